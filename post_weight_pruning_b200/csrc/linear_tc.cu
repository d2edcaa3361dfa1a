// act(x W^T + bias) (* (x W_up^T + bias_up)) + residual on the 5th-generation tensor cores
// (bf16 operands, fp32 accumulation in tensor memory).  Both operands are stored with k
// contiguous, the K-major form the tensor core reads, so tiles go from memory to the MMA
// through TMA with no transpose.  Two kernels:
//
// pair_kernel, for many rows.  Two CTAs of a cluster share one 256 x 256 output tile
// (tcgen05.mma.cta_group::2, M = 256, N = 256): each loads 128 rows of x and 128 rows of W per
// 64 columns of k, half of what two CTAs with a tile each would read, and keeps the 128 x 256
// fp32 accumulator of its own rows.  For the gated product the two CTAs' halves of W are 128
// rows of W and the same 128 rows of W_up: a CTA's accumulator then holds both sums of an
// output element (columns c and 128 + c of one lane) and the product needs no exchange.  Two
// accumulators alternate, so the epilogue of a tile runs beside the next tile's MMAs.
//
// skinny_kernel, for few rows, where the weights' bytes bound the time: the roles are swapped
// (128 rows of W are the M side, up to 256 rows of x the N side, padded to 16), k is split
// over the CTAs of a cluster so that every SM streams weights.  Each CTA then stores its
// partial sums straight from tensor memory into the shared memory of the CTA that finishes
// those rows (stores do not wait for the other side, loads from it would), which adds them
// in rank order -- no atomics, no workspace.  One row of 4096 x 4096 bf16 weights: 11.3 us a call
// on fresh data (5.1 at the copy rate), 8.9 replayed with the weights in L2; 33 rows of two
// 11008 x 4096: 37.9 us a call, 32.2 replayed (27.6).
//
// Accumulators are fp32, but the tensor core truncates when it adds: over 11008 terms 6 in 1000
// outputs are rounded to bf16 the other way than a plain fp32 sum's, and the error against 64 bits
// stays that of the rounding (0.00166 of the size).  Bias, activation, product and residual are applied in fp32 and the
// result is rounded to bf16 once.  Every wait is bounded: a wait that runs out records
// PWP_ETIMEOUT and the rows concerned come out NaN; copies and MMAs in flight are waited for
// before a CTA leaves.
#include "block_ops.cuh"
#include "tc_common.cuh"

namespace pwp {
namespace {

using namespace tc;
typedef __nv_bfloat16 bf16;

constexpr int TK = 64;                            // k per stage: one 128-byte swizzled row
constexpr int ROW_BYTES = TK * 2;

__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A tile load of a CTA pair: into this CTA's shared memory, counted by the barrier at `bar`
// (a cluster address: the leader's).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(idesc), "r"(acc)
      : "memory");
}

// D fp32, A and B bf16 and K-major
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ---------------------------------------------------------------- epilogue pieces

struct Epilogue {
  int vec, pairs;      // rows of out and residual can be read and written 16, 4 bytes at a time
  const bf16* bias;
  const bf16* bias_up;
  const bf16* residual;
  bf16* out;
  long long residual_stride, out_stride;
  int act;
};

__device__ __forceinline__ void unpack8(uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// v[i] += p[i], i < avail (avail > 0); 16-byte loads when all 32 are there and p allows it
__device__ __forceinline__ void add32(float (&v)[32], const bf16* p, int avail) {
  if (avail >= 32 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float t[8];
      unpack8(*reinterpret_cast<const uint4*>(p + 8 * q), t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * q + i] += t[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < avail) v[i] += to_f32(p[i]);
  }
}
// One switch per 32 values, not per value.
__device__ __forceinline__ void activate32(int act, float (&v)[32]) {
  switch (act) {
    case PWP_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate<bf16>(PWP_ACT_RELU, v[i]);
      break;
    case PWP_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate<bf16>(PWP_ACT_SILU, v[i]);
      break;
    case PWP_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate<bf16>(PWP_ACT_GELU, v[i]);
      break;
    case PWP_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate<bf16>(PWP_ACT_GELU_TANH, v[i]);
      break;
    default: break;
  }
}

// ---------------------------------------------------------------- many rows

constexpr int P_ROWS = 128;                       // rows of x, and of W, per CTA
constexpr int P_STAGES = 6;
constexpr int P_STAGE_BYTES = 2 * P_ROWS * ROW_BYTES;   // 32 KB
constexpr int P_EPI_WARPS = 16, P_THREADS = 32 * (2 + P_EPI_WARPS);
constexpr int P_TURN = 32 * 64;                         // a warp's 32 rows of 32 bf16, for its output
constexpr int P_SMEM = P_STAGES * P_STAGE_BYTES + P_EPI_WARPS * P_TURN + 1024 + 256;
constexpr int P_ACC_COLS = 256;
constexpr int P_GROUP = 8;                        // row tiles that share W tiles while they are in L2

// Tile t of the raster: groups of P_GROUP row tiles, inside a group the row tile runs fastest.
__device__ __forceinline__ void pair_tile(int t, int mt, int nt, int& m, int& n) {
  const int per = P_GROUP * nt;
  const int g = t / per, r = t - g * per;
  const int rows = min(P_GROUP, mt - g * P_GROUP);
  n = r / rows;
  m = g * P_GROUP + (r - n * rows);
}

// Two neighbouring columns of a row in a warp's 32 x 32 tile of outputs (see the epilogue).
__device__ __forceinline__ uint8_t* turn_at(uint8_t* turn, int row, int col) {
  return turn + row * 64 + (((col >> 3) ^ ((row >> 1) & 3)) << 4) + (col & 7) * 2;
}

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1)
    pair_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                const __grid_constant__ CUtensorMap umap, long long rows, int n, int nk, Epilogue ep, pwp_stats* st,
                long long spin) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* turn_all = smem + P_STAGES * P_STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(turn_all + P_EPI_WARPS * P_TURN);   // the leader's are used
  uint64_t* empty = full + P_STAGES;
  uint64_t* afull = empty + P_STAGES;
  uint64_t* aempty = afull + 2;                                                    // the leader's are used
  uint64_t* drain = aempty + 2;
  uint64_t* peer = drain + 1;                                                      // the other CTA's copies are all issued
  __shared__ uint32_t tmem_slot, peer_steps;
  __shared__ int abort_flag;
  volatile int* abortp = &abort_flag;

  constexpr int NT = GATED ? 128 : 256;           // output columns of a tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int mt = (int)((rows + 2 * P_ROWS - 1) / (2 * P_ROWS)), nt = (n + NT - 1) / NT;
  const int tiles = mt * nt, pairs = gridDim.x / 2, first = blockIdx.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&afull[a], 1);
      mbar_init(&aempty[a], 2 * P_EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(peer, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_flag = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(2 * P_ACC_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  pdl_enter();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_map(&xmap);
      prefetch_map(&wmap);
      const uint32_t sbase = smem_u32(smem);
      const uint32_t bar0 = map_rank(smem_u32(&full[0]), 0);
      uint32_t s = 0, phase = 0, filled = 0;      // next stage, its phase; stages ever filled (capped)
      uint32_t steps = 0;                         // steps of k loaded
      bool ok = true;
      int t = first, kt = 0, m, c;
      auto load = [&](const CUtensorMap* bmap, int y, int yb) {
        if (rank == 0) mbar_expect_tx(&full[s], 2 * P_STAGE_BYTES);
        const uint32_t dst = sbase + s * P_STAGE_BYTES, bar = bar0 + s * 8u;
        tma_load_pair(dst, &xmap, bar, kt * TK, y);
        tma_load_pair(dst + P_ROWS * ROW_BYTES, bmap, bar, kt * TK, yb);
        ++steps;
        if (++s == P_STAGES) {
          s = 0;
          phase ^= 1u;
        }
      };
      const CUtensorMap* bmap = GATED && rank ? &umap : &wmap;
      while (t < tiles) {
        pair_tile(t, mt, nt, m, c);
        const int y = m * 2 * P_ROWS + (int)rank * P_ROWS;
        const int yb = GATED ? c * NT : c * NT + (int)rank * P_ROWS;
        for (; kt < nk; ++kt) {
          if (filled < P_STAGES) {
            ++filled;
          } else if (!mbar_wait(&empty[s], phase ^ 1u, abortp, spin)) {
            ok = false;
            break;
          }
          load(bmap, y, yb);
        }
        if (!ok) break;
        kt = 0;
        t += pairs;
      }
      if (!ok) *abortp = 1;
      // Both CTAs' copies land before either leaves.  They are counted by the leader's barriers,
      // which complete only when both CTAs have loaded a stage: one that gave up a wait the
      // other did not loads as far as the other (which saw those stages free).
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(smem_u32(&peer_steps), rank ^ 1)), "r"(steps)
                   : "memory");
      remote_arrive(map_rank(smem_u32(peer), rank ^ 1));
      bool met = false;
      for (int i = 0; i < 4 && !met; ++i) met = mbar_wait(peer, 0, kDrainLimit);   // the other's own waits come before
      asm volatile("fence.acq_rel.cluster;" ::: "memory");
      while (met && (int)(*(volatile uint32_t*)&peer_steps - steps) > 0 && t < tiles) {
        pair_tile(t, mt, nt, m, c);
        load(bmap, m * 2 * P_ROWS + (int)rank * P_ROWS, GATED ? c * NT : c * NT + (int)rank * P_ROWS);
        if (++kt == nk) {
          kt = 0;
          t += pairs;
        }
      }
      if (rank == 0) {
        for (uint32_t i = 0; i < filled; ++i) {
          if (s == 0) phase ^= 1u;
          s = s == 0 ? P_STAGES - 1 : s - 1;
          mbar_wait(&full[s], phase, kDrainLimit);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elected()) {
      // descriptors of stage 0; a stage, and a step of 16 along k, on are additions
      const uint64_t da0 = sw128_desc(smem_u32(smem), 16, 1024);
      const uint64_t db0 = sw128_desc(smem_u32(smem) + P_ROWS * ROW_BYTES, 16, 1024);
      constexpr uint32_t idesc = idesc_bf16(256, 256);
      uint32_t s = 0, phase = 0;
      int i = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += pairs, ++i) {
        const int a = i & 1;
        if (i >= 2 && !mbar_wait(&aempty[a], (uint32_t)((i >> 1) - 1) & 1, abortp, spin)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t d = tmem + (uint32_t)(a * P_ACC_COLS);
        for (int kt = 0; kt < nk; ++kt) {
          if (!mbar_wait(&full[s], phase, abortp, spin)) {
            ok = false;
            break;
          }
          fence_after();
          const uint64_t off = s * (P_STAGE_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < TK / 16; ++kk) mma_pair(d, da0 + off + 2 * kk, db0 + off + 2 * kk, idesc, (kt | kk) != 0);
          commit_pair(&empty[s]);
          if (++s == P_STAGES) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (ok) commit_pair(&afull[a]);
      }
      if (!ok) *abortp = 1;
      commit_pair(drain);      // every MMA issued has finished before tensor memory is released
    }
    __syncwarp();
  } else {
    // warp e reads the tensor-memory lanes 32 (e % 4).. and a quarter of the tile's columns
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    int i = 0;
    bool ok = true;
    for (int t = first; t < tiles; t += pairs, ++i) {
      const int a = i & 1;
      if (ok) {
        ok = mbar_wait(&afull[a], (uint32_t)(i >> 1) & 1, abortp, spin);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) {
          *abortp = 1;
          if (st) set_error(st, PWP_ETIMEOUT, kSiteLinear);
        }
      }
      fence_after();
      int m, c;
      pair_tile(t, mt, nt, m, c);
      const long long rw = (long long)m * 2 * P_ROWS + rank * P_ROWS + quarter * 32;      // the warp's first row
      const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(a * P_ACC_COLS);
      uint8_t* turn = turn_all + (warp - 2) * P_TURN;
      // 32 columns at a time.  A thread holds a row, but 32 rows' 16-byte pieces make 32 separate
      // writes; turned through shared memory (16-byte pieces swizzled by row) a warp writes, and
      // reads of the residual, eight rows' whole 64 bytes.  Sixteen warps, because each spends
      // most of its time waiting: at 16384 x 128 x 8192, where the epilogue is the bound, plain
      // 108 us with eight warps of 64 columns and 97 with these, with erf-GELU 300 and 209.
      // Rows that are not 16-byte aligned go two at a time, 4 or 2 bytes a store (8000 x 1000 x 300:
      // 31.5 us with a row per thread, 13.8 this way).
      const int prow = lane >> 2, pcol = lane & 3, brow = lane >> 4, bcol = 2 * (lane & 15);
#pragma unroll 1
      for (int i32 = 0; i32 < NT / 128; ++i32) {
        const int ch = part * (NT / 128) + i32, c0 = c * NT + ch * 32, avail = n - c0;
        if (avail <= 0) break;
        const bool on = 8 * pcol < avail;
        if (ep.vec && ep.residual) {
          uint4 w[4];
          const bf16* p = ep.residual + (rw + prow) * ep.residual_stride + c0 + 8 * pcol;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (on && rw + prow + 8 * q < rows) w[q] = *reinterpret_cast<const uint4*>(p + 8 * q * ep.residual_stride);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int z = prow + 8 * q;
            *reinterpret_cast<uint4*>(turn + z * 64 + ((pcol ^ ((z >> 1) & 3)) << 4)) = w[q];
          }
          __syncwarp();
        } else if (ep.residual) {
          // two rows at a time, a lane two neighbouring columns
          const bf16* p = ep.residual + (rw + brow) * ep.residual_stride + c0 + bcol;
#pragma unroll 8
          for (int q = 0; q < 16; ++q, p += 2 * ep.residual_stride) {
            uint32_t w = 0;
            if (rw + brow + 2 * q < rows && bcol < avail) {
              if (ep.pairs && bcol + 1 < avail) {
                w = *reinterpret_cast<const uint32_t*>(p);
              } else {
                w = *reinterpret_cast<const uint16_t*>(p);
                if (bcol + 1 < avail) w |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 1) << 16;
              }
            }
            *reinterpret_cast<uint32_t*>(turn_at(turn, brow + 2 * q, bcol)) = w;
          }
          __syncwarp();
        }
        float v[32], u[32];
        tmem_ld32_nowait(base + (uint32_t)(ch * 32), v);
        if (GATED) tmem_ld32_nowait(base + (uint32_t)(128 + ch * 32), u);
        tmem_wait_ld();
        pin32(v);
        if (GATED) pin32(u);
        if (ep.bias) add32(v, ep.bias + c0, avail);
        activate32(ep.act, v);
        if (GATED) {
          if (ep.bias_up) add32(u, ep.bias_up + c0, avail);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= u[j];
        }
        if (!ok) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __int_as_float(0x7fc00000);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4* at = reinterpret_cast<uint4*>(turn + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4));
          if (ep.residual) {
            float w[8];
            unpack8(*at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * q + j] += w[j];
          }
          *at = make_uint4(pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                           pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7]));
        }
        __syncwarp();
        if (ep.vec) {
          bf16* p = ep.out + (rw + prow) * ep.out_stride + c0 + 8 * pcol;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int z = prow + 8 * q;
            const uint4 w = *reinterpret_cast<const uint4*>(turn + z * 64 + ((pcol ^ ((z >> 1) & 3)) << 4));
            if (on && rw + z < rows) *reinterpret_cast<uint4*>(p + 8 * q * ep.out_stride) = w;
          }
        } else {
          bf16* p = ep.out + (rw + brow) * ep.out_stride + c0 + bcol;
#pragma unroll 8
          for (int q = 0; q < 16; ++q, p += 2 * ep.out_stride) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(turn_at(turn, brow + 2 * q, bcol));
            if (rw + brow + 2 * q < rows && bcol < avail) {
              if (ep.pairs && bcol + 1 < avail) {
                *reinterpret_cast<uint32_t*>(p) = w;
              } else {
                *reinterpret_cast<uint16_t*>(p) = (uint16_t)w;
                if (bcol + 1 < avail) *reinterpret_cast<uint16_t*>(p + 1) = (uint16_t)(w >> 16);
              }
            }
          }
        }
        __syncwarp();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive(map_rank(smem_u32(&aempty[a]), 0));
    }
  }

  fence_before();
  __syncthreads();
  if (threadIdx.x == 32) mbar_wait(drain, 0, kDrainLimit);   // the MMAs, and their arrivals on this CTA's barriers
  __syncwarp();
  cluster_sync();       // the peer's copies and arrivals on this CTA's barriers are done
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * P_ACC_COLS) : "memory");
}

// ---------------------------------------------------------------- few rows

constexpr int S_FEATURES = 128;                   // rows of W (and W_up) per CTA
constexpr int S_MAX_STAGES = 8, S_THREADS = 256;
constexpr int S_MAX_CLUSTER = 8;

struct Skinny {
  int rows, n, nk;
  int npad;            // rows of x per tile, a multiple of 16 (the tile's tensor-memory columns)
  int row_tiles, split, stages, tmem_cols;
  int f;               // output columns per tile: rows of W, and for the gated product of W_up
};

// Where a feature's four sums of a group of rows lie among the 128 of the tile: the even and the
// odd ones of each half apart, so that a lane which reads slots l and 32 + l of a half has two
// neighbouring features, without bank conflicts.
__device__ __forceinline__ int slot_of(int feature) {
  return (feature & 64) + ((feature & 1) << 5) + ((feature & 63) >> 1);
}

// Adds the ranks' partial sums, part[q][row / 4][slot][row % 4], of `rows` rows and writes them: a
// warp takes four rows of 64 features (for the gated product of the 64 outputs), a lane two
// neighbouring ones.  Branch-free over up to Q ranks (those past the last read its sums again
// and add nothing).  Few warps, so what counts is the instructions of each: pointers step from
// row to row, and whole groups with 4-byte aligned pairs have a path of their own.
template <bool GATED, int ACT, int Q>
__device__ __forceinline__ void finish_rows(const Skinny& g, const Epilogue& ep, const float* part, int per, int row0,
                                            int rows, int c0, int warp, int lane) {
  constexpr int X = GATED ? 4 : 2;
  const int units = (rows + 3) / 4 * (GATED ? 1 : 2);
  for (int unit = warp; unit < units; unit += S_THREADS / 32) {
    const int rg = GATED ? unit : unit >> 1, half = GATED ? 0 : 64 * (unit & 1);
    const int f = half + 2 * lane, c = c0 + f, cols = min(min(g.f - f, 2), g.n - c);
    if (cols <= 0) continue;
    float s[X][4];
    const float* src = part + (rg * S_FEATURES + half + lane) * 4;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(src + 128 * x);
        const bool on = q < g.split;
        s[x][0] = (q ? s[x][0] : 0.f) + (on ? v.x : 0.f);
        s[x][1] = (q ? s[x][1] : 0.f) + (on ? v.y : 0.f);
        s[x][2] = (q ? s[x][2] : 0.f) + (on ? v.z : 0.f);
        s[x][3] = (q ? s[x][3] : 0.f) + (on ? v.w : 0.f);
      }
      if (q + 1 < g.split) src += per * S_FEATURES;
    }
    const bool two = cols == 2;
    if (ep.bias) {
      const float b0 = to_f32(ep.bias[c]), b1 = two ? to_f32(ep.bias[c + 1]) : 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) s[0][t] += b0, s[1][t] += b1;
    }
    if (GATED && ep.bias_up) {
      const float b0 = to_f32(ep.bias_up[c]), b1 = two ? to_f32(ep.bias_up[c + 1]) : 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) s[X - 2][t] += b0, s[X - 1][t] += b1;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s[0][t] = activate<bf16>(ACT, s[0][t]);
      s[1][t] = activate<bf16>(ACT, s[1][t]);
      if (GATED) s[0][t] *= s[X - 2][t], s[1][t] *= s[X - 1][t];
    }
    const long long r = row0 + 4 * rg;
    bf16* o = ep.out + r * ep.out_stride + c;
    const bf16* res = ep.residual ? ep.residual + r * ep.residual_stride + c : nullptr;
    const int left = rows - 4 * rg;
    if (ep.pairs && two && left >= 4) {
      if (res) {
        uint32_t w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint32_t*>(res + t * ep.residual_stride);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          s[0][t] += __uint_as_float(w[t] << 16);
          s[1][t] += __uint_as_float(w[t] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<uint32_t*>(o + t * ep.out_stride) = pack2(s[0][t], s[1][t]);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t >= left) break;
        if (res) {
          s[0][t] += to_f32(res[0]);
          if (two) s[1][t] += to_f32(res[1]);
          res += ep.residual_stride;
        }
        o[0] = from_f32<bf16>(s[0][t]);
        if (two) o[1] = from_f32<bf16>(s[1][t]);
        o += ep.out_stride;
      }
    }
  }
}
template <bool GATED, int ACT>
__device__ __forceinline__ void finish_split(const Skinny& g, const Epilogue& ep, const float* part, int per, int row0,
                                             int rows, int c0, int warp, int lane) {
  if (g.split == 1) finish_rows<GATED, ACT, 1>(g, ep, part, per, row0, rows, c0, warp, lane);
  else if (g.split == 2) finish_rows<GATED, ACT, 2>(g, ep, part, per, row0, rows, c0, warp, lane);
  else if (g.split <= 4) finish_rows<GATED, ACT, 4>(g, ep, part, per, row0, rows, c0, warp, lane);
  else finish_rows<GATED, ACT, S_MAX_CLUSTER>(g, ep, part, per, row0, rows, c0, warp, lane);
}

template <bool GATED>
__global__ void __launch_bounds__(S_THREADS, 2)
    skinny_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                  const __grid_constant__ CUtensorMap umap, const Skinny g, const Epilogue ep, pwp_stats* st,
                  long long spin) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[S_MAX_STAGES], empty[S_MAX_STAGES], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  volatile int* abortp = &abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % g.split), tile = (int)(blockIdx.x / g.split);
  const int c0 = (tile / g.row_tiles) * g.f, r0 = (tile % g.row_tiles) * g.npad;
  const int kt0 = (int)((long long)g.nk * rank / g.split), kt1 = (int)((long long)g.nk * (rank + 1) / g.split);
  const int stage_bytes = (S_FEATURES + g.npad) * ROW_BYTES;

  // The copies start before tensor memory is there: thread 0 sets up the barriers that they
  // need and fills the ring.
  // The tiles of a column of CTAs all read the same rows of x; each starts at another place of
  // its range of k, or they would queue for the same lines of L2 at every step.
  const int range = kt1 - kt0, turn = (int)((unsigned)tile * 37u % (unsigned)range);
  int issued = 0;
  auto load = [&](int i, int s) {
    const int kt = kt0 + (i + turn < range ? i + turn : i + turn - range);
    mbar_expect_tx(&full[s], (uint32_t)(((GATED ? 2 : 1) * g.f + g.npad) * ROW_BYTES));
    uint8_t* a = smem + s * stage_bytes;
    tma_load_2d(a, &wmap, &full[s], kt * TK, c0);
    if (GATED) tma_load_2d(a + 64 * ROW_BYTES, &umap, &full[s], kt * TK, c0);
    tma_load_2d(a + S_FEATURES * ROW_BYTES, &xmap, &full[s], kt * TK, r0);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_flag = 0;
    pdl_wait();
    for (; issued < g.stages && issued < range; ++issued) load(issued, issued);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, (uint32_t)g.tmem_cols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_enter();

  if (warp == 0) {
    if (lane == 0) {
      for (; issued < range; ++issued) {
        const int s = issued % g.stages;
        if (!mbar_wait(&empty[s], (uint32_t)(issued / g.stages - 1) & 1, abortp, spin)) {
          *abortp = 1;
          break;
        }
        load(issued, s);
      }
      for (int i = issued > g.stages ? issued - g.stages : 0; i < issued; ++i)
        mbar_wait(&full[i % g.stages], (uint32_t)(i / g.stages) & 1, kDrainLimit);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t sbase = smem_u32(smem), idesc = idesc_bf16(S_FEATURES, g.npad);
      bool ok = true;
      for (int kt = kt0, i = 0; kt < kt1; ++kt, ++i) {
        const int s = i % g.stages;
        if (!mbar_wait(&full[s], (uint32_t)(i / g.stages) & 1, abortp, spin)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t pa = sbase + s * stage_bytes, pb = pa + S_FEATURES * ROW_BYTES;
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk)
          mma_one(tmem, sw128_desc(pa + kk * 32, 16, 1024), sw128_desc(pb + kk * 32, 16, 1024), idesc, (i | kk) != 0);
        mma_commit(&empty[s]);
      }
      if (!ok) *abortp = 1;
      mma_commit(&done);
      mbar_wait(&done, 0, kDrainLimit);
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();      // every copy has landed, every MMA has finished: the stages are free
  if (g.split > 1) cluster_sync();      // in every CTA of the cluster
  fence_after();

  // Row t of the tile is finished by CTA t / per, which gets the partial sums of rank q at
  // part[q][t % per / 4][slot][t % 4]: four rows of a feature are one 16-byte store, a warp's 32
  // stores two runs of 256 bytes.
  const bool failed_tile = *abortp != 0;
  float* part = reinterpret_cast<float*>(smem);
  const int have = min(g.npad, g.rows - r0);
  const int per = ((have + g.split - 1) / g.split + 3) & ~3;
  const int quarter = warp & 3;
  const uint32_t pbase = smem_u32(part) + (uint32_t)(rank * per * S_FEATURES + slot_of(quarter * 32 + lane) * 4) * 4u;
  for (int j = (warp >> 2) * 16; j < have; j += 32) {
    float v[16];
    tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)j, v);
    if (failed_tile) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __int_as_float(0x7fc00000);
    }
    int to = j / per, at = j - to * per;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      if (j + i < have)
        remote_store4(map_rank(pbase + (uint32_t)(at * S_FEATURES) * 4u, (uint32_t)to),
                      make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
      at += 4;
      if (at == per) {
        at = 0;
        ++to;
      }
    }
  }
  if (failed_tile && threadIdx.x == 0 && st) set_error(st, PWP_ETIMEOUT, kSiteLinear);
  fence_before();
  __syncthreads();
  if (warp == 1) tmem_free(tmem, (uint32_t)g.tmem_cols);
  if (g.split > 1) cluster_sync();      // the others' sums are here

  // one loop per activation: a branch per value costs more than everything else here
  const int t0 = rank * per, mine = min(per, have - t0);
  const float* from = part;
  switch (ep.act) {
    case PWP_ACT_RELU: finish_split<GATED, PWP_ACT_RELU>(g, ep, from, per, r0 + t0, mine, c0, warp, lane); break;
    case PWP_ACT_SILU: finish_split<GATED, PWP_ACT_SILU>(g, ep, from, per, r0 + t0, mine, c0, warp, lane); break;
    case PWP_ACT_GELU: finish_split<GATED, PWP_ACT_GELU>(g, ep, from, per, r0 + t0, mine, c0, warp, lane); break;
    case PWP_ACT_GELU_TANH: finish_split<GATED, PWP_ACT_GELU_TANH>(g, ep, from, per, r0 + t0, mine, c0, warp, lane); break;
    default: finish_split<GATED, PWP_ACT_NONE>(g, ep, from, per, r0 + t0, mine, c0, warp, lane); break;
  }
}

// ---------------------------------------------------------------- host side

// [height][k] bf16, row stride in elements, tiles of box_rows x 64; false when the copies
// cannot take it
bool make_map(CUtensorMap* map, const void* p, long long height, int k, long long stride, int box_rows) {
  if (height <= 1) stride = (k + 7) & ~7;       // a single row: its stride is never used
  if (((uintptr_t)p & 15) || (stride & 7) || stride < k || stride >= (1LL << 38) || height >= (1LL << 32)) return false;
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)height};
  cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  cuuint32_t box[2] = {(cuuint32_t)TK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool GATED>
cudaError_t run_pair(const pwp_linear_args& a, const Epilogue& ep, cudaStream_t s, bool* used) {
  CUtensorMap xm, wm, um;
  if (!make_map(&xm, a.x_dev, a.rows, a.k, a.x_stride, P_ROWS) || !make_map(&wm, a.w_dev, a.n, a.k, a.w_stride, P_ROWS))
    return cudaSuccess;
  um = wm;
  if (GATED && !make_map(&um, a.w_up_dev, a.n, a.k, a.w_up_stride, P_ROWS)) return cudaSuccess;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t ready = on_first_use(attr_done, [] {
    return cudaFuncSetAttribute(pair_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, P_SMEM);
  });
  if (ready != cudaSuccess) return ready;
  constexpr int NT = GATED ? 128 : 256;
  const long long tiles = ((a.rows + 2 * P_ROWS - 1) / (2 * P_ROWS)) * ((a.n + NT - 1) / NT);
  if (tiles > 0x3fffffffLL) return cudaSuccess;
  const int pairs = tiles < kNumSM / 2 ? (int)tiles : kNumSM / 2;
  *used = true;
  const cudaError_t e = launch_pdl(pair_kernel<GATED>, dim3(2 * pairs), dim3(P_THREADS), (size_t)P_SMEM, s, xm, wm, um,
                                   (long long)a.rows, a.n, (a.k + TK - 1) / TK, ep, a.stats_dev, wait_limit());
  count_launches(1);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// How many CTAs of the skinny kernel run at once in clusters of c, one to an SM: all SMs less
// what clusters leave over in a group of SMs.  (The query counts one CTA of a kernel that
// holds tensor memory per SM; two run beside each other when their shared memory fits.)
template <bool GATED>
void resident_ctas(int (&ctas)[S_MAX_CLUSTER + 1]) {
  static std::atomic<int> known[64][S_MAX_CLUSTER + 1];
  int dev = 0;
  const bool ok = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
  for (int c = 2; c <= S_MAX_CLUSTER; ++c) {
    ctas[c] = ok ? known[dev][c].load(std::memory_order_relaxed) : 0;
    if (!ok || ctas[c]) continue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(c * kNumSM));
    cfg.blockDim = dim3(S_THREADS);
    cfg.dynamicSmemBytes = 225 * 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, skinny_kernel<GATED>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      continue;
    }
    ctas[c] = clusters * c;
    known[dev][c].store(ctas[c], std::memory_order_relaxed);
  }
}

template <bool GATED>
cudaError_t run_skinny(const pwp_linear_args& a, const Epilogue& ep, cudaStream_t s, bool* used) {
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t ready = on_first_use(attr_done, [] {
    return cudaFuncSetAttribute(skinny_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
  });
  if (ready != cudaSuccess) return ready;
  constexpr int F = GATED ? S_FEATURES / 2 : S_FEATURES;
  Skinny g;
  g.rows = (int)a.rows;
  g.n = a.n;
  g.nk = (a.k + TK - 1) / TK;
  // All CTAs of a split are resident at once: a second round of clusters costs as much as the
  // first (601 x 4096 x 1000: 17 us split 5 ways, 29 us split 6).
  int resident[S_MAX_CLUSTER + 1];
  resident_ctas<GATED>(resident);
  const int col_tiles = (a.n + F - 1) / F;
  int split = 1, per_sm = 1;
  if (g.rows <= 64) {
    // Bound by the weights' bytes: the largest split.  Up to 64 rows two CTAs fit an SM.
    g.npad = (g.rows + 15) & ~15;
    per_sm = 2;
    for (int c = 2; c <= S_MAX_CLUSTER && c <= g.nk; ++c)
      if ((long long)col_tiles * c <= 2LL * resident[c]) split = c;
  } else {
    // Rows per tile and split of k by a model of the time fitted to stamps of the kernel's phases
    // (us): copies come at 75 KB an SM; a split costs two barriers of the cluster, and its sums
    // go through distributed shared memory at 24 KB an SM; finishing 64 rows takes 1.5.
    float best = 1e30f;
    for (int most = 256; most >= 64; most -= most > 128 ? 64 : 32) {
      const int rt = (g.rows + most - 1) / most, npad = ((g.rows + rt - 1) / rt + 15) & ~15, here = npad <= 64 ? 2 : 1;
      const long long t = (long long)col_tiles * ((g.rows + npad - 1) / npad);
      for (int c = 1; c <= S_MAX_CLUSTER && c <= g.nk; ++c) {
        if (c > 1 && t * c > (long long)resident[c] * here) continue;
        const float on_sm = (float)((t * c + kNumSM - 1) / kNumSM);      // CTAs an SM runs, together or in turn
        float us = on_sm * ((g.nk + c - 1) / c) * (S_FEATURES + npad) * (ROW_BYTES / 75e3f);
        us += on_sm * ((npad + c - 1) / c) * (1.5f / 64);
        if (c > 1) us += 1.8f + on_sm * npad * (c - 1) / c * (S_FEATURES * 4 / 24e3f);
        if (us < best) {
          best = us;
          split = c;
          per_sm = here;
          g.npad = npad;
        }
      }
    }
  }
  g.row_tiles = (g.rows + g.npad - 1) / g.npad;
  g.tmem_cols = 32;
  while (g.tmem_cols < g.npad) g.tmem_cols *= 2;
  const int stage_bytes = (S_FEATURES + g.npad) * ROW_BYTES;
  const int room = (per_sm == 2 ? 112 : 224) * 1024 - 1024;
  g.stages = room / stage_bytes < S_MAX_STAGES ? room / stage_bytes : S_MAX_STAGES;
  long long tiles = (long long)col_tiles * g.row_tiles;
  g.f = F;
  if (split == 1 && g.rows <= 64) {
    // As many rounds of CTAs as that takes anyway, with equal shares of the columns.  (With more
    // rows every share reads too much of x again: 1024^3 in 288 CTAs 11.6 us, in 128 10.4.)
    const long long slots = kNumSM * per_sm, rounds = (tiles + slots - 1) / slots;
    g.f = (int)((a.n + slots * rounds - 1) / (slots * rounds));
    g.f = (g.f + 3) & ~3;
    if (g.f > F) g.f = F;
    tiles = (a.n + g.f - 1) / g.f;
  }
  g.split = split;
  if (tiles > 0x7fffffffLL / split) return cudaSuccess;
  int smem = g.stages * stage_bytes;
  const int parts = (g.npad + 4 * g.split) * S_FEATURES * (int)sizeof(float);
  if (smem < parts) smem = parts;
  smem += 1024;
  CUtensorMap xm, wm, um;
  if (!make_map(&xm, a.x_dev, a.rows, a.k, a.x_stride, g.npad) || !make_map(&wm, a.w_dev, a.n, a.k, a.w_stride, g.f))
    return cudaSuccess;
  um = wm;
  if (GATED && !make_map(&um, a.w_up_dev, a.n, a.k, a.w_up_stride, g.f)) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(S_THREADS);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  *used = true;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, skinny_kernel<GATED>, xm, wm, um, g, ep, a.stats_dev, wait_limit());
  count_launches(1);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

// ---------------------------------------------------------------- operands that are not 16-byte aligned

namespace {

// Rows of k values from a stride of their own to one of `kp` (a multiple of 8), for up to three
// operands in one launch (blockIdx.y); one 16-byte piece per thread and step.  What lies between
// k and kp is never read as data.
struct AlignRows {
  const bf16* src[3];
  bf16* dst[3];
  long long stride[3], rows[3];
};
__global__ void __launch_bounds__(256) align_rows_kernel(const AlignRows a, int k, int kp) {
  pdl_enter();
  const int which = blockIdx.y, pieces = kp / 8;
  const long long total = a.rows[which] * pieces;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += 256LL * gridDim.x) {
    const long long r = i / pieces;
    const int c = (int)(i - r * pieces) * 8;
    const bf16* p = a.src[which] + r * a.stride[which] + c;
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < k ? *reinterpret_cast<const uint16_t*>(p + j) : (uint16_t)0;
    *reinterpret_cast<uint4*>(a.dst[which] + r * kp + c) =
        make_uint4(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16, v[4] | (uint32_t)v[5] << 16,
                   v[6] | (uint32_t)v[7] << 16);
  }
}

bool misaligned(const void* p, long long stride, long long rows) {
  return p && (((uintptr_t)p & 15) != 0 || (rows > 1 && (stride & 7) != 0));
}
size_t copy_bytes(long long rows, int k) { return ((size_t)rows * ((k + 7) & ~7) * 2 + 255) & ~(size_t)255; }

}  // namespace

// Copying costs one more launch and one more read and write of an operand.  A small product over
// a short k is done as soon on the CUDA cores (4 x 33 x 50: 6.7 us, 7.2 with copies); they take
// longer with k (30 x 101 x 100: 13.5, 7.2; 30 x 1001 x 500: 18.5, 7.3).
size_t linear_align_bytes(const pwp_linear_args& a) {
  if (a.type != PWP_BF16 || (a.k < 64 && (double)a.rows * a.k * a.n < (double)(1 << 24))) return 0;
  size_t n = 0;
  if (misaligned(a.x_dev, a.x_stride, a.rows)) n += copy_bytes(a.rows, a.k);
  if (misaligned(a.w_dev, a.w_stride, a.n)) n += copy_bytes(a.n, a.k);
  if (misaligned(a.w_up_dev, a.w_up_stride, a.n)) n += copy_bytes(a.n, a.k);
  return n;
}

// Copies the misaligned operands into a.ws_dev and points `a` at the copies.
cudaError_t launch_linear_align(pwp_linear_args& a, cudaStream_t s) {
  char* ws = (char*)a.ws_dev;
  const int kp = (a.k + 7) & ~7;
  AlignRows r = {};
  int count = 0;
  long long most = 0;
  auto copy = [&](const void*& p, int64_t& stride, long long rows) {
    if (!misaligned(p, stride, rows)) return;
    r.src[count] = (const bf16*)p;
    r.dst[count] = (bf16*)ws;
    r.stride[count] = stride;
    r.rows[count++] = rows;
    if (rows > most) most = rows;
    p = ws;
    stride = kp;
    ws += copy_bytes(rows, a.k);
  };
  copy(a.x_dev, a.x_stride, a.rows);
  copy(a.w_dev, a.w_stride, a.n);
  copy(a.w_up_dev, a.w_up_stride, a.n);
  const long long blocks = (most * (kp / 8) + 255) / 256;
  const cudaError_t e = launch_pdl(align_rows_kernel, dim3((unsigned)(blocks < 16 * kNumSM ? blocks : 16 * kNumSM), (unsigned)count),
                                   dim3(256), (size_t)0, s, r, a.k, kp);
  count_launches(1);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// Declines (used = false) when the tensors do not meet the copies' rules (16-byte aligned
// bases, row strides a multiple of 16 bytes).
cudaError_t launch_linear_tc(const pwp_linear_args& a, cudaStream_t s, bool* used) {
  *used = false;
  if (a.type != PWP_BF16) return cudaSuccess;
  const long long os = a.rows > 1 ? a.out_stride : 8, rs = a.rows > 1 ? a.residual_stride : 8;
  const bool vec = (a.n & 7) == 0 && (os & 7) == 0 && ((uintptr_t)a.out_dev & 15) == 0 &&
                   (!a.residual_dev || ((rs & 7) == 0 && ((uintptr_t)a.residual_dev & 15) == 0));
  const bool pairs = (os & 1) == 0 && ((uintptr_t)a.out_dev & 3) == 0 &&
                     (!a.residual_dev || ((rs & 1) == 0 && ((uintptr_t)a.residual_dev & 3) == 0));
  const Epilogue ep{vec ? 1 : 0, pairs ? 1 : 0, (const bf16*)a.bias_dev, (const bf16*)a.bias_up_dev, (const bf16*)a.residual_dev, (bf16*)a.out_dev,
                    a.residual_stride, a.out_stride, a.activation};
  const bool gated = a.w_up_dev != nullptr;
  // Too few tiles of CTA pairs for the SMs: split k instead.  Alone on their SMs the pairs take
  // about 5.9 + 0.29 us per 64 of k, the other kernel 6.5 + 0.0095 per 64 of k and tile (200 x 4096
  // x 4096, 16 tiles: 24.3 us in pairs, 16.4; 700 x 2000 x 2000, 24 tiles: 15.3, 13.7; 2048 x 1024 x
  // 1024, 32 tiles: 10.6, 12.3; gated 600 x 4096 x 2000, 48 tiles: 26.5, 32.9).
  const long long tiles = ((a.rows + 255) / 256) * ((a.n + (gated ? 127 : 255)) / (gated ? 128 : 256));
  const int nk = (a.k + TK - 1) / TK;
  const bool skinny = a.rows <= 128 || (tiles < 40 && (40 - tiles) * nk > 256);
  if (skinny) return gated ? run_skinny<true>(a, ep, s, used) : run_skinny<false>(a, ep, s, used);
  return gated ? run_pair<true>(a, ep, s, used) : run_pair<false>(a, ep, s, used);
}

}  // namespace pwp
