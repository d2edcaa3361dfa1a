// Attention within packed sequences on the 5th-generation tensor cores (bf16 operands, fp32
// scores, statistics and sums).
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(c (s_ij - m_i)),  s = q k^T,  c = scale log2(e)
//
// in one pass over the keys, 128 at a time (the online softmax of Milakov and Gimelshein, with its
// rescaling put off), with a reference m_i that is the running maximum
// or lags behind it by at most 8 in the exponent: o and the sum are rescaled only when the
// maximum has grown by more (p then stays below 2^8, far from any overflow, and bf16 keeps
// its relative precision).
//
// A persistent CTA takes pairs of tiles of 128 query rows.  A tile's rows are tokens times the
// query heads that share a key head (row = token * group + head), so grouped heads read their
// keys once and short sequences fill tiles; one TMA box gathers them.  Roles:
//   warp 0         finds the items (tile pairs), hands them to the others through a short queue,
//                  and copies: q of both tiles, then K_0, V_0, K_1, V_1, ... through a ring
//   warp 1         MMA: S_w = Q_w K_j^T and O_w += P_w V_j for the two tiles w in turn, so the
//                  tensor core works on one tile while the other's softmax runs.  P_w
//                  (bf16) overlays S_w in tensor memory and is the A operand from there.
//   warps 2, 3     keep what no query may see out of V: rows behind the sequence's end are
//                  zeroed in shared memory (0 * NaN is NaN), and in the blocks the causal mask
//                  cuts, non-finite values are zeroed and added back at the end to the rows
//                  that do see them
//   warps 4-7, 8-11  softmax of tile 0 and 1, one row per thread, and the rows' output
// S_w(j) becoming full implies that O_w holds block j-1's product (the MMAs of a thread complete
// in order), so a softmax thread may rescale its row of O_w without another barrier.
//
// P is rounded to bf16 (2^-8 of each at most) because the tensor core takes both operands in one
// type, V's: the output's error against 64 bits grows from 0.0016 to 0.0021 of its size (the
// output's own rounding is 0.0016).  Scores, statistics, sums and O are fp32; the sum adds the
// probabilities before that rounding.  The products accumulate in the tensor core, which truncates.
//
// What bounds it (16 x 2048 tokens, 32 heads of 128: causal 632 us twenty in a row, 736 a thousand in a
// row under the power cap, 870 and 750 TFLOP/s; full 1.07 and 1.15 ms, 1025 and 955): a tile's chain of
// softmax (about 1700 cycles per 128 keys: 900 of exponentials at 16 a cycle and SM, seven eighths of
// them, the rest issue and latency), its two MMA groups of 512 and the hand-overs between them, which
// the other tile fills only in part: the tensor pipe is busy 38 % of the time causal and
// 52 % full (profiled at 4 x 2048, caches cold).  The single-thread roles are bound by
// instruction issue and fetch, so they hold little code: running slots and descriptors and no item
// search were worth 0.09 ms of 0.70.
// Tried and slower (full attention, when it took 0.95 ms): P handed over in halves (1.24 ms, and 1.15 with an MMA warp
// per tile); blocks of 64 keys with two S per tile (1.42); 32 keys at a time (1.31); two threads
// to a row, 16 softmax warps of 104 registers (1.09); the sum in
// place of the maximum as the reference's guard (0.99); none (0.97) or three of eight pairs of
// exponentials (1.19) on the FMA pipe.
//
// Every wait is bounded: one that runs out records PWP_ETIMEOUT and the rows come out NaN;
// copies and MMAs in flight are waited for before a CTA leaves.
#include <climits>

#include "block_ops.cuh"
#include "tc_common.cuh"

namespace pwp {
namespace {

using namespace tc;
typedef __nv_bfloat16 bf16;

constexpr int BOX = 128 * 128;                 // 128 rows of 64 bf16
constexpr int KEYS = 128;
constexpr int kThreadsAtt = 384;
constexpr int kPolyPairs = 1;                      // of 8 pairs of exponentials, on the FMA pipe
constexpr int kQueue = 4;                      // items handed out ahead

template <int D>
struct Cfg {
  static constexpr int BOXES = D / 64;
  static constexpr int TILE = BOXES * BOX;               // a tile of q, k or v
  static constexpr int SLOTS = D == 128 ? 5 : 8;
  static constexpr int SMEM = (2 + SLOTS) * TILE + 1024;
};

struct Att {
  const int* cu;
  pwp_stats* st;
  bf16* out;
  const bf16* v;
  long long n, os0, os1, vs0, vs1;
  int nseq, hk, group, tq, d, causal;          // tq: tokens per tile
  float c;                                     // scale * log2(e)
  int vec;                                     // 16-byte stores of out are possible
  int* next;                                   // items taken beyond the first of each CTA, or NULL
};

// The items: the sequences' tile pairs (the last, longest one of a sequence first) with the key
// heads running fastest.  A CTA starts with the item of its number and takes the next free one
// when the copies of its last one are out (a counter in the caller's workspace), or without one
// every gridDim-th: the heaviest CTA then has 1.05 times the mean work at 16 sequences of 2048
// tokens, 1.14 at 4, 1.5 at one, against 1.01 to 1.05 with the counter.  Warp 0 finds them and hands them to the other
// roles through a short queue in shared memory.
struct Items {
  int t, s0, base;        // last item (-1: none yet); the first sequence of the scan's chunk; tiles before it
};
struct __align__(16) Item {
  int begin, len, hk;     // sequence (len < 0: no more items), key head
  int tok;                // first token of tile 0; tile 1 starts tq tokens on
  int nb[2];              // key blocks of each tile (0: no rows)
  int fix;                // first block of V that the fixers look at
  int steps;              // key blocks of the item
};

// The next item of this CTA (whole warp); false past the last one.
__device__ __forceinline__ bool next_item(const Att& a, Items& it, Item& x, bool& bad) {
  const int lane = threadIdx.x & 31;
  const int per = 2 * a.tq;
  if (it.t < 0) {
    it.t = blockIdx.x;
  } else if (a.next) {
    int taken = 0;
    if (lane == 0) taken = atomicAdd(a.next, 1);
    it.t = gridDim.x + __shfl_sync(0xffffffffu, taken, 0);
  } else {
    it.t += gridDim.x;
  }
  const int tile = it.t / a.hk;
  x.hk = it.t - tile * a.hk;
  for (; it.s0 < a.nseq; it.s0 += 32) {
    const int s = it.s0 + lane;
    int b = 0, e = 0;
    if (s < a.nseq) {
      b = a.cu[s];
      e = a.cu[s + 1];
    }
    const bool ok = b >= 0 && e >= b && (long long)e <= a.n;
    const unsigned broken = ~__ballot_sync(0xffffffffu, ok);
    if (broken) bad = true;
    const int len = (broken & (0xffffffffu >> (31 - lane))) ? 0 : e - b;
    const int tiles = (int)(((long long)len + per - 1) / per);
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, tile < it.base + sum);
    if (hit) {
      const int l = __ffs(hit) - 1;
      x.begin = __shfl_sync(0xffffffffu, b, l);
      x.len = __shfl_sync(0xffffffffu, len, l);
      const int after = __shfl_sync(0xffffffffu, sum, l);      // tiles up to and with this sequence's
      x.tok = (it.base + after - 1 - tile) * per;              // its tiles from the last one
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int first = x.tok + w * a.tq;
        x.nb[w] = first >= x.len ? 0 : ((a.causal ? min(x.len, first + a.tq) : x.len) + KEYS - 1) / KEYS;
      }
      x.fix = a.causal ? (x.tok + 1) / KEYS : x.len / KEYS;
      x.steps = max(x.nb[0], x.nb[1]);
      return true;
    }
    if (broken) {
      it.s0 = a.nseq;
      return false;
    }
    it.base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// MMAs of one tile product, issued by one thread: descriptors are a base plus constants.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t ta, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(ta), "l"(db), "r"(idesc), "r"(acc)
      : "memory");
}
// S (128 x 128) = Q (128 x 64 BOXES) K^T: steps of 16 are 32 bytes inside a swizzled row, a box of
// 64 further on after four.
template <int BOXES>
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t dq, uint64_t dk, uint32_t idesc) {
#pragma unroll
  for (int i = 0; i < 4 * BOXES; ++i) {
    const uint32_t off = (i / 4) * (BOX >> 4) + (i % 4) * 2;
    mma_ss(d, dq + off, dk + off, idesc, i != 0);
  }
}
// O += P V over 128 keys: P in tensor memory (16 keys are 8 columns), V MN-major (16 keys are
// 2048 bytes).
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t p, uint64_t dv, uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int i = 0; i < KEYS / 16; ++i) mma_ts(d, p + 8 * i, dv + i * 128, idesc, i != 0 ? 1u : acc);
}
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r != 0;
}
// Position in a ring of N slots: the slot, and the phase of its barriers.
template <uint32_t N>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};
// A wait the whole warp takes part in; every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort, long long limit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x of two values on the FMA pipe, after Cody and Waite: x = n + f with n the nearest whole number, f in [-1/2, 1/2],
// and 2^f by the cubic 1 + f (a + f (b + f c)) of least largest relative error (found by linear
// programming over 4001 points: 1.02e-4 = 2^-13.3, a fortieth of a bf16 half step).  The
// constant term is exactly 1, so x clamped at -127 gives exactly 0 (1's exponent field of 127,
// less 127).
__device__ __forceinline__ float2 exp2_poly(float2 x) {
  const f32x2 big = pair(12582912.f, 12582912.f);      // 1.5 * 2^23: the sum's low bits are n
  const f32x2 v = pair(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f));
  const f32x2 t = add2(v, big);
  const f32x2 n = add2(t, pair(-12582912.f, -12582912.f));
  const f32x2 f = fma2(n, pair(-1.f, -1.f), v);
  f32x2 p = fma2(f, pair(0.05500893294811249f, 0.05500893294811249f), pair(0.2422109693288803f, 0.2422109693288803f));
  p = fma2(p, f, pair(0.6932829022407532f, 0.6932829022407532f));
  p = fma2(p, f, pair(1.f, 1.f));
  const float2 pf = unpair(p), tf = unpair(t);
  return make_float2(__int_as_float(__float_as_int(pf.x) + (__float_as_int(tf.x) << 23)),
                     __int_as_float(__float_as_int(pf.y) + (__float_as_int(tf.y) << 23)));
}
// maximum of three, NaN if any is
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_of(const float* s) {
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i + 8 <= KEYS; i += 8) {
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = max3(m[q], s[i + 2 * q], s[i + 2 * q + 1]);
  }
  return max3(max3(m[0], m[1], m[2]), max3(m[3], s[KEYS - 4], s[KEYS - 3]), max3(s[KEYS - 2], s[KEYS - 1], s[KEYS - 1]));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// D fp32, A bf16 K-major, B bf16 (K-major, or MN-major: `bt`)
__device__ __forceinline__ constexpr uint32_t idesc_of(int n, int bt) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)bt << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

struct Bars {
  uint64_t full[8], empty[8], fixed[8];        // ring slots
  uint64_t qfull[2], qempty[2], sfull[2], pfull[2], ofull[2], oempty[2];
  uint64_t drain;
  uint64_t ifull[kQueue], iempty[kQueue];
  Item item[kQueue];
  int vbad[kQueue];                            // item + 1: a non-finite value was taken out of its V
  // for when a wait runs out: the last items taken, each softmax warp's first one that it did not
  // finish, and where warp 0 was
  Item taken[2 * kQueue];
  int ntaken, done[8];
  Items it;
  int abort_flag;
  uint32_t tmem;
};

template <int D>
__global__ void __launch_bounds__(kThreadsAtt, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const Att a, long long spin) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = smem + 2 * C::TILE;
  __shared__ Bars sb;
  volatile int* abortp = &sb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&sb.full[s], 1);
      mbar_init(&sb.empty[s], 3);      // the MMAs and both fixers
      mbar_init(&sb.fixed[s], 2);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sb.qfull[w], 1);
      mbar_init(&sb.qempty[w], 1);
      mbar_init(&sb.sfull[w], 1);
      mbar_init(&sb.pfull[w], 4);
      mbar_init(&sb.ofull[w], 1);
      mbar_init(&sb.oempty[w], 4);
    }
    mbar_init(&sb.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sb.abort_flag = 0;
    sb.ntaken = 0;
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&sb.ifull[i], 1);
      mbar_init(&sb.iempty[i], 11);     // the MMA warp, the fixers and the softmax warps
      sb.vbad[i] = 0;
    }
  }
  if (warp == 1) tmem_alloc(&sb.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  pdl_enter();
  const uint32_t tmem = sb.tmem;
  const uint32_t tS = tmem, tO = tmem + 256;      // S_w at 128 w, O_w at 256 + 128 w

  // Registers: the softmax warps hold a row of 128 scores.  The CTA was launched with 384 * 168;
  // 128 * 88 + 256 * 208 is exactly that.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
    // ---------------------------------------------------------------- items and copies
    Items it{-1, 0, 0};
    Ring<C::SLOTS> rg;
    Ring<kQueue> iq;
    uint32_t filled = 0, items = 0, qn[2] = {0, 0};       // slots ever filled (capped), items, q tiles so far
    bool ok = true, more = true, bad = false;
    const uint32_t qbytes = (uint32_t)(C::BOXES * a.tq * a.group * 128);
    while (ok && more) {
      Item x;
      more = next_item(a, it, x, bad);
      if (elected()) {
        if (!more) {
          x.len = -1;
        } else {
          sb.taken[items % (2 * kQueue)] = x;
          sb.ntaken = items + 1;
        }
        if (items >= kQueue) ok = mbar_wait(&sb.iempty[iq.slot], iq.phase ^ 1u, abortp, spin);
        if (ok) {
          sb.item[iq.slot] = x;
          mbar_arrive(&sb.ifull[iq.slot]);
        }
        for (int w = 0; w < 2 && ok && more; ++w) {
          if (!x.nb[w]) continue;
          if (qn[w]) ok = mbar_wait(&sb.qempty[w], (qn[w] - 1) & 1, abortp, spin);
          if (!ok) break;
          mbar_expect_tx(&sb.qfull[w], qbytes);
          for (int b = 0; b < C::BOXES; ++b)
            tma_load_4d(smem + w * C::TILE + b * BOX, &qmap, &sb.qfull[w], 64 * b, 0, x.hk, x.begin + x.tok + w * a.tq);
          ++qn[w];
        }
        for (int j2 = 0; ok && more && j2 < 2 * x.steps; ++j2) {
          if (filled < C::SLOTS)
            ++filled;
          else
            ok = mbar_wait(&sb.empty[rg.slot], rg.phase ^ 1u, abortp, spin);
          if (!ok) break;
          mbar_expect_tx(&sb.full[rg.slot], C::TILE);
          for (int b = 0; b < C::BOXES; ++b)
            tma_load_3d(ring + rg.slot * C::TILE + b * BOX, (j2 & 1) ? &vmap : &kmap, &sb.full[rg.slot], 64 * b, x.hk,
                        x.begin + (j2 >> 1) * KEYS);
          rg.step();
        }
        if (!ok) *abortp = 1;
      }
      ++items;
      iq.step();
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elected()) {
      if (bad && a.st) set_error(a.st, PWP_EINVAL, kSiteAttention);
      for (uint32_t i = 0; i < filled; ++i) {
        if (rg.slot == 0) rg.phase ^= 1u;
        rg.slot = rg.slot == 0 ? C::SLOTS - 1 : rg.slot - 1;
        mbar_wait(&sb.full[rg.slot], rg.phase, kDrainLimit);
      }
      for (int w = 0; w < 2; ++w)
        if (qn[w]) mbar_wait(&sb.qfull[w], (qn[w] - 1) & 1, kDrainLimit);
      sb.it = it;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    // descriptors of slot 0 and tile 0; slots and tiles further on are additions
    const uint64_t dq0 = sw128_desc(smem_u32(smem), 16, 1024), dk0 = sw128_desc(smem_u32(ring), 16, 1024);
    const uint64_t dv0 = sw128_desc(smem_u32(ring), BOX, 1024);
    constexpr uint32_t id_qk = idesc_of(KEYS, 0), id_pv = idesc_of(D, 1);
    constexpr uint32_t STEP = C::TILE >> 4;
    uint32_t slot = 0, phase = 0, fixpar = 0;       // the ring's next slot, the phase of its barriers
    uint32_t nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};   // q tiles, blocks and outputs so far
    bool ok = true;
    auto advance = [&]() {
      if (++slot == C::SLOTS) {
        slot = 0;
        phase ^= 1u;
      }
    };
    if (elected()) {
      Ring<kQueue> iq;
      while (ok) {
        ok = mbar_wait(&sb.ifull[iq.slot], iq.phase, abortp, spin);
        if (!ok) break;
        const Item x = sb.item[iq.slot];
        if (x.len < 0) break;
        // S_w(0), then for every block O_w += P_w V_j and S_w(j + 1), the tiles in turn.  K_j and
        // V_j follow each other in the ring; K_{j+1} is one slot past V_j.
        for (int j = -1; j < x.steps && ok; ++j) {
          const uint32_t vs = slot, vphase = phase;
          if (j >= 0) {
            advance();
            ok = mbar_wait(&sb.full[vs], vphase, abortp, spin);
            if (ok && j >= x.fix) {
              ok = mbar_wait(&sb.fixed[vs], (fixpar >> vs) & 1, abortp, spin);
              fixpar ^= 1u << vs;
            }
          }
          const uint32_t ks = slot;
          if (ok && j + 1 < x.steps) ok = mbar_wait(&sb.full[ks], phase, abortp, spin);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (ok && j >= 0 && j < x.nb[w]) {
              if (j == 0 && no[w]) ok = mbar_wait(&sb.oempty[w], (no[w] - 1) & 1, abortp, spin);
              ok = ok && mbar_wait(&sb.pfull[w], np[w] & 1, abortp, spin);
              ++np[w];
              if (ok) {
                fence_after();
                mma_pv(tO + 128 * w, tS + 128 * w, dv0 + vs * STEP, id_pv, j != 0);
                if (j == x.nb[w] - 1) {
                  mma_commit(&sb.ofull[w]);
                  ++no[w];
                }
              }
            }
            if (ok && j + 1 < x.nb[w]) {
              if (j < 0) {
                ok = mbar_wait(&sb.qfull[w], nq[w] & 1, abortp, spin);
                ++nq[w];
              }
              if (ok) {
                fence_after();
                mma_qk<C::BOXES>(tS + 128 * w, dq0 + w * STEP, dk0 + ks * STEP, id_qk);
                mma_commit(&sb.sfull[w]);
                if (j + 2 == x.nb[w]) mma_commit(&sb.qempty[w]);
              }
            }
          }
          if (ok && j >= 0) mma_commit(&sb.empty[vs]);
          if (ok && j + 1 < x.steps) {
            mma_commit(&sb.empty[ks]);
            advance();
          }
        }
        mbar_arrive(&sb.iempty[iq.slot]);
        iq.step();
      }
      if (!ok) *abortp = 1;
      mma_commit(&sb.drain);     // every MMA issued has finished before tensor memory is released
      mbar_wait(&sb.drain, 0, kDrainLimit);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- unseen values of V
    Ring<C::SLOTS> rg;
    Ring<kQueue> iq;
    int item = 0;
    bool ok = true;
    const int tid = threadIdx.x - 64;
    while (ok) {
      ok = warp_wait(&sb.ifull[iq.slot], iq.phase, abortp, spin);
      if (!ok) break;
      const Item x = sb.item[iq.slot];
      if (x.len < 0) break;
      // The fixers pass every slot in order, also those they leave alone: a slot's barrier is
      // waited on by parity, which tells neighbouring phases apart and no more.
      for (int j2 = 0; j2 < 2 * x.steps; ++j2, rg.step()) {
        const int j = j2 >> 1;
        ok = warp_wait(&sb.full[rg.slot], rg.phase, abortp, spin);
        if (!ok) break;
        if (!(j2 & 1) || j < x.fix) {
          if (lane == 0) mbar_arrive(&sb.empty[rg.slot]);
          continue;
        }
        const int live = x.len - j * KEYS;        // rows of this block inside the sequence
        uint4* tile = reinterpret_cast<uint4*>(ring + rg.slot * C::TILE);
        bool found = false;
        for (int i0 = tid; i0 < C::TILE / 16; i0 += 64 * 8) {
          uint4 u[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) u[q] = tile[i0 + 64 * q];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t wd[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
            if ((((i0 + 64 * q) >> 3) & 127) >= live) {
              tile[i0 + 64 * q] = make_uint4(0, 0, 0, 0);
            } else if (a.causal) {
              bool hit = false;
#pragma unroll
              for (int z = 0; z < 4; ++z)
                hit = hit || (wd[z] & 0x7f80u) == 0x7f80u || (wd[z] & 0x7f800000u) == 0x7f800000u;
              if (hit) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  if ((wd[z] & 0x7f80u) == 0x7f80u) wd[z] &= 0xffff0000u;
                  if ((wd[z] & 0x7f800000u) == 0x7f800000u) wd[z] &= 0x0000ffffu;
                }
                tile[i0 + 64 * q] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
                found = true;
              }
            }
          }
        }
        if (found) *(volatile int*)&sb.vbad[iq.slot] = item + 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sb.fixed[rg.slot]);
          mbar_arrive(&sb.empty[rg.slot]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.iempty[iq.slot]);
      iq.step();
      ++item;
    }
    if (!ok && lane == 0) *abortp = 1;
  }
  } else {
    // ---------------------------------------------------------------- softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int w = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int tok_in = row / a.group, head_in = row - tok_in * a.group;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t myS = tS + 128 * w + lanes, myO = tO + 128 * w + lanes;
    Ring<kQueue> iq;
    uint32_t ns = 0, no = 0;         // blocks and outputs so far
    int item = 0;
    bool ok = true;
    while (true) {
      ok = warp_wait(&sb.ifull[iq.slot], iq.phase, abortp, spin);
      if (!ok) break;
      const Item& xi = sb.item[iq.slot];
      const int begin = xi.begin, len = xi.len, hk = xi.hk, tok0 = xi.tok + w * a.tq, nb = xi.nb[w], fix = xi.fix;
      if (len < 0) break;
      const int tok = tok0 + tok_in;
      const int seen = a.causal ? min(len, tok + 1) : len;         // keys this row sees
      const int whole = a.causal ? min(len, tok0 + 1) : len;       // keys every row of the tile sees
      const bool mine = tok_in < a.tq && tok < len;                // a row of the output
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j) {
        ok = warp_wait(&sb.sfull[w], ns & 1, abortp, spin);
        if (!ok) break;
        ++ns;
        fence_after();
        float s[KEYS];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_ld32_nowait(myS + 32 * ch, s + 32 * ch);
        tmem_wait_ld();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) pin32(s + 32 * ch);
        if ((j + 1) * KEYS > whole) {
          const int vis = seen - j * KEYS;
#pragma unroll
          for (int i = 0; i < KEYS; ++i)
            if (i >= vis) s[i] = -INFINITY;
        }
        if (j == 0) m = max_of(s);
        // The probabilities are formed against the reference of the blocks before, and this
        // block's maximum beside them; only when it has left the reference by more than 8 in
        // the exponent are o and the sum rescaled and the probabilities formed again.  A row
        // moves to a reference that differs from its own, so at most twice (an infinite maximum
        // stays); a row of -inf alone has the reference 0 and the sum 0, until it sees more.
        f32x2 sum2[2];
        while (true) {
          const float mc = m == -INFINITY ? 0.f : -m * a.c;
          const f32x2 c2 = pair(a.c, a.c), mc2 = pair(mc, mc);
          float mx4[4] = {m, m, m, m};
          sum2[0] = sum2[1] = pair(0.f, 0.f);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float s0 = s[32 * ch + 2 * i], s1 = s[32 * ch + 2 * i + 1];
              mx4[i & 3] = max3(mx4[i & 3], s0, s1);
              const float2 e = unpair(fma2(pair(s0, s1), c2, mc2));
              const float2 v = (i & 7) < kPolyPairs ? exp2_poly(e) : make_float2(ex2(e.x), ex2(e.y));
              sum2[i & 1] = add2(sum2[i & 1], pair(v.x, v.y));
              p[i] = pack2(v.x, v.y);
            }
            tmem_st16(myS + 16 * ch, p);
          }
          const float mx = max3(max3(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]);
          const bool move = mine && mx != m && !((mx - m) * a.c <= 8.f) && m == m;
          if (!__any_sync(0xffffffffu, move)) break;
          const float fix = move ? ex2((m - mx) * a.c) : 1.f;
#pragma unroll 1
          for (int ch = 0; ch < D; ch += 16) {
            float o[16];
            tmem_ld16(myO + ch, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= fix;
            tmem_st16(myO + ch, reinterpret_cast<const uint32_t*>(o));
          }
          if (move) {
            l *= fix;
            m = mx;
          }
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sb.pfull[w]);
        const float2 l2 = unpair(add2(sum2[0], sum2[1]));
        l += l2.x + l2.y;
      }
      if (!ok) break;
      if (nb > 0) {
        ok = warp_wait(&sb.ofull[w], no & 1, abortp, spin);
        if (!ok) break;
        ++no;
        fence_after();
        const float inv = 1.f / l;
        bf16* out = a.out + (long long)(begin + tok) * a.os0 + (long long)(hk * a.group + head_in) * a.os1;
        const bool vbad = *(volatile int*)&sb.vbad[iq.slot] == item + 1;
#pragma unroll 1
        for (int ch = 0; ch < D; ch += 64) {
          float o[64];
          tmem_ld32_nowait(myO + ch, o);
          tmem_ld32_nowait(myO + ch + 32, o + 32);
          tmem_wait_ld();
          pin32(o);
          pin32(o + 32);
          if (ch + 64 >= D) {        // the last read of O
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.oempty[w]);
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) o[i] *= inv;
          if (mine && ch < a.d) {
            if (vbad) {
              for (int key = fix * KEYS; key < seen; ++key) {
                const bf16* vp = a.v + (long long)(begin + key) * a.vs0 + (long long)hk * a.vs1 + ch;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                  if (ch + i < a.d) {
                    const float vv = to_f32(vp[i]);
                    if (!(fabsf(vv) < INFINITY)) o[i] += vv;
                  }
              }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              if (a.vec) {       // d is a multiple of 8
                if (ch + 8 * q < a.d)
                  *reinterpret_cast<uint4*>(out + ch + 8 * q) =
                      make_uint4(pack2(o[8 * q], o[8 * q + 1]), pack2(o[8 * q + 2], o[8 * q + 3]),
                                 pack2(o[8 * q + 4], o[8 * q + 5]), pack2(o[8 * q + 6], o[8 * q + 7]));
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (ch + 8 * q + i < a.d) out[ch + 8 * q + i] = from_f32<bf16>(o[8 * q + i]);
              }
            }
          }
          __syncwarp();
        }
      }
      __syncwarp();      // every lane has read the item, also of a tile without rows
      if (lane == 0) mbar_arrive(&sb.iempty[iq.slot]);
      iq.step();
      ++item;
    }
    if (lane == 0) {
      sb.done[warp - 4] = ok ? INT_MAX : item;
      if (!ok) {
        *abortp = 1;
        if (a.st) set_error(a.st, PWP_ETIMEOUT, kSiteAttention);
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free(tmem, 512);
  if (*abortp) {
    // A wait ran out: the rows of the items taken and not finished come out NaN, and those of the
    // items that are left.
    const int w = (warp - 4) >> 2, row = (warp & 3) * 32 + lane, tok_in = row / a.group, head_in = row - tok_in * a.group;
    auto fail = [&](const Item& x) {
      const int tok = x.tok + w * a.tq + tok_in;
      if (tok_in >= a.tq || tok >= x.len) return;
      bf16* out = a.out + (long long)(x.begin + tok) * a.os0 + (long long)(x.hk * a.group + head_in) * a.os1;
      for (int c = 0; c < a.d; ++c) out[c] = from_f32<bf16>(__int_as_float(0x7fc00000));
    };
    if (warp >= 4)
      for (int i = sb.done[warp - 4]; i < sb.ntaken; ++i) fail(sb.taken[i % (2 * kQueue)]);
    Items it = sb.it;
    while (true) {
      __syncthreads();
      if (warp == 0) {
        Item x;
        bool bad = false;
        if (!next_item(a, it, x, bad)) x.len = -1;
        if (lane == 0) sb.item[0] = x;
      }
      __syncthreads();
      const Item x = sb.item[0];
      if (x.len < 0) break;
      if (warp >= 4) fail(x);
    }
  }
}

// [n][heads][d] bf16 as a tensor of {d, inner heads, outer heads, n}; false when the copies
// cannot take its base or strides
bool make_map(CUtensorMap* map, const void* p, int d, int inner, int outer, long long n, const int64_t stride[2],
              int rank, int box_heads, int box_tokens) {
  const long long head = inner * outer > 1 ? stride[1] : ((long long)d + 7) / 8 * 8;
  const long long tok = n > 1 ? stride[0] : head * inner * outer;
  if (((uintptr_t)p & 15) || (head & 7) || (tok & 7) || head <= 0 || tok <= 0 || tok >= (1LL << 38) || head >= (1LL << 30))
    return false;
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r;
  if (rank == 4) {
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)n};
    cuuint64_t strides[3] = {(cuuint64_t)head * 2, (cuuint64_t)head * 2 * inner, (cuuint64_t)tok * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)box_heads, 1, (cuuint32_t)box_tokens};
    r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)outer, (cuuint64_t)n};
    cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)tok * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)box_tokens};
    r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  return r == CUDA_SUCCESS;
}

// At most this many items: a sequence's last tile pair may be partly filled.
long long most_items(const pwp_attention_args& a) {
  return (a.n / (2 * (128 / (a.hq / a.hk))) + a.nseq) * (long long)a.hk;
}
constexpr size_t kAttentionWorkspace = 256;

template <int D>
cudaError_t run(const pwp_attention_args& a, cudaStream_t s, bool* used) {
  const int group = a.hq / a.hk, tq = 128 / group;
  CUtensorMap qm, km, vm;
  if (!make_map(&qm, a.q_dev, a.d, group, a.hk, a.n, a.q_stride, 4, group, tq) ||
      !make_map(&km, a.k_dev, a.d, 1, a.hk, a.n, a.k_stride, 3, 1, KEYS) ||
      !make_map(&vm, a.v_dev, a.d, 1, a.hk, a.n, a.v_stride, 3, 1, KEYS))
    return cudaSuccess;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t ready = on_first_use(attr_done, [] {
    return cudaFuncSetAttribute(attention_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
  });
  if (ready != cudaSuccess) return ready;
  Att x;
  x.cu = a.cu_seqlens_dev;
  x.st = a.stats_dev;
  x.out = (bf16*)a.out_dev;
  x.v = (const bf16*)a.v_dev;
  x.n = a.n;
  x.os0 = a.out_stride[0];
  x.os1 = a.out_stride[1];
  x.vs0 = a.v_stride[0];
  x.vs1 = a.v_stride[1];
  x.next = nullptr;
  x.nseq = a.nseq;
  x.hk = a.hk;
  x.group = group;
  x.tq = tq;
  x.d = a.d;
  x.causal = a.causal != 0;
  x.c = a.scale * 1.4426950408889634f;
  x.vec = ((uintptr_t)a.out_dev & 15) == 0 && (a.out_stride[0] & 7) == 0 && (a.out_stride[1] & 7) == 0;
  const long long items = most_items(a);
  if (items >= 0x7fffffffLL - kNumSM) return cudaSuccess;
  const int grid = items < kNumSM ? (int)items : kNumSM;
  *used = true;
  cudaError_t e;
  if (items <= kNumSM) {
    e = launch_pdl(attention_tc_kernel<D>, dim3(grid), dim3(kThreadsAtt), (size_t)Cfg<D>::SMEM, s, qm, km, vm, x, wait_limit());
  } else {
    // Started after its predecessor: CTAs that start early, on the SMs the predecessor's CTAs leave
    // first, cost more than the start (16 x 2048 tokens of 32 heads one after another: 765 us,
    // 618 this way; 1 x 1024: 28.2 us early, 29.1 this way).
    if (a.ws_dev && a.ws_bytes >= kAttentionWorkspace && attention_workspace(a)) {
      x.next = (int*)a.ws_dev;
      e = cudaMemsetAsync(a.ws_dev, 0, sizeof(int), s);
      if (e != cudaSuccess) return e;
    }
    attention_tc_kernel<D><<<grid, kThreadsAtt, Cfg<D>::SMEM, s>>>(qm, km, vm, x, wait_limit());
    e = cudaSuccess;
  }
  count_launches(1);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

// Not for fp32, head sizes past 128 or no multiple of 8, more than 128 query heads per key head,
// and a scale that is not positive (the running maximum is taken of the unscaled scores).
static bool takes(const pwp_attention_args& a) {
  return a.type == PWP_BF16 && a.d <= 128 && (a.d & 7) == 0 && a.hq / a.hk <= 128 && a.scale > 0.f;
}

// The counter pays where a CTA has few long items: clearing it and asking it cost 3 us and about
// a microsecond an item.  With it and without, us: 1 x 2048 tokens of 32 heads 54, 64; 4 x 2048
// 175, 180; 10 sequences of 0 to 4095 tokens 276, 301; but 16 x 2048 (28 items a CTA) 644, 636,
// and 64 x 128 71, 67.
size_t attention_workspace(const pwp_attention_args& a) {
  const long long items = takes(a) ? most_items(a) : 0;
  return items > kNumSM && items <= 16 * kNumSM && a.n >= 512LL * a.nseq ? kAttentionWorkspace : 0;
}

// Declines (used = false) also for tensors the copies cannot take.
cudaError_t launch_attention_tc(const pwp_attention_args& a, cudaStream_t s, bool* used) {
  *used = false;
  if (!takes(a)) return cudaSuccess;
  return a.d <= 64 ? run<64>(a, s, used) : run<128>(a, s, used);
}

}  // namespace pwp
