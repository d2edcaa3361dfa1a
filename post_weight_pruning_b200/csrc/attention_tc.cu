// Attention within packed sequences on the 5th-generation tensor cores (bf16 operands, fp32
// scores, statistics and sums).
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(c (s_ij - m_i)),  s = q k^T,  c = scale log2(e)
//
// in one pass over the keys, 128 at a time, with a reference m_i that is the running maximum
// or lags behind it by at most 8 in the exponent: o and the sum are rescaled only when the
// maximum has grown by more (p then stays below 2^8, far from any overflow, and bf16 keeps
// its relative precision).
//
// A persistent CTA takes pairs of tiles of 128 query rows.  A tile's rows are tokens times the
// query heads that share a key head (row = token * group + head), so grouped heads read their
// keys once and short sequences fill tiles; one TMA box gathers them.  Roles:
//   warp 0         TMA: q of both tiles, then K_0, V_0, K_1, V_1, ... through a ring of slots
//   warp 1         MMA: S_w = Q_w K_j^T and O_w += P_w V_j for the two tiles w in turn, so the
//                  tensor core works on one tile while the other's softmax runs.  P_w
//                  (bf16) overlays S_w in tensor memory and is the A operand from there.
//   warps 2, 3     keep what no query may see out of V: rows behind the sequence's end are
//                  zeroed in shared memory (0 * NaN is NaN), and in the blocks the causal mask
//                  cuts, non-finite values are zeroed and added back at the end to the rows
//                  that do see them
//   warps 4-7, 8-11  softmax of tile 0 and 1, one row per thread, and the rows' output
// S_w(j) becoming full implies that O_w holds block j-1's product (the MMAs of a CTA complete
// in order), so a softmax thread may rescale its row of O_w without another barrier.
//
// What bounds it (16 x 2048 tokens, 32 heads of 128, timers in the roles): a tile's chain of
// softmax (about 1700 cycles per 128 keys: 1024 of exponentials at 16 a cycle and SM, the rest issue
// and latency), two MMA groups of 512 and the hand-overs between them (about 600), which the
// other tile fills only in part: 3400 cycles per block and pair of tiles, of which the tensor
// core works 2048.  Tried and slower, full attention at that size against 1.09 ms: blocks of 64
// keys with two S per tile, so that QK runs two blocks ahead (1.42, the MMA warp's waits double);
// P handed over in halves (1.24 to 1.36, the MMA warp then waits on one tile while the other is
// ready); one MMA warp per tile with 32 keys at a time (1.31); more exponentials on the FMA pipe
// than one pair in eight (1.13 at two, 1.19 at three).
//
// Every wait is bounded: one that runs out records PWP_ETIMEOUT and the rows come out NaN;
// copies and MMAs in flight are waited for before a CTA leaves.
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
constexpr int kFlags = 8;                      // items a fixer can be ahead of an epilogue, at least

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
};

// The items of a CTA, in order: the sequences' tile pairs (the last, longest one of a
// sequence first) with the key heads running fastest.
struct Items {
  int t, s0, base;        // next item; the first sequence of the scan's chunk; tiles before it
};
struct Item {
  int begin, len, hk;     // sequence, key head
  int tok[2];             // first token of each tile
  int nb[2];              // key blocks of each tile (0: no rows)
  int fix;                // first block of V that the fixer looks at
};

__device__ __forceinline__ bool next_item(const Att& a, Items& it, Item& x, bool& bad) {
  const int lane = threadIdx.x & 31;
  const int per = 2 * a.tq;
  const int tile = it.t / a.hk;
  x.hk = it.t - tile * a.hk;
  it.t += gridDim.x;
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
      const int p = it.base + after - 1 - tile;                // its tiles from the last one
      x.tok[0] = p * per;
      x.tok[1] = x.tok[0] + a.tq;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int last = min(x.len, x.tok[w] + a.tq);
        x.nb[w] = x.tok[w] >= x.len ? 0 : ((a.causal ? last : x.len) + KEYS - 1) / KEYS;
      }
      x.fix = a.causal ? (x.tok[0] + 1) / KEYS : x.len / KEYS;
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
// The MMAs of one tile product are issued by one elected lane of a converged warp, in one
// statement with the operands advanced inside it (measured in this kernel: a statement per MMA
// costs 0.1 ms more; under a lane test with descriptors formed in between, 0.2 ms).
//
// S (128 x 128) = Q (128 x 64 BOXES) K^T: steps of 16 are 32 bytes inside a swizzled row, a box of
// 64 further on after four.
template <int BOXES>
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred q, f, t;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
      "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(idesc)
      : "memory");
  if (BOXES == 2)
    asm volatile(
        "{\n\t.reg .pred q, t;\n\t.reg .b64 x, y;\n\t"
        "setp.eq.b32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "add.s64 x, %1, 1024;\n\tadd.s64 y, %2, 1024;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
        "add.s64 x, %1, 1026;\n\tadd.s64 y, %2, 1026;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
        "add.s64 x, %1, 1028;\n\tadd.s64 y, %2, 1028;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
        "add.s64 x, %1, 1030;\n\tadd.s64 y, %2, 1030;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc)
        : "memory");
}
// O += P V over 64 keys: P in tensor memory (16 keys are 8 columns), V MN-major (16 keys are
// 2048 bytes).
__device__ __forceinline__ void mma_pv64(uint32_t d, uint32_t ta, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred q, p, t;\n\t.reg .b64 y;\n\t.reg .b32 a;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 y, %2, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, t;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 y, %2, 256;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, t;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 y, %2, 384;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, t;\n\t}" ::"r"(d),
      "r"(ta), "l"(db), "r"(idesc), "r"(acc)
      : "memory");
}
// One arrival on `bar` when the MMAs issued so far have completed (the whole warp calls it).
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
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
// Two fp32 operations in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x of two values on the FMA pipe: x = n + f with n the nearest whole number, f in [-1/2, 1/2],
// and 2^f by the cubic 1 + f (a + f (b + f c)) of least largest relative error (found by linear
// programming over 4001 points: 1.02e-4 = 2^-13.3, a sixteenth of a bf16 half step).  The
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
  int vbad[kFlags];                            // item + 1: a non-finite value was taken out of its V
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
    for (int i = 0; i < kFlags; ++i) sb.vbad[i] = 0;
  }
  if (warp == 1) tmem_alloc(&sb.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  pdl_enter();
  const uint32_t tmem = sb.tmem;
  const uint32_t tS = tmem, tO = tmem + 256;      // S_w at 128 w, O_w at 256 + 128 w

  Items it{(int)blockIdx.x, 0, 0};
  Item x;
  bool bad = false;

  // Registers: the softmax warps hold a row of 128 scores.  The CTA was launched with 384 * 168;
  // 128 * 72 + 256 * 216 is exactly that.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
    // ---------------------------------------------------------------- copies
    uint32_t r = 0, qn[2] = {0, 0};       // slots filled, q tiles loaded
    bool ok = true;
    const uint32_t qbytes = (uint32_t)(C::BOXES * a.tq * a.group * 128);
    while (ok && next_item(a, it, x, bad)) {
      if (lane == 0) {
        const int nb = max(x.nb[0], x.nb[1]);
        for (int j = 0; j < nb && ok; ++j) {
          if (j == 0) {
            for (int w = 0; w < 2 && ok; ++w) {
              if (!x.nb[w]) continue;
              if (qn[w] && !mbar_wait(&sb.qempty[w], (qn[w] - 1) & 1, abortp, spin)) {
                ok = false;
                break;
              }
              mbar_expect_tx(&sb.qfull[w], qbytes);
              for (int b = 0; b < C::BOXES; ++b)
                tma_load_4d(smem + w * C::TILE + b * BOX, &qmap, &sb.qfull[w], 64 * b, 0, x.hk, x.begin + x.tok[w]);
              ++qn[w];
            }
          }
          for (int kv = 0; kv < 2 && ok; ++kv) {
            const int s = (int)(r % C::SLOTS);
            if (r >= C::SLOTS && !mbar_wait(&sb.empty[s], (r / C::SLOTS - 1) & 1, abortp, spin)) {
              ok = false;
              break;
            }
            mbar_expect_tx(&sb.full[s], C::TILE);
            for (int b = 0; b < C::BOXES; ++b)
              tma_load_3d(ring + s * C::TILE + b * BOX, kv ? &vmap : &kmap, &sb.full[s], 64 * b, x.hk, x.begin + j * KEYS);
            ++r;
          }
        }
        if (!ok) *abortp = 1;
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      if (bad && a.st) set_error(a.st, PWP_EINVAL, kSiteAttention);
      for (uint32_t i = r > C::SLOTS ? r - C::SLOTS : 0; i < r; ++i)
        mbar_wait(&sb.full[i % C::SLOTS], (i / C::SLOTS) & 1, kDrainLimit);
      for (int w = 0; w < 2; ++w)
        if (qn[w]) mbar_wait(&sb.qfull[w], (qn[w] - 1) & 1, kDrainLimit);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    const uint32_t sq = smem_u32(smem), sr = smem_u32(ring);
    constexpr uint32_t id_qk = idesc_of(KEYS, 0), id_pv = idesc_of(D, 1);
    uint32_t r = 0, fixpar = 0;
    uint32_t nq = 0, np[2] = {0, 0}, no[2] = {0, 0};   // items, blocks and outputs so far
    bool ok = true;
    while (ok && next_item(a, it, x, bad)) {
      const int nb = max(x.nb[0], x.nb[1]);
      // S_w(0), then for every block O_w += P_w V_j and S_w(j + 1), the tiles in turn
      for (int j = -1; j < nb && ok; ++j) {
        const uint32_t rk = r + 2 * (uint32_t)(j + 1), rv = rk - 1;
        const int sk = (int)(rk % C::SLOTS), sv = (int)(rv % C::SLOTS);
        const uint32_t kb = sr + sk * C::TILE, vb = sr + sv * C::TILE;
        if (j >= 0) {
          ok = warp_wait(&sb.full[sv], (rv / C::SLOTS) & 1, abortp, spin);
          if (ok && j >= x.fix) {
            ok = warp_wait(&sb.fixed[sv], (fixpar >> sv) & 1, abortp, spin);
            fixpar ^= 1u << sv;
          }
        }
        if (ok && j + 1 < nb) ok = warp_wait(&sb.full[sk], (rk / C::SLOTS) & 1, abortp, spin);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (ok && j >= 0 && j < x.nb[w]) {
            if (j == 0 && no[w]) ok = warp_wait(&sb.oempty[w], (no[w] - 1) & 1, abortp, spin);
            ok = ok && warp_wait(&sb.pfull[w], np[w] & 1, abortp, spin);
            ++np[w];
            if (ok) {
              fence_after();
              mma_pv64(tO + 128 * w, tS + 128 * w, sw128_desc(vb, BOX, 1024), id_pv, j != 0);
              mma_pv64(tO + 128 * w, tS + 128 * w + 32, sw128_desc(vb + 8192, BOX, 1024), id_pv, 1);
              if (j == x.nb[w] - 1) {
                commit_elected(&sb.ofull[w]);
                ++no[w];
              }
            }
          }
          if (ok && j + 1 < x.nb[w]) {
            if (j < 0) ok = warp_wait(&sb.qfull[w], (nq >> (16 * w)) & 1, abortp, spin);
            if (ok) {
              fence_after();
              mma_qk<C::BOXES>(tS + 128 * w, sw128_desc(sq + w * C::TILE, 16, 1024), sw128_desc(kb, 16, 1024), id_qk);
              commit_elected(&sb.sfull[w]);
              if (j + 2 == x.nb[w]) commit_elected(&sb.qempty[w]);
            }
          }
        }
        if (ok && j >= 0) commit_elected(&sb.empty[sv]);
        if (ok && j + 1 < nb) commit_elected(&sb.empty[sk]);
      }
      // q tiles loaded so far, one bit (the phase) per tile
      if (x.nb[0]) nq ^= 1u;
      if (x.nb[1]) nq ^= 1u << 16;
      r += 2 * (uint32_t)nb;
      if (!ok && lane == 0) *abortp = 1;
    }
    commit_elected(&sb.drain);     // every MMA issued has finished before tensor memory is released
    mbar_wait(&sb.drain, 0, kDrainLimit);
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- unseen values of V
    uint32_t r = 0;
    int item = 0;
    bool ok = true;
    const int tid = threadIdx.x - 64;
    while (ok && next_item(a, it, x, bad)) {
      const int nb = max(x.nb[0], x.nb[1]);
      // The fixers pass every slot in order, also those they leave alone: a slot's barrier is
      // waited on by parity, which tells neighbouring phases apart and no more.
      for (int j2 = 0; j2 < 2 * nb; ++j2) {
        const uint32_t rv = r + (uint32_t)j2;
        const int s = (int)(rv % C::SLOTS), j = j2 >> 1;
        ok = mbar_wait(&sb.full[s], (rv / C::SLOTS) & 1, abortp, spin);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) *abortp = 1;
          break;
        }
        if (!(j2 & 1) || j < x.fix) {
          if (lane == 0) mbar_arrive(&sb.empty[s]);
          continue;
        }
        const int live = x.len - j * KEYS;        // rows of this block inside the sequence
        uint4* tile = reinterpret_cast<uint4*>(ring + s * C::TILE);
        bool found = false;
        for (int i = tid; i < C::TILE / 16; i += 64) {
          const int row = (i >> 3) & 127;
          if (row >= live) {
            tile[i] = make_uint4(0, 0, 0, 0);
          } else if (a.causal) {
            uint4 u = tile[i];
            uint32_t wd[4] = {u.x, u.y, u.z, u.w};
            bool hit = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if ((wd[q] & 0x7f80u) == 0x7f80u) {
                wd[q] &= 0xffff0000u;
                hit = true;
              }
              if ((wd[q] & 0x7f800000u) == 0x7f800000u) {
                wd[q] &= 0x0000ffffu;
                hit = true;
              }
            }
            if (hit) {
              tile[i] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
              found = true;
            }
          }
        }
        if (found) *(volatile int*)&sb.vbad[item & (kFlags - 1)] = item + 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sb.fixed[s]);
          mbar_arrive(&sb.empty[s]);
        }
      }
      r += 2 * (uint32_t)nb;
      ++item;
    }
  }
  } else {
    // ---------------------------------------------------------------- softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int tok_in = row / a.group, head_in = row - tok_in * a.group;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t myS = tS + 128 * w + lanes, myO = tO + 128 * w + lanes;
    uint32_t ns = 0, no = 0;
    int item = 0;
    bool ok = true;
    while (next_item(a, it, x, bad)) {
      const int nb = x.nb[w];
      const int tok = x.tok[w] + tok_in;
      const int seen = a.causal ? min(x.len, tok + 1) : x.len;     // keys this row sees
      const int whole = a.causal ? min(x.len, x.tok[w] + 1) : x.len;   // keys every row of the tile sees
      const bool mine = tok_in < a.tq && tok < x.len;              // a row of the output
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j) {
        if (ok) {
          ok = mbar_wait(&sb.sfull[w], ns & 1, abortp, spin);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) {
            *abortp = 1;
            if (a.st) set_error(a.st, PWP_ETIMEOUT, kSiteAttention);
          }
        }
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
        // the exponent are o and the sum rescaled and the probabilities formed again.
        f32x2 sum2[2];
        while (true) {
          const f32x2 c2 = pair(a.c, a.c), mc2 = pair(-m * a.c, -m * a.c);
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
          const bool move = mine && !((mx - m) * a.c <= 8.f) && m == m;
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
      if (nb > 0) {
        if (ok) {
          ok = mbar_wait(&sb.ofull[w], no & 1, abortp, spin);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) {
            *abortp = 1;
            if (a.st) set_error(a.st, PWP_ETIMEOUT, kSiteAttention);
          }
        }
        ++no;
        fence_after();
        const float inv = 1.f / l;
        bf16* out = a.out + (long long)(x.begin + tok) * a.os0 + (long long)(x.hk * a.group + head_in) * a.os1;
        const bool vbad = *(volatile int*)&sb.vbad[item & (kFlags - 1)] == item + 1;
#pragma unroll 1
        for (int ch = 0; ch < D; ch += 16) {
          float o[16];
          tmem_ld16(myO + ch, o);
          if (ch + 16 >= D) {        // the last read of O
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.oempty[w]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = ok ? o[i] * inv : __int_as_float(0x7fc00000);
          if (mine && ch < a.d) {
            if (vbad) {
              for (int key = x.fix * KEYS; key < seen; ++key) {
                const bf16* vp = a.v + (long long)(x.begin + key) * a.vs0 + (long long)x.hk * a.vs1 + ch;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (ch + i < a.d) {
                    const float vv = to_f32(vp[i]);
                    if (!(fabsf(vv) < INFINITY)) o[i] += vv;
                  }
              }
            }
            if (a.vec && ch + 16 <= a.d) {
              *reinterpret_cast<uint4*>(out + ch) =
                  make_uint4(pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]), pack2(o[6], o[7]));
              *reinterpret_cast<uint4*>(out + ch + 8) =
                  make_uint4(pack2(o[8], o[9]), pack2(o[10], o[11]), pack2(o[12], o[13]), pack2(o[14], o[15]));
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (ch + i < a.d) out[ch + i] = from_f32<bf16>(o[i]);
            }
          }
          __syncwarp();
        }
      }
      ++item;
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free(tmem, 512);
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

template <int D>
cudaError_t run(const pwp_attention_args& a, cudaStream_t s, bool* used) {
  const int group = a.hq / a.hk, tq = 128 / group;
  CUtensorMap qm, km, vm;
  if (!make_map(&qm, a.q_dev, a.d, group, a.hk, a.n, a.q_stride, 4, group, tq) ||
      !make_map(&km, a.k_dev, a.d, 1, a.hk, a.n, a.k_stride, 3, 1, KEYS) ||
      !make_map(&vm, a.v_dev, a.d, 1, a.hk, a.n, a.v_stride, 3, 1, KEYS))
    return cudaSuccess;
  static std::atomic<unsigned long long> attr_done{0};
  if (first_on_device(attr_done)) {
    cudaError_t e = cudaFuncSetAttribute(attention_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
  }
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
  x.nseq = a.nseq;
  x.hk = a.hk;
  x.group = group;
  x.tq = tq;
  x.d = a.d;
  x.causal = a.causal != 0;
  x.c = a.scale * 1.4426950408889634f;
  x.vec = ((uintptr_t)a.out_dev & 15) == 0 && (a.out_stride[0] & 7) == 0 && (a.out_stride[1] & 7) == 0;
  // at most this many items: a sequence's last tile pair may be partly filled
  const long long items = (a.n / (2 * tq) + a.nseq) * (long long)a.hk;
  if (items >= 0x7fffffffLL - kNumSM) return cudaSuccess;
  const int grid = items < kNumSM ? (int)items : kNumSM;
  *used = true;
  const cudaError_t e = launch_pdl(attention_tc_kernel<D>, dim3(grid), dim3(kThreadsAtt), (size_t)Cfg<D>::SMEM, s, qm, km,
                                   vm, x, wait_limit());
  count_launches(1);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

// Declines (used = false) for fp32, head sizes past 128 or no multiple of 8, more than 128
// query heads per key head, a scale that is not positive (the running maximum is taken of the
// unscaled scores) and tensors the copies cannot take.
cudaError_t launch_attention_tc(const pwp_attention_args& a, cudaStream_t s, bool* used) {
  *used = false;
  if (a.type != PWP_BF16 || a.d > 128 || (a.d & 7) || a.hq / a.hk > 128 || !(a.scale > 0.f)) return cudaSuccess;
  return a.d <= 64 ? run<64>(a, s, used) : run<128>(a, s, used);
}

}  // namespace pwp
