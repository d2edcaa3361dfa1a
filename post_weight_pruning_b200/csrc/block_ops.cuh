// Internal declarations of the decoder block's forward operators (norms, rotated queries
// and keys, packed attention, projections with their epilogues).
#pragma once

#include <cuda_bf16.h>

#include "pwp_internal.cuh"

namespace pwp {

constexpr int kSiteAttention = 9, kSiteLinear = 10;   // pwp_stats::status_site of these calls

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Phi(-a), a >= 0, of the standard normal distribution to 2^-20 of itself, and past a = 2 to
// a^2 2^-23: e^(-a^2/2) times a polynomial in t = 1 / (1 + 0.362 a), the form of Hastings
// (Abramowitz and Stegun, 26.2.17).  The coefficients have the least largest relative error over
// [0, 13.5] (7.1e-7; found by linear programming over 4000 points).
__device__ __forceinline__ float normal_tail(float a) {
  const float t = __fdividef(1.f, fmaf(a, 0.362f, 1.f));
  float p = fmaf(0.04804705845356076f, t, -0.1803753304984107f);
  p = fmaf(p, t, 0.17710773021334036f);
  p = fmaf(p, t, 0.028496550194732795f);
  p = fmaf(p, t, 0.13955203359788615f);
  p = fmaf(p, t, 0.14266678446936745f);
  p = fmaf(p, t, 0.1445055271023927f);
  return p * t * __expf(-0.5f * a * a);
}

// x / (1 + e^-z), z of the sign of x, as x (e^z / (1 + e^z)).  z is cut at 60, where the fraction
// is 1 to the last bit, so e^z never overflows and results far below zero keep their value
// down to the smallest numbers (e^-z is infinite from z = -88.7 on, where x e^z is still a normal
// number).  bf16 takes the fast exponential (off by 2 + 1.17 |z| steps of 2^-23, a hundredth
// of bf16's half step at |z| = 88); the division is good for divisors up to 2^126 (a full one calls
// a routine, which cost the fp32 kernel's main loop registers: 1024 x 8192 x 4096 1710 us, 1635
// this way).
template <typename T>
__device__ __forceinline__ float times_logistic(float x, float z) {
  z = fminf(z, 60.f);
  const float e = sizeof(T) == 4 ? expf(z) : __expf(z);
  return x * __fdividef(e, 1.f + e);
}

// Activations of pwp_activation in fp32, for results of type T.
//
// erf-GELU: 1 + erf(x / sqrt 2) would cancel below zero (nothing is left from x = -5.8 on), so
// fp32 takes erfc, and bf16, whose half step is 2^-8, normal_tail: 16384 x 128 x 8192, where the epilogue
// is the bound, takes 209 us with it, 208 with erff and 392 with erfcf.
template <typename T>
__device__ __forceinline__ float activate(int act, float x) {
  switch (act) {
    case PWP_ACT_RELU: return x != x ? x : fmaxf(x, 0.f);
    case PWP_ACT_SILU: return times_logistic<T>(x, x);
    case PWP_ACT_GELU: {
      if (sizeof(T) == 4) return 0.5f * x * erfcf(x * -0.70710678118654752f);
      const float q = normal_tail(fabsf(x));
      return x * (x < 0.f ? q : 1.f - q);
    }
    case PWP_ACT_GELU_TANH:      // (1 + tanh t) / 2 = 1 / (1 + e^-2t)
      return times_logistic<T>(x, 1.5957691216057308f * (x + 0.044715f * x * x * x));
    default: return x;
  }
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
// Thread-block clusters: this CTA's rank, a barrier of all its threads, and stores into another
// CTA's shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address, in the cluster's window, of a shared-memory address of this CTA as CTA `rank` has it
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void remote_store4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// One tile of a packed batch: rows [begin + first, begin + first + per) of the sequence
// [begin, begin + len).
struct SeqTile {
  int begin, len, first;
};
// Where a search stands: the first sequence of its chunk of 32, and the tiles before it.
struct SeqScan {
  int s0 = 0, base = 0;
};

// Finds tile `t` when every sequence is cut into tiles of `per` rows (whole warp, all lanes
// get the answer).  `scan` goes on from call to call: t never decreases, and a CTA that takes many
// tiles reads the offsets once, however many sequences there are.  The first sequence whose
// offsets decrease or leave [0, n] and all behind it count as empty, so the sequences taken
// never overlap; `bad` is set when one is met.  Returns false past the last tile.
__device__ __forceinline__ bool find_seq_tile(const int* __restrict__ cu, int nseq, long long n, int per, int t,
                                              SeqScan& scan, SeqTile& out, bool& bad) {
  const int lane = threadIdx.x & 31;
  for (; scan.s0 < nseq; scan.s0 += 32) {
    const int s = scan.s0 + lane;
    int a = 0, b = 0;
    if (s < nseq) {
      a = cu[s];
      b = cu[s + 1];
    }
    const bool ok = a >= 0 && b >= a && (long long)b <= n;
    const unsigned broken = ~__ballot_sync(0xffffffffu, ok);
    if (broken) bad = true;
    const int len = (broken & (0xffffffffu >> (31 - lane))) ? 0 : b - a;
    const int tiles = (int)(((long long)len + per - 1) / per);
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, t < scan.base + sum);
    if (hit) {
      const int l = __ffs(hit) - 1;
      out.begin = __shfl_sync(0xffffffffu, a, l);
      out.len = __shfl_sync(0xffffffffu, len, l);
      out.first = (t - scan.base - __shfl_sync(0xffffffffu, sum - tiles, l)) * per;
      return true;
    }
    if (broken) {
      scan.s0 = nseq;
      return false;
    }
    scan.base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

cudaError_t launch_rms_norm(const void* x, int type, long long rows, int width, long long xs, const void* w, float eps,
                            void* out, long long os, cudaStream_t s);
cudaError_t launch_qk_norm_rope(const pwp_rope_args& a, cudaStream_t s);
cudaError_t launch_attention_simt(const pwp_attention_args& a, cudaStream_t s);
size_t attention_workspace(const pwp_attention_args& a);
cudaError_t launch_attention_tc(const pwp_attention_args& a, cudaStream_t s, bool* used);
cudaError_t launch_linear_simt(const pwp_linear_args& a, cudaStream_t s);
size_t linear_align_bytes(const pwp_linear_args& a);
cudaError_t launch_linear_align(pwp_linear_args& a, cudaStream_t s);
cudaError_t launch_linear_tc(const pwp_linear_args& a, cudaStream_t s, bool* used);

}  // namespace pwp
