// Row norms, and the norm and position rotation of queries and keys.
//
// rms_norm: y = x / sqrt(mean(x^2) + eps) * w.  One CTA per row: a thread keeps its share of
// the row as partial sums, the CTA adds them, and the row is read again (from L1 or L2) to
// be scaled.
//
// qk_norm_rope: one CTA per token.  The token's rot/2 angles position * f_i are formed once in
// double precision -- at position 10^6 an fp32 product would be off by 0.06 rad -- reduced to
// a turn in [-1/2, 1/2] and only then rounded to fp32 for sincospi; every head of the token
// uses them.  One warp takes a head at a time through shared memory.
#include "block_ops.cuh"

namespace pwp {
namespace {

constexpr int kNormThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const T* x, long long xs, int width,
                                                                const T* __restrict__ w, float eps, T* out,
                                                                long long os) {
  __shared__ float part[kNormThreads / 32];
  const T* xr = x + (long long)blockIdx.x * xs;
  T* yr = out + (long long)blockIdx.x * os;
  float sum = 0.f;
  for (int i = threadIdx.x; i < width; i += kNormThreads) {
    const float v = to_f32(xr[i]);
    sum += v * v;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 32; ++i) sum += part[i];
  const float r = 1.f / sqrtf(sum / (float)width + eps);
  for (int i = threadIdx.x; i < width; i += kNormThreads) {
    const float v = to_f32(xr[i]) * r;
    yr[i] = from_f32<T>(w ? v * to_f32(w[i]) : v);
  }
}

constexpr int kRopeWarps = 8;

// cosine and sine of position * f, both times `factor`
__device__ __forceinline__ float2 turn_of(long long position, double f, float factor) {
  const double t = (double)position * f * 0.15915494309189533577;   // turns
  const float r = (float)(t - rint(t));
  float s, c;
  sincospif(2.f * r, &s, &c);
  return make_float2(c * factor, s * factor);
}

template <typename T>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const pwp_rope_args a) {
  extern __shared__ float smem[];
  const long long t = blockIdx.x;
  const int half = a.rot / 2, d = a.d;
  float2* cs = reinterpret_cast<float2*>(smem);
  float* head = smem + 2 * half + (threadIdx.x >> 5) * d;
  const int lane = threadIdx.x & 31;
  const long long pos = half ? a.positions_dev[t] : 0;
  for (int i = threadIdx.x; i < half; i += blockDim.x) cs[i] = turn_of(pos, a.freqs_dev[i], a.factor);
  __syncthreads();
  for (int h = threadIdx.x >> 5; h < a.hq + a.hk; h += kRopeWarps) {
    const bool is_q = h < a.hq;
    const int hh = is_q ? h : h - a.hq;
    const int64_t* is = is_q ? a.q_stride : a.k_stride;
    const int64_t* os = is_q ? a.q_out_stride : a.k_out_stride;
    const T* x = (const T*)(is_q ? a.q_dev : a.k_dev) + t * is[0] + hh * is[1];
    T* y = (T*)(is_q ? a.q_out_dev : a.k_out_dev) + t * os[0] + hh * os[1];
    const T* w = (const T*)(is_q ? a.q_weight_dev : a.k_weight_dev);
    float sum = 0.f;
    for (int i = lane; i < d; i += 32) {
      const float v = to_f32(x[i]);
      head[i] = v;
      sum += v * v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    if (w) {
      const float r = 1.f / sqrtf(sum / (float)d + a.eps);
      for (int i = lane; i < d; i += 32) head[i] = head[i] * r * to_f32(w[i]);
      __syncwarp();
    }
    for (int i = lane; i < half; i += 32) {
      const int ia = a.layout == PWP_ROPE_HALF ? i : 2 * i;
      const int ib = a.layout == PWP_ROPE_HALF ? i + half : 2 * i + 1;
      const float u = head[ia], v = head[ib];
      const float2 c = cs[i];
      y[ia] = from_f32<T>(u * c.x - v * c.y);
      y[ib] = from_f32<T>(v * c.x + u * c.y);
    }
    for (int i = a.rot + lane; i < d; i += 32) y[i] = from_f32<T>(head[i]);
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_rms_norm(const void* x, int type, long long rows, int width, long long xs, const void* w, float eps,
                            void* out, long long os, cudaStream_t s) {
  if (type == PWP_BF16)
    rms_norm_kernel<__nv_bfloat16><<<(unsigned)rows, kNormThreads, 0, s>>>(
        (const __nv_bfloat16*)x, xs, width, (const __nv_bfloat16*)w, eps, (__nv_bfloat16*)out, os);
  else
    rms_norm_kernel<float><<<(unsigned)rows, kNormThreads, 0, s>>>((const float*)x, xs, width, (const float*)w, eps,
                                                                   (float*)out, os);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const pwp_rope_args& a, cudaStream_t s) {
  const size_t smem = sizeof(float) * (size_t)(a.rot + kRopeWarps * a.d);   // at most 36 KB (d <= 1024)
  if (a.type == PWP_BF16)
    rope_kernel<__nv_bfloat16><<<(unsigned)a.n, 32 * kRopeWarps, smem, s>>>(a);
  else
    rope_kernel<float><<<(unsigned)a.n, 32 * kRopeWarps, smem, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace pwp
