// act(x W^T + bias) (* (x W_up^T + bias_up)) + residual on the CUDA cores: fp32 tensors, and
// bf16 ones whose bases or strides the tensor-core kernels' copies cannot take.
//
// One CTA of 256 threads per 64 x 64 output tile; 16 columns of x and W at a time go through
// shared memory as fp32 and every thread keeps a 4 x 4 piece (two for the gated product) in
// registers.  Bound by the FMA pipe (128 lanes a cycle and SM).
#include "block_ops.cuh"

namespace pwp {
namespace {

constexpr int TS = 64, KS = 16;

template <typename T, bool GATED>
__global__ void __launch_bounds__(256) linear_simt_kernel(const pwp_linear_args a, int act) {
  __shared__ float xs[KS][TS + 4], ws[GATED ? 2 : 1][KS][TS + 4];
  const int tn = (a.n + TS - 1) / TS;
  const long long r0 = (long long)(blockIdx.x / tn) * TS;
  const int c0 = (int)(blockIdx.x % tn) * TS;
  const T* x = (const T*)a.x_dev;
  const T* w[2] = {(const T*)a.w_dev, (const T*)a.w_up_dev};
  const long long wst[2] = {a.w_stride, a.w_up_stride};
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[GATED ? 2 : 1][4][4] = {};
  for (int k0 = 0; k0 < a.k; k0 += KS) {
    for (int i = threadIdx.x; i < TS * KS; i += 256) {
      const int r = i / KS, k = i % KS;
      const bool in_k = k0 + k < a.k;
      xs[k][r] = in_k && r0 + r < a.rows ? to_f32(x[(r0 + r) * a.x_stride + k0 + k]) : 0.f;
#pragma unroll
      for (int m = 0; m < (GATED ? 2 : 1); ++m)
        ws[m][k][r] = in_k && c0 + r < a.n ? to_f32(w[m][(long long)(c0 + r) * wst[m] + k0 + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const float4 xv = *reinterpret_cast<const float4*>(&xs[k][ty * 4]);
      const float xa[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int m = 0; m < (GATED ? 2 : 1); ++m) {
        const float4 wv = *reinterpret_cast<const float4*>(&ws[m][k][tx * 4]);
        const float wa[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][i][j] += xa[i] * wa[j];
      }
    }
    __syncthreads();
  }
  const T* b = (const T*)a.bias_dev;
  const T* bu = (const T*)a.bias_up_dev;
  const T* res = (const T*)a.residual_dev;
  T* out = (T*)a.out_dev;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = r0 + ty * 4 + i;
    if (r >= a.rows) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + tx * 4 + j;
      if (c >= a.n) break;
      float v = activate(act, acc[0][i][j] + (b ? to_f32(b[c]) : 0.f));
      if (GATED) v *= acc[GATED ? 1 : 0][i][j] + (bu ? to_f32(bu[c]) : 0.f);
      if (res) v += to_f32(res[r * a.residual_stride + c]);
      out[r * a.out_stride + c] = from_f32<T>(v);
    }
  }
}

}  // namespace

cudaError_t launch_linear_simt(const pwp_linear_args& a, cudaStream_t s) {
  const long long tiles = ((a.rows + TS - 1) / TS) * ((a.n + TS - 1) / TS);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)tiles;
  const bool gated = a.w_up_dev != nullptr;
  if (a.type == PWP_BF16) {
    if (gated) linear_simt_kernel<__nv_bfloat16, true><<<grid, 256, 0, s>>>(a, a.activation);
    else linear_simt_kernel<__nv_bfloat16, false><<<grid, 256, 0, s>>>(a, a.activation);
  } else {
    if (gated) linear_simt_kernel<float, true><<<grid, 256, 0, s>>>(a, a.activation);
    else linear_simt_kernel<float, false><<<grid, 256, 0, s>>>(a, a.activation);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace pwp
