// act(x W^T + bias) (* (x W_up^T + bias_up)) + residual on the CUDA cores: fp32 tensors, and
// bf16 ones whose bases or strides the tensor-core kernels' copies cannot take.
//
// A CTA of 256 threads forms a tile of BM rows x 128 columns of products (for the gated product 64
// columns of W and the same 64 of W_up) from 16 columns of x and W at a time, which go through
// shared memory as fp32, transposed, the next ones loaded into registers meanwhile.  A thread
// keeps 8 x 8 sums (2 x 8 in the 32-row tile) as fp32 pairs, columns 4 tx.. and 64 + 4 tx.., so
// the two products of an output meet in one thread.  Bound by the FMA pipe at 128 rows: the
// tensor cores' fp32 accumulation truncates, which over thousands of additions costs fp32
// results two digits, so they are not used here.
//
// Few tiles: k is split over a cluster's CTAs, whose sums go to the CTA that finishes the row
// through distributed shared memory and are added in rank order.  1024 rows by 4096 x 8192 fp32
// weights: 1.64 ms, 42 TFLOP/s of the 74 that the FMA pipe could do (3.28 ms with tiles of 64 and single
// products; the library 1.20), 8192 rows by 4096 x 4096 5.5 ms, 50 TFLOP/s (library 4.2).  A few rows
// are bound by shared memory, whatever their number: 1 and 16 rows by 4096 x 4096 56 us (library 11
// and 66).
#include <type_traits>

#include "block_ops.cuh"

namespace pwp {
namespace {

constexpr int BN = 128, BK = 16, kThreadsSimt = 256, kMaxSplit = 8;

// four consecutive values from column k of a row, zero from `left` on
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, int left, bool vec) {
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (vec && left >= 4) {
    if (sizeof(T) == 4) return *reinterpret_cast<const float4*>(p);
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) v[i] = to_f32(p[i]);
  return make_float4(v[0], v[1], v[2], v[3]);
}

// f(std::integral_constant<int, act>): one branch, not one per value
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
  switch (act) {
    case PWP_ACT_RELU: f(std::integral_constant<int, PWP_ACT_RELU>()); break;
    case PWP_ACT_SILU: f(std::integral_constant<int, PWP_ACT_SILU>()); break;
    case PWP_ACT_GELU: f(std::integral_constant<int, PWP_ACT_GELU>()); break;
    case PWP_ACT_GELU_TANH: f(std::integral_constant<int, PWP_ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, PWP_ACT_NONE>()); break;
  }
}

// Four neighbouring outputs from their sum(s).
template <typename T, bool GATED, int ACT>
__device__ __forceinline__ void finish4(const pwp_linear_args& a, long long r, int c, float4 v4, float4 u4) {
  if (r >= a.rows || c >= a.n) return;
  float v[4] = {v4.x, v4.y, v4.z, v4.w};
  const float u[4] = {u4.x, u4.y, u4.z, u4.w};
  const T* bias = (const T*)a.bias_dev;
  const T* bias_up = (const T*)a.bias_up_dev;
  const T* res = a.residual_dev ? (const T*)a.residual_dev + r * a.residual_stride : nullptr;
  T* out = (T*)a.out_dev + r * a.out_stride;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < a.n) {
      v[i] = activate<T>(ACT, v[i] + (bias ? to_f32(bias[c + i]) : 0.f));
      if (GATED) v[i] *= u[i] + (bias_up ? to_f32(bias_up[c + i]) : 0.f);
      if (res) v[i] += to_f32(res[c + i]);
    }
  if (sizeof(T) == 4 && c + 4 <= a.n && ((uintptr_t)(out + c) & 15) == 0) {
    *reinterpret_cast<float4*>(out + c) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < a.n) out[c + i] = from_f32<T>(v[i]);
  }
}

template <typename T, bool GATED, int BM>
__global__ void __launch_bounds__(kThreadsSimt, 2) linear_simt_kernel(const pwp_linear_args a, int split, int vec) {
  constexpr int OUT = GATED ? 64 : 128;             // output columns of a tile
  constexpr int TM = BM / 16;                       // rows per thread: 8 or 2
  constexpr int LX = BM * BK / 4 / kThreadsSimt > 0 ? BM * BK / 4 / kThreadsSimt : 1, LW = BN * BK / 4 / kThreadsSimt;
  extern __shared__ __align__(16) float sm[];
  float* xs = sm;                                   // [2][BK][BM + 4]
  float* ws = sm + 2 * BK * (BM + 4);               // [2][BK][BN + 4]
  const int rank = (int)(blockIdx.x % split);
  const long long tile = blockIdx.x / split;
  const int tn = (a.n + OUT - 1) / OUT;
  const long long r0 = tile / tn * BM;
  const int c0 = (int)(tile % tn) * OUT;
  const int nk = (a.k + BK - 1) / BK;
  const int kt0 = (int)((long long)nk * rank / split), kt1 = (int)((long long)nk * (rank + 1) / split);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* x = (const T*)a.x_dev;

  // this thread's pieces of the two tiles: piece i is row id / 4, columns 4 (id % 4)..
  float4 gx[LX], gw[LW];
  auto fetch = [&](int kt) {
#pragma unroll
    for (int i = 0; i < LX; ++i) {
      const int id = threadIdx.x + i * kThreadsSimt, row = id >> 2, k = kt * BK + 4 * (id & 3);
      gx[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < BM && r0 + row < a.rows && k < a.k) gx[i] = load4(x + (r0 + row) * a.x_stride + k, a.k - k, vec & 1);
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int id = threadIdx.x + i * kThreadsSimt, row = id >> 2, k = kt * BK + 4 * (id & 3);
      const bool up = GATED && row >= 64;
      const int c = c0 + (up ? row - 64 : row);
      const T* w = up ? (const T*)a.w_up_dev + (long long)c * a.w_up_stride : (const T*)a.w_dev + (long long)c * a.w_stride;
      gw[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < a.n && k < a.k) gw[i] = load4(w + k, a.k - k, vec & 2);
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < LX; ++i) {
      const int id = threadIdx.x + i * kThreadsSimt, row = id >> 2, k = 4 * (id & 3);
      if (row < BM) {
        float* d = xs + (b * BK + k) * (BM + 4) + row;
        d[0] = gx[i].x, d[BM + 4] = gx[i].y, d[2 * (BM + 4)] = gx[i].z, d[3 * (BM + 4)] = gx[i].w;
      }
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int id = threadIdx.x + i * kThreadsSimt, row = id >> 2, k = 4 * (id & 3);
      float* d = ws + (b * BK + k) * (BN + 4) + row;
      d[0] = gw[i].x, d[BN + 4] = gw[i].y, d[2 * (BN + 4)] = gw[i].z, d[3 * (BN + 4)] = gw[i].w;
    }
  };

  f32x2 acc[TM][4];      // columns 4 tx + {0 1, 2 3}, 64 + 4 tx + {0 1, 2 3}
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = pair(0.f, 0.f);
  if (kt0 < kt1) {
    fetch(kt0);
    put(0);
  }
  __syncthreads();
  for (int kt = kt0; kt < kt1; ++kt) {
    const int b = (kt - kt0) & 1;
    if (kt + 1 < kt1) fetch(kt + 1);
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      const float* xr = xs + (b * BK + k) * (BM + 4);
      const float* wr = ws + (b * BK + k) * (BN + 4) + 4 * tx;
      const float4 w0 = *reinterpret_cast<const float4*>(wr), w1 = *reinterpret_cast<const float4*>(wr + 64);
      const f32x2 wv[4] = {pair(w0.x, w0.y), pair(w0.z, w0.w), pair(w1.x, w1.y), pair(w1.z, w1.w)};
      float xv[TM];
      if (TM == 8) {
        const float4 x0 = *reinterpret_cast<const float4*>(xr + 4 * ty), x1 = *reinterpret_cast<const float4*>(xr + 64 + 4 * ty);
        xv[0] = x0.x, xv[1] = x0.y, xv[TM - 6] = x0.z, xv[TM - 5] = x0.w;
        xv[TM - 4] = x1.x, xv[TM - 3] = x1.y, xv[TM - 2] = x1.z, xv[TM - 1] = x1.w;
      } else {
        const float2 x0 = *reinterpret_cast<const float2*>(xr + 2 * ty);
        xv[0] = x0.x, xv[1] = x0.y;
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const f32x2 xx = pair(xv[i], xv[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fma2(xx, wv[j], acc[i][j]);
      }
    }
    if (kt + 1 < kt1) put(b ^ 1);
    __syncthreads();
  }

  // row i of this thread inside the tile
  auto row_of = [&](int i) { return TM == 8 ? (i < 4 ? 4 * ty + i : 64 + 4 * ty + i - 4) : 2 * ty + i; };
  if (split == 1) {
    with_activation(a.activation, [&](auto act) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const long long r = r0 + row_of(i);
        const float2 p0 = unpair(acc[i][0]), p1 = unpair(acc[i][1]), q0 = unpair(acc[i][2]), q1 = unpair(acc[i][3]);
        const float4 p = make_float4(p0.x, p0.y, p1.x, p1.y), q = make_float4(q0.x, q0.y, q1.x, q1.y);
        finish4<T, GATED, act>(a, r, c0 + 4 * tx, p, q);
        if (!GATED) finish4<T, GATED, act>(a, r, c0 + 64 + 4 * tx, q, q);
      }
    });
    return;
  }
  // Row t of the tile is finished by rank t / per; it gets rank q's sums at sm[q][t % per][column].
  const int per = (BM + split - 1) / split;
  cluster_sync();      // every CTA is done with its tiles of x and W
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(sm) + (uint32_t)(rank * per * BN + 4 * tx) * 4u;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int t = row_of(i), to = t / per;
    const uint32_t dst = map_rank(base + (uint32_t)((t - to * per) * BN) * 4u, (uint32_t)to);
    const float2 p0 = unpair(acc[i][0]), p1 = unpair(acc[i][1]), q0 = unpair(acc[i][2]), q1 = unpair(acc[i][3]);
    remote_store4(dst, make_float4(p0.x, p0.y, p1.x, p1.y));
    remote_store4(dst + 64 * 4, make_float4(q0.x, q0.y, q1.x, q1.y));
  }
  cluster_sync();      // the others' sums are here
  const int mine = min(per, BM - rank * per);
  with_activation(a.activation, [&](auto act) {
    for (int e = threadIdx.x; e < mine * (OUT / 4); e += kThreadsSimt) {
      const int t = e / (OUT / 4), c = 4 * (e % (OUT / 4));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f), u = v;
      for (int q = 0; q < split; ++q) {
        const float4 x4 = *reinterpret_cast<const float4*>(sm + (q * per + t) * BN + c);
        v.x += x4.x, v.y += x4.y, v.z += x4.z, v.w += x4.w;
        if (GATED) {
          const float4 y4 = *reinterpret_cast<const float4*>(sm + (q * per + t) * BN + 64 + c);
          u.x += y4.x, u.y += y4.y, u.z += y4.z, u.w += y4.w;
        }
      }
      finish4<T, GATED, act>(a, r0 + rank * per + t, c0 + c, v, u);
    }
  });
}

long long tiles_of(const pwp_linear_args& a, int bm, int out) {
  return ((a.rows + bm - 1) / bm) * ((a.n + out - 1) / out);
}
// Two CTAs fit an SM; a CTA keeps at least 4 steps of k.
int split_of(const pwp_linear_args& a, long long tiles) {
  const int nk = (a.k + BK - 1) / BK;
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= 2 * kNumSM && nk >= 8 * split) split *= 2;
  return split;
}

template <typename T, bool GATED, int BM>
cudaError_t launch(const pwp_linear_args& a, cudaStream_t s) {
  constexpr int OUT = GATED ? 64 : 128;
  const long long tiles = tiles_of(a, BM, OUT);
  const int split = split_of(a, tiles);
  if (tiles > 0x7fffffffLL / split) return cudaErrorInvalidValue;
  const int work = 2 * BK * (BM + 4 + BN + 4), sums = (BM + kMaxSplit) * BN;
  const int smem = (int)sizeof(float) * (split > 1 && sums > work ? sums : work);
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t ready = on_first_use(attr_done, [&] {
    return cudaFuncSetAttribute(linear_simt_kernel<T, GATED, BM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(float) * (sums > work ? sums : work));
  });
  if (ready != cudaSuccess) return ready;
  auto vec4 = [](const void* p, long long stride) {
    return ((uintptr_t)p % (4 * sizeof(T))) == 0 && stride % 4 == 0;
  };
  const int vec = (vec4(a.x_dev, a.x_stride) ? 1 : 0) |
                  (vec4(a.w_dev, a.w_stride) && (!GATED || vec4(a.w_up_dev, a.w_up_stride)) ? 2 : 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(kThreadsSimt);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_simt_kernel<T, GATED, BM>, a, split, vec);
  count_launches(1);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <typename T, bool GATED>
cudaError_t launch_rows(const pwp_linear_args& a, cudaStream_t s) {
  // 32 rows where more would mostly be padding, or leave most SMs without a tile
  const long long tiles = tiles_of(a, 128, GATED ? 64 : 128);
  return a.rows <= 96 || tiles * split_of(a, tiles) <= kNumSM / 2 ? launch<T, GATED, 32>(a, s) : launch<T, GATED, 128>(a, s);
}

}  // namespace

cudaError_t launch_linear_simt(const pwp_linear_args& a, cudaStream_t s) {
  const bool gated = a.w_up_dev != nullptr;
  if (a.type == PWP_BF16)
    return gated ? launch_rows<__nv_bfloat16, true>(a, s) : launch_rows<__nv_bfloat16, false>(a, s);
  return gated ? launch_rows<float, true>(a, s) : launch_rows<float, false>(a, s);
}

}  // namespace pwp
