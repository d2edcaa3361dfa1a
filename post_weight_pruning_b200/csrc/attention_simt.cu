// Attention within packed sequences on the CUDA cores: fp32 tensors, and bf16 ones whose
// bases, strides or head sizes the tensor-core kernel's copies cannot take.
//
// o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = exp(scale q_i k_j - m_i), in one pass over the keys
// with the running maximum m_i and sum (both fp32) corrected when the maximum grows.  One CTA
// of 256 threads takes 64 queries of one head at a time; 32 keys and values at a time go through shared
// memory as fp32.  Four threads share a query: each forms the scores of 8 keys and keeps a
// quarter of the output row.  A query's loops end at its last visible key, so what lies
// behind it (another sequence, a later token) is never multiplied.  Bound by the reads of
// shared memory: 2048 fp32 tokens, 40 heads of 128 on 8 key heads, 3.0 ms, 14 TFLOP/s; bf16, whose
// values are loaded one at a time: 3 x 1000 tokens, 8 heads on 2, of 256 1.24 ms (10 TFLOP/s), of
// 136 1.23 ms.
#include "block_ops.cuh"

namespace pwp {
namespace {

constexpr int QT = 64, KT = 32;
constexpr int kCtas = 16 * kNumSM;

template <typename T, int D>
__global__ void __launch_bounds__(256) attention_simt_kernel(const pwp_attention_args a, int vec) {
  constexpr int LD = D + 4;
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                 // QT x LD
  float* ks = qs + QT * LD;       // KT x LD
  float* vs = ks + KT * LD;       // KT x LD
  float* ps = vs + KT * LD;       // QT x (KT + 1)
  SeqScan scan;
  // items: the tiles with the heads running fastest
  for (long long item = blockIdx.x;; item += gridDim.x) {
    const int h = (int)(item % a.hq), hk = h / (a.hq / a.hk);
    SeqTile tile;
    bool bad = false;
    const bool have = find_seq_tile(a.cu_seqlens_dev, a.nseq, a.n, QT, (int)(item / a.hq), scan, tile, bad);
    if (bad && a.stats_dev && threadIdx.x == 0) set_error(a.stats_dev, PWP_EINVAL, kSiteAttention);
    if (!have) return;
    __syncthreads();      // the last item's tiles have been read
    const T* q = (const T*)a.q_dev + (long long)(tile.begin + tile.first) * a.q_stride[0] + h * a.q_stride[1];
    const T* k = (const T*)a.k_dev + (long long)tile.begin * a.k_stride[0] + hk * a.k_stride[1];
    const T* v = (const T*)a.v_dev + (long long)tile.begin * a.v_stride[0] + hk * a.v_stride[1];
    T* out = (T*)a.out_dev + (long long)(tile.begin + tile.first) * a.out_stride[0] + h * a.out_stride[1];
    const int rows = min(QT, tile.len - tile.first);
    for (int i = threadIdx.x; i < QT * D; i += 256) {
      const int r = i / D, c = i % D;
      qs[r * LD + c] = r < rows && c < a.d ? to_f32(q[r * a.q_stride[0] + c]) * a.scale : 0.f;
    }
    const int r = threadIdx.x >> 2, x = threadIdx.x & 3;
    const int seen = r < rows ? (a.causal ? tile.first + r + 1 : tile.len) : 0;   // keys this query sees
    const int last = a.causal ? tile.first + rows : tile.len;                    // keys any query of the tile sees
    float m = -INFINITY, l = 0.f, o[D / 4];
#pragma unroll
    for (int i = 0; i < D / 4; ++i) o[i] = 0.f;
    for (int k0 = 0; k0 < last; k0 += KT) {
      __syncthreads();
      if (sizeof(T) == 4 && vec) {       // four values at a time, the block's loads in flight together
        constexpr int P = KT * D / 4 / 256;
        float4 kv[P], vv[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int i = threadIdx.x + 256 * p, j = i / (D / 4), c = 4 * (i % (D / 4));
          kv[p] = vv[p] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + j < last && c < a.d) {
            kv[p] = *reinterpret_cast<const float4*>(k + (long long)(k0 + j) * a.k_stride[0] + c);
            vv[p] = *reinterpret_cast<const float4*>(v + (long long)(k0 + j) * a.v_stride[0] + c);
          }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int i = threadIdx.x + 256 * p, j = i / (D / 4), c = 4 * (i % (D / 4));
          *reinterpret_cast<float4*>(ks + j * LD + c) = kv[p];
          *reinterpret_cast<float4*>(vs + j * LD + c) = vv[p];
        }
      } else {
        for (int i = threadIdx.x; i < KT * D; i += 256) {
          const int j = i / D, c = i % D;
          const bool in = k0 + j < last && c < a.d;
          ks[j * LD + c] = in ? to_f32(k[(long long)(k0 + j) * a.k_stride[0] + c]) : 0.f;
          vs[j * LD + c] = in ? to_f32(v[(long long)(k0 + j) * a.v_stride[0] + c]) : 0.f;
        }
      }
      __syncthreads();
      float s[8] = {};
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        const float4 qv = *reinterpret_cast<const float4*>(qs + r * LD + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 kv = *reinterpret_cast<const float4*>(ks + (x + 4 * i) * LD + c);
          s[i] += qv.x * kv.x + qv.y * kv.y + qv.z * kv.z + qv.w * kv.w;
        }
      }
      float mx = m;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (k0 + x + 4 * i >= seen) s[i] = -INFINITY;
        mx = fmaxf(mx, s[i]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float base = mx == -INFINITY ? 0.f : mx;      // no visible key so far
      const float fix = expf(m - base);
      m = mx;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool on = k0 + x + 4 * i < seen;
        const float p = on ? expf(s[i] - base) : 0.f;
        ps[r * (KT + 1) + x + 4 * i] = p;
        sum += p;
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      l = l * fix + sum;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) o[i] *= fix;
      __syncwarp();
      const int nj = min(KT, seen - k0);
      for (int j = 0; j < nj; ++j) {
        const float p = ps[r * (KT + 1) + j];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const float4 vv = *reinterpret_cast<const float4*>(vs + j * LD + 4 * x + 16 * i);
          o[4 * i] += p * vv.x;
          o[4 * i + 1] += p * vv.y;
          o[4 * i + 2] += p * vv.z;
          o[4 * i + 3] += p * vv.w;
        }
      }
      __syncwarp();
    }
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < D / 4; ++i) {
        const int c = 4 * x + 16 * (i / 4) + (i & 3);
        if (c < a.d) out[r * a.out_stride[0] + c] = from_f32<T>(o[i] / l);
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch(const pwp_attention_args& a, cudaStream_t s) {
  constexpr int smem = (int)sizeof(float) * ((QT + 2 * KT) * (D + 4) + QT * (KT + 1));
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t ready = on_first_use(attr_done, [] {
    return cudaFuncSetAttribute(attention_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (ready != cudaSuccess) return ready;
  // No sequence's tiles are known here: an upper bound of their number.  CTAs past kCtas take the
  // next tiles in turn, or a batch of very many sequences would be searched once for each of them.
  const long long items = (a.n / QT + a.nseq) * a.hq;
  const long long grid = items < kCtas ? items : kCtas;
  auto even = [&](const void* p, const int64_t* st) { return ((uintptr_t)p & 15) == 0 && ((st[0] | st[1]) & 3) == 0; };
  const int vec = a.type == PWP_FP32 && (a.d & 3) == 0 && even(a.k_dev, a.k_stride) && even(a.v_dev, a.v_stride);
  attention_simt_kernel<T, D><<<(unsigned)grid, 256, smem, s>>>(a, vec);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const pwp_attention_args& a, cudaStream_t s) {
  if (a.d <= 64) return launch<T, 64>(a, s);
  if (a.d <= 128) return launch<T, 128>(a, s);
  return launch<T, 256>(a, s);
}

}  // namespace

cudaError_t launch_attention_simt(const pwp_attention_args& a, cudaStream_t s) {
  return a.type == PWP_BF16 ? launch_type<__nv_bfloat16>(a, s) : launch_type<float>(a, s);
}

}  // namespace pwp
