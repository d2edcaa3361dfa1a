// Row norms, and the norm and position rotation of queries and keys.  Both are bound by memory:
// each value is read once and written once, sums are fp32, one rounding at the end.
//
// rms_norm: y = x / sqrt(mean(x^2) + eps) * w.  A row is held in registers between its sum of
// squares and its scaling, in 16-byte pieces: by a warp (rows up to 1024 bf16) or by a CTA of 256
// threads (up to 16384 bf16).  Longer rows, and rows that are not 16-byte aligned, are read
// twice.
//
// qk_norm_rope: a token's rot/2 angles position * f_i are formed once per warp in double
// precision -- at position 10^6 an fp32 product would be off by 0.06 rad -- reduced to a turn
// in [-1/2, 1/2] and only then rounded to fp32; every head of the token uses them.  A head is
// held by d / 2N lanes with two vectors of N values each (16, 8 or 4 bytes, as sizes and
// alignment allow), in the half layout the two a rotation pairs, so a pair never leaves its
// thread; a lane meets the same elements, angles and weights in every head and keeps them in
// registers.  Warps are independent: each takes a token's heads a few at a time, the next ones'
// loads in flight meanwhile; several tokens at once when they have few heads; a share of a
// token's heads when there are few tokens.  Other head sizes go through shared memory, a warp
// per head.
//
// Measured.  rms_norm, 32768 rows: 4096 bf16 90 us (5.9 TB/s), 4096 fp32 160 us (6.7); rows that are
// not 16-byte aligned, 4097 bf16 124 us (4.3), and long ones, 16384 x 20000 bf16 552 us (2.4), are
// read twice.  qk_norm_rope, 16384 tokens without and with head norms: 32 + 32 heads of 128 bf16 93
// and 110 us (5.8 and 4.9 TB/s), 32 + 8 bf16 63 and 76 (5.4 and 4.4), 32 + 8 fp32 107 and 124 (6.3 and
// 5.4), 4 + 1 of 96 bf16 19 and 27 (1.7 and 1.2), 4 + 1 of 96 fp32 20 and 35 (3.2 and 1.8).  With few heads
// a warp's chain of position, angle, sine and one round of heads bounds it, with norms the sums
// over a head's lanes, one shuffle after another.
#include "block_ops.cuh"

namespace pwp {
namespace {

constexpr int kNormThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const T* x, long long xs, int width,
                                                                const T* __restrict__ w, float eps, T* out,
                                                                long long os) {
  __shared__ float part[kNormThreads / 32];
  pdl_enter();
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
  const float r = rsqrtf(sum / (float)width + eps);
  for (int i = threadIdx.x; i < width; i += kNormThreads) {
    const float v = to_f32(xr[i]) * r;
    yr[i] = from_f32<T>(w ? v * to_f32(w[i]) : v);
  }
}

// N values of T as one load, in fp32 and back
template <int BYTES>
struct Raw;
template <>
struct Raw<16> { typedef uint4 type; };
template <>
struct Raw<8> { typedef uint2 type; };
template <>
struct Raw<4> { typedef uint32_t type; };
template <typename T, int N>
struct Vec {
  typedef typename Raw<N * (int)sizeof(T)>::type raw;
  static constexpr int WORDS = N * (int)sizeof(T) / 4;
  __device__ static __forceinline__ void unpack(const raw& u, float* v) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
  __device__ static __forceinline__ raw pack(const float* v) {
    raw u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if (sizeof(T) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = __float_as_uint(v[i]);
      }
    }
    return u;
  }
};
template <typename T>
using Vec16 = Vec<T, 16 / (int)sizeof(T)>;

// Rows of `nv` 16-byte vectors, THREADS threads (a warp or the CTA) to a row, VPT vectors a
// thread.
template <typename T, int THREADS, int VPT>
__global__ void __launch_bounds__(kNormThreads) rms_norm_vec_kernel(const T* x, long long xs, long long rows, int nv,
                                                                    const T* __restrict__ w, float eps, T* out,
                                                                    long long os) {
  using V = Vec16<T>;
  constexpr int VN = 16 / (int)sizeof(T);
  __shared__ float part[kNormThreads / 32];
  const long long r = (long long)blockIdx.x * (kNormThreads / THREADS) + threadIdx.x / THREADS;
  const int t = threadIdx.x % THREADS;
  pdl_enter();
  if (r >= rows) return;      // whole warps, and only where a row is a warp's
  const uint4* xr = reinterpret_cast<const uint4*>(x + r * xs);
  uint4 u[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * THREADS < nv) u[i] = xr[t + i * THREADS];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * THREADS < nv) {
      float v[VN];
      V::unpack(u[i], v);
#pragma unroll
      for (int k = 0; k < VN; ++k) sum += v[k] * v[k];
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (THREADS > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) sum += part[i];
  }
  const float inv = rsqrtf(sum / (float)(nv * VN) + eps);
  const uint4* wr = reinterpret_cast<const uint4*>(w);
  uint4* yr = reinterpret_cast<uint4*>(out + r * os);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * THREADS < nv) {
      float v[VN];
      V::unpack(u[i], v);
#pragma unroll
      for (int k = 0; k < VN; ++k) v[k] *= inv;
      if (w) {
        float wv[VN];
        V::unpack(wr[t + i * THREADS], wv);
#pragma unroll
        for (int k = 0; k < VN; ++k) v[k] *= wv[k];
      }
      yr[t + i * THREADS] = V::pack(v);
    }
}

constexpr int kRopeWarps = 8;

// Cosine and sine of position * f, both times `factor`.  The reduced angle has a head in fp32,
// whose sine and cosine sincospif gives, and a rest of up to 2^-26 turns, which would move them by
// up to 2^-23.3: they are turned by it to first order (the next term is below 2^-47).
__device__ __forceinline__ float2 turn_of(long long position, double f, float factor) {
  const double t = (double)position * f * 0.15915494309189533577;   // turns
  const double r = t - rint(t);
  const float head = (float)r, rest = (float)(r - (double)head) * 6.28318530717958648f;
  float s, c;
  sincospif(2.f * head, &s, &c);
  return make_float2(fmaf(-s, rest, c) * factor, fmaf(c, rest, s) * factor);
}

template <typename T>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const pwp_rope_args a) {
  extern __shared__ float smem[];
  pdl_enter();
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
      const float r = rsqrtf(sum / (float)d + a.eps);
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

// Cosine and sine for bf16 results: the hardware's approximations on [-pi, pi] are good to
// 2^-20 absolutely, a two-thousandth of the result's half step of the pair.
template <typename T>
__device__ __forceinline__ float2 turn_as(long long position, double f, float factor) {
  return turn_of(position, f, factor);
}
template <>
__device__ __forceinline__ float2 turn_as<__nv_bfloat16>(long long position, double f, float factor) {
  const double t = (double)position * f * 0.15915494309189533577;   // turns
  const float r = (float)(t - rint(t)) * 6.28318530717958648f;
  return make_float2(__cosf(r) * factor, __sinf(r) * factor);
}

constexpr int kRopeBatch = 2;      // heads a lane turns at once, and as many on their way

// How a launch divides the work (host side, run_rope).
struct RopeSplit {
  int lph;           // lanes per head
  int hpt, tpw;      // heads of a token a warp holds at once, and tokens
  int wpt;           // warps per token
};

template <typename T, int N, bool HALF, bool NORM>
__global__ void __launch_bounds__(32 * kRopeWarps, 2) rope_vec_kernel(const pwp_rope_args a, const RopeSplit sp) {
  using V = Vec<T, N>;
  typedef typename V::raw raw;
  extern __shared__ float2 cs_all[];
  const int half = a.rot / 2, heads = a.hq + a.hk;
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);   // this warp among all
  const long long t0 = gw / sp.wpt * sp.tpw;                                       // its first token
  pdl_enter();
  if (t0 >= a.n) return;
  float2* cs = cs_all + (threadIdx.x >> 5) * (sp.tpw * half);
  const int sub = lane / sp.lph, col = lane - sub * sp.lph;      // head slot of the warp, place in the head
  const int tsub = sub / sp.hpt, hsub = sub - tsub * sp.hpt;     // token and head of the slot
  const long long t = t0 + tsub;
  const bool live = sub < sp.hpt * sp.tpw && t < a.n;
  // elements e0 .. e0 + N and e1 .. e1 + N of the head
  const bool turned = col < a.rot / (2 * N);
  const int e0 = HALF && turned ? col * N : col * 2 * N;
  const int e1 = HALF && turned ? e0 + half : e0 + N;

  const T* qi = (const T*)a.q_dev + t * a.q_stride[0];
  const T* ki = (const T*)a.k_dev + t * a.k_stride[0];
  const int step = sp.wpt * sp.hpt;
  raw u[kRopeBatch][2] = {};
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int h = h0 + i * step;
      if (live && h < heads) {
        const T* p = h < a.hq ? qi + h * a.q_stride[1] : ki + (h - a.hq) * a.k_stride[1];
        u[i][0] = *reinterpret_cast<const raw*>(p + e0);
        u[i][1] = *reinterpret_cast<const raw*>(p + e1);
      }
    }
  };
  const int w0 = (int)(gw % sp.wpt) * sp.hpt;      // the warp's first head
  load(w0 + hsub);
  raw wt[2][2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const T* w = (const T*)(i ? a.k_weight_dev : a.q_weight_dev);
    if (NORM && live && w) {
      wt[i][0] = *reinterpret_cast<const raw*>(w + e0);
      wt[i][1] = *reinterpret_cast<const raw*>(w + e1);
    }
  }
  for (int i = lane; i < sp.tpw * half; i += 32) {
    const int q = i / half;
    if (t0 + q < a.n) cs[i] = turn_as<T>(a.positions_dev[t0 + q], a.freqs_dev[i - q * half], a.factor);
  }
  __syncwarp();
  float2 c[N];
#pragma unroll
  for (int k = 0; k < N; ++k) c[k] = turned && live ? cs[tsub * half + (HALF ? e0 : e0 / 2) + k] : make_float2(1.f, 0.f);

  const float inv_d = 1.f / (float)a.d;
  T* qo = (T*)a.q_out_dev + t * a.q_out_stride[0];
  T* ko = (T*)a.k_out_dev + t * a.k_out_stride[0];
  // every lane takes part in the shuffles, so the loop runs on the warp's first head
  for (int g = w0; g < heads; g += kRopeBatch * step) {
    raw r[kRopeBatch][2];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      r[i][0] = u[i][0];
      r[i][1] = u[i][1];
    }
    load(g + hsub + kRopeBatch * step);      // the next heads are on their way while these are turned
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (g + i * step >= heads) break;
      const int h = g + hsub + i * step;
      const bool on = live && h < heads, is_q = h < a.hq;
      float v0[N], v1[N];
      V::unpack(r[i][0], v0);
      V::unpack(r[i][1], v1);
      if (NORM) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) sum += v0[k] * v0[k] + v1[k] * v1[k];
        if ((sp.lph & (sp.lph - 1)) == 0) {
          for (int o = sp.lph >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        } else {
          float all = 0.f;
          for (int k = 0; k < sp.lph; ++k) all += __shfl_sync(0xffffffffu, sum, min(sub * sp.lph + k, 31));
          sum = all;
        }
        if (is_q ? a.q_weight_dev != nullptr : a.k_weight_dev != nullptr) {
          const float inv = rsqrtf(sum * inv_d + a.eps);
          float x0[N], x1[N];
          V::unpack(is_q ? wt[0][0] : wt[1][0], x0);
          V::unpack(is_q ? wt[0][1] : wt[1][1], x1);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            v0[k] = v0[k] * inv * x0[k];
            v1[k] = v1[k] * inv * x1[k];
          }
        }
      }
      if (HALF) {
        if (turned) {
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float p = v0[k], q = v1[k];
            v0[k] = p * c[k].x - q * c[k].y;
            v1[k] = q * c[k].x + p * c[k].y;
          }
        }
      } else if (turned) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          const float p = v0[2 * k], q = v0[2 * k + 1], y = v1[2 * k], z = v1[2 * k + 1];
          v0[2 * k] = p * c[k].x - q * c[k].y;
          v0[2 * k + 1] = q * c[k].x + p * c[k].y;
          v1[2 * k] = y * c[N / 2 + k].x - z * c[N / 2 + k].y;
          v1[2 * k + 1] = z * c[N / 2 + k].x + y * c[N / 2 + k].y;
        }
      }
      if (on) {
        T* p = is_q ? qo + h * a.q_out_stride[1] : ko + (h - a.hq) * a.k_out_stride[1];
        *reinterpret_cast<raw*>(p + e0) = V::pack(v0);
        *reinterpret_cast<raw*>(p + e1) = V::pack(v1);
      }
    }
  }
}

// Grids that the GPU takes at once are scheduled while their predecessor ends (a rotation of 37
// tokens, one after another: 6.1 us, 4.8 this way; a row's norm 4.2, 3.7); larger ones gain nothing.
template <typename... KArgs, typename... Args>
void launch_row_kernel(void (*kernel)(KArgs...), long long grid, int block, size_t smem, cudaStream_t s, Args... args) {
  if (grid <= 2 * kNumSM)
    launch_pdl(kernel, dim3((unsigned)grid), dim3(block), smem, s, args...);
  else
    kernel<<<(unsigned)grid, block, smem, s>>>(args...);
}

template <typename T>
bool aligned16(const void* p, long long stride) {
  return ((uintptr_t)p & 15) == 0 && (stride * (long long)sizeof(T)) % 16 == 0;
}

template <typename T>
cudaError_t run_rms_norm(const T* x, long long rows, int width, long long xs, const T* w, float eps, T* out,
                         long long os, cudaStream_t s) {
  constexpr int VN = 16 / (int)sizeof(T);
  if (rows == 1) xs = os = width;      // a single row: its stride is never used
  const int nv = width / VN;
  count_launches(1);
  if (width % VN == 0 && aligned16<T>(x, xs) && aligned16<T>(out, os) && aligned16<T>(w, 0) && nv <= 8 * kNormThreads) {
#define PWP_NORM(TH, VPT)                                                                                         \
  launch_row_kernel(rms_norm_vec_kernel<T, TH, VPT>, (rows + kNormThreads / TH - 1) / (kNormThreads / TH), kNormThreads, \
                    0, s, x, xs, rows, nv, w, eps, out, os)
    if (nv <= 32) PWP_NORM(32, 1);
    else if (nv <= 64) PWP_NORM(32, 2);
    else if (nv <= 128) PWP_NORM(32, 4);
    else if (nv <= 256) PWP_NORM(256, 1);
    else if (nv <= 512) PWP_NORM(256, 2);
    else if (nv <= 1024) PWP_NORM(256, 4);
    else PWP_NORM(256, 8);
#undef PWP_NORM
  } else {
    launch_row_kernel(rms_norm_kernel<T>, rows, kNormThreads, 0, s, x, xs, width, w, eps, out, os);
  }
  return cudaGetLastError();
}

// Whether a head can be held as pairs of N-value vectors.
template <typename T, int N>
bool rope_fits(const pwp_rope_args& a) {
  const long long bytes = N * (long long)sizeof(T);
  auto ok = [&](const void* p, long long stride) {
    return ((uintptr_t)p % bytes) == 0 && (stride * (long long)sizeof(T)) % bytes == 0;
  };
  if (a.d % (2 * N) != 0 || a.rot % (2 * N) != 0 || a.d > 32 * 2 * N) return false;
  for (int i = 0; i < 2; ++i) {
    if (a.hq && !(ok(a.q_dev, a.q_stride[i]) && ok(a.q_out_dev, a.q_out_stride[i]))) return false;
    if (a.hk && !(ok(a.k_dev, a.k_stride[i]) && ok(a.k_out_dev, a.k_out_stride[i]))) return false;
  }
  return ok(a.q_weight_dev, 0) && ok(a.k_weight_dev, 0);
}

template <typename T, int N>
void launch_rope(const pwp_rope_args& a, cudaStream_t s) {
  const int heads = a.hq + a.hk;
  RopeSplit sp;
  sp.lph = a.d / (2 * N);
  const int hpw = 32 / sp.lph;
  sp.hpt = heads < hpw ? heads : hpw;
  sp.tpw = hpw / sp.hpt;
  // Warps per token: one where the tokens fill the GPU's warps, more, for latency, where they
  // do not.
  const int groups = (heads + sp.hpt - 1) / sp.hpt;
  sp.wpt = 1;
  while (sp.wpt * kRopeBatch < groups && a.n * sp.wpt < 16 * kNumSM) sp.wpt *= 2;
  const long long warps = (a.n + sp.tpw - 1) / sp.tpw * sp.wpt;
  const long long grid = (warps + kRopeWarps - 1) / kRopeWarps;
  const size_t smem = sizeof(float2) * (size_t)(a.rot / 2) * sp.tpw * kRopeWarps;   // at most 16 KB
  const bool norm = a.q_weight_dev || a.k_weight_dev;
  auto kernel = a.layout == PWP_ROPE_HALF
                    ? (norm ? rope_vec_kernel<T, N, true, true> : rope_vec_kernel<T, N, true, false>)
                    : (norm ? rope_vec_kernel<T, N, false, true> : rope_vec_kernel<T, N, false, false>);
  launch_row_kernel(kernel, grid, 32 * kRopeWarps, smem, s, a, sp);
}

template <typename T>
cudaError_t run_rope(const pwp_rope_args& a, cudaStream_t s) {
  constexpr int N = 16 / (int)sizeof(T);
  count_launches(1);
  if (rope_fits<T, N>(a)) {
    launch_rope<T, N>(a, s);
  } else if (rope_fits<T, N / 2>(a)) {
    launch_rope<T, N / 2>(a, s);
  } else if (N == 8 && rope_fits<T, 2>(a)) {
    launch_rope<T, 2>(a, s);
  } else {
    const size_t smem = sizeof(float) * (size_t)(a.rot + kRopeWarps * a.d);   // at most 36 KB (d <= 1024)
    launch_row_kernel(rope_kernel<T>, a.n, 32 * kRopeWarps, smem, s, a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(const void* x, int type, long long rows, int width, long long xs, const void* w, float eps,
                            void* out, long long os, cudaStream_t s) {
  typedef __nv_bfloat16 bf16;
  return type == PWP_BF16
             ? run_rms_norm<bf16>((const bf16*)x, rows, width, xs, (const bf16*)w, eps, (bf16*)out, os, s)
             : run_rms_norm<float>((const float*)x, rows, width, xs, (const float*)w, eps, (float*)out, os, s);
}

cudaError_t launch_qk_norm_rope(const pwp_rope_args& a, cudaStream_t s) {
  return a.type == PWP_BF16 ? run_rope<__nv_bfloat16>(a, s) : run_rope<float>(a, s);
}

}  // namespace pwp
