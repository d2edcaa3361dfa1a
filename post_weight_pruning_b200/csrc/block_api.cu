// C ABI of the decoder block's forward operators: argument checks and the choice of kernel.
// The declarations and their contracts are in include/pwp.h.
#include "block_ops.cuh"

using namespace pwp;

namespace {

bool valid_type(int32_t t) { return t == PWP_BF16 || t == PWP_FP32; }
bool finite_f(float x) { return x - x == 0.f; }
// the kernels' atomics on a record need its own alignment
bool valid_stats(const pwp_stats* st) { return ((uintptr_t)st & (alignof(pwp_stats) - 1)) == 0; }
pwp_status status_of(cudaError_t e) { return e == cudaSuccess ? PWP_OK : PWP_ECUDA; }

}  // namespace

extern "C" {

pwp_status pwp_rms_norm(const void* x, int32_t type, int64_t rows, int32_t width, int64_t xs, const void* w, float eps,
                        void* out, int64_t os, void* stream) {
  if (!valid_type(type) || rows < 0 || rows > 0x7fffffffLL || width < 1 || width > 65536 || xs < 0 || os < 0 ||
      !(eps >= 0.f) || !finite_f(eps))
    return PWP_EINVAL;
  if (rows == 0) return PWP_OK;
  if (!x || !out || (rows > 1 && os < width)) return PWP_EINVAL;
  return status_of(launch_rms_norm(x, type, rows, width, xs, w, eps, out, os, (cudaStream_t)stream));
}

pwp_status pwp_qk_norm_rope(const pwp_rope_args* a, void* stream) {
  if (!a || !valid_type(a->type) || a->n < 0 || a->n > 0x7fffffffLL || a->hq < 0 || a->hk < 0 || a->d < 1 ||
      a->d > 1024 || a->hq > 65536 || a->hk > 65536 || a->rot < 0 || a->rot > a->d || (a->rot & 1) ||
      (a->layout != PWP_ROPE_HALF && a->layout != PWP_ROPE_INTERLEAVED) || !(a->eps >= 0.f) || !finite_f(a->eps) ||
      !finite_f(a->factor))
    return PWP_EINVAL;
  for (int i = 0; i < 2; ++i)
    if (a->q_stride[i] < 0 || a->k_stride[i] < 0 || a->q_out_stride[i] < 0 || a->k_out_stride[i] < 0) return PWP_EINVAL;
  if (a->n == 0 || a->hq + a->hk == 0) return PWP_OK;
  if ((a->hq > 0 && (!a->q_dev || !a->q_out_dev)) || (a->hk > 0 && (!a->k_dev || !a->k_out_dev)) ||
      (a->rot > 0 && (!a->positions_dev || !a->freqs_dev)))
    return PWP_EINVAL;
  return status_of(launch_qk_norm_rope(*a, (cudaStream_t)stream));
}

static bool valid_attention(const pwp_attention_args* a) {
  if (!a || !valid_type(a->type) || a->n < 0 || a->nseq < 0 || a->hq < 1 || a->hk < 1 || a->hq % a->hk != 0 ||
      a->d < 1 || a->d > 256 || a->n > 0x7fffffffLL / a->hq || a->nseq > (1 << 24) || !finite_f(a->scale) ||
      !valid_stats(a->stats_dev))
    return false;
  for (int i = 0; i < 2; ++i)
    if (a->q_stride[i] < 0 || a->k_stride[i] < 0 || a->v_stride[i] < 0 || a->out_stride[i] < 0) return false;
  return true;
}

size_t pwp_attention_workspace_bytes(const pwp_attention_args* a) {
  return valid_attention(a) && a->n > 0 && a->nseq > 0 ? attention_workspace(*a) : 0;
}

pwp_status pwp_attention(const pwp_attention_args* a, void* stream) {
  if (!valid_attention(a)) return PWP_EINVAL;
  if (a->n == 0 || a->nseq == 0) return PWP_OK;
  if (!a->q_dev || !a->k_dev || !a->v_dev || !a->out_dev || !a->cu_seqlens_dev) return PWP_EINVAL;
  if (a->ws_dev && ((uintptr_t)a->ws_dev & 255) != 0) return PWP_EWORKSPACE;
  bool used = false;
  const cudaError_t e = launch_attention_tc(*a, (cudaStream_t)stream, &used);
  return status_of(used || e != cudaSuccess ? e : launch_attention_simt(*a, (cudaStream_t)stream));
}

static bool valid_linear(const pwp_linear_args* a) {
  if (!a || !valid_type(a->type) || a->rows < 0 || a->rows > 0x7fffffffLL || a->k < 1 || a->n < 1 ||
      a->k >= (1 << 24) || a->n >= (1 << 24) || a->activation < PWP_ACT_NONE || a->activation > PWP_ACT_GELU_TANH ||
      a->x_stride < 0 || a->w_stride < 0 || a->w_up_stride < 0 || a->residual_stride < 0 || a->out_stride < 0 ||
      (!a->w_up_dev && a->bias_up_dev) || !valid_stats(a->stats_dev))
    return false;
  return a->rows == 0 || (a->x_dev && a->w_dev && a->out_dev && (a->rows == 1 || a->out_stride >= a->n));
}

size_t pwp_linear_workspace_bytes(const pwp_linear_args* a) {
  return valid_linear(a) && a->rows > 0 ? linear_align_bytes(*a) : 0;
}

pwp_status pwp_linear(const pwp_linear_args* a, void* stream) {
  if (!valid_linear(a)) return PWP_EINVAL;
  if (a->rows == 0) return PWP_OK;
  if (a->ws_dev && ((uintptr_t)a->ws_dev & 255) != 0) return PWP_EWORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  pwp_linear_args b = *a;
  cudaError_t e = cudaSuccess;
  const size_t need = linear_align_bytes(*a);
  if (need && a->ws_dev && a->ws_bytes >= need) e = launch_linear_align(b, s);
  bool used = false;
  if (e == cudaSuccess) e = launch_linear_tc(b, s, &used);
  return status_of(used || e != cudaSuccess ? e : launch_linear_simt(*a, s));
}

}  // extern "C"
