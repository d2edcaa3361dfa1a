"""Forward pass of a decoder block on calibration tokens: the operators that turn a block's
hidden states into the activations its layers are pruned with.

``rms_norm``, ``qk_norm_rope``, ``attention``, ``linear`` and ``gated_linear`` marshal their
arguments to the C entry points of the same names (include/pwp.h), the usual calls in C++
(csrc/fastcall.cpp), all others here; ``rope_frequencies`` forms
the rotation's frequencies.  ``block_forward`` runs them as a decoder block and returns every
distinct layer input beside the block's output, and ``prune_decoder_block`` prunes the block
with those inputs and passes the hidden states through the pruned layers.

They run on the device of their tensors and on the given or the current stream of that device,
and nothing is kept between calls.  The operators do not synchronise; ``block_forward`` copies the
sequences' offsets, and positions that are not given, from the host and waits for each copy.
They compute a forward pass only: an input that requires a gradient is refused while
gradients are recorded, and one that carries a forward-mode tangent always.
"""
from __future__ import annotations

import ctypes
import math
import struct

import numpy as np

import post_weight_pruning_b200 as _pwp

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
LAYOUTS = {"half": 0, "interleaved": 1}
# the layer input each projection of a decoder block reads
FEEDS = {"q_proj": "attn_in", "k_proj": "attn_in", "v_proj": "attn_in", "o_proj": "o_in", "gate_proj": "mlp_in",
         "up_proj": "mlp_in", "down_proj": "down_in"}


# pwp_rope_args, pwp_attention_args and pwp_linear_args field by field, packed in one call: a
# small operator's time is mostly its host side
ROPE_ARGS = struct.Struct("@4P8q4Pq6i2f")
ATTENTION_ARGS = struct.Struct("@4P8q2Pq6ifPN")
LINEAR_ARGS = struct.Struct("@7P5qPq4iPN")

SIGNATURES = {
    "pwp_rms_norm": (_i32, [_vp, _i32, _i64, _i32, _i64, _vp, _f32, _vp, _i64, _vp]),
    "pwp_qk_norm_rope": (_i32, [ctypes.c_char_p, _vp]),
    "pwp_attention": (_i32, [ctypes.c_char_p, _vp]),
    "pwp_attention_workspace_bytes": (ctypes.c_size_t, [ctypes.c_char_p]),
    "pwp_linear": (_i32, [ctypes.c_char_p, _vp]),
    "pwp_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.c_char_p]),
}


_loaded = _current_device = None


def _torch():
    """torch, imported at the first call (looking it up again costs a small operator's call
    as much as its launch checks)."""
    global _loaded, _current_device
    if _loaded is None:
        _loaded = _pwp._torch()
        _current_device = _loaded._C._cuda_getDevice
    return _loaded


class _NoFastCalls:
    """In the place of _fastcall where it is not built (or for another PyTorch): takes no call."""
    rms_norm = qk_norm_rope = attention = linear = staticmethod(lambda *a: None)


_fast = None


def _fast_calls():
    """_fastcall: the usual calls' checks and marshalling in C++ (the same C entry points).  It
    returns None for what it does not take, which the operators below then check and run."""
    global _fast
    if _fast is None:
        torch = _torch()
        try:
            from . import _fastcall
            _fast = _fastcall if torch.__version__.split("+")[0] == _fastcall.torch_version else _NoFastCalls
        except ImportError:
            _fast = _NoFastCalls
    return _fast


# ------------------------------------------------------------------- argument checks

def _away(x, stream):
    """Whether an operator on `x` has to change the current device or stream first."""
    try:
        dev = x.get_device()
    except AttributeError:
        raise TypeError(f"tensor expected, got {type(x).__name__}") from None
    if stream is not None:
        if dev >= 0 and stream.device_index != dev:
            raise ValueError(f"stream of device {stream.device_index}, tensors on device {dev}")
        return True
    return dev >= 0 and dev != (_current_device or _torch()._C._cuda_getDevice)()


def _at(x, stream):
    """The context of an operator that is away: the given stream, or the device of `x`."""
    return _pwp._stream_ctx(stream) if stream is not None else _torch().cuda.device(x.device)


def _on_gpu(t):
    return t.is_cuda


def _stream_of(dev):
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _type_code(x, name, dims):
    """PWP_BF16 or PWP_FP32 of an operator's first tensor, whose form is checked."""
    torch = _torch()
    code = _pwp.BF16 if x.dtype is torch.bfloat16 else _pwp.FP32 if x.dtype is torch.float32 else None
    if code is None:
        _pwp._dtype_code(x)       # raises
    if x.dim() != dims:
        raise ValueError(f"{name}: {dims} dimensions expected, got shape {tuple(x.shape)}")
    if not _on_gpu(x):
        raise ValueError(f"{name}: CUDA tensors expected")
    if x.stride(-1) != 1 and x.shape[-1] > 1:
        raise ValueError(f"{name}: elements of the last dimension must be contiguous")
    return code


def _check_tensor(t, name, shape, like, dtype=None):
    """`t` on the device of `like`, of its element type (or `dtype`) and of `shape`, with
    contiguous elements in its last dimension."""
    dtype = dtype or like.dtype
    if t.dtype is dtype and t.shape == shape and t.get_device() == like.get_device() and t.stride(-1) == 1:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != like.device:
        raise ValueError(f"{name}: on {t.device}, the first tensor on {like.device}")
    if t.shape[-1] > 1:
        raise ValueError(f"{name}: elements of the last dimension must be contiguous")


def _overlap(a, b):
    """Whether the memory of two tensors may have a byte in common.  Slices that interleave
    (heads or columns of one packed buffer) are told apart by their places within a stride
    they share."""
    sizes = [t.element_size() for t in (a, b)]
    dims = [[(st * e, n) for st, n in zip(t.stride(), t.shape) if n != 1] for t, e in zip((a, b), sizes)]
    if any(n == 0 for ds in dims for _, n in ds):
        return False
    reach = [sum(st * (n - 1) for st, n in ds) + e for ds, e in zip(dims, sizes)]
    gap = b.data_ptr() - a.data_ptr()
    if gap >= reach[0] or -gap >= reach[1]:
        return False
    for pitch in {st for st, _ in dims[0]} & {st for st, _ in dims[1]}:
        if pitch == 0 or any(st > pitch and st % pitch for ds in dims for st, _ in ds):
            continue
        inner = [sum(st * (n - 1) for st, n in ds if st < pitch) + e for ds, e in zip(dims, sizes)]
        if inner[0] <= gap % pitch and gap % pitch + inner[1] <= pitch:
            return False
    return True


def _check_out(t, name, shape, like, others, same=None):
    """An output given by the caller: no two of its elements in one place, and apart from the
    `others`, the tensors the call reads or writes elsewhere.  It may be `same`, the tensor whose
    every element is read where the output's is written, element for element; a tensor given a
    second time, as one of the others, is read in other places too."""
    _check_tensor(t, name, shape, like)
    reach = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride < reach:
            raise ValueError(f"{name}: elements overlap (shape {tuple(t.shape)}, strides {t.stride()})")
        reach = stride * size
    if same is not None and same.data_ptr() == t.data_ptr() and \
            all(n == 1 or i == j for n, i, j in zip(shape, same.stride(), t.stride())):
        same = None
    for x in (*others, same):
        if x is not None and _overlap(t, x):
            raise ValueError(f"{name}: overlaps a tensor the call reads or writes")
    _check_plain(t)


def _check_plain(*ts):
    """Refuses tensors that are more than their memory: with a gradient or a forward-mode tangent to
    carry on, or a negation that is still to be done."""
    torch = _torch()
    recording, forward = torch.is_grad_enabled(), torch.autograd.forward_ad
    dual = forward._current_level >= 0
    for t in ts:
        if t is None:
            continue
        if (recording and t.requires_grad) or (dual and forward.unpack_dual(t).tangent is not None):
            raise ValueError("the operators compute a forward pass only: call them under torch.no_grad() "
                             "or on detached tensors, without forward-mode tangents")
        if t.is_neg():
            raise ValueError("a negated view (of a conjugate's imaginary part): resolve_neg() gives its values")


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _stats_ptr(stats, like):
    if stats is None:
        return 0
    _check_tensor(stats, "stats", (ctypes.sizeof(_pwp.Stats),), like, _torch().uint8)
    if stats.data_ptr() % 8:
        raise ValueError("stats: a record at a multiple of 8 bytes expected (new_stats gives one)")
    return stats.data_ptr()


def _call(name, args, dev):
    st = getattr(_pwp.lib(), name)(args, _stream_of(dev))
    if st:
        raise _pwp.PwpError(st, name)


# ------------------------------------------------------------------- operators

def rms_norm(x, weight=None, *, eps=1e-5, out=None, stream=None):
    """x / sqrt(mean(x^2) + eps) * weight over the rows of x ([n, width], bf16 or fp32;
    rows may be strided).  weight: [width] or None.  out: None, a tensor like x, or x itself."""
    if out is None and stream is None:
        y = (_fast or _fast_calls()).rms_norm(x, weight, eps)
        if y is not None:
            return y
    if _away(x, stream):
        with _at(x, stream):
            return rms_norm(x, weight, eps=eps, out=out)
    code = _type_code(x, "x", 2)
    n, width = shape = x.shape
    if width < 1 or width > 65536:
        raise ValueError(f"x: width {width}, 1 to 65536 expected")
    if weight is not None:
        _check_tensor(weight, "weight", (width,), x)
    if not 0 <= eps < math.inf:
        raise ValueError(f"eps: {eps}")
    _check_plain(x, weight)
    if out is None:
        out = x.new_empty(shape)
    else:
        _check_out(out, "out", shape, x, (weight,), x)
    if n:
        st = _pwp.lib().pwp_rms_norm(x.data_ptr(), code, n, width, x.stride(0), _ptr(weight), eps, out.data_ptr(),
                                     out.stride(0), _stream_of(x.get_device()))
        if st:
            raise _pwp.PwpError(st, "pwp_rms_norm")
    return out


def rope_frequencies(rot, *, base=10000.0, scaling=None, device="cuda"):
    """(frequencies, factor) of the rotation of `rot` elements (even) for qk_norm_rope: a
    double-precision tensor [rot / 2] on `device`, f_i = base^(-2 i / rot), and the number
    cosine and sine are multiplied by.  scaling stretches them to longer contexts:
      None                                   as they are, factor 1
      {"type": "linear", "factor": s}        f_i / s: positions closer together
      {"type": "base", "factor": s}          the base times s^(rot / (rot - 2)): the slowest
                                             pair s times slower, the fastest unchanged
      {"type": "bands", "factor": s, "low_freq_factor": l, "high_freq_factor": h,
       "original_max_positions": n0}         pairs that make fewer than l turns over n0
                                             positions slowed by s, those with more than h
                                             unchanged, linear between (in turns)
      {"type": "yarn", "factor": s, "original_max_positions": n0, "beta_fast": 32.0,
       "beta_slow": 1.0}                     the same idea with the ramp linear in the pair's
                                             index, between the pairs that make beta_fast and
                                             beta_slow turns; factor 0.1 ln s + 1 (1 for s up to 1)"""
    torch = _torch()
    rot = int(rot)
    if rot < 0 or rot % 2 or not 0 < base < math.inf:
        raise ValueError(f"rot even and base > 0 expected, got {rot} and {base}")
    i = np.arange(0, rot, 2, dtype=np.float64)
    f = float(base) ** (-i / max(rot, 1))
    factor = 1.0
    if scaling is not None:
        sc = dict(scaling)
        kind = sc.pop("type", None)

        def entry(name, *default, zero=False):
            if name not in sc and not default:
                raise ValueError(f"scaling: {name} missing in {scaling}")
            x = float(sc.pop(name, *default))
            if not (0 < x < math.inf or (zero and x == 0)):
                raise ValueError(f"scaling: {name} {'>=' if zero else '>'} 0 expected, got {x}")
            return x
        s = entry("factor")
        if kind == "linear":
            f = f / s
        elif kind == "base":
            if rot <= 2:
                raise ValueError("scaling by the base needs rot > 2")
            f = (float(base) * s ** (rot / (rot - 2))) ** (-i / rot)
        elif kind == "bands":
            lo, hi, n0 = entry("low_freq_factor", zero=True), entry("high_freq_factor"), entry("original_max_positions")
            if not hi > lo:
                raise ValueError("scaling: high_freq_factor > low_freq_factor expected")
            keep = np.clip((n0 * f / (2 * math.pi) - lo) / (hi - lo), 0.0, 1.0)
            f = f * (keep + (1.0 - keep) / s)
        elif kind == "yarn":
            n0, fast, slow = entry("original_max_positions"), entry("beta_fast", 32.0), entry("beta_slow", 1.0)
            if not base > 1:
                raise ValueError(f"scaling: yarn needs base > 1, got {base}")
            pair = lambda turns: rot * math.log(n0 / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
            slowed = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
            f = f * (1.0 - slowed) + f / s * slowed
            factor = 0.1 * math.log(s) + 1.0 if s > 1 else 1.0
        else:
            raise ValueError(f"scaling: unknown type {kind!r}")
        if sc:
            raise ValueError(f"scaling: unknown entries {sorted(sc)}")
    return torch.from_numpy(np.ascontiguousarray(f, dtype=np.float64)).to(device), factor


def qk_norm_rope(q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-5, layout="half", factor=1.0,
                 q_out=None, k_out=None, stream=None):
    """Queries and keys of n tokens, normalised per head and turned by position in one pass.

    q: [n, hq, d], k: [n, hk, d] (bf16 or fp32; token and head strides free, so slices of a
    packed projection output do); positions: int64 [n]; freqs, factor: from
    ``rope_frequencies`` (the first 2 * len(freqs) elements of a head are turned).
    q_weight, k_weight: [d], the head norms' weights, or None for no norm.  layout "half" pairs
    elements i and i + rot/2, "interleaved" 2i and 2i+1.  q_out / k_out: None, tensors of the
    same shapes, or q / k themselves; each overlaps nothing else.  Returns (q_out, k_out)."""
    if q_out is None and k_out is None and stream is None:
        y = (_fast or _fast_calls()).qk_norm_rope(q, k, positions, freqs, q_weight, k_weight, eps, LAYOUTS.get(layout),
                                                  factor)
        if y is not None:
            return y
    if _away(q, stream):
        with _at(q, stream):
            return qk_norm_rope(q, k, positions, freqs, q_weight=q_weight, k_weight=k_weight, eps=eps, layout=layout,
                                factor=factor, q_out=q_out, k_out=k_out)
    torch = _torch()
    code = _type_code(q, "q", 3)
    n, hq, d = q_shape = q.shape
    if k.dim() != 3:
        raise ValueError(f"k: [n, heads, d] expected, got shape {tuple(k.shape)}")
    hk = k.shape[1]
    k_shape = (n, hk, d)
    _check_tensor(k, "k", k_shape, q)
    _check_tensor(positions, "positions", (n,), q, torch.int64)
    if freqs.dim() != 1:
        raise ValueError(f"freqs: one dimension expected, got shape {tuple(freqs.shape)}")
    rot = 2 * freqs.shape[0]
    _check_tensor(freqs, "freqs", (rot // 2,), q, torch.float64)
    if not 1 <= d <= 1024 or rot > d:
        raise ValueError(f"head size {d} (1 to 1024), {rot} elements turned")
    if layout not in LAYOUTS:
        raise ValueError(f"layout: {layout!r}, one of {sorted(LAYOUTS)} expected")
    if not (0 <= eps < math.inf and math.isfinite(factor)):
        raise ValueError(f"eps {eps}, factor {factor}")
    if q_weight is not None:
        _check_tensor(q_weight, "q_weight", (d,), q)
    if k_weight is not None:
        _check_tensor(k_weight, "k_weight", (d,), q)
    _check_plain(q, k, freqs, q_weight, k_weight)
    if q_out is None:
        q_out = q.new_empty(q_shape)
    else:
        _check_out(q_out, "q_out", q_shape, q, (k, positions, freqs, q_weight, k_weight), q)
    if k_out is None:
        k_out = q.new_empty(k_shape)
    else:
        _check_out(k_out, "k_out", k_shape, q, (q, q_out, positions, freqs, q_weight, k_weight), k)
    if n and hq + hk:
        qs, ks, qos, kos = q.stride(), k.stride(), q_out.stride(), k_out.stride()
        _call("pwp_qk_norm_rope", ROPE_ARGS.pack(
            q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), qs[0], qs[1], ks[0], ks[1], qos[0], qos[1],
            kos[0], kos[1], positions.data_ptr(), freqs.data_ptr(), _ptr(q_weight), _ptr(k_weight), n, code, hq, hk, d,
            rot, LAYOUTS[layout], eps, factor), q.get_device())
    return q_out, k_out


def attention(q, k, v, cu_seqlens, *, causal=True, scale=None, out=None, stats=None, stream=None):
    """Softmax attention within each of the packed sequences.

    q: [n, hq, d], k and v: [n, hk, d] (bf16 or fp32, d <= 256, hq a multiple of hk; token and
    head strides free); cu_seqlens: int32 [sequences + 1] on the device: sequence s is rows
    cu_seqlens[s] to cu_seqlens[s+1].  scale: default 1 / sqrt(d).  Returns out [n, hq, d]
    (a tensor of one's own must not overlap q, k or v); rows in no sequence are left as they
    were (of a fresh output: undefined).  Offsets that decrease or leave 0..n end the batch
    there and set status 1 in `stats` (a ``new_stats`` record, optional), which also receives
    a device-side wait that ran out."""
    if out is None and stream is None:
        y = (_fast or _fast_calls()).attention(q, k, v, cu_seqlens, causal, scale, stats)
        if y is not None:
            return y
    if _away(q, stream):
        with _at(q, stream):
            return attention(q, k, v, cu_seqlens, causal=causal, scale=scale, out=out, stats=stats)
    code = _type_code(q, "q", 3)
    n, hq, d = q_shape = q.shape
    if k.dim() != 3:
        raise ValueError(f"k: [n, heads, d] expected, got shape {tuple(k.shape)}")
    hk = k.shape[1]
    _check_tensor(k, "k", (n, hk, d), q)
    _check_tensor(v, "v", (n, hk, d), q)
    if hk < 1 or hq < 1 or hq % hk:
        raise ValueError(f"{hq} query heads do not divide among {hk} key heads")
    if not 1 <= d <= 256:
        raise ValueError(f"head size {d}, 1 to 256 expected")
    if n * hq >= 1 << 31:
        raise ValueError(f"{n} tokens of {hq} heads: fewer than 2^31 query rows expected")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError(f"cu_seqlens: [sequences + 1] expected, got shape {tuple(cu_seqlens.shape)}")
    _check_tensor(cu_seqlens, "cu_seqlens", cu_seqlens.shape, q, _torch().int32)
    if scale is None:
        scale = d ** -0.5
    elif not math.isfinite(scale):
        raise ValueError(f"scale: {scale}")
    _check_plain(q, k, v)
    stats_p = _stats_ptr(stats, q)
    if out is None:
        out = q.new_empty(q_shape)
    else:
        _check_out(out, "out", q_shape, q, (q, k, v, cu_seqlens, stats))
    nseq = cu_seqlens.shape[0] - 1
    if n and nseq:
        qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
        args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0],
                os[1], cu_seqlens.data_ptr(), stats_p, n, nseq, code, hq, hk, d, 1 if causal else 0, scale)
        need = _pwp.lib().pwp_attention_workspace_bytes(ATTENTION_ARGS.pack(*args, 0, 0))
        scratch = _torch().empty(need, dtype=_torch().uint8, device=q.device) if need else None
        _call("pwp_attention", ATTENTION_ARGS.pack(*args, _ptr(scratch), need), q.get_device())
    return out


def _linear(x, w, w_up, bias, bias_up, activation, residual, out, stats, name):
    code = _type_code(x, "x", 2)
    rows, k = x.shape
    if w.dim() != 2:
        raise ValueError(f"{name}: [n, k] expected, got shape {tuple(w.shape)}")
    n = w.shape[0]
    _check_tensor(w, name, (n, k), x)
    if not (1 <= k < 1 << 24 and 1 <= n < 1 << 24 and rows < 1 << 31):
        raise ValueError(f"sizes out of range: {rows} rows, k {k}, n {n}")
    if w_up is not None:
        _check_tensor(w_up, "w_up", (n, k), x)
    if bias is not None:
        _check_tensor(bias, "bias", (n,), x)
    if bias_up is not None:
        _check_tensor(bias_up, "bias_up", (n,), x)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation: {activation!r}, one of {sorted(ACTIVATIONS)} expected")
    if residual is not None:
        _check_tensor(residual, "residual", (rows, n), x)
    _check_plain(x, w, w_up, bias, bias_up, residual)
    stats_p = _stats_ptr(stats, x)
    if out is None:
        out = x.new_empty((rows, n))
    else:
        _check_out(out, "out", (rows, n), x, (x, w, w_up, bias, bias_up, stats), residual)
    if rows:
        xs, ws = x.stride(0), w.stride(0)
        us = w_up.stride(0) if w_up is not None else 0
        xp, wp, up = x.data_ptr(), w.data_ptr(), _ptr(w_up)
        args = (xp, wp, up, _ptr(bias), _ptr(bias_up), _ptr(residual), out.data_ptr(), xs, ws, us,
                residual.stride(0) if residual is not None else 0, out.stride(0), stats_p, rows, k, n, code, act)
        scratch = None
        if code == _pwp.BF16 and ((xs | ws | us) & 7 or (xp | wp | up) & 15):
            # operands the tensor cores' copies cannot take as they are
            need = _pwp.lib().pwp_linear_workspace_bytes(LINEAR_ARGS.pack(*args, 0, 0))
            if need:
                scratch = _torch().empty(need, dtype=_torch().uint8, device=x.device)
                args += (scratch.data_ptr(), need)
        if scratch is None:
            args += (0, 0)
        _call("pwp_linear", LINEAR_ARGS.pack(*args), x.get_device())
    return out


def linear(x, w, *, bias=None, activation="none", residual=None, out=None, stats=None, stream=None):
    """activation(x w^T + bias) + residual for x [rows, k], w [n, k], bias [n] and residual
    [rows, n] (bf16 or fp32, one type; rows may be strided).  activation: "none", "relu",
    "silu", "gelu" (by the normal distribution) or "gelu_tanh".  out: None or a tensor
    [rows, n], which may be `residual` itself but overlap nothing else.  stats: an optional
    ``new_stats`` record for a device-side wait that ran out (without it the rows concerned
    come out NaN)."""
    if out is None and stream is None:
        y = (_fast or _fast_calls()).linear(x, w, None, bias, None, ACTIVATIONS.get(activation), residual, stats)
        if y is not None:
            return y
    if _away(x, stream):
        with _at(x, stream):
            return linear(x, w, bias=bias, activation=activation, residual=residual, out=out, stats=stats)
    return _linear(x, w, None, bias, None, activation, residual, out, stats, "w")


def gated_linear(x, w_gate, w_up, *, bias_gate=None, bias_up=None, activation="silu", out=None, stats=None,
                 stream=None):
    """activation(x w_gate^T + bias_gate) * (x w_up^T + bias_up): both projections of a gated
    feed-forward block, the activation and the product in one kernel.  Shapes, types and the
    other arguments as for ``linear``."""
    if w_up is None:
        raise TypeError("w_up: tensor expected, got NoneType (without it: linear)")
    if out is None and stream is None:
        y = (_fast or _fast_calls()).linear(x, w_gate, w_up, bias_gate, bias_up, ACTIVATIONS.get(activation), None, stats)
        if y is not None:
            return y
    if _away(x, stream):
        with _at(x, stream):
            return gated_linear(x, w_gate, w_up, bias_gate=bias_gate, bias_up=bias_up, activation=activation, out=out,
                                stats=stats)
    return _linear(x, w_gate, w_up, bias_gate, bias_up, activation, None, out, stats, "w_gate")


# ------------------------------------------------------------------- a decoder block

def block_forward(weights, hidden, seq_lens, *, heads, kv_heads=None, freqs=None, factor=1.0, layout="half",
                  positions=None, norms=None, biases=None, activation="silu", eps=1e-5, causal=True, scale=None,
                  stats=None, stream=None):
    """One decoder block over packed calibration sequences.

    weights: {"q_proj", "k_proj", "v_proj", "o_proj", "gate_proj", "up_proj", "down_proj":
    [n, k] tensors}; hidden: [tokens, width], the block's input, of the weights' type; seq_lens:
    the sequences' lengths (they add up to the tokens).  heads / kv_heads: of the queries and
    of the keys and values (default: the same).  freqs, factor, layout, positions: as for
    ``qk_norm_rope`` (freqs None: no rotation; positions None: 0, 1, ... in each sequence).
    norms: {"attn", "mlp": [width] weights of the block's norms, "q", "k": [d] weights of the
    head norms}, each optional (a missing "attn" or "mlp" norms without a weight, a missing
    "q" or "k" leaves the heads as they are); biases: {projection: [n]}, each optional.

    Returns (activations, out): {"attn_in", "o_in", "mlp_in", "down_in"}, the inputs of
    the projections as ``FEEDS`` names them (``prune_block``'s activations), and the block's
    output, residuals included.  stats: an optional ``new_stats`` record.  The lengths and
    positions are copied from the host, so the call as a whole cannot be captured into a
    graph; its operators can."""
    torch = _torch()
    missing = sorted(set(FEEDS) - set(weights))
    if missing:
        raise ValueError(f"weights: {missing} missing")
    norms, biases = dict(norms or {}), dict(biases or {})
    for name, given, known in (("norms", norms, {"attn", "mlp", "q", "k"}), ("biases", biases, set(FEEDS))):
        if set(given) - known:
            raise ValueError(f"{name}: unknown entries {sorted(set(given) - known)}")
    if hidden.dim() != 2:
        raise ValueError(f"hidden: [tokens, width] expected, got shape {tuple(hidden.shape)}")
    lens = [int(x) for x in seq_lens]
    n = hidden.shape[0]
    if any(x < 0 for x in lens) or sum(lens) != n:
        raise ValueError(f"seq_lens: {sum(lens)} tokens in all, hidden has {n}")
    kv_heads = heads if kv_heads is None else kv_heads
    if heads < 1 or kv_heads < 1 or heads % kv_heads or weights["q_proj"].shape[0] % heads:
        raise ValueError(f"{heads} query heads, {kv_heads} key heads, q_proj {tuple(weights['q_proj'].shape)}")
    d = weights["q_proj"].shape[0] // heads
    if _away(hidden, stream):
        with _at(hidden, stream):
            return block_forward(weights, hidden, lens, heads=heads, kv_heads=kv_heads, freqs=freqs, factor=factor,
                                 layout=layout, positions=positions, norms=norms, biases=biases,
                                 activation=activation, eps=eps, causal=causal, scale=scale, stats=stats)
    dev = hidden.device
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).to(dev)
    w, b = weights, biases.get
    attn_in = rms_norm(hidden, norms.get("attn"), eps=eps)
    packed = torch.empty((n, (heads + 2 * kv_heads) * d), dtype=hidden.dtype, device=dev)
    ends = np.cumsum([0, heads * d, kv_heads * d, kv_heads * d])
    q, k, v = (packed[:, ends[i]:ends[i + 1]] for i in range(3))
    for name, dst in (("q_proj", q), ("k_proj", k), ("v_proj", v)):
        linear(attn_in, w[name], bias=b(name), out=dst, stats=stats)
    q, k, v = q.view(n, heads, d), k.view(n, kv_heads, d), v.view(n, kv_heads, d)
    if freqs is not None or norms.get("q") is not None or norms.get("k") is not None:
        if freqs is None:
            freqs = torch.empty(0, dtype=torch.float64, device=dev)
        if positions is None:
            positions = torch.from_numpy(np.concatenate([np.arange(x, dtype=np.int64) for x in lens])
                                         if lens else np.zeros(0, np.int64)).to(dev)
        qk_norm_rope(q, k, positions, freqs, q_weight=norms.get("q"), k_weight=norms.get("k"), eps=eps, layout=layout,
                     factor=factor, q_out=q, k_out=k)
    o_in = attention(q, k, v, cu, causal=causal, scale=scale, stats=stats).view(n, heads * d)
    mid = linear(o_in, w["o_proj"], bias=b("o_proj"), residual=hidden, stats=stats)
    mlp_in = rms_norm(mid, norms.get("mlp"), eps=eps)
    down_in = gated_linear(mlp_in, w["gate_proj"], w["up_proj"], bias_gate=b("gate_proj"), bias_up=b("up_proj"),
                           activation=activation, stats=stats)
    out = linear(down_in, w["down_proj"], bias=b("down_proj"), residual=mid, stats=stats)
    return {"attn_in": attn_in, "o_in": o_in, "mlp_in": mlp_in, "down_in": down_in}, out


def prune_decoder_block(weights, hidden, seq_lens, *, forward, stream=None, **cfg):
    """One step of pruning a model block by block: the dense block's forward pass gives its
    layers' inputs, every layer is pruned with its input (``prune_block``, H shared by the
    layers that read the same one), and the hidden states pass through the pruned layers.

    weights, hidden, seq_lens and forward (a dict): as for ``block_forward``; cfg: as for
    ``prune_layer`` (method, pattern, sparsity, ...).  Returns (results, out): {layer: (W_hat
    fp32, mask, Stats)} and the pruned block's output, the next block's hidden states.  The
    pruned weights take part in that pass rounded to the weights' type."""
    if _away(hidden, stream):
        with _at(hidden, stream):
            return prune_decoder_block(weights, hidden, seq_lens, forward=forward, **cfg)
    weights = {name: weights[name] for name in FEEDS if name in weights}
    acts, _ = block_forward(weights, hidden, seq_lens, **forward)
    results = _pwp.prune_block(weights, acts, FEEDS, **cfg)
    del acts      # the second pass allocates its own
    pruned = {name: results[name][0].to(weights[name].dtype) for name in FEEDS}
    _, out = block_forward(pruned, hidden, seq_lens, **forward)
    return results, out
