"""Oracle of the decoder block's forward operators: plain NumPy in fp64, straight from the
formulas (inputs are converted, nothing is rounded on the way)."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["rms_norm", "rope_frequencies", "qk_norm_rope", "attention", "activation", "linear", "gated_linear",
           "block_forward"]


def _d(x):
    return np.asarray(x, dtype=np.float64)


def rms_norm(x, weight=None, eps=1e-5):
    """x / sqrt(mean(x^2) + eps) * weight, along the last axis."""
    x = _d(x)
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return y if weight is None else y * _d(weight)


def rope_frequencies(rot, base=10000.0):
    """f_i = base^(-2 i / rot), i = 0 .. rot/2 - 1."""
    return np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=np.float64)


def _turn(x, positions, freqs, layout, factor):
    x = x.copy()
    rot = 2 * len(freqs)
    for i, f in enumerate(freqs):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        angle = _d(positions) * f
        c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
        u, v = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = u * c - v * s, v * c + u * s
    return x


def qk_norm_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps=1e-5, layout="half", factor=1.0):
    """Head norms (where a weight is given) and the rotation by position."""
    out = []
    for x, w in ((q, q_weight), (k, k_weight)):
        y = _d(x) if w is None else rms_norm(x, w, eps)
        out.append(_turn(y, positions, _d(freqs), layout, factor))
    return tuple(out)


def attention(q, k, v, seq_lens, causal=True, scale=None, spread=False):
    """Softmax attention within packed sequences, one query at a time.  With spread=True also
    returns sum_j p_j |v_j|, the size a relative error of the probabilities is scaled by."""
    q, k, v = _d(q), _d(k), _d(v)
    n, hq, d = q.shape
    group = hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, size = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    at = 0
    for length in seq_lens:
        for h in range(hq):
            ks, vs = k[at:at + length, h // group], v[at:at + length, h // group]
            for i in range(length):
                e = i + 1 if causal else length
                s = scale * (ks[:e] @ q[at + i, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[at + i, h] = p @ vs[:e]
                if spread:
                    size[at + i, h] = p @ np.abs(vs[:e])
        at += length
    return (out, size) if spread else out


def activation(name, x):
    x = _d(x)
    if name == "none":
        return x
    if name == "relu":
        return np.where(x > 0, x, 0.0 * x)
    if name == "silu":
        return x / (1.0 + np.exp(-x))
    if name == "gelu":
        return x * 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    raise ValueError(name)


def linear(x, w, bias=None, act="none", residual=None):
    """act(x w^T + bias) + residual."""
    y = _d(x) @ _d(w).T
    if bias is not None:
        y = y + _d(bias)
    y = activation(act, y)
    return y if residual is None else y + _d(residual)


def gated_linear(x, w_gate, w_up, bias_gate=None, bias_up=None, act="silu"):
    """act(x w_gate^T + bias_gate) * (x w_up^T + bias_up)."""
    return linear(x, w_gate, bias_gate, act) * linear(x, w_up, bias_up)


def block_forward(weights, hidden, seq_lens, heads, kv_heads=None, freqs=None, layout="half", norms=None, eps=1e-5):
    """A decoder block without biases: ({layer input: activations}, output)."""
    kv_heads = kv_heads or heads
    norms = norms or {}
    x = _d(hidden)
    n = x.shape[0]
    attn_in = rms_norm(x, norms.get("attn"), eps)
    q, k, v = (linear(attn_in, weights[p]).reshape(n, h, -1)
               for p, h in (("q_proj", heads), ("k_proj", kv_heads), ("v_proj", kv_heads)))
    pos = np.concatenate([np.arange(length) for length in seq_lens])
    q, k = qk_norm_rope(q, k, pos, [] if freqs is None else freqs, norms.get("q"), norms.get("k"), eps, layout)
    o_in = attention(q, k, v, seq_lens).reshape(n, -1)
    mid = linear(o_in, weights["o_proj"], residual=x)
    mlp_in = rms_norm(mid, norms.get("mlp"), eps)
    down_in = gated_linear(mlp_in, weights["gate_proj"], weights["up_proj"])
    out = linear(down_in, weights["down_proj"], residual=mid)
    return {"attn_in": attn_in, "o_in": o_in, "mlp_in": mlp_in, "down_in": down_in}, out
