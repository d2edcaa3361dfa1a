"""GPU parity of the decoder block's forward operators against the fp64 oracle.

Tolerances, elementwise and derived from the arithmetic (u = half a step of the output type:
2^-8 for bf16, 2^-24 for fp32; g = 2^-23, one fp32 step, which bounds an addition rounded
either way):
  rms_norm       the fp32 sum over b terms of one sign is off by less than
                 (b / 32 + 16) g (a thread's chain, then a tree), halved by the root, and four
                 more operations follow: u + (b / 64 + 16) g
  qk_norm_rope   the same for the norm; the turn adds |a c| and |b s| each off by 4 g, so
                 u |y| + ((d / 64 + 16) g) (|a c| + |b s|), bounded by factor * (|a| + |b|)
  linear         products of bf16 are exact in fp32; a sum of k terms in chains of at most
                 k / 16 + 32 additions (16 terms of one instruction, then one accumulator):
                 (k / 16 + 32) g S, S = sum |x w| + |bias|; fp32 tensors: every product is also
                 rounded and the chain is k long: (k + 4) g S.  Activations have slope at most
                 1.13 and are themselves good to 8 g; u |y| and the residual's addition follow.
  attention      probabilities of the tensor-core kernel are rounded to bf16 (2^-8 of each, so
                 2^-8 sum p|v|), the exponential is good to 2^-12 of itself, and a score is off
                 by (d / 16 + 40) g scale sum |q k|, which is a relative error of p and of the
                 sum; output rounding u |o|.
"""
import math

import numpy as np
import pytest

from oracle import forward as F

pytestmark = pytest.mark.gpu
G = 2.0 ** -23


def _torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def _pwp():
    import post_weight_pruning_b200 as pwp
    return pwp


def U(dtype):
    return 2.0 ** -8 if "bf" in str(dtype) else 2.0 ** -24


def dt(name):
    torch = _torch()
    return torch.bfloat16 if name == "bf16" else torch.float32


def rnd(shape, dtype, seed, scale=1.0):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dt(dtype)).cuda()


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, tol, what=""):
    got = np64(got)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300))))


# ------------------------------------------------------------------- rms_norm

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,b", [(1, 1), (1, 4096), (3, 7), (5, 130), (2, 1000), (300, 256), (7, 8192), (2, 11008),
                                 (3, 30001), (9, 72)])
def test_rms_norm(n, b, dtype):
    pwp = _pwp()
    x, w = rnd((n, b), dtype, 1, 3.0), rnd((b,), dtype, 2)
    for weight in (w, None):
        y = pwp.rms_norm(x, weight)
        want = F.rms_norm(np64(x), np64(weight))
        close(y, want, np.abs(want) * (U(x.dtype) + (b / 64 + 16) * G) + 1e-37)


def test_rms_norm_strides_in_place_and_zero_rows():
    torch, pwp = _torch(), _pwp()
    big = rnd((6, 200), "bf16", 3)
    big[2] = 0
    for cut in (slice(0, 96), slice(8, 136), slice(3, 50)):
        keep = big.clone()
        x = keep[:, cut]
        want = F.rms_norm(np64(x))
        y = pwp.rms_norm(x, out=x)
        assert y is x
        close(y, want, np.abs(want) * (U(x.dtype) + 32 * G))
        outside = torch.ones(200, dtype=torch.bool)
        outside[cut] = False
        assert torch.equal(keep[:, outside.cuda()], big[:, outside.cuda()])
    assert torch.equal(pwp.rms_norm(big)[2], torch.zeros_like(big[2]))


# ------------------------------------------------------------------- qk_norm_rope

def rope_tol(q, freqs, weight, eps, layout, factor, want, u, d):
    y = np64(q) if weight is None else F.rms_norm(np64(q), np64(weight), eps)
    mag = np.abs(y)
    rot = 2 * len(freqs)
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        mag[..., a] = mag[..., b] = factor * (mag[..., a] + mag[..., b])
    return u * np.abs(want) + (d / 64 + 16) * G * mag + 1e-37


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,hq,hk,d,rot,layout,norm,first", [
    (1, 1, 1, 2, 2, "half", False, 0),
    (5, 4, 2, 128, 128, "half", True, 0),
    (5, 4, 2, 128, 128, "interleaved", False, 1000000),
    (33, 8, 1, 64, 32, "half", True, 5),
    (9, 3, 3, 80, 80, "half", False, 100000),
    (9, 7, 1, 96, 48, "interleaved", True, 77),
    (4, 2, 0, 128, 64, "half", True, 3),
    (3, 2, 1, 33, 10, "half", True, 9),
    (3, 2, 1, 40, 12, "interleaved", True, 9),
    (2, 1, 1, 256, 256, "half", True, 11),
    (2, 2, 1, 128, 0, "half", True, 11),
    (70, 32, 8, 128, 64, "interleaved", True, 900000),
])
def test_qk_norm_rope(n, hq, hk, d, rot, layout, norm, first, dtype):
    torch, pwp = _torch(), _pwp()
    packed = rnd((n, (hq + 2 * hk) * d), dtype, 5)
    q, k = packed[:, :hq * d].view(n, hq, d), packed[:, hq * d:(hq + hk) * d].view(n, hk, d)
    qw, kw = (rnd((d,), dtype, 6), rnd((d,), dtype, 7)) if norm else (None, None)
    pos = first + 3 * torch.arange(n, device="cuda")
    f, _ = pwp.rope_frequencies(rot, base=1e4)
    factor = 1.25
    want = F.qk_norm_rope(np64(q), np64(k), pos.cpu().numpy(), np64(f), np64(qw), np64(kw), 1e-5, layout, factor)
    got = pwp.qk_norm_rope(q, k, pos, f, q_weight=qw, k_weight=kw, layout=layout, factor=factor)
    for x, w, y, e in ((q, qw, got[0], want[0]), (k, kw, got[1], want[1])):
        close(y, e, rope_tol(x, np64(f), w, 1e-5, layout, factor, e, U(x.dtype), d))
    # in place, on slices of the packed projection: bit for bit the same, v untouched
    before = packed.clone()
    q2, k2 = pwp.qk_norm_rope(q, k, pos, f, q_weight=qw, k_weight=kw, layout=layout, factor=factor, q_out=q, k_out=k)
    assert q2 is q and torch.equal(q, got[0]) and torch.equal(k, got[1])
    assert torch.equal(packed[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


def test_qk_norm_rope_head_major_and_negative_positions():
    torch, pwp = _torch(), _pwp()
    n, h, d = 6, 4, 64
    q = rnd((h, n, d), "bf16", 8).transpose(0, 1)
    pos = torch.tensor([-5, 0, 3, 2 ** 40 + 1, 7, 7], device="cuda")
    f, _ = pwp.rope_frequencies(d)
    qo, ko = pwp.qk_norm_rope(q, q, pos, f)
    # at 2^40 the double angle itself is off by up to 2^-52 of 2^40 radians
    want = F.qk_norm_rope(np64(q), np64(q), pos.cpu().numpy(), np64(f))[0]
    close(qo, want, rope_tol(q, np64(f), None, 0, "half", 1.0, want, U(q.dtype), d) + 2.0 ** -10)
    assert torch.equal(qo, ko)


# ------------------------------------------------------------------- attention

def att_case(lens, hq, hk, d, dtype, seed, extra=0, qscale=1.5):
    torch = _torch()
    n = sum(lens) + extra
    q, k, v = rnd((n, hq, d), dtype, seed, qscale), rnd((n, hk, d), dtype, seed + 1), rnd((n, hk, d), dtype, seed + 2)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return q, k, v, cu


def att_tol(q, k, lens, hq, hk, d, want, size, dtype, scale=None):
    scale = d ** -0.5 if scale is None else scale
    s = scale * float(np.max(np.linalg.norm(np64(q), axis=-1)) * np.max(np.linalg.norm(np64(k), axis=-1)))
    if dtype == "fp32":
        rel = (d + 8) * G * s + 64 * G
        return U(dtype) * np.abs(want) + (2 * rel + (max(lens) + 8) * G) * size + 1e-30
    rel = (d / 16 + 40) * G * s + 2.0 ** -12
    return U(dtype) * np.abs(want) + (2.0 ** -8 + 2 * rel + (max(lens) / 16 + 40) * G) * size + 1e-30


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hq,hk,d,dtype", [
    ([1], 1, 1, 64, "bf16"),
    ([1, 0, 2, 0, 0, 3], 4, 2, 128, "bf16"),
    ([127, 128, 129], 2, 2, 128, "bf16"),
    ([300], 4, 1, 128, "bf16"),
    ([5, 260, 64], 8, 2, 64, "bf16"),
    ([33, 140], 5, 1, 80, "bf16"),          # a group that does not divide a tile
    ([200], 7, 1, 96, "bf16"),
    ([70], 3, 1, 128, "bf16"),
    ([257], 40, 8, 128, "bf16"),
    ([19, 300], 16, 1, 128, "bf16"),
    ([130], 129, 1, 64, "bf16"),            # more heads in a group than a tile has rows
    ([40, 9], 2, 1, 20, "bf16"),            # head size the copies cannot take
    ([50], 2, 1, 136, "bf16"),
    ([70, 1, 33], 4, 2, 128, "fp32"),
    ([100], 2, 1, 33, "fp32"),
    ([65], 1, 1, 256, "fp32"),
])
def test_attention(lens, hq, hk, d, dtype, causal):
    pwp = _pwp()
    q, k, v, cu = att_case(lens, hq, hk, d, dtype, 11)
    want, size = F.attention(np64(q), np64(k), np64(v), lens, causal, spread=True)
    st = pwp.new_stats()
    got = pwp.attention(q, k, v, cu, causal=causal, stats=st)
    assert pwp.read_stats(st).status == 0
    close(got, want, att_tol(q, k, lens, hq, hk, d, want, size, dtype))


def test_attention_strided_scaled_and_rows_left_alone():
    """q, k, v as slices of one packed buffer and head-major; an output with room around it; a
    scale of one's own; rows before the first and behind the last sequence keep their content."""
    torch, pwp = _torch(), _pwp()
    lens, hq, hk, d, extra = [30, 170], 4, 2, 128, 9
    n = sum(lens) + 2 * extra
    packed = rnd((n, (hq + 2 * hk) * d), "bf16", 21)
    q, k, v = (x.view(n, -1, d) for x in packed.split([hq * d, hk * d, hk * d], dim=1))
    v = v.transpose(0, 1).contiguous().transpose(0, 1)
    packed[:extra] = float("nan")
    packed[n - extra:] = float("inf")
    v[:extra] = float("inf")
    v[n - extra:] = float("nan")
    cu = (extra + torch.tensor([0, 30, 200])).to(torch.int32).cuda()
    room = torch.full((n, hq + 3, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, 1:hq + 1, :d]
    s = slice(extra, n - extra)
    got = pwp.attention(q, k, v, cu, scale=0.05, out=out)
    want, size = F.attention(np64(q[s]), np64(k[s]), np64(v[s]), lens, True, 0.05, spread=True)
    close(got[s], want, att_tol(q[s], k[s], lens, hq, hk, d, want, size, "bf16", 0.05))
    room[s, 1:hq + 1, :d] = 7.0
    assert bool((room == 7.0).all())


@pytest.mark.parametrize("hq,hk,dtype", [(2, 2, "bf16"), (8, 2, "bf16"), (2, 1, "fp32")])
def test_attention_later_tokens_never_reach_a_query(hq, hk, dtype):
    """Causal: NaN and infinities in the values and keys of later tokens leave earlier queries
    as they are, bit for bit; the queries that see them get them."""
    torch, pwp = _torch(), _pwp()
    lens, d, at = [300], 128, 140
    q, k, v, cu = att_case(lens, hq, hk, d, dtype, 31)
    clean = pwp.attention(q, k, v, cu)
    v2, k2 = v.clone(), k.clone()
    v2[at, :, 3] = float("nan")
    v2[at + 1, :, 5] = float("inf")
    v2[at + 5, :, 5] = -float("inf")
    got = pwp.attention(q, k, v2, cu)
    assert torch.equal(got[:at], clean[:at])
    assert bool(got[at:, :, 3].isnan().all())
    assert bool((got[at + 1:at + 5, :, 5] == float("inf")).all()) and bool(got[at + 5:, :, 5].isnan().all())
    others = [c for c in range(d) if c not in (3, 5)]
    assert torch.equal(got[:, :, others], clean[:, :, others])
    k2[at] = float("nan")
    got = pwp.attention(q, k2, v, cu)
    assert torch.equal(got[:at], clean[:at]) and bool(got[at:].isnan().all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("at,value", [((0, 140), -math.inf), ((0, 1), -math.inf), ((5, 6), math.inf), ((200, 201), math.inf),
                                      ((0, 300), -math.inf), ((130, 260), -math.inf)])
def test_attention_infinite_scores(at, value, dtype, causal):
    """Keys whose scores are infinite: -inf weighs nothing, also when a whole block or all that a
    query sees so far is -inf (NaN where it sees nothing else), and +inf makes NaN."""
    pwp = _pwp()
    lens, d = [300], 64
    q, k, v, cu = att_case(lens, 2, 1, d, dtype, 43)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    bad = k.clone()
    bad[at[0]:at[1], 0, 0] = value
    with np.errstate(invalid="ignore"):
        want, size = F.attention(np64(q), np64(bad), np64(v), lens, causal, spread=True)
        k[at[0]:at[1], 0, 0] = 0.0
        tol = att_tol(q, k, lens, 2, 1, d, want, size, dtype)
        close(pwp.attention(q, bad, v, cu, causal=causal), want, tol)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_several_rounds_of_work(causal):
    """More work than one round of the SMs: with the counter and without (the C entry point given
    no scratch) the same bits; the rows behind the last sequence stay."""
    torch, pwp = _torch(), _pwp()
    from post_weight_pruning_b200 import block as B
    lens = [700, 0, 1, 333, 1024, 1129, 64, 1700] * 2
    n, extra = sum(lens), 77
    q, k, v, cu = att_case(lens, 16, 8, 64, "bf16", 151, extra=extra)
    out = torch.full_like(q, 7.0)
    pwp.attention(q, k, v, cu, causal=causal, out=out)
    assert bool((out[n:] == 7.0).all())
    again = torch.full_like(q, 7.0)
    args = B.ATTENTION_ARGS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), again.data_ptr(), *q.stride()[:2], *k.stride()[:2],
                                 *v.stride()[:2], *again.stride()[:2], cu.data_ptr(), 0, n + extra, len(lens), pwp.BF16, 16, 8, 64,
                                 int(causal), 0.125, 0, 0)
    assert pwp.lib().pwp_attention_workspace_bytes(args) == 256
    assert pwp.lib().pwp_attention(args, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, again)
    at = 0
    for length in lens[:8]:                         # each sequence by itself
        s = slice(at, at + length)
        if length:
            alone = pwp.attention(q[s], k[s], v[s], torch.tensor([0, length], dtype=torch.int32, device="cuda"), causal=causal)
            assert torch.equal(alone, out[s])
        at += length
    want, size = F.attention(np64(q[701:1034]), np64(k[701:1034]), np64(v[701:1034]), [333], causal, spread=True)
    close(out[701:1034], want, att_tol(q, k, lens, 16, 8, 64, want, size, "bf16"))


def test_attention_several_rounds_when_waits_run_out():
    """Every row of the sequences comes out NaN, also those of work that nobody took."""
    torch, pwp = _torch(), _pwp()
    lens = [1024] * 8
    q, k, v, cu = att_case(lens, 16, 8, 64, "bf16", 152, extra=5)
    want = pwp.attention(q, k, v, cu)
    torch.cuda.synchronize()
    for limit in (0, 2):
        prev = pwp.set_wait_limit(limit)
        try:
            st, out = pwp.new_stats(), torch.full_like(q, 7.0)
            pwp.attention(q, k, v, cu, out=out, stats=st)
            torch.cuda.synchronize()
        finally:
            pwp.set_wait_limit(prev)
        s = pwp.read_stats(st)
        assert s.status in ((5,) if limit == 0 else (0, 5)) and bool((out[8192:] == 7.0).all())
        wrong = out[:8192] != want[:8192]
        assert bool(out[:8192][wrong].isnan().all()) and bool(wrong.any()) == (s.status == 5)
        assert torch.equal(pwp.attention(q, k, v, cu)[:8192], want[:8192])


def test_attention_bad_offsets_are_reported():
    torch, pwp = _torch(), _pwp()
    q, k, v, _ = att_case([100], 2, 1, 64, "bf16", 41)
    good = pwp.attention(q, k, v, torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda"))
    for offsets in ([0, 40, 30, 100], [0, 40, 101], [0, 40, -5, 100], [0, 40, 2 ** 31 - 1]):
        out = torch.full_like(q, 7.0)
        st = pwp.new_stats()
        pwp.attention(q, k, v, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out, stats=st)
        assert pwp.read_stats(st).status == 1
        assert torch.equal(out[:40], good[:40]) and bool((out[40:] == 7.0).all())


def test_attention_many_sequences_and_large_scores():
    torch, pwp = _torch(), _pwp()
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 9, size=150).tolist()
    q, k, v, cu = att_case(lens, 2, 1, 64, "bf16", 51, qscale=40.0)     # nearly one-hot rows
    want, size = F.attention(np64(q), np64(k), np64(v), lens, True, spread=True)
    close(pwp.attention(q, k, v, cu), want, att_tol(q, k, lens, 2, 1, 64, want, size, "bf16"))
    # scores that rise along the keys: the running maximum moves at every tile
    n = 520
    q = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 8.0
    k = torch.zeros_like(q)
    k[:, 0, 0] = torch.arange(n, device="cuda") * 0.25
    v = rnd((n, 1, 64), "bf16", 52)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want, size = F.attention(np64(q), np64(k), np64(v), [n], True, 1.0, spread=True)
    close(pwp.attention(q, k, v, cu, scale=1.0), want, att_tol(q, k, [n], 1, 1, 64, want, size, "bf16", 1.0))


# ------------------------------------------------------------------- linear, gated_linear

def lin_tol(x, w, bias, act, pre, y, res, dtype, slope=1.13):
    k = x.shape[1]
    s = np.abs(np64(x)) @ np.abs(np64(w)).T + (0 if bias is None else np.abs(np64(bias)))
    e = ((k / 16 + 32) if dtype == "bf16" else (k + 4)) * G * s
    return slope * e + 8 * G * np.abs(pre)


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("rows,k,n,dtype", [
    (1, 1, 1, "bf16"), (1, 64, 128, "bf16"), (1, 4096, 520, "bf16"), (3, 200, 24, "bf16"), (17, 1000, 136, "bf16"),
    (64, 256, 256, "bf16"), (129, 72, 1000, "bf16"), (300, 520, 264, "bf16"), (256, 128, 512, "bf16"),
    (700, 640, 1032, "bf16"), (33, 100, 77, "bf16"), (5, 33, 40, "bf16"), (260, 8, 8, "bf16"), (1100, 512, 1536, "bf16"),
    (700, 333, 521, "bf16"), (1400, 401, 1043, "bf16"), (40, 1003, 1001, "bf16"),
    (1, 5, 3, "fp32"), (70, 130, 65, "fp32"), (200, 64, 128, "fp32"), (300, 515, 260, "fp32"), (130, 4100, 132, "fp32"),
    (33, 2000, 36, "fp32"), (1, 700, 200, "fp32"), (1100, 36, 900, "fp32"),
])
def test_linear_and_gated(rows, k, n, dtype):
    pwp = _pwp()
    x, w, wu = rnd((rows, k), dtype, 61), rnd((n, k), dtype, 62, 0.05), rnd((n, k), dtype, 63, 0.05)
    b, bu, r = rnd((n,), dtype, 64), rnd((n,), dtype, 65), rnd((rows, n), dtype, 66)
    u = U(dtype)
    st = pwp.new_stats()
    for i, act in enumerate(ACTS):
        bias, res = (b if i != 1 else None), (r if i % 2 == 0 else None)
        pre = F.linear(np64(x), np64(w), np64(bias))
        want = F.linear(np64(x), np64(w), np64(bias), act, np64(res))
        tol = lin_tol(x, w, bias, act, pre, want, res, dtype)
        if res is not None:
            tol = tol + G * np.abs(np64(res))
        close(pwp.linear(x, w, bias=bias, activation=act, residual=res, stats=st), want, tol + u * np.abs(want) + 1e-37,
              act)
        up = F.linear(np64(x), np64(wu), np64(bu))
        want = F.gated_linear(np64(x), np64(w), np64(wu), np64(bias), np64(bu), act)
        eg = lin_tol(x, w, bias, act, pre, want, None, dtype)
        eu = lin_tol(x, wu, bu, "none", up, want, None, dtype, 1.0)
        g = F.activation(act, pre)
        tol = eg * np.abs(up) + eu * np.abs(g) + eg * eu + 2 * G * np.abs(want)
        close(pwp.gated_linear(x, w, wu, bias_gate=bias, bias_up=bu, activation=act, stats=st), want,
              tol + u * np.abs(want) + 1e-37, "gated " + act)
    assert pwp.read_stats(st).status == 0


@pytest.mark.parametrize("rows", [3, 300, 1100])
def test_linear_strides_and_residual_in_place(rows):
    torch, pwp = _torch(), _pwp()
    k, n = 192, 264
    for off, pad in ((8, 16), (3, 5)):       # what the copies can take, and what they cannot
        xb, rb = rnd((rows, k + off + pad), "bf16", 71), rnd((rows, n + off + pad), "bf16", 72)
        x, r, w = xb[:, off:off + k], rb[:, off:off + n], rnd((n, k), "bf16", 73, 0.05)
        want = F.linear(np64(x), np64(w), None, "silu", np64(r))
        pre = F.linear(np64(x), np64(w))
        tol = lin_tol(x, w, None, "silu", pre, want, r, "bf16") + G * np.abs(np64(r)) + 2.0 ** -8 * np.abs(want)
        before = rb.clone()
        apart = pwp.linear(x, w, activation="silu", residual=r)
        close(apart, want, tol)
        assert pwp.linear(x, w, activation="silu", residual=r, out=r) is r
        assert torch.equal(r, apart)
        assert torch.equal(rb[:, :off], before[:, :off]) and torch.equal(rb[:, off + n:], before[:, off + n:])


@pytest.mark.parametrize("n", [1000, 1001, 1002, 1004, 1028])
@pytest.mark.parametrize("off", [0, 1, 2])
def test_linear_many_rows_of_any_alignment(n, off):
    """Enough rows and columns for the kernel of CTA pairs, output and residual rows aligned to 16, 4
    or 2 bytes, a last tile partly filled both ways; what lies around the output stays."""
    torch, pwp = _torch(), _pwp()
    rows, k = 3001, 136
    x, w, u = rnd((rows, k), "bf16", 161), rnd((n, k), "bf16", 162, 0.05), rnd((n, k), "bf16", 163, 0.05)
    b, room = rnd((n,), "bf16", 164), rnd((rows, n + 5), "bf16", 165)
    r = room[:, off:off + n]
    before = room.clone()
    want = F.linear(np64(x), np64(w), np64(b), "relu", np64(r))
    pre = F.linear(np64(x), np64(w), np64(b))
    tol = lin_tol(x, w, b, "relu", pre, want, r, "bf16") + G * np.abs(np64(r)) + 2.0 ** -8 * np.abs(want)
    close(pwp.linear(x, w, bias=b, activation="relu", residual=r), want, tol)
    pwp.linear(x, w, bias=b, activation="relu", residual=r, out=r)
    close(r, want, tol)
    assert torch.equal(room[:, :off], before[:, :off]) and torch.equal(room[:, off + n:], before[:, off + n:])
    plain = pwp.gated_linear(x, w, u, bias_gate=b)
    pwp.gated_linear(x, w, u, bias_gate=b, out=r)
    assert torch.equal(r, plain)
    up = F.linear(np64(x), np64(u))
    want = F.gated_linear(np64(x), np64(w), np64(u), np64(b), None, "silu")
    eg, eu = lin_tol(x, w, b, "silu", pre, want, None, "bf16"), lin_tol(x, u, None, "none", up, want, None, "bf16", 1.0)
    tol = eg * np.abs(up) + eu * np.abs(F.activation("silu", pre)) + eg * eu + 2 * G * np.abs(want)
    close(plain, want, tol + 2.0 ** -8 * np.abs(want) + 1e-37)
    assert torch.equal(room[:, :off], before[:, :off]) and torch.equal(room[:, off + n:], before[:, off + n:])


def test_linear_non_finite_rows_stay_theirs():
    torch, pwp = _torch(), _pwp()
    for rows in (40, 600):
        x, w = rnd((rows, 256), "bf16", 81), rnd((304, 256), "bf16", 82)
        clean = pwp.linear(x, w)
        x2 = x.clone()
        x2[7, 3] = float("nan")
        got = pwp.linear(x2, w)
        assert bool(got[7].isnan().all())
        got[7] = clean[7]
        assert torch.equal(got, clean)


def test_gated_extremes():
    """Far in the tails silu is x or 0 (and never NaN for finite sums)."""
    torch, pwp = _torch(), _pwp()
    x = torch.tensor([[1.0, 0.0], [0.0, 1.0]], dtype=torch.bfloat16, device="cuda").repeat(1, 32)
    w = torch.full((8, 64), 100.0, dtype=torch.bfloat16, device="cuda")
    w[::2] = -100.0
    up = torch.full((8, 64), 0.5, dtype=torch.bfloat16, device="cuda")
    y = pwp.gated_linear(x, w, up)
    assert torch.equal(y[:, 1::2], torch.full_like(y[:, 1::2], 3200.0 * 16.0))
    assert bool((y[:, ::2] == 0).all())


# ------------------------------------------------------------------- streams, graphs, timeouts

def _ops(pwp, torch):
    """Every operator once over sizes that take each kernel; returns the outputs."""
    q, k, v, cu = att_case([5, 300, 70], 8, 2, 128, "bf16", 91)
    f, _ = pwp.rope_frequencies(128)
    pos = torch.arange(q.shape[0], device="cuda")
    outs = []
    xs = [rnd((r, 512), "bf16", 92 + r) for r in (2, 70, 1500)]
    w, wu = rnd((1040, 512), "bf16", 93, 0.05), rnd((1040, 512), "bf16", 94, 0.05)
    torch.cuda.synchronize()

    def run(stream=None):
        outs.clear()
        qr, kr = pwp.qk_norm_rope(q, k, pos, f, stream=stream)
        outs.extend([qr, kr, pwp.attention(qr, kr, v, cu, stream=stream)])
        for x in xs:
            y = pwp.rms_norm(x, stream=stream)
            outs.extend([y, pwp.linear(y, w, stream=stream), pwp.gated_linear(y, w, wu, stream=stream)])
        return list(outs)
    return run


def test_operators_on_a_stream_of_their_own_and_in_a_graph():
    torch, pwp = _torch(), _pwp()
    run = _ops(pwp, torch)
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kept = run()
    for _ in range(2):
        for t in kept:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31 (4.6 GB buffer), read and written in place of a copy's."""
    torch, pwp = _torch(), _pwp()
    n, pitch, d = 70000, 32768, 64
    buf = torch.empty((n, pitch), dtype=torch.bfloat16, device="cuda")
    x, out = buf[:, 8:8 + d], buf[:, 16384:16384 + d]
    x.copy_(rnd((n, d), "bf16", 120))
    flat, w = x.contiguous(), rnd((d, d), "bf16", 121, 0.2)
    pos = torch.arange(n, device="cuda")
    f, _ = pwp.rope_frequencies(d)
    cu = torch.tensor([0, 100, n - 3000, n], dtype=torch.int32, device="cuda")
    heads = lambda t: t.view(n, 1, d)
    for call in (lambda t, o: pwp.rms_norm(t, out=o), lambda t, o: pwp.linear(t, w, out=o),
                 lambda t, o: pwp.gated_linear(t, w, w, out=o),
                 lambda t, o: pwp.qk_norm_rope(heads(t), heads(t), pos, f, q_out=heads(o)),
                 lambda t, o: pwp.attention(heads(t), heads(t), heads(t), cu[2:], out=heads(o))):
        want = torch.zeros_like(flat)
        out.zero_()
        call(flat, want)
        call(x, out)
        assert torch.equal(out, want) and bool(want[n - 3000:].any())
    want32 = pwp.linear(flat.float(), w.float())
    del buf, x, out
    buf = torch.empty((n, pitch), dtype=torch.float32, device="cuda")
    buf[:, :d] = flat
    pwp.linear(buf[:, :d], w.float(), out=buf[:, d:2 * d])
    assert torch.equal(buf[:, d:2 * d], want32)


def test_broadcast_inputs():
    """Stride 0: one row for all rows, one key head for all, one residual row."""
    torch, pwp = _torch(), _pwp()
    row, w, r = rnd((1, 256), "bf16", 122), rnd((96, 256), "bf16", 123, 0.1), rnd((1, 96), "bf16", 124)
    y = pwp.linear(row.expand(40, 256), w, residual=r.expand(40, 96))
    want = F.linear(np64(row), np64(w), residual=np64(r))
    tol = U(y.dtype) * np.abs(want) + (256 / 16 + 36) * G * (np.abs(np64(row)) @ np.abs(np64(w)).T + np.abs(np64(r)))
    close(y, np.repeat(want, 40, 0), np.repeat(tol, 40, 0))
    y = pwp.linear(rnd((40, 256), "bf16", 125), w[:1].expand(96, 256))
    assert torch.equal(y, y[:, :1].expand(40, 96))
    z = pwp.rms_norm(row.expand(5, 256))
    assert torch.equal(z, pwp.rms_norm(row).expand(5, 256))
    q, k, v, cu = att_case([150], 4, 1, 64, "bf16", 126)
    got = pwp.attention(q, k.expand(150, 4, 64), v.expand(150, 4, 64), cu)
    want, size = F.attention(np64(q), np64(k), np64(v), [150], spread=True)
    close(got, want, att_tol(q, k, [150], 4, 1, 64, want, size, "bf16"))


def test_two_graphs_at_once():
    """Two captured graphs of calls that take scratch, replayed on two streams beside each other
    and beside an eager call, several times."""
    torch, pwp = _torch(), _pwp()
    xs = [rnd((700, 1001), "bf16", 127 + i) for i in range(3)]
    w = rnd((300, 1001), "bf16", 130, 0.1)
    q, k, v, cu = att_case([400, 1, 333], 4, 2, 128, "bf16", 131)
    run = lambda x: (pwp.linear(x, w, activation="silu"), pwp.rms_norm(x), pwp.attention(q, k, v, cu))
    want = [run(x) for x in xs]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(x))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        mine = run(xs[2])
        torch.cuda.synchronize()
        for got, ref in zip(outs + [mine], want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_usual_calls_with_and_without_the_native_marshalling(monkeypatch):
    """The C++ marshalling takes the usual calls and gives what the Python one gives, bit for bit;
    what it does not take runs or is refused as before."""
    torch, pwp = _torch(), _pwp()
    from post_weight_pruning_b200 import block as B
    fast, taken = B._fast_calls(), []
    assert fast is not B._NoFastCalls, "_fastcall.so is not built"

    class Watch:
        pass
    for name in ("rms_norm", "qk_norm_rope", "attention", "linear"):
        def call(*a, f=getattr(fast, name)):
            y = f(*a)
            taken.append(y is not None)
            return y
        setattr(Watch, name, staticmethod(call))
    q, k, v, cu = att_case([40, 3], 4, 2, 64, "bf16", 141)
    pos, (f, s) = torch.arange(43, device="cuda"), pwp.rope_frequencies(32)
    qw, x, w, u = rnd((64,), "bf16", 144), rnd((43, 96), "bf16", 145), rnd((80, 96), "bf16", 146), rnd((80, 96), "bf16", 147)
    b, r, odd = rnd((80,), "bf16", 148), rnd((43, 80), "bf16", 149), rnd((900, 201), "bf16", 150)
    stats = pwp.new_stats()
    calls = [lambda: pwp.rms_norm(x), lambda: pwp.rms_norm(x[:, :48], w[0, :48], eps=0), lambda: pwp.rms_norm(x.float()),
             lambda: pwp.rms_norm(x[:1].expand(4, 96)),
             lambda: pwp.qk_norm_rope(q, k, pos, f, q_weight=qw, layout="interleaved", factor=2.0),
             lambda: pwp.qk_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, pos, f[:0]),
             lambda: pwp.attention(q, k, v, cu), lambda: pwp.attention(q, k, v, cu, causal=False, scale=0.2, stats=stats),
             lambda: pwp.attention(q.float(), k.float(), v.float(), cu),
             lambda: pwp.linear(x, w), lambda: pwp.linear(x, w, bias=b, residual=r, activation="gelu", stats=stats),
             lambda: pwp.linear(odd, odd[:500]), lambda: pwp.linear(x[:, 3:], w[:, 3:]),
             lambda: pwp.gated_linear(x, w, u, bias_up=b), lambda: pwp.gated_linear(x.float(), w.float(), u.float())]
    flat = lambda y: y if isinstance(y, tuple) else (y,)
    for i, call in enumerate(calls):
        monkeypatch.setattr(B, "_fast", Watch)
        got = flat(call())
        assert taken and taken[-1], i
        monkeypatch.setattr(B, "_fast", B._NoFastCalls)
        want = flat(call())
        for g, e in zip(got, want):
            assert torch.equal(g, e) and g.stride() == e.stride() and g.dtype == e.dtype and g.device == e.device, i
    assert pwp.read_stats(stats).status == 0
    monkeypatch.setattr(B, "_fast", Watch)
    needs = w.clone().requires_grad_()
    other = torch.zeros(80, device="cuda")
    for call, err in [(lambda: pwp.rms_norm(x, w), ValueError), (lambda: pwp.rms_norm(x.half()), TypeError),
                      (lambda: pwp.rms_norm(x, eps=-1.0), ValueError), (lambda: pwp.rms_norm(x.cpu()), ValueError),
                      (lambda: pwp.rms_norm(x, eps=math.nan), ValueError), (lambda: pwp.rms_norm(None), TypeError),
                      (lambda: pwp.linear(x, needs), ValueError), (lambda: pwp.linear(x, w, bias=other), TypeError),
                      (lambda: pwp.linear(x, w, bias=b[:79]), ValueError), (lambda: pwp.linear(x, w.T), ValueError),
                      (lambda: pwp.linear(x, w, residual=r[:1]), ValueError), (lambda: pwp.linear(x, w, bias=b.cpu()), ValueError),
                      (lambda: pwp.linear(x, w, activation="tanh"), ValueError), (lambda: pwp.linear(x, w, stats=b), ValueError),
                      (lambda: pwp.gated_linear(x, w, u[:79]), ValueError),
                      (lambda: pwp.attention(q, k, v[:, :1], cu), ValueError), (lambda: pwp.attention(q, k, v, cu.long()), TypeError),
                      (lambda: pwp.attention(q[:, :3], k, v, cu), ValueError), (lambda: pwp.attention(q, k, v, cu, scale=math.inf), ValueError),
                      (lambda: pwp.qk_norm_rope(q, k, pos[:42], f), ValueError), (lambda: pwp.qk_norm_rope(q, k, pos, f.float()), TypeError),
                      (lambda: pwp.qk_norm_rope(q, k, pos, f, layout="x"), ValueError),
                      (lambda: pwp.qk_norm_rope(q, k, pos, torch.cat([f, f, f])), ValueError)]:
        with pytest.raises(err):
            call()
        assert not taken[-1]
    with torch.no_grad():
        assert torch.equal(pwp.linear(x, needs), pwp.linear(x, w)) and taken[-1]
    assert pwp.rms_norm(x[:0]).shape == (0, 96) and not taken[-1]
    with torch.inference_mode():
        assert pwp.rms_norm(x).is_inference()


def test_waits_that_run_out_are_reported():
    torch, pwp = _torch(), _pwp()
    q, k, v, cu = att_case([200], 2, 1, 128, "bf16", 101)
    w = rnd((512, 512), "bf16", 103)
    xs = [rnd((r, 512), "bf16", 102) for r in (4, 2048)]
    want = [pwp.attention(q, k, v, cu)] + [pwp.linear(x, w) for x in xs]
    torch.cuda.synchronize()
    calls = [(lambda st: pwp.attention(q, k, v, cu, stats=st), 9)] + \
            [(lambda st, x=x: pwp.linear(x, w, stats=st), 10) for x in xs]
    for (call, site), ok in zip(calls, want):
        prev = pwp.set_wait_limit(0)
        try:
            st = pwp.new_stats()
            call(st)
            torch.cuda.synchronize()
        finally:
            pwp.set_wait_limit(prev)
        s = pwp.read_stats(st)
        assert (s.status, s.status_site) == (5, site)
        st = pwp.new_stats()
        assert torch.equal(call(st), ok) and pwp.read_stats(st).status == 0


@pytest.mark.parametrize("gated", [False, True])
def test_waits_that_run_out_with_many_rows(gated):
    """The kernel of CTA pairs, several tiles per pair and more steps of k than stages: either CTA
    may give up first; the rows come out NaN and the next call is right."""
    torch, pwp = _torch(), _pwp()
    x, w, u = rnd((16384, 1024), "bf16", 104), rnd((1000, 1024), "bf16", 105), rnd((1000, 1024), "bf16", 106)
    call = (lambda st=None: pwp.gated_linear(x, w, u, stats=st)) if gated else (lambda st=None: pwp.linear(x, w, stats=st))
    want = call()
    torch.cuda.synchronize()
    for limit in (0, 1, 3):
        prev = pwp.set_wait_limit(limit)
        try:
            st = pwp.new_stats()
            got = call(st)
            torch.cuda.synchronize()
        finally:
            pwp.set_wait_limit(prev)
        s = pwp.read_stats(st)
        assert s.status in ((5,) if limit == 0 else (0, 5)) and (s.status == 0 or s.status_site == 10)
        wrong = got != want
        assert bool(got[wrong].isnan().all()) and bool(wrong.any()) == (s.status == 5)
        st = pwp.new_stats()
        assert torch.equal(call(st), want) and pwp.read_stats(st).status == 0


# ------------------------------------------------------------------- the block

def _block(dtype, heads, kv, width, ff, n, seed=111):
    d = width // heads
    w = {p: rnd(s, dtype, seed + i, 1.5 / math.sqrt(s[1])) for i, (p, s) in enumerate(
        {"q_proj": (heads * d, width), "k_proj": (kv * d, width), "v_proj": (kv * d, width), "o_proj": (width, heads * d),
         "gate_proj": (ff, width), "up_proj": (ff, width), "down_proj": (width, ff)}.items())}
    norms = {"attn": 1 + rnd((width,), dtype, seed + 10, 0.1), "mlp": 1 + rnd((width,), dtype, seed + 11, 0.1),
             "q": 1 + rnd((d,), dtype, seed + 12, 0.1), "k": 1 + rnd((d,), dtype, seed + 13, 0.1)}
    return w, rnd((n, width), dtype, seed + 14), norms


@pytest.mark.parametrize("dtype,tol", [("fp32", 1e-5), ("bf16", 0.03)])
def test_block_forward_matches_the_oracle(dtype, tol):
    """All operators in a row, as a block uses them.  bf16: a dozen roundings of 2^-8 in a row,
    each input's of random sign -- the relative Frobenius error of every activation stays
    within 8 * 2^-8; fp32: sums of a few hundred terms, 1e-5."""
    pwp = _pwp()
    lens = [37, 1, 150]
    w, x, norms = _block(dtype, 8, 2, 512, 1000, sum(lens))
    f, _ = pwp.rope_frequencies(64)
    st = pwp.new_stats()
    acts, out = pwp.block_forward(w, x, lens, heads=8, kv_heads=2, freqs=f, norms=norms, stats=st)
    assert pwp.read_stats(st).status == 0
    want, wout = F.block_forward({p: np64(t) for p, t in w.items()}, np64(x), lens, 8, 2, np64(f),
                                 norms={p: np64(t) for p, t in norms.items()})
    assert set(acts) == {"attn_in", "o_in", "mlp_in", "down_in"}
    for name, got, e in [(m, acts[m], want[m]) for m in acts] + [("out", out, wout)]:
        rel = np.linalg.norm(np64(got) - e) / np.linalg.norm(e)
        assert rel <= tol, (name, rel)


def test_prune_decoder_block():
    """The block's layers are pruned with the activations of the dense pass, exactly as
    prune_block does with them, and the hidden states pass through the pruned layers."""
    torch, pwp = _torch(), _pwp()
    lens = [200, 312]
    w, x, norms = _block("bf16", 4, 2, 256, 640, sum(lens), 131)
    f, _ = pwp.rope_frequencies(64)
    fwd = dict(heads=4, kv_heads=2, freqs=f, norms=norms)
    res, out = pwp.prune_decoder_block(w, x, lens, forward=fwd, method="thanos", pattern="nm", nm=(2, 4), block=64)
    acts, dense = pwp.block_forward(w, x, lens, **fwd)
    want = pwp.prune_block(w, acts, pwp.FEEDS, method="thanos", pattern="nm", nm=(2, 4), block=64)
    for layer in w:
        assert torch.equal(res[layer][0], want[layer][0]) and torch.equal(res[layer][1], want[layer][1])
        assert res[layer][2].pruned == w[layer].numel() // 2
    _, again = pwp.block_forward({p: t[0].bfloat16() for p, t in res.items()}, x, lens, **fwd)
    assert torch.equal(out, again) and not torch.equal(out, dense)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    res2, out2 = pwp.prune_decoder_block(w, x, lens, forward=fwd, stream=s, method="thanos", pattern="nm", nm=(2, 4),
                                         block=64)
    s.synchronize()
    assert torch.equal(out2, out) and all(torch.equal(res2[p][0], res[p][0]) for p in w)


# ------------------------------------------------------------------- activations by themselves

def check_activation(act, dtype, lo, hi, rel, atol, want=None):
    """Relative to the result, in the tails too; few rows and many, alone and times an up product of
    2^20, which lifts a small result over what an absolute bound would forgive.  x has the values
    and a column of ones, the weights pick one: both products are exact, and so are the sums.
    Below the least normal number, 2^-126, the steps of a type stay those at 2^-126 (bf16: 2^-133),
    so a result is rounded by up to u 2^-126 (half of that) there."""
    torch, pwp = _torch(), _pwp()
    pick = lambda k, v: torch.zeros(40, 8, device="cuda").index_fill_(1, torch.tensor([k], device="cuda"), v).to(dt(dtype))
    for count, repeat in ((97, 1), (3001, 2)):
        x = torch.zeros(count * repeat, 8, dtype=dt(dtype), device="cuda")
        x[:, 0] = torch.linspace(lo, hi, count, dtype=torch.float64).to(dt(dtype)).cuda().repeat(repeat)
        x[:, 1] = 1.0
        t = np64(x[:, :1])
        y = F.activation(act, t) if want is None else want(t)
        tol = (np.abs(y) * (rel(t) + U(x.dtype)) + atol(t)) * np.ones((1, 40))
        y = y * np.ones((1, 40))
        least = U(x.dtype) * 2.0 ** -126
        close(pwp.linear(x, pick(0, 1.0), activation=act), y, tol + least, act)
        got = pwp.gated_linear(x, pick(0, 1.0), pick(1, 2.0 ** 20), activation=act)
        close(got, y * 2.0 ** 20, tol * 2.0 ** 20 + least, "gated " + act)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lo,hi", [(-8.0, -3.0), (-12.9, -8.0), (-3.0, 3.0), (3.0, 20.0)])
def test_gelu_in_the_tails(lo, hi, dtype):
    """x Phi(x) relative to itself (c = 2^-24, half a step).  fp32, by erfc(t), t = -x / sqrt 2: t is off by
    c (its rounding) and c / 2 (the constant's), and d ln erfc(t) = -2 t^2 (1 + 1 / (2 t^2)) dt / t at
    most for t > 0.5, so by (x^2 + 2) 1.5 c; erfc to 4 steps (its documented bound), two products.
    bf16, by e^(-x^2/2) and a polynomial good to 2^-20: the exponential to 2 + 1.173 x^2 / 2 steps (its
    documented bound), its argument's rounding x^2 / 2 c, ten more operations of a step each.
    Below the least normal number (2^-126) results have fewer bits."""
    rel = (lambda t: (1.5 * (t * t + 2) + 10) * 2.0 ** -24) if dtype == "fp32" else \
        (lambda t: 2.0 ** -20 + (12 + 0.8365 * t * t) * G)
    check_activation("gelu", dtype, lo, hi, rel, lambda t: np.abs(t) * 2.0 ** -148)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act,lo,hi", [("silu", -20.0, 20.0), ("silu", -91.0, -20.0), ("gelu_tanh", -5.0, 5.0),
                                       ("gelu_tanh", -10.5, -5.0), ("gelu_tanh", 5.0, 200.0)])
def test_logistic_activations_in_the_tails(act, lo, hi, dtype):
    """x / (1 + e^-z) relative to itself, z = x (SiLU) or 2 sqrt(2/pi) (x + 0.044715 x^3), which is off by 6
    half steps (four operations, two constants): |z| 6 2^-24 of the result.  fp32: the exponential to 1
    step (its documented bound), the sum and product to half a step each, the quotient to 2
    (documented).  bf16: the exponential to 2 + 1.173 |z| steps (documented), the others as in fp32.
    Exponentials below the least normal number (2^-126) are off by 2^-149."""
    def z(t):
        return t if act == "silu" else 2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)

    def want(t):           # no sum that cancels
        e = np.exp(-np.abs(z(t)))
        return np.where(z(t) < 0, t * e, t) / (1 + e)
    arg = (lambda t: 0 * t) if act == "silu" else (lambda t: 6 * 2.0 ** -24 * np.minimum(np.abs(z(t)), 90.0))
    rel = (lambda t: arg(t) + 4 * G) if dtype == "fp32" else \
        (lambda t: arg(t) + (7 + 1.173 * np.minimum(np.abs(z(t)), 90.0)) * G)
    check_activation(act, dtype, lo, hi, rel, lambda t: np.abs(t) * 2.0 ** -148, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_of_special_values(dtype):
    """What the formulas give: +inf stays, NaN stays, and at -inf only ReLU has a limit the formula takes."""
    torch, pwp = _torch(), _pwp()
    for rows in (4, 3000):
        x = torch.zeros(rows, 8, dtype=dt(dtype), device="cuda")
        x[:4, 0] = torch.tensor([math.inf, -math.inf, math.nan, -3e38], dtype=dt(dtype))
        w = torch.zeros(40, 8, dtype=dt(dtype), device="cuda")
        w[:, 0] = 1.0
        for act in ACTS:
            y = pwp.linear(x, w, activation=act)
            assert bool((y[0] == math.inf).all()) and bool(y[2].isnan().all()), act
            assert act == "none" or bool((y[3] == 0).all()), act
            assert not bool(y[4:].any())
            if act == "relu":
                assert bool((y[1] == 0).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d", [128, 36])                # registers, and (36 turned of 38) shared memory
def test_rotation_angles_in_fp32(d, layout):
    """Cosines and sines by themselves (q = (1, 0) in every pair), relative to each: sincospif to 2 steps
    (documented: 1 for the sine, 1 for the cosine), the turn by the angle's rest to one rounding, half a
    step.  Near a zero the turn is all there is: at most 2^-23.3, its rest rounded twice and times a
    sine off by two steps (six half steps, 2^-44.7) and its second term (2^-47): 2^-44.  The reduced
    angle's 64-bit error is 4 2^-53 of position * f radians (three roundings, and 1 / 2 pi's)."""
    torch, pwp = _torch(), _pwp()
    n, width = 4000, d + (d == 36) * 2
    pos = torch.arange(n, device="cuda")
    f, _ = pwp.rope_frequencies(d, base=500.0)
    q = torch.zeros(n, 1, width, device="cuda")
    one, other = (slice(0, d // 2), slice(d // 2, d)) if layout == "half" else (slice(0, d, 2), slice(1, d, 2))
    q[..., one] = 1.0
    y = pwp.qk_norm_rope(q, q[:, :0], pos, f, layout=layout)[0]
    angle = np.arange(n)[:, None] * np64(f)[None]
    for got, want in ((y[:, 0, one], np.cos(angle)), (y[:, 0, other], np.sin(angle))):
        close(got, want, np.abs(want) * 2.5 * G + 4 * 2.0 ** -53 * angle + 2.0 ** -44)


def test_forward_mode_tangents_are_refused():
    """Also by the usual calls, which the C++ marshalling takes otherwise."""
    torch, pwp = _torch(), _pwp()
    import torch.autograd.forward_ad as fwd
    x, w = rnd((4, 64), "bf16", 171), rnd((16, 64), "bf16", 172)
    q, pos, (f, _) = rnd((4, 2, 64), "bf16", 173), torch.arange(4, device="cuda"), pwp.rope_frequencies(64)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with fwd.dual_level():
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))
        for call in (lambda g: pwp.rms_norm(g(x)), lambda g: pwp.linear(x, g(w)), lambda g: pwp.gated_linear(g(x), w, w),
                     lambda g: pwp.attention(q, q, g(q), cu), lambda g: pwp.qk_norm_rope(g(q), q, pos, f)):
            with torch.no_grad(), pytest.raises(ValueError, match="forward pass"):
                call(dual)
            call(lambda t: t)


@pytest.mark.parametrize("hq,hk,per", [(2, 2, 128), (8, 2, 32)])
def test_attention_many_items_whose_second_tile_is_empty(hq, hk, per):
    """Sequences of at most one tile of queries (`per` tokens): every item's second tile has no rows, and its
    softmax warps release one item after another without work of their own."""
    pwp = _pwp()
    rng = np.random.default_rng(181)
    lens = rng.integers(1, per + 1, size=900).tolist()
    q, k, v, cu = att_case(lens, hq, hk, 64, "bf16", 182)
    want, size = F.attention(np64(q), np64(k), np64(v), lens, True, spread=True)
    tol = att_tol(q, k, lens, hq, hk, 64, want, size, "bf16")
    for _ in range(3):
        st = pwp.new_stats()
        close(pwp.attention(q, k, v, cu, stats=st), want, tol)
        assert pwp.read_stats(st).status == 0


@pytest.mark.parametrize("dtype,d", [("fp32", 33), ("bf16", 64)])
def test_attention_of_a_few_tokens_among_very_many_sequences(dtype, d):
    """A million offsets, nearly all of empty sequences: the offsets are read a bounded number of times."""
    torch, pwp = _torch(), _pwp()
    nseq, hq, n = 1 << 20, 4, 150
    lens = np.zeros(nseq, dtype=np.int64)
    at = np.random.default_rng(191).choice(nseq, size=50, replace=False)
    lens[at] = 3
    assert lens.sum() == n
    q, k, v, cu = att_case(lens.tolist(), hq, 2, d, dtype, 192)
    few = [3] * 50
    want, size = F.attention(np64(q), np64(k), np64(v), few, True, spread=True)
    st = pwp.new_stats()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    got = pwp.attention(q, k, v, cu, stats=st)
    b.record()
    torch.cuda.synchronize()
    assert pwp.read_stats(st).status == 0
    close(got, want, att_tol(q, k, few, hq, 2, d, want, size, dtype))
    assert a.elapsed_time(b) < 2000.0
    cu[-1] = n + 1                                        # the last sequence leaves the batch
    out = torch.full_like(q, 7.0)
    pwp.attention(q, k, v, cu, out=out, stats=st)
    assert pwp.read_stats(st).status == 1
    first = int(cu[-2])
    assert torch.equal(out[:first], got[:first]) and bool((out[first:] == 7.0).all())


@pytest.mark.parametrize("causal", [True, False])
def test_attention_on_the_cuda_cores_several_tiles_a_cta(causal):
    """More tiles than CTAs: each takes several, of several sequences and heads, in one go."""
    torch, pwp = _torch(), _pwp()
    lens = [300, 0, 64, 1, 65, 130] * 12
    n, hq = sum(lens), 24
    q, k, v, cu = att_case(lens, hq, 2, 20, "fp32", 193, extra=3)
    out = torch.full_like(q, 7.0)
    pwp.attention(q, k, v, cu, causal=causal, out=out)
    assert bool((out[n:] == 7.0).all())
    at = 0
    for length in lens:
        s = slice(at, at + length)
        if length:
            alone = pwp.attention(q[s], k[s], v[s], torch.tensor([0, length], dtype=torch.int32, device="cuda"), causal=causal)
            assert torch.equal(alone, out[s])
        at += length
    want, size = F.attention(np64(q[430:560]), np64(k[430:560]), np64(v[430:560]), [130], causal, spread=True)
    close(out[430:560], want, att_tol(q, k, lens, hq, 2, 20, want, size, "fp32"))


def test_two_graphs_whose_attention_shares_its_work_out():
    """Calls that take the counter's scratch, captured twice and replayed several times on two streams beside
    each other and beside an eager call: each replay clears its own counter."""
    torch, pwp = _torch(), _pwp()
    from post_weight_pruning_b200 import block as B
    lens = [1024] * 8
    cases = [att_case(lens, 16, 8, 64, "bf16", 201 + 3 * i, extra=3) for i in range(3)]
    q, k, v, cu = cases[0]
    args = B.ATTENTION_ARGS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), q.data_ptr(), *q.stride()[:2], *k.stride()[:2],
                                 *v.stride()[:2], *q.stride()[:2], cu.data_ptr(), 0, q.shape[0], len(lens), pwp.BF16, 16, 8, 64,
                                 1, 0.125, 0, 0)
    assert pwp.lib().pwp_attention_workspace_bytes(args) > 0
    want = [pwp.attention(*c)[:8192].clone() for c in cases]
    outs = [torch.empty_like(c[0]) for c in cases]
    for o, c in zip(outs, cases):                        # the first call of each stream's pool is not a captured one
        pwp.attention(*c, out=o)
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for o, c in zip(outs[:2], cases):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pwp.attention(*c, out=o)
        graphs.append(g)
    for _ in range(6):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(2):                               # each graph twice in a row
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            pwp.attention(*cases[2], out=outs[2])
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[:8192], w) and bool((o[8192:] == 7.0).all())


def test_operators_repeat_themselves_exactly():
    """The same bits call after call, whichever CTA took which work."""
    torch, pwp = _torch(), _pwp()
    q, k, v, cu = att_case([1500, 3, 700, 64, 900], 16, 4, 128, "bf16", 211)
    calls = [lambda: pwp.attention(q, k, v, cu), lambda: pwp.attention(q.float(), k.float(), v.float(), cu)]
    for rows, kk, n in ((1, 4096, 1000), (37, 2000, 1544), (300, 1024, 1000), (3000, 512, 1032)):
        x, w, u = rnd((rows, kk), "bf16", 212), rnd((n, kk), "bf16", 213, 0.05), rnd((n, kk), "bf16", 214, 0.05)
        calls += [lambda x=x, w=w: pwp.linear(x, w), lambda x=x, w=w, u=u: pwp.gated_linear(x, w, u),
                  lambda x=x, w=w: pwp.linear(x.float(), w.float())]
    for i, call in enumerate(calls):
        first = call()
        for _ in range(5):
            assert torch.equal(call(), first), i
