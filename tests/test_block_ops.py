"""The decoder block's forward operators without a GPU: the oracle's formulas against
independent computations, the frequency scalings, the binding's refusals and marshalling, and
the C entry points' argument checks."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import post_weight_pruning_b200 as pwp  # noqa: E402
from oracle import forward as F  # noqa: E402
from post_weight_pruning_b200 import block as B  # noqa: E402


# ------------------------------------------------------------------- the oracle

def test_oracle_attention_matches_the_dense_softmax():
    rng = np.random.default_rng(0)
    lens, hq, hk, d = [3, 0, 7, 1], 4, 2, 8
    n = sum(lens)
    q, k, v = (rng.normal(size=(n, h, d)) for h in (hq, hk, hk))
    for causal in (True, False):
        out, size = F.attention(q, k, v, lens, causal, spread=True)
        seq = np.repeat(np.arange(len(lens)), lens)
        sees = seq[:, None] == seq[None]
        if causal:
            sees &= np.arange(n)[:, None] >= np.arange(n)[None]
        for h in range(hq):
            s = torch.from_numpy(q[:, h] @ k[:, h // 2].T / math.sqrt(d))
            p = torch.softmax(s.masked_fill(torch.from_numpy(~sees), -math.inf), -1).numpy()
            np.testing.assert_allclose(out[:, h], p @ v[:, h // 2], rtol=1e-12, atol=1e-14)
            np.testing.assert_allclose(size[:, h], p @ np.abs(v[:, h // 2]), rtol=1e-12)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_oracle_rotation_depends_on_distances_only(layout):
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 12))
    f = F.rope_frequencies(8)
    dots = []
    for shift in (0, 5, 1000):
        a, _ = F.qk_norm_rope(q, q, [shift + 7], f, layout=layout)
        b, _ = F.qk_norm_rope(k, k, [shift + 3], f, layout=layout)
        assert np.array_equal(a[..., 8:], q[..., 8:])
        dots.append(float(np.sum(a * b)))
    assert np.allclose(dots, dots[0], rtol=1e-9)


def test_oracle_activations_match_torch():
    x = torch.linspace(-9, 9, 41, dtype=torch.float64)
    for name, f in (("relu", torch.relu), ("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                    ("gelu_tanh", lambda t: torch.nn.functional.gelu(t, approximate="tanh"))):
        np.testing.assert_allclose(F.activation(name, x.numpy()), f(x).numpy(), rtol=1e-9, atol=1e-14)


# ------------------------------------------------------------------- frequencies

def test_plain_frequencies():
    f, s = pwp.rope_frequencies(16, base=500.0, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0
    np.testing.assert_allclose(f.numpy(), F.rope_frequencies(16, 500.0), rtol=1e-14)
    assert pwp.rope_frequencies(0, device="cpu")[0].shape == (0,)


def test_scaled_frequencies():
    plain = F.rope_frequencies(128)
    f, s = pwp.rope_frequencies(128, scaling=dict(type="linear", factor=4.0), device="cpu")
    np.testing.assert_allclose(f.numpy(), plain / 4, rtol=1e-14)
    f, _ = pwp.rope_frequencies(128, scaling=dict(type="base", factor=4.0), device="cpu")
    assert f[0] == 1.0 and math.isclose(float(f[-1]), plain[-1] / 4, rel_tol=1e-12)
    sc = dict(type="bands", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_max_positions=8192)
    f, s = pwp.rope_frequencies(128, scaling=sc, device="cpu")
    turns = 8192 * plain / (2 * math.pi)
    np.testing.assert_allclose(f.numpy()[turns >= 4], plain[turns >= 4], rtol=1e-14)
    np.testing.assert_allclose(f.numpy()[turns <= 1], plain[turns <= 1] / 8, rtol=1e-14)
    assert np.all(np.diff(f.numpy()) < 0) and s == 1.0
    sc = dict(type="yarn", factor=16.0, original_max_positions=4096)
    f, s = pwp.rope_frequencies(128, scaling=sc, device="cpu")
    assert math.isclose(float(f[0]), 1.0) and math.isclose(float(f[-1]), plain[-1] / 16, rel_tol=1e-12)
    assert math.isclose(s, 0.1 * math.log(16) + 1)


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=-2), dict(rot=4, base=0.0), dict(rot=4, scaling=dict(type="x", factor=2)),
                                dict(rot=4, scaling=dict(type="linear")), dict(rot=2, scaling=dict(type="base", factor=2)),
                                dict(rot=4, scaling=dict(type="linear", factor=2, other=1)),
                                dict(rot=4, scaling=dict(type="bands", factor=2, low_freq_factor=4, high_freq_factor=1,
                                                         original_max_positions=10))])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        pwp.rope_frequencies(**kw, device="cpu")


# ------------------------------------------------------------------- refusals and marshalling

# the argument structures of include/pwp.h, for reading packed calls and driving the C entries
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class RopeArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("q_out", _vp), ("k_out", _vp), ("q_stride", _i64 * 2), ("k_stride", _i64 * 2),
                ("q_out_stride", _i64 * 2), ("k_out_stride", _i64 * 2), ("positions", _vp), ("freqs", _vp),
                ("q_weight", _vp), ("k_weight", _vp), ("n", _i64), ("type", _i32), ("hq", _i32), ("hk", _i32),
                ("d", _i32), ("rot", _i32), ("layout", _i32), ("eps", _f32), ("factor", _f32)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("out", _vp), ("q_stride", _i64 * 2), ("k_stride", _i64 * 2),
                ("v_stride", _i64 * 2), ("out_stride", _i64 * 2), ("cu_seqlens", _vp), ("stats", _vp), ("n", _i64),
                ("nseq", _i32), ("type", _i32), ("hq", _i32), ("hk", _i32), ("d", _i32), ("causal", _i32),
                ("scale", _f32), ("ws", _vp), ("ws_bytes", ctypes.c_size_t)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("w", _vp), ("w_up", _vp), ("bias", _vp), ("bias_up", _vp), ("residual", _vp),
                ("out", _vp), ("x_stride", _i64), ("w_stride", _i64), ("w_up_stride", _i64),
                ("residual_stride", _i64), ("out_stride", _i64), ("stats", _vp), ("rows", _i64), ("k", _i32),
                ("n", _i32), ("type", _i32), ("activation", _i32), ("ws", _vp), ("ws_bytes", ctypes.c_size_t)]


ARGS = {"pwp_qk_norm_rope": RopeArgs, "pwp_attention": AttentionArgs, "pwp_linear": LinearArgs,
        "pwp_linear_workspace_bytes": LinearArgs}


class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("pwp_"):
            raise AttributeError(name)
        if name == "pwp_attention_workspace_bytes":
            return lambda a: 0

        def f(*a):
            self.calls.append((name, [ARGS[name].from_buffer_copy(x) if isinstance(x, bytes) else x for x in a]))
            return 0
        return f


@pytest.fixture
def fake(monkeypatch):
    """The library replaced by a recorder, CPU tensors let through as if they were on a GPU."""
    f = _FakeLib()
    monkeypatch.setattr(pwp, "lib", lambda: f)
    monkeypatch.setattr(B, "_stream_of", lambda dev: 7)
    monkeypatch.setattr(B, "_on_gpu", lambda t: True)
    return f


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_operators_refuse_host_tensors():
    for call in (lambda: pwp.rms_norm(z(2, 4)), lambda: pwp.attention(z(2, 1, 4), z(2, 1, 4), z(2, 1, 4), z(2)),
                 lambda: pwp.linear(z(2, 4), z(3, 4)), lambda: pwp.gated_linear(z(2, 4), z(3, 4), z(3, 4)),
                 lambda: pwp.qk_norm_rope(z(2, 1, 4), z(2, 1, 4), z(2), z(2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        pwp.linear(None, z(3, 4))


CU = torch.zeros(2, dtype=torch.int32)
POS = torch.zeros(2, dtype=torch.int64)
FR = torch.zeros(2, dtype=torch.float64)
POS4 = torch.zeros(4, dtype=torch.int64)


@pytest.mark.parametrize("call, err", [
    (lambda: pwp.rms_norm(z(2, 4, dtype=torch.float16)), TypeError),
    (lambda: pwp.rms_norm(z(2, 4, 1)), ValueError),
    (lambda: pwp.rms_norm(z(4, 2).T), ValueError),
    (lambda: pwp.rms_norm(z(2, 4), z(5)), ValueError),
    (lambda: pwp.rms_norm(z(2, 4), z(4, dtype=torch.float32)), TypeError),
    (lambda: pwp.rms_norm(z(2, 4), eps=-1.0), ValueError),
    (lambda: pwp.rms_norm(z(2, 4), eps=math.inf), ValueError),
    (lambda: pwp.rms_norm(z(2, 4), out=z(1, 4).expand(2, 4)), ValueError),
    (lambda: pwp.rms_norm(z(2, 4).requires_grad_()), ValueError),
    (lambda: pwp.rms_norm(z(2, 0)), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 5), POS, FR), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(3, 3, 4), POS, FR), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS.int(), FR), TypeError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS, FR.float()), TypeError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 2), z(2, 3, 2), POS, FR), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS, FR, layout="quarter"), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS, FR, q_weight=z(3)), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS, FR, factor=math.nan), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), torch.zeros(4, dtype=torch.int64)[::2], FR), ValueError),
    (lambda: pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS, FR, k_out=z(2, 1, 4).expand(2, 3, 4)), ValueError),
    (lambda: pwp.attention(z(2, 3, 4), z(2, 2, 4), z(2, 2, 4), CU), ValueError),
    (lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 1, 4), CU), ValueError),
    (lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU.long()), TypeError),
    (lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU[:0]), ValueError),
    (lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4, dtype=torch.float32), CU), TypeError),
    (lambda: pwp.attention(z(2, 2, 257), z(2, 2, 257), z(2, 2, 257), CU), ValueError),
    (lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU, scale=math.inf), ValueError),
    (lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU, stats=z(8)), ValueError),
    (lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU, out=z(2, 2, 4, dtype=torch.float32)), TypeError),
    (lambda: pwp.linear(z(2, 4), z(3, 5)), ValueError),
    (lambda: pwp.linear(z(2, 4), z(3, 4, dtype=torch.float32)), TypeError),
    (lambda: pwp.linear(z(2, 4), z(4, 3).T), ValueError),
    (lambda: pwp.linear(z(2, 4), z(3, 4), bias=z(4)), ValueError),
    (lambda: pwp.linear(z(2, 4), z(3, 4), residual=z(3, 3)), ValueError),
    (lambda: pwp.linear(z(2, 4), z(3, 4), activation="tanh"), ValueError),
    (lambda: pwp.linear(z(2, 4), z(3, 4), out=z(2, 4)), ValueError),
    (lambda: pwp.linear(z(2, 4), z(3, 4), out=z(1, 3).expand(2, 3)), ValueError),
    (lambda: pwp.linear(z(2, 0), z(3, 0)), ValueError),
    (lambda: pwp.linear(z(2, 4), z(3, 4).requires_grad_()), ValueError),
    (lambda: pwp.gated_linear(z(2, 4), z(3, 4), z(2, 4)), ValueError),
    (lambda: pwp.gated_linear(z(2, 4), z(3, 4), z(3, 4), bias_up=z(2)), ValueError),
])
def test_refusals(fake, call, err):
    with pytest.raises(err):
        call()
    assert not fake.calls


X, PACK, BUF = z(4, 8), z(4, 9, 8), z(200)


@pytest.mark.parametrize("call", [
    lambda: pwp.rms_norm(X[:, :4], out=X[:, 2:6]),
    lambda: pwp.rms_norm(X[:2], out=X[1:3]),
    lambda: pwp.rms_norm(X, BUF[:8], out=BUF[4:36].view(4, 8)),
    lambda: pwp.qk_norm_rope(PACK[:, :3], PACK[:, 3:6], POS4, FR, q_out=PACK[:, 3:6]),
    lambda: pwp.qk_norm_rope(PACK[:, :3], PACK[:, :3], POS4, FR, q_out=PACK[:, :3]),
    lambda: pwp.qk_norm_rope(PACK[:, :3], PACK[:, 3:6], POS4, FR, q_out=PACK[:, 6:], k_out=PACK[:, 6:]),
    lambda: pwp.qk_norm_rope(PACK[:, :3], PACK[:, 3:6], POS4, FR, q_out=PACK[:, 2:5]),
    lambda: pwp.attention(PACK[:, :3], PACK[:, 3:6], PACK[:, 6:], CU, out=PACK[:, :3]),
    lambda: pwp.attention(PACK[:, :3], PACK[:, 3:6], PACK[:, 6:], CU, out=PACK[:, 5:8]),
    lambda: pwp.linear(X, z(8, 8), out=X),
    lambda: pwp.linear(X, z(8, 8), residual=BUF[:32].view(4, 8), out=BUF[8:40].view(4, 8)),
    lambda: pwp.linear(z(8, 8), X, out=BUF[:32].view(8, 4), bias=BUF[30:34]),
    lambda: pwp.gated_linear(z(2, 8), z(8, 8), z(8, 8), out=z(2, 8).requires_grad_()),
])
def test_outputs_that_overlap_are_refused(fake, call):
    with pytest.raises(ValueError, match="overlaps|forward pass"):
        call()
    assert not fake.calls


def test_outputs_beside_their_inputs(fake):
    q, k, v = PACK[:, :3], PACK[:, 3:6], PACK[:, 6:]
    pwp.qk_norm_rope(q, k, POS4, FR, q_out=q, k_out=k)
    pwp.qk_norm_rope(q, k, POS4, FR, q_out=q.view(4, 3, 8), k_out=v)
    pwp.qk_norm_rope(PACK[:1, :3], PACK[:1, 3:6], POS4[:1], FR, q_out=PACK[:1, :3], k_out=PACK[:1, 3:6])
    inner = z(4, 3, 2, 8)                                # q and k of a head side by side
    pwp.qk_norm_rope(inner[:, :, 0], inner[:, :, 1], POS4, FR, q_out=inner[:, :, 0], k_out=inner[:, :, 1])
    heads = z(6, 4, 8)                                   # head-major
    pwp.qk_norm_rope(heads[:3].transpose(0, 1), heads[3:].transpose(0, 1), POS4, FR,
                     q_out=heads[:3].transpose(0, 1), k_out=heads[3:].transpose(0, 1))
    room = z(4, 12, 8)
    pwp.attention(room[:, :3], room[:, 3:6], room[:, 6:9], CU, out=room[:, 9:])
    wide = z(4, 24)
    pwp.linear(wide[:, :8], z(8, 8), out=wide[:, 8:16], residual=wide[:, 16:])
    pwp.linear(wide[:, :8], z(8, 8), out=wide[:, 8:16], residual=wide[:, 8:16])
    pwp.rms_norm(wide[:, :8], out=wide[:, :8])
    assert len(fake.calls) == 9


def test_stream_of_another_device_is_refused(fake, monkeypatch):
    class Stream:
        device_index = 1
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    for call in (lambda s: pwp.rms_norm(z(2, 4), stream=s), lambda s: pwp.linear(z(2, 4), z(3, 4), stream=s),
                 lambda s: pwp.gated_linear(z(2, 4), z(3, 4), z(3, 4), stream=s),
                 lambda s: pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU, stream=s),
                 lambda s: pwp.qk_norm_rope(z(2, 1, 4), z(2, 1, 4), POS, FR, stream=s)):
        with pytest.raises(ValueError, match="device"):
            call(Stream())
    assert not fake.calls


def test_no_grad_lets_parameters_through(fake):
    with torch.no_grad():
        pwp.linear(z(2, 4), z(3, 4).requires_grad_())
    assert [name for name, _ in fake.calls].count("pwp_linear") == 1


def test_calls_without_rows_launch_nothing(fake):
    assert pwp.rms_norm(z(0, 4)).shape == (0, 4)
    assert pwp.linear(z(0, 4), z(3, 4)).shape == (0, 3)
    assert pwp.attention(z(0, 2, 4), z(0, 2, 4), z(0, 2, 4), CU).shape == (0, 2, 4)
    assert pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU[:1]).shape == (2, 2, 4)
    q, k = pwp.qk_norm_rope(z(0, 2, 4), z(0, 1, 4), POS[:0], FR)
    assert q.shape == (0, 2, 4) and k.shape == (0, 1, 4)
    assert not fake.calls


def test_marshalling(fake):
    packed = z(5, 40)
    q, k, v = packed[:, :16].view(5, 2, 8), packed[:, 16:24].view(5, 1, 8), packed[:, 32:].view(5, 1, 8)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    out = pwp.attention(q, k, v, cu, causal=False)
    a = fake.calls[-1][1][0]
    assert fake.calls[-1][0] == "pwp_attention"
    assert (a.q, a.k, a.v, a.out, a.cu_seqlens) == tuple(t.data_ptr() for t in (q, k, v, out, cu))
    assert list(a.q_stride) == [40, 8] and list(a.v_stride) == [40, 8] and list(a.out_stride) == [16, 8]
    assert (a.n, a.nseq, a.type, a.hq, a.hk, a.d, a.causal) == (5, 2, pwp.BF16, 2, 1, 8, 0)
    assert a.stats is None and math.isclose(a.scale, 8 ** -0.5, rel_tol=1e-6)

    pos = torch.arange(5)
    fr = torch.ones(2, dtype=torch.float64)
    w = z(8)
    qo, ko = pwp.qk_norm_rope(q, k, pos, fr, k_weight=w, layout="interleaved", factor=1.5, q_out=q)
    a = fake.calls[-1][1][0]
    assert qo is q and a.q_out == q.data_ptr() and a.k_out == ko.data_ptr() and ko.shape == (5, 1, 8)
    assert (a.rot, a.layout, a.q_weight, a.k_weight, a.factor) == (4, 1, None, w.data_ptr(), 1.5)

    x, wg, wu, b, r = z(3, 4), z(6, 4), z(6, 4), z(6), z(3, 6)
    pwp.linear(x, wg, bias=b, activation="gelu", residual=r, out=r)
    a = fake.calls[-1][1][0]
    assert (a.w_up, a.bias, a.residual, a.out) == (None, b.data_ptr(), r.data_ptr(), r.data_ptr())
    assert (a.rows, a.k, a.n, a.activation, a.out_stride) == (3, 4, 6, 3, 6)
    pwp.gated_linear(x, wg, wu, bias_up=b)
    a = fake.calls[-1][1][0]
    assert (a.w, a.w_up, a.bias, a.bias_up, a.activation) == (wg.data_ptr(), wu.data_ptr(), None, b.data_ptr(), 2)
    pwp.rms_norm(x, eps=0.5)
    assert fake.calls[-1][0] == "pwp_rms_norm" and fake.calls[-1][1][6] == 0.5


def test_misaligned_operands_get_scratch(fake, monkeypatch):
    sizes = []
    monkeypatch.setattr(_FakeLib, "pwp_linear_workspace_bytes", lambda self, a: sizes.append(a) or 512, raising=False)
    x = z(3, 24)[:, 1:17]
    pwp.linear(x, z(8, 16))
    a = fake.calls[-1][1][0]
    assert len(sizes) == 1 and a.ws and a.ws_bytes == 512
    pwp.linear(z(3, 16), z(8, 16))
    a = fake.calls[-1][1][0]
    assert a.x % 16 or (len(sizes) == 1 and a.ws is None and a.ws_bytes == 0)


def test_workspace_bytes_of_misaligned_operands():
    L = pwp.lib()

    def need(**kw):
        a = LinearArgs(x=256, w=256, out=256, rows=300, k=1001, n=400, x_stride=1008, w_stride=1008, out_stride=400)
        for key, val in kw.items():
            setattr(a, key, val)
        return L.pwp_linear_workspace_bytes(bytes(a))
    assert need() == 0
    assert need(x_stride=1001) == (300 * 1008 * 2 + 255) // 256 * 256
    assert need(w=258) == (400 * 1008 * 2 + 255) // 256 * 256
    assert need(w_stride=1001, w_up=256, w_up_stride=1001) == 2 * ((400 * 1008 * 2 + 255) // 256 * 256)
    assert need(x_stride=1001, rows=1) == 0                 # too little work, and one row has no stride
    assert need(x_stride=1001, type=1) == 0 and need(k=0) == 0
    a = LinearArgs(x=256, w=256, out=256, rows=2, k=4, n=4, x_stride=4, w_stride=4, out_stride=4, ws=264, ws_bytes=99)
    assert L.pwp_linear(bytes(a), None) == 3


def test_large_batches_get_a_counter(fake, monkeypatch):
    asked = []
    monkeypatch.setattr(_FakeLib, "pwp_attention_workspace_bytes", lambda self, a: asked.append(a) or 256, raising=False)
    q, cu = z(5, 2, 8), torch.tensor([0, 5], dtype=torch.int32)
    pwp.attention(q, q, q, cu)
    a = fake.calls[-1][1][0]
    assert len(asked) == 1 and a.ws and a.ws_bytes == 256


def test_workspace_bytes_of_attention():
    L = pwp.lib()

    def need(**kw):
        a = AttentionArgs(q=256, k=256, v=256, out=256, cu_seqlens=256, n=2048, nseq=1, hq=32, hk=32, d=128, scale=0.1)
        for key, val in kw.items():
            setattr(a, key, val)
        return L.pwp_attention_workspace_bytes(bytes(a))
    assert need() == 256                                    # 8 or 9 tile pairs of 32 heads
    assert need(n=700) == 0 and need(n=0) == 0              # one round of work
    assert need(n=32768, nseq=16) == 0 and need(nseq=5) == 0      # many rounds, short sequences
    assert need(type=1) == 0 and need(d=136) == 0 and need(d=0) == 0 and need(scale=-1.0) == 0
    a = AttentionArgs(q=256, k=256, v=256, out=256, cu_seqlens=256, n=8, nseq=1, hq=1, hk=1, d=8, scale=1.0, ws=264, ws_bytes=256)
    assert L.pwp_attention(bytes(a), None) == 3


def test_block_forward_refusals(fake):
    w = {p: z(8, 8) for p in B.FEEDS}
    with pytest.raises(ValueError, match="missing"):
        pwp.block_forward({}, z(4, 8), [4], heads=1)
    with pytest.raises(ValueError, match="seq_lens"):
        pwp.block_forward(w, z(4, 8), [3], heads=1)
    with pytest.raises(ValueError, match="seq_lens"):
        pwp.block_forward(w, z(4, 8), [5, -1], heads=1)
    with pytest.raises(ValueError, match="heads"):
        pwp.block_forward(w, z(4, 8), [4], heads=3)
    with pytest.raises(ValueError, match="norms"):
        pwp.block_forward(w, z(4, 8), [4], heads=1, norms={"x": z(8)})
    with pytest.raises(ValueError, match="biases"):
        pwp.block_forward(w, z(4, 8), [4], heads=1, biases={"x": z(8)})


def test_struct_sizes_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "pwp.h"\nint main(void) { printf("%zu %zu %zu\\n", sizeof(pwp_rope_args), '
                   'sizeof(pwp_attention_args), sizeof(pwp_linear_args)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [s.size for s in (B.ROPE_ARGS, B.ATTENTION_ARGS, B.LINEAR_ARGS)]
    assert [int(x) for x in got] == [ctypes.sizeof(t) for t in (RopeArgs, AttentionArgs, LinearArgs)]


def test_c_entry_points_check_their_arguments():
    L = pwp.lib()
    p = ctypes.c_void_p(256)   # never dereferenced: every call below is refused first

    def rms(rows=1, width=4, eps=1e-5, x=p, os=4, type=0):
        return L.pwp_rms_norm(x, type, rows, width, 4, None, eps, p, os, None)
    assert rms(rows=-1) == rms(width=0) == rms(eps=-1.0) == rms(eps=math.nan) == rms(x=None) == rms(type=2) == 1
    assert rms(rows=2, os=3) == 1 and rms(rows=0) == 0

    def att(**kw):
        a = AttentionArgs(q=256, k=256, v=256, out=256, cu_seqlens=256, n=4, nseq=1, type=0, hq=2, hk=1, d=8,
                            causal=1, scale=1.0)
        for key, val in kw.items():
            setattr(a, key, val)
        return L.pwp_attention(bytes(a), None)
    for kw in (dict(hq=3, hk=2), dict(hk=0), dict(d=257), dict(d=0), dict(n=-1), dict(n=1 << 31), dict(nseq=-1),
               dict(scale=math.inf), dict(q=None), dict(cu_seqlens=None), dict(type=3)):
        assert att(**kw) == 1, kw
    assert att(n=0) == att(nseq=0) == 0 and L.pwp_attention(None, None) == 1

    def lin(**kw):
        a = LinearArgs(x=256, w=256, out=256, rows=2, k=4, n=4, x_stride=4, w_stride=4, out_stride=4)
        for key, val in kw.items():
            setattr(a, key, val)
        return L.pwp_linear(bytes(a), None)
    for kw in (dict(rows=-1), dict(k=0), dict(n=0), dict(k=1 << 24), dict(activation=5), dict(activation=-1), dict(x=None),
               dict(bias_up=256), dict(out_stride=3), dict(type=9)):
        assert lin(**kw) == 1, kw
    assert lin(rows=0) == 0 and L.pwp_linear(None, None) == 1

    def rope(**kw):
        a = RopeArgs(q=256, k=256, q_out=256, k_out=256, positions=256, freqs=256, n=1, hq=1, hk=1, d=8, rot=8,
                       eps=1e-5, factor=1.0)
        for key, val in kw.items():
            setattr(a, key, val)
        return L.pwp_qk_norm_rope(bytes(a), None)
    for kw in (dict(rot=7), dict(rot=10), dict(d=0), dict(d=1025), dict(layout=2), dict(hq=-1), dict(n=-1), dict(q=None),
               dict(freqs=None), dict(eps=-1.0), dict(factor=math.inf)):
        assert rope(**kw) == 1, kw
    assert rope(n=0) == 0 and L.pwp_qk_norm_rope(None, None) == 1


# ------------------------------------------------------------------- the same tensor twice

SQ = z(8, 8)


@pytest.mark.parametrize("call", [
    lambda: pwp.linear(SQ, z(8, 8), residual=SQ, out=SQ),              # rows of x that other tiles still read
    lambda: pwp.linear(z(8, 8), SQ, residual=SQ, out=SQ),
    lambda: pwp.qk_norm_rope(PACK[:, :3], PACK[:, :3], POS4, FR, q_out=PACK[:, :3], k_out=PACK[:, :3]),
])
def test_outputs_over_a_tensor_given_twice_are_refused(fake, call):
    with pytest.raises(ValueError, match="overlaps"):
        call()
    assert not fake.calls


def test_queries_given_as_keys_too(fake):
    """One tensor as q and k: in place it is read and written at once; apart it may be given."""
    q = z(4, 3, 8)
    for kw in (dict(q_out=q), dict(k_out=q), dict(q_out=q, k_out=q), dict(q_out=q, k_out=z(4, 3, 8))):
        with pytest.raises(ValueError, match="overlaps"):
            pwp.qk_norm_rope(q, q, POS4, FR, **kw)
    assert not fake.calls
    pwp.qk_norm_rope(q, q, POS4, FR)
    pwp.qk_norm_rope(q, q, POS4, FR, q_out=z(4, 3, 8))
    pwp.linear(SQ, z(8, 8), residual=SQ)
    assert len(fake.calls) == 3


# ------------------------------------------------------------------- derivatives

def test_forward_mode_tangents_are_refused(fake):
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        dual = lambda *shape: fwd.make_dual(z(*shape), z(*shape))
        for recording in (True, False):
            with torch.set_grad_enabled(recording):
                for call in (lambda: pwp.rms_norm(dual(2, 4)), lambda: pwp.rms_norm(z(2, 4), dual(4)),
                             lambda: pwp.rms_norm(z(2, 4), out=dual(2, 4)),
                             lambda: pwp.qk_norm_rope(z(2, 3, 4), dual(2, 3, 4), POS, FR),
                             lambda: pwp.attention(z(2, 2, 4), z(2, 2, 4), dual(2, 2, 4), CU),
                             lambda: pwp.linear(z(2, 4), dual(3, 4)), lambda: pwp.linear(z(2, 4), z(3, 4), residual=dual(2, 3)),
                             lambda: pwp.gated_linear(z(2, 4), z(3, 4), dual(3, 4))):
                    with pytest.raises(ValueError, match="forward pass"):
                        call()
        assert not fake.calls
        pwp.rms_norm(z(2, 4))                # a level alone, and what a dual was made of, are no matter
        pwp.rms_norm(fwd.unpack_dual(dual(2, 4)).primal)
    assert len(fake.calls) == 2


def test_frequencies_that_require_a_gradient_are_refused(fake):
    with pytest.raises(ValueError, match="forward pass"):
        pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS, FR.clone().requires_grad_())
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level(), pytest.raises(ValueError, match="forward pass"):
        pwp.qk_norm_rope(z(2, 3, 4), z(2, 3, 4), POS, fwd.make_dual(FR, FR))
    assert not fake.calls


# ------------------------------------------------------------------- frequencies between the ends

def test_yarn_leaves_short_contexts_their_factor():
    for s in (0.5, 1.0):
        sc = dict(type="yarn", factor=s, original_max_positions=4096)
        assert pwp.rope_frequencies(64, scaling=sc, device="cpu")[1] == 1.0
    sc["factor"] = 1.5
    assert math.isclose(pwp.rope_frequencies(64, scaling=sc, device="cpu")[1], 0.1 * math.log(1.5) + 1, rel_tol=1e-15)


def test_scaled_frequencies_on_the_ramp():
    rot, base, s, n0 = 64, 500.0, 8.0, 2000
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    sc = dict(type="bands", factor=s, low_freq_factor=1.0, high_freq_factor=5.0, original_max_positions=n0)
    f, between = pwp.rope_frequencies(rot, base=base, scaling=sc, device="cpu")[0], 0
    for i, p in enumerate(plain):
        turns = n0 * p / (2 * math.pi)
        t = min(max((turns - 1.0) / 4.0, 0.0), 1.0)
        between += 0 < t < 1
        assert math.isclose(float(f[i]), t * p + (1 - t) * p / s, rel_tol=1e-13), i
    assert between >= 3
    sc["low_freq_factor"] = 0                  # a ramp from the slowest pairs on
    f = pwp.rope_frequencies(rot, base=base, scaling=sc, device="cpu")[0]
    t = min(n0 * plain[-1] / (2 * math.pi) / 5.0, 1.0)
    assert math.isclose(float(f[-1]), t * plain[-1] + (1 - t) * plain[-1] / s, rel_tol=1e-13)
    # pairs that make 32 turns and 1 turn over the positions, rounded outwards
    sc = dict(type="yarn", factor=s, original_max_positions=n0)
    place = lambda turns: rot / 2 * math.log(n0 / (2 * math.pi * turns)) / math.log(base)
    lo, hi = math.floor(place(32.0)), math.ceil(place(1.0))
    assert 0 < lo < hi - 3 and hi < rot // 2
    f = pwp.rope_frequencies(rot, base=base, scaling=sc, device="cpu")[0]
    for i, p in enumerate(plain):
        t = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert math.isclose(float(f[i]), (1 - t) * p + t * p / s, rel_tol=1e-13), i


@pytest.mark.parametrize("sc", [
    dict(type="yarn", factor=2), dict(type="yarn", factor=2, original_max_positions=-5),
    dict(type="yarn", factor=2, original_max_positions=0), dict(type="yarn", factor=2, original_max_positions=9, beta_fast=0),
    dict(type="yarn", factor=2, original_max_positions=9, beta_slow=-1), dict(type="yarn", factor=math.inf, original_max_positions=9),
    dict(type="bands", factor=2, low_freq_factor=1, high_freq_factor=4),
    dict(type="bands", factor=2, low_freq_factor=1, original_max_positions=10),
    dict(type="bands", factor=2, low_freq_factor=1, high_freq_factor=4, original_max_positions=-10),
    dict(type="linear", factor=math.nan), dict(type="linear", factor=math.inf)])
def test_scalings_without_their_entries_are_refused(sc):
    with pytest.raises(ValueError, match="scaling"):
        pwp.rope_frequencies(16, scaling=sc, device="cpu")


def test_bases_out_of_range_are_refused():
    for kw in (dict(base=math.inf), dict(base=math.nan), dict(base=1.0, scaling=dict(type="yarn", factor=2, original_max_positions=9))):
        with pytest.raises(ValueError, match="base"):
            pwp.rope_frequencies(16, **kw, device="cpu")


def test_the_dense_activations_are_free_before_the_second_pass(monkeypatch):
    import weakref
    alive = []

    def block_forward(weights, hidden, seq_lens, **kw):
        alive.append(sum(r() is not None for r in refs))
        acts = {name: z(4, 8) for name in set(B.FEEDS.values())}
        refs.extend(weakref.ref(t) for t in acts.values())
        return acts, hidden
    refs = []
    monkeypatch.setattr(B, "block_forward", block_forward)
    monkeypatch.setattr(pwp, "prune_block", lambda weights, acts, feeds, **kw: {p: (w, None, None) for p, w in weights.items()})
    results, out = pwp.prune_decoder_block({p: z(8, 8) for p in B.FEEDS}, z(4, 8), [4], forward={})
    assert set(results) == set(B.FEEDS) and alive == [0, 0]


BLOCK_W = {p: z(8, 8) for p in B.FEEDS}
BLOCK_CALLS = [lambda **kw: pwp.block_forward(BLOCK_W, z(4, 8), [4], heads=1, **kw),
               lambda **kw: pwp.prune_decoder_block(BLOCK_W, z(4, 8), [4], forward=dict(heads=1), **kw)]


@pytest.mark.parametrize("call", BLOCK_CALLS)
def test_the_block_refuses_a_stream_of_another_device(fake, monkeypatch, call):
    class Stream:
        device_index = 1
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(pwp, "_stream_ctx", lambda s: pytest.fail("entered"))
    with pytest.raises(ValueError, match="stream of device 1"):
        call(stream=Stream())
    assert not fake.calls


@pytest.mark.parametrize("call", BLOCK_CALLS)
def test_the_block_runs_on_its_tensors_device(fake, monkeypatch, call):
    """From another current device every kernel, the prune's among them, is launched on the tensors' one."""
    import contextlib
    current, seen = [1], []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(B, "_current_device", lambda: current[-1])

    @contextlib.contextmanager
    def device(d):
        current.append(0)
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "device", device)

    def prune_block(weights, acts, feeds, **kw):
        seen.append(current[-1])
        return {p: (w, None, None) for p, w in weights.items()}
    monkeypatch.setattr(pwp, "prune_block", prune_block)
    record = B._stream_of
    monkeypatch.setattr(B, "_stream_of", lambda dev: seen.append(current[-1]) or record(dev))
    monkeypatch.setattr(B, "_fast", B._NoFastCalls)
    call()
    assert len(seen) >= 8 and set(seen) == {0} and current == [1]


def test_a_gated_product_needs_both_weights(fake):
    for kw in (dict(), dict(out=z(2, 3))):
        with pytest.raises(TypeError, match="w_up"):
            pwp.gated_linear(z(2, 4), z(3, 4), None, **kw)
    assert not fake.calls


def test_status_records_off_their_alignment_are_refused(fake):
    """The kernels' atomics on one would fault; slices of a buffer of records at its multiples may be given."""
    size = ctypes.sizeof(pwp.Stats)
    buf = torch.zeros(3 * size + 64, dtype=torch.uint8)
    at = -buf.data_ptr() % 64
    for off in (1, 2, 4, size + 4):
        rec = buf[at + off:at + off + size]
        with pytest.raises(ValueError, match="stats"):
            pwp.attention(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), CU, stats=rec)
        with pytest.raises(ValueError, match="stats"):
            pwp.linear(z(2, 4), z(3, 4), stats=rec)
    assert not fake.calls
    pwp.linear(z(2, 4), z(3, 4), stats=buf[at + size:at + 2 * size])
    assert len([name for name, _ in fake.calls if name == "pwp_linear"]) == 1


def test_c_entry_points_check_the_record():
    L = pwp.lib()
    a = AttentionArgs(q=256, k=256, v=256, out=256, cu_seqlens=256, stats=260, nseq=0, hq=1, hk=1, d=8, scale=1.0)
    assert L.pwp_attention(bytes(a), None) == 1
    a.stats = 264
    assert L.pwp_attention(bytes(a), None) == 0                  # no sequences: nothing is enqueued
    a = LinearArgs(rows=0, k=4, n=4, stats=260)
    assert L.pwp_linear(bytes(a), None) == 1
    a.stats = 264
    assert L.pwp_linear(bytes(a), None) == 0


ROOM = torch.zeros(4096, dtype=torch.uint8)
ROOM = ROOM[-ROOM.data_ptr() % 64:]
OUT = ROOM[256:384].view(torch.bfloat16)                    # 64 elements


@pytest.mark.parametrize("call", [
    lambda at: pwp.qk_norm_rope(z(4, 2, 8), z(4, 2, 8), ROOM[at:at + 32].view(torch.int64), FR, q_out=OUT.view(4, 2, 8)),
    lambda at: pwp.qk_norm_rope(z(4, 2, 8), z(4, 2, 8), ROOM[at:at + 32].view(torch.int64), FR, k_out=OUT.view(4, 2, 8)),
    lambda at: pwp.qk_norm_rope(z(4, 2, 8), z(4, 2, 8), POS4, ROOM[at:at + 32].view(torch.float64), k_out=OUT.view(4, 2, 8)),
    lambda at: pwp.attention(z(4, 2, 8), z(4, 2, 8), z(4, 2, 8), ROOM[at:at + 32].view(torch.int32), out=OUT.view(4, 2, 8)),
    lambda at: pwp.attention(z(4, 2, 8), z(4, 2, 8), z(4, 2, 8), CU, stats=ROOM[at:at + ctypes.sizeof(pwp.Stats)],
                             out=OUT.view(4, 2, 8)),
    lambda at: pwp.linear(z(4, 8), z(16, 8), stats=ROOM[at:at + ctypes.sizeof(pwp.Stats)], out=OUT.view(4, 16)),
])
def test_outputs_over_what_the_call_reads_on_the_device_are_refused(fake, call):
    """Positions, frequencies, offsets and the status record, whose elements have other sizes."""
    for at in (232, 256, 352, 376):                   # 32 bytes or a record against bytes 256 .. 384
        with pytest.raises(ValueError, match="overlaps"):
            call(at)
    assert not fake.calls
    for at in (192, 384):
        call(at)
    assert len(fake.calls) >= 2


def test_negated_views_are_refused(fake):
    """Their memory holds the values with the other sign."""
    x = torch.zeros(2, 1, dtype=torch.complex64).conj().imag
    assert x.is_neg()
    f = lambda *shape: z(*shape, dtype=torch.float32)
    for call in (lambda: pwp.rms_norm(x), lambda: pwp.rms_norm(f(2, 1), out=x), lambda: pwp.linear(x, f(3, 1)),
                 lambda: pwp.linear(f(4, 1), x), lambda: pwp.attention(f(2, 1, 1), x[:, None], f(2, 1, 1), CU)):
        with pytest.raises(ValueError, match="negated"):
            call()
    assert not fake.calls
    pwp.rms_norm(x.resolve_neg())
    assert len(fake.calls) == 1
