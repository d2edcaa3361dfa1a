"""What is measured of the calibration operators: the forward pass of a decoder block that
gives the layers' inputs to the prune (norms, rotated queries and keys, packed causal
attention, projections with their epilogues, the gated feed-forward product).

Sizes are those of the 7B-shaped decoder block this repository prunes (width 4096, 32 heads
of 128, feed-forward width 11008, sequences of 2048 tokens), and generic odd, ragged and
grouped ones.  Lengths, head counts and switches are plain values of a case; every input is
made from the seed alone.
"""
import math

import numpy as np
import torch

own = False   # True: run() calls the library's operators; False: their plain form

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- the cases

def listed():
    return [
        # the norm before a projection, one row: a single token's hidden state
        dict(name="norm_one_row", op="rms_norm", rows=1, width=4096, dtype="bf16", weight=True),
        # the norm over 16 calibration sequences of 2048 tokens
        dict(name="norm_calibration", op="rms_norm", rows=32768, width=4096, dtype="bf16", weight=True),
        # a short prompt with grouped heads, per-head norms, interleaved pairs in half of the
        # head, at far positions of a scaled long context
        dict(name="rope_short_far", op="qk_norm_rope", tokens=37, hq=32, hk=8, d=128, rot=64, layout="interleaved",
             norm=True, scaling="bands", first=900000, dtype="bf16"),
        # queries and keys of 8 calibration sequences, whole head rotated in halves, no norm,
        # as slices of one packed projection output
        dict(name="rope_calibration", op="qk_norm_rope", tokens=16384, hq=32, hk=32, d=128, rot=128, layout="half",
             norm=False, scaling="none", first=0, dtype="bf16"),
        # one short prompt: latency
        dict(name="attn_short", op="attention", lens="129", hq=32, hk=8, d=128, causal=True, dtype="bf16"),
        # calibration prompts of very different lengths packed together, grouped heads
        dict(name="attn_ragged", op="attention", lens="1,777,2048,65,4095,128,1500,3,0,2901", hq=32, hk=8,
             d=128, causal=True, dtype="bf16"),
        # 16 calibration sequences of 2048 tokens, every head its own keys
        dict(name="attn_calibration", op="attention", lens="2048*16", hq=32, hk=32, d=128, causal=True, dtype="bf16"),
        # one token through the output projection, added to the residual stream
        dict(name="linear_one_row", op="linear", rows=1, k=4096, n=4096, bias=False, act="none", residual=True,
             dtype="bf16"),
        # an odd number of tokens through a projection with bias and activation
        dict(name="linear_odd", op="linear", rows=601, k=4096, n=1000, bias=True, act="gelu", residual=False,
             dtype="bf16"),
        # the down projection of 8 calibration sequences, added to the residual stream
        dict(name="linear_calibration", op="linear", rows=16384, k=11008, n=4096, bias=False, act="none",
             residual=True, dtype="bf16"),
        # a few tokens through the gated feed-forward product
        dict(name="gated_few", op="gated_linear", rows=33, k=4096, n=11008, bias=False, act="silu", dtype="bf16"),
        # 8 calibration sequences through the gated feed-forward product
        dict(name="gated_calibration", op="gated_linear", rows=16384, k=4096, n=11008, bias=False, act="silu",
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _lens(case):
    """The sequence lengths of "a,b*times,c"."""
    out = []
    for part in case["lens"].split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


def _dtype(rng):
    return "fp32" if rng.random() < 0.15 else "bf16"


def draw(rng):
    op = rng.choice(["rms_norm", "qk_norm_rope", "attention", "linear", "gated_linear"])
    if op == "rms_norm":
        return dict(op=op, rows=_log(rng, 1, 32768), width=_log(rng, 64, 8192), dtype=_dtype(rng),
                    weight=rng.random() < 0.8)
    if op == "qk_norm_rope":
        hk = rng.choice([1, 2, 4, 8, 32])
        hq = hk * rng.choice([1, 2, 4, 7])
        d = rng.choice([64, 80, 96, 128])
        return dict(op=op, tokens=_log(rng, 1, 32768 * 32 // (hq + hk)), hq=hq, hk=hk, d=d,
                    rot=rng.choice([d, d // 2]), layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "bands", "yarn"]),
                    first=rng.choice([0, 0, _log(rng, 1, 1000000)]), dtype=_dtype(rng))
    if op == "attention":
        dtype = _dtype(rng)
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 5])
        total = _log(rng, 1, 16384 if dtype == "bf16" else 2048)
        lens = []
        while total > 0:
            n = min(total, _log(rng, 1, 8192))
            lens.append(n)
            total -= n
            if rng.random() < 0.1:
                lens.append(0)
        return dict(op=op, lens=",".join(map(str, lens)), hq=hq, hk=hk, d=rng.choice([64, 80, 128, 128]), causal=rng.random() < 0.8,
                    dtype=dtype)
    dtype = _dtype(rng)
    top = 16384 if dtype == "bf16" else 1024
    rows, k, n = _log(rng, 1, top), _log(rng, 64, 8192), _log(rng, 64, 8192)
    if rng.random() < 0.8:   # widths of models are mostly multiples of eight
        k, n = k + -k % 8, n + -n % 8
    mats = 2 if op == "gated_linear" else 1
    rows = min(rows, int((2.9e12 if dtype == "bf16" else 1e11) / (2.0 * mats * k * n)))
    case = dict(op=op, rows=rows, k=k, n=n, bias=rng.random() < 0.4, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                dtype=dtype)
    if op == "linear":
        case["act"] = rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "relu"])
        case["residual"] = rng.random() < 0.5
    return case


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "rms_norm":
        n = case["rows"] * case["width"]
        return {"bytes": 2 * e * n + (e * case["width"] if case["weight"] else 0), "flops": 4 * n}
    if op == "qk_norm_rope":
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["d"]
        small = 8 * case["tokens"] + 4 * case["rot"] + (2 * e * case["d"] if case["norm"] else 0)
        return {"bytes": 2 * e * n + small, "flops": (7 if case["norm"] else 3) * n}
    if op == "attention":
        n = sum(_lens(case))
        pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in _lens(case))
        return {"bytes": 2 * e * n * case["d"] * (case["hq"] + case["hk"]), "flops": 4 * pairs * case["d"] * case["hq"]}
    rows, k, n = case["rows"], case["k"], case["n"]
    mats = 2 if op == "gated_linear" else 1
    byt = rows * k + mats * n * k + rows * n + (mats * n if case["bias"] else 0)
    byt += rows * n if case.get("residual") else 0
    return {"bytes": e * byt, "flops": 2 * mats * rows * n * k}


# ----------------------------------------------------------------------------- inputs

_SCALINGS = {
    "none": None,
    "linear": dict(type="linear", factor=4.0),
    "base": dict(type="base", factor=4.0),
    "bands": dict(type="bands", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_max_positions=8192),
    "yarn": dict(type="yarn", factor=16.0, beta_fast=32.0, beta_slow=1.0, original_max_positions=4096),
}
_BASE = 500000.0
_EPS = 1e-5


def _frequencies(rot, scaling, base=_BASE):
    """(rot/2 angles per position, factor on cosine and sine) in double precision."""
    i = np.arange(0, rot, 2, dtype=np.float64)
    f = base ** (-i / rot)
    s = _SCALINGS[scaling]
    if s is None:
        return f, 1.0
    if s["type"] == "linear":
        return f / s["factor"], 1.0
    if s["type"] == "base":
        return (base * s["factor"] ** (rot / (rot - 2))) ** (-i / rot), 1.0
    if s["type"] == "bands":
        wavelength = 2 * math.pi / f
        lo, hi, n0 = s["low_freq_factor"], s["high_freq_factor"], s["original_max_positions"]
        t = np.clip((n0 / wavelength - lo) / (hi - lo), 0.0, 1.0)
        return (1 - t) * f / s["factor"] + t * f, 1.0
    n0 = s["original_max_positions"]

    def at(turns):   # the pair whose angle makes `turns` turns over n0 positions
        return rot * math.log(n0 / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(at(s["beta_fast"])), 0), min(math.ceil(at(s["beta_slow"])), rot - 1)
    ramp = np.clip((np.arange(rot // 2, dtype=np.float64) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f / s["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(s["factor"]) + 1.0


def _data(case, seed):
    """The inputs of a case: tensors on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    def features(rows, width):
        # hidden states: normal values with 0.5% outlier features (x50, as the calibration
        # activations of the prune)
        x = torch.randn(rows, width, generator=g, device="cuda")
        out = torch.rand(width, generator=g, device="cuda") < 0.005
        return torch.where(out, x * 50.0, x).to(dt)

    op = case["op"]
    if op == "rms_norm":
        x = features(case["rows"], case["width"])
        w = (1.0 + 0.1 * torch.randn(case["width"], generator=g, device="cuda")).to(dt) if case["weight"] else None
        return dict(x=x, weight=w)
    if op == "qk_norm_rope":
        n, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
        packed = normal(n, (hq + 2 * hk) * d)         # the projection's q, k, v side by side
        q = packed[:, :hq * d].view(n, hq, d)
        k = packed[:, hq * d:(hq + hk) * d].view(n, hk, d)
        pos = case["first"] + torch.arange(n, device="cuda", dtype=torch.int64)
        nw = [(1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2)]
        return dict(q=q, k=k, positions=pos, q_weight=nw[0] if case["norm"] else None,
                    k_weight=nw[1] if case["norm"] else None)
    if op == "attention":
        n, d = sum(_lens(case)), case["d"]
        return dict(q=normal(n, case["hq"], d, scale=1.5), k=normal(n, case["hk"], d), v=normal(n, case["hk"], d))
    rows, k, n = case["rows"], case["k"], case["n"]
    data = dict(x=features(rows, k), w=normal(n, k, scale=0.02))
    if op == "gated_linear":
        data["w_up"] = normal(n, k, scale=0.02)
        data["bias_up"] = normal(n) if case["bias"] else None
    else:
        data["residual"] = normal(rows, n) if case["residual"] else None
    data["bias"] = normal(n) if case["bias"] else None
    return data


def prepare(case, seed):
    st = _data(case, seed)
    st["case"] = case
    if case["op"] == "attention":
        st["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(_lens(case))]), dtype=torch.int32, device="cuda")
    if case["op"] == "qk_norm_rope":
        if own:
            import post_weight_pruning_b200 as pwp
            st["freqs"], st["factor"] = pwp.rope_frequencies(case["rot"], base=_BASE, scaling=_SCALINGS[case["scaling"]],
                                                             device="cuda")
        else:
            f, st["factor"] = _frequencies(case["rot"], case["scaling"])
            st["freqs"] = torch.from_numpy(f).cuda()
    return st


# ----------------------------------------------------------------------------- one pass

def run(st):
    return _run_own(st) if own else _PLAIN[st["case"]["op"]](st)


def _run_own(st):
    import post_weight_pruning_b200 as pwp
    case, op = st["case"], st["case"]["op"]
    if op == "rms_norm":
        return pwp.rms_norm(st["x"], st["weight"], eps=_EPS)
    if op == "qk_norm_rope":
        return pwp.qk_norm_rope(st["q"], st["k"], st["positions"], st["freqs"], q_weight=st["q_weight"],
                                k_weight=st["k_weight"], eps=_EPS, layout=case["layout"], factor=st["factor"])
    if op == "attention":
        return pwp.attention(st["q"], st["k"], st["v"], st["cu_seqlens"], causal=case["causal"])
    if op == "linear":
        return pwp.linear(st["x"], st["w"], bias=st["bias"], activation=case["act"], residual=st["residual"])
    return pwp.gated_linear(st["x"], st["w"], st["w_up"], bias_gate=st["bias"], bias_up=st["bias_up"],
                            activation=case["act"])


def _act(name, y):
    if name == "none":
        return y
    if name == "relu":
        return torch.clamp(y, min=0.0)
    if name == "silu":
        return y / (1.0 + torch.exp(-y))
    if name == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))


def _plain_rms_norm(st):
    x = st["x"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    if st["weight"] is not None:
        y = y * st["weight"].float()
    return y.to(st["x"].dtype)


def _plain_qk_norm_rope(st):
    case, rot = st["case"], st["case"]["rot"]
    angle = st["positions"].double()[:, None] * st["freqs"][None]          # far positions need 64 bits
    cos, sin = ((f(angle) * st["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    outs = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * w.float()
        if case["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], dim=-1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2), y[..., rot:]], dim=-1)
        outs.append(z.to(x.dtype))
    return outs


def _plain_attention(st):
    case = st["case"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    out = torch.empty_like(st["q"])
    at = 0
    for n in _lens(case):
        if n == 0:
            continue
        q, k, v = (st[x][at:at + n].float().transpose(0, 1) for x in ("q", "k", "v"))
        hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1) if case["causal"] else None
        for h in range(hk):          # one group of query heads beside its key head at a time
            s = q[h * (hq // hk):(h + 1) * (hq // hk)] @ k[h].T * (d ** -0.5)
            if hidden is not None:
                s = s.masked_fill_(hidden, float("-inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = (p @ v[h]) / p.sum(-1, keepdim=True)
            out[at:at + n, h * (hq // hk):(h + 1) * (hq // hk)] = o.transpose(0, 1).to(out.dtype)
        at += n
    return out


def _plain_linear(st):
    y = st["x"].float() @ st["w"].float().T
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _act(st["case"]["act"], y)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(st["x"].dtype)


def _plain_gated_linear(st):
    x = st["x"].float()
    g, u = x @ st["w"].float().T, x @ st["w_up"].float().T
    if st["bias"] is not None:
        g, u = g + st["bias"].float(), u + st["bias_up"].float()
    return (_act(st["case"]["act"], g) * u).to(st["x"].dtype)


_PLAIN = {"rms_norm": _plain_rms_norm, "qk_norm_rope": _plain_qk_norm_rope, "attention": _plain_attention,
          "linear": _plain_linear, "gated_linear": _plain_gated_linear}


# ----------------------------------------------------------------------------- the definitions in 64 bits

def _exact_act(name, y):
    if name == "silu":
        return y * torch.sigmoid(y)
    if name == "gelu":
        return y * torch.special.ndtr(y)
    if name == "gelu_tanh":
        # (1 + tanh t) / 2 = sigmoid(2 t)
        return y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
    return torch.relu(y) if name == "relu" else y


def _exact_project(x, w, b):
    y = torch.einsum("ik,jk->ij", x.double(), w.double())
    return y if b is None else y + b.double()


def exact(case, seed):
    data, op = _data(case, seed), case["op"]
    if op == "rms_norm":
        x = data["x"].double()
        y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["width"] + _EPS)
        return y if data["weight"] is None else y * data["weight"].double()
    if op == "qk_norm_rope":
        rot, half = case["rot"], case["rot"] // 2
        freqs, factor = _frequencies(rot, case["scaling"])
        # a pair as one complex number, turned by its angle
        turn = torch.polar(torch.full((case["tokens"], 1, half), factor, dtype=torch.float64, device="cuda"),
                           torch.outer(data["positions"].double(), torch.from_numpy(freqs).cuda())[:, None, :])
        outs = []
        for name in ("q", "k"):
            y = data[name].double()
            if case["norm"]:
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / case["d"] + _EPS) * data[name + "_weight"].double()
            first = torch.arange(half, device="cuda") * (1 if case["layout"] == "half" else 2)
            second = first + (half if case["layout"] == "half" else 1)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            outs.append(y)
        return outs
    if op == "attention":
        hq, hk, d = case["hq"], case["hk"], case["d"]
        out = torch.empty(sum(_lens(case)), hq, d, dtype=torch.float64, device="cuda")
        begin = 0
        for n in _lens(case):
            for h in range(hq):
                q, k, v = (data[t][begin:begin + n, i].double() for t, i in (("q", h), ("k", h * hk // hq), ("v", h * hk // hq)))
                for r in range(0, n, 1024):       # rows in pieces, each against the keys it sees
                    e = min(n, r + 1024)
                    seen = e if case["causal"] else n
                    s = torch.einsum("id,jd->ij", q[r:e], k[:seen]) / math.sqrt(d)
                    if case["causal"]:
                        i, j = torch.arange(r, e, device="cuda"), torch.arange(seen, device="cuda")
                        s = torch.where(j[None] <= i[:, None], s, -math.inf)
                    out[begin + r:begin + e, h] = torch.softmax(s, dim=-1) @ v[:seen]
            begin += n
        return out
    g = _exact_project(data["x"], data["w"], data["bias"])
    if op == "gated_linear":
        return _exact_act(case["act"], g).mul_(_exact_project(data["x"], data["w_up"], data["bias_up"]))
    y = _exact_act(case["act"], g)
    return y if data["residual"] is None else y + data["residual"].double()
