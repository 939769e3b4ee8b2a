"""Workloads of the operators on packed rows in eight bits and of the rotary map: the norm with the residual's
addition (kvr_rows_norm), the gated activation (kvr_rows_swiglu), rows stored and read back (kvr_rows_quantise,
kvr_rows_dequantise), the projection of 8-bit rows by 8-bit weights (kvr_linear) and the rotation of query and key
heads (kvr_rows_rotate).

listed() names the cases, draw() gives more of the same ranges, prepare() builds what a serving or repair loop holds
before the call, run() is one pass (the library's calls where `own` is true, elementary torch operations otherwise),
exact() the same outputs from the definitions in float64.
"""
import math

import torch

own = False

# d_model, query heads, K/V heads, head_dim, FFN width of the models the workloads use
MODELS = {"llama8b": (4096, 32, 8, 128, 14336), "qwen7b": (3584, 28, 4, 128, 18944),
          "qwen1p5b": (1536, 12, 2, 128, 8960), "tiny": (256, 4, 4, 64, 1024)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name=None, **kw):
    base = {"norm": dict(rows=1, d=4096, type="bf16", residual=True),
            "swiglu": dict(rows=1, d=14336, type="bf16"),
            "store": dict(rows=1, d=4096, type="bf16"),
            "linear": dict(rows=1, k=4096, n=4096, out="bf16", bias=False),
            "rotate": dict(rows=1, hq=32, hkv=8, dh=128, rot=128, layout="half", scaling="plain", type="bf16",
                           far=8192)}[kw["op"]]
    c = dict(base, **kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token's residual addition and norm before its projection: latency counts
        _case("norm step", op="norm", rows=1, d=4096),
        # the whole retained suffix of an 8K context
        _case("norm suffix", op="norm", rows=5632, d=4096),
        # fp32 rows of an odd width, nothing added
        _case("norm odd f32", op="norm", rows=333, d=5001, type="f32", residual=False),
        # a 5 % refresh's rows before the down projection
        _case("swiglu refresh", op="swiglu", rows=282, d=14336),
        # a prompt's rows, the widest feed-forward layer
        _case("swiglu prompt", op="swiglu", rows=4097, d=18944),
        # the boundary states of four adapter-drift sequences, stored in 8 bits and read back
        _case("store boundary", op="store", rows=4 * 24576, d=1536),
        # one decode step's fused q, k, v projection
        _case("linear step", op="linear", rows=1, k=4096, n=6144),
        # a serving batch's down projection
        _case("linear batch", op="linear", rows=64, k=14336, n=4096),
        # the refreshed rows' q, k, v projection with biases, fp32 out, more rows than a tile
        _case("linear refresh", op="linear", rows=282, k=3584, n=4608, out="f32", bias=True),
        # a prompt through gate and up: the largest product
        _case("linear prompt", op="linear", rows=7680, k=4096, n=28672),
        # a decode batch: neighbouring dims paired, part of the head turned
        _case("rotate step", op="rotate", rows=64, hq=12, hkv=2, rot=64, layout="interleaved", far=32768),
        # a prompt far beyond the trained length, wavelengths banded
        _case("rotate prompt", op="rotate", rows=7680, scaling="bands", far=131072),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "store", "linear", "linear", "linear", "rotate", "rotate"])
    m = MODELS[rng.choice(sorted(MODELS))]
    if op == "linear":
        d, hq, hkv, dh, f = m
        k, n = rng.choice([(d, (hq + 2 * hkv) * dh), (hq * dh, d), (d, 2 * f), (f, d), (_log(rng, 64, 18944), _log(rng, 64, 28672))])
        rows = min(_log(rng, 1, 7680), 7680 * 4096 * 28672 // (k * n))
        return _case(op=op, rows=rows, k=k, n=n, out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.4)
    if op == "rotate":
        dh = rng.choice([64, 80, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        return _case(op=op, rows=_log(rng, 1, 16384), hq=hkv * rng.choice([1, 4, 6, 7]), hkv=hkv, dh=dh,
                     rot=rng.choice([dh, dh, dh // 2, dh // 4]), layout=rng.choice(["half", "interleaved"]),
                     scaling=rng.choice(["plain", "linear", "ntk", "bands", "yarn"]),
                     type=rng.choice(["bf16", "bf16", "f32"]), far=rng.choice([4096, 32768, 1000000]))
    width = rng.choice([m[0], m[4], _log(rng, 64, 18944)])
    rows = min(_log(rng, 1, 32768), (1 << 27) // width)
    c = _case(op=op, rows=rows, d=width, type=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        c["residual"] = rng.random() < 0.7
    return c


def work(c):
    r = c["rows"]
    if c["op"] == "linear":
        es = 4 if c["out"] == "f32" else 2
        return {"bytes": r * c["k"] + c["n"] * c["k"] + 4 * (r + c["n"]) + (4 * c["n"] if c["bias"] else 0) + es * r * c["n"],
                "flops": 2 * r * c["k"] * c["n"]}
    es = 4 if c["type"] == "f32" else 2
    if c["op"] == "rotate":
        # every head in and out, and a position a row
        heads = r * (c["hq"] + c["hkv"])
        return {"bytes": 2 * es * heads * c["dh"] + 4 * r, "flops": 3 * heads * c["rot"]}
    d = c["d"]
    held = r * (2 * d + 4 + 2 * d)   # codes out and in, the scale, the values read back in bf16
    if c["op"] == "norm":
        return {"bytes": held + es * r * d * (3 if c["residual"] else 1) + es * d, "flops": 8 * r * d}
    if c["op"] == "swiglu":
        return {"bytes": held + 2 * es * r * d, "flops": 12 * r * d}
    return {"bytes": held + es * r * d, "flops": 4 * r * d}


# ---------------------------------------------------------------- rotary frequencies, float64
FACTOR, LOW, HIGH, ORIGINAL, THETA = 8.0, 1.0, 4.0, 8192, 500000.0
YARN_FAST, YARN_SLOW = 32.0, 1.0


def _frequencies(rot, scaling, dev):
    """Radians a position of each pair, and the factor of cos and sin."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    f = THETA ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / FACTOR, 1.0
    if scaling == "ntk":
        return (THETA * FACTOR ** (rot / (rot - 2))) ** (-2.0 * i / rot), 1.0
    if scaling == "bands":
        t = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        return f * (t + (1 - t) / FACTOR), 1.0
    if scaling == "yarn":
        at = lambda turns: rot * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(0, math.floor(at(YARN_FAST))), min(rot - 1, math.ceil(at(YARN_SLOW)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1
    return f, 1.0


# ---------------------------------------------------------------- state
class State:
    pass


def _codes(rows, k, g, spread):
    """8-bit rows and their scales as the quantiser leaves them, each row padded to a multiple of 16 bytes."""
    pad = -(-k // 16) * 16
    c = torch.empty(rows, pad, dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    step = max(1, (1 << 26) // pad)
    for a in range(0, rows, step):
        x = torch.randn(min(step, rows - a), pad, generator=g, device="cuda")
        top = x[:, :k].abs().amax(1)
        c[a:a + step] = (x * (127.0 / top)[:, None]).round().clamp(-127, 127).to(torch.int8)
        scale[a:a + step] = top / 127 * spread
    return c[:, :k], scale


def prepare(case, seed):
    c, st = case, State()
    st.c = c
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = c["rows"]
    st.plan = None
    if c["op"] == "linear":
        st.codes, st.scale = _codes(r, c["k"], g, 1.0)
        st.w, st.w_scale = _codes(c["n"], c["k"], g, 0.02)
        st.bias = torch.randn(c["n"], generator=g, device="cuda") * 0.1 if c["bias"] else None
        st.out = torch.empty(r, c["n"], dtype=TYPES[c["out"]], device="cuda")
        return st
    dt = TYPES[c["type"]]
    if c["op"] == "rotate":
        # the fused projection's output: query heads, key heads, value heads of each row
        st.qkv = torch.randn(r, c["hq"] + 2 * c["hkv"], c["dh"], generator=g, device="cuda").to(dt)
        st.q, st.k = st.qkv[:, :c["hq"]], st.qkv[:, c["hq"]:c["hq"] + c["hkv"]]
        if r > 1000:   # one sequence's rows, up to the farthest
            st.pos = torch.arange(c["far"] - r, c["far"], device="cuda").clamp(min=0).to(torch.int32)
        else:          # the next tokens of many sequences
            st.pos = torch.randint(0, c["far"], (r,), generator=g, device="cuda", dtype=torch.int32)
        st.q_out = torch.empty(r, c["hq"], c["dh"], dtype=dt, device="cuda")
        st.k_out = torch.empty(r, c["hkv"], c["dh"], dtype=dt, device="cuda")
        return st
    d = c["d"]
    # hidden rows: channels of different size, a few of them far larger than the rest
    size = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    size[torch.randint(0, d, (max(1, d // 500),), generator=g, device="cuda")] *= 20.0
    wide = 2 * d if c["op"] == "swiglu" else d
    st.x = torch.empty(r, wide, dtype=dt, device="cuda")
    step = max(1, (1 << 26) // wide)
    for a in range(0, r, step):
        x = torch.randn(min(step, r - a), wide, generator=g, device="cuda")
        st.x[a:a + step] = (x * (1.5 if c["op"] == "swiglu" else size)).to(dt)
    if c["op"] == "norm":
        st.res = torch.randn(r, d, generator=g, device="cuda").to(dt) if c["residual"] else None
        st.sum = torch.empty(r, d, dtype=dt, device="cuda") if c["residual"] else None
        st.weight = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
    st.codes = torch.empty(r, -(-d // 16) * 16, dtype=torch.int8, device="cuda")[:, :d]
    st.scale = torch.empty(r, device="cuda")
    st.values = torch.empty(r, d, dtype=torch.bfloat16, device="cuda")
    return st


def _plan(st):
    """The library's descriptors of a state, made on its first pass as a program makes them at start-up."""
    from selective_kv_cache_gb300 import kvr
    c = st.c
    if c["op"] == "linear":
        st.err = torch.zeros(4, dtype=torch.int32, device="cuda")
        st.weights = kvr.linear_weights(st.w, st.w_scale, st.err, bias=st.bias)
        st.ws = torch.empty(kvr.kvr_linear_workspace_bytes(st.weights, c["rows"]), dtype=torch.uint8, device="cuda")
    if c["op"] == "rotate":
        more = dict(factor=FACTOR) if c["scaling"] != "plain" else {}
        if c["scaling"] == "bands":
            more.update(low=LOW, high=HIGH, original_len=ORIGINAL)
        if c["scaling"] == "yarn":
            more.update(low=YARN_SLOW, high=YARN_FAST, original_len=ORIGINAL)
        st.rope = kvr.rope(c["dh"], c["rot"], layout=c["layout"], theta=THETA, scaling=c["scaling"], **more)
    st.plan = kvr


EPS = 1e-5


def run(state):
    st, c = state, state.c
    if own:
        if st.plan is None:
            _plan(st)
        kvr = st.plan
        if c["op"] == "linear":
            kvr.kvr_linear(st.weights, st.codes, st.scale, st.out, st.ws)
            return {"out": st.out}
        if c["op"] == "rotate":
            kvr.kvr_rows_rotate(st.rope, st.pos, st.q, st.q_out, st.k, st.k_out)
            return {"q": st.q_out, "k": st.k_out}
        if c["op"] == "norm":
            kvr.kvr_rows_norm(st.x, st.weight, EPS, residual=st.res, sum_out=st.sum, codes=st.codes, scales=st.scale)
        elif c["op"] == "swiglu":
            kvr.kvr_rows_swiglu(st.x, codes=st.codes, scales=st.scale)
        else:
            kvr.kvr_rows_quantise(st.x, st.codes, st.scale)
        kvr.kvr_rows_dequantise(st.codes, st.scale, st.values)
        return {"values": st.values, "scale": st.scale, **({"sum": st.sum} if c.get("residual") else {})}
    if c["op"] == "linear":
        y = (st.codes.float() @ st.w.float().T) * st.scale[:, None] * st.w_scale
        return {"out": (y if st.bias is None else y + st.bias).to(st.out.dtype)}
    if c["op"] == "rotate":
        return _plain_rotate(st)
    x = st.x.float()
    more = {}
    if c["op"] == "norm":
        if c["residual"]:
            x = x + st.res.float()
            more["sum"] = x.to(st.x.dtype)
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * st.weight.float()
    elif c["op"] == "swiglu":
        a, b = x[:, :c["d"]], x[:, c["d"]:]
        x = a / (1 + torch.exp(-a)) * b
    scale = x.abs().amax(1) * (1.0 / 127)
    code = (x * (1.0 / scale)[:, None]).round().clamp(-127, 127)
    return {"values": (code * scale[:, None]).bfloat16(), "scale": scale, **more}


def _plain_rotate(st):
    c = st.c
    f, m = _frequencies(c["rot"], c["scaling"], "cuda")
    a = st.pos.double()[:, None] * f
    cos, sin = ((t * m).float()[:, None] for t in (a.cos(), a.sin()))

    def turned(x):
        x, rest = x[..., :c["rot"]].float(), x[..., c["rot"]:]
        u, w = (x[..., 0::2], x[..., 1::2]) if c["layout"] == "interleaved" else x.chunk(2, -1)
        u, w = u * cos - w * sin, w * cos + u * sin
        x = torch.stack([u, w], -1).flatten(-2) if c["layout"] == "interleaved" else torch.cat([u, w], -1)
        return torch.cat([x.to(st.q.dtype), rest], -1)

    return {"q": turned(st.q), "k": turned(st.k)}


# ---------------------------------------------------------------- definitions in float64
def exact(case, seed):
    """Each output from its definition."""
    c, st = case, prepare(case, seed)
    if c["op"] == "linear":
        y = torch.matmul(st.codes.double(), st.w.double().t())
        y *= st.scale.double()[:, None]
        y *= st.w_scale.double()[None, :]
        if c["bias"]:
            y += st.bias.double()
        return {"out": y}
    if c["op"] == "rotate":
        h = c["rot"] // 2
        f, m = _frequencies(c["rot"], c["scaling"], "cuda")
        turn = m * torch.exp(1j * (st.pos.double()[:, None] * f))[:, None]
        got = {}
        for name, x in (("q", st.q), ("k", st.k)):
            x = x.double()
            at = torch.arange(h, device="cuda")
            i, j = (2 * at, 2 * at + 1) if c["layout"] == "interleaved" else (at, at + h)
            z = torch.complex(x[..., i], x[..., j]) * turn
            y = x.clone()
            y[..., i], y[..., j] = z.real, z.imag
            got[name] = y
        return got
    d = c["d"]
    values, scales, sums = [], [], []
    step = max(1, (1 << 25) // d)
    for a in range(0, c["rows"], step):   # some rows at a time: 64-bit copies of all are many gigabytes
        x = st.x[a:a + step].double()
        if c["op"] == "norm":
            if c["residual"]:
                x += st.res[a:a + step].double()
                sums.append(x.clone())
            x = x / torch.sqrt(x.square().sum(1, keepdim=True) / d + EPS) * st.weight.double()
        elif c["op"] == "swiglu":
            x = x[:, :d] * torch.sigmoid(x[:, :d]) * x[:, d:]
        s = x.abs().max(1).values / 127
        values.append(torch.round(x / s[:, None]) * s[:, None])
        scales.append(s)
    got = {"values": torch.cat(values), "scale": torch.cat(scales)}
    if c.get("residual"):
        got["sum"] = torch.cat(sums)
    return got
