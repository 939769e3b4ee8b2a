"""Packed-row operators on the GPU: norms, gated activation, rows in eight
bits and the rotary map against their definitions in float64 (oracle.rows).

Bounds.  r is half a step of the row type (bf16 2^-8, fp32 2^-24).  A value y
before the quantiser is off by rel |y|:
  norm    n/t + 12 additions of the sum of squares (t threads, then the tree),
          halved by the root, two roundings for the mean and eps, 2 ulp of the
          reciprocal root, h, h w and the scale's three products: for n/t <= 40
          (52 / 2 + 2 + 2 + 5) 2^-24 < 2^-18;
  swiglu  bf16: the approximate exponential is off by 2^-21 + |g| 2^-23, its
          division by 2^-22; |g| <= 40 here: below 2^-17.  fp32: 2^-20.
A code is off its value's place by at most half a step and 127 times three
roundings (1/127, 1 / scale, the product): 0.5 + 2^-14 steps; a scale by rel."""
import copy
import ctypes

import numpy as np
import pytest
import torch

from oracle import rows as OR

pytestmark = pytest.mark.gpu

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
REL = 2.0 ** -18
# widths at every kernel's borders: a warp a row (256, 257), one, two and four
# groups of eight a thread, rows that are read twice, odd ones
WIDTHS = [1, 2, 7, 8, 31, 64, 255, 256, 257, 264, 1792, 2047, 2048, 2056, 4096, 5001, 8192, 8200, 14336, 18944, 32768,
          32776, 40001]


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(n, d, dtype, seed, scale=1.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, d + pad, generator=g, device="cuda") * torch.exp(torch.randn(d + pad, generator=g, device="cuda"))
    return (x * scale).to(DTYPES[dtype])[:, :d]


def empty_codes(n, d, pad=0):
    return torch.full((n, d + pad), 77, dtype=torch.int8, device="cuda")[:, :d], torch.full((n,), 5.0, device="cuda")


def check_codes(codes, scale, y, rel):
    want, got = OR.scales(y), f64(scale)
    assert np.all(np.abs(got - want) <= (rel + 2.0 ** -22) * want), "scales"
    off = np.abs(f64(codes) * got[:, None] - y) - (rel * np.abs(y) + (0.5 + 2.0 ** -14) * got[:, None])
    assert off.max() <= 0, f"codes: {off.max()} beyond the bound at {np.unravel_index(off.argmax(), off.shape)}"


def check_values(out, y, dtype, rel):
    assert np.all(np.abs(f64(out) - y) <= (HALF[dtype] + rel) * np.abs(y) + 1e-37)


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(dtype, d, residual):
    n = 5 if d < 20000 else 2
    x, res, w = rows(n, d, dtype, 1), rows(n, d, dtype, 2), (1 + 0.3 * rows(1, d, "f32", 3)[0].tanh()).to(DTYPES[dtype])
    out, summed = torch.empty_like(x), torch.empty_like(x)
    codes, scale = empty_codes(n, d)
    kvr.kvr_rows_norm(x, w, 1e-5, residual=res if residual else None, sum_out=summed, out=out, codes=codes, scales=scale)
    h, y = OR.norm(f64(x), f64(w), 1e-5, f64(res) if residual else None)
    check_values(summed, h, dtype, 2.0 ** -24)
    check_values(out, y, dtype, REL)
    check_codes(codes, scale, y, REL)
    only, (c2, s2) = torch.empty_like(x), empty_codes(n, d)
    kvr.kvr_rows_norm(x, w, 1e-5, residual=res if residual else None, out=only)
    kvr.kvr_rows_norm(x, w, 1e-5, residual=res if residual else None, codes=c2, scales=s2)
    assert torch.equal(only, out) and torch.equal(c2, codes) and torch.equal(s2, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,pad", [(64, 8), (1536, 24), (1537, 0), (4096, 3), (40008, 8)])
def test_norm_in_place_and_strided(dtype, d, pad):
    """sum_out over the residual, out over x, rows further apart than wide;
    what lies between the rows stays."""
    n = 3
    x, res, w = rows(n, d, dtype, 1, pad=pad), rows(n, d, dtype, 2, pad=pad), torch.ones(d, device="cuda").to(DTYPES[dtype])
    h, y = OR.norm(f64(x), f64(w), 1e-6, f64(res))
    wide = torch.full((n, d + 16), 9, dtype=torch.int8, device="cuda")
    scale = torch.empty(n, device="cuda")
    between = [t.as_strided((n, pad), (d + pad, 1), d).clone() for t in (x, res)]
    kvr.kvr_rows_norm(x, w, 1e-6, residual=res, sum_out=res, out=x, codes=wide[:, :d], scales=scale)
    check_values(res, h, dtype, 2.0 ** -24)
    check_values(x, y, dtype, REL)
    check_codes(wide[:, :d], scale, y, REL)
    assert torch.all(wide[:, d:] == 9)
    for t, old in zip((x, res), between):
        assert torch.equal(t.as_strided((n, pad), (d + pad, 1), d), old)


def test_vector_and_single_element_kernels_agree():
    """The same rows aligned and off by one element: the codes lie within one
    step (the sums are added in another order), the scales within 2^-18."""
    for dtype in DTYPES:
        base = torch.zeros(6, 4112, dtype=DTYPES[dtype], device="cuda")
        base[:, 1:4097] = rows(6, 4096, dtype, 4)
        w = torch.ones(4096, dtype=DTYPES[dtype], device="cuda")
        got = []
        for x in (base[:, 1:4097], base[:, 1:4097].contiguous()):
            codes, scale = empty_codes(6, 4096)
            kvr.kvr_rows_norm(x, w, 1e-5, codes=codes, scales=scale)
            got.append((codes.int(), scale))
        assert (got[0][0] - got[1][0]).abs().max() <= 1
        assert ((got[0][1] - got[1][1]).abs() <= 2.0 ** -18 * got[1][1]).all()


# ---------------------------------------------------------------- gated activation
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_swiglu(dtype, d):
    n = 4 if d < 20000 else 2
    x = rows(n, 2 * d, dtype, 5, 2.0, pad=(16 if d % 8 == 0 else 1)).clamp(-40, 40)
    out = torch.empty(n, d, dtype=x.dtype, device="cuda")
    codes, scale = empty_codes(n, d, 16 if d % 8 == 0 else 3)
    kvr.kvr_rows_swiglu(x, out=out, codes=codes, scales=scale)
    y, rel = OR.swiglu(f64(x)), 2.0 ** (-17 if dtype == "bf16" else -20)
    check_values(out, y, dtype, rel)
    check_codes(codes, scale, y, rel)


def test_swiglu_far_from_zero():
    """exp(-g) overflows below g = -88 and vanishes above 88: the gate goes to 0 and to g."""
    g = torch.tensor([[-300.0, -100.0, -89.0, 89.0, 100.0, 3000.0, 0.0, -0.0]], device="cuda")
    for dt in DTYPES.values():
        x = torch.cat([g, torch.full_like(g, 2.0)], 1).to(dt)
        out = torch.empty(1, 8, dtype=dt, device="cuda")
        kvr.kvr_rows_swiglu(x, out=out)
        want = torch.tensor([[0.0, 0, 0, 178, 200, 6000, 0, 0]], device="cuda").to(dt)
        assert torch.allclose(out.float(), want.float(), rtol=2.0 ** -8, atol=1e-30)


# ---------------------------------------------------------------- rows in eight bits
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 16), (130, 64), (7, 255), (5, 1536), (2, 18944), (2, 40000), (3, 333)])
def test_quantise_and_back(dtype, n, d):
    x = rows(n, d, dtype, 6, 3.0)
    codes, scale = empty_codes(n, d, -d % 16)
    kvr.kvr_rows_quantise(x, codes, scale)
    y = f64(x)
    check_codes(codes, scale, y, 0.0)
    assert (codes.int().abs().amax(1) == 127).all()
    for dt in DTYPES.values():
        wide = torch.full((n, d + 8), 3.0, dtype=dt, device="cuda")
        kvr.kvr_rows_dequantise(codes, scale, wide[:, :d])
        want = (codes.cpu().float() * scale.cpu()[:, None]).to(dt)   # one product in fp32, one rounding
        assert torch.equal(wide[:, :d].cpu(), want) and torch.all(wide[:, d:] == 3.0)


@pytest.mark.parametrize("d", [48, 64, 4096, 40000, 777])
def test_quantise_rows_that_hold_nothing_or_no_number(d):
    """Zero rows, rows below 127 * 2^-126, the largest finite values; a NaN or
    an infinity takes its own row alone."""
    x = rows(9, d, "f32", 7)
    x[0] = 0
    x[1] = 1e-37
    x[2, d // 2] = float("nan")
    x[3, d - 1] = float("inf")
    x[4, 0] = float("-inf")
    x[5] *= 3e38 / x[5].abs().amax()
    x[6] *= 1e-30
    x[7] = -2.5
    codes, scale = empty_codes(9, d)
    kvr.kvr_rows_quantise(x, codes, scale)
    assert torch.all(codes[:5] == 0) and torch.all(scale[:2] == 0) and torch.isnan(scale[2:5]).all()
    check_codes(codes[5:], scale[5:], f64(x[5:]), 0.0)
    assert torch.all(codes[7] == -127)
    out = torch.empty(9, d, device="cuda")
    kvr.kvr_rows_dequantise(codes, scale, out)
    assert torch.all(out[:2] == 0) and torch.isnan(out[2:5]).all() and torch.isfinite(out[5:]).all()
    # the norm and the gate hand the same rows on
    w = torch.ones(d, device="cuda")
    kvr.kvr_rows_norm(x, w, 1e-5, codes=codes, scales=scale)
    assert torch.isnan(scale[2:5]).all() and torch.all(codes[2:5] == 0) and torch.all(codes[0] == 0) and scale[0] == 0
    check_codes(codes[6:], scale[6:], OR.norm(f64(x[6:]), 1.0, 1e-5)[1], REL)
    gu = torch.cat([x, x], 1)
    kvr.kvr_rows_swiglu(gu, codes=codes, scales=scale)
    assert torch.isnan(scale[2:4]).all() and torch.all(codes[2:4] == 0) and scale[0] == 0


def test_codes_round_to_even_halves():
    """A scale of exactly 1: halves go to the even code, both signs."""
    x = torch.arange(-254, 255, device="cuda").float()[None] / 2
    x = torch.cat([x, torch.zeros(1, 3, device="cuda")], 1)
    codes, scale = empty_codes(1, 512)
    kvr.kvr_rows_quantise(x, codes, scale)
    s = float(scale)
    assert abs(s - 1) <= 2.0 ** -23
    got = codes.cpu().numpy()[0].astype(int)
    v = x.cpu().numpy()[0].astype(np.float64)
    np.testing.assert_array_equal(got[v % 1 == 0], v[v % 1 == 0])
    assert np.all(np.abs(got - v) <= 0.5 + 2.0 ** -14)


# ---------------------------------------------------------------- rotary map
LAYOUTS = ["half", "interleaved"]


def rotated(x, pos, r, layout, inverse=False):
    return OR.rotate(f64(x), pos, list(r.turns[:r.rotary_dim // 2]), float(r.attn), layout, inverse)


def check_rotated(out, x, pos, r, layout, dtype, inverse=False):
    """cos and sin are off by 2^-22 (sincospi's ulp, the argument's rounding,
    the product with attn), products and sum rounded: 2^-21 of |x| + |y|."""
    want = rotated(x, pos, r, layout, inverse)
    big = np.abs(f64(x)).max(-1, keepdims=True) * max(float(r.attn), 1 / float(r.attn)) * 2
    assert np.all(np.abs(f64(out) - want) <= HALF[dtype] * np.abs(want) + 2.0 ** -21 * big)
    dims = np.arange(r.rotary_dim, r.head_dim)
    assert torch.equal(out[..., dims], x[..., dims])


FAR = [0, 1, 17, 8191, 131071, 1 << 24, (1 << 31) - 1, -1, -513, -(1 << 31)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dh,rot", [(128, 128), (128, 64), (128, 32), (64, 64), (256, 256), (80, 80), (80, 20), (96, 48),
                                    (2, 2), (10, 6), (64, 2)])
def test_rotate(dtype, layout, dh, rot):
    n, hq, hk = 23, 6, 2
    pos = [FAR[i % len(FAR)] for i in range(n)]
    r = kvr.rope(dh, rot, layout=layout, theta=1e4, attn_factor=1.25)
    qkv = rows(n, (hq + 2 * hk) * dh, dtype, 8).reshape(n, hq + 2 * hk, dh)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    p = torch.tensor(pos, dtype=torch.int64, device="cuda").to(torch.int32)
    qo, ko = torch.empty(n, hq, dh, dtype=q.dtype, device="cuda"), torch.empty(n, hk, dh, dtype=q.dtype, device="cuda")
    kvr.kvr_rows_rotate(r, p, q, qo, k, ko)
    check_rotated(qo, q, pos, r, layout, dtype)
    check_rotated(ko, k, pos, r, layout, dtype)
    back = torch.empty_like(ko)
    kvr.kvr_rows_rotate(r, p, k=ko, k_out=back, inverse=True)
    check_rotated(back, ko, pos, r, layout, dtype, inverse=True)
    # in place, inside the fused rows: the same bits, the values untouched
    before = qkv.clone()
    kvr.kvr_rows_rotate(r, p, q, q, k, k)
    assert torch.equal(qkv[:, :hq], qo) and torch.equal(qkv[:, hq:hq + hk], ko)
    assert torch.equal(qkv[:, hq + hk:], before[:, hq + hk:])


@pytest.mark.parametrize("n,hq,hk", [(1, 1, 0), (1, 32, 8), (1000, 3, 1), (7680, 1, 1), (5, 128, 8), (305, 0, 5)])
def test_rotate_row_and_head_counts(n, hq, hk):
    """More units than a block's batch, one unit, many rows a block."""
    r = kvr.rope(64, layout="half")
    pos = [(i * 7919) % 40000 for i in range(n)]
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for h in (hq, hk):
        if h == 0:
            continue
        x = rows(n, h * 64, "bf16", 9).reshape(n, h, 64)
        out = torch.empty_like(x)
        other = torch.empty(n, 1, 64, dtype=x.dtype, device="cuda")
        kvr.kvr_rows_rotate(r, p, x, out, *((other, torch.empty_like(other)) if h == 3 else (None, None)))
        check_rotated(out, x, pos, r, "half", "bf16")


@pytest.mark.parametrize("offset", [1, 3])
def test_rotate_misaligned_rows(offset):
    for dtype in DTYPES:
        flat = rows(4, 3 * 64 + 8, dtype, 10)
        x = flat[:, offset:offset + 192].unflatten(1, (3, 64))
        r, pos = kvr.rope(64, 32, layout="interleaved"), [5, 100, 3, 9999]
        out = torch.empty(4, 3, 64, dtype=x.dtype, device="cuda")
        kvr.kvr_rows_rotate(r, torch.tensor(pos, dtype=torch.int32, device="cuda"), x, out)
        check_rotated(out, x, pos, r, "interleaved", dtype)


@pytest.mark.parametrize("scaling,more", [("plain", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                          ("bands", dict(factor=8.0, low=1.0, high=4.0, original_len=8192)),
                                          ("yarn", dict(factor=16.0, low=1.0, high=32.0, original_len=4096))])
def test_table_of_scaled_positions(scaling, more):
    """(cos, sin) m of the formulas' own angles; the first rows and far ones."""
    r = kvr.rope(128, theta=500000.0, scaling=scaling, **more)
    n = 70001
    table = torch.empty(n, 64, 2, device="cuda")
    kvr.kvr_rope_table(r, n, table)
    f, m = OR.frequencies(128, scaling, 500000.0, **more)
    g = np.array([0, 1, 2, 1000, 65536, n - 1])
    a = g[:, None] * f
    got = f64(table[torch.as_tensor(g, device="cuda")])
    assert np.all(np.abs(got - m * np.stack([np.cos(a), np.sin(a)], -1)) <= 2.0 ** -22 * m)


def test_table_and_rotation_agree():
    """A head of (1, 0) pairs turns into the table's entries, bit for bit."""
    r = kvr.rope(128, scaling="yarn", factor=4.0, low=1.0, high=32.0, original_len=4096)
    table = torch.empty(5000, 64, 2, device="cuda")
    kvr.kvr_rope_table(r, 5000, table)
    x = torch.zeros(5000, 1, 128, device="cuda")
    x[:, :, :64] = 1
    kvr.kvr_rows_rotate(r, torch.arange(5000, dtype=torch.int32, device="cuda"), x, x)
    assert torch.equal(x[:, 0, :64], table[..., 0]) and torch.equal(x[:, 0, 64:], table[..., 1])


# ---------------------------------------------------------------- streams, graphs, devices
def test_rows_follow_their_stream_and_replay():
    """Captured once, replayed with new contents; two streams at once."""
    n, d = 40, 1536
    x, w = rows(n, d, "bf16", 11), torch.ones(d, dtype=torch.bfloat16, device="cuda")
    codes, scale = empty_codes(n, d)
    out, pos = torch.empty(n, 12, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    r = kvr.rope(128)
    s = torch.cuda.Stream()

    def step(stream):
        kvr.kvr_rows_norm(x, w, 1e-5, codes=codes, scales=scale, stream=stream)
        kvr.kvr_rows_rotate(r, pos, x.view(n, 12, 128), out, stream=stream)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for seed in (12, 13):
        x.copy_(rows(n, d, "bf16", seed))
        pos.copy_(torch.arange(seed, seed + n))
        graph.replay()
        torch.cuda.synchronize()
        check_codes(codes, scale, OR.norm(f64(x), 1.0, 1e-5)[1], REL)
        check_rotated(out, x.view(n, 12, 128), list(range(seed, seed + n)), r, "half", "bf16")
    c2, s2 = empty_codes(n, d)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        kvr.kvr_rows_quantise(x, c2, s2)
    step(None)
    torch.cuda.synchronize()
    check_codes(c2, s2, f64(x), 0.0)


def test_rotate_by_copied_and_by_filled_maps():
    """A kvr_rope is plain data: a copy outlives its original, and a caller may fill one."""
    n, dh = 5, 64
    x = rows(n, 3 * dh, "f32", 15).view(n, 3, dh)
    pos = torch.arange(7, 7 + n, dtype=torch.int32, device="cuda")
    want = torch.empty_like(x)
    kvr.kvr_rows_rotate(kvr.rope(dh), pos, x, want)
    first = kvr.rope(dh)
    copied = copy.copy(first)
    ctypes.memset(ctypes.addressof(first), 0, ctypes.sizeof(first))
    filled = kvr.kvr_rope(dh, dh, 0, 1.0)
    for i in range(dh // 2):
        filled.turns[i] = copied.turns[i]
    for r in (copied, filled):
        out = torch.empty_like(x)
        kvr.kvr_rows_rotate(r, pos, x, out)
        assert torch.equal(out, want)


def test_many_rows():
    """More rows than a grid of one wave, the last one checked."""
    n, d = 70001, 64
    x = rows(n, d, "bf16", 14)
    codes, scale = empty_codes(n, d)
    kvr.kvr_rows_quantise(x, codes, scale)
    at = [0, 1, 35000, n - 2, n - 1]
    check_codes(codes[at], scale[at], f64(x[at]), 0.0)
    assert torch.all(codes.int().abs().amax(1) == 127)
    out = torch.empty_like(x)
    kvr.kvr_rows_dequantise(codes, scale, out)
    assert torch.equal(out, (codes.float() * scale[:, None]).bfloat16())


def test_no_rows():
    """Empty tensors, which have no address: nothing happens."""
    x, c, s = torch.empty(0, 64, device="cuda"), torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    w, h, p = torch.ones(64, device="cuda"), torch.empty(0, 2, 64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    kvr.kvr_rows_norm(x, w, 1e-5, codes=c, scales=s)
    kvr.kvr_rows_swiglu(x, codes=c[:, :32], scales=s)
    kvr.kvr_rows_quantise(x, c, s)
    kvr.kvr_rows_dequantise(c, s, x)
    kvr.kvr_rows_rotate(kvr.rope(64), p, h, h)
    codes, scale = empty_codes(32, 64)
    W = kvr.linear_weights(codes, scale, torch.zeros(4, dtype=torch.int32, device="cuda"))
    kvr.kvr_linear(W, c, s, torch.empty(0, 32, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda"))
    kvr.kvr_linear_status(W)


def test_failed_launches_are_reported(monkeypatch):
    """Every launch made to fail on the host: an error from each call, the next ones work."""
    x, (codes, scale) = rows(70, 64, "bf16", 15), empty_codes(70, 64)
    kvr.kvr_rows_quantise(x, codes, scale)
    W = kvr.linear_weights(codes, scale, torch.zeros(4, dtype=torch.int32, device="cuda"))
    out = torch.empty(70, 70, device="cuda")
    ws = torch.empty(max(kvr.kvr_linear_workspace_bytes(W, n) for n in (4, 40, 70)), dtype=torch.uint8, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    h, p, table = x.view(70, 1, 64), torch.zeros(70, dtype=torch.int32, device="cuda"), torch.empty(8, 32, 2, device="cuda")
    calls = [lambda: kvr.kvr_rows_quantise(x, codes, scale), lambda: kvr.kvr_rows_dequantise(codes, scale, x),
             lambda: kvr.kvr_rows_norm(x, w, 1e-5, out=x), lambda: kvr.kvr_rows_swiglu(x, out=torch.empty_like(x[:, :32])),
             lambda: kvr.kvr_rows_rotate(kvr.rope(64), p, h, h), lambda: kvr.kvr_rope_table(kvr.rope(64), 8, table)] + \
        [lambda n=n: kvr.kvr_linear(W, codes[:n], scale[:n], out[:n], ws) for n in (4, 40, 70)]
    monkeypatch.setenv("KVR_FAULT", "launch")
    for call in calls:
        with pytest.raises(kvr.KvrError) as e:
            call()
        assert e.value.status == kvr.KVR_ECUDA
    monkeypatch.delenv("KVR_FAULT")
    for call in calls:
        call()
    kvr.kvr_linear_status(W)
    want = OR.linear(codes.cpu().numpy(), f64(scale), codes.cpu().numpy(), f64(scale))
    assert np.allclose(f64(out), want, rtol=2.0 ** -20, atol=0)


def test_rows_of_every_alignment():
    """All operands off by every number of elements, apart from one another:
    the values of aligned rows, and nothing outside."""
    n, d = 3, 520
    for dtype in DTYPES:
        x, res, w = rows(n, d, dtype, 16), rows(n, d, dtype, 17), rows(1, d, dtype, 18)[0]
        want, wsum = torch.empty_like(x), torch.empty_like(x)
        codes, scale = empty_codes(n, d)
        kvr.kvr_rows_norm(x, w, 1e-5, residual=res, sum_out=wsum, out=want, codes=codes, scales=scale)
        for off in range(8):
            def at(t, k):
                flat = torch.full((t.numel() + n * 9 + 32,), 3.0, dtype=t.dtype, device="cuda")
                v = flat.as_strided((n, t.shape[1]), (t.shape[1] + 9, 1), k)
                v.copy_(t)
                return flat, v
            (_, x2), (_, r2) = at(x, off), at(res, (3 * off + 1) % 8)
            (fo, o2), (fs, s2) = at(want, (5 * off + 2) % 8), at(wsum, (7 * off + 3) % 8)
            (fc, c2) = at(codes, off)
            wo = torch.zeros(d + 8, dtype=w.dtype, device="cuda")
            wo[off:off + d] = w
            before = [t.clone() for t in (fo, fs, fc)]
            for v in (o2, s2, c2):
                v.zero_()
            sc = torch.empty(n, device="cuda")
            kvr.kvr_rows_norm(x2, wo[off:off + d], 1e-5, residual=r2, sum_out=s2, out=o2, codes=c2, scales=sc)
            assert torch.equal(s2, wsum)
            check_values(o2, OR.norm(f64(x), f64(w), 1e-5, f64(res))[1], dtype, REL)
            assert (c2.int() - codes.int()).abs().max() <= 1
            for flat, old, v in zip((fo, fs, fc), before, (o2, s2, c2)):
                keep = torch.ones_like(flat, dtype=torch.bool)
                keep.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
                assert torch.equal(flat[keep], old[keep])
