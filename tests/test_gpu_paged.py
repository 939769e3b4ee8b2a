"""The paged cache on the GPU: kvr_paged_append, kvr_paged_read and
kvr_paged_attend against the plain definitions (oracle.paged).

Rows in and out of pages are compared bit for bit (the definitions fix every
fp32 rounding); attention within the bound derived in check_attend.  Slots
that were never written hold NaN throughout."""
import numpy as np
import pytest
import torch

from oracle import paged as OP

pytestmark = pytest.mark.gpu

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")
from paged_case import THETA, Paged, attend_case, check_attend, i32  # noqa: E402

FORMATS = [("bf16", 128, 0), ("f32", 64, 0), ("f32", 128, 0), ("int4", 128, 32), ("int4", 128, 64), ("int4", 128, 128)]
ATTEND = [("bf16", 128, 0), ("f32", 64, 0), ("int4", 128, 32), ("int4", 128, 128)]


def bits(t):
    return t.contiguous().view(torch.uint8)


# ---------------------------------------------------------------- append and read
def stored(x32, fmt, group):
    """What the pages hold for fp32 rows [n, heads, dh]: (rows, meta) as torch tensors."""
    if fmt == "int4":
        code, meta = OP.quantise(x32, group)
        return torch.from_numpy(OP.pack(code)), torch.from_numpy(meta)
    t = torch.from_numpy(x32)
    return (t if fmt == "f32" else t.bfloat16()), None


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
@pytest.mark.parametrize("layout,page,counts", [("hnd", 16, [1, 0, 37, 3]), ("nhd", 64, [130]), ("hnd", 256, [5] * 70)])
def test_append_writes_the_defined_bits(fmt, dh, group, layout, page, counts):
    """Ragged rows, sequences without rows and rows behind the last sequence:
    every written slot holds the definition's bits, every other byte of the
    pool what it held."""
    hkv, hq = 3, 6
    starts = [7 * b % 50 for b in range(len(counts))]
    c = Paged(fmt, [a + n for a, n in zip(starts, counts)], hkv, dh, page, layout, group, fill=False)
    n, pad = sum(counts), 3
    qkv = torch.randn(n + pad, hq + 2 * hkv, dh, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    qkv = (qkv * 3).to(c.row_dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    rope = OP.rope_table(256, dh, THETA)
    pos = np.concatenate([a + np.arange(m) for a, m in zip(starts, counts)] + [np.full(pad, 99)])
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs) if t is not None]
    q_out = torch.full((n + pad, hq, dh), 5.0, dtype=c.row_dtype, device="cuda")
    cu = i32(np.concatenate([[0], np.cumsum(counts)]))
    kvr.kvr_paged_append(c.p, cu, i32(pos), k, v, torch.from_numpy(rope).cuda(), q, q_out)
    kvr.kvr_paged_status(c.p)
    f = lambda t: t[:n].float().cpu().numpy()  # noqa: E731
    cs = rope[pos[:n]]
    wk, mk = stored(OP.rotate(f(k), cs), fmt, group)
    wv, mv = stored(f(v), fmt, group)
    wq = torch.from_numpy(OP.rotate(f(q), cs)).to(c.row_dtype)
    assert torch.equal(bits(q_out[:n].cpu()), bits(wq)) and torch.all(q_out[n:] == 5.0)
    seq = np.repeat(np.arange(len(counts)), counts)
    pg = torch.as_tensor(c.table_np[seq, pos[:n] // page], device="cuda")
    sl = torch.as_tensor(pos[:n] % page, device="cuda")
    pools = [t for t in (c.k, c.v, c.ks, c.vs) if t is not None]
    for pool, old, want in zip(pools, before, [w for w in (wk, wv, mk, mv) if w is not None]):
        x = old if layout == "nhd" else old.transpose(1, 2)
        x[pg, sl] = want.cuda()
        assert torch.equal(bits(pool), bits(old))


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
def test_read_returns_what_the_pages_hold(fmt, dh, group):
    """Positions out of order and repeated; strided and absent outputs; rows
    behind the last sequence untouched."""
    c = Paged(fmt, [70, 0, 33], 3, dh, 32, "nhd" if group == 64 else "hnd", group, seed=3)
    pos = [69, 0, 5, 5, 64, 32, 0, 31]
    cu = i32([0, 5, 5, 8])
    wide = torch.full((10, 7, dh), 2.0, dtype=c.row_dtype, device="cuda")
    ko, vo = wide[:, :3], wide[:, 4:]
    kvr.kvr_paged_read(c.p, cu, i32(pos + [1, 1]), ko, vo)
    only_v = torch.zeros(8, 3, dh, dtype=c.row_dtype, device="cuda")
    kvr.kvr_paged_read(c.p, cu, i32(pos), None, only_v)
    kvr.kvr_paged_status(c.p)
    for r, (b, g) in enumerate(zip([0] * 5 + [2] * 3, pos)):
        K, V, _ = c.rows64(b)
        assert torch.equal(ko[r].cpu(), torch.from_numpy(K[:, g]).to(c.row_dtype))
        assert torch.equal(vo[r].cpu(), torch.from_numpy(V[:, g]).to(c.row_dtype))
    assert torch.equal(only_v, vo[:8]) and torch.all(wide[8:] == 2.0) and torch.all(wide[:, 3] == 2.0)


def test_quantiser_on_flat_extreme_and_non_finite_groups():
    """A flat group keeps its value, magnitudes saturate at 2^15, and
    a non-finite element stays within its own group."""
    c = Paged("int4", [8], 1, 128, 16, group=32, fill=False)
    x = torch.randn(8, 1, 128, device="cuda").bfloat16()
    x[0] = 0
    x[1] = 7.25
    x[2, 0, 5] = 3e38
    x[6, 0] = torch.linspace(0, 4e4, 128).bfloat16()
    x[3, 0, 40] = float("nan")
    x[4, 0, 99] = float("-inf")
    x[5] *= 1e-30
    kvr.kvr_paged_append(c.p, i32([0, 8]), i32(np.arange(8)), x, x)
    out = torch.zeros(8, 1, 128, dtype=torch.bfloat16, device="cuda")
    kvr.kvr_paged_read(c.p, i32([0, 8]), i32(np.arange(8)), out)
    kvr.kvr_paged_status(c.p)
    ok = [0, 1, 2, 4, 5, 6, 7]
    code, meta = OP.quantise(x.float().cpu().numpy()[ok], 32)
    want = torch.from_numpy(OP.values(OP.pack(code), meta, 32)).bfloat16()
    assert torch.equal(out[ok].cpu(), want)
    keep = [d for d in range(128) if not 32 <= d < 64]
    code, meta = OP.quantise(np.nan_to_num(x.float().cpu().numpy()[3:4]), 32)
    want = torch.from_numpy(OP.values(OP.pack(code), meta, 32)).bfloat16()
    assert torch.equal(out[3:4].cpu()[..., keep], want[..., keep])


def test_append_reports_and_skips_bad_rows():
    """A position below zero, past the table or past the rotary table, one that
    does not ascend, a page outside the pool: the row is not written, the
    others are, and the report is cleared by being read."""
    for pos, rope_len, page1, status, written in [
            ([3, 4, -1, 60], 64, None, "index", [3, 4, 60]), ([3, 4, 64, 65], 99, None, "index", [3, 4]),
            ([3, 4, 50, 60], 50, None, "index", [3, 4]), ([3, 4, 4, 60], 64, None, "ascend", [3, 4, 60]),
            ([3, 4, 2, 60], 64, None, "ascend", [3, 4, 60]), ([3, 4, 20, 60], 64, -7, "index", [3, 4, 60]),
            ([3, 4, 20, 60], 64, 10 ** 6, "index", [3, 4, 60])]:
        c = Paged("bf16", [64], 2, fill=False)
        if page1 is not None:
            c.table[0, 1] = page1
        x = torch.randn(4, 2, 128, device="cuda").bfloat16()
        rope = torch.from_numpy(OP.rope_table(rope_len, 128, THETA)).cuda()
        kvr.kvr_paged_append(c.p, i32([0, 4]), i32(pos), x, x, rope)
        with pytest.raises(kvr.KvrError, match=status) as e:
            kvr.kvr_paged_status(c.p)
        assert e.value.status == kvr.KVR_EDEVICE
        kvr.kvr_paged_status(c.p)
        for pool in (c.k, c.v):
            got = np.isfinite(c.slots(pool, 0)).all((1, 2))
            assert np.flatnonzero(got).tolist() == written
            assert torch.isfinite(pool.float()).any(-1).sum().item() == 2 * len(written)


def test_malformed_row_offsets_touch_nothing_else():
    c = Paged("bf16", [20, 20], 2, seed=1)
    before = bits(c.k).clone()
    x = torch.ones(4, 2, 128, device="cuda", dtype=torch.bfloat16)
    out = torch.full((4, 4, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    for cu in ([0, 9, 4], [-3, 2, 4], [2, 1, 0]):
        ws = torch.empty(kvr.kvr_paged_workspace_bytes(c.p, 4, 4, 4), dtype=torch.uint8, device="cuda")
        kvr.kvr_paged_attend(c.p, None, 4, i32(cu), i32([1, 2, 3, 4]), out, out.clone(), ws)
        with pytest.raises(kvr.KvrError):
            kvr.kvr_paged_status(c.p)
    for cu in ([4, 4, 4], [-3, -1, -1], [3, 2, 1]):
        kvr.kvr_paged_append(c.p, i32(cu), i32([1, 2, 3, 4]), x, x)
        got = torch.full((4, 2, 128), 9.0, device="cuda", dtype=torch.bfloat16)
        kvr.kvr_paged_read(c.p, i32(cu), i32([1, 2, 3, 4]), got)
        if cu[0] > 0:
            with pytest.raises(kvr.KvrError):
                kvr.kvr_paged_status(c.p)
        assert torch.all(got == 9.0)
    assert torch.equal(bits(c.k), before)


# ---------------------------------------------------------------- attention
def tail(lens, counts):
    return np.concatenate([np.arange(n - q, n) for n, q in zip(lens, counts)]).astype(np.int64)


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (14, 2), (12, 2), (16, 1), (3, 3)])
def test_decode_step(fmt, dh, group, hq, hkv):
    """One row per sequence over lengths around every tile and page border, a
    sequence without keys among them (it may hold a row or none)."""
    lens = [1, 2, 15, 16, 17, 0, 31, 33, 63, 64, 65, 127, 128, 129, 255, 300, 1000, 2049]
    c = Paged(fmt, lens, hkv, dh, 16, "hnd", group, seed=11)
    counts = [1 if n else 0 for n in lens]
    counts[5] = 1    # no key: zeros
    pos = np.array([max(n - 1, 0) for n in lens])
    out, q, _ = attend_case(c, hq, counts, pos, spare_rows=2)
    kvr.kvr_paged_status(c.p)
    assert torch.all(out[5] == 0) and torch.all(out[len(lens):] == 7.0)
    check_attend(c, hq, counts, pos, out, q)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("page,layout", [(16, "nhd"), (32, "hnd"), (64, "nhd"), (128, "hnd"), (256, "nhd")])
def test_rows_and_pages(fmt, dh, group, page, layout):
    """A few to a few hundred rows a sequence, ragged, on every page size."""
    lens, counts = [700, 90, 130, 5], [3, 90, 37, 2]
    c = Paged(fmt, lens, 2, dh, page, layout, group, seed=page)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, 8, counts, pos, spare_rows=1)
    kvr.kvr_paged_status(c.p)
    assert torch.all(out[-1] == 7.0)
    check_attend(c, 8, counts, pos, out, q)


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
@pytest.mark.parametrize("hq,hkv", [(8, 2), (14, 2), (12, 1)])
@pytest.mark.parametrize("opts", [dict(), dict(softcap=15.0)])
def test_several_passes(fmt, dh, group, hq, hkv, opts):
    """Rows for several passes over the keys, ragged and one alone."""
    lens, counts = [333, 40, 1100], [17, 9, 1]
    c = Paged(fmt, lens, hkv, dh, 32, "nhd", group, seed=13)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, hq, counts, pos, **opts)
    kvr.kvr_paged_status(c.p)
    check_attend(c, hq, counts, pos, out, q, **opts)


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
@pytest.mark.parametrize("hq,hkv,n", [(4, 4, 260), (14, 2, 75), (6, 1, 300), (16, 1, 33)])
def test_prompt(fmt, dh, group, hq, hkv, n):
    """A prompt against its own cache: many row tiles of every group size."""
    lens, counts = [n + 41, n], [n, n - 1]
    c = Paged(fmt, lens, hkv, dh, 64, "hnd", group, seed=n)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, hq, counts, pos)
    kvr.kvr_paged_status(c.p)
    check_attend(c, hq, counts, pos, out, q)


def intervals(kind, rng, pos, L):
    n = len(pos)
    if kind == "document":
        starts = np.sort(np.concatenate([[0], rng.integers(0, L, 5)]))
        return starts[np.searchsorted(starts, pos, side="right") - 1], None
    if kind == "window":
        return pos + 1 - 37, None
    if kind == "prefix":
        return None, np.maximum(pos + 1, L // 3)
    if kind == "empty rows":     # every third row sees nothing: begin past end, past kv_len, end <= 0
        b, e = np.zeros(n, np.int64), pos + 1
        b[0::9] = pos[0::9] + 1
        b[3::9] = L + 5
        e[6::9] = -3
        return b, e
    a = rng.integers(-5, L + 5, n)
    e = a + rng.integers(-3, 200, n)          # any interval, reaching below 0 and past kv_len,
    e[0::11], a[5::11] = -2 ** 31, 2 ** 31 - 1          # and the types' ends
    a[7::11], e[7::11] = -2 ** 31, 2 ** 31 - 1
    return a, e


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("kind", ["document", "window", "prefix", "empty rows", "any"])
@pytest.mark.parametrize("counts", [[1, 1, 1], [4, 2, 3], [150, 1, 60]])
def test_masks(fmt, dh, group, kind, counts):
    """Per-row key intervals; rows at positions spread over the sequence."""
    lens = [333, 129, 600]
    c = Paged(fmt, lens, 2, dh, 32, "hnd", group, seed=5)
    rng = np.random.default_rng(9)
    pos = np.concatenate([np.sort(rng.choice(n, min(m, n), replace=False)) for n, m in zip(lens, counts)])
    counts = [min(m, n) for n, m in zip(lens, counts)]
    at = np.concatenate([[0], np.cumsum(counts)])
    pairs = [intervals(kind, rng, pos[at[b]:at[b + 1]], lens[b]) for b in range(3)]
    begin = None if pairs[0][0] is None else np.concatenate([x[0] for x in pairs])
    end = None if pairs[0][1] is None else np.concatenate([x[1] for x in pairs])
    out, q, _ = attend_case(c, 14, counts, pos, key_begin=None if begin is None else i32(begin),
                            key_end=None if end is None else i32(end))
    kvr.kvr_paged_status(c.p)
    check_attend(c, 14, counts, pos, out, q, begin=begin, end=end)


def bit_words(m):
    """[batch, n] bool to int32 words [batch, ceil(n / 32)]."""
    b, n = m.shape
    w = np.zeros((b, -(-n // 32) * 32), np.int64)
    w[:, :n] = m
    return i32((w.reshape(b, -1, 32) << np.arange(32)).sum(-1).astype(np.uint32).view(np.int32))


SCORES = [dict(softcap=20.0), dict(slopes=True), dict(alpha=-2.0, beta=-4.0), dict(alpha=-3e38), dict(beta=-3e38),
          dict(scale=0.3), dict(softcap=5.0, slopes=True, alpha=-1.0, beta=2.0, scale=0.2)]


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("opts", SCORES)
@pytest.mark.parametrize("counts", [[1, 1], [70, 5]])
def test_scores(fmt, dh, group, opts, counts):
    """Cap, distance slopes, operator F's bits and the scale; a bias of the
    type's lowest value leaves only the unbiased keys, or, where every visible
    key has it, the plain softmax."""
    lens, hq = [517, 64], 8
    c = Paged(fmt, lens, 2, dh, 16, "hnd", group, seed=2)
    rng = np.random.default_rng(4)
    loc = rng.random((2, c.max_pages * 16)) < 0.5
    snk = rng.random((2, c.max_pages * 16)) < 0.1
    loc[1] = True
    pos = tail(lens, counts)
    slopes = (2.0 ** -np.arange(1, hq + 1)).astype(np.float32)
    kw = dict(opts)
    if kw.pop("slopes", False):
        kw["slopes"] = torch.from_numpy(slopes).cuda()
    if "alpha" in kw:
        kw["local_bits"] = bit_words(loc)
    if "beta" in kw:
        kw["sink_bits"] = bit_words(snk)
    out, q, _ = attend_case(c, hq, counts, pos, **kw)
    kvr.kvr_paged_status(c.p)
    a, b = (max(opts.get(x, 0.0), -1e30) for x in ("alpha", "beta"))
    check_attend(c, hq, counts, pos, out, q, scale=opts.get("scale"), softcap=opts.get("softcap", 0.0), alpha=a, beta=b,
                 loc=loc if "alpha" in opts else None, snk=snk if "beta" in opts else None,
                 slopes=slopes.astype(np.float64) if opts.get("slopes") else None)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1], [60]])
def test_long_sequence_is_split_and_merged(fmt, dh, group, counts):
    lens = [20011]
    c = Paged(fmt, lens, 1, dh, 64, "nhd", group, seed=8)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, 4, counts, pos, q_scale=4.0)
    again, _, _ = attend_case(c, 4, counts, pos, q_scale=4.0)
    kvr.kvr_paged_status(c.p)
    assert torch.equal(bits(out), bits(again))
    check_attend(c, 4, counts, pos, out, q)


@pytest.mark.parametrize("scale_v,q_scale", [(1e-3, 0.01), (300.0, 12.0)])
@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1], [70]])
def test_magnitudes(fmt, dh, group, scale_v, q_scale, counts):
    """Flat and one-key softmaxes; small and large values."""
    c = Paged(fmt, [1500], 2, dh, 64, "hnd", group, seed=8, v_scale=scale_v)
    pos = tail([1500], counts)
    out, q, _ = attend_case(c, 8, counts, pos, q_scale=q_scale)
    kvr.kvr_paged_status(c.p)
    check_attend(c, 8, counts, pos, out, q)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("most", [1, 40])
def test_many_sequences(fmt, dh, group, most):
    """More sequences than a kernel derives its shares of by itself, some
    without keys, some without rows."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 90, 300)
    counts = np.minimum(rng.integers(0, most + 1, 300), lens)
    c = Paged(fmt, lens, 2, dh, 16, "nhd", group, seed=21)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, 8, counts, pos, spare_rows=3)
    kvr.kvr_paged_status(c.p)
    assert torch.all(out[counts.sum():] == 7.0)
    check_attend(c, 8, counts, pos, out, q)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1, 1], [70, 33]])
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** 64])
def test_extreme_scales_of_flat_rows(fmt, dh, group, counts, scale):
    """Queries of zeros: the mean of the visible values, whatever the scale."""
    lens = [400, 77]
    c = Paged(fmt, lens, 2, dh, 32, "hnd", group, seed=5)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, 8, counts, pos, q_scale=0.0, scale=scale)
    kvr.kvr_paged_status(c.p)
    check_attend(c, 8, counts, pos, out, q, scale=scale)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1, 1], [70, 90]])
@pytest.mark.parametrize("shift,pad", [(8, 0), (0, 8), (16, 16)])
def test_rows_at_any_16_bytes(fmt, dh, group, counts, shift, pad):
    """q and out rows that begin between two 32-byte sectors; what lies between
    the rows stays as it was."""
    lens = [300, 200]
    c = Paged(fmt, lens, 2, dh, 64, "hnd", group, seed=6)
    pos = tail(lens, counts)
    n, hq = sum(counts), 8
    view = lambda x: torch.as_strided(x, (n, hq, dh), (hq * dh + pad, dh, 1), shift)  # noqa: E731
    flat = [torch.full((n * (hq * dh + pad) + shift,), 7.0, dtype=c.row_dtype, device="cuda") for _ in range(2)]
    q, out = view(flat[0]), view(flat[1])
    q.copy_(torch.randn(n, hq, dh, device="cuda"))
    ws = torch.empty(kvr.kvr_paged_workspace_bytes(c.p, hq, n, max(counts)), dtype=torch.uint8, device="cuda")
    kvr.kvr_paged_attend(c.p, None, max(counts), i32(np.concatenate([[0], np.cumsum(counts)])), i32(pos), q, out, ws)
    kvr.kvr_paged_status(c.p)
    check_attend(c, hq, counts, pos, out, q)
    out.fill_(7.0)
    assert torch.all(flat[1] == 7.0)


def test_order_of_rows_does_not_matter():
    """Positions in any order and repeated; strided q and out rows."""
    c = Paged("bf16", [400], 2, seed=3)
    pos = np.array([399, 3, 200, 200, 0, 17, 399])
    wide = torch.randn(7, 20, 128, device="cuda").bfloat16()
    q, out = wide[:, :8], wide[:, 12:]
    ws = torch.empty(kvr.kvr_paged_workspace_bytes(c.p, 8, 7, 7), dtype=torch.uint8, device="cuda")
    keep = wide[:, :12].clone()
    kvr.kvr_paged_attend(c.p, None, 7, i32([0, 7]), i32(pos), q, out, ws)
    kvr.kvr_paged_status(c.p)
    assert torch.equal(bits(wide[:, :12]), bits(keep))
    check_attend(c, 8, [7], pos, out, q)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
def test_attend_reports_bad_input(fmt, dh, group):
    """A page outside the pool, a length past the table, more rows than
    max_rows and a negative position are reported; the other sequences are
    right and rows past max_rows are left alone."""
    for fault in ("page", "length", "rows", "position"):
        c = Paged(fmt, [100, 50], 2, dh, 16, "hnd", group, seed=6, max_pages=8)
        counts = [1, 1]
        pos = np.array([99, 49])
        max_rows = 1
        if fault == "page":
            c.table[0, 2] = 10 ** 7
        elif fault == "length":
            c.kv_len[0] = 8 * 16 + 1
            c.table[0] = c.table[0, 0]
        elif fault == "rows":
            counts, pos = [3, 1], np.array([97, 98, 99, 49])
        else:
            pos = np.array([-1, 49])
        out, q, _ = attend_case(c, 8, counts, pos, max_rows=max_rows)
        with pytest.raises(kvr.KvrError) as e:
            kvr.kvr_paged_status(c.p)
        assert e.value.status == kvr.KVR_EDEVICE
        kvr.kvr_paged_status(c.p)
        check_attend(c, 8, counts, pos, out, q, only=[1])
        if fault == "rows":
            assert torch.all(out[1:3] == 7.0)
        if fault == "position":
            assert torch.all(out[0] == 0)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
def test_captured_calls_follow_their_device_arrays(fmt, dh, group):
    """A decode step (append, then attend) captured once and replayed while
    lengths, positions and row counts move on; a second graph shares the
    workspace."""
    lens = [30, 64, 200]
    c = Paged(fmt, lens, 2, dh, 16, "hnd", group, seed=4, max_pages=20, spare=20)
    for b in range(3):   # room to grow
        used = -(-lens[b] // 16)
        free = [i for i in range(c.k.shape[0]) if i not in set(c.table_np[c.table_np >= 0])]
        c.table_np[b, used:used + 2] = free[:2]
    c.table.copy_(i32(c.table_np))
    rope = torch.from_numpy(OP.rope_table(512, dh, THETA)).cuda()
    x = torch.randn(3, 8 + 4, dh, device="cuda").to(c.row_dtype)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    qr, out, out2 = (torch.zeros(3, 8, dh, dtype=c.row_dtype, device="cuda") for _ in range(3))
    pos, cu = i32([n for n in lens]), i32([0, 1, 2, 3])
    ws = torch.empty(kvr.kvr_paged_workspace_bytes(c.p, 8, 3, 1), dtype=torch.uint8, device="cuda")

    def step(o):
        kvr.kvr_paged_append(c.p, cu, pos, k, v, rope, q, qr)
        kvr.kvr_paged_attend(c.p, None, 1, cu, pos, qr, o, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.kv_len += 1
        step(out)       # outside a capture first
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for o in (out, out2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o)
        graphs.append((g, o))
    for t in range(4):
        x.copy_(torch.randn(3, 12, dh, device="cuda").to(c.row_dtype))
        if t == 2:
            cu.copy_(i32([0, 1, 2, 2]))     # the third sequence pauses
            out[2] = 7.0
        g, o = graphs[t % 2]
        g.replay()
        kvr.kvr_paged_status(c.p)
        c.lens = c.kv_len.cpu().tolist()
        counts = (cu[1:] - cu[:-1]).cpu().tolist()
        check_attend(c, 8, counts, pos.cpu().numpy()[:sum(counts)], o, qr)
        if t >= 2:
            assert t != 2 or torch.all(out[2] == 7.0)
        c.kv_len[:sum(counts)] += 1
        pos[:sum(counts)] += 1


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1, 1], [200, 90]])
def test_other_stream_and_two_calls_at_once(fmt, dh, group, counts):
    """Attention calls on two streams at once, each with its own workspace."""
    lens = [3000, 800]
    c = Paged(fmt, lens, 4, dh, 64, "hnd", group, seed=4)
    pos = tail(lens, counts)
    ref, q, _ = attend_case(c, 16, counts, pos)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(attend_case(c, 16, counts, pos)[0])
    torch.cuda.synchronize()
    kvr.kvr_paged_status(c.p)
    for o in outs:
        assert torch.equal(bits(o), bits(ref))


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
def test_captured_prompt(fmt, dh, group):
    """Many rows captured once, replayed with other lengths, positions, row
    counts and an idle sequence; the workspace serves another call in between."""
    lens = [500, 300, 60]
    c = Paged(fmt, lens, 2, dh, 32, "nhd", group, seed=14)
    n = 400
    q = torch.randn(n, 8, dh, device="cuda").to(c.row_dtype)
    out = torch.zeros_like(q)
    cu, pos = i32([0, 200, 350, 400]), i32(tail(lens, [200, 150, 50]))
    ws = torch.empty(kvr.kvr_paged_workspace_bytes(c.p, 8, n, 256), dtype=torch.uint8, device="cuda")
    call = lambda: kvr.kvr_paged_attend(c.p, None, 256, cu, pos, q, out, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new_lens, counts in [(lens, [200, 150, 50]), ([256, 300, 60], [256, 0, 33]), ([17, 300, 1], [17, 100, 1])]:
        c.lens = new_lens
        c.kv_len.copy_(i32(new_lens))
        cu.copy_(i32(np.concatenate([[0], np.cumsum(counts)])))
        p = tail(new_lens, counts)
        pos[:len(p)] = i32(p)
        out.fill_(7.0)
        g.replay()
        kvr.kvr_paged_status(c.p)
        assert torch.all(out[sum(counts):] == 7.0)
        check_attend(c, 8, counts, p, out, q)
        ws.random_(0, 256)


def test_binding_refusals(monkeypatch):
    c = Paged("bf16", [40], 2)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    cu, pos = i32([0, 1]), i32([3])
    ok = dict(cu_rows=cu, positions=pos, q=q, out=q.clone(), workspace=ws)
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :, :64]), dict(out=q[:, :2]), dict(cu_rows=i32([0])),
           dict(positions=pos.long()), dict(q=q.transpose(1, 2)), dict(workspace=ws.view(torch.int8)),
           dict(q=q.expand(2, 4, 128)[:, ::2])]
    for kw in bad:
        with pytest.raises(ValueError):
            kvr.kvr_paged_attend(c.p, None, 1, **{**ok, **kw})
    with pytest.raises(kvr.KvrError) as e:
        kvr.kvr_paged_attend(c.p, None, 1, **{**ok, "workspace": ws[:256]})
    assert e.value.status == kvr.KVR_EINVAL
    with monkeypatch.context() as m:   # another device is the current one
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        with pytest.raises(ValueError, match="current device"):
            kvr.kvr_paged_attend(c.p, None, 1, **ok)
        with pytest.raises(ValueError, match="current device"):
            kvr.kvr_paged_read(c.p, cu, pos, q[:, :2].clone())
        with pytest.raises(ValueError, match="current device"):
            kvr.kvr_paged_append(c.p, cu, pos, q[:, :2], q[:, :2])
    with pytest.raises(ValueError):
        kvr.kvr_paged_attend(c.p, kvr.score_opts(slopes=torch.ones(2, device="cuda")), 1, **ok)
    with pytest.raises(ValueError):
        kvr.kvr_paged_append(c.p, cu, pos, q, q)            # four heads into pages of two
    with pytest.raises(ValueError):
        kvr.kvr_paged_append(c.p, cu, pos, q[:, :2], q[:, :2], q_rows=q)
    with pytest.raises(ValueError):
        kvr.kvr_paged_append(c.p, cu, pos, q[:, :2], q[:, :2], torch.zeros(8, 32, 2, device="cuda"))
    with pytest.raises(ValueError):
        kvr.pages("bf16", c.k, c.v, c.table, c.kv_len, c.err, 2, 16, strides=(32, 16, 2), n_pages=c.k.shape[0])
    with pytest.raises(ValueError):
        kvr.pages("int4", c.k, c.v, c.table, c.kv_len, c.err, 2, 16, group=32)


def test_offsets_past_32_bits():
    """The last pages of a pool whose byte and element offsets pass 2^32."""
    n_pages = (5 << 30) // (2 * 64 * 256)       # 5 GB each of K and V
    k = torch.empty(n_pages, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Paged("bf16", [100], 2, page=64)
    pick = [n_pages - 1, n_pages - 2]
    for pool, src in ((k, c.k), (v, c.v)):
        for i in range(2):
            pool[pick[i]] = src[c.table_np[0, i]]
    table = i32([pick])
    big = kvr.pages("bf16", k, v, table, c.kv_len, c.err, 2, 64)
    small, p = c.p, c.p
    pos = np.array([97, 98, 99])
    ref, q, _ = attend_case(c, 8, [3], pos)
    c.p = big
    out, _, _ = attend_case(c, 8, [3], pos)
    x = torch.randn(1, 2, 128, device="cuda").bfloat16()
    kvr.kvr_paged_append(big, i32([0, 1]), i32([99]), x, x)
    got = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    kvr.kvr_paged_read(big, i32([0, 1]), i32([99]), got)
    kvr.kvr_paged_status(big)
    assert torch.equal(bits(out), bits(ref)) and torch.equal(got, x) and torch.equal(v[pick[1], :, 35], x[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_answering_after_a_repair(dtype):
    """The calls as a repair loop uses them: select and refresh a kvr_cache,
    view its layer as pages in place, append a new token's rows and answer with
    single-token queries under the mixed cache's bias; then the same rows held
    in 4 bits, read back and spliced into the cache."""
    import dataclasses

    from selective_kv_cache_gb300 import workloads as wl
    from selective_kv_cache_gb300.harness import Setup
    from helpers import small_bf16
    if dtype == "bf16":
        w = small_bf16(n_layers=2, selection="isolated", n_select=60, alpha=-2.0, beta=-4.0, capacity=640, n_tokens=600)
    else:
        w = dataclasses.replace(wl.WORKLOADS["tiny"], capacity=640, n_tokens=600, alpha=-2.0, beta=-4.0)
    m = w.model
    rng = np.random.default_rng(3)
    local, sink = rng.random((1, w.capacity)) < 0.5, rng.random((1, w.capacity)) < 0.1
    s = Setup(w, local=local, sink=sink)
    s.select()
    s.refresh()
    s.sync()
    lw, sw = kvr.kvr_read_meta(s.handle, 1, (w.capacity + 31) // 32)
    layer, page, n = m.n_layers - 1, 64, w.n_tokens
    per = w.capacity // page
    table = i32([np.arange(per)])
    kv_len, err = i32([n + 1]), torch.zeros(4, dtype=torch.int32, device="cuda")
    K, V = s.K[0, layer], s.V[0, layer]      # [hkv, capacity, dh]
    p = kvr.pages(dtype, K, V, table, kv_len, err, m.n_kv_heads, page, strides=(page, w.capacity, 1), n_pages=per)
    K0 = K.clone()
    x = torch.randn(1, m.n_q_heads + 2 * m.n_kv_heads, m.head_dim, device="cuda").to(m.torch_dtype)
    q, k, v = x[:, :m.n_q_heads], x[:, m.n_q_heads:-m.n_kv_heads], x[:, -m.n_kv_heads:]
    rope = torch.from_numpy(OP.rope_table(w.capacity, m.head_dim, m.rope_theta)).cuda()
    qr, out = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous())
    cu, pos = i32([0, 1]), i32([n])
    opts = dict(alpha=w.alpha, beta=w.beta, local_bits=i32(lw.view(np.int32)), sink_bits=i32(sw.view(np.int32)))
    ws = torch.empty(kvr.kvr_paged_workspace_bytes(p, m.n_q_heads, 1, 1), dtype=torch.uint8, device="cuda")
    kvr.kvr_paged_append(p, cu, pos, k, v, rope, q, qr)
    kvr.kvr_paged_attend(p, kvr.score_opts(**opts), 1, cu, pos, qr, out, ws)
    kvr.kvr_paged_status(p)
    assert torch.equal(K[:, :n], K0[:, :n])

    class Twin:                                # what check_attend asks of a Paged
        fmt, lens, dh = dtype, [n + 1], m.head_dim

        @staticmethod
        def rows64(b):
            a, z = (t[:, :n + 1].double().cpu().numpy() for t in (K, V))
            return a, z, np.abs(z)

    def mask(words):
        return ((words.view(np.uint32)[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(1, -1).astype(bool)

    check_attend(Twin, m.n_q_heads, [1], np.array([n]), out, qr, alpha=w.alpha, beta=w.beta, loc=mask(lw),
                 snk=mask(sw))
    # the refreshed rows attend through the pages as kvr_attend does in the cache
    U = np.sort(np.asarray(s.positions[0]))
    rows = len(U)
    qs = torch.randn(rows, m.n_q_heads, m.head_dim, device="cuda").to(m.torch_dtype)
    po, ca = torch.zeros_like(qs), torch.zeros(rows, m.n_q_heads * m.head_dim, device="cuda", dtype=m.torch_dtype)
    wide = torch.empty(kvr.kvr_paged_workspace_bytes(p, m.n_q_heads, rows, rows), dtype=torch.uint8, device="cuda")
    kvr.kvr_paged_attend(p, kvr.score_opts(**opts), rows, i32([0, rows]), i32(U), qs, po, wide)
    kvr.kvr_paged_status(p)
    check_attend(Twin, m.n_q_heads, [rows], U, po, qs, alpha=w.alpha, beta=w.beta, loc=mask(lw), snk=mask(sw))
    kvr.kvr_attend(s.handle, layer, qs, ca)
    s.sync()
    check_attend(Twin, m.n_q_heads, [rows], U, ca.view_as(qs), qs, alpha=w.alpha, beta=w.beta, loc=mask(lw),
                 snk=mask(sw))
    if dtype == "bf16":
        c4 = Paged("int4", [n], m.n_kv_heads, 128, 64, group=32, fill=False)
        rows = lambda t: t[:, :n].transpose(0, 1).contiguous()  # noqa: E731
        cu4, pos4 = i32([0, n]), i32(np.arange(n))
        kvr.kvr_paged_append(c4.p, cu4, pos4, rows(K), rows(V))
        back = [torch.empty(n, m.n_kv_heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        kvr.kvr_paged_read(c4.p, cu4, pos4, *back)
        kvr.kvr_paged_status(c4.p)
        block = [t.transpose(0, 1).unsqueeze(0).expand(m.n_layers, -1, -1, -1).contiguous() for t in back]
        kvr.kvr_splice(s.handle, 0, 0, n, *block, src_pos=0)
        kvr.kvr_sync_status(s.handle)
        assert torch.equal(s.K[0, layer, :, :n], block[0][layer]) and torch.equal(s.V[0, 0, :, :n], block[1][0])
    s.close()


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1], [4, 3], [70, 33]])
@pytest.mark.parametrize("cap", [1e3, 1e4, 1e7, 2.0 ** 64])
def test_caps_far_above_the_logits(fmt, dh, group, counts, cap):
    """cap tanh(x / cap) is nearly x there: a logit keeps its own precision,
    not the cap's (a few roundings of logits of about 10, 2^-24 each, well
    inside the bound's term for the cap)."""
    lens = [517, 64]
    c = Paged(fmt, lens, 2, dh, 16, "hnd", group, seed=2)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, 8, counts, pos, softcap=cap)
    kvr.kvr_paged_status(c.p)
    check_attend(c, 8, counts, pos, out, q, softcap=cap)


def attend_rows(c, q, counts, pos, **opts):
    """kvr_paged_attend on the given query rows; returns out."""
    out = torch.full_like(q, 7.0)
    ws = torch.empty(kvr.kvr_paged_workspace_bytes(c.p, q.shape[1], len(q), max(counts)), dtype=torch.uint8,
                     device="cuda")
    kvr.kvr_paged_attend(c.p, kvr.score_opts(**opts), max(counts), i32(np.concatenate([[0], np.cumsum(counts)])),
                         i32(pos), q, out, ws)
    kvr.kvr_paged_status(c.p)
    return out


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
@pytest.mark.parametrize("counts", [[2, 2], [70, 33]])
def test_capped_rows_keep_their_own_precision(fmt, dh, group, counts):
    """Rows whose logits reach the cap beside rows far below it: a row's bound
    knows its own logits only."""
    lens, cap = [517, 64], 2.0 ** 20
    c = Paged(fmt, lens, 2, dh, 16, "hnd", group, seed=2)
    pos = tail(lens, counts)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(sum(counts), 8, dh, generator=g, device="cuda") * 1.5
    q[::2] *= cap
    q = q.to(c.row_dtype)
    out = attend_rows(c, q, counts, pos, softcap=cap)
    check_attend(c, 8, counts, pos, out, q, softcap=cap)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1, 1], [4, 2], [70, 33]])
@pytest.mark.parametrize("opts", [dict(), dict(softcap=30.0), dict(softcap=1e4), dict(softcap=1e4, slopes=True)])
def test_unseen_slots_decide_nothing(fmt, dh, group, counts, opts):
    """The same bits whatever the slots behind a sequence's end, the unused
    pages and the keys no row sees hold: NaN, infinities, the type's largest
    values, small ones."""
    lens = [517, 77]
    c = Paged(fmt, lens, 2, dh, 32, "hnd", group, seed=12)
    pos = tail(lens, counts)
    pools = [c.ks, c.vs] if fmt == "int4" else [c.k, c.v]
    unseen = [torch.isnan(t) for t in pools]
    kw = dict(opts)
    if kw.pop("slopes", False):
        kw["slopes"] = torch.full((8,), 2.0 ** -6, device="cuda")
    kw["key_begin"] = i32(np.full(sum(counts), 3))
    for t, m in zip(pools, unseen):      # the first three keys of sequence 0 are seen by no row
        m[c.table_np[0, 0], :, :3] = True
        m[c.table_np[1, 0], :, :3] = True
    ref = None
    top = torch.finfo(pools[0].dtype).max
    for value in (0.5, float("nan"), top, -top, float("inf"), -float("inf"), 1e3):
        for t, m in zip(pools, unseen):
            t[m] = value
        out, _, _ = attend_case(c, 8, counts, pos, **kw)
        kvr.kvr_paged_status(c.p)
        ref = out if ref is None else ref
        assert torch.isfinite(out).all() and torch.equal(bits(out), bits(ref)), value


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1, 1], [70, 33]])
@pytest.mark.parametrize("scale,cap", [(2.0 ** 64, 2.0 ** -64), (2.0 ** -64, 2.0 ** 64), (2.0 ** -64, 2.0 ** -64)])
def test_extreme_caps_and_scales_of_flat_rows(fmt, dh, group, counts, scale, cap):
    """Queries of zeros under the ends of both ranges: the mean of the visible values."""
    lens = [400, 77]
    c = Paged(fmt, lens, 2, dh, 32, "hnd", group, seed=5)
    pos = tail(lens, counts)
    out, q, _ = attend_case(c, 8, counts, pos, q_scale=0.0, scale=scale, softcap=cap)
    kvr.kvr_paged_status(c.p)
    check_attend(c, 8, counts, pos, out, q, scale=scale, softcap=cap)


MALFORMED = [([0, 9, 4], [0, 1]), ([-3, 2, 4], [0]), ([2, 1, 0], [0, 1]), ([3, 2, 1], [0, 1]), ([1, 2, 4], [0]),
             ([0, 3, 9], [1]), ([0, 4, 9], [1]), ([0, 3, 2], [1]), ([4, 4, 4], [0]), ([-3, -1, -1], [0, 1]),
             ([0, -2 ** 31, 2 ** 31 - 1], [0, 1])]


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("cu,bad", MALFORMED)
def test_malformed_row_offsets_are_alike_in_every_call(fmt, dh, group, cu, bad):
    """Offsets that do not begin at 0, fall or pass n_rows are reported by each
    of the three calls.  Append and read then touch nothing, attention leaves
    alone the rows of the sequences whose offsets they are (bad)."""
    c = Paged(fmt, [20, 20], 2, dh, 16, "hnd", group, seed=1, spare=4)
    pos = np.array([1, 2, 3, 4])
    good = np.full(4, -1)
    for b in {0, 1} - set(bad):
        good[cu[b]:cu[b + 1]] = b
    x = torch.ones(4, 2, dh, device="cuda", dtype=c.row_dtype)
    q = torch.randn(4, 8, dh, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(c.row_dtype)

    def reported():
        with pytest.raises(kvr.KvrError, match="index") as e:
            kvr.kvr_paged_status(c.p)
        assert e.value.status == kvr.KVR_EDEVICE
        kvr.kvr_paged_status(c.p)

    out = torch.full_like(q, 7.0)
    for max_rows in (4, 1):
        ws = torch.empty(kvr.kvr_paged_workspace_bytes(c.p, 8, 4, max_rows), dtype=torch.uint8, device="cuda")
        kvr.kvr_paged_attend(c.p, None, max_rows, i32(cu), i32(pos), q, out, ws)
        reported()
        if max_rows == 4:
            for r in range(4):
                if good[r] >= 0:
                    one = [1 if b == good[r] else 0 for b in range(2)]
                    check_attend(c, 8, one, pos[r:r + 1], out[r:r + 1], q[r:r + 1])
        assert torch.all(out[torch.as_tensor(good < 0)] == 7.0)
    back = torch.full((4, 2, dh), 9.0, device="cuda", dtype=c.row_dtype)
    kvr.kvr_paged_read(c.p, i32(cu), i32(pos), back, back.clone())
    reported()
    assert torch.all(back == 9.0)
    pools = [t for t in (c.k, c.v, c.ks, c.vs) if t is not None]
    before = [bits(t).clone() for t in pools]
    turned = torch.full_like(q, 5.0)
    kvr.kvr_paged_append(c.p, i32(cu), i32(pos), x, x, None, q, turned)
    reported()
    assert all(torch.equal(bits(t), b) for t, b in zip(pools, before)) and torch.all(turned == 5.0)


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
def test_one_row_of_a_wide_tensor_turns_in_place(fmt, dh, group):
    """A single row is packed whatever its stride: a decode step's fused q, k, v."""
    c = Paged(fmt, [40], 2, dh, 16, "hnd", group, seed=1)
    x = torch.randn(1, 12, dh, device="cuda").to(c.row_dtype)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    rope = OP.rope_table(64, dh, THETA)
    want = torch.from_numpy(OP.rotate(q.float().cpu().numpy(), rope[[39]])).to(c.row_dtype)
    rest = x[:, 8:].clone()
    kvr.kvr_paged_append(c.p, i32([0, 1]), i32([39]), k, v, torch.from_numpy(rope).cuda(), q, q)
    kvr.kvr_paged_status(c.p)
    assert torch.equal(bits(q.cpu()), bits(want)) and torch.equal(bits(x[:, 8:]), bits(rest))


@pytest.mark.parametrize("fmt,dh,group", ATTEND)
@pytest.mark.parametrize("counts", [[1], [70]])
@pytest.mark.parametrize("alpha", [-64.0, -1000.0, -2.0 ** 17, 5000.0])
def test_a_bias_that_all_keys_share_costs_its_own_rounding(fmt, dh, group, counts, alpha):
    """The plain softmax, with logits off by 2^-24 of the bias twice: in its
    sum with the logit and in base 2's factor (check_attend's bound without
    the bias, and that)."""
    c = Paged(fmt, [517], 2, dh, 16, "hnd", group, seed=2)
    pos = tail([517], counts)
    bit = torch.full((c.max_pages * 16 // 32 + 1,), -1, dtype=torch.int32, device="cuda")
    out, q, _ = attend_case(c, 8, counts, pos, alpha=alpha, local_bits=bit)
    kvr.kvr_paged_status(c.p)
    K, V, step = c.rows64(0)
    got, q64 = out.double().cpu().numpy(), q.double().cpu().numpy()
    o, spread, noise = OP.attend(q64, K, V, np.zeros(len(pos)), pos + 1, v_step=step)
    f32 = fmt == "f32"
    r = 2.0 ** -24 if f32 else 2.0 ** -8
    d = 128 * 2.0 ** -24 * noise[..., None] * (16 if fmt == "int4" else 1) + (2.0 ** -19 if f32 else 2.0 ** -14)
    d = d + 2 * abs(alpha) * 2.0 ** -24
    assert np.all(np.abs(got - o) <= r * np.abs(o) + ((0 if f32 else r) + 2 * d) * spread + 1e-30)


@pytest.mark.parametrize("fmt,dh,group", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1, 1], [12, 9, 12], [70, 0, 33]])
def test_tables_far_wider_than_their_sequences(fmt, dh, group, counts):
    """A serving table of 131072 positions; two of its sequences share their
    first pages.  The masks' words follow the table's width."""
    lens, wide = [300, 400, 77], 131072 // 16
    c = Paged(fmt, lens, 2, dh, 16, "hnd", group, seed=17, max_pages=wide)
    c.table_np[1, :5] = c.table_np[0, :5]
    c.table.copy_(i32(c.table_np))
    pos = tail(lens, counts)
    loc = np.random.default_rng(1).random((3, wide * 16)) < 0.3
    out, q, _ = attend_case(c, 8, counts, pos, alpha=-2.0, local_bits=bit_words(loc))
    kvr.kvr_paged_status(c.p)
    check_attend(c, 8, counts, pos, out, q, alpha=-2.0, loc=loc)
