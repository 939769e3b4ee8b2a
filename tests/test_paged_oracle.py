"""The paged cache's plain definitions against each other, and every refusal
of the paged entry points that needs no GPU (CPU only: the addresses passed
are never read)."""
import ctypes as C

import numpy as np
import pytest

import oracle
from oracle import paged as OP


def test_pack_is_a_permutation_of_codes():
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, (5, 3, 128), dtype=np.uint8)
    np.testing.assert_array_equal(OP.unpack(OP.pack(code)), code)
    # dim 4u + e: bits 4e.. of the two-byte unit at place 4 (u % 8) + u // 8
    one = np.zeros(128, np.uint8)
    one[77] = 9    # u = 19, e = 1
    assert OP.pack(one).view("<u2")[4 * 3 + 2] == 9 << 4


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantised_values_are_within_half_a_step(group):
    """|value - x| <= s/2 inside [o, o + 15 s]; the roundings of o and of s
    (fp16, half-step 2^-11 each) move the range's ends by at most |o| 2^-11
    and 15 s 2^-11 beside the range's own 15 s >= hi - lo less that."""
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((64, 2, 128)) * 10 ** rng.uniform(-3, 3, (64, 2, 1)) + rng.standard_normal((64, 2, 1)) * 5)
    x = x.astype(np.float32)
    code, meta = OP.quantise(x, group)
    v = OP.values(OP.pack(code), meta, group)
    m = np.repeat(meta.astype(np.float64), group, -2)
    s, o = m[..., 0], m[..., 1]
    bound = s / 2 + 2.0 ** -11 * np.abs(o) + 15 * s * 2.0 ** -10 + 2.0 ** -24
    assert np.all(np.abs(v - x) <= bound)


def test_flat_and_extreme_groups():
    x = np.zeros((3, 1, 128), np.float32)
    x[1] = 7.25
    x[2, 0, 5] = 1e6    # saturates at 2^15
    code, meta = OP.quantise(x, 64)
    v = OP.values(OP.pack(code), meta, 64)
    np.testing.assert_array_equal(v[0], 0)
    np.testing.assert_array_equal(v[1], 7.25)
    assert np.isfinite(v).all() and v[2, 0, 5] == v.max() and v.max() < 65504


def test_rotation_composes_with_the_refresh_oracle():
    """The table's rotation at g equals the refresh oracle's rotary map."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 2, 128)).astype(np.float32)
    pos = np.array([0, 1, 17, 400, 1023, 2000])
    got = OP.rotate(x, OP.rope_table(2001, 128, 5e5)[pos])
    want = oracle.rope(x.astype(np.float64).swapaxes(0, 1), pos, 5e5).swapaxes(0, 1)
    # one fp32 table rounding and three fp32 operations on values up to sqrt(2) |x|
    assert np.max(np.abs(got - want)) <= 4 * 2.0 ** -24 * 2 * np.max(np.abs(x))


def test_attend_empty_rows_and_plain_softmax():
    rng = np.random.default_rng(4)
    q, K, V = rng.standard_normal((3, 4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    o, _, _ = OP.attend(q, K, V, [0, 5, 3], [9, 5, 4])
    assert np.all(o[1] == 0)
    np.testing.assert_allclose(o[2], np.repeat(V[:, 3], 2, 0))
    x = np.einsum("hd,jd->hj", q[0, :2], K[0]) / np.sqrt(8)
    w = np.exp(x) / np.exp(x).sum(-1, keepdims=True)
    np.testing.assert_allclose(o[0, :2], w @ V[0])


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def kvr():
    from selective_kv_cache_gb300 import build
    build.build()
    from selective_kv_cache_gb300 import kvr
    return kvr


A = 0x100000   # an aligned address that no call may read


def _pages(kvr, **kw):
    p = kvr.kvr_pages(kvr.KVR_BF16, 2, 128, 16, 0, 8, 2, 4, 32, 16, 1, A, A, None, None, A, A, A)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _append(kvr, p, n=4, cu=A, pos=A, k=A, ks=256, v=A, vs=256, rope=A, rope_len=64, q=A, qs=512, qo=A, hq=4):
    return kvr.lib.kvr_paged_append(C.byref(p) if p else None, n, cu, pos, k, ks, v, vs, rope, rope_len, q, qs, qo, hq,
                                    None)


def _attend(kvr, p, opts=None, hq=4, n=4, m=1, cu=A, pos=A, q=A, qs=512, o=A, os_=512, ws=A, wb=1 << 40):
    return kvr.lib.kvr_paged_attend(C.byref(p) if p else None, C.byref(opts) if opts else None, hq, n, m, cu, pos, q,
                                    qs, o, os_, ws, wb, None)


def _read(kvr, p, n=4, cu=A, pos=A, k=A, ks=256, v=A, vs=256):
    return kvr.lib.kvr_paged_read(C.byref(p) if p else None, n, cu, pos, k, ks, v, vs, None)


BAD_PAGES = [
    (dict(format=7), "EINVAL"), (dict(n_kv_heads=0), "EINVAL"), (dict(n_pages=0), "EINVAL"), (dict(batch=0), "EINVAL"),
    (dict(max_pages=0), "EINVAL"), (dict(head_dim=64), "EUNSUPPORTED"), (dict(head_dim=96), "EUNSUPPORTED"),
    (dict(page_size=8), "EUNSUPPORTED"), (dict(page_size=48), "EUNSUPPORTED"), (dict(page_size=512), "EUNSUPPORTED"),
    (dict(group=32), "EINVAL"), (dict(page_stride=0), "EINVAL"), (dict(head_stride=-1), "EINVAL"),
    (dict(slot_stride=0), "EINVAL"), (dict(k=None), "EINVAL"), (dict(v=A + 8), "EINVAL"),
    (dict(page_table=None), "EINVAL"), (dict(kv_len=None), "EINVAL"), (dict(err=None), "EINVAL"),
    (dict(page_table=A + 2), "EINVAL"), (dict(batch=1 << 21), "EUNSUPPORTED"),
    (dict(page_stride=(1 << 21) + 1), "EUNSUPPORTED"), (dict(slot_stride=1 << 22), "EUNSUPPORTED"),
    (dict(head_stride=1 << 32), "EUNSUPPORTED"), (dict(max_pages=1 << 27), "EUNSUPPORTED"),
    (dict(format=2, group=0, k_scale=A, v_scale=A), "EINVAL"), (dict(format=2, group=16, k_scale=A, v_scale=A), "EINVAL"),
    (dict(format=2, group=32, k_scale=None, v_scale=A), "EINVAL"),
    (dict(format=2, group=32, k_scale=A, v_scale=A + 4), "EINVAL"),
]


@pytest.mark.parametrize("bad,status", BAD_PAGES)
def test_bad_pages_are_refused_by_every_call(kvr, bad, status):
    p = _pages(kvr, **bad)
    for call in (_append, _read, _attend):
        assert kvr.STATUS_NAMES[call(kvr, p)] == status, call
    assert kvr.kvr_paged_workspace_bytes(p, 4, 4, 1) == 0
    assert kvr.kvr_last_error()


def test_null_pages(kvr):
    for call in (_append, _read, _attend):
        assert call(kvr, None) == kvr.KVR_EINVAL
    assert kvr.lib.kvr_paged_workspace_bytes(None, 4, 4, 1) == 0
    assert kvr.lib.kvr_paged_status(None, None) == kvr.KVR_EINVAL
    assert kvr.lib.kvr_paged_status(C.byref(_pages(kvr, err=None)), None) == kvr.KVR_EINVAL


@pytest.mark.parametrize("kw", [dict(n=-1), dict(cu=None), dict(pos=None), dict(cu=A + 1), dict(k=None), dict(v=A + 4),
                                dict(ks=255), dict(ks=257), dict(vs=128), dict(rope_len=0), dict(rope=A + 4),
                                dict(q=None), dict(qo=None), dict(qo=A + 8), dict(hq=0), dict(qs=256),
                                dict(qs=1024, qo=A)])
def test_append_refusals(kvr, kw):
    assert _append(kvr, _pages(kvr), **kw) == kvr.KVR_EINVAL


@pytest.mark.parametrize("kw", [dict(n=-1), dict(cu=None), dict(pos=None), dict(k=A + 8), dict(ks=255), dict(vs=264 - 4)])
def test_read_refusals(kvr, kw):
    assert _read(kvr, _pages(kvr), **kw) == kvr.KVR_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), "EINVAL"), (dict(m=0), "EINVAL"), (dict(hq=3), "EINVAL"), (dict(hq=0), "EINVAL"),
    (dict(hq=34), "EUNSUPPORTED"), (dict(cu=None), "EINVAL"), (dict(pos=None), "EINVAL"), (dict(q=None), "EINVAL"),
    (dict(q=A + 8), "EINVAL"), (dict(qs=511), "EINVAL"), (dict(o=None), "EINVAL"), (dict(os_=508), "EINVAL"),
    (dict(ws=None), "EINVAL"), (dict(ws=A + 128), "EINVAL"), (dict(wb=1024), "EINVAL")])
def test_attend_refusals(kvr, kw, status):
    assert kvr.STATUS_NAMES[_attend(kvr, _pages(kvr), **kw)] == status


@pytest.mark.parametrize("kw", [dict(scale=-1.0), dict(scale=float("nan")), dict(softcap=-2.0),
                                dict(softcap=float("inf")), dict(scale=1e-20), dict(scale=1e20),
                                dict(softcap=1e-20), dict(softcap=2e19), dict(alpha=float("nan")), dict(beta=float("-inf")),
                                dict(slopes=A + 2), dict(key_begin=A + 1), dict(local_bits=A + 3)])
def test_score_option_refusals(kvr, kw):
    o = kvr.kvr_score_opts()
    for k, v in kw.items():
        setattr(o, k, v)
    assert _attend(kvr, _pages(kvr), opts=o) == kvr.KVR_EINVAL


def test_no_rows_enqueue_nothing(kvr):
    p = _pages(kvr)
    assert _append(kvr, p, n=0, cu=None, pos=None, k=None, v=None) == kvr.KVR_OK
    assert _read(kvr, p, n=0) == kvr.KVR_OK
    assert _attend(kvr, p, n=0, q=None, o=None, ws=None) == kvr.KVR_OK


def test_call_too_large_is_refused(kvr):
    p = _pages(kvr, batch=1 << 20, max_pages=1 << 22, page_size=256)
    assert _attend(kvr, p) == kvr.KVR_EUNSUPPORTED


@pytest.mark.parametrize("kw,n,m", [
    (dict(batch=1 << 20, max_pages=1 << 22, page_size=256, n_kv_heads=65535), 1 << 16, 1 << 16),
    (dict(batch=1 << 18, max_pages=1 << 22, page_size=256, n_kv_heads=65535), 1 << 18, 1 << 18)])
def test_call_too_large_for_64_bits_is_refused(kvr, kw, n, m):
    """Items times units times heads past 2^63 is too large as well."""
    p = _pages(kvr, **kw)
    assert kvr.kvr_paged_workspace_bytes(p, kw["n_kv_heads"], n, m) == 0
    assert _attend(kvr, p, hq=kw["n_kv_heads"], n=n, m=m) == kvr.KVR_EUNSUPPORTED


def test_binding_refuses_host_tensors(kvr):
    import torch
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        kvr.pages("bf16", k, k.clone(), t, t[0, :1], t[0], 2, 16)
