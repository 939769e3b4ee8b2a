"""Packed-row operators on the CPU: the rotary frequencies of kvr_rope_init,
the oracle's own identities, and what the entry points refuse before any
launch."""
import ctypes
import math

import numpy as np
import pytest

from oracle import rows as OR

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")
lib = kvr.lib
P1, P3 = 1 << 20, (1 << 20) + 1   # an aligned and a misaligned address; nothing is ever read


# ---------------------------------------------------------------- rotary frequencies
SCALINGS = [("plain", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
            ("bands", dict(factor=8.0, low=1.0, high=4.0, original_len=8192)),
            ("yarn", dict(factor=16.0, low=1.0, high=32.0, original_len=4096)),
            ("yarn", dict(factor=2.0, low=0.5, high=1.0, original_len=7))]


@pytest.mark.parametrize("scaling,more", SCALINGS)
@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (64, 10000.0), (4, 10000.0), (256, 1e6)])
def test_rope_init_gives_the_formulas_frequencies(scaling, more, rot, theta):
    """turns = f / 2 pi * 2^64, truncated: off by one unit and by the few
    double roundings of f, 2^-49 of it."""
    r = kvr.rope(256, rot, theta=theta, scaling=scaling, **more)
    f, m = OR.frequencies(rot, scaling, theta, **more)
    got = np.array([int(t) for t in r.turns[:rot // 2]], np.float64) / 2.0 ** 64
    assert np.all(np.abs(got - f / (2 * math.pi)) <= 2.0 ** -49 * f + 2.0 ** -63)
    assert abs(r.attn - m) <= 2.0 ** -24 * m
    assert all(t == 0 for t in r.turns[rot // 2:])
    assert kvr.rope(256, rot, theta=theta, scaling=scaling, attn_factor=0.5, **more).attn == 0.5


def test_rotation_identities():
    """Lengths stay, the inverse takes it out, turns add up, both layouts are
    permutations of one another."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 12))
    r = kvr.rope(12, 8, theta=100.0)
    t = list(r.turns[:4])
    g = [0, 1, -7, 2**31 - 1, -2**31]
    y = OR.rotate(x, g, t)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    np.testing.assert_array_equal(y[0], x[0])
    np.testing.assert_allclose(OR.rotate(y, g, t, inverse=True), x, atol=1e-13)
    np.testing.assert_allclose(OR.rotate(OR.rotate(x, [3] * 5, t), [-10] * 5, t), OR.rotate(x, [-7] * 5, t), atol=1e-13)
    perm = [0, 2, 4, 6, 1, 3, 5, 7, 8, 9, 10, 11]   # interleaved dims in half order
    np.testing.assert_allclose(OR.rotate(x, g, t, layout="interleaved")[..., perm], OR.rotate(x[..., perm], g, t), atol=0)
    np.testing.assert_allclose(y[1, 0, 0], x[1, 0, 0] * math.cos(1) - x[1, 0, 4] * math.sin(1), rtol=1e-13)


@pytest.mark.parametrize("change", [dict(head_dim=0), dict(head_dim=258), dict(head_dim=127), dict(rotary_dim=130),
                                    dict(rotary_dim=0), dict(rotary_dim=63), dict(layout=2), dict(layout=-1),
                                    dict(scaling=5), dict(scaling=-1), dict(theta=1.0), dict(theta=math.inf),
                                    dict(theta=math.nan), dict(factor=0.5), dict(factor=math.nan),
                                    dict(scaling=3, low=0.0), dict(scaling=4, high=1.0), dict(scaling=3, high=math.inf),
                                    dict(scaling=4, original_len=0), dict(scaling=2, rotary_dim=2),
                                    dict(attn_factor=-1.0), dict(attn_factor=math.nan), dict(attn_factor=math.inf)])
def test_rope_init_refuses(change):
    a = dict(head_dim=128, rotary_dim=64, layout=0, scaling=0, theta=1e4, factor=2.0, low=1.0, high=4.0,
             original_len=64, attn_factor=0.0)
    kvr.kvr_rope_init(*a.values())
    with pytest.raises(kvr.KvrError) as e:
        kvr.kvr_rope_init(*{**a, **change}.values())
    assert e.value.status == kvr.KVR_EINVAL
    assert lib.kvr_rope_init(None, 128, 64, 0, 0, 1e4, 1.0, 0.0, 0.0, 0, 0.0) == kvr.KVR_EINVAL


# ---------------------------------------------------------------- refusals
def refused(call, good, **change):
    """The call with these arguments is refused; no argument set here reaches a launch."""
    return call(*{**good, **change}.values()) == kvr.KVR_EINVAL


def test_norm_refuses():
    good = dict(dtype=1, n=0, d=64, x=P1, xs=64, res=P1, rs=64, sum=P1, ss=64, w=P1, eps=1e-5, out=P1 + 4096, os=64,
                codes=P1, cs=64, scales=P1, stream=None)
    assert lib.kvr_rows_norm(*good.values()) == kvr.KVR_OK   # no rows: nothing is enqueued
    assert lib.kvr_rows_norm(*{**good, "res": None, "sum": None, "out": None}.values()) == kvr.KVR_OK
    assert lib.kvr_rows_norm(*{**good, "codes": None, "scales": None}.values()) == kvr.KVR_OK
    for change in (dict(dtype=2), dict(dtype=-1), dict(n=-1), dict(d=0), dict(d=(1 << 20) + 1), dict(x=None), dict(x=P3),
                   dict(xs=63), dict(xs=1 << 30), dict(res=P3), dict(rs=63), dict(sum=P3), dict(ss=-1), dict(w=None),
                   dict(w=P3), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(out=P3), dict(os=63),
                   dict(codes=None), dict(scales=None), dict(scales=P1 + 2), dict(cs=63),
                   dict(out=None, codes=None, scales=None), dict(n=2, xs=65), dict(n=2, rs=65, sum=P1),
                   dict(out=P1), dict(n=2, out=P1, sum=P1 + 8192, os=65)):
        assert refused(lib.kvr_rows_norm, good, **change), change
        assert kvr.kvr_last_error()


def test_swiglu_quantise_and_dequantise_refuse():
    good = dict(dtype=0, n=0, d=64, x=P1, xs=128, out=P1 + 4096, os=64, codes=P1, cs=64, scales=P1, stream=None)
    assert lib.kvr_rows_swiglu(*good.values()) == kvr.KVR_OK
    for change in (dict(dtype=3), dict(n=-1), dict(d=0), dict(x=None), dict(x=P1 + 2), dict(xs=127), dict(out=P1),
                   dict(out=P1 + 2), dict(os=63), dict(codes=None), dict(scales=None), dict(cs=1),
                   dict(out=None, codes=None, scales=None)):
        assert refused(lib.kvr_rows_swiglu, good, **change), change
    good = dict(dtype=0, n=0, d=64, x=P1, xs=64, codes=P1, cs=64, scales=P1, stream=None)
    assert lib.kvr_rows_quantise(*good.values()) == kvr.KVR_OK
    for change in (dict(dtype=2), dict(n=-1), dict(d=0), dict(x=None), dict(xs=63), dict(codes=None), dict(scales=None),
                   dict(cs=63), dict(scales=P3)):
        assert refused(lib.kvr_rows_quantise, good, **change), change
    good = dict(dtype=0, n=0, d=64, codes=P1, cs=64, scales=P1, out=P1, os=64, stream=None)
    assert lib.kvr_rows_dequantise(*good.values()) == kvr.KVR_OK
    for change in (dict(dtype=2), dict(n=-1), dict(d=0), dict(out=None), dict(out=P3), dict(os=63), dict(codes=None),
                   dict(scales=None), dict(cs=63)):
        assert refused(lib.kvr_rows_dequantise, good, **change), change


def test_rotate_and_table_refuse():
    r = kvr.rope(128)
    good = dict(rope=ctypes.addressof(r), dtype=1, n=0, pos=P1, q=P1, qs=512, hq=4, qo=P1, qos=512, k=P1, ks=256, hk=2, ko=P1, kos=256,
                flags=0, stream=None)
    assert lib.kvr_rows_rotate(*good.values()) == kvr.KVR_OK
    none = dict(q=None, hq=0, qo=None)
    assert lib.kvr_rows_rotate(*{**good, **none}.values()) == kvr.KVR_OK
    bad = kvr.rope(128)
    bad.rotary_dim = 130
    flat = kvr.rope(128)
    flat.attn = 0.0
    for change in (dict(rope=None), dict(rope=ctypes.addressof(bad)), dict(rope=ctypes.addressof(flat)), dict(dtype=2),
                   dict(n=-1), dict(pos=None), dict(pos=P3), dict(q=None), dict(qo=None), dict(q=P3), dict(qs=511),
                   dict(hq=-1), dict(hq=65536), dict(hk=0), dict(k=None, ko=None), dict(ko=P3), dict(kos=255),
                   dict(flags=2), dict(n=2, qos=520), {**none, "k": None, "hk": 0, "ko": None}):
        assert refused(lib.kvr_rows_rotate, good, **change), change
    assert lib.kvr_rope_table(ctypes.addressof(r), 0, P1, None) == kvr.KVR_OK
    for a in ((None, 4, P1, None), (ctypes.addressof(r), -1, P1, None), (ctypes.addressof(r), 4, None, None), (ctypes.addressof(r), 4, P1 + 4, None)):
        assert lib.kvr_rope_table(*a) == kvr.KVR_EINVAL


def test_binding_checks_tensors():
    """A wrong type, width, stride or a host tensor does not reach the library."""
    import torch
    x, c, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    w = torch.zeros(64)
    for call in (lambda: kvr.kvr_rows_norm(x, w, 1e-5, out=torch.zeros(4, 64)), lambda: kvr.kvr_rows_quantise(x, c, s),
                 lambda: kvr.kvr_rows_norm(x.half(), w.half(), 1e-5, out=x.half()), lambda: kvr.kvr_rows_swiglu(x[:, :63]),
                 lambda: kvr.kvr_rows_dequantise(c, s, x), lambda: kvr.kvr_rows_quantise(x[0], c, s),
                 lambda: kvr.kvr_rows_rotate(kvr.rope(64), torch.zeros(4, dtype=torch.int32)),
                 lambda: kvr.rope(64, layout="other"), lambda: kvr.kvr_rope_table(kvr.rope(64), 4, torch.zeros(4, 32, 2))):
        with pytest.raises(ValueError):
            call()


def test_divisions_by_multiplication():
    """The quotients of rows_rotate.cu: umulhi with ceil(2^(31 + l) / d) and a
    shift by l - 1 is the quotient for every numerator below 2^31."""
    rng = np.random.default_rng(1)
    for d in list(range(2, 300)) + [511, 512, 513, 65535, 131070] + [int(v) for v in rng.integers(2, 1 << 24, 300)]:
        bits = (d - 1).bit_length()
        mul = -(-(1 << (31 + bits)) // d)
        assert mul < 1 << 32
        for x in [0, 1, d - 1, d, d + 1, (1 << 31) - 1, (1 << 31) // d * d - 1, ((1 << 31) - 1) // d * d] + \
                [int(v) for v in rng.integers(0, 1 << 31, 20)]:
            assert (mul * x >> 32) >> (bits - 1) == x // d


def test_linear_refuses():
    good = dict(n_out=64, k=128, stride=128, codes=P1, scales=P1, bias=None, err=P1)
    args = dict(n=0, codes=P1, stride=128, scales=P1, dtype=1, out=P1, os=64, ws=P1, bytes=1 << 40, stream=None)

    def call(w=None, **change):
        s = kvr.kvr_linear_weights(*{**good, **(w or {})}.values())
        return lib.kvr_linear(ctypes.addressof(s), *{**args, **change}.values())

    assert call() == kvr.KVR_OK and call(dict(bias=P1)) == kvr.KVR_OK
    for w in (dict(n_out=0), dict(n_out=(1 << 20) + 1), dict(k=0), dict(k=65537), dict(stride=127), dict(stride=136),
              dict(codes=None), dict(codes=P1 + 8), dict(scales=None), dict(scales=P1 + 2), dict(bias=P3), dict(err=None)):
        assert call(w) == kvr.KVR_EINVAL, w
        s = kvr.kvr_linear_weights(*{**good, **w}.values())
        assert lib.kvr_linear_workspace_bytes(ctypes.addressof(s), 4) == 0
    for change in (dict(n=-1), dict(n=(1 << 22) + 1), dict(codes=None), dict(codes=P1 + 8), dict(stride=112),
                   dict(stride=136), dict(scales=None), dict(dtype=2), dict(out=None), dict(out=P3), dict(os=63),
                   dict(n=4, ws=None), dict(n=4, ws=P1 + 128), dict(n=4, bytes=255)):
        assert call(**change) == kvr.KVR_EINVAL, change
    assert lib.kvr_linear(None, *args.values()) == kvr.KVR_EINVAL
    assert lib.kvr_linear_workspace_bytes(None, 4) == 0
    s = kvr.kvr_linear_weights(*good.values())
    assert lib.kvr_linear_workspace_bytes(ctypes.addressof(s), 0) == 0
    assert lib.kvr_linear_status(None, None) == kvr.KVR_EINVAL


@pytest.mark.parametrize("n_out,k", [(1, 1), (2048, 1536), (4096, 14336), (28672, 4096)])
def test_linear_workspace_grows_with_the_rows(n_out, k):
    """A program that sizes it for its largest batch calls with fewer rows too."""
    s = kvr.kvr_linear_weights(n_out, k, -(-k // 16) * 16, P1, P1, None, P1)
    sizes = [lib.kvr_linear_workspace_bytes(ctypes.addressof(s), n) for n in range(1, 6000)]
    assert sizes[0] >= 1 and all(a <= b for a, b in zip(sizes, sizes[1:]))
