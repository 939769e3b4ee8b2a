"""kvr_rows_swiglu over every bf16 gate, to fp32's precision: a row of one
element has its value, 127 times its scale, in fp32.

Bounds, relative to the value, in units of 2^-23.  bf16 rows: the approximate
exponential is documented to 2 + 1.173 |g| ulp, the approximate division to 2,
the sum, the product with u and the scale's two roundings take half of one each:
6 + 1.2 |g| with what is of second order.  fp32 rows: 2 ulp of the exponential
and five halves: 8 is 2^-20."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("up", [1.0, -2.0 ** 60])
def test_every_gate(dtype, up):
    bits = torch.arange(1 << 16, dtype=torch.int32)
    g = (bits << 16).view(torch.float32)
    g = g[torch.isfinite(g) & (g.abs() < 2.0 ** 60)]
    x = torch.stack([g, torch.full_like(g, up)], 1).to(dtype).cuda()
    n = x.shape[0]
    codes, scale = torch.full((n, 1), 9, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    kvr.kvr_rows_swiglu(x, codes=codes, scales=scale)
    v = g.double().numpy()
    with np.errstate(over="ignore"):
        y = v / (1 + np.exp(-v)) * up
    got = scale.cpu().double().numpy() * codes.cpu().numpy()[:, 0]
    # exp(-g) past the range that the division takes: 2^126 (bf16), fp32's (fp32), and the quotient below 2^-119 counts as 0
    cut = -126 * np.log(2) if dtype == torch.bfloat16 else -128 * np.log(2)
    gone, near = v < cut - 0.01, np.abs(v - cut) <= 0.01
    assert not near.any() and (got[gone] == 0).all() and (np.abs(y[gone]) <= 2.0 ** -119 * abs(up)).all()
    tiny = np.abs(y) / 127 < 2.0 ** -126
    assert (got[tiny] == 0).all()
    ok = ~gone & ~tiny
    rel = (6 + 1.2 * np.abs(v[ok])) * 2.0 ** -23 if dtype == torch.bfloat16 else 2.0 ** -20
    # a positive gate's exponential vanishes next to 1: it counts at most as itself
    off = np.abs(got[ok] - y[ok]) / np.abs(y[ok])
    assert (off <= rel).all(), (off / rel).max()
    assert (np.abs(codes.cpu().numpy()[ok]) == 127).all()
