"""Packed rows at the ends of their ranges: the quantiser's formula bit for bit,
norms whose squares or products leave fp32's middle, and rows in their
thousands, every one of them checked."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")
from test_gpu_rows import DTYPES, HALF, REL, empty_codes, f64  # noqa: E402


def test_codes_are_the_formulas_bits():
    """scale = top * fp32(1/127), code = rint(y * (1 / scale)) with the product
    rounded to fp32 before it goes to an integer: where that lands on a half,
    the code is the even one."""
    y = np.random.default_rng(0).standard_normal((4000, 2048)).astype(np.float32)
    scale = np.abs(y).max(1) * np.float32(1 / 127)
    inv = np.float32(1) / scale
    want = np.rint(y * inv[:, None])
    once = np.rint(y.astype(np.float64) * inv[:, None].astype(np.float64))
    assert (want != once).any()   # the inputs tell the two apart
    for pad in (0, 3):            # aligned rows, and rows that are not
        x = torch.from_numpy(np.pad(y, ((0, 0), (0, pad)))).cuda()[:, :2048]
        codes, got = empty_codes(4000, 2048, pad)
        kvr.kvr_rows_quantise(x, codes, got)
        np.testing.assert_array_equal(got.cpu().numpy(), scale)
        np.testing.assert_array_equal(codes.cpu().numpy(), want)


# ---------------------------------------------------------------- norms far from one
SMALLEST = 2.0 ** -126


def check_norm(x, w, eps):
    """Rows of any size against the definition.  A row whose sum of squares
    passes fp32's range, or whose mean(h^2) + eps lies below 2^-126, is NaN.
    For the others, to the bounds of test_gpu_rows: h w rounds to multiples of
    2^-149 below 2^-126, so y is off by 2^-150 r more; subnormal outputs round
    to the multiples of their type (fp32 2^-149, bf16 2^-133)."""
    dtype = "f32" if x.dtype == torch.float32 else "bf16"
    n, d = x.shape
    out, (codes, scale) = torch.empty_like(x), empty_codes(n, d)
    kvr.kvr_rows_norm(x, w, eps, out=out, codes=codes, scales=scale)
    h, q = f64(x), (f64(x) ** 2).mean(1) + eps
    over, under = q * d / 2.0 ** 128, q / SMALLEST
    lost = (over >= 1) | (under < 1)
    assert not ((np.abs(over - 1) < 0.01) | ((np.abs(under - 1) < 0.01) & (eps == 0))).any(), "a case next to a border"
    with np.errstate(divide="ignore", invalid="ignore"):
        r = 1 / np.sqrt(q)
        y = h * r[:, None] * f64(w)
    codes, scale, out = f64(codes), f64(scale), f64(out)
    assert np.isnan(scale[lost]).all() and (codes[lost] == 0).all() and np.isnan(out[lost]).all()
    y, r, codes, scale, out = (t[~lost] for t in (y, r, codes, scale, out))
    fine = 2.0 ** -150 * r[:, None]
    least = 2.0 ** (-150 if dtype == "f32" else -134)
    assert np.all(np.abs(out - y) <= (HALF[dtype] + REL) * np.abs(y) + fine + 2.0 ** -149 + least)
    s = np.abs(y).max(1) / 127
    assert not (np.abs(s / SMALLEST - 1) < 0.01).any(), "a scale next to the border"
    none = s < SMALLEST
    assert (scale[none] == 0).all() and (codes[none] == 0).all()
    s, y, fine, codes, scale = s[~none], y[~none], fine[~none], codes[~none], scale[~none]
    assert np.all(np.abs(scale - s) <= (REL + 2.0 ** -22) * s + fine[:, 0] / 64)
    assert np.all(np.abs(codes * scale[:, None] - y) <= REL * np.abs(y) + (0.5 + 2.0 ** -14) * scale[:, None] + 2 * fine)
    return lost, none


def rows_of_size(exponents, d, dtype, seed):
    """Rows of magnitude 2^e, from half of it to one and a half."""
    g = np.random.default_rng(seed)
    x = np.exp2(np.asarray(exponents, np.float64))[:, None] * g.uniform(0.5, 1.5, (len(exponents), d)) * g.choice([-1, 1], (len(exponents), d))
    return torch.from_numpy(x).to(DTYPES[dtype]).cuda()


# a warp a row, a block a row with one to four units a thread, unaligned, read twice
NORM_WIDTHS = [64, 300, 1024, 4096, 4099, 9000, 24000]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", NORM_WIDTHS)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -126, 1e-30, 1e-5])
def test_norm_of_large_and_of_tiny_squares(dtype, d, eps):
    """Magnitudes whose squares overflow, sum to more than fp32 holds, or
    vanish: the row is NaN, not zeros or a wrong root; all others are right."""
    x = rows_of_size([-100, -80, -70, -66, -62, -50, -20, 0, 20, 50, 54, 57, 59, 62, 63, 66, 100, 120], d, dtype, d)
    lost, _ = check_norm(x, torch.ones(d, dtype=x.dtype, device="cuda"), eps)
    assert lost[-2:].all() and not lost[4:11].any() and (lost[:4] == (eps == 0)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", NORM_WIDTHS)
@pytest.mark.parametrize("eps,size", [(0.0, 0), (1e-12, -40), (2.0 ** -126, 0), (1e-30, -70), (1e-12, 0), (1e-5, 0), (1e-5, 20)])
def test_norm_of_tiny_products_keeps_its_codes(dtype, d, eps, size):
    """A row's own scale decides whether it stands for zeros, not the one
    before the root: h = 1e-37 with eps = 1e-12 is y = 1e-31.  Weights of 2^size."""
    x = rows_of_size([-145, -135, -128, -123, -117, -110, -101, -92, -90, -88, -70, -62, -40, 0], d, dtype, d + 1)
    w = rows_of_size([size], d, dtype, 1)[0].abs()
    lost, none = check_norm(x, w, eps)
    assert not lost[-3:].any()
    if (eps, size) == (1e-12, 0):
        assert not none[2:].any()
