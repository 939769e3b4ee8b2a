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


@pytest.mark.parametrize("d", NORM_WIDTHS)
@pytest.mark.parametrize("eps,zeros", [(0.0, False), (1e-44, True), (1e-40, True), (1e-12, True)])
def test_norm_of_zero_rows(d, eps, zeros):
    """0 / sqrt(eps) is 0 for any eps above 0, and no number for eps = 0."""
    for dtype in DTYPES.values():
        x, w = torch.zeros(3, d, dtype=dtype, device="cuda"), torch.ones(d, dtype=dtype, device="cuda")
        out, (codes, scale) = torch.full_like(x, 3), empty_codes(3, d)
        kvr.kvr_rows_norm(x, w, eps, out=out, codes=codes, scales=scale)
        assert (codes == 0).all()
        assert ((scale == 0).all() and (out == 0).all()) if zeros else (scale.isnan().all() and out.isnan().all())


# ---------------------------------------------------------------- more rows than blocks
def off_by(codes, scale, y, rel):
    """The furthest of every row from check_codes' bounds, on the GPU: at most 0 where all hold."""
    top = y.abs().amax(1) / 127
    s = scale.double()
    a = (s - top).abs() - (rel + 2.0 ** -22) * top
    b = ((codes.double() * s[:, None] - y).abs() - rel * y.abs()).amax(1) - (0.5 + 2.0 ** -14) * s
    return float(torch.maximum(a, b).amax())


def many(n, d, dtype, seed, pad):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, d + pad, generator=g, device="cuda") * torch.exp(torch.randn(n, 1, generator=g, device="cuda"))
    return x.to(DTYPES[dtype])[:, :d]


# (rows, width): more rows than the GPU holds blocks, or warps, of every kernel
MANY = [(20000, 40), (20000, 264), (20000, 500), (6000, 520), (6000, 1792), (6000, 2056), (2500, 4096), (2500, 8200), (2500, 14336), (1200, 20488)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", MANY)
@pytest.mark.parametrize("off", [0, 1])
def test_every_row_of_thousands(dtype, n, d, off):
    """Norm, gate and quantiser where a block or a warp takes many rows in turn,
    aligned rows and rows (off = 1) of odd widths that begin anywhere."""
    d, pad = d - off, 7 * off if off else 8
    code = torch.zeros(n, d + pad, dtype=torch.int8, device="cuda")
    codes, scale = code[:, :d], torch.empty(n, device="cuda")
    x = many(n, d, dtype, d, pad)
    kvr.kvr_rows_quantise(x, codes, scale)
    assert off_by(codes, scale, x.double(), 0.0) <= 0
    # the gate: |g| below 40
    gu = many(n, 2 * d, dtype, d + 1, pad).clamp(-40, 40)
    out = torch.empty(n, d + pad, dtype=x.dtype, device="cuda")[:, :d]
    codes.fill_(99)
    kvr.kvr_rows_swiglu(gu, out=out, codes=codes, scales=scale)
    y, rel = gu[:, :d].double() * torch.sigmoid(gu[:, :d].double()) * gu[:, d:].double(), 2.0 ** (-17 if dtype == "bf16" else -20)
    assert off_by(codes, scale, y, rel) <= 0
    assert bool(((out.double() - y).abs() <= (HALF[dtype] + rel) * y.abs() + 1e-37).all())
    del gu, y
    # the norm, both outputs in place
    res, w = many(n, d, dtype, d + 2, pad), (1 + 0.3 * many(1, d, "f32", 3, 0)[0].tanh()).to(x.dtype)
    h = x.double() + res.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * w.double()
    codes.fill_(99)
    kvr.kvr_rows_norm(x, w, 1e-5, residual=res, sum_out=res, out=x, codes=codes, scales=scale)
    # n/t + 12 additions of the sum are at most 52 (see test_gpu_rows): a thread has up to 32 elements
    assert off_by(codes, scale, y, REL) <= 0
    assert bool(((x.double() - y).abs() <= (HALF[dtype] + REL) * y.abs() + 1e-37).all())
    assert bool(((res.double() - h).abs() <= HALF[dtype] * h.abs() + 2.0 ** -24 * h.abs()).all())
    assert int(torch.count_nonzero(code[:, d:])) == 0


@pytest.mark.parametrize("n,d", [((1 << 23) + 1000, 1), ((1 << 28) + 1000, 16)])
def test_read_back_of_more_rows_than_a_grid(n, d):
    """Rows behind the grid's last block are its first ones' again."""
    g = torch.Generator(device="cuda").manual_seed(d)
    codes = torch.empty(n, d, dtype=torch.int8, device="cuda").random_(-127, 128, generator=g)
    scale = torch.rand(n, generator=g, device="cuda")
    out = torch.full((n, d), 3.0, dtype=torch.bfloat16, device="cuda")
    kvr.kvr_rows_dequantise(codes, scale, out)
    for a in range(0, n, 1 << 26):
        b = min(n, a + (1 << 26))
        assert torch.equal(out[a:b], (codes[a:b].float() * scale[a:b, None]).bfloat16())
