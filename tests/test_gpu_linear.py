"""kvr_linear on the GPU against integer sums (oracle.rows.linear).

Bound: the integer sum is exact (in fp32 up to 2^24; above, every one of the
k / 16 steps that add to it rounds by at most 2^-23 of the largest running
sum), its conversion, two products and the bias' addition round by 2^-24 each,
the output by half a step of its type."""
import numpy as np
import pytest
import torch

from oracle import rows as OR

pytestmark = pytest.mark.gpu

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def codes(n, k, seed, pad=None, lo=-128, hi=128):
    """int8 [n, k] whose rows lie a multiple of 16 bytes apart; what lies between them is not zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pad = -k % 16 if pad is None else pad
    return torch.randint(lo, hi, (n, k + pad), generator=g, device="cuda", dtype=torch.int8)[:, :k]


def scales(n, seed, size=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp(torch.randn(n, generator=g, device="cuda")) * size


class Case:
    def __init__(self, rows, n_out, k, dtype="bf16", bias=False, seed=0, pad=None, lo=-128, hi=128, out_pad=0):
        self.a, self.w = codes(rows, k, seed, pad, lo, hi), codes(n_out, k, seed + 1, pad, lo, hi)
        self.sa, self.sw = scales(rows, seed + 2), scales(n_out, seed + 3)
        self.bias = scales(n_out, seed + 4, 1.0) if bias else None
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.weights = kvr.linear_weights(self.w, self.sw, self.err, self.bias)
        self.wide = torch.full((rows + 1, n_out + out_pad), 7.0, dtype=DTYPES[dtype], device="cuda")
        self.out, self.dtype = self.wide[:rows, :n_out], dtype
        self.ws = torch.full((kvr.kvr_linear_workspace_bytes(self.weights, rows),), 255, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        kvr.kvr_linear(self.weights, self.a, self.sa, self.out, self.ws, stream)

    def check(self):
        kvr.kvr_linear_status(self.weights)
        # sums of products below 2^14: exact in float64, and fast there on the CPU
        acc = self.a.cpu().double().numpy() @ self.w.cpu().double().numpy().T
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        s = f(self.sa)[:, None] * f(self.sw)
        want = acc * s + (0 if self.bias is None else f(self.bias))
        k = self.a.shape[1]
        big = np.abs(acc) if k <= 1024 else np.maximum(np.abs(acc), 2.0 ** 24)   # running sums: see large_sums
        steps = 0.0 if np.abs(acc).max() < 2.0 ** 23 else k / 16 * 2.0 ** -23 * big * s
        bound = HALF[self.dtype] * np.abs(want) + 4 * 2.0 ** -24 * (np.abs(acc) * s + np.abs(want)) + steps + 1e-37
        got = f(self.out)
        off = np.abs(got - want) / bound
        assert np.isfinite(got).all() and off.max() <= 1, f"{(off > 1).sum()} of {off.size} off, worst {off.max():.3g} at " \
            f"{np.unravel_index(off.argmax(), off.shape)}"
        assert torch.all(self.wide[-1] == 7.0) and torch.all(self.wide[:, self.out.shape[1]:] == 7.0)


ROWS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 128, 129, 256, 257, 282, 300, 513]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("n_out,k", [(1, 1), (16, 64), (31, 63), (33, 65), (128, 128), (257, 1000), (640, 4096), (130, 5001),
                                     (1000, 333)])
def test_linear(rows, n_out, k):
    """Every row count around the kernels' borders; widths and lengths that end inside every tile."""
    for dtype, bias in (("f32", True), ("bf16", False)):
        c = Case(rows, n_out, k, dtype, bias, seed=rows + n_out + k, out_pad=3 if n_out % 2 else 8)
        c.run()
        c.check()


@pytest.mark.parametrize("rows,n_out,k", [(1, 6144, 4096), (8, 4096, 14336), (16, 2048, 1536), (64, 4096, 14336),
                                          (282, 4608, 3584), (96, 37888, 3584), (1024, 1536, 8960), (2000, 5000, 777),
                                          (7, 300, 65536), (40, 300, 65536), (8, 1530, 8960), (5, 1300, 8200),
                                          (8, 1100, 8192), (1, 3584, 18944), (64, 3584, 18944), (48, 12288, 4096),
                                          (33, 4600, 3600), (100, 4100, 4100), (20, 1000, 9000), (57, 1024, 12288),
                                          (64, 28672, 4096), (50, 28500, 4000), (9, 37888, 3584), (30, 20000, 1111),
                                          (64, 55000, 900), (128, 13000, 2000)])
def test_linear_of_model_shapes(rows, n_out, k):
    c = Case(rows, n_out, k, "f32", True, seed=3, lo=-100, hi=101)
    c.run()
    c.check()


@pytest.mark.parametrize("rows,n_out,k", [(64, 28672, 4096), (64, 6144, 4096), (128, 3584, 18944), (16, 4096, 14336),
                                          (282, 4608, 3584), (8, 4096, 14336)])
def test_linear_holds_over_many_launches(rows, n_out, k):
    """Every bit of a hundred launches, weights from HBM or from L2: no stage of
    codes is overwritten before it was read.  Sums below 2^24 are exact."""
    a, w = codes(rows, k, 3, lo=-100, hi=101), codes(n_out, k, 4, lo=-100, hi=101)
    want = a.double() @ w.double().T
    assert want.abs().max() < 2 ** 23
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    W = kvr.linear_weights(w, torch.ones(n_out, device="cuda"), err)
    ws = torch.empty(kvr.kvr_linear_workspace_bytes(W, rows), dtype=torch.uint8, device="cuda")
    out, one, wrong = torch.empty(rows, n_out, device="cuda"), torch.ones(rows, device="cuda"), torch.zeros((), device="cuda")
    other = torch.empty(200 << 20, dtype=torch.uint8, device="cuda")
    for i in range(100):
        out.fill_(float("nan"))
        if i % 3 == 0:
            other.fill_(i)
        kvr.kvr_linear(W, a, one, out, ws)
        wrong += (out != want).any()
    kvr.kvr_linear_status(W)
    assert wrong.item() == 0


@pytest.mark.parametrize("rows", [1, 8, 16, 40, 300])
def test_sums_are_integers(rows):
    """Scales of one: the output is the integer itself, bit for bit, wherever every running sum stays below 2^24."""
    c = Case(rows, 200, 1000, "f32", seed=5)
    c.sa.fill_(1)
    c.sw.fill_(1)
    c.run()
    kvr.kvr_linear_status(c.weights)
    want = c.a.cpu().double() @ c.w.cpu().double().T
    assert want.abs().max() < 2 ** 24 and torch.equal(c.out.cpu().double(), want)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("value", [127, -128])
def test_large_sums(rows, value):
    """All codes at an end of their range, k at its limit: up to 2^30."""
    c = Case(rows, 40, 65536, "f32", seed=6)
    c.a.fill_(value)
    c.w.fill_(value)
    c.sa.fill_(1)
    c.sw.fill_(2.0 ** -20)
    c.run()
    kvr.kvr_linear_status(c.weights)
    want = value * value * 65536 * 2.0 ** -20
    # integers are exact; fp32 sums round k / 16 times, each by at most 2^-23 of the largest
    assert (c.out.double() - want).abs().max() <= (0 if rows <= 16 else 65536 / 16 * 2.0 ** -23) * want


@pytest.mark.parametrize("rows", [1, 9, 40])
def test_rows_and_channels_without_a_number(rows):
    """A NaN scale is its own row's or channel's; zero scales give the bias."""
    c = Case(rows, 70, 256, "f32", True, seed=7)
    c.sa[rows - 1] = float("nan")
    c.sw[3] = float("nan")
    c.sw[5] = 0
    c.run()
    kvr.kvr_linear_status(c.weights)
    nan = torch.isnan(c.out)
    want = torch.zeros_like(nan)
    want[rows - 1] = True
    want[:, 3] = True
    assert torch.equal(nan, want)
    assert torch.equal(c.out[:-1, 5], c.bias[5].expand(rows - 1))


@pytest.mark.parametrize("rows", [1, 16, 64, 300])
def test_same_bits_every_time(rows):
    c = Case(rows, 4096, 1536, "bf16", seed=8)
    c.run()
    first = c.out.clone()
    for _ in range(3):
        c.ws.random_(0, 256)   # whatever the workspace holds
        c.out.fill_(0)
        c.run()
        assert torch.equal(c.out, first)


@pytest.mark.parametrize("rows", [5, 50, 400])
def test_captured_and_on_two_streams(rows):
    """A captured call replayed with other rows and weights, beside an eager one on another stream."""
    c, e = Case(rows, 520, 640, "f32", seed=9), Case(rows, 520, 640, "bf16", True, seed=10)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    c.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        c.run(s)
    for seed in (11, 12):
        c.a.copy_(codes(rows, 640, seed))
        c.w.copy_(codes(520, 640, seed + 5))
        c.out.fill_(0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        e.run()
        torch.cuda.synchronize()
        c.check()
        e.check()


def test_kernels_of_two_streams_side_by_side():
    """Batches that split k over clusters, shared tiles, many rows and few, in
    turn on two streams: whichever blocks meet on an SM, both finish."""
    shapes = [(64, 4096, 2048), (40, 640, 9000), (64, 24000, 800), (300, 2048, 1536), (4, 4096, 2048), (12, 2048, 1536)]
    cases = [[Case(*shape, "f32", seed=21 + i, lo=-100, hi=101) for i, shape in enumerate(shapes)] for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for turn in range(20):
        for i in range(len(shapes)):
            cases[0][i].run(streams[0])
            cases[1][(i + turn) % len(shapes)].run(streams[1])
    torch.cuda.synchronize()
    for c in cases[0] + cases[1]:
        c.check()


def test_binding_refuses():
    c = Case(20, 64, 128)
    ok = (c.weights, c.a, c.sa, c.out, c.ws)
    for i, bad in ((1, c.a[:, :127]), (1, c.a.int()), (1, c.a.cpu()), (2, c.sa[:-1]), (2, c.sa.double()),
                   (3, c.out[:, :63]), (3, c.out.half()), (4, c.ws.int())):
        with pytest.raises(ValueError):
            kvr.kvr_linear(*ok[:i], bad, *ok[i + 1:])
    with pytest.raises(kvr.KvrError):
        kvr.kvr_linear(*ok[:4], c.ws[:128])
    with pytest.raises(ValueError):
        kvr.linear_weights(c.w, c.sw[:-1], c.err)
    odd = torch.zeros(4, 130, dtype=torch.int8, device="cuda")[:, :128]   # rows 130 bytes apart
    w = kvr.linear_weights(odd, torch.ones(4, device="cuda"), c.err)
    assert kvr.kvr_linear_workspace_bytes(w, 4) == 0
    with pytest.raises(kvr.KvrError):
        kvr.kvr_linear(w, c.a[:4], c.sa[:4], torch.empty(4, 4, device="cuda"), c.ws)
