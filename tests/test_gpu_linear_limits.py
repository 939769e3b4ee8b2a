"""kvr_linear at the ends of its range: a call of more than a second; weights
that the caller fills or copies; sums up to the last that fp32 holds exactly."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")
from test_gpu_linear import Case  # noqa: E402


def test_a_call_of_more_than_a_second():
    """Waits are bounded by a second each, calls are not: 3.4e15 operations take
    the GPU 1.7 s and more.  The status is good and the sums are right."""
    torch.cuda.empty_cache()
    rows, n, k = 400000, 65536, 65536
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.empty(rows, k, dtype=torch.int8, device="cuda").random_(-8, 9, generator=g)
    w = torch.empty(n, k, dtype=torch.int8, device="cuda").random_(-8, 9, generator=g)
    ones = torch.ones(rows, device="cuda")
    W = kvr.linear_weights(w, ones[:n], torch.zeros(4, dtype=torch.int32, device="cuda"))
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kvr.kvr_linear_workspace_bytes(W, rows), dtype=torch.uint8, device="cuda")
    kvr.kvr_linear(W, a, ones, out, ws)
    kvr.kvr_linear_status(W)
    at = torch.tensor([0, 1, 255, 256, 131071, 200000, rows - 257, rows - 1], device="cuda")
    ch = torch.tensor([0, 127, 128, 255, 256, 40000, n - 1], device="cuda")
    want = (a[at].cpu().double() @ w[ch].cpu().double().T).bfloat16()   # sums of 65536 products up to 64: below 2^23, exact
    assert torch.equal(out[at][:, ch].cpu(), want)
    del a, w, out, ws, W
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_weights_filled_by_the_caller_and_copied(rows):
    c = Case(rows, 200, 320, "f32", True, seed=30)
    c.run()
    c.check()
    want, made = c.out.clone(), c.weights
    p = lambda t: t.data_ptr()  # noqa: E731
    filled = kvr.kvr_linear_weights(200, 320, c.w.stride(0), p(c.w), p(c.sw), p(c.bias), p(c.err))
    copied = kvr.kvr_linear_weights.from_buffer_copy(made)
    ctypes.memset(ctypes.addressof(made), 0, ctypes.sizeof(made))
    for w in (filled, copied):
        c.weights = w
        c.out.fill_(0)
        assert kvr.kvr_linear_workspace_bytes(w, rows) == c.ws.numel()
        c.run()
        kvr.kvr_linear_status(w)
        assert torch.equal(c.out, want)


@pytest.mark.parametrize("rows,n_out", [(1, 200), (8, 200), (9, 200), (40, 6000), (64, 200), (64, 25000), (300, 4608), (5000, 200)])
@pytest.mark.parametrize("k,most", [(1040, 127), (1023, -128), (4096, 127), (18944, -127)])
def test_sums_up_to_two_to_the_24(rows, n_out, k, most):
    """Running sums that climb to 2^24 - 3056 (or 2^24 - 16384 of -128 by -128) and
    stay there are exact, of either sign: a step is a multiple of one, and no sum
    on the way is above the last.  Ones in the last places climb to it by one."""
    a, w = torch.zeros(rows, k, dtype=torch.int8), torch.zeros(n_out, k, dtype=torch.int8)
    top = 1040 if abs(most) == 127 else 1023
    a[:, :top], w[:, :top] = most, abs(most) if most != -128 else most
    a[1::2] = -a[1::2].clamp(min=-127)              # odd rows downwards
    w[1::3, top - 2:top] = torch.tensor([1, -1], dtype=torch.int8)   # some channels end on other units
    c = Case(rows, n_out, k, "f32")
    c.a.copy_(a)
    c.w.copy_(w)
    c.sa.fill_(1)
    c.sw.fill_(1)
    c.run()
    kvr.kvr_linear_status(c.weights)
    want = a.double() @ w.double().T
    assert 2 ** 24 - 20000 < want.abs().max() < 2 ** 24
    assert torch.equal(c.out.cpu().double(), want)
