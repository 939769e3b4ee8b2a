"""The packed-row operators as a program uses them: decode steps of a decoder
layer over the paged cache with weights in eight bits, each operator against
its definition in float64 on the inputs that it got, eager and captured; keys
moved between positions; tables for the paged append; sizes past 2^31 bytes."""
import numpy as np
import pytest
import torch

from oracle import rows as OR

pytestmark = pytest.mark.gpu

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")
from paged_case import Paged, check_attend, i32  # noqa: E402
from test_gpu_rows import check_codes, check_rotated, check_values, f64  # noqa: E402

D, HQ, HK, DH, F = 512, 4, 2, 128, 1408
EPS = 1e-5


def weights(n, k, seed, bias=False):
    """A matrix of N(0, 1/sqrt k) in eight bits, by the library's own quantiser."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(n, k, generator=g, device="cuda") / k ** 0.5
    codes, scale = torch.empty(n, k, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    kvr.kvr_rows_quantise(w, codes, scale)
    check_codes(codes, scale, f64(w), 0.0)
    b = torch.randn(n, generator=g, device="cuda") * 0.1 if bias else None
    return kvr.linear_weights(codes, scale, torch.zeros(4, dtype=torch.int32, device="cuda"), b)


class Layer:
    """One decoder layer's decode step over `lens` sequences, a row each."""

    def __init__(self, lens, layout="half", rot=DH):
        n = self.n = len(lens)
        self.c = Paged("bf16", lens, HK, DH, 16, "nhd", seed=2, spare=3 * n, max_pages=max(lens) // 16 + 3)
        for b, m in enumerate(lens):   # pages for the rows to come
            need = -(-m // 16)
            spare = [p for p in range(self.c.k.shape[0]) if p not in set(self.c.table_np[self.c.table_np >= 0].tolist())]
            self.c.table_np[b, need:need + 2] = spare[:2]
        self.c.table.copy_(i32(self.c.table_np))
        self.rope = kvr.rope(DH, rot, layout=layout, theta=10000.0, scaling="bands", factor=4.0, low=1.0, high=4.0,
                             original_len=256)
        self.layout = layout
        self.qkv, self.o, self.gate_up, self.down = (weights((HQ + 2 * HK) * DH, D, 1, True), weights(D, HQ * DH, 2),
                                                     weights(2 * F, D, 3), weights(D, F, 4))
        t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.w1, self.w2 = t(D) + 1.1, t(D) + 0.9
        self.x = torch.randn(n, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).bfloat16()
        self.codes, self.scale = t(n, F, dt=torch.int8), t(n, dt=torch.float32)
        self.h, self.att, self.y, self.z = t(n, HQ + 2 * HK, DH), t(n, HQ, DH), t(n, D), t(n, D)
        self.gu = t(n, 2 * F)
        self.pos, self.cu = i32(lens), i32(np.arange(n + 1))
        self.key_len = self.c.kv_len
        self.linear_ws = torch.empty(max(kvr.kvr_linear_workspace_bytes(w, n) for w in
                                         (self.qkv, self.o, self.gate_up, self.down)), dtype=torch.uint8, device="cuda")
        self.attend_ws = torch.empty(kvr.kvr_paged_workspace_bytes(self.c.p, HQ, n, 1), dtype=torch.uint8, device="cuda")
        self.seen = None

    def note(self, name, *tensors):
        if self.seen is not None:
            self.seen[name] = [t.clone() for t in tensors]

    def step(self):
        n, cd = self.n, self.codes[:, :D]
        self.note("x", self.x)
        kvr.kvr_rows_norm(self.x, self.w1, EPS, codes=cd, scales=self.scale)
        self.note("norm1", cd, self.scale)
        kvr.kvr_linear(self.qkv, cd, self.scale, self.h.view(n, -1), self.linear_ws)
        self.note("qkv", self.h)
        q, k, v = self.h[:, :HQ], self.h[:, HQ:HQ + HK], self.h[:, HQ + HK:]
        kvr.kvr_rows_rotate(self.rope, self.pos, q, q, k, k)
        self.note("turned", self.h)
        kvr.kvr_paged_append(self.c.p, self.cu, self.pos, k, v)
        self.key_len += 1
        kvr.kvr_paged_attend(self.c.p, None, 1, self.cu, self.pos, q, self.att, self.attend_ws)
        self.note("att", self.att)
        cd = self.codes[:, :HQ * DH]
        kvr.kvr_rows_quantise(self.att.view(n, -1), cd, self.scale)
        kvr.kvr_linear(self.o, cd, self.scale, self.y, self.linear_ws)
        self.note("o", cd, self.scale, self.y)
        kvr.kvr_rows_norm(self.x, self.w2, EPS, residual=self.y, sum_out=self.x, codes=self.codes[:, :D], scales=self.scale)
        self.note("norm2", self.x, self.codes[:, :D], self.scale)
        kvr.kvr_linear(self.gate_up, self.codes[:, :D], self.scale, self.gu, self.linear_ws)
        self.note("gu", self.gu)
        kvr.kvr_rows_swiglu(self.gu, codes=self.codes, scales=self.scale)
        self.note("gated", self.codes, self.scale)
        kvr.kvr_linear(self.down, self.codes, self.scale, self.z, self.linear_ws)
        self.x += self.z
        self.pos += 1
        self.note("z", self.z)

    def check_linear(self, w, codes, scale, out):
        want = OR.linear(codes.cpu().numpy(), f64(scale), w.tensors[0].cpu().numpy(), f64(w.tensors[1]),
                         None if w.tensors[2] is None else f64(w.tensors[2]))
        bias = 0 if w.tensors[2] is None else np.abs(f64(w.tensors[2]))
        # sums below 2^24 are exact; conversion, two products and the bias' addition round in fp32, the output in bf16
        assert np.all(np.abs(f64(out) - want) <= (2.0 ** -8 + 2.0 ** -21) * np.abs(want) + 2.0 ** -21 * bias + 1e-30)

    def check(self, lens):
        """Every operator of the last step, from the inputs it got."""
        s = self.seen
        check_codes(*s["norm1"], OR.norm(f64(s["x"][0]), f64(self.w1), EPS)[1], 2.0 ** -18)
        self.check_linear(self.qkv, *s["norm1"], s["qkv"][0].view(self.n, -1))
        before, after = s["qkv"][0], s["turned"][0]
        check_rotated(after[:, :HQ + HK], before[:, :HQ + HK], lens, self.rope, self.layout, "bf16")
        assert torch.equal(after[:, HQ + HK:], before[:, HQ + HK:])
        self.c.lens = [m + 1 for m in lens]
        check_attend(self.c, HQ, [1] * self.n, np.asarray(lens), s["att"][0], after[:, :HQ])
        check_codes(*s["o"][:2], f64(s["att"][0].view(self.n, -1)), 0.0)
        self.check_linear(self.o, *s["o"])
        h, y = OR.norm(f64(s["x"][0]), f64(self.w2), EPS, f64(s["o"][2]))
        check_values(s["norm2"][0], h, "bf16", 2.0 ** -24)
        check_codes(*s["norm2"][1:], y, 2.0 ** -18)
        self.check_linear(self.gate_up, *s["norm2"][1:], s["gu"][0])
        check_codes(*s["gated"], OR.swiglu(f64(s["gu"][0])), 2.0 ** -17)
        self.check_linear(self.down, *s["gated"], s["z"][0])
        for w in (self.qkv, self.o, self.gate_up, self.down):
            kvr.kvr_linear_status(w)
        kvr.kvr_paged_status(self.c.p)


@pytest.mark.parametrize("lens", [[100], [37, 5, 64, 130, 16, 1], list(range(20, 40))])
@pytest.mark.parametrize("layout,rot", [("half", DH), ("interleaved", 64)])
def test_decode_steps(lens, layout, rot):
    """Three eager steps, then a fourth that is captured and replayed: two
    replays give what two eager steps of a twin give, bit for bit."""
    a, b = Layer(lens, layout, rot), Layer(lens, layout, rot)
    for t in range(3):
        a.seen = {}
        a.step()
        torch.cuda.synchronize()
        a.check([m + t for m in lens])
        a.seen = None
        b.step()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.step()
    for _ in range(2):
        graph.replay()
        b.step()
    torch.cuda.synchronize()
    assert torch.equal(a.x, b.x) and torch.equal(a.z, b.z) and torch.equal(a.pos, b.pos)


def test_moved_keys():
    """Keys read out of the pages, turned by the distance that their block
    moves and appended there, against the rows turned once at the new
    positions: two roundings to bf16 more, of rows of the same length."""
    n, move = 40, -23
    r = kvr.rope(DH, theta=500000.0)
    c = Paged("bf16", [64, 64], HK, DH, 16, seed=3)
    cu, old = i32([0, n, n]), i32(np.arange(n) + 24)
    raw = torch.randn(n, HK, DH, device="cuda").bfloat16()
    k, v = torch.empty_like(raw), torch.randn_like(raw)
    kvr.kvr_rows_rotate(r, old, k=raw, k_out=k)
    kvr.kvr_paged_append(c.p, cu, old, k, v)
    got_k, got_v = torch.empty_like(raw), torch.empty_like(raw)
    kvr.kvr_paged_read(c.p, cu, old, got_k, got_v)
    kvr.kvr_rows_rotate(r, i32(np.full(n, move)), k=got_k, k_out=got_k)
    kvr.kvr_paged_append(c.p, i32([0, 0, n]), i32(np.arange(n) + 24 + move), got_k, got_v)
    kvr.kvr_paged_status(c.p)
    want = OR.rotate(f64(raw), (np.arange(n) + 24 + move).tolist(), list(r.turns[:64]))
    K, V, _ = c.rows64(1)
    pair = np.hypot(f64(raw)[..., :64], f64(raw)[..., 64:])
    bound = (3 * 2.0 ** -8 + 2.0 ** -18) * np.concatenate([pair, pair], -1)
    assert np.all(np.abs(K[:, 1:1 + n].transpose(1, 0, 2) - want) <= bound)
    np.testing.assert_array_equal(V[:, 1:1 + n].transpose(1, 0, 2), f64(v))


@pytest.mark.parametrize("scaling,more", [("plain", {}), ("bands", dict(factor=8.0, low=1.0, high=4.0, original_len=512)),
                                          ("yarn", dict(factor=4.0, low=1.0, high=32.0, original_len=512))])
def test_scaled_table_in_the_paged_append(scaling, more):
    """Rows turned by kvr_paged_append with the library's table, and by
    kvr_rows_rotate before it: the same pages, bit for bit."""
    n = 90
    r = kvr.rope(DH, theta=500000.0, scaling=scaling, **more)
    table = torch.empty(128, DH // 2, 2, device="cuda")
    kvr.kvr_rope_table(r, 128, table)
    a, b = (Paged("bf16", [100], HK, DH, 32, seed=5) for _ in range(2))
    cu, pos = i32([0, n]), i32(np.arange(n) + 5)
    q, k, v = (torch.randn(n, h, DH, device="cuda").bfloat16() for h in (HQ, HK, HK))
    qa, qb, kb = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    kvr.kvr_paged_append(a.p, cu, pos, k, v, table, q, qa)
    kvr.kvr_rows_rotate(r, pos, q, qb, k, kb)
    kvr.kvr_paged_append(b.p, cu, pos, kb, v)
    kvr.kvr_paged_status(a.p)
    kvr.kvr_paged_status(b.p)
    assert torch.equal(qa, qb)
    for x, y in zip(a.rows64(0, 95)[:2], b.rows64(0, 95)[:2]):
        np.testing.assert_array_equal(x, y)


def test_boundary_states_in_eight_bits():
    """Stored boundary states read back feed a refresh: kvr_reselect takes the
    dequantised rows where it took the stored ones."""
    from selective_kv_cache_gb300 import workloads as wl
    from selective_kv_cache_gb300.harness import Setup
    m = wl.ModelShape(1, 512, 8, 2, 128, 1024, 500000.0, 1e-5, "bf16", True, vocab=1000)
    s = Setup(wl.Workload("boundary", 7, m, 1, 320, 300, 100, 48, selection="isolated"))
    s.select()
    rows = s.positions[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    state = torch.randn(1, 320, 512, generator=g, device="cuda").bfloat16()
    codes, scale = torch.empty(320, 512, dtype=torch.int8, device="cuda"), torch.empty(320, device="cuda")
    kvr.kvr_rows_quantise(state[0], codes, scale)
    fill = torch.empty_like(state)
    kvr.kvr_rows_dequantise(codes, scale, fill[0])
    wide = np.arange(100, 300, dtype=np.int32)
    out = torch.empty(200, 512, dtype=torch.bfloat16, device="cuda")
    kvr.kvr_reselect(s.handle, wide, np.array([200], np.int32), s.hidden, fill, out)
    torch.cuda.synchronize()
    new = [i for i, p in enumerate(wide) if p not in set(np.asarray(rows).tolist())]
    assert torch.equal(out[new], fill[0][torch.as_tensor(wide[new].astype(np.int64), device="cuda")])
    step = f64(scale)[wide[new]][:, None]
    assert np.all(np.abs(f64(out[new]) - f64(state[0])[wide[new]]) <= (0.5 + 2.0 ** -14) * step + 2.0 ** -8 * 128 * step)
    s.close()


# ---------------------------------------------------------------- offsets past 31 and 32 bits
def test_rows_past_four_gigabytes():
    n, d = 1050000, 2056   # 4.3 GB in bf16, 2.2 GB of codes
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 522000, 1044400, 1044401, n - 1]
    x[at] = torch.randn(len(at), d, device="cuda").bfloat16()
    first = x[at].clone()
    codes, scale = torch.full((n, d), 3, dtype=torch.int8, device="cuda"), torch.full((n,), 9.0, device="cuda")
    kvr.kvr_rows_quantise(x, codes, scale)
    check_codes(codes[at], scale[at], f64(x[at]), 0.0)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert float(scale[keep].abs().amax()) == 0 and int(torch.count_nonzero(codes[n - 1000:n - 1])) == 0
    out = torch.empty_like(x)
    kvr.kvr_rows_dequantise(codes, scale, out)
    assert torch.equal(out[at], (codes[at].float() * scale[at][:, None]).bfloat16()) and \
        int(torch.count_nonzero(out[n - 1000:n - 1])) == 0
    kvr.kvr_rows_norm(x, torch.ones(d, dtype=torch.bfloat16, device="cuda"), EPS, residual=x, sum_out=x, codes=codes,
                      scales=scale)
    check_codes(codes[at], scale[at], OR.norm(f64(x[at]), 1.0, EPS)[1], 2.0 ** -17)
    heads = x.view(n, 257, 8)   # twice the rows by now
    r = kvr.rope(8)
    kvr.kvr_rows_rotate(r, torch.full((n,), 5, dtype=torch.int32, device="cuda"), heads, heads)
    want = OR.rotate(2 * f64(first).reshape(len(at), 257, 8), [5] * len(at), list(r.turns[:4]))
    pair = np.hypot(want[..., :4], want[..., 4:])
    assert np.all(np.abs(f64(heads[at]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.concatenate([pair, pair], -1))


@pytest.mark.parametrize("rows", [3, 20, 100])
def test_weights_past_four_gigabytes(rows):
    n, k = 1 << 20, 4112   # 4.3 GB of codes
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(n, k, dtype=torch.int8, device="cuda")
    w.random_(-100, 100, generator=g)
    a = torch.randint(-100, 100, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    ones = torch.ones(n, device="cuda")
    W = kvr.linear_weights(w, ones, torch.zeros(4, dtype=torch.int32, device="cuda"))
    out = torch.empty(rows, n, device="cuda")
    ws = torch.empty(kvr.kvr_linear_workspace_bytes(W, rows), dtype=torch.uint8, device="cuda")
    kvr.kvr_linear(W, a, ones[:rows], out, ws)
    kvr.kvr_linear_status(W)
    at = torch.cat([torch.arange(0, 300), torch.arange(522000, 522600), torch.arange(n - 300, n)]).cuda()
    want = a.cpu().double() @ w[at].cpu().double().T
    assert torch.equal(out[:, at].cpu().double(), want)   # below 2^24: exact


@pytest.mark.parametrize("rows", [70000])
def test_outputs_past_four_gigabytes(rows):
    n, k = 32000, 64   # 4.5 GB of bf16
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(-3, 4, (n, k), generator=g, device="cuda", dtype=torch.int8)
    a = torch.randint(-3, 4, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    ones = torch.ones(rows, device="cuda")
    W = kvr.linear_weights(w, ones[:n], torch.zeros(4, dtype=torch.int32, device="cuda"))
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kvr.kvr_linear_workspace_bytes(W, rows), dtype=torch.uint8, device="cuda")
    kvr.kvr_linear(W, a, ones, out, ws)
    kvr.kvr_linear_status(W)
    at = torch.cat([torch.arange(0, 100), torch.arange(67000, 67300), torch.arange(rows - 100, rows)]).cuda()
    want = (a[at].cpu().double() @ w.cpu().double().T).bfloat16()   # sums below 577: two roundings are one
    assert torch.equal(out[at].cpu(), want)
