"""A paged cache on the GPU with its plain float64 twin, for the paged tests."""
import numpy as np
import torch

from oracle import paged as OP
from selective_kv_cache_gb300 import kvr

THETA = 500000.0


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Paged:
    """Sequences of the given lengths in shuffled pages; slots nothing was
    written to hold NaN (codes: NaN scales)."""

    def __init__(self, fmt, lens, hkv=2, dh=128, page=16, layout="hnd", group=0, seed=0, spare=2, fill=True,
                 max_pages=None, v_scale=1.0):
        self.fmt, self.lens, self.hkv, self.dh, self.page, self.layout = fmt, list(lens), hkv, dh, page, layout
        self.group = group
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.max_pages = max(max_pages or 1, max(need) if need else 1, 1)
        n_pages = sum(need) + spare
        ids = rng.permutation(n_pages)
        table = np.full((len(lens), self.max_pages), -12345, np.int64)   # never read past a sequence's end
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = ids[at:at + k]
            at += k
        self.table_np = table
        self.table, self.kv_len = i32(table), i32(lens)
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")
        shape = (n_pages, hkv, page) if layout == "hnd" else (n_pages, page, hkv)
        self.ks = self.vs = None
        if fmt == "int4":
            self.k, self.v = (torch.randint(0, 256, shape + (64,), generator=g, device="cuda", dtype=torch.uint8)
                              for _ in range(2))
            self.ks, self.vs = (torch.full(shape + (128 // group, 2), float("nan"), dtype=torch.float16, device="cuda")
                                for _ in range(2))
        else:
            dt = torch.float32 if fmt == "f32" else torch.bfloat16
            self.k, self.v = (torch.full(shape + (dh,), float("nan"), dtype=dt, device="cuda") for _ in range(2))
        self.row_dtype = torch.float32 if fmt == "f32" else torch.bfloat16
        self.p = kvr.pages(fmt, self.k, self.v, self.table, self.kv_len, self.err, hkv, page, layout, self.ks, self.vs,
                           group)
        if fill and sum(lens):
            cu = np.concatenate([[0], np.cumsum(lens)])
            pos = np.concatenate([np.arange(n) for n in lens])
            self.K = torch.randn(len(pos), hkv, dh, generator=g, device="cuda").to(self.row_dtype)
            self.V = (torch.randn(len(pos), hkv, dh, generator=g, device="cuda") * v_scale).to(self.row_dtype)
            kvr.kvr_paged_append(self.p, i32(cu), i32(pos), self.K, self.V)
            kvr.kvr_paged_status(self.p)

    def slots(self, pool, b, n=None):
        """[n, hkv, ...] numpy rows of sequence b's first n positions (raw bytes or elements)."""
        n = self.lens[b] if n is None else n
        x = pool if self.layout == "nhd" else pool.transpose(1, 2)
        g = np.arange(n)
        pg = torch.as_tensor(self.table_np[b, g // self.page], device="cuda")
        x = x[pg, torch.as_tensor(g % self.page, device="cuda")]
        return x.float().cpu().numpy() if x.dtype == torch.bfloat16 else x.cpu().numpy()

    def rows64(self, b, n=None):
        """float64 K, V [hkv, n, dh] of sequence b as held, and the largest |scale * centred code| of V."""
        out = []
        for pool, meta in ((self.k, self.ks), (self.v, self.vs)):
            x = self.slots(pool, b, n)
            if self.fmt == "int4":
                m = self.slots(meta, b, n)
                step = np.repeat(8.0 * m[..., 0].astype(np.float64), self.group, -1)
                x = OP.values(x, m, self.group)
            else:
                x = x.astype(np.float64)
                step = np.abs(x)
            out += [x.transpose(1, 0, 2), np.maximum(step, np.abs(x)).transpose(1, 0, 2)]
        return out[0], out[2], out[3]


def attend_case(c, hq, counts, pos, max_rows=None, seed=7, q_scale=1.5, spare_rows=0, stream=None, workspace=None,
                **opts):
    """Runs kvr_paged_attend on packed rows; returns (out, q, cu)."""
    n = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(n + spare_rows, hq, c.dh, generator=g, device="cuda") * q_scale).to(c.row_dtype)
    out = torch.full((n + spare_rows, hq, c.dh), 7.0, dtype=c.row_dtype, device="cuda")
    cu = i32(np.concatenate([[0], np.cumsum(counts)]))
    p = i32(np.concatenate([pos, np.zeros(spare_rows, np.int64)]))
    m = max_rows or max(max(counts), 1)
    ws = workspace
    if ws is None:
        ws = torch.full((kvr.kvr_paged_workspace_bytes(c.p, hq, n + spare_rows, m),), 255, dtype=torch.uint8,
                        device="cuda")
    kvr.kvr_paged_attend(c.p, kvr.score_opts(**opts) if opts else None, m, cu, p, q, out, ws, stream)
    return out, q, cu


def check_attend(c, hq, counts, pos, out, q, *, begin=None, end=None, scale=None, softcap=0.0, alpha=0.0, beta=0.0,
                 loc=None, snk=None, slopes=None, only=None):
    """out against the float64 definition.

    Bound per element, r = half a step of the row type (bf16 2^-8, fp32
    2^-24), sums over the visible keys' exact weights w:
      r |o|                       the output's rounding;
      r16 sum w a                 the weights' rounding to 16 bits before the
                                  product with V (bf16: 2^-8; none in fp32), a
                                  = |v|, or 8 scales for 4-bit rows, whose
                                  products are with centred codes;
      2 d sum w a                 logits off by d: fp32 accumulation of 128
                                  products, 128 * 2^-24 of sum |q k| scale
                                  (4-bit keys: codes and offset summed apart, 16
                                  times that), the approximate exp2, the cap and
                                  the biases 2^-14 (bf16) or 2^-19 (fp32)."""
    out = out.float().cpu().numpy().astype(np.float64)
    q64 = q.float().cpu().numpy().astype(np.float64)
    row = 0
    for b, n in enumerate(counts):
        rows = slice(row, row + n)
        row += n
        if n == 0 or (only is not None and b not in only):
            continue
        p = np.asarray(pos[rows])
        K, V, step = c.rows64(b)
        lo = np.zeros(n, np.int64) if begin is None else np.asarray(begin[rows])
        hi = p + 1 if end is None else np.asarray(end[rows])
        bias = None
        if loc is not None or snk is not None:
            bias = np.zeros(c.lens[b])
            for m, w in ((loc, alpha), (snk, beta)):
                if m is not None:
                    bias += w * m[b, :c.lens[b]]
        o, spread, noise = OP.attend(q64[rows], K, V, lo, hi, pos=p, scale=scale, softcap=softcap, bias=bias,
                                     slopes=slopes, v_step=step)
        f32 = c.fmt == "f32"
        r = 2.0 ** -24 if f32 else 2.0 ** -8
        d = 128 * 2.0 ** -24 * noise[..., None] * (16 if c.fmt == "int4" else 1) + (2.0 ** -19 if f32 else 2.0 ** -14)
        bound = r * np.abs(o) + ((0 if f32 else r) + 2 * d) * spread + 1e-30
        bad = np.abs(out[rows] - o) > bound
        assert np.isfinite(out[rows]).all() and not bad.any(), (
            f"sequence {b}: {bad.sum()} of {bad.size} off; worst "
            f"{np.max(np.abs(out[rows] - o) / bound):.2f} bounds at {np.argwhere(bad)[:3].tolist()}")
