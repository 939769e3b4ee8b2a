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
