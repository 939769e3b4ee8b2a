"""kvr_linear_weights in the binding is plain data: filled by the caller, or a
copy that outlives its original (CPU only: sizes of the workspace)."""
import ctypes

import pytest

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")
P = 1 << 20   # an aligned address; nothing is read


def filled(n_out=4096, k=1000):
    return kvr.kvr_linear_weights(n_out, k, -(-k // 16) * 16, P, P, None, P)


def test_filled_weights():
    w = filled()
    for n in (1, 64, 65, 500):
        want = kvr.lib.kvr_linear_workspace_bytes(ctypes.addressof(w), n)
        assert want >= 256 and kvr.kvr_linear_workspace_bytes(w, n) == want


def test_copied_weights_do_not_read_their_original():
    first, other = filled(), filled(k=2000)
    first.tensors, first.device = (), 0   # as linear_weights leaves them
    copied = kvr.kvr_linear_weights.from_buffer_copy(first)
    want = kvr.kvr_linear_workspace_bytes(first, 500)
    ctypes.memset(ctypes.addressof(first), 0, ctypes.sizeof(first))
    assert kvr.kvr_linear_workspace_bytes(copied, 500) == want != kvr.kvr_linear_workspace_bytes(other, 500)
