"""Which blocks of the batch projection (csrc/linear_few.cu) meet on an SM, by
the library's own sizes (CPU only).

An allocation of tensor memory waits without a limit until its columns are free.
A block holds its columns until its whole cluster is done, so two clusters that
each hold what the other's second block waits for would wait for ever: blocks
that fit an SM's shared memory together have to fit its columns too, whatever
their register count allows."""
import ctypes
import itertools

import pytest

kvr = pytest.importorskip("selective_kv_cache_gb300.kvr")

SM_BYTES, RESERVED, SM_COLUMNS = 228 * 1024, 1024, 512
BLOCK_MOST = 227 * 1024
COLUMNS = {2: 256, 4: 512}


def shape(sets, n):
    f = kvr.lib._ZN3kvr15linear_few_smemEiiPi   # kvr::linear_few_smem(int, int, int*)
    f.argtypes, f.restype = [ctypes.c_int, ctypes.c_int, ctypes.c_void_p], ctypes.c_int
    stages = ctypes.c_int()
    return f(sets, n, ctypes.addressof(stages)), stages.value


BLOCKS = [(sets, n) for sets in COLUMNS for n in (16, 32, 48, 64)]


def test_blocks_that_meet_have_their_columns():
    for count in (2, 3, 4):
        for group in itertools.combinations_with_replacement(BLOCKS, count):
            if sum(shape(*b)[0] + RESERVED for b in group) <= SM_BYTES:
                assert sum(COLUMNS[sets] for sets, _ in group) <= SM_COLUMNS, group


@pytest.mark.parametrize("sets,n", BLOCKS)
def test_a_block_holds_its_ring(sets, n):
    """Alignment, ring, widened rows of every set, barriers; stages a multiple of
    the sets; the ring has room for two tiles of sums where clusters share tiles."""
    size, stages = shape(sets, n)
    assert stages >= sets and stages % sets == 0
    barriers = 8 * (2 * stages + 2 * sets + 1) + 8
    assert 1024 + stages * (128 * 128 + 128 * n) + 2 * sets * 128 * n + barriers <= size <= BLOCK_MOST
    assert stages * (128 * 128 + 128 * n) >= (2 if sets == 4 else 1) * n * 128 * 4
