"""The table's gradient at every border of the sorted list's chunks: runs of
equal ids of every length at every offset within a chunk, for each of the chunk
lengths that the sizes choose, and runs on both sides of the number of partial
rows from which a run is added up by more than one wave."""

import numpy as np
import pytest
import torch

from test_gpu_embed import check_grad
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu

H = 8  # one eight of columns: the chunk length depends on the tokens alone
SHORT_PARTS = 32  # a run of more partial rows is a long one
# the fewest and the most tokens of each chunk length: the longest of which the
# list has 2,048 chunks (up to 1,024 tokens need no list)
SPANS = {4: (1025, 16383), 8: (16384, 32767), 16: (32768, 65535), 32: (65536, 1 << 30)}


def workspace_of(n, C):
    """The workspace's bytes for chunks of C entries: four lists, a byte a chunk,
    two partial rows of 8 floats a chunk."""
    def up(x):
        return (x + 255) // 256 * 256

    chunks = -(-n // C)
    return 4 * up(4 * n) + up(chunks) + chunks * 2 * 8 * 4


def sorted_list(C, runs, last=()):
    """The sorted ids of `runs`, (offset in a chunk, length) each, single ids
    between them to reach the offsets; then single ids up to the fewest tokens
    of the chunk length, and `last`, a run that ends the list."""
    out, v = [], 0

    def single(count):
        nonlocal v
        out.extend(range(v, v + count))
        v += count

    for off, length in list(runs) + list(last):
        if last and (off, length) == last[0] and len(out) < SPANS[C][0]:
            single(SPANS[C][0] - len(out))
        single((off - len(out)) % C)
        out.extend([v] * length)
        v += 1
    if len(out) < SPANS[C][0]:
        single(SPANS[C][0] - len(out))
    return np.array(out, dtype=np.int32), v


def check(C, runs, dtype, accumulate, last=()):
    ids, V = sorted_list(C, runs, last)
    n = len(ids)
    assert SPANS[C][0] <= n <= SPANS[C][1]
    assert B.mdlm_embed_grad_workspace_bytes(n, H) == workspace_of(n, C)
    at = np.flatnonzero(np.diff(ids, prepend=-1))  # where each run begins
    length = np.diff(at, append=n)
    assert set(runs) <= set(zip(at % C, length))
    np.random.default_rng(n).shuffle(ids)
    check_grad(ids, n, H, V + 1, dtype, accumulate, 1.0, n)


@pytest.mark.parametrize("C", SPANS)
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.bfloat16, True)])
def test_every_run_at_every_offset(C, dtype, accumulate):
    """Lengths up to two chunks and a bit: runs within a chunk, across one
    border, ending on one, and cut into partial rows."""
    runs = [(off, length) for length in range(2, 2 * C + 7) for off in range(C)]
    if C == 4:  # (and up to 18 chunks)
        runs += [(off, length) for length in range(15, 71) for off in range(C)]
    check(C, runs, dtype, accumulate)


@pytest.mark.parametrize("C", SPANS)
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, True), (torch.bfloat16, False)])
def test_runs_of_about_the_long_ones_length(C, dtype, accumulate):
    """Runs of 31 to 34 partial rows, the last row full or of one token, at
    every offset."""
    runs = [(off, parts * C - off + more) for off in range(C)
            for parts in range(SHORT_PARTS - 1, SHORT_PARTS + 2) for more in (0, 1)]
    half = runs if C < 16 else runs[::2]  # (the tokens of one chunk length)
    check(C, half, dtype, accumulate)
    if C >= 16:
        check(C, runs[1::2], dtype, accumulate)


@pytest.mark.parametrize("C", SPANS)
def test_a_run_that_ends_the_list(C):
    """The last run of the list: within the last chunk, cut short of it, of 32
    and of 33 partial rows."""
    for off in (0, 1, C - 1):
        for length in (1, C - off, C + 1, 2 * C - off, 2 * C - off + 1, SHORT_PARTS * C - off,
                       SHORT_PARTS * C - off + 1, (SHORT_PARTS + 9) * C + 1):
            check(C, [], torch.float32, bool(off), [(off, length)])
