"""Edges of attention over prompts and over the paged cache on the GPU, against the float64 oracle (needs an sm_103a GPU).

Bounds are those of tests/test_gpu_attention.py.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_tma_gb300 as fl
import oracle
from test_gpu_attention import (FMT, U, Paged, attend_case, attend_check, attention_case, check, f64, gen, ints,  # noqa: F401
                                library, put, sums)  # (library: the fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# many rows of a sequence over the cache
# ---------------------------------------------------------------------------
def widened(cache, positions):
    """The same pages in a table of `positions` positions at least."""
    more = -(-positions // cache.page) - cache.table.shape[1]
    if more > 0:
        cache.table = np.concatenate((cache.table, np.full((len(cache.table), more), -1, dtype=np.int32)), 1)
    return cache


def row_blocks(q, cache, n_rows):
    """Rows of a row block, 128 or 256, if the call is the many-row kernel's, else 0: by its workspace, sums and statistics of 304
    pieces of so many rows (the other kernel has 608 of 32 at most) and a record of 9760 bytes."""
    need = fl.kv_attend_workspace_size(q, cache.k, ints(cache.table), ints(sums(n_rows)))
    width = 64 if cache.D <= 64 else 128
    return {304 * m * (width + 4) * 4 + 9760: m for m in (128, 256)}.get(need, 0)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,group,D,page,n_rows,start", [
    (1, 4, 128, 16, [48], [2600]),
    (2, 1, 64, 8, [100, 40], [1900, 1100]),
    (1, 2, 96, 30, [64], [1500]),
])
def test_kv_attend_many_rows_gaps_that_differ_from_block_to_block(dt, fmt, H, group, D, page, n_rows, start):
    """Every block of 128 positions lacks other pages than the blocks before it; scales of missing places are not read."""
    rng = gen(80, H, group, D, page)
    cache = Paged(rng, [a + b for a, b in zip(n_rows, start)], H, D, page, fmt)
    gone = rng.random(cache.table.shape) < rng.choice([0.0, 0.2, 0.7], cache.table.shape)
    cache.table[gone] = np.where(rng.random(gone.sum()) < 0.5, -1, cache.pages + 5)
    unused = torch.ones(cache.pages, dtype=torch.bool)
    unused[torch.from_numpy(cache.table[(cache.table >= 0) & (cache.table < cache.pages)]).long()] = False
    for t in (cache.ks, cache.vs):
        t[unused.cuda()] = float("nan")
    for tree in (None, rng.random((sum(n_rows), max(n_rows))) < 0.4):
        got, ref, q = attend_case(rng, dt, cache, H * group, n_rows, start, tree)
        assert row_blocks(q, cache, n_rows) > 0
        with pytest.raises(fl.FusedLinError) as e:
            fl.device_status()
        assert e.value.status == 7
        attend_check(got, ref, dt, cache, n_rows, start)
        again = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)),
                             tree=None if tree is None else put(tree))
        with pytest.raises(fl.FusedLinError):
            fl.device_status()
        assert torch.equal(again, got)
