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


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,group,D,page,n_rows,start", [
    (1, 4, 128, 16, [48], [0]),
    (1, 4, 128, 16, [48, 33], [100, 5]),
    (2, 4, 64, 16, [64, 64], [700, 129]),
    (1, 1, 96, 7, [129, 40], [300, 3]),
    (1, 1, 16, 16, [300], [64]),
    (1, 4, 96, 9, [50], [1500]),
    (1, 3, 128, 1000, [70, 1, 0], [130, 2000, 77]),
    (1, 40, 64, 32, [1, 1], [90, 1029]),
])
def test_kv_attend_many_rows_in_wide_tables(dt, fmt, H, group, D, page, n_rows, start):
    """Short and empty contexts, pages that do not divide a tile, blocks of one and of two tiles of rows: tables of 1024
    positions at least, so that the many-row kernel has them. A wider table changes nothing, in no bit."""
    rng = gen(81, H, group, D, page, sum(start))
    cache = widened(Paged(rng, [a + b for a, b in zip(n_rows, start)], H, D, page, fmt), 1024)
    for tree in (None, rng.random((sum(n_rows), max(max(n_rows) - 1, 1))) < 0.3):
        got, ref, q = attend_case(rng, dt, cache, H * group, n_rows, start, tree)
        fl.device_status()
        assert row_blocks(q, cache, n_rows) == (128 if sum(n_rows) * group <= 128 * len(n_rows) else 256)
        attend_check(got, ref, dt, cache, n_rows, start)
        table = widened(cache, 6000).table
        again = fl.kv_attend(q, *cache.tensors(), ints(table), ints(start), cu_rows=ints(sums(n_rows)),
                             tree=None if tree is None else put(tree))
        assert torch.equal(again, got)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [0, 1100])
def test_kv_attend_many_rows_junk_in_places_that_are_not_seen(dt, fmt, D, far):
    """NaN codes and scales in unused places, drafts that hold no number, rows that see nothing, rows behind the last
    sequence, one row of q that is not finite: each stays where it belongs. (The warps' rows choose together how the weights
    are formed, so that beside rows that are not finite the others are compared with the oracle, not in each bit.)"""
    rng = gen(82, D, far)
    n_rows, start = [40, 50], [137 + far, 0]
    cache = widened(Paged(rng, [177 + far, 50], 1, D, 16, fmt), 1024)
    tree = rng.random((95, 50)) < 0.4
    tree[:, 7] = False
    tree[3, 7] = tree[60, 7] = True
    tree[45] = False                                # sees nothing: its context is empty
    q = put(rng.standard_normal((95, 4, D)), dt)
    out = torch.full_like(q, 7.0)
    clean, ref, _ = attend_case(rng, dt, cache, 4, n_rows, start, tree, q=q, out=out)
    clean = clean.clone()
    assert row_blocks(q, cache, n_rows) == 256
    assert (clean[90:] == 7).all() and (clean[45] == 0).all()
    attend_check(clean[:90], ref, dt, cache, n_rows, start)
    used = np.zeros((cache.pages, 16), dtype=bool)
    for b, n in ((0, 177 + far), (1, 50)):
        for p in range(n):
            used[cache.table[b, p // 16], p % 16] = True
    junk = torch.from_numpy(~used).cuda()
    for t in (cache.ks, cache.vs):
        t[junk] = float("nan")
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[junk] = 0x7f            # a NaN in e4m3

    def call():
        r = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(sums(n_rows)), tree=put(tree), out=out)
        fl.device_status()
        assert (r[90:] == 7).all()
        return r
    assert torch.equal(call(), clean)

    def others(got, bad):
        """All rows but `bad` as the oracle has them."""
        keep = [i for i in range(90) if i not in bad]
        attend_check(got[keep], {n: x[keep] for n, x in ref.items()}, dt, cache, n_rows, start)
    # draft 7 of each sequence holds no number: rows 3 and 60 see it, no others
    held = [x.clone() for x in cache.tensors()]
    for b, pos in ((0, 144 + far), (1, 7)):
        page, at = int(cache.table[b, pos // 16]), pos % 16
        for t in (cache.k, cache.v):
            t.view(torch.uint8)[page, at] = 0
        for t in (cache.ks, cache.vs):
            t[page, at] = float("nan")
    got = call()
    assert torch.isnan(got[3]).all() and torch.isnan(got[60]).all()
    others(got, (3, 60))
    for t, x in zip(cache.tensors(), held):
        t.view(torch.uint8).copy_(x.view(torch.uint8))
    # so does a row of q, of itself and one head
    for bad in (float("inf"), float("nan")):
        keep = q[20, 2, 1].clone()
        q[20, 2, 1] = bad
        got = call()
        assert torch.isnan(got[20, 2]).any()
        others(got, (20,))
        heads = [0, 1, 3]
        attend_check(got[20:21, heads], {n: x[20:21, heads] for n, x in ref.items()}, dt, cache, n_rows, start)
        q[20, 2, 1] = keep
    assert torch.equal(call(), clean)
    # pages that are not there
    cache = widened(Paged(rng, [177 + far, 50], 1, D, 16, fmt), 1024)
    cache.table[0, 4] = -1
    cache.table[0, (137 + far) // 16] = 1 << 30
    got, ref, _ = attend_case(rng, dt, cache, 4, n_rows, start)
    with pytest.raises(fl.FusedLinError) as e:
        fl.device_status()
    assert e.value.status == 7
    attend_check(got, ref, dt, cache, n_rows, start)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_kv_attend_many_rows_scales_and_scores_far_apart(dt, D):
    """Values whose scales lie 2^18 apart, scores that grow towards the end so that weights formed with the maxima so far do not
    do, and rows of bf16 far outside fp16's range, over contexts that the many-row kernel has."""
    rng = gen(83, D)
    n, n_rows, start = 60, [60], [1300]
    cache = Paged(rng, [1360], 1, D, 16, "int8")
    assert cache.table.shape[1] * 16 >= 1024
    cache.scale[1] = np.where(rng.random(cache.scale[1].shape) < 0.5, 2.0 ** -6, 2.0 ** -24).astype(np.float32)
    pos = np.zeros((cache.pages, 16))
    for p in range(1360):
        pos[cache.table[0, p // 16], p % 16] = p
    for grow in (1.003, 1.0):
        cache.scale[0] = (0.002 * grow ** pos)[..., None].astype(np.float32)
        cache.ks, cache.vs = put(cache.scale[0]), put(cache.scale[1])
        for size in ((2.0 ** -50, 1.0, 2.0 ** 40) if dt == "bf16" else (2.0 ** -4, 2.0 ** 4)):
            q = put(rng.standard_normal((n, 1, D)) * size * np.exp2(rng.integers(-6, 6, (n, 1, 1))), dt)
            scale = 0.08 / size
            got, ref, _ = attend_case(rng, dt, cache, 1, n_rows, start, q=q, scale=scale)
            fl.device_status()
            assert row_blocks(q, cache, n_rows) == 128
            vals = cache.values()[0]
            floor = np.zeros((n, 1))
            for i in range(n):
                x = vals[0][:1301 + i, 0] @ f64(q)[i, 0] * scale
                w = np.exp(x - x.max())
                vs = cache.scale[1][cache.table[0][:85]].reshape(-1)[:len(w)]
                floor[i, 0] = len(w) * 2.0 ** -25 * 127 * (w / w.sum() * vs).max()
            check(got, ref, U[dt], 2.0 ** -11, 2.0 ** -18, floor, f"{grow} {size}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,start", [(64, 9000), (128, 12100)])
def test_kv_attend_many_rows_of_more_pieces_than_a_warp_has_lanes(dt, fmt, D, start):
    """One row block over 71 and 95 tiles is split into pieces of two: 36 and 48 to be joined."""
    rng = gen(84, D)
    cache = Paged(rng, [start + 48], 1, D, 64, fmt)
    got, ref, q = attend_case(rng, dt, cache, 4, [48], [start])
    fl.device_status()
    assert row_blocks(q, cache, [48]) == 256
    attend_check(got, ref, dt, cache, [48], [start])
    for _ in range(3):
        again = fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints([start]), cu_rows=ints([0, 48]))
        assert torch.equal(again, got)


# ---------------------------------------------------------------------------
# few rows of a sequence over the cache
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,group,D,n_rows", [(1, 4, 128, [1, 1]), (8, 1, 64, [16, 5]), (2, 3, 256, [5, 1])])
def test_kv_attend_tables_around_the_shortest_that_may_be_split(dt, fmt, H, group, D, n_rows):
    """512 positions, filled to the last, need no workspace; one page more does."""
    for pages in (32, 33):
        rng = gen(85, H, D, pages)
        start = [16 * pages - n_rows[0], 16 * pages - 20]
        cache = Paged(rng, [a + b for a, b in zip(n_rows, start)], H, D, 16, fmt)
        cache.table = cache.table[:, :pages]
        got, ref, q = attend_case(rng, dt, cache, H * group, n_rows, start)
        fl.device_status()
        need = fl.kv_attend_workspace_size(q, cache.k, ints(cache.table), ints(sums(n_rows)))
        assert (need == 0) == (pages == 32)
        attend_check(got, ref, dt, cache, n_rows, start)
        # the same pages in a wide table: the same plan of the same lengths, the same bits
        wide = widened(cache, 4096).table
        again = fl.kv_attend(q, *cache.tensors(), ints(wide), ints(start), cu_rows=ints(sums(n_rows)))
        fl.device_status()
        if sum(n_rows) * group <= 32 * len(n_rows):
            assert torch.equal(again, got)
        attend_check(again, ref, dt, cache, n_rows, start)


# ---------------------------------------------------------------------------
# attention over 16-bit keys and values
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk,is_causal", [([200, 150, 20], [60, 0, 3], True), ([5, 3], [0, 4], False), ([300, 1], [1, 700], True)])
def test_attention_rows_with_keys_beside_rows_without(dt, D, lq, lk, is_causal):
    got, ref, (*_, floor) = attention_case(dt, 2, 1, D, lq, lk, is_causal, 86)
    check(got, ref, U[dt], U[dt], 2.0 ** -20, floor)
    sees = ref["top"] > 0
    assert (f64(got)[~sees] == 0).all() and not sees.all()


def test_attention_keys_for_longer_than_a_wait_may_take():
    """The values of the last block are mended once it is there, however long the blocks in front of it take."""
    rng = gen(87)
    n, hq, D, m = 256, 80, 64, 1000003
    q = put(rng.standard_normal((n, hq, D)), "bf16")
    g = torch.Generator(device="cuda")
    g.manual_seed(87)
    k, v = (torch.randn(m, 1, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    torch.cuda.synchronize()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    fl.set_option("timeout_ms", 2)
    try:
        a.record()
        got = fl.attention(q, k, v, causal=False)
        b.record()
        fl.device_status()
    finally:
        fl.set_option("timeout_ms", 2000)
    assert a.elapsed_time(b) > 4
    rows, heads = [0, 131, 255], [0, 41, 79]
    ref = {x: np.zeros((3, 3, D)) for x in ("out", "mag", "sq")}
    ref["size"] = np.zeros((3, 3))
    kd, vd = k[:, 0].double(), v[:, 0].double()
    for i, r in enumerate(rows):
        for j, h in enumerate(heads):
            x = q[r, h].double()
            w = torch.softmax(kd @ x / 8, 0)
            for name, val in (("out", w @ vd), ("mag", w @ vd.abs()), ("sq", w ** 2 @ vd ** 2)):
                ref[name][i, j] = val.cpu().numpy()
            ref["size"][i, j] = float((kd.abs() @ x.abs()).max()) / 8 / np.log(2.0)
    check(got[rows][:, heads], ref, U["bf16"], U["bf16"], 2.0 ** -20, np.zeros((3, 3)))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m", [(700, 700), (40, 3000)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_values_that_are_not_finite(dt, D, n, m, bad):
    """A value that is not finite, early enough that blocks are seen as a whole: its channel is not finite in the rows that see it
    (an infinity where their weight is not 0, else NaN), and nothing else changes."""
    rng = gen(91, D, n)
    q, k, v = (put(rng.standard_normal((x, h, D)), dt) for x, h in ((n, 2), (m, 1), (m, 1)))
    clean = fl.attention(q, k, v)
    at = m - n + 10
    v[at, 0, 3] = bad
    got = fl.attention(q, k, v)
    fl.device_status()
    rest = [c for c in range(D) if c != 3]
    assert torch.equal(got[:10], clean[:10]) and torch.equal(got[..., rest], clean[..., rest])
    hit = got[10:, :, 3]
    assert (torch.isnan(hit) | (hit == bad)).all()
    if bad != bad:
        assert torch.isnan(hit).all()
    k[at] = 40 * q[10, 0]                               # all the weight that fp32 has, in row 10
    got = fl.attention(q, k, v)
    fl.device_status()
    assert torch.isnan(got[10, 0, 3]) if bad != bad else got[10, 0, 3] == bad


# ---------------------------------------------------------------------------
# scores of any size
# ---------------------------------------------------------------------------
SIZES = [2.0 ** 12, 2.0 ** 20, 2.0 ** 24, 2.0 ** 27, 2.0 ** 31, 2.0 ** 62, 2.0 ** 99]


def winners(q, k, sees, scale):
    """The key with the largest score of each row of q [n, D] over k [m, D], and whether it is certain to have all the weight: in
    front of the next by 2^60 in weight and by more than the scores are off by."""
    x = np.where(sees, q @ k.T, -np.inf)
    size = (np.abs(q) @ np.abs(k).T * sees).max(1)
    two = np.sort(np.concatenate((np.full((len(x), 1), -np.inf), x), 1), 1)[:, -2:]
    with np.errstate(invalid="ignore"):
        gap = two[:, 1] - two[:, 0]
    return x.argmax(1), sees.any(1) & (gap * scale > 42) & (gap > 2.0 ** -18 * size)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m", [(300, 300), (5, 3000)])
@pytest.mark.parametrize("scale", SIZES)
def test_attention_scores_of_any_size(dt, D, n, m, scale):
    """A row whose largest score stands alone gets its key's value. Its weight is 2^r, r the rounding of a score of 2^20 at most (larger
    ones are differences of rounded products, r = 0); rounded to the dtype, divided by itself and multiplied, then rounded
    once more: 2 u and some 2^-23 together."""
    rng = gen(88, D, n)
    q, k, v = (put(rng.standard_normal((x, h, D)), dt) for x, h in ((n, 2), (m, 1), (m, 1)))
    got = f64(fl.attention(q, k, v, scale=scale))
    fl.device_status()
    assert np.isfinite(got).all()
    for h in range(2):
        best, sure = winners(f64(q)[:, h], f64(k)[:, 0], oracle.causal(n, m), scale)
        assert sure.mean() > 0.9
        y = f64(v)[best[sure], 0]
        assert (np.abs(got[sure, h] - y) <= (2 * U[dt] + 2.0 ** -20) * np.abs(y) + 2.0 ** -25 * (dt == "f16")).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group,D,n_rows,start", [(4, 64, [1, 3], [700, 90]), (4, 128, [1, 3], [2900, 90]), (1, 256, [9], [300]),
                                                  (4, 128, [6], [1000]), (4, 64, [48], [1200]), (2, 128, [48], [2700])])
@pytest.mark.parametrize("far", [False, True])
def test_kv_attend_scores_of_any_size(dt, fmt, group, D, n_rows, start, far):
    """The same over the cache, with values of one size and of sizes that lie 2^44 apart: the weight times the value's scale and the output
    are rounded (the scale's logarithm, 2^-19 of it, is one more term)."""
    rng = gen(89, D, sum(start))
    cache = Paged(rng, [a + b for a, b in zip(n_rows, start)], 1, D, 16, fmt)
    if far:
        cache.scale[1] = np.where(rng.random(cache.scale[1].shape) < 0.5, 2.0 ** -6, 2.0 ** -50).astype(np.float32)
        cache.vs = put(cache.scale[1])
    q = put(rng.standard_normal((sum(n_rows), group, D)), dt)
    cu = sums(n_rows)
    vals = cache.values()
    certain = []
    for scale in SIZES:
        got = f64(fl.kv_attend(q, *cache.tensors(), ints(cache.table), ints(start), cu_rows=ints(cu), scale=scale))
        fl.device_status()
        assert np.isfinite(got).all()
        for b, (n, at) in enumerate(zip(n_rows, start)):
            for h in range(group):
                best, sure = winners(f64(q)[cu[b]:cu[b + 1], h], vals[b][0][:at + n, 0], oracle.causal(n, at + n), scale)
                certain.append(sure.mean())
                y = vals[b][1][best[sure], 0]
                err = np.abs(got[cu[b]:cu[b + 1], h][sure] - y)
                # (the others' weights together are below (at + n) 2^-60)
                rest = (at + n) * 2.0 ** -60 * np.abs(vals[b][1]).max() + 2.0 ** -25 * (dt == "f16")
                assert (err <= (U[dt] + 2.0 ** -11 + 2.0 ** -16) * np.abs(y) + rest).all(), (scale, b, h)
    assert np.mean(certain) > 0.5


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def forks_that_are_not_defined(rng, B, kind):
    if kind == "child twice":
        children = rng.integers(B // 2, B, 40)
        parents = rng.integers(0, B // 2 - 2, 40)
    else:                                              # some sequences are children and parents
        children = rng.permutation(np.arange(2, B - 2))[:40]
        parents = rng.integers(0, B - 2, 40)
    return parents, children


@pytest.mark.parametrize("kind", ["child twice", "child and parent"])
@pytest.mark.parametrize("B,per", [(60, 9), (80, 300)])
def test_kv_fork_of_one_sequence_twice_leaves_the_others_alone(kind, B, per):
    """What such a child then holds is not defined. Every other sequence keeps its pages and what they hold, and no page is
    counted less than it is held."""
    for seed in range(4):
        rng = gen(90, B, per, seed)
        lens = rng.integers(0, 16 * per + 1, B).tolist()
        cache = Paged(rng, lens, 1, 64, 16, "int8", spare=90)
        cache.table = cache.table[:, :per]
        shared = np.flatnonzero(np.asarray(lens) >= 32)[-1]
        cache.table[B - 1] = -1
        cache.table[B - 1, :2] = cache.table[shared, :2]  # pages that two sequences hold
        refs = np.bincount(cache.table[cache.table >= 0], minlength=cache.pages).astype(np.int32)
        parents, children = forks_that_are_not_defined(rng, B, kind)
        lengths = [int(rng.integers(0, lens[p] + 1)) for p in parents]
        t, r = ints(cache.table), ints(refs)
        before = [x.clone() for x in cache.tensors()]
        fl.kv_fork(*cache.tensors(), t, r, ints(parents), ints(children), ints(lengths))
        try:
            fl.device_status()
        except fl.FusedLinError as e:
            assert e.status == 7
        table, counts = t.cpu().numpy(), r.cpu().numpy()
        others = np.setdiff1d(np.arange(B), children)
        assert np.array_equal(table[others], cache.table[others])
        assert ((table >= -1) & (table < cache.pages)).all()
        held = np.bincount(table[table >= 0], minlength=cache.pages)
        assert (counts >= held).all()
        pages = np.unique(cache.table[others])
        pages = torch.from_numpy(pages[pages >= 0]).long().cuda()
        for x, y in zip(cache.tensors(), before):
            x, y = (z if z.dtype == torch.float32 else z.view(torch.uint8) for z in (x, y))
            assert torch.equal(x[pages], y[pages])
