"""Attention and the cache's page keeping without a GPU: refusals of the C ABI and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

import gemm_epilogue_tma_gb300 as fl
import oracle
from gemm_epilogue_tma_gb300 import _build

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE, CUDA, TIMEOUT, RANGE = range(8)
BASE = 0x7F0000000000
PASSES = (UNSUPPORTED,)  # validation passed: the device query fails on this machine


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fl.lib()


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a device")


def addr(i, off=0):
    return BASE + i * (1 << 36) + off


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def passed(L, status):
    return status in PASSES and b"no CUDA device" in L.fl_last_error()


@no_gpu
def test_attention_refusals(L):
    good = dict(dtype=0, rows_q=300, rows_k=400, heads_q=8, heads_k=2, head_dim=64, n_seqs=3, causal=1, scale=0.125,
                cu_q=addr(4), cu_k=addr(5), q=addr(0), k=addr(1), v=addr(2), out=addr(3), q_row=512, q_head=64, k_row=128,
                k_head=64, v_row=128, v_head=64, out_row=512, out_head=64)

    def call(**kw):
        return L.fl_attention(ctypes.byref(fl.AttentionDesc(**{**good, **kw})), None)
    assert passed(L, call()) and passed(L, call(causal=0)) and passed(L, call(cu_q=None, cu_k=None, n_seqs=1))
    assert passed(L, call(rows_k=0, k=None, v=None))
    assert L.fl_attention(None, None) == INVALID
    assert call(rows_q=0, q=None, out=None) == OK
    assert call(dtype=2) == INVALID
    for n in ("rows_q", "rows_k", "heads_q", "heads_k", "head_dim", "n_seqs"):
        assert call(**{n: -1}) == INVALID
    for n in ("heads_q", "heads_k", "head_dim", "n_seqs"):
        assert call(**{n: 0}) == INVALID
    assert call(heads_q=7) == INVALID and call(heads_k=3) == INVALID
    assert call(head_dim=60) == ALIGN and call(head_dim=136) == UNSUPPORTED
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == INVALID
    assert call(cu_q=None) == INVALID and call(cu_k=None) == INVALID and call(cu_q=None, cu_k=None) == INVALID
    assert call(cu_q=addr(4, 2)) == ALIGN and call(cu_k=addr(5, 1)) == ALIGN
    for n, i in (("q", 0), ("k", 1), ("v", 2), ("out", 3)):
        assert call(**{n: None}) == INVALID and call(**{n: addr(i, 8)}) == ALIGN
    for n in ("q_row", "k_row", "v_head", "out_row", "out_head"):
        assert call(**{n: 132}) == ALIGN and call(**{n: -64}) == INVALID
    assert call(out_head=56) == INVALID and call(out_row=504) == INVALID
    assert call(k_head=0) == UNSUPPORTED and "expanded" in fl.last_error()
    assert call(v_row=0) == UNSUPPORTED and call(q_row=1 << 40) == UNSUPPORTED
    for n, i in (("q", 0), ("k", 1), ("v", 2), ("cu_q", 4), ("cu_k", 5)):
        assert call(out=addr(i)) == INVALID and "overlaps" in fl.last_error()
        assert call(**{n: addr(3, 512)}) == INVALID
    # out beside q, k and v in one matrix
    wide = dict(q_row=2048, k_row=2048, v_row=2048, out_row=2048)
    assert passed(L, call(**wide, k=addr(0, 1024), v=addr(0, 1280), out=addr(0, 2048)))
    assert call(**wide, k=addr(0, 1024), v=addr(0, 1280), out=addr(0, 1408)) == INVALID
    assert call(rows_q=1 << 30, n_seqs=1 << 30, heads_q=128, heads_k=1) == UNSUPPORTED and "too many rows" in fl.last_error()
    assert call(n_seqs=(1 << 30) + 1) == UNSUPPORTED


ATTEND = dict(dtype=0, format=0, rows=6, heads_q=8, heads_k=2, head_dim=64, page_size=16, n_pages=100, n_seqs=3,
              table_pages=40, tree_cols=5, scale=0.125, table_stride=40, tree_stride=5, page_table=addr(2), cu_rows=addr(3),
              start=addr(4), tree=addr(5), q=addr(0), out=addr(1), q_row=512, q_head=64, out_row=512, out_head=64,
              k_cache=addr(6), v_cache=addr(7), k_scale=addr(8), v_scale=addr(9))


def attend_desc(**kw):
    return fl.KvAttendDesc(**{**ATTEND, **kw})


@no_gpu
def test_kv_attend_refusals(L):
    def call(ws=addr(10), size=1 << 30, **kw):
        return L.fl_kv_attend(ctypes.byref(attend_desc(**kw)), ws, size, None)
    assert passed(L, call()) and passed(L, call(tree=None, cu_rows=None)) and passed(L, call(format=1, head_dim=256, q_row=2048,
                                                                                             q_head=256, out_row=2048, out_head=256))
    assert L.fl_kv_attend(None, None, 0, None) == INVALID
    assert call(rows=0, q=None, out=None) == OK
    assert call(dtype=2) == INVALID and call(format=2) == INVALID
    for n in ("heads_q", "heads_k", "head_dim", "page_size", "n_pages", "n_seqs", "table_pages"):
        assert call(**{n: 0}) == INVALID
    assert call(rows=-1) == INVALID and call(heads_q=7) == INVALID
    assert call(head_dim=60) == ALIGN and call(head_dim=264) == UNSUPPORTED
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == INVALID
    assert call(table_stride=39) == INVALID and call(table_stride=-40) == INVALID and passed(L, call(n_seqs=1, table_stride=0))
    assert call(tree_stride=4) == INVALID and call(tree_cols=-1) == INVALID and passed(L, call(tree=None, tree_cols=9))
    for n, i in (("q", 0), ("out", 1), ("k_cache", 6), ("v_cache", 7), ("k_scale", 8), ("v_scale", 9)):
        assert call(**{n: None}) == INVALID and call(**{n: addr(i, 8)}) == ALIGN
    for n, i in (("page_table", 2), ("start", 4)):
        assert call(**{n: None}) == INVALID and call(**{n: addr(i, 2)}) == ALIGN
    assert call(cu_rows=addr(3, 2)) == ALIGN
    assert call(q_row=508) == ALIGN and call(out_head=-64) == INVALID and call(out_row=504) == INVALID
    for i in range(2, 10):
        assert call(out=addr(i)) == INVALID and call(ws=addr(i)) == INVALID
    assert call(out=addr(0)) == INVALID and call(ws=addr(1)) == INVALID and call(ws=addr(0)) == INVALID
    need = L.fl_kv_attend_workspace_size(ctypes.byref(attend_desc()))
    assert 0 < need <= 11 << 20
    assert call(ws=None) == WORKSPACE and call(size=need - 1) == WORKSPACE and call(ws=addr(10, 8)) == ALIGN
    # contexts of 256 positions at most are never split
    short = dict(table_pages=16, table_stride=16)
    assert L.fl_kv_attend_workspace_size(ctypes.byref(attend_desc(**short))) == 0 and passed(L, call(ws=None, size=0, **short))
    assert L.fl_kv_attend_workspace_size(ctypes.byref(attend_desc(head_dim=60))) == 0
    assert L.fl_kv_attend_workspace_size(None) == 0
    assert call(rows=(1 << 31) - 1) == UNSUPPORTED and call(n_seqs=(1 << 30) + 1) == UNSUPPORTED


PAGES = dict(heads=2, head_dim=64, page_size=16, n_pages=100, n_seqs=3, table_pages=40, table_stride=40, page_table=addr(0),
             k_cache=addr(1), v_cache=addr(2), k_scale=addr(3), v_scale=addr(4))
SIZES = ("page_size", "n_pages", "n_seqs", "table_pages")


def check_pages(L, call, cache):
    for n in SIZES:
        assert call(**{n: 0}) == INVALID
    assert call(table_stride=39) == INVALID and call(page_table=None) == INVALID and call(page_table=addr(0, 2)) == ALIGN
    assert call(n_seqs=(1 << 30) + 1) == UNSUPPORTED
    if not cache:
        return
    assert call(heads=0) == INVALID and call(head_dim=0) == INVALID and call(head_dim=60) == ALIGN and call(head_dim=264) == UNSUPPORTED
    assert call(heads=1 << 21) == UNSUPPORTED
    for i, n in enumerate(("k_cache", "v_cache", "k_scale", "v_scale")):
        assert call(**{n: None}) == INVALID and call(**{n: addr(1 + i, 8)}) == ALIGN
        assert call(**{n: addr(0)}) == INVALID


@no_gpu
def test_kv_resize_refusals(L):
    def call(refs=addr(5), lengths=addr(6), ws=addr(7), size=1 << 20, **kw):
        d = fl.KvPages(**{**PAGES, "heads": 0, "head_dim": 0, "k_cache": None, "v_cache": None, "k_scale": None,
                          "v_scale": None, **kw})
        return L.fl_kv_resize(ctypes.byref(d), refs, lengths, ws, size, None)
    assert passed(L, call())
    assert L.fl_kv_resize(None, addr(5), addr(6), addr(7), 1 << 20, None) == INVALID
    check_pages(L, call, False)
    assert call(refs=None) == INVALID and call(lengths=None) == INVALID and call(refs=addr(5, 2)) == ALIGN
    assert L.fl_kv_pages_workspace_size(100) == 400 and L.fl_kv_pages_workspace_size(0) == 0
    assert call(ws=None) == WORKSPACE and call(size=399) == WORKSPACE and call(ws=addr(7, 4)) == ALIGN
    assert call(refs=addr(0)) == INVALID and call(lengths=addr(5)) == INVALID and call(ws=addr(6)) == INVALID
    assert call(ws=addr(0)) == INVALID


@no_gpu
def test_kv_fork_refusals(L):
    def call(refs=addr(5), parents=addr(6), children=addr(7), lengths=addr(8), n=4, ws=addr(9), size=1 << 20, **kw):
        return L.fl_kv_fork(ctypes.byref(fl.KvPages(**{**PAGES, **kw})), refs, parents, children, lengths, n, ws, size, None)
    assert passed(L, call()) and call(n=0) == OK and call(n=-1) == INVALID
    assert L.fl_kv_fork(None, addr(5), addr(6), addr(7), addr(8), 4, addr(9), 1 << 20, None) == INVALID
    check_pages(L, call, True)
    for n, i in (("refs", 5), ("parents", 6), ("children", 7), ("lengths", 8)):
        assert call(**{n: None}) == INVALID and call(**{n: addr(i, 1)}) == ALIGN
        assert call(**{n: addr(0)}) == INVALID and call(**{n: addr(9)}) == INVALID and call(**{n: addr(1)}) == INVALID
    assert passed(L, call(parents=addr(8)))          # inputs may be one tensor
    assert call(ws=None) == WORKSPACE and call(size=399) == WORKSPACE


@no_gpu
def test_kv_compact_refusals(L):
    def call(start=addr(5), accepted=addr(6), most=4, **kw):
        return L.fl_kv_compact(ctypes.byref(fl.KvPages(**{**PAGES, **kw})), start, accepted, most, None)
    assert passed(L, call()) and call(most=0) == OK and call(most=-1) == INVALID
    assert L.fl_kv_compact(None, addr(5), addr(6), 4, None) == INVALID
    check_pages(L, call, True)
    assert call(start=None) == INVALID and call(accepted=None) == INVALID and call(start=addr(5, 2)) == ALIGN
    assert call(start=addr(1)) == INVALID and call(accepted=addr(4)) == INVALID


def test_binding_refuses_tensors_that_do_not_fit():
    """The checks of the Python binding that need no GPU."""
    t = torch.zeros((4, 2, 64), dtype=torch.float16)
    if torch.cuda.is_available():
        with pytest.raises(ValueError):
            fl.attention(t, t, t)
    fl.ops()
    for call in (lambda: fl.ops().attention(1, 2), lambda: fl.ops().kv_attend(t), lambda: fl.ops().kv_resize()):
        with pytest.raises(TypeError):
            call()


# ---------------------------------------------------------------------------
# pins of the oracle
# ---------------------------------------------------------------------------
def test_oracle_attention_is_softmax():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((n, h, 16)) for n, h in ((7, 4), (9, 2), (9, 2)))
    got = oracle.attention(q, k, v, [0, 3, 7], [0, 5, 9], True, 0.25)["out"]
    tq, tk, tv = (torch.from_numpy(x) for x in (q, k, v))
    for b, (i, j, m, n) in enumerate(((0, 3, 0, 5), (3, 7, 5, 9))):
        for h in range(4):
            x = tq[i:j, h] @ tk[m:n, h // 2].T * 0.25
            x.masked_fill_(~torch.ones(j - i, n - m, dtype=torch.bool).tril(n - m - (j - i)), -np.inf)
            assert np.allclose(got[i:j, h], (torch.softmax(x, 1) @ tv[m:n, h // 2]).numpy(), rtol=1e-13, atol=1e-14)
    # one key: its value; none: zeros; equal keys: the mean
    one = oracle.attention(q[:1], k[:1], v[:1], [0, 1], [0, 1], True, 3.0)["out"]
    assert np.allclose(one[0, 3], v[0, 1])
    assert (oracle.attention(q[:3], k[:1], v[:1], [0, 3], [0, 1], True, 1.0)["out"][:2] == 0).all()
    same = oracle.attention(q[:1], np.ones((5, 2, 16)), v[:5], [0, 1], [0, 5], False, 1.0)["out"]
    assert np.allclose(same[0, 0], v[:5, 0].mean(0))


def test_oracle_tree_of_a_chain_is_causal():
    rng = np.random.default_rng(2)
    q = rng.standard_normal((4, 2, 8))
    k, v = (rng.standard_normal((12, 1, 8)) for _ in "kv")
    there = np.ones(12, dtype=bool)
    a = oracle.kv_attend(q, [k], [v], [there], [0, 4], [8], None, 1.0)["out"]
    b = oracle.kv_attend(q, [k], [v], [there], [0, 4], [8], np.tril(np.ones((4, 4), dtype=bool)), 1.0)["out"]
    c = oracle.attention(q, k, v, [0, 4], [0, 12], True, 1.0)["out"]
    assert np.array_equal(a, b) and np.allclose(a, c)
    # a branch: row 2 does not see draft 1
    tree = np.tril(np.ones((4, 4), dtype=bool))
    tree[2, 1] = False
    d = oracle.kv_attend(q, [k], [v], [there], [0, 4], [8], tree, 1.0)["out"]
    keep = [p for p in range(11) if p != 9]
    e = oracle.attention(q[2:3], k[keep], v[keep], [0, 1], [0, 10], False, 1.0)["out"]
    assert np.allclose(d[2], e[0]) and np.array_equal(d[[0, 1, 3]], a[[0, 1, 3]])


def test_oracle_pages_by_hand():
    table = np.array([[4, 2, -1], [0, -1, -1], [-1, -1, -1]])
    refs = np.array([1, 0, 1, 0, 1, 0])
    # sequence 0 keeps page 4 and gives 2 back; sequence 1 keeps 0 and takes 1 and 2; sequence 2 takes 3
    t, r, fine = oracle.kv_resize(table, refs, [5, 25, 1], 10)
    assert fine and t.tolist() == [[4, -1, -1], [0, 1, 2], [3, -1, -1]] and r.tolist() == [1, 1, 1, 1, 1, 0]
    t, r, fine = oracle.kv_resize(t, r, [30, 25, 31], 10)
    assert not fine and t.tolist() == [[4, 5, -1], [0, 1, 2], [3, -1, -1]] and r.tolist() == [1, 1, 1, 1, 1, 1]
    t, r, copies, fine = oracle.kv_fork(np.array([[4, 2, -1], [0, -1, -1], [-1, -1, -1]]), refs, [0, 0], [1, 2], [17, 20], 10)
    assert fine and t.tolist() == [[4, 2, -1], [4, 0, -1], [4, 2, -1]] and r.tolist() == [1, 0, 2, 0, 3, 0] and copies == [(2, 0, 7)]
    moves, fine = oracle.kv_compact(np.array([[3, 1]]), 6, [8], [[0, 2, 5, -1, 9]], 10)
    assert fine and moves == [((1, 0), (3, 9)), ((1, 3), (1, 0))]


def test_oracle_mistakes_are_seen():
    """Planted mistakes change the answers that the tests compare with."""
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((n, h, 8)) for n, h in ((6, 4), (9, 2), (9, 2)))
    good = oracle.attention(q, k, v, [0, 6], [0, 9], True, 0.35)["out"]
    assert not np.allclose(good, oracle.attention(q, k, v, [0, 6], [0, 9], False, 0.35)["out"])
    assert not np.allclose(good, oracle.attention(q, k[:, ::-1], v[:, ::-1], [0, 6], [0, 9], True, 0.35)["out"])
    assert not np.allclose(good, oracle.attention(q, k, v, [0, 6], [0, 9], True, 0.36)["out"])
    assert not np.allclose(good, oracle.attention(q, k[:6], v[:6], [0, 6], [0, 6], True, 0.35)["out"])


@no_gpu
def test_kv_attend_sizes_next_to_32_bits(L):
    """Row blocks of up to 256 rows are counted in 32 bits on the GPU: rows times heads of a group up to 2^31 - 513."""
    def call(rows, **kw):
        kw = {**dict(n_seqs=1, table_stride=40, tree=None, heads_q=1, heads_k=1, head_dim=16, q_row=16, q_head=16, out_row=16,
                     out_head=16, q=1 << 40, out=1 << 41, page_size=64), **kw}
        return L.fl_kv_attend(ctypes.byref(attend_desc(rows=rows, **kw)), addr(10), 1 << 30, None)
    for kw in ({}, dict(page_size=8), dict(head_dim=256, q_row=256, q_head=256, out_row=256, out_head=256)):
        assert passed(L, call((1 << 31) - 513, **kw))
        for less in (512, 300, 255, 65, 64, 1):
            assert call((1 << 31) - less, **kw) == UNSUPPORTED and "too many rows" in fl.last_error()
    four = dict(heads_q=4, q_row=64, out_row=64)
    assert passed(L, call((1 << 29) - 129, **four)) and call((1 << 29) - 128, **four) == UNSUPPORTED
    assert "too many rows" in fl.last_error()


def test_kv_attend_workspace_of_the_shortest_table_that_may_be_split(L):
    """Up to 512 positions a sequence is never split (the GPU's plan goes by its lengths alone) and no workspace is needed."""
    for size, pages in ((16, 32), (1, 512), (512, 1), (19, 26), (300, 1)):
        for kw in ({}, dict(head_dim=256), dict(rows=300, n_seqs=1), dict(cu_rows=None), dict(head_dim=24)):
            need = [L.fl_kv_attend_workspace_size(ctypes.byref(attend_desc(page_size=size, table_pages=n, table_stride=n, **kw)))
                    for n in (pages, 512 // size + 1)]
            assert need[0] == 0 and 0 < need[1] <= 42 << 20
