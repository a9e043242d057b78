"""Cases of attention over prompts and over the paged 8-bit cache, and of the keeping of the cache's pages.

attention    a prompt's rows over 16-bit k and v: grouped heads, packed sequences, causal or not
kv_attend    new tokens, one or a tree of drafted ones per sequence, over the cache's codes
kv_compact   the rows of accepted drafts moved to the end of their contexts
kv_fork      sequences that share another's full pages, with a copy of its last one
kv_resize    page tables brought to new lengths: pages given back, pages taken

Sizes are those of the library's own workloads (32 and 8 heads of 128 channels, pages of 16 and 64 positions, 61
sequences, 60001 cached positions) and ragged ones around them.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CACHES = {"int8": (torch.int8, 127.0), "fp8": (torch.float8_e4m3fn, 448.0)}


def listed():
    return [
        # the smallest call: a short question to a small model
        {"name": "attention bf16 1x37 h8 d64", "op": "attention", "dtype": "bf16", "seqs": 1, "rows": 37, "context": 0,
         "hq": 8, "hkv": 8, "D": 64, "causal": True, "pad": 0},
        # a step of chunked prompts: parts of five prompts behind what the cache holds of them already
        {"name": "attention f16 5 chunks", "op": "attention", "dtype": "f16", "seqs": 5, "rows": 2051, "context": 1500,
         "hq": 32, "hkv": 8, "D": 128, "causal": True, "pad": 13},
        # one long prompt
        {"name": "attention bf16 1x8192", "op": "attention", "dtype": "bf16", "seqs": 1, "rows": 8192, "context": 0,
         "hq": 32, "hkv": 8, "D": 128, "causal": True, "pad": 0},
        # a decode step of many short conversations
        {"name": "kv_attend int8 bf16 61x1", "op": "kv_attend", "dtype": "bf16", "cache": "int8", "seqs": 61, "rows": 61,
         "total": 9150, "hq": 32, "hkv": 8, "D": 128, "page": 16, "tree": False, "pad": 0},
        # a decode step of a batch of long contexts
        {"name": "kv_attend fp8 f16 16 long", "op": "kv_attend", "dtype": "f16", "cache": "fp8", "seqs": 16, "rows": 16,
         "total": 60001, "hq": 32, "hkv": 8, "D": 128, "page": 64, "tree": False, "pad": 0},
        # four sequences, each with a tree of drafted tokens to be verified
        {"name": "kv_attend int8 bf16 4 trees", "op": "kv_attend", "dtype": "bf16", "cache": "int8", "seqs": 4, "rows": 4 * 48,
         "total": 23003, "hq": 32, "hkv": 8, "D": 128, "page": 16, "tree": True, "pad": 0},
        # the accepted tokens of one tree
        {"name": "kv_compact int8 1x4 of 48", "op": "kv_compact", "cache": "int8", "seqs": 1, "drafts": 48, "most": 4,
         "context": 700, "H": 8, "D": 128, "page": 16},
        # those of a large batch of deep trees
        {"name": "kv_compact fp8 61x16 of 64", "op": "kv_compact", "cache": "fp8", "seqs": 61, "drafts": 64, "most": 16,
         "context": 700, "H": 8, "D": 128, "page": 64},
        # three more answers to one short prompt
        {"name": "kv_fork fp8 1 to 3", "op": "kv_fork", "cache": "fp8", "parents": 1, "each": 3, "length": 150, "H": 8,
         "D": 128, "page": 16},
        # eight prompts, seven more answers to each
        {"name": "kv_fork int8 8 to 56", "op": "kv_fork", "cache": "int8", "parents": 8, "each": 7, "length": 3001, "H": 8,
         "D": 128, "page": 64},
        # a step of speculative decoding: room for the drafts, then back to what was accepted
        {"name": "kv_resize 7 drafts", "op": "kv_resize", "seqs": 7, "most": 16, "page": 16, "spare": 30, "turnover": False},
        # a large server: sequences that have ended give their pages back, new prompts take theirs
        {"name": "kv_resize 256 turnover", "op": "kv_resize", "seqs": 256, "most": 1024, "page": 16, "spare": 9001,
         "turnover": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "kv_attend", "kv_attend", "kv_compact", "kv_fork", "kv_resize"])
    c = {"op": op}
    if op in ("attention", "kv_attend"):
        c["dtype"] = rng.choice(["f16", "bf16"])
        c["D"] = rng.choice([64, 80, 96, 128])
        c["hkv"] = rng.choice([1, 2, 5, 8])
        c["hq"] = c["hkv"] * rng.choice([1, 3, 4])
        c["pad"] = rng.choice([0, 0, 5])
    if op == "attention":
        c["rows"] = _log(rng, 1, 4500)
        c["seqs"] = min(c["rows"], _log(rng, 1, 40))
        c["causal"] = rng.random() < 0.7
        c["context"] = rng.choice([0, _log(rng, 1, 1 + 4000 // c["seqs"])])
    elif op == "kv_attend":
        c["cache"] = rng.choice(["int8", "fp8"])
        c["seqs"] = _log(rng, 1, 64)
        c["tree"] = rng.random() < 0.5
        c["rows"] = c["seqs"] * (_log(rng, 2, 64) if c["tree"] and c["seqs"] < 9 else 1)
        c["total"] = c["rows"] + _log(rng, 64, 20000)
        c["page"] = rng.choice([16, 32, 64])
    elif op == "kv_compact":
        c["cache"] = rng.choice(["int8", "fp8"])
        c["seqs"] = _log(rng, 1, 61)
        c["drafts"] = _log(rng, 4, 64)
        c["most"] = rng.randint(1, max(1, c["drafts"] // 4))
        c["context"] = _log(rng, 1, 1000)
        c["H"] = rng.choice([1, 2, 5, 8])
        c["D"] = rng.choice([64, 80, 128])
        c["page"] = rng.choice([16, 32, 64])
    elif op == "kv_fork":
        c["cache"] = rng.choice(["int8", "fp8"])
        c["parents"] = _log(rng, 1, 8)
        c["each"] = rng.randint(1, 7)
        c["length"] = _log(rng, 1, 3000)
        c["H"] = rng.choice([1, 2, 5, 8])
        c["D"] = rng.choice([64, 80, 128])
        c["page"] = rng.choice([16, 32, 64])
    else:
        c["seqs"] = _log(rng, 3, 256)
        c["most"] = _log(rng, 8, 1024)
        c["page"] = rng.choice([16, 32, 64])
        c["spare"] = _log(rng, 30, 9001)
        c["turnover"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# inputs: lengths go by the case alone, values by the seed
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _spread(seqs, rows, least=1):
    """`rows` rows over `seqs` sequences, unevenly, `least` for each at least."""
    r = random.Random(1000003 * seqs + rows)
    w = [r.random() + 0.05 for _ in range(seqs)]
    n = [least + int(x / sum(w) * (rows - least * seqs)) for x in w]
    n[0] += rows - sum(n)
    return n


def _sums(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def _lengths(c):
    """Of an attention case: rows of q and of k of each sequence."""
    lq = _spread(c["seqs"], c["rows"])
    r = random.Random(c["context"] + 7 * c["rows"])
    return lq, [n + (r.randint(0, 2 * c["context"]) if c["context"] else 0) for n in lq]


def _contexts(c):
    """Of a kv_attend case: positions of each sequence in front of its new rows."""
    each = c["rows"] // c["seqs"]
    return [n - each for n in _spread(c["seqs"], max(c["total"], c["rows"]), each)]


def _tables(g, need, per, spare):
    """A pool of pages in random order over sequences that hold `need` pages each; a row ends with -1."""
    first = _sums(need)
    order = torch.randperm(first[-1] + spare, generator=g, device="cuda")
    j = torch.arange(per, device="cuda")
    n = torch.tensor(need, device="cuda")[:, None]
    at = torch.tensor(first[:-1], device="cuda")[:, None] + j
    table = order[at.clamp(max=order.shape[0] - 1)]
    return torch.where(j < n, table, -1).to(torch.int32), order.shape[0]


def _cache(g, s, pages, page, H, D, cache):
    code, top = CACHES[cache]
    shape = (pages, page, H, D)
    for n in "kv":
        s[n + "_cache"] = (_randn(g, *shape) * top / 4).clamp_(-top, top).to(code)
        # (a head's row of unit variance has its largest value near 2.7)
        s[n + "_scale"] = (0.8 + 0.4 * torch.rand(shape[:3], generator=g, device="cuda")) * 4.0 / top


def _tree(drafts, seqs):
    """Whether a drafted row sees another of its sequence: itself and its ancestors, parents being drawn in front."""
    r = random.Random(drafts)
    sees = [[False] * drafts for _ in range(drafts)]
    for i in range(drafts):
        if i:
            sees[i] = list(sees[r.randint(max(0, i // 4 - 1), i - 1 if r.random() < 0.3 else i // 3)])
        sees[i][i] = True
    return torch.tensor(sees * seqs, device="cuda")


def _accepted(c):
    """Drafts that were accepted, in order, -1 behind them: the root, then a path through rows that lie behind the places
    they move to, so that the same pass can be made again."""
    r = random.Random(c["drafts"] + 77 * c["seqs"])
    rows = []
    for b in range(c["seqs"]):
        n = r.randint(1, c["most"]) if b else c["most"]
        path = [0] + sorted(r.sample(range(n, c["drafts"]), n - 1))
        rows.append(path + [-1] * (c["most"] - n))
    return rows


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op = c["op"]
    s = {"case": c}
    if op == "attention":
        dt, hq, hkv, D, T = DTYPES[c["dtype"]], c["hq"], c["hkv"], c["D"], c["rows"] + c["pad"]
        lq, lk = _lengths(c)
        if c["context"]:  # k and v as they were read back from a cache
            s["q"] = _randn(g, T, hq, D).to(dt)
            s["k"], s["v"] = (_randn(g, sum(lk), hkv, D).to(dt) for _ in "kv")
        else:  # as the stacked projection leaves them, side by side in one row
            qkv = _randn(g, T, (hq + 2 * hkv) * D).to(dt)
            s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
            s["k"] = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
            s["v"] = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        s["cu_q"], s["cu_k"] = _ints(_sums(lq)), _ints(_sums(lk))
        s["out"] = torch.zeros(T, hq, D, dtype=dt, device="cuda")
    elif op == "kv_attend":
        dt, B, page = DTYPES[c["dtype"]], c["seqs"], c["page"]
        each, ctx = c["rows"] // B, _contexts(c)
        need = [-(-(n + each) // page) for n in ctx]
        s["page_table"], pages = _tables(g, need, max(need) + 1, 3)
        _cache(g, s, pages, page, c["hkv"], c["D"], c["cache"])
        s["q"] = _randn(g, c["rows"] + c["pad"], c["hq"], c["D"]).to(dt)
        s["start"], s["cu_rows"] = _ints(ctx), _ints([each * b for b in range(B + 1)])
        s["tree"] = _tree(each, B) if c["tree"] else None
        if c["tree"] and c["pad"]:
            s["tree"] = torch.cat((s["tree"], s["tree"][:1].expand(c["pad"], -1)))
        s["out"] = torch.zeros_like(s["q"])
    elif op == "kv_compact":
        r = random.Random(c["context"])
        start = [r.randint(0, 2 * c["context"]) for _ in range(c["seqs"])]
        need = [-(-(n + c["drafts"]) // c["page"]) for n in start]
        s["page_table"], pages = _tables(g, need, max(need), 2)
        _cache(g, s, pages, c["page"], c["H"], c["D"], c["cache"])
        s["start"], s["accepted"] = _ints(start), _ints(_accepted(c))
    elif op == "kv_fork":
        P, E, page = c["parents"], c["each"], c["page"]
        lens = _spread(P, c["length"] * P)
        need = [-(-n // page) for n in lens] + [0] * (P * E)
        table, pages = _tables(g, need, max(need) + 1, P * E + 5)
        s["page_table"] = table
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        s["refs"][table[table >= 0].long()] = 1
        _cache(g, s, pages, page, c["H"], c["D"], c["cache"])
        s["parents"] = _ints([p for p in range(P) for _ in range(E)])
        s["children"] = _ints(list(range(P, P + P * E)))
        s["lengths"] = _ints([n for n in lens for _ in range(E)])
    else:
        B, most, page = c["seqs"], c["most"], c["page"]
        before, first, second = _turns(c)
        s["page_table"], pages = _tables(g, [-(-n // page) for n in before], most, c["spare"])
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        s["refs"][s["page_table"][s["page_table"] >= 0].long()] = 1
        s["first"], s["second"] = _ints(first), _ints(second)
    return s


def _turns(c):
    """Of a kv_resize case: each sequence's length before, after the first call and after the second."""
    r = random.Random(c["seqs"] + 13 * c["most"])
    cap = c["most"] * c["page"]
    if c["turnover"]:
        before = [r.randint(cap // 4, cap) if b % 4 < 3 else 0 for b in range(c["seqs"])]
        first = [0 if b % 3 == 1 else n for b, n in enumerate(before)]
        second = [(before[(b + 1) % c["seqs"]] + 1) // 2 if n == 0 else n for b, n in enumerate(first)]
    else:
        before = [r.randint(cap // 4, cap - 64) for _ in range(c["seqs"])]
        first = [min(cap, n + 48) for n in before]
        second = [min(cap, n + 1 + b % 5) for b, n in enumerate(before)]
    return before, first, second


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _values(s, n, page, at):
    """Rows of a cache in 32 bits. (By bytes: not every torch version indexes 8-bit floats.)"""
    code = s[n + "_cache"].view(torch.uint8)[page, at].view(s[n + "_cache"].dtype).float()
    return code * s[n + "_scale"][page, at][..., None]


def _plain_softmax(x, sees):
    x = torch.where(sees, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    return w / torch.where(total == 0.0, 1.0, total)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import gemm_epilogue_tma_gb300 as fl
        if op == "attention":
            return fl.attention(s["q"], s["k"], s["v"], cu_q=s["cu_q"], cu_k=s["cu_k"], causal=c["causal"], out=s["out"])
        if op == "kv_attend":
            return fl.kv_attend(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["start"],
                                cu_rows=s["cu_rows"], tree=s["tree"], out=s["out"])
        if op == "kv_compact":
            fl.kv_compact(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["start"], s["accepted"])
            return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        if op == "kv_fork":
            fl.kv_fork(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["refs"], s["parents"],
                       s["children"], s["lengths"])
            return s["page_table"], s["refs"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        fl.kv_resize(s["page_table"], s["refs"], s["first"], c["page"])
        fl.kv_resize(s["page_table"], s["refs"], s["second"], c["page"])
        return s["page_table"], s["refs"]
    if op == "attention":
        T, D = c["rows"], c["D"]
        U = s["k"].shape[0] if c["context"] else T  # (rows behind the last sequence belong to none)
        cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
        i, j = torch.arange(T, device="cuda"), torch.arange(U, device="cuda")
        a, b = (torch.searchsorted(cu[1:].contiguous(), x, right=True) for cu, x in ((cu_q, i), (cu_k, j)))
        sees = (a[:, None] == b[None, :])
        if c["causal"]:
            # the last rows of q and k stand at the same position
            sees &= (cu_k[b + 1] - j)[None, :] >= (cu_q[a + 1] - i)[:, None]
        q = s["q"][:T].float().unflatten(1, (c["hkv"], -1)).permute(1, 2, 0, 3)  # [hkv, group, T, D]
        k, v = (s[n].float()[:U].permute(1, 0, 2)[:, None] for n in "kv")
        w = _plain_softmax(q @ k.transpose(-1, -2) / math.sqrt(D), sees)
        s["out"][:T] = (w @ v).permute(2, 0, 1, 3).flatten(1, 2).to(s["out"].dtype)
        return s["out"]
    if op == "kv_attend":
        B, page, T = c["seqs"], c["page"], c["rows"]
        each = T // B
        table, start = s["page_table"].long(), s["start"].long()
        p = torch.arange(table.shape[1] * page, device="cuda")
        place = table.clamp(min=0)[:, p // page], (p % page).expand(B, -1)
        draft = p - start[:, None]  # [B, positions]; negative in the context
        i = torch.arange(each, device="cuda")
        if s["tree"] is None:
            new = draft[:, None, :] <= i[:, None]
        else:
            tree = s["tree"][:T].unflatten(0, (B, each))
            new = tree.gather(2, draft[:, None, :].clamp(0, each - 1).expand(-1, each, -1))
        sees = (draft[:, None, :] < 0) | (new & (draft[:, None, :] < each))
        k, v = (_values(s, n, *place).transpose(1, 2)[:, :, None] for n in "kv")  # [B, hkv, 1, positions, D]
        q = s["q"][:T].float().reshape(B, each, c["hkv"], -1, c["D"]).permute(0, 2, 3, 1, 4)
        w = _plain_softmax(q @ k.transpose(-1, -2) / math.sqrt(c["D"]), sees[:, None, None])
        s["out"][:T] = (w @ v).permute(0, 3, 1, 2, 4).reshape(T, c["hq"], c["D"]).to(s["out"].dtype)
        return s["out"]
    if op == "kv_compact":
        table, start, acc = s["page_table"].long(), s["start"].long()[:, None], s["accepted"].long()
        j = torch.arange(acc.shape[1], device="cuda")
        # behind the accepted ones a row moves onto itself
        src, dst = start + torch.where(acc < 0, 0, acc), start + torch.where(acc < 0, 0, j)
        (ps, rs), (pd, rd) = ((table.gather(1, p // c["page"]), p % c["page"]) for p in (src, dst))
        for t in (s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8), s["k_scale"], s["v_scale"]):
            t[pd, rd] = t[ps, rs]
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    table, refs = s["page_table"], s["refs"]
    if op == "kv_fork":
        page = c["page"]
        mine, theirs = s["children"].long(), s["parents"].long()
        n = s["lengths"].long()[:, None]
        old = table[mine]
        refs.scatter_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).int().flatten())
        j = torch.arange(table.shape[1], device="cuda")
        new = torch.where(j < n // page, table[theirs], -1)
        refs.scatter_add_(0, new.clamp(min=0).flatten().long(), (new >= 0).int().flatten())
        part = n[:, 0] % page
        free = torch.argsort((refs > 0).int(), stable=True)  # free pages first, in order
        fresh = free[((part > 0).cumsum(0) - 1).clamp(min=0)].int()
        refs.scatter_add_(0, fresh.long(), (part > 0).int())
        # (a sequence that ends with its page copies its first page onto itself)
        last = torch.where(part > 0, n[:, 0] // page, 0)
        tail = table[theirs].gather(1, last[:, None])[:, 0].long()
        table[mine] = torch.where((j == n // page) & (part > 0)[:, None], fresh[:, None], new)
        at = torch.arange(page, device="cuda")
        keep = (at < part[:, None])
        to = torch.where(part > 0, fresh.long(), tail)
        for t in (s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8), s["k_scale"], s["v_scale"]):
            m = keep.reshape(keep.shape + (1,) * (t.dim() - 2))
            t[to] = torch.where(m, t[tail], t[to])
        return table, refs, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    _plain_resize(table, refs, s["first"], c["page"])
    _plain_resize(table, refs, s["second"], c["page"])
    return table, refs


def _plain_resize(table, refs, lengths, page):
    need = (lengths[:, None] + page - 1) // page
    j = torch.arange(table.shape[1], device="cuda")
    held = table >= 0
    drop = held & (j >= need)
    refs.scatter_add_(0, table.clamp(min=0).flatten().long(), -drop.int().flatten())
    want = ~held & (j < need)
    rank = want.flatten().cumsum(0).reshape(want.shape) - 1
    free = refs == 0
    order = torch.argsort((~free).int(), stable=True)
    page_of = order[rank.clamp(0, refs.shape[0] - 1)].int()
    got = want & (rank < free.sum())
    refs.scatter_add_(0, page_of.flatten().long(), got.int().flatten())
    table.copy_(torch.where(got, page_of, torch.where(drop, -1, table)))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    op = c["op"]
    if op == "attention":
        lq, lk = _lengths(c)
        pairs = sum(a * b - (a * (a - 1) // 2 if c["causal"] else 0) for a, b in zip(lq, lk))
        b = 2 * c["D"] * (2 * sum(lq) * c["hq"] + 2 * sum(lk) * c["hkv"])
        return {"bytes": b + 8 * (c["seqs"] + 1), "flops": 4 * pairs * c["hq"] * c["D"]}
    if op == "kv_attend":
        each = c["rows"] // c["seqs"]
        cached = sum(_contexts(c)) + c["rows"]
        pages = sum(-(-(n + each) // c["page"]) for n in _contexts(c))
        pairs = each * sum(_contexts(c)) + c["seqs"] * each * (each + 1) // 2
        b = cached * c["hkv"] * (2 * c["D"] + 8) + 4 * c["rows"] * c["hq"] * c["D"] + 4 * (2 * c["seqs"] + pages)
        return {"bytes": b + (c["rows"] * each if c["tree"] else 0), "flops": 4 * pairs * c["hq"] * c["D"]}
    if op == "kv_compact":
        moved = sum(j != a for row in _accepted(c) for j, a in enumerate(row) if a >= 0)
        return {"bytes": 2 * moved * c["H"] * (2 * c["D"] + 8) + 4 * c["seqs"] * (1 + c["most"]) + 8 * moved, "flops": 0}
    if op == "kv_fork":
        lens = [n for n in _spread(c["parents"], c["length"] * c["parents"]) for _ in range(c["each"])]
        rows = sum(n % c["page"] for n in lens)
        entries = sum(-(-n // c["page"]) for n in lens)
        return {"bytes": 2 * rows * c["H"] * (2 * c["D"] + 8) + 16 * entries + 12 * len(lens), "flops": 0}
    before, first, second = _turns(c)
    pages = sum(-(-n // c["page"]) for n in before) + c["spare"]
    moved = sum(abs(-(-a // c["page"]) - -(-b // c["page"])) for a, b in list(zip(second, first)) * 2)
    # both calls: which pages are free, the lengths, and each entry that changes with its page's count
    return {"bytes": 2 * (4 * pages + 4 * c["seqs"]) + 12 * moved, "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(q, k, v, sees):
    """q [rows, hq, D] over k, v [keys, hkv, D], one head at a time; sees [rows, keys]."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    if k.shape[0] == 0 or q.shape[0] == 0:
        return out
    group = q.shape[1] // k.shape[1]
    none = ~sees.any(1)
    for h in range(q.shape[1]):
        x = torch.matmul(q[:, h].double(), k[:, h // group].double().T) * q.shape[2] ** -0.5
        x.masked_fill_(~sees, -math.inf)
        w = torch.softmax(x, 1)
        w[none] = 0.0
        out[:, h] = torch.matmul(w, v[:, h // group].double())
    return out


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    op = c["op"]
    if op == "attention":
        out = s["out"].double()
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(c["seqs"]):
            n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
            sees = torch.ones(n, m, dtype=torch.bool, device="cuda")
            if c["causal"]:
                sees = torch.tril(sees, m - n)
            out[cq[b]:cq[b + 1]] = _exact_rows(s["q"][cq[b]:cq[b + 1]], s["k"][ck[b]:ck[b + 1]], s["v"][ck[b]:ck[b + 1]], sees)
        return out
    if op == "kv_attend":
        out = s["out"].double()
        each = c["rows"] // c["seqs"]
        for b, n in enumerate(s["start"].tolist()):
            p = torch.arange(n + each, device="cuda")
            place = s["page_table"][b].long()[p // c["page"]] * c["page"] + p % c["page"]
            k, v = (s[x + "_cache"].float().flatten(0, 1)[place].double()
                    * s[x + "_scale"].double().flatten(0, 1)[place].unsqueeze(2) for x in "kv")
            rows = slice(b * each, (b + 1) * each)
            new = torch.tril(torch.ones(each, each, dtype=torch.bool, device="cuda")) if s["tree"] is None else s["tree"][rows]
            sees = torch.cat((torch.ones(each, n, dtype=torch.bool, device="cuda"), new), 1)
            out[rows] = _exact_rows(s["q"][rows], k, v, sees)
        return out
    if op == "kv_compact":
        # codes are whole numbers, or 8-bit floats: what is left to compare is the scales
        outs = [None, None]
        for n in "kv":
            flat = s[n + "_scale"].double().flatten(0, 1)
            old = flat.clone()
            for b, row in enumerate(s["accepted"].tolist()):
                place = lambda p: int(s["page_table"][b, p // c["page"]]) * c["page"] + p % c["page"]  # noqa: E731
                at = int(s["start"][b])
                for j, a in enumerate(row):
                    if a >= 0:
                        flat[place(at + j)] = old[place(at + a)]
            outs.append(flat.reshape(s[n + "_scale"].shape))
        return tuple(outs)
    if op == "kv_fork":
        outs = [None] * 4
        taken = set(s["page_table"].flatten().tolist())
        free = [p for p in range(s["refs"].shape[0]) if p not in taken]
        scales = [s[n + "_scale"].double() for n in "kv"]
        for parent, n in zip(s["parents"].tolist(), s["lengths"].tolist()):
            if n % c["page"]:
                tail, to = int(s["page_table"][parent, n // c["page"]]), free.pop(0)
                for t in scales:
                    t[to, :n % c["page"]] = t[tail, :n % c["page"]].clone()
        return tuple(outs + scales)
    return None
