"""Float64 CPU oracle of attention and of the cache's page keeping.

TEST INFRASTRUCTURE ONLY, like fusedlin_oracle: plain definitions in NumPy, imported by tests only.
"""
from __future__ import annotations

import numpy as np


def softmax_rows(q, k, v, sees, scale):
    """One head: q [n, D], k and v [m, D], sees [n, m]. Returns out, sum of w |v|, sum of (w v)^2, the largest sum of
    |q| |k| scale / ln 2 of a row's scores, and the largest weight."""
    n, D = q.shape
    out, mag, sq = np.zeros((n, D)), np.zeros((n, D)), np.zeros((n, D))
    size, top = np.zeros(n), np.zeros(n)
    for i in range(n):
        j = np.flatnonzero(sees[i])
        if len(j) == 0:
            continue
        x = k[j] @ q[i] * scale
        w = np.exp(x - x.max())
        w /= w.sum()
        out[i], mag[i], sq[i] = w @ v[j], w @ np.abs(v[j]), (w ** 2) @ (v[j] ** 2)
        size[i] = (np.abs(k[j]) @ np.abs(q[i])).max() * scale / np.log(2.0)
        top[i] = w.max()
    return out, mag, sq, size, top


def causal(n, m):
    """Row i of n sees keys 0 .. i + m - n."""
    return np.arange(m)[None, :] <= np.arange(n)[:, None] + (m - n)


def attention(q, k, v, cu_q, cu_k, is_causal, scale):
    """q [rows, hq, D], k and v [keys, hkv, D]: a dict of what softmax_rows returns, laid out like q."""
    group = q.shape[1] // k.shape[1]
    out, mag, sq = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    size, top = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for b in range(len(cu_q) - 1):
        r, s = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        sees = causal(n, m) if is_causal else np.ones((n, m), dtype=bool)
        for h in range(q.shape[1]):
            out[r, h], mag[r, h], sq[r, h], size[r, h], top[r, h] = softmax_rows(q[r, h], k[s, h // group], v[s, h // group],
                                                                                 sees, scale)
    return {"out": out, "mag": mag, "sq": sq, "size": size, "top": top}


def kv_attend(q, k, v, k_there, cu_rows, start, tree, scale):
    """q [rows, hq, D]; k, v: for each sequence the values [positions, hkv, D] its table gives, k_there: which of the
    positions have a page. tree [rows, drafts] or None."""
    hkv = k[0].shape[1]
    group = q.shape[1] // hkv
    out, mag, sq = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    size, top = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for b in range(len(start)):
        r = slice(cu_rows[b], cu_rows[b + 1])
        n = cu_rows[b + 1] - cu_rows[b]
        m = min(max(int(start[b]) + n, 0), len(k_there[b]))
        sees = np.zeros((n, m), dtype=bool)
        for i in range(n):
            for p in range(m):
                j = p - int(start[b])
                if not k_there[b][p]:
                    continue
                if j < 0:
                    sees[i, p] = True
                elif tree is None:
                    sees[i, p] = j <= i
                else:
                    sees[i, p] = j < tree.shape[1] and bool(tree[cu_rows[b] + i, j])
        for h in range(q.shape[1]):
            out[r, h], mag[r, h], sq[r, h], size[r, h], top[r, h] = softmax_rows(
                q[r, h], k[b][:m, h // group], v[b][:m, h // group], sees, scale)
    return {"out": out, "mag": mag, "sq": sq, "size": size, "top": top}


def kv_resize(table, refs, lengths, page):
    """The table and the counts after, and whether every entry that wants a page has one."""
    table, refs = table.copy(), refs.copy()
    B, per = table.shape
    fine = True
    need = [0 if n <= 0 else -(-int(n) // page) for n in lengths]
    for b in range(B):
        fine &= need[b] <= per
        for j in range(per):
            e = table[b, j]
            if j >= need[b] and 0 <= e < len(refs):
                refs[e] -= 1
                table[b, j] = -1
    free = [p for p in range(len(refs)) if refs[p] == 0]
    for b in range(B):
        for j in range(min(need[b], per)):
            if 0 <= table[b, j] < len(refs):
                continue
            if free:
                table[b, j] = free.pop(0)
                refs[table[b, j]] = 1
            else:
                table[b, j] = -1
                fine = False
    return table, refs, fine


def kv_fork(table, refs, parents, children, lengths, page):
    """The table and the counts after, the copies made (page from, page to, rows), and whether every entry has its page."""
    table, refs = table.copy(), refs.copy()
    B, per = table.shape
    fine, copies = True, []
    held = lambda e: 0 <= e < len(refs)  # noqa: E731
    use = [i for i in range(len(parents)) if 0 <= parents[i] < B and 0 <= children[i] < B]
    fine &= len(use) == len(parents)
    for i in use:
        for e in table[children[i]]:
            if held(e):
                refs[e] -= 1
    wants = []
    for i in use:
        n = max(0, int(lengths[i]))
        full, part = n // page, n % page
        if full >= per:
            fine &= full == per and part == 0
            full, part = per, 0
        row = np.full(per, -1, dtype=table.dtype)
        for j in range(full):
            e = table[parents[i], j]
            if held(e):
                row[j] = e
                refs[e] += 1
            else:
                fine = False
        if part:
            if held(table[parents[i], full]):
                wants.append((i, full, part))
            else:
                fine = False
        table[children[i]] = row
    free = [p for p in range(len(refs)) if refs[p] == 0]
    for i, full, part in wants:
        if free:
            to = free.pop(0)
            refs[to] = 1
            table[children[i], full] = to
            copies.append((int(table[parents[i], full]), to, part))
        else:
            fine = False
    return table, refs, copies, fine


def kv_compact(table, n_pages, start, accepted, page):
    """The moves, in order: (from (page, row), to (page, row)); and whether every row has its pages."""
    fine, moves = True, []

    def place(b, p):
        if not 0 <= p < table.shape[1] * page or not 0 <= table[b, p // page] < n_pages:
            return None
        return int(table[b, p // page]), p % page

    for b in range(len(start)):
        for j, a in enumerate(accepted[b]):
            if a < 0:
                break
            if a == j:
                continue
            src, dst = place(b, int(start[b]) + int(a)), place(b, int(start[b]) + j)
            if src is None or dst is None:
                fine = False
            else:
                moves.append((src, dst))
    return moves, fine
