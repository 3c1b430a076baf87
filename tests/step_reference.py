"""Plain 64-bit definitions of the batched paged step's operators (numpy,
one request at a time, no code shared with the CUDA path)."""
import math

import numpy as np

PAGE = 64


def page_plan(cache_len, new_len, table, stack, max_pages, n_pages, max_rows, held_len=None):
    """stack: the free pages, top last.  Returns kv_len, cu_rows, slot_map, table, stack, waited, bad, held_len."""
    table, stack, cap = np.array(table), list(stack), max_pages * PAGE
    bad = waited = False
    hold = [max(h, c) for h, c in zip(cache_len if held_len is None else held_len, cache_len)]
    held_out = [int(h) for h in (held_len if held_len is not None else cache_len)]
    for b, (c, m) in enumerate(zip(cache_len, new_len)):
        if m == -1 and 0 <= c and hold[b] <= cap:
            stack += [int(p) for p in table[b, :-(-hold[b] // PAGE)]]
            held_out[b] = 0
    kv, cu, slots, blocked = [], [0], [], False
    for b, (c, m) in enumerate(zip(cache_len, new_len)):
        if c < 0 or hold[b] > cap or m < -1:
            bad, c, m = True, 0, 0
        elif m == -1:
            c, m = 0, 0
        else:
            if c + m > cap:
                bad, m = True, 0
            else:
                have = -(-hold[b] // PAGE)
                want = max(-(-(c + m) // PAGE), have)
                if blocked or want - have > len(stack) or cu[-1] + m > max_rows:
                    waited |= m > 0
                    blocked, m = True, 0
                else:
                    for i in range(have, want):
                        table[b, i] = stack.pop()
                    slots += [int(table[b, (c + t) // PAGE]) * PAGE + (c + t) % PAGE for t in range(m)]
            held_out[b] = max(held_out[b], c + m)
        kv.append(c + m)
        cu.append(cu[-1] + m)
    return (kv, cu, slots + [-1] * (max_rows - len(slots)), table, stack[:n_pages], waited, bad or len(stack) > n_pages,
            held_out)


def mrope_axis(sections, interleaved, j):
    n = len(sections)
    if interleaved:
        return j % n if j < n * sections[j % n] else 0
    a = 0
    while j >= sections[a]:
        j -= sections[a]
        a += 1
    return a


def mrope(x, pos, sections, base, rot, interleaved):
    """x [rows, heads, D] float64, pos [axes, rows]."""
    y = np.array(x, dtype=np.float64)
    half = rot // 2
    for j in range(half):
        th = pos[mrope_axis(sections, interleaved, j)].astype(np.float64) * float(base) ** (-2.0 * j / rot)
        c, s = np.cos(th)[:, None], np.sin(th)[:, None]
        y[:, :, j] = x[:, :, j] * c - x[:, :, j + half] * s
        y[:, :, j + half] = x[:, :, j + half] * c + x[:, :, j] * s
    return y


def verify(p, q, ids, u, us, n_draft):
    """One sequence: p [K+1, V], q [K, V] or None, all float64 values of the inputs.  (k, out_ids, bad)."""
    V, k, bad = p.shape[1], 0, False
    K = len(ids)
    while k < n_draft:
        x = ids[k]
        if not 0 <= x < V:
            bad = True
            break
        if not u[k] * (1.0 if q is None else q[k, x]) < p[k, x]:
            break
        k += 1

    def clean(a, b):
        with np.errstate(invalid="ignore"):
            return np.where((a > b) & np.isfinite(a), a - np.where(a > b, b, 0.0), 0.0)

    other = np.zeros(V)
    if k < n_draft:
        if q is not None:
            other = q[k]
        elif 0 <= ids[k] < V:
            other = np.zeros(V)
            other[ids[k]] = 1.0
    r = clean(p[k], other)
    if not r.sum() > 0:
        r = clean(p[k], np.zeros(V))
    if not r.sum() > 0:
        return k, list(ids[:k]) + [0] + [-1] * (K - k), True
    us = min(max(us, 0.0), 1.0 - 2.0 ** -24) if not math.isnan(us) else 0.0
    total, run, token = math.fsum(r), 0.0, None
    target = us * total
    c = np.cumsum(r)
    hit = np.flatnonzero((c > target) & (r > 0))
    token = int(hit[0]) if len(hit) else int(np.flatnonzero(r > 0)[-1])
    return k, list(ids[:k]) + [token] + [-1] * (K - k), bad


def chunk_attention(q, k_pages, v_pages, table, kv_len, n_noisy, n_hidden, scale):
    """One request: q [n, Hq, D]; pages K [pages, Hkv, 64, D], V^T [pages, Hkv, D, 64]; all
    float64.  Returns (out [n, Hq, D], lse [n, Hq]): rows that see nothing give 0 and -inf."""
    n, Hq, D = q.shape
    Hkv = k_pages.shape[1]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    pages = np.asarray(table[:-(-kv_len // PAGE)], dtype=int)
    k = k_pages[pages].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)
    v = v_pages[pages].transpose(1, 0, 3, 2).reshape(Hkv, -1, D)
    for t in range(n):
        end = kv_len if t >= n - n_noisy else kv_len - n + t + 1
        if end <= n_hidden:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = scale * (k[g, n_hidden:end] @ q[t, h])
            m = s.max()
            e = np.exp(s - m)
            out[t, h] = (e / e.sum()) @ v[g, n_hidden:end]
            lse[t, h] = m + math.log(e.sum())
    return out, lse
