"""The operators of one batched step over a paged KV cache, as they are timed.

A ragged batch of requests goes through four operators, in this order:

* ``page_plan``: block tables, row offsets, slot map and the stack of free
  pages from the requests' lengths;
* ``mrope`` / ``mrope_append``: rotary positions with several axes (time,
  height, width) on rows, and the same fused with the write of the new keys
  and values into their pages;
* ``chunk_attn``: attention of every request's new rows (one, a block, or a
  prompt chunk) over its paged cache;
* ``verify``: drafted tokens verified against the target's probabilities with
  given random numbers.

``own`` selects between the plain form (elementary torch operations) and the
library's kernels.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step of a small server: one 16-token block each
        {"name": "plan_blocks_8", "op": "page_plan", "n": 8, "kind": "blocks", "max_len": 1600, "max_new": 16,
         "layout": 1},
        # a large server's step: prompt chunks, blocks, idle and finished requests
        {"name": "plan_mixed_512", "op": "page_plan", "n": 512, "kind": "mixed", "max_len": 32768, "max_new": 2048,
         "layout": 2},
        # one block of the 16/2-head decoder (latency)
        {"name": "append_block_16", "op": "mrope_append", "rows": 16, "Hq": 16, "Hkv": 2, "D": 128,
         "sections": "16,24,24", "interleaved": 0, "layout": 3},
        # a batch of prompt chunks, ragged, smaller heads, interleaved axes
        {"name": "append_ragged_1357", "op": "mrope_append", "rows": 1357, "Hq": 14, "Hkv": 2, "D": 64,
         "sections": "12,10,10", "interleaved": 1, "layout": 4},
        # the largest step: many prompt chunks at once
        {"name": "append_chunks_16384", "op": "mrope_append", "rows": 16384, "Hq": 16, "Hkv": 2, "D": 128,
         "sections": "16,24,24", "interleaved": 0, "layout": 5},
        # image rows with height/width positions in fp32
        {"name": "mrope_image_fp32", "op": "mrope", "rows": 4999, "heads": 16, "D": 80, "rot": 80,
         "sections": "20,20", "interleaved": 0, "dtype": "fp32", "layout": 6},
        # the decode shape: one 16-row noisy block over a 1344-slot context
        {"name": "attn_block_1x16", "op": "chunk_attn", "n": 1, "kind": "blocks", "new": 16, "min_len": 1344,
         "max_len": 1344, "Hq": 16, "Hkv": 2, "D": 128, "hidden": 0, "layout": 7},
        # batched single tokens over long ragged caches (bandwidth)
        {"name": "attn_tokens_64x1", "op": "chunk_attn", "n": 64, "kind": "tokens", "new": 1, "min_len": 900,
         "max_len": 16000, "Hq": 16, "Hkv": 2, "D": 128, "hidden": 0, "layout": 8},
        # chunks, blocks and single tokens together, hidden image rows, other heads
        {"name": "attn_mixed_24", "op": "chunk_attn", "n": 24, "kind": "mixed", "new": 517, "min_len": 40,
         "max_len": 4100, "Hq": 14, "Hkv": 2, "D": 64, "hidden": 1, "layout": 9},
        # a prompt chunk over a long cached context (compute)
        {"name": "attn_chunk_4096", "op": "chunk_attn", "n": 1, "kind": "chunks", "new": 4096, "min_len": 8192,
         "max_len": 8192, "Hq": 16, "Hkv": 2, "D": 128, "hidden": 0, "layout": 10},
        # one request's drafts against both distributions (latency)
        {"name": "verify_1x4_fp32", "op": "verify", "b": 1, "K": 4, "V": 151936, "dtype": "fp32", "draft_p": 1,
         "layout": 11},
        # a batch of argmax-drafted blocks
        {"name": "verify_128x15_bf16", "op": "verify", "b": 128, "K": 15, "V": 151936, "dtype": "bf16",
         "draft_p": 0, "layout": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["page_plan", "mrope_append", "mrope", "chunk_attn", "chunk_attn", "verify"])
    case = {"op": op, "layout": rng.randrange(1 << 20)}
    if op == "page_plan":
        case.update(n=_log(rng, 1, 512), kind=rng.choice(["blocks", "mixed"]), max_len=_log(rng, 64, 32768),
                    max_new=_log(rng, 1, 2048))
    elif op == "mrope_append":
        D, sections = rng.choice([(128, "16,24,24"), (128, "64"), (64, "12,10,10"), (64, "8,12,12")])
        Hq, Hkv = rng.choice([(16, 2), (8, 1), (14, 2), (12, 4), (8, 8)])
        case.update(rows=_log(rng, 1, 8000), Hq=Hq, Hkv=Hkv, D=D, sections=sections, interleaved=rng.randrange(2))
    elif op == "mrope":
        D, rot, sections = rng.choice([(80, 80, "20,20"), (128, 128, "16,24,24"), (64, 32, "4,6,6"), (72, 72, "18,18")])
        case.update(rows=_log(rng, 1, 8000), heads=rng.choice([1, 3, 16, 20]), D=D, rot=rot, sections=sections,
                    interleaved=rng.randrange(2), dtype=rng.choice(["bf16", "fp32"]))
    elif op == "chunk_attn":
        D = rng.choice([64, 128])
        Hq, Hkv = rng.choice([(16, 2), (8, 1), (14, 2), (12, 4), (8, 8)])
        kind = rng.choice(["blocks", "tokens", "mixed", "chunks"])
        n = _log(rng, 1, 64) if kind != "chunks" else _log(rng, 1, 4)
        new = {"blocks": _log(rng, 2, 32), "tokens": 1, "mixed": _log(rng, 2, 600), "chunks": _log(rng, 64, 1500)}[kind]
        hi = _log(rng, 70, 8000)
        case.update(n=n, kind=kind, new=new, min_len=_log(rng, 1, hi), max_len=hi, Hq=Hq, Hkv=Hkv, D=D,
                    hidden=rng.randrange(2))
    else:
        case.update(b=_log(rng, 1, 64), K=rng.randint(1, 15), V=rng.choice([151936, 32000, 50257, 4099, 128256]),
                    dtype=rng.choice(["fp32", "bf16"]), draft_p=rng.randrange(2))
    return case


# ------------------------------------------------------- lengths of one case
def _plan_lens(case):
    """(cached, new) lengths: blocks of max_new rows, or a mix of chunks, blocks, idle (0) and finished (-1)."""
    r = random.Random(case["layout"])
    cached, new = [], []
    for _ in range(case["n"]):
        cached.append(r.randint(0, case["max_len"]))
        if case["kind"] == "blocks":
            new.append(case["max_new"])
        else:
            p = r.random()
            new.append(-1 if p < 0.1 else 0 if p < 0.2 else min(16, case["max_new"]) if p < 0.7
                       else r.randint(1, case["max_new"]))
    return cached, new


def _attn_lens(case):
    """Per request (new rows, slots with the new rows, noisy rows of the new, hidden leading slots)."""
    r = random.Random(case["layout"])
    out = []
    for _ in range(case["n"]):
        L = r.randint(case["min_len"], case["max_len"])
        kind = case["kind"]
        if kind == "mixed":
            kind = r.choice(["blocks", "tokens", "chunks", "chunks", "idle"] if out else ["chunks"])
        n = {"blocks": min(16, case["new"]) if case["kind"] == "mixed" else case["new"], "tokens": 1, "idle": 0,
             "chunks": case["new"] if case["n"] == 1 else r.randint(1, case["new"])}[kind]
        noisy = n if kind == "blocks" else 0
        hidden = r.randint(0, L + n // 2) if case["hidden"] and r.random() < 0.5 else 0   # may leave rows empty
        out.append((n, L + n, noisy, hidden))
    return out


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _append_pages(case):
    return -(-case["rows"] // PAGE) * 2 + 8


def _visible(case):
    """Visible (row, slot) pairs of one head, and the slots some row sees."""
    pairs = slots = 0
    for n, kv, noisy, hidden in _attn_lens(case):
        base = kv - n
        for_t = n - noisy
        lo = max(0, min(for_t, hidden - base))       # causal rows before the first visible slot see nothing
        pairs += sum(range(base + lo + 1 - hidden, base + for_t + 1 - hidden)) if lo < for_t else 0
        pairs += noisy * max(0, kv - hidden)
        slots += max(0, kv - hidden) if n else 0
    return pairs, slots


def work(case):
    op = case["op"]
    if op == "page_plan":
        cached, new = _plan_lens(case)
        rows = sum(max(0, m) for m in new)
        pages = sum(-(-(c + max(0, m)) // PAGE) - -(-c // PAGE) for c, m in zip(cached, new) if m >= 0)
        freed = sum(-(-c // PAGE) for c, m in zip(cached, new) if m < 0)
        n = case["n"]
        return {"bytes": 8 * n + 4 + 8 * pages + 8 * freed + 4 * n + 4 * (n + 1) + 4 * rows + 4, "flops": 4 * rows}
    if op == "mrope_append":
        el = case["rows"] * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
        rot = case["rows"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": 4 * el + case["rows"] * (4 * len(_sections(case)) + 4), "flops": 3 * rot}
    if op == "mrope":
        el = case["rows"] * case["heads"] * case["D"]
        return {"bytes": 2 * el * (4 if case["dtype"] == "fp32" else 2) + 4 * case["rows"] * len(_sections(case)),
                "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    if op == "chunk_attn":
        pairs, slots = _visible(case)
        rows = sum(n for n, *_ in _attn_lens(case))
        return {"bytes": 4 * rows * case["Hq"] * case["D"] + 4 * slots * case["Hkv"] * case["D"],
                "flops": 4 * pairs * case["Hq"] * case["D"]}
    es = 4 if case["dtype"] == "fp32" else 2
    b, K, V = case["b"], case["K"], case["V"]
    two = 2 if case["draft_p"] else 1
    return {"bytes": b * (two * V * es + K * (8 + two * es) + 12 + 4 * (K + 2)), "flops": 3 * b * V}


# --------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + salt * 7919 + 17) % (1 << 62))
    return g


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _positions(g, n_axes, rows):
    """Text rows count up on every axis; stretches of image rows hold time still and walk a grid."""
    base = int(torch.randint(0, 40000, (1,), generator=g, device=DEV))
    t = torch.arange(rows, device=DEV) + base
    pos = t.repeat(n_axes, 1)
    img = (t // 97) % 2 == 0
    for a in range(n_axes):
        w = [t - t % 97, t // 24 % 41 + base, t % 24 + base, t % 7][min(a, 3)]
        pos[a] = torch.where(img, w, pos[a])
    return pos.to(torch.int32).contiguous()


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed, case["layout"])
    s = {"case": case}
    if op == "page_plan":
        cached, new = _plan_lens(case)
        n = case["n"]
        held = [-(-c // PAGE) for c in cached]
        max_pages = -(-(case["max_len"] + case["max_new"]) // PAGE)
        spare = n * (-(-case["max_new"] // PAGE) + 1) + 3
        n_pages = sum(held) + spare
        perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((n, max_pages), -1, dtype=torch.int32, device=DEV)
        hd = _i32(held)
        idx = torch.arange(max_pages, device=DEV)[None, :].expand(n, -1)
        first = (torch.cumsum(hd, 0) - hd)[:, None]
        has = idx < hd[:, None]
        table[has] = perm[(first + idx)[has]]
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
        free[:spare] = perm[sum(held):]
        max_rows = sum(max(0, m) for m in new) + 37      # the row buffer is a little longer than this step needs
        s.update(cache_len=_i32(cached), new_len=_i32(new), table=table, free=free, count=_i32([spare]),
                 max_pages=max_pages, n_pages=n_pages, max_rows=max_rows, kv_len=_i32([0] * n),
                 cu=_i32([0] * (n + 1)), slots=_i32([0] * max_rows), count_out=_i32([0]))
    elif op == "mrope_append":
        rows, D, Hq, Hkv = case["rows"], case["D"], case["Hq"], case["Hkv"]
        n_pages = _append_pages(case)
        slots, pages = [], torch.randperm(n_pages, generator=g, device=DEV).tolist()
        r = random.Random(case["layout"])
        while len(slots) < rows:                          # requests of odd lengths, each from some slot of its page
            n, at = min(rows - len(slots), r.randint(1, 700)), r.randrange(PAGE)
            at = 0 if len(pages) < 4 + (rows - len(slots)) // PAGE else at
            while n > 0:
                m, page = min(n, PAGE - at), pages.pop()
                slots += range(page * PAGE + at, page * PAGE + at + m)
                n, at = n - m, 0
            if len(pages) < 4 + (rows - len(slots)) // PAGE and len(slots) < rows:
                m = rows - len(slots)                      # the rest as one request
                while m > 0:
                    page, k = pages.pop(), min(m, PAGE)
                    slots += range(page * PAGE, page * PAGE + k)
                    m -= k
        s.update(qkv=_randn(g, rows, (Hq + 2 * Hkv) * D), pos=_positions(g, len(_sections(case)), rows),
                 slots=_i32(slots), k_pages=_randn(g, n_pages, Hkv, PAGE, D), v_pages=_randn(g, n_pages, Hkv, D, PAGE),
                 q=torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=DEV), n_pages=n_pages)
    elif op == "mrope":
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        s.update(x=_randn(g, case["rows"], case["heads"], case["D"], dtype=dt),
                 pos=_positions(g, len(_sections(case)), case["rows"]))
        s["out"] = torch.zeros_like(s["x"])
    elif op == "chunk_attn":
        lens = _attn_lens(case)
        D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
        rows = sum(n for n, *_ in lens)
        held = [-(-kv // PAGE) for _, kv, _, _ in lens]
        n_pages, max_pages = sum(held) + 5, max(held)
        perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros((case["n"], max_pages), dtype=torch.int32, device=DEV)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = perm[at:at + h]
            at += h
        cu = [0]
        for n, *_ in lens:
            cu.append(cu[-1] + n)
        s.update(q=_randn(g, max(1, rows), Hq, D), k_pages=_randn(g, n_pages, Hkv, PAGE, D),
                 v_pages=_randn(g, n_pages, Hkv, D, PAGE), table=table, cu=_i32(cu), lens=lens, rows=rows,
                 kv_len=_i32([x[1] for x in lens]), noisy=_i32([x[2] for x in lens]), hidden=_i32([x[3] for x in lens]),
                 out=torch.zeros(max(1, rows), Hq, D, dtype=torch.bfloat16, device=DEV), n_pages=n_pages,
                 max_pages=max_pages)
        if own:
            import block_diffusion_vlm_b200 as dv
            nb = dv.chunk_attn_paged_workspace_size(case["n"], max(1, rows), Hq, Hkv, D)
            s["ws"] = torch.zeros((nb + 3) // 4 + 1, dtype=torch.int32, device=DEV)
    else:
        b, K, V = case["b"], case["K"], case["V"]
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        p = torch.empty(b, K + 1, V, dtype=dt, device=DEV)
        q = torch.empty(b, K, V, dtype=dt, device=DEV) if case["draft_p"] else None
        ids = torch.empty(b, K, dtype=torch.int32, device=DEV)
        for i in range(b):       # the draft model is the target with noise on its logits
            z = 4.0 * torch.randn(K + 1, V, generator=g, device=DEV)
            p[i] = torch.softmax(z, -1).to(dt)
            d = torch.softmax(z[:K] + 0.3 * torch.randn(K, V, generator=g, device=DEV), -1)
            if q is not None:
                q[i] = d.to(dt)
                ids[i] = torch.multinomial(d, 1, generator=g)[:, 0].to(torch.int32)
            else:                # argmax drafts, of a sharper target
                p[i] = torch.softmax(3.0 * z, -1).to(dt)
                ids[i] = d.argmax(-1).to(torch.int32)
        s.update(p=p, q=q, ids=ids, u=torch.rand(b, K, generator=g, device=DEV),
                 us=torch.rand(b, generator=g, device=DEV), len=_i32([1344 + K] * b),
                 acc=_i32([0] * b), out=torch.zeros(b, K + 1, dtype=torch.int32, device=DEV), len_out=_i32([0] * b))
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import block_diffusion_vlm_b200 as dv
    case = s["case"]
    op = case["op"]
    if op == "page_plan":
        dv.page_plan(s["cache_len"], s["new_len"], s["table"], s["free"], s["count"], n_batch=case["n"],
                     max_pages=s["max_pages"], n_pages=s["n_pages"], max_rows=s["max_rows"], kv_len=s["kv_len"],
                     cu_rows=s["cu"], slot_map=s["slots"], free_count_out=s["count_out"])
        return [s["kv_len"], s["cu"], s["slots"], s["table"], s["free"], s["count_out"]]
    if op == "mrope_append":
        dv.mrope_append_paged(s["qkv"], s["pos"], s["slots"], s["q"], s["k_pages"], s["v_pages"], n_rows=case["rows"],
                              Hq=case["Hq"], Hkv=case["Hkv"], D=case["D"], n_pages=s["n_pages"],
                              sections=_sections(case), rope_base=1e6, interleaved=case["interleaved"])
        return [s["q"], s["k_pages"], s["v_pages"]]
    if op == "mrope":
        dv.mrope(s["x"], s["out"], s["pos"], n_rows=case["rows"], n_heads=case["heads"], D=case["D"],
                 rot_dim=case["rot"], sections=_sections(case), rope_base=1e4, interleaved=case["interleaved"],
                 dtype=dv.DVLM_FP32 if case["dtype"] == "fp32" else dv.DVLM_BF16)
        return s["out"]
    if op == "chunk_attn":
        dv.chunk_attn_paged(s["q"], s["out"], s["k_pages"], s["v_pages"], s["table"], s["kv_len"], s["cu"],
                            n_batch=case["n"], n_rows=s["q"].shape[0], n_pages=s["n_pages"], max_pages=s["max_pages"],
                            Hq=case["Hq"], Hkv=case["Hkv"], D=case["D"], scale=case["D"] ** -0.5, n_noisy=s["noisy"],
                            n_hidden=s["hidden"], workspace=s["ws"])
        return s["out"]
    dv.spec_verify_sample(s["p"], s["q"], s["ids"], s["u"], s["us"], b=case["b"], K=case["K"], V=case["V"],
                          dtype=dv.DVLM_FP32 if case["dtype"] == "fp32" else dv.DVLM_BF16, accept_len=s["acc"],
                          out_ids=s["out"], cache_len=s["len"], cache_len_out=s["len_out"])
    return [s["acc"], s["out"], s["len_out"]]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "page_plan":
        return _plan_plain(s)
    if op == "mrope_append":
        rows, D, Hq, Hkv = case["rows"], case["D"], case["Hq"], case["Hkv"]
        x = s["qkv"].float().view(rows, Hq + 2 * Hkv, D)
        y = _rotate_plain(x[:, :Hq + Hkv], s["pos"], _sections(case), 1e6, D, case["interleaved"])
        q, k = y[:, :Hq].to(torch.bfloat16), y[:, Hq:].to(torch.bfloat16)
        slots = s["slots"].long()
        s["k_pages"][slots // PAGE, :, slots % PAGE, :] = k
        s["v_pages"][slots // PAGE, :, :, slots % PAGE] = s["qkv"].view(rows, Hq + 2 * Hkv, D)[:, Hq + Hkv:]
        return [q, s["k_pages"], s["v_pages"]]
    if op == "mrope":
        y = _rotate_plain(s["x"].float(), s["pos"], _sections(case), 1e4, case["rot"], case["interleaved"])
        return y.to(s["x"].dtype)
    if op == "chunk_attn":
        return _attn_plain(s)
    return _verify_plain(s)


def _plan_plain(s):
    case = s["case"]
    n = case["n"]
    cached, new = s["cache_len"].long(), s["new_len"].long()
    held = (cached + PAGE - 1) // PAGE
    live = new >= 0
    ok = live & (cached + new <= s["max_pages"] * PAGE)
    want = torch.where(ok, new, 0)
    need = (cached + want + PAGE - 1) // PAGE - held
    need = torch.where(ok, need, 0)
    freed = torch.where(live, 0, held)
    count = s["count"].long()
    R = freed.sum()
    fits = (torch.cumsum(need, 0) <= count + R) & (torch.cumsum(want, 0) <= s["max_rows"])
    want = torch.where(fits, want, 0)
    need = torch.where(fits, need, 0)
    kv = torch.where(live, cached + want, 0)
    # the stack: returned pages on top, then the new pages off the top
    col = torch.arange(s["max_pages"], device=DEV)[None, :]
    returned = s["table"][(col < freed[:, None])]
    top = count + R
    a0 = torch.cumsum(need, 0) - need
    take = (col >= held[:, None]) & (col < (held + need)[:, None])
    index = (top - 1 - (a0[:, None] + col - held[:, None]))[take]
    if returned.numel():
        got = torch.where(index < count, s["free"][index.clamp(max=s["n_pages"] - 1)],
                          returned[(index - count).clamp(0, returned.numel() - 1)])
    else:
        got = s["free"][index]
    s["table"][take] = got
    left = top - need.sum()
    at = torch.arange(s["n_pages"], device=DEV)
    back = (at >= count) & (at < left)
    if returned.numel():
        s["free"][back] = returned[(at - count)[back]]
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(want, 0)])
    row = torch.arange(s["max_rows"], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    real = row < cu[-1]
    seq = torch.where(real, seq, 0).clamp(max=n - 1)
    slot = cached[seq] + row - cu[seq]
    page = s["table"].long()[seq, torch.where(real, slot // PAGE, 0)]
    slots = torch.where(real, page * PAGE + slot % PAGE, -1)
    return [kv.to(torch.int32), cu.to(torch.int32), slots.to(torch.int32), s["table"], s["free"], left.to(torch.int32)]


def _axes(sections, interleaved, half):
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    m = len(sections)
    return [j % m if j < m * sections[j % m] else 0 for j in range(half)]


def _rotate_plain(x, pos, sections, base, rot, interleaved):
    half = rot // 2
    axis = torch.tensor(_axes(sections, interleaved, half), device=DEV)
    inv = base ** (-2.0 * torch.arange(half, dtype=torch.float64, device=DEV) / rot)
    ang = pos.double()[axis].t() * inv                     # far positions: the angle needs 64 bits
    c, sn = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    a, b = x[..., :half], x[..., half:rot]
    return torch.cat([a * c - b * sn, b * c + a * sn, x[..., rot:]], -1)


def _attn_plain(s):
    case = s["case"]
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    out, at = s["out"], 0
    for b, (n, kv, noisy, hidden) in enumerate(s["lens"]):
        if n == 0:
            continue
        pages = s["table"][b, :-(-kv // PAGE)].long()
        k = s["k_pages"][pages].float().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :kv]
        v = s["v_pages"][pages].float().permute(1, 0, 3, 2).reshape(Hkv, -1, D)[:, :kv]
        q = s["q"][at:at + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3)
        sc = torch.matmul(q, k[:, None].transpose(-1, -2)) * D ** -0.5
        t = torch.arange(n, device=DEV)[:, None]
        j = torch.arange(kv, device=DEV)[None, :]
        see = ((j <= kv - n + t) | (t >= n - noisy)) & (j >= hidden)
        sc = torch.where(see, sc, float("-inf"))
        m = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - torch.where(torch.isinf(m), 0.0, m))
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v[:, None]) / torch.where(l > 0, l, 1.0)
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(torch.bfloat16)
        at += n
    return out


def _verify_plain(s):
    case = s["case"]
    b, K, V = case["b"], case["K"], case["V"]
    ids = s["ids"].long()
    px = s["p"][:, :K].gather(2, ids[..., None])[..., 0].double()
    qx = s["q"].gather(2, ids[..., None])[..., 0].double() if s["q"] is not None else 1.0
    ok = s["u"].double() * qx < px
    k = torch.cumprod(ok.long(), 1).sum(1)
    rows = torch.arange(b, device=DEV)
    p = s["p"][rows, k].double()
    if s["q"] is not None:
        q = torch.where((k < K)[:, None], s["q"][rows, k.clamp(max=K - 1)].double(), 0.0)
    else:
        hot = torch.arange(V, device=DEV)[None, :] == ids.gather(1, k.clamp(max=K - 1)[:, None])
        q = (hot & (k < K)[:, None]).double()
    r = torch.where(p > q, p - q, 0.0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, torch.where(p > 0, p, 0.0))
    C = torch.cumsum(r, 1)                                 # long sums next to a border: 64 bits
    hit = C > s["us"].double()[:, None] * C[:, -1:]
    v = torch.arange(V, device=DEV)[None, :]
    first = torch.where(hit, v, V).amin(1)
    last = torch.where(r > 0, v, -1).amax(1)
    tok = torch.where(first < V, first, last)
    j = torch.arange(K + 1, device=DEV)[None, :]
    full = torch.cat([ids, ids[:, :1]], 1)
    out = torch.where(j < k[:, None], full, torch.where(j == k[:, None], tok[:, None], -1))
    return [k.to(torch.int32), out.to(torch.int32), (s["len"] - K + k).to(torch.int32)]


# ---------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "page_plan":
        return _plan_exact(s)
    if op in ("mrope_append", "mrope"):
        sec = _sections(case)
        if op == "mrope":
            return _turn(s["x"].double(), s["pos"], sec, 1e4, case["rot"], case["interleaved"])
        rows, D, Hq, Hkv = case["rows"], case["D"], case["Hq"], case["Hkv"]
        x = s["qkv"].double().reshape(rows, Hq + 2 * Hkv, D)
        q = _turn(x[:, :Hq], s["pos"], sec, 1e6, D, case["interleaved"])
        k = _turn(x[:, Hq:Hq + Hkv], s["pos"], sec, 1e6, D, case["interleaved"])
        kp = s["k_pages"].double().transpose(1, 2).reshape(-1, Hkv, D)
        vp = s["v_pages"].double().permute(0, 3, 1, 2).reshape(-1, Hkv, D)
        kp[s["slots"].long()] = k
        vp[s["slots"].long()] = x[:, Hq + Hkv:]
        return [q, kp.reshape(-1, PAGE, Hkv, D).transpose(1, 2), vp.reshape(-1, PAGE, Hkv, D).permute(0, 2, 3, 1)]
    if op == "chunk_attn":
        return _attn_exact(s)
    return _verify_exact(s)


def _plan_exact(s):
    """Request by request on the host."""
    cached, new = s["cache_len"].tolist(), s["new_len"].tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    stack = free[:int(s["count"])].tolist()
    for b, (c, m) in enumerate(zip(cached, new)):
        if m < 0:
            stack += table[b, :-(-c // PAGE)].tolist()
    kv, cu, slots, blocked = [], [0], [], False
    for b, (c, m) in enumerate(zip(cached, new)):
        if m < 0:
            kv.append(0)
            cu.append(cu[-1])
            continue
        h, e = -(-c // PAGE), -(-(c + m) // PAGE)
        if c + m > s["max_pages"] * PAGE:
            m = 0
        elif blocked or e - h > len(stack) or cu[-1] + m > s["max_rows"]:
            blocked, m = True, 0
        else:
            for i in range(h, e):
                table[b, i] = stack.pop()
        slots += [int(table[b, (c + i) // PAGE]) * PAGE + (c + i) % PAGE for i in range(m)]
        kv.append(c + m)
        cu.append(cu[-1] + m)
    slots += [-1] * (s["max_rows"] - len(slots))
    old = int(s["count"])
    free[old:max(old, len(stack))] = stack[old:]
    return [_i32(kv), _i32(cu), _i32(slots), torch.from_numpy(table).to(DEV), torch.from_numpy(free).to(DEV),
            _i32([len(stack)])]


def _turn(x, pos, sections, base, rot, interleaved):
    """Each pair (j, j + rot/2) as a complex number times exp(i angle)."""
    half = rot // 2
    y = x.clone()
    for j in range(half):
        if interleaved:
            a = j % len(sections)
            a = a if j < len(sections) * sections[a] else 0
        else:
            a = int(np.searchsorted(np.cumsum(sections), j, side="right"))
        th = pos[a].double() * math.exp(-2.0 * j / rot * math.log(base))
        z = torch.complex(x[..., j], x[..., j + half]) * torch.polar(torch.ones_like(th), th)[:, None]
        y[..., j], y[..., j + half] = z.real, z.imag
    return y


def _attn_exact(s):
    case = s["case"]
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    pairs, _ = _visible(case)
    if pairs * Hq * D > 2e12:
        return None
    out = s["out"].double()
    at = 0
    for b, (n, kv, noisy, hidden) in enumerate(s["lens"]):
        slot = torch.arange(kv, device=DEV)
        page = s["table"][b].long()[slot // PAGE]
        for h in range(Hq if n else 0):
            k = s["k_pages"][page, h * Hkv // Hq, slot % PAGE].double()
            v = s["v_pages"][page, h * Hkv // Hq, :, slot % PAGE].double()
            for t0 in range(0, n, 1024):
                t = torch.arange(t0, min(n, t0 + 1024), device=DEV)
                last = torch.where(t >= n - noisy, kv - 1, kv - n + t)
                sc = s["q"][at + t, h].double() @ k.t() / math.sqrt(D)
                sc = sc.masked_fill((slot[None] > last[:, None]) | (slot[None] < hidden), -math.inf)
                out[at + t, h] = torch.nan_to_num(torch.softmax(sc, -1)) @ v
        at += n
    return out


def _verify_exact(s):
    case = s["case"]
    b, K, V = case["b"], case["K"], case["V"]
    acc, out, length = [], [], []
    ids, u, us, lens = s["ids"].tolist(), s["u"].double().tolist(), s["us"].double().tolist(), s["len"].tolist()
    for i in range(b):
        k = 0
        while k < K:
            x = ids[i][k]
            q = float(s["q"][i, k, x]) if s["q"] is not None else 1.0
            if not u[i][k] * q < float(s["p"][i, k, x]):
                break
            k += 1
        r = s["p"][i, k].double().cpu().numpy()
        if k < K:
            if s["q"] is not None:
                r = np.maximum(r - s["q"][i, k].double().cpu().numpy(), 0.0)
            else:
                r[ids[i][k]] = max(r[ids[i][k]] - 1.0, 0.0)
        if not r.sum() > 0:
            r = s["p"][i, k].double().cpu().numpy()
        c = np.cumsum(r)
        v = int(np.searchsorted(c, us[i] * c[-1], side="right"))
        acc.append(k)
        out.append(ids[i][:k] + [min(v, int(np.flatnonzero(r > 0)[-1]))] + [-1] * (K - k))
        length.append(lens[i] - K + k)
    return [_i32(acc), _i32(out), _i32(length)]
