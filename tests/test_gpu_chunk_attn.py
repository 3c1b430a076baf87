"""Attention of ragged chunks over paged caches against its plain 64-bit
definition (step_reference.chunk_attention).

Tolerance.  The kernel rounds each probability p_j (relative to a reference
maximum) to bf16, half a step 2^-8 relative, before the product with V; sums
are fp32.  With A = sum_j p_j |v_j| / sum_j p_j the products therefore err by
at most 2^-8 A; fp32 scores (an error of 128 * 2^-24 of sum |q_i k_i| * scale,
below 1e-4 for the N(0, 1) inputs here), exponentials and sums add less than
2^-12 A; the store rounds once more, 2^-8 |o|.  lse carries the scores' 1e-4
and fp32 roundings of a value below 32 (2^-19): 2e-4."""
import numpy as np
import pytest
import torch

import block_diffusion_vlm_b200 as dv
import step_reference as ref
from gpu_util import assert_ok, status, ws_tensor

pytestmark = pytest.mark.gpu
BOUNDS = 8


def make_case(reqs, Hq, Hkv, D, seed=0, extra_rows=3, q_gap=0):
    """reqs: (n, kv, noisy, hidden).  Pages in random order; every slot that no
    row may see (page tails, hidden slots, unused pages) holds NaN."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-kv // 64) for _, kv, _, _ in reqs]
    n_pages, max_pages = sum(held) + 3, max(1, max(held)) + 1
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((len(reqs), max_pages), -1, dtype=torch.int32)
    kp = torch.randn(n_pages, Hkv, 64, D, generator=g).to(torch.bfloat16)
    vp = torch.randn(n_pages, Hkv, D, 64, generator=g).to(torch.bfloat16)
    live = torch.zeros(n_pages, 64, dtype=torch.bool)
    at = 0
    for b, (n, kv, noisy, hid) in enumerate(reqs):
        table[b, :held[b]] = perm[at:at + held[b]].to(torch.int32)
        s = torch.arange(min(max(hid, 0), kv), kv)
        live[table[b].long()[s // 64], s % 64] = True
        at += held[b]
    kp.transpose(1, 2)[~live] = float("nan")
    vp.permute(0, 3, 1, 2)[~live] = float("nan")
    rows = sum(r[0] for r in reqs)
    q = torch.randn(rows + extra_rows, Hq * D + q_gap, generator=g).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum([r[0] for r in reqs])])
    return dict(q=q, kp=kp, vp=vp, table=table, cu=cu, n_pages=n_pages, max_pages=max_pages, rows=rows, reqs=reqs,
                Hq=Hq, Hkv=Hkv, D=D)


def launch(cuda, c, scale=None, masks=True, lse=True, ws=None, out=None, stream=None):
    n_rows = c["q"].shape[0]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    i32 = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device=cuda)
    out = torch.full((n_rows, Hq, D), 7.0, dtype=torch.bfloat16, device=cuda) if out is None else out
    ls = torch.full((n_rows, Hq), 7.0, device=cuda) if lse else None
    if ws is None:      # any contents will do
        ws = torch.full_like(ws_tensor(dv.chunk_attn_paged_workspace_size(len(c["reqs"]), n_rows, Hq, Hkv, D), cuda), -1)
    st = status(cuda)
    qd = c["q"].to(cuda)
    dv.chunk_attn_paged(qd[:, :Hq * D], out, c["kp"].to(cuda), c["vp"].to(cuda), c["table"].to(cuda),
                        i32([r[1] for r in c["reqs"]]), i32(c["cu"]), n_batch=len(c["reqs"]), n_rows=n_rows,
                        n_pages=c["n_pages"], max_pages=c["max_pages"], Hq=Hq, Hkv=Hkv, D=D,
                        scale=D ** -0.5 if scale is None else scale, workspace=ws,
                        n_noisy=i32([r[2] for r in c["reqs"]]) if masks else None,
                        n_hidden=i32([r[3] for r in c["reqs"]]) if masks else None, lse=ls, status=st, stream=stream)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None, int(st.item())


def check(c, out, lse, scale=None, rows_of=None):
    D, Hq = c["D"], c["Hq"]
    scale = D ** -0.5 if scale is None else scale
    q = c["q"][:, :Hq * D].double().numpy().reshape(-1, Hq, D)
    kp, vp = np.nan_to_num(c["kp"].double().numpy()), np.nan_to_num(c["vp"].double().numpy())
    for b, (n, kv, noisy, hid) in enumerate(c["reqs"]):
        if n == 0 or (rows_of is not None and b not in rows_of):
            continue
        at = int(c["cu"][b])
        noisy, hid = min(max(noisy, 0), n), min(max(hid, 0), kv)
        args = (c["table"][b].tolist(), kv, noisy, hid, scale)
        want, wlse = ref.chunk_attention(q[at:at + n], kp, vp, *args)
        mag, _ = ref.chunk_attention(q[at:at + n], kp, np.abs(vp), *args)
        got = out[at:at + n]
        bound = mag * (2.0 ** -8 + 2.0 ** -12) + (np.abs(want) + mag * 2.0 ** -8) * 2.0 ** -8
        err = np.abs(got - want)
        assert (err <= bound).all(), (b, float(np.nanmax(err - bound)), np.argwhere(~(err <= bound))[:4].tolist())
        if lse is not None:
            assert (np.isneginf(lse[at:at + n]) == np.isneginf(wlse)).all()
            seen = ~np.isneginf(wlse)
            assert (np.abs(lse[at:at + n][seen] - wlse[seen]) <= 2e-4).all()
    assert (out[c["rows"]:] == 7.0).all()      # rows behind the last request are left as they were


HEADS = [(16, 2, 128), (8, 1, 128), (14, 2, 64), (8, 8, 128), (12, 4, 64), (5, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("reqs", [
    [(1, 1, 0, 0)], [(1, 64, 0, 0)], [(1, 65, 1, 0)], [(1, 128, 0, 0)], [(1, 129, 0, 3)], [(16, 16, 16, 0)],
    [(16, 200, 16, 0)], [(5, 300, 2, 0)], [(17, 17, 0, 0)], [(33, 700, 0, 0)],
], ids=lambda r: "_".join(map(str, r[0])))
def test_single_request(cuda, reqs, Hq, Hkv, D):
    c = make_case(reqs, Hq, Hkv, D)
    out, lse, st = launch(cuda, c)
    assert st == 0
    check(c, out, lse)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS + [(128, 1, 64), (130, 2, 128)])
def test_ragged_batch(cuda, Hq, Hkv, D):
    """Single tokens, blocks, chunks, idle requests, noisy tails, hidden prefixes, rows that see nothing."""
    reqs = [(1, 777, 0, 0), (0, 50, 0, 0), (16, 130, 16, 0), (40, 40, 0, 0), (7, 400, 3, 0), (0, 0, 0, 0),
            (1, 64, 0, 64), (20, 90, 0, 80), (9, 300, 9, 200), (65, 66, 0, 1), (3, 1000, 0, 128), (2, 513, 1, 512),
            (10, 10, 0, 10), (6, 70, 6, 70), (12, 140, 99, -5)]
    c = make_case(reqs, Hq, Hkv, D, seed=1, q_gap=16)
    out, lse, st = launch(cuda, c)
    assert st == 0
    check(c, out, lse)
    assert (out[c["cu"][12]:c["cu"][14]] == 0).all()


@pytest.mark.parametrize("Hq,Hkv,D,reqs", [
    (16, 2, 128, [(300, 1000, 0, 0)]), (16, 2, 128, [(257, 257, 0, 0), (1, 4000, 0, 0)]),
    (14, 2, 64, [(400, 900, 30, 130)]), (8, 8, 64, [(500, 500, 0, 0)]), (4, 1, 128, [(700, 1300, 0, 650)]),
    (2, 2, 128, [(1000, 1111, 1000, 0)]), (8, 1, 128, [(1, 30000, 0, 0)]), (16, 2, 128, [(16, 9000, 16, 0)])])
def test_chunks_and_long_caches(cuda, Hq, Hkv, D, reqs):
    """Several tiles per request, work split over many CTAs and merged."""
    c = make_case(reqs, Hq, Hkv, D, seed=2)
    out, lse, st = launch(cuda, c)
    assert st == 0
    check(c, out, lse)


def test_many_requests(cuda):
    """More requests than threads of a CTA; whole and cut items side by side."""
    rng = np.random.default_rng(5)
    reqs = []
    for _ in range(700):
        n = int(rng.choice([0, 1, 1, 1, 4]))
        L = int(rng.integers(0, 300))
        reqs.append((n, n + L, int(rng.integers(0, n + 1)), 0))
    c = make_case(reqs, 8, 2, 64, seed=3)
    out, lse, st = launch(cuda, c)
    assert st == 0
    check(c, out, lse, rows_of=set(range(0, 700, 9)) | {699})


def test_peaked_and_growing_scores(cuda):
    """Large scores, and maxima that grow along the cache (the reference maximum moves often)."""
    c = make_case([(20, 900, 0, 0), (1, 1500, 0, 0)], 8, 1, 128, seed=4)
    for b in range(2):
        kv = c["reqs"][b][1]
        s = torch.arange(kv)
        page = c["table"][b].long()[s // 64]
        c["kp"][page, :, s % 64] *= (s.float() / 200).to(torch.bfloat16)[:, None, None]
    out, lse, st = launch(cuda, c)
    assert st == 0
    scale = 128 ** -0.5
    q = c["q"].double().numpy().reshape(-1, 8, 128)
    kp, vp = np.nan_to_num(c["kp"].double().numpy()), np.nan_to_num(c["vp"].double().numpy())
    for b, (n, kv, noisy, hid) in enumerate(c["reqs"]):
        at = int(c["cu"][b])
        want, wl = ref.chunk_attention(q[at:at + n], kp, vp, c["table"][b].tolist(), kv, 0, 0, scale)
        mag, _ = ref.chunk_attention(q[at:at + n], kp, np.abs(vp), c["table"][b].tolist(), kv, 0, 0, scale)
        # keys up to 7.5 x: scores' fp32 error up to 7.5 times the docstring's 1e-4
        bound = mag * (2.0 ** -8 + 2 * 7.5e-4) + (np.abs(want) + mag * 2.0 ** -8) * 2.0 ** -8
        assert (np.abs(out[at:at + n] - want) <= bound).all()
        assert (np.abs(lse[at:at + n] - wl) <= 1e-3).all()


def test_no_masks_and_same_bits(cuda):
    """NULL noisy / hidden mean zero; a second call, and one in a captured graph on another stream, give the same bits."""
    reqs = [(16, 500, 0, 0), (1, 3000, 0, 0), (130, 300, 0, 0)]
    c = make_case(reqs, 16, 2, 128, seed=6)
    a, la, st = launch(cuda, c)
    b, lb, st2 = launch(cuda, c, masks=False)
    assert st == st2 == 0 and np.array_equal(a, b) and np.array_equal(la, lb)
    check(c, a, la)
    i32 = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device=cuda)
    n_rows = c["q"].shape[0]
    out = torch.full((n_rows, 16, 128), 7.0, dtype=torch.bfloat16, device=cuda)
    ws = ws_tensor(dv.chunk_attn_paged_workspace_size(3, n_rows, 16, 2, 128), cuda)
    t = [c["q"].to(cuda), c["kp"].to(cuda), c["vp"].to(cuda), c["table"].to(cuda), i32([r[1] for r in reqs]), i32(c["cu"])]
    st = status(cuda)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dv.chunk_attn_paged(t[0], out, *t[1:], n_batch=3, n_rows=n_rows, n_pages=c["n_pages"],
                            max_pages=c["max_pages"], Hq=16, Hkv=2, D=128, scale=128 ** -0.5, workspace=ws, status=st)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
    assert_ok(st)
    assert np.array_equal(out.double().cpu().numpy(), a)


def test_bad_requests_take_no_part(cuda):
    """Lengths that do not fit and page numbers outside the store are reported; the other requests' rows are right."""
    reqs = [(4, 100, 0, 0), (5, 60, 0, 0), (3, 200, 0, 0), (2, 70, 0, 0)]
    for what in ("kv_short", "kv_long", "kv_negative", "cu_down", "cu_past", "page"):
        c = make_case(reqs, 8, 1, 128, seed=7)
        kv = [r[1] for r in reqs]
        left = [7.0]
        if what == "kv_short":
            kv[1] = 4
        elif what == "kv_long":
            kv[1] = c["max_pages"] * 64 + 1
        elif what == "kv_negative":
            kv[1] = -60
        elif what == "cu_down":
            c["cu"][2] = 3
        elif what == "cu_past":
            c["cu"][4] = 10 ** 6
        else:
            c["table"][1, 0] = c["n_pages"] + 3
            c["kp"], c["vp"] = torch.nan_to_num(c["kp"]), torch.nan_to_num(c["vp"])
        # cu_down: request 2 then owns rows 3 .. 11, row 3 of request 0 among them
        good = {"cu_down": {3}, "cu_past": {0, 1, 2}}.get(what, {0, 2, 3})
        full = c["reqs"]
        c["reqs"] = [(r[0], k, r[2], r[3]) for r, k in zip(full, kv)]
        out, lse, st = launch(cuda, c)
        c["reqs"] = full
        assert st == BOUNDS, what
        if what == "cu_down":
            c["reqs"] = [full[0], (0, 0, 0, 0), (0, 0, 0, 0), full[3]]
        if what == "cu_past":
            c["reqs"] = full[:3]
        c["rows"] = out.shape[0]
        check(c, out, lse, rows_of=good)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv,n", [(16, 1, 1), (15, 2, 1), (17, 1, 1), (8, 2, 2), (8, 1, 3), (1, 3, 16), (1, 2, 17),
                                     (5, 2, 3), (5, 2, 4), (2, 1, 9)])
def test_few_rows(cuda, G, Hkv, n, D):
    """Rows times heads at and around 16 (products of 64 rows), alone, behind whole tiles, and cut over many CTAs; a
    maximum that moves late."""
    tile = 2 * (128 // G)
    reqs = [(n, 700, 0, 0), (n, 64 * 3, n, 65), (n, n, 0, 0), (n, 5000, 0, 130), (tile + n, 400 + tile, 1, 0)]
    c = make_case(reqs, G * Hkv, Hkv, D, seed=n + G)
    out, lse, st = launch(cuda, c)
    assert st == 0
    check(c, out, lse)
    out, lse, st = launch(cuda, c, scale=3.0 * D ** -0.5)
    assert st == 0
    check(c, out, lse, scale=3.0 * D ** -0.5)
