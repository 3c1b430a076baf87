"""The batched paged step around requests that take no rows, and at the edges
of its page numbers, drafts and values, against the plain 64-bit definitions
(step_reference.py).  Integers are equal; attention is held to the bound of
test_gpu_chunk_attn.py."""
import numpy as np
import pytest
import torch

import block_diffusion_vlm_b200 as dv
import step_reference as ref
from gpu_util import assert_ok, status
from test_gpu_chunk_attn import check, launch, make_case
from test_gpu_step import run_verify
from test_gpu_step_run import Server, host

pytestmark = pytest.mark.gpu
OVERFLOW, BOUNDS = 4, 8


def i32(v, dev):
    return torch.tensor(np.asarray(v, dtype=np.int32), device=dev)


# ------------------------------------------------- requests without rows in a step
class StepServer(Server):
    """A server whose verification knows which requests got rows."""

    def step(self, verify, n_draft=True):
        super().step(False)                     # (the cache then counts every new row)
        if verify:
            dv.spec_verify_sample(self.p, None, self.ids, self.u, self.us, b=self.n, K=self.K, V=self.V,
                                  dtype=dv.DVLM_FP32, accept_len=self.acc, out_ids=self.tok,
                                  n_draft=self.nd if n_draft else None, cache_len=self.kv, cache_len_out=self.cache,
                                  cu_rows=self.cu, status=self.st)


def check_verified(s, n_draft):
    """Tokens, accepted lengths and cut caches of a step; returns the requests that ran."""
    cu, kv, acc, tok, cut = host(s.cu), host(s.kv), host(s.acc), host(s.tok), host(s.cache)
    ran = []
    for b in range(s.n):
        rows = int(cu[b + 1] - cu[b])
        if rows == 0:
            assert (acc[b], tok[b].tolist(), cut[b]) == (0, [-1] * (s.K + 1), kv[b]), b
            continue
        ran.append(b)
        nd = min(n_draft[b], rows)
        k, ids, bad = ref.verify(host(s.p[b]).astype(np.float64), None, host(s.ids[b]).tolist(),
                                 host(s.u[b]).astype(np.float64), float(s.us[b]), nd)
        assert (acc[b], tok[b].tolist(), cut[b]) == (k, ids, kv[b] - (nd - k)) and not bad, b
    return ran


@pytest.mark.parametrize("graph", [False, True])
def test_requests_without_rows_keep_their_caches(cuda, graph):
    """Waiting, idle, finished and refused requests beside drafted ones: no token, no cut, no matter what n_draft says;
    the waiting one goes on with its whole cache once another's pages come back."""
    s = StepServer(cuda, n=6, max_pages=3, n_pages=10, max_rows=460)
    put = lambda t, v: t.copy_(i32(v, cuda))
    put(s.new, [60, 50, 20, 192, 63, 64])        # 1 + 1 + 1 + 3 + 1 + 1 pages of 10
    s.fill()
    s.step(False)
    assert_ok(s.st)
    if graph:
        s.nd.fill_(6)
        s.new.zero_()
        s.step(True)                             # (warm-up: nothing runs, nothing changes)
        assert_ok(s.st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step(True)

    def step(new, n_draft, st):
        put(s.new, new)
        put(s.nd, n_draft)
        s.fill()
        s.st.zero_()
        before, table, held = host(s.cache), host(s.table), host(s.held)
        stack = host(s.free)[:int(s.count)].tolist()
        g.replay() if graph else s.step(True)
        torch.cuda.synchronize()
        assert int(s.st) in st
        want = ref.page_plan(before, new, table, stack, s.max_pages, s.n_pages, s.max_rows, held)
        for got, w in zip((s.kv, s.cu, s.slots, s.table), want):
            np.testing.assert_array_equal(host(got), w)
        return check_verified(s, n_draft)

    # two pages are left: the first three need one between them (60 + 6), then 3 is refused (192 + 1 slots), 4 takes
    # the last page and 5 (64 + 6) waits
    ran = step([6, 6, 0, 1, 6, 6], [6, 6, 6, 6, 6, 6], (OVERFLOW, BOUNDS))
    assert ran == [0, 1, 4]
    assert host(s.cache)[[2, 3, 5]].tolist() == [20, 192, 64] and int(s.count) == 0
    # 3 finishes (its three pages come back), 5 goes on with all of its cache; one row holds no second draft
    ran = step([0, 0, 1, -1, 0, 6], [6, 6, 0, 6, 6, 6], (0,))
    assert ran == [2, 5] and host(s.kv)[[3, 5]].tolist() == [0, 70] and host(s.cache)[3] == 0
    # more drafts than rows: cut to the rows, and said so
    ran = step([0, 2, 0, 0, 0, 0], [6, 6, 6, 6, 6, 6], (BOUNDS,))
    assert ran == [1]


def test_verify_without_draft_counts(cuda):
    """n_draft NULL means K for the sequences that ran; rows that descend count as none."""
    s = StepServer(cuda, n=4, max_pages=2, n_pages=8, max_rows=64)
    s.fill()
    s.kv.copy_(i32([30, 40, 50, 60], cuda))
    for cu, st in (([0, 6, 6, 13, 20], 0), ([0, 6, 4, 13, 16], BOUNDS)):
        s.cu.copy_(i32(cu, cuda))
        s.st.zero_()
        dv.spec_verify_sample(s.p, None, s.ids, s.u, s.us, b=4, K=6, V=s.V, dtype=dv.DVLM_FP32, accept_len=s.acc,
                              out_ids=s.tok, cache_len=s.kv, cache_len_out=s.cache, cu_rows=s.cu, status=s.st)
        torch.cuda.synchronize()
        assert int(s.st) == st
        got = host(s.cu)
        s.cu.copy_(torch.cat([s.cu[:1], s.cu[:1] + torch.cumsum((s.cu[1:] - s.cu[:-1]).clamp(min=0), 0)]))
        assert check_verified(s, [6] * 4) == [b for b in range(4) if got[b + 1] > got[b]]


@pytest.mark.parametrize("with_held", [False, True])
@pytest.mark.parametrize("bad", [-2, -2 ** 31])
def test_a_bad_new_length_loses_no_cache_in_place(cuda, with_held, bad):
    """kv_len in cache_len's place: a request refused for its new length keeps its length, and gives all of its pages
    back when it finishes; beside it the others go on."""
    n, max_pages, n_pages = 3, 4, 12
    table = np.full((n, max_pages), -1, dtype=np.int32)
    table[0, :2], table[1, :3] = [3, 5], [7, 8, 9]
    free = np.zeros(n_pages, dtype=np.int32)
    free[:7] = [0, 1, 2, 4, 6, 10, 11]
    t, f, count, st = i32(table, cuda), i32(free, cuda), i32([7], cuda), status(cuda)
    cache, held = i32([100, 150, 0], cuda), i32([100, 190, 0], cuda) if with_held else None
    cu, slots = i32([0] * (n + 1), cuda), i32([0] * 70, cuda)

    def plan(new):
        st.zero_()
        dv.page_plan(cache, i32(new, cuda), t, f, count, n_batch=n, max_pages=max_pages, n_pages=n_pages, max_rows=70,
                     kv_len=cache, cu_rows=cu, slot_map=slots, free_count_out=count, held_len=held, status=st)
        torch.cuda.synchronize()
        return int(st)

    assert plan([10, bad, 5]) == BOUNDS
    assert host(cache).tolist() == [110, 150, 5] and host(cu).tolist() == [0, 10, 10, 15] and int(count) == 6
    assert plan([0, -1, 0]) == 0
    assert host(cache).tolist() == [110, 0, 5] and int(count) == 9
    assert sorted(host(f)[:9].tolist() + [3, 5, int(host(t)[2, 0])]) == list(range(12))


# ----------------------------------------------------------------- page numbers
def plan_of(cuda, cache, new, table, stack, n_pages, max_rows):
    n, max_pages = np.shape(table)
    free = np.zeros(n_pages, dtype=np.int32)
    free[:len(stack)] = stack
    t = i32(table, cuda)
    kv, cu, slots, count, st = i32([0] * n, cuda), i32([0] * (n + 1), cuda), i32([0] * max_rows, cuda), \
        i32([len(stack)], cuda), status(cuda)
    dv.page_plan(i32(cache, cuda), i32(new, cuda), t, i32(free, cuda), count, n_batch=n, max_pages=max_pages,
                 n_pages=n_pages, max_rows=max_rows, kv_len=kv, cu_rows=cu, slot_map=slots, free_count_out=count,
                 status=st)
    assert_ok(st)
    return slots, t


def append_status(cuda, slots, rows, n_pages):
    """Status of an append of `rows` rows of ones; the rows of q that were written."""
    D = 64
    bf = dict(dtype=torch.bfloat16, device=cuda)
    q, st = torch.zeros(rows, 2, D, **bf), status(cuda)
    dv.mrope_append_paged(torch.ones(rows, 4 * D, **bf), i32(np.zeros((1, rows)), cuda), slots, q,
                          torch.zeros(n_pages, 1, 64, D, **bf), torch.zeros(n_pages, 1, D, 64, **bf), n_rows=rows,
                          Hq=2, Hkv=1, D=D, n_pages=n_pages, sections=(32,), rope_base=1e4, status=st)
    torch.cuda.synchronize()
    return int(st), (q != 0).all(dim=(1, 2)).cpu().tolist()


@pytest.mark.parametrize("wild", [-1, -2, -3, -2 ** 25, 4, 2 ** 25])
def test_no_live_row_looks_like_padding(cuda, wild):
    """A table entry or a stack entry that is no page (-1: the usual filler) gives slots that the append reports, the
    last of the page too (slot -1 is padding: skipped without a word)."""
    slots, _ = plan_of(cuda, [0], [64], [[-7]], [wild], 4, 66)       # off the stack
    got = host(slots)
    assert got[64:].tolist() == [-1, -1] and ((got[:64] >= 4 * 64) | (got[:64] < -1)).all()
    assert (got[:64].astype(np.int64) % 64 == np.arange(64)).all()
    for at in (0, 40, 63):                                           # a cached page, one row alone
        slots, table = plan_of(cuda, [at], [1], [[wild if at else -7]], [] if at else [wild], 4, 1)
        assert host(table).tolist() == [[wild]]                      # the table keeps what it was given
        st, written = append_status(cuda, slots, 1, 4)
        assert st == BOUNDS and written == [False], at
    # the next request's rows are right all the same
    slots, _ = plan_of(cuda, [63, 63], [1, 1], [[wild], [2]], [], 4, 3)
    assert host(slots)[1:].tolist() == [2 * 64 + 63, -1]
    st, written = append_status(cuda, slots, 3, 4)
    assert st == BOUNDS and written == [False, True, False]


# ------------------------------------------------------- slots that no row may see
@pytest.mark.parametrize("D", [64, 128])
def test_stale_values_beside_two_tiles(cuda, D):
    """Pairs of row tiles whose first or last page is partly outside the cache, with NaN there (one tile's warps clear
    V for both): hidden prefixes and ends at every kind of place, rows that see only such a page, again and again."""
    reqs = [(256, 256 + kv, noisy, hid) for kv, noisy, hid in ((1, 0, 0), (63, 0, 63), (7, 256, 5), (130, 40, 129),
                                                               (0, 0, 200), (300, 0, 1), (65, 256, 320), (64, 0, 64))]
    c = make_case(reqs, 8, 1, D, seed=21)
    out0, lse0, st = launch(cuda, c)
    assert st == 0
    check(c, out0, lse0, rows_of={0, 1, 3, 6})
    assert np.isfinite(out0).all()
    for _ in range(20):
        out, lse, st = launch(cuda, c)
        assert st == 0 and np.array_equal(out, out0) and np.array_equal(lse, lse0)


# ------------------------------------------------------ values that are no numbers
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 128), (14, 2, 64), (8, 8, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries_that_are_no_numbers(cuda, Hq, Hkv, D, bad):
    """A query with a NaN, or with an infinity (scores of both signs: inf - inf), gives NaN and not 0, which stands for
    a row that sees nothing; the other rows and heads keep their bits.  Whole tiles, pairs of tiles, single tokens, and
    items cut over many CTAs."""
    reqs = [(1, 300, 0, 0), (16, 130, 16, 0), (40, 40, 0, 0), (300, 900, 0, 0), (1, 9000, 0, 0), (16, 7000, 16, 0),
            (4, 70, 0, 70)]
    c = make_case(reqs, Hq, Hkv, D, seed=11)
    out0, lse0, st = launch(cuda, c)
    assert st == 0
    rows = [int(c["cu"][b]) + t for b, t in ((0, 0), (1, 7), (2, 39), (3, 0), (3, 171), (3, 299), (4, 0), (5, 3))]
    head = Hq - 1
    for r in rows:
        c["q"][r, head * D + 5] = bad
    hidden = int(c["cu"][6])                                          # a row that sees nothing is 0 whatever it holds
    c["q"][hidden, head * D + 5] = bad
    out, lse, st = launch(cuda, c)
    assert st == 0
    assert np.isnan(out[rows, head]).all() and np.isnan(lse[rows, head]).all()
    assert (out[hidden:hidden + 4] == 0).all() and np.isneginf(lse[hidden:hidden + 4]).all()
    keep = np.ones(out.shape[:2], dtype=bool)
    keep[rows, head] = False
    assert np.array_equal(out[keep], out0[keep]) and np.array_equal(lse[keep], lse0[keep])


# ------------------------------------------------------------------------ drafts
@pytest.mark.parametrize("K", [3, 31, 33, 64])
def test_drafts_behind_a_refused_one_are_not_looked_at(cuda, K):
    """Ids outside the vocabulary are reported where the verification gets to them, and not behind a refused draft."""
    V, b = 96, 4
    p = torch.full((b, K + 1, V), 1.0 / V)
    ids, u = np.full((b, K), 7), np.zeros((b, K), dtype=np.float32)
    u[0, 0], u[1, K - 2] = 1.0, 1.0                     # sequences 0 and 1 refuse a draft; 2 and 3 take every one
    p[:2, :, 7] = 0.0
    p[1, :K - 2, 7] = 1.0 / V
    for bad in ([(0, 1)], [(0, K - 1), (1, K - 1)], [(0, j) for j in range(1, K)]):
        x = ids.copy()
        for i, j in bad:
            x[i, j] = -1 if j % 2 else V
        for q in (None, torch.full((b, K, V), 1.0 / V)):
            acc, out, _, st = run_verify(cuda, p, q, x, u, np.full(b, 0.25))
            assert st == 0 and acc.tolist() == [0, K - 2, K, K], bad
    for i, j in ((2, K - 1), (3, 0), (1, K - 2), (0, 0)):               # reached: reported
        x = ids.copy()
        x[i, j] = V + 3
        acc, out, _, st = run_verify(cuda, p, None, x, u, np.full(b, 0.25))
        assert st == BOUNDS and acc[i] == j
        k, want, bad = ref.verify(p[i].double().numpy(), None, x[i].tolist(), u[i].astype(np.float64), 0.25, K)
        assert bad and out[i].tolist() == want


def test_a_request_alone_and_in_a_batch(cuda):
    """The other requests move the cuts of a request's work and with them the reference maxima against which P is
    rounded: alone and in any batch a row keeps to the bound around its exact value, so the two are within twice that
    bound of each other (they are not the same bits)."""
    Hq, Hkv, D = 16, 2, 128
    mine = [(16, 900, 16, 0), (1, 5000, 0, 0), (200, 700, 0, 100)]
    other = [(1, 3000, 0, 0), (300, 2000, 0, 0), (16, 64, 16, 0), (33, 1500, 0, 0)]
    c = make_case(mine + other, Hq, Hkv, D, seed=12)
    outs = []
    for take in ([0], [1], [2], [0, 1, 2], list(range(7))):
        part = dict(c, reqs=[c["reqs"][b] for b in take], table=c["table"][take])
        part["q"] = torch.cat([c["q"][c["cu"][b]:c["cu"][b + 1]] for b in take] + [c["q"][-3:]])
        part["cu"] = np.concatenate([[0], np.cumsum([r[0] for r in part["reqs"]])])
        part["rows"] = int(part["cu"][-1])
        out, lse, st = launch(cuda, part)
        assert st == 0
        check(part, out, lse)                              # each within the bound of the exact value
        outs.append({b: out[part["cu"][i]:part["cu"][i + 1]] for i, b in enumerate(take)})
    kp, vp = np.nan_to_num(c["kp"].double().numpy()), np.nan_to_num(c["vp"].double().numpy())
    for b in range(3):
        n, kv, noisy, hid = c["reqs"][b]
        q = c["q"][c["cu"][b]:c["cu"][b + 1]].double().numpy().reshape(n, Hq, D)
        args = (c["table"][b].tolist(), kv, noisy, hid, D ** -0.5)
        want, _ = ref.chunk_attention(q, kp, vp, *args)
        mag, _ = ref.chunk_attention(q, kp, np.abs(vp), *args)
        one = mag * (2.0 ** -8 + 2.0 ** -12) + (np.abs(want) + mag * 2.0 ** -8) * 2.0 ** -8
        for o in outs[3:]:
            assert (np.abs(o[b] - outs[b][b]) <= 2 * one).all()


# --------------------------------------------------------------- batches together
def test_two_batches_at_once_all_steps(cuda):
    """Two batches, each on its own stream with its own workspace, through steps that all fit: the same lengths,
    tokens, attention, log-sum-exp and page stores as one by one, and no error."""
    def make():
        out = []
        for seed, new in ((1, [100, 1, 17]), (2, [3, 90, 64])):
            s = StepServer(cuda, n=3, max_pages=12, n_pages=30, max_rows=300, seed=seed)
            s.new.copy_(i32(new, cuda))
            s.nd.copy_(i32([3, 1, 0], cuda))
            s.fill()
            out.append(s)
        return out

    alone, both = make(), make()
    torch.cuda.synchronize()
    for s in alone:
        for _ in range(6):
            s.step(True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(6):
        for s, stream in zip(both, streams):
            with torch.cuda.stream(stream):
                s.step(True)
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        assert_ok(x.st)
        assert_ok(y.st)
        assert torch.equal(x.cu[1:] - x.cu[:-1], x.new)               # every request had its rows in the last step too
        for k in ("kv", "cache", "held", "table", "slots", "free", "count", "acc", "tok", "lse"):
            assert torch.equal(getattr(x, k), getattr(y, k)), k
        for k in ("q", "out", "kp", "vp"):
            assert torch.equal(getattr(x, k).view(torch.int16), getattr(y, k).view(torch.int16)), k


@pytest.mark.parametrize("dtype,V", [(torch.float32, 151936), (torch.bfloat16, 50257)])
@pytest.mark.parametrize("b", [1, 5])
def test_sequences_without_rows_among_large_vocabularies(cuda, dtype, V, b):
    """Several CTAs a sequence: the ones that have nothing to do leave, the others' tokens are right."""
    K = 4
    g = torch.Generator().manual_seed(b)
    p = torch.softmax(2.0 * torch.randn(b, K + 1, V, generator=g), -1).to(dtype)
    q = torch.softmax(2.0 * torch.randn(b, K, V, generator=g), -1).to(dtype)
    ids, u, us = torch.randint(0, V, (b, K), generator=g), torch.rand(b, K, generator=g), torch.rand(b, generator=g)
    for rows in ([0] * b, [5] * b, [5 * (i % 2) for i in range(b)]):
        acc, tok, cache, st = i32([9] * b, cuda), i32([[9] * (K + 1)] * b, cuda), i32([100] * b, cuda), status(cuda)
        dv.spec_verify_sample(p.to(cuda), q.to(cuda), ids.to(torch.int32).to(cuda), u.to(cuda), us.to(cuda), b=b, K=K,
                              V=V, dtype=dv.DVLM_FP32 if dtype == torch.float32 else dv.DVLM_BF16, accept_len=acc,
                              out_ids=tok, cache_len=cache, cache_len_out=cache,
                              cu_rows=i32(np.concatenate([[0], np.cumsum(rows)]), cuda), status=st)
        assert_ok(st)
        for i in range(b):
            want = (0, [-1] * (K + 1), 100)
            if rows[i]:
                k, out, bad = ref.verify(p[i].double().numpy(), q[i].double().numpy(), ids[i].tolist(),
                                         u[i].double().numpy(), float(us[i]), K)
                assert not bad
                want = (k, out, 100 - (K - k))
            assert (int(acc[i]), tok[i].tolist(), int(cache[i])) == want
