"""The batched paged step's operators on the GPU against their plain 64-bit
definitions (step_reference.py): the page plan (integers: equal), multi-axis
rotary positions alone and with the paged write, verification by rejection
sampling (integers: equal).

Tolerances.  Rotary rows: the angle is reduced in fp64 (absolute error below
1e-9 radians at the positions used), its cosine and sine carry at most 2 fp32
ulps (2^-22 relative to 1), the two products and the sum at most three fp32
roundings: |error| <= (|x_j| + |x_j'|) * (2^-22 + 2 * 2^-24) before the
store; the store rounds once, half a step of the type (2^-8 relative for
bf16's 8 bits, finfo.eps / 2; fp32 2^-24)."""
import numpy as np
import pytest
import torch

import block_diffusion_vlm_b200 as dv
import step_reference as ref
from gpu_util import assert_ok, status

pytestmark = pytest.mark.gpu
OVERFLOW, BOUNDS = 4, 8


def i32(a, dev):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=dev)


# ------------------------------------------------------------------ page plan
def run_plan(cuda, cache, new, table, stack, n_pages, max_rows, in_place=False, offset=0, stream=None, held=None):
    n, max_pages = table.shape
    free = np.full(n_pages, -7, dtype=np.int32)
    free[:len(stack)] = stack
    d = dict(cache=i32(cache, cuda), new=i32(new, cuda), table=i32(table, cuda), free=i32(free, cuda),
             count=i32([len(stack)], cuda))
    kv = d["cache"] if in_place else i32([-9] * n, cuda)
    co = d["count"] if in_place else i32([-9], cuda)
    cu = i32([-9] * (n + 1), cuda)
    slots = torch.full((max_rows + offset,), -9, dtype=torch.int32, device=cuda)[offset:]
    st, hd = status(cuda), i32(held, cuda) if held is not None else None
    dv.page_plan(d["cache"], d["new"], d["table"], d["free"], d["count"], n_batch=n, max_pages=max_pages,
                 n_pages=n_pages, max_rows=max_rows, kv_len=kv, cu_rows=cu, slot_map=slots, free_count_out=co,
                 held_len=hd, status=st, stream=stream)
    torch.cuda.synchronize()
    got = [t.cpu().numpy() for t in (kv, cu, slots, d["table"], d["free"], co)] + [int(st.item())]
    return got + [hd.cpu().numpy() if hd is not None else None]


def check_plan(cuda, cache, new, table, stack, n_pages, max_rows, held=None, **kw):
    want = ref.page_plan(cache, new, table, stack, table.shape[1], n_pages, max_rows, held)
    kv, cu, slots, tab, free, count, st, hd = run_plan(cuda, cache, new, table, stack, n_pages, max_rows, held=held, **kw)
    if held is not None:
        np.testing.assert_array_equal(hd, want[7])
    np.testing.assert_array_equal(kv, want[0])
    np.testing.assert_array_equal(cu, want[1])
    np.testing.assert_array_equal(slots, want[2])
    np.testing.assert_array_equal(tab, want[3])
    assert int(count[0]) == len(want[4])
    np.testing.assert_array_equal(free[:len(want[4])], want[4][:len(free)])
    if len(stack) > len(want[4]):            # entries above the new top keep what they held
        np.testing.assert_array_equal(free[len(want[4]):len(stack)], stack[len(want[4]):])
    if not want[5] and not want[6]:
        assert st == 0
    else:
        assert st in ([OVERFLOW] if want[5] else []) + ([BOUNDS] if want[6] else [])


def plan_case(rng, n, max_pages, max_new, spare, finished=True):
    cache = rng.integers(0, max_pages * 64 + 1, n)
    new = np.array([rng.choice([-1 if finished else 0, 0, 1, 16, int(rng.integers(0, max_new + 1))]) for _ in range(n)])
    new = np.where(cache + new > max_pages * 64, np.minimum(new, 0), new)
    held = -(-cache // 64)
    n_pages = int(held.sum()) + spare
    perm = rng.permutation(n_pages)
    table = np.full((n, max_pages), -1, dtype=np.int32)
    at = 0
    for b in range(n):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    return cache, new, table, perm[at:].tolist(), n_pages


@pytest.mark.parametrize("n,max_pages,max_new,spare,rows", [
    (1, 1, 1, 1, 1), (1, 3, 130, 3, 200), (7, 5, 64, 40, 450), (33, 9, 257, 300, 9000), (1000, 4, 16, 900, 16001),
    (1025, 3, 16, 900, 12000), (4096, 2, 40, 3000, 8191), (4096, 2, 40, 3000, 70000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_plan(cuda, n, max_pages, max_new, spare, rows, in_place):
    for seed in range(3):
        cache, new, table, stack, n_pages = plan_case(np.random.default_rng(seed), n, max_pages, max_new, spare)
        check_plan(cuda, cache, new, table, stack, n_pages, rows, in_place=in_place)


@pytest.mark.parametrize("n,rows", [(1, 64), (40, 3000), (300, 9000)])
def test_page_plan_after_a_cut(cuda, n, rows):
    """Caches cut back behind their last step keep their pages: none is taken twice, all go back at the end."""
    rng = np.random.default_rng(n)
    held, new, table, stack, n_pages = plan_case(rng, n, 6, 40, 60)
    cache = np.maximum(held - rng.integers(0, 90, n), 0)
    for h in (held, np.where(rng.random(n) < 0.3, -5, held)):      # a held length below the cached one counts as that
        check_plan(cuda, np.where(h < 0, held, cache), new, table, stack, n_pages, rows, held=h)
    bad = held.copy()
    bad[0] = 6 * 64 + 1
    check_plan(cuda, cache, new, table, stack, n_pages, rows, held=bad)
    # a run of steps: what the requests hold and the stack together stay the whole store
    stack = list(stack)
    for step in range(6):
        new = np.array([rng.choice([0, 1, 16, 30]) for _ in range(n)])
        new = np.where(cache + new > 6 * 64, 0, new)
        kv, cu, slots, table, free, count, st, held = run_plan(cuda, cache, new, table, stack, n_pages, rows, held=held)
        stack = free[:int(count[0])].tolist()
        owned = [int(p) for b in range(n) for p in table[b, :-(-int(held[b]) // 64)]]
        assert sorted(owned + stack) == list(range(n_pages))
        cache = np.maximum(kv - rng.integers(0, 14, n), 0)


def test_page_plan_waits_in_order(cuda):
    """Too few pages or rows: the first request that does not fit and all behind it add nothing."""
    rng = np.random.default_rng(2)
    for spare in (0, 1, 5, 20):
        cache, new, table, stack, n_pages = plan_case(rng, 40, 6, 150, spare, finished=spare == 5)
        check_plan(cuda, cache, new, table, stack, n_pages, 4000)
    cache, new, table, stack, n_pages = plan_case(rng, 40, 6, 150, 500)
    for rows in (1, 17, 333):
        check_plan(cuda, cache, new, table, stack, n_pages, rows)


def test_page_plan_bad_lengths(cuda):
    """Lengths outside the table take no part, the others go on; nothing is read or written out of range."""
    rng = np.random.default_rng(3)
    cache, new, table, stack, n_pages = plan_case(rng, 9, 4, 60, 60)
    cache[2], new[4], new[6] = -5, -3, 2 ** 31 - 1
    cache[7], new[7] = 2 ** 31 - 1, -1
    check_plan(cuda, cache, new, table, stack, n_pages, 1000, offset=1)
    # a count outside the stack is cut to it
    n, max_pages = table.shape
    for bad, kept in ((-4, 0), (n_pages + 9, n_pages)):
        st, co = status(cuda), i32([0], cuda)
        zero = i32([0] * n, cuda)
        dv.page_plan(zero, zero, i32(table, cuda), i32([0] * n_pages, cuda), i32([bad], cuda), n_batch=n,
                     max_pages=max_pages, n_pages=n_pages, max_rows=8, kv_len=i32([0] * n, cuda),
                     cu_rows=i32([0] * (n + 1), cuda), slot_map=i32([0] * 8, cuda), free_count_out=co, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == BOUNDS and int(co.item()) == kept


# ------------------------------------------------------------ rotary positions
def mrope_bound(x, want, half, rot, eps):
    """Per-element bound of the module's docstring."""
    mag = np.abs(x).astype(np.float64)
    pair = np.array(mag)
    pair[..., :half] = mag[..., :half] + mag[..., half:rot]
    pair[..., half:rot] = pair[..., :half]
    pair[..., rot:] = 0.0
    near = pair * (2.0 ** -22 + 2 * 2.0 ** -24) + 1e-30
    return near + (np.abs(want) + near) * (eps / 2)


ROPE_CASES = [
    # rows, heads, D, rot, sections, interleaved
    (1, 1, 2, 2, (1,), 0), (3, 5, 72, 72, (18, 18), 0), (33, 3, 80, 80, (20, 20), 1), (64, 2, 128, 128, (16, 24, 24), 0),
    (65, 4, 128, 128, (24, 20, 20), 1), (31, 7, 64, 32, (4, 6, 6), 0), (257, 1, 256, 256, (32, 32, 32, 32), 1),
    (100, 3, 66, 30, (5, 5, 5), 0), (5, 70, 128, 64, (0, 32, 0), 0), (2000, 2, 64, 64, (32,), 0),
    (6007, 2, 80, 80, (20, 20), 0), (12001, 1, 128, 64, (8, 12, 12), 1)]


@pytest.mark.parametrize("rows,heads,D,rot,sections,interleaved", ROPE_CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mrope(cuda, rows, heads, D, rot, sections, interleaved, dtype):
    g = torch.Generator().manual_seed(rows + D)
    x = torch.randn(rows, heads, D, generator=g).to(dtype)
    pos = torch.randint(-200, 200000, (len(sections), rows), generator=g, dtype=torch.int32)
    dt = dv.DVLM_BF16 if dtype == torch.bfloat16 else dv.DVLM_FP32
    xs = x.double().numpy()
    want = ref.mrope(xs, pos.numpy(), sections, 1e6, rot, interleaved)
    bound = mrope_bound(xs, want, rot // 2, rot, torch.finfo(dtype).eps)
    kw = dict(n_rows=rows, n_heads=heads, D=D, rot_dim=rot, sections=sections, rope_base=1e6, interleaved=interleaved,
              dtype=dt)
    xd, pd = x.to(cuda), pos.to(cuda)
    out = torch.full_like(xd, 9.0)
    dv.mrope(xd, out, pd, **kw)
    torch.cuda.synchronize()
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / bound).max())
    # rows of a wider buffer, at an odd element offset, in place: the same values, and nothing beside them changes
    wide = torch.full((rows, heads * D + 3), 5.0, dtype=dtype, device=cuda)
    view = wide[:, 1:1 + heads * D]
    view.copy_(xd.view(rows, -1))
    dv.mrope(view, view, pd, **kw)
    torch.cuda.synchronize()
    assert torch.equal(view.reshape(rows, heads, D), out)
    assert (wide[:, 0] == 5).all() and (wide[:, 1 + heads * D:] == 5).all()


@pytest.mark.parametrize("rows,Hq,Hkv,D,sections,rot,interleaved", [
    (1, 16, 2, 128, (16, 24, 24), 0, 0), (16, 8, 1, 128, (24, 20, 20), 0, 1), (77, 14, 2, 64, (12, 10, 10), 0, 1),
    (200, 3, 3, 64, (7, 8), 30, 0), (1030, 16, 2, 128, (64,), 0, 0), (6100, 2, 1, 64, (12, 10, 10), 0, 0),
    (12011, 2, 1, 128, (8, 12, 12), 64, 1)])
def test_mrope_append(cuda, rows, Hq, Hkv, D, sections, rot, interleaved):
    rot = rot or D
    g = torch.Generator().manual_seed(rows)
    heads, n_pages = Hq + 2 * Hkv, rows // 64 + 4
    qkv = torch.randn(rows, heads * D + 8, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 100000, (len(sections), rows), generator=g, dtype=torch.int32)
    slots = torch.randperm(n_pages * 64, generator=g)[:rows].to(torch.int32)
    if rows > 100:                       # a run of consecutive slots too, and padding rows
        run = torch.arange(65) + 64 * (n_pages - 2) + 3
        slots = torch.cat([slots[~torch.isin(slots, run.to(torch.int32))], run.to(torch.int32)])[-rows:]
        rows = len(slots)
        slots[5] = slots[rows - 70] = -1
    qkv, pos = qkv[:rows], pos[:, :rows].contiguous()
    kp = torch.randn(n_pages, Hkv, 64, D, generator=g).to(torch.bfloat16)
    vp = torch.randn(n_pages, Hkv, D, 64, generator=g).to(torch.bfloat16)
    q0 = torch.full((rows, Hq, D), 3.0, dtype=torch.bfloat16)
    qd, kd, vd, st = q0.to(cuda), kp.to(cuda), vp.to(cuda), status(cuda)
    dv.mrope_append_paged(qkv.to(cuda)[:, :heads * D], pos.to(cuda), slots.to(cuda), qd, kd, vd, n_rows=rows, Hq=Hq,
                          Hkv=Hkv, D=D, n_pages=n_pages, sections=sections, rot_dim=rot, rope_base=1e6,
                          interleaved=interleaved, status=st)
    assert_ok(st)
    x = qkv[:, :heads * D].reshape(rows, heads, D)
    xs = x[:, :Hq + Hkv].double().numpy()
    want = ref.mrope(xs, pos.numpy(), sections, 1e6, rot, interleaved)
    bound = mrope_bound(xs, want, rot // 2, rot, 2.0 ** -7)
    live = slots.numpy() >= 0
    page, row = slots.numpy()[live] // 64, slots.numpy()[live] % 64
    got_q = qd.cpu().double().numpy()
    assert (np.abs(got_q - want[:, :Hq])[live] <= bound[:, :Hq][live]).all()
    assert (got_q[~live] == 3.0).all()
    got_k = kd.cpu()[page, :, row].double().numpy()
    assert (np.abs(got_k - want[live, Hq:]) <= bound[live, Hq:]).all()
    want_v = vp.clone()
    want_v[page, :, :, row] = x[:, Hq + Hkv:][torch.from_numpy(live)]
    assert torch.equal(vd.cpu(), want_v)
    untouched = torch.ones(n_pages, 64, dtype=torch.bool)
    untouched[page, row] = False
    assert torch.equal(kd.cpu().transpose(1, 2)[untouched], kp.transpose(1, 2)[untouched])


def test_mrope_append_bad_slots(cuda):
    """Slots outside the pages are reported and skipped."""
    Hq, Hkv, D, n_pages = 2, 1, 64, 2
    for bad in (-2, 128, 2 ** 31 - 1, -2 ** 31):
        qkv = torch.ones(3, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device=cuda)
        q = torch.zeros(3, Hq, D, dtype=torch.bfloat16, device=cuda)
        kp = torch.zeros(n_pages, Hkv, 64, D, dtype=torch.bfloat16, device=cuda)
        vp = torch.zeros(n_pages, Hkv, D, 64, dtype=torch.bfloat16, device=cuda)
        st = status(cuda)
        dv.mrope_append_paged(qkv, i32([[0, 0, 0]], cuda), i32([1, bad, 127], cuda), q, kp, vp, n_rows=3, Hq=Hq,
                              Hkv=Hkv, D=D, n_pages=n_pages, sections=(32,), rope_base=1e4, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == BOUNDS
        assert (q[1] == 0).all() and (q[0] == 1).all() and (q[2] == 1).all()
        assert int((kp != 0).sum()) == 2 * D and int((vp != 0).sum()) == 2 * D


# ------------------------------------------------------- rejection sampling
def run_verify(cuda, p, q, ids, u, us, n_draft=None, cache=None, in_place=False):
    b, K = ids.shape
    V = p.shape[2]
    acc, out, st = i32([-9] * b, cuda), i32(np.full((b, K + 1), -9), cuda), status(cuda)
    cl = i32(cache, cuda) if cache is not None else None
    co = (cl if in_place else i32([-9] * b, cuda)) if cache is not None else None
    dv.spec_verify_sample(p.to(cuda), q.to(cuda) if q is not None else None, i32(ids, cuda),
                          torch.tensor(u, dtype=torch.float32, device=cuda),
                          torch.tensor(us, dtype=torch.float32, device=cuda), b=b, K=K, V=V,
                          dtype=dv.DVLM_FP32 if p.dtype == torch.float32 else dv.DVLM_BF16, accept_len=acc, out_ids=out,
                          n_draft=i32(n_draft, cuda) if n_draft is not None else None, cache_len=cl, cache_len_out=co,
                          status=st)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), out.cpu().numpy(), co.cpu().numpy() if co is not None else None, int(st.item())


def check_verify(cuda, p, q, ids, u, us, n_draft=None, **kw):
    b, K = ids.shape
    u, us = np.asarray(u, dtype=np.float32), np.asarray(us, dtype=np.float32)
    cache = np.arange(b) * 3 + 500
    acc, out, co, st = run_verify(cuda, p, q, ids, u, us, n_draft, cache, **kw)
    bad = False
    for i in range(b):
        nd = K if n_draft is None else n_draft[i]
        nd_c = min(max(nd, 0), K)
        bad |= nd_c != nd
        k, want, wrong = ref.verify(p[i].double().numpy(), q[i].double().numpy() if q is not None else None,
                                    ids[i].tolist(), u[i].astype(np.float64), float(us[i]), nd_c)
        bad |= wrong
        assert acc[i] == k, i
        assert out[i].tolist() == want, i
        assert co[i] == cache[i] - (nd_c - k)
    assert st == (BOUNDS if bad else 0)
    return acc


@pytest.mark.parametrize("b,K,V", [(1, 1, 1), (1, 4, 7), (3, 5, 33), (2, 15, 1000), (4, 7, 4099), (2, 33, 2048),
                                   (3, 3, 50257), (2, 4, 151936), (5, 64, 640)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_q", [True, False])
def test_verify_sample(cuda, b, K, V, dtype, with_q):
    g = torch.Generator().manual_seed(V + K)
    z = 2.0 * torch.randn(b, K + 1, V, generator=g)
    p = torch.softmax(z, -1).to(dtype)
    d = torch.softmax(z[:, :K] + 0.3 * torch.randn(b, K, V, generator=g), -1)
    ids = torch.multinomial(d.view(-1, V), 1, generator=g).view(b, K).numpy() if with_q else d.argmax(-1).numpy()
    q = d.to(dtype) if with_q else None
    u = torch.rand(b, K, generator=g).numpy() * (1.0 if with_q else 0.1)
    us = torch.rand(b, generator=g).numpy()
    check_verify(cuda, p, q, ids, u, us)
    u[:] = 0.0                                            # all drafts of positive probability accepted
    check_verify(cuda, p, q, ids, u, us, in_place=True)
    n_draft = [int(v) for v in torch.randint(0, K + 1, (b,), generator=g)]
    check_verify(cuda, p, q, ids, torch.rand(b, K, generator=g).numpy(), us, n_draft)


def test_verify_edges(cuda):
    """Exact steps of the cumulative sum, u 0 and near 1, holes of probability 0, an empty residual, NaN and
    infinities, refused drafts outside the vocabulary."""
    V, K = 160, 2
    p = torch.zeros(8, K + 1, V)
    q = torch.zeros(8, K, V)
    ids = np.zeros((8, K), dtype=np.int64)
    u, us = np.full((8, K), 0.5, dtype=np.float32), np.zeros(8, dtype=np.float32)
    p[:, :, [3, 40, 41, 150]] = 0.25
    q[:, :, 7] = 1.0
    ids[:] = 7                                           # p(7) = 0: always refused, the draw is from p
    for i, v in enumerate([0.0, 0.25, 0.5, 0.75, 1 - 2 ** -24, 0.2499999, 1.0, -1.0]):
        us[i] = v
    acc, out, _, st = run_verify(cuda, p, q, ids, u, us)
    assert st == 0 and (acc == 0).all()
    assert out[:, 0].tolist() == [3, 40, 41, 150, 150, 3, 150, 3]     # C(v) > u: a step itself goes to the next token
    check_verify(cuda, p, q, ids, u, us)
    # p == q and refused (u = 1): nothing left of the residual, the draw is from p; a zero row is an error
    q = p[:, :K].clone()
    ids[:] = 40
    check_verify(cuda, p, q, ids, np.ones((8, K)), us)
    p0 = p.clone()
    p0[2] = 0.0
    check_verify(cuda, p0, q, ids, np.ones((8, K)), us)
    # NaN and infinities count as 0
    p1 = p.clone()
    p1[:, :, 3], p1[:, :, 41], p1[:, :, 9] = float("nan"), float("inf"), 1e-30
    check_verify(cuda, p1, q, ids, np.ones((8, K)), us)
    ids[1, 0], ids[3, 1], ids[5] = -1, V, [2 ** 31 - 1, 0]
    u[:] = 0.0
    check_verify(cuda, p, q, ids, u, us)
    check_verify(cuda, p, None, ids, u, us)
    check_verify(cuda, p, q, ids, u, us, n_draft=[0, -1, 3, 2, 1, 0, 2, 2 ** 31 - 1])


def test_verify_draws_the_target(cuda):
    """Accepted and drawn first tokens follow the target's distribution: with the
    same number of evenly spaced u, the empirical frequencies match p (a
    lattice of 64 x 64 pairs (u_accept, u_sample), draft ids in q's
    proportions: exact shares up to one lattice step per token)."""
    V, n = 16, 64
    g = torch.Generator().manual_seed(4)
    p = torch.randint(1, 9, (V,), generator=g).float()
    q = torch.randint(1, 9, (V,), generator=g).float()
    p, q = p / p.sum(), q / q.sum()
    want = np.zeros(V)
    grid = (np.arange(n) + 0.5) / n
    uu, us = np.meshgrid(grid, grid, indexing="ij")
    got = np.zeros(V)
    for x in range(V):
        b = n * n
        acc, out, _, st = run_verify(cuda, p.expand(b, 2, V).contiguous(), q.expand(b, 1, V).contiguous(),
                                     np.full((b, 1), x), uu.reshape(b, 1), us.reshape(b))
        assert st == 0
        got += float(q[x]) * np.bincount(out[:, 0], minlength=V) / b
    # each token's share: an acceptance step and V sampling steps of the lattice, each within 1/n
    assert np.abs(got - p.numpy()).max() <= 2.0 / n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_infinite_drafts(cuda, dtype):
    """NaN and infinities of either sign in the draft's or the target's row: no such token is accepted or drawn, and
    every sequence gets its token."""
    V, K, inf = 2560, 1, float("inf")
    p = torch.zeros(6, K + 1, V)
    p[:, :, 40:48] = 0.125
    q = torch.zeros(6, K, V)
    q[:, :, 40] = 0.5
    ids = np.full((6, K), 40, dtype=np.int64)
    us = np.array([0.0, 0.5, 0.99, 0.0, 0.5, 0.99], dtype=np.float32)
    q[0:3, :, 41] = -inf                                    # p - q would be infinite
    q[0:3, :, 42], q[0:3, :, 43] = inf, float("nan")
    p[3:6, :, 41], p[3:6, :, 42], p[3:6, :, 43] = -inf, inf, float("nan")
    acc, out, _, st = run_verify(cuda, p.to(dtype), q.to(dtype), ids, np.ones((6, K)), us)
    assert st == 0 and (acc == 0).all()
    assert out[:, 0].tolist() == [44, 46, 47, 44, 46, 47]   # 44 .. 47 are left, a quarter each
    # as drafts: u = 0 accepts whatever has a finite probability, and only that
    for tok, ok in ((41, 0), (42, 0), (43, 0), (45, 1)):
        ids[:] = tok
        acc, out, _, st = run_verify(cuda, p.to(dtype), q.to(dtype), ids, np.zeros((6, K)), us)
        assert st == 0 and acc.tolist() == [ok] * 6
        assert ok or set(out[:, 0].tolist()) <= {40, 44, 45, 46, 47}


def test_page_plan_wild_pages(cuda):
    """Page numbers whose slots would wrap around 32 bits into the store give slots outside it."""
    wild = [2 ** 26 + 1, 2 ** 31 - 1, -2 ** 31, -2 ** 26 + 2, 2 ** 25, -2 ** 25 - 1]
    n = len(wild)
    table = np.full((n, 2), -1, dtype=np.int32)
    table[:, 0] = wild
    kv, cu, slots, tab, free, count, st, _ = run_plan(cuda, [5] * n, [3] * n, table, [], 4, 3 * n + 2)
    assert kv.tolist() == [8] * n and cu.tolist() == [3 * i for i in range(n + 1)]
    assert (tab == table).all() and int(count[0]) == 0
    for i, page in enumerate(wild):
        got = slots[3 * i:3 * i + 3].astype(np.int64)
        assert ((got >= 4 * 64) if page > 0 else (got < -1)).all()
        assert (got % 64 == [5, 6, 7]).all()
    assert slots[3 * n:].tolist() == [-1, -1]
    # a stack's wild number reaches the table as it is
    kv, cu, slots, tab, free, count, st, _ = run_plan(cuda, [0], [2], np.full((1, 1), -1, dtype=np.int32), [2 ** 27], 4, 2)
    assert tab.tolist() == [[2 ** 27]] and (slots >= 4 * 64).all()
