"""The batched paged step as it is used: plan, rotary append, attention and
verification one behind the other over several steps of a small batch (prompt
chunks with image positions, noisy blocks, drafted tokens that are partly
refused, a request that finishes and one that takes its pages), all on the
GPU, without a host read in between.  Each stage is held to its plain
definition on the stage's own inputs (the tolerances of test_gpu_step.py and
test_gpu_chunk_attn.py).  Also: the whole step in one captured graph, two
batches at once on two streams, and caches whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import block_diffusion_vlm_b200 as dv
import step_reference as ref
from gpu_util import assert_ok, status, ws_tensor
from test_gpu_chunk_attn import check as check_attn
from test_gpu_step import mrope_bound

pytestmark = pytest.mark.gpu
Hq, Hkv, D, SEC, BASE = 8, 1, 128, (16, 24, 24), 1e6
HEADS = Hq + 2 * Hkv


class Server:
    """One batch's device state and the calls of a step."""

    def __init__(self, dev, n, max_pages, n_pages, max_rows, K=6, V=512, seed=0):
        i = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device=dev)
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.n, self.max_pages, self.n_pages, self.max_rows, self.K, self.V = n, max_pages, n_pages, max_rows, K, V
        self.g = torch.Generator(device=dev).manual_seed(seed)
        self.cache, self.held, self.new, self.kv = i(n), i(n), i(n), i(n)
        self.table, self.cu, self.slots = i(n, max_pages, v=-1), i(n + 1), i(max_rows)
        self.free, self.count = torch.randperm(n_pages, generator=self.g, device=dev).to(torch.int32), i(1, v=n_pages)
        self.noisy, self.hidden = i(n), i(n)
        self.kp = torch.full((n_pages, Hkv, 64, D), float("nan"), **bf)
        self.vp = torch.full((n_pages, Hkv, D, 64), float("nan"), **bf)
        self.qkv, self.pos = torch.zeros(max_rows, HEADS * D, **bf), i(3, max_rows)
        self.q, self.out = torch.zeros(max_rows, Hq, D, **bf), torch.full((max_rows, Hq, D), 7.0, **bf)
        self.lse = torch.zeros(max_rows, Hq, device=dev)
        self.ws = ws_tensor(dv.chunk_attn_paged_workspace_size(n, max_rows, Hq, Hkv, D), dev)
        self.ids, self.acc, self.tok = i(n, K), i(n), i(n, K + 1)
        self.p = torch.zeros(n, K + 1, V, device=dev)
        self.u, self.us, self.nd = torch.zeros(n, K, device=dev), torch.zeros(n, device=dev), i(n)
        self.st = status(dev)

    def fill(self):
        """New rows and random numbers (in place: a captured step replays on them)."""
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g, device=self.qkv.device))
        t = torch.arange(self.max_rows, device=self.pos.device) + int(torch.randint(0, 9000, (1,), generator=self.g,
                                                                                    device=self.pos.device))
        for a in range(3):
            self.pos[a] = torch.where(t // 40 % 2 == 0, [t - t % 40, t // 8 % 5, t % 8][a], t)
        z = 3.0 * torch.randn(self.p.shape, generator=self.g, device=self.p.device)
        self.p.copy_(torch.softmax(z, -1))
        self.ids.copy_(z[:, :self.K].argmax(-1))
        self.u.copy_(0.8 * torch.rand(self.u.shape, generator=self.g, device=self.u.device))
        self.us.copy_(torch.rand(self.us.shape, generator=self.g, device=self.us.device))

    def step(self, verify):
        dv.page_plan(self.cache, self.new, self.table, self.free, self.count, n_batch=self.n,
                     max_pages=self.max_pages, n_pages=self.n_pages, max_rows=self.max_rows, kv_len=self.kv,
                     cu_rows=self.cu, slot_map=self.slots, free_count_out=self.count, held_len=self.held, status=self.st)
        dv.mrope_append_paged(self.qkv, self.pos, self.slots, self.q, self.kp, self.vp, n_rows=self.max_rows, Hq=Hq,
                              Hkv=Hkv, D=D, n_pages=self.n_pages, sections=SEC, rope_base=BASE, status=self.st)
        dv.chunk_attn_paged(self.q, self.out, self.kp, self.vp, self.table, self.kv, self.cu, n_batch=self.n,
                            n_rows=self.max_rows, n_pages=self.n_pages, max_pages=self.max_pages, Hq=Hq, Hkv=Hkv, D=D,
                            scale=D ** -0.5, n_noisy=self.noisy, n_hidden=self.hidden, lse=self.lse, workspace=self.ws,
                            status=self.st)
        if verify:
            dv.spec_verify_sample(self.p, None, self.ids, self.u, self.us, b=self.n, K=self.K, V=self.V,
                                  dtype=dv.DVLM_FP32, accept_len=self.acc, out_ids=self.tok, n_draft=self.nd,
                                  cache_len=self.kv, cache_len_out=self.cache, status=self.st)
        else:
            self.cache.copy_(self.kv)


def host(t):
    return t.cpu().numpy().copy()


def run_and_check(s, new, noisy, hidden=None, n_draft=None):
    """One step against the definitions."""
    dev = s.cache.device
    put = lambda t, v: t.copy_(torch.tensor(np.asarray(v, dtype=np.int32), device=dev))
    put(s.new, new)
    put(s.noisy, noisy)
    put(s.hidden, hidden if hidden is not None else [0] * s.n)
    if n_draft is not None:
        put(s.nd, n_draft)
    s.fill()
    s.out.fill_(7.0)
    before = dict(cache=host(s.cache), held=host(s.held), table=host(s.table),
                  stack=host(s.free)[:int(s.count)].tolist())
    q0 = s.q.clone()
    s.step(n_draft is not None)
    assert_ok(s.st)
    want = ref.page_plan(before["cache"], new, before["table"], before["stack"], s.max_pages, s.n_pages, s.max_rows,
                         before["held"])
    assert not want[5] and not want[6]
    kv, cu, slots, table = host(s.kv), host(s.cu), host(s.slots), host(s.table)
    np.testing.assert_array_equal(kv, want[0])
    np.testing.assert_array_equal(cu, want[1])
    np.testing.assert_array_equal(slots, want[2])
    np.testing.assert_array_equal(table, want[3])
    np.testing.assert_array_equal(host(s.free)[:int(s.count)], want[4])
    np.testing.assert_array_equal(host(s.held), want[7])
    # rotary rows and their pages
    rows = int(cu[-1])
    x = s.qkv.view(s.max_rows, HEADS, D)[:rows].double().cpu().numpy()
    turned = ref.mrope(x[:, :Hq + Hkv], host(s.pos)[:, :rows], SEC, BASE, D, 0)
    bound = mrope_bound(x[:, :Hq + Hkv], turned, D // 2, D, 2.0 ** -7)
    page, row = slots[:rows] // 64, slots[:rows] % 64
    assert (np.abs(s.q[:rows].double().cpu().numpy() - turned[:, :Hq]) <= bound[:, :Hq]).all()
    assert (np.abs(s.kp.cpu()[page, :, row].double().numpy() - turned[:, Hq:]) <= bound[:, Hq:]).all()
    assert (s.vp.cpu()[page, :, :, row].double().numpy() == x[:, Hq + Hkv:]).all()
    assert torch.equal(s.q[rows:], q0[rows:])          # padding rows are left as they were
    # attention over what the pages now hold
    reqs = [(max(0, int(cu[b + 1] - cu[b])), int(kv[b]), int(noisy[b]), int(hidden[b]) if hidden else 0)
            for b in range(s.n)]
    c = dict(q=s.q.reshape(s.max_rows, -1).cpu(), kp=s.kp.cpu(), vp=s.vp.cpu(), table=torch.from_numpy(table), cu=cu,
             rows=rows, reqs=reqs, Hq=Hq, Hkv=Hkv, D=D)
    check_attn(c, s.out.double().cpu().numpy(), s.lse.double().cpu().numpy())
    if n_draft is not None:
        acc, tok, cut = host(s.acc), host(s.tok), host(s.cache)
        for b in range(s.n):
            k, ids, bad = ref.verify(host(s.p[b]).astype(np.float64), None, host(s.ids[b]).tolist(),
                                     host(s.u[b]).astype(np.float64), float(s.us[b]), n_draft[b])
            assert (acc[b], tok[b].tolist(), cut[b]) == (k, ids, kv[b] - (n_draft[b] - k)) and not bad
        return acc
    return None


def test_steps_of_a_batch(cuda):
    s = Server(cuda, n=4, max_pages=8, n_pages=14, max_rows=400)
    run_and_check(s, [130, 20, 0, 65], [0] * 4)                       # prompts
    run_and_check(s, [70, 16, 33, 1], [0, 16, 0, 0])                  # a second chunk, a block, a new request, a token
    accepted = []
    for i in range(4):                                                # drafted blocks, partly refused
        accepted.append(run_and_check(s, [6, 6, 0, 4], [6, 6, 0, 4], [100, 0, 0, 0], n_draft=[6, 6, 0, 4]))
    assert len({int(a) for acc in accepted for a in acc}) > 2         # several accepted lengths came up
    run_and_check(s, [-1, 16, 250, 0], [0, 16, 0, 0])                 # one finishes, its pages go to another
    run_and_check(s, [64, 1, 1, 1], [0] * 4)                          # and its place is taken
    owned = int(sum(-(-h // 64) for h in host(s.held).tolist()))
    assert owned + int(s.count) == s.n_pages


def test_step_in_a_graph(cuda):
    """The whole step captured once and replayed: lengths, pages and rows all come from the device."""
    a, b = (Server(cuda, n=3, max_pages=6, n_pages=18, max_rows=64, seed=5) for _ in range(2))
    for s in (a, b):
        s.new.copy_(torch.tensor([9, 16, 1], device=cuda))
        s.nd.copy_(torch.tensor([6, 3, 0], device=cuda))
        s.fill()
        s.step(True)                                                  # (warm-up, outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = {k: v.clone() for k, v in vars(b).items() if isinstance(v, torch.Tensor)}
    with torch.cuda.graph(graph):
        b.step(True)
    for k, v in keep.items():
        getattr(b, k).copy_(v)
    for _ in range(5):
        a.fill()
        b.fill()
        a.step(True)
        graph.replay()
    assert_ok(a.st)
    assert_ok(b.st)
    rows = int(a.cu[-1])
    for k in ("kv", "cache", "held", "cu", "slots", "table", "free", "count", "acc", "tok"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k
    assert torch.equal(a.out[:rows], b.out[:rows]) and torch.equal(a.kp.view(torch.int16), b.kp.view(torch.int16))


def test_two_batches_on_two_streams(cuda):
    """Two batches at once, each on its own stream with its own workspace, equal the same batches one by one."""
    def make():
        out = []
        for seed, new in ((1, [200, 1, 17]), (2, [3, 150, 64])):
            s = Server(cuda, n=3, max_pages=8, n_pages=20, max_rows=300, seed=seed)
            s.new.copy_(torch.tensor(new, device=cuda))
            s.nd.copy_(torch.tensor([3, 1, 0], device=cuda))
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
        assert int(x.st) == int(y.st)
        for k in ("kv", "cache", "table", "slots", "acc", "tok"):
            assert torch.equal(getattr(x, k), getattr(y, k)), k
        assert torch.equal(x.out, y.out)


def test_offsets_past_32_bits(cuda):
    """Pages whose first elements lie past 2^31 elements into the stores."""
    n_pages, kv = 150000, 130
    kp = torch.empty(n_pages, 2, 64, D, dtype=torch.bfloat16, device=cuda)
    vp = torch.empty(n_pages, 2, D, 64, dtype=torch.bfloat16, device=cuda)
    assert n_pages * 2 * 64 * D > 2 ** 31
    pages = [n_pages - 1, 131073, n_pages - 2]
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(kv, (16 + 4) * D, generator=g).to(torch.bfloat16)
    pos = torch.arange(kv, dtype=torch.int32).repeat(3, 1)
    slots = torch.tensor([pages[i // 64] * 64 + i % 64 for i in range(kv)], dtype=torch.int32)
    q = torch.zeros(kv, 16, D, dtype=torch.bfloat16, device=cuda)
    out = torch.zeros_like(q)
    st = status(cuda)
    dv.mrope_append_paged(qkv.to(cuda), pos.to(cuda), slots.to(cuda), q, kp, vp, n_rows=kv, Hq=16, Hkv=2, D=D,
                          n_pages=n_pages, sections=SEC, rope_base=BASE, status=st)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda)
    ws = ws_tensor(dv.chunk_attn_paged_workspace_size(1, kv, 16, 2, D), cuda)
    dv.chunk_attn_paged(q, out, kp, vp, i32([pages]), i32([kv]), i32([0, kv]), n_batch=1, n_rows=kv, n_pages=n_pages,
                        max_pages=3, Hq=16, Hkv=2, D=D, scale=D ** -0.5, workspace=ws, status=st)
    assert_ok(st)
    small = torch.tensor(pages, device=cuda)
    c = dict(q=q.reshape(kv, -1).cpu(), kp=kp[small].cpu(), vp=vp[small].cpu(),
             table=torch.tensor([[0, 1, 2]]), cu=np.array([0, kv]), rows=kv, reqs=[(kv, kv, 0, 0)], Hq=16, Hkv=2, D=D)
    assert torch.equal(c["vp"][0, :, :, 5], qkv[5].view(20, D)[18:])
    check_attn(c, out.double().cpu().numpy(), None)
