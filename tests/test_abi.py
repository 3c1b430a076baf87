"""C-ABI checks that need no GPU: the library loads, exports every entry
point include/dvlm.h declares, validates arguments on the host (returning a
status before any launch) and lays its structs out as the header does."""
import ctypes
import os
import subprocess


import block_diffusion_vlm_b200 as dv
from block_diffusion_vlm_b200 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK, INVALID, SHAPE, UNSUPPORTED, OVERFLOW, TIMEOUT, CUDA, WORKSPACE, BOUNDS = range(9)


def test_library_exports_every_declared_symbol(dvlm_lib):
    names = dv.declared_symbols()
    assert len(names) >= 19
    for n in names:
        assert hasattr(dvlm_lib, n), n
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True, text=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert set(names) == {e for e in exported if e.startswith("dvlm_")}


def test_status_strings_and_version(dvlm_lib):
    assert dv.status_string(0) == "ok"
    assert "timed out" in dv.status_string(TIMEOUT)
    assert dv.status_string(999) == "unknown status"
    assert dvlm_lib.dvlm_version() == 100


def test_struct_layouts_match_header(tmp_path):
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dvlm.h"\n'
                   'int main(){printf("%zu %zu %zu %zu %zu\\n", sizeof(dvlm_model), sizeof(dvlm_decode_cfg),'
                   ' sizeof(dvlm_stats), offsetof(dvlm_model, lm_head), offsetof(dvlm_stats, accept_hist));}\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = [ctypes.sizeof(dv.Model), ctypes.sizeof(dv.DecodeCfg), ctypes.sizeof(dv.Stats),
            dv.Model.lm_head.offset, dv.Stats.accept_hist.offset]
    assert got == want


def _attn(**kw):
    a = dict(q=16, out=16, k=16, v=16, nb=1, n_rows=16, n_clean=0, L=64, Lmax=128, Hq=16, Hkv=2, D=128,
             scale=0.088, dt=0)
    a.update(kw)
    return dv.lib().dvlm_block_attn(a["q"], a["out"], a["k"], a["v"], a["nb"], a["n_rows"], a["n_clean"], a["L"],
                                    a["Lmax"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["dt"], None, None)


def test_attention_host_validation(dvlm_lib):
    assert _attn(q=None) == INVALID
    assert _attn(dt=7) == INVALID
    assert _attn(scale=float("inf")) == INVALID
    assert _attn(n_clean=17) == SHAPE
    assert _attn(Hq=15) == SHAPE
    assert _attn(L=120) == OVERFLOW
    assert _attn(D=64) == UNSUPPORTED
    assert _attn(Hq=8) == UNSUPPORTED
    assert _attn(Lmax=130, L=64) == SHAPE
    assert _attn(q=18) == INVALID      # misaligned for the TMA path


def _lm(**kw):
    a = dict(h=16, w=16, R=16, H=2048, V=151936, dt=0, norm=0, eps=1e-6, masked=None, tokens=None, thr=0.9,
             aid=None, aconf=None, cert=None, ws=16, wsb=1 << 40)
    a.update(kw)
    return dv.lib().dvlm_lmhead_conf_commit(a["h"], a["w"], a["R"], a["H"], a["V"], a["dt"], a["norm"], a["eps"],
                                            a["masked"], a["tokens"], a["thr"], None, None, None, None, a["aid"],
                                            a["aconf"], a["cert"], a["ws"], a["wsb"], None, None)


def test_lmhead_host_validation(dvlm_lib):
    assert _lm(h=None) == INVALID
    assert _lm(R=0) == SHAPE and _lm(R=129) == SHAPE
    assert _lm(tokens=64) == INVALID                 # tokens need masked
    assert _lm(aid=64) == INVALID                    # certificate is all-or-none
    assert _lm(thr=float("nan")) == INVALID
    assert _lm(ws=None) == WORKSPACE
    assert _lm(wsb=100) == WORKSPACE
    assert _lm(H=100) == UNSUPPORTED
    assert _lm(h=24) == INVALID
    assert dv.lmhead_workspace_size(0, 10, 10, 0) == 0
    assert dv.lmhead_workspace_size(16, 151936, 2048, 0) > 0


def test_spec_host_validation(dvlm_lib):
    L = dv.lib()
    f = L.dvlm_spec_verify_accept
    assert f(None, 16, None, 1, 16, 100, 16, None, 0, None, None, 0, 0, 0, 0, None, 0, None, None) == INVALID
    assert f(None, None, 16, 1, 16, 100, 16, None, 0, None, None, 0, 0, 0, 0, None, 0, None, None) == INVALID
    assert f(None, 16, 16, 1, 16, 100, None, None, 0, None, None, 0, 0, 0, 0, None, 0, None, None) == INVALID
    assert f(None, 16, 16, 1, 65, 100, 16, None, 0, None, None, 0, 0, 0, 0, None, 0, None, None) == SHAPE
    assert f(16, None, 16, 1, 16, 100, 16, None, 0, None, None, 0, 0, 0, 0, None, 0, None, None) == WORKSPACE
    assert f(None, 16, 16, 1, 16, 100, 16, None, 1, None, None, 0, 0, 0, 0, None, 0, None, None) == INVALID


def test_topk_host_validation(dvlm_lib):
    f = dv.lib().dvlm_topk_commit
    assert f(None, 16, 16, 16, 4, 1, None, None, None, None) == INVALID
    assert f(16, 16, 16, None, 4, 1, None, None, None, None) == INVALID
    assert f(16, 16, 16, 16, 0, 1, None, None, None, None) == SHAPE
    assert f(16, 16, 16, 16, 129, 1, None, None, None, None) == SHAPE
    assert f(16, 16, 16, 16, 4, -1, None, None, None, None) == SHAPE
    g = dv.lib().dvlm_divergence_first_commit
    assert g(16, 16, None, 16, 16, 4, 1, None, None, None, None) == INVALID
    assert g(16, 16, 16, 16, 16, 129, 1, None, None, None, None) == SHAPE
    assert g(16, 16, 16, 16, 16, 4, -2, None, None, None, None) == SHAPE


def _dims_model(**kw):
    import dvlm_gen as gen
    m = dv.make_model(gen.QWEN3B, embed=None, wqkv=None, wo=None, wgate=None, wup=None, wdown=None,
                      lm_head=None, dtype=0)
    for name in ("embed", "wqkv", "wo", "wgate", "wup", "wdown", "lm_head"):
        setattr(m, name, 4096)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


def test_engine_host_validation(dvlm_lib):
    L = dv.lib()
    m = _dims_model()
    ws = dv.engine_workspace_size(m, 1600, 16, 1344)
    assert ws > 0
    assert dv.engine_workspace_size(_dims_model(n_kv_heads=3), 1600, 16, 1344) == 0
    assert dv.engine_workspace_size(_dims_model(mask_id=151936), 1600, 16, 1344) == 0
    assert dv.engine_workspace_size(m, 1600, 17, 1344) == 0
    h = ctypes.c_void_p()
    assert L.dvlm_engine_create(ctypes.byref(m), 4096, 4096, 1600, 16, 0, 4096, ws, None, None) == INVALID
    assert L.dvlm_engine_create(ctypes.byref(m), None, 4096, 1600, 16, 0, 4096, ws, None, ctypes.byref(h)) == INVALID
    assert L.dvlm_engine_create(ctypes.byref(_dims_model(head_dim=64)), 4096, 4096, 1600, 16, 0, 4096, ws, None,
                                ctypes.byref(h)) == UNSUPPORTED
    assert L.dvlm_engine_create(ctypes.byref(m), 4096, 4096, 1601, 16, 0, 4096, ws, None,
                                ctypes.byref(h)) == INVALID
    assert L.dvlm_engine_create(ctypes.byref(m), 4096, 4096, 1600, 16, 0, None, ws, None,
                                ctypes.byref(h)) == WORKSPACE
    assert L.dvlm_engine_destroy(None) == INVALID
    assert L.dvlm_prefill(None, None, 0, None, 0, None) == INVALID
    assert L.dvlm_decode_block(None, None, None, None, None, None) == INVALID
    assert L.dvlm_forward_text_only(None, 4096, None, 16, 32, None, None) == INVALID


def test_missing_library_fails_loudly(monkeypatch, tmp_path):
    """No fallback: without the built library every entry point raises."""
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "LIB_PATH", str(tmp_path / "libdvlm.so"))
    import pytest
    with pytest.raises(RuntimeError, match="missing"):
        binding.lib()
    with pytest.raises(RuntimeError, match="missing"):
        dv.topk_commit(None, None, None, None, R=1, k=1)


def test_binding_declares_every_header_entry_point():
    """Every entry point of include/dvlm.h has a ctypes signature in the
    binding (so no call goes through ctypes' int defaults)."""
    import inspect
    import re
    src = inspect.getsource(binding._declare)
    assert set(re.findall(r'"(dvlm_\w+)"', src)) == set(dv.declared_symbols())


def _plan(**kw):
    a = dict(cache=16, new=16, table=16, free=16, count=16, n=4, mp=8, np=32, rows=64, kv=16, cu=16, slots=16, out=16)
    a.update(kw)
    return dv.lib().dvlm_page_plan(a["cache"], a["new"], a["table"], a["free"], a["count"], a["n"], a["mp"], a["np"],
                                   a["rows"], a["kv"], a["cu"], a["slots"], a["out"], None, None, None)


def test_page_plan_host_validation(dvlm_lib):
    for name in ("cache", "new", "table", "free", "count", "kv", "cu", "slots", "out"):
        assert _plan(**{name: None}) == INVALID
    for kw in (dict(n=0), dict(n=4097), dict(mp=0), dict(mp=1 << 25), dict(np=0), dict(np=1 << 25), dict(rows=0)):
        assert _plan(**kw) == SHAPE


def _mrope(**kw):
    a = dict(x=16, out=32, pos=16, rows=4, heads=2, D=64, x_ld=128, o_ld=128, rot=64, n=3, sec=(12, 10, 10), base=1e4,
             il=0, dt=0)
    a.update(kw)
    sec = (ctypes.c_int * len(a["sec"]))(*a["sec"]) if a["sec"] is not None else None
    return dv.lib().dvlm_mrope(a["x"], a["out"], a["pos"], a["rows"], a["heads"], a["D"], a["x_ld"], a["o_ld"],
                               a["rot"], a["n"], sec, a["base"], a["il"], a["dt"], None, None)


def _append(**kw):
    a = dict(qkv=16, pos=16, slots=16, q=16, k=16, v=16, rows=4, Hq=2, Hkv=1, D=64, np=4, ld=256, rot=64, n=3,
             sec=(12, 10, 10), base=1e4, il=0)
    a.update(kw)
    sec = (ctypes.c_int * len(a["sec"]))(*a["sec"]) if a["sec"] is not None else None
    return dv.lib().dvlm_mrope_append_paged(a["qkv"], a["pos"], a["slots"], a["q"], a["k"], a["v"], a["rows"], a["Hq"],
                                            a["Hkv"], a["D"], a["np"], a["ld"], a["rot"], a["n"], sec, a["base"],
                                            a["il"], None, None)


def test_mrope_host_validation(dvlm_lib):
    for f in (_mrope, _append):
        assert f(pos=None) == INVALID and f(sec=None) == INVALID
        assert f(il=2) == INVALID and f(base=0.0) == INVALID and f(base=float("nan")) == INVALID
        assert f(n=0) == SHAPE and f(n=5, sec=(12, 10, 10, 0, 0)) == SHAPE
        assert f(sec=(12, 10, 11)) == SHAPE and f(sec=(42, -10, 0)) == SHAPE
        assert f(rot=63) == SHAPE and f(rot=66, sec=(13, 10, 10)) == SHAPE and f(rot=0, sec=(0, 0, 0)) == SHAPE
        assert f(rows=0) == SHAPE
    assert _mrope(x=None) == INVALID and _mrope(out=None) == INVALID and _mrope(dt=2) == INVALID
    assert _mrope(x=17) == INVALID and _mrope(dt=1, x=18) == INVALID
    assert _mrope(D=258, x_ld=1000, o_ld=1000) == SHAPE and _mrope(x_ld=127) == SHAPE and _mrope(o_ld=127) == SHAPE
    assert _mrope(out=16, o_ld=136) == SHAPE and _mrope(heads=0) == SHAPE
    for name in ("qkv", "slots", "q", "k", "v"):
        assert _append(**{name: None}) == INVALID
    for name in ("qkv", "q", "k", "v"):
        assert _append(**{name: 24}) == INVALID
    assert _append(D=80, rot=64, ld=400) == UNSUPPORTED
    assert _append(ld=248) == SHAPE and _append(ld=260) == SHAPE
    assert _append(np=0) == SHAPE and _append(np=1 << 25) == SHAPE and _append(Hkv=0) == SHAPE


def _verify(**kw):
    a = dict(p=16, q=16, ids=16, nd=None, u=16, us=16, b=1, K=4, V=100, dt=0, acc=16, out=16, cl=None, co=None)
    a.update(kw)
    return dv.lib().dvlm_spec_verify_sample(a["p"], a["q"], a["ids"], a["nd"], a["u"], a["us"], a["b"], a["K"], a["V"],
                                            a["dt"], a["acc"], a["out"], a["cl"], a["co"], None, None)


def test_verify_sample_host_validation(dvlm_lib):
    for name in ("p", "ids", "u", "us", "acc", "out"):
        assert _verify(**{name: None}) == INVALID
    assert _verify(cl=16) == INVALID and _verify(co=16) == INVALID
    assert _verify(dt=2) == INVALID and _verify(p=17) == INVALID and _verify(dt=1, q=18) == INVALID
    for kw in (dict(b=0), dict(b=65536), dict(K=0), dict(K=65), dict(V=0), dict(V=(1 << 30) + 1)):
        assert _verify(**kw) == SHAPE


def test_step_binding_refuses_what_it_would_misread(dvlm_lib):
    """Wrong types, sizes and devices raise before the library is called."""
    import pytest
    import torch
    i = torch.zeros(8, dtype=torch.int32)
    kw = dict(n_batch=4, max_pages=2, n_pages=8, max_rows=8, kv_len=i, cu_rows=i, slot_map=i, free_count_out=i)
    with pytest.raises(dv.DvlmError):
        dv.page_plan(i.long(), i, i, i, i, **kw)
    with pytest.raises(dv.DvlmError):
        dv.page_plan(i, i, i[:7], i, i, **kw)
    with pytest.raises(dv.DvlmError):
        dv.page_plan(i, i, i, i, i, **kw)               # host tensors
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    mk = dict(n_rows=4, n_heads=2, D=64, sections=(32,), rope_base=1e4, dtype=dv.DVLM_BF16)
    for bad in (x.float(), x[:, :1], x[:3], x.transpose(0, 1)):
        with pytest.raises(dv.DvlmError):
            dv.mrope(bad, x, i, **mk)
    p = torch.zeros(1, 5, 100)
    vk = dict(b=1, K=4, V=100, dtype=dv.DVLM_FP32, accept_len=i, out_ids=i)
    u = torch.zeros(4)
    for args in ((p.bfloat16(), None, i, u, u), (p[:, :4], None, i, u, u), (p, p[:, :3], i, u, u), (p, None, i, u.double(), u)):
        with pytest.raises(dv.DvlmError):
            dv.spec_verify_sample(*args, **vk)


def _chunk(**kw):
    a = dict(q=16, out=16, k=16, v=16, table=16, kv=16, cu=16, nb=2, rows=8, np=4, mp=4, Hq=8, Hkv=1, D=128, ld=1024,
             scale=0.09, ws=16, wsb=1 << 40)
    a.update(kw)
    return dv.lib().dvlm_chunk_attn_paged(a["q"], a["out"], a["k"], a["v"], a["table"], a["kv"], a["cu"], None, None,
                                          None, a["nb"], a["rows"], a["np"], a["mp"], a["Hq"], a["Hkv"], a["D"],
                                          a["ld"], a["scale"], a["ws"], a["wsb"], None, None)


def test_chunk_attention_host_validation(dvlm_lib):
    for name in ("q", "out", "k", "v", "table", "kv", "cu"):
        assert _chunk(**{name: None}) == INVALID
    for name in ("q", "out", "k", "v", "ws"):
        assert _chunk(**{name: 24}) == INVALID
    for s in (0.0, -0.1, float("inf"), float("nan")):
        assert _chunk(scale=s) == INVALID
    for kw in (dict(nb=0), dict(rows=0), dict(np=0), dict(np=1 << 25), dict(mp=0), dict(Hq=0), dict(Hkv=3),
               dict(ld=1016), dict(ld=1028), dict(np=1 << 24, Hkv=1), dict(np=1 << 20, Hkv=16, Hq=16, ld=2048)):
        assert _chunk(**kw) == SHAPE, kw
    assert _chunk(D=96) == UNSUPPORTED and _chunk(Hq=129, Hkv=1, ld=129 * 128) == UNSUPPORTED
    assert _chunk(ws=None) == WORKSPACE and _chunk(wsb=1000) == WORKSPACE
    assert dv.chunk_attn_paged_workspace_size(1, 1, 16, 2, 96) == 0
    assert dv.chunk_attn_paged_workspace_size(0, 1, 16, 2, 128) == 0
    assert 0 < dv.chunk_attn_paged_workspace_size(1, 1, 16, 2, 64) < dv.chunk_attn_paged_workspace_size(1, 1, 16, 2, 128)


def test_step_limits(dvlm_lib):
    """Sizes whose offsets or counts would pass what the kernels hold in 31 bits."""
    assert _plan(rows=(1 << 30) + 1) == SHAPE and _plan(rows=2 ** 31 - 1) == SHAPE
    assert _plan(n=4096, mp=1 << 20) == SHAPE

    def chunk(n=1, rows=4, scale=0.1, ws=16, ws_bytes=0):
        return dv.lib().dvlm_chunk_attn_paged(16, 16, 16, 16, 16, 16, 16, None, None, None, n, rows, 4, 8, 8, 2, 64, 512,
                                              scale, ws, ws_bytes, None, None)
    assert chunk() == WORKSPACE
    for n in ((1 << 24) + 1, 2 ** 31 - 1):
        assert chunk(n=n) == SHAPE
    for rows in ((1 << 30) + 1, 2 ** 31 - 1):
        assert chunk(rows=rows) == SHAPE
    for scale in (3e38, 1e-46, 0.0, -1.0, float("inf"), float("nan")):
        assert chunk(scale=scale) == INVALID
