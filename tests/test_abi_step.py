"""Host-side refusals of the batched paged step's entry points (no GPU needed)."""
import pytest
import torch

import block_diffusion_vlm_b200 as dv

OK, INVALID, SHAPE = 0, 1, 2


def _verify_rows(**kw):
    a = dict(p=16, q=16, ids=16, nd=None, u=16, us=16, b=1, K=4, V=100, dt=0, acc=16, out=16, cl=None, co=None, cu=16)
    a.update(kw)
    return dv.lib().dvlm_spec_verify_sample_rows(a["p"], a["q"], a["ids"], a["nd"], a["u"], a["us"], a["b"], a["K"],
                                                 a["V"], a["dt"], a["acc"], a["out"], a["cl"], a["co"], a["cu"], None,
                                                 None)


def test_verify_rows_host_validation(dvlm_lib):
    for name in ("p", "ids", "u", "us", "acc", "out", "cu"):
        assert _verify_rows(**{name: None}) == INVALID
    assert _verify_rows(cl=16) == INVALID and _verify_rows(co=16) == INVALID
    assert _verify_rows(dt=2) == INVALID and _verify_rows(p=17) == INVALID and _verify_rows(dt=1, q=18) == INVALID
    for kw in (dict(b=0), dict(b=65536), dict(K=0), dict(K=65), dict(V=0), dict(V=(1 << 30) + 1)):
        assert _verify_rows(**kw) == SHAPE


def test_verify_binding_refuses_wrong_row_offsets(dvlm_lib):
    i, p, u = torch.zeros(8, dtype=torch.int32), torch.zeros(1, 5, 100), torch.zeros(4)
    for cu in (i.long(), i[:1], i):              # type, length, a host tensor
        with pytest.raises(dv.DvlmError):
            dv.spec_verify_sample(p, None, i, u, u, b=1, K=4, V=100, dtype=dv.DVLM_FP32, accept_len=i, out_ids=i,
                                  cu_rows=cu)
