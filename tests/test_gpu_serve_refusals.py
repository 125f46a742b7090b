"""What the binding refuses on the device: types, shapes and strides that the C
calls could not see.  Nothing is launched by any of these."""
import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_kv import I32, new_cache

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

Z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")


def refused(fn, *kinds):
    with pytest.raises(kinds or (TypeError, ValueError, RuntimeError)):
        fn()


def test_norm_calls():
    q, k, p = Z(4, 6, 64), Z(4, 2, 64), Z(4, dtype=torch.int64)
    f, _ = sv.sv_rope_frequencies(64, device="cuda")
    fwd = lambda q=q, k=k, p=p, f=f, **kw: sv.sv_qk_norm_rope(q, k, p, f, **kw)
    fwd()
    refused(lambda: fwd(q=q.half()), TypeError)
    refused(lambda: fwd(k=k.float()), TypeError)
    refused(lambda: fwd(k=Z(3, 2, 64)), ValueError)
    refused(lambda: fwd(k=Z(4, 2, 32)), ValueError)
    refused(lambda: fwd(q=Z(4, 6 * 64)), ValueError)
    refused(lambda: fwd(q=Z(4, 64, 6).transpose(1, 2)), ValueError)
    refused(lambda: fwd(k="keys"), TypeError)
    refused(lambda: fwd(p=None), ValueError)
    refused(lambda: fwd(p=p.int()), TypeError)
    refused(lambda: fwd(p=p[:3]), ValueError)
    refused(lambda: fwd(f=f.float()), TypeError)
    refused(lambda: fwd(f=torch.zeros(33, dtype=torch.float64, device="cuda")), RuntimeError)
    refused(lambda: fwd(q_weight=Z(63)), ValueError)
    refused(lambda: fwd(q_weight=Z(64), k_weight=Z(64).float()), TypeError)
    refused(lambda: fwd(q_weight=Z(64).half()), TypeError)
    refused(lambda: fwd(eps=0.0), RuntimeError)
    refused(lambda: fwd(eps=1e-40), RuntimeError)
    refused(lambda: fwd(layout="pairs"), ValueError)
    refused(lambda: fwd(out=dict(q=Z(4, 6, 32))), ValueError)
    refused(lambda: fwd(out=dict(k=Z(4, 1, 64).expand(4, 2, 64))), RuntimeError)
    bwd = lambda q=q, k=k, dq=q, dk=k, **kw: sv.sv_qk_norm_rope_backward(q, k, dq, dk, p, f, **kw)
    bwd()
    refused(lambda: bwd(dq=Z(4, 5, 64)), ValueError)
    refused(lambda: bwd(dk=None), ValueError)
    refused(lambda: bwd(k=None), ValueError)
    refused(lambda: bwd(dq=q.float()), TypeError)
    refused(lambda: bwd(out=dict(dq_weight=Z(64))), TypeError)
    refused(lambda: bwd(out=dict(dk_weight=Z(65, dtype=torch.float32))), ValueError)
    refused(lambda: bwd(workspace=Z(8, dtype=torch.uint8)), RuntimeError)
    assert set(sv.sv_qk_norm_rope_backward(q, None, q, None)) == {"dq", "dq_weight"}


def test_append_normed():
    c = new_cache("bf16", 5, 16, 2, 64)
    k, a = Z(4, 2, 64), (I32([[0, 1]]), I32([0, 4]), I32([9]))
    call = lambda k=k, v=k, **kw: sv.sv_kv_append_normed(k, v, c["k_cache"], c["v_cache"], *a, **kw)
    call()
    refused(lambda: call(v=Z(4, 1, 64)), ValueError)
    refused(lambda: call(k=Z(4, 2, 32)), ValueError)
    refused(lambda: call(k_weight=Z(32)), ValueError)
    refused(lambda: call(q=Z(5, 2, 64)), ValueError)
    refused(lambda: call(eps=float("nan")), RuntimeError)


def test_pages():
    i = lambda *s: Z(*s, dtype=torch.int32)
    ok = dict(page_table=i(3, 4) - 1, pages_held=i(3), free_pages=torch.arange(9, device="cuda").int(), free_count=I32([9]),
              kv_len=i(3), page_size=16)
    call = lambda **kw: sv.sv_kv_pages(**{**ok, **kw})
    call()
    for n in ("page_table", "pages_held", "free_pages", "free_count", "kv_len"):
        refused(lambda: call(**{n: ok[n].long()}), TypeError)
        refused(lambda: call(**{n: ok[n].cpu()}), ValueError)
    refused(lambda: call(page_table=i(2, 4)), ValueError)
    refused(lambda: call(page_table=i(4, 3).t()), ValueError)
    refused(lambda: call(page_table=i(1, 4).expand(3, 4)), RuntimeError)
    refused(lambda: call(pages_held=i(4)), ValueError)
    refused(lambda: call(free_count=i(2)), ValueError)
    refused(lambda: call(shared_pages=i(2)), ValueError)
    refused(lambda: call(query_start=i(3), rows=4), ValueError)
    refused(lambda: call(query_start=i(4), rows=-1), ValueError)
    refused(lambda: call(query_start=i(4), rows=sv.SV_ATTN_MAX_ROWS + 1), ValueError)
    refused(lambda: call(query_start=i(4), rows=3, out=dict(slots=i(3))), TypeError)
    refused(lambda: call(page_size=24), RuntimeError)
    refused(lambda: call(page_size=0), RuntimeError)
    assert ok["free_count"].tolist() == [9] and (ok["page_table"] == -1).all()


def test_attention():
    c = new_cache("bf16", 5, 16, 2, 64)
    a = (Z(4, 4, 64), c["k_cache"], c["v_cache"], I32([[0, 1]]), I32([0, 4]), I32([9]))
    sinks = lambda *b, **kw: sv.sv_paged_attention_sinks(*(b or a), **{**dict(window=4, sinks=2), **kw})
    sinks()
    refused(lambda: sinks(window=-1), RuntimeError)
    refused(lambda: sinks(sinks=-1), RuntimeError)
    refused(lambda: sinks(scale=0.0), RuntimeError)
    refused(lambda: sinks(a[0].float(), *a[1:]), TypeError)
    refused(lambda: sinks(Z(4, 3, 64), *a[1:]), RuntimeError)
    refused(lambda: sinks(max_kv_len=-1), RuntimeError)
    shared = lambda gs=I32([0, 1]), sl=I32([4]), **kw: sv.sv_paged_attention_shared(*a, gs, sl, **kw)
    shared()
    refused(lambda: shared(gs=I32([0])), ValueError)
    refused(lambda: shared(sl=I32([4]).long()), TypeError)
    refused(lambda: shared(gs=I32([0, 1]).cpu()), ValueError)
    refused(lambda: shared(max_group_len=-1), RuntimeError)
    refused(lambda: shared(max_shared_len=-4), RuntimeError)
    refused(lambda: shared(workspace=Z(64, dtype=torch.uint8)), RuntimeError)
    refused(lambda: shared(out=dict(lse=Z(4, 4))), TypeError)
