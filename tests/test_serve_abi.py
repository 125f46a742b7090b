"""Refusals of the norm, page and attention variants' calls of specverify_attn.h:
made on the host before anything is launched (no GPU)."""
import ctypes
import math
import os

import pytest
import torch

import draft_token_verification_spec_amd as sv
from draft_token_verification_spec_amd import attn
from test_attn_abi import BAD_CACHES, FAKE, cache

pytestmark = pytest.mark.skipif(not os.path.exists(sv.lib_path()), reason="libspecverify.so not built")


def norm(**kw):
    a = dict(stream=None, T=4, q_heads=4, k_heads=2, D=64, rotary=64, layout=0, dtype=1, q=FAKE, qt=256, qh=64, k=FAKE,
             kt=128, kh=64, wtype=0, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, freq=FAKE, mscale=1.0, qo=FAKE, qot=256, qoh=64,
             ko=FAKE, kot=128, koh=64)
    return attn._attn_lib().sv_qk_norm_rope(*{**a, **kw}.values())


def norm_backward(**kw):
    a = dict(stream=None, T=4, q_heads=4, k_heads=2, D=64, rotary=64, layout=0, dtype=1, q=FAKE, qt=256, qh=64, k=FAKE,
             kt=128, kh=64, gq=FAKE, gqt=256, gqh=64, gk=FAKE, gkt=128, gkh=64, wtype=0, qw=FAKE, kw=FAKE, eps=1e-6,
             pos=FAKE, freq=FAKE, mscale=1.0, qo=FAKE, qot=256, qoh=64, ko=FAKE, kot=128, koh=64, dqw=FAKE, dkw=FAKE,
             ws=FAKE, bytes=1 << 40)
    return attn._attn_lib().sv_qk_norm_rope_backward(*{**a, **kw}.values())


NORM = [
    (dict(T=-1), -1), (dict(q_heads=-1), -1), (dict(k_heads=-1), -1), (dict(D=0), -1), (dict(rotary=-2), -1),
    (dict(rotary=63), -1), (dict(rotary=66), -1), (dict(layout=2), -1), (dict(dtype=2), -1), (dict(wtype=2), -1),
    (dict(mscale=math.nan), -1), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=math.nan), -1),
    (dict(eps=math.inf), -1), (dict(D=257), -2), (dict(q_heads=1025), -2), (dict(k_heads=1025), -2),
    (dict(T=(1 << 23) + 1), -2), (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(pos=None), -1), (dict(freq=None), -1), (dict(qt=-1), -1), (dict(kh=-1), -1), (dict(qot=0), -1),
    (dict(koh=63), -1),
]


@pytest.mark.parametrize("kw,status", NORM + [(dict(T=0, q=None), 0), (dict(q_heads=0, k_heads=0, q=None, k=None), 0)])
def test_norm_refuses_before_launch(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(gq=None), -1), (dict(gk=None), -1), (dict(gqt=-1), -1), (dict(ws=None), -3), (dict(ws=FAKE + 8), -3),
    (dict(bytes=256 + 4 * 2 * 64 * 4 - 1), -3), (dict(T=0, q=None, dqw=None, dkw=None, ws=None), 0),
])
def test_norm_backward_refuses_before_launch(kw, status):
    assert norm_backward(**kw) == status


def test_norm_backward_workspace_size():
    size = sv.sv_qk_norm_rope_backward_workspace_size
    assert size(0, 64) == 256 and size(10, 128) == 256 + 10 * 2 * 128 * 4 and size(10 ** 6, 128) == size(5000, 128)
    for bad in ((-1, 64), ((1 << 23) + 1, 64), (4, 0), (4, 257)):
        assert size(*bad) == 0


def append_normed(c=None, **kw):
    a = dict(stream=None, B=4, T=9, q_heads=4, dtype=1, rotary=64, layout=0, freq=FAKE, mscale=1.0, pos=None, wtype=1,
             qw=FAKE, kw=None, eps=1e-5, q=FAKE, qt=256, qh=64, qo=FAKE, qot=256, qoh=64, k=FAKE, kt=128, kh=64, v=FAKE,
             vt=128, vh=64, qs=FAKE, kl=FAKE)
    c = cache() if c is None else c
    return attn._attn_lib().sv_kv_append_normed(*{**a, **kw}.values(), ctypes.addressof(c))


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(B=(1 << 18) + 1), -2), (dict(q_heads=1025), -2), (dict(dtype=2), -1),
    (dict(rotary=66), -1), (dict(layout=5), -1), (dict(freq=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(q=None), -1), (dict(qo=None), -1), (dict(qs=None), -1), (dict(kl=None), -1), (dict(kt=-1), -1),
    (dict(qot=32), -1), (dict(wtype=2), -1), (dict(wtype=-1), -1), (dict(eps=0.0), -1), (dict(eps=math.nan), -1),
    (dict(T=0, k=None), 0), (dict(B=0, k=None, q=None), 0),
])
def test_append_normed_refuses_before_launch(kw, status):
    assert append_normed(**kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_append_normed_refuses_bad_caches(kw, status):
    assert append_normed(cache(**kw)) == status


def pages(**kw):
    a = dict(stream=None, B=4, T=9, page=16, max_pages=8, num_pages=40, kl=FAKE, shared=None, qs=FAKE, table=FAKE, stride=8,
             held=FAKE, free=FAKE, count=FAKE, granted=FAKE, slots=FAKE, positions=None, ws=None, bytes=0)
    return attn._attn_lib().sv_kv_pages(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(B=(1 << 18) + 1), -2), (dict(T=(1 << 23) + 1), -2), (dict(page=0), -1),
    (dict(page=24), -1), (dict(page=1 << 17), -2), (dict(max_pages=-1), -1), (dict(num_pages=-1), -1),
    (dict(max_pages=1 << 27), -2), (dict(kl=None), -1), (dict(table=None), -1), (dict(held=None), -1),
    (dict(free=None), -1), (dict(count=None), -1), (dict(stride=7), -1), (dict(stride=0), -1), (dict(stride=-8), -1),
    (dict(qs=None), -1), (dict(B=2000), -3), (dict(T=100000), -3), (dict(B=2000, ws=FAKE, bytes=1000), -3),
    (dict(B=2000, ws=FAKE + 8, bytes=1 << 30), -3), (dict(B=0, kl=None), 0),
])
def test_pages_refuse_before_launch(kw, status):
    assert pages(**kw) == status


def test_pages_workspace_size():
    size = sv.sv_kv_pages_workspace_size
    assert size(1024, 0) == 256 and size(1025, 0) >= 256 + 1025 * 20 and size(3, 1 << 20) > 256
    assert size(-1, 0) == 0 and size(1, -1) == 0 and size((1 << 18) + 1, 0) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    i = lambda *n: torch.zeros(n, dtype=torch.int32)
    for call in (lambda: sv.sv_qk_norm_rope(x, x), lambda: sv.sv_qk_norm_rope_backward(x, x, x, x),
                 lambda: sv.sv_kv_append_normed(x, x, c, c, i(1, 2), i(2), i(1)),
                 lambda: sv.sv_kv_pages(i(1, 2), i(1), i(3), i(1), i(1), page_size=16)):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def sinks(c=None, **kw):
    a = dict(stream=None, B=4, T=9, q_heads=4, q=FAKE, qt=256, qh=64)
    b = dict(qs=FAKE, kl=FAKE, max_q=5, max_kv=100, scale=0.125, window=0, sinks=4, out=FAKE, ot=256, oh=64, lse=None,
             ws=FAKE, bytes=1 << 40)
    c = cache() if c is None else c
    a.update({k: v for k, v in kw.items() if k in a})
    b.update({k: v for k, v in kw.items() if k in b})
    return attn._attn_lib().sv_paged_attention_sinks(*a.values(), ctypes.addressof(c), *b.values())


def shared(c=None, **kw):
    a = dict(stream=None, B=4, T=9, q_heads=4, q=FAKE, qt=256, qh=64)
    b = dict(qs=FAKE, kl=FAKE, groups=2, gs=FAKE, sl=FAKE, max_q=5, max_group=5, max_shared=100, max_own=100, scale=0.125,
             out=FAKE, ot=256, oh=64, lse=None, ws=FAKE, bytes=1 << 40)
    c = cache() if c is None else c
    a.update({k: v for k, v in kw.items() if k in a})
    b.update({k: v for k, v in kw.items() if k in b})
    return attn._attn_lib().sv_paged_attention_shared(*a.values(), ctypes.addressof(c), *b.values())


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused_by_the_attention_calls(kw, status):
    for call in (sinks, shared):
        assert call(cache(**kw)) == status, call.__name__


ATTENTION = [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(B=(1 << 18) + 1), -2), (dict(q_heads=3), -1), (dict(q_heads=0), -1),
    (dict(q_heads=1026), -2), (dict(q=None), -1), (dict(q=FAKE + 8), -1), (dict(out=None), -1), (dict(out=FAKE + 2), -1),
    (dict(qt=250), -1), (dict(qh=4), -1), (dict(ot=-8), -1), (dict(ot=0), -1), (dict(oh=32), -1), (dict(qs=None), -1),
    (dict(kl=None), -1), (dict(max_q=-1), -1), (dict(scale=0.0), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(T=0, q=None), 0), (dict(B=0, q=None), 0),
]


@pytest.mark.parametrize("kw,status", ATTENTION + [
    (dict(max_kv=-1), -1), (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(sinks=-1, T=0), -1),
    (dict(ws=None, max_kv=5000), -3), (dict(ws=FAKE + 4, max_kv=5000), -3),
    (dict(bytes=8, max_kv=50000, window=3000), -3),
])
def test_sinks_refuse_before_launch(kw, status):
    assert sinks(**kw) == status


@pytest.mark.parametrize("kw,status", ATTENTION + [
    (dict(max_group=-1), -1), (dict(max_shared=-1), -1), (dict(max_own=-1), -1), (dict(groups=-1), -1),
    (dict(groups=(1 << 18) + 1), -2), (dict(gs=None), -1), (dict(sl=None), -1), (dict(ws=None), -3), (dict(ws=FAKE + 4), -3),
    (dict(bytes=8), -3), (dict(groups=0, gs=None, sl=None, ws=None, max_own=5000), -3),
])
def test_shared_refuses_before_launch(kw, status):
    assert shared(**kw) == status


def test_attention_workspace_sizes():
    size = sv.sv_paged_attention_sinks_workspace_size
    plain = sv.sv_paged_attention_workspace_size
    assert size(4, 4, 32, 8, 128, 1, 100000, 0, 4) == plain(4, 4, 32, 8, 128, 1, 100000)
    assert size(4, 4, 32, 8, 128, 1, 100000, 200, 4) == 256  # what a row sees is not divided
    assert 256 < size(4, 4, 32, 8, 128, 1, 100000, 4096, 4) < plain(4, 4, 32, 8, 128, 1, 100000)
    assert size(4, 4, 32, 8, 128, 1, 2 ** 40, 2 ** 40, 2 ** 40) == plain(4, 4, 32, 8, 128, 1, 2 ** 40)
    for bad in ((-1, 4, 32, 8, 128, 1, 5, 1, 1), (4, 4, 30, 8, 128, 1, 5, 1, 1), (4, 4, 32, 8, 128, 1, 5, -1, 1),
                (4, 4, 32, 8, 128, 1, 5, 1, -1)):
        assert size(*bad) == 0
    size = sv.sv_paged_attention_shared_workspace_size
    assert size(4, 4, 1, 32, 8, 128, 1, 4, 100, 100) >= 256 + 2 * 4 * 32 * (128 * 4 + 8)
    assert size(4, 4, 0, 32, 8, 128, 1, 4, 100, 5000) == plain(4, 4, 32, 8, 128, 1, 5000)
    for bad in ((-1, 4, 1, 32, 8, 128), (4, 4, -1, 32, 8, 128), (4, 4, (1 << 18) + 1, 32, 8, 128), (4, 4, 1, 30, 8, 128),
                (4, 4, 1, 32, 8, 128, -1), (4, 4, 1, 32, 8, 128, 1, -1), (4, 4, 1, 32, 8, 128, 1, 1, -1),
                (4, 4, 1, 32, 8, 128, 1, 1, 1, -1)):
        assert size(*bad) == 0, bad
