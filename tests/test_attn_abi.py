"""specverify_attn.h without a GPU: exported symbols, binding signatures,
frequency tables, and refusals made on the host before anything is launched."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from draft_token_verification_spec_amd import attn
from oracle import attn as oa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "specverify_attn.h")

pytestmark = pytest.mark.skipif(not os.path.exists(sv.lib_path()), reason="libspecverify.so not built")

FAKE = 0x10000  # never dereferenced: the calls below fail host checks or have nothing to do


class PagedCache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("dtype", "heads", "head_dim", "page_size", "num_pages", "max_pages")]
                + [("page_table", ctypes.c_void_p), ("page_table_stride", ctypes.c_int64), ("k", ctypes.c_void_p),
                   ("v", ctypes.c_void_p)]
                + [(f"{kv}_{n}_stride", ctypes.c_int64) for kv in "kv" for n in ("page", "token", "head")]
                + [("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)])


def text():
    return re.sub(r"/\*.*?\*/", " ", open(HEADER).read(), flags=re.S)


def prototypes():
    out = {}
    for m in re.finditer(r"^\s*(size_t|int)\s+(sv_\w+)\s*\(([^;]*)\)\s*;", text(), re.M):
        out[m.group(2)] = (m.group(1), [" ".join(q.split()) for q in m.group(3).split(",")])
    return out


def ctype_of(decl):
    if "*" in decl:
        return ctypes.c_void_p
    return {"int": ctypes.c_int, "size_t": ctypes.c_size_t, "int64_t": ctypes.c_int64, "float": ctypes.c_float,
            "double": ctypes.c_double, "int32_t": ctypes.c_int32}[decl.replace("const ", "").split()[0]]


def test_binding_signatures_match_header_prototypes():
    protos = prototypes()
    assert set(protos) == set(attn._SIGNATURES)
    lib = ctypes.CDLL(sv.lib_path())
    for name, (ret, params) in protos.items():
        assert hasattr(lib, name) and name in sv.__all__ and hasattr(sv, name)
        res, args = attn._SIGNATURES[name]
        assert res == ctype_of(ret), name
        assert args == [ctype_of(p) for p in params], name


def test_cache_struct_matches_header():
    body = re.search(r"typedef struct \{(.*?)\} sv_paged_cache;", text(), re.S).group(1)
    letters = {ctypes.c_int: "i", ctypes.c_int64: "q", ctypes.c_void_p: "P"}
    fields = []
    for decl in filter(None, (" ".join(d.split()) for d in body.split(";"))):
        kind, names = re.match(r"((?:const )?\w+\s?\*?)\s*(.*)", decl).groups()
        fields += [(n.strip(), ctype_of(kind)) for n in names.split(",")]
    assert fields == PagedCache._fields_
    packed = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), attn._CACHE.format.lstrip("@"))
    assert packed == "".join(letters[t] for _, t in fields) and attn._CACHE.size == ctypes.sizeof(PagedCache)


def test_header_constants_match_binding():
    t = text()
    for name in ("SV_E4M3", "SV_ATTN_MAX_HEAD_DIM", "SV_ATTN_MAX_HEADS", "SV_ATTN_MAX_PAGE", "SV_ATTN_MAX_TOKENS"):
        assert int(re.search(rf"#define {name} (\d+)", t).group(1)) == getattr(sv, name), name
    assert re.search(r"#define SV_ATTN_MAX_ROWS \(1 << 23\)", t) and sv.SV_ATTN_MAX_ROWS == 1 << 23
    for prefix, table in (("SV_ROPE_", sv.SV_ROPE_SCALINGS), ("SV_ROPE_", sv.SV_ROPE_LAYOUTS)):
        for word, value in table.items():
            assert re.search(rf"{prefix}{word.upper()} = {value}\b", t), word


@pytest.mark.parametrize("kind,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("ramp", dict(factor=16.0, original_len=4096.0)), ("ramp", dict(factor=1.0, original_len=40.0)),
    ("ramp", dict(factor=4.0, original_len=1.0, low=30.0, high=32.0)),
    ("bands", dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0)),
])
@pytest.mark.parametrize("rotary,base", [(128, 10000.0), (64, 500000.0), (6, 100.0)])
def test_frequencies(kind, kw, rotary, base):
    f, m = sv.sv_rope_frequencies(rotary, base, kind, **kw)
    want, wm = oa.frequencies(rotary, base, kind, **{"high": 32.0, **kw})
    # each side: one pow and a few roundings of binary64; pow's argument log(base) * 2 i / d is under 2^4 * ulp
    assert np.allclose(f.numpy(), want, rtol=1e-14, atol=0) and m == pytest.approx(wm, rel=2 ** -23)
    assert f.dtype == torch.float64 and f.shape == (rotary // 2,)


def test_frequencies_refusals():
    ok = dict(rotary_dim=64, base=1e4, scaling="plain")
    for bad in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(base=0.0), dict(base=-1.0), dict(base=math.nan),
                dict(base=math.inf), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.nan),
                dict(scaling="base", factor=math.inf), dict(scaling="base", factor=2.0, rotary_dim=2),
                dict(scaling="ramp", factor=2.0), dict(scaling="bands", factor=2.0, original_len=10.0, low=4.0, high=4.0),
                dict(scaling="bands", factor=2.0, original_len=10.0, low=0.0, high=4.0),
                dict(scaling="ramp", factor=2.0, original_len=10.0, base=1.0)):
        with pytest.raises(RuntimeError, match="invalid argument"):
            a = {**ok, **bad}
            sv.sv_rope_frequencies(a.pop("rotary_dim"), a.pop("base"), a.pop("scaling"), **a)
    with pytest.raises(ValueError):
        sv.sv_rope_frequencies(64, scaling="other")
    f, m = sv.sv_rope_frequencies(0)
    assert f.numel() == 0 and m == 1.0
    lib = attn._attn_lib()
    assert lib.sv_rope_frequencies(8, 1e4, 7, 1.0, 0.0, 1.0, 2.0, FAKE, FAKE) == -1
    assert lib.sv_rope_frequencies(8, 1e4, 0, 1.0, 0.0, 1.0, 2.0, None, FAKE) == -1
    assert lib.sv_rope_frequencies(8, 1e4, 0, 1.0, 0.0, 1.0, 2.0, FAKE, None) == -1


def rope(**kw):
    a = dict(stream=None, T=4, heads=2, D=64, rotary=64, layout=0, backward=0, dtype=1, x=FAKE, xt=128, xh=64, pos=FAKE,
             freq=FAKE, mscale=1.0, out=FAKE, ot=128, oh=64)
    return attn._attn_lib().sv_rope(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(heads=-1), -1), (dict(D=0), -1), (dict(rotary=-2), -1), (dict(rotary=63), -1),
    (dict(rotary=66), -1), (dict(layout=2), -1), (dict(dtype=2), -1), (dict(mscale=math.nan), -1),
    (dict(D=257), -2), (dict(heads=1025), -2), (dict(T=(1 << 23) + 1), -2), (dict(x=None), -1), (dict(out=None), -1),
    (dict(pos=None), -1), (dict(freq=None), -1), (dict(xt=-1), -1), (dict(ot=0), -1), (dict(oh=63), -1),
    (dict(T=0, x=None), 0), (dict(heads=0, x=None), 0),
])
def test_rope_refuses_before_launch(kw, status):
    assert rope(**kw) == status


def cache(**kw):
    a = dict(dtype=1, heads=2, head_dim=64, page_size=16, num_pages=5, max_pages=3, page_table=FAKE, page_table_stride=3,
             k=FAKE, v=FAKE, k_page_stride=2048, k_token_stride=128, k_head_stride=64, v_page_stride=2048,
             v_token_stride=128, v_head_stride=64, k_scale=None, v_scale=None)
    return PagedCache(**{**a, **kw})


BAD_CACHES = [
    (dict(dtype=0), -1), (dict(dtype=3), -1), (dict(heads=0), -1), (dict(head_dim=8), -1), (dict(head_dim=72), -1),
    (dict(page_size=0), -1), (dict(page_size=24), -1), (dict(num_pages=-1), -1), (dict(max_pages=-1), -1),
    (dict(head_dim=272), -2), (dict(heads=1025), -2), (dict(page_size=1 << 17), -2), (dict(max_pages=1 << 27), -2),
    (dict(page_table=None), -1), (dict(page_table_stride=2), -1), (dict(page_table_stride=-3), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(k=FAKE + 8), -1), (dict(k_head_stride=60), -1),
    (dict(k_token_stride=32), -1), (dict(v_head_stride=0), -1), (dict(v_page_stride=0), -1), (dict(k_page_stride=-8), -1),
    (dict(dtype=2), -1), (dict(dtype=2, k_scale=FAKE), -1),
    (dict(dtype=2, k_scale=FAKE, v_scale=FAKE, k_head_stride=72), -1),
]


def append(c=None, **kw):
    a = dict(stream=None, B=4, T=9, q_heads=4, dtype=1, rotary=64, layout=0, freq=FAKE, mscale=1.0, pos=None,
             q=FAKE, qt=256, qh=64, qo=FAKE, qot=256, qoh=64, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, qs=FAKE,
             kl=FAKE)
    c = cache() if c is None else c
    return attn._attn_lib().sv_kv_append(*{**a, **kw}.values(), ctypes.addressof(c))


def gather(c=None, **kw):
    a = dict(stream=None, B=4, T=9, dtype=1)
    b = dict(rs=FAKE, kb=None, ko=FAKE, vo=FAKE)
    c = cache() if c is None else c
    a.update({k: v for k, v in kw.items() if k in a})
    b.update({k: v for k, v in kw.items() if k in b})
    return attn._attn_lib().sv_kv_gather(*a.values(), ctypes.addressof(c), *b.values())


def attention(c=None, **kw):
    a = dict(stream=None, B=4, T=9, q_heads=4, q=FAKE, qt=256, qh=64)
    b = dict(qs=FAKE, kl=FAKE, max_q=5, max_kv=100, scale=0.125, window=0, out=FAKE, ot=256, oh=64, lse=None, ws=FAKE,
             bytes=1 << 40)
    c = cache() if c is None else c
    a.update({k: v for k, v in kw.items() if k in a})
    b.update({k: v for k, v in kw.items() if k in b})
    return attn._attn_lib().sv_paged_attention(*a.values(), ctypes.addressof(c), *b.values())


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(kw, status):
    for call in (append, gather, attention):
        # a queries' count that divides by the cache's heads is not what is refused here
        assert call(cache(**kw)) == status, call.__name__


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(B=(1 << 18) + 1), -2), (dict(T=(1 << 23) + 1), -2),
    (dict(q_heads=-1), -1), (dict(q_heads=1025), -2), (dict(dtype=2), -1), (dict(rotary=66), -1), (dict(rotary=31), -1),
    (dict(layout=5), -1), (dict(freq=None), -1), (dict(mscale=math.inf), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(q=None), -1), (dict(qo=None), -1), (dict(qs=None), -1), (dict(kl=None), -1), (dict(kt=-1), -1),
    (dict(qot=32), -1), (dict(qoh=0), -1), (dict(T=0, k=None), 0), (dict(B=0, k=None, q=None), 0),
])
def test_append_refuses_before_launch(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(T=(1 << 23) + 1), -2), (dict(dtype=2), -1), (dict(rs=None), -1),
    (dict(ko=FAKE + 4), -1), (dict(T=0), 0), (dict(B=0), 0), (dict(ko=None, vo=None), 0),
])
def test_gather_refuses_before_launch(kw, status):
    assert gather(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(B=(1 << 18) + 1), -2), (dict(q_heads=3), -1), (dict(q_heads=0), -1),
    (dict(q_heads=1026), -2), (dict(q=None), -1), (dict(q=FAKE + 8), -1), (dict(out=None), -1), (dict(out=FAKE + 2), -1),
    (dict(qt=250), -1), (dict(qh=4), -1), (dict(ot=-8), -1), (dict(ot=0), -1), (dict(oh=32), -1), (dict(qs=None), -1),
    (dict(kl=None), -1), (dict(max_q=-1), -1), (dict(max_kv=-1), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(window=-1), -1), (dict(ws=None, max_kv=5000), -3),
    (dict(ws=FAKE + 4, max_kv=5000), -3), (dict(bytes=8, max_kv=5000), -3), (dict(T=0, q=None), 0), (dict(B=0, q=None), 0),
])
def test_attention_refuses_before_launch(kw, status):
    assert attention(**kw) == status


def test_missing_cache_is_refused():
    lib = attn._attn_lib()
    assert lib.sv_kv_gather(None, 4, 9, 1, None, FAKE, None, FAKE, FAKE) == -1


def test_attention_workspace_size():
    size = sv.sv_paged_attention_workspace_size
    assert size(4, 20, 32, 8, 128, 5, 300) == 256  # no context is split: no workspace is needed
    assert size(4, 20, 32, 8, 128, 5, 5000) > 256 + 20 * 32 * 128 * 4
    assert size(0, 0, 32, 8, 128) >= 256
    for bad in ((-1, 20, 32, 8, 128), (4, -1, 32, 8, 128), (4, 20, 30, 8, 128), (4, 20, 32, 0, 128), (4, 20, 32, 8, 24),
                (4, 20, 32, 8, 512), (4, 20, 2048, 8, 128)):
        assert size(*bad) == 0, bad


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    i = lambda *n: torch.zeros(n, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="HIP device"):
        sv.sv_rope(x, torch.zeros(2, dtype=torch.int64), f)
    with pytest.raises(ValueError, match="HIP device"):
        sv.sv_kv_append(x, x, c, c, i(1, 2), i(2), i(1))
    with pytest.raises(ValueError, match="HIP device"):
        sv.sv_kv_gather(c, c, i(1, 2), i(2), 3)
    with pytest.raises(ValueError, match="HIP device"):
        sv.sv_paged_attention(x, c, c, i(1, 2), i(2), i(1))


def test_attention_rows_and_heads_stay_within_32_bits():
    """A request's rows times its query heads are counted in 32 bits."""
    assert attention(T=1 << 23, q_heads=256, max_kv=100) == -2
    assert sv.sv_paged_attention_workspace_size(4, 1 << 23, 256, 2, 64) == 0
    assert sv.sv_paged_attention_workspace_size(4, (1 << 23) - 1, 256, 2, 64) >= 256
