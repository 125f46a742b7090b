"""sv_kv_append and sv_kv_gather on the GPU against the oracle.

Tolerances.  Values (not turned) are rounded once from the input, so stored
rows are compared exactly.  Turned keys carry the rotation's error (see
test_gpu_rope) into the rounding: a bf16 key is off by at most that and 2^-8 of
its value, an 8-bit one by at most that and half a step of its type, 2^-4 of its
value and at least 2^-10 of its scale; its scale may be the neighbouring power
of two only where the largest magnitude is within the rotation's error of a
border."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import attn as oa

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
I32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")


def new_cache(kind, pages, page, heads, D, order="tokens"):
    """Caches full of a marker, so that what is not written shows."""
    shape = (pages, page, heads, D) if order == "tokens" else (pages, heads, page, D)
    c = {}
    for n in ("k", "v"):
        x = torch.full(shape, 3.0, device="cuda", dtype=torch.bfloat16)
        if kind == "e4m3":
            x = x.float().to(torch.float8_e4m3fn)
            c[n + "_scale"] = torch.full((pages, heads, page), 128, dtype=torch.uint8, device="cuda")
        else:
            c[n + "_scale"] = None
        c[n + "_cache"] = x if order == "tokens" else x.transpose(1, 2)
    return c


def values(c, n):
    x = c[n + "_cache"].float().double().cpu().numpy()
    if c[n + "_scale"] is None:
        return x
    return x * np.exp2(c[n + "_scale"].cpu().numpy().astype(float) - 127).transpose(0, 2, 1)[..., None]


def tables(new, total, page, spare=2, seed=0):
    need = [-(-max(t, 0) // page) for t in total]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(total), max(max(need), 1)), -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return sum(need) + spare, table, np.cumsum([0] + list(new))


CASES = [  # new tokens and lengths with them, page, kv heads, q heads, D, rotary
    ([5, 5, 5], [5, 37, 100], 16, 2, 8, 128, 128),
    ([1], [1], 16, 1, 1, 64, 64),
    ([1, 1, 1, 1], [1000, 1, 64, 65], 64, 8, 32, 128, 128),
    ([0, 3, 0, 17, 0], [9, 3, 0, 40, 5], 8, 5, 5, 80, 40),
    ([130, 1, 70], [130, 4, 200], 32, 4, 0, 96, 96),
    ([6, 4], [3, 4], 1, 3, 6, 16, 16),  # the first request's first rows lie before its place 0
    ([33, 2], [50, 2], 128, 1, 7, 256, 64),
]


@pytest.mark.parametrize("cache,order", [("bf16", "tokens"), ("bf16", "heads"), ("e4m3", "tokens"), ("e4m3", "heads")])
@pytest.mark.parametrize("dtype,layout", [("bf16", "half"), ("f32", "interleaved")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_matches_the_oracle(cache, order, dtype, layout, case):
    new, total, page, heads, q_heads, D, rotary = CASES[case]
    g = torch.Generator(device="cuda").manual_seed(case)
    pages, table, start = tables(new, total, page, seed=case)
    c = new_cache(cache, pages, page, heads, D, order)
    T = start[-1] + 3  # rows behind the last request
    qkv = (torch.randn((T, q_heads + 2 * heads, D), generator=g, device="cuda")
           * torch.exp(2 * torch.randn((T, 1, 1), generator=g, device="cuda"))).to(DT[dtype])
    q, k, v = qkv.split([q_heads, heads, heads], 1)
    f, _ = sv.sv_rope_frequencies(rotary, device="cuda")
    out = {"q": torch.full((T, q_heads, D), 7.0, device="cuda", dtype=DT[dtype])}
    o = sv.sv_kv_append(k, v, c["k_cache"], c["v_cache"], I32(table), I32(start), I32(total), q=q if q_heads else None,
                        freq=f, layout=layout, mscale=1.125, k_scale=c["k_scale"], v_scale=c["v_scale"], out=out)
    place = np.array([oa.place_of(start, total, b, i) for b in range(len(new)) for i in range(new[b])], int)
    n = lambda x: x.double().cpu().numpy()
    turned = lambda x: oa.rope(n(x)[: start[-1]], place, f.cpu().numpy(), layout, 1.125)
    rot_err = lambda x: (np.abs(n(x)[: start[-1]]).max(-1, keepdims=True) * 2 * 1.125 * 2.0 ** -21)
    if q_heads:
        want = turned(q)
        tol = rot_err(q) + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 0) * (1 + 2.0 ** -8)
        assert (np.abs(n(o["q"])[: start[-1]] - want) <= tol).all()
        assert (n(o["q"])[start[-1]:] == 7.0).all()
    written = np.zeros((pages, page), bool)
    kv, vv = values(c, "k"), values(c, "v")
    kw, kerr, vn = turned(k), rot_err(k), n(v)
    for b in range(len(new)):
        for i in range(new[b]):
            r, p = start[b] + i, oa.place_of(start, total, b, i)
            if p < 0:
                continue
            at = (table[b, p // page], p % page)
            assert not written[at]
            written[at] = True
            if cache == "bf16":
                assert np.array_equal(vv[at], n(v[r].to(torch.bfloat16)))
                assert (np.abs(kv[at] - kw[r]) <= kerr[r] + np.abs(kw[r]) * 2.0 ** -8 * (1 + 2.0 ** -8)).all()
            else:
                codes, e = oa.quantise(vn[r])
                assert np.array_equal(c["v_scale"][at[0], :, at[1]].cpu().numpy(), e + 127)
                assert np.array_equal(vv[at], oa.e4m3_values()[codes] * 2.0 ** e[:, None])
                lo, hi = oa.quantise(kw[r] * (1 - 2.0 ** -19))[1], oa.quantise(kw[r] * (1 + 2.0 ** -19))[1]
                e = c["k_scale"][at[0], :, at[1]].cpu().numpy().astype(int) - 127
                assert ((lo <= e) & (e <= hi)).all()
                half = np.maximum(np.abs(kw[r]) * 2.0 ** -4, 2.0 ** (e[:, None] - 10))
                assert (np.abs(kv[at] - kw[r]) <= (kerr[r] + half) * (1 + 2.0 ** -4)).all()
    for x in (kv, vv):
        assert (x[~written] == (3.0 if cache == "bf16" else 6.0)).all()


def test_append_drops_absent_pages_and_reads_nothing_beyond():
    page, heads, D = 8, 2, 64
    for kind in ("bf16", "e4m3"):
        c = new_cache(kind, 4, page, heads, D)
        table = I32([[0, -1, 9], [2147483647, 1, -5]])
        x = torch.randn((44, heads, D), device="cuda").bfloat16()
        # request 0: 40 rows over three table entries and beyond them; request 1: 4 rows on a good page
        sv.sv_kv_append(x, x, c["k_cache"], c["v_cache"], table, I32([0, 40, 44]), I32([40, 12]), k_scale=c["k_scale"],
                        v_scale=c["v_scale"])
        for n in ("k", "v"):
            got = values(c, n)
            mark = 3.0 if kind == "bf16" else 6.0
            assert (got[2:] == mark).all() and (got[1, 4:] == mark).all()
            back = sv.sv_kv_gather(c["k_cache"], c["v_cache"], table, I32([0, 30, 44]), 44, k_scale=c["k_scale"],
                                   v_scale=c["v_scale"], dtype=torch.float32)[n].double().cpu().numpy()
            assert np.array_equal(back[:8], got[0]) and (back[8:38] == 0).all() and np.array_equal(back[38:42], got[1, :4])
            if kind == "bf16":
                assert np.array_equal(got[0], x[:8].double().cpu().numpy())
                assert np.array_equal(got[1, :4], x[40:].double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_special_values(dtype):
    rows = torch.randn((12, 1, 64), device="cuda").to(DT[dtype])
    rows[0] = 0
    rows[1] = -0.0
    rows[2, 0, 5] = float("inf")
    rows[3, 0, 6] = float("nan")
    rows[4] = float("-inf")
    rows[5] *= 2.0 ** -130
    rows[6] = torch.finfo(DT[dtype]).max
    rows[7] = 448.0
    rows[8] = 449.0 if dtype == "f32" else 450.0
    rows[9] = 2.0 ** -126
    rows[10, 0, 1:] = 0
    c = new_cache("e4m3", 2, 16, 1, 64)
    t = I32([[1]])
    a = lambda: sv.sv_kv_append(rows, rows, c["k_cache"], c["v_cache"], t, I32([0, 12]), I32([12]), k_scale=c["k_scale"],
                                v_scale=c["v_scale"])
    a()
    codes, e = oa.quantise(rows.double().cpu().numpy())
    for n in ("k", "v"):
        got = c[n + "_cache"][1, :12].view(torch.uint8).cpu().numpy()
        nan = (codes & 127) == 127
        assert np.array_equal(c[n + "_scale"][1, 0, :12].cpu().numpy(), e[:, 0] + 127)
        assert (((got & 127) == 127) == nan).all() and np.array_equal(got[~nan], codes[~nan])


def test_append_positions_and_page_sharing():
    """Explicit positions turn keys and queries in place of the places; two requests read one shared page."""
    f, _ = sv.sv_rope_frequencies(64, device="cuda")
    c = new_cache("bf16", 4, 4, 1, 64)
    x = torch.randn((5, 1, 64), device="cuda").bfloat16()
    pos = torch.tensor([1000, 2, 77, 5, 123456], device="cuda")
    o = sv.sv_kv_append(x, x, c["k_cache"], c["v_cache"], I32([[2, 0], [2, 1]]), I32([0, 3, 5]), I32([7, 6]), q=x, freq=f,
                        positions=pos)
    want = sv.sv_rope(x, pos, f)
    assert torch.equal(o["q"], want)
    assert torch.equal(c["k_cache"][0, :3], want[:3]) and torch.equal(c["k_cache"][1, :2], want[3:])
    assert torch.equal(c["v_cache"][1, :2], x[3:])


def test_append_queries_in_place():
    f, _ = sv.sv_rope_frequencies(128, device="cuda")
    c = new_cache("bf16", 2, 16, 2, 128)
    qkv = torch.randn((9, 8, 128), device="cuda").bfloat16()
    keep = qkv.clone()
    q, k, v = qkv.split([4, 2, 2], 1)
    sv.sv_kv_append(k, v, c["k_cache"], c["v_cache"], I32([[1]]), I32([0, 9]), I32([9]), q=q, freq=f, out={"q": q})
    pos = torch.arange(9, device="cuda")
    assert torch.equal(q, sv.sv_rope(keep[:, :4], pos, f)) and torch.equal(qkv[:, 4:], keep[:, 4:])
    assert torch.equal(c["k_cache"][1, :9], sv.sv_rope(keep[:, 4:6], pos, f))


@pytest.mark.parametrize("cache,order,dtype", [("bf16", "tokens", "bf16"), ("bf16", "heads", "f32"),
                                               ("e4m3", "tokens", "f32"), ("e4m3", "heads", "bf16")])
@pytest.mark.parametrize("lengths,begin,page,heads,D", [
    ([1], [0], 16, 1, 16), ([100, 0, 37], [0, 5, 11], 16, 2, 128), ([5, 64, 129], [3, 0, 1], 64, 5, 80),
    ([700], [1], 8, 8, 256), ([3, 2, 1, 0], [0, 0, 0, 0], 1, 3, 48),
])
def test_gather_matches_the_oracle(cache, order, dtype, lengths, begin, page, heads, D):
    g = np.random.default_rng(len(lengths) + D)
    pages, table, start = tables(lengths, [n + b for n, b in zip(lengths, begin)], page)
    table[-1, -1] = pages + 5  # absent
    c = new_cache(cache, pages, page, heads, D, order)
    for n in ("k", "v"):
        x = torch.from_numpy(g.standard_normal((pages, page, heads, D)).astype(np.float32)).cuda()
        c[n + "_cache"].copy_(x.to(c[n + "_cache"].dtype))
        if cache == "e4m3":
            c[n + "_scale"].copy_(torch.from_numpy(g.integers(10, 230, (pages, heads, page)).astype(np.uint8)))
    start = start + 2
    T = int(start[-1]) + 2
    out = {n: torch.full((T, heads, D), -1.0, device="cuda", dtype=DT[dtype]) for n in ("k", "v")}
    sv.sv_kv_gather(c["k_cache"], c["v_cache"], I32(table), I32(start), T, kv_begin=I32(begin), k_scale=c["k_scale"],
                    v_scale=c["v_scale"], dtype=DT[dtype], out=out)
    want = oa.gather(dict(k=values(c, "k"), v=values(c, "v"), table=table), start, T, begin)
    for n in out:
        w = np.where(np.isnan(want[n]), -1.0, want[n])
        assert np.array_equal(out[n].double().cpu().numpy(), w), n


def test_gather_of_one_of_the_two():
    """The C call with one output missing writes the other alone."""
    from draft_token_verification_spec_amd import attn

    c = new_cache("bf16", 2, 8, 1, 16)
    c["v_cache"].copy_(torch.randn((2, 8, 1, 16)))
    dev = torch.cuda.current_device()
    table, start = I32([[1]]), I32([0, 5])
    p = attn._paged(dev, 1, c["k_cache"], c["v_cache"], table, None, None)[0]
    out = torch.zeros((5, 1, 16), device="cuda")
    attn._call(dev, "sv_kv_gather", 1, 5, sv.SV_F32, p, start.data_ptr(), None, None, out.data_ptr())
    assert torch.equal(out, c["v_cache"][1, :5].float())


def test_round_trip_through_an_8_bit_cache():
    """Written and read back, a row is off by at most half a step of the type."""
    x = (torch.randn((300, 4, 128), device="cuda") * torch.exp(3 * torch.randn((300, 4, 1), device="cuda"))).bfloat16()
    pages, table, start = tables([100, 200], [100, 200], 32)
    c = new_cache("e4m3", pages, 32, 4, 128)
    cache = (c["k_cache"], c["v_cache"], I32(table))
    s = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    sv.sv_kv_append(x, -x, *cache, I32(start), I32([100, 200]), **s)
    back = sv.sv_kv_gather(*cache, I32(start), 300, **s)
    assert torch.equal(back["k"], -back["v"])
    top = x.double().abs().amax(-1, keepdim=True)
    half = torch.maximum(x.double().abs() * 2.0 ** -4, top / 224 * 2.0 ** -10)
    assert ((back["k"].double() - x.double()).abs() <= half).all()


def test_kv_refusals():
    c = new_cache("bf16", 2, 8, 2, 64)
    x = torch.randn((4, 2, 64), device="cuda").bfloat16()
    t, qs, kl = I32([[0]]), I32([0, 4]), I32([4])
    ok = (x, x, c["k_cache"], c["v_cache"], t, qs, kl)
    sv.sv_kv_append(*ok)

    def swap(i, y):
        a = list(ok)
        a[i] = y
        return a

    for i, y, err in ((0, x[:, :1], ValueError), (0, x.float(), TypeError), (1, x[:3], ValueError),
                      (2, c["k_cache"].float(), TypeError), (3, c["v_cache"][:1], ValueError),
                      (4, t.long(), TypeError), (4, I32([[0], [0]]), ValueError), (5, I32([0]), ValueError),
                      (5, qs.cpu(), ValueError), (6, kl.long(), TypeError), (0, None, TypeError),
                      (0, x.half(), TypeError)):
        with pytest.raises(err):
            sv.sv_kv_append(*swap(i, y))
    with pytest.raises(ValueError, match="scales"):
        sv.sv_kv_append(*ok, k_scale=torch.zeros((2, 2, 8), dtype=torch.uint8, device="cuda"))
    e = new_cache("e4m3", 2, 8, 2, 64)
    with pytest.raises(ValueError, match="k_scale"):
        sv.sv_kv_append(x, x, e["k_cache"], e["v_cache"], t, qs, kl)
    with pytest.raises(ValueError):
        sv.sv_kv_append(x, x, e["k_cache"], e["v_cache"], t, qs, kl, k_scale=e["k_scale"][:, :1], v_scale=e["v_scale"])
    with pytest.raises(RuntimeError, match="invalid argument"):  # page size
        odd = torch.zeros((2, 6, 2, 64), device="cuda", dtype=torch.bfloat16)
        sv.sv_kv_append(x, x, odd, odd, t, qs, kl)
    with pytest.raises(RuntimeError, match="invalid argument"):  # rows that overlap
        flat = torch.zeros((2, 1, 2, 64), device="cuda", dtype=torch.bfloat16).expand(2, 8, 2, 64)
        sv.sv_kv_append(x, x, flat, flat, t, qs, kl)
    with pytest.raises(TypeError):
        sv.sv_kv_gather(c["k_cache"], c["v_cache"], t, qs, 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        sv.sv_kv_gather(c["k_cache"], c["v_cache"], t, I32([0, 1, 2]), 4)
    assert sv.sv_kv_gather(c["k_cache"], c["v_cache"], t, qs, 0)["k"].shape == (0, 2, 64)
