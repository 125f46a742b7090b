"""sv_qk_norm_rope, its gradients, and sv_kv_append_normed on the GPU against
the oracle.

Tolerances, u = 2^-24.  The sum of at most 256 squares takes 8 fused steps and 5
levels of a tree: 14 u of itself; the division by D, eps, the root (which halves
what came before) and the reciprocal: r is off by at most (14 + 2) / 2 + 2 = 10
u, a normed channel x (r w) by 12 u < 2^-20 of itself.  The turn adds 2^-21 of
the pair's sum (see test_gpu_rope), so a turned channel is off by at most 2^-19
of mscale (|a| + |c|), a channel that is not turned by 2^-20 of itself.

Gradients, with g = R^T dy off by e_g = 2^-21 mscale (|dy| + |dy'|), n = x r off
by 2^-20 of itself and a = g w off by e_a = e_g |w| + u |a|: the mean c = sum a n
/ D is off by e_c = sum(e_a |n|) / D + (2^-20 + 16 u) sum |a n| / D; dx =
r (a - n c) by r (e_a + |n| e_c + (2^-20 + 2 u) |n c| + u |a|) + 12 u |dx|.  A
weight's gradient sums g n: off by sum e_g |n| + (2^-20 + k u) sum |g n|, k the
longest chain of additions: rows of a workgroup times heads of a group, 8 in a
wave and between waves, 16 workgroups a thread and 6 levels, the product's
rounding."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import attn as oa
from oracle import serve as osv
from test_gpu_kv import I32, new_cache, tables, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
N = lambda t: t.detach().double().cpu().numpy()


def other(x, rotary, layout):
    """What each turned channel is paired with (0 for the others)."""
    y = np.zeros_like(x)
    h = rotary // 2
    if layout == "half":
        y[..., :h], y[..., h:rotary] = x[..., h:rotary], x[..., :h]
    else:
        y[..., 0:rotary:2], y[..., 1:rotary:2] = x[..., 1:rotary:2], x[..., 0:rotary:2]
    return y


def half_step(y, dtype):
    return np.abs(y) * (2.0 ** -8 * (1 + 2.0 ** -8) if dtype == torch.bfloat16 else U)


def turned(x, w, eps, pos, f, layout, mscale):
    """(normed and turned rows, how far off binary32 may be)."""
    xn, wn = N(x), np.ones(x.shape[-1]) if w is None else N(w)
    want = osv.norm_rope(xn, wn, eps, pos, f, layout, mscale)
    n = np.abs(osv.norm_rope(xn, wn, eps, pos, f[:0]))
    r = 2 * len(f)
    pair = n + other(n, r, layout)
    return want, np.where(np.arange(n.shape[-1]) < r, pair * mscale * 2.0 ** -19, n * 2.0 ** -20)


def check_forward(x, out, w, eps, pos, f, layout, mscale):
    want, tol = turned(x, w, eps, pos, f, layout, mscale)
    err = np.abs(N(out) - want)
    assert (err <= tol + half_step(want, x.dtype)).all(), (err - tol - half_step(want, x.dtype)).max()


def check_backward(x, dy, dx, dw, w, eps, pos, f, layout, mscale, heads):
    xn, dn, wn = N(x), N(dy), np.ones(x.shape[-1]) if w is None else N(w)
    T, H, D = xn.shape
    want, want_w = osv.norm_rope_backward(xn, wn, eps, dn, pos, f, layout, mscale)
    r2 = 2 * len(f)
    r = 1 / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps)
    n, g = np.abs(xn * r), np.abs(oa.rope(dn, pos, f, layout, mscale, backward=True))
    e_g = np.where(np.arange(D) < r2, 2.0 ** -21 * mscale * (np.abs(dn) + other(np.abs(dn), r2, layout)), 0)
    a = g * np.abs(wn)
    e_a = e_g * np.abs(wn) + U * a
    c = np.abs((osv.oa.rope(dn, pos, f, layout, mscale, backward=True) * wn * xn * r).mean(-1, keepdims=True))
    e_c = (e_a * n).mean(-1, keepdims=True) + (2.0 ** -20 + 16 * U) * (a * n).mean(-1, keepdims=True)
    tol = r * (e_a + n * e_c + (2.0 ** -20 + 2 * U) * n * c + U * a) + 12 * U * np.abs(want)
    err = np.abs(N(dx) - want)
    tol = tol + half_step(want, x.dtype) + half_step(tol, x.dtype)
    assert (err <= tol).all(), (err - tol).max()
    if dw is not None:
        k = -(-T // 1024) * -(-heads // 8) + 8 + 16 + 6 + 2
        tol = (e_g * n).sum((0, 1)) + (2.0 ** -20 + k * U) * (g * n).sum((0, 1))
        assert dw.dtype == torch.float32 and (np.abs(N(dw) - want_w) <= tol).all(), (np.abs(N(dw) - want_w) - tol).max()


SHAPES = [  # rows, q heads, k heads, D, rotary, far
    (1, 1, 1, 128, 128, 0), (7, 32, 8, 128, 128, 900001), (33, 5, 5, 128, 64, 1 << 20), (3, 2, 1, 64, 16, 1 << 39),
    (5, 3, 1, 80, 80, 12345), (5, 4, 2, 96, 48, 12345), (2, 1, 1, 256, 256, 77), (4, 40, 8, 256, 32, 3),
    (9, 2, 1, 6, 4, 5), (9, 3, 1, 7, 6, 100000), (2, 3, 3, 1, 0, 9), (600, 2, 1, 66, 22, 4000), (3, 1000, 1, 16, 16, 1),
    (2100, 4, 2, 64, 64, 0),
]


def inputs(shape, dtype, weights, seed=0):
    T, Hq, Hk, D, rotary, far = shape
    g = torch.Generator(device="cuda").manual_seed(seed + T * 1000 + D)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    rows = lambda h: (rn(T, h, D) * torch.exp(2 * rn(T, h, 1))).to(DT[dtype])
    s = dict(q=rows(Hq), k=rows(Hk), dq_out=rows(Hq), dk_out=rows(Hk))
    s["pos"] = far + torch.randint(-3, 4, (T,), generator=g, device="cuda")
    s["f"] = sv.sv_rope_frequencies(rotary, device="cuda")[0]
    s["w"] = dict(q_weight=None, k_weight=None) if weights is None else {
        n: (1 + rn(D)).to(DT[weights]) for n in ("q_weight", "k_weight")}
    return s


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,weights,eps,mscale", [("f32", "f32", 1e-6, 1.0), ("bf16", "bf16", 1e-5, 1.25),
                                                      ("bf16", "f32", 0.5, 1.0), ("f32", None, 1e-6, 1.0)])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_rope_and_its_gradients(layout, dtype, weights, eps, mscale, shape):
    s = inputs(shape, dtype, weights)
    kw = dict(eps=eps, layout=layout, mscale=mscale, **s["w"])
    o = sv.sv_qk_norm_rope(s["q"], s["k"], s["pos"], s["f"], **kw)
    d = sv.sv_qk_norm_rope_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], s["pos"], s["f"], **kw)
    pos, f = s["pos"].cpu().numpy(), N(s["f"])
    for n in "qk":
        w = s["w"][n + "_weight"]
        check_forward(s[n], o[n], w, eps, pos, f, layout, mscale)
        check_backward(s[n], s[f"d{n}_out"], d["d" + n], d[f"d{n}_weight"], w, eps, pos, f, layout, mscale,
                       s["q"].shape[1] + s["k"].shape[1])
    again = sv.sv_qk_norm_rope_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], s["pos"], s["f"], **kw)
    assert all(torch.equal(d[n], again[n]) for n in d)


def test_gradients_against_differences():
    """The backward pass against central differences of the forward one, in a direction of length about 1 for each input.
    With steps of h = 2^-4 the outputs' errors, 2^-19 of their pair's size each, come to at most 2^-19 sum |y dy| / h: the
    1920 products have a mean of some 2/3, 0.04 in all.  The differences' own error, h^2 / 6 of the third derivative,
    which is below 15 |dy w| 8 / |x|^3 for a row of length |x| = 8 and |dy w| up to 16: 0.003."""
    s = inputs((6, 3, 2, 64, 32, 50), "f32", "f32")
    for n in ("q", "k"):
        s[n] = torch.randn_like(s[n])
    args = (s["pos"], s["f"])
    dy = {n: torch.randn_like(s[n]) for n in "qk"}
    d = sv.sv_qk_norm_rope_backward(s["q"], s["k"], dy["q"], dy["k"], *args, **s["w"])
    loss = lambda q, k, w: sum((v.double() * dy[n].double()).sum().item()
                               for n, v in sv.sv_qk_norm_rope(q, k, *args, **w).items())
    h = 2.0 ** -4
    for n in ("q", "k", "q_weight", "k_weight"):
        v = {**s, **s["w"]}
        e = torch.randn_like(v[n]) / v[n].numel() ** 0.5
        at = lambda x: loss(*[x if m == n else v[m] for m in ("q", "k")],
                            {m: x if m == n else v[m] for m in ("q_weight", "k_weight")})
        num = (at(v[n] + h * e) - at(v[n] - h * e)) / (2 * h)
        assert abs(num - (d["d" + n].double() * e.double()).sum().item()) < 0.05, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_alignment_and_in_place(dtype, layout):
    """Heads of a fused projection, head-major rows, rows an element off, one row for all; outputs over their inputs."""
    f, _ = sv.sv_rope_frequencies(64, device="cuda")
    pos = torch.arange(11, device="cuda")
    t = DT[dtype]
    base = torch.randn((11, 6, 128), device="cuda").to(t)
    major = torch.randn((6, 11, 128), device="cuda").to(t).transpose(0, 1)
    off = torch.randn(11 * 6 * 131 + 1, device="cuda").to(t)[1:].as_strided((11, 6, 128), (6 * 131, 131, 1), 1)
    w = dict(q_weight=torch.randn(128, device="cuda"), k_weight=torch.randn(128, device="cuda"))
    for x in (base[:, 1:5], major, off, base[:1].expand(11, 6, 128)):
        k, dy = x[:, :2], torch.randn((11, 6, 128), device="cuda").to(t)[:, :x.shape[1]]
        c = x.contiguous()
        want = sv.sv_qk_norm_rope(c, c[:, :2].contiguous(), pos, f, layout=layout, **w)
        got = sv.sv_qk_norm_rope(x, k, pos, f, layout=layout, **w)
        back = lambda a, b: sv.sv_qk_norm_rope_backward(a, b, dy, dy[:, :2], pos, f, layout=layout, **w)
        want_d, got_d = back(c, c[:, :2].contiguous()), back(x, k)
        check_forward(x, got["q"], w["q_weight"], 1e-6, pos.cpu().numpy(), N(f), layout, 1.0)
        for a, b in ((want, got), (want_d, got_d)):
            for n in a:  # (an output's address or stride may choose another order of the same operations: none today)
                assert torch.equal(a[n], b[n]), n
        if x.stride(0) == 0:
            continue
        y, kk = c.clone(), c[:, :2].clone()
        o = sv.sv_qk_norm_rope(y, kk, pos, f, layout=layout, out=dict(q=y, k=kk), **w)
        assert o["q"] is y and torch.equal(y, want["q"]) and torch.equal(kk, want["k"])
        for over in ("grad", "input"):
            a, b, ga, gb = c.clone(), c[:, :2].clone(), dy.clone(), dy[:, :2].clone()
            out = dict(dq=ga, dk=gb) if over == "grad" else dict(dq=a, dk=b)
            d = sv.sv_qk_norm_rope_backward(a, b, ga, gb, pos, f, layout=layout, out=out, **w)
            assert all(torch.equal(d[n], want_d[n]) for n in want_d)


def test_parts_of_a_call():
    """No keys; no rotation; no weights' gradients; one weight alone; no rows; a scratch of the caller's."""
    s = inputs((40, 4, 2, 64, 64, 9), "bf16", "bf16")
    both = sv.sv_qk_norm_rope(s["q"], s["k"], s["pos"], s["f"], **s["w"])
    alone = sv.sv_qk_norm_rope(s["q"], None, s["pos"], s["f"], q_weight=s["w"]["q_weight"])
    assert set(alone) == {"q"} and torch.equal(alone["q"], both["q"])
    plain = sv.sv_qk_norm_rope(s["q"], s["k"], **s["w"])
    still = sv.sv_qk_norm_rope(s["q"], s["k"], torch.zeros_like(s["pos"]), s["f"], **s["w"])
    assert all(torch.equal(plain[n], still[n]) for n in "qk")
    grads = (s["q"], s["k"], s["dq_out"], s["dk_out"], s["pos"], s["f"])
    d = sv.sv_qk_norm_rope_backward(*grads, **s["w"])
    less = sv.sv_qk_norm_rope_backward(*grads, want_weights=False, **s["w"])
    assert set(less) == {"dq", "dk"} and all(torch.equal(less[n], d[n]) for n in less)
    dw = torch.full((64,), 9.0, device="cuda")
    one = sv.sv_qk_norm_rope_backward(*grads, want_weights=False, out=dict(dk_weight=dw), **s["w"])
    assert set(one) == {"dq", "dk", "dk_weight"} and torch.equal(dw, d["dk_weight"])
    size = sv.sv_qk_norm_rope_backward_workspace_size(40, 64)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    own = sv.sv_qk_norm_rope_backward(*grads, workspace=ws[:size], **s["w"])
    assert all(torch.equal(own[n], d[n]) for n in d) and (ws[size:] == 255).all()
    with pytest.raises(RuntimeError, match="workspace"):
        sv.sv_qk_norm_rope_backward(*grads, workspace=ws[:size - 1], **s["w"])
    none = [x[:0] for x in grads[:5]]
    d = sv.sv_qk_norm_rope_backward(*none, s["f"], **s["w"])
    assert d["dq"].shape == (0, 4, 64) and (d["dq_weight"] == 0).all() and (d["dk_weight"] == 0).all()


def test_rows_of_zeros_and_of_extremes():
    """A row of zeros stays one and has the gradient r w g; tiny rows are ruled by eps; NaN stays in its row."""
    x = torch.randn((4, 2, 128), device="cuda")
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e15
    pos, (f, _) = torch.arange(4, device="cuda"), sv.sv_rope_frequencies(128, device="cuda")
    o = sv.sv_qk_norm_rope(x, None, pos, f)["q"]
    assert (o[0] == 0).all()
    check_forward(x, o, None, 1e-6, pos.cpu().numpy(), N(f), "half", 1.0)
    dy = torch.randn_like(x)
    d = sv.sv_qk_norm_rope_backward(x, None, dy, None, pos, f)
    check_backward(x, dy, d["dq"], d["dq_weight"], None, 1e-6, pos.cpu().numpy(), N(f), "half", 1.0, 2)
    x[3, 1, 5] = float("nan")
    p = sv.sv_qk_norm_rope(x, None, pos, f)["q"]
    keep = torch.ones((4, 2), dtype=torch.bool, device="cuda")
    keep[3, 1] = False
    assert torch.equal(p[keep], o[keep]) and torch.isnan(p[3, 1]).all()


CASES = [  # new tokens and lengths with them, page, kv heads, q heads, D, rotary
    ([5, 5, 5], [5, 37, 100], 16, 2, 8, 128, 128),
    ([1], [1], 16, 1, 1, 64, 64),
    ([0, 3, 0, 17, 0], [9, 3, 0, 40, 5], 8, 5, 5, 80, 40),
    ([130, 1, 70], [130, 4, 200], 32, 4, 0, 96, 96),
    ([6, 4], [3, 4], 1, 3, 6, 16, 16),  # the first request's first rows lie before its place 0
    ([33, 2], [50, 2], 128, 1, 7, 256, 64),
]


@pytest.mark.parametrize("cache,order", [("bf16", "tokens"), ("e4m3", "heads")])
@pytest.mark.parametrize("dtype,weights,layout", [("bf16", "bf16", "half"), ("f32", "f32", "interleaved"),
                                                  ("bf16", None, "interleaved")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_normed(cache, order, dtype, weights, layout, case):
    """Queries and stored keys against the oracle; values, slots and rows of no request as sv_kv_append leaves them."""
    new, total, page, heads, q_heads, D, rotary = CASES[case]
    g = torch.Generator(device="cuda").manual_seed(case)
    pages, table, start = tables(new, total, page, seed=case)
    c, plain = new_cache(cache, pages, page, heads, D, order), new_cache(cache, pages, page, heads, D, order)
    T = int(start[-1]) + 3
    qkv = (torch.randn((T, q_heads + 2 * heads, D), generator=g, device="cuda")
           * torch.exp(2 * torch.randn((T, 1, 1), generator=g, device="cuda"))).to(DT[dtype])
    q, k, v = qkv.split([q_heads, heads, heads], 1)
    f, _ = sv.sv_rope_frequencies(rotary, device="cuda")
    w = {n: None if weights is None else (1 + torch.randn(D, generator=g, device="cuda")).to(DT[weights])
         for n in ("q_weight", "k_weight")}
    marked = lambda: {"q": torch.full((T, q_heads, D), 7.0, device="cuda", dtype=DT[dtype])}
    kw = dict(q=q if q_heads else None, freq=f, layout=layout, mscale=1.125)
    at = (I32(table), I32(start), I32(total))
    o = sv.sv_kv_append_normed(k, v, c["k_cache"], c["v_cache"], *at, k_scale=c["k_scale"], v_scale=c["v_scale"],
                               eps=1e-5, out=marked(), **w, **kw)
    sv.sv_kv_append(k, v, plain["k_cache"], plain["v_cache"], *at, k_scale=plain["k_scale"], v_scale=plain["v_scale"],
                    out=marked(), **kw)
    place = np.array([oa.place_of(start, total, b, i) for b in range(len(new)) for i in range(new[b])], int)
    rows = int(start[-1])
    if q_heads:
        check_forward(q[:rows], o["q"][:rows], w["q_weight"], 1e-5, place, N(f), layout, 1.125)
        assert (o["q"][rows:] == 7.0).all()
    assert torch.equal(c["v_cache"].contiguous().view(torch.uint8), plain["v_cache"].contiguous().view(torch.uint8))
    kv, untouched = values(c, "k"), values(new_cache(cache, pages, page, heads, D, order), "k")
    want, tol = turned(k[:rows], w["k_weight"], 1e-5, place, N(f), layout, 1.125)
    written = np.zeros((pages, page), bool)
    r = 0
    for b in range(len(new)):
        for i in range(new[b]):
            p = oa.place_of(start, total, b, i)
            if p >= 0:
                to = (table[b, p // page], p % page)
                written[to] = True
                if cache == "bf16":
                    half = np.abs(want[r]) * 2.0 ** -8 * (1 + 2.0 ** -8)
                else:
                    e = c["k_scale"][to[0], :, to[1]].cpu().numpy().astype(int) - 127
                    top = np.abs(want[r]).max(-1)
                    # the least exponent for the largest magnitude, or its neighbour where that is within 2^-17 of a border
                    lo, hi = (oa.quantise(want[r] * (1 + d))[1] for d in (-2.0 ** -17, 2.0 ** -17))
                    assert ((lo <= e) & (e <= hi)).all() and np.isfinite(top).all()
                    half = np.maximum(np.abs(want[r]) * 2.0 ** -4, 2.0 ** (e[:, None] - 10)) * (1 + 2.0 ** -4)
                assert (np.abs(kv[to] - want[r]) <= tol[r] * (1 + 2.0 ** -4) + half).all()
            r += 1
    assert np.array_equal(kv[~written], untouched[~written])


def test_norm_calls_captured_and_on_two_streams():
    ss = [inputs((300, 8, 2, 128, 128, 5), "bf16", "bf16", seed) for seed in (1, 2)]
    run = lambda s: {**sv.sv_qk_norm_rope(s["q"], s["k"], s["pos"], s["f"], **s["w"]),
                     **sv.sv_qk_norm_rope_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], s["pos"], s["f"], **s["w"])}
    want = [{k: v.clone() for k, v in run(s).items()} for s in ss]
    torch.cuda.synchronize()
    graphs = []
    for s in ss:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(s)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in ss]
    for rep in range(4):
        for s, w in zip(ss, want):
            s["q"].mul_(1.5)
            w.update({k: v.clone() for k, v in run(s).items()})
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = []
        for s, st in zip(ss, streams):
            with torch.cuda.stream(st):
                eager.append(run(s))
        torch.cuda.synchronize()
        for w, (_, out), e in zip(want, graphs, eager):
            for k in w:
                assert torch.equal(out[k], w[k]) and torch.equal(e[k], w[k]), (rep, k)
