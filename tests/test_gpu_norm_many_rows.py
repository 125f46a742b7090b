"""sv_qk_norm_rope and its gradients over so many rows that a workgroup takes four
at a time (from 4096 on): against the oracle, and bit by bit against calls of
fewer rows, which take one.  Tolerances as derived in test_gpu_norm.py; the
longest chain of a weight's gradient is there ceil(T / 1024) ceil(heads / 8)
additions, here ceil(T / 4096) ceil(4 heads / 8) <= ceil(T / 1024) ceil(2 heads /
8) for more than 4096 rows (and equal to ceil(heads / 2) <= 4 ceil(heads / 4) for
4096)."""
import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_norm import DT, N, check_backward, check_forward

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

FEW = 4095  # rows that are still taken one at a time

SHAPES = [  # rows, q heads, k heads, D, rotary
    (4096, 2, 1, 64, 64),
    (4097, 1, 1, 128, 128),
    (4099, 5, 2, 80, 48),
    (4098, 3, 3, 256, 256),
    (8191, 3, 2, 128, 64),
    (8195, 9, 1, 16, 16),
    (4101, 1, 1, 7, 6),
    (5003, 2, 1, 66, 22),
]


def inputs(shape, dtype, unaligned, seed=0):
    T, Hq, Hk, D, rotary = shape
    g = torch.Generator(device="cuda").manual_seed(seed + T * 1000 + D)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")

    def rows(h):
        x = (rn(T, h, D) * torch.exp(rn(T, h, 1))).to(DT[dtype])
        if not unaligned:
            return x
        wide = torch.zeros(T * h * D + 1, dtype=x.dtype, device="cuda")  # an element off
        wide[1:] = x.flatten()
        return wide[1:].view(T, h, D)

    s = dict(q=rows(Hq), k=rows(Hk), dq_out=rows(Hq), dk_out=rows(Hk))
    s["pos"] = 1000 + torch.arange(T, device="cuda") + torch.randint(0, 9, (T,), generator=g, device="cuda")
    s["f"] = sv.sv_rope_frequencies(rotary, device="cuda")[0]
    s["w"] = {n: (1 + 0.3 * rn(D)).to(DT[dtype]) for n in ("q_weight", "k_weight")}
    return s


@pytest.mark.parametrize("unaligned", [False, True])
@pytest.mark.parametrize("dtype,layout", [("bf16", "half"), ("bf16", "interleaved"), ("f32", "half"), ("f32", "interleaved")])
@pytest.mark.parametrize("shape", SHAPES)
def test_many_rows(dtype, layout, unaligned, shape):
    s = inputs(shape, dtype, unaligned)
    kw = dict(layout=layout, mscale=1.25, **s["w"])
    rows = [s[n] for n in ("q", "k", "dq_out", "dk_out", "pos")]
    o = sv.sv_qk_norm_rope(*rows[:2], rows[4], s["f"], **kw)
    d = sv.sv_qk_norm_rope_backward(*rows, s["f"], **kw)
    pos, f, heads = s["pos"].cpu().numpy(), N(s["f"]), shape[1] + shape[2]
    for n in "qk":
        w = s["w"][n + "_weight"]
        check_forward(s[n], o[n], w, 1e-6, pos, f, layout, 1.25)
        check_backward(s[n], s[f"d{n}_out"], d["d" + n], d[f"d{n}_weight"], w, 1e-6, pos, f, layout, 1.25, 2 * heads)
    # a row's bits do not depend on how many are taken at a time
    for part in (slice(0, FEW), slice(shape[0] - FEW, shape[0])):
        a = [x[part] for x in rows]
        few = sv.sv_qk_norm_rope(*a[:2], a[4], s["f"], **kw)
        less = sv.sv_qk_norm_rope_backward(*a, s["f"], want_weights=False, **kw)
        assert all(torch.equal(o[n][part], few[n]) for n in "qk")
        assert all(torch.equal(d[n][part], less[n]) for n in ("dq", "dk"))
    again = sv.sv_qk_norm_rope_backward(*rows, s["f"], **kw)
    assert all(torch.equal(d[n], again[n]) for n in d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_many_rows_in_place(dtype, layout):
    """Outputs over inputs, gradients over either of theirs; queries alone; gradients of 8195 rows that lie in a fused
    projection."""
    s = inputs((8195, 3, 2, 64, 32), dtype, False)
    kw = dict(layout=layout, **s["w"])
    names = ("q", "k", "dq_out", "dk_out")
    want = sv.sv_qk_norm_rope(s["q"], s["k"], s["pos"], s["f"], **kw)
    grad = sv.sv_qk_norm_rope_backward(*[s[n] for n in names], s["pos"], s["f"], **kw)
    q, k = s["q"].clone(), s["k"].clone()
    sv.sv_qk_norm_rope(q, k, s["pos"], s["f"], out=dict(q=q, k=k), **kw)
    assert torch.equal(q, want["q"]) and torch.equal(k, want["k"])
    alone = sv.sv_qk_norm_rope(s["q"], None, s["pos"], s["f"], layout=layout, q_weight=s["w"]["q_weight"])
    assert torch.equal(alone["q"], want["q"])
    for over in (names[:2], names[2:]):
        a = {n: s[n].clone() for n in names}
        d = sv.sv_qk_norm_rope_backward(*a.values(), s["pos"], s["f"], out=dict(dq=a[over[0]], dk=a[over[1]]), **kw)
        assert all(torch.equal(d[n], grad[n]) for n in grad)
    fused = [torch.cat([s[a], s[b], s[b]], 1) for a, b in (names[:2], names[2:])]
    parts = [x.split([3, 2, 2], 1)[:2] for x in fused]
    d = sv.sv_qk_norm_rope_backward(*parts[0], *parts[1], s["pos"], s["f"], **kw)
    assert all(torch.equal(d[n], grad[n]) for n in grad)
