"""sv_rope on the GPU against the oracle.

Tolerance.  An angle's whole turns are dropped in binary64; what is left, at
most half a turn, is rounded once to binary32 (2^-25 half turns = 2^-23.3
radians), cos and sin are off by at most 2 units of the last place (2^-23) and
the two products and their sum by three roundings (2^-24 each) of at most
(|a| + |c|) mscale: under 2^-21 of that.  A bf16 result is rounded once more, by
at most 2^-8 of its value."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import attn as oa

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def bound(x, y, rotary, layout, mscale, dtype):
    x = np.abs(x)
    other = x.copy()
    h = rotary // 2
    if layout == "half":
        other[..., :h], other[..., h:rotary] = x[..., h:rotary], x[..., :h]
    else:
        other[..., 0:rotary:2], other[..., 1:rotary:2] = x[..., 1:rotary:2], x[..., 0:rotary:2]
    tol = (x + other) * mscale * 2.0 ** -21
    tol[..., rotary:] = 0
    return tol + (np.abs(y) * 2.0 ** -8 if dtype == "bf16" else 0) * (1 + 2.0 ** -8) * (np.arange(x.shape[-1]) < rotary)


def check(x, out, positions, f, layout, mscale, backward, dtype):
    xn = x.double().cpu().numpy()
    want = oa.rope(xn, positions.cpu().numpy(), f.cpu().numpy(), layout, mscale, backward)
    got = out.double().cpu().numpy()
    err = np.abs(got - want)
    tol = bound(xn, want, 2 * len(f), layout, mscale, dtype)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,D,rotary,far", [
    (1, 1, 128, 128, 0), (7, 32, 128, 128, 900001), (33, 5, 128, 64, 1 << 20), (3, 2, 64, 16, 1 << 39),
    (5, 3, 80, 80, 12345), (5, 3, 96, 48, 12345), (2, 1, 256, 256, 77), (4, 40, 256, 32, 3), (9, 2, 6, 4, 5),
    (9, 3, 7, 6, 100000), (2, 3, 1, 0, 9), (600, 2, 66, 22, 4000), (3, 1024, 16, 16, 1),
])
def test_rope_forward_and_backward(layout, dtype, T, H, D, rotary, far):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + D)
    x = torch.randn((T, H, D), generator=g, device="cuda").to(DT[dtype])
    pos = far + torch.randint(-3, 4, (T,), generator=g, device="cuda")
    f, _ = sv.sv_rope_frequencies(rotary, device="cuda")
    for mscale, backward in ((1.0, False), (1.25, True)):
        out = sv.sv_rope(x, pos, f, layout=layout, mscale=mscale, backward=backward)
        check(x, out, pos, f, layout, mscale, backward, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strided_unaligned_and_in_place(dtype, layout):
    f, _ = sv.sv_rope_frequencies(64, device="cuda")
    pos = torch.arange(11, device="cuda")
    # heads of a fused projection (aligned), head-major rows, rows one element off, odd row stride
    base = torch.randn((11, 6, 128), device="cuda").to(DT[dtype])
    major = torch.randn((6, 11, 128), device="cuda").to(DT[dtype]).transpose(0, 1)
    flat = torch.randn(11 * 6 * 131 + 1, device="cuda").to(DT[dtype])
    off = flat[1:].as_strided((11, 6, 128), (6 * 131, 131, 1), 1)
    for x in (base[:, 1:5], major, off, base[:1].expand(11, 6, 128)):
        want = sv.sv_rope(x.contiguous(), pos, f, layout=layout)
        check(x, want, pos, f, layout, 1.0, False, dtype)
        assert torch.equal(sv.sv_rope(x, pos, f, layout=layout), want)
    for x in (base[:, 1:5], major, off):
        want = sv.sv_rope(x, pos, f, layout=layout)
        y = x.clone(memory_format=torch.preserve_format) if x is not off else x
        rest = base.clone()
        got = sv.sv_rope(y, pos, f, layout=layout, out=y)
        assert got is y and torch.equal(y, want) and torch.equal(base, rest)


def test_rope_gradient_is_that_of_the_formula_and_of_differences():
    f, m = sv.sv_rope_frequencies(32, scaling="ramp", factor=4.0, original_len=64.0, device="cuda")
    x = torch.randn((6, 3, 48), device="cuda")
    w = torch.randn_like(x)
    pos = torch.tensor([0, 1, 17, 300, 5000, 70000], device="cuda")
    for layout in ("half", "interleaved"):
        grad = sv.sv_rope(w, pos, f, layout=layout, mscale=m, backward=True)
        # the map is linear: <w, R(x + h d) - R(x - h d)> / 2h is <w, R d>, up to the bounds of the three calls (doubled
        # for the roundings of x + h d and x - h d themselves, 2^-24 of their values)
        d = torch.randn_like(x)
        h = 0.5
        diff = (sv.sv_rope(x + h * d, pos, f, layout=layout, mscale=m).double()
                - sv.sv_rope(x - h * d, pos, f, layout=layout, mscale=m).double()) / (2 * h)
        lhs, rhs = (w.double() * diff).sum(), (grad.double() * d.double()).sum()
        n = lambda z: z.double().cpu().numpy()
        b = lambda z: bound(n(z), np.zeros_like(n(z)), 32, layout, m, "f32") + np.abs(n(z)) * 2.0 ** -24
        tol = 2 * (np.abs(n(w)) * (b(x + h * d) + b(x - h * d)) + np.abs(n(d)) * b(w)).sum()
        assert abs(lhs - rhs).item() <= tol
        # and torch's own gradient of the formula in 64 bits
        xd = x.double().requires_grad_()
        t = pos.double()[:, None] * f
        cos, sin = (t.cos() * m)[:, None], (t.sin() * m)[:, None]
        a, c = (xd[..., :16], xd[..., 16:32]) if layout == "half" else (xd[..., 0:32:2], xd[..., 1:32:2])
        wa, wc = (w[..., :16], w[..., 16:32]) if layout == "half" else (w[..., 0:32:2], w[..., 1:32:2])
        ((a * cos - c * sin) * wa + (a * sin + c * cos) * wc).sum().add((xd[..., 32:] * w[..., 32:]).sum()).backward()
        tol = bound(w.double().cpu().numpy(), xd.grad.cpu().numpy(), 32, layout, m, "f32")
        assert (np.abs((grad.double() - xd.grad).cpu().numpy()) <= tol).all()


def test_rope_empty_and_refusals():
    f, _ = sv.sv_rope_frequencies(64, device="cuda")
    pos = torch.arange(4, device="cuda")
    x = torch.randn((4, 2, 64), device="cuda")
    assert sv.sv_rope(x[:0], pos[:0], f).shape == (0, 2, 64)
    assert sv.sv_rope(x[:, :0], pos, f).shape == (4, 0, 64)
    with pytest.raises(TypeError):
        sv.sv_rope(x.half(), pos, f)
    with pytest.raises(TypeError):
        sv.sv_rope(x, pos.int(), f)
    with pytest.raises(TypeError):
        sv.sv_rope(x, pos, f.float())
    with pytest.raises(ValueError):
        sv.sv_rope(x, pos[:3], f)
    with pytest.raises(ValueError):
        sv.sv_rope(x.transpose(1, 2), pos, f)
    with pytest.raises(ValueError):
        sv.sv_rope(x, pos, f, layout="other")
    with pytest.raises(ValueError):
        sv.sv_rope(x, pos.cpu(), f)
    with pytest.raises(ValueError):
        sv.sv_rope(x, pos, f, out=x[:3])
    with pytest.raises(RuntimeError, match="invalid argument"):
        sv.sv_rope(x[..., :32], pos, f)  # more turned channels than a head has
    with pytest.raises(RuntimeError, match="unsupported"):
        sv.sv_rope(torch.randn((1, 1, 300), device="cuda"), pos[:1], f)
