"""Pins of the rotary, cache and attention oracle: closed forms, enumeration
and library routines; no GPU."""
import math

import numpy as np
import pytest
import torch

from oracle import attn as oa


def cache_of(k, v, table):
    return dict(k=np.asarray(k, float), v=np.asarray(v, float), table=np.asarray(table))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_a_rotation_by_relative_positions(layout):
    g = np.random.default_rng(1)
    f, m = oa.frequencies(8)
    assert m == 1.0 and f[0] == 1.0 and f[1] == pytest.approx(0.1) and len(f) == 4
    a, c = g.standard_normal((1, 2, 12)), g.standard_normal((1, 2, 12))
    dots = []
    for p, q in ((3, 10), (1003, 1010), (0, 7)):
        x, y = oa.rope(a, [p], f, layout), oa.rope(c, [q], f, layout)
        assert np.array_equal(x[..., 8:], a[..., 8:])
        assert np.allclose((x ** 2).sum(-1), (a ** 2).sum(-1))
        dots.append((x[..., :8] * y[..., :8]).sum(-1))
    assert np.allclose(dots[0], dots[1]) and np.allclose(dots[0], dots[2])


def test_rope_of_a_quarter_turn_and_its_backward():
    f = np.array([math.pi / 2])
    x = np.array([[[1.0, 2.0, 5.0]]])
    for layout in ("half", "interleaved"):  # one pair: the layouts agree
        y = oa.rope(x, [1], f, layout, mscale=2.0)
        assert np.allclose(y, [[[-4.0, 2.0, 5.0]]])
    g = np.random.default_rng(2)
    f, _ = oa.frequencies(6)
    for layout in ("half", "interleaved"):
        x, d = g.standard_normal((3, 2, 8)), g.standard_normal((3, 2, 8))
        pos = [0, 5, 1 << 30]
        # the transpose: <R x, d> = <x, R' d>
        lhs = (oa.rope(x, pos, f, layout, 1.5)[..., :6] * d[..., :6]).sum()
        rhs = (x[..., :6] * oa.rope(d, pos, f, layout, 1.5, backward=True)[..., :6]).sum()
        assert lhs == pytest.approx(rhs, rel=1e-12)


def test_frequency_scalings():
    plain, _ = oa.frequencies(64, 10000.0)
    assert np.allclose(oa.frequencies(64, 10000.0, "linear", 4.0)[0] * 4, plain)
    # the changed base leaves the fastest pair alone and slows the slowest by the factor
    b, _ = oa.frequencies(64, 10000.0, "base", 8.0)
    assert b[0] == 1.0 and b[-1] * 8 == pytest.approx(plain[-1])
    for kind, kw in (("ramp", dict(low=1.0, high=32.0)), ("bands", dict(low=1.0, high=4.0))):
        f, m = oa.frequencies(64, 10000.0, kind, 8.0, original_len=4096.0, **kw)
        turns = 4096.0 * plain / (2 * math.pi)
        assert np.all(f <= plain * (1 + 1e-15)) and np.all(f >= plain / 8 * (1 - 1e-15)) and np.all(np.diff(f) < 0)
        fast, slow = turns > 1.2 * kw["high"] * (1.35 if kind == "ramp" else 1), turns < kw["low"] / 1.4
        assert fast.any() and slow.any()
        assert np.allclose(f[fast], plain[fast]) and np.allclose(f[slow] * 8, plain[slow])
        assert m == (pytest.approx(0.1 * math.log(8.0) + 1) if kind == "ramp" else 1.0)


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(oa.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


def test_quantise_rounds_as_torch_and_scales_tightly():
    g = np.random.default_rng(3)
    x = (g.standard_normal((500, 16)) * np.exp(3 * g.standard_normal((500, 1)))).astype(np.float32)
    x[0], x[1, :], x[2, 3], x[3, 5] = 0, 448.0, np.inf, np.nan
    x[4] = np.linspace(-448, 448, 16)
    x[5, 0] = 449.0
    x[6] = np.arange(16) / 16 + 1  # ties between codes
    x[6, 15] = 448
    codes, e = oa.quantise(x)
    assert e[0] == -9 and e[1] == 0 and e[5] == 1
    top = np.where(np.isfinite(x), np.abs(x), 0).max(-1).astype(np.float64)
    live = top > 0
    assert np.all(top <= 448 * 2.0 ** e) and np.all(top[live] > 224 * 2.0 ** e[live])
    want = torch.from_numpy(np.where(np.isfinite(x), x, np.nan) / np.exp2(e)[:, None].astype(np.float32))
    want = want.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ok = (codes == want) | ((codes & 127 == 127) & (want & 127 == 127))
    assert ok.all()
    tiny, e = oa.quantise(np.array([[2.0 ** -140, 0.0]]))
    assert e[0] == -117 and tiny[0, 0] == 0


def test_gather_places_and_holes():
    k = np.arange(3 * 2).reshape(3, 2, 1, 1) + 10.0
    c = cache_of(k, -k, [[2, 0], [1, 7]])
    o = oa.gather(c, [1, 4, 6], 7, kv_begin=[0, 1])
    assert o["k"][:, 0, 0].tolist()[1:6] == [14.0, 15.0, 10.0, 13.0, 0.0]
    assert np.isnan(o["k"][0]).all() and np.isnan(o["v"][6]).all() and o["v"][1, 0, 0] == -14.0


def test_attention_closed_forms():
    g = np.random.default_rng(4)
    k, v = g.standard_normal((4, 4, 2, 8)), g.standard_normal((4, 4, 2, 8))
    c = cache_of(k, v, [[3, 1, 0]])
    rows = np.concatenate([k[3], k[1], k[0]]), np.concatenate([v[3], v[1], v[0]])
    # q = 0: the mean of the values seen, lse the log of their number
    o = oa.attention(np.zeros((3, 4, 8)), c, [0, 3], [10], 0.5)
    for i in range(3):
        for h in range(4):
            assert np.allclose(o["out"][i, h], rows[1][: 8 + i, h // 2].mean(0))
            assert o["lse"][i, h] == pytest.approx(math.log(8 + i))
    o = oa.attention(np.zeros((3, 4, 8)), c, [0, 3], [10], 0.5, window=2)
    assert np.allclose(o["out"][1, 0], rows[1][7:9, 0].mean(0))
    # torch's routine, in double
    q = g.standard_normal((5, 4, 8))
    o = oa.attention(q, c, [0, 5], [12], 0.3)
    mask = torch.arange(12)[None] <= (7 + torch.arange(5))[:, None]
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).transpose(0, 1)
    ref = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(rows[0].repeat(2, 1)), t(rows[1].repeat(2, 1)), attn_mask=mask, scale=0.3)
    assert np.allclose(o["out"], ref.transpose(0, 1).numpy())


def test_attention_rows_that_see_nothing():
    c = cache_of(np.ones((2, 2, 1, 8)), np.ones((2, 2, 1, 8)), [[0, 5], [9, 9]])
    o = oa.attention(np.ones((6, 1, 8)), c, [0, 4, 5], [3, 2], 1.0)
    assert np.isneginf(o["lse"][0, 0]) and not o["out"][0].any()  # place -1
    assert o["lse"][1, 0] == pytest.approx(8.0) and o["lse"][3, 0] == pytest.approx(8 + math.log(2))
    assert np.isneginf(o["lse"][4, 0])  # only absent pages
    assert np.isnan(o["out"][5]).all()
