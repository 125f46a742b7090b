"""What binary32 drops of sv_rope's reduced angles is put back.

The half turns t / pi that are left of an angle, up to 1, are rounded to binary32
for cos and sin, by up to 2^-25: 9.4e-8 radians, more than a unit of the last
place of most results.  That angle d is known here, so its share of the errors
can be told from every other rounding by regression: were it not put back, cos t
would be off by d sin t, sin t by -d cos t, and the slope of the errors over
these would be 1.  Put back to first order, d^2 / 2 < 2^-47 remains and the slope
is 0, but for the other roundings: they are below 2^-22 each and know nothing of
d, whose root mean square is above 2^-26, so that over N = 10^5 results the
slope's standard deviation is below 2^-22 / (2^-26 sqrt(N)) = 0.05."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("most", [5000, 1 << 22])
def test_rope_puts_dropped_angles_back(layout, most):
    g = np.random.default_rng(most)
    T, D = 800, 256
    f = g.uniform(0.2, 1, D // 2)
    pos = g.integers(1, most + 1, T)
    one, zero = np.ones((T, 1, D // 2)), np.zeros((T, 1, D // 2))
    x = np.concatenate([one, zero], -1) if layout == "half" else np.stack([one, zero], -1).reshape(T, 1, D)
    cuda = lambda a, t: torch.from_numpy(a).to("cuda", t)
    y = sv.sv_rope(cuda(x, torch.float32), cuda(pos, torch.int64), cuda(f, torch.float64), layout=layout)
    y = y.double().cpu().numpy()[:, 0]
    c, s = (y[:, : D // 2], y[:, D // 2:]) if layout == "half" else (y[:, 0::2], y[:, 1::2])
    pi = np.longdouble("3.14159265358979323846264338327950288")
    half = pos.astype(np.longdouble)[:, None] * f.astype(np.longdouble) / pi
    half -= 2 * np.rint(half / 2)
    d = ((half - half.astype(np.float32)) * pi).astype(np.float64)
    t = (half * pi).astype(np.float64)
    assert np.sqrt((d ** 2).mean()) > 2.0 ** -26
    err, share = np.concatenate([c - np.cos(t), s - np.sin(t)]), np.concatenate([d * np.sin(t), -d * np.cos(t)])
    slope = (err * share).sum() / (share ** 2).sum()
    assert np.abs(err).max() < 2.0 ** -22
    assert abs(slope) < 0.25, slope
