"""Pins of oracle/serve.py: gradients against differences, norms against closed
forms, pages' invariants."""
import numpy as np
import pytest

from oracle import attn as oa
from oracle import serve as os_


def test_norm_closed_forms():
    """A row of equal magnitudes is its signs over sqrt(1 + eps / m^2); weights scale channels; a turn keeps pairs' size."""
    f, _ = oa.frequencies(8)
    x = np.where(np.random.default_rng(0).random((3, 2, 8)) < 0.5, -1.0, 1.0) * 5
    y = os_.norm_rope(x, np.ones(8), 1e-9, [0, 0, 0], f)
    assert np.allclose(y, np.sign(x), atol=1e-10)
    w = np.arange(1.0, 9)
    assert np.allclose(os_.norm_rope(x, w, 25.0, [0, 0, 0], f), np.sign(x) * w / np.sqrt(2))
    z = os_.norm_rope(x, w, 1e-9, [3, 70, 900], f)
    assert np.allclose(np.hypot(z[..., :4], z[..., 4:]), np.hypot(w[:4], w[4:]))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rotary", [0, 4, 10])
def test_norm_gradients_against_differences(layout, rotary):
    rng = np.random.default_rng(rotary)
    x, dy, w = rng.normal(size=(3, 2, 10)), rng.normal(size=(3, 2, 10)), rng.normal(size=10)
    f = oa.frequencies(rotary)[0]
    args = ([5, 0, 77], f, layout, 1.25)
    dx, dw = os_.norm_rope_backward(x, w, 0.01, dy, *args)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        d = (os_.norm_rope(x + e, w, 0.01, *args) - os_.norm_rope(x - e, w, 0.01, *args)) / (2 * h)
        assert abs((d * dy).sum() - dx[i]) < 1e-8
    for i in range(10):
        e = np.zeros(10)
        e[i] = h
        d = (os_.norm_rope(x, w + e, 0.01, *args) - os_.norm_rope(x, w - e, 0.01, *args)) / (2 * h)
        assert abs((d * dy).sum() - dw[i]) < 1e-8


def test_pages_are_neither_lost_nor_doubled():
    rng = np.random.default_rng(1)
    B, most, size, capacity = 7, 9, 4, 30
    table, held, free = [[-1] * most for _ in range(B)], [0] * B, rng.permutation(capacity).tolist()
    refused = 0
    for _ in range(200):
        before = [h for h in held]
        kv_len = rng.integers(-2, 45, B)
        granted = os_.pages(table, held, free, kv_len, size, capacity)
        refused += B - sum(granted)
        out = [p for b in range(B) for p in table[b][:held[b]]]
        assert sorted(out + free) == list(range(capacity))
        for b in range(B):
            need = -(-max(int(kv_len[b]), 0) // size)
            assert held[b] == (need if granted[b] else before[b]) and table[b][held[b]:] == [-1] * (most - held[b])
    assert refused > 20


def test_giving_back_undoes_taking():
    table, held, free = [[-1] * 5 for _ in range(3)], [0, 0, 0], list(range(11))
    os_.pages(table, held, free, [3, 4, 1], 2, 11)
    state = ([r[:] for r in table], held[:], free[:])
    assert os_.pages(table, held, free, [9, 4, 6], 2, 11) == [1, 1, 1] and held == [5, 2, 3]
    os_.pages(table, held, free, [3, 4, 1], 2, 11)
    assert (table, held, free) == state


def test_shared_pages_stay_and_refusals_go_in_order():
    table, held, free = [[7, 8, 9, -1], [7, 8, -1, -1], [7, 8, -1, -1]], [3, 2, 2], [1, 0]
    # the first gives one page back, the second lacks two, the third (two more, of which one is there) is refused
    assert os_.pages(table, held, free, [0, 8, 8], 2, 10, shared=[2, 2, 2]) == [1, 1, 0]
    assert table == [[7, 8, -1, -1], [7, 8, 9, 0], [7, 8, -1, -1]] and held == [2, 4, 2] and free == [1]
    assert os_.slots(table, held, [0, 8, 5], [0, 0, 2, 4], 2, 9) == ([0, 1, 17, -1], [6, 7, 3, 4])


def small_cache(seed, B=3, pages=9, size=4, heads=2, D=8):
    rng = np.random.default_rng(seed)
    c = dict(k=rng.normal(size=(pages, size, heads, D)), v=rng.normal(size=(pages, size, heads, D)),
             table=rng.permutation(pages)[:9].reshape(3, 3))
    return c, rng.normal(size=(6, 4, D))


def test_attention_without_sinks_and_groups_is_the_older_oracle():
    c, q = small_cache(0)
    for window in (0, 1, 3):
        a = oa.attention(q, c, [0, 1, 3, 6], [12, 2, 9], 0.4, window)
        b = os_.attention(q, c, [0, 1, 3, 6], [12, 2, 9], 0.4, window)
        assert all(np.allclose(a[n], b[n], atol=1e-14) for n in a)


def test_attention_sinks_join_what_is_before_the_window():
    """Weights of two disjoint sets of tokens add: the window's result and that of the first tokens, by their lse."""
    c, q = small_cache(1)
    start, length = [0, 1, 1, 1], [12, 0, 0]
    whole = os_.attention(q[:1], c, start, length, 0.4, 5, 3)
    near = os_.attention(q[:1], c, start, length, 0.4, 5)
    first = os_.attention(q[:1], c, start, [3, 0, 0], 0.4)
    a, b = np.exp(near["lse"] - whole["lse"]), np.exp(first["lse"] - whole["lse"])
    assert np.allclose(a + b, 1) and np.allclose(a[..., None] * near["out"] + b[..., None] * first["out"], whole["out"])
    assert np.allclose(os_.attention(q[:1], c, start, length, 0.4, 9, 3)["out"], os_.attention(q[:1], c, start, length, 0.4)["out"])


def test_attention_reads_shared_tokens_from_the_first_row():
    c, q = small_cache(2)
    start, length = [0, 2, 4, 6], [5, 9, 10]
    shared = os_.attention(q, c, start, length, 0.4, group_start=[0, 1, 3], shared_len=[2, 6])
    wide = dict(c, table=c["table"].copy())
    wide["table"][2, 0] = c["table"][1, 0]  # the third request's tokens 0 .. 3, and of the next page 4 and 5
    k = {n: c[n].copy() for n in "kv"}
    for n in "kv":
        k[n][c["table"][2, 1], :2] = c[n][c["table"][1, 1], :2]
    want = oa.attention(q, dict(wide, **k), start, length, 0.4)
    assert all(np.allclose(shared[n], want[n], atol=1e-14) for n in want)
