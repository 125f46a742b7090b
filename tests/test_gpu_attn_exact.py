"""sv_paged_attention where its result is known to the last bit or nearly so, and
one wrong row of keys or values among thousands shows.

Means.  With queries of zero every weight is exactly 1, whatever the keys hold.
Values of +1 and -1 at random have integer sums S over the n tokens that a row
sees, exact in binary32, so its result is S / n, off by the quotient's roundings
(2^-22 of it) and one to bf16 (2^-8).  A row left out, seen twice or taken from
elsewhere changes S by 1 or 2 in half of the channels or all, which shows in each
whose |S| is below 100: a standard deviation is sqrt(n) (50 for 2500 tokens).
lse is log(n).

Single tokens.  With keys of equal lengths and queries that are one of them times
64, that token has all the weight: the others' scores are 42 bits below (the test
asserts it), 2500 of them weigh 2^-30 together.  A score is below 2^15 in base 2,
so its own product and the reference's, one of them rounded, are 2^-10 apart at
most and its weight within 2^-10 of 1: it is 1 as bf16, and the result within
2^-10 of the value, a bf16 number of magnitude 1 to 2 from which that does not
round away (half a step is 2^-8)."""
import numpy as np
import pytest
import torch

from test_gpu_attn import call
from test_gpu_kv import new_cache, tables

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


def marked(f):
    for m in gpu:
        f = m(f)
    return f


SIZES = {  # new tokens and lengths with them, for 4 query heads a key head: 16, 32 and 128 rows a workgroup
    "16": ([3, 1, 4, 0], [2500, 130, 4, 9]),
    "32": ([7, 8, 2], [300, 2100, 77]),
    "128": ([40, 9, 65], [1500, 9, 333]),
}
CASES = [(rows, D, page) for rows in SIZES for D in (48, 64, 128, 256) for page in (4, 16, 64)]


def sequences(c, table, total, page, name):
    """Per request: its cached rows in 64 bits [total, heads, D], and which of them a page holds."""
    x = c[name + "_cache"].double()
    if c[name + "_scale"] is not None:
        x = x * torch.exp2(c[name + "_scale"].double() - 127).transpose(1, 2)[..., None]
    out = []
    for b, n in enumerate(total):
        at = torch.as_tensor(table[b])[torch.arange(n) // page].cuda()
        held = (at >= 0) & (at < x.shape[0])
        out.append((x[at.clamp(0, x.shape[0] - 1), torch.arange(n, device="cuda") % page], held))
    return out


def put(c, name, x, g):
    """Stores x, of few bits, in a cache; an 8-bit row at a scale of its own."""
    if c[name + "_scale"] is None:
        c[name + "_cache"].copy_(x.bfloat16())
    else:
        e = torch.randint(0, 6, c[name + "_scale"].shape, generator=g, device="cuda")
        c[name + "_scale"].copy_(127 + e)
        c[name + "_cache"].copy_((x * torch.exp2(-e.double()).transpose(1, 2)[..., None]).float().to(torch.float8_e4m3fn))


def inputs(rows, D, page, cache, seed):
    new, total = SIZES[rows]
    pages, table, start = tables(new, total, page, seed=seed)
    table[1, 1] = -1  # 4 to 64 tokens of the second request are absent
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = new_cache(cache, pages, page, 2, D)
    put(c, "k", torch.randn(c["k_cache"].shape, generator=g, device="cuda").double(), g)
    put(c, "v", torch.randint(0, 2, c["v_cache"].shape, generator=g, device="cuda").double() * 2 - 1, g)
    return new, total, table, start, g, c


def tolerance(mean):
    return np.abs(mean) * (2.0 ** -8 + 2.0 ** -21)


def ways(new, total):
    """Hints: divided as the lengths allow for, undivided, and without."""
    return dict(max_q_len=max(new), max_kv_len=max(total)), dict(max_q_len=max(new), max_kv_len=500), {}


WINDOWS = (0, 1, 70, 1100)


@marked
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,D,page", CASES)
def test_means_of_exact_values(rows, D, page, cache):
    new, total, table, start, g, c = inputs(rows, D, page, cache, D + page)
    q = torch.zeros((start[-1], 8, D), device="cuda", dtype=torch.bfloat16)
    seq = sequences(c, table, total, page, "v")
    for window, kw in ((w, kw) for w in WINDOWS for kw in ways(new, total)):
        o = call(q, c, table, start, total, window=window, **kw)
        for b, (v, held) in enumerate(seq):
            sums = torch.cat([torch.zeros_like(v[:1]), (v * held[:, None, None]).cumsum(0)])
            count = torch.cat([held[:1].long() * 0, held.long().cumsum(0)])
            place = torch.arange(total[b] - new[b], total[b], device="cuda")
            first = (place - window + 1).clamp(min=0) if window else place * 0
            n = (count[place + 1] - count[first]).double()
            mean = (sums[place + 1] - sums[first]) / n.clamp(min=1)[:, None, None]
            got, lse = (o[x][start[b]:start[b + 1]].double().cpu().numpy() for x in ("out", "lse"))
            want = mean.repeat_interleave(4, 1).cpu().numpy()
            assert (np.abs(got - want) <= tolerance(want)).all(), (window, kw, b)
            n = n.cpu().numpy()[:, None]
            assert (np.isneginf(lse) == (n == 0)).all()
            want = np.log(np.maximum(n, 1))
            assert (np.abs(lse - want) <= want * 2.0 ** -21 + 2.0 ** -22)[np.broadcast_to(n, lse.shape) > 0].all()


@marked
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,D,page", CASES)
def test_single_tokens(rows, D, page, cache):
    new, total, table, start, g, c = inputs(rows, D, page, cache, D + page + 1)
    k = torch.randn(c["k_cache"].shape, generator=g, device="cuda").double()
    put(c, "k", k / k.norm(dim=-1, keepdim=True) * D ** 0.5, g)
    sign = torch.randint(0, 2, c["v_cache"].shape, generator=g, device="cuda") * 2 - 1
    put(c, "v", sign * (1 + torch.randint(0, 8, c["v_cache"].shape, generator=g, device="cuda").double() / 8), g)
    ks, vs = sequences(c, table, total, page, "k"), sequences(c, table, total, page, "v")
    rng = np.random.default_rng(D + page)
    head = torch.arange(8, device="cuda") // 4
    for window in WINDOWS:
        q = torch.zeros((start[-1], 8, D), device="cuda", dtype=torch.bfloat16)
        want = torch.zeros((start[-1], 8, D), device="cuda", dtype=torch.float64)
        for b in range(len(new)):
            held = ks[b][1].cpu().numpy()
            for i in range(new[b]):
                p = total[b] - new[b] + i
                see = np.flatnonzero(held[: p + 1])
                see = see[see > p - window] if window else see
                if len(see) == 0:
                    continue
                at = rng.integers(0, len(see), 8)
                at[0], at[7] = 0, len(see) - 1  # the ends of what the row sees
                at, see = torch.from_numpy(at).cuda(), torch.from_numpy(see).cuda()
                q[start[b] + i] = (ks[b][0][see[at], head] * 64).bfloat16()
                want[start[b] + i] = vs[b][0][see[at], head]
                s = (q[start[b] + i].double() * ks[b][0][see][:, head]).sum(-1)  # [tokens, heads]
                top = s[at, torch.arange(8, device="cuda")].clone()
                s[at, torch.arange(8, device="cuda")] = -1e30
                assert (top - s).min() > 42 * np.log(2)
        for kw in ways(new, total):
            o = call(q, c, table, start, total, scale=1.0, window=window, **kw)
            assert torch.equal(o["out"].double(), want), (window, kw)


def test_the_bounds_see_one_row():
    """On the CPU: means over one row too few, and over one row in another's place, lie outside the tolerance."""
    g = np.random.default_rng(1)
    for n in (2, 40, 700, 2500):
        v = g.integers(0, 2, (n, 48)) * 2.0 - 1
        mean = v.mean(0)
        bf16 = lambda x: torch.from_numpy(x).bfloat16().double().numpy()
        assert (np.abs(bf16(mean) - mean) <= tolerance(mean)).all()
        for j in g.integers(0, n, 20):
            less, other = v.copy(), v.copy()
            less[j] = 0
            other[j] = g.integers(0, 2, 48) * 2.0 - 1
            for wrong in (less, other):
                assert (np.abs(bf16(wrong.mean(0)) - mean) > tolerance(mean)).any()
