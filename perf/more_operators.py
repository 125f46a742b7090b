"""The cases by which the operators of a served batch's step are measured, and their plain forms.

A verification step of speculative decoding takes pages for the new tokens, norms and turns their queries and keys,
writes keys and values to the cache and attends to what it holds.  Five operators of that pass:

  norm       norms of each query and key head and their rotary positions in one pass, forward and backward
  append     the same on the new tokens, whose keys and values go into a paged cache
  pages      pages of a cache taken and given back as requests' lengths say, and the slots of the new tokens
  sinks      attention over a paged cache with a sliding window and a few first tokens that stay visible
  shared     attention of requests whose first tokens are the same, which are read once for all of them

`run` computes them with elementary torch operations, or, where `own` is true, with the calls of
draft_token_verification_spec_amd; `exact` gives the same outputs from their definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GOLD = 0.6180339887498949
EPS = 1e-6
GRADIENTS = ("dq", "dk", "dq_weight", "dk_weight")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of a small batch, far into a long context: queries and keys of 64 tokens
        dict(name="norm_step", op="norm", tokens=64, q_heads=32, kv_heads=8, head_dim=128, rotary=128, layout="half",
             dtype="bf16", backward=False, first=900001),
        # a training step of a draft model on a packed batch: gradients of queries, keys and both weights
        dict(name="norm_backward", op="norm", tokens=8191, q_heads=32, kv_heads=8, head_dim=128, rotary=128, layout="half",
             dtype="bf16", backward=True, first=0),
        # the verification step of 256 requests with 4 drafts each into a bf16 cache
        dict(name="append_verify", op="append", batch=256, new=5, context=100, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=16, dtype="bf16", cache="bf16", rotary=128, layout="half"),
        # prompts of different lengths into an 8-bit cache, half of each head turned, and what the cache then holds
        dict(name="append_prompt_e4m3", op="append", batch=8, new=1500, context=0, ragged=True, q_heads=32, kv_heads=8,
             head_dim=128, page=64, dtype="f32", cache="e4m3", rotary=64, layout="interleaved"),
        # pages of the same verification step: 256 requests of up to 4000 tokens grow by 5
        dict(name="pages_step", op="pages", batch=256, new=5, context=4000, ragged=True, page=16, pool=1.0, shared=0),
        # many prompts admitted at once, a few more than the cache has pages for
        dict(name="pages_prompts", op="pages", batch=1500, new=1000, context=64, ragged=True, page=16, pool=0.95, shared=4),
        # one token of one request behind a long context: latency
        dict(name="sinks_single", op="sinks", batch=1, new=1, context=100000, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=16, cache="bf16", window=4096, sinks=4),
        # a decoding step of a batch of long conversations
        dict(name="sinks_decode", op="sinks", batch=64, new=1, context=30000, ragged=True, q_heads=32, kv_heads=8,
             head_dim=128, page=16, cache="bf16", window=2048, sinks=4),
        # a chunk of a long prompt in an 8-bit cache
        dict(name="sinks_chunk", op="sinks", batch=1, new=2048, context=8192, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, page=64, cache="e4m3", window=4096, sinks=128),
        # 8 samples drawn from one prompt
        dict(name="shared_samples", op="shared", batch=8, groups=1, new=1, shared=16000, context=100, ragged=True,
             q_heads=32, kv_heads=8, head_dim=128, page=16, cache="bf16"),
        # a decoding step of a batch behind one long system prompt
        dict(name="shared_decode", op="shared", batch=128, groups=1, new=1, shared=8000, context=500, ragged=True,
             q_heads=32, kv_heads=8, head_dim=128, page=16, cache="bf16"),
        # verification of 256 requests with 4 drafts each behind 8 prompts of a few shots
        dict(name="shared_verify_e4m3", op="shared", batch=256, groups=8, new=5, shared=4090, context=300, ragged=True,
             q_heads=32, kv_heads=8, head_dim=128, page=64, cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "pages", "sinks", "sinks", "shared", "shared"])
    head_dim = rng.choice([64, 80, 96, 128, 128, 256])
    kv_heads, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 4, 4, 7, 8])
    page, cache = rng.choice([8, 16, 32, 64, 128]), rng.choice(["bf16", "e4m3"])
    heads = dict(q_heads=min(32, kv_heads * group) // kv_heads * kv_heads, kv_heads=kv_heads, head_dim=head_dim)
    turned = dict(rotary=rng.choice([head_dim, head_dim // 2, 32]), layout=rng.choice(["half", "interleaved"]),
                  dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        return dict(op=op, tokens=_log(rng, 1, 4000), **heads, **turned, backward=rng.random() < 0.6,
                    first=_log(rng, 1, 1 << 20))
    if op == "append":
        batch = _log(rng, 1, 256)
        return dict(op=op, batch=batch, new=_log(rng, 1, max(2, 8000 // batch)), context=_log(rng, 1, 200),
                    ragged=rng.random() < 0.5, page=page, cache=cache, **heads, **turned)
    if op == "pages":
        batch = _log(rng, 1, 3000)
        return dict(op=op, batch=batch, new=_log(rng, 1, max(2, 1000000 // batch)), context=_log(rng, 1, 5000),
                    ragged=rng.random() < 0.7, page=page, pool=rng.choice([1.0, 1.0, rng.uniform(0.3, 1.0)]),
                    shared=rng.choice([0, 0, 3]))
    if op == "sinks":
        if rng.random() < 0.3:
            batch = rng.choice([1, 2, 5])
            new, context = _log(rng, 18, 2000 // batch), _log(rng, 1, 8000 // batch)
        else:
            batch = _log(rng, 1, 64)
            new, context = rng.choice([1, 1, rng.randint(2, 17)]), _log(rng, 1, 1000000 // batch)
        return dict(op=op, batch=batch, new=new, context=context, ragged=rng.random() < 0.7, page=page, cache=cache,
                    window=_log(rng, 1, 4096), sinks=rng.choice([1, 4, 4, _log(rng, 1, 200)]), **heads)
    groups = rng.choice([1, 1, 2, 5])
    batch = _log(rng, groups, 200)
    new = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, max(11, 1000 // batch))])
    return dict(op=op, batch=batch, groups=groups, new=new, shared=_log(rng, 16, 16000 // groups),
                context=_log(rng, 1, max(2, 50000 // batch)), ragged=rng.random() < 0.7, page=page, cache=cache, **heads)


def _lengths(n, most, ragged):
    """n lengths up to `most`, spread over three quarters of it where they are ragged."""
    if not ragged:
        return [most] * n
    return [max(min(1, most), most - int(0.75 * most * ((b * GOLD) % 1.0))) for b in range(n)]


def _plan(c):
    """(new tokens, cached tokens with them) of each sequence."""
    few = c["new"] <= 17  # a decoding or verification step: the contexts are ragged; a prompt: the prompts are
    new = _lengths(c["batch"], c["new"], c["ragged"] and not few)
    context = _lengths(c["batch"], c["context"], c["ragged"])
    return new, [n + m + (c["shared"] if c["op"] == "shared" else 0) for n, m in zip(new, context)]


def _groups(c):
    """The first sequence of each group, and the end of the last; tokens that each group shares."""
    first = [c["batch"] * i // c["groups"] for i in range(c["groups"] + 1)]
    return first, _lengths(c["groups"], c["shared"], c["ragged"])


def _pages_before(c, lengths):
    """Pages that each sequence of that length holds; the first ones it may share."""
    return [max(-(-n // c["page"]), c["shared"]) for n in lengths]


def work(c):
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "norm":
        heads = c["q_heads"] + c["kv_heads"]
        n = c["tokens"] * heads * c["head_dim"]
        return {"bytes": (3 if c["backward"] else 2) * n * size[c["dtype"]] + 8 * c["tokens"],
                "flops": n * (12 if c["backward"] else 4) + 3 * c["tokens"] * heads * c["rotary"]}
    new, total = _plan(c)
    t = sum(new)
    if c["op"] == "pages":
        held, need = _pages_before(c, [a - n for a, n in zip(total, new)]), _pages_before(c, total)
        moved = sum(b - a for a, b in zip(held, need))
        return {"bytes": 32 * c["batch"] + 20 * int(moved * c["pool"]) + 16 * t, "flops": 0}
    row = c["kv_heads"] * (2 * c["head_dim"] if c["cache"] == "bf16" else c["head_dim"] + 1)  # of keys or of values
    q = c["q_heads"] * c["head_dim"]
    if c["op"] == "append":
        kv = c["kv_heads"] * c["head_dim"]
        back = 4 * t * kv if c["cache"] == "e4m3" else 0  # the read-back's rows
        return {"bytes": t * (2 * q + 2 * kv) * size[c["dtype"]] + 2 * t * row * (2 if back else 1) + back,
                "flops": t * (c["q_heads"] + c["kv_heads"]) * (3 * c["rotary"] + 4 * c["head_dim"])}
    if c["op"] == "sinks":
        w, k = c["window"], c["sinks"]
        sees = lambda p: min(p, w) + min(max(p - w, 0), k)  # tokens seen by the p-th
        seen = sum(sees(p) for n, s in zip(new, total) for p in range(s - n + 1, s + 1))
        read = sum(min(n + w - 1, s) + min(max(s - n - w + 1, 0), k) for n, s in zip(new, total))
    else:
        first, shared = _groups(c)
        seen = sum(n * (2 * s - n + 1) // 2 for n, s in zip(new, total))
        of = [g for g in range(c["groups"]) for _ in range(first[g + 1] - first[g])]
        read = sum(shared) + sum(s - shared[of[b]] for b, s in enumerate(total))
    return {"bytes": 2 * read * row + 4 * t * q + 4 * t * c["q_heads"], "flops": 4 * seen * q}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _tables(c, gen, total, shared):
    """A page table whose pages lie in the cache in random order, a few of them unused.  The full pages of what a
    group shares are the same for its sequences; of a page that it shares in part each has a copy."""
    page, B = c["page"], len(total)
    need = [-(-t // page) for t in total]
    full = [s // page for s in shared]
    own_pages = [n - f for n, f in zip(need, full)]
    first, group_len = _groups(c) if c["op"] == "shared" else ([0], [])
    group_full = [s // page for s in group_len]
    num_pages = sum(own_pages) + sum(group_full) + 3
    order = torch.randperm(num_pages, generator=gen, device=DEV).to(torch.int32)
    at = torch.full((B, max(max(need), 1)), num_pages - 1, dtype=torch.int64)
    used = 0
    for g, n in enumerate(group_full):
        at[first[g]:first[g + 1], :n] = torch.arange(used, used + n)
        used += n
    for b in range(B):
        at[b, full[b]:need[b]] = torch.arange(used, used + own_pages[b])
        used += own_pages[b]
    return num_pages, order[at.to(DEV)].contiguous()


def _cache(c, gen, num_pages):
    shape = (num_pages, c["page"], c["kv_heads"], c["head_dim"])
    s = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
        if c["cache"] == "e4m3":
            s[name + "_cache"] = (x * 96).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[name + "_scale"] = torch.randint(119, 122, (num_pages, c["kv_heads"], c["page"]), generator=gen, device=DEV,
                                               dtype=torch.uint8)
        else:
            s[name + "_cache"], s[name + "_scale"] = x, None
    return s


def _starts(lengths):
    return torch.tensor([0] + lengths, device=DEV).cumsum(0).to(torch.int32)


def _int32(values):
    return torch.tensor(values, device=DEV, dtype=torch.int32)


def _heads(c, gen, rows, heads):
    """Rows whose heads' channels differ in size, as they do in trained models."""
    size = torch.exp(torch.randn((heads, c["head_dim"]), generator=gen, device=DEV) * 0.7)
    x = torch.randn((rows, heads, c["head_dim"]), generator=gen, device=DEV)
    return (x * size).to(TYPES[c["dtype"]])


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] in ("norm", "append"):
        i = torch.arange(0, c["rotary"], 2, device=DEV, dtype=torch.float64)
        s["freq"] = 10000.0 ** (-i / c["rotary"])  # radians a position
        for n in ("q", "k"):
            w = 1 + 0.3 * torch.randn(c["head_dim"], generator=gen, device=DEV)
            s[n + "_weight"] = w.to(TYPES[c["dtype"]])
    if c["op"] == "norm":
        # a projection writes the queries, keys and values of a token side by side
        qkv = _heads(c, gen, c["tokens"], c["q_heads"] + 2 * c["kv_heads"])
        s["q"], s["k"] = qkv.split([c["q_heads"], c["kv_heads"], c["kv_heads"]], 1)[:2]
        jump = torch.randint(0, 7, (c["tokens"],), generator=gen, device=DEV)
        s["positions"] = c["first"] + torch.arange(c["tokens"], device=DEV) + jump
        if c["backward"]:
            s["dq"], s["dk"] = _heads(c, gen, c["tokens"], c["q_heads"]), _heads(c, gen, c["tokens"], c["kv_heads"])
        return s
    new, total = _plan(c)
    s["max_new"], s["max_total"], s["rows"] = max(new), max(total), sum(new)
    s["query_start"], s["kv_len"] = _starts(new), _int32(total)
    if c["op"] == "pages":
        before = [t - n for t, n in zip(total, new)]
        held, need = _pages_before(c, before), _pages_before(c, total)
        s["before"], s["pages_held"], s["shared_pages"] = _int32(before), _int32(held), _int32([c["shared"]] * c["batch"])
        most = [b - a for a, b in zip(held, need)]
        free = int(sum(most) * c["pool"])
        num_pages = sum(held) - c["shared"] * (c["batch"] - 1) + free
        order = torch.randperm(num_pages, generator=gen, device=DEV).to(torch.int32)
        s["free_pages"], s["free_count"] = order.clone(), _int32([free])  # those above the count are in use
        s["page_table"] = torch.full((c["batch"], max(need) + 2), -1, device=DEV, dtype=torch.int32)
        at = free
        shared = order[at:at + c["shared"]]
        at += c["shared"]
        for b, n in enumerate(held):
            s["page_table"][b, :c["shared"]] = shared
            s["page_table"][b, c["shared"]:n] = order[at:at + n - c["shared"]]
            at += n - c["shared"]
        s["most"] = max(max(most), 1)
        return s
    shared = [0] * c["batch"]
    if c["op"] == "shared":
        first, group_len = _groups(c)
        s["group_start"], s["shared_len"] = _int32(first), _int32(group_len)
        s["max_shared"], s["max_group"] = max(group_len), max(sum(new[a:b]) for a, b in zip(first, first[1:]))
        shared = [n for g, n in enumerate(group_len) for _ in range(first[g], first[g + 1])]
        s["max_own"] = max(t - n for t, n in zip(total, shared))
    num_pages, s["page_table"] = _tables(c, gen, total, shared)
    s.update(_cache(c, gen, num_pages))
    if c["op"] == "shared":
        for g, n in enumerate(group_len):  # the copies of what is shared of a page
            i, part = n // c["page"], n % c["page"]
            if part:
                pages = s["page_table"][first[g]:first[g + 1], i].long()
                for x in ("k", "v"):
                    rows = s[x + "_cache"].view(torch.uint8)
                    rows[pages[1:], :part] = rows[pages[0], :part].clone()
                    if s[x + "_scale"] is not None:
                        s[x + "_scale"][pages[1:], :, :part] = s[x + "_scale"][pages[0], :, :part].clone()
    if c["op"] == "append":
        qkv = _heads(c, gen, s["rows"], c["q_heads"] + 2 * c["kv_heads"])
        s["q"], s["k"], s["v"] = qkv.split([c["q_heads"], c["kv_heads"], c["kv_heads"]], 1)
        s["begin"] = s["kv_len"] - _int32(new)
    else:
        s["q"] = torch.randn((s["rows"], c["q_heads"], c["head_dim"]), generator=gen, device=DEV, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rotate(x, positions, freq, layout, backward=False):
    """x in 32 bits [rows, heads, head_dim] with its first 2 * len(freq) channels turned; angles in 64 bits."""
    angle = positions.double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if backward:
        sin = -sin
    r = 2 * freq.numel()
    y = x.clone()
    if layout == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _normed(x, weight):
    """(normed rows, their inverse norms) in 32 bits."""
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r * weight.float(), r


def _plain_norm(s, c):
    out = {}
    for n in ("q", "k"):
        if not c["backward"]:
            out[n] = _rotate(_normed(s[n], s[n + "_weight"])[0], s["positions"], s["freq"], c["layout"]).to(s[n].dtype)
            continue
        r = _normed(s[n], s[n + "_weight"])[1]
        unit = s[n].float() * r
        g = _rotate(s["d" + n].float(), s["positions"], s["freq"], c["layout"], backward=True)
        out["d" + n + "_weight"] = (g * unit).sum((0, 1), dtype=torch.float64).float()
        g = g * s[n + "_weight"].float()
        out["d" + n] = (r * (g - unit * (g * unit).mean(-1, keepdim=True))).to(s[n].dtype)
    return {n: out[n] for n in (GRADIENTS if c["backward"] else ("q", "k"))}


def _rows(start, count):
    """The sequence of each of `count` rows and its place there."""
    row = torch.arange(count, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(start, row, right=True) - 1
    return seq, (row - start[seq]).long()


def _slots(table, seq, place, page):
    return table[seq, place // page].long(), place % page


def _quantise(x):
    """8-bit values of rows [..., head_dim] and the biased exponents of their scales: the least power of two that
    brings the largest magnitude to at most 448."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = (torch.where(m > 0.875, e - 8, e - 9)).clamp(-126, 127)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _read(cache, scale, page, slot):
    """Rows of a cache in 32 bits."""
    if scale is None:
        return cache[page, slot].float()
    x = cache.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
    e = scale.transpose(1, 2)[page, slot].int() - 127
    return torch.ldexp(x, e[..., None])


def _write(cache, scale, page, slot, x):
    if scale is None:
        cache[page, slot] = x.to(cache.dtype)
    else:
        q, e = _quantise(x)
        cache.view(torch.uint8)[page, slot] = q.view(torch.uint8)
        scale.transpose(1, 2)[page, slot] = e


def _plain_append(s, c):
    seq, i = _rows(s["query_start"], s["rows"])
    place = i + s["begin"][seq]
    q = _rotate(_normed(s["q"], s["q_weight"])[0], place, s["freq"], c["layout"]).to(s["q"].dtype)
    k = _rotate(_normed(s["k"], s["k_weight"])[0], place, s["freq"], c["layout"])
    page, slot = _slots(s["page_table"], seq, place, c["page"])
    _write(s["k_cache"], s["k_scale"], page, slot, k)
    _write(s["v_cache"], s["v_scale"], page, slot, s["v"].float())
    if c["cache"] == "bf16":
        return dict(q=q, k=s["k_cache"], v=s["v_cache"])
    return dict(q=q, k=_read(s["k_cache"], s["k_scale"], page, slot).to(torch.bfloat16),
                v=_read(s["v_cache"], s["v_scale"], page, slot).to(torch.bfloat16))


def _put(to, at, on, values):
    """to[at] = values where `on`."""
    wide = torch.cat([to, to.new_zeros(1)])
    wide[torch.where(on, at, to.numel()).flatten()] = values.flatten()
    to.copy_(wide[:-1])


def _move_pages(s, c, lengths):
    """Pages given back and taken so that each sequence holds what its length needs; 1 for each that has got them.
    Given back, and taken, from the top of the free pages: sequences in order, their pages in order."""
    table, held, free, count = s["page_table"], s["pages_held"], s["free_pages"], s["free_count"]
    need = torch.maximum((lengths.clamp(min=0) + c["page"] - 1) // c["page"], torch.minimum(s["shared_pages"], held))
    give, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    i = torch.arange(s["most"], device=DEV)
    # given back: the first sequence's first page ends up on top
    before = give.cumsum(0) - give
    at = (count + give.sum() - 1 - before)[:, None] - i
    on = i < give[:, None]
    page = table.gather(1, (need[:, None] + i).clamp(max=table.shape[1] - 1))
    _put(free, at, on, page)
    column = torch.arange(table.shape[1], device=DEV)
    table.masked_fill_((column >= need[:, None]) & (column < held[:, None]), -1)
    count += give.sum()
    # taken, while there are enough
    upto = take.cumsum(0)
    granted = (take == 0) | (upto <= count)
    take = torch.where(granted, take, 0)
    at = (count - 1 - (upto - take))[:, None] - i
    on = i < take[:, None]
    row = torch.arange(table.shape[0], device=DEV)[:, None] * table.shape[1]
    _put(table.view(-1), row + held[:, None] + i, on, free[at.clamp(min=0)])
    held.copy_(torch.where(granted, need, held))
    count -= take.sum()
    return granted.int()


def _plain_pages(s, c):
    granted = _move_pages(s, c, s["kv_len"])
    seq, i = _rows(s["query_start"], s["rows"])
    place = i + (s["kv_len"] - s["query_start"].diff())[seq]
    page, slot = _slots(s["page_table"], seq, place, c["page"])
    slots = torch.where(place // c["page"] < s["pages_held"][seq], page * c["page"] + slot, -1)
    again = _move_pages(s, c, s["before"])
    return dict(granted=granted, slots=slots, positions=place, again=again, table=s["page_table"], held=s["pages_held"],
                free=s["free_pages"], count=s["free_count"])


def _padded(s, c):
    """Queries [batch, kv head, group * n, d] in 32 bits and the place of each of the n rows [batch, n]."""
    batch, n, d, hkv = c["batch"], s["max_new"], c["head_dim"], c["kv_heads"]
    start = s["query_start"].long()
    row = torch.arange(n, device=DEV)
    at = (start[:-1, None] + row).clamp(max=s["rows"] - 1)
    q = s["q"][at].float().view(batch, n, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    return q, (s["kv_len"] - s["query_start"].diff())[:, None] + row


def _unpadded(s, c, out, lse):
    batch, n, heads = c["batch"], s["max_new"], c["q_heads"]
    g = heads // c["kv_heads"]
    out = out.view(batch, -1, g, n, c["head_dim"]).permute(0, 3, 1, 2, 4).reshape(batch, n, heads, -1)
    lse = lse.view(batch, -1, g, n).permute(0, 3, 1, 2).reshape(batch, n, heads)
    seq, i = _rows(s["query_start"], s["rows"])
    return dict(out=out[seq, i].to(torch.bfloat16), lse=lse[seq, i])


def _keys(s, name, page, slot):
    """Cached rows [batch, kv head, tokens, d] in 32 bits."""
    return _read(s[name + "_cache"], s[name + "_scale"], page, slot).transpose(1, 2).contiguous()


def _plain_sinks(s, c):
    # the first tokens, and those that some row's window reaches
    reach = min(s["max_total"], c["window"] + s["max_new"] - 1)
    head = torch.arange(min(c["sinks"], s["max_total"]), device=DEV).expand(c["batch"], -1)
    tail = s["kv_len"].long()[:, None] - reach + torch.arange(reach, device=DEV)
    token = torch.cat([head, torch.where(tail >= c["sinks"], tail, -1)], 1)
    page, slot = _slots(s["page_table"], torch.arange(c["batch"], device=DEV)[:, None], token.clamp(min=0), c["page"])
    q, place = _padded(s, c)
    score = torch.matmul(q, _keys(s, "k", page, slot).transpose(2, 3)).mul_(c["head_dim"] ** -0.5)
    j, p = token[:, None], place[..., None]
    see = (j >= 0) & (j <= p) & ((j > p - c["window"]) | (j < c["sinks"]))
    score.view(c["batch"], c["kv_heads"], -1, *see.shape[1:]).masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    mass = p.sum(-1, keepdim=True)
    return _unpadded(s, c, torch.matmul(p, _keys(s, "v", page, slot)) / mass, top + mass.log())


def _plain_shared(s, c):
    batch, d, n = c["batch"], c["head_dim"], s["max_new"]
    first, shared = _groups(c)
    q, place = _padded(s, c)
    # each sequence's own tokens
    of = torch.tensor([shared[g] for g in range(c["groups"]) for _ in range(first[g], first[g + 1])], device=DEV)
    token = of[:, None] + torch.arange(s["max_own"], device=DEV)
    at = token.clamp(max=s["page_table"].shape[1] * c["page"] - 1)
    page, slot = _slots(s["page_table"], torch.arange(batch, device=DEV)[:, None], at, c["page"])
    score = torch.matmul(q, _keys(s, "k", page, slot).transpose(2, 3)).mul_(d ** -0.5)
    hide = token[:, None] > place[..., None]
    score.view(batch, c["kv_heads"], -1, *hide.shape[1:]).masked_fill_(hide[:, None, None], -math.inf)
    own_top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(own_top == -math.inf, 0, own_top)).exp_()
    mass, out = p.sum(-1, keepdim=True), torch.matmul(p, _keys(s, "v", page, slot))
    top = torch.empty_like(own_top)
    for g in range(c["groups"]):  # what a group shares, once for all its rows
        a, b, m = first[g], first[g + 1], shared[g]
        place = torch.arange(m, device=DEV)
        page, slot = _slots(s["page_table"][a:a + 1], torch.zeros_like(place), place, c["page"])
        k, v = (_read(s[x + "_cache"], s[x + "_scale"], page, slot).transpose(0, 1).contiguous() for x in ("k", "v"))
        rows = q[a:b].transpose(0, 1).reshape(c["kv_heads"], -1, d)
        score = torch.matmul(rows, k.transpose(1, 2)).mul_(d ** -0.5)
        back = lambda x: x.view(c["kv_heads"], b - a, -1, x.shape[-1]).transpose(0, 1)
        t = score.amax(-1, keepdim=True)
        top[a:b] = torch.maximum(back(t), own_top[a:b])
        p = score.sub_(t).exp_()
        scale, own_scale = torch.exp(back(t) - top[a:b]), torch.exp(own_top[a:b] - top[a:b])
        mass[a:b] = mass[a:b] * own_scale + back(p.sum(-1, keepdim=True)) * scale
        out[a:b] = out[a:b] * own_scale + back(torch.matmul(p, v)) * scale
    return _unpadded(s, c, out / mass, top + mass.log())


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"norm": _plain_norm, "append": _plain_append, "pages": _plain_pages, "sinks": _plain_sinks,
            "shared": _plain_shared}[c["op"]](s, c)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s, c):
    import draft_token_verification_spec_amd as sv

    if c["op"] == "norm":
        kw = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, layout=c["layout"])
        if c["backward"]:
            return sv.sv_qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["positions"], s["freq"], **kw)
        return sv.sv_qk_norm_rope(s["q"], s["k"], s["positions"], s["freq"], **kw)
    if c["op"] == "pages":
        pool = (s["page_table"], s["pages_held"], s["free_pages"], s["free_count"])
        kw = dict(page_size=c["page"], shared_pages=s["shared_pages"])
        o = sv.sv_kv_pages(*pool, s["kv_len"], query_start=s["query_start"], rows=s["rows"], **kw)
        again = sv.sv_kv_pages(*pool, s["before"], **kw)
        return dict(granted=o["granted"], slots=o["slots"], positions=o["positions"], again=again["granted"],
                    table=s["page_table"], held=s["pages_held"], free=s["free_pages"], count=s["free_count"])
    cache = (s["k_cache"], s["v_cache"], s["page_table"])
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "append":
        o = sv.sv_kv_append_normed(s["k"], s["v"], *cache, s["query_start"], s["kv_len"], q=s["q"], freq=s["freq"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, layout=c["layout"], **scales)
        if c["cache"] == "bf16":
            return dict(q=o["q"], k=s["k_cache"], v=s["v_cache"])
        back = sv.sv_kv_gather(*cache, s["query_start"], s["rows"], kv_begin=s["begin"], **scales)
        return dict(q=o["q"], k=back["k"], v=back["v"])
    kw = dict(max_q_len=s["max_new"], want_lse=True, **scales)
    if c["op"] == "sinks":
        return sv.sv_paged_attention_sinks(s["q"], *cache, s["query_start"], s["kv_len"], window=c["window"],
                                           sinks=c["sinks"], max_kv_len=s["max_total"], **kw)
    return sv.sv_paged_attention_shared(s["q"], *cache, s["query_start"], s["kv_len"], s["group_start"], s["shared_len"],
                                        max_group_len=s["max_group"], max_shared_len=s["max_shared"],
                                        max_own_len=s["max_own"], **kw)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(x):
    """The nearest value of the 8-bit type (ties to an even last bit), for magnitudes of at most 448: its step is
    2^-3 of the value's power of two, and at least 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _stored(x, kind):
    """What the cache stands for after rows x were written to it."""
    if kind == "bf16":
        return x.to(torch.bfloat16).double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    return _e4m3(x * torch.exp2(-e)) * torch.exp2(e)


def _turned(x, place, freq, layout):
    z = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), place.double()[:, None, None] * freq)
    r = 2 * freq.numel()
    pairs = x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2) if layout == "half" else x[..., :r].unflatten(-1, (-1, 2))
    w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    w = w.transpose(-1, -2) if layout == "half" else w
    return torch.cat([w.flatten(-2), x[..., r:]], -1)


def _of_unit_size(x, weight):
    return weight * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _held(s, name, b, place):
    """Cached rows of sequence b at these places."""
    page = s["case"]["page"]
    at, slot = s["page_table"][b][place // page].long(), place % page
    if s[name + "_scale"] is None:
        return s[name + "_cache"][at, slot].double()
    x = s[name + "_cache"].view(torch.uint8)[at, slot].view(torch.float8_e4m3fn).double()
    return x * torch.exp2(s[name + "_scale"][at, :, slot].double() - 127)[..., None]


def _exact_pages(s, c):
    """One sequence and one page at a time."""
    table, held = s["page_table"].tolist(), s["pages_held"].tolist()
    free, count = s["free_pages"].tolist(), int(s["free_count"])

    def move(lengths):
        nonlocal count
        granted = []
        need = [max(-(-max(n, 0) // c["page"]), min(c["shared"], h)) for n, h in zip(lengths, held)]
        back = [table[b].pop(need[b]) for b in range(c["batch"]) for _ in range(need[b], held[b])]
        for b in range(c["batch"]):
            held[b] = min(held[b], need[b])
            table[b] += [-1] * (s["page_table"].shape[1] - len(table[b]))
        for page in reversed(back):
            free[count] = page
            count += 1
        refused = False
        for b in range(c["batch"]):
            lack = need[b] - held[b]
            refused = refused or lack > count
            granted.append(int(lack == 0 or not refused))
            for _ in range(lack if granted[b] else 0):
                count -= 1
                table[b][held[b]] = free[count]
                held[b] += 1
        return granted

    new, total = _plan(c)
    granted = move(total)
    slots, positions = [], []
    for b, (n, t) in enumerate(zip(new, total)):
        places = range(t - n, t)
        positions += places
        slots += [table[b][p // c["page"]] * c["page"] + p % c["page"] if p // c["page"] < held[b] else -1 for p in places]
    again = move([t - n for n, t in zip(new, total)])
    whole = lambda x: torch.tensor(x, device=DEV)
    return dict(granted=whole(granted), slots=whole(slots), positions=whole(positions), again=whole(again),
                table=whole(table), held=whole(held), free=whole(free), count=whole([count]))


def _exact_norm(s, c):
    with torch.enable_grad():
        out = {}
        for n in ("q", "k"):
            x, w = (t.double().contiguous().requires_grad_() for t in (s[n], s[n + "_weight"]))
            y = _turned(_of_unit_size(x, w), s["positions"], s["freq"], c["layout"])
            if c["backward"]:
                out["d" + n], out["d" + n + "_weight"] = torch.autograd.grad(y, (x, w), s["d" + n].double())
            else:
                out[n] = y.detach()
    return {n: out[n] for n in (GRADIENTS if c["backward"] else ("q", "k"))}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        return _exact_norm(s, c)
    if c["op"] == "pages":
        return _exact_pages(s, c)
    new, total = _plan(c)
    starts = [sum(new[:b]) for b in range(len(new))]
    if c["op"] == "append":
        place = torch.cat([torch.arange(t - n, t, device=DEV) for n, t in zip(new, total)])
        q = _turned(_of_unit_size(s["q"].double(), s["q_weight"].double()), place, s["freq"], c["layout"])
        k = _turned(_of_unit_size(s["k"].double(), s["k_weight"].double()), place, s["freq"], c["layout"])
        k, v = _stored(k, c["cache"]), _stored(s["v"].double(), c["cache"])
        if c["cache"] == "e4m3":
            return dict(q=q, k=k, v=v)
        hold = dict(k=s["k_cache"].double(), v=s["v_cache"].double())
        for b, (at, n, t) in enumerate(zip(starts, new, total)):
            p = torch.arange(t - n, t, device=DEV)
            where = (s["page_table"][b][p // c["page"]].long(), p % c["page"])
            hold["k"][where], hold["v"][where] = k[at:at + n], v[at:at + n]
        return dict(q=q, **hold)
    d, g = c["head_dim"], c["q_heads"] // c["kv_heads"]
    out = torch.empty((s["rows"], c["q_heads"], d), device=DEV, dtype=torch.float64)
    lse = torch.empty((s["rows"], c["q_heads"]), device=DEV, dtype=torch.float64)
    for b, (at, n, t) in enumerate(zip(starts, new, total)):
        token, place = torch.arange(t, device=DEV), torch.arange(t - n, t, device=DEV)[:, None]
        if c["op"] == "sinks":
            token = token[(token < c["sinks"]) | (token > t - n - c["window"])]
            hide = (token > place) | ((token <= place - c["window"]) & (token >= c["sinks"]))
        else:
            hide = token > place
        k, v = _held(s, "k", b, token), _held(s, "v", b, token)
        for h in range(c["q_heads"]):
            z = (s["q"][at:at + n, h].double() @ k[:, h // g].T.contiguous()) / math.sqrt(d)
            z[hide] = -math.inf
            lse[at:at + n, h] = torch.logsumexp(z, -1)
            out[at:at + n, h] = torch.softmax(z, -1) @ v[:, h // g].contiguous()
    return dict(out=out, lse=lse)
