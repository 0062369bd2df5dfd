"""Measured cases of the cache operators: append with rotary positions, attention weight per key,
eviction by that weight, and cross attention.

Every case is a call that a serving program makes next to ``splitkv_decode``. With ``own`` false the
operators run in their plain form (elementary torch operations in 32 bits), with ``own`` true through the
library's entry points. Caches are paged: pools of pages, one block table row for each sequence.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
#: How the pairs of a rotated head are dealt to three position axes (time, height, width).
SECTIONS = {(64, 1): (64,), (64, 3): (24, 20, 20), (32, 1): (32,), (32, 3): (12, 10, 10)}


def listed():
    return [
        # one new token of one request at the default decode workload's context: latency alone
        dict(name="append_token_b1", op="append", batch=1, lo=1, hi=1, cached=5900, heads=16, kv_heads=2, dim=128,
             rot=128, axes=1, paired="halves", page=16, dtype="bf16", layout="HND", lens_seed=1),
        # one decode step of a batch over an e4m3 cache, image and video positions
        dict(name="append_token_b32_e4m3", op="append", batch=32, lo=1, hi=1, cached=4000, heads=32, kv_heads=8, dim=128,
             rot=128, axes=3, paired="halves", page=16, dtype="e4m3", layout="NHD", lens_seed=2),
        # the prompts of eight requests, of unequal lengths, entering the cache at once
        dict(name="append_prompts", op="append", batch=8, lo=700, hi=9000, cached=0, heads=32, kv_heads=4, dim=128,
             rot=128, axes=3, paired="halves", page=16, dtype="bf16", layout="HND", lens_seed=3),
        # which keys the default decode workload's token looked at
        dict(name="weights_ctx5900", op="weights", batch=1, tokens=1, lo=5900, hi=5900, heads=16, kv_heads=2, page=16,
             dtype="bf16", layout="HND", lens_seed=4),
        # the same for a batch of long contexts over an e4m3 cache
        dict(name="weights_b8_32k_e4m3", op="weights", batch=8, tokens=1, lo=28672, hi=32768, heads=32, kv_heads=4, page=16,
             dtype="e4m3", layout="HND", lens_seed=5),
        # a batch of very unequal contexts, an observation window of four tokens
        dict(name="weights_mixed_b32_t4", op="weights", batch=32, tokens=4, lo=256, hi=131072, heads=32, kv_heads=8, page=16,
             dtype="bf16", layout="HND", lens_seed=6),
        # one request's context cut to a third
        dict(name="evict_ctx5900", op="evict", batch=1, lo=5900, hi=5900, budget=2048, sink=4, recent=256, kv_heads=2,
             dim=128, page=16, dtype="bf16", layout="HND", lens_seed=7),
        # a latent cache of 64k rows in 8 bits cut to a quarter
        dict(name="evict_latent_64k_e4m3", op="evict", batch=1, lo=65536, hi=65536, budget=16384, sink=4, recent=1024, kv_heads=1,
             dim=576, page=64, dtype="e4m3", layout="HND", lens_seed=8),
        # a batch of unequal contexts: some under the budget, some cut to an eighth
        dict(name="evict_mixed_b32", op="evict", batch=32, lo=256, hi=131072, budget=16001, sink=16, recent=2000, kv_heads=8,
             dim=128, page=16, dtype="bf16", layout="HND", lens_seed=9),
        # one decoder token of eight requests over encoder states (no shared heads)
        dict(name="cross_token_b8", op="cross", batch=8, tlo=1, thi=1, lo=900, hi=1500, heads=16, kv_heads=16, page=16,
             layout="HND", lens_seed=10),
        # decoder prompts of unequal lengths over encoder states of other lengths
        dict(name="cross_ragged_b4", op="cross", batch=4, tlo=37, thi=900, lo=1, hi=4100, heads=32, kv_heads=8, page=16,
             layout="NHD", lens_seed=11),
        # long prompts over long encoder states: matrix products
        dict(name="cross_long_b2", op="cross", batch=2, tlo=4001, thi=4096, lo=8000, hi=8192, heads=32, kv_heads=4, page=64,
             layout="HND", lens_seed=12),
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "weights", "evict", "cross"])
    seed = rng.randrange(1 << 30)
    layout = rng.choice(["HND", "NHD"])
    dtype = rng.choice(["bf16", "e4m3"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64])
    if op == "append":
        latent = rng.random() < 0.25
        batch = between(1, 32)
        hi = between(1, max(1, 30000 // batch))
        rot = 64 if latent else rng.choice([64, 128])
        return dict(op=op, batch=batch, lo=max(1, hi // 9), hi=hi, cached=rng.choice([0, between(1, 3000)]),
                    heads=128 if latent else kv * group, kv_heads=1 if latent else kv, dim=576 if latent else 128, rot=rot,
                    axes=1 if latent else rng.choice([1, 3]), paired="neighbours" if latent else rng.choice(["halves", "neighbours"]),
                    page=page, dtype=dtype, layout="HND" if latent else layout, lens_seed=seed)
    if op == "weights":
        batch = between(1, 32)
        hi = between(2, max(40, 2000000 // (batch * kv)))
        return dict(op=op, batch=batch, tokens=rng.choice([1, 1, 2, 3, 4]), lo=max(1, hi // 20), hi=hi, heads=kv * group,
                    kv_heads=kv, page=page, dtype=dtype, layout=layout, lens_seed=seed)
    if op == "evict":
        latent = rng.random() < 0.25
        kv = 1 if latent else kv
        batch = between(1, 32)
        hi = between(100, 2000000 // (batch * kv) if not latent else 400000 // batch)
        budget = between(16, max(20, hi))
        return dict(op=op, batch=batch, lo=max(1, hi // 20), hi=hi, budget=budget, sink=rng.choice([0, 4]),
                    recent=rng.choice([0, budget // 8]), kv_heads=kv, dim=576 if latent else 128, page=page, dtype=dtype,
                    layout="HND" if latent else layout, lens_seed=seed)
    batch = between(1, 8)
    thi = between(1, 2000 // batch + 40)
    hi = between(16, 8192)
    return dict(op=op, batch=batch, tlo=max(1, thi // 5), thi=thi, lo=max(1, hi // 5), hi=hi, heads=kv * group, kv_heads=kv,
                page=page, layout=layout, lens_seed=seed)


# ------------------------------------------------------------------ inputs

def _lengths(case, lo, hi, salt):
    """Log-uniform lengths, the case's own (they do not depend on the inputs' seed)."""
    rng = random.Random(case["lens_seed"] * 7 + salt)
    return [min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))) for _ in range(case["batch"])]


def _cache_lengths(case):
    if case["op"] == "append":
        new = _lengths(case, case["lo"], case["hi"], 1)
        old = [c if c < 2 else c - (i * 131) % (c // 2) for i, c in enumerate([case["cached"]] * case["batch"])]
        return [n + o for n, o in zip(new, old)]
    if case["op"] == "weights":
        return [max(case["tokens"], n) for n in _lengths(case, case["lo"], case["hi"], 1)]
    return _lengths(case, case["lo"], case["hi"], 1)


def _query_counts(case):
    if case["op"] == "append":
        return _lengths(case, case["lo"], case["hi"], 1)
    if case["op"] == "cross":
        return _lengths(case, case["tlo"], case["thi"], 2)
    return [case.get("tokens", 1)] * case["batch"]


def _tables(lens, page, seed):
    """A block table over randomly placed pages: (table [B][max_pages], pages in the pool)."""
    counts = [-(-n // page) for n in lens]
    order = list(range(sum(counts)))
    random.Random(seed).shuffle(order)
    width = max(1, max(counts))
    rows, at = [], 0
    for c in counts:
        rows.append(order[at:at + c] + [0] * (width - c))
        at += c
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), max(1, sum(counts))


def _pool(g, pages, heads, page, dim, case):
    shape = (pages, heads, page, dim) if case["layout"] == "HND" else (pages, page, heads, dim)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if case.get("dtype") == "e4m3":  # codes whose values times kv_scale are the cache's
        return (x * 64.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


def _offsets(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens = _cache_lengths(case)
    counts = _query_counts(case)
    table, pages = _tables(lens, case["page"], seed)
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), pages=pages,
             max_len=max(lens), width=table.shape[1] * case["page"])
    getattr(_Inputs, case["op"])(s, case, g, lens, counts)
    return s


class _Inputs:
    @staticmethod
    def append(s, case, g, lens, counts):
        n, heads, kv, dim = sum(counts), case["heads"], case["kv_heads"], case["dim"]
        latent = dim == 576
        # the projections' output holds queries, keys and values of a token side by side
        wide = (heads + kv) * dim if latent else (heads + 2 * kv) * dim
        rows = torch.randn((n, wide), generator=g, device="cuda", dtype=torch.bfloat16)
        s["q"] = rows[:, :heads * dim].view(n, heads, dim)
        s["k"] = rows[:, heads * dim:(heads + kv) * dim].view(n, kv, dim)
        s["v"] = None if latent else rows[:, (heads + kv) * dim:].view(n, kv, dim)
        s["k_pages"] = _pool(g, s["pages"], kv, case["page"], dim, case)
        s["v_pages"] = None if latent else _pool(g, s["pages"], kv, case["page"], dim, case)
        s["kv_scale"] = 1.0 / 64.0
        s["cu"] = torch.tensor(_offsets(counts), dtype=torch.int32, device="cuda")
        # a token's index in its sequence, and for three axes its place on a grid of 8 by 8 patches in a frame
        at = torch.cat([torch.arange(length - c, length, device="cuda") for length, c in zip(lens, counts)])
        at = at + int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
        pos = [at] if case["axes"] == 1 else [at // 64, at // 64 + at % 64 // 8, at // 64 + at % 8]
        s["positions"] = torch.stack(pos).to(torch.int32)
        s["rot_offset"] = 512 if latent else 0
        half = case["rot"] // 2
        s["freqs"] = [1e6 ** (-i / half) for i in range(half)]
        s["sections"] = SECTIONS[(half, case["axes"])]
        s["key_weights"] = torch.rand((case["batch"], kv, s["width"]), generator=g, device="cuda")
        s["key_positions"] = torch.zeros((case["batch"], kv, s["width"]), dtype=torch.int32, device="cuda")

    @staticmethod
    def weights(s, case, g, lens, counts):
        heads, kv, t = case["heads"], case["kv_heads"], case["tokens"]
        s["k_pages"] = _pool(g, s["pages"], kv, case["page"], 128, case)
        s["kv_scale"] = 1.0 / 64.0 if case["dtype"] == "e4m3" else 1.0
        s["scale"] = 128 ** -0.5
        s["decay"] = 0.97
        s["q"] = torch.randn((case["batch"], t, heads, 128), generator=g, device="cuda", dtype=torch.bfloat16)
        # of the size of what one call adds
        s["key_weights"] = torch.rand((case["batch"], kv, s["width"]), generator=g, device="cuda") * (2.0 * heads // kv / s["max_len"])
        lse = []
        for b, n in enumerate(lens):  # what the decode call before this one gave
            k = _rows(s["k_pages"], s["table"][b, :-(-n // case["page"])], case)[:n].float() * s["kv_scale"]
            q = s["q"][b].float().view(t, kv, heads // kv, 128).permute(1, 0, 2, 3).reshape(kv, -1, 128)
            x = torch.matmul(q, k.permute(1, 2, 0)).view(kv, t, heads // kv, n) * s["scale"]
            far = torch.arange(n, device="cuda")[None, :] > (n - t + torch.arange(t, device="cuda"))[:, None]
            x = x.masked_fill(far[None, :, None, :], -math.inf)
            lse.append(torch.logsumexp(x, -1).permute(1, 0, 2).reshape(t, heads))
        s["lse"] = torch.stack(lse)

    @staticmethod
    def evict(s, case, g, lens, counts):
        kv = case["kv_heads"]
        s["k_pages"] = _pool(g, s["pages"], kv, case["page"], case["dim"], case)
        s["v_pages"] = None if case["dim"] == 576 else _pool(g, s["pages"], kv, case["page"], case["dim"], case)
        # accumulated softmax weights: a few keys hold most of it
        s["key_weights"] = torch.exp(2.0 * torch.randn((case["batch"], kv, s["width"]), generator=g, device="cuda") - 6.0)
        s["key_positions"] = torch.arange(s["width"], dtype=torch.int32, device="cuda").expand(case["batch"], kv, -1).contiguous()

    @staticmethod
    def cross(s, case, g, lens, counts):
        heads, kv, n = case["heads"], case["kv_heads"], sum(counts)
        s["k_pages"] = _pool(g, s["pages"], kv, case["page"], 128, case)
        s["v_pages"] = _pool(g, s["pages"], kv, case["page"], 128, case)
        s["scale"] = 128 ** -0.5
        s["q"] = torch.randn((n, heads, 128), generator=g, device="cuda", dtype=torch.bfloat16)
        s["cu"] = torch.tensor(_offsets(counts), dtype=torch.int32, device="cuda")
        s["max_tokens"] = max(counts)


def _rows(pool, pages, case):
    """The rows of the given pages in order, [..., keys, heads, dim]; codes as the numbers that they stand for."""
    x = pool[pages.long()]
    if pool.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn)
    if case["layout"] == "HND":
        x = x.transpose(-3, -2)
    return x.flatten(-4, -3)


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _shown(pool):
    """The pool as its values: what is held in 8 bits as numbers of 8 bits."""
    return pool.view(torch.float8_e4m3fn) if pool is not None and pool.dtype == torch.uint8 else pool


def _plain_append(s):
    case = s["case"]
    page, kv = case["page"], case["kv_heads"]
    n = s["q"].shape[0]
    token = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], token, right=True) - 1
    slot = (s["lens"][b] - (s["cu"][b + 1] - token)).long()
    pages = s["table"][b, slot // page].long()
    # angles in 64 bits: a far position times a frequency has no digits left in 32
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"), torch.tensor(s["sections"], device="cuda"))
    angle = s["positions"].double()[axis].t() * torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        x = x.float()
        at, half = s["rot_offset"], case["rot"] // 2
        r = x[..., at:at + case["rot"]]
        if case["paired"] == "halves":
            u, v = r[..., :half], r[..., half:]
            r = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
        else:
            u, v = r[..., 0::2], r[..., 1::2]
            r = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
        return torch.cat([x[..., :at], r, x[..., at + case["rot"]:]], -1)

    def put(pool, x):
        if case["dtype"] == "e4m3":
            x = (x / s["kv_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = x.to(torch.bfloat16)
        view = pool.transpose(1, 2) if case["layout"] == "HND" else pool
        view[pages, slot % page] = x

    q = turned(s["q"]).to(torch.bfloat16)
    put(s["k_pages"], turned(s["k"]))
    if s["v"] is not None:
        put(s["v_pages"], s["v"].float())
    head = torch.arange(kv, device="cuda")
    s["key_weights"][b[:, None], head, slot[:, None]] = 0.0
    s["key_positions"][b[:, None], head, slot[:, None]] = s["positions"][0][:, None].expand(n, kv)
    return q, _shown(s["k_pages"]), _shown(s["v_pages"]), s["key_weights"], s["key_positions"]


def _plain_weights(s):
    case = s["case"]
    t, kv, group = case["tokens"], case["kv_heads"], case["heads"] // case["kv_heads"]
    k = _rows(s["k_pages"], s["table"], case).float()  # [B][width][kv][128]
    q = s["q"].float().view(-1, t, kv, group, 128).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B][kv][t*group][128]
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (s["scale"] * s["kv_scale"])
    lse = s["lse"].view(-1, t, kv, group).permute(0, 2, 1, 3).flatten(2)
    w = torch.exp(x - lse[..., None])
    slot = torch.arange(s["width"], device="cuda")
    last = s["lens"][:, None] - t + torch.arange(t, device="cuda")
    seen = slot <= last.repeat_interleave(group, 1)[:, :, None]
    w = torch.where(seen[:, None], w, 0.0).sum(2)
    inside = slot < s["lens"][:, None, None]
    return torch.where(inside, s["decay"] * s["key_weights"] + w, 0.0)


def _plain_evict(s):
    case = s["case"]
    page = case["page"]
    lens, width = s["lens"][:, None, None], s["width"]
    n = lens.clamp(max=case["budget"])
    slot = torch.arange(width, device="cuda")
    inside = slot < lens
    pos = s["key_positions"]
    top = torch.where(inside, pos, -1).amax(-1, keepdim=True)
    guarded = (pos < case["sink"]) | (pos > top - case["recent"])
    rank = s["key_weights"].clamp(min=0.0).view(torch.int32).long() + (guarded.long() << 31)
    order = torch.sort(torch.where(inside, rank, -1), dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(inside.expand(pos.shape)).scatter(-1, order, (slot < n).expand(pos.shape))
    b, h, to = torch.nonzero(~kept & (slot < n), as_tuple=True)
    at = torch.nonzero(kept & (slot >= n), as_tuple=True)[2]  # as many for each sequence and head, in the same order
    to_page, at_page = s["table"][b, to // page].long(), s["table"][b, at // page].long()
    for pool in (s["k_pages"], s["v_pages"]):
        if pool is not None:
            view = pool if case["layout"] == "HND" else pool.transpose(1, 2)
            view[to_page, h, to % page] = view[at_page, h, at % page]
    weights, positions = s["key_weights"].clone(), pos.clone()
    weights[b, h, to] = weights[b, h, at]
    positions[b, h, to] = positions[b, h, at]
    mine = slot < n
    return (_shown(s["k_pages"]), _shown(s["v_pages"]), torch.where(mine, weights, 0.0), torch.where(mine, positions, 0),
            n.flatten())


def _plain_cross(s):
    case = s["case"]
    heads, kv = case["heads"], case["kv_heads"]
    group = heads // kv
    n = s["q"].shape[0]
    token = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], token, right=True) - 1
    i = (token - s["cu"][b]).long()
    q = torch.zeros((case["batch"], s["max_tokens"], heads, 128), device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(case["batch"], -1, kv, group, 128).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B][kv][group*T][128]
    k = _rows(s["k_pages"], s["table"], case).float().permute(0, 2, 3, 1)
    v = _rows(s["v_pages"], s["table"], case).float().transpose(1, 2)
    x = torch.matmul(q, k) * s["scale"]
    x.masked_fill_((torch.arange(s["width"], device="cuda") >= s["lens"][:, None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / total
    lse = (total.log() + top).view(case["batch"], heads, -1).transpose(1, 2)
    out = out.view(case["batch"], heads, -1, 128).transpose(1, 2)
    return out[b, i].to(torch.bfloat16), lse[b, i]


_PLAIN = dict(append=_plain_append, weights=_plain_weights, evict=_plain_evict, cross=_plain_cross)


# ------------------------------------------------------------------ the library's calls

def _handle(s):
    """What a program makes once and keeps: the cache's description, rotary tables, outputs, workspaces."""
    import split_kv_paged_splitkv_gb300 as skv
    case = s["case"]
    op, dim = case["op"], case.get("dim", 128)
    desc = skv.make_desc(
        case["batch"], case.get("tokens", 1), case.get("heads", case["kv_heads"]), case["kv_heads"], dim, 512 if dim == 576 else dim,
        case["page"], s["table"].shape[1], s["pages"], skv.SPLITKV_FP8_E4M3 if case.get("dtype") == "e4m3" else skv.SPLITKV_BF16,
        v_shares_k=int(dim == 576), kv_layout=skv.SPLITKV_LAYOUT_NHD if case["layout"] == "NHD" else skv.SPLITKV_LAYOUT_HND)
    h = dict(skv=skv, desc=desc)
    if op == "append":
        h["rope"] = skv.splitkv_rope_create(
            case["rot"], s["sections"], freqs=s["freqs"], rot_offset=s["rot_offset"],
            pairing=skv.SPLITKV_ROPE_HALVES if case["paired"] == "halves" else skv.SPLITKV_ROPE_NEIGHBOURS)
        h["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    elif op == "weights":
        h["weights"] = torch.zeros_like(s["key_weights"])
    elif op == "evict":
        size = skv.splitkv_evict_workspace_size(desc, case["budget"])
        h["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
        h["weights"], h["positions"] = torch.zeros_like(s["key_weights"]), torch.zeros_like(s["key_positions"])
        h["lens"] = torch.empty_like(s["lens"])
    elif op == "cross":
        n = s["q"].shape[0]
        size = skv.splitkv_cross_workspace_size(desc, n)
        h["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
        h["out"] = torch.empty_like(s["q"])
        h["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    s["handle"] = h
    return h


def _own_append(s):
    h = s.get("handle") or _handle(s)
    h["skv"].splitkv_append(h["desc"], h["rope"], s["positions"], s["q"], s["k"], s["v"], s["table"], s["lens"], h["q_out"],
                            s["k_pages"], s["v_pages"], cu_tokens=s["cu"], kv_scale=s["kv_scale"],
                            key_weights=s["key_weights"], key_positions=s["key_positions"])
    return h["q_out"], _shown(s["k_pages"]), _shown(s["v_pages"]), s["key_weights"], s["key_positions"]


def _own_weights(s):
    h = s.get("handle") or _handle(s)
    h["skv"].splitkv_key_weights(h["desc"], s["q"], s["k_pages"], s["table"], s["lens"], s["lse"], s["scale"], s["kv_scale"],
                                 s["decay"], s["key_weights"], h["weights"])
    return h["weights"]


def _own_evict(s):
    h = s.get("handle") or _handle(s)
    case = s["case"]
    h["skv"].splitkv_evict(h["desc"], case["budget"], case["sink"], case["recent"], s["k_pages"], s["v_pages"], s["table"],
                           s["lens"], s["key_weights"], s["key_positions"], h["weights"], h["positions"], h["lens"],
                           h["workspace"])
    return _shown(s["k_pages"]), _shown(s["v_pages"]), h["weights"], h["positions"], h["lens"]


def _own_cross(s):
    h = s.get("handle") or _handle(s)
    h["skv"].splitkv_cross_attend(h["desc"], s["cu"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scale"],
                                  h["out"], h["lse"], h["workspace"])
    return h["out"], h["lse"]


_OWN = dict(append=_own_append, weights=_own_weights, evict=_own_evict, cross=_own_cross)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    lens, counts, kv = _cache_lengths(case), _query_counts(case), case["kv_heads"]
    size = 1 if case.get("dtype") == "e4m3" else 2
    if case["op"] == "append":
        n, heads, dim = sum(counts), case["heads"], case["dim"]
        values = dim if dim == 576 else 2 * dim  # of a key and its value
        moved = n * (heads * dim * 4 + kv * values * (2 + size))
        return {"bytes": moved + n * (4 * case["axes"] + 8 * kv), "flops": 3 * n * (heads + kv) * case["rot"]}
    if case["op"] == "weights":
        t, rows = case["tokens"], case["heads"] // kv * case["tokens"]
        return {"bytes": sum(lens) * kv * (128 * size + 8) + case["batch"] * t * case["heads"] * (256 + 4),
                "flops": 2 * sum(lens) * kv * rows * 128}
    if case["op"] == "evict":
        row = case["dim"] * size * (1 if case["dim"] == 576 else 2)
        total = 0.0
        for length in lens:
            n = min(length, case["budget"])
            free = length - case["sink"] - case["recent"]
            # kept keys behind the first n, for weights that do not go by a key's place: each row read and written once
            m = (length - n) * max(0, n - case["sink"]) / free if length > n and free > 0 else 0
            total += kv * (8 * length + 8 * n + 2 * row * m)
        return {"bytes": total, "flops": 0}
    n = sum(counts)
    flops = 4 * 128 * case["heads"] * sum(c * length for c, length in zip(counts, lens))
    return {"bytes": n * case["heads"] * (512 + 4) + sum(lens) * kv * 512, "flops": flops}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _key_rows(s, pool, b, n):
    """Keys 0 .. n-1 of sequence b by their places: (page, offset)."""
    j = torch.arange(n, device="cuda")
    return s["table"][b].long()[j // s["case"]["page"]], j % s["case"]["page"]


def _pick(pool, page, off, case):
    """[keys][heads][dim] in 64 bits."""
    x = pool[page, :, off] if case["layout"] == "HND" else pool[page, off]
    return _shown(x).double()


def exact(case, seed):
    s = prepare(case, seed)
    return getattr(_Exact, case["op"])(s, case, _cache_lengths(case), _query_counts(case))


class _Exact:
    @staticmethod
    def append(s, case, lens, counts):
        half, at, kv = case["rot"] // 2, s["rot_offset"], case["kv_heads"]
        kp = _shown(s["k_pages"]).double()
        vp = None if s["v"] is None else _shown(s["v_pages"]).double()
        weights, positions = s["key_weights"].double(), s["key_positions"].clone()
        queries, begin = [], 0
        first = [sum(s["sections"][:a]) for a in range(case["axes"])] + [half]
        for b, c in enumerate(counts):
            rows = slice(begin, begin + c)
            turn = torch.zeros((c, half), dtype=torch.float64, device="cuda")
            for a in range(case["axes"]):
                f = torch.tensor(s["freqs"][first[a]:first[a + 1]], dtype=torch.float64, device="cuda")
                turn[:, first[a]:first[a + 1]] = torch.outer(s["positions"][a, rows].double(), f)
            unit = torch.polar(torch.ones_like(turn), turn)[:, None]

            def rotated(x):
                x = x.double().clone()
                r = x[..., at:at + 2 * half]
                if case["paired"] == "halves":
                    z = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * unit
                    x[..., at:at + half], x[..., at + half:at + 2 * half] = z.real, z.imag
                else:
                    z = torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * unit
                    x[..., at:at + 2 * half:2], x[..., at + 1:at + 2 * half:2] = z.real, z.imag
                return x

            queries.append(rotated(s["q"][rows]))
            page, off = (z[lens[b] - c:] for z in _key_rows(s, None, b, lens[b]))
            for pool, new in ((kp, rotated(s["k"][rows])), (vp, None if vp is None else s["v"][rows].double())):
                if pool is not None:
                    if case["dtype"] == "e4m3":
                        new = (new / s["kv_scale"]).clamp(-E4M3_MAX, E4M3_MAX)
                    if case["layout"] == "HND":
                        pool[page, :, off] = new
                    else:
                        pool[page, off] = new
            weights[b, :, lens[b] - c:lens[b]] = 0
            positions[b, :, lens[b] - c:lens[b]] = s["positions"][0, rows]
            begin += c
        return torch.cat(queries), kp, vp, weights, positions

    @staticmethod
    def weights(s, case, lens, counts):
        t, kv, group = case["tokens"], case["kv_heads"], case["heads"] // case["kv_heads"]
        w = torch.zeros_like(s["key_weights"], dtype=torch.float64)
        for b, n in enumerate(lens):
            k = _pick(s["k_pages"], *_key_rows(s, None, b, n), case) * s["kv_scale"]
            add = torch.zeros((kv, n), dtype=torch.float64, device="cuda")
            for i in range(t):
                q, seen = s["q"][b, i].double().view(kv, group, 128), n - t + i + 1
                x = torch.einsum("hgd,jhd->hgj", q, k[:seen]) * s["scale"]
                add[:, :seen] += (x - s["lse"][b, i].double().view(kv, group, 1)).exp().sum(1)
            w[b, :, :n] = s["decay"] * s["key_weights"][b, :, :n].double() + add
        return w

    @staticmethod
    def evict(s, case, lens, counts):
        kp, vp = s["k_pages"].clone(), None if s["v_pages"] is None else s["v_pages"].clone()
        weights, positions = torch.zeros_like(s["key_weights"]), torch.zeros_like(s["key_positions"])
        final = []
        for b, length in enumerate(lens):
            n = min(length, case["budget"])
            final.append(n)
            page, off = _key_rows(s, None, b, length)
            for h in range(case["kv_heads"]):
                w, p = s["key_weights"][b, h, :length], s["key_positions"][b, h, :length]
                safe = (p < case["sink"]) | (p > p.max() - case["recent"])
                # two stable sorts: by weight, then the guarded keys first
                by = torch.argsort(w, descending=True, stable=True)
                by = by[torch.argsort((~safe[by]).long(), stable=True)]
                best = torch.sort(by[:n]).values
                late = best[best >= n]
                place = torch.ones(n, dtype=torch.bool, device="cuda")
                place[best[best < n]] = False
                holes = torch.arange(n, device="cuda")[place]
                source = torch.arange(n, device="cuda")
                source[holes] = late
                weights[b, h, :n], positions[b, h, :n] = w[source], p[source]
                for new, old in ((kp, s["k_pages"]), (vp, s["v_pages"])):
                    if new is not None:
                        if case["layout"] == "HND":
                            new[page[holes], h, off[holes]] = old[page[late], h, off[late]]
                        else:
                            new[page[holes], off[holes], h] = old[page[late], off[late], h]
        kp, vp = _shown(kp).double(), None if vp is None else _shown(vp).double()
        return kp, vp, weights.double(), positions, torch.tensor(final, dtype=torch.int32, device="cuda")

    @staticmethod
    def cross(s, case, lens, counts):
        kv, group = case["kv_heads"], case["heads"] // case["kv_heads"]
        out, lse, begin = [], [], 0
        for b, (c, n) in enumerate(zip(counts, lens)):
            where = _key_rows(s, None, b, n)
            k, v = _pick(s["k_pages"], *where, case), _pick(s["v_pages"], *where, case)
            heads, norms = [], []
            for h in range(kv * group):
                x = s["q"][begin:begin + c, h].double() @ k[:, h // group].T * s["scale"]
                z = torch.logsumexp(x, -1)
                heads.append(torch.softmax(x, -1) @ v[:, h // group])
                norms.append(z)
            out.append(torch.stack(heads, 1))
            lse.append(torch.stack(norms, 1))
            begin += c
        return torch.cat(out), torch.cat(lse)
