"""Measured cases of speculative decoding over a paged cache: append with norms and rotary positions,
attention of a tree of drafted tokens, and the commit of the tokens that were accepted.

Every case is a call that a serving program makes between its draft model and the next step. With
``own`` false the operators run in their plain form (elementary torch operations in 32 bits), with ``own``
true through the library's entry points. Caches are paged: pools of pages, one block table row for each
sequence.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
#: How the pairs of a rotated head are dealt to three position axes (time, height, width).
SECTIONS = {(64, 1): (64,), (64, 3): (24, 20, 20), (32, 1): (32,)}


def listed():
    return [
        # one new token of one request at the default decode workload's context: latency alone
        dict(name="norm_token_b1", op="norm", batch=1, tlo=1, thi=1, lo=5900, hi=5900, heads=16, kv_heads=2, dim=128, rot=128,
             axes=1, paired="halves", per_head=False, page=16, dtype="bf16", layout="HND", shape_seed=1),
        # the drafted trees of a batch entering an e4m3 cache before they are verified
        dict(name="norm_drafts_b32_e4m3", op="norm", batch=32, tlo=5, thi=64, lo=500, hi=4000, heads=32, kv_heads=8, dim=128,
             rot=128, axes=1, paired="halves", per_head=False, page=16, dtype="e4m3", layout="NHD", shape_seed=2),
        # the prompts of eight requests, of unequal lengths, image and video positions, a weight for each head
        dict(name="norm_prompts", op="norm", batch=8, tlo=700, thi=9000, lo=1, hi=1, heads=32, kv_heads=4, dim=128, rot=128,
             axes=3, paired="halves", per_head=True, page=16, dtype="bf16", layout="HND", shape_seed=3),
        # prompts entering a latent cache in 8 bits: its 512 latent columns are normalised, its last 64 rotated
        dict(name="norm_latent_prompts_e4m3", op="norm", batch=2, tlo=500, thi=2000, lo=1, hi=1, heads=128, kv_heads=1, dim=576,
             rot=64, axes=1, paired="neighbours", per_head=False, page=64, dtype="e4m3", layout="HND", shape_seed=4),
        # a small tree of one request at the default decode workload's context
        dict(name="tree_b1", op="tree", batch=1, tlo=8, thi=8, lo=5900, hi=5900, heads=16, kv_heads=2, dim=128, page=16,
             dtype="bf16", layout="HND", shape_seed=5),
        # trees of a batch of long contexts over an e4m3 cache
        dict(name="tree_b8_32k_e4m3", op="tree", batch=8, tlo=16, thi=61, lo=28672, hi=32768, heads=32, kv_heads=4, dim=128,
             page=16, dtype="e4m3", layout="HND", shape_seed=6),
        # a batch of very unequal contexts and trees
        dict(name="tree_mixed_b32", op="tree", batch=32, tlo=4, thi=24, lo=256, hi=131072, heads=32, kv_heads=8, dim=128, page=16,
             dtype="bf16", layout="HND", shape_seed=7),
        # many young requests: trees nearly as long as their contexts
        dict(name="tree_short_b64", op="tree", batch=64, tlo=20, thi=64, lo=1, hi=300, heads=32, kv_heads=8, dim=128, page=32,
             dtype="bf16", layout="NHD", shape_seed=8),
        # a tree of one request over 64k latent rows
        dict(name="tree_latent_64k", op="tree", batch=1, tlo=12, thi=12, lo=65536, hi=65536, heads=128, kv_heads=1, dim=576,
             page=64, dtype="bf16", layout="HND", shape_seed=9),
        # the accepted path of one request's tree: latency alone
        dict(name="commit_b1", op="commit", batch=1, tlo=8, thi=8, lo=5900, hi=5900, kv_heads=2, dim=128, page=16, dtype="bf16",
             layout="HND", shape_seed=10),
        # the accepted paths of a batch, with the state that eviction keeps
        dict(name="commit_b64_e4m3", op="commit", batch=64, tlo=31, thi=64, lo=200, hi=1500, kv_heads=8, dim=128, page=16,
             dtype="e4m3", layout="NHD", shape_seed=11),
        # the accepted paths of a large batch over a latent cache
        dict(name="commit_latent_b256", op="commit", batch=256, tlo=9, thi=16, lo=200, hi=1500, kv_heads=1, dim=576, page=64,
             dtype="bf16", layout="HND", shape_seed=12),
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "tree", "commit"])
    latent = rng.random() < 0.25
    kv = 1 if latent else rng.choice([1, 2, 4, 8])
    case = dict(op=op, batch=between(1, 64), kv_heads=kv, heads=128 if latent else kv * rng.choice([1, 2, 4, 5, 8]),
                dim=576 if latent else 128, page=rng.choice([16, 32, 64]), dtype=rng.choice(["bf16", "e4m3"]),
                layout="HND" if latent else rng.choice(["HND", "NHD"]), shape_seed=rng.randrange(1 << 30))
    if op == "norm":
        hi = between(1, max(1, (2000 if latent else 16000) // case["batch"]))
        case.update(tlo=max(1, hi // 9), thi=hi, lo=1, hi=between(1, 4000), rot=64 if latent else rng.choice([64, 128]),
                    axes=1, paired="neighbours" if latent else rng.choice(["halves", "neighbours"]),
                    per_head=not latent and rng.random() < 0.5)
        if case["rot"] == 128:
            case["axes"] = rng.choice([1, 3])
    elif op == "tree":
        if latent:
            case["batch"] = between(1, 8)
        thi = between(1, 16 if latent else 128)
        hi = between(1, max(40, (40000 if latent else 1000000 // kv) // case["batch"]))
        if not latent:
            # (no more work than the listed cases have)
            hi = max(1, min(hi, 400000000 // (case["batch"] * case["heads"] * thi)))
        case.update(tlo=thi if latent else max(1, thi // 5), thi=thi, lo=max(1, hi // 20), hi=hi)
    else:
        thi = between(1, 128)
        case.update(tlo=max(1, thi // 3), thi=thi, lo=1, hi=between(1, 1500))
    return case


# ------------------------------------------------------------------ shapes

def _between(case, lo, hi, salt):
    """Log-uniform numbers, the case's own (they do not depend on the inputs' seed)."""
    rng = random.Random(case["shape_seed"] * 7 + salt)
    return [min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))) for _ in range(case["batch"])]


def _counts(case):
    """New tokens of every sequence."""
    return _between(case, case["tlo"], case["thi"], 2)


def _lengths(case):
    """Keys of every sequence, the new tokens among them."""
    return [n - 1 + c if case["lo"] == 1 else max(n, c) for n, c in zip(_between(case, case["lo"], case["hi"], 1), _counts(case))]


def _parents(case):
    """For every sequence the parent of each drafted token (-1: the first)."""
    rng = random.Random(case["shape_seed"] * 7 + 3)
    return [[-1] + [rng.randrange(max(0, i - 9), i) for i in range(1, c)] for c in _counts(case)]


def _ancestors(parents):
    """For every drafted token the bits of the tokens that it sees: itself and those on the way to the first."""
    seen = []
    for i, p in enumerate(parents):
        seen.append(1 << i | (seen[p] if p >= 0 else 0))
    return seen


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


def _offsets(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return cu


# ------------------------------------------------------------------ inputs

def _pool(g, pages, heads, page, dim, case):
    shape = (pages, heads, page, dim) if case["layout"] == "HND" else (pages, page, heads, dim)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if case["dtype"] == "e4m3":  # codes whose values times kv_scale are the cache's
        return (x * 64.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, counts = _lengths(case), _counts(case)
    table, pages = _tables(lens, case["page"], seed)
    latent, kv = case["dim"] == 576, case["kv_heads"]
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), pages=pages,
             width=table.shape[1] * case["page"], cu=torch.tensor(_offsets(counts), dtype=torch.int32, device="cuda"),
             k_pages=_pool(g, pages, kv, case["page"], case["dim"], case),
             v_pages=None if latent else _pool(g, pages, kv, case["page"], case["dim"], case),
             kv_scale=1.0 / 64.0 if case["dtype"] == "e4m3" else 1.0)
    getattr(_Inputs, case["op"])(s, case, g, lens, counts)
    return s


class _Inputs:
    @staticmethod
    def norm(s, case, g, lens, counts):
        n, heads, kv, dim = sum(counts), case["heads"], case["kv_heads"], case["dim"]
        latent = dim == 576
        # the projections' output holds queries, keys and values of a token side by side
        wide = (heads + kv) * dim if latent else (heads + 2 * kv) * dim
        rows = torch.randn((n, wide), generator=g, device="cuda", dtype=torch.bfloat16)
        # (a projection's rows are of very different lengths)
        rows *= torch.exp(1.5 * torch.randn((n, 1), generator=g, device="cuda")).to(torch.bfloat16)
        s["q"] = rows[:, :heads * dim].view(n, heads, dim)
        s["k"] = rows[:, heads * dim:(heads + kv) * dim].view(n, kv, dim)
        s["v"] = None if latent else rows[:, (heads + kv) * dim:].view(n, kv, dim)

        def weight(count, columns):
            shape = (count, columns) if case["per_head"] else (columns,)
            return 1.0 + 0.2 * torch.randn(shape, generator=g, device="cuda")

        # a latent row's first 512 columns are normalised, its queries are not
        s["q_weight"] = None if latent else weight(heads, dim)
        s["k_weight"] = weight(kv, 512 if latent else dim)
        # a token's index in its sequence, and for three axes its place on a grid of 8 by 8 patches in a frame
        at = torch.cat([torch.arange(length - c, length, device="cuda") for length, c in zip(lens, counts)])
        at = at + int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
        pos = [at] if case["axes"] == 1 else [at // 64, at // 64 + at % 64 // 8, at // 64 + at % 8]
        s["positions"] = torch.stack(pos).to(torch.int32)
        s["rot_offset"] = 512 if latent else 0
        half = case["rot"] // 2
        s["freqs"] = [1e6 ** (-i / half) for i in range(half)]
        s["sections"] = SECTIONS[(half, case["axes"])]

    @staticmethod
    def tree(s, case, g, lens, counts):
        words = -(-max(counts) // 32)
        rows = [[(bits >> 32 * w & 0xffffffff) - (bits >> 32 * w + 31 & 1) * (1 << 32) for w in range(words)]
                for parents in _parents(case) for bits in _ancestors(parents)]
        s["mask"] = torch.tensor(rows, dtype=torch.int32, device="cuda")  # [tokens][words], bit i: the tree's token i is seen
        s["q"] = torch.randn((sum(counts), case["heads"], case["dim"]), generator=g, device="cuda", dtype=torch.bfloat16)
        s["scale"] = case["dim"] ** -0.5
        s["counts"], s["host_lens"] = counts, lens  # (the plain form's loop; the library reads them on the GPU)

    @staticmethod
    def commit(s, case, g, lens, counts):
        # what the verification gave: a way down from the tree's first token, ended anywhere
        rng = random.Random(int(torch.randint(0, 1 << 30, (1,), generator=g, device="cuda")))
        paths = []
        for parents in _parents(case):
            path = [0]
            while True:
                children = [i for i, p in enumerate(parents) if p == path[-1]]
                if not children or rng.random() < 0.15:
                    break
                path.append(rng.choice(children))
            paths.append(path)
        longest = case["thi"]
        s["path"] = torch.tensor([p + [0] * (longest - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        s["path_lens"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        s["key_weights"] = torch.rand((case["batch"], case["kv_heads"], s["width"]), generator=g, device="cuda")
        s["key_positions"] = torch.arange(s["width"], dtype=torch.int32, device="cuda").expand(
            case["batch"], case["kv_heads"], -1).contiguous()


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _shown(pool):
    """The pool as its values: what is held in 8 bits as numbers of 8 bits."""
    return pool.view(torch.float8_e4m3fn) if pool is not None and pool.dtype == torch.uint8 else pool


def _rows(pool, pages, case):
    """The rows of the given pages in order, [keys][heads][dim]; codes as the numbers that they stand for."""
    x = _shown(pool[pages.long()])
    if case["layout"] == "HND":
        x = x.transpose(1, 2)
    return x.flatten(0, 1)


def _plain_norm(s):
    case = s["case"]
    page, n = case["page"], s["q"].shape[0]
    token = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], token, right=True) - 1
    slot = (s["lens"][b] - (s["cu"][b + 1] - token)).long()
    pages = s["table"][b, slot // page].long()
    # angles in 64 bits: a far position times a frequency has no digits left in 32
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"), torch.tensor(s["sections"], device="cuda"))
    angle = s["positions"].double()[axis].t() * torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def normed(x, weight):
        x = x.float()
        if weight is None:
            return x
        c = weight.shape[-1]
        y = x[..., :c] * torch.rsqrt((x[..., :c] * x[..., :c]).mean(-1, keepdim=True) + EPS) * weight
        return torch.cat([y, x[..., c:]], -1)

    def turned(x):
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

    q = turned(normed(s["q"], s["q_weight"])).to(torch.bfloat16)
    put(s["k_pages"], turned(normed(s["k"], s["k_weight"])))
    if s["v"] is not None:
        put(s["v_pages"], s["v"].float())
    return q, _shown(s["k_pages"]), _shown(s["v_pages"])


def _plain_tree(s):
    case = s["case"]
    heads, kv = case["heads"], case["kv_heads"]
    group, columns = heads // kv, 512 if case["dim"] == 576 else case["dim"]
    out, lse, begin = [], [], 0
    for b, (c, n) in enumerate(zip(s["counts"], s["host_lens"])):
        pages = s["table"][b, :-(-n // case["page"])]
        k = _rows(s["k_pages"], pages, case)[:n].float() * s["kv_scale"]
        v = k[..., :columns] if s["v_pages"] is None else _rows(s["v_pages"], pages, case)[:n].float() * s["kv_scale"]
        q = s["q"][begin:begin + c].float().view(c, kv, group, -1).permute(1, 0, 2, 3).reshape(kv, c * group, -1)
        x = torch.matmul(q, k.permute(1, 2, 0)) * s["scale"]  # [kv][c * group][n]
        drafted = torch.arange(c, device="cuda")
        sees = (s["mask"][begin:begin + c][:, drafted // 32] >> (drafted % 32) & 1).bool()
        sees = torch.cat([torch.ones((c, n - c), dtype=torch.bool, device="cuda"), sees], 1).repeat_interleave(group, 0)
        x = torch.where(sees, x, -math.inf)
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - top)
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x, v.permute(1, 0, 2)) / total
        out.append(o.view(kv, c, group, columns).permute(1, 0, 2, 3).reshape(c, heads, columns))
        lse.append((total.log() + top).view(kv, c, group).permute(1, 0, 2).reshape(c, heads))
        begin += c
    return torch.cat(out).to(torch.bfloat16), torch.cat(lse)


def _plain_commit(s):
    case = s["case"]
    page = case["page"]
    i = torch.arange(s["path"].shape[1], device="cuda")
    first = s["lens"] - (s["cu"][1:] - s["cu"][:-1])
    b, i = torch.nonzero(i < s["path_lens"][:, None], as_tuple=True)
    to = (first[b] + i).long()
    at = (first[b] + s["path"][b, i]).long()
    to_page, at_page = s["table"][b, to // page].long(), s["table"][b, at // page].long()
    for pool in (s["k_pages"], s["v_pages"]):
        if pool is not None:
            view = pool.transpose(1, 2) if case["layout"] == "HND" else pool
            view[to_page, to % page] = view[at_page, at % page]
    for state in (s["key_weights"], s["key_positions"]):
        state[b, :, to] = state[b, :, at]
    return _shown(s["k_pages"]), _shown(s["v_pages"]), s["key_weights"], s["key_positions"], first + s["path_lens"]


_PLAIN = dict(norm=_plain_norm, tree=_plain_tree, commit=_plain_commit)


# ------------------------------------------------------------------ the library's calls

def _handle(s):
    """What a program makes once and keeps: the cache's description, rotary tables, outputs, workspaces."""
    import split_kv_paged_splitkv_gb300 as skv
    case = s["case"]
    op, dim = case["op"], case["dim"]
    latent = dim == 576
    # (a latent cache's trees have one size, which the description names)
    tokens = case["thi"] if op == "tree" and latent else 1
    desc = skv.make_desc(
        case["batch"], tokens, case.get("heads", case["kv_heads"]), case["kv_heads"], dim, 512 if latent else dim, case["page"],
        s["table"].shape[1], s["pages"], skv.SPLITKV_FP8_E4M3 if case["dtype"] == "e4m3" else skv.SPLITKV_BF16,
        v_shares_k=int(latent), kv_layout=skv.SPLITKV_LAYOUT_NHD if case["layout"] == "NHD" else skv.SPLITKV_LAYOUT_HND)
    h = dict(skv=skv, desc=desc)
    if op == "norm":
        h["rope"] = skv.splitkv_rope_create(
            case["rot"], s["sections"], freqs=s["freqs"], rot_offset=s["rot_offset"],
            pairing=skv.SPLITKV_ROPE_HALVES if case["paired"] == "halves" else skv.SPLITKV_ROPE_NEIGHBOURS)
        h["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    elif op == "tree":
        n = s["q"].shape[0]
        size = skv.splitkv_tree_workspace_size(desc, n)
        h["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
        h["out"] = torch.empty((n, case["heads"], 512 if latent else dim), dtype=torch.bfloat16, device="cuda")
        h["lse"] = torch.empty((n, case["heads"]), dtype=torch.float32, device="cuda")
    else:
        h["lens"] = torch.empty_like(s["lens"])
    s["handle"] = h
    return h


def _own_norm(s):
    h = s.get("handle") or _handle(s)
    h["skv"].splitkv_append_norm(h["desc"], h["rope"], s["positions"], s["q"], s["k"], s["v"], s["table"], s["lens"], h["q_out"],
                                 s["k_pages"], s["v_pages"], norm_q=s["q_weight"] is not None, q_weight=s["q_weight"],
                                 k_weight=s["k_weight"], eps=EPS, cu_tokens=s["cu"], kv_scale=s["kv_scale"])
    return h["q_out"], _shown(s["k_pages"]), _shown(s["v_pages"])


def _own_tree(s):
    h = s.get("handle") or _handle(s)
    h["skv"].splitkv_tree_attend(h["desc"], None if s["v_pages"] is None else s["cu"], s["mask"], s["q"], s["k_pages"],
                                 s["v_pages"], s["table"], s["lens"], s["scale"], h["out"], h["lse"], h["workspace"],
                                 kv_scale=s["kv_scale"])
    return h["out"], h["lse"]


def _own_commit(s):
    h = s.get("handle") or _handle(s)
    h["skv"].splitkv_tree_commit(h["desc"], s["path"], s["path_lens"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                 h["lens"], cu_tokens=s["cu"], key_weights=s["key_weights"],
                                 key_positions=s["key_positions"])
    return _shown(s["k_pages"]), _shown(s["v_pages"]), s["key_weights"], s["key_positions"], h["lens"]


_OWN = dict(norm=_own_norm, tree=_own_tree, commit=_own_commit)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    lens, counts, kv, dim = _lengths(case), _counts(case), case["kv_heads"], case["dim"]
    size = 1 if case["dtype"] == "e4m3" else 2
    values = dim if dim == 576 else 2 * dim  # of a key and its value
    if case["op"] == "norm":
        n, heads = sum(counts), case["heads"]
        moved = n * (heads * dim * 4 + kv * values * (2 + size))
        normed = kv * 512 if dim == 576 else (heads + kv) * dim
        return {"bytes": moved + n * 4 * case["axes"], "flops": n * (3 * (heads + kv) * case["rot"] + 4 * normed)}
    if case["op"] == "tree":
        heads, columns = case["heads"], 512 if dim == 576 else dim
        words = -(-max(counts) // 32)
        seen = sum(c * (n - c) + sum(bin(bits).count("1") for bits in _ancestors(parents))
                   for c, n, parents in zip(counts, lens, _parents(case)))
        return {"bytes": sum(counts) * (heads * (2 * dim + 2 * columns + 4) + 4 * words) + sum(lens) * kv * values * size,
                "flops": 2 * (dim + columns) * heads * seen}
    # a path's tokens, of which most moves, each row read and written once, and its state
    path = [0.0] * len(counts)
    for b, parents in enumerate(_parents(case)):
        depth = []
        for p in parents:
            depth.append(1 + (depth[p] if p >= 0 else 0))
        path[b] = sum(depth) / len(depth)
    return {"bytes": sum(path) * kv * 2 * (values * size + 8), "flops": 0}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _places(s, b, n):
    """Keys 0 .. n-1 of sequence b by their places: (page, offset)."""
    j = torch.arange(n, device="cuda")
    return s["table"][b].long()[j // s["case"]["page"]], j % s["case"]["page"]


def _pick(pool, page, off, case):
    """[keys][heads][dim] in 64 bits."""
    x = pool[page, :, off] if case["layout"] == "HND" else pool[page, off]
    return _shown(x).double()


def exact(case, seed):
    s = prepare(case, seed)
    return getattr(_Exact, case["op"])(s, case, _lengths(case), _counts(case))


class _Exact:
    @staticmethod
    def norm(s, case, lens, counts):
        half, at = case["rot"] // 2, s["rot_offset"]
        kp = _shown(s["k_pages"]).double()
        vp = None if s["v"] is None else _shown(s["v_pages"]).double()
        queries, begin = [], 0
        first = [sum(s["sections"][:a]) for a in range(case["axes"])] + [half]
        for b, c in enumerate(counts):
            rows = slice(begin, begin + c)
            turn = torch.zeros((c, half), dtype=torch.float64, device="cuda")
            for a in range(case["axes"]):
                f = torch.tensor(s["freqs"][first[a]:first[a + 1]], dtype=torch.float64, device="cuda")
                turn[:, first[a]:first[a + 1]] = torch.outer(s["positions"][a, rows].double(), f)
            unit = torch.polar(torch.ones_like(turn), turn)[:, None]

            def finished(x, weight):
                x = x.double().clone()
                if weight is not None:
                    size = weight.shape[-1]
                    root = (x[..., :size].pow(2).sum(-1, keepdim=True) / size + EPS).sqrt()
                    x[..., :size] = x[..., :size] / root * weight.double()
                r = x[..., at:at + 2 * half].clone()
                if case["paired"] == "halves":
                    z = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * unit
                    x[..., at:at + half], x[..., at + half:at + 2 * half] = z.real, z.imag
                else:
                    z = torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * unit
                    x[..., at:at + 2 * half:2], x[..., at + 1:at + 2 * half:2] = z.real, z.imag
                return x

            queries.append(finished(s["q"][rows], s["q_weight"]))
            page, off = (z[lens[b] - c:] for z in _places(s, b, lens[b]))
            for pool, new in ((kp, finished(s["k"][rows], s["k_weight"])), (vp, None if vp is None else s["v"][rows].double())):
                if pool is not None:
                    if case["dtype"] == "e4m3":
                        new = (new / s["kv_scale"]).clamp(-E4M3_MAX, E4M3_MAX)
                    if case["layout"] == "HND":
                        pool[page, :, off] = new
                    else:
                        pool[page, off] = new
            begin += c
        return torch.cat(queries), kp, vp

    @staticmethod
    def tree(s, case, lens, counts):
        group, columns = case["heads"] // case["kv_heads"], 512 if case["dim"] == 576 else case["dim"]
        out, lse, begin = [], [], 0
        for b, parents in enumerate(_parents(case)):
            c, n = counts[b], lens[b]
            where = _places(s, b, n)
            k = _pick(s["k_pages"], *where, case) * s["kv_scale"]
            v = k[..., :columns] if s["v_pages"] is None else _pick(s["v_pages"], *where, case) * s["kv_scale"]
            hidden = torch.ones((c, c), dtype=torch.bool)
            for i in range(c):
                j = i
                while j >= 0:
                    hidden[i, j] = False
                    j = parents[j]
            hidden = hidden.cuda()
            heads, norms = [], []
            for h in range(case["heads"]):
                x = s["q"][begin:begin + c, h].double() @ k[:, h // group].T * s["scale"]
                x[:, n - c:][hidden] = -math.inf
                heads.append(torch.softmax(x, -1) @ v[:, h // group])
                norms.append(torch.logsumexp(x, -1))
            out.append(torch.stack(heads, 1))
            lse.append(torch.stack(norms, 1))
            begin += c
        return torch.cat(out), torch.cat(lse)

    @staticmethod
    def commit(s, case, lens, counts):
        kp, vp = s["k_pages"].clone(), None if s["v_pages"] is None else s["v_pages"].clone()
        weights, positions = s["key_weights"].clone(), s["key_positions"].clone()
        final = []
        for b, (n, c) in enumerate(zip(lens, counts)):
            path = s["path"][b, :int(s["path_lens"][b])].tolist()
            final.append(n - c + len(path))
            page, off = _places(s, b, n)
            source = torch.tensor([n - c + p for p in path], device="cuda")
            new = slice(n - c, n - c + len(path))
            for after, before in ((kp, s["k_pages"]), (vp, s["v_pages"])):
                if after is not None:
                    if case["layout"] == "HND":
                        after[page[new], :, off[new]] = before[page[source], :, off[source]]
                    else:
                        after[page[new], off[new]] = before[page[source], off[source]]
            weights[b, :, new], positions[b, :, new] = s["key_weights"][b][:, source], s["key_positions"][b][:, source]
        kp, vp = _shown(kp).double(), None if vp is None else _shown(vp).double()
        return kp, vp, weights.double(), positions, torch.tensor(final, dtype=torch.int32, device="cuda")
