"""Plain 64-bit implementations of the cache operators (numpy loops over sequences) and the
inputs that their tests share."""
import math

import numpy as np
import torch

import split_kv_paged_splitkv_gb300 as skv

EPS16 = 2.0 ** -8  # half a step of bf16, relative


class Cache:
    """Pools, block table and lengths of a paged cache with random contents, on ``device``."""

    def __init__(self, lens, kv_heads=2, page=16, dtype="bf16", layout="HND", dim=128, v_dim=None, shares=False,
                 seed=0, device="cpu", cap_pages=None, heads=None, tokens=1, std=1.0):
        rng = np.random.default_rng(seed)
        self.lens_host = [int(x) for x in lens]
        self.B, self.Hkv, self.P, self.dim = len(lens), kv_heads, page, dim
        self.v_dim = dim if v_dim is None else v_dim
        self.layout, self.dtype, self.shares = layout, dtype, shares
        counts = [-(-n // page) for n in self.lens_host]
        self.width = cap_pages or max(1, max(counts))
        self.N = sum(max(c, 1) for c in counts) + 3
        perm = rng.permutation(self.N)
        table = np.full((self.B, self.width), perm[-1], np.int32)
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = perm[at:at + c]
            at += c
        self.table = torch.from_numpy(table).to(device)
        self.lens = torch.tensor(self.lens_host, dtype=torch.int32, device=device)
        self.cap = self.width * page
        g = torch.Generator().manual_seed(seed)

        def pool(d):
            shape = (self.N, kv_heads, page, d) if layout == "HND" else (self.N, page, kv_heads, d)
            x = torch.randn(shape, generator=g) * std
            if dtype == "e4m3":
                return (x * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).to(device)
            return x.to(torch.bfloat16).to(device)

        self.k = pool(dim)
        self.v = None if shares else pool(self.v_dim)
        self.heads = heads or 4 * kv_heads
        self.desc = skv.make_desc(self.B, tokens, self.heads, kv_heads, dim, self.v_dim, page, self.width, self.N,
                                  skv.SPLITKV_FP8_E4M3 if dtype == "e4m3" else skv.SPLITKV_BF16, int(shares),
                                  skv.SPLITKV_COMBINE_SEPARATE,
                                  skv.SPLITKV_LAYOUT_NHD if layout == "NHD" else skv.SPLITKV_LAYOUT_HND)

    def values(self, pool):
        """The pool as float64 numpy, [N][Hkv][P][dim]."""
        x = pool.cpu()
        x = (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).double()
        return (x if self.layout == "HND" else x.transpose(1, 2)).numpy().copy()

    def rows(self, values, b, n):
        """Keys 0 .. n-1 of sequence b: [n][Hkv][dim]."""
        t = self.table[b].cpu().numpy()
        return np.stack([values[t[j // self.P], :, j % self.P] for j in range(n)]) if n else \
            np.zeros((0,) + values.shape[1:2] + values.shape[3:])


def rotated(x, positions, freqs, sections, offset, pairing):
    """x [n][heads][dim] float64, positions [axes][n]."""
    half = len(freqs)
    axis = np.repeat(np.arange(len(sections)), sections)
    # the exact product of an integer position and a frequency, reduced modulo a turn
    ang = np.array([[math.fmod(float(positions[axis[i]][n]) * freqs[i], 2 * math.pi) for i in range(half)]
                    for n in range(x.shape[0])]).reshape(x.shape[0], half)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = x.copy()
    iu = offset + (np.arange(half) if pairing == skv.SPLITKV_ROPE_HALVES else 2 * np.arange(half))
    iv = iu + (half if pairing == skv.SPLITKV_ROPE_HALVES else 1)
    u, v = x[..., iu], x[..., iv]
    y[..., iu], y[..., iv] = u * c - v * s, u * s + v * c
    return y


def key_weights(q, keys, lse, scale, T):
    """q [T][Hq][128], keys [L][Hkv][128], lse [T][Hq] -> [Hkv][L] (all float64)."""
    L, Hkv = keys.shape[:2]
    G = q.shape[1] // Hkv
    w = np.zeros((Hkv, L))
    for t in range(T):
        seen = L - T + t + 1
        for h in range(q.shape[1]):
            if seen > 0 and lse[t, h] != -np.inf:
                w[h // G, :seen] += np.exp(keys[:seen, h // G] @ q[t, h] * scale - lse[t, h])
    return w


def lse_of(q, keys, scale, T):
    L, Hkv = keys.shape[:2]
    G = q.shape[1] // Hkv
    out = np.full(q.shape[:2], -np.inf)
    for t in range(T):
        seen = L - T + t + 1
        for h in range(q.shape[1]):
            if seen > 0:
                x = keys[:seen, h // G] @ q[t, h] * scale
                out[t, h] = x.max() + np.log(np.exp(x - x.max()).sum())
    return out


def evict_moves(weights, positions, L, budget, sink, recent):
    """(n, [(destination, source)]) of one head; weights and positions are numpy arrays of L entries."""
    n = min(L, budget)
    if n == L:
        return n, []
    w = np.where(weights[:L] > 0, weights[:L], 0).astype(np.float64)
    safe = np.zeros(L, bool)
    if positions is not None:
        p = positions[:L].astype(np.int64)
        safe = (p < sink) | (p > p.max() - recent)
    order = sorted(range(L), key=lambda j: (not safe[j], -w[j], j))
    kept = set(order[:n])
    holes = [j for j in range(n) if j not in kept]
    return n, list(zip(holes, sorted(j for j in kept if j >= n)))
