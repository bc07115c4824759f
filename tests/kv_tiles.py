"""Attention in which every tile of 32 tokens shows by itself.

Keys are such that the softmax is nearly even, and of a tile's values one element
of each head is not zero, that of the tile's number modulo the head size.  An
output element is then a sum of a few tiles' weights, all positive: leaving one
tile out, or taking it twice, changes it by a good part of itself, whereas what
the arithmetic may do to it is a small part of itself too."""

import numpy as np

from tests import kv_ref as R
from tests.test_gpu_kv_attention import Setup

TILE = 32


class Tiled(Setup):
    def __init__(self, K, lens, new, qh, kh, dim, page, quant, window=0, sinks=0, room=0, seed=0):
        """room: tokens that the table has room for (0: those of the longest request)."""
        width = -(-room // page) if room else None
        super().__init__(K, lens, new, qh, kh, dim, page, quant, seed=seed, spread=0.05, width=width)
        self.window, self.sinks = window, sinks
        rng = np.random.default_rng(seed + 1)
        zero, one = (7, 15) if quant == "nf4" else (0, 7)  # the codes of 0 and of 1
        codes, scales = np.full_like(self.codes[1], 17 * zero), self.scales[1]
        for i, n in enumerate(self.lens):
            t = np.arange(n)
            page_of, at = self.table[i, t // page], t % page
            for h in range(kh):
                e = self.element(t // TILE, h)
                codes[page_of, h, at, e // 2] = np.where(e % 2, 16 * zero + one, 16 * one + zero)
        self.codes[1] = codes
        new_scales = (1 + rng.integers(0, 8, scales.shape) / 8).astype(np.float32)  # bf16 numbers
        self.scales[1] = np.where(np.isnan(scales), scales, new_scales)

    def element(self, tile, head):
        return (tile + 7 * head) % self.dim

    def rows(self, i, head):
        """For request i's queries and the heads of a cache head: the outputs [n, G, dim] in
        float64, the part of themselves that they may be off by [n, G], and each
        tile's share of the softmax and of its element [n, G, tiles]."""
        G, L, n = self.qh // self.kh, int(self.lens[i]), int(self.new[i])
        k, v, _ = self.kv(i, head)
        q = self.q[self.cu[i]: self.cu[i + 1], head * G: (head + 1) * G].astype(np.float64)
        scale = self.dim ** -0.5
        t, p = np.arange(L), L - n + np.arange(n)[:, None]
        seen = t <= p
        if self.window:
            seen &= (t > p - self.window) | (t < self.sinks)
        s = np.where(seen[:, None], q @ k.T * scale, -np.inf)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        out = w @ v
        # A level in fp16 is off by 2^-12 of itself (the values' nonzero one as well
        # as the keys'), a query by 2^-24 of its row's largest, a weight by 2^-12, and
        # float32 sums of dim products by dim 2^-24 of the products' sizes: a score
        # moves by d, a weight by 2 d of itself (its own score and the sum), and the
        # result by as much.  The sums over the tokens are chains of at most a
        # step for each tile and 64 more, at 2^-23 each (numerator and sum); the
        # output is rounded to bf16, 2^-9 of itself.
        d = ((2.0 ** -12 + self.dim * 2.0 ** -24) * (np.abs(q) @ np.abs(k).T).max(-1)
             + 2.0 ** -24 * np.abs(q).max(-1) * np.abs(k).sum(-1).max()) * scale
        part = 2 * d * (1 + d) + 2.0 ** -11 + 2.0 ** -9 + (L / TILE + 64) * 2.0 ** -22
        of = -(-L // TILE)
        pad = [(0, 0), (0, 0), (0, of * TILE - L)]
        share = np.pad(w, pad).reshape(n, G, of, TILE).sum(-1)
        e = self.element(np.arange(of), head)
        at_e = v[t, e[t // TILE]]
        mine = np.pad(w * at_e, pad).reshape(n, G, of, TILE).sum(-1)
        with np.errstate(invalid="ignore", divide="ignore"):
            return out, part, share, mine / out[..., e]

    def shows(self, i, head):
        """What leaving out, or doubling, a tile does to its element, or to the others
        through the sum, as a multiple of what passes unseen: of each tile that some row sees, the row where it shows
        most; of those, the tile that shows least.  (A row's only tile counts
        once however often it is taken.)"""
        out, part, share, mine = self.rows(i, head)
        seen, only = share > 0, share > 1 - 1e-9
        with np.errstate(invalid="ignore", divide="ignore"):
            without = np.where(only, 1.0, np.abs((1 - mine) / (1 - share) - 1))
            twice = np.where(only, np.inf, np.abs((1 + mine) / (1 + share) - 1))
        # (an element of other tiles goes up, or down, by the tile's share)
        others = np.where(mine > 1 - 1e-9, share / (1 + share), 0)
        without, twice = np.maximum(without, others), np.maximum(twice, others)
        # the result itself may be off by `part`, and as much more passes
        times = np.where(seen, np.minimum(without, twice) / (2 * part[..., None]), 0).max((0, 1))
        return times[seen.any((0, 1))].min() if seen.any() else np.inf

    def check_tiles(self, got, heads):
        from tests import gpu_util as U

        got = U.bf16_to_f64(got).reshape(len(self.q), self.qh, self.dim)
        G, worst = self.qh // self.kh, 0.0
        for i in range(len(self.lens)):
            if not self.new[i]:
                continue
            for h in heads:
                mine = got[self.cu[i]: self.cu[i + 1], h * G: (h + 1) * G]
                if not self.lens[i]:
                    assert not mine.any()
                    continue
                out, part, _, _ = self.rows(i, h)
                err = np.abs(mine - out)
                assert np.all(err <= part[..., None] * out), "request %d head %d: %.3g of the bound" % (
                    i, h, (err / np.maximum(part[..., None] * out, 1e-300)).max())
                worst = max(worst, float((err / np.maximum(part[..., None] * out, 1e-300)).max()))
        print("worst error %.3f of the bound" % worst, flush=True)


def old_bound_sees(s, i, head):
    """Of a request's tiles, how many the bound of kv_ref.attention sees missing."""
    G = s.qh // s.kh
    k, v, amax = s.kv(i, head)
    q = s.q[s.cu[i]: s.cu[i + 1], head * G: (head + 1) * G].astype(np.float64)
    out, bound = R.attention(q, k, v, amax, s.dim ** -0.5, int(s.new[i]), getattr(s, "window", 0), getattr(s, "sinks", 0))
    w = np.exp(q @ k.T * s.dim ** -0.5)
    hits = 0
    for t0 in range(0, len(k), TILE):
        keep = np.r_[0:t0, t0 + TILE: len(k)]
        if not len(keep):
            hits += 1
            continue
        ref = (w[..., keep] / w[..., keep].sum(-1, keepdims=True)) @ v[keep]
        hits += bool((np.abs(ref - out) > bound).any())
    return hits, -(-len(k) // TILE)
