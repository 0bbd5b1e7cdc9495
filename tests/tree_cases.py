"""Inputs and references for sampling, drafted trees and forked rows (used by their GPU tests only).  The
references are written from the formulas in numpy and Python integers; nothing of the library computes them."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

ONE = 1 << 40


# ---- sampling ----------------------------------------------------------------------

def share(x, s: int) -> int:
    """floor(x * s) for x in [0, 1); below 0 and NaN count as 0."""
    x = float(np.float32(x))
    return (Fraction(x) * s).__floor__() if x > 0 else 0


def weights(l, heat):
    """(x, w, W) of one row of logits: 32-bit steps, the exponential as CUDA's expf rounds it, whole multiples of 2^-40."""
    l = np.where(np.isnan(l), -np.inf, l).astype(np.float32)
    with np.errstate(all="ignore"):
        x = np.where(l == l.max(), np.float32(0), (l - l.max()) * np.float32(np.float32(1) / np.float32(heat)))
    x = np.where(np.isnan(x) | (l == -np.inf), -np.inf, x).astype(np.float32)
    w = torch.exp(torch.from_numpy(x).cuda()).cpu().numpy()
    # expf is off by two units in the last place at most
    with np.errstate(all="ignore"):
        true = np.exp(x.astype(np.float64))
    assert (np.abs(w - true) <= 2.0 ** -22 * true + 2.0 ** -149).all()
    return x, w, np.rint(w.astype(np.float64) * ONE).astype(np.int64)


def kept_weights(l, heat=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """W of the tokens that the filters keep (0 for the others); None: a row without any logit."""
    l = np.where(np.isnan(l), -np.inf, l)
    if l.max() == -np.inf:
        return None
    with np.errstate(all="ignore"):
        greedy = not heat > 0 or np.isinf(np.float32(1) / np.float32(heat))
    if greedy:
        out = np.zeros(l.size, np.int64)
        out[l.argmax()] = ONE
        return out
    x, w, W = weights(l, heat)
    order = np.lexsort((np.arange(x.size), -x.astype(np.float64)))
    kept = np.ones(x.size, bool)
    if 0 < top_k < x.size:
        kept[order[top_k:]] = False
    if top_p < 1:
        mine = np.where(kept, W, 0)[order]
        before = np.cumsum(mine) - mine
        out = before >= share(top_p, int(mine.sum()))
        out[0] = False
        kept[order[out]] = False
    if min_p > 0:
        kept &= w >= np.float32(min(min_p, 1.0))
    return np.where(kept, W, 0)


def sample_reference(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Tokens and probabilities (f64) of logits [batch, tokens, vocab] by the definition."""
    l = logits.float().cpu().numpy()
    batch, each, vocab = l.shape
    get = lambda t, b, off: off if t is None else float(t[b])
    tokens, probs = np.zeros((batch, each), np.int32), np.zeros(l.shape)
    for b in range(batch):
        for t in range(each):
            W = kept_weights(l[b, t], get(temperature, b, 1.0), int(get(top_k, b, 0)), get(top_p, b, 1.0), get(min_p, b, 0.0))
            if W is None:
                tokens[b, t] = -1
                continue
            total = int(W.sum())
            probs[b, t] = W / total
            if u is not None:
                limit = total - 1 if float(u[b, t]) >= 1 else share(float(u[b, t]), total)
                tokens[b, t] = int((np.cumsum(W) > limit).argmax())
    return tokens, probs


# ---- trees -------------------------------------------------------------------------

def random_masks(rng, batch, tokens, roots=0.0):
    """Ancestor masks [batch, tokens] (uint64) of random trees, token 0 the first root."""
    out = np.zeros((batch, tokens), np.uint64)
    for b in range(batch):
        for t in range(tokens):
            own = np.uint64(1) << np.uint64(t)
            out[b, t] = own if t == 0 or rng.random() < roots else out[b, rng.integers(0, t)] | own
    return out


def i64(masks):
    return torch.from_numpy(np.ascontiguousarray(masks).view(np.int64)).cuda()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def walk_reference(drafts, masks, sampled):
    """verify_tree's definition, token by token."""
    batch, T = drafts.shape
    tokens, path, kept = np.full((batch, T), -1, np.int32), np.full((batch, T), -1, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        def parent(t):
            below = int(masks[b, t]) & ((1 << t) - 1)
            return below.bit_length() - 1
        at = [0]
        while True:
            s = sampled[b, at[-1]]
            nxt = [t for t in range(1, T) if parent(t) == at[-1] and drafts[b, t] == s and s >= 0]
            if not nxt:
                break
            at.append(nxt[0])
        kept[b] = len(at)
        path[b, :len(at)] = at
        tokens[b, :len(at)] = sampled[b, at]
    return tokens, path, kept


# ---- caches ------------------------------------------------------------------------

class Cache:
    """Pools of some layers with random contents, tables of shuffled pages; the host keeps copies."""

    SHAPES = dict(split512=(4, 512, 512, 256, torch.bfloat16), split256=(3, 256, 256, 64, torch.bfloat16),
                  folded=(2, 128, 512, 32, torch.bfloat16), f32=(2, 256, 256, 16, torch.float32),
                  latent512=(1, 576, 0, 64, torch.bfloat16), latent256=(1, 320, 0, 48, torch.bfloat16))

    def __init__(self, seed, kind, lens, layers=1, stride=0, spare=0):
        import paged_split_kv_attn_gb300 as pskv
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        heads, dk, dv, self.page, kind_ = self.SHAPES[kind]
        need = [-(-n // self.page) for n in lens]
        self.stride = max(stride, max(need), 1)
        ids = rng.permutation(sum(need) + spare + 1).astype(np.int32)
        self.table = np.full((len(lens), self.stride), -7, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.spare = ids[at:]
        pages = len(ids)
        new = lambda d: torch.randn(layers, pages, heads, self.page, d, generator=gen, device="cuda").to(kind_)
        self.pools = [new(dk)] + ([new(dv)] if dv else [])
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.layouts = [pskv.paged_kv_layout_create(self.pools[0][l], self.pools[1][l] if dv else None,
                                                    self.status if l == 0 else None) for l in range(layers)]
        self.lens, self.leases = np.array(lens, np.int32), np.array(need, np.int32)
        self.dev_table, self.dev_lens, self.dev_leases = i32(self.table), i32(self.lens), i32(self.leases)

    def host(self):
        return [p.clone() for p in self.pools]

    def faults(self):
        return int(self.status[0].item())
