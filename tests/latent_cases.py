"""Inputs and 64-bit references for the latent-cache operators and the draft
verification (used by their GPU tests only).  The references are written from
the formulas in plain torch (f64) and Python integers; nothing of the library
computes them."""
from __future__ import annotations

import numpy as np
import torch

import paged_split_kv_attn_gb300 as pskv

ROT = 64
HALF_BF16 = 2.0 ** -8  # a rounding to bf16 is off by at most this share of the value


def normal(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


class LatentCase:
    """A latent pool with rows of the given lengths.  Every pool row no key occupies
    (behind a row's end, and the last page, which table entries behind a
    row's pages name) is NaN: none of it may reach an output."""

    def __init__(self, seed, lens, dc=512, page=64, heads=32, tokens=1, scale=None, extra=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens_host, self.dc, self.page, self.tokens, self.heads = list(lens), dc, page, tokens, heads
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 1 + extra
        self.pool = torch.full((pages, 1, page, dc + ROT), float("nan"), dtype=torch.bfloat16, device="cuda")
        stride = max(1, max(need))
        table = np.full((len(lens), stride), pages - 1, np.int32)
        ids = rng.permutation(pages - 1).astype(np.int32)
        at = 0
        self.keys = []
        for b, n in enumerate(lens):
            table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            k = normal(gen, n, dc + ROT)
            self.keys.append(k)
            flat = self.pool.view(-1, dc + ROT)
            i = torch.arange(n, device="cuda")
            where = torch.from_numpy(table[b].astype(np.int64)).cuda()[i // page] * page + i % page
            flat[where] = k
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = normal(gen, len(lens), tokens, heads, dc + ROT)
        self.scale = (128 + ROT) ** -0.5 if scale is None else scale
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.layout = pskv.paged_kv_layout_create(self.pool, None, self.status)

    def run(self, **kw):
        return pskv.decode_attn_latent(self.layout, self.q, self.table, self.lens, self.lens_host,
                                       self.scale, **kw)

    def reference(self, hidden=None):
        """f64 attention; ``hidden``[b] marks keys (a bool mask) no token sees."""
        out = torch.zeros(len(self.lens_host), self.tokens, self.heads, self.dc, dtype=torch.float64,
                          device="cuda")
        for b, n in enumerate(self.lens_host):
            if n == 0:
                continue
            k = self.keys[b].double()
            s = torch.einsum("thd,kd->thk", self.q[b].double(), k) * self.scale
            own = n - self.tokens + torch.arange(self.tokens, device="cuda")
            s[(torch.arange(n, device="cuda") > own[:, None])[:, None].expand_as(s)] = -float("inf")
            if hidden is not None and hidden[b] is not None:
                s[:, :, hidden[b]] = -float("inf")
            w = torch.softmax(s, -1)
            w = torch.where(torch.isnan(w), torch.zeros_like(w), w)  # a token without any key
            out[b] = torch.einsum("thk,kd->thd", w, k[:, :self.dc])
        return out


def check_attention(out, ref, values_max):
    """Output against the f64 reference.

    Scores come from exact products of bf16 values added in f32: for the n <= 640
    terms of these inputs (|sum of |q k|| * scale < 60) the error stays below n * 2^-24 * 60
    < 2.3e-3 at the very worst and around sqrt(n) * 2^-24 * 60 ~ 1e-4 in practice; a
    relative error d of every weight moves an output by at most 2 d max|v|.
    bf16 output: weights rounded to bf16 (2^-8 each) and the output once more
    (2^-8); over many elements both errors have independent signs, so the 2-norm is off by
    less than 2 * 2^-8.  f32 output: weights as a bf16 pair (2^-16)."""
    half = HALF_BF16 if out.dtype == torch.bfloat16 else 2.0 ** -16
    y = out.double()
    assert torch.isfinite(y).all()
    err = (y - ref).abs()
    bound = 2 * (2.3e-3 + half) * values_max + (half if out.dtype == torch.bfloat16 else 2.0 ** -24) * ref.abs()
    assert (err <= bound).all(), float((err - bound).max())
    norm = float(ref.norm())
    if norm > 0:
        limit = 2 * HALF_BF16 if out.dtype == torch.bfloat16 else 1e-4
        assert float(err.norm()) <= limit * norm, float(err.norm()) / norm


# ---- the drafts' verification, in whole numbers ----------------------------------

def fixed(p) -> int:
    """The nearest multiple of 2^-60 (ties to the even one), NaN and below 0 as 0, above 1 as 1."""
    from fractions import Fraction
    p = float(p)
    if not p > 0:
        return 0
    return 1 << 60 if p >= 1 else round(Fraction(p) * (1 << 60))


def verify_reference(target, draft, drafts, u, num_drafts=None):
    """The verification's definition in Python integers and fractions."""
    from fractions import Fraction
    target, u = target.float().cpu().numpy(), u.cpu().numpy()
    draft = None if draft is None else draft.float().cpu().numpy()
    drafts = drafts.cpu().numpy()
    batch, t, vocab = target.shape[0], target.shape[1] - 1, target.shape[2]
    clamp = lambda x: Fraction(0) if not x > 0 else min(Fraction(1), Fraction(float(x))) if np.isfinite(x) else Fraction(1)
    tokens, accepted = [], []
    for b in range(batch):
        d = t if num_drafts is None else min(max(int(num_drafts[b]), 0), t)
        a = 0
        while a < d:
            x = int(drafts[b, a])
            if not 0 <= x < vocab:
                break
            q = Fraction(1) if draft is None else clamp(draft[b, a, x])
            if not clamp(u[b, a]) * q < clamp(target[b, a, x]):
                break
            a += 1
        p = [fixed(v) for v in target[b, a]]
        r = p
        if a < d:
            if draft is None:
                r = list(p)
                if 0 <= drafts[b, a] < vocab:
                    r[drafts[b, a]] = 0
            else:
                r = [max(x - fixed(y), 0) for x, y in zip(p, draft[b, a])]
            if sum(r) == 0:
                r = p
        total, token = sum(r), -1
        if total:
            uu = clamp(u[b, t])
            limit = total - 1 if uu >= 1 else (uu.numerator * total) // uu.denominator
            run = 0
            for v, x in enumerate(r):
                run += x
                if run > limit:
                    token = v
                    break
        tokens.append([int(drafts[b, i]) for i in range(a)] + [token] + [-1] * (t - a))
        accepted.append(a)
    return np.array(tokens, np.int32), np.array(accepted, np.int32)
