"""The operators of a drafted tree's step and of forked rows: what a pass of each is, in plain form and by this library.

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs a serving program has in hand, ``run()`` one pass
through an operator (``own`` False: elementary torch operations in 32 or 64 bits; True: the library's entry points),
``exact()`` the same outputs from the definition in 64 bits, ``work()`` the bytes and operations a pass cannot do
without.  Nothing here is needed to use the library.

A serving step over drafted trees attends over the window (``decode_attn_latent_tree``), draws the target's own token at
each of its tokens (``sample_tokens``), walks the path that stands (``verify_tree``) and moves that path's rows together in
every layer's cache (``kv_keep_tokens``); several continuations of one prompt begin with ``kv_fork_rows``.
"""
import math
from fractions import Fraction

import numpy as np
import torch

own = False

ROT = 64             # rotated columns of a latent row and of a query
ONE = float(1 << 40)  # weights are whole multiples of 2^-40

# (KV heads, stored K columns, V columns, page size) of a pool; latent ones have no V
POOLS = dict(split512=(4, 512, 512, 256), split256=(16, 256, 256, 64), folded512=(4, 128, 512, 256),
             latent512=(1, 512 + ROT, 0, 256), latent256=(1, 256 + ROT, 0, 64))


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # one stream's next token: every filter, a vocabulary of odd size, logits in bf16; latency is all
        dict(name="sample_1_v32001", op="sample", batch=1, tokens=1, vocab=32001, dtype="bf16", heat=True, top_k=50,
             top_p=0.9, min_p=0.02, masked=0.0, probs="", padded=False),
        # a served batch with a temperature and a top-p of its own for each request
        dict(name="sample_64_v131072", op="sample", batch=64, tokens=1, vocab=131072, dtype="f32", heat=True, top_k=0,
             top_p=0.95, min_p=0.0, masked=0.0, probs="", padded=False),
        # the same without filters: the draw alone
        dict(name="draw_256_v32001", op="sample", batch=256, tokens=1, vocab=32001, dtype="f32", heat=True, top_k=0,
             top_p=1.0, min_p=0.0, masked=0.0, probs="", padded=False),
        # a draft's filtered distributions for verify_drafts, bf16 logits in rows padded to a multiple of 64, a grammar's mask
        dict(name="probs_16x5_v32001", op="sample", batch=16, tokens=5, vocab=32001, dtype="bf16", heat=True, top_k=200,
             top_p=0.9, min_p=0.0, masked=0.3, probs="f32", padded=True),
        # a tree of eight drafts over one long context
        dict(name="tree_1x8x40002", op="tree", rows=1, tokens=8, keys=40002, heads=32, latent=512, page=256),
        # wider trees over several ragged contexts
        dict(name="tree_4x16x10602", op="tree", rows=4, tokens=16, keys=10602, heads=32, latent=512, page=256),
        # one tree, where latency counts
        dict(name="walk_1x8", op="walk", rows=1, tokens=8),
        # a served batch of the widest windows
        dict(name="walk_64x64", op="walk", rows=64, tokens=64),
        # one stream's standing path in one latent layer
        dict(name="keep_1x8_latent", op="keep", rows=1, tokens=8, context=1000, layers=1, pool="latent512"),
        # a batch's paths in four layers of whole K and V rows
        dict(name="keep_32x16_split", op="keep", rows=32, tokens=16, context=300, layers=4, pool="split512"),
        # three more continuations of one prompt in one latent layer
        dict(name="fork_1x3_latent", op="fork", rows=1, forks=3, context=1000, layers=1, pool="latent512"),
        # four continuations of each of sixteen prompts, four layers
        dict(name="fork_16x4_split", op="fork", rows=16, forks=4, context=700, layers=4, pool="split512"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "tree", "tree", "walk", "keep", "fork"])
    if op == "sample":
        vocab = _log(rng, 1000, 131072)
        rows = _log(rng, 1, min(256, 64 * 131072 // vocab))  # the largest listed ones' values
        tokens = rng.choice([1, 1, rng.randint(1, min(8, rows))])
        probs = rng.choice(["", "", "f32", "bf16"])
        return dict(op=op, batch=max(1, rows // tokens // (2 if probs else 1)), tokens=tokens, vocab=vocab,
                    dtype=rng.choice(["bf16", "f32"]), heat=rng.random() < 0.8,
                    top_k=rng.choice([0, 0, 1, _log(rng, 2, min(1000, vocab))]),
                    top_p=rng.choice([1.0, 1.0, 0.5, 0.9, 0.95, 0.99]), min_p=rng.choice([0.0, 0.0, 0.05]),
                    masked=rng.choice([0.0, 0.0, 0.5]), probs=probs, padded=rng.random() < 0.5)
    if op == "tree":
        rows, tokens = _log(rng, 1, 32), _log(rng, 1, 64)
        heads = rng.choice([8, 16, 20, 32, 40, 64, 128])
        # the largest listed one: 4 x 16 tokens x 10,602 keys under 32 heads
        most = min(40002, 4 * 16 * 10602 * 32 // (rows * tokens * heads), 4 * 40002 // rows)
        return dict(op=op, rows=rows, tokens=tokens, keys=_log(rng, tokens, max(tokens, most)), heads=heads,
                    latent=rng.choice([256, 512, 512]), page=rng.choice([64, 256]))
    if op == "walk":
        return dict(op=op, rows=_log(rng, 1, 64), tokens=_log(rng, 1, 64))
    pool = rng.choice(sorted(POOLS))
    layers, context = rng.randint(1, 4), _log(rng, 64, 1000)
    if op == "keep":
        return dict(op=op, rows=_log(rng, 1, 32 * 300 // max(300, context)), tokens=_log(rng, 2, 64), context=context,
                    layers=layers, pool=pool)
    rows = _log(rng, 1, 16 * 300 // max(300, context))
    return dict(op=op, rows=rows, forks=rng.randint(1, 4), context=context, layers=layers, pool=pool)


# ---- inputs ----------------------------------------------------------------------

def _dev(x, kind=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=kind).cuda()


def _lengths(case):
    """Keys of each row: ragged, the last row's a little over half the first's; its own window at least."""
    n, hi = case["rows"], case["keys"]
    return [max(case["tokens"], hi - hi * b // (2 * n)) for b in range(n)]


def _kept(case):
    """Standing tokens of each row, and how many of them lie where they are: the rest come from behind the kept ones
    (as a branch's do), so that a pass can be made again on the same state."""
    t, out = case["tokens"], []
    for b in range(case["rows"]):
        kept = 1 + (5 * b + 3) % max(1, min(9, t // 2))
        still = 1 + b % 2 if kept > 1 else 1
        out.append((kept, min(still, kept)))
    return out


def _contexts(case):
    """Keys of each forked row: around the case's, their last pages filled to different heights."""
    return [case["context"] + (97 * b) % 61 for b in range(case["rows"])]


def _tables(lens, page, rng, more=0):
    """Pages of each row, drawn without order from one pool (with ``more`` left over); -1 behind a row's last page."""
    need = [max(1, -(-n // page)) for n in lens]
    ids = rng.permutation(sum(need) + more).astype(np.int32)
    table, at = np.full((len(lens), max(need)), -1, np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, need, ids[at:]


def _normal(gen, *shape, scale=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, scale, generator=gen)


def _trees(rng, rows, tokens):
    """Random trees: each later token below an earlier one, mostly a late one; masks of ancestors, and the parents."""
    parent = np.full((rows, tokens), -1, np.int64)
    mask = np.zeros((rows, tokens), np.uint64)
    mask[:, 0] = 1
    for t in range(1, tokens):
        parent[:, t] = np.minimum(t - 1, (t * rng.random(rows) ** 0.7).astype(np.int64))
        mask[:, t] = mask[np.arange(rows), parent[:, t]] | (np.uint64(1) << np.uint64(t))
    return mask.view(np.int64), parent


def _pools(st, case, gen, pages):
    """A cache of some layers: [layers, pages, heads, page size, columns]; V None for latent rows."""
    heads, dk, dv, page = POOLS[case["pool"]]
    st["k"] = _normal(gen, case["layers"], pages, heads, page, dk)
    st["v"] = _normal(gen, case["layers"], pages, heads, page, dv) if dv else None


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "sample":
        b, t, v = case["batch"], case["tokens"], case["vocab"]
        wide = -(-v // 64) * 64 if case["padded"] else v
        logits = torch.empty(b, t, wide, device="cuda").normal_(0.0, 2.5, generator=gen)
        # every other request is sure of itself: some tokens stand far above the others
        peaks = torch.randint(v, (b, t, 12), device="cuda", generator=gen)
        lift = 12.0 * torch.rand(b, t, 12, device="cuda", generator=gen)
        lift[1::2] = 0.0
        logits.scatter_add_(2, peaks, lift)
        if case["masked"]:
            logits.masked_fill_(torch.rand(b, 1, wide, device="cuda", generator=gen) < case["masked"], -math.inf)
        logits = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        st["logits"] = logits[..., :v]                                      # rows may be padded
        st["u"] = torch.rand(b, t, device="cuda", generator=gen)
        st["temperature"] = 0.5 + torch.rand(b, device="cuda", generator=gen) if case["heat"] else None
        i = np.arange(b)
        st["top_k"] = _dev(case["top_k"] + i % 3) if case["top_k"] else None
        st["top_p"] = _dev(case["top_p"] - 0.02 * (i % 4), torch.float32) if case["top_p"] < 1.0 else None
        st["min_p"] = _dev(case["min_p"] * (1 + i % 2), torch.float32) if case["min_p"] else None
        kind = torch.bfloat16 if case["probs"] == "bf16" else torch.float32
        st["probs"] = torch.empty(b, t, v, dtype=kind, device="cuda") if case["probs"] else None
    elif case["op"] == "tree":
        lens, d = _lengths(case), case["latent"] + ROT
        table, need, _ = _tables(lens, case["page"], rng)
        st["table"] = _dev(table)
        st["pool"] = _normal(gen, sum(need), 1, case["page"], d)            # normalised latents and rotated keys
        st["q"] = _normal(gen, case["rows"], case["tokens"], case["heads"], d)
        st["lens_host"], st["lens"] = lens, _dev(lens)
        st["mask"] = _dev(_trees(rng, case["rows"], case["tokens"])[0], torch.int64)
        st["scale"] = (128 + ROT) ** -0.5
    elif case["op"] == "walk":
        rows, t = case["rows"], case["tokens"]
        mask, parent = _trees(rng, rows, t)
        # drafts and the target's tokens from a few likely ones: siblings differ or not, paths stand for some tokens
        drafts, sampled = rng.integers(0, 4, (rows, t)), rng.integers(0, 4, (rows, t))
        take = rng.random((rows, t)) < 0.5
        for i in range(1, t):  # half of the drafts are what the target says at their parent
            drafts[:, i] = np.where(take[:, i], sampled[np.arange(rows), parent[:, i]], drafts[:, i])
        st["mask"], st["drafts"], st["sampled"] = _dev(mask, torch.int64), _dev(drafts), _dev(sampled)
    elif case["op"] == "keep":
        t, page = case["tokens"], POOLS[case["pool"]][3]
        lens = [max(t, case["context"] + 5 * b % 97) for b in range(case["rows"])]
        table, need, _ = _tables(lens, page, rng)
        _pools(st, case, gen, sum(need))
        path = np.full((case["rows"], t), -1, np.int64)
        for b, (kept, still) in enumerate(_kept(case)):
            path[b, :still] = np.arange(still)
            path[b, still:kept] = np.sort(rng.choice(np.arange(kept, t), kept - still, replace=False))
        st["table"], st["lens"] = _dev(table), _dev(lens)
        st["path"], st["kept"] = _dev(path), _dev([k for k, _ in _kept(case)])
    else:
        n, page = case["rows"] * case["forks"], POOLS[case["pool"]][3]
        lens = _contexts(case)
        table, need, spare = _tables(lens, page, rng, more=n)
        _pools(st, case, gen, sum(need) + n)
        # the forks' rows lie behind the prompts', still empty
        st["table"] = _dev(np.concatenate([table, np.full((n, table.shape[1]), -1, np.int32)]))
        st["lens"], st["pages"] = _dev(lens + [0] * n), _dev(need + [0] * n)
        st["src"] = _dev(np.repeat(np.arange(case["rows"]), case["forks"]))
        st["dst"] = _dev(case["rows"] + rng.permutation(n))
        st["new"] = _dev(spare)
    return st


# ---- one pass --------------------------------------------------------------------

def _share(x, s):
    """floor(x * s) exactly, for 32-bit x in [0, 1) and whole numbers s below 2^58."""
    m, e = torch.frexp(x)
    m, shift = (m * 16777216.0).long(), (4 - e.long()).clamp(max=63)        # x = m * 2^(e - 24)
    return ((s >> 20) * m + ((s & 1048575) * m >> 20)) >> shift


def _plain_sample(st):
    case = st["case"]
    b, t, v = case["batch"], case["tokens"], case["vocab"]
    each = lambda p: None if p is None else p.repeat_interleave(t)[:, None]  # a request's setting at each of its tokens
    l = st["logits"].reshape(b * t, v).float()
    x = l - l.amax(-1, keepdim=True)
    if st["temperature"] is not None:
        x = x * each(1.0 / st["temperature"])
    w = torch.exp(x)
    whole = torch.round(w.double() * ONE).long()
    if st["top_k"] is not None or st["top_p"] is not None:
        x, order = torch.sort(x, dim=-1, descending=True, stable=True)      # ties: the lowest index first
        run = whole.gather(1, order)
        place = torch.arange(v, device="cuda")
        if st["top_k"] is not None:
            run = run * (place < each(st["top_k"]))
        keep = run > 0
        if st["top_p"] is not None:
            before = run.cumsum(1) - run
            keep &= (before < _share(each(st["top_p"]), run.sum(1, keepdim=True))) | (place == 0)
        whole = whole * torch.zeros_like(keep).scatter_(1, order, keep)
    if st["min_p"] is not None:
        whole = whole * (w >= each(st["min_p"]))
    run = whole.cumsum(1)
    total = run[:, -1:]
    token = (run > _share(st["u"].reshape(-1, 1), total)).int().argmax(1).to(torch.int32).reshape(b, t)
    if st["probs"] is None:
        return dict(tokens=token)
    st["probs"].copy_((whole.double() / total).to(torch.float32).reshape(b, t, v))
    return dict(tokens=token, probs=st["probs"])


def _plain_tree(st):
    case, dc = st["case"], st["case"]["latent"]
    rows, t, heads = case["rows"], case["tokens"], case["heads"]
    table = st["table"].long().clamp(min=0)
    keys = st["pool"][table, 0].flatten(1, 2).float()                       # [rows, longest, latent + 64]
    s = torch.matmul(st["q"].flatten(1, 2).float(), keys.transpose(1, 2)) * st["scale"]
    at = torch.arange(keys.shape[1], device="cuda") - (st["lens"].long()[:, None] - t)  # place in the window
    marked = (st["mask"][:, :, None] >> at.clamp(0, 63)[:, None]) & 1
    seen = (at < 0)[:, None] | ((marked != 0) & (at < t)[:, None])          # [rows, tokens, keys]
    s = s.view(rows, t, heads, -1).masked_fill_(~seen[:, :, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s.flatten(1, 2), keys[..., :dc]).view(rows, t, heads, dc) / s.sum(-1, keepdim=True)
    return o.to(torch.bfloat16)


def _plain_walk(st):
    rows, t = st["case"]["rows"], st["case"]["tokens"]
    i = torch.arange(t, device="cuda")
    anc = ((st["mask"][:, :, None] >> i) & 1).bool()                        # [rows, token, ancestor or itself]
    parent = torch.where(anc & (i < i[:, None]), i, -1).amax(-1)            # -1: a root
    says = st["sampled"].gather(1, parent.clamp(min=0))
    right = (parent >= 0) & (st["drafts"] == says) & (says >= 0)
    twin = (parent[:, :, None] == parent[:, None]) & right[:, None] & (i < i[:, None])
    right = (right & ~twin.any(-1)) | (i == 0)                              # the lowest of equal siblings
    stands = (~anc | right[:, None]).all(-1) & anc[:, :, 0]
    kept = stands.sum(1)
    path = torch.where(stands, i, t).sort(-1)[0]
    tokens = torch.where(i < kept[:, None], st["sampled"].gather(1, path.clamp(max=t - 1)), -1)
    path = torch.where(i < kept[:, None], path, -1)
    return dict(tokens=tokens.to(torch.int32), path=path.to(torch.int32), kept=kept.to(torch.int32))


def _cache(st):
    return dict(k=st["k"], **({} if st["v"] is None else dict(v=st["v"])))


def _plain_keep(st):
    t, page = st["case"]["tokens"], POOLS[st["case"]["pool"]][3]
    i = torch.arange(t, device="cuda")
    first = (st["lens"] - t).long()[:, None]
    real = i < st["kept"][:, None]
    source, target = (first + st["path"])[real].long(), (first + i)[real]
    row = torch.arange(first.shape[0], device="cuda")[:, None].expand_as(real)[real]
    a, c = st["table"][row, source // page].long(), st["table"][row, target // page].long()
    for pool in _cache(st).values():
        pool[:, c, :, target % page] = pool[:, a, :, source % page]
    return dict(_cache(st), lens=(first[:, 0] + st["kept"]).to(torch.int32))


def _plain_fork(st):
    page = POOLS[st["case"]["pool"]][3]
    src, dst = st["src"].long(), st["dst"].long()
    length = st["lens"][src].long()
    last, rest = length // page, length % page
    slot = torch.arange(st["table"].shape[1], device="cuda")
    mine = (slot == last[:, None]) & (rest > 0)[:, None]                    # the page that is not full
    old = st["table"][src].long()
    shared = torch.where(slot < last[:, None], st["table"][src], st["table"][dst])
    st["table"][dst] = torch.where(mine, st["new"][:, None], shared)
    st["lens"][dst] = length.to(torch.int32)
    st["pages"][dst] = (last + (rest > 0)).to(torch.int32)
    from_page = old.gather(1, last.clamp(max=old.shape[1] - 1)[:, None])[:, 0]
    n, i = torch.nonzero(torch.arange(page, device="cuda") < rest[:, None], as_tuple=True)
    for pool in _cache(st).values():
        pool[:, st["new"].long()[n], :, i] = pool[:, from_page[n], :, i]
    return dict(_cache(st), table=st["table"], lens=st["lens"], pages=st["pages"])


def _own_sample(st):
    import paged_split_kv_attn_gb300 as pskv
    tokens = pskv.sample_tokens(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                                top_p=st["top_p"], min_p=st["min_p"], probs=st["probs"])
    return dict(tokens=tokens, **({} if st["probs"] is None else dict(probs=st["probs"])))


def _own_tree(st):
    import paged_split_kv_attn_gb300 as pskv
    if "layout" not in st:
        case = st["case"]
        st["layout"] = pskv.paged_kv_layout_create(st["pool"], None)
        st["workspace"] = pskv.latent_workspace(st["layout"], st["lens_host"], case["tokens"], case["heads"])
    return pskv.decode_attn_latent_tree(st["layout"], st["q"], st["table"], st["lens"], st["lens_host"], st["mask"],
                                        st["scale"], workspace=st["workspace"])


def _own_walk(st):
    import paged_split_kv_attn_gb300 as pskv
    tokens, path, kept = pskv.verify_tree(st["drafts"], st["mask"], st["sampled"])
    return dict(tokens=tokens, path=path, kept=kept)


def _layouts(st):
    import paged_split_kv_attn_gb300 as pskv
    if "layouts" not in st:
        st["layouts"] = [pskv.paged_kv_layout_create(st["k"][l], None if st["v"] is None else st["v"][l])
                         for l in range(st["case"]["layers"])]
    return st["layouts"]


def _own_keep(st):
    import paged_split_kv_attn_gb300 as pskv
    lens = pskv.kv_keep_tokens(_layouts(st), st["table"], st["lens"], st["path"], st["kept"])
    return dict(_cache(st), lens=lens)


def _own_fork(st):
    import paged_split_kv_attn_gb300 as pskv
    pskv.kv_fork_rows(_layouts(st), st["src"], st["dst"], st["new"], st["table"], st["lens"], st["pages"])
    return dict(_cache(st), table=st["table"], lens=st["lens"], pages=st["pages"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(sample=_own_sample, tree=_own_tree, walk=_own_walk, keep=_own_keep, fork=_own_fork)[op](state)
    return dict(sample=_plain_sample, tree=_plain_tree, walk=_plain_walk, keep=_plain_keep, fork=_plain_fork)[op](state)


# ---- the definition in 64 bits -----------------------------------------------------

def _probabilities64(l, heat, top_k, top_p, min_p):
    """One row's filtered distribution.  What is drawn from is defined on the scaled logits as 32-bit numbers."""
    x = (l - l.max()).astype(np.float32)
    if heat is not None:
        x = x * np.float32(np.float32(1) / np.float32(heat))
    w = np.rint(np.exp(x.astype(np.float64)).astype(np.float32).astype(np.float64) * ONE).astype(np.int64)
    order = np.lexsort((np.arange(x.size), -x.astype(np.float64)))
    kept = np.ones(x.size, bool)
    if top_k is not None:
        kept[order[int(top_k):]] = False
    if top_p is not None:
        mine = np.where(kept, w, 0)[order]
        run = np.cumsum(mine)
        out = run - mine >= math.floor(Fraction(float(np.float32(top_p))) * int(run[-1]))
        out[0] = False
        kept[order[out]] = False
    if min_p is not None:
        kept &= np.exp(x.astype(np.float64)).astype(np.float32) >= np.float32(min_p)
    w = np.where(kept, w, 0)
    return w.astype(np.float64) / float(w.sum())


def exact(case, seed):
    if case["op"] == "sample" and case["probs"]:
        st = prepare(case, seed)
        logits = st["logits"].float().cpu().numpy()
        per = {k: None if st[k] is None else st[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p")}
        out = np.empty(logits.shape)
        for b in range(case["batch"]):
            for t in range(case["tokens"]):
                out[b, t] = _probabilities64(logits[b, t], *[None if per[k] is None else per[k][b] for k in per])
        return dict(tokens=None, probs=torch.from_numpy(out))
    if case["op"] != "tree":
        return None  # whole numbers, or rows moved as they are
    st = prepare(case, seed)
    t, dc, out = case["tokens"], case["latent"], []
    masks = st["mask"].cpu().numpy().view(np.uint64)
    for b, n in enumerate(st["lens_host"]):
        k = st["pool"][st["table"][b, :-(-n // case["page"])].long(), 0].reshape(-1, dc + ROT)[:n].double()
        s = torch.einsum("thd,kd->thk", st["q"][b].double(), k) * st["scale"]
        for i in range(t):
            hidden = [j for j in range(t) if not (int(masks[b, i]) >> j) & 1]
            s[i, :, [n - t + j for j in hidden]] = -math.inf
        out.append(torch.einsum("thk,kd->thd", torch.softmax(s, -1), k[:, :dc]))
    return torch.stack(out)


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    if case["op"] == "sample":
        n = case["batch"] * case["tokens"]
        size = 2 if case["dtype"] == "bf16" else 4
        out = {"": 0, "f32": 4, "bf16": 2}[case["probs"]]
        return dict(bytes=n * (case["vocab"] * (size + out) + 24), flops=n * case["vocab"] * 3)
    if case["op"] == "tree":
        dc, n, keys = case["latent"], case["rows"] * case["tokens"] * case["heads"], sum(_lengths(case))
        pairs = case["tokens"] * case["heads"] * keys
        return dict(bytes=keys * (dc + ROT) * 2 + n * (2 * dc + ROT) * 2 + case["rows"] * case["tokens"] * 8,
                    flops=2 * pairs * (2 * dc + ROT))
    if case["op"] == "walk":
        return dict(bytes=case["rows"] * (case["tokens"] * 24 + 4), flops=case["rows"] * case["tokens"])
    heads, dk, dv, page = POOLS[case["pool"]]
    row = heads * (dk + dv) * 2 * case["layers"]
    if case["op"] == "keep":
        moved = sum(k - s for k, s in _kept(case))
        return dict(bytes=2 * moved * row + case["rows"] * (case["tokens"] * 4 + 12), flops=0)
    rest = sum(n % page for n in _contexts(case))
    tables = sum(-(-n // page) for n in _contexts(case)) * 4
    return dict(bytes=(1 + case["forks"]) * (rest * row + tables) + case["rows"] * (case["forks"] * 20 + 8), flops=0)
