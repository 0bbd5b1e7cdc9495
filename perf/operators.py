"""The latent-cache and draft-verification operators: what a pass of each is, in plain form and by this library.

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs a serving program has in hand, ``run()`` one pass
through an operator (``own`` False: elementary torch operations in 32 or 64 bits; True: the library's entry points),
``exact()`` the same outputs from the definition in 64 bits, ``work()`` the bytes and operations a pass cannot do
without.  Nothing here is needed to use the library.
"""
import math

import numpy as np
import torch

own = False

ROT = 64    # rotated columns of a latent row and of a query
NOPE = 128  # unrotated columns of an expanded query or key
VAL = 128   # columns of an expanded value
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # a decode step's new tokens, one a row: latents normalised, keys rotated, rows into their pages
        dict(name="append_step_64", op="append", rows=64, tokens=1, context=5000, heads=32, latent=512, page=256,
             pairs="halves", dense=False),
        # a prompt chunk of 8 rows: the dense copy feeds the up-projection, the queries turn for the expanded form
        dict(name="append_chunk_8x1021", op="append", rows=8, tokens=1021, context=300, heads=32, latent=512, page=256,
             pairs="adjacent", dense=True),
        # one short conversation, where latency is all
        dict(name="decode_1x1000", op="decode", lens="flat", rows=1, keys=1000, tokens=1, heads=32, latent=512, page=256),
        # one long context
        dict(name="decode_1x40002", op="decode", lens="flat", rows=1, keys=40002, tokens=1, heads=32, latent=512, page=256),
        # a ragged batch, lengths spread evenly in their logarithm up to 131,072
        dict(name="decode_ragged_16", op="decode", lens="log", rows=16, keys=131072, tokens=1, heads=32, latent=512, page=256),
        # many heads on one latent row: as much arithmetic as bytes
        dict(name="decode_8x10602_h128", op="decode", lens="flat", rows=8, keys=10602, tokens=1, heads=128, latent=512, page=256),
        # small latents in small pages, a batch of short rows (a window's worth of keys and a page)
        dict(name="decode_32x1040_c256", op="decode", lens="flat", rows=32, keys=1040, tokens=1, heads=16, latent=256, page=64),
        # drafted windows: five tokens a row over long contexts
        dict(name="window_4x5x20001", op="decode", lens="flat", rows=4, keys=20001, tokens=5, heads=32, latent=512, page=256),
        # a whole prompt in expanded form
        dict(name="prefill_1x4096", op="prefill", rows=1, tokens=4096, context=0, heads=32),
        # ragged chunks behind cached contexts
        dict(name="prefill_6_ragged", op="prefill", rows=6, tokens=517, context=1900, heads=16),
        # one stream's four drafts, a vocabulary of odd size, probabilities kept in bf16, the draft a plain guess
        dict(name="verify_1x4_v32001", op="verify", rows=1, drafts=4, vocab=32001, dtype="bf16", guess=True),
        # a served batch: seven drafts a row, the draft's own distribution given
        dict(name="verify_64x7_v131072", op="verify", rows=64, drafts=7, vocab=131072, dtype="f32", guess=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "decode", "prefill", "verify"])
    if op == "append":
        rows = _log(rng, 1, 96)
        return dict(op=op, rows=rows, tokens=_log(rng, 1, max(1, 8168 // rows)), context=_log(rng, 1, 6000),
                    heads=rng.randint(1, 32), latent=rng.choice([256, 512]), page=rng.choice([64, 256]),
                    pairs=rng.choice(["halves", "adjacent"]), dense=rng.random() < 0.5)
    if op == "decode":
        rows, tokens, heads = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4, 5, 8]), rng.choice([8, 16, 20, 32, 40, 64, 96, 128])
        lens = rng.choice(["flat", "log"])
        # the largest listed ones: 16 rows of up to 131,072 keys, 8 x 10,602 keys under 128 heads
        most = min(131072, 16 * 131072 // (8 * rows), 8 * 10602 * 128 // (rows * tokens * heads))
        return dict(op=op, lens=lens, rows=rows, keys=_log(rng, 9, max(9, most)), tokens=tokens, heads=heads,
                    latent=rng.choice([256, 512, 512]), page=rng.choice([64, 256]))
    if op == "prefill":
        rows, heads = _log(rng, 1, 12), rng.choice([4, 8, 16, 32])
        # no more than 4,096 x 4,096 / 2 pairs under 32 heads
        side = int(math.sqrt(4096 * 4096 / 2 * 32 / (heads * rows)))
        tokens = _log(rng, 1, min(4096, side))
        return dict(op=op, rows=rows, tokens=tokens, context=rng.choice([0, _log(rng, 1, max(1, min(4096, side - tokens + 1)))]),
                    heads=heads)
    rows = _log(rng, 1, 64)
    return dict(op="verify", rows=rows, drafts=rng.randint(1, 7), vocab=_log(rng, 1000, 131072), dtype=rng.choice(["bf16", "f32"]),
                guess=rng.random() < 0.4)


# ---- inputs ----------------------------------------------------------------------

def _lengths(case, rng):
    """Keys of each row: all the case's, or spread evenly in their logarithm; a row holds its own new tokens at least."""
    n, hi, least = case["rows"], case["keys"], case["tokens"]
    if case["lens"] == "flat":
        return [max(least, hi)] * n
    return [max(least, int(math.exp(rng.uniform(0.0, math.log(max(2, hi)))))) for _ in range(n)]


def _tables(lens, page, rng):
    """Pages of each row, drawn without order from one pool; -1 behind a row's last page."""
    need = [max(1, -(-n // page)) for n in lens]
    ids = rng.permutation(sum(need)).astype(np.int32)
    table, at = np.full((len(lens), max(need)), -1, np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    return torch.from_numpy(table).cuda(), torch.tensor(need, dtype=torch.int32, device="cuda"), sum(need)


def _normal(gen, *shape, scale=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, scale, generator=gen)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "append":
        n, dc = case["rows"] * case["tokens"], case["latent"]
        lens = [case["context"] + case["tokens"] + b % 7 for b in range(case["rows"])]
        st["table"], st["pages"], pages = _tables(lens, case["page"], rng)
        st["pool"] = _normal(gen, pages, 1, case["page"], dc + ROT)
        st["x"] = _normal(gen, n, dc + ROT, scale=2.0)                      # the down-projection's rows: latent, rotated key
        st["q"] = _normal(gen, n, case["heads"], NOPE + ROT)                # the queries' rows
        st["q_out"] = _normal(gen, n, case["heads"], dc + ROT)              # absorbed queries, their rotated columns to come
        st["row_of"] = torch.arange(case["rows"], dtype=torch.int32, device="cuda").repeat_interleave(case["tokens"])
        first = torch.tensor([k - case["tokens"] for k in lens], dtype=torch.int32, device="cuda")
        st["pos_of"] = (first[:, None] + torch.arange(case["tokens"], dtype=torch.int32, device="cuda")).reshape(-1).contiguous()
        st["w"] = torch.empty(dc, device="cuda").normal_(1.0, 0.1, generator=gen)
        angle = np.arange(max(lens))[:, None] * (1e4 ** (-np.arange(ROT // 2) / (ROT // 2)))
        st["cos"] = torch.from_numpy(np.cos(angle).astype(np.float32)).cuda()
        st["sin"] = torch.from_numpy(np.sin(angle).astype(np.float32)).cuda()
        st["dense"] = torch.empty(n, dc + ROT, dtype=torch.bfloat16, device="cuda") if case["dense"] else None
    elif case["op"] == "decode":
        lens, d = _lengths(case, rng), case["latent"] + ROT
        st["table"], st["pages"], pages = _tables(lens, case["page"], rng)
        st["pool"] = _normal(gen, pages, 1, case["page"], d)                # normalised latents and rotated keys
        st["q"] = _normal(gen, case["rows"], case["tokens"], case["heads"], d)
        st["lens_host"], st["lens"] = lens, torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["scale"] = (NOPE + ROT) ** -0.5
    elif case["op"] == "prefill":
        new = [max(1, case["tokens"] - (37 * b) % max(1, case["tokens"] // 2 + 1)) for b in range(case["rows"])]
        old = [case["context"] * (b + 1) // case["rows"] for b in range(case["rows"])]
        st["cu_q_host"] = [0] + np.cumsum(new).tolist()
        st["cu_k_host"] = [0] + np.cumsum([a + b for a, b in zip(new, old)]).tolist()
        st["cu_q"] = torch.tensor(st["cu_q_host"], dtype=torch.int32, device="cuda")
        st["cu_k"] = torch.tensor(st["cu_k_host"], dtype=torch.int32, device="cuda")
        st["q"] = _normal(gen, st["cu_q_host"][-1], case["heads"], NOPE + ROT)
        st["kv"] = _normal(gen, st["cu_k_host"][-1], case["heads"], NOPE + VAL)   # the up-projection's rows: keys, values
        st["k_rot"] = _normal(gen, st["cu_k_host"][-1], ROT)
        st["scale"] = (NOPE + ROT) ** -0.5
    else:
        b, t, v = case["rows"], case["drafts"], case["vocab"]
        kind = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        logits = torch.empty(b, t + 1, v, device="cuda").normal_(0.0, 2.5, generator=gen)
        st["target"] = torch.softmax(logits, -1).to(kind)
        logits = logits[:, :t] + torch.empty(b, t, v, device="cuda").normal_(0.0, 0.7, generator=gen)
        draft = torch.softmax(logits, -1)
        if case["guess"]:
            # a draft without a distribution of its own: the likelier tokens, now and then another
            st["drafts"] = torch.where(torch.rand(b, t, device="cuda", generator=gen) < 0.8, logits.argmax(-1),
                                       torch.randint(v, (b, t), device="cuda", generator=gen)).to(torch.int32)
            st["draft"] = None
        else:
            st["drafts"] = torch.multinomial(draft.reshape(-1, v), 1, generator=gen).reshape(b, t).to(torch.int32)
            st["draft"] = draft.to(kind)
        st["given"] = torch.from_numpy(np.maximum(t - np.arange(b) % 3, 0).astype(np.int32)).cuda()  # drafts of each row
        st["u"] = torch.rand(b, t + 1, device="cuda", generator=gen)
    return st


# ---- one pass --------------------------------------------------------------------

def _turn(x, cos, sin, pairs):
    """Rotate the last dimension's pairs (i, i + half) or (2i, 2i + 1)."""
    if pairs == "halves":
        a, b = x[..., :ROT // 2], x[..., ROT // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_append(st):
    case, dc = st["case"], st["case"]["latent"]
    pos = st["pos_of"].long()
    cos, sin = st["cos"][pos], st["sin"][pos]
    x = st["x"].float()
    c = x[:, :dc] * torch.rsqrt(x[:, :dc].square().mean(-1, keepdim=True) + EPS) * st["w"]
    row = torch.cat([c, _turn(x[:, dc:], cos, sin, case["pairs"])], -1).to(torch.bfloat16)
    page = st["table"][st["row_of"].long(), pos // case["page"]].long()
    st["pool"].view(-1, dc + ROT)[page * case["page"] + pos % case["page"]] = row
    st["q_out"][..., dc:] = _turn(st["q"][..., NOPE:].float(), cos[:, None], sin[:, None], case["pairs"]).to(torch.bfloat16)
    if st["dense"] is not None:
        st["dense"].copy_(row)
    return dict(pool=st["pool"], q_out=st["q_out"], **({} if st["dense"] is None else dict(dense=st["dense"])))


def _plain_decode(st):
    case, dc = st["case"], st["case"]["latent"]
    rows, t, heads = case["rows"], case["tokens"], case["heads"]
    pool, table = st["pool"], st["table"].long().clamp(min=0)
    keys = pool[table, 0].flatten(1, 2).float()                             # [rows, longest, latent + 64]
    s = torch.matmul(st["q"].flatten(1, 2).float(), keys.transpose(1, 2)) * st["scale"]
    own_key = st["lens"].long()[:, None] - t + torch.arange(t, device="cuda")  # [rows, tokens]
    hidden = torch.arange(keys.shape[1], device="cuda") > own_key[..., None]
    s = s.view(rows, t, heads, -1).masked_fill_(hidden[:, :, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s.flatten(1, 2), keys[..., :dc]).view(rows, t, heads, dc) / s.sum(-1, keepdim=True)
    return o.to(torch.bfloat16)


def _padded(cu, longest, total):
    """Index [rows, longest] into `total` packed rows, which of its entries are real, and how many a row has."""
    start, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    i = torch.arange(longest, device="cuda")
    return (start[:, None] + i).clamp(max=total - 1), i < n[:, None], n


def _plain_prefill(st):
    rows, heads = st["case"]["rows"], st["case"]["heads"]
    most_q = max(b - a for a, b in zip(st["cu_q_host"], st["cu_q_host"][1:]))
    most_k = max(b - a for a, b in zip(st["cu_k_host"], st["cu_k_host"][1:]))
    iq, real_q, nq = _padded(st["cu_q"], most_q, st["q"].shape[0])
    ik, _, nk = _padded(st["cu_k"], most_k, st["kv"].shape[0])
    q, kv = st["q"].float()[iq].transpose(1, 2), st["kv"].float()[ik].transpose(1, 2)   # [rows, heads, longest, .]
    k = torch.cat([kv[..., :NOPE], st["k_rot"].float()[ik][:, None].expand(rows, heads, most_k, ROT)], -1)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"])
    own_key = (nk - nq)[:, None] + torch.arange(most_q, device="cuda")                  # [rows, longest query]
    hidden = torch.arange(most_k, device="cuda") > own_key[..., None]
    s = s.masked_fill_(hidden[:, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s, kv[..., NOPE:]) / s.sum(-1, keepdim=True)
    return o.transpose(1, 2)[real_q].to(torch.bfloat16)


def _plain_verify(st):
    b, t, v = st["case"]["rows"], st["case"]["drafts"], st["case"]["vocab"]
    at = st["drafts"].long()[..., None]
    p = st["target"][:, :t].gather(2, at)[..., 0].double()
    q = torch.ones_like(p) if st["draft"] is None else st["draft"].gather(2, at)[..., 0].double()
    u = st["u"].double()
    ok = (u[:, :t] * q < p) & (torch.arange(t, device="cuda") < st["given"][:, None])
    taken = ok.long().cumprod(1).sum(1)                                     # drafts accepted in each row
    row = torch.arange(b, device="cuda")
    rest = st["target"][row, taken].double()                                # what is left to draw from
    drafted = (taken < st["given"])[:, None]                                # a refused draft: without its own share
    k = taken.clamp(max=t - 1)
    if st["draft"] is None:
        less = torch.zeros_like(rest).scatter_(1, at[row, k], 1.0)
    else:
        less = st["draft"][row, k].double()
    left = torch.where(drafted, (rest - less).clamp(min=0.0), rest)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, rest)
    run = left.cumsum(1)
    token = (run > u[:, t:] * run[:, -1:]).int().argmax(1)
    i = torch.arange(t + 1, device="cuda")
    drafts = torch.cat([st["drafts"], st["drafts"][:, :1]], 1).long()
    out = torch.where(i < taken[:, None], drafts, torch.where(i == taken[:, None], token[:, None], -1))
    return dict(tokens=out.to(torch.int32), accepted=taken.to(torch.int32))


def _own_append(st):
    import paged_split_kv_attn_gb300 as pskv
    dc = st["case"]["latent"]
    if "layout" not in st:
        st["layout"] = pskv.paged_kv_layout_create(st["pool"], None)
    pskv.kv_prep_append_latent(st["layout"], st["x"], st["row_of"], st["pos_of"], st["table"], st["pages"], EPS, st["w"],
                               st["cos"], st["sin"], pairs=st["case"]["pairs"], q=st["q"][..., NOPE:],
                               q_out=st["q_out"][..., dc:], dense=st["dense"])
    return dict(pool=st["pool"], q_out=st["q_out"], **({} if st["dense"] is None else dict(dense=st["dense"])))


def _own_decode(st):
    import paged_split_kv_attn_gb300 as pskv
    if "layout" not in st:
        case = st["case"]
        st["layout"] = pskv.paged_kv_layout_create(st["pool"], None)
        st["workspace"] = pskv.latent_workspace(st["layout"], st["lens_host"], case["tokens"], case["heads"])
    return pskv.decode_attn_latent(st["layout"], st["q"], st["table"], st["lens"], st["lens_host"], st["scale"],
                                   workspace=st["workspace"])


def _own_prefill(st):
    import paged_split_kv_attn_gb300 as pskv
    return pskv.prefill_attn_expanded(st["q"], st["kv"], st["k_rot"], st["cu_q"], st["cu_q_host"], st["cu_k"],
                                      st["cu_k_host"], st["scale"])


def _own_verify(st):
    import paged_split_kv_attn_gb300 as pskv
    tokens, accepted = pskv.verify_drafts(st["target"], st["draft"], st["drafts"], st["u"], num_drafts=st["given"])
    return dict(tokens=tokens, accepted=accepted)


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(append=_own_append, decode=_own_decode, prefill=_own_prefill, verify=_own_verify)[op](state)
    return dict(append=_plain_append, decode=_plain_decode, prefill=_plain_prefill, verify=_plain_verify)[op](state)


# ---- the definition in 64 bits -----------------------------------------------------

def _attend64(q, k, v, scale, own_key):
    """softmax(scale q k^T) v over the keys up to each query's own: q [n, heads, d], k [keys, (heads,) d]."""
    shared = k.dim() == 2
    s = torch.einsum("nhd,kd->hnk" if shared else "nhd,khd->hnk", q, k) * scale
    s[:, torch.arange(k.shape[0], device=k.device)[None, :] > own_key[:, None]] = -math.inf
    w = torch.softmax(s, -1)
    return torch.einsum("hnk,kd->nhd" if shared else "hnk,khd->nhd", w, v)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        dc, half = case["latent"], ROT // 2
        first, second = (range(half), range(half, ROT)) if case["pairs"] == "halves" else (range(0, ROT, 2), range(1, ROT, 2))
        first, second = torch.tensor(list(first)).cuda(), torch.tensor(list(second)).cuda()

        def turned(y, pos):
            z = torch.complex(y[..., first], y[..., second])
            z = z * torch.complex(st["cos"].double()[pos], st["sin"].double()[pos]).reshape(pos.shape[0], *[1] * (y.dim() - 2), half)
            out = torch.empty_like(y)
            out[..., first], out[..., second] = z.real, z.imag
            return out

        pos, x = st["pos_of"].long(), st["x"].double()
        row = x.clone()
        row[:, :dc] = st["w"].double() * x[:, :dc] / torch.sqrt((x[:, :dc] ** 2).sum(1, keepdim=True) / dc + EPS)
        row[:, dc:] = turned(x[:, dc:], pos)
        pool, q_out = st["pool"].double(), st["q_out"].double()
        for b in range(case["rows"]):
            mine = st["row_of"] == b
            where = pos[mine]
            pool[st["table"][b, where // case["page"]].long(), 0, where % case["page"]] = row[mine]
        q_out[..., dc:] = turned(st["q"].double()[..., NOPE:], pos)
        return dict(pool=pool, q_out=q_out, **(dict(dense=row) if case["dense"] else {}))
    if case["op"] == "decode":
        t, dc, out = case["tokens"], case["latent"], []
        for b, n in enumerate(st["lens_host"]):
            k = st["pool"][st["table"][b, :-(-n // case["page"])].long(), 0].reshape(-1, dc + ROT)[:n].double()
            out.append(_attend64(st["q"][b].double(), k, k[:, :dc], st["scale"], n - t + torch.arange(t, device="cuda")))
        return torch.stack(out)
    if case["op"] == "prefill":
        out = []
        for b in range(case["rows"]):
            a, e, c, f = st["cu_q_host"][b], st["cu_q_host"][b + 1], st["cu_k_host"][b], st["cu_k_host"][b + 1]
            piece = torch.empty(e - a, case["heads"], VAL, dtype=torch.float64, device="cuda")
            for h in range(case["heads"]):
                kv = st["kv"][c:f, h].double()
                k = torch.cat([kv[:, :NOPE], st["k_rot"][c:f].double()], 1)
                piece[:, h:h + 1] = _attend64(st["q"][a:e, h:h + 1].double(), k, kv[:, NOPE:], st["scale"],
                                              f - c - (e - a) + torch.arange(e - a, device="cuda"))
            out.append(piece)
        return torch.cat(out)
    return None  # whole numbers


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    if case["op"] == "append":
        n, dc, h = case["rows"] * case["tokens"], case["latent"], case["heads"]
        moved = n * 2 * ((2 + bool(case["dense"])) * (dc + ROT) + 2 * h * ROT) + n * 4 * ROT + n * 8
        return dict(bytes=moved, flops=n * (4 * dc + 3 * ROT + 3 * h * ROT))
    if case["op"] == "decode":
        dc, n = case["latent"], case["rows"] * case["tokens"] * case["heads"]
        # rows spread in their logarithm hold hi / ln(hi) keys on average
        keys = case["keys"] if case["lens"] == "flat" else (case["keys"] - 1) / math.log(max(2, case["keys"]))
        keys = max(keys, case["tokens"])
        return dict(bytes=int(case["rows"] * keys * (dc + ROT) * 2 + n * (2 * dc + ROT) * 2),
                    flops=int(2 * n * keys * (2 * dc + ROT)))
    if case["op"] == "prefill":
        new = [max(1, case["tokens"] - (37 * b) % max(1, case["tokens"] // 2 + 1)) for b in range(case["rows"])]
        old = [case["context"] * (b + 1) // case["rows"] for b in range(case["rows"])]
        pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
        tq, tk, h = sum(new), sum(new) + sum(old), case["heads"]
        return dict(bytes=2 * (tq * h * (NOPE + ROT + VAL) + tk * (h * (NOPE + VAL) + ROT)),
                    flops=2 * h * pairs * (NOPE + ROT + VAL))
    size, v = (2 if case["dtype"] == "bf16" else 4), case["vocab"]
    # one distribution of the target (and of the draft where it has one) decides a row
    return dict(bytes=case["rows"] * (v * size * (1 if case["guess"] else 2) + case["drafts"] * 20 + 8),
                flops=case["rows"] * 3 * v)
