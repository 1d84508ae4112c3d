"""What is measured of the operators that keep a paged latent cache between attention calls,
and their plain forms.

A serving loop verifies drafted tokens, keeps some of them, cuts the sequences back, takes
blocks for the next ones, lets sequences share what they have in common, and now and then
moves the blocks in use to the front of the pool. The operators:

    accept    which drafted tokens stand, by the target's and the draft's probabilities and
              given random numbers, and the token that follows them
    resize    sequences get other lengths: they give blocks back or take free ones
    fork      new sequences begin as others did: they share the full blocks of these, and get
              a block of their own for the tokens behind them
    compact   the blocks in use move to the front of the pool
    copy      the rows that a fork, a cut or a compaction has to move, in the caches of
              many layers

The pool's books are three arrays of 32-bit whole numbers: the block table, the sequences'
lengths, and how many table entries hold each block (0: it is free). Free blocks are taken
lowest first. A case holds plain values; lengths are drawn from its own "lens" seed, so that
they are the same for every seed of the inputs.
"""
import math
import random

import torch

own = False

R, ROPE = 512, 64             # a token's latent and rope key
GROUP = 32                    # values of the 8-bit cache that share a scale


def listed():
    return [
        # one user's answer, a few drafts of a small vocabulary: all latency
        {"name": "accept one", "op": "accept", "B": 1, "K": 4, "V": 32000, "dtype": "fp32", "sure": False, "ragged": False},
        # a batch's drafts are verified, seven behind each sequence's last token
        {"name": "accept batch", "op": "accept", "B": 32, "K": 7, "V": 131072, "dtype": "fp32", "sure": False, "ragged": True},
        # drafts that were looked up, so that their proposal is certain; bf16, rows of odd length
        {"name": "accept looked up", "op": "accept", "B": 64, "K": 3, "V": 50257, "dtype": "bf16", "sure": True, "ragged": True},
        # a decoding step's lengths: a few drafts were refused, or the next ones need room
        {"name": "resize step", "op": "resize", "B": 32, "L": 1024, "L_max": 8192, "bs": 64, "change": "step", "spare": 100, "lens": 1},
        # many sequences over long contexts: some end, some begin, some are cut back far
        {"name": "resize turnover", "op": "resize", "B": 512, "L": 0, "L_max": 65536, "bs": 64, "change": "turnover", "spare": 20000, "lens": 2},
        # four answers to one prompt
        {"name": "fork prompt", "op": "fork", "B": 1, "n": 3, "L": 2000, "L_max": 2000, "bs": 64, "spare": 40, "lens": 3},
        # beams over long documents, each taken several times
        {"name": "fork documents", "op": "fork", "B": 16, "n": 200, "L": 32768, "L_max": 131072, "bs": 64, "spare": 3000, "lens": 4},
        # a small pool with holes
        {"name": "compact small", "op": "compact", "B": 16, "L": 100, "L_max": 3000, "bs": 64, "spare": 150, "lens": 5},
        # a large pool of small blocks, less than half in use, part of them shared
        {"name": "compact large", "op": "compact", "B": 300, "L": 100, "L_max": 16384, "bs": 16, "spare": 200000, "lens": 6},
        # the last blocks of a fork's sequences in one layer
        {"name": "copy tails", "op": "copy", "kind": "bf16", "layers": 1, "n": 8, "rows": 1, "bs": 64, "lens": 7},
        # the same in all layers
        {"name": "copy tails layers", "op": "copy", "kind": "bf16", "layers": 32, "n": 24, "rows": 1, "bs": 64, "lens": 8},
        # whole blocks of the 8-bit cache, as a compaction moves them
        {"name": "copy blocks", "op": "copy", "kind": "mxfp8", "layers": 24, "n": 200, "rows": 64, "bs": 64, "lens": 9},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["accept", "accept", "resize", "fork", "compact", "copy"])
    lens = rng.randrange(1 << 30)
    if op == "accept":
        V, K, bf16 = _log(rng, 500, 200000), rng.randint(0, 8), rng.random() < 0.4
        top = max(1, min(256, (33000000 if not bf16 else 12000000) // (V * (K + 1)), 4000000 // V))
        return {"op": op, "B": _log(rng, 1, top), "K": K, "V": V, "dtype": "bf16" if bf16 else "fp32", "sure": rng.random() < 0.4, "ragged": rng.random() < 0.5}
    bs = rng.choice([16, 32, 64, 64, 128])
    if op == "copy":
        kind, layers = rng.choice(["bf16", "mxfp8"]), _log(rng, 1, 32)
        n = _log(rng, 1, max(1, min(400, 170000 // (layers * bs))))
        return {"op": op, "kind": kind, "layers": layers, "n": n, "rows": rng.choice([1, 1, bs]), "bs": bs, "lens": lens}
    top = _log(rng, 100, 65536)
    L = rng.randint(0, top)
    if op == "fork":
        B = _log(rng, 1, max(1, min(64, 50000 * bs // top)))
        return {"op": op, "B": B, "n": _log(rng, 1, max(1, min(300, 150000 * bs // top))), "L": L, "L_max": top, "bs": bs, "spare": _log(rng, 10, 5000), "lens": lens}
    B = _log(rng, 1, max(1, min(512, 250000 * bs // top)))
    case = {"op": op, "B": B, "L": L, "L_max": top, "bs": bs, "spare": _log(rng, 10, 50000), "lens": lens}
    if op == "resize":
        case["change"] = rng.choice(["step", "turnover"])
    return case


# ------------------------------------------------------------------ lengths

def _cdiv(a, b):
    return -(-a // b)


def _books(case):
    """Lengths of the slots, which sequence a slot shares its first blocks with and how many
    blocks, and what is asked of the pool, as plain lists."""
    r = random.Random(case["lens"])
    B, bs = case["B"], case["bs"]
    lens = [r.randint(case["L"], case["L_max"]) for _ in range(B)]
    if not sum(lens):
        lens[0] = 1
    shared = [0] * B                          # first blocks that are those of the slot before
    for b in range(1, B):
        if r.random() < 0.4:
            shared[b] = r.randint(0, min(lens[b - 1], lens[b]) // bs)
    held = [_cdiv(l, bs) for l in lens]
    used = sum(h - s for h, s in zip(held, shared))
    ask = {}
    if case["op"] == "resize":
        new = []
        for l in lens:
            x = r.random()
            if case["change"] == "step":      # refused drafts go, or the next ones need room
                new.append(max(0, l - r.randint(0, 7)) if x < 0.5 else l + 8)
            elif x < 0.25:
                new.append(0)
            elif x < 0.5:
                new.append(r.randint(0, l))
            else:
                new.append(l + r.randint(0, max(1, case["L_max"] // 8)))
        ask["new"] = new
        room = sum(max(0, _cdiv(n, bs) - h) for n, h in zip(new, held)) + B
        blocks, width = used + room + case["spare"], max(held + [_cdiv(n, bs) for n in new]) + 2
    elif case["op"] == "fork":
        n = case["n"]
        ask["parents"] = [r.randrange(B) for _ in range(n)]
        slots = list(range(B, B + n + 2))     # two slots stay empty
        r.shuffle(slots)
        ask["children"] = slots[:n]
        ask["lens_asked"] = [lens[p] if r.random() < 0.7 else r.randint(0, lens[p]) for p in ask["parents"]]
        lens, shared, held = lens + [0] * (n + 2), shared + [0] * (n + 2), held + [0] * (n + 2)
        blocks, width = used + n + case["spare"], max(held) + 2
    else:
        ask["moves"] = used + 1               # room in the list for every block
        blocks, width = used + case["spare"], max(held) + 2
    return {"lens": lens, "shared": shared, "held": held, "used": used, "blocks": blocks, "width": width, **ask}


def _copies(case):
    """(first row, rows) of every entry."""
    r = random.Random(case["lens"])
    some = [r.randint(case["rows"], case["bs"]) for _ in range(case["n"])]
    return [(r.randint(0, case["bs"] - k) if r.random() < 0.2 else 0, k) for k in some]


def work(case):
    """Each input read once, each output written once."""
    if case["op"] == "accept":
        rows = 1 if case["sure"] or not case["K"] else 2       # the target's row, and the draft's where one was refused
        return {"bytes": case["B"] * (rows * case["V"] * (4 if case["dtype"] == "fp32" else 2) + (case["K"] + 1) * 16), "flops": 0}
    if case["op"] == "copy":
        row = 2 * (R + ROPE) if case["kind"] == "bf16" else R + R // GROUP + 2 * ROPE
        return {"bytes": 2 * row * case["layers"] * sum(k for _, k in _copies(case)), "flops": 0}
    k = _books(case)
    bs, slots = case["bs"], len(k["lens"])
    base = 4 * k["blocks"] + 12 * slots                        # counts; lengths in and out
    if case["op"] == "resize":
        touched = sum(abs(_cdiv(n, bs) - h) for n, h in zip(k["new"], k["held"]))
        return {"bytes": base + touched * 16, "flops": 0}      # an entry and a count, read and written
    if case["op"] == "fork":                                   # a parent's entries once, its blocks' counts read and written
        once = sum(k["held"][p] for p in set(k["parents"]))
        return {"bytes": base + 12 * once + sum(4 * _cdiv(n, bs) + 16 for n in k["lens_asked"]), "flops": 0}
    moved = k["used"] * (k["blocks"] - k["used"]) // k["blocks"]     # blocks lie anywhere: so many behind the first `used`
    return {"bytes": base + 4 * sum(k["held"]) + 32 * moved, "flops": 0}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "accept":
        return _prepare_accept(case, g)
    if case["op"] == "copy":
        return _prepare_copy(case, g)
    return _prepare_pool(case, g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_accept(case, g):
    B, K, V = case["B"], case["K"], case["V"]
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    logits = torch.randn((B, K + 1, V), generator=g, device="cuda") * 3
    near = logits[:, :K] + torch.randn((B, K, V), generator=g, device="cuda") * 0.8      # what the draft model makes of it
    p, q = torch.softmax(logits, -1), torch.softmax(near, -1)
    del logits, near
    if K == 0:
        x = torch.empty((B, 0), dtype=torch.int32, device="cuda")
    elif case["sure"]:                        # the likeliest token, as a lookup that is mostly right has it
        x = p[:, :K].argmax(-1).int()
    else:
        x = torch.multinomial(q.view(B * K, V), 1, generator=g).view(B, K).int()
    s = {"case": case, "p": p.to(dtype), "q": None if case["sure"] or K == 0 else q.to(dtype), "x": x,
         "u": torch.rand((B, K + 1), generator=g, device="cuda"),
         "lens": torch.randint(K + 1, 8192, (B,), generator=g, device="cuda", dtype=torch.int32), "counts": None}
    if case["ragged"]:                        # some sequences have fewer drafts
        s["counts"] = torch.randint(0, K + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if own:
        s.update(accepted=_ints([0] * B), new_lens=_ints([0] * B), tokens=torch.zeros((B, K + 1), dtype=torch.int32, device="cuda"))
    return s


def _prepare_copy(case, g):
    bs, layers, some = case["bs"], case["layers"], _copies(case)
    n = len(some)
    pool = 2 * n + 3
    ids = torch.randperm(pool, generator=g, device="cuda").int()
    copies = torch.zeros((n + 5, 4), dtype=torch.int32, device="cuda")       # the list has room for more
    copies[:n, 0], copies[:n, 1] = ids[:n], ids[n:2 * n]
    copies[:n, 2:] = _ints(some)
    s = {"case": case, "copies": copies, "count": n, "num_copies": _ints([n]), "rows": sum(k for _, k in some)}
    if case["kind"] == "bf16":
        s["planes"] = {"latent": torch.randn((layers, pool, bs, R + ROPE), generator=g, device="cuda", dtype=torch.bfloat16)}
    else:
        values = torch.randn((layers, pool, bs, R), generator=g, device="cuda", dtype=torch.bfloat16) * 50
        s["planes"] = {"codes": values.to(torch.float8_e4m3fn).view(torch.uint8),
                       "scale_zero": torch.randint(100, 130, (layers, pool, bs, R // GROUP), generator=g, device="cuda", dtype=torch.uint8),
                       "rope": torch.randn((layers, pool, bs, ROPE), generator=g, device="cuda", dtype=torch.bfloat16)}
    if own:
        import mla_latent_kv_08_gb300 as mla
        shape = mla.Shape(num_heads=128, kv_lora_rank=R, rope_dim=ROPE, v_head_dim=128, block_size=bs, num_blocks=pool,
                          kind=mla.MLA_KV_BF16 if case["kind"] == "bf16" else mla.MLA_KV_MXFP8)
        s["caches"] = mla.Caches([mla.Cache(shape, **{k: v[i] for k, v in s["planes"].items()}) for i in range(layers)])
    return s


def _prepare_pool(case, g):
    k = _books(case)
    slots, width, blocks, bs = len(k["lens"]), k["width"], k["blocks"], case["bs"]
    # the books lie in one array, so that one copy brings them back: a pass starts from the same ones
    before = torch.empty(slots * width + slots + blocks, dtype=torch.int32, device="cuda")
    s = {"case": case, "before": before, "slots": slots, "width": width, "blocks": blocks}
    table, lens, ref = _views(s, before)
    ids = torch.randperm(blocks, generator=g, device="cuda").int()
    held, shared = _ints(k["held"]), _ints(k["shared"])
    table.fill_(-1)
    lens.copy_(_ints(k["lens"]))
    j = torch.arange(width, device="cuda")
    mine = (j >= shared[:, None]) & (j < held[:, None])
    table[mine] = ids[:k["used"]]
    for b in range(1, slots):                 # in order: what the slot before shares with the one before it
        if k["shared"][b]:
            table[b, :k["shared"][b]] = table[b - 1, :k["shared"][b]]
    ref.copy_(torch.bincount(table[table >= 0].long(), minlength=blocks).int())
    if case["op"] == "resize":
        s["new"], room = _ints(k["new"]), slots
    elif case["op"] == "fork":
        s.update(parents=_ints(k["parents"]), children=_ints(k["children"]), asked=_ints(k["lens_asked"]))
        room = len(k["parents"])
    else:
        room = k["moves"]
    s.update(copies=torch.zeros((room, 4), dtype=torch.int32, device="cuda"), num_copies=_ints([0]), blocks_left=_ints([0]))
    if own:
        import mla_latent_kv_08_gb300 as mla
        shape = mla.Shape(num_heads=128, kv_lora_rank=R, rope_dim=ROPE, v_head_dim=128, block_size=bs, num_blocks=blocks)
        s["now"] = before.clone()
        s["pool"] = mla.Pool(shape, *_views(s, s["now"]))
    return s


def _views(s, books):
    """The books' parts: block table, lengths, counts."""
    n, w = s["slots"], s["width"]
    return books[:n * w].view(n, w), books[n * w:n * w + n], books[n * w + n:]


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"accept": _accept, "resize": _resize, "fork": _fork, "compact": _compact, "copy": _copy}[op](s)


def _own(s, op):
    import mla_latent_kv_08_gb300 as mla
    if op == "accept":
        mla.mla_draft_accept(s["p"], s["x"], s["u"], s["accepted"], s["tokens"], draft_probs=s["q"], draft_counts=s["counts"],
                             seq_lens=s["lens"], new_lens=s["new_lens"])
        return {"accepted": s["accepted"], "tokens": s["tokens"], "new_lens": s["new_lens"]}
    if op == "copy":
        mla.mla_cache_copy(s["caches"], s["copies"], s["num_copies"])
        return _planes(s["planes"])
    s["now"].copy_(s["before"])               # the calls change the books: each pass brings them back, within its time
    if op == "resize":
        mla.mla_pool_resize(s["pool"], s["new"], s["copies"], s["num_copies"], num_free=s["blocks_left"])
    elif op == "fork":
        mla.mla_pool_fork(s["pool"], s["parents"], s["children"], s["copies"], s["num_copies"], lens=s["asked"], num_free=s["blocks_left"])
    else:
        mla.mla_pool_compact(s["pool"], s["copies"], s["num_copies"], num_live=s["blocks_left"])
    return _answer(s, *_views(s, s["now"]), s["copies"], s["num_copies"], s["blocks_left"])


def _answer(s, table, lens, ref, copies, num_copies, blocks_left):
    return {"table": table, "lens": lens, "ref": ref, "copies": copies, "num_copies": num_copies, "blocks_left": blocks_left}


def _planes(planes):
    """8-bit codes as the values they stand for."""
    return {k: v.view(torch.float8_e4m3fn) if k == "codes" else v for k, v in planes.items()}


def _accept(s):
    """In 64 bits: an acceptance is a comparison, and a token's number depends on a long sum."""
    p, q, u = s["p"], s["q"], s["u"].double()
    (B, K1, V), x = p.shape, s["x"].long()
    K = K1 - 1
    counts = torch.full((B,), K, device="cuda") if s["counts"] is None else s["counts"].long()
    px = p[:, :K].gather(-1, x[..., None]).squeeze(-1).double()
    qx = torch.ones_like(px) if q is None else q.gather(-1, x[..., None]).squeeze(-1).double()
    stands = (u[:, :K] * qx < px) & (torch.arange(K, device="cuda") < counts[:, None])
    n = stands.long().cumprod(-1).sum(-1)
    each = torch.arange(B, device="cuda")
    row = p[each, n].double()
    w = row
    if K:
        at = n.clamp(max=K - 1)
        less = q[each, at].double() if q is not None else torch.zeros_like(row).scatter_(-1, x[each, at][:, None], 1.0)
        rest = (row - less).clamp_(min=0)
        w = torch.where((n < counts)[:, None] & (rest.sum(-1, keepdim=True) > 0), rest, row)
    c = w.cumsum(-1)
    token = (c <= u[:, K:] * c[:, -1:]).sum(-1).clamp(max=V - 1)
    i = torch.arange(K1, device="cuda")
    drafts = torch.cat([x, x.new_zeros((B, 1))], -1)
    tokens = torch.where(i < n[:, None], drafts, torch.where(i == n[:, None], token[:, None], -1))
    return {"accepted": n.int(), "tokens": tokens.int(), "new_lens": (s["lens"] - K + n).int()}


def _fresh(ref, need):
    """For every place that needs a block one of the free ones, lowest first."""
    order = torch.argsort((ref != 0).int(), stable=True)
    rank = need.view(-1).long().cumsum(0) - 1
    return order[rank.clamp(0, ref.numel() - 1)].view(need.shape).int()


def _listed(s, ok, src, dst, rows):
    """Entries where `ok`, one behind the other, over the list as it was; and their number."""
    n, room = ok.numel(), s["copies"].shape[0]
    entry = torch.stack([src, dst, torch.zeros_like(src), rows], -1)
    at = torch.where(ok, ok.long().cumsum(0) - 1, room + torch.arange(n, device="cuda")).clamp(max=room + n)
    copies = torch.cat([s["copies"], s["copies"].new_zeros((n + 1, 4))])
    copies[at] = entry
    return copies[:room], ok.sum().int().view(1)


def _resize(s):
    table, lens, ref = _views(s, s["before"])
    bs, new = s["case"]["bs"], s["new"]
    held, wanted = -(-lens // bs), -(-new // bs)
    j = torch.arange(s["width"], device="cuda")
    grow = (j >= held[:, None]) & (j < wanted[:, None])
    cut = (j >= wanted[:, None]) & (j < held[:, None])
    last = table.gather(1, (wanted - 1).clamp(min=0).long()[:, None]).squeeze(1)
    split = (new < lens) & (new % bs > 0) & (ref[last.clamp(min=0).long()] > 1)        # a cut inside a block that others hold
    need = grow | (split[:, None] & (j == wanted[:, None] - 1))
    fresh = _fresh(ref, need)
    change = torch.zeros(ref.numel() + 1, dtype=torch.int32, device="cuda")
    lost = torch.where(cut, table, ref.numel())
    change.index_add_(0, lost.view(-1).long(), torch.full_like(lost.view(-1), -1))
    change.index_add_(0, torch.where(need, fresh, ref.numel()).view(-1).long(), torch.ones_like(fresh.view(-1)))
    change.index_add_(0, torch.where(split, last, ref.numel()).long(), torch.full_like(last, -1))
    counts = ref + change[:-1]
    out = torch.where(need, fresh, torch.where(cut, -1, table))
    tail = out.gather(1, (wanted - 1).clamp(min=0).long()[:, None]).squeeze(1)
    copies, n = _listed(s, split, last, tail, new % bs)
    return _answer(s, out, new.clone(), counts, copies, n, (counts == 0).sum().int().view(1))


def _fork(s):
    table, lens, ref = _views(s, s["before"])
    bs, parents, children, asked = s["case"]["bs"], s["parents"].long(), s["children"].long(), s["asked"]
    full, rest = asked // bs, asked % bs
    j = torch.arange(s["width"], device="cuda")
    rows = table[parents]
    common, tail = j < full[:, None], (j == full[:, None]) & (rest[:, None] > 0)
    fresh = _fresh(ref, tail)
    out = table.clone()
    out[children] = torch.where(common, rows, torch.where(tail, fresh, -1))
    lengths = lens.clone()
    lengths[children] = asked
    change = torch.zeros(ref.numel() + 1, dtype=torch.int32, device="cuda")
    change.index_add_(0, torch.where(common, rows, ref.numel()).view(-1).long(), torch.ones_like(rows.view(-1)))
    change.index_add_(0, torch.where(tail, fresh, ref.numel()).view(-1).long(), torch.ones_like(rows.view(-1)))
    counts = ref + change[:-1]
    at = full.clamp(max=s["width"] - 1).long()[:, None]
    copies, n = _listed(s, rest > 0, rows.gather(1, at).squeeze(1), fresh.gather(1, at).squeeze(1), rest)
    return _answer(s, out, lengths, counts, copies, n, (counts == 0).sum().int().view(1))


def _compact(s):
    table, lens, ref = _views(s, s["before"])
    N = ref.numel()
    used = ref > 0
    live = used.sum()
    i = torch.arange(N, device="cuda", dtype=torch.int32)
    moves, holes = used & (i >= live), ~used & (i < live)
    room = s["copies"].shape[0]
    src, dst = (torch.full((N + 1,), -1, dtype=torch.int32, device="cuda").index_put_((torch.where(m, m.cumsum(0) - 1, N),), i)[:N] for m in (moves, holes))
    n = moves.sum()
    ok = (i < n) & (i < room)                 # the k-th of these goes to the k-th hole
    to = torch.cat([i, i.new_full((1,), -1)])
    to.index_put_((torch.where(ok, src, N).long(),), torch.where(ok, dst, -1))
    counts = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    counts.index_add_(0, to[:N].long(), ref)
    copies, count = _listed(s, ok, src, dst, torch.full_like(src, s["case"]["bs"]))
    return _answer(s, to[torch.where(table < 0, N, table).long()], lens.clone(), counts[:N], copies, count, live.int().view(1))


def _copy(s):
    bs, n = s["case"]["bs"], s["count"]
    src, dst, first, rows = s["copies"][:n].long().unbind(-1)
    e = torch.repeat_interleave(torch.arange(n, device="cuda"), rows, output_size=s["rows"])
    at = torch.arange(s["rows"], device="cuda") - (rows.cumsum(0) - rows)[e] + first[e]
    for plane in s["planes"].values():
        v = plane.view(plane.shape[0], -1, plane.shape[-1])
        v[:, dst[e] * bs + at] = v[:, src[e] * bs + at]
    return _planes(s["planes"])


# ------------------------------------------------------------------ by the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"accept": _exact_accept, "resize": _exact_resize, "fork": _exact_fork, "compact": _exact_compact, "copy": _exact_copy}[case["op"]](s)


def _exact_accept(s):
    p, q, x, u = s["p"], s["q"], s["x"].tolist(), s["u"].double().tolist()
    B, K = p.shape[0], p.shape[1] - 1
    counts = [K] * B if s["counts"] is None else s["counts"].tolist()
    ps = [[p[b, i, x[b][i]].double() for i in range(K)] for b in range(B)]
    ps = torch.stack([v for r in ps for v in r]).tolist() if K else []
    qs = [1.0] * (B * K) if q is None else torch.stack([q[b, i, x[b][i]].double() for b in range(B) for i in range(K)]).tolist()
    accepted, tokens = [], []
    for b in range(B):
        n = 0
        while n < counts[b] and u[b][n] * qs[b * K + n] < ps[b * K + n]:
            n += 1
        row = p[b, n].double()
        w = row
        if n < counts[b]:
            w = row.clone()
            if q is None:
                w[x[b][n]] -= 1
            else:
                w -= q[b, n].double()
            w[w < 0] = 0
            w = w if bool((w > 0).any()) else row
        c = torch.cumsum(w, 0)
        token = torch.searchsorted(c, c[-1:] * u[b][K], right=True)
        accepted.append(n)
        tokens.append(x[b][:n] + [min(int(token), p.shape[2] - 1)] + [-1] * (K - n))
    lens = [l - K + n for l, n in zip(s["lens"].tolist(), accepted)]
    return {"accepted": _ints(accepted), "tokens": _ints(tokens), "new_lens": _ints(lens)}


class _Books:
    """The pool as lists, changed step by step."""

    def __init__(self, s):
        table, lens, ref = _views(s, s["before"])
        self.bs, self.copies = s["case"]["bs"], s["copies"].tolist()
        self.lens, self.ref = lens.tolist(), ref.tolist()
        self.table = [[i for i in row if i >= 0] for row in table.tolist()]
        self.width, self.free, self.n = s["width"], (i for i, c in enumerate(ref.tolist()) if not c), 0

    def take(self):
        i = next(self.free)                   # of those free before the call
        self.ref[i] = 1
        return i

    def note(self, src, dst, rows):
        if self.n < len(self.copies):
            self.copies[self.n] = [src, dst, 0, rows]
            self.n += 1

    def answer(self, left):
        table = [row + [-1] * (self.width - len(row)) for row in self.table]
        return {"table": _ints(table), "lens": _ints(self.lens), "ref": _ints(self.ref), "copies": _ints(self.copies),
                "num_copies": _ints([self.n]), "blocks_left": _ints([left])}


def _exact_resize(s):
    k = _Books(s)
    counts = list(k.ref)
    for b, n in enumerate(s["new"].tolist()):
        row, keep = k.table[b], _cdiv(n, k.bs)
        if n < k.lens[b] and n % k.bs and counts[row[keep - 1]] > 1:
            old = row[keep - 1]
            row[keep - 1] = k.take()
            k.ref[old] -= 1
            k.note(old, row[keep - 1], n % k.bs)
        while len(row) < keep:
            row.append(k.take())
        for i in row[keep:]:
            k.ref[i] -= 1
        del row[keep:]
        k.lens[b] = n
    return k.answer(k.ref.count(0))


def _exact_fork(s):
    k = _Books(s)
    for a, c, n in zip(s["parents"].tolist(), s["children"].tolist(), s["asked"].tolist()):
        full = n // k.bs
        k.table[c] = k.table[a][:full]
        for i in k.table[c]:
            k.ref[i] += 1
        if n % k.bs:
            k.table[c].append(k.take())
            k.note(k.table[a][full], k.table[c][full], n % k.bs)
        k.lens[c] = n
    return k.answer(k.ref.count(0))


def _exact_compact(s):
    k = _Books(s)
    live = sum(c > 0 for c in k.ref)
    high = [i for i, c in enumerate(k.ref) if c and i >= live]
    to = {}
    for src, dst in zip(high, k.free):
        to[src] = dst
        k.note(src, dst, k.bs)
        k.ref[dst], k.ref[src] = k.ref[src], 0
    k.table = [[to.get(i, i) for i in row] for row in k.table]
    return k.answer(live)


def _exact_copy(s):
    bs = s["case"]["bs"]
    out = {k: v.clone() if k == "scale_zero" else v.double() for k, v in _planes(s["planes"]).items()}
    for src, dst, first, rows in s["copies"][:s["count"]].tolist():
        for k, v in out.items():
            v[:, dst, first:first + rows] = _planes(s["planes"])[k][:, src, first:first + rows].to(v.dtype)
    return out
