"""What is measured of the operators around an 8-bit latent cache, and their plain forms.

The cache keeps, for each token, a latent of r values and a rope key of d_R values that
every head shares. Its 8-bit kind holds the latent as e4m3 codes with one power-of-two
scale for every 32 values, and the rope key in bf16. The operators:

    append    new tokens' latents are quantised as they are written into the paged cache
    read      cached tokens of many sequences are read back as dense bf16 rows
    decode    one new token a sequence attends over its cached tokens, in latent space
    verify    a few draft tokens a sequence do, each seeing its predecessors
    prefill   chunks of new tokens, of any length, attend over what is cached before them
              and over one another, with per-head keys and values made from the latents

A case holds plain values. Lengths of sequences are drawn from its own "lens" seed, so
that they are the same for every seed of the inputs.
"""
import math
import random

import torch

own = False

GROUP = 32                    # values that share a scale
R, ROPE, NOPE, DV = 512, 64, 128, 128
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
BLOCK = 64


def listed():
    return [
        # one decoding step of a batch: the call is all latency
        {"name": "append step", "op": "append", "B": 32, "new": 1, "new_max": 1, "past": 0, "past_max": 8000, "lens": 1},
        # prompts of many lengths enter the cache
        {"name": "append prompts", "op": "append", "B": 24, "new": 64, "new_max": 4096, "past": 0, "past_max": 300, "lens": 2},
        # a few short prefixes, of one token upwards, are looked at again
        {"name": "read short", "op": "read", "kind": "mxfp8", "B": 5, "L": 1, "L_max": 333, "lens": 3},
        # a batch's whole context is read back
        {"name": "read batch", "op": "read", "kind": "mxfp8", "B": 32, "L": 1024, "L_max": 8192, "lens": 4},
        # one user at the start of an answer
        {"name": "decode one", "op": "decode", "B": 1, "H": 128, "q_len": 1, "L": 90, "L_max": 200, "lens": 5},
        # the framework's headline batch: 32 sequences of 1k to 8k tokens, all heads
        {"name": "decode batch", "op": "decode", "B": 32, "H": 128, "q_len": 1, "L": 1024, "L_max": 8192, "lens": 6},
        # two long documents on half the heads
        {"name": "decode long", "op": "decode", "B": 2, "H": 64, "q_len": 1, "L": 32768, "L_max": 131072, "lens": 7},
        # speculative drafts of eight tokens are verified
        {"name": "verify drafts", "op": "decode", "B": 16, "H": 128, "q_len": 8, "L": 4096, "L_max": 32768, "lens": 8},
        # short turns of a chat, some sequences with nothing new
        {"name": "prefill turns", "op": "prefill", "kind": "mxfp8", "B": 6, "H": 128, "new": 0, "new_max": 200, "past": 0, "past_max": 300, "lens": 9},
        # whole prompts with nothing before them
        {"name": "prefill prompts", "op": "prefill", "kind": "mxfp8", "B": 4, "H": 128, "new": 1024, "new_max": 4096, "past": 0, "past_max": 0, "lens": 10},
        # the same on an eighth of the heads, over what is cached already
        {"name": "prefill some heads", "op": "prefill", "kind": "mxfp8", "B": 8, "H": 16, "new": 100, "new_max": 2000, "past": 0, "past_max": 4096, "lens": 11},
        # the next chunks of two long documents, bf16 cache
        {"name": "prefill chunks", "op": "prefill", "kind": "bf16", "B": 2, "H": 128, "new": 2048, "new_max": 2048, "past": 8192, "past_max": 24576, "lens": 12},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "verify", "prefill", "prefill"])
    lens = rng.randrange(1 << 30)
    if op == "append":
        new_max = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, 100000 // new_max)))
        return {"op": op, "B": B, "new": rng.randint(0, new_max), "new_max": new_max, "past": 0, "past_max": _log(rng, 1, 4000), "lens": lens}
    if op == "read":
        top = _log(rng, 8, 32768)
        return {"op": op, "kind": rng.choice(["mxfp8", "mxfp8", "bf16"]), "B": _log(rng, 1, max(1, min(64, 150000 // top))),
                "L": rng.randint(0, top), "L_max": top, "lens": lens}
    if op in ("decode", "verify"):
        q_len = 1 if op == "decode" else rng.randint(2, 8)
        top = _log(rng, 16, 65536)
        H = rng.choice([8, 16, 20, 32, 64, 96, 128, 128])
        return {"op": "decode", "B": _log(rng, 1, max(1, min(64, 250000 // top))), "H": H, "q_len": q_len, "L": rng.randint(q_len, top), "L_max": top, "lens": lens}
    new_max = _log(rng, 1, 4096)
    past_max = rng.choice([0, _log(rng, 16, 16384)])
    H = rng.choice([8, 16, 20, 32, 64, 128])
    B = _log(rng, 1, max(1, min(16, 16000000 // (new_max * (new_max + past_max) + 1), 40000 // (new_max + past_max))))
    return {"op": op, "kind": rng.choice(["mxfp8", "bf16"]), "B": B, "H": H, "new": rng.randint(0, new_max), "new_max": new_max,
            "past": rng.randint(0, past_max), "past_max": past_max, "lens": lens}


def _lengths(case):
    """(cached tokens with the new ones, new tokens) of each sequence."""
    r = random.Random(case["lens"])
    if "L" in case:
        L = [r.randint(case["L"], case["L_max"]) for _ in range(case["B"])]
        return L, [case.get("q_len", 0)] * case["B"]
    new = [r.randint(case["new"], case["new_max"]) for _ in range(case["B"])]
    if not sum(new):
        new[0] = 1
    return [n + r.randint(case["past"], case["past_max"]) for n in new], new


def work(case):
    """Each input read once, each output written once; the fewer of the two forms' multiplications."""
    L, new = _lengths(case)
    row = R + R // GROUP + 2 * ROPE if case.get("kind", "mxfp8") == "mxfp8" else 2 * (R + ROPE)
    dense = 2 * (R + ROPE)
    if case["op"] == "append":
        return {"bytes": sum(new) * (dense + row), "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(L) * (dense + row), "flops": 0}
    H = case["H"]
    pairs = [n * l - n * (n - 1) // 2 for l, n in zip(L, new)]     # (new token, cached token) that it sees
    if case["op"] == "decode":
        rows = sum(new) * H
        return {"bytes": sum(L) * row + rows * (2 * (R + ROPE) + 2 * DV + 4) + H * R * DV * 2,
                "flops": 2 * H * sum(pairs) * (2 * R + ROPE) + 2 * rows * R * DV}
    flops = 0
    for l, n, p in zip(L, new, pairs):
        heads = 2 * l * R * (NOPE + DV) + 2 * p * (NOPE + ROPE + DV)       # keys and values made for each head
        latent = 2 * n * R * (NOPE + DV) + 2 * p * (2 * R + ROPE)          # in latent space
        flops += H * min(heads, latent) if n else 0
    used = sum(l for l, n in zip(L, new) if n)
    return {"bytes": used * row + sum(new) * H * 2 * (NOPE + ROPE + DV) + H * R * (NOPE + DV) * 2, "flops": flops}


# ------------------------------------------------------------------ inputs

def _quantise(c):
    """The latents' e4m3 codes (as bytes) and their scales' biased exponents. The scale of a
    group is the least power of two, from 2^-110 to 2^119, that brings its largest magnitude to
    448 or less; what 2^119 leaves above that becomes 448."""
    g = c.float().unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(g.abs().amax(-1))                 # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, -110, e.clamp(-110, 119))
    codes = torch.ldexp(g, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, GROUP))
    return torch.ldexp(v, (scales.int() - 127)[..., None]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(bf16)

    def latents(n):              # the latent's directions differ widely in variance
        sigma = torch.exp(torch.rand(R, generator=g, device="cuda") * math.log(30.0)) * 0.1
        return (torch.randn((n, R), generator=g, device="cuda") * sigma).to(bf16)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    L, new = _lengths(case)
    B = case["B"]
    blocks = [-(-l // BLOCK) for l in L]
    pool, width = sum(blocks) + 3, max(1, max(blocks))
    ids = torch.randperm(pool, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = ids[at:at + n]
        at += n
    s = {"case": case, "table": table, "L": ints(L), "B": B, "pool": pool, "tokens": sum(L), "lengths": L, "new": new,
         "kind": case.get("kind", "mxfp8")}
    if case["op"] == "append":
        past = [l - n for l, n in zip(L, new)]
        s.update(c=latents(sum(new)), k=normal(sum(new), ROPE), past=ints(past),
                 cu=ints([sum(new[:b]) for b in range(B + 1)]),
                 seq=torch.repeat_interleave(torch.arange(B, device="cuda"), ints(new).long()),
                 codes=torch.zeros((pool, BLOCK, R), dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros((pool, BLOCK, R // GROUP), dtype=torch.uint8, device="cuda"),
                 rope=torch.zeros((pool, BLOCK, ROPE), dtype=bf16, device="cuda"))
        return s
    # every slot of the pool holds some token, also those behind a sequence's end
    c = latents(pool * BLOCK)
    if s["kind"] == "mxfp8":
        codes, scales = _quantise(c)
        s.update(codes=codes.view(pool, BLOCK, R), scales=scales.view(pool, BLOCK, R // GROUP), rope=normal(pool, BLOCK, ROPE))
    else:
        s["latent"] = torch.cat([c, normal(pool * BLOCK, ROPE)], -1).view(pool, BLOCK, R + ROPE)
    if case["op"] == "read":
        s.update(first=ints([0] * B), cu=ints([sum(L[:b]) for b in range(B + 1)]),
                 seq=torch.repeat_interleave(torch.arange(B, device="cuda"), s["L"].long()))
        return s
    H = case["H"]
    s["W_UV"] = normal(H, R, DV, std=R ** -0.5)
    if case["op"] == "decode":
        s["q"] = normal(B, case["q_len"], H, R + ROPE)
    else:
        s.update(q=normal(sum(new), H, NOPE + ROPE), W_UK=normal(H, NOPE, R, std=R ** -0.5),
                 cu=ints([sum(new[:b]) for b in range(B + 1)]))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"append": _append, "read": _read, "decode": _decode, "prefill": _prefill}[op](s)


def _own(s, op):
    import mla_latent_kv_08_gb300 as mla
    H = s["case"].get("H", 1)
    shape = mla.Shape(num_heads=H, kv_lora_rank=R, rope_dim=ROPE, v_head_dim=DV, block_size=BLOCK, num_blocks=s["pool"],
                      kind=mla.MLA_KV_MXFP8 if s["kind"] == "mxfp8" else mla.MLA_KV_BF16)
    if s["kind"] == "mxfp8":
        cache = mla.Cache(shape, codes=s["codes"], scale_zero=s["scales"], rope=s["rope"])
    else:
        cache = mla.Cache(shape, latent=s["latent"])
    if op == "append":
        mla.mla_latent_append(cache, s["table"], s["past"], s["cu"], s["c"], s["k"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"], "rope": s["rope"]}
    if op == "read":
        rows = torch.empty((s["tokens"], R + ROPE), dtype=torch.bfloat16, device="cuda")
        mla.mla_latent_read(cache, s["table"], s["first"], s["cu"], rows)
        return rows
    q = s["q"]
    if op == "decode":
        if "workspace" not in s:
            s["workspace"] = mla.alloc_workspace(shape, s["B"], q.shape[1])
        out = torch.empty((*q.shape[:3], DV), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
        call = mla.mla_decode if q.shape[1] == 1 else mla.mla_verify
        call(cache, s["table"], s["L"], q, s["W_UV"], SCALE, out, lse, s["workspace"])
        return {"out": out, "lse": lse}
    if "workspace" not in s:
        s["workspace"] = mla.alloc_prefill_workspace(shape, s["B"], q.shape[0], s["tokens"], NOPE)
    out = torch.empty((q.shape[0], H, DV), dtype=torch.bfloat16, device="cuda")
    mla.mla_prefill(cache, s["table"], s["L"], s["cu"], q, s["W_UK"], s["W_UV"], SCALE, out, s["workspace"], max_tokens=s["tokens"])
    return out


def _slots(s, seq, pos):
    """Token rows of the pool that hold positions `pos` of sequences `seq`."""
    return s["table"][seq, pos // BLOCK].long() * BLOCK + pos % BLOCK


def _append(s):
    n = torch.arange(s["c"].shape[0], device="cuda")
    at = _slots(s, s["seq"], n - s["cu"][s["seq"]] + s["past"][s["seq"]])
    codes, scales = _quantise(s["c"])
    s["codes"].view(-1, R)[at] = codes
    s["scales"].view(-1, R // GROUP)[at] = scales
    s["rope"].view(-1, ROPE)[at] = s["k"]
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"], "rope": s["rope"]}


def _rows(s, at):
    """The pool's token rows `at`, in 32 bits: latent, then rope key."""
    if s["kind"] != "mxfp8":
        return s["latent"].view(-1, R + ROPE)[at].float()
    return torch.cat([_values(s["codes"].view(-1, R)[at], s["scales"].view(-1, R // GROUP)[at]), s["rope"].view(-1, ROPE)[at].float()], -1)


def _read(s):
    n = torch.arange(s["tokens"], device="cuda")
    return _rows(s, _slots(s, s["seq"], n - s["cu"][s["seq"]] + s["first"][s["seq"]])).to(torch.bfloat16)


def _decode(s):
    q, B = s["q"].float(), s["B"]
    n, H = q.shape[1], q.shape[2]
    top = max(s["lengths"])
    pos = torch.arange(top, device="cuda")
    seen = pos < s["L"][:, None] - n + 1 + torch.arange(n, device="cuda")[:, None, None]       # [n, B, top]
    rows = _rows(s, _slots(s, torch.arange(B, device="cuda")[:, None], pos.minimum(s["L"][:, None] - 1)))
    x = torch.bmm(q.view(B, n * H, R + ROPE), rows.transpose(1, 2)).view(B, n, H, top).mul_(SCALE)
    x.masked_fill_(~seen.transpose(0, 1)[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B, n * H, top), rows[..., :R]).view(B, n, H, R) / l
    out = torch.einsum("bnhr,hrv->bnhv", o, s["W_UV"].float())
    return {"out": out.to(torch.bfloat16), "lse": (m + l.log()).squeeze(-1)}


def _prefill(s):
    q, H = s["q"], s["q"].shape[1]
    out = torch.empty((q.shape[0], H, DV), dtype=torch.bfloat16, device="cuda")
    first = 0
    for b, (l, n) in enumerate(zip(s["lengths"], s["new"])):
        if not n:
            continue
        pos = torch.arange(l, device="cuda")
        rows = _rows(s, _slots(s, b, pos))
        some = max(1, min(H, (1 << 29) // (n * l)))       # heads at a time: all heads' scores can fill the memory
        hidden = pos > l - n + torch.arange(n, device="cuda")[:, None]
        for h in range(0, H, some):
            k = torch.matmul(rows[:, :R], s["W_UK"][h:h + some].float().transpose(1, 2))
            v = torch.matmul(rows[:, :R], s["W_UV"][h:h + some].float())
            x = q[first:first + n, h:h + some].float().transpose(0, 1)
            y = torch.matmul(x[..., :NOPE], k.transpose(1, 2)) + torch.matmul(x[..., NOPE:], rows[:, R:].T)
            y.mul_(SCALE).masked_fill_(hidden, -math.inf)
            p = y.sub_(y.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
            out[first:first + n, h:h + some] = o.transpose(0, 1).to(torch.bfloat16)
        first += n
    return out


# ------------------------------------------------------------------ in 64 bits

def _table64():
    """The 256 values of e4m3 by its definition: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    v = []
    for code in range(256):
        e, f = code >> 3 & 15, code & 7
        x = math.ldexp(f / 8, -6) if e == 0 else math.ldexp(1 + f / 8, e - 7)
        v.append(math.nan if code & 127 == 127 else -x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _cached64(s, b, l):
    """Latents and rope keys of the first l tokens of sequence b, block by block."""
    blocks = s["table"][b, :-(-l // BLOCK)].long()
    if s["kind"] != "mxfp8":
        both = s["latent"][blocks].double().reshape(-1, R + ROPE)[:l]
        return both[:, :R], both[:, R:]
    c = _table64()[s["codes"][blocks].reshape(-1, R)[:l].long()]
    scale = torch.exp2(s["scales"][blocks].reshape(-1, R // GROUP)[:l].double() - 127)
    return c * scale.repeat_interleave(GROUP, -1), s["rope"][blocks].reshape(-1, ROPE)[:l].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(s)
    if op == "read":
        parts = [torch.cat(_cached64(s, b, l), -1) for b, l in enumerate(s["lengths"])]
        return torch.cat(parts)
    outs, lses, at = [], [], 0
    for b, (l, n) in enumerate(zip(s["lengths"], s["new"])):
        if not n:
            continue
        c, k = _cached64(s, b, l)
        late = torch.arange(l, device="cuda") > torch.arange(l - n, l, device="cuda")[:, None]
        o, e = [], []
        for h in range(case["H"]):
            w_uv = s["W_UV"][h].double()
            if op == "decode":
                q = s["q"][b, :, h].double()
                x = q[:, :R] @ c.T
            else:
                q = s["q"][at:at + n, h].double()
                x = (q[:, :NOPE] @ s["W_UK"][h].double()) @ c.T if n < l / 4 else q[:, :NOPE] @ (c @ s["W_UK"][h].double().T).T
            x = ((x + q[:, -ROPE:] @ k.T) * SCALE).masked_fill(late, -math.inf)
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[:, None])
            o.append((p @ c) @ w_uv if n < l / 4 else p @ (c @ w_uv))
            e.append(lse)
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(e, 1))
        at += n
    if op == "decode":
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    return torch.cat(outs)


def _exact_append(s):
    """Codes' values and rope keys in place; the scales, whole numbers, are compared as such."""
    values = torch.zeros(s["codes"].shape, dtype=torch.float64, device="cuda").view(-1, R)
    rope = torch.zeros(s["rope"].shape, dtype=torch.float64, device="cuda").view(-1, ROPE)
    c = s["c"].double()
    for b in range(s["B"]):
        lo, hi = int(s["cu"][b]), int(s["cu"][b + 1])
        pos = torch.arange(hi - lo, device="cuda") + int(s["past"][b])
        at = s["table"][b, pos // BLOCK].long() * BLOCK + pos % BLOCK
        g = c[lo:hi].reshape(-1, R // GROUP, GROUP)
        e = torch.ceil(torch.log2(g.abs().amax(-1, keepdim=True) / 448)).clamp(-110, 119)
        values[at] = (g * torch.exp2(-e)).clamp(-448, 448).reshape(-1, R)
        rope[at] = s["k"][lo:hi].double()
    return {"codes": values.view(s["codes"].shape), "scales": None, "rope": rope.view(s["rope"].shape)}
