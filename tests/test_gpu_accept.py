"""mla_draft_accept against the oracle, which decides in whole numbers of any length: outputs
are whole numbers and have to be equal."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import upkeep

pytestmark = pytest.mark.gpu


def _case(seed, B, K, V, dtype="fp32", sure=False, ragged=False, near=0.8, device="cuda"):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    logits = torch.randn((B, K + 1, V), generator=g) * 3
    q = torch.softmax(logits[:, :K] + near * torch.randn((B, K, V), generator=g), -1).to(dt)
    x = torch.multinomial(q.float().view(B * K, V), 1, generator=g).view(B, K).int() if K else torch.empty((B, 0), dtype=torch.int32)
    c = dict(p=torch.softmax(logits, -1).to(dt), q=None if sure or not K else q, x=x, u=torch.rand((B, K + 1), generator=g),
             counts=torch.randint(-1, K + 1, (B,), generator=g).int() if ragged else None,
             lens=torch.randint(K, 9000, (B,), generator=g).int())
    return {k: v.to(device) if v is not None else None for k, v in c.items()}


def _outputs(B, K, device="cuda"):
    import torch
    return [torch.full(s, -7, dtype=torch.int32, device=device) for s in ((B,), (B, K + 1), (B,))] + [
        torch.zeros(1, dtype=torch.int32, device=device)]


def _call(c, outs, **kw):
    import mla_latent_kv_08_gb300 as mla
    accepted, tokens, new_lens, status = outs
    mla.mla_draft_accept(c["p"], c["x"], c["u"], accepted, tokens, draft_probs=c["q"], draft_counts=c["counts"],
                         seq_lens=c["lens"], new_lens=new_lens if c["lens"] is not None else None, status=status, **kw)


def _floats(t):
    return None if t is None else t.double().cpu().numpy().tolist()


def _want(c):
    ints = {k: None if c[k] is None else c[k].cpu().numpy().tolist() for k in ("x", "counts", "lens")}
    return upkeep.accept(_floats(c["p"]), _floats(c["q"]), ints["x"], _floats(c["u"]), ints["counts"], ints["lens"])


def _check(c, outs):
    want = _want(c)
    accepted, tokens, new_lens, status = (t.cpu().numpy() for t in outs)
    np.testing.assert_array_equal(accepted, [w[1] for w in want])
    np.testing.assert_array_equal(tokens, np.array([w[2] for w in want]).reshape(tokens.shape))
    if c["lens"] is not None:
        np.testing.assert_array_equal(new_lens, [w[3] for w in want])
    assert int(status[0]) == int(np.bitwise_or.reduce([w[0] for w in want]))


def _want_long(c):
    """What the oracle says, row by row in numpy's 64-bit whole numbers: for long rows whose values
    are all in range."""
    B, K1, V = c["p"].shape
    K, out = K1 - 1, []
    x, u = c["x"].cpu().tolist(), c["u"].double().cpu().tolist()
    counts = [K] * B if c["counts"] is None else c["counts"].cpu().tolist()
    lens = [0] * B if c["lens"] is None else c["lens"].cpu().tolist()

    def whole(t):
        return np.rint(t.double().cpu().numpy() * 2.0 ** 46).astype(np.int64)
    for b in range(B):
        if counts[b] < 0:
            out.append((0, 0, [-1] * K1, lens[b]))
            continue
        n = 0
        while n < counts[b] and Fraction(u[b][n]) * (1 if c["q"] is None else Fraction(float(c["q"][b, n, x[b][n]]))) < Fraction(float(c["p"][b, n, x[b][n]])):
            n += 1
        row = whole(c["p"][b, n])
        w = row
        if n < counts[b]:
            less = np.zeros(V, np.int64)
            if c["q"] is None:
                less[x[b][n]] = 2 ** 46
            w = np.maximum(row - (less if c["q"] is None else whole(c["q"][b, n])), 0)
            w = w if w.any() else row
        upto = np.cumsum(w)
        border = Fraction(u[b][K]) * int(upto[-1])
        token = int(np.flatnonzero(w)[-1]) if u[b][K] == 1 else int(np.searchsorted(upto, border.numerator // border.denominator, side="right"))
        out.append((0, n, x[b][:n] + [token] + [-1] * (K - n), lens[b] - K + n))
    return out


def _check_long(c, outs):
    want = _want_long(c)
    accepted, tokens, new_lens, status = (t.cpu().numpy() for t in outs)
    np.testing.assert_array_equal(accepted, [w[1] for w in want])
    np.testing.assert_array_equal(tokens, [w[2] for w in want])
    if c["lens"] is not None:
        np.testing.assert_array_equal(new_lens, [w[3] for w in want])
    assert int(status[0]) == 0


def test_the_long_oracle_is_the_oracle(gpu_lib):
    for sure in (False, True):
        c = _case(40, 6, 3, 700, sure=sure, ragged=True, near=2.0)
        assert [w for w in _want_long(c)] == [w for w in _want(c)]


@pytest.mark.parametrize("sure", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,K,V", [(1, 0, 1), (1, 1, 1), (3, 2, 2), (5, 4, 31), (2, 3, 32), (2, 7, 33), (4, 1, 511), (1, 5, 4097),
                                   (7, 3, 1000), (33, 2, 257), (2, 8, 16385), (1, 256, 40), (300, 1, 65)])
def test_against_the_oracle(gpu_lib, B, K, V, dtype, sure):
    for ragged in (False, True):
        c = _case(B * 1000 + K * 10 + V, B, K, V, dtype, sure, ragged)
        outs = _outputs(B, K)
        _call(c, outs)
        _check(c, outs)


@pytest.mark.parametrize("B", [1, 2, 5, 9, 20, 40, 80, 200])
def test_every_split_of_a_row(gpu_lib, B):
    """The rows of few sequences are split over more CTAs."""
    for dtype in ("fp32", "bf16"):
        c = _case(B, B, 1, 3001, dtype, near=4.0)            # most drafts are refused
        outs = _outputs(B, 1)
        _call(c, outs)
        _check(c, outs)


def test_one_token_has_everything(gpu_lib):
    """The token wherever in the row it is, from every random number."""
    import torch
    V = 5000
    at = [0, 1, 31, 32, 255, 256, 511, 512, 1023, 2500, 4095, 4096, 4998, 4999]
    p = torch.zeros(len(at), 1, V)
    for b, i in enumerate(at):
        p[b, 0, i] = 0.7
    for v in (0.0, 2.0 ** -30, 0.5, 1 - 2.0 ** -24, 1.0):
        c = dict(p=p.cuda(), q=None, x=torch.empty((len(at), 0), dtype=torch.int32, device="cuda"),
                 u=torch.full((len(at), 1), v, device="cuda"), counts=None, lens=None)
        outs = _outputs(len(at), 0)
        _call(c, outs)
        np.testing.assert_array_equal(outs[1].cpu().numpy()[:, 0], at)
        _check(c, outs)


def test_borders(gpu_lib):
    """Sums that the random number meets exactly: the token behind the border. Tokens without
    weight are never drawn."""
    import torch
    p = torch.tensor([0.0, 0.25, 0.0, 0.25, 0.5, 0.0]).expand(6, 1, 6).contiguous()
    u = torch.tensor([0.0, 0.25 - 2.0 ** -26, 0.25, 0.5 - 2.0 ** -25, 0.5, 1.0])
    c = dict(p=p.cuda(), q=None, x=torch.empty((6, 0), dtype=torch.int32, device="cuda"), u=u.view(6, 1).cuda(), counts=None, lens=None)
    outs = _outputs(6, 0)
    _call(c, outs)
    assert outs[1].cpu().view(-1).tolist() == [1, 1, 3, 3, 4, 4]
    _check(c, outs)


def test_the_smallest_random_numbers(gpu_lib):
    """A border of 16 units that a random number of 2^-42 and a bit passes by less than a unit's
    millionth; then random ones down to where every border is 0."""
    import torch
    p = torch.tensor([2.0 ** -42, 1 - 2.0 ** -24, (2 ** 22 - 17) * 2.0 ** -46]).expand(3, 1, 3).contiguous()
    u = torch.tensor([2.0 ** -42, 2.0 ** -42 * (1 + 2.0 ** -23), 2.0 ** -42 * (1 + 2.0 ** -22)])
    c = dict(p=p.cuda(), q=None, x=torch.empty((3, 0), dtype=torch.int32, device="cuda"), u=u.view(3, 1).cuda(), counts=None, lens=None)
    outs = _outputs(3, 0)
    _call(c, outs)
    assert outs[1].cpu().view(-1).tolist() == [0, 1, 1]
    _check(c, outs)
    B, V = 400, 130
    g = torch.Generator().manual_seed(31)
    p = torch.randint(0, 3, (B, 1, V), generator=g).float() * 2.0 ** -46
    p[:, 0, V - 1], p[:, 0, V - 2] = 1 - 2.0 ** -24, 2.0 ** -25
    u = torch.exp2(-torch.randint(38, 62, (B, 1), generator=g).float()) * (1 + torch.rand((B, 1), generator=g))
    u[0], u[1], u[2] = 2.0 ** -149, 2.0 ** -126, 0.0
    c = dict(p=p.cuda(), q=None, x=torch.empty((B, 0), dtype=torch.int32, device="cuda"), u=u.cuda(), counts=None, lens=None)
    outs = _outputs(B, 0)
    _call(c, outs)
    _check(c, outs)


def test_rows_that_add_up_to_two(gpu_lib):
    """As much as a row may: none is refused, however it is split and added."""
    import torch
    for B, V in ((200, 12000), (60, 12000), (3, 70001)):
        g = torch.Generator().manual_seed(B)
        w = torch.rand((B, V), generator=g, dtype=torch.float64) + 1
        p = (w / w.sum(-1, keepdim=True) * 2).float()
        units = (p.double() * 2.0 ** 60).long().sum(-1)      # whole ones: p is above 2^-36
        p[:, 0] = (p[:, 0].double() - (units - 2 ** 61).clamp(min=0).double() * 2.0 ** -60 - 2.0 ** -40).float()
        units = (p.double() * 2.0 ** 60).long().sum(-1)
        assert int(units.max()) <= 2 ** 61 and int(units.min()) > 2 ** 61 - 2 ** 38
        c = dict(p=p.view(B, 1, V).cuda(), q=None, x=torch.empty((B, 0), dtype=torch.int32, device="cuda"),
                 u=torch.rand((B, 1), generator=g).cuda(), counts=None, lens=None)
        outs = _outputs(B, 0)
        _call(c, outs)
        assert int(outs[3]) == 0 and int(outs[1].min()) >= 0
        want = _want_long(c)
        np.testing.assert_array_equal(outs[1].cpu().numpy()[:, 0], [w[2][0] for w in want])


def test_an_equal_product_is_refused(gpu_lib):
    """u q = p exactly, and one unit of u to either side."""
    import torch
    B, p, q = 3, 0.375, 0.75
    c = _case(5, B, 1, 8)
    c["p"], c["q"] = torch.full((B, 2, 8), 0.09, device="cuda"), torch.full((B, 1, 8), 0.03, device="cuda")
    c["x"].fill_(2)
    c["p"][:, 0, 2], c["q"][:, 0, 2] = p, q
    c["u"][:, 0] = torch.tensor([np.nextafter(np.float32(0.5), np.float32(0)), 0.5, np.nextafter(np.float32(0.5), np.float32(1))])
    outs = _outputs(B, 1)
    _call(c, outs)
    assert outs[0].tolist() == [1, 0, 0]
    _check(c, outs)


def test_nothing_left_of_the_difference(gpu_lib):
    """A refused draft (certain to be: its p is 0) where p is nowhere above q: p itself."""
    import torch
    c = _case(6, 4, 2, 300)
    c["q"][:, 0] = c["p"][:, 0]
    c["x"][:, 0] = 7
    c["p"][:, 0, 7] = 0
    c["p"][1, 0] = 0
    c["p"][1, 0, 33] = 1e-30                                 # below 2^-47: no weight at all, an error
    c["q"][1, 0] = 0.001
    outs = _outputs(4, 2)
    _call(c, outs)
    assert outs[0].tolist() == [0, 0, 0, 0] and int(outs[3]) == upkeep.VALUE and outs[1][1].tolist() == [-1] * 3
    _check(c, outs)


def test_small_and_denormal_weights(gpu_lib):
    import torch
    c = _case(7, 6, 1, 900)
    c["p"] = torch.exp2(torch.randint(-70, -10, (6, 2, 900), device="cuda").float()) * (1 + torch.rand(6, 2, 900, device="cuda"))
    c["p"][0, :, ::3] = 1e-42
    c["q"] = torch.exp2(torch.randint(-70, -10, (6, 1, 900), device="cuda").float())
    c["u"][:, 0] = 0.9
    outs = _outputs(6, 1)
    _call(c, outs)
    _check(c, outs)


@pytest.mark.parametrize("what", ["nan", "inf", "negative", "above one", "sum", "token", "low token", "count", "u", "u nan", "last u", "q", "empty", "length"])
def test_values_out_of_range(gpu_lib, what):
    """The sequence that has them is refused with a flag; the others are as ever."""
    import torch
    c = _case(8, 5, 3, 700)
    c["u"][:, :3] = 1.0                                      # the first draft whose p <= q is refused
    c["x"][2] = 11
    c["p"][2, :, 11], c["q"][2, :, 11] = 0.001, 0.002        # of sequence 2, the first
    bad = {"nan": math.nan, "inf": math.inf, "negative": -1e-9, "above one": 1.5}
    if what in bad:
        c["p"][2, 0, 650] = bad[what]
    elif what == "sum":
        c["p"][2, 0, 100:103] = 0.9
    elif what in ("token", "low token"):
        c["x"][2, 2] = 700 if what == "token" else -1
    elif what == "count":
        c["counts"] = torch.tensor([3, 2, 4, 0, -1], dtype=torch.int32, device="cuda")
    elif what in ("u", "u nan"):
        c["u"][2, 1] = 1.0001 if what == "u" else math.nan
    elif what == "last u":
        c["u"][2, 3] = -0.25
    elif what == "q":
        c["q"][2, 0, 0] = math.nan
    elif what == "empty":
        c["p"][2, 0] = 0
    else:
        c["lens"][2] = 2
    outs = _outputs(5, 3)
    _call(c, outs)
    assert outs[1][2].tolist() == [-1] * 4 and int(outs[0][2]) == 0
    assert int(outs[3]) == (upkeep.BOUNDS if what == "length" else upkeep.VALUE)
    _check(c, outs)
    import mla_latent_kv_08_gb300 as mla
    assert mla.mla_read_status_word(outs[3])[0] == (mla.MLA_ERR_BOUNDS if what == "length" else mla.MLA_ERR_VALUE)


def test_what_is_not_read_does_not_count(gpu_lib):
    """NaN in rows that draw nothing, in drafts behind a sequence's count, in its random numbers
    there, and in the vocabulary's padding."""
    import torch
    c = _case(9, 4, 4, 640)
    c["counts"] = torch.tensor([2, 0, -1, 1], dtype=torch.int32, device="cuda")
    c["u"][:, :4] = 0.0
    for b, n in enumerate([2, 0, 0, 1]):                     # all stand: row n alone is read as a whole
        for i in range(5):
            if i != n:
                keep = c["p"][b, i, c["x"][b, i]].clone() if i < n else None
                c["p"][b, i] = math.nan
                if keep is not None:
                    c["p"][b, i, c["x"][b, i]] = keep
        c["x"][b, n:] = 10 ** 6
        c["u"][b, n:4] = math.nan
    c["p"][2] = math.nan
    c["u"][2] = math.nan
    wide = torch.full((4, 5, 700), math.nan, device="cuda")
    wide[:, :, :640] = c["p"]
    c["p"] = wide[:, :, :640]
    outs = _outputs(4, 4)
    _call(c, outs)
    assert outs[0].tolist() == [2, 0, 0, 1] and int(outs[3]) == 0
    _check(c, outs)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_of_a_wider_vocabulary(gpu_lib, dtype):
    import torch
    c = _case(10, 6, 3, 1001, dtype)
    for k, pad in (("p", 1100), ("q", 1023)):
        wide = torch.full((*c[k].shape[:2], pad), 0.5, dtype=c[k].dtype, device="cuda")
        wide[:, :, 5:1006] = c[k]
        c[k] = wide[:, :, 5:1006]
    outs = _outputs(6, 3)
    _call(c, outs)
    _check(c, outs)


def test_lengths_in_place_and_left_out(gpu_lib):
    import torch
    c = _case(11, 40, 3, 400, ragged=True)
    want = _want(c)
    outs = _outputs(40, 3)
    outs[2] = c["lens"]                                      # the lengths themselves
    _call(c, outs)
    np.testing.assert_array_equal(c["lens"].cpu().numpy(), [w[3] for w in want])
    np.testing.assert_array_equal(outs[0].cpu().numpy(), [w[1] for w in want])
    c["lens"] = None
    _call(c, outs)
    np.testing.assert_array_equal(outs[0].cpu().numpy(), [w[1] for w in want])


def test_captured_twice_and_on_two_streams(gpu_lib):
    """Two graphs of different sizes replayed in turn over other inputs, then both calls at once."""
    import torch
    a, b = _case(12, 3, 4, 3000), _case(13, 50, 2, 700, "bf16", sure=True)
    oa, ob = _outputs(3, 4), _outputs(50, 2)
    graphs = []
    for c, o in ((a, oa), (b, ob)):
        _call(c, o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _call(c, o)
        graphs.append(g)
    for seed in (14, 15):
        for c, n in ((a, _case(seed, 3, 4, 3000)), (b, _case(seed, 50, 2, 700, "bf16", sure=True))):
            for k in c:
                if c[k] is not None:
                    c[k].copy_(n[k])
        for o in (oa, ob):
            for t in o[:3]:
                t.fill_(-9)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        _check(a, oa)
        _check(b, ob)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        _call(a, oa, stream=s1)
        _call(b, ob, stream=s2)
    torch.cuda.synchronize()
    _check(a, oa)
    _check(b, ob)


def test_rows_past_32_bits(gpu_lib):
    """256 drafts over five million tokens: the last row begins 5 GB behind the first."""
    import torch
    K, V = 256, 5000003
    p = torch.zeros((1, K + 1, V), device="cuda")
    x = (torch.arange(K, device="cuda") * 19531 + 7).int().view(1, K)
    p[0, torch.arange(K), x[0].long()] = 1.0
    p[0, K, V - 3], p[0, K, 5] = 0.5, 0.5
    for v, token in ((0.25, 5), (0.75, V - 3)):
        c = dict(p=p, q=None, x=x, u=torch.full((1, K + 1), v, device="cuda"), counts=None, lens=None)
        outs = _outputs(1, K)
        _call(c, outs)
        assert int(outs[0]) == K and int(outs[1][0, K]) == token and torch.equal(outs[1][:, :K], x) and int(outs[3]) == 0


def test_a_long_row_captured(gpu_lib):
    """16 CTAs a sequence, asked for while a graph is captured."""
    import torch
    c, o = _case(21, 1, 2, 40000), _outputs(1, 2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(c, o)
    for seed in (22, 23):
        n = _case(seed, 1, 2, 40000)
        for k in c:
            if c[k] is not None:
                c[k].copy_(n[k])
        g.replay()
        torch.cuda.synchronize()
        _check(c, o)


# Sequences and a vocabulary whose warps each have more than 1024 tokens, with 1, 2, 4, 8 and 16 CTAs a
# row; and one whose warps have 800.
LONG = [(160, 8195), (80, 16389), (40, 32771), (13, 65539), (1, 131075), (3, 131075), (2, 102401)]


@pytest.mark.parametrize("sure", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,V", LONG)
def test_long_parts_of_every_split(gpu_lib, B, V, dtype, sure):
    """Every kind of weights in the loop over many tokens at a time: p alone (no drafts, or all stand), the
    difference, p without the draft."""
    for K, near in ((0, 1.0), (1, 4.0)):
        c = _case(B + V, B, K, V, dtype, sure, near=near)
        outs = _outputs(B, K)
        _call(c, outs)
        _check_long(c, outs)
        for v in (0.0, 1 - 2.0 ** -24, 1.0):                 # the first token that has weight, and the last
            c["u"][:, K] = v
            if K:
                c["u"][:, 0] = 1.0
            _call(c, outs)
            _check_long(c, outs)


@pytest.mark.parametrize("B,V", LONG)
def test_long_rows_with_nothing_left(gpu_lib, B, V):
    """p <= q throughout, p = 0 at the draft: the second pass over the row, in p's own weights."""
    for dtype in ("fp32", "bf16"):
        c = _case(V, B, 1, V, dtype)
        c["q"][:, 0] = c["p"][:, 0]
        c["x"][:, 0] = V - 2
        c["p"][:, 0, V - 2] = 0
        outs = _outputs(B, 1)
        _call(c, outs)
        assert not outs[0].any()
        _check_long(c, outs)


@pytest.mark.parametrize("B,V", LONG)
def test_values_out_of_range_deep_in_a_long_row(gpu_lib, B, V):
    """One value of one row, wherever it is: that sequence is refused, the others are as ever."""
    import torch
    c = _case(V + 1, B, 1, V, near=2.0)
    c["u"][:, 0], c["x"][:, 0] = 1.0, 5                      # the draft is refused: both rows are read
    c["p"][:, 0, 5], c["q"][:, 0, 5] = 1e-6, 2e-6
    good, negative_zero = _outputs(B, 1), _outputs(B, 1)
    _call(c, good)
    _check_long(c, good)
    b = B // 2
    for which in ("p", "q"):
        for i in (6, 31, 1023, 1024, V // 2 + 1, V - 1030, V - 1):
            for value in (math.nan, -2.0 ** -140, 1 + 2.0 ** -23):
                keep = c[which][b, 0, i].clone()
                c[which][b, 0, i] = value
                outs = _outputs(B, 1)
                _call(c, outs)
                assert int(outs[3]) == upkeep.VALUE and int(outs[0][b]) == 0 and outs[1][b].tolist() == [-1, -1], (which, i, value)
                rest = torch.arange(B, device="cuda") != b
                assert torch.equal(outs[1][rest], good[1][rest])
                c[which][b, 0, i] = keep
    c["p"][b, 0, V - 7] = c["q"][b, 0, V - 7] = -0.0         # is a probability
    _call(c, negative_zero)
    _check_long(c, negative_zero)


def test_sizes_past_32_bits_are_refused(gpu_lib):
    """A vocabulary of 2^32 + 3: not one of 3."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    for B, K, V in ((1, 0, 2 ** 32 + 3), (2 ** 32 + 1, 0, 1)):
        p = torch.empty((B, K + 1, V), dtype=torch.bfloat16, device="cuda")
        i = torch.zeros((B, K + 1), dtype=torch.int32, device="cuda")
        o = torch.full((B, K + 1), -7, dtype=torch.int32, device="cuda")
        n = torch.full((B,), -7, dtype=torch.int32, device="cuda")
        u = torch.zeros((B, K + 1), device="cuda")
        with pytest.raises(mla.MlaError) as e:
            mla.mla_draft_accept(p, i[:, :K], u, n, o)
        assert e.value.code == mla.MLA_ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert int(n[0]) == -7 and int(o[0, 0]) == -7
        del p, i, o, n, u


def test_the_binding_refuses(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    import torch
    c = _case(16, 3, 2, 50)
    o = _outputs(3, 2)
    good = dict(c)
    for k, v in (("p", c["p"].double()), ("p", c["p"].half()), ("p", c["p"].cpu()), ("p", c["p"][:, :, ::2]), ("p", c["p"][:2]),
                 ("q", c["q"].bfloat16()), ("q", c["q"][:, :1]), ("x", c["x"].long()), ("x", c["x"][:, :1]),
                 ("u", c["u"].double()), ("u", c["u"][:, :2]), ("u", c["u"].T.contiguous().T), ("counts", c["lens"][:2]),
                 ("lens", c["lens"].cpu())):
        with pytest.raises(mla.MlaError) as e:
            _call({**good, k: v}, o)
        assert e.value.code == mla.MLA_ERR_INVALID, k
    torch.cuda.synchronize()
    assert all(int(t.max()) == -7 for t in o[:3])
