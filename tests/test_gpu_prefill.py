"""mla_prefill on the GPU against the decompressed attention in 64 bits.

Tolerances. Keys, values and softmax weights are rounded to bf16 (half a step: 2^-8 of the
value, spread evenly, so a standard deviation below u = 2^-8 / sqrt 3 of it), everything
else is held in 32 bits. A score then has a deviation of at most
    ds = u scale sqrt(sum_j q_j^2 k_j^2)     over the nope dims,
an output sum_t p_t v_t one of sqrt(sum_t p_t^2 ((v_t - out)^2 ds_t^2 + 2 v_t^2 u^2)), and
the output's own rounding adds at most 2^-8 |out|. Held to six deviations (two in 10^9 for
a normal error, and a uniform one never gets there), plus 2e-5 of the largest value for
the 32-bit sums. The fp32 kind has none of the roundings: its bars are the framework's.
"""
import numpy as np
import pytest

import workloads
from oracle import mx as omx
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

U = 2.0 ** -8 / np.sqrt(3.0)


class Case:
    def __init__(self, seed, new, past, H=16, r=512, dR=64, dn=128, dv=128, bs=64, kind="bf16", scale=None):
        rng = np.random.default_rng(seed)
        self.new, self.L = np.array(new), np.array(new) + np.array(past)
        self.H, self.r, self.dR, self.dn, self.dv, self.bs, self.kind = H, r, dR, dn, dv, bs, kind
        self.scale = (dn + dR) ** -0.5 if scale is None else scale

        def f(*shape, std=1.0):
            return workloads.bf16_round((rng.standard_normal(shape) * std).astype(np.float32))
        sigma = np.exp(rng.uniform(np.log(0.1), np.log(3.0), size=r))
        self.lat = [f(L, r, std=sigma) for L in self.L]
        self.rope = [f(L, dR) for L in self.L]
        self.q = f(int(sum(new)), H, dn + dR)
        self.W_UK, self.W_UV = f(H, dn, r, std=r ** -0.5), f(H, r, dv, std=r ** -0.5)
        self.table, self.pool = workloads.make_paging(rng, np.maximum(self.L, 1), bs, spare_blocks=2)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)

    def shape(self, mla, **kw):
        kinds = {"bf16": mla.MLA_KV_BF16, "fp32": mla.MLA_KV_FP32, "mxfp8": mla.MLA_KV_MXFP8}
        return mla.Shape(num_heads=self.H, kv_lora_rank=self.r, rope_dim=self.dR, v_head_dim=self.dv, block_size=self.bs,
                         num_blocks=self.pool, kind=kinds[self.kind], **kw)

    def cache(self, mla, shape, poison=False):
        import torch
        c = mla.Cache.allocate(shape)
        if poison:                         # every slot that no token is written to
            for t, v in ((c.latent, float("nan")), (c.codes, 0x7F), (c.scale_zero, 0xFF), (c.rope, float("nan"))):
                if t is not None:
                    t.fill_(v)
        dt = torch.float32 if self.kind == "fp32" else torch.bfloat16
        cu = np.concatenate([[0], np.cumsum(self.L)]).astype(np.int32)
        if cu[-1]:
            mla.mla_latent_append(c, gu.dev(self.table), gu.dev(np.zeros(len(self.L), np.int32)), gu.dev(cu),
                                  gu.dev(np.concatenate(self.lat), dt),
                                  gu.dev(np.concatenate(self.rope), dt) if self.dR else torch.zeros(8, dtype=dt, device="cuda"))
        return c

    def args(self, mla, shape):
        import torch
        dt = torch.float32 if self.kind == "fp32" else torch.bfloat16
        n = int(self.cu[-1])
        a = dict(block_table=gu.dev(self.table), seq_lens=gu.dev(self.L.astype(np.int32)), cu_q=gu.dev(self.cu),
                 q=gu.dev(self.q, dt), W_UK=gu.dev(self.W_UK, dt), W_UV=gu.dev(self.W_UV, dt), scale=self.scale,
                 out=torch.full((n, self.H, self.dv), 5.0, dtype=dt, device="cuda"),
                 lse=torch.full((n, self.H), 5.0, dtype=torch.float32, device="cuda"))
        a["max_tokens"] = int(sum(L for L, k in zip(self.L, self.new) if k))
        a["workspace"] = mla.alloc_prefill_workspace(shape, len(self.L), n, a["max_tokens"], self.dn)
        return a

    def check(self, out, lse, seqs=None, heads=None, rows=None):
        """Against the definition, at the tolerances above; `rows`: of each sequence's new tokens."""
        for b in range(len(self.L)) if seqs is None else seqs:
            n, L = int(self.new[b]), int(self.L[b])
            if not n:
                continue
            c = (omx.decode(*omx.encode(self.lat[b])) if self.kind == "mxfp8" else self.lat[b]).astype(np.float64)
            kr = self.rope[b].astype(np.float64)
            pick = np.arange(n) if rows is None else np.unique(np.clip(np.asarray(rows), 0, n - 1))
            hidden = np.arange(L) > (L - n + pick)[:, None]
            for h in range(self.H) if heads is None else heads:
                k, v = c @ self.W_UK[h].T.astype(np.float64), c @ self.W_UV[h].astype(np.float64)
                q = self.q[self.cu[b] + pick, h].astype(np.float64)
                s = self.scale * (q[:, :self.dn] @ k.T + q[:, self.dn:] @ kr.T)
                s[hidden] = -np.inf
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                l = e.sum(1, keepdims=True)
                p, want_l = e / l, (m + np.log(l))[:, 0]
                want = p @ v
                got, got_l = out[self.cu[b] + pick, h], lse[self.cu[b] + pick, h]
                if self.kind == "fp32":
                    assert gu.rel_err(got, want) <= gu.FP32_REL_TOL and np.max(np.abs(got_l - want_l)) <= gu.FP32_LSE_TOL, (b, h)
                    continue
                ds2 = (U * self.scale) ** 2 * ((q[:, :self.dn] ** 2) @ (k.T ** 2))
                ds2[hidden] = 0
                p2 = p * p
                a = p2 * ds2                                # sum_t a_t (v - out)^2, expanded
                var = a @ (v * v) - 2 * want * (a @ v) + want ** 2 * a.sum(1, keepdims=True) + 2 * U * U * (p2 @ (v * v))
                tol = 6 * np.sqrt(np.maximum(var, 0)) + 2.0 ** -8 * np.abs(want) + 2e-5 * np.abs(v).max()
                err = np.abs(got - want)
                assert np.all(err <= tol), (b, h, float((err - tol).max()), np.argwhere(~(err <= tol))[:4])
                tol_l = 6 * np.sqrt((p2 * ds2).sum(1)) + 2e-5 * (1 + np.abs(want_l))
                assert np.all(np.abs(got_l - want_l) <= tol_l), (b, h, float((np.abs(got_l - want_l) - tol_l).max()))


def _run(mla, case, shape=None, poison=True, **change):
    import torch
    shape = shape or case.shape(mla)
    cache = case.cache(mla, shape, poison)
    a = case.args(mla, shape)
    a.update(change)
    mla.mla_prefill(cache, **a)
    torch.cuda.synchronize()
    lse = a["lse"].cpu().numpy() if a["lse"] is not None else None
    return a["out"].double().cpu().numpy(), lse, mla.mla_get_status(a["workspace"])


# ------------------------------------------------------------------ numerics

NEW, PAST = [0, 1, 5, 17, 130, 0, 40], [9, 0, 63, 64, 1, 0, 129]


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("impl", [0, 1])
@pytest.mark.parametrize("new,past,H,bs", [
    (NEW, PAST, 4, 64), ([1], [0], 1, 64), ([256, 257], [0, 255], 3, 64), ([128, 127, 129], [128, 1, 0], 2, 16),
    ([600], [700], 2, 256), ([513, 100, 700], [0, 400, 63], 2, 64), ([512, 1, 300], [1, 900, 128], 1, 64), ([2, 2], [1500, 126], 2, 64), ([1] * 40, list(range(40)), 1, 64),
])
def test_latent_512(gpu_lib, kind, impl, new, past, H, bs):
    import mla_latent_kv_08_gb300 as mla
    case = Case(7 + H, new, past, H=H, bs=bs, kind=kind)
    out, lse, status = _run(mla, case, case.shape(mla, impl=impl))
    assert status == (mla.MLA_OK, 0)
    case.check(out, lse)


@pytest.mark.parametrize("kind,r,dR,dn,dv,H,bs", [
    ("fp32", 64, 16, 32, 32, 8, 256), ("fp32", 8, 0, 8, 1, 1, 1), ("bf16", 96, 24, 40, 20, 3, 10), ("bf16", 512, 64, 64, 128, 2, 64),
    ("bf16", 512, 64, 128, 64, 2, 64), ("mxfp8", 160, 8, 16, 300, 2, 7), ("mxfp8", 1024, 128, 512, 1024, 1, 32), ("bf16", 512, 0, 128, 128, 2, 64),
])
def test_other_shapes(gpu_lib, kind, r, dR, dn, dv, H, bs):
    import mla_latent_kv_08_gb300 as mla
    case = Case(90, [3, 20, 70], [0, 33, 5], H=H, r=r, dR=dR, dn=dn, dv=dv, bs=bs, kind=kind)
    out, lse, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0)
    case.check(out, lse)


def test_all_heads_long(gpu_lib):
    """Every head's workspace pass, and rows at both ends of a long chunk."""
    import mla_latent_kv_08_gb300 as mla
    case = Case(91, [1500, 300], [900, 8000], H=128, kind="mxfp8")
    out, lse, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0)
    case.check(out, lse, heads=[0, 31, 77, 127], rows=[0, 1, 127, 128, 255, 256, 299, 700, 1499])


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales(gpu_lib, scale):
    """No, a negative and a large scale (a softmax on one token)."""
    import mla_latent_kv_08_gb300 as mla
    case = Case(92, [150, 9], [30, 400], H=2, scale=scale)
    out, lse, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0)
    case.check(out, lse)


def test_growing_maxima(gpu_lib):
    """Scores that grow along the cache: the running maximum moves at every step."""
    import mla_latent_kv_08_gb300 as mla
    case = Case(93, [300], [700], H=2)
    ramp = np.linspace(0, 60, 1000, dtype=np.float32)[:, None]
    case.rope[0] = workloads.bf16_round(np.abs(case.rope[0]) * 0.1 + ramp / 8)
    case.q[..., case.dn:] = workloads.bf16_round(np.abs(case.q[..., case.dn:]))
    out, lse, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0)
    case.check(out, lse)


def test_without_lse_and_spare_room(gpu_lib):
    """lse may be NULL; num_q and max_tokens may be upper bounds, and rows behind the last stay."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    case = Case(94, [20, 3], [5, 80], H=4)
    shape = case.shape(mla)
    want, lse, _ = _run(mla, case)
    a = case.args(mla, shape)
    q = torch.zeros((40, 4, 192), dtype=torch.bfloat16, device="cuda")
    q[:23] = a["q"]
    out = torch.full((40, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = mla.alloc_prefill_workspace(shape, 2, 40, 1000, 128)
    got, _, status = _run(mla, case, lse=None, q=q, out=out, workspace=ws, max_tokens=1000)
    assert status == (mla.MLA_OK, 0)
    np.testing.assert_array_equal(got[:23], want)
    assert (got[23:] == 3.0).all()


def test_nothing_new(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    case = Case(95, [0, 0], [5, 80], H=4)
    out, lse, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0) and out.shape[0] == 0


# ------------------------------------------------------------------ refusals on the device

@pytest.mark.parametrize("impl", [0, 1])
def test_bad_lengths_and_blocks(gpu_lib, impl):
    import mla_latent_kv_08_gb300 as mla
    case = Case(96, [30, 30, 30, 30], [100, 100, 0, 0], H=2)
    shape = case.shape(mla, impl=impl)
    lens = gu.dev(np.array([130, 130, 29, 10 ** 6], np.int32))          # fewer cached than new; past the table
    table = case.table.copy()
    table[1, 1] = case.pool
    out, lse, (code, flags) = _run(mla, case, shape, seq_lens=lens, block_table=gu.dev(table))
    assert code == mla.MLA_ERR_BOUNDS and flags & 3 == 3
    assert np.isnan(out[30:]).all() and np.isnan(lse[30:]).all()
    case.check(out, lse, seqs=[0])


def test_more_tokens_than_the_workspace(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    case = Case(97, [10, 10, 10], [300, 900, 20], H=2)
    shape = case.shape(mla)
    ws = mla.alloc_prefill_workspace(shape, 3, 30, 310, 128)
    out, lse, (code, flags) = _run(mla, case, workspace=ws, max_tokens=310)
    assert code == mla.MLA_ERR_BOUNDS
    assert np.isnan(out[10:20]).all()
    case.check(out, lse, seqs=[0])


def test_bad_prefix_sums(gpu_lib):
    """Prefix sums that fall, or pass num_q, take their own sequences out and touch nothing else."""
    import mla_latent_kv_08_gb300 as mla
    case = Case(98, [10, 10, 10], [30, 40, 20], H=2)
    out, lse, (code, flags) = _run(mla, case, cu_q=gu.dev(np.array([0, 10, 4, 1000], np.int32)))
    assert code == mla.MLA_ERR_BOUNDS
    assert (out[10:] == 5.0).all() and (lse[10:] == 5.0).all()
    case.check(out, lse, seqs=[0])


def test_capture_and_replay_with_other_lengths(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    import torch
    case = Case(99, [140, 60], [200, 0], H=4, kind="mxfp8")
    shape = case.shape(mla)
    cache, a = case.cache(mla, shape), case.args(mla, shape)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.mla_prefill(cache, **a)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        mla.mla_prefill(cache, **a)
    # the same rows cut another way
    case.new, case.cu = np.array([60, 140]), np.array([0, 60, 200], np.int32)
    case.L = np.array([300, 150])
    case.lat = [case.lat[0][:300], np.zeros((0, 512))]
    a["cu_q"].copy_(torch.from_numpy(case.cu))
    a["seq_lens"].copy_(torch.tensor([300, 0], dtype=torch.int32))       # sequence 1: fewer cached than new
    a["out"].fill_(2.0)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    out, lse = a["out"].double().cpu().numpy(), a["lse"].cpu().numpy()
    case.rope = [case.rope[0][:300], None]
    case.check(out, lse, seqs=[0])
    assert np.isnan(out[60:]).all() and mla.mla_get_status(a["workspace"])[0] == mla.MLA_ERR_BOUNDS


@pytest.mark.parametrize("B", [31, 33, 1023, 1024, 1100])
def test_many_sequences(gpu_lib, B):
    """Numbers of sequences about the plan's warp and block sizes, some without new tokens."""
    import mla_latent_kv_08_gb300 as mla
    new = [(i * 7) % 5 for i in range(B)]
    case = Case(103, new, [i % 40 + (k == 0) for i, k in enumerate(new)], H=1, r=64, dR=16, dn=32, dv=32, bs=16)
    out, lse, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0)
    case.check(out, lse, seqs=sorted({*range(0, B, 37), *range(max(0, B - 80), B)}))


@pytest.mark.parametrize("kind,impl", [("bf16", 0), ("bf16", 1), ("mxfp8", 0), ("mxfp8", 1), ("fp32", 1)])
def test_not_a_number_in_a_later_token(gpu_lib, kind, impl):
    """A cached token with a NaN or an infinity makes the new tokens that see it NaN and leaves
    those before it as they are."""
    import mla_latent_kv_08_gb300 as mla
    case = Case(102, [300, 130, 40, 200, 9], [50, 0, 100, 250, 30], H=3, kind=kind)
    at = [349, 1, 139, 300, 38]                                          # the token, of each sequence
    for b, t in enumerate(at):
        if b < 4:
            case.lat[b][t, [0, 511, 255, 100][b]] = [np.nan, np.inf, -np.inf, np.nan][b]
        else:
            case.rope[b][t, 63] = np.nan
    out, lse, status = _run(mla, case, case.shape(mla, impl=impl))
    assert status == (mla.MLA_OK, 0)
    for b, t in enumerate(at):
        case.lat[b][t], case.rope[b][t] = 0, 0                           # hidden from the rows that are held to it
        n, L = int(case.new[b]), int(case.L[b])
        first = t - (L - n)                                              # the first new token that sees it
        mine = slice(int(case.cu[b]) + first, int(case.cu[b]) + n)
        assert np.isnan(out[mine]).all() and np.isnan(lse[mine]).all(), b
        case.check(out, lse, seqs=[b], rows=np.arange(first))


# ------------------------------------------------------------------ as they are used together

def test_prompt_then_steps(gpu_lib):
    """A server's life of a sequence: prompt appended and prefilled in two chunks, then decode
    steps, drafts verified, the cache read back; all on the 8-bit kind and one cache."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    from oracle import attention
    case = Case(100, [90, 40], [0, 0], H=16, kind="mxfp8")
    shape = case.shape(mla)
    cache = mla.Cache.allocate(shape)
    bf = torch.bfloat16
    table = gu.dev(case.table)

    def append(lo, hi):
        cu = np.concatenate([[0], np.cumsum([h - l for l, h in zip(lo, hi)])]).astype(np.int32)
        mla.mla_latent_append(cache, table, gu.dev(np.array(lo, np.int32)), gu.dev(cu),
                              gu.dev(np.concatenate([c[l:h] for c, l, h in zip(case.lat, lo, hi)]), bf),
                              gu.dev(np.concatenate([c[l:h] for c, l, h in zip(case.rope, lo, hi)]), bf))
    done = [0, 0]
    W_UK, W_UV = gu.dev(case.W_UK, bf), gu.dev(case.W_UV, bf)
    for upto in ([50, 7], [80, 30]):                                     # two chunks of unequal lengths
        append(done, upto)
        rows = np.concatenate([np.arange(case.cu[b] + done[b], case.cu[b] + upto[b]) for b in range(2)])
        cu = np.array([0, upto[0] - done[0], len(rows)], np.int32)
        out = torch.empty((len(rows), 16, 128), dtype=bf, device="cuda")
        lse = torch.empty((len(rows), 16), dtype=torch.float32, device="cuda")
        ws = mla.alloc_prefill_workspace(shape, 2, len(rows), sum(upto), 128)
        mla.mla_prefill(cache, table, gu.dev(np.array(upto, np.int32)), gu.dev(cu), gu.dev(case.q[rows], bf), W_UK, W_UV,
                        case.scale, out, ws, sum(upto), lse=lse)
        torch.cuda.synchronize()
        assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
        part = Case.__new__(Case)
        part.__dict__.update(case.__dict__)
        part.new, part.L, part.cu = np.array(upto) - done, np.array(upto), cu
        part.lat, part.rope, part.q = [c[:u] for c, u in zip(case.lat, upto)], [c[:u] for c, u in zip(case.rope, upto)], case.q[rows]
        part.check(out.double().cpu().numpy(), lse.cpu().numpy())
        done = list(upto)
    stored = [omx.decode(*omx.encode(c)) for c in case.lat]
    for q_len in (1, 3):                                                 # one token, then three drafts
        upto = [d + q_len for d in done]
        q = workloads.bf16_round(np.random.default_rng(q_len).standard_normal((2, q_len, 16, 576)).astype(np.float32))
        append(done, upto)
        out = torch.empty((2, q_len, 16, 128), dtype=bf, device="cuda")
        lse = torch.empty((2, q_len, 16), dtype=torch.float32, device="cuda")
        ws = mla.alloc_workspace(shape, 2, q_len)
        call = mla.mla_decode if q_len == 1 else mla.mla_verify
        call(cache, table, gu.dev(np.array(upto, np.int32)), gu.dev(q, bf), W_UV, case.scale, out, lse, ws)
        for b in range(2):
            ro, rl = attention.absorbed(q[b], stored[b][:upto[b]], case.rope[b][:upto[b]], case.W_UV, case.scale)
            assert gu.rel_err(out[b].float().cpu().numpy(), ro) <= gu.BF16_REL_TOL
            assert np.max(np.abs(lse[b].cpu().numpy() - rl)) <= gu.BF16_LSE_TOL
        done = upto
    rows = torch.empty((sum(done), 576), dtype=bf, device="cuda")
    mla.mla_latent_read(cache, table, gu.dev(np.zeros(2, np.int32)), gu.dev(np.array([0, done[0], sum(done)], np.int32)), rows)
    want = np.concatenate([np.concatenate([stored[b][:done[b]], case.rope[b][:done[b]]], 1) for b in range(2)])
    np.testing.assert_array_equal(rows.double().cpu().numpy(), want)
