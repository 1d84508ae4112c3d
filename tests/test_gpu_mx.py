"""The 8-bit latent cache on the GPU: codes and scales bit-exact against the definition,
reading back exact for every kind, decode and verify over it at the framework's bars
against the attention over what the codes stand for (a bf16 each, so the operands of the
products are exact), and the refusals that the device reports."""
import numpy as np
import pytest

import workloads
from oracle import attention, layout
from oracle import int2 as oint2
from oracle import mx as omx
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _shape(mla, w, **kw):
    s = gu.shape_for(w, kind=mla.MLA_KV_MXFP8)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _workload(seed, lens, H=128, r=512, d_rope=64, d_v=128, block_size=64, q_len=1):
    """Paged sequences of the given lengths; r = 512 with latent directions of unequal variance."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    sigma = np.exp(rng.uniform(np.log(0.1), np.log(3.0), size=r)).astype(np.float32)
    lat = [workloads.bf16_round(rng.standard_normal((L, r)).astype(np.float32) * sigma) for L in lens]
    rope = [workloads.bf16_round(rng.standard_normal((L, d_rope)).astype(np.float32)) for L in lens]
    q = workloads.bf16_round(rng.standard_normal((len(lens), q_len, H, r + d_rope)).astype(np.float32))
    W = workloads.bf16_round((rng.standard_normal((H, r, d_v)) / np.sqrt(r)).astype(np.float32))
    table, pool = workloads.make_paging(rng, lens, block_size, spare_blocks=2)
    return workloads.Workload("mx", "bf16", len(lens), q_len, H, r, d_rope, 128, d_v, (128 + d_rope) ** -0.5, block_size,
                              lens, lat, rope, q, W, table, pool)


def _stored(w):
    """Per sequence: what the cache's codes stand for."""
    return [omx.decode(*omx.encode(c)) for c in w.latent]


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("r,d_rope,bs", [(512, 64, 64), (32, 8, 1), (160, 24, 5), (1024, 128, 16)])
def test_append_bit_exact(gpu_lib, r, d_rope, bs):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(1, [1, 37, 64, 2 * bs], H=2, r=r, d_rope=d_rope, block_size=bs)
    w.latent[1][3, :32] = 0                                             # a group of zeros
    w.latent[1][4, :] *= np.float32(2.0 ** 100)
    w.latent[1][5, :] = workloads.bf16_round(w.latent[1][5, :] * np.float32(2.0 ** -122))
    w.latent[1][6, :] = workloads.bf16_round(np.linspace(-1.75, 1.75, r).astype(np.float32))   # the border 1.75
    w.latent[1][7, 0] = np.float32(3.3895314e38)                        # the largest bf16
    w.latent[1][8, :] = np.float32(-1.7578125)                          # one step past the border
    shape = _shape(mla, w)
    cache = mla.Cache.allocate(shape)
    cache.codes.fill_(0xAA), cache.scale_zero.fill_(0x11)
    st = gu.append_tokens(cache, w, w.latent, w.rope, np.zeros(w.B, np.int32))
    torch.cuda.synchronize()
    assert mla.mla_read_status_word(st)[0] == mla.MLA_OK
    enc = [omx.encode(c) for c in w.latent]
    ref = layout.write_paged(w.num_blocks, bs, r, w.block_table, [e[0] for e in enc], [0] * w.B, np.uint8, 0xAA)
    np.testing.assert_array_equal(cache.codes.cpu().numpy(), ref)
    ref = layout.write_paged(w.num_blocks, bs, r // 32, w.block_table, [e[1] for e in enc], [0] * w.B, np.uint8, 0x11)
    np.testing.assert_array_equal(cache.scale_zero.cpu().numpy(), ref)
    ref = layout.write_paged(w.num_blocks, bs, d_rope, w.block_table, w.rope, [0] * w.B)
    np.testing.assert_array_equal(cache.rope.float().cpu().numpy(), ref)


def test_append_non_finite_groups(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(2, [5], H=1, r=96, d_rope=8, block_size=4)
    w.latent[0][1, 40] = np.inf
    w.latent[0][2, 0] = np.nan
    w.latent[0][3, 95] = -np.inf
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    rows = torch.empty((5, 104), dtype=torch.bfloat16, device="cuda")
    mla.mla_latent_read(cache, gu.dev(w.block_table), gu.dev(np.zeros(1, np.int32)), gu.dev(np.array([0, 5], np.int32)), rows)
    got = rows.float().cpu().numpy()
    want = np.concatenate([_stored(w)[0], w.rope[0]], 1)
    np.testing.assert_array_equal(got, want.astype(np.float32))
    assert np.isnan(got[1, 32:64]).all() and np.isfinite(got[1, :32]).all() and np.isfinite(got[1, 64:]).all()


def test_every_code_reads_back(gpu_lib):
    """All finite codes under scales across the range, exactly."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    finite = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    exps = np.array([-110, -109, -9, -1, 0, 1, 7, 8, 100, 118, 119])
    n = len(exps)
    codes = np.resize(finite, (n, 256))
    shape = mla.Shape(num_heads=1, kv_lora_rank=256, rope_dim=8, v_head_dim=8, block_size=n, num_blocks=1, kind=mla.MLA_KV_MXFP8)
    cache = mla.Cache.allocate(shape)
    cache.codes.copy_(torch.from_numpy(codes)[None])
    scales = np.repeat((exps + 127).astype(np.uint8)[:, None], 8, 1)
    cache.scale_zero.copy_(torch.from_numpy(scales)[None])
    rows = torch.empty((n, 264), dtype=torch.bfloat16, device="cuda")
    mla.mla_latent_read(cache, gu.dev(np.zeros((1, 1), np.int32)), gu.dev(np.zeros(1, np.int32)),
                        gu.dev(np.array([0, n], np.int32)), rows)
    np.testing.assert_array_equal(rows[:, :256].double().cpu().numpy(), omx.decode(codes, scales))


def test_append_flags_a_bad_block(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(3, [70, 10], H=1)
    w.block_table[0, 1] = 10 ** 6
    shape = _shape(mla, w)
    cache = mla.Cache.allocate(shape)
    st = gu.append_tokens(cache, w, w.latent, w.rope, np.zeros(2, np.int32))
    torch.cuda.synchronize()
    assert mla.mla_read_status_word(st)[0] == mla.MLA_ERR_BOUNDS
    got = layout.read_paged(cache.codes.cpu().numpy(), w.block_table[1], 10, 64)
    np.testing.assert_array_equal(got, omx.encode(w.latent[1])[0])


# ------------------------------------------------------------------ reading back

def _rotated(kind, w):
    rng = np.random.default_rng(9)
    d = w.r + w.d_rope if kind == "joint" else w.r
    R = workloads.haar_orthogonal(rng, d).astype(np.float32)
    T = np.full((w.r + w.d_rope) // 32, 4.0, np.float32)
    return R, T


@pytest.mark.parametrize("kind", ["bf16", "bf16+index", "fp32", "mxfp8", "rot", "rot_qr", "joint"])
def test_read_back(gpu_lib, kind):
    """Ranges of sequences, empty ones among them, of every kind; rows behind the last range stay."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(4, [130, 1, 64, 200], H=1)
    kinds = {"bf16": mla.MLA_KV_BF16, "fp32": mla.MLA_KV_FP32, "mxfp8": mla.MLA_KV_MXFP8, "rot": mla.MLA_KV_INT2_ROT,
             "rot_qr": mla.MLA_KV_INT2_ROT_QR, "joint": mla.MLA_KV_INT2_JOINT}
    shape = gu.shape_for(w, kind=kinds[kind.split("+")[0]])
    if kind == "bf16+index":
        shape.index_dim = 8
    R = T = None
    if kind in ("rot", "rot_qr", "joint"):
        R, T = _rotated(kind, w)
    cache, st = gu.fill_cache(w, shape, R, T)
    first, count = [60, 0, 0, 199], [70, 1, 0, 1]
    cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    n = int(cu[-1])
    dt = torch.bfloat16 if kind.startswith("bf16") or kind == "mxfp8" else torch.float32
    rows = torch.full((n + 5, 576), 7.0, dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_latent_read(cache, gu.dev(w.block_table), gu.dev(np.array(first, np.int32)), gu.dev(cu), rows, status=status)
    torch.cuda.synchronize()
    assert mla.mla_read_status_word(status) == (mla.MLA_OK, 0)
    got = rows.float().cpu().numpy()
    assert (got[n:] == 7.0).all()
    if R is None:
        lat = _stored(w) if kind == "mxfp8" else w.latent
        want = [np.concatenate([c, k], 1) for c, k in zip(lat, w.rope)]
    else:
        codes = cache.codes.cpu().numpy()
        sz = cache.scale_zero.cpu().numpy()
        qd = codes.shape[-1] * 4
        want = []
        for b, L in enumerate(w.seq_lens):
            c = layout.read_paged(codes, w.block_table[b], int(L), 64)
            z = layout.read_paged(sz.reshape(*sz.shape[:2], -1), w.block_table[b], int(L), 64).reshape(int(L), -1, 2)
            v = (c[..., None] >> np.array([0, 2, 4, 6])) & 3
            v = v.reshape(int(L), qd).astype(np.float64)
            s, z = (np.repeat(z[..., i].astype(np.float64), 32, 1) for i in (0, 1))
            y = (v * s + z).astype(np.float32)                # exact in fp64, rounded once, as fmaf
            want.append(np.concatenate([y, w.rope[b]], 1) if qd == 512 else y)
    want = np.concatenate([x[f:f + k] for x, f, k in zip(want, first, count)])
    np.testing.assert_array_equal(got[:n], want.astype(np.float32))


def test_read_outside_the_cache_gives_nan_rows(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(5, [130, 100], H=1)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    w.block_table[0, 1] = w.num_blocks                       # one past the pool
    width = w.block_table.shape[1]
    first = np.array([60, width * 64 - 2], np.int32)         # sequence 1 runs past its table (unused entries are -1)
    cu = np.array([0, 10, 15], np.int32)
    rows = torch.zeros((15, 576), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_latent_read(cache, gu.dev(w.block_table), gu.dev(first), gu.dev(cu), rows, status=status)
    assert mla.mla_read_status_word(status)[0] == mla.MLA_ERR_BOUNDS
    bad = torch.isnan(rows).all(1).cpu().numpy()
    np.testing.assert_array_equal(bad, [False] * 4 + [True] * 6 + [True] * 5)


# ------------------------------------------------------------------ decode and verify

def _roomy(w):
    """The same sequences under a block table that has room for long ones: by that room the
    library takes its kernel for few query rows."""
    wide = np.full((w.B, 20000 // w.B + 10), -1, np.int32)
    wide[:, :w.block_table.shape[1]] = w.block_table
    w.block_table = wide
    return w


def _check(w, out, lse, lat, seqs=None):
    for b in range(w.B) if seqs is None else seqs:
        ro, rl = attention.absorbed(w.q[b], lat[b], w.rope[b], w.W_UV, w.scale)
        assert gu.rel_err(out[b], ro) <= gu.BF16_REL_TOL, (b, gu.rel_err(out[b], ro))
        assert np.max(np.abs(lse[b] - rl)) <= gu.BF16_LSE_TOL, (b, np.max(np.abs(lse[b] - rl)))


IMPLS = ["auto", "roomy", "simt"]


def _impl(mla, name):
    return mla.MLA_IMPL_SIMT if name == "simt" else mla.MLA_IMPL_AUTO


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("H,q_len,lens", [(128, 1, [1, 63, 64, 65, 127, 128, 129, 700]), (16, 1, [300, 2]), (20, 3, [3, 130, 64]),
                                          (1, 1, [77]), (128, 2, [513, 2]), (96, 8, [8, 9, 200]),
                                          (32, 1, [1, 64, 128, 400, 2000]), (64, 1, [63, 65, 129, 1500]), (8, 8, [8, 70, 300]),
                                          (4, 8, [130, 9]), (65, 1, [200])])
def test_decode_and_verify(gpu_lib, impl, H, q_len, lens):
    import mla_latent_kv_08_gb300 as mla
    w = _workload(20 + H + q_len, lens, H=H, q_len=q_len)
    if impl == "roomy":
        _roomy(w)
    shape = _shape(mla, w, impl=_impl(mla, impl))
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q, q_len=q_len)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    _check(w, out, lse, _stored(w))


@pytest.mark.parametrize("r,d_rope,d_v,H,bs", [(64, 16, 32, 8, 256), (160, 24, 20, 3, 10), (1024, 128, 128, 2, 64), (512, 64, 64, 16, 64)])
def test_decode_other_shapes(gpu_lib, r, d_rope, d_v, H, bs):
    import mla_latent_kv_08_gb300 as mla
    w = _workload(40, [1, 33, 150], H=H, r=r, d_rope=d_rope, d_v=d_v, block_size=bs)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    _check(w, out, lse, _stored(w))


@pytest.mark.parametrize("H", [32, 128])
@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("splits", [1, 7, 200])
def test_split_count_does_not_matter(gpu_lib, impl, splits, H):
    import mla_latent_kv_08_gb300 as mla
    w = _workload(50, [2100, 64, 900], H=H)
    if impl == "roomy":
        _roomy(w)
    shape = _shape(mla, w, impl=_impl(mla, impl), num_splits_hint=splits)
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    _check(w, out, lse, _stored(w), [0, 2])


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("impl", IMPLS)
def test_stale_slots_are_not_read(gpu_lib, impl, H):
    """NaN codes, scales and rope keys behind a sequence's end (in its last block, and in
    blocks it does not use) leave no trace."""
    import mla_latent_kv_08_gb300 as mla
    w = _workload(51, [1, 63, 65, 190], H=H)
    if impl == "roomy":
        _roomy(w)
    shape = _shape(mla, w, impl=_impl(mla, impl))
    cache = mla.Cache.allocate(shape)
    cache.codes.fill_(0x7F), cache.scale_zero.fill_(0xFF), cache.rope.fill_(float("nan"))
    gu.append_tokens(cache, w, w.latent, w.rope, np.zeros(w.B, np.int32))
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    _check(w, out, lse, _stored(w))


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("H,q_len", [(16, 1), (16, 2), (16, 4), (64, 1), (128, 1), (128, 3), (40, 6)])
def test_not_a_number_in_a_draft(gpu_lib, impl, H, q_len):
    """A cached token with a NaN or an infinity makes the rows that see it NaN and leaves
    those whose mask hides it as they are."""
    import mla_latent_kv_08_gb300 as mla
    lens = [200, 129, 66, 700, 385, 30]
    w = _workload(55, lens, H=H, q_len=q_len)
    if impl == "roomy":
        _roomy(w)
    at = [199, 128 - (q_len > 1), 65, 350, 385 - q_len, None]           # the token, of each sequence
    dim = [0, 511, 255, 100, 290, None]
    for b, (t, d) in enumerate(zip(at, dim)):
        if t is not None:
            w.latent[b][t, d] = [np.nan, np.inf, -np.inf][b % 3]
    w.rope[5][29, 63] = np.nan                                          # and in a rope key
    at[5] = 29
    shape = _shape(mla, w, impl=_impl(mla, impl), num_splits_hint=5)
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q, q_len=q_len)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    for b, (t, L) in enumerate(zip(at, lens)):
        w.latent[b][t], w.rope[b][t] = 0, 0                             # hidden from the rows that are held to it
    lat = _stored(w)
    for b, (t, L) in enumerate(zip(at, lens)):
        sees = L - q_len + np.arange(q_len) >= t
        assert np.isnan(out[b][sees]).all() and np.isnan(lse[b][sees]).all(), b
        if not sees.all():
            ro, rl = attention.absorbed(w.q[b], lat[b], w.rope[b], w.W_UV, w.scale)
            assert gu.rel_err(out[b][~sees], ro[~sees]) <= gu.BF16_REL_TOL, b
            assert np.max(np.abs(lse[b][~sees] - rl[~sees])) <= gu.BF16_LSE_TOL, b


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("impl", IMPLS)
def test_bad_lengths_and_blocks_give_nan_rows(gpu_lib, impl, H):
    import mla_latent_kv_08_gb300 as mla
    w = _workload(52, [200, 300, 100, 70], H=H)
    if impl == "roomy":
        _roomy(w)
    shape = _shape(mla, w, impl=_impl(mla, impl))
    cache, _ = gu.fill_cache(w, shape)
    lat = _stored(w)
    w.block_table[1, 2] = -5
    w.seq_lens = np.array([200, 300, 10 ** 7, 0], np.int32)
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    code, flags = mla.mla_get_status(ws)
    assert code == mla.MLA_ERR_BOUNDS and flags & 3 == 3
    assert np.isnan(out[1:]).all() and np.isnan(lse[1:]).all()
    _check(w, out, lse, lat, [0])


@pytest.mark.parametrize("H,room", [(16, False), (16, True), (128, False)])
@pytest.mark.parametrize("k", [1, 3, 700])
def test_append_decode_is_append_then_decode(gpu_lib, k, H, room):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(53, [900, 800, 1000, 750, 801, 720], H=H)
    if room:
        _roomy(w)
    shape = _shape(mla, w)
    pos = (w.seq_lens - k).astype(np.int32)
    one, _ = gu.fill_cache(w, shape)
    two = mla.Cache.allocate(shape)
    gu.append_tokens(two, w, [c[:-k] for c in w.latent], [c[:-k] for c in w.rope], np.zeros(w.B, np.int32))
    out1, lse1, _ = gu.attend(w, shape, one, w.q)
    bf = torch.bfloat16
    out2 = torch.empty((w.B, 1, w.H, w.d_v), dtype=bf, device="cuda")
    lse2 = torch.empty((w.B, 1, w.H), dtype=torch.float32, device="cuda")
    ws = mla.alloc_workspace(shape, w.B, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_append_decode(two, gu.dev(w.block_table), gu.dev(pos), gu.dev((k * np.arange(w.B + 1)).astype(np.int32)),
                          gu.dev(np.concatenate([c[-k:] for c in w.latent]), bf), gu.dev(np.concatenate([c[-k:] for c in w.rope]), bf),
                          gu.dev(w.seq_lens), gu.dev(w.q, bf), gu.dev(w.W_UV, bf), w.scale, out2, lse2, ws, append_status=st)
    torch.cuda.synchronize()
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0) and mla.mla_read_status_word(st) == (mla.MLA_OK, 0)
    for name in ("codes", "scale_zero"):
        assert torch.equal(getattr(one, name), getattr(two, name)), name
    np.testing.assert_array_equal(out2.float().cpu().numpy(), out1)
    np.testing.assert_array_equal(lse2.cpu().numpy(), lse1)


def test_noalloc_decode(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(54, [500, 90], H=64)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    out1, lse1, _ = gu.attend(w, shape, cache, w.q)
    out = torch.empty((w.B, 1, w.H, w.d_v), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((w.B, 1, w.H), dtype=torch.float32, device="cuda")
    mla.mla_decode_noalloc(cache, gu.dev(w.block_table), gu.dev(w.seq_lens), gu.dev(w.q, torch.bfloat16),
                           gu.dev(w.W_UV, torch.bfloat16), w.scale, out, lse)
    assert gu.rel_err(out.float().cpu().numpy(), out1) <= gu.BF16_REL_TOL
    assert np.max(np.abs(lse.cpu().numpy() - lse1)) <= gu.BF16_LSE_TOL


@pytest.mark.parametrize("H,room", [(128, False), (32, True)])
def test_decode_captured_and_replayed_on_a_side_stream(gpu_lib, H, room):
    """A captured step follows its buffers: new codes and lengths under a replay."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(55, [400, 129], H=H)
    if room:
        _roomy(w)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    bf = torch.bfloat16
    bt, sl, q, W = gu.dev(w.block_table), gu.dev(w.seq_lens), gu.dev(w.q, bf), gu.dev(w.W_UV, bf)
    out = torch.empty((w.B, 1, w.H, w.d_v), dtype=bf, device="cuda")
    lse = torch.empty((w.B, 1, w.H), dtype=torch.float32, device="cuda")
    ws = mla.alloc_workspace(shape, w.B, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.mla_decode(cache, bt, sl, q, W, w.scale, out, lse, ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        mla.mla_decode(cache, bt, sl, q, W, w.scale, out, lse, ws)
    w.seq_lens = np.array([131, 64], np.int32)
    sl.copy_(torch.from_numpy(w.seq_lens))
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    lat = [c[:L] for c, L in zip(_stored(w), w.seq_lens)]
    w.rope = [c[:L] for c, L in zip(w.rope, w.seq_lens)]
    _check(w, out.float().cpu().numpy(), lse.cpu().numpy(), lat)


@pytest.mark.parametrize("H,room", [(32, True), (64, True), (64, False), (128, False)])
def test_maxima_that_keep_rising(gpu_lib, H, room):
    """Scores that grow along the cache: every step raises the running maximum past its bound."""
    import mla_latent_kv_08_gb300 as mla
    w = _workload(56, [1000, 130], H=H)
    if room:
        _roomy(w)
    for b, L in enumerate(w.seq_lens):
        ramp = np.linspace(0, 60, L, dtype=np.float32)[:, None]
        w.rope[b] = workloads.bf16_round(np.abs(w.rope[b]) * np.float32(0.1) + ramp / 8)
    w.q[..., 512:] = workloads.bf16_round(np.abs(w.q[..., 512:]))
    w.q[:, :, ::3, 512:] *= -1                                   # and rows whose scores fall
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    lat = _stored(w)
    for b in range(2):
        ro, rl = attention.absorbed(w.q[b], lat[b], w.rope[b], w.W_UV, w.scale)
        assert gu.rel_err(out[b], ro) <= gu.BF16_REL_TOL
        assert np.max(np.abs(lse[b] - rl)) <= gu.BF16_LSE_TOL


@pytest.mark.parametrize("H,room", [(16, True), (16, False), (64, True), (128, False)])
@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0])
def test_scales_of_either_sign(gpu_lib, H, room, scale):
    import mla_latent_kv_08_gb300 as mla
    w = _workload(57, [200, 65], H=H)
    if room:
        _roomy(w)
    w.scale = scale
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    _check(w, out, lse, _stored(w))


def test_scales_above_one(gpu_lib):
    """Latents whose groups' scales are above 1 and below it take both ways through the expansion."""
    import mla_latent_kv_08_gb300 as mla
    for H, room in ((16, True), (64, True), (128, False)):
        w = _workload(58, [300, 70], H=H)
        if room:
            _roomy(w)
        for c in w.latent:
            c[::7] = workloads.bf16_round(c[::7] * np.float32(2000))
        w.scale = 1e-4
        shape = _shape(mla, w)
        cache, _ = gu.fill_cache(w, shape)
        out, lse, ws = gu.attend(w, shape, cache, w.q)
        assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
        assert int(cache.scale_zero.max()) > 127
        lat = _stored(w)
        for b in range(2):
            ro, rl = attention.absorbed(w.q[b], lat[b], w.rope[b], w.W_UV, w.scale)
            assert gu.rel_err(out[b], ro) <= gu.BF16_REL_TOL
            assert np.max(np.abs(lse[b] - rl)) <= gu.BF16_LSE_TOL


def test_low_scores_on_the_few_row_kernel(gpu_lib):
    """Scores far below 0 at a sequence's start, and a few far above later: both leave the range
    that the few-row kernel takes without looking for maxima."""
    import mla_latent_kv_08_gb300 as mla
    w = _workload(59, [700, 129], H=32)
    w.q[...] = workloads.bf16_round(np.abs(w.q))
    for b, L in enumerate(w.seq_lens):
        w.latent[b] = np.zeros_like(w.latent[b])
        level = np.where(np.arange(L) < 300, -3.0, -1.0).astype(np.float32)
        level[L // 2] = 8.0
        w.rope[b] = workloads.bf16_round(np.repeat(level[:, None], 64, 1) + w.rope[b] * np.float32(0.05))
        w.latent[b][:, :32] = workloads.bf16_round(np.random.default_rng(b).standard_normal((L, 32)).astype(np.float32))
    _roomy(w)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    lat = _stored(w)
    for b in range(2):
        ro, rl = attention.absorbed(w.q[b], lat[b], w.rope[b], w.W_UV, w.scale)
        assert gu.rel_err(out[b], ro) <= gu.BF16_REL_TOL
        assert np.max(np.abs(lse[b] - rl)) <= gu.BF16_LSE_TOL


def test_few_rows_many_sequences(gpu_lib):
    """More sequences than CTAs, so that a CTA takes several work items, of all lengths."""
    import mla_latent_kv_08_gb300 as mla
    w = _workload(60, [1 + 7 * i % 200 for i in range(400)], H=4)
    for room in (True, False):
        if room:
            _roomy(w)
        shape = _shape(mla, w)
        cache, _ = gu.fill_cache(w, shape)
        out, lse, ws = gu.attend(w, shape, cache, w.q)
        assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
        _check(w, out, lse, _stored(w), range(0, 400, 13))
        w = _workload(60, [1 + 7 * i % 200 for i in range(400)], H=4)
