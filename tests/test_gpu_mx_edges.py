"""Decode, verify and reading of the 8-bit cache at the ends of their ranges. Tolerances are
the framework's bars for bf16 caches, but for what is exact."""
import numpy as np
import pytest

from oracle import attention
from tests import gpu_util as gu
from tests.test_gpu_mx import IMPLS, _impl, _roomy, _shape, _stored, _workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,q_len,blocks", [(64, 1, 625000), (16, 4, 2200000), (128, 1, 625000), (32, 2, 1100001)])
def test_tokens_times_heads_past_31_bits(gpu_lib, H, q_len, blocks):
    """A table that repeats two blocks of the cache, the first one over the sequence's oldest
    eighth: as the softmax over their 128 tokens, each counted as often as it stands there."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(80 + H, [128], H=H, q_len=q_len)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    a, b = (int(x) for x in w.block_table[0, :2])
    L = 64 * blocks
    assert (L - q_len) * H > 2 ** 31
    old = blocks // 8
    table = np.full((1, blocks), b, np.int32)
    table[0, :old] = a
    bf = torch.bfloat16
    out = torch.empty((1, q_len, H, 128), dtype=bf, device="cuda")
    lse = torch.empty((1, q_len, H), dtype=torch.float32, device="cuda")
    ws = mla.alloc_workspace(shape, 1, q_len)
    call = mla.mla_decode if q_len == 1 else mla.mla_verify
    call(cache, gu.dev(table), gu.dev(np.array([L], np.int32)), gu.dev(w.q, bf), gu.dev(w.W_UV, bf), w.scale, out, lse, ws)
    torch.cuda.synchronize()
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    c = _stored(w)[0]
    s = w.scale * w.q[0].astype(np.float64) @ np.concatenate([c, w.rope[0].astype(np.float64)], 1).T        # [q_len, H, 128]
    count = np.repeat([[old] * 64 + [blocks - old] * 64], q_len, 0).astype(np.float64)
    for i in range(q_len):
        count[i, 128 - (q_len - 1 - i):] -= 1                    # hidden from this draft's row
    m = s.max(-1, keepdims=True)
    e = count[:, None, :] * np.exp(s - m)
    l = e.sum(-1, keepdims=True)
    want = np.einsum("qhr,hrv->qhv", e / l @ c, w.W_UV.astype(np.float64))
    assert gu.rel_err(out[0].float().cpu().numpy(), want) <= gu.BF16_REL_TOL
    assert np.max(np.abs(lse[0].cpu().numpy() - (m + np.log(l))[..., 0])) <= gu.BF16_LSE_TOL


@pytest.mark.parametrize("kind,H", [("mxfp8", 16), ("mxfp8", 128), ("bf16", 128)])
@pytest.mark.parametrize("over", [0, 254])
def test_a_length_at_the_end_of_31_bits_is_refused(gpu_lib, kind, H, over):
    """2^31 - 255 tokens and more, under a table with room for them: the flag and NaN rows; the
    sequence beside it as it is."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(84, [64, 70], H=H)
    shape = _shape(mla, w, kind=mla.MLA_KV_MXFP8 if kind == "mxfp8" else mla.MLA_KV_BF16)
    cache, _ = gu.fill_cache(w, shape)
    table = torch.full((2, 2 ** 25), -1, dtype=torch.int32, device="cuda")
    table[0] = int(w.block_table[0, 0])
    table[1, :2] = gu.dev(w.block_table[1, :2])
    bf = torch.bfloat16
    out = torch.empty((2, 1, H, 128), dtype=bf, device="cuda")
    lse = torch.empty((2, 1, H), dtype=torch.float32, device="cuda")
    ws = mla.alloc_workspace(shape, 2, 1)
    mla.mla_decode(cache, table, gu.dev(np.array([2 ** 31 - 255 + over, 70], np.int32)), gu.dev(w.q, bf), gu.dev(w.W_UV, bf),
                   w.scale, out, lse, ws)
    torch.cuda.synchronize()
    code, flags = mla.mla_get_status(ws)
    assert code == mla.MLA_ERR_BOUNDS and flags == 2            # a length
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    lat = _stored(w) if kind == "mxfp8" else w.latent
    ro, rl = attention.absorbed(w.q[1], lat[1], w.rope[1], w.W_UV, w.scale)
    assert gu.rel_err(out[1].float().cpu().numpy(), ro) <= gu.BF16_REL_TOL
    assert np.max(np.abs(lse[1].cpu().numpy() - rl)) <= gu.BF16_LSE_TOL


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("H,q_len", [(16, 1), (16, 4), (64, 1), (8, 3), (128, 1), (128, 2)])
def test_scores_of_minus_infinity(gpu_lib, impl, H, q_len):
    """A sequence's first tokens score past the 32-bit range, and the others far below 0: weight
    0 for the former, the softmax over the latter."""
    import mla_latent_kv_08_gb300 as mla
    lens, gone = [700, 128 + q_len, q_len], [400, 128, 0]
    w = _workload(83, lens, H=H, q_len=q_len)
    w.q[..., 512], w.q[..., 513] = np.float32(2.0 ** 100), 30
    for b, n in enumerate(gone):
        w.rope[b][:, 0] = 0
        w.rope[b][:n, 0] = -np.float32(2.0 ** 60)
        w.rope[b][:, 1] = -500
    if impl == "roomy":
        _roomy(w)
    shape = _shape(mla, w, impl=_impl(mla, impl), num_splits_hint=1)
    cache, _ = gu.fill_cache(w, shape)
    out, lse, ws = gu.attend(w, shape, cache, w.q, q_len=q_len)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    lat = _stored(w)
    for b in range(3):
        ro, rl = attention.absorbed(w.q[b], lat[b], w.rope[b], w.W_UV, w.scale)
        assert gu.rel_err(out[b], ro) <= gu.BF16_REL_TOL, b
        assert np.max(np.abs(lse[b] - rl)) <= gu.BF16_LSE_TOL, b


def _nan_codes(w, cache, at):
    """Codes that are not a number at (sequence, token, latent dim); `_stored` with them."""
    lat = _stored(w)
    for i, (b, t, d) in enumerate(at):
        cache.codes[int(w.block_table[b, t // 64]), t % 64, d] = (0x7F, 0xFF)[i % 2]
        lat[b][t, d] = np.nan
    return lat


def test_a_code_that_is_not_a_number_reads_as_one(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(81, [130, 4200], H=1)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    lat = _nan_codes(w, cache, [(0, 0, 0), (0, 129, 511), (1, 7, 31), (1, 7, 32), (1, 4199, 300)])
    for b, L in enumerate((130, 4200)):                          # few rows, many rows
        rows = torch.empty((L, 576), dtype=torch.bfloat16, device="cuda")
        mla.mla_latent_read(cache, gu.dev(w.block_table[b:b + 1]), gu.dev(np.zeros(1, np.int32)),
                            gu.dev(np.array([0, L], np.int32)), rows)
        np.testing.assert_array_equal(rows.double().cpu().numpy(), np.concatenate([lat[b], w.rope[b]], 1))


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("H,q_len", [(16, 1), (16, 4), (64, 1), (128, 1), (128, 3)])
def test_a_code_that_is_not_a_number_in_a_draft(gpu_lib, impl, H, q_len):
    """It makes the rows that see it NaN and leaves those whose mask hides it as they are."""
    import mla_latent_kv_08_gb300 as mla
    lens = [200, 129, 66, 700, 385]
    w = _workload(82, lens, H=H, q_len=q_len)
    if impl == "roomy":
        _roomy(w)
    at = [(0, 199, 0), (1, 128 - (q_len > 1), 511), (2, 65, 255), (3, 350, 256), (4, 385 - q_len, 100)]
    shape = _shape(mla, w, impl=_impl(mla, impl), num_splits_hint=5)
    cache, _ = gu.fill_cache(w, shape)
    _nan_codes(w, cache, at)
    out, lse, ws = gu.attend(w, shape, cache, w.q, q_len=q_len)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    for b, t, _ in at:
        w.latent[b][t], w.rope[b][t] = 0, 0                      # hidden from the rows that are held to it
    lat = _stored(w)
    for b, t, _ in at:
        sees = lens[b] - q_len + np.arange(q_len) >= t
        assert np.isnan(out[b][sees]).all() and np.isnan(lse[b][sees]).all(), b
        if not sees.all():
            ro, rl = attention.absorbed(w.q[b], lat[b], w.rope[b], w.W_UV, w.scale)
            assert gu.rel_err(out[b][~sees], ro[~sees]) <= gu.BF16_REL_TOL, b
            assert np.max(np.abs(lse[b][~sees] - rl[~sees])) <= gu.BF16_LSE_TOL, b


@pytest.mark.parametrize("kind,impl,H,q_len", [("mxfp8", "auto", 128, 1), ("mxfp8", "roomy", 16, 2), ("mxfp8", "simt", 16, 1),
                                               ("bf16", "auto", 128, 1), ("bf16", "auto", 20, 3), ("int2", "auto", 128, 1)])
def test_rows_are_nan_after_a_wait_that_gave_up(gpu_lib, kind, impl, H, q_len):
    """As if a wait of a call's kernel had given up: NaN in every row, the flag, and the next
    call on the same workspace as ever."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(85, [700, 64, 129], H=H, q_len=q_len)
    if impl == "roomy":
        _roomy(w)
    kinds = {"mxfp8": mla.MLA_KV_MXFP8, "bf16": mla.MLA_KV_BF16, "int2": mla.MLA_KV_INT2_ROT}
    shape = _shape(mla, w, kind=kinds[kind], impl=_impl(mla, impl))
    R, T = (np.eye(512, dtype=np.float32), np.full(16, 4.0, np.float32)) if kind == "int2" else (None, None)
    cache, _ = gu.fill_cache(w, shape, R, T)
    want, want_l, _ = gu.attend(w, shape, cache, w.q, R=R, q_len=q_len)
    mla.mla_selftest_gave_up(1)
    try:
        out, lse, ws = gu.attend(w, shape, cache, w.q, R=R, q_len=q_len)
    finally:
        mla.mla_selftest_gave_up(0)
    assert mla.mla_get_status(ws) == (mla.MLA_ERR_TIMEOUT, 4)
    assert np.isnan(out).all() and np.isnan(lse).all()
    out, lse, ws = gu.attend(w, shape, cache, w.q, R=R, q_len=q_len)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    np.testing.assert_array_equal(out, want)
    np.testing.assert_array_equal(lse, want_l)
