"""The pool's books, copies of cached rows and the acceptance of drafts without a GPU: the
oracle's own pins, and the arguments that are refused before anything is launched."""
import ctypes

import pytest

from oracle import upkeep


@pytest.fixture(scope="module")
def lib():
    from mla_latent_kv_08_gb300 import build
    build.build()
    import mla_latent_kv_08_gb300 as mla
    return mla.load_library()


def _shape(**kw):
    import mla_latent_kv_08_gb300 as mla
    base = dict(num_heads=128, kv_lora_rank=512, rope_dim=64, v_head_dim=128, block_size=64, num_blocks=10)
    base.update(kw)
    return mla.Shape(**base)


# ------------------------------------------------------------------ the oracle

def test_oracle_books():
    k = upkeep.Books(4, 5, 8, 4)
    assert k.resize([9, 4, 0, 0]) == (0, [], 4)
    assert k.table()[:2] == [[0, 1, 2, -1, -1], [3, -1, -1, -1, -1]]
    assert k.fork([0, 0], [2, 3], [9, 4]) == (0, [[2, 4, 0, 1]], 3)
    assert k.rows[2] == [0, 1, 4] and k.rows[3] == [0] and k.ref == [3, 2, 1, 1, 1, 0, 0, 0]
    # a cut inside the shared block 1: a block of its own; block 4 is free again, block 2 is not touched
    assert k.resize([9, 4, 6, 4]) == (0, [[1, 5, 0, 2]], 3)
    assert k.rows[2] == [0, 5] and k.ref == [3, 1, 1, 1, 0, 1, 0, 0]
    assert k.resize([9, 4, 6, 20])[0] == upkeep.FULL and k.lens == [9, 4, 6, 4]
    assert k.compact(9) == (0, [[5, 4, 0, 4]], 5) and k.rows[2] == [0, 4]


def test_oracle_accept():
    p, close = [[[0.5, 0.25, 0.25], [0.0, 0.5, 0.5]]], [[[0.5, 0.25, 0.25]]]

    def accept(q, x, u):
        return upkeep.accept(p, q, [[x]], [u], lens=[7])[0]
    assert accept(None, 0, [0.49, 0.5]) == (0, 1, [0, 2], 7)             # 0.49 < 0.5: it stands
    assert accept(None, 0, [0.5, 0.0]) == (0, 0, [1, -1], 6)             # not: one of the others
    assert accept(None, 0, [0.5, 0.5]) == (0, 0, [2, -1], 6)
    assert accept(close, 0, [1.0, 0.6]) == (0, 0, [1, -1], 6)            # nothing left of p - q: p itself
    assert accept(None, 0, [0.0, 1.0]) == (0, 1, [0, 2], 7)
    assert accept(None, 3, [0.0, 1.0]) == (upkeep.VALUE, 0, [-1, -1], 6)


# ------------------------------------------------------------------ refusals of the library

FAKE = ctypes.c_void_p(4096)         # never dereferenced: every call here is refused on the host
FAKE2, FAKE3, FAKE4 = ctypes.c_void_p(8192), ctypes.c_void_p(12288), ctypes.c_void_p(16384)
ODD = ctypes.c_void_p(4100)


def _pool(mla, **kw):
    f = dict(block_table=4096, seq_lens=4096, ref_count=4096, max_seqs=3, max_blocks_per_seq=4)
    f.update(kw)
    return mla.mla_pool(*f.values())


BAD_POOLS = [dict(block_table=None), dict(seq_lens=None), dict(ref_count=None), dict(max_seqs=0), dict(max_blocks_per_seq=0)]


def test_status_strings(lib):
    import mla_latent_kv_08_gb300 as mla
    assert mla.MLA_ERR_FULL == -7 and mla.MLA_ERR_VALUE == -8
    for code in (mla.MLA_ERR_FULL, mla.MLA_ERR_VALUE):
        assert mla.status_string(code) != "unknown status"


def test_resize_arguments(lib):
    import mla_latent_kv_08_gb300 as mla

    def call(shape=_shape(), pool=None, new=FAKE2, copies=FAKE, n=FAKE):
        pool = pool or _pool(mla)
        return lib.mla_pool_resize(ctypes.byref(shape.c()), ctypes.byref(pool), new, copies, n, None, None, None)
    for kw in [dict(pool=_pool(mla, **b)) for b in BAD_POOLS] + [
            dict(new=None), dict(new=FAKE), dict(copies=None), dict(copies=ODD), dict(n=None), dict(shape=_shape(kv_lora_rank=7))]:
        assert call(**kw) == mla.MLA_ERR_INVALID, kw
    pool, s = _pool(mla), _shape().c()
    for outs in ((FAKE, None), (None, FAKE), (FAKE2, FAKE2)):            # of num_copies (FAKE), num_free and status two the same
        assert lib.mla_pool_resize(ctypes.byref(s), ctypes.byref(pool), FAKE2, FAKE, FAKE, *outs, None) == mla.MLA_ERR_INVALID
    assert call(pool=_pool(mla, max_seqs=16385)) == mla.MLA_ERR_UNSUPPORTED
    assert call(pool=_pool(mla, max_seqs=16384, max_blocks_per_seq=1 << 17)) == mla.MLA_ERR_UNSUPPORTED
    assert lib.mla_pool_resize(ctypes.byref(_shape().c()), None, FAKE, FAKE, FAKE, None, None, None) == mla.MLA_ERR_INVALID


def test_fork_arguments(lib):
    import mla_latent_kv_08_gb300 as mla

    def call(pool=None, n=2, parents=FAKE, children=FAKE, copies=FAKE, num=FAKE):
        return lib.mla_pool_fork(ctypes.byref(_shape().c()), ctypes.byref(pool or _pool(mla)), n, parents, children, None,
                                 copies, num, None, None, None)
    for kw in [dict(pool=_pool(mla, **b)) for b in BAD_POOLS] + [
            dict(n=0), dict(n=-1), dict(parents=None), dict(children=None), dict(copies=None), dict(copies=ODD), dict(num=None)]:
        assert call(**kw) == mla.MLA_ERR_INVALID, kw
    assert call(n=16385) == mla.MLA_ERR_UNSUPPORTED


def test_compact_arguments(lib):
    import mla_latent_kv_08_gb300 as mla

    def call(pool=None, room=2, copies=FAKE, num=FAKE):
        return lib.mla_pool_compact(ctypes.byref(_shape().c()), ctypes.byref(pool or _pool(mla)), room, copies, num, None,
                                    None, None)
    for kw in [dict(pool=_pool(mla, **b)) for b in BAD_POOLS] + [dict(room=-1), dict(copies=None), dict(copies=ODD), dict(num=None)]:
        assert call(**kw) == mla.MLA_ERR_INVALID, kw


def test_copy_arguments(lib):
    import mla_latent_kv_08_gb300 as mla
    dense = mla.mla_cache(4096, None, None, None)

    def call(shape=_shape(), cache=dense, n=1, copies=FAKE, num=FAKE, room=3):
        return lib.mla_cache_copy(ctypes.byref(shape.c()), ctypes.byref(cache) if cache else None, n, copies, num, room, None, None)
    mx, int2 = _shape(kind=mla.MLA_KV_MXFP8), _shape(kind=mla.MLA_KV_INT2_ROT)
    for kw in (dict(cache=None), dict(n=0), dict(copies=None), dict(copies=ODD), dict(num=None), dict(room=-1),
               dict(cache=mla.mla_cache(4100, None, None, None)), dict(cache=mla.mla_cache(None, 4096, 4096, 4096)),
               dict(shape=mx), dict(shape=int2), dict(shape=mx, cache=mla.mla_cache(None, 4096, 4096, None)),
               dict(shape=int2, cache=mla.mla_cache(None, 4096, 4096, None)), dict(shape=_shape(kind=9))):
        assert call(**kw) == mla.MLA_ERR_INVALID, kw
    assert call(room=1 << 26) == mla.MLA_ERR_UNSUPPORTED
    assert call(room=0, copies=None) == mla.MLA_OK                       # nothing to copy
    # every cache is looked at, also those of a later launch
    many = (mla.mla_cache * 70)(*([dense] * 69 + [mla.mla_cache(None, None, None, None)]))
    assert lib.mla_cache_copy(ctypes.byref(_shape().c()), many, 70, FAKE, FAKE, 0, None, None) == mla.MLA_ERR_INVALID


def test_accept_arguments(lib):
    import mla_latent_kv_08_gb300 as mla

    def call(B=2, K=3, V=100, dtype=mla.MLA_DTYPE_F32, p=FAKE, ps=100, q=FAKE, qs=100, x=FAKE, counts=None, u=FAKE, lens=None,
             accepted=FAKE2, tokens=FAKE3, new=None, status=None):
        return lib.mla_draft_accept(B, K, V, dtype, p, ps, q, qs, x, counts, u, lens, accepted, tokens, new, status, None)
    for kw in (dict(B=0), dict(K=-1), dict(V=0), dict(dtype=mla.MLA_DTYPE_F64), dict(dtype=9), dict(p=None), dict(ps=99),
               dict(qs=99), dict(x=None), dict(u=None), dict(accepted=None), dict(tokens=None), dict(lens=FAKE4),
               dict(new=FAKE4), dict(tokens=FAKE), dict(tokens=FAKE2), dict(accepted=FAKE), dict(new=FAKE2, lens=FAKE4),
               dict(new=FAKE3, lens=FAKE4), dict(lens=FAKE2, new=FAKE4), dict(counts=FAKE2), dict(status=FAKE3),
               dict(counts=FAKE4, lens=FAKE, new=FAKE4)):
        assert call(**kw) == mla.MLA_ERR_INVALID, kw
    for kw in (dict(K=257), dict(V=(1 << 30) + 1, ps=1 << 31, qs=1 << 31)):
        assert call(**kw) == mla.MLA_ERR_UNSUPPORTED, kw


def test_lists_that_no_copy_call_takes(lib):
    """A list that mla_cache_copy refuses is refused before the books change."""
    import mla_latent_kv_08_gb300 as mla
    dense = mla.mla_cache(4096, None, None, None)
    for shape, room in ((_shape(), 1 << 26), (_shape(), 1 << 25), (_shape(block_size=1 << 20), 16385), (_shape(block_size=131069), 16385)):
        s = ctypes.byref(shape.c())
        assert lib.mla_cache_copy(s, ctypes.byref(dense), 1, FAKE, FAKE, room, None, None) == mla.MLA_ERR_UNSUPPORTED
        assert lib.mla_pool_compact(s, ctypes.byref(_pool(mla)), room, FAKE, FAKE, None, None, None) == mla.MLA_ERR_UNSUPPORTED


def test_a_copy_counts_apart_from_its_flags(lib):
    import mla_latent_kv_08_gb300 as mla
    dense = mla.mla_cache(4096, None, None, None)
    assert lib.mla_cache_copy(ctypes.byref(_shape().c()), ctypes.byref(dense), 1, FAKE, FAKE2, 3, FAKE2, None) == mla.MLA_ERR_INVALID


# ------------------------------------------------------------------ refusals of the binding

def test_handles_check_their_tensors():
    import mla_latent_kv_08_gb300 as mla
    import torch
    s = _shape()
    pool = mla.Pool.allocate(s, 3, 4, device="cpu")
    assert pool.block_table.shape == (3, 4) and int(pool.block_table.max()) == -1 and not pool.ref_count.any()
    t, l, r = pool.block_table, pool.seq_lens, pool.ref_count
    for bad in ((t[0], l, r), (t, l[:2], r), (t, l, r[:9]), (t.long(), l, r), (t, l.float(), r), (t.T.contiguous().T, l, r)):
        with pytest.raises(mla.MlaError):
            mla.Pool(s, *bad)
    with pytest.raises(AttributeError):
        pool.seq_lens = l                         # the handle keeps the pointers
    assert pool == pool and pool != mla.Pool(s, t, l, r) and len({pool, pool}) == 1
    one, other = mla.Cache.allocate(s, device="cpu"), mla.Cache.allocate(_shape(num_blocks=9), device="cpu")
    mla.Caches([one, one])
    for bad in ([], [one, other], [mla.Cache(s)], [mla.Cache(s, latent=other.latent)],
                [mla.Cache(s, latent=one.latent.transpose(0, 1))]):
        with pytest.raises(mla.MlaError):
            mla.Caches(bad)


def test_sizes_past_32_bits_are_refused():
    """Sizes that a 32-bit argument would cut to small ones."""
    import mla_latent_kv_08_gb300 as mla
    import torch

    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device="meta")
    s = _shape()
    for S, W in ((1, 2 ** 32 + 4), (2 ** 32 + 1, 1), (1, 2 ** 31)):
        with pytest.raises(mla.MlaError) as e:
            mla.Pool(s, ints(S, W), ints(S), ints(10))
        assert e.value.code == mla.MLA_ERR_UNSUPPORTED
    for n in (2 ** 31, 2 ** 32 + 1):
        with pytest.raises(mla.MlaError) as e:
            mla._check_list("a list", ints(n, 4), ints(1), 0)
        assert e.value.code == mla.MLA_ERR_UNSUPPORTED


def test_every_array_of_a_cache_has_its_size():
    import mla_latent_kv_08_gb300 as mla
    import torch
    for kind in (mla.MLA_KV_MXFP8, mla.MLA_KV_INT2_ROT, mla.MLA_KV_INT2_ROT_QR, mla.MLA_KV_INT2_JOINT):
        s = _shape(kind=kind)
        c = mla.Cache.allocate(s, device="cpu")
        mla.Caches([c])
        swapped = mla.Cache(s, codes=c.scale_zero, scale_zero=c.codes, rope=c.rope)          # as many bytes in all
        rest = c.codes.numel() + c.scale_zero.numel() * c.scale_zero.element_size() - 1
        moved = mla.Cache(s, codes=torch.zeros(rest, dtype=torch.uint8), scale_zero=torch.zeros(1, dtype=torch.uint8), rope=c.rope)
        for bad in (swapped, moved, mla.Cache(s, codes=c.codes, rope=c.rope), mla.Cache(s, latent=c.codes, scale_zero=c.scale_zero, rope=c.rope)):
            with pytest.raises(mla.MlaError):
                mla.Caches([c, bad])
    for kind in (mla.MLA_KV_BF16, mla.MLA_KV_FP32):
        mla.Caches([mla.Cache.allocate(_shape(kind=kind, index_dim=64), device="cpu")])


def test_row_strides():
    import mla_latent_kv_08_gb300 as mla
    import torch
    wide = torch.zeros(3, 4, 50)
    for t, want in ((wide, 50), (wide[:, :, :49], 50), (wide[:, :1].contiguous(), 50), (wide[:, 2:3], 200), (wide[1:2, 1:3], 50),
                    (wide[:1, :1, :7], 7), (wide[:, :0], 50)):
        assert mla._row_stride(t) == (want, True), (t.shape, t.stride())
    for t in (wide[:, :3], wide[:, :, ::2], wide.transpose(0, 1), wide[:, ::2, :], wide[:1].expand(3, 4, 50)):
        s, ok = mla._row_stride(t)
        assert not ok or (t.shape[1] == 2 and s == 100), (t.shape, t.stride())
