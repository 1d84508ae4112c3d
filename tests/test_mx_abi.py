"""The 8-bit cache kind, reading back and prefill without a GPU: the oracle's own pins,
layout, the shapes and arguments that are refused before anything is launched."""
import ctypes

import numpy as np
import pytest

from oracle import mx as omx


@pytest.fixture(scope="module")
def lib():
    from mla_latent_kv_08_gb300 import build
    build.build()
    import mla_latent_kv_08_gb300 as mla
    return mla.load_library()


def _shape(**kw):
    import mla_latent_kv_08_gb300 as mla
    base = dict(num_heads=128, kv_lora_rank=512, rope_dim=64, v_head_dim=128, block_size=64, num_blocks=10,
                kind=mla.MLA_KV_MXFP8)
    base.update(kw)
    return mla.Shape(**base)


# ------------------------------------------------------------------ the oracle

def test_e4m3_table():
    v = omx.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448 and v[0x38] == 1.0
    assert np.all(np.diff(v) > 0)


def test_oracle_rounds_to_nearest_even():
    # halfway between 1 (0x38) and 1.125 (0x39); between 1.125 and 1.25 (0x3a)
    np.testing.assert_array_equal(omx.nearest_code(np.array([1.0625, 1.1875, -1.0625, 448.0, 0.0, 2.0 ** -10])),
                                  [0x38, 0x3A, 0xB8, 126, 0, 0])
    import torch
    x = np.random.default_rng(0).standard_normal(4000) * np.exp2(np.random.default_rng(1).integers(-12, 8, 4000))
    x = np.clip(x.astype(np.float32), -448, 448)
    np.testing.assert_array_equal(omx.nearest_code(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("top,e", [(448.0, 0), (449.0, 1), (1.0, -8), (1.75, -8), (1.76, -7), (0.0, -110),
                                   (2.0 ** -130, -110), (2.0 ** 127 * 1.75, 119), (2.0 ** 127 * 1.99, 119)])
def test_oracle_scale(top, e):
    x = np.zeros((1, 32))
    x[0, 5] = -top
    codes, scales = omx.encode(x)
    assert int(scales[0, 0]) == e + 127
    got = omx.decode(codes, scales)
    assert abs(got[0, 5] + top) <= max(top * 2.0 ** -4, top - 448 * 2.0 ** 119) + 2.0 ** -120


def test_oracle_relative_error():
    x = np.random.default_rng(3).standard_normal((50, 128)) * 3
    y = omx.decode(*omx.encode(x))
    amax = np.abs(x.reshape(50, 4, 32)).max(-1).repeat(32, 1)
    # half a step: 2^-4 of the value, or 2^-10 of a scale that is below amax / 224
    assert np.all(np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, amax / 224 * 2.0 ** -10))


# ------------------------------------------------------------------ the library's refusals

def test_cache_layout():
    import mla_latent_kv_08_gb300 as mla
    c = mla.Cache.allocate(_shape(num_blocks=3), device="cpu")
    assert c.bytes_per_token() == 512 + 16 + 128
    assert c.latent is None
    assert sum(x.numel() * x.element_size() for x in (c.codes, c.scale_zero, c.rope)) == 656 * 3 * 64


def test_shapes(lib):
    import mla_latent_kv_08_gb300 as mla
    assert mla.mla_resolve_impl(_shape()) >= 0
    assert mla.mla_resolve_impl(_shape(kv_lora_rank=64, rope_dim=16, block_size=7)) == mla.MLA_IMPL_SIMT
    for bad in (dict(kv_lora_rank=520), dict(group_size=16), dict(group_size=64), dict(rope_dim=0),
                dict(index_dim=64), dict(flags=mla.MLA_FLAG_WUV_FOLDED), dict(flags=mla.MLA_FLAG_Q_ROTATED)):
        assert mla.mla_resolve_impl(_shape(**bad)) == mla.MLA_ERR_INVALID, bad


def test_a_changed_shape_counts(lib):
    """Calls go by the shape's fields at the time, and a struct handed out is the caller's own."""
    import mla_latent_kv_08_gb300 as mla
    s = _shape()
    before = mla.mla_workspace_bytes(s, 4)
    s.c().num_heads = 1
    assert mla.mla_workspace_bytes(s, 4) == before
    s.kv_lora_rank = 520
    assert mla.mla_resolve_impl(s) == mla.MLA_ERR_INVALID
    s.kv_lora_rank = 512
    assert mla.mla_workspace_bytes(s, 4) == before


FAKE = ctypes.c_void_p(4096)         # never dereferenced: every call here is refused on the host
ODD = ctypes.c_void_p(4100)


def _cache(mla, **kw):
    f = dict(latent=None, codes=4096, scale_zero=4096, rope=4096)
    f.update(kw)
    return mla.mla_cache(f["latent"], f["codes"], f["scale_zero"], f["rope"])


@pytest.mark.parametrize("change", [dict(codes=None), dict(scale_zero=None), dict(rope=None), dict(codes=4100),
                                    dict(rope=4104), dict(scale_zero=4097)])
def test_cache_pointers_refused(lib, change):
    import mla_latent_kv_08_gb300 as mla
    s, c = _shape().c(), _cache(mla, **change)
    assert lib.mla_latent_append(ctypes.byref(s), ctypes.byref(c), FAKE, 4, 2, FAKE, FAKE, 3, FAKE, FAKE, None, None,
                                 None, None) == mla.MLA_ERR_INVALID
    assert lib.mla_latent_read(ctypes.byref(s), ctypes.byref(c), FAKE, 4, 2, FAKE, FAKE, 3, FAKE, None,
                               None) == mla.MLA_ERR_INVALID
    n = 1 << 40
    assert lib.mla_decode(ctypes.byref(s), ctypes.byref(c), FAKE, 4, FAKE, 2, FAKE, FAKE, None, ctypes.c_float(0.1),
                          FAKE, FAKE, FAKE, n, None) == mla.MLA_ERR_INVALID
    assert lib.mla_prefill(ctypes.byref(s), ctypes.byref(c), FAKE, 4, FAKE, FAKE, 2, 3, 100, 128, FAKE, FAKE, FAKE,
                           ctypes.c_float(0.1), FAKE, None, FAKE, n, None) == mla.MLA_ERR_INVALID


def test_read_arguments(lib):
    import mla_latent_kv_08_gb300 as mla
    s, c = _shape().c(), _cache(mla)

    def call(shape=s, cache=c, table=FAKE, mb=4, B=2, start=FAKE, cu=FAKE, n=3, rows=FAKE):
        return lib.mla_latent_read(ctypes.byref(shape), ctypes.byref(cache), table, mb, B, start, cu, n, rows, None, None)
    for kw in (dict(table=None), dict(mb=0), dict(B=0), dict(start=None), dict(cu=None), dict(n=-1), dict(rows=None),
               dict(rows=ODD), dict(shape=_shape(kv_lora_rank=7).c())):
        assert call(**kw) == mla.MLA_ERR_INVALID, kw
    assert call(n=0, rows=None) == mla.MLA_OK               # nothing to read


def test_index_append_refused(lib):
    import mla_latent_kv_08_gb300 as mla
    s, c = _shape(index_dim=64).c(), _cache(mla)
    assert lib.mla_latent_append_index(ctypes.byref(s), ctypes.byref(c), FAKE, 4, 2, FAKE, FAKE, 3, FAKE, None,
                                       None) == mla.MLA_ERR_INVALID


def test_prefill_arguments(lib):
    import mla_latent_kv_08_gb300 as mla
    nan = float("nan")

    def call(shape=None, cache=None, table=FAKE, mb=4, lens=FAKE, cu=FAKE, B=2, nq=3, mt=100, dn=128, q=FAKE, wk=FAKE,
             wv=FAKE, scale=0.1, out=FAKE, ws=FAKE, size=1 << 40):
        s = (shape or _shape()).c()
        c = cache or _cache(mla)
        return lib.mla_prefill(ctypes.byref(s), ctypes.byref(c), table, mb, lens, cu, B, nq, mt, dn, q, wk, wv,
                               ctypes.c_float(scale), out, None, ws, size, None)
    for kw in (dict(table=None), dict(mb=0), dict(lens=None), dict(cu=None), dict(B=0), dict(nq=-1), dict(mt=-1),
               dict(dn=0), dict(dn=12), dict(q=None), dict(q=ODD), dict(wk=None), dict(wk=ODD), dict(wv=None), dict(wv=ODD),
               dict(scale=nan), dict(out=None), dict(out=ODD), dict(ws=None), dict(ws=ODD),
               dict(shape=_shape(kind=9))):
        assert call(**kw) == mla.MLA_ERR_INVALID, kw
    for kw in (dict(shape=_shape(kind=mla.MLA_KV_INT2_ROT)), dict(shape=_shape(kind=mla.MLA_KV_INT2_JOINT)),
               dict(dn=520), dict(shape=_shape(v_head_dim=1032)), dict(mt=2 ** 31 - 1), dict(nq=2 ** 31 - 1)):
        assert call(**kw) == mla.MLA_ERR_UNSUPPORTED, kw
    assert call(size=1000) == mla.MLA_ERR_WORKSPACE
    need = mla.mla_prefill_workspace_bytes(_shape(), 2, 3, 100, 128)
    assert call(size=need - 1) == mla.MLA_ERR_WORKSPACE


def test_prefill_workspace(lib):
    import mla_latent_kv_08_gb300 as mla
    small = mla.mla_prefill_workspace_bytes(_shape(), 1, 1, 1, 128)
    big = mla.mla_prefill_workspace_bytes(_shape(), 4, 4096, 100000, 128)
    assert 0 < small < big < 5 << 30          # keys and values of some heads at a time
    for bad in (dict(B=0), dict(num_q=-1), dict(nope_dim=7)):
        a = dict(B=1, num_q=1, max_tokens=1, nope_dim=128)
        a.update(bad)
        with pytest.raises(mla.MlaError):
            mla.mla_prefill_workspace_bytes(_shape(), **a)


def test_prefill_selftest_arguments(lib):
    import mla_latent_kv_08_gb300 as mla
    for calls in (-1, 17):
        assert lib.mla_selftest_gave_up(calls) == mla.MLA_ERR_INVALID
    mla.mla_selftest_gave_up(0)
