"""mla_prefill at the ends of its ranges. Tolerances: those of tests/test_gpu_prefill.py, from
its head."""
import numpy as np
import pytest

from tests.test_gpu_prefill import Case, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,impl,dims,bound", [
    ("mxfp8", 0, {}, 3500000), ("bf16", 0, {}, 3500000), ("mxfp8", 1, {}, 1800000),
    ("fp32", 1, dict(r=64, dR=16, dn=32, dv=32, bs=16), 7000000)])
def test_several_passes_over_the_heads(gpu_lib, kind, impl, dims, bound):
    """Keys and values of two heads fill the library's 4 GiB under a bound of so many cached
    tokens, so five heads take three passes, the last one a head short. The workspace starts as
    NaN, and two calls follow one another."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    case = Case(110, [300, 0, 140, 7], [200, 9, 0, 600], H=5, kind=kind, **dims)
    shape = case.shape(mla, impl=impl)
    head = (case.dn + case.dv) * (2 if impl == 0 else 4) * bound
    assert 2 * head <= 4 << 30 < 3 * head
    cache, a = case.cache(mla, shape, poison=True), case.args(mla, shape)
    a["max_tokens"] = bound
    a["workspace"] = mla.alloc_prefill_workspace(shape, 4, int(case.cu[-1]), bound, case.dn)
    a["workspace"].fill_(0xFF)
    for _ in range(2):
        a["out"].fill_(float("nan")), a["lse"].fill_(float("nan"))
        mla.mla_prefill(cache, **a)
        mla.mla_prefill(cache, **a)
        torch.cuda.synchronize()
        assert mla.mla_get_status(a["workspace"]) == (mla.MLA_OK, 0)
        case.check(a["out"].double().cpu().numpy(), a["lse"].cpu().numpy())


@pytest.mark.parametrize("above", [False, True])
def test_either_order_of_the_tiles(gpu_lib, above):
    """Chunks of unequal lengths, some empty, on as many heads as give just below and just
    above eight tiles (at their bound) for each SM: sequence by sequence, and head by head."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    new, past = [1500, 0, 700, 1, 0, 900, 257], [100, 30, 0, 2000, 0, 129, 0]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sum(new) // 256 + len(new)
    H = (8 * sms - 1) // tiles + above
    case = Case(111 + above, new, past, H=H, kind="mxfp8")
    out, lse, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0)
    assert np.isfinite(out).all() and np.isfinite(lse).all() and not (lse == 5.0).any()
    case.check(out, lse, heads=sorted({0, 1, H // 2, H - 2, H - 1}),
               rows=[0, 1, 127, 128, 255, 256, 257, 511, 512, 699, 899, 1023, 1280, 1499])


@pytest.mark.parametrize("kind,impl", [("mxfp8", 0), ("mxfp8", 1), ("fp32", 1)])
def test_scores_of_minus_infinity(gpu_lib, kind, impl):
    """The first cached tokens score past the 32-bit range: weight 0, and the softmax over the
    others as it is."""
    import mla_latent_kv_08_gb300 as mla
    case = Case(113, [100, 40, 9], [300, 65, 129], H=2, kind=kind)
    case.q[..., case.dn] = np.float32(2.0 ** 100)
    for r in case.rope:
        r[:, 0] = 0
        r[:64, 0] = -np.float32(2.0 ** 60)
    out, lse, status = _run(mla, case, case.shape(mla, impl=impl))
    assert status == (mla.MLA_OK, 0)
    case.check(out, lse)


@pytest.mark.parametrize("impl", [0, 1])
def test_a_code_that_is_not_a_number(gpu_lib, impl):
    """New tokens that see such a code are NaN; those before it stay as they are."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    case = Case(114, [300, 130, 40], [50, 0, 100], H=3, kind="mxfp8")
    at = [(0, 349, 0, 0x7F), (1, 1, 511, 0xFF), (2, 120, 255, 0x7F)]
    shape = case.shape(mla, impl=impl)
    cache, a = case.cache(mla, shape), case.args(mla, shape)
    for b, t, d, code in at:
        cache.codes[int(case.table[b, t // 64]), t % 64, d] = code
    mla.mla_prefill(cache, **a)
    torch.cuda.synchronize()
    assert mla.mla_get_status(a["workspace"]) == (mla.MLA_OK, 0)
    out, lse = a["out"].double().cpu().numpy(), a["lse"].cpu().numpy()
    for b, t, _, _ in at:
        first = t - int(case.L[b] - case.new[b])                         # the first new token that sees it
        mine = slice(int(case.cu[b]) + first, int(case.cu[b + 1]))
        assert np.isnan(out[mine]).all() and np.isnan(lse[mine]).all(), b
        case.lat[b][t], case.rope[b][t] = 0, 0                           # hidden from the rows that are held to it
        case.check(out, lse, seqs=[b], rows=np.arange(first))


@pytest.mark.parametrize("kind,lse", [("mxfp8", True), ("bf16", False)])
def test_rows_are_nan_after_an_expansion_that_gave_up(gpu_lib, kind, lse):
    """As if a wait of the kernel that makes keys and values had given up: NaN in every new
    token's rows, the flag, and the next call as ever."""
    import mla_latent_kv_08_gb300 as mla
    case = Case(115, [300, 0, 40, 1], [50, 9, 100, 700], H=3, kind=kind)
    change = {} if lse else {"lse": None}
    mla.mla_selftest_gave_up(1)
    try:
        out, got, status = _run(mla, case, **change)
    finally:
        mla.mla_selftest_gave_up(0)
    assert status == (mla.MLA_ERR_TIMEOUT, 4)
    assert np.isnan(out).all() and (got is None or np.isnan(got).all())
    out, got, status = _run(mla, case)
    assert status == (mla.MLA_OK, 0)
    case.check(out, got)
