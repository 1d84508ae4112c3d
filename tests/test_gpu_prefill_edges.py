"""mla_prefill at the ends of its ranges. Tolerances: those of tests/test_gpu_prefill.py, from
its head."""
import numpy as np
import pytest

from tests.test_gpu_prefill import Case, _run

pytestmark = pytest.mark.gpu


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
