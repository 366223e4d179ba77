"""Scored decode and prefill over the whole range of accepted caps, against fp64 attention.

Tolerances: those of scored_ref without its growth with the cap.  A capped score (log2 domain,
below 10 in size here) is off by at most 9e-5 where the cap is at most 128 and by 2^-20 of itself,
1e-5, above: 2 ln 2 * 9e-5 * 5 = 6.3e-4 in an output, and 1.2e-3 for P's bits, together below
2e-3.  fp32 pools: a cap off by three steps of the score, 10 * 3 * 2^-24 * 2 = 3.6e-6, moves an
output by 2 ln 2 * 3.6e-6 * 5 = 2.5e-5, which with 1e-5 stays below the tolerance that scored_ref
gives a bias."""
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import test_gpu_scored_decode as decode
from tests import test_gpu_scored_prefill as prefill
from tests.scored_ref import check, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


CAPS = [0.125, 128.0, 129.0, 1e3, 1e5, 1e6]


def run(c, tol=None):
    out = c.run()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    check(out, c.ref(), tol or tolerance(c.dtype, 0.0, True))


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("form", decode.FORMS)
def test_decode(form, cap, alibi):
    n_q, n_kv, d, bs, dtype, nq, fp8 = decode.FORMS[form]
    run(decode.Case(3000 + sorted(decode.FORMS).index(form), [32, 16, 300, 1001], n_q, n_kv, d, bs, dtype, nq,
                    fp8=fp8, softcap=cap, alibi=alibi, window=700))


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("form", prefill.FORMS)
def test_prefill(form, cap, alibi):
    n_q, n_kv, d, bs, dtype, fp8 = prefill.FORMS[form]
    run(prefill.Case(3100 + sorted(prefill.FORMS).index(form), [(5, 5), (3, 400), (130, 333)], n_q, n_kv, d, bs,
                     dtype, fp8=fp8, softcap=cap, alibi=alibi, prefix=150))


@pytest.mark.parametrize("cap", [1e3, 1e6])
@pytest.mark.parametrize("form", ["bf16-g4", "fp16-g2-d64", "fp8-g4"])
def test_split_prefill(form, cap):
    n_q, n_kv, d, bs, dtype, fp8 = prefill.FORMS[form]
    run(prefill.Case(3200, [(40, 4200), (3, 90)], n_q, n_kv, d, bs, dtype, fp8=fp8, softcap=cap, doc=3000))


def large(c):
    """Scores of +-150 under a cap of 200, on both sides of |x| = 3/8.  A score is
    off by 2^-20 of 183 and by 16 roundings of a sum of 313 in size, 5e-4 together: 2 ln 2 * 5e-4 *
    5 = 3.5e-3 in an output, and 1.2e-3 for P's bits."""
    c.q = (c.q.float() * 30).to(c.q.dtype)
    c.qd = c.q.cuda()
    run(c, 5e-3)


@pytest.mark.parametrize("form", ["bf16-g4", "bf16-q4", "fp8-g4", "fp8-q3", "fp8-g8"])
def test_decode_of_large_scores(form):
    n_q, n_kv, d, bs, dtype, nq, fp8 = decode.FORMS[form]
    large(decode.Case(3300, [17, 40, 500], n_q, n_kv, d, bs, dtype, nq, fp8=fp8, softcap=200.0))


@pytest.mark.parametrize("form", ["bf16-g4", "fp16-g3", "fp8-g4"])
def test_prefill_of_large_scores(form):
    n_q, n_kv, d, bs, dtype, fp8 = prefill.FORMS[form]
    large(prefill.Case(3400, [(5, 5), (3, 400), (130, 333)], n_q, n_kv, d, bs, dtype, fp8=fp8, softcap=200.0))
