"""The measurement hook of the decode calls covers all of a shared decode's attention."""
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from tests import test_gpu_shared as shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_25_gb300 import build
    build.build()
    assert pa.pa_get_device_error() == 0


def test_a_shared_decode_is_timed_with_its_prefix():
    """Nearly all keys are the prefix's: its pass takes most of the call (the merge is the rest)."""
    c = shared.Case(900, [(16384, [1 + i % 3 for i in range(100)])], [], *shared.FORMS["bf16-g4"][:5])
    inner, outer = ([torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(2))
    for e in inner + outer:
        e.record()
    out = c.run()
    torch.cuda.synchronize()
    shares = []
    pa.pa_set_profile_events(*inner)
    try:
        for _ in range(9):
            torch.cuda._sleep(2_000_000)        # the launches below are enqueued meanwhile
            outer[0].record()
            c.run(out=out)
            outer[1].record()
            torch.cuda.synchronize()
            shares.append(inner[0].elapsed_time(inner[1]) / outer[0].elapsed_time(outer[1]))
    finally:
        pa.pa_set_profile_events()
    assert sorted(shares)[4] > 0.5, shares
    assert pa.pa_get_device_error() == 0
