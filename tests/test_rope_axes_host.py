"""CPU checks of the map from pairs to axes, as the several-axes rotary write takes it."""
import numpy as np
import pytest
import torch

from paged_kv_cache_25_gb300 import binding as pa
from paged_kv_cache_25_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    return pa.lib()


class Seen(Exception):
    pass


@pytest.fixture
def taken(monkeypatch):
    """what reaches the library's marshalling as the map"""
    class Marshal:
        def rope(self, *args):
            raise Seen(args[-1])

    monkeypatch.setattr(pa, "_marshal", Marshal)

    def call(axis):
        with pytest.raises(Seen) as e:
            pa.pa_rope_axes_and_cache(*[None] * 5, axis, *[None] * 4)
        return bytes(e.value.args[0])
    return call


@pytest.mark.parametrize("bad", [64, 0, True, np.int64(64), np.uint8(8), torch.tensor(64), None, 1.5], ids=repr)
def test_a_number_is_no_map(bad, taken):
    with pytest.raises(TypeError):
        taken(bad)


@pytest.mark.parametrize("bad", [[0, 256], [-1], [0, 1.5], ["0"]], ids=repr)
def test_numbers_that_are_no_axis(bad, taken):
    with pytest.raises((TypeError, ValueError)):
        taken(bad)


def test_maps(taken):
    want = bytes([0, 1, 2, 0] * 4)
    for axis in (want, list(want), tuple(want), bytearray(want), memoryview(want), np.frombuffer(want, np.uint8),
                 torch.tensor(list(want), dtype=torch.uint8), iter(want)):
        assert taken(axis) == want
