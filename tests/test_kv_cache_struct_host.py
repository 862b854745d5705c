"""The cache's struct at the C level: what the library would read at another
object's address is refused before the call."""
import ctypes

import pytest

import rank_sum_residual_gb300 as farn

A = 1 << 40


def calls(cache):
    yield lambda: farn.farn_kv_write(0, 4, A, 64, 2 * A, 64, cache, 3 * A)
    yield lambda: farn.farn_kv_read(0, cache, A, 2, 3, 2 * A, 40, 3 * A, 4 * A)
    yield lambda: farn.farn_qk_norm_rope_cache(0, 4, 64, A, 2, 128, 2 * A, 64, 3 * A, 64, 1, 0, 0,
                                               1e-6, 0, 0, None, 0, 0, 0, 4 * A, 128, cache, 5 * A)


class Other(ctypes.Structure):
    _fields_ = farn.KvCache._fields_[:2]


@pytest.mark.parametrize("cache", [ctypes.c_int(1), Other(1, 16), 0, A, b"cache", (1, 16)])
def test_other_objects_are_refused(cache):
    farn.build_library()
    for call in calls(cache):
        with pytest.raises(TypeError, match="KvCache"):
            call()


def test_the_struct_and_none_are_taken():
    farn.build_library()
    for cache in (None, farn.KvCache(), farn.KvCache(farn.FARN_CACHE_FP8, 16, 8, 1, 64)):
        for call in calls(cache):
            assert call() == farn.FARN_ERR_INVALID_ARG          # no context
