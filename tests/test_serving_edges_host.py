"""More refusals of the shared-prefix decode and the budget cache on the CPU, with dummy pointers:
every call here is refused before anything is enqueued."""
import pytest

from sliding_window_causal_b200 import _native, build

P0 = 0x10000
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def test_scales_beyond_fp32_are_refused(lib):
    """scale log2(e) is an fp32 factor of the scores; as infinity it would make a score of 0 NaN."""
    size = (2, 38, 2, 5, 3, 64)
    ws = lib.swa_prefix_decode_workspace_bytes(*size)
    for scale in (3e38, 1e300):
        assert lib.swa_prefix_decode(*[P0] * 8, ws, *size, scale, None, None) == UNSUPPORTED, scale
        assert lib.swa_last_error()
        assert lib.swa_cache_decode(*[P0] * 9, 1 << 30, *size, scale, None, None) == UNSUPPORTED, scale
        for dtype in (0, 1):
            for sign in (1, -1):
                assert lib.swa_key_weights(P0, P0, P0, None, P0, 2, 4, 2, 9, 64, 3, 9, sign * scale, None, dtype,
                                           None) == UNSUPPORTED
