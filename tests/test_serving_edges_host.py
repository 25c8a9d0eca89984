"""More refusals of the shared-prefix decode and the budget cache on the CPU, with dummy pointers:
every call here is refused before anything is enqueued."""
import pytest

from sliding_window_causal_b200 import _native, build

P0 = 0x10000
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


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


def test_key_weights_of_no_query_heads_need_their_output(lib):
    """H = 0 is a call like any other: the weights are written (as zeros), so they must be there."""
    f = lambda **c: lib.swa_key_weights(*{**dict(q=None, k=None, lse=None, lens=None, w=P0, B=2, H=0, Hkv=2, T=9, D=64, W=3,
                                                 last=9, scale=0.125, st=None, dtype=1, stream=None), **c}.values())
    assert f(w=None) == INVALID and f(w=P0 + 2) == MISALIGNED and f(lens=P0 + 4) == MISALIGNED
    assert f(Hkv=1 << 40) == UNSUPPORTED and f(Hkv=1 << 62) == UNSUPPORTED and f(D=80) == UNSUPPORTED
    assert f(Hkv=0, w=None) == OK and f(T=0, w=None) == OK
