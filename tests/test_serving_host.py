"""Refusals of the shared-prefix decode and the budget cache on the CPU: at the C ABI with dummy
pointers (every call is refused or a no-op) and in the Python binding."""
import ctypes

import pytest
import torch

import sliding_window_causal_b200 as swa
from sliding_window_causal_b200 import _native, build

P0 = 0x10000
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def strides(*vals):
    return (ctypes.c_int64 * len(vals))(*vals)


def call(fn, base, n_ptr, **change):
    """fn with the arguments of dict base, some replaced."""
    args = {**base, **change}
    assert set(change) <= set(base)
    return fn(*args.values())


def test_key_weights_refusals(lib):
    base = dict(q=P0, k=P0, lse=P0, lens=None, w=P0, B=2, H=4, Hkv=2, T=9, D=64, W=3, last=9, scale=0.125, st=None,
                dtype=1, stream=None)
    f = lambda **c: call(lib.swa_key_weights, base, 5, **c)
    for bad in (dict(B=-1), dict(H=-4), dict(Hkv=3), dict(Hkv=0), dict(T=-1), dict(D=0), dict(W=0), dict(last=0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=2), dict(q=None), dict(lse=None),
                dict(w=None), dict(st=strides(-8, 576, 64, 1152, 576, 64))):
        assert f(**bad) == INVALID, bad
        assert lib.swa_last_error()
    for bad in (dict(D=96), dict(D=5000, dtype=0), dict(T=1 << 31), dict(H=4096, Hkv=2), dict(H=1 << 40, Hkv=1 << 40),
                dict(B=1 << 16, H=1 << 15, Hkv=1 << 15, T=64)):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=P0 + 8), dict(k=P0 + 2), dict(lse=P0 + 2), dict(w=P0 + 1), dict(lens=P0 + 4),
                dict(q=P0 + 2, dtype=0), dict(st=strides(2304, 576, 68, 1152, 576, 64))):
        assert f(**bad) == MISALIGNED, bad
    for empty in (dict(B=0), dict(H=0, Hkv=0), dict(T=0)):
        assert f(**empty, ) == OK


def test_cache_seed_refusals(lib):
    base = dict(k=P0, v=P0, w=P0, lens=None, kc=P0, vc=P0, wc=P0, pc=P0, B=2, Hkv=2, T=9, D=64, S=4, recent=1, st=None,
                stream=None)
    f = lambda **c: call(lib.swa_cache_seed, base, 8, **c)
    for bad in (dict(B=-1), dict(Hkv=-1), dict(T=-2), dict(S=0), dict(recent=-1), dict(recent=4), dict(k=None),
                dict(w=None), dict(pc=None), dict(D=0)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(D=80), dict(T=1 << 31), dict(S=1 << 31)):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(k=P0 + 8), dict(vc=P0 + 2), dict(wc=P0 + 2), dict(pc=P0 + 4), dict(lens=P0 + 4),
                dict(st=strides(1152, 576, 65, 1152, 576, 64))):
        assert f(**bad) == MISALIGNED, bad
    assert f(B=0) == OK and f(Hkv=0) == OK and f(T=0) == OK


def test_cache_append_refusals(lib):
    base = dict(k=P0, v=P0, kc=P0, vc=P0, wc=P0, pc=P0, pos=P0, slots=P0, B=2, Hkv=2, D=64, S=4, recent=1, stream=None)
    f = lambda **c: call(lib.swa_cache_append, base, 8, **c)
    for bad in (dict(B=-1), dict(S=0), dict(recent=-1), dict(recent=4), dict(pos=None), dict(slots=None), dict(D=0)):
        assert f(**bad) == INVALID, bad
    assert f(D=96) == UNSUPPORTED and f(S=1 << 31) == UNSUPPORTED
    for bad in (dict(k=P0 + 8), dict(kc=P0 + 8), dict(wc=P0 + 2), dict(pos=P0 + 4), dict(slots=P0 + 4)):
        assert f(**bad) == MISALIGNED, bad
    assert f(B=0) == OK and f(Hkv=0) == OK


def test_decode_refusals(lib):
    size = dict(B=2, H=38, Hkv=2, S=5, P=3, D=64)  # more than 8 query heads to a key head: a workspace
    for fn, need in ((lib.swa_cache_decode, lib.swa_cache_decode_workspace_bytes),
                     (lib.swa_prefix_decode, lib.swa_prefix_decode_workspace_bytes)):
        ws = need(*size.values())
        assert ws > 0
        if fn is lib.swa_cache_decode:
            base = dict(q=P0, k=P0, v=P0, w=P0, pos=P0, kp=P0, vp=P0, out=P0, ws=P0)
        else:
            base = dict(q=P0, kp=P0, vp=P0, k=P0, v=P0, pos=P0, out=P0, ws=P0)
        base |= dict(nbytes=ws, **size, scale=0.125, st=None, stream=None)
        f = lambda **c: call(fn, base, 9, **c)
        for bad in (dict(B=-1), dict(Hkv=3), dict(S=0), dict(P=-1), dict(D=0), dict(scale=float("nan")), dict(q=None),
                    dict(kp=None), dict(vp=None), dict(out=None), dict(ws=None), dict(nbytes=ws - 1), dict(pos=None),
                    dict(st=strides(-8, 64, 192, 64))):
            assert f(**bad) == INVALID, bad
            assert lib.swa_last_error()
        for bad in (dict(D=96), dict(scale=0.0), dict(scale=-1.0), dict(S=1 << 31), dict(P=1 << 31), dict(H=4096)):
            assert f(**bad) == UNSUPPORTED, bad
        for bad in (dict(q=P0 + 8), dict(k=P0 + 8), dict(kp=P0 + 8), dict(out=P0 + 2), dict(ws=P0 + 128),
                    dict(pos=P0 + 4), dict(st=strides(192, 68, 192, 64))):
            assert f(**bad) == MISALIGNED, bad
        assert f(B=0) == OK and f(H=0) == OK
        assert need(2, 4, 2, 5, 3, 64) == 0  # one cluster a key head needs none
        assert f(H=4, ws=None, nbytes=0, q=None) == INVALID
        assert need(2, 4, 3, 5, 3, 64) == -1 and need(2, 4, 2, 0, 3, 64) == -1 and need(2, 4, 2, 5, 3, 80) == -1
        assert need(0, 4, 2, 5, 3, 64) == 0
    assert lib.swa_cache_decode(P0, P0, P0, P0 + 2, P0, None, None, P0, P0, 1 << 30, 2, 4, 2, 5, 0, 64, 0.125, None,
                                None) == MISALIGNED  # weights


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refusals():
    B, H, Hkv, S, D, T = 2, 4, 2, 6, 64, 9
    q, pos = cpu(B, H, D), cpu(B, dtype=torch.int64)
    kc, w, p = cpu(B, Hkv, S, D), cpu(B, Hkv, S, dtype=torch.float32), cpu(B, Hkv, S, dtype=torch.int64)
    pre = cpu(Hkv, 5, D)
    with pytest.raises(ValueError, match="CUDA"):
        swa.prefix_decode(q, pre, pre, kc, kc, pos, S)
    with pytest.raises(ValueError, match="rings"):
        swa.prefix_decode(q, pre, pre, kc, kc, pos, S + 1)
    with pytest.raises(ValueError, match="multiple"):
        swa.prefix_decode(cpu(B, 3, D), pre, pre, kc, kc, pos, S)
    with pytest.raises(ValueError, match="prefix"):
        swa.prefix_decode(q, cpu(1, 5, D), cpu(1, 5, D), kc, kc, pos, S)
    with pytest.raises(ValueError, match="both"):
        swa.prefix_decode(q, pre, None, kc, kc, pos, S)
    with pytest.raises(ValueError, match="pos"):
        swa.prefix_decode(q, pre, pre, kc, kc, pos.int(), S)
    with pytest.raises(TypeError, match="bf16"):
        swa.prefix_decode(q.float(), pre, pre, kc, kc, pos, S)
    with pytest.raises(ValueError, match="wcache"):
        swa.cache_decode(q, kc, kc, w.double(), pos)
    with pytest.raises(ValueError, match="cache"):
        swa.cache_decode(cpu(B, H, 128), kc, kc, w, pos)
    with pytest.raises(ValueError, match="CUDA"):
        swa.cache_decode(q, kc, kc, w, pos)
    with pytest.raises(ValueError, match="pcache"):
        swa.cache_append(kc[:, :, 0], kc[:, :, 0], kc, kc, w, p.int(), pos, 1)
    with pytest.raises(ValueError, match="k and v"):
        swa.cache_append(q, q, kc, kc, w, p, pos, 1)
    with pytest.raises(ValueError, match="weights"):
        swa.cache_seed(cpu(B, Hkv, T, D), cpu(B, Hkv, T, D), w, kc, kc, w, p, 1)
    with pytest.raises(ValueError, match="fits"):
        swa.cache_seed(cpu(B, 1, T, D), cpu(B, 1, T, D), w, kc, kc, w, p, 1)
    x = cpu(B, H, T, D)
    with pytest.raises(ValueError, match="lse"):
        swa.key_weights(x, cpu(B, Hkv, T, D), cpu(B, H, T), 4)
    with pytest.raises(ValueError, match="multiple"):
        swa.key_weights(x, cpu(B, 3, T, D), cpu(B, H, T, dtype=torch.float32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        swa.key_weights(x, cpu(B, Hkv, T, D), cpu(B, H, T, dtype=torch.float32), 4)
