"""Calls at the edges of the serving operators' documented ranges."""
import math

import pytest
import torch

import serving_ref as ref
import sliding_window_causal_b200 as swa
from test_gpu_serving import BF, DEV, band_lse, gen, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("lens", [None, [9, 0], [4, 9]])
def test_key_weights_of_no_query_heads_are_zeros(dtype, lens):
    """The sum over no head: 0 for every key, also in memory that held something else."""
    k = rand(gen(1), 2, 3, 9, 64, dtype=dtype)
    dirty = torch.full((2, 3, 9), 5.0, device=DEV)
    del dirty  # the allocator hands the same memory out again
    w = swa.key_weights(k[:, :0], k, torch.empty(2, 0, 9, device=DEV), 3,
                        lens=None if lens is None else torch.tensor(lens, device=DEV))
    assert w.shape == (2, 3, 9) and bool((w == 0).all())
    swa.device_status()


def test_key_weights_of_no_query_heads_report_a_length_out_of_range():
    k = rand(gen(2), 2, 3, 9, 64)
    w = swa.key_weights(k[:, :0], k, torch.empty(2, 0, 9, device=DEV), 3, lens=torch.tensor([9, 10], device=DEV))
    with pytest.raises(swa.SwaError) as e:
        swa.device_status()
    assert e.value.code == 1 and bool((w == 0).all())


def test_tensors_of_a_device_that_is_not_current(monkeypatch):
    """Each call launches on its tensors' device and that device's current stream. With one GPU the
    other current device is claimed: the calls then enter the tensors' device themselves."""
    B, Hkv, G, D, S, P, T = 2, 2, 2, 64, 12, 40, 30
    g = gen(3)
    q, k, v = rand(g, B, Hkv * G, T, D), rand(g, B, Hkv, T, D), rand(g, B, Hkv, T, D)
    kp, vp = rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    lse = band_lse(q, k, 7)
    pos = torch.tensor([T, T + 3], device=DEV)

    def steps():
        w = swa.key_weights(q, k, lse, 7)
        cache = [torch.zeros(B, Hkv, S, D, dtype=BF, device=DEV) for _ in range(2)] + \
            [torch.zeros(B, Hkv, S, device=DEV), torch.zeros(B, Hkv, S, dtype=torch.int64, device=DEV)]
        swa.cache_seed(k, v, w, *cache, 3)
        slots = swa.cache_append(k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), *cache, pos, 3)
        return [w, slots, swa.cache_decode(q[:, :, 0].contiguous(), *cache[:3], pos, kp, vp),
                swa.prefix_decode(q[:, :, 1].contiguous(), kp, vp, cache[0], cache[1], pos, S), *cache]

    want = steps()
    current, stream = swa._cuda()
    entered = []
    monkeypatch.setattr(swa, "_cuda", lambda: (lambda: -1, lambda dev: entered.append(dev) or stream(dev)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = steps()
    torch.cuda.current_stream().wait_stream(side)
    assert entered == [pos.get_device()] * 5 and all(torch.equal(a, b) for a, b in zip(got, want))
    swa.device_status()


@pytest.mark.parametrize("B,G,P", [(3, 12, 200), (3, 12, 5000), (2, 70, 3000), (9, 20, 3000)])
def test_a_strided_prefix_of_more_than_8_query_heads(B, G, P):
    """A slice of a [P,Hkv,D] buffer whose other rows hold NaN, read by splits of the slots' kernel
    and the prefix's with one and two row tiles."""
    Hkv, D, S = 2, 128, 90
    g = gen(P + G)
    q, kc, vc = rand(g, B, Hkv * G, D), rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    buf = torch.full((2, P + 90, Hkv, D), math.nan, dtype=BF, device=DEV)
    buf[:, 30:30 + P] = rand(g, 2, P, Hkv, D)
    kp, vp = (buf[x, 30:30 + P].transpose(0, 1) for x in range(2))
    pos = torch.randint(0, 2 * S, (B,), generator=g, device=DEV)
    out = swa.prefix_decode(q, kp, vp, kc, vc, pos, S)
    want, spread, _, ez = ref.decode(q, kc, vc, pos, kp, vp)
    assert bool(((out.double() - want).abs() <= ref.decode_tol(want, spread, ez, P + S, 2.0 ** -16)).all())
    assert torch.equal(out, swa.prefix_decode(q, kp.contiguous(), vp.contiguous(), kc, vc, pos, S))
    swa.device_status()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_key_weights_of_one_key_repeated(dtype):
    """Keys and queries expanded along the tokens (stride 0): as their copies."""
    B, H, T, D, W = 2, 2, 300, 64, 77
    g = gen(4)
    q, k = rand(g, B, H, 1, D, dtype=dtype).expand(B, H, T, D), rand(g, B, H, 1, D, dtype=dtype).expand(B, H, T, D)
    lse = band_lse(q, k, W)
    w = swa.key_weights(q, k, lse, W)
    assert torch.equal(w, swa.key_weights(q.contiguous(), k.contiguous(), lse, W))
    want, bound = ref.key_weights(q, k, lse, W)
    assert bool(((w.double() - want).abs() <= bound + want * ref.U32).all())
    swa.device_status()


def test_seed_of_one_row_repeated():
    B, Hkv, T, D, S = 2, 3, 500, 128, 40
    g = gen(5)
    k, v = (rand(g, B, Hkv, 1, D).expand(B, Hkv, T, D) for _ in range(2))
    w = torch.rand(B, Hkv, T, generator=g, device=DEV)
    caches = [[torch.zeros(B, Hkv, S, D, dtype=BF, device=DEV) for _ in range(2)] +
              [torch.zeros(B, Hkv, S, device=DEV), torch.zeros(B, Hkv, S, dtype=torch.int64, device=DEV)] for _ in range(2)]
    swa.cache_seed(k, v, w, *caches[0], 7)
    swa.cache_seed(k.contiguous(), v.contiguous(), w, *caches[1], 7)
    assert all(torch.equal(a, b) for a, b in zip(*caches))
    swa.device_status()
