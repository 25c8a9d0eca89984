"""The plain float64 forms that the serving tests compare with, pinned on the CPU: to the oracle
where it covers the same case, to closed forms elsewhere."""
import math

import numpy as np
import torch

import oracle
import serving_ref as ref


def rand(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def test_decode_without_prefix_is_the_ring_decode():
    B, H, D, W = 3, 2, 16, 7
    q, k, v = rand(B, H, D, seed=1), rand(B, H, W, D, seed=2), rand(B, H, W, D, seed=3)
    pos = torch.tensor([0, 4, 50])
    out = ref.decode(q, k, v, pos)[0]
    want = oracle.decode(q.double().numpy(), k.double().numpy(), v.double().numpy(), pos.numpy(), W)
    assert np.abs(out.numpy() - want).max() < 1e-12


def test_prefix_keys_are_as_keys_of_the_ring():
    B, H, D, P, n = 2, 4, 8, 5, 3
    q = rand(B, H, D, seed=4)
    kp, vp = rand(2, P, D, seed=5), rand(2, P, D, seed=6)
    k, v = rand(B, 2, n, D, seed=7), rand(B, 2, n, D, seed=8)
    pos = torch.full((B,), n - 1)
    a = ref.decode(q, k, v, pos, kp, vp)
    whole_k = torch.cat([kp.expand(B, 2, P, D), k], 2)
    whole_v = torch.cat([vp.expand(B, 2, P, D), v], 2)
    b = ref.decode(q, whole_k, whole_v, torch.full((B,), P + n - 1))
    assert (a[0] - b[0]).abs().max() < 1e-12
    assert (a[2] - b[2][:, :, P:]).abs().max() < 1e-12
    assert abs(float(b[2].sum()) - B * H) < 1e-12  # a query's probabilities sum to 1


def test_key_weights_sum_to_the_number_of_counted_queries():
    B, H, Hkv, T, D, W = 2, 4, 2, 23, 8, 6
    q, k = rand(B, H, T, D, seed=9), rand(B, Hkv, T, D, seed=10)
    kk = k.repeat_interleave(2, 1)
    d = torch.arange(T)[:, None] - torch.arange(T)[None]
    s = (q @ kk.transpose(2, 3) / math.sqrt(D)).masked_fill((d < 0) | (d >= W), -math.inf)
    lse = s.double().logsumexp(3).float()
    for last in (None, 1, 5, 100):
        w, bound = ref.key_weights(q, k, lse, W, last=last)
        assert (w.sum((1, 2)) - H * min(T, last or T)).abs().max() < 1e-4
        assert (bound >= 0).all()
    w, _ = ref.key_weights(q, k, lse, W, lens=torch.tensor([0, 9]))
    assert (w[0] == 0).all() and (w[1, :, 9:] == 0).all()
    assert abs(float(w[1].sum()) - 9 * H) < 1e-4


def test_choices():
    w = [3.0, 1.0, math.nan, 1.0, -0.0, 0.0, 9.0, 2.0]
    assert ref.seed_choice(w, 8, 4, 1) == [0, 2, 6, 7]
    assert ref.seed_choice(w, 8, 5, 1) == [0, 1, 2, 6, 7]      # 1 and 3 tie: the lower
    assert ref.seed_choice(w, 3, 4, 2) == [0, 1, 2]
    assert ref.append_slot([2.0, math.nan, 0.0, -0.0], [3, 0, 1, 2], 4, 4, 1) == 2  # -0 ties with 0
    assert ref.append_slot([2.0, 1.0, 0.0, 0.5], [0, 1, 3, 2], 4, 4, 2) == 3        # 3 is recent
    assert ref.append_slot([2.0, 1.0, 0.0, 0.5], [0, 1, 4, 2], 4, 4, 2) == 2        # held already
    assert ref.append_slot([0.0] * 4, [9, 9, 9, 9], 5, 4, 0) == -1
    assert ref.append_slot([0.0] * 4, [0] * 4, 3, 4, 0) == 3 and ref.append_slot([0.0], [0], -1, 1, 0) == -1
