"""GPU parity of the shared-prefix decode and of the budget cache against plain float64 forms.
The tolerances are the error bounds of serving_ref: roundings counted, none fitted."""
import math

import pytest
import torch

import serving_ref as ref
import sliding_window_causal_b200 as swa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


# -------------------------------------------------------------------------- key weights
def band_lse(q, k, W, scale=None):
    """The log-sum-exp of every row, rounded to fp32, in blocks of rows."""
    B, H, T, D = q.shape
    kd = k.double().repeat_interleave(H // k.shape[1], 1)
    out = torch.empty(B, H, T, device=DEV)
    c = 1 / math.sqrt(D) if scale is None else scale
    for i0 in range(0, T, 512):
        i1 = min(T, i0 + 512)
        d = torch.arange(i0, i1, device=DEV)[:, None] - torch.arange(T, device=DEV)
        s = (q[:, :, i0:i1].double() @ kd.transpose(2, 3)) * c
        out[:, :, i0:i1] = s.masked_fill((d < 0) | (d >= W), -math.inf).logsumexp(3).float()
    return out


def check_key_weights(q, k, lse, W, **kw):
    w = swa.key_weights(q, k, lse, W, **kw)
    swa.device_status()
    want, bound = ref.key_weights(q, k, lse, W, **kw)
    off = (w.double() - want).abs()
    assert bool((off <= bound + want * ref.U32).all()), float((off - bound).max())
    return w


KEY_CASES = [
    # B, Hkv, G, T, D, W, last, ragged, dtype
    (1, 1, 1, 1, 64, 1, None, False, BF),
    (2, 2, 1, 2, 128, 5, None, False, BF),
    (1, 2, 3, 63, 64, 64, None, False, BF),
    (1, 1, 2, 64, 128, 1, None, False, BF),
    (2, 1, 1, 65, 128, 17, 1, False, BF),
    (1, 2, 1, 128, 64, 128, None, False, BF),
    (1, 1, 1, 129, 128, 128, None, False, BF),
    (2, 2, 2, 300, 128, 77, None, True, BF),
    (1, 1, 8, 777, 64, 200, 33, True, BF),
    (3, 1, 4, 1025, 128, 512, None, True, BF),
    (1, 2, 1, 1500, 64, 1500, 64, False, BF),
    (2, 1, 2, 1111, 128, 257, 300, True, BF),
    (1, 1, 1, 4100, 128, 4096, None, False, BF),
    (4, 8, 1, 1300, 64, 40, None, True, BF),       # more key tiles than CTAs
    (6, 8, 1, 1000, 128, 130, 20, True, BF),       # most of them seen by no counted query
    (7, 7, 1, 900, 128, 300, 1, True, BF),         # one slice a tile
    (1, 1, 1, 1, 1, 1, None, False, torch.float32),
    (2, 2, 2, 70, 40, 9, None, True, torch.float32),
    (1, 1, 1, 333, 80, 100, 50, False, torch.float32),
    (1, 3, 1, 130, 300, 64, None, False, torch.float32),
]


@pytest.mark.parametrize("B,Hkv,G,T,D,W,last,ragged,dtype", KEY_CASES)
def test_key_weights(B, Hkv, G, T, D, W, last, ragged, dtype):
    g = gen(T + D + W)
    q, k = rand(g, B, Hkv * G, T, D, dtype=dtype), rand(g, B, Hkv, T, D, dtype=dtype)
    lens = torch.randint(0, T + 1, (B,), generator=g, device=DEV) if ragged else None
    w = check_key_weights(q, k, band_lse(q, k, W), W, lens=lens, last=last)
    assert torch.equal(w, swa.key_weights(q, k, band_lse(q, k, W), W, lens=lens, last=last))


def test_key_weights_takes_the_forward_lse_and_strides():
    """q and k as views of [B,T,H,D] tensors, another scale, the lse of the training forward."""
    B, H, T, D, W = 2, 2, 257, 128, 100
    g = gen(5)
    q, k, v = (rand(g, B, T, H, D).transpose(1, 2) for _ in range(3))
    _, lse = swa.forward_lse(q.contiguous(), k.contiguous(), v.contiguous(), W, scale=0.2)
    w = check_key_weights(q, k, lse, W, scale=0.2)
    assert abs(float(w.sum()) - B * H * T) < 1e-3 * B * H * T


def test_key_weights_ignores_padding():
    """Rows at or past a stream's length may hold anything; keys there get 0."""
    B, H, T, D, W = 3, 2, 200, 64, 90
    g = gen(6)
    q, k = rand(g, B, H, T, D), rand(g, B, H, T, D)
    lse = band_lse(q, k, W)
    lens = torch.tensor([0, 131, 200], device=DEV)
    want = check_key_weights(q, k, lse, W, lens=lens)
    for b, n in enumerate(lens.tolist()):
        q[b, :, n:], k[b, :, n:], lse[b, :, n:] = math.nan, math.inf, math.nan
        assert bool((want[b, :, n:] == 0).all())
    assert torch.equal(swa.key_weights(q, k, lse, W, lens=lens), want)
    swa.device_status()


def test_key_weights_of_sharp_rows():
    """Scores of +-100: weights near 1 and far below fp32's range, none lost or infinite."""
    B, H, T, D, W = 1, 2, 300, 64, 128
    g = gen(7)
    q, k = rand(g, B, H, T, D, scale=4.0), rand(g, B, H, T, D, scale=4.0)
    check_key_weights(q, k, band_lse(q, k, W), W)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_key_weights_reports_a_length_out_of_range(dtype):
    g = gen(8)
    q, k = rand(g, 3, 1, 40, 64, dtype=dtype), rand(g, 3, 1, 40, 64, dtype=dtype)
    lse = band_lse(q, k, 7)
    w = swa.key_weights(q, k, lse, 7, lens=torch.tensor([41, 40, -1], device=DEV))
    with pytest.raises(swa.SwaError) as e:
        swa.device_status()
    assert e.value.code == 1
    assert bool((w[0] == 0).all()) and bool((w[2] == 0).all())
    assert torch.equal(w[1], swa.key_weights(q, k, lse, 7)[1])


def test_key_weights_empty():
    e = torch.empty(2, 4, 0, 64, dtype=BF, device=DEV)
    assert swa.key_weights(e, e, torch.empty(2, 4, 0, device=DEV), 3).shape == (2, 4, 0)
    swa.device_status()


# -------------------------------------------------------------------------- seed
def heavy(g, *shape):
    w = torch.exp(2 * torch.randn(shape, generator=g, device=DEV) - 2)
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.1, 0.0, w)


def empty_cache(B, Hkv, S, D):
    """A cache whose slots hold marks that a call must leave or replace."""
    return (torch.full((B, Hkv, S, D), 7.0, device=DEV, dtype=BF), torch.full((B, Hkv, S, D), -7.0, device=DEV, dtype=BF),
            torch.full((B, Hkv, S), 3.5, device=DEV), torch.full((B, Hkv, S), -9, device=DEV, dtype=torch.int64))


def check_seed(k, v, w, S, recent, lens=None):
    B, Hkv, T, D = k.shape
    cache = empty_cache(B, Hkv, S, D)
    want = [t.clone() for t in cache]
    swa.cache_seed(k, v, w, *cache, recent, lens=lens)
    swa.device_status()
    wh = w.cpu()
    for b in range(B):
        n = T if lens is None else int(lens[b])
        for h in range(Hkv):
            kept = torch.tensor(ref.seed_choice(wh[b, h].tolist(), n, S, recent), dtype=torch.int64, device=DEV)
            m = len(kept)
            want[0][b, h, :m], want[1][b, h, :m] = k[b, h, kept], v[b, h, kept]
            want[2][b, h, :m], want[3][b, h, :m] = w[b, h, kept], kept
    for a, c in zip(cache, want):
        assert torch.equal(a.nan_to_num(1e30) if a.is_floating_point() else a,
                           c.nan_to_num(1e30) if c.is_floating_point() else c)
    return cache


@pytest.mark.parametrize("B,Hkv,T,D,S,recent,ragged", [
    (1, 1, 1, 64, 1, 0, False), (2, 3, 5, 128, 1, 0, True), (1, 2, 100, 64, 100, 10, False), (2, 1, 101, 64, 100, 99, False),
    (3, 2, 700, 128, 33, 7, True), (2, 2, 5000, 64, 1024, 128, True), (1, 3, 16384, 128, 2000, 256, False),
    (2, 1, 1023, 64, 1022, 0, False), (1, 1, 70000, 64, 4096, 1, False), (1, 2, 40000, 64, 31000, 5000, False),
])
def test_cache_seed(B, Hkv, T, D, S, recent, ragged):
    g = gen(T + S)
    k, v, w = rand(g, B, Hkv, T, D), rand(g, B, Hkv, T, D), heavy(g, B, Hkv, T)
    lens = torch.randint(0, T + 1, (B,), generator=g, device=DEV) if ragged else None
    check_seed(k, v, w, S, recent, lens)


def test_cache_seed_orders_weights_as_numbers():
    """Ties, zeros of both signs, infinities, negative weights and NaN; every weight equal."""
    g = gen(11)
    T, S, D = 500, 120, 64
    k, v = rand(g, 1, 4, T, D), rand(g, 1, 4, T, D)
    pool = torch.tensor([0.0, -0.0, 1.0, 1.0, math.inf, -math.inf, math.nan, -math.nan, -2.5, 1e-40, 3e38], device=DEV)
    w = pool[torch.randint(0, len(pool), (1, 4, T), generator=g, device=DEV)]
    w[:, 1], w[:, 2] = 0.0, math.nan
    check_seed(k, v, w, S, 20)


def test_cache_seed_strided_inputs():
    g = gen(12)
    k, v = rand(g, 2, 300, 3, 64).transpose(1, 2), rand(g, 2, 300, 3, 64).transpose(1, 2)
    check_seed(k, v, heavy(g, 2, 3, 300), 50, 5)


def test_cache_seed_reports_a_length_out_of_range():
    g = gen(13)
    k, v, w = rand(g, 3, 2, 40, 64), rand(g, 3, 2, 40, 64), heavy(g, 3, 2, 40)
    cache = empty_cache(3, 2, 8, 64)
    marks = [t.clone() for t in cache]
    swa.cache_seed(k, v, w, *cache, 2, lens=torch.tensor([-1, 20, 41], device=DEV))
    with pytest.raises(swa.SwaError) as e:
        swa.device_status()
    assert e.value.code == 1
    for a, m in zip(cache, marks):
        assert torch.equal(a[0], m[0]) and torch.equal(a[2], m[2]) and not torch.equal(a[1], m[1])


# -------------------------------------------------------------------------- append
def check_append(cache, pos, recent, g):
    kc, vc, wc, pc = cache
    B, Hkv, S, D = kc.shape
    k, v = rand(g, B, Hkv, D), rand(g, B, Hkv, D)
    want = [t.clone() for t in cache]
    slots = swa.cache_append(k, v, *cache, pos, recent)
    expect = torch.empty(B, Hkv, dtype=torch.int64)
    for b in range(B):
        for h in range(Hkv):
            s = ref.append_slot(want[2][b, h].tolist(), want[3][b, h].tolist(), int(pos[b]), S, recent)
            expect[b, h] = s
            if s >= 0:
                want[0][b, h, s], want[1][b, h, s] = k[b, h], v[b, h]
                want[2][b, h, s], want[3][b, h, s] = 0.0, int(pos[b])
    assert torch.equal(slots.cpu(), expect)
    for a, c in zip(cache, want):
        assert torch.equal(a.nan_to_num(1e30) if a.is_floating_point() else a,
                           c.nan_to_num(1e30) if c.is_floating_point() else c)


@pytest.mark.parametrize("B,Hkv,S,D,recent", [(1, 1, 1, 64, 0), (3, 2, 7, 128, 0), (2, 3, 33, 64, 32), (2, 1, 1001, 64, 33),
                                              (5, 4, 2100, 128, 512), (1, 2, 20000, 64, 100)])
def test_cache_append(B, Hkv, S, D, recent):
    g = gen(S + recent)
    pos = torch.randint(S, S + 50000, (B,), generator=g, device=DEV)
    pos[0] = S // 2  # a stream that still has room
    cache = [rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D), heavy(g, B, Hkv, S), torch.zeros(B, Hkv, S, dtype=torch.int64, device=DEV)]
    for b in range(B):
        for h in range(Hkv):
            p = torch.randperm(int(pos[b]) + 1, generator=g, device=DEV)[:S] - 1  # some -1: older than all
            cache[3][b, h, :len(p)] = p
    check_append(cache, pos, recent, g)
    check_append(cache, pos, recent, g)      # again: the slot that holds the position
    check_append(cache, pos + 1, recent, g)


def test_cache_append_orders_weights_and_reports_full_heads():
    g = gen(21)
    S = 300
    pool = torch.tensor([0.0, -0.0, 1.0, math.inf, -math.inf, math.nan, -1.0, 1e-42], device=DEV)
    cache = [rand(g, 1, 4, S, 64), rand(g, 1, 4, S, 64), pool[torch.randint(0, 8, (1, 4, S), generator=g, device=DEV)],
             torch.randint(0, 900, (1, 4, S), generator=g, device=DEV)]
    cache[2][:, 0] = math.nan
    cache[2][:, 1] = 0.0
    check_append(cache, torch.tensor([1000], device=DEV), 100, g)
    swa.device_status()
    cache[3][:, 2] = 1500  # every position too new: this head has no slot to give
    check_append(cache, torch.tensor([1001], device=DEV), 100, g)
    with pytest.raises(swa.SwaError) as e:
        swa.device_status()
    assert e.value.code == 1
    check_append(cache, torch.tensor([-3], device=DEV), 100, g)
    with pytest.raises(swa.SwaError):
        swa.device_status()


# -------------------------------------------------------------------------- decode


def check_decode(q, kc, vc, pos, kp=None, vp=None, scale=None, wc=None, **kw):
    """One call through the package, with or without weights, against float64."""
    S = kc.shape[2]
    # Softmax weights are carried as two bf16 parts (2 ** -16 of a weight), except over a prefix
    # that more than 128 query rows share: there as one, each weight off by half a step of bf16,
    # 2 ** -8 of itself, so an output sum p (1 + e) v by at most 2 ** -8 of sum p |v|.
    p_step = ref.UBF if kp is not None and q.shape[0] * (q.shape[1] // kc.shape[1]) > 128 else 2.0 ** -16
    want, spread, gain, ez = ref.decode(q, kc, vc, pos, kp, vp, scale)
    keys = S + (0 if kp is None else kp.shape[1])
    if wc is None:
        out = swa.prefix_decode(q, kp, vp, kc, vc, pos, S, scale=scale, **kw)
    else:
        before = wc.clone()
        out = swa.cache_decode(q, kc, vc, wc, pos, kp, vp, scale=scale, **kw)
        got = wc.double()
        # one addition to the old weight, and each probability off by 2 ez and fp32 sums
        G = q.shape[1] // kc.shape[1]
        tol = ref.U32 * (before.double().abs() + gain) * 2 + gain * (2 * ez + 2.0 ** -20 + (keys + G) * ref.U32)
        off = (got - (before.double() + gain)).abs()
        assert bool((off <= tol).all()), float((off - tol).max())
        assert torch.equal(wc[gain == 0], before[gain == 0])
    swa.device_status()
    off = (out.double() - want).abs()
    tol = ref.decode_tol(want, spread, ez, keys, p_step)
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-30)).max())
    return out


DECODE_CASES = [
    # B, Hkv, G, D, S, P
    (1, 1, 1, 64, 1, 0), (1, 1, 1, 128, 1, 1), (3, 2, 1, 64, 5, 7), (2, 1, 3, 128, 16, 15), (2, 3, 8, 64, 17, 33),
    (4, 2, 1, 128, 100, 300), (5, 1, 9, 64, 64, 129), (8, 2, 4, 128, 130, 1000), (3, 2, 2, 64, 1001, 0),
    (24, 1, 4, 128, 333, 2000), (33, 2, 1, 64, 40, 777), (130, 1, 1, 128, 3, 257), (64, 1, 5, 64, 20, 4100),
    (2, 1, 1, 128, 5000, 9), (100, 2, 8, 128, 9, 1500), (1, 1, 70, 64, 129, 128), (16, 1, 1, 128, 64, 128),
    (32, 2, 8, 64, 31, 640),
    # prefixes too long for each stream to read by itself
    (24, 2, 4, 128, 50, 1100), (60, 2, 2, 64, 70, 2100), (100, 2, 3, 64, 33, 700), (16, 1, 8, 128, 40, 4000),
    (2, 1, 1, 128, 30, 140000), (3, 2, 12, 64, 500, 5000), (9, 1, 1, 64, 100, 40001), (40, 8, 1, 128, 600, 300),
    (100, 2, 3, 64, 33, 1500), (70, 1, 7, 128, 900, 2500), (200, 2, 2, 64, 1, 3000),
]


@pytest.mark.parametrize("B,Hkv,G,D,S,P", DECODE_CASES)
def test_decode_over_cache_ring_and_prefix(B, Hkv, G, D, S, P):
    g = gen(B + S + P + D)
    q = rand(g, B, Hkv * G, D)
    kc, vc = rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    kp, vp = (rand(g, Hkv, P, D), rand(g, Hkv, P, D)) if P else (None, None)
    pos = torch.randint(0, 3 * S, (B,), generator=g, device=DEV)
    pos[0] = 0
    a = check_decode(q, kc, vc, pos, kp, vp)
    wc = heavy(g, B, Hkv, S)
    b = check_decode(q, kc, vc, pos, kp, vp, wc=wc.clone())
    again = wc.clone()
    assert torch.equal(b, swa.cache_decode(q, kc, vc, again, pos, kp, vp))
    assert torch.equal(a, swa.prefix_decode(q, kp, vp, kc, vc, pos, S))


@pytest.mark.parametrize("G", [1, 40])
def test_decode_never_reads_slots_without_a_token(G):
    B, Hkv, D, S, P = 4, 2, 128, 300, 50
    g = gen(31)
    q, kc, vc, kp, vp = rand(g, B, Hkv * G, D), rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D), rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    pos = torch.tensor([0, 7, 200, 298], device=DEV)
    wc = heavy(g, B, Hkv, S)
    w1 = wc.clone()
    a, c = swa.prefix_decode(q, kp, vp, kc, vc, pos, S), swa.cache_decode(q, kc, vc, w1, pos, kp, vp)
    for b, p in enumerate(pos.tolist()):
        kc[b, :, p + 1:], vc[b, :, p + 1:] = math.nan, math.inf
    assert torch.equal(a, swa.prefix_decode(q, kp, vp, kc, vc, pos, S))
    w2 = wc.clone()
    assert torch.equal(c, swa.cache_decode(q, kc, vc, w2, pos, kp, vp)) and torch.equal(w1, w2)
    for b, p in enumerate(pos.tolist()):
        assert torch.equal(w2[b, :, p + 1:], wc[b, :, p + 1:])
    swa.device_status()


@pytest.mark.parametrize("B,G,P", [(2, 1, 200), (40, 4, 200), (40, 4, 1000), (20, 4, 2000), (40, 4, 2500)])
def test_decode_reads_a_strided_prefix_and_nothing_past_it(B, G, P):
    """A prefix that is a slice of a longer [P,Hkv,D] buffer whose other rows hold NaN."""
    Hkv, D, S = 3, 64, 20
    g = gen(32)
    q, kc, vc = rand(g, B, Hkv * G, D), rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    buf = torch.full((2, P + 90, Hkv, D), math.nan, dtype=BF, device=DEV)
    buf[:, 30:30 + P] = rand(g, 2, P, Hkv, D)
    kp, vp = (buf[x, 30:30 + P].transpose(0, 1) for x in range(2))
    pos = torch.randint(0, 50, (B,), generator=g, device=DEV)
    out = check_decode(q, kc, vc, pos, kp, vp)
    assert torch.equal(out, swa.prefix_decode(q, kp.contiguous(), vp.contiguous(), kc, vc, pos, S))


@pytest.mark.parametrize("B,G,P", [(1, 1, 300), (3, 8, 500), (80, 2, 700), (80, 2, 2000), (40, 2, 4000), (80, 2, 4000)])
def test_decode_of_sharp_and_growing_scores(B, G, P):
    """Scores that grow along the keys by hundreds, so that every running maximum is replaced
    many times, and rows where one key far outweighs the rest."""
    Hkv, D, S = 1, 64, 130
    g = gen(33)
    q = rand(g, B, G, D).abs() + 1
    ramp = torch.linspace(-3, 3, P + S, device=DEV)[:, None]
    keys = (rand(g, P + S, D).float() * 0.1 + ramp).to(BF)
    kp = keys[None, :P]
    kc = keys[None, None, P:].expand(B, 1, S, D).contiguous()
    vp, vc = rand(g, Hkv, P, D), rand(g, B, Hkv, S, D)
    pos = torch.randint(0, 2 * S, (B,), generator=g, device=DEV)
    check_decode(q, kc, vc, pos, kp, vp, wc=heavy(g, B, Hkv, S))
    check_decode(q, kc.flip(2).contiguous(), vc, pos, kp.flip(1).contiguous(), vp, scale=1.5)


def test_decode_reports_a_negative_position():
    B, H, D, S, P = 3, 2, 64, 16, 40
    g = gen(34)
    q, kc, vc, kp, vp = rand(g, B, H, D), rand(g, B, H, S, D), rand(g, B, H, S, D), rand(g, H, P, D), rand(g, H, P, D)
    wc = heavy(g, B, H, S)
    for call in (lambda p: swa.prefix_decode(q, kp, vp, kc, vc, p, S), lambda p: swa.cache_decode(q, kc, vc, w, p, kp, vp)):
        w = wc.clone()
        good = call(torch.tensor([5, 6, 70], device=DEV))
        swa.device_status()
        w = wc.clone()
        out = call(torch.tensor([5, -1, 70], device=DEV))
        with pytest.raises(swa.SwaError) as e:
            swa.device_status()
        assert e.value.code == 1
        assert bool((out[1] == 0).all()) and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        assert torch.equal(w[1], wc[1])


@pytest.mark.parametrize("B,G,P", [(2, 1, 0), (2, 9, 0), (2, 2, 100), (40, 2, 4000), (80, 2, 2000), (3, 12, 5000)])
def test_decode_of_nan_keys(B, G, P):
    """A NaN key that a query sees makes its output NaN, wherever the key is and also where every
    key of a split is NaN; the other streams' and heads' outputs do not change."""
    Hkv, D, S = 2, 64, 700
    g = gen(39)
    q, kc, vc = rand(g, B, Hkv * G, D), rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    kp, vp = (rand(g, Hkv, P, D), rand(g, Hkv, P, D)) if P else (None, None)
    pos = torch.full((B,), 2 * S, device=DEV)
    good = swa.prefix_decode(q, kp, vp, kc, vc, pos, S)
    for n in (1, 640):
        bad = kc.clone()
        bad[0, 1, :n] = math.nan
        wc = torch.zeros(B, Hkv, S, device=DEV)
        for out in (swa.prefix_decode(q, kp, vp, bad, vc, pos, S), swa.cache_decode(q, bad, vc, wc, pos, kp, vp)):
            assert bool(out[0, G:].isnan().all())
            assert torch.equal(out[0, :G], good[0, :G]) and torch.equal(out[1:], good[1:])
        assert bool(wc[0, 1].isnan().all()) and not bool(wc[0, 0].isnan().any()) and not bool(wc[1:].isnan().any())
    if P:
        bad = kp.clone()
        bad[1, P // 2] = math.nan
        out = swa.prefix_decode(q, bad, vp, kc, vc, pos, S)
        assert bool(out[:, G:].isnan().all()) and torch.equal(out[:, :G], good[:, :G])
    swa.device_status()


def test_decode_of_the_last_position():
    B, H, D, S = 2, 2, 64, 33
    g = gen(37)
    q, kc, vc = rand(g, B, H, D), rand(g, B, H, S, D), rand(g, B, H, S, D)
    far = torch.full((B,), torch.iinfo(torch.int64).max, device=DEV)
    assert torch.equal(swa.prefix_decode(q, None, None, kc, vc, far, S),
                       swa.prefix_decode(q, None, None, kc, vc, torch.full_like(far, S), S))
    swa.device_status()


def test_decode_of_broadcast_prefix_heads():
    """A prefix whose key heads are one head, expanded (stride 0), and an expanded prompt."""
    B, Hkv, G, D, S, P = 40, 4, 2, 64, 10, 3000
    g = gen(38)
    q, kc, vc = rand(g, B, Hkv * G, D), rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    kp, vp = (rand(g, 1, P, D).expand(Hkv, P, D) for _ in range(2))
    pos = torch.full((B,), 20, device=DEV)
    a = check_decode(q, kc, vc, pos, kp, vp)
    assert torch.equal(a, swa.prefix_decode(q, kp.contiguous(), vp.contiguous(), kc, vc, pos, S))
    k = rand(g, 1, 1, 300, D).expand(2, 3, 300, D)
    qq = rand(g, 2, 6, 300, D)
    lse = band_lse(qq, k, 50)
    assert torch.equal(swa.key_weights(qq, k, lse, 50), swa.key_weights(qq, k.contiguous(), lse, 50))
    swa.device_status()


def test_decode_offsets_past_32_bits():
    """The last stream of a cache of more than 2^31 elements a tensor."""
    B, S, D = 5, 1 << 22, 128
    g = gen(35)
    kc = torch.empty(B, 1, S, D, dtype=BF, device=DEV).normal_(generator=g)
    vc = torch.empty(B, 1, S, D, dtype=BF, device=DEV).normal_(generator=g)
    q, pos = rand(g, B, 1, D), torch.full((B,), 10 * S, device=DEV)
    wc = torch.zeros(B, 1, S, device=DEV)
    out = swa.cache_decode(q, kc, vc, wc, pos)
    swa.device_status()
    want, spread, gain, ez = ref.decode(q[-1:], kc[-1:], vc[-1:], pos[-1:])
    assert bool(((out[-1:].double() - want).abs() <= ref.decode_tol(want, spread, ez, S, 2.0 ** -16)).all())
    assert float((wc[-1:].double() - gain).abs().max()) <= float((gain * (2 * ez + 2.0 ** -19 + S * ref.U32)).max())
    slots = swa.cache_append(q[:, :1], q[:, :1], kc, vc, wc, torch.arange(S, device=DEV).expand(B, 1, S).contiguous(),
                             pos, 5)
    assert torch.equal(kc[-1, 0, slots[-1, 0]], q[-1, 0])
    swa.device_status()


def test_decode_workspace_and_out_of_the_caller():
    B, H, Hkv, D, S, P = 3, 18, 2, 64, 70, 90
    g = gen(36)
    q, kc, vc, kp, vp = rand(g, B, H, D), rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D), rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    pos = torch.tensor([3, 69, 500], device=DEV)
    need = swa.prefix_decode_workspace_bytes(B, H, Hkv, S, P, D)
    guard = 256
    buf = torch.full((need + guard,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    r = swa.prefix_decode(q, kp, vp, kc, vc, pos, S, out=out, workspace=buf[:need])
    assert r is out and torch.equal(out, swa.prefix_decode(q, kp, vp, kc, vc, pos, S))
    assert bool((buf[need:] == 0xA5).all())
    with pytest.raises(swa.SwaError):
        swa.prefix_decode(q, kp, vp, kc, vc, pos, S, workspace=buf[:max(need, 256) - 256])
    need = swa.cache_decode_workspace_bytes(B, H, Hkv, S, P, D)
    buf = torch.full((need + guard,), 0x5A, dtype=torch.uint8, device=DEV)
    w1, w2 = heavy(g, B, Hkv, S), None
    w2 = w1.clone()
    a = swa.cache_decode(q, kc, vc, w1, pos, kp, vp, workspace=buf[:need])
    assert torch.equal(a, swa.cache_decode(q, kc, vc, w2, pos, kp, vp)) and torch.equal(w1, w2)
    assert bool((buf[need:] == 0x5A).all())


# -------------------------------------------------------------------------- together
def serve(B, Hkv, G, D, T, S, recent, W, P, steps, seed):
    """A prompt behind a shared prefix into the cache, then tokens; every call is checked."""
    H = Hkv * G
    g = gen(seed)
    lens = torch.randint(1, T + 1, (B,), generator=g, device=DEV)
    q, k, v = rand(g, B, H, T, D), rand(g, B, Hkv, T, D), rand(g, B, Hkv, T, D)
    kp, vp = rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    wide = [t.repeat_interleave(G, 1).contiguous() for t in (k, v)]
    _, lse = swa.forward_lse(q, *wide, W)
    w = check_key_weights(q, k, lse, W, lens=lens)
    cache = check_seed(k, v, w, S, recent, lens)
    pos = lens.clone()
    for _ in range(steps):
        check_append(cache, pos, recent, g)
        check_decode(rand(g, B, H, D), cache[0], cache[1], pos, kp, vp, wc=cache[2])
        pos += 1
    held = cache[3]
    for b in range(B):
        n = int(pos[b])
        for h in range(Hkv):  # no position twice, and the newest are there
            p = held[b, h, :min(n, S)]
            assert len(set(p.tolist())) == len(p) and set(range(max(0, n - max(recent, 1)), n)) <= set(p.tolist())


def test_serving_a_prompt_and_its_tokens():
    serve(3, 2, 2, 64, 90, 40, 8, 64, 77, 12, 41)
    serve(2, 1, 1, 128, 300, 129, 0, 300, 130, 6, 42)


@pytest.mark.parametrize("P", [300, 5000])
def test_captured_steps_replay(P):
    """append + decode captured into a graph: two graphs of their own workspaces, replayed in
    turn on other data, give what plain calls give."""
    B, H, Hkv, D, S, recent = 6, 4, 2, 128, 50, 9
    g = gen(51)
    kp, vp = rand(g, Hkv, P, D), rand(g, Hkv, P, D)

    def fresh(seed):
        g = gen(seed)
        pos = torch.randint(S, 999, (B,), generator=g, device=DEV)
        pc = torch.stack([torch.randperm(S, generator=g, device=DEV) for _ in range(B * Hkv)]).view(B, Hkv, S)
        return dict(q=rand(g, B, H, D), k=rand(g, B, Hkv, D), v=rand(g, B, Hkv, D), kc=rand(g, B, Hkv, S, D),
                    vc=rand(g, B, Hkv, S, D), wc=heavy(g, B, Hkv, S), pc=pc, pos=pos)

    def step(s):
        slots = swa.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["wc"], s["pc"], s["pos"], recent)
        out = swa.cache_decode(s["q"], s["kc"], s["vc"], s["wc"], s["pos"], kp, vp)
        ring = swa.prefix_decode(s["q"], kp, vp, s["kc"], s["vc"], s["pos"], S)
        return slots, out, ring

    states = [fresh(52), fresh(53)]
    graphs = []
    for s in states:
        step(fresh(60))  # first calls outside the capture
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = step(s)
        graphs.append((gr, outs))
    for seeds in ((54, 55), (56, 57)):
        for s, seed in zip(states, seeds):
            for name, t in fresh(seed).items():
                s[name].copy_(t)
        for gr, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for s, (_, outs), seed in zip(states, graphs, seeds):
            plain = fresh(seed)
            want = step(plain)
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
            for name in ("kc", "vc", "wc", "pc"):
                assert torch.equal(s[name], plain[name])
    swa.device_status()


@pytest.mark.parametrize("P", [900, 9000])
def test_two_streams_at_once(P):
    """Calls on two streams with workspaces of their own, interleaved, equal calls alone."""
    B, H, D, S = 12, 8, 64, 700
    g = gen(61)
    sets = [(rand(g, B, H, D), rand(g, 8, P, D), rand(g, 8, P, D), rand(g, B, 8, S, D), rand(g, B, 8, S, D),
             torch.randint(0, 2000, (B,), generator=g, device=DEV)) for _ in range(2)]
    want = [swa.prefix_decode(*s, S) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for x in range(2):
            with torch.cuda.stream(streams[x]):
                outs[x].append(swa.prefix_decode(*sets[x], S))
    torch.cuda.synchronize()
    for x in range(2):
        assert all(torch.equal(o, want[x]) for o in outs[x])
    swa.device_status()


def test_empty_batches():
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device=DEV)
    pos = z(0, dtype=torch.int64)
    assert swa.prefix_decode(z(0, 4, 64), z(2, 5, 64), z(2, 5, 64), z(0, 2, 8, 64), z(0, 2, 8, 64), pos, 8).shape == (0, 4, 64)
    cache = (z(0, 2, 8, 64), z(0, 2, 8, 64), z(0, 2, 8, dtype=torch.float32), z(0, 2, 8, dtype=torch.int64))
    assert swa.cache_append(z(0, 2, 64), z(0, 2, 64), *cache, pos, 1).shape == (0, 2)
    assert swa.cache_decode(z(0, 4, 64), *cache[:3], pos).shape == (0, 4, 64)
    cache = empty_cache(1, 2, 8, 64)
    swa.cache_seed(z(1, 2, 0, 64), z(1, 2, 0, 64), z(1, 2, 0, dtype=torch.float32), *cache, 1)
    assert bool((cache[2] == 3.5).all())
    one = z(1, dtype=torch.int64)  # a prefix of no keys is no prefix
    r = z(1, 2, 8, 64) + 1
    assert torch.equal(swa.prefix_decode(z(1, 2, 64), z(2, 0, 64), z(2, 0, 64), r, r, one, 8), r[:, :, 0])
    swa.device_status()
