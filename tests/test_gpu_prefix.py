"""The shared prefix's kernel where a whole batch's rows are 129 and more to a key head (two row
tiles a CTA) and where a CTA takes many key tiles: rows that few keys dominate, every key once,
reference values that move far. Bounds are roundings counted, none fitted."""
import math

import pytest
import torch

import serving_ref as ref
import sliding_window_causal_b200 as swa
from test_gpu_serving import BF, DEV, gen, heavy, rand

pytestmark = pytest.mark.gpu


def exact_rows(q, kc, vc, pos, kp, vp, c=None):
    """(out, spread, gain, ez) in float64: out, the sums of p |v|, the weight that each slot gets,
    and how far fp32 scores may move an exponent."""
    B, H, D = q.shape
    Hkv, S = kc.shape[1], kc.shape[2]
    G, c = H // Hkv, 1 / math.sqrt(D) if c is None else c
    out, spread = (torch.zeros(B, H, D, dtype=torch.float64, device=DEV) for _ in range(2))
    gain = torch.zeros(B, Hkv, S, dtype=torch.float64, device=DEV)
    ez = 0.0
    for b in range(B):
        n = min(int(pos[b]) + 1, S)
        for hk in range(Hkv):
            ks, vs = (torch.cat([p[hk], r[b, hk, :n]]).double() for p, r in ((kp, kc), (vp, vc)))
            qd = q[b, hk * G:(hk + 1) * G].double()
            p = torch.softmax(c * (qd @ ks.T), 1)
            out[b, hk * G:(hk + 1) * G] = p @ vs
            spread[b, hk * G:(hk + 1) * G] = p @ vs.abs()
            gain[b, hk, :n] = p[:, -n:].sum(0)
            ez = max(ez, (D + 4) * ref.U32 * c * float((qd.abs() @ ks.abs().T).max()))
    return out, spread, gain, ez


TWO_PARTS = 2.0 ** -16  # a weight as hi + lo bf16 parts, relative


@pytest.mark.parametrize("B,Hkv,G,D,S,P,scale", [
    (100, 2, 3, 64, 33, 1500, 4), (40, 2, 4, 128, 20, 4000, 8), (48, 1, 4, 128, 9, 9000, 8), (200, 2, 2, 64, 1, 3000, 8),
    (129, 1, 1, 128, 5, 3300, 16)])
def test_rows_that_few_keys_dominate(B, Hkv, G, D, S, P, scale):
    """Queries scaled up, so that one or a few keys hold most of a row's weight: the bounds of two
    parts and the 1e-2 of the other bf16 calls, whatever the number of rows."""
    g = gen(B + P + scale)
    q = rand(g, B, Hkv * G, D, scale=float(scale))
    kc, vc, kp, vp = rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D), rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    pos = torch.randint(0, 2 * S, (B,), generator=g, device=DEV)
    want, spread, gain, ez = exact_rows(q, kc, vc, pos, kp, vp)
    tol = ref.decode_tol(want, spread, ez, P + S, TWO_PARTS)
    before = heavy(g, B, Hkv, S)
    after = before.clone()
    for out in (swa.prefix_decode(q, kp, vp, kc, vc, pos, S), swa.cache_decode(q, kc, vc, after, pos, kp, vp)):
        off = (out.double() - want).abs()
        assert bool((off <= tol).all()), float((off / tol).max())
        assert float(off[want.abs() < 4].max()) <= 1e-2  # above 4 the steps of bf16 are coarser
    swa.device_status()
    # The slots' weights keep the fp32 sums: exponents and sums as in test_gpu_serving, and each of
    # the G probabilities below fp32's normal numbers may be taken as 0, so 2^-126 each.
    tol = ref.U32 * (before.double() + gain) * 2 + gain * (2 * ez + 2.0 ** -20 + (P + S + G) * ref.U32) + G * 2.0 ** -126
    off = (after.double() - (before.double() + gain)).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


@pytest.mark.parametrize("B,Hkv,G,D,S,P", [
    (200, 2, 2, 64, 5, 3000), (40, 2, 4, 128, 5, 30011),     # two row tiles a CTA: 2 and 5 key tiles each
    (9, 1, 1, 64, 5, 40001), (2, 1, 1, 128, 5, 140000),      # one row tile, alternate key tiles on two lanes
    (3, 1, 2, 64, 700, 100)])                                # the streams read it by themselves
def test_scores_that_rise_beyond_every_power_of_two(B, Hkv, G, D, S, P):
    """Scores that rise by 2^21 (powers of two) from one key tile to the next: a row's weight is
    all on the last tile's keys, in equal shares, and nothing of the others is left or infinite.
    Queries (1, 0, ..) and keys (tile, 0, ..) make every score exact."""
    g = gen(P)
    step = 2.0 ** 21 / math.log2(math.e)
    q = torch.zeros(B, Hkv * G, D, dtype=BF, device=DEV)
    q[..., 0] = 1
    tile = torch.arange(P, device=DEV) // 128
    kp = torch.zeros(Hkv, P, D, dtype=BF, device=DEV)
    kp[..., 0] = (tile - int(tile[-1])).clamp_min(-256).to(BF)  # whole numbers that bf16 holds
    vp, vc = rand(g, Hkv, P, D), rand(g, B, Hkv, S, D)
    kc = torch.zeros(B, Hkv, S, D, dtype=BF, device=DEV)
    kc[..., 0] = -1
    pos = torch.full((B,), S, device=DEV)
    for flip in (False, True):  # rising and falling
        if flip:
            kp, vp = kp.flip(1).contiguous(), vp.flip(1).contiguous()
        top = (kp[0, :, 0] == 0).nonzero().flatten()
        want = vp[:, top].double().mean(1)[None, :, None].expand(B, Hkv, G, D).reshape(B, Hkv * G, D)
        out = swa.prefix_decode(q, kp, vp, kc, vc, pos, S, scale=step)
        spread = vp[:, top].double().abs().mean(1)[None, :, None].expand(B, Hkv, G, D).reshape(B, Hkv * G, D)
        swa.device_status()
        tol = ref.decode_tol(want, spread, 0.0, 128, 2.0 ** -8)
        assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("B,Hkv,G,P", [(100, 2, 3, 1500), (24, 2, 4, 1100), (2, 2, 2, 100), (2, 1, 12, 300)])
def test_a_scale_below_fp32(B, Hkv, G, P):
    """A scale that fp32 holds only as 0 gives equal weights: the keys past a ragged end stay out."""
    D, S = 128, 9
    g = gen(P + 1)
    q, kp, vp = rand(g, B, Hkv * G, D), rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    kc, vc = rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    vs = torch.cat([vp.expand(B, Hkv, P, D), vc], 2).double()
    want = vs.mean(2).repeat_interleave(G, 1)
    tol = ref.decode_tol(want, vs.abs().mean(2).repeat_interleave(G, 1), 0.0, P + S, ref.UBF)
    for scale in (1e-38, 1e-46, 1e-300):
        out = swa.prefix_decode(q, kp, vp, kc, vc, torch.full((B,), S, device=DEV), S, scale=scale)
        assert bool(((out.double() - want).abs() <= tol).all()), scale
    swa.device_status()


def few_units(g, heads, n, D):
    """[heads, n, D] of -1, 0 and 1 in random order, whose columns sum to at most 100 in magnitude."""
    half = max(0, (n - 100) // 2)
    a = torch.randint(-1, 2, (heads, half, D), generator=g, device=DEV)
    v = torch.cat([a, -a, torch.randint(-1, 2, (heads, n - 2 * half, D), generator=g, device=DEV)], 1)
    return v[:, torch.randperm(n, generator=g, device=DEV)]


# B, Hkv, G, D, P; key tiles that a CTA takes, and what follows the prefix's kernel
MANY_TILES = [
    (40, 8, 4, 128, 33000),   # two row tiles, 15, then the streams
    (40, 8, 4, 64, 33001),    # 15
    (128, 8, 4, 128, 65536),  # 57
    (200, 4, 2, 64, 50003),   # 22
    (70, 1, 7, 128, 60011),   # 8, the streams beside it
    (33, 3, 12, 128, 20000),  # 7, then the splits of more than 8 heads
    (64, 8, 1, 64, 70001),    # one row tile on two lanes, 31, then the streams
    (64, 32, 1, 128, 8192),   # 16
    (2, 1, 1, 128, 140000),   # 9, the streams beside it
    (3, 2, 12, 64, 150001),   # then splits
]


@pytest.mark.parametrize("B,Hkv,G,D,P", MANY_TILES)
def test_every_key_of_a_long_prefix_counts_once(B, Hkv, G, D, P):
    """Queries of zeros give every key the same weight, 1, and values of -1, 0 and 1 make every sum
    a whole number of at most 120: one key lost, doubled or out of place changes its columns by
    1 in 120 or more, twice the step of bf16. Nothing but the output is rounded."""
    S = 20
    g = gen(P + B)
    q = torch.zeros(B, Hkv * G, D, dtype=BF, device=DEV)
    kp, kc = rand(g, Hkv, P, D), rand(g, B, Hkv, S, D)
    pv, sv = few_units(g, Hkv, P, D), torch.randint(-1, 2, (B, Hkv, S, D), generator=g, device=DEV)
    pos = torch.randint(0, 2 * S, (B,), generator=g, device=DEV)
    n = (pos + 1).clamp_max(S)
    seen = torch.arange(S, device=DEV) < n[:, None]
    total = pv.sum(1) + (sv * seen[:, None, :, None]).sum(2)
    assert int(total.abs().max()) <= 120
    want = (total.double() / (P + n)[:, None, None]).repeat_interleave(G, 1)
    wc = torch.zeros(B, Hkv, S, device=DEV)
    vp, vc = pv.to(BF), sv.to(BF)
    for out in (swa.prefix_decode(q, kp, vp, kc, vc, pos, S), swa.cache_decode(q, kc, vc, wc, pos, kp, vp)):
        off = (out.double() - want).abs()
        assert bool((off <= want.abs() * (ref.UBF + 2.0 ** -16)).all()), int((off > want.abs() * 0.004).sum())
    gain = torch.where(seen, G / (P + n).double()[:, None], 0.0)[:, None].expand(B, Hkv, S)
    assert bool(((wc.double() - gain).abs() <= gain * 2.0 ** -18).all())  # log2 and exp2 of 18 bits and less
    swa.device_status()


@pytest.mark.parametrize("scale", [None, 1.0])
@pytest.mark.parametrize("B,Hkv,G,D,P", MANY_TILES)
def test_scores_that_grow_along_a_long_prefix(B, Hkv, G, D, P, scale):
    """Scores that rise by 0.3 to 10 (powers of two) a key tile, so that a CTA moves its reference in
    tiles after its first ones: a few streams in float64, the others by repeating the call."""
    S = 30
    g = gen(P + D)
    q = rand(g, B, Hkv * G, D).abs() + 1
    ramp = torch.linspace(-3, 3, P, device=DEV)[:, None]
    kp = (rand(g, Hkv, P, D).float() * 0.1 + ramp).to(BF)
    kc, vp, vc = rand(g, B, Hkv, S, D), rand(g, Hkv, P, D), rand(g, B, Hkv, S, D)
    pos = torch.randint(0, 2 * S, (B,), generator=g, device=DEV)
    for _ in range(2):
        out = swa.prefix_decode(q, kp, vp, kc, vc, pos, S, scale=scale)
        assert torch.equal(out, swa.prefix_decode(q, kp, vp, kc, vc, pos, S, scale=scale))
        some = [0, B // 2, B - 1]
        c = 1 / math.sqrt(D) if scale is None else scale
        want, spread, _, ez = exact_rows(q[some], kc[some], vc[some], pos[some], kp, vp, c)
        off = (out[some].double() - want).abs()
        tol = ref.decode_tol(want, spread, ez, 2000, TWO_PARTS)  # additions in a row: 16 products a tile, 57 tiles, and joins
        assert bool((off <= tol).all()), float((off / tol).max())
        kp, vp = kp.flip(1).contiguous(), vp.flip(1).contiguous()
    swa.device_status()


@pytest.mark.parametrize("B,Hkv,G,D,S,P", [
    (130, 1, 1, 128, 3, 257), (32, 2, 8, 64, 31, 640), (100, 2, 3, 64, 33, 700),       # the streams read them by themselves
    (100, 2, 3, 64, 33, 1500), (70, 1, 7, 128, 900, 2500), (200, 2, 2, 64, 1, 3000),   # a kernel of its own
    (128, 1, 1, 128, 8, 3000), (129, 1, 1, 128, 8, 3000)])
def test_weights_of_many_rows_keep_two_parts(B, Hkv, G, D, S, P):
    """More than 128 rows share these prefixes, whichever kernel takes them: 2^-16 of a weight."""
    g = gen(B + P)
    q, kp, vp = rand(g, B, Hkv * G, D), rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    kc, vc = rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    pos = torch.randint(0, 2 * S, (B,), generator=g, device=DEV)
    want, spread, _, ez = ref.decode(q, kc, vc, pos, kp, vp)
    off = (swa.prefix_decode(q, kp, vp, kc, vc, pos, S).double() - want).abs()
    assert bool((off <= ref.decode_tol(want, spread, ez, P + S, TWO_PARTS)).all())
    swa.device_status()


@pytest.mark.parametrize("D,P", [(64, 33001), (128, 30011)])
def test_a_stream_does_not_depend_on_its_neighbours(D, P):
    """Rows of 40 streams share tiles and warps: another stream's queries must not change a bit of
    this one's output."""
    B, Hkv, G, S = 40, 2, 4, 10
    g = gen(P)
    q, kp, vp = rand(g, B, Hkv * G, D), rand(g, Hkv, P, D), rand(g, Hkv, P, D)
    kc, vc = rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D)
    pos = torch.full((B,), 2 * S, device=DEV)
    a = swa.prefix_decode(q, kp, vp, kc, vc, pos, S)
    q[::2] *= 8
    b = swa.prefix_decode(q, kp, vp, kc, vc, pos, S)
    assert torch.equal(a[1::2], b[1::2]) and not torch.equal(a[::2], b[::2])
    swa.device_status()


@pytest.mark.parametrize("P", [4000, 30011])
def test_two_streams_at_once_and_replayed(P):
    """More than 128 rows to a key head: calls on two streams with workspaces of their own, and the
    same calls captured into two graphs that replay side by side, equal calls alone."""
    B, Hkv, G, D, S = 40, 2, 4, 128, 200
    g = gen(P + 7)
    sets = [(rand(g, B, Hkv * G, D), rand(g, Hkv, P, D), rand(g, Hkv, P, D), rand(g, B, Hkv, S, D), rand(g, B, Hkv, S, D),
             torch.randint(0, 2 * S, (B,), generator=g, device=DEV)) for _ in range(2)]
    want = [swa.prefix_decode(*s, S) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for x in range(2):
            with torch.cuda.stream(streams[x]):
                outs[x].append(swa.prefix_decode(*sets[x], S))
    torch.cuda.synchronize()
    graphs, kept = [], []
    for x in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=streams[x]):
            kept.append([swa.prefix_decode(*sets[x], S) for _ in range(5)])
        graphs.append(gr)
    for _ in range(3):
        for o in kept[0] + kept[1]:
            o.zero_()
        torch.cuda.synchronize()
        for x in range(2):
            with torch.cuda.stream(streams[x]):
                graphs[x].replay()
        torch.cuda.synchronize()
        for x in range(2):
            assert all(torch.equal(o, want[x]) for o in outs[x] + kept[x])
    swa.device_status()
