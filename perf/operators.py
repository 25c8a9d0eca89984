"""Measured cases of the serving operators beside the W-slot ring: a prefix shared by a whole
batch, and a cache of a fixed budget that forgets by accumulated attention weight.

    key_weights    the attention weight each key of a prompt received, summed over queries
    cache_seed     the budget cache after a prompt: the newest keys and the heaviest others
    cache_append   one new token per stream into the budget cache, evicting the lightest
    cache_decode   one query per stream over the budget cache (and a shared prefix),
                   the weights added to the cache's accumulators
    prefix_decode  one query per stream over a shared prefix and the stream's ring

Each runs in a plain form (elementary torch operations in fp32) or, with `own` set, through
the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a short fp32 prompt of a small model, head width that is no power of two
        dict(name="key_weights_small_f32", op="key_weights", B=2, H=4, G=1, T=777, D=80, W=200, last=0, ragged=False, f32=True),
        # a whole 16K prompt, every query counted: the prefill workload's shape
        dict(name="key_weights_prompt", op="key_weights", B=1, H=32, G=1, T=16384, D=128, W=4096, last=0, ragged=False, f32=False),
        # a padded batch of prompts, shared key heads, only the last 64 queries of each observed
        dict(name="key_weights_observed", op="key_weights", B=4, H=32, G=4, T=8191, D=128, W=4096, last=64, ragged=True, f32=False),
        # a 16K prompt cut to 2048 slots a head, 256 of them the newest tokens
        dict(name="cache_seed_prompt", op="cache_seed", B=1, Hkv=32, T=16384, D=128, S=2048, R=256, ragged=False),
        # a padded batch, some prompts shorter than the budget
        dict(name="cache_seed_ragged", op="cache_seed", B=16, Hkv=8, T=5000, D=64, S=1024, R=128, ragged=True),
        # 64 streams take their next token
        dict(name="cache_append_streams", op="cache_append", B=64, Hkv=32, D=128, S=4096, R=512),
        # a single stream, odd budget: launch latency
        dict(name="cache_append_single", op="cache_append", B=1, Hkv=8, D=64, S=1001, R=33),
        # the streaming decode workload with a budget cache in the ring's place
        dict(name="cache_decode_streams", op="cache_decode", B=64, H=32, G=1, D=128, S=4096, P=0),
        # a moderate batch with shared key heads and a system prompt
        dict(name="cache_decode_prefix", op="cache_decode", B=24, H=32, G=4, D=128, S=1000, P=2000),
        # two streams of a small model: launch latency
        dict(name="prefix_decode_few", op="prefix_decode", B=2, H=8, G=1, D=64, W=128, P=300),
        # 64 streams behind an 8K prefix, memory bound
        dict(name="prefix_decode_streams", op="prefix_decode", B=64, H=32, G=1, D=128, W=1024, P=8192),
        # 128 streams with shared key heads behind a 64K prefix: matrix products bound it
        dict(name="prefix_decode_long", op="prefix_decode", B=128, H=32, G=4, D=128, W=256, P=65536),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["key_weights", "cache_seed", "cache_append", "cache_decode", "prefix_decode"])
    D = rng.choice([64, 128])
    while True:
        if op == "key_weights":
            f32 = rng.random() < 0.25
            G = rng.choice([1, 1, 2, 4, 8])
            Hkv = rng.choice([1, 2, 3, 4, 8])
            T = _log(rng, 1, 2500 if f32 else 16384)
            c = dict(op=op, B=_log(rng, 1, 4), H=Hkv * G, G=G, T=T, D=rng.choice([16, 40, 64, 96]) if f32 else D,
                     W=_log(rng, 1, T), last=rng.choice([0, 0, min(T, _log(rng, 1, 256))]),
                     ragged=rng.random() < 0.5, f32=f32)
            most = 5.0e11 if not f32 else 1.0e10
        elif op == "cache_seed":
            S = _log(rng, 1, 4096)
            c = dict(op=op, B=_log(rng, 1, 16), Hkv=rng.choice([1, 2, 5, 8, 32]), T=_log(rng, 1, 16384), D=D, S=S,
                     R=rng.randrange(0, S), ragged=rng.random() < 0.5)
            most = 1.0e12
        elif op == "cache_append":
            S = _log(rng, 1, 8192)
            c = dict(op=op, B=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 5, 8, 32]), D=D, S=S, R=rng.randrange(0, S))
            most = 1.0e12
        else:
            G = rng.choice([1, 1, 2, 3, 4, 8])
            Hkv = rng.choice([1, 2, 5, 8])
            size = "S" if op == "cache_decode" else "W"
            c = dict(op=op, B=_log(rng, 1, 128), H=Hkv * G, G=G, D=D)
            c[size] = _log(rng, 1, 4096)
            c["P"] = 0 if op == "cache_decode" and rng.random() < 0.3 else _log(rng, 1, 32768)
            most = 1.3e11
        w = work(c)
        if w["flops"] <= most and w["bytes"] <= 4.0e9:
            return c


# ------------------------------------------------------------------------------- work
def _pairs(T, W, last):
    """Pairs (i, j) with T - last <= i < T and 0 <= i - j < W, j >= 0."""
    f = lambda n: n * (n + 1) // 2 if n <= W else W * (W + 1) // 2 + (n - W) * W
    return f(T) - f(T - last)


def _mean_len(case):
    """Ragged lengths are uniform in [T/2, T]; the expected counts use their mean."""
    return (3 * case["T"]) // 4 if case["ragged"] else case["T"]


def work(case):
    op = case["op"]
    if op == "key_weights":
        B, H, Hkv, D = case["B"], case["H"], case["H"] // case["G"], case["D"]
        n, e = _mean_len(case), 4 if case["f32"] else 2
        last = min(case["last"], n) if case["last"] else n
        keys = min(n, last + case["W"] - 1)  # keys that some counted query sees
        nbytes = B * H * last * (D * e + 4) + B * Hkv * keys * D * e + B * Hkv * case["T"] * 4
        return {"bytes": nbytes, "flops": 2 * D * B * H * _pairs(n, case["W"], last)}
    if op == "cache_seed":
        n = _mean_len(case)
        s = min(n, case["S"])
        return {"bytes": case["B"] * case["Hkv"] * (4 * n + s * (8 * case["D"] + 12)), "flops": case["B"] * case["Hkv"] * n}
    if op == "cache_append":
        return {"bytes": case["B"] * case["Hkv"] * (12 * case["S"] + 8 * case["D"] + 20),
                "flops": case["B"] * case["Hkv"] * case["S"]}
    B, H, Hkv, D, P = case["B"], case["H"], case["H"] // case["G"], case["D"], case["P"]
    S = case["S"] if op == "cache_decode" else case["W"]
    nbytes = Hkv * P * 4 * D + B * Hkv * S * (4 * D + (8 if op == "cache_decode" else 0)) + B * H * 4 * D
    return {"bytes": nbytes, "flops": 4 * B * H * (P + S) * D}


# ------------------------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype) if dtype != torch.bfloat16 else \
        torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _lens(g, B, T):
    return torch.randint((T + 1) // 2, T + 1, (B,), generator=g, device=DEV, dtype=torch.int64)


def _positions(g, B, Hkv, S, R, pos):
    """The positions that S slots of each head hold once a stream is at pos (its next token's
    position): all of 0 .. pos-1 in order below S, else the newest max(R - 1, 0), and others
    spread over the older ones, in any order of slots."""
    newest = max(R - 1, 0)
    old = S - newest
    room = (pos - newest).clamp_min(old).double()[:, None, None]
    i = torch.arange(old, device=DEV, dtype=torch.float64)
    u = torch.rand(B, Hkv, old, generator=g, device=DEV, dtype=torch.float64)
    lo = torch.floor(i * room / old)
    hi = torch.floor((i + 1) * room / old)
    older = (lo + torch.floor(u * (hi - lo))).to(torch.int64)
    new = (pos[:, None] - newest + torch.arange(newest, device=DEV))[:, None, :].expand(B, Hkv, newest)
    p = torch.cat([older, new], dim=2)
    order = torch.rand(B, Hkv, S, generator=g, device=DEV).argsort(dim=2)
    p = p.gather(2, order)
    return torch.where((pos < S)[:, None, None], torch.arange(S, device=DEV).expand(B, Hkv, S), p).contiguous()


def _heavy(g, *shape):
    """Accumulated attention weights: a few keys hold most of the mass; some are exactly 0."""
    w = torch.exp(2.0 * torch.randn(shape, generator=g, device=DEV) - 2.0)
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.05, torch.zeros_like(w), w)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "key_weights":
        B, H, Hkv, T, D, W = case["B"], case["H"], case["H"] // case["G"], case["T"], case["D"], case["W"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        s["q"], s["k"] = _randn(g, B, H, T, D, dtype=dt), _randn(g, B, Hkv, T, D, dtype=dt)
        s["lens"] = _lens(g, B, T) if case["ragged"] else None
        s["last"] = case["last"] or None
        # the forward pass's log-sum-exp of every row, which such a program already has
        k = s["k"].float().repeat_interleave(case["G"], dim=1)
        lse = torch.empty(B, H, T, device=DEV)
        for i0 in range(0, T, 1024):
            i1, j0 = min(T, i0 + 1024), max(0, i0 - W + 1)
            d = torch.arange(i0, i1, device=DEV)[:, None] - torch.arange(j0, i1, device=DEV)[None, :]
            sc = torch.matmul(s["q"][:, :, i0:i1].float(), k[:, :, j0:i1].transpose(2, 3)) / math.sqrt(D)
            lse[:, :, i0:i1] = sc.masked_fill((d < 0) | (d >= W), -math.inf).logsumexp(dim=3)
        s["lse"] = lse
    elif op == "cache_seed":
        B, Hkv, T, D, S = case["B"], case["Hkv"], case["T"], case["D"], case["S"]
        s["k"], s["v"] = _randn(g, B, Hkv, T, D), _randn(g, B, Hkv, T, D)
        s["weights"] = _heavy(g, B, Hkv, T)
        s["lens"] = _lens(g, B, T) if case["ragged"] else None
        s["kc"], s["vc"] = torch.zeros(B, Hkv, S, D, device=DEV, dtype=torch.bfloat16), torch.zeros(B, Hkv, S, D, device=DEV, dtype=torch.bfloat16)
        s["wc"], s["pc"] = torch.zeros(B, Hkv, S, device=DEV), torch.zeros(B, Hkv, S, device=DEV, dtype=torch.int64)
    elif op == "cache_append":
        B, Hkv, D, S, R = case["B"], case["Hkv"], case["D"], case["S"], case["R"]
        s["pos"] = torch.randint(0, 100000, (B,), generator=g, device=DEV, dtype=torch.int64)
        s["k"], s["v"] = _randn(g, B, Hkv, D), _randn(g, B, Hkv, D)
        s["kc"], s["vc"] = _randn(g, B, Hkv, S, D), _randn(g, B, Hkv, S, D)
        s["wc"], s["pc"] = _heavy(g, B, Hkv, S), _positions(g, B, Hkv, S, R, s["pos"])
    else:
        B, H, Hkv, D, P = case["B"], case["H"], case["H"] // case["G"], case["D"], case["P"]
        S = case["S"] if op == "cache_decode" else case["W"]
        s["pos"] = torch.randint(0, 100000, (B,), generator=g, device=DEV, dtype=torch.int64)
        s["q"] = _randn(g, B, H, D)
        s["kc"], s["vc"] = _randn(g, B, Hkv, S, D), _randn(g, B, Hkv, S, D)
        s["kp"], s["vp"] = (_randn(g, Hkv, P, D), _randn(g, Hkv, P, D)) if P else (None, None)
        if op == "cache_decode":
            s["wc"] = _heavy(g, B, Hkv, S)
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_key_weights(q, k, lse, W, G, lens, last):
    B, H, T, D = q.shape
    last = T if last is None else min(last, T)
    out = torch.zeros(B, H // G, T, device=DEV)
    kf = k.float().repeat_interleave(G, dim=1)
    n = lens if lens is not None else torch.full((B,), T, device=DEV)
    for r0 in range(0, last, 1024):  # rows in blocks, so that the scores fit in memory
        r1 = min(last, r0 + 1024)
        if lens is None:  # the rows are the same for every stream: a slice, and only its band's keys
            i = torch.arange(T - last + r0, T - last + r1, device=DEV)[None, :].expand(B, -1)
            j0, j1 = max(0, T - last + r0 - W + 1), T - last + r1
            qs, ls = q[:, :, T - last + r0:j1], lse[:, :, T - last + r0:j1]
        else:
            i = (n - last)[:, None] + torch.arange(r0, r1, device=DEV)
            j0, j1 = 0, T
            at = i.clamp_min(0)[:, None, :].expand(B, H, -1)
            qs, ls = q.gather(2, at[..., None].expand(-1, -1, -1, D)), lse.gather(2, at)
        d = i[:, :, None] - torch.arange(j0, j1, device=DEV)
        seen = ((d >= 0) & (d < W) & (i >= 0)[:, :, None])[:, None]
        p = torch.matmul(qs.float(), kf[:, :, j0:j1].transpose(2, 3)).div_(math.sqrt(D)).sub_(ls[..., None]).exp_()
        p = p.masked_fill_(~seen, 0.0).sum(dim=2)
        out[:, :, j0:j1] += p.view(B, H // G, G, j1 - j0).sum(dim=2)
    return out


def _plain_seed(k, v, weights, kc, vc, wc, pc, R, lens):
    B, Hkv, T, D = k.shape
    S = kc.shape[2]
    n = (lens if lens is not None else torch.full((B,), T, device=DEV))[:, None, None]
    j = torch.arange(T, device=DEV).expand(B, Hkv, T)
    rank = torch.where(j >= n - R, torch.full_like(weights, math.inf), weights)  # the newest are kept
    rank = torch.where(j >= n, torch.full_like(weights, -math.inf), rank)
    keep = min(S, T)
    kept = rank.sort(dim=2, descending=True, stable=True).indices[:, :, :keep].sort(dim=2).values
    real = kept < n  # at most min(n, S) of them; a sorted order puts them first
    at = kept[..., None].expand(-1, -1, -1, D)
    kc[:, :, :keep] = torch.where(real[..., None], k.gather(2, at), kc[:, :, :keep])
    vc[:, :, :keep] = torch.where(real[..., None], v.gather(2, at), vc[:, :, :keep])
    wc[:, :, :keep] = torch.where(real, weights.gather(2, kept), wc[:, :, :keep])
    pc[:, :, :keep] = torch.where(real, kept, pc[:, :, :keep])
    return kc, vc, wc, pc


def _plain_append(k, v, kc, vc, wc, pc, pos, R):
    B, Hkv, S, D = kc.shape
    p = pos[:, None, None]
    used = torch.arange(S, device=DEV) < p
    victim = torch.where(pc <= p - R, wc, torch.full_like(wc, math.inf)).argmin(dim=2)
    same = (pc == p) & used
    slot = torch.where(same.any(dim=2), same.int().argmax(dim=2), victim)
    slot = torch.where((pos < S)[:, None], pos[:, None], slot)
    at = slot[..., None]
    kc.scatter_(2, at[..., None].expand(-1, -1, 1, D), k[:, :, None])
    vc.scatter_(2, at[..., None].expand(-1, -1, 1, D), v[:, :, None])
    wc.scatter_(2, at, 0.0)
    pc.scatter_(2, at, p.expand(B, Hkv, 1))
    return slot, kc, vc, wc, pc


def _plain_attend(q, kc, vc, pos, kp, vp):
    """(out, probabilities of the cache's slots [B,Hkv,G,S])."""
    B, H, D = q.shape
    Hkv, S = kc.shape[1], kc.shape[2]
    G = H // Hkv
    qf = q.float().view(B, Hkv, G, D) / math.sqrt(D)
    sc = torch.matmul(qf, kc.float().transpose(2, 3))
    sc = sc.masked_fill(torch.arange(S, device=DEV) >= (pos + 1)[:, None, None, None], -math.inf)
    if kp is not None:
        rows = qf.transpose(0, 1).reshape(Hkv, B * G, D)
        sp = torch.matmul(rows, kp.float().transpose(1, 2)).view(Hkv, B, G, -1).transpose(0, 1)
        m = torch.maximum(sc.amax(dim=3), sp.amax(dim=3))[..., None]
        ep, es = torch.exp(sp - m), torch.exp(sc - m)
        z = ep.sum(dim=3, keepdim=True) + es.sum(dim=3, keepdim=True)
        o = torch.matmul(ep.transpose(0, 1).reshape(Hkv, B * G, -1), vp.float()).view(Hkv, B, G, D).transpose(0, 1)
        p = es / z
        out = o / z + torch.matmul(p, vc.float())
    else:
        es = torch.exp(sc - sc.amax(dim=3, keepdim=True))
        p = es / es.sum(dim=3, keepdim=True)
        out = torch.matmul(p, vc.float())
    return out.reshape(B, H, D).to(q.dtype), p


def run(state):
    s = state
    op = s["op"]
    if own:
        import sliding_window_causal_b200 as swa

        if op == "key_weights":
            return swa.key_weights(s["q"], s["k"], s["lse"], s["W"], lens=s["lens"], last=s["last"])
        if op == "cache_seed":
            swa.cache_seed(s["k"], s["v"], s["weights"], s["kc"], s["vc"], s["wc"], s["pc"], s["R"], lens=s["lens"])
            return s["kc"], s["vc"], s["wc"], s["pc"]
        if op == "cache_append":
            slots = swa.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["wc"], s["pc"], s["pos"], s["R"])
            return slots, s["kc"], s["vc"], s["wc"], s["pc"]
        if op == "cache_decode":
            return swa.cache_decode(s["q"], s["kc"], s["vc"], s["wc"], s["pos"], kprefix=s["kp"], vprefix=s["vp"]), s["wc"]
        return swa.prefix_decode(s["q"], s["kp"], s["vp"], s["kc"], s["vc"], s["pos"], s["W"])
    if op == "key_weights":
        return _plain_key_weights(s["q"], s["k"], s["lse"], s["W"], s["G"], s["lens"], s["last"])
    if op == "cache_seed":
        return _plain_seed(s["k"], s["v"], s["weights"], s["kc"], s["vc"], s["wc"], s["pc"], s["R"], s["lens"])
    if op == "cache_append":
        return _plain_append(s["k"], s["v"], s["kc"], s["vc"], s["wc"], s["pc"], s["pos"], s["R"])
    out, p = _plain_attend(s["q"], s["kc"], s["vc"], s["pos"], s["kp"], s["vp"])
    if op == "cache_decode":
        s["wc"] += p.sum(dim=2)
        return out, s["wc"]
    return out


# ------------------------------------------------------------------------------- exact values
def exact(case, seed):
    """The definitions in float64, one (stream, key head) at a time."""
    s, op = prepare(case, seed), case["op"]
    if op in ("cache_seed", "cache_append"):
        return None  # copies and choices: nothing is computed
    G, D = case["G"], case["D"]
    c = 1.0 / math.sqrt(D)
    if op == "key_weights":
        B, Hkv, T, W = case["B"], case["H"] // G, case["T"], case["W"]
        out = torch.zeros(B, Hkv, T, device=DEV, dtype=torch.float64)
        for b in range(B):
            n = T if s["lens"] is None else int(s["lens"][b])
            first = max(0, n - (s["last"] or n))
            for h in range(Hkv * G):
                kd = s["k"][b, h // G].double()
                for i0 in range(first, n, 2048):
                    i1, j0 = min(n, i0 + 2048), max(0, i0 - W + 1)
                    z = s["q"][b, h, i0:i1].double() @ kd[j0:i1].T * c - s["lse"][b, h, i0:i1].double()[:, None]
                    gap = torch.arange(i0, i1, device=DEV)[:, None] - torch.arange(j0, i1, device=DEV)[None]
                    out[b, h // G, j0:i1] += torch.where((gap >= 0) & (gap < W), z.exp(), 0.0).sum(0)
        return out
    B, Hkv = case["B"], case["H"] // G
    S = s["kc"].shape[2]
    out = torch.zeros(B, Hkv, G, D, device=DEV, dtype=torch.float64)
    w = s["wc"].double() if op == "cache_decode" else None
    kpd = None if s["kp"] is None else s["kp"].double()
    vpd = None if s["vp"] is None else s["vp"].double()
    for b in range(B):
        n = min(int(s["pos"][b]) + 1, S)
        ks, vs = s["kc"][b, :, :n].double(), s["vc"][b, :, :n].double()
        if kpd is not None:
            ks, vs = torch.cat([kpd, ks], dim=1), torch.cat([vpd, vs], dim=1)
        p = torch.softmax(torch.bmm(s["q"][b].double().view(Hkv, G, D) * c, ks.transpose(1, 2)), dim=2)
        out[b] = torch.bmm(p, vs)
        if w is not None:
            w[b, :, :n] += p[:, :, -n:].sum(1)
    out = out.reshape(B, Hkv * G, D)
    return (out, w) if op == "cache_decode" else out
