"""Plain float64 forms of the shared-prefix decode and of the budget cache, on torch tensors of
any device, and the error bounds that the tests of the kernels use. Loops and elementary
operations only."""
import math

import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
UBF = 2.0 ** -8    # half a step of bf16, relative


def key_weights(q, k, lse, W, lens=None, last=None, scale=None):
    """(weights, bound): bound[b,hk,j] is how far fp32 scores, exponentials and sums may be."""
    B, H, T, D = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    c = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(B, Hkv, T, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b in range(B):
        n = T if lens is None else int(lens[b])
        first = max(0, n - (T if last is None else last))
        if n <= 0:
            continue
        i = torch.arange(first, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        seen = (i >= j) & (i - j < W)
        for h in range(H):
            qd, kd = q[b, h, first:n].double(), k[b, h // G, :n].double()
            ld = lse[b, h, first:n].double()[:, None]
            p = torch.where(seen, torch.exp(c * (qd @ kd.T) - ld), 0.0)
            # a dot of D terms and one multiply-add in fp32, as an absolute error of the exponent
            ez = (D + 4) * U32 * (abs(c) * (qd.abs() @ kd.abs().T) + ld.abs())
            out[b, h // G, :n] += p.sum(0)
            # exp itself: a few units of fp32; the sum: at most T G additions
            bound[b, h // G, :n] += (p * (ez + 2.0 ** -20 + T * G * U32)).sum(0)
    return out, bound


def _order(w):
    """A weight as it is compared: NaN counts as +infinity."""
    w = float(w)
    return math.inf if w != w else w


def seed_choice(weights, n, S, recent):
    """Positions that a cache of S slots keeps of n tokens with these weights, ascending."""
    if n <= S:
        return list(range(n))
    old = n - recent
    heavy = sorted(range(old), key=lambda j: (-_order(weights[j]), j))[:S - recent]
    return sorted(heavy) + list(range(old, n))


def append_slot(w, p, pos, S, recent):
    """The slot that a token at position pos takes, or -1."""
    if pos < 0:
        return -1
    if pos < S:
        return pos
    for s in range(S):
        if int(p[s]) == pos:
            return s
    may = [s for s in range(S) if int(p[s]) <= pos - recent]
    return min(may, key=lambda s: (_order(w[s]), s)) if may else -1


def decode(q, kc, vc, pos, kp=None, vp=None, scale=None):
    """(out, out_spread, gain, gain_bound, ez): out and each slot's added weight in float64;
    out_spread = sum of p |v| of each output and ez the largest absolute error of an
    exponent, from which a test builds its tolerance."""
    B, H, D = q.shape
    Hkv, S = kc.shape[1], kc.shape[2]
    G = H // Hkv
    c = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(B, H, D, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    gain = torch.zeros(B, Hkv, S, dtype=torch.float64, device=q.device)
    ez = 0.0
    for b in range(B):
        n = min(int(pos[b]) + 1, S)
        if n <= 0:
            continue
        for h in range(H):
            hk = h // G
            ks, vs = kc[b, hk, :n].double(), vc[b, hk, :n].double()
            if kp is not None:
                ks, vs = torch.cat([kp[hk].double(), ks]), torch.cat([vp[hk].double(), vs])
            qd = q[b, h].double()
            p = torch.softmax(c * (ks @ qd), 0)
            ez = max(ez, (D + 4) * U32 * abs(c) * float((ks.abs() @ qd.abs()).max()))
            out[b, h] = p @ vs
            spread[b, h] = p @ vs.abs()
            gain[b, hk, :n] += p[-n:]
    return out, spread, gain, ez


def decode_tol(ref, spread, ez, keys, p_step):
    """Bound on |bf16 output - ref|: the rounding of the output, of the weights to p_step
    relative, errors of 2 ez of each weight (numerator and sum) and fp32 sums over the keys."""
    return UBF * ref.abs() + (p_step + 2 * ez + 2.0 ** -20 + 2 * keys * U32) * spread * (1 + UBF)
