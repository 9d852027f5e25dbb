"""The shared-prefix attention, the attention mass and the cache eviction from their definitions, in 64 bits.

Plain loops over sequences and heads on torch tensors (any device); contiguous layouts only: the paged tests gather
their pages first.
"""
import math

import torch


def visible_new(mode, k, R):
    """[R, R] bool: new key n visible to new row r (mode 0: the hybrid decode mask, 1: causal)."""
    m = torch.zeros((R, R), dtype=torch.bool)
    for r in range(R):
        if mode == 1 or r < k:
            m[r, :r + 1] = True
        else:
            j = (r - k) // k
            m[r, :j] = True
            m[r, k + j * k:k + (j + 1) * k] = True
    return m


def attn_shared(q, kn, vn, ks, vs, S, kc, vc, lens, mode, k, scale):
    """q [B,R,Hq,D]; ks, vs [Hkv,>=S,D]; kc, vc [B,Hkv,>=len,D].  Returns out, lse, and per output the weighted mean
    of |v| and the largest |v| among the row's keys (what rounding errors scale with), all in 64 bits."""
    B, R, Hq, D = q.shape
    Hkv = kn.shape[2]
    G = Hq // Hkv
    dev = q.device
    out = torch.zeros((B, R, Hq, D), dtype=torch.float64, device=dev)
    absum, vmax = torch.zeros_like(out), torch.zeros((B, R, Hq, 1), dtype=torch.float64, device=dev)
    lse = torch.zeros((B, R, Hq), dtype=torch.float64, device=dev)
    seen = visible_new(mode, k, R).to(dev)
    for b in range(B):
        n = S + int(lens[b])
        vis = torch.cat([torch.ones((R, n), dtype=torch.bool, device=dev), seen], 1)
        for h in range(Hkv):
            K = torch.cat([ks[h, :S], kc[b, h, :int(lens[b])], kn[b, :, h]]).double()
            V = torch.cat([vs[h, :S], vc[b, h, :int(lens[b])], vn[b, :, h]]).double()
            for g in range(G):
                x = (q[b, :, h * G + g].double() @ K.T) * scale
                x = x.masked_fill(~vis, -math.inf)
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - z[:, None])
                out[b, :, h * G + g] = p @ V
                absum[b, :, h * G + g] = p @ V.abs()
                lse[b, :, h * G + g] = z
                vmax[b, :, h * G + g] = V.abs().max()
    return out, lse, absum, vmax


def attn_tolerance(out, absum, vmax):
    """Each softmax weight is rounded to bf16 before it multiplies V (half a step: 2^-8 of sum p |v|), partial rows pass
    as fp16 over their own largest magnitude (2^-11 of at most max |v|), sums in fp32 (2^-12 of sum p |v| covers 4096
    terms' steps of 2^-24), and the result is rounded to bf16 (2^-8)."""
    return 2.0**-8 * (absum + out.abs()) + 2.0**-11 * vmax + 2.0**-12 * absum


def mass_update(mass, q, lse, kc, n, a, scale, decay):
    """One (layer, sequence): mass [Hkv,P], q [R,Hq,D], lse [R,Hq], kc [Hkv,>=n,D].  Returns the new mass in 64 bits."""
    Hkv = kc.shape[0]
    G = q.shape[1] // Hkv
    new = mass.double().clone()
    for h in range(Hkv):
        w = torch.zeros(n, dtype=torch.float64, device=q.device)
        K = kc[h, :n].double()
        for j in range(a):
            for g in range(G):
                x = (K @ q[j, h * G + g].double()) * scale - lse[j, h * G + g].double()
                x[n - a + j + 1:] = -math.inf
                w += torch.exp(x)
        new[h, :n - a] = decay * new[h, :n - a] + w[:n - a]
        new[h, n - a:n] = w[n - a:]
    return new


# A score is a sum of D <= 128 exact products in fp32: off by at most D 2^-24 times the sum of their magnitudes, which
# for the tests' inputs (q ~ 1.5 N(0,1), k ~ N(0,1), scale D^-1/2) stays below 1.5 * 128 * 128^-1/2 = 17: 1.3e-4 in the
# exponent, and as much relative to the weight; the exponential and the sum add less than 1e-5.
MASS_RTOL = 2e-4


def evict_moves(mass, n, budget, sink, recent):
    """One head's mass (sequence of n floats): (destinations, sources) of the rows that move, or two empty lists."""
    if n <= budget:
        return [], []
    zone = budget - recent
    heavy = [(0, 0.0) if math.isnan(x) else (1, -x) for x in mass[:n]]  # NaN first, then the greatest mass
    cand = sorted(range(sink, n - recent), key=lambda i: (heavy[i], i))
    kept = set(cand[:zone - sink])
    holes = [i for i in range(sink, min(zone, n - recent)) if i not in kept]
    tails = [i for i in range(zone, n - recent) if i in kept]
    assert len(holes) == len(tails)
    return holes + list(range(zone, budget)), tails + list(range(n - recent, n))
