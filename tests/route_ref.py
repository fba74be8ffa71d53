"""Plain 64-bit forms of the general router, the activation with dropout and the AWQ product, for the tests (torch and
numpy on the CPU)."""
from __future__ import annotations

import numpy as np
import torch

INF = float("inf")
SOFTMAX, SIGMOID = 0, 1


# ---------------------------------------------------------------- router

def scores(l, score):
    """Scores of the experts, l float64 [M, E]; an expert at -inf has none (0)."""
    if score == SIGMOID:
        t = torch.exp(-l.abs())
        return torch.where(l >= 0, 1 / (1 + t), t / (1 + t))
    m = l.amax(dim=1, keepdim=True)
    p = torch.exp(l - torch.where(m > -INF, m, torch.zeros_like(m)))
    return p / p.sum(dim=1, keepdim=True).clamp(min=5e-324)


def route(logits, k, score=SOFTMAX, bias=None, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    """(ids int64 [M, k], weights float64 [M, k], the smallest gap that decided something for each token)."""
    l = logits.double()
    M, E = l.shape
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double()
    bad = ~(l < INF) | ~(b < INF)
    l = torch.where(bad, -INF, l)
    s = scores(l, score)
    off = (l == -INF) | (b == -INF)
    by = torch.where(off, -INF, l if bias is None else s + b)
    value = torch.where(off, -INF, s) if bias is None and group_top == 2 else by
    ids = torch.full((M, k), -1, dtype=torch.int64)
    gap = torch.full((M,), INF, dtype=torch.float64)
    n = E // groups
    for t in range(M):
        live = np.ones(E, dtype=bool)
        if groups > 1:
            best = []
            for g in range(groups):
                v = np.sort(value[t, g * n:(g + 1) * n].numpy())[::-1]
                v = [x for x in v[:group_top] if x > -INF]
                best.append(float(sum(v)) if v else -INF)
            order = sorted(range(groups), key=lambda g: (-best[g], g))
            live = np.isin(np.arange(E) // n, order[:topk_groups])
            if topk_groups < groups and best[order[topk_groups]] > -INF:
                d = best[order[topk_groups - 1]] - best[order[topk_groups]]
                if d:
                    gap[t] = min(gap[t], d)
        v = by[t].numpy()
        order = [e for e in np.argsort(-v, kind="stable") if live[e] and v[e] > -INF]
        for j, e in enumerate(order[:k]):
            ids[t, j] = int(e)
            if bias is not None and j + 1 < len(order) and v[e] != v[order[j + 1]]:
                gap[t] = min(gap[t], v[e] - v[order[j + 1]])
    ok = ids >= 0
    w = weights(l, ids, score, renorm, scale)
    w = torch.where(bad.any(dim=1, keepdim=True), float("nan"), w)
    return ids, torch.where(ok | bad.any(dim=1, keepdim=True), w, 0.0), gap


def weights(l, ids, score, renorm, scale):
    """The weights of given ids (differentiable in l float64)."""
    ok = ids >= 0
    at = ids.clamp(min=0)
    if renorm:
        ls = torch.nn.functional.logsigmoid(l) if score == SIGMOID else l
        c = torch.where(ok, ls.gather(1, at), -INF)
        m = c.detach().amax(dim=1, keepdim=True)
        p = torch.where(ok, torch.exp(c - torch.where(m > -INF, m, torch.zeros_like(m))), 0.0)
        return scale * p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return torch.where(ok, scale * scores(l, score).gather(1, at), 0.0)


def route_bwd(dw, logits, ids, score, renorm, scale):
    """(dlogits, sum of its terms' magnitudes), float64; every slot of an expert adds to it."""
    l, dw = logits.double(), dw.double()
    ok = ids >= 0
    at, dw = ids.clamp(min=0), torch.where(ok, dw, 0.0)
    w, s = weights(l, ids, score, renorm, scale), scores(l, score)
    g, mag = w * dw, w * dw.abs()
    if renorm:
        mag = mag + w * mag.sum(dim=1, keepdim=True) / scale
        g = g - w * g.sum(dim=1, keepdim=True) / scale
    if score == SIGMOID:
        c = scores(-l, score).gather(1, at)
        g, mag = g * c, mag * c
    dl = torch.zeros_like(l).scatter_add_(1, at, torch.where(ok, g, 0.0))
    dm = torch.zeros_like(l).scatter_add_(1, at, torch.where(ok, mag, 0.0))
    if score == SOFTMAX and not renorm:
        dl, dm = dl - s * (w * dw).sum(dim=1, keepdim=True), dm + s * (w * dw.abs()).sum(dim=1, keepdim=True)
    return dl, dm


# ---------------------------------------------------------------- dropout

def philox(counter, key):
    """Philox4x32 with 10 rounds; counter [..., 4] and key (two numbers), all below 2^32."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k = [np.uint64(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ k[0], p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ k[1], p0 & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(c, axis=-1)


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def kept(R, I, p, seed, offset, row0=0):
    """Which elements [R, I] are kept; the first row has the number row0."""
    n = -(-I // 8)
    c = np.zeros((R, n, 4), dtype=np.uint64)
    c[..., 0] = np.arange(n)
    c[..., 1] = (row0 + np.arange(R))[:, None]
    c[..., 2], c[..., 3] = offset % 2 ** 32, offset % 2 ** 64 >> 32
    v = philox(c, (seed % 2 ** 32, seed % 2 ** 64 >> 32))
    bits = np.stack([v & np.uint64(0xFFFF), v >> np.uint64(16)], axis=-1).reshape(R, 8 * n)[:, :I]
    return torch.from_numpy(bits.astype(np.int64) >= threshold(p))


def swiglu(gu, p, keep):
    """(h, dg's and du's functions) in float64: h, and from dh the gradient [dg | du] and its terms' magnitudes."""
    g, u = gu.double().chunk(2, dim=1)
    f = 65536.0 / (65536 - threshold(p))
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    zero = torch.zeros((), dtype=torch.float64)
    h = torch.where(keep, f * g * s * u, zero)

    def bwd(dh):
        d = f * dh.double()
        dg, du = torch.where(keep, d * u * s * (1 + g * c), zero), torch.where(keep, d * g * s, zero)
        mag = torch.where(keep, (d * u * s).abs() * (1 + (g * c).abs()), zero)
        return torch.cat([dg, du], dim=1), torch.cat([mag, du.abs()], dim=1)

    return h, bwd


# ---------------------------------------------------------------- AWQ

def awq_values(q, scale, zero):
    """float64 [E, N, K]."""
    E, N, W = q.shape
    sh = torch.arange(8) * 4
    v = ((q.long().unsqueeze(3) >> sh) & 15).view(E, N, 8 * W)
    z = ((zero.long().unsqueeze(2) >> sh.view(1, 1, 8, 1)) & 15).reshape(E, N, W // 16)
    r = lambda t: t.repeat_interleave(128, dim=2)  # noqa: E731
    return (v - r(z)).double() * r(scale.double())


def awq_random(E, N, K, g, scales=None):
    """(q, scale, zero) of random codes; scales drawn from the given values, or around 0.004."""
    q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=g).int()
    zero = torch.randint(-2 ** 31, 2 ** 31, (E, N // 8, K // 128), generator=g).int()
    if scales is None:
        scale = torch.exp(0.3 * torch.randn((E, N, K // 128), generator=g)).mul_(0.004).half()
    else:
        scale = torch.tensor(scales)[torch.randint(0, len(scales), (E, N, K // 128), generator=g)].half()
    return q, scale, zero
