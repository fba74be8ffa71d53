"""Measured cases of the general router, the experts' activation with dropout, and the 4-bit integer product.

  route  ids and weights of the k experts of each token: softmax or sigmoid scores, a bias that only the choice sees,
         a limit to the best groups of experts, weights renormalised or as they are, times a constant
  step   the same in training: also the tokens that each expert got, and the gradient of the logits from the weights'
  act    h = keep * silu(g) * u / (1 - p) of rows [g | u] and, from dh, the gradient of [g | u]; `keep` comes from a
         counter-based generator in both directions and is stored in neither
  mv     y[r] = W_e x[r] for the rows r of expert e, few of them: W in 4 bits, a scale and a zero per 128 elements

`own` selects the library's kernels; otherwise run() computes the same in elementary torch operations, in 32 bits, and
in 64 where a choice depends on the last bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token through a large layer's router: 4 of 8 groups, a balance bias, top-8 of 256; latency
        dict(name="route_token", op="route", M=1, E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
             group_top=2, renorm=True, scale=2.5, dt="fp32"),
        # a batch of 512 tokens over 128 experts, 16-bit logits (many equal ones), weights as the softmax gives them
        dict(name="route_batch", op="route", M=512, E=128, k=8, score="softmax", bias=False, groups=1, topk_groups=1,
             group_top=1, renorm=False, scale=1.0, dt="bf16"),
        # an odd number of tokens, groups of 20 experts ranked by their best one
        dict(name="route_odd", op="route", M=4099, E=160, k=6, score="softmax", bias=False, groups=8, topk_groups=3,
             group_top=1, renorm=False, scale=16.0, dt="fp16"),
        # a long prefill through the large layer's router
        dict(name="route_prefill", op="route", M=65536, E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
             group_top=2, renorm=True, scale=2.5, dt="bf16"),
        # a training step's routing of 4096 tokens over 128 experts
        dict(name="step_batch", op="step", M=4096, E=128, k=8, score="softmax", bias=False, groups=1, topk_groups=1,
             group_top=1, renorm=False, scale=1.0, dt="fp32"),
        # a training step's routing of 65536 tokens over 256 experts, balanced by the bias
        dict(name="step_large", op="step", M=65536, E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
             group_top=2, renorm=True, scale=2.5, dt="bf16"),
        # fine-tuning on few rows, a width that no vector divides
        dict(name="act_odd", op="act", R=777, I=1001, p=0.1, dt="fp16"),
        # the routes of 512 tokens, top-8
        dict(name="act_batch", op="act", R=4096, I=768, p=0.1, dt="bf16"),
        # a training step of the large layer on one expert-parallel rank: a stream over memory
        dict(name="act_large", op="act", R=38400, I=2048, p=0.3, dt="bf16"),
        # one token's 8 routes through the gate/up projection: latency, weight-bound
        dict(name="mv_token", op="mv", R=8, E=128, N=1536, K=2048, spread="distinct", dt="bf16", out="bf16", pad=0),
        # one token through a shared expert's gate/up projection in the large layer
        dict(name="mv_dense", op="mv", R=1, E=1, N=4096, K=7168, spread="even", dt="fp16", out="fp32", pad=0),
        # 64 decoded tokens, top-8, Zipf-routed: most experts' weights once, up to some tens of rows for the popular
        dict(name="mv_batch", op="mv", R=512, E=128, N=1536, K=2048, spread="zipf", dt="bf16", out="bf16", pad=23),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "step", "act", "mv"])
    if op in ("route", "step"):
        groups = rng.choice([1, 1, 2, 4, 8, 8, 16, 5])
        while True:
            E = groups * (_log(rng, 8, 512) // groups or 1)
            topk_groups = rng.randrange(1, groups + 1)
            k = rng.choice([1, 2, 4, 6, 8, 8, 12])
            if k <= topk_groups * (E // groups):
                break
        M = _log(rng, 1, 65536)
        dt = rng.choice(["bf16", "fp16", "fp32"])
        M = max(1, min(M, 65536 * 256 // E // (2 if dt == "fp32" else 1) * 15 // 16))
        bias = rng.random() < 0.5
        return dict(op=op, M=M, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=bias, groups=groups,
                    topk_groups=topk_groups, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5, 16.0]), dt=dt)
    if op == "act":
        dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        I = _log(rng, 16, 4096)
        if rng.random() < 0.7:
            I = max(8, I // 8 * 8)
        most = 38400 * 2048 // (2 if dt == "fp32" else 1)
        return dict(op=op, R=max(1, min(_log(rng, 1, 38400), most // I)), I=I, p=rng.choice([0.05, 0.1, 0.2, 0.5]), dt=dt)
    while True:
        E = rng.choice([1, 1, _log(rng, 2, 256)])
        N, K = max(8, _log(rng, 64, 8192) // 8 * 8), max(128, _log(rng, 128, 8192) // 128 * 128)
        if rng.random() < 0.5:
            N = max(64, N // 64 * 64)
        R = _log(rng, 1, 32 if E == 1 else min(512, 8 * E))
        spread = rng.choice(["even", "zipf"])
        sizes = _sizes(dict(E=E, R=R, spread=spread))
        if (sizes > 0).sum() * N * K <= 2.9e8 and E * N * K <= 8e8 and sizes.max() <= 96:
            break
    dt = rng.choice(["bf16", "fp16"])
    return dict(op=op, R=R, E=E, N=N, K=K, spread=spread, dt=dt, out=rng.choice([dt, "fp32"]),
                pad=rng.choice([0, 0, rng.randrange(1, 40)]))


def _sizes(c):
    """Rows of each expert, fixed by the case: `distinct` one row each on R experts, `even` and `zipf` R independent
    routes with equal and with (1 + rank)^-1.1 chances."""
    E, R = c["E"], c["R"]
    g = np.random.RandomState(1000 * R + E)
    if c["spread"] == "distinct":
        n = np.zeros(E, dtype=np.int64)
        n[g.permutation(E)[:R]] = 1
        return n
    p = np.ones(E) if c["spread"] == "even" else (1.0 + g.permutation(E)) ** -1.1
    return g.multinomial(R, p / p.sum())


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, std, dt=torch.float32):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(0.0, std, generator=g)

    s = dict(case=c)
    if c["op"] in ("route", "step"):
        # logits of tokens that agree on some experts more than on others, and the bias that makes up for a part of it
        liking = normal((c["E"],), 0.5)
        s["logits"] = (normal((c["M"], c["E"]), 1.0) + liking).to(DTYPES[c["dt"]])
        s["bias"] = -0.1 * liking + normal((c["E"],), 0.01) if c["bias"] else None
        s["dw"] = normal((c["M"], c["k"]), 1.0) if c["op"] == "step" else None
        return s
    if c["op"] == "act":
        dt = DTYPES[c["dt"]]
        s["gu"] = normal((c["R"], 2 * c["I"]), 1.0, dt)
        s["dh"] = normal((c["R"], c["I"]), 0.1, dt)
        s["rng"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=g, device="cuda", dtype=torch.int64)
        return s
    E, N, K, R = c["E"], c["N"], c["K"], c["R"] + c["pad"]
    s["x"] = normal((R, K), 1.0, DTYPES[c["dt"]])
    s["q"] = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=g, device="cuda", dtype=torch.int64).int()
    s["scale"] = torch.exp(normal((E, N, K // 128), 0.3)).mul_(0.004).half()
    zero = torch.zeros((E, N // 8, K // 128), dtype=torch.int32, device="cuda")
    for i in range(8):                          # zeros around the middle of the 16 codes
        zero |= torch.randint(5, 11, zero.shape, generator=g, device="cuda", dtype=torch.int32) << (4 * i)
    s["zero"] = zero
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(_sizes(c))]).astype(np.int32)).cuda()
    if own:                                     # the handle that a program keeps of its weights
        import top_moe_expert_gb300 as moe
        s["w"] = moe.Weights(moe.MOE_W_AWQ4, s["q"], s["scale"], s["zero"])
    return s


# ------------------------------------------------------------------ plain forms

def _scores(l, score):
    """Scores of all experts, of l's type: a softmax over the experts, or each logit's sigmoid."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(dim=1, keepdim=True))
    return p / p.sum(dim=1, keepdim=True)


def _choose(s):
    """Ids [M, k]: by score plus bias in 64 bits (by the logit where there is no bias), equal ones by id."""
    c, l = s["case"], s["logits"].double()
    M, E, G = c["M"], c["E"], c["groups"]
    score = _scores(l, c["score"])
    by = l if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        of = by if s["bias"] is not None or c["group_top"] == 1 else score
        top = torch.sort(of.view(M, G, E // G), dim=2, descending=True)[0][:, :, :c["group_top"]].sum(dim=2)
        best = torch.sort(top, dim=1, descending=True, stable=True)[1][:, :c["topk_groups"]]
        live = torch.zeros((M, G), dtype=torch.bool, device=l.device).scatter_(1, best, True)
        by = torch.where(live.repeat_interleave(E // G, dim=1), by, -math.inf)
    return torch.sort(by, dim=1, descending=True, stable=True)[1][:, :c["k"]]


def _weights(s, ids):
    """Weights [M, k] and the scores of all experts, in 32 bits."""
    c = s["case"]
    score = _scores(s["logits"].float(), c["score"])
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return w * c["scale"], score


def _weights_bwd(s, ids, w, score):
    """The logits' gradient from the weights'."""
    c, dw = s["case"], s["dw"]
    chosen = score.gather(1, ids)
    if c["renorm"]:
        d = w * (dw - (w * dw).sum(dim=1, keepdim=True) / c["scale"])
        if c["score"] == "sigmoid":
            d = d * (1.0 - chosen)
        return torch.zeros_like(score).scatter_(1, ids, d)
    if c["score"] == "sigmoid":
        return torch.zeros_like(score).scatter_(1, ids, c["scale"] * dw * chosen * (1.0 - chosen))
    dp = torch.zeros_like(score).scatter_(1, ids, c["scale"] * dw)
    return score * (dp - (score * dp).sum(dim=1, keepdim=True))


def _philox(c, key):
    """Philox4x32 with 10 rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011): counters c, four
    int64 tensors below 2^32, and a key of two such numbers."""
    k0, k1 = key
    mask = 0xFFFFFFFF
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57          # 64-bit products, their upper halves shifted down
        c = [(p1 >> 32 & mask) ^ c[1] ^ k0, p1 & mask, (p0 >> 32 & mask) ^ c[3] ^ k1, p0 & mask]
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return c


def _keep(c, rng):
    """The factor of each element [R, I]: 0 for a share of threshold / 65536, else 65536 / (65536 - threshold).  Element
    i of row r has the 16 bits i % 8 of the generator's value at counter (i / 8, r, offset)."""
    R, I = c["R"], c["I"]
    t = math.floor(c["p"] * 65536 + 0.5)
    lo, hi = rng & 0xFFFFFFFF, rng >> 32 & 0xFFFFFFFF           # seed, offset
    n = -(-I // 8)
    r = torch.arange(R, device=rng.device).view(R, 1).expand(R, n)
    j = torch.arange(n, device=rng.device).view(1, n).expand(R, n)
    words = torch.stack(_philox([j, r, lo[1].expand(R, n), hi[1].expand(R, n)], (lo[0], hi[0])), dim=2)
    bits = torch.stack([words & 0xFFFF, words >> 16], dim=3).reshape(R, 8 * n)[:, :I]
    return (bits >= t).float() * (65536.0 / (65536 - t))


def _values(q, scale, zero):
    """[E, N, K] fp32 of 4-bit codes, scales and zeros."""
    E, N, W = q.shape
    sh = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    v = ((q.unsqueeze(3) >> sh) & 15).float().view(E, N, W // 16, 128)
    z = ((zero.unsqueeze(2) >> sh.view(1, 1, 8, 1)) & 15).float().view(E, N, W // 16, 1)
    return ((v - z) * scale.float().unsqueeze(3)).view(E, N, 8 * W)


def _product(s):
    """Each row by its expert's weights; the weights of the experts that have rows are widened."""
    c, x, off = s["case"], s["x"].float(), s["offsets"].long()
    n, R = _sizes(c), x.shape[0]
    live = torch.from_numpy(np.flatnonzero(n)).to(x.device)
    w = _values(s["q"][live], s["scale"][live], s["zero"][live])
    rows = off[live][:, None] + torch.arange(int(n.max()), device=x.device)          # [live experts, most rows]
    p = torch.bmm(x[rows.clamp(max=R - 1)], w.transpose(1, 2))
    r = torch.arange(R, device=x.device)
    e = torch.searchsorted(off[1:], r, right=True)
    k = torch.searchsorted(live, e).clamp(max=live.numel() - 1)
    y = p[k, (r - off[live[k]]).clamp(0, p.shape[1] - 1)]
    return y * (r < off[-1])[:, None]


def run(state):
    c, s = state["case"], state
    if own:
        import top_moe_expert_gb300 as moe
    if c["op"] in ("route", "step"):
        if own:
            how = dict(score=moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                       renorm=c["renorm"], scale=c["scale"])
            load = torch.zeros(c["E"], dtype=torch.int32, device="cuda") if c["op"] == "step" else None
            ids, w = moe.moe_route(s["logits"], c["k"], bias=s["bias"], groups=c["groups"], topk_groups=c["topk_groups"],
                                   group_top=c["group_top"], load=load, **how)
            if c["op"] == "route":
                return {"ids": ids, "w": w}
            return {"ids": ids, "w": w, "load": load, "dlogits": moe.moe_route_bwd(s["dw"], s["logits"], ids, **how)}
        ids = _choose(s)
        w, score = _weights(s, ids)
        if c["op"] == "route":
            return {"ids": ids.int(), "w": w}
        ones = torch.ones(ids.numel(), dtype=torch.int32, device=ids.device)
        load = torch.zeros(c["E"], dtype=torch.int32, device=ids.device).index_add_(0, ids.reshape(-1), ones)
        return {"ids": ids.int(), "w": w, "load": load, "dlogits": _weights_bwd(s, ids, w, score).to(s["logits"].dtype)}
    if c["op"] == "act":
        if own:
            return {"h": moe.moe_swiglu_dropout(s["gu"], c["p"], s["rng"]),
                    "dgu": moe.moe_swiglu_dropout_bwd(s["dh"], s["gu"], c["p"], s["rng"])}
        dt = s["gu"].dtype
        g, u = s["gu"].float().chunk(2, dim=1)
        a = 1.0 / (1.0 + torch.exp(-g))
        h = _keep(c, s["rng"]) * (g * a * u)
        d = _keep(c, s["rng"]) * s["dh"].float()          # each direction makes its own: neither stores it for the other
        return {"h": h.to(dt), "dgu": torch.cat([d * u * a * (1.0 + g * (1.0 - a)), d * g * a], dim=1).to(dt)}
    out = DTYPES[c["out"]]
    if own:
        return moe.moe_grouped_mm_awq(s["x"], s["w"], s["offsets"], out_dtype=out)
    return _product(s).to(out)


# ------------------------------------------------------------------ work

def _bytes(name):
    return torch.empty((), dtype=DTYPES[name]).element_size()


def work(case):
    c = case
    if c["op"] in ("route", "step"):
        M, E, k = c["M"], c["E"], c["k"]
        b = M * E * _bytes(c["dt"]) + 8.0 * M * k + (4 * E if c["bias"] else 0)
        f = 10.0 * M * E
        if c["op"] == "step":
            b += M * E * _bytes(c["dt"]) + 4.0 * M * k + 4 * E
            f += 10.0 * M * k
        return {"bytes": float(b), "flops": f}
    if c["op"] == "act":
        n = c["R"] * c["I"]                                # [g | u] and dh read, h and the gradient written
        return {"bytes": float(n * 6 * _bytes(c["dt"])), "flops": 30.0 * n}
    n = _sizes(c)
    R, N, K, live = c["R"] + c["pad"], c["N"], c["K"], int((n > 0).sum())
    return {"bytes": live * N * K * (0.5 + 2 / 128 + 0.5 / 128) + 2.0 * c["R"] * K + R * N * _bytes(c["out"])
            + 4.0 * (c["E"] + 1), "flops": 2.0 * c["R"] * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_route(c, s):
    l, b = s["logits"].double(), s["bias"]
    M, E = l.shape
    if c["score"] == "sigmoid":
        score = torch.where(l >= 0, 1 / (1 + torch.exp(-l.abs())), torch.exp(-l.abs()) / (1 + torch.exp(-l.abs())))
    else:
        score = torch.exp(l - torch.logsumexp(l, dim=1, keepdim=True))
    want = score + b.double() if b is not None else l
    live = torch.ones_like(want, dtype=torch.bool)
    rows = torch.arange(M, device=l.device)
    if c["groups"] > 1:
        n = E // c["groups"]
        value = []
        for g in range(c["groups"]):
            part = (score if b is None and c["group_top"] == 2 else want)[:, g * n:(g + 1) * n]
            first = part.max(dim=1)
            v = first[0]
            if c["group_top"] == 2 and n > 1:
                v = v + part.scatter(1, first[1][:, None], -math.inf).amax(dim=1)
            value.append(v)
        value = torch.stack(value, dim=1)
        live = torch.zeros_like(value, dtype=torch.bool)
        for _ in range(c["topk_groups"]):
            m = torch.where(live, -math.inf, value)
            at = (m == m.amax(dim=1, keepdim=True)).int().argmax(dim=1)          # the first of equal ones
            live[rows, at] = True
        live = live.repeat_interleave(n, dim=1)
    want = torch.where(live, want, -math.inf)
    ids = []
    for _ in range(c["k"]):
        at = (want == want.amax(dim=1, keepdim=True)).int().argmax(dim=1)
        ids.append(at)
        want[rows, at] = -math.inf
    ids = torch.stack(ids, dim=1)
    w = score[rows[:, None], ids]
    total = w.sum(dim=1, keepdim=True) if c["renorm"] else torch.ones((M, 1), dtype=torch.float64, device=l.device)
    w = w * (c["scale"] / total)
    out = {"ids": ids.int(), "w": w}
    if c["op"] == "step":
        # dw/dl of slot j and expert e by the chain rule: through the scores, and through their sum where it divides
        dw, chosen = s["dw"].double(), score[rows[:, None], ids]
        ds = c["scale"] * dw / total
        if c["renorm"]:
            ds = ds - (w * dw).sum(dim=1, keepdim=True) / total
        dl = torch.zeros_like(score)
        if c["score"] == "sigmoid":
            dl[rows[:, None], ids] = ds * chosen * (1 - chosen)
        else:
            dl[rows[:, None], ids] = ds * chosen
            dl -= score * (ds * chosen).sum(dim=1, keepdim=True)
        out["load"] = torch.bincount(ids.reshape(-1), minlength=E).int()
        out["dlogits"] = dl
    return out


def _exact_keep(c, rng):
    """The generator's bits by 16-bit partial products."""
    def mul(a, m):
        """Upper and lower 32 bits of a times the constant m."""
        low = a * (m & 0xFFFF)                                # below 2^48
        high = a * (m >> 16)
        total = (low >> 16) + high                            # the product divided by 2^16
        return total >> 16, ((total & 0xFFFF) << 16) | (low & 0xFFFF)

    seed, offset = (int(v) % 2 ** 64 for v in rng.tolist())
    n = (c["I"] + 7) // 8
    dev = rng.device
    x = [torch.arange(n, device=dev).repeat(c["R"]), torch.arange(c["R"], device=dev).repeat_interleave(n),
         torch.full((c["R"] * n,), offset % 2 ** 32, device=dev), torch.full((c["R"] * n,), offset // 2 ** 32, device=dev)]
    for i in range(10):
        h0, l0 = mul(x[0], 0xD2511F53)
        h1, l1 = mul(x[2], 0xCD9E8D57)
        a, b = (seed + i * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
        x = [h1 ^ x[1] ^ a, l1, h0 ^ x[3] ^ b, l0]
    halves = []
    for v in x:
        halves += [v % 65536, v // 65536]
    bits = torch.stack(halves, dim=1).view(c["R"], n * 8)[:, :c["I"]]
    t = int(c["p"] * 65536 + 0.5)
    return torch.where(bits < t, 0.0, 65536.0 / (65536.0 - t)).double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("route", "step"):
        return _exact_route(c, s)
    if c["op"] == "act":
        f = _exact_keep(c, s["rng"])
        g, u, dh = s["gu"][:, :c["I"]].double(), s["gu"][:, c["I"]:].double(), s["dh"].double()
        sig = torch.sigmoid(g)
        du = f * dh * g * sig
        dg = f * dh * u * (sig + g * sig * torch.sigmoid(-g))
        return {"h": f * g * sig * u, "dgu": torch.cat([dg, du], dim=1)}
    off = s["offsets"].tolist()
    y = torch.zeros((c["R"] + c["pad"], c["N"]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        codes = torch.stack([(s["q"][e].long() >> (4 * i)) & 15 for i in range(8)], dim=2).reshape(c["N"], c["K"])
        zero = torch.stack([(s["zero"][e].long() >> (4 * i)) & 15 for i in range(8)], dim=1).reshape(c["N"], c["K"] // 128)
        w = (codes - zero.repeat_interleave(128, dim=1)).double() * s["scale"][e].double().repeat_interleave(128, dim=1)
        y[lo:hi] = s["x"][lo:hi].double() @ w.T
    return y
