"""Cases that measure a block around the expert layer: the norm before it, softmax routing, 8-bit integer experts.

Five operators, each reached through the C-ABI binding (biased_top_routing_amd._lib):

  norm        h = x + residual, rounded to the activation type; y = h r w with r = (mean(h^2) + eps)^-1/2, and y in 8
              bits: int8 with one scale a token, s = r max|h w| / 127, code = round(127 h w / max|h w|), or E4M3 with
              one a 1 x 128 tile, s = r max|h w| / 448.  Rows behind the live tokens stay as they were.
  norm_grad   its gradients: with g = dy w and m = mean(g h), dx = r (g - h r^2 m) + dh, dw = sum over the tokens of
              dy h r.  Rows of dx behind the live tokens are zero.
  route       softmax affinities s = softmax(x Wr^T + o), rounded once to fp32; q = s + b; the M groups with the
              largest sum of their top-r q, the k largest q in them; gates scale s / sum s, or scale s.
  route_grad  the gradients of the gates and of the sequence balance loss through the softmax and the router.
  experts     the SwiGLU experts on int8 weights (one scale an output channel) and activations (one a token):
              h = bf16(silu(q(x) Wg^T) * (q(x) Wu^T)), y = q(h) Wd^T, q(v) = round(127 v / max|v|) max|v| / 127
              over a row.  The shared experts are one FFN of S I columns: their Wd has one scale a channel.

`own` chooses the library's kernels or the plain torch form.
"""
import math

import torch

own = False

DEV = "cuda"
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token's hidden row before the layer: residual added, normed, in int8 for the experts (latency)
        dict(name="norm_token", op="norm", T=1, live=1, H=7168, act="bf16", residual=True, y=True, codes="int8"),
        # the FP8 layer's prefill batch, padded, normed for the router (bf16) and the experts (E4M3)
        dict(name="norm_prefill", op="norm", T=32768, live=32011, H=7168, act="bf16", residual=True, y=True,
             codes="fp8_e4m3"),
        # the training step of the V3-like layer: gradients of the norm, the residual branch's one coming in
        dict(name="norm_grad_prefill", op="norm_grad", T=16384, live=16384, H=7168, act="bf16", dh=True),
        # the small fp32 layer's training step, padded
        dict(name="norm_grad_small", op="norm_grad", T=256, live=201, H=128, act="f32", dh=False),
        # a decode step through a softmax router, gates renormalised
        dict(name="route_decode", op="route", T=128, H=7168, E=256, G=8, M=4, k=8, topr=2, act="bf16", offset=False,
             raw=False, keep=False),
        # the prefill batch of a training step: affinities kept for the backward pass, some experts masked
        dict(name="route_prefill", op="route", T=16384, H=7168, E=256, G=8, M=4, k=8, topr=2, act="bf16", offset=True,
             raw=True, keep=True),
        # the router's gradients of that step
        dict(name="route_grad_prefill", op="route_grad", T=16384, H=7168, E=256, k=8, seq=4096, alpha=1e-3, raw=True),
        # the same of a mid-size layer, gates renormalised, no balance loss
        dict(name="route_grad_mid", op="route_grad", T=4096, H=2048, E=64, k=6, seq=0, alpha=0.0, raw=False),
        # prefill of a V3-like layer on the norm's codes
        dict(name="experts_prefill", op="experts", T=16384, H=7168, E=256, k=8, S=1, I=2048, skew=0.0, rows="codes"),
        # a mid-size layer on a skewed batch, rows already sorted and quantised; I is an odd multiple of 128
        dict(name="experts_mid", op="experts", T=4096, H=2048, E=64, k=6, S=2, I=1408, skew=1.1, rows="sorted"),
        # decode of a V3-like layer from bf16 rows: a few rows an expert, the weights streamed once
        dict(name="experts_decode", op="experts", T=128, H=7168, E=256, k=8, S=1, I=2048, skew=0.0, rows="gather"),
        # a single token through the same layer
        dict(name="experts_token", op="experts", T=1, H=7168, E=256, k=8, S=1, I=2048, skew=0.0, rows="codes"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "route", "route_grad", "experts", "experts"])
    if op in ("norm", "norm_grad"):
        act = rng.choice(["bf16", "bf16", "f32"])
        H = 128 * _log(rng, 1, 64) if act == "bf16" else 4 * _log(rng, 1, 1024)
        T = _log(rng, 1, 32768 if op == "norm" and act == "bf16" else 16384)
        live = rng.choice([T, rng.randint(0, T)])
        if op == "norm_grad":
            return dict(op=op, T=T, live=live, H=min(H, 7168), act=act, dh=rng.choice([True, False]))
        codes = rng.choice(["int8", "fp8_e4m3", None]) if act == "bf16" else None
        y = True if codes is None else rng.choice([True, False])
        return dict(op=op, T=T, live=live, H=min(H, 7168), act=act, residual=rng.choice([True, False]), y=y, codes=codes)
    if op in ("route", "route_grad"):
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * rng.randint(max(1, 4 // G), 256 // G)
        M = rng.randint(1, G)
        k = rng.randint(1, min(8, M * E // G))
        T = _log(rng, 1, 16384)
        if op == "route_grad":
            H = 64 * _log(rng, 1, 112)
            seq = rng.choice([0] + [d for d in (2, 4, 64, 100) if T % d == 0])
            return dict(op=op, T=T, H=H, E=E, k=k, seq=seq, alpha=rng.choice([0.0, 1e-3, 1e-2]), raw=rng.choice([True, False]))
        act = rng.choice(["bf16", "bf16", "bf16", "f32"])
        H = 64 * _log(rng, 1, 112 if act == "bf16" else 8)
        return dict(op=op, T=T, H=H, E=E, G=G, M=M, k=k, topr=rng.randint(1, min(4, E // G)), act=act,
                    offset=rng.choice([True, False]), raw=rng.choice([True, False]), keep=rng.choice([True, False]))
    while True:
        H, I = 128 * _log(rng, 1, 64), 128 * _log(rng, 1, 24)
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(8, E))
        S = rng.choice([0, 1, 1, 2, 3])
        T = _log(rng, 1, 16384)
        c = dict(op=op, T=T, H=H, E=E, k=k, S=S, I=I, skew=rng.choice([0.0, 0.5, 1.1]),
                 rows=rng.choice(["gather", "sorted", "codes"]))
        if E * H * I <= 256 * 7168 * 2048 and T * (k + S) * H * max(I, S * I) <= 16384 * 9 * 7168 * 2048:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + salt)
    return g


def _q8(v):
    """fp32 rows of bf16 values (or of products of two): int8 codes as fp32, and the largest magnitude.  127 v is exact
    and the quotient is rounded once, so a code is the nearest whole number."""
    a = v.abs().amax(-1, keepdim=True).clamp_(min=2.0 ** -100)
    return (v * 127 / a).round(), a


def _weights(n, rows, cols, sigma, g, joint=False):
    """n random matrices in int8, made some at a time: codes [n, rows, cols] and scales [n, rows], or [rows] over
    all of them together."""
    codes = torch.empty((n, rows, cols), dtype=torch.int8, device=DEV)
    if joint:
        v = (torch.randn((n, rows, cols), generator=g, device=DEV) * sigma).to(BF).float()
        q, a = _q8(v.permute(1, 0, 2).reshape(rows, n * cols))
        codes.copy_(q.reshape(rows, n, cols).permute(1, 0, 2))
        return codes, (a / 127).reshape(rows)
    scale = torch.empty((n, rows), dtype=F32, device=DEV)
    step = max(1, (1 << 26) // (rows * cols))
    for i in range(0, n, step):
        m = min(step, n - i)
        q, a = _q8((torch.randn((m, rows, cols), generator=g, device=DEV) * sigma).to(BF).float())
        codes[i:i + m] = q
        scale[i:i + m] = (a / 127).squeeze(-1)
    return codes, scale


def _choose(T, E, k, skew, g):
    """k distinct experts a token, popularity ~ rank^-skew (ranks shuffled)."""
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1
    u = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    return (-skew * rank.log() - (-u.log()).log()).topk(k, dim=1).indices.to(I32).contiguous()


def _sorted(idx, E):
    """offsets and perm of the pairs, stably sorted by expert."""
    key = idx.reshape(-1).long()
    perm = torch.sort(key, stable=True).indices
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets.to(I32), perm.to(I32)


def _outlying(shape, g):
    """Rows of a residual stream: normal, a few channels far larger."""
    v = torch.randn(shape, generator=g, device=DEV)
    v *= 1 + 20 * (torch.rand(shape[-1], generator=g, device=DEV) > 0.995)
    return v


def _grid(shape, sigma, unit, most, g):
    """Normal values rounded to multiples of `unit` up to `most` of them."""
    return (torch.randn(shape, generator=g, device=DEV) * (sigma / unit)).round_().clamp_(-most, most) * unit


def prepare(case, seed):
    op, T, H = case["op"], case["T"], case["H"]
    s = dict(case=case)
    if op in ("norm", "norm_grad"):
        g = _gen(seed, 1)
        dt = F32 if case["act"] == "f32" else BF
        s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(dt)
        s["eps"] = 1e-6
        s["n"] = torch.tensor([case["live"]], dtype=I32, device=DEV) if case["live"] < T else None
        s["x"] = _outlying((T, H), g).to(dt)
        if op == "norm":
            s["residual"] = _outlying((T, H), g).to(dt) if case["residual"] else None
        else:
            s["dy"] = torch.randn((T, H), generator=g, device=DEV).to(dt)
            s["dh"] = torch.randn((T, H), generator=g, device=DEV).to(dt) if case["dh"] else None
        if own:
            from biased_top_routing_amd import _lib as L
            s["L"] = L
            wgt = case["act"] if op == "norm_grad" or case["codes"] is None else case["codes"]
            s["cfg"] = L.make_cfg(T, H, 1, 1, 1, 1, 0, 128, 1, 1.0, case["act"], wgt)
            zero = lambda *sh, d=dt: torch.zeros(sh, dtype=d, device=DEV)
            if op == "norm":
                s["h"] = zero(T, H) if case["residual"] else None
                s["y"] = zero(T, H) if case["y"] else None
                s["codes"] = None if case["codes"] is None else \
                    zero(T, H, d=torch.int8 if case["codes"] == "int8" else torch.float8_e4m3fn)
                s["scale"] = None if case["codes"] is None else zero(T, *([H // 128] if case["codes"] != "int8" else []), d=F32)
            else:
                s["dx"], s["dw"] = zero(T, H), zero(H, d=F32)
                s["ws"] = torch.empty(L.moe_workspace_bytes(s["cfg"], L.MOE_WS_NORM_BWD), dtype=torch.uint8, device=DEV)
        return s
    E, k = case["E"], case["k"]
    if op == "route":
        g = _gen(seed, 2)
        dt = F32 if case["act"] == "f32" else BF
        # activations and router weights on grids coarse enough for the logits to be exact in fp32 whatever the order
        # of the sums (32 x 61 x 8192 < 2^24 units): the chosen experts can then be compared number by number
        s["x"] = _grid((T, H), 1.0, 2.0 ** -3, 32, g).to(dt)
        s["wr"] = _grid((E, H), 1.0 / math.sqrt(H), 2.0 ** -11, 61, g).to(dt)
        s["bias"] = (torch.rand(E, generator=g, device=DEV) * 2 - 1) * (0.1 / E)
        s["offset"] = None
        if case["offset"]:
            o = torch.randn(E, generator=g, device=DEV)
            o[torch.rand(E, generator=g, device=DEV) < 0.02] = -math.inf      # experts taken out of service
            s["offset"] = o
        if own:
            from biased_top_routing_amd import _lib as L
            s["L"] = L
            s["cfg"] = L.make_cfg(T, H, E, case["G"], case["M"], k, 0, 128, case["topr"], 2.5, case["act"], case["act"])
            s["flags"] = L.MOE_SOFTMAX | (L.MOE_GATES_RAW if case["raw"] else 0)
            s["scores"] = torch.empty((T, E), dtype=F32, device=DEV) if case["keep"] else None
            s["ws"] = torch.empty(L.moe_workspace_bytes(s["cfg"], L.MOE_WS_ROUTE), dtype=torch.uint8, device=DEV)
            s["idx"] = torch.empty((T, k), dtype=I32, device=DEV)
            s["gates"] = torch.empty((T, k), dtype=F32, device=DEV)
        return s
    if op == "route_grad":
        g = _gen(seed, 3)
        s["x"] = torch.randn((T, H), generator=g, device=DEV).to(BF)
        s["wr"] = (torch.randn((E, H), generator=g, device=DEV) / math.sqrt(H)).to(BF)
        s["scores"] = torch.softmax(s["x"].float() @ s["wr"].float().T, 1)
        s["idx"] = s["scores"].topk(k, dim=1).indices.to(I32).contiguous()
        s["dgate"] = torch.randn((T, k), generator=g, device=DEV)
        if own:
            from biased_top_routing_amd import _lib as L
            s["L"] = L
            s["cfg"] = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 2.5, "bf16", "bf16")
            s["flags"] = L.MOE_SOFTMAX | (L.MOE_GATES_RAW if case["raw"] else 0)
            s["dx"] = torch.empty((T, H), dtype=F32, device=DEV)
            s["dw"] = torch.empty((E, H), dtype=F32, device=DEV)
            s["loss"] = torch.empty(1, dtype=F32, device=DEV)
            s["ws"] = torch.empty(L.moe_workspace_bytes(s["cfg"], L.MOE_WS_ROUTE_BWD_SOFTMAX), dtype=torch.uint8, device=DEV)
        return s
    g = _gen(seed, 4)
    S, I, P = case["S"], case["I"], T * k
    s["x"] = _outlying((T, H), g).to(BF)
    s["offsets"], s["perm"] = _sorted(_choose(T, E, k, case["skew"], g), E)
    s["bounds"] = s["offsets"].tolist()
    sg, sd = 1.0 / math.sqrt(H), 1.0 / math.sqrt(I)
    s["wgu"], s["wgu_s"] = _weights(E, 2 * I, H, sg, g)
    s["wd"], s["wd_s"] = _weights(E, H, I, sd, g)
    s["sgu"], s["sgu_s"] = _weights(S, 2 * I, H, sg, g)
    s["sd"], s["sd_s"] = _weights(S, H, I, sd, g, joint=True) if S else (None, None)
    if case["rows"] != "gather":
        q, a = _q8(s["x"].float())
        s["xq"], s["xs"] = q.to(torch.int8), (a / 127).reshape(T)
        if case["rows"] == "sorted":
            tok = (s["perm"] // k).long()
            s["x_perm"], s["x_perm_s"] = s["xq"][tok].contiguous(), s["xs"][tok].contiguous()
    if own:
        from biased_top_routing_amd import _lib as L
        s["L"] = L
        s["cfg"] = L.make_cfg(T, H, E, 1, 1, k, S, I, 1, 1.0, "bf16", "int8")
        sh = (s["sgu"], s["sd"]) if S else (None, None)
        shs = (s["sgu_s"], s["sd_s"]) if S else (None, None)
        s["w"] = L.expert_weights(s["wgu"], s["wd"], *sh, s["wgu_s"], s["wd_s"], *shs)
        s["ws"] = torch.empty(L.moe_workspace_bytes(s["cfg"], L.MOE_WS_FFN), dtype=torch.uint8, device=DEV)
        s["y_perm"] = torch.empty((P, H), dtype=BF, device=DEV)
        s["y_shared"] = torch.empty((T, H), dtype=BF, device=DEV) if S else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"norm": _norm, "norm_grad": _norm_grad, "route": _route, "route_grad": _route_grad,
            "experts": _experts}[s["case"]["op"]](s, s["case"])


def _norm(s, case):
    names = [n for n in ("h", "y", "codes", "scale") if n in s]
    if own:
        s["L"].moe_norm(s["cfg"], s["n"], s["x"], s["residual"], s["w"], s["eps"], s["h"], s["y"], s["codes"], s["scale"])
        return {n: s[n] for n in names if s[n] is not None}
    T, H, live = case["T"], case["H"], case["live"]
    dt = s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
    v = h.float()
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + s["eps"])
    p = v * s["w"].float()
    out = {}
    if case["residual"]:
        out["h"] = h
    if case["y"]:
        out["y"] = (p * r).to(dt)
    if case["codes"] == "int8":
        q, a = _q8(p)
        out["codes"], out["scale"] = q.to(torch.int8), (a / 127 * r).reshape(T)
    elif case["codes"]:
        t = p.reshape(T, H // 128, 128)
        a = t.abs().amax(-1, keepdim=True) / 448
        out["codes"] = (t / a).reshape(T, H).to(torch.float8_e4m3fn)
        out["scale"] = a.squeeze(-1) * r
    if live < T:                                       # rows behind the live ones stay as they were: zero
        for o in out.values():
            o.view(torch.uint8)[live:] = 0
    return out


def _norm_grad(s, case):
    if own:
        s["L"].moe_norm_backward(s["cfg"], s["n"], s["x"], s["w"], s["eps"], s["dy"], s["dh"], s["dx"], s["dw"], s["ws"])
        return s["dx"], s["dw"]
    live = case["live"]
    h, dy = s["x"][:live].float(), s["dy"][:live].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"])
    g = dy * s["w"].float()
    d = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        d = d + s["dh"][:live].float()
    dx = torch.zeros_like(s["x"])
    dx[:live] = d.to(dx.dtype)
    return dx, (dy * (h * r)).sum(0)


def _pick(scores, bias, case):
    """The k experts of each token in order, from fp32 affinities."""
    T, E, G, M = case["T"], case["E"], case["G"], case["M"]
    q = scores + bias
    top = q.reshape(T, G, E // G).topk(case["topr"], dim=2).values
    gs = top[..., 0].clone()
    for i in range(1, case["topr"]):
        gs += top[..., i]
    groups = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :M]
    ok = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, groups, True).repeat_interleave(E // G, 1)
    order = torch.sort(torch.where(ok, q, -math.inf), dim=1, descending=True, stable=True).indices
    return order[:, :case["k"]]


def _gates(s, idx, raw):
    sel = s.gather(1, idx)
    return 2.5 * sel if raw else 2.5 * sel / sel.sum(1, keepdim=True).clamp(min=1e-300 if s.dtype == F64 else 1e-37)


def _route(s, case):
    if own:
        s["L"].moe_route(s["cfg"], s["x"], s["wr"], s["offset"], s["bias"], s["scores"], s["flags"], s["idx"], s["gates"],
                         None if case["keep"] else s["ws"])
        return (s["idx"], s["gates"], s["scores"]) if case["keep"] else (s["idx"], s["gates"])
    logits = s["x"].float() @ s["wr"].float().T
    if s["offset"] is not None:
        logits = logits + s["offset"]
    scores = torch.softmax(logits.double(), 1).float()  # 64 bits: neighbouring affinities keep their order
    idx = _pick(scores, s["bias"], case)
    out = idx.to(I32), _gates(scores, idx, case["raw"])
    return (*out, scores) if case["keep"] else out


def _route_grad(s, case):
    if own:
        s["L"].moe_route_backward_flags(s["cfg"], s["flags"], s["x"], s["wr"], s["scores"], s["idx"], s["dgate"],
                                        case["alpha"], case["seq"], s["dx"], s["dw"], s["loss"], s["ws"])
        return s["dx"], s["dw"], s["loss"]
    T, E, k = case["T"], case["E"], case["k"]
    p, idx = s["scores"], s["idx"].long()
    sel = p.gather(1, idx)
    if case["raw"]:
        d = 2.5 * s["dgate"]
    else:
        S = sel.sum(1, keepdim=True)
        d = 2.5 / S * (s["dgate"] - (s["dgate"] * sel).sum(1, keepdim=True) / S)
    ds = torch.zeros_like(p).scatter_add_(1, idx, d)
    Lq = case["seq"] or T
    n = T // Lq
    total = p.sum(1, keepdim=True)
    norm = p / total
    chosen = torch.zeros_like(p).scatter_add_(1, idx, torch.ones_like(sel)).reshape(n, Lq, E).sum(1)
    f = chosen * (E / (k * Lq))
    loss = (case["alpha"] / n * (f * norm.reshape(n, Lq, E).mean(1)).sum()).reshape(1)
    c = (f * (case["alpha"] / (n * Lq))).repeat_interleave(Lq, 0)
    ds += (c - (c * norm).sum(1, keepdim=True)) / total
    dl = p * (ds - (p * ds).sum(1, keepdim=True))
    return dl @ s["wr"].float(), dl.T @ s["x"].float(), loss


def _swiglu(a, sa, w, sw, I):
    """int8 rows (as fp32) through gate and up weights, to bf16 and back to fp32."""
    gu = (a @ w.float().T) * (sa * sw)
    g, u = gu[:, :I], gu[:, I:]
    return (g * torch.sigmoid(g) * u).to(BF).float()


def _experts(s, case):
    T, H, S, I, k = case["T"], case["H"], case["S"], case["I"], case["k"]
    if own:
        L = s["L"]
        if case["rows"] == "sorted":
            L.moe_expert_ffn(s["cfg"], s["x_perm"], s["x_perm_s"], s["offsets"], s["w"], s["x"], s["y_perm"],
                             s["y_shared"], s["ws"])
        elif case["rows"] == "codes":
            L.moe_expert_ffn_codes(s["cfg"], s["xq"], s["xs"], s["perm"], s["offsets"], s["w"], s["y_perm"],
                                   s["y_shared"], s["ws"])
        else:
            L.moe_expert_ffn_gather(s["cfg"], s["x"], s["perm"], s["offsets"], s["w"], s["y_perm"], s["y_shared"],
                                    s["ws"])
        return (s["y_perm"], s["y_shared"]) if S else s["y_perm"]
    y = torch.empty((T * k, H), dtype=BF, device=DEV)
    tok = (s["perm"] // k).long()
    if case["rows"] == "codes":
        xq, xs = s["xq"].float(), s["xs"].unsqueeze(1)
    else:
        xq, a = _q8(s["x"].float())
        xs = a / 127
    for e in range(case["E"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if a == b:
            continue
        if case["rows"] == "sorted":
            rows, rs = s["x_perm"][a:b].float(), s["x_perm_s"][a:b].unsqueeze(1)
        else:
            rows, rs = xq[tok[a:b]], xs[tok[a:b]]
        hq, ha = _q8(_swiglu(rows, rs, s["wgu"][e], s["wgu_s"][e], I))
        y[a:b] = (hq @ s["wd"][e].float().T) * (ha / 127 * s["wd_s"][e])
    if not S:
        return y
    h = torch.cat([_swiglu(xq, xs, s["sgu"][e], s["sgu_s"][e], I) for e in range(S)], 1)
    hq, ha = _q8(h)
    ys = (hq @ s["sd"].float().permute(1, 0, 2).reshape(H, S * I).T) * (ha / 127 * s["sd_s"])
    return y, ys.to(BF)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, T, H = case["op"], case["T"], case["H"]
    if op == "norm":
        b = 4 if case["act"] == "f32" else 2
        row = H * b * (1 + 2 * case["residual"] + case["y"])
        row += {"int8": H + 4, "fp8_e4m3": H + H // 32, None: 0}[case["codes"]]
        return dict(bytes=case["live"] * row + H * b, flops=5 * case["live"] * H)
    if op == "norm_grad":
        b = 4 if case["act"] == "f32" else 2
        return dict(bytes=case["live"] * H * b * (2 + case["dh"]) + T * H * b + H * (b + 4), flops=10 * case["live"] * H)
    E, k = case["E"], case["k"]
    if op == "route":
        b = 4 if case["act"] == "f32" else 2
        return dict(bytes=(T + E) * H * b + T * k * 8 + (T * E * 4 if case["keep"] else 0), flops=2 * T * H * E)
    if op == "route_grad":
        return dict(bytes=(T + E) * H * 2 + T * E * 4 + T * k * 8 + (T + E) * H * 4, flops=2 * 2 * T * H * E)
    S, I = case["S"], case["I"]
    touched = E * (1 - (1 - k / E) ** T)              # experts that get a row, expected
    w = (touched + S) * 3 * H * I
    rows = T * k * H + (T * H * 2 if S else 0) if case["rows"] == "sorted" else T * H * (1 if case["rows"] == "codes" else 2)
    return dict(bytes=w + rows + (T * k + (T if S else 0)) * H * 2, flops=2 * 3 * H * I * T * (k + S))


# ------------------------------------------------------------------ the definition in 64 bits
def _whole(v):
    """int8 codes of float64 rows and their largest magnitudes: the nearest whole number of 127 v / max, ties to even."""
    top = v.abs().max(1, keepdim=True).values
    return torch.where(top > 0, torch.round(127.0 * v / torch.where(top > 0, top, 1.0)), 0.0), top


def exact(case, seed):
    s = prepare(case, seed)
    op, T, H = case["op"], case["T"], case["H"]
    if op == "norm":
        live = case["live"]
        w = s["w"].double()
        zero = lambda *sh, d=F64: torch.zeros(sh, dtype=d, device=DEV)
        out = {}
        if case["residual"]:
            out["h"] = zero(T, H)
        if case["y"]:
            out["y"] = zero(T, H)
        if case["codes"] == "int8":
            out["codes"], out["scale"] = zero(T, H, d=torch.int8), zero(T)
        elif case["codes"]:
            out["codes"], out["scale"] = None, zero(T, H // 128)       # (E4M3 codes are y / scale in 8 bits)
        for part in torch.arange(live, device=DEV).split(2048):
            h = s["x"][part].double()
            if case["residual"]:
                out["h"][part] = h + s["residual"][part].double()
                h = out["h"][part].to(s["x"].dtype).double()           # (the stored sum is what is normed)
            n = (h.square().sum(1, keepdim=True) / H + s["eps"]).sqrt()
            if case["y"]:
                out["y"][part] = h * w / n
            if case["codes"] == "int8":
                q, top = _whole(h * w)
                out["codes"][part] = q.to(torch.int8)
                out["scale"][part] = (top / (127.0 * n)).squeeze(1)
            elif case["codes"]:
                t = (h * w).reshape(part.numel(), H // 128, 128)
                top = t.abs().max(2, keepdim=True).values
                out["scale"][part] = (top / 448.0).squeeze(2) / n
        return out
    if op == "norm_grad":
        live = case["live"]
        w = s["w"].double()
        dx = torch.zeros((T, H), dtype=F64, device=DEV)
        dw = torch.zeros(H, dtype=F64, device=DEV)
        for part in torch.arange(live, device=DEV).split(2048):
            h, dy = s["x"][part].double(), s["dy"][part].double()
            n = (h.square().sum(1, keepdim=True) / H + s["eps"]).sqrt()
            u = h / n                                                  # y = u w, du/dh = (1 - u u^T / H) / n
            dw += (dy * u).sum(0)
            du = dy * w
            dx[part] = (du - u * (du * u).sum(1, keepdim=True) / H) / n
            if case["dh"]:
                dx[part] += s["dh"][part].double()
        return dx, dw
    E, k = case["E"], case["k"]
    if op == "route":
        logits = s["x"].double() @ s["wr"].double().transpose(0, 1).contiguous()
        if s["offset"] is not None:
            logits = (logits + s["offset"].double()).float().double()  # (the logit is an fp32 number)
        e = torch.exp(logits - logits.max(1, keepdim=True).values)
        p = e / e.sum(1, keepdim=True)
        q = p.float() + s["bias"]
        G, M, r = case["G"], case["M"], case["topr"]
        desc = torch.sort(q.reshape(T, G, E // G), dim=2, descending=True).values
        gs = desc[:, :, 0]
        for i in range(1, r):
            gs = gs + desc[:, :, i]
        mine, other = gs.unsqueeze(2), gs.unsqueeze(1)                 # rank: better groups, or as good and earlier
        earlier = torch.ones((G, G), dtype=torch.bool, device=DEV).tril(-1)
        chosen = ((other > mine) | ((other == mine) & earlier)).sum(2) < M
        left = torch.where(chosen.unsqueeze(2).expand(T, G, E // G).reshape(T, E), q.double(), -math.inf)
        picks = []
        at = torch.arange(E, device=DEV)
        for _ in range(k):
            best = left.max(1, keepdim=True).values
            i = torch.where(left == best, at, E).min(1, keepdim=True).values
            picks.append(i)
            left = left.scatter(1, i, -math.inf)
        idx = torch.cat(picks, 1)
        out = idx.to(I32), _gates(p, idx, case["raw"])
        return (*out, p) if case["keep"] else out
    if op == "route_grad":
        p, idx, dg = s["scores"].double(), s["idx"].long(), s["dgate"].double()
        Lq = case["seq"] or T
        n = T // Lq
        f = torch.zeros((n, E), dtype=F64, device=DEV)
        seq = (torch.arange(T, device=DEV) // Lq).unsqueeze(1).expand(T, k)
        f.index_put_((seq, idx), torch.ones((T, k), dtype=F64, device=DEV), accumulate=True)
        f *= E / (k * Lq)
        total = p.sum(1)
        mean = torch.zeros((n, E), dtype=F64, device=DEV).index_add_(0, seq[:, 0], p / total.unsqueeze(1)) / Lq
        loss = case["alpha"] / n * (f * mean).sum()
        c = case["alpha"] / (n * Lq) * f[seq[:, 0]]
        ds = c / total.unsqueeze(1) - ((c * p).sum(1) / total.square()).unsqueeze(1)
        t = torch.arange(T, device=DEV)
        sel = torch.stack([p[t, idx[:, j]] for j in range(k)], 1)
        S = sel.sum(1)
        for j in range(k):
            dj = 2.5 * dg[:, j] if case["raw"] else 2.5 * (dg[:, j] / S - (dg * sel).sum(1) / S.square())
            ds[t, idx[:, j]] += dj
        dl = p * ds - p * (p * ds).sum(1, keepdim=True)
        return dl @ s["wr"].double(), dl.transpose(0, 1).contiguous() @ s["x"].double(), loss.reshape(1)
    S, I = case["S"], case["I"]
    big = T * k * H > 1 << 27
    y = torch.empty((T * k, H), dtype=F32 if big else F64, device=DEV)
    if case["rows"] == "gather":
        xq, top = _whole(s["x"].double())
        xs = top / 127.0
    elif case["rows"] == "codes" or S:
        xq, xs = s["xq"].double(), s["xs"].double().unsqueeze(1)

    def hidden(q, sc, w, ws):
        gu = (q @ w.double().transpose(0, 1).contiguous()) * sc * ws.double()
        g, u = gu.split(I, 1)
        return (g / (1 + torch.exp(-g)) * u).to(BF).double()

    for e in range(E):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if b > a:
            if case["rows"] == "sorted":
                q, sc = s["x_perm"][a:b].double(), s["x_perm_s"][a:b].double().unsqueeze(1)
            else:
                t = (s["perm"][a:b] // k).long()
                q, sc = xq[t], xs[t]
            hq, top = _whole(hidden(q, sc, s["wgu"][e], s["wgu_s"][e]))
            y[a:b] = (hq @ s["wd"][e].double().transpose(0, 1).contiguous()) * (top / 127.0) * s["wd_s"][e].double()
    if not S:
        return y
    hs = [hidden(xq, xs, s["sgu"][e], s["sgu_s"][e]) for e in range(S)]
    top = torch.stack([h.abs().max(1).values for h in hs]).max(0).values.unsqueeze(1)
    ys = torch.zeros((T, H), dtype=F64, device=DEV)
    for e in range(S):
        q = torch.round(127.0 * hs[e] / torch.where(top > 0, top, 1.0))
        ys += q @ s["sd"][e].double().transpose(0, 1).contiguous()
    return y, ys * (top / 127.0) * s["sd_s"].double()
