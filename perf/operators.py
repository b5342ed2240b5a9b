"""Cases that measure the 4-bit expert path and the shares of a batch.

Four operators of one MoE layer, each reached through the C-ABI binding
(biased_top_routing_amd._lib):

  quantise   MXFP4 quantisation of bf16 rows and reading the codes back: 32
             neighbouring elements share a power of two X = 2^(e - 127) (one
             byte e), an element is a 4-bit E2M1 code c in {0, .5, 1, 1.5, 2, 3,
             4, 6} with a sign, standing for c X.  X is 2^(E - 2) with E the
             exponent of the block's largest magnitude rounded to one mantissa
             bit (so that no element is off by more than half a step), never
             below 2^-126; codes round to nearest, ties to the even code.
  experts    the SwiGLU experts on MXFP4 weights and activations:
             h = silu(q(x) Wg^T) * (q(x) Wu^T), y = q(h) Wd^T, with q() the
             quantisation above; routed experts on their rows, shared experts on
             every token.
  sort       dispatch of a share: the (token, slot) pairs of the first `live`
             tokens whose expert lies in [first, first + E), sorted by expert
             (stably), and their rows of x; every other pair is absent.
  back       combine of a share: y[t] = y_shared[t] + sum over the present
             slots of w[t, j] y_perm[inv[t, j]].
  grad       the gradients of back and sort: dy_perm = w dy, dw = <dy, y_perm>,
             dx[t] = sum over the present slots of dx_perm + dx_shared + dx_router.

`own` chooses the library's kernels or the plain torch form.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token's hidden row, quantised as it arrives (decode, latency)
        dict(name="quantise_row", op="quantise", n=1, rows=1, cols=7168, mag=1.0),
        # loading a checkpoint: the gate/up weights of 32 experts
        dict(name="quantise_weights", op="quantise", n=32, rows=4096, cols=7168, mag=0.006),
        # prefill of a V3-like layer, rows gathered from x
        dict(name="experts_prefill", op="experts", T=16384, H=7168, E=256, k=8, S=1, I=2048, skew=0.0, rows="gather"),
        # a mid-size layer on a skewed batch, rows already sorted and quantised; I is an odd multiple of 128
        dict(name="experts_mid", op="experts", T=4096, H=2048, E=64, k=6, S=2, I=1408, skew=1.1, rows="sorted"),
        # decode of a V3-like layer: a few rows an expert, the weights streamed once
        dict(name="experts_decode", op="experts", T=128, H=7168, E=256, k=8, S=1, I=2048, skew=0.0, rows="gather"),
        # a single token through the same layer
        dict(name="experts_token", op="experts", T=1, H=7168, E=256, k=8, S=1, I=2048, skew=0.0, rows="gather"),
        # one of 8 ranks holding 32 of 256 experts sorts its share of a padded prefill batch
        dict(name="sort_share", op="sort", T=16384, live=16001, H=7168, total=256, first=64, E=32, k=8, skew=0.0,
             act="bf16"),
        # a decode step padded to a graph's batch size, every expert held
        dict(name="sort_decode", op="sort", T=128, live=97, H=7168, total=256, first=0, E=256, k=8, skew=0.0,
             act="bf16"),
        # the same rank adds up its part of the layer's output
        dict(name="back_share", op="back", T=16384, live=16001, H=7168, total=256, first=64, E=32, k=8, skew=0.0,
             S=0, act="bf16"),
        # a small fp32 layer, padded, with a shared expert
        dict(name="back_small", op="back", T=256, live=201, H=128, total=16, first=0, E=16, k=4, skew=0.0, S=1,
             act="f32"),
        # the rank's training step
        dict(name="grad_share", op="grad", T=16384, live=16384, H=7168, total=256, first=96, E=32, k=8, skew=0.0,
             S=0, router=True),
        # a mid-size layer's padded training batch, every expert held, skewed
        dict(name="grad_mid", op="grad", T=4096, live=3801, H=2048, total=64, first=0, E=64, k=6, skew=1.1, S=2,
             router=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "experts", "experts", "sort", "back", "grad"])
    if op == "quantise":
        cols = 128 * _log(rng, 1, 64)
        n = _log(rng, 1, 32)
        rows = min(_log(rng, 1, 8192), (32 * 4096 * 7168) // (n * cols))
        return dict(op=op, n=n, rows=rows, cols=cols, mag=10.0 ** rng.uniform(-3, 2))
    if op == "experts":
        while True:
            H, I = 128 * _log(rng, 1, 64), 128 * _log(rng, 1, 24)
            E = _log(rng, 1, 256)
            k = rng.randint(1, min(8, E))
            S = rng.choice([0, 1, 1, 2, 3])
            T = _log(rng, 1, 16384)
            c = dict(op=op, T=T, H=H, E=E, k=k, S=S, I=I, skew=rng.choice([0.0, 0.5, 1.1]),
                     rows=rng.choice(["gather", "sorted"]))
            if E * H * I <= 256 * 7168 * 2048 and T * (k + S) * H * max(I, S * I) <= 16384 * 9 * 7168 * 2048:
                return c
    total = _log(rng, 2, 256)
    E = rng.choice([total, max(1, total // 2), max(1, total // 8)])
    first = rng.randint(0, total - E)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 16384)
    c = dict(op=op, T=T, live=rng.choice([T, rng.randint(0, T)]), H=64 * _log(rng, 2, 112), total=total, first=first,
             E=E, k=k, skew=rng.choice([0.0, 1.1]))
    if op == "sort":
        c["act"] = rng.choice(["bf16", "bf16", "f32"])
    elif op == "back":
        c.update(S=rng.choice([0, 1]), act=rng.choice(["bf16", "bf16", "f32"]))
    else:
        c.update(S=rng.choice([0, 1]), router=rng.choice([True, False]))
    return c


# ------------------------------------------------------------------ MXFP4, plain
def _block_scale(amax):
    """X of blocks with largest magnitude amax (fp32): its exponent after rounding to one mantissa bit, less 2."""
    bits = amax.view(torch.int32)
    e = (((bits + 0x200000) >> 23) - 2).clamp_(min=1)
    return (e << 23).view(torch.float32)


def _round_e2m1(a):
    """|a| to the nearest E2M1 magnitude, ties to the even code."""
    r = torch.where(a < 2, (a * 2).round() * 0.5, torch.where(a < 4, a.round(), (a * 0.5).round() * 2))
    return r.clamp_(max=6.0)


def _fq(v):
    """The MXFP4 values (fp32) of fp32 rows [..., cols], cols % 32 == 0."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    x = _block_scale(b.abs().amax(-1, keepdim=True))
    q = b / x
    return (torch.copysign(_round_e2m1(q.abs()), q) * x).reshape(v.shape)


def _encode(v):
    """fp32 rows [n, rows, cols] -> packed codes [n, rows, cols/2] (the even element in the low half byte) and
    scale bytes [n, cols/128, rows, 4]."""
    n, rows, cols = v.shape
    b = v.reshape(n, rows, cols // 32, 32)
    x = _block_scale(b.abs().amax(-1, keepdim=True))
    q = b / x
    m = _round_e2m1(q.abs())
    code = torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m * 0.5 + 4)).to(torch.uint8)
    code |= torch.signbit(q).to(torch.uint8) << 3
    code = code.reshape(n, rows, cols // 2, 2)
    packed = code[..., 0] | (code[..., 1] << 4)
    e = (x.view(torch.int32) >> 23).to(torch.uint8).reshape(n, rows, cols // 128, 4)
    return packed.contiguous(), e.permute(0, 2, 1, 3).contiguous()


def _decode(packed, scale, dtype):
    """Packed codes [n, rows, cols/2] and scale bytes [n, cols/128, rows, 4] -> values [n, rows, cols]."""
    n, rows, half = packed.shape
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=packed.device)
    c = torch.stack((packed & 15, packed >> 4), -1).reshape(n, rows, half * 2)
    e = scale.permute(0, 2, 1, 3).reshape(n, rows, half // 16, 1)
    x = (e.to(torch.int32) << 23).view(torch.float32).to(dtype)
    return (lut[c.to(torch.int32)].reshape(n, rows, half // 16, 32) * x).reshape(n, rows, half * 2)


# ------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + salt)
    return g


def _weights(n, rows, cols, sigma, g):
    """n random matrices in MXFP4: packed codes and scale bytes, made one matrix at a time."""
    codes = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((n, cols // 128, rows, 4), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (rows * cols))
    for i in range(0, n, step):
        m = min(step, n - i)
        v = torch.randn((m, rows, cols), generator=g, device=DEV) * sigma
        codes[i:i + m], scale[i:i + m] = _encode(v)
    return codes, scale


def _choose(T, total, k, skew, g):
    """k distinct experts a token, popularity ~ rank^-skew (ranks shuffled), and gates summing to 2.5."""
    rank = torch.randperm(total, generator=g, device=DEV).float() + 1
    u = torch.rand((T, total), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    idx = (-skew * rank.log() - (-u.log()).log()).topk(k, dim=1).indices.to(torch.int32)
    w = torch.rand((T, k), generator=g, device=DEV) + 0.05
    return idx.contiguous(), (2.5 * w / w.sum(1, keepdim=True)).contiguous()


def _present(idx, case):
    t = torch.arange(case["T"], device=DEV).unsqueeze(1)
    rel = idx - case["first"]
    return rel, (rel >= 0) & (rel < case["E"]) & (t < case["live"])


def _sorted(idx, case):
    """counts, offsets, perm and inv of the present pairs (absent: inv -1, rows behind the last 0)."""
    E, P = case["E"], idx.numel()
    rel, here = _present(idx, case)
    key = torch.where(here, rel, E).reshape(-1)
    order = torch.sort(key, stable=True).indices
    counts = (key.unsqueeze(0) == torch.arange(E, device=DEV).unsqueeze(1)).sum(1) if P * E <= 1 << 24 else \
        torch.zeros(E + 1, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(key, dtype=torch.int64))[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts.cumsum(0)
    pos = torch.arange(P, device=DEV)
    live = pos < offsets[E]
    perm = torch.where(live, order, 0)
    inv = torch.empty(P, dtype=torch.int64, device=DEV)
    inv[order] = torch.where(live, pos, -1)
    i32 = torch.int32
    return counts.to(i32), offsets.to(i32), perm.to(i32), inv.to(i32).reshape(idx.shape), live


def prepare(case, seed):
    op = case["op"]
    s = dict(case=case)
    if op == "quantise":
        g = _gen(seed, 1)
        n, rows, cols = case["n"], case["rows"], case["cols"]
        x = torch.empty((n, rows, cols), dtype=torch.bfloat16, device=DEV)
        for i in range(n):
            v = torch.randn((rows, cols), generator=g, device=DEV) * case["mag"]
            v *= 1 + 30 * (torch.rand((rows, cols), generator=g, device=DEV) > 0.999)   # outliers
            x[i] = v
            x[i, rows // 2, : cols // 2 // 32 * 32] = 0                                   # a padded piece of a row
        s["x"] = x
        if own:
            s["codes"] = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=DEV)
            s["scale"] = torch.empty((n, cols // 128, rows, 4), dtype=torch.uint8, device=DEV)
            s["out"] = torch.empty_like(x)
        return s
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    P = T * k
    if op == "experts":
        g = _gen(seed, 2)
        S, I = case["S"], case["I"]
        s["x"] = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
        idx, _ = _choose(T, E, k, case["skew"], g)
        _, s["offsets"], s["perm"], _, _ = _sorted(idx, dict(T=T, first=0, E=E, live=T))
        s["bounds"] = s["offsets"].tolist()
        sg, sd = 1.0 / math.sqrt(H), 1.0 / math.sqrt(I)
        s["wgu"], s["wgu_s"] = _weights(E, 2 * I, H, sg, g)
        s["wd"], s["wd_s"] = _weights(E, H, I, sd, g)
        s["sgu"], s["sgu_s"] = _weights(S, 2 * I, H, sg, g)
        s["sd"], s["sd_s"] = _weights(S, H, I, sd, g)
        if case["rows"] == "sorted":
            xp, xs = _encode(s["x"].float().unsqueeze(0))
            tok = (s["perm"] // k).long()
            s["x_perm"], s["x_perm_s"] = xp[0][tok].contiguous(), xs[0][:, tok].contiguous()
        if own:
            from biased_top_routing_amd import _lib as L
            s["L"] = L
            s["cfg"] = L.make_cfg(T, H, E, 1, 1, k, S, I, 1, 1.0, "bf16", "mxfp4")
            sh = (s["sgu"], s["sd"]) if S else (None, None)
            shs = (s["sgu_s"], s["sd_s"]) if S else (None, None)
            s["w"] = L.expert_weights(s["wgu"], s["wd"], *sh, s["wgu_s"], s["wd_s"], *shs)
            s["ws"] = torch.empty(L.moe_workspace_bytes(s["cfg"], L.MOE_WS_FFN), dtype=torch.uint8, device=DEV)
            s["y_perm"] = torch.empty((P, H), dtype=torch.bfloat16, device=DEV)
            s["y_shared"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV) if S else None
        return s
    g = _gen(seed, 3)
    dt = torch.float32 if case.get("act", "bf16") == "f32" else torch.bfloat16
    s["idx"], s["w"] = _choose(T, case["total"], k, case["skew"], g)
    rand = lambda n, d: torch.randn((n, H), generator=g, device=DEV).to(d)
    s["n"] = torch.tensor([case["live"]], dtype=torch.int32, device=DEV)
    S = case.get("S", 0)
    if op == "sort":
        s["x"] = rand(T, dt)
    else:
        _, _, _, s["inv"], live = _sorted(s["idx"], case)
        s["y_perm"] = rand(P, dt)
        s["y_shared"] = rand(T, dt) if S else None
        if op == "grad":
            s["live_rows"] = live
            s["dy"] = rand(T, dt)
            s["dx_perm"] = rand(P, dt)
            s["dx_shared"] = rand(T, dt) if S else None
            s["dx_router"] = rand(T, torch.float32) if case["router"] else None
    if own:
        from biased_top_routing_amd import _lib as L
        s["L"] = L
        act = case.get("act", "bf16")
        s["cfg"] = L.make_cfg(T, H, E, 1, 1, k, S, 128, 1, 1.0, act, act)
        z = lambda *sh, d=torch.int32: torch.zeros(sh, dtype=d, device=DEV)
        if op == "sort":
            s["ws"] = torch.empty(L.moe_workspace_bytes(s["cfg"], L.MOE_WS_DISPATCH), dtype=torch.uint8, device=DEV)
            # rows behind the last present pair stay as they were: zero
            s["out"] = (z(E), z(E + 1), z(P), z(T, k), z(P, H, d=dt))
        elif op == "back":
            s["y"] = z(T, H, d=dt)
        else:
            s["out"] = (z(P, H, d=dt), z(T, k, d=torch.float32), z(T, H, d=dt))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    return {"quantise": _quantise, "experts": _experts, "sort": _sort, "back": _back, "grad": _grad}[case["op"]](s, case)


def _quantise(s, case):
    x = s["x"]
    if own:
        from biased_top_routing_amd import _lib as L
        L.moe_quantize_fp4(x, case["n"], case["rows"], case["cols"], s["codes"], s["scale"])
        L.moe_dequantize_fp4(s["codes"], s["scale"], case["n"], case["rows"], case["cols"], s["out"])
        return s["out"]
    out = torch.empty_like(x)
    step = max(1, (1 << 28) // (case["rows"] * case["cols"]))
    for i in range(0, case["n"], step):
        out[i:i + step] = _fq(x[i:i + step].float())
    return out


def _swiglu(a, wgu, I):
    g, u = (a @ wgu[:, :I].flatten(0, 1).T), (a @ wgu[:, I:].flatten(0, 1).T)
    return g * torch.sigmoid(g) * u


def _experts(s, case):
    if own:
        L = s["L"]
        if case["rows"] == "sorted":
            L.moe_expert_ffn(s["cfg"], s["x_perm"], s["x_perm_s"], s["offsets"], s["w"], s["x"], s["y_perm"],
                             s["y_shared"], s["ws"])
        else:
            L.moe_expert_ffn_gather(s["cfg"], s["x"], s["perm"], s["offsets"], s["w"], s["y_perm"], s["y_shared"],
                                    s["ws"])
        return (s["y_perm"], s["y_shared"]) if case["S"] else s["y_perm"]
    T, H, S, I, k = case["T"], case["H"], case["S"], case["I"], case["k"]
    y = torch.empty((T * k, H), dtype=torch.bfloat16, device=DEV)
    f32 = torch.float32
    xq = _fq(s["x"].float())
    tok = s["perm"] // k
    for e in range(case["E"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if a == b:
            continue
        if case["rows"] == "sorted":
            rows = _decode(s["x_perm"][None, a:b], s["x_perm_s"][None, :, a:b], f32)[0]
        else:
            rows = xq[tok[a:b]]
        h = _fq(_swiglu(rows, _decode(s["wgu"][e:e + 1], s["wgu_s"][e:e + 1], f32), I))
        y[a:b] = h @ _decode(s["wd"][e:e + 1], s["wd_s"][e:e + 1], f32)[0].T
    if not S:
        return y
    acc = torch.zeros((T, H), dtype=f32, device=DEV)
    for e in range(S):
        h = _fq(_swiglu(xq, _decode(s["sgu"][e:e + 1], s["sgu_s"][e:e + 1], f32), I))
        acc += h @ _decode(s["sd"][e:e + 1], s["sd_s"][e:e + 1], f32)[0].T
    return y, acc.to(torch.bfloat16)


def _sort(s, case):
    if own:
        counts, offsets, perm, inv, x_perm = s["out"]
        s["L"].moe_dispatch_local(s["cfg"], case["first"], s["n"], s["idx"], s["x"], counts, offsets, perm, inv, x_perm,
                                  None, s["ws"])
        return s["out"]
    counts, offsets, perm, inv, live = _sorted(s["idx"], case)
    x_perm = torch.where(live.unsqueeze(1), s["x"][perm // case["k"]], 0)
    return counts, offsets, perm, inv, x_perm


def _back(s, case):
    if own:
        s["L"].moe_combine_local(s["cfg"], s["y_perm"], s["y_shared"], s["inv"], s["w"], s["y"])
        return s["y"]
    acc = torch.zeros((case["T"], case["H"]), dtype=torch.float32, device=DEV)
    if s["y_shared"] is not None:
        acc += s["y_shared"]
    for j in range(case["k"]):
        p = s["inv"][:, j]
        row = s["y_perm"][p.clamp(min=0)].float() * s["w"][:, j:j + 1]
        acc += torch.where((p >= 0).unsqueeze(1), row, 0)
    return acc.to(s["y_perm"].dtype)


def _grad(s, case):
    if own:
        dy_perm, dw, dx = s["out"]
        L = s["L"]
        L.moe_combine_local_backward(s["cfg"], s["dy"], s["y_perm"], s["inv"], s["w"], dy_perm, dw)
        L.moe_dispatch_local_backward(s["cfg"], s["dx_perm"], s["dx_shared"], s["dx_router"], s["inv"], dx)
        return s["out"]
    T, H, k = case["T"], case["H"], case["k"]
    dy = s["dy"].float()
    dy_perm = torch.zeros((T * k + 1, H), dtype=torch.bfloat16, device=DEV)   # absent pairs write the last row
    dw = torch.zeros((T, k), dtype=torch.float32, device=DEV)
    acc = torch.zeros((T, H), dtype=torch.float32, device=DEV)
    for j in range(k):
        p = s["inv"][:, j]
        here = p >= 0
        q = p.clamp(min=0)
        dw[:, j] = torch.where(here, (s["y_perm"][q].float() * dy).sum(1), 0)
        acc += torch.where(here.unsqueeze(1), s["dx_perm"][q].float(), 0)
        dy_perm[torch.where(here, p, T * k).long()] = (dy * s["w"][:, j:j + 1]).to(torch.bfloat16)
    if s["dx_shared"] is not None:
        acc += s["dx_shared"]
    if s["dx_router"] is not None:
        acc += s["dx_router"]
    return dy_perm[:-1], dw, acc.to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantise":   # bf16 in; codes, scale bytes and the values read back out
        return dict(bytes=case["n"] * case["rows"] * case["cols"] * (2 + 0.5 + 1 / 32 + 2), flops=0)
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    if op == "experts":
        S, I = case["S"], case["I"]
        touched = E * (1 - (1 - k / E) ** T)          # experts that get a row, expected
        w = (touched + S) * 3 * H * I * (0.5 + 1 / 32)
        rows = T * k * H * (0.5 + 1 / 32) + (T * H * 2 if S else 0) if case["rows"] == "sorted" else T * H * 2 + T * k * 4
        return dict(bytes=w + rows + (T * k + (T if S else 0)) * H * 2, flops=2 * 3 * H * I * T * (k + S))
    b = 4 if case.get("act", "bf16") == "f32" else 2
    share = E / case["total"]
    pairs = case["live"] * k * share                   # present pairs, expected
    some = case["live"] * (1 - (1 - share) ** k)       # tokens with one at least
    if op == "sort":
        return dict(bytes=T * k * 4 * 2 + pairs * 4 + (some + pairs) * H * b, flops=0)
    if op == "back":
        return dict(bytes=(pairs + T + (T if case["S"] else 0)) * H * b + T * k * 8, flops=2 * pairs * H)
    extra = (2 if case["S"] else 0) + (4 if case["router"] else 0)
    return dict(bytes=(3 * pairs + some + T) * H * 2 + T * H * extra + T * k * 12, flops=4 * pairs * H)


# ------------------------------------------------------------------ the definition in 64 bits
def _pow2(e):
    """2^e in float64, from its bits (a device's pow may be off by a last place)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _x_values(v):
    """MXFP4 values of float64 rows, straight from the definition: the block's power of two, then the nearest
    of the 8 magnitudes (a tie goes to the even code)."""
    rows = v.reshape(-1, 32)
    top = rows.abs().max(1, keepdim=True).values
    m, e = torch.frexp(top)                                   # top = m 2^e, m in [1/2, 1): 1.75 2^(e-1) is m = 7/8
    e = (e - 1 + (m >= 0.875).to(e.dtype) - 2).clamp(min=-126)
    e = torch.where(top == 0, torch.full_like(e, -126), e)
    x = _pow2(e)
    a = rows.abs() / x
    mag = torch.zeros_like(a)
    for i in range(1, 8):
        mid = (E2M1[i - 1] + E2M1[i]) / 2
        mag = torch.where(a >= mid if i % 2 == 0 else a > mid, torch.full_like(a, E2M1[i]), mag)
    return (rows.sign() * mag * x).reshape(v.shape)


def _w64(codes, scale):
    """One MXFP4 matrix in float64: codes [rows, cols/2], scale bytes [cols/128, rows, 4]."""
    rows, half = codes.shape
    table = torch.tensor([(-1.0 if i > 7 else 1.0) * E2M1[i & 7] for i in range(16)], dtype=torch.float64, device=DEV)
    v = torch.empty((rows, half * 2), dtype=torch.float64, device=DEV)
    v[:, 0::2] = table[(codes % 16).long()]
    v[:, 1::2] = table[(codes // 16).long()]
    x = _pow2(scale.transpose(0, 1).reshape(rows, half // 16).to(torch.int64) - 127)
    return v * x.repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "quantise":
        return torch.stack([torch.cat([_x_values(part.double()).to(torch.float32) for part in m.split(512)])
                            for m in s["x"]]) if s["x"].numel() <= 1 << 27 else \
            torch.cat([_x_values(part.double()).to(torch.bfloat16) for part in s["x"].flatten(0, 1).split(4096)]
                      ).reshape(s["x"].shape)
    T, H, k = case["T"], case["H"], case["k"]
    if op == "experts":
        I = case["I"]
        y = torch.empty((T * k, H), dtype=torch.float32 if T * k * H > 1 << 27 else f64, device=DEV)
        xq = _x_values(s["x"].double())

        def expert(rows, wgu, wgu_s, wd, wd_s):
            gu = rows @ _w64(wgu, wgu_s).transpose(0, 1).contiguous()
            g, u = gu[:, :I], gu[:, I:]
            return _x_values(g / (1 + torch.exp(-g)) * u) @ _w64(wd, wd_s).transpose(0, 1).contiguous()

        for e in range(case["E"]):
            a, b = s["bounds"][e], s["bounds"][e + 1]
            if b > a:
                y[a:b] = expert(xq[(s["perm"][a:b] // k).long()], s["wgu"][e], s["wgu_s"][e], s["wd"][e], s["wd_s"][e])
        if not case["S"]:
            return y
        ys = torch.zeros((T, H), dtype=f64, device=DEV)
        for e in range(case["S"]):
            ys += expert(xq, s["sgu"][e], s["sgu_s"][e], s["sd"][e], s["sd_s"][e])
        return y, ys
    if op == "sort":
        idx = s["idx"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(case["E"])]
        for f in range(case["live"] * k):
            e = idx[f] - case["first"]
            if 0 <= e < case["E"]:
                lists[e].append(f)
        perm = [f for one in lists for f in one]
        ends = [0]
        for one in lists:
            ends.append(ends[-1] + len(one))
        inv = [-1] * (T * k)
        for p, f in enumerate(perm):
            inv[f] = p
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
        x_perm = torch.zeros((T * k, H), dtype=s["x"].dtype, device=DEV)
        if perm:
            x_perm[:len(perm)] = s["x"].index_select(0, (i32(perm) // k).long())
        return (i32([len(one) for one in lists]), i32(ends), i32(perm + [0] * (T * k - len(perm))),
                i32(inv).reshape(T, k), x_perm)
    rows = s["inv"].reshape(-1)
    f = torch.nonzero(rows >= 0).reshape(-1)                  # the present pairs
    tok, p = f // k, rows[f].long()
    if op == "back":
        y = torch.zeros((T, H), dtype=f64, device=DEV) if s["y_shared"] is None else s["y_shared"].double()
        w = s["w"].reshape(-1)[f].double().unsqueeze(1)
        for part in torch.arange(f.numel(), device=DEV).split(8192):
            y.index_add_(0, tok[part], s["y_perm"][p[part]].double() * w[part])
        return y
    big = T * k * H > 1 << 27
    dy_perm = torch.zeros((T * k, H), dtype=torch.float32 if big else f64, device=DEV)
    dw = torch.zeros(T * k, dtype=f64, device=DEV)
    dx = torch.zeros((T, H), dtype=f64, device=DEV)
    w = s["w"].reshape(-1)[f].double().unsqueeze(1)
    for part in torch.arange(f.numel(), device=DEV).split(8192):
        d = s["dy"][tok[part]].double()
        dy_perm[p[part]] = (d * w[part]).to(dy_perm.dtype)
        dw[f[part]] = (d * s["y_perm"][p[part]].double()).sum(1)
        dx.index_add_(0, tok[part], s["dx_perm"][p[part]].double())
    for extra in (s["dx_shared"], s["dx_router"]):
        if extra is not None:
            dx += extra.double()
    return dy_perm, dw.reshape(T, k), dx
