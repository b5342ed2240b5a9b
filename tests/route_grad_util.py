"""Helpers of the tests of the router's gradients (no arithmetic of theirs but the bounds)."""
import numpy as np
import torch

from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import to_device
from gpu_util import dev_f32, dev_i32, host
from workloads.inputs import f32_to_bf16_bits

EPS32 = 2.0 ** -24


def grid(g, n, H, sigma, unit, most):
    """Normal values rounded to multiples of `unit` up to `most` of them."""
    return (np.clip(np.rint(g.standard_normal((n, H)) * sigma / unit), -most, most) * unit).astype(np.float32)


def backward(cfg, flags, x, w, s, idx, dg, alpha, seq, with_dx=True):
    """dx, dw and the loss of either entry point, into outputs and a workspace full of NaN."""
    kind = L.MOE_WS_ROUTE_BWD if flags is None else L.MOE_WS_ROUTE_BWD_SOFTMAX
    ws = torch.full((L.moe_workspace_bytes(cfg, kind),), 0xFF, dtype=torch.uint8, device="cuda")
    dx = torch.full((max(cfg.T, 1), cfg.H), float("nan"), device="cuda") if with_dx else None
    dw, loss = (torch.full(sh, float("nan"), device="cuda") for sh in ((cfg.E, cfg.H), (1,)))
    args = (to_device(f32_to_bf16_bits(x)), to_device(f32_to_bf16_bits(w)), dev_f32(s), dev_i32(idx), dev_f32(dg), alpha,
            seq, dx, dw, loss, ws)
    if flags is None:
        L.moe_route_backward(cfg, *args)
    else:
        L.moe_route_backward_flags(cfg, flags, *args)
    torch.cuda.synchronize()
    return None if dx is None else host(dx), host(dw), float(host(loss)[0])


def bounds(x, w, s, idx, dg, alpha, softmax, raw, terms, rows=slice(None)):
    """What dx (of some rows) and dw may be off by: 100 2^-24 of the magnitudes that make dlogit up and half a step of what it is
    stored as, one bf16 number or two, and (2 n + 8) 2^-24 of the sum of magnitudes in a product over n terms."""
    T, E = s.shape
    k = idx.shape[1]
    p = s.astype(np.float64)
    sel = np.take_along_axis(p, idx.astype(np.int64), 1)
    S = sel.sum(axis=1, keepdims=True)
    one = np.where(S == 0, 1.0, S)
    a = 2.5 * np.abs(dg) if raw else 2.5 / one * (np.abs(dg) + (np.abs(dg) * sel).sum(axis=1, keepdims=True) / one)
    A = np.zeros((T, E))
    np.put_along_axis(A, idx.astype(np.int64), a, axis=1)
    if alpha:
        total = p.sum(axis=1, keepdims=True)
        A += np.where(total == 0, 0.0, 2 * alpha * (E / k) / T / np.where(total == 0, 1.0, total))
    mag = p * (A + (p * A).sum(axis=1, keepdims=True)) if softmax else p * A
    # (below 2^-126 fp32 and bf16 have fewer bits, down to none, and a matrix product may take such a number for 0: it and
    # its second term are off by up to themselves, 2^-126 each.  It counts where dlogit itself has vanished.)
    dl = (100 * EPS32 + (2.0 ** -8 if terms == 1 else 2.0 ** -17)) * mag + 2 * 2.0 ** -126
    aw, ax = np.abs(w).astype(np.float64), np.abs(x).astype(np.float64)
    return (dl + (2 * E + 8) * EPS32 * mag)[rows] @ aw, (dl + (2 * T + 8) * EPS32 * mag).T @ ax
