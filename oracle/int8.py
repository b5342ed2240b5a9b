"""Oracle: symmetric int8 quantisation with one scale a row, and experts on it.

TEST INFRASTRUCTURE (see the package docstring).

A row with largest magnitude a stands for code * a / 127, code the whole number
nearest 127 v / a (ties to the even one).  A row of zeros has scale 0 and codes 0,
a row that holds an infinity or a NaN scale NaN and codes 0.  The shared experts
are one FFN of S * I columns: the rows of their W_d, and of their h, are quantised
over all of them.  h is rounded to bf16 before it is quantised.  Sums are exact.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def quantize_int8(v):
    """(codes int8 [R, K], scale fp64 [R]) of rows v [R, K]."""
    v = np.asarray(v, F64)
    a = np.abs(v).max(axis=1)
    bad = ~np.isfinite(v).all(axis=1)
    with np.errstate(invalid="ignore", divide="ignore"):
        codes = np.rint(127.0 * v / a[:, None])
    codes[bad | (a == 0)] = 0
    return codes.astype(np.int8), np.where(bad, np.nan, a / 127.0)


def round_bf16(v):
    """fp64 values rounded to bf16 (nearest, ties to even), as fp64; finite values inside the normal range."""
    v = np.asarray(v, F64)
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def hidden_int8(xc, xs, w_gate_up):
    """h (rounded to bf16, fp64 [n, I]) of rows xc * xs with the bf16 weights [2I, H] quantised by row."""
    wc, ws = quantize_int8(w_gate_up)
    c = (xc.astype(F64) @ wc.astype(F64).T) * xs[:, None] * ws
    I = len(wc) // 2
    a, u = c[:, :I], c[:, I:]
    with np.errstate(over="ignore"):
        return round_bf16(a / (1.0 + np.exp(-a)) * u)


def down_int8(hc, hs, w_down):
    """y [n, H] of rows hc * hs with the bf16 weights [H, I] quantised by row."""
    wc, ws = quantize_int8(w_down)
    return (hc.astype(F64) @ wc.astype(F64).T) * hs[:, None] * ws


def expert_int8(xc, xs, w_gate_up, w_down):
    return down_int8(*quantize_int8(hidden_int8(xc, xs, w_gate_up)), w_down)


def shared_int8(xc, xs, ws_gate_up, ws_down):
    """The shared experts' summed output: one FFN over all of their columns."""
    h = np.concatenate([hidden_int8(xc, xs, w) for w in ws_gate_up], axis=1)
    return down_int8(*quantize_int8(h), np.concatenate(list(ws_down), axis=1))
