"""Device buffers for one MoE layer and the five C-ABI calls in order.

MoeLayerGPU uploads a layer's weights once, allocates every buffer the calls
need for T tokens, and runs route -> dispatch -> expert FFN -> combine ->
bias update on the current stream.  It only allocates and marshals; every step
of the layer runs in libmoe's kernels.  With gather=True, dispatch writes only
the indices and the routed gate/up GEMM reads its rows from x through perm
(moe_expert_ffn_gather); no x_perm is allocated.  With save_gu=True (bf16),
the forward pass keeps the gate and up outputs (moe_expert_ffn_save) and the
backward pass starts from them (moe_expert_ffn_backward_saved) instead of
recomputing the gate/up GEMM.  With keep_scores=False, moe_route writes no
[T, E] affinities (a forward pass that needs no router gradient).

With share=(first, count) the layer holds the routed experts [first, first +
count) only, as one of several ranks does: the router still ranks all E, and
dispatch, combine and their gradients take the pairs that fall on its experts
(moe_dispatch_local and the calls beside it).  forward(n_tokens=...) takes an
int32 device tensor with the number of live tokens of a padded batch.  Either
way y (and dx) is this share's sum; the bias update needs the loads of the whole
batch, so gamma is refused.  The shares of the ranks add up to the layer when what
every rank could compute is given to one of them: the shared experts (the others'
cfg has S = 0) and the balance loss (adds_balance=True; the others pass alpha = 0).

With norm=w [H] the layer begins with a root-mean-square norm (moe_norm):
forward(x, residual=r) adds r to x (the sum stays in .h, for the next block's
residual), norms it, and routes and runs the experts on the result; with
gather=True int8 and FP8 experts take their rows as the norm's codes
(moe_expert_ffn_codes).  backward(dh=...) goes through the norm too.
softmax=True and raw_gates=True are moe_route's MOE_SOFTMAX and MOE_GATES_RAW.
"""
from __future__ import annotations

import numpy as np
import torch

from . import _lib as L


def to_device(arr, device="cuda"):
    """numpy float32 -> float32 tensor; numpy uint16 (bf16 bit patterns) -> bfloat16 tensor."""
    if arr is None:
        return None
    arr = np.ascontiguousarray(arr)
    if arr.dtype == np.uint16:
        return torch.from_numpy(arr.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(arr).to(device)


class MoeLayerGPU:
    norm = residual = graph_residual = codes = code_scale = None
    route_flags = 0
    scores_there = True      # the affinities of the last batch are in .scores

    def __init__(self, cfg, weights, T=None, device="cuda", gather=False, save_gu=False, keep_scores=True, share=None,
                 adds_balance=False, norm=None, eps=1e-6, softmax=False, raw_gates=False):
        self.c = cfg
        self.route_flags = (L.MOE_SOFTMAX if softmax else 0) | (L.MOE_GATES_RAW if raw_gates else 0)
        self.eps = eps
        self.share = share
        first, self.n_exp = (0, cfg.E) if share is None else (int(share[0]), int(share[1]))
        self.adds_balance = adds_balance or self.n_exp == cfg.E
        if first < 0 or self.n_exp < cfg.k or first + self.n_exp > cfg.E:
            raise ValueError(f"share {share} of {cfg.E} experts: needs at least k = {cfg.k} experts inside the layer's")
        if share is not None and len(weights.w_gate_up) not in (cfg.E, self.n_exp):
            raise ValueError(f"{len(weights.w_gate_up)} experts' weights for a share of {self.n_exp} of {cfg.E}")
        held = slice(first, first + self.n_exp) if share is not None and len(weights.w_gate_up) == cfg.E else slice(None)
        self.n_tokens = None
        self.device = device
        self.gather = gather
        self.save_gu = save_gu
        self.keep_scores = keep_scores
        self.fp8 = cfg.wgt == "fp8_e4m3"
        self.fp4 = cfg.wgt == "mxfp4"
        self.int8 = cfg.wgt == "int8"
        self.act_dtype = torch.float32 if cfg.act == "f32" else torch.bfloat16
        dev = lambda a: to_device(a, device)
        self.w_router = dev(weights.w_router)
        self.logit_offset = dev(weights.logit_offset)
        self.norm = dev(norm) if isinstance(norm, np.ndarray) else norm
        if self.norm is not None and (self.norm.shape != (cfg.H,) or self.norm.dtype != self.act_dtype):
            raise ValueError(f"norm is a weight of {cfg.H} values of {self.act_dtype}")
        if self.fp8 or self.fp4 or self.int8:
            self.w_gate_up, self.w_gate_up_scale = self._quantize(weights.w_gate_up[held])
            self.w_down, self.w_down_scale = self._quantize(weights.w_down[held])
            self.ws_gate_up, self.ws_gate_up_scale = self._quantize(weights.ws_gate_up)
            self.ws_down, self.ws_down_scale = self._quantize(weights.ws_down, joint=True)
        else:
            self.w_gate_up, self.w_down = dev(weights.w_gate_up[held]), dev(weights.w_down[held])
            self.ws_gate_up, self.ws_down = dev(weights.ws_gate_up), dev(weights.ws_down)
            self.w_gate_up_scale = self.w_down_scale = self.ws_gate_up_scale = self.ws_down_scale = None
        self.weights = L.expert_weights(self.w_gate_up, self.w_down, self.ws_gate_up, self.ws_down,
                                        self.w_gate_up_scale, self.w_down_scale, self.ws_gate_up_scale,
                                        self.ws_down_scale)
        self.alloc(cfg.T if T is None else T)

    def _quantize(self, w_np, joint=False):
        """bf16 weights [n, rows, cols] -> E4M3 codes + one fp32 scale per 128 x 128 block, or MXFP4 codes
        [n, rows, cols/2] + scale bytes [n, cols/128, rows, 4], or int8 codes + one fp32 scale a row [n, rows]
        (joint: [rows], over all n matrices) (on the GPU)."""
        n, rows, cols = w_np.shape
        if self.int8:
            codes = torch.empty((n, rows, cols), dtype=torch.int8, device=self.device)
            scales = torch.empty((rows,) if joint else (n, rows), dtype=torch.float32, device=self.device)
            if n:
                src = to_device(w_np, self.device)
                L.moe_quantize_int8(src, n, rows, cols, n if joint else 1, codes, scales)
                torch.cuda.current_stream().synchronize()
                del src
            return codes, scales
        if self.fp4:
            codes = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=self.device)
            scales = torch.empty((n, cols // 128, rows, 4), dtype=torch.uint8, device=self.device)
            if n:
                src = to_device(w_np, self.device)
                L.moe_quantize_fp4(src, n, rows, cols, codes, scales)
                torch.cuda.current_stream().synchronize()
                del src
            return codes, scales
        codes = torch.empty((n, rows, cols), dtype=torch.uint8, device=self.device)
        scales = torch.empty((n, rows // 128, cols // 128), dtype=torch.float32, device=self.device)
        if n:
            src = to_device(w_np, self.device)
            L.moe_quantize_fp8(src, n, rows, cols, 128, codes, scales)
            torch.cuda.current_stream().synchronize()
            del src
        return codes, scales

    def alloc(self, T):
        c = self.c
        self.T = T
        self.cfg = L.cfg_from(c, T=T)
        # the experts' configuration: the share's, whose experts form one group
        self.cfg_x = self.cfg if self.share is None else L.cfg_from(c, T=T, E=self.n_exp, G=1, M=1, group_topr=1)
        d, P = self.device, T * c.k
        f32, i32 = torch.float32, torch.int32
        # the [T, E] affinities (the backward pass reads them); without them moe_route
        # gets a workspace instead and a fused router kernel keeps them on chip
        self.scores = torch.empty((T, c.E), dtype=f32, device=d)
        self.ws_route = torch.empty(L.moe_workspace_bytes(self.cfg, L.MOE_WS_ROUTE), dtype=torch.uint8, device=d)
        self.topk_idx = torch.empty((T, c.k), dtype=i32, device=d)
        self.topk_w = torch.empty((T, c.k), dtype=f32, device=d)
        self.counts = torch.empty(self.n_exp, dtype=i32, device=d)
        self.offsets = torch.empty(self.n_exp + 1, dtype=i32, device=d)
        self.perm = torch.empty(P, dtype=i32, device=d)
        self.inv = torch.empty((T, c.k), dtype=i32, device=d)
        if self.gather:
            self.x_perm = self.x_perm_scale = None
        elif self.fp4:
            self.x_perm = torch.empty((P, c.H // 2), dtype=torch.uint8, device=d)
            self.x_perm_scale = torch.empty((c.H // 128, P, 4), dtype=torch.uint8, device=d)
        elif self.int8:
            self.x_perm = torch.empty((P, c.H), dtype=torch.int8, device=d)
            self.x_perm_scale = torch.empty(P, dtype=f32, device=d)
        elif self.fp8:
            self.x_perm = torch.empty((P, c.H), dtype=torch.uint8, device=d)
            self.x_perm_scale = torch.empty((P, c.H // 128), dtype=f32, device=d)
        else:
            self.x_perm = torch.empty((P, c.H), dtype=self.act_dtype, device=d)
            self.x_perm_scale = None
        self.y_perm = torch.empty((P, c.H), dtype=self.act_dtype, device=d)
        self.y_shared = torch.empty((T, c.H), dtype=self.act_dtype, device=d) if c.S > 0 else None
        self.y = torch.empty((T, c.H), dtype=self.act_dtype, device=d)
        self.ws_dispatch = torch.empty(L.moe_workspace_bytes(self.cfg_x, L.MOE_WS_DISPATCH), dtype=torch.uint8,
                                       device=d)
        self.ws_ffn = torch.empty(L.moe_workspace_bytes(self.cfg_x, L.MOE_WS_FFN), dtype=torch.uint8, device=d)
        self.codes = self.code_scale = None
        if self.norm is not None:
            # (zero: the rows behind the live tokens of a padded batch are not written)
            self.h = torch.zeros((T, c.H), dtype=self.act_dtype, device=d)
            self.xn = torch.zeros((T, c.H), dtype=self.act_dtype, device=d)
            if self.gather and (self.int8 or self.fp8):
                self.codes = torch.zeros((T, c.H), dtype=torch.int8 if self.int8 else torch.uint8, device=d)
                self.code_scale = torch.zeros((T,) if self.int8 else (T, c.H // 128), dtype=f32, device=d)
        if self.save_gu:
            bf = torch.bfloat16
            self.g = torch.empty((P, c.I), dtype=bf, device=d)
            self.u = torch.empty((P, c.I), dtype=bf, device=d)
            self.gs = torch.empty((T, c.S * c.I), dtype=bf, device=d) if c.S > 0 else None
            self.us = torch.empty((T, c.S * c.I), dtype=bf, device=d) if c.S > 0 else None
            self.saved = L.ffn_saved(self.g, self.u, self.gs, self.us)

    # ---------------------------------------------------------------- the five calls
    def add_and_norm(self, x, residual=None):
        """The norm in front of the layer: self.h = x + residual (h = x without one), returns the normed rows."""
        self.residual = residual
        L.moe_norm(self.cfg, self.n_tokens, x, residual, self.norm, self.eps, None if residual is None else self.h,
                   self.xn, self.codes, self.code_scale)
        return self.xn

    def route(self, x, bias, scores_in=False):
        keep = self.scores_there = self.keep_scores or scores_in
        flags = self.route_flags & ~L.MOE_SOFTMAX | L.MOE_SCORES_IN if scores_in else self.route_flags
        L.moe_route(self.cfg, x, self.w_router, self.logit_offset, bias, self.scores if keep else None,
                    flags, self.topk_idx, self.topk_w, None if keep else self.ws_route)

    @property
    def partial(self):
        """Whether some pairs of the batch may be absent (a share, or a padded batch)."""
        return self.share is not None or self.n_tokens is not None

    def dispatch(self, x):
        if self.partial:
            L.moe_dispatch_local(self.cfg_x, 0 if self.share is None else self.share[0], self.n_tokens, self.topk_idx, x,
                                 self.counts, self.offsets, self.perm, self.inv, self.x_perm, self.x_perm_scale,
                                 self.ws_dispatch)
            return
        L.moe_dispatch(self.cfg, self.topk_idx, x, self.counts, self.offsets, self.perm, self.inv, self.x_perm,
                       self.x_perm_scale, self.ws_dispatch)

    def expert_ffn(self, x, phase=L.MOE_FFN_ALL):
        if self.save_gu:
            L.moe_expert_ffn_save(self.cfg_x, self.x_perm, self.perm, self.offsets, self.weights, x, self.y_perm,
                                  self.y_shared, self.saved, self.ws_ffn, phase)
        elif self.codes is not None:
            L.moe_expert_ffn_codes(self.cfg_x, self.codes, self.code_scale, self.perm, self.offsets, self.weights,
                                   self.y_perm, self.y_shared, self.ws_ffn, phase)
        elif self.gather:
            L.moe_expert_ffn_gather(self.cfg_x, x, self.perm, self.offsets, self.weights, self.y_perm,
                                    self.y_shared, self.ws_ffn, phase)
        else:
            L.moe_expert_ffn(self.cfg_x, self.x_perm, self.x_perm_scale, self.offsets, self.weights, x,
                             self.y_perm, self.y_shared, self.ws_ffn, phase)

    def combine(self):
        combine = L.moe_combine_local if self.partial else L.moe_combine
        combine(self.cfg_x, self.y_perm, self.y_shared, self.inv, self.topk_w, self.y)

    def update_bias(self, bias, gamma):
        if self.partial:
            raise ValueError("the bias update needs the loads of a whole batch over every expert")
        L.moe_update_bias(self.cfg, self.counts, bias, gamma)

    # ---------------------------------------------------------------- backward
    def alloc_backward(self):
        """Gradient buffers for the current T (fp32 weight gradients, bf16 activation gradients)."""
        c, d = self.c, self.device
        T, P = self.T, self.T * c.k
        bf, f32 = torch.bfloat16, torch.float32
        self.dy_perm = torch.empty((P, c.H), dtype=bf, device=d)
        self.d_topk_w = torch.empty((T, c.k), dtype=f32, device=d)
        self.dx_perm = torch.empty((P, c.H), dtype=bf, device=d)
        self.dx_shared = torch.empty((T, c.H), dtype=bf, device=d) if c.S > 0 else None
        self.dx_router = torch.empty((T, c.H), dtype=f32, device=d)
        self.dx = torch.empty((T, c.H), dtype=bf, device=d)
        self.g_w_gate_up = torch.empty((self.n_exp, 2 * c.I, c.H), dtype=f32, device=d)
        self.g_w_down = torch.empty((self.n_exp, c.H, c.I), dtype=f32, device=d)
        self.g_ws_gate_up = torch.empty((c.S, 2 * c.I, c.H), dtype=f32, device=d) if c.S > 0 else None
        self.g_ws_down = torch.empty((c.S, c.H, c.I), dtype=f32, device=d) if c.S > 0 else None
        self.g_w_router = torch.empty((c.E, c.H), dtype=f32, device=d)
        self.loss_bal = torch.empty(1, dtype=f32, device=d)
        self.grads = L.expert_grads(self.g_w_gate_up, self.g_w_down, self.g_ws_gate_up, self.g_ws_down)
        self.ws_ffn_bwd = torch.empty(L.moe_workspace_bytes(self.cfg_x, L.MOE_WS_FFN_BWD), dtype=torch.uint8, device=d)
        kind = L.MOE_WS_ROUTE_BWD_SOFTMAX if self.route_flags else L.MOE_WS_ROUTE_BWD
        self.ws_route_bwd = torch.empty(L.moe_workspace_bytes(self.cfg, kind), dtype=torch.uint8, device=d)
        if self.norm is not None:
            self.dx_in = torch.empty((T, c.H), dtype=bf, device=d)
            self.g_norm = torch.empty(c.H, dtype=f32, device=d)
            self.ws_norm_bwd = torch.empty(L.moe_workspace_bytes(self.cfg, L.MOE_WS_NORM_BWD), dtype=torch.uint8,
                                           device=d)
        self._bwd_T = T

    def backward(self, x, dy, alpha=0.0, seq_len=0, dh=None):
        """Gradients of sum(dy * y) + alpha-weighted sequence balance loss for the last forward pass
        (same x, same routing).  Fills dx, the fp32 weight gradients and loss_bal; returns dx.
        Of a padded batch (n_tokens still holds its live count) they are the live tokens' gradients:
        what lies in the padded rows of x and dy takes no part, and those of dx are zero.
        With a norm dx is the gradient of x and of the residual, dh (or None) the one that reaches their sum from
        elsewhere, and g_norm the norm weight's."""
        if dh is not None and self.norm is None:
            raise ValueError("dh is the gradient of the norm's input sum: the layer has no norm")
        if dh is not None:
            self._check_rows("dh", dh)
        if self.norm is not None and self.residual is None:
            self._check_rows("x", x)                      # (the norm's input; with a residual that is self.h)
        if self.gather:
            raise ValueError("backward reads the permuted rows x_perm: build the layer with gather=False")
        if not self.scores_there:
            raise ValueError("backward reads the affinities: build the layer with keep_scores=True")
        if self.n_tokens is not None and alpha:
            raise ValueError("the balance loss counts every token of the batch: alpha has to be 0 for a padded one")
        if alpha and not self.adds_balance:
            raise ValueError("every share's gradients would hold the whole balance term: build one of them with "
                             "adds_balance=True, and pass alpha = 0 to the others")
        if getattr(self, "_bwd_T", None) != self.T:
            self.alloc_backward()
        cfg = self.cfg_x
        h = x if self.residual is None else self.h        # the norm's input
        if self.norm is not None:
            x = self.xn
        combine_backward = L.moe_combine_local_backward if self.partial else L.moe_combine_backward
        dispatch_backward = L.moe_dispatch_local_backward if self.partial else L.moe_dispatch_backward
        combine_backward(cfg, dy, self.y_perm, self.inv, self.topk_w, self.dy_perm, self.d_topk_w)
        scores = self.scores
        if self.n_tokens is not None:
            x, dy, scores = self._without_padding(x, dy)
        if self.save_gu:
            L.moe_expert_ffn_backward_saved(cfg, self.x_perm, x, self.offsets, self.weights, self.saved, self.dy_perm,
                                            dy, self.dx_perm, self.dx_shared, self.grads, self.ws_ffn_bwd)
        else:
            L.moe_expert_ffn_backward(cfg, self.x_perm, x, self.offsets, self.weights, self.dy_perm, dy,
                                      self.dx_perm, self.dx_shared, self.grads, self.ws_ffn_bwd)
        if self.route_flags:
            L.moe_route_backward_flags(self.cfg, self.route_flags, x, self.w_router, scores, self.topk_idx, self.d_topk_w,
                                       alpha, seq_len, self.dx_router, self.g_w_router, self.loss_bal,
                                       self.ws_route_bwd)
        else:
            L.moe_route_backward(self.cfg, x, self.w_router, scores, self.topk_idx, self.d_topk_w, alpha, seq_len,
                                 self.dx_router, self.g_w_router, self.loss_bal, self.ws_route_bwd)
        dispatch_backward(cfg, self.dx_perm, self.dx_shared, self.dx_router, self.inv, self.dx)
        if self.norm is None:
            return self.dx
        L.moe_norm_backward(self.cfg, self.n_tokens, h, self.norm, self.eps, self.dx, dh, self.dx_in, self.g_norm,
                            self.ws_norm_bwd)
        return self.dx_in

    def _without_padding(self, x, dy):
        """x, dy and the affinities with rows for the padded tokens that add exactly nothing.  The router's and the
        shared experts' gradients contract over all T rows; a padded row's gate gradients are zero, but zero times
        what lies there need not be."""
        live = self.n_tokens.reshape(1).to(self.device, non_blocking=True)   # (pinned host memory will do too)
        pad = (torch.arange(self.T, device=self.device) >= live).unsqueeze(1)
        if self.c.S > 0:
            dy = dy[:self.T].masked_fill(pad, 0)
            if self.save_gu:
                self.gs.masked_fill_(pad, 0)
                self.us.masked_fill_(pad, 0)
        scores = None if self.scores is None else self.scores.masked_fill(pad, 0.5)
        return x[:self.T].masked_fill(pad, 0), dy, scores

    def forward(self, x, bias, gamma=None, scores_in=False, n_tokens=None, residual=None):
        """One batch through the layer; with gamma set, bias is updated in place afterwards.
        n_tokens: int32 device tensor of one element, the live tokens of a padded batch; y of a padded token is the
        shared experts' output for whatever its row of x holds.
        residual: [T, H], added to x before the norm (layers with a norm)."""
        self._check_batch(gamma, n_tokens, residual)
        if self.norm is not None:
            self._check_rows("x", x)
        self.n_tokens = n_tokens
        if self.norm is not None:
            x = self.add_and_norm(x, residual)
        self.route(x, bias, scores_in)
        self.dispatch(x)
        self.expert_ffn(x)
        self.combine()
        if gamma is not None:
            self.update_bias(bias, gamma)
        return self.y

    def _check_batch(self, gamma, n_tokens, residual=None):
        """Refuses what forward() cannot run, before anything is launched."""
        L.live_count(n_tokens)
        if residual is not None:
            if self.norm is None:
                raise ValueError("a residual is added before the norm: the layer has none")
            self._check_rows("residual", residual)
        if gamma is not None and (self.share is not None or n_tokens is not None):
            raise ValueError("the bias update needs the loads of a whole batch over every expert")

    def _check_rows(self, name, t):
        if t.dim() != 2 or t.shape[0] < self.T or t.shape[1] != self.c.H or t.dtype != self.act_dtype:
            raise ValueError(f"{name} of shape {tuple(t.shape)}, {t.dtype}: needs {self.T} rows of {self.c.H}, "
                             f"{self.act_dtype}")

    # ---------------------------------------------------------------- HIP graph
    def capture(self, x, bias, gamma=None, n_tokens=None, residual=None):
        """Record one forward() over the tensors x and bias (and the bias update when
        gamma is set) into a HIP graph; replay() reruns it on whatever they (and n_tokens and residual) then hold.
        One graph serves every batch of this T: each launch is sized by capacity (the
        grouped GEMMs' tile tables are built on the device from the batch's routing)
        and no call allocates, copies or synchronises, so the recorded work is the
        same kernels forward() launches.  A warm-up pass (no bias update) on a side
        stream precedes the capture."""
        self._check_batch(gamma, n_tokens, residual)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward(x, bias, None, n_tokens=n_tokens, residual=residual)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.forward(x, bias, gamma, n_tokens=n_tokens, residual=residual)
        self.graph_inputs, self.graph_residual = (x, bias, n_tokens), residual
        return self.graph

    def replay(self):
        """One replay of the captured step on the current stream; returns y."""
        self.n_tokens = self.graph_inputs[2]     # backward() then takes the pairs that the graph's batch has
        self.residual = self.graph_residual
        self.scores_there = self.keep_scores
        self.graph.replay()
        return self.y
