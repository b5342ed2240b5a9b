"""Calls of the norm, the routing and the int8 experts that the documentation allows beside the usual ones: outputs left out,
live counts past the ends or in pinned memory, empty batches, another stream, two graphs over one workspace.

Each is compared bit for bit with the usual call, whose results are compared with the formulas elsewhere."""
import numpy as np
import pytest
import torch

from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU, to_device
from gpu_util import dev_f32, host, say
from workloads import MID
from workloads.inputs import f32_to_bf16_bits, make_weights, make_x, rng

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _rows(T, H, act, *salt):
    v = rng(251, T, H, *salt).standard_normal((T, H)).astype(np.float32)
    return to_device(v if act == "f32" else f32_to_bf16_bits(v))


def _dt(act):
    return torch.float32 if act == "f32" else torch.bfloat16


def _norm(T, H, act, wgt, n, x, res, w, h=True, y=True, codes=False, fill=3):
    new = lambda *s, d=_dt(act): torch.full(s, fill, dtype=d, device="cuda")
    out = dict(h=new(T, H) if h else None, y=new(T, H) if y else None,
               q=new(T, H, d=torch.int8) if codes else None,
               s=new(*((T,) if wgt == "int8" else (T, H // 128)), d=torch.float32) if codes else None)
    L.moe_norm(L.make_cfg(T, H, 1, 1, 1, 1, 0, 128, 1, 1.0, act, wgt), n, x, res, w, EPS, out["h"], out["y"], out["q"], out["s"])
    torch.cuda.synchronize()
    return out


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T,H,act,wgt", [(5, 256, "bf16", "int8"), (9, 2048, "bf16", "fp8_e4m3"), (9, 7168, "bf16", "int8"),
                                         (3, 16512, "bf16", "int8"), (3, 33408, "bf16", "bf16"), (7, 132, "f32", "f32"),
                                         (2, 20004, "f32", "f32"), (4, 8192, "bf16", "fp8_e4m3")])
def test_norm_with_outputs_left_out(T, H, act, wgt):
    """The sum not stored (rows longer than the registers add it up again), the normed rows or the codes not wanted."""
    say(f"norm, outputs left out, T={T} H={H} {act} {wgt}")
    codes = wgt not in (act, "bf16")
    x, res, w = _rows(T, H, act, 0), _rows(T, H, act, 1), _rows(1, H, act, 2).reshape(H)
    for r in (res, None):
        want = _norm(T, H, act, wgt, None, x, r, w, codes=codes)
        for h in (False, True):
            for y in (False, True) if codes else (True,):
                for q in (False, True) if codes and y else (codes,):
                    got = _norm(T, H, act, wgt, None, x, r, w, h, y, q)
                    for k, v in got.items():
                        assert v is None or _same(v, want[k]), (k, h, y, q)


@pytest.mark.parametrize("wgt", ["int8", "fp8_e4m3"])
def test_live_counts_past_the_ends(wgt):
    """Taken as 0 when negative and as T when larger; on the device or in pinned host memory."""
    T, H = 70, 512
    x, res, w = _rows(T, H, "bf16", 0), _rows(T, H, "bf16", 1), _rows(1, H, "bf16", 2).reshape(H)
    dy = _rows(T, H, "bf16", 3)
    cfg = L.make_cfg(T, H, 1, 1, 1, 1, 0, 128, 1, 1.0, "bf16", wgt)
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_NORM_BWD), dtype=torch.uint8, device="cuda")

    def both(n):
        out = _norm(T, H, "bf16", wgt, n, x, res, w, codes=True)
        dx, dw = torch.full_like(dy, 7), torch.full((H,), 7.0, device="cuda")
        L.moe_norm_backward(cfg, n, x, w, EPS, dy, None, dx, dw, ws)
        torch.cuda.synchronize()
        return [*out.values(), dx, dw]

    count = lambda v, pin=False: torch.tensor([v], dtype=torch.int32).pin_memory() if pin else \
        torch.tensor([v], dtype=torch.int32, device="cuda")
    say(f"live counts past the ends, {wgt}")
    whole, none = both(None), both(count(0))
    for n in (count(T), count(T + 1), count(2 ** 31 - 1), count(T, True), count(T + 9, True)):
        assert all(_same(a, b) for a, b in zip(both(n), whole))
    for n in (count(-1), count(-2 ** 31), count(0, True)):
        assert all(_same(a, b) for a, b in zip(both(n), none))
    assert (none[-2] == 0).all() and (none[-1] == 0).all() and (none[0] == 3).all()


def test_empty_batches():
    """T = 0: nothing is written but what is a sum over the tokens."""
    say("empty batches")
    H, E, I = 256, 8, 128
    one = torch.full((4096,), 3, dtype=torch.uint8, device="cuda")
    for wgt in ("int8", "fp8_e4m3", "bf16"):
        cfg = L.make_cfg(0, H, E, 1, 1, 2, 1, I, 1, 1.0, "bf16", wgt)
        L.moe_norm(cfg, None, None, None, None, EPS, None, None)
        dw = torch.full((H,), 7.0, device="cuda")
        ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_NORM_BWD), dtype=torch.uint8, device="cuda")
        L.moe_norm_backward(cfg, None, None, one, EPS, None, None, None, dw, ws)
        for flags in (0, L.MOE_SOFTMAX, L.MOE_GATES_RAW, L.MOE_SOFTMAX | L.MOE_GATES_RAW):
            L.moe_route(cfg, one, one, None, one, one, flags, one, one)
        if wgt != "bf16":
            w = L.expert_weights(one, one, one, one, one, one, one, one)
            offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
            wsf = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_FFN), dtype=torch.uint8, device="cuda")
            L.moe_expert_ffn_codes(cfg, one, one, one, offsets, w, one, one, wsf)
            L.moe_expert_ffn_gather(cfg, one, one, offsets, w, one, one, wsf)
        torch.cuda.synchronize()
        assert (host(dw) == 0).all() and (host(one) == 3).all()
    L.moe_quantize_int8(None, 0, 4, 16, 1, None, None)


@pytest.mark.parametrize("wgt,kw", [("int8", dict(softmax=True)), ("int8", dict(raw_gates=True)), ("fp8_e4m3", dict(softmax=True)),
                                    ("mxfp4", dict(softmax=True, raw_gates=True)), ("bf16", dict(softmax=True, raw_gates=True))])
def test_another_stream_and_given_affinities(wgt, kw):
    """A block on a side stream, and on its own affinities given back: the bits of the block on the current stream."""
    c = MID.with_(T=260, H=512, E=16, G=4, M=2, k=4, S=1, I=256, wgt=wgt)
    wts = make_weights(c)
    nw = f32_to_bf16_bits((1 + 0.2 * rng(252).standard_normal(c.H)).astype(np.float32))
    layer = MoeLayerGPU(c, wts, gather=wgt in ("int8", "fp8_e4m3"), norm=nw, **kw)
    x, res, bias = to_device(make_x(c)), _rows(c.T, c.H, "bf16", 4), dev_f32(wts.bias0)
    say(f"another stream, given affinities, {wgt} {kw}")
    want = layer.forward(x, bias, residual=res).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    layer.y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x, bias, residual=res)
    side.synchronize()
    assert _same(layer.y, want)
    layer.y.zero_()
    layer.forward(x, bias, residual=res, scores_in=True)
    torch.cuda.synchronize()
    assert _same(layer.y, want)


def test_two_graphs_over_one_layer():
    """Two captured blocks (two batch contents) share the layer's buffers and workspaces: replayed in turn, each gives its
    own batch's bits."""
    c = MID.with_(T=260, H=512, E=16, G=4, M=2, k=4, S=1, I=256, wgt="int8")
    wts = make_weights(c)
    nw = f32_to_bf16_bits(np.ones(c.H, np.float32))
    kw = dict(gather=True, norm=nw, softmax=True)
    layer, eager = MoeLayerGPU(c, wts, **kw), MoeLayerGPU(c, wts, **kw)
    bias = dev_f32(wts.bias0)
    xs = [to_device(make_x(c, i)) for i in range(2)]
    ns = [None, torch.tensor([200], dtype=torch.int32, device="cuda")]
    say("two graphs over one layer")
    graphs = [layer.capture(x, bias, n_tokens=n) for x, n in zip(xs, ns)]
    for turn in (0, 1, 1, 0, 1, 0, 0):
        xs[turn].copy_(to_device(make_x(c, 10 + turn)))
        want = eager.forward(xs[turn], bias, n_tokens=ns[turn]).clone()
        torch.cuda.synchronize()
        graphs[turn].replay()
        torch.cuda.synchronize()
        live = c.T if turn == 0 else 200
        assert _same(layer.y[:live], want[:live])


@pytest.mark.parametrize("phases", [(L.MOE_FFN_ALL,), (L.MOE_FFN_GATE_UP, L.MOE_FFN_DOWN)])
@pytest.mark.parametrize("wgt,S", [("fp8_e4m3", 0), ("fp8_e4m3", 2), ("int8", 0), ("int8", 2)])
def test_experts_on_codes_of_a_share(wgt, S, phases):
    """A share's padded batch given as codes, in one call or in phases, gives what its bf16 rows give; codes of dead tokens
    may be anything."""
    c = MID.with_(T=300, H=384, E=16, G=4, M=2, k=4, S=S, I=256, wgt=wgt)
    wts = make_weights(c)
    layer = MoeLayerGPU(c, wts, share=(3, 9), gather=True)
    x, bias = to_device(make_x(c)), dev_f32(wts.bias0)
    n = torch.tensor([211], dtype=torch.int32, device="cuda")
    say(f"codes of a share {wgt} S={S} {phases}")
    layer.forward(x, bias, n_tokens=n)
    torch.cuda.synchronize()
    m = int(host(layer.offsets)[-1])
    want = [layer.y_perm[:m].clone(), layer.y_shared[:211].clone() if S else None]
    if wgt == "int8":
        codes, scale = torch.empty((c.T, c.H), dtype=torch.int8, device="cuda"), torch.empty(c.T, device="cuda")
        L.moe_quantize_int8(x, 1, c.T, c.H, 1, codes, scale)
    else:
        codes = torch.empty((c.T, c.H), dtype=torch.uint8, device="cuda")
        scale = torch.empty((c.T, c.H // 128), device="cuda")
        L.moe_quantize_fp8(x, 1, c.T, c.H, 1, codes, scale)
    codes[211:], scale[211:] = 77, float("nan")
    layer.y_perm.fill_(5)
    for ph in phases:
        L.moe_expert_ffn_codes(layer.cfg_x, codes, scale, layer.perm, layer.offsets, layer.weights, layer.y_perm,
                               layer.y_shared, layer.ws_ffn, ph)
    torch.cuda.synchronize()
    assert _same(layer.y_perm[:m], want[0]) and (layer.y_perm[m:] == 5).all()
    assert not S or _same(layer.y_shared[:211], want[1])
