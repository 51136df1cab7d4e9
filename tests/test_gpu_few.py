"""The MoE layer for few tokens in one kernel (moe_layer_forward_few) against the
fp64 oracle, element by element.

Tolerances are bounds, not measurements.  A sum of n products in fp32 -- in any
order, each addition truncated at worst -- is off by at most n 2^-23 times the sum
of the products' magnitudes; SiLU's slope is at most 1.1 and its own error 1e-5
relative; a value held in bf16 is off by half a step, 2^-8 relative.  Every output
element gets the bound that follows from those for its own inputs."""
import numpy as np
import pytest
import torch

import expert_ffn_layer_gb300 as moe
import oracle
import workloads as W
from moe_testlib import DeviceLayer, check_selection, host_f64

pytestmark = pytest.mark.gpu

WIDE = W.Workload("few_wide", 5, 256, 256, 16, 64, 64, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 7)
ODD = W.Workload("few_odd", 3, 192, 6, 2, 320, 64, "softmax", 1.0, 1e-8, True, "none", 0.0, 9)
DENSE = W.Workload("few_dense", 4, 256, 1, 1, 128, 128, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 8)
NOSH = W.Workload("few_nosh", 6, 1088, 12, 3, 704, 704, "softmax", 1.0, 1e-8, False, "none", 0.0, 12)
MID = W.Workload("few_mid", 8, 2048, 16, 4, 512, 256, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 13)
TINY = W.WORKLOADS["tiny"].with_(name="few_tiny")

FP32_STEP, BF16_HALF = 2.0 ** -23, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def swiglu_bound(x, wg, wu, wd, act_eps):
    """SwiGLU outputs in float64 and how far a kernel with fp32 sums, whose
    activation keeps a relative error of act_eps, may be from them."""
    x, wg, wu, wd = (np.asarray(oracle.widen_bf16(a), dtype=np.float64) for a in (x, wg, wu, wd))
    g, u = x @ wg.T, x @ wu.T
    c = (x.shape[-1] + 64) * FP32_STEP
    dg, du = c * (np.abs(x) @ np.abs(wg).T), c * (np.abs(x) @ np.abs(wu).T)
    s = oracle.silu(g)
    a = s * u
    da = 1.1 * np.abs(u) * dg + np.abs(s) * du + 1.1 * dg * du + (1e-5 + act_eps) * np.abs(a)
    y = a @ wd.T
    wd = np.abs(wd).T
    return y, da @ wd + (a.shape[-1] + 64) * FP32_STEP * ((np.abs(a) + da) @ wd)


def layer_bound(w, inp, idx, act_eps, y_eps=0.0):
    """The layer's output for the selection idx [T, k] and the bound of each element."""
    x = oracle.widen_bf16(inp["hidden"]).astype(np.float64)
    logits = oracle.router_logits(inp["hidden"], inp["router_w"])
    dl = (w.H + 64) * FP32_STEP * (np.abs(x) @ np.abs(inp["router_w"].astype(np.float64)).T).max(1)
    route = oracle.route_sigmoid(logits, inp["bias"], w.top_k, w.route_scale) if w.score_mode == "sigmoid" else \
        oracle.route_softmax(logits, w.top_k, w.renorm_eps)
    wt = oracle.routing_weights_for(route["scores"], idx, w.score_mode, w.route_scale, w.renorm_eps)
    out, bound = np.zeros((w.T, w.H)), np.zeros((w.T, w.H))
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        y, dy = swiglu_bound(inp["hidden"][t], inp["w_gate"][e], inp["w_up"][e], inp["w_down"][e], act_eps)
        dy = dy + y_eps * np.abs(y)
        c = wt[t, j][:, None]
        out[t] += c * y
        # a weight s / sum(s) moves by at most twice the logits' error, relative
        bound[t] += c * (dy + (2 * dl[t][:, None] + 4e-6 + (w.top_k + 2) * FP32_STEP) * (np.abs(y) + dy))
    if w.has_shared:
        z, dz = swiglu_bound(inp["hidden"], inp["ws_gate"], inp["ws_up"], inp["ws_down"], act_eps)
        out += z
        bound += dz + (y_eps + FP32_STEP) * np.abs(z)
    return out, bound + BF16_HALF * (np.abs(out) + bound)


def assert_within(got, ref, bound, what=""):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {got.size} past the bound, worst {over.max():.3e}"


def check_layer(w, inp, got, act_eps, what="", y_eps=0.0):
    """`got` against the oracle; a row whose keys nearly tie may use any valid selection."""
    ref = oracle.layer_forward(inp["hidden"], inp["router_w"], inp["bias"], inp["w_gate"], inp["w_up"],
                               inp["w_down"], inp["ws_gate"], inp["ws_up"], inp["ws_down"], top_k=w.top_k,
                               score_mode=w.score_mode, route_scale=w.route_scale, renorm_eps=w.renorm_eps)
    sure = ref["margin"] >= 1e-5  # the seeds of this file have no nearer keys but by chance
    assert sure.mean() >= 0.9
    out, bound = layer_bound(w, inp, ref["idx"], act_eps, y_eps)
    assert_within(got[sure], out[sure], bound[sure], what)


def few(dl, stream=None, out=None, ws=None):
    out = torch.empty((dl.d.T, dl.d.H), dtype=torch.bfloat16, device="cuda") if out is None else out
    moe.moe_layer_forward_few(dl.d, dl.hidden, dl.router_w, dl.bias, dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate,
                              dl.ws_up, dl.ws_down, out, dl.ws if ws is None else ws, stream)
    return out


@pytest.mark.parametrize("w", [TINY, WIDE, ODD, DENSE, NOSH, MID], ids=lambda w: w.name)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32])
def test_few_parity(w, T):
    w = w.with_(T=T)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    got = host_f64(few(dl))
    assert moe.moe_ws_read_error(dl.ws) == 0
    check_layer(w, inp, got, 2.0 ** -16, f"{w.name} T={T}")
    assert torch.equal(few(dl), few(dl)), "not reproducible"
    assert int(dl.ws[:4096].sum()) == 0, "the workspace header is not left zero"


def test_few_decode_widths():
    """The Hy3 layer's widths (with 24 experts), a few tokens."""
    w = W.WORKLOADS["decode"].with_(name="few_hy3", E=24, T=5)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    check_layer(w, inp, host_f64(few(dl)), 2.0 ** -16, "hy3 widths")


@pytest.mark.parametrize("H,I,Is", [(16384, 64, 128), (64, 16384, 64), (4096, 64, 4096)])
def test_few_extreme_widths(H, I, Is):
    """The widest rows beside the narrowest, and a shared expert far wider than the routed ones."""
    w = W.Workload("few_ext", 3, H, 4, 2, I, Is, "softmax", 1.0, 1e-8, True, "none", 0.0, 31)
    inp = W.layer_inputs(w)
    check_layer(w, inp, host_f64(few(DeviceLayer(w, inp))), 2.0 ** -16, f"H={H} I={I} Is={Is}")


@pytest.mark.parametrize("T", [8, 13, 32])
def test_few_all_tokens_on_the_same_experts(T):
    """A bias that sends every token to the same experts: T tokens in each, the others idle."""
    w = MID.with_(T=T)
    inp = dict(W.layer_inputs(w))
    bias = np.full(w.E, -4.0, dtype=np.float32)
    bias[[1, 5, 6, 15]] = 4.0
    inp["bias"] = bias
    dl = DeviceLayer(w, inp)
    check_layer(w, inp, host_f64(few(dl)), 2.0 ** -16)


def test_few_equal_keys_take_the_lower_expert():
    """A zero router: every logit is 0, so the top-k is experts 0 .. k - 1, equally weighted."""
    w = ODD.with_(T=3)
    inp = dict(W.layer_inputs(w))
    inp["router_w"] = np.zeros_like(inp["router_w"])
    got = host_f64(few(DeviceLayer(w, inp)))
    out, bound = layer_bound(w, inp, np.tile(np.arange(w.top_k, dtype=np.int32), (w.T, 1)), 2.0 ** -16)
    assert_within(got, out, bound)


def test_few_rows_do_not_mix():
    """A row of NaN, one of infinities and one of zeros leave the other rows within their own
    bounds.  (Not their bits: how K is split over the warps depends on how many experts are active,
    and with it the order of the fp32 sums, which the bounds cover.)"""
    w = MID.with_(T=11)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    dl.hidden[3] = float("nan")
    dl.hidden[7] = float("inf")
    dl.hidden[9] = 0
    got = few(dl)
    keep = [t for t in range(11) if t not in (3, 7, 9)]
    part = w.with_(T=len(keep))
    check_layer(part, {**inp, "hidden": inp["hidden"][keep]}, host_f64(got)[keep], 2.0 ** -16)
    assert not torch.isfinite(got[3]).any()
    assert not torch.isfinite(got[7]).all()
    assert (got[9] == 0).all()


def test_few_against_the_chain():
    """The chain of kernels on the same inputs: both within their bounds of the same layer.
    (The chain stores activations and expert outputs in bf16: two more half steps.)"""
    w = MID.with_(T=8)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    check_layer(w, inp, host_f64(dl.forward()), BF16_HALF, "chain", y_eps=BF16_HALF)
    check_layer(w, inp, host_f64(few(dl)), 2.0 ** -16, "few")


def test_few_then_chain_share_a_workspace():
    """The two forms alternate on one workspace, on a side stream, with the bits each has alone."""
    w = MID.with_(T=8)
    dl = DeviceLayer(w, W.layer_inputs(w))
    a, b = few(dl).clone(), dl.forward().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            x, y = few(dl), dl.forward()
    side.synchronize()
    assert torch.equal(x, a) and torch.equal(y, b)


def test_few_two_graphs_share_a_workspace():
    """Two captured graphs (other inputs, the same workspace) replayed in turn."""
    w = MID.with_(T=8)
    dl = DeviceLayer(w, W.layer_inputs(w))
    dl2 = DeviceLayer(w, W.layer_inputs(w.with_(seed=99)))
    ref, ref2 = few(dl).clone(), few(dl2).clone()
    outs, graphs = [], []
    for x in (dl, dl2):
        out = torch.zeros_like(ref)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            few(x, out=out, ws=dl.ws)
        outs.append(out)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref2)


def test_few_two_calls_at_once():
    """Calls on two streams with a workspace each: both need every SM, and take turns."""
    w = MID.with_(T=4)
    dl = DeviceLayer(w, W.layer_inputs(w))
    ref = few(dl).clone()
    ws2 = moe.alloc_workspace(dl.d)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(ref) for _ in range(80)]
    torch.cuda.synchronize()  # the zeros are written on the default stream
    for i in range(0, len(outs), 2):
        few(dl, stream=s1, out=outs[i])
        few(dl, stream=s2, out=outs[i + 1], ws=ws2)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_few_refusals_and_empty_batch():
    w = TINY.with_(T=4)
    dl = DeviceLayer(w, W.layer_inputs(w))
    d33 = moe.dims(33, w.H, w.E, w.I, w.top_k, w.I_shared)
    x, o = (torch.zeros((33, w.H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rest = (dl.router_w, dl.bias, dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate, dl.ws_up, dl.ws_down)
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        moe.moe_layer_forward_few(d33, x, *rest, o, moe.alloc_workspace(d33))
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_layer_forward_few(dl.d, dl.hidden, *rest, o[:4], dl.ws[:4096])
    with pytest.raises(ValueError):
        moe.moe_layer_forward_few(dl.d, dl.hidden[:3], *rest, o[:4], dl.ws)
    d0 = moe.dims(0, w.H, w.E, w.I, w.top_k, w.I_shared)
    moe.moe_layer_forward_few(d0, x[:0], *rest, o[:0], moe.alloc_workspace(d0))


def test_few_selection_matches_the_router():
    """The same experts as moe_route on ordinary inputs (through equal outputs with one expert
    per token whose output alone is non-zero)."""
    w = W.Workload("few_sel", 16, 256, 64, 1, 64, 64, "softmax", 1.0, 1e-8, False, "none", 0.0, 21)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    idx, _, _ = dl.route()
    ref = oracle.layer_forward(inp["hidden"], inp["router_w"], inp["bias"], inp["w_gate"], inp["w_up"],
                               inp["w_down"], None, None, None, top_k=1, score_mode="softmax", route_scale=1.0,
                               renorm_eps=1e-8)
    check_selection(idx.cpu().numpy(), ref, 1)
    check_layer(w, inp, host_f64(few(dl)), 2.0 ** -16)


def test_few_without_a_bias_equals_a_zero_one():
    w = MID.with_(T=5)
    dl = DeviceLayer(w, W.layer_inputs(w))
    dl.bias.zero_()
    ref = few(dl).clone()
    dl.bias = None
    assert torch.equal(few(dl), ref)


def test_few_in_place():
    """The output over the hidden state: every row is read before any is written."""
    w = MID.with_(T=7)
    dl = DeviceLayer(w, W.layer_inputs(w))
    ref = few(dl).clone()
    few(dl, out=dl.hidden)
    assert torch.equal(dl.hidden, ref)
