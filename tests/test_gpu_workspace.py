"""One workspace, made for the largest batch, under smaller batches of every entry: accepted, the same bits as
with a workspace of the batch's own, and nothing written behind its end."""
import pytest
import torch

import expert_ffn_layer_gb300 as moe
import workloads as W
from moe_testlib import DeviceLayer

pytestmark = pytest.mark.gpu

MANY = W.Workload("ws_many", 8, 512, 64, 2, 256, 256, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 3)
WIDE_H = W.Workload("ws_wide_h", 8, 4096, 22, 1, 128, 128, "softmax", 1.0, 1e-8, True, "none", 0.0, 4)
FEW_E = W.Workload("ws_few_e", 8, 512, 4, 4, 512, 512, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 5)
GUARD = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def entries(dl):
    """name -> call(ws), which returns the outputs of one entry (or one chain of stages)."""
    d, dev = dl.d, dict(device="cuda")
    fp8 = moe.quantize_fp8_experts(dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate, dl.ws_up, dl.ws_down)
    mx = moe.quantize_mxfp4_experts(dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate, dl.ws_up, dl.ws_down)
    gu = torch.cat([dl.w_gate, dl.w_up], dim=1).contiguous()
    sgu = torch.cat([dl.ws_gate, dl.ws_up], dim=0).contiguous()
    rest = (dl.hidden, dl.router_w, dl.bias)
    bf = (dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate, dl.ws_up, dl.ws_down)

    def out(rows=d.T):
        return torch.empty((rows, d.H), dtype=torch.bfloat16, **dev)

    def layer(fn, *w):
        def call(ws):
            o = out()
            fn(d, *rest, *w, o, ws)
            return (o,)
        return call

    def stages(ws):
        S = d.T * d.top_k
        idx, wt = torch.empty((d.T, d.top_k), dtype=torch.int32, **dev), torch.empty((d.T, d.top_k), **dev)
        counts, offsets = torch.empty(d.E, dtype=torch.int32, **dev), torch.empty(d.E + 1, dtype=torch.int32, **dev)
        perm, inv = torch.empty(S, dtype=torch.int32, **dev), torch.empty(S, dtype=torch.int32, **dev)
        moe.moe_route(d, *rest, idx, wt, ws)
        moe.moe_permute(d, idx, counts, offsets, perm, inv, ws)
        got = [idx, wt, counts, offsets, perm, inv]
        for fn, w in ((moe.moe_expert_ffn, bf), (moe.moe_expert_ffn_fp8, (fp8,)), (moe.moe_expert_ffn_w8a8, (fp8,)),
                      (moe.moe_expert_ffn_mxfp4, (mx,))):
            y, z = out(S), out()
            fn(d, dl.hidden, perm, offsets, *w, y, z, ws)
            got += [y, z]
        y, z, o = out(S), out(), out()
        moe.moe_expert_gate_up(d, dl.hidden, perm, offsets, dl.w_gate, dl.w_up, dl.ws_gate, dl.ws_up, ws)
        moe.moe_expert_down(d, offsets, dl.w_down, dl.ws_down, y, z, ws)
        moe.moe_fused_moe(d, dl.hidden, idx, wt, gu, dl.w_down, sgu, dl.ws_down, o, ws)
        return got + [y, z, o]

    calls = {"stages": stages, "layer": layer(moe.moe_layer_forward, *bf), "fp8": layer(moe.moe_layer_forward_fp8, fp8),
             "w8a8": layer(moe.moe_layer_forward_w8a8, fp8), "mxfp4": layer(moe.moe_layer_forward_mxfp4, mx)}
    if d.T <= 32:
        calls["few"] = layer(moe.moe_layer_forward_few, *bf)
    return calls


@pytest.mark.parametrize("w", [MANY, WIDE_H, FEW_E], ids=lambda w: w.name)
@pytest.mark.parametrize("made_for,T", [(33, 32), (100, 8), (257, 256), (257, 33), (320, 200), (1025, 1024)])
def test_a_larger_batchs_workspace(w, made_for, T):
    dl = DeviceLayer(w.with_(T=T), W.layer_inputs(w.with_(T=T)))
    n = moe.moe_workspace_bytes(moe.dims(made_for, w.H, w.E, w.I, w.top_k, w.I_shared, w.score_mode, w.route_scale,
                                         w.renorm_eps))
    buf = torch.zeros(n + GUARD, dtype=torch.uint8, device="cuda")
    buf[n:] = 0xA5
    for name, call in entries(dl).items():
        ref = call(moe.alloc_workspace(dl.d))
        got = call(buf[:n])
        for a, b in zip(got, ref):
            assert torch.equal(a, b), name
    assert moe.moe_ws_read_error(buf[:n]) == 0
    assert int(buf[:4096].sum()) == 0
    assert bool((buf[n:] == 0xA5).all())


@pytest.mark.parametrize("w", [MANY, WIDE_H, FEW_E], ids=lambda w: w.name)
@pytest.mark.parametrize("T", [1, 32, 33, 256, 257])
def test_nothing_behind_the_workspace(w, T):
    """A workspace of exactly the batch's size."""
    dl = DeviceLayer(w.with_(T=T), W.layer_inputs(w.with_(T=T)))
    n = moe.moe_workspace_bytes(dl.d)
    buf = torch.zeros(n + GUARD, dtype=torch.uint8, device="cuda")
    buf[n:] = 0xA5
    for call in entries(dl).values():
        call(buf[:n])
    assert moe.moe_ws_read_error(buf[:n]) == 0
    assert bool((buf[n:] == 0xA5).all())
