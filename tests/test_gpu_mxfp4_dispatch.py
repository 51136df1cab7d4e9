"""MXFP4 expert FFN and layer on both sides of the rule that chooses their form, each with the bound of the form
that runs: the one-kernel form keeps fp16's 11 bits of an activation, the converting kernel bf16's 8."""
import numpy as np
import pytest
import torch

import expert_ffn_layer_gb300 as moe
import oracle
import workloads as W
from moe_testlib import DeviceLayer, host_f64, i32_dev
from test_gpu_few import BF16_HALF, MID, TINY, assert_within, check_layer, swiglu_bound
from test_gpu_mxfp4 import HALF_FP16, NOSH, ODD, WIDE, dequantised, experts_of, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def one_kernel(w):
    """include/moe.h: at most 32 tokens, or up to 256 tokens and 2048 slots of at most 12 slots an expert."""
    return w.T <= 32 or (w.T <= 256 and w.S <= 2048 and w.S <= 12 * w.E)


def random_topk(w, seed=0):
    rng = np.random.default_rng(seed + w.T)
    return np.stack([rng.permutation(w.E)[:w.top_k] for _ in range(w.T)]).astype(np.int32)


def check_ffn(w, topk):
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    _, offsets = oracle.histogram_offsets(topk, w.E)
    perm, _ = oracle.permutation(topk, w.E)
    y = torch.full((w.S, w.H), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((w.T, w.H), 7.0, dtype=torch.bfloat16, device="cuda") if w.has_shared else None
    moe.moe_expert_ffn_mxfp4(dl.d, dl.hidden, i32_dev(perm), i32_dev(offsets), experts_of(dl), y, z, dl.ws)
    assert moe.moe_ws_read_error(dl.ws) == 0
    deq, tok, got = dequantised(inp), np.asarray(perm) // w.top_k, host_f64(y)
    act_eps = HALF_FP16 if one_kernel(w) else BF16_HALF

    def check(got, x, *weights, what):
        ref, b = swiglu_bound(x, *weights, act_eps)
        assert_within(got, ref, b + BF16_HALF * (np.abs(ref) + b), what)

    for e in range(w.E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            check(got[lo:hi], inp["hidden"][tok[lo:hi]], deq["w_gate"][e], deq["w_up"][e], deq["w_down"][e],
                  what=f"expert {e}")
    if z is not None:
        check(host_f64(z), inp["hidden"], deq["ws_gate"], deq["ws_up"], deq["ws_down"], what="shared")
    assert int(dl.ws[:4096].sum()) == 0


@pytest.mark.parametrize("w,T", [(TINY, 33), (TINY, 48), (WIDE, 33), (WIDE, 128), (NOSH, 48), (MID, 33), (MID, 48),
                                 (MID.with_(top_k=1), 192)], ids=lambda v: getattr(v, "name", str(v)))
def test_one_kernel_ffn_past_32_tokens(w, T):
    """Up to 12 slots an expert."""
    w = w.with_(T=T)
    assert one_kernel(w)
    check_ffn(w, random_topk(w))


@pytest.mark.parametrize("T,E,k", [(256, 200, 8), (256, 22, 1), (128, 171, 16)])
def test_one_kernel_ffn_limits(T, E, k):
    w = W.Workload("mx_lim", T, 128, E, k, 128, 128, "softmax", 1.0, 1e-8, True, "none", 0.0, 17)
    assert one_kernel(w)
    check_ffn(w, random_topk(w, E))


@pytest.mark.parametrize("w,T", [(TINY, 49), (MID, 49), (MID.with_(top_k=1), 193), (ODD, 37)],
                         ids=lambda v: getattr(v, "name", str(v)))
def test_converting_ffn_just_past_the_rule(w, T):
    w = w.with_(T=T)
    assert not one_kernel(w)
    check_ffn(w, random_topk(w))


LONG = W.Workload("mx_long", 700, 384, 2, 1, 256, 256, "softmax", 1.0, 1e-8, True, "none", 0.0, 23)


@pytest.mark.parametrize("w", [LONG, LONG.with_(T=513), LONG.with_(name="mx_long3", T=500, E=3, top_k=2, I=640, I_shared=128),
                               LONG.with_(name="mx_long1", T=300, E=1, has_shared=False)],
                         ids=lambda w: f"{w.name}-{w.T}")
@pytest.mark.parametrize("uneven", [False, True])
def test_converting_ffn_past_256_slots_an_expert(w, uneven):
    """Experts of several chunks each, taken expert by expert; uneven: the first expert has nearly all."""
    assert w.S > 256 * w.E
    topk = random_topk(w)
    if uneven:
        topk = np.tile(np.arange(w.top_k, dtype=np.int32), (w.T, 1))
        if w.E > 1:
            topk[::97, 0] = w.E - 1
    check_ffn(w, topk)


@pytest.mark.parametrize("w", [LONG, LONG.with_(name="mx_long3", T=500, E=3, top_k=2, I=640, I_shared=128)],
                         ids=lambda w: w.name)
def test_layer_past_256_slots_an_expert(w):
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    got = host_f64(layer(dl, experts_of(dl)))
    assert moe.moe_ws_read_error(dl.ws) == 0
    check_layer(w, dequantised(inp), got, BF16_HALF, w.name, y_eps=BF16_HALF)


@pytest.mark.parametrize("w,T", [(TINY, 33), (MID, 48)], ids=lambda v: getattr(v, "name", str(v)))
def test_layer_with_the_one_kernel_ffn(w, T):
    """Past 32 tokens the layer is the chain of kernels, with the one-kernel FFN as its stage."""
    w = w.with_(T=T)
    assert one_kernel(w)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    got = host_f64(layer(dl, experts_of(dl)))
    assert moe.moe_ws_read_error(dl.ws) == 0
    check_layer(w, dequantised(inp), got, HALF_FP16, w.name, y_eps=BF16_HALF)
