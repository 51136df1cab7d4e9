"""MXFP4 expert weights: the quantiser bit for bit against the oracle, the expert
FFN and the layer against the oracle's layer on the values that the codes stand
for.  Tolerances as in test_gpu_few.py: bounds from half a rounding step."""
import numpy as np
import pytest
import torch

import expert_ffn_layer_gb300 as moe
import oracle
import workloads as W
from moe_testlib import DeviceLayer, bf16_dev, host_f64, i32_dev
from oracle import mx
from test_gpu_few import BF16_HALF, DENSE, MID, TINY, assert_within, check_layer, swiglu_bound

pytestmark = pytest.mark.gpu

# H, I, I_shared multiples of 128; one to three pieces of 128 codes split unevenly over the warps
ODD = W.Workload("mx_odd", 3, 384, 6, 2, 640, 128, "softmax", 1.0, 1e-8, True, "none", 0.0, 9)
NOSH = W.Workload("mx_nosh", 6, 1152, 12, 3, 384, 384, "softmax", 1.0, 1e-8, False, "none", 0.0, 12)
WIDE = W.Workload("mx_wide", 5, 256, 256, 16, 128, 128, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 7)
HALF_FP16 = 2.0 ** -11
NAMES = ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class LazyValues:
    """Stacked weights whose expert e is quantised and dequantised by the oracle when first indexed."""

    def __init__(self, src):
        self.src, self.cache = src, {}

    def __getitem__(self, e):
        if int(e) not in self.cache:
            self.cache[int(e)] = mx.dequantize_mx(*mx.quantize_mx(oracle.widen_bf16(self.src[int(e)]), "e2m1"))
        return self.cache[int(e)]


def dequantised(inp):
    """The inputs with every expert weight replaced by the value its MXFP4 code stands for."""
    out = dict(inp)
    for n in NAMES[:3]:
        out[n] = LazyValues(inp[n])
    for n in NAMES[3:]:
        if inp.get(n) is not None:
            out[n] = mx.dequantize_mx(*mx.quantize_mx(oracle.widen_bf16(inp[n]), "e2m1"))
    return out


def experts_of(dl):
    return moe.quantize_mxfp4_experts(dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate, dl.ws_up, dl.ws_down)


def quantize_dev(w):
    src = bf16_dev(w)
    codes = torch.empty((*src.shape[:-1], src.shape[-1] // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((*src.shape[:-1], src.shape[-1] // 32), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4_rows(src, codes, scales)
    return src, codes, scales


def plain_codes(packed):
    """One code per byte, in order, of packed codes."""
    b = moe.pack_mxfp4(packed).cpu().numpy()
    return np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], -1)


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (37, 640), (129, 1408), (1024, 2048)])
def test_quantize_bit_exact(rows, cols):
    """Ordinary rows, and rows spread over bf16's range, with zero, negative-zero and subnormal blocks."""
    rng = np.random.default_rng(rows + cols)
    w = W.normal_bf16(2, 40, (rows, cols), 0.02)
    if rows >= 37:
        mag = 2.0 ** rng.uniform(-132, 127.9, size=(8, cols // 32, 1)) * 2.0 ** rng.uniform(-6, 0, size=(8, cols // 32, 32))
        v = (np.where(rng.random(mag.shape) < 0.5, -mag, mag)).astype(np.float32)
        w[:8] = (v.reshape(8, cols).view(np.uint32) >> 16).astype(np.uint16)
        w[8] = 0
        w[9, ::2] = 0x8000
        w[10, :32] = 0x0001          # the smallest subnormal
        # every midpoint between element values, at an exact scale
        pos = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
        mids = np.concatenate([(pos[1:] + pos[:-1]) / 2, [6.5, 7.0, 7.5], pos[1:]])
        row = np.zeros(32, dtype=np.float32)
        row[:len(mids)] = mids
        row[-1] = 4.0
        w[11, :32] = (row.view(np.uint32) >> 16).astype(np.uint16)
        w[12, :32] = ((-row).view(np.uint32) >> 16).astype(np.uint16)
    src, codes, scales = quantize_dev(w)
    q, e, _ = mx.quantize_mx(oracle.widen_bf16(w), "e2m1")
    assert np.array_equal(scales.cpu().numpy(), e)
    assert np.array_equal(plain_codes(codes), q)
    back = torch.empty_like(src)
    moe.moe_dequantize_mxfp4_rows(codes, scales, back)
    ref = mx.dequantize_mx(q, e, "e2m1")
    ref = np.where(np.abs(ref) > 3.3895e38, np.copysign(np.inf, ref), ref)  # 6 2^126 and above: past bf16
    got = host_f64(back)
    small = np.abs(ref) < 2.0 ** -126
    assert np.array_equal(got[~small], ref[~small])
    assert np.abs(got[small] - ref[small]).max(initial=0) <= 2.0 ** -134  # half of bf16's last subnormal step


def test_quantize_marks_blocks_that_are_not_finite():
    w = W.normal_bf16(2, 40, (4, 256), 0.02)
    w[1, 40] = 0x7F80   # +inf in block 1
    w[2, 200] = 0xFFC1  # NaN in block 6
    src, codes, scales = quantize_dev(w)
    e = scales.cpu().numpy()
    assert e[1, 1] == 255 and e[2, 6] == 255 and (e == 255).sum() == 2
    back = torch.empty_like(src)
    moe.moe_dequantize_mxfp4_rows(codes, scales, back)
    bad = torch.isnan(back).cpu().numpy()
    assert bad[1, 32:64].all() and bad[2, 192:224].all() and bad.sum() == 64


def test_pack_is_the_documented_layout():
    plain = torch.arange(2 * 128, dtype=torch.int32).reshape(2, 128) % 251
    packed = moe.pack_mxfp4(plain.to(torch.uint8))
    for r in range(2):
        for piece in range(2):
            for q in range(4):
                for t in range(4):
                    a, b = 64 * piece + 4 * (4 * t + q), 64 * piece + 4 * (4 * q + t)
                    assert torch.equal(packed[r, a:a + 4].int(), plain[r, b:b + 4])
    assert torch.equal(moe.pack_mxfp4(packed).int(), plain)


def layer(dl, ex, out=None, stream=None):
    out = torch.empty((dl.d.T, dl.d.H), dtype=torch.bfloat16, device="cuda") if out is None else out
    moe.moe_layer_forward_mxfp4(dl.d, dl.hidden, dl.router_w, dl.bias, ex, out, dl.ws, stream)
    return out


@pytest.mark.parametrize("w", [TINY, WIDE, ODD, DENSE, NOSH, MID], ids=lambda w: w.name)
@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 32])
def test_layer_mxfp4_few(w, T):
    w = w.with_(T=T)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    ex = experts_of(dl)
    got = host_f64(layer(dl, ex))
    assert moe.moe_ws_read_error(dl.ws) == 0
    check_layer(w, dequantised(inp), got, HALF_FP16, f"{w.name} T={T}")
    assert torch.equal(layer(dl, ex), layer(dl, ex)), "not reproducible"
    assert int(dl.ws[:4096].sum()) == 0


def ffn_case(w, inp, topk, seed=0):
    """Expert FFN on a given routing [T, k] against its bounds; returns nothing but asserts."""
    dl = DeviceLayer(w, inp)
    ex = experts_of(dl)
    counts, offsets = oracle.histogram_offsets(topk, w.E)
    perm, _ = oracle.permutation(topk, w.E)
    y = torch.full((w.T * w.top_k, w.H), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((w.T, w.H), 7.0, dtype=torch.bfloat16, device="cuda") if w.has_shared else None
    moe.moe_expert_ffn_mxfp4(dl.d, dl.hidden, i32_dev(perm), i32_dev(offsets), ex, y, z, dl.ws)
    assert moe.moe_ws_read_error(dl.ws) == 0
    deq = dequantised(inp)
    act_eps = HALF_FP16 if w.T <= 32 else BF16_HALF
    tok = np.asarray(perm) // w.top_k
    got = host_f64(y)
    for e in range(w.E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            ref, b = swiglu_bound(inp["hidden"][tok[lo:hi]], deq["w_gate"][e], deq["w_up"][e], deq["w_down"][e], act_eps)
            assert_within(got[lo:hi], ref, b + BF16_HALF * (np.abs(ref) + b), f"expert {e}")
    if z is not None:
        ref, b = swiglu_bound(inp["hidden"], deq["ws_gate"], deq["ws_up"], deq["ws_down"], act_eps)
        assert_within(host_f64(z), ref, b + BF16_HALF * (np.abs(ref) + b), "shared")
    assert int(dl.ws[:4096].sum()) == 0


@pytest.mark.parametrize("w", [TINY, WIDE, ODD, NOSH, MID], ids=lambda w: w.name)
@pytest.mark.parametrize("T", [1, 5, 8, 16, 27, 32])
def test_expert_ffn_mxfp4_few(w, T):
    w = w.with_(T=T)
    rng = np.random.default_rng(T)
    topk = np.stack([rng.permutation(w.E)[:w.top_k] for _ in range(T)]).astype(np.int32)
    ffn_case(w, W.layer_inputs(w), topk)


@pytest.mark.parametrize("w", [TINY, WIDE, ODD, NOSH, MID], ids=lambda w: w.name)
@pytest.mark.parametrize("T", [33, 64, 65, 128, 129, 300])
def test_expert_ffn_mxfp4_many(w, T):
    """Batches past 32 tokens: the expert kernel with converter warps."""
    w = w.with_(T=T)
    rng = np.random.default_rng(T)
    topk = np.stack([rng.permutation(w.E)[:w.top_k] for _ in range(T)]).astype(np.int32)
    ffn_case(w, W.layer_inputs(w), topk)


@pytest.mark.parametrize("T", [700, 1040])
def test_expert_ffn_mxfp4_skewed(T):
    """One expert holding every token (several chunks), idle experts."""
    w = MID.with_(T=T, top_k=2)
    topk = np.zeros((T, 2), dtype=np.int32)
    topk[:, 0] = 3
    topk[:, 1] = np.where(np.arange(T) < 512, 6, 1)
    ffn_case(w, W.layer_inputs(w), topk)


@pytest.mark.parametrize("w", [TINY, MID, NOSH], ids=lambda w: w.name)
@pytest.mark.parametrize("T", [33, 200])
def test_layer_mxfp4_many(w, T):
    w = w.with_(T=T)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    got = host_f64(layer(dl, experts_of(dl)))
    assert moe.moe_ws_read_error(dl.ws) == 0
    # the chain's router: 1e-5 of the logits' norm, from the split of the router weight
    check_layer(w, dequantised(inp), got, BF16_HALF, f"{w.name} T={T}", y_eps=BF16_HALF)


@pytest.mark.parametrize("T,E,k", [(256, 200, 8), (256, 22, 1), (128, 171, 16), (129, 171, 16)])
def test_expert_ffn_mxfp4_one_kernel_limits(T, E, k):
    """The largest batches of the one-kernel form (256 tokens, 2048 slots, 12 slots an expert), and one past it."""
    w = W.Workload("mx_lim", T, 128, E, k, 128, 128, "softmax", 1.0, 1e-8, True, "none", 0.0, 17)
    rng = np.random.default_rng(T + E)
    topk = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ffn_case(w, W.layer_inputs(w), topk)


@pytest.mark.parametrize("H,I,Is", [(16384, 128, 128), (128, 16384, 128), (2048, 128, 4096)])
def test_expert_ffn_mxfp4_extreme_widths(H, I, Is):
    w = W.Workload("mx_ext", 3, H, 4, 2, I, Is, "softmax", 1.0, 1e-8, True, "none", 0.0, 31)
    ffn_case(w, W.layer_inputs(w), np.array([[0, 3], [3, 1], [1, 0]], dtype=np.int32))


@pytest.mark.parametrize("T", [4, 64])
def test_mxfp4_scale_bytes_at_the_ends(T):
    """A scale byte of 255 makes the outputs that read its block non-finite and no others; 0 counts as
    zero.  T = 4 runs the one-kernel form, T = 64 (16 slots an expert) the converting kernel."""
    w = TINY.with_(T=T)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    ex = experts_of(dl)
    topk = np.tile(np.arange(4, dtype=np.int32), (T, 1))
    _, offsets = oracle.histogram_offsets(topk, w.E)
    perm, _ = oracle.permutation(topk, w.E)
    y = torch.empty((T * 4, w.H), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((T, w.H), dtype=torch.bfloat16, device="cuda")

    def run():
        moe.moe_expert_ffn_mxfp4(dl.d, dl.hidden, i32_dev(perm), i32_dev(offsets), ex, y, z, dl.ws)
        return y.clone(), z.clone()

    clean, clean_z = run()
    codes, scales = ex.t["down"]
    kept = scales.clone()
    scales[2, 77, 1] = 255
    scales[1, 50, :] = 0
    got, got_z = run()
    rows2 = slice(int(offsets[2]), int(offsets[3]))
    rows1 = slice(int(offsets[1]), int(offsets[2]))
    assert not torch.isfinite(got[rows2, 77]).any()
    assert (got[rows1, 50] == 0).all()
    got[rows2, 77] = clean[rows2, 77]
    got[rows1, 50] = clean[rows1, 50]
    assert torch.equal(got, clean) and torch.equal(got_z, clean_z)
    scales.copy_(kept)


def test_expert_ffn_mxfp4_repeated_expert():
    """A routing that names the same expert twice for a token, and one expert for all."""
    w = ODD.with_(T=9)
    ffn_case(w, W.layer_inputs(w), np.full((9, 2), 4, dtype=np.int32))


def test_expert_ffn_mxfp4_spread_inputs():
    """Tokens of very different sizes, rows with values far apart and a zero row: each row is
    scaled by its own power of two, so the bound holds relative to the row."""
    w = MID.with_(T=6)
    inp = dict(W.layer_inputs(w))
    x = oracle.widen_bf16(inp["hidden"]).astype(np.float32).copy()
    x[0] *= 2.0 ** 20
    x[1] *= 2.0 ** -20
    x[2, ::7] *= 2.0 ** 15
    x[3] = 0
    x[4, 5] = 1e6
    inp["hidden"] = (x.view(np.uint32) >> 16).astype(np.uint16)
    topk = np.tile(np.arange(4, dtype=np.int32), (6, 1))
    ffn_case(w, inp, topk)


def test_expert_ffn_mxfp4_bad_routing_is_recorded():
    """Offsets that do not end at S, and a slot out of range: flagged, nothing read out of range."""
    w = TINY.with_(T=4)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    ex = experts_of(dl)
    topk = np.tile(np.arange(4, dtype=np.int32), (4, 1))
    _, offsets = oracle.histogram_offsets(topk, w.E)
    perm, _ = oracle.permutation(topk, w.E)
    y = torch.zeros((16, w.H), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((4, w.H), dtype=torch.bfloat16, device="cuda")
    short = np.array(offsets)
    short[-1] = 15
    moe.moe_expert_ffn_mxfp4(dl.d, dl.hidden, i32_dev(perm), i32_dev(short), ex, y, z, dl.ws)
    assert moe.moe_ws_read_error(dl.ws, clear=True) == moe.DEVERR_OFFSETS
    assert (y == 0).all() and (z != 0).any()
    odd = np.array(perm)
    odd[3] = 99
    moe.moe_expert_ffn_mxfp4(dl.d, dl.hidden, i32_dev(odd), i32_dev(offsets), ex, y, z, dl.ws)
    assert moe.moe_ws_read_error(dl.ws, clear=True) == moe.DEVERR_INDEX


def test_layer_mxfp4_equals_its_stages():
    """The one-kernel layer and route, permute, expert FFN, combine: each within its bounds.
    (The stages store expert outputs in bf16: one more half step.)"""
    w = MID.with_(T=8)
    inp = W.layer_inputs(w)
    dl = DeviceLayer(w, inp)
    ex = experts_of(dl)
    idx, wts, _ = dl.route()
    _, offsets, perm, inv = dl.permute(idx)
    y = torch.empty((w.S, w.H), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((w.T, w.H), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_ffn_mxfp4(dl.d, dl.hidden, perm, offsets, ex, y, z, dl.ws)
    deq = dequantised(inp)
    check_layer(w, deq, host_f64(dl.combine(y, z, inv, wts)), HALF_FP16, "stages", y_eps=BF16_HALF)
    check_layer(w, deq, host_f64(layer(dl, ex)), HALF_FP16, "layer")


def test_layer_mxfp4_graph():
    w = TINY.with_(T=8)
    dl = DeviceLayer(w, W.layer_inputs(w))
    ex = experts_of(dl)
    ref = layer(dl, ex).clone()
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(dl, ex, out=out)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_mxfp4_refusals():
    w = TINY.with_(T=4)
    dl = DeviceLayer(w, W.layer_inputs(w))
    ex = experts_of(dl)
    out = torch.empty((4, w.H), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_layer_forward_mxfp4(dl.d, dl.hidden, dl.router_w, dl.bias, ex, out, dl.ws[:4096])
    with pytest.raises(ValueError):
        moe.moe_layer_forward_mxfp4(dl.d, dl.hidden, dl.router_w, dl.bias,
                                    moe.Mxfp4Experts(gate=ex.t["gate"], up=ex.t["up"]), out, dl.ws)
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4_rows(dl.hidden, torch.empty((4, 64), dtype=torch.uint8, device="cuda"),
                                    torch.empty((4, 8), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moe.pack_mxfp4(torch.zeros((2, 96), dtype=torch.uint8))
