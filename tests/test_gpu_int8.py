"""GPU parity of the 8-bit integer experts: the row quantiser code for code, the
expert FFN and the layer against a float64 reference of the same definition.

Tolerance of outputs: the layer's (relative L2 5e-3, 3e-2 absolute).  A bf16 value
is off by at most 2^-8 of itself, in the mean of a binade 2^-8 / sqrt(3) or less:
2.3e-3.  The kernel's activations are within 9e-6 of the reference's before their
rounding to bf16, so about one in 2^8 * 9e-6 = 1/400 of them rounds to the neighbour,
which moves a code by one in at most half of the cases; a code is 1/127 of the row's
largest of I of them, so y moves by less than 1e-3 of itself."""
import numpy as np
import pytest
import torch

import expert_ffn_layer_gb300 as moe
import int8_testlib as ref8
import workloads as W
from moe_testlib import DeviceLayer, assert_layer_close, bf16_dev, check_selection, host_f64, i32_dev, valid_alternatives
from test_gpu_parity import MID, MID_SOFTMAX, NOSHARED, ODD_H, WIDE, inputs_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def quantized(src):
    codes = torch.empty(src.shape, dtype=torch.int8, device="cuda")
    scales = torch.empty(src.shape[:-1], dtype=torch.float32, device="cuda")
    moe.moe_quantize_int8_rows(src, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def values(codes, scales):
    dst = torch.empty(codes.shape, dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_int8_rows(codes, scales, dst)
    torch.cuda.synchronize()
    return dst


def bf16_of(x):
    """A device matrix of values that bf16 holds exactly."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float64)).bfloat16()
    assert torch.equal(t.double(), torch.from_numpy(np.asarray(x, np.float64)))
    return t.cuda()


@pytest.mark.parametrize("shift", [0, 90, -126])
def test_quantizer_every_ratio(shift):
    """Every pair of 8-bit significands a / b at every power of two that matters, signs both: the code is the
    integer nearest to 127 a 2^-k / b, ties to even, by integer arithmetic.  Rows of ordinary, huge and tiny
    (subnormal) magnitudes."""
    a = np.arange(128, 256)
    rows, want = [], []
    for b in range(128, 256):
        vals, codes = [b], [127]
        for k in range(10):
            for x in a[(a <= b << k)]:
                if shift < -100 and x % (1 << k):  # below the normal range only multiples of 2^-133 exist
                    continue
                num, den = 127 * int(x), int(b) << k
                n, rem = divmod(num, den)
                n += 2 * rem > den or (2 * rem == den and n % 2 == 1)
                vals.append(x * 2.0 ** -k)
                codes.append(n)
        rows.append(vals)
        want.append(codes)
    wide = (max(map(len, rows)) + 7) // 8 * 8
    x, q = np.zeros((len(rows), wide)), np.zeros((len(rows), wide), np.int64)
    for i, (v, c) in enumerate(zip(rows, want)):
        x[i, :len(v)], q[i, :len(c)] = v, c
    x[:, 1::2] *= -1
    q[:, 1::2] *= -1
    x *= 2.0 ** (shift - 7)
    codes, scales = quantized(bf16_of(x))
    assert np.array_equal(codes.cpu().numpy(), q)
    top = np.abs(x).max(-1).astype(np.float32)
    assert np.array_equal(scales.cpu().numpy(), top / np.float32(127))


@pytest.mark.parametrize("shape", [(1, 8), (3, 24), (37, 520), (7, 2048), (3, 2056), (1300, 4096), (5, 16384), (3, 20008), (2, 3, 64)],
                         ids=str)
def test_quantizer_shapes_and_values(shape):
    src = bf16_dev(W.normal_bf16(2, 51, shape, 0.02))
    codes, scales = quantized(src)
    q, s = ref8.quantize(host_f64(src))
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(scales.cpu().numpy().astype(np.float64), s)
    want = torch.from_numpy((q * s[..., None]).astype(np.float32)).bfloat16()  # one rounding to fp32, one to bf16
    assert torch.equal(values(codes, scales).cpu(), want)


def test_quantizer_special_rows():
    x = torch.zeros((8, 64), dtype=torch.bfloat16)
    x[1] = -0.0
    x[2, 5] = 2.0 ** -133                    # the smallest bf16
    x[3, 7] = torch.finfo(torch.bfloat16).max
    x[3, 9] = -torch.finfo(torch.bfloat16).max
    x[4, 0], x[5, 63], x[6, 1], x[6, 2] = float("inf"), float("nan"), float("-inf"), float("nan")
    x[7] = 3.0
    codes, scales = (t.cpu() for t in quantized(x.cuda()))
    assert not codes[:2].any() and scales[:2].tolist() == [1.0, 1.0]
    assert codes[2, 5] == 127 and codes[2].abs().sum() == 127
    assert codes[3, 7] == 127 and codes[3, 9] == -127 and torch.isfinite(scales[3])
    assert torch.isnan(scales[4:7]).all()
    assert (codes[7] == 127).all()
    assert torch.isnan(values(codes.cuda(), scales.cuda())[4:7]).all()


def test_every_code_back():
    """Codes of a checkpoint may use all of -128 .. 127."""
    codes = torch.arange(-128, 128, dtype=torch.int8, device="cuda").repeat(3, 1)
    scales = torch.tensor([1.0, 0.3, 2.0 ** -120], device="cuda")
    want = (codes.double() * scales.double()[:, None]).float().bfloat16()
    assert torch.equal(values(codes, scales), want)


def test_codes_of_minus_128_in_the_products():
    """Weights whose codes are all -128 or 127, as other quantisers make them."""
    w = W.Workload("codes", 20, 128, 2, 1, 64, 64, "sigmoid", 2.826, 0.0, False, "normal", 0.1, 16)
    inp = W.layer_inputs(w)
    rng = np.random.default_rng(3)
    pair = lambda *s: (np.where(rng.random(s) < 0.5, -128, 127).astype(np.int8), np.full(s[:-1], 2e-4, np.float32))  # noqa: E731
    q = {"w_gate": pair(2, 64, 128), "w_up": pair(2, 64, 128), "w_down": pair(2, 128, 64)}
    r = ref8.layer(w, inp, {n: [(c[e], s[e].astype(np.float64)) for e in range(2)] for n, (c, s) in q.items()})
    dl = DeviceLayer(w, inp)
    ex = moe.Int8Experts(**{n[2:]: (torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()) for n, (c, s) in q.items()})
    y = torch.empty((w.S, w.H), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_ffn_int8(dl.d, dl.hidden, i32_dev(r["perm"]), i32_dev(r["offsets"]), ex, y, None, dl.ws)
    torch.cuda.synchronize()
    assert_layer_close(host_f64(y), r["y_sorted"], "y_sorted")


def dev_experts(dl):
    return moe.quantize_int8_experts(dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate, dl.ws_up, dl.ws_down)


_cache = {}


def weights_of(w, inp):
    if w.name not in _cache:
        _cache.clear()
        _cache[w.name] = ref8.quantize_weights(inp)
    return _cache[w.name]


def ffn(dl, w, perm, offsets):
    y = torch.full((w.S, w.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    z = torch.full((w.T, w.H), float("nan"), dtype=torch.bfloat16, device="cuda") if w.has_shared else None
    moe.moe_expert_ffn_int8(dl.d, dl.hidden, perm, offsets, dev_experts(dl), y, z, dl.ws)
    torch.cuda.synchronize()
    assert moe.moe_ws_read_error(dl.ws) == 0
    return y, z


# widths that are odd multiples of 64 (a ragged row block, a last group of 32-column maxima past the row) on
# every token tile, a shared expert of another width, one expert, one token
ODD_I = W.Workload("odd_i", 300, 320, 8, 2, 192, 448, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 12)
# tiles of 128 and of 240 tokens with I past 256 columns (ragged column blocks in the quantisation tiles), and
# 64-token tiles with several chunks an expert
MANY = W.Workload("many", 600, 192, 8, 1, 576, 320, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 15)
LONG_I = W.Workload("long_i", 260, 128, 3, 1, 1600, 64, "sigmoid", 2.826, 0.0, True, "normal", 0.1, 13)
SHAPES = [W.WORKLOADS["tiny"], MID, MID_SOFTMAX, WIDE, ODD_H, NOSHARED, ODD_I, LONG_I,
          MANY, MANY.with_(name="many_800", T=800), MANY.with_(name="many_360", T=360, E=16),
          *(ODD_I.with_(name=f"odd_i_{T}", T=T) for T in (1, 17, 33, 65, 129)), W.WORKLOADS["decode"]]


@pytest.mark.parametrize("w", SHAPES, ids=lambda w: w.name)
def test_expert_ffn(w):
    inp = inputs_of(w)
    q = weights_of(w, inp)
    r = ref8.layer(w, inp, q)
    dl = DeviceLayer(w, inp)
    y, z = ffn(dl, w, i32_dev(r["perm"]), i32_dev(r["offsets"]))
    assert_layer_close(host_f64(y), r["y_sorted"], f"{w.name} y_sorted")
    if w.has_shared:
        assert_layer_close(host_f64(z), r["z"], f"{w.name} y_shared")


@pytest.mark.parametrize("T", [700, 1040])
def test_expert_ffn_skewed(T):
    """One expert holding every token (several 240-token chunks), empty experts, a ragged last chunk."""
    w = MID.with_(name=f"mid_int8_{T}", T=T)
    inp = W.layer_inputs(w)
    topk = np.zeros((w.T, 2), dtype=np.int32)
    topk[:, 0] = 3
    topk[:, 1] = np.where(np.arange(w.T) < 512, 6, 1)
    r = ref8.layer(w, inp, ref8.quantize_weights(inp), topk_idx=topk)
    y, z = ffn(DeviceLayer(w, inp), w, i32_dev(r["perm"]), i32_dev(r["offsets"]))
    assert_layer_close(host_f64(y), r["y_sorted"], "y_sorted")
    assert_layer_close(host_f64(z), r["z"], "y_shared")


def test_sums_past_24_bits():
    """H = 16384 with every code +-127 and few signs to cancel: sums of code products up to 2.6e8, which fp32 rounds."""
    w = W.Workload("wide_sum", 20, 16384, 1, 1, 64, 64, "sigmoid", 2.826, 0.0, False, "normal", 0.1, 14)
    rng = np.random.default_rng(5)
    sign = np.where(rng.random((w.T, w.H)) < 0.9, 1.0, -1.0)
    inp = W.layer_inputs(w)
    bits = lambda x: (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731  (exact: powers of two)
    inp["hidden"] = bits(sign * 2.0 ** -6)
    for n, share in (("w_gate", 0.5), ("w_up", 0.8)):
        inp[n] = bits(np.where(rng.random((1, w.I, w.H)) < share, 1.0, -1.0) * 2.0 ** -9)
    r = ref8.layer(w, inp, ref8.quantize_weights(inp), topk_idx=np.zeros((w.T, 1), np.int32))
    y, _ = ffn(DeviceLayer(w, inp), w, i32_dev(r["perm"]), i32_dev(r["offsets"]))
    got = host_f64(y)
    # fp32 sums round by at most 2^-24 a step over 1024 steps of 16 products: 6e-5 of the sum of magnitudes, far
    # below the bf16 rounding of the result; the bound is relative, as y is not of order one here
    assert np.linalg.norm(got - r["y_sorted"]) <= 5e-3 * np.linalg.norm(r["y_sorted"])


@pytest.mark.parametrize("w", [W.WORKLOADS["tiny"], MID, MID_SOFTMAX, NOSHARED, ODD_I, W.WORKLOADS["decode"]],
                         ids=lambda w: w.name)
def test_layer(w):
    """moe_layer_forward_int8 against the reference (near-tie rows for the selection the GPU made); the same bits
    when it is called again, and when it is captured into a graph and replayed."""
    inp = inputs_of(w)
    q = weights_of(w, inp)
    dl = DeviceLayer(w, inp)
    experts = dev_experts(dl)
    outs = [torch.empty((w.T, w.H), dtype=torch.bfloat16, device="cuda") for _ in range(3)]

    def call(o):
        moe.moe_layer_forward_int8(dl.d, dl.hidden, dl.router_w, dl.bias, experts, o, dl.ws)

    call(outs[0])
    idx, _, _ = dl.route()
    call(outs[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[2])
    outs[2].zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    gi = idx.cpu().numpy()
    r = ref8.layer(w, inp, q)
    _, ties = check_selection(gi, r, w.top_k)
    want = r["out"].copy()
    for t in ties:
        pick = sorted(gi[t].tolist())
        assert pick in valid_alternatives(r, t, w.top_k)
        want[t] = ref8.layer(w, inp, q, topk_idx=np.array([pick], np.int32), rows=slice(t, t + 1))["out"][0]
    assert_layer_close(host_f64(outs[0]), want, f"{w.name} layer")
    for o in outs[1:]:
        assert torch.equal(outs[0].view(torch.int16), o.view(torch.int16))
    assert moe.moe_ws_read_error(dl.ws) == 0


def test_non_finite_tokens_and_weights_stay_in_their_rows():
    """A token with an infinity or NaN makes its own outputs NaN and no other's; so does a weight row with one, for
    the outputs that read it."""
    w = MID
    inp = dict(inputs_of(w))
    r = ref8.layer(w, inp, weights_of(w, inp))
    dl = DeviceLayer(w, inp)
    y0, z0 = ffn(dl, w, i32_dev(r["perm"]), i32_dev(r["offsets"]))
    dl.hidden[7, 3], dl.hidden[200, 0] = float("inf"), float("nan")
    dl.w_down[2, 33, 5] = float("nan")
    y, z = ffn(dl, w, i32_dev(r["perm"]), i32_dev(r["offsets"]))
    tok = torch.from_numpy(np.asarray(r["perm"], np.int64) // w.top_k).cuda()
    bad = (tok == 7) | (tok == 200)
    assert torch.isnan(y[bad]).all() and torch.isnan(z[[7, 200]]).all()
    of2 = torch.zeros(w.S, dtype=torch.bool, device="cuda")
    of2[int(r["offsets"][2]):int(r["offsets"][3])] = True
    assert torch.isnan(y[of2][:, 33]).all()
    keep = ~bad[:, None] & ~(of2[:, None] & (torch.arange(w.H, device="cuda") == 33))
    assert torch.equal(y[keep], y0[keep])
    rest = torch.ones(w.T, dtype=torch.bool, device="cuda")
    rest[[7, 200]] = False
    assert torch.equal(z[rest], z0[rest])


def test_right_behind_the_quantiser_and_other_layers():
    """Calls back to back, weights quantised anew before each: the same bits as with a synchronize between them."""
    w = MID.with_(name="mid_back", T=40)
    inp = W.layer_inputs(w)
    r = ref8.layer(w, inp, ref8.quantize_weights(inp))
    perm, offsets = i32_dev(r["perm"]), i32_dev(r["offsets"])
    dl = DeviceLayer(w, inp)
    sets = [(dl.w_gate, dl.w_up, dl.w_down), (dl.w_up, dl.w_gate, dl.w_down)]
    want = []
    for s in sets:
        y, z = (torch.empty((n, w.H), dtype=torch.bfloat16, device="cuda") for n in (w.S, w.T))
        ex = moe.quantize_int8_experts(*s, dl.ws_gate, dl.ws_up, dl.ws_down)
        torch.cuda.synchronize()
        moe.moe_expert_ffn_int8(dl.d, dl.hidden, perm, offsets, ex, y, z, dl.ws)
        torch.cuda.synchronize()
        want.append((y, z))
    got = []
    for i in range(20):
        y, z = (torch.empty((n, w.H), dtype=torch.bfloat16, device="cuda") for n in (w.S, w.T))
        ex = moe.quantize_int8_experts(*sets[i & 1], dl.ws_gate, dl.ws_up, dl.ws_down)
        moe.moe_expert_ffn_int8(dl.d, dl.hidden, perm, offsets, ex, y, z, dl.ws)
        got.append((y, z, ex))
    torch.cuda.synchronize()
    for i, (y, z, _) in enumerate(got):
        assert torch.equal(y, want[i & 1][0]) and torch.equal(z, want[i & 1][1]), i


def test_one_workspace_for_a_batch_and_smaller_ones():
    """A workspace made for the largest batch serves smaller ones, and the other entries in between."""
    w = MID
    inp = inputs_of(w)
    dl = DeviceLayer(w, inp)
    experts = dev_experts(dl)
    for T in (300, 1, 64, 300, 33):
        d = moe.dims(T, w.H, w.E, w.I, w.top_k, w.I_shared)
        out, own = (torch.empty((T, w.H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        moe.moe_layer_forward_int8(d, dl.hidden[:T], dl.router_w, dl.bias, experts, out, dl.ws)
        moe.moe_layer_forward(d, dl.hidden[:T], dl.router_w, dl.bias, dl.w_gate, dl.w_up, dl.w_down, dl.ws_gate, dl.ws_up,
                              dl.ws_down, own, dl.ws)
        fresh = torch.empty_like(out)
        moe.moe_layer_forward_int8(d, dl.hidden[:T], dl.router_w, dl.bias, experts, fresh, moe.alloc_workspace(d))
        torch.cuda.synchronize()
        assert torch.equal(out, fresh), T
        # 8-bit rows of normal values: rounding noise of about 1 % of a row's values in each factor
        a, b = host_f64(out), host_f64(own)
        assert np.linalg.norm(a - b) <= 0.05 * np.linalg.norm(b)
    assert moe.moe_ws_read_error(dl.ws) == 0
