"""Operators of the MoE FFN layer for few tokens and for 4-bit experts: cases, plain forms and the library's calls.

Four operators share this file:

quantize   expert weights to MXFP4 and back: blocks of 32 values along a row share a
           power-of-two scale, elements are E2M1 (moe_quantize_mxfp4_rows,
           moe_dequantize_mxfp4_rows)
few        a whole MoE FFN layer for a few tokens, bf16 weights (moe_layer_forward_few)
layer4     a whole MoE FFN layer with MXFP4 expert weights (moe_layer_forward_mxfp4)
ffn4       the grouped expert FFN with MXFP4 weights for a given routing
           (moe_expert_ffn_mxfp4)

Packed codes: a row of K values (K a multiple of 128) is K / 128 pieces of 64 bytes.
The piece's 32-bit word 4 t + q (t, q in 0..3) holds the codes of values
32 q + 8 t .. 32 q + 8 t + 7 of the piece, the first in the lowest four bits.  The
scale of a block of 32 is one byte e that stands for 2^(e - 127).

`own` chooses what run() computes: the plain form in elementary torch operations
(false) or the library's entry points (true).
"""
import functools
import math

import torch

own = False

ROUTE_SCALE = 2.826
BLOCK = 32


# --------------------------------------------------------------------- cases
def listed():
    hy3 = dict(H=4096, E=192, I=1536, k=8, mode="sigmoid", shared=1536)
    return [
        # one expert's gate matrix, as when a single expert is updated in place
        dict(name="quantize one expert", op="quantize", rows=1536, cols=4096),
        # the gate matrices of 64 stacked experts, as when a checkpoint is loaded
        dict(name="quantize stack", op="quantize", rows=64 * 1536, cols=4096),
        # one user's single-token decode step
        dict(name="few T1", op="few", T=1, **hy3),
        # the decode batch that the benchmark measures
        dict(name="few T8", op="few", T=8, **hy3),
        # a softmax-routed layer of odd widths without a shared expert
        dict(name="few T13 odd", op="few", T=13, H=1088, E=48, I=704, k=6, mode="softmax", shared=0),
        # the largest batch of the one-kernel layer: speculative tokens of several users
        dict(name="few T32", op="few", T=32, **hy3),
        # 4-bit experts: one user's single-token step, the decode batch, an odd softmax layer
        dict(name="layer4 T1", op="layer4", T=1, **hy3),
        dict(name="layer4 T8", op="layer4", T=8, **hy3),
        dict(name="layer4 T21 odd", op="layer4", T=21, H=1152, E=40, I=640, k=5, mode="softmax", shared=384),
        # the expert step alone: a decode batch, an uneven middle batch with idle experts, a prompt
        dict(name="ffn4 T8", op="ffn4", T=8, skew=0.0, **hy3),
        dict(name="ffn4 T300 uneven", op="ffn4", T=300, H=1152, E=40, I=640, k=5, mode="softmax", shared=384, skew=2.5),
        dict(name="ffn4 T4096", op="ffn4", T=4096, skew=0.0, **hy3),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "few", "layer4", "ffn4"])
    if op == "quantize":
        return dict(op=op, rows=_spread(rng, 1, 98304), cols=128 * _spread(rng, 1, 32))
    unit = 64 if op == "few" else 128
    E = _spread(rng, 2, 192)
    c = dict(op=op, H=unit * _spread(rng, 2, 4096 // unit), E=E, I=unit * _spread(rng, 1, 1536 // unit),
             k=rng.randint(1, min(8, E)), mode=rng.choice(["sigmoid", "softmax"]))
    c["T"] = _spread(rng, 1, 4096 if op == "ffn4" else 32)
    c["shared"] = rng.choice([0, c["I"], unit * _spread(rng, 1, 1536 // unit)])
    if op == "ffn4":
        c["skew"] = rng.choice([0.0, 1.0, 2.5])
    return c


def _active(c):
    """Experts that a batch reaches when its tokens choose evenly."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(c):
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        # read bf16, write codes and scales; read those, write bf16
        return {"bytes": 2 * n + 2 * (n / 2 + n / BLOCK) + 2 * n, "flops": 2 * n}
    T, H, I, S = c["T"], c["H"], c["I"], c["T"] * c["k"]
    per = 2.0 if c["op"] == "few" else 0.5 + 1.0 / BLOCK
    weights = 3 * H * (I * _active(c) + c["shared"]) * per
    flops = 6.0 * H * (S * I + T * c["shared"])
    if c["op"] == "ffn4":
        return {"bytes": weights + 2 * T * H + 4 * (S + c["E"] + 1) + 2 * H * (S + (T if c["shared"] else 0)), "flops": flops}
    return {"bytes": weights + 4 * c["E"] * (H + 1) + 4 * T * H, "flops": flops + 2.0 * T * H * c["E"]}


# -------------------------------------------------------------------- inputs
def _normal(gen, shape, sigma, dtype):
    """N(0, sigma^2) of `dtype`, drawn in pieces so that the fp32 draws stay small."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, device="cuda", generator=gen) * sigma
    return out


def _exponents(blocks):
    """Biased scale exponent of blocks [..., 32] in fp32: floor(log2 max|v|) - 2, at least -127."""
    bits = blocks.abs().amax(-1).view(torch.int32)
    return ((bits >> 23) - 2).clamp(min=0)


def _element_codes(scaled):
    """E2M1 codes (sign, then 0 .. 7 for 0, .5, 1, 1.5, 2, 3, 4, 6) of fp32 values: nearest, ties to the even code."""
    a = scaled.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c | (torch.signbit(scaled).to(torch.uint8) << 3)


def _power(e):
    """2^(e - 127) in fp32 for biased exponents e in 1 .. 254."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _pack_rows(w):
    """Packed codes [R, K / 2] and scale bytes [R, K / 32] of rows [R, K] in fp32."""
    R, K = w.shape
    blocks = w.view(R, K // BLOCK, BLOCK)
    e = _exponents(blocks)
    codes = _element_codes(blocks / _power(e.clamp(min=1))[..., None])
    pairs = codes.view(R, K // 128, 4, 4, 4, 2)          # piece, q, t, byte, nibble
    packed = pairs[..., 0] | (pairs[..., 1] << 4)
    return packed.transpose(2, 3).reshape(R, K // 2), e.to(torch.uint8)


def _mxfp4_normal(gen, shape, sigma):
    K, R = shape[-1], math.prod(shape[:-1])
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((R, K // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // K)
    for i in range(0, R, step):
        n = min(step, R - i)
        w = (torch.randn((n, K), device="cuda", generator=gen) * sigma).bfloat16().float()
        codes[i:i + n], scales[i:i + n] = _pack_rows(w)
    return codes.view(*shape[:-1], K // 2), scales.view(*shape[:-1], K // BLOCK)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    if c["op"] == "quantize":
        return {"case": c, "src": _normal(gen, (c["rows"], c["cols"]), 0.02, torch.bfloat16)}
    T, H, E, I, k, Is = (c[n] for n in ("T", "H", "E", "I", "k", "shared"))
    s = {"case": c, "hidden": _normal(gen, (T, H), 1.0, torch.bfloat16)}
    make = (lambda shape: _normal(gen, shape, 0.02, torch.bfloat16)) if c["op"] == "few" else (
        lambda shape: _mxfp4_normal(gen, shape, 0.02))
    s["gate"], s["up"], s["down"] = make((E, I, H)), make((E, I, H)), make((E, H, I))
    if Is:
        s["s_gate"], s["s_up"], s["s_down"] = make((Is, H)), make((Is, H)), make((H, Is))
    if c["op"] == "ffn4":
        # a routing: each token's k experts by noisy popularity, slots sorted by expert
        liking = torch.randn(E, device="cuda", generator=gen) * c["skew"]
        idx = torch.topk(liking + torch.randn((T, E), device="cuda", generator=gen), k, dim=1).indices
        s["perm"] = torch.sort(idx.reshape(-1), stable=True).indices.int()
        counts = torch.bincount(idx.reshape(-1), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    else:
        s["router_w"] = _normal(gen, (E, H), 0.02, torch.float32)
        s["bias"] = _normal(gen, (E,), 0.01, torch.float32)
    return s


# --------------------------------------------------------------- plain forms
def _element(code):
    """fp32 values of E2M1 codes."""
    m = code & 7
    mag = torch.where(m < 2, m * 0.5, (1 + (m & 1) * 0.5) * (1 << (m >> 1)) * 0.5)
    return torch.where(code > 7, -mag, mag)


@functools.cache
def _byte_values(device):
    """The two values (low nibble, high nibble) of each byte of codes: [256, 2], a constant."""
    table = _element(torch.arange(16, device=device))
    return torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)


def _values(weight):
    """fp32 values of a weight: bf16 as it is, or (codes, scales) of MXFP4."""
    if not isinstance(weight, tuple):
        return weight.float()
    codes, e = weight
    lead, K = codes.shape[:-1], codes.shape[-1] * 2
    both = _byte_values(codes.device)
    byte = codes.view(*lead, K // 128, 4, 4, 4).transpose(-3, -2)             # piece, q, t, byte
    v = both[byte.int()].reshape(*lead, K // BLOCK, BLOCK)
    return (v * _power(e)[..., None]).view(*lead, K)


def _of(weight, index):
    return tuple(x[index] for x in weight) if isinstance(weight, tuple) else weight[index]


def _swiglu(x, gate, up, down):
    """x [n, t, H] or [t, H] through stacked (or single) expert weights, in fp32."""
    g, u = x @ _values(gate).mT, x @ _values(up).mT
    return (g * torch.sigmoid(g) * u) @ _values(down).mT


def _slot_outputs(s, expert, token):
    """FFN of each slot's token by the slot's expert: [S, H] in fp32."""
    x, E = s["hidden"].float(), s["case"]["E"]
    if expert.numel() <= E:  # the slots' own weights, gathered
        w = [_of(s[n], expert) for n in ("gate", "up", "down")]
        return _swiglu(x[token][:, None], *w)[:, 0]
    return _swiglu(x.expand(E, -1, -1), s["gate"], s["up"], s["down"])[expert, token]


def _shared(s):
    return _swiglu(s["hidden"].float(), s["s_gate"], s["s_up"], s["s_down"]) if s["case"]["shared"] else None


def _route(s):
    """Experts and weights of each token.  The keys decide between experts: 64 bits."""
    c = s["case"]
    logits = s["hidden"].double() @ s["router_w"].double().T
    score = torch.sigmoid(logits) if c["mode"] == "sigmoid" else torch.softmax(logits, -1)
    key = score + s["bias"].double() if c["mode"] == "sigmoid" else score
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    sel = score.gather(1, idx)
    w = sel / sel.sum(-1, keepdim=True) * ROUTE_SCALE if c["mode"] == "sigmoid" else sel / sel.sum(-1, keepdim=True).clamp(min=1e-8)
    return idx, w.float()


def _plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        blocks = s["src"].float().view(c["rows"], -1, BLOCK)
        e = _exponents(blocks)
        p = _power(e.clamp(min=1))[..., None]
        values = _element(_element_codes(blocks / p).int()) * p
        return {"values": values.view(c["rows"], c["cols"]).bfloat16(), "scales": e.to(torch.uint8)}
    if c["op"] == "ffn4":
        slot = torch.arange(c["T"] * c["k"], device="cuda")
        expert = torch.searchsorted(s["offsets"].long(), slot, right=True) - 1
        y = _slot_outputs(s, expert, s["perm"].long() // c["k"]).bfloat16()
        z = _shared(s)
        return {"y": y} if z is None else {"y": y, "z": z.bfloat16()}
    idx, w = _route(s)
    token = torch.arange(c["T"], device="cuda").repeat_interleave(c["k"])
    y = _slot_outputs(s, idx.reshape(-1), token).view(c["T"], c["k"], c["H"])
    out = (y * w[..., None]).sum(1)
    z = _shared(s)
    return {"out": (out if z is None else out + z).bfloat16()}


# -------------------------------------------------------- the library's calls
def _handle(s):
    """What a program keeps beside its weights: the layer's dims, a workspace and the output buffers."""
    if "d" in s:
        return s
    import expert_ffn_layer_gb300 as moe

    c = s["case"]
    if c["op"] == "quantize":
        r, n = c["rows"], c["cols"]
        s["codes"] = torch.empty((r, n // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((r, n // BLOCK), dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty((r, n), dtype=torch.bfloat16, device="cuda")
        s["d"] = None
        return s
    sigmoid = c["mode"] == "sigmoid"
    s["d"] = moe.dims(c["T"], c["H"], c["E"], c["I"], c["k"], I_shared=c["shared"], score_mode=c["mode"],
                      route_scale=ROUTE_SCALE if sigmoid else 1.0, renorm_eps=0.0 if sigmoid else 1e-8,
                      has_shared=c["shared"] > 0)
    s["ws"] = moe.alloc_workspace(s["d"])
    if c["op"] != "few":
        s["experts"] = moe.Mxfp4Experts(**{n: s[n] for n in moe.Mxfp4Experts.NAMES if n in s})
    if c["op"] == "ffn4":
        s["y"] = torch.empty((c["T"] * c["k"], c["H"]), dtype=torch.bfloat16, device="cuda")
        s["z"] = torch.empty((c["T"], c["H"]), dtype=torch.bfloat16, device="cuda") if c["shared"] else None
    else:
        s["out"] = torch.empty((c["T"], c["H"]), dtype=torch.bfloat16, device="cuda")
    return s


def _library(s):
    import expert_ffn_layer_gb300 as moe

    s, c = _handle(s), s["case"]
    if c["op"] == "quantize":
        moe.moe_quantize_mxfp4_rows(s["src"], s["codes"], s["scales"])
        moe.moe_dequantize_mxfp4_rows(s["codes"], s["scales"], s["values"])
        return {"values": s["values"], "scales": s["scales"]}
    if c["op"] == "ffn4":
        moe.moe_expert_ffn_mxfp4(s["d"], s["hidden"], s["perm"], s["offsets"], s["experts"], s["y"], s["z"], s["ws"])
        return {"y": s["y"]} if s["z"] is None else {"y": s["y"], "z": s["z"]}
    if c["op"] == "few":
        moe.moe_layer_forward_few(s["d"], s["hidden"], s["router_w"], s["bias"], s["gate"], s["up"], s["down"],
                                  s.get("s_gate"), s.get("s_up"), s.get("s_down"), s["out"], s["ws"])
    else:
        moe.moe_layer_forward_mxfp4(s["d"], s["hidden"], s["router_w"], s["bias"], s["experts"], s["out"], s["ws"])
    return {"out": s["out"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------- 64-bit answers
def _exact_matrix(weight):
    """fp64 matrix [R, K] of one expert's weight, by walking the packed layout's definition."""
    if not isinstance(weight, tuple):
        return weight.double()
    codes, e = weight
    R, K = codes.shape[0], codes.shape[1] * 2
    j = torch.arange(K, device=codes.device)
    piece, q, t, i = j // 128, j // 32 % 4, j // 8 % 4, j % 8
    at = 64 * piece + 4 * (4 * t + q) + i // 2
    nibble = (codes[:, at].long() >> (4 * (i % 2))) & 15
    exponent, mantissa = (nibble >> 1) & 3, (nibble & 1).double()
    mag = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * torch.exp2((exponent - 1).double()))
    sign = 1.0 - 2.0 * (nibble >> 3).double()
    return sign * mag * torch.exp2(e.double() - 127).repeat_interleave(BLOCK, 1)


def _exact_ffn(x, s, names, e=None):
    w = [_exact_matrix(s[n] if e is None else _of(s[n], e)) for n in names]
    g, u = x @ w[0].T, x @ w[1].T
    return (g / (1 + torch.exp(-g)) * u) @ w[2].T


def _exact_quantize(src):
    """Values and scale bytes of rows by distance to every element value, in pieces."""
    e_out, v_out = [], []
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    odd = torch.arange(8, device="cuda") % 2
    for rows in src.split(max(1, (1 << 22) // src.shape[1])):
        b = rows.double().view(rows.shape[0], -1, BLOCK)
        top = b.abs().amax(-1)
        e = torch.where(top > 0, torch.frexp(top).exponent - 1 - 2, torch.full_like(top, -127).int()).clamp(min=-127)
        scale = torch.exp2(e.double())[..., None]
        a = b.abs() / scale
        off = (a[..., None] - table).abs()
        near = off == off.amin(-1, keepdim=True)                    # one value, or two at a tie
        code = torch.where(near, odd, 2).argmin(-1)                 # the even one of a tie
        v_out.append((torch.sign(b) * table[code] * scale).view(rows.shape))
        e_out.append(e + 127)
    return {"values": torch.cat(v_out), "scales": torch.cat(e_out)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        return _exact_quantize(s["src"])
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    x = s["hidden"].double()
    z = _exact_ffn(x, s, ("s_gate", "s_up", "s_down")) if c["shared"] else None
    if c["op"] == "ffn4":
        y = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(E):
            if off[e + 1] > off[e]:
                token = s["perm"][off[e]:off[e + 1]].long() // k
                y[off[e]:off[e + 1]] = _exact_ffn(x[token], s, ("gate", "up", "down"), e)
        return {"y": y} if z is None else {"y": y, "z": z}
    logits = x @ s["router_w"].double().T
    if c["mode"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
        key = score + s["bias"].double()
    else:
        score = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
        key = score.clone()
    weight = torch.zeros_like(score)
    for _ in range(k):  # the largest key left; the first of equal ones
        best = (key == key.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
        weight.scatter_(1, best, score.gather(1, best))
        key.scatter_(1, best, -math.inf)
    total = weight.sum(-1, keepdim=True)
    weight = weight / total * ROUTE_SCALE if c["mode"] == "sigmoid" else weight / total.clamp(min=1e-8)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda") if z is None else z
    for e in torch.nonzero(weight.sum(0)).flatten().tolist():
        token = torch.nonzero(weight[:, e]).flatten()
        out[token] += weight[token, e, None] * _exact_ffn(x[token], s, ("gate", "up", "down"), e)
    return {"out": out}
