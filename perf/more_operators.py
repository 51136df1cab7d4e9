"""Operators of the MoE FFN layer for 8-bit integer experts and for training its router: cases, plain forms and the library's calls.

Five operators share this file:

rows8         rows of bf16 values to 8-bit integers with one scale a row, and back
              (moe_quantize_int8_rows, moe_dequantize_int8_rows)
ffn8          the grouped expert FFN for a given routing, weights and activations in
              8-bit integers: a scale for each token and one for each weight row
              (moe_expert_ffn_int8)
balance       per-expert counts of each sequence, the balance loss and the z loss of
              the router's logits, and their gradient with respect to the logits
              (moe_balance_loss, moe_route_backward without a routing gradient)
route_grad    gradients of the combine weights and of both losses with respect to the
              logits, the hidden state and the router weight (moe_route_backward)
combine_grad  gradients of the combine with respect to its weights and to the experts'
              outputs (moe_combine_backward)

A row's scale is its largest magnitude over 127 (1 for a row of zeros), its codes are
127 w / max|row| to the nearest integer, ties to the even one.

A token belongs to sequence seq_id[t]; a negative number marks padding, which counts
nowhere and gets no gradient.

`own` chooses what run() computes: the plain form in elementary torch operations
(false) or the library's entry points (true).
"""
import math

import torch

own = False

ROUTE_SCALE = 2.826


# --------------------------------------------------------------------- cases
def listed():
    hy3 = dict(H=4096, E=192, I=1536, k=8, mode="sigmoid", shared=1536)
    router = dict(H=4096, E=192, k=8, mode="sigmoid")
    return [
        # one expert's gate matrix, as when a single expert is updated in place
        dict(name="rows8 one expert", op="rows8", rows=1536, cols=4096),
        # the gate matrices of 64 stacked experts, as when a checkpoint is loaded
        dict(name="rows8 stack", op="rows8", rows=64 * 1536, cols=4096),
        # the expert step of the decode batch that the benchmark measures
        dict(name="ffn8 T8", op="ffn8", T=8, skew=0.0, **hy3),
        # a middle batch of odd widths with idle and crowded experts
        dict(name="ffn8 T300 uneven", op="ffn8", T=300, H=1088, E=40, I=704, k=5, mode="softmax", shared=320, skew=2.5),
        # a prompt
        dict(name="ffn8 T4096", op="ffn8", T=4096, skew=0.0, **hy3),
        # the losses of a training step's tokens, one sequence
        dict(name="balance T4096", op="balance", T=4096, seqs=1, pad=0.0, **router),
        # a packed batch of uneven sequences with padding, softmax routing
        dict(name="balance T16384 packed", op="balance", T=16384, seqs=23, pad=0.1, H=4096, E=64, k=8, mode="softmax"),
        # the smallest router step: a few tokens, where launches count
        dict(name="route_grad T8", op="route_grad", T=8, seqs=1, pad=0.0, **router),
        # an odd softmax router over packed uneven sequences with padding
        dict(name="route_grad T1000 packed", op="route_grad", T=1000, seqs=7, pad=0.15, H=1088, E=40, k=5, mode="softmax"),
        # a training step's tokens
        dict(name="route_grad T4096", op="route_grad", T=4096, seqs=4, pad=0.0, **router),
        # a few tokens of an odd layer, and a training step's tokens
        dict(name="combine_grad T13 odd", op="combine_grad", T=13, H=1088, k=6),
        dict(name="combine_grad T4096", op="combine_grad", T=4096, H=4096, k=8),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows8", "ffn8", "balance", "route_grad", "combine_grad"])
    if op == "rows8":
        return dict(op=op, rows=_spread(rng, 1, 98304), cols=64 * _spread(rng, 1, 64))
    c = dict(op=op, T=_spread(rng, 1, 4096 if op == "ffn8" else 16384), H=64 * _spread(rng, 2, 64))
    if op == "combine_grad":
        return dict(c, k=rng.randint(1, 8))
    E = _spread(rng, 2, 192 if op == "ffn8" else 256)
    c.update(E=E, k=rng.randint(1, min(8, E)), mode=rng.choice(["sigmoid", "softmax"]))
    if op == "ffn8":
        c["I"] = 64 * _spread(rng, 1, 24)
        c["shared"] = rng.choice([0, c["I"], 64 * _spread(rng, 1, 24)])
        c["skew"] = rng.choice([0.0, 1.0, 2.5])
    else:
        c["seqs"] = _spread(rng, 1, 64)
        c["pad"] = rng.choice([0.0, 0.1, 0.5])
    return c


def work(c):
    if c["op"] == "rows8":
        n = c["rows"] * c["cols"]
        # read bf16, write codes and scales; read those, write bf16
        return {"bytes": 6 * n + 8 * c["rows"], "flops": 3 * n}
    T, H, k = c["T"], c["H"], c["k"]
    S = T * k
    if c["op"] == "combine_grad":
        return {"bytes": 2 * T * H + 2 * S * H + 8 * S + 2 * S * H + 4 * S, "flops": 3 * S * H}
    E = c["E"]
    if c["op"] == "ffn8":
        active = E * (1.0 - (1.0 - k / E) ** T)  # experts that a batch reaches when its tokens choose evenly
        I, Is = c["I"], c["shared"]
        weights = 3 * H * (I * active + Is) + 4 * (active * (2 * I + H) + (2 * Is + H if Is else 0))
        return {"bytes": weights + 2 * T * H + 4 * (S + E + 1) + 2 * H * (S + (T if Is else 0)),
                "flops": 6.0 * H * (S * I + T * Is)}
    read = 4 * T * E + 4 * S + 4 * T
    if c["op"] == "balance":
        return {"bytes": read + 4 * c["seqs"] * (E + 1) + 16 + 4 * T * E, "flops": 16 * T * E}
    return {"bytes": read + 4 * S + 4 * T * E + 4 * T * H + 8 * E * H, "flops": 4.0 * T * E * H}


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


def _row_codes(x):
    """Codes (whole numbers in fp32) and scales of rows [.., K] in fp32."""
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / torch.full_like(top, 127.0), torch.ones_like(top))
    return torch.round(x * 127 / torch.where(top > 0, top, torch.ones_like(top))[..., None]), scale


def _int8_normal(gen, shape, sigma):
    K, R = shape[-1], math.prod(shape[:-1])
    codes = torch.empty((R, K), dtype=torch.int8, device="cuda")
    scales = torch.empty(R, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 25) // K)
    for i in range(0, R, step):
        n = min(step, R - i)
        q, s = _row_codes((torch.randn((n, K), device="cuda", generator=gen) * sigma).bfloat16().float())
        codes[i:i + n], scales[i:i + n] = q.to(torch.int8), s
    return codes.view(shape), scales.view(shape[:-1])


def _routing(gen, T, E, k, skew):
    """Each token's k experts by noisy popularity: slots sorted by expert, offsets, and the largest count."""
    liking = torch.randn(E, device="cuda", generator=gen) * skew
    idx = torch.topk(liking + torch.randn((T, E), device="cuda", generator=gen), k, dim=1).indices
    perm = torch.sort(idx.reshape(-1), stable=True).indices
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    return perm.int(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(), int(counts.max())


def _sequences(gen, T, seqs, pad):
    """seq_id of a packed batch: `seqs` uneven runs (some empty where they are many), the last tokens padding."""
    real = T - int(pad * T)
    cuts = torch.sort(torch.randint(0, real + 1, (seqs - 1,), device="cuda", generator=gen)).values
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cuts, t, right=True)
    return torch.where(t < real, b, torch.full_like(b, -1)).int()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 29)
    if c["op"] == "rows8":
        return {"case": c, "src": _normal(gen, (c["rows"], c["cols"]), 0.02, torch.bfloat16)}
    T, H, k = c["T"], c["H"], c["k"]
    if c["op"] == "combine_grad":
        w = torch.rand((T, k), device="cuda", generator=gen) + 0.05
        return {"case": c, "grad_out": _normal(gen, (T, H), 1e-3, torch.bfloat16),
                "y": _normal(gen, (T * k, H), 1.0, torch.bfloat16),
                "inv": torch.randperm(T * k, device="cuda", generator=gen).int(),
                "w": w / w.sum(-1, keepdim=True) * ROUTE_SCALE}
    E = c["E"]
    s = {"case": c, "hidden": _normal(gen, (T, H), 1.0, torch.bfloat16)}
    if c["op"] == "ffn8":
        I, Is = c["I"], c["shared"]
        s["gate"], s["up"] = _int8_normal(gen, (E, I, H), 0.02), _int8_normal(gen, (E, I, H), 0.02)
        s["down"] = _int8_normal(gen, (E, H, I), 0.02)
        if Is:
            s["s_gate"], s["s_up"] = _int8_normal(gen, (Is, H), 0.02), _int8_normal(gen, (Is, H), 0.02)
            s["s_down"] = _int8_normal(gen, (H, Is), 0.02)
        s["perm"], s["offsets"], s["most"] = _routing(gen, T, E, k, c["skew"])
        return s
    # what the forward step left: the router's logits, each token's experts, the loss's counts
    s["router_w"] = _normal(gen, (E, H), 0.02, torch.float32)
    s["logits"] = s["hidden"].float() @ s["router_w"].T
    bias = _normal(gen, (E,), 0.01, torch.float32)
    key = torch.sigmoid(s["logits"]) + bias if c["mode"] == "sigmoid" else s["logits"]
    s["idx"] = torch.topk(key, k, dim=1).indices.int()
    s["seq_id"] = _sequences(gen, T, c["seqs"], c["pad"])
    s["grad_losses"] = torch.tensor([1e-2, 1e-3], device="cuda")
    if c["op"] == "route_grad":
        s["counts"], s["tokens"] = _counts(s)
        s["grad_w"] = _normal(gen, (T, k), 1e-3, torch.float32)
    return s


# --------------------------------------------------------------- plain forms
def _swiglu(x, gate, up, down):
    """x [.., t, H] in fp32 through stacked (or single) int8 weights; the sums of codes in fp32."""
    q, sx = _row_codes(x)
    g = q @ gate[0].float().mT * sx[..., None] * gate[1][..., None, :]
    u = q @ up[0].float().mT * sx[..., None] * up[1][..., None, :]
    q, sa = _row_codes((g * torch.sigmoid(g) * u).bfloat16().float())
    return q @ down[0].float().mT * sa[..., None] * down[1][..., None, :]


def _of(weight, index):
    return tuple(x[index] for x in weight)


def _plain_ffn(s):
    c = s["case"]
    x, S = s["hidden"].float(), c["T"] * c["k"]
    token = s["perm"].long() // c["k"]
    experts = [s[n] for n in ("gate", "up", "down")]
    first, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    if S <= c["E"]:  # the slots' own weights, gathered
        expert = torch.searchsorted(end, torch.arange(S, device="cuda"), right=True)
        y = _swiglu(x[token][:, None], *(_of(w, expert) for w in experts))[:, 0]
    else:  # every expert's tokens in rows of their own, as many as the busiest expert has
        at = first[:, None] + torch.arange(s["most"], device="cuda")
        live = at < end[:, None]
        y = _swiglu(x[token[at.clamp(max=S - 1)]], *experts)[live]  # in the order of the experts, as the slots are sorted
    out = {"y": y.bfloat16()}
    if c["shared"]:
        out["z"] = _swiglu(x, s["s_gate"], s["s_up"], s["s_down"]).bfloat16()
    return out


def _counts(s):
    """Choices of each expert by each sequence's tokens, and the sequences' tokens: whole numbers."""
    c, b = s["case"], s["seq_id"].long()
    here = b >= 0
    cell = torch.where(here, b * c["E"], torch.zeros_like(b))[:, None] + s["idx"].long()
    size = c["seqs"] * c["E"]
    counts = torch.zeros(size, dtype=torch.int32, device="cuda").scatter_add_(
        0, cell.reshape(-1), here.int()[:, None].expand(-1, c["k"]).reshape(-1))
    tokens = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda").scatter_add_(0, b.clamp(min=0), here.int())
    return counts.view(c["seqs"], c["E"]), tokens


def _loads(c, counts, tokens):
    """d balance / d (score of a token of sequence b for expert e), per token: [B, E] in fp32."""
    n = tokens.clamp(min=1).float()
    return counts.float() * (c["E"] / c["k"]) / (n * n)[:, None] / (tokens > 0).sum().clamp(min=1)


def _shares(c, logits):
    """Each token's scores normalised over all experts."""
    if c["mode"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
    else:
        e = torch.sigmoid(logits)
    return e / e.sum(-1, keepdim=True)


def _log_sum(logits):
    top = logits.amax(-1)
    return top + torch.log(torch.exp(logits - top[:, None]).sum(-1))


def _plain_balance(s):
    c, l = s["case"], s["logits"]
    counts, tokens = _counts(s)
    b = s["seq_id"].long()
    here = b >= 0
    F, q, lse = _loads(c, counts, tokens)[b.clamp(min=0)], _shares(c, l), _log_sum(l)
    mean = (F * q).sum(-1)
    n = here.sum().clamp(min=1)
    losses = torch.stack([torch.where(here, mean, torch.zeros_like(mean)).double().sum(),
                          torch.where(here, lse * lse, torch.zeros_like(lse)).double().sum() / n]).float()
    d = _loss_grad(s, F, q, lse, n)
    return {"counts": counts, "tokens": tokens, "losses": losses, "logits": torch.where(here[:, None], d, torch.zeros_like(d))}


def _loss_grad(s, F, q, lse, n):
    """Gradient of both losses, weighted by grad_losses, with respect to the logits of counted tokens."""
    l = s["logits"]
    d = s["grad_losses"][0] * q * (F - (F * q).sum(-1, keepdim=True))
    if s["case"]["mode"] == "sigmoid":
        d = d * torch.sigmoid(-l)  # 1 - sigmoid(l)
    return d + s["grad_losses"][1] * 2 / n * lse[:, None] * torch.exp(l - lse[:, None])


def _plain_route_grad(s):
    c, l = s["case"], s["logits"]
    b = s["seq_id"].long()
    here = b >= 0
    idx, g, q = s["idx"].long(), s["grad_w"], _shares(c, l)
    d = _loss_grad(s, _loads(c, s["counts"], s["tokens"])[b.clamp(min=0)], q, _log_sum(l), here.sum().clamp(min=1))
    sel = (torch.sigmoid(l) if c["mode"] == "sigmoid" else q).gather(1, idx)
    u = sel / sel.sum(-1, keepdim=True)
    slope = g - (g * u).sum(-1, keepdim=True)
    if c["mode"] == "sigmoid":
        slope = ROUTE_SCALE * slope * torch.sigmoid(-l).gather(1, idx)
    d = d.scatter_add(1, idx, u * slope)
    d = torch.where(here[:, None], d, torch.zeros_like(d))
    return {"logits": d, "hidden": (d @ s["router_w"]).bfloat16(), "router_w": d.T @ s["hidden"].float()}


def _plain(s):
    c = s["case"]
    if c["op"] == "rows8":
        q, scale = _row_codes(s["src"].float())
        return {"values": (q * scale[:, None]).bfloat16(), "scales": scale}
    if c["op"] == "ffn8":
        return _plain_ffn(s)
    if c["op"] == "balance":
        return _plain_balance(s)
    if c["op"] == "route_grad":
        return _plain_route_grad(s)
    T, H, k = c["T"], c["H"], c["k"]
    at, dout = s["inv"].long(), s["grad_out"].float()
    grad_w = (s["y"].float()[at].view(T, k, H) * dout[:, None]).sum(-1)
    grad_y = torch.empty_like(s["y"])
    grad_y[at] = (s["w"][..., None] * dout[:, None]).bfloat16().view(T * k, H)
    return {"w": grad_w, "y": grad_y}


# -------------------------------------------------------- the library's calls
def _handle(s):
    """What a program keeps beside its inputs: the layer's dims, a workspace and the output buffers."""
    if "d" in s:
        return s
    import expert_ffn_layer_gb300 as moe

    c = s["case"]
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "rows8":
        s["codes"], s["scales"] = new((c["rows"], c["cols"]), torch.int8), new(c["rows"], torch.float32)
        s["values"] = new((c["rows"], c["cols"]), torch.bfloat16)
        s["d"] = None
        return s
    T, H, k = c["T"], c["H"], c["k"]
    sigmoid, Is = c.get("mode", "sigmoid") == "sigmoid", c.get("shared", 0)
    s["d"] = moe.dims(T, H, c.get("E", k), c.get("I", 64), k, I_shared=Is, score_mode="sigmoid" if sigmoid else "softmax",
                      route_scale=ROUTE_SCALE if sigmoid else 1.0, renorm_eps=0.0 if sigmoid else 1e-8, has_shared=Is > 0)
    if c["op"] == "combine_grad":
        s["out_w"], s["out_y"] = new((T, k), torch.float32), new((T * k, H), torch.bfloat16)
        return s
    s["ws"] = moe.alloc_workspace(s["d"])
    E = c["E"]
    if c["op"] == "ffn8":
        s["experts"] = moe.Int8Experts(**{n: s[n] for n in moe.Int8Experts.NAMES if n in s})
        s["out_y"] = new((T * k, H), torch.bfloat16)
        s["out_z"] = new((T, H), torch.bfloat16) if Is else None
    elif c["op"] == "balance":
        s["counts"], s["tokens"] = new((c["seqs"], E), torch.int32), new(c["seqs"], torch.int32)
        s["losses"] = new(2, torch.float32)
    if c["op"] != "ffn8":
        s["out_l"] = new((T, E), torch.float32)
    if c["op"] == "route_grad":
        s["out_x"], s["out_w"] = new((T, H), torch.bfloat16), new((E, H), torch.float32)
    return s


def _library(s):
    import expert_ffn_layer_gb300 as moe

    s, c = _handle(s), s["case"]
    if c["op"] == "rows8":
        moe.moe_quantize_int8_rows(s["src"], s["codes"], s["scales"])
        moe.moe_dequantize_int8_rows(s["codes"], s["scales"], s["values"])
        return {"values": s["values"], "scales": s["scales"]}
    if c["op"] == "ffn8":
        moe.moe_expert_ffn_int8(s["d"], s["hidden"], s["perm"], s["offsets"], s["experts"], s["out_y"], s["out_z"], s["ws"])
        return {"y": s["out_y"]} if s["out_z"] is None else {"y": s["out_y"], "z": s["out_z"]}
    if c["op"] == "balance":
        moe.moe_balance_loss(s["d"], s["logits"], s["idx"], s["counts"], s["tokens"], s["losses"], s["ws"], seq_id=s["seq_id"])
        moe.moe_route_backward(s["d"], s["logits"], s["idx"], s["ws"], grad_losses=s["grad_losses"], counts=s["counts"],
                               tokens=s["tokens"], seq_id=s["seq_id"], grad_logits=s["out_l"])
        return {"counts": s["counts"], "tokens": s["tokens"], "losses": s["losses"], "logits": s["out_l"]}
    if c["op"] == "route_grad":
        moe.moe_route_backward(s["d"], s["logits"], s["idx"], s["ws"], grad_w=s["grad_w"], grad_losses=s["grad_losses"],
                               counts=s["counts"], tokens=s["tokens"], seq_id=s["seq_id"], hidden=s["hidden"],
                               router_w=s["router_w"], grad_logits=s["out_l"], grad_hidden=s["out_x"], grad_router_w=s["out_w"])
        return {"logits": s["out_l"], "hidden": s["out_x"], "router_w": s["out_w"]}
    moe.moe_combine_backward(s["d"], s["grad_out"], s["y"], s["inv"], s["w"], s["out_w"], s["out_y"])
    return {"w": s["out_w"], "y": s["out_y"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------- 64-bit answers
def _exact_rows(x):
    """Codes and scales of rows [R, K] in fp64: the scale is kept in 32 bits, the code is the integer nearest to 127 w / max."""
    top = x.abs().amax(-1)
    top = torch.where(top > 0, top, torch.full_like(top, 127.0))
    return torch.round(127 * x / top[:, None]), (top / 127).float().double()


def _exact_ffn(x, gate, up, down):
    q, sx = _exact_rows(x)
    g = (q @ gate[0].double().T) * torch.outer(sx, gate[1].double())
    u = (q @ up[0].double().T) * torch.outer(sx, up[1].double())
    q, sa = _exact_rows((g / (1 + torch.exp(-g)) * u).bfloat16().double())
    return (q @ down[0].double().T) * torch.outer(sa, down[1].double())


def _exact_losses(s):
    """Counts, tokens and both losses, sequence by sequence, and their derivative by the logits."""
    c, E = s["case"], s["case"]["E"]
    l = s["logits"].double()
    counts = torch.zeros((c["seqs"], E), dtype=torch.int64, device="cuda")
    tokens = torch.zeros(c["seqs"], dtype=torch.int64, device="cuda")
    members = [torch.nonzero(s["seq_id"] == b).flatten() for b in range(c["seqs"])]
    full = sum(1 for m in members if m.numel())
    total = sum(m.numel() for m in members)
    balance, z = l.new_zeros(()), l.new_zeros(())
    d_balance, d_z = torch.zeros_like(l), torch.zeros_like(l)
    for b, m in enumerate(members):
        n = m.numel()
        if not n:
            continue
        counts[b], tokens[b] = torch.bincount(s["idx"][m].long().flatten(), minlength=E), n
        f = counts[b].double() * E / (c["k"] * n)
        lse = torch.logsumexp(l[m], -1)
        p = torch.exp(l[m] - lse[:, None])
        if c["mode"] == "softmax":
            q, slope = p, torch.ones_like(p)
        else:
            score = 1 / (1 + torch.exp(-l[m]))
            q, slope = score / score.sum(-1, keepdim=True), 1 / (1 + torch.exp(l[m]))
        balance += (f * q.mean(0)).sum() / full
        z += lse.square().sum() / total
        d_balance[m] = q * slope * (f - (q * f).sum(-1, keepdim=True)) / (n * full)
        d_z[m] = 2 * lse[:, None] * p / total
    return counts, tokens, torch.stack([balance, z]), d_balance, d_z


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rows8":
        q, scale = _exact_rows(s["src"].double())
        return {"values": q * scale[:, None], "scales": scale}
    T, H, k = c["T"], c["H"], c["k"]
    if c["op"] == "combine_grad":
        grad_w = torch.empty((T, k), dtype=torch.float64, device="cuda")
        grad_y = torch.empty((T * k, H), dtype=torch.float64, device="cuda")
        for j in range(k):
            p = s["inv"].view(T, k)[:, j].long()
            grad_w[:, j] = (s["y"][p].double() * s["grad_out"].double()).sum(-1)
            grad_y[p] = s["w"][:, j, None].double() * s["grad_out"].double()
        return {"w": grad_w, "y": grad_y}
    if c["op"] == "ffn8":
        x = s["hidden"].double()
        y = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(c["E"]):
            if off[e + 1] > off[e]:
                rows = slice(off[e], off[e + 1])
                one = [(s[n][0][e], s[n][1][e]) for n in ("gate", "up", "down")]
                y[rows] = _exact_ffn(x[s["perm"][rows].long() // k], *one)
        return {"y": y, "z": _exact_ffn(x, s["s_gate"], s["s_up"], s["s_down"])} if c["shared"] else {"y": y}
    counts, tokens, losses, d_balance, d_z = _exact_losses(s)
    d = s["grad_losses"][0].double() * d_balance + s["grad_losses"][1].double() * d_z
    if c["op"] == "balance":
        return {"counts": counts, "tokens": tokens, "losses": losses, "logits": d}
    l, g, here = s["logits"].double(), s["grad_w"].double(), (s["seq_id"] >= 0)[:, None]
    score = 1 / (1 + torch.exp(-l)) if c["mode"] == "sigmoid" else torch.softmax(l, -1)
    sel = score.gather(1, s["idx"].long())
    w = sel / sel.sum(-1, keepdim=True)
    slope = g - (g * w).sum(-1, keepdim=True)
    if c["mode"] == "sigmoid":
        slope = slope * ROUTE_SCALE / (1 + torch.exp(l.gather(1, s["idx"].long())))
    d = d.scatter_add(1, s["idx"].long(), torch.where(here, w * slope, torch.zeros_like(w)))
    return {"logits": d, "hidden": d @ s["router_w"].double(), "router_w": d.T @ s["hidden"].double()}
