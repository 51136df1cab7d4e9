"""The 8-bit integer expert FFN and layer in float64 numpy, for the tests of the
int8 entries: rows quantised from their definition, one expert after the other."""
import numpy as np

import oracle


def quantize(rows):
    """Codes (int64) and scales (float64 holding fp32 values) of rows [.., K] of bf16 values."""
    x = np.asarray(rows, np.float64)
    m = np.abs(x).max(-1)
    safe = np.where(m > 0, m, 1.0)
    scale = np.where(m > 0, safe.astype(np.float32) / np.float32(127), np.float32(1)).astype(np.float64)
    return np.rint(127 * x / safe[..., None]).astype(np.int64), scale  # rint: ties to even


def ffn(x, gate, up, down):
    """x [t, H] float64; weights (codes, scales).  Sums of codes are exact (under 2^53)."""
    q, sx = quantize(x)
    g, u = (q.astype(np.float64) @ np.asarray(w[0], np.float64).T * sx[:, None] * w[1] for w in (gate, up))
    q, sa = quantize(oracle.bf16_round(g / (1 + np.exp(-g)) * u))
    return q.astype(np.float64) @ np.asarray(down[0], np.float64).T * sa[:, None] * down[1]


def quantize_weights(inp):
    """(codes, scales) of every expert matrix that a workload's inputs hold."""
    names = ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")
    return {n: _Lazy(inp[n]) if n.startswith("w_") else quantize(oracle.widen_bf16(inp[n]))
            for n in names if inp.get(n) is not None}


class _Lazy:
    """Stacked matrices, each quantised when it is first asked for."""

    def __init__(self, src):
        self.src, self.cache = src, {}

    def __getitem__(self, e):
        if e not in self.cache:
            self.cache[e] = quantize(oracle.widen_bf16(self.src[e]))
        return self.cache[e]


def experts_sorted(hidden, q, perm, offsets, top_k):
    x = oracle.widen_bf16(hidden)
    y = np.zeros((len(perm), x.shape[1]))
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi] = ffn(x[np.asarray(perm[lo:hi], np.int64) // top_k], *(q[n][e] for n in ("w_gate", "w_up", "w_down")))
    return y


def shared(hidden, q):
    return ffn(oracle.widen_bf16(hidden), q["ws_gate"], q["ws_up"], q["ws_down"])


def layer(w, inp, q, topk_idx=None, rows=None):
    """The layer of a workload (or of some of its tokens), with the oracle's routing or a given selection."""
    hidden = inp["hidden"] if rows is None else inp["hidden"][rows]
    logits = oracle.router_logits(hidden, inp["router_w"])
    r = (oracle.route_sigmoid(logits, inp["bias"], w.top_k, w.route_scale) if w.score_mode == "sigmoid"
         else oracle.route_softmax(logits, w.top_k, w.renorm_eps))
    idx, wt = r["idx"], r["w"]
    if topk_idx is not None:
        idx = np.asarray(topk_idx, np.int32)
        wt = oracle.routing_weights_for(r["scores"], idx, w.score_mode, w.route_scale, w.renorm_eps)
    counts, offsets = oracle.histogram_offsets(idx, w.E)
    perm, inv = oracle.permutation(idx, w.E)
    y = experts_sorted(hidden, q, perm, offsets, w.top_k)
    z = shared(hidden, q) if w.has_shared else None
    return {**r, "idx": idx, "w": wt, "perm": perm, "inv": inv, "offsets": offsets, "y_sorted": y, "z": z,
            "out": oracle.combine(y, inv, wt, z)}
