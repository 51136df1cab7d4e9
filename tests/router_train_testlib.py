"""The router's losses and the backward passes of routing and combine in float64
numpy, from their definitions, for the tests of moe_balance_loss, moe_route_backward
and moe_combine_backward.  Counts are constants of the losses' gradients."""
import numpy as np


def counts_of(idx, seq, n_seq, E):
    counts, tokens = np.zeros((n_seq, E), np.int64), np.zeros(n_seq, np.int64)
    for t, b in enumerate(seq):
        if 0 <= b < n_seq:
            tokens[b] += 1
            for e in idx[t]:
                counts[b, e] += 1
    return counts, tokens


def sigmoid(l):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-l))


def softmax(l):
    e = np.exp(l - l.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def lse_of(l):
    m = l.max(-1)
    return m + np.log(np.exp(l - m[..., None]).sum(-1))


def losses(l, counts, tokens, seq, mode, k):
    """(balance, z) over the tokens of sequences in [0, n_seq)."""
    n_seq, E = counts.shape
    q = softmax(l) if mode == "softmax" else sigmoid(l) / sigmoid(l).sum(-1, keepdims=True)
    per = [(counts[b] * E / (k * tokens[b])) @ q[seq == b].mean(0) for b in range(n_seq) if tokens[b]]
    live = (seq >= 0) & (seq < n_seq)
    return (np.mean(per) if per else 0.0), (np.square(lse_of(l[live])).mean() if live.any() else 0.0)


def weights(l, idx, mode, scale, eps):
    """The combine weights of a given selection."""
    s = softmax(l) if mode == "softmax" else sigmoid(l)
    sel = np.take_along_axis(s, idx, 1)
    total = sel.sum(-1, keepdims=True)
    return sel / np.maximum(total, eps) if mode == "softmax" else sel / total * scale


def grad_logits(l, idx, seq, n_seq, mode, *, scale=1.0, eps=0.0, grad_w=None, grad_losses=None, counts=None, tokens=None):
    """The gradient, and a bound's magnitudes: the sum of what is added and subtracted in each element, with every
    exponential's argument (at most the logits' range R) and lse's own size taken into account."""
    T, E = l.shape
    k = idx.shape[1]
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        b = seq[t]
        if not 0 <= b < n_seq:
            continue
        p, s = softmax(l[t]), sigmoid(l[t])
        miss = sigmoid(-l[t])
        if grad_losses is not None:
            full, n = (tokens > 0).sum(), tokens.sum()
            F = counts[b] * E / (k * float(tokens[b]) ** 2 * full)
            q, slope = (p, np.ones(E)) if mode == "softmax" else (s / s.sum(), miss)
            d[t] += grad_losses[0] * q * slope * (F - F @ q)
            mag[t] += abs(grad_losses[0]) * q * slope * (F + F @ q)
            lse = lse_of(l[t])
            d[t] += grad_losses[1] * 2 * lse / n * p
            mag[t] += abs(grad_losses[1]) * 2 * (abs(l[t].max()) + np.log(E) + 1) / n * p
        if grad_w is not None:
            g, e = grad_w[t], idx[t]
            if mode == "softmax":
                total = p[e].sum()
                if total >= eps:
                    u = p[e] / total
                    v, m = u * (g - g @ u), u * (abs(g) + abs(g) @ u)
                else:
                    v, m = g / eps * p[e], abs(g) / eps * p[e]
                    d[t] -= p * v.sum()
                    mag[t] += p * m.sum()
            else:
                u = s[e] / s[e].sum()
                v, m = scale * u * (g - g @ u) * miss[e], abs(scale) * u * (abs(g) + abs(g) @ u) * miss[e]
            np.add.at(d[t], e, v)
            np.add.at(mag[t], e, m)
    return d, mag
