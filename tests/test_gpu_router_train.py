"""The router's losses and the backward passes of routing and combine on the GPU,
against the float64 reference.

Tolerances.  u = 2^-24 is fp32's rounding.  A logit's gradient is formed from
exponentials of arguments up to the logits' range R (off by R u and 2 units each),
sums of at most 256 terms in trees (13 additions), and about ten further roundings:
(64 + 4 R) u of the magnitudes that are added in it.  The losses likewise."""
import numpy as np
import pytest
import torch

import expert_ffn_layer_gb300 as moe
import router_train_testlib as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dims(T, E, k, mode, H=64, eps=1e-8):
    return moe.dims(T, H, E, 64, k, score_mode=mode, route_scale=2.826 if mode == "sigmoid" else 1.0,
                    renorm_eps=0.0 if mode == "sigmoid" else eps)


class Case:
    def __init__(self, T, E, k, mode, n_seq=1, pad=0.0, H=64, spread=1.3, eps=1e-8, sort=True, seed=0, seqs=None):
        rng = self.rng = np.random.default_rng(1000 * T + 10 * E + k + seed)
        self.mode, self.n_seq, self.k, self.eps = mode, n_seq, k, eps
        self.d = dims(T, E, k, mode, H, eps)
        self.logits = (rng.normal(size=(T, E)) * spread).astype(np.float32)
        self.idx = np.argsort(-(self.logits + rng.normal(size=(T, E)) * 0.1), 1, kind="stable")[:, :k].astype(np.int32)
        seq = rng.integers(0, n_seq, T) if seqs is None else np.asarray(seqs)
        self.seq = (np.sort(seq) if sort else seq).astype(np.int32)
        if pad:
            self.seq[rng.random(T) < pad] = -1
        self.grad_w = rng.normal(size=(T, k)).astype(np.float32)
        self.grad_losses = np.array([0.01, 0.001], np.float32) * T
        self.ws = moe.alloc_workspace(self.d)
        self.counts, self.tokens = ref.counts_of(self.idx.clip(0, E - 1), self.seq, n_seq, E)

    def dev(self, name):
        return torch.from_numpy(np.ascontiguousarray(getattr(self, name))).cuda()

    def seq_dev(self):
        return self.dev("seq")

    def balance(self, losses=True):
        d = self.d
        counts = torch.full((self.n_seq, d.E), -7, dtype=torch.int32, device="cuda")
        tokens = torch.full((self.n_seq,), -7, dtype=torch.int32, device="cuda")
        out = torch.full((2,), float("nan"), device="cuda") if losses else None
        moe.moe_balance_loss(d, self.dev("logits"), self.dev("idx"), counts, tokens, out, self.ws, seq_id=self.seq_dev())
        torch.cuda.synchronize()
        return counts, tokens, out

    def backward(self, w=True, loss=True, hidden=None, router_w=None, **kw):
        d = self.d
        new = lambda *s, dtype=torch.float32: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        out = dict(grad_logits=new(d.T, d.E))
        if router_w is not None:
            out["grad_hidden"] = new(d.T, d.H, dtype=torch.bfloat16)
        if hidden is not None:
            out["grad_router_w"] = new(d.E, d.H)
        args = dict(hidden=hidden, router_w=router_w, seq_id=self.seq_dev(), n_seq=self.n_seq, **out)
        if w:
            args["grad_w"] = self.dev("grad_w")
        if loss:
            args.update(grad_losses=self.dev("grad_losses"), counts=torch.from_numpy(self.counts).int().cuda(),
                        tokens=torch.from_numpy(self.tokens).int().cuda())
        moe.moe_route_backward(d, self.dev("logits"), self.dev("idx"), self.ws, **args, **kw)
        torch.cuda.synchronize()
        return out

    def want(self, w=True, loss=True):
        l = self.logits.astype(np.float64)
        d, mag = ref.grad_logits(l, self.idx, self.seq, self.n_seq, self.mode, scale=np.float64(np.float32(2.826)),
                                 eps=np.float64(np.float32(self.eps)),
                                 grad_w=self.grad_w.astype(np.float64) if w else None,
                                 grad_losses=self.grad_losses.astype(np.float64) if loss else None,
                                 counts=self.counts, tokens=self.tokens)
        live = l[(self.seq >= 0) & (self.seq < self.n_seq)]
        live = live[np.isfinite(live)]
        R = float(np.abs(live).max() * 2) if live.size else 0.0
        return d, (64 + 4 * R) * U * mag + 1e-37


CASES = [dict(T=1, E=1, k=1), dict(T=1, E=192, k=8), dict(T=2, E=33, k=16), dict(T=8, E=192, k=8, n_seq=3),
         dict(T=257, E=256, k=16, n_seq=5, pad=0.2), dict(T=300, E=40, k=5, n_seq=64, pad=0.5, sort=False),
         dict(T=63, E=64, k=8, spread=12.0), dict(T=1500, E=31, k=3, n_seq=9, pad=0.1),
         dict(T=100, E=7, k=7, n_seq=200), dict(T=50, E=100, k=1, pad=0.9, n_seq=2)]
IDS = lambda c: "-".join(f"{k}{v}" for k, v in c.items())  # noqa: E731


# more choices, and more counters, than one cluster counts
MANY = [dict(T=9000, E=16, k=8, n_seq=3, pad=0.1), dict(T=300, E=200, k=8, n_seq=60), dict(T=8500, E=8, k=8, sort=False, n_seq=5)]


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("c", CASES + MANY, ids=IDS)
def test_balance_loss(c, mode):
    a = Case(mode=mode, **c)
    counts, tokens, out = a.balance()
    assert np.array_equal(counts.cpu().numpy(), a.counts) and np.array_equal(tokens.cpu().numpy(), a.tokens)
    l = a.logits.astype(np.float64)
    b, z = ref.losses(l, a.counts, a.tokens, a.seq, mode, a.k)
    R = 2 * np.abs(l).max()
    got = out.cpu().numpy().astype(np.float64)
    assert abs(got[0] - b) <= (64 + 4 * R) * U * b + 1e-37
    assert abs(got[1] - z) <= (64 + 4 * R) * U * (np.abs(l).max() + np.log(c["E"]) + 1) ** 2
    assert moe.moe_ws_read_error(a.ws) == 0
    again = a.balance()
    assert torch.equal(again[2], out)
    only = a.balance(losses=False)
    assert torch.equal(only[0], counts) and torch.equal(only[1], tokens)


@pytest.mark.parametrize("parts", ["both", "weights", "losses"])
@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_grad_logits(c, mode, parts):
    a = Case(mode=mode, **c)
    on = dict(w=parts != "losses", loss=parts != "weights")
    got = a.backward(**on)["grad_logits"].cpu().numpy().astype(np.float64)
    d, tol = a.want(**on)
    assert (np.abs(got - d) <= tol).all(), np.abs(got - d).max()
    assert not got[a.seq < 0].any()
    assert moe.moe_ws_read_error(a.ws) == 0


def test_clamped_sum():
    """renorm_eps above the selected probabilities of some tokens: weights p / eps, whose gradient reaches every expert."""
    a = Case(T=200, E=24, k=3, mode="softmax", eps=0.6, spread=1.5)
    p = np.take_along_axis(ref.softmax(a.logits.astype(np.float64)), a.idx.astype(np.int64), 1).sum(-1)
    assert (p < 0.59).sum() > 20 and (p > 0.61).sum() > 20 and not (abs(p - 0.6) < 1e-5).any()
    got = a.backward()["grad_logits"].cpu().numpy().astype(np.float64)
    d, tol = a.want()
    assert (np.abs(got - d) <= tol).all()


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
def test_masked_experts_and_saturated_logits(mode):
    """Experts shut out by a logit of -infinity or of the type's lowest value, and logits far from zero."""
    a = Case(T=40, E=48, k=4, mode=mode, spread=1.0)
    a.logits[:, 5] = -np.inf
    a.logits[:, 9] = -1e30
    a.logits[:, 11] = np.finfo(np.float32).min
    a.logits[3:6] += 60.0
    a.logits[7, :4] = 80.0
    a.logits[8, 10] = -60.0
    order = np.argsort(-a.logits, 1, kind="stable")
    a.idx = order[:, :4].astype(np.int32)
    a.counts, a.tokens = ref.counts_of(a.idx, a.seq, 1, 48)
    with np.errstate(over="ignore"):
        d, _ = a.want()
    got = a.backward()["grad_logits"].cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    # the logits' range here is 140: (64 + 4 * 140) u of the row's largest magnitude
    top = np.abs(d).max(-1, keepdims=True)
    assert (np.abs(got - d) <= 1000 * U * (top + 1)).all()
    assert not got[:, 5].any()


def test_padding_is_not_read():
    """NaN and infinities in padded tokens' logits and hidden rows, weights' gradients among them: zeros come out, and
    every other output keeps its bits."""
    a = Case(T=130, E=40, k=4, mode="sigmoid", n_seq=3, pad=0.3, H=192)
    gen = torch.Generator(device="cuda").manual_seed(1)
    hidden = torch.randn((130, 192), device="cuda", generator=gen).bfloat16()
    router_w = torch.randn((40, 192), device="cuda", generator=gen) * 0.02
    clean_loss, clean = a.balance(), a.backward(hidden=hidden, router_w=router_w)
    off = a.seq < 0
    a.logits[off] = np.nan
    a.logits[off, 3] = np.inf
    a.grad_w[off] = np.nan
    hidden[torch.from_numpy(off).cuda()] = float("nan")
    hidden[int(np.nonzero(off)[0][0]), 0] = float("inf")
    loss, got = a.balance(), a.backward(hidden=hidden, router_w=router_w)
    assert torch.equal(loss[2], clean_loss[2])
    for n in clean:
        assert torch.equal(got[n], clean[n]), n
    assert not got["grad_hidden"][torch.from_numpy(off).cuda()].any()


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
def test_all_padding_and_no_tokens(mode):
    a = Case(T=5, E=8, k=2, mode=mode, seqs=[-1, -3, -1, -1, -2147483648], n_seq=2, sort=False)
    counts, tokens, out = a.balance()
    assert not counts.any() and not tokens.any() and out.tolist() == [0.0, 0.0]
    h, w = torch.ones((5, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((8, 64), device="cuda")
    for v in a.backward(hidden=h, router_w=w).values():
        assert not v.any()
    d = dims(0, 8, 2, mode)
    counts, tokens = torch.ones((2, 8), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    losses, gw = torch.ones(2, device="cuda"), torch.ones((8, 64), device="cuda")
    none = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    ws = moe.alloc_workspace(dims(1, 8, 2, mode))
    moe.moe_balance_loss(d, none(0, 8), none(0, 2, t=torch.int32), counts, tokens, losses, ws, seq_id=none(0, t=torch.int32))
    moe.moe_route_backward(d, none(0, 8), none(0, 2, t=torch.int32), ws, grad_w=none(0, 2), grad_router_w=gw,
                           hidden=none(0, 64, t=torch.bfloat16))
    torch.cuda.synchronize()
    assert not counts.any() and not tokens.any() and not losses.any() and not gw.any()


def test_an_expert_named_twice_counts_twice():
    a = Case(T=30, E=9, k=3, mode="sigmoid")
    a.idx[:, 2] = a.idx[:, 0]
    a.counts, a.tokens = ref.counts_of(a.idx, a.seq, 1, 9)
    counts, _, _ = a.balance()
    assert np.array_equal(counts.cpu().numpy(), a.counts)
    d, tol = a.want()
    assert (np.abs(a.backward()["grad_logits"].cpu().numpy() - d) <= tol).all()


def test_bad_indices_are_clamped_and_flagged():
    for field, value in (("idx", -1), ("idx", 12), ("seq", 3)):
        a = Case(T=20, E=12, k=2, mode="softmax", n_seq=3)
        if field == "idx":
            a.idx[7, 1] = value
            a.counts, a.tokens = ref.counts_of(a.idx.clip(0, 11), a.seq, 3, 12)
        else:
            a.seq[7] = value
            a.counts, a.tokens = ref.counts_of(a.idx, a.seq, 3, 12)
        counts, tokens, out = a.balance()
        assert np.array_equal(counts.cpu().numpy(), a.counts) and np.array_equal(tokens.cpu().numpy(), a.tokens)
        assert moe.moe_ws_read_error(a.ws, clear=True) == moe.DEVERR_INDEX
        got = a.backward()["grad_logits"].cpu().numpy()
        assert moe.moe_ws_read_error(a.ws, clear=True) == moe.DEVERR_INDEX
        if field == "idx":
            a.idx = a.idx.clip(0, 11)
        d, tol = a.want()
        assert (np.abs(got - d) <= tol).all()


PRODUCTS = [dict(T=1, E=1, k=1, H=64), dict(T=1, E=192, k=8, H=4096), dict(T=8, E=192, k=8, H=1024),
            dict(T=127, E=40, k=5, H=1088, n_seq=3, pad=0.3), dict(T=129, E=64, k=8, H=128),
            dict(T=300, E=256, k=16, H=320, n_seq=2), dict(T=513, E=17, k=2, H=192, pad=0.5, n_seq=40),
            dict(T=640, E=255, k=3, H=704), dict(T=1300, E=130, k=4, H=256, pad=0.1), dict(T=40, E=2, k=1, H=16384),
            dict(T=2100, E=33, k=3, H=128, n_seq=3, pad=0.05), dict(T=100, E=20, k=2, H=64, n_seq=2, pad=0.2),
            dict(T=17, E=192, k=8, H=192), dict(T=16, E=256, k=16, H=64, n_seq=3, pad=0.3)]


@pytest.mark.parametrize("c", PRODUCTS, ids=IDS)
def test_grad_hidden_and_router_w(c):
    """The products with the logits' gradient that the call itself returns.  grad_hidden: a bf16 rounding (2^-8), and
    the factors taken as two bf16 pieces or better (2^-16 each, 2^-15 with what is left out) and summed in fp32: 2^-14
    of the magnitudes.  grad_router_w: factors exact, fp32 sums of at most 2 + T / 16 steps for each of three pieces
    that round by 2^-23 of the sum so far or better."""
    a = Case(mode="sigmoid", **c)
    T, H, E = c["T"], c["H"], c["E"]
    gen = torch.Generator(device="cuda").manual_seed(T)
    hidden = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    router_w = torch.randn((E, H), device="cuda", generator=gen) * 0.02
    got = a.backward(hidden=hidden, router_w=router_w)
    dl = got["grad_logits"].double()
    want, mag = dl @ router_w.double(), dl.abs() @ router_w.double().abs()
    assert ((got["grad_hidden"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * mag + 1e-37).all()
    want, mag = dl.T @ hidden.double(), dl.T.abs() @ hidden.double().abs()
    steps = 3 * (2 + T / 16) + 16
    assert ((got["grad_router_w"].double() - want).abs() <= steps * 2.0 ** -23 * mag + 1e-37).all()
    # in the mean far less: errors of the steps are independent
    err = (got["grad_router_w"].double() - want).norm() / want.norm().clamp(min=1e-300)
    assert err <= 4e-6, err
    again = a.backward(hidden=hidden, router_w=router_w)
    for n in got:
        assert torch.equal(got[n], again[n]), n
    one = a.backward(hidden=hidden)
    assert torch.equal(one["grad_router_w"], got["grad_router_w"])
    two = a.backward(router_w=router_w)
    assert torch.equal(two["grad_hidden"], got["grad_hidden"])


def test_more_tokens_than_one_pass():
    """grad_router_w over several rounds of both accumulators and grad_hidden over several token tiles a CTA: sums and
    rows far from the first, with padding in between."""
    c = dict(T=5000, E=72, k=4, H=8192, n_seq=4, pad=0.05)
    a = Case(mode="softmax", **c)
    gen = torch.Generator(device="cuda").manual_seed(9)
    hidden = torch.randn((5000, 8192), device="cuda", generator=gen).bfloat16()
    router_w = torch.randn((72, 8192), device="cuda", generator=gen) * 0.02
    got = a.backward(hidden=hidden, router_w=router_w)
    dl = got["grad_logits"].double()
    at = torch.cat([torch.arange(0, 40), torch.arange(2040, 2060), torch.arange(4970, 5000)]).cuda()
    want, mag = dl[at] @ router_w.double(), dl[at].abs() @ router_w.double().abs()
    assert ((got["grad_hidden"][at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * mag + 1e-37).all()
    cols = torch.cat([torch.arange(0, 64), torch.arange(8100, 8192)]).cuda()
    x = hidden[:, cols].double()
    want, mag = dl.T @ x, dl.T.abs() @ x.abs()
    # at most 128 tokens, 3 * 8 steps, in an accumulator, then 40 sums in registers and 8 of the cluster
    assert ((got["grad_router_w"][:, cols].double() - want).abs() <= (24 * 2.0 ** -23 + 48 * U) * mag + 1e-37).all()
    assert (got["grad_router_w"][:, cols].double() - want).norm() <= 1e-6 * want.norm()


def test_wide_ranges_of_gradients():
    """Tokens whose gradients differ by many powers of two, and a router weight that does: pieces keep their digits."""
    a = Case(T=64, E=32, k=4, mode="sigmoid", H=128)
    a.grad_w *= (2.0 ** np.linspace(-40, 30, 64)).astype(np.float32)[:, None]
    gen = torch.Generator(device="cuda").manual_seed(2)
    hidden = torch.randn((64, 128), device="cuda", generator=gen).bfloat16()
    router_w = torch.randn((32, 128), device="cuda", generator=gen) * torch.exp2(torch.linspace(-60, 20, 128, device="cuda"))
    got = a.backward(loss=False, hidden=hidden, router_w=router_w)
    dl = got["grad_logits"].double()
    want, mag = dl @ router_w.double(), dl.abs() @ router_w.double().abs()
    assert ((got["grad_hidden"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * mag + 1e-37).all()
    want, mag = dl.T @ hidden.double(), dl.T.abs() @ hidden.double().abs()
    assert ((got["grad_router_w"].double() - want).abs() <= 2.0 ** -18 * mag + 1e-37).all()


COMBINE = [dict(T=1, H=64, k=1), dict(T=13, H=1088, k=6), dict(T=3, H=16384, k=16), dict(T=700, H=192, k=2),
           dict(T=2500, H=128, k=8), dict(T=5, H=4096, k=8), dict(T=9, H=2112, k=7), dict(T=1300, H=1024, k=16), dict(T=9001, H=64, k=1), dict(T=1250, H=1088, k=3), dict(T=1301, H=2048, k=2)]


@pytest.mark.parametrize("c", COMBINE, ids=IDS)
def test_combine_backward(c):
    T, H, k = c["T"], c["H"], c["k"]
    d = moe.dims(T, H, 16, 64, k)
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    g = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    y = torch.randn((T * k, H), device="cuda", generator=gen).bfloat16()
    inv = torch.randperm(T * k, device="cuda", generator=gen).int()
    w = torch.rand((T, k), device="cuda", generator=gen)
    gw, gy = torch.full((T, k), float("nan"), device="cuda"), torch.full_like(y, float("nan"))
    moe.moe_combine_backward(d, g, y, inv, w, gw, gy)
    rows = y.double()[inv.long()].view(T, k, H)
    want, mag = (rows * g.double()[:, None]).sum(-1), (rows * g.double()[:, None]).abs().sum(-1)
    # a thread adds 8 ceil(H / 2048) products at most, or where a warp has a row of at most 2048 values 8 ceil(H / 256),
    # then 13 sums follow
    steps = 8 * ((H + 255) // 256 if H <= 2048 else (H + 2047) // 2048) + 16
    assert ((gw.double() - want).abs() <= steps * U * mag).all()
    expect = torch.empty_like(y)
    expect[inv.long()] = (w[..., None] * g.float()[:, None]).bfloat16().view(T * k, H)
    assert torch.equal(gy, expect)
    gw2, gy2 = torch.empty_like(gw), torch.empty_like(gy)
    moe.moe_combine_backward(d, g, y, inv, None, gw2, None)
    moe.moe_combine_backward(d, g, None, inv, w, None, gy2)
    torch.cuda.synchronize()
    assert torch.equal(gw, gw2) and torch.equal(gy, gy2)


@pytest.mark.parametrize("mode", ["sigmoid", "softmax"])
def test_a_router_step(mode):
    """A step that tunes the router of a layer whose experts are frozen in 8-bit integers, as a program would run it,
    captured into a graph and replayed on another stream: the router weight's gradient against the float64 formula
    (with the experts' outputs as they came) and against differences of the float64 loss along a direction."""
    T, H, E, I, k = 150, 256, 24, 128, 4
    gen = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s, sigma=1.0: torch.randn(s, device="cuda", generator=gen) * sigma  # noqa: E731
    d = moe.dims(T, H, E, I, k, score_mode=mode, route_scale=2.826 if mode == "sigmoid" else 1.0,
                 renorm_eps=0.0 if mode == "sigmoid" else 1e-8)
    hidden, router_w, bias = rnd(T, H).bfloat16(), rnd(E, H, sigma=0.05), rnd(E, sigma=0.01)
    ex = moe.quantize_int8_experts(*(rnd(*s, sigma=0.05).bfloat16() for s in ((E, I, H), (E, I, H), (E, H, I), (I, H), (I, H), (H, I))))
    seq = torch.arange(T, device="cuda").div(40, rounding_mode="floor").int()
    seq[-20:] = -1
    n_seq, coef = 4, torch.tensor([0.02, 0.003], device="cuda") * T
    grad_out = rnd(T, H).bfloat16()
    grad_out[-20:] = 0
    e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    i32, b16 = torch.int32, torch.bfloat16
    ws = moe.alloc_workspace(d)
    idx, w, logits = e(T, k, t=i32), e(T, k), e(T, E)
    cnt, off, perm, inv = e(E, t=i32), e(E + 1, t=i32), e(T * k, t=i32), e(T * k, t=i32)
    y, z, out = e(T * k, H, t=b16), e(T, H, t=b16), e(T, H, t=b16)
    counts, tokens, losses = e(n_seq, E, t=i32), e(n_seq, t=i32), e(2)
    gw, gl, gx, grw = e(T, k), e(T, E), e(T, H, t=b16), e(E, H)

    def step():
        moe.moe_route(d, hidden, router_w, bias, idx, w, ws, logits_out=logits)
        moe.moe_permute(d, idx, cnt, off, perm, inv, ws)
        moe.moe_expert_ffn_int8(d, hidden, perm, off, ex, y, z, ws)
        moe.moe_combine(d, y, z, inv, w, out)
        moe.moe_balance_loss(d, logits, idx, counts, tokens, losses, ws, seq_id=seq)
        moe.moe_combine_backward(d, grad_out, y, inv, w, gw)
        moe.moe_route_backward(d, logits, idx, ws, grad_w=gw, grad_losses=coef, counts=counts, tokens=tokens, seq_id=seq,
                               hidden=hidden, router_w=router_w, grad_logits=gl, grad_hidden=gx, grad_router_w=grw)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (out, losses, counts, tokens, gl, gx, grw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (out, losses, counts, tokens, gl, gx, grw):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (out, losses, counts, tokens, gl, gx, grw)):
        assert torch.equal(a, b)
    assert moe.moe_ws_read_error(ws) == 0

    host = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    x, W, i64, s = host(hidden), host(router_w), idx.cpu().numpy().astype(np.int64), seq.cpu().numpy()
    rows, go = host(y)[inv.cpu().numpy()].reshape(T, k, H), host(grad_out)
    c64, t64 = counts.cpu().numpy().astype(np.int64), tokens.cpu().numpy().astype(np.int64)
    assert np.array_equal(c64, ref.counts_of(i64, s, n_seq, E)[0])
    assert int(cnt.sum()) == T * k
    scale, eps, co = float(np.float32(d.route_scale)), float(np.float32(d.renorm_eps)), host(coef)

    def loss(M):
        l = x @ M.T
        b, zz = ref.losses(l, c64, t64, s, mode, k)
        return co[0] * b + co[1] * zz + (go[:, None] * rows * ref.weights(l, i64, mode, scale, eps)[..., None]).sum()

    dw = (go[:, None] * rows).sum(-1)
    dl, _ = ref.grad_logits(x @ W.T, i64, s, n_seq, mode, scale=scale, eps=eps, grad_w=dw, grad_losses=co, counts=c64, tokens=t64)
    want = dl.T @ x
    # logits are within 1e-5 of their norm (the router's bound), which the scores' slopes pass on: 1e-4 in all
    assert np.linalg.norm(host(grw) - want) <= 1e-4 * np.linalg.norm(want)
    assert np.linalg.norm(host(gx) - dl @ W) <= 4e-3 * np.linalg.norm(dl @ W)
    direction = np.random.default_rng(0).normal(size=W.shape)
    h = 1e-5
    slope = (loss(W + h * direction) - loss(W - h * direction)) / (2 * h)
    assert abs(slope - (want * direction).sum()) <= 1e-6 * np.abs(want * direction).sum()
    assert abs((host(grw) * direction).sum() - slope) <= 1e-4 * np.abs(want * direction).sum()


def test_two_streams_with_their_own_workspaces():
    cases = [Case(T=400, E=64, k=4, mode="softmax", n_seq=5, seed=i) for i in range(2)]
    want = [(c.balance()[2], c.backward()["grad_logits"]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ins = [[c.dev("logits"), c.dev("idx"), c.seq_dev(), c.dev("grad_w"), c.dev("grad_losses")] for c in cases]
    outs = []
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, (l, i, q, g, gl) in zip(cases, streams, ins):
            with torch.cuda.stream(s):
                counts = torch.empty((5, 64), dtype=torch.int32, device="cuda")
                tokens, losses = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
                dl = torch.empty((400, 64), device="cuda")
                moe.moe_balance_loss(c.d, l, i, counts, tokens, losses, c.ws, seq_id=q)
                moe.moe_route_backward(c.d, l, i, c.ws, grad_w=g, grad_losses=gl, counts=counts, tokens=tokens, seq_id=q,
                                       grad_logits=dl)
                outs.append((counts, tokens, losses, dl))
    torch.cuda.synchronize()
    for n, (_, _, losses, dl) in enumerate(outs):
        assert torch.equal(losses, want[n % 2][0]) and torch.equal(dl, want[n % 2][1])
