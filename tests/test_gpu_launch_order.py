"""moe_fused_moe right behind kernels of this library that let the next one launch
while they still write: what its early tiles read (hidden, the shared expert's
weights) and count with (the workspace header) has to be complete.  Every sequence
is run once with a synchronize between its calls and then many times without; the
bits have to be the same."""
import pytest
import torch

import expert_ffn_layer_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _normal(gen, shape, sigma):
    return (torch.randn(shape, device="cuda", generator=gen) * sigma).bfloat16()


class Layer:
    def __init__(self, T, H, E, k, I, Is, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.gen = gen
        self.d = moe.dims(T, H, E, I, k, I_shared=Is, score_mode="softmax", route_scale=1.0)
        self.hidden = _normal(gen, (T, H), 1.0)
        self.gu, self.down = _normal(gen, (E, 2 * I, H), 0.02), _normal(gen, (E, H, I), 0.02)
        self.sgu, self.sdown = _normal(gen, (2 * Is, H), 0.02), _normal(gen, (H, Is), 0.02)
        self.idx = torch.stack([torch.randperm(E, device="cuda", generator=gen)[:k] for _ in range(T)]).int()
        self.w = torch.full((T, k), 1.0 / k, device="cuda")
        self.ws = moe.alloc_workspace(self.d)

    def fused(self, hidden, out):
        moe.moe_fused_moe(self.d, hidden, self.idx, self.w, self.gu, self.down, self.sgu, self.sdown, out, self.ws)
        return out

    def new_out(self):
        return torch.empty((self.d.T, self.d.H), dtype=torch.bfloat16, device="cuda")


def _codes(x):
    codes = torch.empty((*x.shape[:-1], x.shape[-1] // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((*x.shape[:-1], x.shape[-1] // 32), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4_rows(x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("T", [8, 1200])  # the permutation in one kernel, and (9600 slots) in two
def test_fused_moe_behind_the_dequantiser(T):
    """The shared expert's stacked weights are expanded from MXFP4 anew before each call, from two sets in turn."""
    a = Layer(T, 1024, 16, 8, 128, 4096)
    sets = [_codes(_normal(a.gen, a.sgu.shape, 0.02)) for _ in range(2)]
    ref = []
    for s in sets:
        moe.moe_dequantize_mxfp4_rows(*s, a.sgu)
        torch.cuda.synchronize()
        ref.append(a.fused(a.hidden, a.new_out()))
        torch.cuda.synchronize()
    assert not torch.equal(ref[0], ref[1])
    outs = [a.new_out() for _ in range(40)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        moe.moe_dequantize_mxfp4_rows(*sets[i & 1], a.sgu)
        a.fused(a.hidden, o)
    torch.cuda.synchronize()
    assert moe.moe_ws_read_error(a.ws) == 0
    for i, o in enumerate(outs):
        assert torch.equal(o, ref[i & 1]), f"call {i}"


@pytest.mark.parametrize("T", [8, 2048])
def test_fused_moe_behind_its_own_combine(T):
    """Layer after layer: each call's output, written by its combine, is the next one's hidden state."""
    a = Layer(T, 1024, 16, 4, 128, 1024)
    n = 3  # the outputs shrink from layer to layer
    ref, x = [], a.hidden
    for _ in range(n):
        x = a.fused(x, a.new_out())
        torch.cuda.synchronize()
        ref.append(x)
    assert all(float(r.abs().max()) > 0 for r in ref)
    for _ in range(15):
        outs = [a.new_out() for _ in range(n)]
        torch.cuda.synchronize()
        x = a.hidden
        for o in outs:
            x = a.fused(x, o)
        torch.cuda.synchronize()
        assert moe.moe_ws_read_error(a.ws) == 0
        for i, o in enumerate(outs):
            assert torch.equal(o, ref[i]), f"layer {i}"


@pytest.mark.parametrize("T", [8, 512])
def test_fused_moe_behind_an_expert_ffn_on_the_same_workspace(T):
    """Both claim tiles from the header's counter and keep activations in the workspace."""
    a = Layer(T, 1024, 16, 4, 256, 1024)
    d, E, I, Is = a.d, 16, 256, 1024
    gate, up = a.gu[:, :I].contiguous(), a.gu[:, I:].contiguous()
    sgate, sup = a.sgu[:Is].contiguous(), a.sgu[Is:].contiguous()
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    perm, inv = (torch.empty(T * 4, dtype=torch.int32, device="cuda") for _ in range(2))
    moe.moe_permute(d, a.idx, counts, offsets, perm, inv, a.ws)
    y = torch.empty((T * 4, 1024), dtype=torch.bfloat16, device="cuda")
    z = a.new_out()

    def ffn():
        moe.moe_expert_ffn(d, a.hidden, perm, offsets, gate, up, a.down, sgate, sup, a.sdown, y, z, a.ws)

    ffn()
    torch.cuda.synchronize()
    ref_y, ref_z = y.clone(), z.clone()
    ref = a.fused(a.hidden, a.new_out())
    torch.cuda.synchronize()
    outs = [a.new_out() for _ in range(30)]
    torch.cuda.synchronize()
    for o in outs:
        ffn()
        a.fused(a.hidden, o)
    torch.cuda.synchronize()
    assert moe.moe_ws_read_error(a.ws) == 0
    assert torch.equal(y, ref_y) and torch.equal(z, ref_z)
    assert all(torch.equal(o, ref) for o in outs)
    assert int(a.ws[:4096].sum()) == 0


def test_fused_moe_behind_the_dequantiser_in_a_graph():
    a = Layer(8, 1024, 16, 4, 128, 4096)
    sets = [_codes(_normal(a.gen, a.sgu.shape, 0.02)) for _ in range(2)]
    ref = []
    for s in sets:
        moe.moe_dequantize_mxfp4_rows(*s, a.sgu)
        torch.cuda.synchronize()
        ref.append(a.fused(a.hidden, a.new_out()))
        torch.cuda.synchronize()
    outs = [a.new_out() for _ in range(16)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i, o in enumerate(outs):
            moe.moe_dequantize_mxfp4_rows(*sets[i & 1], a.sgu)
            a.fused(a.hidden, o)
    for _ in range(5):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert torch.equal(o, ref[i & 1]), f"call {i}"
