"""Host-side checks of the router's losses and backward entries that need no GPU:
refusals before any launch, and the binding's checks."""
import ctypes

import pytest
import torch

import __graft_entry__
import expert_ffn_layer_gb300 as moe

G = 0x100000  # an aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    moe._lib = None  # another file reloads the module: take its current struct classes
    return moe.load()


def test_balance_loss_refusals(lib):
    d, ref = moe.dims(8, 256, 16, 128, 4), ctypes.byref
    call = lambda *a: lib.moe_balance_loss(ref(d), *a)  # noqa: E731  logits, idx, seq_id, n_seq, counts, tokens, losses, ws
    assert call(None, G, None, 1, G, G, G, G, BIG, None) == 1      # losses without logits
    assert call(G, None, None, 1, G, G, G, G, BIG, None) == 1
    assert call(G, G, None, 1, None, G, G, G, BIG, None) == 1
    assert call(G, G, None, 1, G, None, G, G, BIG, None) == 1
    assert call(G, G, None, 2, G, G, G, G, BIG, None) == 1         # several sequences without seq_id
    assert call(G, G, G, 0, G, G, G, G, BIG, None) == 1
    assert call(G, G, G + 4, 2, G, G, G, G, BIG, None) == 1
    assert call(G, G, G, 65537, G, G, G, G, BIG, None) == 2
    assert call(G, G, None, 1, G, G, G + 2, G, BIG, None) == 1     # losses' alignment
    assert call(G + 4, G, None, 1, G, G, G, G, BIG, None) == 1
    assert call(G, G, None, 1, G, G, G, None, BIG, None) == 1
    assert call(G, G, None, 1, G, G, G, G, 4096, None) == 3
    bad = moe.dims(8, 256, 300, 128, 4)
    assert lib.moe_balance_loss(ref(bad), G, G, None, 1, G, G, G, G, BIG, None) == 2


def test_route_backward_refusals(lib):
    d, ref = moe.dims(8, 256, 16, 128, 4), ctypes.byref
    names = ("hidden", "router_w", "logits", "topk_idx", "grad_topk_w", "seq_id", "n_seq", "counts", "tokens", "grad_losses",
             "grad_logits", "grad_hidden", "grad_router_w", "ws", "ws_bytes", "stream")
    good = dict.fromkeys(names, G)
    good.update(seq_id=None, n_seq=1, ws_bytes=BIG, stream=None)

    def call(dims=d, **over):
        return lib.moe_route_backward(ref(dims), *({**good, **over}[n] for n in names))

    for n in ("hidden", "router_w", "logits", "topk_idx", "counts", "tokens", "ws"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: G + 4}) == 1, n
    assert call(grad_logits=None, grad_hidden=None, grad_router_w=None) == 1
    assert call(grad_topk_w=None, grad_losses=None) == 1
    for n in ("grad_topk_w", "grad_logits", "grad_hidden", "grad_router_w", "seq_id"):
        assert call(**{n: G + 4}) == 1, n
    assert call(grad_losses=G + 2) == 1
    assert call(n_seq=2) == 1 and call(seq_id=G, n_seq=0) == 1
    assert call(seq_id=G, n_seq=65537) == 2
    assert call(ws_bytes=4096) == 3
    empty = moe.dims(0, 256, 16, 128, 4)
    assert call(empty, grad_router_w=None, **dict.fromkeys(("hidden", "logits", "topk_idx", "ws"))) == 0


def test_combine_backward_refusals(lib):
    d, ref = moe.dims(8, 256, 16, 128, 4), ctypes.byref
    good = [G] * 6  # grad_out, y_sorted, inv_perm, topk_w, grad_topk_w, grad_y_sorted
    for at in range(4):
        for bad in (None, G + 4):
            args = list(good)
            args[at] = bad
            assert lib.moe_combine_backward(ref(d), *args, None) == 1, at
    assert lib.moe_combine_backward(ref(d), G, G, G, G, None, None, None) == 1
    assert lib.moe_combine_backward(ref(d), G, G, G, G, G + 4, G, None) == 1
    assert lib.moe_combine_backward(ref(d), G, G, G, G, G, G + 4, None) == 1
    assert lib.moe_combine_backward(ref(moe.dims(0, 256, 16, 128, 4)), *[None] * 6, None) == 0


def test_binding_checks():
    d = moe.dims(4, 64, 4, 64, 2)
    l, idx, ws = torch.zeros(4, 4), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(8, dtype=torch.uint8)
    tokens, counts = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="n_seq"):
        moe.moe_route_backward(d, l, idx, ws, grad_w=torch.zeros(4, 2), seq_id=torch.zeros(4, dtype=torch.int32), grad_logits=l)
    with pytest.raises(ValueError, match="counts"):
        moe.moe_balance_loss(d, l, idx, counts[:2], tokens, torch.zeros(2), ws)
    with pytest.raises(TypeError, match="seq_id"):
        moe.moe_balance_loss(d, l, idx, counts, tokens, torch.zeros(2), ws, seq_id=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError, match="grad_router_w"):
        moe.moe_route_backward(d, l, idx, ws, grad_w=torch.zeros(4, 2), grad_router_w=torch.zeros((4, 64), dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="grad_y_sorted"):
        moe.moe_combine_backward(d, torch.zeros((4, 64), dtype=torch.bfloat16), None, torch.zeros(8, dtype=torch.int32),
                                 torch.zeros(4, 2), grad_y_sorted=torch.zeros(8, 64))
