"""moe_workspace_bytes on the host: it covers the one-kernel forms' pieces, and a
workspace made for a batch serves every smaller batch of the same layer."""
import ctypes
import random

import pytest

import __graft_entry__
import expert_ffn_layer_gb300 as moe

G = 0x100000  # an aligned address that is never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    moe._lib = None  # another file reloads the module: take its current struct classes
    return moe.load()


def _up(n):
    return (n + 255) // 256 * 256


SHAPES = [dict(H=4096, E=192, I=1536, k=8), dict(H=4096, E=64, I=2048, k=8), dict(H=2048, E=4, I=1024, k=4),
          dict(H=256, E=256, I=128, k=1), dict(H=16384, E=22, I=128, k=1), dict(H=1024, E=2, I=16384, k=2),
          dict(H=128, E=8, I=128, k=2, Is=8192), dict(H=192, E=16, I=64, k=3, Is=0)]


def _dims(T, H, E, I, k, Is=None):
    return moe.dims(T, H, E, I, k, I_shared=I if Is is None else Is, has_shared=Is != 0)


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: "-".join(str(v) for v in s.values()))
def test_workspace_does_not_fall_as_the_batch_grows(lib, s):
    rng = random.Random(0)
    Ts = sorted({*range(0, 300), 511, 512, 513, *(b + d for i in range(6) for b in [1024 << i] for d in (-1, 0, 1, 129)),
                 *(rng.randint(300, 40000) for _ in range(200))})
    sizes = [moe.moe_workspace_bytes(_dims(T, **s)) for T in Ts]
    for a, b, ta, tb in zip(sizes, sizes[1:], Ts, Ts[1:]):
        assert a <= b, f"T = {ta}: {a}, T = {tb}: {b}"


def _few_layer_bytes(T, H, E, I, k, Is):
    """The one-kernel layer's pieces behind the 4 KiB header: logits, fp16 hidden and its scales, activations in
    fp32 and in fp16 with their exponents, outputs in fp32."""
    n_act = T * k * I + T * Is
    return 4096 + sum(map(_up, (T * E * 4, T * H * 2, T * 4, n_act * 4, n_act * 2, n_act // 32, (T * k + T) * H * 4)))


@pytest.mark.parametrize("T", [1, 8, 32])
@pytest.mark.parametrize("s", [dict(H=2048, E=4, I=1024, k=4, Is=1024), dict(H=1024, E=2, I=16384, k=2, Is=128)],
                         ids=["narrow", "wide"])
def test_workspace_covers_the_one_kernel_layer_where_it_needs_more(lib, s, T):
    """Few experts and wide ones, so that these pieces and not the chain's set the size; a byte less is refused."""
    d, need = _dims(T, **s), _few_layer_bytes(T, **s)
    assert moe.moe_workspace_bytes(d) >= need
    ref = ctypes.byref
    ex = moe.MoeMxfp4Experts(**{n: G for n, _ in moe.MoeMxfp4Experts._fields_})
    assert lib.moe_layer_forward_few(ref(d), *([G] * 11), need - 1, None) == 3
    assert lib.moe_layer_forward_mxfp4(ref(d), G, G, None, ref(ex), G, G, need - 1, None) == 3
    assert lib.moe_expert_ffn_mxfp4(ref(d), G, G, G, ref(ex), G, G, G, need - 1, None) == 3


@pytest.mark.parametrize("T", [33, 100, 256])
def test_workspace_covers_the_one_kernel_expert_ffn(lib, T):
    """Past 32 tokens: the chain's outputs (kept for the combine) and behind them the FFN's own pieces."""
    s = dict(H=16384, E=22, I=128, k=1, Is=128)
    d, n_act = _dims(T, **s), 2 * T * 128
    need = 4096 + 2 * T * 16384 * 2 + n_act * 2 + T * 16384 * 2 + T * 4 + n_act // 32  # outputs, activations, hidden
    assert moe.moe_workspace_bytes(d) >= need
    ex = moe.MoeMxfp4Experts(**{n: G for n, _ in moe.MoeMxfp4Experts._fields_})
    assert lib.moe_expert_ffn_mxfp4(ctypes.byref(d), G, G, G, ctypes.byref(ex), G, G, G, need, None) == 3
