"""Host-side checks of the 8-bit integer entry points that need no GPU: refusals
before any launch, the struct mirror, the workspace's size and the reference's
quantiser."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import expert_ffn_layer_gb300 as moe
import int8_testlib as ref8
from test_abi_cpu import _c_struct_fields
from test_workspace_cpu import SHAPES, _dims, _up

G = 0x100000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    moe._lib = None  # another file reloads the module: take its current struct classes
    return moe.load()


def _experts(**over):
    return moe.MoeInt8Experts(**{n: over.get(n, G) for n, _ in moe.MoeInt8Experts._fields_})


def test_struct_matches_the_header():
    fields = _c_struct_fields("moe_int8_experts")
    assert [n for n, _ in fields] == [n for n, _ in moe.MoeInt8Experts._fields_]
    assert all(t.endswith("*") for _, t in fields)


def test_quantizer_refusals(lib):
    assert lib.moe_quantize_int8_rows(G, 4, 12, G, G, None) == 1         # cols % 8
    assert lib.moe_quantize_int8_rows(G, -1, 64, G, G, None) == 1
    assert lib.moe_quantize_int8_rows(G, 4, 0, G, G, None) == 1
    assert lib.moe_quantize_int8_rows(G, 1 << 60, 64, G, G, None) == 1   # rows * cols past 64 bits
    assert lib.moe_quantize_int8_rows(None, 4, 64, G, G, None) == 1
    assert lib.moe_quantize_int8_rows(G, 4, 64, G + 8, G, None) == 1
    assert lib.moe_quantize_int8_rows(G, 4, 64, G, G + 2, None) == 1
    assert lib.moe_quantize_int8_rows(None, 0, 64, None, None, None) == 0
    assert lib.moe_dequantize_int8_rows(G, G, 4, 20, G, None) == 1
    assert lib.moe_dequantize_int8_rows(G, None, 4, 64, G, None) == 1
    assert lib.moe_dequantize_int8_rows(G, G, 4, 64, G + 4, None) == 1
    assert lib.moe_dequantize_int8_rows(None, None, 0, 64, None, None) == 0


def test_layer_refusals(lib):
    d, ref = moe.dims(8, 256, 16, 128, 4), ctypes.byref
    ex, big = _experts(), 1 << 40
    assert lib.moe_layer_forward_int8(ref(d), None, None, None, None, None, None, 0, None) == 1
    assert lib.moe_expert_ffn_int8(ref(d), G, G, G, None, G, G, G, big, None) == 1
    for n, _ in moe.MoeInt8Experts._fields_:  # every array has to be there and aligned
        for bad in (None, G + 4):
            assert lib.moe_expert_ffn_int8(ref(d), G, G, G, ref(_experts(**{n: bad})), G, G, G, big, None) == 1, n
    for at in range(3):  # hidden, perm, offsets
        args = [G, G, G]
        args[at] = None
        assert lib.moe_expert_ffn_int8(ref(d), *args, ref(ex), G, G, G, big, None) == 1
    assert lib.moe_expert_ffn_int8(ref(d), G, G, G, ref(ex), G, None, G, big, None) == 1    # no y_shared
    assert lib.moe_expert_ffn_int8(ref(d), G, G, G, ref(ex), G, G, G + 16, big, None) == 1  # ws alignment
    assert lib.moe_expert_ffn_int8(ref(d), G, G, G, ref(ex), G, G, G, 16, None) == 3
    assert lib.moe_layer_forward_int8(ref(d), G, G, G + 4, ref(ex), G, G, big, None) == 1   # bias alignment
    bad = moe.dims(8, 4000, 192, 1536, 8)
    assert lib.moe_expert_ffn_int8(ref(bad), G, G, G, ref(ex), G, G, G, big, None) == 2
    empty = moe.dims(0, 256, 16, 128, 4)
    assert lib.moe_layer_forward_int8(ref(empty), None, None, None, None, None, None, 0, None) == 0
    assert lib.moe_expert_ffn_int8(ref(empty), None, None, None, None, None, None, None, 0, None) == 0


def test_binding_refuses_tensors_of_other_shapes_and_types(lib):
    d = moe.dims(4, 128, 2, 64, 1, has_shared=False)
    pair = lambda *s: (torch.zeros(s, dtype=torch.int8), torch.zeros(s[:-1]))  # noqa: E731
    good = dict(gate=pair(2, 64, 128), up=pair(2, 64, 128), down=pair(2, 128, 64))

    class OnHost(moe.Int8Experts):  # the checks alone: no device pointers are taken
        def __init__(self, **t):
            self.t, self.fits = t, None

    OnHost(**good).check(d)
    with pytest.raises(ValueError):
        OnHost(**{**good, "down": pair(2, 64, 128)}).check(d)
    with pytest.raises(TypeError):
        OnHost(**{**good, "up": (good["up"][0].to(torch.uint8), good["up"][1])}).check(d)
    with pytest.raises(ValueError):
        OnHost(gate=good["gate"], up=good["up"]).check(d)
    with pytest.raises(ValueError):
        OnHost(**good).check(moe.dims(4, 128, 2, 64, 1))  # a shared expert is missing


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: "-".join(str(v) for v in s.values()))
def test_workspace_covers_the_int8_pieces(lib, s):
    """The header and the hidden state's codes in two bytes at least; fewer bytes are refused."""
    for T in (1, 33, 500):
        d = _dims(T, **s)
        need = 4096 + _up(T * s["H"] * 2) + _up(T * 4)
        assert moe.moe_workspace_bytes(d) >= need
        ref, ex = ctypes.byref, _experts()
        assert lib.moe_expert_ffn_int8(ref(d), G, G, G, ref(ex), G, G, G, need - 1, None) == 3


def test_reference_quantiser():
    x = np.array([[2.0, 1.0, -1.0, 0.0], [0.0, 0.0, 0.0, 0.0], [127.0, 2.5, -3.5, 0.5], [-127.0, 126.5, 1.49, 1.51]])
    q, s = ref8.quantize(x)
    assert q.tolist() == [[127, 64, -64, 0], [0, 0, 0, 0], [127, 2, -4, 0], [-127, 126, 1, 2]]
    assert s.tolist() == [float(np.float32(2) / np.float32(127)), 1.0, 1.0, 1.0]
