"""Host-side checks of the MXFP4 and few-token entry points that need no GPU:
refusals before any launch, the struct mirror and the packed layout."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import expert_ffn_layer_gb300 as moe
from test_abi_cpu import _c_struct_fields

G = 0x100000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    moe._lib = None  # another file reloads the module: take its current struct classes
    return moe.load()


def _experts(**over):
    return moe.MoeMxfp4Experts(**{n: over.get(n, G) for n, _ in moe.MoeMxfp4Experts._fields_})


def test_struct_matches_the_header():
    fields = _c_struct_fields("moe_mxfp4_experts")
    assert [n for n, _ in fields] == [n for n, _ in moe.MoeMxfp4Experts._fields_]
    assert all(t.endswith("*") for _, t in fields)


def test_quantizer_refusals(lib):
    assert lib.moe_quantize_mxfp4_rows(G, 4, 64, G, G, None) == 1         # cols % 128
    assert lib.moe_quantize_mxfp4_rows(G, -1, 128, G, G, None) == 1
    assert lib.moe_quantize_mxfp4_rows(G, 1 << 60, 128, G, G, None) == 1  # rows * cols past 64 bits
    assert lib.moe_quantize_mxfp4_rows(None, 4, 128, G, G, None) == 1
    assert lib.moe_quantize_mxfp4_rows(G, 4, 128, G + 8, G, None) == 1
    assert lib.moe_quantize_mxfp4_rows(None, 0, 128, None, None, None) == 0
    assert lib.moe_dequantize_mxfp4_rows(G, G, 4, 96, G, None) == 1
    assert lib.moe_dequantize_mxfp4_rows(G, None, 4, 128, G, None) == 1
    assert lib.moe_dequantize_mxfp4_rows(None, None, 0, 128, None, None) == 0


def test_layer_refusals(lib):
    d, ref = moe.dims(8, 256, 16, 128, 4), ctypes.byref
    ex = _experts()
    big = 1 << 40
    assert lib.moe_layer_forward_mxfp4(ref(d), None, None, None, None, None, None, 0, None) == 1
    assert lib.moe_expert_ffn_mxfp4(ref(d), G, G, G, None, G, G, G, big, None) == 1
    for n, _ in moe.MoeMxfp4Experts._fields_:  # every array has to be there and aligned
        for bad in (None, G + 4):
            assert lib.moe_expert_ffn_mxfp4(ref(d), G, G, G, ref(_experts(**{n: bad})), G, G, G, big, None) == 1, n
    assert lib.moe_expert_ffn_mxfp4(ref(d), G, G, G, ref(ex), G, None, G, big, None) == 1   # no y_shared
    assert lib.moe_expert_ffn_mxfp4(ref(d), G, G, G, ref(ex), G, G, G + 16, big, None) == 1  # ws alignment
    assert lib.moe_expert_ffn_mxfp4(ref(d), G, G, G, ref(ex), G, G, G, 16, None) == 3
    assert lib.moe_layer_forward_mxfp4(ref(d), G, G, G + 4, ref(ex), G, G, big, None) == 1  # bias alignment
    for bad in (moe.dims(8, 192, 16, 128, 4), moe.dims(8, 256, 16, 64, 4), moe.dims(8, 256, 16, 128, 4, I_shared=64)):
        assert lib.moe_expert_ffn_mxfp4(ref(bad), G, G, G, ref(ex), G, G, G, big, None) == 2
        assert lib.moe_layer_forward_mxfp4(ref(bad), G, G, G, ref(ex), G, G, big, None) == 2
    assert lib.moe_layer_forward_few(ref(d), *([None] * 11), 0, None) == 1
    assert lib.moe_layer_forward_few(ref(moe.dims(33, 256, 16, 128, 4)), *([G] * 11), big, None) == 2
    assert lib.moe_layer_forward_few(ref(d), *([G] * 11), 16, None) == 3
    empty = moe.dims(0, 256, 16, 128, 4)
    assert lib.moe_layer_forward_few(ref(empty), *([None] * 11), 0, None) == 0
    assert lib.moe_layer_forward_mxfp4(ref(empty), None, None, None, None, None, None, 0, None) == 0
    assert lib.moe_expert_ffn_mxfp4(ref(empty), None, None, None, None, None, None, None, 0, None) == 0


def test_pack_is_its_own_inverse_and_moves_whole_words():
    plain = torch.from_numpy(np.random.default_rng(0).integers(0, 256, (3, 5, 192), dtype=np.uint8))
    packed = moe.pack_mxfp4(plain)
    assert torch.equal(moe.pack_mxfp4(packed), plain)
    words, moved = plain.reshape(-1, 16, 4), packed.reshape(-1, 16, 4)
    for q in range(4):
        for t in range(4):
            assert torch.equal(moved[:, 4 * t + q], words[:, 4 * q + t])


@pytest.mark.parametrize("T", [1, 8, 32, 33])
def test_workspace_covers_the_one_kernel_layer(lib, T):
    d = moe.dims(T, 4096, 192, 1536, 8)
    fp32 = 4 * ((8 * T + T) * (4096 + 1536)) if T <= 32 else 0
    assert moe.moe_workspace_bytes(d) >= fp32
