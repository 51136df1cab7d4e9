"""MXFP4 expert FFN at the ends of its number ranges, in both forms: T = 4 (and 48) runs the one-kernel form,
T = 64 (16 slots an expert) the converting kernel."""
import numpy as np
import pytest
import torch

import expert_ffn_layer_gb300 as moe
import oracle
import workloads as W
from moe_testlib import DeviceLayer, i32_dev
from test_gpu_few import TINY
from test_gpu_mxfp4 import experts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Ffn:
    """Tokens to experts 0..3 in turn order; run() returns y_sorted and y_shared."""

    def __init__(self, T):
        w = TINY.with_(T=T)
        self.dl = DeviceLayer(w, W.layer_inputs(w))
        self.ex = experts_of(self.dl)
        topk = np.tile(np.arange(4, dtype=np.int32), (T, 1))
        _, self.offsets = oracle.histogram_offsets(topk, w.E)
        self.perm, _ = oracle.permutation(topk, w.E)
        self.y = torch.empty((T * 4, w.H), dtype=torch.bfloat16, device="cuda")
        self.z = torch.empty((T, w.H), dtype=torch.bfloat16, device="cuda")

    def run(self):
        dl = self.dl
        moe.moe_expert_ffn_mxfp4(dl.d, dl.hidden, i32_dev(self.perm), i32_dev(self.offsets), self.ex, self.y, self.z, dl.ws)
        assert moe.moe_ws_read_error(dl.ws) == 0
        return self.y.clone(), self.z.clone()


@pytest.mark.parametrize("T", [4, 48, 64])
@pytest.mark.parametrize("gate,up,down", [(0, -60, 60), (0, 60, -60), (0, 90, -90), (0, -90, 90), (0, 100, -100)])
def test_scales_moved_by_powers_of_two(T, gate, up, down):
    """Factors that cancel between the up and the down weights leave every bit of the outputs."""
    f = Ffn(T)
    y, z = f.run()
    for names, by in ((("gate", "s_gate"), gate), (("up", "s_up"), up), (("down", "s_down"), down)):
        for n in names:
            s = f.ex.t[n][1]
            moved = s.int() + by
            assert int(moved.min()) >= 1 and int(moved.max()) <= 223
            s.copy_(moved.to(torch.uint8))
    y2, z2 = f.run()
    assert torch.equal(y, y2) and torch.equal(z, z2)


@pytest.mark.parametrize("T", [4, 48, 64])
@pytest.mark.parametrize("by", [-100, -40, 40, 90])
def test_hidden_moved_against_the_weights(T, by):
    """Hidden rows 2^by times as large and gate and up scales 2^-by times: the same products."""
    f = Ffn(T)
    y, z = f.run()
    f.dl.hidden.copy_((f.dl.hidden.double() * 2.0 ** by).bfloat16())
    for n in ("gate", "up", "s_gate", "s_up"):
        s = f.ex.t[n][1]
        moved = s.int() - by
        assert int(moved.min()) >= 1 and int(moved.max()) <= 223
        s.copy_(moved.to(torch.uint8))
    y2, z2 = f.run()
    assert torch.equal(y, y2) and torch.equal(z, z2)


@pytest.mark.parametrize("T", [4, 48, 64])
@pytest.mark.parametrize("name", ["gate", "up"])
def test_a_scale_byte_of_255_in_gate_or_up(T, name):
    """Expert 2's activation 5 is then not finite for any token, and with it every output of that expert."""
    f = Ffn(T)
    y, z = f.run()
    f.ex.t[name][1][2, 5, 1] = 255
    y2, z2 = f.run()
    rows = slice(int(f.offsets[2]), int(f.offsets[3]))
    assert not torch.isfinite(y2[rows]).any()
    y2[rows] = y[rows]
    assert torch.equal(y, y2) and torch.equal(z, z2)


@pytest.mark.parametrize("T", [4, 48, 64])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_one_hidden_value_that_is_not_finite(T, value):
    """The token's outputs are not finite; the other tokens keep every bit."""
    f = Ffn(T)
    y, z = f.run()
    f.dl.hidden[1, 17] = value
    y2, z2 = f.run()
    mine = torch.from_numpy(np.asarray(f.perm) // 4 == 1).cuda()
    assert not torch.isfinite(y2[mine]).any() and not torch.isfinite(z2[1]).any()
    y2[mine], z2[1] = y[mine], z[1]
    assert torch.equal(y, y2) and torch.equal(z, z2)
