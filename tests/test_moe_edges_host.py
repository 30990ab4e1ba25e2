"""CPU checks of the mixture-of-experts calls at the edges of what they take."""
import pytest
import torch

import quantized_gemm_decode_b200 as qgd
from quantized_gemm_decode_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    qgd.lib()


HEADER = 64 * 1024  # the dense calls' arrival counters, zero between calls


def test_workspaces_leave_room_for_the_dense_calls_counters():
    # two blocks of pairs, 8 experts: 2 x 8 counts
    assert qgd.qgd_moe_sort_workspace_size(4096, 8) >= HEADER + 2 * 8 * 4
    assert qgd.qgd_moe_sort_workspace_size(2048, 8) == 0  # one block needs none
    for fmt in (qgd.FMT_W8A8_INT8, qgd.FMT_FP8_DYNAMIC):
        # codes and scales of one row, and an arrival counter per SM
        assert qgd.qgd_experts_workspace_size(fmt, 1, 1, 4, 64, 256) >= HEADER + 148 * 4 + 256 + 4


def test_layer_quantizes_its_weights_on_their_own_device(monkeypatch):
    # the quantizer launches on the current device, which need not be the weights'
    from quantized_gemm_decode_b200.linear import QuantizedExperts
    current = ["the caller's"]

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *exc):
            current.pop()

    seen = []

    def quantizer(w, qtype):
        seen.append((current[-1], w.device))
        return torch.zeros(w.shape, dtype=torch.int8), torch.ones(w.shape[0])

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(qgd, "quant_weight_per_channel", quantizer)
    layer = QuantizedExperts(torch.zeros((2, 32, 64)), torch.zeros((2, 64, 16)), 1)
    assert layer.gate_up.shape == (2, 32, 64) and layer.down_s.shape == (2, 64)
    assert len(seen) == 2 and all(cur == dev for cur, dev in seen)


def test_sizes_and_strides_past_32_bits_are_refused():
    # (the library takes ints: a stride of 2**32 + 64 would arrive as 64)
    for stride in (1 << 31, (1 << 32) + 64):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            qgd._row_stride(torch.empty_strided((2, 64), (stride, 1), device="meta"), "x")
    assert qgd._row_stride(torch.empty_strided((2, 64), ((1 << 31) - 8, 1), device="meta"), "x") == (1 << 31) - 8
    assert qgd._row_stride(torch.empty_strided((1, 64), (1 << 40, 1), device="meta"), "x") == 64  # one row: unused
    for n in (1 << 31, (1 << 32) + 2, 1 << 40):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            qgd._below_2_31(n | 5, "x")
        with pytest.raises(ValueError, match="2\\*\\*31"):
            qgd._route_desc(n, 0, 1, 1, 1, 1, 1.0)
    qgd._below_2_31((1 << 31) - 1, "x")


@pytest.mark.parametrize("rows,unsupported", [((1 << 31) - 1, True), ((1 << 31) - (1 << 20), True), (1 << 30, True),
                                              ((1 << 30) - 1, False)])
@pytest.mark.parametrize("act", [0, 1])
def test_rows_whose_tiles_would_pass_32_bits_are_refused(rows, unsupported, act):
    # 2**31 - 2**20 rows of one expert: rows + token tiles wrap, and tiles would start at negative rows
    at = 1 << 20  # an aligned address; without a workspace nothing is launched with it
    st = qgd.lib().qlinear_experts_bf16(1, at, 16, 8, at, 2, at, 1, rows, at, at, at, 16, 16, act, None, 0, None)
    assert st != 0 and (st == -2) == unsupported
