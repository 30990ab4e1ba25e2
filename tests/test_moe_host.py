"""CPU checks of the mixture-of-experts calls: what they refuse, workspace
sizes, and the tests' own 64-bit forms on hand-made cases."""
import ctypes

import numpy as np
import pytest
import torch

import moelib
import quantized_gemm_decode_b200 as qgd
from quantized_gemm_decode_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    qgd.lib()


P = ctypes.c_void_p
A = P(1 << 20)  # an aligned address: nothing is launched with it


def _route(**kw):
    d = dict(top_k=2, score=0, groups=1, topk_groups=1, group_top=1, renormalize=1, scale=1.0)
    d.update(kw)
    return ctypes.byref(qgd._Route(**d))


def _call_route(dtype=1, T=4, E=16, ldl=16, logits=A, weights=A, ids=A, bias=None, **kw):
    return qgd.lib().moe_route(logits, dtype, T, E, ldl, bias, _route(**kw), weights, ids, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -1), (dict(T=-1), -1), (dict(E=0), -1), (dict(E=1040, ldl=1040), -2), (dict(ldl=15), -1),
    (dict(top_k=0), -1), (dict(top_k=17), -1), (dict(E=64, ldl=64, top_k=33), -1), (dict(score=2), -1),
    (dict(groups=0), -1), (dict(groups=3), -1), (dict(groups=4, topk_groups=5), -1), (dict(groups=4, topk_groups=0), -1),
    (dict(groups=4, topk_groups=1, top_k=5), -1), (dict(group_top=3), -1), (dict(E=64, ldl=64, groups=64), -1),
    (dict(logits=None), -1), (dict(weights=None), -1), (dict(ids=P((1 << 20) + 2)), -1),
    (dict(logits=P((1 << 20) + 2)), -1), (dict(bias=P((1 << 20) + 1)), -1), (dict(T=0), 0)])
def test_route_refusals(kw, status):
    assert _call_route(**kw) == status
    if status:
        assert qgd.lib().qgd_last_error_message()


def test_route_takes_no_null_descriptor():
    assert qgd.lib().moe_route(A, 1, 4, 16, 16, None, None, A, A, None) == -1


@pytest.mark.parametrize("kw,status", [
    (dict(pairs=-1), -1), (dict(E=0), -1), (dict(E=1025), -2), (dict(offsets=None), -1), (dict(ids=None), -1),
    (dict(order=P((1 << 20) + 1)), -1), (dict(pairs=100000, ws=None), -3), (dict(pairs=100000, ws=A, ws_bytes=16), -3)])
def test_sort_refusals(kw, status):
    d = dict(ids=A, pairs=10, E=4, offsets=A, order=A, pos=A, ws=None, ws_bytes=0)
    d.update(kw)
    assert qgd.lib().moe_sort(d["ids"], d["pairs"], d["E"], d["offsets"], d["order"], d["pos"], d["ws"],
                              d["ws_bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=-1), -1), (dict(fmt=5), -1), (dict(fmt=2), -2), (dict(fmt=3), -2), (dict(fmt=4), -2), (dict(act=2), -1),
    (dict(rows=-1), -1), (dict(N=24), -2), (dict(N=0), -1), (dict(K=40), -2), (dict(K=16400, ldx=16400), -2),
    (dict(E=0), -1), (dict(E=2000), -2), (dict(ldx=56), -1), (dict(ldx=68), -1), (dict(top_k=0), -1),
    (dict(order=None, rows=9), -1), (dict(x_rows=0), -1), (dict(x=None), -1), (dict(wq=P((1 << 20) + 8)), -1), (dict(y=P((1 << 20) + 8)), -1),
    (dict(sw=P((1 << 20) + 2)), -1), (dict(offsets=None), -1), (dict(N=1 << 20, E=1024), -2), (dict(rows=0), 0),
    (dict(rows=1 << 28, E=1024, N=16), -2), (dict(rows=1 << 28, N=4096, K=16384, ldx=16384), -2)])
def test_experts_refusals(kw, status):
    d = dict(fmt=1, x=A, ldx=64, x_rows=8, order=A, top_k=2, offsets=A, E=4, rows=16, wq=A, sw=A, y=A, N=32, K=64, act=0,
             ws=A, ws_bytes=1 << 40)
    d.update(kw)
    assert qgd.lib().qlinear_experts_bf16(d["fmt"], d["x"], d["ldx"], d["x_rows"], d["order"], d["top_k"],
                                          d["offsets"], d["E"], d["rows"], d["wq"], d["sw"], d["y"], d["N"], d["K"],
                                          d["act"], d["ws"], d["ws_bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(T=-1), -1), (dict(H=12), -2), (dict(H=0), -1), (dict(k=0), -1), (dict(k=33), -1),
    (dict(add=A, lda=24), -1), (dict(add=A, lda=36), -1), (dict(h=None), -1), (dict(pos=None), -1),
    (dict(h=P((1 << 20) + 8)), -1), (dict(w=P((1 << 20) + 2)), -1), (dict(T=0), 0)])
def test_combine_refusals(kw, status):
    d = dict(h=A, rows=8, pos=A, w=A, add=None, lda=0, y=A, T=4, k=2, H=32)
    d.update(kw)
    assert qgd.lib().moe_combine(d["h"], d["rows"], d["pos"], d["w"], d["add"], d["lda"], d["y"], d["T"], d["k"], d["H"],
                                 None) == status


def test_python_checks_reject_cpu_tensors_and_wrong_types():
    f = torch.zeros
    with pytest.raises(ValueError):
        qgd.moe_route(f(4, 8), 2)
    with pytest.raises(ValueError):
        qgd.moe_route(f(4, 8), 2, score="tanh")
    with pytest.raises(ValueError):
        qgd.moe_sort(f(4, 2, dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        qgd.moe_sort(f(4, 2, dtype=torch.int64), 8)
    with pytest.raises(ValueError):
        qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, f(4, 64).bfloat16(), None, None, None)
    with pytest.raises(ValueError):
        qgd.moe_combine(f(4, 64).bfloat16(), None, None)


def test_workspace_sizes():
    assert qgd.qgd_moe_sort_workspace_size(1, 8) == 0
    assert qgd.qgd_moe_sort_workspace_size(0, 8) == 0
    assert qgd.qgd_moe_sort_workspace_size(1 << 20, 256) >= 256 * 4
    assert qgd.qgd_experts_workspace_size(qgd.FMT_BLOCK_FP8, 8, 4, 8, 64, 64) == 0
    assert qgd.qgd_experts_workspace_size(qgd.FMT_W8A8_INT8, 0, 4, 8, 64, 64) == 0
    # the codes and scales of the sorted rows at least
    assert qgd.qgd_experts_workspace_size(qgd.FMT_W8A8_INT8, 1000, 0, 8, 64, 512) >= 1000 * 516


# ---------------------------------------------------------------------------
# the 64-bit forms themselves, on cases worked out by hand
# ---------------------------------------------------------------------------
def test_oracle_route_by_hand():
    logits = torch.tensor([[0.0, 1.0, 1.0, -1.0], [float("-inf"), float("nan"), 3.0, float("-inf")]])
    w, ids = moelib.route(logits, 2)
    np.testing.assert_array_equal(ids, [[1, 2], [2, -1]])
    np.testing.assert_allclose(w, [[0.5, 0.5], [1.0, 0.0]])
    # the bias moves the choice, not the weight
    w, ids = moelib.route(logits[:1], 1, score="sigmoid", bias=torch.tensor([0.0, 0.0, 0.0, 1.0]), renormalize=False)
    assert ids[0, 0] == 3 and w[0, 0] == pytest.approx(1 / (1 + np.e))
    # groups {0, 1} and {2, 3}: sums 0.5 + 0.731 against 0.731 + 0.269
    w, ids = moelib.route(logits[:1], 2, score="sigmoid", groups=2, topk_groups=1, group_top=2)
    np.testing.assert_array_equal(ids, [[1, 0]])


def test_oracle_sort_by_hand():
    off, order, pos = moelib.sort(torch.tensor([[1, 0], [-1, 1], [0, 7]], dtype=torch.int32), 2)
    np.testing.assert_array_equal(off, [0, 2, 4])
    np.testing.assert_array_equal(order, [1, 4, 0, 3, -1, -1])
    np.testing.assert_array_equal(pos, [[2, 0], [-1, 3], [1, -1]])


def test_oracle_notices_a_swapped_expert():
    # a planted mistake: two experts' weights exchanged
    g = torch.Generator().manual_seed(0)
    wq = torch.randint(-127, 128, (2, 16, 32), generator=g, dtype=torch.int8)
    sw = torch.full((2, 16), 1e-3)
    x = torch.randn((4, 32), generator=g).bfloat16()
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    ref, mag = moelib.experts(x, wq, sw, off, None, 1, False, True)
    bad, _ = moelib.experts(x, wq.flip(0), sw, off, None, 1, False, True)
    moelib.close(ref, ref, moelib.experts_tolerance(ref, mag, 32, False, True))
    with pytest.raises(AssertionError):
        moelib.close(bad, ref, moelib.experts_tolerance(ref, mag, 32, False, True))
