"""Mixture-of-experts operators on the GPU: expert routing, the sort of the
pairs, the grouped quantized products and the weighted sum, each against its
64-bit form, and a run of them together."""
import numpy as np
import pytest
import torch

import moelib
import quantized_gemm_decode_b200 as qgd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    qgd.lib()
    yield
    torch.cuda.synchronize()
    assert qgd.qgd_device_error() == 0


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ids(T, k, E, seed, dropped=0.0):
    g = _gen(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32) if T else \
        torch.zeros((0, k), dtype=torch.int32)
    if dropped:
        ids[torch.rand(ids.shape, generator=g) < dropped] = -1
    return ids


# ---------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E,dropped", [(1, 1, 1, 0.0), (1, 8, 64, 0.0), (7, 3, 5, 0.3), (33, 8, 128, 0.1),
                                           (257, 6, 60, 0.0), (512, 8, 1024, 0.0), (4096, 1, 3, 0.0),
                                           (4097, 1, 33, 0.5), (5000, 4, 256, 0.2), (3000, 8, 1000, 0.0)])
def test_sort_matches_a_stable_sort(T, k, E, dropped):
    ids = _ids(T, k, E, 11 * T + k, dropped)
    off, order, pos = qgd.moe_sort(ids.cuda(), E)
    ro, rr, rp = moelib.sort(ids, E)
    np.testing.assert_array_equal(off.cpu().numpy(), ro)
    np.testing.assert_array_equal(order.cpu().numpy(), rr)
    np.testing.assert_array_equal(pos.cpu().numpy(), rp)


@pytest.mark.parametrize("ids,E", [([], 4), ([-1, -1, 9, 4], 4), ([2] * 70, 3), ([3, 3, 0, -5, 2147483647, 0], 4)])
def test_sort_edges(ids, E):
    t = torch.tensor(ids, dtype=torch.int32)
    off, order, pos = qgd.moe_sort(t.cuda(), E)
    ro, rr, rp = moelib.sort(t, E)
    np.testing.assert_array_equal(off.cpu().numpy(), ro)
    np.testing.assert_array_equal(order.cpu().numpy(), rr)
    np.testing.assert_array_equal(pos.cpu().numpy(), rp)


# ---------------------------------------------------------------------------
# combine
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,H,add,dropped", [(1, 1, 8, False, 0.0), (1, 8, 4096, True, 0.0), (5, 3, 24, True, 0.4),
                                               (3, 32, 520, False, 0.1), (67, 9, 1032, True, 0.2), (300, 6, 2048, False, 1.0)])
def test_combine(T, k, H, add, dropped):
    g = _gen(T + H)
    P = T * k
    h = torch.randn((P, H), generator=g).bfloat16()
    pos = torch.randperm(P, generator=g).to(torch.int32).view(T, k)
    pos[torch.rand((T, k), generator=g) < dropped] = -1
    w = torch.randn((T, k), generator=g)
    w[pos < 0] = float("nan")  # a dropped pair's weight is not read
    wide = torch.randn((T, H + 8), generator=g).bfloat16().cuda()
    a = wide[:, :H] if add else None
    y = qgd.moe_combine(h.cuda(), pos.cuda(), w.cuda(), add=a)
    ref, mag = moelib.combine(h, pos, torch.nan_to_num(w), a)
    moelib.close(y, ref, moelib.combine_tolerance(ref, mag, k))


def test_combine_in_place_and_positions_outside():
    g = _gen(5)
    h = torch.randn((6, 64), generator=g).bfloat16()
    pos = torch.tensor([[0, 6], [-7, 3], [1 << 30, 5]], dtype=torch.int32)
    w = torch.rand((3, 2), generator=g)
    y = torch.randn((3, 64), generator=g).bfloat16()
    ref, mag = moelib.combine(h, pos, w, y)
    yd = y.cuda()
    out = qgd.moe_combine(h.cuda(), pos.cuda(), w.cuda(), add=yd, y=yd)
    assert out is yd
    moelib.close(yd, ref, moelib.combine_tolerance(ref, mag, 2))


# ---------------------------------------------------------------------------
# route
# ---------------------------------------------------------------------------
def _check_route(logits, k, **kw):
    bias = kw.get("bias")
    w, ids = qgd.moe_route(logits.cuda(), k, **{**kw, "bias": None if bias is None else bias.cuda()})
    rw, ri = moelib.route(logits, k, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), ri)
    # weights: one rounding to fp32 of a value computed to a few fp32 steps (2^-20 together)
    err = np.abs(w.double().cpu().numpy() - rw)
    assert (err <= np.abs(rw) * 2.0 ** -20 + 2.0 ** -140).all(), (err / np.maximum(np.abs(rw), 1e-300)).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,groups,keep,top", [(1, 1, 1, 1, 1, 1), (3, 5, 5, 1, 1, 1), (9, 33, 7, 1, 1, 1),
                                                   (40, 60, 5, 4, 2, 1), (65, 256, 8, 8, 4, 2), (10, 96, 6, 32, 5, 2),
                                                   (6, 512, 32, 1, 1, 1), (5, 1024, 10, 16, 3, 2), (8, 48, 2, 16, 7, 1)])
@pytest.mark.parametrize("bias", [False, True])
def test_route(score, dtype, T, E, k, groups, keep, top, bias):
    g = _gen(T * E + k)
    logits = (2 * torch.randn((T, E), generator=g)).to(dtype)
    b = 0.2 * torch.randn(E, generator=g) if bias else None
    _check_route(logits, k, score=score, bias=b, groups=groups, topk_groups=keep, group_top=top,
                 renormalize=(T + E) % 2 == 0, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_ties_masks_and_infinities(score, bias):
    g = _gen(3)
    E, k = 64, 6
    logits = torch.randint(-3, 4, (40, E), generator=g).float()  # many equal logits
    logits[0] = float("-inf")
    logits[1, 3:] = float("-inf")
    logits[2] = float("nan")
    logits[3, 10] = float("nan")
    logits[4, 20] = float("inf")
    logits[5, 5:9] = float("inf")
    logits[6] = torch.finfo(torch.float32).min
    logits[7, ::2] = torch.finfo(torch.float32).min
    logits[8] = 0.0
    logits[9] = -0.0
    logits[9, 7] = 0.0
    logits[10] = 80.0
    logits[11] = -120.0 + torch.randn(E, generator=g)  # scores far below fp32's range for sigmoid
    b = (torch.randint(0, 2, (E,), generator=g).float() * 0.25) if bias else None
    for groups, keep, top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        for renorm in (False, True):
            _check_route(logits, k, score=score, bias=b, groups=groups, topk_groups=keep, group_top=top,
                         renormalize=renorm)


def test_route_near_ties_are_decided_in_64_bits():
    # scores equal in 32 bits, told apart in 64: neighbouring fp32 logits under a bias
    E = 32
    base = torch.full((16, E), 1.0)
    for t in range(16):
        base[t, 5] = 1.0 + 2.0 ** -23
        base[t, 9 + t % 8] = 1.0 + 2.0 ** -22
    b = torch.full((E,), 0.5)
    for score in ("softmax", "sigmoid"):
        _check_route(base, 4, score=score, bias=b)
        _check_route(base, 4, score=score, bias=b, groups=4, topk_groups=2, group_top=2)


def test_route_reads_a_column_slice():
    g = _gen(8)
    wide = torch.randn((20, 100), generator=g)
    w, ids = qgd.moe_route(wide.cuda()[:, 3:67], 4)
    rw, ri = moelib.route(wide[:, 3:67], 4)
    np.testing.assert_array_equal(ids.cpu().numpy(), ri)


# ---------------------------------------------------------------------------
# grouped products
# ---------------------------------------------------------------------------
def _weights(E, rows, K, int8, seed):
    g = _gen(seed)
    if int8:
        wq = torch.randint(-127, 128, (E, rows, K), generator=g, dtype=torch.int8)
        sw = 3e-4 * (0.5 + torch.rand((E, rows), generator=g))
    else:
        wq = (100 * torch.randn((E, rows, K), generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        sw = 2e-4 * (0.5 + torch.rand((E, rows), generator=g))
    return wq, sw


def _run_experts(fmt, T, k, E, K, N, act, gather, seed, dropped=0.0, ids=None, ldx=None):
    int8 = fmt == "w8a8_int8"
    g = _gen(seed)
    ids = _ids(T, k, E, seed, dropped) if ids is None else ids
    off, order, _ = (torch.from_numpy(v) for v in moelib.sort(ids, E))
    n_x = T if gather else ids.numel()
    x = torch.randn((n_x, ldx or K), generator=g).bfloat16()
    wq, sw = _weights(E, N * (2 if act else 1), K, int8, seed)
    xd = x.cuda()[:, :K]
    y = torch.full((ids.numel(), N), 7.0, dtype=torch.bfloat16, device="cuda")
    order = order if gather else None
    out = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC, xd, wq.cuda(), sw.cuda(),
                                   off.cuda(), order=None if order is None else order.cuda(), top_k=ids.shape[1],
                                   act=qgd.ACT_SILU_MUL if act else qgd.ACT_NONE, y=y)
    torch.cuda.synchronize()
    assert out is y and qgd.qgd_device_error() == 0
    n = int(off[-1])
    ref, mag = moelib.experts(x[:, :K], wq, sw, off, order, ids.shape[1], act, int8)
    moelib.close(y[:n], ref[:n], moelib.experts_tolerance(ref, mag, K, act, int8)[:n],
                 f"{fmt} T={T} k={k} E={E} K={K} N={N} act={act}")
    assert (y[n:] == 7.0).all()  # rows behind the last expert's are left as they were
    return y


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("T,k,E,K,N", [(1, 1, 1, 16, 16), (1, 2, 4, 128, 128), (1, 8, 16, 1024, 256), (3, 2, 5, 272, 80),
                                       (17, 3, 6, 144, 176), (40, 4, 8, 512, 144), (64, 2, 3, 640, 208),
                                       (200, 1, 2, 1408, 96), (130, 6, 60, 256, 64)])
def test_experts_small(fmt, act, T, k, E, K, N):
    _run_experts(fmt, T, k, E, K, N, act, gather=act, seed=T + K)


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("T,k,E,K,N", [(128, 1, 1, 256, 128), (257, 1, 1, 144, 48), (700, 3, 8, 384, 272),
                                       (1500, 2, 5, 528, 160)])
def test_experts_many_rows(fmt, act, T, k, E, K, N):
    _run_experts(fmt, T, k, E, K, N, act, gather=act, seed=T + K, dropped=0.1)


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
def test_experts_rows_taken_often(fmt):
    # enough rows that each row of x is coded once and its codes are copied; odd widths, dropped pairs
    _run_experts(fmt, 1400, 8, 16, 1520, 48, True, gather=True, seed=3, dropped=0.05)
    _run_experts(fmt, 1100, 9, 12, 2064, 144, False, gather=True, seed=5)


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("act", [False, True])
def test_experts_many_tiles_back_to_back(fmt, act):
    # several tiles per CTA pair and wrapped rings, calls queued behind one another
    int8 = fmt == "w8a8_int8"
    T, k, E, K, N = 1500, 4, 4, 1536, 640
    ids = _ids(T, k, E, 3)
    off, order, _ = (torch.from_numpy(v) for v in moelib.sort(ids, E))
    x = torch.randn((T, K), generator=_gen(3)).bfloat16()
    wq, sw = _weights(E, N * (2 if act else 1), K, int8, 3)
    args = (qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC, x.cuda(), wq.cuda(), sw.cuda(), off.cuda())
    kw = dict(order=order.cuda(), top_k=k, act=qgd.ACT_SILU_MUL if act else qgd.ACT_NONE)
    ys = [qgd.qlinear_experts_bf16(*args, **kw) for _ in range(12)]
    torch.cuda.synchronize()
    for y in ys[1:]:
        assert torch.equal(y.view(torch.int16), ys[0].view(torch.int16))
    ref, mag = moelib.experts(x, wq, sw, off, order, k, act, int8)
    moelib.close(ys[0], ref, moelib.experts_tolerance(ref, mag, K, act, int8))


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("counts", [[0, 0, 5, 0], [0, 0, 0, 0], [64, 65, 0, 1], [16, 17, 128, 129], [255, 256, 257, 1],
                                    [600, 0, 3, 0]])
def test_experts_uneven_loads(fmt, counts):
    ids = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(counts)] +
                    [torch.full((3,), -1, dtype=torch.int32)])
    ids = ids[torch.randperm(ids.numel(), generator=_gen(1))][:, None]
    for act in (False, True):
        _run_experts(fmt, ids.shape[0], 1, 4, 208, 112, act, gather=True, seed=9, ids=ids)


def test_experts_wide_rows_and_plain_gather():
    _run_experts("w8a8_int8", 30, 2, 4, 256, 128, False, gather=True, seed=2, ldx=264)
    _run_experts("fp8_dynamic", 30, 2, 4, 256, 128, True, gather=False, seed=2, ldx=512)


def test_experts_long_rows():
    _run_experts("w8a8_int8", 2, 2, 3, 16384, 64, False, gather=False, seed=4)
    _run_experts("fp8_dynamic", 3, 1, 2, 8208, 32, True, gather=True, seed=4)


def test_experts_bad_offsets_and_rows_stay_in_bounds():
    # offsets past the rows are cut, source rows outside x count as zeros
    E, K, N = 3, 64, 32
    wq, sw = _weights(E, N, K, True, 1)
    x = torch.randn((4, K), generator=_gen(1)).bfloat16()
    off = torch.tensor([-5, 2, 1 << 30, 7], dtype=torch.int32)
    order = torch.tensor([0, 9, -3, 2, 1], dtype=torch.int32)
    y = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, x.cuda(), wq.cuda(), sw.cuda(), off.cuda(), order=order.cuda())
    torch.cuda.synchronize()
    fixed = torch.tensor([0, 2, 5, 5], dtype=torch.int32)
    padded = torch.cat([x, torch.zeros((1, K), dtype=torch.bfloat16)])
    src = torch.tensor([0, 4, 4, 2, 1], dtype=torch.int32)
    ref, mag = moelib.experts(padded, wq, sw, fixed, src, 1, False, True)
    moelib.close(y, ref, moelib.experts_tolerance(ref, mag, K, False, True))


def _awkward_rows(rows, K, qmax, seed):
    """bf16 rows whose quotients by the row scale crowd around the codes'
    rounding boundaries, with zeros, subnormals, infinities and NaNs."""
    g = _gen(seed)
    x = torch.randn((rows, K), generator=g).double()
    amax = torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).double()) * (1 + torch.rand((rows, 1), generator=g))
    amax = amax.bfloat16().double()
    step = amax / qmax
    half = torch.randint(0, 2 * int(qmax), (rows, K), generator=g).double() + 0.5
    near = half * step * 0.5 * torch.where(torch.rand((rows, K), generator=g) < 0.5, 1.0, -1.0)
    fine = step * torch.exp2(-torch.randint(0, 12, (rows, K), generator=g).double()) * torch.randint(1, 16, (rows, K), generator=g)
    pick = torch.rand((rows, K), generator=g)
    x = torch.where(pick < 0.5, near, torch.where(pick < 0.9, fine, x * step))
    x = torch.where(x.abs() > amax, amax, x).bfloat16()
    x[:, 0] = amax[:, 0].bfloat16()
    x[0] = 0
    x[1, :] = 1e-40
    x[2, 3], x[2, 4] = float("inf"), float("-inf")
    x[3, 5] = float("nan")
    x[4] = -0.0
    x[4, 7] = 3e38
    return x


@pytest.mark.parametrize("fmt,qmax", [("w8a8_int8", 127.0), ("fp8_dynamic", 448.0)])
@pytest.mark.parametrize("rows", [48, 700])
def test_experts_same_bits_as_the_dense_layer(fmt, qmax, rows):
    # unit weights give back the codes: they have to be the dense quantizer's, bit for bit
    K = 1024
    int8 = fmt == "w8a8_int8"
    fid = qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC
    x = _awkward_rows(rows, K, qmax, 17).cuda()
    one = 1 if int8 else 0x38  # e4m3 1.0
    wq = (torch.eye(K) * one).to(torch.int8 if int8 else torch.uint8).cuda()
    sw = torch.ones(K, device="cuda")
    dense = qgd.qlinear_bf16(fid, x, wq, sw)
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    y = qgd.qlinear_experts_bf16(fid, x, torch.stack([wq, wq]), torch.stack([sw, sw]), off)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), dense.view(torch.int16))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("T", [1, 5, 90])
def test_a_layer_of_experts(fmt, T):
    E, k, H, I = 8, 3, 256, 96
    int8 = fmt == "w8a8_int8"
    fid = qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC
    g = _gen(T)
    x = torch.randn((T, H), generator=g).bfloat16()
    logits = torch.randn((T, E), generator=g)
    logits[T // 2, :6] = float("-inf")  # fewer experts than slots
    gu, sgu = _weights(E, 2 * I, H, int8, 1)
    dn, sdn = _weights(E, H, I, int8, 2)
    w, ids = qgd.moe_route(logits.cuda(), k)
    off, order, pos = qgd.moe_sort(ids, E)
    h = qgd.qlinear_experts_bf16(fid, x.cuda(), gu.cuda(), sgu.cuda(), off, order=order, top_k=k, act=qgd.ACT_SILU_MUL)
    o = qgd.qlinear_experts_bf16(fid, h, dn.cuda(), sdn.cuda(), off)
    y = qgd.moe_combine(o, pos, w, add=x.cuda())
    torch.cuda.synchronize()
    rw, ri = moelib.route(logits, k)
    np.testing.assert_array_equal(ids.cpu().numpy(), ri)
    n = int(off[-1])
    # stage by stage, each on the stage before as the GPU gave it
    ref, mag = moelib.experts(x, gu, sgu, off, order, k, True, int8)
    moelib.close(h[:n], ref[:n], moelib.experts_tolerance(ref, mag, H, True, int8)[:n])
    hc = h.cpu().clone()
    hc[n:] = 0
    ref, mag = moelib.experts(hc, dn, sdn, off, None, 1, False, int8)
    moelib.close(o[:n], ref[:n], moelib.experts_tolerance(ref, mag, I, False, int8)[:n])
    oc = o.cpu().clone()
    oc[n:] = 0
    ref, mag = moelib.combine(oc, pos.cpu(), w.cpu(), x)
    moelib.close(y, ref, moelib.combine_tolerance(ref, mag, k))


# ---------------------------------------------------------------------------
# streams, graphs, devices, the layer class
# ---------------------------------------------------------------------------
def _layer(fmt="w8a8_int8", E=8, H=256, I=96, k=3, **route):
    from quantized_gemm_decode_b200.linear import QuantizedExperts
    g = _gen(E + H)
    gu = (0.05 * torch.randn((E, 2 * I, H), generator=g)).bfloat16().cuda()
    dn = (0.05 * torch.randn((E, H, I), generator=g)).bfloat16().cuda()
    return QuantizedExperts(gu, dn, k, fmt, route=route), gu, dn


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
def test_layer_class_graphs_match_direct_calls(fmt):
    layer, _, _ = _layer(fmt, score="sigmoid", groups=4, topk_groups=2, group_top=2)
    layer.capture(buckets=(1, 4, 8))
    g = _gen(1)
    for M in (1, 2, 4, 3, 7, 8, 9, 40, 1):
        x = torch.randn((M, 256), generator=g).bfloat16().cuda()
        lg = torch.randn((M, 8), generator=g).cuda()
        add = torch.randn((M, 256), generator=g).bfloat16().cuda() if M % 2 else None
        y = layer(x, lg, add=add).clone()
        ref = layer.layer(x, lg, add=add)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), ref.view(torch.int16)), M


def test_layer_class_against_its_formula():
    layer, gu, dn = _layer()
    T, k, E = 21, 3, 8
    g = _gen(2)
    x = torch.randn((T, 256), generator=g).bfloat16()
    lg = torch.randn((T, E), generator=g)
    y = layer.layer(x.cuda(), lg.cuda()).double().cpu()
    w, ids = moelib.route(lg, k)
    ref = torch.zeros((T, 256), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            v = gu[e].double().cpu() @ x[t].double()
            h = v[:96] / (1 + torch.exp(-v[:96])) * v[96:]
            ref[t] += w[t, j] * (dn[e].double().cpu() @ h)
    # the whole layer in 8 bits against none: a sanity check on the error's norm
    assert (y - ref).norm() / ref.norm() < 0.05


def test_layer_class_refuses_what_does_not_fit():
    layer, gu, dn = _layer()
    from quantized_gemm_decode_b200.linear import QuantizedExperts
    with pytest.raises(ValueError):
        QuantizedExperts(gu, dn[:, :, :64], 2)
    with pytest.raises(ValueError):
        QuantizedExperts(gu, dn, 2, "block_fp8")
    with pytest.raises(ValueError):
        layer.layer(torch.zeros((2, 256), device="cuda").bfloat16(), torch.zeros((3, 8), device="cuda"))
    with pytest.raises(qgd.QGDError):
        qgd.moe_route(torch.zeros((2, 8), device="cuda"), 9)
    assert layer(torch.zeros((0, 256), device="cuda").bfloat16(), torch.zeros((0, 8), device="cuda")).shape == (0, 256)


def test_layer_class_graphs_take_what_direct_calls_take():
    layer, _, _ = _layer()
    layer.capture(buckets=(4,))
    g = _gen(6)
    x, lg = torch.randn((4, 256), generator=g).bfloat16().cuda(), torch.randn((4, 8), generator=g).cuda()
    for call in (layer, layer.layer):
        for bad in ((x[:, :1], lg, None), (x, lg[:1], None), (x, lg[:, :1], None), (x.float(), lg, None),
                    (x, lg, x[:1]), (x, lg, x.float())):
            with pytest.raises(ValueError):
                call(*bad)
    # logits of another type than the graph's keep their own values
    y = layer(x, lg.bfloat16())
    assert torch.equal(y.view(torch.int16), layer.layer(x, lg.bfloat16()).view(torch.int16))


def test_two_graphs_and_two_streams_at_once():
    # each call brings its own workspace: graphs captured separately may run side by side
    layer, _, _ = _layer(E=16, H=512, I=208, k=4)
    ins, refs, graphs, outs = [], [], [], []
    for i in range(2):
        g = _gen(50 + i)
        x = torch.randn((24 + 200 * i, 512), generator=g).bfloat16().cuda()
        lg = torch.randn((24 + 200 * i, 16), generator=g).cuda()
        refs.append(layer.layer(x, lg).clone())
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y = layer.layer(x, lg)
        ins.append((x, lg))
        graphs.append(gr)
        outs.append(y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for y, r in zip(outs, refs):
        assert torch.equal(y.view(torch.int16), r.view(torch.int16))
    # and direct calls on two streams, given as an argument
    got = [None, None]
    for rep in range(10):
        for i, s in enumerate(streams):
            x, lg = ins[i]
            w, ids = qgd.moe_route(lg, 4, stream=s)
            off, order, pos = qgd.moe_sort(ids, 16, stream=s)
            h = qgd.qlinear_experts_bf16(layer.fmt_id, x, layer.gate_up, layer.gate_up_s, off, order=order, top_k=4,
                                         act=qgd.ACT_SILU_MUL, stream=s)
            o = qgd.qlinear_experts_bf16(layer.fmt_id, h, layer.down, layer.down_s, off, stream=s.cuda_stream)
            got[i] = qgd.moe_combine(o, pos, w, stream=s)
    torch.cuda.synchronize()
    for y, r in zip(got, refs):
        assert torch.equal(y.view(torch.int16), r.view(torch.int16))


def test_replay_follows_new_routings():
    layer, _, _ = _layer(E=8, H=256, I=96, k=2)
    x = torch.randn((40, 256), generator=_gen(4)).bfloat16().cuda()
    lg = torch.randn((40, 8), generator=_gen(5)).cuda()
    layer.layer(x, lg)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = layer.layer(x, lg)
    for seed in range(3):
        new = torch.randn((40, 8), generator=_gen(60 + seed))
        if seed == 1:
            new[:, 1:] = float("-inf")  # everything to one expert, one slot each
        if seed == 2:
            new[:] = float("-inf")      # nothing to anyone
        lg.copy_(new)
        gr.replay()
        torch.cuda.synchronize()
        ref = layer.layer(x, new.cuda())
        assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
        if seed == 2:
            assert not y.any()


def test_caller_workspace_and_buffers():
    E, K, N, T, k = 6, 256, 96, 33, 2
    wq, sw = _weights(E, N, K, True, 1)
    ids = _ids(T, k, E, 8)
    x = torch.randn((T, K), generator=_gen(8)).bfloat16().cuda()
    off, order, pos = qgd.moe_sort(ids.cuda(), E)
    need = qgd.qgd_experts_workspace_size(qgd.FMT_W8A8_INT8, T * k, T, E, N, K)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # no zero-filling needed
    a = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, x, wq.cuda(), sw.cuda(), off, order=order, top_k=k, ws=ws)
    b = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, x, wq.cuda(), sw.cuda(), off, order=order, top_k=k,
                                 ws=qgd.Workspace(16))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    with pytest.raises(qgd.QGDError):
        qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, x, wq.cuda(), sw.cuda(), off, order=order, top_k=k, ws=ws[:64])


def test_a_row_listed_twice():
    # an order that names rows of x itself (top_k 1), the same one several times
    E, K, N = 3, 128, 32
    wq, sw = _weights(E, N, K, False, 1)
    x = torch.randn((4, K), generator=_gen(1)).bfloat16()
    order = torch.tensor([2, 2, 0, 3, 2, 2, 1], dtype=torch.int32)
    off = torch.tensor([0, 3, 3, 7], dtype=torch.int32)
    y = qgd.qlinear_experts_bf16(qgd.FMT_FP8_DYNAMIC, x.cuda(), wq.cuda(), sw.cuda(), off.cuda(), order=order.cuda())
    ref, mag = moelib.experts(x, wq, sw, off, order, 1, False, False)
    moelib.close(y, ref, moelib.experts_tolerance(ref, mag, K, False, False))
    assert torch.equal(y[0].view(torch.int16), y[1].view(torch.int16))
