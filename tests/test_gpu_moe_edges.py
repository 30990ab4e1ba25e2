"""Mixture-of-experts calls on the GPU at the edges of what they take: shared
workspaces, extreme values, other streams, refusals."""
import pytest
import torch

import moelib
import quantized_gemm_decode_b200 as qgd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    qgd.lib()
    yield
    for f in (qgd.FMT_FP8_DYNAMIC, qgd.FMT_W8A8_INT8):
        qgd.qgd_set_override(f)
    torch.cuda.synchronize()
    assert qgd.qgd_device_error() == 0


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bits(t):
    return t.view(torch.int16)


def _weights(E, rows, K, int8, seed):
    g = _gen(seed)
    if int8:
        wq = torch.randint(-127, 128, (E, rows, K), generator=g, dtype=torch.int8)
    else:
        wq = (100 * torch.randn((E, rows, K), generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return wq, 2e-4 * (0.5 + torch.rand((E, rows), generator=g))


# ---------------------------------------------------------------------------
# one workspace for expert calls and dense calls
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("reduce", [qgd.REDUCE_LAST_CTA, qgd.REDUCE_TWO_PASS])
def test_a_workspace_serves_expert_and_dense_calls(fmt, reduce):
    int8 = fmt == "w8a8_int8"
    fid = qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC
    E, K, N, M = 6, 1024, 512, 4
    wq, sw = (t.cuda() for t in _weights(E, N, K, int8, 1))
    x = torch.randn((M, K), generator=_gen(2)).bfloat16().cuda()
    qgd.qgd_set_override(fid, qgd.VARIANT_SWAP_AB, 4, reduce, 0, 0, qgd.SCHEDULE_GRID)
    assert qgd.qgd_workspace_size(fid, M, N, K) > 0  # the dense plan counts arrivals in its workspace
    ref = qgd.qlinear_bf16(fid, x, wq[0], sw[0], ws=qgd.Workspace(1 << 23)).clone()
    shared = qgd.Workspace(1 << 23)
    for T, k in ((3, 2), (700, 3), (5000, 2)):  # split tiles, pair tiles, several blocks of pairs
        ids = torch.randint(0, E, (T, k), generator=_gen(T), dtype=torch.int32).cuda()
        xe = torch.randn((T, K), generator=_gen(T)).bfloat16().cuda()
        own = qgd.moe_sort(ids, E)
        off, order, pos = qgd.moe_sort(ids, E, ws=shared)
        for a, b in zip(own, (off, order, pos)):
            assert torch.equal(a, b)
        y = qgd.qlinear_experts_bf16(fid, xe, wq, sw, off, order=order, top_k=k, ws=shared)
        assert not shared.buf[:64 * 1024].any()
        dense = qgd.qlinear_bf16(fid, x, wq[0], sw[0], ws=shared)
        again = qgd.qlinear_experts_bf16(fid, xe, wq, sw, off, order=order, top_k=k, ws=shared)
        assert torch.equal(_bits(dense), _bits(ref))
        assert torch.equal(_bits(y), _bits(again))


# ---------------------------------------------------------------------------
# the gated activation over fp32's range
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("rows", [1, 60, 300])
def test_gates_far_below_zero(fmt, rows):
    # One live input per row, whose code is the largest (scale 1), times weights of 1: the
    # products are qmax * sw, so the scales place gates and ups anywhere.
    int8 = fmt == "w8a8_int8"
    qmax = 127.0 if int8 else 448.0
    gates = [0.0, -1.0, 5.0, 60.0, -60.0, -79.5, -80.5, -86.0, -88.5, -89.0, -95.0, -100.0, -103.0, -120.0, -1e20, -1e36]
    ups = [1.0, -3.0, 1e10, 1e30]
    N, K = len(gates) * len(ups), 16
    g = torch.tensor(gates).repeat(len(ups)) / qmax
    u = torch.tensor(ups).repeat_interleave(len(gates)) / qmax
    sw = torch.cat([g, u])[None]
    wq = torch.zeros((1, 2 * N, K), dtype=torch.int8 if int8 else torch.uint8)
    wq[:, :, 0] = 1 if int8 else 0x38  # e4m3 1.0
    x = torch.zeros((rows, K), dtype=torch.bfloat16)
    x[:, 0] = qmax
    off = torch.tensor([0, rows], dtype=torch.int32)
    y = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC, x.cuda(), wq.cuda(), sw.cuda(),
                                 off.cuda(), act=qgd.ACT_SILU_MUL)
    ref, mag = moelib.experts(x, wq, sw, off, None, 1, True, int8)
    # Half a bf16 step; up to g = -104 the exponential's (2 + 1.2 * 104) 2^-23 and the gate's two
    # roundings, 2^-23 together, times |g|: 2^-14 in all; the subnormal exponential's step times
    # |g u|; and half of bf16's smallest step.
    size_g, size_u = mag[:, :N], mag[:, N:]
    tol = abs(ref) * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -149 * (size_g.clip(max=110.0) + 2) * size_u + 2.0 ** -133
    moelib.close(y, ref, tol, fmt)


@pytest.mark.parametrize("rows", [1, 300])
def test_infinite_gates(rows):
    # inf / (1 + 0) = inf, and -inf / (1 + inf) = NaN
    N, K, inf = 16, 16, float("inf")
    sw = torch.ones((1, 2 * N))
    sw[0, :4] = torch.tensor([inf, -inf, 1.0, float("nan")])
    wq = torch.zeros((1, 2 * N, K), dtype=torch.int8)
    wq[:, :, 0] = 1
    x = torch.zeros((rows, K), dtype=torch.bfloat16)
    x[:, 0] = 127.0
    off = torch.tensor([0, rows], dtype=torch.int32)
    y = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, x.cuda(), wq.cuda(), sw.cuda(), off.cuda(),
                                 act=qgd.ACT_SILU_MUL).float().cpu()
    assert (y[:, 0] == inf).all() and y[:, 1].isnan().all() and y[:, 3].isnan().all()
    assert (y[:, 2] == 16128.0).all()  # 127 * 127 in bf16


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_route_infinite_logits_over_masked_ones(dtype, score, renormalize, bias):
    # differences of logits outside fp32's range, with experts left over at finite logits
    inf, low, E = float("inf"), torch.finfo(dtype).min, 64
    rows = [[inf, inf, low, 0.0], [inf, low, low, low], [1e38, 1e38, -3e38, -1e38], [low] * 4, [0.0, low, low, -inf],
            [inf, inf, -inf, low], [3e38, 3e38, 3e38, -3e38]]
    logits = torch.full((len(rows), E), low)
    for t, r in enumerate(rows):
        logits[t, 5:9] = torch.tensor(r)
    logits[-1, 40:] = -inf
    logits = logits.to(dtype)
    b = torch.linspace(-0.25, 0.25, E) if bias else None
    w, ids = qgd.moe_route(logits.cuda(), 4, score=score, renormalize=renormalize, bias=None if b is None else b.cuda())
    rw, ri = moelib.route(logits, 4, score=score, renormalize=renormalize, bias=b)
    assert (ids.cpu().numpy() == ri).all()
    # one rounding to fp32 of a value computed to a few fp32 steps (2^-20 together)
    moelib.close(w, rw, abs(rw) * 2.0 ** -20 + 2.0 ** -140)


# ---------------------------------------------------------------------------
# the layer class
# ---------------------------------------------------------------------------
def _layer(E=8, H=256, I=96, k=3, fmt="w8a8_int8", **route):
    from quantized_gemm_decode_b200.linear import QuantizedExperts
    g = _gen(E + H)
    gu = (0.05 * torch.randn((E, 2 * I, H), generator=g)).bfloat16().cuda()
    dn = (0.05 * torch.randn((E, H, I), generator=g)).bfloat16().cuda()
    return QuantizedExperts(gu, dn, k, fmt, route=route)


def _inputs(M, seed, H=256, E=8):
    g = _gen(seed)
    return torch.randn((M, H), generator=g).bfloat16().cuda(), torch.randn((M, E), generator=g).cuda()


@pytest.mark.parametrize("captured", [False, True])
def test_results_of_earlier_calls_stay_as_they_were(captured):
    layer = _layer()
    if captured:
        layer.capture(buckets=(1, 4))
    ins = [_inputs(M, 30 + i) for i, M in enumerate((4, 4, 3, 1, 1))]
    got = [layer(x, lg) for x, lg in ins]
    for (x, lg), y in zip(ins, got):
        assert torch.equal(_bits(y), _bits(layer.layer(x, lg)))
    got[0].zero_()  # and are the caller's to write
    assert torch.equal(_bits(layer(*ins[1])), _bits(got[1]))


@pytest.mark.parametrize("captured", [False, True])
def test_operands_on_the_host_are_refused(captured):
    layer = _layer()
    if captured:
        layer.capture(buckets=(4,))
    x, lg = _inputs(4, 3)
    for bad in ((x.cpu(), lg, None), (x, lg.cpu(), None), (x, lg, x.cpu()), (x.cpu().pin_memory(), lg, None)):
        with pytest.raises(ValueError, match="cuda|CUDA"):
            layer(*bad)
    assert layer(x, lg, add=x).shape == (4, 256)


def test_graphs_are_captured_on_a_stream_of_the_layers_device(monkeypatch):
    layer, streams, graph = _layer(), [], torch.cuda.graph

    def recording(g, pool=None, stream=None, **kw):
        streams.append(stream)
        return graph(g, pool=pool, stream=stream, **kw)

    monkeypatch.setattr(torch.cuda, "graph", recording)
    layer.capture(buckets=(1, 4))
    assert len(streams) == 2 and all(s is not None and s.device == layer.device for s in streams)
    x, lg = _inputs(3, 4)
    assert torch.equal(_bits(layer(x, lg)), _bits(layer.layer(x, lg)))


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------
def test_streams_given_by_address():
    side = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        for other in (torch.cuda.default_stream(), torch.cuda.Stream()):
            with torch.cuda.stream(other), qgd._on(0, stream.cuda_stream):
                assert torch.cuda.current_stream().cuda_stream == stream.cuda_stream
    # on the default stream, a call by its address follows the work queued there
    ids = torch.randint(0, 16, (4000, 4), generator=_gen(1), dtype=torch.int32).cuda()
    ref = [t.clone() for t in qgd.moe_sort(ids, 16)]
    for _ in range(10):
        late = torch.zeros_like(ids)
        torch.cuda._sleep(2_000_000)
        late.copy_(ids)
        got = qgd.moe_sort(late, 16, stream=torch.cuda.default_stream().cuda_stream)
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_sizes_and_strides_past_32_bits_are_refused():
    # (nothing of the buffer is written or read)
    n = (1 << 32) + 64
    buf = torch.empty(n, dtype=torch.int32, device="cuda")
    wide = buf.view(torch.bfloat16)
    far = wide.as_strided((2, 64), (n, 1))
    wq, sw = (t.cuda() for t in _weights(2, 32, 64, True, 1))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    h, one = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((2, 1), device="cuda")
    pos = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: qgd.moe_route(far, 2), lambda: qgd.moe_route(wide[:n, None], 1),
                 lambda: qgd.moe_route(h, (1 << 32) + 1),
                 lambda: qgd.moe_sort(buf, 8), lambda: qgd.moe_sort(pos, (1 << 32) + 8),
                 lambda: qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, far, wq, sw, off),
                 lambda: qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, h, wq, sw, off, order=buf),
                 lambda: qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, h, wq, sw, off, order=pos.view(-1), top_k=1 << 32),
                 lambda: qgd.moe_combine(h, pos, one, add=far)):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            call()


def test_route_as_many_rows_as_an_int_counts():
    # one expert, so every row's choice is known; 22 GB
    T = (1 << 31) - 1
    logits = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    logits[-1] = float("-inf")
    w, ids = qgd.moe_route(logits, 1, score="sigmoid", renormalize=False)
    assert w[-4:].flatten().tolist() == [0.5, 0.5, 0.5, 0.0] and ids[-4:].flatten().tolist() == [0, 0, 0, -1]
    assert w[:2].flatten().tolist() == [0.5, 0.5]
    assert int((ids[1 << 30:].view(-1) == 0).sum()) == T - (1 << 30) - 1


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("E,scale", [(4, 1), (4, 20), (4, 150), (400, 1), (400, 150)])
def test_offsets_that_descend_write_nothing(fmt, E, scale):
    # rows could belong to several experts, and those at offsets[E] and behind have no codes
    int8 = fmt == "w8a8_int8"
    K, N, rows = 128, 48, 10 * scale
    wq, sw = _weights(E, N, K, int8, 1)
    x = torch.randn((rows, K), generator=_gen(1)).bfloat16()
    args = (qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC, x.cuda(), wq.cuda(), sw.cuda())
    need = qgd.qgd_experts_workspace_size(args[0], rows, 0, E, N, K)
    for place in {0, E - 4}:  # descents among the first and the last experts
        for offsets in ([0, 3, 8, 9, 6], [0, 8, 8, 7, 6], [2, 9, 4, 4, -3], [7, 6, 9, 8, 0], [0, 3, 5, 8, 9]):
            off = torch.full((E + 1,), offsets[-1] if place == 0 else offsets[0], dtype=torch.int32)
            off[place:place + 5] = torch.tensor(offsets, dtype=torch.int32)
            off *= scale
            y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
            ws = torch.full((need,), 0x55, dtype=torch.uint8, device="cuda")  # what uncoded rows would hold
            qgd.qlinear_experts_bf16(*args, off.cuda(), y=y, ws=ws)
            if offsets == sorted(offsets):
                ref, mag = moelib.experts(x, wq, sw, off, None, 1, False, int8)
                n = int(off[-1])
                moelib.close(y[:n], ref[:n], moelib.experts_tolerance(ref, mag, K, False, int8)[:n])
                assert (y[n:] == 7.0).all()
            else:
                assert (y == 7.0).all()


# ---------------------------------------------------------------------------
# sort of many pairs
# ---------------------------------------------------------------------------
def _check_sort(ids, E):
    off, order, pos = qgd.moe_sort(ids, E)
    P = ids.numel()
    live = (ids >= 0) & (ids < E)
    ref = torch.sort(torch.where(live, ids, E), stable=True).indices
    n = int(live.sum())
    assert torch.equal(off[1:].long(), torch.bincount(ids[live].long(), minlength=E).cumsum(0)) and off[0] == 0
    assert torch.equal(order[:n].long(), ref[:n]) and (order[n:] == -1).all()
    want = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    want[ref[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(pos, want)


# 2048 pairs a block; above 65536 counts the blocks' counts are summed by a kernel of their own
@pytest.mark.parametrize("P,E", [(64 * 2048, 1024), (64 * 2048 + 1, 1024), (257 * 2048 - 1, 256), (8192 * 2048, 7),
                                 (8192 * 2048 + 5, 7), (5_000_003, 33), (4_500_000, 1023), (9_000_001, 257)])
def test_sort_of_many_pairs(P, E):
    g = torch.Generator(device="cuda").manual_seed(P)
    ids = torch.randint(0, E, (P,), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(P, generator=g, device="cuda") < 0.1] = -1
    _check_sort(ids, E)


def test_sort_as_many_pairs_as_an_int_counts():
    # all but the last pairs go to expert 1; 34 GB
    P, tail = (1 << 31) - 1, [2, -1, 0, 1, 2, 7]
    ids = torch.ones(P, dtype=torch.int32, device="cuda")
    ids[-6:] = torch.tensor(tail, dtype=torch.int32)
    off, order, pos = qgd.moe_sort(ids, 3)
    assert off.tolist() == [0, 1, P - 4, P - 2]
    assert order[0] == P - 4 and order[P - 5] == P - 3 and order[P - 4:].tolist() == [P - 6, P - 2, -1, -1]
    assert pos[-6:].tolist() == [P - 4, -1, 0, P - 5, P - 3, -1]
    for a in range(0, P - 6, 1 << 29):  # the others keep their order, one place up
        b = min(a + (1 << 29), P - 6)
        run = torch.arange(a, b, dtype=torch.int32, device="cuda")
        assert torch.equal(order[a + 1:b + 1], run)
        assert torch.equal(pos[a:b], run + 1)


def test_sort_time_grows_with_the_pairs():
    # (with every block adding up all blocks' counts, 64 M pairs took 780 ms, and 2 G would take minutes)
    def ms(P):
        ids = torch.zeros(P, dtype=torch.int32, device="cuda")
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            qgd.moe_sort(ids, 1024)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert ms(1 << 26) < 64 * ms(1 << 22)  # 16 times the pairs


def _moe_args():
    E, K, N = 4, 64, 32
    wq, sw = (t.cuda() for t in _weights(E, N, K, True, 1))
    f = dict(dtype=torch.float32, device="cuda")
    i = dict(dtype=torch.int32, device="cuda")
    return dict(logits=torch.zeros((6, 16), **f), ids=torch.zeros((6, 2), **i), wq=wq, sw=sw,
                x=torch.zeros((6, K), dtype=torch.bfloat16, device="cuda"), offsets=torch.zeros(E + 1, **i),
                order=torch.zeros(12, **i), h=torch.zeros((12, N), dtype=torch.bfloat16, device="cuda"),
                pos=torch.zeros((6, 2), **i), weights=torch.zeros((6, 2), **f))


def _call(name, a):
    if name == "route":
        return qgd.moe_route(a["logits"], 2, score=a.get("score", "softmax"), bias=a.get("bias"),
                             weights=a.get("weights_out"), ids=a.get("ids_out"), stream=a.get("stream"))
    if name == "sort":
        return qgd.moe_sort(a["ids"], 4, offsets=a.get("offsets_out"), order=a.get("order_out"), pos=a.get("pos_out"))
    if name == "experts":
        return qgd.qlinear_experts_bf16(a.get("fmt", qgd.FMT_W8A8_INT8), a["x"], a["wq"], a["sw"], a["offsets"],
                                        order=a["order"], top_k=2, act=a.get("act", qgd.ACT_NONE), y=a.get("y"),
                                        ws=a.get("ws"))
    return qgd.moe_combine(a["h"], a["pos"], a["weights"], add=a.get("add"), y=a.get("y"))


@pytest.mark.parametrize("name", ["route", "sort", "experts", "combine"])
def test_the_refusals_start_from_calls_that_pass(name):
    _call(name, _moe_args())


# each case changes one operand of a call that passes, and has to be refused for that operand
@pytest.mark.parametrize("name,key,change,match", [
    ("route", "score", lambda a: "tanh", "score must be one of"),
    ("route", "logits", lambda a: a["logits"].double(), "logits has type torch.float64"),
    ("route", "logits", lambda a: a["logits"][0], "logits must be 2-D"),
    ("route", "logits", lambda a: a["logits"].t(), "unit column stride"),
    ("route", "logits", lambda a: a["logits"][:1].expand(6, 16), "row stride of at least"),
    ("route", "logits", lambda a: a["logits"].cpu(), "logits must be a CUDA tensor"),
    ("route", "bias", lambda a: torch.zeros(15, device="cuda"), "bias has shape"),
    ("route", "bias", lambda a: torch.zeros(16, device="cuda").bfloat16(), "bias has type"),
    ("route", "bias", lambda a: torch.zeros(16), "bias is on cpu"),
    ("route", "bias", lambda a: torch.zeros(32, device="cuda")[::2], "bias must be contiguous"),
    ("route", "weights_out", lambda a: torch.zeros((6, 3), device="cuda"), "weights has shape"),
    ("route", "ids_out", lambda a: torch.zeros((6, 2), device="cuda").long(), "ids has type"),
    ("sort", "ids", lambda a: a["ids"].long(), "ids has type torch.int64"),
    ("sort", "ids", lambda a: a["ids"][:, :1], "ids must be contiguous"),
    ("sort", "ids", lambda a: a["ids"].cpu(), "ids must be a CUDA tensor"),
    ("sort", "offsets_out", lambda a: torch.zeros(4, dtype=torch.int32, device="cuda"), "offsets has shape"),
    ("sort", "order_out", lambda a: torch.zeros(11, dtype=torch.int32, device="cuda"), "order has shape"),
    ("sort", "pos_out", lambda a: torch.zeros(12, dtype=torch.int32, device="cuda"), "pos has shape"),
    ("experts", "x", lambda a: a["x"].float(), "x has type"),
    ("experts", "x", lambda a: a["x"][0], "x must be 2-D"),
    ("experts", "x", lambda a: torch.zeros((6, 128), device="cuda").bfloat16()[:, ::2], "unit column stride"),
    ("experts", "x", lambda a: torch.zeros((6, 80), device="cuda").bfloat16(), "wq must be"),
    ("experts", "wq", lambda a: a["wq"].view(torch.uint8), "wq has type"),
    ("experts", "fmt", lambda a: qgd.FMT_FP8_DYNAMIC, "wq has type torch.int8"),
    ("experts", "wq", lambda a: a["wq"][0], "wq must be"),
    ("experts", "wq", lambda a: a["wq"].transpose(0, 1).contiguous().transpose(0, 1), "wq must be contiguous"),
    ("experts", "wq", lambda a: a["wq"].cpu(), "wq is on cpu"),
    ("experts", "sw", lambda a: a["sw"][:, :16].contiguous(), "sw has shape"),
    ("experts", "sw", lambda a: a["sw"].double(), "sw has type"),
    ("experts", "offsets", lambda a: a["offsets"][:4], "offsets has shape"),
    ("experts", "offsets", lambda a: a["offsets"].long(), "offsets has type"),
    ("experts", "order", lambda a: a["order"].long(), "order has type"),
    ("experts", "order", lambda a: a["order"].tolist(), "order must be a tensor"),
    ("experts", "act", lambda a: 2, "act must be"),
    ("experts", "y", lambda a: torch.zeros((12, 64), device="cuda").bfloat16(), "y has shape"),
    ("experts", "ws", lambda a: torch.zeros(1 << 20, dtype=torch.uint8), "ws must be"),
    ("combine", "h", lambda a: a["h"].float(), "h has type"),
    ("combine", "h", lambda a: a["h"][0], "h must be"),
    ("combine", "pos", lambda a: a["pos"].long(), "pos has type"),
    ("combine", "pos", lambda a: a["pos"].view(-1), "pos \\[tokens"),
    ("combine", "weights", lambda a: a["weights"].bfloat16(), "weights has type"),
    ("combine", "weights", lambda a: a["weights"][:, :1].contiguous(), "weights has shape"),
    ("combine", "add", lambda a: a["h"][:5], "add has shape"),
    ("combine", "add", lambda a: a["h"][:1].expand(6, 32), "row stride of at least"),
    ("combine", "y", lambda a: torch.zeros((6, 32), device="cuda"), "y has type"),
])
def test_refusals_name_their_operand(name, key, change, match):
    a = _moe_args()
    a[key] = change(a)
    with pytest.raises(ValueError, match=match):
        _call(name, a)


# ---------------------------------------------------------------------------
# behind copies, wide layers
# ---------------------------------------------------------------------------
def test_calls_wait_for_the_copies_before_them():
    # copies of a few microseconds in front of the calls, on a stream and inside a graph
    T, E, k, K, N = 16384, 256, 8, 512, 64
    wq, sw = (t.cuda() for t in _weights(E, N, K, True, 1))
    lg, x = torch.empty((T, E), device="cuda"), torch.empty((T, K), device="cuda").bfloat16()
    ids, w, pos = (torch.empty((T, k), dtype=d, device="cuda") for d in (torch.int32, torch.float32, torch.int32))
    h = torch.empty((T * k, N), device="cuda").bfloat16()

    def calls(src):
        lg.copy_(src["lg"])
        rw, ri = qgd.moe_route(lg, k)
        ids.copy_(src["ids"])
        off, order, p = qgd.moe_sort(ids, E)
        x.copy_(src["x"])
        y = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, x, wq, sw, off, order=order, top_k=k)
        w.copy_(src["w"])
        pos.copy_(p)
        h.copy_(y)
        return [rw, ri, off, order, p, y, qgd.moe_combine(h, pos, w)]

    def source(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return dict(lg=torch.randn((T, E), generator=g, device="cuda"),
                    ids=torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32),
                    x=torch.randn((T, K), generator=g, device="cuda").bfloat16(),
                    w=torch.rand((T, k), generator=g, device="cuda"))

    def settled(src):  # every copy and call on its own
        out = []
        for fn in (lambda: qgd.moe_route(src["lg"], k), lambda: qgd.moe_sort(src["ids"], E)):
            out += fn()
            torch.cuda.synchronize()
        out.append(qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8, src["x"], wq, sw, out[2], order=out[3], top_k=k))
        torch.cuda.synchronize()
        return out + [qgd.moe_combine(out[5], out[4], src["w"])]

    src = source(0)
    calls(src)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls(src)
    for seed in range(1, 4):
        new = source(seed)
        want = settled(new)
        for got in (calls(new), None):
            if got is None:
                for n, t in src.items():
                    t.copy_(new[n])
                graph.replay()
                got = held
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("fmt", ["w8a8_int8", "fp8_dynamic"])
@pytest.mark.parametrize("T,k,E,K,N,act", [(1, 8, 256, 7168, 64, True), (33, 8, 256, 7168, 32, False),
                                           (90, 6, 1024, 256, 32, True), (2600, 8, 1024, 64, 16, False),
                                           (300, 8, 8, 7168, 48, True), (700, 2, 4, 16384, 32, False)])
def test_experts_wide_and_many(fmt, T, k, E, K, N, act):
    int8 = fmt == "w8a8_int8"
    g = _gen(T + E)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    off, order, _ = (torch.from_numpy(v) for v in moelib.sort(ids, E))
    x = torch.randn((T, K), generator=g).bfloat16()
    wq, sw = _weights(E, N * (2 if act else 1), K, int8, 5)
    y = qgd.qlinear_experts_bf16(qgd.FMT_W8A8_INT8 if int8 else qgd.FMT_FP8_DYNAMIC, x.cuda(), wq.cuda(), sw.cuda(),
                                 off.cuda(), order=order.cuda(), top_k=k,
                                 act=qgd.ACT_SILU_MUL if act else qgd.ACT_NONE)
    ref, mag = moelib.experts(x, wq, sw, off, order, k, act, int8)
    moelib.close(y, ref, moelib.experts_tolerance(ref, mag, K, act, int8))
