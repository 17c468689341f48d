"""The block-scaled e4m3 operators where a call goes wrong or two ways of making
it meet: offsets out of order, launches that fail, waits that ran out, streams
and graphs, and each way in which few rows are cut into pieces.  References and
tolerances are those of test_gpu_block_fp8.py."""
import ctypes
import threading

import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from tests import block_ref as br
from tests.test_gpu_block_fp8 import BF, F32, _check_bwd, _check_fwd, _ffn_weights, _normal, _offsets, _product, _quantize_rows, _ws, lib  # noqa: F401

pytestmark = [pytest.mark.gpu]


# ---------------------------------------------------------------- offsets out of order
@pytest.mark.parametrize("R", [9, 300])
@pytest.mark.parametrize("cuts", ["down", "past the end", "all in the first", "below zero"])
def test_feed_forward_with_offsets_out_of_order(lib, R, cuts):  # noqa: F811
    """Clamped into order and recorded: the rows of the groups as clamped, none of what an earlier call left in the workspace."""
    E, h, f = 4, 256, 320
    offsets, counts = {
        "down": ([0, 5, 3, R, 2], [5, 0, R - 5, 0]),
        "past the end": ([0, 2, 7, R + 1000, 2 ** 31 - 1], [2, 5, R - 7, 0]),
        "all in the first": ([0, R, 0, 0, 0], [R, 0, 0, 0]),
        "below zero": ([0, -3, 7, 6, -2 ** 31], [0, 7, 0, 0]),
    }[cuts]
    n = sum(counts)
    w = _ffn_weights(E, h, f, 41)
    codes = [t for q, s, _ in w for t in (q, s)]
    x, dy = _normal((R, h), 42), _normal((R, h), 43)
    A, B, H = (torch.full((R, f), 55.0, dtype=BF, device="cuda") for _ in range(3))
    y, dx = torch.full_like(x, 55.0), torch.full_like(x, 55.0)
    dW = [torch.full(v[0].shape, 55.0, dtype=F32, device="cuda") for v in w]
    fd = mb.ffn_dims(R, h, f, E)
    ws = _ws(max(mb.moe_ffn_workspace_bytes(fd, b) for b in (0, 1)))
    # other rows through the same workspace first
    x0, dy0, o0 = _normal((R, h), 44, 50.0), _normal((R, h), 45, 50.0), _offsets([R, 0, 0, 0])
    A0, B0, H0 = (torch.empty_like(A) for _ in range(3))
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    mb.moe_gated_ffn_fwd(fd, x0, o0, *codes, A0, B0, H0, torch.empty_like(y), ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    mb.moe_gated_ffn_fwd(fd, x, o, *codes, A, B, H, y, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_ERR_DEVICE_INDEX
    _check_fwd(x, A, B, H, y, w, counts)
    for t in (A, B, H, y):
        assert (t[n:] == 55).all()
    mb.moe_gated_ffn_bwd(fd, x0, dy0, o0, *codes, A0, B0, H0, torch.empty_like(dx), None, None, None, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    mb.moe_gated_ffn_bwd(fd, x, dy, o, *codes, A, B, H, dx, *dW, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_ERR_DEVICE_INDEX
    _check_bwd(x, dy, A, B, H, w, counts, dx, dW, n)
    assert (dx[n:] == 55).all()


@pytest.mark.parametrize("at", [1, 31, 32, 33, 63, 64])
def test_the_furthest_of_64_ends_in_any_place(lib, at):  # noqa: F811
    """The group that ends there has all rows; every later offset is smaller."""
    R, h, f, E = 70, 128, 192, 64
    w, x = _ffn_weights(E, h, f, 46), _normal((R, h), 47)
    codes = [t for q, s, _ in w for t in (q, s)]
    o = torch.tensor([0] * at + [R] + [3] * (E - at), dtype=torch.int32, device="cuda")
    counts = [0] * (at - 1) + [R] + [0] * (E - at)
    A, B, H = (torch.full((R, f), 55.0, dtype=BF, device="cuda") for _ in range(3))
    y, fd = torch.full_like(x, 55.0), mb.ffn_dims(R, h, f, E)
    ws = _ws(mb.moe_ffn_workspace_bytes(fd, 0))
    mb.moe_gated_ffn_fwd(fd, x, o, *codes, A, B, H, y, ws)
    assert mb.moe_read_device_status(ws) == (mb.MOE_OK if at == 64 else mb.MOE_ERR_DEVICE_INDEX)
    _check_fwd(x, A, B, H, y, w, counts)


# ---------------------------------------------------------------- after a wait that ran out
@pytest.mark.parametrize("counts,K,N", [([3], 4096, 512), ([2, 0, 5], 4096, 1408), ([70], 4096, 512)])
def test_a_status_of_a_timeout_read_leaves_the_workspace_as_new(lib, counts, K, N):  # noqa: F811
    """What blocks that gave up leave in the header: the status, and pieces counted of tiles that nobody joined."""
    R, E = sum(counts), len(counts)
    x = _normal((R, K), 51)
    aq, sa = _quantize_rows(x)
    bq, sb, w = br.weights(E, K, N, seed=52)
    gd, o = mb.gemm_dims(R, K, N, E, out_f32=True), _offsets(counts)
    ws = _ws(mb.moe_gemm_workspace_bytes(gd))
    want, C = (torch.full((R, N), 77.0, dtype=F32, device="cuda") for _ in range(2))
    mb.moe_gemm_fp8_block(gd, aq, sa, bq, sb, o, want, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK and (want != 77).all()
    ws[64:224] = 100
    ws[:4] = torch.tensor([mb.MOE_ERR_DEVICE_TIMEOUT, 0, 0, 0], dtype=torch.uint8)
    assert mb.moe_read_device_status(ws) == mb.MOE_ERR_DEVICE_TIMEOUT
    mb.moe_gemm_fp8_block(gd, aq, sa, bq, sb, o, C, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    assert torch.equal(C, want)


# ---------------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("R,n", [(8192, 100), (8192, 300), (9000, 256), (4096, 4000), (300, 40)])
def test_a_graph_gives_the_bits_of_a_stream(lib, R, n, f32):  # noqa: F811
    """Also where the rows that there are would make fewer tiles than the rows that there could be."""
    K, N = 4096, 512
    aq, sa = _quantize_rows(_normal((R, K), 61))
    bq, sb, _ = br.weights(1, K, N, seed=62)
    gd, o = mb.gemm_dims(R, K, N, 1, out_f32=f32), _offsets([n])
    ws = _ws(mb.moe_gemm_workspace_bytes(gd))
    C = torch.full((R, N), 77.0, dtype=F32 if f32 else BF, device="cuda")
    mb.moe_gemm_fp8_block(gd, aq, sa, bq, sb, o, C, ws)
    torch.cuda.synchronize()
    want = C.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mb.moe_gemm_fp8_block(gd, aq, sa, bq, sb, o, C, ws)
    C.fill_(77)
    graph.replay()
    assert torch.equal(C, want) and (C[n:] == 77).all()


# ---------------------------------------------------------------- launches that fail
@pytest.mark.parametrize("call", ["rows", "weights", "few", "many", "forward"])
def test_an_error_of_one_call_is_not_the_next_ones(lib, call):  # noqa: F811
    """A launch that the runtime refuses (the legacy stream beside a capture of a stream that waits for it) is that call's error;
    the next call has none."""
    E, h, f, R = 2, 256, 384, 300 if call == "many" else 5
    w = _ffn_weights(E, h, f, 71)
    codes = [t for q, s, _ in w for t in (q, s)]
    x, o, W = _normal((R, h), 72), _offsets([R - 2, 2]), _normal((E, h, f), 73)
    aq, sa = _quantize_rows(x)
    fd, gd = mb.ffn_dims(R, h, f, E), mb.gemm_dims(R, h, f, E)
    ws = _ws(max(mb.moe_ffn_workspace_bytes(fd, 0), mb.moe_gemm_workspace_bytes(gd)))
    q, s = torch.empty_like(aq), torch.empty_like(sa)
    wq, wsc = torch.empty(W.shape, dtype=torch.uint8, device="cuda"), torch.empty((E, 2, 3), dtype=F32, device="cuda")
    C, y = torch.empty((R, f), dtype=BF, device="cuda"), torch.empty_like(x)

    def run():
        if call == "rows":
            mb.moe_quantize_rows_fp8_block(x, R, h, None, 1, R, q, s, stream=0)
        elif call == "weights":
            mb.moe_quantize_weights_fp8_block(W, E, h, f, wq, wsc, stream=0)
        elif call == "forward":
            mb.moe_gated_ffn_fwd(fd, x, o, *codes, None, None, None, y, ws, stream=0)
        else:
            mb.moe_gemm_fp8_block(gd, aq, sa, codes[0], codes[1], o, C, ws, stream=0)

    run()
    torch.cuda.synchronize()
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
    try:
        assert cu.cuStreamBeginCapture_v2(stream, 2) == 0
        with pytest.raises(mb.MoeError) as e:
            run()
        cu.cuStreamEndCapture(stream, ctypes.byref(graph))
        assert e.value.status == mb.MOE_ERR_CUDA
        run()
        torch.cuda.synchronize()
    finally:
        cu.cuStreamDestroy_v2(stream)


@pytest.mark.parametrize("R", [1, 20, 300])
def test_calls_behind_copies_and_other_streams_in_a_graph(lib, R):  # noqa: F811
    """Kernels that may begin early, behind a copy, behind a fill and behind two streams that join."""
    h, f = 512, 384
    w = _ffn_weights(1, h, f, 81)
    codes = [t for q, s, _ in w for t in (q, s)]
    xs = [_normal((R, h), 82 + i) for i in range(4)]
    x, x2, y, C = (torch.empty_like(xs[0]), torch.empty_like(xs[0]), torch.empty_like(xs[0]), torch.empty((R, f), dtype=BF, device="cuda"))
    aq, sa = torch.empty((R, h), dtype=torch.uint8, device="cuda"), torch.empty((h // 128, R), dtype=F32, device="cuda")
    src = torch.empty_like(x)
    fd, gd = mb.ffn_dims(R, h, f), mb.gemm_dims(R, h, f)
    wss = [_ws(mb.moe_ffn_workspace_bytes(fd, 0)), _ws(mb.moe_gemm_workspace_bytes(gd))]
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        x.copy_(src)
        mb.moe_gated_ffn_fwd(fd, x, None, *codes, None, None, None, y, wss[0])
        side.wait_stream(here)
        with torch.cuda.stream(side):
            x2.copy_(src)
            mb.moe_quantize_rows_fp8_block(x2, R, h, None, 1, R, aq, sa)
        C.zero_()
        here.wait_stream(side)
        mb.moe_gemm_fp8_block(gd, aq, sa, codes[0], codes[1], None, C, wss[1])
        x.zero_()

    want = []
    for t in xs:
        src.copy_(t)
        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        want.append((y.clone(), C.clone()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        for t, (a, b) in zip(xs, want):
            src.copy_(t)
            graph.replay()
            assert torch.equal(y, a) and torch.equal(C, b)


def test_host_threads_with_a_stream_each(lib):  # noqa: F811
    """Four threads at once, each with its stream, workspace and sizes: the same bits as alone."""
    E, h, f = 4, 512, 384
    w = _ffn_weights(E, h, f, 84)
    codes = [t for q, s, _ in w for t in (q, s)]
    jobs = []
    for i, R in enumerate((3, 30, 200, 600)):
        fd, gd, o = mb.ffn_dims(R, h, f, E), mb.gemm_dims(R, h, f, E), _offsets([R - 2, 0, 2, 0])
        x, dy = _normal((R, h), 85 + i), _normal((R, h), 185 + i)
        outs = [torch.empty(shape, dtype=BF, device="cuda") for shape in [(R, f)] * 4 + [(R, h)] * 2]
        outs += [torch.empty(q.shape, dtype=F32, device="cuda") for q, _, _ in w]
        q, s = torch.empty((R, h), dtype=torch.uint8, device="cuda"), torch.empty((h // 128, R), dtype=F32, device="cuda")
        wss = [_ws(mb.moe_ffn_workspace_bytes(fd, 0)), _ws(mb.moe_ffn_workspace_bytes(fd, 1)), _ws(mb.moe_gemm_workspace_bytes(gd))]
        jobs.append((R, fd, gd, o, x, dy, outs, q, s, wss, torch.cuda.Stream()))

    def step(R, fd, gd, o, x, dy, outs, q, s, wss, stream):
        A, B, H, C, y, dx = outs[:6]
        mb.moe_quantize_rows_fp8_block(x, R, h, None, 1, R, q, s, stream=stream)
        mb.moe_gemm_fp8_block(gd, q, s, codes[0], codes[1], o, C, wss[2], stream=stream)
        mb.moe_gated_ffn_fwd(fd, x, o, *codes, A, B, H, y, wss[0], stream=stream)
        mb.moe_gated_ffn_bwd(fd, x, dy, o, *codes, A, B, H, dx, *outs[6:], wss[1], stream=stream)

    want = []
    for j in jobs:
        step(*j)
        torch.cuda.synchronize()
        want.append([t.clone() for t in j[6]])
        for t in j[6]:
            t.fill_(3)
    torch.cuda.synchronize()
    errors = []

    def work(j):
        try:
            for _ in range(30):
                step(*j)
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for j, first in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip(first, j[6]))
        assert all(mb.moe_read_device_status(ws) == mb.MOE_OK for ws in j[9])


# ---------------------------------------------------------------- few rows: every cut, every tile
FEW = [([3] * 64, 2048, 1408), ([1] * 8, 4096, 2816), ([9, 0, 1, 16, 0, 2] * 8, 1104, 1552),   # pieces that hold parts of two tiles
       ([32], 4096, 16512), ([17], 4096, 16512), ([40, 3, 0, 5], 2048, 8320), ([12] * 8, 4096, 2816)]   # the tile of 32 rows


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts,K,N", FEW)
def test_product_of_few_rows(lib, counts, K, N, trans, f32):  # noqa: F811
    C, ref, bound = _product(counts, K, N, trans, f32, seed=len(counts) + K + N)
    assert ((C.double() - ref).abs() <= bound).all()


FEW_FFN = [([3, 0, 2, 7, 0, 1, 4, 3] * 8, 2048, 1408), ([1] * 8, 4096, 1408), ([9, 0, 30, 2, 0, 2] * 4, 1088, 2112), ([14] * 8, 2816, 4096)]


@pytest.mark.parametrize("counts,h,f", FEW_FFN)
def test_feed_forward_of_few_rows_cut_inside_tiles(lib, counts, h, f):  # noqa: F811
    E, R = len(counts), sum(counts)
    w, x, o = _ffn_weights(E, h, f, 91), _normal((R, h), 92), _offsets(counts)
    codes = [t for q, s, _ in w for t in (q, s)]
    fd = mb.ffn_dims(R, h, f, E)
    ws = _ws(mb.moe_ffn_workspace_bytes(fd, 0))
    A, B, H = (torch.empty(R, f, dtype=BF, device="cuda") for _ in range(3))
    y = torch.empty_like(x)
    first = None
    for _ in range(20):
        for t in (A, B, H, y):
            t.fill_(3)
        mb.moe_gated_ffn_fwd(fd, x, o, *codes, A, B, H, y, ws)
        got = [t.clone() for t in (A, B, H, y)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    _check_fwd(x, A, B, H, y, w, counts)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK and not ws[:256].any()


# ---------------------------------------------------------------- the gate at its ends
@pytest.mark.parametrize("R", [1, 16, 30, 300])
def test_gate_values_from_one_end_to_the_other(lib, R):  # noqa: F811
    """A from -1e37 to 1e37.  Past A = -87.3 the sigmoid's quotient is 0: silu is off by less than 88.8 * 2^-126 there.  In the
    backward a value of dA or dB that rounds to the other side is off by one bf16 step, 2^-7 of it at most."""
    h, f = 64, 320
    gate = torch.empty(f, device="cuda")  # the values of a block of 128 columns are codes under one scale
    gate[:128] = torch.linspace(-300, -1, 128)
    gate[128:256] = torch.logspace(32, 37, 128) * torch.tensor([1.0, -1.0]).repeat(64)
    gate[256:] = torch.logspace(-6, -1, 64) * torch.tensor([1.0, -1.0]).repeat(32)
    W1 = torch.zeros((1, h, f), dtype=BF, device="cuda")
    W1[0, 0] = gate.to(BF)
    q1, s1, v1 = br.code_weights(W1)
    q3, s3, v3 = br.weights(1, h, f, seed=95)
    q2, s2, v2 = br.weights(1, f, h, seed=96)
    codes = (q1, s1, q3, s3, q2, s2)
    x = _normal((R, h), 97, 2.0 ** -10)
    x[:, 0] = 1 + torch.arange(R, device="cuda") % 128 * 2.0 ** -7
    fd = mb.ffn_dims(R, h, f)
    ws = _ws(max(mb.moe_ffn_workspace_bytes(fd, b) for b in (0, 1)))
    A, B, H = (torch.empty((R, f), dtype=BF, device="cuda") for _ in range(3))
    y = torch.empty_like(x)
    mb.moe_gated_ffn_fwd(fd, x, None, *codes, A, B, H, y, ws)
    v = br.coded_rows(x.double())
    a, b = v @ v1[0], v @ v3[0]
    ea, eb = (11 * 2.0 ** -23 * (v.abs() @ w[0].abs()) for w in (v1, v3))
    hh = br.silu(a) * b
    off = 1.1 * (b.abs() + eb) * ea + br.silu(a).abs() * eb + (16 + a.abs().clamp(max=200)) * 2.0 ** -23 * hh.abs() + 88.8 * 2.0 ** -126 * (b.abs() + eb)
    assert torch.isfinite(H).all() and torch.isfinite(y).all()
    assert ((H.double() - hh).abs() <= off + 2.0 ** -8 * (hh.abs() + off) + 2.0 ** -134).all()
    assert (H[a < -1000] == 0).all()
    # the backward, from A at once
    A[:] = torch.cat([-torch.logspace(36, -3, f // 2, device="cuda"), torch.logspace(-3, 36, f // 2, device="cuda")]).to(BF)
    A[:, :40] = torch.linspace(-120, -60, 40, device="cuda").to(BF)
    B, dy = _normal((R, f), 98), _normal((R, h), 99)
    H = torch.zeros_like(A)
    dx, dW = torch.empty_like(x), [torch.empty(t.shape, dtype=F32, device="cuda") for t in (q1, q3, q2)]
    mb.moe_gated_ffn_bwd(fd, x, dy, None, *codes, A, B, H, dx, *dW, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    dh, aa = br.coded_rows(dy.double()) @ v2[0].t(), A.double()
    sg = torch.sigmoid(aa)
    da, db = br.kept(dh * B.double() * sg * (1 + aa * (1 - sg))), br.kept(dh * aa * sg)
    assert all(torch.isfinite(t).all() for t in (dx, *dW))
    for got, ref in ((dW[0][0], x.double().t() @ da), (dW[1][0], x.double().t() @ db)):
        n = ref.norm(dim=0)  # each column by itself: its A sets its size
        assert ((got.double() - ref).norm(dim=0) <= (2.0 ** -7 + 1e-4) * n + 1e-30).all()
