"""The block-scaled e4m3 operators at the ends of their sizes: codes, weights and
outputs whose last elements lie past 2^31, contractions and rows of a million,
and a workspace that two captured graphs use in turn.  References and
tolerances are those of test_gpu_block_fp8.py, on the rows and groups that lie
last."""
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from tests import block_ref as br
from tests.test_gpu_block_fp8 import BF, F32, _check_fwd, _ffn_bwd, _ffn_fwd, _ffn_weights, _groups, _normal, _offsets, _quantize_rows, _rel, _ws, lib  # noqa: F401

pytestmark = [pytest.mark.gpu]


def _gemm(aq, sa, bq, sb, offsets, R, K, N, E, trans=False, f32=True):
    gd = mb.gemm_dims(R, K, N, E, trans_b=trans, out_f32=f32)
    ws = _ws(mb.moe_gemm_workspace_bytes(gd))
    C = torch.full((R, N), 77.0, dtype=F32 if f32 else BF, device="cuda")
    mb.moe_gemm_fp8_block(gd, aq, sa, bq, sb, offsets, C, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    return C


def _near(C, a, w, K, f32):
    ref = a @ w
    bound = (8 + 3 * -(-K // 128)) * 2.0 ** -23 * (a.abs() @ w.abs()) + (0 if f32 else 2.0 ** -8 * ref.abs())
    return bool(((C.double() - ref).abs() <= bound).all())


def test_row_codes_past_31_bits(lib):  # noqa: F811
    R, n, last = 2 ** 31 // 4096 + 300, 4096, 310
    x = _normal((R, n), 1)
    q, s = _quantize_rows(x)
    rq, rs = br.quantize(x[-last:].double(), 1)
    assert torch.equal(q[-last:].double(), rq) and torch.equal(s[:, -last:].t().double(), rs)
    del x
    bq, sb, w = br.weights(1, n, 16, seed=2)
    C = _gemm(q, s, bq, sb, None, R, n, 16, 1)
    assert _near(C[-last:], br.value(rq, rs, 1), w[0], n, True)


@pytest.mark.parametrize("f32", [False, True])
def test_outputs_past_31_bits(lib, f32):  # noqa: F811
    R, K, N, last = 2 ** 31 // 4096 + 300, 16, 4096, 310
    q, s = _quantize_rows(_normal((R, K), 3))
    bq, sb, w = br.weights(2, K, N, seed=4)
    C = _gemm(q, s, bq, sb, _offsets([R - 200, 150]), R, K, N, 2, f32=f32)
    a = br.value(q[-last:].double(), s[:, -last:].t(), 1)
    assert _near(C[-last:-200], a[:-200], w[0], K, f32) and _near(C[-200:-50], a[-200:-50], w[1], K, f32)
    assert (C[-50:] == 77).all()


def test_weights_past_31_bits(lib):  # noqa: F811
    E, K, N = 38, 4096, 14336  # the last weight's codes begin past 2^31
    W = _normal((E, K, N), 5, K ** -0.5)
    q = torch.empty((E, K, N), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, K // 128, N // 128), dtype=F32, device="cuda")
    mb.moe_quantize_weights_fp8_block(W, E, K, N, q, s)
    rq, rs = br.quantize(W[-1].double(), 128)
    del W
    assert torch.equal(q[-1].view(torch.float8_e4m3fn).double(), rq) and torch.equal(s[-1].double(), rs)
    w = br.value(rq, rs, 128)
    for rows in (3, 17 * E):  # the kernel for few rows, and the one for many
        counts = [0] * (E - 1) + [rows]
        x = _normal((rows, K), 6)
        aq, sa = _quantize_rows(x)
        assert _near(_gemm(aq, sa, q, s, _offsets(counts), rows, K, N, E), br.coded_rows(x.double()), w, K, True)
        x = _normal((rows, N), 7)
        aq, sa = _quantize_rows(x)
        C = _gemm(aq, sa, q, s, _offsets(counts), rows, N, K, E, trans=True)
        assert _near(C, br.coded_rows(x.double()), w.t(), N, True)


def test_feed_forward_past_31_bits(lib):  # noqa: F811
    h, f, last = 64, 8192, 270
    R = 2 ** 31 // f + 300
    x, w = _normal((R, h), 8), _ffn_weights(1, h, f, 9)
    A, B, H, y = _ffn_fwd(x, None, w, f, 1)
    _check_fwd(x[-last:], A[-last:], B[-last:], H[-last:], y[-last:], w, [last])
    dy = _normal((R, h), 10)
    dx, _ = _ffn_bwd(x, dy, None, w, A, B, H, 1, wgrads=False)
    want = br.ffn_bwd(*[t[-last:].double() for t in (x, dy, A, B, H)], *[v[2] for v in w], [slice(0, last)])
    assert _rel(dx[-last:], want[0]) <= 5e-3
    # gradients of weights whose last rows alone count
    dy[:-last] = 0
    _, dW = _ffn_bwd(x, dy, None, w, A, B, H, 1)
    assert _rel(dW[0], want[1]) <= 3e-3 and _rel(dW[1], want[2]) <= 3e-3 and _rel(dW[2], want[3]) <= 2e-5


@pytest.mark.parametrize("rows", [3, 130])
@pytest.mark.parametrize("K,N", [(1 << 20, 16), (16, 1 << 20)])
def test_a_side_of_a_million(lib, rows, K, N):  # noqa: F811
    x = _normal((rows, K), 11)
    aq, sa = _quantize_rows(x)
    W = _normal((1, K, N), 12, K ** -0.5)
    bq, sb, w = br.code_weights(W)
    C = _gemm(aq, sa, bq, sb, None, rows, K, N, 1)
    assert _near(C, br.coded_rows(x.double()), w[0], K, True)
    del C
    wt = W.transpose(1, 2).contiguous()
    bq, sb, w = br.code_weights(wt)
    C = _gemm(aq, sa, bq, sb, None, rows, K, N, 1, trans=True)
    assert _near(C, br.coded_rows(x.double()), w[0].t(), K, True)


def test_two_graphs_on_one_workspace(lib):  # noqa: F811
    """Graphs of few rows and of many, replayed in turn on one workspace, leave its header as the other needs it."""
    E, h, f = 4, 1024, 704
    w = _ffn_weights(E, h, f, 13)
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    rows = (9, 400)
    fds = [mb.ffn_dims(r, h, f, E) for r in rows]
    gd = mb.gemm_dims(rows[0], h, f, E)
    ws = _ws(max(mb.moe_ffn_workspace_bytes(fds[1], 0), mb.moe_gemm_workspace_bytes(gd)))
    os = [_offsets(c) for c in ([2, 0, 6, 1], [100, 30, 0, 270])]
    xs = [_normal((r, h), 14 + r) for r in rows]
    want = [_ffn_fwd(x, o, w, f, E, keep=False)[3] for x, o in zip(xs, os)]
    aq, sa = _quantize_rows(xs[0])
    C0 = _gemm(aq, sa, q1, s1, os[0], rows[0], h, f, E, f32=False)
    ys, C = [torch.empty_like(x) for x in xs], torch.empty_like(C0)
    graphs = []
    for i in range(2):
        def step():
            mb.moe_gated_ffn_fwd(fds[i], xs[i], os[i], q1, s1, q3, s3, q2, s2, None, None, None, ys[i], ws)
            if i == 0:
                mb.moe_gemm_fp8_block(gd, aq, sa, q1, s1, os[0], C, ws)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for _ in range(10):
        for t in (*ys, C):
            t.fill_(3)
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, ys)) and torch.equal(C, C0)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    assert not ws[:256].any()


@pytest.mark.parametrize("counts,h,f", [([30], 1024, 640), ([50], 4096, 1152), ([130, 0, 300], 2048, 256), ([20, 0, 40], 192, 8192)])
def test_shared_tiles_give_the_same_bits_each_time(lib, counts, h, f):  # noqa: F811
    """Few tiles with a long contraction: pieces of a tile are joined in their order, whichever arrives last."""
    E, R = len(counts), sum(counts)
    w, x, dy, o = _ffn_weights(E, h, f, 21), _normal((R, h), 22), _normal((R, h), 23), _offsets(counts)
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    fd = mb.ffn_dims(R, h, f, E)
    ws = _ws(max(mb.moe_ffn_workspace_bytes(fd, b) for b in (0, 1)))
    A, B, H = (torch.empty(R, f, dtype=BF, device="cuda") for _ in range(3))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    first = None
    for _ in range(40):
        for t in (A, B, H, y, dx):
            t.fill_(3)
        mb.moe_gated_ffn_fwd(fd, x, o, q1, s1, q3, s3, q2, s2, A, B, H, y, ws)
        mb.moe_gated_ffn_bwd(fd, x, dy, o, q1, s1, q3, s3, q2, s2, A, B, H, dx, None, None, None, ws)
        got = [t.clone() for t in (A, B, H, y, dx)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    _check_fwd(x, A, B, H, y, w, counts)
    want = br.ffn_bwd(*[t.double() for t in (x, dy, A, B, H)], *[v[2] for v in w], _groups(counts))
    assert _rel(dx, want[0]) <= 5e-3
    assert mb.moe_read_device_status(ws) == mb.MOE_OK and not ws[:256].any()


@pytest.mark.parametrize("rows", [2, 60, 300])
def test_weights_written_just_before(lib, rows):  # noqa: F811
    """Launches that begin early read the weights, offsets and rows that the launches just before them wrote."""
    E, h, f, n = 2, 512, 384, 24
    g = torch.Generator("cuda").manual_seed(31)
    Ws = [torch.empty((n, E, a, b), dtype=BF, device="cuda").normal_(0.0, a ** -0.5, generator=g) for a, b in ((h, f), (h, f), (f, h))]
    xs = torch.empty((n, rows, h), dtype=BF, device="cuda").normal_(0.0, 1.0, generator=g)
    cuts = [(7 * i) % (rows + 1) for i in range(n)]
    offs = torch.tensor([[0, c, rows] for c in cuts], dtype=torch.int32, device="cuda")
    q = [torch.empty(W.shape[1:], dtype=torch.uint8, device="cuda") for W in Ws]
    s = [torch.empty((E, -(-W.shape[2] // 128), -(-W.shape[3] // 128)), dtype=F32, device="cuda") for W in Ws]
    x, o = torch.empty_like(xs[0]), torch.empty_like(offs[0])
    aq, sa = torch.empty((rows, h), dtype=torch.uint8, device="cuda"), torch.empty((h // 128, rows), dtype=F32, device="cuda")
    fd, gd = mb.ffn_dims(rows, h, f, E), mb.gemm_dims(rows, h, f, E)
    ws = _ws(max(mb.moe_ffn_workspace_bytes(fd, 0), mb.moe_gemm_workspace_bytes(gd)))
    y = torch.empty_like(xs)
    C = torch.empty((n, rows, f), dtype=BF, device="cuda")

    def step(i, wait):
        def then():
            if wait:
                torch.cuda.synchronize()
        x.copy_(xs[i])
        o.copy_(offs[i])
        mb.moe_quantize_rows_fp8_block(x, rows, h, None, 1, rows, aq, sa)
        then()
        mb.moe_quantize_weights_fp8_block(Ws[0][i], E, h, f, q[0], s[0])
        then()
        mb.moe_gemm_fp8_block(gd, aq, sa, q[0], s[0], o, C[i], ws)
        then()
        for j in (1, 2):
            mb.moe_quantize_weights_fp8_block(Ws[j][i], *Ws[j].shape[1:], q[j], s[j])
        then()
        mb.moe_gated_ffn_fwd(fd, x, o, q[0], s[0], q[1], s[1], q[2], s[2], None, None, None, y[i], ws)
        then()

    for i in range(n):
        step(i, True)
    want = y.clone(), C.clone()
    for _ in range(5):
        y.fill_(3)
        C.fill_(3)
        for i in range(n):
            step(i, False)
        assert torch.equal(y, want[0]) and torch.equal(C, want[1])
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
