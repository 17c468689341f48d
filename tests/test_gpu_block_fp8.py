"""The e4m3 operators with a float32 scale for each block of 128 against their
64-bit formulas: the quantisers (bit for bit), the grouped product, the gated
feed-forward block in both directions, and the layer calls built from them.

Tolerances.  A product's fp32 sum of K terms has its value off by at most a few
roundings of 2^-23 for each block of 128, relative to the sum S of the terms'
magnitudes: (8 + 3 ceil(K/128)) 2^-23 S covers four partial sums a block in the
tensor core, the scaling and the running sum.  A bf16 store adds 2^-8 of the
value.  H adds the exponential's and the division's few ulps and what A and B
are off.  Behind dA and dB, whose bf16 rounding (2^-8, uniform: 2^-8/sqrt(3) of
the largest, 1.7e-3 in the mean) can fall to either side, results are compared
in the 2-norm: 5e-3, as everywhere in these tests."""
import numpy as np
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests import block_ref as br

pytestmark = [pytest.mark.gpu]

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    return mb.load()


def _normal(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _ws(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _groups(counts):
    o = np.concatenate([[0], np.cumsum(counts)])
    return [slice(int(a), int(b)) for a, b in zip(o[:-1], o[1:])]


def _quantize_rows(x, idx=None, div=1, rows=None):
    rows = x.shape[0] if rows is None else rows
    n = x.shape[1]
    q = torch.full((rows, n), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-n // 128), rows), -1.0, dtype=F32, device="cuda")
    mb.moe_quantize_rows_fp8_block(x, rows, n, idx, div, x.shape[0], q, s)
    return q.view(torch.float8_e4m3fn), s


# ---------------------------------------------------------------- quantisers
@pytest.mark.parametrize("rows,n", [(1, 16), (1, 4096), (3, 128), (37, 144), (300, 2064), (5, 14336), (2000, 272)])
def test_row_codes_bit_exact(lib, rows, n):
    x = _normal((rows, n), rows + n)
    x[rows // 2, : min(n, 128)] = 0  # a block of zeros: scale 1
    # magnitudes from far below e4m3's least code to bf16's largest, and scales that leave the normal range
    x[-1] *= torch.exp2(torch.linspace(-30, 30, n, device="cuda")).to(BF)
    q, s = _quantize_rows(x)
    rq, rs = br.quantize(x.double(), 1)
    assert torch.equal(s.t().double(), rs)
    assert torch.equal(q.double(), rq)


@pytest.mark.parametrize("scale", [2.0 ** -133, 2.0 ** -120, 2.0 ** -99, 2.0 ** -70, 2.0 ** 60, 2.0 ** 110, 2.0 ** 126])
def test_row_codes_at_the_ends_of_the_range(lib, scale):
    x = (_normal((64, 256), 3, dtype=F32).clamp(-1.9, 1.9).double() * scale).to(BF)
    q, s = _quantize_rows(x)
    rq, rs = br.quantize(x.double(), 1)
    assert torch.equal(s.t().double(), rs)
    assert torch.equal(q.double(), rq)


def test_every_quotient_of_two_bf16_rounds_as_division_does(lib):
    """All 128 significands of a block's largest value against every value of the ten binades below it."""
    top = (1 + torch.arange(128, device="cuda") / 128).double()
    v = torch.zeros(11 * 127, dtype=torch.float64, device="cuda")     # 1280 values and zeros, 127 to a block
    v[:1280] = torch.stack([top * 2.0 ** -j for j in range(10)]).reshape(-1)
    x = torch.where(v <= top[:, None], v, 0.0).view(128, 11, 127)
    x = torch.cat([top[:, None, None].expand(128, 11, 1), x], 2).reshape(128, 11 * 128).to(BF)
    q, s = _quantize_rows(x)
    rq, rs = br.quantize(x.double(), 1)
    assert torch.equal(s.t().double(), rs) and torch.equal(q.double(), rq)


def test_row_codes_gathered(lib):
    T, k, n = 97, 3, 400
    x = _normal((T, n), 9)
    idx = torch.randperm(T * k, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.int32)
    q, s = _quantize_rows(x, idx, k, T * k)
    rq, rs = br.quantize(x[idx.long() // k].double(), 1)
    assert torch.equal(q.double(), rq) and torch.equal(s.t().double(), rs)


def test_row_indices_out_of_range_are_recorded(lib):
    mb.moe_clear_device_status(None)
    x, idx = _normal((10, 256), 2), torch.tensor([3, -1, 9, 10, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    q, s = _quantize_rows(x, idx, 1, 5)
    assert mb.moe_read_device_status(None) == mb.MOE_ERR_DEVICE_INDEX
    assert mb.moe_read_device_status(None) == mb.MOE_OK
    rq, _ = br.quantize(x[[3, 9]].double(), 1)
    assert torch.equal(q[[0, 2]].double(), rq)
    bad = torch.tensor([1, 3, 4], device="cuda")
    assert (q.view(torch.uint8)[bad] == 0).all() and (s[:, bad] == 1).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_a_block_that_is_not_finite(lib, what):
    x = _normal((4, 384), 4)
    clean, cs = _quantize_rows(x)
    x[2, 130] = what
    q, s = _quantize_rows(x)
    assert not torch.isfinite(s[1, 2])
    assert not torch.isfinite(q.float()[2, 130] * s[1, 2])
    keep = torch.ones(4, 384, dtype=torch.bool, device="cuda")
    keep[2, 128:256] = False
    assert torch.equal(q.view(torch.uint8)[keep], clean.view(torch.uint8)[keep])
    s[1, 2] = cs[1, 2]
    assert torch.equal(s, cs)


@pytest.mark.parametrize("E,K,N", [(1, 16, 16), (3, 128, 128), (2, 144, 400), (1, 4096, 272), (5, 80, 1040)])
def test_weight_codes_bit_exact(lib, E, K, N):
    W = _normal((E, K, N), K + N, K ** -0.5)
    W[0, : min(K, 128), : min(N, 128)] = 0
    q = torch.empty((E, K, N), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, -(-K // 128), -(-N // 128)), dtype=F32, device="cuda")
    mb.moe_quantize_weights_fp8_block(W, E, K, N, q, s)
    for e in range(E):
        rq, rs = br.quantize(W[e].double(), 128)
        assert torch.equal(s[e].double(), rs)
        assert torch.equal(q[e].view(torch.float8_e4m3fn).double(), rq)


# ---------------------------------------------------------------- the product
def _product(counts, K, N, trans, f32, seed, behind=0, dense=False):
    """Runs the product on random codes; returns (C, reference, bound) with `behind` rows past the last group's."""
    R, E = int(sum(counts)) + behind, len(counts)
    x = _normal((R, K), seed)
    if behind:
        x[R - behind:] = float("nan")
    q, s = br.quantize(x[: R - behind].double(), 1)
    aq = torch.full((R, K), 0x7F, dtype=torch.uint8, device="cuda")
    sa = torch.full((-(-K // 128), R), float("nan"), dtype=F32, device="cuda")
    aq[: R - behind] = q.float().to(torch.float8_e4m3fn).view(torch.uint8)
    sa[:, : R - behind] = s.t().float()
    bq, sb, w = br.weights(E, N if trans else K, K if trans else N, std=K ** -0.5, seed=seed + 1)
    C = torch.full((R, N), 77.0, dtype=F32 if f32 else BF, device="cuda")
    gd = mb.gemm_dims(R, K, N, E, trans_b=trans, out_f32=f32)
    ws = _ws(mb.moe_gemm_workspace_bytes(gd))
    mb.moe_gemm_fp8_block(gd, aq, sa, bq, sb, None if dense else _offsets(counts), C, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    a = br.value(q, s, 1)
    ref, S = torch.empty(R - behind, N, dtype=torch.float64, device="cuda"), torch.empty(R - behind, N, dtype=torch.float64, device="cuda")
    for e, r in enumerate(_groups(counts)):
        m = w[e].t() if trans else w[e]
        ref[r], S[r] = a[r] @ m, a[r].abs() @ m.abs()
    bound = (8 + 3 * -(-K // 128)) * 2.0 ** -23 * S + (0 if f32 else 2.0 ** -8 * ref.abs())
    return C, ref, bound


SHAPES = [
    ([1], 128, 128), ([1], 4096, 272), ([2], 16, 16), ([3], 144, 400), ([17], 272, 144), ([64], 512, 640),
    ([127], 400, 272), ([128], 256, 256), ([129], 384, 528), ([300], 1104, 720), ([1000], 640, 1040),
    ([0, 5, 0, 130, 1, 0], 400, 272), ([33, 0, 64, 1, 200], 1088, 704), ([0, 0, 7], 128, 1408), ([600, 3, 500], 272, 1552),
    ([4] * 64, 2048, 144), ([0] * 63 + [9], 256, 384), ([257, 255, 0, 1], 896, 640),
    ([1, 400, 0, 3], 400, 272), ([2, 0, 290, 1, 70], 1040, 592), ([65], 1408, 2048), ([30] * 9, 640, 272), ([200, 1, 0, 3, 40], 1936, 400),
    ([16], 8320, 400), ([17], 8320, 272), ([48], 8192, 144), ([49], 8192, 144), ([10, 40, 0, 30], 8192, 272), ([12] * 3, 2048, 2064),
    ([16], 272, 128), ([17], 272, 640), ([5, 43, 0], 640, 1040), ([33, 64, 31], 400, 272), ([32] * 4, 640, 528), ([96, 160], 272, 384),
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_product(lib, counts, K, N, trans, f32):
    C, ref, bound = _product(counts, K, N, trans, f32, seed=len(counts) + K + N)
    assert ((C.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts,K,N,behind", [([5], 256, 272, 40), ([130, 0, 20], 400, 144, 1), ([300, 260], 640, 528, 200), ([0, 0], 128, 128, 9)])
def test_product_leaves_rows_behind_the_last_group(lib, counts, K, N, behind, trans):
    C, ref, bound = _product(counts, K, N, trans, False, seed=K + N + behind, behind=behind)
    n = int(sum(counts))
    assert ((C[:n].double() - ref).abs() <= bound).all()
    assert (C[n:] == 77).all()


@pytest.mark.parametrize("rows", [1, 16, 40, 200, 700])
def test_product_without_offsets(lib, rows):
    C, ref, bound = _product([rows], 528, 400, False, True, seed=rows, dense=True)
    assert ((C.double() - ref).abs() <= bound).all()


def test_product_without_rows(lib):
    gd = mb.gemm_dims(0, 128, 128, 2)
    bq, sb, _ = br.weights(2, 128, 128)
    mb.moe_gemm_fp8_block(gd, None, None, bq, sb, _offsets([0, 0]), None, _ws(mb.moe_gemm_workspace_bytes(gd)))
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [9, 300])
def test_offsets_out_of_order_are_recorded(lib, rows):
    """Clamped into order: the results of the groups as clamped, nothing out of bounds."""
    K, N, E = 256, 272, 4
    q, s = br.quantize(_normal((rows, K), 1).double(), 1)
    bq, sb, w = br.weights(E, K, N, seed=2)
    gd = mb.gemm_dims(rows, K, N, E, out_f32=True)
    ws = _ws(mb.moe_gemm_workspace_bytes(gd))
    C = torch.full((rows, N), 77.0, dtype=F32, device="cuda")
    o = torch.tensor([0, 5, 3, rows + 1000, 2], dtype=torch.int32, device="cuda")
    mb.moe_gemm_fp8_block(gd, q.float().to(torch.float8_e4m3fn), s.t().float().contiguous(), bq, sb, o, C, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_ERR_DEVICE_INDEX
    a = br.value(q, s, 1)
    want = torch.cat([a[:5] @ w[0], a[5:] @ w[2]])  # 0, 5, 5, rows, rows
    assert ((C.double() - want).norm() / want.norm()) < 1e-6


def test_rows_that_are_not_finite_stay_apart(lib):
    """A row with an infinity, or a NaN, makes its own outputs not finite and no other's."""
    counts, K, N = [70, 200], 400, 272
    for rows in (None, 8):
        c = counts if rows is None else [3, 5]
        R = sum(c)
        x = _normal((R, K), 5)
        x[1, 7], x[R - 2, 300] = float("inf"), float("nan")
        aq, sa = _quantize_rows(x)
        bq, sb, w = br.weights(2, K, N, seed=6)
        gd = mb.gemm_dims(R, K, N, 2)
        C = torch.empty(R, N, dtype=BF, device="cuda")
        mb.moe_gemm_fp8_block(gd, aq, sa, bq, sb, _offsets(c), C, _ws(mb.moe_gemm_workspace_bytes(gd)))
        bad = torch.zeros(R, dtype=torch.bool, device="cuda")
        bad[[1, R - 2]] = True
        assert torch.equal(torch.isfinite(C).all(1), ~bad) and not torch.isfinite(C[bad]).any()


# ---------------------------------------------------------------- the gated feed-forward block
def _ffn_weights(E, h, f, seed):
    return br.weights(E, h, f, seed=seed), br.weights(E, h, f, seed=seed + 1), br.weights(E, f, h, seed=seed + 2)


def _ffn_fwd(x, offsets, w, f, E, keep=True, y=None):
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    R, h = x.shape
    fd = mb.ffn_dims(R, h, f, E)
    ws = _ws(mb.moe_ffn_workspace_bytes(fd, False))
    A, B, H = (torch.full((R, f), 55.0, dtype=BF, device="cuda") if keep else None for _ in range(3))
    y = torch.full((R, h), 55.0, dtype=BF, device="cuda") if y is None else y
    mb.moe_gated_ffn_fwd(fd, x, offsets, q1, s1, q3, s3, q2, s2, A, B, H, y, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    return A, B, H, y


FFN = [([1], 64, 64), ([1], 4096, 448), ([5], 192, 320), ([64], 256, 128), ([130], 704, 1088), ([700], 320, 640),
       ([0, 9, 0, 33, 1], 448, 704), ([140, 0, 256, 3], 1088, 320), ([3] * 64, 128, 192), ([513, 129], 256, 2112),
       ([16], 128, 8256), ([17], 320, 448), ([48], 192, 8256), ([20, 0, 40], 704, 320), ([40, 7, 0, 17], 256, 8192)]


def _check_fwd(x, A, B, H, y, w, counts):
    (_, _, w1), (_, _, w3), (_, _, w2) = w
    h, f = x.shape[1], A.shape[1]
    hb, fb = (8 + 3 * -(-h // 128)) * 2.0 ** -23, (8 + 3 * -(-f // 128)) * 2.0 ** -23
    for e, r in enumerate(_groups(counts)):
        if r.stop == r.start:
            continue
        v = br.coded_rows(x[r].double())
        a, b, ea, eb = v @ w1[e], v @ w3[e], hb * (v.abs() @ w1[e].abs()), hb * (v.abs() @ w3[e].abs())
        assert ((A[r].double() - a).abs() <= ea + 2.0 ** -8 * a.abs()).all()
        assert ((B[r].double() - b).abs() <= eb + 2.0 ** -8 * b.abs()).all()
        hh = br.silu(a) * b
        # |silu'| < 1.1; the exponential, the quotient and the products: 16 ulps; the exponential's argument adds |a| of them
        off = 1.1 * (b.abs() + eb) * ea + br.silu(a).abs() * eb + (16 + a.abs()) * 2.0 ** -23 * hh.abs()
        assert ((H[r].double() - hh).abs() <= off + 2.0 ** -8 * (hh.abs() + off)).all()
        u = br.coded_rows(H[r].double())
        yy = u @ w2[e]
        assert ((y[r].double() - yy).abs() <= fb * (u.abs() @ w2[e].abs()) + 2.0 ** -8 * yy.abs()).all()


@pytest.mark.parametrize("counts,h,f", FFN)
def test_ffn_forward(lib, counts, h, f):
    x, E = _normal((sum(counts), h), h + f), len(counts)
    w = _ffn_weights(E, h, f, h + 3 * f)
    A, B, H, y = _ffn_fwd(x, _offsets(counts), w, f, E)
    _check_fwd(x, A, B, H, y, w, counts)
    _, _, _, y2 = _ffn_fwd(x, _offsets(counts), w, f, E, keep=False)
    assert torch.equal(y, y2)
    if E == 1:
        assert torch.equal(y, _ffn_fwd(x, None, w, f, E)[3])


@pytest.mark.parametrize("counts,behind", [([4, 3], 6), ([150, 0, 20], 90)])
def test_ffn_leaves_rows_behind_the_last_group(lib, counts, behind):
    h, f, E, n = 320, 448, len(counts), sum(counts)
    x = _normal((n + behind, h), 3)
    x[n:] = float("nan")
    w = _ffn_weights(E, h, f, 8)
    A, B, H, y = _ffn_fwd(x, _offsets(counts), w, f, E)
    _check_fwd(x, A, B, H, y, w, counts)
    for t in (A, B, H, y):
        assert (t[n:] == 55).all()
    dy = _normal((n + behind, h), 4)
    dy[n:] = float("nan")
    for t in (A, B, H):
        t[n:] = float("inf")
    dx, dW = _ffn_bwd(x, dy, _offsets(counts), w, A, B, H, E)
    assert (dx[n:] == 55).all()
    _check_bwd(x, dy, A, B, H, w, counts, dx, dW, n)


def _ffn_bwd(x, dy, offsets, w, A, B, H, E, dtype=F32, wgrads=True):
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    R, h = x.shape
    f = A.shape[1]
    fd = mb.ffn_dims(R, h, f, E, dw_bf16=dtype == BF)
    ws = _ws(mb.moe_ffn_workspace_bytes(fd, True))
    dx = torch.full((R, h), 55.0, dtype=BF, device="cuda")
    dW = [torch.full(q.shape, 55.0, dtype=dtype, device="cuda") if wgrads else None for q in (q1, q3, q2)]
    mb.moe_gated_ffn_bwd(fd, x, dy, offsets, q1, s1, q3, s3, q2, s2, A, B, H, dx, *dW, ws)
    assert mb.moe_read_device_status(ws) == mb.MOE_OK
    return dx, dW


def _rel(a, b):
    n = b.norm()
    return float((a.double() - b).norm() / n) if n > 0 else float((a.double() - b).norm())


def _check_bwd(x, dy, A, B, H, w, counts, dx, dW, n=None):
    n = x.shape[0] if n is None else n
    args = [t[:n].double() for t in (x, dy, A, B, H)]
    want = br.ffn_bwd(*args, *[v[2] for v in w], _groups(counts))
    assert _rel(dx[:n], want[0]) <= 5e-3
    lim = 5e-3 if dW[0].dtype == BF else 3e-3   # dA, dB in bf16; and the gradient's own rounding
    assert _rel(dW[0], want[1]) <= lim and _rel(dW[1], want[2]) <= lim
    assert _rel(dW[2], want[3]) <= (3e-3 if dW[0].dtype == BF else 2e-5)
    for e, r in enumerate(_groups(counts)):
        if r.stop == r.start:
            assert all((g[e] == 0).all() for g in dW)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("counts,h,f", FFN)
def test_ffn_backward(lib, counts, h, f, dtype):
    R, E = sum(counts), len(counts)
    x, dy, A, B = (_normal(s, h + i) for i, s in enumerate([(R, h), (R, h), (R, f), (R, f)]))
    H = (br.silu(A.double()) * B.double()).to(BF)
    w = _ffn_weights(E, h, f, 2 * h + f)
    dx, dW = _ffn_bwd(x, dy, _offsets(counts), w, A, B, H, E, dtype)
    _check_bwd(x, dy, A, B, H, w, counts, dx, dW)
    dx2, _ = _ffn_bwd(x, dy, _offsets(counts), w, A, B, H, E, dtype, wgrads=False)
    assert torch.equal(dx, dx2)
    if E == 1:
        dx3, dW3 = _ffn_bwd(x, dy, None, w, A, B, H, E, dtype)
        assert torch.equal(dx, dx3) and all(torch.equal(a, b) for a, b in zip(dW, dW3))


def test_ffn_gradient_against_differences(lib):
    """<dx, v> and <dW, V> against central differences of <y, dy> in 64 bits at the coded weights.  The kernel's x is coded
    exactly (its values are codes under a scale of 1), so the forward's function is the same but for H's codes; dy, dA and
    dB lose up to 2^-4 of each value to their codes, independent of sign: 2^-4 / sqrt(3) / sqrt(terms) of the sum, under
    3% of |dx| |v| by a wide margin."""
    R, h, f = 64, 256, 192
    w = _ffn_weights(1, h, f, 71)
    w1, w3, w2 = (v[2][0] for v in w)
    g = torch.Generator("cuda").manual_seed(5)
    x = br.e4m3(torch.randn(R, h, generator=g, device="cuda", dtype=torch.float64))
    x[:, ::128] = 448 * 2.0 ** -8
    x = br.e4m3(x * 2.0 ** 8) * 2.0 ** -8
    dy = torch.randn(R, h, generator=g, device="cuda").to(BF)
    xb = x.to(BF)
    A, B, H, _ = _ffn_fwd(xb, None, w, f, 1)
    dx, dW = _ffn_bwd(xb, dy, None, w, A, B, H, 1)

    def loss(x, w1, w3, w2):
        a, b = x @ w1, x @ w3
        return float(((br.silu(a) * b) @ w2 * dy.double()).sum())

    base, grads = [xb.double(), w1, w3, w2], [dx.double(), dW[0][0].double(), dW[1][0].double(), dW[2][0].double()]
    for i in range(4):
        v = grads[i] + grads[i].norm() / grads[i].numel() ** 0.5 * torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-4 * float(base[i].norm() / v.norm())
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + eps * v, base[i] - eps * v
        slope = (loss(*hi) - loss(*lo)) / (2 * eps)
        assert abs(slope - float((grads[i] * v).sum())) <= 0.03 * float(grads[i].norm() * v.norm()), i


def test_ffn_without_rows(lib):
    w = _ffn_weights(2, 128, 192, 1)
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    fd = mb.ffn_dims(0, 128, 192, 2)
    ws = _ws(mb.moe_ffn_workspace_bytes(fd, True))
    dW = [torch.full(q.shape, 5.0, dtype=F32, device="cuda") for q in (q1, q3, q2)]
    o = _offsets([0, 0])
    mb.moe_gated_ffn_fwd(fd, None, o, q1, s1, q3, s3, q2, s2, None, None, None, None, ws)
    mb.moe_gated_ffn_bwd(fd, None, None, o, q1, s1, q3, s3, q2, s2, None, None, None, None, *dW, ws)
    assert all((g == 0).all() for g in dW)


def test_ffn_of_a_next_expert_that_is_not_finite(lib):
    """An expert whose rows hold infinities leaves the weight gradients of the one before it alone."""
    counts, h, f = [70, 90], 256, 192
    R = sum(counts)
    x, dy, A, B = (_normal(s, 30 + i) for i, s in enumerate([(R, h), (R, h), (R, f), (R, f)]))
    H = (br.silu(A.double()) * B.double()).to(BF)
    w = _ffn_weights(2, h, f, 33)
    _, clean = _ffn_bwd(x, dy, _offsets(counts), w, A, B, H, 2)
    for t in (x, dy, H):
        t[counts[0]] = float("inf")
    dx, dW = _ffn_bwd(x, dy, _offsets(counts), w, A, B, H, 2)
    assert all(torch.equal(a[0], b[0]) for a, b in zip(clean, dW))
    assert torch.isfinite(dx[: counts[0]]).all() and not torch.isfinite(dx[counts[0]]).any()


# ---------------------------------------------------------------- together, streams, graphs
def test_quantise_then_ffn_as_a_program_runs_them(lib):
    """Weights quantised by the library, two steps on one workspace of the largest size, on another stream and in a graph."""
    E, h, f, R = 4, 256, 320, 300
    Ws = [_normal((E, a, b), 50 + i, a ** -0.5) for i, (a, b) in enumerate([(h, f), (h, f), (f, h)])]
    w = []
    for W in Ws:
        q = torch.empty(W.shape, dtype=torch.uint8, device="cuda")
        s = torch.empty((E, -(-W.shape[1] // 128), -(-W.shape[2] // 128)), dtype=F32, device="cuda")
        mb.moe_quantize_weights_fp8_block(W, *W.shape, q, s)
        rq, rs, v = br.code_weights(W)
        assert torch.equal(q, rq.view(torch.uint8)) and torch.equal(s, rs)
        w.append((q, s, v))
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    fd = mb.ffn_dims(R, h, f, E)
    ws = _ws(max(mb.moe_ffn_workspace_bytes(fd, b) for b in (0, 1)))
    counts = [100, 0, 150, 50]
    x, dy, o = _normal((R, h), 1), _normal((R, h), 2), _offsets(counts)
    A, B, H = (torch.empty(R, f, dtype=BF, device="cuda") for _ in range(3))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dW = [torch.empty(W.shape, dtype=F32, device="cuda") for W in Ws]

    def step():
        mb.moe_gated_ffn_fwd(fd, x, o, q1, s1, q3, s3, q2, s2, A, B, H, y, ws)
        mb.moe_gated_ffn_bwd(fd, x, dy, o, q1, s1, q3, s3, q2, s2, A, B, H, dx, *dW, ws)

    step()
    _check_fwd(x, A, B, H, y, w, counts)
    _check_bwd(x, dy, A, B, H, w, counts, dx, dW)
    first = [t.clone() for t in (y, dx, *dW)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in (y, dx, *dW):
            t.fill_(3)
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, *dW)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (y, dx, *dW):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, *dW)))
    x2 = _normal((R, h), 91)
    x.copy_(x2)
    o.copy_(_offsets([0, 120, 100, 80]))
    graph.replay()
    _check_fwd(x, A, B, H, y, w, [0, 120, 100, 80])
    assert mb.moe_read_device_status(ws) == mb.MOE_OK


def test_two_streams_with_a_workspace_each(lib):
    E, h, f, R = 3, 512, 384, 90
    w = _ffn_weights(E, h, f, 17)
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    fd, o = mb.ffn_dims(R, h, f, E), _offsets([30, 20, 40])
    xs = [_normal((R, h), 60 + i) for i in range(2)]
    want = [_ffn_fwd(x, o, w, f, E, keep=False)[3] for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [_ws(mb.moe_ffn_workspace_bytes(fd, 0)) for _ in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            mb.moe_gated_ffn_fwd(fd, xs[i], o, q1, s1, q3, s3, q2, s2, None, None, None, ys[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, ys))


@pytest.mark.parametrize("n", [1, 2, 3])
def test_injected_launch_failure(lib, n):
    w = _ffn_weights(1, 128, 128, 1)
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    fd = mb.ffn_dims(4, 128, 128)
    x, ws = _normal((4, 128), 1), _ws(mb.moe_ffn_workspace_bytes(fd, 0))
    y = torch.empty_like(x)
    mb.moe_test_fail_launch_after(n)
    with pytest.raises(mb.MoeError) as e:
        mb.moe_gated_ffn_fwd(fd, x, None, q1, s1, q3, s3, q2, s2, None, None, None, y, ws)
    assert e.value.status == mb.MOE_ERR_CUDA
    mb.moe_gated_ffn_fwd(fd, x, None, q1, s1, q3, s3, q2, s2, None, None, None, y, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, _ffn_fwd(x, None, w, 128, 1)[3])


# ---------------------------------------------------------------- the layer
def _layer(T, h, f, E, k, capacity=0, seed=0):
    d = mb.dims(T, h, f, E, k, capacity=capacity)
    w = _ffn_weights(E, h, f, seed)
    x, dy, Wg = _normal((T, h), seed + 5), _normal((T, h), seed + 6), _normal((h, E), seed + 7, h ** -0.5, F32)
    return d, w, x, dy, Wg


def _run_layer(d, w, x, dy, Wg):
    (q1, s1, _), (q3, s3, _), (q2, s2, _) = w
    saved = _ws(mb.moe_saved_bytes(d))
    wf, wb = (_ws(mb.moe_workspace_bytes(d, op)) for op in (mb.OP_LAYER_FWD_FP8_BLOCK, mb.OP_LAYER_BWD_FP8_BLOCK))
    y, dx, dWg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(Wg)
    dW = [torch.empty(q.shape, dtype=F32, device="cuda") for q in (q1, q3, q2)]
    mb.moe_layer_fwd_fp8_block(d, x, Wg, None, q1, s1, q3, s3, q2, s2, y, saved, wf)
    mb.moe_layer_bwd_fp8_block(d, x, dy, Wg, q1, s1, q3, s3, q2, s2, saved, dx, dWg, *dW, wb)
    assert mb.moe_read_device_status(wf) == mb.MOE_OK and mb.moe_read_device_status(wb) == mb.MOE_OK

    def view(name, shape, dtype):
        off = mb.moe_saved_view(d, saved, name) - saved.data_ptr()
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        return saved[off:off + n].view(dtype).view(shape)

    return y, dx, dWg, dW, view


@pytest.mark.parametrize("T,h,f,E,k,cap", [(1, 128, 192, 4, 2, 0), (33, 256, 128, 8, 2, 0), (300, 320, 448, 8, 3, 0), (700, 256, 320, 5, 1, 0), (200, 128, 192, 4, 2, 60)])
def test_layer(lib, T, h, f, E, k, cap):
    d, w, x, dy, Wg = _layer(T, h, f, E, k, cap, seed=T)
    y, dx, dWg, dW, view = _run_layer(d, w, x, dy, Wg)
    counts = view("counts", (E,), torch.int32).cpu().numpy()
    R = T * k
    n = int(counts.sum())
    psrc, pdst = view("perm_src", (R,), torch.int32).long(), view("perm_dst", (R,), torch.int32).long()
    gates = view("gates", (T, k), F32)
    A, B, H = (view(m, (R, f), BF) for m in "ABH")
    O, xp = view("O", (R, h), BF), view("x_perm", (R, h), BF)
    assert torch.equal(xp[:n], x[psrc[:n] // k])
    _check_fwd(xp[:n], A[:n], B[:n], H[:n], O[:n], w, counts)
    slot = torch.where(pdst >= 0, pdst, 0).view(T, k)
    wts = gates.double() * (pdst.view(T, k) >= 0)
    want = (O[:n].double()[slot.clamp(max=max(n - 1, 0))] * wts[..., None]).sum(1)
    mag = (O[:n].double()[slot.clamp(max=max(n - 1, 0))] * wts[..., None]).abs().sum(1)
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + k * 2.0 ** -22 * mag).all()
    # the backward, from what the forward kept
    dO = (gates.view(-1)[psrc[:n]][:, None] * dy[psrc[:n] // k].float()).to(BF)
    dxp, g1, g3, g2 = br.ffn_bwd(*[t[:n].double() for t in (xp, dO, A, B, H)], *[v[2] for v in w], _groups(counts))
    for got, ref in zip(dW, (g1, g3, g2)):
        assert _rel(got, ref) <= 5e-3
    dg = torch.zeros(R, dtype=torch.float64, device="cuda")
    dg[psrc[:n]] = (dy[psrc[:n] // k].double() * O[:n].double()).sum(1)
    dg = dg.view(T, k)
    dl = gates.double() * (dg - (gates.double() * dg).sum(1, keepdim=True))
    idx = view("topk_idx", (T, k), torch.int32).long()
    dense = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_add_(1, idx, dl)
    want = torch.zeros(T, h, dtype=torch.float64, device="cuda").index_add_(0, psrc[:n] // k, dxp) + dense @ Wg.double().t()
    assert _rel(dx, want) <= 5e-3
    ref = x.double().t() @ dense
    assert float((dWg.double() - ref).norm()) <= 1e-2 * float(ref.norm()) + 1e-5 * float(x.double().norm() * dg.norm())


def test_layer_of_one_expert_each_is_the_feed_forward_block(lib):
    """Top 1 has gates of 1: the layer's experts get the calls' own rows, bit for bit."""
    T, h, f, E = 260, 256, 320, 4
    d, w, x, dy, Wg = _layer(T, h, f, E, 1, seed=3)
    y, dx, dWg, dW, view = _run_layer(d, w, x, dy, Wg)
    psrc, o = view("perm_src", (T,), torch.int32).long(), view("offsets", (E + 1,), torch.int32)
    A, B, H, yp = _ffn_fwd(x[psrc].contiguous(), o, w, f, E)
    assert torch.equal(y[psrc], yp)
    dxp, dWp = _ffn_bwd(x[psrc].contiguous(), dy[psrc].contiguous(), o, w, A, B, H, E)
    assert torch.equal(dx[psrc], dxp)
    assert all(torch.equal(a, b) for a, b in zip(dW, dWp))


def test_layer_is_near_the_bf16_layer(lib):
    """On weights whose values are their codes' the two layers differ by the activations' codes: 2^-4 / sqrt(3) of a value at
    most, 2.6% in the mean of a uniform significand; three codings in a row (x, H and the products' cross terms) stay under 8%."""
    T, h, f, E, k = 400, 256, 384, 8, 2
    d, w, x, dy, Wg = _layer(T, h, f, E, k, seed=12)
    y, dx, dWg, dW, view = _run_layer(d, w, x, dy, Wg)
    W = [v[2].to(BF) for v in w]
    saved, wf, wb = _ws(mb.moe_saved_bytes(d)), _ws(mb.moe_workspace_bytes(d, mb.OP_LAYER_FWD)), _ws(mb.moe_workspace_bytes(d, mb.OP_LAYER_BWD))
    y2, dx2, dWg2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(Wg)
    dW2 = [torch.empty_like(g) for g in dW]
    mb.moe_layer_fwd(d, x, Wg, None, *W, y2, saved, wf)
    mb.moe_layer_bwd(d, x, dy, Wg, *W, saved, dx2, dWg2, *dW2, wb)
    for a, b in [(y, y2), (dx, dx2)] + list(zip(dW, dW2)):
        assert _rel(a, b.double()) < 0.08
