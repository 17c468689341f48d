"""The norms around the block (moe_block_norm_fwd, moe_block_norm_bwd) against
a plain 64-bit implementation, and the gradients against differences.

Tolerances.  Everything is fp32 inside and rounded once on the way out: bf16
outputs have a relative error of at most 2^-8 for each element (half a step of
8 significant bits; plus the fp32 sums), fp32 ones of a few 2^-24 for each operation.  Forward: u is the norm of
the stored r_out, so with a bf16 residual the reference takes the kernel's
r_out.  Per element |err| <= 2^-8 |ref| + 2e-6 * row scale in bf16, and
2e-6 * row scale in fp32.  Column sums run over T rows in fp32: relative L2
2e-6 * sqrt(T) of the sum of magnitudes would be a worst case; their terms'
errors are independent, so 1e-5 of the L2 norm is used (T <= 1100 here).
"""
import pytest
import torch

from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild

pytestmark = pytest.mark.gpu

EPS = 1e-5
KINDS = {"none": mb.GATE_NONE, "channel": mb.GATE_CHANNEL, "token": mb.GATE_TOKEN}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mbuild.build()
    return mb.load()


def make(T, h, f32, gate, post=True, pre=True, first=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    res = torch.float32 if f32 else torch.bfloat16
    v = {"r": (2 * n(T, h)).to(res), "y": None if first else (0.7 * n(T, h)).bfloat16(),
         "w_post": 1 + 0.1 * n(h) if post and not first else None, "w_pre": 1 + 0.1 * n(h) if pre else None,
         "gate": None if first else {"none": None, "channel": 0.5 * n(h), "token": torch.sigmoid(n(T))}[gate],
         "du": n(T, h).bfloat16() if pre else None, "dr_out": n(T, h).to(res)}
    return v


def rms(v):
    return torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def forward64(v, alpha, beta, gate, stored=None):
    """r_out, u of the formula; `stored` (the stored r_out) feeds the second norm where given."""
    d = {n: None if t is None else t.double() for n, t in v.items()}
    r = d["r"]
    if d["y"] is not None:
        z = d["y"] if d["w_post"] is None else d["y"] / rms(d["y"]) * d["w_post"]
        if d["gate"] is not None:
            z = z * (d["gate"][:, None] if gate == "token" else d["gate"])
        r = alpha * d["r"] + beta * z
    s = r if stored is None else stored.double()
    return r, None if d["w_pre"] is None else s / rms(s) * d["w_pre"]


def dims(T, h, f32, gate, alpha, beta):
    return mb.norm_dims(T, h, res_f32=f32, gate=KINDS[gate], eps=EPS, alpha=alpha, beta=beta)


def cuda(v):
    return {n: None if t is None else t.cuda() for n, t in v.items()}


def run_fwd(nd, v, stream=None):
    c = cuda(v)
    r_out = None if v["y"] is None else torch.full_like(c["r"], 9.0)
    u = None if v["w_pre"] is None else torch.full(c["r"].shape, 9.0, dtype=torch.bfloat16, device="cuda")
    mb.moe_block_norm_fwd(nd, c["r"], c["y"], c["w_post"], c["gate"], c["w_pre"], r_out, u, stream=stream)
    torch.cuda.synchronize()
    return None if r_out is None else r_out.cpu(), None if u is None else u.cpu()


def run_bwd(nd, v, gate):
    """v["r"] is taken for r_out."""
    c = cuda(v)
    like = lambda t: None if t is None else torch.full_like(t, 9.0)  # noqa: E731
    out = {"dr": like(c["r"]), "dy": like(c["y"]), "dw_post": like(c["w_post"]), "dgate": like(c["gate"]),
           "dw_pre": like(c["w_pre"])}
    ws = torch.full((mb.moe_norm_workspace_bytes(nd),), 0xFF, dtype=torch.uint8, device="cuda")
    mb.moe_block_norm_bwd(nd, c["r"] if v["w_pre"] is not None else None, c["y"], c["w_post"], c["gate"], c["w_pre"],
                          c["du"], c["dr_out"], out["dr"], out["dy"], out["dw_post"], out["dgate"], out["dw_pre"], ws)
    torch.cuda.synchronize()
    return {n: None if t is None else t.cpu() for n, t in out.items()}


def backward64(v, alpha, beta, gate):
    """Reverse mode by torch's autograd on the 64-bit formula, with r_out a leaf of the second norm."""
    leaf = {n: None if t is None else t.double().clone().requires_grad_(True) for n, t in v.items()}
    G = torch.zeros(v["r"].shape, dtype=torch.float64) if v["dr_out"] is None else v["dr_out"].double()
    out = {}
    if v["w_pre"] is not None:
        u = leaf["r"] / rms(leaf["r"]) * leaf["w_pre"]
        gr, out["dw_pre"] = torch.autograd.grad(u, (leaf["r"], leaf["w_pre"]), v["du"].double())
        G = G + gr
    if v["y"] is None:
        return dict(out, dr=G)
    out["dr"] = alpha * G
    z = leaf["y"] if v["w_post"] is None else leaf["y"] / rms(leaf["y"]) * leaf["w_post"]
    if v["gate"] is not None:
        z = z * (leaf["gate"][:, None] if gate == "token" else leaf["gate"])
    names = [n for n in ("y", "w_post", "gate") if v[n] is not None]
    for n, t in zip(names, torch.autograd.grad(beta * z, [leaf[n] for n in names], G)):
        out["d" + n] = t
    return out


def close(got, ref, what):
    got64 = got.double()
    scale = ref.abs().amax(-1, keepdim=True)
    lim = 2e-6 * scale + (2.0 ** -8 * ref.abs() if got.dtype == torch.bfloat16 else 0.0)
    worst = ((got64 - ref).abs() - lim).max().item()
    assert worst <= 0, (what, worst)


def close_sum(got, ref, what):
    err = ((got.double() - ref).norm() / ref.norm().clamp_min(1e-300)).item()
    assert err <= 1e-5, (what, err)


SIZES = [(1, 8), (1, 64), (3, 520), (5, 1024), (7, 6400), (33, 2056), (40, 4096), (2, 8192), (1100, 256), (9, 8184),
         (2000, 768), (650, 4352), (11, 5120), (310, 4096), (613, 5128), (477, 7176)]  # other numbers of threads and of rows side by side


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gate", list(KINDS))
@pytest.mark.parametrize("T,h", SIZES)
def test_forward(T, h, gate, f32):
    v = make(T, h, f32, gate, seed=T + h)
    r_out, u = run_fwd(dims(T, h, f32, gate, 1.25, 0.5), v)
    ref_r, _ = forward64(v, 1.25, 0.5, gate)
    close(r_out, ref_r, "r_out")
    close(u, forward64(v, 1.25, 0.5, gate, stored=r_out)[1], "u")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gate", list(KINDS))
@pytest.mark.parametrize("T,h", SIZES)
def test_backward(T, h, gate, f32):
    v = make(T, h, f32, gate, seed=T + h + 1)
    got, ref = run_bwd(dims(T, h, f32, gate, 1.25, 0.5), v, gate), backward64(v, 1.25, 0.5, gate)
    close(got["dr"], ref["dr"], "dr")
    close(got["dy"], ref["dy"], "dy")
    for n in ("dw_post", "dw_pre", "dgate"):
        if got[n] is not None:
            close_sum(got[n], ref[n], n)


PARTS = [dict(post=False), dict(pre=False), dict(post=False, pre=False), dict(first=True)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gate", list(KINDS))
@pytest.mark.parametrize("parts", PARTS, ids=["no_post", "no_pre", "residual_only", "first_norm"])
def test_optional_parts(parts, gate, f32):
    check_parts(37, 1032, parts, gate, f32)


@pytest.mark.parametrize("T,h,f32", [(700, 1536, False), (310, 4096, True), (307, 5120, False), (309, 7168, False), (5, 6400, True)])
@pytest.mark.parametrize("parts", PARTS, ids=["no_post", "no_pre", "residual_only", "first_norm"])
def test_optional_parts_of_longer_rows(parts, T, h, f32):
    check_parts(T, h, parts, "channel", f32)


def check_parts(T, h, parts, gate, f32):
    v = make(T, h, f32, gate, seed=5, **parts)
    nd = dims(T, h, f32, gate, 0.75, 2.0)
    r_out, u = run_fwd(nd, v)
    ref_r, ref_u = forward64(v, 0.75, 2.0, gate, stored=r_out)
    if r_out is not None:
        close(r_out, ref_r, "r_out")
    if u is not None:
        close(u, ref_u, "u")
    for without in (False, True):  # with and without a gradient of r_out's other uses
        if without and v["w_pre"] is None:
            continue
        w = dict(v, dr_out=None) if without else v
        got, ref = run_bwd(nd, w, gate), backward64(w, 0.75, 2.0, gate)
        close(got["dr"], ref["dr"], "dr")
        if v["y"] is not None:
            close(got["dy"], ref["dy"], "dy")
        for n in ("dw_post", "dw_pre", "dgate"):
            if got[n] is not None:
                close_sum(got[n], ref[n], n)


@pytest.mark.parametrize("gate", list(KINDS))
def test_gradients_against_differences(gate):
    """The loss sum(du u) + sum(dr_out r_out) of the 64-bit forward, moved by +-1e-5 along a random direction of each
    input; the difference quotient's own error is about 1e-9 of the loss's scale, the gradients' 2^-8 (dy) or 1e-6."""
    T, h, alpha, beta = 6, 264, 1.25, 0.5
    v = make(T, h, True, gate, seed=8)
    r_out = forward64(v, alpha, beta, gate)[0].float()
    got = run_bwd(dims(T, h, True, gate, alpha, beta), dict(v, r=r_out), gate)
    gen = torch.Generator().manual_seed(9)

    def loss(w):
        r, u = forward64(w, alpha, beta, gate)
        return (w["du"].double() * u).sum() + (w["dr_out"].double() * r).sum()

    for name, grad in (("r", "dr"), ("y", "dy"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("gate", "dgate")):
        if v[name] is None:
            continue
        dirn = torch.randn(v[name].shape, generator=gen, dtype=torch.float64)
        moved = [loss(dict(v, **{name: v[name].double() + s * dirn})) for s in (1e-5, -1e-5)]
        num = ((moved[0] - moved[1]) / 2e-5).item()
        ana = (got[grad].double() * dirn).sum().item()
        size = (got[grad].double().norm() * dirn.norm()).item()
        tol = (2.0 ** -8 if grad == "dy" else 1e-5) * size / dirn.numel() ** 0.5 * 4 + 1e-6 * abs(num)
        assert abs(num - ana) <= tol, (name, num, ana, tol)


@pytest.mark.parametrize("f32", [False, True])
def test_in_place(f32):
    T, h = 50, 1536
    v = cuda(make(T, h, f32, "token", seed=12))
    nd = dims(T, h, f32, "token", 1.25, 0.5)
    want, u, u2 = torch.empty_like(v["r"]), torch.empty_like(v["y"]), torch.empty_like(v["y"])
    mb.moe_block_norm_fwd(nd, v["r"], v["y"], v["w_post"], v["gate"], v["w_pre"], want, u)
    r = v["r"].clone()
    mb.moe_block_norm_fwd(nd, r, v["y"], v["w_post"], v["gate"], v["w_pre"], r, u2)
    assert torch.equal(r, want) and torch.equal(u, u2)
    ws = torch.zeros(mb.moe_norm_workspace_bytes(nd), dtype=torch.uint8, device="cuda")
    outs = []
    for dr in (torch.empty_like(v["r"]), v["dr_out"].clone()):
        src = v["dr_out"] if not outs else dr
        o = [torch.empty_like(v["y"]), torch.empty_like(v["w_post"]), torch.empty_like(v["gate"]), torch.empty_like(v["w_pre"])]
        mb.moe_block_norm_bwd(nd, r, v["y"], v["w_post"], v["gate"], v["w_pre"], v["du"], src, dr, *o, ws)
        outs.append([dr] + o)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_zero_rows_zero_gates_and_rows_that_are_not_finite():
    T, h = 12, 640
    v = make(T, h, False, "token", seed=13)
    v["r"][2] = 0
    v["y"][2] = 0
    v["gate"][5] = 0
    clean = make(T, h, False, "token", seed=13)
    v["y"][9, 3] = float("nan")
    v["r"][10, 600] = float("inf")
    nd = dims(T, h, False, "token", 1.0, 1.0)
    r_out, u = run_fwd(nd, v)
    assert (r_out[2] == 0).all() and (u[2] == 0).all()
    assert torch.equal(r_out[5], v["r"][5])
    base_r, base_u = run_fwd(nd, clean)
    rest = [t for t in range(T) if t not in (2, 5, 9, 10)]
    assert torch.equal(r_out[rest], base_r[rest]) and torch.equal(u[rest], base_u[rest])
    got, ref = run_bwd(nd, v, "token"), backward64(v, 1.0, 1.0, "token")
    fine = [t for t in range(T) if t not in (9, 10)]
    close(got["dr"][fine], ref["dr"][fine], "dr")
    close(got["dy"][fine], ref["dy"][fine], "dy")
    assert (got["dy"][5] == 0).all()
    assert ((got["dgate"].double() - ref["dgate"])[fine].abs() <= 1e-5 * h ** 0.5 * 4).all()


def test_no_rows():
    nd = dims(0, 512, False, "channel", 1.0, 1.0)
    w = torch.ones(512, device="cuda")
    mb.moe_block_norm_fwd(nd, None, None, w, w, w, None, None)
    ws = torch.zeros(mb.moe_norm_workspace_bytes(nd), dtype=torch.uint8, device="cuda")
    outs = [torch.full((512,), 9.0, device="cuda") for _ in range(3)]
    mb.moe_block_norm_bwd(nd, None, None, w, w, w, None, None, None, None, *outs, ws)
    for o in outs:
        assert (o == 0).all()


def test_same_bits_each_time_and_on_a_side_stream():
    v, gate = make(1000, 1160, False, "channel", seed=14), "channel"
    nd = dims(1000, 1160, False, gate, 1.0, 0.5)
    first = run_bwd(nd, v, gate)
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            again = run_bwd(nd, v, gate)
        for n, t in first.items():
            assert t is None or torch.equal(t, again[n]), n


def test_in_a_graph():
    v = cuda(make(6, 2048, False, "channel", seed=15))
    nd = dims(6, 2048, False, "channel", 1.0, 1.0)
    r_out, u = torch.empty_like(v["r"]), torch.empty_like(v["y"])
    call = lambda: mb.moe_block_norm_fwd(nd, v["r"], v["y"], v["w_post"], v["gate"], v["w_pre"], r_out, u)  # noqa: E731
    call()
    torch.cuda.synchronize()
    want = (r_out.clone(), u.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    r_out.zero_()
    u.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r_out, want[0]) and torch.equal(u, want[1])


def test_offsets_past_32_bits():
    """T * h just over 2^31 elements: the last rows are those of a small call."""
    T, h = 2 ** 31 // 8192 + 3, 8192
    nd = mb.norm_dims(T, h, gate=mb.GATE_TOKEN, eps=EPS)
    r = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(r)
    v = cuda(make(2, h, False, "token", seed=16))
    r[-2:], y[-2:] = v["r"], v["y"]
    gate = torch.zeros(T, device="cuda")
    gate[-2:] = v["gate"]
    u = torch.empty_like(y)
    mb.moe_block_norm_fwd(nd, r, y, v["w_post"], gate, v["w_pre"], r, u)
    small = [torch.empty_like(v["r"]) for _ in range(2)]
    mb.moe_block_norm_fwd(mb.norm_dims(2, h, gate=mb.GATE_TOKEN, eps=EPS), v["r"], v["y"], v["w_post"], v["gate"], v["w_pre"], *small)
    torch.cuda.synchronize()
    assert torch.equal(r[-2:], small[0]) and torch.equal(u[-2:], small[1])
    assert not u[:-2].any()
