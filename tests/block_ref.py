"""Plain 64-bit references of the e4m3 operators with a scale for each block of
128: codes from their definition (the float32 quotient to the nearest e4m3
value, ties to even), products of the values that codes and scales stand for."""
import torch

BLOCK = 128


def _up(n):
    return -(-n // BLOCK)


def e4m3(v):
    """The nearest e4m3 value to each float64 in v: spacing 2^-3 of the power of two below, 2^-9 at the least."""
    e = torch.frexp(v.abs())[1].double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def quantize(v, bk):
    """v [R, n] float64 -> (codes' values [R, n], scales [ceil(R/bk), ceil(n/128)]) for blocks of bk x 128."""
    R, n = v.shape
    top = torch.zeros(-(-R // bk), _up(n), dtype=torch.float64, device=v.device)
    rows, cols = torch.arange(R, device=v.device) // bk, torch.arange(n, device=v.device) // BLOCK
    top.view(-1).scatter_reduce_(0, (rows[:, None] * _up(n) + cols).reshape(-1), v.abs().reshape(-1), "amax")
    s = torch.where(top > 0, (top / 448.0).float().double(), torch.ones_like(top))
    q = e4m3((v / s[rows][:, cols]).float().double())
    return q, s


def value(q, s, bk):
    """Codes [R, n] times their blocks' scales, float64."""
    rows = torch.arange(q.shape[0], device=q.device) // bk
    cols = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * s.double()[rows][:, cols]


def coded_rows(v):
    return value(*quantize(v, 1), 1)


def kept(v):
    """Rounded to bf16 and back."""
    return v.to(torch.bfloat16).double()


def silu(a):
    return a * torch.sigmoid(a)


def weights(E, K, N, std=None, seed=0, device="cuda"):
    """Random weights as (codes float8 [E, K, N], scales, values float64), quantised by this reference."""
    g = torch.Generator(device).manual_seed(seed)
    W = torch.empty(E, K, N, dtype=torch.bfloat16, device=device).normal_(0.0, K ** -0.5 if std is None else std, generator=g)
    return code_weights(W)


def code_weights(W):
    qs = [quantize(w.double(), BLOCK) for w in W]
    q = torch.stack([a for a, _ in qs]).float().to(torch.float8_e4m3fn)
    s = torch.stack([b for _, b in qs]).float().contiguous()
    return q, s, torch.stack([value(a, b, BLOCK) for a, b in qs])


def ffn_bwd(x, dy, A, B, H, w1, w3, w2, groups):
    """(dx, dW1, dW3, dW2) in float64, dA and dB kept in bf16; groups: a slice of rows for each expert."""
    dx = torch.zeros_like(x)
    dW1, dW3, dW2 = torch.zeros_like(w1), torch.zeros_like(w3), torch.zeros_like(w2)
    for e, r in enumerate(groups):
        if r.stop <= r.start:
            continue
        dh = coded_rows(dy[r]) @ w2[e].t()
        g = torch.sigmoid(A[r])
        da, db = kept(dh * B[r] * g * (1 + A[r] * (1 - g))), kept(dh * A[r] * g)
        dx[r] = coded_rows(da) @ w1[e].t() + coded_rows(db) @ w3[e].t()
        dW1[e], dW3[e], dW2[e] = x[r].t() @ da, x[r].t() @ db, H[r].t() @ dy[r]
    return dx, dW1, dW3, dW2
