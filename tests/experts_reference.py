"""The grouped and 4-bit operators written out in 64 bits on the CPU, and how far a result
that is summed in fp32 and rounded once may be from them.

Bounds.  A sum of K products in fp32 is off by at most about K steps of 2^-23 (a step of an
addition that need not round to nearest) relative to the sum S of the magnitudes, whatever
the order; (K + 4) * 2^-23 * S covers the factor alpha and beta * C_old as well.  The final
rounding adds half a step of the output type, eps / 2 relative to the value, and below the
smallest normal number half of the smallest one that is not.  1 / (1 + e^-g) from the
hardware's exp2 and reciprocal: the exponent's argument is off by 2^-24 relative, so e^-g by
|g| * 2^-23.5, and each of the few other steps by 2^-23: (|g| + 8) * 2^-22 covers them.
|SiLU'| <= 1.1 and |SiLU''| <= 0.5 carry an error of g on."""
import torch

STEP = 2.0 ** -23


def half_step(y, dtype):
    f = torch.finfo(dtype)
    return f.eps / 2 * y.abs() + f.smallest_normal * f.eps / 2


def parts(offsets):
    o = offsets.tolist()
    return [slice(a, b) for a, b in zip(o, o[1:])]


def matmul(a, b):
    """(a @ b, the bound of an fp32 sum's error) for 64-bit a, b."""
    return a @ b, (a.shape[1] + 4) * STEP * (a.abs() @ b.abs())


def silu_error(g):
    return (g.abs() + 8) * 2.0 ** -22


def gemm_rows(A, B, offsets, trans, alpha, scale, C_old, beta, out_dtype):
    """C [M, N] and its tolerance; rows of no expert NaN."""
    N = B.shape[1] if trans == "T" else B.shape[2]
    C = torch.full((A.shape[0], N), float("nan"), dtype=torch.float64)
    T = C.clone()
    for e, p in enumerate(parts(offsets)):
        b = B[e].double()
        s, err = matmul(A[p].double(), b.t() if trans == "T" else b)
        f = alpha * (1.0 if scale is None else float(scale[e]))
        C[p], T[p] = f * s, abs(f) * (err + 2 * STEP * s.abs())
        if beta:
            C[p] += beta * C_old[p].double()
            T[p] += 4 * STEP * (C_old[p].double() * beta).abs()
    return C, T + half_step(C, out_dtype)


def wgrad(A, D, offsets, alpha, C_old, beta, out_dtype):
    E = len(offsets) - 1
    C = torch.zeros(E, A.shape[1], D.shape[1], dtype=torch.float64)
    T = C.clone()
    for e, p in enumerate(parts(offsets)):
        s, err = matmul(A[p].double().t(), D[p].double())
        C[e], T[e] = alpha * s, abs(alpha) * (err + 2 * STEP * s.abs())
        if beta:
            C[e] += beta * C_old[e].double()
            T[e] += 4 * STEP * (C_old[e].double() * beta).abs()
    return C, T + half_step(C, out_dtype)


def gate_up(a, w):
    """gate, up and their errors from a [m, K] and interleaved w [K, 2N]."""
    g, dg = matmul(a, w[:, 0::2])
    u, du = matmul(a, w[:, 1::2])
    return g, u, dg, du


def swiglu(g, u, dg, du, out_dtype, s=1.0):
    """y and its tolerance, gate and up both times s."""
    g, u, dg, du = s * g, s * u, s * dg + 2 * STEP * (s * g).abs(), s * du + 2 * STEP * (s * u).abs()
    silu = g / (1 + torch.exp(-g))
    y = silu * u
    t = 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + silu_error(g) * y.abs()
    return y, t + half_step(y, out_dtype)


def swiglu_rows(A, W, offsets, alpha, scale, out_dtype):
    N = W.shape[2] // 2
    Y = torch.full((A.shape[0], N), float("nan"), dtype=torch.float64)
    T = Y.clone()
    for e, p in enumerate(parts(offsets)):
        f = alpha * (1.0 if scale is None else float(scale[e]))
        Y[p], T[p] = swiglu(*gate_up(A[p].double(), W[e].double()), out_dtype, f)
    return Y, T


def swiglu_bwd_rows(A, W, dY, offsets, out_dtype):
    H = torch.full((A.shape[0], W.shape[2]), float("nan"), dtype=torch.float64)
    T = H.clone()
    for e, p in enumerate(parts(offsets)):
        g, u, eg, eu = gate_up(A[p].double(), W[e].double())
        dy = dY[p].double()
        s = 1 / (1 + torch.exp(-g))
        d = s * (1 + g * (1 - s))
        H[p, 0::2], H[p, 1::2] = dy * u * d, dy * g * s
        T[p, 0::2] = dy.abs() * (1.1 * eu + 0.5 * (u.abs() + eu) * eg
                                 + u.abs() * s * (1 + g.abs() * (1 - s)) * silu_error(g)
                                 + u.abs() * s * g.abs() * STEP)
        T[p, 1::2] = dy.abs() * (1.1 * eg + g.abs() * s * silu_error(g))
    return H, T + half_step(H, out_dtype)


# ------------------------------------------------------------------ 4-bit
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def quantize(X):
    """Codes [R, 16*ceil(K/32)] and scales [R, ceil(K/32)] of X [R, K], and the values."""
    R, K = X.shape
    nb = -(-K // 32)
    x = torch.zeros(R, nb * 32, dtype=torch.float64)
    x[:, :K] = X.double()
    x = x.view(R, nb, 32)
    bad = ~torch.isfinite(x).all(2)
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2)
    s = (torch.frexp(top).exponent.long() - 3 + 127).clamp(min=0)
    s = torch.where(top > 0, s, 0)
    y = torch.where(bad[..., None], 0.0, x) * torch.exp2(127.0 - s.double())[..., None]
    dist = (y.abs()[..., None] - GRID).abs()
    low = dist.argmin(3)                                 # the first of two at one distance
    up = (low + 1).clamp(max=7)
    tie = (dist.gather(3, up[..., None]) == dist.gather(3, low[..., None])).squeeze(3) & (up != low)
    code = torch.where(tie & (low % 2 == 1), up, low)
    sign = torch.signbit(y).long()
    s = torch.where(bad, 255, s)
    code = (code + 8 * sign).view(R, nb * 32)
    code = torch.where(bad.repeat_interleave(32, 1), 0, code)
    codes = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    return codes, s.to(torch.uint8), values(codes, s.to(torch.uint8))[:, :K]


def values(codes, scales):
    """64-bit values of codes [.., R, 16 nb] and row-major scales [.., R, nb]."""
    table = torch.cat([GRID, -GRID])
    v = table[torch.stack([codes & 15, codes >> 4], -1).long()].flatten(-2)
    f = torch.exp2(scales.double() - 127.0)
    f = torch.where(scales == 255, float("nan"), f)
    return v * f.repeat_interleave(32, -1)


def tile_scales(S):
    """Row-major scales [R, nb] in tiles of 32 rows x 8 blocks, by the formula of the header."""
    R, nb = S.shape
    tk = -(-nb // 8)
    out = torch.zeros(-(-R // 32) * tk * 256, dtype=torch.uint8)
    r, b = torch.meshgrid(torch.arange(R), torch.arange(nb), indexing="ij")
    out[256 * ((r // 32) * tk + b // 8) + 128 * ((b // 4) % 2) + 4 * (r % 32) + b % 4] = S
    return out


def untile_scales(T, R, nb):
    tk = -(-nb // 8)
    r, b = torch.meshgrid(torch.arange(R), torch.arange(nb), indexing="ij")
    return T[256 * ((r // 32) * tk + b // 8) + 128 * ((b // 4) % 2) + 4 * (r % 32) + b % 4]


def check(got, want, tol, what=""):
    """Every element within its tolerance; where `want` is NaN (a row of no expert) any value.
    Rounding to nearest makes an infinity of any value from half a step past the largest number
    of the type on (65520 in fp16): there, and only there, an infinity of its sign is right."""
    f = torch.finfo(got.dtype)
    over = f.max * (1 + f.eps / (4 - 2 * f.eps))          # max = (2 - eps) 2^e, a step eps 2^e
    got = got.double().cpu()
    assert got.shape == want.shape
    inside = ~torch.isnan(want)
    off = torch.where(inside, (got - want).abs() - tol, -1.0)
    gone = torch.isinf(got) & (got.sign() == want.sign()) & (want.abs() + tol >= over)
    off = torch.where(gone, -1.0, off)
    bad = inside & ~(off <= 0)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError("%s: %d of %d outside their bound; first at %s: got %r want %r +- %r"
                             % (what, int(bad.sum()), bad.numel(), i, got[i].item(),
                                want[i].item(), tol[i].item()))
