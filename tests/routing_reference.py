"""The routing operators and 4-bit integer weights written out in 64 bits on the CPU, and how far a
result computed in fp32 and rounded once may be from them.

Bounds, u = 2^-23 (a step of an operation that need not round to nearest).  e^d with d = x - top
rounded: off by |d| u / 2 from the argument and 2 u of its own; a sum of positive terms carries
their errors in proportion, and each addition or division adds u.  A log score min(x, 0) -
log1p(e^-|x|) is off by (4 + |l|) u in all: e^-|x| by 2 u of at most 1, log1p by 2 u of at most 0.7,
the difference by u / 2 of itself."""
import torch

from experts_reference import half_step, swiglu

U = 2.0 ** -23


def route(X, top_k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=2,
          renormalize=True, scale=1.0, mask=None):
    """(ids, weights, the weights' tolerance) row by row."""
    T, E = X.shape
    ids = torch.full((T, top_k), -1, dtype=torch.int32)
    w, tol = torch.zeros(T, top_k, dtype=torch.float64), torch.zeros(T, top_k, dtype=torch.float64)
    per = E // groups
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        x = X[t].double()
        on = x != -float("inf")
        if not on.any():
            continue
        if scoring == "softmax":
            s = torch.exp(x - x[on].max())
            s = s / s.sum()
        else:
            s = 1 / (1 + torch.exp(-x))
        c = s if bias is None else s + bias.double()
        on = on & (c != -float("inf")) & ~torch.isnan(c)
        key = x if bias is None else c
        if groups > 1 and top_groups < groups:
            value = []
            for g in range(groups):
                inside = sorted((float(c[e]) for e in range(g * per, g * per + per) if on[e]), reverse=True)
                value.append(sum(inside[:group_top]) if inside else -float("inf"))
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            on = on & torch.tensor([e // per in kept for e in range(E)])
        pick = sorted((e for e in range(E) if on[e]), key=lambda e: (-float(key[e]), e))[:top_k]
        n = len(pick)
        if n == 0:
            continue
        ids[t, :n] = torch.tensor(pick, dtype=torch.int32)
        w[t, :n], tol[t, :n] = weights(x, s, torch.tensor(pick), scoring, renormalize, scale)
    return ids, w, tol


def weights(x, s, pick, scoring, renormalize, scale):
    """Weights of the chosen experts and their tolerance."""
    if renormalize:
        l = x[pick] if scoring == "softmax" else torch.minimum(x[pick], torch.zeros(())) - torch.log1p(
            torch.exp(-x[pick].abs()))
        q = torch.softmax(l, 0)
        el = torch.zeros(()) if scoring == "softmax" else 2 * (4 + l.abs().max())
        d = l.max() - l
        rel = (d + (q * d).sum() + 2 * el + len(pick) + 10) * U
    elif scoring == "softmax":
        q = s[pick]
        d = x.max() - x
        d = torch.where(torch.isinf(d), 0.0, d)
        rel = (d[pick] + (s * d).sum() + 24 + len(x) / 64) * U
    else:
        q, rel = s[pick], 8 * U
    return scale * q, abs(scale) * (q * rel + 2.0 ** -126) + 2.0 ** -149


def route_bwd(X, ids, dweights, scoring="softmax", renormalize=True, scale=1.0):
    """dX and its tolerance (the type's rounding included)."""
    T, E = X.shape
    dX = torch.zeros(T, E, dtype=torch.float64)
    tol = dX.clone()
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not at:
            continue
        pick, x = ids[t, at].long(), X[t].double()
        G = scale * dweights[t, at].double()
        s = torch.softmax(x, 0) if scoring == "softmax" else 1 / (1 + torch.exp(-x))
        q, e = weights(x, s, pick, scoring, renormalize, 1.0)
        rel = (e / q.clamp(min=1e-300)).clamp(max=1.0)
        worst = rel.max() + 16 * U
        if renormalize:
            d = q * (G - (G * q).sum())
            m = q * (G.abs() + (G * q).abs().sum())
            if scoring == "sigmoid":
                f = 1 / (1 + torch.exp(x[pick]))
                d, m = d * f, m * f
            dX[t].index_add_(0, pick, d)
            tol[t].index_add_(0, pick, 3 * worst * m)
        elif scoring == "sigmoid":
            f = q / (1 + torch.exp(x[pick]))
            dX[t].index_add_(0, pick, G * f)
            tol[t].index_add_(0, pick, (G * f).abs() * 24 * U)
        else:
            full, size = torch.zeros(E, dtype=torch.float64), torch.zeros(E, dtype=torch.float64)
            full.index_add_(0, pick, G)
            size.index_add_(0, pick, G.abs())
            dX[t] = s * (full - (full * s).sum())
            every = weights(x, s, torch.arange(E), scoring, False, 1.0)[1]
            rel = (every / s.clamp(min=1e-300)).clamp(max=1.0)
            sums = (rel * s * size).sum() + (s * size).sum() * (24 + E / 64) * U
            tol[t] = every * (size + (s * size).sum()) + s * (sums + 8 * U * (size + (s * size).sum()))
    return dX, tol + half_step(dX, X.dtype) + 2.0 ** -149


def sort(ids, experts):
    flat = ids.flatten().tolist()
    lists = [[i for i, v in enumerate(flat) if v == e] for e in range(experts)]
    offsets = [0]
    for v in lists:
        offsets.append(offsets[-1] + len(v))
    order = [i for v in lists for i in v]
    place = [-1] * len(flat)
    for r, i in enumerate(order):
        place[i] = r
    order += [-1] * (len(flat) - len(order))
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)
    return as_int(offsets), as_int(order), as_int(place).view(ids.shape)


def spread(X, place, Y, weights=None):
    """Y with the rows of X at their places, 64 bits, rounded once to Y's type."""
    Y = Y.clone()
    for t in range(place.shape[0]):
        for j in range(place.shape[1]):
            r = int(place[t, j])
            if 0 <= r < Y.shape[0]:
                f = 1.0 if weights is None else weights[t, j].double()
                Y[r] = (X[t].double() * f).to(Y.dtype)
    return Y


def combine(Z, place, weights=None, residual=None):
    """out in 64 bits and its tolerance."""
    T, k = place.shape
    out = torch.zeros(T, Z.shape[1], dtype=torch.float64)
    size = out.clone()
    if residual is not None:
        out, size = out + residual.double(), size + residual.double().abs()
    for t in range(T):
        for j in range(k):
            r = int(place[t, j])
            if 0 <= r < Z.shape[0]:
                v = Z[r].double() * (1.0 if weights is None else weights[t, j].double())
                out[t] += v
                size[t] += v.abs()
    return out, (k + 1) * U * size + half_step(out, Z.dtype)


def combine_bwd(dOut, Z, place, weights):
    """dZ (NaN where no place names the row), its tolerance, dweights and theirs."""
    T, k = place.shape
    dZ = torch.full(Z.shape, float("nan"), dtype=torch.float64)
    dw, tol = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            r = int(place[t, j])
            if 0 <= r < Z.shape[0]:
                dZ[r] = weights[t, j].double() * dOut[t].double()
                p = dOut[t].double() * Z[r].double()
                dw[t, j], tol[t, j] = p.sum(), (len(p) + 8) * U * p.abs().sum()
    return dZ, U * dZ.abs() + half_step(dZ, Z.dtype), dw, tol + 2.0 ** -149


# ------------------------------------------------------------------ 4-bit integers
def int4_quantize(W, group, zero_points, scale_dtype):
    """codes [N, K], scales [N, groups], zeros [N, groups] of W [N, K] by the formulas; the scale in
    fp32 steps as they say, the rest in 64 bits."""
    N, K = W.shape
    n = -(-K // group)
    codes = torch.full((N, K), 8, dtype=torch.uint8)
    scales = torch.zeros(N, n, dtype=scale_dtype)
    zeros = torch.full((N, n), 8, dtype=torch.uint8)
    for g in range(n):
        w = W[:, g * group:(g + 1) * group].float()
        bad = ~torch.isfinite(w).all(1)
        lo, hi = w.clamp(max=0).amin(1), w.clamp(min=0).amax(1)
        s = ((hi - lo) / 15 if zero_points else torch.maximum(hi, -lo) / 7).to(scale_dtype)
        bad |= ~torch.isfinite(s)
        f = torch.where(bad, 0.0, s.double())[:, None]
        live = f > 0
        z = torch.full((N, 1), 8.0, dtype=torch.float64)
        if zero_points:
            z = torch.where(live, torch.round(-lo.double()[:, None] / f).clamp(0, 15), 8.0)
        c = torch.where(live, (torch.round(w.double() / f) + z).clamp(0, 15), 8.0)
        codes[:, g * group:(g + 1) * group] = torch.where(live, c, 8.0).to(torch.uint8)
        scales[:, g] = torch.where(bad, float("nan"), s.double()).to(scale_dtype)
        zeros[:, g] = torch.where(live, z, 8.0)[:, 0].to(torch.uint8)
    return codes, scales, zeros if zero_points else None


def int4_values(codes, scales, zeros, group):
    """64-bit values of codes [.., N, K]."""
    K = codes.shape[-1]
    wide = lambda f: f.double().repeat_interleave(group, -1)[..., :K]
    return wide(scales) * (codes.double() - (8.0 if zeros is None else wide(zeros)))


def int4_layout(codes, scales, zeros, group):
    """The kernels' layout of one weight, element by element."""
    N, K = codes.shape
    tk, tn, n = -(-K // 128), -(-N // 16), -(-K // group)
    tg = -(-n // 4)
    out = torch.zeros(tn * tk * 1024, dtype=torch.uint8)
    r, c = torch.meshgrid(torch.arange(N), torch.arange(K), indexing="ij")
    i = c % 8
    nibble = i // 2 + 4 * (i % 2)
    at = ((r // 16) * tk + c // 128) * 1024 + 16 * (16 * (c % 32 // 8) + r % 16) + 4 * (c % 128 // 32)
    at, high = at + nibble // 2, nibble % 2 == 1
    out[at[~high]] = codes[~high]
    out[at[high]] += codes[high] * 16
    r, g = torch.meshgrid(torch.arange(N), torch.arange(n), indexing="ij")
    at = ((r // 16) * tg + g // 4) * 64 + 4 * (r % 16) + g % 4
    s = torch.zeros(tn * tg * 64, dtype=scales.dtype)
    s[at] = scales
    z = None
    if zeros is not None:
        z = torch.zeros(tn * tg * 64, dtype=torch.uint8)
        z[at] = zeros
    return out, s, z


def int4_sums(A, codes, scales, zeros, group):
    """A @ W^T in 64 bits and the bound of its fp32 sums.  fp16: products a * (code - zero); bf16:
    a * (16 + code) less (16 + zero) * a.  Each group's sum takes one more product and addition."""
    wide = lambda f: f.double().repeat_interleave(group, -1)[..., :codes.shape[-1]]
    z = torch.full_like(codes, 8, dtype=torch.float64) if zeros is None else wide(zeros)
    c, s, a = codes.double(), wide(scales), A.double()
    size = (c - z).abs() if A.dtype == torch.float16 else 32 + c + z
    total = a @ (s * (c - z)).t().contiguous()
    return total, (codes.shape[-1] + 8) * U * (a.abs() @ (s.abs() * size).t().contiguous())


def int4_rows(A, weights, group, offsets, order, top_k, M, out_dtype, swiglu_form, alpha=1.0):
    """The product's rows and their tolerance; rows of no expert NaN.  weights: one (codes, scales,
    zeros) for each expert."""
    outs, tols = None, None
    ends = [0, M] if offsets is None else offsets.tolist()
    for (lo, hi), (codes, scales, zeros) in zip(zip(ends, ends[1:]), weights):
        rows = torch.arange(lo, hi) if order is None else order[lo:hi].long() // top_k
        y, t = int4_sums(A[rows], codes, scales, zeros, group)
        if swiglu_form:
            y, t = swiglu(y[:, 0::2], y[:, 1::2], t[:, 0::2], t[:, 1::2], out_dtype)
        else:
            y, t = alpha * y, abs(alpha) * (t + U * y.abs())
            t = t + half_step(y, out_dtype)
        if outs is None:
            outs = torch.full((M, y.shape[1]), float("nan"), dtype=torch.float64)
            tols = outs.clone()
        outs[lo:hi], tols[lo:hi] = y, t
    return outs, tols
