"""The operators of a mixture-of-experts layer around its products, and products with 4-bit integer
weights, on real work: the cases, their inputs, and two ways to compute them: the plain form in
elementary torch operations, and the library's own calls.

    route_experts         each token's top_k experts and their weights, from the router's logits
    sort_experts          rows sorted by expert: offsets, the order of the rows and its inverse
    spread_rows           the tokens' rows in that order
    combine_rows          each token's weighted sum of its experts' rows; backward
    int4_gemm / _swiglu   products with weights of 4-bit codes, a scale (and zero) for each group

`own` selects the library's calls; the inputs do not depend on it.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a small mixture in serving: latency counts
        dict(name="route one token", op="route", dtype="f32", tokens=1, experts=64, top_k=6,
             scoring="softmax", bias=False, groups=1, top_groups=1, renormalize=True, scale=1.0,
             padded=0.0, off=0, train=False),
        # a decode batch of many experts in groups, balanced by a bias, some places of it empty
        dict(name="route decode", op="route", dtype="f32", tokens=77, experts=256, top_k=8,
             scoring="sigmoid", bias=True, groups=8, top_groups=4, renormalize=True, scale=2.5,
             padded=0.2, off=0, train=False),
        # the same router on a long prefill
        dict(name="route prefill", op="route", dtype="f32", tokens=16384, experts=256, top_k=8,
             scoring="sigmoid", bias=True, groups=8, top_groups=4, renormalize=True, scale=2.5,
             padded=0.0, off=0, train=False),
        # a training step through a softmax router: ids, weights and the logits' gradient
        dict(name="route training", op="route", dtype="bf16", tokens=8192, experts=64, top_k=8,
             scoring="softmax", bias=False, groups=1, top_groups=1, renormalize=False, scale=1.0,
             padded=0.0, off=0, train=True),
        # rows of a decode batch to their experts
        dict(name="rows decode", op="rows", dtype="bf16", tokens=32, experts=64, top_k=8, width=2048,
             padded=0.0, skew=0.5),
        # rows of a prefill, the end of the batch padded
        dict(name="rows prefill", op="rows", dtype="bf16", tokens=8192, experts=64, top_k=8,
             width=2048, padded=0.1, skew=0.5),
        # a decode batch's rows back, onto the residual stream
        dict(name="combine decode", op="combine", dtype="f16", tokens=16, experts=32, top_k=4,
             width=4096, padded=0.0, skew=0.5, residual=True, train=False),
        # the same in training, with the gradients of the rows and of the router's weights
        dict(name="combine training", op="combine", dtype="bf16", tokens=8191, experts=32, top_k=4,
             width=2048, padded=0.0, skew=0.7, residual=False, train=True),
        # one token through a square projection
        dict(name="int4 one token", op="int4", dtype="bf16", swiglu=False, grouped=False, tokens=1,
             top_k=1, experts=1, k=4096, n=4096, group=128, zeros=False, skew=0.0),
        # gate and up projections of a decode batch, weights with zero points
        dict(name="int4 swiglu decode", op="int4", dtype="f16", swiglu=True, grouped=False, tokens=16,
             top_k=1, experts=1, k=4096, n=11008, group=128, zeros=True, skew=0.0),
        # a decode batch through experts' gate and up projections, rows taken where they lie
        dict(name="int4 experts decode", op="int4", dtype="bf16", swiglu=True, grouped=True,
             tokens=32, top_k=8, experts=64, k=2048, n=1408, group=64, zeros=True, skew=0.5),
        # a short prefill through the same projections as the decode batch
        dict(name="int4 prefill", op="int4", dtype="bf16", swiglu=False, grouped=False, tokens=512,
             top_k=1, experts=1, k=4096, n=11008, group=128, zeros=False, skew=0.0),
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, evenly over its logarithm, a multiple of step."""
    return max(step, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


def draw(rng):
    op = rng.choice(["route", "route", "rows", "combine", "int4", "int4", "int4"])
    if op == "route":
        experts = rng.choice([8, 16, 40, 60, 64, 128, 160, 256])
        groups = rng.choice([1, 1, 4, 8] if experts % 8 == 0 else [1, 4])
        top_groups = max(1, groups // 2)
        top_k = min(rng.choice([1, 2, 4, 6, 8]), experts // groups * top_groups)
        return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                    tokens=_spread(rng, 1, 16384), experts=experts, top_k=top_k,
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.choice([False, True]),
                    groups=groups, top_groups=top_groups, renormalize=rng.choice([False, True]),
                    scale=rng.choice([1.0, 2.5]), padded=rng.choice([0.0, 0.2]),
                    off=rng.choice([0, 0, experts // 4]), train=rng.choice([False, True]))
    experts = rng.choice([4, 8, 16, 32, 60, 64, 128])
    top_k = min(experts, rng.choice([1, 2, 4, 6, 8]))
    skew = rng.choice([0.0, 0.5, 1.0])
    if op != "int4":
        width = _spread(rng, 256, 8192, rng.choice([1, 8, 64]))
        most = 8192 * 8 * 2048 // (top_k * width) if op == "rows" else 8192 * 4 * 2048 // (top_k * width)
        c = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), tokens=min(_spread(rng, 1, 16384), most),
                 experts=experts, top_k=top_k, width=width, padded=rng.choice([0.0, 0.1]), skew=skew)
        if c["dtype"] == "f32":
            c["tokens"] = max(1, c["tokens"] // 2)
        if op == "combine":
            c.update(residual=rng.choice([False, True]), train=rng.choice([False, True]))
        return c
    grouped = rng.choice([False, True])
    if not grouped:
        experts = top_k = 1
    k = _spread(rng, 256, 8192, rng.choice([1, 8, 128]))
    n = _spread(rng, 256, 4096 if grouped else 16384, rng.choice([1, 8, 64]))
    if grouped:
        k = min(k, 4096)
        experts = min(experts, max(top_k, 64 * 2048 * 2816 // (2 * n * k)))
    tokens = min(_spread(rng, 1, 512), max(1, 512 * 4096 * 11008 // (2 * n * k * top_k)))
    return dict(op=op, dtype=rng.choice(["bf16", "f16"]), swiglu=rng.choice([False, True]),
                grouped=grouped, tokens=tokens, top_k=top_k, experts=experts, k=k, n=n,
                group=rng.choice([32, 64, 128, 128]), zeros=rng.choice([False, True]), skew=skew)


# ------------------------------------------------------------------ inputs
def _choices(case, seed):
    """(tokens, top_k) different experts of each token, some experts more often, best first; -1 for
    the tokens of the padded end."""
    rng = np.random.default_rng(seed)
    e, t = case["experts"], case["tokens"]
    liking = -case["skew"] * np.log(np.arange(1, e + 1))[rng.permutation(e)]
    scores = liking + rng.gumbel(size=(t, e))
    ids = np.argsort(-scores, axis=1)[:, :case["top_k"]].astype(np.int32)
    ids[t - int(case.get("padded", 0.0) * t):] = -1
    return torch.tensor(ids, device="cuda")


def _plan(ids, experts):
    """offsets, order and place of rows sorted by expert."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.argsort(key, stable=True)
    bounds = torch.arange(experts + 1, device=flat.device)
    offsets = torch.searchsorted(key[order].contiguous(), bounds)
    row = torch.arange(len(flat), device=flat.device)
    place = torch.empty_like(flat)
    place[order] = row
    place = torch.where(flat < 0, -1, place).view(ids.shape)
    order = torch.where(row < offsets[-1], order, -1)
    return offsets.int(), order.int(), place.int()


def _normal(shape, std, dtype, gen):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], case["dtype"]
    s = {"case": case}
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        x = 2 * torch.randn((t, e), generator=gen, device="cuda")
        if case["off"]:       # experts that are out of service
            x[:, torch.randperm(e, generator=gen, device="cuda")[:case["off"]]] = -math.inf
        s["X"] = x.to(DTYPES[dt])
        s["bias"] = 0.2 * torch.randn(e, generator=gen, device="cuda") if case["bias"] else None
        s["mask"] = torch.rand(t, generator=gen, device="cuda") >= case["padded"] if case["padded"] else None
        if case["train"]:
            s["dW"] = torch.randn((t, k), generator=gen, device="cuda")
        return s
    if op in ("rows", "combine"):
        t, k, d = case["tokens"], case["top_k"], case["width"]
        s["ids"] = _choices(case, seed)
        if op == "rows":
            s["X"] = _normal((t, d), 1.0, dt, gen)
            s["Y"] = torch.zeros((t * k, d), dtype=DTYPES[dt], device="cuda")
            return s
        s["place"] = _plan(s["ids"], case["experts"])[2]
        s["Z"] = _normal((t * k, d), 1.0, dt, gen)
        s["weights"] = torch.rand((t, k), generator=gen, device="cuda")
        s["R"] = _normal((t, d), 1.0, dt, gen) if case["residual"] else None
        if case["train"]:
            s["dOut"] = _normal((t, d), 0.1, dt, gen)
            s["dZ"] = torch.zeros((t * k, d), dtype=DTYPES[dt], device="cuda")
        return s
    e, k, n = case["experts"], case["k"], case["n"]
    rows = 2 * n if case["swiglu"] else n
    s["A"] = _normal((case["tokens"], k), 1.0, dt, gen)
    s["offsets"] = s["order"] = None
    if case["grouped"]:
        s["offsets"], s["order"], _ = _plan(_choices(case, seed), e)
    # codes spread over their range, scales around those of weights of size K^-1/2
    groups = -(-k // case["group"])
    codes = torch.randn((e, rows, k), generator=gen, device="cuda").mul_(3).add_(8).round_()
    codes = codes.clamp_(0, 15).to(torch.uint8)
    size = 0.5 + torch.rand((e, rows, groups), generator=gen, device="cuda")
    s["scales"] = (size * (k ** -0.5 / 3)).to(DTYPES[dt])
    s["zeros"] = torch.randint(5, 12, (e, rows, groups), generator=gen, device="cuda",
                               dtype=torch.uint8) if case["zeros"] else None
    s["packed"] = _packed(codes, s["scales"], s["zeros"])
    if not case["grouped"]:
        s["packed"] = tuple(None if p is None else p[0] for p in s["packed"])
    return s


def _packed(codes, scales, zeros):
    """A weight (experts, rows, k) as a user holds it.  Codes: tiles of 16 rows x 128 columns, 1024
    bytes each; byte 16 * (16 * q + r) + 4 * s + b of a tile holds elements 32 * s + 8 * q + 2 * c and
    the one behind it of row r, in nibbles c and c + 4 of the four bytes.  Scales and zeros: tiles of
    16 rows x 4 groups."""
    e, n, k = codes.shape
    c = torch.nn.functional.pad(codes, (0, -k % 128, 0, -n % 16))
    c = c.view(e, -(-n // 16), 16, -(-k // 128), 4, 4, 4, 2)    # tile, r, tile, s, q, c, odd
    c = c.permute(0, 1, 3, 5, 2, 4, 7, 6)                        # tile, tile, q, r, s, odd, c
    c = c.reshape(e, c.shape[1], c.shape[2], 1024, 2)
    out = [c[..., 0] + 16 * c[..., 1]]
    out[0] = out[0].contiguous().flatten(1)
    for f in (scales, zeros):
        if f is None:
            out.append(None)
            continue
        f = torch.nn.functional.pad(f, (0, -f.shape[2] % 4, 0, -n % 16))
        f = f.view(e, -(-n // 16), 16, f.shape[2] // 4, 4).permute(0, 1, 3, 2, 4)
        out.append(f.contiguous().flatten(1))
    return tuple(out)


# ------------------------------------------------------------------ plain form
def _unpacked(s):
    """The weight (experts, rows, k) in fp32 of its packed form."""
    case = s["case"]
    e, k, g = case["experts"], case["k"], case["group"]
    n = 2 * case["n"] if case["swiglu"] else case["n"]
    tn, tk, tg = -(-n // 16), -(-k // 128), -(-(-(-k // g)) // 4)
    codes, scales, zeros = (None if p is None else p.view(e, -1) for p in s["packed"])
    c = torch.stack([codes & 15, codes >> 4], 2).view(e, tn, tk, 4, 16, 4, 2, 4)
    c = c.permute(0, 1, 4, 2, 5, 3, 7, 6).reshape(e, tn * 16, tk * 128).float()

    def by_column(f):
        f = f.view(e, tn, tg, 16, 4).permute(0, 1, 3, 2, 4).reshape(e, tn * 16, tg * 4).float()
        return f.repeat_interleave(g, 2)[:, :n, :k]
    z = by_column(zeros) if zeros is not None else 8.0
    return (c[:, :n, :k] - z) * by_column(scales)


def _chosen(s):
    """The ids of each token, chosen by values in 64 bits."""
    case, x = s["case"], s["X"].double()
    t, e = x.shape
    if s["mask"] is not None:
        x = x.masked_fill(~s["mask"][:, None], -math.inf)
    # a row without an expert: any finite stand-in, the row's ids are -1 all the same
    safe = torch.where(torch.isinf(x).all(1, keepdim=True), 0.0, x)
    if case["scoring"] == "softmax":
        p = torch.exp(safe - safe.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-safe))
    out = torch.isinf(x)
    c = p if s["bias"] is None else p + s["bias"].double()
    c = c.masked_fill(out, -math.inf)
    allowed = ~out
    if case["groups"] > 1:
        inside = c.view(t, case["groups"], -1)
        best = torch.sort(inside, dim=2, descending=True).values[:, :, :2]
        best = torch.where(torch.isinf(best), 0.0, best).sum(2)
        best = best.masked_fill(torch.isinf(inside).all(2), -math.inf)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        on = torch.zeros(best.shape, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        allowed &= on.repeat_interleave(e // case["groups"], 1)
    key = (x if s["bias"] is None else c).masked_fill(~allowed, -math.inf)
    value, ids = torch.sort(key, dim=1, descending=True, stable=True)
    value, ids = value[:, :case["top_k"]], ids[:, :case["top_k"]]
    return torch.where(torch.isinf(value), -1, ids)


def _route(s):
    case, x = s["case"], s["X"].float()
    ids = _chosen(s)
    there = ids >= 0
    if case["scoring"] == "softmax":
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    else:
        p = 1 / (1 + torch.exp(-x))
    at = ids.clamp(min=0)
    w = torch.where(there, p.gather(1, at), 0.0)
    q = w
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        q = w / torch.where(total > 0, total, 1.0)
    out = [ids.int(), q * case["scale"]]
    if case["train"]:
        g = torch.where(there, s["dW"] * case["scale"], 0.0)
        if case["renormalize"]:
            d = q * (g - (g * q).sum(1, keepdim=True))
            if case["scoring"] == "sigmoid":
                d = d * (1 - w)
            dx = torch.zeros_like(x).scatter_add_(1, at, torch.where(there, d, 0.0))
        else:
            full = torch.zeros_like(x).scatter_add_(1, at, g)
            if case["scoring"] == "sigmoid":
                dx = full * p * (1 - p)
            else:
                dx = p * (full - (full * p).sum(1, keepdim=True))
        if s["mask"] is not None:
            dx = torch.where(s["mask"][:, None], dx, 0.0)
        out.append(dx.to(s["X"].dtype))
    return out


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "route":
        return _route(s)
    if op == "rows":
        offsets, order, place = _plan(s["ids"], case["experts"])
        y = s["X"][order.clamp(min=0).long() // case["top_k"]]
        return [offsets, order, place, torch.where(order[:, None] >= 0, y, 0.0).to(y.dtype)]
    if op == "combine":
        place = s["place"].long()
        there = (place >= 0).float()[..., None]
        z = s["Z"].float()[place.clamp(min=0)]
        w = s["weights"][..., None] * there
        y = (w * z).sum(1)
        if s["R"] is not None:
            y = y + s["R"].float()
        out = [y.to(s["Z"].dtype)]
        if case["train"]:
            do = s["dOut"].float()[:, None]
            dz = torch.zeros(s["Z"].shape, device=z.device)
            dz.index_add_(0, place.clamp(min=0).flatten(), (w * do).flatten(0, 1))
            out += [dz.to(s["Z"].dtype), (z * do * there).sum(2)]
        return out
    w = _unpacked(s)
    a = s["A"].float()
    if case["grouped"]:
        # the rows of each expert as a block of the longest run's height, zeros behind
        off = s["offsets"].long()
        row = torch.arange(len(s["order"]), device=a.device)
        expert = torch.searchsorted(off[1:].contiguous(), row, right=True)
        at = row - off[expert]
        block = torch.zeros((case["experts"], case["tokens"], a.shape[1]), device=a.device)
        block[expert, at] = a[s["order"].long() // case["top_k"]]
        h = torch.bmm(block, w.transpose(1, 2).contiguous())[expert, at]
    else:
        h = a @ w[0].t()
    if case["swiglu"]:
        h = h[:, 0::2] * torch.sigmoid(h[:, 0::2]) * h[:, 1::2]
    return h.to(s["A"].dtype)


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import swiglu_gemm_amd as sg
    case, op = s["case"], s["case"]["op"]
    if op == "route":
        how = dict(scoring=case["scoring"], renormalize=case["renormalize"], scale=case["scale"])
        out = list(sg.route_experts(s["X"], case["top_k"], bias=s["bias"], groups=case["groups"],
                                    top_groups=case["top_groups"], mask=s["mask"], **how))
        if case["train"]:
            out.append(sg.route_experts_bwd(s["X"], out[0], s["dW"], torch.empty_like(s["X"]), **how))
        return out
    if op == "rows":
        offsets, order, place = sg.sort_experts(s["ids"], case["experts"])
        sg.spread_rows(s["X"], place, s["Y"])
        return [offsets, order, place, s["Y"]]
    if op == "combine":
        out = [sg.combine_rows(s["Z"], s["place"], s["Z"].new_empty((case["tokens"], case["width"])),
                               weights=s["weights"], residual=s["R"])]
        if case["train"]:
            out += sg.combine_rows_bwd(s["dOut"], s["Z"], s["place"], s["weights"], s["dZ"],
                                       torch.empty_like(s["weights"]))
        return out
    codes, scales, zeros = s["packed"]
    m = case["tokens"] * case["top_k"]
    out = s["A"].new_empty((m, case["n"]))
    product = sg.int4_swiglu_gemm if case["swiglu"] else sg.int4_gemm
    return product(s["A"], codes, scales, out, zeros=zeros, group=case["group"],
                   offsets=s["offsets"], order=s["order"], top_k=case["top_k"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, t, k = case["op"], case["tokens"], case["top_k"]
    size = SIZES[case["dtype"]]
    if op == "route":
        e = case["experts"]
        b = t * e * size + t * k * 8
        if case["train"]:      # the logits again, their gradient, ids and the weights' gradient
            b += t * e * size + t * k * 4
        return {"bytes": b, "flops": (20 if case["train"] else 10) * t * e}
    if op == "rows":
        d = case["width"] * size
        live = t - int(case["padded"] * t)
        return {"bytes": live * d * (1 + k) + t * k * 12, "flops": t * k}
    if op == "combine":
        d = case["width"] * size
        live = t - int(case["padded"] * t)
        b = live * k * d + t * d * (2 if case["residual"] else 1) + t * k * 8
        f = 2 * t * k * case["width"]
        if case["train"]:
            b, f = b + t * d + live * k * d + t * k * 4, 3 * f
        return {"bytes": b, "flops": f}
    e, n, m = case["experts"], case["n"], t * k
    rows = 2 * n if case["swiglu"] else n
    met = e * (1 - (1 - k / e) ** t)          # experts with at least one row
    weight = rows * case["k"] / 2 + rows * -(-case["k"] // case["group"]) * (3 if case["zeros"] else 2)
    return {"bytes": t * case["k"] * size + met * weight + m * n * size,
            "flops": 2 * m * rows * case["k"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_route(s):
    case = s["case"]
    x = s["X"].double().cpu().numpy()
    t, e = x.shape
    k, per = case["top_k"], e // case["groups"]
    live = np.ones(t, bool) if s["mask"] is None else s["mask"].cpu().numpy()
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    g = s["dW"].double().cpu().numpy() * case["scale"] if case["train"] else None
    ids, w, dx = np.full((t, k), -1, np.int32), np.zeros((t, k)), np.zeros((t, e))
    for i in np.flatnonzero(live):
        on = np.isfinite(x[i])
        if not on.any():
            continue
        if case["scoring"] == "softmax":
            p = np.exp(x[i] - x[i][on].max())
            p /= p.sum()
        else:
            p = 1 / (1 + np.exp(-x[i]))
        c = p if bias is None else p + bias
        key = np.where(on, x[i] if bias is None else c, -np.inf)
        if case["groups"] > 1:
            value = []
            for j in range(case["groups"]):
                best = np.sort(c[j * per:(j + 1) * per][on[j * per:(j + 1) * per]])[::-1][:2]
                value.append(best.sum() if len(best) else -np.inf)
            kept = np.argsort(-np.array(value), kind="stable")[:case["top_groups"]]
            key = np.where(np.isin(np.arange(e) // per, kept), key, -np.inf)
        pick = np.argsort(-key, kind="stable")[:k]
        pick = pick[np.isfinite(key[pick])]
        n = len(pick)
        if not n:
            continue
        ids[i, :n] = pick
        q = p[pick] / p[pick].sum() if case["renormalize"] else p[pick]
        w[i, :n] = case["scale"] * q
        if g is None:
            continue
        gi = g[i, :n]
        if case["renormalize"]:
            d = q * (gi - gi @ q)
            dx[i, pick] = d * (1 - p[pick]) if case["scoring"] == "sigmoid" else d
        elif case["scoring"] == "sigmoid":
            dx[i, pick] = gi * q * (1 - q)
        else:
            dx[i] = -p * (gi @ q)
            dx[i, pick] += q * gi
    out = [ids, w] + ([dx] if case["train"] else [])
    return [torch.from_numpy(a) for a in out]


def _exact_rows(s):
    case = s["case"]
    ids = s["ids"].cpu().numpy()
    t, k = ids.shape
    flat = ids.ravel()
    lists = [np.flatnonzero(flat == e) for e in range(case["experts"])]
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists])]).astype(np.int32)
    order = np.full(t * k, -1, np.int32)
    order[:offsets[-1]] = np.concatenate(lists)
    place = np.full(t * k, -1, np.int32)
    place[order[:offsets[-1]]] = np.arange(offsets[-1])
    x = s["X"].double().cpu()
    y = torch.zeros(t * k, case["width"], dtype=torch.float64)
    y[:offsets[-1]] = x[torch.from_numpy(order[:offsets[-1]].astype(np.int64) // k)]
    return [torch.from_numpy(offsets), torch.from_numpy(order), torch.from_numpy(place.reshape(t, k)), y]


def _exact_combine(s):
    case = s["case"]
    place = s["place"].long()
    z, w = s["Z"].double(), s["weights"].double()
    y = torch.zeros(place.shape[0], case["width"], dtype=torch.float64, device=z.device)
    if s["R"] is not None:
        y += s["R"].double()
    dz, dw = torch.zeros_like(z) if case["train"] else None, torch.zeros_like(w)
    for j in range(place.shape[1]):
        live = torch.nonzero(place[:, j] >= 0).flatten()
        at = place[live, j]
        y[live] += w[live, j, None] * z[at]
        if case["train"]:
            do = s["dOut"][live].double()
            dz[at] = w[live, j, None] * do
            dw[live, j] = (do * z[at]).sum(1)
    return [y, dz, dw] if case["train"] else [y]


def _exact_int4(s):
    case = s["case"]
    k, g = case["k"], case["group"]
    n = 2 * case["n"] if case["swiglu"] else case["n"]
    groups = -(-k // g)
    dev = s["A"].device
    codes, scales, zeros = (None if p is None else p.view(case["experts"], -1) for p in s["packed"])
    r = torch.arange(n, device=dev)[:, None]
    c = torch.arange(k, device=dev)[None]
    tile = (r // 16) * -(-k // 128) + c // 128
    inner, pair = c % 128, c % 8 // 2
    nibble = pair + 4 * (c % 2)                                 # of the four bytes of eight columns
    at = 1024 * tile + 16 * (16 * (inner % 32 // 8) + r % 16) + 4 * (inner // 32) + nibble // 2
    high = nibble % 2 == 1
    f = torch.arange(groups, device=dev)[None]
    fat = ((r // 16) * -(-groups // 4) + f // 4) * 64 + 4 * (r % 16) + f % 4
    a = s["A"].double()
    ends = [0, case["tokens"]] if s["offsets"] is None else s["offsets"].tolist()
    outs = []
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        byte = codes[i][at]
        w = torch.where(high, byte >> 4, byte & 15).double()
        z = zeros[i][fat].double() if zeros is not None else torch.full((1, 1), 8.0, device=dev).double()
        w = w - (z.repeat_interleave(g, 1)[:, :k] if zeros is not None else z)
        w = w * scales[i][fat].double().repeat_interleave(g, 1)[:, :k]
        x = a if s["order"] is None else a[s["order"][lo:hi].long() // case["top_k"]]
        if case["swiglu"]:
            u, v = x @ w[0::2].T.contiguous(), x @ w[1::2].T.contiguous()
            outs.append(u / (1 + torch.exp(-u)) * v)
        else:
            outs.append(x @ w.T.contiguous())
    return torch.cat(outs)


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "rows": _exact_rows, "combine": _exact_combine,
            "int4": _exact_int4}[case["op"]](s)
