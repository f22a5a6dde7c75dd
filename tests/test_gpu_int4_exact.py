"""4-bit integer weights where every sum is exact: whole activations, scales that are powers of two, so that
no order of summing rounds and a product without SwiGLU is compared bit for bit, at any depth.  Each case is
also held against planted mistakes, in the reference and without a GPU: a column, a group, a zero point, a
row or an expert that is left out or taken for its neighbour has to show in it."""
import pytest

torch = pytest.importorskip("torch")

import routing_reference as ref
from experts_reference import check, swiglu

HALF = {"f16": torch.float16, "bf16": torch.bfloat16}
U8 = torch.uint8


class Case:
    """Activations [T, K] and one weight for each expert, the rows of C through order where top_k > 0.  A is
    whole, its first and last columns without a zero; W = scale * (code - zero) with scales of +-q and
    +-2 q, the first and last columns' codes away from their zero points."""

    def __init__(self, dtype, M, N, K, group, zeros, sizes=None, top_k=0):
        g = torch.Generator().manual_seed(M * 7 + N * 3 + K + group)
        self.dtype, self.N, self.K, self.group = HALF[dtype], N, K, group
        most = max(1, min(8, 2 ** 24 // (K * 132)))
        n = -(-K // group)
        self.weights = []
        # q: sums near 2, where SiLU bends; fp32 holds them to q / 2^24
        self.q = 2.0 ** -round((3 + torch.tensor(float(K)).log2().item()) / 2 + torch.tensor(most / 2.0).log2().item())
        for _ in range(1 if sizes is None else len(sizes)):
            codes = torch.randint(0, 16, (N, K), generator=g, dtype=U8)
            scales = (self.q * 2.0 ** torch.randint(0, 2, (N, n), generator=g)).to(self.dtype)
            scales[torch.rand(N, n, generator=g) < 0.5] *= -1
            z = torch.randint(0, 16, (N, n), generator=g, dtype=U8) if zeros else None
            for c in (0, K - 1):
                at = 8 if z is None else z[:, c // group].long()
                codes[:, c] = ((at + 1 + torch.randint(0, 15, (N,), generator=g)) % 16).to(U8)
            if zeros:
                z[N // 2, 0] = 255                    # codes' range is not the zero points'
            self.weights.append((codes, scales, z))
        self.offsets = self.order = None
        self.top_k, T, self.M = max(top_k, 1), M, M
        if sizes is not None:
            self.offsets = torch.tensor([0] + list(sizes), dtype=torch.int32).cumsum(0).int()
            self.M = T = int(self.offsets[-1])
        if top_k:
            T = -(-self.M // top_k)
            self.order = torch.randperm(T * top_k, generator=g)[:self.M].to(torch.int32)
        self.A = torch.randint(-most, most + 1, (T, K), generator=g).to(self.dtype)
        for c in (0, K - 1):
            self.A[:, c] = (2 * torch.randint(0, 2, (T,), generator=g) - 1).to(self.dtype)
        # every product and partial sum is a multiple of q and below 2^24 q
        for codes, scales, z in self.weights:
            wide = lambda f: f.double().repeat_interleave(group, 1)[:, :K]
            size = wide(scales).abs() * (48 + (8 if z is None else wide(z)))
            assert (self.A.double().abs() @ size.t()).max() < 2 ** 24 * self.q

    def sums(self, weights=None, A=None, order=None):
        """C [M, N] in 64 bits; the arguments take the place of the case's own."""
        weights, A = weights or self.weights, self.A if A is None else A
        order = self.order if order is None else order
        rows = torch.arange(self.M) if order is None else order.long() // self.top_k
        ends = [0, self.M] if self.offsets is None else self.offsets.tolist()
        return torch.cat([A[rows[lo:hi]].double() @ ref.int4_values(*w, self.group).t()
                          for lo, hi, w in zip(ends, ends[1:], weights)])

    def swiglu(self, sums):
        """SwiGLU of exact sums, and its tolerance: SiLU's and one rounding."""
        none = torch.zeros_like(sums[:, 0::2])
        return swiglu(sums[:, 0::2], sums[:, 1::2], none, none, self.dtype)

    def changed(self):
        """The sums with one mistake each."""
        def each(f):
            out = []
            for c, s, z in self.weights:
                c, s, z = c.clone(), s.clone(), None if z is None else z.clone()
                f(c, s, z)
                out.append((c, s, z))
            return out

        def dropped(column):
            A = self.A.clone()
            A[:, column] = 0
            return self.sums(A=A)
        yield "first column", dropped(0)
        yield "last column", dropped(self.K - 1)
        yield "last group", self.sums(each(lambda c, s, z: s[:, -1].zero_()))
        yield "first group", self.sums(each(lambda c, s, z: s[:, 0].zero_()))
        yield "last codes", self.sums(each(lambda c, s, z: c[:, -1].bitwise_xor_(1)))
        yield "last row", self.sums(each(lambda c, s, z: c[-2:].bitwise_xor_(8)))
        if self.weights[0][2] is not None:
            yield "last zero point", self.sums(each(lambda c, s, z: z[:, -1].bitwise_xor_(1)))
        if len(self.weights) > 1:
            yield "next expert", self.sums(self.weights[1:] + self.weights[:1])
        if self.order is not None and self.A.shape[0] > 1:
            other = (self.order + self.top_k) % (self.A.shape[0] * self.top_k)
            yield "other token", self.sums(order=other)



def outside(got, want, tol):
    return bool(((got - want).abs() > tol).any())


# rows, columns, depth, group, zero points
SIZES = [(1, 16, 128, 128, False), (70, 210, 1100, 64, True), (65, 130, 2304, 128, True),
         (16, 98, 4000, 32, False), (3, 34, 40, 32, True), (40, 50, 640, 128, True), (33, 60, 384, 64, False),
         (34, 36, 4000, 32, True), (2, 33, 130, 64, True), (5, 20, 20011, 128, True), (35, 18, 65535, 64, False)]
# rows of each expert, top_k (0: rows as they lie), columns, depth, group, zero points
GROUPED = [([5, 0, 64, 1, 130, 16], 0, 150, 200, 64, True), ([1, 0, 5, 2], 3, 50, 2000, 128, False),
           ([40, 33, 0, 70], 4, 66, 1032, 32, True), ([2] * 70, 8, 18, 260, 128, True)]


def cases(dtype):
    for M, N, K, group, zeros in SIZES:
        yield Case(dtype, M, N, K, group, zeros)
    for sizes, top_k, N, K, group, zeros in GROUPED:
        yield Case(dtype, 0, N, K, group, zeros, sizes, top_k)


@pytest.mark.parametrize("dtype", sorted(HALF))
def test_mistakes_show(dtype):
    for c in cases(dtype):
        want = c.sums()
        y, tol = c.swiglu(want) if c.N % 2 == 0 else (None, None)
        assert torch.equal(want.float().double(), want)
        for what, got in c.changed():
            assert not torch.equal(got, want), (what, c.N, c.K)
            if y is not None:
                assert outside(c.swiglu(got)[0], y, tol), (what, c.N, c.K)


def layouts(c):
    parts = [ref.int4_layout(*w, c.group) for w in c.weights]
    out = [None if p[0] is None else torch.stack(p).cuda() for p in zip(*parts)]
    return out if c.offsets is not None else [None if p is None else p[0] for p in out]


def compare(c):
    import swiglu_gemm_amd as sg
    cuda = lambda t: None if t is None else t.cuda()
    codes, scales, zeros = layouts(c)
    kw = dict(zeros=zeros, group=c.group, offsets=cuda(c.offsets), order=cuda(c.order), top_k=c.top_k)
    A, want = c.A.cuda(), c.sums()
    for alpha in (1.0, -0.5):
        for out in (torch.float32, c.dtype):
            C = sg.int4_gemm(A, codes, scales, torch.full((c.M, c.N), 7.0, dtype=out, device="cuda:0"), alpha=alpha, **kw)
            assert torch.equal(C.cpu(), (alpha * want).to(out)), (out, alpha)
    if c.N % 2 == 0:
        Y = torch.full((c.M, c.N // 2), 7.0, dtype=c.dtype, device="cuda:0")
        check(sg.int4_swiglu_gemm(A, codes, scales, Y, **kw), *c.swiglu(want), "swiglu")


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", sorted(HALF))
def test_exact(dtype):
    need_gpu()
    for c in cases(dtype):
        print("int4 exact %s %d x %d x %d, groups of %d" % (dtype, c.M, c.N, c.K, c.group), flush=True)
        compare(c)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", range(9))
@pytest.mark.parametrize("dtype", sorted(HALF))
def test_exact_of_every_tile(dtype, cfg, monkeypatch):
    need_gpu()
    monkeypatch.setenv("SG_FORCE_INT4", str(cfg))
    for c in cases(dtype):
        print("int4 exact, tile %d %s %d x %d x %d" % (cfg, dtype, c.M, c.N, c.K), flush=True)
        compare(c)


@pytest.mark.gpu
def test_exact_past_32_bits():
    """Five experts of 16384 x 65536, 512 MiB of codes each: the first and last columns of each expert's
    product, whole activations of -1, 0 and 1 and scales of 2^-9 and 2^-8."""
    need_gpu()
    import swiglu_gemm_amd as sg
    E, N, K, q = 5, 16384, 65536, 2.0 ** -9
    g = torch.Generator(device="cuda:0").manual_seed(6)
    nc, ns = sg.int4_shapes(N, K)
    codes = torch.randint(0, 256, (E, nc), dtype=U8, device="cuda:0", generator=g)
    scales = (q * 2.0 ** torch.randint(0, 2, (E, ns), device="cuda:0", generator=g)).half()
    A = torch.randint(-1, 2, (7, K), device="cuda:0", generator=g).half()
    offsets = torch.tensor([0, 1, 2, 3, 5, 7], dtype=torch.int32, device="cuda:0")
    C = sg.int4_gemm(A, codes, scales, torch.empty(7, N, device="cuda:0"), offsets=offsets).cpu()
    for n in (torch.arange(16), torch.arange(N - 16, N)):
        r, c = torch.meshgrid(n, torch.arange(K), indexing="ij")
        nib = c % 8 // 2 + 4 * (c % 2)
        at = ((r // 16) * (K // 128) + c // 128) * 1024 + 16 * (16 * (c % 32 // 8) + r % 16) + 4 * (c % 128 // 32)
        f = torch.arange(K // 128)[None]
        fat = ((n[:, None] // 16) * (K // 512) + f // 4) * 64 + 4 * (n[:, None] % 16) + f % 4
        for e in range(E):
            byte = codes[e][(at + nib // 2).cuda()].cpu()
            held = torch.where(nib % 2 == 1, byte >> 4, byte & 15), scales[e].cpu()[fat], None
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            want = A[lo:hi].cpu().double() @ ref.int4_values(*held, 128).t()
            assert torch.equal(C[lo:hi][:, n], want.float()), e
