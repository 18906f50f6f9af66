"""The 8-bit and ragged products against plain implementations in 64 bits.

Tolerances (fixed before the first run, by arithmetic):

* 16-bit operands: a product of two BF16 or F16 values is exact in FP32, so what is left
  are the FP32 additions of c terms. Each costs at most one unit in the last place (2^-23
  relative, rounding towards zero included) of a partial sum that is itself at most
  S = sum |a b|: an error of at most c * 2^-23 * S, whatever the order. Rounding to the
  output type adds half a step: eps / 2 of the value (plus half the smallest subnormal
  where the value is that small).
* int8: the sum is exact. float(sum), the product of the scales and its product with the
  sum round once each (2^-24): 4 * 2^-24 of the value with room for the second-order
  terms, then the output type's half step.
* accumulate: one more FP32 addition, 2^-24 of |base + value|.
* whole-number operands small enough that every partial sum stays below 2^24: exact.
* the quantiser: codes and scales equal (SwiGLU: see there).
"""
import math

import pytest
import torch

import nvfp4_mixture_experts_03_b200 as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def no_tf32():
    assert not torch.backends.cuda.matmul.allow_tf32
    yield
    assert nv.products_status() == 0      # no bounded wait gave up in any of these tests


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def padded(shape, dtype, extra=0, fill=None):
    """Rows that start every whole number of 16 bytes (plus `extra` such units), the gaps filled with NaN
    (or the extreme codes of int8) to show a read of them."""
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    ld = -(-shape[-1] // unit) * unit + extra * unit
    buf = torch.full((*shape[:-1], ld), (-128 if dtype == torch.int8 else NAN) if fill is None else fill, dtype=dtype, device=DEV)
    return buf[..., :shape[-1]]


def normal(shape, dtype, seed, std=1.0, extra=0):
    t = padded(shape, dtype, extra)
    t.copy_(torch.randn(*shape, generator=gen(seed), device=DEV) * std)
    return t


def codes(shape, seed, lo=-127, hi=127, extra=0):
    t = padded(shape, torch.int8, extra)
    t.copy_(torch.randint(lo, hi + 1, shape, generator=gen(seed), device=DEV, dtype=torch.int32))
    return t


def offsets_of(counts, first=0):
    off = [first]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def half_step(dtype, v):
    return v.abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def assert_within(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
                          f"{got[tuple(bad.nonzero()[0].tolist())].item()} for {ref[tuple(bad.nonzero()[0].tolist())].item()}"


def ref_fwd(x, w, off):
    """Value and sum of magnitudes, [rows][n] in 64 bits; rows of no group are NaN."""
    rows, n = x.shape[0], w.shape[1]
    y = torch.full((rows, n), NAN, dtype=torch.float64, device=DEV)
    s = y.clone()
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if hi > lo:
            a, b = x[lo:hi].double(), w[e].double()
            y[lo:hi], s[lo:hi] = a @ b.T, a.abs() @ b.abs().T
    return y, s


def tol16(c, s, y, out):
    return c * 2.0 ** -23 * s + (half_step(out, y) * (1 + 2.0 ** -8) if out != F32 else 0)


# ---------------------------------------------------------------- the product

# (counts of the groups, rows before the first, rows after the last)
SPLITS = [
    ((1,), 0, 0), ((8,), 0, 0), ((33,), 0, 0), ((300,), 0, 0),
    ((0, 5, 0, 1, 70, 0), 0, 0), ((129, 0, 257, 3), 0, 0), ((0, 0, 0), 0, 9),
    ((17, 64, 255), 5, 7), ((1,) * 40, 0, 0), ((256, 512, 31), 3, 0),
]


@pytest.mark.parametrize("n,k", [(256, 128), (1, 1), (40, 72), (129, 65), (300, 200), (513, 31), (128, 1000)])
@pytest.mark.parametrize("split", SPLITS, ids=lambda s: "-".join(map(str, s[0][:6])) + f"+{s[1]}+{s[2]}")
def test_forward_16bit(split, n, k):
    counts, before, after = split
    rows, E = before + sum(counts) + after, len(counts)
    off = offsets_of(counts, before)
    for dtype, out_dtype, extra in ((BF16, BF16, 0), (F16, F32, 2)):
        x = normal((rows, k), dtype, 1, extra=extra)
        w = normal((E, n, k), dtype, 2, 0.1)
        x[:before], x[before + sum(counts):] = NAN, math.inf
        out = torch.full((rows, n), 7.0, dtype=out_dtype, device=DEV)
        got = nv.grouped_gemm(x, w, off, out=out)
        assert got is out
        y, s = ref_fwd(x, w, off.tolist())
        mine = ~y.isnan().any(1)
        assert (out[~mine] == 7.0).all(), "a row of no group was written"
        assert_within(out[mine], y[mine], tol16(k, s[mine], y[mine], out_dtype), f"{dtype}")


@pytest.mark.parametrize("n,k", [(256, 128), (1, 1), (40, 80), (129, 65), (300, 200), (128, 1000)])
@pytest.mark.parametrize("split", SPLITS, ids=lambda s: "-".join(map(str, s[0][:6])) + f"+{s[1]}+{s[2]}")
def test_forward_int8(split, n, k):
    counts, before, after = split
    rows, E = before + sum(counts) + after, len(counts)
    off = offsets_of(counts, before)
    x, w = codes((rows, k), 3, extra=1), codes((E, n, k), 4)
    xs = torch.rand(rows, generator=gen(5), device=DEV) + 0.5
    ws = (torch.rand(E, n, generator=gen(6), device=DEV) + 0.5) * 1e-3
    y, _ = ref_fwd(x, w, off.tolist())
    for out_dtype in (F32, BF16):
        out = torch.full((rows, n), 7.0, dtype=out_dtype, device=DEV)
        nv.grouped_gemm(x, w, off, x_scale=xs, w_scale=ws, out=out)
        ref = y.clone()
        for e, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
            ref[lo:hi] *= xs[lo:hi, None].double() * ws[e].double()
        mine = ~ref.isnan().any(1)
        assert (out[~mine] == 7.0).all()
        tol = 4 * 2.0 ** -24 * ref.abs() + (half_step(out_dtype, ref) * (1 + 2.0 ** -8) if out_dtype != F32 else 0)
        assert_within(out[mine], ref[mine], tol[mine], f"int8 to {out_dtype}")


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 16, 17, 31, 32, 33, 64, 65, 200, 1025])
@pytest.mark.parametrize("n,k", [(1536, 2048), (2048, 768), (77, 333)])
def test_int8_dense(rows, n, k):
    x, w = codes((rows, k), 7), codes((n, k), 8)
    xs = torch.rand(rows, generator=gen(9), device=DEV) + 0.5
    ws = torch.rand(n, generator=gen(10), device=DEV) + 0.5
    ref = (x.double() @ w.double().T) * xs[:, None].double() * ws.double()
    assert_within(nv.gemm_int8(x, w, xs, ws), ref, 4 * 2.0 ** -24 * ref.abs(), "int8")
    base = torch.randn(rows, n, generator=gen(11), device=DEV)
    out = base.clone()
    nv.gemm_int8(x, w, xs, ws, out=out, accumulate=True)
    total = ref + base.double()
    assert_within(out, total, 4 * 2.0 ** -24 * ref.abs() + 2.0 ** -24 * (total.abs() + 2.0 ** -20 * ref.abs()), "int8 accumulated")


@pytest.mark.parametrize("rows,n,k", [(1, 48, 128), (20, 136, 256), (300, 264, 512), (600, 256, 8208)], ids=["token", "streamed", "tiles", "a split sum"])
@pytest.mark.parametrize("xs,ws", [(1e-30, 1e-10), (3e-38, 2e-5), (1e-41, 1e3), (1e33, 1e-33), (1e-33, 1e33), (1e25, 1e25), (-1e30, 1e-30),
                                   (1.2e-38, -1.2e-38), (3e38, 1e-44)])
def test_int8_scales_of_any_size(rows, n, k, xs, ws):
    """float(sum) and its two products round once each: 3 * 2^-24 of the value, 4 of them with room for the second order;
    a result below 2^-126 may lose half a step of 2^-149 (the first product is a whole multiple of that step, so it is
    exact wherever it is subnormal). A sum of zero gives zero, whatever the scales. The values pass FP32's largest number
    where the definition does."""
    x, w = codes((rows, k), 241), codes((n, k), 242)
    x[rows // 2] = 0
    w[n // 3] = 0
    vary = torch.linspace(0.75, 1.0, rows, device=DEV, dtype=torch.float64)
    xs = (vary * xs).float()
    ws = torch.full((n,), ws, device=DEV)
    ref = (x.double() @ w.double().T) * xs[:, None].double() * ws.double()
    most = torch.finfo(F32).max
    near = ((ref.abs() / most - 1).abs() < 1e-5)
    for out_dtype in (F32, BF16):
        got = nv.gemm_int8(x, w, xs, ws, out_dtype=out_dtype).double()
        assert (got[rows // 2] == 0).all() and (got[:, n // 3] == 0).all()
        inside = ref.abs() < torch.finfo(out_dtype).max * (1 - 2.0 ** -6)
        outside = (ref.abs() > most) & ~near
        assert (got[outside] == ref[outside].sign() * math.inf).all()
        tol = 4 * 2.0 ** -24 * ref.abs() + 2.0 ** -150 + (half_step(out_dtype, ref) * (1 + 2.0 ** -8) if out_dtype != F32 else 0)
        assert_within(got[inside], ref[inside], tol[inside], f"scales to {out_dtype}")


@pytest.mark.parametrize("counts,n,k", [((2, 1, 0, 3), 77, 200), ((300, 0, 33, 400), 200, 264), ((1300, 700), 520, 1040)],
                         ids=["streamed", "tiles", "pairs"])
def test_int8_rows_with_unusual_scales_beside_others(counts, n, k):
    """A few rows far too small or too large, a NaN and zeros among usual ones: the usual rows keep their bits, the others are
    within four roundings (below 2^-126: within half a step of 2^-149), also where they are added to something."""
    off, rows, E = offsets_of(counts), sum(counts), len(counts)
    x, w = codes((rows, k), 243), codes((E, n, k), 244)
    xs, ws = torch.rand(rows, generator=gen(245), device=DEV) + 0.5, torch.rand(E, n, generator=gen(246), device=DEV) + 0.5
    ws[:, n // 2] = 1e-12
    usual = {o: nv.grouped_gemm(x, w, off, x_scale=xs, w_scale=ws, out_dtype=o) for o in (F32, BF16)}
    odd = torch.zeros(rows, dtype=torch.bool, device=DEV)
    odd[::5] = True
    odd[-1] = True
    some = xs.clone()
    some[::5] = torch.tensor([1e-36, 1e30, 2e-41], device=DEV).repeat(rows)[: some[::5].numel()]
    some[-1] = NAN
    y, _ = ref_fwd(x, w, off.tolist())
    for e, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        y[lo:hi] *= some[lo:hi, None].double() * ws[e].double()
    for o in (F32, BF16):
        got = nv.grouped_gemm(x, w, off, x_scale=some, w_scale=ws, out_dtype=o)
        assert torch.equal(got[~odd], usual[o][~odd])
        assert got[-1].isnan().all()
        tol = 4 * 2.0 ** -24 * y[:-1].abs() + 2.0 ** -150 + (half_step(o, y[:-1]) * (1 + 2.0 ** -8) if o != F32 else 0)
        assert_within(got[:-1], y[:-1], tol, f"to {o}")
    base = torch.randn(rows, n, generator=gen(247), device=DEV)
    out = base.clone()
    nv.grouped_gemm(x, w, off, x_scale=some, w_scale=ws, out=out, accumulate=True)
    total = y[:-1] + base[:-1].double()
    assert_within(out[:-1], total, 4 * 2.0 ** -24 * y[:-1].abs() + 2.0 ** -24 * (total.abs() + 2.0 ** -20 * y[:-1].abs()), "added")


@pytest.mark.parametrize("rows", [1, 24, 200])
def test_int8_sums_are_exact_up_to_the_last_k(rows):
    """All codes -128 at the largest k: every sum is 2^14 * 131071, just below 2^31; with one code of x
    turned to 127 the sum is that less 255 * 128."""
    k, n = 131071, 40
    x, w = padded((rows, k), torch.int8), padded((n, k), torch.int8)
    x.fill_(-128)
    w.fill_(-128)
    x[rows // 2, k - 1] = 127
    one = torch.ones(rows, device=DEV)
    out = nv.gemm_int8(x, w, one, torch.ones(n, device=DEV))
    want = torch.full((rows, n), float(2 ** 14 * k), dtype=torch.float64, device=DEV)
    want[rows // 2] -= 255 * 128
    assert torch.equal(out, want.float())


@pytest.mark.parametrize("rows,n,k,counts", [(24, 96, 160, (24,)), (700, 384, 320, (0, 400, 1, 299)), (5000, 257, 520, (5000,))])
def test_16bit_accumulate(rows, n, k, counts):
    off = offsets_of(counts)
    x, w = normal((rows, k), BF16, 12), normal((len(counts), n, k), BF16, 13, 0.1)
    base = torch.randn(rows, n, generator=gen(14), device=DEV)
    out = base.clone()
    nv.grouped_gemm(x, w, off, out=out, accumulate=True)
    y, s = ref_fwd(x, w, off.tolist())
    assert_within(out, y + base, k * 2.0 ** -23 * s + 2.0 ** -24 * ((y + base).abs() + k * 2.0 ** -23 * s), "accumulate")


# -------------------------------------------------------------- the gradients

@pytest.mark.parametrize("n,k", [(256, 128), (1, 1), (40, 72), (129, 65), (65, 300), (31, 513), (1000, 128)])
@pytest.mark.parametrize("split", SPLITS, ids=lambda s: "-".join(map(str, s[0][:6])) + f"+{s[1]}+{s[2]}")
def test_gradients(split, n, k):
    counts, before, after = split
    rows, E = before + sum(counts) + after, len(counts)
    off = offsets_of(counts, before)
    for dtype, out_dtype in ((BF16, F32), (F16, F16)):
        x, dy = normal((rows, k), dtype, 21, extra=1), normal((rows, n), dtype, 22, 0.5)
        w = normal((E, n, k), dtype, 23, 0.1)
        for t in (x, dy):      # rows of no group reach neither gradient
            t[:before], t[before + sum(counts):] = NAN, math.inf
        # dx[p] = dy[p] W_e: the product with each matrix transposed
        y, s = ref_fwd(dy, w.transpose(1, 2), off.tolist())
        dx = torch.full((rows, k), 7.0, dtype=out_dtype, device=DEV)
        nv.grouped_gemm_dx(dy, w, off, out=dx)
        mine = ~y.isnan().any(1)
        assert (dx[~mine] == 7.0).all(), "a row of no group was written"
        assert_within(dx[mine], y[mine], tol16(n, s[mine], y[mine], out_dtype), "dx")
        dw = nv.grouped_gemm_dw(dy, x, off, out_dtype=out_dtype)
        assert dw.shape == (E, n, k)
        for e, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
            a, b = dy[lo:hi].double(), x[lo:hi].double()
            ref, s = a.T @ b, a.abs().T @ b.abs()
            if hi == lo:
                assert (dw[e] == 0).all(), "an expert without rows has no gradient"
            assert_within(dw[e], ref, tol16(max(hi - lo, 1), s, ref, out_dtype), f"dw of {e}")


def test_gradients_are_the_formulas_and_the_differences():
    """Small whole numbers, so that every sum is exact in FP32: the three products satisfy the adjoint identity
    and the differences of the bilinear form as equations, not up to a tolerance."""
    counts, n, k = (40, 0, 7, 130), 72, 104
    rows, E, off = sum(counts), len(counts), offsets_of(counts)

    def whole(shape, seed, dtype=BF16):
        t = padded(shape, dtype)
        t.copy_(torch.randint(-4, 5, shape, generator=gen(seed), device=DEV))
        return t

    x, w, dy = whole((rows, k), 31), whole((E, n, k), 32), whole((rows, n), 33)
    y = nv.grouped_gemm(x, w, off, out_dtype=F32).double()
    dx = nv.grouped_gemm_dx(dy, w, off, out_dtype=F32).double()
    dw = nv.grouped_gemm_dw(dy, x, off).double()
    loss = (y * dy.double()).sum()
    assert loss == (dx * x.double()).sum() == (dw * w.double()).sum()
    ddx, ddw = whole((rows, k), 34), whole((E, n, k), 35)
    up = nv.grouped_gemm((x + ddx), w, off, out_dtype=F32).double()
    down = nv.grouped_gemm((x - ddx), w, off, out_dtype=F32).double()
    assert ((up - down) * dy.double()).sum() / 2 == (dx * ddx.double()).sum()
    up = nv.grouped_gemm(x, padded_copy(w + ddw), off, out_dtype=F32).double()
    down = nv.grouped_gemm(x, padded_copy(w - ddw), off, out_dtype=F32).double()
    assert ((up - down) * dy.double()).sum() / 2 == (dw * ddw.double()).sum()


def padded_copy(t):
    out = padded(tuple(t.shape), t.dtype)
    out.copy_(t)
    return out


def test_dw_without_rows_and_accumulated():
    n, k, E = 96, 200, 3
    none = torch.empty(0, n, dtype=BF16, device=DEV), torch.empty(0, k, dtype=BF16, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    assert (nv.grouped_gemm_dw(*none, off) == 0).all()
    base = torch.randn(E, n, k, generator=gen(41), device=DEV)
    out = base.clone()
    nv.grouped_gemm_dw(*none, off, out=out, accumulate=True)
    assert torch.equal(out, base)
    dy, x = normal((100, n), BF16, 42), normal((100, k), BF16, 43)
    off = offsets_of((60, 0, 40))
    nv.grouped_gemm_dw(dy, x, off, out=out, accumulate=True)
    assert torch.equal(out[1], base[1])
    for e, lo, hi in ((0, 0, 60), (2, 60, 100)):
        ref = dy[lo:hi].double().T @ x[lo:hi].double()
        s = dy[lo:hi].double().abs().T @ x[lo:hi].double().abs()
        t = ref + base[e].double()
        assert_within(out[e], t, 60 * 2.0 ** -23 * s + 2.0 ** -24 * (t.abs() + 60 * 2.0 ** -23 * s), f"dw {e}")


# ------------------------------------------------------------- the quantiser

def ref_codes(v):
    """v in 64 bits -> (codes, scale as FP32): the definition."""
    scale = (v.abs().amax(1) / 127.0).float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    q = (v / safe[:, None]).round().clamp(-127, 127) * (scale > 0)[:, None]
    return q.to(torch.int8), scale


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (3, 7), (5, 8), (2, 33), (700, 96), (2500, 2048), (4, 5000),
                                       (3, 70001), (1300, 100), (149, 20000)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize_codes_are_exact(dtype, rows, cols):
    for tight in (True, False):
        x = normal((rows, cols), dtype, 51, extra=1)
        x[:, ::17] *= 20
        x[rows // 2] = 0
        x[0, : cols // 2] = x[0].abs().max() / 2      # 63.5 steps: a tie that 1 / scale rounds either way
        if tight:
            x = x.contiguous()
        q, scale = nv.quantize_int8(x)
        rq, rs = ref_codes(x.double())
        assert torch.equal(scale, rs)
        assert torch.equal(q, rq)


def test_quantize_borders():
    """Every half step k + 1/2 of rows whose scale is exact and of rows whose scale is not, and their FP32 neighbours."""
    rows = []
    for amax in (127.0, 254.0, 1.0, 3.1415927, 1.1754944e-38, 2.0 ** -140, 3.4028235e38, 190 * 2.0 ** -149, 63 * 2.0 ** -149,
                 64 * 2.0 ** -149):
        a = torch.tensor(amax, dtype=F32)
        s = (a.double() / 127).float().double()
        h = ((torch.arange(-127, 128).double() + 0.5) * s).float()
        v = torch.cat([h, torch.nextafter(h, torch.tensor(math.inf)), torch.nextafter(h, torch.tensor(-math.inf))]).clamp(-a, a)
        rows.append(torch.cat([v, a[None]]))
    x = torch.stack(rows).to(DEV)
    for cols in (x.shape[1], x.shape[1] - 3):
        y = x[:, x.shape[1] - cols:]
        q, scale = nv.quantize_int8(y)
        rq, rs = ref_codes(y.double())
        assert torch.equal(scale, rs)
        assert torch.equal(q, rq)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("swiglu", [False, True])
def test_quantize_non_finite_rows_are_reported_in_their_scale(dtype, swiglu):
    x = normal((8, 512), dtype, 61)
    clean_q, clean_s = nv.quantize_int8(x.clone(), swiglu=swiglu)
    x[2, 5], x[4, 100], x[6, 300], x[7, 511] = NAN, math.inf, -math.inf, NAN
    q, scale = nv.quantize_int8(x, swiglu=swiglu)
    for r in range(8):
        if r in (2, 4, 6, 7):
            assert scale[r].isnan() and (q[r] == 0).all()
        else:
            assert scale[r] == clean_s[r] and torch.equal(q[r], clean_q[r])


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 768), (4, 768), (3, 9), (700, 96), (3000, 768), (2, 9000), (1300, 101)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_swiglu_quantize(dtype, rows, cols):
    """h = SiLU(g) u in FP32: exp's argument rounds (|g| 2^-24 of the value, |g| <= 88 where the value counts) and the
    exponential, the sum, the quotient and the product add at most 8 * 2^-24; with |g| <= 32 here that is below 2^-18.
    So the scale agrees to 2^-18, and a code differs from the quotient's by less than half plus 127 * 2^-17."""
    x = normal((rows, 2 * cols), dtype, 71, 3.0).clamp(-32, 32)
    q, scale = nv.quantize_int8(x, swiglu=True)
    g, u = x.double().split(cols, 1)
    h = g * torch.sigmoid(g) * u
    amax = h.abs().amax(1)
    assert ((scale.double() * 127 - amax).abs() <= 2.0 ** -18 * amax).all()
    t = h / torch.where(amax > 0, amax / 127, torch.ones_like(amax))[:, None]
    assert ((q.double() - t).abs() <= 0.5 + 127 * 2.0 ** -17).all()
    assert (q[torch.arange(rows, device=DEV), h.abs().argmax(1)].abs() == 127).all()


@pytest.mark.parametrize("lo,hi", [(-87.0, -60.0), (-60.0, -30.0), (-30.0, -10.0), (-87.0, -86.0), (-5.0, 5.0), (20.0, 88.0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_swiglu_values_at_every_gate(dtype, lo, hi):
    """Rows of one value, whose scale is |SiLU(g) u| / 127, and rows of many such values, which their codes show. In units of
    2^-24: the exponential is off by up to 4 (2^-22.5 and a rounding), 1 + it by 1, its inverse by 2, the products with g and u by 1
    each, the scale's quotient by 1: 10, below 2^-20."""
    rows = 4000
    g = (torch.rand(rows, generator=gen(271), device=DEV, dtype=torch.float64) * (hi - lo) + lo).to(dtype)
    u = ((torch.rand(rows, generator=gen(272), device=DEV, dtype=torch.float64) + 0.5) * 1e3).to(dtype)
    h = g.double() * torch.sigmoid(g.double()) * u.double()
    q, scale = nv.quantize_int8(torch.stack([g, u], 1).contiguous(), swiglu=True)
    assert ((scale.double() * 127 - h.abs()).abs() <= 2.0 ** -20 * h.abs()).all()
    assert torch.equal(q[:, 0], (h.sign() * 127).to(torch.int8))
    wide = torch.cat([g.view(40, 100), u.view(40, 100)], 1)
    q, scale = nv.quantize_int8(wide, swiglu=True)
    t = h.view(40, 100) / (h.view(40, 100).abs().amax(1, keepdim=True) / 127)
    assert ((q.double() - t).abs() <= 0.5 + 127 * 2.0 ** -19).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_swiglu_rows_at_the_ends_of_the_range(dtype):
    """Gates of any size, infinities and NaN, each with ordinary, huge and non-finite ups: a row that holds something not finite,
    or whose value passes FP32's largest number, has scale NaN and code 0; else its scale is that of the definition, or 0 below -87."""
    inf = math.inf
    pairs = [(g, u) for g in (-inf, inf, NAN, -3e38, 3e38, -1e30, 1e30, -88.5, -87.5, -87.0, 88.0, 89.0, 0.0, -0.0)
             for u in (1.0, 0.0, -2.0, inf, -inf, NAN, 1e30)]
    x = torch.tensor(pairs, device=DEV).to(dtype)
    q, scale = nv.quantize_int8(x, swiglu=True)
    g, u = x.double().unbind(1)
    h = (g * torch.sigmoid(g) * u).abs()
    bad = ~x.isfinite().all(1) | ~(h <= torch.finfo(F32).max)
    assert scale[bad].isnan().all() and (q[bad] == 0).all()
    near = (scale.double() * 127 - h).abs() <= 2.0 ** -20 * h
    assert (near | ((g < -87) & (scale == 0)))[~bad].all()


def test_swiglu_quantize_far_gates():
    """Gates whose exponential leaves FP32 either way: SiLU is 0 or the gate itself."""
    g = torch.tensor([[-1e30, -200.0, -89.0, -87.5, 200.0, 1e5, 0.0, 88.9]], device=DEV)
    u = torch.tensor([[1.0, 1.0, 1.0, 1.0, 500.0, 1.0, 3.0, 1.0]], device=DEV)
    q, scale = nv.quantize_int8(torch.cat([g, u], 1), swiglu=True)
    assert scale.item() == torch.tensor(1e5 / 127).item()
    assert q[0].tolist() == [0, 0, 0, 0, 127, 127, 0, 0]


def test_quantize_writes_its_rows_only():
    x = normal((20, 100), BF16, 81)
    q = torch.full((22, 128), 99, dtype=torch.int8, device=DEV)
    scale = torch.full((22,), -1.0, device=DEV)
    nv.quantize_int8(x, q=q[1:21, :100], scale=scale[1:21])
    assert (q[0] == 99).all() and (q[21] == 99).all() and (q[:, 100:] == 99).all()
    assert scale[0] == -1 and scale[21] == -1
    assert torch.equal(q[1:21, :100], ref_codes(x.double())[0])


# ------------------------------------------------------- how it may be called

def _all_calls(rows=300, n=136, k=264, seed=91):
    counts = (0, 1, rows - 40, 39)
    off = offsets_of(counts)
    x, dy = normal((rows, k), BF16, seed), normal((rows, n), BF16, seed + 1)
    w = normal((4, n, k), BF16, seed + 2)
    wq, ws = codes((4, n, k), seed + 3), torch.rand(4, n, generator=gen(seed + 4), device=DEV)

    def run(**kw):
        q, s = nv.quantize_int8(x, **kw)
        hq, hs = nv.quantize_int8(x, swiglu=True, **kw)
        return [q, s, hq, hs, nv.grouped_gemm(x, w, off, **kw), nv.grouped_gemm(q, wq, off, x_scale=s, w_scale=ws, **kw),
                nv.gemm_int8(q, wq[1], s, ws[1], **kw), nv.gemm_int8(q[:1], wq[1], s[:1], ws[1], **kw),
                nv.grouped_gemm(x[:2], w, offsets_small, **kw), nv.grouped_gemm_dx(dy, w, off, **kw), nv.grouped_gemm_dw(dy, x, off, **kw)]

    offsets_small = offsets_of((0, 1, 0, 1))
    return run, (x, dy, w)


def test_the_same_bits_on_every_run_and_stream():
    run, _ = _all_calls()
    want = run()
    torch.cuda.synchronize()
    other = [torch.cuda.Stream() for _ in range(3)]
    several = [run(stream=s) for s in other for _ in range(3)]     # calls side by side
    torch.cuda.synchronize()
    for got in [run()] + several:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    run, inputs = _all_calls()
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for seed in (1, 2):
        for i, t in enumerate(inputs):
            t.copy_(torch.randn(*t.shape, generator=gen(100 * seed + i), device=DEV))
        g.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_wrong_offsets_stay_in_range():
    """Offsets past the rows, below zero or out of order are clamped: rows go wrong, nothing is written out of range."""
    rows, n, k = 100, 64, 64
    x, dy, w = normal((rows, k), BF16, 95), normal((rows, n), BF16, 96), normal((3, n, k), BF16, 97)
    for off in ([0, 50, 200, 300], [-7, 20, 10, 100], [90, 40, 1 << 30, 3], [2 ** 31 - 1, -2 ** 31, 50, 100]):
        off = torch.tensor(off, dtype=torch.int32, device=DEV)
        for fn, a, b, cols in ((nv.grouped_gemm, x, w, n), (nv.grouped_gemm_dx, dy, w, k)):
            out = torch.full((rows + 20, cols), 7.0, device=DEV)
            fn(a, b, off, out=out[10:-10], out_dtype=F32)
            torch.cuda.synchronize()
            assert (out[:10] == 7.0).all() and (out[-10:] == 7.0).all()
        assert nv.grouped_gemm_dw(dy, x, off).shape == (3, n, k)
    torch.cuda.synchronize()


@pytest.mark.parametrize("off", [[0, 50, 200, 300], [-7, 20, 10, 100], [90, 40, 1 << 30, 3], [2 ** 31 - 1, -2 ** 31, 50, 100],
                                 [30, 10, 20, 60], [0, 60, 59, 61], [5, 99, 98, 97], [-1, -2, -3, -4], [100, 100, 100, 100], [0, 0, 7, 5]])
@pytest.mark.parametrize("n,k", [(64, 64), (1024, 64), (64, 1024)])
def test_wrong_offsets_are_clamped_alike_in_every_kernel(off, n, k):
    """The same rows for the same offsets, whichever kernel takes the call: each offset clamped into [0, rows] and to no less
    than those before it. (100 rows of 64 columns are streamed, of 1024 not.)"""
    rows, E = 100, 3
    x, dy, w = normal((rows, k), BF16, 251), normal((rows, n), BF16, 252), normal((E, n, k), BF16, 253, 0.1)
    clamped, top = [], 0
    for v in off:
        top = max(top, min(max(v, 0), rows))
        clamped.append(top)
    off = torch.tensor(off, dtype=torch.int32, device=DEV)
    for fn, a, m, cols in ((nv.grouped_gemm, x, w, n), (nv.grouped_gemm_dx, dy, w.transpose(1, 2), k)):
        out = torch.full((rows, cols), 7.0, device=DEV)
        fn(a, w, off, out=out)
        y, s = ref_fwd(a, m, clamped)
        mine = ~y.isnan().any(1)
        assert (out[~mine] == 7.0).all()
        assert_within(out[mine], y[mine], tol16(a.shape[1], s[mine], y[mine], F32), fn.__name__)
    dw = nv.grouped_gemm_dw(dy, x, off)
    for e, (lo, hi) in enumerate(zip(clamped[:-1], clamped[1:])):
        a, b = dy[lo:hi].double(), x[lo:hi].double()
        assert_within(dw[e], a.T @ b, tol16(max(hi - lo, 1), a.abs().T @ b.abs(), a.T @ b, F32), f"dw of {e}")


def test_element_offsets_past_32_bits():
    """Rows whose elements start past 2^31 from the first, in x and in the output, and matrices that do."""
    k, ld = 136, (1 << 26) + 8
    buf = torch.empty(40 * ld, dtype=torch.int8, device=DEV)
    q = torch.as_strided(buf, (40, k), (ld * 1, 1)) if ld % 16 == 0 else torch.as_strided(buf, (40, k), (ld + 8, 1))[:38]
    rows = q.shape[0]
    x = normal((rows, k), F32, 98)
    scale = torch.empty(rows, device=DEV)
    nv.quantize_int8(x, q=q, scale=scale)
    assert torch.equal(q, ref_codes(x.double())[0])
    w, ws = codes((48, k), 99), torch.ones(48, device=DEV)
    out = nv.gemm_int8(q, w, scale, ws)
    ref = (q.double() @ w.double().T) * scale[:, None].double()
    assert_within(out, ref, 4 * 2.0 ** -24 * ref.abs(), "far rows")
    del buf, q
    E, n = 600, 2048
    wide = torch.zeros(E, n, 2048, dtype=BF16, device=DEV)      # 2.5e9 elements
    wide[E - 1].copy_(torch.randn(n, 2048, generator=gen(100), device=DEV) * 0.1)
    for rows in (3, 150):
        x, dy = normal((rows, 2048), BF16, 101), normal((rows, n), BF16, 102)
        off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        off[E] = rows
        ref, s = x.double() @ wide[-1].double().T, x.double().abs() @ wide[-1].double().abs().T
        assert_within(nv.grouped_gemm(x, wide, off), ref, tol16(2048, s, ref, BF16), "far matrix")
        ref, s = dy.double() @ wide[-1].double(), dy.double().abs() @ wide[-1].double().abs()
        assert_within(nv.grouped_gemm_dx(dy, wide, off), ref, tol16(n, s, ref, BF16), "far matrix, dx")
    dw = nv.grouped_gemm_dw(dy, x, off, out_dtype=BF16)
    ref, s = dy.double().T @ x.double(), dy.double().abs().T @ x.double().abs()
    assert_within(dw[-1], ref, tol16(150, s, ref, BF16), "far matrix, dw")
    assert not dw[:-1].any()


def test_dw_of_the_most_rows_in_one_of_many_groups():
    """2^30 rows, all but a few of them in one of 1024 groups: a single CTA's sum of more than three seconds."""
    rows, c, E, e = nv.products.MAX_EXTENT, 8, nv.products.MAX_GROUPS, 700
    x, dy = (torch.zeros(rows, c, dtype=BF16, device=DEV) for _ in range(2))
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[: e + 1], off[e + 1:] = 5, rows - 3
    some = torch.tensor([5, 6, 63, 64, 2 ** 21 + 3, 2 ** 29, rows - 70, rows - 5, rows - 4], device=DEV)
    x[some] = torch.randint(-4, 5, (some.numel(), c), generator=gen(261), device=DEV).to(BF16)
    dy[some] = torch.randint(-4, 5, (some.numel(), c), generator=gen(262), device=DEV).to(BF16)
    x[:5], dy[:5], x[-3:], dy[-3:] = NAN, NAN, NAN, NAN
    dw = nv.grouped_gemm_dw(dy, x, off)
    assert nv.products_status() == 0
    assert torch.equal(dw[e], dy[some].float().T @ x[some].float())
    assert not dw[:e].any() and not dw[e + 1:].any()


def test_values_outside_a_groups_rows_do_not_reach_it():
    """NaN and infinities in the neighbouring expert's rows and matrices stay there."""
    counts, n, k = (70, 33, 100), 200, 136
    off, rows = offsets_of(counts), sum(counts)
    x, dy, w = normal((rows, k), BF16, 111), normal((rows, n), BF16, 112), normal((3, n, k), BF16, 113)
    want = nv.grouped_gemm(x, w, off), nv.grouped_gemm_dx(dy, w, off), nv.grouped_gemm_dw(dy, x, off)
    for t in (x, dy):
        t[:70], t[103:] = NAN, math.inf
    w[0], w[2] = math.inf, NAN
    got = nv.grouped_gemm(x, w, off), nv.grouped_gemm_dx(dy, w, off), nv.grouped_gemm_dw(dy, x, off)
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a[70:103], b[70:103])
    assert torch.equal(got[2][1], want[2][1])


def _check_all(x, dy, w, off, out_fwd, out_dx, out_dw, dw_dtype):
    """All three products of one set of operands against 64 bits."""
    n, k = w.shape[1:]
    y, s = ref_fwd(x, w, off)
    mine = ~y.isnan().any(1)
    assert_within(out_fwd[mine], y[mine], tol16(k, s[mine], y[mine], out_fwd.dtype), "product")
    y, s = ref_fwd(dy, w.transpose(1, 2), off)
    assert_within(out_dx[mine], y[mine], tol16(n, s[mine], y[mine], out_dx.dtype), "dx")
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        ref, s = dy[lo:hi].double().T @ x[lo:hi].double(), dy[lo:hi].double().abs().T @ x[lo:hi].double().abs()
        assert_within(out_dw[e], ref, tol16(max(hi - lo, 1), s, ref, dw_dtype), f"dw of {e}")


@pytest.mark.parametrize("counts,n,k", [
    ((3000,), 512, 512),                                   # whole pair tiles
    ((1999, 0, 513, 70, 2), 576, 640),                     # ragged ones, 64-column boxes
    ((700, 1300), 520, 1032),                              # columns that no 64 divides
    ((257, 255, 256, 31, 33, 63, 65, 127, 129, 1), 768, 264),
    ((5000, 1), 136, 2048), ((40,) * 60, 640, 256),
])
@pytest.mark.parametrize("dtype,wide", [(BF16, BF16), (F16, F32)])
def test_large_tiles(counts, n, k, dtype, wide):
    off, rows, E = offsets_of(counts), sum(counts), len(counts)
    x, dy, w = normal((rows, k), dtype, 141), normal((rows, n), dtype, 142, 0.5), normal((E, n, k), dtype, 143, 0.1)
    _check_all(x, dy, w, off.tolist(), nv.grouped_gemm(x, w, off, out_dtype=wide), nv.grouped_gemm_dx(dy, w, off, out_dtype=wide),
               nv.grouped_gemm_dw(dy, x, off, out_dtype=wide), wide)


@pytest.mark.parametrize("counts,n,k", [
    ((10000,), 200, 304), ((3001,), 130, 72), ((2000, 0, 71, 900), 96, 136), ((16384,), 64, 64), ((700,), 520, 40),
    ((5, 4000), 33, 129), ((300,), 256, 4104), ((300,), 4104, 256),
])
def test_long_sums_of_few_tiles(counts, n, k):
    """Sums that several CTAs share: the three products, accumulated ones too."""
    off, rows, E = offsets_of(counts), sum(counts), len(counts)
    x, dy, w = normal((rows, k), BF16, 145), normal((rows, n), BF16, 146, 0.5), normal((E, n, k), BF16, 147, 0.1)
    for wide in (BF16, F32):
        _check_all(x, dy, w, off.tolist(), nv.grouped_gemm(x, w, off, out_dtype=wide),
                   nv.grouped_gemm_dx(dy, w, off, out_dtype=wide), nv.grouped_gemm_dw(dy, x, off, out_dtype=wide), wide)
    base = torch.randn(E, n, k, generator=gen(148), device=DEV)
    out = base.clone()
    nv.grouped_gemm_dw(dy, x, off, out=out, accumulate=True)
    assert (out == base + nv.grouped_gemm_dw(dy, x, off)).all()
    for _ in range(3):
        assert torch.equal(nv.grouped_gemm_dw(dy, x, off), nv.grouped_gemm_dw(dy, x, off))


@pytest.mark.parametrize("rows,n,k", [(600, 256, 8208), (257, 40, 16384), (70, 130, 4000)])
def test_int8_long_sums(rows, n, k):
    x, w = codes((rows, k), 175), codes((n, k), 176)
    xs, ws = torch.rand(rows, generator=gen(177), device=DEV) + 0.5, torch.rand(n, generator=gen(178), device=DEV) + 0.5
    ref = (x.double() @ w.double().T) * xs[:, None].double() * ws.double()
    for out_dtype in (F32, BF16):
        got = nv.gemm_int8(x, w, xs, ws, out_dtype=out_dtype)
        assert_within(got, ref, 4 * 2.0 ** -24 * ref.abs() + (half_step(out_dtype, ref) * (1 + 2.0 ** -8) if out_dtype != F32 else 0), "int8")


def test_no_rows():
    w = normal((3, 40, 64), BF16, 179)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert nv.grouped_gemm(torch.empty(0, 64, dtype=BF16, device=DEV), w, off).shape == (0, 40)
    assert nv.grouped_gemm_dx(torch.empty(0, 40, dtype=BF16, device=DEV), w, off).shape == (0, 64)
    q, scale = nv.quantize_int8(torch.empty(0, 64, dtype=BF16, device=DEV))
    assert q.shape == (0, 64) and scale.shape == (0,)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_outputs_with_rows_of_any_alignment(dtype):
    """Outputs whose rows start anywhere, with what lies between and around them left alone."""
    counts, n, k = (900, 3, 411), 517, 531
    off, rows, E = offsets_of(counts, 2), sum(counts), len(counts)
    x, dy, w = normal((rows + 5, k), BF16, 151), normal((rows + 5, n), BF16, 152), normal((E, n, k), BF16, 153, 0.1)
    size = dtype.itemsize

    def around(lead, cols):
        buf = torch.full((lead * (cols + 4) + 1,), 7.0, dtype=dtype, device=DEV)
        return buf, torch.as_strided(buf, (lead, cols), (cols + 4 if size == 4 else cols + 3, 1), 1)

    bf, of = around(rows + 5, n)
    bx, ox = around(rows + 5, k)
    bw, ow = around(E * n, k)
    nv.grouped_gemm(x, w, off, out=of)
    nv.grouped_gemm_dx(dy, w, off, out=ox)
    ow3 = torch.as_strided(bw, (E, n, k), (n * ow.stride(0), ow.stride(0), 1), 1)
    nv.grouped_gemm_dw(dy, x, off, out=ow3)
    _check_all(x, dy, w, off.tolist(), of, ox, ow3, dtype)
    for buf, o, last in ((bf, of, rows + 2), (bx, ox, rows + 2), (bw, ow, E * n)):
        written = torch.zeros_like(buf, dtype=torch.bool)
        first = 0 if o is ow else 2
        torch.as_strided(written, o.shape, o.stride(), 1)[first:last] = True
        assert (buf[~written] == 7.0).all()


@pytest.mark.parametrize("rows,n,k", [(6000, 200, 264), (20, 40, 72), (300, 264, 520)])
def test_the_most_groups(rows, n, k):
    """1024 groups, most of them small, some empty, one large."""
    E = nv.products.MAX_GROUPS
    p = torch.rand(E, generator=gen(161), device=DEV) ** 6
    p[700] = 30.0
    counts = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=gen(162)), minlength=E).tolist()
    off = offsets_of(counts)
    x, dy, w = normal((rows, k), BF16, 163), normal((rows, n), BF16, 164, 0.5), normal((E, n, k), BF16, 165, 0.1)
    _check_all(x, dy, w, off.tolist(), nv.grouped_gemm(x, w, off), nv.grouped_gemm_dx(dy, w, off),
               nv.grouped_gemm_dw(dy, x, off, out_dtype=BF16), BF16)


def test_int8_large_tiles():
    counts, n, k = (1300, 0, 700, 31, 257), 520, 1040
    off, rows, E = offsets_of(counts), sum(counts), len(counts)
    x, w = codes((rows, k), 171), codes((E, n, k), 172)
    xs, ws = torch.rand(rows, generator=gen(173), device=DEV) + 0.5, torch.rand(E, n, generator=gen(174), device=DEV) + 0.5
    y, _ = ref_fwd(x, w, off.tolist())
    for e, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        y[lo:hi] *= xs[lo:hi, None].double() * ws[e].double()
    for out_dtype in (F32, BF16, F16):
        x_s = xs * (1e-4 if out_dtype == F16 else 1.0)
        ref = y * (x_s / xs)[:, None].double()
        got = nv.grouped_gemm(x, w, off, x_scale=x_s, w_scale=ws, out_dtype=out_dtype)
        tol = 5 * 2.0 ** -24 * ref.abs() + (half_step(out_dtype, ref) * (1 + 2.0 ** -8) if out_dtype != F32 else 0)
        assert_within(got, ref, tol, f"int8 to {out_dtype}")      # (x_s / xs rounds once more)


def test_first_calls_of_a_process_may_be_captured():
    """A fresh process whose first calls of the library run inside a capture, twice over the same buffers."""
    import os
    import subprocess
    import sys
    from conftest import ROOT
    code = """
import torch, nvfp4_mixture_experts_03_b200 as nv
torch.manual_seed(0)
x = torch.randn(300, 256, device="cuda", dtype=torch.bfloat16)
w = torch.randn(4, 512, 256, device="cuda", dtype=torch.bfloat16)
off = torch.tensor([0, 100, 100, 260, 300], device="cuda", dtype=torch.int32)
torch.cuda.synchronize()
def run():
    q, s = nv.quantize_int8(x)
    y = nv.grouped_gemm(x, w, off)
    return [q, s, y, nv.grouped_gemm(x[:1], w[:1]), nv.grouped_gemm_dx(y, w, off), nv.grouped_gemm_dw(y, x, off)]
g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
with torch.cuda.graph(g1):
    a = run()
with torch.cuda.graph(g2):
    b = run()
s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
for _ in range(5):
    with torch.cuda.stream(s1):
        g1.replay()
    with torch.cuda.stream(s2):
        g2.replay()
torch.cuda.synchronize()
c = run()
for u, v, z in zip(a, b, c):
    assert torch.equal(u, v) and torch.equal(u, z)
assert nv.products_status() == 0
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def _chain(steps, sync, layer):
    """Calls that each read what the one before wrote, through buffers that are written again and again; the
    routed layer's decode kernel and torch's own among them."""
    done = torch.cuda.synchronize if sync else (lambda: None)
    E, H, I = 4, 256, 192
    w, wq = normal((E, I, H), BF16, 201, 0.06), codes((H, I), 202)
    w2, ws = normal((E, I, H), BF16, 203, 0.06), torch.full((H,), 4e-4, device=DEV)
    x = normal((60, H), F32, 204)
    xb, h = torch.empty(60, H, dtype=BF16, device=DEV), torch.empty(60, I, dtype=BF16, device=DEV)
    q, s = torch.empty(60, I, dtype=torch.int8, device=DEV), torch.empty(60, device=DEV)
    dx, dw = torch.empty(60, H, dtype=BF16, device=DEV), torch.empty(E, I, H, device=DEV)
    logits, square = torch.randn(4, 8, generator=gen(205), device=DEV), codes((H, H), 206)
    off, small = offsets_of((9, 0, 40, 11)), offsets_of((1, 0, 2, 1))
    xq, xs = torch.empty(4, H, dtype=torch.int8, device=DEV), torch.empty(4, device=DEV)
    out = torch.empty(4, H, device=DEV)
    for _ in range(steps):
        xb.copy_(x); done()
        nv.grouped_gemm(xb, w, off, out=h); done()
        nv.grouped_gemm(xb[:4], w, small, out=h[:4]); done()          # streamed
        nv.quantize_int8(h, q=q, scale=s); done()
        nv.gemm_int8(q, wq, s, ws, out=x, accumulate=True); done()
        nv.grouped_gemm_dx(h, w2, off, out=dx); done()
        nv.grouped_gemm_dw(h, xb, off, out=dw); done()
        nv.quantize_int8(dx[:4], q=xq, scale=xs); done()
        layer.forward(xq, x_scale=xs, logits=logits, out=out); done()
        nv.gemm_int8(xq, square, xs, ws, out=out, accumulate=True); done()
        x.mul_(0.5)
        x[:4].add_(out, alpha=1e-3); done()
    torch.cuda.synchronize()
    return [t.clone() for t in (x, h, q, s, dx, dw, xq, xs, out)]


def test_chains_of_dependent_calls():
    """A kernel may start before the one ahead of it has ended, but touches nothing until then: a chain without a
    wait gives the bits of one that waits after every call; so does its capture, replayed."""
    import synth
    dims = synth.LayerDims(E=8, H=256, I=128, K=2)
    layer = nv.MoELayer.from_layer(synth.make_layer(dims, seed=9).to(DEV), top_k=dims.K, max_tokens=4)
    want = _chain(25, True, layer)
    for _ in range(4):
        for a, b in zip(_chain(25, False, layer), want):
            assert torch.equal(a, b)
    assert layer.status() == 0
    layer.close()


def test_captured_across_two_streams():
    x, w = normal((300, 256), BF16, 211), normal((2, 320, 256), BF16, 212, 0.1)
    off = offsets_of((100, 200))
    y, z, u = (torch.empty(300, n, dtype=BF16, device=DEV) for n in (320, 256, 320))

    def run(side):
        main = torch.cuda.current_stream()
        nv.grouped_gemm(x, w, off, out=y)
        side.wait_stream(main)
        nv.grouped_gemm_dx(y, w, off, out=z, stream=side)
        q, s = nv.quantize_int8(y)
        main.wait_stream(side)
        nv.grouped_gemm(z, w, off, out=u)
        return q, s

    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    run(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        q, s = run(side)
    for seed in (1, 2, 3):
        x.copy_(torch.randn(*x.shape, generator=gen(213 + seed), device=DEV))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, z, u, q, s)]
        nv.grouped_gemm(x, w, off, out=y); torch.cuda.synchronize()
        nv.grouped_gemm_dx(y, w, off, out=z); torch.cuda.synchronize()
        nv.grouped_gemm(z, w, off, out=u); torch.cuda.synchronize()
        want = [y, z, u, *nv.quantize_int8(y)]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_both_bindings_make_the_same_calls(monkeypatch):
    """The native marshalling of the common calls and the Python one behind it: the same outputs, types and strides,
    and what one does not take the other does or refuses."""
    P = nv.products
    run, (x, dy, w) = _all_calls(rows=210, n=77, k=134, seed=183)
    run()
    assert P._native is not None, "_marshal.so is not built"
    native = run()
    q, s = native[:2]
    off = offsets_of((0, 1, 170, 39))
    taken = P._native.product(0, x, w, off, None, None, None)
    assert taken.dtype == BF16 and tuple(taken.shape) == (210, 77) and taken.stride(0) == 80
    assert P._native.product(0, x, w, None, None, None, None) is None          # four matrices, no offsets
    assert P._native.product(0, x, w, off.long(), None, None, None) is None
    assert P._native.product(0, x.t(), w, off, None, None, None) is None
    assert P._native.product(0, x, w, off, s, s, None) is None                 # scales without codes
    assert P._native.product(0, q, w, off, None, None, None) is None           # two types
    assert P._native.product(0, x.cpu(), w, off, None, None, None) is None
    assert P._native.product(1, q, q, None, None, None, None) is None
    assert P._native.product(3, x, w, off, None, None, None) is None
    assert P._native.product(0, "x", w, off, None, None, None) is None
    assert P._native.product(0, x, w, off, None, None, torch.int8) is None
    assert P._native.quantize(q, False) is None and P._native.quantize(x[:, :7], True) is None
    with pytest.raises(nv.NVFP4MoEError):       # rows that do not start every 16 bytes: the library's own refusal
        nv.grouped_gemm(x[:, 1:], w[:, :, 1:], off)
    monkeypatch.setattr(P, "_native", None)
    monkeypatch.setattr(P, "_marshal", None)
    for a, b in zip(native, run()):
        assert torch.equal(a, b) and a.dtype == b.dtype and a.stride() == b.stride()
    with pytest.raises(nv.NVFP4MoEError):
        nv.grouped_gemm(x[:, 1:], w[:, :, 1:], off)


@pytest.mark.parametrize("call,counts,n,k", [
    ("fwd", (200, 300), 200, 264), ("dx", (16384,), 512, 512), ("dw", (1001,) * 8, 1024, 1024), ("dw", (9000,), 96, 136),
], ids=["one CTA", "a pair", "a pair with rows to zero", "a split sum"])
def test_a_wait_that_runs_out_is_reported(call, counts, n, k):
    """The first CTA's copies are left out by the test hook: the bounded waits end (about 2 s), the status says so once,
    and the next call is whole again."""
    off, rows, E = offsets_of(counts), sum(counts), len(counts)
    x, dy, w = normal((rows, k), BF16, 221), normal((rows, n), BF16, 222), normal((E, n, k), BF16, 223, 0.1)
    run = {"fwd": lambda: nv.grouped_gemm(x, w, off), "dx": lambda: nv.grouped_gemm_dx(dy, w, off),
           "dw": lambda: nv.grouped_gemm_dw(dy, x, off)}[call]
    want = run()
    assert nv.products_status() == 0
    nv.nvfp4_moe_test_products_stall(1)
    run()
    assert nv.products_status() == -8
    assert nv.products_status() == 0
    assert torch.equal(run(), want)
    assert nv.products_status() == 0


@pytest.mark.parametrize("rows,n,k", [(6000, 1536, 512), (300, 256, 4104), (257, 200, 264)], ids=["many tiles", "a split sum", "few tiles"])
@pytest.mark.parametrize("call", ["fwd", "dx", "dw"])
def test_a_wait_that_runs_out_leaves_the_next_call_alone(call, rows, n, k):
    """A dense call enqueued right behind a stalled one starts before that has ended, on the SMs that it leaves free; its
    own bounded waits must not run meanwhile."""
    x, dy, w = normal((rows, k), BF16, 231), normal((rows, n), BF16, 232), normal((n, k), BF16, 233, 0.1)
    run = {"fwd": lambda: nv.grouped_gemm(x, w), "dx": lambda: nv.grouped_gemm_dx(dy, w), "dw": lambda: nv.grouped_gemm_dw(dy, x)}[call]
    few, one = normal((500, 264), BF16, 234), normal((2, 200, 264), BF16, 235)
    off = offsets_of((200, 300))
    want = run()
    nv.grouped_gemm(few, one, off)
    assert nv.products_status() == 0
    nv.nvfp4_moe_test_products_stall(1)
    nv.grouped_gemm(few, one, off)
    got = run()
    assert nv.products_status() == -8
    assert torch.equal(got, want)
    assert nv.products_status() == 0


def test_calls_from_several_threads():
    import threading
    run, _ = _all_calls(rows=200, n=264, k=328, seed=181)
    want = run()
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(5):
                got[i] = run(stream=s)
            s.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_calls_from_several_threads_on_their_current_streams():
    """The native calls, which drop the interpreter lock: each thread with a current stream of its own."""
    import threading
    run, _ = _all_calls(rows=200, n=264, k=328, seed=191)
    want = run()
    torch.cuda.synchronize()
    assert nv.products._native is not None
    got, errors = [[] for _ in range(4)], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i].append(run())
            s.synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for g in got:
        assert len(g) == 20
        for outs in g:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_outputs_are_detached_and_empty_offsets_refused():
    x, w = normal((30, 64), BF16, 281), torch.nn.Parameter(normal((2, 40, 64), BF16, 282))
    off = offsets_of((10, 20))
    y = nv.grouped_gemm(x, w, off)
    assert not y.requires_grad
    assert torch.equal(y, nv.grouped_gemm(x, w.detach(), off))
    for n in (0, 1):
        with pytest.raises(ValueError, match="offsets"):
            nv.grouped_gemm_dw(y, x, torch.zeros(n, dtype=torch.int32, device=DEV))


# --------------------------------------------------- together, as they are used

def test_shared_expert_in_8_bits_beside_the_routed_layer():
    """A prompt chunk and a few decode tokens: the chunk's activations are quantised on the GPU and routed through
    the NVFP4 layer; a shared expert in 8 bits (gate and up in one product, SwiGLU with its quantiser, down) adds to
    the same output. The reference: the FP64 oracle for the layer, 64-bit products of the GPU's own codes for the
    shared expert, whose codes the quantiser's tests pin."""
    import numpy as np
    import oracle
    import synth
    dims = synth.LayerDims(E=16, H=256, I=128, K=4)
    layer = synth.make_layer(dims, seed=5)
    wide = normal((2 * 96, dims.H), F32, 121, 0.05)
    down = normal((dims.H, 96), F32, 122, 0.05)
    wq, ws = nv.quantize_int8(wide)
    dq, ds = nv.quantize_int8(down)
    for T in (5, 90):
        x = synth.make_x_bf16(T, dims.H, 6)
        logits = synth.make_logits(T, dims.E, 6)
        q, s = nv.quantize_int8(x.to(DEV))
        m = nv.MoELayer.from_layer(layer.to(DEV), top_k=dims.K, max_tokens=T)
        out = m.forward(q, x_scale=s, logits=logits.to(DEV))
        routed = out.clone()
        h = nv.gemm_int8(q, wq, s, ws)
        hq, hs = nv.quantize_int8(h, swiglu=True)
        nv.gemm_int8(hq, dq, hs, ds, out=out, accumulate=True)
        assert m.status() == 0
        m.close()
        ref = oracle.forward(layer, q.cpu(), K=dims.K, logits=logits, x_scale=s.cpu())["out"]
        from helpers import assert_close
        assert_close(routed.double().cpu().numpy(), ref, "routed")
        hr = (q.double() @ wq.double().T) * s[:, None].double() * ws.double()
        g, u = hr.split(96, 1)
        v = g * torch.sigmoid(g) * u
        assert ((hq.double() * hs[:, None].double() - v).abs() <= hs[:, None].double() * (0.5 + 2.0 ** -9)).all()
        shared = (hq.double() @ dq.double().T) * hs[:, None].double() * ds.double()
        total = shared + routed.double()
        assert_within(out, total, 4 * 2.0 ** -24 * shared.abs() + 2.0 ** -23 * total.abs(), "routed + shared")
        assert np.isfinite(ref).all()


def test_bf16_experts_on_the_layers_own_routing_with_a_training_step():
    """Rows sorted by the permutation and the offsets that the layer's routing gives, through experts in BF16 (gate | up,
    SwiGLU, down), and back: gradients against 64-bit autograd on the same BF16 intermediates."""
    import synth
    dims, T = synth.LayerDims(E=16, H=256, I=128, K=4), 120
    layer = synth.make_layer(dims, seed=7)
    x, logits = synth.make_x_bf16(T, dims.H, 8).to(DEV), synth.make_logits(T, dims.E, 8).to(DEV)
    m = nv.MoELayer.from_layer(layer.to(DEV), top_k=dims.K, max_tokens=T)
    dbg = nv.debug_buffers(T, dims.E, dims.K, torch.device(DEV))
    m.forward(x, logits=logits, debug=dbg)
    assert m.status() == 0
    m.close()
    off, token = dbg["offsets"], dbg["perm"].long() // dims.K
    xs = x[token].contiguous()
    w1, w2 = normal((dims.E, 2 * dims.I, dims.H), BF16, 131, 0.05), normal((dims.E, dims.H, dims.I), BF16, 132, 0.05)
    gu = nv.grouped_gemm(xs, w1, off)
    h = (torch.nn.functional.silu(gu[:, :dims.I].float()) * gu[:, dims.I:].float()).to(BF16)
    y = nv.grouped_gemm(h, w2, off, out_dtype=F32)
    dy = normal((T * dims.K, dims.H), BF16, 133, 0.1)
    dh, dw2 = nv.grouped_gemm_dx(dy, w2, off), nv.grouped_gemm_dw(dy, h, off)
    pos = off.tolist()
    for e in range(dims.E):
        r = slice(pos[e], pos[e + 1])
        hd, wd, dd = h[r].double().requires_grad_(), w2[e].double().requires_grad_(), dy[r].double()
        yd = hd @ wd.T
        yd.backward(dd)
        s = h[r].double().abs() @ w2[e].double().abs().T
        assert_within(y[r], yd.detach(), tol16(dims.I, s, yd.detach(), F32), "y")
        s = dd.abs() @ w2[e].double().abs()
        assert_within(dh[r], hd.grad, tol16(dims.H, s, hd.grad, BF16), "dh")
        s = dd.abs().T @ h[r].double().abs()
        assert_within(dw2[e], wd.grad, tol16(max(1, pos[e + 1] - pos[e]), s, wd.grad, F32), "dw2")
