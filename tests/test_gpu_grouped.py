"""The grouped products by expert, their gradients, the block quantiser and the fp8 block products on the GPU,
against plain references in 64 bits.

Bounds.  A sum of n products held in fp32 is off by at most n * 2^-23 * S from the exact one, S the sum of the
products' magnitudes: each of at most n additions, in whatever order, is off by one unit 2^-23 (twice what
rounding to nearest allows) of a partial sum that S bounds.  The fp8 products add one scaling (two roundings)
and one addition per block of 128.  Storing the result adds eps / 2 of its type.  Integer-valued inputs whose
sums stay below 2^24 must come out exactly in fp32.
"""
import numpy as np
import pytest
import torch

import quantized_moe_expert_topk_amd as qm

pytestmark = pytest.mark.gpu

DEV = "cuda"
FP8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(torch.bfloat16)


def ints(g, *shape, most=3):
    return torch.randint(-most, most + 1, shape, device=DEV, generator=g).to(torch.bfloat16)


def ranges(counts, gap=0, step=1, lead=0):
    """Starts [E + 1] of runs with these counts, each start on a multiple of step plus lead, gap rows between."""
    off, at = [], lead
    for c in counts:
        off.append(at)
        at = -(-(at + c + gap) // step) * step
    off.append(at)
    return torch.tensor(off, dtype=torch.int32, device=DEV), torch.tensor(counts, dtype=torch.int32, device=DEV), at


def rows_of(off, cnt):
    o, c = off.tolist(), cnt.tolist()
    return [slice(o[e], o[e] + c[e]) for e in range(len(c))]


def fill_outside(x, off, cnt, value):
    """Rows of nobody hold `value`."""
    keep = torch.zeros(x.shape[0], dtype=torch.bool, device=DEV)
    for r in rows_of(off, cnt):
        keep[r] = True
    x[~keep] = value
    return ~keep


def check(name, got, ref, S, terms):
    half = torch.finfo(got.dtype).eps / 2
    sums = terms * 2.0 ** -23 * S
    bound = sums + half * (ref.abs() + sums) + 1e-38
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), name
    worst = float((err / bound).max()) if err.numel() else 0.0
    print(f"[grouped] {name}: worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, name


COUNTS = {
    "one": [1],
    "tiny": [3, 0, 1, 2],
    "empty": [0, 0, 0, 0, 0],
    "ragged": [37, 0, 128, 1, 129, 64, 0, 250],
    "edges": [31, 32, 33, 63, 64, 65, 127, 128, 129],
    "long": [700, 0, 513],
    "many": [((7 * i) % 5) for i in range(130)],
    "wide": [300, 257, 255, 256],
    "huge": [1300, 0, 900],
    # enough experts for each tile that the launchers pick by the mean number of rows
    "mean 12": [((5 * i) % 25) for i in range(130)],
    "mean 24": [((7 * i) % 49) for i in range(130)],
    "mean 48": [((11 * i) % 97) for i in range(130)],
    "mean 80": [((13 * i) % 161) for i in range(130)],
    "forty": [((13 * i) % 151) for i in range(40)],  # fewer tiles than CUs, but not few
}
SIZES = [(8, 8), (64, 64), (136, 72), (264, 200), (256, 512), (520, 1032),
         (1024, 512)]  # (N, K); the last: rows of whole lines, of outputs too large for L2


@pytest.mark.parametrize("NK", SIZES, ids=str)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_forward_and_gradients(counts, NK):
    """All three products on integer-valued inputs (exact in fp32) and on normal ones (bound)."""
    N, K = NK
    if counts.startswith("mean") and NK not in ((264, 200), (520, 1032), (1024, 512)):
        pytest.skip("many experts at three sizes are enough")
    off, cnt, M = ranges(COUNTS[counts])
    E = len(COUNTS[counts])
    g = gen(len(counts) * 1000 + N + K)
    for kind in ("ints", "normal"):
        make = ints if kind == "ints" else bf16
        x, w, dy = make(g, M, K), make(g, E, N, K), make(g, M, N)
        for dt in (torch.float32, torch.bfloat16):
            print(f"[grouped] {counts} N={N} K={K} {kind} {dt}", flush=True)
            y = qm.moe_grouped_mm(x, w, off, out_dtype=dt)
            dx = qm.moe_grouped_mm_dgrad(dy, w, off, out_dtype=dt)
            dw = qm.moe_grouped_mm_wgrad(dy, x, off, out_dtype=dt)
            torch.cuda.synchronize()
            assert y.shape == (M, N) and dx.shape == (M, K) and dw.shape == (E, N, K) and y.dtype == dt
            for e, r in enumerate(rows_of(off, cnt)):
                X, W, D = x[r].double(), w[e].double(), dy[r].double()
                for name, got, a, b in (("y", y[r], X, W.t()), ("dx", dx[r], D, W), ("dw", dw[e], D.t(), X)):
                    ref = a @ b
                    if kind == "ints" and dt == torch.float32:
                        assert torch.equal(got.double(), ref), (name, e)
                    else:
                        n = max(1, a.shape[1])
                        bound = n * 2.0 ** -23 * (a.abs() @ b.abs())
                        bound = bound + torch.finfo(dt).eps / 2 * (ref.abs() + bound) + 1e-38
                        assert bool(((got.double() - ref).abs() <= bound).all()), (name, e)


@pytest.mark.parametrize("step,gap,lead", [(16, 0, 0), (128, 0, 0), (1, 3, 5), (1, 300, 129)])
def test_rows_of_nobody(step, gap, lead):
    """NaN in rows of nobody reaches no output, and their output rows, and the memory around, stay as they were."""
    counts = [5, 0, 130, 16, 1, 0, 70]
    off, cnt, M = ranges(counts, gap, step, lead)
    N, K, E, g = 72, 136, len(counts), gen(3)
    x, w, dy = ints(g, M, K), ints(g, E, N, K), ints(g, M, N)
    fill_outside(dy, off, cnt, float("nan"))
    idle = fill_outside(x, off, cnt, float("nan"))
    ybuf = torch.full((M + 8, N), 7.0, device=DEV)
    xbuf = torch.full((M + 8, K), 7.0, device=DEV)
    wbuf = torch.full((E + 2, N, K), 7.0, device=DEV)
    qm.moe_grouped_mm(x, w, off, cnt, sum(counts), out=ybuf[4:M + 4])
    qm.moe_grouped_mm_dgrad(dy, w, off, cnt, sum(counts), out=xbuf[4:M + 4])
    qm.moe_grouped_mm_wgrad(dy, x, off, cnt, sum(counts), out=wbuf[1:E + 1])
    torch.cuda.synchronize()
    for buf in (ybuf, xbuf):
        assert bool((buf[:4] == 7).all()) and bool((buf[M + 4:] == 7).all())
        assert bool((buf[4:M + 4][idle] == 7).all())
    assert bool((wbuf[0] == 7).all()) and bool((wbuf[-1] == 7).all())
    for e, r in enumerate(rows_of(off, cnt)):
        X, W, D = x[r].double(), w[e].double(), dy[r].double()
        assert torch.equal(ybuf[4:M + 4][r].double(), X @ W.t())
        assert torch.equal(xbuf[4:M + 4][r].double(), D @ W)
        assert torch.equal(wbuf[1 + e].double(), D.t() @ X)


# --------------------------------------------------------------------------------------- fp8


def fp8_rows(g, M, K, kind="normal"):
    """e4m3 codes and block-major scales: from the quantiser's formula, or integers with powers of two."""
    KB = -(-K // 128)
    if kind == "ints":
        q = torch.randint(-4, 5, (M, K), device=DEV, generator=g).float().to(FP8)
        return q, torch.randint(0, 3, (KB, M), device=DEV, generator=g).float().exp2()
    q = (torch.randn(M, K, device=DEV, generator=g) * 100).clamp(-448, 448).to(FP8)
    return q, torch.rand(KB, M, device=DEV, generator=g) * 0.01 + 1e-3


def fp8_weights(g, E, N, K, kind="normal"):
    NB, KB = -(-N // 128), -(-K // 128)
    if kind == "ints":
        q = torch.randint(-4, 5, (E, N, K), device=DEV, generator=g).float().to(FP8)
        return q, torch.randint(0, 3, (E, NB, KB), device=DEV, generator=g).float().exp2()
    q = (torch.randn(E, N, K, device=DEV, generator=g) * 100).clamp(-448, 448).to(FP8)
    return q, torch.rand(E, NB, KB, device=DEV, generator=g) * 1e-3 + 1e-4


def tile16(q):
    E, N, K = q.shape
    b = q.view(torch.uint8).view(E, N // 16, 16, K // 16, 16).permute(0, 1, 3, 2, 4)
    return b.contiguous().view(E, N, K).view(FP8)


def dequant_rows(q, s):
    M, K = q.shape
    return q.float().double() * s.t().double().repeat_interleave(128, 1)[:, :K]


def dequant_weights(q, s):
    N, K = q.shape
    return q.float().double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def check_fp8(name, got, X, W, kind):
    """fp32 outputs: the sums' bound, exact for the integer inputs.  bf16 outputs may come from the fp8 matrix
    cores, which add the products of 8 consecutive k with what lies below 2^-13 of the largest cut off: each of
    the other 7 loses less than 2^-13 of the largest, so a group loses less than 7 * 2^-13 times its largest
    product (the groups' sum is bounded here with the largest of each row's and column's 8 values)."""
    ref = X @ W.t()
    if kind == "ints" and got.dtype == torch.float32:
        assert torch.equal(got.double(), ref), name
        return
    K = X.shape[1]
    sums = (K + K // 128 + 3) * 2.0 ** -23 * (X.abs() @ W.abs().t())
    if got.dtype == torch.bfloat16:
        largest = X.abs().unfold(1, 8, 8).amax(2) @ W.abs().unfold(1, 8, 8).amax(2).t()
        sums = sums + 7 * 2.0 ** -13 * largest
    bound = sums + torch.finfo(got.dtype).eps / 2 * (ref.abs() + sums) + 1e-38
    assert bool(((got.double() - ref).abs() <= bound).all()), name


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 1024, 2048), (3, 1, 128), (17, 130, 144), (33, 257, 400), (64, 64, 64),
                                   (100, 384, 1040), (129, 515, 256), (256, 256, 512), (300, 1000, 272),
                                   (513, 128, 8208), (1000, 2050, 272), (2000, 2064, 144), (2100, 4096, 272)])
def test_block_mm(M, N, K):
    g = gen(M + N + K)
    for kind in ("ints", "normal"):
        xq, xs = fp8_rows(g, M, K, kind)
        wq, ws = fp8_weights(g, 1, N, K, kind)
        X, W = dequant_rows(xq, xs), dequant_weights(wq[0], ws[0])
        for dt in (torch.float32, torch.bfloat16):
            for layout in (qm.MOE_LAYOUT_ROWS, qm.MOE_LAYOUT_TILE16):
                if layout == qm.MOE_LAYOUT_TILE16 and N % 16:
                    continue
                print(f"[block_mm] {M} {N} {K} {kind} {dt} layout {layout}", flush=True)
                w = (tile16(wq) if layout == qm.MOE_LAYOUT_TILE16 else wq)[0]
                y = qm.moe_block_mm(xq, xs, w, ws[0], layout, out_dtype=dt)
                torch.cuda.synchronize()
                check_fp8(f"{kind} {dt} {layout}", y, X, W, kind)


@pytest.mark.parametrize("N,K", [(16, 16), (144, 272), (1, 128), (131, 144), (256, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_grouped_block_mm(counts, N, K):
    for step in (1, 16):
        off, cnt, M = ranges(COUNTS[counts], 0, step)
        E, g = len(COUNTS[counts]), gen(N + K + M)
        for kind in ("ints", "normal"):
            xq, xs = fp8_rows(g, M, K, kind)
            wq, ws = fp8_weights(g, E, N, K, kind)
            for layout in (qm.MOE_LAYOUT_ROWS, qm.MOE_LAYOUT_TILE16):
                if layout == qm.MOE_LAYOUT_TILE16 and N % 16:
                    continue
                print(f"[grouped_block_mm] {counts} {N} {K} step {step} {kind} layout {layout}", flush=True)
                w = tile16(wq) if layout == qm.MOE_LAYOUT_TILE16 else wq
                out = torch.full((M + 2, N), 7.0, device=DEV)
                qm.moe_grouped_block_mm(xq, xs, w, ws, off, cnt, sum(COUNTS[counts]), layout, out=out[:M])
                torch.cuda.synchronize()
                idle = torch.ones(M + 2, dtype=torch.bool, device=DEV)
                for e, r in enumerate(rows_of(off, cnt)):
                    idle[r] = False
                    check_fp8(f"{kind} {layout} {e}", out[:M][r], dequant_rows(xq[r], xs[:, r]), dequant_weights(wq[e], ws[e]), kind)
                assert bool((out[idle] == 7).all())


@pytest.mark.parametrize("N,K", [(131, 144), (144, 272), (1024, 272), (1040, 128)])
@pytest.mark.parametrize("counts", ["ragged", "wide", "mean 24", "mean 48", "mean 80", "forty"])
def test_grouped_block_mm_bf16(counts, N, K):
    off, cnt, M = ranges(COUNTS[counts])
    E, g = len(COUNTS[counts]), gen(N + K + M)
    for kind in ("ints", "normal"):
        xq, xs = fp8_rows(g, M, K, kind)
        wq, ws = fp8_weights(g, E, N, K, kind)
        print(f"[grouped_block_mm] {counts} {N} {K} {kind} bf16", flush=True)
        y = qm.moe_grouped_block_mm(xq, xs, wq, ws, off, out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        for e, r in enumerate(rows_of(off, cnt)):
            check_fp8(f"{kind} {e}", y[r], dequant_rows(xq[r], xs[:, r]), dequant_weights(wq[e], ws[e]), kind)


# --------------------------------------------------------------------------------------- quantiser


def quantize_ref(x):
    """Codes' values and scales by the definition: fp32 quotients (64-bit division rounded once), e4m3 by grid."""
    M, K = x.shape
    KB = -(-K // 128)
    z = torch.zeros(M, KB * 128, dtype=torch.float64, device=DEV)
    z[:, :K] = x.double()
    z = z.view(M, KB, 128)
    s = (z.abs().amax(2) / 448).float()
    v = (z / torch.where(s == 0, torch.ones_like(s), s).double()[:, :, None]).float().double()
    m, e = torch.frexp(v.abs())
    step = ((e.long() - 1).clamp_min(-6) - 3 + 1023 << 52).view(torch.float64)  # a power of two, made of its bits
    return (torch.round(v / step) * step).view(M, KB * 128)[:, :K], s.t()


@pytest.mark.parametrize("M,K", [(1, 16), (1, 2048), (31, 128), (33, 400), (64, 4096), (1000, 1040), (5, 8208)])
def test_quantize_blocks(M, K):
    g = gen(M + K)
    x = bf16(g, M, K)
    x[:, ::7] *= 20
    x[M // 2, :128] = 0
    x[0, K // 2:] *= 2.0 ** -120  # tiny blocks: subnormal scales
    x[-1, :16] *= 2.0 ** 100
    q, s = qm.moe_quantize_blocks(x)
    torch.cuda.synchronize()
    v, rs = quantize_ref(x)
    assert torch.equal(s, rs)
    assert torch.equal(q.float().double(), v)


def test_quantize_blocks_all_values():
    """Every finite bf16 magnitude against a range of block maxima: each rounding and tie of the format."""
    bits = torch.arange(0x0000, 0x7F80, dtype=torch.int32, device=DEV)
    for top in (448.0, 3.0, 1.0, 1.75, 251.0, 2.0 ** -110, 1e30):
        v = (bits << 16).view(torch.float32)
        v = v[v <= top]
        v = v[-127 * 64:]  # the values within reach of the maximum
        v = v[: len(v) // 127 * 127].view(-1, 127)
        t = torch.tensor(top, device=DEV).to(torch.bfloat16).float()
        x = torch.cat([t.expand(len(v), 1), v.minimum(t)], 1).to(torch.bfloat16)
        x[:, 1::2] *= -1
        q, s = qm.moe_quantize_blocks(x)
        torch.cuda.synchronize()
        rv, rs = quantize_ref(x)
        assert torch.equal(s, rs) and torch.equal(q.float().double(), rv), top


def test_quantize_blocks_not_finite():
    x = bf16(gen(0), 4, 256)
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    q, s = qm.moe_quantize_blocks(x)
    torch.cuda.synchronize()
    assert torch.isnan(s[0, 1]) and bool(torch.isnan(q[1, :128].float()).all())
    assert torch.isinf(s[1, 2]) and torch.isnan(q[2, 200].float()) and int((q[2, 128:].float() == 0).sum()) == 127
    v, rs = quantize_ref(x[[0, 3]])
    assert torch.equal(q[[0, 3]].float().double(), v)


# --------------------------------------------------------------------------------------- how the calls are made


def ragged(seed=0, N=264, K=392, counts=(70, 0, 1, 33, 200, 16)):
    off, cnt, M = ranges(list(counts))
    g = gen(seed)
    return dict(off=off, cnt=cnt, M=M, E=len(counts), N=N, K=K, x=ints(g, M, K), w=ints(g, len(counts), N, K),
                dy=ints(g, M, N))


def every_product(c, y, dx, dw, stream=None):
    qm.moe_grouped_mm(c["x"], c["w"], c["off"], c["cnt"], c["M"], out=y, stream=stream)
    qm.moe_grouped_mm_dgrad(c["dy"], c["w"], c["off"], c["cnt"], c["M"], out=dx, stream=stream)
    qm.moe_grouped_mm_wgrad(c["dy"], c["x"], c["off"], c["cnt"], c["M"], out=dw, stream=stream)


def outputs(c):
    f32 = dict(dtype=torch.float32, device=DEV)
    return (torch.zeros(c["M"], c["N"], **f32), torch.zeros(c["M"], c["K"], **f32),
            torch.zeros(c["E"], c["N"], c["K"], **f32))


def check_every(c, y, dx, dw):
    for e, r in enumerate(rows_of(c["off"], c["cnt"])):
        X, W, D = c["x"][r].double(), c["w"][e].double(), c["dy"][r].double()
        assert torch.equal(y[r].double(), X @ W.t()) and torch.equal(dx[r].double(), D @ W)
        assert torch.equal(dw[e].double(), D.t() @ X)


def test_gradients_against_differences():
    """y is linear in x and in w: for integers L(x + d) - L(x) with L = sum(y * dy) is sum(dx * d) exactly."""
    c = ragged(1)
    y, dx, dw = outputs(c)
    every_product(c, y, dx, dw)
    g = gen(2)
    d, dW = ints(g, c["M"], c["K"], most=1), ints(g, c["E"], c["N"], c["K"], most=1)
    lin = (qm.moe_grouped_mm(c["x"] + d, c["w"], c["off"], out_dtype=torch.float32).double() - y.double())
    assert float((lin * c["dy"].double()).sum()) == float((dx.double() * d.double()).sum())
    lin = (qm.moe_grouped_mm(c["x"], c["w"] + dW, c["off"], out_dtype=torch.float32).double() - y.double())
    assert float((lin * c["dy"].double()).sum()) == float((dw.double() * dW.double()).sum())


@pytest.mark.parametrize("E,N,K", [(6, 264, 392), (40, 264, 392), (130, 520, 1032), (130, 256, 1024)])
def test_wgrad_accumulates(E, N, K):
    c = ragged(3, N, K, [(17 * i) % 40 for i in range(E)])
    base = ints(gen(4), E, N, K).float()
    dw = base.clone()
    for n in (1, 2):
        qm.moe_grouped_mm_wgrad(c["dy"], c["x"], c["off"], out=dw, accumulate=True)
    for e, r in enumerate(rows_of(c["off"], c["cnt"])):
        assert torch.equal(dw[e].double(), base[e].double() + 2 * (c["dy"][r].double().t() @ c["x"][r].double()))


def test_no_rows_at_all():
    w = ints(gen(5), 3, 16, 24)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x, dy = torch.empty(0, 24, dtype=torch.bfloat16, device=DEV), torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    assert qm.moe_grouped_mm(x, w, off).shape == (0, 16) and qm.moe_grouped_mm_dgrad(dy, w, off).shape == (0, 24)
    dw = torch.full((3, 16, 24), 7.0, device=DEV)
    qm.moe_grouped_mm_wgrad(dy, x, off, out=dw, accumulate=True)
    assert bool((dw == 7).all())
    qm.moe_grouped_mm_wgrad(dy, x, off, out=dw)
    assert bool((dw == 0).all())
    q, s = qm.moe_quantize_blocks(torch.empty(0, 32, dtype=torch.bfloat16, device=DEV))
    assert q.shape == (0, 32) and s.shape == (1, 0)


def test_not_finite_stays_in_its_row_and_expert():
    c = ragged(6)
    y, dx, dw = outputs(c)
    bad = 70 + 1 + 5  # a row of expert 3
    c["x"][bad, 9] = float("nan")
    c["dy"][bad, 3] = float("inf")
    every_product(c, y, dx, dw)
    assert bool(torch.isnan(y[bad]).all())
    keep = torch.ones(c["M"], dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert bool(torch.isfinite(y[keep]).all()) and bool(torch.isfinite(dx[keep]).all())
    assert not bool(torch.isfinite(dx[bad]).all())
    for e in range(c["E"]):
        assert bool(torch.isfinite(dw[e]).all()) == (e != 3)


def test_bad_ranges_stay_inside():
    """Device values that name rows outside the matrices are cut to them: what is asked for inside is right, and
    no byte around the outputs changes."""
    N, K, M, E = 136, 72, 100, 6
    g = gen(7)
    x, w, dy = ints(g, M, K), ints(g, E, N, K), ints(g, M, N)
    off = torch.tensor([-50, 20, 90, 5000, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    cnt = torch.tensor([20, 30, 2 ** 31 - 1, 9, 5, -3], dtype=torch.int32, device=DEV)
    inside = [slice(0, 20), slice(20, 50), slice(90, 100), slice(0, 0), slice(0, 0), slice(0, 0)]
    ybuf, xbuf = torch.full((M + 600, N), 7.0, device=DEV), torch.full((M + 600, K), 7.0, device=DEV)
    y, dx = ybuf[300:300 + M], xbuf[300:300 + M]
    dw = torch.full((E, N, K), 7.0, device=DEV)
    qm.moe_grouped_mm(x, w, off, cnt, 60, out=y)
    qm.moe_grouped_mm_dgrad(dy, w, off, cnt, 60, out=dx)
    qm.moe_grouped_mm_wgrad(dy, x, off, cnt, 60, out=dw)
    xq, xs = fp8_rows(g, M, 80, "ints")
    wq, ws = fp8_weights(g, E, N, 80, "ints")
    fbuf = torch.full((M + 600, N), 7.0, device=DEV)
    qm.moe_grouped_block_mm(xq, xs, wq, ws, off, cnt, 60, out=fbuf[300:300 + M])
    torch.cuda.synchronize()
    for buf in (ybuf, xbuf, fbuf):
        assert bool((buf[:300] == 7).all()) and bool((buf[300 + M:] == 7).all()) and bool((buf[350:390] == 7).all())
    for e, r in enumerate(inside):
        X, W, D = x[r].double(), w[e].double(), dy[r].double()
        assert torch.equal(y[r].double(), X @ W.t()) and torch.equal(dx[r].double(), D @ W)
        assert torch.equal(dw[e].double(), D.t() @ X)
        check_fp8("bad ranges", fbuf[300:300 + M][r], dequant_rows(xq[r], xs[:, r]), dequant_weights(wq[e], ws[e]), "ints")


@pytest.mark.parametrize("E,M", [(1024, 5000), (7, 300)])
def test_overlapping_ranges_end(E, M):
    """Every expert claims every row: the outputs are undefined, but the calls end, write rows of the matrix only,
    and a call with proper ranges after them is right."""
    N, K = 72, 80
    g = gen(9)
    x, w = ints(g, M, K), ints(g, E, N, K)
    xq, xs = fp8_rows(g, M, K, "ints")
    wq, ws = fp8_weights(g, E, N, K, "ints")
    off = torch.zeros(E, dtype=torch.int32, device=DEV)
    cnt = torch.full((E,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    for hint in (1, M):  # the kernel for few rows and a tiled one
        buf = torch.full((M + 600, N), 7.0, device=DEV)
        qm.moe_grouped_mm(x, w, off, cnt, hint, out=buf[300:300 + M])
        qm.moe_grouped_block_mm(xq, xs, wq, ws, off, cnt, hint, out=buf[300:300 + M])
        torch.cuda.synchronize()
        assert bool((buf[:300] == 7).all()) and bool((buf[300 + M:] == 7).all())
    cnt.zero_()
    cnt[E - 1] = M
    y = qm.moe_grouped_mm(x, w, off, cnt, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w[E - 1].double().t())


def test_matrices_past_4_gib():
    """Weights, gradients and rows whose byte offsets need more than 32 bits."""
    E, N, K = 260, 4104, 2056  # 4.4 GB of bf16 weights, 8.8 GB of fp32 gradient
    cnt = [0] * E
    cnt[0], cnt[E - 1] = 3, 5
    off, counts, M = ranges(cnt)
    g = gen(8)
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    w[0], w[E - 1] = ints(g, N, K), ints(g, N, K)
    x, dy = ints(g, M, K), ints(g, M, N)
    y = qm.moe_grouped_mm(x, w, off, out_dtype=torch.float32)
    dx = qm.moe_grouped_mm_dgrad(dy, w, off, out_dtype=torch.float32)
    dw = qm.moe_grouped_mm_wgrad(dy, x, off, out_dtype=torch.float32)
    for e, r in ((0, slice(0, 3)), (E - 1, slice(3, 8))):
        X, W, D = x[r].double(), w[e].double(), dy[r].double()
        assert torch.equal(y[r].double(), X @ W.t()) and torch.equal(dx[r].double(), D @ W)
        assert torch.equal(dw[e].double(), D.t() @ X)
    assert not bool(dw[E // 2].any())
    del w, dw
    M, N, K = 1_100_000, 72, 2048  # 4.5 GB of rows
    lo = torch.tensor([5, M - 300], dtype=torch.int32, device=DEV)
    n = torch.tensor([2, 300], dtype=torch.int32, device=DEV)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[5:7], x[M - 300:] = ints(g, 2, K), ints(g, 300, K)
    w = ints(g, 2, N, K)
    y = torch.zeros(M, N, dtype=torch.float32, device=DEV)
    qm.moe_grouped_mm(x, w, lo, n, 302, out=y)
    assert torch.equal(y[5:7].double(), x[5:7].double() @ w[0].double().t())
    assert torch.equal(y[M - 300:].double(), x[M - 300:].double() @ w[1].double().t())
    assert not bool(y[7:M - 300].any())
    xq = torch.zeros(M * 2, 2048, dtype=FP8, device=DEV)
    xs = torch.ones(16, M * 2, device=DEV)
    xq[-40:], xs[:, -40:] = fp8_rows(g, 40, 2048, "ints")
    wq, ws = fp8_weights(g, 1, N, 2048, "ints")
    lo, n = torch.tensor([2 * M - 40], dtype=torch.int32, device=DEV), torch.tensor([40], dtype=torch.int32, device=DEV)
    y = torch.zeros(2 * M, N, dtype=torch.float32, device=DEV)
    qm.moe_grouped_block_mm(xq, xs, wq, ws, lo, n, 40, out=y)
    check_fp8("rows past 4 GiB", y[-40:], dequant_rows(xq[-40:], xs[:, -40:]), dequant_weights(wq[0], ws[0]), "ints")


def test_streams_and_repeats():
    """Calls on two streams at once, each result as alone; the same call twice gives the same bits."""
    cases = [ragged(10 + i, 520, 1032, [(17 * j + i) % 90 for j in range(60)]) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [outputs(c) for c in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, o, s in zip(cases, outs, streams):
            every_product(c, *o, stream=s)
    with torch.cuda.stream(streams[0]):  # the current stream of the device
        third = outputs(cases[0])
        every_product(cases[0], *third)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        check_every(c, *o)
    assert all(torch.equal(a, b) for a, b in zip(outs[0], third))
    g = gen(12)
    x, w = bf16(g, 900, 1032), bf16(g, 9, 520, 1032)
    off, _, _ = ranges([100] * 9)
    a, b = qm.moe_grouped_mm(x, w, off), qm.moe_grouped_mm(x, w, off)
    assert torch.equal(a, b)


def test_captured_and_replayed():
    """A graph of every call, replayed with new inputs and new row ranges, and eager calls between the replays."""
    c = ragged(20)
    y, dx, dw = outputs(c)
    xb = bf16(gen(21), c["M"], 400)
    wq, ws = fp8_weights(gen(22), c["E"], 144, 400)
    q, s = qm.moe_quantize_blocks(xb)
    z = torch.zeros(c["M"], 144, device=DEV)
    zd = torch.zeros(c["M"], 144, dtype=torch.bfloat16, device=DEV)

    def step():
        every_product(c, y, dx, dw)
        qm.moe_quantize_blocks(xb, q, s)
        qm.moe_grouped_block_mm(q, s, wq, ws, c["off"], c["cnt"], c["M"], out=z)
        qm.moe_block_mm(q, s, wq[0], ws[0], out=zd)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(4):
        counts = torch.tensor([[70, 0, 1, 33, 200, 16], [0, 0, 0, 320, 0, 0], [53] * 6, [1, 2, 3, 4, 5, 6]][n], dtype=torch.int32)
        c["cnt"].copy_(counts)
        c["off"][:6].copy_(torch.cumsum(counts, 0) - counts)
        for t in ("x", "dy"):
            c[t].copy_(ints(gen(30 + n), *c[t].shape))
        xb.copy_(bf16(gen(40 + n), *xb.shape))
        for t in (y, dx, dw, z):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw, q.view(torch.uint8), s, z, zd)]
        check_every(c, y, dx, dw)
        for t in (y, dx, dw, z):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw, q.view(torch.uint8), s, z, zd))), n


def test_expected_rows_changes_no_result():
    c = ragged(50)
    for hint in (0, 1, 100, 10 ** 9):
        y = torch.zeros(c["M"], c["N"], device=DEV)
        qm.moe_grouped_mm(c["x"], c["w"], c["off"], c["cnt"], hint, out=y)
        for e, r in enumerate(rows_of(c["off"], c["cnt"])):
            assert torch.equal(y[r].double(), c["x"][r].double() @ c["w"][e].double().t())


# --------------------------------------------------------------------------------------- together


def _layer(fmt, T=75):
    from oracle import oracle as O
    from synth import synth as S
    from tests.gpu_util import bf16_dev, device_bank, to_dev
    cfg = S.LayerConfig(90, "small layer", fmt, 256, 8, 2, 256, False, (T,), ((0, 256),))
    inp = S.layer_inputs(cfg, T)
    x = bf16_dev(inp.x)
    _, ids, wts, al = qm.moe_route_align(x, bf16_dev(inp.router), None, cfg.k, 16)
    pairs = torch.cat([torch.arange(T * cfg.k, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)])
    slots = al.sorted_ids.long().clamp(max=T * cfg.k)
    return O, cfg, inp, x, ids, wts, al, pairs[slots] // cfg.k, slots, device_bank, to_dev


def _combine(y, slots, wts, T, k):
    """Row sums of the pairs by their weights."""
    out = torch.zeros(T * k + 1, y.shape[1], dtype=torch.float64, device=DEV)
    out[slots] = y.double()
    return (out[:T * k].view(T, k, -1) * wts.double()[:, :, None]).sum(1)


def test_a_layer_of_bf16_products_and_its_backward():
    """gather, gate_up, SwiGLU, down and combine from the alignment's own arrays, against moe_expert_forward; then
    the layer's backward against torch's on the same formula in 64 bits."""
    O, cfg, inp, x, ids, wts, al, tok, slots, device_bank, to_dev = _layer("bf16")
    T, k, I, H = 75, cfg.k, cfg.I, cfg.H
    wg = to_dev(inp.routed.gate_up).view(torch.bfloat16)
    wd = to_dev(inp.routed.down).view(torch.bfloat16)
    rows = x[tok].contiguous()
    ranges_of = (al.offsets, al.counts, T * k)
    gu = qm.moe_grouped_mm(rows, wg, *ranges_of, out=torch.zeros(al.capacity, 2 * I, device=DEV))
    act = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).to(torch.bfloat16)
    y = qm.moe_grouped_mm(act, wd, *ranges_of, out=torch.zeros(al.capacity, H, device=DEV))
    got = _combine(y, slots, wts, T, k)
    want = qm.moe_expert_forward(device_bank(inp.routed), None, x, wts, al, 0, I)
    # the same sums of the same bf16 products in another order; act may round to its other neighbour
    assert float((got - want.double()).abs().max()) <= 1e-2 * float(want.abs().max())

    # backward of sum(out * G) for the rows of the pairs (G and the weights as bf16 gradients of y)
    G = torch.randn(T, H, device=DEV, generator=gen(1))
    pair_w = torch.cat([wts.reshape(-1), torch.zeros(1, device=DEV)])[slots]
    dy = (G[tok] * pair_w[:, None]).to(torch.bfloat16)
    da = qm.moe_grouped_mm_dgrad(dy, wd, *ranges_of, out=torch.zeros(al.capacity, I, device=DEV))
    dwd = qm.moe_grouped_mm_wgrad(dy, act, *ranges_of, out_dtype=torch.float32)
    sig = torch.sigmoid(gu[:, :I])
    dgu = torch.cat([da * gu[:, I:] * sig * (1 + gu[:, :I] * (1 - sig)), da * gu[:, :I] * sig], 1).to(torch.bfloat16)
    dx = qm.moe_grouped_mm_dgrad(dgu, wg, *ranges_of, out=torch.zeros(al.capacity, H, device=DEV))
    dwg = qm.moe_grouped_mm_wgrad(dgu, rows, *ranges_of, out_dtype=torch.float32)
    for e, r in enumerate(rows_of(al.offsets, al.counts)):
        X = rows[r].double().requires_grad_()
        Wg, Wd = wg[e].double().requires_grad_(), wd[e].double().requires_grad_()
        z = X @ Wg.t()
        a = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        (a @ Wd.t() * dy[r].double()).sum().backward()
        # act and dgu were rounded to bf16 (half a step 2^-9 of values that then spread over the sums) and gu's
        # sums are fp32: the norms agree to a few steps
        for a_, b_ in ((dwd[e], Wd.grad), (dwg[e], Wg.grad), (dx[r], X.grad)):
            assert float((a_.double() - b_).norm()) <= 2 ** -7 * float(b_.norm()) + 1e-30


def test_a_layer_of_fp8_products_on_a_packed_bank():
    """quantise, gate_up, SwiGLU, quantise, down on a TILE16 bank: each product against 64 bits on its own
    operands, the whole against moe_expert_forward within what e4m3 activations can do."""
    O, cfg, inp, x, ids, wts, al, tok, slots, device_bank, to_dev = _layer("fp8blk")
    T, k, I, H = 75, cfg.k, cfg.I, cfg.H
    bank = device_bank(inp.routed)
    rows = x[tok].contiguous()
    ranges_of = (al.offsets, al.counts, T * k)
    xq, xs = qm.moe_quantize_blocks(rows)
    gu = qm.moe_grouped_block_mm(xq, xs, bank.gate_up, bank.gate_up_scale, *ranges_of, layout=bank.layout,
                                 out=torch.zeros(al.capacity, 2 * I, device=DEV))
    act = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).to(torch.bfloat16)
    aq, as_ = qm.moe_quantize_blocks(act)
    y = qm.moe_grouped_block_mm(aq, as_, bank.down, bank.down_scale, *ranges_of, layout=bank.layout,
                                out=torch.zeros(al.capacity, H, device=DEV))
    for e, r in enumerate(rows_of(al.offsets, al.counts)):
        codes = to_dev(inp.routed.gate_up)[e].view(FP8), to_dev(inp.routed.down)[e].view(FP8)
        check_fp8("gate_up", gu[r], dequant_rows(xq[r], xs[:, r]), dequant_weights(codes[0], to_dev(inp.routed.gate_up_scale)[e]), "")
        check_fp8("down", y[r], dequant_rows(aq[r], as_[:, r]), dequant_weights(codes[1], to_dev(inp.routed.down_scale)[e]), "")
    got = _combine(y, slots, wts, T, k)
    want = qm.moe_expert_forward(bank, None, x, wts, al, 0, I).double()
    # each activation is off by at most 2^-4 of itself, evenly over +- that: 2^-4 / sqrt(3) = 3.6% in the norm for
    # each of the three rounded inputs (x in gate and in up, and the activation): under 3 * 3.6% + a margin
    assert float((got - want).norm() / want.norm()) <= 0.125
