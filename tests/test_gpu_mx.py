"""The MXFP4 quantiser and products on the GPU, against plain references in 64 bits.

Bounds: those of test_gpu_grouped's ``check``: a sum of n products held in fp32 is off by at most n 2^-23 S, S the sum of the
products' magnitudes, and storing it adds eps / 2 of its type.  Codes with equal scales have products that are multiples of
a quarter: their sums come out exactly in fp32.  The quantiser and its inverse are exact.
"""
import numpy as np
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import COUNTS, check, gen, ranges, rows_of
from tests.test_gpu_rows import routing, some_slots, there

pytestmark = pytest.mark.gpu

DEV = "cuda"
BOTH = (torch.bfloat16, torch.float32)
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
ROWS, TILE16 = qm.MOE_LAYOUT_ROWS, qm.MOE_LAYOUT_TILE16


# ------------------------------------------------------------------------------------------- references

def quantize_np(x):
    """Codes [M, K] and scale bytes [M, K / 32] of float64 rows."""
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    fine = np.isfinite(b).all(2)
    top = np.where(fine, np.abs(np.where(np.isfinite(b), b, 0)).max(2), 1.0)
    e = np.full(top.shape, -126)
    for p in range(-126, 127):
        e[top > 6 * 2.0 ** p] = p + 1
    q = np.abs(np.where(fine[:, :, None], b, 0)) / (2.0 ** e)[:, :, None]
    d = np.abs(q[..., None] - VALUES)
    order = [0, 2, 4, 6, 1, 3, 5, 7]  # of equal distances the even code
    code = np.array(order)[np.argmin(d[..., order], axis=-1)] + 8 * np.signbit(b)
    code = np.where(fine[:, :, None], code, 0)
    return code.reshape(M, K).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def pack(code):
    return code[:, 0::2] | code[:, 1::2] << 4


def group(byte):
    """Scale bytes [R, K / 32] in the quantiser's order [ceil(K / 128), R, 4]."""
    R, S = byte.shape
    p = byte.new_zeros(R, -(-S // 4) * 4)
    p[:, :S] = byte
    return p.view(R, p.shape[1] // 4, 4).permute(1, 0, 2).contiguous()


def ungroup(scale, K):
    return scale.permute(1, 0, 2).reshape(scale.shape[1], scale.shape[0] * 4)[:, :K // 32]


def decode(codes, byte):
    """Values in 64 bits of codes [R, K / 2] and scale bytes [R, K / 32]."""
    v = torch.tensor(np.concatenate([VALUES, -VALUES]), device=DEV)
    one = torch.stack([v[(codes & 15).long()], v[(codes >> 4).long()]], 2).view(*byte.shape, 32)
    unit = (byte.to(torch.int64) - 127 + 1023 << 52).view(torch.float64)  # made of its bits: torch's ldexp is not exact here
    return (one * torch.where(byte == 255, float("nan"), unit)[:, :, None]).view(codes.shape[0], codes.shape[1] * 2)


def operand(g, R, K, kind):
    """Random codes [R, K / 2] and scale bytes [R, K / 32]: one scale for all ("ints"), or of 15 binades."""
    q = torch.randint(0, 256, (R, K // 2), device=DEV, generator=g, dtype=torch.uint8)
    b = torch.randint(120, 135, (R, K // 32), device=DEV, generator=g, dtype=torch.uint8)
    return q, torch.full_like(b, 127) if kind == "ints" else b


def tile16(t, unit):
    E, N, P = t.shape
    return t.view(E, N // 16, 16, P // unit, unit).permute(0, 1, 3, 2, 4).contiguous().view(E, N, P)


def weights(g, E, N, K, kind, layout):
    """(codes, scales) as the calls take them, and the values [E, N, K]."""
    q, b = operand(g, E * N, K, kind)
    values = decode(q, b).view(E, N, K)
    if layout == TILE16:
        return tile16(q.view(E, N, -1), 16), tile16(b.view(E, N, -1), 1), values
    return q.view(E, N, -1), group(b), values


def check_product(name, got, x, w, kind):
    ref = x @ w.t()
    if kind == "ints" and got.dtype == torch.float32:
        assert torch.equal(got.double(), ref), name
    else:
        check(name, got, ref, x.abs() @ w.abs().t(), x.shape[1])


# ------------------------------------------------------------------------------------------- quantiser

def bf16_of(bits):
    return torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16).to(DEV)


def same_as_reference(x, slots=None):
    q, s = qm.moe_quantize_mx(x)
    code, byte = quantize_np(x.double().cpu().numpy())
    assert (s.cpu().numpy() == group(torch.from_numpy(byte)).numpy()).all()
    assert (q.cpu().numpy() == pack(code)).all()
    return q, s


def test_quantize_every_value_of_a_block():
    """Every bf16 number of at most 6, both signs, in blocks whose largest is 6 (X = 1), 4.03, 3.02 (the least of X = 1)."""
    for top in (0x40C0, 0x4081, 0x4041):
        mags = np.arange(top + 1)
        bits = np.concatenate([mags, mags | 0x8000])
        bits = np.concatenate([bits, np.zeros(-len(bits) % 31, dtype=bits.dtype)]).reshape(-1, 31)
        bits = np.concatenate([bits[:, :17], np.full((len(bits), 1), top), bits[:, 17:]], axis=1)
        bits = np.concatenate([bits, np.zeros((-len(bits) % 4, 32), dtype=bits.dtype)])
        same_as_reference(bf16_of(bits.reshape(-1, 128)))


def test_quantize_every_largest_value():
    """Blocks for every positive bf16 number as the largest value, with smaller ones at the borders between codes."""
    rng = np.random.default_rng(0)
    tops = np.arange(0x7F80)
    unit = 2.0 ** np.clip(np.floor(np.log2(np.maximum(bf16_of(tops).double().cpu().numpy(), 2.0 ** -140))) - 2, -126, None)
    some = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2501, 0.7499, 1.251, 2.49, 3.51, 4.99, 0.0, 0.1])
    x = np.concatenate([some, -some])[None, :] * unit[:, None] * rng.choice([0.5, 1.0, 2.0], size=(len(tops), 1))
    x = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    top = bf16_of(tops)
    x = torch.where(x.abs() > top[:, None], torch.zeros_like(x), x)
    x = torch.cat([x[:, :9], top[:, None], x[:, 9:], -top[:, None]], 1)
    assert x.shape[1] == 32
    same_as_reference(x.contiguous().view(-1, 32))
    same_as_reference(torch.cat([x, x.flip(0)], 1).contiguous())


@pytest.mark.parametrize("T,K", [(1, 32), (1, 2048), (3, 96), (70, 544), (33, 4128), (1000, 160), (5, 8192)])
def test_quantize_rows(T, K):
    x = torch.randn(T, K, device=DEV, generator=gen(T)) * torch.exp2(torch.randint(-40, 40, (T, 1), device=DEV, generator=gen(K)).float())
    x[:, ::29] = 0
    x[T // 2] = 0
    x = x.to(torch.bfloat16)
    q, s = same_as_reference(x)
    for dt in BOTH:
        got = qm.moe_dequantize_mx(q, s, out_dtype=dt)
        assert got.dtype == dt and torch.equal(got.double(), decode(q, ungroup(s, K)))


def test_quantize_values_that_are_not_finite():
    x = torch.randn(8, 256, device=DEV, generator=gen(2)).to(torch.bfloat16)
    want_q, want_s = qm.moe_quantize_mx(x)
    x[1, 40] = float("nan")
    x[3, 255] = float("inf")
    x[4, 0] = -float("inf")
    q, s = same_as_reference(x)
    assert sorted(torch.nonzero(ungroup(s, 256) == 255).tolist()) == [[1, 1], [3, 7], [4, 0]]
    same = ungroup(s, 256) != 255
    assert torch.equal(q.view(8, 8, 16)[same], want_q.view(8, 8, 16)[same])
    y = qm.moe_dequantize_mx(q, s).view(8, 8, 32)
    assert bool(y[~same].isnan().all()) and bool(torch.isfinite(y[same]).all())


def test_dequantize_every_code_and_scale():
    """Every code with every scale byte, in both types: exact, infinite past the type's range, NaN at 255."""
    q = torch.arange(256, device=DEV).to(torch.uint8).view(1, 256).repeat(256, 1)  # 512 columns
    byte = torch.arange(256, device=DEV).to(torch.uint8)[:, None].repeat(1, 16)
    want = decode(q, byte)
    for dt in BOTH:
        got = qm.moe_dequantize_mx(q, group(byte), out_dtype=dt)
        most = torch.finfo(dt).max
        ref = torch.where(want.abs() > most, torch.sign(want) * float("inf"), want)
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.double().nan_to_num(7.0), ref.nan_to_num(7.0))
        assert torch.equal(torch.signbit(got[1:255]), torch.signbit(want[1:255]))


@pytest.mark.parametrize("T,k,K", [(1, 8, 2048), (5, 3, 160), (300, 2, 96), (64, 70, 64), (2, 1, 32)])
def test_quantize_into_slots(T, k, K):
    """Each token's row in each of its slots; other rows, and the memory around, stay as they were."""
    M, G = T * k + 9, -(-K // 128)
    x = torch.randn(T, K, device=DEV, generator=gen(T)).to(torch.bfloat16)
    slots = some_slots(T, k, M, T)
    ok = there(slots, M)
    qbuf = torch.full((M + 2, K // 2), 99, dtype=torch.uint8, device=DEV)
    sbuf = torch.full((G + 2, M, 4), 98, dtype=torch.uint8, device=DEV)
    if K // 2 % 16 == 0:
        qm.moe_quantize_mx(x, slots, q=qbuf[1:M + 1], scale=sbuf[1:G + 1])
        q1, s1 = qm.moe_quantize_mx(x)
        want_q, want_s = torch.full_like(qbuf, 99), torch.full_like(sbuf, 98)
        at, token = slots[ok].long(), torch.nonzero(ok)[:, 0]
        want_q[1 + at] = q1[token]
        want_s[1:G + 1][:, at] = s1[:, token]
        assert torch.equal(qbuf, want_q) and torch.equal(sbuf, want_s)
    q, s = qm.moe_quantize_mx(x, slots, rows=M)
    assert q.shape == (M, K // 2) and s.shape == (G, M, 4)


# ------------------------------------------------------------------------------------------- products

SIZES = [(16, 32), (64, 64), (144, 96), (272, 224), (256, 512), (528, 1056), (1040, 2080)]  # (N, K)


@pytest.mark.parametrize("layout", [ROWS, TILE16])
@pytest.mark.parametrize("N,K", SIZES, ids=str)
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 65, 129, 300, 1000])
def test_dense(M, N, K, layout):
    g = gen(M + N + K)
    for kind in ("ints", "binades"):
        xq, xb = operand(g, M, K, kind)
        w, ws, values = weights(g, 1, N, K, kind, layout)
        ws = ws if layout == ROWS else ws[0]
        for dt in BOTH:
            print(f"[mx] {M} {N} {K} {kind} {dt} layout {layout}", flush=True)
            buf = torch.full((M + 2, N), 7.0, dtype=dt, device=DEV)
            got = qm.moe_mx_mm(xq, group(xb), w[0], ws, layout=layout, out=buf[1:M + 1])
            check_product(f"{M} {N} {K}", got, decode(xq, xb), values[0], kind)
            assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


@pytest.mark.parametrize("N", [1, 7, 24, 33, 100, 250, 513])
def test_dense_odd_widths(N):
    """Row-major weights of any N."""
    g = gen(N)
    for M, K in ((1, 64), (40, 288), (260, 640)):
        xq, xb = operand(g, M, K, "binades")
        w, ws, values = weights(g, 1, N, K, "binades", ROWS)
        for dt in BOTH:
            buf = torch.full((M * N + 16,), 7.0, dtype=dt, device=DEV)
            got = qm.moe_mx_mm(xq, group(xb), w[0], ws, out=buf[:M * N].view(M, N))
            check_product(f"{M} {N} {K}", got, decode(xq, xb), values[0], "binades")
            assert bool((buf[M * N:] == 7).all())


@pytest.mark.parametrize("layout", [ROWS, TILE16])
@pytest.mark.parametrize("N,K", [(64, 64), (272, 224), (528, 1056)], ids=str)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_grouped(counts, N, K, layout):
    if len(COUNTS[counts]) > 100 and N == 272:
        pytest.skip("many experts at two sizes are enough")
    off, cnt, M = ranges(COUNTS[counts])
    E, g = len(COUNTS[counts]), gen(len(counts) * 1000 + N + K)
    for kind in ("ints", "binades"):
        xq, xb = operand(g, M, K, kind)
        w, ws, values = weights(g, E, N, K, kind, layout)
        X = decode(xq, xb)
        for dt in BOTH:
            print(f"[mx] {counts} {N} {K} {kind} {dt} layout {layout}", flush=True)
            y = qm.moe_grouped_mx_mm(xq, group(xb), w, ws, off, layout=layout, out_dtype=dt)
            assert y.shape == (M, N) and y.dtype == dt
            for e, r in enumerate(rows_of(off, cnt)):
                if r.stop > r.start:
                    check_product(f"{counts} {e}", y[r], X[r], values[e], kind)


@pytest.mark.parametrize("layout", [ROWS, TILE16])
@pytest.mark.parametrize("step,gap,lead", [(16, 0, 0), (128, 0, 0), (1, 3, 5), (1, 300, 129)])
@pytest.mark.parametrize("hint", [None, 0, 7, 1 << 40])
def test_rows_of_nobody(step, gap, lead, layout, hint):
    """NaN scales in rows of nobody reach no output, whose rows stay as they were, whatever the hint says."""
    counts = [5, 0, 130, 16, 1, 0, 70]
    off, cnt, M = ranges(counts, gap, step, lead)
    N, K, E, g = 80, 160, len(counts), gen(3)
    xq, xb = operand(g, M, K, "binades")
    idle = torch.ones(M, dtype=torch.bool, device=DEV)
    for r in rows_of(off, cnt):
        idle[r] = False
    xb[idle] = 255
    w, ws, values = weights(g, E, N, K, "binades", layout)
    buf = torch.full((M + 8, N), 7.0, device=DEV)
    y = qm.moe_grouped_mx_mm(xq, group(xb), w, ws, off, cnt, hint, layout=layout, out=buf[4:M + 4])
    assert bool((y[idle] == 7).all()) and bool((buf[:4] == 7).all()) and bool((buf[M + 4:] == 7).all())
    X = decode(xq, xb)
    for e, r in enumerate(rows_of(off, cnt)):
        if r.stop > r.start:
            check_product(str(e), y[r], X[r], values[e], "binades")


@pytest.mark.parametrize("layout", [ROWS, TILE16])
@pytest.mark.parametrize("M", [9, 200])
def test_values_that_are_not_finite(M, layout):
    """A scale of 255 makes its own row (of x) or column (of a weight row) NaN and nothing else."""
    N, K, E, g = 96, 224, 2, gen(5)
    off = torch.tensor([0, M // 2, M], dtype=torch.int32, device=DEV)
    xq, xb = operand(g, M, K, "binades")
    q, b = operand(g, E * N, K, "binades")
    xb[3, 2] = 255
    b[N + 11, K // 32 - 1] = 255
    w, ws = (q.view(E, N, -1), group(b)) if layout == ROWS else (tile16(q.view(E, N, -1), 16), tile16(b.view(E, N, -1), 1))
    y = qm.moe_grouped_mx_mm(xq, group(xb), w, ws, off, layout=layout, out_dtype=torch.float32)
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[3] = True
    want[M // 2:, 11] = True
    assert torch.equal(y.isnan(), want)


@pytest.mark.parametrize("M", [4, 400])
def test_scales_at_the_ends(M):
    """The smallest and largest scales meet: only their product has to be in fp32's range.  Sums past it are infinite."""
    N, K = 64, 256
    xq, _ = operand(gen(1), M, K, "ints")
    wq, _ = operand(gen(2), N, K, "ints")
    xb, wb = torch.full((M, K // 32), 254, dtype=torch.uint8, device=DEV), torch.zeros(N, K // 32, dtype=torch.uint8, device=DEV)
    ref = decode(xq, torch.full_like(xb, 127)) @ decode(wq, torch.full_like(wb, 127)).t()
    assert torch.equal(qm.moe_mx_mm(xq, group(xb), wq, group(wb), out_dtype=torch.float32).double(), ref)
    assert torch.equal(qm.moe_mx_mm(xq, group(torch.zeros_like(xb)), wq, group(wb + 254), out_dtype=torch.float32).double(), ref)
    ones = torch.full_like(xq, 0x22)
    y = qm.moe_mx_mm(ones, group(xb), torch.full_like(wq, 0x22), group(wb + 254))
    assert bool((y == float("inf")).all())
    y = qm.moe_mx_mm(ones, group(torch.zeros_like(xb)), torch.full_like(wq, 0x22), group(wb))
    assert bool((y == 0).all())


@pytest.mark.parametrize("M", [4, 400])
def test_sums_that_cancel(M):
    """Blocks 2^18 apart whose large parts cancel: what is left is exact in fp32."""
    N, K = 48, 512
    g = gen(8)
    xq, _ = operand(g, M, K, "ints")
    wq, _ = operand(g, N, K, "ints")
    xb = torch.full((M, K // 32), 127, dtype=torch.uint8, device=DEV)
    wb = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    # codes of 1 and -1 in blocks 0 and 9, scaled by 2^18; small integers elsewhere: |sum| < 2^19 on a grid of a quarter
    for q, value in ((xq, 0x22), (wq, 0x22)):
        q[:, :16] = value
        q[:, 9 * 16:10 * 16] = value
    wq[:, 9 * 16:10 * 16] = 0xAA
    xq[:, 1 * 16:9 * 16] = 0  # few terms: every partial sum is below 2^24 quarters
    xq[:, 12 * 16:] = 0
    xb[:, 0] += 13
    xb[:, 9] += 13
    ref = decode(xq, xb) @ decode(wq, wb).t()
    assert float(ref.abs().max()) < 2.0 ** 13
    assert torch.equal(qm.moe_mx_mm(xq, group(xb), wq, group(wb), out_dtype=torch.float32).double(), ref)


def test_ranges_that_are_not_ranges():
    """Whatever the device arrays hold, nothing outside y is written, and the call ends."""
    N, K, E, M = 64, 128, 6, 90
    g = gen(4)
    xq, xb = operand(g, M, K, "ints")
    w, ws, _ = weights(g, E, N, K, "ints", ROWS)
    big, small = 2 ** 31 - 1, -2 ** 31
    for off, cnt in (([0, 50, 20, 90, 10, 60, 90], None), ([big] * 7, None), ([small, 0, big, 5, small, 90, big], None),
                     ([0, 0, 0, 0, 0, 0, 0], [big] * 6), ([-5, 80, 200, 0, 10, 10, 0], [30, 30, 5, small, 90, 0])):
        buf = torch.full((M + 16, N), 7.0, device=DEV)
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        c = None if cnt is None else torch.tensor(cnt, dtype=torch.int32, device=DEV)
        print("[mx]", off, cnt, flush=True)
        qm.moe_grouped_mx_mm(xq, group(xb), w, ws, o, c, out=buf[8:M + 8])
        torch.cuda.synchronize()
        assert bool((buf[:8] == 7).all()) and bool((buf[M + 8:] == 7).all())


def test_packed_bank_matrices():
    """gate_up and down of a packed MXFP4 bank, as the fused layer takes it."""
    E, H, I, M = 4, 256, 96, 50
    g = gen(6)
    gq, gb = operand(g, E * 2 * I, H, "binades")
    dq, db = operand(g, E * H, I, "binades")
    bank = qm.moe_pack_bank(qm.DeviceBank("mxfp4", E, H, I, gq.view(E, 2 * I, -1), gb.view(E, 2 * I, -1), dq.view(E, H, -1),
                                          db.view(E, H, -1)))
    off = torch.tensor([0, 20, 20, 33, M], dtype=torch.int32, device=DEV)
    for codes, scales, q, b, K in ((bank.gate_up, bank.gate_up_scale, gq, gb, H), (bank.down, bank.down_scale, dq, db, I)):
        xq, xb = operand(g, M, K, "binades")
        y = qm.moe_grouped_mx_mm(xq, group(xb), codes, scales, off, layout=bank.layout, out_dtype=torch.float32)
        rows = qm.moe_grouped_mx_mm(xq, group(xb), q.view(E, -1, K // 2), group(b), off, out_dtype=torch.float32)
        assert torch.equal(y, rows)
        W = decode(q, b).view(E, -1, K)
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            if r.stop > r.start:
                check_product(str(e), y[r], decode(xq, xb)[r], W[e], "binades")


def test_offsets_past_32_bits():
    """Codes, scales and outputs whose byte offsets need more than 32 bits."""
    M, N, K = 1_100_000, 1024, 8192  # 4.5 GB of codes, 2.2 GB of bf16 outputs
    xq = torch.zeros(M, K // 2, dtype=torch.uint8, device=DEV)
    xs = torch.full((K // 128, M, 4), 127, dtype=torch.uint8, device=DEV)
    g = gen(1)
    w, ws, values = weights(g, 1, N, K, "ints", ROWS)
    at = torch.tensor([0, 5, M // 2, M - 257, M - 2, M - 1], device=DEV)
    xq[at], _ = operand(g, len(at), K, "ints")
    xs[:, M - 1] = 125
    y = qm.moe_mx_mm(xq, xs, w[0], ws)
    byte = torch.full((len(at), K // 32), 127, dtype=torch.uint8, device=DEV)
    byte[-1] = 125
    check_product("far rows", y[at], decode(xq[at], byte), values[0], "binades")
    idle = torch.ones(M, dtype=torch.bool, device=DEV)
    idle[at] = False
    assert not bool(y[idle].any())


def test_quantised_layer_run_captured_and_replayed():
    """Routing, alignment, slots, tokens quantised into their rows, both products of a packed bank with the activation
    between, and the rows back, in a graph: every replay, on new inputs, gives what the calls give one by one."""
    T, k, E, H, I = 96, 4, 16, 256, 128
    g = gen(11)
    gq, gb = operand(g, E * 2 * I, H, "binades")
    dq, db = operand(g, E * H, I, "binades")
    bank = qm.moe_pack_bank(qm.DeviceBank("mxfp4", E, H, I, gq.view(E, 2 * I, -1), gb.view(E, 2 * I, -1) - 8,
                                          dq.view(E, H, -1), db.view(E, H, -1) - 8))
    router = (torch.randn(E, H, device=DEV, generator=g) * 0.1).to(torch.bfloat16)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    M = qm.moe_align_capacity(T, k, E, 16)

    def step():
        _, ids, wts = qm.moe_route(x, router, None, k)
        al = qm.moe_align(ids, E, 16)
        slots = qm.moe_pair_slots(ids, al.sorted_ids, al.offsets, al.counts)
        q, s = qm.moe_quantize_mx(x, slots, rows=M)
        gu = qm.moe_grouped_mx_mm(q, s, bank.gate_up, bank.gate_up_scale, al.offsets, al.counts, T * k, layout=bank.layout)
        a = torch.nn.functional.silu(gu[:, :I].float()) * gu[:, I:].float()
        q2, s2 = qm.moe_quantize_mx(a.nan_to_num(0, 0, 0).to(torch.bfloat16))  # rows of nobody hold anything
        y = qm.moe_grouped_mx_mm(q2, s2, bank.down, bank.down_scale, al.offsets, al.counts, T * k, layout=bank.layout)
        return ids, slots, wts, qm.moe_combine_rows(y, slots, wts, out_dtype=torch.float32)

    x.copy_(torch.randn(T, H, device=DEV, generator=gen(0)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2, 3):
        x.copy_(torch.randn(T, H, device=DEV, generator=gen(seed)))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), seed
    # the last step against the layer's formula on the quantised tokens, with its own roundings
    ids, _, wts, out = outs
    xq, xs = qm.moe_quantize_mx(x)
    X = decode(xq, ungroup(xs, H))
    G, D = decode(gq, gb - 8).view(E, 2 * I, H), decode(dq, db - 8).view(E, H, I)
    ref = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    worst = 0.0
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            gu = (X[t] @ G[e].t()).to(torch.bfloat16).double()
            a = (torch.nn.functional.silu(gu[:, :I].float()) * gu[:, I:].float()).to(torch.bfloat16)
            q2, s2 = qm.moe_quantize_mx(a)
            y = decode(q2, ungroup(s2, I)) @ D[e].t()
            ref.index_add_(0, t, y * wts[t, j].double()[:, None])
            worst = max(worst, float((decode(q2, ungroup(s2, I)).abs() @ D[e].abs().t()).max()))
    # a sum within 2^-16 of a rounding border may fall to its other side (bf16, then a code: half of it at most), in a few
    # of a row's I activations, and y is rounded to bf16
    assert float((out.double() - ref).abs().max()) <= worst * (2.0 ** -8 + 0.5 * 4 / I)


def test_straight_through_gradients():
    """Training through quantised operands: the product is that of the values, and the values give the gradients."""
    E, N, K, M = 3, 96, 128, 60
    g = gen(7)
    off = torch.tensor([0, 25, 25, M], dtype=torch.int32, device=DEV)
    x = torch.randn(M, K, device=DEV, generator=g).to(torch.bfloat16)
    w = (torch.randn(E * N, K, device=DEV, generator=g) * 0.1).to(torch.bfloat16)
    (xq, xs), (wq, ws) = qm.moe_quantize_mx(x), qm.moe_quantize_mx(w)
    y = qm.moe_grouped_mx_mm(xq, xs, wq.view(E, N, -1), ws, off, out_dtype=torch.float32)
    xv, wv = qm.moe_dequantize_mx(xq, xs), qm.moe_dequantize_mx(wq, ws).view(E, N, K)
    dy = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16)
    dx = qm.moe_grouped_mm_dgrad(dy, wv, off, out_dtype=torch.float32)
    dw = qm.moe_grouped_mm_wgrad(dy, xv, off, out_dtype=torch.float32)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.stop > r.start:
            X, W, D = xv[r].double(), wv[e].double(), dy[r].double()
            check("y", y[r], X @ W.t(), X.abs() @ W.abs().t(), K)
            check("dx", dx[r], D @ W, D.abs() @ W.abs(), N)
            check("dw", dw[e], D.t() @ X, D.abs().t() @ X.abs(), r.stop - r.start)
        else:
            assert not bool(dw[e].any())


# ------------------------------------------------------------------------------------------- how they are called

def test_no_rows():
    q, s = torch.empty(0, 64, dtype=torch.uint8, device=DEV), torch.empty(1, 0, 4, dtype=torch.uint8, device=DEV)
    w, ws, _ = weights(gen(0), 2, 32, 128, "ints", ROWS)
    assert qm.moe_mx_mm(q, s, w[0], group(torch.zeros(32, 4, dtype=torch.uint8, device=DEV))).shape == (0, 32)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert qm.moe_grouped_mx_mm(q, s, w, ws, off).shape == (0, 32)
    a, b = qm.moe_quantize_mx(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV))
    assert a.shape == (0, 64) and b.shape == (1, 0, 4)
    assert qm.moe_dequantize_mx(a, b).shape == (0, 128)


def test_on_a_stream_of_its_own():
    M, N, K, T, k = 300, 256, 512, 100, 3
    g = gen(2)
    xq, xb = operand(g, M, K, "binades")
    xs = group(xb)
    w, ws, _ = weights(g, 1, N, K, "binades", ROWS)
    x = torch.randn(T, K, device=DEV, generator=g).to(torch.bfloat16)
    slots = some_slots(T, k, M, 2, lost=0.0)

    def calls(stream):
        q, s = qm.moe_quantize_mx(x, slots, rows=M, stream=stream)
        return [qm.moe_mx_mm(xq, xs, w[0], ws, stream=stream), qm.moe_dequantize_mx(xq, xs, stream=stream),
                q[:, slots.new_zeros(1).long()], *qm.moe_quantize_mx(x, stream=stream)]

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    S = torch.cuda.Stream()
    with torch.cuda.stream(S):
        got = calls(S)
    S.synchronize()
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(got, want)) if i != 2)


def test_results_do_not_vary():
    g = gen(3)
    for M in (3, 700):
        xq, xb = operand(g, M, 2048, "binades")
        w, ws, _ = weights(g, 1, 512, 2048, "binades", ROWS)
        want = qm.moe_mx_mm(xq, group(xb), w[0], ws, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(qm.moe_mx_mm(xq, group(xb), w[0], ws, out_dtype=torch.float32), want)
