"""Cases of the rows' way to the experts and back (with its gradients), and of MXFP4: quantiser and products.

With ``own`` false every operator is computed in its plain form (elementary torch operations in 32 bits,
rounded once at the end); with ``own`` true through the library's entry points.

T tokens choose k of E experts each; pair f = t k + j is token t's j-th choice.  Row matrices hold the pairs
sorted by expert, as ``moe_align`` lays them out: ``align`` 1 packs the experts' runs tightly; 16 or 128 starts
every run at a multiple of that many rows, and the rows between the runs are nobody's: they keep the zeros that
the output buffers start with.  ``slots`` [T, k] is the row of each pair, or -1 for a pair that has none.

MXFP4: e2m1 codes, two a byte (the even column in the low nibble), with a power of two (e8m0) for each 32
columns.  ``rows`` banks hold the scales as the quantiser gives them, four of a row together, [K / 128, rows, 4];
``tile16`` banks hold codes and scales as ``moe_pack_bank`` lays them out.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases

def _case(name, **c):
    return dict(c, name=name) if name else c


def _dispatch(name, T, k, E, H, skew, align, dtype, absent=0.0):
    return _case(name, op="dispatch", T=T, k=k, E=E, H=H, skew=skew, align=align, dtype=dtype, absent=absent)


def _combine(name, T, k, E, H, skew, align, dtype, out, add, absent=0.0):
    return _case(name, op="combine", T=T, k=k, E=E, H=H, skew=skew, align=align, dtype=dtype, out=out, add=add, absent=absent)


def _grad(name, T, k, E, H, skew, align, dtype, out, absent=0.0):
    return _case(name, op="grad", T=T, k=k, E=E, H=H, skew=skew, align=align, dtype=dtype, out=out, absent=absent)


def _quantize(name, T, k, E, K, skew, align):
    return _case(name, op="quantize", T=T, k=k, E=E, K=K, skew=skew, align=align, absent=0.0)


def _mm(name, T, k, E, N, K, skew, align, out, layout):
    return _case(name, op="mm", T=T, k=k, E=E, N=N, K=K, skew=skew, align=align, out=out, layout=layout, absent=0.0)


def _dense(name, M, N, K, out, layout):
    return _case(name, op="dense", M=M, N=N, K=K, out=out, layout=layout)


def listed():
    return [
        # one token sent to its eight experts: latency
        _dispatch("dispatch one token", 1, 8, 256, 2048, 1.0, 16, "bf16"),
        # a prefill batch sent to its experts, uneven ones
        _dispatch("dispatch prefill", 8192, 8, 256, 2048, 1.0, 1, "bf16"),
        # a decode batch's pair rows back to their tokens, added to the shared expert's output
        _combine("combine decode", 64, 8, 256, 2048, 1.0, 16, "f32", "f32", True),
        # the same for a prefill batch in bf16
        _combine("combine prefill", 8192, 8, 256, 2048, 1.0, 128, "bf16", "bf16", True),
        # gradients of both ways in a small layer, some pairs dropped
        _grad("grad small", 101, 2, 8, 200, 0.5, 1, "f32", "f32", 0.1),
        # gradients of both ways in training
        _grad("grad training", 8192, 8, 256, 2048, 0.7, 1, "bf16", "bf16"),
        # one token's activations quantised for its eight experts
        _quantize("quantize one token", 1, 8, 256, 2048, 1.0, 16),
        # a prefill batch's activations quantised for their experts
        _quantize("quantize prefill", 8192, 8, 256, 2048, 1.0, 1),
        # one token's eight experts, gate_up of a packed bank: latency and weight streaming
        _mm("mm one token", 1, 8, 256, 1024, 2048, 1.0, 16, "bf16", "tile16"),
        # a decode batch's down projection of a packed bank, two rows an expert on average
        _mm("mm decode", 64, 8, 256, 2048, 1024, 1.0, 16, "f32", "tile16"),
        # a prefill batch's gate_up of a packed bank, uneven experts
        _mm("mm prefill", 8192, 8, 256, 1024, 2048, 1.0, 1, "bf16", "tile16"),
        # a prefill batch through a dense projection, both sides from the quantiser
        _dense("dense prefill", 8192, 4096, 4096, "bf16", "rows"),
    ]


def _log(rng, lo, hi, step=1):
    """A size in [lo, hi], spread over its logarithm, a multiple of `step`."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return min(hi, max(lo, v // step * step))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "grad", "quantize", "mm", "mm", "dense"])
    if op == "dense":
        layout = rng.choice(["rows", "tile16"])
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 64, 8192, 16 if layout == "tile16" else 1), _log(rng, 128, 8192, 32)
            if M * N * K <= 8192 * 4096 * 4096:
                return _dense(None, M, N, K, rng.choice(["bf16", "f32"]), layout)
    E = rng.choice([4, 8, 16, 32, 60, 64, 128, 160, 256])
    skew, align = rng.choice([0.0, 0.5, 1.0]), rng.choice([1, 1, 16, 128])
    dtype, out, absent = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.choice([0.0, 0.0, 0.1])
    while True:
        k, T = rng.choice([1, 2, 4, 6, 8]), _log(rng, 1, 8192)
        if k > E:
            continue
        if op == "mm":
            layout = rng.choice(["rows", "tile16"])
            N, K = _log(rng, 64, 4096, 16 if layout == "tile16" else 1), _log(rng, 64, 4096, 32)
            if T * k * N * K <= 65536 * 1024 * 2048 and E * N * K <= 256 * 1024 * 2048:
                return _mm(None, T, k, E, N, K, skew, align, out, layout)
        if op == "quantize":
            K = _log(rng, 32, 8192, 32)
            if T * k * K <= 65536 * 2048:
                return _quantize(None, T, k, E, K, skew, align)
        H = _log(rng, 64, 8192, 8)
        if T * k * H * (2 if dtype == "f32" else 1) <= 65536 * 2048:
            if op == "dispatch":
                return _dispatch(None, T, k, E, H, skew, align, dtype, absent)
            if op == "combine":
                return _combine(None, T, k, E, H, skew, align, dtype, out, rng.choice([True, False]), absent)
            if op == "grad":
                return _grad(None, T, k, E, H, skew, align, dtype, out, absent)


# ------------------------------------------------------------------------------------------- inputs

def _routing(c, rng):
    """Expert of each pair [T, k] when T tokens choose k different experts each, some experts liked more; a share
    `absent` of the pairs has none (-1)."""
    like = rng.standard_normal(c["E"]) * c["skew"]
    score = like + rng.gumbel(size=(c["T"], c["E"]))
    ids = np.argsort(-score, axis=1, kind="stable")[:, :c["k"]].astype(np.int32)
    ids[rng.random(ids.shape) < c["absent"]] = -1
    return np.ascontiguousarray(ids)


def _alignment(c, ids):
    """moe_align's outputs for ids: sorted_ids [M], offsets [E + 1], counts [E]."""
    P, E, step = ids.size, c["E"], c["align"]
    flat = ids.ravel()
    counts = np.bincount(flat[flat >= 0], minlength=E)
    room = (P + E * (step - 1) + step - 1) // step * step
    offsets = np.concatenate([[0], np.cumsum((counts + step - 1) // step * step)])
    pairs = np.flatnonzero(flat >= 0)
    pairs = pairs[np.argsort(flat[pairs], kind="stable")]
    e = flat[pairs]
    first = np.cumsum(counts) - counts
    sorted_ids = np.full(room, P, dtype=np.int32)
    sorted_ids[offsets[e] + np.arange(len(pairs)) - first[e]] = pairs
    return sorted_ids, offsets.astype(np.int32), counts.astype(np.int32)


def _activations(g, M, K):
    """Rows of N(0, 1) with every 61st channel eight times as large."""
    x = torch.randn(M, K, device="cuda", generator=g)
    x[:, 7::61] *= 8
    return x


def _codes_of_rows(x):
    """Packed codes [M, K / 2] and scales [K / 128, M, 4] of rows (inputs of the products): any valid ones do."""
    M, K = x.shape
    G = -(-K // 128)
    b = x.view(M, K // 32, 32)
    e = (torch.frexp(b.abs().amax(2))[1] - 3).clamp(-126, 127)
    v = b / torch.exp2(e.float())[:, :, None]
    near = torch.bucketize(v.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda"))
    code = (near + 8 * (v < 0)).to(torch.uint8).view(M, K // 2, 2)
    s = torch.zeros(M, G * 4, dtype=torch.uint8, device="cuda")
    s[:, :K // 32] = (e + 127).to(torch.uint8)
    return code[:, :, 0] | code[:, :, 1] << 4, s.view(M, G, 4).permute(1, 0, 2).contiguous()


def _weights(g, E, N, K):
    """Random codes [E, N, K / 2] that use the whole format, and scale bytes [E, N, K / 32] of four binades."""
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    for e in range(E):
        q[e] = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
        s[e] = torch.randint(118, 122, (N, K // 32), device="cuda", generator=g, dtype=torch.uint8)
    return q, s


def _tile16(t, unit):
    """Bytes [E, N, P] in the banks' packed order: 16-row tiles, each stored as its units column by column."""
    E, N, P = t.shape
    return t.view(E, N // 16, 16, P // unit, unit).permute(0, 1, 3, 2, 4).contiguous().view(E, N, P)


def _untile16(t, unit):
    E, N, P = t.shape
    return t.view(E, N // 16, P // unit, 16, unit).permute(0, 1, 3, 2, 4).contiguous().view(E, N, P)


def _scales_by_128(s):
    """Scale bytes [R, K / 32] in the quantiser's order [K / 128, R, 4], zeros past the last."""
    R, S = s.shape
    p = torch.zeros(R, -(-S // 4) * 4, dtype=torch.uint8, device="cuda")
    p[:, :S] = s
    return p.view(R, -1, 4).permute(1, 0, 2).contiguous()


def _bank(c, g, E):
    q, s = _weights(g, E, c["N"], c["K"])
    if c["layout"] == "tile16":
        return _tile16(q, 16), _tile16(s, 1)
    return q, _scales_by_128(s.view(E * c["N"], -1))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": c["op"], "out": DTYPES.get(c.get("out")), "layout": c.get("layout")}
    if c["op"] == "dense":
        s["xq"], s["xs"] = _codes_of_rows(_activations(g, c["M"], c["K"]).bfloat16().float())
        w, ws = _bank(c, g, 1)
        s["w"], s["ws"] = w[0], ws if c["layout"] == "rows" else ws[0]
        s["y"] = torch.zeros(c["M"], c["N"], dtype=s["out"], device="cuda")
        return s
    ids = _routing(c, np.random.default_rng(seed))
    sorted_ids, offsets, counts = _alignment(c, ids)
    T, k, M = c["T"], c["k"], len(sorted_ids)
    s["pairs"], s["most"] = int(counts.sum()), int(counts.max())
    s["ids"], s["sorted"] = torch.from_numpy(ids).cuda(), torch.from_numpy(sorted_ids).cuda()
    s["offsets"], s["counts"] = torch.from_numpy(offsets).cuda(), torch.from_numpy(counts).cuda()
    slots = np.full(T * k + 1, -1, dtype=np.int32)
    slots[sorted_ids] = np.arange(M)
    slots = slots[:-1]
    s["slots"] = torch.from_numpy(slots.reshape(T, k)).cuda()
    dtype = DTYPES.get(c.get("dtype"))
    if c["op"] == "dispatch":
        s["x"] = _activations(g, T, c["H"]).to(dtype)
        s["rows"] = torch.zeros(M, c["H"], dtype=dtype, device="cuda")
        s["slots"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    elif c["op"] == "quantize":
        s["x"] = _activations(g, T, c["K"]).bfloat16()
        s["q"] = torch.zeros(M, c["K"] // 2, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros(-(-c["K"] // 128), M, 4, dtype=torch.uint8, device="cuda")
        s["values"] = torch.zeros(M, c["K"], dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "mm":
        s["xq"], s["xs"] = _codes_of_rows(_activations(g, M, c["K"]).bfloat16().float())
        s["w"], s["ws"] = _bank(c, g, c["E"])
        s["y"] = torch.zeros(M, c["N"], dtype=s["out"], device="cuda")
    else:
        H = c["H"]
        s["rows"] = _activations(g, M, H).to(dtype)
        s["weights"] = torch.softmax(torch.randn(T, k, device="cuda", generator=g), dim=1)
        if c["op"] == "combine":
            s["add"] = _activations(g, T, H).to(s["out"]) if c["add"] else None
            s["y"] = torch.empty(T, H, dtype=s["out"], device="cuda")
        else:
            s["dout"] = torch.randn(T, H, device="cuda", generator=g).to(s["out"])
            s["dx_rows"] = torch.randn(M, H, device="cuda", generator=g).to(dtype)  # the experts' gradients of their rows
            s["drows"] = torch.zeros(M, H, dtype=dtype, device="cuda")
            s["dweights"] = torch.empty(T, k, device="cuda")
            s["dx"] = torch.empty(T, H, dtype=s["out"], device="cuda")
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _token_rows(s, rows):
    """rows[slots] as [T, k, H] in 32 bits, zeros for pairs without a row."""
    got = rows[s["slots"].clamp_min(0).long()].float()
    return got.masked_fill_((s["slots"] < 0)[:, :, None], 0.0)


def _plain_dispatch(s):
    T, k = s["ids"].shape
    P = T * k
    taken = s["sorted"] < P
    pair = s["sorted"].long()
    at = torch.arange(len(pair), device="cuda", dtype=torch.int32)
    slots = torch.full((P + 1,), -1, dtype=torch.int32, device="cuda")
    slots[pair] = at  # the last entry takes the rows of nobody
    rows = s["x"][(pair // k).clamp_max(T - 1)] * taken[:, None]
    return slots[:P].view(T, k), rows


def _plain_combine(s):
    y = (_token_rows(s, s["rows"]) * s["weights"][:, :, None]).sum(1)
    return (y if s["add"] is None else y + s["add"].float()).to(s["out"])


def _plain_grad(s):
    T, k = s["slots"].shape
    there = s["slots"] >= 0
    dweights = (_token_rows(s, s["rows"]) * s["dout"].float()[:, None, :]).sum(2)
    d = s["dout"].float()[:, None, :] * s["weights"][:, :, None]
    drows = torch.zeros(len(s["rows"]) + 1, s["rows"].shape[1], dtype=s["rows"].dtype, device="cuda")
    at = torch.where(there, s["slots"], len(s["rows"])).long().view(-1)  # pairs without a row go to one past the last
    drows[at] = d.view(T * k, -1).to(drows.dtype)
    return drows[:-1], dweights, _token_rows(s, s["dx_rows"]).sum(1).to(s["out"])


def _grid(v):
    """The e2m1 value nearest to each number, ties to the even code, at most 6 in magnitude."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp_max(6.0) * torch.sign(v)


def _plain_quantize(s):
    T, K = s["x"].shape
    x = s["x"].float().view(T, K // 32, 32)
    top = x.abs().amax(2)
    # the smallest power of two that leaves nothing above 6 = 1.5 * 2^2, and 2^-126 at least
    m, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1
    e = (e - 3 + (m > 0.75).int()).clamp_min(-126)
    unit = ((e + 127) << 23).view(torch.float32)
    values = (_grid(x / unit[:, :, None]) * unit[:, :, None]).view(T, K).to(torch.bfloat16)
    pair = s["sorted"].long()
    taken = pair < s["slots"].numel()
    token = (pair // s["slots"].shape[1]).clamp_max(T - 1)
    byte = torch.zeros(T, -(-K // 128) * 4, dtype=torch.uint8, device="cuda")
    byte[:, :K // 32] = (e + 127).to(torch.uint8)
    scale = (byte[token] * taken[:, None]).view(len(pair), -1, 4).permute(1, 0, 2).contiguous()
    return values[token] * taken[:, None], scale


def _values(codes, scale_bytes):
    """Codes [..., K / 2] times scales [..., K / 32], in 32 bits, as [..., K]."""
    of_code = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    of_byte = torch.stack([of_code.repeat(16), of_code.repeat_interleave(16)], 1)  # the low nibble first
    v = torch.nn.functional.embedding(codes.int(), of_byte).view(*scale_bytes.shape, 32)
    unit = (scale_bytes.int() << 23).view(torch.float32)
    return v.mul_(unit[..., None]).view(*codes.shape[:-1], -1)


def _scale_rows(s, K):
    """Scales [K / 128, R, 4] as [R, K / 32]."""
    return s.permute(1, 0, 2).reshape(s.shape[1], -1)[:, :K // 32]


def _plain_weights(w, ws, layout):
    K = w.shape[-1] * 2
    if layout == "tile16":
        three, ws = w.view(-1, *w.shape[-2:]), ws.view(-1, *ws.shape[-2:])
        return _values(_untile16(three, 16), _untile16(ws, 1)).view(*w.shape[:-1], K)
    return _values(w, _scale_rows(ws, K).reshape(*w.shape[:-1], K // 32))


def _plain_dense(s):
    x = _values(s["xq"], _scale_rows(s["xs"], s["xq"].shape[1] * 2))
    return torch.mm(x, _plain_weights(s["w"], s["ws"], s["layout"]).t()).to(s["out"])


def _plain_mm(s):
    (E, N, _), G = s["w"].shape, len(s["xs"])
    used = torch.nonzero(s["counts"]).view(-1)  # experts that have rows
    w = s["w"][used]
    ws = s["ws"][used] if s["layout"] == "tile16" else s["ws"].view(G, E, N, 4)[:, used].reshape(G, -1, 4)
    pair = torch.nonzero(s["sorted"] < s["slots"].numel()).view(-1)  # rows of some expert
    e = s["ids"].view(-1)[s["sorted"][pair].long()].long()
    place, e = pair - s["offsets"][e], torch.searchsorted(used, e)
    x = _values(s["xq"], _scale_rows(s["xs"], s["xq"].shape[1] * 2))
    z = torch.zeros(len(used), s["most"], x.shape[1], device="cuda")
    z[e, place] = x[pair]
    z = torch.bmm(z, _plain_weights(w, ws, s["layout"]).transpose(1, 2).contiguous())
    y = torch.zeros(len(s["sorted"]), N, dtype=s["out"], device="cuda")
    y[pair] = z[e, place].to(s["out"])
    return y


PLAIN = {"dispatch": _plain_dispatch, "combine": _plain_combine, "grad": _plain_grad, "quantize": _plain_quantize,
         "mm": _plain_mm, "dense": _plain_dense}


def run(state):
    s = state
    if not own:
        return PLAIN[s["op"]](s)
    import quantized_moe_expert_topk_amd as qm
    if s["op"] == "dispatch":
        slots = qm.moe_pair_slots(s["ids"], s["sorted"], s["offsets"], s["counts"], slots=s["slots"])
        return slots, qm.moe_gather_rows(s["x"], slots, out=s["rows"])
    if s["op"] == "combine":
        return qm.moe_combine_rows(s["rows"], s["slots"], s["weights"], add=s["add"], out=s["y"])
    if s["op"] == "grad":
        drows, dweights = qm.moe_combine_rows_grad(s["dout"], s["rows"], s["slots"], s["weights"], drows=s["drows"],
                                                   dweights=s["dweights"])
        return drows, dweights, qm.moe_combine_rows(s["dx_rows"], s["slots"], out=s["dx"])
    if s["op"] == "quantize":
        q, scale = qm.moe_quantize_mx(s["x"], s["slots"], q=s["q"], scale=s["scale"])
        return qm.moe_dequantize_mx(q, scale, out=s["values"]), scale
    layout = qm.MOE_LAYOUT_TILE16 if s["layout"] == "tile16" else qm.MOE_LAYOUT_ROWS
    if s["op"] == "dense":
        return qm.moe_mx_mm(s["xq"], s["xs"], s["w"], s["ws"], layout=layout, out=s["y"])
    return qm.moe_grouped_mx_mm(s["xq"], s["xs"], s["w"], s["ws"], s["offsets"], s["counts"], s["pairs"],
                                   layout=layout, out=s["y"])


# ------------------------------------------------------------------------------------------- work

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "dense":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * (K // 2 + K // 32) + size[c["out"]] * M * N, "flops": 2 * M * N * K}
    T, P, E = c["T"], c["T"] * c["k"], c["E"]
    if c["op"] == "dispatch":
        return {"bytes": (T + P) * c["H"] * size[c["dtype"]] + 12 * P + 8 * E, "flops": P}
    if c["op"] == "combine":
        out = T * c["H"] * size[c["out"]] * (2 if c["add"] else 1)
        return {"bytes": P * c["H"] * size[c["dtype"]] + out + 8 * P, "flops": 2 * P * c["H"]}
    if c["op"] == "grad":
        return {"bytes": 3 * P * c["H"] * size[c["dtype"]] + 2 * T * c["H"] * size[c["out"]] + 16 * P, "flops": 4 * P * c["H"]}
    if c["op"] == "quantize":  # quantised, and the values that the codes stand for
        K = c["K"]
        return {"bytes": 2 * T * K + 2 * P * (K // 2 + K // 32) + 2 * P * K + 4 * P, "flops": 3 * T * K + P * K}
    N, K = c["N"], c["K"]
    active = len(np.unique(_routing(c, np.random.default_rng(0))))  # weights of idle experts are not needed
    return {"bytes": (P + active * N) * (K // 2 + K // 32) + size[c["out"]] * P * N + 8 * E, "flops": 2 * P * N * K}


# ------------------------------------------------------------------------------------------- 64 bits

def _rows_of_tokens(slots, M):
    """For each row its (token, choice), or -1."""
    t = np.full((M, 2), -1, dtype=np.int64)
    at = np.argwhere(slots >= 0)
    t[slots[at[:, 0], at[:, 1]]] = at
    return torch.from_numpy(t[:, 0]).cuda(), torch.from_numpy(t[:, 1]).cuda()


def _decode(codes, scale_bytes):
    """Codes [n, K / 2] and scale bytes [n, K / 32] as 64-bit values [n, K], from the bits of each code."""
    n = codes.shape[0]
    c = torch.stack([codes & 15, codes >> 4], 2).view(n, -1).to(torch.int64)
    e, m = c >> 1 & 3, (c & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.where(e == 3, 4.0, torch.where(e == 2, 2.0, 1.0)).double())
    v = torch.where(c >= 8, -v, v)
    unit = (scale_bytes.to(torch.int64) - 127 + 1023 << 52).view(torch.float64)
    return (v.view(n, -1, 32) * unit[:, :, None]).view(n, -1)


def _weights_of(c, s, e):
    w = s["w"] if c["op"] == "dense" else s["w"][e]
    N, K = c["N"], c["K"]
    if c["layout"] == "tile16":
        ws = s["ws"] if c["op"] == "dense" else s["ws"][e]
        w = w.reshape(N // 16, K // 32, 16, 16).transpose(1, 2).reshape(N, K // 2)
        return _decode(w, ws.reshape(N // 16, K // 32, 16).transpose(1, 2).reshape(N, K // 32))
    ws = s["ws"][:, e * N:e * N + N]
    return _decode(w, torch.cat(list(ws), 1)[:, :K // 32])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "dense":
        x = _decode(s["xq"], torch.cat(list(s["xs"]), 1)[:, :c["K"] // 32])
        return x @ _weights_of(c, s, 0).t()
    if c["op"] == "mm":
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        xs = torch.cat(list(s["xs"]), 1)[:, :c["K"] // 32]
        starts, counts = s["offsets"].tolist(), s["counts"].tolist()
        for e in range(c["E"]):
            if counts[e]:
                rows = slice(starts[e], starts[e] + counts[e])
                y[rows] = _decode(s["xq"][rows], xs[rows]) @ _weights_of(c, s, e).t()
        return y
    M = len(s["sorted"])
    ids = s["ids"].cpu().numpy()
    if c["op"] == "dispatch":
        slots, nxt = np.full(ids.shape, -1, dtype=np.int32), s["offsets"].cpu().numpy().copy()
        for t in range(c["T"]):  # in the pairs' order, each to its expert's next row
            for j in range(c["k"]):
                if ids[t, j] >= 0:
                    slots[t, j] = nxt[ids[t, j]]
                    nxt[ids[t, j]] += 1
        token, _ = _rows_of_tokens(slots, M)
        rows = torch.zeros(M, c["H"], dtype=torch.float64, device="cuda")
        rows[token >= 0] = s["x"].double()[token[token >= 0]]
        return torch.from_numpy(slots).cuda(), rows
    token, choice = _rows_of_tokens(s["slots"].cpu().numpy(), M)
    there = token >= 0
    if c["op"] == "quantize":
        x = s["x"].double()
        T, K = x.shape
        grid = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device="cuda")  # even codes first: the first of equals wins
        of = torch.tensor([0, 1, 2, 4, .5, 1.5, 3, 6], dtype=torch.float64, device="cuda")
        values, byte = torch.zeros_like(x), torch.zeros(T, -(-K // 128) * 4, dtype=torch.int64, device="cuda")
        for b in range(K // 32):
            part = x[:, 32 * b:32 * b + 32]
            top, e = part.abs().amax(1), torch.full((T,), -126, device="cuda")
            for p in range(-126, 126):
                at = (6.0 * 2.0 ** p < top)
                if not bool(at.any()):
                    break
                e[at] = p + 1
            unit = (e.to(torch.int64) + 1023 << 52).view(torch.float64)
            near = ((part / unit[:, None]).abs()[:, :, None] - of).abs()
            first = torch.zeros(near.shape[:2], dtype=torch.int64, device="cuda")
            least = near[:, :, 0].clone()
            for i in range(1, len(grid)):
                less = near[:, :, i] < least
                first[less] = i
                least = torch.minimum(least, near[:, :, i])
            values[:, 32 * b:32 * b + 32] = of[first] * torch.sign(part) * unit[:, None]
            byte[:, b] = e + 127
        out = torch.zeros(M, K, dtype=torch.float64, device="cuda")
        out[there] = values[token[there]]
        scale = torch.zeros(M, byte.shape[1], dtype=torch.uint8, device="cuda")
        scale[there] = byte[token[there]].to(torch.uint8)
        return out, torch.stack(list(scale.split(4, dim=1)), 0).contiguous()
    rows, w = s["rows"].double(), s["weights"].double()
    T, H = len(ids), c["H"]
    if c["op"] == "combine":
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
        return y.index_add(0, token[there], rows[there] * w[token[there], choice[there]][:, None])
    dout = s["dout"].double()[token[there]]
    drows = torch.zeros(M, H, dtype=torch.float64, device="cuda")
    drows[there] = dout * w[token[there], choice[there]][:, None]
    dweights = torch.zeros(T, c["k"], dtype=torch.float64, device="cuda")
    dweights[token[there], choice[there]] = (dout * rows[there]).sum(1)
    dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    return drows, dweights, dx.index_add(0, token[there], s["dx_rows"].double()[there])
