"""Measured cases of the microscaled (MX) operators and of the experts' layer
built on them: rows quantized into MX blocks and read back, products with
e2m1 weights, a router with the tokens sorted by expert, the experts'
products, and the way back with the router's weights.

`run` computes each case in its plain form (elementary torch operations in 32
bits) or, where `own` is true, through the library's entry points. `exact`
gives the same outputs from the operators' definitions in 64 bits.

MX rows: 32 consecutive elements of a row share a scale byte s, which stands
for 2^(s - 127) (255: NaN). Elements are e2m1 (two to a byte, even k in the
low nibble) or e4m3 (one a byte). Scale rows are padded to whole 4 bytes.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
DT = {F32: torch.float32, BF16: torch.bfloat16}
E2M1, E4M3 = "e2m1", "e4m3"
EMAX = {E2M1: 2, E4M3: 8}
INF = float("inf")


def listed():
    return [
        # the hidden rows of one decode step before a product (latency)
        dict(name="quant_64x2048", op="quant", dtype=F32, fmt=E4M3, rows=64, k=2048, pad=0),
        # the inner rows of a long prompt, parts of wider rows
        dict(name="quant_16411x6144", op="quant", dtype=BF16, fmt=E2M1, rows=16411, k=6144, pad=128),
        # one token through one projection (latency)
        dict(name="gemm_1x6144x2048", op="gemm", fmt=E4M3, out=F32, n=1, m=6144, k=2048, silu=0),
        # a batch of decoding requests through a gate and up projection
        dict(name="gemm_77x17408x5120_silu", op="gemm", fmt=E4M3, out=BF16, n=77, m=17408, k=5120, silu=1),
        # a long prompt through a wide projection
        dict(name="gemm_10240x17408x5120", op="gemm", fmt=E2M1, out=BF16, n=10240, m=17408, k=5120, silu=0),
        # the experts of a decode step chosen (latency)
        dict(name="route_64x128", op="route", dtype=F32, rows=64, experts=128, top=8, renorm=1, pad=0, masked=0),
        # the experts of a long prompt, some of them masked, rows without any among them
        dict(name="route_16411x256", op="route", dtype=BF16, rows=16411, experts=256, top=6, renorm=0, pad=0, masked=1),
        # one token through the gate and up products of its experts
        dict(name="experts_1_of_128_silu", op="experts", fmt=E4M3, out=F32, rows=1, experts=128, top=8, m=1024, k=2048, silu=1,
             gather=1, skew=0.5),
        # a decode step's rows, sorted by expert, through the experts' down products
        dict(name="experts_64_of_128_down", op="experts", fmt=E4M3, out=F32, rows=64, experts=128, top=8, m=2048, k=1024, silu=0,
             gather=0, skew=0.5),
        # a prompt through the gate and up products, experts unevenly liked
        dict(name="experts_4099_of_64_silu", op="experts", fmt=E2M1, out=BF16, rows=4099, experts=64, top=8, m=1024, k=2048, silu=1,
             gather=1, skew=0.7),
        # the way back of a decode step
        dict(name="combine_64x8x2048", op="combine", dtype=F32, out=F32, rows=64, top=8, m=2048, dropped=0),
        # the way back of a prompt, some pairs being another card's
        dict(name="combine_16411x8x2048", op="combine", dtype=BF16, out=BF16, rows=16411, top=8, m=2048, dropped=1),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "route", "experts", "experts", "combine"])
    if op == "quant":
        k = _log_int(rng, 64, 16384, 32)
        return dict(op=op, dtype=rng.choice([F32, BF16]), fmt=rng.choice([E2M1, E4M3]), rows=_log_int(rng, 1, max(2, 100000000 // k)),
                    k=k, pad=rng.choice([0, 8, 128]))
    if op == "route":
        experts = rng.choice([8, 16, 60, 64, 100, 128, 256, 512])
        return dict(op=op, dtype=rng.choice([F32, BF16]), rows=_log_int(rng, 1, 16411), experts=experts,
                    top=rng.choice([t for t in (1, 2, 4, 6, 8, 10) if t <= experts]), renorm=rng.choice([0, 1]),
                    pad=rng.choice([0, 0, 3]), masked=rng.choice([0, 1]))
    if op == "combine":
        return dict(op=op, dtype=rng.choice([F32, BF16]), out=rng.choice([F32, BF16]), rows=_log_int(rng, 1, 12000),
                    top=rng.choice([1, 2, 4, 6, 8]), m=_log_int(rng, 256, 4096, 8), dropped=rng.choice([0, 1]))
    fmt, out, silu = rng.choice([E2M1, E4M3]), rng.choice([F32, BF16]), rng.choice([0, 1])
    if op == "gemm":
        m, k = _log_int(rng, 64, 20000), _log_int(rng, 256, 16384, 32)
        n = _log_int(rng, 1, max(2, min(10240, 10 ** 12 // (m * k * (1 + silu)))))
        return dict(op=op, fmt=fmt, out=out, n=n, m=m, k=k, silu=silu)
    experts = rng.choice([8, 16, 60, 64, 128])
    m, k = _log_int(rng, 256, 4096, 4), _log_int(rng, 256, 4096, 32)
    while experts * m * k > 64 * 2048 * 2048:
        experts //= 2
    top = rng.choice([t for t in (1, 2, 4, 6, 8) if t <= experts])
    return dict(op=op, fmt=fmt, out=out, rows=_log_int(rng, 1, 8192 if m * k * top < 2 ** 24 else 2048), experts=experts, top=top, m=m, k=k,
                silu=silu, gather=rng.choice([0, 1]), skew=rng.choice([0.0, 0.5, 1.0]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)


def _normal(g, *shape):
    return torch.empty(*shape, device="cuda").normal_(generator=g)


def _pitch(k):
    """Bytes of a row of scales."""
    return (k // 32 + 3) // 4 * 4


def _tables():
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(mags + [-v for v in mags], device="cuda")


def _elements(x, fmt):
    """x float32 [..., 32] as (elements, their float32 values before the
    shared scale, scale bytes [...]): the scale's power of two is the largest
    magnitude's, less the element type's largest exponent."""
    big = x.abs().amax(-1).contiguous()
    exp = (big.view(torch.int32) >> 23) & 0xFF
    byte = (exp - EMAX[fmt]).clamp(min=0)
    y = torch.ldexp(x, (127 - byte)[..., None].float())
    if fmt == E4M3:
        code = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return code.view(torch.uint8), code.float(), byte
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= edge) if i % 2 else (a > edge)          # a tie goes to the even code
    code |= torch.signbit(y).to(torch.uint8) << 3
    return code, _tables()[code.long()], byte


def _quantized(x, fmt):
    """Rows x float32 [rows][k] as (codes, scales) bytes."""
    rows, k = x.shape
    code, _, byte = _elements(x.reshape(rows, k // 32, 32), fmt)
    code = code.reshape(rows, k)
    if fmt == E2M1:
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = torch.zeros(rows, _pitch(k), dtype=torch.uint8, device="cuda")
    scales[:, :k // 32] = byte.to(torch.uint8)
    return code.contiguous(), scales


def _weights(g, rows, k):
    """e2m1 weights: a bell of values whose size differs from row to row."""
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, _pitch(k), dtype=torch.uint8, device="cuda")
    step = max(1, 2 ** 26 // k)
    for at in range(0, rows, step):
        n = min(step, rows - at)
        w = _normal(g, n, k) * torch.exp(0.3 * _normal(g, n, 1)) * (1.5 / math.sqrt(k))
        codes[at:at + n], scales[at:at + n] = _quantized(w, E2M1)
    return codes, scales


def _activations(g, rows, k, fmt):
    """Rows with a few channels much larger than the others."""
    gain = torch.exp(0.4 * _normal(g, k)) * torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 12.0, 1.0)
    return _quantized(_normal(g, rows, k) * gain, fmt)


def _liked(g, rows, experts, skew):
    """A router's logits: some experts are liked more than others."""
    return 1.5 * _normal(g, rows, experts) + 2.0 * skew * _normal(g, experts)


def _sorted_by_expert(ids, experts):
    """offsets, order, slots of ids int32 [rows][top]."""
    flat = ids.reshape(-1).long()
    mine = (flat >= 0) & (flat < experts)
    key = torch.where(mine, flat, torch.full_like(flat, experts))
    at = torch.sort(key, stable=True).indices
    count = torch.zeros(experts + 1, dtype=torch.long, device="cuda").scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([count.new_zeros(1), count[:experts].cumsum(0)])
    place = torch.arange(flat.numel(), device="cuda")
    real = place < offsets[-1]
    none = torch.full_like(place, -1)
    slots = torch.empty_like(place).scatter_(0, at, torch.where(real, place, none))
    return offsets.int(), torch.where(real, at, none).int(), slots.reshape(ids.shape).int()


def _best(x, top):
    """The first `top` of rows x float32 by larger value, then lower index:
    (values, indices)."""
    bits = (x + 0.0).contiguous().view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    j = torch.arange(x.shape[-1], device="cuda")
    key = torch.topk(order * (1 << 32) + (0xFFFFFFFF - j), top, dim=-1).values
    at = 0xFFFFFFFF - (key & 0xFFFFFFFF)
    return x.gather(-1, at), at


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "quant":
        spread = torch.exp(0.6 * _normal(g, case["k"]))
        x = torch.zeros(case["rows"], case["k"] + case["pad"], dtype=DT[case["dtype"]], device="cuda")
        step = max(1, 2 ** 26 // case["k"])
        for at in range(0, case["rows"], step):
            n = min(step, case["rows"] - at)
            x[at:at + n, :case["k"]] = _normal(g, n, case["k"]) * spread
        s.update(x=x)
    elif op == "gemm":
        s.update(w=_weights(g, case["m"] * (1 + case["silu"]), case["k"]), x=_activations(g, case["n"], case["k"], case["fmt"]))
    elif op == "route":
        x = _liked(g, case["rows"], case["experts"] + case["pad"], 0.5).to(DT[case["dtype"]])
        if case["masked"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < 0.1, -INF)
            x.masked_fill_(torch.rand(case["rows"], 1, generator=g, device="cuda") < 0.02, -INF)
        s.update(x=x)
    elif op == "experts":
        ids = _best(_liked(g, case["rows"], case["experts"], case["skew"]), case["top"])[1].int()
        offsets, order, slots = _sorted_by_expert(ids, case["experts"])
        pairs = case["rows"] * case["top"]
        s.update(w=_weights(g, case["experts"] * case["m"] * (1 + case["silu"]), case["k"]),
                 x=_activations(g, case["rows"] if case["gather"] else pairs, case["k"], case["fmt"]),
                 offsets=offsets, order=order, counts=(offsets[1:] - offsets[:-1]).tolist())
    else:
        pairs = case["rows"] * case["top"]
        slots = torch.randperm(pairs, generator=g, device="cuda").int().reshape(case["rows"], case["top"])
        if case["dropped"]:
            slots = torch.where(torch.rand(slots.shape, generator=g, device="cuda") < 0.2, -1, slots).int()
        w = torch.rand(case["rows"], case["top"], generator=g, device="cuda") + 0.05
        s.update(y=_normal(g, pairs, case["m"]).to(DT[case["dtype"]]), slots=slots, weights=w / w.sum(-1, keepdim=True))
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _values(codes, scales, k, fmt):
    """float32 values of MX rows."""
    if fmt == E2M1:
        t = _tables()
        v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], -1)
    else:
        v = codes.view(torch.float8_e4m3fn).float()
    size = scales[:, :k // 32].int()
    factor = torch.ldexp(torch.ones(size.shape, device="cuda"), (size - 127).float())
    return (v.reshape(-1, k // 32, 32) * factor[..., None]).reshape(-1, k)


def _plain_product(x, w, silu):
    y = torch.matmul(x, w.t().contiguous())
    if silu:
        gate, up = y.chunk(2, dim=-1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y


def _plain_quant(s):
    c = s["case"]
    out = torch.empty(c["rows"], c["k"], device="cuda")
    step = max(1, 2 ** 25 // c["k"])
    for at in range(0, c["rows"], step):
        x = s["x"][at:at + step, :c["k"]].float()
        _, v, byte = _elements(x.reshape(x.shape[0], -1, 32), c["fmt"])
        out[at:at + step] = torch.ldexp(v, (byte - 127)[..., None].float()).reshape(x.shape)
    return out


def _plain_gemm(s):
    c = s["case"]
    y = _plain_product(_values(*s["x"], c["k"], c["fmt"]), _values(*s["w"], c["k"], E2M1), c["silu"])
    return y.to(DT[c["out"]])


def _plain_route(s):
    c = s["case"]
    x = s["x"][:, :c["experts"]].float()
    value, at = _best(x, c["top"])
    m = value[:, :1]
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    z = torch.exp((value if c["renorm"] else x) - m).sum(-1, keepdim=True)
    weights = torch.exp(value - m) / torch.where(z == 0, torch.ones_like(z), z)
    ids = torch.where(value == -INF, torch.full_like(at, -1), at).int()
    offsets, order, slots = _sorted_by_expert(ids, c["experts"])
    return dict(ids=ids, weights=weights, offsets=offsets, order=order, slots=slots)


def _plain_experts(s):
    c = s["case"]
    x = _values(*s["x"], c["k"], c["fmt"])
    if c["gather"]:
        x = x[s["order"].long() // c["top"]]
    y = torch.empty(c["rows"] * c["top"], c["m"], dtype=DT[c["out"]], device="cuda")
    at, wide = 0, c["m"] * (1 + c["silu"])
    for e, n in enumerate(s["counts"]):
        if n:
            w = _values(s["w"][0][e * wide:(e + 1) * wide], s["w"][1][e * wide:(e + 1) * wide], c["k"], E2M1)
            y[at:at + n] = _plain_product(x[at:at + n], w, c["silu"]).to(y.dtype)
        at += n
    return y


def _plain_combine(s):
    c = s["case"]
    out = torch.zeros(c["rows"], c["m"], device="cuda")
    for j in range(c["top"]):
        at = s["slots"][:, j].long()
        row = torch.where((at >= 0)[:, None], s["y"][at.clamp(min=0)].float(), torch.zeros((), device="cuda"))
        out = out + s["weights"][:, j:j + 1] * row
    return out.to(DT[c["out"]])


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _once(s, key, make):
    """A buffer that a user's program keeps from one call to the next."""
    if key not in s:
        s[key] = make()
    return s[key]


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _scratch(need):
    return _empty(need, dtype=torch.uint8) if need else None


def _names(q, c):
    return dict(dtype=q.QG_F32 if c.get("dtype") == F32 else q.QG_BF16, out=q.QG_F32 if c.get("out") == F32 else q.QG_BF16,
                fmt=q.QMX_E2M1 if c.get("fmt") == E2M1 else q.QMX_E4M3, act=q.QMX_SILU_MUL if c.get("silu") else q.QMX_NONE)


def _own_quant(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    R, K, t = c["rows"], c["k"], _names(q, c)
    codes, scales, back = _once(s, "out", lambda: (_empty(R, K // 2 if c["fmt"] == E2M1 else K, dtype=torch.uint8),
                                                   _empty(R, q.qmx_scale_pitch(K), dtype=torch.uint8), _empty(R, K)))
    q.qmx_quant(t["dtype"], s["x"], K + c["pad"], R, K, t["fmt"], codes, scales)
    q.qmx_dequant(t["fmt"], codes, scales, R, K, q.QG_F32, back, K)
    return back


def _own_gemm(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    N, M, K, t = c["n"], c["m"], c["k"], _names(q, c)
    ws = _once(s, "ws", lambda: _scratch(q.qmx_gemm_workspace_bytes(t["fmt"], t["act"], M, K, N)))
    y = _once(s, "y", lambda: _empty(N, M, dtype=DT[c["out"]]))
    q.qmx_gemm(t["fmt"], *s["x"], *s["w"], t["act"], t["out"], y, M, K, N, ws)
    return y


def _own_route(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    R, E, top = c["rows"], c["experts"], c["top"]
    ws = _once(s, "ws", lambda: _scratch(q.qmoe_plan_workspace_bytes(R, E, top)))
    o = _once(s, "out", lambda: dict(ids=_empty(R, top, dtype=torch.int32), weights=_empty(R, top), offsets=_empty(E + 1, dtype=torch.int32),
                                     order=_empty(R * top, dtype=torch.int32), slots=_empty(R, top, dtype=torch.int32)))
    q.qmoe_route(_names(q, c)["dtype"], s["x"], E + c["pad"], R, E, top, c["renorm"], o["ids"], o["weights"], o["offsets"], o["order"],
                 o["slots"], ws)
    return o


def _own_experts(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    R, E, top, M, K, t = c["rows"], c["experts"], c["top"], c["m"], c["k"], _names(q, c)
    ws = _once(s, "ws", lambda: _scratch(q.qmoe_gemm_workspace_bytes(t["fmt"], t["act"], R, E, top, M, K)))
    y = _once(s, "y", lambda: _empty(R * top, M, dtype=DT[c["out"]]))
    q.qmoe_gemm(t["fmt"], *s["x"], *s["w"], s["offsets"], s["order"] if c["gather"] else None, R, E, top, t["act"], t["out"], y, M, K, ws)
    return y


def _own_combine(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    t = _names(q, c)
    out = _once(s, "out", lambda: _empty(c["rows"], c["m"], dtype=DT[c["out"]]))
    q.qmoe_combine(t["dtype"], s["y"], s["slots"], s["weights"], c["rows"], c["top"], c["m"], t["out"], out)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"quant": _own_quant, "gemm": _own_gemm, "route": _own_route, "experts": _own_experts, "combine": _own_combine}[op](state)
    return {"quant": _plain_quant, "gemm": _plain_gemm, "route": _plain_route, "experts": _plain_experts, "combine": _plain_combine}[op](state)


# ---------------------------------------------------------------------------
# Work and the definitions in 64 bits
# ---------------------------------------------------------------------------

def _row_bytes(k, fmt):
    return (k // 2 if fmt == E2M1 else k) + k // 32


def work(case):
    op = case["op"]
    size, out = (4 if case.get("dtype") == F32 else 2), (4 if case.get("out") == F32 else 2)
    if op == "quant":
        n = case["rows"] * case["k"]
        return {"bytes": n * (size + 4) + 2 * case["rows"] * _row_bytes(case["k"], case["fmt"]), "flops": 4 * n}
    if op == "route":
        pairs = case["rows"] * case["top"]
        return {"bytes": case["rows"] * case["experts"] * size + 16 * pairs + 4 * case["experts"] + 4,
                "flops": 6 * case["rows"] * case["experts"]}
    if op == "combine":
        pairs = case["rows"] * case["top"]
        kept = 0.8 if case["dropped"] else 1.0
        return {"bytes": int(kept * pairs * case["m"] * size) + case["rows"] * case["m"] * out + 8 * pairs, "flops": int(2 * kept * pairs * case["m"])}
    wide = case["m"] * (1 + case["silu"])
    if op == "gemm":
        n, rows, sets = case["n"], case["n"], 1
    else:
        n = case["rows"] * case["top"]
        rows = case["rows"] if case["gather"] else n
        sets = min(case["experts"], n)               # at most: how many are chosen depends on the inputs
        if n > sets:
            sets = min(sets, max(1, round(case["experts"] * (1 - (1 - 1 / case["experts"]) ** n))))
    return {"bytes": sets * wide * _row_bytes(case["k"], E2M1) + rows * _row_bytes(case["k"], case["fmt"]) + n * case["m"] * out,
            "flops": 2 * n * wide * case["k"]}


def _wide(codes, scales, k, fmt):
    """float64 values of MX rows, from the bit fields."""
    if fmt == E2M1:
        c = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], k).long()
        sign, exp, man = c >> 3, (c >> 1) & 3, c & 1
        bias, one = 1, 2.0
    else:
        c = codes.long()
        sign, exp, man = c >> 7, (c >> 3) & 15, c & 7
        bias, one = 7, 8.0
    mag = torch.where(exp == 0, man.double() / one * 2.0 ** (1 - bias), (1.0 + man.double() / one) * torch.exp2((exp - bias).double()))
    size = torch.exp2(scales[:, :k // 32].double() - 127.0)
    return torch.where(sign == 1, -mag, mag) * size.repeat_interleave(32, dim=1)


def _exact_rows(xs, ws, m, k, fmt, silu):
    """Outputs float64 of some rows, the weights taken in pieces."""
    x = _wide(*xs, k, fmt)
    out = torch.empty(x.shape[0], m, dtype=torch.float64, device="cuda")
    step = max(1, 2 ** 25 // k)
    for a in range(0, m, step):
        b = min(m, a + step)
        y = x @ _wide(ws[0][a:b], ws[1][a:b], k, E2M1).T
        if silu:
            y = y * torch.sigmoid(y) * (x @ _wide(ws[0][m + a:m + b], ws[1][m + a:m + b], k, E2M1).T)
        out[:, a:b] = y
    return out


def _exact_quant(case, s):
    k, fmt = case["k"], case["fmt"]
    bits, low = (1, 0) if fmt == E2M1 else (3, -6)           # mantissa bits, least exponent
    top = 6.0 if fmt == E2M1 else 448.0
    out = torch.empty(case["rows"], k, dtype=torch.float64, device="cuda")
    step = max(1, 2 ** 24 // k)
    for at in range(0, case["rows"], step):
        x = s["x"][at:at + step, :k].double().reshape(-1, 32)
        big = x.abs().max(1, keepdim=True).values
        e = torch.frexp(big).exponent.double() - 1.0         # 2^e <= big < 2^(e + 1)
        size = torch.exp2(torch.where(big > 0, e - EMAX[fmt], torch.full_like(e, -127.0)).clamp(min=-127.0))
        v = x / size
        ulp = torch.exp2((torch.frexp(v).exponent.double() - 1.0).clamp(min=low) - bits)
        out[at:at + step] = ((v / ulp).round() * ulp).clamp(-top, top).mul(size).reshape(-1, k)
    return out


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "quant":
        return _exact_quant(case, s)
    if op == "gemm":
        return _exact_rows(s["x"], s["w"], case["m"], case["k"], case["fmt"], case["silu"])
    if op == "experts":
        out = torch.empty(case["rows"] * case["top"], case["m"], dtype=torch.float64, device="cuda")
        row = s["order"].long() // case["top"] if case["gather"] else torch.arange(case["rows"] * case["top"], device="cuda")
        at, wide = 0, case["m"] * (1 + case["silu"])
        for e, n in enumerate(s["counts"]):
            if n:
                mine = row[at:at + n]
                out[at:at + n] = _exact_rows([t[mine] for t in s["x"]], [t[e * wide:(e + 1) * wide] for t in s["w"]], case["m"], case["k"],
                                             case["fmt"], case["silu"])
            at += n
        return out
    if op == "combine":
        rows = []
        for a in range(0, case["rows"], 512):
            at, w = s["slots"][a:a + 512].long(), s["weights"][a:a + 512].double()
            y = s["y"][at.clamp(min=0).reshape(-1)].double().reshape(*at.shape, case["m"])
            rows.append((torch.where(at >= 0, w, torch.zeros_like(w))[..., None] * y).sum(1))
        return torch.cat(rows)
    x = s["x"][:, :case["experts"]].double()
    value = torch.sort(x, dim=1, descending=True, stable=True).values[:, :case["top"]]
    total = torch.logsumexp(value if case["renorm"] else x, 1, keepdim=True)
    weights = torch.where(value == -INF, torch.zeros_like(value), torch.exp(value - total))
    return dict(ids=None, weights=weights, offsets=None, order=None, slots=None)
