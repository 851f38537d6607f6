"""Measured cases of the serving-step operators: the page plan, the 4-bit
key/value cache (append and read back), attention over that cache, and the
log probabilities of given tokens with entropy and top alternatives.

`run` computes each case in its plain form (elementary torch operations in 32
bits) or, where `own` is true, through the library's entry points. `exact`
gives the same outputs from the operators' definitions in 64 bits.

Cache layout (one page of one key/value head is one block of bytes):
codes of K [page][D/2], scale and bias of K bf16 [page][D/64][2], then the
same two parts for V; blocks are ordered [num_pages][kv_heads]. Code k of a
row sits in byte k // 2, even k in the low nibble; value = scale * code + bias.
"""
import math
import random

import numpy as np
import torch

own = False

F32, BF16 = "f32", "bf16"
DT = {F32: torch.float32, BF16: torch.bfloat16}
INF = float("inf")


def listed():
    return [
        # one decode step of a 64-request batch: a few requests need a page,
        # a few have ended and give theirs back (latency)
        dict(name="plan_decode_64", op="plan", batch=64, page=16, max_len=8192, tokens=64, pool=40000, mode="decode"),
        # admission of new prompts beside 400 running requests
        dict(name="plan_prompts_512", op="plan", batch=512, page=16, max_len=16384, tokens=65536, pool=400000, mode="mixed"),
        # the new token of each of 64 requests written to the cache, and read back
        dict(name="append_decode_64", op="append", dtype=F32, tokens=64, kv_heads=8, dim=128, page=16, pages=4096, pad=0),
        # a chunk of prompt tokens, keys and values being parts of wider rows
        dict(name="append_prompt_16411", op="append", dtype=BF16, tokens=16411, kv_heads=8, dim=128, page=64, pages=300, pad=64),
        # a single request, short context, 64-wide heads (latency)
        dict(name="decode_1x701", op="attn", dtype=F32, batch=1, q_heads=32, kv_heads=4, dim=64, page=16, new=1,
             max_kv=701, window=0, ragged=0),
        # a single request, long context: the keys split over the chip
        dict(name="decode_1x131071", op="attn", dtype=F32, batch=1, q_heads=32, kv_heads=8, dim=128, page=64, new=1,
             max_kv=131071, window=0, ragged=0),
        # a batch of decoding requests of mixed lengths
        dict(name="decode_64x8192_ragged", op="attn", dtype=BF16, batch=64, q_heads=32, kv_heads=8, dim=128, page=16, new=1,
             max_kv=8192, window=0, ragged=1),
        # five speculated tokens a request checked at once, wide heads, a sliding window
        dict(name="verify_16x6000_window", op="attn", dtype=F32, batch=16, q_heads=16, kv_heads=2, dim=256, page=32, new=5,
             max_kv=6000, window=4096, ragged=1),
        # a chunk of 2048 prompt tokens after 8192 cached ones
        dict(name="prompt_2048_after_8192", op="attn", dtype=F32, batch=1, q_heads=32, kv_heads=8, dim=128, page=64, new=2048,
             max_kv=10240, window=0, ragged=0),
        # several prompts of mixed lengths, nothing cached before
        dict(name="prompts_6x4001_ragged", op="attn", dtype=BF16, batch=6, q_heads=32, kv_heads=4, dim=64, page=16, new=4001,
             max_kv=4001, window=0, ragged=1),
        # the sampled token of one request, with the 20 best alternatives
        dict(name="logprob_1x151936", op="logprob", rows=1, vocab=151936, top=20, pad=0, masked=0),
        # a prompt's tokens scored
        dict(name="logprob_1024x151936", op="logprob", rows=1024, vocab=151936, top=5, pad=0, masked=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "logprob"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        batch = _log_int(rng, 1, 600)
        mode = rng.choice(["decode", "mixed"])
        tokens = batch if mode == "decode" else _log_int(rng, max(batch, 64), 65536)
        return dict(op=op, batch=batch, page=page, max_len=rng.choice([4096, 8192, 16384]), tokens=tokens,
                    pool=600000, mode=mode)
    if op == "append":
        tokens = _log_int(rng, 1, 16000)
        return dict(op=op, dtype=rng.choice([F32, BF16]), tokens=tokens, kv_heads=rng.choice([1, 2, 4, 5, 8]),
                    dim=rng.choice([64, 128, 256]), page=page, pages=tokens // page + 40, pad=rng.choice([0, 8, 64]))
    if op == "logprob":
        return dict(op=op, rows=_log_int(rng, 1, 700), vocab=_log_int(rng, 1000, 200000), top=rng.choice([0, 1, 5, 20, 32]),
                    pad=rng.choice([0, 0, 3, 64]), masked=rng.choice([0, 1]))
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    while kv_heads * group > 64:
        group = max(1, group // 2)
    kind = rng.choice(["decode", "verify", "prompt"])
    if kind == "decode":
        new, batch, max_kv = 1, _log_int(rng, 1, 64), _log_int(rng, 1, 16000)
    elif kind == "verify":
        new, batch, max_kv = rng.randint(2, 9), _log_int(rng, 1, 32), _log_int(rng, 16, 12000)
    else:
        new, batch = _log_int(rng, 17, 2048), rng.randint(1, 4)
        max_kv = new + rng.choice([0, _log_int(rng, 1, 4000)])
    heads = kv_heads * group
    while batch > 1 and batch * heads * dim * new * max_kv > 128 * 32 * 2048 * 6000:
        batch -= 1
    while batch > 1 and batch * max_kv * kv_heads * dim > 64 * 8192 * 8 * 128:
        batch -= 1
    while heads * dim * new * max_kv > 128 * 32 * 2048 * 6000 and group > 1:
        group //= 2
        heads = kv_heads * group
    return dict(op="attn", dtype=rng.choice([F32, BF16]), batch=batch, q_heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                new=new, max_kv=max_kv, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), ragged=rng.choice([0, 1]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """(tokens in the cache with the new ones, new tokens) of each request: a
    property of the case, the same for every seed."""
    r = random.Random("%(batch)d %(max_kv)d %(new)d" % case)
    lens = []
    for b in range(case["batch"]):
        if b == 0 or not case["ragged"]:
            kv, n = case["max_kv"], case["new"]
        else:
            n = case["new"] if case["new"] < 10 else r.randint(max(1, case["new"] // 8), case["new"])
            kv = r.randint(case["max_kv"] // 8, case["max_kv"])
            kv = max(kv, n) if case["max_kv"] > case["new"] else n
            n = min(n, kv)
        lens.append((kv, min(n, kv)))
    return lens


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _block_bytes(case):
    return case["page"] * case["dim"] + case["page"] * (case["dim"] // 64) * 8


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _prepare_plan(case, seed):
    r = np.random.default_rng([int(seed), 5])
    B, page, width = case["batch"], case["page"], case["max_len"] // case["page"]
    old = r.integers(1, case["max_len"] * 3 // 4, size=B)
    keep, new = old.copy(), np.ones(B, np.int64)
    if case["mode"] == "mixed":
        prompts = r.random(B) < 0.2
        old[prompts], keep[prompts] = 0, 0
        room = max(0, case["tokens"] - B)
        share = r.random(B) * prompts
        new += np.minimum((room * share / max(share.sum(), 1e-9)).astype(np.int64), case["max_len"] - 2)
        keep -= np.minimum(keep, r.integers(0, 5, size=B) * (r.random(B) < 0.3))     # rejected speculation
    ended = r.random(B) < 0.06
    keep[ended], new[ended] = 0, 0
    have = -(-old // page)
    perm = r.permutation(case["pool"]).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = np.cumsum(have) - have
    cols = np.arange(width)
    mine = cols[None, :] < have[:, None]
    table[mine] = perm[(at[:, None] + cols[None, :])[mine]]
    used = int(have.sum())
    ring = np.roll(np.concatenate([perm[used:], np.full(used, -1, np.int32)]), 12345)
    head = 12345 + 3 * case["pool"]
    s = dict(case=case, old=_ints(old), keep=_ints(keep), new=_ints(new), table=_ints(table), ring=_ints(ring),
             state=_ints([head, head + case["pool"] - used], torch.int64))
    return s


def _prepare_append(case, seed):
    g = _gen(seed)
    T, H, D = case["tokens"], case["kv_heads"], case["dim"]
    wide = H * D + case["pad"]
    spread = torch.exp(0.5 * torch.randn(H * D, generator=g, device="cuda"))
    middle = 2.0 * torch.randn(H * D, generator=g, device="cuda")
    kv = []
    for _ in range(2):
        t = torch.zeros(T, wide, dtype=DT[case["dtype"]], device="cuda")
        t[:, :H * D] = torch.randn(T, H * D, generator=g, device="cuda") * spread + middle
        kv.append(t)
    slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:T].to(torch.int32)
    data = torch.zeros(case["pages"] * H * _block_bytes(case), dtype=torch.uint8, device="cuda")
    return dict(case=case, k=kv[0], v=kv[1], slots=slots, data=data)


def _bits16(x):
    """bf16 bit patterns (int16) of float32 values."""
    return x.to(torch.bfloat16).view(torch.int16)


def _prepare_attn(case, seed):
    g = _gen(seed)
    D, H, page, G = case["dim"], case["kv_heads"], case["page"], case["q_heads"] // case["kv_heads"]
    lens = _lengths(case)
    width = -(-case["max_kv"] // page)
    used = [-(-kv // page) for kv, _ in lens]
    pages = sum(used) + 7
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    # keys and values as quantizing real ones leaves them: a bell of codes in
    # each group of 64, scales and minima that go with it
    data = torch.empty(pages, H, _block_bytes(case), dtype=torch.uint8, device="cuda")
    n_code, n_coef = page * D // 2, page * (D // 64) * 4
    for part in range(2):
        lo = part * (n_code + n_coef)
        z = torch.randn(pages, H, n_code, generator=g, device="cuda").mul_(2.9).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        y = torch.randn(pages, H, n_code, generator=g, device="cuda").mul_(2.9).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        data[:, :, lo:lo + n_code] = z | (y << 4)
        del z, y
        s = 0.15 + 0.3 * torch.rand(pages, H, n_coef // 4, generator=g, device="cuda")
        b = -7.5 * s + 0.4 * torch.randn(pages, H, n_coef // 4, generator=g, device="cuda")
        co = torch.stack([_bits16(s), _bits16(b)], -1).reshape(pages, H, n_coef // 2).contiguous()
        data[:, :, lo + n_code:lo + n_code + n_coef] = co.view(torch.uint8)
    # what is behind a request's last token in its last page is left over from
    # other requests, or was never written: any bits
    for b, (kv, _) in enumerate(lens):
        if kv % page:
            blk, tail = data[int(perm[sum(used[:b + 1]) - 1])], page - kv % page
            for part in range(2):
                lo = part * (n_code + n_coef) + n_code
                blk[:, lo + (page - tail) * (D // 64) * 4:lo + n_coef] = 0xFF
    starts = np.concatenate([[0], np.cumsum([n for _, n in lens])])
    total = int(starts[-1])
    q = torch.randn(total, case["q_heads"], D, generator=g, device="cuda") * 1.2
    return dict(case=case, q=q.to(DT[case["dtype"]]), data=data, table=table, cu_q=_ints(starts), kv_len=_ints([kv for kv, _ in lens]),
                total=total, pages=pages, scale=1.0 / math.sqrt(D), max_q=max(n for _, n in lens))


def _prepare_logprob(case, seed):
    g = _gen(seed)
    R, M = case["rows"], case["vocab"]
    buf = torch.empty(R, M + case["pad"], device="cuda")
    buf.normal_(generator=g).mul_(2.3)
    peaks = torch.randint(0, M, (R, 40), generator=g, device="cuda")
    buf.scatter_add_(1, peaks, torch.rand(R, 40, generator=g, device="cuda") * 12)
    if case["masked"]:     # part of the vocabulary excluded, as by a grammar
        gone = torch.randint(0, M, (R, max(1, M // 50)), generator=g, device="cuda")
        buf.scatter_(1, gone, -INF)
    ids = torch.where(torch.rand(R, generator=g, device="cuda") < 0.7, peaks[:, 0],
                      torch.randint(0, M, (R,), generator=g, device="cuda")).to(torch.int32)
    return dict(case=case, logits=buf, ids=ids)


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn,
            "logprob": _prepare_logprob}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_plan(s):
    """Pages and slots from lengths. Requests that shrink put their last pages
    behind the free ones of the ring; requests that grow take free pages from
    its front, in request order, as long as the pages that were free before
    the call last; a request that gets none keeps `keep` tokens."""
    c = s["case"]
    page, width = c["page"], s["table"].shape[1]
    cap, T = s["ring"].numel(), c["tokens"]
    old, keep, new = s["old"].long(), s["keep"].long(), s["new"].long()
    head, tail = s["state"][0], s["state"][1]
    have, want = (old + page - 1) // page, (keep + new + page - 1) // page
    grow = torch.where(want <= width, (want - have).clamp(min=0), torch.zeros_like(have))
    granted = (want <= width) & ((grow == 0) | (grow.cumsum(0) <= tail - head))
    after = torch.where(granted, want, (keep + page - 1) // page)
    take = torch.where(granted, grow, torch.zeros_like(grow))
    take_at = take.cumsum(0) - take
    give = (have - after).clamp(min=0)
    give_at = give.cumsum(0) - give
    cols = torch.arange(width, device="cuda")[None, :]
    fresh = (cols >= have[:, None]) & (cols < after[:, None])
    from_ring = s["ring"][(head + take_at[:, None] + cols - have[:, None]) % cap]
    table = torch.where(fresh, from_ring, s["table"])
    freed = (cols >= after[:, None]) & (cols < have[:, None])
    to = torch.where(freed, (tail + give_at[:, None] + cols - after[:, None]) % cap, torch.full_like(cols, cap))
    ring = torch.cat([s["ring"], s["ring"][:1]]).scatter(0, to.reshape(-1), s["table"].reshape(-1))[:cap]
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=old.numel() - 1)
    pos = keep[b] + t - cu[b]
    real = t < cu[-1]
    at = table[b, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    none = torch.full_like(pos, -1)
    return dict(table=table, ring=ring, state=torch.stack([head + take.sum(), tail + give.sum()]),
                kv_len=torch.where(granted, keep + new, keep).int(), cu_q=cu.int(),
                slots=torch.where(real & granted[b], at, none).int(), pos=torch.where(real, pos, none).int(),
                denied=(~granted).sum().int().reshape(1))


def _plain_quantize(x):
    """x float32 [..., 64]: bf16 scale and bias (as float32) and codes (as
    float32) of each group: scale (max - min) / 15 and bias min, both rounded
    to bf16, codes against the rounded ones."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).to(torch.bfloat16).float()
    b = lo.to(torch.bfloat16).float()
    flat = s < 2.0 ** -126
    code = ((x - b) / torch.where(flat, torch.full_like(s, INF), s)).round().clamp(0, 15)
    return torch.where(flat, torch.zeros_like(s), s), b, code


def _plain_append(s):
    """Each token's keys and values put into its slot's place in the cache,
    then read back (what a slot stands for, in float32)."""
    c = s["case"]
    T, H, D, page = c["tokens"], c["kv_heads"], c["dim"], c["page"]
    n_code, n_coef = page * D // 2, page * (D // 64) * 4
    data = s["data"].view(c["pages"], H, _block_bytes(c))
    slots = s["slots"].long()
    pg, off = (slots // page)[:, None, None], (slots % page)[:, None, None]
    heads = torch.arange(H, device="cuda")[None, :, None]
    out = {}
    for part, name in enumerate(("k", "v")):
        x = s[name][:, :H * D].float().reshape(T, H, D // 64, 64)
        sc, bi, code = _plain_quantize(x)
        u = code.to(torch.uint8).reshape(T, H, D // 2, 2)
        lo = part * (n_code + n_coef)
        at_code = lo + off * (D // 2) + torch.arange(D // 2, device="cuda")
        at_coef = lo + n_code + off * (D // 16) + torch.arange(D // 16, device="cuda")
        data[pg, heads, at_code] = u[..., 0] | (u[..., 1] << 4)
        coef = torch.stack([_bits16(sc), _bits16(bi)], -1).reshape(T, H, D // 32).contiguous().view(torch.uint8)
        data[pg, heads, at_coef] = coef
        byte = data[pg, heads, at_code]
        back = torch.stack([byte & 15, byte >> 4], -1).float().reshape(T, H, D // 64, 64)
        co = data[pg, heads, at_coef].view(torch.bfloat16).float().reshape(T, H, D // 64, 2)
        out[name] = (co[..., :1] * back + co[..., 1:]).reshape(T, H * D)
    return out


def _cache_values(s, part, table, double=False):
    """Values [batch][kv_heads][positions][D] that the pages of `table`
    [batch][width] stand for (entries outside the cache read as page 0)."""
    c = s["case"]
    D, page, H = c["dim"], c["page"], c["kv_heads"]
    n_code, n_coef = page * D // 2, page * (D // 64) * 4
    lo = part * (n_code + n_coef)
    B, W = table.shape
    blk = s["data"][table.clamp(min=0).long().reshape(-1)]
    byte = blk[:, :, lo:lo + n_code]
    co = blk[:, :, lo + n_code:lo + n_code + n_coef].contiguous().view(torch.bfloat16).float().reshape(B * W, H, page, D // 64, 2)
    code = torch.stack([byte & 15, byte >> 4], -1).float().reshape(B * W, H, page, D // 64, 64)
    if double:
        co, code = co.double(), code.double()
    x = (code * co[..., :1] + co[..., 1:]).reshape(B, W, H, page, D)
    return x.transpose(1, 2).reshape(B, H, W * page, D)


def _plain_attn(s):
    c = s["case"]
    D, H, Hq = c["dim"], c["kv_heads"], c["q_heads"]
    G, B, N = Hq // H, c["batch"], s["max_q"]
    k, v = (_cache_values(s, part, s["table"]) for part in range(2))
    L = k.shape[2]
    cu, kv_len = s["cu_q"].long(), s["kv_len"].long()
    n_q = cu[1:] - cu[:-1]
    i = torch.arange(N, device="cuda")
    row = (cu[:-1, None] + i[None, :]).clamp(max=s["total"] - 1)
    q = s["q"].float()[row]                                                        # [B][N][Hq][D]
    q = q.reshape(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    j = torch.arange(L, device="cuda")
    dead = (j[None, :] >= kv_len[:, None])[:, None, :, None]
    k = torch.where(dead, torch.zeros((), device="cuda"), k)
    v = torch.where(dead, torch.zeros((), device="cuda"), v)
    at = (kv_len - n_q)[:, None] + i[None, :]                                       # position of each new token
    seen = (j[None, None, :] <= at[:, :, None]) & (j[None, None, :] < kv_len[:, None, None])
    if c["window"]:
        seen = seen & (j[None, None, :] > at[:, :, None] - c["window"])
    seen = seen[:, None, :, None, :].expand(B, 1, N, G, L).reshape(B, 1, N * G, L)
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    x = x.masked_fill_(~seen, -INF)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == -INF, torch.zeros_like(m), m)
    x = x.sub_(m0).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(z == 0, torch.ones_like(z), z)
    lse = (m0 + torch.log(z)).reshape(B, H, N, G).permute(0, 2, 1, 3).reshape(B, N, Hq)
    o = o.reshape(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return dict(out=o[b, t - cu[b]].to(s["q"].dtype), lse=lse[b, t - cu[b]])


def _plain_logprob(s):
    c = s["case"]
    M, top = c["vocab"], c["top"]
    x = s["logits"][:, :M]
    ids = s["ids"].long()[:, None]
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = d.exp()
    z = e.sum(-1, keepdim=True)
    lse = (m + z.log())
    given = x.gather(1, ids)
    j = torch.arange(M, device="cuda")[None, :]
    out = dict(logprob=(given - lse)[:, 0],
               entropy=(z.log() - torch.where(e == 0, e, e * d).sum(-1, keepdim=True) / z)[:, 0],
               rank=(1 + ((x > given) | ((x == given) & (j < ids))).sum(-1)).int())
    if top:
        bits = (x + 0.0).contiguous().view(torch.int32).long()
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)                      # as signed, in the values' order
        best = torch.topk(order * (1 << 32) + (0xFFFFFFFF - j), top, dim=-1).values
        at = 0xFFFFFFFF - (best & 0xFFFFFFFF)
        out.update(top_ids=at.int(), top_logprobs=x.gather(1, at) - lse)
    return out


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


def _own_plan(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    B, T = c["batch"], c["tokens"]
    o = _once(s, "out", lambda: dict(state=_empty(2, dtype=torch.int64), kv_len=_empty(B, dtype=torch.int32),
                                     cu_q=_empty(B + 1, dtype=torch.int32), slots=_empty(T, dtype=torch.int32),
                                     pos=_empty(T, dtype=torch.int32), denied=_empty(1, dtype=torch.int32)))
    q.qkv_plan(s["old"], s["keep"], s["new"], B, c["page"], s["table"], s["table"].shape[1], s["ring"], s["ring"].numel(),
               s["state"], o["state"], o["kv_len"], o["cu_q"], o["slots"], o["pos"], T, o["denied"])
    return dict(o, table=s["table"], ring=s["ring"])


def _own_append(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    T, H, D = c["tokens"], c["kv_heads"], c["dim"]
    dt = q.QG_F32 if c["dtype"] == F32 else q.QG_BF16
    cache = _once(s, "cache", lambda: q.KVCache(s["data"], c["pages"], c["page"], H, D))
    k, v = _once(s, "back", lambda: (_empty(T, H * D), _empty(T, H * D)))
    q.qkv_append(dt, s["k"], H * D + c["pad"], s["v"], H * D + c["pad"], s["slots"], T, cache)
    q.qkv_read(q.QG_F32, cache, s["slots"], T, k, H * D, v, H * D)
    return dict(k=k, v=v)


def _own_attn(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    B, Hq, D, T = c["batch"], c["q_heads"], c["dim"], s["total"]
    dt = q.QG_F32 if c["dtype"] == F32 else q.QG_BF16
    cache = _once(s, "cache", lambda: q.KVCache(s["data"], s["pages"], c["page"], c["kv_heads"], D))
    need = _once(s, "need", lambda: q.qkv_attn_workspace_bytes(cache, B, T, s["max_q"], c["max_kv"], Hq))
    ws = _once(s, "ws", lambda: _empty(need, dtype=torch.uint8) if need else None)
    out, lse = _once(s, "out", lambda: (_empty(T, Hq, D, dtype=DT[c["dtype"]]), _empty(T, Hq)))
    q.qkv_attn(dt, s["q"], Hq * D, cache, s["table"], s["table"].shape[1], s["cu_q"], s["kv_len"], B, T, s["max_q"], c["max_kv"],
               Hq, s["scale"], c["window"], out, Hq * D, lse, ws)
    return dict(out=out, lse=lse)


def _own_logprob(s):
    import gemm_qgemv_amd as q
    c = s["case"]
    R, M, top = c["rows"], c["vocab"], c["top"]
    need = _once(s, "need", lambda: q.qlogprobs_workspace_bytes(R, M, top))
    ws = _once(s, "ws", lambda: _empty(need, dtype=torch.uint8) if need else None)

    def buffers():
        o = dict(logprob=_empty(R), entropy=_empty(R), rank=_empty(R, dtype=torch.int32))
        if top:
            o.update(top_ids=_empty(R, top, dtype=torch.int32), top_logprobs=_empty(R, top))
        return o
    o = _once(s, "out", buffers)
    q.qlogprobs(s["logits"], M + c["pad"], R, M, s["ids"], top, o["logprob"], o["entropy"], o["rank"], o.get("top_ids"),
                o.get("top_logprobs"), ws)
    return o


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "attn": _own_attn, "logprob": _own_logprob}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn, "logprob": _plain_logprob}[op](state)


# ---------------------------------------------------------------------------
# Work and the definitions in 64 bits
# ---------------------------------------------------------------------------

def _pairs(case):
    """(query, key) pairs that a head looks at, and keys that any query of
    its request sees."""
    pairs, keys = 0, 0
    w = case["window"] or (1 << 60)
    for kv, n in _lengths(case):
        first = kv - n
        for_rows = np.minimum(np.arange(first + 1, kv + 1), w)
        pairs += int(for_rows.sum())
        keys += min(kv, n - 1 + w)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "plan":
        # lengths in, lengths and starts out, slots and positions out, about
        # one table entry read or written for each page of new tokens
        entries = max(case["batch"] // 16, case["tokens"] // case["page"])
        return {"bytes": case["batch"] * 20 + case["tokens"] * 8 + entries * 12 + 40, "flops": 4 * (case["batch"] + case["tokens"])}
    if op == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"] * 2
        return {"bytes": n * (4 if case["dtype"] == F32 else 2) + n * 9 // 16 * 2 + n * 4 + case["tokens"] * 8, "flops": 8 * n}
    if op == "attn":
        pairs, keys = _pairs(case)
        rows = sum(n for _, n in _lengths(case))
        size = 4 if case["dtype"] == F32 else 2
        cache = keys * case["kv_heads"] * (case["dim"] + case["dim"] // 8)
        return {"bytes": cache + rows * case["q_heads"] * (case["dim"] * size * 2 + 4), "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    n = case["rows"] * case["vocab"]
    return {"bytes": 4 * n + case["rows"] * (16 + 8 * case["top"]), "flops": 8 * n}


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    T, H, D = case["tokens"], case["kv_heads"], case["dim"]
    out = {}
    for name in ("k", "v"):
        x = s[name][:, :H * D].double().reshape(-1, 64)
        lo, hi = x.min(1, keepdim=True).values, x.max(1, keepdim=True).values
        step = ((hi - lo).float() / 15).bfloat16().double()      # the stored scale is a bf16 number
        base = lo.bfloat16().double()
        code = torch.round((x - base) / torch.where(step > 0, step, torch.ones_like(step))).clamp(0, 15)
        out[name] = (base + step * code).reshape(T, H * D)
    return out


def _exact_attn(case, seed):
    pairs, _ = _pairs(case)
    if pairs * case["q_heads"] * case["dim"] > 4e11:
        return None
    s = _prepare_attn(case, seed)
    G = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["total"], case["q_heads"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], case["q_heads"], dtype=torch.float64, device="cuda")
    at = 0
    for b, (kv, n) in enumerate(_lengths(case)):
        width = -(-kv // case["page"])
        k = _cache_values(s, 0, s["table"][b:b + 1, :width], True)[0, :, :kv]
        v = _cache_values(s, 1, s["table"][b:b + 1, :width], True)[0, :, :kv]
        pos = torch.arange(kv - n, kv, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None, :]
        hide = j > pos
        if case["window"]:
            hide = hide | (j <= pos - case["window"])
        for h in range(case["q_heads"]):
            x = (s["q"][at:at + n, h].double() @ k[h // G].T) * s["scale"]
            x = x.masked_fill(hide, -INF)
            lse[at:at + n, h] = torch.logsumexp(x, -1)
            out[at:at + n, h] = torch.softmax(x, -1) @ v[h // G]
        at += n
    return dict(out=out, lse=lse)


def _exact_logprob(case, seed):
    s = _prepare_logprob(case, seed)
    M, rows = case["vocab"], []
    for r in range(0, case["rows"], 64):
        x = s["logits"][r:r + 64, :M].double()
        lp = x - torch.logsumexp(x, 1, keepdim=True)
        ent = -torch.where(lp == -INF, torch.zeros_like(lp), lp.exp() * lp).sum(1)
        best = torch.sort(lp, dim=1, descending=True, stable=True).values[:, :case["top"]]
        rows.append((lp.gather(1, s["ids"][r:r + 64].long()[:, None])[:, 0], ent, best))
    out = dict(logprob=torch.cat([r[0] for r in rows]), entropy=torch.cat([r[1] for r in rows]), rank=None)
    if case["top"]:
        out.update(top_ids=None, top_logprobs=torch.cat([r[2] for r in rows]))
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None          # whole numbers only
    return {"append": _exact_append, "attn": _exact_attn, "logprob": _exact_logprob}[case["op"]](case, seed)
