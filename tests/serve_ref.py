"""Plain reference forms of the serving-step operators, in numpy: loops and
64-bit arithmetic, written from include/qg.h alone. Test infrastructure."""
import numpy as np


def bf16_bits(x):
    """Nearest-even bf16 bits of float32 values (finite or not)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32)
    nan = (u & 0x7FFFFFFF) > 0x7F800000
    return np.where(nan, 0x7FC0, r).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


# --- the cache -------------------------------------------------------------

def block_bytes(page, D):
    return page * (D + D // 8)


def parts(page, D, part):
    """Byte ranges of a block's codes and coefficients, K (0) or V (1)."""
    lo = part * block_bytes(page, D) // 2
    return lo, lo + page * D // 2, lo + page * D // 2 + page * (D // 64) * 4


def quantize(x):
    """One group of 64 float32 values -> (codes uint8[64], scale bits, bias bits)."""
    x = np.asarray(x, np.float32)
    if not np.all(np.isfinite(x)):
        return np.zeros(64, np.uint8), 0x7FC0, 0x7FC0
    with np.errstate(over="ignore"):
        s_bits = int(bf16_bits(np.float32(np.float32(x.max() - x.min()) * np.float32(1 / 15)))[0])
        b_bits = int(bf16_bits(np.float32(x.min()))[0])
    if (s_bits & 0x7F80) == 0x7F80 or (b_bits & 0x7F80) == 0x7F80:
        return np.zeros(64, np.uint8), 0x7FC0, 0x7FC0
    if (s_bits & 0x7F80) == 0:
        return np.zeros(64, np.uint8), 0, b_bits
    s, b = bf16_value(s_bits), bf16_value(b_bits)
    with np.errstate(over="ignore"):
        q = np.rint(((x - b).astype(np.float32) / s).astype(np.float32))
    return np.clip(q, 0, 15).astype(np.uint8), s_bits, b_bits


def append(data, page, H, D, k, v, slots):
    """data uint8 [num_pages][H][block], in place; k, v float32 [n][H*D]."""
    for t, slot in enumerate(slots):
        if slot < 0 or slot // page >= data.shape[0]:
            continue
        for part, rows in enumerate((k, v)):
            lo, mid, _ = parts(page, D, part)
            for h in range(H):
                blk = data[slot // page, h]
                at = slot % page
                for g in range(D // 64):
                    codes, sb, bb = quantize(rows[t, h * D + g * 64:h * D + g * 64 + 64])
                    blk[lo + at * D // 2 + g * 32:lo + at * D // 2 + g * 32 + 32] = codes[0::2] | (codes[1::2] << 4)
                    c = mid + (at * (D // 64) + g) * 4
                    blk[c:c + 4] = np.array([sb, bb], "<u2").view(np.uint8)


def slot_values(data, page, D, part, slot, h, bound=False):
    """float64 values [D] a slot's head stands for; with `bound`, instead the
    sizes of the terms they are summed from, 8 |scale| + |bias + 8 scale|."""
    lo, mid, _ = parts(page, D, part)
    blk, at = data[slot // page, h], slot % page
    byte = blk[lo + at * D // 2:lo + (at + 1) * D // 2]
    code = np.stack([byte & 15, byte >> 4], -1).reshape(D).astype(np.float64)
    co = bf16_value(np.ascontiguousarray(blk[mid + at * (D // 64) * 4:mid + (at + 1) * (D // 64) * 4]).view("<u2")).astype(np.float64)
    co = co.reshape(D // 64, 2)
    if bound:
        return np.repeat(8 * np.abs(co[:, 0]) + np.abs(co[:, 1] + 8 * co[:, 0]), 64)
    return np.repeat(co[:, 0], 64) * code + np.repeat(co[:, 1], 64)


def read(data, page, H, D, slots, part):
    """float32 rows of qkv_read."""
    out = np.full((len(slots), H * D), np.nan, np.float32)
    for t, slot in enumerate(slots):
        if 0 <= slot and slot // page < data.shape[0]:
            out[t] = np.concatenate([slot_values(data, page, D, part, slot, h) for h in range(H)]).astype(np.float32)
    return out


# --- attention ---------------------------------------------------------------

def attn(q, data, page, H, D, table, cu, kv_len, scale, window):
    """q float64 [total][Hq][D] -> out, lse, spread, amp (float64): what error
    bounds scale with, the sizes of the terms of the output (spread) and of
    the largest score (amp)."""
    total, Hq = q.shape[:2]
    G = Hq // H
    out = np.zeros((total, Hq, D))
    lse = np.full((total, Hq), -np.inf)
    spread = np.zeros((total, Hq, D))
    amp = np.zeros((total, Hq))
    for b in range(len(kv_len)):
        n, kv = cu[b + 1] - cu[b], kv_len[b]
        if n == 0:
            continue
        slots = [int(table[b, j // page]) * page + j % page for j in range(kv)]
        for h in range(H):
            K = np.array([slot_values(data, page, D, 0, s, h) for s in slots]).reshape(kv, D)
            V = np.array([slot_values(data, page, D, 1, s, h) for s in slots]).reshape(kv, D)
            KB = np.array([slot_values(data, page, D, 0, s, h, True) for s in slots]).reshape(kv, D)
            VB = np.array([slot_values(data, page, D, 1, s, h, True) for s in slots]).reshape(kv, D)
            for i in range(n):
                p = kv - n + i
                lo = max(0, p - window + 1) if window else 0
                if p < 0 or lo > p:
                    continue
                k, v = K[lo:p + 1], V[lo:p + 1]
                for g in range(G):
                    x = q[cu[b] + i, h * G + g]
                    s = (k @ x) * scale
                    m = s.max()
                    w = np.exp(s - m)
                    z = w.sum()
                    out[cu[b] + i, h * G + g] = (w @ v) / z
                    lse[cu[b] + i, h * G + g] = m + np.log(z)
                    spread[cu[b] + i, h * G + g] = (w @ VB[lo:p + 1]) / z
                    amp[cu[b] + i, h * G + g] = (KB[lo:p + 1] @ np.abs(x)).max() * scale
    return out, lse, spread, amp


# --- the page plan -----------------------------------------------------------

def plan(old, keep, new, page, table, ring, state, total):
    """Sequential form of qkv_plan; returns copies of everything it writes."""
    table, ring = table.copy(), ring.copy()
    B, width = table.shape
    cap = len(ring)
    head, tail = int(state[0]), int(state[1])
    free = min(max(tail - head, 0), cap)
    ceil = lambda a: -(-a // page)                    # noqa: E731
    clamp = lambda a, hi: max(0, min(int(a), hi))     # noqa: E731
    kv, cu, slots, pos = [], [0], [], []
    wanted, took, gave, denied = 0, 0, 0, 0
    writes = []
    for b in range(B):
        o = clamp(old[b], 1 << 30)
        k, n = clamp(keep[b], o), clamp(new[b], 1 << 30)
        have, want = min(ceil(o), width), ceil(k + n)
        grow = max(0, want - have) if want <= width else 0
        wanted += grow
        ok = want <= width and (grow == 0 or wanted <= free)
        after = want if ok else min(ceil(k), width)
        pages = [int(table[b, c]) for c in range(have)]
        if ok:
            for c in range(have, want):
                page_no = int(ring[(head + took) % cap])
                table[b, c] = page_no
                pages.append(page_no)
                took += 1
        else:
            denied += 1
        for c in range(after, have):
            writes.append(((tail + gave) % cap, pages[c]))
            gave += 1
        kv.append(k + n if ok else k)
        cu.append(cu[-1] + n)
        for i in range(n):
            if len(slots) >= total:
                break
            slots.append(pages[(k + i) // page] * page + (k + i) % page if ok else -1)
            pos.append(k + i)
    for at, v in writes:
        ring[at] = v
    slots += [-1] * (total - len(slots))
    pos += [-1] * (total - len(pos))
    i32 = np.int32
    return dict(table=table, ring=ring, state=np.array([head + took, tail + gave]), kv_len=np.array(kv, i32),
                cu_q=np.array(cu, i32), slots=np.array(slots[:total], i32), pos=np.array(pos[:total], i32),
                denied=np.array([denied], i32))


# --- token log probabilities ---------------------------------------------------

def logprobs(x, ids, top):
    """x float32 [rows][vocab]: logprob, entropy, rank, top_ids, top_logprobs."""
    rows, M = x.shape
    lp, ent, rank = np.full(rows, np.nan), np.full(rows, np.nan), np.zeros(rows, np.int32)
    tid, tlp = np.zeros((rows, top), np.int32), np.full((rows, top), np.nan)
    for n in range(rows):
        r = x[n].astype(np.float64)
        order = sorted(range(M), key=lambda j: (-r[j], j)) if not np.isnan(r).any() else list(range(M))
        tid[n] = order[:top]
        i = int(ids[n])
        if 0 <= i < M:
            rank[n] = order.index(i) + 1
        if np.isnan(r).any() or np.isposinf(r).any() or np.isneginf(r).all():
            continue
        m = r.max()
        z = np.exp(r - m).sum()
        l = r - m - np.log(z)
        p = np.exp(l)
        ent[n] = -sum(a * b for a, b in zip(p, l) if a > 0)
        tlp[n] = l[order[:top]]
        if 0 <= i < M:
            lp[n] = l[i]
    return lp, ent, rank, tid, tlp
