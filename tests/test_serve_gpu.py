"""GPU parity of the serving-step operators against their plain forms
(serve_ref: numpy, 64 bits), through the C ABI: the page plan and the cache's
bytes exactly, attention and log probabilities within bounds derived from the
float32 arithmetic of the operators' definitions.

Bounds. Attention: a score is a float32 sum of terms whose sizes add up to
`amp`, and each weight 2^(f x - R) has a rounded argument: relative error of
a weight at most 2^-21 (1 + amp). The output is a sum of weighted terms of
total size `spread` over the sum of the weights, each carrying that error
once, plus 2^-24 for each of the float32 additions along a sum (one in 16
tokens of a row is an addition a lane makes). bfloat16 adds the rounding of
the result (2^-9, taken as 2^-8) and of the weights to binary16 (2^-12, taken
as 2^-11). Log probabilities: sums of float32 exponentials of rounded
arguments, 2^-20 beside 2^-22 of the value.
"""
import numpy as np
import pytest

import gemm_qgemv_amd as q
import serve_ref as ref
from gemm_qgemv_amd import tensors

pytestmark = pytest.mark.gpu
GUARD = 32


def say(*a):
    print(*a, flush=True)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "these tests need the GPU"
    return t


def dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Guarded:
    """A device buffer with guard bands around it."""

    def __init__(self, torch, n, dtype, fill=77):
        self.n, self.fill = n, fill
        self.full = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")
        self.t = self.full[GUARD:GUARD + n]

    def numpy(self):
        f = self.full.float().cpu().numpy() if self.full.is_floating_point() else self.full.cpu().numpy()
        assert np.all(f[:GUARD] == self.fill) and np.all(f[GUARD + self.n:] == self.fill), "guard band overwritten"
        return f[GUARD:GUARD + self.n]


# --- the page plan -------------------------------------------------------------

def run_plan(torch, old, keep, new, page, table, ring, state, total):
    B = len(old)
    tab, rng_ = Guarded(torch, table.size, torch.int32), Guarded(torch, ring.size, torch.int32)
    tab.t.copy_(dev(torch, table.reshape(-1)))
    rng_.t.copy_(dev(torch, ring))
    o = {n: Guarded(torch, k, torch.int32) for n, k in (("kv_len", B), ("cu_q", B + 1), ("slots", total), ("pos", total), ("denied", 1))}
    state_out = torch.full((2,), -5, dtype=torch.int64, device="cuda")
    i32 = np.int32
    # twice: the same inputs plan the same step
    for _ in range(2):
        q.qkv_plan(dev(torch, np.asarray(old, i32)), dev(torch, np.asarray(keep, i32)), dev(torch, np.asarray(new, i32)), B, page,
                   tab.t, table.shape[1], rng_.t, ring.size, dev(torch, np.asarray(state, np.int64)), state_out,
                   o["kv_len"].t, o["cu_q"].t, o["slots"].t, o["pos"].t, total, o["denied"].t)
        torch.cuda.synchronize()
    got = {n: g.numpy() for n, g in o.items()}
    got.update(table=tab.numpy().reshape(table.shape), ring=rng_.numpy(), state=state_out.cpu().numpy())
    return got


def check_plan(torch, *args):
    got, want = run_plan(torch, *args), ref.plan(*args)
    for n in want:
        assert np.array_equal(got[n], want[n]), (n, got[n], want[n])
    return want


def plan_case(rng, B, page, width, spare, growth):
    old = rng.integers(0, width * page + 1, size=B)
    keep = old.copy()
    back = rng.random(B) < 0.3
    keep[back] -= np.minimum(keep[back], rng.integers(0, 3 * page, size=back.sum()))
    new = rng.integers(0, growth + 1, size=B)
    ended = rng.random(B) < 0.15
    keep[ended], new[ended] = 0, 0
    have = -(-old // page)
    used = int(have.sum())
    cap = used + spare
    perm = rng.permutation(cap).astype(np.int32)
    table = np.full((B, width), -9, np.int32)
    n = 0
    for b in range(B):
        table[b, :have[b]] = perm[n:n + have[b]]
        n += have[b]
    head = int(rng.integers(0, 10 * cap + 1))
    ring = np.full(cap, -3, np.int32)
    for i in range(spare):
        ring[(head + i) % cap] = perm[used + i]
    return old, keep, new, page, table, ring, [head, head + spare], int(new.sum())


@pytest.mark.parametrize("B,page,width,spare,growth", [
    (1, 16, 4, 3, 20), (3, 1, 9, 5, 3), (64, 16, 32, 40, 1), (64, 16, 32, 0, 30), (257, 32, 8, 100, 60), (1000, 64, 3, 2000, 200),
    (2500, 16, 5, 700, 8)])
def test_plan(torch, B, page, width, spare, growth):
    rng = np.random.default_rng([7, B, page])
    for k in range(3):
        say("plan", B, page, k)
        args = plan_case(rng, B, page, width, spare, growth)
        check_plan(torch, *args)
        # room for more tokens than there are, and for fewer
        check_plan(torch, *args[:-1], args[-1] + 37)
        check_plan(torch, *args[:-1], args[-1] // 2)


def test_plan_contents_out_of_range(torch):
    """Lengths below 0, keep past the length, lengths past the table, a ring
    count below 0: taken as the header says, nothing outside written."""
    table = np.arange(12, dtype=np.int32).reshape(4, 3)
    ring = np.arange(100, 116, dtype=np.int32)
    check_plan(torch, [-5, 40, 3, 5], [7, 99, -2, 5], [2, 0, -1, 4], 4, table, ring, [5, 13], 12)
    check_plan(torch, [4, 4, 0, 1], [4, 4, 0, 1], [3, 9, 5, 1], 4, table, ring, [9, 4], 18)
    check_plan(torch, [0, 0, 0, 0], [0, 0, 0, 0], [0, 0, 0, 0], 4, table, ring, [-7, -2], 0)


def test_plan_serves_a_whole_run(torch):
    """Forty steps of requests that come, grow and end: no page is held
    twice, none is lost, slots lie in the pages held."""
    rng = np.random.default_rng(11)
    page, width, cap, B = 4, 6, 40, 9
    table, ring, state = np.full((B, width), -1, np.int32), np.arange(cap, dtype=np.int32), [0, cap]
    length = np.zeros(B, np.int64)
    for step in range(40):
        keep, new = length.copy(), rng.integers(0, 6, size=B)
        end = rng.random(B) < 0.15
        keep[end], new[end] = 0, 0
        total = int(new.sum())
        w = check_plan(torch, length, keep, new, page, table, ring, state, total)
        table, ring, state, length = w["table"], w["ring"], w["state"].tolist(), w["kv_len"].astype(np.int64)
        held = [int(p) for b in range(B) for p in table[b, :-(-length[b] // page)]]
        free = [int(ring[i % cap]) for i in range(state[0], state[1])]
        assert sorted(held + free) == list(range(cap)), step


# --- append and read -------------------------------------------------------------

def make_rows(rng, n, H, D):
    """Rows whose groups hit the quantizer's corners."""
    x = rng.standard_normal((n, H * D)).astype(np.float32) * np.exp(rng.normal(0, 1, (n, H * D // 64))).repeat(64, 1).astype(np.float32)
    x += rng.normal(0, 2, (n, H * D // 64)).repeat(64, 1).astype(np.float32)
    for i in range(n):
        g = slice((i % (H * D // 64)) * 64, (i % (H * D // 64)) * 64 + 64)
        kind = i % 11
        if kind == 1: x[i, g] = 1.25                                        # noqa: E701
        elif kind == 2: x[i, g] = 0.0                                       # noqa: E701
        elif kind == 3: x[i, g.start + 5] = np.nan                          # noqa: E701
        elif kind == 4: x[i, g.start + 63] = np.inf                         # noqa: E701
        elif kind == 5: x[i, g] *= np.float32(1e-38)                        # noqa: E701
        elif kind == 6: x[i, g] = np.float32(3.3e38) * np.sign(x[i, g])     # noqa: E701
        elif kind == 7: x[i, g] = rng.integers(-15, 16, 64)                 # noqa: E701  halves between codes
        elif kind == 8: x[i, g] = -0.0                                      # noqa: E701
        elif kind == 9: x[i, g] = 1e6 + rng.integers(0, 3, 64)              # noqa: E701  a range below the bias's steps
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,H,D,page,pad", [(1, 1, 64, 16, 0), (33, 5, 64, 32, 8), (60, 2, 128, 16, 16), (45, 3, 256, 64, 0),
                                            (23, 16, 256, 16, 8), (200, 1, 128, 128, 64)])
def test_append_and_read(torch, dtype, n, H, D, page, pad):
    say("append", dtype, n, H, D, page, pad)
    rng = np.random.default_rng([3, n, H, D])
    pages = n // page + 3
    k, v = make_rows(rng, n, H, D), make_rows(rng, n, H, D)[::-1].copy()
    W = H * D + pad
    dt, td = (q.QG_F32, torch.float32) if dtype == "f32" else (q.QG_BF16, torch.bfloat16)
    rows = []
    for x in (k, v):
        t = torch.full((n, W), float("nan"), dtype=td, device="cuda")
        t[:, :H * D] = dev(torch, x).to(td)
        rows.append(t)
    k, v = (t[:, :H * D].float().cpu().numpy() for t in rows)
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    if n > 3:
        slots[1], slots[2] = -1, pages * page
        slots[3] = 2 ** 31 - 1
    start = rng.integers(0, 256, size=(pages, H, ref.block_bytes(page, D)), dtype=np.uint8)
    buf = Guarded(torch, start.size, torch.uint8)
    buf.t.copy_(dev(torch, start.reshape(-1)))
    cache = q.KVCache(buf.t, pages, page, H, D)
    q.qkv_append(dt, rows[0], W, rows[1], W, dev(torch, slots), n, cache)
    torch.cuda.synchronize()
    want = start.copy()
    ref.append(want, page, H, D, k, v, slots)
    assert np.array_equal(buf.numpy().reshape(want.shape), want)

    ok, ov = Guarded(torch, n * W, td), Guarded(torch, n * W, td)
    q.qkv_read(dt, cache, dev(torch, slots), n, ok.t, W, ov.t, W)
    only = Guarded(torch, n * W, td)
    q.qkv_read(dt, cache, dev(torch, slots), n, None, 0, only.t, W)
    torch.cuda.synchronize()
    for part, g in ((0, ok), (1, ov), (1, only)):
        got = g.numpy().reshape(n, W)
        assert np.all(got[:, H * D:] == 77)
        w = torch.from_numpy(ref.read(want, page, H, D, slots, part)).to(td).float().numpy()
        assert np.array_equal(got[:, :H * D], w, equal_nan=True)


def test_append_scales_between_bf16_numbers(torch):
    """Ranges of 15 times the middle of two bf16 numbers: the product with 1/15
    may lie on either side of the middle, and decides."""
    rng = np.random.default_rng(15)
    n, page = 512, 64
    middle = (256 + np.arange(1, 256, 2)) / 256.0                          # 9 significant bits, the last one set
    x = rng.random((n, 64)).astype(np.float32)
    x[:, 0], x[:, 63] = 0.0, np.tile(15 * middle, 4) * np.repeat(2.0 ** np.array([-9, -1, 0, 20]), 128)
    x[:, 1:63] *= x[:, 63:]
    cache = q.KVCache(torch.zeros(n // page * ref.block_bytes(page, 64), dtype=torch.uint8, device="cuda"), n // page, page, 1, 64)
    t, slots = dev(torch, x), np.arange(n, dtype=np.int32)
    q.qkv_append(q.QG_F32, t, 64, t, 64, dev(torch, slots), n, cache)
    torch.cuda.synchronize()
    data = cache.data.cpu().numpy().reshape(n // page, 1, -1)
    want = np.zeros_like(data)
    ref.append(want, page, 1, 64, x, x, slots)
    assert np.array_equal(data, want)
    _, mid, end = ref.parts(page, 64, 0)
    scales = np.ascontiguousarray(data[:, 0, mid:end]).view("<u2")[:, ::2].reshape(-1)
    assert np.array_equal(scales, (t[:, 63] / 15.0).bfloat16().view(torch.int16).cpu().numpy().view(np.uint16))


def test_append_slots_past_2_gib(torch):
    """A cache of 4.8 GB: byte offsets past 32 bits, the last slot included."""
    page, H, D = 256, 8, 256
    pages = 4100 * 2
    data = torch.zeros(pages * H * ref.block_bytes(page, D) // 1, dtype=torch.uint8, device="cuda")
    assert data.numel() > 2 ** 32
    cache = q.KVCache(data, pages, page, H, D)
    x = torch.randn(4, H * D, device="cuda")
    slots = torch.tensor([0, pages * page - 1, pages * page // 2 + 3, 5], dtype=torch.int32, device="cuda")
    q.qkv_append(q.QG_F32, x, H * D, x, H * D, slots, 4, cache)
    k, v = torch.empty_like(x), torch.empty_like(x)
    q.qkv_read(q.QG_F32, cache, slots, 4, k, H * D, v, H * D)
    torch.cuda.synchronize()
    assert torch.equal(k, v)
    step = (x.reshape(4, H * 4, 64).amax(-1) - x.reshape(4, H * 4, 64).amin(-1)) / 15
    assert ((k - x).abs().reshape(4, H * 4, 64).amax(-1) <= 0.6 * step + 0.02).all()
    # attention over a context that lies in the last pages
    table = torch.arange(pages - 2, pages, dtype=torch.int32, device="cuda").reshape(1, 2)
    data.view(pages, -1)[-2:] = 0
    q.qkv_append(q.QG_F32, x, H * D, x, H * D, torch.arange(4, dtype=torch.int32, device="cuda") + (pages - 2) * page, 4, cache)
    out = torch.empty(1, H * D, device="cuda")
    q.qkv_attn(q.QG_F32, x[3:], H * D, cache, table, 2, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
               torch.tensor([1], dtype=torch.int32, device="cuda"), 1, 1, 1, 1, H, 0.1, 0, out, H * D)
    torch.cuda.synchronize()
    assert torch.allclose(out[0], v[0], rtol=1e-5, atol=1e-5)


# --- attention -------------------------------------------------------------------

class AttnCase:
    def __init__(self, torch, dtype, H, G, D, page, lens, window=0, seed=0, pad=0, tame=1.0):
        rng = np.random.default_rng([5, D, page, seed])
        self.torch, self.H, self.G, self.D, self.page, self.window = torch, H, G, D, page, window
        self.dt, self.td = (q.QG_F32, torch.float32) if dtype == "f32" else (q.QG_BF16, torch.bfloat16)
        self.lens, self.B = lens, len(lens)
        self.kv_len = np.array([kv for kv, _ in lens], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
        self.total = int(self.cu[-1])
        self.max_kv = max(1, int(self.kv_len.max()))
        self.width = -(-self.max_kv // page) + 1
        used = [-(-kv // page) for kv in self.kv_len]
        self.pages = sum(used) + 3
        perm = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((self.B, self.width), 2 ** 30, np.int32)        # unused entries: nonsense
        self.data = rng.integers(0, 256, size=(self.pages, H, ref.block_bytes(page, D)), dtype=np.uint8)
        for part in range(2):                                               # unwritten places: NaN coefficients
            _, mid, end = ref.parts(page, D, part)
            self.data[:, :, mid:end] = 0xFF
        n = 0
        for b, kv in enumerate(self.kv_len):
            self.table[b, :used[b]] = perm[n:n + used[b]]
            n += used[b]
            slots = [int(self.table[b, j // page]) * page + j % page for j in range(kv)]
            x = rng.standard_normal((2, kv, H * D)).astype(np.float32)
            x[0] += rng.normal(0, 1, H * D).astype(np.float32)
            ref.append(self.data, page, H, D, x[0], x[1], slots)
        self.scale = tame / np.sqrt(D)
        self.Hq, self.W = H * G, H * G * D + pad
        qq = rng.standard_normal((self.total, self.Hq * D)).astype(np.float32) * 1.5
        self.q = torch.zeros(self.total, self.W, dtype=self.td, device="cuda")
        self.q[:, :self.Hq * D] = dev(torch, qq).to(self.td)

    def run(self, ws_fill=None, stream=None, max_q=None, max_kv=None, data=None, table=None, lse=True):
        torch = self.torch
        self.cache = q.KVCache(dev(torch, self.data if data is None else data), self.pages, self.page, self.H, self.D)
        max_q = max_q or max(1, max(n for _, n in self.lens))
        max_kv = max_kv or self.max_kv
        out, l = Guarded(torch, self.total * self.W, self.td), Guarded(torch, self.total * self.Hq, torch.float32)
        need = q.qkv_attn_workspace_bytes(self.cache, self.B, self.total, max_q, max_kv, self.Hq)
        ws = torch.full((need,), ws_fill if ws_fill is not None else 0xFF, dtype=torch.uint8, device="cuda") if need else None
        args = (dev(torch, self.table if table is None else table), dev(torch, self.cu), dev(torch, self.kv_len))
        torch.cuda.synchronize()
        q.qkv_attn(self.dt, self.q, self.W, self.cache, args[0], self.width, args[1], args[2], self.B, self.total, max_q, max_kv,
                   self.Hq, self.scale, self.window, out.t, self.W, l.t if lse else None, ws, stream=stream)
        torch.cuda.synchronize()
        o = out.numpy().reshape(self.total, self.W)
        assert np.all(o[:, self.Hq * self.D:] == 77), "written between the rows"
        self.splits = need > 0
        return o[:, :self.Hq * self.D].reshape(self.total, self.Hq, self.D), l.numpy().reshape(self.total, self.Hq)

    def want(self):
        x = self.q[:, :self.Hq * self.D].double().cpu().numpy().reshape(self.total, self.Hq, self.D)
        return ref.attn(x, self.data, self.page, self.H, self.D, self.table, self.cu, self.kv_len, self.scale, self.window)

    def check(self, got=None):
        out, lse = got or self.run()
        o, l, spread, amp = self.want()
        kv = float(self.kv_len.max())
        tol = spread * (2.0 ** -21 * 2 * (1 + amp[..., None]) + 2.0 ** -24 * (kv / 16 + 16))
        if self.dt == q.QG_BF16:
            tol = tol + 2.0 ** -8 * np.abs(o) + 2.0 ** -11 * spread
        bad = ~(np.abs(out - o) <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(out - o) / np.maximum(tol, 1e-30))}, first {np.argwhere(bad)[0]}"
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(lse), empty)
        assert np.all(np.abs(lse - l)[~empty] <= (2.0 ** -20 * (1 + amp) + 2.0 ** -22 * np.abs(l))[~empty])


LENS = {
    "one": [(1, 1)],
    "edges": [(15, 1), (16, 1), (17, 1), (63, 1), (64, 1), (65, 1), (255, 1), (256, 1), (257, 1)],
    "decode": [(701, 1), (3, 1), (130, 1)],
    "empty": [(0, 1), (40, 0), (33, 1), (0, 0), (2, 5)],
    "verify": [(300, 5), (7, 7), (129, 2), (64, 3)],
    "prompt": [(150, 150), (77, 20), (1, 1)],
    "chunk": [(333, 70)],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,G,D,page", [(1, 1, 64, 16), (2, 4, 64, 32), (1, 8, 128, 16), (2, 3, 128, 64), (1, 2, 256, 32),
                                        (1, 16, 64, 128), (1, 5, 256, 16)])
@pytest.mark.parametrize("lens", list(LENS))
def test_attention(torch, dtype, H, G, D, page, lens):
    say("attention", dtype, H, G, D, page, lens)
    AttnCase(torch, dtype, H, G, D, page, LENS[lens]).check()


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200])
@pytest.mark.parametrize("H,G,D,page,lens", [(1, 4, 64, 16, "decode"), (2, 2, 128, 32, "verify"), (1, 3, 128, 16, "prompt"),
                                             (1, 2, 256, 64, "chunk"), (1, 20, 64, 16, "edges")])
def test_attention_window(torch, window, H, G, D, page, lens):
    say("window", window, D, lens)
    AttnCase(torch, "f32", H, G, D, page, LENS[lens], window=window).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,G,D,lens", [(1, 7, 64, [(2300, 1)]), (1, 30, 128, [(1500, 1), (900, 1)]), (1, 16, 64, [(1200, 3), (10, 1)]),
                                        (1, 8, 128, [(1100, 40)]), (1, 4, 256, [(1300, 2)])])
def test_attention_split_tokens(torch, dtype, H, G, D, lens):
    """Few rows and many tokens: split over workgroups and joined."""
    say("split", dtype, D, lens)
    c = AttnCase(torch, dtype, H, G, D, 16, lens)
    got = c.run()
    assert c.splits
    c.check(got)
    again = c.run(ws_fill=0)
    assert np.array_equal(again[0], got[0]) and np.array_equal(again[1], got[1])


def test_attention_strides_and_hints(torch):
    """Rows that are parts of wider ones; max_q below the longest request and
    sizes above the real ones give the same values within the bound."""
    c = AttnCase(torch, "f32", 2, 3, 64, 16, LENS["verify"], pad=40)
    c.check()
    c.check(c.run(max_q=1))
    c.check(c.run(max_q=200))
    c.check(c.run(max_kv=c.width * 16))
    out, _ = c.run(lse=False)
    assert np.array_equal(out, c.run()[0])
    AttnCase(torch, "bf16", 1, 4, 128, 16, LENS["chunk"], pad=8).check()


def test_attention_large_scores(torch):
    """Scores of some hundreds: weights that underflow, a reference that moves
    often; and a query of zeros (uniform weights)."""
    AttnCase(torch, "f32", 1, 4, 64, 16, LENS["decode"], tame=60.0).check()
    AttnCase(torch, "f32", 1, 4, 128, 16, LENS["prompt"], tame=30.0).check()
    c = AttnCase(torch, "f32", 1, 4, 64, 16, LENS["decode"])
    c.q[0] = 0
    c.check()
    c.q *= 1e-25
    c.check()
    c.q *= 1e-15      # subnormal queries
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,G,D", [(1, 2, 64), (1, 8, 128), (1, 3, 256)])
def test_attention_what_is_masked_does_not_matter(torch, dtype, H, G, D):
    """NaN and infinite coefficients at token j reach the rows that see it,
    and change no bit of the others."""
    lens = [(90, 40)]
    c = AttnCase(torch, dtype, H, G, D, 16, lens)
    clean, clean_lse = c.run()
    for j, word in ((70, 0x7FC0), (55, 0x7F80), (89, 0xFF80)):
        d = c.data.copy()
        slot = int(c.table[0, j // 16]) * 16 + j % 16
        for part in range(2):
            _, mid, _ = ref.parts(16, D, part)
            at = mid + (slot % 16) * (D // 64) * 4
            d[slot // 16, :, at:at + (D // 64) * 4] = np.array([word] * (D // 64 * 2), "<u2").view(np.uint8)
        out, lse = c.run(data=d)
        sees = np.arange(50, 90) >= j
        assert np.array_equal(out[~sees], clean[~sees]) and np.array_equal(lse[~sees], clean_lse[~sees])
        assert np.isnan(out[sees]).all()


def test_attention_window_hides_what_it_masks(torch):
    """A token that left the window may be anything."""
    c = AttnCase(torch, "f32", 1, 4, 64, 16, [(100, 1), (80, 20)], window=10)
    clean = c.run()[0]
    d = c.data.copy()
    for b, j in ((0, 89), (0, 64), (1, 50)):
        slot = int(c.table[b, j // 16]) * 16 + j % 16
        for part in range(2):
            _, mid, _ = ref.parts(16, 64, part)
            d[slot // 16, :, mid + (slot % 16) * 4:mid + (slot % 16) * 4 + 4] = 0xFF
    assert np.array_equal(c.run(data=d)[0], clean)


def test_attention_contents_out_of_range(torch):
    """A length past max_kv and page numbers outside the cache give NaN in the
    rows concerned and leave the others as they are."""
    c = AttnCase(torch, "f32", 1, 4, 64, 16, [(40, 1), (200, 1), (60, 1)])
    clean, _ = c.run()
    t = c.table.copy()
    t[2, 1] = -1
    out, lse = c.run(table=t)
    assert np.array_equal(out[:2], clean[:2]) and np.isnan(out[2]).all() and np.isnan(lse[2]).all()
    t[2, 1] = c.pages
    assert np.isnan(c.run(table=t)[0][2]).all()
    out, lse = c.run(max_kv=100)
    assert np.isnan(out[1]).all() and np.isnan(lse[1]).all() and np.isfinite(out[[0, 2]]).all()
    c.kv_len[0] = -3
    out, lse = c.run()
    assert np.all(out[0] == 0) and np.isneginf(lse[0]).all()
    # row starts that are not in order or past the batch: no rows, or no fault
    c.cu = np.array([0, 5, 1, 9], np.int32)
    c.run()
    c.cu = np.array([-4, 1, 2, 3], np.int32)
    assert np.array_equal(c.run()[0][1], clean[1])


def test_attention_nan_query(torch):
    c = AttnCase(torch, "f32", 1, 4, 64, 16, LENS["verify"])
    clean, _ = c.run()
    c.q[2, 64:128] = float("nan")
    c.q[4, 5] = float("inf")
    out, _ = c.run()
    assert np.isnan(out[2, 1]).all() and np.isnan(out[4, 0]).all()
    keep = np.ones(clean.shape[:2], bool)
    keep[2, 1] = keep[4, 0] = False
    assert np.array_equal(out[keep], clean[keep])


def test_attention_on_another_stream_and_in_a_graph(torch):
    for lens in (LENS["prompt"], [(1400, 1)]):
        c = AttnCase(torch, "f32", 1, 4, 64, 16, lens)
        want, want_lse = c.run()
        side = torch.cuda.Stream()
        assert np.array_equal(c.run(stream=side)[0], want)
        out, lse = torch.zeros(c.total, c.W, device="cuda"), torch.zeros(c.total, c.Hq, device="cuda")
        ws = tensors.attn_workspace(c.cache, c.B, c.total, max(n for _, n in lens), c.max_kv, c.Hq)
        args = (dev(torch, c.table), dev(torch, c.cu), dev(torch, c.kv_len))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q.qkv_attn(c.dt, c.q, c.W, c.cache, args[0], c.width, args[1], args[2], c.B, c.total, max(n for _, n in lens), c.max_kv,
                       c.Hq, c.scale, 0, out, c.W, lse, ws)
        for _ in range(3):
            out.zero_()
            lse.zero_()
            if ws is not None:
                ws.fill_(255)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(out.cpu().numpy().reshape(want.shape), want)
            assert np.array_equal(lse.cpu().numpy(), want_lse)


# --- log probabilities -------------------------------------------------------------

def run_logprobs(torch, x, ids, top, ld=None, skew=0, stream=None):
    R, M = x.shape
    ld = ld or M
    buf = torch.full((skew + R * ld + 8,), float("nan"), device="cuda")
    view = buf[skew:skew + R * ld].view(R, ld)
    view[:, :M] = dev(torch, x)
    o = dict(lp=Guarded(torch, R, torch.float32), ent=Guarded(torch, R, torch.float32), rank=Guarded(torch, R, torch.int32))
    if top:
        o.update(tid=Guarded(torch, R * top, torch.int32), tlp=Guarded(torch, R * top, torch.float32))
    ws = tensors.logprobs_workspace(R, M, top)
    if ws is not None:
        ws.fill_(255)
    idd = dev(torch, np.asarray(ids, np.int32))
    torch.cuda.synchronize()
    q.qlogprobs(view, ld, R, M, idd, top, o["lp"].t, o["ent"].t, o["rank"].t, o["tid"].t if top else None,
                o["tlp"].t if top else None, ws, stream=stream)
    torch.cuda.synchronize()
    tid = o["tid"].numpy().reshape(R, top) if top else np.zeros((R, 0), np.int32)
    tlp = o["tlp"].numpy().reshape(R, top) if top else np.zeros((R, 0), np.float32)
    return o["lp"].numpy(), o["ent"].numpy(), o["rank"].numpy(), tid, tlp


def check_logprobs(torch, x, ids, top, **kw):
    got = run_logprobs(torch, x, ids, top, **kw)
    want = ref.logprobs(x, ids, top)
    sane = ~np.isnan(want[1])
    for i, n in ((0, "logprob"), (1, "entropy"), (4, "top_logprobs")):
        g, w = got[i], want[i]
        assert np.array_equal(np.isnan(g), np.isnan(w)), (n, g, w)
        assert np.array_equal(np.isneginf(g), np.isneginf(w)), n
        f = np.isfinite(w)
        assert np.all(np.abs(g[f] - w[f]) <= 2.0 ** -20 + 2.0 ** -22 * np.abs(w[f])), (n, np.abs(g[f] - w[f]).max())
    inside = np.array([0 <= i < x.shape[1] for i in ids])
    assert np.array_equal(got[2][sane & inside], want[2][sane & inside])
    assert np.all(got[2][~inside] == 0)
    assert np.array_equal(got[3][sane], want[3][sane])
    return got


@pytest.mark.parametrize("M,ld,skew", [(1, 1, 0), (2, 3, 1), (3, 3, 3), (63, 64, 0), (257, 257, 2), (1023, 1025, 1), (1024, 1024, 0),
                                       (4096, 4096, 0), (5001, 5004, 0), (16390, 16391, 3)])
@pytest.mark.parametrize("top", [0, 1, 5, 64])
def test_logprobs(torch, M, ld, skew, top):
    say("logprobs", M, ld, skew, top)
    rng = np.random.default_rng([9, M, top])
    R = 5
    x = (rng.standard_normal((R, M)) * rng.choice([0.1, 3, 20], (R, 1))).astype(np.float32)
    ids = np.array([0, M - 1, rng.integers(0, M), -1, M])
    check_logprobs(torch, x, ids, min(top, M), ld=ld, skew=skew)


def test_logprobs_ties_and_masks(torch):
    """Equal logits come lowest index first; excluded tokens (-infinity, or
    the lowest finite value) take no part; rows without a distribution are
    NaN and do not disturb the others."""
    rng = np.random.default_rng(4)
    M = 9000
    x = np.zeros((12, M), np.float32)
    x[1] = rng.integers(0, 3, M)
    x[2] = np.where(rng.random(M) < 0.5, np.float32(-0.0), np.float32(0.0))
    x[3] = -np.inf
    x[3, 7000] = 2.0
    x[4] = -np.inf
    x[5] = np.where(rng.random(M) < 0.99, -np.inf, 1.0)
    x[6] = np.float32(-3.4028235e38)
    x[7] = np.float32(-3.4028235e38)
    x[7, 5:9] = [1, 2, 3, 3]
    x[8, 100] = np.nan
    x[9, 8999] = np.inf
    x[10] = rng.standard_normal(M)
    x[10, ::2] = -np.inf
    x[11] = np.arange(M) * 1e-3
    ids = np.array([4500, 8000, 17, 7000, 3, 100, 8999, 8, 100, 8999, 4, 0])
    got = check_logprobs(torch, x, ids, 64)
    assert got[3][0].tolist() == list(range(64)) and got[2][0] == 4501
    check_logprobs(torch, x[::-1].copy(), ids[::-1], 3, skew=1, ld=M + 1)
    # a given token that is excluded
    lp = check_logprobs(torch, x[10:11], [6], 2)
    assert np.isneginf(lp[0][0]) and lp[2][0] == 4503 + (6 // 2 + 1) - 3


def test_logprobs_many_rows_and_descending_values(torch):
    """Rows whose best values come last, first, or all in one lane's share."""
    rng = np.random.default_rng(8)
    M = 12345
    x = rng.standard_normal((40, M)).astype(np.float32)
    x[0] = np.sort(x[0])
    x[1] = np.sort(x[1])[::-1]
    x[2, 64:64 + 64 * 16:16] += 50
    x[3, 1024:1088] += 50
    x[4, :4] += 50
    x[5, -5:] += 50
    for top in (1, 20, 33):
        check_logprobs(torch, x, rng.integers(0, M, 40), top)


def test_logprobs_rows_far_apart(torch):
    """Row offsets past 32 bits."""
    M, ld = 1000, (1 << 31) + 4
    buf = torch.empty(ld + M, device="cuda")
    a, b = torch.randn(M, device="cuda"), torch.randn(M, device="cuda")
    buf[:M], buf[ld:ld + M] = a, b
    out = [torch.empty(2, device="cuda") for _ in range(2)]
    ws = tensors.logprobs_workspace(2, M, 0)
    q.qlogprobs(buf, ld, 2, M, torch.tensor([1, 2], dtype=torch.int32, device="cuda"), 0, out[0], out[1], None, None, None, ws)
    torch.cuda.synchronize()
    w = ref.logprobs(np.stack([a.cpu().numpy(), b.cpu().numpy()]), [1, 2], 0)
    assert np.allclose(out[0].cpu().numpy(), w[0], atol=1e-5) and np.allclose(out[1].cpu().numpy(), w[1], atol=1e-5)


def test_logprobs_optional_outputs(torch):
    x = torch.randn(3, 777, device="cuda")
    ent = torch.empty(3, device="cuda")
    ws = tensors.logprobs_workspace(3, 777, 0)
    q.qlogprobs(x, 777, 3, 777, None, 0, None, ent, None, None, None, ws)
    torch.cuda.synchronize()
    p = torch.softmax(x.double(), -1)
    assert torch.allclose(ent.double(), -(p * p.log()).sum(-1), atol=1e-5)


def test_logprobs_repeat_on_another_stream_and_in_a_graph(torch):
    rng = np.random.default_rng(2)
    x, ids = rng.standard_normal((2, 60000)).astype(np.float32), [5, 70]
    want = run_logprobs(torch, x, ids, 8)
    for a, b in zip(want, run_logprobs(torch, x, ids, 8, stream=torch.cuda.Stream())):
        assert np.array_equal(a, b)
    xd, idd = dev(torch, x), dev(torch, np.asarray(ids, np.int32))
    o = [torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
         torch.zeros(2, 8, dtype=torch.int32, device="cuda"), torch.zeros(2, 8, device="cuda")]
    ws = tensors.logprobs_workspace(2, 60000, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlogprobs(xd, 60000, 2, 60000, idd, 8, *o, ws)
    for _ in range(3):
        for t in o:
            t.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, t in zip(want, o):
            assert np.array_equal(a, t.cpu().numpy())
