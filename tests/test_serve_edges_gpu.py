"""GPU tests of the serving-step operators at the edges of their contents and
sizes: row starts out of order, requests cut off by the call's row count, value
scales far apart, page numbers past 32-bit slots, interleaved read-back.
References and bounds are those of test_serve_gpu.py."""
import numpy as np
import pytest

import gemm_qgemv_amd as q
import serve_ref as ref
from gemm_qgemv_amd import tensors
from test_serve_gpu import AttnCase, Guarded, dev, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "these tests need the GPU"
    return t


# --- row starts --------------------------------------------------------------------

@pytest.mark.parametrize("cu", [[50, 100, 0, 0], [100, 0, 50, 100], [0, 100, 30, 40], [90, 80, 70, 3], [-7, 300, 20, 60]])
@pytest.mark.parametrize("G,D,kv", [(3, 64, 60), (24, 128, 60), (3, 64, 1500)])
@pytest.mark.parametrize("max_q", [1, 50])
def test_attention_row_starts_out_of_order(torch, cu, G, D, kv, max_q):
    """No place outside the rows is written (the guard bands and the gaps of a
    head's width between the rows are looked at by run), and rows before the
    least and behind the last start stay as they were."""
    say("row starts", cu, G, D, kv, max_q)
    c = AttnCase(torch, "f32", 1, G, D, 16, [(kv, 50), (40, 50), (30, 0)], pad=D)
    c.cu = np.array(cu, np.int32)
    out, lse = c.run(max_q=max_q)
    inside = [min(max(s, 0), c.total) for s in cu]
    for lo, hi in ((0, min(inside)), (max(inside), c.total)):
        assert np.all(out[lo:hi] == 77) and np.all(lse[lo:hi] == 77)


@pytest.mark.parametrize("G,D,lens,cut", [(2, 64, [(40, 6), (30, 5)], 8), (8, 128, [(90, 3), (70, 40)], 25), (4, 64, [(1500, 3)], 2),
                                          (3, 256, [(60, 30)], 11), (24, 64, [(20, 1), (300, 100)], 61)])
@pytest.mark.parametrize("window", [0, 9])
def test_attention_rows_cut_off(torch, G, D, lens, cut, window):
    """A call with fewer rows than cu_q counts: the rows that exist stand for
    the same tokens as in the whole call."""
    say("cut off", G, D, lens, cut, window)
    c = AttnCase(torch, "f32", 1, G, D, 16, lens, window=window)
    o, l, spread, amp = c.want()
    c.total, c.q = cut, c.q[:cut].contiguous()
    out, lse = c.run()
    kv = float(c.kv_len.max())
    tol = spread * (2.0 ** -21 * 2 * (1 + amp[..., None]) + 2.0 ** -24 * (kv / 16 + 16))
    assert np.all(np.abs(out - o[:cut]) <= tol[:cut])
    assert np.all(np.abs(lse - l[:cut]) <= 2.0 ** -20 * (1 + amp[:cut]) + 2.0 ** -22 * np.abs(l[:cut]))


# --- the page plan -----------------------------------------------------------------

@pytest.mark.parametrize("page,number", [(16, 1 << 28), (1 << 20, 4096), (16, (1 << 28) + 1), (1 << 20, 2047), (256, 2 ** 31 - 1),
                                         (16, -(1 << 28)), (1 << 20, -2048), (4, -3)])
def test_plan_slots_past_32_bits(torch, page, number):
    """A page whose slots are no 32-bit numbers, in the table and in the ring:
    its tokens get slot -1, never the slot of another page."""
    say("plan slots", page, number)
    i32 = np.int32
    table = Guarded(torch, 4, torch.int32)
    table.t.copy_(dev(torch, np.array([number, -1, 5, -1], i32)))
    ring = dev(torch, np.array([number, 7], i32))
    o = {n: Guarded(torch, k, torch.int32) for n, k in (("kv_len", 2), ("cu_q", 3), ("slots", 6), ("pos", 6), ("denied", 1))}
    state_out = torch.zeros(2, dtype=torch.int64, device="cuda")
    q.qkv_plan(dev(torch, np.array([page - 2, page - 1], i32)), dev(torch, np.array([page - 2, page - 1], i32)),
               dev(torch, np.array([1, 3], i32)), 2, page, table.t, 2, ring, 2, torch.tensor([0, 2], device="cuda"), state_out,
               o["kv_len"].t, o["cu_q"].t, o["slots"].t, o["pos"].t, 6, o["denied"].t)
    torch.cuda.synchronize()

    def slot(number, at):
        v = number * page + at
        return v if -2 ** 31 <= v < 2 ** 31 else -1
    assert table.numpy().tolist() == [number, -1, 5, number]
    assert o["slots"].numpy().tolist() == [slot(number, page - 2), slot(5, page - 1), slot(number, 0), slot(number, 1), -1, -1]
    assert o["pos"].numpy().tolist() == [page - 2, page - 1, page, page + 1, -1, -1]
    assert o["denied"].numpy().tolist() == [0] and state_out.tolist() == [1, 2]


def test_plan_length_past_32_bits(torch):
    """The longest length kept and the most new tokens: their sum is no int32
    and is the largest one instead, as the row starts are."""
    page, width, most = 1 << 20, 2048, 1 << 30
    table = torch.arange(2 * width, dtype=torch.int32, device="cuda")
    ring = torch.arange(width, dtype=torch.int32, device="cuda") + 2 * width
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")     # noqa: E731
    kv_len, cu, slots, pos, denied = ints(0, 0), ints(0, 0, 0), ints(9, 9), ints(9, 9), ints(9)
    state_out = torch.zeros(2, dtype=torch.int64, device="cuda")
    q.qkv_plan(ints(most, 5), ints(most, 5), ints(most, most), 2, page, table, width, ring, width, torch.tensor([0, width], device="cuda"),
               state_out, kv_len, cu, slots, pos, 2, denied)
    torch.cuda.synchronize()
    # request 0 goes from 1024 to 2048 pages, request 1 from 1 to 1025: all that are free
    assert kv_len.tolist() == [2 ** 31 - 1, most + 5] and cu.tolist() == [0, most, 2 ** 31 - 1] and denied.tolist() == [0]
    assert state_out.tolist() == [width, width] and pos.tolist() == [most, most + 1]
    assert table[1024:2048].tolist() == ring[:1024].tolist()
    assert table[2049:3073].tolist() == ring[1024:].tolist()


# --- value scales far apart ----------------------------------------------------------

def scale_values(c, exponents, part=1):
    """Values (part 0: keys) of request b's token j, group g, times
    2^exponents(b, j, g): the stored bfloat16 scale and bias change by an exact
    power of two."""
    G = c.D // 64
    _, mid, _ = ref.parts(c.page, c.D, part)
    for b, kv in enumerate(c.kv_len):
        for j in range(kv):
            page, at = int(c.table[b, j // c.page]), j % c.page
            for h in range(c.H):
                co = np.ascontiguousarray(c.data[page, h, mid + at * G * 4:mid + (at + 1) * G * 4]).view("<u2")
                x = ref.bf16_value(co).astype(np.float64) * np.repeat([2.0 ** exponents(b, j, g) for g in range(G)], 2)
                c.data[page, h, mid + at * G * 4:mid + (at + 1) * G * 4] = ref.bf16_bits(x.astype(np.float32)).view(np.uint8)


def constant_values(c, which, value):
    """Values of the groups that which(b, j, g) names become `value`: scale 0."""
    G = c.D // 64
    _, mid, _ = ref.parts(c.page, c.D, 1)
    for b, kv in enumerate(c.kv_len):
        for j in range(kv):
            page, at = int(c.table[b, j // c.page]), j % c.page
            for g in range(G):
                if which(b, j, g):
                    o = mid + (at * G + g) * 4
                    c.data[page, :, o:o + 4] = np.array([0, ref.bf16_bits(np.array([value], np.float32))[0]], "<u2").view(np.uint8)


KINDS = ["few", "drafts", "rows", "prompt", "split"]


def value_case(torch, dtype, kind, D, **kw):
    H, G, lens = {"few": (2, 4, [(150, 1), (64, 1), (7, 1)]), "drafts": (1, 8, [(200, 3), (130, 4)]), "rows": (1, 6, [(170, 9), (90, 2)]),
                  "prompt": (1, 4, [(220, 60)]), "split": (1, 4, [(1500, 2)])}[kind]
    return AttnCase(torch, dtype, H, G, D, 16, lens, seed=3, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,apart", [(128, 10), (128, 20), (256, 14), (128, 40), (256, -30)])
def test_attention_value_groups_of_other_sizes(torch, dtype, kind, D, apart):
    """Every channel group keeps its bits, whatever the others' size (the bound
    of a channel is made of its own values)."""
    say("value groups", dtype, kind, D, apart)
    c = value_case(torch, dtype, kind, D)
    scale_values(c, lambda b, j, g: -apart if g & 1 else 0)
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,low,high,tame", [(64, 0, 12, 1.0), (64, -20, 20, 1.0), (128, -50, 50, 20.0), (256, 0, 30, 40.0)])
def test_attention_value_tokens_of_other_sizes(torch, dtype, kind, D, low, high, tame):
    """Tokens whose values differ by many binary orders, with weights that are
    alike (large values decide) and that are not."""
    say("value tokens", dtype, kind, D, low, high, tame)
    rng = np.random.default_rng(9)
    c = value_case(torch, dtype, kind, D, tame=tame)
    e = rng.integers(low, high + 1, size=(c.B, int(c.kv_len.max()), D // 64))
    scale_values(c, lambda b, j, g: int(e[b, j, g]))
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,size", [(64, 105), (128, 112), (64, 60), (128, -45), (256, -70), (64, -100)])
def test_attention_values_of_any_size(torch, dtype, kind, D, size):
    """Values that append stores and read-back returns as finite numbers."""
    say("value size", dtype, kind, D, size)
    c = value_case(torch, dtype, kind, D)
    scale_values(c, lambda b, j, g: size)
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_attention_constant_value_groups(torch, dtype, kind):
    """Groups of scale 0, everywhere, in some tokens, large and small ones;
    and a large value among them that has next to no weight."""
    say("constant values", dtype, kind)
    for D, which, value in ((128, lambda b, j, g: g == 1, 0.0), (128, lambda b, j, g: True, 3.0), (64, lambda b, j, g: True, 2.0 ** 100),
                            (256, lambda b, j, g: g == (j // 40) % 4, 1.0), (64, lambda b, j, g: j < 70, 0.0),
                            (128, lambda b, j, g: j >= 70 and g == 0, 2.0 ** 60)):
        c = value_case(torch, dtype, kind, D, tame=8.0)
        constant_values(c, which, value)
        c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [30, 110])
def test_attention_a_large_value_without_weight(torch, dtype, kind, size):
    """One token of far larger values whose score is far below the others':
    what it does not weigh it must not cost."""
    say("weightless", dtype, kind, size)
    c = value_case(torch, dtype, kind, 64)
    for b, kv in enumerate(c.kv_len):
        j = int(kv) // 3
        slot = int(c.table[b, j // 16]) * 16 + j % 16
        # its key, alike in all channels, is far from every query once these lean to one side
        k = np.full((1, c.H * 64), -40.0, np.float32)
        v = np.zeros((1, c.H * 64), np.float32)
        v[0, ::2] = 1.0
        ref.append(c.data, 16, c.H, 64, k, v, [slot])
    c.q[:, :c.Hq * 64] += 2.0
    scale_values(c, lambda b, j, g: size if j == int(c.kv_len[b]) // 3 else 0)
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,G,D,lens", [(1, 4, 128, [(900, 1), (640, 1)]), (1, 8, 64, [(800, 4)]), (1, 6, 256, [(700, 9)]), (1, 4, 64, [(800, 33)]),
                                        (1, 4, 128, [(700, 40)])])
@pytest.mark.parametrize("tame,window", [(1.0, 0), (25.0, 0), (4.0, 333)])
def test_attention_values_that_change_size_along_a_request(torch, dtype, H, G, D, lens, tame, window):
    """Runs of tokens whose values are alike, at sizes far apart, a few tokens
    of other sizes among them: kernels go from one way of taking tiles to the
    other and back."""
    say("runs", dtype, D, lens, tame, window)
    rng = np.random.default_rng(21)
    c = AttnCase(torch, dtype, H, G, D, 16, lens, seed=5, tame=tame, window=window)
    run = [0, -18, 14, 0, -33, 3, 40, -6]
    odd = rng.integers(-30, 30, size=2000) * (rng.random(2000) < 0.004)
    scale_values(c, lambda b, j, g: run[j // 131 % 8] + int(odd[j]) - 5 * (g & 1))
    c.check()


# --- more rows than one launch takes ---------------------------------------------------

def test_logprobs_of_more_rows_than_a_launch(torch):
    R = 2 ** 24 + 3
    x = torch.zeros(R, 2, device="cuda")
    x[:, 1] = torch.arange(R, device="cuda") % 7 - 3.0
    ids = torch.ones(R, dtype=torch.int32, device="cuda")
    lp, ent = torch.full((R + 8,), 77.0, device="cuda"), torch.empty(R, device="cuda")
    rank, tid = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    tlp = torch.empty(R, device="cuda")
    assert q.qlogprobs_workspace_bytes(R, 2, 1) == 0
    q.qlogprobs(x, 2, R, 2, ids, 1, lp, ent, rank, tid, tlp)
    torch.cuda.synchronize()
    d = x[:, 1].double()
    want = -torch.log1p(torch.exp(-d))
    assert ((lp[:R].double() - want).abs() <= 2.0 ** -20 + 2.0 ** -22 * want.abs()).all() and (lp[R:] == 77).all()
    assert torch.equal(rank, 1 + (d <= 0).int()) and torch.equal(tid, (d > 0).int())
    assert ((tlp.double() + torch.log1p(torch.exp(-d.abs()))).abs() <= 2.0 ** -20).all()
    p = torch.sigmoid(d)
    assert ((ent.double() + p * want + (1 - p) * -torch.log1p(torch.exp(d))).abs() <= 2.0 ** -20).all()


def test_append_and_read_of_more_tokens_than_a_launch(torch):
    """A token of 17 heads of 64 channels is a workgroup's (36 GB of bfloat16
    rows; nearly all slots lie outside the cache)."""
    H, D, page, n = 17, 64, 16, 2 ** 24 + 5
    W = H * D
    at = [0, 2 ** 24 - 2, 2 ** 24 - 1, 2 ** 24, n - 1]
    x = torch.empty(n, W, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for t in at:
        x[t] = torch.randn(W, generator=g, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[torch.tensor(at, device="cuda")] = torch.tensor([3, 17, 2, 31, 8], dtype=torch.int32, device="cuda")
    data = Guarded(torch, 2 * H * ref.block_bytes(page, D), torch.uint8)
    cache = q.KVCache(data.t, 2, page, H, D)
    q.qkv_append(q.QG_BF16, x, W, x, W, slots, n, cache)
    torch.cuda.synchronize()
    rows = torch.stack([x[t] for t in at]).float().cpu().numpy()
    want = np.full((2, H, ref.block_bytes(page, D)), 77, np.uint8)
    ref.append(want, page, H, D, rows, rows, [3, 17, 2, 31, 8])
    assert np.array_equal(data.numpy().reshape(want.shape), want)
    x.fill_(1.0)
    q.qkv_read(q.QG_BF16, cache, slots, n, None, 0, x, W)
    torch.cuda.synchronize()
    got = torch.stack([x[t] for t in at]).float().cpu().numpy()
    w = torch.from_numpy(ref.read(want, page, H, D, [3, 17, 2, 31, 8], 1)).bfloat16().float().numpy()
    assert np.array_equal(got, w)
    assert torch.isnan(x[1:n - 1:4099]).all() and torch.isnan(x[n - 2]).all()


# --- rows that are parts of wider ones ---------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,H,D,gap", [(1, 1, 64, 0), (37, 2, 128, 0), (50, 3, 64, 24), (9, 2, 256, 64)])
def test_read_into_parts_of_one_buffer(torch, dtype, n, H, D, gap):
    """Keys and values side by side in the rows of one buffer, as append takes
    them; what lies between them stays."""
    say("side by side", dtype, n, H, D, gap)
    dt, td = (q.QG_F32, torch.float32) if dtype == "f32" else (q.QG_BF16, torch.bfloat16)
    W, page = H * D, 16
    wide = 2 * (W + gap)
    rng = np.random.default_rng(6)
    cache = tensors.kv_cache(n // page + 1, page, H, D)
    cache.data.fill_(0xFF)
    x = dev(torch, rng.standard_normal((n, wide)).astype(np.float32)).to(td)
    slots = dev(torch, rng.permutation(cache.num_pages * page)[:n].astype(np.int32))
    q.qkv_append(dt, x, wide, x[:, W + gap:], wide, slots, n, cache)
    k, v = torch.empty(n, W, dtype=td, device="cuda"), torch.empty(n, W, dtype=td, device="cuda")
    q.qkv_read(dt, cache, slots, n, k, W, v, W)
    for first, second in ((0, W + gap), (W + gap, 0)):
        buf = Guarded(torch, n * wide, td)
        rows = buf.t.view(n, wide)
        q.qkv_read(dt, cache, slots, n, rows[:, first:], wide, rows[:, second:], wide)
        torch.cuda.synchronize()
        got = buf.numpy().reshape(n, wide)
        assert np.array_equal(got[:, first:first + W], k.float().cpu().numpy())
        assert np.array_equal(got[:, second:second + W], v.float().cpu().numpy())
        assert np.all(got[:, W:W + gap] == 77) and np.all(got[:, 2 * W + gap:] == 77)


def test_attention_beside_its_queries(torch):
    """Outputs in the same wider rows as the queries."""
    c = AttnCase(torch, "f32", 2, 3, 64, 16, [(40, 7), (90, 2)])
    want, want_lse = c.run()
    W = c.Hq * c.D
    both = torch.full((c.total, 2 * W + 8), 5.0, device="cuda")
    both[:, :W] = c.q[:, :W]
    lse = torch.empty(c.total, c.Hq, device="cuda")
    q.qkv_attn(c.dt, both, 2 * W + 8, c.cache, dev(torch, c.table), c.width, dev(torch, c.cu), dev(torch, c.kv_len), c.B, c.total, 7,
               c.max_kv, c.Hq, c.scale, 0, both[:, W + 4:], 2 * W + 8, lse)
    torch.cuda.synchronize()
    assert np.array_equal(both[:, W + 4:2 * W + 4].cpu().numpy().reshape(want.shape), want)
    assert torch.equal(both[:, :W], c.q[:, :W]) and (both[:, W:W + 4] == 5).all() and (both[:, 2 * W + 4:] == 5).all()
    assert np.array_equal(lse.cpu().numpy(), want_lse)


# --- long contexts, windows in bfloat16, neighbours -----------------------------------------

class LongCase:
    """Requests of many tokens with random codes and coefficients, on the GPU;
    sampled rows are compared with 64 bits there."""

    def __init__(self, torch, dtype, H, G, D, page, lens, window=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.H, self.G, self.D, self.page, self.window, self.lens = torch, H, G, D, page, window, lens
        self.dt, self.td = (q.QG_F32, torch.float32) if dtype == "f32" else (q.QG_BF16, torch.bfloat16)
        self.B, self.Hq = len(lens), H * G
        self.width = -(-max(kv for kv, _ in lens) // page)
        used = [-(-kv // page) for kv, _ in lens]
        self.pages = sum(used) + 1
        perm = torch.randperm(self.pages, generator=g, device="cuda").int()
        self.table = torch.full((self.B, self.width), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(used):
            self.table[b, :n] = perm[sum(used[:b]):sum(used[:b]) + n]
        n_code, n_coef = page * D // 2, page * (D // 64) * 4
        self.data = torch.empty(self.pages, H, ref.block_bytes(page, D), dtype=torch.uint8, device="cuda")
        for part in range(2):
            lo = part * (n_code + n_coef)
            z = torch.randn(2, self.pages, H, n_code, generator=g, device="cuda").mul_(2.9).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
            self.data[:, :, lo:lo + n_code] = z[0] | (z[1] << 4)
            s = 0.15 + 0.3 * torch.rand(self.pages, H, n_coef // 4, generator=g, device="cuda")
            b = -7.5 * s + 0.4 * torch.randn(self.pages, H, n_coef // 4, generator=g, device="cuda")
            co = torch.stack([s, b], -1).bfloat16().view(torch.int16).reshape(self.pages, H, n_coef // 2).contiguous()
            self.data[:, :, lo + n_code:lo + n_code + n_coef] = co.view(torch.uint8)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
        self.total, self.scale = int(self.cu[-1]), D ** -0.5
        self.q = (torch.randn(self.total, self.Hq, D, generator=g, device="cuda") * 1.2).to(self.td)

    def run(self):
        torch = self.torch
        cache = q.KVCache(self.data, self.pages, self.page, self.H, self.D)
        max_q, max_kv = max(n for _, n in self.lens), max(kv for kv, _ in self.lens)
        out, lse = torch.empty_like(self.q), torch.empty(self.total, self.Hq, device="cuda")
        ws = tensors.attn_workspace(cache, self.B, self.total, max_q, max_kv, self.Hq)
        kv_len = torch.tensor([kv for kv, _ in self.lens], dtype=torch.int32, device="cuda")
        q.qkv_attn(self.dt, self.q, self.Hq * self.D, cache, self.table, self.width, dev(torch, self.cu), kv_len, self.B, self.total, max_q,
                   max_kv, self.Hq, self.scale, self.window, out, self.Hq * self.D, lse, ws)
        torch.cuda.synchronize()
        return out, lse

    def values(self, b, h, part, kv):
        torch = self.torch
        lo, mid, end = ref.parts(self.page, self.D, part)
        blk = self.data[self.table[b, :-(-kv // self.page)].long(), h]
        byte = blk[:, lo:mid]
        code = torch.stack([byte & 15, byte >> 4], -1).double().reshape(-1, self.D // 64, 64)
        co = blk[:, mid:end].contiguous().view(torch.bfloat16).double().reshape(-1, self.D // 64, 2)
        size = (8 * co[..., :1].abs() + (co[..., 1:] + 8 * co[..., :1]).abs()).expand_as(code)
        return (code * co[..., :1] + co[..., 1:]).reshape(-1, self.D)[:kv], size.reshape(-1, self.D)[:kv]

    def check(self, got):
        """Weights' rounding errors (2^-21 (1 + amp) each; bfloat16: 2^-12) and
        those of the sums (kv / 32 additions, 2^-24 of the terms' sizes; 8 times
        that for bfloat16's small codes) add up like random ones: six times
        their root."""
        torch = self.torch
        out, lse = got
        for b, (kv, n) in enumerate(self.lens):
            for h in range(self.H):
                k, kb = self.values(b, h, 0, kv)
                v, vb = self.values(b, h, 1, kv)
                for i in sorted({0, 1, n // 2, n - 1} & set(range(n))):
                    p = kv - n + i
                    lo = max(0, p - self.window + 1) if self.window else 0
                    for j in sorted({h * self.G, (h + 1) * self.G - 1}):
                        x = self.q[self.cu[b] + i, j].double()
                        s = (k[lo:p + 1] @ x) * self.scale
                        w = torch.softmax(s, 0)
                        want, spread = w @ v[lo:p + 1], w @ vb[lo:p + 1]
                        amp = float((kb[lo:p + 1] @ x.abs()).max()) * self.scale
                        root = ((w * w) @ (vb[lo:p + 1] ** 2)).sqrt()
                        tol = 6 * 2.0 ** -21 * (1 + amp) * root + 6 * 2.0 ** -24 * (p / 32 + 1) ** 0.5 * spread
                        if self.dt == q.QG_BF16:
                            tol = 8 * tol + 6 * 2.0 ** -12 * root + 2.0 ** -8 * want.abs()
                        err = (out[self.cu[b] + i, j].double() - want).abs()
                        assert (err <= tol).all(), (b, h, i, j, float((err / tol).max()))
                        ref_lse = float(torch.logsumexp(s, 0))
                        assert abs(float(lse[self.cu[b] + i, j]) - ref_lse) <= 2.0 ** -20 * (1 + amp) + 2.0 ** -22 * abs(ref_lse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,G,D,page,lens,window", [
    (2, 4, 128, 64, [(131071, 1)], 0), (2, 16, 64, 16, [(40001, 1), (9000, 1), (65536, 1)], 0), (1, 7, 256, 32, [(30000, 4), (20011, 5)], 0),
    (1, 8, 64, 128, [(65537, 30)], 0), (8, 4, 128, 64, [(131072, 2048)], 0), (2, 4, 128, 16, [(50000, 1), (30000, 7)], 20011)])
def test_attention_long_contexts(torch, dtype, H, G, D, page, lens, window):
    """Up to 131072 tokens, in one piece (2048 rows) and in many; pages all over
    a cache of up to 300 MB."""
    say("long", dtype, H, G, D, lens, window)
    c = LongCase(torch, dtype, H, G, D, page, lens, window)
    c.check(c.run())


@pytest.mark.parametrize("window", [1, 16, 65, 200])
@pytest.mark.parametrize("H,G,D,page,lens", [(1, 4, 64, 16, [(701, 1), (3, 1), (130, 1)]), (2, 2, 128, 32, [(300, 5), (129, 2)]),
                                             (1, 3, 128, 16, [(150, 150), (77, 20)]), (1, 2, 256, 64, [(333, 70)])])
def test_attention_window_bf16(torch, window, H, G, D, page, lens):
    say("window bf16", window, D, lens)
    AttnCase(torch, "bf16", H, G, D, page, lens, window=window).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_alone_and_among_others(torch, dtype, D):
    """A request's rows in a call of their own, and beside requests that bring
    other tile heights and splits: each within the bound, so their difference
    within twice that (their rounding may differ)."""
    say("neighbours", dtype, D)
    one = [(700, 2)]
    alone = AttnCase(torch, dtype, 1, 4, D, 16, one, seed=7)
    _, l, spread, amp = alone.want()
    got = alone.run()
    alone.check(got)
    tol = spread * (2.0 ** -20 * (1 + amp[..., None]) + 2.0 ** -24 * (700 / 16 + 16))
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(got[0]) + 2.0 ** -11 * spread
    for others in ([(90, 3)], [(300, 90)], [(40, 1)] * 30):
        c = AttnCase(torch, dtype, 1, 4, D, 16, one + others, seed=7)
        # the same tokens and queries for the first request
        for j in range(700):
            a, b = (int(x.table[0, j // 16]) for x in (alone, c))
            for part in range(2):
                lo, mid, _ = ref.parts(16, D, part)
                for at, size in ((lo, D // 2), (mid, D // 16)):
                    at += j % 16 * size
                    c.data[b, :, at:at + size] = alone.data[a, :, at:at + size]
        c.q[:2] = alone.q
        out, lse = c.run()
        assert np.all(np.abs(out[:2] - got[0]) <= 2 * tol)
        assert np.all(np.abs(lse[:2] - got[1]) <= 2 * (2.0 ** -20 * (1 + amp) + 2.0 ** -22 * np.abs(l)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,by", [(64, 60), (128, -60), (128, 95), (64, -95), (256, 95)])
def test_attention_keys_and_queries_of_any_size(torch, dtype, kind, D, by):
    """Keys 2^by as large and queries 2^-by: the scores are as before."""
    say("key size", dtype, kind, D, by)
    c = value_case(torch, dtype, kind, D)
    scale_values(c, lambda b, j, g: by, part=0)
    c.q *= 2.0 ** -by
    c.check()
