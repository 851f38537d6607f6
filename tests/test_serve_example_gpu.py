"""The serving example: its steps against plain references on what each
operator was given, its pages, and its drafts."""
import os
import sys

import numpy as np
import pytest

import serve_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import serve  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def model():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("needs a GPU")
    return serve.Model(serve.Shape())


def check_step(session, trace, before):
    shape, page = session.model.shape, session.page
    D, H, Hq = shape.head_dim, shape.kv_heads, shape.q_heads
    table = session.table.cpu().numpy()
    for t in trace[:-1]:
        cache, cu, kv = t["cache"], t["cu_q"].cpu().numpy(), t["kv_len"].cpu().numpy()
        qkv, out = t["qkv"].cpu().numpy(), t["out"].cpu().numpy()
        data = cache.data.cpu().numpy().reshape(cache.num_pages, H, ref.block_bytes(page, D))
        # the cache holds what was appended, and else what it held
        want = before[id(cache)].copy()
        ref.append(want, page, H, D, qkv[:, Hq * D:(Hq + H) * D], qkv[:, (Hq + H) * D:], t["slots"].cpu().numpy())
        assert np.array_equal(data, want)
        x = qkv[:, :Hq * D].astype(np.float64).reshape(-1, Hq, D)
        o, _, spread, amp = ref.attn(x, data, page, H, D, table, cu, kv, D ** -0.5, 0)
        tol = spread * (2.0 ** -21 * 2 * (1 + amp[..., None]) + 2.0 ** -24 * (float(kv.max()) / 16 + 16))
        assert np.all(np.abs(out.reshape(o.shape) - o) <= tol)


def data_of(session):
    shape, page = session.model.shape, session.page
    return {id(c): c.data.cpu().numpy().reshape(c.num_pages, shape.kv_heads, ref.block_bytes(page, shape.head_dim)).copy()
            for c in session.caches}


def test_steps(model):
    import torch
    rng = np.random.default_rng(11)
    B, vocab = 3, model.shape.vocab
    s = serve.Session(model, B, 128)
    for c in s.caches:
        c.data.fill_(0xFF)
    lens = [0] * B
    for keep, n_new, rows in (([0, 0, 0], [37, 5, 16], 1),       # prompts
                              ([37, 5, 16], [1, 1, 1], 1),       # a token each
                              ([38, 6, 17], [4, 0, 2], 4),       # drafts; one request waits
                              ([39, 0, 18], [1, 21, 3], 2)):     # three rejected; one ended, another took its row
        print("step", keep, n_new, flush=True)
        before, trace = data_of(s), []
        new = [rng.integers(0, vocab, size=n).tolist() for n in n_new]
        r = s.step(keep, new, rows_wanted=rows, trace=trace)
        torch.cuda.synchronize()
        check_step(s, trace, before)
        lens = [k + n for k, n in zip(keep, n_new)]
        assert s.kv_len.tolist() == lens
        used = [p for b in range(B) for p in s.table[b, :-(-lens[b] // s.page)].tolist()]
        head, tail = s.state.tolist()
        free = [int(s.ring[i % s.ring.numel()]) for i in range(head, tail)]
        assert sorted(used + free) == list(range(s.ring.numel()))
        logits = trace[-1]["logits"].cpu().numpy()
        assert logits.shape[0] == sum(min(n, rows) for n in n_new)
        assert np.array_equal(r.tokens, logits.argmax(1))
        lp, ent, rank, ids, top = ref.logprobs(logits, r.tokens, 4)
        assert np.array_equal(trace[-1]["rank"].cpu().numpy(), rank) and np.all(rank == 1)
        assert np.array_equal(r.top_ids, ids)
        for g, w in ((r.logprob, lp), (r.entropy, ent), (r.top_logprobs, top)):
            assert np.all(np.abs(g - w) <= 2.0 ** -20 + 2.0 ** -22 * np.abs(w))


def test_generate_and_pages(model):
    rng = np.random.default_rng(12)
    prompts = [rng.integers(0, model.shape.vocab, size=n).tolist() for n in (9, 70, 1)]
    for draft in (0, 3):
        done, (steps, tried, kept), s = serve.generate(model, prompts, 12, draft)
        assert [len(d) for d in done] == [12] * 3
        assert all(l < 0 for d in done for _, l in d) and kept <= tried
        assert steps == 11 if draft == 0 else steps <= 11
        head, tail = s.state.tolist()
        assert tail - head == s.ring.numel() and s.kv_len.tolist() == [0, 0, 0]
        again, _, _ = serve.generate(model, prompts, 12, draft)
        assert again == done


def test_out_of_pages(model):
    s = serve.Session(model, 2, 64, pages=3)
    assert s.step([0, 0], [[1] * 20, [2] * 10]) is not None
    with pytest.raises(RuntimeError, match="free pages"):
        s.step([20, 10], [[3] * 1, [4] * 30])
