"""Greedy serving of several requests at once, every heavy step a call of the
library: a small decoder with random 4-bit weights whose keys and values stay
in the paged 4-bit cache.

    python examples/serve.py [--requests 4] [--tokens 24] [--draft 3]

One step (Session.step) takes some new tokens of every request -- a prompt, one
token, or a drafted continuation to be checked -- and runs

    qkv_plan      pages, lengths and slots of the step, on the device
    qembed        the new tokens' rows of the tied 4-bit matrix
    per layer     qgemm (queries, keys and values in one product), qkv_append,
                  qkv_attn, qgemm (output projection)
    qgemv_argmax  logits and the greedy token of the rows that are asked for
    qlogprobs     log probability, entropy and the best alternatives

A drafted continuation is what followed the last two tokens where they last
stood in the request: tokens that the greedy choice does not confirm are
dropped by keeping fewer tokens in the next step's plan, which takes their
pages back. torch holds the memory and does the residual sums and norms.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_qgemv_amd as q  # noqa: E402
from gemm_qgemv_amd import synth, tensors  # noqa: E402


@dataclasses.dataclass
class Shape:
    vocab: int = 4099
    hidden: int = 512
    layers: int = 2
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64


class Model:
    """Random weights in the 4-bit format, their mean near 0, on the device."""

    def __init__(self, shape: Shape, seed: int = 0, device="cuda"):
        rng = np.random.default_rng([41, seed])
        self.shape, self.device = shape, device
        wide = shape.q_heads * shape.head_dim

        def draw(M, K):
            w = synth.draw_weights(synth.U4_G64, M, K, rng)
            scale = (w.scales.astype(np.uint32) << 16).view(np.float32)
            w.biases = synth.to_bf16_bits(-7.5 * scale)
            return tensors.to_device(w, device)
        self.embed = draw(shape.vocab, shape.hidden)
        self.layers = [(draw(wide + 2 * shape.kv_heads * shape.head_dim, shape.hidden), draw(shape.hidden, wide))
                       for _ in range(shape.layers)]


@dataclasses.dataclass
class StepResult:
    tokens: np.ndarray       # greedy token of each row asked for
    logprob: np.ndarray      # its log probability
    entropy: np.ndarray
    top_ids: np.ndarray      # [rows][top] best alternatives
    top_logprobs: np.ndarray


class Session:
    """A batch of requests and their cache: one block table for all layers."""

    def __init__(self, model: Model, batch: int, max_len: int, page: int = 16, pages: int | None = None):
        import torch
        s, dev = model.shape, model.device
        self.torch, self.model, self.batch, self.page = torch, model, batch, page
        self.width = -(-max_len // page)
        pages = pages or batch * self.width
        self.caches = [tensors.kv_cache(pages, page, s.kv_heads, s.head_dim, dev) for _ in range(s.layers)]
        self.table = torch.full((batch, self.width), -1, dtype=torch.int32, device=dev)
        self.ring = torch.arange(pages, dtype=torch.int32, device=dev)
        self.state = torch.tensor([0, pages], dtype=torch.int64, device=dev)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.length = [0] * batch                # the same, as the host knows it

    def _norm(self, x):
        return x * self.torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)

    def _product(self, w, x):
        y = self.torch.empty(x.shape[0], w.M, dtype=self.torch.float32, device=x.device)
        ws = tensors.workspace(q.QG_OP_GEMM, w.fmt, w.M, w.K, x.shape[0], x.device)
        q.qgemm(w.fmt, w.codes, w.scales, w.biases, x, y, w.M, w.K, x.shape[0], ws)
        return y

    def step(self, keep, new, rows_wanted=1, top=4, trace=None) -> StepResult | None:
        """Request b keeps its first keep[b] tokens and gets the tokens new[b].
        Returns what the head says at the last rows_wanted rows of each
        request (fewer where a request has fewer new ones), in order."""
        torch, m, s = self.torch, self.model, self.model.shape
        dev = m.device

        def ints(v):
            return torch.tensor(v, dtype=torch.int32, device=dev)
        n_new = [len(t) for t in new]
        total = sum(n_new)
        kv_len, cu_q = torch.empty_like(self.kv_len), torch.empty(self.batch + 1, dtype=torch.int32, device=dev)
        slots, pos = (torch.empty(max(total, 1), dtype=torch.int32, device=dev) for _ in range(2))
        state, denied = torch.empty_like(self.state), torch.empty(1, dtype=torch.int32, device=dev)
        q.qkv_plan(self.kv_len, ints(keep), ints(n_new), self.batch, self.page, self.table, self.width, self.ring,
                   self.ring.numel(), self.state, state, kv_len, cu_q, slots, pos, total, denied)
        if int(denied) > 0:                      # pages or table ran out: a request must end first
            raise RuntimeError(f"{int(denied)} requests found no free pages")
        self.kv_len, self.state = kv_len, state
        self.length = [k + n for k, n in zip(keep, n_new)]
        if total == 0:
            return None

        ids = ints([t for row in new for t in row])
        x = torch.empty(total, s.hidden, dtype=torch.float32, device=dev)
        q.qembed(m.embed.fmt, m.embed.codes, m.embed.scales, m.embed.biases, ids, x, s.vocab, s.hidden, total)
        D, wide, kv_wide = s.head_dim, s.q_heads * s.head_dim, s.kv_heads * s.head_dim
        row = wide + 2 * kv_wide
        max_q, max_kv = max(n_new), max(self.length)
        ws = tensors.attn_workspace(self.caches[0], self.batch, total, max_q, max_kv, s.q_heads, dev)
        for cache, (w_qkv, w_out) in zip(self.caches, m.layers):
            # queries, keys and values are parts of one product's rows
            qkv = self._product(w_qkv, self._norm(x))
            k, v = qkv[:, wide:], qkv[:, wide + kv_wide:]
            q.qkv_append(q.QG_F32, k, row, v, row, slots, total, cache)
            out = torch.empty(total, wide, dtype=torch.float32, device=dev)
            q.qkv_attn(q.QG_F32, qkv, row, cache, self.table, self.width, cu_q, kv_len, self.batch, total, max_q,
                       max_kv, s.q_heads, D ** -0.5, 0, out, wide, None, ws)
            if trace is not None:
                trace.append(dict(qkv=qkv, out=out, cache=cache, cu_q=cu_q, kv_len=kv_len, slots=slots))
            x = x + self._product(w_out, out)

        first = np.concatenate([[0], np.cumsum(n_new)])
        pick = [r for b, n in enumerate(n_new) for r in range(first[b] + max(0, n - rows_wanted), first[b] + n)]
        x = self._norm(x)[torch.tensor(pick, device=dev)]
        n = len(pick)
        logits = torch.empty(n, s.vocab, dtype=torch.float32, device=dev)
        idx = torch.empty(n, dtype=torch.int32, device=dev)
        e = m.embed
        for at in range(0, n, q.QG_MAX_ARGMAX_BATCH):
            part = slice(at, min(n, at + q.QG_MAX_ARGMAX_BATCH))
            rows = part.stop - part.start
            xp, lp = x[part].contiguous(), torch.empty(rows, s.vocab, dtype=torch.float32, device=dev)
            ip = torch.empty(rows, dtype=torch.int32, device=dev)
            hw = tensors.workspace(q.QG_OP_GEMV_ARGMAX, e.fmt, e.M, e.K, rows, dev)
            q.qgemv_argmax(e.fmt, e.codes, e.scales, e.biases, xp, lp, ip, e.M, e.K, rows, hw)
            logits[part], idx[part] = lp, ip
        logprob, entropy = (torch.empty(n, dtype=torch.float32, device=dev) for _ in range(2))
        rank = torch.empty(n, dtype=torch.int32, device=dev)
        top_ids = torch.empty(n, top, dtype=torch.int32, device=dev)
        top_lp = torch.empty(n, top, dtype=torch.float32, device=dev)
        q.qlogprobs(logits, s.vocab, n, s.vocab, idx, top, logprob, entropy, rank, top_ids, top_lp,
                    tensors.logprobs_workspace(n, s.vocab, top, dev))
        if trace is not None:
            trace.append(dict(logits=logits, idx=idx, rank=rank))
        return StepResult(*(t.cpu().numpy() for t in (idx, logprob, entropy, top_ids, top_lp)))


def drafted(tokens, most):
    """What followed the last two tokens where they last stood, `most` times."""
    text = list(tokens)
    while len(text) < len(tokens) + most:
        at = next((i for i in range(len(text) - 3, -1, -1) if text[i:i + 2] == text[-2:]), None)
        if at is None:
            break
        text.append(text[at + 2])
    return text[len(tokens):]


def generate(model, prompts, tokens=24, draft=3, page=16):
    """Greedy continuations [(token, log probability), ...] of each prompt and
    (steps, drafted tokens, confirmed ones)."""
    B = len(prompts)
    s = Session(model, B, max(map(len, prompts)) + tokens + draft + 1, page)
    text = [list(p) for p in prompts]
    done = [[] for _ in range(B)]
    r = s.step([0] * B, text)
    for b in range(B):
        done[b].append((int(r.tokens[b]), float(r.logprob[b])))
        text[b].append(done[b][-1][0])
    steps = tried = kept = 0
    while any(len(d) < tokens for d in done):
        live = [len(d) < tokens for d in done]
        guess = [drafted(text[b], draft) if live[b] else [] for b in range(B)]
        # the last token chosen is not in the cache yet; an ended request gives its pages back
        keep = [len(text[b]) - 1 if live[b] else 0 for b in range(B)]
        new = [[text[b][-1]] + guess[b] if live[b] else [] for b in range(B)]
        r = s.step(keep, new, rows_wanted=draft + 1)
        at = 0
        for b in range(B):
            for j in range(len(new[b])):
                done[b].append((int(r.tokens[at + j]), float(r.logprob[at + j])))
                text[b].append(done[b][-1][0])
                if j < len(guess[b]) and guess[b][j] != text[b][-1]:
                    break                        # the tokens behind it answered another text
                kept += j < len(guess[b])
            at += len(new[b])
            tried += len(guess[b])
            del done[b][tokens:]
        steps += 1
    s.step([0] * B, [[] for _ in range(B)])      # all pages back
    return done, (steps, tried, kept), s


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--draft", type=int, default=3)
    a = ap.parse_args()
    model = Model(Shape())
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, model.shape.vocab, size=int(n)).tolist()
               for n in rng.integers(5, 200, size=a.requests)]
    done, (steps, tried, kept), s = generate(model, prompts, a.tokens, a.draft)
    for b, d in enumerate(done):
        print(f"request {b}: {len(prompts[b])} tokens of prompt, then", " ".join(str(t) for t, _ in d),
              f"(log probability {sum(l for _, l in d):.2f})")
    head, tail = s.state.tolist()
    print(f"{steps} steps, {tried} tokens drafted, {kept} confirmed; {tail - head} of {s.ring.numel()} pages free")


if __name__ == "__main__":
    main()
