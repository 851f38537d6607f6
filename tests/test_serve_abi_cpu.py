"""Refusals of the serving-step entry points: every argument error is found
on the host, before anything is enqueued, so no call here reaches a GPU. And
the reference forms the GPU tests compare with, held to hand-worked values."""
import numpy as np
import pytest

import gemm_qgemv_amd as q
import serve_ref as ref

A = 1 << 20    # fake, 16-byte aligned "device" addresses, far apart, never dereferenced


def at(i):
    return A + (i << 32)


def err(fn, *args, **kw):
    with pytest.raises(q.QGError) as e:
        fn(*args, stream=0, **kw)
    return e.value.status


def cache(data=at(40), pages=8, page=16, heads=2, dim=64):
    return q.KVCache(data, pages, page, heads, dim)


BAD_CACHES = [dict(page=8), dict(page=24), dict(page=512), dict(pages=0), dict(pages=1 << 28), dict(heads=0),
              dict(heads=1025), dict(dim=32), dict(dim=96), dict(dim=512)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_cache_geometry(bad):
    c = cache(**bad)
    assert q.qkv_cache_bytes(c) == 0
    assert q.qkv_attn_workspace_bytes(c, 1, 1, 1, 16, 4) == 0
    assert err(q.qkv_append, q.QG_F32, at(1), 1 << 20, at(2), 1 << 20, at(3), 4, c) == q.QG_ERR_SHAPE
    assert err(q.qkv_read, q.QG_F32, c, at(3), 4, at(1), 1 << 20, at(2), 1 << 20) == q.QG_ERR_SHAPE
    assert attn_err(cache=c) == q.QG_ERR_SHAPE


def test_cache_bytes():
    assert q.qkv_cache_bytes(cache(pages=3, page=16, heads=2, dim=64)) == 3 * 2 * 16 * (64 + 8)
    assert q.qkv_cache_bytes(cache(pages=5, page=64, heads=1, dim=256)) == 5 * 64 * (256 + 32)
    with pytest.raises(ValueError):
        import torch
        q.KVCache(torch.empty(100, dtype=torch.uint8), 3, 16, 2, 64)


PLAN = dict(len_old=at(1), keep=at(2), n_new=at(3), batch=4, page_size=16, block_table=at(4), table_stride=8, ring=at(5),
            ring_size=64, state_in=at(6), state_out=at(7), kv_len=at(8), cu_q=at(9), slots=at(10), pos=at(11), total=9,
            denied=at(12))


def plan_err(**kw):
    return err(q.qkv_plan, **dict(PLAN, **kw))


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, "NULL") for n in ("len_old", "keep", "n_new", "block_table", "ring", "state_in", "state_out", "kv_len",
                                    "cu_q", "slots", "pos", "denied")],
    (dict(batch=0), "SHAPE"), (dict(batch=8193), "SHAPE"), (dict(page_size=0), "SHAPE"), (dict(page_size=24), "SHAPE"),
    (dict(page_size=1 << 21), "SHAPE"), (dict(table_stride=0), "SHAPE"), (dict(ring_size=0), "SHAPE"),
    (dict(ring_size=1 << 31), "SHAPE"), (dict(total=-1), "SHAPE"), (dict(total=1 << 31), "SHAPE"),
    (dict(len_old=at(1) + 2), "ALIGN"), (dict(slots=at(10) + 1), "ALIGN"), (dict(state_in=at(6) + 4), "ALIGN"),
    (dict(state_out=at(7) + 4), "ALIGN"),
    (dict(state_out=at(6)), "ALIAS"), (dict(kv_len=at(1)), "ALIAS"), (dict(ring=at(4) + 64), "ALIAS"),
    (dict(slots=at(11)), "ALIAS"), (dict(cu_q=at(3)), "ALIAS")])
def test_plan_refusals(kw, status):
    assert plan_err(**kw) == getattr(q, "QG_ERR_" + status)


def test_append_and_read_refusals():
    c = cache()
    ok = dict(dtype=q.QG_F32, k=at(1), k_stride=128, v=at(2), v_stride=128, slots=at(3), n=4, cache=c)
    rd = dict(dtype=q.QG_F32, cache=c, slots=at(3), n=4, k=at(1), k_stride=128, v=at(2), v_stride=128)
    for kw, status in [(dict(dtype=0), "FORMAT"), (dict(dtype=3), "FORMAT"), (dict(k=None), "NULL"), (dict(v=None), "NULL"),
                       (dict(slots=None), "NULL"), (dict(n=-1), "SHAPE"), (dict(k_stride=127), "SHAPE"),
                       (dict(v_stride=130), "SHAPE"), (dict(k=at(1) + 8), "ALIGN"), (dict(slots=at(3) + 2), "ALIGN"),
                       (dict(cache=cache(data=at(40) + 8)), "ALIGN"), (dict(cache=cache(data=None)), "NULL"),
                       (dict(k=at(40) + 64), "ALIAS"), (dict(slots=at(40)), "ALIAS")]:
        assert err(q.qkv_append, **dict(ok, **kw)) == getattr(q, "QG_ERR_" + status), kw
    for kw, status in [(dict(dtype=9), "FORMAT"), (dict(k=None, v=None), "NULL"), (dict(slots=None), "NULL"),
                       (dict(n=1 << 31), "SHAPE"), (dict(v_stride=64), "SHAPE"), (dict(v=at(2) + 4), "ALIGN"),
                       (dict(v=at(40)), "ALIAS"), (dict(v=at(1) + 256), "ALIAS"), (dict(k=at(3)), "ALIAS")]:
        assert err(q.qkv_read, **dict(rd, **kw)) == getattr(q, "QG_ERR_" + status), kw
    # bfloat16 rows: strides are multiples of 8 elements
    assert err(q.qkv_append, **dict(ok, dtype=q.QG_BF16, k_stride=132)) == q.QG_ERR_SHAPE
    # nothing to do is no error, whatever the pointers
    q.qkv_append(q.QG_F32, None, 0, None, 0, None, 0, c, stream=0)
    q.qkv_read(q.QG_F32, c, None, 0, None, 0, None, 0, stream=0)


ATTN = dict(dtype=q.QG_F32, q=at(1), q_stride=256, cache=None, block_table=at(2), table_stride=8, cu_q=at(3), kv_len=at(4),
            batch=2, total_q=3, max_q=2, max_kv=100, q_heads=4, scale=0.125, window=0, out=at(5), out_stride=256, lse=at(6),
            ws=at(7), ws_bytes=1 << 24)


def attn_err(**kw):
    a = dict(ATTN, **kw)
    a["cache"] = a["cache"] or cache()
    return err(q.qkv_attn, **a)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), "FORMAT"), *[({n: None}, "NULL") for n in ("q", "block_table", "cu_q", "kv_len", "out")],
    (dict(batch=0), "SHAPE"), (dict(batch=65536), "SHAPE"), (dict(total_q=0), "SHAPE"), (dict(max_q=0), "SHAPE"),
    (dict(max_kv=0), "SHAPE"), (dict(max_kv=129), "SHAPE"), (dict(max_kv=(1 << 30) + 1, table_stride=1 << 30), "SHAPE"),
    (dict(q_heads=3), "SHAPE"), (dict(q_heads=0), "SHAPE"), (dict(q_heads=1026), "SHAPE"), (dict(scale=0.0), "SHAPE"),
    (dict(scale=-1.0), "SHAPE"), (dict(scale=float("nan")), "SHAPE"), (dict(scale=float("inf")), "SHAPE"),
    (dict(scale=3e38), "SHAPE"), (dict(window=-1), "SHAPE"), (dict(table_stride=0), "SHAPE"), (dict(q_stride=255), "SHAPE"),
    (dict(q_stride=258), "SHAPE"), (dict(out_stride=128), "SHAPE"), (dict(q=at(1) + 4), "ALIGN"), (dict(out=at(5) + 8), "ALIGN"),
    (dict(block_table=at(2) + 2), "ALIGN"), (dict(lse=at(6) + 1), "ALIGN"), (dict(out=at(1)), "ALIAS"),
    (dict(lse=at(5) + 16), "ALIAS"), (dict(out=at(40)), "ALIAS"), (dict(lse=at(4)), "ALIAS"), (dict(out=at(2)), "ALIAS")])
def test_attn_refusals(kw, status):
    assert attn_err(**kw) == getattr(q, "QG_ERR_" + status)


def test_attn_workspace():
    c = cache(pages=4096)
    big = dict(cache=c, max_kv=4096, table_stride=512)
    need = q.qkv_attn_workspace_bytes(c, 2, 3, 2, 4096, 4)
    assert need > 0 and need % 256 == 0
    assert attn_err(**big, ws_bytes=need - 1) == q.QG_ERR_WORKSPACE
    assert attn_err(**big, ws=None, ws_bytes=need) == q.QG_ERR_WORKSPACE
    assert attn_err(**big, ws=at(7) + 8, ws_bytes=need) == q.QG_ERR_ALIGN
    assert attn_err(**big, ws=at(5), ws_bytes=need) == q.QG_ERR_ALIAS
    assert attn_err(**big, ws=at(4), ws_bytes=need) == q.QG_ERR_ALIAS
    # sizes the entry point refuses report no workspace
    assert q.qkv_attn_workspace_bytes(c, 0, 3, 2, 4096, 4) == 0
    assert q.qkv_attn_workspace_bytes(c, 2, 3, 2, 4096, 5) == 0


LP = dict(logits=at(1), ld=1000, rows=3, vocab=999, ids=at(2), top=4, logprob=at(3), entropy=at(4), rank=at(5),
          top_ids=at(6), top_logprobs=at(7), ws=at(8), ws_bytes=1 << 24)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), "NULL"), (dict(ids=None), "NULL"), (dict(top_ids=None), "NULL"), (dict(top_logprobs=None), "NULL"),
    (dict(top=0), "NULL"), (dict(rows=0), "SHAPE"), (dict(vocab=0), "SHAPE"), (dict(vocab=(1 << 30) + 1, ld=1 << 31), "SHAPE"),
    (dict(ld=998), "SHAPE"), (dict(top=65), "SHAPE"), (dict(top=-1), "SHAPE"), (dict(vocab=3, top=4), "SHAPE"),
    (dict(logits=at(1) + 2), "ALIGN"), (dict(ids=at(2) + 1), "ALIGN"), (dict(entropy=at(4) + 3), "ALIGN"),
    (dict(logprob=at(1) + 64), "ALIAS"), (dict(rank=at(2)), "ALIAS"), (dict(entropy=at(3)), "ALIAS"),
    (dict(top_ids=at(7)), "ALIAS")])
def test_logprobs_refusals(kw, status):
    assert err(q.qlogprobs, **dict(LP, **kw)) == getattr(q, "QG_ERR_" + status)


def test_logprobs_workspace():
    need = q.qlogprobs_workspace_bytes(1, 151936, 20)
    assert need > 0
    big = dict(LP, ld=151936, rows=1, vocab=151936, top=20)
    assert err(q.qlogprobs, **dict(big, ws_bytes=need - 1)) == q.QG_ERR_WORKSPACE
    assert err(q.qlogprobs, **dict(big, ws=None, ws_bytes=need)) == q.QG_ERR_WORKSPACE
    assert err(q.qlogprobs, **dict(big, ws=at(8) + 4, ws_bytes=need)) == q.QG_ERR_ALIGN
    assert err(q.qlogprobs, **dict(big, ws=at(1), ws_bytes=need)) == q.QG_ERR_ALIAS
    assert q.qlogprobs_workspace_bytes(0, 10, 1) == 0 and q.qlogprobs_workspace_bytes(1, 10, 11) == 0


# --- the reference forms -------------------------------------------------------

def test_reference_quantizer_by_hand():
    """A group from 0 to 15 has scale 1 and bias 0: the codes are the rounded
    values, halves to even. The pages' worked example: range -0.5..0.8."""
    x = np.zeros(64, np.float32)
    x[:8] = [0, 15, 0.5, 1.5, 2.5, 7.4, 14.5, 13.5]
    codes, s, b = ref.quantize(x)
    assert (s, b) == (0x3F80, 0x0000) and codes[:8].tolist() == [0, 15, 0, 2, 2, 7, 14, 14]
    x = np.full(64, 0.28, np.float32)
    x[0], x[1] = -0.5, 0.8
    codes, s, b = ref.quantize(x)
    assert codes[:3].tolist() == [0, 15, 9] and abs(ref.bf16_value(s) - 1.3 / 15) < 4e-4 and ref.bf16_value(b) == -0.5
    assert ref.quantize(np.full(64, 3.0, np.float32))[1:] == (0, 0x4040)
    assert ref.quantize(np.array([np.inf] + [0] * 63, np.float32))[1:] == (0x7FC0, 0x7FC0)
    assert ref.quantize(np.array([3e38, -3e38] + [0] * 62, np.float32))[1:] == (0x7FC0, 0x7FC0)


def test_reference_attention_by_hand():
    """Two tokens with scores 0 and log 3: weights 1/4 and 3/4."""
    D, page = 64, 16
    data = np.zeros((1, 1, ref.block_bytes(page, D)), np.uint8)
    k, v = np.zeros((2, D), np.float32), np.zeros((2, D), np.float32)
    k[1, :] = 1.0                      # a constant group is its bias
    v[0, :], v[1, :] = 2.0, -2.0
    ref.append(data, page, 1, D, k, v, [0, 1])
    x = np.full((1, 1, D), np.log(3.0) / D)
    out, lse, _, _ = ref.attn(x, data, page, 1, D, np.zeros((1, 1), int), [0, 1], [2], 1.0, 0)
    assert np.allclose(out, -1.0) and np.allclose(lse, np.log(4.0))
    out, lse, _, _ = ref.attn(x, data, page, 1, D, np.zeros((1, 1), int), [0, 1], [2], 1.0, 1)
    assert np.allclose(out, -2.0) and np.allclose(lse, np.log(3.0))


def test_reference_plan_by_hand():
    """Pages of 4: request 0 grows by a page, 1 ends (two pages back), 2 is
    denied (one page is left), 3 still fits its page."""
    t = np.array([[7, -1, -1], [3, 9, -1], [-1, -1, -1], [5, -1, -1]], np.int32)
    r = ref.plan([4, 6, 0, 2], [4, 0, 0, 1], [1, 0, 7, 2], 4, t, np.array([20, 21, -1, -1], np.int32), [0, 2], 11)
    assert r["table"].tolist() == [[7, 20, -1], [3, 9, -1], [-1, -1, -1], [5, -1, -1]]
    assert r["ring"].tolist() == [20, 21, 3, 9] and r["state"].tolist() == [1, 4] and r["denied"][0] == 1
    assert r["kv_len"].tolist() == [5, 0, 0, 3] and r["cu_q"].tolist() == [0, 1, 1, 8, 10]
    assert r["slots"].tolist() == [80] + [-1] * 7 + [21, 22, -1] and r["pos"].tolist() == [4] + list(range(7)) + [1, 2, -1]


def test_reference_logprobs_by_hand():
    x = np.array([[0.0, np.log(2.0), -np.inf, 0.0]], np.float32)
    lp, ent, rank, tid, tlp = ref.logprobs(x, [3], 3)
    assert np.allclose(lp, -np.log(4.0)) and rank[0] == 3 and tid[0].tolist() == [1, 0, 3]
    assert np.allclose(ent, 1.5 * np.log(2.0)) and np.allclose(tlp[0], [-np.log(2.0), -np.log(4.0), -np.log(4.0)])
