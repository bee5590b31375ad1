"""The INT8 paged KV cache on a host without a GPU: what the entry points
refuse (fake pointers are never dereferenced), what the binding refuses
before the C call, and the plain reference against worked values."""
import ctypes

import numpy as np
import pytest
import torch

from int8_gemm_token_b200 import w8a8 as W
from tests import kv_reference as R

P = 0x10000   # a 16-byte aligned fake device address (never dereferenced)
ODD = 0x10008


def cache(**kw):
    a = dict(k=P, v=P, ks=P, vs=P, pages=10, heads=2, page=16, d=128)
    a.update(kw)
    return ctypes.byref(W._CacheStruct(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["heads"], a["page"], a["d"]))


def batch(**kw):
    a = dict(table=P, ld=4, start=P, kv=P, batch=3, max_pages=4, max_q=1, max_kv=64)
    a.update(kw)
    return ctypes.byref(W._BatchStruct(a["table"], a["ld"], a["start"], a["kv"], a["batch"], a["max_pages"], a["max_q"],
                                       a["max_kv"]))


BAD_CACHES = [(dict(page=24), 3), (dict(page=256), 3), (dict(page=0), 3), (dict(d=80), 3), (dict(d=256), 3),
              (dict(heads=0), 1), (dict(heads=-1), 1), (dict(pages=-1), 1), (dict(k=None), 1), (dict(vs=None), 1),
              (dict(k=ODD), 2), (dict(v=ODD), 2), (dict(ks=P + 2), 2)]
BAD_BATCHES = [(dict(batch=-1), 1), (dict(ld=3), 1), (dict(max_pages=-1), 1), (dict(max_q=-1), 1), (dict(max_kv=65), 1),
               (dict(max_kv=-1), 1), (dict(start=None), 1), (dict(kv=None), 1), (dict(table=None), 1),
               (dict(start=P + 2), 2), (dict(table=P + 1), 2), (dict(batch=70000), 1),
               (dict(max_pages=1 << 27, ld=1 << 27), 3)]


def append(c=None, b=None, tokens=3, k=P, kt=256, kh=128, v=P, vt=256, vh=128, cos=P, sin=P, rope=64, rot=128, il=0,
           q=P, qt=512, qh=128, hq=4, qo=P):
    return W.lib().w8a8_kv_append(c or cache(), b or batch(), tokens, k, kt, kh, v, vt, vh, cos, sin, rope, rot, il, q, qt,
                                  qh, hq, qo, None)


def attention(c=None, b=None, tokens=3, q=P, qt=512, qh=128, hq=4, scores=(0.1, 0.0, None, 0, None), out=P, ws=P,
              wsb=1 << 40):
    s = None if scores is None else ctypes.byref(W._ScoresStruct(*scores))
    return W.lib().w8a8_kv_attention(c or cache(), b or batch(), tokens, q, qt, qh, hq, s, out, ws, wsb, None)


def gather(c=None, table=P, ld=4, n=3, max_pages=4, first=P, start=P, rows=5, ko=P, vo=P, dt=0):
    return W.lib().w8a8_kv_gather(c or cache(), table, ld, n, max_pages, first, start, rows, ko, vo, dt, None)


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(bad, code):
    assert append(c=cache(**bad)) == code
    assert attention(c=cache(**bad)) == code
    assert gather(c=cache(**bad)) == code
    assert W.lib().w8a8_kv_attention_workspace_size(cache(**bad), batch(), 3, 4) == 0


@pytest.mark.parametrize("bad,code", BAD_BATCHES)
def test_append_and_attention_refuse_a_bad_batch(bad, code):
    assert append(b=batch(**bad)) == code
    assert attention(b=batch(**bad)) == code


def test_append_refusals():
    assert append(c=0) == 10 or torch.cuda.is_available()  # the good call: no device here
    assert W.lib().w8a8_kv_append(None, batch(), 3, P, 256, 128, P, 256, 128, None, None, 0, 0, 0, None, 0, 0, 0, None, None) == 1
    assert W.lib().w8a8_kv_append(cache(), None, 3, P, 256, 128, P, 256, 128, None, None, 0, 0, 0, None, 0, 0, 0, None, None) == 1
    assert append(tokens=-1) == 1
    assert append(tokens=(1 << 30) + 1) == 3
    assert append(k=None) == 1 and append(v=None) == 1
    assert append(k=ODD) == 2 and append(vt=260) == 2 and append(kh=4) == 2 and append(kt=-8) == 1
    assert append(cos=None) == 1 and append(sin=None) == 1
    assert append(rot=8) == 3 and append(rot=144) == 3 and append(rot=24) == 3
    assert append(cos=P + 4) == 2 and append(rope=-1) == 1
    assert append(q=None) == 1 and append(qo=None) == 1
    assert append(hq=0) == 1 and append(qo=ODD) == 2 and append(q=ODD) == 2 and append(qt=4) == 2
    assert append(tokens=0) == 0 and append(b=batch(batch=0, max_q=0)) == 0 and append(b=batch(max_q=0)) == 0


def test_attention_refusals():
    assert attention(tokens=-1) == 1
    assert attention(hq=0) == 1 and attention(hq=3) == 3 and attention(c=cache(heads=1), hq=129) == 3
    assert attention(scores=None) == 1
    for bad in ((float("nan"), 0.0, None, 0, None), (float("inf"), 0.0, None, 0, None), (1.0, -1.0, None, 0, None),
                (1.0, float("nan"), None, 0, None), (1.0, 0.0, None, -1, None)):
        assert attention(scores=bad) == 1
    assert attention(scores=(1.0, 0.0, P + 1, 0, None)) == 2 and attention(scores=(1.0, 0.0, None, 0, P + 2)) == 2
    assert attention(q=None) == 1 and attention(out=None) == 1
    assert attention(q=ODD) == 2 and attention(out=ODD) == 2 and attention(ws=ODD) == 2 and attention(qh=12) == 2
    assert attention(qt=0) == 1 and attention(qh=0) == 1  # a broadcast axis
    assert attention(tokens=0, q=None, out=None) == 0 and attention(b=batch(batch=0)) == 0
    f = W.lib().w8a8_kv_attention_requant
    s = ctypes.byref(W._ScoresStruct(1.0, 0.0, None, 0, None))
    assert f(cache(), batch(), 3, P, 512, 128, 4, s, None, P, P, P, 1 << 40, None) == 1
    assert f(cache(), batch(), 3, P, 512, 128, 4, s, P, None, P, P, 1 << 40, None) == 1
    assert f(cache(), batch(), 3, P, 512, 128, 4, s, P, P + 2, P, P, 1 << 40, None) == 2


def test_attention_refuses_caps_that_fp32_does_not_hold():
    for bad in ((1.0, 5000.0, None, 0, None), (1.0, float("inf"), None, 0, None), (1.0, 1e-39, None, 0, None),
                (1e30, 1e-10, None, 0, None)):
        assert attention(scores=bad) == 1
    for good in ((1.0, 4096.0, None, 0, None), (1.0, 1e-30, None, 0, None), (0.0, 1e-39, None, 0, None)):
        assert attention(tokens=0, scores=good) == 0


def test_gather_refusals():
    assert gather(dt=2) == 4
    assert gather(rows=-1) == 1 and gather(rows=(1 << 30) + 1) == 3
    assert gather(ko=None, vo=None) == 1 and gather(first=None) == 1 and gather(start=None) == 1
    assert gather(ko=ODD) == 2 and gather(ld=3) == 1 and gather(n=-1) == 1 and gather(table=None) == 1
    assert gather(rows=0) == 0 and gather(n=0) == 0


def test_status_names():
    assert W.status_string(11) == "W8A8_ERR_BAD_PAGE" and W.status_string(12) == "W8A8_ERR_BAD_SEQUENCE"


def host_cache(pages=4, heads=2, page=16, d=64):
    return W.PagedKVCache(*(torch.zeros((pages, heads, page, d), dtype=torch.int8) for _ in range(2)),
                          *(torch.zeros((pages, heads)) for _ in range(2)))


def host_batch(**kw):
    a = dict(page_table=torch.zeros((2, 2), dtype=torch.int32), seq_start=torch.zeros(3, dtype=torch.int32),
             kv_len=torch.zeros(2, dtype=torch.int32), max_q_len=1)
    a.update(kw)
    return W.KVBatch(**a)


def test_binding_refuses_bad_caches_and_batches():
    z8 = torch.zeros((4, 2, 16, 64), dtype=torch.int8)
    f = torch.zeros((4, 2))
    for args in ((z8.float(), z8, f, f), (z8, z8[:3], f, f), (z8, z8, f[:3], f), (z8, z8, f, f.double()),
                 (z8.transpose(1, 2), z8, f, f), (z8[0], z8[0], f, f),
                 (z8.view(4, 2, 8, 128), z8.view(4, 2, 8, 128), f, f), (z8.view(4, 2, 32, 32), z8.view(4, 2, 32, 32), f, f)):
        with pytest.raises(ValueError):
            W.PagedKVCache(*args)
    for bad in (dict(page_table=torch.zeros((2, 2))), dict(page_table=torch.zeros(4, dtype=torch.int32)),
                dict(seq_start=torch.zeros(2, dtype=torch.int32)), dict(kv_len=torch.zeros(2, dtype=torch.int64)),
                dict(page_table=torch.zeros((2, 4), dtype=torch.int32)[:, ::2])):
        with pytest.raises(ValueError):
            host_batch(**bad)


def test_binding_refuses_bad_tensors_before_the_c_call():
    c, b = host_cache(), host_batch()
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    cos = torch.zeros((32, 32))
    for bad, what in ((dict(k=k.float()), "k"), (dict(v=k[:1]), "v"), (dict(k=torch.zeros((2, 3, 64), dtype=torch.bfloat16)), "k"),
                      (dict(cos=cos), "cos"), (dict(cos=cos, sin=cos[:5]), "sin"), (dict(cos=cos.double(), sin=cos), "cos"),
                      (dict(q_out=q), "q_out"), (dict(q=q, q_out=q[:1]), "q_out"), (dict(q=q[:1]), "q"),
                      (dict(k=torch.zeros((2, 64, 2), dtype=torch.bfloat16).transpose(1, 2)), "k")):
        a = dict(k=k, v=k, cache=c, batch=b)
        a.update(bad)
        with pytest.raises(ValueError, match=what):
            W.w8a8_kv_append(**a)
    for bad, what in ((dict(q=q.float()), "q"), (dict(slopes=torch.zeros(3)), "slopes"), (dict(out=q[:1]), "out"),
                      (dict(prefix_len=torch.zeros(2)), "prefix_len"), (dict(out=q.float()), "out")):
        a = dict(q=q, cache=c, batch=b)
        a.update(bad)
        with pytest.raises(ValueError, match=what):
            W.w8a8_kv_attention(**a)
    i = torch.zeros(2, dtype=torch.int32)
    i3 = torch.zeros(3, dtype=torch.int32)
    t = b.page_table
    for bad, what in ((dict(first_pos=i3), "first_pos"), (dict(row_start=i), "row_start"), (dict(rows=None), "rows"),
                      (dict(k_out=torch.zeros((5, 2, 32))), "k_out"), (dict(out_dtype=torch.int8), "k_out"),
                      (dict(k_out=torch.zeros((5, 2, 64)), v_out=torch.zeros((5, 2, 64), dtype=torch.bfloat16)), "v_out")):
        a = dict(cache=c, page_table=t, first_pos=i, row_start=i3, rows=5)
        a.update(bad)
        with pytest.raises(ValueError, match=what):
            W.w8a8_kv_gather(**a)
    with pytest.raises(ValueError, match="CUDA"):  # well-formed, but host memory
        W.w8a8_kv_append(k, k, c, b)


# ------------------------------------------------------------------ the reference itself
def test_reference_append_worked_values():
    """Two tokens in a page of four slots: absmax 2 gives S = 2 / 127 and codes
    127 and -64 (rne(-63.5)); a third token of absmax 8 makes S four times as
    large, the old codes become rne(code / 4), halves to even."""
    c = R.Cache(*(np.zeros((1, 1, 16, 64), np.int8) for _ in range(2)), *(np.zeros((1, 1), np.float32) for _ in range(2)))
    x = np.zeros((3, 1, 64), np.float32)
    x[0, 0, :2], x[1, 0, :2], x[2, 0, 0] = (2.0, -1.0), (0.5, 1.5), -8.0
    t = np.zeros((1, 1), np.int32)
    c = R.append(c, R.Seqs(t, np.array([0, 2]), np.array([2])), x[:2], x[:2])
    assert c.ks[0, 0] == np.float32(2.0) / np.float32(127)
    assert c.k[0, 0, 0, :2].tolist() == [127, -64] and c.k[0, 0, 1, :2].tolist() == [32, 95]
    c = R.append(c, R.Seqs(t, np.array([0, 1]), np.array([3])), x[2:], x[2:])
    assert c.ks[0, 0] == np.float32(8.0) / np.float32(127)
    assert c.k[0, 0, 0, :2].tolist() == [32, -16] and c.k[0, 0, 1, :2].tolist() == [8, 24] and c.k[0, 0, 2, 0] == -127


def test_reference_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 1, 64))
    cos, sin = R.angles(5, 32)
    for il in (False, True):
        y = R.rotate(x, cos[:, None], sin[:, None], il, np.float64)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-6)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
        # the product of two rotated vectors depends on the distance alone
        z = R.rotate(np.repeat(x[:1], 5, 0), cos[:, None], sin[:, None], il, np.float64)
        dots = [(z[i] * z[i + 1]).sum() for i in range(4)]
        assert np.allclose(dots, dots[0], rtol=1e-5)


def test_reference_attention_against_a_plain_softmax():
    """One sequence, no options: torch's softmax in 64 bits on the dense values."""
    rng = np.random.default_rng(1)
    s, pages = R.make_seqs(rng, [4], [9], 16)
    c = R.random_cache(rng, pages, 2, 16, 64)
    q = rng.standard_normal((4, 4, 64)).astype(np.float32)
    out, tol = R.attention(c, s, q, 0.125)
    k, v = (torch.from_numpy(R.dense(c, s.table[0], 13, n)).repeat_interleave(2, 0) for n in "kv")
    z = torch.einsum("ihd,hjd->hij", torch.from_numpy(q).double(), k) * 0.125
    z = z.masked_fill(torch.arange(13)[None] > 9 + torch.arange(4)[:, None], float("-inf"))
    want = torch.einsum("hij,hjd->ihd", z.softmax(-1), v).numpy()
    assert np.allclose(out, want, rtol=1e-12, atol=1e-12) and (tol > 0).all()


def test_a_batch_serves_caches_of_several_page_sizes():
    """What one cache's call was given does not change when another's is prepared (two threads, one batch)."""
    b = W.KVBatch(torch.zeros((3, 5), dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                  torch.zeros(3, dtype=torch.int32), 1)
    small, large = W.PagedKVCache.empty(6, 2, 16, 64, "cpu"), W.PagedKVCache.empty(6, 2, 128, 64, "cpu")
    one, two = b._for(small), b._for(large)
    assert one._obj.max_kv_len == 5 * 16 and two._obj.max_kv_len == 5 * 128
    assert b._for(small)._obj.max_kv_len == 5 * 16 and one._obj.batch == two._obj.batch == 3


def test_empty_cache():
    c = W.PagedKVCache.empty(6, 2, 32, 96, "cpu")
    assert c.k_codes.shape == c.v_codes.shape == (6, 2, 32, 96) and c.k_codes.dtype == torch.int8
    assert c.k_scale.shape == c.v_scale.shape == (6, 2) and c.k_scale.dtype == torch.float32
    assert not any(t.any() for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale))
    with pytest.raises(ValueError):
        W.PagedKVCache.empty(6, 2, 24, 96, "cpu")
