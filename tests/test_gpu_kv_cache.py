"""The INT8 paged KV cache on the GPU: append and read-back bit for bit
against the plain fp32 reference, attention against the 64-bit reference
within the bound that tests/kv_reference.py derives."""
import numpy as np
import pytest
import torch

from int8_gemm_token_b200 import synth
from int8_gemm_token_b200 import w8a8 as W
from tests import kv_reference as R
from tests.gpu_util import dev, dev_bf16, diff_report, host, host_bf16

pytestmark = pytest.mark.gpu


def to_dev(c: R.Cache) -> W.PagedKVCache:
    return W.PagedKVCache(dev(c.k), dev(c.v), dev(c.ks), dev(c.vs))


def batch_of(s: R.Seqs, max_kv=None) -> W.KVBatch:
    return W.KVBatch(dev(s.table), dev(s.start), dev(s.kv), int(max(s.new.max(), 0)), max_kv)


def bf16_rows(rng, tokens, heads, d, gain=1.0):
    return synth.bf16_bits(rng.standard_normal((tokens, heads, d), dtype=np.float32) * np.float32(gain))


def assert_same(got, want, what):
    assert got.shape == want.shape and got.dtype == want.dtype, what
    assert np.array_equal(got, want), f"{what}: {diff_report(got, want)}"


def assert_cache(c: W.PagedKVCache, want: R.Cache):
    assert_same(host(c.k_scale), want.ks, "k_scale")
    assert_same(host(c.v_scale), want.vs, "v_scale")
    assert_same(host(c.k_codes), want.k, "k_codes")
    assert_same(host(c.v_codes), want.v, "v_codes")


def status():
    return W.w8a8_check_device_error()


# ------------------------------------------------------------------ append
LENGTHS = {
    "one_token_each": dict(new=[1, 1, 1, 1], ctx=[0, 15, 16, 77]),
    "few": dict(new=[8, 3, 0, 5, 1], ctx=[9, 14, 40, 0, 127], spare=3),
    "many": dict(new=[67, 1, 130, 0, 16], ctx=[5, 31, 0, 3, 48], spare=2),
    "one_long": dict(new=[301], ctx=[0]),
    "padding_few": dict(new=[4, 1, 2], ctx=[0, 0, 0], kv=[2, 0, 20]),
    "padding_many": dict(new=[40, 9, 33], ctx=[0, 0, 0], kv=[21, 0, 64], spare=1),
}


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("d,page,hq,hkv,rot,interleaved", [
    (128, 64, 8, 2, 128, False), (64, 16, 3, 3, 32, True), (96, 32, 4, 1, 48, False), (128, 128, 2, 2, 128, True),
    (96, 16, 5, 5, 96, False), (64, 128, 6, 2, 0, False)])
def test_append(lengths, d, page, hq, hkv, rot, interleaved):
    rng = np.random.default_rng(7)
    s, pages = R.make_seqs(rng, page=page, **LENGTHS[lengths])
    cache = R.random_cache(rng, pages, hkv, page, d)
    # keys, values and queries as views of one projection's rows, k's values larger in some pages than the cache's
    fused = bf16_rows(rng, s.tokens, hq + 2 * hkv, d, 1.5)
    x = synth.bits_to_f32(fused)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    cos, sin = R.angles(int(s.kv.max()) + 1, rot) if rot else (None, None)
    want = R.append(cache, s, k, v, cos, sin, interleaved)
    keep = bf16_rows(rng, s.tokens, hq, d)
    want_q = R.rotate_queries(s, q, cos, sin, interleaved, keep)
    f = dev_bf16(fused)
    c, q_out = to_dev(cache), dev_bf16(keep)
    W.w8a8_kv_append(f[:, hq:hq + hkv], f[:, hq + hkv:], c, batch_of(s), cos=None if cos is None else dev(cos),
                     sin=None if sin is None else dev(sin), q=f[:, :hq], q_out=q_out, interleaved=interleaved)
    assert_cache(c, want)
    assert_same(host_bf16(q_out), want_q, "q_out")
    assert status() == 0


@pytest.mark.parametrize("gain", [0.0, 1e-30, 2e-38, 1e30])
def test_append_extreme_magnitudes(gain):
    """Zero tokens, tokens so small that 1 / S overflows, and very large ones; into a fresh and a started page."""
    rng = np.random.default_rng(3)
    s, pages = R.make_seqs(rng, [5, 20], [0, 9], 16)
    cache = R.random_cache(rng, pages, 2, 16, 64)
    k, v = bf16_rows(rng, s.tokens, 2, 64, gain), bf16_rows(rng, s.tokens, 2, 64, gain)
    c = to_dev(cache)
    W.w8a8_kv_append(dev_bf16(k), dev_bf16(v), c, batch_of(s))
    assert_cache(c, R.append(cache, s, synth.bits_to_f32(k), synth.bits_to_f32(v)))


def test_append_token_by_token_equals_reference_and_stays_near_the_values():
    """40 single appends into pages of 16: scales grow, old codes are
    re-rounded. Against the values themselves each code is off by half a step
    of the page's last scale, plus half a step of the scale at each growth
    (no more than the last one), however many there were."""
    rng = np.random.default_rng(11)
    page, heads, d, n = 16, 2, 64, 40
    cache = R.Cache(*(np.zeros((4, heads, page, d), np.int8) for _ in range(2)),
                    *(np.zeros((4, heads), np.float32) for _ in range(2)))
    table = np.array([[2, 0, 3]], np.int32)
    x = synth.bits_to_f32(bf16_rows(rng, n, heads, d)) * np.exp2(rng.integers(-3, 3, (n, 1, 1))).astype(np.float32)
    bits = synth.bf16_bits(x)
    x = synth.bits_to_f32(bits)
    c = to_dev(cache)
    growths = np.zeros((4, heads))
    for i in range(n):
        s = R.Seqs(table, np.array([0, 1], np.int32), np.array([i + 1], np.int32))
        before = cache.ks.copy()
        cache = R.append(cache, s, x[i:i + 1], x[i:i + 1])
        growths += (cache.ks > before) & (i % page > 0)
        t = dev_bf16(bits[i:i + 1])
        W.w8a8_kv_append(t, t, c, batch_of(s))
    assert_cache(c, cache)
    assert growths.max() >= 2
    for p, pi in enumerate(table[0]):
        m = min(n, (p + 1) * page) - p * page
        vals = cache.k[pi, :, :m].astype(np.float64) * cache.ks[pi].astype(np.float64)[:, None, None]
        err = np.abs(vals - x[p * page:p * page + m].transpose(1, 0, 2))
        step = cache.ks[pi].astype(np.float64)[:, None, None]
        assert (err <= step * (0.5 * (1 + growths[pi])[:, None, None] + 1e-4)).all()


def test_append_in_place_queries_and_repeated_call():
    """q_out may be q; appending the same tokens again changes nothing."""
    rng = np.random.default_rng(5)
    s, pages = R.make_seqs(rng, [30, 2], [3, 18], 16)
    cache = R.random_cache(rng, pages, 2, 16, 128)
    k, v, q = (bf16_rows(rng, s.tokens, 2, 128) for _ in range(3))
    cos, sin = R.angles(64, 128)
    want_q = R.rotate_queries(s, synth.bits_to_f32(q), cos, sin, False, q)
    c, qd = to_dev(cache), dev_bf16(q)
    W.w8a8_kv_append(dev_bf16(k), dev_bf16(v), c, batch_of(s), dev(cos), dev(sin), q=qd, q_out=qd)
    assert_same(host_bf16(qd), want_q, "q in place")
    first = [host(t).copy() for t in c._tensors]
    W.w8a8_kv_append(dev_bf16(k), dev_bf16(v), c, batch_of(s), dev(cos), dev(sin))
    for a, t in zip(first, c._tensors):
        assert_same(host(t), a, "second append of the same tokens")


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,page,heads", [(128, 64, 3), (64, 16, 1), (96, 32, 5), (64, 128, 8)])
def test_gather(d, page, heads, dtype):
    rng = np.random.default_rng(13)
    s, pages = R.make_seqs(rng, [0, 0, 0, 0], [200, 1, 0, 65], page)
    cache = R.random_cache(rng, pages, heads, page, d)
    first = np.array([37, 0, 0, 64], np.int32)
    start = np.concatenate([[0], np.cumsum(s.kv - first)]).astype(np.int32)
    rows = int(start[-1]) + 3
    keep = rng.standard_normal((rows, heads, d), dtype=np.float32)
    keep = synth.bits_to_f32(synth.bf16_bits(keep))
    wk, wv = R.gather(cache, s.table, first, start, keep)
    k_out, v_out = (torch.from_numpy(keep.copy()).cuda().to(dtype) for _ in range(2))
    W.w8a8_kv_gather(to_dev(cache), dev(s.table), dev(first), dev(start), k_out=k_out, v_out=v_out)
    for got, want in ((k_out, wk), (v_out, wv)):
        if dtype == torch.float32:
            assert_same(host(got), want, "gather")
        else:
            assert_same(host_bf16(got), synth.bf16_bits(want), "gather")
    only = torch.from_numpy(keep.copy()).cuda().to(dtype)
    W.w8a8_kv_gather(to_dev(cache), dev(s.table), dev(first), dev(start), v_out=only)
    assert torch.equal(only, v_out)
    assert status() == 0


# ------------------------------------------------------------------ attention
def check_attention(rng, s, cache, hq, **kw):
    d, heads = cache.d, cache.k.shape[1]
    q = bf16_rows(rng, s.tokens, hq, d)
    scale = kw.pop("scale", d ** -0.5)
    few = R.few_rows(s.new.max(), hq, cache, s)
    want, tol = R.attention(cache, s, synth.bits_to_f32(q), np.float32(scale), few=few,
                            slopes=kw.get("slopes"), prefix=kw.get("prefix"), softcap=kw.get("softcap", 0.0),
                            window=kw.get("window", 0))
    keep = bf16_rows(rng, s.tokens, hq, d)
    out = dev_bf16(keep)
    args = dict(scale=scale, softcap=kw.get("softcap", 0.0), window=kw.get("window", 0),
                slopes=None if kw.get("slopes") is None else dev(kw["slopes"]),
                prefix_len=None if kw.get("prefix") is None else dev(kw["prefix"]))
    W.w8a8_kv_attention(dev_bf16(q), to_dev(cache), batch_of(s), out=out, **args)
    got_bits = host_bf16(out)
    got = synth.bits_to_f32(got_bits).astype(np.float64)
    nobody = np.isnan(want)
    assert np.array_equal(got_bits[nobody], keep[nobody]), "rows of no sequence were written"
    err = np.abs(got - want)
    bad = ~nobody & ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} outside the bound; worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} times; "
                           f"first {np.argwhere(bad)[0]} got {got[bad][0]} want {want[bad][0]} tol {tol[bad][0]}")
    assert status() == 0
    return q, args, out


SHAPES = [(128, 64, 4, 4), (128, 16, 8, 2), (64, 16, 8, 1), (96, 32, 6, 2), (128, 128, 5, 1), (64, 64, 21, 3), (96, 16, 3, 3)]


@pytest.mark.parametrize("d,page,hq,hkv", SHAPES)
@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 31, 63, 255, 300, 1025])
def test_attention_single_tokens(d, page, hq, hkv, ctx):
    rng = np.random.default_rng(ctx + d)
    s, pages = R.make_seqs(rng, [1, 1, 1], [ctx, ctx // 2, 3 * ctx], page, spare=1)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, page, d), hq)


MASKS = {
    "plain": {},
    "softcap": dict(softcap=20.0),
    "window_1": dict(window=1),
    "window_33": dict(window=33),
    "alibi": dict(slopes=True),
    "prefix": dict(prefix=[40, 0, 1000]),
    "window_prefix": dict(window=50, prefix=[40, 70, 3]),
    "all": dict(window=120, prefix=[33, 0, 16], slopes=True, softcap=5.0),
    "sharp": dict(scale=3.0),
}


def mask_args(name, hq):
    kw = dict(MASKS[name])
    if kw.get("slopes"):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, hq + 1) / hq).astype(np.float32)
    if "prefix" in kw:
        kw["prefix"] = np.array(kw["prefix"], np.int32)
    return kw


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("d,page,hq,hkv", SHAPES[:4])
@pytest.mark.parametrize("new", [(1, 1, 1), (4, 2, 3), (8, 0, 5), (70, 33, 129)])
def test_attention_masks(mask, d, page, hq, hkv, new):
    rng = np.random.default_rng(len(mask) + 10 * new[0])
    s, pages = R.make_seqs(rng, list(new), [700, 90, 15], page)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, page, d), hq, **mask_args(mask, hq))


@pytest.mark.parametrize("d,page,hq,hkv", SHAPES)
@pytest.mark.parametrize("new,ctx", [([5], [0]), ([64], [0]), ([65], [0]), ([257], [0]), ([300, 1, 40], [0, 513, 100]),
                                     ([16, 128, 127, 129], [1000, 0, 1, 255])])
def test_attention_chunks(d, page, hq, hkv, new, ctx):
    rng = np.random.default_rng(new[0])
    s, pages = R.make_seqs(rng, new, ctx, page, spare=2)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, page, d), hq)


@pytest.mark.parametrize("d,page,hq,hkv", [(128, 64, 4, 1), (96, 16, 3, 1), (64, 32, 4, 4)])
@pytest.mark.parametrize("mask", ["plain", "window_prefix", "all"])
def test_attention_few_long_blocks(d, page, hq, hkv, mask):
    """Few query blocks behind long contexts: their key tiles are split over the SMs and joined."""
    rng = np.random.default_rng(d)
    s, pages = R.make_seqs(rng, [70, 40, 300], [5000, 3, 1500], page, spare=1)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, page, d), hq, **mask_args(mask, hq))


@pytest.mark.parametrize("B", [31, 32, 33, 95, 96, 97, 129])
def test_attention_single_tokens_of_several_scans_of_sequences(B):
    rng = np.random.default_rng(B)
    ctx = [int(c) for c in rng.integers(0, 90, B)]
    ctx[B // 2] = 2100  # cut into parts
    s, pages = R.make_seqs(rng, [1] * B, ctx, 32, kv=[0 if b % 7 == 3 else ctx[b] + 1 for b in range(B)], spare=1)
    check_attention(rng, s, R.random_cache(rng, pages, 2, 32, 64), 4, prefix=rng.integers(0, 99, B).astype(np.int32))


@pytest.mark.parametrize("mask", ["plain", "softcap", "window_33", "window_prefix", "all"])
@pytest.mark.parametrize("new,ctx,hq,hkv", [
    ([33, 1, 64], [100, 700, 0], 1, 1), ([11, 16, 2], [40, 0, 1200], 8, 2), ([1, 3, 2], [5, 900, 63], 21, 1),
    ([40, 64, 7], [4100, 0, 33], 23, 23)])
def test_attention_up_to_64_rows_of_a_head(new, ctx, hq, hkv, mask):
    rng = np.random.default_rng(new[0] + hq)
    s, pages = R.make_seqs(rng, new, ctx, 32, spare=1)
    assert R.few_rows(max(new), hq, R.random_cache(rng, 1, hkv, 32, 64), s)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, 32, 64), hq, **mask_args(mask, hq))


@pytest.mark.parametrize("hq,hkv,new", [(4, 4, 40), (8, 4, 31), (12, 4, 21)])
def test_attention_up_to_64_rows_of_many_short_sequences(hq, hkv, new):
    rng = np.random.default_rng(new)
    s, pages = R.make_seqs(rng, [new, 1, 0, 17] * 5, [60, 0, 33, 200] * 5, 16, spare=1)
    assert not R.few_rows(new, hq, R.random_cache(rng, 1, hkv, 16, 128), s)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, 16, 128), hq)


@pytest.mark.parametrize("new,kv", [([1, 1, 1], [0, 5, 0]), ([3, 2], [1, 0]), ([50, 70, 40], [30, 70, 0])])
@pytest.mark.parametrize("prefix", [None, [4, 4, 4]])
def test_attention_padding_rows_are_zero(new, kv, prefix):
    """Rows at negative positions (empty slots of a captured step) see nothing, not even the prefix."""
    rng = np.random.default_rng(1)
    s, pages = R.make_seqs(rng, new, new, 16, kv=kv, spare=1)
    kw = {} if prefix is None else {"prefix": np.array(prefix[:len(new)], np.int32)}
    check_attention(rng, s, R.random_cache(rng, pages, 2, 16, 128), 4, **kw)


def test_attention_requant_equals_quantizing_the_output():
    rng = np.random.default_rng(2)
    r, Z = torch.tensor([31.7], device="cuda"), torch.tensor([-9], dtype=torch.int32, device="cuda")
    for new, ctx in (([1] * 5, [3, 40, 100, 900, 0]), ([80, 1], [7, 30])):
        s, pages = R.make_seqs(rng, new, ctx, 32, spare=2)
        cache = R.random_cache(rng, pages, 2, 32, 128)
        q, args, out = check_attention(rng, s, cache, 8)
        codes = torch.full((s.tokens, 8, 128), 77, dtype=torch.int8, device="cuda")
        W.w8a8_kv_attention_requant(dev_bf16(q), to_dev(cache), batch_of(s), r, Z, out=codes, **args)
        n = int(s.start[-1])
        want = W.w8a8_quant_per_tensor(out.view(s.tokens, -1), r, Z).view_as(codes)
        assert torch.equal(codes[:n], want[:n])
        assert (codes[n:] == 77).all()


# ------------------------------------------------------------------ what the host cannot check
def test_bad_pages_and_sequences_are_reported_and_skipped():
    rng = np.random.default_rng(4)
    page, hkv, hq, d = 16, 2, 4, 64
    s, pages = R.make_seqs(rng, [3, 3, 3], [30, 30, 30], page)
    cache = R.random_cache(rng, pages, hkv, page, d)
    bits = bf16_rows(rng, s.tokens, hq, d)
    k = dev_bf16(bits[:, :hkv])
    x = synth.bits_to_f32(bits[:, :hkv])
    assert status() == 0
    for bad in (-1, pages, 2 ** 30):
        t = s.table.copy()
        t[1, 2] = bad  # sequence 1's last page: it holds position 32, its last new token
        bb = W.KVBatch(dev(t), dev(s.start), dev(s.kv), 3)
        c = to_dev(cache)
        W.w8a8_kv_append(k, k, c, bb)
        assert status() == 11
        want = R.append(cache, R.Seqs(s.table[[0, 2]], np.array([0, 3, 6], np.int32), s.kv[[0, 2]]), x[[0, 1, 2, 6, 7, 8]],
                        x[[0, 1, 2, 6, 7, 8]])
        part = R.append(want, R.Seqs(s.table[[1]], np.array([0, 2], np.int32), np.array([32], np.int32)), x[3:5], x[3:5])
        assert_cache(c, part)
        out = W.w8a8_kv_attention(dev_bf16(bits), c, bb)
        assert status() == 11
        # the tokens of the missing page are not seen
        want, tol = R.attention(part, R.Seqs(s.table[[1]], np.array([0, 2], np.int32), np.array([32], np.int32)),
                                synth.bits_to_f32(bits[3:5]), np.float32(d ** -0.5))
        got = synth.bits_to_f32(host_bf16(out))[3:5]
        assert (np.abs(got - want) <= tol).all()
        ko, _ = W.w8a8_kv_gather(c, dev(t), dev(np.zeros(3, np.int32)), dev(np.array([0, 33, 66, 99], np.int32)), rows=99)
        assert status() == 11
        assert (ko[33 + 32] == 0).all() and (ko[33 + 31] != 0).any()
    # lengths and offsets outside the call's limits
    keep = bf16_rows(rng, s.tokens, hq, d)
    for start, kv, max_q, max_kv in (([0, 3, 2, 9], s.kv, 9, None), ([0, 3, 6, 12], s.kv, 6, None),
                                     ([0, 3, 6, 9], [33, 49, 33], 3, 48), ([0, 3, 6, 9], [33, -1, 33], 3, None),
                                     ([0, 2, 7, 9], s.kv, 4, None), ([-3, 0, 6, 9], s.kv, 6, None)):
        bb = W.KVBatch(dev(s.table), dev(np.array(start, np.int32)), dev(np.array(kv, np.int32)), max_q, max_kv)
        c = to_dev(cache)
        qo = dev_bf16(keep)
        W.w8a8_kv_append(k, k, c, bb, q=dev_bf16(bits), q_out=qo)
        assert status() == 12
        out = dev_bf16(keep)
        W.w8a8_kv_attention(dev_bf16(bits), c, bb, out=out)
        assert status() == 12
    for first, start in (([0, -1, 0], [0, 3, 6, 9]), ([0, 46, 0], [0, 3, 6, 9]), ([0, 0, 0], [0, 5, 4, 9])):
        ko = torch.full((9, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
        W.w8a8_kv_gather(to_dev(cache), dev(s.table[:, :3].copy()), dev(np.array(first, np.int32)),
                         dev(np.array(start, np.int32)), k_out=ko)
        assert status() == 12
    # a sequence past the rotation table
    cos, sin = R.angles(32, 64)
    c = to_dev(cache)
    W.w8a8_kv_append(k, k, c, batch_of(s), dev(cos), dev(sin))
    assert status() == 12
    assert_cache(c, cache)


@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [40, 300, 7]), ([5, 12, 1], [0, 90, 33]), ([70, 33, 129], [100, 0, 15])])
@pytest.mark.parametrize("d,page,hq,hkv", [(128, 32, 8, 2), (96, 16, 3, 3), (64, 64, 5, 1)])
def test_attention_query_strides(new, ctx, d, page, hq, hkv):
    """Queries inside a fused projection's rows, and head-major: the same bits as dense ones."""
    rng = np.random.default_rng(d + new[0])
    s, pages = R.make_seqs(rng, new, ctx, page, spare=1)
    cache = R.random_cache(rng, pages, hkv, page, d)
    q, args, out = check_attention(rng, s, cache, hq)
    n = int(s.start[-1])
    fused = torch.full((s.tokens, hq + 2 * hkv + 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 1:1 + hq] = dev_bf16(q)
    heads_first = dev_bf16(q).transpose(0, 1).contiguous().transpose(0, 1)
    for view in (fused[:, 1:1 + hq], heads_first):
        got = W.w8a8_kv_attention(view, to_dev(cache), batch_of(s), **args)
        assert torch.equal(got[:n], out[:n])
    assert status() == 0


@pytest.mark.parametrize("new", [(1, 3, 2), (40, 70, 9)])
def test_rows_in_front_of_the_first_sequence_are_nobodys(new):
    rng = np.random.default_rng(new[0])
    s, pages = R.make_seqs(rng, list(new), [20, 0, 70], 16, spare=2)
    s = R.Seqs(s.table, s.start + 21, s.kv, spare=2)
    cache = R.random_cache(rng, pages, 2, 16, 64)
    check_attention(rng, s, cache, 4)
    x = bf16_rows(rng, s.tokens, 2, 64)
    c = to_dev(cache)
    keep = dev_bf16(bf16_rows(rng, s.tokens, 2, 64))
    q_out = keep.clone()
    W.w8a8_kv_append(dev_bf16(x), dev_bf16(x), c, batch_of(s), q=dev_bf16(x), q_out=q_out)
    f = synth.bits_to_f32(x)
    assert_cache(c, R.append(cache, s, f, f))
    first, last = int(s.start[0]), int(s.start[-1])
    assert torch.equal(q_out[:first], keep[:first]) and torch.equal(q_out[last:], keep[last:])
    assert torch.equal(q_out[first:last], dev_bf16(x)[first:last])
    assert status() == 0


@pytest.mark.parametrize("hq,new", [(2, 1), (2, 40), (64, 3)])
def test_a_call_whose_contexts_are_all_empty(hq, new):
    c = W.PagedKVCache.empty(4, 2, 16, 64)
    rows = 3 * new
    b = W.KVBatch(torch.zeros((3, 2), dtype=torch.int32, device="cuda"), dev(np.arange(4, dtype=np.int32) * new),
                  torch.zeros(3, dtype=torch.int32, device="cuda"), new, 0)
    x = torch.ones((rows, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((rows, hq, 64), dtype=torch.bfloat16, device="cuda")
    turned = W.w8a8_kv_append(x, x, c, b, q=q)
    assert not turned.any() and not c.k_codes.any() and not c.k_scale.any()
    assert not W.w8a8_kv_attention(q, c, b).any()
    assert status() == 0


def test_many_sequences():
    """More sequences than a warp scans at once, for each of the kernels."""
    rng = np.random.default_rng(21)
    for new, ctx in (([1, 0, 2] * 400, [3, 17, 40] * 400), ([70, 1, 0] * 40, [5, 40, 3] * 40)):
        s, pages = R.make_seqs(rng, new, ctx, 16, spare=1)
        cache = R.random_cache(rng, pages, 1, 16, 64)
        check_attention(rng, s, cache, 2)
        x = bf16_rows(rng, s.tokens, 1, 64)
        c = to_dev(cache)
        W.w8a8_kv_append(dev_bf16(x), dev_bf16(x), c, batch_of(s))
        f = synth.bits_to_f32(x)
        assert_cache(c, R.append(cache, s, f, f))
    assert status() == 0


@pytest.mark.parametrize("new", [(1, 1, 1), (70, 33, 129)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 600])
def test_a_window_of_all_positions_is_none(new, window):
    rng = np.random.default_rng(3)
    s, pages = R.make_seqs(rng, list(new), [400, 0, 15], 32, kv=[400 + new[0], 0, 15 + new[2]])
    check_attention(rng, s, R.random_cache(rng, pages, 2, 32, 64), 4, window=window, prefix=np.array([30, 5, 0], np.int32))


@pytest.mark.parametrize("most", [20, 201])
def test_attention_reports_descending_starts(most):
    """Every sequence is checked by itself; those that hold may have been served."""
    rng = np.random.default_rng(8)
    start = np.array([0, 20, 40, 60, 5, 6, 26, 27], np.int32)
    kv = np.array([100, 10, 10, 10, 1, 20, 1], np.int32)
    table = np.arange(7 * 16, dtype=np.int32).reshape(7, 16)
    c = to_dev(R.random_cache(rng, 7 * 16, 2, 16, 64))
    assert status() == 0
    W.w8a8_kv_attention(dev_bf16(bf16_rows(rng, 60, 8, 64)), c, W.KVBatch(dev(table), dev(start), dev(kv), most))
    assert status() == 12


@pytest.mark.parametrize("new,ctx", [([1, 1], [100, 2]), ([3, 130], [1, 40])])
@pytest.mark.parametrize("d,hq", [(64, 128), (128, 128), (96, 65), (128, 43)])
def test_attention_large_groups(d, hq, new, ctx):
    rng = np.random.default_rng(hq)
    s, pages = R.make_seqs(rng, new, ctx, 64, spare=1)
    check_attention(rng, s, R.random_cache(rng, pages, 1, 64, d), hq)


def test_descending_starts_are_reported_and_stay_in_the_table():
    """A search over starts that descend may end at a sequence whose pages lie behind: it takes none in front of its row."""
    rng = np.random.default_rng(6)
    start = np.array([0, 100, 110, 120, 5, 6, 200, 201], np.int32)
    kv = np.array([100, 10, 10, 10, 1, 194, 1], np.int32)
    batch, wide = len(kv), 16
    # the call's table is the right half of a wider one, whose left half names a page of no sequence
    table = np.full((batch, 2 * wide), batch * wide, np.int32)
    table[:, wide:] = np.arange(batch * wide).reshape(batch, wide)
    full = dev(table)
    cache = R.random_cache(rng, batch * wide + 1, 2, 16, 64)
    c = to_dev(cache)
    x = dev_bf16(bf16_rows(rng, 201, 2, 64))
    assert status() == 0
    W.w8a8_kv_append(x, x, c, W.KVBatch(full[:, wide:], dev(start), dev(kv), 201))
    assert status() == 12
    for got, was in ((c.k_codes, cache.k), (c.v_codes, cache.v), (c.k_scale, cache.ks), (c.v_scale, cache.vs)):
        assert_same(host(got)[-1], was[-1], "a page in front of the table's rows")
    W.w8a8_kv_gather(to_dev(cache), full[:, wide:], dev(np.zeros(batch, np.int32)), dev(start), rows=201)
    assert status() == 12


def test_masked_pages_may_hold_anything():
    """Scales of infinity and NaN in pages that no row sees do not reach the output."""
    rng = np.random.default_rng(6)
    for new in ([1], [40]):
        s, pages = R.make_seqs(rng, new, [200], 16)
        cache = R.random_cache(rng, pages, 2, 16, 128)
        first = 200 - 50 + 1  # the first position that a window of 50 shows to the first new token
        for p in range(first // 16):
            cache.ks[s.table[0, p]], cache.vs[s.table[0, p]] = np.inf, np.nan
        q = bf16_rows(rng, s.tokens, 4, 128)
        clean = cache.copy()
        for p in range(first // 16):
            clean.ks[s.table[0, p]] = clean.vs[s.table[0, p]] = 1.0
        args = dict(window=50)
        a = W.w8a8_kv_attention(dev_bf16(q), to_dev(cache), batch_of(s), **args)
        b = W.w8a8_kv_attention(dev_bf16(q), to_dev(clean), batch_of(s), **args)
        assert torch.equal(a, b) and torch.isfinite(a).all()


# ------------------------------------------------------------------ together, as a program uses them
def test_captured_decode_steps_follow_growing_sequences():
    """A captured step (append, attention) replayed while kv_len grows equals eager steps on a second cache."""
    rng = np.random.default_rng(8)
    page, hkv, hq, d, B, steps = 16, 2, 8, 128, 3, 20
    table = rng.permutation(B * 5).astype(np.int32).reshape(B, 5)
    base = R.random_cache(rng, B * 5, hkv, page, d)
    ctx = np.array([0, 13, 50], np.int32)
    start = np.arange(B + 1, dtype=np.int32)
    cos, sin = (dev(x) for x in R.angles(80, d))
    fused = [dev_bf16(bf16_rows(rng, B, hq + 2 * hkv, d)) for _ in range(steps)]
    caches = [to_dev(base), to_dev(base)]
    kv = [dev(ctx + 1), dev(ctx + 1)]
    batches = [W.KVBatch(dev(table), dev(start), n, 1, 80) for n in kv]
    outs = [torch.empty((B, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qo = [torch.empty((B, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = [torch.empty((max(16, W.w8a8_kv_attention_workspace_size(caches[0], batches[0], B, hq)),), dtype=torch.uint8,
                      device="cuda") for _ in range(2)]
    x = fused[0].clone()

    def step(i, f):
        W.w8a8_kv_append(f[:, hq:hq + hkv], f[:, hq + hkv:], caches[i], batches[i], cos, sin, q=f[:, :hq], q_out=qo[i])
        W.w8a8_kv_attention(qo[i], caches[i], batches[i], out=outs[i], workspace=ws[i])

    step(0, x)  # the step again below: appending the same tokens changes nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0, x)
    for i in range(steps):
        x.copy_(fused[i])
        kv[0].copy_(torch.from_numpy(ctx + 1 + i))
        kv[1].copy_(torch.from_numpy(ctx + 1 + i))
        graph.replay()
        step(1, fused[i])
        assert torch.equal(outs[0], outs[1]), f"step {i}"
    for a, b in zip(caches[0]._tensors, caches[1]._tensors):
        assert torch.equal(a, b)
    assert status() == 0


def test_layer_chain_from_projection_to_output_projection():
    """A Prefill chunk and a Decode step of one attention layer: INT8
    projection, append with rotation, attention, INT8 output projection (the
    Decode step hands the attention result over as static codes)."""
    rng = np.random.default_rng(9)
    hid, hq, hkv, d, page = 512, 4, 2, 128, 16
    wide = (hq + 2 * hkv) * d
    Wqkv = W.w8a8_quant_weight_per_channel(dev(synth.weight(rng, hid, wide) * 3))
    Wo = W.w8a8_quant_weight_per_channel(dev(synth.weight(rng, hq * d, hid)))
    cos, sin = R.angles(128, d)
    new, ctx = [50, 33], [0, 0]
    s, pages = R.make_seqs(rng, new, ctx, page, width_extra=3, extra_pages=8)
    spare = [p for p in range(pages) if p not in set(s.table[s.table >= 0].tolist())]
    cache = R.Cache(*(np.zeros((pages, hkv, page, d), np.int8) for _ in range(2)),
                    *(np.zeros((pages, hkv), np.float32) for _ in range(2)))
    c = to_dev(cache)

    def project(x):
        Xq, S = W.w8a8_quant_per_token(x)
        return W.w8a8_gemm_dequant(Xq, S, Wqkv[0], Wqkv[1]).view(-1, hq + 2 * hkv, d)

    def layer(x, s):
        f = project(x)
        q = W.w8a8_kv_append(f[:, hq:hq + hkv], f[:, hq + hkv:], c, batch_of(s), dev(cos), dev(sin), q=f[:, :hq])
        fx = synth.bits_to_f32(host_bf16(f))
        nonlocal cache
        cache = R.append(cache, s, fx[:, hq:hq + hkv], fx[:, hq + hkv:], cos, sin)
        assert_cache(c, cache)
        few = R.few_rows(s.new.max(), hq, cache, s)
        want, tol = R.attention(cache, s, synth.bits_to_f32(host_bf16(q)), np.float32(d ** -0.5),
                                few=few)
        return q, want, tol

    x = dev_bf16(synth.activations(rng, s.tokens, hid))
    q, want, tol = layer(x, s)
    y = W.w8a8_kv_attention(q, c, batch_of(s))
    assert (np.abs(synth.bits_to_f32(host_bf16(y)) - want) <= tol).all()
    S, r, Z = W.w8a8_calibrate_static(y.view(s.tokens, -1))
    # one decode step: position 50 is in the fourth page of sequence 0 (there), 33 in the third of sequence 1
    table = s.table.copy()
    for b in range(2):
        need = -(-(int(s.kv[b]) + 1) // page)
        for i in range(need):
            if table[b, i] < 0:
                table[b, i] = spare.pop()
    s1 = R.Seqs(table, np.array([0, 1, 2], np.int32), s.kv + 1)
    x1 = dev_bf16(synth.activations(rng, 2, hid))
    q1, want, tol = layer(x1, s1)
    y1 = W.w8a8_kv_attention(q1, c, batch_of(s1))
    assert (np.abs(synth.bits_to_f32(host_bf16(y1)) - want) <= tol).all()
    codes = W.w8a8_kv_attention_requant(q1, c, batch_of(s1), r, Z)
    got = W.w8a8_gemm_dequant(codes.view(2, -1), S, Wo[0], Wo[1], colsum=Wo[2], Z=Z)
    assert torch.equal(got, W.w8a8_linear_static(y1.view(2, -1), S, r, Z, *Wo))
    assert status() == 0


def test_two_streams_at_once_equal_one_after_the_other():
    rng = np.random.default_rng(10)
    work = []
    for new in ([1] * 6, [90, 5]):
        s, pages = R.make_seqs(rng, new, [500] * len(new), 32)
        cache = to_dev(R.random_cache(rng, pages, 4, 32, 128))
        q = dev_bf16(bf16_rows(rng, s.tokens, 8, 128))
        b = batch_of(s)
        ws = torch.empty((max(16, W.w8a8_kv_attention_workspace_size(cache, b, s.tokens, 8)),), dtype=torch.uint8, device="cuda")
        work.append((q, cache, b, ws, W.w8a8_kv_attention(q, cache, b, workspace=ws).clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    outs = [torch.empty_like(w[4]) for w in work]
    for _ in range(20):
        for st, (q, cache, b, ws, _), out in zip(streams, work, outs):
            W.w8a8_kv_attention(q, cache, b, out=out, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for w, out in zip(work, outs):
        assert torch.equal(out, w[4])


def test_what_a_call_allocates_belongs_to_the_given_stream():
    """A workspace given back to the current stream could be written there while the call on the other one runs."""
    rng = np.random.default_rng(12)
    s, pages = R.make_seqs(rng, [300, 200], [500, 0], 16)
    cache = R.random_cache(rng, pages, 2, 16, 64)
    q = dev_bf16(bf16_rows(rng, s.tokens, 4, 64))
    c, b = to_dev(cache), batch_of(s)
    want = W.w8a8_kv_attention(q, c, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    taken = set()
    n = W.w8a8_kv_attention_workspace_size(c, b, s.tokens, 4)
    for _ in range(3):
        call = W._kv_call

        def spy(fn, dev_, stream, *args):
            taken.add(args[-2])  # (workspace, its bytes)
            call(fn, dev_, stream, *args)

        W._kv_call = spy
        try:
            out = W.w8a8_kv_attention(q, c, b, stream=side)
        finally:
            W._kv_call = call
        taken.add(out.data_ptr())
        mine = [torch.zeros((size,), dtype=torch.uint8, device="cuda") for size in (n, out.numel() * 2)]
        assert not taken & {t.data_ptr() for t in mine}
        side.synchronize()
        assert torch.equal(out, want)
        del out
    assert status() == 0


def test_offsets_past_32_bits():
    """Pages whose codes lie past 2^32 bytes of the cache."""
    page, hkv, hq, d = 128, 8, 8, 128
    pages = (1 << 32) // (page * hkv * d) + 40
    rng = np.random.default_rng(12)
    k = torch.empty((pages, hkv, page, d), dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = (torch.ones((pages, hkv), device="cuda") for _ in range(2))
    table = (pages - 1 - rng.permutation(8)).astype(np.int32).reshape(2, 4)
    small = R.random_cache(rng, 8, hkv, page, d)
    at = torch.from_numpy(np.sort(table.reshape(-1)).astype(np.int64)).cuda()
    for full, part in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
        full[at] = dev(part)
    c = W.PagedKVCache(k, v, ks, vs)
    low = table - (pages - 8)
    for new, ctx in (([1, 1], [400, 130]), ([60, 90], [300, 0])):
        s = R.Seqs(table, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), np.array(new, np.int32) + np.array(ctx, np.int32))
        s_low = R.Seqs(low, s.start, s.kv)
        x = bf16_rows(rng, s.tokens, hkv, d)
        W.w8a8_kv_append(dev_bf16(x), dev_bf16(x), c, batch_of(s))
        f = synth.bits_to_f32(x)
        small = R.append(small, s_low, f, f)
        assert_same(host(k[at]), small.k, "codes far in the cache")
        assert_same(host(vs[at]), small.vs, "scales far in the cache")
        q = bf16_rows(rng, s.tokens, hq, d)
        out = W.w8a8_kv_attention(dev_bf16(q), c, batch_of(s))
        few = R.few_rows(max(new), hq, small, s_low)
        want, tol = R.attention(small, s_low, synth.bits_to_f32(q), np.float32(d ** -0.5), few=few)
        assert (np.abs(synth.bits_to_f32(host_bf16(out)) - want) <= tol).all()
        ko, vo = W.w8a8_kv_gather(c, dev(table), dev(np.zeros(2, np.int32)),
                                  dev(np.concatenate([[0], np.cumsum(s.kv)]).astype(np.int32)), rows=int(s.kv.sum()),
                                  out_dtype=torch.float32)
        keep = np.zeros((int(s.kv.sum()), hkv, d), np.float32)
        wk, wv = R.gather(small, low, np.zeros(2, np.int32), np.concatenate([[0], np.cumsum(s.kv)]), keep)
        assert_same(host(ko), wk, "k read back")
        assert_same(host(vo), wv, "v read back")
    assert status() == 0


@pytest.mark.parametrize("B,hkv,G,ctx", [(2, 2, 4, 30000), (3, 40, 1, 4300), (40, 8, 2, 600), (9, 3, 8, 1500), (1, 1, 1, 70000)])
def test_attention_single_tokens_at_the_ranges_of_the_cut(B, hkv, G, ctx):
    """Few and many segments, short and long: pieces of warps and of blocks, against the 64-bit reference."""
    rng = np.random.default_rng(ctx)
    ctxs = [ctx] + [int(c) for c in rng.integers(0, ctx, B - 1)]
    s, pages = R.make_seqs(rng, [1] * B, ctxs, 64)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, 64, 128), hkv * G)
