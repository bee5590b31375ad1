"""The INT8 paged KV cache on the GPU at its edges: table entries that no call
needs, ranges of nothing, weights far below a row's largest, bounds
far above the lengths, captured chunks."""
import numpy as np
import pytest
import torch

from int8_gemm_token_b200 import synth
from int8_gemm_token_b200 import w8a8 as W
from tests import kv_reference as R
from tests.gpu_util import dev, dev_bf16, host_bf16
from tests.test_gpu_kv_cache import batch_of, bf16_rows, check_attention, mask_args, status, to_dev

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ pages that no query sees
def unseen_pages(s, page, window, prefix):
    """(sequence, index in its row) of the pages of which no query of the sequence sees a position."""
    for b in range(len(s.kv)):
        n = int(s.kv[b])
        first = max(n - int(s.new[b]), 0)
        low = max(0, first - window + 1) if window else 0
        for p in range(-(-n // page)):
            if p * page >= min(int(prefix[b]), n) and (p + 1) * page <= low:
                yield b, p


@pytest.mark.parametrize("window,prefix", [(16, (0, 0, 0)), (16, (17, 5, 64)), (50, (0, 130, 1)), (129, (33, 0, 400))])
@pytest.mark.parametrize("new", [(1, 1, 1), (6, 1, 3), (40, 1, 65), (130, 90, 7)])
@pytest.mark.parametrize("d,page,hq,hkv", [(128, 16, 4, 4), (64, 32, 8, 2), (96, 16, 16, 1)])
def test_entries_of_pages_that_no_query_sees_are_not_needed(d, page, hq, hkv, new, window, prefix):
    """A sliding window's program gives its oldest pages away: what their entries say is not looked at."""
    rng = np.random.default_rng(window + new[0])
    s, pages = R.make_seqs(rng, list(new), [63, 700, 255], page, spare=1)
    cache = to_dev(R.random_cache(rng, pages, hkv, page, d))
    q = dev_bf16(bf16_rows(rng, s.tokens, hq, d))
    args = dict(window=window, prefix_len=dev(np.array(prefix, np.int32)))
    n = int(s.start[-1])
    assert status() == 0
    want = W.w8a8_kv_attention(q, cache, batch_of(s), **args)[:n].clone()
    given_away = list(unseen_pages(s, page, window, prefix))
    assert given_away
    for entry in (-1, pages, 2 ** 30):
        t = s.table.copy()
        for at in given_away:
            t[at] = entry
        got = W.w8a8_kv_attention(q, cache, batch_of(R.Seqs(t, s.start, s.kv, spare=1)), **args)[:n]
        assert status() == 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("new", [1, 12, 70])
@pytest.mark.parametrize("at", [0, 1, 3, 4, 8])
def test_entries_of_pages_that_a_query_sees_are_needed(new, at):
    """144 positions, of which a prefix of 17 and the last key of page 3 onwards are seen."""
    rng = np.random.default_rng(at)
    s, pages = R.make_seqs(rng, [new], [144 - new], 16)
    cache = to_dev(R.random_cache(rng, pages, 2, 16, 64))
    s.table[0, at] = -1
    assert status() == 0
    W.w8a8_kv_attention(dev_bf16(bf16_rows(rng, s.tokens, 4, 64)), cache, batch_of(s), window=144 - new - 63 + 1,
                        prefix_len=dev(np.array([17], np.int32)))
    assert status() == 11


# ------------------------------------------------------------------ nothing to read
@pytest.mark.parametrize("first", [5, 15, 16, 17, 40])
def test_an_empty_range_reads_no_page(first):
    rng = np.random.default_rng(first)
    cache = to_dev(R.random_cache(rng, 4, 2, 16, 64))
    table = np.full((3, 4), -1, np.int32)
    table[2, :2] = 3, 1
    ko = torch.full((9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    assert status() == 0
    W.w8a8_kv_gather(cache, dev(table), dev(np.array([first, first, 13], np.int32)), dev(np.array([0, 0, 0, 9], np.int32)),
                     k_out=ko)
    assert status() == 0
    x = cache.k_codes.float() * cache.k_scale[:, :, None, None]
    want = torch.cat([x[3, :, 13:], x[1, :, :6]], 1).transpose(0, 1).bfloat16()
    assert torch.equal(ko, want)


# ------------------------------------------------------------------ weights far below the largest
@pytest.mark.parametrize("B,hq,n", [(1776, 1, 1 << 18), (1, 1, 1 << 20), (1, 16, 1 << 20), (1, 1, 1000), (3, 1, 3000)])
@pytest.mark.parametrize("log2_weight", [-26.0, -28.0])
def test_small_weights_of_many_keys_add_up(B, hq, n, log2_weight):
    """B sequences on the same pages, each: one key that takes nearly all the
    weight and holds zeros, in front of a tail of equal keys that hold ones. T =
    (n - 1) 2^log2_weight against the first key's 1 is the tail's, so the output
    is T / (1 + T). Each weight keeps fp16's rounding of 2^-32 of the row's
    largest, so the output is off by at most n 2^-32, and by its rounding to
    bf16. The score is off by a few roundings of its 28 (2^-18), the exponential
    by 2^-22. In the fp32 sum of the weights the one lane of eight that holds
    the 1 may lose its keys of the tail (T / 8); the other lanes' roundings are
    of sums of at most T (2^-13 with all the above)."""
    page, d = 128, 64
    pages = -(-n // page)
    codes = [torch.zeros((pages, 1, page, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    k, v = codes
    k[0, 0, 0, 0] = 64
    v[:] = 1
    v[0, 0, 0] = 0
    ones = torch.ones((pages, 1), device="cuda")
    q = torch.zeros((B, hq, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    b = W.KVBatch(table, dev(np.arange(B + 1, dtype=np.int32)), dev(np.full(B, n, np.int32)), 1)
    scale = -log2_weight * np.log(2.0) / 64
    out = W.w8a8_kv_attention(q, W.PagedKVCache(k, v, ones, ones.clone()), b, scale=scale)
    T = (n - 1) * np.exp(-64 * np.float64(np.float32(scale)))
    want = T / (1 + T)
    got = synth.bits_to_f32(host_bf16(out)).astype(np.float64)
    tol = n * 2.0 ** -32 + want * (2.0 ** -8 + T / 8 + 2.0 ** -13)
    assert (np.abs(got - want) <= tol).all(), (got.min(), got.max(), want, tol)
    assert status() == 0


# ------------------------------------------------------------------ bounds that say little
@pytest.mark.parametrize("mask", ["plain", "window_prefix", "all"])
@pytest.mark.parametrize("d,page,hq,hkv", [(128, 64, 8, 2), (64, 16, 4, 4), (96, 32, 16, 1)])
@pytest.mark.parametrize("new", [(1, 1, 1), (3, 1, 2), (200, 1, 1), (1, 70, 300)])
def test_tables_much_wider_than_the_contexts(d, page, hq, hkv, new, mask):
    """The bound that a table of 40000 positions implies chooses kernels and sizes the workspace, and a batch may mix
    chunks with single tokens."""
    rng = np.random.default_rng(new[0] + d)
    s, pages = R.make_seqs(rng, list(new), [40, 500, 0], page, spare=1, width_extra=40000 // page)
    check_attention(rng, s, R.random_cache(rng, pages, hkv, page, d), hq, **mask_args(mask, hq))


# ------------------------------------------------------------------ many rows in a graph
def test_a_captured_chunk_follows_its_lengths():
    """One captured call (append, attention) of up to 260 new tokens a sequence, replayed for chunks of other lengths,
    equals eager calls."""
    rng = np.random.default_rng(8)
    page, hkv, hq, d, B, rows, most, bound = 16, 2, 8, 128, 3, 420, 260, 800
    table = dev(rng.permutation(B * bound // page).astype(np.int32).reshape(B, -1))
    base = R.random_cache(rng, B * bound // page, hkv, page, d)
    chunks = [([130, 1, 260], [0, 40, 17]), ([260, 160, 0], [540, 0, 300]), ([1, 1, 1], [799, 0, 31]), ([0, 0, 0], [5, 9, 0]),
              ([99, 200, 121], [3, 600, 256])]
    start, kv = dev(np.zeros(B + 1, np.int32)), dev(np.zeros(B, np.int32))
    caches = [to_dev(base), to_dev(base)]
    batch = W.KVBatch(table, start, kv, most, bound)
    cos, sin = (dev(x) for x in R.angles(bound, d))
    x = torch.zeros((rows, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    n = W.w8a8_kv_attention_workspace_size(caches[0], batch, rows, hq)
    ws = [torch.empty((n,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs, qs = ([torch.empty((rows, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2))

    def step(i):
        W.w8a8_kv_append(x[:, hq:hq + hkv], x[:, hq + hkv:], caches[i], batch, cos, sin, q=x[:, :hq], q_out=qs[i])
        W.w8a8_kv_attention(qs[i], caches[i], batch, out=outs[i], workspace=ws[i])

    step(0)  # (no new tokens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    for new, ctx in chunks:
        start.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        kv.copy_(torch.from_numpy(np.array(new, np.int32) + np.array(ctx, np.int32)))
        x.copy_(dev_bf16(bf16_rows(rng, rows, hq + 2 * hkv, d)))
        for t in (*outs, *qs):
            t.fill_(7.0)
        graph.replay()
        step(1)
        assert torch.equal(outs[0], outs[1]) and torch.equal(qs[0], qs[1]), new
        assert (outs[0][sum(new):] == 7).all() and torch.isfinite(outs[0]).all()
        for a, b in zip(caches[0]._tensors, caches[1]._tensors):
            assert torch.equal(a, b)
    assert status() == 0
    graph.reset()
