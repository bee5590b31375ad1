"""The INT8 paged KV cache on the GPU at its edges: table entries that no call
needs, ranges of nothing."""
import numpy as np
import pytest
import torch

from int8_gemm_token_b200 import w8a8 as W
from tests import kv_reference as R
from tests.gpu_util import dev, dev_bf16
from tests.test_gpu_kv_cache import batch_of, bf16_rows, status, to_dev

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
