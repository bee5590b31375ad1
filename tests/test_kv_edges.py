"""What the binding of the INT8 paged KV cache hands to the C calls, on a host
without a GPU: row strides of page tables, bounds of any size; and
calls whose grids would pass what a launch holds."""
import pytest
import torch

from int8_gemm_token_b200 import w8a8 as W
from tests.test_kv_cache import append, batch, cache, gather


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


# ------------------------------------------------------------------ page tables whose rows lie in one another
OVERLAPPING = {
    "one row for all": lambda: i32(1, 4).expand(3, 4),
    "one entry for all": lambda: i32(1, 1).expand(3, 1),
    "rows one apart": lambda: i32(6).as_strided((3, 4), (1, 1)),
    "rows three apart": lambda: i32(10).as_strided((3, 4), (3, 1)),
}


@pytest.mark.parametrize("table", OVERLAPPING)
def test_tables_whose_rows_overlap_are_refused(table):
    """Their rows are not max_pages apart: read so, they end past the tensor."""
    t = OVERLAPPING[table]()
    cache = W.PagedKVCache.empty(4, 2, 16, 64, "cpu")
    with pytest.raises(ValueError, match="page_table.*overlap"):
        W.KVBatch(t, i32(4), i32(3), 1)
    with pytest.raises(ValueError, match="page_table.*overlap"):
        W.w8a8_kv_gather(cache, t, i32(3), i32(4), rows=5)
    W.KVBatch(t.contiguous(), i32(4), i32(3), 1)


@pytest.mark.parametrize("table,ld", [
    (lambda: i32(3, 4), 4), (lambda: i32(3, 9)[:, 2:6], 9), (lambda: i32(6, 4)[::2], 8), (lambda: i32(1, 4).expand(1, 4), 4),
    (lambda: i32(8).as_strided((1, 4), (1, 1)), 4), (lambda: i32(3, 0), 1), (lambda: i32(0, 4), 4)])
def test_the_row_stride_of_a_table_is_its_own(table, ld):
    """Of one row (or none) any stride is as good as the row's length."""
    t = table()
    b = W.KVBatch(t, i32(t.shape[0] + 1), i32(t.shape[0]), 1)
    c = b._for(W.PagedKVCache.empty(4, 2, 16, 64, "cpu"))._obj
    assert c.page_table_ld == ld >= t.shape[1]


# ------------------------------------------------------------------ host bounds past the C int
@pytest.mark.parametrize("bound", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63])
def test_bounds_past_int32_stay_bounds(bound):
    """As the C int they would be a small number, or a negative one."""
    cache = W.PagedKVCache.empty(4, 2, 16, 64, "cpu")
    c = W.KVBatch(i32(3, 4), i32(4), i32(3), bound)._for(cache)._obj
    assert c.max_q_len == 2 ** 31 - 1 and c.max_kv_len == 64
    big = W.KVBatch(i32(3, 4), i32(4), i32(3), 1, bound)
    assert big._for(cache)._obj.max_kv_len == 2 ** 31 - 1  # more than the table holds, which the C calls refuse
    assert W.KVBatch(i32(3, 4), i32(4), i32(3), -bound)._for(cache)._obj.max_q_len == -2 ** 31  # refused too
    assert W.w8a8_kv_attention_workspace_size(cache, big, 3, bound + 4) == 0


@pytest.mark.parametrize("window,handed", [(7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                           (-1, -1), (-2 ** 32, -2 ** 31)])
def test_windows_past_int32_stay_windows(monkeypatch, window, handed):
    seen = []
    monkeypatch.setattr(W, "_same_gpu", lambda *a: None)
    monkeypatch.setattr(W, "w8a8_kv_attention_workspace_size", lambda *a: 0)
    monkeypatch.setattr(W, "_kv_call", lambda fn, dev, stream, *args: seen.append(args[7]._obj.window))
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    W.w8a8_kv_attention(q, W.PagedKVCache.empty(4, 2, 16, 64, "cpu"), W.KVBatch(i32(3, 4), i32(4), i32(3), 1), window=window)
    assert seen == [handed]
    with pytest.raises(TypeError):
        W.w8a8_kv_attention(q, W.PagedKVCache.empty(4, 2, 16, 64, "cpu"), W.KVBatch(i32(3, 4), i32(4), i32(3), 1), window=2.5)


# ------------------------------------------------------------------ grids past 2^31 - 1 blocks
def test_appends_of_more_blocks_than_a_launch_holds_are_refused():
    """They would have been cut to the count's low 32 bits, or not been launched at all."""
    plain = dict(cos=None, sin=None, q=None, qo=None)
    wide = dict(c=cache(heads=65535, page=128, d=64), tokens=9)
    # 9 new tokens: a block of 256 threads for each slot of a page, head and of k and v, two slots a sequence
    for n in (8193, 16384, 65535):  # 2^31 blocks and a little more; about 2^32, whose low bits are few; the largest batch
        assert append(b=batch(batch=n, max_q=9), **wide, **plain) == 3
    # query rows: a warp for each 32 heads of 64, 8 of them a block
    assert append(c=cache(d=64), tokens=1 << 30, hq=65535, b=batch(max_q=8), cos=None, sin=None) == 3


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
def test_appends_of_fewer_blocks_are_taken():
    plain = dict(cos=None, sin=None, q=None, qo=None)
    wide = dict(c=cache(heads=65535, page=128, d=64), tokens=9)
    assert append(b=batch(batch=8192, max_q=9), **wide, **plain) == 10  # no device here
    assert append(b=batch(batch=65535, max_q=8), **wide, **plain) == 10  # a warp for each sequence, head and of k and v
    assert gather(c=cache(heads=65535), rows=1 << 20) == 10


def test_read_backs_of_more_blocks_than_a_launch_holds_are_refused():
    assert gather(c=cache(heads=65535), rows=1 << 30) == 3
    assert gather(c=cache(heads=1 << 14, d=64), rows=1 << 24, n=60000) == 3


# ------------------------------------------------------------------ made-up addresses stay on hosts without a GPU
def test_good_calls_with_made_up_addresses_are_skipped_where_a_gpu_is(monkeypatch):
    """test_append_refusals begins with one, whose kernel a GPU would run."""
    from tests import conftest

    class Item:
        def __init__(self, nodeid):
            self.nodeid, self.marks = nodeid, []

        def add_marker(self, mark):
            self.marks.append(mark.name)

    ids = ["tests/test_kv_cache.py::test_append_refusals", "test_kv_cache.py::test_append_refusals",
           "tests/test_kv_cache.py::test_gather_refusals"]
    for gpu, want in ((True, [["skip"], ["skip"], []]), (False, [[], [], []])):
        monkeypatch.setattr(torch.cuda, "is_available", lambda gpu=gpu: gpu)
        items = [Item(i) for i in ids]
        conftest.pytest_collection_modifyitems(items)
        assert [i.marks for i in items] == want


# ------------------------------------------------------------------ what was checked once stays what it was
def test_caches_and_batches_cannot_be_given_other_tensors():
    """The addresses were taken when the object was made: another tensor would not be looked at."""
    c, b = W.PagedKVCache.empty(4, 2, 16, 64, "cpu"), W.KVBatch(i32(3, 4), i32(4), i32(3), 1)
    for obj, names in ((c, ("k_codes", "v_codes", "k_scale", "v_scale", "page_size", "num_pages")),
                       (b, ("page_table", "seq_start", "kv_len", "max_q_len", "max_kv_len"))):
        for name in names:
            was = getattr(obj, name)
            with pytest.raises(AttributeError, match=name):
                setattr(obj, name, torch.ones_like(was) if isinstance(was, torch.Tensor) else 7)
            assert getattr(obj, name) is was
    b.kv_len.fill_(5)  # the contents may change
    b.note = "anything else is the caller's"
    b.note = "and stays so"
