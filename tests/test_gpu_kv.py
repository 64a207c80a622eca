"""The paged key-value cache on the GPU: rows appended, attention of single tokens and of prompts,
pages handed out, shared, given up, moved and copied, against models in 64 bits and in Python."""
import numpy as np
import pytest
import torch

from kv_common import BAD, E4M3, NO_PAGE, Batch, TableModel, cache_values, nan_cache, quantize_rows

pytestmark = pytest.mark.gpu

bt = pytest.importorskip("binarized_transformer_b200")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    bt.load_library()


def cu(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(news):
    return cu([0] + list(np.cumsum(news)))


# ------------------------------------------------------------------ append
def rows_for_append(n, H, D, kind, seed):
    r = np.random.default_rng([9, seed])
    x = r.standard_normal((n, H, D)) * np.exp(2 * r.standard_normal((n, H, 1)))
    x[r.random((n, H)) < 0.1] = 0.0                           # rows of zeros
    x[r.random((n, H)) < 0.1] *= 2.0 ** -18                   # towards fp16's smallest
    x[r.random((n, H)) < 0.1] *= 2.0 ** 12
    hit = r.random((n, H)) < 0.1                              # a largest value on the border 448 * 2^e
    x[hit, 0] = 448.0 * 2.0 ** r.integers(-15, 7, hit.sum())
    x = np.clip(x, -65504, 65504)
    x[r.random((n, H, D)) < 0.02] = -0.0
    return x.astype(np.float16 if kind == "f16" else np.float32)


@pytest.mark.parametrize("H,D,ps,news,lens,pad", [
    (1, 8, 16, [1, 1, 1], [1, 16, 17], 0),
    (2, 64, 16, [1] * 5, [5, 100, 33, 32, 1], 16),
    (3, 128, 48, [7, 0, 60, 1], [7, 20, 200, 49], 0),
    (8, 96, 32, [33, 64], [40, 64], 32),
    (1, 40, 64, [130], [130], 0),
])
@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append(H, D, ps, news, lens, pad, kind, e4m3):
    b = Batch(bt, [0] * len(lens), ps, H, D, e4m3, pad=pad)
    m = TableModel(b.table.pages.shape[0], b.table.pages.shape[1], 0, ps)
    # a pool and rows of its own for these lengths
    need = [-(-n // ps) for n in lens]
    cache = nan_cache(bt, sum(need) + 2, ps, H, D, e4m3, pad)
    n_slots = len(lens) + 1
    order = np.random.default_rng(3).permutation(sum(need) + 2)
    slot_of = np.random.default_rng(4).permutation(n_slots)[:len(lens)].astype(np.int32)
    pages = np.full((n_slots, max(need)), -1, np.int32)
    at = 0
    for s, k in enumerate(need):
        pages[slot_of[s], :k] = order[at:at + k]
        at += k
    kv_len = np.zeros(n_slots, np.int32)
    kv_len[slot_of] = lens
    table = bt.KvTable(torch.from_numpy(pages).cuda(), cu(kv_len.tolist()))
    n = sum(news)
    step = all(x == 1 for x in news)
    extra = 0 if step else 3                                  # rows behind the last sequence
    k, v = (rows_for_append(n + extra, H, D, kind, i) for i in (0, 1))
    before = cache_values(cache)
    raw = [t.clone() for t in (cache.k, cache.v)]
    status = bt.new_status()
    wide = torch.zeros((n + extra, H * D + 16), dtype=torch.float16 if kind == "f16" else torch.float32, device="cuda")
    wide[:, :H * D] = torch.from_numpy(k.reshape(n + extra, -1)).cuda()
    bt.bwta_kv_append(cache, table, wide[:, :H * D], torch.from_numpy(v).cuda(), slots=cu(slot_of.tolist()),
                      cu_q=None if step else offsets(news), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for x, t, sc, old in ((k, cache.k, cache.k_scale, raw[0]), (v, cache.v, cache.v_scale, raw[1])):
        want = old.cpu().numpy().copy()
        wsc = None if sc is None else np.full(sc.shape, np.nan, np.float32)
        codes, scales = quantize_rows(x) if e4m3 else (None, None)
        row = 0
        for s in range(len(lens)):
            for p in range(lens[s] - news[s], lens[s]):
                page = pages[slot_of[s], p // ps]
                if e4m3:
                    want[page, :, p % ps] = codes[row]
                    wsc[page, :, p % ps] = scales[row]
                else:
                    want[page, :, p % ps] = x[row].astype(np.float16)
                row += 1
        got = t.cpu().numpy()
        bits = np.uint8 if e4m3 else np.uint16
        np.testing.assert_array_equal(np.ascontiguousarray(got).view(bits), np.ascontiguousarray(want).view(bits))
        if e4m3:
            np.testing.assert_array_equal(sc.cpu().numpy(), wsc)


def test_append_bad_entries_and_values():
    H, D, ps = 2, 64, 16
    cache = nan_cache(bt, 4, ps, H, D, False)
    # slot 0: page past the pool; 1: negative page; 2: longer than its row; 3: fine; 4: empty
    table = bt.KvTable(cu([[4, 0], [-1, 0], [1, 2], [3, 0], [0, 0]]), cu([1, 1, 33, 1, 0]))
    x = torch.ones((6, H * D), device="cuda")
    status = bt.new_status()
    before = cache.k.clone()
    bt.bwta_kv_append(cache, table, x, x, slots=cu([0, 1, 2, 4, 5, -1]), status=status)
    torch.cuda.synchronize()
    assert status.item() == BAD
    assert torch.equal(before.view(torch.int16), cache.k.view(torch.int16))
    status.zero_()
    bt.bwta_kv_append(cache, table, x[:1], x[:1], slots=cu([3]), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and (cache.k[3, :, 0] == 1).all()
    for e4m3 in (False, True):
        for value in (float("nan"), float("inf"), 70000.0, 65520.0):
            c = nan_cache(bt, 4, ps, H, D, e4m3)
            status.zero_()
            y = x[:1].clone()
            y[0, 77] = value
            bt.bwta_kv_append(c, table, y, x[:1], slots=cu([3]), status=status)
            torch.cuda.synchronize()
            assert status.item() == bt.STATUS_NONFINITE, (e4m3, value)
            # the other head's row is what it should be
            assert (cache_values(c)[0][3, 0, 0] == 1).all()


# ------------------------------------------------------------------ attention of single tokens
DECODE = [
    # H, G, D, ps, lens, window, sinks
    (1, 1, 64, 16, [1], 0, 0),
    (2, 1, 128, 16, [0, 1, 15, 16, 17, 63, 64, 65], 0, 0),
    (1, 8, 128, 32, [129, 1000, 2], 0, 0),
    (3, 5, 40, 16, [77, 300, 31], 0, 0),
    (2, 16, 96, 48, [511, 48, 47], 0, 0),
    (1, 20, 64, 64, [200, 1], 0, 0),
    (2, 4, 128, 128, [900, 128, 5], 100, 0),
    (2, 2, 64, 16, [700, 33, 1, 260], 37, 5),
    (1, 3, 8, 16, [100, 400], 1, 0),
    (4, 1, 112, 256, [1000, 300], 64, 100),
    (2, 8, 128, 16, [5000, 3], 0, 0),
    (1, 2, 80, 16, [3000, 2999], 1024, 65),
    (12, 1, 64, 16, [40] * 30, 0, 0),
]


@pytest.mark.parametrize("H,G,D,ps,lens,window,sinks", DECODE)
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode(H, G, D, ps, lens, window, sinks, e4m3):
    b = Batch(bt, lens, ps, H, D, e4m3, seed=len(lens) + D)
    heads = H * G
    q = b.queries(len(lens), heads)
    wide = torch.zeros((len(lens), heads * D + 8), dtype=torch.float16, device="cuda")
    wide[:, :heads * D] = torch.from_numpy(q.reshape(len(lens), -1)).cuda()
    qt = wide[:, :heads * D].unflatten(1, (heads, D))
    status = bt.new_status()
    out = bt.bwta_attn_decode_paged(qt, b.cache, b.table, D ** -0.5, window, sinks, slots=b.slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    b.check(q, out, [1 if n else 0 for n in lens] if 0 not in lens else [1] * len(lens), D ** -0.5, window, sinks)


@pytest.mark.parametrize("H,G,D,ps,lens,window,sinks", DECODE)
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_in_long_rows(H, G, D, ps, lens, window, sinks, e4m3):
    """The same sequences in a table with room for long ones: the lengths are not bounded by its rows,
    and the tiles of all sequences are shared out over the GPU."""
    b = Batch(bt, lens, ps, H, D, e4m3, seed=len(lens) + D)
    rows = torch.full((b.table.pages.shape[0], (1 << 20) // ps), -1, dtype=torch.int32, device="cuda")
    rows[:, :b.max_pages] = b.table.pages
    table = bt.KvTable(rows, b.table.kv_len)
    q = b.queries(len(lens), H * G)
    qt = torch.from_numpy(q).cuda()
    status = bt.new_status()
    out = bt.bwta_attn_decode_paged(qt, b.cache, table, D ** -0.5, window, sinks, slots=b.slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    b.check(q, out, [1] * len(lens), D ** -0.5, window, sinks)


@pytest.mark.parametrize("n,H,G,ps,most", [(1, 1, 1, 16, 333), (1, 32, 1, 16, 333), (3, 8, 8, 32, 1000), (5, 12, 1, 16, 700),
                                           (17, 8, 4, 64, 500), (1, 4, 16, 16, 4000), (27, 8, 3, 16, 100)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_of_few_items(n, H, G, ps, most, e4m3):
    """Around the sizes at which clusters of 8, 4 and 2 blocks take an item, empty sequences among them."""
    r = np.random.default_rng(n)
    lens = [most] + r.integers(0, most, n - 1).tolist()
    if n > 2:
        lens[1] = 0
    b = Batch(bt, lens, ps, H, 64, e4m3, seed=n)
    q = b.queries(n, H * G)
    qt = torch.from_numpy(q).cuda()
    for window, sinks in ((0, 0), (100, 7)):
        status = bt.new_status()
        out = bt.bwta_attn_decode_paged(qt, b.cache, b.table, 0.125, window, sinks, slots=b.slots, status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        b.check(q, out, [1] * n, 0.125, window, sinks)
        assert torch.equal(out, bt.bwta_attn_decode_paged(qt, b.cache, b.table, 0.125, window, sinks, slots=b.slots))


def test_decode_long_split():
    """One long sequence beside empty and short ones: the length is split over many blocks and joined."""
    lens = [70001, 0, 3, 20000]
    b = Batch(bt, lens, 64, 2, 64, True, seed=5)
    q = b.queries(4, 8, size=2.0)
    out = bt.bwta_attn_decode_paged(torch.from_numpy(q).cuda(), b.cache, b.table, 0.2, slots=b.slots)
    torch.cuda.synchronize()
    b.check(q, out, [1] * 4, 0.2)
    again = bt.bwta_attn_decode_paged(torch.from_numpy(q).cuda(), b.cache, b.table, 0.2, slots=b.slots)
    assert torch.equal(out, again)                            # the same order of sums in every run


# ------------------------------------------------------------------ attention of prompts
PROMPT = [
    # H, G, D, ps, lens, news, window, sinks
    (1, 1, 64, 16, [1], [1], 0, 0),
    (2, 1, 128, 16, [17, 128, 129], [17, 128, 129], 0, 0),
    (1, 4, 128, 32, [300, 40, 500], [300, 0, 77], 0, 0),
    (2, 3, 64, 48, [260, 131], [260, 131], 0, 0),
    (1, 8, 128, 64, [1000], [333], 0, 0),
    (1, 7, 96, 16, [200, 90, 3], [5, 90, 3], 0, 0),
    (2, 1, 64, 128, [700, 520], [700, 300], 100, 0),
    (1, 2, 128, 16, [900], [900], 130, 4),
    (1, 1, 40, 256, [600], [100], 1, 0),
    (2, 2, 80, 16, [1500], [400], 257, 140),
    (1, 16, 32, 16, [333, 50], [333, 50], 64, 1),
    (1, 100, 64, 16, [70], [9], 0, 0),
    (12, 1, 64, 16, [100, 31, 257], [100, 31, 257], 0, 0),
]


@pytest.mark.parametrize("H,G,D,ps,lens,news,window,sinks", PROMPT)
@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt(H, G, D, ps, lens, news, window, sinks, e4m3):
    b = Batch(bt, lens, ps, H, D, e4m3, seed=len(lens) + D)
    heads, n = H * G, sum(news)
    q = b.queries(n + 3, heads)
    qt = torch.from_numpy(q).cuda()
    out = torch.full((n + 3, heads, D), 7.5, dtype=torch.float16, device="cuda")
    status = bt.new_status()
    bt.bwta_attn_prompt_paged(qt, offsets(news), b.cache, b.table, D ** -0.5, window, sinks, slots=b.slots,
                              status=status, out=out)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert (out[n:] == 7.5).all()
    b.check(q, out, news, D ** -0.5, window, sinks, rows=24)


@pytest.mark.parametrize("H,G,D,ps,lens,news,window,sinks", [
    (1, 1, 64, 16, [5000], [3], 0, 0),
    (2, 8, 128, 32, [3000, 9, 700], [5, 9, 1], 0, 0),
    (1, 4, 128, 64, [6000], [70], 2000, 300),
    (1, 3, 40, 48, [2000, 1], [50, 1], 0, 0),
    (4, 2, 96, 16, [513, 0, 1500], [130, 0, 200], 900, 1),
    (1, 1, 128, 16, [1030], [300], 0, 0),
    (1, 16, 80, 128, [4000], [17], 100, 2000),
])
@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_of_few_rows(H, G, D, ps, lens, news, window, sinks, e4m3):
    """Few rows over long caches: the keys of a tile are shared out and the parts added up."""
    b = Batch(bt, lens, ps, H, D, e4m3, seed=len(lens) + D)
    q = b.queries(sum(news), H * G, size=2.0)
    status = bt.new_status()
    args = (torch.from_numpy(q).cuda(), offsets(news), b.cache, b.table, D ** -0.5, window, sinks)
    out = bt.bwta_attn_prompt_paged(*args, slots=b.slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    b.check(q, out, news, D ** -0.5, window, sinks, rows=24)
    assert torch.equal(out, bt.bwta_attn_prompt_paged(*args, slots=b.slots))


def test_prompt_rows_before_the_first_token_are_zero():
    b = Batch(bt, [5, 0], 16, 1, 64)
    q = torch.from_numpy(b.queries(12, 2)).cuda()
    out = bt.bwta_attn_prompt_paged(q, cu([0, 8, 12]), b.cache, b.table, 0.125, slots=b.slots)
    torch.cuda.synchronize()
    assert (out[:3] == 0).all() and (out[8:] == 0).all()
    b.check(q.cpu().numpy()[3:8], out[3:8], [5], 0.125)


def test_prompt_and_single_tokens_agree():
    """The last row of a prompt is the single-token call's row."""
    b = Batch(bt, [777], 16, 2, 128, True)
    q = b.queries(1, 8)
    qt = torch.from_numpy(q).cuda()
    a = bt.bwta_attn_decode_paged(qt, b.cache, b.table, 0.09, 200, 9, slots=b.slots)
    c = bt.bwta_attn_prompt_paged(qt, cu([0, 1]), b.cache, b.table, 0.09, 200, 9, slots=b.slots)
    b.check(q, a, [1], 0.09, 200, 9)
    b.check(q, c, [1], 0.09, 200, 9)


def test_large_scores_and_equal_scores():
    """Scores of thousands (one key takes all) and rows of equal scores (the mean of V)."""
    b = Batch(bt, [300, 200], 16, 1, 64, k_scale=30.0)
    q = b.queries(2, 4, size=30.0)
    qt = torch.from_numpy(q).cuda()
    out = bt.bwta_attn_decode_paged(qt, b.cache, b.table, 1.0, slots=b.slots)
    b.check(q, out, [1, 1], 1.0)
    out = bt.bwta_attn_prompt_paged(qt, cu([0, 1, 2]), b.cache, b.table, 1.0, slots=b.slots)
    b.check(q, out, [1, 1], 1.0)
    zero = np.zeros_like(q)
    for o in (bt.bwta_attn_decode_paged(torch.zeros_like(qt), b.cache, b.table, 1.0, slots=b.slots),
              bt.bwta_attn_prompt_paged(torch.zeros_like(qt), cu([0, 1, 2]), b.cache, b.table, 1.0, slots=b.slots)):
        b.check(zero, o, [1, 1], 1.0)


@pytest.mark.parametrize("D,slope", [(64, 0.05), (128, 0.02), (64, -0.05), (40, 0.5)])
def test_scores_that_keep_rising(D, slope):
    """Each key scores above (or below) the one before: the running maximum moves all the way."""
    t, n = 1300, 400
    b = Batch(bt, [t], 16, 1, D)
    k = np.repeat((np.arange(t) * slope % 64.0)[:, None], D, 1) if abs(slope) > 0.1 else \
        np.repeat((np.arange(t) * slope)[:, None], D, 1)
    b.k[0] = k[None].astype(np.float16).astype(np.float64)
    for i in range(-(-t // 16)):
        m = min(16, t - i * 16)
        page = b.table.pages[b.slot_of[0], i].item()
        b.cache.k[page, 0, :m] = torch.from_numpy(b.k[0][0, i * 16:i * 16 + m].astype(np.float16)).cuda()
    q = np.abs(b.queries(n, 2)) + np.float16(0.5)
    qt = torch.from_numpy(q).cuda()
    status = bt.new_status()
    out = bt.bwta_attn_prompt_paged(qt, cu([0, n]), b.cache, b.table, 0.125, slots=b.slots, status=status)
    b.check(q, out, [n], 0.125, rows=40)
    out = bt.bwta_attn_decode_paged(qt[-1:], b.cache, b.table, 0.125, slots=b.slots, status=status)
    b.check(q[-1:], out, [1], 0.125)
    assert status.item() == 0


def test_nonfinite_keys_are_flagged_wherever_they_lie():
    b = Batch(bt, [300], 16, 1, 64)
    q = torch.from_numpy(b.queries(10, 3)).cuda()
    for j in (0, 1, 15, 16, 63, 64, 127, 128, 200, 289):
        page = b.table.pages[b.slots[0].item(), j // 16].item()
        for value in (float("nan"), float("inf")):
            was = b.cache.k[page, 0, j % 16, 7].item()
            b.cache.k[page, 0, j % 16, 7] = value
            for f in (lambda **kw: bt.bwta_attn_decode_paged(q[-1:], b.cache, b.table, 0.125, **kw),
                      lambda **kw: bt.bwta_attn_prompt_paged(q, cu([0, 10]), b.cache, b.table, 0.125, **kw)):
                status = bt.new_status()
                f(slots=b.slots, status=status)
                torch.cuda.synchronize()
                assert status.item() == bt.STATUS_NONFINITE, (j, value)
            b.cache.k[page, 0, j % 16, 7] = was


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_with_bad_entries(e4m3):
    """Pages and slots outside, lengths past the row: flagged, nothing else disturbed."""
    b = Batch(bt, [100, 60, 40], 16, 2, 64, e4m3)
    pages = b.table.pages.clone()
    pages[b.slots[0].item(), 2] = b.num_pages + 5
    pages[b.slots[1].item(), 1] = -7
    kv_len = b.table.kv_len.clone()
    t = bt.KvTable(pages, kv_len)
    q = b.queries(3, 4)
    qt = torch.from_numpy(q).cuda()
    for news in (None, [1, 1, 1]):
        status = bt.new_status()
        args = dict(slots=b.slots, status=status)
        out = (bt.bwta_attn_decode_paged(qt, b.cache, t, 0.125, **args) if news is None else
               bt.bwta_attn_prompt_paged(qt, offsets(news), b.cache, t, 0.125, **args))
        torch.cuda.synchronize()
        assert status.item() & BAD
        assert status.item() & ~(BAD | bt.STATUS_NONFINITE) == 0
        sub = Batch.__new__(Batch)
        sub.__dict__.update(b.__dict__)
        sub.lens, sub.k, sub.v = [40], b.k[2:], b.v[2:]
        sub.check(q[2:], out[2:], [1], 0.125)
    status = bt.new_status()
    long = bt.KvTable(b.table.pages, torch.full_like(kv_len, 1 << 20))
    bt.bwta_attn_decode_paged(qt, b.cache, long, 0.125, slots=cu([0, 99, -1]), status=status)
    torch.cuda.synchronize()
    assert status.item() & BAD


def test_nonfinite_inputs_are_flagged():
    b = Batch(bt, [50], 16, 1, 64)
    page = b.table.pages[b.slots[0].item(), 0].item()
    b.cache.v[page, 0, 3, 5] = float("inf")
    q = torch.from_numpy(b.queries(1, 1)).cuda()
    for f in (lambda **kw: bt.bwta_attn_decode_paged(q, b.cache, b.table, 0.125, **kw),
              lambda **kw: bt.bwta_attn_prompt_paged(q, cu([0, 1]), b.cache, b.table, 0.125, **kw)):
        status = bt.new_status()
        f(slots=b.slots, status=status)
        torch.cuda.synchronize()
        assert status.item() == bt.STATUS_NONFINITE
        status.zero_()
        f(window=40, slots=b.slots, status=status)            # key 3 is hidden now
        torch.cuda.synchronize()
        assert status.item() == 0


def far_batch(lens, ps, H, D, e4m3, seed, gap):
    """A batch whose pages lie `gap` elements apart: offsets pass 32 bits."""
    b = Batch(bt, lens, ps, H, D, e4m3, seed=seed)
    n = H * ps * D
    ns = H * ps

    def spread(t, step, inner):
        buf = torch.empty(b.num_pages * step, dtype=t.dtype, device="cuda")
        far = buf.as_strided(t.shape, (step, *inner))
        far.copy_(t)
        return far
    k, v = (spread(t, gap, (ps * D, D, 1)) for t in (b.cache.k, b.cache.v))
    sc = [None if t is None else spread(t, ns + 4, (ps, 1)) for t in (b.cache.k_scale, b.cache.v_scale)]
    assert gap >= n and (b.num_pages - 1) * gap > 1 << 32
    b.cache = bt.KvCache(k, v, *sc)
    return b


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_32_bits(e4m3):
    """Pages 2^28 elements apart (a pool of 2^32 and more): append, both attentions, copies."""
    lens = [200, 90]
    b = far_batch(lens, 16, 2, 64, e4m3, 3, 1 << 28)
    q = b.queries(2, 4)
    qt = torch.from_numpy(q).cuda()
    out = bt.bwta_attn_decode_paged(qt, b.cache, b.table, 0.125, slots=b.slots)
    b.check(q, out, [1, 1], 0.125)
    out = bt.bwta_attn_prompt_paged(qt, cu([0, 1, 2]), b.cache, b.table, 0.125, slots=b.slots)
    b.check(q, out, [1, 1], 0.125)
    slot = b.slot_of[0]
    last = b.table.pages[slot, (lens[0] - 1) // 16].item()
    ones = torch.ones((1, 2, 64), device="cuda")
    bt.bwta_kv_append(b.cache, b.table, ones, ones, slots=b.slots[:1])
    assert (cache_values(type("C", (), dict(k=b.cache.k[last:last + 1], v=b.cache.v[last:last + 1],
                                            k_scale=b.cache.k_scale[last:last + 1] if e4m3 else None,
                                            v_scale=b.cache.v_scale[last:last + 1] if e4m3 else None)))[0]
            [0, :, (lens[0] - 1) % 16] == 1).all()
    free = b.num_pages - 1 if last != b.num_pages - 1 else b.num_pages - 2
    bt.bwta_kv_copy_pages(b.cache, b.cache, cu([last]), cu([free]))
    torch.cuda.synchronize()
    assert torch.equal(b.cache.k[last].view(torch.uint8), b.cache.k[free].view(torch.uint8))
    assert torch.equal(b.cache.v[last].view(torch.uint8), b.cache.v[free].view(torch.uint8))


@pytest.mark.parametrize("H,G,D,ps,lens,news,window,sinks", [
    (1, 2, 8, 16, [150, 33], [150, 20], 0, 0),
    (2, 1, 24, 1024, [1500, 1024], [260, 129], 0, 0),
    (1, 9, 104, 48, [400], [90], 70, 40),
    (1, 2, 120, 65536, [700, 1], [300, 1], 0, 0),
    (3, 2, 72, 112, [333, 112], [111, 112], 50, 3),
    (1, 128, 64, 16, [40], [3], 0, 0),
])
@pytest.mark.parametrize("e4m3", [False, True])
def test_odd_widths_pages_and_strides(H, G, D, ps, lens, news, window, sinks, e4m3):
    """Head widths that are not multiples of 16, long pages, rows of q and out further apart than dense."""
    b = Batch(bt, lens, ps, H, D, e4m3, seed=D)
    heads, n = H * G, sum(news)
    q = b.queries(n, heads)
    for prompt in (True, False):
        rows = n if prompt else len(lens)
        buf = torch.full((2, rows, heads * D + 24), 3.25, dtype=torch.float16, device="cuda")
        qt, out = (x[:, :heads * D].unflatten(1, (heads, D)) for x in buf)
        qt.copy_(torch.from_numpy(q[:rows]))
        status = bt.new_status()
        args = dict(slots=b.slots, status=status, out=out)
        if prompt:
            bt.bwta_attn_prompt_paged(qt, offsets(news), b.cache, b.table, D ** -0.5, window, sinks, **args)
        else:
            bt.bwta_attn_decode_paged(qt, b.cache, b.table, D ** -0.5, window, sinks, **args)
        torch.cuda.synchronize()
        assert status.item() == 0 and (buf[:, :, heads * D:] == 3.25).all()
        b.check(q, out, news if prompt else [1] * len(lens), D ** -0.5, window, sinks, rows=16)


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_prompt_follows_the_lengths(e4m3):
    """One graph, replayed while the sequences grow: short, then long enough to be shared out."""
    b = Batch(bt, [2500, 1800], 32, 2, 64, e4m3, seed=9)
    q = b.queries(40, 6)
    qt = torch.from_numpy(q).cuda()
    off = cu([0, 30, 40])
    full = b.table.kv_len.clone()
    out = torch.empty_like(qt)
    bt.bwta_attn_prompt_paged(qt, off, b.cache, b.table, 0.125, slots=b.slots, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.bwta_attn_prompt_paged(qt, off, b.cache, b.table, 0.125, slots=b.slots, out=out)
    for cut in ((2500, 1800), (35, 10), (130, 700), (2500, 11)):
        b.table.kv_len[b.slots.long()] = cu(list(cut))
        graph.replay()
        torch.cuda.synchronize()
        sub = Batch.__new__(Batch)
        sub.__dict__.update(b.__dict__)
        sub.lens = list(cut)
        sub.k, sub.v = ([x[:, :t] for x, t in zip(y, cut)] for y in (b.k, b.v))
        sub.check(q, out, [30, 10], 0.125, rows=16)
    b.table.kv_len.copy_(full)
    graph.reset()


def test_two_streams_at_once():
    """Both attentions on two streams, many calls each, beside one another: no result depends on the other."""
    b = Batch(bt, [3000, 500, 77], 16, 2, 128, True, seed=12)
    q = torch.from_numpy(b.queries(60, 8)).cuda()
    off = cu([0, 20, 40, 60])
    want_d = bt.bwta_attn_decode_paged(q[:3], b.cache, b.table, 0.09, slots=b.slots)
    want_p = bt.bwta_attn_prompt_paged(q, off, b.cache, b.table, 0.09, slots=b.slots)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            got.append((bt.bwta_attn_decode_paged(q[:3], b.cache, b.table, 0.09, slots=b.slots),
                        bt.bwta_attn_prompt_paged(q, off, b.cache, b.table, 0.09, slots=b.slots)))
    torch.cuda.synchronize()
    assert all(torch.equal(d, want_d) and torch.equal(p, want_p) for d, p in got)


# ------------------------------------------------------------------ pages
def mirror(table, m):
    assert table.pages.cpu().tolist() == m.pages
    assert table.kv_len.cpu().tolist() == m.len
    assert table.refcount.cpu().tolist() == m.ref


@pytest.mark.parametrize("seed,num_pages,ps,n_slots,max_pages", [
    (0, 40, 16, 6, 12), (1, 7, 16, 5, 9), (2, 300, 32, 40, 20), (3, 33, 16, 12, 4), (4, 3000, 16, 64, 100),
    (5, 1, 16, 3, 2), (6, 100, 48, 9, 1100),
])
def test_pages_random_walk(seed, num_pages, ps, n_slots, max_pages):
    """Random requests, valid and not, against the Python model; every page's bytes follow."""
    r = np.random.default_rng([11, seed])
    e4m3 = bool(seed % 2)
    layers = [nan_cache(bt, num_pages, ps, 1, 8, e4m3, 16 * (seed % 3)) for _ in range(1 + seed % 3)]
    for c in layers:                                          # every page distinct
        for t in (c.k, c.v) + ((c.k_scale, c.v_scale) if e4m3 else ()):
            src = r.integers(1, 100, t.shape)
            t.copy_(torch.from_numpy(src))
    data = [[t.cpu().clone() for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None] for c in layers]
    table = bt.KvTable.empty(n_slots, max_pages, num_pages)
    m = TableModel(n_slots, max_pages, num_pages, ps)
    status = bt.new_status()

    def pick(n, junk=0.1):
        s = r.integers(0, n_slots, n)
        return [int(x) if r.random() > junk else int(r.choice([-1, n_slots, 1 << 30, -(1 << 31)])) for x in s]

    for _ in range(40):
        do = r.integers(0, 4)
        n = int(r.integers(1, 2 * n_slots))
        copies = []
        if do == 0:
            s = pick(n)
            g = [int(x) for x in r.integers(-1, max(2, num_pages * ps // n_slots), n)]
            m.reserve(s, g)
            bt.bwta_kv_reserve(table, ps, cu(s), cu(g), status=status)
        elif do == 1:
            s = pick(max(1, n // 3))
            m.free(s)
            bt.bwta_kv_free(table, ps, cu(s), status=status)
        elif do == 2:
            a, d = pick(n, 0.03), pick(n, 0.03)
            copies = m.fork(a, d)
            bt.bwta_kv_fork(layers, table, cu(a), cu(d), status=status)
        else:
            copies, used = m.compact()
            assert bt.bwta_kv_compact(layers, table, status=status).item() == used
        for c in data:
            for t in c:
                if copies:
                    t[[b for _, b in copies]] = t[[a for a, _ in copies]]
        torch.cuda.synchronize()
        mirror(table, m)
        assert status.item() == m.status
        status.zero_()
        m.status = 0
    for c, want in zip(layers, data):
        for t, w in zip([t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None], want):
            assert torch.equal(t.cpu(), w)


def test_reserve_all_or_nothing_order():
    t = bt.KvTable.empty(4, 8, 5)
    m = TableModel(4, 8, 5, 16)
    status = bt.new_status()
    for s, g in (([0, 1, 2], [33, 40, 1]), ([3, 0, 1], [0, 15, 1]), ([0, 0], [1, 1]), ([2], [129]), ([2], [1 << 30])):
        m.reserve(s, g)
        bt.bwta_kv_reserve(t, 16, cu(s), cu(g), status=status)
        torch.cuda.synchronize()
        mirror(t, m)
        assert status.item() == m.status
    assert m.status == BAD | NO_PAGE


@pytest.mark.parametrize("n", [1, 700, 2048])
def test_long_lists(n):
    t, m = bt.KvTable.empty(n, 3, 4 * n), TableModel(n, 3, 4 * n, 16)
    r = np.random.default_rng(n)
    s, g = r.permutation(n).tolist(), r.integers(0, 48, n).tolist()
    m.reserve(s, g)
    bt.bwta_kv_reserve(t, 16, cu(s), cu(g))
    torch.cuda.synchronize()
    mirror(t, m)


def test_pages_with_broken_tables():
    """Rows that name pages outside the pool, pages that nobody counts, lengths past the row."""
    ps, num = 16, 6
    cache = nan_cache(bt, num, ps, 1, 8, False)
    status = bt.new_status()
    t = bt.KvTable(cu([[9, 1, -1], [5, 5, 2], [-1, -1, -1], [-1, -1, -1]]), cu([32, 40, 0, 0]), cu([0, 1, 1, 0, 0, 0]))
    bt.bwta_kv_fork([cache], t, cu([0]), cu([2]), status=status)
    torch.cuda.synchronize()
    assert status.item() == BAD and t.pages[2].tolist() == [9, 1, -1] and t.refcount.tolist() == [0, 2, 1, 0, 0, 0]
    status.zero_()
    n = bt.bwta_kv_compact([cache], t, status=status)         # pages 1, 2 in use: 2 -> 0; slot 1 names 5, uncounted
    torch.cuda.synchronize()
    assert n.item() == 2 and status.item() == BAD
    assert t.pages.tolist() == [[9, 1, -1], [5, 5, 0], [9, 1, -1], [-1, -1, -1]]
    assert t.refcount.tolist() == [1, 2, 0, 0, 0, 0]
    status.zero_()
    bt.bwta_kv_free(t, ps, cu([0, 1, 0]), status=status)
    torch.cuda.synchronize()
    assert status.item() == BAD and t.refcount.tolist() == [0, 1, 0, 0, 0, 0]
    status.zero_()
    t = bt.KvTable(cu([[0, 1], [-1, -1]]), cu([33, 0]), cu([1, 1, 0, 0, 0, 0]))
    bt.bwta_kv_reserve(t, ps, cu([0]), cu([1]), status=status)
    bt.bwta_kv_fork([cache], t, cu([0]), cu([1]), status=status)
    torch.cuda.synchronize()
    assert status.item() == BAD and t.pages.tolist() == [[0, 1], [-1, -1]] and t.kv_len.tolist() == [33, 0]


@pytest.mark.parametrize("e4m3", [False, True])
def test_copy_pages(e4m3):
    ps, H, D, n = 16, 3, 40, 50
    r = np.random.default_rng(2)
    a = [nan_cache(bt, n, ps, H, D, e4m3) for _ in range(2)]
    b = [nan_cache(bt, n + 9, ps, H, D, e4m3, 16) for _ in range(2)]

    def tensors(c):
        return [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]
    for c in a + b:
        for t in tensors(c):
            t.copy_(torch.from_numpy(r.integers(1, 100, t.shape)))
    src, dst = [0, 7, 49, 50, 3, 3, 8, -1, 12], [58, 0, 5, 1, 59, -1, 6, 2, 6]
    want = [[t.cpu().clone() for t in tensors(c)] for c in b]
    for c, w in zip(a, want):
        for t, x in zip(tensors(c), w):
            for s, d in ((0, 58), (7, 0), (49, 5)):           # the others: out of range, or 6 written twice
                x[d] = t[s].cpu()
    status = bt.new_status()
    bt.bwta_kv_copy_pages(a, b, cu(src), cu(dst), status=status)
    torch.cuda.synchronize()
    assert status.item() == BAD
    for c, w in zip(b, want):
        assert all(torch.equal(t.cpu(), x) for t, x in zip(tensors(c), w))
    # within one pool: 1 -> 2 -> 3 is refused where it reads what the list writes
    status.zero_()
    want = [t.cpu().clone() for t in tensors(a[0])]
    for x in want:
        x[2] = x[1]
        x[4] = x[0]
    bt.bwta_kv_copy_pages(a[0], a[0], cu([1, 2, 0, 5]), cu([2, 3, 4, 5]), status=status)
    torch.cuda.synchronize()
    assert status.item() == BAD
    assert all(torch.equal(t.cpu(), x) for t, x in zip(tensors(a[0]), want))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_run(e4m3):
    """Prompts, forks, single tokens, a compaction and single tokens again, as a server would: every
    attention against 64 bits over the tokens that the cache should hold."""
    H, G, D, ps, n_slots = 2, 4, 64, 16, 6
    r = np.random.default_rng(21)
    cache = nan_cache(bt, 60, ps, H, D, e4m3)
    layers = bt.kv_layers(cache)
    table = bt.KvTable.empty(n_slots, 20, 60)
    status = bt.new_status()
    hist = {s: (np.zeros((H, 0, D)), np.zeros((H, 0, D))) for s in range(n_slots)}

    def held(x):
        if not e4m3:
            return x.astype(np.float16).astype(np.float64)
        codes, sc = quantize_rows(x)
        return E4M3[codes] * sc[..., None]

    def step(slots, news, window=0, sinks=0):
        n = sum(news)
        k, v = (r.standard_normal((n, H, D)).astype(np.float32) for _ in range(2))
        q = r.standard_normal((n, H * G, D)).astype(np.float16)
        single = all(x == 1 for x in news)
        off = None if single else offsets(news)
        bt.bwta_kv_reserve(table, ps, cu(slots), cu(news), status=status)
        bt.bwta_kv_append(cache, table, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), slots=cu(slots),
                          cu_q=off, status=status)
        qt = torch.from_numpy(q).cuda()
        out = (bt.bwta_attn_decode_paged(qt, cache, table, 0.125, window, sinks, slots=cu(slots), status=status)
               if single else bt.bwta_attn_prompt_paged(qt, off, cache, table, 0.125, window, sinks,
                                                        slots=cu(slots), status=status))
        torch.cuda.synchronize()
        assert status.item() == 0
        at = 0
        sub = Batch.__new__(Batch)
        sub.H, sub.D, sub.lens, sub.k, sub.v = H, D, [], [], []
        for s, m in zip(slots, news):
            hk, hv = hist[s]
            hist[s] = (np.concatenate([hk, held(k[at:at + m]).transpose(1, 0, 2)], 1),
                       np.concatenate([hv, held(v[at:at + m]).transpose(1, 0, 2)], 1))
            at += m
            sub.lens.append(hist[s][0].shape[1])
            sub.k.append(hist[s][0])
            sub.v.append(hist[s][1])
        sub.check(q, out, news, 0.125, window, sinks)

    step([2, 0], [37, 64])
    step([0, 2], [1, 1])
    bt.bwta_kv_fork(layers, table, cu([2, 0, 2]), cu([1, 3, 4]), status=status)
    for a, d in ((2, 1), (0, 3), (2, 4)):
        hist[d] = hist[a]
    for _ in range(3):
        step([4, 1, 0, 2, 3], [1] * 5, window=20, sinks=3)
    bt.bwta_kv_free(table, ps, cu([2, 0]), status=status)
    hist[2] = hist[0] = (np.zeros((H, 0, D)), np.zeros((H, 0, D)))
    n = bt.bwta_kv_compact(layers, table, status=status)
    step([1, 4], [1, 1])
    step([0, 3, 1], [90, 5, 40], window=33, sinks=2)
    assert n.item() <= 60
    bt.bwta_kv_free(table, ps, cu(list(range(n_slots))), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert (table.refcount == 0).all() and (table.kv_len == 0).all() and (table.pages == -1).all()


def test_captured_step_replays():
    """reserve + append + attention in a graph: each replay is the next step."""
    H, G, D, ps = 2, 2, 64, 16
    cache = nan_cache(bt, 20, ps, H, D, False)
    table = bt.KvTable.empty(2, 6, 20)
    one = cu([1, 1])
    slots = cu([1, 0])
    r = np.random.default_rng(31)
    k = torch.zeros((2, H, D), device="cuda")
    v = torch.zeros((2, H, D), device="cuda")
    q = torch.from_numpy(r.standard_normal((2, H * G, D)).astype(np.float16)).cuda()
    status = bt.new_status()

    def step():
        bt.bwta_kv_reserve(table, ps, slots, one, status=status)
        bt.bwta_kv_append(cache, table, k, v, slots=slots, status=status)
        return bt.bwta_attn_decode_paged(q, cache, table, 0.125, slots=slots, status=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                # a first call outside of the capture
    torch.cuda.current_stream().wait_stream(side)
    bt.bwta_kv_free(table, ps, slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    ks, vs = [], []
    for _ in range(20):
        k.copy_(torch.from_numpy(r.standard_normal((2, H, D)).astype(np.float32)))
        v.copy_(torch.from_numpy(r.standard_normal((2, H, D)).astype(np.float32)))
        ks.append(k.half().cpu().double().numpy())
        vs.append(v.half().cpu().double().numpy())
        graph.replay()
    torch.cuda.synchronize()
    assert status.item() == 0 and table.kv_len.tolist() == [20, 20]
    sub = Batch.__new__(Batch)
    sub.H, sub.D, sub.lens = H, D, [20, 20]
    sub.k = [np.stack([x[s] for x in ks], 1) for s in range(2)]
    sub.v = [np.stack([x[s] for x in vs], 1) for s in range(2)]
    sub.check(q.cpu().numpy(), out, [1, 1], 0.125)
    graph.reset()
