"""The paged key-value cache where its arithmetic can go wrong: values that are not finite, weights of very
unlike sizes, scores past what fp32 resolves, lengths that grow from launch to launch, each against 64 bits."""
import math

import numpy as np
import pytest
import torch

import kv_common
from kv_common import E4M3, Batch
from kv_edges import quantize_many

pytestmark = pytest.mark.gpu

bt = pytest.importorskip("binarized_transformer_b200")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    bt.load_library()


@pytest.fixture(autouse=True)
def _quick(monkeypatch):
    """Long sequences: the model quantizes all rows at once."""
    monkeypatch.setattr(kv_common, "quantize_rows", quantize_many)


def cu(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def put(b, s, k=None, v=None):
    """Replace all keys or values of sequence s ([heads, tokens, dim], 64 bits) in the cache and the model."""
    e4m3 = b.cache.k_scale is not None
    for x, pool, sc, keep in ((k, b.cache.k, b.cache.k_scale, b.k), (v, b.cache.v, b.cache.v_scale, b.v)):
        if x is None:
            continue
        t = x.shape[1]
        if e4m3:
            codes, scale = quantize_many(x)
            keep[s] = E4M3[codes] * scale[..., None]
        else:
            codes = x.astype(np.float16)
            keep[s] = codes.astype(np.float64)
        rows = b.table.pages[b.slot_of[s], :-(-t // b.ps)].long()
        whole = torch.zeros((b.H, len(rows) * b.ps, b.D), dtype=pool.dtype, device="cuda")
        whole[:, :t] = torch.from_numpy(codes).cuda()
        pool[rows] = whole.unflatten(1, (len(rows), b.ps)).transpose(0, 1)
        if e4m3:
            ws = torch.ones((b.H, len(rows) * b.ps), device="cuda")
            ws[:, :t] = torch.from_numpy(scale.astype(np.float32)).cuda()
            sc[rows] = ws.unflatten(1, (len(rows), b.ps)).transpose(0, 1)


def long_rows(b, tokens=1 << 20):
    """The batch's table with room for `tokens` tokens in a row: no bound on the lengths is known to the host."""
    rows = torch.full((b.table.pages.shape[0], tokens // b.ps), -1, dtype=torch.int32, device="cuda")
    rows[:, :b.max_pages] = b.table.pages
    return bt.KvTable(rows, b.table.kv_len, b.table.refcount)


def place(b, s, j):
    return b.table.pages[b.slots[s].item(), j // b.ps].item(), j % b.ps


# ------------------------------------------------------------------ keys that are not finite
@pytest.mark.parametrize("length,window,sinks", [(65, 0, 0), (129, 0, 0), (257, 0, 0), (300, 1, 3), (385, 1, 200)])
@pytest.mark.parametrize("rows", ["short", "long"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_newest_key_alone_in_its_share_is_nan(length, window, sinks, rows, e4m3):
    """The newest token is alone in the last tile and its key is NaN: no finite score stands beside it there."""
    b = Batch(bt, [length], 16, 2, 64, e4m3)
    page, at = place(b, 0, length - 1)
    if e4m3:
        b.cache.k[page, 1, at] = 0x7f
    else:
        b.cache.k[page, 1, at] = math.nan
    table = b.table if rows == "short" else long_rows(b)
    q = b.queries(1, 6)
    status = bt.new_status()
    out = bt.bwta_attn_decode_paged(torch.from_numpy(q).cuda(), b.cache, table, 0.125, window, sinks, slots=b.slots,
                                    status=status)
    torch.cuda.synchronize()
    assert status.item() == bt.STATUS_NONFINITE
    assert torch.isnan(out[0, 3:]).all()
    one = Batch.__new__(Batch)                                # the other key head's queries are as ever
    one.H, one.D, one.lens, one.k, one.v = 1, 64, b.lens, [b.k[0][:1]], [b.v[0][:1]]
    one.check(q[:, :3], out[:, :3], [1], 0.125, window, sinks)


# ------------------------------------------------------------------ weights of unlike sizes
def attend_tight(q, k, v, p, scale, window=0, sinks=0):
    """One query row at position p against 64 bits: (o [D], bound [D]).

    With w the weights over their sum, A = sum w |v|, n keys, fp16's half step 2^-11 and fp32's 2^-24:
    * a weight is rounded to fp16. The largest one is held as at least 2^7 (the reference is 7 below the
      maximum), so a weight is normal down to 2^-21 of the largest and rounded by 2^-11 of itself; below,
      by half a subnormal step, 2^-25 / 2^7 of the largest, and by no more than itself
    * a score is an fp32 sum of D products and the exponent's multiplication and subtraction: an absolute
      error d, a relative one of each weight, met by the weights and by their sum; exp2 within 2^-22
    * the sums run in fp32: at most n / 16 steps of the products, whose additions may cut instead of
      round (2^-23 of the sum so far, at most A), and n / 32 + 64 additions of the weights (2^-24)
    * the result is rounded to fp16: 2^-11 of it, or half the smallest step, 2^-25"""
    j = np.arange(min(len(k), p + 1))
    if window:
        j = j[(j > p - window) | (j < sinks)]
    x = (k[j] @ q) * scale
    w = np.exp(x - x.max())
    w /= w.sum()
    o, a, n = w @ v[j], w @ np.abs(v[j]), len(j)
    d = (k.shape[1] + 2) * 2.0 ** -24 * scale * (np.abs(k[j]) @ np.abs(q)).max() + 2.0 ** -22 * np.abs(x).max()
    per_key = np.minimum(w, np.maximum(2.0 ** -11 * w, 2.0 ** -32 * w.max())) @ np.abs(v[j])
    sums = n / 16 * 2.0 ** -23 + (n / 32 + 64) * 2.0 ** -24
    return o, 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + per_key + (2 * d + 2.0 ** -21 + sums) * a


def check_tight(b, q, out, seqs, positions, scale, window=0, sinks=0, rows=None):
    """Rows of q, out [n, heads, D]: row i is sequence seqs[i]'s query at positions[i]."""
    got, g, worst = out.cpu().double().numpy(), q.shape[1] // b.H, 0.0
    pick = range(len(q)) if rows is None or len(q) <= rows else np.unique(np.linspace(0, len(q) - 1, rows).astype(int))
    for i in pick:
        for h in range(q.shape[1]):
            o, bound = attend_tight(q[i, h].astype(np.float64), b.k[seqs[i]][h // g], b.v[seqs[i]][h // g], positions[i],
                                    scale, window, sinks)
            err = np.abs(got[i, h] - o)
            assert (err <= bound).all(), (i, h, float(np.nanmax(err / bound)))
            worst = max(worst, float((err / bound).max()))
    return worst


@pytest.mark.parametrize("call", ["decode", "decode_cluster", "prompt", "prompt_cluster"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_dominant_first_token_and_a_long_tail(call, D, e4m3):
    """A sink takes 99.9% of the weight and its value is zero: the output is the tail's, weights of 2^-25 of
    the largest each. Many rows, so that one block walks a whole sequence, or few, which share one."""
    t = 3500 if call == "decode_cluster" else 32768
    b = Batch(bt, [t], 64, 1, D, e4m3, seed=D)
    k, v = b.k[0].copy(), b.v[0].copy()
    k[0, :, 0] = 0.0
    k[0, 0] = 0.0
    k[0, 0, 0] = 64.0
    v[0, 0] = 0.0
    put(b, 0, k, v)
    n = {"decode": 450, "decode_cluster": 1, "prompt": 150, "prompt_cluster": 3}[call]
    q = b.queries(n, 1, size=(64.0 / D) ** 0.5)
    scale = 0.125
    tail = math.log(t) + 0.5                                  # log of the sum of weights with scores of variance 1
    q[:, :, 0] = (tail + math.log(999.0)) / (64.0 * scale)
    slots = b.slots.repeat(n)
    status = bt.new_status()
    qt = torch.from_numpy(q).cuda()
    if call.startswith("decode"):
        table = b.table if call == "decode_cluster" else long_rows(b)
        out = bt.bwta_attn_decode_paged(qt, b.cache, table, scale, slots=slots, status=status)
    else:
        out = bt.bwta_attn_prompt_paged(qt, cu(list(range(n + 1))), b.cache, b.table, scale, slots=slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    check_tight(b, q, out, [0] * n, [t - 1] * n, scale, rows=8)


@pytest.mark.parametrize("rows", ["short", "long"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_every_unit_of_a_long_sequence_counts(rows, e4m3):
    """Scores next to equal, V marks the unit of 64 tokens (column c: units c, c + D, ...): a unit lost or
    counted twice at a cut changes a column by more than a twentieth."""
    lens = [70001, 0, 3, 20000] if rows == "long" else [4000, 0, 3, 2900]
    b = Batch(bt, lens, 64, 2, 64, e4m3, seed=6)
    for s, t in enumerate(lens):
        if t:
            mark = (np.arange(t)[:, None] // 64 % 64 == np.arange(64)).astype(np.float64)
            put(b, s, v=np.broadcast_to(mark, (2, t, 64)).copy())
    q = b.queries(4, 8, size=0.1)
    qt = torch.from_numpy(q).cuda()
    status = bt.new_status()
    table = b.table if rows == "short" else long_rows(b)
    picks = [0, 2, 3]
    for window, sinks in ((0, 0), (1700, 129)):
        out = bt.bwta_attn_decode_paged(qt, b.cache, table, 0.125, window, sinks, slots=b.slots, status=status)
        assert (out[1] == 0).all()
        check_tight(b, q[picks], out[picks], picks, [lens[s] - 1 for s in picks], 0.125, window, sinks)
        out = bt.bwta_attn_prompt_paged(qt, cu([0, 1, 2, 3, 4]), b.cache, table, 0.125, window, sinks, slots=b.slots,
                                        status=status)
        assert (out[1] == 0).all()
        check_tight(b, q[picks], out[picks], picks, [lens[s] - 1 for s in picks], 0.125, window, sinks)
    assert status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_every_unit_of_a_long_prompt_counts(e4m3):
    """The same for many rows of a prompt, each of which sees another number of keys."""
    t, n = 9000, 3000
    b = Batch(bt, [t], 64, 2, 64, e4m3, seed=7)
    mark = (np.arange(t)[:, None] // 64 % 64 == np.arange(64)).astype(np.float64)
    put(b, 0, v=np.broadcast_to(mark, (2, t, 64)).copy())
    q = b.queries(n, 4, size=0.1)
    qt = torch.from_numpy(q).cuda()
    for window, sinks in ((0, 0), (1700, 129)):
        status = bt.new_status()
        out = bt.bwta_attn_prompt_paged(qt, cu([0, n]), b.cache, b.table, 0.125, window, sinks, slots=b.slots, status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        check_tight(b, q, out, [0] * n, list(range(t - n, t)), 0.125, window, sinks, rows=60)


# ------------------------------------------------------------------ scores of minus infinity
@pytest.mark.parametrize("t,n", [(40, 40), (300, 7), (5000, 3)])
def test_rows_whose_every_score_is_minus_infinity(t, n):
    """0 / 0 is not the zero of a row that sees nothing: NaN, and flagged, by both calls."""
    b = Batch(bt, [t], 16, 2, 64)
    q = np.abs(b.queries(n + 2, 4)) + np.float16(0.5)
    b.cache.k[:, 1, :, 5] = -math.inf                         # key head 1
    b.table.kv_len[b.slots.long()] = t
    qt = torch.from_numpy(q).cuda()
    status = bt.new_status()
    # two rows more than the sequence has when n = t: these see nothing
    out = bt.bwta_attn_prompt_paged(qt, cu([0, n + 2]), b.cache, b.table, 0.125, slots=b.slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == bt.STATUS_NONFINITE
    blind = max(0, n + 2 - t)
    assert (out[:blind] == 0).all() and torch.isnan(out[blind:, 2:]).all()
    one = Batch.__new__(Batch)
    one.H, one.D, one.lens, one.k, one.v = 1, 64, b.lens, [b.k[0][:1]], [b.v[0][:1]]
    one.check(q[blind:, :2], out[blind:, :2], [n + 2 - blind], 0.125, rows=8)
    status.zero_()
    out = bt.bwta_attn_decode_paged(qt[:1], b.cache, b.table, 0.125, slots=b.slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == bt.STATUS_NONFINITE and torch.isnan(out[:, 2:]).all()
    one.check(q[:1, :2], out[:, :2], [1], 0.125)


# ------------------------------------------------------------------ scores past what fp32 resolves
LN2 = float(np.float32(math.log(2.0)))                        # softmax_scale * log2(e) is 1 in fp32


def one_hot_queries(n, heads, D, cols):
    q = np.zeros((n, heads, D), np.float16)
    for c, x in cols.items():
        q[:, :, c] = x
    return q


@pytest.mark.parametrize("call", ["decode", "decode_long", "prompt", "prompt_cluster"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_of_millions_and_billions(call, e4m3):
    """fp16's largest queries and keys: one key takes all, wherever it lies. One product a score, so the scores
    are exact in fp32, and the keys' differ by 10^5 at least. The prompt call takes scores up to 2^27; beyond, a
    row is NaN and flagged."""
    t = 700
    b = Batch(bt, [t], 16, 1, 64, e4m3)
    table = b.table if call in ("decode", "prompt_cluster") else long_rows(b)
    n = {"prompt": 200, "decode_long": 450}.get(call, 1)      # many rows: one block walks a whole sequence
    for scale in (0.0011, 0.035, 0.37, 1.0):
        for top in (0, 77, 128, 699):
            for sign in (1.0, -1.0):
                k = np.zeros((1, t, 64))
                k[0, :, 3] = np.where(np.arange(t) == top, 57344.0, 53248.0 - 4096.0 * (np.arange(t) % 5))
                if sign < 0:                                  # all scores far below zero
                    k[0, :, 3] = -np.where(np.arange(t) == top, 36864.0, 40960.0 + 4096.0 * (np.arange(t) % 5))
                put(b, 0, k)
                q = one_hot_queries(n, 2, 64, {3: 65504.0})
                qt = torch.from_numpy(q).cuda()
                status = bt.new_status()
                slots = b.slots.repeat(n)
                if call.startswith("decode"):
                    out = bt.bwta_attn_decode_paged(qt, b.cache, table, scale, slots=slots, status=status)
                else:
                    out = bt.bwta_attn_prompt_paged(qt, cu(list(range(n + 1))), b.cache, table, scale, slots=slots,
                                                    status=status)
                torch.cuda.synchronize()
                if call.startswith("prompt") and scale > 0.1:
                    assert status.item() == bt.STATUS_NONFINITE and torch.isnan(out).all(), (scale, top, sign)
                    continue
                want = b.v[0][0, top]
                # the largest weight is rounded to fp16 and the sum is not; the result is rounded to fp16
                bound = (2.0 ** -10 + 2.0 ** -20) * np.abs(want) + 2.0 ** -25
                err = np.abs(out.cpu().double().numpy() - want)
                assert status.item() == 0, (scale, top, sign)
                assert (err <= bound).all(), (scale, top, sign)


@pytest.mark.parametrize("call", ["decode", "prompt"])
def test_steps_of_the_score_around_the_slack(call):
    """Scores of 2^27 + 16 r (exact, fp32's own steps there are 16): the next tile's maximum passes the
    reference by 16 = 2^16 of a weight, more than fp16 holds."""
    t, n = 512, 450                                           # many rows: one block walks a whole sequence
    for r0 in (1, 2, 3, 4):
        b = Batch(bt, [t], 16, 1, 64)
        k = np.zeros((1, t, 64))
        k[0, :, 0] = 8192.0
        k[0, :, 1] = r0 + np.arange(t) // 64                  # one more in each 64 tokens
        k[0, :, 1] += np.arange(t) % 64 == 63
        k[0, 64:, 1] -= 1
        put(b, 0, k)
        q = one_hot_queries(n, 1, 64, {0: 16384.0, 1: 16.0})
        qt = torch.from_numpy(q).cuda()
        status = bt.new_status()
        slots = b.slots.repeat(n)
        if call == "decode":
            out = bt.bwta_attn_decode_paged(qt, b.cache, long_rows(b), LN2, slots=slots, status=status)
        else:
            out = bt.bwta_attn_prompt_paged(qt, cu(list(range(n + 1))), b.cache, b.table, LN2, slots=slots, status=status)
        torch.cuda.synchronize()
        x = 16.0 * k[0, :, 1]
        w = 2.0 ** (x - x.max())
        w /= w.sum()
        o, a = w @ b.v[0][0], w @ np.abs(b.v[0][0])
        # scores and their differences are exact; weights, exp2, sums and the result are rounded
        bound = 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + (2.0 ** -11 + 2.0 ** -20) * a + t * 2.0 ** -32 * 4
        assert status.item() == 0, r0
        assert (np.abs(out[:, 0].cpu().double().numpy() - o) <= bound).all(), r0


# ------------------------------------------------------------------ values at fp16's largest
@pytest.mark.parametrize("call", ["decode", "decode_long", "prompt", "prompt_cluster"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_means_of_the_largest_value_stay_finite(call, sign):
    """Every value is 65504, so every mean is. The weights of 15 keys of 16 are just past the middle of
    two fp16 numbers and are rounded up while their sum is not: half a step above 65504 without a limit."""
    t = 700
    b = Batch(bt, [t], 16, 1, 128)
    k = np.zeros((1, t, 128))
    k[0, np.arange(t) % 16 != 0, 0] = -1.0                    # one of 16 keys holds the maximum: every share sees it
    put(b, 0, k, np.full((1, t, 128), sign * 65504.0))
    scale = -math.log(0.5 + 1.1 * 2.0 ** -12)
    n = 150 if call == "prompt" else 1
    q = one_hot_queries(n, 2, 128, {0: 1.0})
    qt = torch.from_numpy(q).cuda()
    table = b.table if call in ("decode", "prompt_cluster") else long_rows(b)
    slots = b.slots.repeat(n)
    status = bt.new_status()
    if call.startswith("decode"):
        out = bt.bwta_attn_decode_paged(qt, b.cache, table, scale, slots=slots, status=status)
    else:
        out = bt.bwta_attn_prompt_paged(qt, cu(list(range(n + 1))), b.cache, table, scale, slots=slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and (out == sign * 65504.0).all()


@pytest.mark.parametrize("call", ["decode", "decode_long", "prompt", "prompt_cluster"])
def test_infinite_values_stay_infinite(call):
    """A value of Inf that every row sees: that column of the output is Inf, the others are what they were."""
    t, n = 700, 150 if call == "prompt" else 1
    b = Batch(bt, [t], 16, 1, 64)
    for j, d, x in ((3, 5, math.inf), (77, 8, -math.inf)):
        page, at = place(b, 0, j)
        b.cache.v[page, 0, at, d] = x
    q = b.queries(n, 2)
    qt = torch.from_numpy(q).cuda()
    table = b.table if call in ("decode", "prompt_cluster") else long_rows(b)
    slots = b.slots.repeat(n)
    status = bt.new_status()
    if call.startswith("decode"):
        out = bt.bwta_attn_decode_paged(qt, b.cache, table, 0.125, slots=slots, status=status)
    else:
        out = bt.bwta_attn_prompt_paged(qt, cu(list(range(n + 1))), b.cache, table, 0.125, slots=slots, status=status)
    torch.cuda.synchronize()
    assert status.item() == bt.STATUS_NONFINITE
    assert (out[:, :, 5] == math.inf).all() and (out[:, :, 8] == -math.inf).all()
    out[:, :, [5, 8]] = 0.0
    b.v[0][:, :, [5, 8]] = 0.0
    check_tight(b, q, out, [0] * n, [t - 1] * n, 0.125, rows=8)


# ------------------------------------------------------------------ lengths that grow from launch to launch
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_joined_pieces_follow_the_lengths(e4m3, captured):
    """reserve, append, decode over and over with nothing between them, in a table whose rows are too long for
    clusters: every step is cut by lengths that the step before it in the stream has just written."""
    H, G, D, ps, steps = 2, 4, 64, 16, 24
    lens, grow = [2990, 100, 63, 1], [1, 1, 1, 1]
    b = Batch(bt, lens, ps, H, D, e4m3, seed=8)
    pool = b.num_pages + 40
    kind = torch.uint8 if e4m3 else torch.float16
    cache = bt.KvCache.empty(pool, ps, H, D, e4m3=e4m3)
    for x, y in ((cache.k, b.cache.k), (cache.v, b.cache.v), (cache.k_scale, b.cache.k_scale), (cache.v_scale, b.cache.v_scale)):
        if x is not None:
            x[:b.num_pages] = y
    assert cache.k.dtype == kind
    ref = torch.zeros(pool, dtype=torch.int32, device="cuda")
    held = b.table.pages[b.table.pages >= 0].long()
    ref[held] = 1
    b.table.refcount = ref
    table = long_rows(b, 1 << 15)
    r = np.random.default_rng(41)
    ks, vs, qs = (r.standard_normal((steps, 4, heads, D)) for heads in (H, H, H * G))
    ks, vs = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (ks, vs))
    qs = torch.from_numpy(qs.astype(np.float16)).cuda()
    k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
    status, new, ws = bt.new_status(), cu(grow), bt.decode_workspace(H * G, cache)

    def step():
        bt.bwta_kv_reserve(table, ps, b.slots, new, status=status)
        bt.bwta_kv_append(cache, table, k, v, slots=b.slots, status=status)
        return bt.bwta_attn_decode_paged(q, cache, table, 0.125, slots=b.slots, workspace=ws, status=status)

    bt.bwta_attn_decode_paged(q, cache, table, 0.125, slots=b.slots, workspace=ws)  # once outside of the capture
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
    got = []
    for i in range(steps):
        k.copy_(ks[i])
        v.copy_(vs[i])
        q.copy_(qs[i])
        if captured:
            graph.replay()
        else:
            out = step()
        got.append(out.clone())
    torch.cuda.synchronize()
    assert status.item() == 0
    for i in range(steps):
        for s in range(4):
            for x, keep in ((ks, b.k), (vs, b.v)):
                row = x[i, s].cpu().double().numpy()[:, None]
                if e4m3:
                    codes, sc = quantize_many(row)
                    row = E4M3[codes] * sc[..., None]
                else:
                    row = row.astype(np.float16).astype(np.float64)
                keep[s] = np.concatenate([keep[s], row], 1)
        check_tight(b, qs[i].cpu().numpy(), got[i], [0, 1, 2, 3], [n + i for n in lens], 0.125)
    if captured:
        graph.reset()


# ------------------------------------------------------------------ pools without pages
@pytest.mark.parametrize("e4m3", [False, True])
def test_copies_where_a_pool_is_empty(e4m3):
    """No page can be named: each copy is refused on the device, the call is not (empty pools have no buffers,
    and that both sides' are NULL says nothing)."""
    void = [bt.KvCache.empty(0, 16, 2, 64, e4m3=e4m3) for _ in range(4)]
    some = [bt.KvCache.empty(3, 16, 2, 64, e4m3=e4m3) for _ in range(2)]
    for c in some:
        c.k.zero_()
    for a, b in ((void[:1], void[1:2]), (void[:2], void[2:]), (void[:2], some), (some, void[:2]), (void[:2], void[:2])):
        status = bt.new_status()
        bt.bwta_kv_copy_pages(a, b, cu([0, 1]), cu([1, 2]), status=status)
        torch.cuda.synchronize()
        assert status.item() == kv_common.BAD
    assert all((c.k == 0).all() for c in some)


# ------------------------------------------------------------------ a table of one page size
def test_a_table_refuses_another_page_size():
    """Pages handed out by one size and read by another would be the wrong ones, without a flag."""
    table = bt.KvTable.empty(2, 4, 8, page_size=32)
    small, right = (bt.KvCache.empty(8, ps, 1, 64) for ps in (16, 32))
    one, slots = cu([1, 1]), cu([0, 1])
    k = torch.zeros((2, 64), device="cuda")
    q = torch.zeros((2, 1, 64), dtype=torch.float16, device="cuda")

    def calls(c):
        ps = c.page_size
        return [lambda: bt.bwta_kv_reserve(table, ps, slots, one), lambda: bt.bwta_kv_append(c, table, k, k),
                lambda: bt.bwta_attn_decode_paged(q, c, table, 0.125),
                lambda: bt.bwta_attn_prompt_paged(q, cu([0, 1, 2]), c, table, 0.125),
                lambda: bt.bwta_kv_fork(c, table, slots[:1], slots[1:]), lambda: bt.bwta_kv_compact(c, table),
                lambda: bt.bwta_kv_free(table, ps, slots)]
    for call in calls(small):
        with pytest.raises(AssertionError):
            call()
    assert (table.kv_len == 0).all()
    for call in calls(right):
        call()
    torch.cuda.synchronize()
    assert (table.kv_len == 0).all() and (table.refcount == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_sequences_of_unlike_lengths(e4m3):
    """A thousand sequences, empty ones among them: a share of the cut's prefix sums is several of them, and
    pieces of a sequence lie in many blocks or one."""
    r = np.random.default_rng(17)
    lens = [0, 1, 63, 64, 65, 128, 129, 1000, 5000] + r.integers(0, 700, 15).tolist()
    b = Batch(bt, lens, 16, 2, 64, e4m3, seed=17)
    n = 1000
    who = r.integers(0, len(lens), n)
    q = b.queries(n, 4)
    status = bt.new_status()
    for window, sinks in ((0, 0), (100, 20)):
        out = bt.bwta_attn_decode_paged(torch.from_numpy(q).cuda(), b.cache, long_rows(b), 0.125, window, sinks,
                                        slots=b.slots[torch.from_numpy(who).cuda()], status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        empty = np.array([lens[s] == 0 for s in who])
        assert (out.cpu().numpy()[empty] == 0).all()
        rows = np.nonzero(~empty)[0]
        check_tight(b, q[rows], out[torch.from_numpy(rows).cuda()], who[rows], [lens[s] - 1 for s in who[rows]], 0.125,
                    window, sinks)
