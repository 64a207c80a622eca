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
