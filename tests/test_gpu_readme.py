"""The serving step of the README, as it stands there, on the outputs of real projections."""
import os

import numpy as np
import pytest
import torch

from kv_common import E4M3, quantize_rows

pytestmark = pytest.mark.gpu

bt = pytest.importorskip("binarized_transformer_b200")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def serving_step():
    text = open(os.path.join(ROOT, "README.md")).read().split("## A serving step")[1].split("\n## ")[0]
    return "\n".join(line[4:] for line in text.splitlines() if line.startswith("    "))


def test_the_serving_step_runs_as_written():
    n_heads, n_kv_heads, head_dim, K, rows = 8, 2, 64, 512, 3
    r = np.random.default_rng(3)
    X = torch.from_numpy(r.standard_normal((rows, K)).astype(np.float16)).cuda()
    jobs = []
    for n in (n_heads, n_kv_heads, n_kv_heads):
        W = torch.from_numpy(r.standard_normal((n * head_dim, K)).astype(np.float32)).cuda()
        jobs.append((X, *bt.bwta_pack_weights(W, 128), 128))
    q, k, v = (y[0] if isinstance(y, tuple) else y for y in bt.bwta_linear_decode_batched(jobs))
    assert q.dtype == torch.float32 and q.shape == (rows, n_heads * head_dim)
    names = dict(num_pages=10, n_kv_heads=n_kv_heads, n_heads=n_heads, head_dim=head_dim, n_layers=2, n_slots=5,
                 max_pages=4, q=q, k=k, v=v, slots=torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda"),
                 new_tokens=torch.ones(rows, dtype=torch.int32, device="cuda"))
    exec(serving_step(), names)
    torch.cuda.synchronize()
    # one token each: its value, as the cache holds it; the one weight is rounded to fp16 and so is the result
    codes, scale = quantize_rows(v.cpu().double().numpy().reshape(rows, n_kv_heads, head_dim))
    want = np.repeat(E4M3[codes] * scale[..., None], n_heads // n_kv_heads, axis=1)
    err = np.abs(names["o"].cpu().double().numpy() - want)
    assert (err <= (2.0 ** -10 + 2.0 ** -20) * np.abs(want) + 2.0 ** -25).all()
    assert names["table"].kv_len.tolist() == [1, 0, 1, 0, 1]
