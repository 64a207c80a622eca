"""The models that the cache's edge tests use, against those of kv_common, on the CPU."""
import numpy as np

from kv_common import quantize_rows
from kv_edges import quantize_many


def test_many_rows_quantize_as_one_by_one():
    r = np.random.default_rng(5)
    x = r.standard_normal((3, 200, 40)) * np.exp(4 * r.standard_normal((3, 200, 1)))
    x[r.random((3, 200)) < 0.05] = 0.0
    hit = r.random((3, 200)) < 0.2                            # a largest value on the border 448 * 2^e
    x[hit, 0] = 448.0 * 2.0 ** r.integers(-16, 8, hit.sum())
    x[r.random(x.shape) < 0.05] = -0.0
    x = np.clip(x, -65504, 65504)
    for y in (x, x.astype(np.float16).astype(np.float64)):
        for a, b in zip(quantize_rows(y), quantize_many(y)):
            np.testing.assert_array_equal(a, b)
