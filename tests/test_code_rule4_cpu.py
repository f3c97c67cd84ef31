"""The 4-bit code without a division per value: with r = fl(1 / s), the code of
x = fl(z - m) is k + [x > h s, or x = h s and k odd], h = k + 1/2, where k is
rint(x r - 1/2) clamped to [0, 14].  Checked in numpy fp32 against the oracle's
division, on groups built around every rounding midpoint and on workload data
(the kernels run the same groups in test_gpu_int4.py)."""
import numpy as np
import pytest

from int2_kv_cache_rotate_b200 import workloads as WL
from oracle import okv_oracle as O
from tests.test_gpu_int4 import boundary_vectors, special_rows

f = np.float32


def rule(z, s16, m16, group):
    x = (z.reshape(*s16.shape, group) - m16.astype(f)[..., None]).astype(f)
    s = s16.astype(f)[..., None]
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        r = (f(1) / s).astype(f)
        k = np.clip(np.rint((x.astype(np.float64) * r - 0.5).astype(f)), 0, 14).astype(f)
    thr = (k * s + f(0.5) * s).astype(f)      # exact: 5 + 11 bits
    c = k + ((x > thr) | ((x == thr) & (k % 2 == 1)))
    return np.where(s == 0, 0, c).astype(np.uint8).reshape(z.shape)


@pytest.mark.parametrize("group", [128, 64, 32])
def test_rule_equals_division(group):
    rows = np.concatenate([boundary_vectors(9, 700, group), special_rows()] +
                          [WL.sample_rotated(0, 0, 0, 0, 1000, 0, scale=sc) for sc in (1e-6, 1.0, 300.0)])
    c, s16, m16 = O.quantize(rows, group, 4)
    shape = (rows.shape[0], 128 // group)
    assert np.array_equal(rule(rows, s16.reshape(shape), m16.reshape(shape), group), c)
    assert set(np.unique(c)) == set(range(16))
