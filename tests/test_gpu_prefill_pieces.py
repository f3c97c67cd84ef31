"""The 4-bit prefill where a tile's keys are cut into 30 and 31 pieces, the most
that a sweep of the cut finds on 148 SMs (the merge has room for 32), in all
three group sizes: every row against 64 bits, at the bar of the other prefills."""
import math

import numpy as np
import pytest

from tests.test_gpu_int4 import TOL, _okv, _t, check_rows, fill, queries
from tests.test_prefill_split_cpu import MANY

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("tokens,length,hq,hkv", [m[:4] for m in MANY])
def test_tiles_in_thirty_pieces(group, tokens, length, hq, hkv):
    okv = _okv()
    gc, oc, lay, _ = fill(63, hq, hkv, [length], group, sinks=16)
    q, qn = queries(63, tokens, hq, hkv)
    out = torch.full((tokens, hq, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    okv.prefill_attention(gc, q, 0, length, _t(lay.table), out=out)
    again = torch.empty_like(out)
    okv.prefill_attention(gc, q, 0, length, _t(lay.table), out=again)
    assert gc.device_status() == 0 and torch.equal(out, again)
    got = out.float().cpu().numpy()
    seen = np.arange(length)[None] <= np.arange(length - tokens, length)[:, None]
    for h in range(hkv):
        keys, vals = (oc.values(0, kind, h, length) for kind in (0, 1))
        for j in range(h * hq // hkv, (h + 1) * hq // hkv):
            x = np.where(seen, (qn[:, j].astype(np.float64) @ oc.r[0][h]) @ keys.T / math.sqrt(128), -np.inf)
            w = np.exp(x - x.max(1, keepdims=True))
            check_rows(got[:, j], (w / w.sum(1, keepdims=True)) @ vals @ oc.r[1][h].T, TOL + 2.0 ** -8)
