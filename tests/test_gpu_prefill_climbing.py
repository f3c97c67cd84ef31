"""The 4-bit prefill with bf16 output where the running maximum moves in every
batch of 32 keys, so that the weights a thread has stored in TMEM are read back
and scaled again and again, in the first chunk of keys and in later ones.

Bar: that of the other 4-bit prefill tests, 2e-3 and half a bf16 step.  Scores
reach 66 log2 units here; a key's own fp16 rounding (2^-11 of each of 128
products of either sign, so about 2^-11 sqrt(2/3) / sqrt(40) of the score) moves
its weight by 0.3 %, which the 32 keys that share a row's weight average to
0.05 %: a quarter of the 2e-3."""
import math

import numpy as np
import pytest

from oracle import okv_oracle as O
from tests import gpu_helpers as H
from tests.test_gpu_int4 import TOL, _okv, _t, check_rows, fill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

STEP, SLACK = 5.5, 4.0  # climb of a batch, and what the running maximum lets pass (log2 units)


def moves(score, pos):
    """How often, by batch of the chunk, the lazy maximum of a row at `pos` moves after the row's first batch."""
    seen = np.zeros(4, int)
    m = -math.inf
    for b in range(pos // 32 + 1):
        top = score[32 * b:min(32 * b + 32, pos + 1)].max()
        if top > m + SLACK:
            seen[b % 4] += m > -math.inf
            m = top
    return seen


@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2)])
@pytest.mark.parametrize("length,tokens", [(128, 90), (384, 40), (384, 384), (383, 1)])
def test_maximum_moves_in_every_batch(group, hq, hkv, length, tokens):
    okv = _okv()
    seed, g = 71, hq // hkv
    r = np.random.default_rng(seed)
    u = r.standard_normal((hkv, 128))
    u /= np.linalg.norm(u, axis=-1, keepdims=True)
    amp = 8.0
    uk, _ = H.rotations(seed, hkv)
    rot = [O.rotation(uk[h].astype(np.float64)) for h in range(hkv)]
    climb = STEP * (np.arange(length) // 32) / (amp * math.log2(math.e) / math.sqrt(128))

    def put(kind, b, z):
        if kind == 0:
            for h in range(hkv):
                z[:, h] = climb[:, None] * (u[h] @ rot[h]) + 0.05 * r.standard_normal((length, 128))
    gc, oc, lay, _ = fill(seed, hq, hkv, [length], group, extra=put)
    q = amp * np.repeat(u, g, 0)[None] + 0.01 * r.standard_normal((tokens, hq, 128))
    q = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    qn = q.float().numpy()
    keys = oc.values(0, 0, 0, length)
    score = keys @ (qn[-1, 0].astype(np.float64) @ oc.r[0][0]) * (math.log2(math.e) / math.sqrt(128))
    seen = moves(score, length - 1)
    assert (seen[1:] >= max(1, length // 128)).all() and (length <= 128 or seen[0] >= length // 128 - 1), seen
    out = torch.full((tokens, hq, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    okv.prefill_attention(gc, q.cuda(), 0, length, _t(lay.table), out=out)
    assert gc.device_status() == 0
    check_rows(out.float().cpu().numpy(), O.prefill(oc, qn, 0, length, hq), TOL + 2.0 ** -8)
