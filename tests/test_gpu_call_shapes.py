"""Shapes of the binding's tensors beside the usual ones: rows with the heads and
channels in one dimension or in more than two, and block tables and slot lengths
with fewer rows than the cache has sequence slots, as a caller has them who uses
the first slots only.  Results have the bits of the usual call; a slot beyond the
rows given is skipped and flagged."""
import pytest

from tests.test_gpu_int4 import _okv, _t, queries

import numpy as np

from tests import gpu_helpers as H

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
HQ, HKV, LENS = 8, 2, [300, 40, 500, 17]


def filled(bits=4):
    okv = _okv()
    lay = H.Layout(56, [n + 1 for n in LENS])
    uk, uv = H.rotations(56, HKV)
    c = okv.Cache(HQ, HKV, lay.num_blocks, 4, lay.mbps, uk, uv, bits=bits, num_sink=16)
    r = np.random.default_rng(56)
    slots = np.concatenate([np.full(n, b, np.int32) for b, n in enumerate(LENS)])
    pos = np.concatenate([np.arange(n, dtype=np.int32) for n in LENS])
    k, v = (torch.from_numpy(r.standard_normal((len(slots), HKV, 128)).astype(np.float32)).bfloat16().cuda()
            for _ in range(2))
    return okv, c, lay, k, v, _t(slots), _t(pos), _t(lay.table), _t(np.array(LENS, np.int32))


@pytest.mark.parametrize("shape", [lambda x: x.flatten(1), lambda x: x.unsqueeze(1), lambda x: x.view(len(x), -1, 2, 64)])
def test_heads_and_channels_in_other_dimensions(shape):
    okv, c, lay, k, v, slots, pos, table, lens = filled()
    okv.append_quantize(c, k, v, slots, pos, table, lens)
    pages = c.pages.clone()
    c.pages.zero_()
    okv.append_quantize(c, shape(k), shape(v), slots, pos, table, lens)
    assert torch.equal(c.pages, pages)
    q, _ = queries(56, 4, HQ, HKV)
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    want = okv.decode_attention(c, q, seq, table, lens)
    assert torch.equal(okv.decode_attention(c, shape(q), seq, table, lens), want)
    assert torch.equal(okv.decode_attention_noalloc(c, shape(q), seq, table, lens), want)
    assert torch.equal(okv.prefill_attention(c, shape(q), 2, 500, table), okv.prefill_attention(c, q, 2, 500, table))
    more = lens + 1
    want = okv.decode_step(c, k[:4], v[:4], seq, lens, more, q, seq, table, more)
    assert torch.equal(okv.decode_step(c, shape(k[:4]), shape(v[:4]), seq, lens, more, shape(q), seq, table, more), want)
    assert c.device_status() == 0
    for bad in (q.flatten(), q.flatten(0, 1), q[:, :4], q.flatten(1)[:, :-128].contiguous()):
        with pytest.raises(ValueError, match="q must"):
            okv.decode_attention(c, bad.contiguous(), seq, table, lens)


@pytest.mark.parametrize("rows", [1, 3])
def test_fewer_rows_than_the_cache_has_slots(rows):
    okv, c, lay, k, v, slots, pos, table, lens = filled()
    okv.append_quantize(c, k, v, slots, pos, table, lens)
    pages, ring, sink = c.pages.clone(), c.ring.clone(), c.sink.clone()
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    q, _ = queries(56, 4, HQ, HKV)
    dense = okv.dequantize(c, seq, table, lens, 500, 1)
    want = okv.decode_attention(c, q, seq, table, lens)
    chunk = okv.prefill_attention(c, q, rows - 1, LENS[rows - 1], table)
    # the rows behind them belong to somebody else, and would send a reader out of the cache
    few = torch.full((4, lay.mbps), 1 << 30, dtype=torch.int32, device="cuda")
    few[:rows] = table[:rows]
    few, few_lens = few[:rows], lens[:rows]
    n = sum(LENS[:rows])
    c.pages.zero_(), c.ring.zero_(), c.sink.zero_()
    okv.append_quantize(c, k[:n], v[:n], slots[:n], pos[:n], few, few_lens)
    assert c.device_status() == 0
    okv.append_quantize(c, k[n:], v[n:], slots[n:], pos[n:], few, few_lens)   # slots that have no row
    assert c.device_status() == okv.DEV_BAD_SLOT
    c.clear_status()
    assert torch.equal(c.ring[:rows], ring[:rows]) and (c.ring[rows:] == 0).all() and (c.sink[rows:] == 0).all()
    assert torch.equal(okv.decode_attention(c, q[:rows], seq[:rows], few, lens[:rows]), want[:rows])
    assert torch.equal(okv.prefill_attention(c, q, rows - 1, LENS[rows - 1], few), chunk)
    assert torch.equal(okv.dequantize(c, seq[:rows], few, lens[:rows], 500, 1), dense[:rows])
    assert c.device_status() == 0
    got = okv.decode_attention(c, q, seq, few, lens)
    assert torch.equal(got[:rows], want[:rows]) and (got[rows:] == 0).all()
    assert c.device_status() == okv.DEV_BAD_SLOT
    with pytest.raises(okv.OkvError, match="slot"):
        okv.prefill_attention(c, q, rows, LENS[rows], few)
    # the step: append and decode, with one row more than the lengths have
    c.clear_status()
    c.pages.copy_(pages), c.ring.copy_(ring), c.sink.copy_(sink)
    more = lens + 1
    want = okv.decode_step(c, k[:4], v[:4], seq, lens, more, q, seq, table, more)
    c.pages.copy_(pages), c.ring.copy_(ring), c.sink.copy_(sink)
    got = okv.decode_step(c, k[:4], v[:4], seq, lens, more[:rows], q, seq, table, more)
    assert torch.equal(got[:rows], want[:rows]) and c.device_status() == okv.DEV_BAD_SLOT
    with pytest.raises(ValueError, match="block_table"):
        okv.decode_attention(c, q, seq, table.flatten()[:lay.mbps - 1], lens)
