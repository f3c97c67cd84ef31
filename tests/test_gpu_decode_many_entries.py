"""More sequences than split-K CTAs: a CTA goes through several entries, whose
window scratch and merge buffers lie over the ring that the next entry's blocks
are copied into.  Against the oracle, at the bar of the other decode tests."""
import numpy as np
import pytest

from oracle import okv_oracle as O
from tests import gpu_helpers as H
from tests.test_gpu_int4 import TOL, _okv, _t

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("hq,hkv,group", [(8, 2, 128), (4, 1, 32), (8, 8, 64), (16, 2, 128)])
def test_several_entries_per_cta(bits, hq, hkv, group):
    okv = _okv()
    r = np.random.default_rng(59)
    lens = [int(x) for x in r.integers(1, 420, 900)]
    lay = H.Layout(59, lens)
    uk, uv = H.rotations(59, hkv)
    c = okv.Cache(hq, hkv, lay.num_blocks, len(lens), lay.mbps, uk, uv, bits=bits, group=group)
    oc = O.Cache(hkv, uk.astype(np.float64), uv.astype(np.float64), bits=bits, group=group)
    slots, pos = lay.flat()
    z = [r.standard_normal((len(slots), hkv, 128)).astype(np.float32) for _ in range(2)]
    n = np.array(lens, np.int32)
    okv.append_quantize(c, _t(z[0]), _t(z[1]), _t(slots), _t(pos), _t(lay.table), _t(n), pre_rotated=True)
    q = torch.from_numpy(r.standard_normal((len(lens), hq, 128)).astype(np.float32)).bfloat16()
    seq = np.arange(len(lens), dtype=np.int32)
    got = okv.decode_attention(c, q.cuda(), _t(seq), _t(lay.table), _t(n)).cpu().numpy()
    again = okv.decode_attention(c, q.cuda(), _t(seq), _t(lay.table), _t(n)).cpu().numpy()
    assert c.device_status() == 0 and np.array_equal(got, again)
    some = np.arange(0, len(lens), 7)
    ends = np.cumsum(lens)
    for b in some:
        a = ends[b] - lens[b]
        oc.append(int(b), 0, z[0][a:ends[b]], z[1][a:ends[b]], pre_rotated=True)
    want = O.decode(oc, q.float().numpy()[some], some, [lens[b] for b in some], hq)
    assert H.rel_err_rows(got[some], want).max() <= TOL
