"""okv_decode_step equals the append followed by the decode also where a token of
the step is written far behind the sequence's end, among the blocks that the
attention kernel starts to copy while the append still runs.  The rewritten key
holds nearly all of the row's weight, so that an old copy of it shows."""
import numpy as np
import pytest

from tests import gpu_helpers as H
from tests.test_gpu_int4 import _okv, _t

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 2])
@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (4, 1), (64, 8)])
@pytest.mark.parametrize("tokens", [1, 40, 127])
def test_a_token_rewritten_among_the_blocks(bits, group, hq, hkv, tokens):
    okv = _okv()
    lens, sinks = [3000, 700, 129], 16
    lay = H.Layout(58, lens)
    uk, uv = H.rotations(58, hkv)
    r = np.random.default_rng(58)
    bf = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    c = okv.Cache(hq, hkv, lay.num_blocks, 3, lay.mbps, uk, uv, bits=bits, group=group, num_sink=sinks)
    slots, pos = lay.flat()
    table, n = _t(lay.table), _t(np.array(lens, np.int32))
    okv.append_quantize(c, bf(len(slots), hkv, 128), bf(len(slots), hkv, 128), _t(slots), _t(pos), table, n)
    first = [x.clone() for x in (c.pages, c.ring, c.sink)]
    seq = torch.arange(3, dtype=torch.int32, device="cuda")
    # one token far back in each of the first two sequences, the rest at the first one's end
    new_slot = np.zeros(tokens, np.int32)
    new_pos = lens[0] - tokens + np.arange(tokens, dtype=np.int32)
    new_pos[0] = 16
    if tokens > 1:
        new_slot[tokens - 1], new_pos[tokens - 1] = 1, 300
    k, v, q = bf(tokens, hkv, 128), bf(tokens, hkv, 128), bf(3, hq, 128)
    for b, t in ((0, 0), (1, tokens - 1)):
        k[t] = 4 * q[b].view(hkv, hq // hkv, 128)[:, 0]
    args = (_t(new_slot), _t(new_pos))
    okv.append_quantize(c, k, v, *args, table, n)
    want = okv.decode_attention(c, q, seq, table, n)
    after = [x.clone() for x in (c.pages, c.ring, c.sink)]
    for _ in range(5):
        for x, y in zip((c.pages, c.ring, c.sink), first):
            x.copy_(y)
        got = okv.decode_step(c, k, v, *args, n, q, seq, table, n)
        assert torch.equal(got, want)
        assert all(torch.equal(x, y) for x, y in zip((c.pages, c.ring, c.sink), after))
    assert c.device_status() == 0
