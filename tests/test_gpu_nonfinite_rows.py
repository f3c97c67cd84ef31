"""A query row that holds an infinity or a NaN gives NaN in its own output row
and nothing but rounding in the others, in every decode and prefill kernel and
whether or not the work over its keys is cut into pieces.

Bar for the other rows: prefill rows keep their bits (a row shares nothing with
the next one).  A decode warp flushes all its heads' sums when one of them moves
its reference, so the others' fp32 sums are added up at other moments: a few
2^-24 per flush and 2^-16 of a weight, under 1e-3 of a row's largest value."""
import numpy as np
import pytest

from tests import gpu_helpers as H

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
L = 3000


def cache(bits, group, hq, hkv):
    from int2_kv_cache_rotate_b200 import okv
    lay = H.Layout(3, [L])
    uk, uv = H.rotations(3, hkv)
    c = okv.Cache(hq, hkv, lay.num_blocks, 1, lay.mbps, uk, uv, group=group, bits=bits)
    r = np.random.default_rng(0)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    k, v = (d(r.standard_normal((L, hkv, 128)).astype(np.float32)) for _ in range(2))
    slots, pos = lay.flat()
    okv.append_quantize(c, k, v, d(slots), d(pos), d(lay.table), d(np.array([L], np.int32)), pre_rotated=True)
    return okv, c, d(lay.table)


def query(n, hq, val):
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn(n, hq, 128, generator=g, device="cuda").bfloat16()
    bad = q.clone()
    bad[n - 1, 1, 5] = val
    keep = torch.ones(n, hq, dtype=torch.bool, device="cuda")
    keep[n - 1, 1] = False
    return q, bad, keep


@pytest.mark.parametrize("val", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (64, 8), (4, 1), (16, 1), (6, 3)])
def test_decode(val, bits, group, hq, hkv):
    okv, c, table = cache(bits, group, hq, hkv)
    q, bad, keep = query(3, hq, val)
    args = (torch.zeros(3, dtype=torch.int32, device="cuda"), table, torch.full((3,), L, dtype=torch.int32, device="cuda"))
    want, got = (okv.decode_attention(c, x, *args) for x in (q, bad))
    assert got[2, 1].isnan().all()
    assert H.rel_err_rows(got[keep].cpu().numpy(), want[keep].cpu().numpy()).max() <= 1e-3
    assert c.device_status() == 0


@pytest.mark.parametrize("val", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (4, 1), (6, 3)])
@pytest.mark.parametrize("tokens", [1, 40, 700, 2500])   # few rows: every tile is cut; many: most are whole
def test_prefill(val, bits, group, hq, hkv, tokens):
    okv, c, table = cache(bits, group, hq, hkv)
    q, bad, keep = query(tokens, hq, val)
    for dtype in (torch.float32, torch.bfloat16):
        outs = [torch.empty(tokens, hq, 128, dtype=dtype, device="cuda") for _ in range(2)]
        for x, o in zip((q, bad), outs):
            okv.prefill_attention(c, x, 0, L, table, out=o)
        assert outs[1][-1, 1].isnan().all(), dtype
        assert torch.equal(outs[0][keep], outs[1][keep]), dtype
    assert c.device_status() == 0
