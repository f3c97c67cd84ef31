"""okv_qk_norm_rope against the formula in 64 bits.  The outputs are bf16:
half a step is 2^-8 of the value.  What the kernel computes before that in fp32
(sum of 128 squares, square root, division, the product with the weight, the
sine and cosine of an fp32 angle within half a turn, two products and a sum) is
off by less than 32 steps of 2^-24 of sqrt(a^2 + b^2) of the rotated pair, so
|got - want| <= 2^-8 |want| + 2^-18 |pair|, with the pair's norm as a bound on
the terms that cancel."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D = 128


def _okv():
    from int2_kv_cache_rotate_b200 import okv
    return okv


def formula(x, w, pos, freq, eps, interleaved, norm, scale):
    """fp64 [T][H][128] and, per channel, the norm of its rotated pair."""
    x = x.double()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
    half = freq.numel()
    i = torch.arange(half, device=x.device)
    a_, b_ = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    ang = pos.double()[:, None, None] * freq.double()
    a, b = x[..., a_], x[..., b_]
    y = x.clone()
    y[..., a_] = (a * ang.cos() - b * ang.sin()) * scale
    y[..., b_] = (b * ang.cos() + a * ang.sin()) * scale
    size = x.abs().clone()
    size[..., a_] = size[..., b_] = torch.sqrt(a * a + b * b) * scale
    return y, size


def close(got, want, size):
    off = (got.double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -18 * size)
    assert off.max().item() <= 0, off.max().item()


def freqs(rot):
    return (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()


def inputs(seed, t, hq, hkv, dtype, far=100000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (torch.randn(t, (hq + 2 * hkv) * D, generator=g, device="cuda") * 2).to(dtype)
    pos = torch.randint(0, far, (t,), generator=g, device="cuda", dtype=torch.int32)
    w = [1 + 0.3 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    return qkv, pos, w


def views(qkv, hq, hkv):
    t = qkv.shape[0]
    return (qkv[:, :hq * D].view(t, hq, D), qkv[:, hq * D:(hq + hkv) * D].view(t, hkv, D),
            qkv[:, (hq + hkv) * D:].view(t, hkv, D))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("t,hq,hkv", [(1, 4, 1), (3, 32, 8), (64, 8, 8), (17, 5, 5), (2501, 24, 3)])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (96, False), (96, True), (16, False),
                                             (0, False)])
def test_norm_rope_matches_the_formula(dtype, t, hq, hkv, rot, interleaved):
    okv = _okv()
    qkv, pos, (wq, wk) = inputs(7, t, hq, hkv, dtype)
    q, k, v = views(qkv, hq, hkv)
    f = freqs(rot)
    got = okv.qk_norm_rope(q, k, pos, f, wq, wk, eps=1e-6, v=v, interleaved=interleaved)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        close(y, *formula(x, w, pos, f, 1e-6, interleaved, True, 1.0))
    assert torch.equal(got[2], v.to(torch.bfloat16))


def test_without_values_weights_or_norm_and_with_a_scale():
    okv = _okv()
    qkv, pos, (wq, _) = inputs(8, 33, 8, 2, torch.bfloat16)
    q, k, _ = views(qkv, 8, 2)
    f = freqs(128)
    for wq_, norm, scale in ((None, True, 1.0), (wq, True, 1.25), (None, False, 0.5)):
        got = okv.qk_norm_rope(q, k, pos, f, wq_, None, norm=norm, rope_scale=scale)
        assert len(got) == 2
        close(got[0], *formula(q, wq_, pos, f, 1e-6, False, norm, scale))
        close(got[1], *formula(k, None, pos, f, 1e-6, False, norm, scale))


@pytest.mark.parametrize("far", [1, 131072, 2 ** 24 + 1, 2 ** 31 - 1])
def test_far_positions_keep_their_angle(far):
    okv = _okv()
    qkv, _, _ = inputs(9, 8, 4, 1, torch.float32)
    q, k, _ = views(qkv, 4, 1)
    pos = torch.arange(far - 1, far - 9, -1, dtype=torch.int64, device="cuda").clamp(min=0).to(torch.int32)
    f = freqs(128)
    got = okv.qk_norm_rope(q, k, pos, f, norm=False)
    close(got[0], *formula(q, None, pos, f, 0, False, False, 1.0))


def test_padding_rows_stay_as_they_were_and_in_place():
    okv = _okv()
    qkv, pos, (wq, wk) = inputs(10, 70, 8, 2, torch.bfloat16)
    q, k, v = (x.contiguous() for x in views(qkv, 8, 2))
    pos[[0, 13, 14, 69]] = -1
    f = freqs(64)
    outs = [torch.full_like(x, 7.0) for x in (q, k, v)]
    okv.qk_norm_rope(q, k, pos, f, wq, wk, v=v, q_out=outs[0], k_out=outs[1], v_out=outs[2])
    dead = pos < 0
    for o in outs:
        assert torch.equal(o[dead], torch.full_like(o[dead], 7.0))
    want, size = formula(q, wq, pos, f, 1e-6, False, True, 1.0)
    close(outs[0][~dead], want[~dead], size[~dead])
    a, b = q.clone(), k.clone()
    okv.qk_norm_rope(a, b, pos, f, wq, wk, q_out=a, k_out=b)   # in place
    assert torch.equal(a[~dead], outs[0][~dead]) and torch.equal(a[dead], q[dead])
    assert torch.equal(b[~dead], outs[1][~dead]) and torch.equal(b[dead], k[dead])


def test_head_major_views_and_extreme_rows():
    okv = _okv()
    g = torch.Generator(device="cuda").manual_seed(3)
    qt = torch.randn(8, 40, D, generator=g, device="cuda")          # [heads][tokens][128]
    kt = torch.randn(2, 40, D, generator=g, device="cuda")
    qt[0, 0] = 0                                                    # a zero row: eps alone
    qt[1, 1] = 1e-20
    qt[2, 2] *= 1e15
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    f = freqs(128)
    q, k = qt.transpose(0, 1), kt.transpose(0, 1)
    got = okv.qk_norm_rope(q, k, pos, f)
    close(got[0], *formula(q, None, pos, f, 1e-6, False, True, 1.0))
    close(got[1], *formula(k, None, pos, f, 1e-6, False, True, 1.0))
    # an infinity or NaN stays in its own row (and, without a norm, in its own pair)
    bad = q.contiguous().clone()
    bad[5, 3, 9], bad[6, 1, 2] = math.inf, math.nan
    out = okv.qk_norm_rope(bad, k, pos, f[:16], norm=False)[0]
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[5, 3, [9, 25]] = False
    keep[6, 1, [2, 18]] = False
    assert torch.isfinite(out[keep]).all() and not torch.isfinite(out[~keep]).any()


def test_one_token_and_one_head_at_any_stride():
    okv = _okv()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(2000, generator=g, device="cuda")
    q = x.as_strided((1, 4, D), (3, 136, 1), 0)           # one token: its stride is never used
    k = x.as_strided((1, 1, D), (5, 7, 1), 1000)
    pos, f = torch.tensor([77], dtype=torch.int32, device="cuda"), freqs(64)
    got = okv.qk_norm_rope(q, k, pos, f)
    for y, t in zip(got, (q, k)):
        close(y, *formula(t, None, pos, f, 1e-6, False, True, 1.0))
    q = torch.randn(D, generator=g, device="cuda").expand(6, 3, D)  # one row broadcast over tokens and heads
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    y, _ = okv.qk_norm_rope(q, q, pos, f)
    close(y, *formula(q, None, pos, f, 1e-6, False, True, 1.0))
    with pytest.raises(ValueError, match="inv_freq"):
        okv.qk_norm_rope(q, q, pos, None)


def test_streams_and_graph():
    okv = _okv()
    qkv, pos, (wq, wk) = inputs(11, 200, 32, 8, torch.bfloat16)
    q, k, v = views(qkv, 32, 8)
    f = freqs(128)
    want = okv.qk_norm_rope(q, k, pos, f, wq, wk, v=v)
    outs = [torch.empty_like(x) for x in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        okv.qk_norm_rope(q, k, pos, f, wq, wk, v=v, q_out=outs[0], k_out=outs[1], v_out=outs[2])
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_refusals_on_the_device():
    okv = _okv()
    qkv, pos, _ = inputs(12, 4, 4, 1, torch.bfloat16)
    q, k, v = views(qkv, 4, 1)
    f = freqs(128)
    wide = torch.zeros(4, 4, 2 * D, dtype=torch.bfloat16, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        okv.qk_norm_rope(wide, k, pos, f)
    odd = torch.zeros(4 * 4 * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 4, D)
    with pytest.raises(okv.OkvError, match="16-byte"):
        okv.qk_norm_rope(odd, k, pos, f)
    with pytest.raises(ValueError, match="positions"):
        okv.qk_norm_rope(q, k, pos[:3], f)
    with pytest.raises(ValueError, match="heads"):
        okv.qk_norm_rope(q, k, pos, f, v=q)
    with pytest.raises(okv.OkvError, match="rot_dim"):
        okv.qk_norm_rope(q, k, pos, f[:5])
