"""The cache held in 4 bits: append, gather, decode, fused step and chunked
prefill through the C ABI, against the oracle with 16 levels per group.

Bars.  Codes, scales, minima and fp16 rows are whole bits and have to be equal
(to the oracle's quantiser on the kernel's own fp32 rotation where the kernel
rotates).  Attention with fp32 output keeps the bar of the 2-bit cache, 2e-3 of
a row's largest value: the formula is the same, the codes are exact operands in
both, and the roundings in between (16-bit query limbs, 16-bit weights, the
approximate exponent) do not depend on the code's width.  With bf16 output half
a step of the value, 2^-8, comes on top."""
import math

import numpy as np
import pytest

from int2_kv_cache_rotate_b200 import workloads as WL
from oracle import okv_oracle as O
from tests import gpu_helpers as H

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 2e-3
GROUPS = (128, 64, 32)


def _okv():
    from int2_kv_cache_rotate_b200 import okv
    return okv


def _t(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def read_codes(pages, table, slot, h, hkv, n, kind, group):
    """Codes [n][128] and fp16 scale and minimum [n][128 / group] by the layout that the header documents."""
    ng = 128 // group
    bhb = 2048 + 128 * ng
    pos = np.arange(n)
    base = ((table[slot, pos // 16].astype(np.int64) * hkv + h) * bhb)[:, None]
    t = (pos % 16)[:, None]
    b = np.arange(64)[None]
    w = b >> 2
    off = t * 64 + (4 * (w & 3) + (w >> 2)) * 4 + (b & 3) if kind == 0 else \
        1024 + (b >> 5) * 512 + ((b & 7) * 4 + (t >> 2)) * 16 + ((b >> 3) & 3) * 4 + (t & 3)
    byte = pages[base + off]
    codes = np.stack([byte & 15, byte >> 4], -1).reshape(n, 128)
    so = base + 2048 + 64 * ng * kind + 4 * (t * ng + np.arange(ng)[None])
    half = [(pages[so + 2 * i].astype(np.uint16) | (pages[so + 2 * i + 1].astype(np.uint16) << 8)).view(np.float16)
            for i in (0, 1)]
    return codes, half[0], half[1]


def oracle_codes(z, group):
    c, s, m = O.quantize(z, group, 4)
    shape = (z.shape[0], 128 // group)
    return c, s.reshape(shape), m.reshape(shape)


def boundary_vectors(seed, n, group):
    """Rows whose values sit within 8 fp32 steps of every rounding midpoint m + (k + 1/2) s, k = 0 .. 14, of their
    group's own quantiser, ties included; scales over fp16's normal and subnormal range, minima on both sides."""
    r = np.random.default_rng(np.random.SeedSequence([seed, 77]))
    rows = np.empty((n, 128 // group, group), np.float32)
    for i in range(n):
        for j in range(128 // group):
            s_t = max(np.float64(np.float16(r.uniform(1, 2) * 2.0 ** int(r.integers(-24, 9)))), 2.0 ** -24)
            m_t = np.float32(np.float16(np.clip(r.uniform(-1, 1) * s_t * 2.0 ** int(r.integers(0, 8)), -60000, 60000)))
            row = np.full(group, m_t, np.float32)
            row[1] = np.float32(np.float64(m_t) + 15 * s_t)
            _, s16, m16 = O.quantize_rows(row[None], 4)
            s, m = np.float64(s16[0]), np.float64(m16[0])
            vals = np.empty(group - 2, np.float32)
            for x in range(group - 2):
                c = np.float32(m + (int(r.integers(0, 15)) + 0.5) * s)
                for _ in range(int(r.integers(0, 9))):
                    c = np.nextafter(c, np.float32(np.inf if x & 1 else -np.inf))
                vals[x] = c
            row[2:] = np.clip(vals, row[0], row[1])
            rows[i, j] = row[r.permutation(group)]
    return rows.reshape(n, 128)


def special_rows():
    j = np.arange(128)
    return np.concatenate([H.special_vectors(), np.stack([
        (j % 16).astype(np.float32), np.float32(-7.5) + (j % 16), np.where(j == 5, 1e-6, 0).astype(np.float32),
        np.where(j == 3, 1e38, -1e38).astype(np.float32), np.where(j < 64, 4e-7, 0).astype(np.float32)
        ]).astype(np.float32)])


def fill(seed, hq, hkv, lens, group, sinks=0, special=False, extra=None, **kw):
    """A 4-bit cache and the oracle's, filled with the same rotated vectors."""
    okv = _okv()
    lay = H.Layout(seed, lens)
    uk, uv = H.rotations(seed, hkv)
    gc = okv.Cache(hq, hkv, lay.num_blocks, len(lens), lay.mbps, uk, uv, num_sink=sinks, group=group, bits=4, **kw)
    oc = O.Cache(hkv, uk.astype(np.float64), uv.astype(np.float64), sinks=sinks, group=group, bits=4)
    zs = {0: [], 1: []}
    for kind in (0, 1):
        for b, n in enumerate(lens):
            z = np.stack([WL.sample_rotated(seed, 0, 0, h, n, kind, extra=b) for h in range(hkv)], axis=1) \
                if n else np.zeros((0, hkv, 128), np.float32)
            if special and n:
                sp = special_rows()
                z[:min(n, len(sp)), 0] = sp[:n]
            if extra is not None:
                extra(kind, b, z)
            zs[kind].append(z)
    for b, n in enumerate(lens):
        if n:
            oc.append(b, 0, zs[0][b], zs[1][b], pre_rotated=True)
    slots, pos = lay.flat()
    if len(slots):
        okv.append_quantize(gc, _t(np.concatenate(zs[0])), _t(np.concatenate(zs[1])), _t(slots), _t(pos), _t(lay.table),
                            _t(np.array(lens, np.int32)), pre_rotated=True)
    return gc, oc, lay, zs


def queries(seed, n, hq, hkv, extra=0, scale=1.0):
    q = np.stack([WL.sample_queries(seed, 0, 0, h, n, hq // hkv, extra=extra) for h in range(hkv)], 1)
    q = torch.from_numpy(np.ascontiguousarray(q.reshape(n, hq, 128)) * scale).to(torch.bfloat16)
    return q.cuda(), q.float().numpy()


def check_rows(got, want, tol):
    err = H.rel_err_rows(got, want)
    assert np.isfinite(got).all() and err.max() <= tol, err.max()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("hkv", [1, 3])
def test_pre_rotated_append_is_bit_exact(group, hkv):
    gc, oc, lay, zs = fill(21, hkv, hkv, [1, 15, 16, 17, 300], group, sinks=16, special=True)
    torch.cuda.synchronize()
    assert gc.device_status() == 0
    pages, ring, sink = gc.pages.cpu().numpy(), gc.ring.cpu().numpy(), gc.sink.cpu().numpy()
    for b, n in enumerate(lay.lens):
        for h in range(hkv):
            for kind in (0, 1):
                got = read_codes(pages, lay.table, b, h, hkv, n, kind, group)
                z = zs[kind][b][:, h]
                for x, y in zip(got, oracle_codes(z, group)):
                    assert np.array_equal(x.view(np.uint8), y.view(np.uint8)), (b, h, kind)
                z16 = O.fp16_saturate(z)
                for p in range(max(0, n - 128), n):
                    assert np.array_equal(ring[b, h, kind, p % 128].view(np.uint16), z16[p].view(np.uint16))
                assert np.array_equal(sink[b, h, kind, :min(n, 16)].view(np.uint16), z16[:16].view(np.uint16))


@pytest.mark.parametrize("group", GROUPS)
def test_codes_at_every_rounding_midpoint(group):
    n = 1200
    z = boundary_vectors(5, n, group)

    def put(kind, b, x):
        x[:, 0] = z
    gc, _, lay, _ = fill(22, 1, 1, [n], group, extra=put)
    pages = gc.pages.cpu().numpy()
    want = oracle_codes(z, group)
    t = (z.reshape(n, -1, group) - want[2].astype(np.float32)[..., None]) / want[1].astype(np.float32)[..., None]
    assert ((t - np.floor(t)) == 0.5).sum() > 1000       # ties really occur
    for kind in (0, 1):
        for x, y in zip(read_codes(pages, lay.table, 0, 0, 1, n, kind, group), want):
            assert np.array_equal(x.view(np.uint8), y.view(np.uint8))


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("tokens,offset,stage", [(1, 0, True), (37, 0, True), (127, 0, True), (128, 0, True),
                                                 (745, 0, True), (745, 0, False), (745, 1, True)])
def test_rotating_append_quantises_its_own_rotation_exactly(group, tokens, offset, stage):
    okv = _okv()
    seed, hq, hkv = 23, 8, 2
    lay = H.Layout(seed, [tokens])
    uk, uv = H.rotations(seed, hkv)
    gc = okv.Cache(hq, hkv, lay.num_blocks, 1, lay.mbps, uk, uv, group=group, bits=4, stage_r=stage, num_sink=32)
    k, v = (np.stack([f(seed, 0, 0, h, tokens) for h in range(hkv)], 1) for f in (WL.sample_keys, WL.sample_values))
    dev = []
    for x in (k, v):  # offset 1: rows that TMA cannot take
        flat = torch.zeros(x.size + offset, dtype=torch.bfloat16, device="cuda")[offset:]
        dev.append(flat.view(tokens, hkv, 128).copy_(torch.from_numpy(x)))
    rot = torch.zeros(tokens, 2, hkv, 128, device="cuda")
    slots, pos = lay.flat()
    okv.append_quantize(gc, *dev, _t(slots), _t(pos), _t(lay.table), _t(np.array([tokens], np.int32)), rotated_out=rot)
    torch.cuda.synchronize()
    assert gc.device_status() == 0
    rot, pages, ring = rot.cpu().numpy(), gc.pages.cpu().numpy(), gc.ring.cpu().numpy()
    for kind, (x, u) in enumerate(((dev[0], uk), (dev[1], uv))):
        x = x.float().cpu().numpy().astype(np.float64)
        for h in range(hkv):
            z64 = x[:, h] @ O.rotation(u[h].astype(np.float64))
            assert (np.abs(rot[:, kind, h] - z64).max(1) <= 1e-5 * np.abs(z64).max(1)).all()
            for a, b in zip(read_codes(pages, lay.table, 0, h, hkv, tokens, kind, group),
                            oracle_codes(rot[:, kind, h], group)):
                assert np.array_equal(a.view(np.uint8), b.view(np.uint8)), (kind, h)
            z16 = O.fp16_saturate(rot[:, kind, h])
            for p in range(max(0, tokens - 128), tokens):
                assert np.array_equal(ring[0, h, kind, p % 128].view(np.uint16), z16[p].view(np.uint16))


@pytest.mark.parametrize("tokens", [5, 40, 300])
def test_padding_rows_are_skipped_and_flagged_only_without_the_format_bit(tokens):
    okv = _okv()
    seed, hkv = 24, 2
    lay = H.Layout(seed, [tokens])
    uk, uv = H.rotations(seed, hkv)
    k, v = (np.stack([f(seed, 0, 0, h, tokens) for h in range(hkv)], 1) for f in (WL.sample_keys, WL.sample_values))
    slots, pos = lay.flat()
    slots, pos = slots.copy(), pos.copy()
    slots[[1, tokens - 1]] = -1
    pos[[1, tokens - 1]] = -1
    for bits in (2, 4):
        got = []
        for pad in (True, False):
            c = okv.Cache(4, hkv, lay.num_blocks, 1, lay.mbps, uk, uv, bits=bits, pad_rows=pad)
            c.pages.fill_(0x5A)
            okv.append_quantize(c, _t(k, torch.bfloat16), _t(v, torch.bfloat16), _t(slots), _t(pos), _t(lay.table),
                                _t(np.array([tokens], np.int32)))
            torch.cuda.synchronize()
            assert c.device_status() == (0 if pad else okv.DEV_BAD_SLOT)
            got.append(c.pages.clone())
        assert torch.equal(*got)


# ------------------------------------------------------------------ gather

@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("source", [0, 1])
def test_dequantise(group, source):
    okv = _okv()
    lens, hkv = [0, 5, 130, 401], 2
    gc, oc, lay, zs = fill(25, hkv, hkv, lens, group, sinks=16)
    seq, ctx = _t(np.arange(4, dtype=np.int32)), _t(np.array(lens, np.int32))
    for which in (0, 1):
        got = okv.dequantize(gc, seq, _t(lay.table), ctx, 410, which, 0, source)
        half = torch.full(got.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        okv.dequantize(gc, seq, _t(lay.table), ctx, 410, which, 0, source, out=half)
        assert torch.equal(half, got.to(torch.bfloat16))
        orig = okv.dequantize(gc, seq, _t(lay.table), ctx, 410, which, 1, source).cpu().numpy()
        got = got.cpu().numpy()
        for b, n in enumerate(lens):
            assert (got[b, :, n:] == 0).all()
            for h in range(hkv):
                if not n:
                    continue
                c, s, m = oracle_codes(zs[which][b][:, h], group)
                want = O.dequantize(c, s if group < 128 else s[:, 0], m if group < 128 else m[:, 0], group)
                if source == 1:
                    want = oc.values(b, which, h, n).astype(np.float32)
                assert np.array_equal(got[b, h, :n], want)
                back = want.astype(np.float64) @ oc.r[which][h].T
                assert np.abs(orig[b, h, :n] - back).max() <= 1e-5 * np.abs(back).max()
    assert gc.device_status() == 0


# ------------------------------------------------------------------ decode

LENS = [0, 1, 15, 16, 17, 127, 128, 129, 143, 144, 145, 160, 161, 300, 577, 1024, 3001]


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("hq,hkv", [(8, 8), (16, 8), (32, 8), (64, 8), (128, 8), (4, 1), (8, 1), (1, 1), (16, 2), (16, 4),
                                    (24, 3), (5, 5)])
def test_decode_matches_the_oracle(group, hq, hkv):
    okv = _okv()
    lens = LENS if hkv <= 3 else [0, 1, 16, 129, 145, 300, 1500]
    gc, oc, lay, _ = fill(26, hq, hkv, lens, group)
    q, qn = queries(26, len(lens), hq, hkv)
    seq = np.arange(len(lens), dtype=np.int32)
    args = (_t(seq), _t(lay.table), _t(np.array(lens, np.int32)))
    got = okv.decode_attention(gc, q, *args)
    want = O.decode(oc, qn, seq, lens, hq)
    torch.cuda.synchronize()
    assert gc.device_status() == 0
    check_rows(got.cpu().numpy(), want, TOL)
    assert (got[0] == 0).all()
    out = torch.empty(len(lens), hq, 128, dtype=torch.bfloat16, device="cuda")
    okv.decode_attention(gc, q, *args, out=out)
    assert torch.equal(out, got.to(torch.bfloat16))
    if okv.decode_workspace_bytes(gc, len(lens)) <= 8 << 20:  # what the built-in scratch holds
        assert torch.equal(okv.decode_attention_noalloc(gc, q, *args), got)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("sinks", [16, 48, 192])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 4), (64, 8), (3, 3)])
def test_decode_with_sinks_and_block_order_of_the_batch(group, sinks, hq, hkv):
    okv = _okv()
    lens = [0, 7, 16, sinks, sinks + 1, sinks + 127, sinks + 128, sinks + 145, 700]
    gc, oc, lay, _ = fill(27, hq, hkv, lens, group, sinks=sinks)
    order = np.array([8, 0, 3, 5, 1, 7, 2, 6, 4], np.int32)     # requests in another order than the slots
    q, qn = queries(27, len(lens), hq, hkv)
    ctx = np.array(lens, np.int32)[order]
    got = okv.decode_attention(gc, q, _t(order), _t(lay.table), _t(ctx)).cpu().numpy()
    check_rows(got, O.decode(oc, qn, order, ctx.tolist(), hq), TOL)
    assert gc.device_status() == 0


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("hq,hkv", [(32, 8), (64, 8), (4, 1)])
def test_decode_long_and_peaked(group, hq, hkv):
    """One key far above a flat context of 30,000 tokens (its weight dwarfs the tail's), early and late."""
    okv = _okv()
    n, hot = 30000, (17, 15000, 29999 - 200)
    g = hq // hkv

    def put(kind, b, z):
        if kind == 0:
            z *= 0.05
    gc, oc, lay, zs = fill(28, hq, hkv, [n] * len(hot), group, extra=put)
    q, qn = queries(28, len(hot), hq, hkv)
    # the hot key of each sequence and head points along its first query, 10 nats up
    for b, p in enumerate(hot):
        kz = np.zeros((1, hkv, 128), np.float32)
        for h in range(hkv):
            qr = qn[b, h * g].astype(np.float64) @ oc.r[0][h]
            kz[0, h] = (qr / (qr @ qr) * 10 * math.sqrt(128)).astype(np.float32)
        vz = zs[1][b][p:p + 1]
        oc.append(b, p, kz, vz, pre_rotated=True)
        okv.append_quantize(gc, _t(kz), _t(vz), _t(np.array([b], np.int32)), _t(np.array([p], np.int32)), _t(lay.table),
                            _t(np.array([n] * len(hot), np.int32)), pre_rotated=True)
    seq = np.arange(len(hot), dtype=np.int32)
    got = okv.decode_attention(gc, q, _t(seq), _t(lay.table), _t(np.array([n] * len(hot), np.int32))).cpu().numpy()
    check_rows(got, O.decode(oc, qn, seq, [n] * len(hot), hq), TOL)


@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_decode_flat_and_large_logits(group, scale):
    okv = _okv()
    lens, hq, hkv = [2000, 333], 32, 8
    gc, oc, lay, _ = fill(29, hq, hkv, lens, group)
    q, qn = queries(29, 2, hq, hkv, scale=scale)
    seq = np.arange(2, dtype=np.int32)
    got = okv.decode_attention(gc, q, _t(seq), _t(lay.table), _t(np.array(lens, np.int32))).cpu().numpy()
    check_rows(got, O.decode(oc, qn, seq, lens, hq), TOL)


@pytest.mark.parametrize("group", GROUPS)
def test_decode_value_scales_from_subnormal_to_the_top_of_fp16(group):
    okv = _okv()
    lens, hq, hkv = [900, 900, 900], 8, 2
    gain = {0: 1e-6, 1: 2e4, 2: 1.0}

    def put(kind, b, z):
        if kind == 1:
            z *= gain[b]
            if b == 2:  # growing scales: the weight scale is raised again and again
                z *= np.geomspace(1e-3, 1e3, len(z)).astype(np.float32)[:, None, None]
    gc, oc, lay, _ = fill(30, hq, hkv, lens, group, extra=put)
    q, qn = queries(30, 3, hq, hkv)
    seq = np.arange(3, dtype=np.int32)
    got = okv.decode_attention(gc, q, _t(seq), _t(lay.table), _t(np.array(lens, np.int32))).cpu().numpy()
    check_rows(got, O.decode(oc, qn, seq, lens, hq), TOL)


def test_decode_flags_bad_blocks_and_keeps_other_entries():
    okv = _okv()
    lens, hq, hkv = [700, 700, 700], 32, 8
    gc, oc, lay, _ = fill(31, hq, hkv, lens, 128)
    table = lay.table.copy()
    table[1, 3] = lay.num_blocks + 7
    q, qn = queries(31, 3, hq, hkv)
    seq, ctx = np.array([0, 1, 9], np.int32), np.array(lens, np.int32)
    got = okv.decode_attention(gc, q, _t(seq), _t(table), _t(ctx)).cpu().numpy()
    assert gc.device_status() == okv.DEV_BAD_BLOCK | okv.DEV_BAD_SLOT
    check_rows(got[:1], O.decode(oc, qn[:1], [0], [700], hq), TOL)
    assert np.isfinite(got).all() and (got[2] == 0).all()


@pytest.mark.parametrize("bits", [2, 4])
def test_fused_step_equals_append_then_decode_and_replays(bits):
    okv = _okv()
    seed, hq, hkv = 32, 32, 8
    lens = [1, 17, 128, 129, 1000, 2049]
    outs = {}
    for how in ("two", "step", "graph"):
        lay = H.Layout(seed, [n + 4 for n in lens])
        uk, uv = H.rotations(seed, hkv)
        c = okv.Cache(hq, hkv, lay.num_blocks, len(lens), lay.mbps, uk, uv, group=64, bits=bits, num_sink=16)
        slots = np.concatenate([np.full(n - 1, b, np.int32) for b, n in enumerate(lens)])
        pos = np.concatenate([np.arange(n - 1, dtype=np.int32) for n in lens])
        r = np.random.default_rng(seed)
        z = [r.standard_normal((len(slots), hkv, 128)).astype(np.float32) for _ in range(2)]
        okv.append_quantize(c, _t(z[0]), _t(z[1]), _t(slots), _t(pos), _t(lay.table), _t(np.array(lens, np.int32) - 1),
                            pre_rotated=True)
        seq, p, ctx = (_t(x) for x in (np.arange(6, dtype=np.int32), np.array(lens, np.int32) - 1,
                                       np.array(lens, np.int32)))
        table = _t(lay.table)
        k, v, q = (torch.zeros(6, h, 128, dtype=torch.bfloat16, device="cuda") for h in (hkv, hkv, hq))
        out = torch.zeros(6, hq, 128, dtype=torch.bfloat16, device="cuda")
        call = okv.DecodeStepCall(c, k, v, seq, p, ctx, q, seq, table, ctx, out=out, graph=how == "graph")
        got = []
        for i in range(3):
            for x in (k, v, q):
                x.copy_(torch.from_numpy(r.standard_normal(x.shape).astype(np.float32)))
            if how == "two":
                okv.append_quantize(c, k, v, seq, p, table, ctx)
                okv.decode_attention(c, q, seq, table, ctx, out=out)
            else:
                call()
            got.append(out.clone())
            p += 1
            ctx += 1
        torch.cuda.synchronize()
        assert c.device_status() == 0
        outs[how] = (torch.stack(got), c.pages.clone(), c.ring.clone(), c.sink.clone())
    for how in ("step", "graph"):
        for a, b in zip(outs[how], outs["two"]):
            assert torch.equal(a, b), how


# ------------------------------------------------------------------ chunked prefill

@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("tokens,length,sinks", [(1, 1, 0), (1, 500, 0), (16, 16, 16), (63, 200, 0), (129, 129, 48),
                                                 (130, 901, 16), (200, 777, 0)])
def test_chunked_prefill_matches_the_oracle(group, hq, hkv, tokens, length, sinks):
    okv = _okv()
    gc, oc, lay, _ = fill(33, hq, hkv, [length, 40], group, sinks=sinks)
    q, qn = queries(33, tokens, hq, hkv)
    got = okv.prefill_attention(gc, q, 0, length, _t(lay.table))
    want = O.prefill(oc, qn, 0, length, hq)
    assert gc.device_status() == 0
    check_rows(got.cpu().numpy(), want, TOL)
    out = torch.empty(tokens, hq, 128, dtype=torch.bfloat16, device="cuda")
    okv.prefill_attention(gc, q, 0, length, _t(lay.table), out=out)
    check_rows(out.float().cpu().numpy(), want, TOL + 2.0 ** -8)


@pytest.mark.parametrize("group", GROUPS)
def test_chunked_prefill_skips_bad_blocks_and_takes_large_scales(group):
    okv = _okv()

    def put(kind, b, z):
        if kind == 1:
            z *= 2e3
    gc, oc, lay, _ = fill(34, 8, 2, [600], group, extra=put)
    q, qn = queries(34, 100, 8, 2)
    got = okv.prefill_attention(gc, q, 0, 600, _t(lay.table)).cpu().numpy()
    check_rows(got, O.prefill(oc, qn, 0, 600, 8), TOL)
    table = lay.table.copy()
    table[0, 5] = -1
    got = okv.prefill_attention(gc, q, 0, 600, _t(table)).cpu().numpy()
    assert np.isfinite(got).all() and gc.device_status() == okv.DEV_BAD_BLOCK


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("length,tokens,lost", [(600, 40, 29), (598, 150, 29), (597, 5, 3), (600, 600, 29)])
@pytest.mark.parametrize("bf16", [False, True])
def test_chunked_prefill_with_a_lost_block_reads_the_rest(group, length, tokens, lost, bf16):
    """A block id outside the pool: its code positions are skipped, window positions in the same block are not
    (block 29 holds positions 464 .. 479, the window of 600 tokens starts at 472)."""
    okv = _okv()
    hq, hkv = 8, 2
    gc, oc, lay, _ = fill(35, hq, hkv, [length], group)
    q, qn = queries(35, tokens, hq, hkv)
    table = lay.table.copy()
    table[0, lost] = lay.num_blocks + 1
    out = torch.empty(tokens, hq, 128, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    okv.prefill_attention(gc, q, 0, length, _t(table), out=out)
    assert gc.device_status() == okv.DEV_BAD_BLOCK
    gone = np.arange(16 * lost, min(16 * lost + 16, length - 128))
    want = np.zeros((tokens, hq, 128))
    for h in range(hkv):
        keys, vals = (oc.values(0, kind, h, length) for kind in (0, 1))
        for t in range(tokens):
            seen = np.setdiff1d(np.arange(length - tokens + t + 1), gone)
            if not len(seen):
                continue
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                x = keys[seen] @ (qn[t, j].astype(np.float64) @ oc.r[0][h]) / math.sqrt(128)
                w = np.exp(x - x.max())
                want[t, j] = (w / w.sum()) @ vals[seen] @ oc.r[1][h].T
    check_rows(out.float().cpu().numpy(), want, TOL + (2.0 ** -8 if bf16 else 0))


@pytest.mark.parametrize("group", [128, 32])
def test_chunked_prefill_rows_keep_apart(group):
    """An infinite query row leaves the other rows alone; values at the top of fp16 saturate and stay finite."""
    okv = _okv()

    def put(kind, b, z):
        if kind == 1:
            z[::7] *= 3e4
    gc, oc, lay, _ = fill(36, 8, 2, [500], group, extra=put)
    q, qn = queries(36, 90, 8, 2)
    out = torch.empty(90, 8, 128, dtype=torch.bfloat16, device="cuda")
    okv.prefill_attention(gc, q, 0, 500, _t(lay.table), out=out)
    assert torch.isfinite(out).all() and gc.device_status() == 0
    bad = q.clone()
    bad[33, 5, 7] = float("inf")
    got = torch.empty_like(out)
    okv.prefill_attention(gc, bad, 0, 500, _t(lay.table), out=got)
    keep = torch.ones(90, 8, dtype=torch.bool, device="cuda")
    keep[33, 5] = False
    assert torch.equal(got[keep], out[keep])


@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("hq,hkv,length,tokens", [(32, 8, 700, 300), (40, 2, 1333, 251), (64, 64, 400, 390), (6, 2, 2100, 2100)])
@pytest.mark.parametrize("stage_r,off", [(True, 0), (False, 0), (True, 3)])
def test_chunked_prefill_with_many_rows(group, hq, hkv, length, tokens, stage_r, off):
    """Chunks whose rotations run on the tensor cores, without the staged image of R, and into an output off 16
    bytes (both take the other rotations): every row against 64 bits, rows in front of the output untouched."""
    okv = _okv()
    gc, oc, lay, _ = fill(41, hq, hkv, [length], group, sinks=16, stage_r=stage_r)
    q, qn = queries(41, tokens, hq, hkv)
    buf = torch.full((off + tokens * hq * 128 + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[off:off + tokens * hq * 128].view(tokens, hq, 128)
    okv.prefill_attention(gc, q, 0, length, _t(lay.table), out=out)
    assert gc.device_status() == 0
    assert (buf[:off] == 7).all() and (buf[off + tokens * hq * 128:] == 7).all()
    got = out.float().cpu().numpy()
    seen = np.arange(length)[None] <= np.arange(length - tokens, length)[:, None]
    for h in range(hkv):
        keys, vals = (oc.values(0, kind, h, length) for kind in (0, 1))
        for j in range(h * hq // hkv, (h + 1) * hq // hkv):
            x = np.where(seen, (qn[:, j].astype(np.float64) @ oc.r[0][h]) @ keys.T / math.sqrt(128), -np.inf)
            w = np.exp(x - x.max(1, keepdims=True))
            check_rows(got[:, j], (w / w.sum(1, keepdims=True)) @ vals @ oc.r[1][h].T, TOL + 2.0 ** -8)


def test_chunked_prefill_with_many_rows_scales_and_keeps_rows_apart():
    """Values times 2^k give the output times 2^k: a row's scale leaves nothing of its 2^-12 to the values' size.
    An infinite query row leaves the others alone."""
    okv = _okv()
    outs = []
    for k in (0, -9, 10):
        def put(kind, b, z):
            if kind == 1:
                z *= 2.0 ** k
        gc, oc, lay, _ = fill(42, 32, 8, [500], 128, extra=put)
        q, _ = queries(42, 310, 32, 8)
        outs.append(torch.empty(310, 32, 128, dtype=torch.bfloat16, device="cuda"))
        okv.prefill_attention(gc, q, 0, 500, _t(lay.table), out=outs[-1])
        assert gc.device_status() == 0
    # 2^-9: (scale, min) pairs and fp16 rows near 2^-9 keep 11 bits down to 2^-14, a unit of 2^-24 below: against
    # rows of norm ~2^-9 their rounding is 2^-15 a value; both bf16 outputs round by 2^-9, values and weights 2^-11
    for o, k in zip(outs[1:], (-9, 10)):
        a, b = outs[0].double(), o.double() * 2.0 ** -k
        assert ((a - b).norm(dim=-1) / a.norm(dim=-1)).max() <= 2 * 2.0 ** -9 + 2.0 ** -8
    bad = q.clone()
    bad[77, 9, 3] = float("inf")
    got = torch.empty_like(outs[-1])
    okv.prefill_attention(gc, bad, 0, 500, _t(lay.table), out=got)
    keep = torch.ones(310, 32, dtype=torch.bool, device="cuda")
    keep[77, 9] = False
    assert torch.equal(got[keep], outs[-1][keep])


@pytest.mark.parametrize("val", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", [5, 100, 260])   # a sink row, codes, the window
@pytest.mark.parametrize("kind", [0, 1])
def test_chunked_prefill_rows_before_a_token_that_is_not_finite(val, where, kind):
    """The cache holds such a token's channel as zero or at fp16's end, so it reaches nobody through the mask."""
    okv = _okv()

    def put(k, b, z):
        if k == kind:
            z[where, 1, 17] = val
    outs = []
    for extra in (None, put):
        gc, _, lay, _ = fill(45, 8, 2, [300], 64, sinks=16, extra=extra)
        q, _ = queries(45, 300, 8, 2)
        outs.append(torch.empty(300, 8, 128, dtype=torch.bfloat16, device="cuda"))
        okv.prefill_attention(gc, q, 0, 300, _t(lay.table), out=outs[-1])
    assert torch.equal(outs[0][:where], outs[1][:where]) and torch.equal(outs[0][:, :4], outs[1][:, :4])
    assert torch.isfinite(outs[1]).all()
