"""Operators of the 4-bit serving path and the cases they are measured on.

Four operators, in the order in which a serving step runs them:

  plan     block tables and slot maps built on the GPU from request lengths
  rope     norms of queries and keys for each head with the position rotation
  decode   one decode step over a cache held in 4 bits (append, then attention)
  prefill  one prompt chunk into that cache and its causal attention over it

`run` computes them in plain torch operations, or, where `own` is set, makes
the calls that a user makes of the package.  Both take what `prepare` gives.
"""
import math

import numpy as np
import torch

own = False

D, BLOCK, WINDOW = 128, 16, 128


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # every running request of a server gains one token; a few entries are padding of a captured batch
        dict(name="plan_decode_256", op="plan", batch=256, tokens=256, most=1, low=1000, high=65536, pad=6, slots=256,
             blocks=4352, short=False),
        # 64 prompts of 1K to 64K tokens admitted at once
        dict(name="plan_prompts_64", op="plan", batch=64, tokens=1 << 20, most=65536, low=0, high=0, pad=0, slots=64,
             blocks=4096, short=False),
        # decode steps and prompt chunks mixed, odd sizes, a pool that runs out before the last requests
        dict(name="plan_mixed_1001", op="plan", batch=1001, tokens=70001, most=513, low=1, high=9000, pad=17,
             slots=1200, blocks=611, short=True),
        # one decode step's queries and keys
        dict(name="rope_decode_64", op="rope", tokens=64, hq=32, hkv=8, rot=128, interleaved=False, type="bf16",
             far=100000, pad=0),
        # a prompt chunk's, taken from one fused projection
        dict(name="rope_chunk_8192", op="rope", tokens=8192, hq=32, hkv=8, rot=128, interleaved=False, type="bf16",
             far=32768, pad=0),
        # half the channels rotated, adjacent pairs, far positions, fp16 projections, padding rows at the end
        dict(name="rope_partial_1021", op="rope", tokens=1021, hq=64, hkv=8, rot=64, interleaved=True, type="fp16",
             far=1000003, pad=5),
        # the smallest decode step: one sequence, one KV head
        dict(name="decode_1x2048", op="decode", batch=1, low=2048, high=2048, hq=4, hkv=1, group=128, sinks=0),
        # four sequences of 100,000 tokens
        dict(name="decode_4x100k", op="decode", batch=4, low=100001, high=100001, hq=32, hkv=8, group=128, sinks=0),
        # a ragged batch, two scales per vector, sink tokens kept in fp16
        dict(name="decode_ragged_16", op="decode", batch=16, low=1000, high=32768, hq=32, hkv=8, group=64, sinks=64),
        # eight query heads per KV head, one sequence of 131,072 tokens
        dict(name="decode_1x131k_g8", op="decode", batch=1, low=131072, high=131072, hq=64, hkv=8, group=128, sinks=0),
        # a 1,024-token chunk at the end of 32,768 tokens
        dict(name="prefill_1024_32k", op="prefill", tokens=1024, context=32768, hq=32, hkv=8, group=128),
        # a short odd chunk of a short prompt, four scales per vector
        dict(name="prefill_203_2999", op="prefill", tokens=203, context=2999, hq=8, hkv=2, group=32),
    ]


def _spread(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "decode", "decode", "prefill"])
    if op == "plan":
        most = rng.choice([1, _spread(rng, 2, 65536)])
        batch = _spread(rng, 1, 2000 if most == 1 else max(1, min(2000, (1 << 20) // most)))
        low = _spread(rng, 1, 4000)
        high = _spread(rng, low, 65536)
        return dict(op=op, batch=batch, tokens=max(1, min(1 << 20, batch * most - rng.randint(0, most // 3))),
                    most=most, low=low, high=high, pad=rng.randint(0, 1 + batch // 20), slots=batch + rng.randint(0, 99),
                    blocks=(high + most + 15) // 16 + rng.randint(0, 9), short=rng.random() < 0.3)
    if op == "rope":
        hq, hkv = rng.choice([(4, 1), (32, 8), (64, 8), (8, 8), (24, 3), (40, 5)])
        tokens = _spread(rng, 1, 8192 * 48 // (hq + 2 * hkv) if hq + 2 * hkv > 48 else 8192)
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, rot=rng.choice([128, 128, 64, 96, 32]),
                    interleaved=rng.random() < 0.4, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    far=_spread(rng, 1000, 1 << 20), pad=rng.randint(0, tokens // 8))
    hq, hkv = rng.choice([(4, 1), (8, 1), (8, 2), (16, 8), (32, 8), (64, 8), (8, 8)])
    group = rng.choice([128, 64, 32])
    if op == "decode":
        batch = _spread(rng, 1, 32)
        high = _spread(rng, 300, max(300, min(131072, 400000 * 8 // (batch * hkv))))
        return dict(op=op, batch=batch, low=max(1, high // rng.choice([1, 3, 16, 200])), high=high, hq=hq, hkv=hkv,
                    group=group, sinks=rng.choice([0, 0, 16, 192]))
    tokens = _spread(rng, 1, 1024)
    return dict(op=op, tokens=tokens, context=tokens + _spread(rng, 1, 32768 - 1024), hq=min(hq, 32), hkv=hkv, group=group)


def work(case):
    if case["op"] == "plan":
        # lengths, slots and the popped block ids in; token maps, table entries, lengths and offsets out
        b, t = case["batch"], case["tokens"]
        return {"bytes": 12 * b + 8 * t + 2 * 4 * (t / BLOCK) + 12 * b, "flops": 0}
    if case["op"] == "rope":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
        rows, live = case["hq"] + 2 * case["hkv"], case["tokens"] - case["pad"]
        return {"bytes": live * rows * D * (size + 2) + 4 * case["tokens"],
                "flops": live * (case["hq"] + case["hkv"]) * (4 * D + 3 * case["rot"])}
    ng = D // case["group"]
    if case["op"] == "decode":
        lens, hq, hkv = _lengths(case), case["hq"], case["hkv"]
        full = sum(min(n, WINDOW) + min(case["sinks"], max(0, n - WINDOW)) for n in lens)
        packed = sum(max(0, n - WINDOW - case["sinks"]) for n in lens)
        io = len(lens) * (hq * D * 4 + 2 * hkv * D * 2 + 2 * hkv * (64 + 4 * ng) + 2 * hkv * D * 2)
        return {"bytes": hkv * (packed * (128 + 8 * ng) + full * 512) + io + 2 * hkv * D * D * 4,
                "flops": 4 * D * hq * sum(lens) + 2 * D * D * len(lens) * (2 * hq + 2 * hkv)}
    t, n, hq, hkv = case["tokens"], case["context"], case["hq"], case["hkv"]
    seen = t * (n - t) + t * (t + 1) // 2
    io = t * (hq * D * 4 + 2 * hkv * D * 2 + 2 * hkv * (64 + 4 * ng)) + min(t, WINDOW) * hkv * 512
    return {"bytes": hkv * (n * (128 + 8 * ng)) + io + 2 * hkv * D * D * 4,
            "flops": 4 * D * hq * seen + 2 * D * D * t * (2 * hq + 2 * hkv)}


def _lengths(case):
    """Lengths of a decode batch: spread over [low, high] by their logarithm, the longest first."""
    b, low, high = case["batch"], case["low"], case["high"]
    return [int(round(high * (low / high) ** (i / max(1, b - 1)))) for i in range(b)]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _orthogonal(gen, heads):
    """[heads][128][128] orthogonal matrices in fp32: the bases of a calibration."""
    q, r = torch.linalg.qr(_normal(gen, heads, D, D, dtype=torch.float64))
    return (q * torch.sign(torch.diagonal(r, dim1=-2, dim2=-1))[:, None, :]).float().contiguous()


def _rotation(u):
    """R = U H P_br (fp64): H the normalised Hadamard matrix, P_br the 7-bit reversal of columns."""
    i = np.arange(D)
    bits = i[:, None] & i[None, :]
    parity = np.zeros_like(bits)
    for k in range(7):
        parity ^= (bits >> k) & 1
    rev = sum(((i >> k) & 1) << (6 - k) for k in range(7))
    h = torch.from_numpy((1.0 - 2.0 * parity)[:, rev] / math.sqrt(D)).cuda()
    return u.double() @ h


def _quantise(z, group):
    """Codes 0..15 (uint8) and fp16 scale and minimum of every `group` channels of z (fp32 [..., 128])."""
    x = z.reshape(*z.shape[:-1], D // group, group)
    lo, hi = x.amin(-1), x.amax(-1)
    s, m = ((hi - lo) / 15.0).clamp(-65504, 65504).half(), lo.clamp(-65504, 65504).half()
    sf, mf = s.float()[..., None], m.float()[..., None]
    c = torch.where(sf > 0, torch.round((x - mf) / torch.where(sf > 0, sf, 1.0)).clamp(0, 15), 0.0)
    return c.to(torch.uint8).reshape(z.shape), s, m


def _pack(z_k, z_v, group):
    """Blocks of 16 tokens in the cache's 4-bit layout from rotated values [blocks][16][hkv][128]:
    keys token by token, 64 bytes each, their 32-bit words w stored in the order 4 (w % 4) + w / 4; values
    as 16-byte chunks of four tokens' bytes; then fp16 (scale, minimum) pairs of keys and of values."""
    n, _, hkv, _ = z_k.shape
    parts = []
    (kc, ks, km), (vc, vs, vm) = (_quantise(z.permute(0, 2, 1, 3), group) for z in (z_k, z_v))
    k = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(n, hkv, 16, 4, 4, 4).permute(0, 1, 2, 4, 3, 5)
    v = (vc[..., 0::2] | (vc[..., 1::2] << 4)).reshape(n, hkv, 4, 4, 2, 4, 8).permute(0, 1, 4, 6, 2, 5, 3)
    parts += [k.reshape(n, hkv, 1024), v.reshape(n, hkv, 1024)]
    for s, m in ((ks, km), (vs, vm)):
        parts.append(torch.stack([s, m], -1).reshape(n, hkv, -1).contiguous().view(torch.uint8))
    return torch.cat(parts, -1)


def _history(gen, lens, after, hkv, group, sinks, mbps):
    """A cache that holds `lens[b]` tokens of sequence b and has blocks for `after[b]`: pages (blocks in a shuffled
    order), block table, fp16 rows of the last 128 tokens at row position % 128, and of the first `sinks` tokens."""
    slots = len(lens)
    blocks = [(n + BLOCK - 1) // BLOCK for n in after]
    total = sum(blocks)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((slots, mbps), -1, dtype=torch.int32, device="cuda")
    for b, part in enumerate(order.split(blocks)):
        table[b, :blocks[b]] = part
    pages = torch.zeros(total, hkv, 2048 + 128 * (D // group), dtype=torch.uint8, device="cuda")
    ring = torch.zeros(slots, hkv, 2, WINDOW, D, dtype=torch.float16, device="cuda")
    sink = torch.zeros(slots, hkv, 2, sinks, D, dtype=torch.float16, device="cuda")
    for b, n in enumerate(lens):
        if not n:
            continue
        held = (n + BLOCK - 1) // BLOCK
        z = [_normal(gen, held, BLOCK, hkv, D) * sd for sd in (2.0, 1.0)]  # keys spread wider than values
        pages[table[b, :held].long()] = _pack(z[0], z[1], group)
        first = max(0, n - WINDOW)
        for kind in (0, 1):
            rows = z[kind].reshape(-1, hkv, D)
            ring[b, :, kind, torch.arange(first, n, device="cuda") % WINDOW] = \
                rows[first:n].permute(1, 0, 2).half()
            kept = min(n, sinks)
            sink[b, :, kind, :kept] = rows[:kept].permute(1, 0, 2).half()
    return pages, table, ring, sink


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    if op == "plan":
        b, slots, cols, tokens = case["batch"], case["slots"], case["blocks"], case["tokens"]
        slot = torch.randperm(slots, generator=gen, device="cuda")[:b].to(torch.int32)
        live = b - case["pad"] if case["pad"] < b else b
        slot[live:] = -1

        def lengths(low, high, size):
            x = torch.rand(size, generator=gen, device="cuda", dtype=torch.float64)
            return (low * (high / low) ** x).round().to(torch.int32)

        cached = lengths(case["low"], case["high"], b) if case["low"] else torch.zeros(b, dtype=torch.int32, device="cuda")
        new = torch.ones(b, dtype=torch.int32, device="cuda") if case["most"] == 1 else \
            lengths(1 if case["low"] else 1000, case["most"], b)
        need = int(((cached + new + 15) // 16 - (cached + 15) // 16)[:live].sum())
        pool = max(1, need * 2 // 3 if case["short"] else need + 50)
        table = torch.randint(0, 1 << 20, (slots, cols), generator=gen, device="cuda", dtype=torch.int32)
        st = dict(op=op, slot=slot, cached=cached, new=new, table=table, tokens=tokens,
                  slot_lens=torch.randint(0, 1000, (slots,), generator=gen, device="cuda", dtype=torch.int32),
                  free=torch.randperm(pool + 9, generator=gen, device="cuda").to(torch.int32),
                  count=torch.tensor([pool], dtype=torch.int32, device="cuda"))
        if own:
            from int2_kv_cache_rotate_b200 import okv
            st["plan"] = okv.AppendPlan(b, tokens)
        return st
    if op == "rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        kind = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["type"]]
        qkv = (_normal(gen, t, (hq + 2 * hkv) * D) * 1.5).to(kind)
        pos = torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        if case["pad"]:
            pos[t - case["pad"]:] = -1
        rot = case["rot"]
        freq = (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        out = [torch.zeros(t, h, D, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
        return dict(op=op, q=qkv[:, :hq * D].view(t, hq, D), k=qkv[:, hq * D:(hq + hkv) * D].view(t, hkv, D),
                    v=qkv[:, (hq + hkv) * D:].view(t, hkv, D), pos=pos, freq=freq, out=out,
                    wq=1.0 + 0.2 * _normal(gen, D), wk=1.0 + 0.2 * _normal(gen, D), eps=1e-6,
                    interleaved=case["interleaved"])
    hq, hkv, group = case["hq"], case["hkv"], case["group"]
    sinks = case.get("sinks", 0)
    lens = [n - 1 for n in _lengths(case)] if op == "decode" else [case["context"] - case["tokens"]]
    after = [n + (1 if op == "decode" else case["tokens"]) for n in lens]
    mbps = (max(after) + BLOCK - 1) // BLOCK
    u_k, u_v = _orthogonal(gen, hkv), _orthogonal(gen, hkv)
    pages, table, ring, sink = _history(gen, lens, after, hkv, group, sinks, mbps)
    t = len(lens) if op == "decode" else case["tokens"]
    i32 = dict(dtype=torch.int32, device="cuda")
    st = dict(op=op, hq=hq, hkv=hkv, group=group, sinks=sinks, table=table, after=after,
              q=_normal(gen, t, hq, D).bfloat16(), k=(2.0 * _normal(gen, t, hkv, D)).bfloat16(),
              v=_normal(gen, t, hkv, D).bfloat16(),
              slots=torch.arange(t, **i32) if op == "decode" else torch.zeros(t, **i32),
              pos=torch.tensor(lens, **i32) if op == "decode" else lens[0] + torch.arange(t, **i32),
              lens=torch.tensor(after, **i32))
    if own:
        from int2_kv_cache_rotate_b200 import okv
        c = okv.Cache(hq, hkv, pages.shape[0], len(lens), mbps, u_k.cpu(), u_v.cpu(), num_sink=sinks, group=group, bits=4)
        c.pages.copy_(pages.reshape(-1))
        c.ring.copy_(ring)
        c.sink.copy_(sink)
        st["cache"] = c
        st["out"] = torch.empty(t, hq, D, dtype=torch.bfloat16, device="cuda")
        size = okv.decode_workspace_bytes(c, t) if op == "decode" else okv.prefill_workspace_bytes(c, t)
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    else:
        st.update(pages=pages, ring=ring, sink=sink, r_k=_rotation(u_k).float(), r_v=_rotation(u_v).float())
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if own:
        return _own(state)
    if op == "plan":
        return _plan_plain(state)
    if op == "rope":
        return _rope_plain(state)
    return _attend_plain(state)


def _own(st):
    from int2_kv_cache_rotate_b200 import okv
    if st["op"] == "plan":
        p = st["plan"]
        p.build(st["slot"], st["cached"], st["new"], st["table"], st["slot_lens"], st["free"], st["count"])
        return [st["table"], st["slot_lens"], p.tok_slot, p.tok_pos, p.context_lens, p.cu_tokens, p.free_count]
    if st["op"] == "rope":
        q, k, v = st["out"]
        okv.qk_norm_rope(st["q"], st["k"], st["pos"], st["freq"], q_weight=st["wq"], k_weight=st["wk"], eps=st["eps"],
                         v=st["v"], interleaved=st["interleaved"], q_out=q, k_out=k, v_out=v)
        return [q, k, v]
    c = st["cache"]
    if st["op"] == "decode":
        okv.decode_step(c, st["k"], st["v"], st["slots"], st["pos"], st["lens"], st["q"], st["slots"], st["table"],
                        st["lens"], out=st["out"], ws=st["ws"])
    else:
        okv.append_quantize(c, st["k"], st["v"], st["slots"], st["pos"], st["table"], st["lens"])
        okv.prefill_attention(c, st["q"], 0, st["after"][0], st["table"], out=st["out"], ws=st["ws"])
    return [st["out"], c.ring]


def _plan_plain(st):
    """Requests in order: each gets ceil((old + new) / 16) - ceil(old / 16) blocks from the end of the free list and a
    row (slot, position) for each new token.  The first request that the pool or the token rows do not hold, and all
    after it, get nothing; rows behind the last token are -1."""
    slot, old, new, free = st["slot"].long(), st["cached"].long(), st["new"].long(), st["free"]
    count, tokens = st["count"].long(), st["tokens"]
    table, slot_lens = st["table"], st["slot_lens"]
    live = slot >= 0
    have, want = (old + 15) // 16, (old + new + 15) // 16
    blocks, rows = torch.where(live, want - have, 0), torch.where(live, new, 0)
    sum_b, sum_t = blocks.cumsum(0), rows.cumsum(0)
    took = live & (sum_b <= count) & (sum_t <= tokens)
    rows, blocks = torch.where(took, rows, 0), torch.where(took, blocks, 0)
    end = rows.cumsum(0)
    lens = torch.where(live, old + rows, 0)
    index = torch.arange(tokens, device="cuda")
    owner = torch.searchsorted(end, index, right=True).clamp(max=len(slot) - 1)
    there = index < end[-1]
    tok_slot = torch.where(there, slot[owner], -1).int()
    tok_pos = torch.where(there, old[owner] + index - (end - rows)[owner], -1).int()
    col = torch.arange(table.shape[1], device="cuda")
    gets = (took[:, None]) & (col >= have[:, None]) & (col < want[:, None])
    source = count - 1 - ((blocks.cumsum(0) - blocks)[:, None] + col - have[:, None])
    # entries of padding requests go to a row of their own, behind the table
    grown = torch.cat([table, table[:1]])
    at = torch.where(live, slot, table.shape[0])
    grown[at] = torch.where(gets, free[source.clamp(0, len(free) - 1)], grown[at])
    grown_lens = torch.cat([slot_lens, slot_lens[:1]])
    grown_lens[at] = lens.int()
    cu = torch.cat([end.new_zeros(1), end]).int()
    return [grown[:-1], grown_lens[:-1], tok_slot, tok_pos, lens.int(), cu, (count - blocks.sum()).int()]


def _rope_plain(st):
    pos = st["pos"]
    angle = torch.remainder(pos.double()[:, None] * st["freq"].double(), 2 * math.pi)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot = 2 * st["freq"].shape[0]
    live = (pos >= 0)[:, None, None]

    def one(x, w, out):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w
        if st["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.where(live, torch.cat([turned, y[..., rot:]], -1).bfloat16(), out)

    q, k, v = st["out"]
    return [one(st["q"], st["wq"], q), one(st["k"], st["wk"], k),
            torch.where(live, st["v"].bfloat16(), v)]


def _unpack(pg, kind, group):
    """fp32 values [..., 16, 128] of blocks pg [..., 2048 + 128 ng] (uint8)."""
    lead, ng = pg.shape[:-1], D // group
    if kind == 0:
        b = pg[..., :1024].reshape(*lead, 16, 4, 4, 4).transpose(-3, -2)
    else:
        b = pg[..., 1024:2048].reshape(*lead, 2, 8, 4, 4, 4)
        n = len(lead)
        b = b.permute(*range(n), n + 2, n + 4, n, n + 3, n + 1)
    b = b.reshape(*lead, 16, 64)
    code = torch.stack([b & 15, b >> 4], -1).reshape(*lead, 16, ng, group).float()
    start = 2048 + 64 * ng * kind
    sm = pg[..., start:start + 64 * ng].contiguous().view(torch.float16).float().reshape(*lead, 16, ng, 2)
    return (code * sm[..., :1] + sm[..., 1:]).reshape(*lead, 16, D)


def _cache_plain(st, kind, z_new, new_slot, new_pos, ring):
    """What attention reads for each sequence, fp32 [batch][hkv][length][128]: 4-bit values, and the fp16 rows of sink
    tokens and of the last 128 positions.  z_new: the rotated new tokens, written first."""
    table, group, lens = st["table"], st["group"], st["lens"].long()
    n = max(st["after"])
    val = _unpack(st["pages"][table.long()], kind, group)              # [batch][blocks][hkv][16][128]
    val = val.permute(0, 2, 1, 3, 4).reshape(len(lens), st["hkv"], -1, D)[:, :, :n].clone()
    code, s, m = _quantise(z_new, group)
    ng = D // group
    back = code.reshape(*code.shape[:-1], ng, group).float() * s.float()[..., None] + m.float()[..., None]
    val[new_slot, :, new_pos] = back.reshape(z_new.shape)
    at = torch.arange(n, device="cuda")
    fresh = (at >= (lens - WINDOW)[:, None]) & (at < lens[:, None])
    val = torch.where(fresh[:, None, :, None], ring[:, :, kind].float()[:, :, at % WINDOW], val)
    if st["sinks"]:
        k = min(n, st["sinks"])
        first = (at[:k] < lens[:, None])[:, None, :, None]
        val[:, :, :k] = torch.where(first, st["sink"][:, :, kind, :k].float(), val[:, :, :k])
    return val


def _attend_plain(st):
    hq, hkv, lens = st["hq"], st["hkv"], st["lens"].long()
    new_slot, new_pos = st["slots"].long(), st["pos"].long()
    z = [torch.einsum("thc,hcd->thd", x.float(), r) for x, r in ((st["k"], st["r_k"]), (st["v"], st["r_v"]))]
    ring = st["ring"].clone()
    if st["sinks"]:  # new tokens that are sink tokens too
        st = dict(st, sink=st["sink"].clone())
    kept = new_pos >= lens[new_slot] - WINDOW
    spare = torch.cat([ring, ring[:1]])  # rows that leave the window go to a slot of their own
    at = torch.where(kept, new_slot, ring.shape[0])
    for_sink = torch.where(new_pos < st["sinks"], new_slot, ring.shape[0]) if st["sinks"] else None
    both = torch.stack(z, 2).half()                                     # [tokens][hkv][2][128]
    spare[at, :, :, new_pos % WINDOW] = both
    ring = spare[:-1]
    if for_sink is not None:
        grown = torch.cat([st["sink"], st["sink"][:1]])
        grown[for_sink, :, :, new_pos.clamp(max=st["sinks"] - 1)] = both
        st["sink"] = grown[:-1]
    q = torch.einsum("thgc,hcd->thgd", st["q"].float().reshape(-1, hkv, hq // hkv, D), st["r_k"])
    keys = _cache_plain(st, 0, z[0], new_slot, new_pos, ring)
    at = torch.arange(keys.shape[2], device="cuda")
    if st["op"] == "decode":                                            # [batch][hkv][g][length]
        score = torch.einsum("bhgd,bhnd->bhgn", q, keys)
        seen = (at < lens[:, None])[:, None, None]
    else:                                                               # [hkv][tokens * g][length]
        score = torch.einsum("thgd,hnd->htgn", q, keys[0])
        seen = (at <= new_pos[:, None])[None, :, None]
    del keys
    score = torch.where(seen, score / math.sqrt(D), -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    del score
    p = p / p.sum(-1, keepdim=True)
    values = _cache_plain(st, 1, z[1], new_slot, new_pos, ring)
    if st["op"] == "decode":
        o = torch.einsum("bhgn,bhnd->bhgd", p, values)
    else:
        o = torch.einsum("htgn,hnd->thgd", p, values[0])
    o = torch.einsum("bhgd,hcd->bhgc", o, st["r_v"])
    return [o.reshape(-1, hq, D).bfloat16(), ring]


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    global own
    if case["op"] == "plan":
        return None  # whole numbers throughout
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        return _rope_exact(st)
    return _attend_exact(st)


def _rope_exact(st):
    """x / rms(x) * w, then each pair (a, b) of channels turned by position * frequency, as a complex product."""
    pos, rot = st["pos"].double(), 2 * st["freq"].shape[0]
    half = rot // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + half)
    unit = torch.polar(torch.ones(len(pos), half, dtype=torch.float64, device="cuda"),
                       torch.outer(pos, st["freq"].double()))
    got = []
    for x, w, out in ((st["q"], st["wq"], st["out"][0]), (st["k"], st["wk"], st["out"][1])):
        y = out.double().clone()
        for h in range(x.shape[1]):
            a = x[:, h].double()
            a = a / ((a * a).sum(1, keepdim=True) / D + st["eps"]).sqrt() * w.double()
            c = torch.complex(a[:, first], a[:, second]) * unit
            a[:, first], a[:, second] = c.real.contiguous(), c.imag.contiguous()
            y[:, h] = torch.where((pos >= 0)[:, None], a, y[:, h])
        got.append(y)
    v = torch.where((pos >= 0)[:, None, None], st["v"].double(), st["out"][2].double())
    return got + [v]


def _attend_exact(st):
    hq, hkv, group = st["hq"], st["hkv"], st["group"]
    g, ng, sinks = hq // hkv, D // group, st["sinks"]
    r = [st[n].double() for n in ("r_k", "r_v")]
    pages, table = st["pages"], st["table"].long()
    ring = st["ring"].double().clone()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    ch = torch.arange(D, device="cuda")
    byte, high = ch // 2, (ch % 2).bool()
    word = byte // 4
    k_off = 16 * (word % 4) + 4 * (word // 4) + byte % 4                 # within a token's 64 bytes
    tile, lane = byte // 8, byte % 8
    v_off = 1024 + 512 * (tile // 4) + 64 * lane + 4 * (tile % 4)         # of tokens 0..3; 16 bytes on per four tokens
    new_pos, new_slot = st["pos"].long(), st["slots"].long()
    for b, n in enumerate(st["after"]):
        mine = torch.nonzero(new_slot == b)[:, 0]
        at = torch.arange(n, device="cuda")
        blk, t = table[b, at // BLOCK], at % BLOCK
        for h in range(hkv):
            val = []
            for kind, x in ((0, st["k"]), (1, st["v"])):
                rows = pages[:, h]
                off = (t * 64)[:, None] + k_off if kind == 0 else (16 * (t // 4) + t % 4)[:, None] + v_off
                code = rows[blk[:, None], off].to(torch.int16)
                code = torch.where(high, code >> 4, code & 15).double()
                pair = 2048 + 64 * ng * kind + 4 * (t[:, None] * ng + ch // group)
                half = [(rows[blk[:, None], pair + 2 * i].to(torch.int32)
                         | (rows[blk[:, None], pair + 2 * i + 1].to(torch.int32) << 8)) for i in (0, 1)]
                s, m = [x_.to(torch.int16).view(torch.float16).double() for x_ in half]
                y = code * s + m
                z = x[mine, h].double() @ r[kind][h]
                zg = z.reshape(len(mine), ng, group)
                lo, hi = zg.amin(-1, keepdim=True), zg.amax(-1, keepdim=True)
                sn, mn = ((hi - lo) / 15).half().double(), lo.half().double()
                y[new_pos[mine]] = (((zg - mn) / sn).round().clamp(0, 15) * sn + mn).reshape(z.shape)
                last = max(0, n - WINDOW)
                row = ring[b, h, kind].clone()
                keep = new_pos[mine] >= last
                row[new_pos[mine][keep] % WINDOW] = z[keep]
                ring[b, h, kind] = row
                fresh = at[last:]
                seen_row = row.half().double()
                y[last:] = seen_row[fresh % WINDOW]
                if sinks:
                    k = min(n, sinks)
                    first = st["sink"][b, h, kind, :k].double().clone()
                    early = new_pos[mine] < k
                    first[new_pos[mine][early]] = z[early].half().double()
                    y[:k] = first
                val.append(y)
            q = st["q"][mine, h * g:(h + 1) * g].double() @ r[0][h]       # [new][g][128]
            score = q.reshape(-1, D) @ val[0].T / math.sqrt(D)
            limit = (new_pos[mine] if st["op"] == "prefill" else new_pos[mine] * 0 + n - 1).repeat_interleave(g)
            score = score.masked_fill(at[None] > limit[:, None], -math.inf)
            o = torch.softmax(score, -1) @ val[1] @ r[1][h].T
            out[mine, h * g:(h + 1) * g] = o.reshape(len(mine), g, D)
    return [out, ring]
