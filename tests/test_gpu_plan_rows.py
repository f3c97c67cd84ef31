"""Decode over the plan's token rows: whatever requests of a batch are padding,
dropped, without a new token or with several, row i of the queries and of the
output belongs to token row i, and a row without a query of its own gives zeros.

Bar: 2e-3 of a row's largest value for the attention and half a bf16 step."""
import numpy as np
import pytest

from oracle import okv_oracle as O
from tests import gpu_helpers as H
from tests.test_gpu_plan import _case, _dev, _run, plan_loop

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TOL = 2e-3 + 2.0 ** -8


def row_lens(want, tokens):
    lens = np.zeros(tokens, np.int64)
    for b, n in enumerate(want["lens"]):
        if want["cu"][b + 1] > want["cu"][b]:
            lens[want["cu"][b + 1] - 1] = n
    return lens


@pytest.mark.parametrize("batch,slots,cols,max_old,max_new,pool,tokens,pad,bad", [
    (0, 3, 4, 0, 0, 7, 5, 0, 0), (1, 1, 1, 0, 1, 1, 1, 0, 0), (7, 9, 64, 500, 1, 50, 7, 2, 0),
    (33, 40, 64, 500, 40, 1000, 2000, 5, 0), (64, 64, 64, 0, 1000, 6000, 64001, 0, 0),
    (100, 120, 40, 600, 33, 900, 4000, 9, 1), (100, 120, 40, 600, 33, 900, 9001, 9, 1),
    (200, 250, 80, 1200, 50, 90, 9000, 11, 0), (200, 250, 80, 1200, 50, 9000, 1003, 11, 0),
    (2049, 2500, 70, 1000, 3, 3000, 8000, 20, 1), (5000, 6000, 70, 1000, 20, 9000, 60000, 99, 1)])
def test_row_lengths_equal_the_loop(batch, slots, cols, max_old, max_new, pool, tokens, pad, bad):
    for seed in (1, 2):
        case = _case(seed, batch, slots, cols, max_old, max_new, pool, tokens, pad, bad)
        plan, _, _ = _run(case)
        assert np.array_equal(plan.tok_lens.cpu().numpy(), row_lens(plan_loop(*case), tokens))


@pytest.mark.parametrize("bits", [4, 2])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_with_holes_in_the_batch(bits, graph):
    from int2_kv_cache_rotate_b200 import okv
    hq, hkv, slots, cols, blocks, rows = 8, 2, 6, 24, 90, 12
    r = np.random.default_rng(7)
    uk, uv = H.rotations(51, hkv)
    cache = okv.Cache(hq, hkv, blocks, slots, cols, uk, uv, bits=bits, pad_rows=True)
    oc = O.Cache(hkv, uk.astype(np.float64), uv.astype(np.float64), bits=bits)
    free, count = r.permutation(blocks), blocks
    table, slot_lens = torch.full((slots, cols), -1, dtype=torch.int32, device="cuda"), _dev(np.zeros(slots))
    state = (np.full((slots, cols), -1), np.zeros(slots, np.int64))
    # the batch's slots and new tokens, step by step: prompts first, then decode steps with a padding entry, a
    # request without a new token, two that name one slot (both dropped) and one that gains several, all in the middle
    steps = [([3, 5, 0, 1], [3, 3, 3, 3]), ([3, -1, 5, 1], [1, 1, 1, 1]), ([3, 5, 0, 1], [1, 0, 1, 1]),
             ([0, 2, 2, 5], [1, 1, 1, 1]), ([5, 9, 3, 0], [1, 1, 1, 1]), ([1, 3, -1, 5], [1, 6, 1, 1]),
             ([-1, -1, -1, 0], [1, 1, 1, 1]), ([-1, 1, 3, 5], [0, 0, 0, 0])]
    B = 4
    plan = okv.AppendPlan(B, rows)
    d_seq, d_old, d_new, d_free = (_dev(x) for x in (np.zeros(B), np.zeros(B), np.zeros(B), free))
    plan.free_count.fill_(blocks)
    k, v, q = (torch.zeros(rows, h, 128, dtype=torch.bfloat16, device="cuda") for h in (hkv, hkv, hq))
    out = torch.zeros(rows, hq, 128, dtype=torch.bfloat16, device="cuda")
    ws = okv.workspace(cache, rows)

    def run():
        plan.build(d_seq, d_old, d_new, table, slot_lens, d_free, plan.free_count)
        okv.decode_step(cache, k, v, plan.tok_slot, plan.tok_pos, slot_lens, q, plan.tok_slot, table, plan.tok_lens,
                        out=out, ws=ws)

    recorded = None
    if graph:
        torch.cuda.synchronize()
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            run()
    held = np.zeros(slots, np.int64)
    for seq, new in steps:
        seq, new = np.array(seq), np.array(new)
        old = np.array([held[s] if 0 <= s < slots else 0 for s in seq])
        for dst, src in ((d_seq, seq), (d_old, old), (d_new, new)):
            dst.copy_(_dev(src))
        for x in (k, v, q):
            x.copy_(torch.from_numpy(r.standard_normal(x.shape).astype(np.float32)))
        out.fill_(7)
        recorded.replay() if graph else run()
        torch.cuda.synchronize()
        w = plan_loop(seq, old, new, *state, free, count, rows)
        state, count = (w["table"], w["slot_lens"]), w["count"]
        want = np.zeros((rows, hq, 128))
        for b, s in enumerate(seq):
            a, e = int(w["cu"][b]), int(w["cu"][b + 1])
            if e > a:
                oc.append(int(s), int(old[b]), k[a:e].float().cpu().numpy(), v[a:e].float().cpu().numpy())
                held[s] = w["lens"][b]
        for b, s in enumerate(seq):
            e = int(w["cu"][b + 1])
            if e > int(w["cu"][b]):
                want[e - 1] = O.decode(oc, q[e - 1:e].float().cpu().numpy(), [int(s)], [int(w["lens"][b])], hq)[0]
        got = out.float().cpu().numpy()
        assert (got[want.any((1, 2)) == 0] == 0).all()
        assert H.rel_err_rows(got, want).max() <= TOL
    assert cache.device_status() == 0 and plan.device_status() == okv.DEV_BAD_SLOT  # slot 9, and the slot named twice
