"""okv_plan_append against a plain loop over the requests: block tables, slot
maps, lengths, offsets and the free count are whole numbers and have to be
equal, in the one-launch and the two-launch form, whatever is padding, dropped
or out of room."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _okv():
    from int2_kv_cache_rotate_b200 import okv
    return okv


def plan_loop(slot, old, new, table, slot_lens, free, count, tokens):
    """The definition, request by request (numpy int64)."""
    okv = _okv()
    table, slot_lens = table.copy(), slot_lens.copy()
    count = min(max(count, 0), len(free))
    left, row, flags, open_ = count, 0, 0, True
    tok_slot, tok_pos = np.full(tokens, -1), np.full(tokens, -1)
    lens, cu = np.zeros(len(slot), np.int64), [0]
    n_slots, cols = table.shape
    names = {}
    for s in slot:
        names[int(s)] = names.get(int(s), 0) + 1
    for b, (s, o, n) in enumerate(zip(slot, old, new)):
        s, o, n = int(s), int(o), int(n)
        if s == -1:
            pass
        elif s < 0 or s >= n_slots or names[s] > 1:
            flags |= okv.DEV_BAD_SLOT
        elif o < 0 or n < 0 or o + n > cols * 16:
            flags |= okv.DEV_BAD_POS
        else:
            first, last = -(-o // 16), -(-(o + n) // 16)
            lens[b] = o
            # a request that does not fit closes the step for every later one; what it asked for
            # still counts when a later one is judged, as in a sum over all requests
            if open_ and last - first <= left and row + n <= tokens:
                for c in range(first, last):
                    left -= 1
                    table[s, c] = free[left]
                for i in range(n):
                    tok_slot[row + i], tok_pos[row + i] = s, o + i
                row += n
                lens[b] = o + n
            else:
                open_ = False
            slot_lens[s] = lens[b]
        cu.append(row)
    return dict(table=table, slot_lens=slot_lens, tok_slot=tok_slot, tok_pos=tok_pos, lens=lens,
                cu=np.array(cu), count=left, flags=flags, closed=not open_)


def _case(seed, batch, slots, cols, max_old, max_new, pool, tokens, pad=0, bad=0):
    r = np.random.default_rng(seed)
    slot = r.permutation(slots)[:batch].astype(np.int64)
    old = r.integers(0, max_old + 1, batch)
    new = r.integers(0, max_new + 1, batch)
    if batch:
        for i in r.integers(0, batch, pad):
            slot[i] = -1
    if bad and batch >= 8:
        i = r.permutation(batch)[:8]
        slot[i[0]] = slots + 3
        slot[i[1]] = -5
        slot[i[2]] = slot[i[3]]          # the same slot twice: both dropped
        old[i[4]] = -1
        new[i[5]] = -2
        old[i[6]], new[i[6]] = cols * 16, 1
        old[i[7]], new[i[7]] = 2 ** 31 - 1, 2 ** 31 - 1
    free = r.permutation(pool + 5).astype(np.int64)
    table = r.integers(0, 1 << 20, (slots, cols))
    slot_lens = r.integers(0, 99, slots)
    return slot, old, new, table, slot_lens, free, pool, tokens


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _run(case, plan=None, stream=None):
    okv = _okv()
    slot, old, new, table, slot_lens, free, count, tokens = case
    plan = plan or okv.AppendPlan(len(slot), tokens)
    t, sl = _dev(table), _dev(slot_lens)
    plan.build(_dev(slot), _dev(old), _dev(new), t, sl, _dev(free), _dev([count]), stream=stream)
    return plan, t, sl


def _check(case, plan, t, sl):
    okv = _okv()
    w = plan_loop(*case)
    for name, got, want in (("table", t, w["table"]), ("slot_lens", sl, w["slot_lens"]),
                            ("tok_slot", plan.tok_slot, w["tok_slot"]), ("tok_pos", plan.tok_pos, w["tok_pos"]),
                            ("context_lens", plan.context_lens, w["lens"]), ("cu_tokens", plan.cu_tokens, w["cu"])):
        assert np.array_equal(got.cpu().numpy(), want), name
    assert int(plan.free_count) == w["count"]
    st = plan.device_status()
    full = okv.DEV_NO_BLOCKS | okv.DEV_NO_ROWS
    assert (st & ~full) == w["flags"] and bool(st & full) == w["closed"]


@pytest.mark.parametrize("batch,slots,cols,max_old,max_new,pool,tokens,pad,bad", [
    (0, 1, 1, 0, 0, 0, 0, 0, 0),             # nothing at all
    (0, 3, 4, 0, 0, 7, 5, 0, 0),             # no request: every row is padding
    (1, 1, 1, 0, 1, 1, 1, 0, 0),
    (1, 5, 70, 900, 200, 100, 300, 0, 0),
    (7, 9, 64, 500, 1, 50, 7, 2, 0),         # a decode step with padding entries
    (33, 40, 64, 500, 40, 1000, 2000, 5, 0),
    (64, 64, 64, 0, 1000, 6000, 8192, 0, 0),  # prompts; the largest one-launch size
    (64, 64, 64, 0, 1000, 6000, 64001, 0, 0),  # the same, split over two launches
    (100, 120, 40, 600, 33, 900, 4000, 9, 1),  # bad slots, lengths and a slot named twice
    (100, 120, 40, 600, 33, 900, 9001, 9, 1),
    (200, 250, 80, 1200, 50, 90, 9000, 11, 0),  # the pool runs out
    (200, 250, 80, 1200, 50, 9000, 1003, 11, 0),  # the rows run out
    (1024, 1100, 70, 1000, 3, 3000, 4000, 20, 0),
    (1025, 1100, 70, 1000, 3, 3000, 4000, 20, 1),
    (2048, 2500, 70, 1000, 3, 3000, 8000, 20, 0),
    (2049, 2500, 70, 1000, 3, 3000, 8000, 20, 1),
    (5000, 6000, 70, 1000, 20, 9000, 60000, 99, 1),
])
def test_plan_equals_the_loop(batch, slots, cols, max_old, max_new, pool, tokens, pad, bad):
    for seed in (1, 2):
        case = _case(seed, batch, slots, cols, max_old, max_new, pool, tokens, pad, bad)
        _check(case, *_run(case))


def test_one_long_prompt_and_the_block_edges():
    # lengths on both sides of a block edge, alone and after a history that ends inside and at one
    for old in (0, 1, 15, 16, 17, 31, 32):
        for new in (0, 1, 15, 16, 17, 100000):
            case = (np.array([2]), np.array([old]), np.array([new]), np.zeros((4, 6260), np.int64),
                    np.zeros(4, np.int64), np.arange(6300)[::-1].copy(), 6270, max(1, new))
            _check(case, *_run(case))


@pytest.mark.parametrize("count", [-3, 0, 1, 999])
def test_count_outside_the_pool_is_clamped(count):
    case = (np.array([0, 1]), np.array([0, 0]), np.array([16, 16]), np.zeros((2, 4), np.int64), np.zeros(2, np.int64),
            np.arange(5), count, 64)
    _check(case, *_run(case))


@pytest.mark.parametrize("tokens", [64, 9000])
def test_a_captured_step_feeds_itself(tokens):
    """cached_lens = context_lens and free_count in place: each replay is one more step."""
    okv = _okv()
    batch, cols = 6, 40
    slot = np.array([3, 0, -1, 5, 1, 2])
    plan = okv.AppendPlan(batch, tokens)
    table, slot_lens = torch.full((7, cols), -1, dtype=torch.int32, device="cuda"), _dev(np.zeros(7))
    free = np.random.default_rng(0).permutation(400)
    d_slot, d_new, d_free = _dev(slot), _dev(np.full(batch, 7)), _dev(free)
    start = np.array([0, 5, 0, 16, 31, 100])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        plan.context_lens.copy_(_dev(start))
        plan.free_count.fill_(390)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            plan.build(d_slot, plan.context_lens, d_new, table, slot_lens, d_free, plan.free_count)
        lens, count = start.copy(), 390
        tab, sl = np.full((7, cols), -1), np.zeros(7, np.int64)
        for _ in range(5):
            g.replay()
            w = plan_loop(slot, lens, np.full(batch, 7), tab, sl, free, count, tokens)
            torch.cuda.synchronize()
            assert np.array_equal(table.cpu().numpy(), w["table"])
            assert np.array_equal(plan.context_lens.cpu().numpy(), w["lens"])
            assert np.array_equal(plan.tok_pos.cpu().numpy(), w["tok_pos"])
            assert int(plan.free_count) == w["count"]
            lens, count, tab, sl = w["lens"], w["count"], w["table"], w["slot_lens"]
    assert plan.device_status() == 0


def test_two_plans_on_two_streams():
    okv = _okv()
    cases = [_case(s, 500, 600, 70, 1000, 60, 9000, 20000, 9, 0) for s in (5, 6)]
    plans = [okv.AppendPlan(500, 20000) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [_run(c, p, s) for c, p, s in zip(cases, plans, streams)]
    torch.cuda.synchronize()
    for c, g in zip(cases, got):
        _check(c, *g)
