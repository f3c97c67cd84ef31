"""The serving calls together, as a server uses them: prompts planned on the
GPU, normed, rotated, appended and attended in chunks, then decode steps of a
padded batch (plan, norm and rotation, append and attention) captured once in a
CUDA graph and replayed with lengths that feed themselves.  Every step's
attention is checked against the fp64 oracle on the queries, keys and values
that the norm and rotation produced, those against their formula, and the plan
against the loop over requests."""
import numpy as np
import pytest

from oracle import okv_oracle as O
from tests import gpu_helpers as H
from tests.test_gpu_norm_rope import close, formula, freqs
from tests.test_gpu_plan import plan_loop

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _d(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("bits", [4, 2])
@pytest.mark.parametrize("group,sinks", [(128, 0), (64, 16), (32, 0)])
def test_prompts_then_captured_decode_steps(bits, group, sinks):
    from int2_kv_cache_rotate_b200 import okv
    hq, hkv, slots, cols, blocks = 8, 2, 6, 24, 60
    tol = 2e-3 + 2.0 ** -8   # the attention's bar, and the bf16 output's half step
    g = torch.Generator(device="cuda").manual_seed(5)
    uk, uv = H.rotations(50, hkv)
    cache = okv.Cache(hq, hkv, blocks, slots, cols, uk, uv, num_sink=sinks, group=group, bits=bits, pad_rows=True)
    oc = O.Cache(hkv, uk.astype(np.float64), uv.astype(np.float64), sinks=sinks, group=group, bits=bits)
    f = freqs(128)
    wq, wk = (1 + 0.2 * torch.randn(128, generator=g, device="cuda") for _ in range(2))
    free = np.random.default_rng(1).permutation(blocks)
    table, slot_lens = torch.full((slots, cols), -1, dtype=torch.int32, device="cuda"), _d(np.zeros(slots))
    state = dict(table=table.cpu().numpy(), slot_lens=np.zeros(slots, np.int64))

    def project(n):
        return (torch.randn(n, (hq + 2 * hkv) * 128, generator=g, device="cuda") * 1.3).bfloat16()

    def split(x):
        n = x.shape[0]
        return (x[:, :hq * 128].view(n, hq, 128), x[:, hq * 128:(hq + hkv) * 128].view(n, hkv, 128),
                x[:, (hq + hkv) * 128:].view(n, hkv, 128))

    def check_rope(x, pos, got):
        q, k, v = split(x)
        close(got[0], *formula(q, wq, pos, f, 1e-6, False, True, 1.0))
        close(got[1], *formula(k, wk, pos, f, 1e-6, False, True, 1.0))
        assert torch.equal(got[2], v)

    def attend_ok(got, want):
        assert H.rel_err_rows(got.float().cpu().numpy(), want).max() <= tol

    # ---- prompts: one plan, one norm and rotation, one append for all of them, chunked attention per sequence
    seq, new = np.array([4, 1, 3]), np.array([37, 200, 129])
    rows = 384                                       # room for more tokens than come: padding rows at the end
    plan = okv.AppendPlan(3, rows).build(_d(seq), _d(np.zeros(3)), _d(new), table, slot_lens, _d(free), _d([blocks]))
    x = project(rows)
    q, k, v = okv.qk_norm_rope(*split(x)[:2], plan.tok_pos, f, wq, wk, v=split(x)[2])
    okv.append_quantize(cache, k, v, plan.tok_slot, plan.tok_pos, table, slot_lens)
    torch.cuda.synchronize()
    assert cache.device_status() == 0 and plan.device_status() == 0
    w = plan_loop(seq, np.zeros(3), new, state["table"], state["slot_lens"], free, blocks, rows)
    assert np.array_equal(table.cpu().numpy(), w["table"]) and np.array_equal(plan.cu_tokens.cpu().numpy(), w["cu"])
    n = int(w["cu"][-1])
    check_rope(x[:n], plan.tok_pos[:n], (q[:n], k[:n], v[:n]))
    for b, s in enumerate(seq):
        a, e = w["cu"][b], w["cu"][b + 1]
        oc.append(int(s), 0, k[a:e].float().cpu().numpy(), v[a:e].float().cpu().numpy())
    for b, s in enumerate(seq):
        a, e = int(w["cu"][b]), int(w["cu"][b + 1])
        out = torch.empty(e - a, hq, 128, dtype=torch.bfloat16, device="cuda")
        okv.prefill_attention(cache, q[a:e].contiguous(), int(s), e - a, table, out=out)
        attend_ok(out, O.prefill(oc, q[a:e].float().cpu().numpy(), int(s), e - a, hq))

    # ---- decode: a batch of five entries, two of them padding, captured once
    B = 5
    dseq = np.array([1, 4, 3, -1, -1])
    step = okv.AppendPlan(B, B)
    d_seq, d_new, d_free = _d(dseq), _d(np.ones(B)), _d(free)
    step.context_lens.copy_(_d([200, 37, 129, 0, 0]))
    step.free_count.copy_(plan.free_count)
    x = project(B)
    q, k, v = (torch.zeros(B, h, 128, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    out = torch.zeros(B, hq, 128, dtype=torch.bfloat16, device="cuda")
    ws = okv.workspace(cache, B)

    def run():
        step.build(d_seq, step.context_lens, d_new, table, slot_lens, d_free, step.free_count)
        okv.qk_norm_rope(*split(x)[:2], step.tok_pos, f, wq, wk, v=split(x)[2], q_out=q, k_out=k, v_out=v)
        okv.decode_step(cache, k, v, step.tok_slot, step.tok_pos, slot_lens, q, d_seq, table, step.context_lens, out=out,
                        ws=ws)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    lens = np.array([200, 37, 129, 0, 0])
    count = w["count"]
    for i in range(20):                               # past two block edges of every sequence
        x.copy_(project(B))
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            graph.replay()
        torch.cuda.synchronize()
        p = plan_loop(dseq, lens, np.ones(B), w["table"], w["slot_lens"], free, count, B)
        assert np.array_equal(table.cpu().numpy(), p["table"]) and int(step.free_count) == p["count"]
        assert np.array_equal(step.context_lens.cpu().numpy(), p["lens"])
        w, lens, count = p, p["lens"], p["count"]
        check_rope(x[:3], step.tok_pos[:3], (q[:3], k[:3], v[:3]))
        for b in range(3):
            oc.append(int(dseq[b]), int(lens[b]) - 1, k[b:b + 1].float().cpu().numpy(), v[b:b + 1].float().cpu().numpy())
        if i in (0, 1, 9, 19):
            attend_ok(out[:3], O.decode(oc, q[:3].float().cpu().numpy(), dseq[:3], lens[:3].tolist(), hq))
        assert (out[3:] == 0).all()
    assert cache.device_status() == 0 and step.device_status() == 0
