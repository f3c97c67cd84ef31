"""The 4-bit calls on other streams: with workspaces they make themselves,
two at once, captured and replayed on new inputs, and two captured graphs over
one workspace replayed in turn.  Every result has the bits of the plain call."""
import pytest

from tests.test_gpu_int4 import _okv, _t, fill, queries

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

L, HQ, HKV = 3000, 32, 8


def setup(seed=51):
    gc, _, lay, _ = fill(seed, HQ, HKV, [L], 128)
    return gc, _t(lay.table)


def prefill(gc, table, q, **kw):
    return _okv().prefill_attention(gc, q, 0, L, table, out=torch.empty_like(q), **kw)


@pytest.mark.parametrize("tokens", [1, 40, 400])
def test_own_workspace_on_another_stream(tokens):
    """The call's own workspace must outlive it: a buffer of its size, taken and filled on the current stream while
    the call waits behind a long kernel, is other memory."""
    okv = _okv()
    gc, table = setup()
    q, _ = queries(51, tokens, HQ, HKV)
    want = prefill(gc, table, q)
    seq, n = torch.zeros(1, dtype=torch.int32, device="cuda"), _t([L], torch.int32)
    dwant = okv.decode_attention(gc, q[:1], seq, table, n)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for size, call, ref in ((okv.prefill_workspace_bytes(gc, tokens), lambda: prefill(gc, table, q, stream=s), want),
                            (okv.decode_workspace_bytes(gc, 1),
                             lambda: okv.decode_attention(gc, q[:1], seq, table, n, stream=s), dwant)):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        got = call()
        other = torch.full((max(size, 256),), 0x7F, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(got, ref) and (other == 0x7F).all() and gc.device_status() == 0


def test_two_calls_at_once():
    okv = _okv()
    gc, table = setup()
    qs = [queries(52 + i, n, HQ, HKV)[0] for i, n in enumerate((400, 333))]
    wants = [prefill(gc, table, q) for q in qs]
    ws = [torch.empty(okv.prefill_workspace_bytes(gc, len(q)), dtype=torch.uint8, device="cuda") for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [prefill(gc, table, q, ws=w, stream=s) for q, w, s in zip(qs, ws, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, wants)) and gc.device_status() == 0


@pytest.mark.parametrize("tokens", [(400, 400), (400, 17), (5, 300)])
def test_two_graphs_over_one_workspace(tokens):
    okv = _okv()
    gc, table = setup()
    ws = torch.empty(max(okv.prefill_workspace_bytes(gc, n) for n in tokens), dtype=torch.uint8, device="cuda")
    ins = [torch.empty(n, HQ, 128, dtype=torch.bfloat16, device="cuda") for n in tokens]
    outs = [torch.empty_like(q) for q in ins]
    graphs = []
    for q, out in zip(ins, outs):
        q.zero_()
        okv.prefill_attention(gc, q, 0, L, table, out=out, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            okv.prefill_attention(gc, q, 0, L, table, out=out, ws=ws)
        graphs.append(g)
    for seed in (61, 62):
        for q in ins:
            q.copy_(queries(seed, len(q), HQ, HKV)[0])
        for i in (0, 1, 0):
            outs[i].fill_(9)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], prefill(gc, table, ins[i])) and gc.device_status() == 0
