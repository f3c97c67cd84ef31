"""Calls on a stream of their own that make their outputs and workspaces
themselves: memory that work queued on the caller's stream still reads is not
handed to them, and an output that the caller drops is not overwritten before
the caller's stream is past it.  Results have the bits of the plain call."""
import pytest

from tests.test_gpu_int4 import _okv, _t, fill, queries
from tests.test_gpu_norm_rope import freqs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
L, HQ, HKV = 3000, 32, 8


def calls():
    """(bytes of a tensor that the call makes, the call on a stream) of every call with a `stream` argument."""
    okv = _okv()
    gc, _, lay, _ = fill(54, HQ, HKV, [L], 128)
    table = _t(lay.table)
    q, _ = queries(54, 300, HQ, HKV)
    seq, n = torch.zeros(1, dtype=torch.int32, device="cuda"), _t([L], torch.int32)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    k = q[:, :HKV].contiguous()
    f = freqs(128)
    where = n - 1
    return gc, [
        (okv.decode_workspace_bytes(gc, 1), lambda s: okv.decode_attention(gc, q[:1], seq, table, n, stream=s)),
        (okv.decode_workspace_bytes(gc, 1),
         lambda s: okv.decode_step(gc, k[:1], k[:1], seq, where, n, q[:1], seq, table, n, stream=s)),
        (HQ * 512, lambda s: okv.decode_attention_noalloc(gc, q[:1], seq, table, n, stream=s)),
        (okv.prefill_workspace_bytes(gc, 300), lambda s: okv.prefill_attention(gc, q, 0, L, table, stream=s)),
        (300 * HQ * 512, lambda s: okv.prefill_attention(gc, q, 0, L, table, stream=s)),
        (300 * HQ * 256, lambda s: okv.qk_norm_rope(q, k, pos, f, v=k, stream=s)),
        (HKV * L * 512, lambda s: okv.dequantize(gc, seq, table, n, L, 1, 1, 1, stream=s)),
    ]


def whole(x):
    return x if isinstance(x, tuple) else (x,)


def test_memory_in_use_on_the_callers_stream_is_left_alone():
    gc, made = calls()
    s = torch.cuda.Stream()
    for size, call in made:
        want = [x.clone() for x in whole(call(None))]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()   # the block freed below is the one that fits
        x = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        y = x.clone()
        x.fill_(0x11)
        del x                      # free for this stream, but read and written behind the sleep
        got = whole(call(s))
        torch.cuda.synchronize()
        assert (y == 0x5A).all()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and gc.device_status() == 0


def test_a_dropped_output_stays_until_the_callers_stream_has_read_it():
    gc, made = calls()
    s = torch.cuda.Stream()
    for _, call in made:
        want = [x.clone() for x in whole(call(None))]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        got = whole(call(s))
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(20_000_000)
        kept = [x.clone() for x in got]
        sizes = [x.numel() * x.element_size() for x in got]
        del got
        with torch.cuda.stream(s):   # takes the stream's free memory at once
            other = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)) and all((o == 0x7F).all() for o in other)


def test_a_prepared_step_on_a_stream():
    okv = _okv()
    gc, _, lay, _ = fill(55, HQ, HKV, [L], 128)
    table, n = _t(lay.table), _t([L], torch.int32)
    q, _ = queries(55, 1, HQ, HKV)
    k, seq, pos = q[:, :HKV].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"), n - 1
    want = okv.decode_step(gc, k, k, seq, pos, n, q, seq, table, n)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    x = torch.full((okv.decode_workspace_bytes(gc, 1),), 0x5A, dtype=torch.uint8, device="cuda")
    y = x.clone()
    del x
    for graph in (False, True):
        step = okv.DecodeStepCall(gc, k, k, seq, pos, n, q, seq, table, n, stream=s, graph=graph)
        for _ in range(3):
            out = step()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert (y == 0x5A).all() and gc.device_status() == 0
