"""Tensors that do not lie where a call runs are refused on the host: each
argument in host memory, a workspace in host memory or not contiguous, and
tensors on another GPU than the cache (the cache's device number is changed for
that: one GPU is enough)."""
import numpy as np
import pytest

from tests import gpu_helpers as H
from tests.test_gpu_int4 import _okv, _t

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def setup():
    okv = _okv()
    lay = H.Layout(57, [40])
    uk, uv = H.rotations(57, 2)
    c = okv.Cache(8, 2, lay.num_blocks, 1, lay.mbps, uk, uv, bits=4)
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = i + 1
    return okv, c, dict(k=x, v=x, q=q, i=i, n=n, table=_t(lay.table), out=torch.zeros(1, 8, 128, device="cuda"),
                        ws=okv.workspace(c, 1), rot=torch.zeros(1, 2, 2, 128, device="cuda"),
                        pws=torch.empty(okv.prefill_workspace_bytes(c, 1), dtype=torch.uint8, device="cuda"))


# each call, and the arguments that one test after another replaces
CALLS = {
    "append": (lambda o, c, a: o.append_quantize(c, a["k"], a["v"], a["i"], a["i"], a["table"], a["n"]),
               ["k", "v", "i", "n", "table"]),
    "append, rotated": (lambda o, c, a: o.append_quantize(c, a["k"], a["v"], a["i"], a["i"], a["table"], a["n"],
                                                          rotated_out=a["rot"]), ["rot"]),
    "decode": (lambda o, c, a: o.decode_attention(c, a["q"], a["i"], a["table"], a["n"], out=a["out"], ws=a["ws"]),
               ["q", "i", "table", "n", "out", "ws"]),
    "noalloc": (lambda o, c, a: o.decode_attention_noalloc(c, a["q"], a["i"], a["table"], a["n"], out=a["out"]),
                ["q", "i", "table", "n", "out"]),
    "step": (lambda o, c, a: o.decode_step(c, a["k"], a["v"], a["i"], a["i"], a["n"], a["q"], a["i"], a["table"], a["n"],
                                           out=a["out"], ws=a["ws"]), ["k", "v", "i", "n", "q", "table", "out", "ws"]),
    "prepared step": (lambda o, c, a: o.DecodeStepCall(c, a["k"], a["v"], a["i"], a["i"], a["n"], a["q"], a["i"],
                                                       a["table"], a["n"], out=a["out"], ws=a["ws"])(),
                      ["k", "v", "i", "n", "q", "table", "out", "ws"]),
    "prefill": (lambda o, c, a: o.prefill_attention(c, a["q"], 0, 1, a["table"], out=a["out"], ws=a["pws"]),
                ["q", "table", "out", "pws"]),
    "gather": (lambda o, c, a: o.dequantize(c, a["i"], a["table"], a["n"], 1, 0, out=a["out"]),
               ["i", "table", "n", "out"]),
}


@pytest.mark.parametrize("name", CALLS)
def test_arguments_off_the_device_are_refused(name):
    okv, c, a = setup()
    call, args = CALLS[name]
    call(okv, c, a)                                        # as it should be
    for x in args:
        with pytest.raises(ValueError):
            call(okv, c, {**a, x: a[x].cpu()})
        if x in ("ws", "pws"):
            with pytest.raises(ValueError, match="contiguous"):
                call(okv, c, {**a, x: a[x][:1].expand(a[x].numel())})
            with pytest.raises(okv.OkvError, match="workspace too small"):
                call(okv, c, {**a, x: a[x][:-256]})
            call(okv, c, {**a, x: torch.empty(a[x].numel() // 4, dtype=torch.float32, device="cuda")})  # bytes count
    c.dev = 1
    with pytest.raises(ValueError, match="device"):
        call(okv, c, a)
    c.dev = 0
    call(okv, c, a)
    torch.cuda.synchronize()
    assert c.device_status() == 0
