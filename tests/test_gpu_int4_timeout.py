"""The timeout paths of the 4-bit kernels, in a child process that loads the
short-wait build (every bounded wait gives up after 64 cycles): the tcgen05
append, the split-K decode and both chunked-prefill kernels (exact codes with
fp32 output, fp16 tiles with bf16 output, one key range and several) raise
OKV_DEV_TIMEOUT, wind down and leave the CUDA context usable."""
import os
import subprocess
import sys

import pytest

from tests.test_gpu_timeout import ROOT, _short_wait_lib

pytestmark = pytest.mark.gpu

CHILD = r"""
import numpy as np, torch
from int2_kv_cache_rotate_b200 import okv
from int2_kv_cache_rotate_b200 import workloads as WL
torch.cuda.set_device(0)
seed, hq, hkv, L = 62, 32, 8, 4096
r = np.random.default_rng(seed)
uk = np.stack([WL.haar_orthogonal(r) for _ in range(hkv)]).astype(np.float32)
uv = np.stack([WL.haar_orthogonal(r) for _ in range(hkv)]).astype(np.float32)
table, nb = WL.block_table(seed, 0, [L], extra_tokens=16)
dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
got = []
for group in (128, 32):
    cache = okv.Cache(hq, hkv, nb, 1, table.shape[1], uk, uv, group=group, bits=4)
    def flag():
        torch.cuda.synchronize()
        s = cache.device_status()
        cache.clear_status()
        got.append(s)
    k, v = (dev(r.standard_normal((L, hkv, 128)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    zero, n = dev(np.zeros(L, np.int32)), dev(np.array([L], np.int32))
    okv.append_quantize(cache, k, v, zero, dev(np.arange(L, dtype=np.int32)), dev(table), n)
    flag()
    q = dev(r.standard_normal((256, hq, 128)).astype(np.float32)).to(torch.bfloat16)
    okv.decode_attention(cache, q[:1], zero[:1], dev(table), n)
    flag()
    okv.prefill_attention(cache, q, 0, L, dev(table))
    flag()
    for T in (256, 16):
        out = torch.empty(T, hq, 128, dtype=torch.bfloat16, device="cuda")
        okv.prefill_attention(cache, q[:T], 0, L, dev(table), out=out)
        flag()
x = torch.arange(1 << 20, device="cuda", dtype=torch.float32)
assert float(x.sum().item()) == float((1 << 20) * ((1 << 20) - 1) // 2)
print("STATUS", *got)
"""


def test_four_bit_timeouts_wind_down_cleanly():
    env = dict(os.environ, OKV_LIBRARY=_short_wait_lib(), PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    line = [ln for ln in res.stdout.splitlines() if ln.startswith("STATUS")][-1]
    from int2_kv_cache_rotate_b200 import okv
    flags = [int(x) for x in line.split()[1:]]
    assert len(flags) == 10 and all(s & okv.DEV_TIMEOUT for s in flags), flags


def test_four_bit_prefill_of_many_rows_winds_down_cleanly():
    """400 x 32 rows: the rotations' own waits run out as well."""
    child = CHILD.replace("(256, hq, 128)", "(400, hq, 128)").replace("for T in (256, 16):", "for T in (400, 300):")
    env = dict(os.environ, OKV_LIBRARY=_short_wait_lib(), PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    res = subprocess.run([sys.executable, "-c", child], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    line = [ln for ln in res.stdout.splitlines() if ln.startswith("STATUS")][-1]
    from int2_kv_cache_rotate_b200 import okv
    flags = [int(x) for x in line.split()[1:]]
    assert len(flags) == 10 and all(s & okv.DEV_TIMEOUT for s in flags), flags
