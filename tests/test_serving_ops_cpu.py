"""Refusals of the serving calls that need no GPU: the plan of a step
(okv_plan_append) and the norm and rotation (okv_qk_norm_rope) check their
arguments on the host before any launch."""
import ctypes

import pytest

from int2_kv_cache_rotate_b200 import okv

torch = pytest.importorskip("torch")
FAKE = 1 << 20


def _plan(**kw):
    a = okv.PlanArgs(4, 8, 16, 32, 100)
    for n in ("seq_slot", "cached_lens", "new_lens", "free_blocks", "free_count", "block_table", "slot_lens",
              "context_lens", "cu_tokens", "tok_slot", "tok_pos", "free_count_out"):
        setattr(a, n, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(num_requests=-1), okv.ERR_INVALID_ARG), (dict(max_tokens=-1), okv.ERR_INVALID_ARG),
    (dict(num_free=-1), okv.ERR_INVALID_ARG), (dict(num_seq_slots=0), okv.ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), okv.ERR_INVALID_ARG), (dict(max_blocks_per_seq=1 << 27), okv.ERR_INVALID_ARG),
    (dict(num_seq_slots=524289), okv.ERR_UNSUPPORTED), (dict(max_tokens=1 << 30), okv.ERR_INVALID_ARG),
    (dict(num_free=1 << 30), okv.ERR_INVALID_ARG), (dict(seq_slot=None), okv.ERR_INVALID_ARG),
    (dict(cached_lens=None), okv.ERR_INVALID_ARG), (dict(new_lens=None), okv.ERR_INVALID_ARG),
    (dict(free_blocks=None), okv.ERR_INVALID_ARG), (dict(free_count=None), okv.ERR_INVALID_ARG),
    (dict(block_table=None), okv.ERR_INVALID_ARG), (dict(slot_lens=None), okv.ERR_INVALID_ARG),
    (dict(context_lens=None), okv.ERR_INVALID_ARG), (dict(cu_tokens=None), okv.ERR_INVALID_ARG),
    (dict(tok_slot=None), okv.ERR_INVALID_ARG), (dict(tok_pos=None), okv.ERR_INVALID_ARG),
    (dict(free_count_out=None), okv.ERR_INVALID_ARG), (dict(tok_pos=FAKE + 2), okv.ERR_INVALID_ARG),
    (dict(status_word=FAKE + 1), okv.ERR_INVALID_ARG),
])
def test_plan_refuses_bad_arguments(change, status):
    a = _plan(**change)
    assert okv.lib().okv_plan_append(ctypes.byref(a), FAKE, 1 << 20, None) == status
    assert okv.lib().okv_last_error_string()


def test_plan_refuses_bad_workspace_and_null():
    lib = okv.lib()
    assert lib.okv_plan_append(None, FAKE, 1 << 20, None) == okv.ERR_INVALID_ARG
    a = _plan(max_tokens=100000)  # the split form reads the workspace
    need = lib.okv_plan_workspace_bytes(4)
    assert need >= 36 and lib.okv_plan_workspace_bytes(-1) == 0
    assert lib.okv_plan_append(ctypes.byref(a), None, need, None) == okv.ERR_INVALID_ARG
    assert lib.okv_plan_append(ctypes.byref(a), FAKE + 2, need, None) == okv.ERR_INVALID_ARG
    assert lib.okv_plan_append(ctypes.byref(a), FAKE, need - 1, None) == okv.ERR_INVALID_ARG
    assert b"workspace" in lib.okv_last_error_string()


def _rope(**kw):
    a = okv.NormRopeArgs(4, 8, 2, 128, 0, 128, 0, 1, 1e-6, 1.0, FAKE, FAKE, FAKE, 1024, 128, 256, 128, 256, 128, FAKE,
                         FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=64), okv.ERR_UNSUPPORTED), (dict(num_tokens=-1), okv.ERR_INVALID_ARG),
    (dict(num_q_heads=0), okv.ERR_INVALID_ARG), (dict(num_kv_heads=0), okv.ERR_INVALID_ARG),
    (dict(rot_dim=130), okv.ERR_UNSUPPORTED), (dict(rot_dim=24), okv.ERR_UNSUPPORTED),
    (dict(rot_dim=-16), okv.ERR_UNSUPPORTED), (dict(in_type=3), okv.ERR_UNSUPPORTED),
    (dict(eps=-1.0), okv.ERR_INVALID_ARG), (dict(eps=float("nan")), okv.ERR_INVALID_ARG),
    (dict(rope_scale=0.0), okv.ERR_INVALID_ARG), (dict(v=None), okv.ERR_INVALID_ARG),
    (dict(v_out=None), okv.ERR_INVALID_ARG), (dict(q=None), okv.ERR_INVALID_ARG), (dict(k_out=None), okv.ERR_INVALID_ARG),
    (dict(positions=None), okv.ERR_INVALID_ARG), (dict(inv_freq=None), okv.ERR_INVALID_ARG),
    (dict(q=FAKE + 8), okv.ERR_INVALID_ARG), (dict(k_out=FAKE + 2), okv.ERR_INVALID_ARG),
    (dict(q_token_stride=1028), okv.ERR_INVALID_ARG), (dict(v_head_stride=132), okv.ERR_INVALID_ARG),
    (dict(k_token_stride=-256), okv.ERR_INVALID_ARG), (dict(q_weight=FAKE + 2), okv.ERR_INVALID_ARG),
])
def test_norm_rope_refuses_bad_arguments(change, status):
    a = _rope(**change)
    assert okv.lib().okv_qk_norm_rope(ctypes.byref(a), None) == status
    assert okv.lib().okv_last_error_string()


def test_norm_rope_empty_call_and_null():
    lib = okv.lib()
    assert lib.okv_qk_norm_rope(None, None) == okv.ERR_INVALID_ARG
    a = _rope(num_tokens=0, q=None, positions=None)
    assert lib.okv_qk_norm_rope(ctypes.byref(a), None) == okv.OK


def test_binding_checks_types_and_shapes_on_the_host():
    q, k = torch.zeros(2, 4, 128), torch.zeros(2, 1, 128)
    pos, freq = torch.zeros(2, dtype=torch.int32), torch.zeros(64)
    with pytest.raises(TypeError, match="bfloat16"):
        okv.qk_norm_rope(q.double(), k.double(), pos, freq)
    with pytest.raises(TypeError, match="like q"):
        okv.qk_norm_rope(q, k.half(), pos, freq)
    with pytest.raises(ValueError, match="CUDA"):
        okv.qk_norm_rope(q, k, pos, freq)
    with pytest.raises(ValueError):
        okv.AppendPlan(-1, 4, device="cpu")
    p = okv.AppendPlan(2, 4, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="seq_slot"):
        p.build(i.long(), i, i, i, i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        p.build(i, i, i, i.view(1, 2), i, i, i)


def _desc(group=128, **kw):
    d = okv.CacheDesc(32, 8, 128, group, 16, 128, 64, 4, 16, 0, 4096, 8192, 16384, 32768, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_format_bits_of_the_group():
    lib = okv.lib()
    for bits in (0, okv.OUT_BF16, okv.PAD_ROWS, okv.OUT_BF16 | okv.PAD_ROWS):
        assert [lib.okv_block_head_bytes(g | bits) for g in (128, 64, 32, 16, 0)] == [1152, 1280, 1536, 0, 0]
        assert [lib.okv_block_head_bytes(g | bits | okv.INT4) for g in (128, 64, 32, 16, 0)] == [2176, 2304, 2560, 0, 0]
    assert lib.okv_pages_bytes(10, 8, 64 | okv.INT4) == 10 * 8 * 2304
    for group in (okv.INT4, 16 | okv.INT4, 128 | 0x80000, 256 | okv.OUT_BF16, -128):
        d = _desc(group)
        assert lib.okv_append_quantize(ctypes.byref(d), FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, 0, None, None) \
            == okv.ERR_UNSUPPORTED, group
    for group in (128 | okv.INT4, 32 | okv.INT4 | okv.OUT_BF16 | okv.PAD_ROWS):
        d = _desc(group)
        assert lib.okv_append_quantize(ctypes.byref(d), None, None, 0, None, None, None, None, 0, None, None) == okv.OK
        assert lib.okv_decode_workspace_bytes(ctypes.byref(d), 4) > 0


def test_attention_refuses_misaligned_tensors():
    lib = okv.lib()
    ws = 1 << 24
    for group, odd in ((128, 2), (128 | okv.OUT_BF16, 1), (128 | okv.INT4, 2)):
        d = _desc(group)
        assert lib.okv_decode_attention(ctypes.byref(d), FAKE, 4, FAKE, FAKE, FAKE, FAKE + odd, ws, 1 << 30, None) \
            == okv.ERR_INVALID_ARG
        assert lib.okv_decode_attention_noalloc(ctypes.byref(d), FAKE, 4, FAKE, FAKE, FAKE, FAKE + odd, None) \
            == okv.ERR_INVALID_ARG
        assert lib.okv_prefill_attention(ctypes.byref(d), FAKE, 4, 0, 64, FAKE, FAKE + odd, ws, 1 << 30, None) \
            == okv.ERR_INVALID_ARG
        # the prefill's query rotation reads 16 bytes at a time
        for off in (2, 8):
            assert lib.okv_prefill_attention(ctypes.byref(d), FAKE + off, 4, 0, 64, FAKE, FAKE, ws, 1 << 30, None) \
                == okv.ERR_INVALID_ARG


def test_cache_takes_two_or_four_bits():
    with pytest.raises(ValueError, match="bits"):
        okv.Cache(4, 1, 4, 1, 4, None, None, bits=3)
