"""Thin ctypes binding over ``libokv.so`` (argument marshalling only).

Every step of the hot path runs in the library's CUDA kernels; this module
checks dtypes/devices/shapes of torch tensors, passes raw pointers and the
current CUDA stream, and turns non-OK statuses into ``OkvError``.  Nothing
here computes any part of the method.  If the library is missing the first
call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# OKV_LIBRARY names another in-tree build of the same library (the short-wait
# test build); by default the binding loads libokv.so
LIB_PATH = os.environ.get("OKV_LIBRARY") or os.path.join(_HERE, "libokv.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "okv.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_NUMERIC, ERR_IO = range(6)
DEV_BAD_BLOCK, DEV_BAD_POS, DEV_BAD_SLOT, DEV_TIMEOUT, DEV_NO_BLOCKS, DEV_NO_ROWS = 1, 2, 4, 8, 16, 32
PRE_ROTATED = 1
INT4, OUT_BF16, PAD_ROWS = 0x10000, 0x20000, 0x40000  # format bits of CacheDesc.group
HEAD_DIM, BLOCK_TOKENS, WINDOW, BLOCK_HEAD_BYTES = 128, 16, 128, 1152


class OkvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status}: {msg}")
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("block_tokens", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("num_seq_slots", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("num_sink", ctypes.c_int32),
        ("pages", ctypes.c_void_p),
        ("window_ring", ctypes.c_void_p),
        ("u_k", ctypes.c_void_p),
        ("u_v", ctypes.c_void_p),
        ("status_word", ctypes.c_void_p),
        ("sink_rows", ctypes.c_void_p),
        ("r_image", ctypes.c_void_p),
    ]


class PlanArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_requests", "max_tokens", "num_seq_slots", "max_blocks_per_seq",
                                              "num_free")] + \
               [(n, ctypes.c_void_p) for n in ("seq_slot", "cached_lens", "new_lens", "free_blocks", "free_count",
                                               "block_table", "slot_lens", "context_lens", "cu_tokens", "tok_slot",
                                               "tok_pos", "free_count_out", "status_word", "tok_lens")]


class NormRopeArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_q_heads", "num_kv_heads", "head_dim", "in_type",
                                              "rot_dim", "interleaved", "norm")] + \
               [("eps", ctypes.c_float), ("rope_scale", ctypes.c_float)] + \
               [(n, ctypes.c_void_p) for n in ("q", "k", "v")] + \
               [(n, ctypes.c_int64) for n in ("q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride",
                                              "v_token_stride", "v_head_stride")] + \
               [(n, ctypes.c_void_p) for n in ("positions", "inv_freq", "q_weight", "k_weight", "q_out", "k_out",
                                               "v_out")]


# the same two structures as bytes, for calls that fill every field at once
_PLAN, _ROPE = struct.Struct("5i4x14P"), struct.Struct("8i2f3P6q7P")
_WEIGHT = (HEAD_DIM,)
assert _PLAN.size == ctypes.sizeof(PlanArgs) and _ROPE.size == ctypes.sizeof(NormRopeArgs)

_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_U32 = ctypes.c_uint32
_SZ = ctypes.c_size_t
_DESC = ctypes.POINTER(CacheDesc)

_SIGNATURES = {
    "okv_calibrate_rotations": (_I32, [_P, _I64, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _P, _P]),
    "okv_pages_bytes": (_SZ, [_I32, _I32, _I32]),
    "okv_block_head_bytes": (_SZ, [_I32]),
    "okv_window_bytes": (_SZ, [_I32, _I32]),
    "okv_sink_bytes": (_SZ, [_I32, _I32, _I32]),
    "okv_r_image_bytes": (_SZ, [_I32]),
    "okv_build_r_image": (_I32, [_DESC, _P]),
    "okv_append_quantize": (_I32, [_DESC, _P, _P, _I32, _P, _P, _P, _P, _U32, _P, _P]),
    "okv_decode_workspace_bytes": (_SZ, [_DESC, _I32]),
    "okv_decode_attention": (_I32, [_DESC, _P, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "okv_dequantize": (_I32, [_DESC, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P]),
    "okv_status_string": (ctypes.c_char_p, [_I32]),
    "okv_last_error_string": (ctypes.c_char_p, []),
    "okv_version": (_I32, []),
    "okv_time_next_decode_kernel": (_I32, [_P, _P]),
    "okv_decode_attention_noalloc": (_I32, [_DESC, _P, _I32, _P, _P, _P, _P, _P]),
    "okv_prefill_workspace_bytes": (_SZ, [_DESC, _I32]),
    "okv_prefill_attention": (_I32, [_DESC, _P, _I32, _I32, _I32, _P, _P, _P, _SZ, _P]),
    "okv_decode_step": (_I32, [_DESC, _P, _P, _I32, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "okv_plan_workspace_bytes": (_SZ, [_I32]),
    "okv_plan_append": (_I32, [_P, _P, _SZ, _P]),
    "okv_qk_norm_rope": (_I32, [_P, _P]),
    "okv_save_rotations": (_I32, [ctypes.c_char_p, _I32, _I32, _I32, _P, _P, ctypes.c_char_p]),
    "okv_rotations_file_shape": (_I32, [ctypes.c_char_p, _P, _P, _P, _P]),
    "okv_load_rotations": (_I32, [ctypes.c_char_p, _I32, _I32, _I32, _P, _P, _P, _SZ, _I32]),
}


def lib() -> ctypes.CDLL:
    """Load ``libokv.so`` (built in-tree); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OkvError(-1, f"{LIB_PATH} is missing: run `python -m int2_kv_cache_rotate_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def header_functions() -> list:
    """Names of the functions ``include/okv.h`` declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(okv_[a-z0-9_]+)\s*\(", text)))


def _check(status: int):
    if status != OK:
        msg = lib().okv_last_error_string().decode()
        raise OkvError(status, msg)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


_torch = None


def _t():
    """torch, imported on first use (the host-only calls do not need it)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _stream(stream) -> int:
    return (_t().cuda.current_stream() if stream is None else stream).cuda_stream


def _current_device() -> int:
    """The current GPU's number.  torch's own short cuts here and below save 3 us of a call; they are not public, so a
    torch without them takes the public functions."""
    fast = getattr(_t()._C, "_cuda_getDevice", None)
    return _torch.cuda.current_device() if fast is None else fast()


def _current_stream(dev: int) -> int:
    """The handle of GPU dev's current stream."""
    fast = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return _torch.cuda.current_stream(dev).cuda_stream if fast is None else fast(dev)


def _run(t, stream, fn, *args):
    """fn(*args, stream handle) with the device of tensor t as the current one: a launch, and the default current
    stream, belong to the current device."""
    dev = t.get_device()
    if dev == _current_device():
        status = fn(*args, _current_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with _torch.cuda.device(dev):
            status = fn(*args, _stream(stream))
    if status != OK:
        _check(status)


def _need(t, dtype, name, dev=None):
    """t: a contiguous tensor of that type on GPU `dev` (any GPU when None)."""
    if t is not None and t.dtype is dtype and t.is_contiguous():
        on = t.get_device()
        if on >= 0 and (on == dev or dev is None):
            return t
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on the device of the call's other tensors, got {t.device}")


def _device(cache, t, name):
    """The GPU of a call: that of its first tensor t, which the cache has to be on too."""
    if t is None:
        raise ValueError(f"{name} is required")
    dev = t.get_device()
    if dev >= 0 and cache is not None and dev != cache.dev:
        raise ValueError(f"{name} must be on the cache's device, got {t.device}")
    return dev


def _ws(ws, dev):
    """Address and bytes of a workspace that the caller gives."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on the device of the call's other tensors, got {ws.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _heads(t, dtype, name, heads, dev):
    """t: contiguous [rows][heads][128] on GPU dev, in any dimensions behind the first; returns its rows."""
    return _rows(_need(t, dtype, name, dev), name, heads)


def _rows(t, name, heads):
    """The rows of a tensor that _need has passed."""
    n = t.numel()
    rows = n // (heads * HEAD_DIM)
    if n == 0 or (t.shape and t.shape[0] == rows and n == rows * heads * HEAD_DIM):
        return rows
    raise ValueError(f"{name} must be [rows][{heads}][{HEAD_DIM}], got {tuple(t.shape)}")


def _ints(t, name, least, dev):
    """t: contiguous int32 on GPU dev with `least` values or more."""
    if t is not None and t.dtype is _torch.int32 and t.get_device() == dev and t.is_contiguous() and t.numel() >= least:
        return t.data_ptr()
    _need(t, _t().int32, name, dev)
    raise ValueError(f"{name} must hold at least {least} values, got {t.numel()}")


def _new(shape, dtype, device, stream):
    """A tensor that a call makes for itself and writes on `stream`: from that stream's pool, so that nothing queued on
    another stream still uses its memory, and kept from reuse until the caller's current stream is past it."""
    torch = _t()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _scratch(nbytes, device, stream):
    """A workspace that a call makes for itself."""
    return _new(max(nbytes, 256), _t().uint8, device, stream)


def _for_slots(cache, desc, block_table, slot_lens=None):
    """desc, or where the block table or slot_lens have fewer rows than the cache has sequence slots, a copy with as
    many slots as they have: the kernels then skip and flag a slot beyond them like one beyond the cache's."""
    slots = block_table.numel() // cache.max_blocks_per_seq
    if slot_lens is not None:
        slots = min(slots, slot_lens.numel())
    if slots >= cache.num_seq_slots:
        return desc
    d = CacheDesc.from_buffer_copy(desc)
    d.num_seq_slots = slots
    return d


def _out(cache, out, rows, device, stream):
    """The output of `rows` query rows (a new fp32 tensor when None) and the descriptor that writes its type."""
    if out is None:
        return _new((rows, cache.hq, HEAD_DIM), _torch.float32, device, stream), cache.desc
    desc = _desc_for(cache, out, device.index)
    if out.numel() < rows * cache.hq * HEAD_DIM:
        raise ValueError(f"out must hold [{rows}][{cache.hq}][{HEAD_DIM}] values, got {tuple(out.shape)}")
    return out, desc


# ---------------------------------------------------------------- calibration

def calibrate_rotations(q: np.ndarray, k: np.ndarray, v: np.ndarray, hq: int, hkv: int) -> dict:
    """Host fp64 calibration.  q [nq, hq, 128], k/v [nk, hkv, 128] (float32)."""
    q = np.ascontiguousarray(q, dtype=np.float32)
    k = np.ascontiguousarray(k, dtype=np.float32)
    v = np.ascontiguousarray(v, dtype=np.float32)
    out = {n: np.zeros((hkv, HEAD_DIM, HEAD_DIM), np.float32) for n in ("R_K", "R_V", "U_K", "U_V")}
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(lib().okv_calibrate_rotations(p(q), q.shape[0], p(k), p(v), k.shape[0], hq, hkv, q.shape[-1],
                                         p(out["R_K"]), p(out["R_V"]), p(out["U_K"]), p(out["U_V"])))
    return out


# ---------------------------------------------------------------------- cache

class Cache:
    """Device buffers of one layer's quantised cache plus its C descriptor.

    bits: 2 (INT2 codes, the default) or 4 (INT4).  pad_rows: appended rows
    whose sequence slot is -1 are padding (else they raise DEV_BAD_SLOT).
    Memory comes from torch (the caller's allocator); the library only
    receives pointers."""

    def __init__(self, hq: int, hkv: int, num_blocks: int, num_seq_slots: int, max_blocks_per_seq: int,
                 u_k, u_v, device="cuda", num_sink: int = 0, group: int = HEAD_DIM, stage_r: bool = True,
                 bits: int = 2, pad_rows: bool = False):
        import torch
        if bits not in (2, 4):
            raise ValueError(f"bits must be 2 or 4, got {bits}")
        self.hq, self.hkv, self.num_sink, self.group, self.bits = hq, hkv, num_sink, group, bits
        if bits == 4:
            group |= INT4
        self.num_blocks, self.num_seq_slots, self.max_blocks_per_seq = num_blocks, num_seq_slots, max_blocks_per_seq
        self.block_head_bytes = int(lib().okv_block_head_bytes(group))
        nbytes = lib().okv_pages_bytes(num_blocks, hkv, group)
        self.pages = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=device)
        self.ring = torch.zeros((num_seq_slots, hkv, 2, WINDOW, HEAD_DIM), dtype=torch.float16, device=device)
        self.u_k = torch.as_tensor(np.asarray(u_k, dtype=np.float32)).to(device).contiguous()
        self.u_v = torch.as_tensor(np.asarray(u_v, dtype=np.float32)).to(device).contiguous()
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self.dev = self.pages.get_device()
        # first num_sink positions of every sequence, fp16 (sink tokens)
        self.sink = torch.zeros((num_seq_slots, hkv, 2, max(num_sink, 0), HEAD_DIM), dtype=torch.float16,
                                device=device)
        # the prefill append's staged R of every (KV head, K|V), built once from U
        self.r_image = torch.empty(max(int(lib().okv_r_image_bytes(hkv)), 16), dtype=torch.uint8, device=device) \
            if stage_r else None
        self.desc = CacheDesc(hq, hkv, HEAD_DIM, group | (PAD_ROWS if pad_rows else 0), BLOCK_TOKENS, WINDOW, num_blocks, num_seq_slots,
                              max_blocks_per_seq, num_sink, self.pages.data_ptr(), self.ring.data_ptr(),
                              self.u_k.data_ptr(), self.u_v.data_ptr(), self.status.data_ptr(),
                              self.sink.data_ptr() if num_sink > 0 else None,
                              self.r_image.data_ptr() if stage_r else None)
        if stage_r:
            self.rebuild_r_image()

    def rebuild_r_image(self, stream=None):
        """Stage R from u_k, u_v into the image buffer again (after changing them)."""
        _run(self.pages, stream, lib().okv_build_r_image, ctypes.byref(self.desc))

    def device_status(self) -> int:
        return int(self.status[0].item())

    def clear_status(self):
        self.status.zero_()


def _desc_for(cache: Cache, out, dev):
    """The cache's descriptor for a call that writes `out`: fp32, or bf16 (the OUT_BF16 format bit)."""
    torch = _t()
    if out.dtype is not torch.bfloat16:
        _need(out, torch.float32, "out", dev)
        return cache.desc
    _need(out, torch.bfloat16, "out", dev)
    d = CacheDesc.from_buffer_copy(cache.desc)
    d.group |= OUT_BF16
    return d


def save_rotations(path, u_k, u_v, tag: str = "") -> None:
    """Write U_K and U_V (host fp32 [layers][Hkv][128][128], or [Hkv][128][128]
    for one layer) to a rotations file."""
    uk = np.ascontiguousarray(u_k, dtype=np.float32)
    uv = np.ascontiguousarray(u_v, dtype=np.float32)
    if uk.ndim == 3:
        uk, uv = uk[None], uv[None]
    if uk.ndim != 4 or uv.shape != uk.shape or uk.shape[2] != uk.shape[3]:
        raise ValueError(f"u_k {uk.shape} and u_v {uv.shape} must both be [layers][Hkv][d][d]")
    layers, hkv, d, _ = uk.shape
    _check(lib().okv_save_rotations(os.fsencode(path), layers, hkv, d, uk.ctypes.data, uv.ctypes.data,
                                    tag.encode("utf-8")))


def load_rotations(path, verify: bool = True) -> dict:
    """Read a rotations file: {"U_K", "U_V": fp32 [layers][Hkv][d][d], "tag": str}."""
    p = os.fsencode(path)
    layers, hkv, d, tag_len = (ctypes.c_int32() for _ in range(4))
    _check(lib().okv_rotations_file_shape(p, ctypes.byref(layers), ctypes.byref(hkv), ctypes.byref(d),
                                          ctypes.byref(tag_len)))
    shape = (layers.value, hkv.value, d.value, d.value)
    uk, uv = np.empty(shape, np.float32), np.empty(shape, np.float32)
    tag = ctypes.create_string_buffer(tag_len.value + 1)
    _check(lib().okv_load_rotations(p, layers.value, hkv.value, d.value, uk.ctypes.data, uv.ctypes.data, tag,
                                    tag_len.value + 1, int(verify)))
    return {"U_K": uk, "U_V": uv, "tag": tag.value.decode("utf-8")}


def append_quantize(cache: Cache, k, v, seq_slot, pos, block_table, slot_lens, pre_rotated=False,
                    rotated_out=None, stream=None):
    torch = _t()
    dt = torch.float32 if pre_rotated else torch.bfloat16
    dev = _device(cache, k, "k")
    T = _heads(k, dt, "k", cache.hkv, dev)
    if _heads(v, dt, "v", cache.hkv, dev) != T:
        raise ValueError("k and v must have the same number of rows")
    if rotated_out is not None:
        _need(rotated_out, torch.float32, "rotated_out", dev)
        if rotated_out.numel() < 2 * k.numel():
            raise ValueError("rotated_out must hold [T][2][Hkv][128] values")
    args = (k.data_ptr(), v.data_ptr(), T, _ints(seq_slot, "seq_slot", T, dev), _ints(pos, "pos", T, dev),
            _ints(block_table, "block_table", cache.max_blocks_per_seq if T else 0, dev),
            _ints(slot_lens, "slot_lens", 1 if T else 0, dev), PRE_ROTATED if pre_rotated else 0, _ptr(rotated_out))
    desc = _for_slots(cache, cache.desc, block_table, slot_lens) if T else cache.desc
    _run(k, stream, lib().okv_append_quantize, ctypes.byref(desc), *args)


def decode_workspace_bytes(cache: Cache, batch: int) -> int:
    return int(lib().okv_decode_workspace_bytes(ctypes.byref(cache.desc), batch))


def workspace(cache: Cache, batch: int):
    return _t().empty(max(decode_workspace_bytes(cache, batch), 256), dtype=_torch.uint8, device=cache.pages.device)


def _least(t, name, least):
    """The address of an integer tensor that _need has passed, with `least` values or more."""
    if t.numel() < least:
        raise ValueError(f"{name} must hold at least {least} values, got {t.numel()}")
    return t.data_ptr()


def _decode_args(cache, q, seq_slot, block_table, context_lens, dev):
    """Rows of q (which _need has passed), and the pointers of a decode call's integer arrays."""
    B = _rows(q, "q", cache.hq)
    return (B, _ints(seq_slot, "seq_slot", B, dev),
            _ints(block_table, "block_table", cache.max_blocks_per_seq if B else 0, dev),
            _ints(context_lens, "context_lens", B, dev))


def decode_attention(cache: Cache, q, seq_slot, block_table, context_lens, out=None, ws=None, stream=None):
    """Decode attention of one query per sequence; out: fp32 (a new tensor when None) or bf16 [B, Hq, 128]."""
    dev = _device(cache, q, "q")
    _need(q, _t().bfloat16, "q", dev)
    B, seq, table, ctx = _decode_args(cache, q, seq_slot, block_table, context_lens, dev)
    out, desc = _out(cache, out, B, q.device, stream)
    if B:
        desc = _for_slots(cache, desc, block_table)
    if ws is None:
        ws = _scratch(decode_workspace_bytes(cache, B), q.device, stream)
    _run(q, stream, lib().okv_decode_attention, ctypes.byref(desc), q.data_ptr(), B, seq, table, ctx, out.data_ptr(),
         *_ws(ws, dev))
    return out


def _step_args(cache, k, v, new_seq_slot, new_pos, slot_lens, q, seq_slot, block_table, context_lens, out, ws, stream):
    """Output, the library's arguments but for the stream, and what they point into."""
    bf16, dev = _t().bfloat16, _device(cache, q, "q")
    _need(k, bf16, "k", dev), _need(v, bf16, "v", dev), _need(q, bf16, "q", dev)
    for name, t in (("new_seq_slot", new_seq_slot), ("new_pos", new_pos), ("slot_lens", slot_lens)):
        _need(t, _torch.int32, name, dev)
    B, seq, table, ctx = _decode_args(cache, q, seq_slot, block_table, context_lens, dev)
    T = _rows(k, "k", cache.hkv)
    if _rows(v, "v", cache.hkv) != T:
        raise ValueError("k and v must have the same number of rows")
    if T and not B:
        _ints(block_table, "block_table", cache.max_blocks_per_seq, dev)
    out, desc = _out(cache, out, B, q.device, stream)
    if T or B:
        desc = _for_slots(cache, desc, block_table, slot_lens if T else None)
    if ws is None:
        ws = _scratch(decode_workspace_bytes(cache, B), q.device, stream)
    args = (ctypes.byref(desc), k.data_ptr(), v.data_ptr(), T, _least(new_seq_slot, "new_seq_slot", T),
            _least(new_pos, "new_pos", T), _least(slot_lens, "slot_lens", 1 if T else 0), q.data_ptr(), B, seq, table, ctx,
            out.data_ptr(), *_ws(ws, dev))
    return out, args, (desc, ws)


def decode_step(cache: Cache, k, v, new_seq_slot, new_pos, slot_lens, q, seq_slot, block_table, context_lens,
                out=None, ws=None, stream=None):
    """Append this step's bf16 tokens, then decode (one call; see okv_decode_step); out: fp32 or bf16 [B, Hq, 128]."""
    out, args, _ = _step_args(cache, k, v, new_seq_slot, new_pos, slot_lens, q, seq_slot, block_table, context_lens,
                              out, ws, stream)
    _run(q, stream, lib().okv_decode_step, *args)
    return out


class DecodeStepCall:
    """okv_decode_step prepared once for fixed buffers: the arguments are
    checked and marshalled here, and each call only invokes the library, for
    serving loops that refill the same input tensors every step.  The tensors
    must stay alive, and their shapes, for as long as the object is used.

    graph=True: the first call runs eagerly and then records the step's three
    launches in a CUDA graph; later calls replay it (one launch per step)."""

    def __init__(self, cache: Cache, k, v, new_seq_slot, new_pos, slot_lens, q, seq_slot, block_table,
                 context_lens, out=None, ws=None, stream=None, graph: bool = False):
        self.out, self._args, keep = _step_args(cache, k, v, new_seq_slot, new_pos, slot_lens, q, seq_slot, block_table,
                                                context_lens, out, ws, stream)
        self._keep = (cache, k, v, new_seq_slot, new_pos, slot_lens, q, seq_slot, block_table, context_lens, keep)
        self._fn = lib().okv_decode_step
        self._stream = stream
        self._want_graph, self._graph = graph, None

    def __call__(self):
        import torch
        if self._graph is not None:
            if self._stream is None:
                self._graph.replay()  # (on the current stream of the device it was recorded on)
            else:
                with torch.cuda.stream(self._stream):
                    self._graph.replay()
            return self.out
        _run(self.out, self._stream, self._fn, *self._args)
        if self._want_graph:
            with torch.cuda.device(self.out.device):
                # record the same call (the library allocates nothing and only launches)
                cap = torch.cuda.Stream()
                cap.wait_stream(torch.cuda.current_stream() if self._stream is None else self._stream)
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=cap):
                    status = self._fn(*self._args, cap.cuda_stream)
                _check(status)
                self._graph = g
        return self.out


def decode_attention_noalloc(cache: Cache, q, seq_slot, block_table, context_lens, out=None, stream=None):
    """Decode attention with the library's static scratch (no workspace, no allocation in the library)."""
    dev = _device(cache, q, "q")
    _need(q, _t().bfloat16, "q", dev)
    B, seq, table, ctx = _decode_args(cache, q, seq_slot, block_table, context_lens, dev)
    out, desc = _out(cache, out, B, q.device, stream)
    if B:
        desc = _for_slots(cache, desc, block_table)
    _run(q, stream, lib().okv_decode_attention_noalloc, ctypes.byref(desc), q.data_ptr(), B, seq, table, ctx,
         out.data_ptr())
    return out


def prefill_workspace_bytes(cache: Cache, T: int) -> int:
    return int(lib().okv_prefill_workspace_bytes(ctypes.byref(cache.desc), T))


def prefill_attention(cache: Cache, q, slot: int, context_len: int, block_table, out=None, ws=None, stream=None):
    """Causal attention of a prefill chunk (q: bf16 [T, Hq, 128], already appended at positions
    context_len - T .. context_len - 1 of sequence `slot`) over the cache; returns [T, Hq, 128] in fp32 (a new tensor
    when out is None) or in out's type, fp32 or bf16."""
    dev = _device(cache, q, "q")
    T = _heads(q, _t().bfloat16, "q", cache.hq, dev)
    table = _ints(block_table, "block_table", cache.max_blocks_per_seq if T else 0, dev)
    out, desc = _out(cache, out, T, q.device, stream)
    if T:
        desc = _for_slots(cache, desc, block_table)
    if ws is None:
        ws = _scratch(prefill_workspace_bytes(cache, T), q.device, stream)
    _run(q, stream, lib().okv_prefill_attention, ctypes.byref(desc), q.data_ptr(), T, int(slot), int(context_len),
         table, out.data_ptr(), *_ws(ws, dev))
    return out


class AppendPlan:
    """Block tables and slot maps of serving steps of up to `batch` requests and
    `max_tokens` new tokens, built on the GPU (okv_plan_append).  Holds the
    outputs that the step's other calls take:

      tok_slot, tok_pos  int32 [max_tokens]: sequence slot and position of every new token, -1 behind the last
      tok_lens           int32 [max_tokens]: tokens of the request after the step in the row of its last new token,
                         0 in every other row: with tok_slot, what a decode call over the token rows takes
      context_lens       int32 [batch]: tokens of every request after the step
      cu_tokens          int32 [batch + 1]: first token row of every request
      free_count         int32 [1]: blocks left in the pool

    The buffers stay the same from call to call, so a step can be captured in a
    CUDA graph.  They are one set per plan, workspace included: builds of one
    plan, captured ones among them, have to follow one another.  Steps that are
    built at the same time, on two streams, take a plan each (two plans share
    nothing)."""

    def __init__(self, batch: int, max_tokens: int, device="cuda"):
        import torch
        if batch < 0 or max_tokens < 0:
            raise ValueError("batch and max_tokens must be >= 0")
        self.batch, self.max_tokens = batch, max_tokens
        i32 = dict(dtype=torch.int32, device=device)
        self.tok_slot = torch.full((max_tokens,), -1, **i32)
        self.tok_pos = torch.full((max_tokens,), -1, **i32)
        self.tok_lens = torch.zeros(max_tokens, **i32)
        self.context_lens = torch.zeros(batch, **i32)
        self.cu_tokens = torch.zeros(batch + 1, **i32)
        self.free_count = torch.zeros(1, **i32)
        self.status = torch.zeros(4, **i32)
        self.ws = torch.empty(int(lib().okv_plan_workspace_bytes(batch)), dtype=torch.uint8, device=device)
        self._fn, self._dev = lib().okv_plan_append, self.tok_slot.get_device()
        self._outs = tuple(t.data_ptr() for t in (self.context_lens, self.cu_tokens, self.tok_slot, self.tok_pos,
                                                  self.free_count, self.status, self.tok_lens))
        self._ws = (self.ws.data_ptr(), self.ws.numel())

    def build(self, seq_slot, cached_lens, new_lens, block_table, slot_lens, free_blocks, free_count, stream=None):
        """Plan one step: request b (sequence slot seq_slot[b], -1 for padding) holds cached_lens[b] tokens and
        gains new_lens[b].  Updates block_table [slots][columns] and slot_lens [slots]; takes blocks from the end
        of free_blocks[:free_count].  cached_lens may be this plan's context_lens and free_count its free_count
        (a step that feeds the next).  Returns self."""
        i32, dev = _t().int32, self._dev
        for name, t in (("seq_slot", seq_slot), ("cached_lens", cached_lens), ("new_lens", new_lens),
                        ("block_table", block_table), ("slot_lens", slot_lens), ("free_blocks", free_blocks),
                        ("free_count", free_count)):
            if t.dtype is not i32 or not t.is_contiguous() or t.get_device() != dev or dev < 0:
                _need(t, i32, name)
                raise ValueError(f"{name} must be on {self.tok_slot.device}")
        n = self.batch
        for name, t in (("seq_slot", seq_slot), ("cached_lens", cached_lens), ("new_lens", new_lens)):
            if t.dim() != 1 or t.shape[0] != n:
                raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
        if block_table.dim() != 2 or slot_lens.dim() != 1 or slot_lens.shape[0] != block_table.shape[0]:
            raise ValueError("block_table must be [slots][columns] and slot_lens [slots]")
        if free_blocks.dim() != 1 or free_count.numel() != 1:
            raise ValueError("free_blocks must be one-dimensional and free_count hold one value")
        a = _PLAN.pack(n, self.max_tokens, *block_table.shape, free_blocks.shape[0], seq_slot.data_ptr(),
                       cached_lens.data_ptr(), new_lens.data_ptr(), free_blocks.data_ptr(), free_count.data_ptr(),
                       block_table.data_ptr(), slot_lens.data_ptr(), *self._outs)
        _run(self.tok_slot, stream, self._fn, a, *self._ws)
        return self

    def device_status(self) -> int:
        return int(self.status[0].item())

    def clear_status(self):
        self.status.zero_()


def _rope_refuse(q, k, v, positions, inv_freq, weights, outs):
    """The error of a qk_norm_rope call whose tensors do not fit, found one by one."""
    torch = _t()
    dt, dev = q.dtype, q.get_device()
    if dt not in (torch.bfloat16, torch.float16, torch.float32):
        raise TypeError(f"q must be bfloat16, float16 or float32, got {dt}")
    given = [(n, t) for n, t in (("q", q), ("k", k), ("v", v)) if t is not None]
    for name, t in given:
        if t.dtype is not dt:
            raise TypeError(f"{name} must be {dt} like q, got {t.dtype}")
    for name, t in given:
        if dev < 0 or t.get_device() != dev:
            raise ValueError(f"{name} must be a CUDA tensor on one device with q")
        if t.dim() != 3 or t.shape[2] != HEAD_DIM or t.stride(2) != 1 or t.shape[0] != q.shape[0]:
            raise ValueError(f"{name} must be [T][heads][{HEAD_DIM}] with contiguous rows, got {tuple(t.shape)}")
    if v is not None and v.shape[1] != k.shape[1]:
        raise ValueError("k and v must have the same number of heads")
    for (name, t), out in zip(given, outs):
        if out is not None and (_need(out, torch.bfloat16, name + "_out").shape != t.shape or out.get_device() != dev):
            raise ValueError(f"{name}_out must have shape {tuple(t.shape)} on {q.device}")
    for name, t, dtype, n in (("positions", positions, torch.int32, q.shape[0]), ("inv_freq", inv_freq, torch.float32, -1),
                              ("q_weight", weights[0], torch.float32, HEAD_DIM),
                              ("k_weight", weights[1], torch.float32, HEAD_DIM)):
        if t is None and name.endswith("weight"):
            continue
        if _need(t, dtype, name).get_device() != dev or t.dim() != 1:
            raise ValueError(f"{name} must be one-dimensional on {q.device}")
        if n >= 0 and t.shape[0] != n:
            raise ValueError(f"{name} must have shape ({n},)")
    raise ValueError("the tensors do not fit")


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6, v=None,
                 interleaved: bool = False, norm: bool = True, rope_scale: float = 1.0, q_out=None, k_out=None,
                 v_out=None, stream=None):
    """Norms of queries and keys for each head with the position rotation (okv_qk_norm_rope): q [T][Hq][128], k and
    v [T][Hkv][128] in bf16, fp16 or fp32, views of one fused projection included (the last dimension contiguous,
    rows on 16-byte boundaries); positions int32 [T] (negative: a padding row, left as it is); inv_freq fp32
    [rot_dim/2]; weights fp32 [128].  Returns contiguous bf16 (q, k), or (q, k, v) when v is given."""
    torch = _t()
    bf16, f32, dt, dev = torch.bfloat16, torch.float32, q.dtype, q.get_device()
    kind = 0 if dt is bf16 else 1 if dt is torch.float16 else 2 if dt is f32 else -1
    fits = (kind >= 0 and dev >= 0 and k.dtype is dt and k.get_device() == dev and q.dim() == 3 and k.dim() == 3
            and positions is not None and inv_freq is not None)
    if fits:
        (tokens, hq, d), (qt, qh, q1) = q.shape, q.stride()
        (kt_, hkv, kd), (kt, kh, k1) = k.shape, k.stride()
        fits = d == HEAD_DIM and kd == HEAD_DIM and q1 == 1 and k1 == 1 and kt_ == tokens
    if fits and v is not None:
        fits = v.dtype is dt and v.get_device() == dev and v.shape == k.shape
        if fits:
            vt, vh, v1 = v.stride()
            fits = v1 == 1
    if fits:
        for t, x in ((q_out, q), (k_out, k), (v_out, v)):
            if t is not None and x is not None and not (t.dtype is bf16 and t.shape == x.shape and t.is_contiguous()
                                                        and t.get_device() == dev):
                fits = False
        fits = (fits and positions.dtype is torch.int32 and positions.shape == (tokens,) and positions.is_contiguous()
                and positions.get_device() == dev and inv_freq.dtype is f32 and inv_freq.dim() == 1
                and inv_freq.is_contiguous() and inv_freq.get_device() == dev)
        for t in (q_weight, k_weight):
            if t is not None and not (t.dtype is f32 and t.shape == _WEIGHT and t.is_contiguous() and t.get_device() == dev):
                fits = False
    if not fits:
        _rope_refuse(q, k, v, positions, inv_freq, (q_weight, k_weight), (q_out, k_out, v_out))
    if q_out is None:
        q_out = _new(q.shape, bf16, q.device, stream)
    if k_out is None:
        k_out = _new(k.shape, bf16, q.device, stream)
    if v is None:
        vp = vo = vt = vh = 0
    else:
        if v_out is None:
            v_out = _new(v.shape, bf16, q.device, stream)
        vp, vo = v.data_ptr(), v_out.data_ptr()
    if tokens == 1:  # the stride of a dimension of one is never used, whatever it says
        qt = kt = vt = 0
    if hq == 1:
        qh = 0
    if hkv == 1:
        kh = vh = 0
    a = _ROPE.pack(tokens, hq, hkv, HEAD_DIM, kind, 2 * inv_freq.shape[0], bool(interleaved), bool(norm), eps, rope_scale,
                   q.data_ptr(), k.data_ptr(), vp, qt, qh, kt, kh, vt, vh, positions.data_ptr(), inv_freq.data_ptr(),
                   0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(),
                   q_out.data_ptr(), k_out.data_ptr(), vo)
    _run(q, stream, lib().okv_qk_norm_rope, a)
    return (q_out, k_out) if v is None else (q_out, k_out, v_out)


def time_next_decode_kernel(start_event, stop_event):
    """Record two torch.cuda.Event objects around the next decode call's split-K kernel."""
    for e in (start_event, stop_event):
        if not e.cuda_event:  # torch creates the CUDA event lazily, on first record
            e.record()
    _check(lib().okv_time_next_decode_kernel(start_event.cuda_event, stop_event.cuda_event))


def dequantize(cache: Cache, seq_slot, block_table, context_lens, max_ctx: int, which: int, basis: int = 0,
               source: int = 0, out=None, stream=None):
    torch, dev = _t(), _device(cache, seq_slot, "seq_slot")
    for name, t in (("seq_slot", seq_slot), ("block_table", block_table), ("context_lens", context_lens)):
        _need(t, torch.int32, name, dev)
    batch = seq_slot.shape[0]
    if out is None:
        out = _new((batch, cache.hkv, max_ctx, HEAD_DIM), torch.float32, seq_slot.device, stream)
    desc = _desc_for(cache, out, dev)
    if out.numel() < batch * cache.hkv * max(max_ctx, 0) * HEAD_DIM:
        raise ValueError(f"out must hold [{batch}][{cache.hkv}][{max_ctx}][{HEAD_DIM}] values, got {tuple(out.shape)}")
    table = _ints(block_table, "block_table", cache.max_blocks_per_seq if batch else 0, dev)
    if batch:
        desc = _for_slots(cache, desc, block_table)
    _run(out, stream, lib().okv_dequantize, ctypes.byref(desc), batch, seq_slot.data_ptr(), table,
         _ints(context_lens, "context_lens", batch, dev), max_ctx, which, basis, source, out.data_ptr())
    return out
