"""8-bit paged KV cache: append with position rotation, decode attention and
prompt attention (tq_kv8_* in include/tq.h, which has the formulas).

A cache is a dict of tensors: kcodes, vcodes [num_blocks, Hkv, block_size, d]
(float8_e4m3fn) and kscale, vscale [num_blocks, Hkv] (float32); kv8_empty makes
one.  block_table is int32 [B, max_blocks], seq_lens int32 [B] (lengths
including the call's own rows), cu_q int32 [B + 1] (rows cu_q[b] .. cu_q[b + 1]
- 1 of a ragged batch are the last tokens of sequence b).

Calls run on the given stream, else on the current one, of the current
device, where every tensor must live.  Like all of libtq they only enqueue
kernels; outputs and a workspace that are not given are allocated by torch for
the call, on its stream.
"""
from __future__ import annotations

import math

import torch

from . import _DTYPES, TQ_ERR_ARG, TQError, _check, _lib

FP8 = torch.float8_e4m3fn
_I32, _F32 = torch.int32, torch.float32
# A torch built without CUDA has neither; it has no tensor that gets as far as these.
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_append, _decode, _prefill = _lib.tq_kv8_append, _lib.tq_kv8_attn_decode, _lib.tq_kv8_attn_prefill
_decode_ws, _prefill_ws = _lib.tq_kv8_decode_workspace_bytes, _lib.tq_kv8_prefill_workspace_bytes


def rope_table(max_pos: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos | sin of position * base^(-2 i / rot), i < rot / 2: float32
    [max_pos, rot], from angles in 64 bits."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * base ** (-i / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def kv8_empty(num_blocks: int, Hkv: int, block_size: int, d: int, device="cuda") -> dict:
    """A cache of zeros."""
    shape = (num_blocks, Hkv, block_size, d)
    return {"kcodes": torch.zeros(shape, dtype=FP8, device=device),
            "kscale": torch.zeros(shape[:2], dtype=torch.float32, device=device),
            "vcodes": torch.zeros(shape, dtype=FP8, device=device),
            "vscale": torch.zeros(shape[:2], dtype=torch.float32, device=device)}


# The checks below run on every call, where a few microseconds count: they
# compare device numbers and dtype objects, and say more only when refusing.
def _bad(msg: str):
    raise TQError(TQ_ERR_ARG, msg)


def _stream(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device)
    if stream.device.index != device:
        _bad(f"a stream of {stream.device} for tensors of cuda:{device}")
    return stream.cuda_stream


def _like(stream, q: torch.Tensor) -> torch.Tensor:
    """An output like q that the given stream (else the current one) may use at
    once: it comes from that stream's own pool."""
    if stream is None:
        return torch.empty_like(q)
    with torch.cuda.stream(stream):
        return torch.empty_like(q)


def _scratch(stream, q: torch.Tensor, n: int) -> torch.Tensor:
    if stream is None:
        return q.new_empty(n, dtype=torch.uint8)
    with torch.cuda.stream(stream):
        return q.new_empty(n, dtype=torch.uint8)


def _device(name: str, t: torch.Tensor) -> int:
    device = t.get_device()
    if device < 0 or device != _current_device():
        _bad(f"{name}: tensors on {t.device}, which is not the current CUDA device")
    return device


def _ints(name: str, what: str, t: torch.Tensor, n: int, device: int) -> int:
    if t.dtype is not _I32 or t.shape != (n,) or t.get_device() != device or not t.is_contiguous():
        _bad(f"{name}: {what} must be contiguous int32 [{n}] on cuda:{device}")
    return t.data_ptr()


def _cache(name: str, cache: dict, table: torch.Tensor, device: int):
    """The C arguments of cache and block table, and Hkv, d, B."""
    kc, ks, vc, vs = cache["kcodes"], cache["kscale"], cache["vcodes"], cache["vscale"]
    shape = kc.shape
    if len(shape) != 4 or vc.shape != shape or kc.dtype is not FP8 or vc.dtype is not FP8:
        _bad(f"{name}: kcodes and vcodes must be float8_e4m3fn [num_blocks, Hkv, block_size, d]")
    nb, hkv, bs, d = shape
    heads = (nb, hkv)
    if ks.shape != heads or vs.shape != heads or ks.dtype is not _F32 or vs.dtype is not _F32:
        _bad(f"{name}: kscale and vscale must be float32 [num_blocks, Hkv]")
    if not (kc.get_device() == ks.get_device() == vc.get_device() == vs.get_device() == device and kc.is_contiguous()
            and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
        _bad(f"{name}: the cache must be contiguous, on cuda:{device}")
    size = table.shape
    if len(size) != 2 or table.dtype is not _I32 or table.get_device() != device or not table.is_contiguous():
        _bad(f"{name}: block_table must be contiguous int32 [B, max_blocks] on cuda:{device}")
    B, blocks = size
    return (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), table.data_ptr(), blocks, bs, nb), hkv, d, B


def _rows(name: str, what: str, x: torch.Tensor, shape: tuple, dtype, device: int) -> int:
    """Row stride of x [n, heads, d], whose rows are dense."""
    if x.shape != shape or x.dtype is not dtype or x.get_device() != device:
        _bad(f"{name}: {what} must be {list(shape)} of {dtype} on cuda:{device}")
    row, head, one = x.stride()
    n, heads, d = shape
    if n and (one != 1 or (heads > 1 and head != d)):
        _bad(f"{name}: the heads of a row of {what} must be dense")
    return row if n > 1 else heads * d


def kv8_append(cache: dict, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor,
               seq_lens: torch.Tensor, q: torch.Tensor | None = None, rope: torch.Tensor | None = None,
               interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Rotate k (and q) [n, heads, d] by their positions with the table `rope`
    [>= max_blocks * block_size, rot] and append k and v [n, Hkv, d] to the
    cache.  Rows may be strided (slices of one projection's output).  Returns
    the rotated queries: q_out, which may be q, or a new tensor."""
    name = "kv8_append"
    dev = _device(name, k)
    c, hkv, d, B = _cache(name, cache, block_table, dev)
    dtype = k.dtype
    if k.dim() != 3 or dtype not in _DTYPES:
        _bad(f"{name}: k must be [n, Hkv, d] of float32, bfloat16 or float16")
    n = k.shape[0]
    shape = (n, hkv, d)
    ldk, ldv = _rows(name, "k", k, shape, dtype, dev), _rows(name, "v", v, shape, dtype, dev)
    cu, lens = _ints(name, "cu_q", cu_q, B + 1, dev), _ints(name, "seq_lens", seq_lens, B, dev)
    hq = ldq = ldo = qp = op = 0
    if q is not None:
        if q.dim() != 3:
            _bad(f"{name}: q must be [n, Hq, d]")
        hq = q.shape[1]
        shape = (n, hq, d)
        ldq = _rows(name, "q", q, shape, dtype, dev)
        if q_out is None:
            q_out = _like(stream, q)
        ldo = _rows(name, "q_out", q_out, shape, dtype, dev)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        _bad(f"{name}: q_out without q")
    rows = rot = rp = 0
    if rope is not None:
        if rope.dim() != 2 or rope.dtype is not _F32 or rope.get_device() != dev or not rope.is_contiguous():
            _bad(f"{name}: rope must be contiguous float32 [positions, rot] on cuda:{dev}")
        rows, rot = rope.shape
        rp = rope.data_ptr()
    status = _append(qp, ldq, op, ldo, k.data_ptr(), ldk, v.data_ptr(), ldv, _DTYPES[dtype], n, B, hq, hkv, d, cu, lens,
                     rp, rows, rot, interleaved, *c, _stream(stream, dev))
    if status:
        _check(status)
    return q_out


def _attention(name, prefill, cache, q, block_table, cu_q, seq_lens, scale, window, out, workspace, stream):
    dev = _device(name, q)
    c, hkv, d, B = _cache(name, cache, block_table, dev)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3 or shape[2] != d or dtype not in _DTYPES or not q.is_contiguous():
        _bad(f"{name}: q must be contiguous [rows, Hq, {d}] of bfloat16 or float16")
    n, hq, _ = shape
    lens = _ints(name, "seq_lens", seq_lens, B, dev)
    if not prefill and n != B:
        _bad(f"{name}: q has {n} rows for {B} sequences")
    if out is None:
        out = _like(stream, q)
    elif out.shape != shape or out.dtype is not dtype or out.get_device() != dev or not out.is_contiguous():
        _bad(f"{name}: out must be like q")
    if workspace is None:
        workspace = _scratch(stream, q, _prefill_ws(n, B, hq, hkv, d) if prefill else _decode_ws(B, hq, hkv, d))
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _bad(f"{name}: workspace must be contiguous, on cuda:{dev}")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if not 0 <= window < 1 << 31:   # ctypes would keep its low 32 bits
        if window < 0:
            _bad(f"{name}: window={window}")
        window = (1 << 31) - 1
    tail = (window, scale, out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream(stream, dev))
    if prefill:
        status = _prefill(q.data_ptr(), _DTYPES[dtype], n, B, hq, hkv, d, *c, _ints(name, "cu_q", cu_q, B + 1, dev), lens,
                          *tail)
    else:
        status = _decode(q.data_ptr(), _DTYPES[dtype], B, hq, hkv, d, *c, lens, *tail)
    if status:
        _check(status)
    return out


def kv8_decode_workspace_bytes(B: int, Hq: int, Hkv: int, d: int) -> int:
    return _decode_ws(B, Hq, Hkv, d)


def kv8_prefill_workspace_bytes(n: int, B: int, Hq: int, Hkv: int, d: int) -> int:
    return _prefill_ws(n, B, Hq, Hkv, d)


def kv8_set_wait_limit(tries: int) -> None:
    """Test diagnostic: attention kernels launched by this process give up
    their bounded waits after `tries` tries (0: without looking; negative: the
    full limit), and report it in tq_device_fault."""
    _check(_lib.tq_kv8_set_wait_limit(tries))


def kv8_attn_decode(cache: dict, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [B, Hq, d] (the newest token of each sequence) attends over its
    sequence's cached tokens, the last `window` of them if window > 0.  out may
    be q."""
    return _attention("kv8_attn_decode", False, cache, q, block_table, None, seq_lens, scale, window, out, workspace,
                      stream)


def kv8_attn_prefill(cache: dict, q: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor,
                     seq_lens: torch.Tensor, scale: float | None = None, window: int = 0,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """q [n, Hq, d], a ragged batch of rows whose keys and values have been
    appended: each attends over the tokens up to its own position, the last
    `window` of them if window > 0.  out may be q."""
    return _attention("kv8_attn_prefill", True, cache, q, block_table, cu_q, seq_lens, scale, window, out, workspace,
                      stream)
