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
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


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


def _bad(msg: str):
    raise TQError(TQ_ERR_ARG, msg)


def _stream(stream, device) -> int:
    if stream is None:
        return _raw_stream(device.index)
    if stream.device != device:
        _bad(f"a stream of {stream.device} for tensors of {device}")
    return stream.cuda_stream


def _new(stream, q: torch.Tensor, *shape, dtype=None) -> torch.Tensor:
    """Memory like q's that the given stream (else the current one) may use at
    once: it comes from that stream's own pool."""
    if stream is None:
        return q.new_empty(*shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return q.new_empty(*shape, dtype=dtype)


def _here(name: str, device) -> None:
    if device.type != "cuda" or device.index != _current_device():
        _bad(f"{name}: tensors on {device}, which is not the current CUDA device")


def _ints(name: str, what: str, t: torch.Tensor, n: int, device) -> None:
    if t.dtype != _I32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.device != device:
        _bad(f"{name}: {what} must be contiguous int32 [{n}] on {device}")


def _cache(name: str, cache: dict, table: torch.Tensor, device):
    """The C arguments of cache and block table, and Hkv, d, B."""
    kc, ks, vc, vs = cache["kcodes"], cache["kscale"], cache["vcodes"], cache["vscale"]
    shape = kc.shape
    if len(shape) != 4 or vc.shape != shape or kc.dtype != FP8 or vc.dtype != FP8:
        _bad(f"{name}: kcodes and vcodes must be float8_e4m3fn [num_blocks, Hkv, block_size, d]")
    if ks.shape != shape[:2] or vs.shape != shape[:2] or ks.dtype != _F32 or vs.dtype != _F32:
        _bad(f"{name}: kscale and vscale must be float32 [num_blocks, Hkv]")
    for t in (kc, ks, vc, vs):
        if t.device != device or not t.is_contiguous():
            _bad(f"{name}: the cache must be contiguous, on {device}")
    if table.dim() != 2 or table.dtype != _I32 or not table.is_contiguous() or table.device != device:
        _bad(f"{name}: block_table must be contiguous int32 [B, max_blocks] on {device}")
    nb, hkv, bs, d = shape
    B, blocks = table.shape
    return (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), table.data_ptr(), blocks, bs, nb), hkv, d, B


def _rows(name: str, what: str, x: torch.Tensor, heads: int, d: int, like: torch.Tensor) -> int:
    """Row stride of x [n, heads, d], whose rows are dense."""
    n = like.shape[0]
    if x.shape != (n, heads, d) or x.dtype != like.dtype or x.device != like.device:
        _bad(f"{name}: {what} must be [{n}, {heads}, {d}] of {like.dtype} on {like.device}")
    row, head, one = x.stride()
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
    dev = k.device
    _here(name, dev)
    c, hkv, d, B = _cache(name, cache, block_table, dev)
    if k.dim() != 3 or k.dtype not in _DTYPES:
        _bad(f"{name}: k must be [n, Hkv, d] of float32, bfloat16 or float16")
    n = k.shape[0]
    ldk, ldv = _rows(name, "k", k, hkv, d, k), _rows(name, "v", v, hkv, d, k)
    _ints(name, "cu_q", cu_q, B + 1, dev)
    _ints(name, "seq_lens", seq_lens, B, dev)
    hq = ldq = ldo = qp = op = 0
    if q is not None:
        if q.dim() != 3:
            _bad(f"{name}: q must be [n, Hq, d]")
        hq = q.shape[1]
        ldq = _rows(name, "q", q, hq, d, k)
        if q_out is None:
            q_out = _new(stream, q, q.shape)
        ldo = _rows(name, "q_out", q_out, hq, d, k)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        _bad(f"{name}: q_out without q")
    rows = rot = rp = 0
    if rope is not None:
        if rope.dim() != 2 or rope.dtype != _F32 or not rope.is_contiguous() or rope.device != dev:
            _bad(f"{name}: rope must be contiguous float32 [positions, rot] on {dev}")
        rows, rot = rope.shape
        rp = rope.data_ptr()
    _check(_lib.tq_kv8_append(qp, ldq, op, ldo, k.data_ptr(), ldk, v.data_ptr(), ldv, _DTYPES[k.dtype], n, B, hq, hkv, d,
                              cu_q.data_ptr(), seq_lens.data_ptr(), rp, rows, rot, int(interleaved), *c,
                              _stream(stream, dev)))
    return q_out


def _attention(name, prefill, cache, q, block_table, cu_q, seq_lens, scale, window, out, workspace, stream):
    dev = q.device
    _here(name, dev)
    c, hkv, d, B = _cache(name, cache, block_table, dev)
    if q.dim() != 3 or q.shape[2] != d or q.dtype not in _DTYPES or not q.is_contiguous():
        _bad(f"{name}: q must be contiguous [rows, Hq, {d}] of bfloat16 or float16")
    n, hq, _ = q.shape
    _ints(name, "seq_lens", seq_lens, B, dev)
    if prefill:
        _ints(name, "cu_q", cu_q, B + 1, dev)
    elif n != B:
        _bad(f"{name}: q has {n} rows for {B} sequences")
    if out is None:
        out = _new(stream, q, q.shape)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.device != dev:
        _bad(f"{name}: out must be like q")
    if workspace is None:
        need = kv8_prefill_workspace_bytes(n, B, hq, hkv, d) if prefill else kv8_decode_workspace_bytes(B, hq, hkv, d)
        workspace = _new(stream, q, need, dtype=torch.uint8)
    elif workspace.device != dev or not workspace.is_contiguous():
        _bad(f"{name}: workspace must be contiguous, on {dev}")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    tail = (int(window), scale, out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream(stream, dev))
    if prefill:
        _check(_lib.tq_kv8_attn_prefill(q.data_ptr(), _DTYPES[q.dtype], n, B, hq, hkv, d, *c, cu_q.data_ptr(),
                                        seq_lens.data_ptr(), *tail))
    else:
        _check(_lib.tq_kv8_attn_decode(q.data_ptr(), _DTYPES[q.dtype], B, hq, hkv, d, *c, seq_lens.data_ptr(), *tail))
    return out


def kv8_decode_workspace_bytes(B: int, Hq: int, Hkv: int, d: int) -> int:
    return _lib.tq_kv8_decode_workspace_bytes(B, Hq, Hkv, d)


def kv8_prefill_workspace_bytes(n: int, B: int, Hq: int, Hkv: int, d: int) -> int:
    return _lib.tq_kv8_prefill_workspace_bytes(n, B, Hq, Hkv, d)


def kv8_attn_decode(cache: dict, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [B, Hq, d] (the newest token of each sequence) attends over its
    sequence's cached tokens, the last `window` of them if window > 0."""
    return _attention("kv8_attn_decode", False, cache, q, block_table, None, seq_lens, scale, window, out, workspace,
                      stream)


def kv8_attn_prefill(cache: dict, q: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor,
                     seq_lens: torch.Tensor, scale: float | None = None, window: int = 0,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """q [n, Hq, d], a ragged batch of rows whose keys and values have been
    appended: each attends over the tokens up to its own position, the last
    `window` of them if window > 0."""
    return _attention("kv8_attn_prefill", True, cache, q, block_table, cu_q, seq_lens, scale, window, out, workspace,
                      stream)
