"""Python binding of the paged-cache operators (``include/sv_paged.h``).

Argument marshalling only, in a small native module (``lib/_svkv.*.so``): shapes
and types are checked there, sizes and alignments by the library, and the work
is done by its CUDA kernels on the current (or given) stream.

The cache.  ``k_cache`` and ``v_cache`` [num_blocks, kv heads, block size,
head dim], bf16, fp16 or float8_e4m3fn, their last three dimensions dense and
their strides equal (they may be two halves of one buffer).  An e4m3 cache has
``k_scale`` and ``v_scale`` [num_blocks, kv heads, block size, head dim / 32]
uint8: value = code * 2^(scale - 127).  A cache of 4 bits is uint8 [..., head
dim / 2], element 2i in the low half of byte i, with scales of the same shape:
value = (code - 8) * 2^(scale // 8 - 14) * (1 + scale % 8 / 8), scale <= 215
(larger bytes are NaN).  It halves e4m3's memory.  Attention from single tokens
takes two thirds of the time over e4m3, from chains of six 1 to 1.25 times it, from
prompts 1.4 to 2.1 times and from trees of 64 2 to 3 times.  ``block_tables`` [B, max_blocks] int32
(-1 = no block) and ``seq_lens`` [B] int32 (committed tokens L) are those of
``kv_rollback``; ``new_lens`` [B] int32 or None (all T) counts the new tokens
of a request, at positions L .. L + n - 1.  ``status`` is None or a 1-element
int32/uint32 tensor that receives SV_KV_* bits (the caller zeroes it).
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
from typing import Optional, Tuple

import torch

from . import api as _api
from . import build as _build
from .api import SpecVerifyError

SV_F16 = 2
SV_E4M3 = 3
SV_I4 = 4

SV_KV_BAD_BLOCK = 0x10
SV_KV_BAD_PATH = 0x20
SV_KV_NO_BLOCKS = 0x40
SV_KV_GROUP = 32
SV_KV_I4_MAX_SCALE = 215

_native = None


def load_binding():
    """The native module, loaded once (it must have been built)."""
    global _native
    if _native is None:
        lib = _api.load_library()
        path = _build.binding_path()
        if not path.exists():
            raise RuntimeError(
                f"{path} is not built (for this Python and PyTorch): run `python -m "
                "speculative_decoding_verification_75_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_svkv", str(path))
        mod = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_svkv", loader))
        loader.exec_module(mod)
        mod.bind_library(lib._name)
        _native = mod
    return _native


def _raise(rc: int):
    raise SpecVerifyError(rc, _api.load_library())


def kv_reserve(seq_lens: torch.Tensor, new_lens: Optional[torch.Tensor],
               block_tables: torch.Tensor, block_size: int, free_list: torch.Tensor,
               free_count: torch.Tensor, tree_mask: Optional[torch.Tensor] = None, *,
               max_new: Optional[int] = None, slots: Optional[torch.Tensor] = None,
               positions: Optional[torch.Tensor] = None, reserved: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Places for a step's new tokens, through ``sv_kv_reserve``: blocks from the
    free list go into ``block_tables`` (in place, ``free_count`` goes down), the
    inverse of ``kv_rollback`` on the same tensors.

    Requests are served in order while blocks last; one that is refused is
    reported (SV_KV_NO_BLOCKS) and left as it was.  Returns (slots, positions,
    reserved): slots [B, T] int64, block * block_size + row of each new token, -1
    where there is none; positions [B, T] int32, seq_lens[b] + i, or by the depth
    of node i in ``tree_mask`` ([B, T, T] or [T, T] bool, as for
    ``tree_attention``); reserved [B] int32, the new tokens that have places
    (new_lens[b], or 0), which is the new_lens of the calls that follow,
    ``kv_rollback`` among them (its num_accepted at most that); it may be the
    tensor new_lens itself.  T is ``max_new``, or that of ``slots`` or ``tree_mask``."""
    rc, *res = (_native or load_binding()).kv_reserve(
        seq_lens, new_lens, block_tables, block_size, free_list, free_count, tree_mask, max_new,
        slots, positions, reserved, status, None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return tuple(res)


def qk_norm_rope(query: torch.Tensor, key: torch.Tensor, cos_sin: torch.Tensor,
                 positions: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                 interleaved: bool = False, out: Optional[torch.Tensor] = None,
                 key_out: Optional[torch.Tensor] = None, value: Optional[torch.Tensor] = None,
                 k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                 slots: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None
                 ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Root-mean-square norm of each query and key head and rotation by the
    tokens' positions, through ``sv_qk_norm_rope``; with a cache, keys and values
    go into it in the same pass.

    query [B, T, heads, head dim], key and value [B, T, kv heads, head dim] bf16
    or fp16, last dimension dense, other strides free (views of a fused
    projection); q_weight, k_weight [head dim] of their type, or None: no norm.
    cos_sin [positions, rotary dim] fp32, cosines then sines; positions [B, T]
    int32.  The first rotary dim elements turn in pairs: (i, i + rotary dim / 2),
    or neighbours if ``interleaved``.

    k_cache, v_cache of any type, with ``value`` and ``slots`` [B, T] int64
    (``kv_reserve``): each token's key and value go to its slot as ``kv_write``
    would put the result there; a token with a negative slot is left out, its
    outputs as they were.  Returns (out, key_out): ``out`` like query and
    ``key_out`` like key, or new tensors (not initialised); the tensors
    themselves are fine, in place.  With a cache key_out is None unless given."""
    rc, out, key_out = (_native or load_binding()).qk_norm_rope(
        query, key, cos_sin, positions, q_weight, k_weight, eps, interleaved, out, key_out, value,
        k_cache, v_cache, slots, k_scale, v_scale, status,
        None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return out, key_out


def kv_write(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
             v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
             new_lens: Optional[torch.Tensor] = None, *,
             k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> None:
    """New tokens' keys and values into the cache, in place, through
    ``sv_kv_write``; an e4m3 or 4-bit cache gets codes and scales.

    key, value [B, T, kv heads, head dim] bf16 or fp16 (the cache's own type,
    or either where it holds codes), last dimension dense, other strides free."""
    rc = (_native or load_binding()).kv_write(
        key, value, k_cache, v_cache, block_tables, seq_lens, new_lens, k_scale, v_scale, status,
        None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)


def kv_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
            lens: torch.Tensor, starts: Optional[torch.Tensor] = None, *,
            max_len: Optional[int] = None, dtype: torch.dtype = torch.bfloat16,
            out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
            k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cached tokens as dense tensors through ``sv_kv_read``: positions
    starts[b] + i (None: i) for i < lens[b].

    Returns (key, value) [B, T, kv heads, head dim]: ``out``, or new zeroed
    tensors of ``dtype`` with T = ``max_len``.  Rows at or past lens[b] are
    left as they were."""
    native = _native or load_binding()
    if out is None:
        if max_len is None:
            raise ValueError("max_len is needed when out is None")
        for t, name, dims in ((k_cache, "k_cache", 4), (block_tables, "block_tables", 2)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dim() != dims:
                raise ValueError(f"{name} must have {dims} dimensions")
        per = 2 if k_cache.dtype == torch.uint8 else 1
        shape = (block_tables.shape[0], max_len, k_cache.shape[1], k_cache.shape[3] * per)
        with torch.cuda.stream(stream):
            out = tuple(torch.zeros(shape, dtype=dtype, device=k_cache.device) for _ in range(2))
    key, value = out
    rc = native.kv_read(k_cache, v_cache, block_tables, lens, starts, key, value, k_scale, v_scale,
                        status, None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return key, value


def kv_compact(path: torch.Tensor, num_accepted: torch.Tensor, seq_lens: torch.Tensor,
               block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *,
               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
    """The accepted tree path's entries moved together, in place, through
    ``sv_kv_compact``: position seq_lens[b] + path[b, i] goes to seq_lens[b] +
    i for i < num_accepted[b].

    path [B, P] int32, strictly increasing per request.  num_accepted [B] int32
    counts the entries to keep: where the last emitted token was written with the
    drafts, as node 0, that is ``verify``'s num_accepted + 1.  The caches (and
    scales) may have a layers dimension in front: one call then moves every
    layer.  ``kv_rollback`` with the same count cuts the sequence afterwards
    (its draft_lens: the new tokens, the emitted one among them)."""
    rc = (_native or load_binding()).kv_compact(
        path, num_accepted, seq_lens, block_tables, k_cache, v_cache, k_scale, v_scale, status,
        None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)


def tree_attention_workspace_bytes(B: int, T: int, num_heads: int, num_kv_heads: int,
                                   head_dim: int) -> int:
    """Bytes of workspace ``tree_attention`` needs for batches of up to B
    requests and T new tokens."""
    return int(_api.load_library().sv_tree_attention_workspace_bytes(
        B, T, num_heads, num_kv_heads, head_dim))


def tree_attention(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, seq_lens: torch.Tensor,
                   tree_mask: Optional[torch.Tensor] = None,
                   new_lens: Optional[torch.Tensor] = None, *,
                   scale: Optional[float] = None,
                   k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the new tokens over the paged cache, which holds them
    already (``kv_write``), through ``sv_tree_attention``.

    query [B, T, heads, head dim] bf16 or fp16 (the cache's own type, or
    either where it holds codes), last dimension dense, other strides free; heads is a
    multiple of the cache's.  New token i sees the seq_lens[b] committed
    tokens and new token c < new_lens[b] where tree_mask[b, i, c] is true
    (tree_mask [B, T, T] or [T, T] bool; None: c <= i).  T = 1 is plain
    decoding.  A row that sees nothing is 0.

    scale defaults to head_dim ** -0.5.  Returns ``out`` [B, T, heads, head
    dim], contiguous; rows at or past new_lens[b] are left as they were (a
    new ``out`` is not initialised).  ``lse`` [B, T, heads] fp32 receives the
    log of the softmax denominators.  ``workspace``: a uint8 tensor of
    ``tree_attention_workspace_bytes`` on a 256-byte boundary, allocated per
    call if None; calls that share one must be ordered on one stream.

    Fast for head dims 64 and 128, block sizes that are a multiple of 8 and
    query rows on 16-byte boundaries.  Like the other operators here it is not
    differentiable."""
    rc, out = (_native or load_binding()).tree_attention(
        query, k_cache, v_cache, block_tables, seq_lens, tree_mask, new_lens, scale, k_scale,
        v_scale, out, lse, workspace, status, None if stream is None else stream.cuda_stream)
    if rc:
        _raise(rc)
    return out
