"""Python binding of the paged-cache operators (``include/sv_paged.h``).

Argument marshalling only: shapes and types are checked here, sizes and
alignments by the library, and the work is done by its CUDA kernels on the
current (or given) stream.  Every call packs its arguments into one struct of
8-byte words, so that a call costs a few microseconds of host time.

The cache.  ``k_cache`` and ``v_cache`` [num_blocks, kv heads, block size,
head dim], bf16, fp16 or float8_e4m3fn, their last three dimensions dense and
their strides equal (they may be two halves of one buffer).  An e4m3 cache has
``k_scale`` and ``v_scale`` [num_blocks, kv heads, block size, head dim / 32]
uint8: value = code * 2^(scale - 127).  ``block_tables`` [B, max_blocks] int32
(-1 = no block) and ``seq_lens`` [B] int32 (committed tokens L) are those of
``kv_rollback``; ``new_lens`` [B] int32 or None (all T) counts the new tokens
of a request, at positions L .. L + n - 1.  ``status`` is None or a 1-element
int32/uint32 tensor that receives SV_KV_* bits (the caller zeroes it).
"""
from __future__ import annotations

import struct
from typing import Optional, Tuple

import torch

from . import api as _api
from .api import SV_BF16, SV_F32, SV_OK, SpecVerifyError

SV_F16 = 2
SV_E4M3 = 3

SV_KV_BAD_BLOCK = 0x10
SV_KV_BAD_PATH = 0x20
SV_KV_GROUP = 32

_CODES = {torch.bfloat16: SV_BF16, torch.float16: SV_F16, torch.float8_e4m3fn: SV_E4M3}
_OUT_CODES = {torch.bfloat16: SV_BF16, torch.float16: SV_F16, torch.float32: SV_F32}
_I32 = torch.int32
_CACHE_WORDS = 16

# The structs of include/sv_paged.h: struct_bytes, the cache, the rest.
_WRITE = struct.Struct(f"@{1 + _CACHE_WORDS + 4 + 6 + 4}q")
_READ = struct.Struct(f"@{1 + _CACHE_WORDS + 4 + 6 + 4}q")
_COMPACT = struct.Struct(f"@{1 + _CACHE_WORDS + 3 + 3}q")
_ATTN = struct.Struct(f"@{1 + _CACHE_WORDS + 3 + 3 + 4}qd{4 + 3}q")


def _dev(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _ids(t, name, shape, dev) -> int:
    """Pointer of an int32 tensor of this shape on this device (0 for None)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _I32:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {_I32}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _status(t, dev) -> int:
    if t is None:
        return 0
    if t.get_device() != dev or t.numel() != 1 or t.dtype not in (torch.int32, torch.uint32):
        raise ValueError("status must be a 1-element int32/uint32 tensor on the same device")
    return t.data_ptr()


def _same(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _pool(k, v, what, lead):
    """Strides (layer, block) of a k / v pair whose last three dimensions are
    dense.  Dimensions of one element may have any stride."""
    s, h = k.stride(), k.shape
    want = 1
    for d in (-1, -2, -3):
        if h[d] != 1 and s[d] != want:
            raise ValueError(f"{what}: the last three dimensions must be dense")
        want *= h[d]
    if v.stride() != s:
        for a, b, n in zip(s, v.stride(), h):
            if n > 1 and a != b:
                raise ValueError(f"{what}: k and v must have the same strides")
    return (s[0] if lead else 0), s[1 if lead else 0]


def _cache(k, v, ks, vs, tables, dev, lead=False):
    """The sv_kv_cache words, and (heads, head dim, dtype)."""
    if not isinstance(k, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    code = _CODES.get(k.dtype)
    if code is None:
        raise TypeError(f"unsupported cache dtype {k.dtype}")
    shape = k.shape
    if len(shape) != (5 if lead else 4):
        raise ValueError("k_cache and v_cache must be [num_blocks, kv heads, block size, head dim]"
                         + (", with the layers in front" if lead else ""))
    if k.get_device() != dev:
        raise ValueError(f"k_cache is on {k.device}, expected cuda:{dev}")
    _same(v, "v_cache", shape, k.dtype, dev)
    if 0 in shape[-3:]:
        raise ValueError("k_cache has an empty dimension")
    layer, block = _pool(k, v, "k_cache and v_cache", lead)
    D = shape[-1]
    if code == SV_E4M3:
        if ks is None or vs is None:
            raise ValueError("an e4m3 cache needs k_scale and v_scale")
        if D % SV_KV_GROUP:
            raise ValueError(f"the head dim of an e4m3 cache is a multiple of {SV_KV_GROUP}")
        sshape = shape[:-1] + (D // SV_KV_GROUP,)
        _same(ks, "k_scale", sshape, torch.uint8, dev)
        _same(vs, "v_scale", sshape, torch.uint8, dev)
        slayer, sblock = _pool(ks, vs, "k_scale and v_scale", lead)
        sk, sv = ks.data_ptr(), vs.data_ptr()
    else:
        if ks is not None or vs is not None:
            raise ValueError("k_scale and v_scale belong to an e4m3 cache")
        sk = sv = slayer = sblock = 0
    if not isinstance(tables, torch.Tensor) or tables.dim() != 2:
        raise ValueError("block_tables must be [B, max_blocks]")
    tb = _ids(tables, "block_tables", tables.shape, dev)
    return (k.data_ptr(), v.data_ptr(), sk, sv, layer, block, slayer, sblock,
            shape[0] if lead else 1, shape[-4], shape[-3], shape[-2], D, code, tb, tables.shape[1])


def _dense(t, name, shape, dtype, dev):
    """Pointer and (b, t, head) strides of a [B, T, heads, D] tensor."""
    _same(t, name, shape, dtype, dev)
    s = t.stride()
    if s[3] != 1 and shape[3] != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    return t.data_ptr(), s[0], s[1], s[2]


def _no_overlap(t, name):
    """Refuses an output with two elements in one place (an expanded view)."""
    for n, s in zip(t.shape, t.stride()):
        if n > 1 and s == 0:
            raise ValueError(f"{name} must not be an expanded tensor")


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else None


def _call(fn, args: bytes, dev: int, stream) -> None:
    if stream is not None:
        handle = stream.cuda_stream
    elif _raw_stream is not None:
        handle = _raw_stream(dev)
    else:
        handle = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev:
        rc = fn(args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(args, handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, _api.load_library())


def kv_write(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
             v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
             new_lens: Optional[torch.Tensor] = None, *,
             k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> None:
    """New tokens' keys and values into the cache, in place, through
    ``sv_kv_write``; an e4m3 cache gets codes and scales.

    key, value [B, T, kv heads, head dim] bf16 or fp16 (the cache's own type,
    or either for e4m3), last dimension dense, other strides free."""
    lib = _api.load_library()
    dev = _dev(key, "key")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, block_tables, dev)
    if key.dim() != 4:
        raise ValueError("key must be [B, T, kv heads, head dim]")
    shape = key.shape
    code = _CODES.get(key.dtype)
    if code is None or code == SV_E4M3:
        raise TypeError(f"unsupported key dtype {key.dtype}")
    if cache[13] != SV_E4M3 and cache[13] != code:
        raise TypeError(f"a {k_cache.dtype} cache takes no {key.dtype} keys")
    B, T = shape[0], shape[1]
    if shape[2] != cache[10] or shape[3] != cache[12] or block_tables.shape[0] != B:
        raise ValueError(f"key {tuple(shape)}, k_cache {tuple(k_cache.shape)} and block_tables "
                         f"{tuple(block_tables.shape)} do not belong together")
    kp, ksb, kst, ksh = _dense(key, "key", shape, key.dtype, dev)
    vp, vsb, vst, vsh = _dense(value, "value", shape, key.dtype, dev)
    sl = _ids(seq_lens, "seq_lens", (B,), dev)
    nl = _ids(new_lens, "new_lens", (B,), dev)
    _call(lib.sv_kv_write,
          _WRITE.pack(_WRITE.size, *cache, sl, nl, kp, vp, ksb, kst, ksh, vsb, vst, vsh,
                      B, T, code, _status(status, dev)), dev, stream)


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
    lib = _api.load_library()
    dev = _dev(k_cache, "k_cache")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, block_tables, dev)
    B = block_tables.shape[0]
    if out is None:
        if max_len is None:
            raise ValueError("max_len is needed when out is None")
        with torch.cuda.stream(stream):
            out = tuple(torch.zeros(B, max_len, cache[10], cache[12], dtype=dtype,
                                    device=k_cache.device) for _ in range(2))
    key, value = out
    if not isinstance(key, torch.Tensor) or key.dim() != 4:
        raise ValueError("out must be two [B, T, kv heads, head dim] tensors")
    shape = key.shape
    code = _OUT_CODES.get(key.dtype)
    if code is None:
        raise TypeError(f"unsupported output dtype {key.dtype}")
    if shape[0] != B or shape[2] != cache[10] or shape[3] != cache[12]:
        raise ValueError(f"out {tuple(shape)}, k_cache {tuple(k_cache.shape)} and block_tables "
                         f"{tuple(block_tables.shape)} do not belong together")
    kp, ksb, kst, ksh = _dense(key, "out[0]", shape, key.dtype, dev)
    vp, vsb, vst, vsh = _dense(value, "out[1]", shape, key.dtype, dev)
    _no_overlap(key, "out[0]")
    _no_overlap(value, "out[1]")
    ln = _ids(lens, "lens", (B,), dev)
    sp = _ids(starts, "starts", (B,), dev)
    _call(lib.sv_kv_read,
          _READ.pack(_READ.size, *cache, sp, ln, kp, vp, ksb, kst, ksh, vsb, vst, vsh,
                     B, shape[1], code, _status(status, dev)), dev, stream)
    return key, value


def kv_compact(path: torch.Tensor, num_accepted: torch.Tensor, seq_lens: torch.Tensor,
               block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *,
               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
    """The accepted tree path's entries moved together, in place, through
    ``sv_kv_compact``: position seq_lens[b] + path[b, i] goes to seq_lens[b] +
    i for i < num_accepted[b].

    path [B, P] int32, strictly increasing per request.  The caches (and
    scales) may have a layers dimension in front: one call then moves every
    layer.  ``kv_rollback`` with the same num_accepted cuts the sequence
    afterwards."""
    lib = _api.load_library()
    dev = _dev(k_cache, "k_cache")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, block_tables, dev, k_cache.dim() == 5)
    B = block_tables.shape[0]
    if not isinstance(path, torch.Tensor) or path.dim() != 2:
        raise ValueError("path must be [B, P]")
    P = path.shape[1]
    pp = _ids(path, "path", (B, P), dev)
    na = _ids(num_accepted, "num_accepted", (B,), dev)
    sl = _ids(seq_lens, "seq_lens", (B,), dev)
    _call(lib.sv_kv_compact,
          _COMPACT.pack(_COMPACT.size, *cache, pp, na, sl, B, P, _status(status, dev)),
          dev, stream)


_ws_bytes: dict = {}  # sizes only


def tree_attention_workspace_bytes(B: int, T: int, num_heads: int, num_kv_heads: int,
                                   head_dim: int) -> int:
    """Bytes of workspace ``tree_attention`` needs for batches of these sizes."""
    key = (B, T, num_heads, num_kv_heads, head_dim)
    n = _ws_bytes.get(key)
    if n is None:
        n = int(_api.load_library().sv_tree_attention_workspace_bytes(*key))
        if len(_ws_bytes) > 4096:
            _ws_bytes.clear()
        _ws_bytes[key] = n
    return n


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
    either for e4m3), last dimension dense, other strides free; heads is a
    multiple of the cache's.  New token i sees the seq_lens[b] committed
    tokens and new token c < new_lens[b] where tree_mask[b, i, c] is true
    (tree_mask [B, T, T] or [T, T] bool; None: c <= i).  T = 1 is plain
    decoding.  A row that sees nothing is 0.

    scale defaults to head_dim ** -0.5.  Returns ``out`` [B, T, heads, head
    dim], contiguous; rows at or past new_lens[b] are left as they were (a
    new ``out`` is not initialised).  ``lse`` [B, T, heads] fp32 receives the
    log of the softmax denominators.  ``workspace``: a uint8 tensor of
    ``tree_attention_workspace_bytes`` on a 256-byte boundary, allocated per
    call if None; calls that share one must be ordered on one stream."""
    lib = _api.load_library()
    dev = _dev(query, "query")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, block_tables, dev)
    if query.dim() != 4:
        raise ValueError("query must be [B, T, heads, head dim]")
    shape = query.shape
    B, T, H, D = shape
    code = _CODES.get(query.dtype)
    if code is None or code == SV_E4M3:
        raise TypeError(f"unsupported query dtype {query.dtype}")
    if cache[13] != SV_E4M3 and cache[13] != code:
        raise TypeError(f"{query.dtype} queries do not read a {k_cache.dtype} cache")
    if D != cache[12] or H % cache[10] or block_tables.shape[0] != B:
        raise ValueError(f"query {tuple(shape)}, k_cache {tuple(k_cache.shape)} and block_tables "
                         f"{tuple(block_tables.shape)} do not belong together")
    qp, qsb, qst, qsh = _dense(query, "query", shape, query.dtype, dev)
    sl = _ids(seq_lens, "seq_lens", (B,), dev)
    nl = _ids(new_lens, "new_lens", (B,), dev)
    mp = msb = 0
    if tree_mask is not None:
        if not isinstance(tree_mask, torch.Tensor) or tree_mask.dtype is not torch.bool:
            raise TypeError("tree_mask must be a bool tensor")
        if tree_mask.shape != (T, T) and tree_mask.shape != (B, T, T):
            raise ValueError(f"tree_mask has shape {tuple(tree_mask.shape)}, expected "
                             f"{(T, T)} or {(B, T, T)}")
        if tree_mask.get_device() != dev:
            raise ValueError(f"tree_mask is on {tree_mask.device}, expected cuda:{dev}")
        ms = tree_mask.stride()
        if T > 1 and ms[-2:] != (T, 1):
            raise ValueError("tree_mask: the last two dimensions must be dense")
        mp = tree_mask.data_ptr()
        if tree_mask.dim() == 3 and B > 1:
            msb = ms[0]
    with_out = out is not None
    if with_out:
        _same(out, "out", shape, query.dtype, dev)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
    if lse is not None:
        _same(lse, "lse", (B, T, H), torch.float32, dev)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    need = tree_attention_workspace_bytes(B, T, H, cache[10], D)
    if workspace is not None:
        _same(workspace, "workspace", workspace.shape, torch.uint8, dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    if not with_out or workspace is None:
        # New tensors belong to the stream that uses them.
        if stream is None:
            out, workspace = _new(out, workspace, shape, query, need)
        else:
            with torch.cuda.stream(stream):
                out, workspace = _new(out, workspace, shape, query, need)
    _call(lib.sv_tree_attention,
          _ATTN.pack(_ATTN.size, *cache, sl, nl, qp, qsb, qst, qsh, mp, msb, out.data_ptr(),
                     0 if lse is None else lse.data_ptr(),
                     float(D ** -0.5 if scale is None else scale), B, T, H, code,
                     workspace.data_ptr(), workspace.numel(), _status(status, dev)),
          dev, stream)
    return out


def _new(out, workspace, shape, query, need):
    if out is None:
        out = torch.empty(shape, dtype=query.dtype, device=query.device)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=query.device)
    return out, workspace
