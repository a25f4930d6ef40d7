"""GB300-native speculative-decoding verification (vectorised rejection sampler).

``verify`` runs one verification step of a batch on the GPU through the C ABI
of ``lib/libspecverify.so`` (declared in ``include/spec_verify.h``);
``bind`` fixes the tensors of a loop once and re-runs the step cheaply;
``verify_host`` does the same from host tensors, copies included.

Around it, the target model's paged KV cache (``include/sv_paged.h``):
``kv_reserve`` gives the new tokens blocks, slots and positions,
``qk_norm_rope`` normalises and rotates their queries and keys and puts keys and
values there, ``kv_write`` puts ready keys and values into the cache (quantised
if it holds codes of 8 or 4 bits), ``tree_attention`` attends from the drafted tokens,
a chain or a tree, to the cache, ``kv_compact`` moves an accepted tree path
together, ``kv_rollback`` cuts the sequence behind it and ``kv_read`` reads a
sequence back.
"""
from .api import (BoundVerify, SpecVerifyError, bind, kv_rollback, last_error,  # noqa: F401
                  load_library, verify, verify_host, workspace_bytes)
from .kv import (kv_compact, kv_read, kv_reserve, kv_write, qk_norm_rope,  # noqa: F401
                 tree_attention, tree_attention_workspace_bytes)
