"""torch.library custom ops over the C ABI: ``torch.ops.w4a16.gemm`` and the serving operators.

The PR #51453 report ("register Triton W4A16 GEMM as custom op", motivation and implementation
breakdown) traces a decode throughput regression to torch.compile tracing the Python tile
selection and freezing the prefill configuration into decode calls; the fix is an opaque custom op
with a fake implementation, so that the compiled graph holds one call node and tile selection sees
the real runtime shape. Here the tile, split-K and cluster choice already live inside the library
(chosen per call from the runtime M), and this module makes the call opaque to torch.compile:

* the real implementation forwards to ``w4a16_gemm`` of the binding (no computation in Python);
* the fake implementation only states the output metadata, as the pages' fake impl does:
  shape (a.size(0), b_q.size(1) * 8), dtype and device of ``a``; it checks nothing;
* ``mutates_args=()``: inputs are not written, the output is a new tensor.

The serving operators (``rope``, ``kv_write``, ``kv_write_q``, ``kv_read``, ``tree_attention``, ``tree_attention_lse``,
``token_logprobs``) are opaque calls in the same way: each forwards to the binding's function of that name, its fake
implementation states the outputs' metadata, and the two writes say that they change the cache.

Import this module to register the ops.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import serving as _serving
from . import w4a16_gemm as _w4a16_gemm


@torch.library.custom_op("w4a16::gemm", mutates_args=())
def gemm(a: torch.Tensor, b_q: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor],
         group_size: int, zp_bias: int = 8, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out = cast(a @ dequant(b_q, scales, qzeros | zp_bias) + bias); runs libw4a16.so."""
    return _w4a16_gemm(a, b_q, scales, qzeros, group_size, zp_bias, bias)


@gemm.register_fake
def _gemm_fake(a, b_q, scales, qzeros, group_size, zp_bias=8, bias=None):
    return a.new_empty((a.size(0), b_q.size(1) * 8))


def w4a16_linear(a: torch.Tensor, b_q: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor],
                 group_size: int, zp_bias: int = 8, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Facade with the signature of the pages' ``triton_w4a16_gemm`` (plus bias), routed through the op."""
    return torch.ops.w4a16.gemm(a, b_q, scales, qzeros, group_size, zp_bias, bias)


@torch.library.custom_op("w4a16::rope", mutates_args=())
def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False) -> torch.Tensor:
    """Heads of x turned to their tokens' positions, in a new tensor."""
    return _serving.w4a16_rope(x, positions, table, interleaved)


@rope.register_fake
def _rope_fake(x, positions, table, interleaved=False):
    return x.new_empty(x.shape)


@torch.library.custom_op("w4a16::kv_write", mutates_args=("cache",))
def kv_write(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
             positions: Optional[torch.Tensor] = None, table: Optional[torch.Tensor] = None, interleaved: bool = False) -> None:
    """Quantises k (turned first, with positions and table) and v into the cache's slots."""
    _serving.w4a16_kv_write(k, v, cache, slots, positions=positions, table=table, interleaved=interleaved)


@kv_write.register_fake
def _kv_write_fake(k, v, cache, slots, positions=None, table=None, interleaved=False):
    return None


@torch.library.custom_op("w4a16::kv_write_q", mutates_args=("cache",))
def kv_write_q(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
               positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False) -> torch.Tensor:
    """The same with the rotation of q in the call: returns the turned q."""
    return _serving.w4a16_kv_write(k, v, cache, slots, q=q, positions=positions, table=table, interleaved=interleaved)


@kv_write_q.register_fake
def _kv_write_q_fake(q, k, v, cache, slots, positions, table, interleaved=False):
    return q.new_empty(q.shape)


@torch.library.custom_op("w4a16::kv_read", mutates_args=())
def kv_read(cache: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values of the given slots."""
    return _serving.w4a16_kv_read(cache, slots, head_dim, dtype)


@kv_read.register_fake
def _kv_read_fake(cache, slots, head_dim, dtype):
    shape = (slots.size(0), cache.size(1), head_dim)
    return cache.new_empty(shape, dtype=dtype), cache.new_empty(shape, dtype=dtype)


@torch.library.custom_op("w4a16::tree_attention", mutates_args=())
def tree_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                   q_start: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                   softmax_scale: Optional[float] = None, max_q: Optional[int] = None) -> torch.Tensor:
    """Attention of the query tokens over their sequences' cached tokens."""
    return _serving.w4a16_tree_attention(q, cache, page_table, kv_lens, q_start, tree_mask, softmax_scale, max_q)


@tree_attention.register_fake
def _tree_attention_fake(q, cache, page_table, kv_lens, q_start=None, tree_mask=None, softmax_scale=None, max_q=None):
    return q.new_empty(q.shape)


@torch.library.custom_op("w4a16::tree_attention_lse", mutates_args=())
def tree_attention_lse(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                       q_start: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                       softmax_scale: Optional[float] = None, max_q: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The same with the log-sum-exp of each row."""
    return _serving.w4a16_tree_attention(q, cache, page_table, kv_lens, q_start, tree_mask, softmax_scale, max_q, return_lse=True)


@tree_attention_lse.register_fake
def _tree_attention_lse_fake(q, cache, page_table, kv_lens, q_start=None, tree_mask=None, softmax_scale=None, max_q=None):
    return q.new_empty(q.shape), q.new_empty((q.size(0), q.size(1)), dtype=torch.float32)


@torch.library.custom_op("w4a16::token_logprobs", mutates_args=())
def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None,
                   top_k: int = 0) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(logprobs, entropy, top_ids, top_logprobs) of rows of logits."""
    return _serving.w4a16_token_logprobs(logits, tokens, top_k)


@token_logprobs.register_fake
def _token_logprobs_fake(logits, tokens=None, top_k=0):
    rows = logits.size(0)
    f = lambda *shape: logits.new_empty(shape, dtype=torch.float32)
    return f(*(tokens.shape if tokens is not None else (rows, 0))), f(rows), logits.new_empty((rows, top_k), dtype=torch.int64), f(rows, top_k)
