"""GB300-native paged KV-cache decode path (PagedAttention) behind a C ABI.

The compute lives in libpagedkv.so (CUDA kernels for sm_103a plus the C++
block manager); ``pagedkv`` is its thin ctypes binding and ``workloads`` the
seeded synthetic inputs.  Build with ``python -m paged_kv_cache_05_gb300.build``.
"""
from .pagedkv import (BlockManager, OutOfBlocks, PagedKVError, alloc_grouped_workspace,
                      alloc_latent_workspace, alloc_workspace, copy_blocks,
                      contiguous_attention_decode, contiguous_workspace_size,
                      decode_grouped_workspace_size,
                      decode_shared_workspace_size, decode_workspace_size, gather_latent, get_device_error,
                      latent_attention_decode, latent_attention_prefill,
                      latent_decode_workspace_size, latent_norm_rope_and_cache,
                      latent_prefill_workspace_size, lib,
                      paged_attention_decode, paged_attention_decode_append, paged_attention_decode_grouped,
                      paged_attention_decode_noalloc, paged_attention_decode_shared,
                      norm_rope_and_cache, paged_attention_prefill,
                      paged_attention_prefill_grouped, paged_attention_prefill_write,
                      prefill_grouped_workspace_size,
                      reshape_and_cache, rope_inv_freq, rope_phases, set_decode_wait_limit,
                      swap_blocks, version)

__all__ = ["BlockManager", "OutOfBlocks", "PagedKVError", "alloc_grouped_workspace",
           "alloc_latent_workspace", "alloc_workspace", "copy_blocks",
           "contiguous_attention_decode", "contiguous_workspace_size",
           "decode_grouped_workspace_size",
           "decode_shared_workspace_size", "decode_workspace_size", "gather_latent", "get_device_error",
           "latent_attention_decode", "latent_attention_prefill", "latent_decode_workspace_size",
           "latent_norm_rope_and_cache", "latent_prefill_workspace_size", "lib", "paged_attention_decode",
           "paged_attention_decode_append", "paged_attention_decode_grouped",
           "paged_attention_decode_noalloc", "paged_attention_decode_shared",
           "norm_rope_and_cache", "paged_attention_prefill",
           "paged_attention_prefill_grouped", "paged_attention_prefill_write",
           "prefill_grouped_workspace_size",
           "reshape_and_cache", "rope_inv_freq", "rope_phases", "set_decode_wait_limit",
           "swap_blocks", "version"]
