"""Paged-KV attention for one continuous-batching step on GB300 (sm_103a).

The computation lives in libpa.so (hand-written CUDA kernels behind a C ABI,
declared in include/pa.h); `binding` exposes the same calls on torch tensors.
"""
from .binding import (PA_BF16, PA_DEV_BLOCK_RANGE, PA_DEV_CAPACITY, PA_DEV_LENGTHS, PA_DEV_QSL,
                      PA_DEV_POSITION, PA_DEV_SLOT_RANGE, PA_DEV_TIMEOUT, PA_ERR_CUDA, PA_ERR_INVALID,
                      PA_ERR_UNSUPPORTED, PA_F32, PA_FP8_E4M3, PA_INT4, PA_INT4_LIMIT, PA_OK,
                      PA_ROPE_HALVES, PA_ROPE_PAIRS, PaError,
                      alloc_latent_workspace, alloc_workspace, cache_shape, last_error, latent_cache_shape,
                      latent_layout_of, layout_of, lib, make_latent_layout, make_layout,
                      pa_cache_read, pa_cache_write, pa_expanded_forward, pa_expanded_layout,
                      pa_expanded_workspace_size, pa_forward,
                      pa_forward_noalloc, pa_forward_workspace_size, pa_latent_forward, pa_latent_layout,
                      pa_latent_read, pa_latent_workspace_size, pa_latent_write, pa_layout, pa_rope,
                      pa_rope_cache_write,
                      pa_set_prefill_overlap, pa_set_prefill_profile_events,
                      pa_set_profile_events)

__all__ = ["PA_BF16", "PA_DEV_BLOCK_RANGE", "PA_DEV_CAPACITY", "PA_DEV_LENGTHS", "PA_DEV_QSL",
           "PA_DEV_POSITION", "PA_DEV_SLOT_RANGE", "PA_DEV_TIMEOUT", "PA_ERR_CUDA", "PA_ERR_INVALID",
           "PA_ERR_UNSUPPORTED", "PA_F32", "PA_FP8_E4M3", "PA_INT4", "PA_INT4_LIMIT", "PA_OK",
           "PA_ROPE_HALVES", "PA_ROPE_PAIRS", "PaError",
           "alloc_latent_workspace", "alloc_workspace", "cache_shape", "last_error", "latent_cache_shape",
           "latent_layout_of", "layout_of", "lib", "make_latent_layout", "make_layout",
           "pa_cache_read", "pa_cache_write", "pa_expanded_forward", "pa_expanded_layout",
           "pa_expanded_workspace_size", "pa_forward",
           "pa_forward_noalloc", "pa_forward_workspace_size", "pa_latent_forward", "pa_latent_layout",
           "pa_latent_read", "pa_latent_workspace_size", "pa_latent_write", "pa_layout", "pa_rope",
           "pa_rope_cache_write",
           "pa_set_prefill_overlap", "pa_set_prefill_profile_events", "pa_set_profile_events"]
