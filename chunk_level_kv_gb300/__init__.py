"""ChunkKV chunk-level KV-cache compression on one GB300: Python binding of libchunkkv.so."""
from .api import (ChunkKVError, CompressResult, Params, chunkkv_compress_layers, chunkkv_compress_tail,
                  chunkkv_tail_sizes, compress_tail, chunkkv_gather,
                  chunkkv_launch_count, chunkkv_set_phase_events, PHASES, chunkkv_selftest_wait_timeout,
                  chunkkv_layer_overlap, chunkkv_probe_ex2,
                  chunkkv_out_capacity, chunkkv_score, chunkkv_score_noalloc, chunkkv_score_path, chunkkv_select,
                  chunkkv_status_check, chunkkv_workspace_size, compress_layers, make_params,
                  params_for)
from .serve import (Q8_PAGE, PrefillParams, Q4Cache, Q8Cache, chunkkv_prefill_attention, chunkkv_prefill_path,
                    chunkkv_prefill_workspace_size, chunkkv_q4_append, chunkkv_q4_attention, chunkkv_q4_load,
                    chunkkv_q4_path, chunkkv_q4_resize, chunkkv_q4_workspace_size, chunkkv_q8_append, chunkkv_q8_attention, chunkkv_q8_load,
                    chunkkv_q8_resize, chunkkv_q8_workspace_size, prefill_attention, prefill_params_for, q4_attention,
                    q4_cache, q4_page_bytes, q8_attention, q8_cache)

__all__ = [
    "ChunkKVError", "CompressResult", "Params", "chunkkv_compress_layers", "chunkkv_compress_tail",
    "chunkkv_tail_sizes", "compress_tail", "chunkkv_gather", "chunkkv_launch_count",
    "chunkkv_set_phase_events", "PHASES", "chunkkv_selftest_wait_timeout", "chunkkv_layer_overlap",
    "chunkkv_probe_ex2",
    "chunkkv_out_capacity", "chunkkv_score", "chunkkv_score_noalloc", "chunkkv_score_path", "chunkkv_select",
    "chunkkv_status_check", "chunkkv_workspace_size", "compress_layers", "make_params", "params_for",
    "PrefillParams", "Q4Cache", "Q8Cache", "Q8_PAGE", "chunkkv_prefill_attention", "chunkkv_prefill_path",
    "chunkkv_prefill_workspace_size", "chunkkv_q4_append", "chunkkv_q4_attention", "chunkkv_q4_load", "chunkkv_q4_path",
    "chunkkv_q4_resize", "chunkkv_q4_workspace_size", "chunkkv_q8_append", "chunkkv_q8_attention", "chunkkv_q8_load",
    "chunkkv_q8_resize", "chunkkv_q8_workspace_size", "prefill_attention", "prefill_params_for", "q4_attention",
    "q4_cache", "q4_page_bytes", "q8_attention", "q8_cache",
]
