"""Selective state update (Mamba-style SSM decode, prefill, MTP replay and tree
verify), per-channel selective scan, gated delta rule, causal convolution and
draft verification over a paged recurrent-state pool, with the RMS norm and the
log probabilities around them, as hand-written HIP kernels for AMD Instinct
MI355X.

The compute lives in libssu.so (C ABI declared in include/ssu.h); this package
only marshals torch GPU tensors into those calls.
"""
from .ssu import (SsuError, SsuPool, DeviceArray, ReplayLayerTable, StateLayerTable,
                  load_library, ssu_decode, ssu_prefill, ssu_replay, ssu_tree_verify,
                  ssu_tree_verify_noalloc, TREE_SCRATCH_BYTES,
                  ssu_replay_layers, ssu_state_clear_layers, ssu_state_gather,
                  ssu_state_scatter, ssu_state_pack, ssu_state_unpack, pack_workspace_bytes,
                  ssu_conv_prefill, ssu_conv_decode, ssu_scan_prefill, ssu_scan_decode,
                  ssu_draft_verify, scan_workspace_bytes, verify_workspace_bytes,
                  ssu_delta_prefill, ssu_delta_decode, delta_workspace_bytes, ssu_rms_norm,
                  ssu_token_logprobs, logprobs_workspace_bytes,
                  ssu_gdn_decode, gdn_workspace_bytes, tree_workspace_bytes,
                  LIB_PATH, EXPORTS)

__all__ = ["SsuError", "SsuPool", "DeviceArray", "ReplayLayerTable", "StateLayerTable",
           "load_library", "ssu_decode", "ssu_prefill", "ssu_replay", "ssu_tree_verify",
           "ssu_tree_verify_noalloc", "TREE_SCRATCH_BYTES",
           "ssu_replay_layers", "ssu_state_clear_layers", "ssu_state_gather", "ssu_state_scatter",
           "ssu_state_pack", "ssu_state_unpack", "pack_workspace_bytes", "ssu_gdn_decode", "gdn_workspace_bytes",
           "ssu_conv_prefill", "ssu_conv_decode", "ssu_scan_prefill", "ssu_scan_decode",
           "ssu_draft_verify", "scan_workspace_bytes", "verify_workspace_bytes", "tree_workspace_bytes",
           "ssu_delta_prefill", "ssu_delta_decode", "delta_workspace_bytes", "ssu_rms_norm",
           "ssu_token_logprobs", "logprobs_workspace_bytes",
           "LIB_PATH", "EXPORTS"]
