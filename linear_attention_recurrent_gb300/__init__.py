"""Recurrent linear-attention decode over a paged fp32 state pool, on GB300.

GDN (gated delta rule, scalar decay), KDA (per-key-channel decay), Lightning
Attention and the selective state space scan, the short causal convolution in
front of them, the verification of drafted tokens, the draw of tokens, and the paged key/value
cache with the attention that reads it: hand-written sm_103a kernels behind the C ABI in
include/lar.h (liblar.so, built in-tree by ``_build.build()``).  This package
is the thin torch-facing binding; see ``binding`` for the calls.
"""
from .binding import (LAR_BETA_RAW, LAR_DEVERR_ACCEPTED, LAR_DEVERR_READ_SLOT, LAR_DEVERR_SEQLEN,
                      LAR_DEVERR_TIMEOUT, LAR_DEVERR_WRITE_SLOT, LAR_GATE_RAW, LAR_QK_L2NORM, LAR_STATE_KV, LarError,
                      LAR_DEVERR_DRAFT, LAR_DEVERR_PROBS, LAR_DT_SOFTPLUS, LAR_SILU,
                      PreparedCall, StepGraph,
                      gdn_decode, gdn_decode_tokens, gdn_decode_varlen, kda_decode, kda_decode_tokens,
                      kda_decode_varlen, la_decode, la_decode_varlen, gdn_prefill, kda_prefill, la_prefill,
                      conv_decode, conv_decode_tokens, conv_prefill, ssm_decode, ssm_decode_tokens, ssm_prefill,
                      spec_verify, LAR_DEVERR_PAGE, LAR_ROPE_INTERLEAVED, attn_decode, attn_workspace, kv_append,
                      sample_tokens, library_path, load)

__all__ = ["gdn_decode", "kda_decode", "la_decode", "gdn_decode_tokens", "kda_decode_tokens",
           "gdn_decode_varlen", "kda_decode_varlen", "la_decode_varlen", "gdn_prefill", "kda_prefill", "la_prefill",
           "conv_decode", "conv_decode_tokens", "conv_prefill", "ssm_decode", "ssm_decode_tokens", "ssm_prefill",
           "spec_verify", "LAR_SILU", "LAR_DT_SOFTPLUS", "LAR_DEVERR_DRAFT", "LAR_DEVERR_PROBS", "PreparedCall", "StepGraph", "LarError", "load", "library_path", "LAR_QK_L2NORM", "LAR_GATE_RAW",
           "LAR_BETA_RAW", "LAR_STATE_KV", "LAR_DEVERR_READ_SLOT", "LAR_DEVERR_WRITE_SLOT", "LAR_DEVERR_ACCEPTED",
           "LAR_DEVERR_SEQLEN", "LAR_DEVERR_TIMEOUT", "kv_append", "attn_decode", "attn_workspace", "sample_tokens",
           "LAR_ROPE_INTERLEAVED", "LAR_DEVERR_PAGE"]
