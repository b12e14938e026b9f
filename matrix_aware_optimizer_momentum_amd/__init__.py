"""MI355X-native Muon-family optimizer step (Sign-Muon, CacheMuon, LionMuon),
the AdamW step of the parameters beside the matrices, and the feed-forward
layers whose gradients the steps read.

The step runs in the HIP library libsm.so (C ABI in include/sm.h); this
package is its Python binding.  Importing it does not load the library; the
first call does, and fails loudly if it has not been built.
"""
from ._binding import (ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, BF16, CACHE_MUON, ENC_BITS, ENC_INT8, F32, LION_MUON, MODE_FORCE_FRESH,
                       MODE_FORCE_REUSE, MODE_TRIGGER, ROUND_NEAREST, ROUND_STOCHASTIC, SIGN_MUON,
                       UPDATE_POLAR, UPDATE_VOTE, SmError, lib)
from .api import (Act8, AdamWConfig, MatrixBuffers, NSParams, ParamBuffers, ParamSet, StepCall, StepConfig,
                  StepGraph, act8_pack, act8_unpack, adamw, gated, gated_grad, grad_norm, gram_ns_cached, gram_ns_cached_ws, linear, linear_grad, mfma_ceiling, ns_polar, ns_polar_noalloc, ns_polar_ws, polar_update, profile_enable,
                  profile_read, profile_read_bytes, profile_reset, sign_int8, sign_pack, spectral_norm, state8_pack,
                  state8_unpack, step, step_ws, vote, vote_update, vote_update_int8)

__all__ = [
    "AdamWConfig", "ParamBuffers", "ParamSet", "ROUND_NEAREST", "ROUND_STOCHASTIC", "adamw",
    "grad_norm", "state8_pack", "state8_unpack",
    "ACT_GELU", "ACT_GELU_TANH", "ACT_NONE", "ACT_RELU", "ACT_SILU", "Act8", "act8_pack",
    "act8_unpack", "gated", "gated_grad", "linear", "linear_grad",
    "BF16", "CACHE_MUON", "ENC_BITS", "ENC_INT8", "F32", "LION_MUON", "MODE_FORCE_FRESH",
    "MODE_FORCE_REUSE", "MODE_TRIGGER", "SIGN_MUON", "UPDATE_POLAR", "UPDATE_VOTE", "SmError",
    "lib", "MatrixBuffers", "NSParams", "StepCall", "StepConfig", "StepGraph", "gram_ns_cached",
    "gram_ns_cached_ws", "mfma_ceiling", "ns_polar", "ns_polar_noalloc", "ns_polar_ws", "polar_update", "profile_enable",
    "profile_read", "profile_read_bytes", "profile_reset", "sign_int8", "sign_pack", "spectral_norm", "step",
    "step_ws", "vote",
    "vote_update", "vote_update_int8",
]
