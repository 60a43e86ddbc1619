"""MI355X-native verify-and-resample step of speculative sampling.

The computation lives in libspecverify.so (HIP kernels for gfx950 behind a C ABI declared in
include/spec_verify.h); this package is its thin Python binding.
"""

from ._lib import (PagedCache, SpecVerifyError, expected_tokens, ops_factor,  # noqa: F401
                   optimal_gamma, release_workspaces, rotary_frequencies, sample_summary,
                   spec_acceptance_rate, spec_build_tree, spec_cache_append, spec_cache_commit,
                   spec_cache_evict, spec_cache_fork, spec_cache_resize, spec_cache_weigh,
                   spec_philox_uniform, spec_rotary, spec_rotary_append, spec_sample,
                   spec_token_logprobs, spec_tree_attention, spec_verify, spec_verify_noalloc,
                   spec_verify_tree, status_string, walltime_speedup)

__all__ = ["spec_verify", "spec_verify_noalloc", "spec_sample", "spec_verify_tree",
           "spec_build_tree", "spec_philox_uniform", "spec_acceptance_rate", "expected_tokens",
           "walltime_speedup", "ops_factor", "optimal_gamma", "SpecVerifyError", "status_string",
           "sample_summary", "release_workspaces", "PagedCache", "spec_tree_attention",
           "spec_cache_append", "spec_cache_commit", "spec_cache_resize", "spec_cache_fork",
           "rotary_frequencies", "spec_rotary", "spec_rotary_append", "spec_cache_weigh",
           "spec_cache_evict", "spec_token_logprobs"]
