"""spec_verify_gb300: a batched next-token sampler and speculative-decoding
verifier for NVIDIA GB300 (sm_103a), with the cached step that feeds them.

The compute lives in libsmp.so (C ABI: include/smp.h, include/smp_cache.h),
built in-tree by `python -m spec_verify_gb300.build`.
`spec_verify_gb300.binding` wraps the sampler and the verifier for PyTorch
tensors, `spec_verify_gb300.cache` the speculative step over a paged 8-bit
cache; `spec_verify_gb300.workloads` makes seeded synthetic inputs.
"""

__all__ = ["binding", "build", "cache", "workloads"]
