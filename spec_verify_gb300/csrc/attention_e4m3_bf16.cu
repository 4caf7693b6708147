#include "cache_attention.cuh"

namespace smp {
SMP_ATTENTION_INSTANCE(SMP_CACHE_E4M3, false)
}  // namespace smp
