#include "cache_attention.cuh"

namespace smp {
SMP_ATTENTION_INSTANCE(SMP_CACHE_I8, false)
}  // namespace smp
