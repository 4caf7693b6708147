// The rows per key head that the host expects of a call's requests: with them
// it chooses the attention kernel (cache_attention.cuh), without waiting for
// the lengths on the device.
#pragma once

#include <stdint.h>

namespace smp {

// Tokens that divide evenly: the requests of a step of equal drafts add
// tokens / batch each, and so do the places of a captured step of that
// capacity.  Else the step is ragged, and most requests are nearer the longest
// than the average: a quarter more.  Measured on 32 requests of up to 4 K
// keys, heads of 128, four to a key head: 5 tokens each 61.7 us as they are
// (88.0 with a quarter more), 4 each 48.0 (54.5), 6 each 63.7 (89.1).  Ragged
// steps whose tokens divide evenly by chance pay for it: 128 tokens in
// requests of 1 and 5 take 68.0 us (60.2).
inline int64_t attention_rows(int64_t tokens, int64_t batch, int64_t group) {
  if (tokens % batch == 0) return tokens / batch * group;
  return (tokens * group * 5 / 4 + batch - 1) / batch;
}

}  // namespace smp
