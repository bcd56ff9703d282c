// The 4-bit cache's layout (include/pks.h), shared by the kernels that write, read
// and attend over it.
#pragma once

#include <stdint.h>

namespace pks {
namespace q4 {

constexpr int kGroup = 32;  // values that share an (s, m) pair

// bytes of one head's record: codes, then an (s, m) pair of fp16 a group
__host__ __device__ constexpr int record_bytes(int D) { return D / 2 + D / kGroup * 4; }
__host__ __device__ constexpr int token_bytes(int heads, int D) {
  return (heads * record_bytes(D) + 15) / 16 * 16;
}

}  // namespace q4
}  // namespace pks
