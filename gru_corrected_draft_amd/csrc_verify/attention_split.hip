// bf16 attention over a bf16 cache.
#include "attention_split.h"

// workspace: two parts of the most rows, their outputs and (m, l), for each
// workgroup
size_t attend_split_floats(int head_dim, int cus) {
  return (size_t)2 * cus * (head_dim == 256 ? 128 : 256) * (head_dim + 2);
}

hipError_t attend_split_prepare(int head_dim) { return prepare<false>(head_dim); }

void launch_attend_split(int head_dim, const AttendArgs& a, int cus, hipStream_t st) {
  launch_dim<false>(head_dim, a, cus, st);
}
