// bf16 attention over a bf16 cache.
#include "attention_split.h"

namespace {

template <int D>
hipError_t allow_lds_d() {
  hipError_t e = allow_lds<D, 1, false>();
  if (e == hipSuccess) e = allow_lds<D, 4, false>();
  if constexpr (D < 256) {
    if (e == hipSuccess) e = allow_lds<D, 2, false>();
    if (e == hipSuccess) e = allow_lds<D, 8, false>();
  }
  return e;
}

// The fewest rows to a workgroup that hold a request's, so that its keys are
// read once; beyond 128 rows the largest.  A wave costs the same whether its
// rows are there or not.
template <int D>
void launch_d(const AttendArgs& a, int cus, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.group;
  if (rows <= 32) return launch<D, 1, false>(a, cus, st);
  if constexpr (D == 256) {
    launch<D, 4, false>(a, cus, st);
  } else {
    if (rows <= 64) return launch<D, 2, false>(a, cus, st);
    if (rows <= 128) return launch<D, 4, false>(a, cus, st);
    launch<D, 8, false>(a, cus, st);
  }
}

}  // namespace

// workspace: two parts of the most rows, their outputs and (m, l), for each
// workgroup
size_t attend_split_floats(int head_dim, int cus) {
  return (size_t)2 * cus * (head_dim == 256 ? 128 : 256) * (head_dim + 2);
}

hipError_t attend_split_prepare(int head_dim) {
  return head_dim == 64 ? allow_lds_d<64>() : head_dim == 128 ? allow_lds_d<128>() : allow_lds_d<256>();
}

void launch_attend_split(int head_dim, const AttendArgs& a, int cus, hipStream_t st) {
  if (head_dim == 64)
    launch_d<64>(a, cus, st);
  else if (head_dim == 128)
    launch_d<128>(a, cus, st);
  else
    launch_d<256>(a, cus, st);
}
