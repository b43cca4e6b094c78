// prefill_tc.cu — instances of the tcgen05 multi-token kernel (prefill_tc.cuh)
// for 16-bit and E4M3 caches.
#include "prefill_tc.cuh"

namespace paged {

cudaError_t launch_prefill_tc(const PrefillArgs& a, const CUtensorMap& kmap,
                              const CUtensorMap& vmap, int q_dtype, int cache_dtype,
                              int head_dim, int group, int32_t max_query_len,
                              cudaStream_t stream) {
  // two row groups (256 rows) when the chunks fill them
  const bool two = static_cast<int64_t>(max_query_len) * group >= 2 * kTcRows;
#define PAGED_TC(QF, CF, d, g)                                                          \
  if (head_dim == d && group == g)                                                      \
    return two ? launch_tc<QF, CF, d, g, 2>(a, {kmap, vmap}, max_query_len, stream)    \
               : launch_tc<QF, CF, d, g, 1>(a, {kmap, vmap}, max_query_len, stream);
#define PAGED_TC_ALL(QF)                                                              \
  PAGED_TC(QF, QF, 64, 1) PAGED_TC(QF, QF, 64, 2) PAGED_TC(QF, QF, 64, 4)             \
  PAGED_TC(QF, QF, 64, 8) PAGED_TC(QF, QF, 128, 1) PAGED_TC(QF, QF, 128, 2)           \
  PAGED_TC(QF, QF, 128, 4) PAGED_TC(QF, QF, 128, 8)
#define PAGED_TC_FP8(QF)                                                              \
  PAGED_TC(QF, E4M3, 128, 1) PAGED_TC(QF, E4M3, 128, 2) PAGED_TC(QF, E4M3, 128, 4)    \
  PAGED_TC(QF, E4M3, 128, 8)
  const bool fp8 = cache_dtype == kE4M3;
  if (q_dtype == kF16) {
    if (fp8) {
      PAGED_TC_FP8(F16)
    } else {
      PAGED_TC_ALL(F16)
    }
  } else if (q_dtype == kBF16) {
    if (fp8) {
      PAGED_TC_FP8(BF16)
    } else {
      PAGED_TC_ALL(BF16)
    }
  }
#undef PAGED_TC_FP8
#undef PAGED_TC_ALL
#undef PAGED_TC
  return cudaErrorNotSupported;
}

}  // namespace paged
