// prefill_mxfp4.cu — instances of the tcgen05 multi-token kernel
// (prefill_tc.cuh) for an MXFP4 cache. On a B200: 8 draft tokens for 64
// sequences of 1 024 to 4 096 tokens, 64 heads on 8, bf16, 112 us (16-bit cache
// 118); 512-token chunks of 16 contexts of 512 to 4 096 tokens, 32 heads, f16,
// 226 us (204), of which the pass over the scales is 18.
#include "prefill_tc.cuh"

namespace paged {

cudaError_t launch_prefill_mxfp4(const PrefillArgs& a, const uint8_t* const (&planes)[4],
                                 int q_dtype, int head_dim, int group, int32_t max_query_len,
                                 bool two, cudaStream_t stream) {
  const TcCache<Mxfp4> cache{{planes[0], planes[1]}, {planes[2], planes[3]}};
#define PAGED_TC(QF, d, g)                                                              \
  if (head_dim == d && group == g)                                                      \
    return two ? launch_tc<QF, Mxfp4, d, g, 2>(a, cache, max_query_len, stream)         \
               : launch_tc<QF, Mxfp4, d, g, 1>(a, cache, max_query_len, stream);
#define PAGED_TC_ALL(QF)                                                                \
  PAGED_TC(QF, 64, 1) PAGED_TC(QF, 64, 2) PAGED_TC(QF, 64, 4) PAGED_TC(QF, 64, 8)       \
  PAGED_TC(QF, 128, 1) PAGED_TC(QF, 128, 2) PAGED_TC(QF, 128, 4) PAGED_TC(QF, 128, 8)
  if (q_dtype == kF16) {
    PAGED_TC_ALL(F16)
  } else if (q_dtype == kBF16) {
    PAGED_TC_ALL(BF16)
  }
#undef PAGED_TC_ALL
#undef PAGED_TC
  return cudaErrorNotSupported;
}

}  // namespace paged
