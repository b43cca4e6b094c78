// mxfp4_cache.cu — writing new K/V rows into a 4-bit (MXFP4) cache, and
// reading rows back as 16-bit values.
//
// Write: for each 32-element block of a row, amax = max |x|,
//   b = clamp(floor(log2 amax) - 2, -126, 125) + 127   (255 if amax is not finite)
//   code_i = E2M1(x_i * 2^(127 - b)), nearest even, saturating at 6
// (OCP Microscaling v1.0, the conversion to MXFP4; the product with a power of
// two is exact, so the result does not depend on the arithmetic's width).
// Read: x_i = code_i * 2^(b - 127), rounded to the row's type (exact within
// its range).
//
// Both move 2 + 17/32 bytes an element and nothing else: memory bound. A write
// thread takes one block of K and of V (32 elements, eight 16-byte loads in
// flight): the maximum needs no exchange between lanes, and the indices and the
// scale are worked out once per 32 elements (with 8 elements a thread and two
// shuffles the instructions bound it: 8 191 tokens of 32 heads written in 44 us
// and read in 34; now 23 and 24, 55 with both launches). The 16-bit rows pass
// through the caches as streams (58 us without the hints). A read
// thread takes 8 elements of four rows' chunks, so that a warp's stores are
// whole lines.
#include <algorithm>
#include <type_traits>

#include "decode_args.h"
#include "device_common.cuh"
#include "mxfp4.cuh"

namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxRows = 1 << 24;  // rows (token, head) of a launch at most: 31-bit indices

// n / d for 0 <= n < 2^31 as (n * mul) >> shift.
struct FastDiv {
  uint32_t mul, shift;
};

__device__ __forceinline__ uint32_t fast_div(uint32_t n, FastDiv f) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * f.mul) >> f.shift);
}

struct RowArgs {
  const int32_t* slots;  // of the launch's first token
  uint32_t rows;         // tokens x heads
  uint32_t hkv;
  FastDiv by_hkv;
  int32_t bs_log;
  int64_t pool_slots;
};

// Cache row of (token, head) row r, or -1 where its slot is not in the pool.
__device__ __forceinline__ int64_t cache_row(const RowArgs& a, uint32_t r) {
  const uint32_t n = fast_div(r, a.by_hkv), h = r - n * a.hkv;
  const int32_t slot = a.slots[n];
  if (slot < 0 || slot >= a.pool_slots) return -1;
  const int32_t bs = 1 << a.bs_log;
  return ((static_cast<int64_t>(slot >> a.bs_log) * a.hkv + h) << a.bs_log) + (slot & (bs - 1));
}

// Larger magnitudes of two pairs; a NaN goes through.
__device__ __forceinline__ uint32_t max_abs2(F16, uint32_t m, uint32_t x) {
  x &= 0x7fff7fffu;
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&m),
                                *reinterpret_cast<const __half2*>(&x));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_abs2(BF16, uint32_t m, uint32_t x) {
  x &= 0x7fff7fffu;
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                       *reinterpret_cast<const __nv_bfloat162*>(&x));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One block of 32 elements -> 16 bytes of codes and the scale byte.
template <class F>
__device__ __forceinline__ void write_block(const uint4 (&x)[4], uint8_t* codes, uint8_t* scale) {
  const uint32_t w[16] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w,
                          x[2].x, x[2].y, x[2].z, x[2].w, x[3].x, x[3].y, x[3].z, x[3].w};
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = max_abs2(F{}, m, w[j]);
  const float2 mm = cvt2(F{}, m);
  // fmaxf passes over a NaN: as bits it is above infinity
  const float amax = __uint_as_float(max(__float_as_uint(mm.x) & 0x7fffffffu,
                                         __float_as_uint(mm.y) & 0x7fffffffu));
  const int b = mx_scale_byte(amax);
  uint32_t c[4] = {0u, 0u, 0u, 0u};  // a block that is not finite: NaN scale, zero codes
  if (b != kMxNan) {
    const float s = mx_inverse(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = cvt2(F{}, w[4 * i + j]);
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      c[i] = mx_pack8(v);
    }
  }
  *reinterpret_cast<uint4*>(codes) = make_uint4(c[0], c[1], c[2], c[3]);
  *scale = static_cast<uint8_t>(b);
}

template <class F, int D>
__global__ void __launch_bounds__(kThreads)
    mxfp4_write_kernel(const uint4* __restrict__ key, const uint4* __restrict__ value,
                       uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                       uint8_t* __restrict__ ks, uint8_t* __restrict__ vs, const RowArgs a) {
  // the next kernel may be scheduled now; one that reads the cache waits for
  // this grid's completion before it does
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int NB = D / 32;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x, r = i / NB;
  if (r >= a.rows) return;
  const int64_t row = cache_row(a, r);
  if (row < 0) return;
  uint4 k[4], v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    k[j] = __ldcs(key + static_cast<int64_t>(i) * 4 + j);
    v[j] = __ldcs(value + static_cast<int64_t>(i) * 4 + j);
  }
  const int64_t at = row * NB + i % NB;
  write_block<F>(k, kc + at * 16, ks + at);
  write_block<F>(v, vc + at * 16, vs + at);
}

template <class F>
__device__ __forceinline__ uint4 read_chunk(uint32_t code, int b) {
  uint32_t h[4];
  mx_unpack8(code, h);
  const float s = mx_scale(b);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = cvt2(F16{}, h[j]);
    if constexpr (std::is_same<F, BF16>::value) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(f.x * s, f.y * s);
      o[j] = *reinterpret_cast<const uint32_t*>(&t);
    } else {
      const __half2 t = __floats2half2_rn(f.x * s, f.y * s);
      o[j] = *reinterpret_cast<const uint32_t*>(&t);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int kReadChunks = 4;  // 8-element chunks of K and of V per read thread

template <class F, int D>
__global__ void __launch_bounds__(kThreads)
    mxfp4_read_kernel(uint4* __restrict__ key, uint4* __restrict__ value,
                      const uint32_t* __restrict__ kc, const uint32_t* __restrict__ vc,
                      const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs,
                      const RowArgs a) {
  constexpr int CPR = D / 8;
  const uint32_t i0 = blockIdx.x * (kThreads * kReadChunks) + threadIdx.x;
  uint32_t kw[kReadChunks], vw[kReadChunks];
  int kb[kReadChunks], vb[kReadChunks];
  bool real[kReadChunks];
#pragma unroll
  for (int j = 0; j < kReadChunks; ++j) {
    const uint32_t i = i0 + j * kThreads, r = i / CPR, chunk = i % CPR;
    const int64_t row = r < a.rows ? cache_row(a, r) : -1;
    real[j] = row >= 0;
    if (!real[j]) continue;
    const int64_t c = row * CPR + chunk, s = row * (CPR / 4) + chunk / 4;
    kw[j] = kc[c];
    vw[j] = vc[c];
    kb[j] = ks[s];
    vb[j] = vs[s];
  }
#pragma unroll
  for (int j = 0; j < kReadChunks; ++j) {
    if (!real[j]) continue;
    const int64_t i = i0 + j * kThreads;
    __stcs(key + i, read_chunk<F>(kw[j], kb[j]));
    __stcs(value + i, read_chunk<F>(vw[j], vb[j]));
  }
}

FastDiv make_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

// Calls launch(args, first token) for ranges of tokens of at most kMaxRows rows.
template <class L>
cudaError_t for_token_ranges(const int32_t* slots, int32_t num_tokens, int32_t hkv,
                             int32_t block_size, int64_t num_blocks, L launch) {
  const int32_t step = std::max(1, kMaxRows / hkv);
  for (int32_t n = 0; n < num_tokens; n += step) {
    const int32_t count = std::min(step, num_tokens - n);
    const RowArgs a{slots + n, static_cast<uint32_t>(count) * hkv, static_cast<uint32_t>(hkv),
                    make_div(hkv), block_size == 32 ? 5 : 4, num_blocks * block_size};
    launch(a, n);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (num_tokens - n <= step) break;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_mxfp4_write(const void* key, const void* value, uint8_t* kc, uint8_t* vc,
                               uint8_t* ks, uint8_t* vs, const int32_t* slots,
                               int32_t num_tokens, int32_t hkv, int32_t head_dim,
                               int32_t block_size, int64_t num_blocks, int kv_dtype,
                               cudaStream_t stream) {
  return for_token_ranges(slots, num_tokens, hkv, block_size, num_blocks, [&](const RowArgs& a,
                                                                              int32_t first) {
    const int64_t at = static_cast<int64_t>(first) * hkv * (head_dim / 8);
    auto k = static_cast<const uint4*>(key) + at;
    auto v = static_cast<const uint4*>(value) + at;
    const unsigned grid = (a.rows * (head_dim / 32) + kThreads - 1) / kThreads;
#define PAGED_W(F, d) mxfp4_write_kernel<F, d><<<grid, kThreads, 0, stream>>>(k, v, kc, vc, ks, vs, a)
    if (kv_dtype == kF16 && head_dim == 64) PAGED_W(F16, 64);
    else if (kv_dtype == kF16) PAGED_W(F16, 128);
    else if (head_dim == 64) PAGED_W(BF16, 64);
    else PAGED_W(BF16, 128);
#undef PAGED_W
  });
}

cudaError_t launch_mxfp4_read(void* key, void* value, const uint8_t* kc, const uint8_t* vc,
                              const uint8_t* ks, const uint8_t* vs, const int32_t* slots,
                              int32_t num_tokens, int32_t hkv, int32_t head_dim,
                              int32_t block_size, int64_t num_blocks, int kv_dtype,
                              cudaStream_t stream) {
  auto kw = reinterpret_cast<const uint32_t*>(kc);
  auto vw = reinterpret_cast<const uint32_t*>(vc);
  return for_token_ranges(slots, num_tokens, hkv, block_size, num_blocks, [&](const RowArgs& a,
                                                                              int32_t first) {
    const int64_t at = static_cast<int64_t>(first) * hkv * (head_dim / 8);
    auto k = static_cast<uint4*>(key) + at;
    auto v = static_cast<uint4*>(value) + at;
    constexpr unsigned kPer = kThreads * kReadChunks;
    const unsigned grid = (a.rows * (head_dim / 8) + kPer - 1) / kPer;
#define PAGED_R(F, d) mxfp4_read_kernel<F, d><<<grid, kThreads, 0, stream>>>(k, v, kw, vw, ks, vs, a)
    if (kv_dtype == kF16 && head_dim == 64) PAGED_R(F16, 64);
    else if (kv_dtype == kF16) PAGED_R(F16, 128);
    else if (head_dim == 64) PAGED_R(BF16, 64);
    else PAGED_R(BF16, 128);
#undef PAGED_R
  });
}

}  // namespace paged
