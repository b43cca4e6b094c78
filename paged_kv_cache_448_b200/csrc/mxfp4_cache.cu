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
// Both move 2 + 17/32 bytes an element and nothing else: memory bound. One
// thread takes 8 elements (16 bytes of the row) of K and of V; the 4 threads
// of a block share their maxima by two shuffles, and a warp writes whole rows.
#include "decode_args.h"
#include "device_common.cuh"
#include "mxfp4.cuh"

namespace paged {
namespace {

constexpr int kThreads = 256;

// Where the 8 elements of thread i sit: token n and slot, and the element
// offset of the cache row's chunk.
struct Place {
  int64_t n, row, slot;  // token, cache row ((block * hkv + head) * block_size + offset), slot
  int chunk;             // 8-element chunk of the row
};

template <int D>
__device__ __forceinline__ Place place(int64_t i, const int32_t* slots, int32_t hkv,
                                       int32_t block_size) {
  constexpr int CPR = D / 8;
  Place p;
  const int64_t per_token = static_cast<int64_t>(hkv) * CPR;
  p.n = i / per_token;
  const int r = static_cast<int>(i - p.n * per_token);
  const int h = r / CPR;
  p.chunk = r % CPR;
  p.slot = slots[p.n];
  const int64_t blk = p.slot / block_size;
  p.row = (blk * hkv + h) * block_size + p.slot % block_size;
  return p;
}

template <class F>
__device__ __forceinline__ void write_chunk(uint4 x, uint8_t* codes, uint8_t* scales, int64_t row,
                                            int chunk, int row_chunks, bool store) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float v[8], amax = 0.f;
  bool bad = false;  // fmaxf passes over a NaN, so it is looked for
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = cvt2(F{}, w[j]);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
    bad |= f.x != f.x || f.y != f.y;
    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  if (bad) amax = CUDART_INF_F;
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int b = mx_scale_byte(amax);
  uint32_t code = 0u;  // a block that is not finite: NaN scale, zero codes
  if (b != kMxNan) {
    const float s = mx_inverse(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s;
    code = mx_pack8(v);
  }
  if (!store) return;
  reinterpret_cast<uint32_t*>(codes)[row * row_chunks + chunk] = code;
  if (chunk % 4 == 0) scales[row * (row_chunks / 4) + chunk / 4] = static_cast<uint8_t>(b);
}

template <class F, int D>
__global__ void __launch_bounds__(kThreads)
    mxfp4_write_kernel(const uint4* __restrict__ key, const uint4* __restrict__ value,
                       uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                       uint8_t* __restrict__ ks, uint8_t* __restrict__ vs,
                       const int32_t* __restrict__ slots, int64_t total, int32_t hkv,
                       int32_t block_size, int64_t pool_slots) {
  // the next kernel may be scheduled now; one that reads the cache waits for
  // this grid's completion before it does
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  // whole warps stay for the shuffles; total is a multiple of D / 8 threads
  const bool in = i < total;
  const Place p = place<D>(in ? i : 0, slots, hkv, block_size);
  const bool store = in && p.slot >= 0 && p.slot < pool_slots;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 k = store ? key[i] : zero, v = store ? value[i] : zero;
  write_chunk<F>(k, kc, ks, p.row, p.chunk, D / 8, store);
  write_chunk<F>(v, vc, vs, p.row, p.chunk, D / 8, store);
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
    if constexpr (F::kIsBf16) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(f.x * s, f.y * s);
      o[j] = *reinterpret_cast<const uint32_t*>(&t);
    } else {
      const __half2 t = __floats2half2_rn(f.x * s, f.y * s);
      o[j] = *reinterpret_cast<const uint32_t*>(&t);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct OutF16 {
  static constexpr bool kIsBf16 = false;
};
struct OutBF16 {
  static constexpr bool kIsBf16 = true;
};

template <class F, int D>
__global__ void __launch_bounds__(kThreads)
    mxfp4_read_kernel(uint4* __restrict__ key, uint4* __restrict__ value,
                      const uint32_t* __restrict__ kc, const uint32_t* __restrict__ vc,
                      const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs,
                      const int32_t* __restrict__ slots, int64_t total, int32_t hkv,
                      int32_t block_size, int64_t pool_slots) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= total) return;
  const Place p = place<D>(i, slots, hkv, block_size);
  if (p.slot < 0 || p.slot >= pool_slots) return;
  constexpr int CPR = D / 8;
  const int64_t c = p.row * CPR + p.chunk, s = p.row * (CPR / 4) + p.chunk / 4;
  key[i] = read_chunk<F>(kc[c], ks[s]);
  value[i] = read_chunk<F>(vc[c], vs[s]);
}

}  // namespace

cudaError_t launch_mxfp4_write(const void* key, const void* value, uint8_t* kc, uint8_t* vc,
                               uint8_t* ks, uint8_t* vs, const int32_t* slots,
                               int32_t num_tokens, int32_t hkv, int32_t head_dim,
                               int32_t block_size, int64_t num_blocks, int kv_dtype,
                               cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(num_tokens) * hkv * (head_dim / 8);
  const unsigned grid = static_cast<unsigned>((total + kThreads - 1) / kThreads);
  auto k = static_cast<const uint4*>(key);
  auto v = static_cast<const uint4*>(value);
#define PAGED_W(F, d)                                                                        \
  mxfp4_write_kernel<F, d><<<grid, kThreads, 0, stream>>>(k, v, kc, vc, ks, vs, slots, total, \
                                                          hkv, block_size,                   \
                                                          num_blocks * block_size)
  if (kv_dtype == kF16 && head_dim == 64) PAGED_W(F16, 64);
  else if (kv_dtype == kF16) PAGED_W(F16, 128);
  else if (head_dim == 64) PAGED_W(BF16, 64);
  else PAGED_W(BF16, 128);
#undef PAGED_W
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_read(void* key, void* value, const uint8_t* kc, const uint8_t* vc,
                              const uint8_t* ks, const uint8_t* vs, const int32_t* slots,
                              int32_t num_tokens, int32_t hkv, int32_t head_dim,
                              int32_t block_size, int64_t num_blocks, int kv_dtype,
                              cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(num_tokens) * hkv * (head_dim / 8);
  const unsigned grid = static_cast<unsigned>((total + kThreads - 1) / kThreads);
  auto k = static_cast<uint4*>(key);
  auto v = static_cast<uint4*>(value);
  auto kw = reinterpret_cast<const uint32_t*>(kc);
  auto vw = reinterpret_cast<const uint32_t*>(vc);
  const int64_t pool = num_blocks * block_size;
#define PAGED_R(F, d)                                                                   \
  mxfp4_read_kernel<F, d><<<grid, kThreads, 0, stream>>>(k, v, kw, vw, ks, vs, slots, total, \
                                                         hkv, block_size, pool)
  if (kv_dtype == kF16 && head_dim == 64) PAGED_R(OutF16, 64);
  else if (kv_dtype == kF16) PAGED_R(OutF16, 128);
  else if (head_dim == 64) PAGED_R(OutBF16, 64);
  else PAGED_R(OutBF16, 128);
#undef PAGED_R
  return cudaGetLastError();
}

}  // namespace paged
