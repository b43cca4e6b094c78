// decode_mxfp4.cu — decode over a 4-bit (MXFP4) paged cache.
//
// For each (sequence, query head): out = sum_t softmax_t(scale q . K_t) V_t
// over the context, K_t and V_t being code * 2^(b - 127) per 32-element block
// (mxfp4.cuh). One CTA per (kv-head, sequence, partition); each warp owns
// every NW-th step of 32 tokens and streams it through its own ring of
// shared-memory stages with 16-byte asynchronous copies (136 bytes a token and
// kv-head at head_dim 128; one block and head is 1 KB of codes). Plain copies
// and not TMA boxes: a step has eight boxes (K and V, codes and scales, two
// blocks), whose issue took an eighth of the instructions, and a launch
// encodes no tensor maps. A warp waits for its own copies alone, which always
// complete: nothing here can run out of time.
//
// Arithmetic on a step, per warp, on mma.sync m16n8k16 (f16 in, fp32
// accumulators) with the tokens (S) or the dims (O) on M and the group's
// query heads on N:
//  * ldmatrix hands lane (g, c) [g = lane / 4, c = lane % 4] word c of the 16
//    bytes a block of token g has: 8 codes, dims 32 b + 8 c .. + 7. One
//    conversion instruction per byte makes the f16 pair that A wants (every
//    E2M1 value is an f16 value). The contraction order within a block is
//    permuted to match, in the query fragments too, and every MMA stays inside
//    one block, so the block's scale is applied to the fp32 partial sums:
//      S[t, h] = sum_b 2^(bK[t, b] - 127) (codes . q)_b.
//  * ldmatrix.trans of the same bytes gives lane (g, c) the codes of dims
//    32 b + 4 g .. + 3 for tokens 2 c and 2 c + 1, the A operand of V^T P once
//    the two tokens' codes are interleaved. The V scale belongs to the
//    contracted index, so it multiplies P, per block of dims:
//      O[d, h] += V~[t, d] (P[t, h] 2^(bV[t, b(d)] - r_b)),
//    r_b being a running reference for the block's scales (undone at the end)
//    that keeps the product within f16.
// P and O follow a base-2 online softmax whose maximum m moves only when a
// logit passes it by more than 8, so P <= 2^8; r_b moves only when a scale
// passes it by more than 7, so P 2^(bV - r_b) <= 2^15 < 65504. Scales more
// than 8 below r_b would lose P's low bits, or all of it: a step that holds
// one takes its tokens band by band (15 powers of two each, relative to the
// band's largest scale) and adds the bands in fp32. All three conditions are
// checked with one vote per step; the slow paths run a few times a unit.
// A probability is rounded to f16 (2^-12 relative) before the product with V;
// sums, maxima, logits and O are fp32.
// A bf16 query row is scaled by a power of two that puts its largest element
// in [1, 2) and held in f16: exact for elements down to 2^-17 of the largest,
// an error of at most 2^-25 of it below.
//
// Not bound by memory, and by no unit that is full: a step of 32 tokens takes
// 650 (850 with MxState) instructions a warp, of which the conversions are 128,
// and with the 16 warps an SM that 128 registers a thread leave, dependent
// chains keep 57 (61) % of the issue slots and 64 % of the integer pipe busy.
// On a B200, 32 sequences of 2 030 tokens with 32 heads, f16: 68 us, 4.15 TB/s
// of codes and scales (an E4M3 cache 90 us, 16 bit 155); 24 sequences of 1 024
// to 32 768 tokens, 64 query heads on 8, bf16: 89 us (141 and 153).
#include <math_constants.h>

#include <type_traits>

#include "consumer_mma.cuh"
#include "decode_args.h"
#include "decode_kernel.cuh"
#include "device_common.cuh"
#include "mxfp4.cuh"

namespace paged {
namespace {

constexpr int kStep = 32;  // tokens per step

template <int D_, int NW_>
struct MxCfg {
  static constexpr int D = D_, NW = NW_;
  static constexpr int RB = D / 2;                    // code bytes of a row
  static constexpr int SB = D / 32;                   // scale bytes of a row = blocks
  static constexpr int CODES = kStep * RB;            // K (or V) codes of a step
  static constexpr int SCALES = kStep * SB;           // K (or V) scales of a step
  static constexpr int SWZ = RB == 64 ? 0x30 : 0x10;  // 16-byte chunks of a row XOR its number / 2 (4)
  static constexpr int R = 2;                         // stages of a warp's ring
  static constexpr int STAGE = 2 * CODES + 2 * SCALES;  // K codes, V codes, K scales, V scales
  static constexpr int OFF_IDS = NW * R * STAGE;
  static_assert(NW * 8 * (D + 1) * 4 + NW * 16 * 4 <= OFF_IDS, "merge buffer fits");
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit values held one pair a lane.
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float fast_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^n, 0 below the normal numbers.
__device__ __forceinline__ float pow2i(int n) {
  return n < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
}

// e such that mq 2^e lies in [1, 2) (2^e and 2^-e normal numbers; 0 for a row
// of zeros or one that is not finite).
__device__ __forceinline__ int row_exponent(float mq) {
  const int field = static_cast<int>(__float_as_uint(mq) >> 23);
  return mq > 0.f && field < 255 ? min(max(127 - field, -126), 126) : 0;
}

// Each 16-bit half v of x where lo <= v <= hi, the other halves as 0.
__device__ __forceinline__ uint32_t halves_within(uint32_t x, int lo, int hi) {
  const int a = static_cast<int>(x & 0xffffu), b = static_cast<int>(x >> 16);
  return (a >= lo && a <= hi ? x & 0x0000ffffu : 0u) | (b >= lo && b <= hi ? x & 0xffff0000u : 0u);
}

// f16 of 2^(v - r) for each 16-bit half v of x, r - 14 <= v <= r + 15: its
// exponent field is v - r + 15 (exact in integer arithmetic on the word).
__device__ __forceinline__ uint32_t f16_pow2(uint32_t x, int r) {
  return x * 0x400u + static_cast<uint32_t>(15 - r) * 0x04000400u;
}

// f16 of 2^(v - r) for the halves v of x with max(r - 14, 1) <= v <= r, 0 for the others.
__device__ __forceinline__ uint32_t band_pow2(uint32_t x, int r) {
  const uint32_t in = halves_within(x, max(r - 14, 1), r);
  const uint32_t keep = ((in & 0xffffu) ? 0x0000ffffu : 0u) | ((in >> 16) ? 0xffff0000u : 0u);
  // the halves left out take the value r first: no carry into the other half
  return f16_pow2(in | (static_cast<uint32_t>(r) * 0x10001u & ~keep), r) & keep;
}

// The halves v of x with max(r - 8, 1) <= v <= r + 7 as they are, the others
// such that f16_pow2 gives 0 (a scale byte of 0 reads as 0).
__device__ __forceinline__ uint32_t window_only(uint32_t x, int r) {
  const int a = static_cast<int>(x & 0xffffu), b = static_cast<int>(x >> 16);
  const int lo = max(r - 8, 1), hi = r + 7;
  return static_cast<uint32_t>(b >= lo && b <= hi ? b : r - 15) * 0x10000u +
         static_cast<uint32_t>(a >= lo && a <= hi ? a : r - 15);
}

// m's bits of x, the others of y.
__device__ __forceinline__ uint32_t bit_select(uint32_t m, uint32_t x, uint32_t y) {
  return ((x ^ y) & m) ^ y;
}

// One word of V codes as ldmatrix.trans gives it (dims 4 g .. + 3 of tokens
// 2 c, 2 c + 1) -> per dim the f16 pair of the two tokens.
__device__ __forceinline__ void v_pairs(uint32_t w, uint32_t (&h)[4]) {
  // bytes: (token 2c, token 2c + 1) codes of dims 0, 2, 1, 3
  const uint32_t x =
      bit_select(0x0f0f0000u, w << 12, bit_select(0xf0f00f0fu, w, w >> 12));
  uint32_t t[4];
  mx_unpack8(x, t);
  h[0] = t[0];
  h[2] = t[1];
  h[1] = t[2];
  h[3] = t[3];
}

// Codes of rows 16 u .. + 15 of a staged tile: per 8 rows i one word a block.
// K (trans false): lane (g, c) gets word c of row 8 i + g; V: transposed.
template <int D, int SWZ, bool TRANS>
__device__ __forceinline__ void load_codes(const uint8_t* tile, int u, int lane,
                                           uint32_t (&r)[2][D / 32]) {
  constexpr int RB = D / 2;
  auto ld = [](const uint8_t* p, uint32_t (&x)[4]) {
    if constexpr (TRANS) ldsm_x4_trans(p, x);
    else ldsm_x4(p, x);
  };
  if constexpr (D == 128) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int off = (16 * u + 8 * i + (lane & 7)) * RB + (lane >> 3) * 16;
      ld(tile + (off ^ ((off >> 3) & SWZ)), r[i]);
    }
  } else {
    uint32_t t[4];
    const int off = (16 * u + 8 * (lane >> 4) + (lane & 7)) * RB + ((lane >> 3) & 1) * 16;
    ld(tile + (off ^ ((off >> 3) & SWZ)), t);
    r[0][0] = t[0];
    r[0][1] = t[1];
    r[1][0] = t[2];
    r[1][1] = t[3];
  }
}

// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The attention state of one warp: query heads 2c and 2c+1 of lane (g, c),
// tokens shared out over g.
template <class QF, int D>
struct MxState {
  static constexpr int NB = D / 32;  // blocks of a row
  uint32_t q[NB][4];   // query fragments: block b, k-step i: q[b][2 i], q[b][2 i + 1]
  float qs[2];         // base-2 logit scale of the two heads
  float m[2], l[2];    // running maximum; this lane's part of the sum
  float o[NB][2][4];   // O: block b, dims 32 b + 4 g + 2 i (+1) x heads 2c, 2c+1
  int ref[NB];         // r_b: scale byte the V scales are taken relative to (-1: none yet)
  uint32_t nan_blocks; // blocks of V with a NaN scale in the context
  bool low;            // a reference so low that the window below it holds the byte 0
  uint32_t off;        // added to a row's scale bytes: 0x80 .. 0x8f within the window

  __device__ __forceinline__ void init(const DecodeArgs& a, const uint8_t* query, int group,
                                       int lane) {
    const int g = lane >> 2, c = lane & 3;
    const uint4* row = reinterpret_cast<const uint4*>(query + static_cast<int64_t>(g) * D * 2);
    uint4 w[NB];
    float mq = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      w[b] = g < group ? row[b * 4 + c] : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (std::is_same<QF, BF16>::value) {
        const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = cvt2(BF16{}, x[j]);
          mq = fmaxf(mq, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
    }
    int e = 0;  // power of two of this row (head g)
    if constexpr (std::is_same<QF, BF16>::value) {
      mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 1));
      mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 2));
      e = row_exponent(mq);
    }
    const float up = pow2i(e);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (std::is_same<QF, BF16>::value) {
          const float2 f = cvt2(BF16{}, x[j]);
          const __half2 h = __floats2half2_rn(f.x * up, f.y * up);
          q[b][j] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          q[b][j] = x[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int eh = __shfl_sync(0xffffffffu, e, (2 * c + i) * 4);
      qs[i] = a.scale_log2 * pow2i(-eh);
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      ref[b] = -1;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[b][i][j] = 0.f;
    }
    nan_blocks = 0u;
    low = true;
    off = 0u;
  }

  // The NB scale bytes of a row.
  static __device__ __forceinline__ uint32_t scale_word(const uint8_t* p) {
    if constexpr (NB == 4) return *reinterpret_cast<const uint32_t*>(p);
    return *reinterpret_cast<const uint16_t*>(p);
  }
  static __device__ __forceinline__ int byte_of(uint32_t w, int b) { return (w >> (8 * b)) & 255; }

  // One step: kStep rows of codes at kc / vc (swizzled), scales at ks / vs;
  // if PARTIAL, rows from `valid` on are not of the context and may hold
  // anything (a copy of its own: masks would cost every step a tenth).
  template <int SWZ, bool PARTIAL>
  __device__ __forceinline__ void step(const uint8_t* kc, const uint8_t* vc, const uint8_t* ks,
                                       const uint8_t* vs, int valid, int lane) {
    constexpr int SB = NB;
    constexpr unsigned FULL = 0xffffffffu;
    const int g = lane >> 2, c = lane & 3;
    // ---- logits: x[u][i][j] = token 16 u + 8 i + g, head 2 c + j
    float x[2][2][2];
    uint32_t ff = 0u;  // a K scale of 255 among this lane's tokens
    uint32_t kw[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t r[2][NB];  // [rows g / g + 8][block]
      load_codes<D, SWZ, false>(kc, u, lane, r);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        kw[u][i] = scale_word(ks + (16 * u + 8 * i + g) * SB);
        if (PARTIAL && 16 * u + 8 * i + g >= valid) kw[u][i] = 0u;
        ff |= has_ff(kw[u][i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) x[u][i][j] = 0.f;
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t h0[4], h1[4];
        mx_unpack8(r[0][b], h0);
        mx_unpack8(r[1][b], h1);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816(s, h0[0], h1[0], h0[1], h1[1], q[b][0], q[b][1]);
        mma16816(s, h0[2], h1[2], h0[3], h1[3], q[b][2], q[b][3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f =
              __uint_as_float((b == 3 ? kw[u][i] >> 1 : kw[u][i] << (23 - 8 * b)) & 0x7f800000u);
          x[u][i][0] = fmaf(f, s[2 * i], x[u][i][0]);
          x[u][i][1] = fmaf(f, s[2 * i + 1], x[u][i][1]);
        }
      }
    }
    // ---- scales of V: words of tokens 16 u + 8 i + 2 c, + 1
    uint32_t vw[2][2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* p = vs + (16 * u + 8 * i + 2 * c) * SB;
        if constexpr (NB == 4) {
          const uint2 t = *reinterpret_cast<const uint2*>(p);
          vw[u][i][0] = t.x;
          vw[u][i][1] = t.y;
        } else {
          const uint32_t t = *reinterpret_cast<const uint32_t*>(p);
          vw[u][i][0] = t & 0xffffu;
          vw[u][i][1] = t >> 16;
        }
      }
    float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = x[u][i][j] * qs[j];
          if (PARTIAL && 16 * u + 8 * i + g >= valid) t = -CUDART_INF_F;
          x[u][i][j] = t;
          mx[j] = fmaxf(mx[j], t);
        }
    if constexpr (PARTIAL) {  // rows that are not of the context: scales within the window
      uint32_t in = 0u;
#pragma unroll
      for (int b = 0; b < NB; ++b) in |= static_cast<uint32_t>(max(ref[b], 1)) << (8 * b);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (16 * u + 8 * i + 2 * c + j >= valid) vw[u][i][j] = in;
    }
    const bool lift = mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f || outside(vw) || ff ||
                      (low && far_above(vw));
    bool wide = low;  // V scales below the window (the same in every lane)
    if (__any_sync(FULL, lift)) {
      update(x, mx, kw, ff, vw);
      wide = low || __any_sync(FULL, outside(vw));
    }
    // ---- probabilities, their sum, and P as B operand (tokens x heads)
    const float mu0 = m[0] == -CUDART_INF_F ? 0.f : m[0];
    const float mu1 = m[1] == -CUDART_INF_F ? 0.f : m[1];
    uint32_t p[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float p0 = fast_ex2(x[u][i][0] - mu0), p1 = fast_ex2(x[u][i][1] - mu1);
        l[0] += p0;
        l[1] += p1;
        const __half2 h = __floats2half2_rn(p0, p1);
        p[u][i] = movm_trans(*reinterpret_cast<const uint32_t*>(&h));
      }
    if (wide) {  // the bands below the window; those tokens weigh nothing after this
      bands<SWZ>(vc, p, vw, lane);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t w = 0u;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const int v = byte_of(vw[u][i][j], b);
              const bool in = v >= max(ref[b] - 8, 1) && v <= ref[b] + 7;
              w |= static_cast<uint32_t>(in ? v : (ref[b] - 15) & 31) << (8 * b);  // factor 0
            }
            vw[u][i][j] = w;
          }
    }
    // ---- O += V^T (P 2^(bV - r))
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t r[2][NB];
      load_codes<D, SWZ, true>(vc, u, lane, r);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t f0 = factor(vw[u][0], b), f1 = factor(vw[u][1], b);
        uint32_t h[2][4];
        v_pairs(r[0][b], h[0]);
        v_pairs(r[1][b], h[1]);
        const uint32_t b0 = hmul2u(p[u][0], f0), b1 = hmul2u(p[u][1], f1);
        mma16816(o[b][0], h[0][0], h[0][1], h[1][0], h[1][1], b0, b1);
        mma16816(o[b][1], h[0][2], h[0][3], h[1][2], h[1][3], b0, b1);
      }
    }
  }

  // Nonzero if some V scale of the step is not within [r_b - 8, r_b + 7] of its
  // block's reference: whole words of scales at once. w + off has an upper
  // nibble of 8 in every byte when every byte is within its window, and not in
  // the lowest one that is outside it, but for a byte so far above that the sum
  // runs through to the nibble again: r_b + 248 and more. Those need r_b <= 7
  // (low is set then) and are what far_above finds.
  __device__ __forceinline__ uint32_t outside(const uint32_t (&vw)[2][2][2]) const {
    uint32_t bits = 0u;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) bits |= (vw[u][i][j] + off) ^ 0x80808080u;
    return bits & (NB == 4 ? 0xf0f0f0f0u : 0x0000f0f0u);
  }

  // Nonzero if some V scale of the step is 248 or more (NaN, 255, among them).
  static __device__ __forceinline__ uint32_t far_above(const uint32_t (&vw)[2][2][2]) {
    uint32_t bits = 0u;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) bits |= has_ff(vw[u][i][j] | 0x07070707u);
    return bits;
  }

  // The V scales of block b of two tokens (words w) as halves.
  static __device__ __forceinline__ uint32_t halves(const uint32_t (&w)[2], int b) {
    return prmt(w[0], w[1], static_cast<uint32_t>(b | (b + 4) << 8)) & 0x00ff00ffu;
  }

  // f16 of 2^(bV - r_b) for the two tokens, both within the window: the byte
  // twice in each half, so that no sum carries into the other; the five bits of
  // the exponent field are kept.
  __device__ __forceinline__ uint32_t factor(const uint32_t (&w)[2], int b) const {
    const uint32_t v = prmt(w[0], w[1], static_cast<uint32_t>(b * 0x11 | (b + 4) * 0x1100));
    return (v * 0x400u + static_cast<uint32_t>((15 - ref[b]) & 31) * 0x04000400u) & 0x7c007c00u;
  }

  // The step's tokens whose V scale lies below the window of its block: bands
  // of 15 powers of two from the largest such scale down, each a product of
  // its own added to O in fp32.
  template <int SWZ>
  __device__ __forceinline__ void bands(const uint8_t* vc, const uint32_t (&p)[2][2],
                                        const uint32_t (&vw)[2][2][2], int lane) {
    constexpr int RB = D / 2;
    constexpr unsigned FULL = 0xffffffffu;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      int hi = ref[b] - 9;
      while (hi > 0) {  // the same in every lane
        int t = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t in = halves_within(halves(vw[u][i], b), 1, hi);
            t = max(t, max(static_cast<int>(in & 0xffffu), static_cast<int>(in >> 16)));
          }
        t = max(t, __shfl_xor_sync(FULL, t, 1));
        t = max(t, __shfl_xor_sync(FULL, t, 2));
        if (t == 0) break;
        float add[2][4] = {};
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          // 16 rows x the 16 bytes of this block, transposed
          uint32_t r[4];
          const int off = (16 * u + (lane & 15)) * RB + b * 16;
          ldsm_x4_trans(vc + (off ^ ((off >> 3) & SWZ)), r);
          uint32_t h[2][4];
          v_pairs(r[0], h[0]);
          v_pairs(r[1], h[1]);
          const uint32_t e0 = u ? halves(vw[1][0], b) : halves(vw[0][0], b);
          const uint32_t e1 = u ? halves(vw[1][1], b) : halves(vw[0][1], b);
          const uint32_t p0 = u ? p[1][0] : p[0][0], p1 = u ? p[1][1] : p[0][1];
          const uint32_t b0 = hmul2u(p0, band_pow2(e0, t));
          const uint32_t b1 = hmul2u(p1, band_pow2(e1, t));
          mma16816(add[0], h[0][0], h[0][1], h[1][0], h[1][1], b0, b1);
          mma16816(add[1], h[0][2], h[0][3], h[1][2], h[1][3], b0, b1);
        }
        const float f = pow2i(t - ref[b]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[b][i][j] = fmaf(add[i][j], f, o[b][i][j]);
        hi = t - 15;
      }
    }
  }

  // The scale references move to the largest V scale of the step; a NaN scale
  // is remembered for its block.
  __device__ __forceinline__ void update_scales(uint32_t (&vw)[2][2][2]) {
    constexpr unsigned FULL = 0xffffffffu;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      int t = -1;
      bool bad = false;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int v = byte_of(vw[u][i][j], b);
            if (v == kMxNan) {
              bad = true;
              vw[u][i][j] &= ~(255u << (8 * b));  // as 0: no weight
            } else {
              t = max(t, v);
            }
          }
      t = max(t, __shfl_xor_sync(FULL, t, 1));
      t = max(t, __shfl_xor_sync(FULL, t, 2));
      if (__any_sync(FULL, bad)) nan_blocks |= 1u << b;
      t = min(t, 247);  // 248 .. 254 stay within the 7 powers of two above r_b
      if (t > ref[b]) {
        const float f = ref[b] < 0 ? 0.f : pow2i(ref[b] - t);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[b][i][j] *= f;
        ref[b] = t;
      }
    }
    low = false;
    off = NB == 4 ? 0x88888888u : 0x00008888u;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      low |= ref[b] <= 8;
      off -= static_cast<uint32_t>(ref[b]) << (8 * b);
    }
  }

  // A maximum or a scale reference has to move, or a scale is NaN (a K scale:
  // the token's logit is NaN for every head).
  __device__ __forceinline__ void update(float (&x)[2][2][2], float (&mx)[2],
                                         const uint32_t (&kw)[2][2], uint32_t ff,
                                         uint32_t (&vw)[2][2][2]) {
    constexpr unsigned FULL = 0xffffffffu;
    if (ff) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (has_ff(kw[u][i])) x[u][i][0] = x[u][i][1] = CUDART_NAN_F;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) mx[j] = fmaxf(mx[j], __shfl_xor_sync(FULL, mx[j], d));
      if (mx[j] > m[j]) {
        const float f = m[j] == -CUDART_INF_F ? 0.f : fast_ex2(m[j] - mx[j]);
        l[j] *= f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o[b][i][j] *= f;
            o[b][i][2 + j] *= f;
          }
        m[j] = mx[j];
      }
    }
    update_scales(vw);
  }

  // (m, l) of each head and O in true units to shared memory.
  __device__ __forceinline__ void finish(float* ml, float* ob, int group, int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[j] += __shfl_xor_sync(FULL, l[j], d);
      if (g == 0 && 2 * c + j < group) {
        ml[2 * (2 * c + j)] = m[j];
        ml[2 * (2 * c + j) + 1] = l[j];
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float f = nan_blocks >> b & 1 ? CUDART_NAN_F
                      : ref[b] <= 0       ? 0.f
                                          : pow2i(ref[b] - 127);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int head = 2 * c + j, dim = 32 * b + 4 * g + 2 * i + k;
            if (head < group) ob[head * D + dim] = o[b][i][2 * k + j] * f;
          }
    }
  }
};

// The same for kv-heads with few query heads (heads x blocks <= 8 columns of
// N): column n is block n % NB of query head n / NB. For S the column's query
// fragment is zero outside its block, so one chain of MMAs gives the partial
// sums of all blocks, and lane (g, c) applies two scales to its two columns;
// for O the column's P carries its block's scale, so a step needs one scaled P
// instead of one per block (of O's columns those of a tile's own block count).
// The scale work and the exponentials shrink by NB against MxState, where they
// are a third of a step's instructions.
template <class QF, int D>
struct MxStateN {
  static constexpr int NB = D / 32;
  uint32_t q[NB][4];    // query fragments of column g: zero but in its block
  float qs;             // base-2 logit scale of this lane's head (columns 2c, 2c+1)
  float m, l;           // running maximum; this lane's part of the sum
  float o[NB][2][4];    // O: block b, dims 32 b + 4 g + 2 i (+1) x columns 2c, 2c+1
  int ref[NB];          // r_b: scale byte the V scales are taken relative to (-1: none yet)
  int own;              // r_b of column g's block
  uint32_t nan_blocks;
  bool low;

  static __device__ __forceinline__ int head_of(int col) { return col / NB; }

  __device__ __forceinline__ void init(const DecodeArgs& a, const uint8_t* query, int group,
                                       int lane) {
    const int g = lane >> 2, c = lane & 3;
    const int hq = head_of(g), bq = g % NB;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4* row = reinterpret_cast<const uint4*>(query + static_cast<int64_t>(hq) * D * 2);
    const uint4 w = hq < group ? row[bq * 4 + c] : zero;
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
    int e = 0;  // power of two of this head's row
    if constexpr (std::is_same<QF, BF16>::value) {
      float mq = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = cvt2(BF16{}, x[j]);
        mq = fmaxf(mq, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
#pragma unroll
      for (int d = 1; d < 4 * NB; d *= 2) mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, d));
      e = row_exponent(mq);
      const float up = pow2i(e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = cvt2(BF16{}, x[j]);
        const __half2 h = __floats2half2_rn(f.x * up, f.y * up);
        x[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int j = 0; j < 4; ++j) q[b][j] = b == bq ? x[j] : 0u;
      ref[b] = -1;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[b][i][j] = 0.f;
    }
    const int eh = __shfl_sync(0xffffffffu, e, head_of(2 * c) * NB * 4);
    qs = a.scale_log2 * pow2i(-eh);
    m = -CUDART_INF_F;
    l = 0.f;
    own = -1;
    nan_blocks = 0u;
    low = true;
  }

  template <int SWZ, bool PARTIAL>
  __device__ __forceinline__ void step(const uint8_t* kc, const uint8_t* vc, const uint8_t* ks,
                                       const uint8_t* vs, int valid, int lane) {
    constexpr int SB = NB;
    constexpr unsigned FULL = 0xffffffffu;
    const int g = lane >> 2, c = lane & 3;
    // ---- logits: x[u][i] = token 16 u + 8 i + g, the head of columns 2c, 2c+1
    float x[2][2];
    float fs[2][2], top = 0.f;  // larger scale of the two columns: infinity for a byte of 255
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t r[2][NB];
      load_codes<D, SWZ, false>(kc, u, lane, r);
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t h0[4], h1[4];
        mx_unpack8(r[0][b], h0);
        mx_unpack8(r[1][b], h1);
        mma16816(s, h0[0], h1[0], h0[1], h1[1], q[b][0], q[b][1]);
        mma16816(s, h0[2], h1[2], h0[3], h1[3], q[b][2], q[b][3]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // the scale bytes of this lane's two columns
        uint32_t y = *reinterpret_cast<const uint16_t*>(ks + (16 * u + 8 * i + g) * SB +
                                                        (2 * c) % NB);
        if (PARTIAL && 16 * u + 8 * i + g >= valid) y = 0u;
        const float f0 = __uint_as_float((y << 23) & 0x7f800000u);
        const float f1 = __uint_as_float((y << 15) & 0x7f800000u);
        fs[u][i] = fmaxf(f0, f1);
        top = fmaxf(top, fs[u][i]);
        x[u][i] = fmaf(f0, s[2 * i], f1 * s[2 * i + 1]);
        if constexpr (NB == 4) x[u][i] += __shfl_xor_sync(FULL, x[u][i], 1);
      }
    }
    // ---- V scales of column g's block, tokens 16 u + 8 i + 2 c, + 1 as halves
    uint32_t ex[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* p = vs + (16 * u + 8 * i + 2 * c) * SB;
        const uint32_t b = g % NB;
        if constexpr (NB == 4) {
          const uint2 t = *reinterpret_cast<const uint2*>(p);
          ex[u][i] = prmt(t.x, t.y, b | (b + 4) << 8) & 0x00ff00ffu;
        } else {
          const uint32_t t = *reinterpret_cast<const uint32_t*>(p);
          ex[u][i] = prmt(t, 0u, b | (b + 2) << 8) & 0x00ff00ffu;
        }
      }
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t = x[u][i] * qs;
        if (PARTIAL && 16 * u + 8 * i + g >= valid) t = -CUDART_INF_F;
        x[u][i] = t;
        mx = fmaxf(mx, t);
      }
    if constexpr (PARTIAL) {  // rows that are not of the context: a scale within the window
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = valid - (16 * u + 8 * i + 2 * c);
          const uint32_t keep = t <= 0 ? 0u : t == 1 ? 0x0000ffffu : 0xffffffffu;
          ex[u][i] = (ex[u][i] & keep) | (static_cast<uint32_t>(max(own, 1)) * 0x10001u & ~keep);
        }
    }
    const bool lift = mx > m + 8.f || outside(ex) || top == CUDART_INF_F;
    bool wide = low;  // (the same in every lane)
    if (__any_sync(FULL, lift)) {
      update(x, mx, fs, ex, lane);
      wide = low || __any_sync(FULL, outside(ex));
    }
    // ---- probabilities, their sum, and P as B operand (tokens x columns)
    const float mu = m == -CUDART_INF_F ? 0.f : m;
    uint32_t p[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float e = fast_ex2(x[u][i] - mu);
        l += e;
        const __half2 h = __floats2half2_rn(e, e);
        p[u][i] = movm_trans(*reinterpret_cast<const uint32_t*>(&h));
      }
    if (wide) {  // the bands below the window; those tokens weigh nothing after this
      bands<SWZ>(vc, p, ex, lane);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) ex[u][i] = window_only(ex[u][i], own);
    }
    // ---- O += V^T (P 2^(bV - r))
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t r[2][NB];
      load_codes<D, SWZ, true>(vc, u, lane, r);
      const uint32_t b0 = hmul2u(p[u][0], f16_pow2(ex[u][0], own));
      const uint32_t b1 = hmul2u(p[u][1], f16_pow2(ex[u][1], own));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t h[2][4];
        v_pairs(r[0][b], h[0]);
        v_pairs(r[1][b], h[1]);
        mma16816(o[b][0], h[0][0], h[0][1], h[1][0], h[1][1], b0, b1);
        mma16816(o[b][1], h[0][2], h[0][3], h[1][2], h[1][3], b0, b1);
      }
    }
  }

  // Nonzero if a V scale of the step is not within [r_b - 8, r_b + 7].
  __device__ __forceinline__ uint32_t outside(const uint32_t (&ex)[2][2]) const {
    const uint32_t add = static_cast<uint32_t>(0x8000 + 8 - own) * 0x10001u;
    return (((ex[0][0] + add) ^ 0x80008000u) | ((ex[0][1] + add) ^ 0x80008000u) |
            ((ex[1][0] + add) ^ 0x80008000u) | ((ex[1][1] + add) ^ 0x80008000u)) &
           0xfff0fff0u;
  }

  // Tokens whose V scale lies below the window: bands of 15 powers of two per
  // block, from its largest such scale down (MxState::bands).
  template <int SWZ>
  __device__ __forceinline__ void bands(const uint8_t* vc, const uint32_t (&p)[2][2],
                                        const uint32_t (&ex)[2][2], int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    int hi = own - 9;
    for (;;) {
      int t = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t in = hi > 0 ? halves_within(ex[u][i], 1, hi) : 0u;
          t = max(t, max(static_cast<int>(in & 0xffffu), static_cast<int>(in >> 16)));
        }
      t = max(t, __shfl_xor_sync(FULL, t, 1));
      t = max(t, __shfl_xor_sync(FULL, t, 2));
      if (!__any_sync(FULL, t > 0)) break;
      float f[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int tb = __shfl_sync(FULL, t, b * 4);  // (column b is block b)
        f[b] = tb > 0 ? pow2i(tb - ref[b]) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t r[2][NB];
        load_codes<D, SWZ, true>(vc, u, lane, r);
        const uint32_t b0 = t > 0 ? hmul2u(p[u][0], band_pow2(ex[u][0], t)) : 0u;
        const uint32_t b1 = t > 0 ? hmul2u(p[u][1], band_pow2(ex[u][1], t)) : 0u;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t h[2][4];
          v_pairs(r[0][b], h[0]);
          v_pairs(r[1][b], h[1]);
          float add[2][4] = {};
          mma16816(add[0], h[0][0], h[0][1], h[1][0], h[1][1], b0, b1);
          mma16816(add[1], h[0][2], h[0][3], h[1][2], h[1][3], b0, b1);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[b][i][j] = fmaf(add[i][j], f[b], o[b][i][j]);
        }
      }
      hi = t > 0 ? t - 15 : 0;
    }
  }

  // MxState::update: maxima and references move, NaN scales are looked at.
  __device__ __forceinline__ void update(float (&x)[2][2], float mx, const float (&fs)[2][2],
                                         uint32_t (&ex)[2][2], int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    const int g = lane >> 2;
    // a NaN K scale of any column makes the token's logit NaN for every head
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t = fs[u][i];
        if constexpr (NB == 4) t = fmaxf(t, __shfl_xor_sync(FULL, t, 1));
        if (t == CUDART_INF_F) x[u][i] = CUDART_NAN_F;
      }
#pragma unroll
    for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, d));
    if (mx > m) {
      const float f = m == -CUDART_INF_F ? 0.f : fast_ex2(m - mx);
      l *= f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[b][i][j] *= f;
      m = mx;
    }
    // references
    int t = -1;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int v = (ex[u][i] >> (16 * j)) & 0xffff;
          if (v == kMxNan) {
            bad = true;
            ex[u][i] &= j ? 0x0000ffffu : 0xffff0000u;  // as 0: no weight
          } else {
            t = max(t, v);
          }
        }
    low = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bool mine = g % NB == b;
      if (__any_sync(FULL, mine && bad)) nan_blocks |= 1u << b;
      const int tb = min(__reduce_max_sync(FULL, mine ? t : -1), 247);  // (MxState::update_scales)
      if (tb > ref[b]) {
        const float f = ref[b] < 0 ? 0.f : pow2i(ref[b] - tb);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[b][i][j] *= f;
        ref[b] = tb;
      }
      low |= ref[b] <= 8;
      if (mine) own = ref[b];
    }
  }

  __device__ __forceinline__ void finish(float* ml, float* ob, int group, int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(FULL, l, d);
    const int head = head_of(2 * c);
    if (g == 0 && (2 * c) % NB == 0 && head < group) {
      ml[2 * head] = m;
      ml[2 * head + 1] = l;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float f = nan_blocks >> b & 1 ? CUDART_NAN_F
                      : ref[b] <= 0       ? 0.f
                                          : pow2i(ref[b] - 127);
      // the lanes and the column that hold this block's own
      if (head < group && (2 * c) % NB == (b & ~1)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            ob[head * D + 32 * b + 4 * g + 2 * i + k] = o[b][i][2 * k + (b & 1)] * f;
      }
    }
  }
};

// The planes of the cache: K codes, V codes, K scales, V scales.
struct MxPlanes {
  const uint8_t* p[4];
};

// Four CTAs (16 warps) per SM: 128 registers a thread; with five the state
// spills (32 x 32 heads x 2 030 tokens 82 us against 67), with three 75. (With
// four, MxStateN at head_dim 128 spills 30 bytes.)
template <class QF, int D, int NW, bool BLOCKS_ON_N>
__global__ void __launch_bounds__(NW * 32, 4)
    paged_decode_mxfp4_kernel(const DecodeArgs a, const MxPlanes planes) {
  using C = MxCfg<D, NW>;
  constexpr int R = C::R, RB = C::RB, SB = C::SB;
  extern __shared__ __align__(128) uint8_t smem[];
  int32_t* ids = reinterpret_cast<int32_t*>(smem + C::OFF_IDS);

  const int kvh = blockIdx.x, s = blockIdx.y, part = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.num_heads / a.num_kv_heads;
  // everything below reads what earlier kernels of the stream wrote
  asm volatile("griddepcontrol.wait;" ::: "memory");

  int ctx = a.context_lens[s];
  if (ctx > a.ctx_limit || ctx < 0) {
    if (threadIdx.x == 0 && part == 0) report(a.err, kErrContextClipped);
    ctx = ctx < 0 ? 0 : a.ctx_limit;
  }
  const int bs = a.block_size;
  const int nblk = (ctx + bs - 1) / bs;
  const int parts = nblk == 0 ? 1 : (nblk + a.partition_blocks - 1) / a.partition_blocks;
  if (part >= parts) return;
  const int b_begin = part * a.partition_blocks;
  const int nlocal = min(b_begin + a.partition_blocks, nblk) - b_begin;
  const int tokens = max(0, min(ctx, (b_begin + nlocal) * bs) - b_begin * bs);
  const int nsteps = (tokens + kStep - 1) / kStep;

  // block ids of this unit -> shared memory, validated once
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  for (int i = threadIdx.x; i < nlocal; i += NW * 32) {
    int32_t id = table[b_begin + i];
    if (id < 0 || id >= a.num_blocks) {
      report(a.err, kErrBadBlockId);
      id = -1;  // zero codes and scales
    }
    ids[i] = id;
  }
  __syncthreads();

  const int my_count = nsteps > warp ? (nsteps - warp + NW - 1) / NW : 0;
  uint8_t* ring = smem + warp * R * C::STAGE;
  // Copies of this warp's k-th step (one group of asynchronous copies each,
  // empty past the last). Rows 16 u .. of a step are 16 rows of one block:
  // contiguous codes and scales, of which lane l copies the 16 bytes from 16 l.
  const int32_t cstride = a.num_kv_heads * bs * RB, sstride = a.num_kv_heads * bs * SB;
  const uint32_t ring0 = smem_addr(ring);
  const int lane16 = lane * 16, swizzled = lane16 ^ ((lane16 >> 3) & C::SWZ);
  // scale copies: SL lanes for K, as many for V, half of them for each 16 rows
  constexpr int SL = C::SCALES / 16;
  const int sv = lane / SL, sc = lane % SL, su = sc / (SL / 2);
  const uint8_t* scale_plane = (sv ? planes.p[3] : planes.p[2]) +
                               static_cast<int64_t>(kvh) * bs * SB + sc % (SL / 2) * 16;
  const uint8_t* k_plane = planes.p[0] + static_cast<int64_t>(kvh) * bs * RB + lane16;
  const uint8_t* v_plane = planes.p[1] + static_cast<int64_t>(kvh) * bs * RB + lane16;
  auto issue = [&](int k) {
    if (k < my_count) {
      const int t0 = (warp + k * NW) * kStep;
      const uint32_t dst = ring0 + (k % R) * C::STAGE;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int blk = bs == 16 ? t0 / 16 + u : t0 / 32, row = bs == 16 ? 0 : 16 * u;
        if (blk >= nlocal) break;
        const int32_t id = ids[blk];
        const int32_t b = max(id, 0);
        const uint8_t* k_src = k_plane + static_cast<int64_t>(b) * cstride + row * RB;
        const uint8_t* v_src = v_plane + static_cast<int64_t>(b) * cstride + row * RB;
#pragma unroll
        for (int i = 0; i < RB / 32; ++i) {  // 512 bytes each
          copy16(dst + (u * (RB / 32) + i) * 512 + swizzled, k_src + i * 512, id >= 0);
          copy16(dst + C::CODES + (u * (RB / 32) + i) * 512 + swizzled, v_src + i * 512,
                 id >= 0);
        }
        if (su == u && sv < 2)
          copy16(dst + 2 * C::CODES + lane16, scale_plane + static_cast<int64_t>(b) * sstride + row * SB, id >= 0);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < R; ++k) issue(k);

  typename std::conditional<BLOCKS_ON_N, MxStateN<QF, D>, MxState<QF, D>>::type st;
  const int64_t row0 = static_cast<int64_t>(s) * a.num_heads + kvh * group;
  if (my_count > 0)  // (a warp without steps has nothing to set up or to hand over)
    st.init(a, static_cast<const uint8_t*>(a.query) + row0 * D * 2, group, lane);
  for (int k = 0; k < my_count; ++k) {
    copy_wait<R - 1>();
    __syncwarp();  // every lane's copies of the step
    const uint8_t* stage = ring + (k % R) * C::STAGE;
    const uint8_t* scales = stage + 2 * C::CODES;
    const int valid = tokens - (warp + k * NW) * kStep;
    if (valid >= kStep)
      st.template step<C::SWZ, false>(stage, stage + C::CODES, scales, scales + C::SCALES, kStep,
                                      lane);
    else
      st.template step<C::SWZ, true>(stage, stage + C::CODES, scales, scales + C::SCALES, valid,
                                     lane);
    __syncwarp();
    issue(k + R);
  }
  copy_wait<0>();

  // merge the warps through shared memory (every copy has landed)
  __syncthreads();
  const bool single = parts == 1;
  float* mbuf = reinterpret_cast<float*>(smem);  // [NW][8][2]: m, l
  float* obuf = mbuf + NW * 16;                  // [NW][8][D]
  if (my_count > 0) {
    st.finish(mbuf + warp * 16, obuf + warp * 8 * D, group, lane);
  } else if (lane < group) {
    mbuf[warp * 16 + 2 * lane] = -CUDART_INF_F;
    mbuf[warp * 16 + 2 * lane + 1] = 0.f;
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < group * D; idx += NW * 32) {
    const int h = idx / D, d = idx % D;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, mbuf[w * 16 + 2 * h]);
    float L = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = mbuf[w * 16 + 2 * h], lw = mbuf[w * 16 + 2 * h + 1];
      // a warp that saw no token has m = -inf and l = 0; one that saw only
      // NaN logits has m = -inf and l = NaN, which must survive
      const float f = mw == -CUDART_INF_F ? (lw == 0.f ? 0.f : 1.f) : exp2f(mw - M);
      L += lw * f;
      // not written by a warp without steps; a NaN block of V counts whatever
      // its weight, so a weight that underflowed to 0 is multiplied all the same
      const float v = obuf[(w * 8 + h) * D + d];
      o = lw != 0.f ? fmaf(v, f, o) : o;
    }
    o = L == 0.f ? 0.f : o / L;
    if (single) {
      store_out(QF{}, a.out, (row0 + h) * D + d, o);
    } else {
      const int64_t pi = (row0 + h) * a.max_parts + part;
      a.ws_o[pi * D + d] = o;
      // the combine kernel leaves out a partial whose sum is not positive: one
      // that is NaN (o is NaN then) goes in with a weight of its own
      if (d == 0) a.ws_ml[pi] = L == L ? make_float2(M, L) : make_float2(0.f, 1.f);
    }
  }
}

template <class QF, int D, int NW, bool BLOCKS_ON_N>
cudaError_t launch_mx(const DecodeArgs& a, const MxPlanes& planes, cudaStream_t stream) {
  using C = MxCfg<D, NW>;
  if (a.partition_blocks > kMaxUnitBlocks || kStep % a.block_size != 0)
    return cudaErrorNotSupported;
  const size_t smem = C::OFF_IDS + 4 * static_cast<size_t>(a.partition_blocks);
  auto kern = paged_decode_mxfp4_kernel<QF, D, NW, BLOCKS_ON_N>;
  cudaError_t e = configure_kernel(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.num_kv_heads, a.num_seqs, a.max_parts), NW * 32, smem, stream, a,
                    planes);
}

}  // namespace

cudaError_t decode_mxfp4(const DecodeArgs& a, const uint8_t* const (&planes)[4], int q_dtype,
                         int head_dim, cudaStream_t stream) {
  const MxPlanes pl{{planes[0], planes[1], planes[2], planes[3]}};
  const int group = a.num_heads / a.num_kv_heads;
  // blocks on the columns of N wherever heads x blocks fit there (32 kv-heads of
  // one head each, 32 x 2 030 tokens: 101 us against 117 at that stage)
  const bool n = group * (head_dim / 32) <= 8;
#define PAGED_MX(QT, QF, d)                                                     \
  if (q_dtype == QT && head_dim == d)                                          \
    return n ? launch_mx<QF, d, 4, true>(a, pl, stream) : launch_mx<QF, d, 4, false>(a, pl, stream);
  PAGED_MX(kF16, F16, 64)
  PAGED_MX(kF16, F16, 128)
  PAGED_MX(kBF16, BF16, 64)
  PAGED_MX(kBF16, BF16, 128)
#undef PAGED_MX
  return cudaErrorNotSupported;
}

}  // namespace paged
