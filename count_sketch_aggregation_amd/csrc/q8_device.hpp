// q8_device.hpp -- device code shared by the 8-bit training kernels: element types, the
// 128-element scale and the rounding to 8 bits (internal to libs2r).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "s2r_q8.h"

namespace s2r {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kQ8Block = 128;    // elements of a row, or rows and columns, under one scale
constexpr int kQ8MinScale = 17;  // 2^-110: below it a stored value would not be a normal bf16

// ---- element types -----------------------------------------------------------------------
// Storage of one element, and of the 16 consecutive ones that a lane handles at a time.
template <int DT> struct ElemT;
template <> struct ElemT<S2R_BF16> { using type = uint16_t; };
template <> struct ElemT<S2R_F16> { using type = uint16_t; };
template <> struct ElemT<S2R_F32> { using type = uint32_t; };

template <int DT>
constexpr int elem_bytes() { return DT == S2R_F32 ? 4 : 2; }

// 16 elements in 16-byte pieces: `piece` 0..(2 or 4)-1
template <int DT>
struct Raw16 {
  static constexpr int kPieces = elem_bytes<DT>();
  static constexpr int kPer = 16 / kPieces;  // elements of a piece
  u32x4 p[kPieces];
};

// The pieces of elements [col, col + 16) of a row that hold a column below `cols`; the
// others, and the elements at or beyond `cols`, are zero.  A piece that holds a valid column
// lies inside the row (ld is a multiple of 16 bytes).
template <int DT>
__device__ inline Raw16<DT> load_raw16(const void* row, uint32_t col, uint32_t cols) {
  Raw16<DT> r;
  constexpr int per = Raw16<DT>::kPer;
  const auto* src = static_cast<const typename ElemT<DT>::type*>(row) + col;
  if (col + 16 <= cols) {
#pragma unroll
    for (int i = 0; i < Raw16<DT>::kPieces; ++i)
      r.p[i] = *reinterpret_cast<const u32x4*>(src + i * per);
    return r;
  }
#pragma unroll
  for (int i = 0; i < Raw16<DT>::kPieces; ++i) {
    u32x4 v = {0, 0, 0, 0};
    const uint32_t c = col + i * per;
    if (c < cols) {
      v = *reinterpret_cast<const u32x4*>(src + i * per);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (DT == S2R_F32) {
          if (c + w >= cols) v[w] = 0;
        } else {
          if (c + 2 * w >= cols) v[w] = 0;
          else if (c + 2 * w + 1 >= cols) v[w] &= 0xffffu;
        }
      }
    }
    r.p[i] = v;
  }
  return r;
}

template <int DT>
__device__ inline void unpack16(const Raw16<DT>& r, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < Raw16<DT>::kPieces; ++i)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t v = r.p[i][w];
      if (DT == S2R_F32) {
        x[4 * i + w] = __uint_as_float(v);
      } else if (DT == S2R_BF16) {
        x[8 * i + 2 * w] = __uint_as_float(v << 16);
        x[8 * i + 2 * w + 1] = __uint_as_float(v & 0xffff0000u);
      } else {
        const f16x2 h = __builtin_bit_cast(f16x2, v);
        x[8 * i + 2 * w] = (float)h[0];
        x[8 * i + 2 * w + 1] = (float)h[1];
      }
    }
}

// fp32 -> bf16 and fp16, to nearest with ties to even, two at a time
template <int DT>
__device__ inline uint32_t pack2(float a, float b) {
  if (DT == S2R_BF16) {
    bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  f16x2 v = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// 16 fp32 values to a row's elements [col, col + 16), those at or beyond `cols` left alone.
template <int DT>
__device__ inline void store16(void* row, uint32_t col, uint32_t cols, const float (&x)[16]) {
  auto* dst = static_cast<typename ElemT<DT>::type*>(row) + col;
  constexpr int per = Raw16<DT>::kPer;
#pragma unroll
  for (int i = 0; i < Raw16<DT>::kPieces; ++i) {
    u32x4 v;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      v[w] = DT == S2R_F32 ? __float_as_uint(x[4 * i + w])
                           : pack2<DT>(x[8 * i + 2 * w], x[8 * i + 2 * w + 1]);
    const uint32_t c = col + i * per;
    if (c + per <= cols) {
      *reinterpret_cast<u32x4*>(dst + i * per) = v;
    } else {
#pragma unroll
      for (int e = 0; e < per; ++e)
        if (c + e < cols)
          dst[i * per + e] = DT == S2R_F32 ? v[e & 3] : (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Four fp32 values to columns c .. c + 3 of row m, c a multiple of 4; those at or beyond `cols`
// are left alone.
__device__ inline void store4(const s2r_mat& o, uint32_t m, uint32_t c, uint32_t cols, f32x4 v) {
  const uint64_t at = (uint64_t)m * o.ld + c;
  if (o.dtype == S2R_F32) {
    float* p = static_cast<float*>(o.data) + at;
    if (c + 4 <= cols) *reinterpret_cast<f32x4*>(p) = v;
    else
      for (uint32_t e = 0; c + e < cols; ++e) p[e] = e == 0 ? v[0] : e == 1 ? v[1] : v[2];
    return;
  }
  const bool bf = o.dtype == S2R_BF16;
  const u32x2 h = {bf ? pack2<S2R_BF16>(v[0], v[1]) : pack2<S2R_F16>(v[0], v[1]),
                   bf ? pack2<S2R_BF16>(v[2], v[3]) : pack2<S2R_F16>(v[2], v[3])};
  uint16_t* p = static_cast<uint16_t*>(o.data) + at;
  if (c + 4 <= cols) *reinterpret_cast<u32x2*>(p) = h;
  else
    for (uint32_t e = 0; c + e < cols; ++e)
      p[e] = (uint16_t)(e == 0 ? h[0] : e == 1 ? h[0] >> 16 : h[1]);
}

// Eight values to columns c .. c + 7 of row m, c a multiple of 8.
__device__ inline void store8(const s2r_mat& o, uint32_t m, uint32_t c, uint32_t cols, f32x4 lo,
                              f32x4 hi) {
  if (c + 8 <= cols && o.dtype != S2R_F32) {
    const bool bf = o.dtype == S2R_BF16;
    u32x4 v;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float x = w < 2 ? lo[2 * w] : hi[2 * w - 4], y = w < 2 ? lo[2 * w + 1] : hi[2 * w - 3];
      v[w] = bf ? pack2<S2R_BF16>(x, y) : pack2<S2R_F16>(x, y);
    }
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(o.data) + (uint64_t)m * o.ld + c) = v;
    return;
  }
  store4(o, m, c, cols, lo);
  if (c + 4 < cols) store4(o, m, c + 4, cols, hi);
}

// ---- the scale ----------------------------------------------------------------------------
template <int FMT>
constexpr int scale_bias() { return FMT == S2R_E4M3 ? 8 : 15; }

// Scale byte of a block whose largest finite magnitude has the fp32 bits `amax`: MAX is
// 1.75 * 2^8 (e4m3) or 1.75 * 2^15 (e5m2), so the least power of two s with amax <= MAX * s is
// amax's own power of two over 2^8 or 2^15, one more where amax's mantissa exceeds 1.75;
// adding 0x1fffff carries into the exponent exactly then.
template <int FMT>
__device__ inline uint32_t scale_byte(uint32_t amax) {
  const int b = (int)((amax + 0x1fffffu) >> 23) - scale_bias<FMT>();
  return b < kQ8MinScale ? kQ8MinScale : b;
}

__device__ inline float scale_value(uint32_t b) { return __uint_as_float(b << 23); }

__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Magnitude bits of the largest finite of 16 values.  As integers fp32 magnitudes order as their
// values, with infinity and every NaN above them; a floating maximum would return a quieted
// signalling NaN and then drop it together with all that came before.
__device__ inline uint32_t amax16(const float (&x)[16]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) most = umax(most, __float_as_uint(x[i]) & 0x7fffffffu);
  if (most >= 0x7f800000u) {  // rare: once more, without infinities and NaN
    most = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
      most = umax(most, b >= 0x7f800000u ? 0u : b);
    }
  }
  return most;
}

// Maximum over aligned groups of 8 lanes (a 128-element block at 16 elements per lane): two
// exchanges within quads, then the mirrored half row.
__device__ inline uint32_t max_over_8(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));
  return v;
}

// ---- codes --------------------------------------------------------------------------------
// Four values to four codes: the conversion divides by the scale (a power of two: exact, or far
// below the format's least code), rounds to nearest even and cannot overflow, because
// the block's scale covers its largest finite value; infinities and NaN convert as the
// format has them.
template <int FMT>
__device__ inline uint32_t encode4(float a, float b, float c, float d, float scale) {
  s16x2 v = {};
  if (FMT == S2R_E4M3) {
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, a, b, scale, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, c, d, scale, true);
  } else {
    v = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(v, a, b, scale, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(v, c, d, scale, true);
  }
  return __builtin_bit_cast(uint32_t, v);
}

// 16 values to codes under the scale byte sb.  The largest scale is that of blocks with values next to
// fp32's largest, some of which round to 2^128: that is code 0x78 in both formats, and the
// code below it is within a step of them too.
template <int FMT>
__device__ inline u32x4 encode16(const float (&x)[16], uint32_t sb) {
  const float scale = scale_value(sb);
  u32x4 q;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    q[w] = encode4<FMT>(x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3], scale);
  if (sb == 255 - scale_bias<FMT>()) {  // rare
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t off = (q[w] & 0x7f7f7f7fu) ^ 0x78787878u;  // 0 in the bytes meant
      q[w] -= (~(off + 0x7f7f7f7fu) & 0x80808080u) >> 7;
    }
  }
  return q;
}

// Four codes to four values, exact.
template <int FMT>
__device__ inline f32x4 decode4(uint32_t q, float scale) {
  f32x2 lo, hi;
  if (FMT == S2R_E4M3) {
    lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, scale, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, scale, true);
  } else {
    lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(q, scale, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(q, scale, true);
  }
  return {lo[0], lo[1], hi[0], hi[1]};
}

// Four codes to bf16: exact, as a scale is a power of two and a stored value a normal bf16.
template <int FMT>
__device__ inline u32x2 to_bf16(uint32_t q, float scale) {
  if (FMT == S2R_E4M3)
    return {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, scale, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, scale, true))};
  return {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(q, scale, false)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(q, scale, true))};
}

template <int FMT>
__device__ inline void decode16(u32x4 q, float scale, float (&x)[16]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const f32x4 v = decode4<FMT>(q[w], scale);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * w + e] = v[e];
  }
}

// Code pieces of a row: [col, col + 16) with the codes at or beyond `cols` zero; and back.
__device__ inline u32x4 load_codes16(const uint8_t* row, uint32_t col, uint32_t cols) {
  u32x4 v = {0, 0, 0, 0};
  if (col < cols) v = *reinterpret_cast<const u32x4*>(row + col);
  if (col + 16 > cols) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int left = (int)cols - (int)col - 4 * w;
      if (left <= 0) v[w] = 0;
      else if (left < 4) v[w] &= (1u << (8 * left)) - 1;
    }
  }
  return v;
}

__device__ inline void store_codes16(uint8_t* row, uint32_t col, uint32_t cols, u32x4 q) {
  if (col + 16 <= cols) {
    *reinterpret_cast<u32x4*>(row + col) = q;
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (col + e < cols) row[col + e] = (uint8_t)(q[e / 4] >> (8 * (e & 3)));
  }
}

}  // namespace s2r
