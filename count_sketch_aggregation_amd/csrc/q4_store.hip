// q4_store.hip -- matrices to 4 bits and back: s2r_q4_save, s2r_q4_load.
//
// For each 32 elements of a row: a = the largest magnitude, scale = the least power of two with
// a <= 6 scale, code = value / scale to nearest even.  The transpose has blocks of 32 rows of a column and so
// scales and codes of its own; both are written from one read of x.  Measured on MI355X, where a large copy moves 5.18
// TB/s: rows of 8192 x 8192 bf16 to 4 bits 34 us (5.0 TB/s), back to bf16 28 to 32 (5.3 and more): bound by HBM.  With the
// transpose 52 us, 3.9 TB/s, and 64 (3.2) right behind two loads of 134 MB each: most likely since a tile leaves
// half lines of the transpose's codes, and its scales as single bytes.  1001 x 1000 fp32 3.1, and back to bf16 3.2.
#include "q4_device.hpp"
#include "q4_launch.hpp"
#include "q8_tile.hpp"

namespace s2r {

constexpr int kQ4Threads = 256;

// Maximum over aligned pairs of lanes (a block at 16 elements per lane).
__device__ inline uint32_t max_over_2(uint32_t v) {
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));
}

__device__ inline uint32_t bits16(const float (&x)[16]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) most = umax(most, __float_as_uint(x[i]) & 0x7fffffffu);
  return most;
}

// Codes of columns c .. c + 15 of a row of `cols`.  Of the last byte of an odd row the upper half is 0,
// as the values beyond the row are.
__device__ inline void q4_store16(uint8_t* row, uint32_t c, uint32_t cols, u32x2 q) {
  if (c + 16 <= cols) {
    *reinterpret_cast<u32x2*>(row + c / 2) = q;
  } else {
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
      if (c + 2 * e < cols) row[c / 2 + e] = (uint8_t)(q[e / 4] >> 8 * (e % 4));
  }
}

// ---- rows ---------------------------------------------------------------------------------
// 16 elements to a lane, 2 lanes to a block, 64 lanes to 1024 columns; ROWS rows to a wave.
template <int DT, int ROWS>
__global__ __launch_bounds__(kQ4Threads) void k_q4_save(s2r_mat x, s2r_q4_mat out, uint32_t R, uint32_t C,
                                                        uint32_t spans) {
  const uint32_t span = blockIdx.x % spans, lane = threadIdx.x % 64;
  const uint32_t r0 = (blockIdx.x / spans * (kQ4Threads / 64) + threadIdx.x / 64) * ROWS;
  const uint32_t c = span * 1024 + lane * 16;
  Raw16<DT> raw[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    raw[i] = load_raw16<DT>(static_cast<const uint8_t*>(x.data) +
                                (uint64_t)min(r0 + i, R - 1) * x.ld * elem_bytes<DT>(), c, C);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float v[16];
    unpack16<DT>(raw[i], v);
    const uint32_t b = q4_scale_byte(max_over_2(bits16(v)));
    if (r0 + i >= R || c >= C) continue;
    q4_store16(out.q + (uint64_t)(r0 + i) * out.ld, c, C, u32x2{q4_encode8(v, b), q4_encode8(v + 8, b)});
    if (lane % 2 == 0) out.scale[(uint64_t)(r0 + i) * out.lds + c / kQ4Block] = (uint8_t)b;
  }
}

// ---- rows and columns -----------------------------------------------------------------------
// A workgroup takes 128 x 128 elements: their rows as above, 8 lanes to a row, and through LDS, as they
// came, their columns: a lane takes 32 rows of one column, one block, and writes its 16 bytes.  Tiles that share
// lines run on one die, one soon after the other (128.5 us instead of 133 for 8192 x 8192 and back).
constexpr int kSide = 128;

template <int DT>
__global__ __launch_bounds__(kQ4Threads) void k_q4_save_both(s2r_mat x, s2r_q4_mat out, s2r_q4_mat out_t,
                                                             uint32_t R, uint32_t C, uint32_t col_tiles) {
  using E = typename ElemT<DT>::type;
  // 16 bytes more than a row: the lanes of a write, 8 to a row, meet the banks evenly
  constexpr int kStride = kSide + 16 / sizeof(E);
  __shared__ __attribute__((aligned(16))) E tile[kSide * kStride];
  const TileAt tile_of = tile_at(blockIdx.x, gridDim.x / col_tiles, col_tiles, gridDim.x);
  const uint32_t ct = tile_of.col, rt = tile_of.row, t = threadIdx.x;
  const uint32_t c = ct * kSide + t % 8 * 16;
  Raw16<DT> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = rt * kSide + t / 8 + 32 * i;
    raw[i] = load_raw16<DT>(static_cast<const uint8_t*>(x.data) + (uint64_t)min(r, R - 1) * x.ld * elem_bytes<DT>(),
                            c, r < R ? C : 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = rt * kSide + t / 8 + 32 * i;
#pragma unroll
    for (int p = 0; p < Raw16<DT>::kPieces; ++p)
      *reinterpret_cast<u32x4*>(tile + (t / 8 + 32 * i) * kStride + t % 8 * 16 + p * Raw16<DT>::kPer) = raw[i].p[p];
    if (!out.q) continue;
    float v[16];
    unpack16<DT>(raw[i], v);
    const uint32_t b = q4_scale_byte(max_over_2(bits16(v)));
    if (r >= R || c >= C) continue;
    q4_store16(out.q + (uint64_t)r * out.ld, c, C, u32x2{q4_encode8(v, b), q4_encode8(v + 8, b)});
    if (t % 2 == 0) out.scale[(uint64_t)r * out.lds + c / kQ4Block] = (uint8_t)b;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t col = t % kSide, block = t / kSide + 2 * i;
    const uint32_t n = ct * kSide + col, r0 = rt * kSide + block * kQ4Block;
    float v[32];
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const E raw1 = tile[(block * kQ4Block + e) * kStride + col];
      if (DT == S2R_F32) v[e] = __uint_as_float((uint32_t)raw1);
      else if (DT == S2R_BF16) v[e] = __uint_as_float((uint32_t)raw1 << 16);
      else v[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)raw1);
      most = umax(most, __float_as_uint(v[e]) & 0x7fffffffu);
    }
    if (n >= C || r0 >= R) continue;
    const uint32_t b = q4_scale_byte(most);
    const u32x4 q = {q4_encode8(v, b), q4_encode8(v + 8, b), q4_encode8(v + 16, b), q4_encode8(v + 24, b)};
    uint8_t* const to = out_t.q + (uint64_t)n * out_t.ld;
    if (r0 + 32 <= R) {
      *reinterpret_cast<u32x4*>(to + r0 / 2) = q;
    } else {
      q4_store16(to, r0, R, u32x2{q[0], q[1]});
      q4_store16(to, r0 + 16, R, u32x2{q[2], q[3]});
    }
    out_t.scale[(uint64_t)n * out_t.lds + r0 / kQ4Block] = (uint8_t)b;
  }
}

// ---- back -----------------------------------------------------------------------------------
// A lane takes the codes of one 16-byte piece of x, a wave 64 pieces of kLoadRows rows.
constexpr int kQ4LoadRows = 4;

template <int DT>
__global__ __launch_bounds__(kQ4Threads) void k_q4_load(s2r_q4_mat in, s2r_mat x, uint32_t R, uint32_t C,
                                                        uint32_t spans) {
  using E = typename ElemT<DT>::type;
  constexpr uint32_t kPer = 16 / elem_bytes<DT>();
  const uint32_t span = blockIdx.x % spans, lane = threadIdx.x % 64;
  const uint32_t r0 = (blockIdx.x / spans * (kQ4Threads / 64) + threadIdx.x / 64) * kQ4LoadRows;
  const uint32_t c = (span * 64 + lane) * kPer;
  if (c >= C) return;
  uint32_t code[kQ4LoadRows], sb[kQ4LoadRows];
#pragma unroll
  for (int i = 0; i < kQ4LoadRows; ++i) {
    const uint64_t r = min(r0 + i, R - 1);
    const uint8_t* at = in.q + r * in.ld + c / 2;
    code[i] = kPer == 8 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
    sb[i] = in.scale[r * in.lds + c / kQ4Block];
  }
#pragma unroll
  for (int i = 0; i < kQ4LoadRows; ++i) {
    if (r0 + i >= R) return;
    // a scale byte of 255 is an infinity here, which no code may meet: NaN, as the format has it
    const float s = sb[i] == kQ4NanScale ? __uint_as_float(0x7fc00000u) : scale_value(sb[i]);
    float v[8];
    const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 0);
    const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 1);
    const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 2);
    const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], 1.0f, 3);
    v[0] = v0[0] * s, v[1] = v0[1] * s, v[2] = v1[0] * s, v[3] = v1[1] * s;
    v[4] = v2[0] * s, v[5] = v2[1] * s, v[6] = v3[0] * s, v[7] = v3[1] * s;
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = DT == S2R_F32 ? __float_as_uint(v[j]) : pack2<DT>(v[2 * j], v[2 * j + 1]);
    E* const to = static_cast<E*>(x.data) + (uint64_t)(r0 + i) * x.ld + c;
    if (c + kPer <= C) {
      *reinterpret_cast<u32x4*>(to) = w;
    } else {
#pragma unroll
      for (uint32_t e = 0; e < kPer; ++e)
        if (c + e < C) to[e] = DT == S2R_F32 ? (E)w[e % 4] : (E)(w[e / 2 % 4] >> 16 * (e % 2));
    }
  }
}

#define S2R_Q4_TYPES(dtype, CALL)                                      \
  do {                                                                 \
    if ((dtype) == S2R_BF16) { constexpr int DT = S2R_BF16; CALL; }    \
    else if ((dtype) == S2R_F16) { constexpr int DT = S2R_F16; CALL; } \
    else { constexpr int DT = S2R_F32; CALL; }                         \
  } while (0)

hipError_t launch_q4_save(uint64_t R, uint64_t C, const s2r_mat& x, const s2r_q4_mat* out,
                          const s2r_q4_mat* out_t, hipStream_t s) {
  if (out_t) {
    // ld and with it R is at most 2^23 and C below 2^22, so a launch has below 2^31 workgroups, but its
    // threads may pass 2^32: ranges of whole tiles of rows, whose transpose begins at whole bytes
    const uint64_t ct = (C + kSide - 1) / kSide;
    trace_mark(s, "k_q4_save_both");
    by_rows(R, kSide, ct, [&](uint64_t r, uint64_t n) {
      const s2r_mat f = from_row(x, r);
      const s2r_q4_mat o = out ? from_row(*out, r) : s2r_q4_mat{};
      const s2r_q4_mat ot = {out_t->q + r / 2, out_t->ld, out_t->scale + r / kQ4Block, out_t->lds};
      const dim3 grid((uint32_t)(ct * ((n + kSide - 1) / kSide)));
      S2R_Q4_TYPES(x.dtype, hipLaunchKernelGGL((k_q4_save_both<DT>), grid, dim3(kQ4Threads), 0, s, f, o, ot,
                                               (uint32_t)n, (uint32_t)C, (uint32_t)ct));
    });
    return hipGetLastError();
  }
  // four rows to a wave, or one where that leaves compute units without work (1001 x 1000 fp32: 3.1 us, 5.4 with
  // four)
  const uint64_t spans = (C + 1023) / 1024;
  const bool few = spans * ((R + 15) / 16) < 2 * 256;
  const uint64_t each = kQ4Threads / 64 * (few ? 1 : 4);
  trace_mark(s, "k_q4_save");
  by_rows(R, each, spans, [&](uint64_t r, uint64_t n) {
    const s2r_mat f = from_row(x, r);
    const s2r_q4_mat o = from_row(*out, r);
    const dim3 grid((uint32_t)(spans * ((n + each - 1) / each)));
#define S2R_SAVE(ROWS)                                                                                         \
  S2R_Q4_TYPES(x.dtype, hipLaunchKernelGGL((k_q4_save<DT, ROWS>), grid, dim3(kQ4Threads), 0, s, f, o, (uint32_t)n, \
                                           (uint32_t)C, (uint32_t)spans))
    if (few) S2R_SAVE(1);
    else S2R_SAVE(4);
#undef S2R_SAVE
  });
  return hipGetLastError();
}

hipError_t launch_q4_load(uint64_t R, uint64_t C, const s2r_q4_mat& in, const s2r_mat& x, hipStream_t s) {
  const uint64_t cols = 1024 / (x.dtype == S2R_F32 ? 4 : 2), spans = (C + cols - 1) / cols;
  const uint64_t each = kQ4Threads / 64 * kQ4LoadRows;
  trace_mark(s, "k_q4_load");
  by_rows(R, each, spans, [&](uint64_t r, uint64_t n) {
    const s2r_q4_mat f = from_row(in, r);
    const s2r_mat t = from_row(x, r);
    const dim3 grid((uint32_t)(spans * ((n + each - 1) / each)));
    S2R_Q4_TYPES(x.dtype, hipLaunchKernelGGL((k_q4_load<DT>), grid, dim3(kQ4Threads), 0, s, f, t, (uint32_t)n,
                                             (uint32_t)C, (uint32_t)spans));
  });
  return hipGetLastError();
}

}  // namespace s2r
