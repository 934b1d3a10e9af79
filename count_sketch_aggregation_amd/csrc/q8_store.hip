// q8_store.hip -- matrices to 8 bits and back: s2r_q8_save, s2r_q8_load, s2r_q8_weight.
//
// For each block of 128 (a row's 128 elements, or 128 x 128): a = the largest finite
// magnitude, scale = the least power of two with a <= MAX * scale, code = value / scale to
// nearest even.  One read and one write of everything: bound by HBM.  Measured on MI355X, where a
// large copy moves 5.2 TB/s: 16384 x 8192 bf16 to e4m3 72 us (5.6 TB/s), 8192 x 4096 weights with their
// transpose 28 us from bf16 (4.8), 41 from fp32 (5.0), 5001 x 1000 e5m2 to fp32 7 us.
#include "q8_device.hpp"
#include "q8_launch.hpp"

namespace s2r {

constexpr int kStoreThreads = 256;
constexpr int kStoreRows = kStoreThreads / 8;  // rows of a workgroup's tile: 8 lanes per block
constexpr int kStoreBlocks = 4;                // blocks of 128 columns of its tile

// Lanes 8 j .. 8 j + 7 of a wave hold one row's block, 16 elements each; the 8 rows of a wave
// are consecutive, so that their scale bytes are.
template <int DT, int FMT>
__global__ __launch_bounds__(kStoreThreads) void k_q8_save(
    const void* __restrict__ x, uint64_t ldx, uint8_t* __restrict__ q, uint64_t ldq,
    uint8_t* __restrict__ scale, uint64_t lds, uint32_t M, uint32_t K, uint32_t col_tiles) {
  const uint32_t ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
  const uint32_t m = rt * kStoreRows + threadIdx.x / 8;
  if (m >= M) return;  // whole groups of 8 lanes leave together
  const uint32_t c0 = ct * (kStoreBlocks * kQ8Block) + (threadIdx.x % 8) * 16;
  const auto* row = static_cast<const typename ElemT<DT>::type*>(x) + (uint64_t)m * ldx;
  uint8_t* qrow = q + (uint64_t)m * ldq;
  Raw16<DT> r[kStoreBlocks];
#pragma unroll
  for (int b = 0; b < kStoreBlocks; ++b) r[b] = load_raw16<DT>(row, c0 + b * kQ8Block, K);
#pragma unroll
  for (int b = 0; b < kStoreBlocks; ++b) {
    const uint32_t c = c0 + b * kQ8Block;
    float v[16];
    unpack16<DT>(r[b], v);
    const uint32_t sb = scale_byte<FMT>(max_over_8(amax16(v)));
    if (c < K) store_codes16(qrow, c, K, encode16<FMT>(v, sb));
    if (threadIdx.x % 8 == 0 && c < K) scale[(uint64_t)(c / kQ8Block) * lds + m] = (uint8_t)sb;
  }
}

// A lane takes the codes of one 16-byte piece of x, a wave 64 pieces of a row: what is written, two
// to four times what is read, leaves as whole lines.
constexpr int kLoadRows = 4;  // of a wave
template <int DT, int FMT>
__global__ __launch_bounds__(kStoreThreads) void k_q8_load(
    const uint8_t* __restrict__ q, uint64_t ldq, const uint8_t* __restrict__ scale, uint64_t lds,
    void* __restrict__ x, uint64_t ldx, uint32_t M, uint32_t K, uint32_t col_tiles) {
  using E = typename ElemT<DT>::type;
  constexpr uint32_t kPer = 16 / elem_bytes<DT>();
  const uint32_t ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
  const uint32_t m0 = (rt * (kStoreThreads / 64) + threadIdx.x / 64) * kLoadRows;
  const uint32_t c = (ct * 64 + threadIdx.x % 64) * kPer;
  if (c >= K) return;
  uint32_t code[kLoadRows][kPer / 4], sb[kLoadRows];
#pragma unroll
  for (int i = 0; i < kLoadRows; ++i) {
    const uint32_t m = min(m0 + i, M - 1);
    const uint8_t* at = q + (uint64_t)m * ldq + c;
    if (kPer == 8) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(at);
      code[i][0] = v[0], code[i][kPer / 4 - 1] = v[1];
    } else {
      code[i][0] = *reinterpret_cast<const uint32_t*>(at);
    }
    sb[i] = scale[(uint64_t)(c / kQ8Block) * lds + m];
  }
#pragma unroll
  for (int i = 0; i < kLoadRows; ++i) {
    const uint32_t m = m0 + i;
    if (m >= M) return;
    const f32x4 lo = decode4<FMT>(code[i][0], scale_value(sb[i]));
    const f32x4 hi = decode4<FMT>(code[i][kPer / 4 - 1], scale_value(sb[i]));
    E* const to = static_cast<E*>(x) + (uint64_t)m * ldx + c;
    u32x4 v;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (DT == S2R_F32) v[w] = __float_as_uint(lo[w]);
      else v[w] = w < 2 ? pack2<DT>(lo[2 * w], lo[2 * w + 1]) : pack2<DT>(hi[2 * w - 4], hi[2 * w - 3]);
    }
    if (c + kPer <= K) {
      *reinterpret_cast<u32x4*>(to) = v;
    } else {
#pragma unroll
      for (uint32_t e = 0; e < kPer; ++e)
        if (c + e < K) to[e] = DT == S2R_F32 ? (E)v[e % 4] : (E)(v[e / 2 % 4] >> 16 * (e % 2));
    }
  }
}

// One workgroup per 128 x 128 block: row t / 8 + 32 i of the block, 16 elements per lane.  The
// transposed codes go through LDS, where each lane takes 16 rows x 4 columns as dwords and
// transposes them 4 x 4 bytes at a time.
constexpr int kWtStride = kQ8Block + 4;  // bytes of an LDS row: dword columns on distinct banks

__device__ inline void transpose4(const uint32_t (&a)[4], uint32_t (&t)[4]) {
  const uint32_t p = __builtin_amdgcn_perm(a[1], a[0], 0x05010400);  // a0.0 a1.0 a0.1 a1.1
  const uint32_t q = __builtin_amdgcn_perm(a[1], a[0], 0x07030602);  // a0.2 a1.2 a0.3 a1.3
  const uint32_t r = __builtin_amdgcn_perm(a[3], a[2], 0x05010400);
  const uint32_t s = __builtin_amdgcn_perm(a[3], a[2], 0x07030602);
  t[0] = __builtin_amdgcn_perm(r, p, 0x05040100);
  t[1] = __builtin_amdgcn_perm(r, p, 0x07060302);
  t[2] = __builtin_amdgcn_perm(s, q, 0x05040100);
  t[3] = __builtin_amdgcn_perm(s, q, 0x07060302);
}

template <int DT, int FMT>
__global__ __launch_bounds__(kStoreThreads) void k_q8_weight(
    const void* __restrict__ w, uint64_t ldw, uint8_t* __restrict__ q, uint64_t ldq,
    uint8_t* __restrict__ scale, uint64_t lds, uint8_t* __restrict__ qt, uint64_t ldt,
    uint8_t* __restrict__ scale_t, uint64_t ldst, uint32_t N, uint32_t K, uint32_t col_blocks) {
  __shared__ uint32_t wave_max[kStoreThreads / 64];
  __shared__ uint32_t tile[kQ8Block * kWtStride / 4];
  const uint32_t kb = blockIdx.x % col_blocks, nb = blockIdx.x / col_blocks;
  const uint32_t t = threadIdx.x;
  const uint32_t c = kb * kQ8Block + (t % 8) * 16;
  Raw16<DT> r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t n = nb * kQ8Block + t / 8 + 32 * i;
    const auto* row = static_cast<const typename ElemT<DT>::type*>(w) + (uint64_t)n * ldw;
    r[i] = load_raw16<DT>(row, c, n < N ? K : 0);
  }
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[16];
    unpack16<DT>(r[i], v);
    am = umax(am, amax16(v));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) am = umax(am, (uint32_t)__shfl_xor((int)am, o));
  if (t % 64 == 0) wave_max[t / 64] = am;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kStoreThreads / 64; ++i) am = umax(am, wave_max[i]);
  const uint32_t sb = scale_byte<FMT>(am);
  if (t == 0) {
    scale[(uint64_t)kb * lds + nb] = (uint8_t)sb;
    if (qt) scale_t[(uint64_t)nb * ldst + kb] = (uint8_t)sb;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t rr = t / 8 + 32 * i, n = nb * kQ8Block + rr;
    float v[16];
    unpack16<DT>(r[i], v);
    const u32x4 code = encode16<FMT>(v, sb);
    if (n < N && c < K) store_codes16(q + (uint64_t)n * ldq, c, K, code);
    if (qt) {
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[(rr * kWtStride + (t % 8) * 16) / 4 + j] = code[j];
    }
  }
  if (!qt) return;
  __syncthreads();
  const uint32_t ng = t % 8, kg = t / 8;  // 16 rows n, 4 columns k
  u32x4 out[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    uint32_t in[4], tr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) in[j] = tile[(ng * 16 + a * 4 + j) * (kWtStride / 4) + kg];
    transpose4(in, tr);
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j][a] = tr[j];
  }
  const uint32_t n0 = nb * kQ8Block + ng * 16;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t k = kb * kQ8Block + kg * 4 + j;
    if (k < K && n0 < N) store_codes16(qt + (uint64_t)k * ldt, n0, N, out[j]);
  }
}

#define S2R_Q8_DISPATCH(dtype, format, CALL)                                       \
  do {                                                                             \
    if ((format) == S2R_E4M3) {                                                    \
      constexpr int FMT = S2R_E4M3;                                                \
      if ((dtype) == S2R_BF16) { constexpr int DT = S2R_BF16; CALL; }              \
      else if ((dtype) == S2R_F16) { constexpr int DT = S2R_F16; CALL; }           \
      else { constexpr int DT = S2R_F32; CALL; }                                   \
    } else {                                                                       \
      constexpr int FMT = S2R_E5M2;                                                \
      if ((dtype) == S2R_BF16) { constexpr int DT = S2R_BF16; CALL; }              \
      else if ((dtype) == S2R_F16) { constexpr int DT = S2R_F16; CALL; }           \
      else { constexpr int DT = S2R_F32; CALL; }                                   \
    }                                                                              \
  } while (0)

hipError_t launch_q8_save(uint64_t M, uint64_t K, const s2r_mat& x, const s2r_q8_mat& out,
                          hipStream_t s) {
  const uint64_t ct = (K + kStoreBlocks * kQ8Block - 1) / (kStoreBlocks * kQ8Block);
  trace_mark(s, "k_q8_save");
  by_rows(M, kStoreRows, ct, [&](uint64_t m, uint64_t rows) {
    const s2r_mat f = from_row(x, m);
    const s2r_q8_mat t = from_row(out, m);
    const uint32_t grid = (uint32_t)(ct * ((rows + kStoreRows - 1) / kStoreRows));
    S2R_Q8_DISPATCH(x.dtype, out.format,
                    hipLaunchKernelGGL((k_q8_save<DT, FMT>), dim3(grid), dim3(kStoreThreads), 0, s,
                                       f.data, f.ld, t.q, t.ld, t.scale, t.lds, (uint32_t)rows,
                                       (uint32_t)K, (uint32_t)ct));
  });
  return hipGetLastError();
}

hipError_t launch_q8_load(uint64_t M, uint64_t K, const s2r_q8_mat& in, const s2r_mat& x,
                          hipStream_t s) {
  const uint64_t cols = 1024 / (x.dtype == S2R_F32 ? 4 : 2), each = kStoreThreads / 64 * kLoadRows;
  const uint64_t ct = (K + cols - 1) / cols;
  trace_mark(s, "k_q8_load");
  by_rows(M, each, ct, [&](uint64_t m, uint64_t rows) {
    const s2r_q8_mat f = from_row(in, m);
    const s2r_mat t = from_row(x, m);
    const uint32_t grid = (uint32_t)(ct * ((rows + each - 1) / each));
    S2R_Q8_DISPATCH(x.dtype, in.format,
                    hipLaunchKernelGGL((k_q8_load<DT, FMT>), dim3(grid), dim3(kStoreThreads), 0, s,
                                       f.q, f.ld, f.scale, f.lds, t.data, t.ld, (uint32_t)rows,
                                       (uint32_t)K, (uint32_t)ct));
  });
  return hipGetLastError();
}

hipError_t launch_q8_weight(uint64_t N, uint64_t K, const s2r_mat& w, const s2r_q8_mat& out,
                            const s2r_q8_mat* out_t, hipStream_t s) {
  const uint64_t kb = (K + kQ8Block - 1) / kQ8Block, nb = (N + kQ8Block - 1) / kQ8Block;
  trace_mark(s, "k_q8_weight");
  S2R_Q8_DISPATCH(w.dtype, out.format,
                  hipLaunchKernelGGL((k_q8_weight<DT, FMT>), dim3((uint32_t)(kb * nb)),
                                     dim3(kStoreThreads), 0, s, w.data, w.ld, out.q, out.ld,
                                     out.scale, out.lds, out_t ? out_t->q : nullptr,
                                     out_t ? out_t->ld : 0, out_t ? out_t->scale : nullptr,
                                     out_t ? out_t->lds : 0, (uint32_t)N, (uint32_t)K,
                                     (uint32_t)kb));
  return hipGetLastError();
}

}  // namespace s2r
