// q8_gemm.hip -- C = A B^T of 8-bit matrices with a power-of-two scale for each block of 128:
//   c[m][n] = sum_k a[m][k] sa[k / 128][m] b[n][k] sb[k / 128][n / 128].
// The scaled matrix instruction multiplies both operands by their scales itself, so one fp32
// accumulator runs over the whole sum.  The first operand is B, so that a lane's results
// are consecutive columns of C.
#include "q8_launch.hpp"
#include "q8_tile.hpp"

namespace s2r {

// ---- fragments ----------------------------------------------------------------------------
// The matrix instruction takes 16 rows x 128 bytes from each side: lane l holds row l % 16,
// bytes 32 (l / 16) .. + 31.
__device__ inline i32x8 join(u32x4 lo, u32x4 hi) {
  i32x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (int)lo[i];
    v[4 + i] = (int)hi[i];
  }
  return v;
}

// `at` is the byte of `sa` that holds this fragment's scale.
template <int FA, int FB>
__device__ inline f32x4 mma(const i32x8& b, const i32x8& a, const f32x4& c, uint32_t sb,
                            uint32_t sa, int at) {
  switch (at) {
    case 0:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 0, (int)sa);
    case 1:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 1, (int)sa);
    case 2:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 2, (int)sa);
    default:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 3, (int)sa);
  }
}

// ---- tiles --------------------------------------------------------------------------------
// WM x WN waves, each 64 IM rows of A by 64 rows of B; a step is one block of 128 of the sum.
// LDS holds 128 bytes of every row of both operands, twice: one half is filled directly from
// global memory while the other is multiplied.  16-byte piece s of LDS row p lies at
// s ^ (p / 2 % 8): the 16 lanes that read together, one piece of 16 rows, meet every bank once.
// Rows of A are taken in the order m = 64 I + 4 r + i (fragment i of group I, lane r), so the
// scales of a lane's four fragments are one dword; rows of B in the order
// n = 16 g + 4 j + t (fragment j, row 4 g + t), so a lane's results are 16 consecutive columns.
template <int FA, int FB, int WM, int WN, int IM>
__global__ __launch_bounds__(64 * WM * WN) void k_q8_gemm(s2r_q8_mat a, s2r_q8_mat b, s2r_mat c,
                                                          uint64_t part_bytes, uint32_t M, uint32_t N,
                                                          uint32_t K, uint32_t m_tiles,
                                                          uint32_t n_tiles, uint32_t part_steps) {
  constexpr int kWaves = WM * WN, TM = 64 * IM * WM, TN = 64 * WN;
  constexpr int kLoadsA = TM / 8 / kWaves, kLoadsB = TN / 8 / kWaves;
  constexpr int kBytes = (TM + TN) * kQ8Block;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBytes];

  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const TileAt t = tile_at(blockIdx.x, m_tiles, n_tiles, gridDim.x);
  const uint32_t m0 = t.row * TM, n0 = t.col * TN;
  const uint32_t wm = wave / WN * (64 * IM), wn = wave % WN * 64;
  const uint32_t steps = (K + kQ8Block - 1) / kQ8Block;
  const uint32_t s0 = t.part * part_steps, s1 = min(s0 + part_steps, steps);

  // where this lane's pieces of a step come from, relative to the tile's first row
  uint32_t from_a[kLoadsA], from_b[kLoadsB];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j) {
    const uint32_t p = (wave * kLoadsA + j) * 8 + lane / 8;
    const uint32_t row = p / 64 * 64 + 4 * (p % 16) + p % 64 / 16;
    from_a[j] = min(row, M - 1 - m0) * (uint32_t)a.ld + (lane % 8 ^ p / 2 % 8) * 16;
  }
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) {
    const uint32_t p = (wave * kLoadsB + j) * 8 + lane / 8;
    const uint32_t row = p / 64 * 64 + 16 * (p % 16 / 4) + 4 * (p % 64 / 16) + p % 4;
    from_b[j] = min(row, N - 1 - n0) * (uint32_t)b.ld + (lane % 8 ^ p / 2 % 8) * 16;
  }
  const uint64_t base_a = (uint64_t)a.q + (uint64_t)m0 * a.ld, len_a = (uint64_t)(M - m0) * a.ld;
  const uint64_t base_b = (uint64_t)b.q + (uint64_t)n0 * b.ld, len_b = (uint64_t)(N - n0) * b.ld;
  const uint8_t* scale_a[IM];
#pragma unroll
  for (int I = 0; I < IM; ++I)
    scale_a[I] = a.scale + min(m0 + wm + 64 * I + 4 * r, (uint32_t)a.lds - 4);
  const uint8_t* scale_b = b.scale + min(n0 + wn, N - 1) / kQ8Block;

  auto load = [&](uint8_t* lds, uint32_t step) {
    const uint64_t k = (uint64_t)step * kQ8Block;
    const auto ra = rsrc_of(base_a + k, len_a - k), rb = rsrc_of(base_b + k, len_b - k);
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j)
      load_to_lds(ra, lds + (wave * kLoadsA + j) * 1024, from_a[j]);
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j)
      load_to_lds(rb, lds + TM * kQ8Block + (wave * kLoadsB + j) * 1024, from_b[j]);
  };
  auto load_scales = [&](uint32_t (&sa)[IM], uint32_t& sb, uint32_t step) {
#pragma unroll
    for (int I = 0; I < IM; ++I)
      sa[I] = *reinterpret_cast<const uint32_t*>(scale_a[I] + (uint64_t)step * a.lds);
    sb = scale_b[(uint64_t)step * b.lds];
  };

  f32x4 acc[4 * IM][4] = {};
  const uint32_t lo = r * kQ8Block + (2 * g ^ r / 2) * 16;
  const uint32_t hi = r * kQ8Block + ((2 * g + 1) ^ r / 2) * 16;
  auto frag = [&](const uint8_t* p) {
    return join(*reinterpret_cast<const u32x4*>(p + lo), *reinterpret_cast<const u32x4*>(p + hi));
  };
  auto multiply = [&](const uint8_t* lds, const uint32_t (&sa)[IM], uint32_t sb) {
    i32x8 fb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) fb[j] = frag(lds + (TM + wn + 16 * j) * kQ8Block);
    i32x8 fa = frag(lds + wm * kQ8Block);
#pragma unroll
    for (int i = 0; i < 4 * IM; ++i) {
      i32x8 next = fa;
      if (i + 1 < 4 * IM) next = frag(lds + (wm + 16 * (i + 1)) * kQ8Block);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = mma<FA, FB>(fb[j], fa, acc[i][j], sb, sa[i / 4], i % 4);
      fa = next;
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // codes at or beyond K in the last block of the sum
  auto clear_tail = [&](uint8_t* lds) {
    const int left = (int)(K % kQ8Block);
    for (uint32_t e = threadIdx.x; e < (TM + TN) * 8; e += 64 * kWaves) {
      const int keep = left - 16 * (int)(e % 8 ^ e / 16 % 8);
      if (keep >= 16) continue;
      u32x4* at = reinterpret_cast<u32x4*>(lds + e * 16);
      u32x4 v = *at;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        v[w] &= keep - 4 * w <= 0 ? 0u : keep - 4 * w >= 4 ? ~0u : (1u << 8 * (keep - 4 * w)) - 1;
      *at = v;
    }
    drain_and_sync();
  };

  uint32_t sa[IM], sb, sa_next[IM], sb_next;
  auto step = [&](uint8_t* here, uint8_t* there, uint32_t s) {
    if (s + 1 < s1) {
      load(there, s + 1);
      load_scales(sa_next, sb_next, s + 1);
    } else if ((s + 1) * kQ8Block > K) {
      clear_tail(here);
    }
    multiply(here, sa, sb);
    drain_and_sync();
#pragma unroll
    for (int I = 0; I < IM; ++I) sa[I] = sa_next[I];
    sb = sb_next;
  };
  if (s0 < s1) {
    load(lds, s0);
    load_scales(sa, sb, s0);
    drain_and_sync();
    uint32_t half = 0;
    for (uint32_t s = s0; s < s1; ++s) {
      step(lds + half, lds + (kBytes - half), s);
      half = kBytes - half;
    }
  }

  c.data = static_cast<uint8_t*>(c.data) + t.part * part_bytes;
#pragma unroll
  for (int i = 0; i < 4 * IM; ++i) {
    const uint32_t m = m0 + wm + 64 * (i / 4) + 4 * r + i % 4, n = n0 + wn + 16 * g;
    if (m >= M || n >= N) continue;
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = acc[i][e / 4][e % 4];
    if (c.dtype == S2R_F32)
      store16<S2R_F32>(static_cast<uint32_t*>(c.data) + (uint64_t)m * c.ld, n, N, v);
    else if (c.dtype == S2R_BF16)
      store16<S2R_BF16>(static_cast<uint16_t*>(c.data) + (uint64_t)m * c.ld, n, N, v);
    else
      store16<S2R_F16>(static_cast<uint16_t*>(c.data) + (uint64_t)m * c.ld, n, N, v);
  }
}

// ---- few rows -----------------------------------------------------------------------------
// Up to 16 FM rows of A: the rows of B are read once, straight into registers, and bound the
// call.  A workgroup takes 16 of them and cuts the sum among its waves, block by block in
// turn; the partial sums meet in LDS and are added in the order of the waves.
constexpr int kFewBatch = 2;  // blocks of the sum a wave has in flight

__device__ inline i32x8 load_frag(const uint8_t* row, uint32_t k, uint32_t K) {
  return join(load_codes16(row, k, K), load_codes16(row, k + 16, K));
}

template <int FA, int FB, int FM, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_q8_gemm_few(s2r_q8_mat a, s2r_q8_mat b, s2r_mat c,
                                                            uint32_t M, uint32_t N, uint32_t K) {
  __shared__ f32x4 part[WAVES][FM][64];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const uint32_t n0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * FM);
  const uint32_t n = min(n0 + r, N - 1);
  const uint8_t* rows_a[FM];
  uint32_t ms[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    ms[i] = min(m0 + 16 * i + r, M - 1);
    rows_a[i] = a.q + (uint64_t)ms[i] * a.ld;
  }
  const uint8_t* row_b = b.q + (uint64_t)n * b.ld;
  const uint8_t* scale_b = b.scale + n0 / kQ8Block;
  f32x4 acc[FM] = {};
  const uint32_t steps = (K + kQ8Block - 1) / kQ8Block;
  for (uint32_t s = wave; s < steps; s += WAVES * kFewBatch) {
    i32x8 fb[kFewBatch], fa[kFewBatch][FM];
    uint32_t sb[kFewBatch], sa[kFewBatch][FM];
#pragma unroll
    for (int e = 0; e < kFewBatch; ++e) {
      const uint32_t at = s + e * WAVES, k = at * kQ8Block + 32 * g;
      if (at >= steps) continue;
      fb[e] = load_frag(row_b, k, K);
      sb[e] = scale_b[(uint64_t)at * b.lds];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        fa[e][i] = load_frag(rows_a[i], k, K);
        sa[e][i] = a.scale[(uint64_t)at * a.lds + ms[i]];
      }
    }
#pragma unroll
    for (int e = 0; e < kFewBatch; ++e) {
      if (s + e * WAVES >= steps) continue;
#pragma unroll
      for (int i = 0; i < FM; ++i)
        acc[i] = mma<FA, FB>(fb[e], fa[e][i], acc[i], sb[e], sa[e][i], 0);
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < FM * 64; e += 64 * WAVES) {
    f32x4 v = part[0][e / 64][e % 64];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += part[w][e / 64][e % 64];
    const uint32_t m = m0 + e / 64 * 16 + e % 16, at = n0 + e % 64 / 16 * 4;
    if (m < M) store4(c, m, at, N, v);
  }
}

size_t q8_gemm_workspace(uint64_t, uint64_t, uint64_t) { return 0; }

namespace {

template <int FA, int FB>
void go_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat& a, const s2r_q8_mat& b,
             const s2r_mat& c, hipStream_t s) {
  const uint32_t m = (uint32_t)M, n = (uint32_t)N, k = (uint32_t)K;
  if (M <= 64) {
    trace_mark(s, "k_q8_gemm_few");
    const dim3 grid((n + 15) / 16);
    if (M <= 16)
      hipLaunchKernelGGL((k_q8_gemm_few<FA, FB, 1, 8>), grid, dim3(512), 0, s, a, b, c, m, n, k);
    else if (M <= 32)
      hipLaunchKernelGGL((k_q8_gemm_few<FA, FB, 2, 8>), grid, dim3(512), 0, s, a, b, c, m, n, k);
    else
      hipLaunchKernelGGL((k_q8_gemm_few<FA, FB, 4, 8>), grid, dim3(512), 0, s, a, b, c, m, n, k);
    return;
  }
  trace_mark(s, "k_q8_gemm");
  const uint32_t mt = (m + 255) / 256, nt = (n + 255) / 256, steps = (k + kQ8Block - 1) / kQ8Block;
  hipLaunchKernelGGL((k_q8_gemm<FA, FB, 2, 4, 2>), dim3(mt * nt), dim3(512), 0, s, a, b, c, 0, m, n,
                     k, mt, nt, steps);
}

}  // namespace

hipError_t launch_q8_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat& a,
                          const s2r_q8_mat& b, const s2r_mat& c, void*, hipStream_t s) {
  if (a.format == S2R_E4M3) {
    if (b.format == S2R_E4M3) go_gemm<S2R_E4M3, S2R_E4M3>(M, N, K, a, b, c, s);
    else go_gemm<S2R_E4M3, S2R_E5M2>(M, N, K, a, b, c, s);
  } else {
    if (b.format == S2R_E4M3) go_gemm<S2R_E5M2, S2R_E4M3>(M, N, K, a, b, c, s);
    else go_gemm<S2R_E5M2, S2R_E5M2>(M, N, K, a, b, c, s);
  }
  return hipGetLastError();
}

}  // namespace s2r
