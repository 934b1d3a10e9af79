// moe.hip -- tokens sorted by expert and back: s2r_moe_route, s2r_moe_gather, s2r_moe_combine and
// s2r_moe_combine_grad.
//
//   place[t][k] = first[e] + the number of choices of e before (t, k),  e = expert[t][k]
//   out[place[t][k]] = x[t]                      y[t] = sum_k w[t][k] rows[place[t][k]]
//   drows[place[t][k]] = w[t][k] dy[t]           dw[t][k] = dy[t] . rows[place[t][k]]
//
// Everything goes by tokens and not by rows: a token is read (or written) once, its K rows are
// whole lines wherever they lie, and no list of a row's token is needed.  Bound by HBM; measured on
// MI355X, where a large copy moves 5.18 TB/s:
//   gather 16384 x 4096 bf16, 4 choices, to 8 bits         81 us (5.0 TB/s); as it is 129 (5.2), both 210
//   combine 8192 x 4096 bf16, 4 choices                    68 us (4.9); 1001 x 1000 fp16, 6 choices 6.0
//   its gradient to 8 bits, with that of the weights       89 us (5.2); to bf16 116 (5.2), of fp32 to fp32 247 (4.9)
//   route 65536 choices among 64                           two launches of 4.8 us in a trace, 7.0 a call among others
//                                                          in a graph; 192 choices 2.8 and 3.0 in one launch
#include "moe_launch.hpp"
#include "q8_device.hpp"
#include "s2r_device.hpp"

namespace s2r {

// ---- route --------------------------------------------------------------------------------
// A stable counting sort.  A workgroup takes a chunk of choices, a wave a segment of it; counts of each
// expert by wave in LDS.  With several chunks a first launch leaves every chunk's counts, and
// each workgroup of the second adds up those before its own: integers, the same in any order.
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr uint64_t kRouteChunk = 2048;   // at least, of several
constexpr uint64_t kRouteAlone = 4096;   // choices up to which one workgroup takes them all
constexpr uint64_t kRouteChunks = 256;   // at most: one for every compute unit

struct RouteCut {
  uint32_t chunk, chunks;
};
// A call among others in a graph: 192 choices take 3.0 us, 2000 4.1, 4096 5.7 (6.3 in two chunks), 65536 7.0.
inline RouteCut route_cut(uint64_t A) {
  if (A <= kRouteAlone) return {A <= 1024 ? 1024u : A <= 2048 ? 2048u : 4096u, 1};
  uint64_t chunk = (A + kRouteChunks - 1) / kRouteChunks;
  chunk = (chunk + kRouteThreads - 1) / kRouteThreads * kRouteThreads;
  if (chunk < kRouteChunk) chunk = kRouteChunk;
  return {(uint32_t)chunk, (uint32_t)((A + chunk - 1) / chunk)};
}

__global__ __launch_bounds__(kRouteThreads) void k_moe_count(const int32_t* __restrict__ expert, uint32_t A,
                                                             uint32_t E, uint32_t chunk,
                                                             uint32_t* __restrict__ counts) {
  __shared__ uint32_t hist[S2R_MAX_EXPERTS];
  for (uint32_t e = threadIdx.x; e < E; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  const uint32_t begin = blockIdx.x * chunk, end = min(begin + chunk, A);
  for (uint32_t i = begin + threadIdx.x; i < end; i += kRouteThreads) {
    const uint32_t e = (uint32_t)expert[i];
    if (e < E) atomicAdd(&hist[e], 1u);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < E; e += kRouteThreads) counts[(uint64_t)blockIdx.x * E + e] = hist[e];
}

__device__ inline uint32_t up4(uint32_t n) { return (n + 3) & ~3u; }

// MOST: experts that LDS has room for.  counts: of every chunk, NULL where there is one.
template <int MOST>
__global__ __launch_bounds__(kRouteThreads) void k_moe_place(const int32_t* __restrict__ expert, uint32_t A,
                                                             uint32_t E, uint32_t chunk, uint32_t chunks,
                                                             const uint32_t* __restrict__ counts,
                                                             uint32_t* __restrict__ first,
                                                             uint32_t* __restrict__ rows,
                                                             int32_t* __restrict__ place) {
  __shared__ uint32_t hist[kRouteWaves][MOST];
  __shared__ uint32_t total[MOST], before[MOST], wave_sum[kRouteWaves];
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  for (uint32_t i = tid; i < kRouteWaves * MOST; i += kRouteThreads) hist[i / MOST][i % MOST] = 0;
  for (uint32_t e = tid; e < MOST; e += kRouteThreads) total[e] = 0, before[e] = 0;
  __syncthreads();
  const uint32_t segment = chunk / kRouteWaves;  // a multiple of 64
  const uint32_t from = blockIdx.x * chunk + wave * segment, end = min(from + segment, A);
  for (uint32_t i = from + lane; i < end; i += 64) {
    const uint32_t e = (uint32_t)expert[i];
    if (e < E) atomicAdd(&hist[wave][e], 1u);
  }
  __syncthreads();
  if (counts) {
    // as many experts side by side as there are, and the chunks in as many stripes as remain
    const uint32_t width = 1u << (32 - __builtin_clz(max(E, 2u) - 1)), stripes = kRouteThreads / width;
    const uint32_t e = tid % width;
    if (e < E) {
      uint32_t all = 0, mine = 0;
      for (uint32_t c = tid / width; c < chunks; c += stripes) {
        const uint32_t n = counts[(uint64_t)c * E + e];
        all += n;
        if (c < blockIdx.x) mine += n;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], mine);
    }
  } else if (tid < E) {
    uint32_t n = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) n += hist[w][tid];
    total[tid] = n;
  }
  __syncthreads();
  // first[e]: the sum of the experts before, one to a thread (kRouteThreads is S2R_MAX_EXPERTS)
  static_assert(kRouteThreads >= S2R_MAX_EXPERTS, "");
  const uint32_t n = tid < E ? total[tid] : 0;
  uint32_t sum = up4(n);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = (uint32_t)__shfl_up((int)sum, o);
    if (lane >= (uint32_t)o) sum += v;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  uint32_t at = sum - up4(n);
  for (uint32_t w = 0; w < wave; ++w) at += wave_sum[w];
  if (tid < E) {
    if (blockIdx.x == 0) {
      first[tid] = at;
      rows[tid] = n;
    }
    at += before[tid];
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
      const uint32_t count = hist[w][tid];
      hist[w][tid] = at;
      at += count;
    }
  }
  __syncthreads();
  // 64 choices at a time, in order: a lane's place is behind those of the lanes before it that chose
  // the same expert, which ballots over the bits of their numbers find
  volatile uint32_t* const next = hist[wave];
  for (uint32_t base = from; base < end; base += 64) {
    const uint32_t i = base + lane;
    const uint32_t e = i < end ? (uint32_t)expert[i] : ~0u;
    const bool some = e < E;
    uint64_t same = __ballot(some);
    for (uint32_t b = 0; (1u << b) < E; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      same &= (e >> b & 1) ? set : ~set;
    }
    const uint64_t ahead = same & ((1ull << lane) - 1);
    uint32_t p = 0;
    if (some) p = next[e];
    __builtin_amdgcn_wave_barrier();
    if (some && (same >> lane) == 1) next[e] = p + (uint32_t)__popcll(same);  // the last of them
    __builtin_amdgcn_wave_barrier();
    if (i < end) place[i] = some ? (int32_t)(p + (uint32_t)__popcll(ahead)) : -1;
  }
}

size_t moe_route_workspace(uint64_t T, uint32_t K, uint32_t E) {
  const RouteCut cut = route_cut(T * K);
  return cut.chunks > 1 ? (size_t)cut.chunks * E * sizeof(uint32_t) : 0;
}

hipError_t launch_moe_route(uint64_t T, uint32_t K, uint32_t E, const int32_t* expert,
                            uint32_t* first, uint32_t* rows, int32_t* place, void* workspace,
                            hipStream_t s) {
  const uint32_t A = (uint32_t)(T * K);
  const RouteCut cut = route_cut(A);
  uint32_t* counts = nullptr;
  if (cut.chunks > 1) {
    counts = static_cast<uint32_t*>(workspace);
    trace_mark(s, "k_moe_count");
    hipLaunchKernelGGL(k_moe_count, dim3(cut.chunks), dim3(kRouteThreads), 0, s, expert, A, E, cut.chunk, counts);
  }
  trace_mark(s, "k_moe_place");
  const dim3 grid(cut.chunks > 1 ? cut.chunks : 1);
  if (E <= 128)
    hipLaunchKernelGGL((k_moe_place<128>), grid, dim3(kRouteThreads), 0, s, expert, A, E, cut.chunk, cut.chunks,
                       counts, first, rows, place);
  else
    hipLaunchKernelGGL((k_moe_place<S2R_MAX_EXPERTS>), grid, dim3(kRouteThreads), 0, s, expert, A, E, cut.chunk,
                       cut.chunks, counts, first, rows, place);
  return hipGetLastError();
}

// ---- the choices of a token ----------------------------------------------------------------
constexpr int kMoeThreads = 256;
constexpr int kMoeWaves = kMoeThreads / 64;

// Lane k holds choice k's row and weight; ~0 where there is no row of the R.  They are asked for
// where all lanes run: the compiler may move their loads down to there.
struct Choices {
  uint32_t row;
  float weight;
  __device__ Choices(const int32_t* place, const float* w, uint32_t t, uint32_t K, uint32_t R) {
    const uint32_t lane = threadIdx.x % 64;
    const uint64_t at = (uint64_t)t * K + lane;
    row = lane < K ? (uint32_t)place[at] : ~0u;
    row = row < R ? row : ~0u;
    weight = w && lane < K ? w[at] : 1.0f;
  }
  __device__ uint32_t row_of(uint32_t k) const { return __builtin_amdgcn_readlane(row, k); }
  __device__ float weight_of(uint32_t k) const {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), k));
  }
};

// ---- gather -------------------------------------------------------------------------------
// A wave takes PIECES KB of a token's row to all of its choices' rows.  SIZE: of an element.
template <int SIZE, int PIECES>
__global__ __launch_bounds__(kMoeThreads) void k_moe_gather(const uint8_t* __restrict__ x, uint64_t ldx,
                                                            const int32_t* __restrict__ place, uint32_t T,
                                                            uint32_t K, uint32_t bytes, uint32_t R,
                                                            uint8_t* __restrict__ out, uint64_t ldo,
                                                            uint32_t spans) {
  const uint32_t span = blockIdx.x % spans, lane = threadIdx.x % 64;
  const uint32_t t = __builtin_amdgcn_readfirstlane(blockIdx.x / spans * kMoeWaves + threadIdx.x / 64);
  if (t >= T) return;
  const Choices of(place, nullptr, t, K, R);
  const uint32_t c = span * (PIECES * 1024) + lane * 16;
  const uint8_t* from = x + (uint64_t)t * ldx;
  u32x4 v[PIECES];
#pragma unroll
  for (int u = 0; u < PIECES; ++u)
    if (c + u * 1024 < bytes) v[u] = *reinterpret_cast<const u32x4*>(from + c + u * 1024);
  for (uint32_t k = 0; k < K; ++k) {
    const uint32_t row = of.row_of(k);
    if (row == ~0u) continue;
    uint8_t* const to = out + (uint64_t)row * ldo;
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      const uint32_t at = c + u * 1024;
      if (at + 16 <= bytes) {
        *reinterpret_cast<u32x4*>(to + at) = v[u];
      } else {
#pragma unroll
        for (int e = 0; e < 16 / SIZE; ++e) {
          if (at + e * SIZE >= bytes) continue;
          if (SIZE == 4) *reinterpret_cast<uint32_t*>(to + at + e * 4) = v[u][e % 4];
          else *reinterpret_cast<uint16_t*>(to + at + e * 2) = (uint16_t)(v[u][e / 2] >> 16 * (e % 2));
        }
      }
    }
  }
}

// The same in 8 bits: a wave takes 1024 columns, 16 to a lane, 8 lanes to a block of 128, and stores
// what it has once converted to every row.
template <int DT, int FMT>
__global__ __launch_bounds__(kMoeThreads) void k_moe_gather_q8(s2r_mat x, const int32_t* __restrict__ place,
                                                               uint32_t T, uint32_t K, uint32_t D, uint32_t R,
                                                               s2r_q8_mat out, uint32_t spans) {
  const uint32_t span = blockIdx.x % spans, lane = threadIdx.x % 64;
  const uint32_t t = __builtin_amdgcn_readfirstlane(blockIdx.x / spans * kMoeWaves + threadIdx.x / 64);
  if (t >= T) return;
  const Choices of(place, nullptr, t, K, R);
  const uint32_t c = span * 1024 + lane * 16;
  float v[16];
  unpack16<DT>(load_raw16<DT>(static_cast<const uint8_t*>(x.data) + (uint64_t)t * x.ld * elem_bytes<DT>(), c, D), v);
  const uint32_t sb = scale_byte<FMT>(max_over_8(amax16(v)));
  const u32x4 q = encode16<FMT>(v, sb);
  uint8_t* const scales = out.scale + (uint64_t)(c / kQ8Block) * out.lds;
  for (uint32_t k = 0; k < K; ++k) {
    const uint32_t row = of.row_of(k);
    if (row == ~0u || c >= D) continue;
    store_codes16(out.q + (uint64_t)row * out.ld, c, D, q);
    if (lane % 8 == 0) scales[row] = (uint8_t)sb;
  }
}

#define S2R_MOE_TYPES(dtype, CALL)                                \
  do {                                                            \
    if ((dtype) == S2R_BF16) { constexpr int DT = S2R_BF16; CALL; } \
    else if ((dtype) == S2R_F16) { constexpr int DT = S2R_F16; CALL; } \
    else { constexpr int DT = S2R_F32; CALL; }                    \
  } while (0)

hipError_t launch_moe_gather(uint64_t T, uint32_t K, uint64_t D, const s2r_mat& x,
                             const int32_t* place, uint64_t R, const s2r_mat* out,
                             const s2r_q8_mat* outq, hipStream_t s) {
  const uint64_t size = x.dtype == S2R_F32 ? 4 : 2;
  if (out) {
    // a token's row in pieces of 4 KB to a wave, or of 1 KB where that leaves compute units without one (24
    // tokens of 4 KB: 3.4 us, 4.6 in pieces of 4 KB)
    const uint64_t bytes = D * size;
    const bool few = T * ((bytes + 4095) / 4096) < 4 * 256;
    const uint64_t spans = few ? (bytes + 1023) / 1024 : (bytes + 4095) / 4096;
    trace_mark(s, "k_moe_gather");
    by_rows(T, kMoeWaves, spans, [&](uint64_t t, uint64_t n) {
      const s2r_mat f = from_row(x, t);
      const dim3 grid((uint32_t)(spans * ((n + kMoeWaves - 1) / kMoeWaves)));
#define S2R_GATHER(SIZE, PIECES)                                                                     \
  hipLaunchKernelGGL((k_moe_gather<SIZE, PIECES>), grid, dim3(kMoeThreads), 0, s,                    \
                     static_cast<const uint8_t*>(f.data), f.ld * size, place + t * K, (uint32_t)n, K, \
                     (uint32_t)bytes, (uint32_t)R, static_cast<uint8_t*>(out->data), out->ld * size, (uint32_t)spans)
      if (size == 4 && few) S2R_GATHER(4, 1);
      else if (size == 4) S2R_GATHER(4, 4);
      else if (few) S2R_GATHER(2, 1);
      else S2R_GATHER(2, 4);
#undef S2R_GATHER
    });
  }
  if (outq) {
    const uint64_t spans = (D + 1023) / 1024;
    trace_mark(s, "k_moe_gather_q8");
    by_rows(T, kMoeWaves, spans, [&](uint64_t t, uint64_t n) {
      const s2r_mat f = from_row(x, t);
      const dim3 grid((uint32_t)(spans * ((n + kMoeWaves - 1) / kMoeWaves)));
#define S2R_GATHER(FMT)                                                                            \
  S2R_MOE_TYPES(x.dtype, hipLaunchKernelGGL((k_moe_gather_q8<DT, FMT>), grid, dim3(kMoeThreads), 0, s, f, \
                                            place + t * K, (uint32_t)n, K, (uint32_t)D, (uint32_t)R, *outq, \
                                            (uint32_t)spans))
      if (outq->format == S2R_E4M3) S2R_GATHER(S2R_E4M3);
      else S2R_GATHER(S2R_E5M2);
#undef S2R_GATHER
    });
  }
  return hipGetLastError();
}

// ---- combine ------------------------------------------------------------------------------
// Eight values of a row from column c on; those at or beyond `cols` are whatever the row's padding
// holds, and zeros beyond its last 16-byte piece.
template <int DT>
__device__ inline void load8(const uint8_t* row, uint32_t c, uint32_t cols, float (&v)[8]) {
  if (DT == S2R_F32) {
    const float* p = reinterpret_cast<const float*>(row) + c;
    const f32x4 z = {0, 0, 0, 0};
    const f32x4 lo = c < cols ? *reinterpret_cast<const f32x4*>(p) : z;
    const f32x4 hi = c + 4 < cols ? *reinterpret_cast<const f32x4*>(p + 4) : z;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
    return;
  }
  u32x4 r = {0, 0, 0, 0};
  if (c < cols) r = *reinterpret_cast<const u32x4*>(row + 2 * c);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (DT == S2R_BF16) {
      v[2 * w] = __uint_as_float(r[w] << 16);
      v[2 * w + 1] = __uint_as_float(r[w] & 0xffff0000u);
    } else {
      const f16x2 h = __builtin_bit_cast(f16x2, (uint32_t)r[w]);
      v[2 * w] = (float)h[0];
      v[2 * w + 1] = (float)h[1];
    }
  }
}

// A wave takes PIECES x 512 columns of a token, eight to a lane at a time, and reads ROWS of its rows at once.
template <int DT, int PIECES, int ROWS>
__global__ __launch_bounds__(kMoeThreads) void k_moe_combine(s2r_mat rows, uint32_t R,
                                                             const int32_t* __restrict__ place,
                                                             const float* __restrict__ weight, uint32_t T,
                                                             uint32_t K, uint32_t D, s2r_mat y, uint32_t spans) {
  const uint32_t span = blockIdx.x % spans, lane = threadIdx.x % 64;
  const uint32_t t = __builtin_amdgcn_readfirstlane(blockIdx.x / spans * kMoeWaves + threadIdx.x / 64);
  if (t >= T) return;
  const Choices of(place, weight, t, K, R);
  const uint32_t c = span * (PIECES * 512) + lane * 8;
  const uint64_t ld = rows.ld * elem_bytes<DT>();
  float sum[PIECES][8] = {};
  for (uint32_t k0 = 0; k0 < K; k0 += ROWS) {
    float v[ROWS][PIECES][8];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const uint32_t row = k0 + j < K ? of.row_of(k0 + j) : ~0u;
      if (row == ~0u) continue;
      const uint8_t* from = static_cast<const uint8_t*>(rows.data) + (uint64_t)row * ld;
#pragma unroll
      for (int u = 0; u < PIECES; ++u) load8<DT>(from, c + 512 * u, D, v[j][u]);
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if (k0 + j >= K || of.row_of(k0 + j) == ~0u) continue;  // the same for the wave
      const float w = of.weight_of(k0 + j);
#pragma unroll
      for (int u = 0; u < PIECES; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[u][e] = __builtin_fmaf(w, v[j][u][e], sum[u][e]);
    }
  }
#pragma unroll
  for (int u = 0; u < PIECES; ++u) {
    const f32x4 lo = {sum[u][0], sum[u][1], sum[u][2], sum[u][3]}, hi = {sum[u][4], sum[u][5], sum[u][6], sum[u][7]};
    if (c + 512 * u < D) store8(y, t, c + 512 * u, D, lo, hi);
  }
}

hipError_t launch_moe_combine(uint64_t T, uint32_t K, uint64_t D, const s2r_mat& rows, uint64_t R,
                              const int32_t* place, const float* weight, const s2r_mat& y,
                              hipStream_t s) {
  // 1024 columns to a wave, or 512 with more rows at once where that leaves compute units idle
  const bool few = T * ((D + 1023) / 1024) < 16 * 256;
  const uint64_t each = few ? 512 : 1024, spans = (D + each - 1) / each;
  trace_mark(s, "k_moe_combine");
  by_rows(T, kMoeWaves, spans, [&](uint64_t t, uint64_t n) {
    const s2r_mat to = from_row(y, t);
    const dim3 grid((uint32_t)(spans * ((n + kMoeWaves - 1) / kMoeWaves)));
#define S2R_COMBINE(PIECES, ROWS)                                                                                  \
  S2R_MOE_TYPES(rows.dtype, hipLaunchKernelGGL((k_moe_combine<DT, PIECES, ROWS>), grid, dim3(kMoeThreads), 0, s, rows, \
                                               (uint32_t)R, place + t * K, weight ? weight + t * K : nullptr,      \
                                               (uint32_t)n, K, (uint32_t)D, to, (uint32_t)spans))
    if (few) S2R_COMBINE(1, 8);
    else S2R_COMBINE(2, 4);
#undef S2R_COMBINE
  });
  return hipGetLastError();
}

// ---- its gradient ---------------------------------------------------------------------------
// WAVES waves to a token, 16 columns to a lane at a time as the 8-bit blocks want it; kGradRows choices
// at once.  A weight's gradient is added up in a lane over its columns, then over the lanes, then
// over the waves.
constexpr int kGradRows = 4;

struct GradOut {
  s2r_mat rows, drows;   // data NULL: not wanted
  s2r_q8_mat drowsq;
  float* dweight;
};

__device__ inline void store16_as(const s2r_mat& m, uint32_t row, uint32_t c, uint32_t cols, const float (&v)[16]) {
  uint8_t* const to = static_cast<uint8_t*>(m.data) + (uint64_t)row * m.ld * (m.dtype == S2R_F32 ? 4 : 2);
  if (m.dtype == S2R_BF16) store16<S2R_BF16>(to, c, cols, v);
  else if (m.dtype == S2R_F16) store16<S2R_F16>(to, c, cols, v);
  else store16<S2R_F32>(to, c, cols, v);
}

// FMT: of drowsq, -1 without it
template <int DT, int FMT, int WAVES>
__global__ __launch_bounds__(kMoeThreads) void k_moe_combine_grad(s2r_mat dy, const int32_t* __restrict__ place,
                                                                  const float* __restrict__ weight, uint32_t T,
                                                                  uint32_t K, uint32_t D, uint32_t R, GradOut o) {
  __shared__ float part[kMoeWaves][S2R_MAX_CHOICES];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t t = __builtin_amdgcn_readfirstlane(blockIdx.x * (kMoeWaves / WAVES) + wave / WAVES);
  if (t < T) {
    const Choices of(place, weight, t, K, R);
    const uint8_t* from = static_cast<const uint8_t*>(dy.data) + (uint64_t)t * dy.ld * elem_bytes<DT>();
    for (uint32_t k0 = 0; k0 < K; k0 += kGradRows) {
      uint32_t row[kGradRows];
      float w[kGradRows], dot[kGradRows] = {};
#pragma unroll
      for (int j = 0; j < kGradRows; ++j) {
        row[j] = k0 + j < K ? of.row_of(k0 + j) : ~0u;
        w[j] = of.weight_of((k0 + j) % 64);
      }
      for (uint32_t c = wave % WAVES * 1024 + lane * 16; c < (D + 127) / 128 * 128; c += WAVES * 1024) {
        const Raw16<DT> d = load_raw16<DT>(from, c, D);
        Raw16<DT> r[kGradRows];
        if (o.dweight) {
#pragma unroll
          for (int j = 0; j < kGradRows; ++j) {
            if (row[j] == ~0u) continue;
            r[j] = load_raw16<DT>(static_cast<const uint8_t*>(o.rows.data) +
                                      (uint64_t)row[j] * o.rows.ld * elem_bytes<DT>(), c, D);
          }
        }
        float v[16];
        unpack16<DT>(d, v);
#pragma unroll
        for (int j = 0; j < kGradRows; ++j) {
          if (row[j] == ~0u) continue;
          if (o.dweight) {
            float x[16];
            unpack16<DT>(r[j], x);
#pragma unroll
            for (int e = 0; e < 16; ++e) dot[j] = __builtin_fmaf(v[e], x[e], dot[j]);
          }
          float g[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) g[e] = w[j] * v[e];
          if (o.drows.data && c < D) store16_as(o.drows, row[j], c, D, g);
          if (FMT >= 0) {
            constexpr int F = FMT < 0 ? S2R_E4M3 : FMT;
            const uint32_t sb = scale_byte<F>(max_over_8(amax16(g)));
            if (c < D) {
              store_codes16(o.drowsq.q + (uint64_t)row[j] * o.drowsq.ld, c, D, encode16<F>(g, sb));
              if (lane % 8 == 0) o.drowsq.scale[(uint64_t)(c / kQ8Block) * o.drowsq.lds + row[j]] = (uint8_t)sb;
            }
          }
        }
      }
      if (o.dweight) {
#pragma unroll
        for (int j = 0; j < kGradRows; ++j) {
#pragma unroll
          for (int m = 32; m > 0; m >>= 1) dot[j] += __shfl_xor(dot[j], m);
          if (lane == 0 && k0 + j < K) part[wave][k0 + j] = dot[j];
        }
      }
    }
  }
  if (!o.dweight) return;
  __syncthreads();
  if (t < T && wave % WAVES == 0 && lane < K) {
    float sum = part[wave][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[wave + w][lane];
    o.dweight[(uint64_t)t * K + lane] = sum;
  }
}

hipError_t launch_moe_combine_grad(uint64_t T, uint32_t K, uint64_t D, const s2r_mat& dy,
                                   const int32_t* place, uint64_t R, const float* weight,
                                   const s2r_mat* rows, const s2r_mat* drows,
                                   const s2r_q8_mat* drowsq, float* dweight, hipStream_t s) {
  const int waves = D <= 1024 ? 1 : D <= 2048 ? 2 : 4;
  const uint64_t each = kMoeWaves / waves;
  trace_mark(s, "k_moe_combine_grad");
  by_rows(T, each, 1, [&](uint64_t t, uint64_t n) {
    const s2r_mat f = from_row(dy, t);
    const GradOut o = {rows ? *rows : s2r_mat{}, drows ? *drows : s2r_mat{}, drowsq ? *drowsq : s2r_q8_mat{},
                       dweight ? dweight + t * K : nullptr};
    const dim3 grid((uint32_t)((n + each - 1) / each));
#define S2R_GRAD(FMT, WAVES)                                                                            \
  S2R_MOE_TYPES(dy.dtype, hipLaunchKernelGGL((k_moe_combine_grad<DT, FMT, WAVES>), grid, dim3(kMoeThreads), 0, s, f, \
                                             place + t * K, weight ? weight + t * K : nullptr, (uint32_t)n, K, \
                                             (uint32_t)D, (uint32_t)R, o))
#define S2R_GRAD_WAVES(FMT)              \
  do {                                   \
    if (waves == 1) S2R_GRAD(FMT, 1);    \
    else if (waves == 2) S2R_GRAD(FMT, 2); \
    else S2R_GRAD(FMT, 4);               \
  } while (0)
    if (!drowsq) S2R_GRAD_WAVES(-1);
    else if (drowsq->format == S2R_E4M3) S2R_GRAD_WAVES(S2R_E4M3);
    else S2R_GRAD_WAVES(S2R_E5M2);
#undef S2R_GRAD_WAVES
#undef S2R_GRAD
  });
  return hipGetLastError();
}

}  // namespace s2r
