// q8_glu.hip -- the activation of a feed-forward layer with 8-bit checkpoints, and its
// gradient from them: s2r_q8_glu, s2r_q8_glu_grad.
//
//   forward   y = act(g) u;  g, u and y leave in 8 bits (and y in 16 or 32 if asked)
//   backward  dg = dy u act'(g), du = dy act(g), with g and u as stored
// act and act' share their transcendental:
//   SiLU       s = 1 / (1 + e^-g):           act = g s,  act' = s (1 + g (1 - s))
//   GELU       c = Phi(g):                   act = g c,  act' = c + g e^(-g^2 / 2) / sqrt(2 pi)
//   GELU_TANH  s = 1 / (1 + e^(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3), which is
//              (1 + tanh z) / 2:             act = g s,  act' = s + g s (1 - s) 2 z'
// Element-wise apart from the blocks' largest magnitudes: one read and one write of
// everything, bound by HBM and, where arithmetic comes close, by both.  Measured on MI355X: gated SiLU of
// 8192 x 8192 bf16 with its three 8-bit results 88 us (5.3 TB/s), its gradient 86 us (4.7); with the
// library's exponential and division the gradient took 97.  GELU_TANH takes 90 and 93, GELU 96 and
// 100, bound by arithmetic (98% and 95% of the vector instructions that the cycles hold); with the
// library's error function, whose 1 + erf has no digits left far below zero, GELU took 89 and 108.
#include "q8_device.hpp"
#include "q8_launch.hpp"

namespace s2r {

constexpr int kGluThreads = 256;
constexpr int kGluRows = kGluThreads / 8;
constexpr int kGluBlocks = 2;  // blocks of 128 columns per workgroup: two or three streams each

// e^x within two units in the last place for |x| up to 200: x log2(e) is cut into a whole number and a
// rest that keeps its low bits, and the hardware's 2^x (one unit) takes the rest.  Without that the
// argument's rounding alone costs |x| half units, and a result next to a border of the 8-bit
// grid falls to the other side that much more often.  Beyond that e^x is infinite or zero, as it is at
// 200; a NaN gets lost there, but what exp_of's callers multiply it with is the same NaN.
__device__ inline float exp_within_200(float x) {
  const float n = __builtin_rintf(x * 1.44269504088896f);
  float r = __builtin_fmaf(x, 1.44269504088896f, -n);
  r = __builtin_fmaf(x, 1.925963033500e-8f, r);  // log2(e) beyond 24 bits
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(r), (int)n);
}
__device__ inline float exp_of(float x) {
  return exp_within_200(__builtin_amdgcn_fmed3f(x, -200.0f, 200.0f));
}

// s = 1 / (1 + e^-x) by the hardware's reciprocal with one step of Newton's, and 1 - s as e^-x s: where s
// is near 1 the subtraction would leave few digits.
__device__ inline float sigmoid(float x, float& rest) {
  const float e = exp_of(-x), d = 1.0f + e, r = __builtin_amdgcn_rcpf(d);
  const bool finite = d < __builtin_inff();
  const float s = finite ? __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r) : r;
  rest = finite ? e * s : 1.0f;
  return s;
}

// Phi(g), the normal distribution's integral, and e = e^(-g^2 / 2).  Phi(-a) = e h(a), where h falls
// slowly from 1/2 like 1 / (a sqrt(2 pi)) and so keeps all digits however small Phi is: a quotient
// of polynomials fitted to it over [0, 14.5] in relative error (least squares of the linearised quotient,
// reweighted by the last quotient's denominator and by Lawson's rule until the error is level:
// 6e-9), all of its coefficients positive.  The rest of a^2 that its rounding loses comes back by
// a factor; from a = 14.5 on e is 0 in fp32.  A NaN gets lost as in exp_of.
__device__ inline float normal_cdf(float g, float& e) {
  const float a = __builtin_amdgcn_fmed3f(__builtin_fabsf(g), 0.0f, 15.0f);
  float n = 4.11623903e-3f, d = 1.03177615e-2f;
  n = __builtin_fmaf(n, a, 4.06327881e-2f);
  d = __builtin_fmaf(d, a, 1.01857744e-1f);
  n = __builtin_fmaf(n, a, 1.83233887e-1f);
  d = __builtin_fmaf(d, a, 4.69467312e-1f);
  n = __builtin_fmaf(n, a, 4.38293338e-1f);
  d = __builtin_fmaf(d, a, 1.20249808f);
  n = __builtin_fmaf(n, a, 0.5f);
  d = __builtin_fmaf(d, a, 1.67447162f);
  d = __builtin_fmaf(d, a, 1.0f);
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  const float sq = a * a, rest = __builtin_fmaf(a, a, -sq);
  e = exp_within_200(-0.5f * sq);
  e = __builtin_fmaf(-0.5f * e, rest, e);
  const float tail = e * (n * r);
  return g < 0 ? tail : 1.0f - tail;
}

// 2 z of GELU_TANH, and cubic = 0.044715 g^2.  g^2 is taken no further than 16^2, where the sigmoid
// has long been 0 or 1: an infinite one would meet s (1 - s) = 0 in the derivative.
__device__ inline float tanh_argument(float g, float& cubic) {
  const float h = __builtin_amdgcn_fmed3f(g, -16.0f, 16.0f);
  cubic = 0.044715f * h * h;
  return 1.5957691216057308f * g * (1.0f + cubic);
}

template <int ACT>
__device__ inline float act_value(float g) {
  float rest;
  if (ACT == S2R_ACT_SILU) return g * sigmoid(g, rest);
  if (ACT == S2R_ACT_GELU) {
    float e;
    return g * normal_cdf(g, e);
  }
  float cubic;
  return g * sigmoid(tanh_argument(g, cubic), rest);
}

template <int ACT>
__device__ inline void act_both(float g, float& a, float& d) {
  if (ACT == S2R_ACT_SILU) {
    float rest;
    const float s = sigmoid(g, rest);
    a = g * s;
    d = s * (1.0f + g * rest);
  } else if (ACT == S2R_ACT_GELU) {
    float e;
    const float c = normal_cdf(g, e);
    a = g * c;
    d = c + g * (e * 0.39894228040143268f);
  } else {
    float cubic, rest;
    const float s = sigmoid(tanh_argument(g, cubic), rest);
    a = g * s;
    d = s + a * rest * (1.5957691216057308f * (1.0f + 3.0f * cubic));
  }
}

// Where 16 columns of one row go: in 8 bits, their block's scale over 8 lanes, ...
__device__ inline void put8(const s2r_q8_mat& o, uint32_t m, uint32_t c, uint32_t F,
                            const float (&v)[16]) {
  const uint32_t am = max_over_8(amax16(v));
  uint32_t sb;
  u32x4 code;
  if (o.format == S2R_E4M3) {
    sb = scale_byte<S2R_E4M3>(am);
    code = encode16<S2R_E4M3>(v, sb);
  } else {
    sb = scale_byte<S2R_E5M2>(am);
    code = encode16<S2R_E5M2>(v, sb);
  }
  if (c >= F) return;
  store_codes16(o.q + (uint64_t)m * o.ld, c, F, code);
  if (threadIdx.x % 8 == 0) o.scale[(uint64_t)(c / kQ8Block) * o.lds + m] = (uint8_t)sb;
}

// ... or in 16 or 32.
__device__ inline void put(const s2r_mat& o, uint32_t m, uint32_t c, uint32_t F,
                           const float (&v)[16]) {
  if (c >= F) return;
  if (o.dtype == S2R_BF16)
    store16<S2R_BF16>(static_cast<uint16_t*>(o.data) + (uint64_t)m * o.ld, c, F, v);
  else if (o.dtype == S2R_F16)
    store16<S2R_F16>(static_cast<uint16_t*>(o.data) + (uint64_t)m * o.ld, c, F, v);
  else
    store16<S2R_F32>(static_cast<uint32_t*>(o.data) + (uint64_t)m * o.ld, c, F, v);
}

// Outputs that the caller left out have a null pointer.
template <int DT, int ACT, bool GATED>
__global__ __launch_bounds__(kGluThreads) void k_q8_glu(
    const void* __restrict__ g, uint64_t ldg, const void* __restrict__ u, uint64_t ldu,
    s2r_q8_mat gq, s2r_q8_mat uq, s2r_mat y, s2r_q8_mat yq, uint32_t M, uint32_t F,
    uint32_t col_tiles) {
  using E = typename ElemT<DT>::type;
  const uint32_t ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
  const uint32_t m = rt * kGluRows + threadIdx.x / 8;
  if (m >= M) return;  // whole groups of 8 lanes leave together
  const uint32_t c0 = ct * (kGluBlocks * kQ8Block) + (threadIdx.x % 8) * 16;
  const E* grow = static_cast<const E*>(g) + (uint64_t)m * ldg;
  const E* urow = GATED ? static_cast<const E*>(u) + (uint64_t)m * ldu : nullptr;
  Raw16<DT> rg[kGluBlocks], ru[GATED ? kGluBlocks : 1];
#pragma unroll
  for (int b = 0; b < kGluBlocks; ++b) {
    rg[b] = load_raw16<DT>(grow, c0 + b * kQ8Block, F);
    if (GATED) ru[b] = load_raw16<DT>(urow, c0 + b * kQ8Block, F);
  }
#pragma unroll
  for (int b = 0; b < kGluBlocks; ++b) {
    const uint32_t c = c0 + b * kQ8Block;
    float v[16], w[16];
    unpack16<DT>(rg[b], v);
    if (gq.q) put8(gq, m, c, F, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = act_value<ACT>(v[i]);
    if (GATED) {
      unpack16<DT>(ru[b], w);
      if (uq.q) put8(uq, m, c, F, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= w[i];
    }
    if (y.data) put(y, m, c, F, v);
    if (yq.q) put8(yq, m, c, F, v);
  }
}

template <int FMT, int ACT, bool GATED>
__global__ __launch_bounds__(kGluThreads) void k_q8_glu_grad(
    s2r_q8_mat gq, s2r_q8_mat uq, s2r_mat dy, s2r_mat dg, s2r_mat du, s2r_q8_mat dgq,
    s2r_q8_mat duq, uint32_t M, uint32_t F, uint32_t col_tiles) {
  const uint32_t ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
  const uint32_t m = rt * kGluRows + threadIdx.x / 8;
  if (m >= M) return;
  const uint32_t c0 = ct * (kGluBlocks * kQ8Block) + (threadIdx.x % 8) * 16;
  u32x4 cg[kGluBlocks], cu[GATED ? kGluBlocks : 1];
  uint32_t sg[kGluBlocks], su[GATED ? kGluBlocks : 1];
  Raw16<S2R_BF16> r16[kGluBlocks];
  Raw16<S2R_F32> r32[kGluBlocks];
  const bool wide = dy.dtype == S2R_F32;
#pragma unroll
  for (int b = 0; b < kGluBlocks; ++b) {
    const uint32_t c = c0 + b * kQ8Block;
    const uint64_t sat = (uint64_t)(c / kQ8Block);
    cg[b] = load_codes16(gq.q + (uint64_t)m * gq.ld, c, F);
    sg[b] = c < F ? gq.scale[sat * gq.lds + m] : 127;
    if (GATED) {
      cu[b] = load_codes16(uq.q + (uint64_t)m * uq.ld, c, F);
      su[b] = c < F ? uq.scale[sat * uq.lds + m] : 127;
    }
    if (wide)
      r32[b] = load_raw16<S2R_F32>(static_cast<const uint32_t*>(dy.data) + (uint64_t)m * dy.ld, c, F);
    else
      r16[b] = load_raw16<S2R_BF16>(static_cast<const uint16_t*>(dy.data) + (uint64_t)m * dy.ld, c, F);
  }
#pragma unroll
  for (int b = 0; b < kGluBlocks; ++b) {
    const uint32_t c = c0 + b * kQ8Block;
    float t[16], vg[16], vu[16];
    if (wide) {
      unpack16<S2R_F32>(r32[b], t);
    } else if (dy.dtype == S2R_BF16) {
      unpack16<S2R_BF16>(r16[b], t);
    } else {
      unpack16<S2R_F16>(__builtin_bit_cast(Raw16<S2R_F16>, r16[b]), t);
    }
    decode16<FMT>(cg[b], scale_value(sg[b]), vg);
    if (GATED) decode16<FMT>(cu[b], scale_value(su[b]), vu);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a, d;
      act_both<ACT>(vg[i], a, d);
      if (GATED) {
        vg[i] = t[i] * vu[i] * d;
        vu[i] = t[i] * a;
      } else {
        vg[i] = t[i] * d;
      }
    }
    if (dg.data) put(dg, m, c, F, vg);
    if (dgq.q) put8(dgq, m, c, F, vg);
    if (GATED) {
      if (du.data) put(du, m, c, F, vu);
      if (duq.q) put8(duq, m, c, F, vu);
    }
  }
}

namespace {

template <int DT, int ACT>
void go_glu(uint32_t grid, hipStream_t s, uint64_t M, uint64_t F, uint32_t ct, const s2r_mat& g,
            const s2r_mat* u, const s2r_q8_mat& gq, const s2r_q8_mat& uq, const s2r_mat& y,
            const s2r_q8_mat& yq) {
  if (u)
    hipLaunchKernelGGL((k_q8_glu<DT, ACT, true>), dim3(grid), dim3(kGluThreads), 0, s, g.data, g.ld,
                       u->data, u->ld, gq, uq, y, yq, (uint32_t)M, (uint32_t)F, ct);
  else
    hipLaunchKernelGGL((k_q8_glu<DT, ACT, false>), dim3(grid), dim3(kGluThreads), 0, s, g.data,
                       g.ld, nullptr, 0, gq, uq, y, yq, (uint32_t)M, (uint32_t)F, ct);
}

template <int FMT, int ACT>
void go_grad(uint32_t grid, hipStream_t s, uint64_t M, uint64_t F, uint32_t ct,
             const s2r_q8_mat& gq, const s2r_q8_mat* uq, const s2r_mat& dy, const s2r_mat& dg,
             const s2r_mat& du, const s2r_q8_mat& dgq, const s2r_q8_mat& duq) {
  if (uq)
    hipLaunchKernelGGL((k_q8_glu_grad<FMT, ACT, true>), dim3(grid), dim3(kGluThreads), 0, s, gq, *uq,
                       dy, dg, du, dgq, duq, (uint32_t)M, (uint32_t)F, ct);
  else
    hipLaunchKernelGGL((k_q8_glu_grad<FMT, ACT, false>), dim3(grid), dim3(kGluThreads), 0, s, gq,
                       s2r_q8_mat{}, dy, dg, du, dgq, duq, (uint32_t)M, (uint32_t)F, ct);
}

#define S2R_Q8_ACT(act, CALL)                                              \
  do {                                                                     \
    if ((act) == S2R_ACT_SILU) { constexpr int ACT = S2R_ACT_SILU; CALL; } \
    else if ((act) == S2R_ACT_GELU) { constexpr int ACT = S2R_ACT_GELU; CALL; } \
    else { constexpr int ACT = S2R_ACT_GELU_TANH; CALL; }                  \
  } while (0)

inline s2r_q8_mat or_none(const s2r_q8_mat* m) { return m ? *m : s2r_q8_mat{}; }
inline s2r_mat or_none(const s2r_mat* m) { return m ? *m : s2r_mat{}; }

}  // namespace

hipError_t launch_q8_glu(uint64_t M, uint64_t F, s2r_act act, const s2r_mat& g, const s2r_mat* u,
                         const s2r_q8_mat* gq, const s2r_q8_mat* uq, const s2r_mat* y,
                         const s2r_q8_mat* yq, hipStream_t s) {
  const uint32_t ct = (uint32_t)((F + kGluBlocks * kQ8Block - 1) / (kGluBlocks * kQ8Block));
  trace_mark(s, "k_q8_glu");
  by_rows(M, kGluRows, ct, [&](uint64_t m, uint64_t rows) {
    const uint32_t grid = (uint32_t)((rows + kGluRows - 1) / kGluRows * ct);
    const s2r_mat from = from_row(g, m), up = from_row(or_none(u), m), d = from_row(or_none(y), m);
    const s2r_mat* const gate = u ? &up : nullptr;
    const s2r_q8_mat a = from_row(or_none(gq), m), b = from_row(or_none(uq), m),
                     c = from_row(or_none(yq), m);
    if (g.dtype == S2R_BF16)
      S2R_Q8_ACT(act, (go_glu<S2R_BF16, ACT>(grid, s, rows, F, ct, from, gate, a, b, d, c)));
    else if (g.dtype == S2R_F16)
      S2R_Q8_ACT(act, (go_glu<S2R_F16, ACT>(grid, s, rows, F, ct, from, gate, a, b, d, c)));
    else
      S2R_Q8_ACT(act, (go_glu<S2R_F32, ACT>(grid, s, rows, F, ct, from, gate, a, b, d, c)));
  });
  return hipGetLastError();
}

hipError_t launch_q8_glu_grad(uint64_t M, uint64_t F, s2r_act act, const s2r_q8_mat& gq,
                              const s2r_q8_mat* uq, const s2r_mat& dy, const s2r_mat* dg,
                              const s2r_mat* du, const s2r_q8_mat* dgq, const s2r_q8_mat* duq,
                              hipStream_t s) {
  const uint32_t ct = (uint32_t)((F + kGluBlocks * kQ8Block - 1) / (kGluBlocks * kQ8Block));
  trace_mark(s, "k_q8_glu_grad");
  by_rows(M, kGluRows, ct, [&](uint64_t m, uint64_t rows) {
    const uint32_t grid = (uint32_t)((rows + kGluRows - 1) / kGluRows * ct);
    const s2r_q8_mat from = from_row(gq, m), up = from_row(or_none(uq), m);
    const s2r_q8_mat* const gate = uq ? &up : nullptr;
    const s2r_mat dym = from_row(dy, m), a = from_row(or_none(dg), m), b = from_row(or_none(du), m);
    const s2r_q8_mat c = from_row(or_none(dgq), m), d = from_row(or_none(duq), m);
    if (gq.format == S2R_E4M3)
      S2R_Q8_ACT(act, (go_grad<S2R_E4M3, ACT>(grid, s, rows, F, ct, from, gate, dym, a, b, c, d)));
    else
      S2R_Q8_ACT(act, (go_grad<S2R_E5M2, ACT>(grid, s, rows, F, ct, from, gate, dym, a, b, c, d)));
  });
  return hipGetLastError();
}

}  // namespace s2r
