// moe_api.hip -- the C entry points of s2r_moe.h: argument checks on the host, then the launch.
#include "checks.hpp"
#include "moe_launch.hpp"

using namespace s2r;

namespace {

constexpr uint64_t kMaxChoices = 1ull << 27;

inline bool choices_ok(uint64_t T, uint32_t K, uint32_t E = 1) {
  return K >= 1 && K <= S2R_MAX_CHOICES && E >= 1 && E <= S2R_MAX_EXPERTS && T < kMaxChoices &&
         T * K < kMaxChoices;
}

// What the calls over tokens and rows share: the sizes, and a place for every choice.
void check_choices(Verdict& v, uint64_t T, uint32_t K, uint64_t D, uint64_t R, const int32_t* place) {
  if (!choices_ok(T, K) || !sizes_ok(D, R)) v.add(S2R_ERR_DIM);
  if (T > 0 && D > 0 && !place) v.add(S2R_ERR_NULL);
  if (!aligned(place, 4)) v.add(S2R_ERR_ALIGN);
}

void check_experts(Verdict& v, const s2r_experts* e) {
  if (!e->first || !e->rows) v.add(S2R_ERR_NULL);
  if (e->experts < 1 || e->experts > S2R_MAX_EXPERTS) v.add(S2R_ERR_DIM);
  if (!aligned(e->first, 4) || !aligned(e->rows, 4)) v.add(S2R_ERR_ALIGN);
}

}  // namespace

extern "C" {

uint64_t s2r_moe_rows(uint64_t T, uint32_t K, uint32_t E) {
  if (!choices_ok(T, K, E)) return 0;
  const uint64_t A = T * K;
  return (A + 3 * (E < A ? E : A)) / 4 * 4;
}

size_t s2r_moe_route_workspace_bytes(uint64_t T, uint32_t K, uint32_t E) {
  return choices_ok(T, K, E) ? moe_route_workspace(T, K, E) : 0;
}

s2r_status s2r_moe_route(uint64_t T, uint32_t K, uint32_t E, const int32_t* expert,
                         uint32_t* first, uint32_t* rows, int32_t* place, void* workspace,
                         size_t ws_bytes, void* stream) {
  Verdict v;
  if (!first || !rows || (T > 0 && (!expert || !place))) v.add(S2R_ERR_NULL);
  if (!choices_ok(T, K, E)) v.add(S2R_ERR_DIM);
  if (!aligned(expert, 4) || !aligned(first, 4) || !aligned(rows, 4) || !aligned(place, 4))
    v.add(S2R_ERR_ALIGN);
  if (v.st != S2R_OK) return v.st;
  const size_t need = moe_route_workspace(T, K, E);
  if (need && !aligned(workspace, 16)) return S2R_ERR_ALIGN;
  if (need && (!workspace || ws_bytes < need)) return S2R_ERR_WORKSPACE;
  return done(launch_moe_route(T, K, E, expert, first, rows, place, workspace, on(stream)), stream);
}

s2r_status s2r_moe_gather(uint64_t T, uint32_t K, uint64_t D, const s2r_mat* x,
                          const int32_t* place, uint64_t R, const s2r_mat* out,
                          const s2r_q8_mat* outq, void* stream) {
  if (!x || (!out && !outq)) return S2R_ERR_NULL;
  Verdict v;
  check_choices(v, T, K, D, R, place);
  v.add(check(x, T, D));
  if (out) {
    v.add(check(out, R, D));
    if (out->dtype != x->dtype) v.add(S2R_ERR_DIM);
  }
  if (outq) v.add(check(outq, R, D, R));
  if (v.st != S2R_OK) return v.st;
  if (T == 0 || D == 0 || R == 0) return S2R_OK;
  return done(launch_moe_gather(T, K, D, *x, place, R, out, outq, on(stream)), stream);
}

s2r_status s2r_moe_combine(uint64_t T, uint32_t K, uint64_t D, const s2r_mat* rows, uint64_t R,
                           const int32_t* place, const float* weight, const s2r_mat* y,
                           void* stream) {
  if (!rows || !y) return S2R_ERR_NULL;
  Verdict v;
  check_choices(v, T, K, D, R, place);
  v.add(check(rows, R, D));
  v.add(check(y, T, D));
  if (!aligned(weight, 4)) v.add(S2R_ERR_ALIGN);
  if (v.st != S2R_OK) return v.st;
  if (T == 0 || D == 0) return S2R_OK;
  return done(launch_moe_combine(T, K, D, *rows, R, place, weight, *y, on(stream)), stream);
}

s2r_status s2r_moe_combine_grad(uint64_t T, uint32_t K, uint64_t D, const s2r_mat* dy,
                                const int32_t* place, uint64_t R, const float* weight,
                                const s2r_mat* rows, const s2r_mat* drows,
                                const s2r_q8_mat* drowsq, float* dweight, void* stream) {
  if (!dy || (!drows && !drowsq && !dweight) || (dweight && !rows)) return S2R_ERR_NULL;
  Verdict v;
  check_choices(v, T, K, D, R, place);
  if (dweight && T > 0 && !place) v.add(S2R_ERR_NULL);
  v.add(check(dy, T, D));
  if (dweight) {
    v.add(check(rows, R, D));
    if (rows->dtype != dy->dtype) v.add(S2R_ERR_DIM);
  }
  if (drows) v.add(check(drows, R, D));
  if (drowsq) v.add(check(drowsq, R, D, R));
  if (!aligned(weight, 4) || !aligned(dweight, 4)) v.add(S2R_ERR_ALIGN);
  if (v.st != S2R_OK) return v.st;
  // with no columns or no rows the weights' gradients are empty sums
  if (T == 0 || (!dweight && (D == 0 || R == 0))) return S2R_OK;
  return done(launch_moe_combine_grad(T, K, D, *dy, place, R, weight, dweight ? rows : nullptr, drows,
                                      drowsq, dweight, on(stream)),
              stream);
}

s2r_status s2r_q8_gemm_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts* experts,
                               const s2r_q8_mat* a, const s2r_q8_mat* b, uint64_t b_step,
                               uint64_t b_scale_step, const s2r_mat* c, void* stream) {
  if (!experts || !a || !b || !c) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, N, K)) v.add(S2R_ERR_DIM);
  check_experts(v, experts);
  v.add(check(a, M, K, M));
  v.add(check(b, N, K, blocks128(N)));
  v.add(check(c, M, N));
  uint64_t codes, scales;
  if (!extent(N, b->ld, K, &codes) || !extent_ok(experts->experts, b_step, codes, 1) ||
      !extent(blocks128(K), b->lds, blocks128(N), &scales) ||
      !extent_ok(experts->experts, b_scale_step, scales, 1))
    v.add(S2R_ERR_DIM);
  if (b_step % 16 != 0) v.add(S2R_ERR_ALIGN);
  if (v.st != S2R_OK) return v.st;
  if (M == 0 || N == 0) return S2R_OK;
  return done(launch_q8_gemm_experts(M, N, K, *experts, *a, *b, {b_step, b_scale_step}, *c, on(stream)),
              stream);
}

s2r_status s2r_q8_wgrad_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts* experts,
                                const s2r_mat* dy16, const s2r_q8_mat* dy8, const s2r_q8_mat* x,
                                float* dw, uint64_t lddw, uint64_t dw_step, int accumulate,
                                void* stream) {
  if (!experts || !x || (!dy16 && !dy8)) return S2R_ERR_NULL;
  if (N > 0 && K > 0 && !dw) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, N, K) || (dy16 && dy8) || lddw < K) v.add(S2R_ERR_DIM);
  uint64_t own;
  if (!extent(N, lddw, K, &own) || (experts->experts > 1 && dw_step < own) ||
      !extent_ok(experts->experts, dw_step, own, sizeof(float)))
    v.add(S2R_ERR_DIM);
  check_experts(v, experts);
  if (dy16) {
    v.add(check(dy16, M, N));
    if (dy16->dtype != S2R_BF16) v.add(S2R_ERR_DIM);
  }
  if (dy8) v.add(check(dy8, M, N, M));
  v.add(check(x, M, K, M));
  if (!aligned(dw, 4)) v.add(S2R_ERR_ALIGN);
  if (v.st != S2R_OK) return v.st;
  if (N == 0 || K == 0 || (M == 0 && accumulate)) return S2R_OK;
  return done(launch_q8_wgrad_experts(M, N, K, *experts, dy16, dy8, *x, dw, lddw, dw_step,
                                      accumulate != 0, on(stream)),
              stream);
}

}  // extern "C"
