// q8_api.hip -- the C entry points of s2r_q8.h: argument checks on the host, then the launch.
#include "checks.hpp"
#include "q8_launch.hpp"

using namespace s2r;

namespace {

s2r_status gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat* a, const s2r_q8_mat* b,
                const s2r_mat* c, bool fast, void* workspace, size_t ws_bytes, void* stream) {
  if (!a || !b || !c) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, N, K)) v.add(S2R_ERR_DIM);
  v.add(check(a, M, K, M));
  v.add(check(b, N, K, blocks128(N)));
  v.add(check(c, M, N));
  if (v.st != S2R_OK) return v.st;
  if (M == 0 || N == 0) return S2R_OK;
  v.add(check_workspace(workspace, ws_bytes, q8_gemm_workspace(M, N, K)));
  if (v.st != S2R_OK) return v.st;
  return done(launch_q8_gemm(M, N, K, *a, *b, *c, fast, ws_bytes ? workspace : nullptr, on(stream)),
              stream);
}

}  // namespace

extern "C" {

s2r_status s2r_q8_save(uint64_t M, uint64_t K, const s2r_mat* x, const s2r_q8_mat* out,
                       void* stream) {
  if (!x || !out) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, K)) v.add(S2R_ERR_DIM);
  v.add(check(x, M, K));
  v.add(check(out, M, K, M));
  if (v.st != S2R_OK) return v.st;
  if (M == 0 || K == 0) return S2R_OK;
  return done(launch_q8_save(M, K, *x, *out, on(stream)), stream);
}

s2r_status s2r_q8_load(uint64_t M, uint64_t K, const s2r_q8_mat* in, const s2r_mat* x,
                       void* stream) {
  if (!x || !in) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, K)) v.add(S2R_ERR_DIM);
  v.add(check(x, M, K));
  v.add(check(in, M, K, M));
  if (v.st != S2R_OK) return v.st;
  if (M == 0 || K == 0) return S2R_OK;
  return done(launch_q8_load(M, K, *in, *x, on(stream)), stream);
}

s2r_status s2r_q8_weight(uint64_t N, uint64_t K, const s2r_mat* w, const s2r_q8_mat* out,
                         const s2r_q8_mat* out_t, void* stream) {
  if (!w || !out) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(N, K)) v.add(S2R_ERR_DIM);
  v.add(check(w, N, K));
  v.add(check(out, N, K, blocks128(N)));
  if (out_t) {
    v.add(check(out_t, K, N, blocks128(K)));
    if (out_t->format != out->format) v.add(S2R_ERR_DIM);
  }
  if (v.st != S2R_OK) return v.st;
  if (N == 0 || K == 0) return S2R_OK;
  return done(launch_q8_weight(N, K, *w, *out, out_t, on(stream)), stream);
}

size_t s2r_q8_gemm_workspace_bytes(uint64_t M, uint64_t N, uint64_t K) {
  return sizes_ok(M, N, K) ? q8_gemm_workspace(M, N, K) : 0;
}

s2r_status s2r_q8_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat* a,
                       const s2r_q8_mat* b, const s2r_mat* c, void* workspace, size_t ws_bytes,
                       void* stream) {
  return gemm(M, N, K, a, b, c, false, workspace, ws_bytes, stream);
}

s2r_status s2r_q8_gemm_fast(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat* a,
                            const s2r_q8_mat* b, const s2r_mat* c, void* workspace,
                            size_t ws_bytes, void* stream) {
  return gemm(M, N, K, a, b, c, true, workspace, ws_bytes, stream);
}

size_t s2r_q8_wgrad_workspace_bytes(uint64_t M, uint64_t N, uint64_t K) {
  return sizes_ok(M, N, K) ? q8_wgrad_workspace(M, N, K) : 0;
}

s2r_status s2r_q8_wgrad(uint64_t M, uint64_t N, uint64_t K, const s2r_mat* dy16,
                        const s2r_q8_mat* dy8, const s2r_q8_mat* x, float* dw, uint64_t lddw,
                        int accumulate, void* workspace, size_t ws_bytes, void* stream) {
  if (!x || (!dy16 && !dy8)) return S2R_ERR_NULL;
  if (N > 0 && K > 0 && !dw) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, N, K) || (dy16 && dy8) || lddw < K) v.add(S2R_ERR_DIM);
  uint64_t own;
  if (!extent(N, lddw, K, &own) || !extent_ok(1, 0, own, sizeof(float))) v.add(S2R_ERR_DIM);
  if (dy16) {
    v.add(check(dy16, M, N));
    if (dy16->dtype != S2R_BF16) v.add(S2R_ERR_DIM);
  }
  if (dy8) v.add(check(dy8, M, N, M));
  v.add(check(x, M, K, M));
  if (!aligned(dw, 4)) v.add(S2R_ERR_ALIGN);
  if (v.st != S2R_OK) return v.st;
  if (N == 0 || K == 0 || (M == 0 && accumulate)) return S2R_OK;
  v.add(check_workspace(workspace, ws_bytes, q8_wgrad_workspace(M, N, K)));
  if (v.st != S2R_OK) return v.st;
  return done(launch_q8_wgrad(M, N, K, dy16, dy8, *x, dw, lddw, accumulate != 0,
                              ws_bytes ? workspace : nullptr, on(stream)),
              stream);
}

s2r_status s2r_q8_glu(uint64_t M, uint64_t F, s2r_act act, const s2r_mat* g, const s2r_mat* u,
                      const s2r_q8_mat* gq, const s2r_q8_mat* uq, const s2r_mat* y,
                      const s2r_q8_mat* yq, void* stream) {
  if (!g || (!gq && !uq && !y && !yq) || (uq && !u)) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, F) || (uint32_t)act > S2R_ACT_GELU_TANH) v.add(S2R_ERR_DIM);
  v.add(check(g, M, F));
  if (u) {
    v.add(check(u, M, F));
    if (u->dtype != g->dtype) v.add(S2R_ERR_DIM);
  }
  if (gq) v.add(check(gq, M, F, M));
  if (uq) v.add(check(uq, M, F, M));
  if (y) v.add(check(y, M, F));
  if (yq) v.add(check(yq, M, F, M));
  if (v.st != S2R_OK) return v.st;
  if (M == 0 || F == 0) return S2R_OK;
  return done(launch_q8_glu(M, F, act, *g, u, gq, uq, y, yq, on(stream)), stream);
}

s2r_status s2r_q8_glu_grad(uint64_t M, uint64_t F, s2r_act act, const s2r_q8_mat* gq,
                           const s2r_q8_mat* uq, const s2r_mat* dy, const s2r_mat* dg,
                           const s2r_mat* du, const s2r_q8_mat* dgq, const s2r_q8_mat* duq,
                           void* stream) {
  if (!gq || !dy || (!dg && !du && !dgq && !duq) || ((du || duq) && !uq)) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, F) || (uint32_t)act > S2R_ACT_GELU_TANH) v.add(S2R_ERR_DIM);
  v.add(check(gq, M, F, M));
  if (uq) {
    v.add(check(uq, M, F, M));
    if (uq->format != gq->format) v.add(S2R_ERR_DIM);
  }
  v.add(check(dy, M, F));
  if (dg) v.add(check(dg, M, F));
  if (du) v.add(check(du, M, F));
  if (dgq) v.add(check(dgq, M, F, M));
  if (duq) v.add(check(duq, M, F, M));
  if (v.st != S2R_OK) return v.st;
  if (M == 0 || F == 0) return S2R_OK;
  return done(launch_q8_glu_grad(M, F, act, *gq, uq, *dy, dg, du, dgq, duq, on(stream)), stream);
}

}  // extern "C"
