// q4_api.hip -- the C entry points of s2r_q4.h: argument checks on the host, then the launch.
#include "checks.hpp"
#include "q4_launch.hpp"

using namespace s2r;

namespace {

s2r_status check(const s2r_q4_mat* m, uint64_t rows, uint64_t cols) {
  if (rows > 0 && cols > 0 && (!m->q || !m->scale)) return S2R_ERR_NULL;
  if (m->ld < (cols + 1) / 2 || m->ld > kMaxLd || m->lds < (cols + 31) / 32 || m->lds > kMaxLd)
    return S2R_ERR_DIM;
  if (!aligned(m->q, 16) || m->ld % 16 != 0 || !aligned(m->scale, 8) || m->lds % 8 != 0)
    return S2R_ERR_ALIGN;
  return S2R_OK;
}

}  // namespace

extern "C" {

s2r_status s2r_q4_save(uint64_t R, uint64_t C, const s2r_mat* x, const s2r_q4_mat* out,
                       const s2r_q4_mat* out_t, void* stream) {
  if (!x || (!out && !out_t)) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(R, C)) v.add(S2R_ERR_DIM);
  v.add(check(x, R, C));
  if (out) v.add(check(out, R, C));
  if (out_t) v.add(check(out_t, C, R));
  if (v.st != S2R_OK) return v.st;
  if (R == 0 || C == 0) return S2R_OK;
  return done(launch_q4_save(R, C, *x, out, out_t, on(stream)), stream);
}

s2r_status s2r_q4_load(uint64_t R, uint64_t C, const s2r_q4_mat* in, const s2r_mat* x,
                       void* stream) {
  if (!x || !in) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(R, C)) v.add(S2R_ERR_DIM);
  v.add(check(x, R, C));
  v.add(check(in, R, C));
  if (v.st != S2R_OK) return v.st;
  if (R == 0 || C == 0) return S2R_OK;
  return done(launch_q4_load(R, C, *in, *x, on(stream)), stream);
}

size_t s2r_q4_gemm_workspace_bytes(uint64_t M, uint64_t N, uint64_t K) {
  return sizes_ok(M, N, K) ? q4_gemm_workspace(M, N, K) : 0;
}

s2r_status s2r_q4_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q4_mat* a,
                       const s2r_q4_mat* b, const s2r_mat* c, void* workspace, size_t ws_bytes,
                       void* stream) {
  if (!a || !b || !c) return S2R_ERR_NULL;
  Verdict v;
  if (!sizes_ok(M, N, K)) v.add(S2R_ERR_DIM);
  v.add(check(a, M, K));
  v.add(check(b, N, K));
  v.add(check(c, M, N));
  if (v.st != S2R_OK) return v.st;
  if (M == 0 || N == 0) return S2R_OK;
  v.add(check_workspace(workspace, ws_bytes, q4_gemm_workspace(M, N, K)));
  if (v.st != S2R_OK) return v.st;
  return done(launch_q4_gemm(M, N, K, *a, *b, *c, ws_bytes ? workspace : nullptr, on(stream)), stream);
}

}  // extern "C"
