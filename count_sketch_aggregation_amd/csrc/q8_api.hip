// q8_api.hip -- the C entry points of s2r_q8.h: argument checks on the host, then the launch.
#include "q8_launch.hpp"

using namespace s2r;

namespace {

constexpr uint64_t kMaxSize = 1ull << 28;
constexpr uint64_t kMaxLd = 1ull << 22;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline uint64_t blocks128(uint64_t n) { return (n + 127) / 128; }

// The first broken rule of a matrix of `rows` x `cols`, in the order NULL, size, alignment.
s2r_status check(const s2r_mat* m, uint64_t rows, uint64_t cols) {
  if (rows > 0 && cols > 0 && !m->data) return S2R_ERR_NULL;
  if (m->dtype > S2R_F32 || m->ld < cols || m->ld > kMaxLd) return S2R_ERR_DIM;
  if (!aligned(m->data, 16) || m->ld % (m->dtype == S2R_F32 ? 4 : 8) != 0) return S2R_ERR_ALIGN;
  return S2R_OK;
}

s2r_status check(const s2r_q8_mat* m, uint64_t rows, uint64_t cols, uint64_t scale_rows) {
  if (rows > 0 && cols > 0 && (!m->q || !m->scale)) return S2R_ERR_NULL;
  if (m->format > S2R_E5M2 || m->ld < cols || m->ld > kMaxLd || m->lds < scale_rows ||
      m->lds >= kMaxSize + 4)
    return S2R_ERR_DIM;
  if (!aligned(m->q, 16) || m->ld % 16 != 0 || !aligned(m->scale, 4) || m->lds % 4 != 0)
    return S2R_ERR_ALIGN;
  return S2R_OK;
}

s2r_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || have == 0) return S2R_OK;
  if (!aligned(ws, 16)) return S2R_ERR_ALIGN;
  return have < need ? S2R_ERR_WORKSPACE : S2R_OK;
}

// What several checks found: a NULL anywhere comes before a size, a size before an alignment.
struct Verdict {
  s2r_status st = S2R_OK;
  void add(s2r_status s) {
    if (s != S2R_OK && (st == S2R_OK || s < st)) st = s;
  }
};

inline bool sizes_ok(uint64_t a, uint64_t b, uint64_t c = 0) {
  return a < kMaxSize && b < kMaxSize && c < kMaxSize;
}

inline hipStream_t on(void* stream) { return static_cast<hipStream_t>(stream); }

s2r_status done(hipError_t e, void* stream) {
  if (e != hipSuccess) return S2R_ERR_HIP;
  trace_mark(on(stream), "end");
  return S2R_OK;
}

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
