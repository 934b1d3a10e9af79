// checks.hpp -- the argument checks that the entry points of s2r_q8.h, s2r_moe.h and s2r_q4.h share
// (internal to libs2r).
#pragma once

#include "s2r_launch.hpp"
#include "s2r_q4.h"
#include "s2r_q8.h"

namespace s2r {

constexpr uint64_t kMaxSize = 1ull << 28;
constexpr uint64_t kMaxLd = 1ull << 22;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline uint64_t blocks128(uint64_t n) { return (n + 127) / 128; }

// The first broken rule of a matrix of `rows` x `cols`, in the order NULL, size, alignment.
inline s2r_status check(const s2r_mat* m, uint64_t rows, uint64_t cols) {
  if (rows > 0 && cols > 0 && !m->data) return S2R_ERR_NULL;
  if (m->dtype > S2R_F32 || m->ld < cols || m->ld > kMaxLd) return S2R_ERR_DIM;
  if (!aligned(m->data, 16) || m->ld % (m->dtype == S2R_F32 ? 4 : 8) != 0) return S2R_ERR_ALIGN;
  return S2R_OK;
}

inline s2r_status check(const s2r_q8_mat* m, uint64_t rows, uint64_t cols, uint64_t scale_rows) {
  if (rows > 0 && cols > 0 && (!m->q || !m->scale)) return S2R_ERR_NULL;
  if (m->format > S2R_E5M2 || m->ld < cols || m->ld > kMaxLd || m->lds < scale_rows ||
      m->lds >= kMaxSize + 4)
    return S2R_ERR_DIM;
  if (!aligned(m->q, 16) || m->ld % 16 != 0 || !aligned(m->scale, 4) || m->lds % 4 != 0)
    return S2R_ERR_ALIGN;
  return S2R_OK;
}

inline s2r_status check_workspace(const void* ws, size_t have, size_t need) {
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

// Elements from the first of a matrix [rows][ld] of `cols` columns to behind its last, and of `count` of them `step`
// apart (of `own` elements each) to behind the last one's; false where that, or its bytes, passes 64 bits: a stride like
// -1 would wrap round to a small one.
inline bool extent(uint64_t rows, uint64_t ld, uint64_t cols, uint64_t* n) {
  *n = 0;
  return rows == 0 || cols == 0 ||
         (!__builtin_mul_overflow(rows - 1, ld, n) && !__builtin_add_overflow(*n, cols, n));
}
inline bool extent_ok(uint64_t count, uint64_t step, uint64_t own, uint64_t elem_size) {
  uint64_t n = 0;
  return own == 0 || ((count <= 1 || !__builtin_mul_overflow(count - 1, step, &n)) && !__builtin_add_overflow(n, own, &n) &&
                      n <= UINT64_MAX / elem_size);
}

inline hipStream_t on(void* stream) { return static_cast<hipStream_t>(stream); }

inline s2r_status done(hipError_t e, void* stream) {
  if (e != hipSuccess) return S2R_ERR_HIP;
  trace_mark(on(stream), "end");
  return S2R_OK;
}

}  // namespace s2r
