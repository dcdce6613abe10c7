// Argument checks that the entry points of libssm_block and libssm_delta share:
// the thread's last error (each library has its own), sizes without overflow,
// pointers present, aligned and apart.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "ssm.h"

namespace ssmb {

inline thread_local char g_last_error[512];

// Record a reason (one line) and return `status`.
__attribute__((format(printf, 2, 3))) inline int fail(int status, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return status;
}

inline int ok() {
  g_last_error[0] = 0;
  return SSM_OK;
}

inline int launched(hipError_t e, const char *what) {
  return e == hipSuccess ? ok() : fail(SSM_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
}

inline bool valid_dtype(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }
inline size_t dtype_size(int32_t t) { return t == SSM_F32 ? 4 : 2; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// a * b of sizes, or -1 past 2^62.
inline int64_t mul(int64_t a, int64_t b) {
  int64_t r;
  return a < 0 || b < 0 || __builtin_mul_overflow(a, b, &r) || r > (int64_t{1} << 62) ? -1 : r;
}

// One tensor of a call: `bytes` from `p`.
struct Arg {
  const char *name;
  const void *p;
  size_t bytes;
  size_t align;
  bool required;
};

inline int check_in(const Arg &a) {
  if (a.required && a.bytes > 0 && !a.p) return fail(SSM_ERR_NULL, "%s is required", a.name);
  if (!aligned(a.p, a.align)) return fail(SSM_ERR_ALIGN, "%s must be aligned to %zu bytes", a.name, a.align);
  return SSM_OK;
}

inline bool overlap(const Arg &a, const Arg &b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Pointers present and aligned; no output overlaps an input or another
// output.  Where `same[o]` is set, output o may be exactly that input.
template <size_t NI, size_t NO>
int check_args(const Arg (&ins)[NI], const Arg (&outs)[NO], const void *const (&same)[NO][2]) {
  for (const Arg &a : ins)
    if (const int rc = check_in(a)) return rc;
  for (const Arg &a : outs)
    if (const int rc = check_in(a)) return rc;
  for (size_t o = 0; o < NO; ++o) {
    for (const Arg &a : ins) {
      const bool exact = outs[o].p != nullptr && outs[o].p == a.p && (a.p == same[o][0] || a.p == same[o][1]);
      if (!exact && overlap(outs[o], a)) return fail(SSM_ERR_SHAPE, "%s overlaps %s", outs[o].name, a.name);
    }
    for (size_t k = 0; k < o; ++k)
      if (overlap(outs[o], outs[k])) return fail(SSM_ERR_SHAPE, "%s overlaps %s", outs[o].name, outs[k].name);
  }
  return SSM_OK;
}

// The workspace, last of `ins`: large enough, aligned, and none of the bytes
// that are used lies in an input (check_args() has compared it with outputs).
template <size_t NI>
int check_workspace(const Arg (&ins)[NI], size_t need) {
  Arg ws = ins[NI - 1];
  if (need == 0) return SSM_OK;
  if (!ws.p || ws.bytes < need)
    return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", ws.bytes, need);
  if (!aligned(ws.p, 256)) return fail(SSM_ERR_ALIGN, "workspace must be aligned to 256 bytes");
  ws.bytes = need;
  for (size_t k = 0; k + 1 < NI; ++k)
    if (overlap(ws, ins[k])) return fail(SSM_ERR_SHAPE, "workspace overlaps %s", ins[k].name);
  return SSM_OK;
}

constexpr int64_t kMaxGrid = 2147483647;
constexpr int64_t kMaxToken = int64_t{1} << 24;  // elements between two tokens

}  // namespace ssmb
