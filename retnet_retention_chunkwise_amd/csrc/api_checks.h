// Argument checks of C entry points that take tensors with strides: presence,
// strides, alignment, overlaps.  Internal to each source that includes it.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <numeric>
#include <utility>

#include "abi_internal.h"
#include "kernels.h"
#include "libretention.h"

namespace {

using ret::Strides3;

ret_status fail(ret_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  ret::set_last_error(buf);
  return st;
}

ret_status ok() {
  ret::set_last_error("");
  return RET_OK;
}

ret_status done(const char* fn, hipError_t e) {
  if (e == hipSuccess) return ok();
  return fail(RET_ERR_HIP, "%s: HIP error %d (%s)", fn, static_cast<int>(e), hipGetErrorString(e));
}

constexpr long long kMaxElems = (1LL << 31) - 1;
constexpr long long kMaxExtent = 1LL << 46;  // largest extent of a strided tensor, in elements
constexpr int kMaxT = 1 << 30;
constexpr size_t kBad = static_cast<size_t>(-1);

size_t dsize(ret_dtype dt) { return dt == RET_F32 ? 4 : 2; }

// A tensor argument as the checks see it: n0 x n1 x n2 rows of len elements.
struct Arg {
  const char* name;
  const void* p;
  bool written;
  bool required;
  long long n[3];
  Strides3 s;
  long long len;
  size_t es;
  uintptr_t align;
  bool empty() const { return p == nullptr || n[0] == 0 || n[1] == 0 || n[2] == 0 || len == 0; }
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const {  // one past the last byte
    return lo() + ((n[0] - 1) * s.b + (n[1] - 1) * s.h + (n[2] - 1) * s.t + len) * es;
  }
};

Arg seq(const char* name, const void* p, bool written, int B, int H, int T, int d, const Strides3& s, ret_dtype dt) {
  return Arg{name, p, written, true, {B, H, T}, s, d, dsize(dt), dsize(dt)};
}
Arg flat(const char* name, const void* p, bool written, bool required, long long n) {
  return Arg{name, p, written, required, {1, 1, 1}, {0, 0, 0}, n, 4, 16};
}

Strides3 contiguous_bhtd(int H, int T, int d) {
  return {static_cast<long>(H) * T * d, static_cast<long>(T) * d, static_cast<long>(d)};
}
Strides3 contiguous_bthd(int H, int T, int d) {
  return {static_cast<long>(T) * H * d, static_cast<long>(d), static_cast<long>(H) * d};
}
Strides3 given(const ret_strides* s, int i, const Strides3& otherwise) {
  return s == nullptr ? otherwise : Strides3{static_cast<long>(s[i].b), static_cast<long>(s[i].h), static_cast<long>(s[i].t)};
}

// Whether two non-empty tensors share a byte.  Extents that meet may still be
// disjoint when the tensors are slices of one buffer: dimensions that continue
// a row (a stride of the row's length, as merged heads have) are taken into
// it; every row of either tensor then starts a multiple of the remaining
// strides' common divisor g from the tensor's start, and the tensors are
// disjoint if the rows' places within g bytes do not meet.
bool shares(const Arg& a, const Arg& b) {
  if (a.empty() || b.empty()) return false;
  if (!(a.lo() < b.hi() && b.lo() < a.hi())) return false;
  unsigned long long g = 0, len[2];
  const Arg* both[2] = {&a, &b};
  for (int k = 0; k < 2; ++k) {
    const Arg& t = *both[k];
    const long long st[3] = {t.s.b, t.s.h, t.s.t};
    bool open[3] = {t.n[0] > 1, t.n[1] > 1, t.n[2] > 1};
    long long row = t.len;
    for (int pass = 0; pass < 3; ++pass)
      for (int i = 0; i < 3; ++i)
        if (open[i] && st[i] == row) {
          row *= t.n[i];
          open[i] = false;
        }
    for (int i = 0; i < 3; ++i)
      if (open[i]) g = std::gcd(g, static_cast<unsigned long long>(st[i]) * t.es);
    len[k] = static_cast<unsigned long long>(row) * t.es;
  }
  if (g == 0 || len[0] + len[1] > g) return true;
  const unsigned long long ra = a.lo() % g, rb = b.lo() % g;
  // [ra, ra + len a) and [rb, rb + len b) on a circle of g bytes
  return (rb + g - ra) % g < len[0] || (ra + g - rb) % g < len[1];
}

// Whether the rows of a written tensor are disjoint: dimensions taken by
// growing stride must each step past everything inside them.
bool rows_disjoint(const Arg& a) {
  long long n[3] = {a.n[0], a.n[1], a.n[2]};
  long long st[3] = {a.s.b, a.s.h, a.s.t};
  long long inner = a.len;
  for (int k = 0; k < 3; ++k) {
    int best = -1;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && (best < 0 || st[i] < st[best])) best = i;
    if (best < 0) break;
    if (st[best] < inner) return false;
    inner = st[best] * (n[best] - 1) + inner;
    n[best] = 1;
  }
  return true;
}

bool is(const Arg& a, const char* name) { return std::strcmp(a.name, name) == 0; }

// Checks shared by all entry points: presence, strides, alignment, overlaps.
// same_ok: pairs of arguments that may be one buffer exactly.
ret_status check_args(const char* fn, std::initializer_list<Arg> args,
                      std::initializer_list<std::pair<const char*, const char*>> same_ok = {}) {
  for (const Arg& a : args) {
    const bool none = a.n[0] == 0 || a.n[1] == 0 || a.n[2] == 0 || a.len == 0;
    if (a.p == nullptr) {
      if (a.required && !none) return fail(RET_ERR_INVALID_ARG, "%s: %s is required", fn, a.name);
      continue;
    }
    if (none) continue;
    const long long st[3] = {a.s.b, a.s.h, a.s.t};
    for (int i = 0; i < 3; ++i)  // a dimension of one row has no stride to follow
      if (st[i] < 0 || (a.n[i] > 1 && st[i] > kMaxExtent / (a.n[i] - 1)))
        return fail(RET_ERR_INVALID_ARG, "%s: stride %lld of %s is negative or spans more than 2^46 elements", fn, st[i],
                    a.name);
    if (a.lo() % a.align != 0)
      return fail(RET_ERR_UNSUPPORTED, "%s: %s must be aligned to %zu bytes", fn, a.name, static_cast<size_t>(a.align));
    if (a.written && !rows_disjoint(a))
      return fail(RET_ERR_INVALID_ARG, "%s: rows of %s overlap each other", fn, a.name);
  }
  for (const Arg& a : args) {
    if (!a.written) continue;
    for (const Arg& b : args) {
      if (&a == &b || (b.written && &b < &a)) continue;
      bool may = false;
      for (const auto& pr : same_ok)
        may = may || (a.p == b.p && ((is(a, pr.first) && is(b, pr.second)) || (is(b, pr.first) && is(a, pr.second))));
      if (!may && shares(a, b)) return fail(RET_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, a.name, b.name);
    }
  }
  return RET_OK;
}

ret_status check_sizes(const char* fn, int B, int H, int T, int d, ret_dtype dt) {
  if (B < 1 || H < 1) return fail(RET_ERR_INVALID_ARG, "%s: B=%d and H=%d must be >= 1", fn, B, H);
  if (T < 0) return fail(RET_ERR_INVALID_ARG, "%s: T=%d must be >= 0", fn, T);
  if (d < 1) return fail(RET_ERR_INVALID_ARG, "%s: d=%d must be >= 1", fn, d);
  if (dt != RET_F32 && dt != RET_BF16)
    return fail(RET_ERR_UNSUPPORTED, "%s: dtype %d is not RET_F32 or RET_BF16", fn, static_cast<int>(dt));
  if (T > kMaxT) return fail(RET_ERR_UNSUPPORTED, "%s: T=%d exceeds 2^30", fn, T);
  const long long bh = static_cast<long long>(B) * H;
  if (bh > kMaxElems || bh * d > kMaxElems || bh * d * T > kMaxElems)
    return fail(RET_ERR_UNSUPPORTED, "%s: a tensor has 2^31 or more elements", fn);
  return RET_OK;
}

ret_status check_workspace(const char* fn, const void* ws, size_t given_bytes, size_t need) {
  if (need > 0 && (ws == nullptr || given_bytes < need))
    return fail(RET_ERR_INVALID_ARG, "%s: workspace of %zu bytes required, %zu given", fn, need, given_bytes);
  return RET_OK;
}

}  // namespace
