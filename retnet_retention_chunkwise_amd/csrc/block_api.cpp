// C-ABI layer of the operators around retention in a block (gated scan, gated
// GroupNorm, residual norm): argument checks, kernel arguments and launches.
// Every check happens before the first HIP call, so a rejected call enqueues
// nothing and touches no output.
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

// Launch sizes: a grid has fewer than 2^32 threads, 65535 workgroups along y.
constexpr long long kMaxRuns = 1LL << 21;  // tiles of channels of a scan
constexpr long long kMaxRows = 1LL << 28;  // rows of a norm
constexpr int kMaxNormHeads = 65535;

// A forward call of one token has no runs: its kernel goes by the element.
ret_status check_runs(const char* fn, int B, int H, int T, int d, bool backward) {
  if (T > (backward ? 0 : 1) && static_cast<long long>(B) * H * ret::gated_scan_tiles(d) > kMaxRuns)
    return fail(RET_ERR_UNSUPPORTED, "%s: B*H*%d tiles of channels exceed 2^21", fn, ret::gated_scan_tiles(d));
  return RET_OK;
}

ret_status check_norm(const char* fn, int B, int H, int T, int dv) {
  if (dv > RET_MAX_DV) return fail(RET_ERR_UNSUPPORTED, "%s: dv=%d exceeds %d", fn, dv, RET_MAX_DV);
  if (H > kMaxNormHeads) return fail(RET_ERR_UNSUPPORTED, "%s: H=%d exceeds %d", fn, H, kMaxNormHeads);
  if (static_cast<long long>(B) * H * T > kMaxRows)
    return fail(RET_ERR_UNSUPPORTED, "%s: B*H*T exceeds 2^28", fn);
  return RET_OK;
}

ret_status check_eps(const char* fn, float eps) {
  if (!std::isfinite(eps) || eps < 0.0f)
    return fail(RET_ERR_INVALID_ARG, "%s: eps=%g must be finite and >= 0", fn, static_cast<double>(eps));
  return RET_OK;
}

ret_status check_rates(const char* fn, const float* rate, int H) {
  if (rate == nullptr) return fail(RET_ERR_INVALID_ARG, "%s: rate (host array of H floats) is null", fn);
  for (int h = 0; h < H; ++h)
    if (!std::isfinite(rate[h]) || rate[h] <= 0.0f)
      return fail(RET_ERR_INVALID_ARG, "%s: rate[%d] = %g is not finite and > 0", fn, h, static_cast<double>(rate[h]));
  return RET_OK;
}

Arg rows_arg(const char* name, const void* p, bool written, int rows, int D, long stride, ret_dtype dt) {
  return seq(name, p, written, 1, 1, rows, D, Strides3{0, 0, stride}, dt);
}

ret_status check_rows(const char* fn, int rows, int D, float alpha, ret_dtype dt) {
  if (rows < 0) return fail(RET_ERR_INVALID_ARG, "%s: rows=%d must be >= 0", fn, rows);
  if (D < 1) return fail(RET_ERR_INVALID_ARG, "%s: D=%d must be >= 1", fn, D);
  if (dt != RET_F32 && dt != RET_BF16)
    return fail(RET_ERR_UNSUPPORTED, "%s: dtype %d is not RET_F32 or RET_BF16", fn, static_cast<int>(dt));
  if (D > ret::kResidualMaxD) return fail(RET_ERR_UNSUPPORTED, "%s: D=%d exceeds %d", fn, D, ret::kResidualMaxD);
  if (rows > kMaxRows) return fail(RET_ERR_UNSUPPORTED, "%s: rows=%d exceeds 2^28", fn, rows);
  if (static_cast<long long>(rows) * D > kMaxElems)
    return fail(RET_ERR_UNSUPPORTED, "%s: a tensor has 2^31 or more elements", fn);
  if (!std::isfinite(alpha))
    return fail(RET_ERR_INVALID_ARG, "%s: alpha=%g must be finite", fn, static_cast<double>(alpha));
  return RET_OK;
}

ret_status check_workspace(const char* fn, const void* ws, size_t given_bytes, size_t need) {
  if (need > 0 && (ws == nullptr || given_bytes < need))
    return fail(RET_ERR_INVALID_ARG, "%s: workspace of %zu bytes required, %zu given", fn, need, given_bytes);
  return RET_OK;
}

template <typename F>
ret_status for_head_groups(const char* fn, int H, const float* rate, F&& launch) {
  for (int h0 = 0; h0 < H; h0 += ret::kHeadsPerLaunch) {
    ret::HeadGroup g{h0, H - h0 < ret::kHeadsPerLaunch ? H - h0 : ret::kHeadsPerLaunch, rate + h0};
    const hipError_t e = launch(g);
    if (e != hipSuccess) return done(fn, e);
  }
  return ok();
}

long long checkpoint_floats(int B, int H, int T, int d) {
  const int block = ret::gated_scan_block(d);
  return static_cast<long long>(B) * H * ((T + static_cast<long long>(block) - 1) / block) * d;
}

// Bytes that n bytes of checkpoints take in front of the chain's scratch.
size_t own_offset(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

extern "C" {

size_t retention_gated_scan_workspace_bytes(int B, int H, int T, int d, ret_dtype dt) {
  if (check_sizes("retention_gated_scan_workspace_bytes", B, H, T, d, dt) != RET_OK) return kBad;
  if (check_runs("retention_gated_scan_workspace_bytes", B, H, T, d, false) != RET_OK) return kBad;
  return ret::gated_scan_chain_bytes(B, H, T, d);
}

size_t retention_gated_scan_checkpoint_bytes(int B, int H, int T, int d) {
  if (check_sizes("retention_gated_scan_checkpoint_bytes", B, H, T, d, RET_F32) != RET_OK) return kBad;
  return static_cast<size_t>(checkpoint_floats(B, H, T, d)) * 4;
}

size_t retention_gated_scan_bwd_workspace_bytes(int B, int H, int T, int d, ret_dtype dt, int have_checkpoints) {
  if (check_sizes("retention_gated_scan_bwd_workspace_bytes", B, H, T, d, dt) != RET_OK) return kBad;
  if (check_runs("retention_gated_scan_bwd_workspace_bytes", B, H, T, d, true) != RET_OK) return kBad;
  const size_t kept = have_checkpoints ? 0 : static_cast<size_t>(checkpoint_floats(B, H, T, d)) * 4;
  return own_offset(kept) + ret::gated_scan_chain_bytes(B, H, T, d);
}

ret_status retention_gated_scan_fwd(const void* x, const void* f, const float* rate, const float* state_in,
                                    float* state_out, void* y, float* checkpoints, const ret_strides* strides,
                                    int B, int H, int T, int d, int normalize, ret_dtype dt, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const char* fn = "retention_gated_scan_fwd";
  ret_status st = check_sizes(fn, B, H, T, d, dt);
  if (st == RET_OK) st = check_runs(fn, B, H, T, d, false);
  if (st == RET_OK) st = check_rates(fn, rate, H);
  if (st != RET_OK) return st;
  const Strides3 c = contiguous_bhtd(H, T, d);
  const Strides3 sx = given(strides, 0, c), sf = given(strides, 1, c), sy = given(strides, 2, c);
  const long long ns = static_cast<long long>(B) * H * d;
  const size_t need = retention_gated_scan_workspace_bytes(B, H, T, d, dt);
  st = check_args(fn,
                  {seq("x", x, false, B, H, T, d, sx, dt), seq("f", f, false, B, H, T, d, sf, dt),
                   seq("y", y, true, B, H, T, d, sy, dt), flat("state_in", state_in, false, false, ns),
                   flat("state_out", state_out, true, false, ns),
                   flat("checkpoints", checkpoints, true, false, checkpoint_floats(B, H, T, d)),
                   flat("workspace", need ? workspace : nullptr, true, false, (need + 3) / 4)},
                  {{"state_in", "state_out"}});
  if (st == RET_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != RET_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T == 0)
    return state_out == nullptr || state_out == state_in ? ok() : done(fn, ret::launch_state_copy(state_in, state_out, ns, s));
  const ret::GatedScanFwd p{x, f, state_in, state_out, y, checkpoints, sx, sf, sy, B, H, T, d, normalize != 0,
                            dt == RET_BF16 ? 1 : 0};
  return for_head_groups(fn, H, rate, [&](const ret::HeadGroup& g) { return ret::launch_gated_scan_fwd(p, workspace, g, s); });
}

ret_status retention_gated_scan_bwd(const void* x, const void* f, const float* rate, const float* state_in,
                                    const float* checkpoints, const void* grad_y, const float* grad_state_out,
                                    void* grad_x, void* grad_f, float* grad_state_in, const ret_strides* strides,
                                    int B, int H, int T, int d, int normalize, ret_dtype dt, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const char* fn = "retention_gated_scan_bwd";
  ret_status st = check_sizes(fn, B, H, T, d, dt);
  if (st == RET_OK) st = check_runs(fn, B, H, T, d, true);
  if (st == RET_OK) st = check_rates(fn, rate, H);
  if (st != RET_OK) return st;
  const Strides3 c = contiguous_bhtd(H, T, d);
  Strides3 sx = given(strides, 0, c), sf = given(strides, 1, c), sgy = given(strides, 2, c),
           sgx = given(strides, 3, c), sgf = given(strides, 4, c);
  if (T == 1) sx.t = sf.t = sgy.t = sgx.t = sgf.t = d;  // not followed, but multiplied
  const long long ns = static_cast<long long>(B) * H * d;
  const size_t need = retention_gated_scan_bwd_workspace_bytes(B, H, T, d, dt, checkpoints != nullptr);
  st = check_args(fn,
                  {seq("x", x, false, B, H, T, d, sx, dt), seq("f", f, false, B, H, T, d, sf, dt),
                   seq("grad_y", grad_y, false, B, H, T, d, sgy, dt), seq("grad_x", grad_x, true, B, H, T, d, sgx, dt),
                   seq("grad_f", grad_f, true, B, H, T, d, sgf, dt), flat("state_in", state_in, false, false, ns),
                   flat("grad_state_out", grad_state_out, false, false, ns),
                   flat("grad_state_in", grad_state_in, true, false, ns),
                   flat("checkpoints", checkpoints, false, false, checkpoint_floats(B, H, T, d)),
                   flat("workspace", need ? workspace : nullptr, true, false, (need + 3) / 4)},
                  {{"grad_state_out", "grad_state_in"}});
  if (st == RET_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != RET_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T == 0)
    return grad_state_in == nullptr || grad_state_in == grad_state_out
               ? ok()
               : done(fn, ret::launch_state_copy(grad_state_out, grad_state_in, ns, s));
  const int dti = dt == RET_BF16 ? 1 : 0;
  float* own = static_cast<float*>(workspace);
  void* chain = static_cast<char*>(workspace) +
                (checkpoints != nullptr ? 0 : own_offset(static_cast<size_t>(checkpoint_floats(B, H, T, d)) * 4));
  const ret::GatedScanFwd again{x, f, state_in, nullptr, nullptr, own, sx, sf, sx, B, H, T, d, normalize != 0, dti};
  const ret::GatedScanBwd p{x, f, checkpoints != nullptr ? checkpoints : own, grad_y, grad_state_out, grad_x, grad_f,
                            grad_state_in, sx, sf, sgy, sgx, sgf, B, H, T, d, normalize != 0, dti};
  return for_head_groups(fn, H, rate, [&](const ret::HeadGroup& g) {
    if (checkpoints == nullptr) {
      const hipError_t e = ret::launch_gated_scan_fwd(again, chain, g, s);
      if (e != hipSuccess) return e;
    }
    return ret::launch_gated_scan_bwd(p, chain, g, s);
  });
}

ret_status retention_gated_scan_step(const void* x, const void* f, const float* rate, float* state, void* y,
                                     const ret_strides* strides, int B, int H, int d, int normalize, ret_dtype dt,
                                     void* stream) {
  const char* fn = "retention_gated_scan_step";
  ret_status st = check_sizes(fn, B, H, 1, d, dt);
  if (st == RET_OK) st = check_rates(fn, rate, H);
  if (st != RET_OK) return st;
  const Strides3 c = contiguous_bhtd(H, 1, d);
  Strides3 sx = given(strides, 0, c), sf = given(strides, 1, c), sy = given(strides, 2, c);
  sx.t = sf.t = sy.t = d;
  const long long ns = static_cast<long long>(B) * H * d;
  st = check_args(fn, {seq("x", x, false, B, H, 1, d, sx, dt), seq("f", f, false, B, H, 1, d, sf, dt),
                       seq("y", y, true, B, H, 1, d, sy, dt), flat("state", state, true, true, ns)});
  if (st != RET_OK) return st;
  const ret::GatedScanFwd p{x, f, state, state, y, nullptr, sx, sf, sy, B, H, 1, d, normalize != 0,
                            dt == RET_BF16 ? 1 : 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return for_head_groups(fn, H, rate, [&](const ret::HeadGroup& g) { return ret::launch_gated_scan_fwd(p, nullptr, g, s); });
}

ret_status retention_group_norm_gated(const void* y, const void* gate, const float* weight, const float* bias,
                                      float eps, void* out, const ret_strides* strides, int B, int H, int T, int dv,
                                      ret_dtype dt, void* stream) {
  const char* fn = "retention_group_norm_gated";
  ret_status st = check_sizes(fn, B, H, T, dv, dt);
  if (st == RET_OK) st = check_eps(fn, eps);
  if (st != RET_OK) return st;
  st = check_norm(fn, B, H, T, dv);
  if (st != RET_OK) return st;
  const Strides3 sy = given(strides, 0, contiguous_bhtd(H, T, dv)), sz = given(strides, 1, contiguous_bthd(H, T, dv)),
                 so = given(strides, 2, contiguous_bthd(H, T, dv));
  const long long np = static_cast<long long>(H) * dv;
  Arg g = seq("gate", gate, false, B, H, T, dv, sz, dt);
  g.required = false;
  st = check_args(fn, {seq("y", y, false, B, H, T, dv, sy, dt), g, seq("out", out, true, B, H, T, dv, so, dt),
                       flat("weight", weight, false, false, np), flat("bias", bias, false, false, np)});
  if (st != RET_OK) return st;
  if (T == 0) return ok();
  const ret::GateNormFwd a{y, gate, weight, bias, eps, out, sy, gate != nullptr ? sz : so, so, B, H, T, dv,
                           dt == RET_BF16 ? 1 : 0};
  return done(fn, ret::launch_gate_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t retention_group_norm_gated_bwd_workspace_bytes(int B, int H, int T, int dv) {
  const char* fn = "retention_group_norm_gated_bwd_workspace_bytes";
  if (check_sizes(fn, B, H, T, dv, RET_F32) != RET_OK) return kBad;
  if (check_norm(fn, B, H, T, dv) != RET_OK) return kBad;
  return T == 0 ? 0 : static_cast<size_t>(2) * ret::gate_norm_bwd_slabs(B, H, T, dv) * H * dv * 4;
}

ret_status retention_group_norm_gated_bwd(const void* y, const void* gate, const float* weight, const float* bias,
                                          float eps, const void* grad_out, void* grad_y, void* grad_gate,
                                          float* grad_weight, float* grad_bias, const ret_strides* strides, int B,
                                          int H, int T, int dv, ret_dtype dt, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  const char* fn = "retention_group_norm_gated_bwd";
  ret_status st = check_sizes(fn, B, H, T, dv, dt);
  if (st == RET_OK) st = check_eps(fn, eps);
  if (st != RET_OK) return st;
  st = check_norm(fn, B, H, T, dv);
  if (st != RET_OK) return st;
  if ((gate == nullptr) != (grad_gate == nullptr) && T > 0)
    return fail(RET_ERR_INVALID_ARG, "%s: gate and grad_gate are given together or not at all", fn);
  const Strides3 head = contiguous_bhtd(H, T, dv), token = contiguous_bthd(H, T, dv);
  const Strides3 sy = given(strides, 0, head), sz = given(strides, 1, token), sdo = given(strides, 2, token),
                 sdy = given(strides, 3, head), sdz = given(strides, 4, token);
  const long long np = static_cast<long long>(H) * dv;
  const bool want = grad_weight != nullptr || grad_bias != nullptr;
  const size_t need = want ? retention_group_norm_gated_bwd_workspace_bytes(B, H, T, dv) : 0;
  Arg g = seq("gate", gate, false, B, H, T, dv, sz, dt), gg = seq("grad_gate", grad_gate, true, B, H, T, dv, sdz, dt);
  g.required = gg.required = false;
  st = check_args(
      fn, {seq("y", y, false, B, H, T, dv, sy, dt), g, seq("grad_out", grad_out, false, B, H, T, dv, sdo, dt),
           seq("grad_y", grad_y, true, B, H, T, dv, sdy, dt), gg, flat("weight", weight, false, false, np),
           flat("bias", bias, false, false, np), flat("grad_weight", grad_weight, true, false, np),
           flat("grad_bias", grad_bias, true, false, np),
           flat("workspace", need ? workspace : nullptr, true, false, (need + 3) / 4)});
  if (st == RET_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != RET_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T == 0) {  // no rows: the parameter gradients are empty sums
    for (float* p : {grad_weight, grad_bias}) {
      if (p == nullptr) continue;
      const hipError_t e = ret::launch_fill_u32(p, np, 0, s);
      if (e != hipSuccess) return done(fn, e);
    }
    return ok();
  }
  const ret::GateNormBwd a{y,         gate,        weight,    bias, eps, grad_out,
                           grad_y,    grad_gate,   grad_weight, grad_bias,
                           sy,        gate != nullptr ? sz : sdo, sdo, sdy, gate != nullptr ? sdz : sdo,
                           B,         H,           T,         dv,   dt == RET_BF16 ? 1 : 0};
  return done(fn, ret::launch_gate_norm_bwd(a, want ? static_cast<float*>(workspace) : nullptr, s));
}

ret_status retention_residual_norm(const void* x, const void* f, const float* weight, const float* bias,
                                   const float* scale, float alpha, float eps, int rms, void* r, void* n,
                                   const long long* row_strides, int rows, int D, ret_dtype dt, void* stream) {
  const char* fn = "retention_residual_norm";
  ret_status st = check_rows(fn, rows, D, alpha, dt);
  if (st == RET_OK) st = check_eps(fn, eps);
  if (st != RET_OK) return st;
  auto s = [&](int i) { return row_strides == nullptr ? static_cast<long>(D) : static_cast<long>(row_strides[i]); };
  st = check_args(fn, {rows_arg("x", x, false, rows, D, s(0), dt), rows_arg("f", f, false, rows, D, s(1), dt),
                       rows_arg("r", r, true, rows, D, s(2), dt), rows_arg("n", n, true, rows, D, s(3), dt),
                       flat("weight", weight, false, false, D), flat("bias", bias, false, false, D),
                       flat("scale", scale, false, false, D)});
  if (st != RET_OK) return st;
  if (rows == 0) return ok();
  const ret::ResidualNormFwd a{x, f, weight, bias, scale, alpha, eps, rms != 0, r, n, s(0), s(1), s(2), s(3),
                               rows, D, dt == RET_BF16 ? 1 : 0};
  return done(fn, ret::launch_residual_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t retention_residual_norm_bwd_workspace_bytes(int rows, int D) {
  if (check_rows("retention_residual_norm_bwd_workspace_bytes", rows, D, 1.0f, RET_F32) != RET_OK) return kBad;
  return rows == 0 ? 0 : static_cast<size_t>(3) * ret::residual_norm_bwd_blocks(rows, D) * D * 4;
}

ret_status retention_residual_norm_bwd(const void* r, const void* grad_n, const void* grad_r, const void* f,
                                       const float* weight, const float* scale, float alpha, float eps, int rms,
                                       void* grad_x, void* grad_f, float* grad_weight, float* grad_bias,
                                       float* grad_scale, const long long* row_strides, int rows, int D, ret_dtype dt,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "retention_residual_norm_bwd";
  ret_status st = check_rows(fn, rows, D, alpha, dt);
  if (st == RET_OK) st = check_eps(fn, eps);
  if (st != RET_OK) return st;
  auto s = [&](int i) { return row_strides == nullptr ? static_cast<long>(D) : static_cast<long>(row_strides[i]); };
  const bool want = grad_weight != nullptr || grad_bias != nullptr || grad_scale != nullptr;
  const size_t need = want ? retention_residual_norm_bwd_workspace_bytes(rows, D) : 0;
  Arg gr = rows_arg("grad_r", grad_r, false, rows, D, s(2), dt), ff = rows_arg("f", f, false, rows, D, s(3), dt);
  Arg gx = rows_arg("grad_x", grad_x, true, rows, D, s(4), dt), gf = rows_arg("grad_f", grad_f, true, rows, D, s(5), dt);
  gr.required = gx.required = gf.required = false;
  ff.required = grad_scale != nullptr;
  st = check_args(fn, {rows_arg("r", r, false, rows, D, s(0), dt), rows_arg("grad_n", grad_n, false, rows, D, s(1), dt),
                       gr, ff, gx, gf, flat("weight", weight, false, false, D), flat("scale", scale, false, false, D),
                       flat("grad_weight", grad_weight, true, false, D), flat("grad_bias", grad_bias, true, false, D),
                       flat("grad_scale", grad_scale, true, false, D),
                       flat("workspace", need ? workspace : nullptr, true, false, (need + 3) / 4)});
  if (st == RET_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != RET_OK) return st;
  hipStream_t q = static_cast<hipStream_t>(stream);
  if (rows == 0) {  // no rows: the parameter gradients are empty sums
    for (float* p : {grad_weight, grad_bias, grad_scale}) {
      if (p == nullptr) continue;
      const hipError_t e = ret::launch_fill_u32(p, D, 0, q);
      if (e != hipSuccess) return done(fn, e);
    }
    return ok();
  }
  const ret::ResidualNormBwd a{r, grad_n, grad_r, f, weight, scale, alpha, eps, rms != 0, grad_x, grad_f, grad_weight,
                               grad_bias, grad_scale, s(0), s(1), s(2), s(3), s(4), s(5), rows, D,
                               dt == RET_BF16 ? 1 : 0};
  return done(fn, ret::launch_residual_norm_bwd(a, want ? static_cast<float*>(workspace) : nullptr, q));
}

}  // extern "C"
