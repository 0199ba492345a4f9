// C-ABI layer of the attention calls: argument checks, kernel arguments and
// launches.  Every check happens before the first HIP call, so a rejected call
// enqueues nothing and touches no output.
#include "api_checks.h"
#include "attention.h"

namespace {

constexpr int kMaxLen = 1 << 30;               // tokens, and the offset's magnitude
constexpr long long kMaxAttnRows = 1LL << 25;  // rows of q: a wave each, below 2^32 threads in all
constexpr long long kMaxTiles = 1LL << 23;     // workgroups of 256 threads
// Scales: the kernels form scale log2 e and 8 / (scale log2 e), which leave fp32 below
// 1.6e-38 and above 2.3e38 (the running maximum then never moves, or every score is NaN).
constexpr float kMinScale = 0x1p-100f, kMaxScale = 0x1p+100f;

struct Sizes {
  int B, H, Hk, T, S, dk, dv, maps;
};

ret_status check_heads(const char* fn, int B, int H, int Hk, int dk, int dv, int maps, ret_dtype dt) {
  if (B < 1 || H < 1 || Hk < 1)
    return fail(RET_ERR_INVALID_ARG, "%s: B=%d, H=%d and Hk=%d must be >= 1", fn, B, H, Hk);
  if (H % Hk != 0) return fail(RET_ERR_INVALID_ARG, "%s: H=%d is not a multiple of Hk=%d", fn, H, Hk);
  if (dk < 1 || dv < 1) return fail(RET_ERR_INVALID_ARG, "%s: dk=%d and dv=%d must be >= 1", fn, dk, dv);
  if (maps < 1 || maps > 2) return fail(RET_ERR_INVALID_ARG, "%s: maps=%d must be 1 or 2", fn, maps);
  if (dk % maps != 0) return fail(RET_ERR_INVALID_ARG, "%s: dk=%d does not halve into two maps", fn, dk);
  if (dk > ret::kAttnMaxDk || dv > ret::kAttnMaxDv)
    return fail(RET_ERR_UNSUPPORTED, "%s: dk=%d or dv=%d exceeds %d", fn, dk, dv, ret::kAttnMaxDk);
  if (dt != RET_F32 && dt != RET_BF16)
    return fail(RET_ERR_UNSUPPORTED, "%s: dtype %d is not RET_F32 or RET_BF16", fn, static_cast<int>(dt));
  return RET_OK;
}

// Elements of [B,H,T,d] as a limit; every factor is >= 0 and an int.
bool fits(long long B, long long H, long long T, long long d, long long most) {
  return B * H <= most && B * H * (T > 0 ? T : 1) <= most && B * H * T * d <= most;
}

ret_status check_attn(const char* fn, const Sizes& z, ret_dtype dt) {
  const ret_status st = check_heads(fn, z.B, z.H, z.Hk, z.dk, z.dv, z.maps, dt);
  if (st != RET_OK) return st;
  if (z.T < 0 || z.S < 0) return fail(RET_ERR_INVALID_ARG, "%s: T=%d and S=%d must be >= 0", fn, z.T, z.S);
  if (z.T > kMaxLen || z.S > kMaxLen) return fail(RET_ERR_UNSUPPORTED, "%s: T=%d or S=%d exceeds 2^30", fn, z.T, z.S);
  const int d = z.dk > z.dv ? z.dk : z.dv;
  if (!fits(z.B, z.H, z.T, d, kMaxElems) || !fits(z.B, z.Hk, z.S, d, kMaxElems))
    return fail(RET_ERR_UNSUPPORTED, "%s: a tensor has 2^31 or more elements", fn);
  if (!fits(z.B, z.H, z.T, 1, kMaxAttnRows)) return fail(RET_ERR_UNSUPPORTED, "%s: B*H*T exceeds 2^25", fn);
  if (static_cast<long long>(z.B) * z.H * ((z.T + 63LL) / 64) > kMaxTiles ||
      static_cast<long long>(z.B) * z.Hk * ((z.S + 63LL) / 64) > kMaxTiles)
    return fail(RET_ERR_UNSUPPORTED, "%s: more than 2^23 tiles of 64 tokens", fn);
  return RET_OK;
}

ret_status check_scores(const char* fn, float scale, int offset) {
  if (!std::isfinite(scale) || scale <= 0.0f)
    return fail(RET_ERR_INVALID_ARG, "%s: scale=%g must be finite and > 0", fn, static_cast<double>(scale));
  if (scale < kMinScale || scale > kMaxScale)
    return fail(RET_ERR_UNSUPPORTED, "%s: scale=%g is not within 2^-100..2^100", fn, static_cast<double>(scale));
  if (offset < -kMaxLen || offset > kMaxLen)
    return fail(RET_ERR_INVALID_ARG, "%s: offset=%d is beyond 2^30", fn, offset);
  return RET_OK;
}

// Distances between tokens of tensors that are read in tiles.
ret_status check_token_strides(const char* fn, std::initializer_list<std::pair<const Strides3*, int>> all) {
  for (const auto& x : all)
    if (x.second > 1 && x.first->t > ret::kMaxTokenStride)
      return fail(RET_ERR_UNSUPPORTED, "%s: a distance of %ld elements between tokens exceeds 2^24", fn, x.first->t);
  return RET_OK;
}

Arg optional(Arg a) {
  a.required = false;
  return a;
}
// Contiguous 4-byte values of any 4-byte alignment.
Arg words(const char* name, const void* p, bool written, bool required, long long n) {
  Arg a = flat(name, p, written, required, n);
  a.align = 4;
  return a;
}

// A cache as a tensor of [pages, Hk, page] rows.
Strides3 contiguous_cache(int Hk, int page, int d) { return contiguous_bhtd(Hk, page, d); }

ret_status check_cache(const char* fn, int pages, int page, int max_pages) {
  if (pages < 0 || max_pages < 0 || page < 1)
    return fail(RET_ERR_INVALID_ARG, "%s: pages=%d and max_pages=%d must be >= 0, page=%d >= 1", fn, pages, max_pages,
                page);
  if (static_cast<long long>(max_pages) * page > kMaxLen)
    return fail(RET_ERR_UNSUPPORTED, "%s: max_pages * page exceeds 2^30 tokens", fn);
  return RET_OK;
}

ret::AttnFwd sizes_only(const Sizes& z, ret_dtype dt) {
  static const float two = 0.0f;
  ret::AttnFwd a{};
  a.lam = z.maps > 1 ? &two : nullptr;
  a.B = z.B;
  a.H = z.H;
  a.Hk = z.Hk;
  a.T = z.T;
  a.S = z.S;
  a.d = z.dk / z.maps;
  a.dv = z.dv;
  a.dt = dt == RET_BF16 ? 1 : 0;
  a.whole = true;
  return a;
}

// Whether maps of d and values of dv elements are whole pieces of 16 bytes.
bool whole_rows(int d, int dv, ret_dtype dt) {
  const int piece = dt == RET_BF16 ? 8 : 4;
  return d % piece == 0 && dv % piece == 0;
}
// Whether every row of a tensor starts at a multiple of 16 bytes.
bool rows_aligned(const void* p, const Strides3& s, size_t es) {
  return (reinterpret_cast<uintptr_t>(p) | s.b * es | s.h * es | s.t * es) % 16 == 0;
}

}  // namespace

extern "C" {

size_t retention_attention_workspace_bytes(int B, int H, int Hk, int T, int S, int dk, int dv, int maps, ret_dtype dt) {
  const Sizes z{B, H, Hk, T, S, dk, dv, maps};
  if (check_attn("retention_attention_workspace_bytes", z, dt) != RET_OK) return kBad;
  return T == 0 ? 0 : ret::attention_fwd_workspace(sizes_only(z, dt));
}

size_t retention_attention_bwd_workspace_bytes(int B, int H, int Hk, int T, int S, int dk, int dv, int maps,
                                               ret_dtype dt) {
  const Sizes z{B, H, Hk, T, S, dk, dv, maps};
  if (check_attn("retention_attention_bwd_workspace_bytes", z, dt) != RET_OK) return kBad;
  return ret::attention_bwd_workspace(sizes_only(z, dt));
}

ret_status retention_attention_fwd(const void* q, const void* k, const void* v, const float* lam, const int* lens,
                                   void* o, float* lse, void* second, const ret_strides* strides, int B, int H, int Hk,
                                   int T, int S, int dk, int dv, float scale, int causal, int offset, ret_dtype dt,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "retention_attention_fwd";
  const Sizes z{B, H, Hk, T, S, dk, dv, lam != nullptr ? 2 : 1};
  ret_status st = check_attn(fn, z, dt);
  if (st == RET_OK) st = check_scores(fn, scale, offset);
  if (st != RET_OK) return st;
  if (second != nullptr && lam == nullptr)
    return fail(RET_ERR_INVALID_ARG, "%s: second is an output of two maps, and lam is null", fn);
  ret::AttnFwd a = sizes_only(z, dt);
  a.sq = given(strides, 0, contiguous_bhtd(H, T, dk));
  a.sk = given(strides, 1, contiguous_bhtd(Hk, S, dk));
  a.sv = given(strides, 2, contiguous_bhtd(Hk, S, dv));
  a.so = given(strides, 3, contiguous_bhtd(H, T, dv));
  st = check_token_strides(fn, {{&a.sk, S}, {&a.sv, S}});
  if (st != RET_OK) return st;
  if (S <= 1) a.sk.t = a.sv.t = 0;  // not followed, but multiplied
  const size_t need = T == 0 ? 0 : ret::attention_fwd_workspace(a);
  const long long rows = static_cast<long long>(B) * H * T;
  st = check_args(fn, {seq("q", q, false, B, H, T, dk, a.sq, dt), seq("k", k, false, B, Hk, S, dk, a.sk, dt),
                       seq("v", v, false, B, Hk, S, dv, a.sv, dt), seq("o", o, true, B, H, T, dv, a.so, dt),
                       optional(seq("second", second, true, B, H, T, dv, contiguous_bhtd(H, T, dv), dt)),
                       words("lse", lse, true, false, rows * z.maps), words("lam", lam, false, false, H),
                       words("lens", lens, false, false, B),
                       flat("workspace", need ? workspace : nullptr, true, false, (need + 3) / 4)});
  if (st == RET_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != RET_OK) return st;
  if (T == 0) return ok();
  a.q = q;
  a.k = k;
  a.v = v;
  a.lam = lam;
  a.lens = lens;
  a.o = o;
  a.second = second;
  a.lse = lse;
  a.scale = scale;
  a.causal = causal != 0;
  a.offset = offset;
  a.whole = whole_rows(a.d, dv, dt) &&
            (dt == RET_F32 || (rows_aligned(k, a.sk, dsize(dt)) && rows_aligned(v, a.sv, dsize(dt))));
  return done(fn, ret::launch_attention_fwd(a, workspace, static_cast<hipStream_t>(stream)));
}

ret_status retention_attention_bwd(const void* q, const void* k, const void* v, const float* lam, const int* lens,
                                   const void* o, const float* lse, const void* second, const void* grad_o,
                                   void* grad_q, void* grad_k, void* grad_v, float* grad_lam,
                                   const ret_strides* strides, int B, int H, int Hk, int T, int S, int dk, int dv,
                                   float scale, int causal, int offset, ret_dtype dt, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  const char* fn = "retention_attention_bwd";
  const Sizes z{B, H, Hk, T, S, dk, dv, lam != nullptr ? 2 : 1};
  ret_status st = check_attn(fn, z, dt);
  if (st == RET_OK) st = check_scores(fn, scale, offset);
  if (st != RET_OK) return st;
  if ((grad_lam != nullptr) != (lam != nullptr))
    return fail(RET_ERR_INVALID_ARG, "%s: lam and grad_lam are given together or not at all", fn);
  ret::AttnBwd g{};
  ret::AttnFwd& a = g.f;
  a = sizes_only(z, dt);
  const Strides3 cq = contiguous_bhtd(H, T, dk), ck = contiguous_bhtd(Hk, S, dk), cv = contiguous_bhtd(Hk, S, dv),
                 co = contiguous_bhtd(H, T, dv);
  a.sq = given(strides, 0, cq);
  a.sk = given(strides, 1, ck);
  a.sv = given(strides, 2, cv);
  a.so = given(strides, 3, co);
  g.sdo = given(strides, 4, co);
  g.sdq = given(strides, 5, cq);
  g.sdk = given(strides, 6, ck);
  g.sdv = given(strides, 7, cv);
  st = check_token_strides(fn, {{&a.sq, T}, {&g.sdo, T}, {&a.sk, S}, {&a.sv, S}});
  if (st != RET_OK) return st;
  if (T <= 1) a.sq.t = g.sdo.t = 0;  // not followed, but multiplied
  if (S <= 1) a.sk.t = a.sv.t = 0;
  const size_t need = ret::attention_bwd_workspace(a);
  const long long rows = static_cast<long long>(B) * H * T;
  Arg two = seq("second", second, false, B, H, T, dv, co, dt);
  two.required = z.maps > 1;
  st = check_args(
      fn, {seq("q", q, false, B, H, T, dk, a.sq, dt), seq("k", k, false, B, Hk, S, dk, a.sk, dt),
           seq("v", v, false, B, Hk, S, dv, a.sv, dt), seq("o", o, false, B, H, T, dv, a.so, dt), two,
           seq("grad_o", grad_o, false, B, H, T, dv, g.sdo, dt), words("lse", lse, false, true, rows * z.maps),
           seq("grad_q", grad_q, true, B, H, T, dk, g.sdq, dt), seq("grad_k", grad_k, true, B, Hk, S, dk, g.sdk, dt),
           seq("grad_v", grad_v, true, B, Hk, S, dv, g.sdv, dt), words("lam", lam, false, false, H),
           words("grad_lam", grad_lam, true, false, H), words("lens", lens, false, false, B),
           flat("workspace", need ? workspace : nullptr, true, false, (need + 3) / 4)});
  if (st == RET_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != RET_OK) return st;
  a.q = q;
  a.k = k;
  a.v = v;
  a.lam = lam;
  a.lens = lens;
  a.o = const_cast<void*>(o);
  a.second = const_cast<void*>(second);
  a.lse = const_cast<float*>(lse);
  a.scale = scale;
  a.causal = causal != 0;
  a.offset = offset;
  a.whole = whole_rows(a.d, dv, dt) &&
            (dt == RET_F32 || (rows_aligned(k, a.sk, dsize(dt)) && rows_aligned(v, a.sv, dsize(dt)) &&
                               rows_aligned(q, a.sq, dsize(dt)) && rows_aligned(grad_o, g.sdo, dsize(dt))));
  g.grad_o = grad_o;
  g.grad_q = grad_q;
  g.grad_k = grad_k;
  g.grad_v = grad_v;
  g.grad_lam = grad_lam;
  return done(fn, ret::launch_attention_bwd(g, workspace, static_cast<hipStream_t>(stream)));
}

size_t retention_attention_step_workspace_bytes(int B, int H, int Hk, int dk, int dv, int page, int max_pages, int maps,
                                                ret_dtype dt) {
  const char* fn = "retention_attention_step_workspace_bytes";
  if (check_heads(fn, B, H, Hk, dk, dv, maps, dt) != RET_OK || check_cache(fn, 0, page, max_pages) != RET_OK) return kBad;
  if (!fits(B, H, 1, 1, kMaxTiles)) {
    fail(RET_ERR_UNSUPPORTED, "%s: B*H exceeds 2^23", fn);
    return kBad;
  }
  static const float two = 0.0f;
  ret::AttnStep a{};
  a.lam = maps > 1 ? &two : nullptr;
  a.B = B;
  a.H = H;
  a.Hk = Hk;
  a.d = dk / maps;
  a.dv = dv;
  a.set_page(page);
  a.max_pages = max_pages;
  a.dt = dt == RET_BF16 ? 1 : 0;
  return ret::attention_step_workspace(a);
}

ret_status retention_attention_step(const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
                                    const int* table, const int* lens, const float* lam, void* o,
                                    const ret_strides* strides, int B, int H, int Hk, int dk, int dv, int pages,
                                    int page, int max_pages, float scale, ret_dtype dt, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const char* fn = "retention_attention_step";
  const int maps = lam != nullptr ? 2 : 1;
  ret_status st = check_heads(fn, B, H, Hk, dk, dv, maps, dt);
  if (st == RET_OK) st = check_cache(fn, pages, page, max_pages);
  if (st == RET_OK) st = check_scores(fn, scale, 0);
  if (st != RET_OK) return st;
  if (!fits(B, H, 1, 1, kMaxTiles)) return fail(RET_ERR_UNSUPPORTED, "%s: B*H exceeds 2^23", fn);
  ret::AttnStep a{};
  a.sq = given(strides, 0, contiguous_bhtd(H, 1, dk));
  a.sk = given(strides, 1, contiguous_bhtd(Hk, 1, dk));
  a.sv = given(strides, 2, contiguous_bhtd(Hk, 1, dv));
  a.skc = given(strides, 3, contiguous_cache(Hk, page, dk));
  a.svc = given(strides, 4, contiguous_cache(Hk, page, dv));
  a.so = given(strides, 5, contiguous_bhtd(H, 1, dv));
  const size_t need = retention_attention_step_workspace_bytes(B, H, Hk, dk, dv, page, max_pages, maps, dt);
  st = check_args(
      fn, {seq("q", q, false, B, H, 1, dk, a.sq, dt), seq("k", k, false, B, Hk, 1, dk, a.sk, dt),
           seq("v", v, false, B, Hk, 1, dv, a.sv, dt), seq("k_cache", k_cache, true, pages, Hk, page, dk, a.skc, dt),
           seq("v_cache", v_cache, true, pages, Hk, page, dv, a.svc, dt),
           words("table", table, false, true, static_cast<long long>(B) * max_pages),
           words("lens", lens, false, true, B), words("lam", lam, false, false, H),
           seq("o", o, true, B, H, 1, dv, a.so, dt),
           flat("workspace", need ? workspace : nullptr, true, false, (need + 3) / 4)});
  if (st == RET_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != RET_OK) return st;
  a.q = q;
  a.k = k;
  a.v = v;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.table = table;
  a.lens = lens;
  a.lam = lam;
  a.o = o;
  a.B = B;
  a.H = H;
  a.Hk = Hk;
  a.d = dk / maps;
  a.dv = dv;
  a.pages = pages;
  a.set_page(page);
  a.max_pages = max_pages;
  a.scale = scale;
  a.dt = dt == RET_BF16 ? 1 : 0;
  a.whole = whole_rows(a.d, dv, dt);
  return done(fn, ret::launch_attention_step(a, workspace, static_cast<hipStream_t>(stream)));
}

ret_status retention_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, const int* table,
                                  const int* start, const int* counts, const ret_strides* strides, int B, int Hk,
                                  int T, int dk, int dv, int pages, int page, int max_pages, ret_dtype dt,
                                  void* stream) {
  const char* fn = "retention_cache_append";
  ret_status st = check_attn(fn, {B, Hk, Hk, T, T, dk, dv, 1}, dt);
  if (st == RET_OK) st = check_cache(fn, pages, page, max_pages);
  if (st != RET_OK) return st;
  const Strides3 sk = given(strides, 0, contiguous_bhtd(Hk, T, dk)), sv = given(strides, 1, contiguous_bhtd(Hk, T, dv)),
                 skc = given(strides, 2, contiguous_cache(Hk, page, dk)),
                 svc = given(strides, 3, contiguous_cache(Hk, page, dv));
  st = check_args(
      fn, {seq("k", k, false, B, Hk, T, dk, sk, dt), seq("v", v, false, B, Hk, T, dv, sv, dt),
           seq("k_cache", k_cache, true, pages, Hk, page, dk, skc, dt),
           seq("v_cache", v_cache, true, pages, Hk, page, dv, svc, dt),
           words("table", table, false, true, static_cast<long long>(B) * max_pages),
           words("start", start, false, true, B), words("counts", counts, false, false, B)});
  if (st != RET_OK) return st;
  if (T == 0 || max_pages == 0 || pages == 0) return ok();  // nothing to store, or nowhere
  const ret::CacheAppend a{k,  v,  k_cache, v_cache, table, start, counts, sk,    sv,   skc,
                           svc, B, Hk,      T,       dk,    dv,    pages,  page, max_pages, dt == RET_BF16 ? 1 : 0};
  return done(fn, ret::launch_cache_append(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
