// Launch interface of the attention kernels (attention_*.hip); arguments are
// validated by the caller.
#pragma once

#include <type_traits>

#include "kernels.h"

namespace ret {

constexpr int kAttnMaxDk = 256;  // channels of q and k, all maps together
constexpr int kAttnMaxDv = 256;
// Elements between tokens of a whole sequence's tensors that are read in tiles: a
// tile's rows are addressed in 32 bits from its first.
constexpr long kMaxTokenStride = 1L << 24;

struct AttnFwd {
  const void* q;
  const void* k;
  const void* v;
  const float* lam;  // [H]; null: one map
  const int* lens;   // [B] or null
  void* o;
  void* second;      // nullable: [B,H,T,dv], the second map's output
  float* lse;        // nullable: [B,H,M,T]
  Strides3 sq, sk, sv, so;
  int B, H, Hk, T, S;
  int d, dv;         // channels of one map; of a value
  float scale;       // of the scores, within 2^-100..2^100
  bool causal;
  int offset;        // causal: row t sees the keys up to t + offset
  int dt;
  bool whole;        // rows of whole 16-byte pieces; bf16: also at 16-byte addresses
  int maps() const { return lam != nullptr ? 2 : 1; }
};
struct AttnBwd {
  AttnFwd f;         // the forward's, o, second and lse as it wrote them
  const void* grad_o;
  void* grad_q;
  void* grad_k;
  void* grad_v;
  float* grad_lam;   // null with one map
  Strides3 sdo, sdq, sdk, sdv;
};

// One new token of every sequence over a paged cache of keys and values.
// Strides of a cache: between pages (b), heads (h) and tokens of a page (t).
struct AttnStep {
  const void* q;     // [B,H,M d]
  const void* k;     // [B,Hk,M d], the new token's
  const void* v;     // [B,Hk,dv]
  void* k_cache;     // [pages,Hk,page,M d]
  void* v_cache;     // [pages,Hk,page,dv]
  const int* table;  // [B,max_pages]
  const int* lens;   // [B], keys in the cache
  const float* lam;  // [H]; null: one map
  void* o;           // [B,H,dv]
  Strides3 sq, sk, sv, skc, svc, so;
  int B, H, Hk, d, dv, pages, page, max_pages;
  float scale;
  int dt;
  bool whole;        // rows of whole 16-byte pieces
  int maps() const { return lam != nullptr ? 2 : 1; }
  // key / page by a product, for 0 <= key < 2^30: mul exceeds 2^(30 + s) / page,
  // 2^s >= page, by less than one, which moves no quotient's floor.
  unsigned page_mul;
  int page_shift;
  __host__ __device__ int page_of(int key) const {
    return static_cast<int>(static_cast<unsigned long long>(key) * page_mul >> page_shift);
  }
  void set_page(int n) {
    page = n;
    page_shift = 30;
    while (1LL << (page_shift - 30) < n) ++page_shift;
    page_mul = static_cast<unsigned>(((1ULL << page_shift) + n - 1) / n);
  }
};
// T tokens of every sequence into the cache.
struct CacheAppend {
  const void* k;     // [B,Hk,T,dk]
  const void* v;
  void* k_cache;
  void* v_cache;
  const int* table;
  const int* start;   // [B], position of token 0
  const int* counts;  // [B] or null: T
  Strides3 sk, sv, skc, svc;
  int B, Hk, T, dk, dv, pages, page, max_pages, dt;
};

// Scratch of the calls in bytes, functions of the sizes alone.
size_t attention_fwd_workspace(const AttnFwd& a);
size_t attention_bwd_workspace(const AttnFwd& a);
hipError_t launch_attention_fwd(const AttnFwd& a, void* ws, hipStream_t s);
hipError_t launch_attention_bwd(const AttnBwd& a, void* ws, hipStream_t s);
size_t attention_step_workspace(const AttnStep& a);
hipError_t launch_attention_step(const AttnStep& a, void* ws, hipStream_t s);
hipError_t launch_cache_append(const CacheAppend& a, hipStream_t s);

namespace attn {

// Shares of the keys of a call whose keys are split: outputs not yet divided,
// [split][row][M][dv4] with dv4 = dv rounded up to 4, and their {maximum of
// scale score log2 e, sum}, [split][row][M].
struct Partial {
  float* out;
  float* ml;
  int nsplit;
};
// Shares that so many keys need at least: a sum of weights grows by one key at a
// time in each of four lanes (the step: 16), and stands still at 2^24 equal ones.
constexpr int kMaxRange = 1 << 24;
inline int least_ranges(long keys) { return keys > kMaxRange ? static_cast<int>((keys + kMaxRange - 1) / kMaxRange) : 1; }
inline size_t partial_floats(long rows, int maps, int dv, int nsplit) {
  return nsplit > 1 ? static_cast<size_t>(nsplit) * rows * maps * (((dv + 3) & ~3) + 4) : 0;  // ml in 16 bytes
}
inline Partial partial_at(void* ws, long rows, int maps, int dv, int nsplit) {
  float* out = static_cast<float*>(ws);
  return {out, out + static_cast<size_t>(nsplit) * rows * maps * ((dv + 3) & ~3), nsplit};
}
// Joins the shares into o, second and lse (T rows of every batch element and head).
hipError_t launch_join(const AttnFwd& a, const Partial& p, hipStream_t s);

// The kernels of one type (E: uint16_t, bf16 bits, or float).
template <typename E>
int fwd_rows(const AttnFwd& a);  // rows of a workgroup
template <typename E>
hipError_t launch_fwd(const AttnFwd& a, const Partial& part, hipStream_t s);
// shares > 1: every share of the keys leaves its sums in part
template <typename E>
hipError_t launch_bwd_q(const AttnBwd& a, float* stats, float* lam_part, float* part, int shares, hipStream_t s);
template <typename E>
int bwd_rows(const AttnFwd& a);  // rows of a workgroup
constexpr int kBwdKeys = 64;     // keys of a workgroup, of any size and type
// shares > 1: every share of the rows leaves its sums in part
template <typename E>
hipError_t launch_bwd_kv(const AttnBwd& a, const float* stats, float* part, int shares, hipStream_t s);

// f(maps, channels of all maps, channels of a value, whole), as types, for the
// smallest sizes built that hold the call's.  Where keys or values alone are wide,
// sizes of their own save the narrow side's padding (dk 192 dv 128, B4 H8 T2048
// forward: 83 us, in (256, 256) 122).  Rows that are not whole take code that shifts
// their ends, built for two sizes; a workgroup's rows do not depend on it.
template <typename A, typename F>
auto with_sizes(const A& a, F&& f) {
  typedef std::integral_constant<int, 64> N64;
  typedef std::integral_constant<int, 128> N128;
  typedef std::integral_constant<int, 256> N256;
  auto pick = [&](auto maps) {
    const int dk = a.d * decltype(maps)::value;
    if (!a.whole) {
      if (dk <= 128 && a.dv <= 128) return f(maps, N128(), N128(), std::false_type());
      return f(maps, N256(), N256(), std::false_type());
    }
    if (dk <= 64 && a.dv <= 64) return f(maps, N64(), N64(), std::true_type());
    if (dk <= 128 && a.dv <= 128) return f(maps, N128(), N128(), std::true_type());
    if (a.dv <= 128) return f(maps, N256(), N128(), std::true_type());
    if (dk <= 128) return f(maps, N128(), N256(), std::true_type());
    return f(maps, N256(), N256(), std::true_type());
  };
  return a.maps() > 1 ? pick(std::integral_constant<int, 2>()) : pick(std::integral_constant<int, 1>());
}

}  // namespace attn
}  // namespace ret
