// The attention calls' host side and their per-row kernels: the join of split
// keys, the backward's row statistics and the sums of shares.  All are bound by
// memory where there are many rows (B2 H16 T4096 d128 two maps: statistics 26 us for
// 105 MB, sums of the kv pass 17 us for 84 MB) and by latency where there are few (a
// join of 32 shares 5.6 us).
#include "attention.h"

#include <algorithm>

#include "attention_tiles.h"
#include "row_sum.h"

namespace ret {
namespace attn {
namespace {

constexpr int kWaves = 4;

// Four elements of a row from c on, zeros from n on.
template <typename E>
__device__ __forceinline__ f32x4 load4(const E* row, int c, int n) {
  f32x4 x = {0, 0, 0, 0};
  if (n % 4 == 0) {
    if (c < n) {
      float y[4];
      VecIO<E, 4>::unpack(VecIO<E, 4>::load(row + c), y);
      x = f32x4{y[0], y[1], y[2], y[3]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < n) x[i] = Elem<E>::load(row, c + i);
  }
  return x;
}
template <typename E>
__device__ __forceinline__ void put4(E* row, int c, int n, f32x4 x) {
  if (n % 4 == 0)
    store4<E, true>(row, c, n, x);
  else
    store4<E, false>(row, c, n, x);
}

// WPR waves per row, along the shares; lanes along the channels, four each.  The
// shares' outputs o_i with maxima m_i and sums l_i join as
// sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i, the waves' sums in wave order.
template <typename E, int MAPS, int WPR>
__global__ __launch_bounds__(64 * kWaves) void attention_join_kernel(AttnFwd a, Partial p, long rows) {
  const int lane = threadIdx.x & 63, wave = wave_id() % WPR, ch = 4 * lane;
  const long row = static_cast<long>(blockIdx.x) * (kWaves / WPR) + wave_id() / WPR;
  if (row >= rows) return;  // with a wave per row, which meets no barrier
  const int t = static_cast<int>(row % a.T), dv4 = (a.dv + 3) & ~3;
  const long bh = row / a.T;
  const int h = static_cast<int>(bh % a.H), b = static_cast<int>(bh / a.H);
  const float2* ml = reinterpret_cast<const float2*>(p.ml);
  f32x4 y[MAPS];
  float tops[MAPS], sums[MAPS];
  // this wave's shares: wave, wave + WPR, ..., one maximum a lane to begin with
#pragma unroll
  for (int m = 0; m < MAPS; ++m) {
    float top = -INFINITY;
    for (int i = wave + WPR * lane; i < p.nsplit; i += WPR * 64) top = fmaxf(top, ml[(i * rows + row) * MAPS + m].x);
#pragma unroll
    for (int o = 1; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
    const float at = top == -INFINITY ? 0.0f : top;
    float l = 0.0f;
    f32x4 x = {0, 0, 0, 0};
#pragma unroll 4
    for (int i = wave; i < p.nsplit; i += WPR) {
      const long j = (i * rows + row) * MAPS + m;
      const float2 s = ml[j];
      f32x4 z = {0, 0, 0, 0};
      if (ch < dv4) z = *reinterpret_cast<const f32x4*>(p.out + j * dv4 + ch);
      const float f = fast_exp2(s.x - at);
      l = fmaf(s.y, f, l);
      x += z * f;
    }
    tops[m] = top;
    sums[m] = l;
    y[m] = x;
  }
  if constexpr (WPR > 1) {
    __shared__ float wave_top[WPR][MAPS], wave_sum[WPR][MAPS];
    __shared__ f32x4 wave_out[WPR][MAPS][64];
#pragma unroll
    for (int m = 0; m < MAPS; ++m) {
      if (lane == 0) {
        wave_top[wave][m] = tops[m];
        wave_sum[wave][m] = sums[m];
      }
      wave_out[wave][m][lane] = y[m];
    }
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int m = 0; m < MAPS; ++m) {
      float top = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) top = fmaxf(top, wave_top[w][m]);
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        const float f = wave_top[w][m] == -INFINITY ? 0.0f : fast_exp2(wave_top[w][m] - top);
        l = fmaf(wave_sum[w][m], f, l);
        x += wave_out[w][m][lane] * f;
      }
      tops[m] = top;
      sums[m] = l;
      y[m] = x;
    }
  }
#pragma unroll
  for (int m = 0; m < MAPS; ++m) {
    const float top = tops[m], l = sums[m];
    y[m] *= l == 0.0f ? 0.0f : 1.0f / l;
    if (a.lse != nullptr && lane == 0)
      a.lse[(bh * MAPS + m) * a.T + t] = l == 0.0f ? -INFINITY : top * kLn2 + logf(l);
  }
  if constexpr (MAPS > 1) {
    if (a.second != nullptr) put4<E>(static_cast<E*>(a.second) + row * a.dv, ch, a.dv, y[1]);
    y[0] -= a.lam[h] * y[1];
  }
  put4<E>(static_cast<E*>(a.o) + b * a.so.b + h * a.so.h + t * a.so.t, ch, a.dv, y[0]);
}

// {lse log2 e, D} of every row and map, LPR lanes per row, four channels a lane.
// A row that saw no key gets +inf, so that exp2(score - lse) is zero there.
template <typename E, int MAPS, int LPR>
__global__ __launch_bounds__(64 * kWaves) void attention_stats_kernel(AttnBwd g, float2* stats, long rows) {
  const AttnFwd& a = g.f;
  const int lane = threadIdx.x % LPR, ch = 4 * lane;
  const long at = (static_cast<long>(blockIdx.x) * kWaves * 64 + threadIdx.x) / LPR;
  const long row = at < rows ? at : rows - 1;
  const int t = static_cast<int>(row % a.T);
  const long bh = row / a.T;
  const int h = static_cast<int>(bh % a.H), b = static_cast<int>(bh / a.H);
  const f32x4 d = load4<E>(static_cast<const E*>(g.grad_o) + b * g.sdo.b + h * g.sdo.h + t * g.sdo.t, ch, a.dv);
  const f32x4 o = load4<E>(static_cast<const E*>(a.o) + b * a.so.b + h * a.so.h + t * a.so.t, ch, a.dv);
  float s[2];
  s[0] = d[0] * o[0] + d[1] * o[1] + d[2] * o[2] + d[3] * o[3];
  s[0] = lanes_sum<LPR>(s[0]);
  if constexpr (MAPS > 1) {
    const f32x4 z = load4<E>(static_cast<const E*>(a.second) + row * a.dv, ch, a.dv);
    s[1] = d[0] * z[0] + d[1] * z[1] + d[2] * z[2] + d[3] * z[3];
    s[1] = lanes_sum<LPR>(s[1]);
    s[0] = fmaf(a.lam[h], s[1], s[0]);
  }
  if (lane < MAPS && at < rows) {
    const float l = a.lse[(bh * MAPS + lane) * a.T + t];
    stats[lane * rows + row] = make_float2(l == -INFINITY ? INFINITY : l * kLog2e, lane == 0 ? s[0] : s[1]);
  }
}

// grad_k and grad_v from the shares' sums [share][row][MAPS d4 + dv4], added in
// share order: a thread per four channels of a row (b, hk, key).
template <typename E, int MAPS>
__global__ __launch_bounds__(64 * kWaves) void attention_add_kernel(AttnBwd g, const float* __restrict__ part, int shares,
                                                                    long rows) {
  const AttnFwd& a = g.f;
  const int d4 = (a.d + 3) & ~3, dv4 = (a.dv + 3) & ~3, width = MAPS * d4 + dv4, per = width / 4;
  const long at = static_cast<long>(blockIdx.x) * (64 * kWaves) + threadIdx.x, row = at / per;
  if (row >= rows) return;
  const int c = 4 * static_cast<int>(at % per);
  f32x4 x = {0, 0, 0, 0};
#pragma unroll 4
  for (int i = 0; i < shares; ++i) x += *reinterpret_cast<const f32x4*>(part + (i * rows + row) * width + c);
  const int key = static_cast<int>(row % a.S);
  const long bh = row / a.S;
  const int hk = static_cast<int>(bh % a.Hk), b = static_cast<int>(bh / a.Hk);
  if (c < MAPS * d4) {
    const int m = MAPS > 1 && c >= d4;
    put4<E>(static_cast<E*>(g.grad_k) + b * g.sdk.b + hk * g.sdk.h + key * g.sdk.t + m * a.d, c - m * d4, a.d, x * a.scale);
  } else {
    put4<E>(static_cast<E*>(g.grad_v) + b * g.sdv.b + hk * g.sdv.h + key * g.sdv.t, c - MAPS * d4, a.dv, x);
  }
}

// grad_q from the shares' sums [share][row][MAPS d4], likewise: a thread per four
// channels of a row (b, h, t).
template <typename E, int MAPS>
__global__ __launch_bounds__(64 * kWaves) void attention_add_q_kernel(AttnBwd g, const float* __restrict__ part, int shares,
                                                                      long rows) {
  const AttnFwd& a = g.f;
  const int d4 = (a.d + 3) & ~3, width = MAPS * d4, per = width / 4;
  const long at = static_cast<long>(blockIdx.x) * (64 * kWaves) + threadIdx.x, row = at / per;
  if (row >= rows) return;
  const int c = 4 * static_cast<int>(at % per), m = MAPS > 1 && c >= d4;
  f32x4 x = {0, 0, 0, 0};
#pragma unroll 4
  for (int i = 0; i < shares; ++i) x += *reinterpret_cast<const f32x4*>(part + (i * rows + row) * width + c);
  const int t = static_cast<int>(row % a.T);
  const long bh = row / a.T;
  const int h = static_cast<int>(bh % a.H), b = static_cast<int>(bh / a.H);
  put4<E>(static_cast<E*>(g.grad_q) + b * g.sdq.b + h * g.sdq.h + t * g.sdq.t + m * a.d, c - m * d4, a.d, x);
}

int kv_width(const AttnFwd& a) { return a.maps() * ((a.d + 3) & ~3) + ((a.dv + 3) & ~3); }

template <typename E>
hipError_t add(const AttnBwd& g, const float* part, int shares, hipStream_t s) {
  const long rows = static_cast<long>(g.f.B) * g.f.Hk * g.f.S, n = rows * (kv_width(g.f) / 4);
  auto* kern = g.f.maps() > 1 ? attention_add_kernel<E, 2> : attention_add_kernel<E, 1>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((n + 64 * kWaves - 1) / (64 * kWaves))), dim3(64 * kWaves), 0, s, g,
                     part, shares, rows);
  return hipGetLastError();
}

template <typename E>
hipError_t add_q(const AttnBwd& g, const float* part, int shares, hipStream_t s) {
  const long rows = static_cast<long>(g.f.B) * g.f.H * g.f.T, n = rows * g.f.maps() * ((g.f.d + 3) / 4);
  auto* kern = g.f.maps() > 1 ? attention_add_q_kernel<E, 2> : attention_add_q_kernel<E, 1>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((n + 64 * kWaves - 1) / (64 * kWaves))), dim3(64 * kWaves), 0, s, g,
                     part, shares, rows);
  return hipGetLastError();
}

template <typename E, int LPR>
hipError_t stats_by_width(const AttnBwd& g, float* to, hipStream_t s) {
  const long rows = static_cast<long>(g.f.B) * g.f.H * g.f.T, per = 64 * kWaves / LPR;
  auto* kern = g.f.maps() > 1 ? attention_stats_kernel<E, 2, LPR> : attention_stats_kernel<E, 1, LPR>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(64 * kWaves), 0, s, g,
                     reinterpret_cast<float2*>(to), rows);
  return hipGetLastError();
}
template <typename E>
hipError_t stats(const AttnBwd& g, float* to, hipStream_t s) {
  if (g.f.dv <= 64) return stats_by_width<E, 16>(g, to, s);
  if (g.f.dv <= 128) return stats_by_width<E, 32>(g, to, s);
  return stats_by_width<E, 64>(g, to, s);
}

long rows_of(const AttnFwd& a) { return static_cast<long>(a.B) * a.H * a.T; }

template <typename E, int WPR>
hipError_t join_by(const AttnFwd& a, const Partial& p, hipStream_t s) {
  const long rows = static_cast<long>(a.B) * a.H * a.T, per = kWaves / WPR;
  auto* kern = a.maps() > 1 ? attention_join_kernel<E, 2, WPR> : attention_join_kernel<E, 1, WPR>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(64 * kWaves), 0, s, a, p, rows);
  return hipGetLastError();
}
template <typename E>
hipError_t join(const AttnFwd& a, const Partial& p, hipStream_t s) {
  // one wave reads a row's few shares as fast as four, which then wait for each other
  // (and a workgroup for each of very many rows would be more than a launch takes)
  return p.nsplit > 8 && rows_of(a) < 1 << 23 ? join_by<E, kWaves>(a, p, s) : join_by<E, 1>(a, p, s);
}

// Keys are split where the tiles of rows alone are too few to fill the device's
// 256 compute units, into ranges of at least kRange keys, so that about
// kSplitTarget workgroups share them.  A tile of 32 keys takes a workgroup 1 us
// (fp32 2.6), a second kernel about 4: sequences of fewer than 512 keys (fp32
// 256) are left whole.  Measured, whole against split: B1 H4 T1000 d128 bf16
// training pass 109 and 75 us, B1 H4/2 T1000 d64 fp32 144 and 87, but B1 H4 T300
// d128 bf16 forward 13 and 17.
constexpr int kRange = 128, kSplitTarget = 512;

int key_ranges(const AttnFwd& a, int rows) {  // for tiles of so many rows
  const long wgs = static_cast<long>((a.T + rows - 1) / rows) * a.B * a.H;
  if (wgs == 0 || wgs >= kSplitTarget / 2 || a.S < kRange * (a.dt ? 4 : 2)) return 1;
  const long want = kSplitTarget / wgs, most = a.S / kRange;
  return static_cast<int>(want < most ? want : most);
}
int fwd_splits(const AttnFwd& a) {
  return std::max(key_ranges(a, a.dt ? fwd_rows<uint16_t>(a) : fwd_rows<float>(a)), least_ranges(a.S));
}
int q_shares(const AttnFwd& a) { return key_ranges(a, a.dt ? bwd_rows<uint16_t>(a) : bwd_rows<float>(a)); }
size_t q_floats(const AttnFwd& a) {
  const int n = q_shares(a);
  return n > 1 ? static_cast<size_t>(n) * rows_of(a) * a.maps() * ((a.d + 3) & ~3) : 0;
}

int lam_rows(const AttnFwd& a) {  // workgroups of the q pass, of a head
  const int rows = a.dt ? bwd_rows<uint16_t>(a) : bwd_rows<float>(a);
  return a.B * ((a.T + rows - 1) / rows) * q_shares(a);
}

// The kv pass gives every tile of keys to one workgroup, or to several that share
// the rows: two fit on each of the 256 compute units, and with a causal mask,
// whose tiles differ in length, twice as many even them out.  A share has at
// least kShareRows rows (256 in place of 128: B3 H6/2 T501 fp32 training pass 153
// us and 136, B2 H8/2 T500 d128 bf16 84 and 80).
constexpr int kShareTarget = 1024, kShareRows = 128;

int kv_shares(const AttnFwd& a, bool causal) {
  const long wgs = static_cast<long>((a.S + kBwdKeys - 1) / kBwdKeys) * a.B * a.Hk, rows = static_cast<long>(a.H / a.Hk) * a.T;
  const long target = causal ? kShareTarget : kShareTarget / 2;
  if (wgs == 0 || wgs >= target || rows < 2 * kShareRows) return 1;
  const long want = (target + wgs - 1) / wgs, most = rows / kShareRows;
  return static_cast<int>(want < most ? want : most);
}
size_t kv_floats(const AttnFwd& a) {
  const int n = kv_shares(a, true);
  return n > 1 ? static_cast<size_t>(n) * a.B * a.Hk * a.S * kv_width(a) : 0;
}

// the shares' sums, of the q pass and then of the kv pass
size_t part_floats(const AttnFwd& a) { return std::max(q_floats(a), kv_floats(a)); }

size_t stats_floats(const AttnFwd& a) { return (static_cast<size_t>(rows_of(a)) * a.maps() * 2 + 3) & ~static_cast<size_t>(3); }

}  // namespace

hipError_t launch_join(const AttnFwd& a, const Partial& p, hipStream_t s) {
  return a.dt ? join<uint16_t>(a, p, s) : join<float>(a, p, s);
}

}  // namespace attn

size_t attention_fwd_workspace(const AttnFwd& a) {
  return 4 * attn::partial_floats(attn::rows_of(a), a.maps(), a.dv, attn::fwd_splits(a));
}

size_t attention_bwd_workspace(const AttnFwd& a) {
  return 4 * (attn::stats_floats(a) + attn::part_floats(a) + (a.maps() > 1 ? static_cast<size_t>(attn::lam_rows(a)) * a.H : 0));
}

hipError_t launch_attention_fwd(const AttnFwd& a, void* ws, hipStream_t s) {
  const int n = attn::fwd_splits(a);
  const attn::Partial part = n > 1 ? attn::partial_at(ws, attn::rows_of(a), a.maps(), a.dv, n) : attn::Partial{nullptr, nullptr, 1};
  const hipError_t e = a.dt ? attn::launch_fwd<uint16_t>(a, part, s) : attn::launch_fwd<float>(a, part, s);
  return e != hipSuccess || n == 1 ? e : attn::launch_join(a, part, s);
}

hipError_t launch_attention_bwd(const AttnBwd& g, void* ws, hipStream_t s) {
  const AttnFwd& a = g.f;
  float* stats = static_cast<float*>(ws);
  float* part = stats + attn::stats_floats(a);
  float* lam_part = part + attn::part_floats(a);
  hipError_t e = hipSuccess;
  if (a.T > 0) {
    e = a.dt ? attn::stats<uint16_t>(g, stats, s) : attn::stats<float>(g, stats, s);
    if (e != hipSuccess) return e;
    const int n = attn::q_shares(a);
    e = a.dt ? attn::launch_bwd_q<uint16_t>(g, stats, lam_part, part, n, s) : attn::launch_bwd_q<float>(g, stats, lam_part, part, n, s);
    if (e == hipSuccess && n > 1) e = a.dt ? attn::add_q<uint16_t>(g, part, n, s) : attn::add_q<float>(g, part, n, s);
    if (e != hipSuccess) return e;
  }
  if (a.S > 0) {
    const int n = attn::kv_shares(a, a.causal);
    e = a.dt ? attn::launch_bwd_kv<uint16_t>(g, stats, part, n, s) : attn::launch_bwd_kv<float>(g, stats, part, n, s);
    if (e == hipSuccess && n > 1) e = a.dt ? attn::add<uint16_t>(g, part, n, s) : attn::add<float>(g, part, n, s);
    if (e != hipSuccess) return e;
  }
  if (a.maps() > 1) {
    const ColumnSums c{lam_part, attn::lam_rows(a), a.H, {g.grad_lam, nullptr, nullptr}};
    e = launch_column_sums(c, s);
  }
  return e;
}

}  // namespace ret
