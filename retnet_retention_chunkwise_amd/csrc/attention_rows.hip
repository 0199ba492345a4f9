// The attention calls' host side and their per-row kernels: the join of split
// keys and the backward's row statistics.  Both are bound by memory.
#include "attention.h"

#include "attention_tiles.h"
#include "row_sum.h"

namespace ret {
namespace attn {
namespace {

constexpr int kWaves = 4;

// One wave per row, four channels a lane.  The shares' outputs o_i with maxima
// m_i and sums l_i join as sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i.
template <typename E, int MAPS>
__global__ __launch_bounds__(64 * kWaves) void attention_join_kernel(AttnFwd a, Partial p, long rows) {
  const int lane = threadIdx.x & 63, ch = 4 * lane;
  const long row = static_cast<long>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int t = static_cast<int>(row % a.T), dv4 = (a.dv + 3) & ~3;
  const long bh = row / a.T;
  const int h = static_cast<int>(bh % a.H), b = static_cast<int>(bh / a.H);
  const float2* ml = reinterpret_cast<const float2*>(p.ml);
  f32x4 y[MAPS];
#pragma unroll
  for (int m = 0; m < MAPS; ++m) {
    float top = -INFINITY;
    for (int i = 0; i < p.nsplit; ++i) top = fmaxf(top, ml[(i * rows + row) * MAPS + m].x);
    const float at = top == -INFINITY ? 0.0f : top;
    float l = 0.0f;
    f32x4 x = {0, 0, 0, 0};
    for (int i = 0; i < p.nsplit; ++i) {
      const long j = (i * rows + row) * MAPS + m;
      const float2 s = ml[j];
      if (s.x == -INFINITY) continue;  // a share without keys wrote no outputs
      const float f = fast_exp2(s.x - at);
      l = fmaf(s.y, f, l);
      if (ch < dv4) x += *reinterpret_cast<const f32x4*>(p.out + j * dv4 + ch) * f;
    }
    y[m] = x * (l == 0.0f ? 0.0f : 1.0f / l);
    if (a.lse != nullptr && lane == 0)
      a.lse[(bh * MAPS + m) * a.T + t] = l == 0.0f ? -INFINITY : top * kLn2 + logf(l);
  }
  if constexpr (MAPS > 1) {
    if (a.second != nullptr) store4<E>(static_cast<E*>(a.second) + row * a.dv, ch, a.dv, y[1]);
    y[0] -= a.lam[h] * y[1];
  }
  store4<E>(static_cast<E*>(a.o) + b * a.so.b + h * a.so.h + t * a.so.t, ch, a.dv, y[0]);
}

// {lse log2 e, D} of every row and map, one wave per row.  A row that saw no key
// gets +inf, so that exp2(score - lse) is zero there.
template <typename E, int MAPS>
__global__ __launch_bounds__(64 * kWaves) void attention_stats_kernel(AttnBwd g, float2* stats, long rows) {
  const AttnFwd& a = g.f;
  const int lane = threadIdx.x & 63, ch = 4 * lane;
  const long row = static_cast<long>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int t = static_cast<int>(row % a.T);
  const long bh = row / a.T;
  const int h = static_cast<int>(bh % a.H), b = static_cast<int>(bh / a.H);
  const E* o = static_cast<const E*>(a.o) + b * a.so.b + h * a.so.h + t * a.so.t;
  const E* d = static_cast<const E*>(g.grad_o) + b * g.sdo.b + h * g.sdo.h + t * g.sdo.t;
  const E* z = static_cast<const E*>(a.second) + row * a.dv;
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (ch + i < a.dv) {
      const float x = Elem<E>::load(d, ch + i);
      s[0] = fmaf(x, Elem<E>::load(o, ch + i), s[0]);
      if constexpr (MAPS > 1) s[1] = fmaf(x, Elem<E>::load(z, ch + i), s[1]);
    }
  s[0] = lanes_sum<64>(s[0]);
  if constexpr (MAPS > 1) {
    s[1] = lanes_sum<64>(s[1]);
    s[0] = fmaf(a.lam[h], s[1], s[0]);
  }
  if (lane < MAPS) {
    const float l = a.lse[(bh * MAPS + lane) * a.T + t];
    stats[lane * rows + row] = make_float2(l == -INFINITY ? INFINITY : l * kLog2e, lane == 0 ? s[0] : s[1]);
  }
}

unsigned row_blocks(long rows) { return static_cast<unsigned>((rows + kWaves - 1) / kWaves); }

template <typename E>
hipError_t stats(const AttnBwd& g, float* to, hipStream_t s) {
  const long rows = static_cast<long>(g.f.B) * g.f.H * g.f.T;
  auto* kern = g.f.maps() > 1 ? attention_stats_kernel<E, 2> : attention_stats_kernel<E, 1>;
  hipLaunchKernelGGL(kern, dim3(row_blocks(rows)), dim3(64 * kWaves), 0, s, g, reinterpret_cast<float2*>(to), rows);
  return hipGetLastError();
}

template <typename E>
hipError_t join(const AttnFwd& a, const Partial& p, hipStream_t s) {
  const long rows = static_cast<long>(a.B) * a.H * a.T;
  auto* kern = a.maps() > 1 ? attention_join_kernel<E, 2> : attention_join_kernel<E, 1>;
  hipLaunchKernelGGL(kern, dim3(row_blocks(rows)), dim3(64 * kWaves), 0, s, a, p, rows);
  return hipGetLastError();
}

long rows_of(const AttnFwd& a) { return static_cast<long>(a.B) * a.H * a.T; }

// Keys are split where the tiles of rows alone are too few to fill the device's
// 256 compute units, into ranges of at least kSplitKeys keys.
constexpr int kSplitKeys = 256, kSplitTarget = 512;

int fwd_splits(const AttnFwd& a) {
  const int rows = a.dt ? fwd_rows<uint16_t>(a) : fwd_rows<float>(a);
  const long wgs = static_cast<long>((a.T + rows - 1) / rows) * a.B * a.H;
  if (wgs == 0 || wgs >= kSplitTarget / 2 || a.S < 2 * kSplitKeys) return 1;
  const long want = kSplitTarget / wgs, most = a.S / kSplitKeys;
  return static_cast<int>(want < most ? want : most);
}

int lam_rows(const AttnFwd& a) {  // tiles of the q pass
  const int rows = a.dt ? bwd_q_rows<uint16_t>(a) : bwd_q_rows<float>(a);
  return a.B * ((a.T + rows - 1) / rows);
}

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
  return 4 * (attn::stats_floats(a) + (a.maps() > 1 ? static_cast<size_t>(attn::lam_rows(a)) * a.H : 0));
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
  float* lam_part = stats + attn::stats_floats(a);
  hipError_t e = hipSuccess;
  if (a.T > 0) {
    e = a.dt ? attn::stats<uint16_t>(g, stats, s) : attn::stats<float>(g, stats, s);
    if (e != hipSuccess) return e;
    e = a.dt ? attn::launch_bwd_q<uint16_t>(g, stats, lam_part, s) : attn::launch_bwd_q<float>(g, stats, lam_part, s);
    if (e != hipSuccess) return e;
  }
  if (a.S > 0) {
    e = a.dt ? attn::launch_bwd_kv<uint16_t>(g, stats, s) : attn::launch_bwd_kv<float>(g, stats, s);
    if (e != hipSuccess) return e;
  }
  if (a.maps() > 1) {
    const ColumnSums c{lam_part, attn::lam_rows(a), a.H, {g.grad_lam, nullptr, nullptr}};
    e = launch_column_sums(c, s);
  }
  return e;
}

}  // namespace ret
