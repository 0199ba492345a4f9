// Softmax attention of one new token over a paged cache of keys and values,
// ordinary or differential (attention_fwd.h has the formulas), and the storing
// of new tokens into the pages.
//
// The cache is read once, at the speed of memory.  A workgroup takes up to 16
// query heads that share a key head, as the columns of its products, and a range
// of the keys; its waves take 32 keys at a time: the keys go from memory straight
// into operands, the values through LDS that is the wave's own, so that no wave
// waits for another until the end, where their outputs are joined.  Where
// the sequences and heads alone do not fill the device, the keys are split over
// workgroups and their shares joined by a second launch.  The new token's key
// and value are read from the arguments and stored beside; nobody reads their
// place in the cache during the call.
// Bound by memory: 128 streams of 16/4 heads over up to 2048 tokens, d128 bf16,
// 270 MB in 58 us (4.6 TB/s); 2 of 32/8 over 65536, 537 MB in 97 us and 6 for the
// join.  Few short streams are bound by latency: 8 of 8 over 512, 11 us.
#include "attention.h"

#include <algorithm>

#include "attention_tiles.h"

namespace ret {
namespace attn {
namespace {

constexpr int kKeys = 32;
constexpr float kSlack = 8.0f;  // see attention_fwd.h

template <typename E, int MAPS, int DK, int DV, bool kWhole, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void attention_step_kernel(AttnStep a, Partial part) {
  typedef Mma<E> X;
  typedef typename X::Frag Frag;
  typedef Tile<E, DV, false> VTile;
  constexpr int D = DK / MAPS, KS = D / 32, VB = DV / 16, VLD = VTile::LD;
  constexpr int CE = 16 / static_cast<int>(sizeof(E)), CH = DV / CE;  // pieces of a value row
  constexpr int VR = 64 / CH > 0 ? 64 / CH : 1, VN = kKeys / VR;     // rows of one load of a wave, loads
  static_assert(CH <= 64, "a row per load");
  struct Join {
    float out[kWaves][MAPS][16][DV + 4];
    float2 ml[kWaves][MAPS][16];  // maximum and sum
  };
  union Lds {
    E v[kWaves][kKeys * VLD];
    Join j;
  };
  __shared__ __attribute__((aligned(16))) Lds lds;

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), col = lane & 15, grp = lane >> 4;
  const int G = a.H / a.Hk, blocks = (G + 15) / 16;
  const int gb = blockIdx.x % blocks, bk = blockIdx.x / blocks, b = bk / a.Hk, hk = bk % a.Hk;
  const int split = blockIdx.y;
  const int head = gb * 16 + col;  // of the group
  const bool live = head < G;
  const int h = hk * G + (live ? head : 0);
  const long rows = static_cast<long>(a.B) * a.H, row = static_cast<long>(b) * a.H + h;
  const int len = a.lens[b];
  const int keys = len < 0 ? 0 : min(len, a.max_pages * a.page) + 1;  // the new token's among them
  const int all = (keys + kKeys - 1) / kKeys;
  const int first = static_cast<int>(static_cast<long>(all) * split / part.nsplit);
  const int last = static_cast<int>(static_cast<long>(all) * (split + 1) / part.nsplit);

  const E* knew = static_cast<const E*>(a.k) + b * a.sk.b + hk * a.sk.h;
  const E* vnew = static_cast<const E*>(a.v) + b * a.sv.b + hk * a.sv.h;
  E* kc = static_cast<E*>(a.k_cache) + hk * a.skc.h;
  E* vc = static_cast<E*>(a.v_cache) + hk * a.svc.h;
  const int* table = a.table + static_cast<long>(b) * a.max_pages;

  const float c = a.scale * kLog2e, slack = kSlack / c;
  f32x4 o[MAPS][VB];
  float mx[MAPS], sum[MAPS];
#pragma unroll
  for (int m = 0; m < MAPS; ++m) {
    mx[m] = -INFINITY;
    sum[m] = 0.0f;
#pragma unroll
    for (int i = 0; i < VB; ++i) o[m][i] = f32x4{0, 0, 0, 0};
  }

  // One tile on its way: pieces of the keys' operands and of the value rows, and
  // which keys count.
  constexpr int KP = 8 / CE;  // pieces of an operand
  u32x4 kr[2][MAPS * KS][KP], vr[VN];
  unsigned ok = 0;
  const int vrow = lane / CH, vchunk = (lane % CH) * CE;
  const Piece16<E, kWhole> vpiece(vchunk, a.dv);
  auto kpiece = [&](int e, int i) { return Piece16<E, kWhole>(32 * (e % KS) + CE * grp + 16 * i, a.d); };
  // Lane j finds key j's rows.  Its page is looked up a tile ahead of the rows,
  // which are a memory latency behind it already.
  auto page_of = [&](int tile) {
    const int key = tile * kKeys + (lane & (kKeys - 1));
    return key < keys - 1 ? table[a.page_of(key)] : -1;
  };
  auto load = [&](int tile, int page) {
    // a key without a page (or behind the last) is masked, and the new token's
    // rows are read in its place
    const int key = tile * kKeys + (lane & (kKeys - 1));
    const E *kp = knew, *vp = vnew;
    bool in = key < keys;
    if (key < keys - 1) {
      in = page >= 0 && page < a.pages;
      if (in) {
        const int r = key - a.page_of(key) * a.page;
        kp = kc + page * a.skc.b + r * a.skc.t;
        vp = vc + page * a.svc.b + r * a.svc.t;
      }
    }
    ok = static_cast<unsigned>(__ballot(in));
    auto from = [&](const E* p, int src) {
      const unsigned long x = reinterpret_cast<unsigned long>(p);
      const unsigned lo = __shfl(static_cast<unsigned>(x), src), hi = __shfl(static_cast<unsigned>(x >> 32), src);
      return reinterpret_cast<const E*>(static_cast<unsigned long>(hi) << 32 | lo);
    };
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const E* p = from(kp, 16 * kb + col);
#pragma unroll
      for (int e = 0; e < MAPS * KS; ++e)
#pragma unroll
        for (int i = 0; i < KP; ++i) kr[kb][e][i] = kpiece(e, i).load(reinterpret_cast<const char*>(p + e / KS * a.d), 0, a.d);
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) vr[i] = vpiece.load(reinterpret_cast<const char*>(from(vp, i * VR + vrow)), 0, a.dv);
  };

  E* vs = lds.v[wave];
  int i = first + wave, next_page = -1;
  if (i < last) {
    const int page = page_of(i);
    next_page = page_of(i + kWaves);
    load(i, page);
  }
  Frag qf[MAPS * KS];
  load_columns<E, MAPS, D, kWhole>(static_cast<const E*>(a.q) + b * a.sq.b + h * a.sq.h, live, a.d, lane, qf);
  const float lam = MAPS > 1 ? a.lam[h] : 0.0f;
  // the new token's elements, a thread each, and their page, to be stored below
  const bool stores = len >= 0 && len < a.max_pages * static_cast<long>(a.page) && split == part.nsplit - 1 && gb == 0;
  static_assert(DK <= 64 * kWaves && DV <= 64 * kWaves, "a thread per element");
  int new_page = -1;
  E new_k, new_v;
  if (stores) {
    new_page = table[a.page_of(len)];
    if (tid < MAPS * a.d) new_k = knew[tid];
    if (tid < a.dv) new_v = vnew[tid];
  }
  for (; i < last; i += kWaves) {
#pragma unroll
    for (int j = 0; j < VN; ++j)
      *reinterpret_cast<u32x4*>(vs + (j * VR + vrow) * VLD + vchunk) = vpiece.finish(vr[j]);
    f32x4 s[MAPS][2];
#pragma unroll
    for (int m = 0; m < MAPS; ++m)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        s[m][kb] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = m * KS; e < (m + 1) * KS; ++e) {
          const int left = a.d - 32 * (e - m * KS);
          if (X::kSkip && left <= 0) break;
          u32x4 x[KP];
#pragma unroll
          for (int j = 0; j < KP; ++j) x[j] = kpiece(e, j).finish(kr[kb][e][j]);
          Frag kf;
          __builtin_memcpy(&kf, x, sizeof(kf));
          s[m][kb] = X::mma(kf, qf[e], s[m][kb], left);
        }
      }
    const unsigned seen = ok;
    if (i + kWaves < last) {
      load(i + kWaves, next_page);
      next_page = page_of(i + 2 * kWaves);
    }
    if (seen != 0xffffffffu) {
#pragma unroll
      for (int m = 0; m < MAPS; ++m)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!(seen >> (16 * kb + 4 * grp + r) & 1)) s[m][kb][r] = -INFINITY;
    }
    Frag pf[MAPS];
#pragma unroll
    for (int m = 0; m < MAPS; ++m) {
      float top = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, s[m][kb][r]);
      if (__any(top > mx[m] + slack)) {
        const float next = fmaxf(mx[m], row4_max(top));
        const float f = next == -INFINITY ? 1.0f : fast_exp2((mx[m] - next) * c);
        mx[m] = next;
        sum[m] *= f;
#pragma unroll
        for (int j = 0; j < VB; ++j) o[m][j] *= f;
      }
      const float mc = mx[m] == -INFINITY ? 0.0f : mx[m] * c;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float p = fast_exp2(fmaf(s[m][kb][r], c, -mc));
          s[m][kb][r] = p;
          sum[m] += p;
        }
      pf[m] = X::pack(s[m][0], s[m][1]);
    }
    // the wave's own rows: written above, read by other lanes below
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
#pragma unroll
    for (int vb = 0; vb < VB; ++vb) {
      if (X::kSkip && 16 * vb >= a.dv) break;
      const Frag vf = VTile::cols(vs, 0, 16 * vb, lane);
#pragma unroll
      for (int m = 0; m < MAPS; ++m) o[m][vb] = X::mma(vf, pf[m], o[m][vb]);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
  }

  if (stores && new_page >= 0 && new_page < a.pages) {
    const int r = len - a.page_of(len) * a.page;
    if (tid < MAPS * a.d) kc[new_page * a.skc.b + r * a.skc.t + tid] = new_k;
    if (tid < a.dv) vc[new_page * a.svc.b + r * a.svc.t + tid] = new_v;
  }

  // the waves' shares side by side; every thread adds its part of them onto one
  // maximum, in wave order
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MAPS; ++m) {
    sum[m] = row4_sum(sum[m]);
    if (grp == 0) lds.j.ml[wave][m][col] = make_float2(mx[m], sum[m]);
#pragma unroll
    for (int j = 0; j < VB; ++j) *reinterpret_cast<f32x4*>(&lds.j.out[wave][m][col][16 * j + 4 * grp]) = o[m][j];
  }
  __syncthreads();
  if (!live) return;
  float f[MAPS][kWaves];
#pragma unroll
  for (int m = 0; m < MAPS; ++m) {
    float2 ml[kWaves];
    float top = -INFINITY, l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      ml[w] = lds.j.ml[w][m][col];
      top = fmaxf(top, ml[w].x);
    }
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[m][w] = ml[w].x == -INFINITY ? 0.0f : fast_exp2((ml[w].x - top) * c);
      l = fmaf(ml[w].y, f[m][w], l);
    }
    mx[m] = top;
    sum[m] = l;
  }
  auto joined = [&](int m, int ch) {
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) x += *reinterpret_cast<const f32x4*>(&lds.j.out[w][m][col][ch]) * f[m][w];
    return x;
  };
  // wave w writes channels 4 grp.. of the blocks w, w + kWaves, ...
  const int dv4 = (a.dv + 3) & ~3;
  if (part.nsplit > 1) {
#pragma unroll
    for (int m = 0; m < MAPS; ++m) {
      const long at = (split * rows + row) * MAPS + m;
      if (tid < 16) reinterpret_cast<float2*>(part.ml)[at] = make_float2(mx[m] * c, sum[m]);
      for (int vb = wave; vb < VB; vb += kWaves) {
        const int ch = 16 * vb + 4 * grp;
        if (ch < dv4) *reinterpret_cast<f32x4*>(part.out + at * dv4 + ch) = joined(m, ch);
      }
    }
    return;
  }
  float inv[MAPS];
#pragma unroll
  for (int m = 0; m < MAPS; ++m) inv[m] = sum[m] == 0.0f ? 0.0f : 1.0f / sum[m];
  E* out = static_cast<E*>(a.o) + b * a.so.b + h * a.so.h;
  for (int vb = wave; vb < VB; vb += kWaves) {
    const int ch = 16 * vb + 4 * grp;
    f32x4 y = joined(0, ch) * inv[0];
    if constexpr (MAPS > 1) y -= joined(1, ch) * (inv[1] * lam);
    store4<E, kWhole>(out, ch, a.dv, y);
  }
}

// Rows of keys and values, 16 bytes a lane, LPR lanes a row; a row's last piece
// reaches back over the one before.
template <typename E>
__device__ __forceinline__ void copy_row(const E* from, E* to, int n, int lane) {
  constexpr int CE = 16 / static_cast<int>(sizeof(E));
  typedef RawOf<16, static_cast<int>(sizeof(E))> R;
  int c = lane * CE;
  if (c >= n) return;
  if (n < CE) {
    for (; c < n; ++c) to[c] = from[c];
    return;
  }
  c = min(c, n - CE);
  __builtin_nontemporal_store(__builtin_nontemporal_load(reinterpret_cast<const typename R::at*>(from + c)),
                              reinterpret_cast<typename R::at*>(to + c));
}

// Bound by memory, and read and written once: past the caches.  4 x 2048 tokens of
// 8 heads, 256 + 256 channels bf16: 134 MB in 27 us (5.0 TB/s).
constexpr int kAppendThreads = 256, kAppendRounds = 4;

template <typename E, int LPR>
__global__ __launch_bounds__(kAppendThreads) void cache_append_kernel(CacheAppend a, int tiles) {
  constexpr int STEP = kAppendThreads / LPR;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / a.Hk, h = bh % a.Hk;
  const int lane = threadIdx.x % LPR;
  const int start = a.start[b], count = a.counts != nullptr ? min(a.counts[b], a.T) : a.T;
  if (start < 0) return;
  const E* k = static_cast<const E*>(a.k) + b * a.sk.b + h * a.sk.h;
  const E* v = static_cast<const E*>(a.v) + b * a.sv.b + h * a.sv.h;
#pragma unroll
  for (int i = 0; i < kAppendRounds; ++i) {
    const int t = (tile * kAppendRounds + i) * STEP + static_cast<int>(threadIdx.x) / LPR;
    const long at = static_cast<long>(start) + t;
    if (t >= count || at >= static_cast<long>(a.max_pages) * a.page) return;
    const int page = a.table[static_cast<long>(b) * a.max_pages + static_cast<int>(at) / a.page];
    const int r = static_cast<int>(at) % a.page;
    if (page < 0 || page >= a.pages) continue;
    copy_row(k + t * a.sk.t, static_cast<E*>(a.k_cache) + page * a.skc.b + h * a.skc.h + r * a.skc.t, a.dk, lane);
    copy_row(v + t * a.sv.t, static_cast<E*>(a.v_cache) + page * a.svc.b + h * a.svc.h + r * a.svc.t, a.dv, lane);
  }
}

template <typename E, int LPR>
hipError_t append(const CacheAppend& a, hipStream_t s) {
  constexpr int ROWS = kAppendThreads / LPR * kAppendRounds;
  const int tiles = (a.T + ROWS - 1) / ROWS;
  hipLaunchKernelGGL((cache_append_kernel<E, LPR>), dim3(static_cast<unsigned>(tiles) * a.B * a.Hk),
                     dim3(kAppendThreads), 0, s, a, tiles);
  return hipGetLastError();
}

template <typename E>
hipError_t append_by_width(const CacheAppend& a, hipStream_t s) {
  const int bytes = (a.dk > a.dv ? a.dk : a.dv) * static_cast<int>(sizeof(E));
  if (bytes <= 16 * 16) return append<E, 16>(a, s);
  if (bytes <= 32 * 16) return append<E, 32>(a, s);
  return append<E, 64>(a, s);
}

// Keys are split where the sequences and key heads alone give fewer than
// kStepTarget / 2 workgroups (two fit on a compute unit), into ranges that take a
// wave longer than the second launch: four tiles of bf16, two of fp32, whose
// products are slower.  With four waves a workgroup, 8 streams of 8 heads over 512
// tokens bf16: one range 14.6 us a call, two 18; 15 heads over 3001 tokens fp32: ranges of 256 tokens
// 26.6 us, of 512 35, of 128 31.
constexpr int kStepTarget = 1024;

int step_splits(const AttnStep& a) {
  const int blocks = (a.H / a.Hk + 15) / 16, range = a.dt ? 512 : 256;
  const long wgs = static_cast<long>(a.B) * a.Hk * blocks, keys = static_cast<long>(a.max_pages) * a.page;
  const int least = least_ranges(keys);
  if (wgs >= kStepTarget / 2 || keys < 2 * range) return least;
  const long want = kStepTarget / wgs, most = keys / range;
  return std::max(least, static_cast<int>(want < most ? want : most));
}

template <typename E>
hipError_t step(const AttnStep& a, const Partial& p, hipStream_t s) {
  return with_sizes(a, [&](auto m, auto dk, auto dv, auto whole) {
    constexpr int M = decltype(m)::value, DK = decltype(dk)::value, DV = decltype(dv)::value;
    constexpr bool W = decltype(whole)::value;
    const unsigned wgs = static_cast<unsigned>(a.B) * a.Hk * ((a.H / a.Hk + 15) / 16);
    // Workgroups that have a compute unit each to themselves take eight waves, whose
    // chains of tiles are half as long: 8 streams of 8 heads over 512 tokens 11.2 us,
    // with four 12.4; where all units are taken they only make the join longer (128
    // streams 63.7 us, with four 61).  Wider heads and fp32 have no registers for it.
    if constexpr (sizeof(E) == 2 && DK + DV <= 256) {
      if (static_cast<long>(wgs) * p.nsplit <= 256) {
        hipLaunchKernelGGL((attention_step_kernel<E, M, DK, DV, W, 8>), dim3(wgs, p.nsplit), dim3(64 * 8), 0, s, a, p);
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((attention_step_kernel<E, M, DK, DV, W, 4>), dim3(wgs, p.nsplit), dim3(64 * 4), 0, s, a, p);
    return hipGetLastError();
  });
}

}  // namespace
}  // namespace attn

size_t attention_step_workspace(const AttnStep& a) {
  return 4 * attn::partial_floats(static_cast<long>(a.B) * a.H, a.maps(), a.dv, attn::step_splits(a));
}

hipError_t launch_attention_step(const AttnStep& a, void* ws, hipStream_t s) {
  const int n = attn::step_splits(a);
  const attn::Partial p =
      n > 1 ? attn::partial_at(ws, static_cast<long>(a.B) * a.H, a.maps(), a.dv, n) : attn::Partial{nullptr, nullptr, 1};
  const hipError_t e = a.dt ? attn::step<uint16_t>(a, p, s) : attn::step<float>(a, p, s);
  if (e != hipSuccess || n == 1) return e;
  AttnFwd f{};  // the join's view: one row for every batch element and head
  f.lam = a.lam;
  f.o = a.o;
  f.so = a.so;
  f.B = a.B;
  f.H = a.H;
  f.T = 1;
  f.dv = a.dv;
  f.dt = a.dt;
  return attn::launch_join(f, p, s);
}

hipError_t launch_cache_append(const CacheAppend& a, hipStream_t s) {
  return a.dt ? attn::append_by_width<uint16_t>(a, s) : attn::append_by_width<float>(a, s);
}

}  // namespace ret
