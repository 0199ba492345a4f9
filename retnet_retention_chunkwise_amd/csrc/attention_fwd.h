// Softmax attention over a whole sequence, ordinary (M = 1 map) or differential
// (M = 2):  o[t] = sum_s (A_1 - lam_h A_2)[t,s] v[s],  A_m = softmax over the
// visible s of scale q_m[t] . k_m[s].
//
// A workgroup holds QT rows of q for one query head and streams the keys and
// values through LDS, KT at a time; each wave owns 16 NB rows as the columns of
// its products:
//   S^T[key][row]  = K Q^T    (K from LDS along its rows, Q in registers)
//   O^T[chan][row] += V^T P^T (V from LDS across its rows; P^T is S^T's own
//                              registers, rounded to the tensors' type)
// so a row's scores lie in one lane group's registers and its maximum takes
// two lane swaps.  One pass with a running maximum and sum; the maximum is only
// moved (and O scaled) when a score exceeds it by 2^kSlack: p is then at most
// 2^kSlack instead of 1, which takes as much from the range of the sums and
// nothing from their precision.  Both maps read
// the same value tile once and keep an output each, because they are divided by
// different sums.  Products are bf16 MFMA (fp32: fp32 MFMA); scores, maxima,
// sums and outputs are fp32; p is rounded to bf16 as an operand, which costs as
// much as the output's own rounding and halves the product's time.
//
// 32 rows a wave (bf16, up to 128 channels): a tile's operands are read from LDS
// once for twice the products.  Wider rows leave room for one such wave a SIMD; 16
// rows and two waves are faster (B4 H8 T2048 one map d256: 126 us to 101 when that
// was chosen, 96 now).
// Bound by matrix and vector instructions: a wave does a tile's scores, softmax and
// sums one after the other, and two waves of a SIMD make up for little of that (16
// products of one, 349 clocks, and 32 exponentials of the other, 413, take 617
// together; 16 products with 48 vector instructions in between 453).  About 24 clocks
// of products and 31 of softmax a score at 128 channels and two maps.  B1 H16/4 T8192
// d128 two maps causal: 411 us (1.0 PFLOP/s of visible pairs); B4 H8 T2048 d256: 117
// us (0.88).
#pragma once

#include "attention.h"
#include "attention_tiles.h"

namespace ret {
namespace attn {

constexpr float kSlack = 8.0f;

template <typename E, int MAPS, int DK, int DV, bool kWhole, int NB, int NW, int KT>
__global__ __launch_bounds__(64 * NW, (sizeof(E) == 2 && DV <= 128 ? 2 : 1)) void attention_fwd_kernel(AttnFwd a, Partial part, int tiles) {
  typedef Mma<E> X;
  typedef typename X::Frag Frag;
  constexpr int D = DK / MAPS, THREADS = 64 * NW, QT = 16 * NB * NW;
  constexpr int KB = KT / 16, KS = D / 32, VB = DV / 16;
  constexpr bool kDma = kWhole && sizeof(E) == 2;
  constexpr int SLOTS = DK + DV <= 384 ? 3 : 2;
  typedef Tile<E, DK, kDma> KTile;
  typedef Tile<E, DV, kDma> VTile;
  __shared__ __attribute__((aligned(16))) E K0[KT * KTile::LD], K1[KT * KTile::LD], K2[kDma && SLOTS == 3 ? KT * DK : 16];
  __shared__ __attribute__((aligned(16))) E V0[KT * VTile::LD], V1[KT * VTile::LD], V2[kDma && SLOTS == 3 ? KT * DV : 16];

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), col = lane & 15, grp = lane >> 4;
  // the longest rows of all heads first, so that the last workgroups are short
  const int heads = a.B * a.H, bh = blockIdx.x % heads, tile = tiles - 1 - blockIdx.x / heads;
  const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int split = blockIdx.y;
  const int len = a.lens != nullptr ? min(max(a.lens[b], 0), a.S) : a.S;
  // keys that a row t sees
  auto seen = [&](int t) { return a.causal ? min(max(t + a.offset + 1, 0), len) : len; };
  const int q0 = tile * QT, w0 = q0 + wave * 16 * NB;
  const int kmax = seen(min(q0 + QT, a.T) - 1);  // what lies behind is not read: it may hold anything
  const int all = (kmax + KT - 1) / KT;
  const int first = static_cast<int>(static_cast<long>(all) * split / part.nsplit);
  const int last = static_cast<int>(static_cast<long>(all) * (split + 1) / part.nsplit);
  // keys that some row, and that every row, of this wave sees
  const int wmax = w0 < a.T ? seen(min(w0 + 16 * NB, a.T) - 1) : 0, wall = seen(w0);

  const E* q = static_cast<const E*>(a.q) + b * a.sq.b + h * a.sq.h;
  const E* k = static_cast<const E*>(a.k) + b * a.sk.b + hk * a.sk.h;
  const E* v = static_cast<const E*>(a.v) + b * a.sv.b + hk * a.sv.h;
  Frag qf[NB][MAPS * KS];
  int lim[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int t = w0 + 16 * n + col;
    load_columns<E, MAPS, D, kWhole>(q + min(t, a.T - 1) * a.sq.t, t < a.T, a.d, lane, qf[n]);
    lim[n] = seen(t);
  }

  const float c = a.scale * kLog2e, slack = kSlack / c;
  f32x4 o[MAPS][VB][NB];
  float mx[MAPS][NB], sum[MAPS][NB];
#pragma unroll
  for (int m = 0; m < MAPS; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      mx[m][n] = -INFINITY;
      sum[m][n] = 0.0f;
#pragma unroll
      for (int i = 0; i < VB; ++i) o[m][i][n] = f32x4{0, 0, 0, 0};
    }

  // one tile of keys and values that lie in LDS
  auto use = [&](int i, const E* Ks, const E* Vs) __attribute__((always_inline)) {
    const int k0 = i * KT;
    if (k0 >= wmax) return;
    products_first();
    f32x4 s[MAPS][KB][NB];
#pragma unroll
    for (int m = 0; m < MAPS; ++m)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        Frag kf[KS];
#pragma unroll
        for (int e = 0; e < KS; ++e)
          if (!X::kSkip || 32 * e < a.d) kf[e] = KTile::rows(Ks, 16 * kb, m * D + 32 * e, lane);
#pragma unroll
        for (int n = 0; n < NB; ++n) s[m][kb][n] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < KS; ++e) {
          if (X::kSkip && 32 * e >= a.d) break;
#pragma unroll
          for (int n = 0; n < NB; ++n) s[m][kb][n] = X::mma(kf[e], qf[n][m * KS + e], s[m][kb][n], a.d - 32 * e);
        }
      }
    products_done();
    if (k0 + KT > wall) {  // some row does not see some key
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool out = k0 + 16 * kb + 4 * grp + r >= lim[n];
#pragma unroll
            for (int m = 0; m < MAPS; ++m)
              if (out) s[m][kb][n][r] = -INFINITY;
          }
    }
    float top[MAPS][NB];
    bool over = false;
#pragma unroll
    for (int m = 0; m < MAPS; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        top[m][n] = -INFINITY;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int r = 0; r < 4; ++r) top[m][n] = fmaxf(top[m][n], s[m][kb][n][r]);
        over = over || top[m][n] > mx[m][n] + slack;
      }
    if (__any(over)) {
#pragma unroll
      for (int m = 0; m < MAPS; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const float next = fmaxf(mx[m][n], row4_max(top[m][n]));
          const float f = next == -INFINITY ? 1.0f : fast_exp2((mx[m][n] - next) * c);
          mx[m][n] = next;
          sum[m][n] *= f;
#pragma unroll
          for (int j = 0; j < VB; ++j) o[m][j][n] *= f;
        }
    }
    Frag pf[MAPS][NB][KT / 32];
#pragma unroll
    for (int m = 0; m < MAPS; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float mc = mx[m][n] == -INFINITY ? 0.0f : mx[m][n] * c;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float p = fast_exp2(fmaf(s[m][kb][n][r], c, -mc));
            s[m][kb][n][r] = p;
            sum[m][n] += p;
          }
#pragma unroll
        for (int j = 0; j < KT / 32; ++j) pf[m][n][j] = X::pack(s[m][2 * j][n], s[m][2 * j + 1][n]);
      }
    products_first();
#pragma unroll
    for (int j = 0; j < KT / 32; ++j)
#pragma unroll
      for (int vb = 0; vb < VB; ++vb) {
        if (X::kSkip && 16 * vb >= a.dv) break;
        const Frag vf = VTile::cols(Vs, 32 * j, 16 * vb, lane);
#pragma unroll
        for (int m = 0; m < MAPS; ++m)
#pragma unroll
          for (int n = 0; n < NB; ++n) o[m][vb][n] = X::mma(vf, pf[m][n][j], o[m][vb][n]);
      }
    products_done();
  };
  if constexpr (kDma) {
    const Dma<KT, MAPS, D, NW> kd(a.d, wave, lane);
    const Dma<KT, 1, DV, NW> vd(a.dv, wave, lane);
    E *const Kt[] = {K0, K1, K2}, *const Vt[] = {V0, V1, V2};
    walk_tiles<SLOTS, kd.COUNT + vd.COUNT>(
        first, last,
        [&](int i, auto slot) __attribute__((always_inline)) {
          kd.load(k, a.sk.t, i * KT, kmax, Kt[slot], wave);
          vd.load(v, a.sv.t, i * KT, kmax, Vt[slot], wave);
        },
        [&](int i, auto slot) __attribute__((always_inline)) { use(i, Kt[slot], Vt[slot]); });
  } else {
    // Two tiles in LDS: while one is used the next is written (its loads were sent
    // a tile earlier) and the one after is on its way; one barrier a tile.
    Stage<E, KT, MAPS, D, THREADS, kWhole> ks(a.d, tid);
    Stage<E, KT, 1, DV, THREADS, kWhole> vs(a.dv, tid);
    auto load = [&](int i) {
      ks.load(k, a.sk.t, i * KT, kmax, a.d);
      vs.load(v, a.sv.t, i * KT, kmax, a.dv);
    };
    auto store = [&](int i, int slot) {
      ks.store(slot ? K1 : K0, i * KT, kmax);
      vs.store(slot ? V1 : V0, i * KT, kmax);
    };
    if (first < last) {
      load(first);
      store(first, 0);
      if (first + 1 < last) load(first + 1);
    }
    for (int i = first; i < last; ++i) {
      const int slot = (i - first) & 1;
      lds_barrier();
      if (i + 1 < last) {
        store(i + 1, slot ^ 1);
        if (i + 2 < last) load(i + 2);
      }
      use(i, slot ? K1 : K0, slot ? V1 : V0);
    }
  }

  const float lam = MAPS > 1 ? a.lam[h] : 0.0f;
  const long rows = static_cast<long>(a.B) * a.H * a.T;
#pragma unroll
  for (int m = 0; m < MAPS; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) sum[m][n] = row4_sum(sum[m][n]);
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int t = w0 + 16 * n + col;
    if (t >= a.T) continue;
    const long row = static_cast<long>(bh) * a.T + t;
    if (part.nsplit > 1) {
      const int dv4 = (a.dv + 3) & ~3;
#pragma unroll
      for (int m = 0; m < MAPS; ++m) {
        const long at = (split * rows + row) * MAPS + m;
        if (grp == 0) reinterpret_cast<float2*>(part.ml)[at] = make_float2(mx[m][n] * c, sum[m][n]);
#pragma unroll
        for (int vb = 0; vb < VB; ++vb) {
          const int ch = 16 * vb + 4 * grp;
          if (ch < dv4) *reinterpret_cast<f32x4*>(part.out + at * dv4 + ch) = o[m][vb][n];
        }
      }
      continue;
    }
    float inv[MAPS];
#pragma unroll
    for (int m = 0; m < MAPS; ++m) {
      const float l = sum[m][n];
      inv[m] = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees no key is zero
      if (a.lse != nullptr && grp == 0)
        a.lse[(static_cast<long>(bh) * MAPS + m) * a.T + t] =
            l == 0.0f ? -INFINITY : mx[m][n] * a.scale + logf(l);
    }
    E* out = static_cast<E*>(a.o) + b * a.so.b + h * a.so.h + t * a.so.t;
    E* two = static_cast<E*>(a.second) + row * a.dv;
#pragma unroll
    for (int vb = 0; vb < VB; ++vb) {
      f32x4 y = o[0][vb][n] * inv[0];
      if constexpr (MAPS > 1) {
        const f32x4 z = o[1][vb][n] * inv[1];
        y -= lam * z;
        if (a.second != nullptr) store4<E, kWhole>(two, 16 * vb + 4 * grp, a.dv, z);
      }
      store4<E, kWhole>(out, 16 * vb + 4 * grp, a.dv, y);
    }
  }
}

template <typename E, int DK, int DV>
struct FwdShape {
  static constexpr int NB = sizeof(E) == 2 && DK <= 128 && DV <= 128 ? 2 : 1;
  static constexpr int NW = 4, KT = 32, QT = 16 * NB * NW;
};

// Rows of a tile, for the sizes that hold the call's.
template <typename E>
int fwd_rows(const AttnFwd& a) {
  return with_sizes(a, [](auto, auto dk, auto dv, auto) { return FwdShape<E, decltype(dk)::value, decltype(dv)::value>::QT; });
}

template <typename E>
hipError_t launch_fwd(const AttnFwd& a, const Partial& part, hipStream_t s) {
  return with_sizes(a, [&](auto m, auto dk, auto dv, auto whole) {
    constexpr int M = decltype(m)::value, DK = decltype(dk)::value, DV = decltype(dv)::value;
    constexpr bool W = decltype(whole)::value;
    typedef FwdShape<E, DK, DV> C;
    const int tiles = (a.T + C::QT - 1) / C::QT;
    hipLaunchKernelGGL((attention_fwd_kernel<E, M, DK, DV, W, C::NB, C::NW, C::KT>),
                       dim3(static_cast<unsigned>(tiles) * a.B * a.H, part.nsplit), dim3(64 * C::NW), 0, s, a, part,
                       tiles);
    return hipGetLastError();
  });
}

}  // namespace attn
}  // namespace ret
