// Gradients of softmax attention (attention_fwd.h).  With dP = dO V^T and
// D_m[t] = sum_s A_m dP:
//   dV = (A_1 - lam A_2)^T dO,
//   dS_1 = A_1 (dP - D_1),  dS_2 = -lam A_2 (dP - D_2),
//   dq_m = scale dS_m k_m,  dk_m = scale dS_m^T q_m,  dlam = -sum A_2 dP,
// A_m = exp(scale q_m . k_m - lse_m) from the forward's lse.  Three launches:
//   rows    D_2 = dO . second and D_1 = dO . o + lam D_2 of every row, with
//           lse log2 e beside them;
//   q pass  a wave owns 16 NB rows as columns and streams keys and values
//           through LDS, as the forward does: S^T, dP^T and then
//           dQ^T[chan][row] += K^T dS^T;
//   kv pass a wave owns 16 NB keys as columns and streams q and dO of every
//           head that shares them: S, dP, then dV^T += dO^T P and
//           dK^T += Q^T dS.
// The scores are computed twice (7 products in place of 5) so that every
// gradient is summed by one wave in a fixed order: no atomics, the same bits
// every time.  P and dS are rounded to the tensors' type as operands, all else
// is fp32.  bf16 rounds o, so D from it is off by some 2^-9 of what dP - D
// cancels from; where few keys share a row's weight that is much of what is
// left.  A row that ends in its first tile of keys therefore takes D from the
// tile itself and leaves it to the kv pass.  A longer row keeps the D of the
// rounded o, however few of its keys carry its weight: for unit inputs of 64
// channels dq is off by 0.0024 of itself with the exact D, and by 0.0027, 0.0032
// and 0.0038 where 9, 3 and 2 keys carry the row; where one key does and the
// others weigh e^-12 of it, what little is left is off by a quarter and more.
//
// Bound as the forward is; B2 H16/4 T4096 d128 two maps causal: q pass 257 us,
// kv pass 373 (0.28 TFLOP executed), rows 28.  The kv pass holds 16 keys a wave:
// with 32 the accumulators spill, with a third wave a SIMD they do too (1440 us for
// the whole training pass in place of 924, when measured).  Its operands are read a
// stage ahead, which the compiler would undo without barriers (918 us, 831 with).
// With two maps it reads its head's weight once a tile, behind that tile's loads,
// and waits for all of them with it: a tile is on its way for less than the tile's
// time before it that three slots would allow.
#pragma once

#include "attention.h"
#include "attention_tiles.h"
#include "row_sum.h"

namespace ret {
namespace attn {

// stats: [M][B*H*T] of {lse log2 e, D}: first all of map 1.
template <typename E, int MAPS, int DK, int DV, bool kWhole, int NB, int NW, int KT>
__global__ __launch_bounds__(64 * NW, (sizeof(E) == 2 && DK + DV <= 256 ? 2 : 1)) void attention_bwd_q_kernel(AttnBwd g, float2* stats,
                                                                  float* __restrict__ lam_part, float* __restrict__ part,
                                                                  int tiles, int shares) {
  typedef Mma<E> X;
  typedef typename X::Frag Frag;
  constexpr int D = DK / MAPS, THREADS = 64 * NW, QT = 16 * NB * NW;
  constexpr int KB = KT / 16, KS = D / 32, VS = DV / 32, CB = D / 16;
  constexpr bool kDma = kWhole && sizeof(E) == 2;
  constexpr int SLOTS = DK + DV <= 384 ? 3 : 2;
  typedef Tile<E, DK, kDma> KTile;
  typedef Tile<E, DV, kDma> VTile;
  __shared__ __attribute__((aligned(16))) E K0[KT * KTile::LD], K1[KT * KTile::LD], K2[kDma && SLOTS == 3 ? KT * DK : 16];
  __shared__ __attribute__((aligned(16))) E V0[KT * VTile::LD], V1[KT * VTile::LD], V2[kDma && SLOTS == 3 ? KT * DV : 16];
  __shared__ float wave_lam[NW];

  const AttnFwd& a = g.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), col = lane & 15, grp = lane >> 4;
  // the longest rows of all heads first, so that the last workgroups are short
  const int heads = a.B * a.H, bh = blockIdx.x % heads, tile = tiles - 1 - blockIdx.x / heads;
  const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int len = a.lens != nullptr ? min(max(a.lens[b], 0), a.S) : a.S;
  auto seen = [&](int t) { return a.causal ? min(max(t + a.offset + 1, 0), len) : len; };
  const int q0 = tile * QT, w0 = q0 + wave * 16 * NB;
  // this workgroup's share of the rows' tiles of keys
  const int kmax = seen(min(q0 + QT, a.T) - 1);  // what lies behind is not read: it may hold anything
  const int share = blockIdx.y, all = (kmax + KT - 1) / KT;
  const int first = static_cast<int>(static_cast<long>(all) * share / shares);
  const int last = static_cast<int>(static_cast<long>(all) * (share + 1) / shares);
  const int wmax = w0 < a.T ? seen(min(w0 + 16 * NB, a.T) - 1) : 0, wall = seen(w0);

  const E* q = static_cast<const E*>(a.q) + b * a.sq.b + h * a.sq.h;
  const E* dout = static_cast<const E*>(g.grad_o) + b * g.sdo.b + h * g.sdo.h;
  const E* k = static_cast<const E*>(a.k) + b * a.sk.b + hk * a.sk.h;
  const E* v = static_cast<const E*>(a.v) + b * a.sv.b + hk * a.sv.h;
  const long rows = static_cast<long>(a.B) * a.H * a.T;
  Frag qf[NB][MAPS * KS], gf[NB][VS];
  int lim[NB];
  float2 st[MAPS][NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int t = w0 + 16 * n + col;
    const int row = min(t, a.T - 1);
    load_columns<E, MAPS, D, kWhole>(q + row * a.sq.t, t < a.T, a.d, lane, qf[n]);
    load_columns<E, 1, DV, kWhole>(dout + row * g.sdo.t, t < a.T, a.dv, lane, gf[n]);
    lim[n] = seen(t);
#pragma unroll
    for (int m = 0; m < MAPS; ++m)
      st[m][n] = t < a.T ? stats[m * rows + static_cast<long>(bh) * a.T + t] : make_float2(INFINITY, 0.0f);
  }
  const float c = a.scale * kLog2e;
  f32x4 dq[MAPS][CB][NB];
#pragma unroll
  for (int m = 0; m < MAPS; ++m)
#pragma unroll
    for (int i = 0; i < CB; ++i)
#pragma unroll
      for (int n = 0; n < NB; ++n) dq[m][i][n] = f32x4{0, 0, 0, 0};
  float lam_sum = 0.0f;

  auto use = [&](int i, const E* Ks, const E* Vs) __attribute__((always_inline)) {
    const int k0 = i * KT;
    if (k0 >= wmax) return;
    products_first();
    f32x4 dp[KB][NB], s[MAPS][KB][NB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      Frag vf[VS];
#pragma unroll
      for (int e = 0; e < VS; ++e)
        if (!X::kSkip || 32 * e < a.dv) vf[e] = VTile::rows(Vs, 16 * kb, 32 * e, lane);
#pragma unroll
      for (int n = 0; n < NB; ++n) dp[kb][n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < VS; ++e) {
        if (X::kSkip && 32 * e >= a.dv) break;
#pragma unroll
        for (int n = 0; n < NB; ++n) dp[kb][n] = X::mma(vf[e], gf[n][e], dp[kb][n], a.dv - 32 * e);
      }
    }
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
    if constexpr (sizeof(E) == 2) {
      // Rows that end in their first tile of keys (a wave's first row is its shortest)
      // take D from it, for this pass and the next.
      if (k0 == 0 && wall <= KT) {
#pragma unroll
        for (int m = 0; m < MAPS; ++m)
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            float x = 0.0f;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                x = fmaf(fast_exp2(fmaf(s[m][kb][n][r], c, -st[m][n].x)), dp[kb][n][r], x);
            x = row4_sum(x);
            const bool few = lim[n] <= KT;
            if (few) st[m][n].y = x;
            // another share may read either value: it has no keys for these rows
            const int t = w0 + 16 * n + col;
            if (few && grp == 0 && t < a.T) stats[m * rows + static_cast<long>(bh) * a.T + t].y = x;
          }
      }
    }
#pragma unroll
    for (int m = 0; m < MAPS; ++m) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float p = fast_exp2(fmaf(s[m][kb][n][r], c, -st[m][n].x));
            if (m == 1) lam_sum = fmaf(p, dp[kb][n][r], lam_sum);
            s[m][kb][n][r] = p * (dp[kb][n][r] - st[m][n].y);
          }
      products_first();
#pragma unroll
      for (int j = 0; j < KT / 32; ++j) {
        Frag ds[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) ds[n] = X::pack(s[m][2 * j][n], s[m][2 * j + 1][n]);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          if (X::kSkip && 16 * cb >= a.d) break;
          const Frag kt = KTile::cols(Ks, 32 * j, m * D + 16 * cb, lane);
#pragma unroll
          for (int n = 0; n < NB; ++n) dq[m][cb][n] = X::mma(kt, ds[n], dq[m][cb][n]);
        }
      }
      products_done();
    }
  };
  // tiles in LDS as in the forward
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
    Stage<E, KT, MAPS, D, THREADS, kWhole> ks(a.d, tid);
    Stage<E, KT, 1, DV, THREADS, kWhole> vs(a.dv, tid);
    auto load = [&](int i) {
      ks.load(k, a.sk.t, i * KT, kmax, a.d);
      vs.load(v, a.sv.t, i * KT, kmax, a.dv);
    };
    auto store = [&](int i) {
      ks.store(i & 1 ? K1 : K0, i * KT, kmax);
      vs.store(i & 1 ? V1 : V0, i * KT, kmax);
    };
    if (first < last) {
      load(first);
      store(first);
      if (first + 1 < last) load(first + 1);
    }
    for (int i = first; i < last; ++i) {
      lds_barrier();
      if (i + 1 < last) {
        store(i + 1);
        if (i + 2 < last) load(i + 2);
      }
      use(i, i & 1 ? K1 : K0, i & 1 ? V1 : V0);
    }
  }

  if constexpr (MAPS > 1) {  // this tile's share of the weight's gradient, in a fixed order
    const float w = lanes_sum<64>(lam_sum);
    if (lane == 0) wave_lam[wave] = w;
    __syncthreads();
    if (tid == 0) {
      float x = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) x += wave_lam[i];
      lam_part[((static_cast<long>(b) * tiles + tile) * shares + share) * a.H + h] = -x;
    }
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int t = w0 + 16 * n + col;
    if (t >= a.T) continue;
    E* out = static_cast<E*>(g.grad_q) + b * g.sdq.b + h * g.sdq.h + t * g.sdq.t;
    const int d4 = (a.d + 3) & ~3;
    float* to = part + (share * rows + static_cast<long>(bh) * a.T + t) * (MAPS * d4);
#pragma unroll
    for (int m = 0; m < MAPS; ++m) {
      const float f = m == 0 ? a.scale : -a.lam[h] * a.scale;
      if (shares > 1) {  // fp32 sums of the share, [share][b, h, row][MAPS d4]
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) store4<float, true>(to + m * d4, 16 * cb + 4 * grp, d4, dq[m][cb][n] * f);
        continue;
      }
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) store4<E, kWhole>(out + m * a.d, 16 * cb + 4 * grp, a.d, dq[m][cb][n] * f);
    }
  }
}

template <typename E, int MAPS, int DK, int DV, bool kWhole, int NB, int NW, int QT>
__global__ __launch_bounds__(64 * NW, (sizeof(E) == 2 && (kWhole || DK + DV <= 256) ? 2 : 1)) void attention_bwd_kv_kernel(AttnBwd g, const float2* __restrict__ stats,
                                                                      float* __restrict__ part, int shares) {
  typedef Mma<E> X;
  typedef typename X::Frag Frag;
  constexpr int D = DK / MAPS, THREADS = 64 * NW, KT = 16 * NB * NW;
  constexpr int QB = QT / 16, KS = D / 32, VS = DV / 32, CB = D / 16, VB = DV / 16;
  constexpr bool kDma = kWhole && sizeof(E) == 2;
  constexpr int SLOTS = DK + DV <= 384 ? 3 : 2;
  typedef Tile<E, DK, kDma> QTile;
  typedef Tile<E, DV, kDma> GTile;
  // Operands are read a stage ahead, except beside the sums of wide rows, which
  // leave registers for that or for a second wave on the SIMD: the wave gains more
  // (B2 H8 T2000 one map d256: training pass 308 us, reading ahead 370), though most
  // of these kernels then spill 2 to 11 registers, and what is read back in the loop
  // waits for the loads under way.  Rows that are not whole spill more, and lose by it
  // (T1500 250 and 201 channels: 424 us, reading ahead 401).
  constexpr bool kAhead = sizeof(E) == 2 && (!kWhole || DK + DV <= 256);
  __shared__ __attribute__((aligned(16))) E Q0[QT * QTile::LD], Q1[QT * QTile::LD], Q2[kDma && SLOTS == 3 ? QT * DK : 16];
  __shared__ __attribute__((aligned(16))) E G0[QT * GTile::LD], G1[QT * GTile::LD], G2[kDma && SLOTS == 3 ? QT * DV : 16];
  // statistics of a tile's rows, {lse log2 e, D}; with straight loads every wave
  // brings a map's, so that all have as many loads, and the first copies are used
  constexpr int SC = kDma ? (NW > MAPS ? NW : MAPS) : MAPS;
  __shared__ __attribute__((aligned(16))) float2 S0[SC * QT], S1[SC * QT], S2[kDma && SLOTS == 3 ? SC * QT : 1];
  static_assert(MAPS * QT <= THREADS, "a thread per row's statistics");

  const AttnFwd& a = g.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), col = lane & 15, grp = lane >> 4;
  // the keys that most rows see first, of all heads and shares
  const int heads = a.B * a.Hk, bh = blockIdx.x % heads, share = blockIdx.x / heads % shares, tile = blockIdx.x / heads / shares;
  const int b = bh / a.Hk, hk = bh % a.Hk, G = a.H / a.Hk;
  // keys that some row sees; the others count as zeros, whatever they hold, and have no gradient
  const int all = a.lens != nullptr ? min(max(a.lens[b], 0), a.S) : a.S;
  const int len = a.causal ? min(max(a.T + a.offset, 0), all) : all;
  const int k0 = tile * KT, w0 = k0 + wave * 16 * NB;
  // the first row that sees a key
  auto from = [&](int key) { return a.causal ? min(max(key - a.offset, 0), a.T) : 0; };
  const int t0 = from(k0) / QT * QT, n_tiles = k0 < len ? (a.T - t0 + QT - 1) / QT : 0;
  // rows that see some key, and every key, of this wave
  const int wfirst = w0 < len ? from(w0) : a.T, wall = from(w0 + 16 * NB - 1);

  const E* k = static_cast<const E*>(a.k) + b * a.sk.b + hk * a.sk.h;
  const E* v = static_cast<const E*>(a.v) + b * a.sv.b + hk * a.sv.h;
  const long rows = static_cast<long>(a.B) * a.H * a.T;
  Frag kf[NB][MAPS * KS], vf[NB][VS];
  int lim[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int key = w0 + 16 * n + col, row = min(key, a.S - 1);
    load_columns<E, MAPS, D, kWhole>(k + row * a.sk.t, key < len, a.d, lane, kf[n]);
    load_columns<E, 1, DV, kWhole>(v + row * a.sv.t, key < len, a.dv, lane, vf[n]);
    lim[n] = from(key);
  }
  const float c = a.scale * kLog2e;
  f32x4 dk[MAPS][CB][NB], dv[VB][NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
#pragma unroll
    for (int m = 0; m < MAPS; ++m)
#pragma unroll
      for (int i = 0; i < CB; ++i) dk[m][i][n] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < VB; ++i) dv[i][n] = f32x4{0, 0, 0, 0};
  }

  // this workgroup's share of the heads' tiles
  const int n_all = G * n_tiles;
  const int first = static_cast<int>(static_cast<long>(n_all) * share / shares);
  const int last = static_cast<int>(static_cast<long>(n_all) * (share + 1) / shares);
  auto use = [&](int i, const E* Qs, const E* Gs, const float2* Ss) __attribute__((always_inline)) {
    const int row0 = t0 + i % n_tiles * QT;
    if (row0 + QT <= wfirst) return;
    const float lam = MAPS > 1 ? a.lam[hk * G + i / n_tiles] : 0.0f;
    Frag ga[QB][VS], qa[MAPS][QB][KS], qc[MAPS][QT / 32][CB];
    f32x4 dp[QB][NB], s[MAPS][QB][NB], pv[QB][NB];
    // an operand that was read a stage ahead; fp32 ones, twice as large, are read when they are used
    auto get = [](const Frag& ahead, auto&& now) {
      if constexpr (kAhead) return ahead;
      else return now();
    };
    auto read_q = [&](int m) {
      if constexpr (!kAhead) return;
#pragma unroll
      for (int qb = 0; qb < QB; ++qb)
#pragma unroll
        for (int e = 0; e < KS; ++e) qa[m][qb][e] = QTile::rows(Qs, 16 * qb, m * D + 32 * e, lane);
    };
    auto scores = [&](int m) {
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) {
#pragma unroll
        for (int n = 0; n < NB; ++n) s[m][qb][n] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < KS; ++e) {
          if (X::kSkip && 32 * e >= a.d) break;
#pragma unroll
          for (int n = 0; n < NB; ++n)
            s[m][qb][n] = X::mma(get(qa[m][qb][e], [&] { return QTile::rows(Qs, 16 * qb, m * D + 32 * e, lane); }),
                                 kf[n][m * KS + e], s[m][qb][n], a.d - 32 * e);
        }
      }
    };
    auto mask = [&]() {
      if (row0 < wall || row0 + QT > a.T) {  // some row does not see some key, or is none
#pragma unroll
        for (int qb = 0; qb < QB; ++qb)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int t = row0 + 16 * qb + 4 * grp + r;
              const bool out = t < lim[n] || t >= a.T;
#pragma unroll
              for (int m = 0; m < MAPS; ++m)
                if (out) s[m][qb][n][r] = -INFINITY;
            }
      }
    };
    auto read_qt = [&](int m) {
      if constexpr (!kAhead) return;
#pragma unroll
      for (int j = 0; j < QT / 32; ++j)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) qc[m][j][cb] = QTile::cols(Qs, 32 * j, m * D + 16 * cb, lane);
    };
    // p and ds of a map in place of its scores; pv collects p_1 - lam p_2
    auto weigh = [&](int m) {
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) {
        const f32x4* at = reinterpret_cast<const f32x4*>(&Ss[m * QT + 16 * qb + 4 * grp]);
        const f32x4 s01 = at[0], s23 = at[1], l4 = {s01[0], s01[2], s23[0], s23[2]}, d4 = {s01[1], s01[3], s23[1], s23[3]};
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float p = fast_exp2(fmaf(s[m][qb][n][r], c, -l4[r]));
            if (m == 1) p *= -lam;
            pv[qb][n][r] = m == 0 ? p : pv[qb][n][r] + p;
            s[m][qb][n][r] = p * (dp[qb][n][r] - d4[r]);
          }
      }
    };
    auto add_k = [&](int m) {
#pragma unroll
      for (int j = 0; j < QT / 32; ++j) {
        Frag ds[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) ds[n] = X::pack(s[m][2 * j][n], s[m][2 * j + 1][n]);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          if (X::kSkip && 16 * cb >= a.d) break;
#pragma unroll
          for (int n = 0; n < NB; ++n)
            dk[m][cb][n] = X::mma(get(qc[m][j][cb], [&] { return QTile::cols(Qs, 32 * j, m * D + 16 * cb, lane); }),
                                  ds[n], dk[m][cb][n]);
        }
      }
    };
    if constexpr (kAhead) {
#pragma unroll
      for (int qb = 0; qb < QB; ++qb)
#pragma unroll
        for (int e = 0; e < VS; ++e) ga[qb][e] = GTile::rows(Gs, 16 * qb, 32 * e, lane);
    }
    read_q(0);
    stage_border<E>();
    products_first();
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
#pragma unroll
      for (int n = 0; n < NB; ++n) dp[qb][n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < VS; ++e) {
        if (X::kSkip && 32 * e >= a.dv) break;
#pragma unroll
        for (int n = 0; n < NB; ++n)
          dp[qb][n] = X::mma(get(ga[qb][e], [&] { return GTile::rows(Gs, 16 * qb, 32 * e, lane); }), vf[n][e], dp[qb][n],
                             a.dv - 32 * e);
      }
    }
    stage_border<E>();
    if constexpr (MAPS > 1) read_q(1);
    else read_qt(0);
    stage_border<E>();
    scores(0);
    stage_border<E>();
    if constexpr (MAPS > 1) {
      read_qt(0);
      stage_border<E>();
      scores(1);
      products_done();
      mask();
      weigh(0);
      stage_border<E>();
      read_qt(1);
      stage_border<E>();
      products_first();
      add_k(0);
      products_done();
      weigh(1);
    } else {
      products_done();
      mask();
      weigh(0);
    }
    stage_border<E>();
    constexpr int VG = VB < 4 ? VB : 4;  // blocks of values of a stage
    Frag gc[2][QT / 32][VG];
    auto read_gt = [&](int v0) {
      if constexpr (!kAhead) return;
#pragma unroll
      for (int j = 0; j < QT / 32; ++j)
#pragma unroll
        for (int vb = 0; vb < VG; ++vb) gc[v0 / VG & 1][j][vb] = GTile::cols(Gs, 32 * j, 16 * (v0 + vb), lane);
    };
    read_gt(0);
    stage_border<E>();
    products_first();
    add_k(MAPS - 1);
    Frag pf[QT / 32][NB];
#pragma unroll
    for (int j = 0; j < QT / 32; ++j)
#pragma unroll
      for (int n = 0; n < NB; ++n) pf[j][n] = X::pack(pv[2 * j][n], pv[2 * j + 1][n]);
#pragma unroll
    for (int v0 = 0; v0 < VB; v0 += VG) {
      stage_border<E>();
      if (v0 + VG < VB) read_gt(v0 + VG);
      stage_border<E>();
#pragma unroll
      for (int j = 0; j < QT / 32; ++j)
#pragma unroll
        for (int vb = 0; vb < VG; ++vb) {
          if (X::kSkip && 16 * (v0 + vb) >= a.dv) break;
#pragma unroll
          for (int n = 0; n < NB; ++n)
            dv[v0 + vb][n] = X::mma(
                get(gc[v0 / VG & 1][j][vb], [&] { return GTile::cols(Gs, 32 * j, 16 * (v0 + vb), lane); }), pf[j][n],
                dv[v0 + vb][n]);
        }
    }
    products_done();
  };
  auto q_of = [&](int h) { return static_cast<const E*>(a.q) + b * a.sq.b + h * a.sq.h; };
  auto g_of = [&](int h) { return static_cast<const E*>(g.grad_o) + b * g.sdo.b + h * g.sdo.h; };
  auto stats_of = [&](int h, int m) { return stats + m * rows + (static_cast<long>(b) * a.H + h) * a.T; };
  // tiles in LDS as in the forward
  if constexpr (kDma) {
    const Dma<QT, MAPS, D, NW> qd(a.d, wave, lane);
    const Dma<QT, 1, DV, NW> gd(a.dv, wave, lane);
    static_assert(QT * 8 == 64 * 4, "a wave brings a map's statistics in one load");
    E *const Qt[] = {Q0, Q1, Q2}, *const Gt[] = {G0, G1, G2};
    float2* const St[] = {S0, S1, S2};
    walk_tiles<SLOTS, qd.COUNT + gd.COUNT + 1>(
        first, last,
        [&](int i, auto slot) __attribute__((always_inline)) {
          const int h = hk * G + i / n_tiles, row0 = t0 + i % n_tiles * QT;
          qd.load(q_of(h), a.sq.t, row0, a.T, Qt[slot], wave);
          gd.load(g_of(h), g.sdo.t, row0, a.T, Gt[slot], wave);
          // rows behind the last repeat it; use() masks them
          load_to_lds<4>(stats_of(h, wave % MAPS), 8 * min(row0 + lane / 2, a.T - 1) + 4 * (lane & 1), St[slot] + wave * QT);
        },
        [&](int i, auto slot) __attribute__((always_inline)) { use(i, Qt[slot], Gt[slot], St[slot]); });
  } else {
    Stage<E, QT, MAPS, D, THREADS, kWhole> qs(a.d, tid);
    Stage<E, QT, 1, DV, THREADS, kWhole> gs(a.dv, tid);
    float2 st;
    auto load = [&](int i) {
      const int h = hk * G + i / n_tiles, row0 = t0 + i % n_tiles * QT;
      qs.load(q_of(h), a.sq.t, row0, a.T, a.d);
      gs.load(g_of(h), g.sdo.t, row0, a.T, a.dv);
      if (tid < MAPS * QT) st = stats_of(h, tid / QT)[min(row0 + tid % QT, a.T - 1)];
    };
    auto store = [&](int i) {
      const int row0 = t0 + i % n_tiles * QT;
      qs.store(i & 1 ? Q1 : Q0, row0, a.T);
      gs.store(i & 1 ? G1 : G0, row0, a.T);
      if (tid < MAPS * QT) (i & 1 ? S1 : S0)[tid] = st;
    };
    if (first < last) {
      load(first);
      store(first);
      if (first + 1 < last) load(first + 1);
    }
    for (int i = first; i < last; ++i) {
      lds_barrier();
      if (i + 1 < last) {
        store(i + 1);
        if (i + 2 < last) load(i + 2);
      }
      use(i, i & 1 ? Q1 : Q0, i & 1 ? G1 : G0, i & 1 ? S1 : S0);
    }
  }

#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int key = w0 + 16 * n + col;
    if (key >= a.S) continue;
    const bool in = key < len;
    const f32x4 zero = {0, 0, 0, 0};
    if (shares > 1) {  // fp32 sums of the share, [share][b, hk, key][dk4 + dv4]
      const int d4 = (a.d + 3) & ~3, dv4 = (a.dv + 3) & ~3;
      float* to = part + (share * static_cast<long>(heads) * a.S + static_cast<long>(bh) * a.S + key) * (MAPS * d4 + dv4);
#pragma unroll
      for (int m = 0; m < MAPS; ++m)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          store4<float, true>(to + m * d4, 16 * cb + 4 * grp, d4, in ? dk[m][cb][n] : zero);
#pragma unroll
      for (int vb = 0; vb < VB; ++vb) store4<float, true>(to + MAPS * d4, 16 * vb + 4 * grp, dv4, in ? dv[vb][n] : zero);
      continue;
    }
    E* ok = static_cast<E*>(g.grad_k) + b * g.sdk.b + hk * g.sdk.h + key * g.sdk.t;
    E* ov = static_cast<E*>(g.grad_v) + b * g.sdv.b + hk * g.sdv.h + key * g.sdv.t;
#pragma unroll
    for (int m = 0; m < MAPS; ++m)
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        store4<E, kWhole>(ok + m * a.d, 16 * cb + 4 * grp, a.d, in ? dk[m][cb][n] * a.scale : zero);
#pragma unroll
    for (int vb = 0; vb < VB; ++vb) store4<E, kWhole>(ov, 16 * vb + 4 * grp, a.dv, in ? dv[vb][n] : zero);
  }
}

struct KvShape {
  static constexpr int NB = 1, NW = 4, TILE = 16 * NB * NW, STREAM = 32;
  static_assert(TILE == kBwdKeys, "keys of a workgroup");
};
template <typename E, int DK, int DV>
struct BwdShape {
  static constexpr int NB = sizeof(E) == 2 && DK + DV <= 256 ? 2 : 1;
  static constexpr int NW = 4, TILE = 16 * NB * NW, STREAM = 32;
};

template <typename E>
int bwd_rows(const AttnFwd& a) {
  return with_sizes(a, [](auto, auto dk, auto dv, auto) { return BwdShape<E, decltype(dk)::value, decltype(dv)::value>::TILE; });
}

template <typename E>
hipError_t launch_bwd_q(const AttnBwd& a, float* stats, float* lam_part, float* part, int shares, hipStream_t s) {
  return with_sizes(a.f, [&](auto m, auto dk, auto dv, auto whole) {
    constexpr int M = decltype(m)::value, DK = decltype(dk)::value, DV = decltype(dv)::value;
    constexpr bool W = decltype(whole)::value;
    typedef BwdShape<E, DK, DV> C;
    const int tiles = (a.f.T + C::TILE - 1) / C::TILE;
    hipLaunchKernelGGL((attention_bwd_q_kernel<E, M, DK, DV, W, C::NB, C::NW, C::STREAM>),
                       dim3(static_cast<unsigned>(tiles) * a.f.B * a.f.H, shares), dim3(64 * C::NW), 0, s, a,
                       reinterpret_cast<float2*>(stats), lam_part, part, tiles, shares);
    return hipGetLastError();
  });
}

template <typename E>
hipError_t launch_bwd_kv(const AttnBwd& a, const float* stats, float* part, int shares, hipStream_t s) {
  return with_sizes(a.f, [&](auto m, auto dk, auto dv, auto whole) {
    constexpr int M = decltype(m)::value, DK = decltype(dk)::value, DV = decltype(dv)::value;
    constexpr bool W = decltype(whole)::value;
    typedef KvShape C;
    const int tiles = (a.f.S + C::TILE - 1) / C::TILE;
    hipLaunchKernelGGL((attention_bwd_kv_kernel<E, M, DK, DV, W, C::NB, C::NW, C::STREAM>),
                       dim3(static_cast<unsigned>(tiles) * a.f.B * a.f.Hk * shares), dim3(64 * C::NW), 0, s, a,
                       reinterpret_cast<const float2*>(stats), part, shares);
    return hipGetLastError();
  });
}

}  // namespace attn
}  // namespace ret
