// Gated linear recurrence with token-dependent decays, forward, backward and
// single-token step.  Per batch b, head h and channel, with the head's decay
// exponent rate > 0:
//   a_t = sigmoid(f_t)^rate,  h_t = a_t h_(t-1) + u_t,  y_t = h_t,
//   u_t = x_t, or u_t = (1 - a_t) x_t (normalize).
// The recurrence is carried with c_t = 1 - a_t instead of a_t:
//   h_t = h_(t-1) - c_t h_(t-1) + x_t,   normalize: h_t = h_(t-1) + c_t (x_t - h_(t-1)),
// because a decay near 1 loses its distance to 1 when it is rounded (a memory
// of n tokens would see n times that error), while c_t has 24 good bits.
//
// A tile is CW channels by TT tokens.  Lanes run along channels (VEC per lane,
// one access of up to 16 bytes) and then along time, so a wave reads whole
// runs of CW channels; every thread walks S consecutive tokens of its VEC
// channels in registers.  Affine maps h -> A h + H compose associatively: each
// thread forms the map of its S tokens, one wave composes the maps of the
// NSEG segments in time order, and every thread replays its tokens from its
// incoming value.  x and f are read once and y is written once.
#include "common.h"
#include "kernels.h"
#include "vec_io.h"

// Fused multiply-adds only where they are written: which products the compiler
// joins would differ between the instances of a kernel, and so would their bits.
#pragma clang fp contract(off)

namespace ret {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kPerThread = 16;  // VEC * S

struct HeadRate {
  float r[kHeadsPerLaunch];
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// c = 1 - sigmoid(f)^rate in fp32 from log2 sigmoid(f) = -(max(-f,0) log2e + log2(1+t)),
// t = e^-|f|.  log2(1+t) takes back the rounding of 1+t, and 1 - 2^z goes
// through its Taylor series where 2^z is near 1, so c keeps its relative
// precision down to the smallest decays.  f = -inf gives c = 1 and f = +inf
// gives c = 0 exactly.  *t_out: t.
template <typename E>
__device__ __forceinline__ float decay_complement(float f, float rate, float* t_out) {
  const float af = fabsf(f);
  const float p = af * kLog2e;
  float t = __builtin_amdgcn_exp2f(-p);
  const float w = 1.0f + t;
  const float l = fmaf(t - (w - 1.0f), kLog2e, __builtin_amdgcn_logf(w));
  const float z2 = -rate * fmaf(fmaxf(-f, 0.0f), kLog2e, l);
  const float z = z2 * kLn2;
  // relative error below -0.25: 2^-25 / 0.22; above it the series ends at z^6/5040 < 2^-24
  float s = fmaf(z, 1.0f / 720.0f, 1.0f / 120.0f);
  s = fmaf(z, s, 1.0f / 24.0f);
  s = fmaf(z, s, 1.0f / 6.0f);
  s = fmaf(z, s, 0.5f);
  s = fmaf(z, s, 1.0f);
  const float e = 1.0f - __builtin_amdgcn_exp2f(z2);
  *t_out = t;
  return z > -0.25f ? -z * s : e;
}

// sigmoid(-f) from t = e^-|f|
__device__ __forceinline__ float sigmoid_neg(float f, float t) {
  return (f > 0.0f ? t : 1.0f) * __builtin_amdgcn_rcpf(1.0f + t);
}

struct ScanTile {
  int b, h, hl, c0, ct;
};

__device__ __forceinline__ ScanTile decode_tile(int tile, int nct, int nh, int h0, int cw) {
  ScanTile s;
  s.ct = tile % nct;
  const int hb = tile / nct;
  s.hl = hb % nh;
  s.b = hb / nh;
  s.h = h0 + s.hl;
  s.c0 = s.ct * cw;
  return s;
}

template <typename E, int VEC, int CW, bool kNorm>
__global__ __launch_bounds__(kThreads) void gated_scan_fwd_kernel(GatedScanFwd p, HeadRate rates, int h0, int nh,
                                                                  int nct) {
  constexpr int S = kPerThread / VEC, LC = CW / VEC, TG = 64 / LC, NSEG = kWaves * TG, TT = NSEG * S;
  using IO = VecIO<E, VEC>;
  __shared__ float segA[2][NSEG][CW];
  __shared__ float segH[2][NSEG][CW];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int lc = lane % LC, seg = w * TG + lane / LC;
  const ScanTile tl = decode_tile(blockIdx.x, nct, nh, h0, CW);
  const int c = tl.c0 + lc * VEC;
  const bool active = c < p.d;
  const int cc = active ? c : 0;
  const E* xp = static_cast<const E*>(p.x) + tl.b * p.sx.b + tl.h * p.sx.h + cc;
  const E* fp = static_cast<const E*>(p.f) + tl.b * p.sf.b + tl.h * p.sf.h + cc;
  E* yp = static_cast<E*>(p.y) + tl.b * p.sy.b + tl.h * p.sy.h + cc;
  const float rate = rates.r[tl.hl];
  // the composing wave: one channel per lane
  const int ch = tl.c0 + lane;
  const bool mine = w == 0 && lane < CW;
  const bool kept = mine && ch < p.d;
  const long row = (static_cast<long>(tl.b) * p.H + tl.h) * p.d + ch;
  float carry = kept && p.state_in != nullptr ? p.state_in[row] : 0.0f;
  const int nchunk = (p.T + TT - 1) / TT;

  typename IO::Raw rx[S], rf[S];
  auto load = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const long t = min(chunk * TT + seg * S + s, p.T - 1);  // a row past the end: the last one, masked below
      rx[s] = IO::load(xp + t * p.sx.t);
      rf[s] = IO::load(fp + t * p.sf.t);
    }
  };
  load(0);
  for (int chunk = 0; chunk < nchunk; ++chunk) {
    float x[S][VEC], cm[S][VEC];
    const int t0 = chunk * TT + seg * S;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float f[VEC], t;
      IO::unpack(rx[s], x[s]);
      IO::unpack(rf[s], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        cm[s][e] = t0 + s < p.T ? decay_complement<E>(f[e], rate, &t) : 0.0f;
        x[s][e] = t0 + s < p.T ? x[s][e] : 0.0f;
      }
    }
    if (chunk + 1 < nchunk) load(chunk + 1);
    const int q = chunk & 1;
    float A[VEC], H[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      A[e] = 1.0f;
      H[e] = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        A[e] = fmaf(-cm[s][e], A[e], A[e]);
        H[e] = kNorm ? fmaf(cm[s][e], x[s][e] - H[e], H[e]) : fmaf(-cm[s][e], H[e], H[e]) + x[s][e];
      }
      segA[q][seg][lc * VEC + e] = A[e];
      segH[q][seg][lc * VEC + e] = H[e];
    }
    __syncthreads();
    if (mine) {
      if (kept && p.checkpoints != nullptr)
        p.checkpoints[((static_cast<long>(tl.b) * p.H + tl.h) * nchunk + chunk) * p.d + ch] = carry;
#pragma unroll 8
      for (int i = 0; i < NSEG; ++i) {
        const float a = segA[q][i][lane], hh = segH[q][i][lane];
        segH[q][i][lane] = carry;
        carry = fmaf(a, carry, hh);
      }
    }
    __syncthreads();
    float hcur[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) hcur[e] = segH[q][seg][lc * VEC + e];
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        hcur[e] = kNorm ? fmaf(cm[s][e], x[s][e] - hcur[e], hcur[e]) : fmaf(-cm[s][e], hcur[e], hcur[e]) + x[s][e];
      if (active && p.y != nullptr && t0 + s < p.T) IO::store(yp + (t0 + s) * p.sy.t, hcur);
    }
  }
  if (kept && p.state_out != nullptr) p.state_out[row] = carry;
}

// Backward, walking the tiles of a channel run from the last token to the
// first.  g_t = dL/dh_t = dy_t + a_(t+1) g_(t+1); what crosses a token
// boundary is G_t = a_t g_t, so a token maps G -> a_t (dy_t + G).  h_(t-1)
// comes from replaying the tile forwards from its checkpoint:
//   dx_t = g_t (c_t g_t),  df_t = g_t (h_(t-1) [- x_t]) a_t rate sigmoid(-f_t).
template <typename E, int VEC, int CW, bool kNorm>
__global__ __launch_bounds__(kThreads) void gated_scan_bwd_kernel(GatedScanBwd p, HeadRate rates, int h0, int nh,
                                                                  int nct) {
  constexpr int S = kPerThread / VEC, LC = CW / VEC, TG = 64 / LC, NSEG = kWaves * TG, TT = NSEG * S;
  using IO = VecIO<E, VEC>;
  __shared__ float segA[2][NSEG][CW];
  __shared__ float segH[2][NSEG][CW];
  __shared__ float segG[2][NSEG][CW];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int lc = lane % LC, seg = w * TG + lane / LC;
  const ScanTile tl = decode_tile(blockIdx.x, nct, nh, h0, CW);
  const int c = tl.c0 + lc * VEC;
  const bool active = c < p.d;
  const int cc = active ? c : 0;
  const E* xp = static_cast<const E*>(p.x) + tl.b * p.sx.b + tl.h * p.sx.h + cc;
  const E* fp = static_cast<const E*>(p.f) + tl.b * p.sf.b + tl.h * p.sf.h + cc;
  const E* gyp = static_cast<const E*>(p.grad_y) + tl.b * p.sgy.b + tl.h * p.sgy.h + cc;
  E* gxp = static_cast<E*>(p.grad_x) + tl.b * p.sgx.b + tl.h * p.sgx.h + cc;
  E* gfp = static_cast<E*>(p.grad_f) + tl.b * p.sgf.b + tl.h * p.sgf.h + cc;
  const float rate = rates.r[tl.hl];
  const int ch = tl.c0 + lane;
  const bool kept = w < 2 && lane < CW && ch < p.d;  // wave 0 composes forwards, wave 1 backwards
  const long bh = static_cast<long>(tl.b) * p.H + tl.h;
  float carry = w == 1 && kept && p.grad_state_out != nullptr ? p.grad_state_out[bh * p.d + ch] : 0.0f;
  const int nchunk = (p.T + TT - 1) / TT;

  typename IO::Raw rx[S], rf[S], rg[S];
  auto load = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const long t = min(chunk * TT + seg * S + s, p.T - 1);
      rx[s] = IO::load(xp + t * p.sx.t);
      rf[s] = IO::load(fp + t * p.sf.t);
      rg[s] = IO::load(gyp + t * p.sgy.t);
    }
  };
  load(nchunk - 1);
  for (int chunk = nchunk - 1; chunk >= 0; --chunk) {
    float x[S][VEC], cm[S][VEC], kf[S][VEC], dy[S][VEC];
    const int t0 = chunk * TT + seg * S;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float f[VEC];
      IO::unpack(rx[s], x[s]);
      IO::unpack(rf[s], f);
      IO::unpack(rg[s], dy[s]);
      const bool in = t0 + s < p.T;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float t;
        const float m = decay_complement<E>(f[e], rate, &t);
        cm[s][e] = in ? m : 0.0f;
        kf[s][e] = rate * (1.0f - m) * sigmoid_neg(f[e], t);
        x[s][e] = in ? x[s][e] : 0.0f;
        dy[s][e] = in ? dy[s][e] : 0.0f;
      }
    }
    const float ckpt = w == 0 && kept ? p.checkpoints[(bh * nchunk + chunk) * p.d + ch] : 0.0f;
    if (chunk > 0) load(chunk - 1);
    const int q = chunk & 1;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float A = 1.0f, H = 0.0f, G = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        A = fmaf(-cm[s][e], A, A);
        H = kNorm ? fmaf(cm[s][e], x[s][e] - H, H) : fmaf(-cm[s][e], H, H) + x[s][e];
      }
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const float g = dy[s][e] + G;
        G = fmaf(-cm[s][e], g, g);
      }
      segA[q][seg][lc * VEC + e] = A;
      segH[q][seg][lc * VEC + e] = H;
      segG[q][seg][lc * VEC + e] = G;
    }
    __syncthreads();
    if (w == 0 && lane < CW) {
      float cur = ckpt;
#pragma unroll 8
      for (int i = 0; i < NSEG; ++i) {
        const float a = segA[q][i][lane], hh = segH[q][i][lane];
        segH[q][i][lane] = cur;
        cur = fmaf(a, cur, hh);
      }
    } else if (w == 1 && lane < CW) {
#pragma unroll 8
      for (int i = NSEG - 1; i >= 0; --i) {
        const float a = segA[q][i][lane], gg = segG[q][i][lane];
        segG[q][i][lane] = carry;
        carry = fmaf(a, carry, gg);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float hp = segH[q][seg][lc * VEC + e], G = segG[q][seg][lc * VEC + e];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float xs = x[s][e];
        x[s][e] = kNorm ? hp - xs : hp;  // dh_t / da_t
        hp = kNorm ? fmaf(cm[s][e], xs - hp, hp) : fmaf(-cm[s][e], hp, hp) + xs;
      }
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const float g = dy[s][e] + G;
        G = fmaf(-cm[s][e], g, g);
        dy[s][e] = kNorm ? g * cm[s][e] : g;
        x[s][e] = g * x[s][e] * kf[s][e];
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (active && t0 + s < p.T) {
        IO::store(gxp + (t0 + s) * p.sgx.t, dy[s]);
        IO::store(gfp + (t0 + s) * p.sgf.t, x[s]);
      }
  }
  if (w == 1 && kept && p.grad_state_in != nullptr) p.grad_state_in[bh * p.d + ch] = carry;
}

// One token: state <- a state + u, y = state; one thread per VEC channels.
template <typename E, int VEC, bool kNorm>
__global__ __launch_bounds__(256) void gated_scan_step_kernel(GatedScanFwd p, HeadRate rates, int h0, int nh, long n) {
  using IO = VecIO<E, VEC>;
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const uint32_t per = p.d / VEC, ii = static_cast<uint32_t>(i);  // i < 2^31
  const int c = static_cast<int>(ii % per) * VEC;
  const int bh = static_cast<int>(ii / per);
  const int hl = bh % nh, b = bh / nh, h = h0 + hl;
  float x[VEC], f[VEC], st[VEC];
  IO::unpack(IO::load(static_cast<const E*>(p.x) + b * p.sx.b + h * p.sx.h + c), x);
  IO::unpack(IO::load(static_cast<const E*>(p.f) + b * p.sf.b + h * p.sf.h + c), f);
  const long row = (static_cast<long>(b) * p.H + h) * p.d + c;
  if (p.state_in != nullptr) {
    load_params<VEC>(p.state_in + row, st);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) st[e] = 0.0f;
  }
  if (p.checkpoints != nullptr)  // T = 1: one tile, which starts from the incoming state
#pragma unroll
    for (int e = 0; e < VEC; ++e) p.checkpoints[row + e] = st[e];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float t;
    const float m = decay_complement<E>(f[e], rates.r[hl], &t);
    st[e] = kNorm ? fmaf(m, x[e] - st[e], st[e]) : fmaf(-m, st[e], st[e]) + x[e];
  }
  if (p.state_out != nullptr) VecIO<float, VEC>::store(p.state_out + row, st);
  if (p.y != nullptr) IO::store(static_cast<E*>(p.y) + b * p.sy.b + h * p.sy.h + c, st);
}

HeadRate head_rates(const HeadGroup& g) {
  HeadRate r;
  for (int i = 0; i < kHeadsPerLaunch; ++i) r.r[i] = i < g.nh ? g.gamma[i] : 1.0f;
  return r;
}

template <typename E, int VEC, int CW, bool kNorm>
hipError_t run_fwd(const GatedScanFwd& p, const HeadGroup& g, hipStream_t s) {
  const int nct = (p.d + CW - 1) / CW;
  hipLaunchKernelGGL((gated_scan_fwd_kernel<E, VEC, CW, kNorm>), dim3(p.B * g.nh * nct), dim3(kThreads), 0, s, p,
                     head_rates(g), g.h0, g.nh, nct);
  return hipGetLastError();
}

template <typename E, int VEC, bool kNorm>
hipError_t run_step(const GatedScanFwd& p, const HeadGroup& g, hipStream_t s) {
  const long n = static_cast<long>(p.B) * g.nh * (p.d / VEC);
  hipLaunchKernelGGL((gated_scan_step_kernel<E, VEC, kNorm>), dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256),
                     0, s, p, head_rates(g), g.h0, g.nh, n);
  return hipGetLastError();
}

template <typename E, int VEC, int CW, bool kNorm>
hipError_t run_bwd(const GatedScanBwd& p, const HeadGroup& g, hipStream_t s) {
  const int nct = (p.d + CW - 1) / CW;
  hipLaunchKernelGGL((gated_scan_bwd_kernel<E, VEC, CW, kNorm>), dim3(p.B * g.nh * nct), dim3(kThreads), 0, s, p,
                     head_rates(g), g.h0, g.nh, nct);
  return hipGetLastError();
}

// Tile width for a row of d channels: 64, or the next power of two for
// narrow rows so that lanes are not left idle.
int tile_width(int d) { return d > 32 ? 64 : d > 16 ? 32 : 16; }

template <template <typename, int, int, bool> class F, typename E, int VEC, typename... A>
hipError_t by_width(int cw, bool norm, A&&... a) {
  if (cw == 64) return norm ? F<E, VEC, 64, true>::run(a...) : F<E, VEC, 64, false>::run(a...);
  if (cw == 32) return norm ? F<E, VEC, 32, true>::run(a...) : F<E, VEC, 32, false>::run(a...);
  return norm ? F<E, VEC, 16, true>::run(a...) : F<E, VEC, 16, false>::run(a...);
}
template <template <typename, int, int, bool> class F, typename E, typename... A>
hipError_t by_vec(int vec, int cw, bool norm, A&&... a) {
  switch (vec) {
    case 4: return by_width<F, E, 4>(cw, norm, a...);
    case 2: return by_width<F, E, 2>(cw, norm, a...);
    default: return by_width<F, E, 1>(cw, norm, a...);
  }
}

template <typename E, int VEC, int CW, bool kNorm>
struct Fwd {
  static hipError_t run(const GatedScanFwd& p, const HeadGroup& g, hipStream_t s) {
    return run_fwd<E, VEC, CW, kNorm>(p, g, s);
  }
};
template <typename E, int VEC, int CW, bool kNorm>
struct Bwd {
  static hipError_t run(const GatedScanBwd& p, const HeadGroup& g, hipStream_t s) {
    return run_bwd<E, VEC, CW, kNorm>(p, g, s);
  }
};

template <typename E>
hipError_t step_by_vec(int vec, const GatedScanFwd& p, const HeadGroup& g, hipStream_t s) {
  switch (vec) {
    case 4: return p.normalize ? run_step<E, 4, true>(p, g, s) : run_step<E, 4, false>(p, g, s);
    case 2: return p.normalize ? run_step<E, 2, true>(p, g, s) : run_step<E, 2, false>(p, g, s);
    default: return p.normalize ? run_step<E, 1, true>(p, g, s) : run_step<E, 1, false>(p, g, s);
  }
}

}  // namespace

int gated_scan_block(int d) { return kWaves * (kPerThread * 64 / tile_width(d)); }

hipError_t launch_gated_scan_fwd(const GatedScanFwd& p, const HeadGroup& g, hipStream_t s) {
  const int es = p.dt == 1 ? 2 : 4;
  const int vec = widest_access(p.d, 4, es, {p.x, p.f, p.y}, {p.sx, p.sf, p.sy});
  if (p.T == 1) {
    const int sv = widest_access(p.d, vec, 4, {p.state_in, p.state_out}, {});
    return p.dt == 1 ? step_by_vec<uint16_t>(sv, p, g, s) : step_by_vec<float>(sv, p, g, s);
  }
  const int cw = tile_width(p.d);
  return p.dt == 1 ? by_vec<Fwd, uint16_t>(vec, cw, p.normalize, p, g, s)
                   : by_vec<Fwd, float>(vec, cw, p.normalize, p, g, s);
}

hipError_t launch_gated_scan_bwd(const GatedScanBwd& p, const HeadGroup& g, hipStream_t s) {
  const int es = p.dt == 1 ? 2 : 4;
  const int vec = widest_access(p.d, 4, es, {p.x, p.f, p.grad_y, p.grad_x, p.grad_f}, {p.sx, p.sf, p.sgy, p.sgx, p.sgf});
  const int cw = tile_width(p.d);
  return p.dt == 1 ? by_vec<Bwd, uint16_t>(vec, cw, p.normalize, p, g, s)
                   : by_vec<Bwd, float>(vec, cw, p.normalize, p, g, s);
}

}  // namespace ret
