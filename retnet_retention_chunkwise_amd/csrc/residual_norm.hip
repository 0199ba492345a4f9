// The residual stream after a block and the normalised input of the next one,
// and the gradient of both.  Per row of D channels:
//   r = alpha x + scale f (held in the tensors' type),  n = (r - mu) rstd w + b
// (LayerNorm), or n = r rstd w + b with mu = 0 (RMSNorm); backward, with
// p = dn w, xh = (r - mu) rstd:
//   g = dr + rstd (p - mean(p) - xh mean(p xh)),  dx = alpha g,  df = scale g,
//   dw = sum dn xh,  db = sum dn,  dscale = sum g f   (mean(p) only for LayerNorm).
// A row is held in registers by LPR threads, 8 elements each (16 for the
// widest rows), in 16-byte pieces at any alignment (vec_io.h); every element is
// read and written once, so the call is HBM bound.  Row sums are fp32 (row_sum.h): first sum r (and p),
// then squares and products about the mean, so a mean far from zero costs no
// precision.  mu and rstd are found again in the backward: its rows are in
// registers anyway.  Measured: 16384 x 4096 bf16 backward with all parameter
// gradients 154 us (5.2 TB/s), 8191 x 1111 fp32 forward 28.4 us (5.1 TB/s).
#include "common.h"
#include "kernels.h"
#include "row_sum.h"
#include "vec_io.h"

// Fused multiply-adds only where they are written: which products the compiler
// joins would differ between the instances of a kernel, and so would their bits.
#pragma clang fp contract(off)

namespace ret {
namespace {

template <int VEC>
__device__ __forceinline__ void params(const float* p, int c, float otherwise, float (&x)[VEC]) {
  if (p != nullptr) {
    load_params<VEC>(p + c, x);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = otherwise;
  }
}

template <typename E>
__device__ __forceinline__ float as_held(float x) {
  if constexpr (sizeof(E) == 2)
    return bf16_to_f32(f32_to_bf16(x));
  else
    return x;
}

template <typename E, int VEC, int LPR, int EPT, int THREADS>
__global__ __launch_bounds__(THREADS) void residual_norm_fwd_kernel(ResidualNormFwd a) {
  constexpr int NI = EPT / VEC, G = THREADS / LPR;
  using IO = VecIO<E, VEC>;
  __shared__ RowExchange<THREADS> ex;
  int phase = 0;
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const long row = static_cast<long>(blockIdx.x) * G + g;
  const bool valid = row < a.rows;
  const long rr = valid ? row : a.rows - 1;  // past the end: the last row, not stored
  const E* xp = static_cast<const E*>(a.x) + rr * a.sx;
  const E* fp = static_cast<const E*>(a.f) + rr * a.sf;
  typename IO::Raw rx[NI], rf[NI];
  Piece pc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    pc[i] = Piece(VEC * (l + LPR * i), a.D, VEC);
    rx[i] = IO::load(xp + pc[i].at);
    rf[i] = IO::load(fp + pc[i].at);
  }
  float r[NI][VEC], s = 0.0f, q = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float x[VEC], f[VEC], sc[VEC];
    IO::unpack(rx[i], x);
    IO::unpack(rf[i], f);
    params<VEC>(a.scale, pc[i].at, 1.0f, sc);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      r[i][e] = as_held<E>(fmaf(a.alpha, x[e], sc[e] * f[e]));
      s += pc[i].own(e) ? r[i][e] : 0.0f;
      q = pc[i].own(e) ? fmaf(r[i][e], r[i][e], q) : q;
    }
    if (pc[i].in && valid) IO::store(static_cast<E*>(a.r) + rr * a.sr + pc[i].at, r[i]);
  }
  const float inv = 1.0f / static_cast<float>(a.D);
  row_sums<LPR>(s, q, ex, phase);
  const float mu = a.rms ? 0.0f : s * inv;
  if (!a.rms) {  // uniform
    float none = 0.0f;
    q = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) q = pc[i].own(e) ? fmaf(r[i][e] - mu, r[i][e] - mu, q) : q;
    row_sums<LPR>(q, none, ex, phase);
  }
  const float rstd = 1.0f / sqrtf(q * inv + a.eps);
  if (!valid) return;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = pc[i].at;
    if (!pc[i].in) continue;
    float w[VEC], b[VEC], n[VEC];
    params<VEC>(a.weight, c, 1.0f, w);
    params<VEC>(a.bias, c, 0.0f, b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) n[e] = fmaf((r[i][e] - mu) * rstd, w[e], b[e]);
    IO::store(static_cast<E*>(a.n) + rr * a.sn + c, n);
  }
}

// A workgroup walks rows, G at a time; the parameter sums stay in registers
// until the end, when its G row groups are added through LDS in a fixed order
// and written as partial sums [3][gridDim.x][D] (dw, db, dscale).
template <typename E, int VEC, int LPR, int EPT, int THREADS, bool kParam>
__global__ __launch_bounds__(THREADS) void residual_norm_bwd_kernel(ResidualNormBwd a, float* partial) {
  constexpr int NI = EPT / VEC, G = THREADS / LPR;
  using IO = VecIO<E, VEC>;
  __shared__ RowExchange<THREADS> ex;
  __shared__ float acc[kParam && G > 1 ? G : 1][kParam && G > 1 ? LPR * EPT : 1];
  int phase = 0;
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const float inv = 1.0f / static_cast<float>(a.D);
  const bool with_f = kParam && a.grad_scale != nullptr;
  float w[NI][VEC], sc[NI][VEC], dw[NI][VEC], db[NI][VEC], ds[NI][VEC];
  Piece pc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    pc[i] = Piece(VEC * (l + LPR * i), a.D, VEC);
    params<VEC>(a.weight, pc[i].at, 1.0f, w[i]);
    params<VEC>(a.scale, pc[i].at, 1.0f, sc[i]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = ds[i][e] = 0.0f;
  }
  typename IO::Raw rr[NI], rn[NI], rd[NI], rf[NI];
  auto load = [&](long row) __attribute__((always_inline)) {
    row = row < a.rows ? row : a.rows - 1;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int cc = pc[i].at;
      rr[i] = IO::load(static_cast<const E*>(a.r) + row * a.sr + cc);
      rn[i] = IO::load(static_cast<const E*>(a.grad_n) + row * a.sgn + cc);
      if (a.grad_r != nullptr) rd[i] = IO::load(static_cast<const E*>(a.grad_r) + row * a.sgr + cc);
      if (with_f) rf[i] = IO::load(static_cast<const E*>(a.f) + row * a.sf + cc);
    }
  };
  const long step = static_cast<long>(gridDim.x) * G;
  long first = static_cast<long>(blockIdx.x) * G;
  load(first + g);
  for (; first < a.rows; first += step) {  // uniform over the workgroup
    const long row = first + g;
    const bool valid = row < a.rows;
    float r[NI][VEC], p[NI][VEC], d[NI][VEC], f[NI][VEC], s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      IO::unpack(rr[i], r[i]);
      IO::unpack(rn[i], p[i]);
      if (a.grad_r != nullptr) {
        IO::unpack(rd[i], d[i]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[i][e] = 0.0f;
      }
      if (with_f) IO::unpack(rf[i], f[i]);
    }
    if (first + step < a.rows) load(row + step);
    float mu = 0.0f, mp = 0.0f;
    if (!a.rms) {  // uniform
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s0 += pc[i].own(e) ? r[i][e] : 0.0f;
          s1 = pc[i].own(e) ? fmaf(p[i][e], w[i][e], s1) : s1;
        }
      row_sums<LPR>(s0, s1, ex, phase);
      mu = s0 * inv;
      mp = s1 * inv;
    }
    float q = 0.0f, px = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        r[i][e] -= mu;
        q = pc[i].own(e) ? fmaf(r[i][e], r[i][e], q) : q;
        px = pc[i].own(e) ? fmaf(p[i][e] * w[i][e], r[i][e], px) : px;
      }
    row_sums<LPR>(q, px, ex, phase);
    const float rstd = 1.0f / sqrtf(q * inv + a.eps);
    const float mpx = px * inv * rstd;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float gx[VEC], gf[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = r[i][e] * rstd;
        const float gr = fmaf(rstd, fmaf(-xh, mpx, fmaf(p[i][e], w[i][e], -mp)), d[i][e]);
        gx[e] = a.alpha * gr;
        gf[e] = sc[i][e] * gr;
        if constexpr (kParam) {
          if (valid) {
            dw[i][e] = fmaf(p[i][e], xh, dw[i][e]);
            db[i][e] += p[i][e];
            if (with_f) ds[i][e] = fmaf(gr, f[i][e], ds[i][e]);
          }
        }
      }
      if (pc[i].in && valid) {
        const int c = pc[i].at;
        if (a.grad_x != nullptr) IO::store(static_cast<E*>(a.grad_x) + row * a.sgx + c, gx);
        if (a.grad_f != nullptr) IO::store(static_cast<E*>(a.grad_f) + row * a.sgf + c, gf);
      }
    }
  }
  if constexpr (kParam) {
    for (int k = 0; k < 3; ++k) {
      if ((k == 0 ? a.grad_weight : k == 1 ? a.grad_bias : a.grad_scale) == nullptr) continue;  // uniform
      float* to = partial + (static_cast<long>(k) * gridDim.x + blockIdx.x) * a.D;
      if constexpr (G > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (pc[i].in) acc[g][pc[i].at + e] = k == 0 ? dw[i][e] : k == 1 ? db[i][e] : ds[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += THREADS) {
          float s = acc[0][c];
#pragma unroll
          for (int j = 1; j < G; ++j) s += acc[j][c];
          to[c] = s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (pc[i].in)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              to[pc[i].at + e] = k == 0 ? dw[i][e] : k == 1 ? db[i][e] : ds[i][e];
      }
    }
  }
}

// Threads per row: the fewest that hold it at 8 elements each (16 beyond 8192
// elements), a power of two from 8 to 1024.
int threads_per_row(int D) {
  int n = 8;
  while (n < 1024 && n * 8 < D) n *= 2;
  return n;
}
constexpr int fwd_threads(int lpr) { return lpr > 256 ? lpr : 256; }
constexpr int bwd_threads(int lpr) { return lpr > 512 ? lpr : 512; }

template <typename E, int VEC, int LPR, int EPT>
struct Fwd {
  static hipError_t run(const ResidualNormFwd& a, hipStream_t s) {
    constexpr int THREADS = fwd_threads(LPR), G = THREADS / LPR;
    hipLaunchKernelGGL((residual_norm_fwd_kernel<E, VEC, LPR, EPT, THREADS>),
                       dim3(static_cast<unsigned>((a.rows + G - 1) / G)), dim3(THREADS), 0, s, a);
    return hipGetLastError();
  }
};
template <typename E, int VEC, int LPR, int EPT>
struct Bwd {
  static hipError_t run(const ResidualNormBwd& a, float* partial, int blocks, hipStream_t s) {
    constexpr int THREADS = bwd_threads(LPR);
    if (partial != nullptr)
      hipLaunchKernelGGL((residual_norm_bwd_kernel<E, VEC, LPR, EPT, THREADS, true>), dim3(blocks), dim3(THREADS), 0,
                         s, a, partial);
    else
      hipLaunchKernelGGL((residual_norm_bwd_kernel<E, VEC, LPR, EPT, THREADS, false>), dim3(blocks), dim3(THREADS), 0,
                         s, a, partial);
    return hipGetLastError();
  }
};

template <template <typename, int, int, int> class F, typename E, int VEC, typename... A>
hipError_t by_row(int D, A&&... a) {
  if constexpr (VEC == 1) {
    return F<E, VEC, 8, 8>::run(a...);  // rows of fewer than 8 elements
  } else {
    switch (threads_per_row(D)) {
      case 8: return F<E, VEC, 8, 8>::run(a...);
      case 16: return F<E, VEC, 16, 8>::run(a...);
      case 32: return F<E, VEC, 32, 8>::run(a...);
      case 64: return F<E, VEC, 64, 8>::run(a...);
      case 128: return F<E, VEC, 128, 8>::run(a...);
      case 256: return F<E, VEC, 256, 8>::run(a...);
      case 512: return F<E, VEC, 512, 8>::run(a...);
      default: return D <= 8192 ? F<E, VEC, 1024, 8>::run(a...) : F<E, VEC, 1024, 16>::run(a...);
    }
  }
}

}  // namespace

hipError_t launch_residual_norm_fwd(const ResidualNormFwd& a, hipStream_t s) {
  if (a.dt == 1) return a.D >= 8 ? by_row<Fwd, uint16_t, 8>(a.D, a, s) : by_row<Fwd, uint16_t, 1>(a.D, a, s);
  return a.D >= 4 ? by_row<Fwd, float, 4>(a.D, a, s) : by_row<Fwd, float, 1>(a.D, a, s);
}

// Two workgroups of 512 threads for each compute unit, as many as fit with
// their parameter sums in registers: more would only add partial sums.
int residual_norm_bwd_blocks(long rows, int D) {
  const int lpr = threads_per_row(D), threads = bwd_threads(lpr);
  const long most = (rows + threads / lpr - 1) / (threads / lpr);
  const long want = 256L * (1024 / threads);
  return static_cast<int>(want < most ? want : most);
}

hipError_t launch_residual_norm_bwd(const ResidualNormBwd& a, float* partial, hipStream_t s) {
  const int blocks = residual_norm_bwd_blocks(a.rows, a.D);
  hipError_t e;
  if (a.dt == 1)
    e = a.D >= 8 ? by_row<Bwd, uint16_t, 8>(a.D, a, partial, blocks, s) : by_row<Bwd, uint16_t, 1>(a.D, a, partial, blocks, s);
  else
    e = a.D >= 4 ? by_row<Bwd, float, 4>(a.D, a, partial, blocks, s) : by_row<Bwd, float, 1>(a.D, a, partial, blocks, s);
  if (e != hipSuccess || partial == nullptr) return e;
  return launch_column_sums(ColumnSums{partial, blocks, a.D, {a.grad_weight, a.grad_bias, a.grad_scale}}, s);
}

}  // namespace ret
