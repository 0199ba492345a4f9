// Per-head GroupNorm of a mixer's output followed by its gate, and the
// gradient of both.  For every (b, h, t), over the d_v values of the row:
//   xh = (y - mu) rstd,  n = xh w[h] + bias[h],  out = n z sigmoid(z)   (out = n without a gate)
// and, with s = sigmoid(z), dn = dout z s, p = dn w:
//   dz = dout n (s + z s (1 - s)),  dy = rstd (p - mean(p) - xh mean(p xh)),
//   dw = sum dn xh,  dbias = sum dn   (over b and t).
// Rows move in 16-byte pieces at any alignment, every element once (vec_io.h):
// LPR lanes hold a row in registers (8 elements each), so narrow heads share a
// wave.  Sums over a row
// are fp32: sum y (and p) first, then the squares and products about the
// mean.  HBM bound: 3 elements move per value forward, 5 backward.  Measured:
// B1 H8 T65536 dv512 bf16 forward 307 us (5.2 TB/s), B4 H8 T2048 dv512 bf16
// backward 67 us with the column sums (5.0 TB/s).
#include "common.h"
#include "kernels.h"
#include "row_sum.h"
#include "vec_io.h"

// Fused multiply-adds only where they are written: which products the compiler
// joins would differ between the instances of a kernel, and so would their bits.
#pragma clang fp contract(off)

namespace ret {
namespace {

constexpr int kThreads = 256;
constexpr int kEPT = 8;  // elements of a row per thread

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// The row of sequence tensor p at (b, h, t).
template <typename E>
__device__ __forceinline__ const E* row_of(const void* p, const Strides3& s, int b, int h, int t) {
  return static_cast<const E*>(p) + b * s.b + h * s.h + t * s.t;
}

template <typename E, int VEC, int LPR>
__global__ __launch_bounds__(kThreads) void gate_norm_fwd_kernel(GateNormFwd a, unsigned rows) {
  constexpr int NI = kEPT / VEC, G = kThreads / LPR, kRows = 2;
  using IO = VecIO<E, VEC>;
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const unsigned row0 = (blockIdx.x * G + g) * kRows;
  Piece pc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) pc[i] = Piece(VEC * (l + LPR * i), a.dv, VEC);
  typename IO::Raw ry[kRows][NI], rz[kRows][NI];
  int hh[kRows];
  E* op[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const unsigned row = min(row0 + r, rows - 1);  // past the end: the last row, not stored
    const int t = row % a.T, bh = row / a.T, h = bh % a.H, b = bh / a.H;
    hh[r] = h;
    const E* yp = row_of<E>(a.y, a.sy, b, h, t);
    const E* zp = row_of<E>(a.gate, a.sz, b, h, t);
    op[r] = const_cast<E*>(row_of<E>(a.out, a.so, b, h, t));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      ry[r][i] = IO::load(yp + pc[i].at);
      if (a.gate != nullptr) rz[r][i] = IO::load(zp + pc[i].at);
    }
  }
  const float inv = 1.0f / static_cast<float>(a.dv);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float y[NI][VEC], s = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      IO::unpack(ry[r][i], y[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += pc[i].own(e) ? y[i][e] : 0.0f;
    }
    const float mu = lanes_sum<LPR>(s) * inv;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        y[i][e] -= mu;
        q = pc[i].own(e) ? fmaf(y[i][e], y[i][e], q) : q;
      }
    const float rstd = 1.0f / sqrtf(lanes_sum<LPR>(q) * inv + a.eps);
    if (row0 + r >= rows) continue;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = pc[i].at;
      if (!pc[i].in) continue;
      float w[VEC], bi[VEC], z[VEC], o[VEC];
      if (a.weight != nullptr) load_params<VEC>(a.weight + static_cast<long>(hh[r]) * a.dv + c, w);
      if (a.bias != nullptr) load_params<VEC>(a.bias + static_cast<long>(hh[r]) * a.dv + c, bi);
      if (a.gate != nullptr) IO::unpack(rz[r][i], z);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float n = y[i][e] * rstd;
        if (a.weight != nullptr) n *= w[e];
        if (a.bias != nullptr) n += bi[e];
        o[e] = a.gate != nullptr ? n * (z[e] * sigmoid(z[e])) : n;
      }
      IO::store(op[r] + c, o);
    }
  }
}

// A workgroup walks rows of one head, slab blockIdx.x of gridDim.x; its dw and
// dbias sums stay in registers until the end, when the workgroup's row groups
// are added through LDS in a fixed order and written as partial sums
// [2][gridDim.x][H][dv] for the column sums.
template <typename E, int VEC, int LPR, bool kParam>
__global__ __launch_bounds__(kThreads) void gate_norm_bwd_kernel(GateNormBwd a, unsigned rows, float* partial) {
  constexpr int NI = kEPT / VEC, G = kThreads / LPR;
  using IO = VecIO<E, VEC>;
  __shared__ float acc[kParam ? G : 1][kParam ? LPR * kEPT : 1];
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const int h = blockIdx.y;
  const unsigned step = gridDim.x * G;
  const float inv = 1.0f / static_cast<float>(a.dv);
  float w[NI][VEC], bi[NI][VEC], dw[NI][VEC], db[NI][VEC];
  Piece pc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    pc[i] = Piece(VEC * (l + LPR * i), a.dv, VEC);
    const long k = static_cast<long>(h) * a.dv + pc[i].at;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = 1.0f;
      bi[i][e] = dw[i][e] = db[i][e] = 0.0f;
    }
    if (a.weight != nullptr) load_params<VEC>(a.weight + k, w[i]);
    if (a.bias != nullptr) load_params<VEC>(a.bias + k, bi[i]);
  }
  typename IO::Raw ry[NI], rz[NI], rd[NI];
  auto load = [&](unsigned row) __attribute__((always_inline)) {
    const unsigned rr = min(row, rows - 1);
    const int t = rr % a.T, b = rr / a.T;
    const E* yp = row_of<E>(a.y, a.sy, b, h, t);
    const E* zp = row_of<E>(a.gate, a.sz, b, h, t);
    const E* dp = row_of<E>(a.grad_out, a.sdo, b, h, t);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int cc = pc[i].at;
      ry[i] = IO::load(yp + cc);
      if (a.gate != nullptr) rz[i] = IO::load(zp + cc);
      rd[i] = IO::load(dp + cc);
    }
  };
  unsigned row = blockIdx.x * G + g;
  if (row < rows) load(row);
  for (; row < rows; row += step) {
    float y[NI][VEC], z[NI][VEC], d[NI][VEC];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      IO::unpack(ry[i], y[i]);
      if (a.gate != nullptr) IO::unpack(rz[i], z[i]);
      IO::unpack(rd[i], d[i]);
    }
    if (row + step < rows) load(row + step);
    // d: dout; sg: z sigmoid(z); kz: d silu / dz
    float sg[NI][VEC], kz[NI][VEC], s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (a.gate != nullptr) {
          const float s = sigmoid(z[i][e]);
          sg[i][e] = z[i][e] * s;
          kz[i][e] = d[i][e] * fmaf(sg[i][e], 1.0f - s, s);
          d[i][e] *= sg[i][e];  // dn
        }
        s0 += pc[i].own(e) ? y[i][e] : 0.0f;
        s1 = pc[i].own(e) ? fmaf(d[i][e], w[i][e], s1) : s1;
      }
    const float mu = lanes_sum<LPR>(s0) * inv, mp = lanes_sum<LPR>(s1) * inv;
    float q = 0.0f, px = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        y[i][e] -= mu;
        q = pc[i].own(e) ? fmaf(y[i][e], y[i][e], q) : q;
        px = pc[i].own(e) ? fmaf(d[i][e] * w[i][e], y[i][e], px) : px;
      }
    const float rstd = 1.0f / sqrtf(lanes_sum<LPR>(q) * inv + a.eps);
    const float mpx = lanes_sum<LPR>(px) * inv * rstd;
    const int t = row % a.T, b = row / a.T;
    E* gyp = const_cast<E*>(row_of<E>(a.grad_y, a.sdy, b, h, t));
    E* gzp = const_cast<E*>(row_of<E>(a.grad_gate, a.sdz, b, h, t));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float gy[VEC], gz[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = y[i][e] * rstd, dn = d[i][e];
        gy[e] = rstd * fmaf(-xh, mpx, fmaf(dn, w[i][e], -mp));
        if (a.gate != nullptr) gz[e] = kz[i][e] * fmaf(xh, w[i][e], bi[i][e]);
        if constexpr (kParam) {
          dw[i][e] = fmaf(dn, xh, dw[i][e]);
          db[i][e] += dn;
        }
      }
      if (pc[i].in) {
        IO::store(gyp + pc[i].at, gy);
        if (a.gate != nullptr) IO::store(gzp + pc[i].at, gz);
      }
    }
  }
  if constexpr (kParam) {
    for (int k = 0; k < 2; ++k) {
      if (k == 1) __syncthreads();
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (pc[i].in) acc[g][pc[i].at + e] = k == 0 ? dw[i][e] : db[i][e];  // shared elements have equal sums
      __syncthreads();
      float* to = partial + ((static_cast<long>(k) * gridDim.x + blockIdx.x) * a.H + h) * a.dv;
      for (int c = threadIdx.x; c < a.dv; c += kThreads) {
        float s = acc[0][c];
#pragma unroll
        for (int j = 1; j < G; ++j) s += acc[j][c];
        to[c] = s;
      }
    }
  }
}

int lanes_for(int dv) { return dv > 32 * kEPT ? 64 : dv > 16 * kEPT ? 32 : dv > 8 * kEPT ? 16 : 8; }

template <typename E, int VEC, int LPR>
hipError_t run_fwd(const GateNormFwd& a, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(static_cast<long>(a.B) * a.H * a.T);
  const unsigned per = kThreads / LPR * 2;
  hipLaunchKernelGGL((gate_norm_fwd_kernel<E, VEC, LPR>), dim3(rows / per + (rows % per != 0)), dim3(kThreads), 0, s, a,
                     rows);
  return hipGetLastError();
}
template <typename E, int VEC, int LPR>
hipError_t run_bwd(const GateNormBwd& a, float* partial, int slabs, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(static_cast<long>(a.B) * a.T);
  if (partial != nullptr)
    hipLaunchKernelGGL((gate_norm_bwd_kernel<E, VEC, LPR, true>), dim3(slabs, a.H), dim3(kThreads), 0, s, a, rows,
                       partial);
  else
    hipLaunchKernelGGL((gate_norm_bwd_kernel<E, VEC, LPR, false>), dim3(slabs, a.H), dim3(kThreads), 0, s, a, rows,
                       partial);
  return hipGetLastError();
}

// Rows of at most 4 pieces take 4 lanes.  Against 8 (110 heads of 4454 tokens,
// us, forward and backward): bf16 dv 8 24 + 39 / 35 + 66, dv 32 30 + 52 / 34 + 67;
// fp32 dv 16 37 + 60 / 36 + 63, but dv 32, two pieces to a lane, 51 + 96 / 39 + 79.
template <typename E, int VEC>
hipError_t fwd_by_lanes(const GateNormFwd& a, hipStream_t s) {
  if constexpr (VEC == 1) {
    return run_fwd<E, VEC, 8>(a, s);  // rows of fewer than 8 elements
  } else {
    switch (lanes_for(a.dv)) {
      case 64: return run_fwd<E, VEC, 64>(a, s);
      case 32: return run_fwd<E, VEC, 32>(a, s);
      case 16: return run_fwd<E, VEC, 16>(a, s);
      default: return a.dv > 4 * VEC ? run_fwd<E, VEC, 8>(a, s) : run_fwd<E, VEC, 4>(a, s);
    }
  }
}
template <typename E, int VEC>
hipError_t bwd_by_lanes(const GateNormBwd& a, float* partial, int slabs, hipStream_t s) {
  if constexpr (VEC == 1) {
    return run_bwd<E, VEC, 8>(a, partial, slabs, s);
  } else {
    switch (lanes_for(a.dv)) {
      case 64: return run_bwd<E, VEC, 64>(a, partial, slabs, s);
      case 32: return run_bwd<E, VEC, 32>(a, partial, slabs, s);
      case 16: return run_bwd<E, VEC, 16>(a, partial, slabs, s);
      default: return a.dv > 4 * VEC ? run_bwd<E, VEC, 8>(a, partial, slabs, s) : run_bwd<E, VEC, 4>(a, partial, slabs, s);
    }
  }
}

}  // namespace

hipError_t launch_gate_norm_fwd(const GateNormFwd& a, hipStream_t s) {
  if (a.dt == 1)
    return a.dv >= 8 ? fwd_by_lanes<uint16_t, 8>(a, s) : fwd_by_lanes<uint16_t, 1>(a, s);
  return a.dv >= 4 ? fwd_by_lanes<float, 4>(a, s) : fwd_by_lanes<float, 1>(a, s);
}

int gate_norm_bwd_slabs(int B, int H, int T, int dv) {
  const long groups = static_cast<long>(B) * T;  // rows of one head
  // rows in a workgroup at once (twice that with 4 lanes to a row: of short narrow heads half then get no row)
  const long per = kThreads / lanes_for(dv);
  const long most = (groups + per - 1) / per;
  const long want = (1024 + H - 1) / H;  // about four workgroups on each of 256 compute units
  return static_cast<int>(want < most ? want : most);
}

hipError_t launch_gate_norm_bwd(const GateNormBwd& a, float* partial, hipStream_t s) {
  const int slabs = gate_norm_bwd_slabs(a.B, a.H, a.T, a.dv);
  hipError_t e;
  if (a.dt == 1)
    e = a.dv >= 8 ? bwd_by_lanes<uint16_t, 8>(a, partial, slabs, s) : bwd_by_lanes<uint16_t, 1>(a, partial, slabs, s);
  else
    e = a.dv >= 4 ? bwd_by_lanes<float, 4>(a, partial, slabs, s) : bwd_by_lanes<float, 1>(a, partial, slabs, s);
  if (e != hipSuccess || partial == nullptr) return e;
  return launch_column_sums(
      ColumnSums{partial, slabs, static_cast<long>(a.H) * a.dv, {a.grad_weight, a.grad_bias, nullptr}}, s);
}

}  // namespace ret
