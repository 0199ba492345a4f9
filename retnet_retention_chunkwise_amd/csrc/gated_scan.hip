// Gated linear recurrence with token-dependent decays, forward, backward and
// single-token step.  Per batch b, head h and channel, with the head's decay
// exponent rate > 0:
//   a_t = sigmoid(f_t)^rate,  h_t = a_t h_(t-1) + u_t,  y_t = h_t,
//   u_t = x_t, or u_t = (1 - a_t) x_t (normalize).
// Where a_t >= 1/2 the recurrence is carried with c_t = 1 - a_t instead of a_t:
//   h_t = h_(t-1) - c_t h_(t-1) + x_t,   normalize: h_t = h_(t-1) + c_t (x_t - h_(t-1)),
// because a decay near 1 loses its distance to 1 when it is rounded (a memory
// of n tokens would see n times that error), while c_t has 24 good bits.  Below
// 1/2 it is the other way round, c_t would lose a_t, and
//   h_t = a_t h_(t-1) + x_t,   normalize: h_t = x_t + a_t (h_(t-1) - x_t),
// so that what is forgotten leaves no rounding behind (a_t = 0: h_t = u_t).  A
// decay is held in one number m_t that says which it is: c_t, or -a_t.  Choosing
// by its sign costs where the vector unit is what bounds: B1 H8 T32768 d512
// bf16, forward and backward, 520 us in place of 496 (two versions of every
// product and a branch by the wave's signs: 529).
//
// A tile is CW channels by TT tokens.  Lanes run along channels (VEC per lane,
// one access of up to 16 bytes) and then along time, so a wave reads whole
// runs of CW channels; every thread walks S consecutive tokens of its VEC
// channels in registers.  Affine maps h -> A h + H compose associatively: each
// thread forms the map of its S tokens, the maps are composed in time order
// (within a wave, then over the waves), and every thread replays its tokens
// from its incoming value.  x and f are read once and y is written once.
// Measured, bf16:
// B4 H8 T2048 d512 forward 40 us (5.0 TB/s), B2 H16 T8192 d512 forward and
// backward 432 to 445 us (4.9 TB/s), B1 H8 T65536 d512 forward 334 to 340 us with
// the workspace's fill (4.8 TB/s): the means of passes one after the other;
// single launches vary more, by up to a fifth.
#include "common.h"
#include "gfx950.h"
#include "kernels.h"
#include "vec_io.h"

// Fused multiply-adds only where they are written: which products the compiler
// joins would differ between the instances of a kernel, and so would their bits.
#pragma clang fp contract(off)

namespace ret {
namespace {

constexpr int kPerThread = 16;   // VEC * S of most kernels
constexpr int kBlockElems = 128;  // a checkpoint's block: as many elements per lane (8 waves of 16)
// Tiles of a channel run are chained over workgroups where the runs are fewer
// than kWalkTiles and have kChainSteps blocks of tokens or more; else one
// workgroup walks each run.  Measured in us, walking / chaining, d 64, bf16
// forward (and backward), runs x tokens:
//     32 x 512   13 / 17 (17 / 20)      32 x 1024    16 / 17 (24 / 21)
//     32 x 4096  51 / 25 (85 / 32)     128 x 4096    55 / 54 (92 / 88)
//    192 x 4096  63 / 74 (107 / 130)   256 x 16384  284 / 314 (456 / 639)
//    384 x 4096 124 / 129 (194 / 241)  512 x 4096   145 / 171 (233 / 322)
// and in fp32 128 x 4096 83 / 77 (137 / 117), 256 x 4096 139 / 147 (202 / 230),
// 384 x 4096 214 / 218 (329 / 342).
constexpr int kWalkTiles = 160, kChainSteps = 8;
constexpr int kTableTiles = 4;  // tiles of a workgroup from which on its gate table pays
// A workgroup that walks a run uses a table, and 16 waves, where the run is
// longer than so many blocks of tokens.  With / without, us, 1280 runs of d 64:
//   T 128   29 / 17 (backward 41 / 31)    T 256   32 / 30 (46 / 53)    T 512   51 / 53 (78 / 105)
constexpr int kTableStepsFwd = 2, kTableStepsBwd = 1;

typedef unsigned long long u64;

struct HeadRate {
  float r[kHeadsPerLaunch];
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994531;

// a = sigmoid(f)^rate in fp32, as held (*a_out: as it is), from
// z2 = rate log2 sigmoid(f) = -rate (max(-f,0) log2e + log2(1+t)), t = e^-|f|
// (*t_out).  log2(1+t) takes back the rounding of 1+t, and c = 1 - 2^z2 goes
// through its Taylor series where 2^z2 is near 1, so c keeps its relative
// precision down to the smallest decays.  f = -inf gives a = 0 and f = +inf
// gives c = 0 exactly.
__device__ __forceinline__ float held_decay(float f, float rate, float* t_out, float* a_out) {
  const float p = fabsf(f) * kLog2e;
  const float t = __builtin_amdgcn_exp2f(-p);
  const float w = 1.0f + t;
  const float l = fmaf(t - (w - 1.0f), kLog2e, __builtin_amdgcn_logf(w));
  const float z2 = -rate * fmaf(__builtin_amdgcn_fmed3f(-f, 0.0f, __builtin_inff()), kLog2e, l);
  // relative error below -0.36: 2^-25 / 0.22; above it the series ends at (z2 ln2)^6/5040 < 2^-24
  constexpr double k2 = kLn2 * kLn2 / 2, k3 = k2 * kLn2 / 3, k4 = k3 * kLn2 / 4, k5 = k4 * kLn2 / 5, k6 = k5 * kLn2 / 6;
  float s = fmaf(z2, static_cast<float>(k6), static_cast<float>(k5));
  s = fmaf(z2, s, static_cast<float>(k4));
  s = fmaf(z2, s, static_cast<float>(k3));
  s = fmaf(z2, s, static_cast<float>(k2));
  s = fmaf(z2, s, static_cast<float>(kLn2));
  const float a = __builtin_amdgcn_exp2f(z2);
  *t_out = t;
  *a_out = a;
  // fabs: c is never -0 and never below 0, which a rounding of l could else make it
  return z2 > -0.36f ? fabsf(z2 * s) : a < 0.5f ? -a : 1.0f - a;
}

// Whether a held decay is -a (-0 for a = 0) and not c >= 0.
__device__ __forceinline__ bool holds_a(float m) { return __float_as_int(m) < 0; }
// a h
__device__ __forceinline__ float decayed(float m, float h) { return fmaf(-m, h, holds_a(m) ? 0.0f : h); }
// (1 - a) h
__device__ __forceinline__ float complement(float m, float h) { return fmaf(m, h, holds_a(m) ? h : 0.0f); }
// a h + u
template <bool kNorm>
__device__ __forceinline__ float decay_step(float m, float x, float h) {
  return kNorm ? fmaf(m, x - h, holds_a(m) ? x : h) : decayed(m, h) + x;
}

// sigmoid(-f) from t = e^-|f|
__device__ __forceinline__ float sigmoid_neg(float f, float t) {
  return (f > 0.0f ? t : 1.0f) * __builtin_amdgcn_rcpf(1.0f + t);
}

// ---- Gate table ----
//
// bf16 gates take few values: 31 * 128 magnitudes from 2^-24 to 128 in two
// signs.  A workgroup that works on many tokens of one head evaluates the gate
// once for each of them into LDS and then looks it up, about 5 vector
// instructions and an LDS read per element in place of about 35 (three of them
// at a quarter of the rate), which bounded the kernel.  The entry of a value v
// is at rotate_left(bits(v), 1), so that both signs of a magnitude lie side by
// side.  Magnitudes below 2^-24, of either sign, take the entry of +2^-24: f is
// off by less than 2^-23 there, c by 1.45 x 2^-24 of itself, a by rate 2^-24.
// A wave that meets 128 or more, an infinity or a NaN evaluates its tokens
// directly.
constexpr int kGateLow = 103 << 7, kGateHigh = 134 << 7;  // bf16 bits of 2^-24 and of 128
constexpr int kGateN = 2 * (kGateHigh - kGateLow);
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Table index of two gates; top collects the largest index before clamping
// (kGateN or more: a gate outside the table).
__device__ __forceinline__ u16x2 gate_index(u16x2 bits, u16x2& top) {
  const u16x2 one = 1, fifteen = 15, low = 2 * kGateLow, most = kGateN - 1;
  const u16x2 r = __builtin_elementwise_sub_sat(static_cast<u16x2>((bits << one) | (bits >> fifteen)), low);
  top = __builtin_elementwise_max(top, r);
  return __builtin_elementwise_min(r, most);
}

__device__ __forceinline__ float gate_of_index(int i) {
  return bf16_to_f32(static_cast<uint16_t>((kGateLow + (i >> 1)) | ((i & 1) << 15)));
}

// One gate: a as held and, for the backward, k = rate a sigmoid(-f).
__device__ __forceinline__ void gate_value(float f, float rate, float* out) {
  float t, a;
  *out = held_decay(f, rate, &t, &a);
}
__device__ __forceinline__ void gate_value(float f, float rate, float2* out) {
  float t, a;
  const float m = held_decay(f, rate, &t, &a);
  *out = make_float2(m, rate * a * sigmoid_neg(f, t));
}

template <typename Entry>
__device__ __forceinline__ void build_gate_table(Entry* table, float rate, int threads) {
  for (int i = threadIdx.x; i < kGateN; i += threads) gate_value(gate_of_index(i), rate, &table[i]);
}

// The gates of S rows of VEC elements.
template <typename E, typename Entry, int VEC, int S>
struct Gates {
  using IO = VecIO<E, VEC>;
  __device__ __forceinline__ static void direct(const typename IO::Raw (&rf)[S], float rate, Entry (&out)[S][VEC]) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float f[VEC];
      IO::unpack(rf[s], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) gate_value(f[e], rate, &out[s][e]);
    }
  }
  // by table (bf16 only) or directly
  template <bool kTable>
  __device__ __forceinline__ static void get(const typename IO::Raw (&rf)[S], const Entry* table, float rate,
                                             Entry (&out)[S][VEC]) {
    if constexpr (!kTable) {
      direct(rf, rate, out);
    } else {
      static_assert(sizeof(E) == 2, "gate tables are of bf16 values");
      u16x2 top = 0;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if constexpr (VEC == 1) {
          u16x2 two;
          two[0] = two[1] = rf[s];
          out[s][0] = table[gate_index(two, top)[0]];
        } else if constexpr (VEC == 2) {
          const u16x2 i = gate_index(__builtin_bit_cast(u16x2, rf[s]), top);
          out[s][0] = table[i[0]];
          out[s][1] = table[i[1]];
        } else {
#pragma unroll
          for (int v = 0; v < VEC / 2; ++v) {
            const u16x2 i = gate_index(__builtin_bit_cast(u16x2, static_cast<unsigned>(rf[s][v])), top);
            out[s][2 * v] = table[i[0]];
            out[s][2 * v + 1] = table[i[1]];
          }
        }
      }
      if (__any(top[0] >= kGateN || top[1] >= kGateN)) direct(rf, rate, out);
    }
  }
};

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

// ---- Chaining tiles that run in different workgroups ----
//
// With few channels and many tokens the tiles of one channel run must work at
// the same time, each on its own tokens, and still hand their state on.  The
// workgroups of a head take tickets, which go through the head's tiles of step
// 0 of the walk (the first tokens, or the last ones backwards), then step 1,
// ...  A workgroup publishes its tile's map (A, H), takes the value that enters
// its group of kGroup steps and folds the maps of the group's earlier steps
// into it; the last step of a group publishes the value that enters the next
// group.  The order of all additions is fixed by the sizes, so results do not
// depend on timing.
//
// Every wait ends: a workgroup works on its tickets in order, waits only for
// words of lower tickets and publishes its tile's map before it waits, so the
// lowest ticket that is not yet done is never held up.  A wait of more than
// kSpinLimit polls (two calls on one workspace at the same time, which the
// interface forbids) gives NaN instead of hanging.  Published words carry
// their own "ready": the workspace is filled with ones before the launch and
// no published NaN has that pattern.
//
// A word takes microseconds to reach another workgroup while the memory is
// busy, so the tiles are large and several workgroups share a compute unit.
// (Measured slower: waves that fold all maps of a channel run and publish every
// tile's entering value, with twice the hops; replaying a tile one later.)
constexpr int kGroup = 8;
constexpr int kSpinLimit = 1 << 20;
constexpr int kCounterWords = 16;  // a counter has half a cache line to itself

struct Chain {
  unsigned* counters;  // [heads of the launch][kCounterWords]: the heads' tickets
  u64* maps;           // [steps][tiles][CW]: A in the low word, H in the high word
  unsigned* enter;     // [groups][tiles][CW]: the value that enters a group
  int steps, tiles;
};

__device__ __forceinline__ unsigned quiet(float x) { return x != x ? 0x7fc00000u : __float_as_uint(x); }

template <typename W>
__device__ __forceinline__ W wait_word(const W* p, W seen, W otherwise) {
  for (int n = 0; seen == static_cast<W>(~static_cast<W>(0)); ++n) {
    if (n == kSpinLimit) return otherwise;
    __builtin_amdgcn_s_sleep(1);
    seen = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  return seen;
}

// A word of LDS that the whole wave reads, as a scalar.
__device__ __forceinline__ unsigned uniform(unsigned x) { return __builtin_amdgcn_readfirstlane(x); }

// The next number of a counter (counters start one below 0).
__device__ __forceinline__ unsigned take(unsigned* counter) {
  return __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
}

// Hands a tile's map on: the lane's channel of the tile at step j.  Only step 0
// takes the value that enters the run (first), and publishes the constant map
// of what leaves it: the call's final state may lie over its incoming one, and
// the tile that writes it has waited for words that came from this read.
template <int CW>
__device__ __forceinline__ void publish_map(const Chain& c, int j, int tile, int lane, float A, float H, float first) {
  if (j == 0) {
    H = fmaf(A, first, H);
    A = 0.0f;
  }
  if (j % kGroup == kGroup - 1 || j == c.steps - 1) return;  // nobody folds it
  const long per = static_cast<long>(c.tiles) * CW;
  __hip_atomic_store(c.maps + j * per + static_cast<long>(tile) * CW + lane, static_cast<u64>(quiet(H)) << 32 | quiet(A),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The value that enters the tile at step j, for the lane's channel: begin()
// requests the published words, end() waits for them and folds them.
template <int CW>
struct Entering {
  u64 m[kGroup - 1];
  unsigned e;
  __device__ __forceinline__ void begin(const Chain& c, int j, int tile, int lane) {
    const long per = static_cast<long>(c.tiles) * CW, at = static_cast<long>(tile) * CW + lane;
    const int k = j % kGroup, g = j / kGroup;
    if (g > 0) e = __hip_atomic_load(c.enter + g * per + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const u64* maps = c.maps + static_cast<long>(g) * kGroup * per + at;
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
      if (i < k) m[i] = __hip_atomic_load(maps + i * per, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // (A, H): the tile's map; first: the value that enters step 0, finite at later steps (a constant map follows)
  __device__ __forceinline__ float end(const Chain& c, int j, int tile, int lane, float A, float H, float first) const {
    const long per = static_cast<long>(c.tiles) * CW, at = static_cast<long>(tile) * CW + lane;
    const int k = j % kGroup, g = j / kGroup;
    const u64* maps = c.maps + static_cast<long>(g) * kGroup * per + at;
    float v = g > 0 ? __uint_as_float(wait_word(c.enter + g * per + at, e, 0x7fc00000u)) : first;
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
      if (i < k) {
        const u64 r = wait_word(maps + i * per, m[i], static_cast<u64>(0x7fc000007fc00000ull));
        v = fmaf(__uint_as_float(static_cast<unsigned>(r)), v, __uint_as_float(static_cast<unsigned>(r >> 32)));
      }
    if (k == kGroup - 1 && j != c.steps - 1)
      __hip_atomic_store(c.enter + (g + 1) * per + at, quiet(fmaf(A, v, H)), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    return v;
  }
};

// A head's queue of tiles: ticket -> step and tile (b, column tile).
struct Queue {
  unsigned* counter;
  unsigned per_step, total;
  int hl, h0, nh, nct;
  __device__ __forceinline__ Queue(const Chain& c, int head, int h0_, int nh_, int nct_, int B)
      : counter(c.counters + head * kCounterWords), per_step(B * nct_), total(static_cast<unsigned>(c.steps) * B * nct_),
        hl(head), h0(h0_), nh(nh_), nct(nct_) {}
  __device__ __forceinline__ unsigned take() const { return ret::take(counter); }
  __device__ __forceinline__ int step(unsigned ticket) const { return ticket / per_step; }
  template <int CW>
  __device__ __forceinline__ ScanTile tile(unsigned ticket) const {
    const int i = ticket % per_step;
    return decode_tile((i / nct * nh + hl) * nct + i % nct, nct, nh, h0, CW);
  }
  __device__ __forceinline__ int number(const ScanTile& t) const { return (t.b * nh + hl) * nct + t.ct; }
};

// Where a thread stands in its tile.
template <int VEC, int CW, int NW, int PT = kPerThread>
struct Place {
  static constexpr int S = PT / VEC, LC = CW / VEC, TG = 64 / LC, NSEG = NW * TG, TT = NSEG * S;
  // a tile's checkpoints, one every PER waves
  static constexpr int BLOCKS = NW * PT / kBlockElems, PER = NW / BLOCKS, BLOCK = TT / BLOCKS;
  int lane, wave, lc, seg;
  __device__ Place()
      : lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), lc((threadIdx.x & 63) % LC),
        seg(wave * TG + (threadIdx.x & 63) / LC) {}
};

template <typename E>
__device__ __forceinline__ E* at_row(const void* p, const Strides3& s, const ScanTile& t, int c) {
  return const_cast<E*>(static_cast<const E*>(p)) + t.b * s.b + t.h * s.h + c;
}

// A thread's columns in its tile's LDS rows.  Rows that are whole vectors
// (kWhole): VEC columns from lc * VEC on.  Else the row's last vector reaches
// back over skip elements that belong to the lane before, which this lane
// neither hands on nor stores.
template <int VEC, bool kWhole>
struct Columns {
  int first, skip;
  __device__ __forceinline__ Columns() {}
  __device__ __forceinline__ Columns(const Piece& p, int lc)
      : first(lc * VEC - (kWhole ? 0 : p.skip)), skip(kWhole ? 0 : p.skip) {}
  __device__ __forceinline__ void put(float* row, int e, float x) const {
    if (kWhole || e >= skip) row[first + e] = x;
  }
  __device__ __forceinline__ float get(const float* row, int e) const {
    return kWhole || e >= skip ? row[first + e] : 0.0f;
  }
  template <typename E>
  __device__ __forceinline__ void store(E* p, const float (&x)[VEC]) const {
    if (kWhole || skip == 0) {
      VecIO<E, VEC>::store(p, x);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= skip) Elem<E>::store(p, e, x[e]);
    }
  }
};

// A tile's maps are composed in two steps: every wave those of its own TG
// segments, which only its own lanes have written, then one wave those of the
// NW waves.  With one wave over all segments the others waited longer (bf16:
// B4 H8 T2048 d512 forward 43.7 us in place of 42.0; B1 H8 T32768 d512 forward
// and backward 536 in place of 498).
__device__ __forceinline__ void wave_sync() {  // LDS writes of the wave's lanes before, reads after
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// segA, segH: the segments' maps h -> A h + H, replaced by the map of the
// wave's segments before each; wA, wH: the wave's map.
template <typename P, int CW>
__device__ __forceinline__ void compose_wave(const P& pl, float (*segA)[CW], float (*segH)[CW], float (*wA)[CW],
                                             float (*wH)[CW]) {
  wave_sync();
  if (pl.lane < CW) {
    float a = 1.0f, h = 0.0f;
#pragma unroll
    for (int i = 0; i < P::TG; ++i) {
      const int k = pl.wave * P::TG + i;
      const float ai = segA[k][pl.lane], hi = segH[k][pl.lane];
      segA[k][pl.lane] = a;
      segH[k][pl.lane] = h;
      a *= ai;
      h = fmaf(ai, h, hi);
    }
    wA[pl.wave][pl.lane] = a;
    wH[pl.wave][pl.lane] = h;
  }
  wave_sync();
}

// The same in both directions: also G -> A G + segG from the wave's last
// segment on, replaced with its products segB by the map of the segments
// behind each.
template <typename P, int CW>
__device__ __forceinline__ void compose_wave(const P& pl, float (*segA)[CW], float (*segH)[CW], float (*segB)[CW],
                                             float (*segG)[CW], float (*wA)[CW], float (*wH)[CW], float (*wG)[CW]) {
  wave_sync();
  if (pl.lane < CW) {
    float b = 1.0f, g = 0.0f;
#pragma unroll 2
    for (int i = P::TG - 1; i >= 0; --i) {
      const int k = pl.wave * P::TG + i;
      const float ai = segA[k][pl.lane], gi = segG[k][pl.lane];
      segB[k][pl.lane] = b;
      segG[k][pl.lane] = g;
      b *= ai;
      g = fmaf(ai, g, gi);
    }
    wG[pl.wave][pl.lane] = g;
  }
  compose_wave<P, CW>(pl, segA, segH, wA, wH);
}

// ---- Forward ----
template <typename E, int VEC, int CW, int NW, int PT, bool kNorm, bool kWhole>
struct FwdThread {
  using P = Place<VEC, CW, NW, PT>;
  using IO = VecIO<E, VEC>;
  static constexpr int S = P::S, kAhead = VEC >= 4 ? 2 : 8 / VEC;
  const E *xp, *fp;
  E* yp;
  long sx, sf, sy;
  float rate;
  int T, seg;
  bool store;
  Columns<VEC, kWhole> cols;
  typename IO::Raw rx[S], rf[S];
  float x[S][VEC], cm[S][VEC];

  __device__ __forceinline__ FwdThread(const GatedScanFwd& p, const P& pl, float r)
      : sx(p.sx.t), sf(p.sf.t), sy(p.sy.t), rate(r), T(p.T), seg(pl.seg) {}
  __device__ __forceinline__ void aim_loads(const GatedScanFwd& p, const ScanTile& t, const P& pl) {
    const int c = Piece(t.c0 + pl.lc * VEC, p.d, VEC).at;  // lanes past the row's end read its start
    xp = at_row<E>(p.x, p.sx, t, c);
    fp = at_row<E>(p.f, p.sf, t, c);
  }
  __device__ __forceinline__ void aim_stores(const GatedScanFwd& p, const ScanTile& t, const P& pl) {
    const Piece pc(t.c0 + pl.lc * VEC, p.d, VEC);
    cols = Columns<VEC, kWhole>(pc, pl.lc);
    store = pc.in && p.y != nullptr;
    yp = at_row<E>(p.y, p.sy, t, pc.at);
  }
  __device__ __forceinline__ void load(int chunk) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const long t = min(chunk * P::TT + seg * S + s, T - 1);  // a token past the end: the last one, masked below
      rx[s] = IO::load(xp + t * sx);
      rf[s] = IO::load(fp + t * sf);
    }
  }
  template <bool kTable>
  __device__ __forceinline__ void unpack(int chunk, const float* table) {
    Gates<E, float, VEC, S>::template get<kTable>(rf, table, rate, cm);
#pragma unroll
    for (int s = 0; s < S; ++s) IO::unpack(rx[s], x[s]);
    if ((chunk + 1) * P::TT <= T) return;  // uniform; else tokens past the end leave the state as it is
    const int t0 = chunk * P::TT + seg * S;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (t0 + s >= T) cm[s][e] = x[s][e] = 0.0f;
  }
  __device__ __forceinline__ static float step(float m, float x, float h) { return decay_step<kNorm>(m, x, h); }
  // The map of the thread's tokens; cm and x become the maps up to each of
  // them, which give the tokens' values in one operation.
  __device__ __forceinline__ void map(float (&A)[VEC], float (&H)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      A[e] = 1.0f;
      H[e] = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float m = cm[s][e];
        cm[s][e] = A[e] = decayed(m, A[e]);
        x[s][e] = H[e] = step(m, x[s][e], H[e]);
      }
    }
  }
  // The same straight from the packed registers, row by row.  With a table the
  // gates are looked up again for the replay; without one they stay in cm.
  template <bool kTable>
  __device__ __forceinline__ void packed_map(int chunk, const float* table, float (&A)[VEC], float (&H)[VEC]) {
    const int t0 = chunk * P::TT + seg * S;
    const bool whole = (chunk + 1) * P::TT <= T;  // uniform
    if constexpr (!kTable) Gates<E, float, VEC, S>::direct(rf, rate, cm);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      A[e] = 1.0f;
      H[e] = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      // a few rows' lookups at a time: all at once would take a register for each
      if (kTable && s % kAhead == 0) __builtin_amdgcn_sched_barrier(0);
      float c[1][VEC], u[VEC];
      row<kTable>(s, table, c, u);
      if (!whole && t0 + s >= T) continue;  // tokens past the end leave the state as it is
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        A[e] = decayed(c[0][e], A[e]);
        H[e] = step(c[0][e], u[e], H[e]);
      }
    }
  }
  template <bool kTable>
  __device__ __forceinline__ void packed_replay(int chunk, const float* table, float (&h)[VEC]) {
    const int t0 = chunk * P::TT + seg * S;
    E* py = yp + min(t0, T - 1) * sy;
    if constexpr (kTable) {
      // the compiler would otherwise keep the map's gates in registers, twice as many as the packed ones
#pragma unroll
      for (int s = 0; s < S; ++s) asm("" : "+v"(rx[s]), "+v"(rf[s]));
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      // a few rows' lookups at a time: all at once would take a register for each
      if (kTable && s % kAhead == 0) __builtin_amdgcn_sched_barrier(0);
      float c[1][VEC], u[VEC];
      row<kTable>(s, table, c, u);
      if (t0 + s >= T) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = step(c[0][e], u[e], h[e]);
      if (store) cols.template store<E>(py, h);
      py += sy;
    }
  }
  template <bool kTable>
  __device__ __forceinline__ void row(int s, const float* table, float (&c)[1][VEC], float (&u)[VEC]) {
    if constexpr (kTable) {
      const typename IO::Raw one[1] = {rf[s]};
      Gates<E, float, VEC, 1>::template get<true>(one, table, rate, c);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[0][e] = cm[s][e];
    }
    IO::unpack(rx[s], u);
  }
  // the thread's tokens from their incoming value, by the maps that map() left
  __device__ __forceinline__ void replay(int chunk, const float (&in)[VEC]) const {
    const int t0 = chunk * P::TT + seg * S;
    E* py = yp + min(t0, T - 1) * sy;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float h[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = fmaf(cm[s][e], in[e], x[s][e]);
      if (store && t0 + s < T) cols.template store<E>(py, h);
      py += sy;
    }
  }
};

// One workgroup walks the tiles of a channel run from the first token on.
template <typename E, int VEC, int CW, int NW, bool kNorm, bool kWhole, bool kTable>
__global__ __launch_bounds__(64 * NW) void gated_scan_fwd_walk_kernel(GatedScanFwd p, HeadRate rates, int h0, int nh,
                                                                       int nct) {
  using P = Place<VEC, CW, NW>;
  __shared__ float segA[P::NSEG][CW];
  __shared__ float segH[P::NSEG][CW];
  __shared__ float waveA[2][NW][CW];
  __shared__ float waveH[2][NW][CW];
  const P pl;
  const ScanTile tl = decode_tile(blockIdx.x, nct, nh, h0, CW);
  FwdThread<E, VEC, CW, NW, kPerThread, kNorm, kWhole> th(p, pl, rates.r[tl.hl]);
  th.aim_loads(p, tl, pl);
  th.aim_stores(p, tl, pl);
  // the composing wave: one channel per lane
  const int ch = tl.c0 + pl.lane;
  const bool mine = pl.wave == 0 && pl.lane < CW, kept = mine && ch < p.d;
  const long bh = static_cast<long>(tl.b) * p.H + tl.h;
  float carry = kept && p.state_in != nullptr ? p.state_in[bh * p.d + ch] : 0.0f;
  const int nchunk = (p.T + P::TT - 1) / P::TT, nblock = (p.T + P::BLOCK - 1) / P::BLOCK;
  th.load(0);
  __shared__ float gate[kTable ? kGateN : 1];
  if constexpr (kTable) {
    build_gate_table(gate, th.rate, 64 * NW);
    __syncthreads();
  }
  for (int chunk = 0; chunk < nchunk; ++chunk) {
    th.template unpack<kTable>(chunk, gate);
    if (chunk + 1 < nchunk) th.load(chunk + 1);
    const int q = chunk & 1;
    float A[VEC], H[VEC];
    th.map(A, H);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      th.cols.put(segA[pl.seg], e, A[e]);
      th.cols.put(segH[pl.seg], e, H[e]);
    }
    compose_wave<P, CW>(pl, segA, segH, waveA[q], waveH[q]);
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int k = 0; k < P::BLOCKS; ++k) {
        const int block = chunk * P::BLOCKS + k;
        if (kept && p.checkpoints != nullptr && block < nblock) p.checkpoints[(bh * nblock + block) * p.d + ch] = carry;
#pragma unroll
        for (int i = k * P::PER; i < (k + 1) * P::PER; ++i) {
          const float a = waveA[q][i][pl.lane], hh = waveH[q][i][pl.lane];
          waveH[q][i][pl.lane] = carry;
          carry = fmaf(a, carry, hh);
        }
      }
    }
    __syncthreads();
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      h[e] = fmaf(th.cols.get(segA[pl.seg], e), th.cols.get(waveH[q][pl.wave], e), th.cols.get(segH[pl.seg], e));
    th.replay(chunk, h);
  }
  if (kept && p.state_out != nullptr) p.state_out[bh * p.d + ch] = carry;
}

// Workgroups of one head (blockIdx modulo the heads) on the tiles of its queue.
// A thread keeps its PT elements packed as they were read and evaluates their
// gates twice, for the tile's map and for the replay: by table that is cheap,
// and few registers let two workgroups with 256-token tiles share a compute
// unit.  Without a table the tiles are half as long.
template <typename E, int VEC, int CW, int NW, int PT, bool kNorm, bool kWhole, bool kTable>
__global__ __launch_bounds__(64 * NW, 4) void gated_scan_fwd_chain_kernel(GatedScanFwd p, Chain cn, HeadRate rates,
                                                                       int h0, int nh, int nct) {
  using P = Place<VEC, CW, NW, PT>;
  using Th = FwdThread<E, VEC, CW, NW, PT, kNorm, kWhole>;
  __shared__ float segA[P::NSEG][CW];
  __shared__ float segH[P::NSEG][CW];
  __shared__ float waveA[NW][CW];
  __shared__ float waveH[NW][CW];
  __shared__ float enter[CW];
  __shared__ unsigned ticket;
  __shared__ float gate[kTable ? kGateN : 1];
  const P pl;
  const Queue qu(cn, blockIdx.x % nh, h0, nh, nct, p.B);
  if (threadIdx.x == 0) ticket = qu.take();
  Th th(p, pl, rates.r[qu.hl]);
  if constexpr (kTable) build_gate_table(gate, th.rate, 64 * NW);
  __syncthreads();
  const int nblock = (p.T + P::BLOCK - 1) / P::BLOCK;
  for (unsigned cur = uniform(ticket); cur < qu.total;) {
    const int chunk = qu.step(cur);
    const ScanTile tl = qu.template tile<CW>(cur);
    th.aim_loads(p, tl, pl);
    th.aim_stores(p, tl, pl);
    th.load(chunk);
    float A[VEC], H[VEC];
    th.template packed_map<kTable>(chunk, gate, A, H);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      th.cols.put(segA[pl.seg], e, A[e]);
      th.cols.put(segH[pl.seg], e, H[e]);
    }
    compose_wave<P, CW>(pl, segA, segH, waveA, waveH);
    __syncthreads();
    if (threadIdx.x == 64) ticket = qu.take();
    if (pl.wave == 0 && pl.lane < CW) {
      const int ch = tl.c0 + pl.lane, tile = qu.number(tl);
      const long bh = static_cast<long>(tl.b) * p.H + tl.h;
      const bool kept = ch < p.d;
      Entering<CW> in;
      in.begin(cn, chunk, tile, pl.lane);
      const float first = kept && chunk == 0 && p.state_in != nullptr ? p.state_in[bh * p.d + ch] : 0.0f;
      float a = 1.0f, h = 0.0f, ca[P::BLOCKS], chh[P::BLOCKS];  // the map of the waves so far, and at the blocks
#pragma unroll
      for (int k = 0; k < P::BLOCKS; ++k) {
        ca[k] = a;
        chh[k] = h;
#pragma unroll
        for (int i = k * P::PER; i < (k + 1) * P::PER; ++i) {
          const float ai = waveA[i][pl.lane], hi = waveH[i][pl.lane];
          waveA[i][pl.lane] = a;
          waveH[i][pl.lane] = h;
          a *= ai;
          h = fmaf(ai, h, hi);
        }
      }
      publish_map<CW>(cn, chunk, tile, pl.lane, a, h, first);
      const float v = in.end(cn, chunk, tile, pl.lane, a, h, first);
      enter[pl.lane] = v;
      if (kept) {
        if (p.checkpoints != nullptr)
#pragma unroll
          for (int k = 0; k < P::BLOCKS; ++k)
            if (chunk * P::BLOCKS + k < nblock)
              p.checkpoints[(bh * nblock + chunk * P::BLOCKS + k) * p.d + ch] = fmaf(ca[k], v, chh[k]);
        if (p.state_out != nullptr && chunk == cn.steps - 1) p.state_out[bh * p.d + ch] = fmaf(a, v, h);
      }
    }
    __syncthreads();
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float v = fmaf(th.cols.get(waveA[pl.wave], e), th.cols.get(enter, e), th.cols.get(waveH[pl.wave], e));
      h[e] = fmaf(th.cols.get(segA[pl.seg], e), v, th.cols.get(segH[pl.seg], e));
    }
    cur = uniform(ticket);
    th.template packed_replay<kTable>(chunk, gate, h);
    __syncthreads();  // the waves' maps, the entering values and the ticket are read
  }
}

// ---- Backward ----
// g_t = dL/dh_t = dy_t + a_(t+1) g_(t+1); what crosses a token boundary is
// G_t = a_t g_t, so a token maps G -> a_t (dy_t + G), last token first.
// h_(t-1) comes from replaying the tile forwards from its checkpoint:
//   dx_t = g_t (normalize: c_t g_t),  df_t = g_t (h_(t-1) [- x_t]) a_t rate sigmoid(-f_t).
template <typename E, int VEC, int CW, int NW, bool kNorm, bool kWhole>
struct BwdThread {
  using P = Place<VEC, CW, NW>;
  using IO = VecIO<E, VEC>;
  static constexpr int S = P::S;
  const E *xp, *fp, *gyp;
  E *gxp, *gfp;
  long sx, sf, sgy, sgx, sgf;
  float rate;
  int T, seg;
  bool store;
  Columns<VEC, kWhole> cols;
  typename IO::Raw rx[S], rf[S], rg[S];
  float x[S][VEC], cm[S][VEC], kf[S][VEC], dy[S][VEC];

  __device__ __forceinline__ BwdThread(const GatedScanBwd& p, const P& pl, float r)
      : sx(p.sx.t), sf(p.sf.t), sgy(p.sgy.t), sgx(p.sgx.t), sgf(p.sgf.t), rate(r), T(p.T), seg(pl.seg) {}
  __device__ __forceinline__ void aim_loads(const GatedScanBwd& p, const ScanTile& t, const P& pl) {
    const int c = Piece(t.c0 + pl.lc * VEC, p.d, VEC).at;
    xp = at_row<E>(p.x, p.sx, t, c);
    fp = at_row<E>(p.f, p.sf, t, c);
    gyp = at_row<E>(p.grad_y, p.sgy, t, c);
  }
  __device__ __forceinline__ void aim_stores(const GatedScanBwd& p, const ScanTile& t, const P& pl) {
    const Piece pc(t.c0 + pl.lc * VEC, p.d, VEC);
    cols = Columns<VEC, kWhole>(pc, pl.lc);
    gxp = at_row<E>(p.grad_x, p.sgx, t, pc.at);
    gfp = at_row<E>(p.grad_f, p.sgf, t, pc.at);
    store = pc.in;
  }
  __device__ __forceinline__ void load(int chunk) {
    // one product of token and stride for the rows: products take a quarter of the rate
    const int t0 = chunk * P::TT + seg * S;
    const E* px = xp + min(t0, T - 1) * sx;
    const E* pf = fp + min(t0, T - 1) * sf;
    const E* pg = gyp + min(t0, T - 1) * sgy;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool on = t0 + s < T;  // else another token that exists, masked below
      rx[s] = IO::load(px + (on ? s * sx : 0));
      rf[s] = IO::load(pf + (on ? s * sf : 0));
      rg[s] = IO::load(pg + (on ? s * sgy : 0));
    }
  }
  template <bool kTable>
  __device__ __forceinline__ void unpack(int chunk, const float2* table) {
    float2 g[S][VEC];
    Gates<E, float2, VEC, S>::template get<kTable>(rf, table, rate, g);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      IO::unpack(rx[s], x[s]);
      IO::unpack(rg[s], dy[s]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        cm[s][e] = g[s][e].x;
        kf[s][e] = g[s][e].y;
      }
    }
    if ((chunk + 1) * P::TT <= T) return;
    const int t0 = chunk * P::TT + seg * S;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (t0 + s >= T) cm[s][e] = x[s][e] = dy[s][e] = 0.0f;
  }
  // the maps of the thread's tokens: h -> A h + H forwards, G -> A G + R
  // backwards, where every token's dy has passed the decays up to its own
  __device__ __forceinline__ void map(int e, float& A, float& H, float& R) const {
    A = 1.0f;
    H = R = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      A = decayed(cm[s][e], A);
      R = fmaf(A, dy[s][e], R);
      H = decay_step<kNorm>(cm[s][e], x[s][e], H);
    }
  }
  // replays the tokens of element e forwards from h: kf becomes dy_t -> df_t, a_t h'_t with h'_t = dh_t / da_t
  __device__ __forceinline__ void replay_state(int e, float h) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      kf[s][e] *= kNorm ? h - x[s][e] : h;
      h = decay_step<kNorm>(cm[s][e], x[s][e], h);
    }
  }
  // and backwards from G behind them: g becomes dx, k becomes df
  __device__ __forceinline__ static void replay_grad(int e, float G, const float (&c)[S][VEC], float (&g)[S][VEC],
                                                     float (&k)[S][VEC]) {
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
      const float gs = g[s][e] + G;
      G = decayed(c[s][e], gs);
      g[s][e] = kNorm ? complement(c[s][e], gs) : gs;
      k[s][e] *= gs;
    }
  }
  __device__ __forceinline__ void write(int chunk, const float (&dx)[S][VEC], const float (&df)[S][VEC]) const {
    const int t0 = chunk * P::TT + seg * S;
    E* px = gxp + min(t0, T - 1) * sgx;
    E* pf = gfp + min(t0, T - 1) * sgf;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (store && t0 + s < T) {
        cols.template store<E>(px, dx[s]);
        cols.template store<E>(pf, df[s]);
      }
      px += sgx;
      pf += sgf;
    }
  }
};

// One workgroup walks the tiles of a channel run from the last token on.
template <typename E, int VEC, int CW, int NW, bool kNorm, bool kWhole, bool kTable>
__global__ __launch_bounds__(64 * NW) void gated_scan_bwd_walk_kernel(GatedScanBwd p, HeadRate rates, int h0, int nh,
                                                                       int nct) {
  using P = Place<VEC, CW, NW>;
  __shared__ float segA[P::NSEG][CW];
  __shared__ float segH[P::NSEG][CW];
  __shared__ float segB[P::NSEG][CW];  // products of A behind a segment
  __shared__ float segG[P::NSEG][CW];
  __shared__ float waveA[2][NW][CW];
  __shared__ float waveH[2][NW][CW];
  __shared__ float waveG[2][NW][CW];
  const P pl;
  const ScanTile tl = decode_tile(blockIdx.x, nct, nh, h0, CW);
  BwdThread<E, VEC, CW, NW, kNorm, kWhole> th(p, pl, rates.r[tl.hl]);
  th.aim_loads(p, tl, pl);
  th.aim_stores(p, tl, pl);
  const int ch = tl.c0 + pl.lane;
  const bool kept = pl.wave < 2 && pl.lane < CW && ch < p.d;  // wave 0 composes forwards, wave 1 backwards
  const long bh = static_cast<long>(tl.b) * p.H + tl.h;
  float carry = pl.wave == 1 && kept && p.grad_state_out != nullptr ? p.grad_state_out[bh * p.d + ch] : 0.0f;
  const int nchunk = (p.T + P::TT - 1) / P::TT, nblock = (p.T + P::BLOCK - 1) / P::BLOCK;
  th.load(nchunk - 1);
  __shared__ float2 gate[kTable ? kGateN : 1];
  if constexpr (kTable) {
    build_gate_table(gate, th.rate, 64 * NW);
    __syncthreads();
  }
  for (int chunk = nchunk - 1; chunk >= 0; --chunk) {
    th.template unpack<kTable>(chunk, gate);
    const float ckpt = pl.wave == 0 && kept ? p.checkpoints[(bh * nblock + chunk * P::BLOCKS) * p.d + ch] : 0.0f;
    if (chunk > 0) th.load(chunk - 1);
    const int q = chunk & 1;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float A, H, R;
      th.map(e, A, H, R);
      th.cols.put(segA[pl.seg], e, A);
      th.cols.put(segH[pl.seg], e, H);
      th.cols.put(segG[pl.seg], e, R);
    }
    compose_wave<P, CW>(pl, segA, segH, segB, segG, waveA[q], waveH[q], waveG[q]);
    __syncthreads();
    if (pl.wave == 0 && pl.lane < CW) {
      float cur = ckpt;
#pragma unroll 4
      for (int i = 0; i < NW; ++i) {
        const float a = waveA[q][i][pl.lane], hh = waveH[q][i][pl.lane];
        waveH[q][i][pl.lane] = cur;
        cur = fmaf(a, cur, hh);
      }
    } else if (pl.wave == 1 && pl.lane < CW) {
#pragma unroll 4
      for (int i = NW - 1; i >= 0; --i) {
        const float a = waveA[q][i][pl.lane], gg = waveG[q][i][pl.lane];
        waveG[q][i][pl.lane] = carry;
        carry = fmaf(a, carry, gg);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      // one channel at a time: interleaved they hold more registers (B2 H16 T8192
      // d512 bf16, forward and backward, 452 us in place of 440)
      __builtin_amdgcn_sched_barrier(0);
      th.replay_state(e, fmaf(th.cols.get(segA[pl.seg], e), th.cols.get(waveH[q][pl.wave], e),
                              th.cols.get(segH[pl.seg], e)));
      th.replay_grad(e, fmaf(th.cols.get(segB[pl.seg], e), th.cols.get(waveG[q][pl.wave], e),
                             th.cols.get(segG[pl.seg], e)), th.cm, th.dy, th.kf);
    }
    th.write(chunk, th.dy, th.kf);
  }
  if (pl.wave == 1 && kept && p.grad_state_in != nullptr) p.grad_state_in[bh * p.d + ch] = carry;
}

// Workgroups of one head on the tiles of its queue, from the last token on.
template <typename E, int VEC, int CW, int NW, bool kNorm, bool kWhole, bool kTable>
__global__ __launch_bounds__(64 * NW) void gated_scan_bwd_chain_kernel(GatedScanBwd p, Chain cn, HeadRate rates,
                                                                       int h0, int nh, int nct) {
  using P = Place<VEC, CW, NW>;
  __shared__ float segA[P::NSEG][CW];
  __shared__ float segH[P::NSEG][CW];
  __shared__ float segG[P::NSEG][CW];
  __shared__ float segB[P::NSEG][CW];  // products of A behind a segment
  __shared__ float waveA[NW][CW];
  __shared__ float waveH[NW][CW];
  __shared__ float waveB[NW][CW];
  __shared__ float waveG[NW][CW];
  __shared__ float enter[CW];
  __shared__ unsigned tickets[2];
  __shared__ float2 gate[kTable ? kGateN : 1];
  const P pl;
  const Queue qu(cn, blockIdx.x % nh, h0, nh, nct, p.B);
  auto chunk_of = [&](unsigned ticket) __attribute__((always_inline)) { return cn.steps - 1 - qu.step(ticket); };
  if (threadIdx.x == 0) tickets[0] = qu.take();
  __syncthreads();
  unsigned cur = uniform(tickets[0]);
  if (cur >= qu.total) return;  // the whole workgroup
  if (threadIdx.x == 0) tickets[1] = qu.take();
  const int nblock = (p.T + P::BLOCK - 1) / P::BLOCK;
  BwdThread<E, VEC, CW, NW, kNorm, kWhole> th(p, pl, rates.r[qu.hl]);
  ScanTile tl = qu.template tile<CW>(cur);
  th.aim_loads(p, tl, pl);
  th.load(chunk_of(cur));
  if constexpr (kTable) build_gate_table(gate, th.rate, 64 * NW);
  __syncthreads();  // the table and the second ticket
  unsigned next = uniform(tickets[1]);
  for (;;) {
    const int step = qu.step(cur), chunk = cn.steps - 1 - step;
    const int ch = tl.c0 + pl.lane, tile = qu.number(tl);
    const bool channel = pl.lane < CW, kept = channel && ch < p.d;
    const long bh = static_cast<long>(tl.b) * p.H + tl.h;
    // wave 0: the state before the tile; wave 1: the gradient behind the sequence
    float start = 0.0f;
    if (pl.wave == 0 && kept) start = p.checkpoints[(bh * nblock + chunk * P::BLOCKS) * p.d + ch];
    if (pl.wave == 1 && kept && step == 0 && p.grad_state_out != nullptr) start = p.grad_state_out[bh * p.d + ch];
    th.aim_stores(p, tl, pl);
    th.template unpack<kTable>(chunk, gate);
    if (next < qu.total) {
      tl = qu.template tile<CW>(next);
      th.aim_loads(p, tl, pl);
      th.load(chunk_of(next));
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float A, H, R;
      th.map(e, A, H, R);
      th.cols.put(segA[pl.seg], e, A);
      th.cols.put(segH[pl.seg], e, H);
      th.cols.put(segG[pl.seg], e, R);
    }
    compose_wave<P, CW>(pl, segA, segH, segB, segG, waveA, waveH, waveG);
    __syncthreads();
    if (threadIdx.x == 128 && next < qu.total) tickets[0] = qu.take();
    if (pl.wave == 0 && channel) {
#pragma unroll 4
      for (int i = 0; i < NW; ++i) {
        const float a = waveA[i][pl.lane], hh = waveH[i][pl.lane];
        waveH[i][pl.lane] = start;
        start = fmaf(a, start, hh);
      }
    } else if (pl.wave == 1 && channel) {
      Entering<CW> in;
      in.begin(cn, step, tile, pl.lane);
      float a = 1.0f, g = 0.0f;  // the map of the waves behind
#pragma unroll 4
      for (int i = NW - 1; i >= 0; --i) {
        const float ai = waveA[i][pl.lane], gi = waveG[i][pl.lane];
        waveB[i][pl.lane] = a;
        waveG[i][pl.lane] = g;
        a *= ai;
        g = fmaf(ai, g, gi);
      }
      publish_map<CW>(cn, step, tile, pl.lane, a, g, start);
      const float v = in.end(cn, step, tile, pl.lane, a, g, start);
      enter[pl.lane] = v;
      if (kept && p.grad_state_in != nullptr && chunk == 0) p.grad_state_in[bh * p.d + ch] = fmaf(a, v, g);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      th.replay_state(e, fmaf(th.cols.get(segA[pl.seg], e), th.cols.get(waveH[pl.wave], e),
                              th.cols.get(segH[pl.seg], e)));
      const float v = fmaf(th.cols.get(waveB[pl.wave], e), th.cols.get(enter, e), th.cols.get(waveG[pl.wave], e));
      th.replay_grad(e, fmaf(th.cols.get(segB[pl.seg], e), v, th.cols.get(segG[pl.seg], e)), th.cm, th.dy, th.kf);
    }
    cur = next;
    next = uniform(tickets[0]);
    __syncthreads();  // the waves' maps, the entering values and the ticket are read
    th.write(chunk, th.dy, th.kf);
    if (cur >= qu.total) break;
  }
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
    float t, a;
    st[e] = decay_step<kNorm>(held_decay(f[e], rates.r[hl], &t, &a), x[e], st[e]);
  }
  if (p.state_out != nullptr) VecIO<float, VEC>::store(p.state_out + row, st);
  if (p.y != nullptr) IO::store(static_cast<E*>(p.y) + b * p.sy.b + h * p.sy.h + c, st);
}

HeadRate head_rates(const HeadGroup& g) {
  HeadRate r;
  for (int i = 0; i < kHeadsPerLaunch; ++i) r.r[i] = i < g.nh ? g.gamma[i] : 1.0f;
  return r;
}

// Tile width for a row of d channels: 64, or the next power of two for
// narrow rows so that lanes are not left idle.
int tile_width(int d) { return d > 32 ? 64 : d > 16 ? 32 : 16; }
// Tokens of a tile with elems elements per lane over its waves.
int tile_tokens(int d, int elems) { return elems * 64 / tile_width(d); }

// The chained kernels' part of the workspace for a launch of nh heads.
struct ChainSizes {
  int steps, tiles;
  size_t maps, enter;  // words of 8 and of 4 bytes
};
ChainSizes chain_sizes(int B, int nh, int T, int d, int elems) {
  const int cw = tile_width(d), tt = tile_tokens(d, elems);
  ChainSizes z;
  z.steps = (T + tt - 1) / tt;
  z.tiles = B * nh * ((d + cw - 1) / cw);
  z.maps = static_cast<size_t>(z.steps) * z.tiles * cw;
  z.enter = static_cast<size_t>((z.steps + kGroup - 1) / kGroup) * z.tiles * cw;
  return z;
}

// Whether the tiles of a channel run are chained over workgroups (else one
// workgroup walks them).
bool chained(int B, int H, int T, int d) {
  const ChainSizes z = chain_sizes(B, H < kHeadsPerLaunch ? H : kHeadsPerLaunch, T, d, kBlockElems);
  return z.steps >= kChainSteps && z.tiles < kWalkTiles;
}

// [counters][maps][enter], all ones at the start.
hipError_t make_chain(void* ws, int B, int nh, int T, int d, int elems, Chain* c, hipStream_t s) {
  const ChainSizes z = chain_sizes(B, nh, T, d, elems);
  c->counters = static_cast<unsigned*>(ws);
  c->maps = reinterpret_cast<u64*>(c->counters + nh * kCounterWords);
  c->enter = reinterpret_cast<unsigned*>(c->maps + z.maps);
  c->steps = z.steps;
  c->tiles = z.tiles;
  return launch_fill_u32(ws, static_cast<size_t>(nh) * kCounterWords + z.maps * 2 + z.enter, 0xFFFFFFFFu, s);
}

// Workgroups of a chained launch: per_cu for each compute unit, shared out to
// the heads, at most one for each tile.
int chain_blocks(int steps, int tiles, int nh, int per_cu) {
  const long per_head = static_cast<long>(steps) * (tiles / nh);
  const long want = 256L * per_cu / nh > 1 ? 256L * per_cu / nh : 1;
  return nh * static_cast<int>(want < per_head ? want : per_head);
}
// Whether the workgroups of a chained launch have so many tiles that a gate
// table pays.
bool many_tiles(int B, int nh, int T, int d, int elems, int per_cu) {
  const ChainSizes z = chain_sizes(B, nh, T, d, elems);
  return static_cast<long>(z.steps) * z.tiles >= static_cast<long>(kTableTiles) * chain_blocks(z.steps, z.tiles, nh, per_cu);
}
// Whether a run is longer than so many blocks.
bool longer(int T, int d, int blocks) { return T > blocks * tile_tokens(d, kBlockElems); }

template <typename E, int VEC, int CW, bool kNorm, bool kWhole>
hipError_t run_fwd(const GatedScanFwd& p, void* ws, const HeadGroup& g, hipStream_t s) {
  const int nct = (p.d + CW - 1) / CW;
  if (!chained(p.B, p.H, p.T, p.d)) {
    const dim3 runs(p.B * g.nh * nct);
    if (sizeof(E) == 2 && !longer(p.T, p.d, kTableStepsFwd)) {
      hipLaunchKernelGGL((gated_scan_fwd_walk_kernel<E, VEC, CW, 8, kNorm, kWhole, false>), runs, dim3(64 * 8), 0, s, p,
                         head_rates(g), g.h0, g.nh, nct);
      return hipGetLastError();
    }
    constexpr int NW = VEC == 1 ? 8 : 16;
    hipLaunchKernelGGL((gated_scan_fwd_walk_kernel<E, VEC, CW, NW, kNorm, kWhole, sizeof(E) == 2>), runs, dim3(64 * NW), 0,
                       s, p, head_rates(g), g.h0, g.nh, nct);
    return hipGetLastError();
  }
  constexpr int NW = 8, kLong = sizeof(E) == 2 && VEC > 1 ? 32 : 16;  // elements of a thread: by table, directly
  const bool table = sizeof(E) == 2 && many_tiles(p.B, g.nh, p.T, p.d, NW * kLong, 2);
  Chain c;
  const hipError_t e = make_chain(ws, p.B, g.nh, p.T, p.d, NW * (table ? kLong : 16), &c, s);
  if (e != hipSuccess) return e;
  if (table)
    hipLaunchKernelGGL((gated_scan_fwd_chain_kernel<E, VEC, CW, NW, kLong, kNorm, kWhole, sizeof(E) == 2>),
                       dim3(chain_blocks(c.steps, c.tiles, g.nh, 2)), dim3(64 * NW), 0, s, p, c, head_rates(g), g.h0,
                       g.nh, nct);
  else
    hipLaunchKernelGGL((gated_scan_fwd_chain_kernel<E, VEC, CW, NW, 16, kNorm, kWhole, false>),
                       dim3(chain_blocks(c.steps, c.tiles, g.nh, 3)), dim3(64 * NW), 0, s, p, c, head_rates(g), g.h0,
                       g.nh, nct);
  return hipGetLastError();
}

template <typename E, int VEC, bool kNorm>
hipError_t run_step(const GatedScanFwd& p, const HeadGroup& g, hipStream_t s) {
  const long n = static_cast<long>(p.B) * g.nh * (p.d / VEC);
  hipLaunchKernelGGL((gated_scan_step_kernel<E, VEC, kNorm>), dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256),
                     0, s, p, head_rates(g), g.h0, g.nh, n);
  return hipGetLastError();
}

template <typename E, int VEC, int CW, bool kNorm, bool kWhole>
hipError_t run_bwd(const GatedScanBwd& p, void* ws, const HeadGroup& g, hipStream_t s) {
  const int nct = (p.d + CW - 1) / CW;
  if (!chained(p.B, p.H, p.T, p.d)) {
    const dim3 runs(p.B * g.nh * nct);
    if (sizeof(E) == 2 && !longer(p.T, p.d, kTableStepsBwd)) {
      hipLaunchKernelGGL((gated_scan_bwd_walk_kernel<E, VEC, CW, 8, kNorm, kWhole, false>), runs, dim3(64 * 8), 0, s, p,
                         head_rates(g), g.h0, g.nh, nct);
      return hipGetLastError();
    }
    constexpr int NW = sizeof(E) == 4 || VEC == 1 ? 8 : 16;  // by the registers of a thread, 512 / (NW / 4)
    hipLaunchKernelGGL((gated_scan_bwd_walk_kernel<E, VEC, CW, NW, kNorm, kWhole, sizeof(E) == 2>), runs, dim3(64 * NW), 0,
                       s, p, head_rates(g), g.h0, g.nh, nct);
    return hipGetLastError();
  }
  constexpr int NW = 8;
  Chain c;
  const hipError_t e = make_chain(ws, p.B, g.nh, p.T, p.d, NW * kPerThread, &c, s);
  if (e != hipSuccess) return e;
  const int blocks = chain_blocks(c.steps, c.tiles, g.nh, 1);
  if (sizeof(E) == 2 && many_tiles(p.B, g.nh, p.T, p.d, NW * kPerThread, 1))
    hipLaunchKernelGGL((gated_scan_bwd_chain_kernel<E, VEC, CW, NW, kNorm, kWhole, sizeof(E) == 2>), dim3(blocks), dim3(64 * NW),
                       0, s, p, c, head_rates(g), g.h0, g.nh, nct);
  else
    hipLaunchKernelGGL((gated_scan_bwd_chain_kernel<E, VEC, CW, NW, kNorm, kWhole, false>), dim3(blocks), dim3(64 * NW), 0, s,
                       p, c, head_rates(g), g.h0, g.nh, nct);
  return hipGetLastError();
}

// Rows of 4 channels or more move in vectors of 4 at any alignment, narrower
// ones by the channel.
template <template <typename, int, int, bool, bool> class F, typename E, int VEC, bool kWhole, typename... A>
hipError_t by_width(int cw, bool norm, A&&... a) {
  if (cw == 64) return norm ? F<E, VEC, 64, true, kWhole>::run(a...) : F<E, VEC, 64, false, kWhole>::run(a...);
  if (cw == 32) return norm ? F<E, VEC, 32, true, kWhole>::run(a...) : F<E, VEC, 32, false, kWhole>::run(a...);
  return norm ? F<E, VEC, 16, true, kWhole>::run(a...) : F<E, VEC, 16, false, kWhole>::run(a...);
}
template <template <typename, int, int, bool, bool> class F, typename E, typename... A>
hipError_t by_row(int d, bool norm, A&&... a) {
  if (d < 4) return norm ? F<E, 1, 16, true, true>::run(a...) : F<E, 1, 16, false, true>::run(a...);
  return d % 4 == 0 ? by_width<F, E, 4, true>(tile_width(d), norm, a...) : by_width<F, E, 4, false>(tile_width(d), norm, a...);
}

template <typename E, int VEC, int CW, bool kNorm, bool kWhole>
struct Fwd {
  static hipError_t run(const GatedScanFwd& p, void* ws, const HeadGroup& g, hipStream_t s) {
    return run_fwd<E, VEC, CW, kNorm, kWhole>(p, ws, g, s);
  }
};
template <typename E, int VEC, int CW, bool kNorm, bool kWhole>
struct Bwd {
  static hipError_t run(const GatedScanBwd& p, void* ws, const HeadGroup& g, hipStream_t s) {
    return run_bwd<E, VEC, CW, kNorm, kWhole>(p, ws, g, s);
  }
};

template <typename E>
hipError_t step_by_row(const GatedScanFwd& p, const HeadGroup& g, hipStream_t s) {
  if (p.d % 4 == 0) return p.normalize ? run_step<E, 4, true>(p, g, s) : run_step<E, 4, false>(p, g, s);
  return p.normalize ? run_step<E, 1, true>(p, g, s) : run_step<E, 1, false>(p, g, s);
}

}  // namespace

int gated_scan_block(int d) { return tile_tokens(d, kBlockElems); }
int gated_scan_tiles(int d) { return static_cast<int>((d + static_cast<long>(tile_width(d)) - 1) / tile_width(d)); }

size_t gated_scan_chain_bytes(int B, int H, int T, int d) {
  if (T <= 1 || !chained(B, H, T, d)) return 0;
  const int nh = H < kHeadsPerLaunch ? H : kHeadsPerLaunch;
  const ChainSizes z = chain_sizes(B, nh, T, d, kBlockElems);  // longer tiles are fewer
  return static_cast<size_t>(nh) * kCounterWords * 4 + z.maps * 8 + z.enter * 4;
}

hipError_t launch_gated_scan_fwd(const GatedScanFwd& p, void* ws, const HeadGroup& g, hipStream_t s) {
  if (p.T == 1) return p.dt == 1 ? step_by_row<uint16_t>(p, g, s) : step_by_row<float>(p, g, s);
  return p.dt == 1 ? by_row<Fwd, uint16_t>(p.d, p.normalize, p, ws, g, s)
                   : by_row<Fwd, float>(p.d, p.normalize, p, ws, g, s);
}

hipError_t launch_gated_scan_bwd(const GatedScanBwd& p, void* ws, const HeadGroup& g, hipStream_t s) {
  return p.dt == 1 ? by_row<Bwd, uint16_t>(p.d, p.normalize, p, ws, g, s)
                   : by_row<Bwd, float>(p.d, p.normalize, p, ws, g, s);
}

}  // namespace ret
