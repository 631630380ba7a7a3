// head_norm.cu -- RMS norm of every query and key head with the position
// rotation in the same pass, its form that writes keys and values into a
// paged cache, and its backward pass.
//
// Per token and head x [d], with r = (mean x^2 + eps)^(-1/2) and z = x r w,
// the first `rot` elements of z are turned in pairs by the angle
// position * inv_freq[i] (pairs (i, i + rot/2), or (2i, 2i+1) interleaved).
// Backward: dz = the turned-back gradient, u = dz w, dx = r (u - x r^2
// mean(u x)), dw = sum over tokens and heads of dz x r.
//
// Everything is bound by memory (each element is read and written once, with
// a few dozen operations).  A head is held by a team of TEAM lanes, each
// with the two 16-byte vectors whose elements pair up, so the rotation needs
// no exchange and the norm one shuffle reduction.  A warp takes a token row
// (or a part of its heads) at a time: its lanes form the row's angles once in
// shared memory of the warp's own, one cosine and sine per token and pair
// instead of one per head, and go through the heads with several of them in
// flight; no warp waits for another.
//
// Measured on GB300, bf16: 65536 tokens of 56 + 8 heads of 128, 332 us
// (6.5 TB/s); 256 tokens of 56 + 8 + 8 heads into a cache, 7.1 us (frequencies,
// position, page and heads are read one after the other, although only the
// store's address needs the page); backward over 16384 tokens of 16 + 16 heads, 69 us (5.8
// TB/s, two heads in flight: three take 77 us, four 82) and 4.4 us for the
// weights' sums.
//
// Angles.  A frequency is kept as a 64-bit fraction of a turn per position,
// and position * step wraps modulo one turn exactly, so far positions lose
// nothing: the angle is off by the rounding of inv_freq / 2 pi in 64 bits and
// by 2^-25 of half a turn when its upper 32 bits become an fp32 argument.
// The fraction is formed in integers (the mantissa times 2^66 / 2 pi), since
// fp64 instructions are slow on this GPU.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace attnres {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBackFlight = 2;         // heads a team of the backward kernel has in flight

// inv_freq (radians per position) as 2^-64ths of a turn per position, modulo
// one turn.  The last bit says that inv_freq is no finite number (2^-64 of a
// turn is less than what the angle is rounded by at any position).
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
  const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq);
  const int exponent = (int)((bits >> 52) & 0x7ff) - 1023;
  if (exponent == 1024) return 1;
  if (exponent < -1000 || exponent > 53) return 0;          // nothing, or beyond any use
  const uint64_t mantissa = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  constexpr uint64_t kPerTurn = 11743562013128004906ull;    // 2^66 / (2 pi), rounded
  const uint64_t lo = mantissa * kPerTurn, hi = __umul64hi(mantissa, kPerTurn);
  // the product times 2^(exponent - 52 - 66 + 64)
  const int right = 54 - exponent;
  const uint64_t t = right >= 128 ? 0 : right >= 64 ? hi >> (right - 64) : right == 0 ? lo : (lo >> right) | (hi << (64 - right));
  return (bits >> 63 ? 0 - t : t) & ~1ull;
}

// cosine and sine of `position` steps; NaN for a frequency that is no number.
__device__ __forceinline__ float2 turned(uint64_t step, int position) {
  const uint64_t t = step * (uint64_t)(int64_t)position;
  const float half_turns = step & 1 ? __int_as_float(0x7fffffff) : (float)(int)(t >> 32) * 0x1p-31f;   // [-1, 1)
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

// The two vectors of a lane: byte offsets within the head and how they pair.
// Units 0 .. rot/(2 EPV) - 1 are turned, the others pass through.
template <typename T, bool INTER>
struct Unit {
  static constexpr int EPV = Elt<T>::EPV;
  int off0, off1;     // element offsets of the two vectors
  bool turn;
  int angle;          // index of the unit's first angle
  __device__ __forceinline__ Unit(int u, int rot) {
    const int turned_units = rot / (2 * EPV);
    turn = u < turned_units;
    angle = u * EPV;
    if (INTER || !turn) {
      off0 = u * 2 * EPV;
      off1 = off0 + EPV;
    } else {
      off0 = u * EPV;
      off1 = off0 + rot / 2;
    }
  }
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t swapped(uint64_t a) { return a >> 32 | a << 32; }

// A vector from pairs of fp32 values, rounded to the element type.
template <typename T>
__device__ __forceinline__ uint4 from_pairs(const uint64_t *x) {
  constexpr int NP = Pairs<T>::NP;
  float f[2 * NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) unpair(x[i], f[2 * i], f[2 * i + 1]);
  return Elt<T>::pack(f);
}

// Turn a unit (2 NP pairs of fp32 values: vector 0, then vector 1) by the
// angles at c and s, forwards or back.
template <typename T, bool INTER, bool BACK>
__device__ __forceinline__ void turn(uint64_t *x, const float *c, const float *s) {
  constexpr int NP = Pairs<T>::NP;
  if constexpr (INTER) {
    // a pair is (a, b) itself
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
      const float si = BACK ? -s[i] : s[i];
      x[i] = fma2(x[i], pair(c[i], c[i]), mul2(swapped(x[i]), pair(-si, si)));
    }
  } else {
    // vector 0 holds a, vector 1 b
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint64_t ci = pair(c[2 * i], c[2 * i + 1]);
      const uint64_t up = BACK ? pair(-s[2 * i], -s[2 * i + 1]) : pair(s[2 * i], s[2 * i + 1]);
      const uint64_t down = BACK ? pair(s[2 * i], s[2 * i + 1]) : pair(-s[2 * i], -s[2 * i + 1]);
      const uint64_t a = x[i], b = x[NP + i];
      x[i] = fma2(b, down, mul2(a, ci));
      x[NP + i] = fma2(a, up, mul2(b, ci));
    }
  }
}

// A lane's share of the weight, or ones.
template <typename T>
__device__ __forceinline__ void load_weight(uint64_t *w, const float *src, int off0, int off1) {
  constexpr int NP = Pairs<T>::NP;
#pragma unroll
  for (int j = 0; j < NP; j += 2) {
    const float4 a = src ? ld_f4(src + off0 + 2 * j) : make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 b = src ? ld_f4(src + off1 + 2 * j) : make_float4(1.f, 1.f, 1.f, 1.f);
    w[j] = pair(a.x, a.y);
    w[j + 1] = pair(a.z, a.w);
    w[NP + j] = pair(b.x, b.y);
    w[NP + j + 1] = pair(b.z, b.w);
  }
}

// The frequencies' steps, once per CTA; then each warp forms its rows' angles
// from them.
struct Angles {
  const uint64_t *steps;             // [rot / 2]
  float *c, *s;                      // cosines and sines [rot / 2], the warp's own
  int n;
  __device__ __forceinline__ Angles(char *smem, const double *inv_freq, int rot) {
    n = rot / 2;                     // a multiple of 4
    uint64_t *st = reinterpret_cast<uint64_t *>(smem);
    for (int i = threadIdx.x; i < n; i += kThreads) st[i] = turn_step(inv_freq[i]);
    steps = st;
    c = reinterpret_cast<float *>(st + n) + threadIdx.x / 32 * 2 * n;
    s = c + n;
    __syncthreads();
  }
  __device__ __forceinline__ void form(int position) const {
    __syncwarp();                    // the last row's are read
    for (int i = threadIdx.x % 32; i < n; i += 32) {
      const float2 cs = turned(steps[i], position);
      c[i] = cs.x;
      s[i] = cs.y;
    }
    __syncwarp();
  }
  // A lane's angles (a unit has 2 NP of them), in 16-byte reads.
  template <int N> __device__ __forceinline__ void read(int at, float *cosines, float *sines) const {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(c + at + i), y = *reinterpret_cast<const float4 *>(s + at + i);
      cosines[i] = x.x; cosines[i + 1] = x.y; cosines[i + 2] = x.z; cosines[i + 3] = x.w;
      sines[i] = y.x; sines[i + 1] = y.y; sines[i + 2] = y.z; sines[i + 3] = y.w;
    }
  }
  static size_t bytes(int rot) { return (size_t)(rot / 2) * 8 * (1 + kWarps); }
};

struct HeadParams {
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;       // k_out, v_out: the caches when page > 0
  int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;   // elements from one token row to the next
  const float *wq, *wk;
  const int32_t *positions;          // [rows] or nullptr: the row's index in its sequence
  const double *inv_freq;
  const int32_t *table;              // [B, max_pages]
  int64_t rows, T;
  int Hq, Hk, d, rot;
  int parts, per_part;               // a row's heads (q, then k, then v into a cache) in parts, one per work item
  int64_t num_pages;
  int page, max_pages;
  float eps, inv_d;
};

template <typename T, int TEAM, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kThreads, 2) head_norm_kernel(const HeadParams p) {
  constexpr int E = Elt<T>::EPV, NP = Pairs<T>::NP;
  constexpr int kTeams = 32 / TEAM;              // of a warp
  constexpr int kFlight = 4;                     // heads in flight per team
  extern __shared__ char smem[];
  grid_dependency_wait();
  const Angles ang(smem, p.inv_freq, p.rot);
  const int lane = threadIdx.x % TEAM, team = threadIdx.x % 32 / TEAM;
  const bool active = lane * 2 * E < p.d;
  const Unit<T, INTER> u(lane, p.rot);
  const int64_t items = p.rows * p.parts, stride = (int64_t)gridDim.x * kWarps;
  const int heads = p.Hq + (CACHE ? 2 : 1) * p.Hk;

  for (int64_t item = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; item < items; item += stride) {
    const int64_t row = p.parts == 1 ? item : item / p.parts;
    const int from = p.parts == 1 ? 0 : (int)(item - row * p.parts) * p.per_part, to = min(heads, from + p.per_part);
    const int position = p.positions ? p.positions[row] : (int)(row % p.T);
    // A row without a place in the cache (a negative position, one behind the
    // table, a page outside the pool) is rotated but not stored.
    int64_t slot = -1;
    if (CACHE && position >= 0 && position / p.page < p.max_pages) {
      const int64_t pg = p.table[row / p.T * p.max_pages + position / p.page];
      if (pg >= 0 && pg < p.num_pages) slot = (pg * p.Hk * p.page + position % p.page) * p.d;
    }
    bool formed = false;
    // The queries', then the keys' heads.
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int first = which ? p.Hq : 0, count = which ? p.Hk : p.Hq;
      const int h0 = max(from, first) - first, h1 = min(to, first + count) - first;
      if (h0 >= h1) continue;
      const T *x0 = which ? (const T *)p.k + row * p.k_stride : (const T *)p.q + row * p.q_stride;
      T *y0;
      int64_t step = p.d;                        // from one head of the output to the next
      bool store = true;
      if (!which) y0 = (T *)p.q_out + row * p.qo_stride;
      else if (!CACHE) y0 = (T *)p.k_out + row * p.ko_stride;
      else {
        y0 = (T *)p.k_out + slot;
        step = (int64_t)p.page * p.d;
        store = slot >= 0;
      }
      uint64_t w[2 * NP];
      if (active) load_weight<T>(w, which ? p.wk : p.wq, u.off0, u.off1);
      float c[2 * NP] = {}, sn[2 * NP] = {};     // the lane's angles
      for (int hb = h0; hb < h1; hb += kTeams * kFlight) {
        uint4 va[kFlight], vb[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int h = hb + k * kTeams + team;
          va[k] = vb[k] = make_uint4(0, 0, 0, 0);
          if (active && h < h1) {
            va[k] = *reinterpret_cast<const uint4 *>(x0 + h * p.d + u.off0);
            vb[k] = *reinterpret_cast<const uint4 *>(x0 + h * p.d + u.off1);
          }
        }
        if (!formed) {                           // with the first heads on their way
          ang.form(position);
          formed = true;
        }
        if (hb == h0 && active && u.turn) ang.template read<2 * NP>(u.angle, c, sn);
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int h = hb + k * kTeams + team;
          if (hb + k * kTeams >= h1) break;      // the same for the whole warp
          uint64_t x[2 * NP], sum = 0;
          Pairs<T>::split(va[k], x);
          Pairs<T>::split(vb[k], x + NP);
#pragma unroll
          for (int i = 0; i < 2 * NP; ++i) fma_pair(sum, x[i], x[i]);
          const float ss = team_sum_shfl<TEAM>(pair_sum(sum));
          if (!active || h >= h1 || !store) continue;
          const float rms = rsqrtf(ss * p.inv_d + p.eps);
          const uint64_t rms2 = pair(rms, rms);
#pragma unroll
          for (int i = 0; i < 2 * NP; ++i) x[i] = mul2(mul2(x[i], rms2), w[i]);
          if (u.turn) turn<T, INTER, false>(x, c, sn);
          T *y = y0 + h * step;
          st_vec(y + u.off0, from_pairs<T>(x));
          st_vec(y + u.off1, from_pairs<T>(x + NP));
        }
      }
    }
    if (CACHE && slot >= 0) {
      // the values, as they are
      const int first = p.Hq + p.Hk, h0 = max(from, first) - first, h1 = to - first;
      const T *x0 = (const T *)p.v + row * p.v_stride;
      T *y0 = (T *)p.v_out + slot;
      for (int h = h0 + team; h < h1; h += kTeams) {
        if (!active) continue;
        const uint4 a = *reinterpret_cast<const uint4 *>(x0 + h * p.d + u.off0);
        const uint4 b = *reinterpret_cast<const uint4 *>(x0 + h * p.d + u.off1);
        st_vec(y0 + (int64_t)h * p.page * p.d + u.off0, a);
        st_vec(y0 + (int64_t)h * p.page * p.d + u.off1, b);
      }
    }
  }
}

struct HeadBackwardParams {
  const void *x[2], *g[2];           // q and k: inputs and upstream gradients
  void *dx[2];                       // contiguous
  int64_t stride[2], gstride[2];
  const float *w[2];
  float *partials;                   // [gridDim.x][2][d] or nullptr
  const int32_t *positions;
  const double *inv_freq;
  int64_t rows, T;
  int H[2], d, rot;
  int parts[2], per_part[2];         // a row's heads in parts, one per work item
  float eps, inv_d;
};

template <typename T, int TEAM, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) head_norm_backward_kernel(const HeadBackwardParams p) {
  constexpr int E = Elt<T>::EPV, NP = Pairs<T>::NP;
  constexpr int kTeams = 32 / TEAM;
  constexpr int kFlight = kBackFlight;
  extern __shared__ char smem[];
  grid_dependency_wait();
  const Angles ang(smem, p.inv_freq, p.rot);
  const int lane = threadIdx.x % TEAM, team = threadIdx.x % 32 / TEAM;
  const bool active = lane * 2 * E < p.d;
  const Unit<T, INTER> u(lane, p.rot);
  const int64_t stride = (int64_t)gridDim.x * kWarps;

  // All of the queries' heads, then the keys', so that the sums of one weight
  // are in registers at a time.
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    uint64_t dw[2 * NP], w[2 * NP];
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) dw[i] = 0;
    if (active) load_weight<T>(w, p.w[which], u.off0, u.off1);
    const int parts = p.parts[which], H = p.H[which];
    for (int64_t item = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; item < p.rows * parts; item += stride) {
      const int64_t row = parts == 1 ? item : item / parts;
      const int h0 = parts == 1 ? 0 : (int)(item - row * parts) * p.per_part[which], h1 = min(H, h0 + p.per_part[which]);
      const int position = p.positions ? p.positions[row] : (int)(row % p.T);
      const T *x0 = (const T *)p.x[which] + row * p.stride[which];
      const T *g0 = (const T *)p.g[which] + row * p.gstride[which];
      T *y0 = (T *)p.dx[which] + row * H * p.d;
      for (int hb = h0; hb < h1; hb += kTeams * kFlight) {
        uint4 xa[kFlight], xb[kFlight], ga[kFlight], gb[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int h = hb + k * kTeams + team;
          xa[k] = xb[k] = ga[k] = gb[k] = make_uint4(0, 0, 0, 0);
          if (active && h < h1) {
            xa[k] = *reinterpret_cast<const uint4 *>(x0 + h * p.d + u.off0);
            xb[k] = *reinterpret_cast<const uint4 *>(x0 + h * p.d + u.off1);
            ga[k] = *reinterpret_cast<const uint4 *>(g0 + h * p.d + u.off0);
            gb[k] = *reinterpret_cast<const uint4 *>(g0 + h * p.d + u.off1);
          }
        }
        if (hb == h0) ang.form(position);        // with the first heads on their way
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int h = hb + k * kTeams + team;
          if (hb + k * kTeams >= h1) break;      // the same for the whole warp
          uint64_t x[2 * NP], g[2 * NP], v[2 * NP], sum = 0, dot = 0;
          Pairs<T>::split(xa[k], x);
          Pairs<T>::split(xb[k], x + NP);
          Pairs<T>::split(ga[k], g);
          Pairs<T>::split(gb[k], g + NP);
          if (u.turn && active) {
            float c[2 * NP], sn[2 * NP];
            ang.template read<2 * NP>(u.angle, c, sn);
            turn<T, INTER, true>(g, c, sn);
          }
#pragma unroll
          for (int i = 0; i < 2 * NP; ++i) {
            v[i] = mul2(g[i], w[i]);
            fma_pair(sum, x[i], x[i]);
            fma_pair(dot, v[i], x[i]);
          }
          const bool live = active && h < h1;
          const float ss = team_sum_shfl<TEAM>(live ? pair_sum(sum) : 0.f);
          const float ux = team_sum_shfl<TEAM>(live ? pair_sum(dot) : 0.f);
          if (!live) continue;
          const float r = rsqrtf(ss * p.inv_d + p.eps), rc = -ux * p.inv_d * r * r * r;
          const uint64_t r2 = pair(r, r), rc2 = pair(rc, rc);
#pragma unroll
          for (int i = 0; i < 2 * NP; ++i) {
            fma_pair(dw[i], g[i], mul2(x[i], r2));
            v[i] = fma2(x[i], rc2, mul2(v[i], r2));
          }
          T *y = y0 + h * p.d;
          st_vec(y + u.off0, from_pairs<T>(v));
          st_vec(y + u.off1, from_pairs<T>(v + NP));
        }
      }
    }
    if (!p.partials) continue;
    // The CTA's sums: over the teams of a warp by shuffles, over the warps
    // through shared memory in a fixed order (reproducible).
    float *red = reinterpret_cast<float *>(smem) + p.rot / 2 * 2 * (1 + kWarps);   // [warps][d], behind the angles
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
      float lo, hi;
      unpair(dw[i], lo, hi);
#pragma unroll
      for (int o = TEAM; o < 32; o <<= 1) {
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
        hi += __shfl_xor_sync(0xffffffffu, hi, o);
      }
      if (team == 0 && active) {
        float *at = red + threadIdx.x / 32 * p.d + (i < NP ? u.off0 + 2 * i : u.off1 + 2 * (i - NP));
        at[0] = lo;
        at[1] = hi;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += red[k * p.d + i];
      p.partials[((int64_t)blockIdx.x * 2 + which) * p.d + i] = s;
    }
    __syncthreads();
  }
}

// The weights' gradients: the CTAs' sums added in a fixed order, 32 lanes of
// a warp taking every 32nd CTA.  One warp per element of the two [d] rows.
__global__ void __launch_bounds__(256) head_norm_weights_kernel(const float *partials, int ctas, int d, float *dwq,
                                                                float *dwk) {
  grid_dependency_wait();
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x % 32;
  if (warp >= 2 * d) return;
  float s = 0.f;
  for (int c = lane; c < ctas; c += 32) s += partials[(int64_t)c * 2 * d + warp];
  s = team_sum_shfl<32>(s);
  float *out = warp < d ? dwq : dwk;
  if (lane == 0 && out) out[warp % d] = s;
}

// Parts that a row's heads are cut into so that there are about `want` work
// items, each of a multiple of `round` heads.
int row_parts(int64_t rows, int heads, int round, int64_t want, int &per_part) {
  int64_t parts = (want + rows - 1) / rows;
  const int most = (heads + round - 1) / round;
  if (parts > most) parts = most;
  per_part = (int)((heads + parts - 1) / parts + round - 1) / round * round;
  return (heads + per_part - 1) / per_part;
}

// Call f with the element type, the lanes per head and the pairing as types.
template <typename F>
cudaError_t dispatch(int dtype, int d, int interleaved, F f) {
  const int units = d / (dtype == ATTNRES_BF16 ? 16 : 8);
  auto with_team = [&](auto elt, auto inter) -> cudaError_t {
    if (units <= 4) return f(elt, std::integral_constant<int, 4>{}, inter);
    if (units <= 8) return f(elt, std::integral_constant<int, 8>{}, inter);
    if (units <= 16) return f(elt, std::integral_constant<int, 16>{}, inter);
    return f(elt, std::integral_constant<int, 32>{}, inter);
  };
  auto with_pairs = [&](auto elt) -> cudaError_t {
    return interleaved ? with_team(elt, std::true_type{}) : with_team(elt, std::false_type{});
  };
  return dtype == ATTNRES_BF16 ? with_pairs(__nv_bfloat16{}) : with_pairs(float{});
}

}  // namespace

bool head_norm_supported(int64_t d, int dtype) {
  const int pair = dtype == ATTNRES_BF16 ? 16 : 8;
  return d >= pair && d <= 32 * pair && d % pair == 0;
}

cudaError_t launch_head_norm(const HeadNormArgs &a) {
  HeadParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v;
  p.q_out = a.q_out; p.k_out = a.k_out; p.v_out = a.v_cache;
  p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
  p.qo_stride = a.q_out_stride; p.ko_stride = a.k_out_stride;
  p.wq = a.q_weight; p.wk = a.k_weight;
  p.positions = a.positions; p.inv_freq = a.inv_freq; p.table = a.page_table;
  p.rows = a.rows; p.T = a.T; p.Hq = a.Hq; p.Hk = a.Hk; p.d = a.d; p.rot = a.rot;
  p.num_pages = a.num_pages; p.page = a.page_size; p.max_pages = a.max_pages;
  p.eps = a.eps; p.inv_d = 1.f / (float)a.d;
  const bool cache = a.page_size > 0;
  const int sms = sm_count();
  return dispatch(a.dtype, a.d, a.interleaved, [&](auto elt, auto team, auto inter) -> cudaError_t {
    using T = decltype(elt);
    constexpr int TEAM = decltype(team)::value;
    constexpr bool INTER = decltype(inter)::value;
    // A row per work item, cut into parts of no less than one round of a
    // warp's teams where the rows alone would not give every SM eight warps.
    // Measured, 32 + 8 heads of 128, cut against whole rows: 1 to 64 rows 4.0 against 7.4
    // to 9.0 us, 512 5.8 against 8.3; for 16 warps per SM 512 rows take 6.9, 2048 12.3
    // against 10.2.
    const int heads = a.Hq + (cache ? 2 : 1) * a.Hk;
    p.parts = row_parts(a.rows, heads, 32 / TEAM, 8 * (int64_t)sms, p.per_part);
    const int64_t ctas = (a.rows * p.parts + kWarps - 1) / kWarps, most = (int64_t)sms * 8;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    const size_t smem = Angles::bytes(a.rot);
    return cache ? launch_dependent(head_norm_kernel<T, TEAM, INTER, true>, grid, dim3(kThreads), smem, a.stream, p)
                 : launch_dependent(head_norm_kernel<T, TEAM, INTER, false>, grid, dim3(kThreads), smem, a.stream, p);
  });
}

int head_norm_backward_ctas() { return 2 * sm_count(); }

cudaError_t launch_head_norm_backward(const HeadNormBackwardArgs &a) {
  HeadBackwardParams p{};
  p.x[0] = a.q; p.x[1] = a.k; p.g[0] = a.grad_q; p.g[1] = a.grad_k;
  p.dx[0] = a.dq; p.dx[1] = a.dk;
  p.stride[0] = a.q_stride; p.stride[1] = a.k_stride;
  p.gstride[0] = a.gq_stride; p.gstride[1] = a.gk_stride;
  p.w[0] = a.q_weight; p.w[1] = a.k_weight;
  p.partials = a.workspace;
  p.positions = a.positions; p.inv_freq = a.inv_freq;
  p.rows = a.rows; p.T = a.T; p.H[0] = a.Hq; p.H[1] = a.Hk; p.d = a.d; p.rot = a.rot;
  p.eps = a.eps; p.inv_d = 1.f / (float)a.d;
  const int limit = a.workspace && a.workspace_rows / 2 < head_norm_backward_ctas() ? (int)(a.workspace_rows / 2)
                                                                                : head_norm_backward_ctas();
  int ctas = 0;
  cudaError_t e = dispatch(a.dtype, a.d, a.interleaved, [&](auto elt, auto team, auto inter) -> cudaError_t {
    using T = decltype(elt);
    constexpr int TEAM = decltype(team)::value;
    // The parts with the least work for the busiest warp.  An item costs its
    // heads, in whole rounds of the warp's teams (kBackFlight heads each in
    // flight), and the row's angles, worth six heads.  Against two items per
    // warp: 1024 rows of 32 + 8 heads 14.0 against 15.4 us, 2048 18.3 against 19.7,
    // 512 and 3000 (cut into four and two) the same.
    int64_t most = 0;
    for (int i = 0; i < 2; ++i) {
      const int round = kBackFlight * (32 / TEAM), all = (p.H[i] + round - 1) / round;
      const int64_t warps = (int64_t)limit * kWarps;
      int64_t least = INT64_MAX;
      for (int n = 1; n <= all; ++n) {
        const int per = (all + n - 1) / n * round, parts = (p.H[i] + per - 1) / per;
        const int64_t cost = (a.rows * parts + warps - 1) / warps * (per + 6);
        if (cost < least) {
          least = cost;
          p.parts[i] = parts;
          p.per_part[i] = per;
        }
      }
      if (a.rows * p.parts[i] > most) most = a.rows * p.parts[i];
    }
    const int64_t want = (most + kWarps - 1) / kWarps;
    ctas = (int)(want < limit ? want : limit);
    const size_t smem = Angles::bytes(a.rot) + (size_t)kWarps * a.d * sizeof(float);
    return launch_dependent(head_norm_backward_kernel<T, TEAM, decltype(inter)::value>, dim3((unsigned)ctas),
                            dim3(kThreads), smem, a.stream, p);
  });
  if (e != cudaSuccess || !a.workspace) return e;
  return launch_dependent(head_norm_weights_kernel, dim3((unsigned)((2 * a.d + 7) / 8)), dim3(256), 0, a.stream,
                          (const float *)a.workspace, ctas, a.d, a.grad_q_weight, a.grad_k_weight);
}

}  // namespace attnres
