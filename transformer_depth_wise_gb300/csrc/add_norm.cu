// add_norm.cu -- RMS norm with the residual's addition, its form with an
// output in 8 bits, and its backward pass.
//
// Per token row, with s = x + residual in fp32:  sum = s rounded once,
// y = s r w, r = (mean s^2 + eps)^(-1/2), rounded once to the row's type, or
// in e4m3 with one fp32 scale per group of a row's elements (or per row):
// scale = max|y| / 448 over the group, y8 = y / scale (as products with the
// rounded reciprocals of 448 and of the scale: a division per element would
// change only values within two roundings of a tie).
// Backward at the stored sum s:  u = grad_y w,  dx = grad_sum + r (u - s r^2
// mean(u s)),  grad_weight = sum over rows of grad_y s r.
//
// Memory binds: every tensor passes once.  A thread holds the same vectors of
// each of its team's rows (a CTA per row, or 8 or 32 lanes for narrow rows);
// the next row's loads are issued before the present row's reduction, so that
// the reduction's barriers leave no gap in the loads.
//
// Measured on GB300, bf16: 32768 rows of 7168 with a scale per 128 elements, 261
// us (6.3 TB/s; 364 without the loads ahead, 370 with three CTAs per SM, 309 with
// the per-vector address arithmetic and reductions that bound an earlier form,
// 38 instructions an element); 256 rows with a scale per row, 6 us; backward over
// 16384 rows of 4096, 81 us (6.6 TB/s) and 5 us for the weight's sums.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace attnres {
namespace {

constexpr float kTop = 448.f;              // the largest e4m3 value
constexpr float kLeast = 0x1p-126f;        // the smallest scale: its reciprocal is finite

enum Mode { kPlain, kGroups, kRow8 };      // y in the row's type, in e4m3 by groups, in e4m3 by rows

// Four values in e4m3, to nearest even, held within +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3(uint64_t a, uint64_t b) {
  float f[4];
  unpair(a, f[0], f[1]);
  unpair(b, f[2], f[3]);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
  return (uint32_t)hi << 16 | lo;
}

// The largest magnitude of a pair and of what is there; NaN stays NaN.
__device__ __forceinline__ float top_of(uint64_t x, float top) {
  float lo, hi;
  unpair(x, lo, hi);
  asm("max.NaN.abs.f32 %0, %1, %2, %0;" : "+f"(top) : "f"(lo), "f"(hi));
  return top;
}
__device__ __forceinline__ float larger(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}

// The scale of a group with this largest magnitude (a NaN gives NaN): within a
// rounding of the quotient, and its reciprocal is what y is multiplied by.
__device__ __forceinline__ float scale_of(float top) {
  const float s = top * (1.f / kTop);
  return s < kLeast ? kLeast : s;
}

// The sum over a CTA of at most 16 warps, by warp and then over the warps'
// sums; `red` [2][16], the half taken in turn so that one barrier is enough.
__device__ __forceinline__ float cta_total(float v, float *red, int parity) {
  v = team_sum_shfl<32>(v);
  float *slot = red + parity * 16;
  if (threadIdx.x % 32 == 0) slot[threadIdx.x / 32] = v;
  __syncthreads();
  v = threadIdx.x % 32 < blockDim.x / 32 ? slot[threadIdx.x % 32] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

// The same for two values; `red` [2][2][16].
__device__ __forceinline__ void cta_totals(float &a, float &b, float *red, int parity) {
  a = team_sum_shfl<32>(a);
  b = team_sum_shfl<32>(b);
  float *slot = red + parity * 32;
  const int lane = threadIdx.x % 32;
  if (lane == 0) {
    slot[threadIdx.x / 32] = a;
    slot[16 + threadIdx.x / 32] = b;
  }
  __syncthreads();
  float v = lane % 16 < blockDim.x / 32 ? slot[lane] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  a = __shfl_sync(0xffffffffu, v, 0);
  b = __shfl_sync(0xffffffffu, v, 16);
}

template <typename T>
__device__ __forceinline__ void load_weight(uint64_t *w, const float *src) {
#pragma unroll
  for (int i = 0; i < Pairs<T>::NP; i += 2) {
    const float4 a = src ? ld_f4(src + 2 * i) : make_float4(1.f, 1.f, 1.f, 1.f);
    w[i] = pair(a.x, a.y);
    w[i + 1] = pair(a.z, a.w);
  }
}

struct AddNormParams {
  const void *x, *residual;                // residual: nullptr for none
  void *sum, *y;                           // sum: nullptr if not wanted; y: the row's type or bytes
  float *scales;                           // [rows, D / group] or [rows]
  const float *w;                          // [D] or nullptr
  int64_t rows;
  int nvec, lanes;                         // vectors of a row; lanes of a group (kGroups)
  float inv_D, eps;
};

// Eight (bf16) or four (fp32) values times `inv` in e4m3.
template <int NP>
__device__ __forceinline__ void store_e4m3(char *y, const uint64_t *v, float inv) {
  const uint64_t inv2 = pair(inv, inv);
  uint32_t q[NP / 2];
#pragma unroll
  for (int i = 0; i < NP; i += 2) q[i / 2] = to_e4m3(mul2(v[i], inv2), mul2(v[i + 1], inv2));
  if constexpr (NP == 4) *reinterpret_cast<uint2 *>(y) = make_uint2(q[0], q[1]);
  else *reinterpret_cast<uint32_t *>(y) = q[0];
}

template <typename T, int VPT, int TEAM, int MODE>
__global__ void __launch_bounds__(TEAM ? 256 : 512) add_norm_kernel(const AddNormParams p) {
  constexpr int EPV = Elt<T>::EPV, NP = Pairs<T>::NP;
  __shared__ float red[TEAM ? 1 : 32], top_red[TEAM || MODE != kRow8 ? 1 : 32];
  grid_dependency_wait();
  const int tpr = TEAM ? TEAM : blockDim.x, lt = TEAM ? threadIdx.x % TEAM : threadIdx.x;
  const int teams = TEAM ? blockDim.x / TEAM : 1, team = TEAM ? threadIdx.x / TEAM : 0;
  // the thread's first vector of a row, and from one row of the team to its next
  const int64_t start = (int64_t)blockIdx.x * teams + team, rows = p.rows, turn = (int64_t)gridDim.x * teams;
  const int64_t step = turn * p.nvec * 16;
  const char *x = (const char *)p.x + (start * p.nvec + lt) * 16;
  const char *res = p.residual ? (const char *)p.residual + (start * p.nvec + lt) * 16 : nullptr;
  char *sum = p.sum ? (char *)p.sum + (start * p.nvec + lt) * 16 : nullptr;
  char *y = (char *)p.y + (start * p.nvec + lt) * (MODE == kPlain ? 16 : EPV);
  float *scales = MODE == kGroups ? p.scales + start * (p.nvec / p.lanes) + lt / p.lanes : p.scales + start;
  const float *w = p.w ? p.w + lt * EPV : nullptr;
  bool in[VPT];                            // vectors that a row has
#pragma unroll
  for (int k = 0; k < VPT; ++k) in[k] = lt + k * tpr < p.nvec;
  uint4 xv[VPT], rv[VPT];
  auto load = [&](bool live) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      xv[k] = rv[k] = make_uint4(0, 0, 0, 0);
      if (live && in[k]) {
        xv[k] = ld_once(x + k * tpr * 16);
        if (res) rv[k] = ld_once(res + k * tpr * 16);
      }
    }
  };
  int parity = 0;
  load(start < rows);
  // a team's last turns may be idle ones that its warp's other teams need
  for (int64_t row = start; row - team < rows; row += turn) {
    const bool live = TEAM == 0 || row < rows;
    uint64_t s[VPT * NP], sq = 0;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      Pairs<T>::split(xv[k], s + k * NP);
      if (res) {
        uint64_t b[NP];
        Pairs<T>::split(rv[k], b);
#pragma unroll
        for (int i = 0; i < NP; ++i) s[k * NP + i] = add2(s[k * NP + i], b[i]);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) fma_pair(sq, s[k * NP + i], s[k * NP + i]);
    }
    x += step;
    if (res) res += step;
    load(row + turn < rows);
    float ss = pair_sum(sq);
    if (TEAM) ss = team_sum_shfl<TEAM ? TEAM : 1>(ss);
    else ss = cta_total(ss, red, parity);
    const float r = rsqrtf(fmaf(ss, p.inv_D, p.eps));
    const uint64_t r2 = pair(r, r);
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const bool here = live && in[k];
      uint64_t *v = s + k * NP;
      if (here) {
        if (sum) st_stream(sum + k * tpr * 16, from_pairs<T>(v));
        uint64_t c[NP];
        load_weight<T>(c, w ? w + k * tpr * EPV : nullptr);
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = mul2(mul2(v[i], r2), c[i]);
        if (MODE == kPlain) st_vec(y + k * tpr * 16, from_pairs<T>(v));
      }
      if constexpr (MODE != kPlain) {
        float m = 0.f;
        if (here) {
#pragma unroll
          for (int i = 0; i < NP; ++i) m = top_of(v[i], m);
        }
        if constexpr (MODE == kRow8) {
          top = larger(top, m);
        } else {
          for (int o = p.lanes / 2; o > 0; o >>= 1) m = larger(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (here) {
            const float scale = scale_of(m);
            store_e4m3<NP>(y + k * tpr * EPV, v, 1.f / scale);
            if (lt % p.lanes == 0) scales[k * (tpr / p.lanes)] = scale;
          }
        }
      }
    }
    if constexpr (MODE == kRow8) {
#pragma unroll
      for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (!TEAM) {
        float *slot = top_red + parity * 16;
        if (threadIdx.x % 32 == 0) slot[threadIdx.x / 32] = top;
        __syncthreads();
        top = threadIdx.x % 32 < blockDim.x / 32 ? slot[threadIdx.x % 32] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = __shfl_sync(0xffffffffu, top, 0);
      }
      const float scale = scale_of(top), inv = 1.f / scale;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (live && in[k]) store_e4m3<NP>(y + k * tpr * EPV, s + k * NP, inv);
      if (live && lt == 0) *scales = scale;
    }
    if (sum) sum += step;
    y += MODE == kPlain ? step : step / 16 * EPV;
    if (MODE != kPlain) scales += MODE == kGroups ? turn * (p.nvec / p.lanes) : turn;
    parity ^= 1;
  }
}

struct AddNormBackwardParams {
  const void *s, *gy, *gs;                 // gs: nullptr for none
  void *dx;
  const float *w;                          // [D] or nullptr
  float *partials;                         // [gridDim.x][D] or nullptr
  int64_t rows;
  int nvec;
  float inv_D, eps;
};

template <typename T, int VPT, int TEAM>
__global__ void __launch_bounds__(TEAM ? 256 : 512) add_norm_backward_kernel(const AddNormBackwardParams p) {
  constexpr int EPV = Elt<T>::EPV, NP = Pairs<T>::NP;
  __shared__ float red[TEAM ? 1 : 64];
  extern __shared__ float team_dw[];       // TEAM: [teams][VPT * TEAM * EPV]
  grid_dependency_wait();
  const int tpr = TEAM ? TEAM : blockDim.x, lt = TEAM ? threadIdx.x % TEAM : threadIdx.x;
  const int teams = TEAM ? blockDim.x / TEAM : 1, team = TEAM ? threadIdx.x / TEAM : 0;
  const int64_t start = (int64_t)blockIdx.x * teams + team, rows = p.rows, turn = (int64_t)gridDim.x * teams;
  const int64_t step = turn * p.nvec * 16, at = (start * p.nvec + lt) * 16;
  const char *sp = (const char *)p.s + at, *gp = (const char *)p.gy + at;
  const char *rp = p.gs ? (const char *)p.gs + at : nullptr;
  char *out = (char *)p.dx + at;
  bool in[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) in[k] = lt + k * tpr < p.nvec;
  uint4 sv[VPT], gv[VPT], rv[VPT];
  auto load = [&](bool live) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      sv[k] = gv[k] = rv[k] = make_uint4(0, 0, 0, 0);
      if (live && in[k]) {
        sv[k] = ld_once(sp + k * tpr * 16);
        gv[k] = ld_once(gp + k * tpr * 16);
        if (rp) rv[k] = ld_once(rp + k * tpr * 16);
      }
    }
  };
  uint64_t dw[VPT * NP], w[VPT * NP];
#pragma unroll
  for (int i = 0; i < VPT * NP; ++i) dw[i] = w[i] = 0;
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    if (in[k]) load_weight<T>(w + k * NP, p.w ? p.w + (lt + k * tpr) * EPV : nullptr);
  int parity = 0;
  load(start < rows);
  for (int64_t row = start; row - team < rows; row += turn, out += step) {
    uint64_t s[VPT * NP], g[VPT * NP], sq = 0, dot = 0;
    uint4 gs[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      Pairs<T>::split(sv[k], s + k * NP);
      Pairs<T>::split(gv[k], g + k * NP);
      gs[k] = rv[k];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint64_t a = s[k * NP + i];
        fma_pair(sq, a, a);
        fma_pair(dot, mul2(g[k * NP + i], w[k * NP + i]), a);
      }
    }
    sp += step;
    gp += step;
    if (rp) rp += step;
    load(row + turn < rows);
    float ss = pair_sum(sq), us = pair_sum(dot);
    if (TEAM) {
      ss = team_sum_shfl<TEAM ? TEAM : 1>(ss);
      us = team_sum_shfl<TEAM ? TEAM : 1>(us);
    } else {
      cta_totals(ss, us, red, parity);
      parity ^= 1;
    }
    if (TEAM && row >= rows) continue;
    const float r = rsqrtf(fmaf(ss, p.inv_D, p.eps)), rc = -us * p.inv_D * r * r * r;
    const uint64_t r2 = pair(r, r), rc2 = pair(rc, rc);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (!in[k]) continue;
      uint64_t b[NP];
      Pairs<T>::split(gs[k], b);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint64_t a = s[k * NP + i], gr = mul2(g[k * NP + i], r2);
        fma_pair(dw[k * NP + i], gr, a);
        b[i] = fma2(a, rc2, fma2(gr, w[k * NP + i], b[i]));
      }
      st_stream(out + k * tpr * 16, from_pairs<T>(b));
    }
  }
  if (!p.partials) return;
  float *sums = p.partials + (int64_t)blockIdx.x * p.nvec * EPV;
  if (TEAM) {
    // the teams' sums, in a fixed order
    const int D = p.nvec * EPV;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int j = lt + k * tpr;
      if (j >= p.nvec) continue;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        *reinterpret_cast<uint64_t *>(team_dw + team * D + j * EPV + 2 * i) = dw[k * NP + i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
      float sum = 0.f;
      for (int t = 0; t < teams; ++t) sum += team_dw[t * D + i];
      sums[i] = sum;
    }
  } else {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int j = lt + k * tpr;
      if (j >= p.nvec) continue;
#pragma unroll
      for (int i = 0; i < NP; i += 2) {
        float4 f;
        unpair(dw[k * NP + i], f.x, f.y);
        unpair(dw[k * NP + i + 1], f.z, f.w);
        *reinterpret_cast<float4 *>(sums + (int64_t)j * EPV + 2 * i) = f;
      }
    }
  }
}

// The weight's gradient: the CTAs' sums added in a fixed order, 16 strands of
// every 16th CTA per column, 32 columns per CTA.
constexpr int kStrands = 16;
__global__ void __launch_bounds__(32 * kStrands) add_norm_weight_kernel(const float *partials, int ctas, int D, float *dw) {
  __shared__ float red[kStrands][32];
  grid_dependency_wait();
  const int col = blockIdx.x * 32 + threadIdx.x % 32, strand = threadIdx.x / 32;
  float s = 0.f;
  if (col < D) {
#pragma unroll 8
    for (int c = strand; c < ctas; c += kStrands) s += partials[(int64_t)c * D + col];
  }
  red[strand][threadIdx.x % 32] = s;
  __syncthreads();
  if (strand == 0 && col < D) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kStrands; ++k) s += red[k][threadIdx.x];
    dw[col] = s;
  }
}

// Most shared memory of the backward's teams: 32 rows of 128 elements, 8 of 512.
constexpr size_t kTeamBytes = 16384;

// Lanes of a row (0: a CTA's), vectors per thread and the CTA's threads for
// rows of nvec vectors; `whole`: no less than a warp per row.
struct RowShape {
  int team, vpt, threads;
};
RowShape shape_of(int nvec, bool whole) {
  if (nvec <= 16 && !whole) return {8, 2, 256};
  if (nvec <= 64) return {32, 2, 256};
  const int vpt = nvec <= 1024 ? 2 : 4;
  return {0, vpt, ((nvec + vpt - 1) / vpt + 31) / 32 * 32};
}

// CTAs of `kern` that an SM holds (with the most shared memory it takes),
// asked once per device and CTA size.
template <auto kern>
int resident(int threads, size_t smem) {
  static Kept kept[16][17];
  int dev = 0, n = 1;
  cudaGetDevice(&dev);
  const cudaError_t e = kept[dev & 15][threads / 32].get(
      n, [&](int *v) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kern, threads, smem); });
  return e == cudaSuccess ? n : 1;
}

// Call f with the vectors per thread and the lanes of a row as types.
template <bool WHOLE, typename F>
cudaError_t with_shape(const RowShape &s, F f) {
  using I2 = std::integral_constant<int, 2>;
  if constexpr (!WHOLE)
    if (s.team == 8) return f(I2{}, std::integral_constant<int, 8>{});
  if (s.team == 32) return f(I2{}, std::integral_constant<int, 32>{});
  if (s.vpt == 2) return f(I2{}, std::integral_constant<int, 0>{});
  return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 0>{});
}

template <typename T, int MODE>
cudaError_t forward(const AddNormArgs &a, const AddNormParams &p) {
  const RowShape s = shape_of(p.nvec, MODE != kPlain);
  return with_shape<MODE != kPlain>(s, [&](auto vpt, auto team) -> cudaError_t {
    constexpr int TEAM = decltype(team)::value;
    constexpr auto kern = add_norm_kernel<T, decltype(vpt)::value, TEAM, MODE>;
    const int teams = TEAM ? s.threads / (TEAM ? TEAM : 1) : 1;
    const int64_t steps = (p.rows + teams - 1) / teams, most = (int64_t)resident<kern>(s.threads, 0) * sm_count();
    return launch_dependent(kern, dim3((unsigned)(steps < most ? steps : most)), dim3(s.threads), 0, a.stream, p);
  });
}

template <typename T>
cudaError_t forward(const AddNormArgs &a, const AddNormParams &p) {
  return !a.bits8 ? forward<T, kPlain>(a, p) : a.group ? forward<T, kGroups>(a, p) : forward<T, kRow8>(a, p);
}

int elements(int dtype) { return dtype == ATTNRES_BF16 ? 8 : 4; }

}  // namespace

bool add_norm_supported(int64_t D, int dtype) { return D / elements(dtype) <= 2048; }

cudaError_t launch_add_norm(const AddNormArgs &a) {
  AddNormParams p{};
  p.x = a.x; p.residual = a.residual; p.sum = a.sum_out; p.y = a.y; p.scales = a.scales; p.w = a.weight;
  p.rows = a.rows; p.nvec = a.D / elements(a.dtype); p.lanes = a.group / elements(a.dtype);
  p.inv_D = 1.f / (float)a.D; p.eps = a.eps;
  return a.dtype == ATTNRES_BF16 ? forward<__nv_bfloat16>(a, p) : forward<float>(a, p);
}

// Each CTA leaves one row of partial sums.
int add_norm_backward_ctas() { return 4 * sm_count(); }

cudaError_t launch_add_norm_backward(const AddNormBackwardArgs &a) {
  AddNormBackwardParams p{};
  p.s = a.s; p.gy = a.grad_y; p.gs = a.grad_sum; p.dx = a.dx; p.w = a.weight; p.partials = a.workspace;
  p.rows = a.rows; p.nvec = a.D / elements(a.dtype); p.inv_D = 1.f / (float)a.D; p.eps = a.eps;
  const RowShape s = shape_of(p.nvec, false);
  int ctas = 0;
  auto go = [&](auto elt) -> cudaError_t {
    using T = decltype(elt);
    return with_shape<false>(s, [&](auto vpt, auto team) -> cudaError_t {
      constexpr int TEAM = decltype(team)::value;
      constexpr auto kern = add_norm_backward_kernel<T, decltype(vpt)::value, TEAM>;
      const int teams = TEAM ? s.threads / (TEAM ? TEAM : 1) : 1;
      const size_t smem = TEAM && p.partials ? (size_t)teams * a.D * sizeof(float) : 0;
      int64_t most = (int64_t)resident<kern>(s.threads, TEAM ? kTeamBytes : 0) * sm_count();
      if (most > add_norm_backward_ctas()) most = add_norm_backward_ctas();
      if (p.partials && most > a.workspace_rows) most = a.workspace_rows;
      const int64_t steps = (p.rows + teams - 1) / teams;
      ctas = (int)(steps < most ? steps : most);
      return launch_dependent(kern, dim3((unsigned)ctas), dim3(s.threads), smem, a.stream, p);
    });
  };
  cudaError_t e = a.dtype == ATTNRES_BF16 ? go(__nv_bfloat16{}) : go(float{});
  if (e != cudaSuccess || !a.workspace) return e;
  return launch_dependent(add_norm_weight_kernel, dim3((unsigned)((a.D + 31) / 32)), dim3(32 * kStrands), 0, a.stream,
                          (const float *)a.workspace, ctas, a.D, a.grad_weight);
}

}  // namespace attnres
