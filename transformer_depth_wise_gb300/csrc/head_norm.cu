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
// no exchange and the norm one shuffle reduction.  A CTA takes a few token
// rows at a time: its threads first form the rows' angles once in shared
// memory (one cosine and sine per token and pair instead of one per head),
// with the first heads' loads already in flight.
//
// Angles.  A frequency is kept as a 64-bit fraction of a turn per position,
// and position * step wraps modulo one turn exactly, so far positions lose
// nothing: the angle is off by the rounding of inv_freq / 2 pi in 64 bits and
// by 2^-25 of half a turn when its upper 32 bits become an fp32 argument.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace attnres {
namespace {

constexpr int kThreads = 256;
constexpr double kInvTwoPi = 0.15915494309189533577;

// inv_freq (radians per position) as 2^-64ths of a turn per position.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
  double turns = inv_freq * kInvTwoPi;
  turns -= floor(turns);                       // in [0, 1]: 1 only by rounding of a tiny negative
  return turns < 1.0 ? (uint64_t)(turns * 18446744073709551616.0) : 0ull;
}

// cosine and sine of `position` steps.
__device__ __forceinline__ float2 turned(uint64_t step, int position) {
  const uint64_t t = step * (uint64_t)(int64_t)position;
  const float half_turns = (float)(int)(t >> 32) * 0x1p-31f;   // [-1, 1)
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

// Turn the pairs of x (2 EPV elements: vector 0 then vector 1) by the angles
// in cs, forwards (dir = 1) or back (-1).
template <typename T, bool INTER>
__device__ __forceinline__ void turn(float *x, const float2 *cs, float dir) {
  constexpr int E = Elt<T>::EPV;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float c = cs[i].x, s = cs[i].y * dir;
    const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : i + E;
    const float xa = x[a], xb = x[b];
    x[a] = xa * c - xb * s;
    x[b] = xb * c + xa * s;
  }
}

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
  int H;                             // heads a token has in this pass (q, k and, into a cache, v)
  int R;                             // rows per CTA and pass
  int head_parts, heads_per_part;    // a token's heads over gridDim.y CTAs
  int64_t num_pages;
  int page, max_pages;
  float eps, inv_d;
};

// Rows' angles into shared memory: thread i forms angle i % nang of row
// i / nang.  Also the rows' cache slots (-1: none).
struct RowAngles {
  int nang, row, angle;
  uint64_t step;
  __device__ __forceinline__ RowAngles(const double *inv_freq, int rot) {
    nang = rot / 2;
    row = nang ? threadIdx.x / nang : 0;
    angle = nang ? threadIdx.x % nang : 0;
    step = nang ? turn_step(inv_freq[angle]) : 0;
  }
  __device__ __forceinline__ void form(float2 *cs, const int32_t *positions, int64_t row0, int R, int64_t rows,
                                       int64_t T) const {
    if (nang == 0) return;
    const int per = kThreads / nang;             // rows formed at once (rot <= 512: at least one)
    if (row >= per) return;
    for (int r = row; r < R; r += per) {
      const int64_t t = row0 + r;
      if (t < rows) cs[r * nang + angle] = turned(step, positions ? positions[t] : (int)(t % T));
    }
  }
};

template <typename T, int TEAM, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(const HeadParams p) {
  constexpr int E = Elt<T>::EPV;
  constexpr int kTeams = kThreads / TEAM;
  constexpr int UNROLL = 2;                      // heads in flight per team
  extern __shared__ char smem[];
  float2 *cs = reinterpret_cast<float2 *>(smem);                          // [R][rot / 2]
  int64_t *slot = reinterpret_cast<int64_t *>(cs + p.R * (p.rot / 2));    // [R]: the row's first cache element
  grid_dependency_wait();
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const bool active = lane * 2 * E < p.d;
  const Unit<T, INTER> u(lane, p.rot);
  const RowAngles ang(p.inv_freq, p.rot);
  const int h0 = blockIdx.y * p.heads_per_part, h1 = min(p.H, h0 + p.heads_per_part), nh = h1 - h0;

  for (int64_t row0 = (int64_t)blockIdx.x * p.R; row0 < p.rows; row0 += (int64_t)gridDim.x * p.R) {
    const int nrow = (int)min((int64_t)p.R, p.rows - row0);
    const int units = nrow * nh;
    uint4 va[UNROLL], vb[UNROLL];
    auto load = [&](int i, int k) {
      const int r = i / nh, h = h0 + i % nh;
      const int64_t row = row0 + r;
      const T *x;
      if (h < p.Hq) x = (const T *)p.q + row * p.q_stride + (int64_t)h * p.d;
      else if (!CACHE || h < p.Hq + p.Hk) x = (const T *)p.k + row * p.k_stride + (int64_t)(h - p.Hq) * p.d;
      else x = (const T *)p.v + row * p.v_stride + (int64_t)(h - p.Hq - p.Hk) * p.d;
      va[k] = *reinterpret_cast<const uint4 *>(x + u.off0);
      vb[k] = *reinterpret_cast<const uint4 *>(x + u.off1);
    };
#pragma unroll
    for (int k = 0; k < UNROLL; ++k)
      if (active && team + k * kTeams < units) load(team + k * kTeams, k);
    ang.form(cs, p.positions, row0, nrow, p.rows, p.T);
    if (CACHE && threadIdx.x < nrow) {
      // A row without a place in the cache (a negative position, one behind
      // the table, a page outside the pool) is rotated but not stored.
      const int64_t row = row0 + threadIdx.x;
      const int pos = p.positions ? p.positions[row] : (int)(row % p.T);
      int64_t s = -1;
      if (pos >= 0 && pos / p.page < p.max_pages) {
        const int64_t pg = p.table[(row / p.T) * p.max_pages + pos / p.page];
        if (pg >= 0 && pg < p.num_pages) s = (pg * p.Hk * p.page + pos % p.page) * p.d;
      }
      slot[threadIdx.x] = s;
    }
    __syncthreads();
    for (int i0 = 0; i0 < units; i0 += kTeams * UNROLL) {
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) {
        const int i = i0 + k * kTeams + team;
        const bool live = i < units;               // the same for a whole team
        const int r = live ? i / nh : 0, h = h0 + (live ? i % nh : 0);
        const bool copy = CACHE && h >= p.Hq + p.Hk;
        float x[2 * E];
        float ss = 0.f;
        if (active && live) {
          Elt<T>::unpack(va[k], x);
          Elt<T>::unpack(vb[k], x + E);
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) ss = fmaf(x[e], x[e], ss);
        }
        ss = team_sum_shfl<TEAM>(ss);
        if (!active || !live) continue;
        const int64_t row = row0 + r;
        T *y;
        if (h < p.Hq) y = (T *)p.q_out + row * p.qo_stride + (int64_t)h * p.d;
        else if (!CACHE) y = (T *)p.k_out + row * p.ko_stride + (int64_t)(h - p.Hq) * p.d;
        else {
          if (slot[r] < 0) continue;
          y = (T *)(copy ? p.v_out : p.k_out) + slot[r] + (int64_t)((h - p.Hq) % p.Hk) * p.page * p.d;
        }
        if (copy) {
          st_vec(y + u.off0, va[k]);
          st_vec(y + u.off1, vb[k]);
          continue;
        }
        const float rms = rsqrtf(ss * p.inv_d + p.eps);
        const float *w = h < p.Hq ? p.wq : p.wk;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) x[e] *= rms;
        if (w) {
#pragma unroll
          for (int j = 0; j < E; j += 4) {
            const float4 a = ld_f4(w + u.off0 + j), b = ld_f4(w + u.off1 + j);
            x[j] *= a.x; x[j + 1] *= a.y; x[j + 2] *= a.z; x[j + 3] *= a.w;
            x[E + j] *= b.x; x[E + j + 1] *= b.y; x[E + j + 2] *= b.z; x[E + j + 3] *= b.w;
          }
        }
        if (u.turn) turn<T, INTER>(x, cs + r * (p.rot / 2) + u.angle, 1.f);
        st_vec(y + u.off0, Elt<T>::pack(x));
        st_vec(y + u.off1, Elt<T>::pack(x + E));
      }
      // the next heads (all lanes are done with the vectors above)
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) {
        const int i = i0 + (UNROLL + k) * kTeams + team;
        if (active && i < units) load(i, k);
      }
    }
    __syncthreads();                               // the angles are rewritten
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
  int H[2], d, rot, R;
  float eps, inv_d;
};

template <typename T, int TEAM, bool INTER>
__global__ void __launch_bounds__(kThreads) head_norm_backward_kernel(const HeadBackwardParams p) {
  constexpr int E = Elt<T>::EPV;
  constexpr int kTeams = kThreads / TEAM;
  extern __shared__ char smem[];
  float2 *cs = reinterpret_cast<float2 *>(smem);
  grid_dependency_wait();
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const bool active = lane * 2 * E < p.d;
  const Unit<T, INTER> u(lane, p.rot);
  const RowAngles ang(p.inv_freq, p.rot);

#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = p.H[which];
    float w[2 * E], dw[2 * E];
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) {
      w[e] = 1.f;
      dw[e] = 0.f;
    }
    if (active && p.w[which]) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w[e] = __ldg(p.w[which] + u.off0 + e);
        w[E + e] = __ldg(p.w[which] + u.off1 + e);
      }
    }
    for (int64_t row0 = (int64_t)blockIdx.x * p.R; row0 < p.rows && H > 0; row0 += (int64_t)gridDim.x * p.R) {
      const int nrow = (int)min((int64_t)p.R, p.rows - row0);
      const int units = nrow * H;
      uint4 xa, xb, ga, gb;
      auto load = [&](int i) {
        const int64_t row = row0 + i / H;
        const int h = i % H;
        const T *x = (const T *)p.x[which] + row * p.stride[which] + (int64_t)h * p.d;
        const T *g = (const T *)p.g[which] + row * p.gstride[which] + (int64_t)h * p.d;
        xa = *reinterpret_cast<const uint4 *>(x + u.off0);
        xb = *reinterpret_cast<const uint4 *>(x + u.off1);
        ga = *reinterpret_cast<const uint4 *>(g + u.off0);
        gb = *reinterpret_cast<const uint4 *>(g + u.off1);
      };
      if (active && team < units) load(team);
      ang.form(cs, p.positions, row0, nrow, p.rows, p.T);
      __syncthreads();
      for (int i0 = 0; i0 < units; i0 += kTeams) {
        const int i = i0 + team;
        const bool live = active && i < units;
        float x[2 * E], g[2 * E], ss = 0.f, ux = 0.f;
        if (live) {
          Elt<T>::unpack(xa, x);
          Elt<T>::unpack(xb, x + E);
          Elt<T>::unpack(ga, g);
          Elt<T>::unpack(gb, g + E);
          if (u.turn) turn<T, INTER>(g, cs + (i / H) * (p.rot / 2) + u.angle, -1.f);
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            ss = fmaf(x[e], x[e], ss);
            ux = fmaf(g[e] * w[e], x[e], ux);
          }
        }
        if (active && i + kTeams < units) load(i + kTeams);
        ss = team_sum_shfl<TEAM>(ss);
        ux = team_sum_shfl<TEAM>(ux);
        if (!live) continue;
        const float r = rsqrtf(ss * p.inv_d + p.eps);
        const float c = ux * p.inv_d * r * r;
        float dx[2 * E];
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) {
          dw[e] = fmaf(g[e], x[e] * r, dw[e]);
          dx[e] = r * fmaf(-c, x[e], g[e] * w[e]);
        }
        T *y = (T *)p.dx[which] + ((row0 + i / H) * H + i % H) * p.d;
        st_vec(y + u.off0, Elt<T>::pack(dx));
        st_vec(y + u.off1, Elt<T>::pack(dx + E));
      }
      __syncthreads();
    }
    if (!p.partials) continue;
    // The CTA's sum of dw: over the teams of a warp by shuffles, over the
    // warps through shared memory in a fixed order (reproducible).
    float *red = reinterpret_cast<float *>(smem);      // [warps][d]: the angles are no longer needed
    const int warp = threadIdx.x / 32, wl = threadIdx.x % 32;
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) {
#pragma unroll
      for (int o = TEAM; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
    }
    if (wl < TEAM && active) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        red[warp * p.d + u.off0 + e] = dw[e];
        red[warp * p.d + u.off1 + e] = dw[E + e];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) s += red[k * p.d + i];
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
  p.H = a.Hq + (cache ? 2 : 1) * a.Hk;
  const int sms = sm_count();
  // Rows per pass: as many as the threads form angles for at once, but no
  // more than leave every SM a few CTAs; a token's heads are split over
  // several CTAs where the rows alone would not fill the SMs.
  const int most = a.rot ? kThreads / (a.rot / 2) : 16;
  const int64_t fill = a.rows / (4 * (int64_t)sms);
  p.R = (int)(fill < 1 ? 1 : fill < most ? fill : most);
  if (p.R > 16) p.R = 16;
  return dispatch(a.dtype, a.d, a.interleaved, [&](auto elt, auto team, auto inter) -> cudaError_t {
    using T = decltype(elt);
    constexpr int TEAM = decltype(team)::value, kTeams = kThreads / TEAM;
    constexpr bool INTER = decltype(inter)::value;
    const int64_t ctas = (a.rows + p.R - 1) / p.R;
    int parts = 1;
    while (ctas * parts < 2 * sms && p.H > parts * kTeams) ++parts;
    p.heads_per_part = (p.H + parts - 1) / parts;
    p.head_parts = (p.H + p.heads_per_part - 1) / p.heads_per_part;
    const int64_t most_x = (int64_t)sms * 8;
    dim3 grid((unsigned)(ctas < most_x ? ctas : most_x), (unsigned)p.head_parts);
    const size_t smem = (size_t)p.R * (a.rot / 2) * sizeof(float2) + (size_t)p.R * sizeof(int64_t);
    return cache ? launch_dependent(head_norm_kernel<T, TEAM, INTER, true>, grid, dim3(kThreads), smem, a.stream, p)
                 : launch_dependent(head_norm_kernel<T, TEAM, INTER, false>, grid, dim3(kThreads), smem, a.stream, p);
  });
}

int head_norm_backward_ctas() { return 4 * sm_count(); }

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
  const int sms = sm_count();
  const int most = a.rot ? kThreads / (a.rot / 2) : 16;
  const int64_t fill = a.rows / (4 * (int64_t)sms);
  p.R = (int)(fill < 1 ? 1 : fill < most ? fill : most);
  if (p.R > 16) p.R = 16;
  const int64_t want = (a.rows + p.R - 1) / p.R;
  const int64_t limit = a.workspace ? a.workspace_rows / 2 : head_norm_backward_ctas();
  const int ctas = (int)(want < limit ? want : limit);
  cudaError_t e = dispatch(a.dtype, a.d, a.interleaved, [&](auto elt, auto team, auto inter) -> cudaError_t {
    using T = decltype(elt);
    size_t smem = (size_t)p.R * (a.rot / 2) * sizeof(float2);
    const size_t red = (size_t)(kThreads / 32) * a.d * sizeof(float);
    if (smem < red) smem = red;
    return launch_dependent(head_norm_backward_kernel<T, decltype(team)::value, decltype(inter)::value>,
                            dim3((unsigned)ctas), dim3(kThreads), smem, a.stream, p);
  });
  if (e != cudaSuccess || !a.workspace) return e;
  return launch_dependent(head_norm_weights_kernel, dim3((unsigned)((2 * a.d + 7) / 8)), dim3(256), 0, a.stream,
                          (const float *)a.workspace, ctas, a.d, a.grad_q_weight, a.grad_k_weight);
}

}  // namespace attnres
