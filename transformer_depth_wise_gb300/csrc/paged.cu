// paged.cu -- attention of one new token per sequence over a paged key-value
// cache, split over the cache's length and joined.
//
// For sequence b, query head h and its key head h / G:  s_j = scale q . k_j
// over the sequence's first lengths[b] cached tokens, o = sum_j softmax(s)_j
// v_j, lse = ln sum_j e^{s_j}.  Each key and value row is read once for all G
// query heads that share it; the running maximum and sum of the softmax are
// kept in fp32, so one pass over the cache is enough.
//
// Split.  The tokens of all (sequence, key head) pairs form one axis of
// tiles of kTile tokens, pair after pair, which the grid's CTAs cut into
// equal ranges whatever the sequences' lengths are.  A pair that lies inside
// one CTA's range is written out by it; of one that is cut, each CTA leaves
// its normalised part and lse in one of its two workspace slots (slot 0 for
// the pair its range begins with, slot 1 for the one it ends with), and the
// join kernel merges the parts in order with the same (lse, o) rule as the
// two-phase merge.  The workspace therefore depends on the grid alone, and
// the result on nothing but the inputs and the device.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace attnres {
namespace {

constexpr int kTile = 64;              // tokens per tile of the split
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct PagedParams {
  const void *q, *k, *v;
  int64_t q_stride;                    // elements from one sequence's queries to the next
  const int32_t *table, *lengths;
  int B, Hq, Hk, G, d;
  int page, max_pages;
  int64_t num_pages;
  float scale;
  void *out;                           // [B, Hq, d]
  float *lse;                          // [B, Hq] or nullptr
  float *part_o, *part_lse;            // [ctas][2][G][d], [ctas][2][G]
};

// The sequence's length, held within what its row of the page table covers.
__device__ __forceinline__ int64_t clamped_length(const PagedParams &p, int b) {
  const int64_t most = (int64_t)p.max_pages * p.page;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n < most ? n : most;
}
__device__ __forceinline__ int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

// The tiles of one key head of all sequences before `upto`, by all threads of the CTA.
__device__ __forceinline__ int64_t tiles_before(const PagedParams &p, int upto, int64_t *red /*[kWarps]*/) {
  int64_t s = 0;
  for (int b = threadIdx.x; b < upto; b += kThreads) s += tiles_of(clamped_length(p, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += red[w];
  return s;
}

// Where range c of `ctas` equal ranges of `total` tiles begins.
__device__ __forceinline__ int64_t range_begin(int64_t total, int c, int ctas) { return total * c / ctas; }

// A CTA's walk over its range: one (sequence, key head, tiles) piece after another.
struct Walk {
  int64_t first, at, end;              // the range's first tile, the next piece's, the last + 1
  int64_t base;                        // first tile of sequence b
  int64_t tiles;                       // tiles per key head of sequence b
  int b;
};
// All threads: find the CTA's range and the sequence it begins in.
__device__ __forceinline__ Walk walk_begin(const PagedParams &p, int64_t *red) {
  Walk w;
  const int64_t total = tiles_before(p, p.B, red) * p.Hk;
  w.first = w.at = range_begin(total, blockIdx.x, gridDim.x);
  w.end = range_begin(total, blockIdx.x + 1, gridDim.x);
  // the sequence by bisection over rounds of whole-CTA sums would cost more
  // than a plain scan: a warp scans 32 lengths at a time
  w.base = 0;
  w.b = 0;
  w.tiles = 0;
  if (w.at >= w.end) return w;
  const int lane = threadIdx.x % 32;
  for (int b0 = 0;; b0 += 32) {
    const int64_t n = b0 + lane < p.B ? tiles_of(clamped_length(p, b0 + lane)) * p.Hk : 0;
    int64_t s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, w.base + s > w.at);
    if (past || b0 + 32 >= p.B) {
      const int l = past ? __ffs(past) - 1 : 31;
      w.b = b0 + l;
      w.base += __shfl_sync(0xffffffffu, s - n, l);
      w.tiles = __shfl_sync(0xffffffffu, n, l) / p.Hk;
      return w;
    }
    w.base += __shfl_sync(0xffffffffu, s, 31);
  }
}

// The cache row of token j of sequence b: element offset, or -1 for a page outside the pool.
__device__ __forceinline__ int64_t cache_row(const PagedParams &p, const int32_t *pages, int j, int hk) {
  const int64_t pg = pages[j / p.page];
  if (pg < 0 || pg >= p.num_pages) return -1;
  return ((pg * p.Hk + hk) * p.page + j % p.page) * p.d;
}

// Where a piece's result goes: the output itself when the piece is the whole pair, else one of the CTA's slots.
template <typename T>
__device__ __forceinline__ void store_piece(const PagedParams &p, bool whole, int b, int hk, int slot, int g, int e,
                                            const float *o, int n, float lse, bool first) {
  if (whole) {
    const int64_t row = (int64_t)b * p.Hq + hk * p.G + g;
    T *dst = (T *)p.out + row * p.d + e;
    for (int i = 0; i < n; ++i) {
      if constexpr (std::is_same<T, float>::value) dst[i] = o[i];
      else dst[i] = __float2bfloat16_rn(o[i]);
    }
    if (first && p.lse) p.lse[row] = lse;
  } else {
    const int64_t row = ((int64_t)blockIdx.x * 2 + slot) * p.G + g;
    for (int i = 0; i < n; ++i) p.part_o[row * p.d + e + i] = o[i];
    if (first) p.part_lse[row] = lse;
  }
}

// ---------------------------------------------------------------------------
// The general kernel (fp32, and every head width the matrix kernel does not
// take).  Eight lanes hold one token's row, NV 16-byte vectors each; a warp
// works on four tokens at a time for GQ query heads kept in registers, and
// the CTA's warps are dealt out over the query heads' groups and the tokens.
// Every team of eight lanes keeps its own running maximum, sum and output;
// they are joined at the end of a piece.
// ---------------------------------------------------------------------------
template <typename T, int NV, int GQ>
__global__ void __launch_bounds__(kThreads) paged_general_kernel(const PagedParams p) {
  constexpr int E = Elt<T>::EPV, N = NV * E;
  extern __shared__ float sm[];                     // [kWarps][GQ][d] outputs, then [kWarps][GQ] m, then l
  __shared__ int64_t red[kWarps];
  grid_dependency_wait();
  Walk w = walk_begin(p, red);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, team = lane / 8, l8 = lane % 8;
  const int groups = (p.G + GQ - 1) / GQ;           // of query heads
  const int strips = kWarps / groups;               // warps over the tokens of one group (G <= kWarps * GQ)
  const int group = warp % groups, strip = warp / groups;
  const bool working = strip < strips;
  const int nvec = p.d / E;
  float *so = sm, *smax = sm + kWarps * GQ * p.d, *ssum = smax + kWarps * GQ;

  while (w.at < w.end) {
    while (w.at >= w.base + w.tiles * p.Hk) {       // the next sequence that has tokens
      w.base += w.tiles * p.Hk;
      ++w.b;
      w.tiles = tiles_of(clamped_length(p, w.b));
    }
    const int hk = (int)((w.at - w.base) / w.tiles);
    const int64_t pair = w.base + hk * w.tiles;     // the pair's first tile
    const int64_t stop = min(w.end, pair + w.tiles);
    const int64_t len = clamped_length(p, w.b);
    const int j0 = (int)((w.at - pair) * kTile), j1 = (int)min(len, (stop - pair) * kTile);
    const bool whole = w.at == pair && stop == pair + w.tiles;
    const int slot = w.at == w.first ? 0 : 1;
    const int32_t *pages = p.table + (int64_t)w.b * p.max_pages;

    float q[GQ][N], o[GQ][N], m[GQ], l[GQ];
#pragma unroll
    for (int g = 0; g < GQ; ++g) {
      const int head = group * GQ + g;
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) o[g][i] = q[g][i] = 0.f;
      if (working && head < p.G) {
        const T *src = (const T *)p.q + (int64_t)w.b * p.q_stride + (int64_t)(hk * p.G + head) * p.d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (v * 8 + l8 < nvec)
            Elt<T>::unpack(*reinterpret_cast<const uint4 *>(src + (v * 8 + l8) * E), q[g] + v * E);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) q[g][i] *= p.scale;
      }
    }
    if (working) {
      for (int j = j0 + strip * 4; j < j1; j += strips * 4) {   // the same trip count for a whole warp
        const int tok = j + team;
        const int64_t row = tok < j1 ? cache_row(p, pages, tok, hk) : -1;
        const bool live = row >= 0;                 // a token on a page outside the pool is left out
        uint4 kv[NV], vv[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          kv[v] = vv[v] = make_uint4(0, 0, 0, 0);
          if (row >= 0 && v * 8 + l8 < nvec) {
            kv[v] = ld_stream((const T *)p.k + row + (v * 8 + l8) * E);
            vv[v] = ld_stream((const T *)p.v + row + (v * 8 + l8) * E);
          }
        }
        float s[GQ];
#pragma unroll
        for (int g = 0; g < GQ; ++g) s[g] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float x[E];
          Elt<T>::unpack(kv[v], x);
#pragma unroll
          for (int g = 0; g < GQ; ++g)
#pragma unroll
            for (int i = 0; i < E; ++i) s[g] = fmaf(x[i], q[g][v * E + i], s[g]);
        }
#pragma unroll
        for (int g = 0; g < GQ; ++g) s[g] = team_sum_shfl<8>(s[g]);
        if (!live) continue;
        float pr[GQ];
#pragma unroll
        for (int g = 0; g < GQ; ++g) {
          const float mn = fmaxf(m[g], s[g]);
          const float keep = m[g] == mn ? 1.f : __expf(m[g] - mn);
          pr[g] = s[g] == -INFINITY ? 0.f : __expf(s[g] - mn);
          m[g] = mn;
          l[g] = fmaf(l[g], keep, pr[g]);
          if (keep != 1.f) {
#pragma unroll
            for (int i = 0; i < N; ++i) o[g][i] *= keep;
          }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float x[E];
          Elt<T>::unpack(vv[v], x);
#pragma unroll
          for (int g = 0; g < GQ; ++g)
#pragma unroll
            for (int i = 0; i < E; ++i) o[g][v * E + i] = fmaf(pr[g], x[i], o[g][v * E + i]);
        }
      }
    }
    // Join the teams of a warp (lanes l8, l8 + 8, ...), then the warps.
#pragma unroll
    for (int g = 0; g < GQ; ++g) {
      float M = m[g];
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
      const float f = m[g] == -INFINITY ? 0.f : __expf(m[g] - M);
      float L = l[g] * f;
      L += __shfl_xor_sync(0xffffffffu, L, 8);
      L += __shfl_xor_sync(0xffffffffu, L, 16);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float x = o[g][i] * f;
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        o[g][i] = x;
      }
      if (team == 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (v * 8 + l8 < nvec) {
#pragma unroll
            for (int i = 0; i < E; ++i) so[(warp * GQ + g) * p.d + (v * 8 + l8) * E + i] = o[g][v * E + i];
          }
        }
        if (l8 == 0) {
          smax[warp * GQ + g] = M;
          ssum[warp * GQ + g] = L;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.G * p.d; i += kThreads) {
      const int head = i / p.d, e = i % p.d, g = head % GQ;
      float M = -INFINITY, L = 0.f, x = 0.f;
      for (int k = 0; k < strips; ++k) M = fmaxf(M, smax[(head / GQ + k * groups) * GQ + g]);
      for (int k = 0; k < strips; ++k) {
        const int at = (head / GQ + k * groups) * GQ + g;
        const float f = smax[at] == -INFINITY ? 0.f : __expf(smax[at] - M);
        L = fmaf(ssum[at], f, L);
        x = fmaf(so[at * p.d + e], f, x);
      }
      x = L == 0.f ? 0.f : x / L;
      store_piece<T>(p, whole, w.b, hk, slot, head, e, &x, 1, L == 0.f ? -INFINITY : M + logf(L), e == 0);
    }
    __syncthreads();
    w.at = stop;
  }
}

// One CTA per (sequence, key head): merge the parts of a pair that several
// CTAs share, or write the empty sequence's zeros.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const PagedParams p, int ctas) {
  __shared__ int64_t red[kWarps];
  grid_dependency_wait();
  const int b = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk;
  const int64_t len = clamped_length(p, b), tiles = tiles_of(len);
  if (tiles == 0) {
    for (int i = threadIdx.x; i < p.G * p.d; i += kThreads) {
      const int64_t row = (int64_t)b * p.Hq + hk * p.G + i / p.d;
      ((T *)p.out)[row * p.d + i % p.d] = T(0.f);
      if (i % p.d == 0 && p.lse) p.lse[row] = -INFINITY;
    }
    return;
  }
  const int64_t total = tiles_before(p, p.B, red) * p.Hk;
  const int64_t s = tiles_before(p, b, red) * p.Hk + hk * tiles, e = s + tiles;
  // the CTAs whose ranges hold tiles s and e - 1
  auto owner = [&](int64_t t) {
    int c = (int)(t * ctas / total);
    while (range_begin(total, c + 1, ctas) <= t) ++c;
    while (range_begin(total, c, ctas) > t) --c;
    return c;
  };
  const int c0 = owner(s), c1 = owner(e - 1);
  if (c0 == c1) return;                             // written whole by its CTA
  for (int i = threadIdx.x; i < p.G * p.d; i += kThreads) {
    const int g = i / p.d, x = i % p.d;
    float M = -INFINITY, L = 0.f, o = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const int64_t begin = range_begin(total, c, ctas);
      if (range_begin(total, c + 1, ctas) == begin) continue;   // an empty range
      const int64_t row = ((int64_t)c * 2 + (begin < s ? 1 : 0)) * p.G + g;
      const float lse = p.part_lse[row];
      if (lse == -INFINITY) continue;
      const float mn = fmaxf(M, lse), f = M == -INFINITY ? 0.f : expf(M - mn), h = expf(lse - mn);
      L = fmaf(L, f, h);
      o = fmaf(o, f, p.part_o[row * p.d + x] * h);
      M = mn;
    }
    const int64_t row = (int64_t)b * p.Hq + hk * p.G + g;
    const float y = L == 0.f ? 0.f : o / L;
    if constexpr (std::is_same<T, float>::value) ((float *)p.out)[row * p.d + x] = y;
    else ((__nv_bfloat16 *)p.out)[row * p.d + x] = __float2bfloat16_rn(y);
    if (x == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : M + logf(L);
  }
}

}  // namespace

bool paged_supported(int64_t d, int dtype) {
  const int e = dtype == ATTNRES_BF16 ? 8 : 4;
  return d >= e && d <= 256 && d % e == 0;
}
int paged_ctas() { return 2 * sm_count(); }

cudaError_t launch_paged(const PagedArgs &a) {
  PagedParams p{};
  p.q = a.q; p.k = a.k_cache; p.v = a.v_cache; p.q_stride = a.q_stride;
  p.table = a.page_table; p.lengths = a.lengths;
  p.B = (int)a.B; p.Hq = a.Hq; p.Hk = a.Hk; p.G = a.Hq / a.Hk; p.d = a.d;
  p.page = a.page_size; p.max_pages = a.max_pages; p.num_pages = a.num_pages;
  p.scale = a.scale; p.out = a.out; p.lse = a.lse;
  const int ctas = paged_ctas();
  p.part_o = a.workspace;
  p.part_lse = a.workspace + (int64_t)ctas * 2 * p.G * p.d;
  const int e = a.dtype == ATTNRES_BF16 ? 8 : 4, nv = (a.d / e + 7) / 8;
  auto go = [&](auto elt, auto NV) -> cudaError_t {
    using T = decltype(elt);
    constexpr int N = decltype(NV)::value * Elt<T>::EPV, GQ = N > 16 ? 2 : 4;
    const size_t smem = (size_t)kWarps * GQ * (p.d + 2) * sizeof(float);
    return launch_dependent(paged_general_kernel<T, decltype(NV)::value, GQ>, dim3((unsigned)ctas), dim3(kThreads),
                            smem, a.stream, p);
  };
  cudaError_t err;
  if (a.dtype == ATTNRES_BF16) {
    const __nv_bfloat16 t{};
    err = nv == 1 ? go(t, std::integral_constant<int, 1>{}) : nv == 2 ? go(t, std::integral_constant<int, 2>{})
                  : go(t, std::integral_constant<int, 4>{});
  } else {
    err = nv <= 2 ? go(0.f, std::integral_constant<int, 2>{}) : nv <= 4 ? go(0.f, std::integral_constant<int, 4>{})
                  : go(0.f, std::integral_constant<int, 8>{});
  }
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)(a.B * a.Hk));
  return a.dtype == ATTNRES_BF16
             ? launch_dependent(paged_join_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, a.stream, p, ctas)
             : launch_dependent(paged_join_kernel<float>, grid, dim3(kThreads), 0, a.stream, p, ctas);
}

}  // namespace attnres
