// shared.cu -- attention of one new token per sequence of a batch that shares
// a prefix in the paged cache, each sequence going on with pages of its own.
//
// For sequence b and query head h:  out = softmax of scale q.k over the
// prefix's tokens and the sequence's own ones, times v; lse.  The prefix is
// the same for all sequences, so the query heads of all of them that share a
// key head are the rows of one matrix Q [B G, d], and the prefix costs two
// matrix products, Q K^T and P V, which read the prefix once per tile of rows
// instead of once per sequence.  The rows' tiles and the prefix's ranges are
// dealt out over the CTAs; each leaves its part, normalised, with its lse.
// The sequences' own tokens go through the kernel of attnres_paged_attention,
// which leaves one more part (or several, of a sequence that its split has
// cut), and a last kernel joins the parts by the online-softmax merge (OS2).
//
// This file: the parts of the prefix in fp32, and the join (bf16: shared_tc.cu).
// 64 tokens at a time go through shared memory, the keys and the queries
// transposed; a thread forms the scores of eight rows (or four) with four
// tokens, and then adds to an eighth of its rows' outputs (half of that for
// 64-wide heads), as products of pairs of rows.  The reads from shared memory
// bind: 12 words a lane for 32 multiply-adds, then 16 for 64.  Measured on
// GB300: 64 sequences of 32 heads over 8 behind 8000 tokens, 128 wide 245 us (34
// TFLOP/s), 64 wide and 16000 tokens 251 us, 256 wide and 4000 tokens 356 us (24).
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "shared.cuh"

namespace attnres {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;                // tokens of a tile

// A CTA's shared memory for ROWS query rows of D elements, in floats.
template <int D, int ROWS> struct Shape {
  static constexpr int kQ = ROWS + 4, kK = kKeys + 4, kV = D + 4, kP = ROWS + 4;     // pitches
  static constexpr int kOffK = D * kQ, kOffV = kOffK + D * kK, kOffP = kOffV + kKeys * kV, kEnd = kOffP + kKeys * kP;
  static constexpr size_t kSmem = (size_t)kEnd * sizeof(float);
  static constexpr int kPieces = kKeys * D / 4 / kThreads;            // 16-byte pieces of a tile per thread and tensor
};

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads) shared_f32_kernel(const PrefixParams p) {
  using S = Shape<D, ROWS>;
  constexpr int R = ROWS / 16, R2 = R / 2, C = D / 16, N = S::kPieces;   // rows, pairs of rows and output columns of a thread
  extern __shared__ __align__(16) float sm[];
  float *qs = sm, *ks = sm + S::kOffK, *vs = sm + S::kOffV, *ps = sm + S::kOffP;
  __shared__ int live[kKeys];
  p.begin();
  const int all = p.B * p.G, tiles = (all + ROWS - 1) / ROWS;
  const int hk = blockIdx.x / tiles, row0 = (blockIdx.x - hk * tiles) * ROWS, split = blockIdx.y;
  int j0, j1;
  p.range<kKeys>(p.tokens(), split, j0, j1);
  const int nvec = p.d / 4, ty = threadIdx.x / 16, tx = threadIdx.x % 16;

  // the queries by element, zero behind the batch and behind d, in powers of two
  const float scale2 = p.scale * 1.44269504088896340736f;
  for (int i = threadIdx.x; i < ROWS * (D / 4); i += kThreads) {
    const int r = i % ROWS, c = i / ROWS, row = row0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < all && c < nvec)
      x = *reinterpret_cast<const float4 *>((const float *)p.q + (int64_t)(row / p.G) * p.q_stride +
                                            (int64_t)(hk * p.G + row % p.G) * p.d + c * 4);
    float *to = qs + c * 4 * S::kQ + r;
    to[0] = x.x * scale2;
    to[S::kQ] = x.y * scale2;
    to[2 * S::kQ] = x.z * scale2;
    to[3 * S::kQ] = x.w * scale2;
  }

  // A thread's pieces of a tile: keys with the tokens side by side over the
  // lanes (they are stored by element), values with the elements.
  auto piece = [&](const void *cache, int j, int t, int c, bool &have) -> float4 {
    const int64_t at = j + t < j1 ? p.row(j + t, hk) : -1;
    have = at >= 0;
    return have && c < nvec ? *reinterpret_cast<const float4 *>((const float *)cache + at + c * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto key = [&](int j, int u, bool &have) {
    const int i = threadIdx.x + u * kThreads;
    return piece(p.k, j, i % kKeys, i / kKeys, have);
  };
  auto value = [&](int j, int u) {
    const int i = threadIdx.x + u * kThreads;
    bool have;
    return piece(p.v, j, i / (D / 4), i % (D / 4), have);
  };
  auto store = [&](int u, const float4 &k, const float4 &v, bool have) {
    const int i = threadIdx.x + u * kThreads;
    float *to = ks + i / kKeys * 4 * S::kK + i % kKeys;
    to[0] = k.x;
    to[S::kK] = k.y;
    to[2 * S::kK] = k.z;
    to[3 * S::kK] = k.w;
    *reinterpret_cast<float4 *>(vs + i / (D / 4) * S::kV + i % (D / 4) * 4) = v;
    if (i < kKeys) live[i] = have;
  };
  // the next tile's are on their way while the present one is worked on
  float4 kv[N], vv[N];
  bool have[N];
  auto read = [&](int j) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      kv[u] = key(j, u, have[u]);
      vv[u] = value(j, u);
    }
  };

  float m[R], l[R];
  uint64_t o[R2][C];                       // of two rows each
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) o[r / 2][c] = 0;
  }
  if (j0 < j1) read(j0);
  for (int j = j0; j < j1; j += kKeys) {
    __syncthreads();                       // the last tile is read
#pragma unroll
    for (int u = 0; u < N; ++u) store(u, kv[u], vv[u], have[u]);
    __syncthreads();
    if (j + kKeys < j1) read(j + kKeys);
    // scores of rows R ty .. with tokens tx + 16 i
    uint64_t s[R2][4] = {};
#pragma unroll 8
    for (int c = 0; c < D; ++c) {
      uint64_t a[R2];
#pragma unroll
      for (int r = 0; r < R2; r += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(qs + c * S::kQ + ty * R + 2 * r);
        a[r] = x.x;
        a[r + 1] = x.y;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float k = ks[c * S::kK + tx + 16 * i];
        const uint64_t k2 = pair(k, k);
#pragma unroll
        for (int r = 0; r < R2; ++r) fma_pair(s[r][i], a[r], k2);
      }
    }
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) on[i] = live[tx + 16 * i];
#pragma unroll
    for (int r = 0; r < R2; ++r) {
      float x[2][4], keep[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unpair(s[r][i], x[0][i], x[1][i]);
        if (!on[i]) x[0][i] = x[1][i] = -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
#pragma unroll
        for (int e = 1; e < 16; e <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
        const int at = 2 * r + h;
        const float mn = fmaxf(m[at], top), base = mn == -INFINITY ? 0.f : mn;
        keep[h] = m[at] == mn ? 1.f : exp2_fast(m[at] - mn);
        m[at] = mn;
        l[at] *= keep[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[h][i] = exp2_fast(x[h][i] - base);
          l[at] += x[h][i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[r][i] = pair(x[0][i], x[1][i]);
      if (keep[0] != 1.f || keep[1] != 1.f) {
        const uint64_t k2 = pair(keep[0], keep[1]);
#pragma unroll
        for (int c = 0; c < C; ++c) scale_pair(o[r][c], k2);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < R2; r += 2)
        *reinterpret_cast<ulonglong2 *>(ps + (tx + 16 * i) * S::kP + ty * R + 2 * r) = make_ulonglong2(s[r][i], s[r + 1][i]);
    __syncwarp();                          // a row's weights come from 16 lanes of its own warp
    const int left = min(kKeys, j1 - j);
#pragma unroll 4
    for (int t = 0; t < left; ++t) {
      uint64_t a[R2];
#pragma unroll
      for (int r = 0; r < R2; r += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(ps + t * S::kP + ty * R + 2 * r);
        a[r] = x.x;
        a[r + 1] = x.y;
      }
#pragma unroll
      for (int c = 0; c < C; c += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(vs + t * S::kV + c * 16 + tx * 4);
        const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t v2 = pair(e[i], e[i]);
#pragma unroll
          for (int r = 0; r < R2; ++r) fma_pair(o[r][c + i], a[r], v2);
        }
      }
    }
  }
#pragma unroll
  for (int at = 0; at < R; ++at) {
    const int row = row0 + ty * R + at;
    float L = l[at];
#pragma unroll
    for (int e = 1; e < 16; e <<= 1) L += __shfl_xor_sync(0xffffffffu, L, e);
    if (row >= all) continue;
    const int64_t part = p.part(split, row, hk);
    const float f = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int c = 0; c < C; c += 4) {
      if (c * 16 + tx * 4 >= p.d) continue;
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpair(o[at / 2][c + i], lo, hi);
        x[i] = (at & 1 ? hi : lo) * f;
      }
      *reinterpret_cast<float4 *>(p.part_o + part * p.d + c * 16 + tx * 4) = make_float4(x[0], x[1], x[2], x[3]);
    }
    if (tx == 0) p.part_lse[part] = L == 0.f ? -INFINITY : (m[at] + log2f(L)) * 0.69314718055994530942f;
  }
}

// What the join reads: parts [splits + 1][rows] of the prefix and, where a
// pair's own tokens were not cut, of those; else their pieces.
struct JoinParams {
  const float *part_o, *part_lse, *piece_o, *piece_lse;
  const Pieces *pieces;                    // [B, Hk]
  int splits, Hq, Hk, G, d;
  int rows;                                // B Hq
  Mark ready;                              // of the own tokens' kernel, taken away
  void *out;
  float *lse;
};

struct Sum {
  float4 v[2];                             // elements 4 lane .. and 128 + 4 lane ..
  __device__ __forceinline__ void zero() { v[0] = v[1] = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float *row, int lane, int d) {
    zero();
    if (lane * 4 < d) v[0] = *reinterpret_cast<const float4 *>(row + lane * 4);
    if (d > 128 && lane * 4 + 128 < d) v[1] = *reinterpret_cast<const float4 *>(row + lane * 4 + 128);
  }
  __device__ __forceinline__ void add(const Sum &x, float h) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i].x = fmaf(x.v[i].x, h, v[i].x);
      v[i].y = fmaf(x.v[i].y, h, v[i].y);
      v[i].z = fmaf(x.v[i].z, h, v[i].z);
      v[i].w = fmaf(x.v[i].w, h, v[i].w);
    }
  }
  template <typename T> __device__ __forceinline__ void store(T *row, int lane, int d, float f) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = lane * 4 + i * 128;
      if (e >= d) break;
      const float4 y = make_float4(v[i].x * f, v[i].y * f, v[i].z * f, v[i].w * f);
      if constexpr (std::is_same<T, float>::value) *reinterpret_cast<float4 *>(row + e) = y;
      else *reinterpret_cast<uint2 *>(row + e) = make_uint2(Elt<T>::pack_word(y.x, y.y), Elt<T>::pack_word(y.z, y.w));
    }
  }
};
// A part without tokens, or none with a weight, may hold nothing and is left out.  One whose weight is too small for
// fp32 is not: it may hold an infinity or a NaN, which shows.
__device__ __forceinline__ bool part_counts(float lse) { return lse != -INFINITY; }
__device__ __forceinline__ float part_weight(float lse, float M) { return part_counts(lse) ? expf(lse - M) : 0.f; }
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

constexpr int kJoinWarps = 8;

// A warp per (sequence, query head) and PARTS parts of the prefix: everything
// whose place is known, the own tokens' part of a pair that was not cut among
// it, is on its way at once, and only a cut pair's pieces need a second read.
template <typename T, int PARTS>
__global__ void __launch_bounds__(kJoinWarps * 32) shared_join_few_kernel(const JoinParams p) {
  grid_dependency_wait();
  if (p.ready.at && blockIdx.x == 0 && threadIdx.x == 0) p.ready.take_away();
  const int lane = threadIdx.x % 32, d = p.d;
  const int row = blockIdx.x * kJoinWarps + threadIdx.x / 32;
  if (row >= p.rows) return;
  const int b = row / p.Hq, head = row - b * p.Hq, hk = head / p.G, g = head - hk * p.G;
  float x[PARTS + 1];
  Sum y[PARTS + 1];
#pragma unroll
  for (int k = 0; k <= PARTS; ++k) {
    const int64_t at = (int64_t)k * p.rows + row;
    x[k] = p.part_lse[at];
    y[k].load(p.part_o + at * d, lane, d);
  }
  const Pieces own = p.pieces[b * p.Hk + hk];
  const int pieces = own.first < 0 ? 0 : own.last - own.first + 1;
  if (pieces) x[PARTS] = -INFINITY;
  auto piece = [&](int c) { return ((own.first + c) * 2 + (c == 0 ? own.slot : 0)) * p.G + g; };
  float M = -INFINITY;
  for (int c = lane; c < pieces; c += 32) M = fmaxf(M, p.piece_lse[piece(c)]);
  if (pieces) M = warp_max(M);
#pragma unroll
  for (int k = 0; k <= PARTS; ++k) M = fmaxf(M, x[k]);
  float L = 0.f;
  Sum s;
  s.zero();
#pragma unroll
  for (int k = 0; k <= PARTS; ++k) {
    const float w = part_weight(x[k], M);
    L += w;
    if (part_counts(x[k])) s.add(y[k], w);
  }
#pragma unroll 2
  for (int c = 0; c < pieces; ++c) {
    const int at = piece(c);
    Sum z;
    z.load(p.piece_o + (int64_t)at * d, lane, d);
    const float lse = p.piece_lse[at], w = part_weight(lse, M);
    L += w;
    if (part_counts(lse)) s.add(z, w);
  }
  s.store((T *)p.out + (int64_t)row * d, lane, d, L == 0.f ? 0.f : 1.f / L);
  if (lane == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : M + logf(L);
}

// WARPS warps per (sequence, query head), 32 parts at a time: a lane finds a
// part and its weight by its lse, then a warp adds every WARPS-th part, in an
// order that is always the same.
template <typename T, int WARPS>
__global__ void __launch_bounds__(kJoinWarps * 32) shared_join_kernel(const JoinParams p) {
  __shared__ Sum sums[kJoinWarps][32];
  grid_dependency_wait();
  if (p.ready.at && blockIdx.x == 0 && threadIdx.x == 0) p.ready.take_away();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, first = warp % WARPS, d = p.d;
  const int row = blockIdx.x * (kJoinWarps / WARPS) + warp / WARPS;
  const bool live = row < p.rows;
  const int b = row / p.Hq, head = row - b * p.Hq, hk = head / p.G, g = head - hk * p.G;
  // the lse of the lane's part of the prefix, before the pieces' place is known
  float x0 = live && lane < p.splits ? p.part_lse[(int64_t)lane * p.rows + row] : -INFINITY;
  Pieces own{-1, 0, 0};
  if (live) own = p.pieces[b * p.Hk + hk];
  const int parts = !live ? 0 : own.first < 0 ? p.splits + 1 : p.splits + own.last - own.first + 1;
  // part k's row, in part_o or in piece_o, and its lse
  auto find = [&](int k, const float *&src) -> float {
    src = p.part_o;
    if (k >= parts) return -INFINITY;
    if (k < p.splits || own.first < 0) {
      const int64_t at = (int64_t)k * p.rows + row;
      src = p.part_o + at * d;
      return k < 32 && k < p.splits ? x0 : p.part_lse[at];
    }
    const int c = k - p.splits;
    const int64_t at = ((int64_t)(own.first + c) * 2 + (c == 0 ? own.slot : 0)) * p.G + g;
    src = p.piece_o + at * d;
    return p.piece_lse[at];
  };
  const float *src0, *src;
  x0 = find(lane, src0);
  float M = x0, L = 0.f;
  for (int k = lane + 32; k < parts; k += 32) M = fmaxf(M, find(k, src));
  M = warp_max(M);
  Sum s;
  s.zero();
  for (int k0 = 0; k0 < parts; k0 += 32) {
    src = src0;
    const float lse = k0 == 0 ? x0 : find(k0 + lane, src), w = part_weight(lse, M);
    L += w;
    const unsigned counts = __ballot_sync(0xffffffffu, part_counts(lse));
    const int n = min(32, parts - k0);
#pragma unroll 4
    for (int k = first; k < n; k += WARPS) {
      const float h = __shfl_sync(0xffffffffu, w, k);
      const float *from = reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, (unsigned long long)src, k));
      if (!(counts >> k & 1u)) continue;
      Sum y;
      y.load(from, lane, d);
      s.add(y, h);
    }
  }
  L = team_sum_shfl<32>(L);
  sums[warp][lane] = s;
  __syncthreads();
  if (first > 0 || !live) return;
#pragma unroll
  for (int k = 1; k < WARPS; ++k) s.add(sums[warp + k][lane], 1.f);
  s.store((T *)p.out + (int64_t)row * d, lane, d, L == 0.f ? 0.f : 1.f / L);
  if (lane == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : M + logf(L);
}

// Few parts of the prefix: a warp per row.  More: eight warps per row where the
// rows are few, two where they fill the GPU.
template <typename T> cudaError_t launch_join(const JoinParams &p, cudaStream_t stream) {
  auto few = [&](auto n) -> cudaError_t {
    return launch_dependent(shared_join_few_kernel<T, decltype(n)::value>,
                            dim3((unsigned)((p.rows + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32), 0, stream, p);
  };
  auto many = [&](auto warps) -> cudaError_t {
    constexpr int W = decltype(warps)::value, R = kJoinWarps / W;
    return launch_dependent(shared_join_kernel<T, W>, dim3((unsigned)((p.rows + R - 1) / R)), dim3(kJoinWarps * 32), 0, stream,
                            p);
  };
  switch (p.splits) {
    case 0: return few(std::integral_constant<int, 0>{});
    case 1: return few(std::integral_constant<int, 1>{});
    case 2: return few(std::integral_constant<int, 2>{});
    case 3: return few(std::integral_constant<int, 3>{});
  }
  return p.rows >= 8 * (int64_t)sm_count() ? many(std::integral_constant<int, 2>{}) : many(std::integral_constant<int, 8>{});
}

// Rows of a CTA: 128 where that pads no more than a fifth over 64, but for
// heads wider than 128, whose tiles fill the shared memory with 64.
int f32_rows(int64_t rows, int d) {
  const int64_t by64 = (rows + 63) / 64 * 64, by128 = (rows + 127) / 128 * 128;
  return d <= 128 && by128 * 5 <= by64 * 6 ? 128 : 64;
}

// Ranges of the prefix with the least time, in tiles of a CTA: its start and
// end are worth two, and an SM has one CTA (two with 64-wide heads).
int f32_splits(int64_t B, int G, int Hk, int d, int64_t tokens) {
  const int rows = f32_rows(B * G, d);
  const int64_t items = (B * G + rows - 1) / rows * Hk, tiles = (tokens + kKeys - 1) / kKeys;
  const int64_t slots = (d <= 64 ? 2 : 1) * sm_count();
  int best = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= kMaxPrefixParts && n <= tiles; ++n) {
    const int64_t cost = (items * n + slots - 1) / slots * (2 + (tiles + n - 1) / n);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

cudaError_t launch_shared_f32(const PrefixParams &p, cudaStream_t stream) {
  auto go = [&](auto D, auto rows) -> cudaError_t {
    constexpr int ROWS = decltype(rows)::value;
    using S = Shape<decltype(D)::value, ROWS>;
    constexpr auto kern = shared_f32_kernel<decltype(D)::value, ROWS>;
    const cudaError_t e = allow_smem<kern>(S::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((int64_t)p.Hk * (((int64_t)p.B * p.G + ROWS - 1) / ROWS)), (unsigned)p.splits);
    return launch_dependent(kern, grid, dim3(kThreads), S::kSmem, stream, p);
  };
  using R64 = std::integral_constant<int, 64>;
  using R128 = std::integral_constant<int, 128>;
  if (p.d > 128) return go(std::integral_constant<int, 256>{}, R64{});
  const bool wide = f32_rows((int64_t)p.B * p.G, p.d) == 128;
  if (p.d > 64) return wide ? go(R128{}, R128{}) : go(R128{}, R64{});
  return wide ? go(R64{}, R128{}) : go(R64{}, R64{});
}

// The own tokens' marks.  A call takes the next place and a number that no
// other call has; its prefix's kernel writes the number there, and its join
// takes it away, so that a captured call finds none of its last replay.  Calls
// that share a place at the same time overwrite each other's number, and then
// the own tokens' kernel waits like any other.
constexpr int kMarks = 4096;
__device__ unsigned long long g_marks[kMarks];

Mark next_mark() {
  static std::atomic<unsigned long long> calls{0};
  void *at = nullptr;                    // asked every time: a device that has been reset has the table elsewhere
  if (cudaGetSymbolAddress(&at, g_marks) != cudaSuccess) return {};
  const unsigned long long n = calls.fetch_add(1, std::memory_order_relaxed) + 1;
  return {static_cast<unsigned long long *>(at) + n % kMarks, n};
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

SharedLayout shared_layout(int64_t B, int Hq, int Hk, int64_t d, int dtype, int64_t tokens, int64_t own) {
  SharedLayout w{};
  const int G = Hq / Hk;
  if (B > 0 && tokens > 0)
    w.splits = dtype == ATTNRES_BF16 ? shared_tc_splits(B, G, Hk, d, tokens, own) : f32_splits(B, G, Hk, (int)d, tokens);
  const int64_t rows = B * Hq, parts = w.splits + 1;
  // Behind a prefix's kernel the SMs come free one after the other: ranges
  // of a third of the length even that out, where the tables leave each of
  // them 8 tiles of 64 tokens or more (fp32: 16).  With thirds and without: 256
  // chats of up to 2048 tokens 259 and 269 us (halves, when it was 277 without,
  // 266, sixths 265), 64 of as many behind 2048 tokens 82 and 92, with heads of 256
  // 64 of up to 1024 128 and 141 and of up to 512 130 and 154, 64 of up to 2048 behind
  // 131071 155 and 159; but 128 of up to 1024 with heads of 64 94 and 89.  Below: 64 chats
  // of up to 256 50 and 45, 48 of up to 1024 on two key heads 63 and 57, fp32 with
  // 9 tiles 328 and 320.
  w.own_ctas = paged_ctas(d, dtype);
  const int64_t fine = paged_fine_ctas(d, dtype), least = dtype == ATTNRES_BF16 ? 8 : 16;
  if (w.splits && B * Hk * (own / 64) >= least * fine) w.own_ctas = (int)fine;
  w.pieces = up16(paged_workspace_bytes(G, d, dtype, w.own_ctas));
  w.part_lse = w.pieces + up16(B * Hk * (int64_t)sizeof(Pieces));
  w.part_o = w.part_lse + up16(parts * rows * (int64_t)sizeof(float));
  w.bytes = w.part_o + parts * rows * d * (int64_t)sizeof(float);
  return w;
}

cudaError_t launch_shared(const SharedArgs &a, const SharedLayout &w) {
  // without a pool no table is read
  const int64_t tokens = a.num_pages > 0 ? (int64_t)a.prefix_pages * a.page_size : 0;
  char *ws = static_cast<char *>(a.workspace);
  const int64_t rows = a.B * a.Hq;
  PrefixParams p{};
  p.q = a.q; p.k = a.k_cache; p.v = a.v_cache; p.q_stride = a.q_stride;
  p.table = a.prefix_table; p.length = a.prefix_length;
  p.B = (int)a.B; p.Hq = a.Hq; p.Hk = a.Hk; p.G = a.Hq / a.Hk; p.d = a.d;
  p.page = a.page_size; p.most = (int)tokens; p.num_pages = a.num_pages; p.scale = a.scale;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  p.part_o = reinterpret_cast<float *>(ws + w.part_o);
  p.part_lse = reinterpret_cast<float *>(ws + w.part_lse);
  p.splits = w.splits;
  p.wait_limit = wait_limit_cycles();
  cudaError_t e = cudaSuccess;
  if (w.splits > 0) {
    p.ready = next_mark();
    e = a.dtype == ATTNRES_BF16 ? launch_shared_tc(p, a.stream) : launch_shared_f32(p, a.stream);
  }
  if (e != cudaSuccess) return e;
  // The sequences' own tokens: the last part.  It needs nothing of the prefix's
  // kernel, which lets it start as soon as all of its own CTAs have: by the mark
  // it fills the SMs that that one leaves, and waits for its end at its own (256
  // chats 258 us, 280 where it waits at its start; four chats 14 and 19 us).
  PagedArgs s{};
  s.q = a.q; s.q_stride = a.q_stride; s.k_cache = a.k_cache; s.v_cache = a.v_cache; s.num_pages = a.num_pages;
  s.page_size = a.page_size; s.max_pages = a.max_pages; s.page_table = a.page_table; s.lengths = a.lengths;
  s.B = a.B; s.Hq = a.Hq; s.Hk = a.Hk; s.d = a.d; s.dtype = a.dtype; s.scale = a.scale;
  s.out = p.part_o + w.splits * rows * a.d; s.lse = p.part_lse + w.splits * rows; s.out_f32 = true;
  s.workspace = ws; s.stream = a.stream; s.ready = p.ready; s.ctas = w.own_ctas;
  s.pieces = reinterpret_cast<Pieces *>(ws + w.pieces);
  if ((e = launch_paged(s)) != cudaSuccess) return e;
  JoinParams j{};
  const PagedParts own = paged_parts(ws, p.G, a.d, w.own_ctas);
  j.part_o = p.part_o; j.part_lse = p.part_lse; j.piece_o = own.o; j.piece_lse = own.lse; j.pieces = s.pieces;
  j.splits = w.splits; j.Hq = a.Hq; j.Hk = a.Hk; j.G = p.G; j.d = a.d; j.rows = (int)rows; j.ready = p.ready; j.out = a.out; j.lse = a.lse;
  return a.dtype == ATTNRES_BF16 ? launch_join<__nv_bfloat16>(j, a.stream) : launch_join<float>(j, a.stream);
}

}  // namespace attnres
