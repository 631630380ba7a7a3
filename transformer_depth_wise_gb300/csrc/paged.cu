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
// the pair its range begins with, slot 1 for the one it ends with), the CTA
// that holds the pair's beginning notes it, and the join kernel merges the
// noted pairs' parts in order with the same (lse, o) rule as the two-phase
// merge.  At most one pair per CTA is cut, so the workspace depends on the
// grid alone, and the result on nothing but the inputs and the device.
//
// The cache's bytes bind.  Measured on GB300, bf16, heads of 128: 256 sequences
// of up to 8192 tokens, 56 query over 8 key heads, 4.3 GB in 681 us (6.3 TB/s)
// and 9 us for the join; 65537 and 131071 tokens, 32 over 4, 403 MB in 65 us
// (6.2 TB/s) and 7 us.  fp32, 16 sequences of 2048 to 4096 tokens, 8 key heads of
// 128: 71 us with one or two query heads each, 113 with four, 195 with eight,
// where the CUDA cores bind.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace attnres {
namespace {

constexpr int kTile = 64;              // tokens per tile of the split

struct PagedParams {
  const void *q, *k, *v;
  int64_t q_stride;                    // elements from one sequence's queries to the next
  const int32_t *table, *lengths;
  int B, Hq, Hk, G, d;
  int page, page_shift, max_pages;     // page_shift: log2(page), or -1
  int64_t num_pages;
  float scale;
  void *out;                           // [B, Hq, d]
  Mark ready;                          // of the kernel before, which is waited for at the end only (or none)
  bool out_f32;                        // out in fp32 whatever the type (a part of a longer attention, with pieces)
  float *lse;                          // [B, Hq] or nullptr
  float *part_o, *part_lse;            // [ctas][2][G][d], [ctas][2][G]
  Cut *cuts;                           // [ctas]
  Pieces *pieces;                      // [B, Hk] or nullptr: where each pair's parts are, for a join elsewhere
  __device__ __forceinline__ int page_of(int j) const { return page_shift >= 0 ? j >> page_shift : j / page; }
  __device__ __forceinline__ int slot_of(int j) const { return page_shift >= 0 ? j & (page - 1) : j % page; }
};

// What a kernel starts with, all threads: the wait for what came before.  With
// a mark the kernel before has started this one early, and nothing of that one
// is read here; a thread that finds the mark raised sees all that it waited
// for itself, and one that does not waits for its end.
__device__ __forceinline__ void wait_for_inputs(const PagedParams &p) {
  if (!p.ready.at || !p.ready.raised()) grid_dependency_wait();
}
// What it ends with: one CTA's wait holds the launch's end until the kernel before has ended.
__device__ __forceinline__ void wait_for_last(const PagedParams &p) {
  if (p.ready.at && blockIdx.x + 1 == gridDim.x) grid_dependency_wait();
}

// The sequence's length, held within what its row of the page table covers.
__device__ __forceinline__ int64_t clamped_length(const PagedParams &p, int b) {
  const int64_t most = (int64_t)p.max_pages * p.page;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n < most ? n : most;
}
__device__ __forceinline__ int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

// The tiles of one key head of all sequences, by all threads of the CTA.
__device__ __forceinline__ int64_t all_tiles(const PagedParams &p, int64_t *red /*[warps]*/) {
  int64_t s = 0;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) s += tiles_of(clamped_length(p, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  s = 0;
  for (int w = 0; w < (int)(blockDim.x / 32); ++w) s += red[w];
  return s;
}

// Where range c of `ctas` equal ranges of `total` tiles begins.
__device__ __forceinline__ int64_t range_begin(int64_t total, int c, int ctas) { return total * c / ctas; }

// A walk over a CTA's range: one piece (the tiles of one pair that lie in the range) after another.
struct Walk {
  int64_t at, end;                     // the piece's first tile, the range's last + 1
  int64_t pair;                        // the first tile of the piece's pair
  int tiles;                           // of the pair
  int len, b, hk;                      // the sequence's length, sequence, key head
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ int64_t stop() const { return min(end, pair + tiles); }
  __device__ __forceinline__ bool begins() const { return at == pair; }
  __device__ __forceinline__ bool whole() const { return at == pair && pair + tiles <= end; }
  __device__ __forceinline__ int first_token() const { return (int)(at - pair) * kTile; }
  __device__ __forceinline__ int last_token() const { return (int)min((int64_t)len, (stop() - pair) * kTile); }
  __device__ __forceinline__ void next(const PagedParams &p) {
    at = stop();
    if (at >= end) return;
    pair += tiles;
    if (++hk < p.Hk) return;
    hk = 0;
    do {                               // the next sequence that has tokens
      len = (int)clamped_length(p, ++b);
    } while (len == 0);
    tiles = (int)tiles_of(len);
  }
};

// All threads: the walk over this CTA's range, of `total` tiles in all.
__device__ __forceinline__ Walk walk_begin(const PagedParams &p, int64_t total) {
  Walk w;
  w.at = range_begin(total, blockIdx.x, gridDim.x);
  w.end = range_begin(total, blockIdx.x + 1, gridDim.x);
  w.pair = 0;
  w.tiles = w.len = w.b = w.hk = 0;
  if (w.at >= w.end) return w;
  // every warp finds the sequence by itself, 32 lengths at a time
  const int lane = threadIdx.x % 32;
  for (int b0 = 0;; b0 += 32) {
    const int64_t n = b0 + lane < p.B ? tiles_of(clamped_length(p, b0 + lane)) * p.Hk : 0;
    int64_t s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, w.pair + s > w.at);
    if (past || b0 + 32 >= p.B) {
      const int l = past ? __ffs(past) - 1 : 31;
      w.b = b0 + l;
      w.pair += __shfl_sync(0xffffffffu, s - n, l);
      w.tiles = (int)(__shfl_sync(0xffffffffu, n, l) / p.Hk);
      break;
    }
    w.pair += __shfl_sync(0xffffffffu, s, 31);
  }
  w.len = (int)clamped_length(p, w.b);
  w.hk = (int)((w.at - w.pair) / w.tiles);
  w.pair += (int64_t)w.hk * w.tiles;
  return w;
}

// One thread: note the pair that the walk's piece begins.
__device__ __forceinline__ void note_cut(const PagedParams &p, const Walk &w, int slot, int64_t total) {
  const int64_t last_tile = w.pair + w.tiles - 1;
  const int ctas = gridDim.x;
  if (w.whole()) {
    if (p.pieces) p.pieces[(int64_t)w.b * p.Hk + w.hk] = {-1, 0, 0};
    return;
  }
  int c = (int)(last_tile * ctas / total);
  while (range_begin(total, c + 1, ctas) <= last_tile) ++c;
  while (range_begin(total, c, ctas) > last_tile) --c;
  if (p.pieces) p.pieces[(int64_t)w.b * p.Hk + w.hk] = {(int)blockIdx.x, c, slot};
  else p.cuts[blockIdx.x] = {w.b, w.hk, c, slot};
}

// Sequences without tokens: zeros and -infinity, dealt out over the CTAs.
template <typename T>
__device__ __forceinline__ void write_empty(const PagedParams &p) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (clamped_length(p, b) != 0) continue;
    for (int i = threadIdx.x; i < p.Hq * p.d; i += blockDim.x) {
      const int64_t at = (int64_t)b * p.Hq * p.d + i;
      if (p.out_f32) ((float *)p.out)[at] = 0.f;
      else ((T *)p.out)[at] = T(0.f);
    }
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += blockDim.x) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
    if (p.pieces)
      for (int i = threadIdx.x; i < p.Hk; i += blockDim.x) p.pieces[(int64_t)b * p.Hk + i] = {-1, 0, 0};
  }
}

// The cache row of token j of a sequence with this row of the page table:
// element offset, or -1 for a page outside the pool.
__device__ __forceinline__ int64_t cache_row(const PagedParams &p, int pg, int j, int hk) {
  if (pg < 0 || pg >= p.num_pages) return -1;
  return (((int64_t)pg * p.Hk + hk) * p.page + p.slot_of(j)) * p.d;
}

// Four of a piece's outputs (elements e .. e + 3 of head g) and, with e == 0,
// its lse: to the output when the piece is the whole pair, else to a slot.
template <typename T>
__device__ __forceinline__ void store_piece(const PagedParams &p, const Walk &w, int slot, int g, int e, float4 o,
                                            float lse) {
  if (w.whole()) {
    const int64_t row = (int64_t)w.b * p.Hq + w.hk * p.G + g;
    T *dst = (T *)p.out + row * p.d + e;
    if constexpr (std::is_same<T, float>::value) *reinterpret_cast<float4 *>(dst) = o;
    else if (p.out_f32) *reinterpret_cast<float4 *>((float *)p.out + row * p.d + e) = o;
    else *reinterpret_cast<uint2 *>(dst) = make_uint2(Elt<T>::pack_word(o.x, o.y), Elt<T>::pack_word(o.z, o.w));
    if (e == 0 && p.lse) p.lse[row] = lse;
  } else {
    const int64_t row = ((int64_t)blockIdx.x * 2 + slot) * p.G + g;
    *reinterpret_cast<float4 *>(p.part_o + row * p.d + e) = o;
    if (e == 0) p.part_lse[row] = lse;
  }
}

// ---------------------------------------------------------------------------
// fp32.  Eight lanes hold one token's row, NV 16-byte vectors each; a warp
// works on four tokens at a time for GQ query heads kept in registers, and
// the CTA's warps are dealt out over the query heads' groups and the tokens.
// Every team of eight lanes keeps its own running maximum, sum and output;
// they are joined at the end of a piece.
// ---------------------------------------------------------------------------
constexpr int kWarpsF = 8;

// Whether the next tokens' rows are on their way while the present ones are
// added, and the instances held to 128 registers so that two CTAs run on an SM
// (0: as the compiler chooses).  Measured (16 sequences of 2048 to 4096 tokens, 8
// key heads; reading ahead against two CTAs without): 64 wide with four
// query heads a warp 104 against 58 us, 128 wide with two 119 against 73.  128
// wide with four does not fit twice (ahead 124, without 113), 256 wide neither (two
// query heads: ahead 124, without 128; one: ahead 142, two CTAs 166).
constexpr bool reads_ahead(int nv, int gq) { return nv * gq <= 4 || nv == 8; }
constexpr int resident(int nv, int gq) { return nv < 8 && nv * gq == 8 ? 2 : 0; }

template <int NV, int GQ>
__global__ void __launch_bounds__(kWarpsF * 32, resident(NV, GQ)) paged_f32_kernel(const PagedParams p) {
  constexpr int E = 4, N = NV * E;
  extern __shared__ float sm[];                     // [warps][GQ][d] outputs, then [warps][GQ] m, then l
  __shared__ int64_t red[kWarpsF];
  wait_for_inputs(p);
  const int64_t total = all_tiles(p, red) * p.Hk;
  Walk w = walk_begin(p, total);
  if (threadIdx.x == 0 && !p.pieces) p.cuts[blockIdx.x].b = -1;
  if (!w.more())                                    // an empty range's part weighs nothing
    for (int g = threadIdx.x; g < p.G; g += blockDim.x) p.part_lse[(int64_t)blockIdx.x * 2 * p.G + g] = -INFINITY;
  const int64_t first = w.at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, team = lane / 8, l8 = lane % 8;
  const int groups = (p.G + GQ - 1) / GQ;           // of query heads
  const int strips = kWarpsF / groups;              // warps over the tokens of one group (G <= warps * GQ)
  const int group = warp % groups, strip = warp / groups;
  const bool working = strip < strips;
  const int nvec = p.d / E;
  float *so = sm, *smax = sm + kWarpsF * GQ * p.d, *ssum = smax + kWarpsF * GQ;

  for (; w.more(); w.next(p)) {
    const int j0 = w.first_token(), j1 = w.last_token();
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
        const float *src = (const float *)p.q + (int64_t)w.b * p.q_stride + (int64_t)(w.hk * p.G + head) * p.d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (v * 8 + l8 < nvec)
            Elt<float>::unpack(*reinterpret_cast<const uint4 *>(src + (v * 8 + l8) * E), q[g] + v * E);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) q[g][i] *= p.scale;
      }
    }
    if (working) {
      constexpr bool kAhead = reads_ahead(NV, GQ);
      uint4 nk[NV], nv[NV];
      bool next_live;
      auto read = [&](int j) {
        const int tok = j + team;
        const int64_t row = tok < j1 ? cache_row(p, pages[p.page_of(tok)], tok, w.hk) : -1;
        next_live = row >= 0;                       // a token on a page outside the pool is left out
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          nk[v] = nv[v] = make_uint4(0, 0, 0, 0);
          if (next_live && v * 8 + l8 < nvec) {
            nk[v] = ld_once((const float *)p.k + row + (v * 8 + l8) * E);
            nv[v] = ld_once((const float *)p.v + row + (v * 8 + l8) * E);
          }
        }
      };
      if (kAhead) read(j0 + strip * 4);
      for (int j = j0 + strip * 4; j < j1; j += strips * 4) {   // the same trip count for a whole warp
        uint4 kv[NV], vv[NV];
        if (!kAhead) read(j);
        const bool live = next_live;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          kv[v] = nk[v];
          vv[v] = nv[v];
        }
        if (kAhead) read(j + strips * 4);
        float s[GQ];
#pragma unroll
        for (int g = 0; g < GQ; ++g) s[g] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float x[E];
          Elt<float>::unpack(kv[v], x);
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
          Elt<float>::unpack(vv[v], x);
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
          if (v * 8 + l8 < nvec)
            *reinterpret_cast<float4 *>(so + (warp * GQ + g) * p.d + (v * 8 + l8) * E) =
                make_float4(o[g][v * E], o[g][v * E + 1], o[g][v * E + 2], o[g][v * E + 3]);
        }
        if (l8 == 0) {
          smax[warp * GQ + g] = M;
          ssum[warp * GQ + g] = L;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.G * nvec; i += kWarpsF * 32) {
      const int head = i / nvec, e = i % nvec * E, g = head % GQ;
      float M = -INFINITY, L = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < strips; ++k) M = fmaxf(M, smax[(head / GQ + k * groups) * GQ + g]);
      for (int k = 0; k < strips; ++k) {
        const int at = (head / GQ + k * groups) * GQ + g;
        const float f = smax[at] == -INFINITY ? 0.f : __expf(smax[at] - M);
        const float4 y = *reinterpret_cast<const float4 *>(so + at * p.d + e);
        L = fmaf(ssum[at], f, L);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
      }
      const float r = L == 0.f ? 0.f : 1.f / L;
      x.x *= r; x.y *= r; x.z *= r; x.w *= r;
      store_piece<float>(p, w, w.at == first ? 0 : 1, head, e, x, L == 0.f ? -INFINITY : M + logf(L));
    }
    if (threadIdx.x == 0 && w.begins()) note_cut(p, w, w.at == first ? 0 : 1, total);
    __syncthreads();
  }
  write_empty<float>(p);
  wait_for_last(p);
}

// ---------------------------------------------------------------------------
// bf16, on the warp-level matrix instruction (mma.sync m16n8k16).  The pass is
// bound by the cache's bytes: with up to 16 query heads to a key head it needs
// 2 x 16 multiply-adds per cached element at most, a tenth of what the
// instruction delivers at the memory's rate, while the CUDA cores would be
// the limit from four heads on, and a 5th-generation product, whose smallest
// tile has 64 rows, would want its weights turned round through shared
// memory.  So each warp works alone: it copies tiles of 16 tokens' keys and
// values into a ring of its own (cp.async, 16 bytes a lane, swizzled so that
// the matrix loads meet no bank twice), forms the 16 x 16 scores (query heads
// by tokens), updates the running maximum and sum, and adds the weighted
// values.  The weights enter the second product as two bf16 parts (16 bits in
// all): one part alone would add an error as large as the output's rounding.
// The ring runs on across the pieces of a CTA's range, so the joins of the
// warps' results at a piece's end leave no gap in the copies.
// ---------------------------------------------------------------------------
constexpr int kWarpsM = 4;
constexpr int kRow = 16;               // tokens per warp tile

template <int D> struct MmaShape {
  static constexpr int kPitch = D > 128 ? 512 : (D + 63) / 64 * 128;   // bytes of a token's row in shared memory
  static constexpr int kStage = 2 * kRow * kPitch;              // keys, then values
  static constexpr int kStages = D <= 64 ? 6 : 3;
  static constexpr int kCtas = D <= 128 ? 2 : 1;                // per SM
  static constexpr int kOutPitch = D + 4;                       // floats
  static constexpr size_t kSmem = (size_t)kWarpsM * kStages * kStage + 16 * kOutPitch * sizeof(float);
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A pair of weights as its nearest bf16 pair and the bf16 pair of what is left.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = Elt<__nv_bfloat16>::pack_word(a, b);
  float ha, hb;
  Elt<__nv_bfloat16>::unpack_word(hi, ha, hb);
  lo = Elt<__nv_bfloat16>::pack_word(a - ha, b - hb);
}

template <int D>
__global__ void __launch_bounds__(kWarpsM * 32, MmaShape<D>::kCtas) paged_mma_kernel(const PagedParams p) {
  using S = MmaShape<D>;
  constexpr int KS = D / 16, NT = D / 8;            // 16-wide steps and 8-wide tiles of the head's width
  extern __shared__ __align__(128) char smem[];
  __shared__ int64_t red[kWarpsM];
  __shared__ float smax[kWarpsM][16], ssum[kWarpsM][16];
  __shared__ uint32_t live_bits[kWarpsM][S::kStages];
  float *so = reinterpret_cast<float *>(smem + kWarpsM * S::kStages * S::kStage);   // [16][kOutPitch]
  wait_for_inputs(p);
  const int64_t total = all_tiles(p, red) * p.Hk;
  Walk w = walk_begin(p, total);
  if (threadIdx.x == 0 && !p.pieces) p.cuts[blockIdx.x].b = -1;
  if (!w.more())                                    // an empty range's part weighs nothing
    for (int g = threadIdx.x; g < p.G; g += blockDim.x) p.part_lse[(int64_t)blockIdx.x * 2 * p.G + g] = -INFINITY;
  const int64_t first = w.at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g4 = lane / 4, t4 = lane % 4;
  const uint32_t ring = smem_u32(smem) + warp * S::kStages * S::kStage;
  const int chunks = p.d / 8;                       // 16-byte pieces of a row

  // The copying side: tile after tile of this warp, ahead of the products.
  Walk cw = w;
  int cj = cw.more() ? cw.first_token() + warp * kRow : 0;
  int issue = 0, page_no = -1;                      // stage to fill, the next tile's page of this lane's token
  auto settle = [&]() {                             // to the warp's next tile, in a later piece if need be
    while (cw.more() && cj >= cw.last_token()) {
      cw.next(p);
      if (cw.more()) cj = cw.first_token() + warp * kRow;
    }
    if (cw.more()) {
      const int tok = cj + lane % kRow;
      page_no = tok < cw.last_token() ? p.table[(int64_t)cw.b * p.max_pages + p.page_of(tok)] : -1;
    }
  };
  settle();
  constexpr int CH = S::kPitch / 16;                // pieces of a padded row
  constexpr int kPerRow = kRow * CH / 32;           // copies per lane and tensor
  const bool aligned = p.page % kRow == 0;          // a tile never spans two pages
  auto copy_tile = [&]() {
    if (cw.more()) {
      const int64_t row = cache_row(p, page_no, cj + lane % kRow, cw.hk);
      const unsigned bits = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
      if (lane == 0) live_bits[warp][issue] = bits;
      const uint32_t dst = ring + issue * S::kStage;
      if (aligned && bits == 0xffffu) {
        // sixteen rows side by side in one page
        const int64_t at = __shfl_sync(0xffffffffu, row, 0) + (lane / CH) * p.d + (lane % CH) * 8;
        const __nv_bfloat16 *ks = (const __nv_bfloat16 *)p.k + at, *vs = (const __nv_bfloat16 *)p.v + at;
        const int step = 32 / CH * p.d;
        if (lane % CH < chunks) {
#pragma unroll
          for (int i = 0; i < kPerRow; ++i, ks += step, vs += step) {
            const int r = (i * 32 + lane) / CH;
            const uint32_t to = dst + r * S::kPitch + (((lane % CH) ^ (r & 7)) * 16);
            copy16(to, ks, true);
            copy16(to + kRow * S::kPitch, vs, true);
          }
        } else if (lane % CH * 8 < D) {             // a row's padding
#pragma unroll
          for (int i = 0; i < kPerRow; ++i) {
            const int r = (i * 32 + lane) / CH;
            const uint32_t to = dst + r * S::kPitch + (((lane % CH) ^ (r & 7)) * 16);
            copy16(to, p.k, false);
            copy16(to + kRow * S::kPitch, p.v, false);
          }
        }
      } else {
#pragma unroll 2
        for (int i = 0; i < kPerRow; ++i) {
          const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
          const int64_t off = __shfl_sync(0xffffffffu, row, r);
          const bool live = off >= 0 && c < chunks;
          const int64_t at = live ? off + c * 8 : 0;
          const uint32_t to = dst + r * S::kPitch + ((c ^ (r & 7)) * 16);
          if (c * 8 < D) {
            copy16(to, (const __nv_bfloat16 *)p.k + at, live);
            copy16(to + kRow * S::kPitch, (const __nv_bfloat16 *)p.v + at, live);
          }
        }
      }
      cj += kWarpsM * kRow;
      settle();
    }
    cp_async_commit();                              // empty groups keep the count
    issue = issue + 1 == S::kStages ? 0 : issue + 1;
  };
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) copy_tile();
  int use = 0;

  const float scale2 = p.scale * 1.44269504088896340736f;   // scores in powers of two
  for (; w.more(); w.next(p)) {
    const int j0 = w.first_token(), j1 = w.last_token();
    uint32_t q[KS][4];                              // rows g4 and g4 + 8 (query heads), zero behind G and d
    {
      const __nv_bfloat16 *src = (const __nv_bfloat16 *)p.q + (int64_t)w.b * p.q_stride + (int64_t)w.hk * p.G * p.d;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = g4 + (i & 1) * 8, col = k * 16 + t4 * 2 + (i >> 1) * 8;
          q[k][i] = row < p.G && col < p.d ? *reinterpret_cast<const uint32_t *>(src + row * p.d + col) : 0u;
        }
    }
    float o[NT][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int j = j0 + warp * kRow; j < j1; j += kWarpsM * kRow) {
      copy_tile();
      cp_async_wait<S::kStages - 1>();
      __syncwarp();
      const uint32_t kb = ring + use * S::kStage, vb = kb + kRow * S::kPitch;
      const uint32_t bits = live_bits[warp][use];
      // scores: lane rows of the matrix load: tokens (lane % 8) + 8 (lane / 16), 16-byte piece 2 k + (lane / 8) % 2
      float s[2][4] = {};
      const int kr = lane % 8 + (lane / 16) * 8, kc = (lane / 8) % 2;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        ldmatrix4(b, kb + kr * S::kPitch + (((2 * k + kc) ^ (kr & 7)) * 16));
        mma16816(s[0], q[k], b[0], b[1]);
        mma16816(s[1], q[k], b[2], b[3]);
      }
      // columns n * 8 + t4 * 2 + (i & 1) are tokens, rows g4 (i < 2) and g4 + 8 query heads
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool live = (bits >> (n * 8 + t4 * 2 + (i & 1))) & 1u;
          s[n][i] = live ? s[n][i] * scale2 : -INFINITY;
          top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
        float keep[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mn = fmaxf(m[r], top[r]);
          keep[r] = m[r] == mn ? 1.f : exp2_fast(m[r] - mn);
          m[r] = mn;
          l[r] *= keep[r];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= keep[0];
          o[n][1] *= keep[0];
          o[n][2] *= keep[1];
          o[n][3] *= keep[1];
        }
      }
      const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
      uint32_t hi[4], lo[4];                        // the weights as the second product's left operand
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float a = exp2_fast(s[n][2 * r] - base[r]), b = exp2_fast(s[n][2 * r + 1] - base[r]);
          l[r] += a + b;
          split_pair(a, b, hi[2 * n + r], lo[2 * n + r]);
        }
      }
      // values: rows of the matrix load: tokens lane % 16, piece 2 n + lane / 16
      const int vr = lane % 16, vc = lane / 16;
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        uint32_t b[4];
        ldmatrix4_t(b, vb + vr * S::kPitch + (((2 * n + vc) ^ (vr & 7)) * 16));
        mma16816(o[2 * n], hi, b[0], b[1]);
        mma16816(o[2 * n + 1], hi, b[2], b[3]);
        mma16816(o[2 * n], lo, b[0], b[1]);
        mma16816(o[2 * n + 1], lo, b[2], b[3]);
      }
      __syncwarp();                                 // the stage is read; the next copy may fill it
      use = use + 1 == S::kStages ? 0 : use + 1;
    }
    // Join the warps: common maximum, then the sums one warp after the other.
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t4 == 0) {
        smax[warp][g4 + 8 * r] = m[r];
        ssum[warp][g4 + 8 * r] = l[r];
      }
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarpsM; ++k) M = fmaxf(M, smax[k][g4 + 8 * r]);
      f[r] = m[r] == -INFINITY ? 0.f : exp2_fast(m[r] - M);
    }
#pragma unroll 1
    for (int k = 0; k < kWarpsM; ++k) {
      if (warp == k) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float2 *at = reinterpret_cast<float2 *>(so + (g4 + 8 * r) * S::kOutPitch + n * 8 + t4 * 2);
            float2 x = make_float2(o[n][2 * r] * f[r], o[n][2 * r + 1] * f[r]);
            if (k > 0) {
              const float2 y = *at;
              x.x += y.x;
              x.y += y.y;
            }
            *at = x;
          }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < p.G * (p.d / 4); i += kWarpsM * 32) {
      const int g = i / (p.d / 4), e = i % (p.d / 4) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < kWarpsM; ++k) M = fmaxf(M, smax[k][g]);
      // A warp without a finite score adds nothing, or the NaN that its sum holds: the maximum alone, which
      // passes NaN scores over, does not tell.
#pragma unroll
      for (int k = 0; k < kWarpsM; ++k)
        L += ssum[k][g] * (smax[k][g] == -INFINITY ? 0.f : exp2_fast(smax[k][g] - M));
      float4 x = *reinterpret_cast<const float4 *>(so + g * S::kOutPitch + e);
      const float r = L == 0.f ? 0.f : 1.f / L;
      x.x *= r; x.y *= r; x.z *= r; x.w *= r;
      store_piece<__nv_bfloat16>(p, w, w.at == first ? 0 : 1, g, e, x,
                                 L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f);
    }
    if (threadIdx.x == 0 && w.begins()) note_cut(p, w, w.at == first ? 0 : 1, total);
    __syncthreads();                                // the shared results are read
  }
  cp_async_wait<0>();
  write_empty<__nv_bfloat16>(p);
  wait_for_last(p);
}

// One CTA per (noted pair, query head): the parts' weights, then their sum.
// A warp takes every eighth part, 16 bytes per lane, and the warps' sums meet
// in shared memory in a fixed order.
constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const PagedParams p) {
  // A part without tokens, or none with a weight, may hold nothing and is left out.  One whose weight is too small
  // for fp32 is not: it may hold an infinity or a NaN, which shows.
  constexpr float kNone = -1.f;
  extern __shared__ float weight[];                 // [parts], then the warps' sums [kJoinWarps][d]
  __shared__ float red[kJoinWarps];
  grid_dependency_wait();
  const int c0 = blockIdx.x, g = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Cut cut = p.cuts[c0];
  if (cut.b < 0) return;
  const int parts = cut.last - c0 + 1;
  float *sums = weight + (gridDim.x + 3) / 4 * 4;
  // a later CTA's range begins with its part: slot 0
  auto row_of = [&](int k) { return ((int64_t)(c0 + k) * 2 + (k == 0 ? cut.slot : 0)) * p.G + g; };
  float M = -INFINITY;
  for (int k = threadIdx.x; k < parts; k += kJoinWarps * 32) {
    const float x = p.part_lse[row_of(k)];          // -infinity also where a CTA's range is empty
    weight[k] = x;
    M = fmaxf(M, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp] = M;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) M = fmaxf(M, red[k]);
  for (int k = threadIdx.x; k < parts; k += kJoinWarps * 32)
    weight[k] = weight[k] == -INFINITY ? kNone : expf(weight[k] - M);
  __syncthreads();
  float L = 0.f;
  for (int k = 0; k < parts; ++k) L += weight[k] == kNone ? 0.f : weight[k];
  for (int e = lane * 4; e < p.d; e += 128) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = warp; k < parts; k += kJoinWarps) {
      const float h = weight[k];
      if (h == kNone) continue;
      const float4 y = *reinterpret_cast<const float4 *>(p.part_o + row_of(k) * p.d + e);
      x.x = fmaf(y.x, h, x.x);
      x.y = fmaf(y.y, h, x.y);
      x.z = fmaf(y.z, h, x.z);
      x.w = fmaf(y.w, h, x.w);
    }
    *reinterpret_cast<float4 *>(sums + warp * p.d + e) = x;
  }
  __syncthreads();
  const float r = L == 0.f ? 0.f : 1.f / L;
  const int64_t row = (int64_t)cut.b * p.Hq + cut.hk * p.G + g;
  for (int e = threadIdx.x; e < p.d; e += kJoinWarps * 32) {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) x += sums[k * p.d + e];
    if constexpr (std::is_same<T, float>::value) ((float *)p.out)[row * p.d + e] = x * r;
    else ((__nv_bfloat16 *)p.out)[row * p.d + e] = __float2bfloat16_rn(x * r);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : M + logf(L);
}

}  // namespace

bool paged_supported(int64_t d, int dtype) {
  const int e = dtype == ATTNRES_BF16 ? 8 : 4;
  return d >= e && d <= 256 && d % e == 0;
}
// Two CTAs per SM but for bf16 heads wider than 128, whose rings fill the shared memory.
int paged_ctas(int64_t d, int dtype) { return (dtype == ATTNRES_BF16 && d > 128 ? 1 : 2) * sm_count(); }
int paged_fine_ctas(int64_t d, int dtype) { return 3 * paged_ctas(d, dtype); }

int64_t paged_workspace_bytes(int G, int64_t d, int dtype, int64_t ctas) {
  return ctas * (int64_t)sizeof(Cut) + ctas * 2 * G * (d + 1) * (int64_t)sizeof(float);
}

PagedParts paged_parts(void *workspace, int G, int64_t d, int64_t ctas) {
  float *o = reinterpret_cast<float *>(static_cast<Cut *>(workspace) + ctas);
  return {o, o + ctas * 2 * G * d};
}

cudaError_t launch_paged(const PagedArgs &a) {
  PagedParams p{};
  p.q = a.q; p.k = a.k_cache; p.v = a.v_cache; p.q_stride = a.q_stride;
  p.table = a.page_table; p.lengths = a.lengths;
  p.B = (int)a.B; p.Hq = a.Hq; p.Hk = a.Hk; p.G = a.Hq / a.Hk; p.d = a.d;
  p.page = a.page_size; p.max_pages = a.max_pages; p.num_pages = a.num_pages;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  p.scale = a.scale; p.out = a.out; p.lse = a.lse; p.out_f32 = a.out_f32; p.ready = a.ready; p.pieces = a.pieces;
  const int ctas = a.ctas;
  p.cuts = static_cast<Cut *>(a.workspace);
  const PagedParts parts = paged_parts(a.workspace, p.G, a.d, ctas);
  p.part_o = parts.o;
  p.part_lse = parts.lse;
  const dim3 grid((unsigned)ctas), join((unsigned)ctas, (unsigned)p.G);
  const size_t join_smem = ((size_t)(ctas + 3) / 4 * 4 + (size_t)kJoinWarps * a.d) * sizeof(float);
  cudaError_t err;
  if (a.dtype == ATTNRES_BF16) {
    auto go = [&](auto D) -> cudaError_t {
      using S = MmaShape<decltype(D)::value>;
      auto kern = paged_mma_kernel<decltype(D)::value>;
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
      if (e != cudaSuccess) return e;
      return launch_dependent(kern, grid, dim3(kWarpsM * 32), S::kSmem, a.stream, p);
    };
    err = a.d <= 64 ? go(std::integral_constant<int, 64>{}) : a.d <= 96 ? go(std::integral_constant<int, 96>{})
        : a.d <= 128 ? go(std::integral_constant<int, 128>{}) : a.d <= 192 ? go(std::integral_constant<int, 192>{})
        : go(std::integral_constant<int, 256>{});
    if (err != cudaSuccess || p.pieces) return err;
    return launch_dependent(paged_join_kernel<__nv_bfloat16>, join, dim3(kJoinWarps * 32), join_smem, a.stream, p);
  }
  auto go = [&](auto NV) -> cudaError_t {
    // Query heads per warp: as many as its registers hold, two of them beyond
    // 128 wide, but no more than a key head has.
    constexpr int N = decltype(NV)::value * 4, kMost = N > 16 ? 2 : 4;
    auto with = [&](auto gq) -> cudaError_t {
      constexpr int GQ = decltype(gq)::value;
      const size_t smem = (size_t)kWarpsF * GQ * (p.d + 2) * sizeof(float);
      return launch_dependent(paged_f32_kernel<decltype(NV)::value, GQ>, grid, dim3(kWarpsF * 32), smem, a.stream, p);
    };
    return p.G == 1 ? with(std::integral_constant<int, 1>{}) : p.G == 2 ? with(std::integral_constant<int, 2>{})
                    : with(std::integral_constant<int, kMost>{});
  };
  const int nv = (a.d / 4 + 7) / 8;
  err = nv <= 2 ? go(std::integral_constant<int, 2>{}) : nv <= 4 ? go(std::integral_constant<int, 4>{})
                : go(std::integral_constant<int, 8>{});
  if (err != cudaSuccess || p.pieces) return err;
  return launch_dependent(paged_join_kernel<float>, join, dim3(kJoinWarps * 32), join_smem, a.stream, p);
}

}  // namespace attnres
