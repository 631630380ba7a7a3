// shared.cuh -- what the kernels of a shared prefix's parts have in common.
#pragma once

#include "common.cuh"
#include <stdint.h>

namespace attnres {

// Most ranges of the prefix: what a part adds to the workspace and to the
// join's reads grows with them.  With one key head and up to 256 rows they are
// fewer than the SMs.
constexpr int kMaxPrefixParts = 64;

struct PrefixParams {
  const void *q, *k, *v;
  int64_t q_stride;                      // elements from one sequence's queries to the next
  const int32_t *table, *length;         // the prefix's pages; its tokens
  int B, Hq, Hk, G, d;
  int page, page_shift, most;            // page_shift: log2(page), or -1; most: tokens that the table covers
  int64_t num_pages;
  float scale;
  float *part_o, *part_lse;              // [splits][B Hq][d], [splits][B Hq]
  int splits;
  long long wait_limit;                  // SM clock cycles a wait of the tensor-core kernel may take
  Mark ready;                            // the follower's (none: it waits for this kernel's end)

  // What every thread of a prefix's kernel starts with: the wait for what
  // came before.  Then the own tokens' kernel may start; with `ready` it goes
  // to work at once, and sees by the mark that this thread has waited.
  __device__ __forceinline__ void begin() const {
    grid_dependency_wait();
    if (threadIdx.x != 0) return;
    if (ready.at && blockIdx.x == 0 && blockIdx.y == 0) ready.raise();
    launch_dependents();
  }

  // The prefix's tokens, held within what the table covers.
  __device__ __forceinline__ int tokens() const {
    const int n = *length;
    return n < 0 ? 0 : n < most ? n : most;
  }
  // Range `split` of the first n tokens, in whole tiles of TILE.
  template <int TILE> __device__ __forceinline__ void range(int n, int split, int &from, int &to) const {
    const int64_t tiles = (n + TILE - 1) / TILE;
    from = (int)(tiles * split / splits) * TILE;
    to = min(n, (int)(tiles * (split + 1) / splits) * TILE);
  }
  // The cache row of token j as a number and as an element offset; -1 for a page outside the pool.
  __device__ __forceinline__ int64_t row_number(int j, int hk) const {
    const int64_t pg = table[page_shift >= 0 ? j >> page_shift : j / page];
    if (pg < 0 || pg >= num_pages) return -1;
    return (pg * Hk + hk) * page + (page_shift >= 0 ? j & (page - 1) : j % page);
  }
  __device__ __forceinline__ int64_t row(int j, int hk) const {
    const int64_t r = row_number(j, hk);
    return r < 0 ? r : r * d;
  }
  // The part's row of row r (sequence r / G, head r % G of key head hk).
  __device__ __forceinline__ int64_t part(int split, int r, int hk) const {
    return ((int64_t)split * B + r / G) * Hq + hk * G + r % G;
  }
};

// The parts on the 5th-generation tensor cores (bf16): how many, and the launch.  tokens, own: what the prefix's table
// and a sequence's cover.
int shared_tc_splits(int64_t B, int G, int Hk, int64_t d, int64_t tokens, int64_t own);
cudaError_t launch_shared_tc(const PrefixParams &p, cudaStream_t stream);

}  // namespace attnres
