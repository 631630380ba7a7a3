// shared_tc.cu -- the parts of a shared prefix on the 5th-generation tensor
// cores (bf16; see shared.cu for the operator).
//
// A CTA takes 256 rows (query heads of one key head, over the sequences) as
// two tiles of 128, and one range of the prefix's tokens, 128 at a time (heads
// wider than 128: one tile, and 64):
//   S = Q K^T (M 128, N 128, K d),  P = 2^(scale S - m),  O += P V (M 128, N d, K 128)
// S and O are fp32 in tensor memory; two threads have a row of S, half of the
// tokens each (113 us where one per row took 121); P, rounded to bf16, goes back
// to tensor memory over S, as the left operand of the second product.  While
// one tile's weights are formed, the tensor cores work on the other's products.
//
// m is a reference, not the maximum: it moves, to the maximum, only when the
// weights that a thread forms in a step add up to more than 2^10 (and at the
// first step), and O and the sum are rescaled then; fp32 and bf16 hold what lies
// above it.  So a step needs no maximum.  Rounding P to bf16 adds an error of
// the size of the output's own rounding; the sum is that of the unrounded
// weights.  Two parts of P, as the own tokens' weights have them (paged.cu),
// leave only the output's rounding (0.0017 of the outputs' norm in place of
// 0.0019 to 0.0023), but they make the second product twice as long, and the
// products bind: with 640 threads, whose softmax then has the registers for it,
// 64 questions about 131071 tokens took 164 us instead of 127, 256 chats behind
// 8192 278 instead of 259, 64 behind 8192 with heads of 128 51 instead of 46.
//
// Roles: the two tiles' softmax (two warpgroups each); copies (cp.async of 16
// bytes a lane, a row's page looked up by its own lane, into a ring of tiles
// with the 128-byte swizzle; tokens behind the range or on no page arrive as
// zeros and are masked); and one thread that issues the products.
//
// What bounds it: the products.  One of 128 x 128 x 16 with both operands in
// shared memory takes 94 cycles of the 64 that the tensor cores need (8 KB at
// 87 bytes a cycle, beside the copies' 19), and with the hand-overs between the
// roles a step of both tiles takes some 3400 cycles for 2048.  Measured on GB300:
// 512 rows and 131071 tokens, four key heads of 128: 102 us on 152 SMs (1.35
// PFLOP/s, 67 % of cuBLAS's), 119 on the 136 that the launch takes; 1792 rows
// and 8192 tokens, eight key heads: 67 to 72 us on 112 SMs.  Measured and not
// kept (whole call of the first, 136 us when these were tried): tiles copied by
// tensor-map boxes of 32 rows 136; steps of 80 tokens, whose P fits beside S, so
// that the next scores need not wait for the weights' use, 148; a thread per
// tile that issues, 148; a sixth of the exponentials as polynomials 161.
//
// Every wait is bounded: one that runs out records a flag and an abort mark in
// shared memory, on which every other wait returns at once; what is in flight
// is drained and the CTA ends.
#include "common.cuh"
#include "launch.h"
#include "shared.cuh"
#include "tcgen05.cuh"

ATTNRES_DEFINE_ERROR_FLAG(take_error_shared)

namespace attnres {
namespace {

constexpr int kTileRows = 128;             // rows of a tile: two threads have one
constexpr int kThreads = 768;
constexpr uint32_t kQBlock = 128 * 128;    // bytes: 128 rows of 64 bf16 columns
constexpr int kRegs = 80;                  // a thread's registers at the launch, then the roles' shares
constexpr int kRegsSoftmax = 96, kRegsCopy = 48, kRegsMma = 48;
static_assert(4 * kRegsSoftmax + kRegsCopy + kRegsMma <= 6 * kRegs, "more registers than the launch has");
constexpr float kMost = 1024.f;            // the sum of a thread's weights of a step that the reference may stay for
constexpr int kMasks = 4;                  // steps whose masks are kept

// Heads of up to 64, 128 and 256 elements.  The last take half of the tensor
// memory for one tile's O and half of a step's tokens.
template <int D> struct Layout {
  static constexpr int kTiles = D <= 128 ? 2 : 1, kRows = kTiles * kTileRows;
  static constexpr int kKeys = D <= 128 ? 128 : 64;                   // tokens of a step
  static constexpr uint32_t kBlock = kKeys * 128;                     // bytes: a step's rows of 64 bf16 columns
  static constexpr uint32_t kQTile = D / 64 * kQBlock, kTile = D / 64 * kBlock;
  static constexpr int kRing = D == 64 ? 6 : 5;                       // tiles of K and V, in turn
  static constexpr uint32_t kOffRing = kTiles * kQTile;
  static constexpr uint32_t kOffMask = kOffRing + kRing * kTile;
  static constexpr uint32_t kOffRow = kOffMask + kMasks * 16;         // a float per row
  static constexpr uint32_t kOffBar = kOffRow + kRows * 4;
  // barriers
  static constexpr int kFull = 0, kEmpty = kRing, kMask = 2 * kRing, kScores = kMask + kMasks, kWeights = kScores + 2,
                       kOut = kWeights + 2, kDrain = kOut + 2, kBars = kDrain + 1;
  static constexpr uint32_t kOffCtl = kOffBar + kBars * 8;
  static constexpr uint32_t kBytes = kOffCtl + 16 + 1024;             // and the alignment's slack
  static_assert(kBytes <= 232448, "what a CTA can have");
  // Tensor memory columns: S (P over its first half) of the tiles, O.
  static constexpr uint32_t kColO = 256;
  static_assert(kTiles * kKeys <= (int)kColO && kColO + kTiles * D <= 512, "tensor memory");
};

// This thread's arrival at a barrier, once its copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// The exponents of 32 tokens of a row, from scores, reference and mask, two at
// a time to f.
template <bool MASKED, typename F>
__device__ __forceinline__ void exponents(const uint32_t (&s)[32], uint64_t scale2, uint64_t minus, uint32_t mask, F f) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a, b;
    unpair(fma2((uint64_t)s[2 * i + 1] << 32 | s[2 * i], scale2, minus), a, b);
    if (MASKED) {
      if (!(mask >> (2 * i) & 1u)) a = -INFINITY;
      if (!(mask >> (2 * i + 1) & 1u)) b = -INFINITY;
    }
    f(i, a, b);
  }
}

// Two warps that share rows: a barrier, and one with a vote of their 64 threads.
__device__ __forceinline__ void pair_barrier(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool any_of_pair(int id, bool x) {
  uint32_t any;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.or.pred q, %1, 64, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(any) : "r"(id), "r"(x ? 1u : 0u) : "memory");
  return any != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ PrefixParams p) {
  using L = Layout<D>;
  constexpr int NR = L::kRing, kKeys = L::kKeys;
  extern __shared__ unsigned char smem_raw[];
  p.begin();
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(sm);
  volatile uint32_t *masks = reinterpret_cast<uint32_t *>(sm + L::kOffMask);
  volatile uint32_t *ctl = reinterpret_cast<uint32_t *>(sm + L::kOffCtl);      // TMEM address, skip, abort
  auto bar = [&](int b) { return base + L::kOffBar + 8u * b; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp >> 2, quad = warp & 3;

  const int all = p.B * p.G, tiles = (all + L::kRows - 1) / L::kRows;
  const int hk = blockIdx.x / tiles, row0 = (blockIdx.x - hk * tiles) * L::kRows, split = blockIdx.y;
  const int active = L::kTiles == 2 && all - row0 > kTileRows ? 2 : 1;                          // tiles with rows
  int j0, j1;
  p.range<kKeys>(p.tokens(), split, j0, j1);
  const int steps = j1 > j0 ? (j1 - j0 + kKeys - 1) / kKeys : 0;
  if (steps == 0) {                        // an empty range's part weighs nothing
    for (int i = threadIdx.x; i < L::kRows && row0 + i < all; i += kThreads)
      p.part_lse[p.part(split, row0 + i, hk)] = -INFINITY;
    return;
  }

  if (threadIdx.x == 0) {
    ctl[1] = *reinterpret_cast<volatile unsigned int *>(&g_error_flag) != 0 ? 1u : 0u;
    ctl[2] = 0;
    for (int i = 0; i < NR; ++i) {
      mbar_init(bar(L::kFull + i), 128);
      mbar_init(bar(L::kEmpty + i), 1);
    }
    for (int i = 0; i < kMasks; ++i) mbar_init(bar(L::kMask + i), 4);
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(L::kScores + g), 1);
      mbar_init(bar(L::kWeights + g), 8);
      mbar_init(bar(L::kOut + g), 1);
    }
    mbar_init(bar(L::kDrain), 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (ctl[1]) return;                      // an earlier error has not been taken: nothing is issued
  constexpr int kMmaWarp = 20;
  if (warp == kMmaWarp) tmem_alloc(base + L::kOffCtl, 512);
  // the queries, zero behind the batch and behind d
  {
    const int nvec = p.d / 8;
    for (int i = threadIdx.x; i < L::kRows * (D / 8); i += kThreads) {
      const int r = i / (D / 8) % kTileRows, c = i % (D / 8), tile = i / (D / 8) / kTileRows, row = row0 + tile * kTileRows + r;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < all && c < nvec)
        x = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)p.q + (int64_t)(row / p.G) * p.q_stride +
                                             (int64_t)(hk * p.G + row % p.G) * p.d + c * 8);
      *reinterpret_cast<uint4 *>(sm + tile * L::kQTile + c / 8 * kQBlock + r * 128 + ((c % 8) ^ (r & 7)) * 16) = x;
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl[0];

  // Wait for a phase; false once any wait of the CTA has run out.
  auto wait = [&](int which, uint32_t parity) -> bool {
    const uint32_t at = bar(which);
    if (mbar_try(at, parity & 1)) return true;
    const long long t0 = clock64();
    while (!mbar_try(at, parity & 1)) {
      if (ctl[2]) return false;
      if (clock64() - t0 > p.wait_limit) {
        ctl[2] = 1;
        raise_timeout();
      }
    }
    return true;
  };

  if (group == 4) {
    // ---------------- copies: a quarter of every tile's rows per warp ----------------
    share_registers<kRegsCopy, kRegs>();
    constexpr int CH = D / 8, kPer = 32 / CH, kWord = kKeys / 4;   // 16-byte pieces of a row, rows per instruction, rows
    const int c = lane % CH, sub = lane / CH;
    const bool inside = c * 8 < p.d;
    const bool side = p.page % kWord == 0 && p.d == D;  // the warp's tokens never span two pages, and rows have no padding
    const uint32_t mine = c / 8 * L::kBlock + (quad * kWord + sub) * 128;
    // 16-byte piece c % 8 of row k kPer + sub of the warp, in the swizzle's place
    auto swizzled = [&](int k) -> uint32_t { return ((c % 8) ^ ((k * kPer + sub) & 7)) * 16; };
    bool alive = false;                                 // all of the warp's tokens are on a page
    auto page_row = [&](int step) -> int64_t {          // this lane's token of a step
      const int j = j0 + step * kKeys + quad * kWord + lane;
      return lane < kWord && j < j1 ? p.row(j, hk) : -1;
    };
    int64_t next = page_row(0);
    bool ok = true;
    for (int i = 0; ok && i < steps; ++i) {
      const int64_t row = next;
      if (i + 1 < steps) next = page_row(i + 1);
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int s = 2 * i + kv;
        if (s >= NR && !(ok = __all_sync(0xffffffffu, wait(L::kEmpty + s % NR, s / NR - 1)))) break;
        if (kv == 0) {
          const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
          alive = live == (uint32_t)((1ull << kWord) - 1);
          if (lane == 0) {
            masks[i % kMasks * 4 + quad] = live;
            mbar_arrive(bar(L::kMask + i % kMasks));
          }
        }
        const char *from = reinterpret_cast<const char *>(kv ? p.v : p.k);
        const uint32_t to = base + L::kOffRing + s % NR * L::kTile + mine;
        if (side && alive) {
          // the warp's rows lie side by side in one page
          const char *src = from + (__shfl_sync(0xffffffffu, row, 0) + sub * p.d + c * 8) * 2;
          const int step = kPer * p.d * 2;
#pragma unroll
          for (int k = 0; k < kWord / kPer; ++k, src += step) copy16(to + k * kPer * 128 + swizzled(k), src);
        } else {
#pragma unroll 4
          for (int k = 0; k < kWord / kPer; ++k) {
            const int64_t at = __shfl_sync(0xffffffffu, row, k * kPer + sub);
            const bool live = at >= 0 && inside;
            copy16(to + k * kPer * 128 + swizzled(k), from + (live ? (at + c * 8) * 2 : 0), live);
          }
        }
        copies_arrive(bar(L::kFull + s % NR));
      }
    }
    cp_async_wait<0>();
  } else if (group == 5) {
    share_registers<kRegsMma, kRegs>();
    if (warp == kMmaWarp && elect_one()) {
      // ---------------- products ----------------
      const int ks = (p.d + 15) / 16;                   // K steps over d
      auto scores = [&](int g, int s) {                 // S of tile g with the K tile s
        const Desc q = desc_k(base + g * L::kQTile), k = desc_k(base + L::kOffRing + s % NR * L::kTile);
#pragma unroll 2
        for (int x = 0; x < ks; ++x)
          mma_bf16(tmem + g * kKeys, q.at(x / 4 * kQBlock + x % 4 * 32), k.at(x / 4 * L::kBlock + x % 4 * 32),
                   idesc_bf16(128, kKeys), x > 0);
        mma_commit(bar(L::kScores + g));
      };
      // A tile's copies are seen here through its barrier; the fence orders them before the products' reads.
      auto landed = [&](int s) -> bool {
        if (!wait(L::kFull + s % NR, s / NR)) return false;
        fence_async_smem();
        return true;
      };
      bool ok = landed(0);
      if (ok) {
        tc_fence_after();
        for (int g = 0; g < active; ++g) scores(g, 0);
        mma_commit(bar(L::kEmpty));
      }
      for (int i = 0; ok && i < steps; ++i) {
        const int sv = 2 * i + 1, sk = 2 * i + 2;
        for (int g = 0; ok && g < active; ++g) {
          if (!(ok = (g > 0 || landed(sv)) && wait(L::kWeights + g, i))) break;
          tc_fence_after();
          const Desc v = desc_mn(base + L::kOffRing + sv % NR * L::kTile, L::kBlock);
#pragma unroll
          for (int x = 0; x < kKeys / 16; ++x)
            mma_bf16_ts(tmem + L::kColO + g * D, tmem + g * kKeys + 8 * x, v.at(x * 2048), idesc_bf16(128, D) | kIdescMnB, i + x > 0);
          mma_commit(bar(L::kOut + g));
          if (g + 1 == active) mma_commit(bar(L::kEmpty + sv % NR));
          if (i + 1 == steps) continue;
          // the next scores go over the weights that this product reads
          if (!(ok = (g > 0 || landed(sk)) && wait(L::kOut + g, i))) break;
          tc_fence_after();
          scores(g, sk);
          if (g + 1 == active) mma_commit(bar(L::kEmpty + sk % NR));
        }
      }
      // every product issued has completed before the memory it uses goes
      mma_commit(bar(L::kDrain));
      if (!mbar_wait_for(bar(L::kDrain), 0, kDrainLimitCycles)) raise_timeout();
    }
    __syncwarp();
  } else {
    // ---------------- softmax: two threads per row, half of a step's tokens each ----------------
    share_registers<kRegsSoftmax, kRegs>();
    const int g = group >> 1, half = group & 1, row = row0 + g * kTileRows + quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16), at_s = lanes + g * kKeys, at_o = lanes + L::kColO + g * D + half * (D / 2);
    constexpr int kHalf = kKeys / 2;
    volatile float *slot = reinterpret_cast<float *>(sm + L::kOffRow) + g * kTileRows + quad * 32 + lane;
    const int both = 1 + g * 4 + quad;                  // the barrier of the two warps with these rows
    // f of the two threads' values (the first half's, the second's), for both
    auto joined = [&](float x, auto f) -> float {
      if (half == 0) *slot = x;
      pair_barrier(both);
      if (half == 1) *slot = f(*slot, x);
      pair_barrier(both);
      return *slot;
    };
    const float scale = p.scale * 1.44269504088896340736f;               // scores in powers of two
    const uint64_t scale2 = pair(scale, scale);
    float m = -INFINITY;                                // the reference, the same in both threads
    float l = 0.f;
    if (g < active) {
      for (int i = 0; i < steps; ++i) {
        wait(L::kMask + i % kMasks, i / kMasks);
        uint32_t mask0 = masks[i % kMasks * 4 + half * 2], mask1 = masks[i % kMasks * 4 + half * 2 + 1];
        if (kHalf == 32) mask0 |= mask1 << 16;          // of 32 tokens each
        wait(L::kScores + g, i);
        __syncwarp();
        tc_fence_after();
        uint32_t w[kHalf / 2], a[32], b[32];
        // f of the exponents of this thread's tokens
        auto each = [&](auto f) {
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t minus = pair(-ref, -ref);
          tmem_ld32(at_s + half * kHalf, a);
          tmem_wait_ld();
          if (kHalf == 64) tmem_ld32(at_s + half * kHalf + 32, b);
          if (mask0 == 0xffffffffu) exponents<false>(a, scale2, minus, 0, f);
          else exponents<true>(a, scale2, minus, mask0, f);
          if constexpr (kHalf == 64) {
            tmem_wait_ld();
            auto behind = [&](int i, float x, float y) { f(i + 16, x, y); };
            if (mask1 == 0xffffffffu) exponents<false>(b, scale2, minus, 0, behind);
            else exponents<true>(b, scale2, minus, mask1, behind);
          }
        };
        uint64_t sum, sum1;
        auto form = [&]() {
          sum = sum1 = 0;
          each([&](int i, float x, float y) {
            x = exp2_fast(x);
            y = exp2_fast(y);
            if (i & 1) sum1 = add2(sum1, pair(x, y));
            else sum = add2(sum, pair(x, y));
            w[i] = Elt<__nv_bfloat16>::pack_word(x, y);
          });
          sum = add2(sum, sum1);
        };
        form();
        // The vote also says that both halves have read their scores, which the weights go over.
        tc_fence_before();
        if (any_of_pair(both, m == -INFINITY || pair_sum(sum) > kMost)) {
          // a new reference: the maximum, where it has passed the old one
          float top = -INFINITY;
          const float old = m;
          each([&](int, float x, float y) { top = fmaxf(top, fmaxf(x, y)); });
          top = joined(top, [](float x, float y) { return fmaxf(x, y); });
          if (top > (old == -INFINITY ? -INFINITY : 0.f)) m = (old == -INFINITY ? 0.f : old) + top;
          const float keep = m == old ? 1.f : exp2_fast(old - m);
          l *= keep;
          __syncwarp();                                 // what each lane chose for itself is behind: loads and stores of the warp
          if (i > 0) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float x[16];
              tmem_ld16(at_o + q * 16, x);
              tmem_wait_ld();
              uint32_t y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(x[e] * keep);
              tmem_st16(at_o + q * 16, y);
            }
          }
          form();
          tc_fence_before();
          pair_barrier(both);
        }
        tc_fence_after();
        l += pair_sum(sum);
#pragma unroll
        for (int q = 0; q < kHalf / 32; ++q) {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = w[q * 16 + e];
          tmem_st16(at_s + half * (kHalf / 2) + q * 16, y);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kWeights + g));
      }
      l = joined(l, [](float a, float b) { return a + b; });
      wait(L::kOut + g, steps - 1);
      __syncwarp();
      tc_fence_after();
      const float f = l == 0.f ? 0.f : 1.f / l;
      const int64_t at = row < all ? p.part(split, row, hk) : 0;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float x[16];
        __syncwarp();                                   // lanes behind the batch store nothing; the loads take all of them
        tmem_ld16(at_o + q * 16, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const int c = half * (D / 2) + q * 16 + e;
          if (row < all && c < p.d)
            *reinterpret_cast<float4 *>(p.part_o + at * p.d + c) = make_float4(x[e] * f, x[e + 1] * f, x[e + 2] * f, x[e + 3] * f);
        }
      }
      __syncwarp();
      if (row < all && half == 0) p.part_lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The launch's registers have to be the number that the roles' shares start
// from, or a role would wait for registers that nobody gives.
template <int D> bool registers_as_planned() {
  static const bool ok = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, shared_tc_kernel<D>) == cudaSuccess && a.numRegs == kRegs;
  }();
  return ok;
}

template <int D> cudaError_t launch(const PrefixParams &p, cudaStream_t stream) {
  using L = Layout<D>;
  if (!registers_as_planned<D>()) return cudaErrorInvalidConfiguration;
  const cudaError_t e = allow_smem<shared_tc_kernel<D>>(L::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)p.B * p.G + L::kRows - 1) / L::kRows;
  return launch_dependent(shared_tc_kernel<D>, dim3((unsigned)(tiles * p.Hk), (unsigned)p.splits), dim3(kThreads), L::kBytes,
                          stream, p);
}

}  // namespace

// Ranges of the prefix with the least time, in microseconds: a CTA's start and
// end, its steps (of one tile or two), and the parts that the join reads and
// writes; and the own tokens' kernel, which runs beside the prefix's CTAs where
// they leave a tenth of the SMs free, and else behind them: 4 and its bytes at
// 6 TB/s, where there are own tokens, and no more than 18 (beyond that it
// outlasts them either way).  64 questions about 131071 tokens, us with 16 SMs
// left and with none: no own tokens 125 and 116, a page of 64 at most 126 and 120,
// 256 126 and 125, 512 126 and 132 (137 with 8 left, 132 with 24), 1024 143 and 139, 2048
// 159 and 158; two key heads and 65536 tokens, 1024 own ones 58 and 61; four short
// chats 14 and 18.
int shared_tc_splits(int64_t B, int G, int Hk, int64_t d, int64_t tokens, int64_t own) {
  const int rows = d <= 128 ? Layout<128>::kRows : Layout<256>::kRows, keys = d <= 128 ? Layout<128>::kKeys : Layout<256>::kKeys;
  const int64_t items = (B * G + rows - 1) / rows * Hk, steps = (tokens + keys - 1) / keys;
  const double row_us = (double)B * G * Hk * d * 8e-6 / 4., step_us = B * G > kTileRows && d <= 128 ? 1.8 : 1.2;
  const int64_t slots = sm_count();
  const double own_us = own > 0 ? 4. + (double)B * Hk * own * d * 4. / 6e6 : 0., beside_us = own_us < 18. ? own_us : 18.;
  int best = 1;
  double least = 1e300;
  for (int n = 1; n <= kMaxPrefixParts && n <= steps; ++n) {
    const int64_t waves = (items * n + slots - 1) / slots, free = waves * slots - items * n;
    const double cost = (double)waves * (8. + step_us * (double)((steps + n - 1) / n)) + row_us * n + (10 * free < slots ? beside_us : 0.);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

cudaError_t launch_shared_tc(const PrefixParams &p, cudaStream_t stream) {
  return p.d <= 64 ? launch<64>(p, stream) : p.d <= 128 ? launch<128>(p, stream) : launch<256>(p, stream);
}

}  // namespace attnres
