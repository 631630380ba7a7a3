// linear_tc.cu -- the chunks of linear attention with one decay per head on
// the 5th-generation tensor cores (bf16 inputs; see linear.cu for the form
// F(a, b, c; first) and the segments).
//
// Per chunk of 64 tokens, with S the state before it (da x dc, fp32):
//   P  = a b^T, masked and decayed                    (M 64,  N 64,  K da)
//   O^T = S^T a^T (weighted by token) + c^T P^T       (M dc,  N 64,  K da; K 64)
//   S  <- lambda^n S + b^T (w c), w_j = lambda^{n-1-j} (M da,  N dc,  K 64)
// The outputs are formed transposed, so that every product but the small P
// has M = 128, the full rate.  c^T, S^T and b^T are MN-major operands: the
// tiles are used as they lie in memory, nothing is transposed by threads.
//
// Accuracy.  The state has to keep fp32 accuracy over any number of chunks.
// w c is therefore split into three bf16 parts (24 bits), so its product is
// exact to fp32's rounding, and S itself lives in fp32 registers (a thread
// per row and half of the columns).  P and the copy of S that forms the
// outputs are rounded to bf16 once: each adds an error of the size of the
// output's own rounding at most.
//
// Roles of a CTA, one per SM (a warpgroup of four warps each, but for the
// last): the state (a thread per row of S, all its columns in registers); two
// for the weighted parts; P; the outputs; and two warps that copy tiles
// (cp.async, 16 bytes a lane, straight into the swizzled layout, rows behind
// the sequence and columns behind the width as zeros; tensor-map copies are
// served one box at a time per CTA and would cap one CTA per SM at about
// 4.2 TB/s) beside two threads that issue products, one the updates of S and
// one all others, so that neither waits for the other's operands.  A warp runs
// its dependent instructions one in five cycles or so, so what counts is how
// few instructions each role needs per chunk, and that the roles run side by
// side: with eight warps doing all of the work in turn a chunk took 7900
// cycles.
//
// Every wait is bounded: one that runs out records a flag and an abort mark
// in shared memory, on which every other wait returns at once; the issuing
// roles stop and drain what they have in flight, and the CTA ends.
#include "linear.cuh"
#include "tcgen05.cuh"

ATTNRES_DEFINE_ERROR_FLAG(take_error_linear)

namespace attnres {
namespace {

constexpr int kC = kChunk;
constexpr uint32_t kTile = kC * 128 * 2;              // bytes: 64 tokens x 128 columns, two blocks of 64 columns
constexpr uint32_t kBlock = kTile / 2;
constexpr int kStep = 16;                             // tokens per step of the weighted parts (an MMA's K)
constexpr uint32_t kPart = kStep * 128 * 2;           // a part of them: two blocks of 64 columns
constexpr uint32_t kSBlock = 128 * 128;               // 64 columns of S's 128 rows
constexpr int kOutPitch = 272;                        // bytes per token of the output staging (no bank met twice)
constexpr int kCopiers = 2;                           // warps

// The main kernel's warpgroups: S, parts, parts, P, outputs, copies + products;
// the states' kernel: S, parts, parts, copies + products.
template <bool STATES> struct Shape {
  static constexpr int kGroups = STATES ? 4 : 6;
  static constexpr int kThreads = kGroups * 128;
  static constexpr int kStages = STATES ? 6 : 3;
  // Registers per thread: as launched (checked at the launch), then each
  // role's share; their sum stays within the launch's.
  static constexpr int kRegs = STATES ? 128 : 80;
  static constexpr int kRegsS = STATES ? 184 : 168, kRegsParts = STATES ? 96 : 56, kRegsP = 72, kRegsOut = 88,
                       kRegsCopy = STATES ? 96 : 40;
  static_assert(kRegsS + 2 * kRegsParts + (STATES ? 0 : kRegsP + kRegsOut) + kRegsCopy <= kGroups * kRegs,
                "more registers than the launch has");
  static constexpr uint32_t kStage = (STATES ? 2 : 3) * kTile;      // b, c, [a]
  static constexpr uint32_t kOffParts = kStages * kStage;
  static constexpr uint32_t kOffP = kOffParts + 2 * 3 * kPart;
  static constexpr uint32_t kOffS = kOffP + (STATES ? 0 : kC * 128);
  static constexpr uint32_t kOffOut = kOffS + (STATES ? 0 : 2 * kSBlock);
  static constexpr uint32_t kOffPow = kOffOut + (STATES ? 0 : kC * kOutPitch);
  static constexpr uint32_t kOffBar = kOffPow + 72 * 4;
  static constexpr uint32_t kBytes = kOffBar + 30 * 8 + 1024;       // and the alignment's slack
};

// Tensor memory columns: the update of S by the chunk's parity, P, the outputs' two sums.
constexpr uint32_t kColKV = 0, kColP = 256, kColInter = 320, kColIntra = 384;

// Barriers, one phase per chunk (full, empty and parts: one per use of a
// stage or buffer).  A waiter may be at most one phase behind its barrier, or
// the parity deceives it; the updates of S, which run up to two chunks ahead
// of the state, therefore have a pair of each, by the chunk's parity.
enum Bar { kFull = 0, kEmpty = 6, kPartsFull = 12, kPartsEmpty = 14, kKV = 16, kKVFree = 18, kPV = 20, kOutFree, kQK, kSReady,
           kQS, kPReady, kDrain, kDrainKV, kBars };

// A role's share of the registers: it gives some of the launch's back, or
// takes some that others have given.
template <int N, int LAUNCHED> __device__ __forceinline__ void share_registers() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "what the instruction takes");
  if constexpr (N < LAUNCHED) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
  if constexpr (N > LAUNCHED) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}
// The outputs' four warps.
__device__ __forceinline__ void output_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Descriptors from a tile's address: K-major tiles (groups of eight rows 1024
// bytes apart) and MN-major ones; `d` moves along them by whole 16-byte units.
struct Desc {
  uint32_t lo;
  __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
    return ((uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32) | (lo + (bytes >> 4));
  }
};
__device__ __forceinline__ Desc desc_k(uint32_t addr) { return {((addr & 0x3FFFFu) >> 4) | 1u << 16}; }
__device__ __forceinline__ Desc desc_mn(uint32_t addr, uint32_t lbo) { return {((addr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16}; }

// Two fp32 values in a register pair, from and to bf16 pairs.
__device__ __forceinline__ uint64_t widen(uint32_t w) { return ((uint64_t)(w & 0xffff0000u) << 32) | (uint64_t)(w << 16); }
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  unpair(v, lo, hi);
  return Elt<__nv_bfloat16>::pack_word(lo, hi);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 32 columns of this thread's tensor-memory lane, as pairs.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint64_t (&v)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = ((uint64_t)r[2 * i + 1] << 32) | r[2 * i];
}
// 16 lanes x 32 columns spread over the warp as four matrix fragments of 16 x
// 8: pair 2 i + j of a thread is row lane / 4 + 8 j, columns 8 i + 2 (lane %
// 4) and the next.
__device__ __forceinline__ void tmem_ld_fragments(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ uint64_t joined(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }
// Four 8 x 8 bf16 fragments to shared memory, as they lie or transposed;
// lane l names row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
               ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
__device__ __forceinline__ void stmatrix4_t(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
               ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

template <bool STATES>
__global__ void __launch_bounds__(Shape<STATES>::kThreads, 1) linear_tc_kernel(const LinearParams p) {
  using L = Shape<STATES>;
  extern __shared__ unsigned char smem_raw[];
  grid_dependency_wait();
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(sm);
  float *pw = reinterpret_cast<float *>(sm + L::kOffPow);                       // lambda^0 .. lambda^65
  volatile uint32_t *ctl = reinterpret_cast<uint32_t *>(sm + L::kOffBar + kBars * 8);   // TMEM address, skip, abort
  auto bar = [&](int b) { return base + L::kOffBar + 8u * b; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp >> 2, quad = warp & 3;

  const int seg = blockIdx.x % p.nseg;
  const int64_t bh = blockIdx.x / p.nseg, b = bh / p.H;
  const int h = (int)(bh % p.H);
  const int64_t n = seq_length(p, b);
  const int64_t begin = seg * p.seg_len, end = min(p.T, begin + p.seg_len), stop = min(n, end);
  const float g = p.log_decay[h];
  int64_t from = begin;
  if (STATES && g < 0.f && stop > begin) {
    // Tokens whose weight in the segment's last state is below fp32's
    // smallest number (e^-104) add exactly nothing: start behind them.
    const float reach = 104.f / -g;
    if (reach < (float)(stop - begin)) from = max(begin, (stop - 1 - (int64_t)reach) / kC * kC);
  }
  const int chunks = stop > from ? (int)((stop - from + kC - 1) / kC) : 0;
  const int tail = chunks > 0 ? (int)(stop - from - (int64_t)(chunks - 1) * kC) : 0;   // tokens of the last chunk

  if (threadIdx.x == 0) {
    ctl[1] = *reinterpret_cast<volatile unsigned int *>(&g_error_flag) != 0 ? 1u : 0u;
    ctl[2] = 0;
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar(kFull + i), kCopiers * 32);
      mbar_init(bar(kEmpty + i), STATES ? 1 : 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kPartsFull + i), 8);
      mbar_init(bar(kPartsEmpty + i), 1);
      mbar_init(bar(kKV + i), 1);
      mbar_init(bar(kKVFree + i), 4);
    }
    mbar_init(bar(kQK), 1);
    mbar_init(bar(kSReady), 4);
    mbar_init(bar(kQS), 1);
    mbar_init(bar(kPV), 1);
    mbar_init(bar(kOutFree), 4);
    mbar_init(bar(kPReady), 4);
    mbar_init(bar(kDrain), 1);
    mbar_init(bar(kDrainKV), 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 66) pw[threadIdx.x] = decay_pow(g, threadIdx.x);
  __syncthreads();
  if (ctl[1]) return;                                 // an earlier error has not been taken: nothing is issued
  constexpr int kMmaWarp = L::kGroups * 4 - 1;
  if (warp == kMmaWarp) tmem_alloc(base + L::kOffBar + kBars * 8, STATES ? 256 : 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl[0];

  // Wait for the phase; false once any wait of the CTA has run out.
  auto wait = [&](int which, uint32_t parity) -> bool {
    if (mbar_try(bar(which), parity & 1)) return true;
    const long long since = clock64();
    for (;;) {
      if (mbar_try(bar(which), parity & 1)) return true;
      if (ctl[2]) return false;
      if (clock64() - since > p.wait_limit) {
        ctl[2] = 1;
        raise_timeout();
        return false;
      }
    }
  };
  // A warp's arrival: its shared-memory writes and tensor-memory reads come first.
  auto arrive = [&](int which) {
    tc_fence_before();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(which));
  };
  // Token count of chunk c, and a row's place in the walk.
  auto length_of = [&](int c) { return c + 1 < chunks ? kC : tail; };
  auto place = [&](int r) { return p.reverse ? kC - 1 - r : r; };
  const uint32_t quad_addr = tmem + ((uint32_t)(quad * 32) << 16);

  if (group == L::kGroups - 1) {
    share_registers<L::kRegsCopy, L::kRegs>();
    if (warp < kMmaWarp - 1) {
      // ---------------- copies ----------------
      // Each warp takes half of the rows of every tensor.
      const int chunk8 = lane % 8, row0 = (warp - (kMmaWarp - 3)) * 32 + lane / 8;   // a 16-byte piece of rows row0 + 4 i
      const uint32_t swz0 = row0 * 128 + ((chunk8 ^ (row0 & 7)) << 4), swz1 = swz0 ^ 64;   // i even and odd
      for (int c = 0; c < chunks; ++c) {
        const int s = c % L::kStages;
        if (c >= L::kStages && !wait(kEmpty + s, c / L::kStages - 1)) break;
        const int len = length_of(c);
        const int64_t i0 = from + (int64_t)c * kC;
        const int64_t at = b * p.T + (p.reverse ? n - i0 - kC : i0) + row0;
#pragma unroll 1
        for (int t = 0; t < (STATES ? 2 : 3); ++t) {
          const __nv_bfloat16 *src = (const __nv_bfloat16 *)(t == 0 ? p.b : t == 1 ? p.c : p.a);
          const int64_t stride = t == 0 ? p.b_stride : t == 1 ? p.c_stride : p.a_stride;
          const int d = t == 1 ? p.dc : p.da;
          const bool low = chunk8 * 8 < d, high = 64 + chunk8 * 8 < d;
          const __nv_bfloat16 *x = src + at * stride + (int64_t)h * d + chunk8 * 8;
          const int64_t step = 4 * stride;
          const uint32_t dst = base + s * L::kStage + t * kTile;
          if (len == kC && d == 128) {
#pragma unroll
            for (int i = 0; i < 8; ++i, x += step) {
              copy16(dst + (i & 1 ? swz1 : swz0) + i * 512, x, true);
              copy16(dst + (i & 1 ? swz1 : swz0) + i * 512 + kBlock, x + 64, true);
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < 8; ++i, x += step) {
              const bool live = place(row0 + 4 * i) < len;
              const uint32_t to = dst + (i & 1 ? swz1 : swz0) + i * 512;
              copy16(to, live && low ? x : src, live && low);
              copy16(to + kBlock, live && high ? x + 64 : src, live && high);
            }
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(kFull + s)) : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kMmaWarp - 1) {
      // ---------------- products: the update of S, 16 tokens at a time ----------------
      if (elect_one()) {
        const uint32_t kind = idesc_bf16(128, p.dc <= 64 ? 64 : 128) | kIdescMnA | kIdescMnB;
        bool ok = true;
        for (int c = 0; ok && c < chunks; ++c) {
          const int s = c % L::kStages;
          if (!wait(kFull + s, c / L::kStages)) break;
          fence_async_smem();                           // the copies' writes, before the products read them
          if (c >= 2 && !wait(kKVFree + (c & 1), (c >> 1) - 1)) break;
          const Desc kt = desc_mn(base + s * L::kStage, kBlock);
#pragma unroll 1
          for (int k = 0; k < kC / kStep; ++k) {
            const int use = c * (kC / kStep) + k;
            if (!(ok = wait(kPartsFull + (use & 1), use >> 1))) break;
            tc_fence_after();
            const Desc w = desc_mn(base + L::kOffParts + (use & 1) * 3 * kPart, kPart / 2);
#pragma unroll
            for (int part = 0; part < 3; ++part)
              mma_bf16(tmem + kColKV + 128 * (c & 1), kt.at(k * 2048), w.at(part * kPart), kind, k + part > 0);
            mma_commit(bar(kPartsEmpty + (use & 1)));
          }
          if (!ok) break;
          mma_commit(bar(kKV + (c & 1)));
          mma_commit(bar(kEmpty + s));
        }
        // every product issued has completed before the memory it uses goes
        mma_commit(bar(kDrainKV));
        if (!mbar_wait_for(bar(kDrainKV), 0, kDrainLimitCycles)) raise_timeout();
      }
    } else if (!STATES) {
      // ---------------- products: P, the outputs ----------------
      if (elect_one()) {
        const int ka = (p.da + 15) / 16;                // K steps over da
        const Desc st = desc_mn(base + L::kOffS, kSBlock), pt = desc_k(base + L::kOffP);
        for (int c = 0; c < chunks; ++c) {
          const int s = c % L::kStages;
          const uint32_t tb = base + s * L::kStage;
          if (!wait(kFull + s, c / L::kStages)) break;
          fence_async_smem();
          tc_fence_after();
          const Desc a = desc_k(tb + 2 * kTile), kt = desc_k(tb);
#pragma unroll 4
          for (int k = 0; k < ka; ++k) {
            const uint32_t off = (k / 4) * kBlock + (k % 4) * 32;
            mma_bf16(tmem + kColP, a.at(off), kt.at(off), idesc_bf16(64, 64), k > 0);
          }
          mma_commit(bar(kQK));
          if ((c > 0 && !wait(kOutFree, c - 1)) || !wait(kSReady, c)) break;
          tc_fence_after();
#pragma unroll 4
          for (int k = 0; k < ka; ++k)
            mma_bf16(tmem + kColInter, st.at(k * 2048), a.at((k / 4) * kBlock + (k % 4) * 32),
                     idesc_bf16(128, 64) | kIdescMnA, k > 0);
          mma_commit(bar(kQS));
          if (!wait(kPReady, c)) break;
          tc_fence_after();
          const Desc v = desc_mn(tb + kTile, kBlock);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16(tmem + kColIntra, v.at(k * 2048), pt.at(k * 32), idesc_bf16(128, 64) | kIdescMnA, k > 0);
          mma_commit(bar(kPV));
          mma_commit(bar(kEmpty + s));
        }
        mma_commit(bar(kDrain));
        if (!mbar_wait_for(bar(kDrain), 0, kDrainLimitCycles)) raise_timeout();
      }
    }
  } else if (group == 0) {
    // ---------------- the state ----------------
    share_registers<L::kRegsS, L::kRegs>();
    const int row = quad * 32 + lane;
    const bool has = row < p.da;
    uint64_t st[64];                                    // columns 2 j and 2 j + 1
    float *states = p.states + ((bh * p.nseg + seg) * p.da) * p.dc;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      float x[2] = {0.f, 0.f};
      if (!STATES && has && 2 * j < p.dc) {             // dc is even
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (p.nseg > 1) x[e] = states[(int64_t)row * p.dc + 2 * j + e];
          else if (p.first) x[e] = first_at(p, bh, row, 2 * j + e);
        }
      }
      st[j] = pair(x[0], x[1]);
    }
    // The state's bf16 copy, [da][dc] in blocks of 64 columns.
    auto publish = [&]() {
      const uint32_t dst = base + L::kOffS + row * 128;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = narrow(st[j * 4 + i]);
        sts128(dst + (j / 8) * kSBlock + (((j % 8) ^ (row & 7)) << 4), w);
      }
      arrive(kSReady);
    };
    for (int c = 0; c < chunks; ++c) {
      if (!STATES) {
        if (c > 0) wait(kQS, c - 1);                    // the last copy is read
        publish();
      }
      const int lead = from + (int64_t)c * kC == 0 ? p.first_pow : 1;
      const float keep = decay_pow(g, length_of(c) - 1 + lead);
      const uint64_t keep2 = pair(keep, keep);
      wait(kKV + (c & 1), c >> 1);
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q < 2 || p.dc > 64) {                       // narrow states: the upper columns stay zero
          uint64_t x[16];
          tmem_ld32(quad_addr + kColKV + 128 * (c & 1) + q * 32, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) st[q * 16 + i] = fma2(st[q * 16 + i], keep2, x[i]);
        }
      }
      arrive(kKVFree + (c & 1));
    }
    if (has && (STATES || (p.nseg == 1 && p.last))) {
      float *dst = STATES ? states : p.last + bh * p.da * p.dc;
      // no token at all: the state passes through unchanged
      const float f = STATES ? 1.f : p.last_scale * (n > 0 ? decay_pow(g, p.last_pow) : 1.f);
#pragma unroll
      for (int j = 0; j < 64; j += 2) {
        if (2 * j < p.dc) {                             // dc is a multiple of 8
          float4 x;
          unpair(st[j], x.x, x.y);
          unpair(st[j + 1], x.z, x.w);
          x.x *= f; x.y *= f; x.z *= f; x.w *= f;
          *reinterpret_cast<float4 *>(dst + (int64_t)row * p.dc + 2 * j) = x;
        }
      }
    }
  } else if (group <= 2) {
    // ---------------- w c in three parts, each in the tile's own layout ----------------
    share_registers<L::kRegsParts, L::kRegs>();
    const int tid = threadIdx.x - 128;
    const uint64_t minus = pair(-1.f, -1.f);
    const int row = tid / 8 % kStep;                    // of each step's 16; block tid / 128
    const uint32_t from_tile = tid / 128 * kBlock + row * 128 + tid % 8 * 16;
    const uint32_t to = base + L::kOffParts + tid / 128 * (kPart / 2) + row * 128 + tid % 8 * 16;
    float w[kC / kStep];
#pragma unroll
    for (int k = 0; k < kC / kStep; ++k) w[k] = pw[kC - 1 - place(k * kStep + row)];
    for (int c = 0; c < chunks; ++c) {
      const int s = c % L::kStages, len = length_of(c);
      if (len < kC) {
#pragma unroll
        for (int k = 0; k < kC / kStep; ++k) {
          const int li = place(k * kStep + row);
          w[k] = li < len ? pw[len - 1 - li] : 0.f;
        }
      }
      wait(kFull + s, c / L::kStages);
      uint32_t next[4];
#pragma unroll
      for (int k = 0; k < kC / kStep; ++k) {
        uint32_t v[4], p0[4], p1[4], p2[4];
        if (k == 0) lds128(base + s * L::kStage + kTile + from_tile, next);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = next[e];
        if (k + 1 < kC / kStep) lds128(base + s * L::kStage + kTile + from_tile + (k + 1) * (kStep * 128), next);
        const uint64_t w2 = pair(w[k], w[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint64_t x = widen(v[e]);
          scale_pair(x, w2);
          p0[e] = narrow(x);
          x = fma2(widen(p0[e]), minus, x);
          p1[e] = narrow(x);
          p2[e] = narrow(fma2(widen(p1[e]), minus, x));
        }
        const int use = c * (kC / kStep) + k;
        if (use >= 2) wait(kPartsEmpty + (k & 1), (use >> 1) - 1);
        const uint32_t dst = to + (k & 1) * 3 * kPart;
        sts128(dst, p0);
        sts128(dst + kPart, p1);
        sts128(dst + 2 * kPart, p2);
        arrive(kPartsFull + (k & 1));
      }
    }
  } else if (group == 3) {
    // ---------------- P: 64 rows in the first 16 lanes of each quadrant ----------------
    share_registers<L::kRegsP, L::kRegs>();
    const int row = quad * 16 + lane / 4, col = 2 * (lane % 4);         // of the thread's first element
    float w[32];                                        // its 32 weights (alpha, the decay, the mask) stay the same
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = row + 8 * (j / 2), k = col + 8 * i + j % 2, back = p.reverse ? k - r : r - k;
        w[4 * i + j] = back >= 0 ? p.alpha * pw[back] : 0.f;
      }
    const int srow = quad * 16 + lane % 16;             // the row this lane names for the matrix stores
    const uint32_t dst = base + L::kOffP + srow * 128;
    for (int c = 0; c < chunks; ++c) {
      wait(kQK, c);
      if (c > 0) wait(kPV, c - 1);               // the last copy is read
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t x[16];
        tmem_ld_fragments(quad_addr + kColP + q * 32, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; i += 2) {                // columns 32 q + 8 i: two fragments of 16 x 8
          uint32_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * i + 2 * j;
            uint64_t y = joined(x[e], x[e + 1]);
            scale_pair(y, pair(w[16 * q + e], w[16 * q + e + 1]));
            v[j] = narrow(y);
          }
          stmatrix4(dst + (((q * 4 + i + lane / 16) ^ (srow & 7)) << 4), v);
        }
      }
      arrive(kPReady);
    }
  } else {
    // ---------------- outputs: weights, sum, transposition through shared memory, store ----------------
    share_registers<L::kRegsOut, L::kRegs>();
    const int tid = threadIdx.x - 4 * 128;
    float w[16];                                        // alpha and the decay of the thread's 16 tokens
    int lead = -1;
    // the matrix stores: this lane names a token's row and 8 columns of c
    const uint32_t put = base + L::kOffOut + (8 * (lane / 16) + lane % 8) * kOutPitch + (quad * 4 + lane / 8 % 2) * 16;
    const int col = tid % 16 * 8;
    const uint32_t get = base + L::kOffOut + tid / 16 * kOutPitch + col * 2;
    const int64_t step = (int64_t)8 * p.H * p.dc;
    for (int c = 0; c < chunks; ++c) {
      const int len = length_of(c);
      const int64_t i0 = from + (int64_t)c * kC;
      const int now = i0 == 0 ? p.first_pow : 1;
      if (now != lead) {
        lead = now;
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = p.alpha * pw[place(8 * (i / 2) + 2 * (lane % 4) + i % 2) + lead];
      }
      wait(kPV, c);
      __syncwarp();
      tc_fence_after();
      output_barrier();                                 // the last outputs have left the staging
#pragma unroll
      for (int q = 0; q < 4; ++q) {                     // columns 16 (q / 2) of c, tokens 32 (q % 2)
        const uint32_t at = quad_addr + ((uint32_t)(q / 2 * 16) << 16) + q % 2 * 32;
        uint32_t x[16], y[16];
        tmem_ld_fragments(at + kColInter, x);
        tmem_ld_fragments(at + kColIntra, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * i + 2 * j, t = 8 * (q % 2) + 2 * (i + j / 2);
            v[j] = narrow(fma2(joined(x[e], x[e + 1]), pair(w[t], w[t + 1]), joined(y[e], y[e + 1])));
          }
          stmatrix4_t(put + (q % 2 * 32 + i * 8) * kOutPitch + q / 2 * 32, v);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOutFree));
      output_barrier();
      __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out +
                           ((b * p.T + (p.reverse ? n - i0 - kC : i0) + tid / 16) * p.H + h) * p.dc + col;
#pragma unroll
      for (int i = 0; i < 8; ++i, dst += step) {
        if (place(i * 8 + tid / 16) < len && col < p.dc) {
          uint32_t v[4];
          lds128(get + i * 8 * kOutPitch, v);
          st_vec(dst, make_uint4(v[0], v[1], v[2], v[3]));
        }
      }
    }
    // rows behind the sequence are zero
    const int64_t first_row = max(stop, begin);
    const int v = p.dc / 8;
    for (int64_t k = tid; k < (end - first_row) * v; k += 128)
      st_vec((__nv_bfloat16 *)p.out + ((b * p.T + first_row + k / v) * p.H + h) * p.dc + k % v * 8, make_uint4(0, 0, 0, 0));
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, STATES ? 256 : 512);
  }
}

}  // namespace

// From one full chunk on; shorter prompts stay on the general kernel, whose
// fp32 products also spare a handful of tokens the rounding of P.
bool linear_tc_supported(int64_t T, int dtype) { return dtype == ATTNRES_BF16 && T >= kChunk; }

// Segments: the count with the least waves of CTAs times their length.  A
// CTA's fixed cost is worth about six chunks, and with more than one segment
// the states' kernel and the scan add about half of the main kernel's time.
int linear_tc_segments(int64_t BH, int64_t T) {
  const int64_t slots = sm_count(), chunks = (T + kChunk - 1) / kChunk;
  int best = 1;
  double least = 0.;
  for (int n = 1; n <= 64 && n * 4 <= chunks + 3; ++n) {
    const int64_t per = (chunks + n - 1) / n, waves = (BH * ((chunks + per - 1) / per) + slots - 1) / slots;
    const double cost = (double)waves * (double)(per + 6) * (n > 1 ? 1.5 : 1.0) + (n > 1 ? 8. : 0.);
    if (n == 1 || cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

namespace {
// The shares above start from the registers a launch gives each thread: what
// the compiler chose has to be that number, or a role would wait for
// registers that nobody gives.
template <bool STATES> bool registers_as_planned() {
  static const bool ok = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, linear_tc_kernel<STATES>) == cudaSuccess && a.numRegs == Shape<STATES>::kRegs;
  }();
  return ok;
}
template <bool STATES> cudaError_t launch_chunks(const LinearParams &p, int64_t BH, cudaStream_t stream) {
  using L = Shape<STATES>;
  if (!registers_as_planned<STATES>()) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(linear_tc_kernel<STATES>, dim3((unsigned)(BH * p.nseg)), dim3(L::kThreads), L::kBytes, stream, p);
}
}  // namespace

cudaError_t launch_linear_tc(const LinearParams &p, int64_t BH, bool states, cudaStream_t stream) {
  return states ? launch_chunks<true>(p, BH, stream) : launch_chunks<false>(p, BH, stream);
}

}  // namespace attnres
