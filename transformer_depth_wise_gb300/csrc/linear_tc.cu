// linear_tc.cu -- the chunks of linear attention with one decay per head on
// the 5th-generation tensor cores (bf16 inputs; see linear.cu for the form
// F(a, b, c; first) and the segments).
//
// Per chunk of 64 tokens, with S the state before it (da x dc, fp32):
//   P  = a b^T, masked and decayed                    (M 64,  N 64,  K da)
//   O^T = carry S^T a^T (weighted by token) + c^T P^T (M dc,  N 64,  K da; K 64)
//   S^T <- lambda^n S^T + (w c)^T b, w_j = gain lambda^{n-1-j} (M dc, N da, K 64)
// (one of carry and gain is the call's scale, the other 1).
// The outputs and the state are formed transposed, so that every product but
// the small P has M = 128, the full rate, and S^T is a left operand as it
// lies: a thread's row of it goes to tensor memory as bf16.  c^T, (w c)^T and
// b are MN-major operands: the tiles are used as they lie in memory, nothing
// is transposed by threads.
//
// Accuracy.  The state has to keep fp32 accuracy over any number of chunks:
// S itself lives in fp32 registers, and w c, which the product takes in bf16,
// is split into parts.  Three of them (24 bits) make the product exact to
// fp32's rounding, for a state that may be handed out; two (16 bits, an error
// of 2^-17 at most) serve the main kernel's where the states' kernel has
// formed the exact ones.  P and the copy of S (times carry) that
// forms the outputs are rounded to bf16 once: each adds an error of the size
// of the output's own rounding at most.
//
// Roles of a CTA, one per SM (a warpgroup of four warps each): two for the
// state (a thread per row of S^T and half of its columns, in registers); two
// for the weighted parts; P; the outputs; and one with the lanes that copy
// tiles (tensor-map boxes of 64 tokens x 64 columns, six of them in flight
// per stage: rows outside the tensor and columns behind the width arrive as
// zeros) and two threads that issue products, one the updates of S and one
// all others, so that neither waits for the other's operands.  What bound earlier forms was
// the shared memory's 128 bytes per cycle, which the products' operands, the
// copies and the threads share: 3700 of a chunk's 4370 cycles with S^T as a
// shared-memory operand and tiles copied by threads (cp.async), 2550 of 3000
// with S^T in tensor memory and tensor-map boxes.
//
// Measured on GB300: 65536 tokens, 32 heads of 128 x 128, 331 us for the
// 2.15 GB of inputs and outputs (6.5 TB/s) and 110 us for the segments'
// states (decays e^-2^(-8i/32); without decay the whole call takes 529 instead
// of 456 us, as nothing is left out there); 4 x 4096 tokens, 16 heads, 53 us
// for 268 MB (5.0 TB/s) and 22 us.
//
// What is no number.  By the recurrence a NaN or an infinity in b or c stays in
// the state however small its token's weight becomes, but the states' kernel
// leaves out tokens whose finite traces are zero.  The main kernel sees every
// token: a CTA whose segment's last state holds what is no number marks its
// columns, which also go into the call's last state, and the last CTA of a
// (sequence, head) to finish carries the marks on to the outputs of the later
// segments.  (1.4 us a launch, where heads have such tokens.)
//
// Every wait is bounded: one that runs out records a flag and an abort mark
// in shared memory, on which every other wait returns at once; the issuing
// roles stop and drain what they have in flight, and the CTA ends.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "linear.cuh"
#include "tcgen05.cuh"

ATTNRES_DEFINE_ERROR_FLAG(take_error_linear)

namespace attnres {
namespace {

constexpr int kC = kChunk;
constexpr int kMaxRanked = 512;                       // heads that the states' kernel orders by their decay
constexpr uint32_t kTile = kC * 128 * 2;              // bytes: 64 tokens x 128 columns, two blocks of 64 columns
constexpr uint32_t kBlock = kTile / 2;
constexpr int kOutPitch = 272;                        // bytes per token of the output staging (no bank met twice)

// The main kernel's warpgroups: S, S, parts, parts, P, outputs, copies and
// products; the states' kernel: S, S, four for the parts, copies and products.
template <bool STATES> struct Shape {
  static constexpr int kGroups = 7;
  static constexpr int kThreads = kGroups * 128;
  static constexpr int kStages = STATES ? 4 : 3;
  // Registers per thread: as launched (checked at the launch), then each
  // role's share; their sum stays within the launch's.
  static constexpr int kRegs = 72;
  static constexpr int kPartGroups = STATES ? 4 : 2;
  // The weighted parts are formed in steps of kStep tokens (whole chunks in
  // the states' kernel, half of one where the outputs need the room) by two
  // teams, each with a buffer of its own, that take the steps in turn.
  static constexpr int kStep = STATES ? 64 : 32;
  static constexpr uint32_t kPart = kStep * 128 * 2;                // one part: two blocks of 64 columns
  static constexpr int kTeam = kPartGroups * 64;                    // threads of a team
  static constexpr int kRegsS = 96, kRegsParts = 64, kRegsP = 72, kRegsOut = 80, kRegsMma = 32;
  static_assert(2 * kRegsS + kPartGroups * kRegsParts + (STATES ? 0 : kRegsP + kRegsOut) + kRegsMma <= kGroups * kRegs,
                "more registers than the launch has");
  static constexpr uint32_t kStage = (STATES ? 2 : 3) * kTile;      // b, c, [a]
  static constexpr uint32_t kOffParts = kStages * kStage;
  static constexpr uint32_t kOffP = kOffParts + 2 * 3 * kPart;
  static constexpr uint32_t kOffOut = kOffP + (STATES ? 0 : kC * 128);
  static constexpr uint32_t kOffPow = kOffOut + (STATES ? 0 : kC * kOutPitch);
  static constexpr uint32_t kOffBar = kOffPow + 72 * 4;
  static constexpr uint32_t kBytes = kOffBar + 36 * 8 + 1024;       // and the alignment's slack
};

// Tensor memory columns: the update of S by the chunk's parity, P, the outputs'
// two sums, S^T as bf16 pairs.
constexpr uint32_t kColKV = 0, kColP = 256, kColInter = 320, kColIntra = 384, kColST = 448;

// Barriers, one phase per chunk (full, empty and parts: one per use of a
// stage or buffer).  A waiter may be at most one phase behind its barrier, or
// the parity deceives it; the updates of S, which run up to two chunks ahead
// of the state, therefore have a pair of each, by the chunk's parity.
enum Bar { kFull = 0, kEmpty = 4, kPartsFull = 8, kPartsEmpty = 10, kKV = 12, kKVFree = 14, kPV = 16, kOutFree, kQK, kSReady,
           kQS, kPReady, kClean, kDrain, kDrainKV, kBars };

// A box of a [B][H][T][d] view (coordinates innermost first) to shared memory.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int t, int h, int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(t), "r"(h), "r"(b), "r"(bar) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
// What a CTA of the main kernel has stored, before its first group counts it
// as done: that group waits for the other state's and the outputs'.
__device__ __forceinline__ void stored_arrive() {
  __syncwarp();
  asm volatile("bar.arrive 2, 384;" ::: "memory");
}
__device__ __forceinline__ void stored_wait() {
  __syncwarp();
  asm volatile("bar.sync 2, 384;" ::: "memory");
}
__device__ __forceinline__ void first_group_barrier() {
  __syncwarp();
  asm volatile("bar.sync 3, 128;" ::: "memory");
}
// The outputs' four warps.
__device__ __forceinline__ void output_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Two fp32 values in a register pair, from and to bf16 pairs.
__device__ __forceinline__ uint64_t widen(uint32_t w) { return ((uint64_t)(w & 0xffff0000u) << 32) | (uint64_t)(w << 16); }
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  unpair(v, lo, hi);
  return Elt<__nv_bfloat16>::pack_word(lo, hi);
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

// A token whose weight in its segment's last state is below e^-kReach leaves no
// trace there: even the largest finite product of gain, b and c comes below
// fp32's smallest number (e^-193 of e^88.8).
constexpr float kReach = 193.f;

__device__ __forceinline__ bool no_number(uint32_t bits) { return (bits & 0x7f800000u) == 0x7f800000u; }

// The tensors as [B][H][T][d], boxes of 64 tokens x 64 columns.
struct Maps {
  CUtensorMap b, c, a;
};

template <bool STATES>
__global__ void __launch_bounds__(Shape<STATES>::kThreads, 1)
    linear_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LinearParams p) {
  using L = Shape<STATES>;
  extern __shared__ unsigned char smem_raw[];
  grid_dependency_wait();
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(sm);
  float *pw = reinterpret_cast<float *>(sm + L::kOffPow);                       // lambda^0 .. lambda^65
  volatile uint32_t *ctl = reinterpret_cast<uint32_t *>(sm + L::kOffBar + kBars * 8);   // TMEM address, skip, abort, done
  auto bar = [&](int b) { return base + L::kOffBar + 8u * b; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp >> 2, quad = warp & 3;

  // Neighbouring CTAs take the heads of the same tokens: their rows lie side
  // by side in memory.
  const int64_t BH = gridDim.x / p.nseg;
  int64_t bh = blockIdx.x % BH;
  int seg = (int)(blockIdx.x / BH);
  if (STATES && p.H > 1 && p.H <= kMaxRanked) {
    // A head with a strong decay needs the end of a segment only (below), so
    // the slow ones, a segment's whole length of work, go first: CTAs in
    // the order of the heads' decays.
    int *decays = reinterpret_cast<int *>(sm);          // as integers of the same order (any bits at all have one)
    int *found = reinterpret_cast<int *>(sm + kMaxRanked * 4);
    for (int i = threadIdx.x; i < p.H; i += L::kThreads) {
      const int x = __float_as_int(p.log_decay[i]);
      decays[i] = x ^ ((x >> 31) & 0x7fffffff);
    }
    __syncthreads();
    const int64_t per = BH / p.H * p.nseg, rank = blockIdx.x / per, rest = blockIdx.x % per;
    for (int i = threadIdx.x; i < p.H; i += L::kThreads) {
      int before = 0;
      for (int j = 0; j < p.H; ++j) before += decays[j] > decays[i] || (decays[j] == decays[i] && j < i);
      if (before == rank) *found = i;
    }
    __syncthreads();
    bh = rest % (BH / p.H) * p.H + *found;
    seg = (int)(rest / (BH / p.H));
    fence_async_smem();                               // tensor-map copies will write over what was kept here
    __syncthreads();
  }
  const int64_t b = bh / p.H;
  const int h = (int)(bh % p.H);
  const int64_t n = seq_length(p, b);
  const int64_t begin = seg * p.seg_len, end = min(p.T, begin + p.seg_len), stop = min(n, end);
  const float g = p.log_decay[h];
  int64_t from = begin;
  if (STATES && g < 0.f && stop > begin) {
    // What finite tokens before these add to the segment's last state is
    // exactly nothing: start behind them.
    const float reach = kReach / -g;
    if (reach < (float)(stop - begin)) from = max(begin, (stop - 1 - (int64_t)reach) / kC * kC);
  }
  const int chunks = stop > from ? (int)((stop - from + kC - 1) / kC) : 0;
  // The last chunk of a sequence that ends before the tensor does also gets
  // the rows behind the sequence; they are cleared in shared memory.
  const bool unclean = !p.reverse && n < p.T && stop == n;
  const int tail = chunks > 0 ? (int)(stop - from - (int64_t)(chunks - 1) * kC) : 0;   // tokens of the last chunk

  if (threadIdx.x == 0) {
    ctl[1] = *reinterpret_cast<volatile unsigned int *>(&g_error_flag) != 0 ? 1u : 0u;
    ctl[2] = 0;
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar(kFull + i), 1);
      mbar_init(bar(kEmpty + i), STATES ? 1 : 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kPartsFull + i), L::kTeam / 32);
      mbar_init(bar(kPartsEmpty + i), 1);
      mbar_init(bar(kKV + i), 1);
      mbar_init(bar(kKVFree + i), 8);
    }
    mbar_init(bar(kQK), 1);
    mbar_init(bar(kSReady), 8);
    mbar_init(bar(kQS), 1);
    mbar_init(bar(kPV), 1);
    mbar_init(bar(kOutFree), 4);
    mbar_init(bar(kPReady), 4);
    mbar_init(bar(kClean), 8);
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

  // Wait for the phase; false once any wait of the CTA has run out.  The limit
  // counts from the CTA's start and once more for every 8192 chunks that it
  // goes through (some 10 ms of work), so that no length runs into it; a short
  // loop at every wait keeps the roles' code small.
  const long long deadline = clock64() + p.wait_limit * (1 + chunks / 8192);
  auto wait = [&](int which, uint32_t parity) -> bool {
    const uint32_t at = bar(which);
    while (!mbar_try(at, parity & 1)) {
      if (ctl[2]) return false;
      if (clock64() > deadline) {
        ctl[2] = 1;
        raise_timeout();
      }
    }
    return true;
  };
  // A warp's arrival: its shared-memory writes and tensor-memory reads come first.
  auto arrive = [&](int which) {
    tc_fence_before();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(which));
  };
  // The same where only tensor memory was read.
  auto release = [&](int which) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(which));
  };
  // Token count of chunk c, and a row's place in the walk.
  auto length_of = [&](int c) { return c + 1 < chunks ? kC : tail; };
  auto place = [&](int r) { return p.reverse ? kC - 1 - r : r; };
  // Whether the states' kernel may have left out tokens of this head (its own
  // test divides: a margin for the roundings of both).
  auto left_out = [&]() -> bool { return !STATES && p.nseg > 1 && -g * p.piece > 0.99f * kReach; };
  const bool three = STATES || p.nseg == 1;            // parts of w c: this kernel's state is the one handed out
  const uint32_t quad_addr = tmem + ((uint32_t)(quad * 32) << 16);

  if (group == L::kGroups - 1) {
    share_registers<L::kRegsMma, L::kRegs>();
    auto clean = [&](int c) -> bool { return !(unclean && tail < kC && c + 1 == chunks) || wait(kClean, 0); };
    if (warp == kMmaWarp - 3) {
      // ---------------- copies: a box per lane ----------------
      constexpr int kBoxes = STATES ? 4 : 6;
      const int t = lane >> 1;
      const CUtensorMap *map = t == 0 ? &maps.b : t == 1 ? &maps.c : &maps.a;
      int last = -1;
      for (int c = 0; c < chunks; ++c) {
        const int s = c % L::kStages;
        const bool ok = c < L::kStages || wait(kEmpty + s, c / L::kStages - 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int64_t i0 = from + (int64_t)c * kC;
        if (lane == 0) mbar_expect_tx(bar(kFull + s), L::kStage);
        __syncwarp();
        if (lane < kBoxes)
          copy_box(base + s * L::kStage + lane * kBlock, map, (lane & 1) * 64, (int)(p.reverse ? n - i0 - kC : i0), h, (int)b,
                   bar(kFull + s));
        last = c;
      }
      // what was copied has landed before the CTA may end
      for (int c = max(0, last + 1 - L::kStages); c <= last; ++c)
        if (!mbar_wait_for(bar(kFull + c % L::kStages), (c / L::kStages) & 1, kDrainLimitCycles)) raise_timeout();
    } else if (warp == kMmaWarp - 1) {
      // ---------------- products: the update of S, step by step ----------------
      if (elect_one()) {
        const uint32_t kind = idesc_bf16(128, p.da <= 64 ? 64 : 128) | kIdescMnA | kIdescMnB;
        bool ok = true;
        for (int c = 0; ok && c < chunks; ++c) {
          const int s = c % L::kStages;
          if (!wait(kFull + s, c / L::kStages) || !clean(c)) break;
          if (c >= 2 && !wait(kKVFree + (c & 1), (c >> 1) - 1)) break;
          const Desc x = desc_mn(base + s * L::kStage, kBlock);
#pragma unroll 1
          for (int k = 0; k < kC / L::kStep; ++k) {
            const int use = c * (kC / L::kStep) + k;
            if (!(ok = wait(kPartsFull + (use & 1), use >> 1))) break;
            tc_fence_after();
            const Desc w = desc_mn(base + L::kOffParts + (use & 1) * 3 * L::kPart, L::kPart / 2);
#pragma unroll
            for (int i = 0; i < L::kStep / 16; ++i) {
              const uint64_t y = x.at((L::kStep / 16 * k + i) * 2048);
              mma_bf16(tmem + kColKV + 128 * (c & 1), w.at(i * 2048), y, kind, k + i > 0);
              mma_bf16(tmem + kColKV + 128 * (c & 1), w.at(L::kPart + i * 2048), y, kind, 1);
              if (three) mma_bf16(tmem + kColKV + 128 * (c & 1), w.at(2 * L::kPart + i * 2048), y, kind, 1);
            }
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
    } else if (!STATES && warp == kMmaWarp) {
      // ---------------- products: P, the outputs ----------------
      if (elect_one()) {
        const int ka = (p.da + 15) / 16;                // K steps over da
        const Desc pt = desc_k(base + L::kOffP);
        for (int c = 0; c < chunks; ++c) {
          const int s = c % L::kStages;
          const uint32_t tb = base + s * L::kStage;
          if (!wait(kFull + s, c / L::kStages) || !clean(c)) break;
          tc_fence_after();
          const Desc a = desc_k(tb + 2 * kTile), kt = desc_k(tb);
#pragma unroll 2
          for (int k = 0; k < ka; ++k) {
            const uint32_t off = (k / 4) * kBlock + (k % 4) * 32;
            mma_bf16(tmem + kColP, a.at(off), kt.at(off), idesc_bf16(64, 64), k > 0);
          }
          mma_commit(bar(kQK));
          if ((c > 0 && !wait(kOutFree, c - 1)) || !wait(kSReady, c)) break;
          tc_fence_after();
#pragma unroll 2
          for (int k = 0; k < ka; ++k)
            mma_bf16_ts(tmem + kColInter, tmem + kColST + 8 * k, a.at((k / 4) * kBlock + (k % 4) * 32), idesc_bf16(128, 64),
                        k > 0);
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
  } else if (group <= 1) {
    // ---------------- the state: a row of S^T per thread, 64 columns per group ----------------
    share_registers<L::kRegsS, L::kRegs>();
    const int row = quad * 32 + lane, col0 = group * 64;               // dc, da
    uint64_t st[32];                                    // columns col0 + 2 j and the next
    float *states = p.states + ((bh * p.nstates + seg * p.step) * p.da + col0) * p.dc + row;
    const int cols = row < p.dc ? p.da - col0 : 0;      // of this thread's row that exist (da is even)
    {
      // the segment's first state, or the call's (which may lie transposed)
      const bool own = p.nseg > 1, across = own ? p.states_t : p.first_t;
      const float *src = (own ? p.states + (bh * p.nstates + seg * p.step) * p.da * p.dc : p.first + bh * p.da * p.dc) +
                         (across ? (int64_t)row * p.da + col0 : (int64_t)col0 * p.dc + row);
      const int step = across ? 1 : p.dc;
      const int have = !STATES && (own || p.first) ? cols : 0;
#pragma unroll
      for (int j = 0; j < 32; ++j, src += 2 * step) st[j] = 2 * j < have ? pair(src[0], src[step]) : 0ull;
    }
    const float keep_full = decay_pow(g, kC);
    const uint64_t carry = pair(p.carry, p.carry);
    for (int c = 0; c < chunks; ++c) {
      if (!STATES) {
        // its bf16 copy in tensor memory
        if (c > 0) wait(kQS, c - 1);                    // the last copy is read
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint64_t x = st[q * 16 + i];
            scale_pair(x, carry);
            w[i] = narrow(x);
          }
          tmem_st16(quad_addr + kColST + group * 32 + q * 16, w);
        }
        tmem_wait_st();
        release(kSReady);
      }
      const int lead = from + (int64_t)c * kC == 0 ? p.first_pow : 1;
      const int steps = length_of(c) - 1 + lead;
      const float keep = steps == kC ? keep_full : decay_pow(g, steps);
      const uint64_t keep2 = pair(keep, keep);
      wait(kKV + (c & 1), c >> 1);
      __syncwarp();
      tc_fence_after();
      if (col0 < p.da) {                                // else these columns stay zero
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[16];
          tmem_ld16(quad_addr + kColKV + 128 * (c & 1) + col0 + q * 16, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) st[q * 8 + i] = fma2(st[q * 8 + i], keep2, pair(x[2 * i], x[2 * i + 1]));
        }
      }
      release(kKVFree + (c & 1));
    }
    if (STATES || (p.nseg == 1 && p.last)) {
      float *out = STATES ? states : p.last + (bh * p.da + col0) * p.dc + row;
      // no token at all: the state passes through unchanged
      const float f = STATES || n == 0 ? 1.f : decay_pow(g, p.last_pow);
#pragma unroll
      for (int j = 0; j < 32; ++j, out += 2 * p.dc) {
        if (2 * j < cols) {
          float x, y;
          unpair(st[j], x, y);
          out[0] = x * f;
          out[p.dc] = y * f;
        }
      }
    }
    if (left_out()) {
      // columns behind da hold no number only where those before them do
      uint64_t sum = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) sum = fma2(st[j], 0ull, sum);
      float lo, hi;
      unpair(sum, lo, hi);
      const bool bad = row < p.dc && isnan(lo + hi);
      if (bad && p.last) {
        float *last = p.last + (bh * p.da + col0) * p.dc + row;
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (j < cols && no_number((uint32_t)(st[j / 2] >> (j % 2 * 32)))) last[(int64_t)j * p.dc] = __int_as_float(0x7fffffff);
      }
      uint32_t *marks = p.marks + bh * p.nseg * kMarks;
      const uint32_t word = __ballot_sync(0xffffffffu, bad);
      if (lane == 0) marks[seg * kMarks + group * 4 + quad] = word;
      if (group == 1) {
        stored_arrive();
      } else {
        stored_wait();                                  // this CTA's marks and outputs are stored
        if (threadIdx.x == 0) {
          __threadfence();
          ctl[3] = atomicAdd(p.done + bh, 1u) + 1 == (uint32_t)p.nseg ? 1 : 0;
        }
        first_group_barrier();
        if (ctl[3]) {                                   // and so are all others' of this (sequence, head)
          __threadfence();
          uint32_t any = 0;
          for (int i = threadIdx.x; i < p.nseg * kMarks; i += 128) any |= __ldcg(marks + i);
          if (any) ctl[3] = 2;
          if (threadIdx.x == 0) p.done[bh] = 0;         // for a launch that shares the workspace
          first_group_barrier();
          if (ctl[3] == 2 && row < p.dc) {              // a thread per column
            bool lost = false;
            for (int s = 0; s + 1 < p.nseg; ++s) {
              lost |= ((__ldcg(marks + s * kMarks + quad) | __ldcg(marks + s * kMarks + 4 + quad)) >> lane) & 1u;
              if (!lost) continue;
              for (int64_t i = (s + 1) * p.seg_len; i < min(n, (s + 2) * p.seg_len); ++i)
                ((__nv_bfloat16 *)p.out)[(walk_row(p, b, n, i) * p.H + h) * p.dc + row] = __ushort_as_bfloat16(0x7fff);
            }
          }
        }
      }
    }
  } else if (group < 2 + L::kPartGroups) {
    // ---------------- w c in three parts, each in the tile's own layout ----------------
    share_registers<L::kRegsParts, L::kRegs>();
    constexpr int kSteps = kC / L::kStep;               // per chunk
    constexpr int kRows = L::kTeam / 16, kPer = L::kStep / kRows;
    const int team = (threadIdx.x - 2 * 128) / L::kTeam, tid = (threadIdx.x - 2 * 128) % L::kTeam;
    // 16 bytes of a row at a time; kPer of them per step, kRows rows apart
    const int row = tid / 8 % kRows, block = tid / 8 / kRows;
    const int row0 = (kSteps == 2 ? team * L::kStep : 0) + row;        // of the chunk
    const uint32_t src = base + kTile + block * kBlock + row0 * 128 + tid % 8 * 16;
    const uint32_t dst = base + L::kOffParts + team * 3 * L::kPart + block * (L::kPart / 2) + row * 128 + tid % 8 * 16;
    const uint64_t minus = pair(-1.f, -1.f);
    float w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = p.gain * pw[kC - 1 - place(row0 + i * kRows)];
    for (int use = team; use < chunks * kSteps; use += 2) {
      const int c = use / kSteps, s = c % L::kStages, len = length_of(c);
      wait(kFull + s, c / L::kStages);
      if (len < kC) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int li = place(row0 + i * kRows);
          w[i] = li < len ? p.gain * pw[len - 1 - li] : 0.f;
        }
        if (unclean) {
          // the rows behind the sequence, of b and c (those of a only reach
          // outputs that are not stored), by the 256 threads that work on
          // this chunk
          const uint32_t zero[4] = {0, 0, 0, 0};
          for (int i = kSteps == 2 ? threadIdx.x - 2 * 128 : tid; i < (kC - len) * 16; i += 256) {
            const uint32_t at = base + s * L::kStage + i % 16 / 8 * kBlock + (len + i / 16) * 128 + i % 8 * 16;
            sts128(at, zero);
            sts128(at + kTile, zero);
          }
          arrive(kClean);
          wait(kClean, 0);                              // all of them, before the parts are formed
        }
      }
      if (use >= 2) wait(kPartsEmpty + team, (use >> 1) - 1);
#pragma unroll
      for (int i0 = 0; i0 < kPer; i0 += 2) {
        uint32_t v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) lds128(src + s * L::kStage + (i0 + i) * kRows * 128, v[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t w2 = pair(w[i0 + i], w[i0 + i]);
          uint32_t p0[4], p1[4], p2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint64_t x = widen(v[i][e]);
            scale_pair(x, w2);
            p0[e] = narrow(x);
            x = fma2(widen(p0[e]), minus, x);
            p1[e] = narrow(x);
            if (three) p2[e] = narrow(fma2(widen(p1[e]), minus, x));
          }
          const uint32_t to = dst + (i0 + i) * kRows * 128;
          sts128(to, p0);
          sts128(to + L::kPart, p1);
          if (three) sts128(to + 2 * L::kPart, p2);
        }
      }
      arrive(kPartsFull + team);
    }
  } else if (!STATES && group == 4) {
    // ---------------- P: 64 rows in the first 16 lanes of each quadrant ----------------
    share_registers<L::kRegsP, L::kRegs>();
    const int row = quad * 16 + lane / 4, col = 2 * (lane % 4);         // of P: the thread's first element
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
      if (c > 0) wait(kPV, c - 1);                    // the last copy of P is read
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t x[16];
        tmem_ld_fragments(quad_addr + kColP + q * 32, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; i += 2) {              // columns 32 q + 8 i: two fragments of 16 x 8
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
  } else if (!STATES) {
    // ---------------- outputs: weights, sum, transposition through shared memory, store ----------------
    share_registers<L::kRegsOut, L::kRegs>();
    const int tid = threadIdx.x - 5 * 128;
    float w[16];                                        // the decay of the thread's 16 tokens
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
        for (int i = 0; i < 16; ++i) w[i] = pw[place(8 * (i / 2) + 2 * (lane % 4) + i % 2) + lead];
      }
      wait(kPV, c);
      __syncwarp();
      tc_fence_after();
      output_barrier();                                 // the last outputs have left the staging
#pragma unroll 1
      for (int m = 0; m < 2; ++m) {                     // columns 16 m of this warp's 32
#pragma unroll
        for (int q = 0; q < 2; ++q) {                   // tokens 32 q
          const uint32_t at = quad_addr + ((uint32_t)(m * 16) << 16) + q * 32;
          uint32_t x[16], y[16];
          tmem_ld_fragments(at + kColInter, x);
          tmem_ld_fragments(at + kColIntra, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int e = 4 * i + 2 * j, t = 8 * q + 2 * (i + j / 2);
              v[j] = narrow(fma2(joined(x[e], x[e + 1]), pair(w[t], w[t + 1]), joined(y[e], y[e + 1])));
            }
            stmatrix4_t(put + (q * 32 + i * 8) * kOutPitch + m * 32, v);
          }
        }
      }
      release(kOutFree);
      output_barrier();
      __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out +
                           ((b * p.T + (p.reverse ? n - i0 - kC : i0) + tid / 16) * p.H + h) * p.dc + col;
#pragma unroll 2
      for (int i = 0; i < 8; ++i, dst += step) {
        if (place(i * 8 + tid / 16) < len && col < p.dc) {
          uint32_t v[4];
          lds128(get + i * 8 * kOutPitch, v);
          st_vec(dst, make_uint4(v[0], v[1], v[2], v[3]));
        }
      }
    }
    // rows behind the sequence are zero
    for (int64_t t = max(stop, begin) + tid / 16; t < end; t += 8)
      if (col < p.dc) st_vec((__nv_bfloat16 *)p.out + ((b * p.T + t) * p.H + h) * p.dc + col, make_uint4(0, 0, 0, 0));
    if (left_out()) stored_arrive();
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

// The split with the least cost in waves of CTAs, one per SM, times their
// chunks.  A CTA's fixed cost is worth about eight chunks of the main kernel's,
// a chunk of the states' kernel a bit more than half of one and its fixed cost
// three; the scan and the launches make up for four, and every state written,
// scanned and read for a fiftieth.
// Measured, heads of 128 x 128, the whole call uncut against as the rule cuts it:
// 4 heads, 512 tokens 20 us (uncut; in four segments 24), 1024 33 against 28,
// 4096 100 against 32, 65536 1446 against 97; 32 heads, 512 tokens 22 (uncut; in
// four 28), 1024 33 against 34 to 36, 4096 100 against 62, 65536 1457 against 456;
// 64 pairs of 4096 tokens 100 against 103 (two segments of one piece each, which
// the rule passes over for two of two, 97); 128 pairs 102 (uncut; in two 181);
// 160 pairs 199 to 201 (uncut; in two 236).
Split linear_tc_split(int64_t BH, int64_t T) {
  const int64_t slots = sm_count(), chunks = (T + kChunk - 1) / kChunk;
  auto waves = [&](int64_t ctas) { return (double)((ctas + slots - 1) / slots); };
  Split best{chunks * kChunk, 1, 1};
  double least = waves(BH) * (double)(chunks + 8);
  for (int n = 2; n <= 64 && n * 4 <= chunks; ++n) {
    for (int k = 1; k <= 4 && n * k * 4 <= chunks; k *= 2) {
      const int64_t piece = (chunks + (int64_t)n * k - 1) / ((int64_t)n * k), per = piece * k;
      const int64_t segments = (chunks + per - 1) / per;
      const double cost = waves(BH * segments) * (double)(per + 8) + 0.55 * waves(BH * (segments - 1) * k) * (double)(piece + 3) +
                          4. + 0.02 * (double)(BH * segments * k);
      if (segments > 1 && cost < least) {
        least = cost;
        best = {per * kChunk, (int)segments, k};
      }
    }
  }
  return best;
}

namespace {
// The shares above start from the registers a launch gives each thread: what
// the compiler chose has to be that number, or a role would wait for
// registers that nobody gives.  The build checks it too, so that another
// compiler's choice shows there.
template <bool STATES> bool registers_as_planned() {
  static const bool ok = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, linear_tc_kernel<STATES>) == cudaSuccess && a.numRegs == Shape<STATES>::kRegs;
  }();
  return ok;
}
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}
// A [B, T, H, d] tensor whose token rows are `stride` elements apart.
bool encode(CUtensorMap &m, const void *x, int64_t stride, int64_t B, int64_t T, int H, int d) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)stride * 2, (cuuint64_t)d * 2, (cuuint64_t)(T * stride) * 2};
  const cuuint32_t box[4] = {64, kC, 1, 1}, ones[4] = {1, 1, 1, 1};
  return encode_fn()(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(x), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool STATES> cudaError_t launch_chunks(const LinearParams &p, int64_t BH, cudaStream_t stream) {
  using L = Shape<STATES>;
  if (!registers_as_planned<STATES>() || !encode_fn()) return cudaErrorInvalidConfiguration;
  Maps m;
  const int64_t B = BH / p.H;
  if (!encode(m.b, p.b, p.b_stride, B, p.T, p.H, p.da) || !encode(m.c, p.c, p.c_stride, B, p.T, p.H, p.dc) ||
      !encode(m.a, p.a, p.a_stride, B, p.T, p.H, p.da))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(linear_tc_kernel<STATES>, dim3((unsigned)(BH * p.nseg)), dim3(L::kThreads), L::kBytes, stream, m, p);
}
}  // namespace

cudaError_t launch_linear_tc(const LinearParams &p, int64_t BH, bool states, cudaStream_t stream) {
  return states ? launch_chunks<true>(p, BH, stream) : launch_chunks<false>(p, BH, stream);
}

}  // namespace attnres
