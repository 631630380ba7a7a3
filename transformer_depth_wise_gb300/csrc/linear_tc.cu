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
// Roles of a CTA, one per SM: eight worker warps, two warps that copy tiles
// (cp.async, 16 bytes a lane, straight into the swizzled layout, rows behind
// the sequence and columns behind the width as zeros; tensor-map copies are
// served one box at a time per CTA and would cap one CTA per SM at about
// 4.2 TB/s), one thread that issues the products.  Tensor memory holds P, the
// update of S, and two pairs of output accumulators.  Workers, per chunk c:
// split w c (starts the update of S), form P (starts c^T P^T), store the
// outputs of chunk c - 1, then S (starts S^T a^T of chunk c + 1); so the
// products run beside the next piece of the workers' work.
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
constexpr int kWorkers = 8, kCopiers = 2;             // warps
constexpr int kMmaWarp = kWorkers + kCopiers;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kCopyThreads = kCopiers * 32;
constexpr uint32_t kTile = kC * 128 * 2;              // bytes: 64 tokens x 128 columns, two blocks of 64 columns
constexpr uint32_t kBlock = kTile / 2;
constexpr uint32_t kSBlock = 128 * 128;               // 64 columns of S's 128 rows
constexpr int kOutPitch = 320;                        // bytes per token of the output staging (no bank met twice)

// Tensor memory columns (main kernel): P, update of S, outputs by parity.
constexpr uint32_t kColP = 0, kColKV = 64, kColInter = 192, kColIntra = 320;

template <bool STATES> struct Smem {
  static constexpr uint32_t kStage = (STATES ? 2 : 3) * kTile;      // [a], b, c
  static constexpr uint32_t kOffParts = 2 * kStage;                 // STATES: the first part replaces c itself
  static constexpr uint32_t kOffP = kOffParts + (STATES ? 2 : 3) * kTile;
  static constexpr uint32_t kOffS = kOffP + (STATES ? 0 : kC * 128);
  static constexpr uint32_t kOffOut = kOffS + (STATES ? 0 : 2 * kSBlock);
  static constexpr uint32_t kOffPow = kOffOut + (STATES ? 0 : kC * kOutPitch);
  static constexpr uint32_t kOffBar = kOffPow + 68 * 4;
  static constexpr uint32_t kBytes = kOffBar + 16 * 8 + 1024;       // and the alignment's slack
};

enum Bar { kFull0, kFull1, kEmpty0, kEmpty1, kQK, kS, kV, kKV, kP, kPV, kDrain, kBars };

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
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t w) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(w) : "memory");
}
__device__ __forceinline__ void worker_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kWorkers * 32) : "memory"); }

// A chunk of the walk: its physical rows are t0 .. t0 + 63 of the sequence;
// row r is the chunk's token r, or 63 - r when time runs backwards.
struct Chunk {
  int64_t t0;
  int len;
};
__device__ __forceinline__ Chunk chunk_at(const LinearParams &p, int64_t n, int64_t i0, int64_t stop) {
  Chunk c;
  c.len = (int)min((int64_t)kC, stop - i0);
  c.t0 = p.reverse ? n - i0 - kC : i0;
  return c;
}

template <bool STATES>
__global__ void __launch_bounds__(kThreads, STATES ? 2 : 1) linear_tc_kernel(const LinearParams p) {
  using L = Smem<STATES>;
  extern __shared__ unsigned char smem_raw[];
  grid_dependency_wait();
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(sm);
  float *pw = reinterpret_cast<float *>(sm + L::kOffPow);                       // lambda^0 .. lambda^65
  volatile uint32_t *ctl = reinterpret_cast<uint32_t *>(sm + L::kOffBar + kBars * 8);   // TMEM address, skip, abort
  auto bar = [&](int b) { return base + L::kOffBar + 8u * b; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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

  if (threadIdx.x == 0) {
    ctl[1] = *reinterpret_cast<volatile unsigned int *>(&g_error_flag) != 0 ? 1u : 0u;
    ctl[2] = 0;
    mbar_init(bar(kFull0), kCopyThreads);
    mbar_init(bar(kFull1), kCopyThreads);
    mbar_init(bar(kEmpty0), 1);
    mbar_init(bar(kEmpty1), 1);
    mbar_init(bar(kQK), 1);
    mbar_init(bar(kS), kWorkers);
    mbar_init(bar(kV), kWorkers);
    mbar_init(bar(kKV), 1);
    mbar_init(bar(kP), kWorkers);
    mbar_init(bar(kPV), 1);
    mbar_init(bar(kDrain), 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 66) pw[threadIdx.x] = decay_pow(g, threadIdx.x);
  __syncthreads();
  if (ctl[1]) return;                                 // an earlier error has not been taken: nothing is issued
  if (warp == kMmaWarp) tmem_alloc(base + L::kOffBar + kBars * 8, STATES ? 128 : 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl[0];
  const uint32_t kv_col = STATES ? 0 : kColKV;

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
  // A worker warp's arrival: its shared-memory writes and tensor-memory reads come first.
  auto arrive = [&](int which) {
    tc_fence_before();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(which));
  };

  if (warp >= kWorkers && warp < kMmaWarp) {
    // ---------------- copies ----------------
    const int tid = threadIdx.x - kWorkers * 32;
    const int chunk8 = tid % 8, row0 = tid / 8;         // a 16-byte piece of rows row0 + 8 i
    auto copy_tile = [&](uint32_t dst, const void *src, int64_t stride, int d, const Chunk &ck) {
      const __nv_bfloat16 *x = (const __nv_bfloat16 *)src + (b * p.T + ck.t0) * stride + (int64_t)h * d;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = row0 + 8 * (i % 8), col = (i / 8) * 64 + chunk8 * 8;
        const bool live = (p.reverse ? kC - 1 - r : r) < ck.len && col < d;
        copy16(dst + (i / 8) * kBlock + r * 128 + ((chunk8 ^ (r & 7)) << 4), live ? (const void *)(x + r * stride + col) : src,
               live);
      }
    };
    for (int c = 0; c < chunks; ++c) {
      const int s = c & 1;
      if (c >= 2 && !wait(kEmpty0 + s, ((c >> 1) - 1))) break;
      const Chunk ck = chunk_at(p, n, from + (int64_t)c * kC, stop);
      uint32_t dst = base + s * L::kStage;
      copy_tile(dst, p.b, p.b_stride, p.da, ck);
      copy_tile(dst + kTile, p.c, p.c_stride, p.dc, ck);
      if (!STATES) copy_tile(dst + 2 * kTile, p.a, p.a_stride, p.da, ck);
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(kFull0 + s)) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kMmaWarp) {
    // ---------------- products ----------------
    if (lane == 0) {
      const int ka = (p.da + 15) / 16;                  // K steps over da
      const uint32_t nkv = p.dc <= 64 ? 64 : 128;
      for (int c = 0; c < chunks; ++c) {
        const int s = c & 1;
        const uint32_t tb = base + s * L::kStage, tcl = tb + kTile, ta = tb + 2 * kTile;
        if (!wait(kFull0 + s, c >> 1)) break;
        fence_async_smem();                             // the copies' writes, before the products read them
        tc_fence_after();
        if (!STATES) {
          for (int k = 0; k < ka; ++k) {
            const uint32_t off = (k / 4) * kBlock + (k % 4) * 32;
            mma_bf16(tmem + kColP, sw128_desc(ta + off, 1024), sw128_desc(tb + off, 1024), idesc_bf16(64, 64), k > 0);
          }
          mma_commit(bar(kQK));
          if (!wait(kS, c)) break;
          tc_fence_after();
          for (int k = 0; k < ka; ++k) {
            const uint32_t off = (k / 4) * kBlock + (k % 4) * 32;
            mma_bf16(tmem + kColInter + 64 * s, sw128_desc_mn(base + L::kOffS + k * 2048, kSBlock, 1024),
                     sw128_desc(ta + off, 1024), idesc_bf16(128, 64) | kIdescMnA, k > 0);
          }
        }
        if (!wait(kV, c)) break;
        tc_fence_after();
        for (int part = 0; part < 3; ++part) {
          const uint32_t w = STATES ? (part == 0 ? tcl : base + L::kOffParts + (part - 1) * kTile)
                                    : base + L::kOffParts + part * kTile;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16(tmem + kv_col, sw128_desc_mn(tb + k * 2048, kBlock, 1024), sw128_desc_mn(w + k * 2048, kBlock, 1024),
                     idesc_bf16(128, (int)nkv) | kIdescMnA | kIdescMnB, part > 0 || k > 0);
        }
        mma_commit(bar(kKV));
        if (!STATES) {
          if (!wait(kP, c)) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16(tmem + kColIntra + 64 * s, sw128_desc_mn(tcl + k * 2048, kBlock, 1024),
                     sw128_desc(base + L::kOffP + k * 32, 1024), idesc_bf16(128, 64) | kIdescMnA, k > 0);
          mma_commit(bar(kPV));
        }
        mma_commit(bar(kEmpty0 + s));
      }
      // every product issued has completed before the memory it uses goes
      mma_commit(bar(kDrain));
      if (!mbar_wait_for(bar(kDrain), 0, kDrainLimitCycles)) raise_timeout();
    }
  } else {
    // ---------------- workers ----------------
    const int half = warp / 4, quad = warp % 4;
    const uint32_t quad_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const int row = quad * 32 + lane;                   // of S (and, of the outputs, the column of c)
    const bool has = row < p.da && half * 64 < p.dc;    // this thread's 64 columns of S exist
    float st[64];
    float *states = p.states + ((bh * p.nseg + seg) * p.da) * p.dc;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      const int col = half * 64 + j;
      st[j] = 0.f;
      if (!STATES && has && col < p.dc) {
        if (p.nseg > 1) st[j] = states[(int64_t)row * p.dc + col];
        else if (p.first) st[j] = first_at(p, bh, row, col);
      }
    }
    // The state's bf16 copy, [da][dc] in blocks of 64 columns.
    auto publish_state = [&]() {
      const uint32_t dst = base + L::kOffS + half * kSBlock + row * 128;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = Elt<__nv_bfloat16>::pack_word(st[j * 8 + 2 * i], st[j * 8 + 2 * i + 1]);
        sts128(dst + ((j ^ (row & 7)) << 4), w);
      }
      arrive(kS);
    };
    // The outputs of chunk c: weights, sum, transposition through shared memory, store.
    auto store_outputs = [&](int c) {
      const Chunk ck = chunk_at(p, n, from + (int64_t)c * kC, stop);
      const int lead = from + (int64_t)c * kC == 0 ? p.first_pow : 1;
      const int s = c & 1;
      worker_barrier();                                 // the last outputs have left the staging
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int t0 = half * 32 + q * 16;              // this thread: column `row` of tokens t0 .. t0 + 15
        float x[16], y[16];
        tmem_ld16(quad_addr + kColInter + 64 * s + t0, x);
        tmem_ld16(quad_addr + kColIntra + 64 * s + t0, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = t0 + i;
          x[i] = p.alpha * fmaf(pw[(p.reverse ? kC - 1 - r : r) + lead], x[i], y[i]);
        }
        // neighbouring lanes swap, so that each stores two columns of one token
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? x[i] : x[i + 1], 1);
          const uint32_t w = lane & 1 ? Elt<__nv_bfloat16>::pack_word(other, x[i + 1])
                                      : Elt<__nv_bfloat16>::pack_word(x[i], other);
          sts32(base + L::kOffOut + (t0 + i + (lane & 1)) * kOutPitch + (row & ~1) * 2, w);
        }
      }
      worker_barrier();
      __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out + ((b * p.T + ck.t0) * p.H + h) * p.dc;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = i * (kWorkers * 32) + threadIdx.x, r = k / 16, col = (k % 16) * 8;
        if ((p.reverse ? kC - 1 - r : r) < ck.len && col < p.dc) {
          uint32_t w[4];
          lds128(base + L::kOffOut + r * kOutPitch + col * 2, w);
          st_vec(dst + (int64_t)r * p.H * p.dc + col, make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
    };
    if (!STATES && chunks > 0) publish_state();
    for (int c = 0; c < chunks; ++c) {
      const int s = c & 1;
      const Chunk ck = chunk_at(p, n, from + (int64_t)c * kC, stop);
      const int lead = from + (int64_t)c * kC == 0 ? p.first_pow : 1;
      const uint32_t tcl = base + s * L::kStage + kTile;
      // w c in three parts, each in the tile's own layout
      wait(kFull0 + s, c >> 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = (i * (kWorkers * 32) + threadIdx.x) * 16;
        const int r = (off / 128) % kC, li = p.reverse ? kC - 1 - r : r;
        const float w = li < ck.len ? pw[ck.len - 1 - li] : 0.f;
        uint32_t v[4], p0[4], p1[4], p2[4];
        lds128(tcl + off, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x0, x1, h0, h1;
          Elt<__nv_bfloat16>::unpack_word(v[e], x0, x1);
          x0 *= w;
          x1 *= w;
          p0[e] = Elt<__nv_bfloat16>::pack_word(x0, x1);
          Elt<__nv_bfloat16>::unpack_word(p0[e], h0, h1);
          x0 -= h0;
          x1 -= h1;
          p1[e] = Elt<__nv_bfloat16>::pack_word(x0, x1);
          Elt<__nv_bfloat16>::unpack_word(p1[e], h0, h1);
          p2[e] = Elt<__nv_bfloat16>::pack_word(x0 - h0, x1 - h1);
        }
        if (STATES) {
          sts128(tcl + off, p0);
          sts128(base + L::kOffParts + off, p1);
          sts128(base + L::kOffParts + kTile + off, p2);
        } else {
          sts128(base + L::kOffParts + off, p0);
          sts128(base + L::kOffParts + kTile + off, p1);
          sts128(base + L::kOffParts + 2 * kTile + off, p2);
        }
      }
      arrive(kV);
      if (!STATES) {
        // P: 64 rows in 16 lanes of each quadrant; this warp's half of the columns
        if (c > 0) wait(kPV, c - 1);                    // P's last copy is read
        wait(kQK, c);
        __syncwarp();
        tc_fence_after();
        float x[32];
        tmem_ld16(quad_addr + kColP + half * 32, x);
        tmem_ld16(quad_addr + kColP + half * 32 + 16, x + 16);
        tmem_wait_ld();
        if (lane < 16) {
          const int r = quad * 16 + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int col = half * 32 + j * 8 + i, back = p.reverse ? col - r : r - col;
              x[j * 8 + i] = back >= 0 ? x[j * 8 + i] * pw[back] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = Elt<__nv_bfloat16>::pack_word(x[j * 8 + 2 * i], x[j * 8 + 2 * i + 1]);
            sts128(base + L::kOffP + r * 128 + (((half * 4 + j) ^ (r & 7)) << 4), w);
          }
        }
        arrive(kP);
        if (c > 0) store_outputs(c - 1);
      }
      // S <- lambda^len S + its update
      wait(kKV, c);
      __syncwarp();
      tc_fence_after();
      if (half * 64 < p.dc) {
        const float keep = decay_pow(g, ck.len - 1 + lead);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[16];
          tmem_ld16(quad_addr + kv_col + half * 64 + q * 16, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) st[q * 16 + i] = fmaf(st[q * 16 + i], keep, x[i]);
        }
      }
      if (!STATES && c + 1 < chunks) publish_state();
    }
    if (!STATES && chunks > 0) {
      wait(kPV, chunks - 1);
      store_outputs(chunks - 1);
    }
    if (has && (STATES || (p.nseg == 1 && p.last))) {
      float *dst = STATES ? states : p.last + bh * p.da * p.dc;
      // no token at all: the state passes through unchanged
      const float f = STATES ? 1.f : p.last_scale * (n > 0 ? decay_pow(g, p.last_pow) : 1.f);
#pragma unroll
      for (int j = 0; j < 64; j += 4) {
        const int col = half * 64 + j;                  // dc is a multiple of 8
        if (col < p.dc)
          *reinterpret_cast<float4 *>(dst + (int64_t)row * p.dc + col) =
              make_float4(st[j] * f, st[j + 1] * f, st[j + 2] * f, st[j + 3] * f);
      }
    }
    if (!STATES) {
      // rows behind the sequence are zero
      const int64_t first_row = max(stop, begin);
      const int v = p.dc / 8;
      for (int64_t k = threadIdx.x; k < (end - first_row) * v; k += kWorkers * 32)
        st_vec((__nv_bfloat16 *)p.out + ((b * p.T + first_row + k / v) * p.H + h) * p.dc + k % v * 8, make_uint4(0, 0, 0, 0));
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, STATES ? 128 : 512);
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

cudaError_t launch_linear_tc(const LinearParams &p, int64_t BH, bool states, cudaStream_t stream) {
  auto go = [&](auto kern, uint32_t smem) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)(BH * p.nseg)), dim3(kThreads), smem, stream, p);
  };
  return states ? go(linear_tc_kernel<true>, Smem<true>::kBytes) : go(linear_tc_kernel<false>, Smem<false>::kBytes);
}

}  // namespace attnres
