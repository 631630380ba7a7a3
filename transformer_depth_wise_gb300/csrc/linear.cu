// linear.cu -- linear attention with one decay per head: over prompts
// (chunked), its gradients, and for single tokens (recurrent).
//
// Per sequence and head, with lambda = e^g:
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Written out, o_t = scale (sum_{s <= t} lambda^{t-s} (q_t . k_s) v_s +
// lambda^{t+1} S_0^T q_t), one form F(a, b, c; first) = sum_{j <= i}
// lambda^{i-j} (a_i . b_j) c_j + lambda^{i+1} a_i . first that the gradients
// share: dq = scale F(do, v, k; S_0^T), and with time running backwards
// dk = scale F'(v, do, q) and dv = scale F'(k, q, do) with dS^T and dS as
// their first states, where dS, the gradient of the final state, meets the
// last token undecayed and unscaled: there scale goes into the state with
// the tokens instead of multiplying what is read out of it, and dS_0 is
// lambda times the state that the last of them ends with, dS itself where
// there is no token.
//
// Chunks.  Within a chunk of kC tokens the masked, decayed product matrix
// P_ij = lambda^{i-j} a_i . b_j is formed once and applied to c; what came
// before enters through the state.  Decay weights never exceed one: rows are
// weighted by lambda^{i+1} on the way out and by lambda^{n-1-j} on the way
// into the state, so a strong decay underflows to zero and nothing overflows.
//
// Segments.  The chunks of one (sequence, head) follow one another, so where
// there are too few of those to fill the GPU the time axis is cut into
// segments: one kernel forms every segment's own state, a scan turns them
// into the states that the segments begin with, and the main kernel runs all
// segments at once.
#include <algorithm>
#include <type_traits>

#include "linear.cuh"

namespace attnres {
namespace {

constexpr int kC = kChunk;             // tokens per chunk
constexpr int kThreads = 256;
constexpr int kNS = 64;                // columns of c a CTA takes
constexpr int kMaxDim = 128;

// ---------------------------------------------------------------------------
// The fp32 kernel (and, for no tokens at all, the states of either type), any
// width up to 128, padded with zeros to DA.  A CTA owns kNS columns of c and of
// the state for one segment.
//
// Products.  On the tensor cores: an fp32 operand is split into a tf32 (its upper
// bits) and the nearest tf32 of what is left, both by integer instructions (by
// conversions, which take several issue slots each, the kernel takes 15 % longer).
// x y = xh yh + (xh yl + xl yh); what is missing is below 2^-19 of |x y|, 2^-22
// on average.  The tensor cores' accumulators cut off instead of rounding
// (measured: 1 plus 3/4 of the last place stays 1), so the large and the small
// products have accumulators of their own, none of which runs for longer than a
// chunk: the state itself is kept in fp32 registers and takes one rounded
// addition per chunk.
//
// Roles.  Four warps hold 16 rows of P = a b^T each, which stay in registers as
// the left operand of P c (the pairs of columns that a lane holds name the rows
// of c that it reads), and the four others the state, 32 x 32 elements at a
// time; only the state goes through shared memory, for a S.  In the
// states' kernel all eight warps hold the state.  The next chunk's rows are
// copied while one is worked on.  What binds is the rate at which instructions
// are issued: splitting, loads of operands, and 1100 products a scheduler.
//
// Measured on GB300, 128 x 128: 11.3 us for a chunk and slice (on the CUDA
// cores 24), 2.8 in the states' kernel; 64 heads x 4096 tokens 740 us (1532).
// Twelve and sixteen warps (a S by four of its own, the state in eight) take
// 708 and 738 there, and 4 to 9 % longer with 64 x 64.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy_or_zero(float *dst, const float *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}

// Rows i0 .. i0 + kC of a [.., H, d] tensor, columns col0 .. col0 + W, on their
// way to shared memory [kC][pitch]; rows behind `stop` and columns behind d are zero.
template <int W>
__device__ __forceinline__ void copy_rows(const LinearParams &p, float *dst, int pitch, const void *src, int64_t stride,
                                          int h, int d, int col0, int64_t b, int64_t n, int64_t i0, int64_t stop) {
  constexpr int V = W / 4, kRows = kThreads / V;        // rows per turn
  static_assert(kC % kRows == 0, "whole turns");
  const int r0 = threadIdx.x / V, c = threadIdx.x % V * 4;
  const int rows = col0 + c < d ? (int)min((int64_t)kC, stop - i0) : 0;
  const float *at = (const float *)src + walk_row(p, b, n, i0 + r0) * stride + (int64_t)h * d + col0 + c;
  const int64_t step = (p.reverse ? -kRows : kRows) * stride;
  float *to = dst + r0 * pitch + c;
#pragma unroll
  for (int r = 0; r < kC; r += kRows, at += step, to += kRows * pitch) {
    const bool live = r + r0 < rows;
    copy_or_zero(to, live ? at : (const float *)src, live);
  }
}

struct Tf32 {
  uint32_t hi, lo;
};
__device__ __forceinline__ Tf32 split(float x) {
  constexpr uint32_t kUpper = 0xffffe000u;
  const uint32_t hi = __float_as_uint(x) & kUpper;
  return {hi, (__float_as_uint(x - __uint_as_float(hi)) + 0x1000u) & kUpper};
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A left operand's 16 x 8 elements: rows g, g + 8 at the lane's first k (x0, x1) and its second (x2, x3).
struct Left {
  uint32_t hi[4], lo[4];
  __device__ __forceinline__ Left(float x0, float x1, float x2, float x3) {
    const float x[4] = {x0, x1, x2, x3};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Tf32 s = split(x[i]);
      hi[i] = s.hi;
      lo[i] = s.lo;
    }
  }
};
// One 16 x 8 tile of sums: the large products and the small ones.
struct Tile {
  float big[4] = {}, small[4] = {};
  __device__ __forceinline__ void add(const Left &a, float y0, float y1) {
    const Tf32 b0 = split(y0), b1 = split(y1);
    mma_tf32(big, a.hi, b0.hi, b1.hi);
    mma_tf32(small, a.hi, b0.lo, b1.lo);
    mma_tf32(small, a.lo, b0.hi, b1.hi);
  }
  __device__ __forceinline__ float at(int i) const { return big[i] + small[i]; }
};

// Floats of shared memory: two stages of b, a [kC][DA + 8] and c [kC][kPitchC], the state, the decay's powers.
constexpr int kPitchC = kNS + 8, kPitchS = kNS + 4;
template <int DA, bool STATES> struct Room {
  static constexpr int kPitch = DA + 8;
  static constexpr int kB = 0, kA = kC * kPitch, kCc = (STATES ? 1 : 2) * kC * kPitch;
  static constexpr int kStage = kCc + kC * kPitchC;
  static constexpr int kS = 2 * kStage, kPow = kS + (STATES ? 0 : DA * kPitchS);
  static constexpr int kFloats = kPow + kC + 4;
};

template <int DA, bool STATES>
__global__ void __launch_bounds__(kThreads) linear_general_kernel(const LinearParams p) {
  using R = Room<DA, STATES>;
  constexpr int kPitch = R::kPitch;
  constexpr int kHolders = STATES ? 8 : 4;             // warps with parts of the state
  constexpr int kParts = DA / 32 * (kNS / 32);         // of 32 x 32
  constexpr int kOwn = (kParts + kHolders - 1) / kHolders;
  extern __shared__ float4 smem4[];
  float *sm = reinterpret_cast<float *>(smem4), *ss = sm + R::kS, *pw = sm + R::kPow;
  grid_dependency_wait();
  const int seg = blockIdx.x % p.nseg, slice = blockIdx.x / p.nseg % p.slices;
  const int64_t bh = blockIdx.x / (p.nseg * p.slices), b = bh / p.H;
  const int h = (int)(bh % p.H), col0 = slice * kNS;
  const int64_t n = seq_length(p, b);
  const int64_t begin = seg * p.seg_len, end = min(p.T, begin + p.seg_len), stop = min(n, end);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g8 = lane / 4, t = lane % 4;
  const float g = p.log_decay[h];
  if (threadIdx.x <= kC) pw[threadIdx.x] = decay_pow(g, threadIdx.x);

  // The lane's elements of part i of the state: tile (m, j) holds rows g8, g8 + 8 of 16 and columns 2 t, 2 t + 1 of 8.
  const int holder = STATES ? warp : warp - 4;
  auto part_of = [&](int i) { return holder * kOwn + i; };
  auto row_of = [&](int i, int m, int e) { return part_of(i) / 2 * 32 + m * 16 + g8 + (e / 2) * 8; };
  auto col_of = [&](int i, int j, int e) { return part_of(i) % 2 * 32 + j * 8 + 2 * t + e % 2; };
  const bool holds = holder >= 0 && holder * kOwn < kParts;
  float s[kOwn][2][4][4];
  float *states = p.states + ((bh * p.nstates + seg * p.step) * p.da) * p.dc;
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][m][j][e] = 0.f;
          if (!holds) continue;
          const int row = row_of(i, m, e), col = col0 + col_of(i, j, e);
          if (!STATES && row < p.da && col < p.dc) {
            if (p.nseg > 1)
              s[i][m][j][e] = p.states_t ? states[(int64_t)col * p.da + row] : states[(int64_t)row * p.dc + col];
            else if (p.first) s[i][m][j][e] = first_at(p, bh, row, col);
          }
        }
  auto copy = [&](int64_t i0, int stage) {
    float *to = sm + stage * R::kStage;
    copy_rows<DA>(p, to + R::kB, kPitch, p.b, p.b_stride, h, p.da, 0, b, n, i0, stop);
    if (!STATES) copy_rows<DA>(p, to + R::kA, kPitch, p.a, p.a_stride, h, p.da, 0, b, n, i0, stop);
    copy_rows<kNS>(p, to + R::kCc, kPitchC, p.c, p.c_stride, h, p.dc, col0, b, n, i0, stop);
    cp_async_commit();
  };
  if (begin < stop) copy(begin, 0);
  int stage = 0;
  for (int64_t i0 = begin; i0 < stop; i0 += kC, stage ^= 1) {
    const int len = (int)min((int64_t)kC, stop - i0);
    const int lead = (i0 == 0) ? p.first_pow : 1;      // the first row's weight of the state: lambda^lead
    const float *sb = sm + stage * R::kStage + R::kB, *sa = sm + stage * R::kStage + R::kA;
    const float *sc = sm + stage * R::kStage + R::kCc;
    if (!STATES && holds) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              *reinterpret_cast<float2 *>(ss + row_of(i, m, e) * kPitchS + col_of(i, j, e)) =
                  make_float2(s[i][m][j][e] * p.carry, s[i][m][j][e + 1] * p.carry);
    }
    cp_async_wait<0>();
    __syncthreads();                                   // the chunk and the state are there; the other stage is read
    if (i0 + kC < stop) copy(i0 + kC, stage ^ 1);
    if (!STATES && warp < 4) {
      const int m0 = warp * 16;
      const float *xa = sa + (m0 + g8) * kPitch + 2 * t;
      // P, up to the diagonal: rows m0 + g8 (+ 8), columns 8 j + 2 t (+ 1); k in the order 2 t, 2 t + 1
      float pr[kC / 8][4];
      {
        Tile acc[kC / 8];
#pragma unroll 2
        for (int k = 0; k < DA; k += 8) {
          const float2 x = *reinterpret_cast<const float2 *>(xa + k);
          const float2 y = *reinterpret_cast<const float2 *>(xa + 8 * kPitch + k);
          const Left a(x.x, y.x, x.y, y.y);
#pragma unroll
          for (int j = 0; j < kC / 8; ++j) {
            if (j > 2 * warp + 1) continue;
            const float2 z = *reinterpret_cast<const float2 *>(sb + (8 * j + g8) * kPitch + k + 2 * t);
            acc[j].add(a, z.x, z.y);
          }
        }
#pragma unroll
        for (int j = 0; j < kC / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int back = m0 + g8 + (e / 2) * 8 - (8 * j + 2 * t + e % 2);
            pr[j][e] = back >= 0 ? acc[j].at(e) * (p.alpha * pw[back]) : 0.f;
          }
      }
      // the state's part, weighted by row, then the chunk's own
      float o[kNS / 8][4];
      {
        Tile acc[kNS / 8];
#pragma unroll 2
        for (int k = 0; k < DA; k += 8) {
          const float2 x = *reinterpret_cast<const float2 *>(xa + k);
          const float2 y = *reinterpret_cast<const float2 *>(xa + 8 * kPitch + k);
          const Left a(x.x, y.x, x.y, y.y);
          const float *z = ss + (k + 2 * t) * kPitchS + g8;
#pragma unroll
          for (int j = 0; j < kNS / 8; ++j) acc[j].add(a, z[8 * j], z[kPitchS + 8 * j]);
        }
#pragma unroll
        for (int j = 0; j < kNS / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = acc[j].at(e) * pw[m0 + g8 + (e / 2) * 8 + lead];
      }
      Tile acc[kNS / 8];
#pragma unroll
      for (int i = 0; i < kC / 8; ++i) {
        if (i > 2 * warp + 1) continue;
        const Left a(pr[i][0], pr[i][2], pr[i][1], pr[i][3]);
        const float *z = sc + (8 * i + 2 * t) * kPitchC + g8;
#pragma unroll
        for (int j = 0; j < kNS / 8; ++j) acc[j].add(a, z[8 * j], z[kPitchC + 8 * j]);
      }
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int r = m0 + g8 + (e / 2) * 8;
        if (r >= len) continue;
        float *y = (float *)p.out + (walk_row(p, b, n, i0 + r) * p.H + h) * p.dc + col0 + 2 * t;
#pragma unroll
        for (int j = 0; j < kNS / 8; ++j)
          if (col0 + 8 * j + 2 * t < p.dc)
            *reinterpret_cast<float2 *>(y + 8 * j) = make_float2(o[j][e] + acc[j].at(e), o[j][e + 1] + acc[j].at(e + 1));
      }
    } else if (holds) {
      // S = lambda^len S + gain sum_j lambda^{len-1-j} b_j c_j^T
      const float keep = decay_pow(g, len - 1 + lead);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        Tile acc[2][4];
        const float *xb = sb + part_of(i) / 2 * 32 + g8, *xc = sc + part_of(i) % 2 * 32 + g8;
#pragma unroll 2
        for (int k = 0; k < kC; k += 8) {
          const int k0 = k + t, k1 = k0 + 4;
          const float w0 = k0 < len ? p.gain * pw[len - 1 - k0] : 0.f, w1 = k1 < len ? p.gain * pw[len - 1 - k1] : 0.f;
          const float *x = xb + k0 * kPitch, *y = x + 4 * kPitch;
          const Left a0(x[0], x[8], y[0], y[8]), a1(x[16], x[24], y[16], y[24]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float z0 = xc[k0 * kPitchC + 8 * j] * w0, z1 = xc[k1 * kPitchC + 8 * j] * w1;
            acc[0][j].add(a0, z0, z1);
            acc[1][j].add(a1, z0, z1);
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][m][j][e] = fmaf(s[i][m][j][e], keep, acc[m][j].at(e));
      }
    }
    if (!STATES) __syncthreads();                      // the state is read
  }
  const bool write_last = !STATES && p.nseg == 1 && p.last;
  if ((STATES || write_last) && holds) {
    float *dst = STATES ? states : p.last + bh * p.da * p.dc;
    // no token at all: the state passes through unchanged
    const float f = STATES || n == 0 ? 1.f : decay_pow(g, p.last_pow);
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = row_of(i, m, e), col = col0 + col_of(i, j, e);
            if (row < p.da && col < p.dc) dst[(int64_t)row * p.dc + col] = s[i][m][j][e] * f;
          }
  }
  if (!STATES) {
    // rows behind the sequence are zero
    const int64_t from = max(stop, begin);
    const int w = min(kNS, p.dc - col0);
    for (int64_t k = threadIdx.x; k < (end - from) * w; k += kThreads)
      ((float *)p.out)[((b * p.T + from + k / w) * p.H + h) * p.dc + col0 + k % w] = 0.f;
  }
}

// The segments' own states become the states they begin with; the state
// after the last token is written where it is wanted (else the last segment's
// own state is not used, whatever is there).  Four elements of a row
// per thread, the next segments' on their way while one is added.
__global__ void __launch_bounds__(kThreads) linear_scan_kernel(const LinearParams p) {
  grid_dependency_wait();
  const int per = p.da * p.dc / 4;
  const int64_t bh = blockIdx.y;
  const int e = blockIdx.x * kThreads + threadIdx.x;
  if (e >= per) return;
  if (p.done && e == 0) p.done[bh] = 0;
  const int64_t n = seq_length(p, bh / p.H);
  const float g = p.log_decay[bh % p.H];
  const int row = e * 4 / p.dc, col = e * 4 % p.dc;      // dc is a multiple of 4
  float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.first)
    cur = make_float4(first_at(p, bh, row, col), first_at(p, bh, row, col + 1), first_at(p, bh, row, col + 2),
                      first_at(p, bh, row, col + 3));
  float4 *st = reinterpret_cast<float4 *>(p.states) + bh * p.nstates * per + e;
  const float full = decay_pow(g, p.seg_len);
  auto read = [&](int s) { return s < p.nseg ? st[(int64_t)s * per] : make_float4(0.f, 0.f, 0.f, 0.f); };
  float4 own = read(0), next = read(1), after = read(2);
  for (int s = 0; s < p.nseg; ++s) {
    const float4 later = read(s + 3);
    st[(int64_t)s * per] = cur;
    const int64_t left = n - s * p.seg_len;
    if (left > 0) {
      const float keep = s > 0 && left >= p.seg_len ? full : decay_pow(g, min(p.seg_len, left) - (s == 0 ? 1 - p.first_pow : 0));
      cur = make_float4(fmaf(cur.x, keep, own.x), fmaf(cur.y, keep, own.y), fmaf(cur.z, keep, own.z), fmaf(cur.w, keep, own.w));
    }
    own = next;
    next = after;
    after = later;
  }
  if (p.last) {
    const float f = n > 0 ? decay_pow(g, p.last_pow) : 1.f;
    reinterpret_cast<float4 *>(p.last)[bh * per + e] = make_float4(cur.x * f, cur.y * f, cur.z * f, cur.w * f);
  }
}

// ---------------------------------------------------------------------------
// One token: S' = lambda S + k v^T, o = scale S'^T q.  Bound by the state,
// read and written once.  A CTA takes `cols` columns of one (sequence, head)
// and all its rows, four columns per thread; the row groups' parts of o meet
// in shared memory.
// ---------------------------------------------------------------------------
struct StepParams {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int H, dk, dv, cols;
  const float *log_decay;
  float scale;
  const float *state;
  float *state_out;
  void *out;
};

template <typename T>
__device__ __forceinline__ float elt_at(const T *x, int64_t i) {
  if constexpr (std::is_same<T, float>::value) return x[i];
  else return __bfloat162float(x[i]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(const StepParams p) {
  constexpr int RPT = 4;                               // rows in flight per thread
  __shared__ float sq[kMaxDim], sk[kMaxDim];
  __shared__ float4 red[kThreads];
  grid_dependency_wait();
  const int64_t bh = blockIdx.x, b = bh / p.H;
  const int h = (int)(bh % p.H);
  const int lanes = p.cols / 4, groups = kThreads / lanes;
  const int lane = threadIdx.x % lanes, grp = threadIdx.x / lanes;
  const int col = blockIdx.y * p.cols + lane * 4;
  const bool active = grp < groups && col < p.dv;
  const float lam = expf(p.log_decay[h]);
  if (threadIdx.x < p.dk) {
    sq[threadIdx.x] = elt_at((const T *)p.q, b * p.q_stride + (int64_t)h * p.dk + threadIdx.x);
    sk[threadIdx.x] = elt_at((const T *)p.k, b * p.k_stride + (int64_t)h * p.dk + threadIdx.x);
  }
  float v[4] = {};
  if (active) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = elt_at((const T *)p.v, b * p.v_stride + (int64_t)h * p.dv + col + j);
  }
  __syncthreads();
  float o[4] = {};
  const float *src = p.state + bh * p.dk * p.dv + col;
  float *dst = p.state_out + bh * p.dk * p.dv + col;
  if (active) {
    for (int r0 = grp; r0 < p.dk; r0 += groups * RPT) {
      float4 s[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = r0 + i * groups;
        if (r < p.dk) s[i] = *reinterpret_cast<const float4 *>(src + (int64_t)r * p.dv);
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = r0 + i * groups;
        if (r >= p.dk) continue;
        const float kr = sk[r], qr = sq[r];
        s[i].x = fmaf(lam, s[i].x, kr * v[0]);
        s[i].y = fmaf(lam, s[i].y, kr * v[1]);
        s[i].z = fmaf(lam, s[i].z, kr * v[2]);
        s[i].w = fmaf(lam, s[i].w, kr * v[3]);
        o[0] = fmaf(qr, s[i].x, o[0]);
        o[1] = fmaf(qr, s[i].y, o[1]);
        o[2] = fmaf(qr, s[i].z, o[2]);
        o[3] = fmaf(qr, s[i].w, o[3]);
        *reinterpret_cast<float4 *>(dst + (int64_t)r * p.dv) = s[i];
      }
    }
  }
  red[threadIdx.x] = make_float4(o[0], o[1], o[2], o[3]);
  __syncthreads();
  if (threadIdx.x < lanes && active) {
    float4 t = red[threadIdx.x];
    for (int k = 1; k < groups; ++k) {
      const float4 x = red[k * lanes + threadIdx.x];
      t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
    }
    T *y = (T *)p.out + bh * p.dv + col;
    t.x *= p.scale; t.y *= p.scale; t.z *= p.scale; t.w *= p.scale;
    if constexpr (std::is_same<T, float>::value) *reinterpret_cast<float4 *>(y) = t;
    else *reinterpret_cast<uint2 *>(y) = make_uint2(Elt<T>::pack_word(t.x, t.y), Elt<T>::pack_word(t.z, t.w));
  }
}

int general_slices(int dc) { return (dc + kNS - 1) / kNS; }

template <typename K>
cudaError_t launch_big(K kern, int64_t ctas, size_t smem, cudaStream_t st, const LinearParams &p) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)ctas), dim3(kThreads), smem, st, p);
}

}  // namespace

bool linear_supported(int64_t da, int64_t dc, int dtype) {
  const int e = dtype == ATTNRES_BF16 ? 8 : 4;
  return da >= e && dc >= e && da <= kMaxDim && dc <= kMaxDim && da % e == 0 && dc % e == 0;
}

// Segments of the fp32 kernel: the split with the least cost in waves of CTAs, one
// per SM, times their chunks, in units of a chunk of the main kernel (11.3 us).  A
// chunk of the states' kernel is worth a quarter of one, a CTA's start 0.8 (the
// states' kernel's 0.33), the scan 0.35, a state written, scanned and read 0.001.
// The same with da and dc exchanged, so that two calls can share the segments'
// states.
// Measured, uncut against cut: 4 heads of 128 x 128, 100 tokens 34 against 26 us,
// 512 102 against 27, 4096 728 against 71; 64 heads of 64 x 64, 1024 tokens 110
// against 77; 40 heads of 128 x 128, 4096 tokens 730 against 549, 1024 tokens 191
// against 194 (uncut); 64 heads, 4096 tokens 732 against 917 (uncut).
static Split linear_split(int64_t B, int64_t T, int H, int da, int dc, int dtype) {
  if (B * H < 1 || T < 1) return {kChunk, 1, 1};
  const int64_t chunks = (T + kC - 1) / kC;
  if (B * H > 65535) return {chunks * kC, 1, 1};                 // the scan's grid; and the SMs are full
  if (linear_tc_supported(T, dtype)) return linear_tc_split(B * H, T);
  const int wide = da > dc ? da : dc;
  const int64_t have = B * H * general_slices(wide), slots = sm_count();
  auto waves = [&](int64_t ctas) { return (double)((ctas + slots - 1) / slots); };
  int64_t per = chunks;
  double least = waves(have) * ((double)chunks + 0.8);
  for (int n = 2; n <= 128 && n <= chunks; ++n) {
    const int64_t len = (chunks + n - 1) / n, segments = (chunks + len - 1) / len;
    const double cost = waves(have * segments) * ((double)len + 0.8) +
                        0.25 * waves(have * (segments - 1)) * ((double)len + 1.3) + 0.35 +
                        0.001 * (double)(B * H * segments);
    if (cost < least) {
      least = cost;
      per = len;
    }
  }
  return {per * kC, (int)((chunks + per - 1) / per), 1};
}

int64_t linear_workspace_floats(int64_t B, int64_t T, int H, int da, int dc, int dtype) {
  const Split s = linear_split(B, T, H, da, dc, dtype);
  if (s.nseg == 1) return 0;
  const int64_t marks = linear_tc_supported(T, dtype) ? B * H * (s.nseg * kMarks + 1) : 0;
  return B * H * s.nseg * s.nsub * da * dc + marks;
}

cudaError_t launch_linear(const LinearArgs &a) {
  LinearParams p{};
  p.a = a.a; p.b = a.b; p.c = a.c;
  p.a_stride = a.a_stride; p.b_stride = a.b_stride; p.c_stride = a.c_stride;
  p.out = a.out; p.T = a.T; p.H = a.H; p.da = a.da; p.dc = a.dc;
  p.slices = general_slices(a.dc);
  const Split split = linear_split(a.B, a.T, a.H, a.da, a.dc, a.dtype);
  p.nseg = split.nseg;
  p.seg_len = split.seg_len;
  p.nstates = split.nseg * split.nsub;
  p.step = split.nsub;
  p.log_decay = a.log_decay; p.lengths = a.lengths; p.reverse = a.reverse;
  p.alpha = a.alpha; p.carry = a.carry; p.gain = a.gain;
  p.first = a.first; p.first_t = a.first_t; p.first_pow = a.first_pow;
  p.last = a.last; p.last_pow = a.last_pow;
  p.states = a.workspace;
  p.states_t = a.states_t;
  p.wait_limit = std::min(wait_limit_cycles(), 1ll << 48);    // times a CTA's length, within 63 bits
  const int64_t BH = a.B * a.H;
  const bool tc = linear_tc_supported(a.T, a.dtype);
  if (tc && p.nseg > 1) {
    p.marks = reinterpret_cast<uint32_t *>(p.states + BH * p.nstates * a.da * a.dc);
    p.done = p.marks + BH * p.nseg * kMarks;
    p.piece = (float)(p.seg_len / split.nsub);
  }
  // The states' kernel (states = true) or the main one.
  auto chunks = [&](const LinearParams &p, bool states) -> cudaError_t {
    if (tc) return launch_linear_tc(p, BH, states, a.stream);
    const int64_t ctas = BH * p.nseg * p.slices;
    auto go = [&](auto da) -> cudaError_t {
      constexpr int DA = decltype(da)::value;
      const size_t smem = (size_t)(states ? Room<DA, true>::kFloats : Room<DA, false>::kFloats) * sizeof(float);
      return states ? launch_big(linear_general_kernel<DA, true>, ctas, smem, a.stream, p)
                    : launch_big(linear_general_kernel<DA, false>, ctas, smem, a.stream, p);
    };
    return a.da <= 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
  };
  if (p.nseg > 1 && !a.states_ready) {
    // The pieces' own states (the last segment's only where the final state
    // is wanted), then the states they begin with.
    LinearParams s = p;
    s.seg_len = p.seg_len / split.nsub;
    s.step = 1;
    s.nseg = (a.last ? p.nseg : p.nseg - 1) * split.nsub;
    cudaError_t e = chunks(s, true);
    if (e != cudaSuccess) return e;
    if (!a.last) ++s.nseg;
    e = launch_dependent(linear_scan_kernel, dim3((unsigned)((a.da * a.dc / 4 + kThreads - 1) / kThreads), (unsigned)BH),
                         dim3(kThreads), 0, a.stream, s);
    if (e != cudaSuccess) return e;
  }
  return chunks(p, false);
}

cudaError_t launch_linear_step(const LinearStepArgs &a) {
  StepParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v;
  p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
  p.H = a.H; p.dk = a.dk; p.dv = a.dv;
  p.log_decay = a.log_decay; p.scale = a.scale; p.state = a.state; p.state_out = a.state_out; p.out = a.out;
  // Slices of 32 columns (128 bytes of a row) while there is no (sequence, head)
  // pair for every SM, else whole rows.  Measured, 128 x 128, sliced against
  // whole: 64 pairs 4.2 against 6.5 us, 152 5.7 against 7.1, 176 7.7 against 7.5, 256
  // 8.5 against 7.8, 2048 47.8 against 38.9.
  p.cols = a.dv;
  if (a.B * a.H <= sm_count() && a.dv > 32) p.cols = 32;
  const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.dv + p.cols - 1) / p.cols));
  return a.dtype == ATTNRES_BF16
             ? launch_dependent(linear_step_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, a.stream, p)
             : launch_dependent(linear_step_kernel<float>, grid, dim3(kThreads), 0, a.stream, p);
}

}  // namespace attnres
