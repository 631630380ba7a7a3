// linear.cu -- linear attention with one decay per head: over prompts
// (chunked), its gradients, and for single tokens (recurrent).
//
// Per sequence and head, with lambda = e^g:
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Written out, o_t = scale (sum_{s <= t} lambda^{t-s} (q_t . k_s) v_s +
// lambda^{t+1} S_0^T q_t), one form F(a, b, c; first) = sum_{j <= i}
// lambda^{i-j} (a_i . b_j) c_j + lambda^{i+1} a_i . first that the gradients
// share: dq = scale F(do, v, k; S_0^T), and with time running backwards
// dk = scale F'(v, do, q; dS^T), dv = scale F'(k, q, do; dS), where dS, the
// gradient of the final state, meets the last token undecayed, and
// dS_0 = lambda times the state that the last of them ends with.
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
constexpr int kPadS = kNS + 4;         // row pitch of [.][kNS] tiles (floats)
constexpr int kMaxDim = 128;

// Rows i0 .. i0 + kC of a [.., H, d] tensor, columns col0 .. col0 + W, to fp32
// shared memory [kC][pitch]; rows behind `stop` and columns behind d are zero.
template <int W>
__device__ __forceinline__ void load_rows(const LinearParams &p, float *dst, int pitch, const void *src, int64_t stride,
                                          int h, int d, int col0, int64_t b, int64_t n, int64_t i0, int64_t stop) {
  constexpr int E = Elt<float>::EPV, V = W / E;
  for (int k = threadIdx.x; k < kC * V; k += kThreads) {
    const int r = k / V, c = (k % V) * E;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (i0 + r < stop && col0 + c < d)
      v = ld_stream((const float *)src + walk_row(p, b, n, i0 + r) * stride + (int64_t)h * d + col0 + c);
    float x[E];
    Elt<float>::unpack(v, x);
#pragma unroll
    for (int e = 0; e < E; ++e) dst[r * pitch + c + e] = x[e];
  }
}

// ---------------------------------------------------------------------------
// The general kernel: fp32 on the CUDA cores (and, for no tokens at all, the
// states of either type), any width up to 128 (padded with zeros to DA).  A CTA of 16 x 16 threads owns kNS columns of c
// and of the state for one segment; each thread forms 4 x 4 elements of every
// product.  STATES: only the segment's own state is formed.  The CUDA cores
// bind: about 24 us for a chunk of 64 tokens, 128 x 128, of one slice.
// ---------------------------------------------------------------------------
template <int DA, bool STATES>
__global__ void __launch_bounds__(kThreads) linear_general_kernel(const LinearParams p) {
  constexpr int kPitch = DA + 4, MB = DA / 64;
  extern __shared__ float4 smem4[];
  float *sa = reinterpret_cast<float *>(smem4);        // [kC][kPitch]
  float *sb = sa + kC * kPitch;                        // [kC][kPitch]
  float *sc = sb + kC * kPitch;                        // [kC][kPadS]
  float *sp = sc + kC * kPadS;                         // [kC][kPadS]
  float *ss = sp + kC * kPadS;                         // [DA][kPadS]
  float *pw = ss + DA * kPadS;                         // [kC + 1]
  grid_dependency_wait();
  const int seg = blockIdx.x % p.nseg, slice = blockIdx.x / p.nseg % p.slices;
  const int64_t bh = blockIdx.x / (p.nseg * p.slices), b = bh / p.H;
  const int h = (int)(bh % p.H), col0 = slice * kNS;
  const int64_t n = seq_length(p, b);
  const int64_t begin = seg * p.seg_len, end = min(p.T, begin + p.seg_len), stop = min(n, end);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const float g = p.log_decay[h];
  if (threadIdx.x <= kC) pw[threadIdx.x] = decay_pow(g, threadIdx.x);

  float s[MB * 4][4];                                  // state rows mb * 64 + ty * 4 + i, columns tx * 4 + j
  float *states = p.states + ((bh * p.nstates + seg * p.step) * p.da) * p.dc;
#pragma unroll
  for (int m = 0; m < MB * 4; ++m) {
    const int row = (m / 4) * 64 + ty * 4 + m % 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = col0 + tx * 4 + j;
      s[m][j] = 0.f;
      if (!STATES && row < p.da && col < p.dc) {
        if (p.nseg > 1) s[m][j] = p.states_t ? states[(int64_t)col * p.da + row] : states[(int64_t)row * p.dc + col];
        else if (p.first) s[m][j] = first_at(p, bh, row, col);
      }
    }
  }
  for (int64_t i0 = begin; i0 < stop; i0 += kC) {
    const int len = (int)min((int64_t)kC, stop - i0);
    const int lead = (i0 == 0) ? p.first_pow : 1;      // the first row's weight of the state: lambda^lead
    __syncthreads();                                   // the last chunk's tiles are read
    if (!STATES) load_rows<DA>(p, sa, kPitch, p.a, p.a_stride, h, p.da, 0, b, n, i0, stop);
    load_rows<DA>(p, sb, kPitch, p.b, p.b_stride, h, p.da, 0, b, n, i0, stop);
    load_rows<kNS>(p, sc, kPadS, p.c, p.c_stride, h, p.dc, col0, b, n, i0, stop);
    if (!STATES) {
#pragma unroll
      for (int m = 0; m < MB * 4; ++m) {
        const int row = (m / 4) * 64 + ty * 4 + m % 4;
        *reinterpret_cast<float4 *>(ss + row * kPadS + tx * 4) = make_float4(s[m][0], s[m][1], s[m][2], s[m][3]);
      }
    }
    __syncthreads();
    if (!STATES) {
      // P: rows ty + 16 i, columns tx + 16 j
      float acc[4][4] = {};
#pragma unroll 4
      for (int k = 0; k < DA; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(sa + (ty + 16 * i) * kPitch + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(sb + (tx + 16 * j) * kPitch + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = ty + 16 * i, c = tx + 16 * j;
          sp[r * kPadS + c] = r >= c ? acc[i][j] * pw[r - c] : 0.f;
        }
      __syncthreads();
      // rows ty * 4 + i, columns tx * 4 + j: the state's part, weighted by row, then the chunk's own
      float o[4][4] = {};
#pragma unroll 4
      for (int k = 0; k < DA; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(sa + (ty * 4 + i) * kPitch + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(ss + (k + j) * kPadS + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[i][0] = fmaf(xs[j], y[j].x, o[i][0]);
            o[i][1] = fmaf(xs[j], y[j].y, o[i][1]);
            o[i][2] = fmaf(xs[j], y[j].z, o[i][2]);
            o[i][3] = fmaf(xs[j], y[j].w, o[i][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= pw[ty * 4 + i + lead];
#pragma unroll 4
      for (int k = 0; k < kC; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(sp + (ty * 4 + i) * kPadS + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(sc + (k + j) * kPadS + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[i][0] = fmaf(xs[j], y[j].x, o[i][0]);
            o[i][1] = fmaf(xs[j], y[j].y, o[i][1]);
            o[i][2] = fmaf(xs[j], y[j].z, o[i][2]);
            o[i][3] = fmaf(xs[j], y[j].w, o[i][3]);
          }
        }
      }
      const int col = col0 + tx * 4;
      if (col < p.dc) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = ty * 4 + i;
          if (r >= len) continue;
          float *y = (float *)p.out + (walk_row(p, b, n, i0 + r) * p.H + h) * p.dc + col;
          *reinterpret_cast<float4 *>(y) =
              make_float4(o[i][0] * p.alpha, o[i][1] * p.alpha, o[i][2] * p.alpha, o[i][3] * p.alpha);
        }
      }
    }
    // S = lambda^len S + sum_j lambda^{len-1-j} b_j c_j^T
    const float keep = decay_pow(g, len - 1 + lead);
#pragma unroll
    for (int m = 0; m < MB * 4; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[m][j] *= keep;
#pragma unroll 4
    for (int k = 0; k < len; ++k) {
      float4 y = *reinterpret_cast<const float4 *>(sc + k * kPadS + tx * 4);
      const float wk = pw[len - 1 - k];
      y.x *= wk; y.y *= wk; y.z *= wk; y.w *= wk;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const float4 x = *reinterpret_cast<const float4 *>(sb + k * kPitch + mb * 64 + ty * 4);
        const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[mb * 4 + i][0] = fmaf(xs[i], y.x, s[mb * 4 + i][0]);
          s[mb * 4 + i][1] = fmaf(xs[i], y.y, s[mb * 4 + i][1]);
          s[mb * 4 + i][2] = fmaf(xs[i], y.z, s[mb * 4 + i][2]);
          s[mb * 4 + i][3] = fmaf(xs[i], y.w, s[mb * 4 + i][3]);
        }
      }
    }
  }
  const bool write_last = !STATES && p.nseg == 1 && p.last;
  if (STATES || write_last) {
    float *dst = STATES ? states : p.last + bh * p.da * p.dc;
    // no token at all: the state passes through unchanged
    const float f = STATES ? 1.f : p.last_scale * (n > 0 ? decay_pow(g, p.last_pow) : 1.f);
#pragma unroll
    for (int m = 0; m < MB * 4; ++m) {
      const int row = (m / 4) * 64 + ty * 4 + m % 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = col0 + tx * 4 + j;
        if (row < p.da && col < p.dc) dst[(int64_t)row * p.dc + col] = s[m][j] * f;
      }
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
    const float f = p.last_scale * (n > 0 ? decay_pow(g, p.last_pow) : 1.f);
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

// Segments of the general kernel: the split with the least cost in waves of CTAs
// (two per SM up to 64 wide, else one: 137 KB of shared memory) times their
// chunks, in units of a chunk of the main kernel.  A chunk of the states' kernel
// is worth a third of one, a CTA's start 0.3 (with its state 0.6), the scan and
// the launches 0.4, a state written, scanned and read 0.0015.  Measured, fp32, 128 x 128,
// uncut against cut: 4 heads x 512 tokens 195 against 43 us, 4 heads x 4096
// 1506 against 145, 64 heads x 2048 767 against 1097 (three segments: uncut
// it stays).  The same with da and dc exchanged, so that two calls can share
// the segments' states.
static Split linear_split(int64_t B, int64_t T, int H, int da, int dc, int dtype) {
  if (B * H < 1 || T < 1) return {kChunk, 1, 1};
  const int64_t chunks = (T + kC - 1) / kC;
  if (B * H > 65535) return {chunks * kC, 1, 1};                 // the scan's grid; and the SMs are full
  if (linear_tc_supported(T, dtype)) return linear_tc_split(B * H, T);
  const int wide = da > dc ? da : dc;
  const int64_t have = B * H * general_slices(wide), slots = sm_count() * (int64_t)(wide <= 64 ? 2 : 1);
  auto waves = [&](int64_t ctas) { return (double)((ctas + slots - 1) / slots); };
  int64_t per = chunks;
  double least = waves(have) * ((double)chunks + 0.3);
  for (int n = 2; n <= 128 && n <= chunks; ++n) {
    const int64_t len = (chunks + n - 1) / n, segments = (chunks + len - 1) / len;
    const double cost = waves(have * segments) * ((double)len + 0.3) +
                        0.35 * waves(have * (segments - 1)) * ((double)len + 1.) + 0.4 +
                        0.0015 * (double)(B * H * segments);
    if (cost < least) {
      least = cost;
      per = len;
    }
  }
  return {per * kC, (int)((chunks + per - 1) / per), 1};
}

int64_t linear_workspace_floats(int64_t B, int64_t T, int H, int da, int dc, int dtype) {
  const Split s = linear_split(B, T, H, da, dc, dtype);
  return s.nseg > 1 ? B * H * s.nseg * s.nsub * da * dc : 0;
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
  p.log_decay = a.log_decay; p.lengths = a.lengths; p.alpha = a.alpha; p.reverse = a.reverse;
  p.first = a.first; p.first_t = a.first_t; p.first_pow = a.first_pow; p.first_scale = a.first_scale;
  p.last = a.last; p.last_scale = a.last_scale; p.last_pow = a.last_pow;
  p.states = a.workspace;
  p.states_t = a.states_t;
  p.wait_limit = std::min(wait_limit_cycles(), 1ll << 48);    // times a CTA's length, within 63 bits
  const int64_t BH = a.B * a.H;
  const bool tc = linear_tc_supported(a.T, a.dtype);
  // The states' kernel (states = true) or the main one.
  auto chunks = [&](const LinearParams &p, bool states) -> cudaError_t {
    if (tc) return launch_linear_tc(p, BH, states, a.stream);
    const int64_t ctas = BH * p.nseg * p.slices;
    auto go = [&](auto da) -> cudaError_t {
      constexpr int DA = decltype(da)::value;
      const size_t smem = (size_t)(2 * kC * (DA + 4) + 2 * kC * kPadS + DA * kPadS + kC + 4) * sizeof(float);
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
