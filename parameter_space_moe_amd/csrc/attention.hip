// Linear attention: host side of the walks (attention.hpp), the carry between
// segments, the gradients of the decays and the single-token step.
#include "attention.hpp"

namespace swimba {
namespace {

int checked() { return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP; }

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// First state of every segment from the segments' end states (in place; 13.7 us
// of the 64K-token prompt's 540):
// first(0) = s0, first(i + 1) = decay(i) first(i) + end(i).  One thread per
// state entry; the loads of the next segments do not wait for the sums.
__global__ __launch_bounds__(256) void attn_carry_kernel(AttnParams p) {
  const int64_t n = (int64_t)p.Kd * p.Cd, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t bh = blockIdx.y;
  if (e >= n) return;
  const int64_t row = e / p.Cd, c = e - row * p.Cd;
  float cur = p.s0 != nullptr ? p.s0[bh * n + row * p.sk + c * p.sc] : 0.f;
  float* st = p.seg_state + bh * p.nseg * n + e;
  const float* dec = p.seg_decay + bh * p.nseg;
  constexpr int kAhead = 8;
  float end[kAhead];
  for (int s = 0; s < p.nseg; s += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) end[i] = s + i < p.nseg - 1 ? st[(s + i) * n] : 0.f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s + i >= p.nseg) break;
      st[(s + i) * n] = cur;
      if (s + i < p.nseg - 1) cur = fmaf(dec[s + i], cur, end[i]);
    }
  }
}

// The log decays' gradient (below) where segments meet, from both walks' first
// states: the state before the boundary and the adjoint behind it, joined by the
// decay of the first token behind it.  And before the first token: <h0, dL/dh0>.
struct AnchorParams {
  const float *h, *adj;  // [B, H, nseg, n] first states of the dq and of the dk walk
  const float *h0, *dh0; // null: a first state of zero
  const float* g;
  double* out;           // [B, H, nseg - 1]
  double* begin;         // [B, H]
  int64_t n;
  int H, L, nseg, seg_chunks, token_decay;
  int known;             // values per sequence and head: nseg - 1, and one with h0
};

// out[b, h] = <a, b> over a state, in 64 bits.
constexpr int kDotThreads = 1024;
__device__ __forceinline__ double block_dot(const float* a, const float* b, int64_t n,
                                            double* part) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 8 * kDotThreads) {
    float x[8], y[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t e = i + u * kDotThreads;
      x[u] = a[e < n ? e : 0];
      y[u] = b[e < n ? e : 0];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u * kDotThreads < n) s += (double)x[u] * (double)y[u];
  }
  part[threadIdx.x] = s;
  __syncthreads();
  for (int w = kDotThreads / 2; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) part[threadIdx.x] += part[threadIdx.x + w];
    __syncthreads();
  }
  return part[0];
}

__global__ __launch_bounds__(kDotThreads) void attn_dot_kernel(const float* a, const float* b,
                                                               double* out, int64_t n) {
  __shared__ double part[kDotThreads];
  const int64_t at = (int64_t)blockIdx.x * n;
  const double s = block_dot(a + at, b + at, n, part);
  if (threadIdx.x == 0) out[blockIdx.x] = s;
}

__global__ __launch_bounds__(kDotThreads) void attn_anchor_kernel(AnchorParams p) {
  __shared__ double part[kDotThreads];
  const int64_t bh = blockIdx.x / p.known;
  // the boundary before segment i, or last the sequence's start
  const int i = (int)(blockIdx.x % p.known) + 1;
  if (i == p.nseg) {
    const double s = block_dot(p.h0 + bh * p.n, p.dh0 + bh * p.n, p.n, part);
    if (threadIdx.x == 0) p.begin[bh] = s;
    return;
  }
  const int64_t f = (bh * p.nseg + i) * p.n, r = (bh * p.nseg + p.nseg - i) * p.n;
  const double s = block_dot(p.h + f, p.adj + r, p.n, part);
  if (threadIdx.x == 0) {
    const int64_t t = (int64_t)i * p.seg_chunks * kChunk, b = bh / p.H, h = bh % p.H;
    const double d = (double)p.g[p.token_decay ? (b * p.L + t) * p.H + h : h] * 1.4426950408889634;
    const float e = exp2_sum(d < (double)kLeastLog2 ? (double)kLeastLog2 : d);
    p.out[bh * (p.nseg - 1) + i - 1] = e == 0.f ? 0.0 : s * (double)e;
  }
}

// Gradients of the log decays.  In a chunk, with row_r and col_s the sums of
// (q_r . k_s)(dy_r . v_s) D[r][s] over the pairs s <= r of the chunk (the walks'
// <q, dq> and <k, dk> inside the chunk), a_r what r reads of the chunk's first
// state and b_s what later chunks read of s, the slopes of neighbours differ by
//   dg_t - dg_{t+1} = u_t = row_t - col_t + a_t - b_t,
// and over a whole chunk the pairs' part of that sum is zero.  dg is known behind
// the last token (the product of state and adjoint there), where segments meet,
// and where a state is cleared: zero.  Every other token's is summed up from the
// nearest of these behind it, so that the rounding of what cancels stays inside
// a document and inside a segment (a whole walk is one segment).
// u of a token with an infinity or a NaN in k or v, and of the later ones, is not
// finite, and neither is that sum for the tokens before it, whose gradients do
// not depend on that k or v.  Where it is not, the sum from the nearest known
// value in front (the product of the first state and its gradient at the start)
// is taken if it is finite.
struct DecayGradParams {
  const float *zq, *zk;   // [B, H, ctiles, 2, L] of the dq and dk walks
  const double* x_end;    // [B, H] dg behind the last token, or null for zero
  const double* begin;    // [B, H] dg before the first token, or null for zero
  const double* anchor;   // [B, H, segments - 1] dg where segments meet, or null
  int seg_chunks, nseg;
  struct Chunk {          // the slopes' difference over a chunk
    double back;          // from its first token to its end, or to the first cleared state
    double fore;          // from its first token, or from the last cleared state, to its end
    int32_t cleared;      // whether there is one
  };
  Chunk* chunk;           // [B, H, chunks]
  double* part;           // [B, H, chunks] sums of dg (a decay per head), or null
  const float* g;
  float* dg;              // [B, L, H] or [H]
  int B, L, H, ctiles, nc, token_decay;
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

struct DecayTerms {
  double inside, a, b;
};

__device__ __forceinline__ DecayTerms decay_terms(const DecayGradParams& p, int64_t bh, int t) {
  DecayTerms r = {0.0, 0.0, 0.0};
  if (t < p.L) {
    for (int i = 0; i < p.ctiles; ++i) {
      const int64_t at = (bh * p.ctiles + i) * 2 * p.L + t;
      r.inside += (double)p.zq[at] - (double)p.zk[at];
      r.a += p.zq[at + p.L];
      r.b += p.zk[at + p.L];
    }
  }
  return r;
}

// Whether token t clears the state: nothing passes, whatever g is near by.
__device__ __forceinline__ bool clears(const DecayGradParams& p, int64_t bh, int t) {
  if (t >= p.L) return false;
  const int h = (int)(bh % p.H);
  return hw_exp2((p.token_decay ? p.g[(bh / p.H * p.L + t) * p.H + h] : p.g[h]) * kLog2e) == 0.f;
}

// First lane of a mask, 64 for none; last lane, -1 for none.
__device__ __forceinline__ int first_lane(uint64_t mask) {
  return mask != 0 ? __ffsll((unsigned long long)mask) - 1 : 64;
}
__device__ __forceinline__ int last_lane_of(uint64_t mask) {
  return 63 - __clzll((long long)mask);
}

__global__ __launch_bounds__(256) void attn_decay_diff_kernel(DecayGradParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= (int64_t)p.B * p.H * p.nc) return;
  const int64_t bh = w / p.nc;
  const int t = (int)(w - bh * p.nc) * kChunk + lane;
  const DecayTerms r = decay_terms(p, bh, t);
  const uint64_t mask = __ballot(clears(p, bh, t));
  const double back = wave_sum(lane < first_lane(mask) ? r.a - r.b : 0.0);
  const double fore = wave_sum(lane >= last_lane_of(mask) ? r.a - r.b : 0.0);
  if (lane == 0) {
    p.chunk[w].back = back;
    p.chunk[w].fore = fore;
    p.chunk[w].cleared = mask != 0;
  }
}

__device__ __forceinline__ bool finite(double v) { return fabs(v) < (double)__builtin_inff(); }

__global__ __launch_bounds__(256) void attn_decay_grad_kernel(DecayGradParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= (int64_t)p.B * p.H * p.nc) return;
  const int64_t bh = w / p.nc;
  const int c = (int)(w - bh * p.nc), h = (int)(bh % p.H), t = c * kChunk + lane;
  // up to the next segment's first chunk, or the end, or a chunk that clears
  int stop = p.nc;
  double known = p.x_end != nullptr ? p.x_end[bh] : 0.0;
  if (p.anchor != nullptr) {
    const int next = c / p.seg_chunks + 1;
    if (next < p.nseg) {
      stop = next * p.seg_chunks;
      known = p.anchor[bh * (p.nseg - 1) + next - 1];
    }
  }
  double x = 0.0;
  for (int i = c + 1; i < stop; i += 64) {
    DecayGradParams::Chunk n = {0.0, 0.0, 0};
    if (i + lane < stop) n = p.chunk[bh * p.nc + i + lane];
    const int first = first_lane(__ballot(n.cleared != 0));
    if (lane <= first) x += n.back;
    if (first < 64) {
      known = 0.0;
      break;
    }
  }
  x = wave_sum(x) + known;
  const DecayTerms r = decay_terms(p, bh, t);
  const bool clear = clears(p, bh, t);
  const uint64_t mask = __ballot(clear);
  // the next token that clears, behind this one
  const int next = first_lane(lane < 63 ? mask & (~0ull << (lane + 1)) : 0);
  const double u = r.inside + r.a - r.b;
  double dg = u;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double o = __shfl_down(dg, m);
    if (lane + m < next) dg += o;
  }
  if (next == 64) dg += x;
  const bool lost = t < p.L && !clear && !finite(dg);
  if (__ballot(lost)) {
    const int seg = p.anchor != nullptr ? c / p.seg_chunks : 0;
    double in_front = seg > 0 ? p.anchor[bh * (p.nseg - 1) + seg - 1]
                              : (p.begin != nullptr ? p.begin[bh] : 0.0);
    double y = 0.0;
    for (int i = c - 1; i >= seg * p.seg_chunks; i -= 64) {
      DecayGradParams::Chunk n = {0.0, 0.0, 0};
      if (i - lane >= seg * p.seg_chunks) n = p.chunk[bh * p.nc + i - lane];
      const int first = first_lane(__ballot(n.cleared != 0));
      if (lane <= first) y -= n.fore;
      if (first < 64) {
        in_front = 0.0;
        break;
      }
    }
    y = wave_sum(y) + in_front;
    const int from = last_lane_of(mask & (~0ull >> (63 - lane)));  // this token's document
    double before = u;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double o = __shfl_up(before, m);
      if (lane - m >= (from < 0 ? 0 : from)) before += o;
    }
    before = __shfl_up(before, 1);  // without this token's own
    const double fore = (from < 0 ? y : 0.0) - (lane > 0 ? before : 0.0);
    if (lost && finite(fore)) dg = fore;
  }
  if (clear || t >= p.L) dg = 0.0;
  if (t < p.L && p.token_decay) p.dg[(bh / p.H * p.L + t) * p.H + h] = (float)dg;
  if (p.part != nullptr) {
    dg = wave_sum(dg);
    if (lane == 0) p.part[w] = dg;
  }
}

// dg[h] = sum over sequences and chunks, one workgroup per head.
__global__ __launch_bounds__(256) void attn_decay_sum_kernel(const double* part, float* dg, int B,
                                                             int H, int nc) {
  __shared__ double s[256];
  const int h = blockIdx.x;
  double v = 0.0;
  for (int64_t i = threadIdx.x; i < (int64_t)B * nc; i += 256) {
    const int64_t b = i / nc;
    v += part[(b * H + h) * nc + (i - b * nc)];
  }
  s[threadIdx.x] = v;
  __syncthreads();
  for (int w = 128; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) s[threadIdx.x] += s[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[h] = (float)s[0];
}

// out[t, g, :] = sum over the heads of group g, in order, of in[t, h, :].
template <typename TO>
__global__ __launch_bounds__(256) void attn_share_sum_kernel(const float* in, TO* out, int64_t rows,
                                                             int share, int N) {
  const int ppr = (N + kPack - 1) / kPack;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = i / ppr;
  if (r >= rows) return;
  const int c = (int)(i - r * ppr) * kPack;
  float acc[kPack] = {};
  for (int s = 0; s < share; ++s) {
    const Pack<float> v = load_pack(in + (r * share + s) * N + c, N - c);
#pragma unroll
    for (int k = 0; k < kPack; ++k) acc[k] += v.v[k];
  }
  Pack<TO> o;
#pragma unroll
  for (int k = 0; k < kPack; ++k) o.v[k] = from_f32<TO>(acc[k]);
  store_pack(out + r * N + c, o, N - c);
}

// One token: h' = e^g h + k v^T, y = h'^T q.  The state is read and written
// once (8 bytes per entry against 2 multiply-adds), so the rest only has to
// stay out of the way.  A workgroup takes `slice` columns of one head's state:
// V of them per thread, rows spread over the workgroup's row lanes, and adds
// the row lanes' parts of y in LDS in order.  256 sequences of 40 heads of
// 128 x 128: 265 us, 5.1 TB/s, against 253 us of a plain copy of that state.
struct AttnStepParams {
  const void *q, *k, *v;
  const float* g;
  const float* state;
  float* out;
  void* y;
  int H, share, N, P, token_decay, y_bf16;
  int slice, slices, cg;  // columns per workgroup, workgroups per head, column groups
};

constexpr int kMaxRows = 256;  // N

template <typename TI, int V>
__global__ __launch_bounds__(256) void attn_step_kernel(AttnStepParams p) {
  __shared__ float sq[kMaxRows], sk[kMaxRows];
  __shared__ float part[256 * V];
  const int64_t bh = blockIdx.x / p.slices;
  const int c0 = (int)(blockIdx.x % p.slices) * p.slice;
  const int64_t b = bh / p.H;
  const int h = (int)(bh - b * p.H);
  const int rl = 256 / p.cg;  // row lanes
  const int r0 = threadIdx.x / p.cg, cg = threadIdx.x % p.cg, c = c0 + cg * V;
  const int end = c0 + p.slice < p.P ? c0 + p.slice : p.P;
  const bool on = r0 < rl && c < end;  // V divides P where it is not one
  const float* st = p.state + bh * p.N * p.P + c;
  float* so = p.out + bh * p.N * p.P + c;

  constexpr int kAhead = 16 / V > 8 ? 8 : (V == 4 ? 8 : 16);
  float cur[kAhead][V];
  auto fetch = [&](int base) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int n = base + i * rl;
      if (on && n < p.N) {
        if constexpr (V == 4) {
          const float4 f = *reinterpret_cast<const float4*>(st + (int64_t)n * p.P);
          cur[i][0] = f.x; cur[i][1] = f.y; cur[i][2] = f.z; cur[i][3] = f.w;
        } else {
          cur[i][0] = st[(int64_t)n * p.P];
        }
      }
    }
  };
  fetch(r0);  // in flight while q, k and the decay come
  const TI* q = static_cast<const TI*>(p.q) + (b * (p.H / p.share) + h / p.share) * p.N;
  const TI* k = static_cast<const TI*>(p.k) + (b * (p.H / p.share) + h / p.share) * p.N;
  if ((int)threadIdx.x < p.N) {
    sq[threadIdx.x] = to_f32(q[threadIdx.x]);
    sk[threadIdx.x] = to_f32(k[threadIdx.x]);
  }
  float vv[V], acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    vv[j] = on ? to_f32(static_cast<const TI*>(p.v)[bh * p.P + c + j]) : 0.f;
    acc[j] = 0.f;
  }
  const float e = hw_exp2(p.g[p.token_decay ? bh : h] * kLog2e);
  __syncthreads();
  for (int base = r0; base < p.N; base += kAhead * rl) {
    if (base != r0) fetch(base);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int n = base + i * rl;
      if (!on || n >= p.N) continue;
      const float kn = sk[n], qn = sq[n];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        cur[i][j] = fmaf(e, cur[i][j], kn * vv[j]);
        acc[j] = fmaf(qn, cur[i][j], acc[j]);
      }
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(so + (int64_t)n * p.P) =
            make_float4(cur[i][0], cur[i][1], cur[i][2], cur[i][3]);
      else
        so[(int64_t)n * p.P] = cur[i][0];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) part[threadIdx.x * V + j] = acc[j];
  __syncthreads();
  const int col = threadIdx.x;
  if (col < p.cg * V && c0 + col < end) {
    float s = 0.f;
    for (int r = 0; r < rl; ++r) s += part[r * p.cg * V + col];
    const int64_t at = bh * p.P + c0 + col;
    if (p.y_bf16) static_cast<bf16_t*>(p.y)[at] = from_f32<bf16_t>(s);
    else static_cast<float*>(p.y)[at] = s;
  }
}

__global__ __launch_bounds__(256) void attn_copy_kernel(const float* in, float* out, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    out[i] = in != nullptr ? in[i] : 0.f;
}

// The walks load whole packs inside a tensor.  One of fewer elements than a pack
// (a token of a few features) is first copied to a slot of the workspace.
template <typename T>
__global__ __launch_bounds__(64) void attn_tiny_kernel(const T* in, T* out, int n) {
  if (threadIdx.x < kPack) out[threadIdx.x] = (int)threadIdx.x < n ? in[threadIdx.x] : T(0);
}
bool is_tiny(int64_t n) { return n < kPack; }

// How one walk is laid out over the device.
struct WalkPlan {
  int waves = 1, nseg = 1, seg_chunks = 1;
  size_t state_bytes = 0, decay_bytes = 0;
  size_t bytes() const { return state_bytes + decay_bytes; }
};

WalkPlan plan_walk(bool f32, int B, int L, int H, int share, int Kd, int Cd, int dev) {
  WalkPlan w;
  const int ctiles = (Cd + 31) / 32;
  const int64_t units = (int64_t)share * ctiles;
  w.waves = attn_waves(f32, Kd, Cd, units);
  const int64_t nc = (L + kChunk - 1) / kChunk;
  const int64_t base = (int64_t)B * (H / share) * ((units + w.waves - 1) / w.waves);
  // as many workgroups as the device holds at once, from the independent walks
  // or from segments of them (whose first states cost a pass over k and v)
  const int64_t hold = (int64_t)device_cus(dev) *
                       (f32 ? attn_resident<float>(Kd, w.waves)
                            : attn_resident<bf16_t>(Kd, w.waves));
  int64_t want = base > 0 ? hold / base : 1;
  if (want > nc) want = nc;
  // Four waves of a lone workgroup take every SIMD of a CU: halves of such walks
  // would only add the pass (8 x 4096 tokens, 32 heads of 128 x 128, both on one
  // card: 410 us in halves, 387 us whole).  Two waves leave SIMDs idle, and halves
  // would gain there (4 x 8192, 64 heads of 128 x 64: 1049 us against 1268 us as it
  // is; 3 x 3000, 100 heads of 64 x 64: 214 us against 263 us): not taken yet.
  if (want < 3 || nc < 4) want = 1;
  w.seg_chunks = (int)((nc + want - 1) / want);
  if (w.seg_chunks < 1) w.seg_chunks = 1;
  w.nseg = nc > 0 ? (int)((nc + w.seg_chunks - 1) / w.seg_chunks) : 1;
  if (w.nseg > 1) {
    w.state_bytes = align256((size_t)B * H * w.nseg * Kd * Cd * sizeof(float));
    w.decay_bytes = align256((size_t)B * H * w.nseg * sizeof(float));
  }
  return w;
}

int dispatch(const AttnParams& p, bool f32, bool state, bool exact, hipStream_t s) {
  const int k = p.Kd;
  if (f32) {
    if (k <= 32) return attn_f32_32(p, state, exact, s);
    if (k <= 64) return attn_f32_64(p, state, exact, s);
    if (k <= 128) return attn_f32_128(p, state, exact, s);
    return attn_f32_256(p, state, exact, s);
  }
  if (k <= 32) return attn_bf16_32(p, state, exact, s);
  if (k <= 64) return attn_bf16_64(p, state, exact, s);
  if (k <= 128) return attn_bf16_128(p, state, exact, s);
  return attn_bf16_256(p, state, exact, s);
}

// One walk; ws holds the plan's segment states, or `turned` the transposed first
// states of the same segments from another walk.
int walk(AttnParams p, const WalkPlan& w, bool f32, bool exact, unsigned char* ws, hipStream_t s,
         float* turned = nullptr) {
  p.nseg = w.nseg;
  p.seg_chunks = w.seg_chunks;
  p.ctiles = (p.Cd + 31) / 32;
  p.fk = turned != nullptr ? 1 : p.Cd;
  p.fc = turned != nullptr ? p.Kd : 1;
  if (turned != nullptr) {
    p.seg_state = turned;
  } else if (w.nseg > 1) {
    p.seg_state = reinterpret_cast<float*>(ws);
    p.seg_decay = reinterpret_cast<float*>(ws + w.state_bytes);
    const int rc = dispatch(p, f32, true, true, s);
    if (rc != SWIMBA_OK) return rc;
    const int64_t n = (int64_t)p.Kd * p.Cd;
    hipLaunchKernelGGL(attn_carry_kernel, dim3((unsigned)((n + 255) / 256), (unsigned)(p.B * p.H)),
                       dim3(256), 0, s, p);
    if (checked() != SWIMBA_OK) return SWIMBA_EHIP;
  }
  return dispatch(p, f32, false, exact, s);
}

AttnParams base_params(const swimba_linear_attention_args* a) {
  AttnParams p = {};
  p.g = a->log_decay;
  p.B = a->B;
  p.L = a->L;
  p.H = a->H;
  p.token_decay = a->decay_form == SWIMBA_DECAY_TOKEN;
  return p;
}

int64_t key_elements(const swimba_linear_attention_args* a) {
  return (int64_t)a->B * a->L * a->G * a->N;
}
int64_t value_elements(const swimba_linear_attention_args* a) {
  return (int64_t)a->B * a->L * a->H * a->P;
}
// Slots behind the rest of the workspace for `slots` operands.
size_t tiny_bytes(const swimba_linear_attention_args* a, int slots) {
  return is_tiny(key_elements(a)) || is_tiny(value_elements(a)) ? slots * kTinySlot : 0;
}

struct GradPlan {
  WalkPlan q, v;  // dq and dk walk (states [P][N]), dv walk (states [N][P])
  // The dk and the dv walk have the same states, transposed: cut into the same
  // segments, the second takes the first's (24 heads of 64 x 64: 26 us less of
  // 273; 32 heads of 128 x 128: 50 of 726).  It reads them element by element: four
  // rows of a column per load made walks of 128 rows spill (1.4B-like prompts 388 ->
  // 537 us).
  bool turned = false;
  size_t off_zq = 0, off_zk = 0, off_chunk = 0, off_part = 0, off_x = 0, off_begin = 0, off_end = 0, off_dh0 = 0, off_rows = 0;
  size_t off_tiny = 0, off_adj = 0, off_v = 0, off_anchor = 0;
  size_t bytes = 0;
  int nc = 0, ntiles = 0;
};

GradPlan plan_grad(const swimba_linear_attention_grad_args* g, int dev) {
  const swimba_linear_attention_args* a = &g->fwd;
  const bool f32 = a->in_dtype == SWIMBA_F32;
  GradPlan r;
  r.q = plan_walk(f32, a->B, a->L, a->H, 1, a->P, a->N, dev);
  r.v = plan_walk(f32, a->B, a->L, a->H, a->H / a->G, a->N, a->P, dev);
  r.nc = (a->L + kChunk - 1) / kChunk;
  r.ntiles = (a->N + 31) / 32;
  // segment states of the dq and dk walks (the decays' gradient meets both) and,
  // where they are not the dk walk's, of the dv walk
  size_t o = r.q.bytes();
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  const size_t bh = (size_t)a->B * a->H;
  r.off_adj = take(r.q.bytes());
  r.turned = r.q.nseg > 1 && r.v.nseg == r.q.nseg && r.v.seg_chunks == r.q.seg_chunks;
  r.off_v = take(r.turned ? 0 : r.v.bytes());
  r.off_anchor = take(r.q.nseg > 1 ? bh * (r.q.nseg - 1) * sizeof(double) : 0);
  r.off_zq = take(bh * r.ntiles * 2 * a->L * sizeof(float));
  r.off_zk = take(bh * r.ntiles * 2 * a->L * sizeof(float));
  r.off_chunk = take(bh * r.nc * sizeof(DecayGradParams::Chunk));
  r.off_part = take(a->decay_form == SWIMBA_DECAY_HEAD ? bh * r.nc * sizeof(double) : 0);
  r.off_x = take(bh * sizeof(double));
  r.off_begin = take(a->h0 != nullptr ? bh * sizeof(double) : 0);
  r.off_dh0 = take(a->h0 != nullptr && g->dh0 == nullptr ? bh * a->N * a->P * sizeof(float) : 0);
  r.off_end = take(g->dh_final != nullptr ? bh * a->N * a->P * sizeof(float) : 0);
  // per-head rows of dq, then of dk, where heads share them
  r.off_rows = take(a->H != a->G ? bh * a->L * a->N * sizeof(float) : 0);
  r.off_tiny = take(tiny_bytes(a, 4));
  r.bytes = o;
  return r;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<unsigned char*>(ws) + off);
}

int share_sum(const float* rows, void* out, swimba_dtype d, const swimba_linear_attention_args* a,
              hipStream_t s) {
  return sum_shared_heads(rows, out, d, (int64_t)a->B * a->L * a->G, a->H / a->G, a->N, s);
}

}  // namespace

int copy_or_zero(const float* in, float* out, int64_t n, hipStream_t s) {
  if (n <= 0) return SWIMBA_OK;
  const int64_t wg = (n + 255) / 256 < (1 << 20) ? (n + 255) / 256 : 1 << 20;
  hipLaunchKernelGGL(attn_copy_kernel, dim3((unsigned)wg), dim3(256), 0, s, in, out, n);
  return checked();
}

const void* whole_packs(const void* rows, int64_t n, bool f32, unsigned char* slot, hipStream_t s,
                        int* rc) {
  if (!is_tiny(n) || *rc != SWIMBA_OK) return rows;
  if (f32)
    hipLaunchKernelGGL(attn_tiny_kernel<float>, dim3(1), dim3(64), 0, s,
                       static_cast<const float*>(rows), reinterpret_cast<float*>(slot), (int)n);
  else
    hipLaunchKernelGGL(attn_tiny_kernel<bf16_t>, dim3(1), dim3(64), 0, s,
                       static_cast<const bf16_t*>(rows), reinterpret_cast<bf16_t*>(slot), (int)n);
  *rc = checked();
  return slot;
}

int sum_shared_heads(const float* rows, void* out, swimba_dtype d, int64_t n, int share, int N,
                     hipStream_t s) {
  const int64_t packs = n * ((N + kPack - 1) / kPack);
  const dim3 grid((unsigned)((packs + 255) / 256));
  if (d == SWIMBA_BF16)
    hipLaunchKernelGGL((attn_share_sum_kernel<bf16_t>), grid, dim3(256), 0, s, rows,
                       static_cast<bf16_t*>(out), n, share, N);
  else
    hipLaunchKernelGGL((attn_share_sum_kernel<float>), grid, dim3(256), 0, s, rows,
                       static_cast<float*>(out), n, share, N);
  return checked();
}

int sum_decay_parts(const double* part, float* dg, int B, int H, int nc, hipStream_t s) {
  hipLaunchKernelGGL(attn_decay_sum_kernel, dim3(H), dim3(256), 0, s, part, dg, B, H, nc);
  return checked();
}

size_t attention_bytes(const swimba_linear_attention_args* a, int dev) {
  if (a->B == 0 || a->L == 0) return 0;
  const size_t walk =
      plan_walk(a->in_dtype == SWIMBA_F32, a->B, a->L, a->H, a->H / a->G, a->N, a->P, dev).bytes();
  return walk + tiny_bytes(a, 3);
}

int launch_attention(const swimba_linear_attention_args* a, void* ws, int dev, hipStream_t s) {
  const int64_t states = (int64_t)a->B * a->H * a->N * a->P;
  if (a->B == 0 || a->L == 0)
    return a->h_final != nullptr ? copy_or_zero(a->h0, a->h_final, states, s) : SWIMBA_OK;
  const bool f32 = a->in_dtype == SWIMBA_F32;
  const WalkPlan w = plan_walk(f32, a->B, a->L, a->H, a->H / a->G, a->N, a->P, dev);
  AttnParams p = base_params(a);
  unsigned char* slot = static_cast<unsigned char*>(ws) + w.bytes();
  int rc = SWIMBA_OK;
  p.q = whole_packs(a->q, key_elements(a), f32, slot, s, &rc);
  p.k = whole_packs(a->k, key_elements(a), f32, slot + kTinySlot, s, &rc);
  p.v = whole_packs(a->v, value_elements(a), f32, slot + 2 * kTinySlot, s, &rc);
  if (rc != SWIMBA_OK) return rc;
  p.y = a->y;
  p.qshare = a->H / a->G;
  p.vshare = 1;
  p.Kd = a->N;
  p.Cd = a->P;
  p.y_bf16 = a->y_dtype == SWIMBA_BF16;
  p.s0 = a->h0;
  p.s_final = a->h_final;
  p.sk = a->P;
  p.sc = 1;
  return walk(p, w, f32, a->y_dtype == SWIMBA_F32, static_cast<unsigned char*>(ws), s);
}

size_t attention_backward_bytes(const swimba_linear_attention_grad_args* g, int dev) {
  if (g->fwd.B == 0 || g->fwd.L == 0) return 0;
  return plan_grad(g, dev).bytes;
}

int launch_attention_backward(const swimba_linear_attention_grad_args* g, void* ws, int dev,
                              hipStream_t s) {
  const swimba_linear_attention_args* a = &g->fwd;
  const int64_t states = (int64_t)a->B * a->H * a->N * a->P;
  if (a->B == 0 || a->L == 0) {
    int rc = SWIMBA_OK;
    if (g->dh0 != nullptr) rc = copy_or_zero(g->dh_final, g->dh0, states, s);
    if (rc == SWIMBA_OK && a->decay_form == SWIMBA_DECAY_HEAD)
      rc = copy_or_zero(nullptr, g->dlog_decay, a->H, s);
    return rc;
  }
  const bool f32 = a->in_dtype == SWIMBA_F32, shared = a->H != a->G;
  const GradPlan r = plan_grad(g, dev);
  unsigned char* seg = static_cast<unsigned char*>(ws);
  float *zq = at<float>(ws, r.off_zq), *zk = at<float>(ws, r.off_zk);
  float *rows = at<float>(ws, r.off_rows), *end = at<float>(ws, r.off_end);

  unsigned char* slot = at<unsigned char>(ws, r.off_tiny);
  int rc = SWIMBA_OK;
  const void* q = whole_packs(a->q, key_elements(a), f32, slot, s, &rc);
  const void* k = whole_packs(a->k, key_elements(a), f32, slot + kTinySlot, s, &rc);
  const void* v = whole_packs(a->v, value_elements(a), f32, slot + 2 * kTinySlot, s, &rc);
  const void* dy = whole_packs(g->dy, value_elements(a), f32, slot + 3 * kTinySlot, s, &rc);
  if (rc != SWIMBA_OK) return rc;

  // dq = walk(dY, V, K)
  AttnParams p = base_params(a);
  p.q = dy;
  p.k = v;
  p.v = k;
  p.qshare = 1;
  p.vshare = a->H / a->G;
  p.Kd = a->P;
  p.Cd = a->N;
  p.sk = 1;
  p.sc = a->P;
  p.s0 = a->h0;
  p.s_final = g->dh_final != nullptr ? end : nullptr;
  p.z = q;
  p.zsum = zq;
  p.y = shared ? static_cast<void*>(rows) : g->dq;
  p.y_bf16 = !shared && g->grad_dtype == SWIMBA_BF16;
  rc = walk(p, r.q, f32, true, seg, s);
  if (rc == SWIMBA_OK && shared) rc = share_sum(rows, g->dq, g->grad_dtype, a, s);
  if (rc != SWIMBA_OK) return rc;

  // dk = backward walk(V, dY, Q)
  p.q = v;
  p.k = dy;
  p.v = q;
  p.reverse = 1;
  p.s0 = g->dh_final;
  p.s_final = nullptr;
  p.z = k;
  p.zsum = zk;
  p.y = shared ? static_cast<void*>(rows) : g->dk;
  rc = walk(p, r.q, f32, true, at<unsigned char>(ws, r.off_adj), s);
  if (rc == SWIMBA_OK && shared) rc = share_sum(rows, g->dk, g->grad_dtype, a, s);
  if (rc != SWIMBA_OK) return rc;

  // <h, dL/dh> behind the last token, before dh0 is written (it may be dh_final)
  double* x_end = nullptr;
  if (g->dh_final != nullptr) {
    x_end = at<double>(ws, r.off_x);
    hipLaunchKernelGGL(attn_dot_kernel, dim3(a->B * a->H), dim3(kDotThreads), 0, s, end,
                       g->dh_final, x_end, (int64_t)a->N * a->P);
    if (checked() != SWIMBA_OK) return SWIMBA_EHIP;
  }

  // dv = backward walk(K, Q, dY), whose last state is dh0
  p = base_params(a);
  p.q = k;
  p.k = q;
  p.v = dy;
  p.qshare = a->H / a->G;
  p.vshare = 1;
  p.Kd = a->N;
  p.Cd = a->P;
  p.sk = a->P;
  p.sc = 1;
  p.reverse = 1;
  p.s0 = g->dh_final;
  float* dh0 = g->dh0 == nullptr && a->h0 != nullptr ? at<float>(ws, r.off_dh0) : g->dh0;
  p.s_final = dh0;
  p.y = g->dv;
  p.y_bf16 = g->grad_dtype == SWIMBA_BF16;
  rc = walk(p, r.v, f32, g->grad_dtype == SWIMBA_F32, at<unsigned char>(ws, r.off_v), s,
            r.turned ? at<float>(ws, r.off_adj) : nullptr);
  if (rc != SWIMBA_OK) return rc;

  DecayGradParams d;
  d.zq = zq;
  d.zk = zk;
  d.x_end = x_end;
  d.anchor = nullptr;
  d.begin = nullptr;
  d.seg_chunks = r.q.seg_chunks;
  d.nseg = r.q.nseg;
  d.chunk = at<DecayGradParams::Chunk>(ws, r.off_chunk);
  d.part = a->decay_form == SWIMBA_DECAY_HEAD ? at<double>(ws, r.off_part) : nullptr;
  d.g = a->log_decay;
  d.dg = g->dlog_decay;
  d.B = a->B;
  d.L = a->L;
  d.H = a->H;
  d.ctiles = r.ntiles;
  d.nc = r.nc;
  d.token_decay = a->decay_form == SWIMBA_DECAY_TOKEN;
  AnchorParams x;
  x.known = r.q.nseg - 1 + (a->h0 != nullptr ? 1 : 0);
  if (x.known > 0) {
    x.h = reinterpret_cast<const float*>(seg);
    x.adj = at<float>(ws, r.off_adj);
    x.h0 = a->h0;
    x.dh0 = dh0;
    x.g = a->log_decay;
    x.out = at<double>(ws, r.off_anchor);
    x.begin = at<double>(ws, r.off_begin);
    x.n = (int64_t)a->N * a->P;
    x.H = a->H;
    x.L = a->L;
    x.nseg = r.q.nseg;
    x.seg_chunks = r.q.seg_chunks;
    x.token_decay = d.token_decay;
    hipLaunchKernelGGL(attn_anchor_kernel, dim3((unsigned)(a->B * a->H * x.known)),
                       dim3(kDotThreads), 0, s, x);
    if (r.q.nseg > 1) d.anchor = x.out;
    if (a->h0 != nullptr) d.begin = x.begin;
  }
  const unsigned wg = (unsigned)(((int64_t)a->B * a->H * r.nc + 3) / 4);
  hipLaunchKernelGGL(attn_decay_diff_kernel, dim3(wg), dim3(256), 0, s, d);
  hipLaunchKernelGGL(attn_decay_grad_kernel, dim3(wg), dim3(256), 0, s, d);
  if (d.part != nullptr)
    hipLaunchKernelGGL(attn_decay_sum_kernel, dim3(a->H), dim3(256), 0, s, d.part, g->dlog_decay,
                       a->B, a->H, r.nc);
  return checked();
}

int launch_attention_step(const swimba_linear_attention_step_args* a, int dev, hipStream_t s) {
  AttnStepParams p;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.g = a->log_decay;
  p.state = a->state;
  p.out = a->state_out != nullptr ? a->state_out : a->state;
  p.y = a->y;
  p.H = a->H;
  p.share = a->H / a->G;
  p.N = a->N;
  p.P = a->P;
  p.token_decay = a->decay_form == SWIMBA_DECAY_TOKEN;
  p.y_bf16 = a->y_dtype == SWIMBA_BF16;
  const bool vec = a->P % 4 == 0 && ((reinterpret_cast<uintptr_t>(p.state) |
                                      reinterpret_cast<uintptr_t>(p.out)) & 15) == 0;
  const int V = vec ? 4 : 1;
  // columns per workgroup: narrower slices, down to 64-byte rows, where the
  // heads alone do not give two workgroups per CU
  int slice = vec ? 128 : 64;
  const int64_t heads = (int64_t)a->B * a->H, target = 2LL * device_cus(dev);
  while (slice > 16 && heads * ((a->P + slice - 1) / slice) < target) slice >>= 1;
  p.slice = slice < a->P ? slice : a->P;
  p.slices = (a->P + p.slice - 1) / p.slice;
  p.cg = (p.slice + V - 1) / V;
  const int64_t grid = heads * p.slices;
  const dim3 g((unsigned)grid), t(256);
  const bool bf = a->in_dtype == SWIMBA_BF16;
  if (vec && bf) hipLaunchKernelGGL((attn_step_kernel<bf16_t, 4>), g, t, 0, s, p);
  else if (vec) hipLaunchKernelGGL((attn_step_kernel<float, 4>), g, t, 0, s, p);
  else if (bf) hipLaunchKernelGGL((attn_step_kernel<bf16_t, 1>), g, t, 0, s, p);
  else hipLaunchKernelGGL((attn_step_kernel<float, 1>), g, t, 0, s, p);
  return checked();
}

}  // namespace swimba
