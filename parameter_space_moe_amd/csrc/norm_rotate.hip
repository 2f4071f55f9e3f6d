// Norms of queries and keys for each head, with the rotation of their positions.
//
//   r = (c <x, x> + eps)^-1/2,  c = 1 / N or 1;   n = r x;   y = scale Rot(n w)
// and, for dL/dy,
//   d = scale Rot^T(dy);  dw = sum over tokens and heads of d n;
//   dx = r (d w - c <d w, n> n).
// Both are bound by memory: x is read and y written once (x and dy read, dx written).  A row
// of one head belongs to a power of two of lanes, 8 pairs of elements each, so that what is
// turned together is in one lane and the sums are a few lane exchanges.  A workgroup takes all
// heads of a few tokens and makes these tokens' cosines and sines once, in LDS: the
// angle is a product in 64 bits, whose whole turns are taken off before it is rounded (at
// position 10^6 an fp32 angle would be off by 0.06).  Everything else is fp32.
// 65536 tokens of 48 heads of 64, all turned, in bf16: 148 to 160 us, 5.0 to 5.4 TB/s (a copy:
// 5.3), in fp32 307, 5.2 TB/s.  32768 tokens of 36 heads of 128, bf16: forward 106 to 111 us, 5.4 to
// 5.7 TB/s (a part of it from the caches), backward 176 to 181 us, 5.0 to 5.1 TB/s.  256 tokens
// of 80 heads of 128, not turned: 5.1 us.  Sizes that are no multiple of 16 move element by
// element: 65536 tokens of 48 heads of 72 in 436 us in bf16 and 415 in fp32, backward 1070 and 695.
#include "pack.hpp"
#include "swimba_internal.hpp"

namespace swimba {
namespace {

int checked() { return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP; }

constexpr int kThreads = 256;
constexpr int kPairs = 8;         // per lane
constexpr int kTable = 2048;      // cosines and sines of a workgroup
constexpr int kWeightStride = 2 * kPairs + 4;  // eight lanes' packs in different banks

struct NormParams {
  const void *q, *k;              // x
  const void *gq, *gk;            // dL/dy (backward)
  void *oq, *ok;                  // y, or dx
  const float *wq, *wk;
  const int32_t* pos;
  const float* rates;
  float* part;                    // [workgroups, 2, N] sums of dw, or null
  int64_t T, q_stride, k_stride;
  int Hq, Hk, N, R;
  int tokens, heads;              // of a workgroup at a time
  int64_t groups;                 // of tokens
  float c, eps, q_scale;
  int out_bf16;
};

// Elements of pair `i` of lane `l`: the first R in pairs across the halves or of neighbours,
// the others of neighbours.  whole: eight pairs are two packs of eight.
template <bool NEIGHBOURS>
__device__ __forceinline__ int2 pair_at(int p, int R) {
  const int half = R >> 1;
  if (!NEIGHBOURS && p < half) return make_int2(p, p + half);
  return make_int2(2 * p, 2 * p + 1);
}

template <typename T>
__device__ __forceinline__ void load8(const T* at, float* out) {
  const Pack<T> v = load_pack(at, kPack);
#pragma unroll
  for (int i = 0; i < kPack; ++i) out[i] = to_f32(v.v[i]);
}
template <typename T>
__device__ __forceinline__ void store8(T* at, const float* in) {
  Pack<T> v;
#pragma unroll
  for (int i = 0; i < kPack; ++i) v.v[i] = from_f32<T>(in[i]);
  store_pack(at, v, kPack);
}

// A lane's share of a row: its pairs' first and second elements.
template <bool WHOLE, bool NEIGHBOURS, int LANES>
struct Share {
  int lane, N, R;
  // whole packs: where they start
  __device__ __forceinline__ int first() const {
    const int p = kPairs * lane;
    return !NEIGHBOURS && p < R / 2 ? p : 2 * p;
  }
  __device__ __forceinline__ int second() const {
    const int p = kPairs * lane;
    return !NEIGHBOURS && p < R / 2 ? p + R / 2 : 2 * p + 8;
  }
  __device__ __forceinline__ bool across() const {  // the pairs lie across the packs
    return !NEIGHBOURS && kPairs * lane < R / 2;
  }
  __device__ __forceinline__ int pair(int i) const {
    return WHOLE ? kPairs * lane + i : lane + i * LANES;
  }
  __device__ __forceinline__ bool inside() const { return 2 * kPairs * lane < N; }

  template <typename T>
  __device__ __forceinline__ void load(const T* row, float* a, float* b) const {
    if constexpr (WHOLE) {
      float x[8], y[8];
      const bool in = inside();
      load8(row + (in ? first() : 0), x);
      load8(row + (in ? second() : 0), y);
      const bool cross = across();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n0 = i < 4 ? x[2 * i & 7] : y[2 * i & 7];
        const float n1 = i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7];
        a[i] = in ? (cross ? x[i] : n0) : 0.f;
        b[i] = in ? (cross ? y[i] : n1) : 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int2 e = pair_at<NEIGHBOURS>(pair(i), R);
        a[i] = e.x < N ? to_f32(row[e.x]) : 0.f;
        b[i] = e.y < N ? to_f32(row[e.y]) : 0.f;
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, const float* a, const float* b) const {
    if constexpr (WHOLE) {
      if (!inside()) return;
      float x[8], y[8];
      const bool cross = across();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n0 = i & 1 ? b[i >> 1] : a[i >> 1];
        const float n1 = i & 1 ? b[4 + (i >> 1)] : a[4 + (i >> 1)];
        x[i] = cross ? a[i] : n0;
        y[i] = cross ? b[i] : n1;
      }
      store8(row + first(), x);
      store8(row + second(), y);
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int2 e = pair_at<NEIGHBOURS>(pair(i), R);
        if (e.x < N) row[e.x] = from_f32<T>(a[i]);
        if (e.y < N) row[e.y] = from_f32<T>(b[i]);
      }
    }
  }
};

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v, int lane) {
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) v += xor_lane_any(v, m, lane);
  return v;
}

// TI: x and dy; TO: y or dx.
template <typename TI, typename TO, int LANES, bool WHOLE, bool NEIGHBOURS, bool BACK>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormParams p) {
  __shared__ float2 table[kTable];
  __shared__ __attribute__((aligned(16))) float weights[2 * LANES * kWeightStride];
  __shared__ float sums[BACK ? 4 * 2 * 2 * kPairs * LANES : 1];
  constexpr int kRowsAtOnce = kThreads / LANES;
  const int lane = threadIdx.x & (LANES - 1), r0 = threadIdx.x / LANES;
  const int half = p.R >> 1;
  const Share<WHOLE, NEIGHBOURS, LANES> mine = {lane, p.N, p.R};
  const int h0 = (int)blockIdx.y * p.heads;
  const int heads = p.Hq + p.Hk - h0 < p.heads ? p.Hq + p.Hk - h0 : p.heads;

  // the weights as the lanes take them, in LDS: in registers they cost the backward pass a
  // wave per SIMD (145 instead of 121 registers; 217 us instead of 189)
  if (threadIdx.x < 2 * LANES) {
    const float* w = threadIdx.x < LANES ? p.wq : p.wk;
    float x[2 * kPairs];
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i) x[i] = 1.f;
    if (w != nullptr) mine.load(w, x, x + kPairs);
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i) weights[threadIdx.x * kWeightStride + i] = x[i];
  }
  __syncthreads();
  float dwq[2 * kPairs] = {}, dwk[2 * kPairs] = {};
  const int dt = kRowsAtOnce / heads, dh = kRowsAtOnce - dt * heads;  // to a thread's next row

  for (int64_t grp = blockIdx.x; grp < p.groups; grp += gridDim.x) {
    const int64_t t0 = grp * p.tokens;
    const int tokens = p.T - t0 < p.tokens ? (int)(p.T - t0) : p.tokens;
    if (half > 0) {
      __syncthreads();  // the last group's are done with
      for (int e = threadIdx.x; e < tokens * half; e += kThreads) {
        const int t = e / half, i = e - t * half;
        const double turns = (double)p.pos[t0 + t] * (double)p.rates[i] * 0.15915494309189535;
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        table[e] = make_float2(c, s);
      }
      __syncthreads();
    }
    int t = r0 / heads, h = r0 - t * heads;
    for (; t < tokens; ) {
      const bool isq = h0 + h < p.Hq;
      const int head = isq ? h0 + h : h0 + h - p.Hq;
      const int64_t tok = t0 + t;
      const int64_t from = tok * (isq ? p.q_stride : p.k_stride) + (int64_t)head * p.N;
      const int64_t to = (tok * (isq ? p.Hq : p.Hk) + head) * p.N;
      float a[kPairs], b[kPairs];
      mine.load(static_cast<const TI*>(isq ? p.q : p.k) + from, a, b);
      float ga[kPairs], gb[kPairs];
      if (BACK) mine.load(static_cast<const TI*>(isq ? p.gq : p.gk) + to, ga, gb);
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) sq = fmaf(a[i], a[i], fmaf(b[i], b[i], sq));
      sq = lanes_sum<LANES>(sq, (int)threadIdx.x & 63);
      const float r = __builtin_amdgcn_rsqf(fmaf(sq, p.c, p.eps));
      const float scale = isq ? p.q_scale : 1.f;
      float w[2 * kPairs];
#pragma unroll
      for (int i = 0; i < 2 * kPairs; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(
            weights + ((isq ? 0 : LANES) + lane) * kWeightStride + i);
        w[i] = f.x;
        w[i + 1] = f.y;
        w[i + 2] = f.z;
        w[i + 3] = f.w;
      }
      if constexpr (!BACK) {
        const float f = r * scale;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          a[i] *= f * w[i];
          b[i] *= f * w[kPairs + i];
          const int pi = mine.pair(i);
          if (pi < half) {
            const float2 cs = table[t * half + pi];
            const float x = a[i];
            a[i] = x * cs.x - b[i] * cs.y;
            b[i] = fmaf(b[i], cs.x, x * cs.y);
          }
        }
      } else {
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          ga[i] *= scale;
          gb[i] *= scale;
          const int pi = mine.pair(i);
          if (pi < half) {
            const float2 cs = table[t * half + pi];
            const float x = ga[i];
            ga[i] = fmaf(x, cs.x, gb[i] * cs.y);
            gb[i] = gb[i] * cs.x - x * cs.y;
          }
          a[i] *= r;
          b[i] *= r;
          const float da = ga[i] * a[i], db = gb[i] * b[i];
          dwq[i] += isq ? da : 0.f;
          dwk[i] += isq ? 0.f : da;
          dwq[kPairs + i] += isq ? db : 0.f;
          dwk[kPairs + i] += isq ? 0.f : db;
          ga[i] *= w[i];
          gb[i] *= w[kPairs + i];
          dot = fmaf(ga[i], a[i], fmaf(gb[i], b[i], dot));
        }
        dot = lanes_sum<LANES>(dot, (int)threadIdx.x & 63) * p.c;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          a[i] = r * fmaf(-dot, a[i], ga[i]);
          b[i] = r * fmaf(-dot, b[i], gb[i]);
        }
      }
      mine.store(static_cast<TO*>(isq ? p.oq : p.ok) + to, a, b);
      t += dt;
      h += dh;
      if (h >= heads) {
        h -= heads;
        ++t;
      }
    }
  }
  if constexpr (BACK) {
    if (p.part == nullptr) return;
    // over the wave's rows, then its waves, in order
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i) {
      float vq = dwq[i], vk = dwk[i];
#pragma unroll
      for (int m = LANES; m < 64; m <<= 1) {
        vq += xor_lane_any(vq, m, (int)threadIdx.x & 63);
        vk += xor_lane_any(vk, m, (int)threadIdx.x & 63);
      }
      if ((threadIdx.x & 63) < LANES) {
        sums[((wave * 2 + 0) * 2 * kPairs + i) * LANES + lane] = vq;
        sums[((wave * 2 + 1) * 2 * kPairs + i) * LANES + lane] = vk;
      }
    }
    __syncthreads();
    constexpr int kAll = 2 * 2 * kPairs * LANES;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    for (int e = threadIdx.x; e < kAll; e += kThreads) {
      const float v = (sums[e] + sums[kAll + e]) + (sums[2 * kAll + e] + sums[3 * kAll + e]);
      const int l = e % LANES, i = e / LANES % (2 * kPairs), which = e / (LANES * 2 * kPairs);
      const Share<WHOLE, NEIGHBOURS, LANES> its = {l, p.N, p.R};
      const int2 at = pair_at<NEIGHBOURS>(its.pair(i % kPairs), p.R);
      const int n = i < kPairs ? at.x : at.y;
      if (n < p.N) p.part[(block * 2 + which) * p.N + n] = v;
    }
  }
}

// dw[n] = sum over the workgroups' parts, in order, in 64 bits: 16 columns per workgroup, 64
// threads in turn of each, eight parts of a thread on their way at once.  1024 parts of 2 x 128
// in 5 us (four threads per column: 67).
constexpr int kSumRows = 64, kSumCols = 16;
__global__ __launch_bounds__(kSumRows * kSumCols) void norm_weights_kernel(const float* part,
                                                                          float* dwq, float* dwk,
                                                                          int64_t blocks, int N) {
  __shared__ double s[kSumRows][kSumCols];
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + col;
  double v = 0.0;
  if (c < 2 * N) {
    for (int64_t i = row; i < blocks; i += 8 * kSumRows) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t at = i + u * kSumRows;
        x[u] = part[(at < blocks ? at : 0) * 2 * N + c];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u * kSumRows < blocks) v += x[u];
    }
  }
  s[row][col] = v;
  __syncthreads();
  for (int w = kSumRows / 2; w > 0; w >>= 1) {
    if (row < w) s[row][col] += s[row + w][col];
    __syncthreads();
  }
  if (row == 0 && c < 2 * N) {
    float* out = c < N ? dwq : dwk;
    if (out != nullptr) out[c < N ? c : c - N] = (float)s[0][col];
  }
}

// Lanes of a row: a power of two whose pairs hold it.
int row_lanes(int N) {
  const int need = ((N + 1) / 2 + kPairs - 1) / kPairs;
  int l = 1;
  while (l < need) l <<= 1;
  return l;
}

struct NormGrid {
  int tokens, heads, ysize;
  int64_t groups, blocks;
};

// Tokens and heads of a workgroup.  All heads of a token share its cosines; where the tokens
// alone do not give two workgroups per CU their heads are cut, down to the rows that a
// workgroup takes at once.
NormGrid plan_norm(int64_t T, int H, int N, int R, bool back, int dev) {
  NormGrid g;
  const int rows = kThreads / row_lanes(N), half = R / 2;
  const int64_t target = 2LL * device_cus(dev);
  g.heads = H;
  while (g.heads > rows && T * ((H + g.heads - 1) / g.heads) < target) g.heads = (g.heads + 1) / 2;
  g.ysize = (H + g.heads - 1) / g.heads;
  // Two rounds of rows, if the tokens suffice: fewer repeat the wait for the table, with more
  // the workgroups' streams lie further apart (65536 tokens of 48 heads of 64: 168 us with one
  // token, 148 with 3, 167 with 11, 184 with 32).
  int64_t tokens = (2 * rows + g.heads - 1) / g.heads;
  if (tokens > T * g.ysize / target) tokens = T * g.ysize / target;
  if (half > 0 && tokens > kTable / half) tokens = kTable / half;
  g.tokens = tokens < 1 ? 1 : (int)tokens;
  g.groups = (T + g.tokens - 1) / g.tokens;
  // the gradients of the weights leave a part per workgroup: as many as run at once
  const int64_t most = back ? 4LL * device_cus(dev) : (int64_t)1 << 22;
  g.blocks = g.groups < most ? g.groups : most;
  return g;
}

template <typename TI, typename TO, int LANES, bool BACK>
int launch_lanes(const NormParams& p, const NormGrid& g, bool whole, bool neighbours,
                 hipStream_t s) {
  const dim3 grid((unsigned)g.blocks, (unsigned)g.ysize), t(kThreads);
  if (whole && neighbours)
    hipLaunchKernelGGL((norm_kernel<TI, TO, LANES, true, true, BACK>), grid, t, 0, s, p);
  else if (whole)
    hipLaunchKernelGGL((norm_kernel<TI, TO, LANES, true, false, BACK>), grid, t, 0, s, p);
  else if (neighbours)
    hipLaunchKernelGGL((norm_kernel<TI, TO, LANES, false, true, BACK>), grid, t, 0, s, p);
  else
    hipLaunchKernelGGL((norm_kernel<TI, TO, LANES, false, false, BACK>), grid, t, 0, s, p);
  return checked();
}

template <typename TI, typename TO, bool BACK>
int launch_types(const NormParams& p, const NormGrid& g, bool whole, bool neighbours,
                 hipStream_t s) {
  switch (row_lanes(p.N)) {
    case 1: return launch_lanes<TI, TO, 1, BACK>(p, g, whole, neighbours, s);
    case 2: return launch_lanes<TI, TO, 2, BACK>(p, g, whole, neighbours, s);
    case 4: return launch_lanes<TI, TO, 4, BACK>(p, g, whole, neighbours, s);
    case 8: return launch_lanes<TI, TO, 8, BACK>(p, g, whole, neighbours, s);
    case 16: return launch_lanes<TI, TO, 16, BACK>(p, g, whole, neighbours, s);
    default: return launch_lanes<TI, TO, 32, BACK>(p, g, whole, neighbours, s);
  }
}

template <bool BACK>
int launch_norm(const NormParams& p, const NormGrid& g, bool f32, bool neighbours, hipStream_t s) {
  // two packs per lane: pairs across the halves start at whole packs
  const bool whole = p.N % 16 == 0 && p.R % 16 == 0;
  if (f32)
    return p.out_bf16 ? launch_types<float, bf16_t, BACK>(p, g, whole, neighbours, s)
                      : launch_types<float, float, BACK>(p, g, whole, neighbours, s);
  return p.out_bf16 ? launch_types<bf16_t, bf16_t, BACK>(p, g, whole, neighbours, s)
                    : launch_types<bf16_t, float, BACK>(p, g, whole, neighbours, s);
}

NormParams norm_params(const swimba_norm_rotate_args* a, const NormGrid& g) {
  NormParams p = {};
  p.q = a->q;
  p.k = a->k;
  p.wq = a->wq;
  p.wk = a->wk;
  p.pos = a->positions;
  p.rates = a->rates;
  p.T = a->T;
  p.q_stride = a->q_stride != 0 ? a->q_stride : (int64_t)a->Hq * a->N;
  p.k_stride = a->k_stride != 0 ? a->k_stride : (int64_t)a->Hk * a->N;
  p.Hq = a->Hq;
  p.Hk = a->Hk;
  p.N = a->N;
  p.R = a->R;
  p.tokens = g.tokens;
  p.heads = g.heads;
  p.groups = g.groups;
  p.c = a->norm == SWIMBA_NORM_RMS ? 1.f / (float)a->N : 1.f;
  p.eps = a->eps;
  p.q_scale = a->q_scale;
  return p;
}

}  // namespace

int launch_norm_rotate(const swimba_norm_rotate_args* a, int dev, hipStream_t s) {
  if (a->T == 0) return SWIMBA_OK;
  const NormGrid g = plan_norm(a->T, a->Hq + a->Hk, a->N, a->R, false, dev);
  NormParams p = norm_params(a, g);
  p.oq = a->q_out;
  p.ok = a->k_out;
  p.out_bf16 = a->out_dtype == SWIMBA_BF16;
  return launch_norm<false>(p, g, a->in_dtype == SWIMBA_F32, a->pairs == SWIMBA_PAIRS_NEIGHBOURS,
                            s);
}

size_t norm_rotate_backward_bytes(const swimba_norm_rotate_grad_args* g, int dev) {
  const swimba_norm_rotate_args* a = &g->fwd;
  if (a->T == 0 || (g->dwq == nullptr && g->dwk == nullptr)) return 0;
  const NormGrid n = plan_norm(a->T, a->Hq + a->Hk, a->N, a->R, true, dev);
  return (size_t)n.blocks * n.ysize * 2 * a->N * sizeof(float);
}

int launch_norm_rotate_backward(const swimba_norm_rotate_grad_args* g, void* ws, int dev,
                                hipStream_t s) {
  const swimba_norm_rotate_args* a = &g->fwd;
  const bool weights = g->dwq != nullptr || g->dwk != nullptr;
  const NormGrid n = plan_norm(a->T, a->Hq + a->Hk, a->N, a->R, true, dev);
  float* part = static_cast<float*>(ws);
  if (a->T > 0) {
    NormParams p = norm_params(a, n);
    p.gq = g->dq_out;
    p.gk = g->dk_out;
    p.oq = g->dq;
    p.ok = g->dk;
    p.part = weights ? part : nullptr;
    p.out_bf16 = g->grad_dtype == SWIMBA_BF16;
    const int rc = launch_norm<true>(p, n, a->in_dtype == SWIMBA_F32,
                                     a->pairs == SWIMBA_PAIRS_NEIGHBOURS, s);
    if (rc != SWIMBA_OK) return rc;
  }
  if (!weights) return SWIMBA_OK;
  hipLaunchKernelGGL(norm_weights_kernel,
                     dim3((unsigned)((2 * a->N + kSumCols - 1) / kSumCols)),
                     dim3(kSumRows * kSumCols), 0, s, part, g->dwq, g->dwk,
                     a->T > 0 ? n.blocks * n.ysize : 0, a->N);
  return checked();
}

}  // namespace swimba
