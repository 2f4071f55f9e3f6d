// The gated delta rule: host side of its phases (delta.hpp) and the single-token step.
#include "delta.hpp"

#include <algorithm>
#include <cmath>

namespace swimba {
namespace {

int checked() { return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP; }

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<unsigned char*>(ws) + off);
}

int phase(const DeltaParams& p, bool f32, int which, hipStream_t s) {
  if (f32) {
    if (p.N <= 32) return delta_f32_32(p, which, s);
    if (p.N <= 64) return delta_f32_64(p, which, s);
    return delta_f32_128(p, which, s);
  }
  if (p.N <= 32) return delta_bf16_32(p, which, s);
  if (p.N <= 64) return delta_bf16_64(p, which, s);
  if (p.N <= 128) return delta_bf16_128(p, which, s);
  return delta_bf16_256(p, which, s);
}

int grads(const DeltaGradParams& p, bool f32, hipStream_t s) {
  if (f32) {
    if (p.N <= 32) return delta_f32_32_grad(p, s);
    if (p.N <= 64) return delta_f32_64_grad(p, s);
    return delta_f32_128_grad(p, s);
  }
  if (p.N <= 32) return delta_bf16_32_grad(p, s);
  if (p.N <= 64) return delta_bf16_64_grad(p, s);
  if (p.N <= 128) return delta_bf16_128_grad(p, s);
  return delta_bf16_256_grad(p, s);
}

int carry(const DeltaParams& p, bool back, hipStream_t s) {
  if (p.N <= 32) return back ? delta_carry<1, true>(p, s) : delta_carry<1, false>(p, s);
  if (p.N <= 64) return back ? delta_carry<2, true>(p, s) : delta_carry<2, false>(p, s);
  if (p.N <= 128) return back ? delta_carry<4, true>(p, s) : delta_carry<4, false>(p, s);
  return back ? delta_carry<8, true>(p, s) : delta_carry<8, false>(p, s);
}

int padded_rows(int N) { return N <= 32 ? 32 : N <= 64 ? 64 : N <= 128 ? 128 : 256; }

constexpr size_t kTriBytes = kDeltaTri * sizeof(float);
constexpr size_t kGateBytes = kDeltaGates * sizeof(float);

// Segments of the walks.  A walk's chunks follow each other; where the independent ones leave
// CUs idle, they are cut into segments, whose transitions and ends are made first (a state
// pass over the state's columns and as many more as it has rows) and joined.  Taken is the
// number of the least time, summed up from measured ones.
struct SegPlan {
  int nseg = 1, seg_chunks = 1;
};

// Microseconds of a chunk in a workgroup's walk, with up to one workgroup per CU and where it
// shares its CU with another (traces of 16 chunks by 256 and by 512 workgroups; of fp32
// inputs and of 256 keys a CU's LDS holds one), and of a link of a join forwards and back (8
// heads of 64 columns, 32 segments).
struct WalkTimes {
  double out[2], keep[2], back[2], seg[2], seg_back[2], join[2];
};
constexpr WalkTimes kTimesBf16[4] = {
    {{4.1, 5.8}, {2.6, 4.7}, {4.9, 7.0}, {2.1, 2.9}, {4.1, 5.7}, {0.75, 0.65}},  // 32 keys
    {{4.8, 7.1}, {3.0, 6.1}, {5.4, 8.6}, {2.4, 3.5}, {4.5, 7.3}, {1.0, 0.9}},    // 64
    {{6.2, 9.6}, {4.1, 8.6}, {7.0, 12.0}, {3.2, 4.8}, {5.7, 9.0}, {2.5, 2.6}},   // 128
    {{10.0, 0}, {7.2, 0}, {11.4, 0}, {5.0, 0}, {9.5, 0}, {9.8, 54.0}}};          // 256
constexpr WalkTimes kTimesF32[3] = {
    {{5.4, 0}, {3.2, 0}, {6.0, 0}, {2.6, 0}, {5.0, 0}, {0.75, 0.65}},
    {{6.9, 0}, {4.4, 0}, {7.7, 0}, {3.4, 0}, {6.4, 0}, {1.0, 0.9}},
    {{10.1, 0}, {6.3, 0}, {11.3, 0}, {4.9, 0}, {10.2, 0}, {2.5, 2.6}}};
constexpr double kJoinBytes = 4e6;  // of transitions and states, per microsecond
constexpr double kTwoLaunches = 8;  // microseconds of the state pass and the join on their own

// A chunk's step of `wgs` workgroups, in rounds of all that the CUs hold.
double step_time(double wgs, const double (&us)[2], bool one, double cus) {
  const double round = one ? cus : 2 * cus, whole = std::floor(wgs / round);
  const double rest = wgs - whole * round, shared = one ? us[0] : us[1];
  return whole * shared + (rest <= 0 ? 0.0 : rest <= cus ? us[0] : shared);
}

// Against the best of a sweep over 1 to 128 segments (16 shapes, both ways) its choice takes 4 %
// more at most.  Whole walks, its choice and other cuts, forward: one head of 128 x 128 over
// 65536 tokens 5342, 317 (64 segments), 592 (16), 417 us (128); 8 heads of 64 x 64 over 32768
// tokens 2132, 197 (32), 264 (16), 271 (128); 40 heads of 128 x 64 over 65536 tokens 5721, 2030
// (25), 2294 (5), 2452 (128); 256 heads of 128 x 128 over 4096 tokens 702 (whole), 1028 (2);
// 8 heads of 256 x 128 over 8192 tokens 1015, 352 (11), 489 (20), and back 2084, 1357 (8),
// 2142 (20), whose joins are its longest part.
SegPlan plan_segments(const swimba_delta_rule_args* a, bool back, int dev) {
  const int64_t tiles = (a->P + kWalkCols - 1) / kWalkCols, bh = (int64_t)a->B * a->H;
  const int rows = padded_rows(a->N), size = rows <= 32 ? 0 : rows <= 64 ? 1 : rows <= 128 ? 2 : 3;
  const int64_t more = (rows + kWalkCols - 1) / kWalkCols;
  const int64_t nc = (a->L + kChunk - 1) / kChunk;
  const double cus = device_cus(dev);
  const bool f32 = a->in_dtype == SWIMBA_F32, one = f32 || rows > 128;
  const WalkTimes& us = f32 ? kTimesF32[size] : kTimesBf16[size];
  const double link = (double)(bh * tiles) * rows * (rows + 2 * kWalkCols) * sizeof(float) / kJoinBytes;
  auto time = [&](int64_t n) {
    const double w = (double)(bh * tiles * n);
    double chunk = back ? step_time(w, us.keep, one, cus) + step_time(w, us.back, one, cus)
                        : step_time(w, us.out, one, cus);
    double joins = 0;
    if (n > 1) {
      chunk += step_time((double)(bh * (tiles + more) * (back ? n : n - 1)), us.seg, one, cus);
      if (back) chunk += step_time((double)(bh * tiles * (n - 1)), us.seg_back, one, cus);
      joins = (double)(n - 1) * std::max(us.join[0], link) + kTwoLaunches;
      if (back) joins += (double)(n - 1) * std::max(us.join[1], link) + kTwoLaunches;
    }
    return (double)((nc + n - 1) / n) * chunk + joins;
  };
  SegPlan best;
  best.seg_chunks = (int)nc;
  double least = time(1);
  for (int64_t n = 2; n <= 128 && 2 * n <= nc; ++n) {
    const int64_t len = (nc + n - 1) / n;
    if ((nc + len - 1) / len != n) continue;
    const double t = time(n);
    if (t < least) {
      least = t;
      best.nseg = (int)n;
      best.seg_chunks = (int)len;
    }
  }
  return best;
}

int64_t chunks_of(const swimba_delta_rule_args* a) { return (a->L + kChunk - 1) / kChunk; }

int64_t key_elements(const swimba_delta_rule_args* a) {
  return (int64_t)a->B * a->L * a->G * a->N;
}
int64_t value_elements(const swimba_delta_rule_args* a) {
  return (int64_t)a->B * a->L * a->H * a->P;
}
// Slots for copies of operands of less than a pack.
size_t tiny_bytes(const swimba_delta_rule_args* a) {
  return key_elements(a) < kPack || value_elements(a) < kPack ? 4 * kTinySlot : 0;
}

// Workspace of a forward call: per chunk and head the inverse and the gates.
struct DeltaPlan {
  SegPlan seg;
  size_t off_tri = 0, off_gates = 0, off_tiny = 0, off_seg = 0, off_carry = 0,
         bytes = 0;
};

size_t padded_columns(const swimba_delta_rule_args* a) {
  return (size_t)(a->P + kWalkCols - 1) / kWalkCols * kWalkCols;
}
DeltaPlan plan_delta(const swimba_delta_rule_args* a, int dev) {
  DeltaPlan r;
  r.seg = plan_segments(a, false, dev);
  const size_t units = (size_t)a->B * a->H * chunks_of(a);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  r.off_tri = take(units * kTriBytes);
  r.off_gates = take(units * kGateBytes);
  r.off_tiny = take(tiny_bytes(a));
  const size_t N = padded_rows(a->N), segs = (size_t)a->B * a->H * (r.seg.nseg > 1 ? r.seg.nseg : 0);
  r.off_seg = take(segs * N * padded_columns(a) * sizeof(float));
  r.off_carry = take(segs * N * N * sizeof(float));
  r.bytes = o;
  return r;
}

// And of a backward call.
struct DeltaGradPlan {
  SegPlan seg;
  int parts = 1;
  size_t off_seg = 0, off_carry = 0;
  size_t off_tri = 0, off_tri_t = 0, off_gates = 0, off_states = 0, off_adj = 0,
         off_o = 0, off_dv = 0, off_dq = 0, off_dk = 0, off_part = 0, off_tiny = 0, bytes = 0;
};

// Workgroups of a group of heads that share q and k in the gradients' kernel: one, which adds
// their gradients up in registers, unless that leaves CUs idle.
int grad_parts(const swimba_delta_rule_args* a, int dev) {
  const int share = a->H / a->G;
  const int64_t units = (int64_t)a->B * a->G * chunks_of(a), want = 2LL * device_cus(dev);
  int n = 1;
  while (n < share && (units * n < want || share % n != 0)) ++n;
  return n;
}

DeltaGradPlan plan_delta_grad(const swimba_delta_rule_grad_args* g, int dev) {
  const swimba_delta_rule_args* a = &g->fwd;
  DeltaGradPlan r;
  r.seg = plan_segments(a, true, dev);
  const size_t units = (size_t)a->B * a->H * chunks_of(a), Pp = padded_columns(a);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  r.off_tri = take(units * kTriBytes);
  r.off_tri_t = take(units * kTriBytes);
  r.off_gates = take(units * kGateBytes);
  r.off_states = take(units * padded_rows(a->N) * Pp * sizeof(float));
  r.off_adj = take(units * padded_rows(a->N) * Pp * sizeof(float));
  r.off_o = take(units * kChunk * Pp * sizeof(float));
  r.off_dv = take(units * kChunk * Pp * sizeof(float));
  // rows of dq and dk of the parts of a group of heads
  r.parts = grad_parts(a, dev);
  const size_t rows = r.parts > 1 ? (size_t)a->B * a->L * a->G * r.parts * a->N * sizeof(float) : 0;
  r.off_dq = take(rows);
  r.off_dk = take(rows);
  r.off_part = take(a->decay_form == SWIMBA_DECAY_HEAD ? units * sizeof(double) : 0);
  r.off_tiny = take(tiny_bytes(a));
  const size_t N = padded_rows(a->N), segs = (size_t)a->B * a->H * (r.seg.nseg > 1 ? r.seg.nseg : 0);
  r.off_seg = take(segs * N * Pp * sizeof(float));
  r.off_carry = take(segs * N * N * sizeof(float));
  r.bytes = o;
  return r;
}

DeltaParams base_params(const swimba_delta_rule_args* a, const void* q, const void* k,
                        const void* v) {
  DeltaParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = a->log_decay;
  p.beta = a->beta;
  p.B = a->B;
  p.L = a->L;
  p.H = a->H;
  p.G = a->G;
  p.N = a->N;
  p.P = a->P;
  p.token_decay = a->decay_form == SWIMBA_DECAY_TOKEN;
  p.nc = (int)chunks_of(a);
  p.ctiles = (a->P + kWalkCols - 1) / kWalkCols;
  p.nseg = 1;
  p.seg_chunks = p.nc;
  p.Pp = kWalkCols * p.ctiles;
  return p;
}

// One token: u = beta (v - e^g h^T k), h' = e^g h + k u^T, y = e^g h^T q + (k . q) u.
// The state is read and written once (8 bytes per entry against 4 multiply-adds).  A
// workgroup holds `slice` columns of one head's state in registers, up to kStepRows rows of V
// columns per thread, while both sums over the rows are made: across the wave's row
// lanes, then its waves, in order.  256 sequences of 40 heads of 128 x 128 in 266 us, 5.1 TB/s
// (a copy: 5.3); one of 24 heads of 128 x 64 in 5.3 us, one launch.
struct DeltaStepParams {
  const void *q, *k, *v;
  const float *g, *beta;
  const float* state;
  float* out;
  void* y;
  int H, share, N, P, token_decay, y_bf16;
  int slices, cg_log;  // workgroups per head; log2 of the column groups
};

constexpr int kMaxRows = 256;   // N
constexpr int kStepRows = 16;

template <typename TI, int V>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepParams p) {
  __shared__ float sq[kMaxRows], sk[kMaxRows];
  __shared__ float part[4][2][32 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cgs = 1 << p.cg_log, rl = 256 >> p.cg_log;
  const int64_t bh = blockIdx.x / p.slices;
  const int cg = threadIdx.x & (cgs - 1), r0 = threadIdx.x >> p.cg_log;
  const int c = ((int)(blockIdx.x % p.slices) * cgs + cg) * V;
  const int64_t b = bh / p.H;
  const int h = (int)(bh - b * p.H);
  const bool on = c < p.P;  // V divides P where it is not one
  const float* st = p.state + bh * p.N * p.P + c;
  float* so = p.out + bh * p.N * p.P + c;

  float cur[kStepRows][V];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int n = r0 + i * rl;
#pragma unroll
    for (int j = 0; j < V; ++j) cur[i][j] = 0.f;
    if (i * rl < p.N && on && n < p.N) {
      if constexpr (V == 4) {
        const float4 f = *reinterpret_cast<const float4*>(st + (int64_t)n * p.P);
        cur[i][0] = f.x; cur[i][1] = f.y; cur[i][2] = f.z; cur[i][3] = f.w;
      } else {
        cur[i][0] = st[(int64_t)n * p.P];
      }
    }
  }
  const int64_t row = (b * (p.H / p.share) + h / p.share) * p.N;
  if ((int)threadIdx.x < p.N) {
    sq[threadIdx.x] = to_f32(static_cast<const TI*>(p.q)[row + threadIdx.x]);
    sk[threadIdx.x] = to_f32(static_cast<const TI*>(p.k)[row + threadIdx.x]);
  }
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = on ? to_f32(static_cast<const TI*>(p.v)[bh * p.P + c + j]) : 0.f;
  const float e = hw_exp2(p.g[p.token_decay ? bh : h] * kLog2e), beta = p.beta[bh];
  __syncthreads();
  float kh[V] = {}, qh[V] = {}, qk = 0.f;
  for (int n = lane; n < p.N; n += 64) qk = fmaf(sq[n], sk[n], qk);
  qk = wave_sum64(qk);
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int n = r0 + i * rl;
    if (i * rl < p.N && n < p.N) {
      const float kn = sk[n], qn = sq[n];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        kh[j] = fmaf(kn, cur[i][j], kh[j]);
        qh[j] = fmaf(qn, cur[i][j], qh[j]);
      }
    }
  }
  for (int m = cgs; m < 64; m <<= 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      kh[j] += __shfl_xor(kh[j], m);
      qh[j] += __shfl_xor(qh[j], m);
    }
  }
  if (lane < cgs) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      part[wave][0][cg * V + j] = kh[j];
      part[wave][1][cg * V + j] = qh[j];
    }
  }
  __syncthreads();
  float u[V], y[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = cg * V + j;
    const float k4 = (part[0][0][i] + part[1][0][i]) + (part[2][0][i] + part[3][0][i]);
    const float q4 = (part[0][1][i] + part[1][1][i]) + (part[2][1][i] + part[3][1][i]);
    u[j] = beta * fmaf(-e, k4, v[j]);
    y[j] = fmaf(e, q4, qk * u[j]);
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int n = r0 + i * rl;
    if (i * rl < p.N && on && n < p.N) {
      const float kn = sk[n];
#pragma unroll
      for (int j = 0; j < V; ++j) cur[i][j] = fmaf(e, cur[i][j], kn * u[j]);
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(so + (int64_t)n * p.P) =
            make_float4(cur[i][0], cur[i][1], cur[i][2], cur[i][3]);
      else
        so[(int64_t)n * p.P] = cur[i][0];
    }
  }
  if (on && r0 == 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (p.y_bf16) static_cast<bf16_t*>(p.y)[bh * p.P + c + j] = from_f32<bf16_t>(y[j]);
      else static_cast<float*>(p.y)[bh * p.P + c + j] = y[j];
    }
  }
}

}  // namespace

size_t delta_rule_bytes(const swimba_delta_rule_args* a, int dev) {
  return a->B == 0 || a->L == 0 ? 0 : plan_delta(a, dev).bytes;
}

// A walk, from the first states of its segments if it has some: the state pass `pass`, the
// join and the walk.
int walk(const DeltaParams& p, bool f32, int pass, int which, bool back, hipStream_t s) {
  int rc = SWIMBA_OK;
  if (p.nseg > 1) {
    rc = phase(p, f32, pass, s);
    if (rc == SWIMBA_OK) rc = carry(p, back, s);
  }
  return rc == SWIMBA_OK ? phase(p, f32, which, s) : rc;
}

int launch_delta_rule(const swimba_delta_rule_args* a, void* ws, int dev, hipStream_t s) {
  const int64_t states = (int64_t)a->B * a->H * a->N * a->P;
  if (a->B == 0 || a->L == 0)
    return a->h_final != nullptr ? copy_or_zero(a->h0, a->h_final, states, s) : SWIMBA_OK;
  const bool f32 = a->in_dtype == SWIMBA_F32;
  const DeltaPlan r = plan_delta(a, dev);
  unsigned char* slot = at<unsigned char>(ws, r.off_tiny);
  int rc = SWIMBA_OK;
  const void* q = whole_packs(a->q, key_elements(a), f32, slot, s, &rc);
  const void* k = whole_packs(a->k, key_elements(a), f32, slot + kTinySlot, s, &rc);
  const void* v = whole_packs(a->v, value_elements(a), f32, slot + 2 * kTinySlot, s, &rc);
  DeltaParams p = base_params(a, q, k, v);
  p.tri = at<float>(ws, r.off_tri);
  p.gates = at<float>(ws, r.off_gates);
  p.out = a->y;
  p.out_bf16 = a->y_dtype == SWIMBA_BF16;
  p.s0 = a->h0;
  p.s_final = a->h_final;
  p.nseg = r.seg.nseg;
  p.state_segs = p.nseg - 1;  // the last one's end is not carried on
  p.seg_chunks = r.seg.seg_chunks;
  p.seg_state = at<float>(ws, r.off_seg);
  p.seg_carry = at<float>(ws, r.off_carry);
  if (rc == SWIMBA_OK) rc = phase(p, f32, kPhasePrep, s);
  if (rc == SWIMBA_OK)
    rc = walk(p, f32, kPhaseSeg, kPhaseOut, false, s);
  return rc;
}

size_t delta_rule_backward_bytes(const swimba_delta_rule_grad_args* g, int dev) {
  return g->fwd.B == 0 || g->fwd.L == 0 ? 0 : plan_delta_grad(g, dev).bytes;
}

int launch_delta_rule_backward(const swimba_delta_rule_grad_args* g, void* ws, int dev,
                               hipStream_t s) {
  const swimba_delta_rule_args* a = &g->fwd;
  const int64_t states = (int64_t)a->B * a->H * a->N * a->P;
  if (a->B == 0 || a->L == 0) {
    int rc = SWIMBA_OK;
    if (g->dh0 != nullptr) rc = copy_or_zero(g->dh_final, g->dh0, states, s);
    if (rc == SWIMBA_OK && a->decay_form == SWIMBA_DECAY_HEAD)
      rc = copy_or_zero(nullptr, g->dlog_decay, a->H, s);
    return rc;
  }
  const bool f32 = a->in_dtype == SWIMBA_F32;
  const DeltaGradPlan r = plan_delta_grad(g, dev);
  unsigned char* slot = at<unsigned char>(ws, r.off_tiny);
  int rc = SWIMBA_OK;
  const bool shared = r.parts > 1;
  const void* q = whole_packs(a->q, key_elements(a), f32, slot, s, &rc);
  const void* k = whole_packs(a->k, key_elements(a), f32, slot + kTinySlot, s, &rc);
  const void* v = whole_packs(a->v, value_elements(a), f32, slot + 2 * kTinySlot, s, &rc);
  DeltaParams p = base_params(a, q, k, v);
  p.dy = whole_packs(g->dy, value_elements(a), f32, slot + 3 * kTinySlot, s, &rc);
  p.tri = at<float>(ws, r.off_tri);
  p.tri_t = at<float>(ws, r.off_tri_t);
  p.gates = at<float>(ws, r.off_gates);
  p.out = g->dv;
  p.out_bf16 = g->grad_dtype == SWIMBA_BF16;
  p.s0 = a->h0;
  p.states = at<float>(ws, r.off_states);
  p.rows = at<float>(ws, r.off_o);
  p.nseg = r.seg.nseg;
  p.seg_chunks = r.seg.seg_chunks;
  p.seg_state = at<float>(ws, r.off_seg);
  p.seg_carry = at<float>(ws, r.off_carry);
  p.state_segs = p.nseg;  // walking back, the last one's transition is the first to be passed
  if (rc == SWIMBA_OK) rc = phase(p, f32, kPhasePrepBack, s);
  if (rc == SWIMBA_OK) rc = walk(p, f32, kPhaseSeg, kPhaseKeep, false, s);
  p.s0 = g->dh_final;
  p.s_final = g->dh0;
  p.states = at<float>(ws, r.off_adj);
  p.rows = at<float>(ws, r.off_dv);
  p.state_segs = p.nseg - 1;
  if (rc == SWIMBA_OK) rc = walk(p, f32, kPhaseSegBack, kPhaseBack, true, s);
  if (rc != SWIMBA_OK) return rc;

  DeltaGradParams d = {};
  d.q = q;
  d.k = k;
  d.dy = p.dy;
  d.g = a->log_decay;
  d.beta = a->beta;
  d.B = a->B;
  d.L = a->L;
  d.H = a->H;
  d.G = a->G;
  d.N = a->N;
  d.P = a->P;
  d.Pp = p.Pp;
  d.token_decay = p.token_decay;
  d.nc = p.nc;
  d.parts = r.parts;
  d.heads = a->H / a->G / r.parts;
  d.gates = p.gates;
  d.states = at<float>(ws, r.off_states);
  d.adjoints = at<float>(ws, r.off_adj);
  d.o = at<float>(ws, r.off_o);
  d.dv = at<float>(ws, r.off_dv);
  d.dq = shared ? at<void>(ws, r.off_dq) : g->dq;
  d.dk = shared ? at<void>(ws, r.off_dk) : g->dk;
  d.grad_bf16 = !shared && g->grad_dtype == SWIMBA_BF16;
  d.dg = p.token_decay ? g->dlog_decay : nullptr;
  d.part = p.token_decay ? nullptr : at<double>(ws, r.off_part);
  d.dbeta = g->dbeta;
  rc = grads(d, f32, s);
  if (rc == SWIMBA_OK && shared) {
    const int64_t rows = (int64_t)a->B * a->L * a->G;
    rc = sum_shared_heads(at<float>(ws, r.off_dq), g->dq, g->grad_dtype, rows, r.parts, a->N, s);
    if (rc == SWIMBA_OK)
      rc = sum_shared_heads(at<float>(ws, r.off_dk), g->dk, g->grad_dtype, rows, r.parts, a->N, s);
  }
  if (rc == SWIMBA_OK && d.part != nullptr)
    rc = sum_decay_parts(d.part, g->dlog_decay, a->B, a->H, p.nc, s);
  return rc;
}

int launch_delta_rule_step(const swimba_delta_rule_step_args* a, int dev, hipStream_t s) {
  DeltaStepParams p;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.g = a->log_decay;
  p.beta = a->beta;
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
  // Column groups per workgroup: up to 32 of four columns (16 of one) whose rows fit
  // the registers; fewer where the heads alone do not give two workgroups per CU.
  int cg_log = vec ? 5 : 4;
  const int V = vec ? 4 : 1;
  while (cg_log > 2 && a->N > (256 >> cg_log) * kStepRows) --cg_log;
  while (cg_log > 2 && (V << (cg_log - 1)) >= a->P) --cg_log;
  const int64_t heads = (int64_t)a->B * a->H, target = 2LL * device_cus(dev);
  auto slices = [&](int l) { return ((int64_t)a->P + (V << l) - 1) / (V << l); };
  while (cg_log > 2 && heads * slices(cg_log) < target) --cg_log;
  p.cg_log = cg_log;
  p.slices = (int)slices(cg_log);
  const dim3 g((unsigned)(heads * p.slices)), t(256);
  const bool bf = a->in_dtype == SWIMBA_BF16;
  if (vec && bf) hipLaunchKernelGGL((delta_step_kernel<bf16_t, 4>), g, t, 0, s, p);
  else if (vec) hipLaunchKernelGGL((delta_step_kernel<float, 4>), g, t, 0, s, p);
  else if (bf) hipLaunchKernelGGL((delta_step_kernel<bf16_t, 1>), g, t, 0, s, p);
  else hipLaunchKernelGGL((delta_step_kernel<float, 1>), g, t, 0, s, p);
  return checked();
}

}  // namespace swimba
