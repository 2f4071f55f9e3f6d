// Linear attention with a decay per head, in chunks on the matrix units.
//
// One kernel serves the forward pass and every gradient.  For row operands
// q_t, k_t (size Kd), values v_t (size Cd) and log decays g_t it computes
//   h_t = e^{g_t} h_{t-1} + k_t v_t^T,   y_t = h_t^T q_t
// 64 tokens at a time.  With G_t the running sum of g inside the chunk,
// D[t][s] = e^{G_t - G_s} for s <= t, w_s = e^{G_end - G_s}:
//   y     = e^{G_t} (Q h)_t + ((Q K^T) * D) V
//   h'    = e^{G_end} h + K^T (w * V)
// The gradients are the same computation with the operands' places changed:
//   dq = (q: dY, k: V, v: K),  and walking the tokens backwards, with every
//   decay taken from the token after,  dk = (V, dY, Q),  dv = (K, Q, dY).
//
// Mapping.  A wave owns 32 columns of the state (its 32 x 32 accumulator tiles
// hold h[n][c] in fp32 for the whole walk); a workgroup's waves share the
// staged Q and K rows and the scores Q K^T, which they compute once and keep
// in LDS in fp32; each wave applies its own head's decays.  The accumulator
// layout of h is, register for register, the layout of the other operand of
// Q h when the sum over n runs in the order n = 4 half + j, 8 + 4 half + j, so
// the state never passes through LDS; Q is read in that order.  The decay of a
// token enters on the value side (w * V), which a wave reads for itself, so
// that K stays as it came.
//
// Roundings.  bf16 inputs multiply exactly.  What is computed in fp32 and
// enters a product (decayed scores, state, decayed values) is split into two
// or three bf16 terms that sum to it within 2^-16 or 2^-24 of its size, two
// where the result is rounded to bf16 anyway, three where it is kept in fp32:
// a single bf16 term would leave 2^-9, as much as the output's own rounding,
// and in the state it would stay for the rest of the sequence.  fp32 inputs go
// through the fp32 matrix instruction.  Sums of log decays are taken in 64
// bits and handed on as a high and a low fp32 part: differences of large sums
// would lose the small decays after a document boundary.
#pragma once
#include "pack.hpp"
#include "swimba_internal.hpp"

namespace swimba {

constexpr int kChunk = 64;
constexpr float kLeastLog2 = -300.f;  // e^g is zero in fp32 long before
constexpr int kScoreStride = kChunk + 4;

struct AttnParams {
  const void *q, *k, *v;
  void* y;
  const float* g;         // [H] or [B, L, H]
  int B, L, H;
  int qshare, vshare;     // heads per q/k head and per v head
  int Kd, Cd;
  int token_decay, reverse, y_bf16;
  const float* s0;        // first state or null; entry (n, c) at n * sk + c * sc
  float* s_final;         // or null; the same layout
  int64_t sk, sc;
  int nseg, seg_chunks;   // segments of the walk, chunks in each
  float* seg_state;       // [B, H, nseg, Kd, Cd]: end states out (state pass), first states in
  float* seg_decay;       // [B, H, nseg] out of the state pass
  const void* z;          // null, or rows (B, L, H / vshare, Cd) for the sums below
  float* zsum;            // [B, H, ctiles, 2, L]: <z_t, y_t> inside the chunk, and from the state
  int ctiles;             // ceil(Cd / 32)
};

typedef float f16x __attribute__((ext_vector_type(16)));
typedef __bf16 bf8x __attribute__((ext_vector_type(8)));
typedef short s4x __attribute__((ext_vector_type(4)));

struct Bits8 {
  uint32_t w[4];
};

// Two fp32 values as bf16 in one register, the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return (uint32_t)from_f32<bf16_t>(a) | ((uint32_t)from_f32<bf16_t>(b) << 16);
}
__device__ __forceinline__ float low_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x (8 values) as S bf16 terms.
template <int S>
__device__ __forceinline__ void split_terms(const float* x, bf8x* out) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    Bits8 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = bf16_pair(r[2 * i], r[2 * i + 1]);
    out[s] = __builtin_bit_cast(bf8x, b);
    if (s + 1 < S) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[2 * i] -= low_f32(b.w[i]);
        r[2 * i + 1] -= high_f32(b.w[i]);
      }
    }
  }
}

__device__ __forceinline__ f16x mma(bf8x a, bf8x b, f16x c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x mma(float a, float b, f16x c) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

// Eight rows (half the lanes four each, twice) of one column from a row-major
// LDS tile: the transposing read hands lane i of 16 the column i of a block of
// 4 rows x 16 columns of which it points at row i / 4, columns 4 (i % 4)..
__device__ __forceinline__ bf8x column8(const bf16_t* tile, int stride, int row, int col, int lane) {
  typedef __attribute__((address_space(3))) s4x* lds_s4;
  const bf16_t* p = tile + (row + 8 * (lane >> 5) + ((lane & 15) >> 2)) * stride + col +
                    16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  struct { s4x a, b; } r;
  r.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p));
  r.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + 4 * stride));
  return __builtin_bit_cast(bf8x, r);
}

template <typename TI, int KT, int W>
struct AttnShape {
  static constexpr bool kF32 = sizeof(TI) == 4;
  static constexpr int kRows = 32 * KT;                      // padded Kd
  static constexpr int kRowStride = kRows + (kF32 ? 4 : 16);  // banks of rows apart
  static constexpr int kValStride = 32 + (kF32 ? 4 : 16);
  static constexpr size_t kBytes =
      (size_t)(2 * kChunk * kRowStride + W * kChunk * kValStride) * sizeof(TI) +
      (size_t)(kChunk * kScoreStride + W * 4 * kChunk) * sizeof(float);
};

// Rows of `base` (row r at token(r) * stride) into LDS, zero beyond `len` rows
// and `cols` columns.  PAD columns are written.
template <typename TI, int PAD, int THREADS, typename F>
__device__ __forceinline__ void stage_rows(const TI* base, int64_t stride, int cols, int len,
                                           TI* dst, int dst_stride, int tid, F token) {
  constexpr int kPer = PAD / kPack;
#pragma unroll
  for (int i = 0; i < kChunk * kPer / THREADS; ++i) {
    const int u = i * THREADS + tid;
    const int r = u / kPer, c = (u % kPer) * kPack;
    Pack<TI> v = {};
    if (r < len && c < cols) v = load_pack(base + token(r) * stride + c, cols - c);
    *reinterpret_cast<Pack<TI>*>(dst + r * dst_stride + c) = v;
  }
}

// Sums of 16 registers, each over the 32 lanes of its half: lane l of a half
// returns that of register (l >> 1).
__device__ __forceinline__ float half_sums(const float* v, int lane) {
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 8] : v[i]) + xor_lane<16>(up ? v[i] : v[i + 8], lane);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 4] : a[i]) + xor_lane<8>(up ? a[i] : a[i + 4], lane);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 4;
    c[i] = (up ? b[i + 2] : b[i]) + xor_lane<4>(up ? b[i] : b[i + 2], lane);
  }
  const bool up = lane & 2;
  float s = (up ? c[1] : c[0]) + xor_lane<2>(up ? c[0] : c[1], lane);
  return s + xor_lane<1>(s, lane);
}

// S: bf16 terms of what is computed (2 or 3); STATE: only the segment's end
// state from zero and its decay.
template <typename TI, int KT, int W, int S, bool STATE>
__global__ __launch_bounds__(64 * W, KT > 4 ? 1 : 2) void attn_kernel(AttnParams p) {
  using Sh = AttnShape<TI, KT, W>;
  constexpr bool kF32 = Sh::kF32;
  constexpr int RS = Sh::kRowStride, VS = Sh::kValStride;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
  TI* sQ = reinterpret_cast<TI*>(smem_raw);
  TI* sK = sQ + kChunk * RS;
  TI* sVall = sK + kChunk * RS;
  float* sS = reinterpret_cast<float*>(sVall + W * kChunk * VS);
  float* sGall = sS + kChunk * kScoreStride;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int half = lane >> 5, col = lane & 31;
  TI* sV = sVall + wave * kChunk * VS;
  float* gHi = sGall + wave * 4 * kChunk;  // high and low parts of G, e^G, w
  float *gLo = gHi + kChunk, *gE = gLo + kChunk, *gW = gE + kChunk;

  // workgroup -> (sequence, group of heads sharing q and k, segment, W units)
  const int groups = p.H / p.qshare, units = p.qshare * p.ctiles, nu = (units + W - 1) / W;
  int blk = blockIdx.x;
  const int u = (blk % nu) * W + wave;
  blk /= nu;
  const int segs = STATE ? p.nseg - 1 : p.nseg;  // the last one's end state is not carried
  const int seg = blk % segs;
  blk /= segs;
  const int grp = blk % groups, b = blk / groups;
  const bool active = u < units;
  const int head = grp * p.qshare + (active ? u / p.ctiles : 0);
  const int c0 = active ? (u % p.ctiles) * 32 : 0;
  const int cols = active ? p.Cd - c0 : 0;  // columns of this wave inside the state

  const int hv = p.H / p.vshare;
  const int64_t qstride = (int64_t)groups * p.Kd, vstride = (int64_t)hv * p.Cd;
  const TI* qb = static_cast<const TI*>(p.q) + (int64_t)b * p.L * qstride + (int64_t)grp * p.Kd;
  const TI* kb = static_cast<const TI*>(p.k) + (int64_t)b * p.L * qstride + (int64_t)grp * p.Kd;
  const TI* vb = static_cast<const TI*>(p.v) + (int64_t)b * p.L * vstride +
                 (int64_t)(head / p.vshare) * p.Cd + c0;
  const float* gb = p.g + (p.token_decay ? (int64_t)b * p.L * p.H : 0) + head;
  const int64_t state = ((int64_t)b * p.H + head) * p.Kd * p.Cd;
  const int64_t sstate = (((int64_t)b * p.H + head) * p.nseg + seg) * p.Kd * p.Cd;

  f16x h[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = 32 * kt + 8 * (i >> 2) + 4 * half + (i & 3);
      float v = 0.f;
      if (!STATE && n < p.Kd && col < cols) {
        if (p.nseg > 1) v = p.seg_state[sstate + (int64_t)n * p.Cd + c0 + col];
        else if (p.s0 != nullptr) v = p.s0[state + n * p.sk + (c0 + col) * p.sc];
      }
      h[kt][i] = v;
    }
  double whole = 0.0;  // log2 decay of the segment so far (state pass)

  const int nc = (p.L + kChunk - 1) / kChunk;
  const int j1 = (seg + 1) * p.seg_chunks < nc ? (seg + 1) * p.seg_chunks : nc;
  for (int j = seg * p.seg_chunks; j < j1; ++j) {
    const int t0 = (p.reverse ? nc - 1 - j : j) * kChunk;
    const int len = p.L - t0 < kChunk ? p.L - t0 : kChunk;
    auto token = [&](int r) { return (int64_t)(p.reverse ? t0 + len - 1 - r : t0 + r); };
    __syncthreads();
    if (!STATE) stage_rows<TI, 32 * KT, 64 * W>(qb, qstride, p.Kd, len, sQ, RS, tid, token);
    stage_rows<TI, 32 * KT, 64 * W>(kb, qstride, p.Kd, len, sK, RS, tid, token);
    stage_rows<TI, 32, 64>(vb, vstride, cols, len, sV, VS, lane, token);
    double end;
    {
      // log2 decays, summed over the lanes
      double g = 0.0;
      if (lane < len) {
        float v;
        if (!p.token_decay) {
          v = p.reverse && token(lane) + 1 >= p.L ? 0.f : gb[0];
        } else {
          const int64_t t = token(lane) + (p.reverse ? 1 : 0);
          v = t < p.L ? gb[t * p.H] : 0.f;
        }
        const double d = (double)v * 1.4426950408889634;
        g = d < (double)kLeastLog2 ? (double)kLeastLog2 : d;
      }
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(g, m);
        if (lane >= m) g += o;
      }
      end = __shfl(g, 63);
      const float hi = (float)g;
      gHi[lane] = hi;
      gLo[lane] = (float)(g - (double)hi);
      gE[lane] = hw_exp2(hi);
      gW[lane] = hw_exp2((float)(end - g));
    }
    __syncthreads();

    if (!STATE) {
      // scores Q K^T: the three 32 x 32 tiles on and below the diagonal
      for (int tile = wave; tile < 3; tile += W) {
        const int tt = tile > 0, ss = tile > 1;
        f16x a;
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = 0.f;
        const TI* qr = sQ + (32 * tt + col) * RS;
        const TI* kr = sK + (32 * ss + col) * RS;
        if constexpr (kF32) {
#pragma unroll 4
          for (int n = 0; n < 32 * KT; n += 8) {
            const float4 x = *reinterpret_cast<const float4*>(qr + n + 4 * half);
            const float4 y = *reinterpret_cast<const float4*>(kr + n + 4 * half);
            a = mma(x.x, y.x, a);
            a = mma(x.y, y.y, a);
            a = mma(x.z, y.z, a);
            a = mma(x.w, y.w, a);
          }
        } else {
#pragma unroll
          for (int n = 0; n < 32 * KT; n += 16)
            a = mma(*reinterpret_cast<const bf8x*>(qr + n + 8 * half),
                    *reinterpret_cast<const bf8x*>(kr + n + 8 * half), a);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sS[(32 * tt + 8 * (i >> 2) + 4 * half + (i & 3)) * kScoreStride + 32 * ss + col] = a[i];
      }
      __syncthreads();
    }

    const float carry = hw_exp2((float)end);
    f16x y[2];
    if (!STATE) {
      // from the state: e^{G_t} (Q h)_t
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) y[tt][i] = 0.f;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        if constexpr (kF32) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
              const float4 x = *reinterpret_cast<const float4*>(sQ + (32 * tt + col) * RS + 32 * kt +
                                                                8 * a + 4 * half);
              y[tt] = mma(x.x, h[kt][4 * a], y[tt]);
              y[tt] = mma(x.y, h[kt][4 * a + 1], y[tt]);
              y[tt] = mma(x.z, h[kt][4 * a + 2], y[tt]);
              y[tt] = mma(x.w, h[kt][4 * a + 3], y[tt]);
            }
        } else {
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = h[kt][8 * k2 + i];
            bf8x t[S];
            split_terms<S>(x, t);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
              const TI* r = sQ + (32 * tt + col) * RS + 32 * kt + 16 * k2 + 4 * half;
              struct { uint2 a, b; } qa;
              qa.a = *reinterpret_cast<const uint2*>(r);
              qa.b = *reinterpret_cast<const uint2*>(r + 8);
              const bf8x a = __builtin_bit_cast(bf8x, qa);
#pragma unroll
              for (int s = S - 1; s >= 0; --s) y[tt] = mma(a, t[s], y[tt]);
            }
          }
        }
      }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const float4 e = *reinterpret_cast<const float4*>(gE + 32 * tt + 8 * a + 4 * half);
          y[tt][4 * a] *= e.x;
          y[tt][4 * a + 1] *= e.y;
          y[tt][4 * a + 2] *= e.z;
          y[tt][4 * a + 3] *= e.w;
        }
    }
    f16x zv[2];
    float zstate[2] = {0.f, 0.f};
    if (!STATE && S == 3 && p.z != nullptr) {
      const TI* zb = static_cast<const TI*>(p.z) + (int64_t)b * p.L * vstride +
                     (int64_t)(head / p.vshare) * p.Cd + c0;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        float m[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = 32 * tt + 8 * (i >> 2) + 4 * half + (i & 3);
          zv[tt][i] = t < len && col < cols ? to_f32(zb[token(t) * vstride + col]) : 0.f;
          m[i] = zv[tt][i] * y[tt][i];
          y[tt][i] = y[tt][i];
        }
        zstate[tt] = half_sums(m, lane);
      }
    }
    f16x ystate[2];
    if (!STATE && S == 3 && p.z != nullptr) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        ystate[tt] = y[tt];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[tt][i] = 0.f;
      }
    }

#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) h[kt][i] *= carry;

    // 8 (fp32) or 16 (bf16) tokens s at a time: y += M V, h += K^T (w V)
    constexpr int kStep = kF32 ? 8 : 16;
#pragma unroll
    for (int s0 = 0; s0 < kChunk; s0 += kStep) {
      constexpr int kV = kF32 ? 4 : 8;  // tokens per lane and step
      const int sl = s0 + kV * half;
      float vf[kV];
      bf8x vt;
      if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < kV; ++i) vf[i] = sV[(sl + i) * VS + col];
      } else {
        vt = column8(sV, VS, s0, 0, lane);
        const Bits8 bits = __builtin_bit_cast(Bits8, vt);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vf[2 * i] = low_f32(bits.w[i]);
          vf[2 * i + 1] = high_f32(bits.w[i]);
        }
      }
      if (!STATE) {
        float hs[kV], ls[kV];
#pragma unroll
        for (int i = 0; i < kV; i += 4) {
          *reinterpret_cast<float4*>(hs + i) = *reinterpret_cast<const float4*>(gHi + sl + i);
          *reinterpret_cast<float4*>(ls + i) = *reinterpret_cast<const float4*>(gLo + sl + i);
        }
#pragma unroll
        for (int tt = s0 / 32; tt < 2; ++tt) {
          const int t = 32 * tt + col;
          const float ht = gHi[t], lt = gLo[t];
          float m[kV];
#pragma unroll
          for (int i = 0; i < kV; i += 4)
            *reinterpret_cast<float4*>(m + i) =
                *reinterpret_cast<const float4*>(sS + t * kScoreStride + sl + i);
#pragma unroll
          for (int i = 0; i < kV; ++i) {
            const float d = hw_exp2((ht - hs[i]) + (lt - ls[i]));
            m[i] = (tt > s0 / 32 || sl + i <= t) ? m[i] * d : 0.f;
          }
          if constexpr (kF32) {
#pragma unroll
            for (int i = 0; i < kV; ++i) y[tt] = mma(m[i], vf[i], y[tt]);
          } else {
            bf8x mt[S];
            split_terms<S>(m, mt);
#pragma unroll
            for (int s = S - 1; s >= 0; --s) y[tt] = mma(mt[s], vt, y[tt]);
          }
        }
      }
      float ws[kV];
#pragma unroll
      for (int i = 0; i < kV; i += 4)
        *reinterpret_cast<float4*>(ws + i) = *reinterpret_cast<const float4*>(gW + sl + i);
#pragma unroll
      for (int i = 0; i < kV; ++i) vf[i] *= ws[i];
      if constexpr (kF32) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < kV; ++i) h[kt] = mma(sK[(sl + i) * RS + 32 * kt + col], vf[i], h[kt]);
      } else {
        bf8x wt[3];
        split_terms<3>(vf, wt);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const bf8x a = column8(sK, RS, s0, 32 * kt, lane);
#pragma unroll
          for (int s = 2; s >= 0; --s) h[kt] = mma(a, wt[s], h[kt]);
        }
      }
    }

    if (STATE) {
      whole += end;
      continue;
    }
    if (S == 3 && p.z != nullptr) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        float m[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i] = zv[tt][i] * y[tt][i];
        const float zin = half_sums(m, lane);
        const int i = col >> 1, t = 32 * tt + 8 * (i >> 2) + 4 * half + (i & 3);
        if (active && (lane & 1) == 0 && t < len) {
          float* zs = p.zsum + (((int64_t)b * p.H + head) * p.ctiles + u % p.ctiles) * 2 * p.L;
          zs[token(t)] = zin;
          zs[p.L + token(t)] = zstate[tt];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) y[tt][k] += ystate[tt][k];
      }
    }
    const int64_t ystride = (int64_t)p.H * p.Cd;
    const int64_t yb = (int64_t)b * p.L * ystride + (int64_t)head * p.Cd + c0 + col;
    if (col < cols) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = 32 * tt + 8 * (i >> 2) + 4 * half + (i & 3);
          if (t >= len) continue;
          const int64_t at = yb + token(t) * ystride;
          if (p.y_bf16) static_cast<bf16_t*>(p.y)[at] = from_f32<bf16_t>(y[tt][i]);
          else static_cast<float*>(p.y)[at] = y[tt][i];
        }
    }
  }

  if (STATE) {
    if (active && c0 == 0 && lane == 0)
      p.seg_decay[((int64_t)b * p.H + head) * p.nseg + seg] = hw_exp2((float)whole);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = 32 * kt + 8 * (i >> 2) + 4 * half + (i & 3);
        if (n < p.Kd && col < cols) p.seg_state[sstate + (int64_t)n * p.Cd + c0 + col] = h[kt][i];
      }
  } else if (p.s_final != nullptr && seg == p.nseg - 1) {
    // walking backwards the first token's own decay is still to come
    float f = 1.f;
    if (p.reverse) f = hw_exp2(gb[0] * kLog2e < kLeastLog2 ? kLeastLog2 : gb[0] * kLog2e);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = 32 * kt + 8 * (i >> 2) + 4 * half + (i & 3);
        if (n < p.Kd && col < cols)
          p.s_final[state + n * p.sk + (c0 + col) * p.sc] = h[kt][i] * f;
      }
  }
}

// Host side: launches one walk (or its state pass).
template <typename TI, int KT, int W, int S, bool STATE>
int attn_launch(const AttnParams& p, hipStream_t s) {
  const int groups = p.H / p.qshare, units = p.qshare * p.ctiles;
  const int64_t grid = (int64_t)p.B * groups * (STATE ? p.nseg - 1 : p.nseg) * ((units + W - 1) / W);
  if (grid > 0x7fffffff) return SWIMBA_EUNSUPPORTED;
  constexpr size_t lds = AttnShape<TI, KT, W>::kBytes;
  allow_dynamic_lds(attn_kernel<TI, KT, W, S, STATE>, lds);
  hipLaunchKernelGGL((attn_kernel<TI, KT, W, S, STATE>), dim3((unsigned)grid), dim3(64 * W), lds, s,
                     p);
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

template <typename TI, int KT, int W>
int attn_launch_kind(const AttnParams& p, bool state, bool exact, hipStream_t s) {
  if (state) return attn_launch<TI, KT, W, 3, true>(p, s);
  if constexpr (sizeof(TI) == 2)
    if (!exact) return attn_launch<TI, KT, W, 2, false>(p, s);
  return attn_launch<TI, KT, W, 3, false>(p, s);
}

template <typename TI, int KT>
int attn_launch_waves(const AttnParams& p, int waves, bool state, bool exact, hipStream_t s) {
  // fp32 rows of 256 leave LDS for one wave's values
  constexpr bool kNarrow = sizeof(TI) == 4 && KT == 8;
  if constexpr (!kNarrow) {
    if (waves == 4) return attn_launch_kind<TI, KT, 4>(p, state, exact, s);
    if (waves == 2) return attn_launch_kind<TI, KT, 2>(p, state, exact, s);
  }
  return attn_launch_kind<TI, KT, 1>(p, state, exact, s);
}

// One per dtype and padded row size.
#define SWIMBA_ATTN_DECL(name) \
  int name(const AttnParams& p, int waves, bool state, bool exact, hipStream_t s);
SWIMBA_ATTN_DECL(attn_bf16_32)
SWIMBA_ATTN_DECL(attn_bf16_64)
SWIMBA_ATTN_DECL(attn_bf16_128)
SWIMBA_ATTN_DECL(attn_bf16_256)
SWIMBA_ATTN_DECL(attn_f32_32)
SWIMBA_ATTN_DECL(attn_f32_64)
SWIMBA_ATTN_DECL(attn_f32_128)
SWIMBA_ATTN_DECL(attn_f32_256)
#undef SWIMBA_ATTN_DECL

}  // namespace swimba
