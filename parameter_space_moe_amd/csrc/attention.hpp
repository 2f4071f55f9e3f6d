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
#include <type_traits>

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
  static constexpr int kRows = 32 * KT;  // padded Kd
  // Row strides that keep the reads of 16 lanes on different banks: Q is read
  // along its rows (16 rows at once, 4 banks apart), K mostly by the transposing
  // read (4 rows of 32 bytes at once, 8 banks apart), like V.
  static constexpr int kQStride = kRows + (kF32 ? 4 : 8);
  static constexpr int kKStride = kRows + (kF32 ? 4 : 16);
  static constexpr int kValStride = 32 + (kF32 ? 4 : 16);
  static constexpr size_t kBytes =
      (size_t)(kChunk * (kQStride + kKStride) + W * kChunk * kValStride) * sizeof(TI) +
      (size_t)(kChunk * kScoreStride + W * 4 * kChunk) * sizeof(float);
};

// The pack at element e of a tensor of `total` (at least 8) elements, with the
// elements from n on zero.  Always one whole-pack load inside the tensor, so
// that a run of them is issued without branches between.
template <typename T>
__device__ __forceinline__ Pack<T> pack_inside(const T* base, int64_t e, int64_t total, int n) {
  const int64_t at = e + kPack <= total ? e : total - kPack;
  Pack<T> r = load_pack(base + at, kPack);
  const int shift = (int)(e - at);
  if (__ballot(shift != 0 && n > 0)) {  // the tensor's last elements
    Pack<T> m;
#pragma unroll
    for (int i = 0; i < kPack; ++i) {
      m.v[i] = r.v[i];
#pragma unroll
      for (int j = i + 1; j < kPack; ++j) m.v[i] = shift == j - i ? r.v[j] : m.v[i];
    }
    r = m;
  }
#pragma unroll
  for (int i = 0; i < kPack; ++i) r.v[i] = i < n ? r.v[i] : T(0);
  return r;
}

// Rows of one operand of a chunk, ROUND packs per thread at a time on their way
// to LDS: load() issues the loads of round i without branches between them,
// store() writes them (zero beyond `len` rows and `cols` columns).
template <typename T, int PAD, int THREADS>
struct RowStage {
  static constexpr int kPer = PAD / kPack, kN = kChunk * kPer / THREADS;
  static constexpr int kRound = kN < 8 ? kN : 8, kRounds = kN / kRound;
  const T* base;
  int64_t first, total, stride;  // element of row 0, column 0; elements in all; between rows
  int cols, len, tid;
  bool whole, down;              // rows of whole packs; tokens in falling order
  int64_t t0;                    // token of row 0
  Pack<T> v[kRound];

  __device__ __forceinline__ int64_t at(int r, int c) const {
    return first + (down ? t0 - r : t0 + r) * stride + c;
  }

  __device__ __forceinline__ void load(int round) {
    if (whole) {
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int u = (round * kRound + i) * THREADS + tid, r = u / kPer, c = (u % kPer) * kPack;
        const bool in = r < len && c < cols;
        v[i] = load_pack(base + (in ? at(r, c) : 0), kPack);
      }
    } else if (total >= kPack) {
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int u = (round * kRound + i) * THREADS + tid, r = u / kPer, c = (u % kPer) * kPack;
        const bool in = r < len && c < cols;
        v[i] = pack_inside(base, in ? at(r, c) : 0, total, in ? cols - c : 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int u = (round * kRound + i) * THREADS + tid, r = u / kPer, c = (u % kPer) * kPack;
        v[i] = Pack<T>{};
        if (r < len && c < cols) v[i] = load_pack(base + at(r, c), cols - c);
      }
    }
  }

  __device__ __forceinline__ void store(int round, T* dst, int dst_stride) const {
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      const int u = (round * kRound + i) * THREADS + tid, r = u / kPer, c = (u % kPer) * kPack;
      const bool in = r < len && c < cols;
      Pack<T> p;
#pragma unroll
      for (int k = 0; k < kPack; ++k) p.v[k] = in ? v[i].v[k] : T(0);
      *reinterpret_cast<Pack<T>*>(dst + r * dst_stride + c) = p;
    }
  }
};

// Inclusive sum over the lanes, in 64 bits, on the DPP row shifts and row
// broadcasts (no LDS round trips: the chunk's decays are waited for).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return v + __longlong_as_double(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_prefix(double v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __longlong_as_double(((uint64_t)hi << 32) | lo);
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

// Row of register i of a 32 x 32 accumulator tile.
__device__ __forceinline__ int tile_row(int i, int half) {
  return 8 * (i >> 2) + 4 * half + (i & 3);
}

enum AttnMode {
  kAttnState = 0,  // only the segment's end state from zero, and its decay
  kAttnPlain = 1,
  kAttnSums = 2    // also the sums of z with the results (the gradient of the decays)
};

// S: bf16 terms of what is computed (2 or 3).
template <typename TI, int KT, int W, int S, int MODE>
__global__ __launch_bounds__(64 * W, KT > 4 ? 1 : 2) void attn_kernel(AttnParams p) {
  using Sh = AttnShape<TI, KT, W>;
  constexpr bool kF32 = Sh::kF32, STATE = MODE == kAttnState, SUMS = MODE == kAttnSums;
  constexpr int QS = Sh::kQStride, KS = Sh::kKStride, VS = Sh::kValStride;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
  TI* sQ = reinterpret_cast<TI*>(smem_raw);
  TI* sK = sQ + kChunk * QS;
  TI* sVall = sK + kChunk * KS;
  float* sS = reinterpret_cast<float*>(sVall + W * kChunk * VS);
  float* sGall = sS + kChunk * kScoreStride;

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  TI* sV = sVall + wave * kChunk * VS;
  float* gHi = sGall + wave * 4 * kChunk;  // high and low parts of G, e^G, w
  float *gLo = gHi + kChunk, *gE = gLo + kChunk, *gW = gE + kChunk;

  // workgroup -> (sequence, group of heads sharing q and k, segment, W units),
  // neighbours (which read the same q and k) on one XCD: workgroups go to the
  // eight of them in turn
  const int groups = p.H / p.qshare, units = p.qshare * p.ctiles, nu = (units + W - 1) / W;
  int blk = blockIdx.x;
  {
    const int n = gridDim.x, x = blk & 7, per = n >> 3, more = n & 7;
    blk = x * per + (x < more ? x : more) + (blk >> 3);
  }
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
  const int64_t qtotal = (int64_t)p.B * p.L * qstride, vtotal = (int64_t)p.B * p.L * vstride;
  const int64_t qfirst = (int64_t)b * p.L * qstride + (int64_t)grp * p.Kd;
  const int64_t vfirst = (int64_t)b * p.L * vstride + (int64_t)(head / p.vshare) * p.Cd + c0;
  const bool qwhole = p.Kd % kPack == 0, vwhole = p.Cd % kPack == 0;
  const float* gb = p.g + (p.token_decay ? (int64_t)b * p.L * p.H : 0) + head;
  const int64_t state = ((int64_t)b * p.H + head) * p.Kd * p.Cd;
  const int64_t sstate = (((int64_t)b * p.H + head) * p.nseg + seg) * p.Kd * p.Cd;

  f16x h[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = 32 * kt + tile_row(i, half);
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
    double end;
    const int64_t first = p.reverse ? t0 + len - 1 : t0;
    {
      float g = 0.f;
      if (!p.token_decay) {
        g = lane < len && !(p.reverse && token(lane) + 1 >= p.L) ? gb[0] : 0.f;
      } else {
        const int64_t t = token(lane) + (p.reverse ? 1 : 0);
        const bool in = lane < len && t < p.L;
        g = gb[in ? t * p.H : 0];
        if (!in) g = 0.f;
      }
      using Rows = RowStage<TI, 32 * KT, 64 * W>;
      Rows rk = {static_cast<const TI*>(p.k), qfirst, qtotal, qstride, p.Kd, len, tid, qwhole,
                 (bool)p.reverse, first};
      RowStage<TI, 32, 64> rv = {static_cast<const TI*>(p.v), vfirst, vtotal, vstride, cols, len,
                                 lane, vwhole, (bool)p.reverse, first};
      Rows rq = rk;
      rq.base = static_cast<const TI*>(p.q);
      rv.load(0);
      rk.load(0);
      // four waves or more have all of a chunk in flight at once, fewer go by rounds
      if (!STATE && W == 4 && Rows::kRounds == 1) rq.load(0);

      // log2 decays, summed over the lanes
      const double d = (double)g * 1.4426950408889634;
      const double sum = wave_prefix(d < (double)kLeastLog2 ? (double)kLeastLog2 : d);
      end = last_lane(sum);
      const float hi = (float)sum;
      __syncthreads();  // everyone is done with the last chunk
      gHi[lane] = hi;
      gLo[lane] = (float)(sum - (double)hi);
      gE[lane] = hw_exp2(hi);
      gW[lane] = hw_exp2((float)(end - sum));
      rv.store(0, sV, VS);
      rk.store(0, sK, KS);
#pragma unroll
      for (int r = 1; r < Rows::kRounds; ++r) {
        rk.load(r);
        rk.store(r, sK, KS);
      }
      if (!STATE) {
#pragma unroll
        for (int r = 0; r < Rows::kRounds; ++r) {
          if (!(W == 4 && Rows::kRounds == 1)) rq.load(r);
          rq.store(r, sQ, QS);
        }
      }
    }
    __syncthreads();

    if (!STATE) {
      // scores Q K^T: the three 32 x 32 tiles on and below the diagonal
      for (int tile = wave; tile < 3; tile += W) {
        const int tt = tile > 0, ss = tile > 1;
        f16x a;
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = 0.f;
        const TI* qr = sQ + (32 * tt + col) * QS;
        const TI* kr = sK + (32 * ss + col) * KS;
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
          sS[(32 * tt + tile_row(i, half)) * kScoreStride + 32 * ss + col] = a[i];
      }
      __syncthreads();
    }

    const float carry = hw_exp2((float)end);
    f16x ys[2];  // from the state: e^{G_t} (Q h)_t
    f16x yi[2];  // from the chunk (SUMS: apart, and without the diagonal)
    f16x(&y)[2] = SUMS ? yi : ys;
    if (!STATE) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          ys[tt][i] = 0.f;
          yi[tt][i] = 0.f;
        }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        if constexpr (kF32) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
              const float4 x = *reinterpret_cast<const float4*>(sQ + (32 * tt + col) * QS + 32 * kt +
                                                                8 * a + 4 * half);
              ys[tt] = mma(x.x, h[kt][4 * a], ys[tt]);
              ys[tt] = mma(x.y, h[kt][4 * a + 1], ys[tt]);
              ys[tt] = mma(x.z, h[kt][4 * a + 2], ys[tt]);
              ys[tt] = mma(x.w, h[kt][4 * a + 3], ys[tt]);
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
              const TI* r = sQ + (32 * tt + col) * QS + 32 * kt + 16 * k2 + 4 * half;
              struct { uint2 a, b; } qa;
              qa.a = *reinterpret_cast<const uint2*>(r);
              qa.b = *reinterpret_cast<const uint2*>(r + 8);
              const bf8x a = __builtin_bit_cast(bf8x, qa);
#pragma unroll
              for (int s = S - 1; s >= 0; --s) ys[tt] = mma(a, t[s], ys[tt]);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // keep the operands of few steps in registers
      }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const float4 e = *reinterpret_cast<const float4*>(gE + 32 * tt + 8 * a + 4 * half);
          ys[tt][4 * a] *= e.x;
          ys[tt][4 * a + 1] *= e.y;
          ys[tt][4 * a + 2] *= e.z;
          ys[tt][4 * a + 3] *= e.w;
        }
    }

#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) h[kt][i] *= carry;

    // 8 (fp32) or 16 (bf16) tokens s at a time: y += M V, h += K^T (w V)
    constexpr int kStep = kF32 ? 8 : 16;
#pragma unroll 1
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
        for (int tt = 0; tt < 2; ++tt) {
          if (32 * tt + 31 < s0) continue;
          const int t = 32 * tt + col;
          const float ht = gHi[t], lt = gLo[t];
          float m[kV];
#pragma unroll
          for (int i = 0; i < kV; i += 4)
            *reinterpret_cast<float4*>(m + i) =
                *reinterpret_cast<const float4*>(sS + t * kScoreStride + sl + i);
          const int before = SUMS ? t : t + 1;  // tokens that are read
#pragma unroll
          for (int i = 0; i < kV; ++i) {
            const float d = hw_exp2((ht - hs[i]) + (lt - ls[i]));
            m[i] = sl + i < before ? m[i] * d : 0.f;
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
          for (int i = 0; i < kV; ++i) h[kt] = mma(sK[(sl + i) * KS + 32 * kt + col], vf[i], h[kt]);
      } else {
        bf8x wt[3];
        split_terms<3>(vf, wt);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const bf8x a = column8(sK, KS, s0, 32 * kt, lane);
#pragma unroll
          for (int s = 2; s >= 0; --s) h[kt] = mma(a, wt[s], h[kt]);
        }
      }
    }

    if (STATE) {
      whole += end;
      continue;
    }
    RowStage<TI, 32, 64> rz = {static_cast<const TI*>(p.z), vfirst, vtotal, vstride, cols, len,
                               lane, vwhole, (bool)p.reverse, first};
    if (SUMS) rz.load(0);
    // The wave's V slab is free row by row now: z comes in through it and the
    // results leave through it, 32 rows at a time, as whole packs.
#pragma unroll
    for (int tt = 0; tt < 2; ++tt) {
      f16x o = y[tt];
      if constexpr (SUMS) {
        float m[16], vd[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = 32 * tt + tile_row(i, half);
          vd[i] = sS[t * kScoreStride + t] * to_f32(sV[t * VS + col]);  // the diagonal
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < rz.kN / 2; ++k) {
          const int i = rz.kN / 2 * tt + k, un = i * 64 + lane;
          const int r = un / rz.kPer, c = (un % rz.kPer) * kPack;
          const bool in = r < len && c < cols;
          Pack<TI> zp;
#pragma unroll
          for (int e = 0; e < kPack; ++e) zp.v[e] = in ? rz.v[i].v[e] : TI(0);
          *reinterpret_cast<Pack<TI>*>(sV + r * VS + c) = zp;
        }
        __builtin_amdgcn_wave_barrier();
        float z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          z[i] = to_f32(sV[(32 * tt + tile_row(i, half)) * VS + col]);
          m[i] = z[i] * o[i];
        }
        const float zin = half_sums(m, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i] = z[i] * ys[tt][i];
        const float zst = half_sums(m, lane);
        const int t = 32 * tt + tile_row(col >> 1, half);
        if (active && (lane & 1) == 0 && t < len) {
          float* zs = p.zsum + (((int64_t)b * p.H + head) * p.ctiles + u % p.ctiles) * 2 * p.L;
          zs[token(t)] = zin;
          zs[p.L + token(t)] = zst;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = (o[i] + vd[i]) + ys[tt][i];
        __builtin_amdgcn_wave_barrier();
      }
      const int64_t ystride = (int64_t)p.H * p.Cd;
      const int64_t yfirst = (int64_t)b * p.L * ystride + (int64_t)head * p.Cd + c0;
      auto leave = [&](auto* out) {
        using TO = std::remove_pointer_t<decltype(out)>;
        constexpr int OS = 32 + 16 / (int)sizeof(TO);
        // rows at a time that fit the slab's 32 rows
        constexpr int kOut = sizeof(TO) > sizeof(TI) ? 16 : 32;
        TO* so = reinterpret_cast<TO*>(sV + 32 * tt * VS);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kOut) {
#pragma unroll
          for (int i = r0 / 2; i < (r0 + kOut) / 2; ++i)
            so[(tile_row(i, half) - r0) * OS + col] = from_f32<TO>(o[i]);
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int k = 0; k < kOut / 16; ++k) {
            const int un = k * 64 + lane, r = un >> 2, c = (un & 3) * kPack, t = 32 * tt + r0 + r;
            const Pack<TO> v = *reinterpret_cast<const Pack<TO>*>(so + r * OS + c);
            if (t < len && c < cols) store_pack(out + yfirst + token(t) * ystride + c, v, cols - c);
          }
          __builtin_amdgcn_wave_barrier();
        }
      };
      if (p.y_bf16) leave(static_cast<bf16_t*>(p.y));
      else leave(static_cast<float*>(p.y));
    }
  }

  if (STATE) {
    if (active && c0 == 0 && lane == 0)
      p.seg_decay[((int64_t)b * p.H + head) * p.nseg + seg] = hw_exp2((float)whole);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = 32 * kt + tile_row(i, half);
        if (n < p.Kd && col < cols) p.seg_state[sstate + (int64_t)n * p.Cd + c0 + col] = h[kt][i];
      }
  } else if (p.s_final != nullptr && seg == p.nseg - 1) {
    // walking backwards the first token's own decay is still to come
    float f = 1.f;
    if (p.reverse) {
      const float g = gb[0] * kLog2e;
      f = hw_exp2(g < kLeastLog2 ? kLeastLog2 : g);
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = 32 * kt + tile_row(i, half);
        if (n < p.Kd && col < cols) p.s_final[state + n * p.sk + (c0 + col) * p.sc] = h[kt][i] * f;
      }
  }
}

// Host side: launches one walk (or its state pass).
template <typename TI, int KT, int W, int S, int MODE>
int attn_launch(const AttnParams& p, hipStream_t s) {
  const int groups = p.H / p.qshare, units = p.qshare * p.ctiles;
  const int64_t grid = (int64_t)p.B * groups * (MODE == kAttnState ? p.nseg - 1 : p.nseg) * ((units + W - 1) / W);
  if (grid > 0x7fffffff) return SWIMBA_EUNSUPPORTED;
  constexpr size_t lds = AttnShape<TI, KT, W>::kBytes;
  allow_dynamic_lds(attn_kernel<TI, KT, W, S, MODE>, lds);
  hipLaunchKernelGGL((attn_kernel<TI, KT, W, S, MODE>), dim3((unsigned)grid), dim3(64 * W), lds, s,
                     p);
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

template <typename TI, int KT, int W>
int attn_launch_kind(const AttnParams& p, bool state, bool exact, hipStream_t s) {
  if (state) return attn_launch<TI, KT, W, 3, kAttnState>(p, s);
  if (p.z != nullptr) return attn_launch<TI, KT, W, 3, kAttnSums>(p, s);
  if constexpr (sizeof(TI) == 2)
    if (!exact) return attn_launch<TI, KT, W, 2, kAttnPlain>(p, s);
  return attn_launch<TI, KT, W, 3, kAttnPlain>(p, s);
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
