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
// What bounds it (MI355X, bf16, N = 128; 2560-column 64K-token prompt, 41 chunks
// by each of 500 workgroups, two per CU): 9.0 us per chunk and CU.  Of a CU's busy
// cycles the matrix units take 35 % (98 instructions of 32 cycles per wave and
// chunk) and vector issue 50 % (1115 instructions, most of them the splits
// below; each wave splits the shared scores for itself), and 13 % see a conflict
// of LDS banks; the two hardly overlap with two waves per SIMD, the registers'
// limit (64 of state, 32 of results, 48 of rows on their way).  Memory would
// allow a third of the time.
// Measured on the way: loads issued under per-pack branches waited for each
// other (34 us per chunk); one workgroup per CU, when the LDS passed 80 KB by
// half a KB, cost 1.6 x; an exponential per pair instead of two factors per
// token 1.2 x; a full unroll of the token steps, or the order of matrix and vector
// instructions fixed by hand, 0.95 to 1 x.
//
// Roundings.  bf16 inputs multiply exactly.  What is computed in fp32 and
// enters a product (decayed scores, state, decayed values) is split into two
// or three bf16 terms that sum to it within 2^-16 or 2^-24 of its size, two
// where the result is rounded to bf16 anyway, three where it is kept in fp32:
// a single bf16 term would leave 2^-8, as much as the output's own rounding,
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
  float* seg_state;       // [B, H, nseg, Kd, Cd]: end states out (state pass), first states in,
  int64_t fk, fc;         // whose entry (n, c) is at n * fk + c * fc
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
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
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
__device__ __forceinline__ bf8x column8(const bf16_t* tile, int stride, int row, int col,
                                        int lane) {
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
  static constexpr int kGates = 4 * kChunk;  // floats per wave
  // K rows, values and factors; and the Q rows and scores that the state pass
  // does without
  static constexpr size_t kStateBytes = (size_t)(kChunk * kKStride + W * kChunk * kValStride) *
                                            sizeof(TI) + (size_t)W * kGates * sizeof(float);
  static constexpr size_t kBytes = kStateBytes + (size_t)kChunk * kQStride * sizeof(TI) +
                                   (size_t)kChunk * kScoreStride * sizeof(float);
};

typedef uint32_t u4x __attribute__((ext_vector_type(4)));

// Rows of one operand of a chunk, up to eight packs per thread at a time: load()
// issues the loads of a round, pack() has them with zeros beyond `len` rows and
// `cols` columns, store() writes those to LDS.  The packs stay whole registers
// and no load waits for another: without branches between them where rows are
// whole packs; LOOSE rows take one load per pack inside the tensor, moved back
// from its end where it would pass it.
template <typename T, int PAD, int THREADS, bool LOOSE>
struct RowStage {
  static constexpr int kPer = PAD / kPack, kN = kChunk * kPer / THREADS;
  static constexpr int kMost = sizeof(T) == 4 ? 4 : 8;  // 32 registers
  static constexpr int kRound = kN < kMost ? kN : kMost, kRounds = kN / kRound;
  static constexpr int kStep = THREADS / kPer;      // rows between a thread's packs
  static constexpr int kQuads = sizeof(T) / 2;      // 16-byte registers per pack
  static constexpr int kWords = 4 * kQuads;
  struct __attribute__((packed, aligned(sizeof(T)))) Loose { u4x q[kQuads]; };
  const T* base;
  int64_t total;    // elements of the tensor, a pack at least
  int64_t first;    // element of the chunk's lowest token, column 0
  int64_t stride;   // between tokens
  int cols, len, tid;
  bool down;        // row 0 is the highest token
  u4x v[kRound][kQuads];

  __device__ __forceinline__ int row(int i) const { return i * kStep + tid / kPer; }
  __device__ __forceinline__ int column() const { return tid % kPer * kPack; }
  __device__ __forceinline__ bool inside(int r) const { return r < len && column() < cols; }
  __device__ __forceinline__ int64_t element(int r) const {
    return first + (down ? len - 1 - r : r) * stride + column();
  }

  __device__ __forceinline__ void fetch(int i, const T* at) {
    const Loose l = *reinterpret_cast<const Loose*>(at);
#pragma unroll
    for (int q = 0; q < kQuads; ++q) v[i][q] = l.q[q];
  }

  __device__ __forceinline__ void load(int round) {
    if constexpr (!LOOSE) {
      // a chunk's rows lie within 2^31 bytes (checked on the host): a wave-uniform
      // base and 32-bit offsets
      const char* chunk = reinterpret_cast<const char*>(base + first);
      const uint32_t bytes = (uint32_t)stride * (uint32_t)sizeof(T);
      const uint32_t step = (down ? 0u - bytes : bytes) * (uint32_t)kStep;
      const uint32_t mine = (uint32_t)(down ? len - 1 - tid / kPer : tid / kPer) * bytes +
                            (uint32_t)(column() * (int)sizeof(T));
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int n = round * kRound + i;
        const uint32_t off = inside(row(n)) ? mine + (uint32_t)n * step : 0u;
        fetch(i, reinterpret_cast<const T*>(chunk + off));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int r = row(round * kRound + i);
        const int64_t e = inside(r) ? element(r) : 0;
        fetch(i, base + (e + kPack <= total ? e : total - kPack));
      }
    }
  }

  __device__ __forceinline__ void pack(int round, int i, u4x* out) const {
    const int r = row(round * kRound + i);
    const bool in = inside(r);
#pragma unroll
    for (int q = 0; q < kQuads; ++q) out[q] = in ? v[i][q] : u4x{0, 0, 0, 0};
    if constexpr (LOOSE) {
      uint32_t w[kWords];
      __builtin_memcpy(w, out, sizeof(w));
      const int64_t e = element(r);
      const int shift = in && e + kPack > total ? (int)(e + kPack - total) : 0;
      if (__ballot(shift != 0)) {  // the tensor's last elements
        T m[kPack], o[kPack];
        __builtin_memcpy(m, w, sizeof(m));
#pragma unroll
        for (int k = 0; k < kPack; ++k) {
          o[k] = m[k];
#pragma unroll
          for (int l = k + 1; l < kPack; ++l) o[k] = shift == l - k ? m[l] : o[k];
        }
        __builtin_memcpy(w, o, sizeof(o));
      }
      const int n = cols - column();  // columns of this pack
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < kWords; ++k)
          w[k] = n >= 2 * k + 2 ? w[k] : (n == 2 * k + 1 ? w[k] & 0xffffu : 0u);
      } else {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = n > k ? w[k] : 0u;
      }
      __builtin_memcpy(out, w, sizeof(w));
    }
  }

  // An infinity or a NaN among the packs of a round (or in rows left out).
  __device__ __forceinline__ bool wild() const {
    if constexpr (sizeof(T) == 2) {
      typedef unsigned short us2 __attribute__((ext_vector_type(2)));
      us2 m = {0, 0};
#pragma unroll
      for (int i = 0; i < kRound; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, v[i][0][k] & 0x7fff7fffu));
      return m.x >= 0x7f80 || m.y >= 0x7f80;
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kRound; ++i)
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w = v[i][q][k] & 0x7fffffffu;
            m = m > w ? m : w;
          }
      return m >= 0x7f800000u;
    }
  }

  __device__ __forceinline__ void store(int round, T* dst, int dst_stride) const {
    T* d = dst + row(round * kRound) * dst_stride + column();
    if (!LOOSE && len == kChunk && cols >= PAD) {  // nothing to leave out
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kRound; ++i)
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
          reinterpret_cast<u4x*>(d + i * kStep * dst_stride)[q] = v[i][q];
      return;
    }
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      u4x p[kQuads];
      pack(round, i, p);
#pragma unroll
      for (int q = 0; q < kQuads; ++q) reinterpret_cast<u4x*>(d + i * kStep * dst_stride)[q] = p[q];
    }
  }
};

// Inclusive sum over the lanes, in 64 bits, on the DPP row shifts and row
// broadcasts (no LDS round trips: the chunk's decays are waited for).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
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

// Row of register i of a 32 x 32 accumulator tile.
__device__ __forceinline__ int tile_row(int i, int half) {
  return 8 * (i >> 2) + 4 * half + (i & 3);
}

// A rare branch computes its addresses from these for itself: hoisted out of it
// they would cost registers everywhere.
__device__ __forceinline__ int apart(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

enum AttnMode {
  kAttnState = 0,  // only the segment's end state from zero, and its decay
  kAttnPlain = 1,
  kAttnSums = 2    // also the sums of z with the results (the gradient of the decays)
};

// 2^x of a sum in 64 bits, also where it is large: the part of x that fp32
// leaves out multiplies the result.
__device__ __forceinline__ float exp2_sum(double x) {
  const float hi = (float)x;
  return hw_exp2(hi) * fmaf((float)(x - (double)hi), kLn2, 1.f);
}

// Sums of log2 decays inside a chunk that keep e^{G_t} and e^{-G_s} apart, and
// the product of e^{G_t} and the scale that the state carries on top.  Scaled
// partial sums are at most 1 / kLeastScale times what they stand for: fp32 holds
// them up to 2^127 kLeastScale.
constexpr float kLeastSum = -40.f, kMostSum = 16.f;
constexpr float kLeastScale = 0x1p-40f, kMostScale = 0x1p40f;

// S: bf16 terms of what is computed (2 or 3).
template <typename TI, int KT, int W, int S, int MODE, bool LOOSE>
__global__ __launch_bounds__(64 * W, KT > 4 ? 1 : 2) void attn_kernel(AttnParams p) {
  using Sh = AttnShape<TI, KT, W>;
  constexpr bool kF32 = Sh::kF32, STATE = MODE == kAttnState, SUMS = MODE == kAttnSums;
  constexpr int QS = Sh::kQStride, KS = Sh::kKStride, VS = Sh::kValStride;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
  TI* sK = reinterpret_cast<TI*>(smem_raw);
  TI* sVall = sK + kChunk * KS;
  float* sGall = reinterpret_cast<float*>(sVall + W * kChunk * VS);
  float* sS = sGall + W * Sh::kGates;
  TI* sQ = reinterpret_cast<TI*>(sS + kChunk * kScoreStride);
  // the scores' diagonal (SUMS), in the score rows' part above it that nobody reads
  auto diagonal = [&](int t) -> float& { return sS[(t & 31) * kScoreStride + 32 + (t >> 5)]; };

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  TI* sV = sVall + wave * kChunk * VS;
  float* gHi = sGall + wave * Sh::kGates;  // high and low parts of G
  float *gLo = gHi + kChunk;
  float *gRead = gLo + kChunk, *gWrite = gRead + kChunk;  // factors of y_t and of v_s

  // Row tiles of the state that hold rows: tiles past the middle may not.  An fp32
  // product takes 16 times the cycles of a bf16 one, so there a tile without rows
  // is branched round (8192 tokens of 16 heads: 122 -> 110 us with 96 rows, 1270 ->
  // 1015 us with 160, 1270 -> 1353 us where all eight are used; 16384 bf16 tokens:
  // 140 -> 138 us with 160 rows, 155 -> 162 us with 256, not taken).
  constexpr bool kSkip = kF32;
  auto used = [&](int kt) { return !kSkip || kt <= KT / 2 || 32 * kt < p.Kd; };

  // This column's first token with an infinity or a NaN in v: in a row's padding.
  auto bad_at = [&]() -> void* {
    const int at = apart(col);
    return STATE ? static_cast<void*>(sV + at * VS + 32) : sS + at * kScoreStride + kChunk + wave;
  };
  static_assert(W <= kScoreStride - kChunk, "a place per wave");
  auto first_bad = [&] {
    int t;
    __builtin_memcpy(&t, bad_at(), sizeof(t));
    return t;
  };

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
  // (smaller tensors were copied to whole packs)
  const int64_t qall = (int64_t)p.B * p.L * qstride, vall = (int64_t)p.B * p.L * vstride;
  const int64_t qtotal = qall < kPack ? kPack : qall, vtotal = vall < kPack ? kPack : vall;
  const int64_t qfirst = (int64_t)b * p.L * qstride + (int64_t)grp * p.Kd;
  const int64_t vfirst = (int64_t)b * p.L * vstride + (int64_t)(head / p.vshare) * p.Cd + c0;
  const float* gb = p.g + (p.token_decay ? (int64_t)b * p.L * p.H : 0) + head;
  const int64_t state = ((int64_t)b * p.H + head) * p.Kd * p.Cd;
  const int64_t sstate = (((int64_t)b * p.H + head) * p.nseg + seg) * p.Kd * p.Cd;
  const bool down = p.reverse;

  // The state is c * h: a chunk's decay multiplies c, not every entry.
  f16x h[KT];
  float c = 1.f;
  const bool walked = p.nseg > 1;  // first states of segments are in the workspace
  const float* from = STATE ? nullptr : walked ? p.seg_state + sstate : p.s0;
  if (from != nullptr) {
    if (!walked) from += state;
    const int64_t fk = walked ? p.fk : p.sk, fc = walked ? p.fc : p.sc;
    const int64_t at = (c0 + col) * fc;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = 32 * kt + tile_row(i, half);
        h[kt][i] = from[n < p.Kd && col < cols ? n * fk + at : 0];
      }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (32 * kt + tile_row(i, half) >= p.Kd || col >= cols) h[kt][i] = 0.f;
  } else {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) h[kt][i] = 0.f;
  }
  double whole = 0.0;  // log2 decay of the segment so far (state pass)

  using Rows = RowStage<TI, 32 * KT, 64 * W, LOOSE>;
  using Vals = RowStage<TI, 32, 64, LOOSE>;
  // the next chunk's rows travel while this one is worked on, where registers hold them
  constexpr bool kAhead = !kF32 && KT <= 4 && !SUMS;
  Rows rk, rq;
  Vals rv;
  float g = 0.f;
  const int nc = (p.L + kChunk - 1) / kChunk;
  // segments are the same chunks in either direction
  const int low = (down ? p.nseg - 1 - seg : seg) * p.seg_chunks;
  const int high = low + p.seg_chunks < nc ? low + p.seg_chunks : nc;
  const int j0 = down ? nc - high : low, j1 = down ? nc - low : high;
  auto chunk_first = [&](int j) { return (down ? nc - 1 - j : j) * kChunk; };
  auto fetch = [&](int j) {
    const int t0 = chunk_first(j), len = p.L - t0 < kChunk ? p.L - t0 : kChunk;
    rk.base = static_cast<const TI*>(p.k);
    rk.total = qtotal;
    rk.first = qfirst + t0 * qstride;
    rk.stride = qstride;
    rk.cols = p.Kd;
    rk.len = len;
    rk.tid = tid;
    rk.down = down;
    rv.base = static_cast<const TI*>(p.v);
    rv.total = vtotal;
    rv.first = vfirst + t0 * vstride;
    rv.stride = vstride;
    rv.cols = cols;
    rv.len = len;
    rv.tid = lane;
    rv.down = down;
    if (!p.token_decay) {
      g = lane < len && !(down && t0 + len - 1 - lane + 1 >= p.L) ? gb[0] : 0.f;
    } else {
      const int t = down ? t0 + len - lane : t0 + lane;
      const bool in = lane < len && t < p.L;
      g = gb[in ? (int64_t)t * p.H : 0];
      if (!in) g = 0.f;
    }
    rv.load(0);
    rk.load(0);
    if (!STATE) {
      rq.base = static_cast<const TI*>(p.q);
      rq.total = rk.total;
      rq.first = rk.first;
      rq.stride = rk.stride;
      rq.cols = rk.cols;
      rq.len = rk.len;
      rq.tid = rk.tid;
      rq.down = down;
      if (Rows::kRounds == 1) rq.load(0);
    }
  };
  if (kAhead) fetch(j0);

  for (int j = j0; j < j1; ++j) {
    const int t0 = chunk_first(j), len = p.L - t0 < kChunk ? p.L - t0 : kChunk;
    auto token = [&](int r) { return (int64_t)(down ? t0 + len - 1 - r : t0 + r); };
    if (!kAhead) fetch(j);

    // log2 decays, summed over the lanes
    const double d = (double)g * 1.4426950408889634;
    const double sum = wave_prefix(d < (double)kLeastLog2 ? (double)kLeastLog2 : d);
    const double end = last_lane(sum);
    const float hi = (float)sum;
    // Where no sum is far from zero, D[t][s] = e^{G_t} e^{-G_s}: one factor on y_t
    // and one on v_s, both with the state's scale c in them:
    //   y_t = e^{G_t} c ((Q h)_t + sum_s (q_t . k_s) (e^{-G_s} / c) v_s),
    //   h' = h + K^T ((e^{-G} / c) V),  c' = e^{G_end} c.
    // Elsewhere (a cleared state, a NaN) every pair has its own exponential and
    // h is scaled.
    const bool split = __ballot(!(hi >= kLeastSum && hi <= kMostSum)) == 0;
    float read = exp2_sum(sum) * c;
    if (!split || __ballot(!(read >= kLeastScale && read <= kMostScale))) {
      __builtin_amdgcn_sched_barrier(0);  // rare: a branch, not a product with one
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) h[kt][i] *= c;
      c = 1.f;
      read = exp2_sum(sum);
    }
    const float write = split ? exp2_sum(-sum) / c : exp2_sum(end - sum);
    __syncthreads();  // everyone is done with the last chunk
    gHi[lane] = hi;
    gLo[lane] = (float)(sum - (double)hi);
    gRead[lane] = read;
    gWrite[lane] = write;
    const bool wild = __ballot(rv.wild()) != 0;
    rv.store(0, sV, VS);
    if (wild) {
      // An infinity or a NaN in v_s may reach y_t for t >= s only, and a product of
      // the matrix units with a zero score would spread it.  It is taken out of
      // the slab, and the column's state and its results from it on become NaN
      // behind the products (the results in memory: branches round their registers
      // cost 25 of them, and in LDS on their way out 3 % of a walk).
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_wave_barrier();
      int bad = kChunk;
#pragma unroll 1
      for (int r = 31; r >= 0; --r) {
        TI* at = sV + (32 * half + r) * VS + col;
        if (!(fabsf(to_f32(*at)) < __builtin_inff())) {
          bad = 32 * half + r;
          *at = TI(0);
        }
      }
      const int o = __shfl_xor(bad, 32);
      bad = o < bad ? o : bad;
      __builtin_memcpy(bad_at(), &bad, sizeof(bad));
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
    rk.store(0, sK, KS);
#pragma unroll
    for (int r = 1; r < Rows::kRounds; ++r) {
      rk.load(r);
      rk.store(r, sK, KS);
    }
    if (!STATE) {
#pragma unroll
      for (int r = 0; r < Rows::kRounds; ++r) {
        if (!(Rows::kRounds == 1)) rq.load(r);
        rq.store(r, sQ, QS);
      }
    }
    __syncthreads();
    if (kAhead && j + 1 < j1) fetch(j + 1);

    if (!STATE) {
      // scores Q K^T, zero above the diagonal (SUMS: and on it): the three 32 x 32
      // tiles that are read
      for (int tile = wave; tile < 3; tile += W) {
        const int tt = tile > 0, ss = tile > 1;
        f16x a;
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = 0.f;
        const TI* qr = sQ + (32 * tt + col) * QS;
        const TI* kr = sK + (32 * ss + col) * KS;
        if constexpr (kF32) {
          const int rows = (p.Kd + 31) & ~31;
#pragma unroll 4
          for (int n = 0; n < rows; n += 8) {
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
        const int lead = tt > ss ? 32 : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = tile_row(i, half);
          if (SUMS && lead == 0 && r == col) diagonal(32 * tt + r) = a[i];
          const bool seen = SUMS ? col < r + lead : col <= r + lead;
          sS[(32 * tt + r) * kScoreStride + 32 * ss + col] = seen ? a[i] : 0.f;
        }
      }
    }

    // a wave at its products goes before one that stages rows (2 to 5 % of a walk)
    __builtin_amdgcn_s_setprio(1);
    f16x ys[2];  // from the state
    f16x yi[2];  // from the chunk (SUMS: apart)
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
        if (!used(kt)) continue;
        if constexpr (kF32) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
              const float4 x = *reinterpret_cast<const float4*>(sQ + (32 * tt + col) * QS +
                                                                32 * kt + 8 * a + 4 * half);
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
            bf8x a[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
              const TI* r = sQ + (32 * tt + col) * QS + 32 * kt + 16 * k2 + 4 * half;
              struct { uint2 a, b; } qa;
              qa.a = *reinterpret_cast<const uint2*>(r);
              qa.b = *reinterpret_cast<const uint2*>(r + 8);
              a[tt] = __builtin_bit_cast(bf8x, qa);
            }
#pragma unroll
            for (int s = S - 1; s >= 0; --s)
#pragma unroll
              for (int tt = 0; tt < 2; ++tt) ys[tt] = mma(a[tt], t[s], ys[tt]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // keep the operands of few steps in registers
      }
      __syncthreads();  // the scores are there (the state's part did not need them)
    }
    // y_t's factor, from the state's part before the sums or on all of it after
    auto scale_rows = [&](f16x(&v)[2]) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const float4 e = *reinterpret_cast<const float4*>(gRead + 32 * tt + 8 * a + 4 * half);
          v[tt][4 * a] *= e.x;
          v[tt][4 * a + 1] *= e.y;
          v[tt][4 * a + 2] *= e.z;
          v[tt][4 * a + 3] *= e.w;
        }
    };
    if (!split) {
      __builtin_amdgcn_sched_barrier(0);
      if (!STATE) scale_rows(ys);
      const float carry = exp2_sum(end);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) h[kt][i] *= carry;
    }

    // 8 (fp32) or 16 (bf16) tokens s at a time: y += M V, h += K^T (w V)
    constexpr int kStep = kF32 ? 8 : 16;
#pragma unroll 1
    for (int s0 = 0; s0 < kChunk; s0 += kStep) {
      constexpr int kV = kF32 ? 4 : 8;  // tokens per lane and step
      const int sl = s0 + kV * half;
      float vf[kV], ws[kV];
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
#pragma unroll
      for (int i = 0; i < kV; i += 4)
        *reinterpret_cast<float4*>(ws + i) = *reinterpret_cast<const float4*>(gWrite + sl + i);
      if (!STATE) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          if (32 * tt + 31 < s0) continue;
          const int t = 32 * tt + col;
          float m[kV];
#pragma unroll
          for (int i = 0; i < kV; i += 4)
            *reinterpret_cast<float4*>(m + i) =
                *reinterpret_cast<const float4*>(sS + t * kScoreStride + sl + i);
          if (split) {
#pragma unroll
            for (int i = 0; i < kV; ++i) m[i] *= ws[i];
          } else {
            const float ht = gHi[t], lt = gLo[t];
#pragma unroll
            for (int i = 0; i < kV; ++i) {
              const float e = hw_exp2((ht - gHi[sl + i]) + (lt - gLo[sl + i]));
              m[i] = sl + i <= t ? m[i] * e : 0.f;
            }
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
#pragma unroll
      for (int i = 0; i < kV; ++i) vf[i] *= ws[i];
      if constexpr (kF32) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          if (!used(kt)) continue;
#pragma unroll
          for (int i = 0; i < kV; ++i) h[kt] = mma(sK[(sl + i) * KS + 32 * kt + col], vf[i], h[kt]);
        }
      } else {
        bf8x wt[3];
        split_terms<3>(vf, wt);
        bf8x a[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) a[kt] = column8(sK, KS, s0, 32 * kt, lane);
#pragma unroll
        for (int s = 2; s >= 0; --s)
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
            if (used(kt)) h[kt] = mma(a[kt], wt[s], h[kt]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (split) c *= exp2_sum(end);
    if (wild) {
      __builtin_amdgcn_sched_barrier(0);
      const bool lost = first_bad() < kChunk;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) h[kt][i] = lost ? __builtin_nanf("") : h[kt][i];
    }
    if (STATE) {
      whole += end;
      continue;
    }
    if (split) {
      __builtin_amdgcn_sched_barrier(0);
      scale_rows(ys);
      if (SUMS) scale_rows(yi);
    }

    const int64_t ystride = (int64_t)p.H * p.Cd;
    const int64_t yfirst = (int64_t)b * p.L * ystride + (int64_t)head * p.Cd + c0;
    if constexpr (SUMS) {
      // 16 rows at a time the two parts pass through the wave's V slab (free once
      // the rows for the diagonal are out) to eight columns per lane, four lanes
      // per row, where z comes from memory and the sums stay short.
      Vals rz;
      rz.base = static_cast<const TI*>(p.z);
      rz.total = vtotal;
      rz.first = vfirst + t0 * vstride;
      rz.stride = vstride;
      rz.cols = cols;
      rz.len = len;
      rz.tid = lane;
      rz.down = down;
      rz.load(0);
      Pack<TI> vd[Vals::kN];
#pragma unroll
      for (int k = 0; k < Vals::kN; ++k)
        vd[k] = *reinterpret_cast<const Pack<TI>*>(sV + rz.row(k) * VS + rz.column());
      __builtin_amdgcn_wave_barrier();
      constexpr int OS = 36;
      float* part = reinterpret_cast<float*>(sV);  // [2][16][OS]
      static_assert(2 * 16 * OS * sizeof(float) <= kChunk * VS * sizeof(TI), "the slab");
#pragma unroll
      for (int k = 0; k < Vals::kN; ++k) {
        const int tt = k >> 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = tile_row(i, half) * OS + col;
          part[r] = yi[tt][8 * (k & 1) + i];
          part[16 * OS + r] = ys[tt][8 * (k & 1) + i];
        }
        __builtin_amdgcn_wave_barrier();
        const int t = rz.row(k), cc = rz.column();
        float in[kPack], st[kPack];
#pragma unroll
        for (int i = 0; i < kPack; i += 4) {
          const float* r = part + (lane >> 2) * OS + cc + i;
          *reinterpret_cast<float4*>(in + i) = *reinterpret_cast<const float4*>(r);
          *reinterpret_cast<float4*>(st + i) = *reinterpret_cast<const float4*>(r + 16 * OS);
        }
        u4x zq[Vals::kQuads];
        rz.pack(0, k, zq);
        Pack<TI> z;
        __builtin_memcpy(&z, zq, sizeof(z));
        float zin = 0.f, zst = 0.f;
        const float dg = diagonal(t);
#pragma unroll
        for (int i = 0; i < kPack; ++i) {
          zin = fmaf(to_f32(z.v[i]), in[i], zin);
          zst = fmaf(to_f32(z.v[i]), st[i], zst);
          in[i] = fmaf(dg, to_f32(vd[k].v[i]), in[i]) + st[i];
        }
        zin += xor_lane<1>(zin, lane);
        zst += xor_lane<1>(zst, lane);
        zin += xor_lane<2>(zin, lane);
        zst += xor_lane<2>(zst, lane);
        if (t < len && cc < cols) {
          const int64_t at = yfirst + token(t) * ystride + cc;
          if (p.y_bf16) {
            Pack<bf16_t> o;
#pragma unroll
            for (int i = 0; i < kPack; ++i) o.v[i] = from_f32<bf16_t>(in[i]);
            store_pack(static_cast<bf16_t*>(p.y) + at, o, LOOSE ? cols - cc : kPack);
          } else {
            Pack<float> o;
#pragma unroll
            for (int i = 0; i < kPack; ++i) o.v[i] = in[i];
            store_pack(static_cast<float*>(p.y) + at, o, LOOSE ? cols - cc : kPack);
          }
        }
        if (active && (lane & 3) == 0 && t < len) {
          float* zs = p.zsum + (((int64_t)b * p.H + head) * p.ctiles + u % p.ctiles) * 2 * p.L;
          zs[token(t)] = zin;
          zs[p.L + token(t)] = zst;
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      // The results leave through the wave's V slab, 32 rows at a time (16 where
      // they are wider), as whole packs.
      auto leave = [&](auto* out) {
        using TO = std::remove_pointer_t<decltype(out)>;
        constexpr int OS = 32 + 16 / (int)sizeof(TO);
        constexpr int kOut = sizeof(TO) > sizeof(TI) ? 16 : 32;
        TO* so = reinterpret_cast<TO*>(sV);
        static_assert(kOut * OS * sizeof(TO) <= kChunk * VS * sizeof(TI), "the slab");
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += kOut) {
#pragma unroll
            for (int i = r0 / 2; i < (r0 + kOut) / 2; ++i)
              so[(tile_row(i, half) - r0) * OS + col] = from_f32<TO>(ys[tt][i]);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int k = 0; k < kOut / 16; ++k) {
              const int un = k * 64 + lane, r = un >> 2, cc = (un & 3) * kPack;
              const int t = 32 * tt + r0 + r;
              const Pack<TO> v = *reinterpret_cast<const Pack<TO>*>(so + r * OS + cc);
              if (t < len && cc < cols)
                store_pack(out + yfirst + token(t) * ystride + cc, v, LOOSE ? cols - cc : kPack);
            }
            __builtin_amdgcn_wave_barrier();
          }
      };
      if (p.y_bf16) leave(static_cast<bf16_t*>(p.y));
      else leave(static_cast<float*>(p.y));
    }
    if (wild) {  // over what has left
      __builtin_amdgcn_sched_barrier(0);
      __threadfence();
      const int at = apart(col);
      int bad = first_bad();
#pragma unroll 1
      for (int t = bad + (apart(lane) >> 5); t < len; t += 2) {
        const int64_t to = yfirst + token(t) * ystride + at;
        if (at >= cols) break;
        if (p.y_bf16) static_cast<bf16_t*>(p.y)[to] = from_f32<bf16_t>(__builtin_nanf(""));
        else static_cast<float*>(p.y)[to] = __builtin_nanf("");
      }
      if (SUMS) {
#pragma unroll 1
        for (int m = 1; m < 32; m <<= 1) {
          const int o = __shfl_xor(bad, m);
          bad = o < bad ? o : bad;
        }
        float* zs = p.zsum + (((int64_t)b * p.H + head) * p.ctiles + u % p.ctiles) * 2 * p.L;
        const int t = bad + apart(lane);
        if (active && t < len) zs[p.L + token(t)] = __builtin_nanf("");
      }
    }
  }

  if (STATE) {
    if (active && c0 == 0 && lane == 0)
      p.seg_decay[((int64_t)b * p.H + head) * p.nseg + seg] = exp2_sum(whole);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = 32 * kt + tile_row(i, half);
        if (n < p.Kd && col < cols)
          p.seg_state[sstate + (int64_t)n * p.Cd + c0 + col] = h[kt][i] * c;
      }
  } else if (p.s_final != nullptr && seg == p.nseg - 1) {
    // walking backwards the first token's own decay is still to come
    float f = c;
    if (down) {
      const float l = gb[0] * kLog2e;
      f *= hw_exp2(l < kLeastLog2 ? kLeastLog2 : l);
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
template <typename TI, int KT, int W, int S, int MODE, bool LOOSE>
int attn_launch(const AttnParams& p, hipStream_t s) {
  const int groups = p.H / p.qshare, units = p.qshare * p.ctiles;
  const int64_t grid = (int64_t)p.B * groups * (MODE == kAttnState ? p.nseg - 1 : p.nseg) *
                       ((units + W - 1) / W);
  using Sh = AttnShape<TI, KT, W>;
  constexpr size_t lds = MODE == kAttnState ? Sh::kStateBytes : Sh::kBytes;
  static_assert(lds <= 160 * 1024, "a CU's LDS");
  allow_dynamic_lds(attn_kernel<TI, KT, W, S, MODE, LOOSE>, lds);
  hipLaunchKernelGGL((attn_kernel<TI, KT, W, S, MODE, LOOSE>), dim3((unsigned)grid), dim3(64 * W),
                     lds, s, p);
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

template <typename TI, int KT, int W, bool LOOSE>
int attn_launch_kind(const AttnParams& p, bool state, bool exact, hipStream_t s) {
  if (state) return attn_launch<TI, KT, W, 3, kAttnState, LOOSE>(p, s);
  if (p.z != nullptr) return attn_launch<TI, KT, W, 3, kAttnSums, LOOSE>(p, s);
  if constexpr (sizeof(TI) == 2)
    if (!exact) return attn_launch<TI, KT, W, 2, kAttnPlain, LOOSE>(p, s);
  return attn_launch<TI, KT, W, 3, kAttnPlain, LOOSE>(p, s);
}

// Waves of a workgroup: four where that many units share q and k, else two (two
// everywhere: 1152 against 533 us for the 64K-token prompt, 781 against 388 us for
// the 1.4B-like prompts, whose rows then do not fit the registers).
// Rows that are not whole packs always go by two (fewer kernels; the packs'
// masks cost more than the sharing gives), and fp32 rows of 256 leave LDS for
// one wave's values only.
inline int attn_waves(bool f32, int Kd, int Cd, int64_t units) {
  if (f32 && Kd > 128) return 1;
  if (Kd % kPack != 0 || Cd % kPack != 0) return 2;
  return units >= 3 ? 4 : 2;
}

// Workgroups of a walk that a CU holds at once: by its LDS, and two waves per
// SIMD by the registers (one with rows of more than 128).
template <typename TI, int KT>
int attn_resident_rows(int waves) {
  size_t lds = 0;
  if (waves == 4) lds = AttnShape<TI, KT, 4>::kBytes;
  else if (waves == 2) lds = AttnShape<TI, KT, 2>::kBytes;
  else lds = AttnShape<TI, KT, 1>::kBytes;
  const int by_lds = (int)(160 * 1024 / lds), by_regs = (KT > 4 ? 4 : 8) / waves;
  return by_lds < by_regs ? by_lds : by_regs;
}
template <typename TI>
int attn_resident(int Kd, int waves) {
  if (Kd <= 32) return attn_resident_rows<TI, 1>(waves);
  if (Kd <= 64) return attn_resident_rows<TI, 2>(waves);
  if (Kd <= 128) return attn_resident_rows<TI, 4>(waves);
  return attn_resident_rows<TI, 8>(waves);
}

template <typename TI, int KT>
int attn_launch_waves(const AttnParams& p, bool state, bool exact, hipStream_t s) {
  const int64_t units = (int64_t)p.qshare * p.ctiles;
  const bool loose = p.Kd % kPack != 0 || p.Cd % kPack != 0;
  if constexpr (sizeof(TI) == 4 && KT == 8) {
    return loose ? attn_launch_kind<TI, KT, 1, true>(p, state, exact, s)
                 : attn_launch_kind<TI, KT, 1, false>(p, state, exact, s);
  } else {
    if (loose) return attn_launch_kind<TI, KT, 2, true>(p, state, exact, s);
    if (attn_waves(sizeof(TI) == 4, p.Kd, p.Cd, units) == 4)
      return attn_launch_kind<TI, KT, 4, false>(p, state, exact, s);
    return attn_launch_kind<TI, KT, 2, false>(p, state, exact, s);
  }
}

// One per dtype and padded row size.
#define SWIMBA_ATTN_DECL(name) \
  int name(const AttnParams& p, bool state, bool exact, hipStream_t s);
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
