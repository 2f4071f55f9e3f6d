// The gated delta rule, in chunks on the matrix units.
//
//   h~ = e^{g_t} h_{t-1},  u_t = beta_t (v_t - h~^T k_t),  h_t = h~ + k_t u_t^T,  y_t = h_t^T q_t.
// With h the state before a chunk of 64 tokens, G_t the running sum of g inside it,
// D[t][s] = e^{G_t - G_s}, w_s = e^{G_end - G_s} and o_t = u_t / beta_t:
//   (I + A diag(beta)) O = V - e^G K h,   A[t][s] = D[t][s] k_t . k_s  for s < t
//   y  = e^G Q h + ((Q K^T) * D) (beta O),   h' = e^{G_end} h + K^T (w beta O).
// The 64 x 64 inverse T = (I + A diag(beta))^-1 depends on no state: delta_prep_kernel
// makes it for every chunk and head at once.  delta_walk_kernel carries the state through
// them, with the decayed scores S = (Q K^T) * D, which it makes for itself (written out
// by the preparation they cost as much memory traffic as T).
// Backwards, with a = dL/dh' and dU = dL/d(beta O):
//   dU = S^T dY + w K a,   dV = T^T (beta dU),
//   a0 = e^{G_end} a + Q^T (e^G dY) - K^T (e^G dV),
// the same walk with operands exchanged; delta_grad_kernel makes the other
// gradients from each chunk's h, a, O and dV, every chunk for itself.
//
// Mapping of a walk.  A wave owns 16 columns of the state (its 16 x 16 accumulator
// tiles hold h[n][c] in fp32 for the whole walk).  Register for register the
// accumulator layout of two tiles is the layout of the other operand of a product
// over their 32 rows when these run in the order n = 4 g + j, 16 + 4 g + j
// (g = lane / 16, j < 4): state, O and U go from one product to the next without
// leaving their lane.  K and Q rows lie in LDS in that order.
//
// Roundings.  bf16 inputs multiply exactly.  What is computed in fp32 and enters a
// product, and fp32 inputs, are three bf16 terms, which hold them within 2^-27 of their
// size (2^-9 for each of three round-to-nearests); of a product of two such operands
// the pairs of 2^-27 and below are left out.  Two terms (2^-18) leave 3e-6 of the states in
// the 2-norm, 7e-6 of gradients, 1e-4 of a decay's that cancels over the tokens.  For a y in
// bf16 they would do where it does not cancel, but one in 300 of its values is another
// one then, and of sums |q| |h| that cancel to 2^-10 of them bits are lost: three there as well
// (8 x 4096 tokens of 32 heads of 128 x 128: 680 us instead of 630; 64K tokens of 40 heads
// of 128 x 64: 2053 instead of 1995).
// Sums, states and inverses are fp32; sums of log decays are in 64 bits.
#pragma once
#include "attention.hpp"

namespace swimba {

typedef float f4x __attribute__((ext_vector_type(4)));

constexpr int kDeltaBlocks = 6;               // 16 x 32 blocks of a triangle of 64 x 64
constexpr int kDeltaTri = kDeltaBlocks * 512; // values of a triangle
constexpr int kDeltaTerms = 3;
// Of a chunk and head, 64 floats each: e^G, w, beta, (e^{G_end}, first bad token), and
// G / ln 2 in a high and a low part.
constexpr int kDeltaGates = 6 * kChunk;

struct DeltaParams {
  const void *q, *k, *v, *dy;
  void* out;              // y, or dv
  const float *g, *beta;  // [H] or [B, L, H]; [B, L, H]
  int B, L, H, G, N, P;
  int token_decay, out_bf16;
  int nc;                 // chunks
  int ctiles;             // workgroups for the columns of a state
  int nseg, seg_chunks;   // segments of the walk, chunks in each
  int state_segs;         // segments of a state pass
  float* seg_state;       // [B, H, nseg, N', P'] end states out (state pass), first states in
  float* seg_carry;       // [B, H, nseg, N', N'] the segments' transitions (state pass)
  // workspace, per (b, h, chunk)
  float *tri, *tri_t;     // [kDeltaTri] T in operand order; its transpose (backward)
  float* gates;           // [kDeltaGates]
  const float* s0;        // first state or null, [B, H, N, P]
  float* s_final;         // or null
  float* states;          // [N', P'] the state before (behind: walking back) the chunk
  float* rows;            // [64, P'] O, or dV
  int Pp;                 // P' = P rounded up to 64
};

__device__ __forceinline__ f4x mma16(bf8x a, bf8x b, f4x c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4x mma16(float a, float b, f4x c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// c += a b of operands in terms, smallest products first; pairs of terms beyond the finer
// operand's last one are left out.
template <int NA, int NB>
__device__ __forceinline__ f4x mma_terms(const bf8x* a, const bf8x* b, f4x c) {
  constexpr int kLast = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int n = kLast; n >= 0; --n)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (n - i >= 0 && n - i < NB) c = mma16(a[i], b[n - i], c);
  return c;
}

// The same for M accumulators that share one operand: products of one pair of terms next to
// each other, as none of them waits for another.
template <int NA, int NB, int M>
__device__ __forceinline__ void mma_tiles(const bf8x (*a)[NA], const bf8x* b, f4x* c) {
  constexpr int kLast = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int n = kLast; n >= 0; --n)
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (n - i >= 0 && n - i < NB) c[m] = mma16(a[m][i], b[n - i], c[m]);
}

// x (V values, even) as S bf16 terms, as split_terms() makes them.  What a pair of terms leaves
// is one two-element product each, x - 1 * term + 0 * the other, which is exact: seven
// instructions for a pair's three terms instead of eleven.  The factors come from
// registers: as constants in the instruction they are read as fp32 numbers.
template <int S, int V>
__device__ __forceinline__ void split_pairs(const float* x, uint32_t (*out)[V / 2]) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  uint32_t first = 0x0000bf80u, second = 0xbf800000u;  // (-1, 0) and (0, -1)
  asm("" : "+s"(first), "+s"(second));
  float r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = x[i];
#pragma unroll
  for (int s = 0; s < S; ++s) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) out[s][i] = bf16_pair(r[2 * i], r[2 * i + 1]);
    if (s + 1 < S) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const b2 t = __builtin_bit_cast(b2, out[s][i]);
        r[2 * i] = __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(b2, first), r[2 * i], false);
        r[2 * i + 1] =
            __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(b2, second), r[2 * i + 1], false);
      }
    }
  }
}

template <int S>
__device__ __forceinline__ void split_values(const float* x, bf8x* out) {
  uint32_t w[S][4];
  split_pairs<S, 8>(x, w);
#pragma unroll
  for (int s = 0; s < S; ++s) out[s] = __builtin_bit_cast(bf8x, u4x{w[s][0], w[s][1], w[s][2], w[s][3]});
}

// Two accumulator tiles as one operand in S terms.
template <int S>
__device__ __forceinline__ void split_tiles(f4x lo, f4x hi, bf8x* out) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lo[i];
    x[4 + i] = hi[i];
  }
  split_values<S>(x, out);
}

// First block of row tile rt of a triangle (tiles 0, 1: one block of 32, tiles 2, 3:
// two), and of its transpose (tiles 0, 1: two blocks, tiles 2, 3: the second).
__device__ __forceinline__ constexpr int tri_block(int rt, int b) {
  return rt < 2 ? rt : 2 * rt - 2 + b;
}
__device__ __forceinline__ constexpr int tri_block_t(int rt, int b) {
  return rt < 2 ? 2 * rt + b : 2 + rt;
}

template <typename TI, int KT>
struct DeltaShape {
  static constexpr bool kF32 = sizeof(TI) == 4;
  static constexpr int kTerms = kF32 ? kDeltaTerms : 1;
  static constexpr int kRows = 32 * KT;
  static constexpr int kStride = kRows;
  static constexpr int kTile = kChunk * kStride;  // values of one term

  // Where a row's values lie.  Slots of eight hold what a lane takes of a block of 32
  // columns (4 g.. and 16 + 4 g..), and a row's slots are exchanged by an exclusive or
  // with mix(row): 16 rows at one slot, the 4 rows by 4 slots of a transposing read, and
  // the even or odd slots of four rows that a store has, are then different slots of the
  // 64 banks.
  static __device__ __forceinline__ int mix(int row) {
    if constexpr (KT >= 4) return ((row & 3) << 2) | (((row >> 2) + row) & 3);
    else if constexpr (KT == 2) return ((row & 2) << 1) | ((row >> 2) & 3);
    else return (row >> 2) & 3;
  }
  static __device__ __forceinline__ int slot(int row, int n) { return 8 * (n ^ mix(row)); }
  // Place of column `col` (a multiple of four).
  static __device__ __forceinline__ int place(int row, int col) {
    return row * kStride + slot(row, 4 * (col >> 5) + ((col & 15) >> 2)) + (col & 16) / 4;
  }
};

constexpr int kDeltaThreads = 256, kDeltaWaves = 4;
constexpr int kWalkCols = 16 * kDeltaWaves;  // columns of a walk's workgroup, 16 of a wave

// The staged rows of a chunk into LDS, in operand order and in terms; rows from `len` on
// are zero.
template <typename TI, int KT, bool LOOSE>
struct DeltaRows {
  using Stage = RowStage<TI, 32 * KT, kDeltaThreads, LOOSE>;
  using Sh = DeltaShape<TI, KT>;
  static __device__ __forceinline__ void put(const Stage& st, int round, bf16_t* dst) {
    if (!LOOSE && st.len == kChunk && st.cols >= Sh::kRows) put_as<true>(st, round, dst);
    else put_as<false>(st, round, dst);
  }
  template <bool FULL>  // nothing to leave out
  static __device__ __forceinline__ void put_as(const Stage& st, int round, bf16_t* dst) {
#pragma unroll
    for (int i = 0; i < Stage::kRound; ++i) {
      u4x w[Stage::kQuads];
      if constexpr (FULL) {
#pragma unroll
        for (int q = 0; q < Stage::kQuads; ++q) w[q] = st.v[i][q];
      } else {
        st.pack(round, i, w);
      }
      const int row = st.row(round * Stage::kRound + i);
      bf16_t* d = dst + Sh::place(row, st.column());
      bf16_t* d4 = dst + Sh::place(row, st.column() + 4);
      if constexpr (Sh::kF32) {
        float x[8];
        __builtin_memcpy(x, w, sizeof(x));
        bf8x t[Sh::kTerms];
        split_values<Sh::kTerms>(x, t);
#pragma unroll
        for (int s = 0; s < Sh::kTerms; ++s) {
          struct { uint2 a, b; } o = __builtin_bit_cast(decltype(o), t[s]);
          *reinterpret_cast<uint2*>(d + s * Sh::kTile) = o.a;
          *reinterpret_cast<uint2*>(d4 + s * Sh::kTile) = o.b;
        }
      } else {
        *reinterpret_cast<uint2*>(d) = make_uint2(w[0][0], w[0][1]);
        *reinterpret_cast<uint2*>(d4) = make_uint2(w[0][2], w[0][3]);
      }
    }
  }
  static __device__ __forceinline__ void all(Stage& st, bf16_t* dst) {
#pragma unroll
    for (int r = 0; r < Stage::kRounds; ++r) {
      if (r > 0) st.load(r);
      put(st, r, dst);
    }
  }
  static __device__ __forceinline__ void place(Stage& st, const void* base, const DeltaParams& p,
                                               int b, int grp, int t0, int len, int tid) {
    const int64_t stride = (int64_t)p.G * p.N, all = (int64_t)p.B * p.L * stride;
    st.base = static_cast<const TI*>(base);
    st.total = all < kPack ? kPack : all;  // (smaller tensors were copied to whole packs)
    st.first = ((int64_t)b * p.L + t0) * stride + (int64_t)grp * p.N;
    st.stride = stride;
    st.cols = p.N;
    st.len = len;
    st.tid = tid;
    st.down = false;
  }
};

// Operand of 16 rows (from `row`) by 32 columns (block b) of staged rows.
template <typename Sh>
__device__ __forceinline__ void row_operand(const bf16_t* tile, int row, int b, int lane,
                                            bf8x* out) {
#pragma unroll
  for (int s = 0; s < Sh::kTerms; ++s)
    out[s] = *reinterpret_cast<const bf8x*>(tile + s * Sh::kTile +
                                            (row + (lane & 15)) * Sh::kStride +
                                            Sh::slot(lane & 15, 4 * b + (lane >> 4)));
}

// Operand of 16 columns (tile nt) by 32 rows (block b) of staged rows: the transposing
// read hands lane i of 16 the column i of four rows, of which it points at row
// i / 4, columns 4 (i % 4)..
template <typename Sh>
__device__ __forceinline__ void column_operand(const bf16_t* tile, int nt, int b, int lane,
                                               bf8x* out) {
  typedef __attribute__((address_space(3))) s4x* lds_s4;
  const int i = lane & 15, row = 4 * (lane >> 4) + (i >> 2);
  const bf16_t* p = tile + (32 * b + row) * Sh::kStride + Sh::slot(row, 4 * (nt >> 1) + (i & 3)) +
                    4 * (nt & 1);
#pragma unroll
  for (int s = 0; s < Sh::kTerms; ++s) {
    struct { s4x a, b; } r;
    r.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + s * Sh::kTile));
    r.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + s * Sh::kTile + 16 * Sh::kStride));
    out[s] = __builtin_bit_cast(bf8x, r);
  }
}

// ---- what depends on no state -------------------------------------------------

constexpr int kTriStride = kChunk + 4;

// Blocks of a triangle whose row tile `rt` a wave holds, tile by tile (zero beyond the diagonal),
// in operand order.
template <bool TRANSPOSED>
__device__ __forceinline__ void put_tiles(const f4x* tiles, int rt, float* out, int lane) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (TRANSPOSED ? b < rt / 2 : b > rt / 2) continue;
    const int blk = TRANSPOSED ? tri_block_t(rt, b) : tri_block(rt, b);
    f4x* to = reinterpret_cast<f4x*>(out + (blk * 64 + lane) * 8);
    to[0] = tiles[2 * b];
    to[1] = tiles[2 * b + 1];
  }
}

constexpr int kDiagStride = 20;

// T = (I + A)^-1 of a strictly lower triangular A of 64 x 64, in fp32; `at` holds A^T, its rows
// kTriStride apart.  The four blocks of 16 x 16 on the diagonal by substitution in one
// wave, a lane per row of T: T[i][k] = [i = k] - sum_{m > k} T[i][m] A[m][k], transposed
// into `diag`.
__device__ __forceinline__ void unit_blocks(const float* at, float* diag, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const float* a = at + 16 * g * kTriStride + 16 * g;
  float x[16];
#pragma unroll
  for (int k = 15; k >= 0; --k) {
    float s = i == k ? 1.f : 0.f;
#pragma unroll
    for (int m = k / 4 * 4; m < 16; m += 4) {
      const float4 r = *reinterpret_cast<const float4*>(a + k * kTriStride + m);
      if (m > k) s = fmaf(-r.x, x[m], s);
      if (m + 1 > k) s = fmaf(-r.y, x[m + 1], s);
      if (m + 2 > k) s = fmaf(-r.z, x[m + 2], s);
      if (m + 3 > k) s = fmaf(-r.w, x[m + 3], s);
    }
    x[k] = s;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) diag[(16 * g + k) * kDiagStride + i] = x[k];
}

// The tiles of block row `row` of T, transposed: x[j] = T_row,j^T, by
//   T_ij = -(sum_{j < k <= i} T_ik A_kj) T_jj,
// where a product's result is register for register the next one's right operand.
__device__ __forceinline__ void unit_row(const float* at, const float* diag, int row, int lane,
                                         f4x* x) {
  const int g = lane >> 4, col = lane & 15;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = f4x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i != row) continue;  // (uniform)
#pragma unroll
    for (int r = 0; r < 4; ++r) x[i][r] = diag[(16 * i + 4 * g + r) * kDiagStride + col];
#pragma unroll
    for (int j = 2; j >= 0; --j) {
      if (j >= i) continue;
      f4x s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 3; k >= 1; --k) {
        if (k > i || k <= j) continue;
        const f4x a = *reinterpret_cast<const f4x*>(at + (16 * j + col) * kTriStride + 16 * k +
                                                    4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) s = mma16(a[r], x[k][r], s);
      }
      const f4x d = *reinterpret_cast<const f4x*>(diag + (16 * j + col) * kDiagStride + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[j] = mma16(-d[r], s[r], x[j]);
    }
  }
}

__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) < __builtin_inff()); }

template <typename TI, int KT>
constexpr size_t delta_prep_lds(bool back) {
  using Sh = DeltaShape<TI, KT>;
  const size_t rows = (size_t)Sh::kTerms * Sh::kTile * sizeof(bf16_t);
  const size_t tris = ((back ? 2 : 1) * (size_t)kChunk * kTriStride + kChunk * kDiagStride) *
                      sizeof(float);
  return (rows > tris ? rows : tris) + 4 * kChunk * sizeof(float);
}

// One workgroup per chunk and head.  Tokens from the first one on whose k, beta or decay is not
// finite leave the products, and the walk makes what it reaches NaN.  Wave w holds column
// tile w of the scores K K^T, which go to LDS for the inverse, and then block row w of T,
// transposed, whose accumulators are the triangle's operand register for register.  BACK:
// for the gradients, T both ways.
// 40960 chunks and heads of 128 keys in 260-270 us: 0.57 GB of T and gates written, and the
// substitution in one wave while three wait, which other workgroups fill.  (T written in
// three terms was 0.82 GB and 310 us; the walks split it, which costs them 2 %.)
template <typename TI, int KT, bool LOOSE, bool BACK>
__global__ __launch_bounds__(kDeltaThreads) void delta_prep_kernel(DeltaParams p) {
  using Sh = DeltaShape<TI, KT>;
  using Rows = DeltaRows<TI, KT, LOOSE>;
  constexpr int NT = Sh::kTerms;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
  float* sG = reinterpret_cast<float*>(smem_raw);  // high and low parts of G, beta
  int* bad = reinterpret_cast<int*>(sG + 3 * kChunk);
  bf16_t* sK = reinterpret_cast<bf16_t*>(sG + 4 * kChunk);
  float* sA = reinterpret_cast<float*>(sK);  // once the rows are done with: A^T
  float* sD = sA + kChunk * kTriStride;
  float* sT = sD + kChunk * kDiagStride;     // (BACK) T^T

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int64_t unit = blockIdx.x;
  const int bh = (int)blockIdx.x / p.nc, c = (int)blockIdx.x - bh * p.nc;
  const int b = bh / p.H, h = bh - b * p.H;
  const int t0 = c * kChunk, len = p.L - t0 < kChunk ? p.L - t0 : kChunk;

  typename Rows::Stage rk;
  Rows::place(rk, p.k, p, b, h / (p.H / p.G), t0, len, tid);
  rk.load(0);
  if (tid == 0) *bad = kChunk;
  float gt = 0.f, bt = 0.f;
  if (wave == 0 && lane < len) {
    const int64_t at = ((int64_t)b * p.L + t0 + lane) * p.H + h;
    gt = p.token_decay ? p.g[at] : p.g[h];
    bt = p.beta[at];
  }
  __syncthreads();
  if (wave == 0) {
    if (not_finite(bt) || !(gt < __builtin_inff())) atomicMin(bad, lane);
    if (!(gt < __builtin_inff())) gt = 0.f;
    const double d = (double)gt * 1.4426950408889634;
    const double sum = wave_prefix(d < (double)kLeastLog2 ? (double)kLeastLog2 : d);
    const double end = last_lane(sum);
    const float hi = (float)sum;
    bt = not_finite(bt) ? 0.f : bt;
    sG[lane] = hi;
    sG[kChunk + lane] = (float)(sum - (double)hi);
    sG[2 * kChunk + lane] = bt;
    float* gates = p.gates + unit * kDeltaGates;
    gates[lane] = exp2_sum(sum);
    gates[kChunk + lane] = exp2_sum(end - sum);
    gates[2 * kChunk + lane] = bt;
    if (lane == 0) gates[3 * kChunk] = exp2_sum(end);
    gates[4 * kChunk + lane] = hi;
    gates[5 * kChunk + lane] = (float)(sum - (double)hi);
  }
  static_assert(Rows::Stage::kRounds == 1, "rows in one round");
  if (rk.wild()) {
    for (int i = 0; i < Rows::Stage::kRound; ++i) {
      u4x w[Rows::Stage::kQuads];
      rk.pack(0, i, w);
      TI e[kPack];
      __builtin_memcpy(e, w, sizeof(e));
      bool wild = false;
#pragma unroll
      for (int n = 0; n < kPack; ++n) wild |= not_finite(to_f32(e[n]));
      if (wild) atomicMin(bad, rk.row(i));
    }
  }
  Rows::all(rk, sK);
  __syncthreads();
  const int first_bad = *bad;
  if (first_bad < kChunk) {
    for (int e = tid; e < (kChunk - first_bad) * Sh::kStride; e += kDeltaThreads) {
#pragma unroll
      for (int s = 0; s < NT; ++s) sK[s * Sh::kTile + first_bad * Sh::kStride + e] = 0;
    }
    __syncthreads();
  }
  if (tid == 0) p.gates[unit * kDeltaGates + 3 * kChunk + 1] = __int_as_float(first_bad);

  f4x kk[4];
#pragma unroll
  for (int rt = 0; rt < 4; ++rt) kk[rt] = f4x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = 0; n < KT; ++n) {
    bf8x bk[NT];
    row_operand<Sh>(sK, 16 * wave, n, lane, bk);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      if (rt > wave) continue;
      bf8x a[NT];
      row_operand<Sh>(sK, 16 * rt, n, lane, a);
      kk[rt] = mma_terms<NT, NT>(a, bk, kk[rt]);
    }
  }
  // decays: this lane's column, and four rows per tile
  const int mine = 16 * wave + col;
  const float hi = sG[mine], lo = sG[kChunk + mine];
#pragma unroll
  for (int rt = 0; rt < 4; ++rt) {
    if (rt > wave) continue;
    const int row = 16 * rt + 4 * g;
    const f4x rh = *reinterpret_cast<const f4x*>(sG + row);
    const f4x rl = *reinterpret_cast<const f4x*>(sG + kChunk + row);
    const f4x rb = *reinterpret_cast<const f4x*>(sG + 2 * kChunk + row);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float d = hw_exp2((hi - rh[r]) + (lo - rl[r]));
      kk[rt][r] = row + r < mine ? kk[rt][r] * d * rb[r] : 0.f;
    }
  }
  __syncthreads();  // the rows are done with
#pragma unroll
  for (int rt = 0; rt < 4; ++rt) {
    if (rt > wave) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) sA[(16 * rt + 4 * g + r) * kTriStride + mine] = kk[rt][r];
  }
  __syncthreads();
  const int64_t to = unit * kDeltaTri;
  if (wave == 0) unit_blocks(sA, sD, lane);
  __syncthreads();
  f4x x[4];
  unit_row(sA, sD, wave, lane, x);
  put_tiles<false>(x, wave, p.tri + to, lane);
  if constexpr (BACK) {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) sT[(16 * rt + 4 * g + r) * kTriStride + mine] = x[rt][r];
    __syncthreads();
    // rows of T^T: tile `wave`, columns 32 b + 4 g.., + 16
    f4x t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t[i] = *reinterpret_cast<const f4x*>(sT + mine * kTriStride + 16 * i + 4 * g);
    put_tiles<true>(t, wave, p.tri_t + to, lane);
  }
}

// ---- the walk -------------------------------------------------------------------

enum DeltaMode {
  kDeltaOut = 0,    // y
  kDeltaKeep = 1,   // each chunk's first state, and O
  kDeltaBack = 2,   // dv, each chunk's last adjoint and dV, backwards
  kDeltaSeg = 3,    // only a segment's end state from zero, and its transition
  kDeltaSegBack = 4 // only a segment's adjoint before it from zero
};

template <typename TI, int KT, int MODE>
struct DeltaLds {
  using Sh = DeltaShape<TI, KT>;
  static constexpr bool kQ = MODE != kDeltaKeep && MODE != kDeltaSeg;
  static constexpr size_t kRows = (size_t)(kQ ? 2 : 1) * Sh::kTerms * Sh::kTile;
  static constexpr size_t kTris = (size_t)(kQ ? 2 : 1) * kDeltaTerms * kDeltaTri;
  // values: strides that spread the transposing reads over the banks
  static constexpr int kValStride = kWalkCols + (Sh::kF32 ? 4 : 8);
  static constexpr size_t kVals = (size_t)kChunk * kValStride * (Sh::kF32 ? 4 : 2);
  static constexpr size_t kBytes =
      (kRows + kTris) * sizeof(bf16_t) + kVals + kDeltaGates * sizeof(float);
};

// Element `i` of a wave-uniform base and a byte offset per lane.
template <typename T>
__device__ __forceinline__ T& lane_at(T* base, int64_t i, uint32_t off) {
  return *reinterpret_cast<T*>(reinterpret_cast<char*>(base + i) + off);
}

// A triangle on its way to LDS, where it lies in terms.
struct TriStage {
  static constexpr int THREADS = kDeltaThreads, kN = kDeltaTri / 4 / THREADS;
  static_assert(kN * 4 * THREADS == kDeltaTri, "whole rounds");
  f4x v[kN];
  __device__ __forceinline__ void load(const float* from, int tid) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = reinterpret_cast<const f4x*>(from)[i * THREADS + tid];
  }
  __device__ __forceinline__ void store(bf16_t* to, int tid) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float x[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
      uint32_t w[kDeltaTerms][2];
      split_pairs<kDeltaTerms, 4>(x, w);
#pragma unroll
      for (int s = 0; s < kDeltaTerms; ++s)
        *reinterpret_cast<uint2*>(to + s * kDeltaTri + (i * THREADS + tid) * 4) =
            make_uint2(w[s][0], w[s][1]);
    }
  }
};

// Two workgroups of four waves share a CU where LDS and 256 registers suffice: the stages of a
// chunk (rows to LDS, K h, T R, U, the state's update) follow each other, and one workgroup's
// products run while the other waits.  A chunk of 128 keys and 64 columns takes 6.2 us alone
// and 4.8 us as one of two; its matrix instructions are 1.5 us of that, vector issue and LDS
// about as much again each.  Eight waves on 128 columns share rows, T and scores, but their
// barriers stop the whole CU: 8 % slower for 256 heads of 128 x 128 over 4096 tokens.
template <typename TI, int KT>
constexpr int delta_waves_per_simd() {
  if (sizeof(TI) == 4 || KT > 4) return 1;
  return 2;
}

template <typename TI, int KT, bool LOOSE, int MODE>
__global__ __launch_bounds__(kDeltaThreads) __attribute__((
    amdgpu_waves_per_eu(delta_waves_per_simd<TI, KT>(), delta_waves_per_simd<TI, KT>())))
void delta_walk_kernel(DeltaParams p) {
  constexpr int THREADS = kDeltaThreads, COLS = kWalkCols;
  using Sh = DeltaShape<TI, KT>;
  using Rows = DeltaRows<TI, KT, LOOSE>;
  using Lds = DeltaLds<TI, KT, MODE>;
  constexpr int NT = Sh::kTerms, HT = 2 * KT;  // terms of inputs; 16-row tiles
  constexpr bool BACK = MODE == kDeltaBack || MODE == kDeltaSegBack, QUERY = Lds::kQ;
  constexpr bool OUT = MODE == kDeltaOut;
  constexpr bool CARRY = MODE == kDeltaSeg;  // transitions too
  constexpr bool SEG = CARRY || MODE == kDeltaSegBack;
  constexpr bool KEEP = MODE == kDeltaKeep || MODE == kDeltaBack;
  constexpr int S = kDeltaTerms;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
  bf16_t* sK = reinterpret_cast<bf16_t*>(smem_raw);
  bf16_t* sQ = sK + NT * Sh::kTile;  // (QUERY)
  bf16_t* sT = sK + Lds::kRows;
  bf16_t* sS = sT + S * kDeltaTri;   // (QUERY)
  TI* sV = reinterpret_cast<TI*>(sT + Lds::kTris);
  float* sG = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(sV) + Lds::kVals);

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int g = lane >> 4;
  // neighbours (which read the same rows) on one XCD: workgroups go to the eight in turn
  int blk = blockIdx.x;
  {
    const int n = gridDim.x, x = blk & 7, per = n >> 3, more = n & 7;
    blk = x * per + (x < more ? x : more) + (blk >> 3);
  }
  // the state pass has columns of the transition behind those of the state
  const int all_tiles = CARRY ? p.ctiles + (32 * KT + COLS - 1) / COLS : p.ctiles;
  const int tile = blk % all_tiles;
  blk /= all_tiles;
  const int segs = SEG ? p.state_segs : p.nseg;
  const int seg = blk % segs;
  const int bh = blk / segs, b = bh / p.H, h = bh - b * p.H;
  const bool unit_state = CARRY && tile >= p.ctiles;
  const int c0 = COLS * (unit_state ? tile - p.ctiles : tile);
  const int cw = 16 * wave + (lane & 15);  // this lane's first column in the workgroup
  const int width = unit_state ? 0 : p.P - c0;  // columns with values
  const int grp = h / (p.H / p.G);
  const int64_t vstride = (int64_t)p.H * p.P;
  const int64_t vfirst = (int64_t)b * p.L * vstride + (int64_t)h * p.P + (unit_state ? 0 : c0);
  const int64_t state = (int64_t)bh * p.N * p.P;
  // chunks of this segment; segments are the same either way, counted from where the walk starts
  const int low = (BACK ? p.nseg - 1 - seg : seg) * p.seg_chunks;
  const int high = low + p.seg_chunks < p.nc ? low + p.seg_chunks : p.nc;
  const int nj = high - low;
  auto chunk_of = [&](int j) { return BACK ? high - 1 - j : low + j; };

  f4x st[HT];
#pragma unroll
  for (int i = 0; i < HT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int n = 16 * i + 4 * g + r;
      float v = 0.f;
      if constexpr (SEG) {
        v = unit_state && n == c0 + cw ? 1.f : 0.f;
      } else if (p.nseg > 1) {
        v = p.seg_state[(((int64_t)bh * p.nseg + seg) * (32 * KT) + n) * p.Pp + c0 + cw];
      } else if (p.s0 != nullptr) {
        if (cw < width && n < p.N) v = p.s0[state + (int64_t)n * p.P + c0 + cw];
      }
      st[i][r] = v;
    }

  static_assert(Rows::Stage::kRounds == 1, "rows in one round");
  typename Rows::Stage rk, rq;
  TriStage tri;
  using Vals = RowStage<TI, COLS, THREADS, LOOSE>;
  static_assert(Vals::kRounds == 1, "values in one round");
  Vals rv;
  constexpr int kGateLoads = (kDeltaGates + THREADS - 1) / THREADS;
  float gate[kGateLoads];
  int next_bad = kChunk;
  auto fetch = [&](int j) {
    const int cc = chunk_of(j), t0 = cc * kChunk, len = p.L - t0 < kChunk ? p.L - t0 : kChunk;
    const int64_t unit = (int64_t)bh * p.nc + cc;
    Rows::place(rk, p.k, p, b, grp, t0, len, tid);
    rk.load(0);
    if (QUERY) {
      Rows::place(rq, p.q, p, b, grp, t0, len, tid);
      rq.load(0);
    }
    tri.load((BACK ? p.tri_t : p.tri) + unit * kDeltaTri, tid);
#pragma unroll
    for (int i = 0; i < kGateLoads; ++i) {
      const int e = i * THREADS + tid;
      gate[i] = p.gates[unit * kDeltaGates + (e < kDeltaGates ? e : tid)];
    }
    next_bad = __float_as_int(p.gates[unit * kDeltaGates + 3 * kChunk + 1]);
    const int64_t all = (int64_t)p.B * p.L * vstride;
    rv.base = static_cast<const TI*>(BACK ? p.dy : p.v);
    rv.total = all < kPack ? kPack : all;
    rv.first = vfirst + t0 * vstride;
    rv.stride = vstride;
    rv.cols = width;
    rv.len = len;
    rv.tid = tid;
    rv.down = false;
    rv.load(0);
  };
  // A chunk's results, stored while the next one is worked on.
  f4x late[4];
  const uint32_t state_off = (uint32_t)(4 * g * p.Pp + c0 + cw) * 4u;  // of the workspace's rows
  auto leave_as = [&](auto* out, int64_t first, int len) {
    using TO = std::remove_pointer_t<decltype(out)>;
    const uint32_t off = (uint32_t)(4 * g * (uint32_t)vstride + (uint32_t)cw) * (uint32_t)sizeof(TO);
    out += first;
    if (cw >= width) return;
    if (len == kChunk) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        lane_at(out, (16 * (i >> 2) + (i & 3)) * vstride, off) = from_f32<TO>(late[i >> 2][i & 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * (i >> 2) + 4 * g + (i & 3) < len)
          lane_at(out, (16 * (i >> 2) + (i & 3)) * vstride, off) =
              from_f32<TO>(late[i >> 2][i & 3]);
    }
  };
  auto leave = [&](int cc) {
    const int t0 = cc * kChunk, len = p.L - t0 < kChunk ? p.L - t0 : kChunk;
    if (KEEP) {
      float* to = p.rows + ((int64_t)bh * p.nc + cc) * kChunk * p.Pp;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        lane_at(to, (int64_t)(16 * (i >> 2) + (i & 3)) * p.Pp, state_off) = late[i >> 2][i & 3];
    }
    const int64_t first = vfirst + t0 * vstride;
    if ((OUT || MODE == kDeltaBack) && p.out_bf16)
      leave_as(static_cast<bf16_t*>(p.out), first, len);
    else if (OUT || MODE == kDeltaBack) leave_as(static_cast<float*>(p.out), first, len);
  };
  fetch(0);

  for (int j = 0; j < nj; ++j) {
    const int cc = chunk_of(j), t0 = cc * kChunk, len = p.L - t0 < kChunk ? p.L - t0 : kChunk;
    const int64_t unit = (int64_t)bh * p.nc + cc;
    __syncthreads();  // everyone is done with the last chunk
    // tokens from the first bad one on leave the products
    const int bad = next_bad;
    rk.len = bad < len ? bad : len;
    if (!BACK) rv.len = rk.len;
    Rows::all(rk, sK);
    if (QUERY) Rows::all(rq, sQ);
    tri.store(sT, tid);
#pragma unroll
    for (int i = 0; i < kGateLoads; ++i)
      if (i * THREADS + tid < kDeltaGates) sG[i * THREADS + tid] = gate[i];
    rv.store(0, sV, Lds::kValStride);
    __syncthreads();
    // stores before the loads that the next chunk waits for, not behind them
    if (j > 0 && !SEG) leave(chunk_of(j - 1));
    if (KEEP) {
      float* to = p.states + unit * (32 * KT) * p.Pp;
#pragma unroll
      for (int i = 0; i < HT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          lane_at(to, (int64_t)(16 * i + r) * p.Pp, state_off) = st[i][r];
    }
    if (j + 1 < nj) fetch(j + 1);

    // The decayed scores of K Q^T (walking back: of Q K^T), whose accumulators are the triangle's
    // operand register for register: its six blocks of two tiles, two or three tiles per wave.
    if constexpr (QUERY) {
      static_assert(kDeltaWaves == 4, "blocks by wave");
      const int lane_now = apart(lane), col = lane_now & 15, g4 = 4 * (lane_now >> 4);
      auto block = [&](int rt, int b) {  // operand row tile, 32-block
        f4x sc[2];
        sc[0] = sc[1] = f4x{0.f, 0.f, 0.f, 0.f};
        const int mine = 16 * rt + col;
        const float hi = sG[4 * kChunk + mine], lo = sG[5 * kChunk + mine];
#pragma unroll
        for (int n = 0; n < KT; ++n) {
          bf8x bm[NT];
          row_operand<Sh>(BACK ? sK : sQ, 16 * rt, n, lane_now, bm);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = 2 * b + x;
            if (BACK ? t < rt : t > rt) continue;
            bf8x a[NT];
            row_operand<Sh>(BACK ? sQ : sK, 16 * t, n, lane_now, a);
            sc[x] = mma_terms<NT, NT>(a, bm, sc[x]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = 2 * b + x;
          if (BACK ? t < rt : t > rt) continue;
          const f4x rh = *reinterpret_cast<const f4x*>(sG + 4 * kChunk + 16 * t + g4);
          const f4x rl = *reinterpret_cast<const f4x*>(sG + 5 * kChunk + 16 * t + g4);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float e = BACK ? (rh[r] - hi) + (rl[r] - lo) : (hi - rh[r]) + (lo - rl[r]);
            sc[x][r] *= hw_exp2(e);
            if (t == rt && (BACK ? g4 + r < col : g4 + r > col)) sc[x][r] = 0.f;
          }
        }
        bf8x v[S];
        split_tiles<S>(sc[0], sc[1], v);
        const int blk2 = BACK ? tri_block_t(rt, b) : tri_block(rt, b);
#pragma unroll
        for (int x = 0; x < S; ++x)
          *reinterpret_cast<bf8x*>(sS + x * kDeltaTri + (blk2 * 64 + lane_now) * 8) = v[x];
      };
      if constexpr (BACK) {
        if (wave == 0) block(0, 0);
        else if (wave == 1) { block(0, 1); block(3, 1); }
        else if (wave == 2) { block(1, 0); block(1, 1); }
        else block(2, 1);
      } else {
        if (wave == 0) block(3, 0);
        else if (wave == 1) { block(3, 1); block(0, 0); }
        else if (wave == 2) { block(2, 0); block(2, 1); }
        else block(1, 0);
      }
    }

    // K h, and Q h, the next rows on their way
    f4x z[4], y[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      z[t] = f4x{0.f, 0.f, 0.f, 0.f};
      y[t] = f4x{0.f, 0.f, 0.f, 0.f};
    }
    {
      // two sets of operands where the registers allow it (with queries one does as well: 64K-token
      // prompt 2035 us, with two sets 2033)
      constexpr int kSets = KEEP ? 2 : 1;
      bf8x ak[kSets][4][NT], aq[kSets][4][NT];
      auto rows = [&](int n) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          row_operand<Sh>(sK, 16 * t, n, lane, ak[n % kSets][t]);
          if (OUT) row_operand<Sh>(sQ, 16 * t, n, lane, aq[n % kSets][t]);
        }
      };
      if (kSets == 2) rows(0);
#pragma unroll
      for (int n = 0; n < KT; ++n) {
        bf8x hb[S];
        split_tiles<S>(st[2 * n], st[2 * n + 1], hb);
        if (kSets == 1) rows(n);
        else if (n + 1 < KT) rows(n + 1);
        mma_tiles<NT, S, 4>(ak[n % kSets], hb, z);
        if (OUT) mma_tiles<NT, S, 4>(aq[n % kSets], hb, y);
      }
    }
    if (QUERY) __syncthreads();  // the scores are there

    // this lane's columns of the values; an infinity or a NaN of v reaches its own column from
    // its token on
    f4x vv[4];
    float odd = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (Sh::kF32) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          vv[t][r] = sV[(16 * t + 4 * g + r) * Lds::kValStride + cw];
      } else {
        typedef __attribute__((address_space(3))) s4x* lds_s4;
        const int i = lane & 15;
        const s4x q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s4)(sV + (16 * t + 4 * g + (i >> 2)) * Lds::kValStride + 16 * wave +
                     4 * (i & 3)));
#pragma unroll
        for (int r = 0; r < 4; ++r) vv[t][r] = to_f32((bf16_t)q[r]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) odd = fmaf(vv[t][r], 0.f, odd);
    }
    int limit = bad;
    if constexpr (!BACK) {
      if (!unit_state && __ballot(!(odd == 0.f))) {
        __builtin_amdgcn_sched_barrier(0);
        int first = kChunk;
#pragma unroll
        for (int i = 15; i >= 0; --i)
          if (not_finite(vv[i >> 2][i & 3])) first = 16 * (i >> 2) + 4 * g + (i & 3);
        int o = __shfl_xor(first, 16);
        first = o < first ? o : first;
        o = __shfl_xor(first, 32);
        first = o < first ? o : first;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (16 * (i >> 2) + 4 * g + (i & 3) >= first) vv[i >> 2][i & 3] = 0.f;
        limit = first < bad ? first : bad;
      }
    }
    auto gates = [&](int which, int t) {
      return *reinterpret_cast<const f4x*>(sG + which * kChunk + 16 * t + 4 * g);
    };
    // c += the triangle's (or its transpose's) product with values in terms
    auto triangle = [&](auto terms, const bf16_t* tri_in, int m, const bf8x* v, f4x* acc) {
      constexpr int NB = decltype(terms)::value;
#pragma unroll
      for (int t0 = 0; t0 < 4; t0 += 2) {  // operands of two tiles at a time
        if (BACK ? t0 >= 2 * m + 2 : t0 < 2 * m) continue;
        bf8x a[2][S];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int blk2 = BACK ? tri_block_t(t0 + t, m) : tri_block(t0 + t, m);
#pragma unroll
          for (int s = 0; s < S; ++s)
            a[t][s] =
                *reinterpret_cast<const bf8x*>(tri_in + s * kDeltaTri + blk2 * 512 + lane * 8);
        }
        mma_tiles<S, NB, 2>(a, v, acc + t0);
      }
    };
    using Three = std::integral_constant<int, S>;
    using OfInput = std::integral_constant<int, NT>;
    // state += columns of staged rows times values in terms
    auto update = [&](const bf16_t* tile_in, int m, const bf8x* v) {
      constexpr int kMost = 4, kAtOnce = NT == 1 ? (HT < kMost ? HT : kMost) : 2;
#pragma unroll
      for (int i0 = 0; i0 < HT; i0 += kAtOnce) {
        bf8x a[kAtOnce][NT];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) column_operand<Sh>(tile_in, i0 + i, m, lane, a[i]);
        mma_tiles<NT, S, kAtOnce>(a, v, st + i0);
      }
    };
    const float carry = sG[3 * kChunk];
    f4x o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = f4x{0.f, 0.f, 0.f, 0.f};
    if constexpr (!BACK) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4x e = gates(0, t);
        vv[t] -= e * z[t];
        if (OUT) y[t] *= e;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        bf8x rb[S];
        split_tiles<S>(vv[2 * m], vv[2 * m + 1], rb);
        triangle(Three(), sT, m, rb, o);
      }
      f4x u[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4x e = gates(2, t);
        u[t] = e * o[t];
      }
      if (OUT) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          bf8x ub[S];
          split_tiles<S>(u[2 * m], u[2 * m + 1], ub);
          triangle(Three(), sS, m, ub, y);
        }
      }
#pragma unroll
      for (int i = 0; i < HT; ++i) st[i] *= carry;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        bf8x ub[S];
        const f4x e0 = gates(1, 2 * m), e1 = gates(1, 2 * m + 1);
        split_tiles<S>(u[2 * m] * e0, u[2 * m + 1] * e1, ub);
        update(sK, m, ub);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (!SEG) late[t] = OUT ? y[t] : o[t];
      if (limit < len) {
#pragma unroll
        for (int i = 0; i < HT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) st[i][r] = __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (16 * (i >> 2) + 4 * g + (i & 3) >= limit)
            late[i >> 2][i & 3] = __builtin_nanf("");
      }
    } else {
      // A bad token reaches the adjoints and dV of those columns that anything behind it reaches
      bool reached = false;
      if (bad < len) {  // (uniform)
        bool some = false;
#pragma unroll
        for (int i = 0; i < HT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) some |= !(st[i][r] == 0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          some |= 16 * (i >> 2) + 4 * g + (i & 3) >= bad && !(vv[i >> 2][i & 3] == 0.f);
        const uint64_t rows = __ballot(some);
        reached = ((rows | rows >> 16 | rows >> 32 | rows >> 48) >> (lane & 15) & 1) != 0;
      }
      // dU = w K a + S^T dY, dV = T^T (beta dU)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4x e = gates(1, t);
        z[t] *= e;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        bf8x db[NT];
        split_tiles<NT>(vv[2 * m], vv[2 * m + 1], db);
        triangle(OfInput(), sS, m, db, z);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f4x e = gates(2, t);
        z[t] *= e;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        bf8x ub[S];
        split_tiles<S>(z[2 * m], z[2 * m + 1], ub);
        triangle(Three(), sT, m, ub, o);
      }
#pragma unroll
      for (int i = 0; i < HT; ++i) st[i] *= carry;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        bf8x yb[S], vb[S];
        const f4x e0 = gates(0, 2 * m), e1 = gates(0, 2 * m + 1);
        split_tiles<S>(vv[2 * m] * e0, vv[2 * m + 1] * e1, yb);
        split_tiles<S>(o[2 * m] * -e0, o[2 * m + 1] * -e1, vb);
        update(sQ, m, yb);
        update(sK, m, vb);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) late[t] = o[t];
      if (reached) {
        const float nan = __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < HT; ++i) st[i] = f4x{nan, nan, nan, nan};
#pragma unroll
        for (int t = 0; t < 4; ++t) late[t] = f4x{nan, nan, nan, nan};
      }
    }
  }
  if (!SEG) leave(chunk_of(nj - 1));
  if constexpr (SEG) {
    const int64_t at = (int64_t)bh * p.nseg + seg;
    const int ld = unit_state ? 32 * KT : p.Pp;
    float* to = unit_state ? p.seg_carry + at * (32 * KT) * (32 * KT) : p.seg_state + at * (32 * KT) * p.Pp;
    if (c0 + cw >= ld) return;
#pragma unroll
    for (int i = 0; i < HT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        to[(int64_t)(16 * i + 4 * g + r) * ld + c0 + cw] = st[i][r];
  } else if (p.s_final != nullptr && seg == p.nseg - 1) {
#pragma unroll
    for (int i = 0; i < HT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = 16 * i + 4 * g + r;
        if (cw < width && n < p.N) p.s_final[state + (int64_t)n * p.P + c0 + cw] = st[i][r];
      }
  }
}

// ---- the other gradients, every chunk for itself --------------------------------

struct DeltaGradParams {
  const void *q, *k, *dy;
  const float *g, *beta;
  int B, L, H, G, N, P, Pp;
  int token_decay, nc;
  int parts, heads;                // workgroups of a group of heads that share q and k, heads each
  const float* gates;              // [kDeltaGates] of each chunk and head, for its first bad token
  const float *states, *adjoints;  // [N', P'] before and behind each chunk
  const float *o, *dv;             // [64, P']
  void *dq, *dk;                   // [B, L, G, parts, N]
  int grad_bf16;
  float* dg;                       // [B, L, H], or null
  double* part;                    // sums of dg per chunk (a decay per head), or null
  float* dbeta;                    // [B, L, H]
};

// Sum over the 16 lanes of a row, on each of them.
__device__ __forceinline__ float row_sum(float v) {
  v += xor_lane<1>(v, 0);
  v += xor_lane<2>(v, 0);
  v += xor_lane<4>(v, 0);
  return v + xor_lane<8>(v, 0);
}
// Sum over the four lanes of a column.
__device__ __forceinline__ float column_sum(float v) {
  v = xchg_add<32>(v, v);
  return xchg_add<16>(v, v);
}

constexpr int kGradThreads = 512;

// LDS of the gradients' kernel: K and Q; 32 columns of dY, O, dV, h and a in terms (h and a in
// turn where they do not fit together), later the slopes of the scores; vectors.
template <typename TI, int KT>
struct GradLds {
  using Sh = DeltaShape<TI, KT>;
  static constexpr int S = kDeltaTerms;
  static constexpr size_t kRows = 2 * (size_t)Sh::kTerms * Sh::kTile * sizeof(bf16_t);
  static constexpr size_t kToken = (size_t)kChunk * 32 * sizeof(bf16_t);  // of a term
  static constexpr size_t kState = (size_t)Sh::kRows * 32 * sizeof(bf16_t);
  static constexpr size_t kTokens = (Sh::kTerms + 2 * S) * kToken;
  static constexpr size_t kVectors = 16 * kChunk * sizeof(float);
  static constexpr bool kTogether =
      kRows + kTokens + 2 * S * kState + kVectors <= 160 * 1024;
  static constexpr size_t kStage = kTokens + (kTogether ? 2 : 1) * S * kState;
  static constexpr size_t kSlopes = (size_t)kChunk * kTriStride * sizeof(float);
  static constexpr size_t kBytes = kRows + (kStage > kSlopes ? kStage : kSlopes) + kVectors;
};

// With F = dY O^T and E = dV O^T (pairs s <= t and s < t):
//   dQ = e^G dY h^T + (F D beta) K
//   dK = beta w O a^T - e^G dV h^T + (F D beta)^T Q - (E D beta) K - (E D beta)^T K
//   dbeta_s = sum_t (q_t . k_s) D F - (k_t . k_s) D E + w_s k_s . (O a^T)_s
// and dg_t is the sum of everything that spans t: the pairs s < t <= r of
// beta_s D (q_r . k_s F - k_r . k_s E), what tokens r >= t read of h, what later
// chunks read of tokens s < t, and e^{G_end} <h, a>.  The pairs' sum is taken up from its
// differences between neighbours (column sum less row sum) from the chunk's start or the
// last cleared state, in 64 bits.
//
// One workgroup per chunk and `heads` heads that share its q and k, whose gradients stay in
// registers from head to head.  Wave (rt, half) takes the 16 tokens of tile rt by half
// of the keys; waves of half 0 also take row tile rt of F, of half 1 of E.  dY, O, dV, h
// and a pass through LDS 32 columns at a time, split into terms once for all waves, the next
// ones on their way in registers.
// 2 x 4096 tokens, 32 heads of 128 x 128 over 4 key heads: 331 us, of which a head's four
// column blocks are 60 % (the three-term products, one workgroup per CU for want of LDS and
// registers), slopes 10 %, their products with K and Q 10 % and the sums behind them, in one
// wave, 20 %.  Reading states, adjoints, O and dV in fp32 (805 MB there) alone would take 152 us
// at the copy rate.  Two workgroups per CU (128 registers) spill: 60 % slower for 4 x 2048
// tokens of 24 heads of 64 x 64, which take 163 us.
// From the first bad token on (whose k, beta or decay is not finite) gradients are NaN; earlier
// tokens see the chunk without it, and the NaN that the walk back leaves in dV and a where it
// reaches them.
template <typename TI, int KT, bool LOOSE>
__global__ __launch_bounds__(kGradThreads) void delta_grad_kernel(DeltaGradParams p) {
  using Sh = DeltaShape<TI, KT>;
  using Lds = GradLds<TI, KT>;
  using Rows = DeltaRows<TI, KT, LOOSE>;
  static_assert(kGradThreads == 2 * kDeltaThreads, "half of the threads for K, half for Q");
  constexpr int NT = Sh::kTerms, S = kDeltaTerms, N = Sh::kRows;
  constexpr int kTokenTerm = kChunk * 32, kStateTerm = N * 32;  // values of a term
  constexpr int kStatePacks = (N * 4 + kGradThreads - 1) / kGradThreads;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_raw[];
  bf16_t* sK = reinterpret_cast<bf16_t*>(smem_raw);
  bf16_t* sQ = sK + NT * Sh::kTile;
  bf16_t* sY = sQ + NT * Sh::kTile;
  bf16_t* sO = sY + NT * kTokenTerm;
  bf16_t* sV = sO + S * kTokenTerm;
  bf16_t* sH = sV + S * kTokenTerm;
  bf16_t* sB = Lds::kTogether ? sH + S * kStateTerm : sH;
  // F D beta on and below the diagonal, (E D beta)^T above it
  float* sM = reinterpret_cast<float*>(sY);
  float* vec = reinterpret_cast<float*>(smem_raw + Lds::kBytes - Lds::kVectors);
  float *gHi = vec, *gLo = vec + 64, *gRead = vec + 128, *gWrite = vec + 192, *gBeta = vec + 256;
  float *row = vec + 320, *diag = vec + 384;
  float *seen = vec + 448, *wrote = vec + 576;  // [2][64]: halves of the keys
  float* cols = vec + 704;                      // [4][64]: row tiles
  float* thru = vec + 960;                      // [8]: waves
  static_assert(Lds::kVectors >= 968 * sizeof(float), "the vectors");

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int rt = wave & 3, half = wave >> 2;
  int blk = (int)blockIdx.x;
  const int part = blk % p.parts;
  blk /= p.parts;
  const int c = blk % p.nc;
  blk /= p.nc;
  const int grp = blk % p.G, b = blk / p.G;
  const int t0 = c * kChunk, len = p.L - t0 < kChunk ? p.L - t0 : kChunk;
  const int h0 = grp * (p.H / p.G) + part * p.heads;
  const int blocks = (p.P + 31) / 32;

  // K and Q, by half of the threads each
  {
    DeltaParams rp = {};
    rp.G = p.G;
    rp.N = p.N;
    rp.B = p.B;
    rp.L = p.L;
    typename Rows::Stage st;
    Rows::place(st, half ? p.q : p.k, rp, b, grp, t0, len, tid & (kDeltaThreads - 1));
    st.load(0);
    static_assert(Rows::Stage::kRounds == 1, "rows in one round");
    if (!half && st.wild()) st.drop_wild();
    Rows::all(st, half ? sQ : sK);
  }

  // The next 32 columns: a pack of eight of O or dV and of dY per thread, and of h and a.
  struct Pack8 {
    f4x a, b;
  };
  const int tok = tid & 255, trow = tok >> 2, tslot = tok & 3;
  const int64_t vstride = (int64_t)p.H * p.P;
  Pack8 ro, rh[kStatePacks], ra[kStatePacks];
  Pack<TI> ry;
  float gt = 0.f, bt = 0.f, next_g = 0.f, next_b = 0.f;
  int bad = kChunk, next_bad = kChunk;
  auto load8 = [](const float* at) {
    Pack8 v;
    v.a = *reinterpret_cast<const f4x*>(at);
    v.b = *reinterpret_cast<const f4x*>(at + 4);
    return v;
  };
  auto fetch = [&](int i, int m) {
    const int64_t bh = (int64_t)b * p.H + h0 + i, unit = bh * p.nc + c;
    const int cc = 32 * m + 8 * tslot;
    ro = load8((half ? p.dv : p.o) + (unit * kChunk + trow) * p.Pp + cc);
    if (half == 0) {
      const TI* dy = static_cast<const TI*>(p.dy) + ((int64_t)b * p.L + t0) * vstride +
                     (int64_t)(h0 + i) * p.P;
      const int n = trow < len ? p.P - cc : 0;
      if (LOOSE) ry = load_pack(dy + (n > 0 ? trow * vstride + cc : 0), n);
      else ry = load_pack(dy + (n > 0 ? trow * vstride + cc : 0), kPack);
    }
#pragma unroll
    for (int k = 0; k < kStatePacks; ++k) {
      const int e = k * kGradThreads + tid;
      const int64_t at = (unit * N + (e < N * 4 ? e >> 2 : 0)) * p.Pp + 32 * m + 8 * (e & 3);
      rh[k] = load8(p.states + at);
      ra[k] = load8(p.adjoints + at);
    }
    if (m == 0) next_bad = __float_as_int(p.gates[unit * kDeltaGates + 3 * kChunk + 1]);
    if (m == 0 && wave == 0 && lane < len) {
      const int64_t at = ((int64_t)b * p.L + t0 + lane) * p.H + h0 + i;
      next_g = p.token_decay ? p.g[at] : p.g[h0 + i];
      next_b = p.beta[at];
    }
  };
  auto place = [](int r, int slot) { return ((r >> 4) * 64 + slot * 16 + (r & 15)) * 8; };
  auto put = [&](const Pack8& v, bf16_t* to, int term) {
    bf8x t[S];
    split_tiles<S>(v.a, v.b, t);
#pragma unroll
    for (int s = 0; s < S; ++s) *reinterpret_cast<bf8x*>(to + s * term) = t[s];
  };
  auto put_states = [&](const Pack8* v, bf16_t* to) {
#pragma unroll
    for (int k = 0; k < kStatePacks; ++k) {
      const int e = k * kGradThreads + tid;
      if (N * 4 % kGradThreads == 0 || e < N * 4) put(v[k], to + place(e >> 2, e & 3), kStateTerm);
    }
  };
  auto operand = [&](const bf16_t* from, int tile, int term, int s) {
    return *reinterpret_cast<const bf8x*>(from + s * term + (tile * 64 + lane) * 8);
  };

  f4x dq[KT], dk[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) {
    dq[k] = f4x{0.f, 0.f, 0.f, 0.f};
    dk[k] = f4x{0.f, 0.f, 0.f, 0.f};
  }
  fetch(0, 0);
  __syncthreads();
  // scores of row tile rt, before the decays: Q K^T, or (half 1) K K^T
  f4x sc[4];
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) sc[ct] = f4x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = 0; n < KT; ++n) {
    bf8x a[NT];
    row_operand<Sh>(half ? sK : sQ, 16 * rt, n, lane, a);
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      if (ct > rt) continue;
      bf8x bk[NT];
      row_operand<Sh>(sK, 16 * ct, n, lane, bk);
      sc[ct] = mma_terms<NT, NT>(a, bk, sc[ct]);
    }
  }

  for (int i = 0; i < p.heads; ++i) {
    const int h = h0 + i;
    const int64_t bh = (int64_t)b * p.H + h, unit = bh * p.nc + c;
    // what this wave's tokens read of h, erase of it and write into a; F or E
    f4x reads[KT], erased[KT], written[KT], fe[4];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      reads[k] = f4x{0.f, 0.f, 0.f, 0.f};
      erased[k] = f4x{0.f, 0.f, 0.f, 0.f};
      written[k] = f4x{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) fe[ct] = f4x{0.f, 0.f, 0.f, 0.f};
    float through = 0.f;
    for (int m = 0; m < blocks; ++m) {
      __syncthreads();  // everyone is done with the last ones
      if (m == 0) {
        bad = next_bad;
        gt = lane < bad ? next_g : 0.f;
        bt = lane < bad ? next_b : 0.f;
        if (wave == 0) {
          const double d = (double)gt * 1.4426950408889634;
          const double sum = wave_prefix(d < (double)kLeastLog2 ? (double)kLeastLog2 : d);
          const double end = last_lane(sum);
          const float hi = (float)sum;
          gHi[lane] = hi;
          gLo[lane] = (float)(sum - (double)hi);
          gRead[lane] = exp2_sum(sum);
          gWrite[lane] = exp2_sum(end - sum);
          gBeta[lane] = bt;
        }
      }
      if (half == 0 && trow >= bad) ro.a = ro.b = f4x{0.f, 0.f, 0.f, 0.f};
      put(ro, (half ? sV : sO) + place(trow, tslot), kTokenTerm);
      if (half == 0) {
        const bool in = LOOSE || (trow < len && 32 * m + 8 * tslot < p.P);
        if constexpr (Sh::kF32) {
          Pack8 v;
          __builtin_memcpy(&v, &ry, sizeof(v));
          if (!in) v.a = v.b = f4x{0.f, 0.f, 0.f, 0.f};
          put(v, sY + place(trow, tslot), kTokenTerm);
        } else {
          u4x v = __builtin_bit_cast(u4x, ry);
          if (!in) v = u4x{0, 0, 0, 0};
          *reinterpret_cast<u4x*>(sY + place(trow, tslot)) = v;
        }
      }
      put_states(rh, sH);
      if (Lds::kTogether) put_states(ra, sB);
#pragma unroll
      for (int k = 0; k < kStatePacks; ++k) {
        if (N * 4 % kGradThreads != 0 && k * kGradThreads + tid >= N * 4) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          through = fmaf(rh[k].a[e], ra[k].a[e], fmaf(rh[k].b[e], ra[k].b[e], through));
      }
      __syncthreads();
      const bool more = m + 1 < blocks || i + 1 < p.heads;
      auto ahead = [&] {
        if (more) fetch(m + 1 < blocks ? i : i + 1, m + 1 < blocks ? m + 1 : 0);
      };
      if (Lds::kTogether) ahead();

      bf8x ay[NT], av[S], ao[S];
#pragma unroll
      for (int s = 0; s < NT; ++s) ay[s] = operand(sY, rt, kTokenTerm, s);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        av[s] = operand(sV, rt, kTokenTerm, s);
        ao[s] = operand(sO, rt, kTokenTerm, s);
      }
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) {
        if (ct > rt) continue;
        bf8x bo[S];
#pragma unroll
        for (int s = 0; s < S; ++s) bo[s] = operand(sO, ct, kTokenTerm, s);
        if (half) fe[ct] = mma_terms<S, S>(av, bo, fe[ct]);
        else fe[ct] = mma_terms<NT, S>(ay, bo, fe[ct]);
      }
      // two tiles of keys at a time (four spill), a pair of terms for both in turn
      constexpr int kAtOnce = KT < 2 ? KT : 2;
      auto tiles = [&](auto na, const bf8x* a, const bf8x (*v)[S], f4x* acc) {
        constexpr int NA = decltype(na)::value;
#pragma unroll
        for (int n = S - 1; n >= 0; --n)
#pragma unroll
          for (int x = 0; x < NA; ++x)
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
              if (n - x >= 0) acc[k] = mma16(a[x], v[k][n - x], acc[k]);
      };
      using Three = std::integral_constant<int, S>;
      using OfInput = std::integral_constant<int, NT>;
#pragma unroll
      for (int k0 = 0; k0 < KT; k0 += kAtOnce) {
        bf8x v[kAtOnce][S];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
          for (int s = 0; s < S; ++s) v[k][s] = operand(sH, half * KT + k0 + k, kStateTerm, s);
        tiles(OfInput(), ay, v, reads + k0);
        tiles(Three(), av, v, erased + k0);
      }
      if (!Lds::kTogether) {
        __syncthreads();
        put_states(ra, sB);
        ahead();
        __syncthreads();
      }
#pragma unroll
      for (int k0 = 0; k0 < KT; k0 += kAtOnce) {
        bf8x v[kAtOnce][S];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
          for (int s = 0; s < S; ++s) v[k][s] = operand(sB, half * KT + k0 + k, kStateTerm, s);
        tiles(Three(), ao, v, written + k0);
      }
    }
    through = wave_sum64(through);
    if (lane == 0) thru[wave] = through;
    __syncthreads();  // the columns are done with: slopes in their place

    // (addresses from here on are made anew for each head: kept over the loop they spill, and
    // a load of a spilled one waits for the next head's columns on their way)
    {
      const int lane_now = apart(lane), g = lane_now >> 4, col = lane_now & 15;

      {
        float rs[4] = {}, cs[4];
        const int t = 16 * rt + 4 * g;
        const f4x ht = *reinterpret_cast<const f4x*>(gHi + t);
        const f4x lt = *reinterpret_cast<const f4x*>(gLo + t);
        // pairs in tiles below the diagonal are all seen
        auto slopes = [&](int ct, auto whole) {
          constexpr bool ALL = decltype(whole)::value;
          const int s = 16 * ct + col;
          const float bs = gBeta[s], hs = gHi[s], ls = gLo[s];
          float sum = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float d = fe[ct][r] * hw_exp2((ht[r] - hs) + (lt[r] - ls));
            const float y = d * sc[ct][r];
            const float x = ALL || s < t + r ? y : 0.f;
            // the other triangle's places of the diagonal's tile are the other half's
            float* to = half ? sM + s * kTriStride + t + r : sM + (t + r) * kTriStride + s;
            if (ALL || s < t + r || (half == 0 && s == t + r)) *to = d * bs;
            if (!ALL && half == 0 && s == t + r) diag[s] = y;
            sum += x;
            rs[r] = fmaf(x, bs, rs[r]);
          }
          return column_sum(sum);
        };
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
          cs[ct] = ct < rt ? slopes(ct, std::true_type())
                           : ct == rt ? slopes(ct, std::false_type()) : 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) rs[r] = row_sum(rs[r]);
        if (half == 0) {
          if (g == 0) {
#pragma unroll
            for (int ct = 0; ct < 4; ++ct) cols[rt * 64 + 16 * ct + col] = cs[ct];
          }
          if (col == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) row[16 * rt + 4 * g + r] = rs[r];
          }
        }
        __syncthreads();
        if (half) {  // less those of E
          if (g == 0) {
#pragma unroll
            for (int ct = 0; ct < 4; ++ct) cols[rt * 64 + 16 * ct + col] -= cs[ct];
          }
          if (col == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) row[16 * rt + 4 * g + r] -= rs[r];
          }
        }
      }
      auto element = [&](const bf16_t* tile, int t, int n) {
        const bf16_t* at = tile + Sh::place(t, n & ~3) + (n & 3);
        float v = to_f32(at[0]);
#pragma unroll
        for (int s = 1; s < NT; ++s) v += to_f32(at[s * Sh::kTile]);
        return v;
      };
      const f4x er = *reinterpret_cast<const f4x*>(gRead + 16 * rt + 4 * g);
      const f4x ew = *reinterpret_cast<const f4x*>(gWrite + 16 * rt + 4 * g);
      const f4x eb = *reinterpret_cast<const f4x*>(gBeta + 16 * rt + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * rt + 4 * g + r;
        float x = 0.f, w = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const int n = 16 * (half * KT + k) + col;
          const float kn = element(sK, t, n), qn = element(sQ, t, n);
          x += qn * reads[k][r] - kn * erased[k][r];
          w = fmaf(kn, written[k][r], w);
        }
        x = row_sum(x) * er[r];
        w = row_sum(w) * ew[r];
        if (col == 0) {
          seen[half * 64 + t] = x;
          wrote[half * 64 + t] = w;
        }
      }
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        dq[k] += reads[k] * er;
        dk[k] += written[k] * (ew * eb) - erased[k] * er;
        if (bad < len) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (16 * rt + 4 * g + r >= bad) dq[k][r] = dk[k][r] = __builtin_nanf("");
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int t = 16 * rt + col;
        float fd[8], both[8], ft[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int s = 32 * m + 16 * (e >> 2) + 4 * g + (e & 3);
          const float across = sM[t * kTriStride + s], down = sM[s * kTriStride + t];
          fd[e] = s <= t ? across : 0.f;
          ft[e] = s >= t ? down : 0.f;
          both[e] = s == t ? 0.f : s < t ? -down : -across;
        }
        bf8x af[S], ae[S], at[S];
        split_values<S>(fd, af);
        split_values<S>(both, ae);
        split_values<S>(ft, at);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          bf8x bk[NT], bq[NT];
          column_operand<Sh>(sK, half * KT + k, m, lane_now, bk);
          column_operand<Sh>(sQ, half * KT + k, m, lane_now, bq);
          dq[k] = mma_terms<S, NT>(af, bk, dq[k]);
          dk[k] = mma_terms<S, NT>(ae, bk, dk[k]);
          dk[k] = mma_terms<S, NT>(at, bq, dk[k]);
        }
      }
      __syncthreads();
      if (wave == 0) {
        const float down = cols[lane] + cols[64 + lane] + cols[128 + lane] + cols[192 + lane];
        const float wr = wrote[lane] + wrote[64 + lane];
        const int64_t at = ((int64_t)b * p.L + t0 + lane) * p.H + h;
        if (lane < len) p.dbeta[at] = lane < bad ? down + diag[lane] + wr : __builtin_nanf("");
        const bool clear = lane < len && hw_exp2(gt * kLog2e) == 0.f;
        const double slope = (double)bt * down - (double)row[lane];
        const double upto = wave_prefix(slope) - slope;  // of the tokens before
        const uint64_t mask = __ballot(clear) & (~0ull >> (63 - lane));
        const int from = mask != 0 ? 63 - __clzll((long long)mask) : 0;
        const double base = __shfl(upto, from);
        const double sn = (double)seen[lane] + seen[64 + lane], wb = (double)bt * wr;
        const double all_seen = wave_prefix(sn), all_wrote = wave_prefix(wb);
        double ha = 0.0;
#pragma unroll
        for (int w = 0; w < kGradThreads / 64; ++w) ha += thru[w];
        double dg = (upto - base) + (last_lane(all_seen) - all_seen + sn) + (all_wrote - wb) +
                    (double)exp2_sum((double)gHi[63] + (double)gLo[63]) * ha;
        if (lane >= bad) dg = __builtin_nan("");
        if (clear || lane >= len) dg = 0.0;
        if (p.dg != nullptr && lane < len) p.dg[at] = (float)dg;
        if (p.part != nullptr) {
          dg = wave_prefix(dg);
          if (lane == 63) p.part[unit] = dg;
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < KT; ++k) {
    const int n = 16 * (half * KT + k) + col;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * rt + 4 * g + r;
      if (t < len && n < p.N) {
        const int64_t to =
            ((((int64_t)b * p.L + t0 + t) * p.G + grp) * p.parts + part) * p.N + n;
        if (p.grad_bf16) {
          static_cast<bf16_t*>(p.dq)[to] = from_f32<bf16_t>(dq[k][r]);
          static_cast<bf16_t*>(p.dk)[to] = from_f32<bf16_t>(dk[k][r]);
        } else {
          static_cast<float*>(p.dq)[to] = dq[k][r];
          static_cast<float*>(p.dk)[to] = dk[k][r];
        }
      }
    }
  }
}

// ---- launches -------------------------------------------------------------------

template <typename TI, int KT, bool LOOSE, bool BACK>
int delta_prep(const DeltaParams& p, hipStream_t s) {
  constexpr size_t lds = delta_prep_lds<TI, KT>(BACK);
  static_assert(lds <= 160 * 1024, "a CU's LDS");
  allow_dynamic_lds(delta_prep_kernel<TI, KT, LOOSE, BACK>, lds);
  hipLaunchKernelGGL((delta_prep_kernel<TI, KT, LOOSE, BACK>),
                     dim3((unsigned)((int64_t)p.B * p.H * p.nc)), dim3(kDeltaThreads), lds, s, p);
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

template <typename TI, int KT, bool LOOSE, int MODE>
int delta_walk(const DeltaParams& p, hipStream_t s) {
  constexpr size_t lds = DeltaLds<TI, KT, MODE>::kBytes;
  static_assert(lds <= 160 * 1024, "a CU's LDS");
  const int tiles = p.ctiles + (MODE == kDeltaSeg ? (32 * KT + kWalkCols - 1) / kWalkCols : 0);
  const int segs = MODE >= kDeltaSeg ? p.state_segs : p.nseg;
  allow_dynamic_lds(delta_walk_kernel<TI, KT, LOOSE, MODE>, lds);
  hipLaunchKernelGGL((delta_walk_kernel<TI, KT, LOOSE, MODE>),
                     dim3((unsigned)((int64_t)p.B * p.H * segs * tiles)), dim3(kDeltaThreads), lds,
                     s, p);
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

template <typename TI, int KT, bool LOOSE>
int delta_grad(const DeltaGradParams& p, hipStream_t s) {
  constexpr size_t lds = GradLds<TI, KT>::kBytes;
  static_assert(lds <= 160 * 1024, "a CU's LDS");
  allow_dynamic_lds(delta_grad_kernel<TI, KT, LOOSE>, lds);
  hipLaunchKernelGGL((delta_grad_kernel<TI, KT, LOOSE>),
                     dim3((unsigned)((int64_t)p.B * p.G * p.nc * p.parts)), dim3(kGradThreads), lds,
                     s, p);
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

enum DeltaPhase {
  kPhasePrep, kPhasePrepBack, kPhaseOut, kPhaseKeep, kPhaseBack, kPhaseSeg, kPhaseSegBack
};

template <typename TI, int KT, bool LOOSE>
int delta_phase(const DeltaParams& p, int phase, hipStream_t s) {
  switch (phase) {
    case kPhasePrep: return delta_prep<TI, KT, LOOSE, false>(p, s);
    case kPhasePrepBack: return delta_prep<TI, KT, LOOSE, true>(p, s);
    case kPhaseOut:
      return delta_walk<TI, KT, LOOSE, kDeltaOut>(p, s);
    case kPhaseKeep: return delta_walk<TI, KT, LOOSE, kDeltaKeep>(p, s);
    case kPhaseBack: return delta_walk<TI, KT, LOOSE, kDeltaBack>(p, s);
    case kPhaseSeg: return delta_walk<TI, KT, LOOSE, kDeltaSeg>(p, s);
    default: return delta_walk<TI, KT, LOOSE, kDeltaSegBack>(p, s);
  }
}

// First states of the segments (two at least), h(i + 1) = M_i h(i) + end(i), from the state pass's
// transitions M (walking back: their transposes) and ends, in place.  Four waves take the
// rows of 16 columns of one state in turn of 16-row tiles, in fp32 on the matrix units; the next
// transition is on its way while one is applied.  Bound by its chain: 2.5 to 3 us per segment of
// 128 x 128 (25 segments of 40 heads of 64 columns in 73 us); of 256 x 256 9.8 us, and walking
// back, where the operands spill, 54.  A transition that is not finite (a bad token
// in the segment, or growth beyond fp32) leaves a column that is all zero so: 0 * NaN.
template <int KT, bool BACK>
__global__ __launch_bounds__(kDeltaThreads, 1) void delta_carry_kernel(DeltaParams p) {
  constexpr int N = 32 * KT, HT = 2 * KT, kMine = (HT + 3) / 4, kStride = N + 4;
  constexpr int kPart = KT > 4 ? HT / 2 : HT;  // tiles of a row on their way at once
  __shared__ __attribute__((aligned(16))) float sH[2][16 * kStride];  // [column][row]
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int tiles = p.Pp / 16;
  const int64_t bh = blockIdx.x / tiles;
  const int c = (int)(blockIdx.x % tiles) * 16 + col;
  // (waves without a tile do the work of tile 0 again and keep nothing)
  auto tile = [&](int k) { return wave + 4 * k < HT ? wave + 4 * k : 0; };
  auto mine = [&](int k) { return wave + 4 * k < HT; };
  f4x h[kMine], end[kMine], own_end[kMine], m[kMine][kPart];
  auto load_end = [&](int s) {
    const float* st = p.seg_state + (bh * p.nseg + s) * N * p.Pp + c;
#pragma unroll
    for (int k = 0; k < kMine; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) end[k][r] = st[(int64_t)(16 * tile(k) + 4 * g + r) * p.Pp];
  };
  auto load_part = [&](int s, int part) {
    // the transition over the same tokens, made by the forward state pass
    const float* from = p.seg_carry + (bh * p.nseg + (BACK ? p.nseg - 1 - s : s)) * N * N;
#pragma unroll
    for (int k = 0; k < kMine; ++k)
#pragma unroll
      for (int n = 0; n < kPart; ++n) {
        const int nn = 16 * (part * kPart + n) + 4 * g;
        if (BACK) {
#pragma unroll
          for (int r = 0; r < 4; ++r) m[k][n][r] = from[(nn + r) * N + 16 * tile(k) + col];
        } else {
          m[k][n] = *reinterpret_cast<const f4x*>(from + (16 * tile(k) + col) * N + nn);
        }
      }
  };
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    h[k] = f4x{0.f, 0.f, 0.f, 0.f};
    if (p.s0 != nullptr) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = 16 * tile(k) + 4 * g + r;
        if (c < p.P && n < p.N) h[k][r] = p.s0[(bh * p.N + n) * p.P + c];
      }
    }
  }
  load_end(0);
  load_part(0, 0);
  for (int s = 0; s < p.nseg; ++s) {
    float* st = p.seg_state + (bh * p.nseg + s) * N * p.Pp + c;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      if (!mine(k)) continue;
      *reinterpret_cast<f4x*>(sH[s & 1] + col * kStride + 16 * tile(k) + 4 * g) = h[k];
#pragma unroll
      for (int r = 0; r < 4; ++r) st[(int64_t)(16 * tile(k) + 4 * g + r) * p.Pp] = h[k][r];
    }
    if (s + 1 == p.nseg) break;
    __syncthreads();
    f4x a[kMine][kPart];
#pragma unroll
    for (int k = 0; k < kMine; ++k) h[k] = own_end[k] = end[k];
    const bool more = s + 2 < p.nseg;
#pragma unroll
    for (int part = 0; part < HT / kPart; ++part) {
#pragma unroll
      for (int k = 0; k < kMine; ++k)
#pragma unroll
        for (int n = 0; n < kPart; ++n) a[k][n] = m[k][n];
      if (part + 1 < HT / kPart) load_part(s, part + 1);
      else if (more) {
        load_end(s + 1);
        load_part(s + 1, 0);
      }
#pragma unroll
      for (int n = 0; n < kPart; ++n) {
        const f4x b = *reinterpret_cast<const f4x*>(sH[s & 1] + col * kStride +
                                                    16 * (part * kPart + n) + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int k = 0; k < kMine; ++k) h[k] = mma16(a[k][n][r], b[r], h[k]);
      }
    }
    bool wild = false;
#pragma unroll
    for (int k = 0; k < kMine; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) wild |= not_finite(h[k][r]);
    if (__ballot(wild)) {
      bool some = false;
      for (int n = 4 * g; n < N; n += 16) {
        const f4x b = *reinterpret_cast<const f4x*>(sH[s & 1] + col * kStride + n);
        some |= !(b[0] == 0.f && b[1] == 0.f && b[2] == 0.f && b[3] == 0.f);
      }
      const uint64_t rows = __ballot(some);
      if (((rows | rows >> 16 | rows >> 32 | rows >> 48) >> col & 1) == 0) {
#pragma unroll
        for (int k = 0; k < kMine; ++k) h[k] = own_end[k];
      }
    }
  }
}

template <int KT, bool BACK>
int delta_carry(const DeltaParams& p, hipStream_t s) {
  hipLaunchKernelGGL((delta_carry_kernel<KT, BACK>),
                     dim3((unsigned)((int64_t)p.B * p.H * (p.Pp / 16))), dim3(kDeltaThreads), 0, s,
                     p);
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

// One pair per dtype and padded row size.
#define SWIMBA_DELTA_DECL(name)                                       \
  int name(const DeltaParams& p, int phase, hipStream_t s);           \
  int name##_grad(const DeltaGradParams& p, hipStream_t s);
SWIMBA_DELTA_DECL(delta_bf16_32)
SWIMBA_DELTA_DECL(delta_bf16_64)
SWIMBA_DELTA_DECL(delta_bf16_128)
SWIMBA_DELTA_DECL(delta_bf16_256)
SWIMBA_DELTA_DECL(delta_f32_32)
SWIMBA_DELTA_DECL(delta_f32_64)
SWIMBA_DELTA_DECL(delta_f32_128)
#undef SWIMBA_DELTA_DECL

#define SWIMBA_DELTA_DEFINE(name, TI, KT)                                           \
  int name(const DeltaParams& p, int phase, hipStream_t s) {                        \
    return p.N % kPack != 0 || p.P % kPack != 0 ? delta_phase<TI, KT, true>(p, phase, s) \
                            : delta_phase<TI, KT, false>(p, phase, s);              \
  }                                                                                 \
  int name##_grad(const DeltaGradParams& p, hipStream_t s) {                        \
    return p.N % kPack != 0 || p.P % kPack != 0 ? delta_grad<TI, KT, true>(p, s)    \
                                                : delta_grad<TI, KT, false>(p, s);  \
  }

}  // namespace swimba
