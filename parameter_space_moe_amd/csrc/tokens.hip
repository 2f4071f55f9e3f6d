// Tokens sorted by expert, copied out to the experts' rows, and brought back
// weighted by the gates, with the gradients of the way back.
//
// Slot s = t * k + j is token t's j-th choice.  The sort is a stable counting
// sort over at most 64 experts: every place is (slots of smaller experts) +
// (earlier slots of the same expert), so it does not depend on timing.  All
// of these move bytes: nothing is computed that a copy would not hide.
#include "pack.hpp"
#include "swimba_internal.hpp"

namespace swimba {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;

struct SortParams {
  const int32_t* idx;
  int32_t *order, *pos, *offsets;
  int32_t* counts;  // [blocks][E], null with one block
  int n, E, blocks, per;  // slots, experts, workgroups, slots per workgroup
};

// Lanes of the wave that hold the same expert (0 for a lane without one).
__device__ __forceinline__ uint64_t same_expert(int e, bool valid) {
  uint64_t m = __ballot(valid);
#pragma unroll
  for (int b = 0; b < 6; ++b) {
    const uint64_t s = __ballot((e >> b) & 1);
    m &= ((e >> b) & 1) ? s : ~s;
  }
  return valid ? m : 0;
}

// Calls f(slot, expert, valid, lanes of the same expert) for every slot of this
// wave's part of the workgroup's range, 64 slots at a time, in order.
template <typename F>
__device__ __forceinline__ void each_slot(const SortParams& p, int wave, int lane, F f) {
  const int part = p.per / kSortWaves;
  const int first = blockIdx.x * p.per + wave * part;
  for (int i = 0; i < part; i += kWave) {
    if (first + i >= p.n) break;  // uniform over the wave
    const int s = first + i + lane;
    const int e = s < p.n ? p.idx[s] : -1;
    const bool valid = e >= 0 && e < p.E;
    f(s, e, valid, same_expert(e, valid));
  }
}

__device__ __forceinline__ bool first_of(uint64_t mask, int lane) {
  return mask != 0 && (__ffsll((unsigned long long)mask) - 1) == lane;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams p) {
  __shared__ int32_t cnt[kSortWaves][SWIMBA_MAX_EXPERTS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  cnt[wave][lane] = 0;
  __builtin_amdgcn_wave_barrier();
  each_slot(p, wave, lane, [&](int, int e, bool, uint64_t m) {
    if (first_of(m, lane)) cnt[wave][e] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  });
  __syncthreads();
  if ((int)threadIdx.x < p.E) {
    int32_t s = 0;
    for (int w = 0; w < kSortWaves; ++w) s += cnt[w][threadIdx.x];
    p.counts[(size_t)blockIdx.x * p.E + threadIdx.x] = s;
  }
}

// Each workgroup adds up the counts of all workgroups (at most 256 of them, a
// few KB that the L2 holds) for its own first places, instead of a third
// launch in between.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortParams p) {
  __shared__ int32_t cnt[kSortWaves][SWIMBA_MAX_EXPERTS];
  __shared__ int32_t all[kSortWaves][SWIMBA_MAX_EXPERTS], before[kSortWaves][SWIMBA_MAX_EXPERTS];
  __shared__ int32_t total;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  cnt[wave][lane] = 0;
  __builtin_amdgcn_wave_barrier();
  each_slot(p, wave, lane, [&](int, int e, bool, uint64_t m) {
    if (first_of(m, lane)) cnt[wave][e] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  });
  int32_t a = 0, b = 0;
  if (p.counts != nullptr && lane < p.E) {
    for (int i = wave; i < p.blocks; i += kSortWaves) {
      const int32_t c = p.counts[(size_t)i * p.E + lane];
      a += c;
      b += i < (int)blockIdx.x ? c : 0;
    }
  }
  all[wave][lane] = a;
  before[wave][lane] = b;
  __syncthreads();
  if (wave == 0) {
    int32_t sum = 0, prev = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      sum += p.counts != nullptr ? all[w][lane] : cnt[w][lane];
      prev += before[w][lane];
    }
    int32_t incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int32_t o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    int32_t place = incl - sum + prev;
    for (int w = 0; w < kSortWaves; ++w) {  // the waves' first places
      const int32_t c = cnt[w][lane];
      cnt[w][lane] = place;
      place += c;
    }
    if (lane == 63) total = incl;
    if (blockIdx.x == 0 && lane < p.E) {
      p.offsets[lane] = incl - sum;
      if (lane == p.E - 1) p.offsets[p.E] = incl;
    }
  }
  __syncthreads();
  each_slot(p, wave, lane, [&](int s, int e, bool valid, uint64_t m) {
    int32_t at = -1;
    if (valid) {
      at = cnt[wave][e] + __popcll(m & ((1ull << lane) - 1));
      if (p.order != nullptr) p.order[at] = s;
    }
    if (s < p.n) p.pos[s] = at;
    __builtin_amdgcn_wave_barrier();
    if (first_of(m, lane)) cnt[wave][e] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  });
  if (p.order != nullptr) {  // no row behind the last one
    const int last = blockIdx.x * p.per + p.per < p.n ? blockIdx.x * p.per + p.per : p.n;
    for (int i = blockIdx.x * p.per + threadIdx.x; i < last; i += kSortThreads)
      if (i >= total) p.order[i] = -1;
  }
}

// Workgroups of a sort over n slots: 1024 slots each up to 256 workgroups, more
// slots each beyond.
int sort_blocks(int64_t n) {
  const int64_t b = (n + kSortThreads - 1) / kSortThreads;
  return (int)(b < 256 ? b : 256);
}

// A place a token's slot may have: callers' values are not trusted.
__device__ __forceinline__ bool is_row(int32_t at, int64_t rows) { return at >= 0 && at < rows; }

constexpr int kMoveThreads = 256;
constexpr int kMovePacks = 4;  // packs per thread: 64 bytes of bf16 in flight

struct MoveParams {
  const void* src;
  void* dst;
  const int32_t* pos;
  const float* gate;
  int64_t T, packs;  // tokens, packs in all
  int D, k, ppr;     // row width, slots, packs per row
};

// The packs of a thread: token and first element of each, `on` where there is
// one.  Work is laid out over packs, not rows, so that every row width fills
// the workgroups alike; all of a thread's packs are loaded before any is used
// (one pack after the other, the copy out ran at 3.6 TB/s).
struct Packs {
  int64_t t[kMovePacks];
  int c[kMovePacks];
  bool on[kMovePacks];
};

__device__ __forceinline__ Packs packs_of(const MoveParams& p) {
  const int64_t base = (int64_t)blockIdx.x * (kMoveThreads * kMovePacks);
  const int64_t t0 = base / p.ppr;  // uniform
  const uint32_t r0 = (uint32_t)(base - t0 * p.ppr);
  Packs m;
#pragma unroll
  for (int i = 0; i < kMovePacks; ++i) {
    const uint32_t r = r0 + i * kMoveThreads + threadIdx.x;
    const uint32_t dt = r / (uint32_t)p.ppr;
    m.t[i] = t0 + dt;
    m.c[i] = (int)(r - dt * p.ppr) * kPack;
    m.on[i] = m.t[i] < p.T;
    if (!m.on[i]) {  // reads then take the first row
      m.t[i] = 0;
      m.c[i] = 0;
    }
  }
  return m;
}

// A pack of row `row` (of `rows`, D wide) from column c on.
template <typename T, int ROWS>
struct RowPack {
  Loose<T, kPack> v;
  __device__ __forceinline__ void load(const T* base, int64_t row, int64_t rows, int D, int c) {
    const T* p = base + row * D + c;
    if constexpr (ROWS == kWhole) v.whole(p);
    else if constexpr (ROWS == kLoose) v.whole(p - back_of<kPack>(rows - 1 - row, D, D - c));
    else v.few(p, D - c);
  }
  __device__ __forceinline__ Pack<T> get(int64_t row, int64_t rows, int D, int c) const {
    Pack<T> p;
    if constexpr (ROWS == kWhole) v.get(0, kPack, p.v);
    else v.get(ROWS == kLoose ? back_of<kPack>(rows - 1 - row, D, D - c) : 0, D - c, p.v);
    return p;
  }
};

template <typename T, int ROWS>
__global__ __launch_bounds__(kMoveThreads) void dispatch_kernel(MoveParams p) {
  const T* x = static_cast<const T*>(p.src);
  T* rows = static_cast<T*>(p.dst);
  const int64_t n = p.T * p.k;
  const Packs m = packs_of(p);
  RowPack<T, ROWS> in[kMovePacks];
  Pack<T> v[kMovePacks];
#pragma unroll
  for (int i = 0; i < kMovePacks; ++i) in[i].load(x, m.t[i], p.T, p.D, m.c[i]);
#pragma unroll
  for (int i = 0; i < kMovePacks; ++i)
    v[i] = in[i].get(m.t[i], p.T, p.D, m.c[i]);
  for (int j = 0; j < p.k; ++j) {
    int32_t at[kMovePacks];
#pragma unroll
    for (int i = 0; i < kMovePacks; ++i) at[i] = p.pos[m.t[i] * p.k + j];
#pragma unroll
    for (int i = 0; i < kMovePacks; ++i)
      if (m.on[i] && is_row(at[i], n))
        store_pack(rows + (int64_t)at[i] * p.D + m.c[i], v[i],
                   ROWS == kWhole ? kPack : p.D - m.c[i]);
  }
}

// y_t = sum_j gate_j rows[pos_j], in slot order in fp32 (gate null: ones).
// A slot without a row reads row 0 and leaves it out.
template <typename TI, typename TO, int ROWS>
__global__ __launch_bounds__(kMoveThreads) void combine_kernel(MoveParams p) {
  const TI* rows = static_cast<const TI*>(p.src);
  TO* y = static_cast<TO*>(p.dst);
  const int64_t n = p.T * p.k;
  const Packs m = packs_of(p);
  float acc[kMovePacks][kPack] = {};
  for (int j = 0; j < p.k; ++j) {
    int32_t at[kMovePacks];
    float g[kMovePacks];
    RowPack<TI, ROWS> v[kMovePacks];
    int64_t row[kMovePacks];
#pragma unroll
    for (int i = 0; i < kMovePacks; ++i) {
      at[i] = p.pos[m.t[i] * p.k + j];
      g[i] = p.gate != nullptr ? p.gate[m.t[i] * p.k + j] : 1.f;
    }
#pragma unroll
    for (int i = 0; i < kMovePacks; ++i) {
      row[i] = is_row(at[i], n) ? at[i] : 0;
      v[i].load(rows, row[i], n, p.D, m.c[i]);
    }
#pragma unroll
    for (int i = 0; i < kMovePacks; ++i) {
      const bool in = is_row(at[i], n);
      const Pack<TI> r = v[i].get(row[i], n, p.D, m.c[i]);
#pragma unroll
      for (int u = 0; u < kPack; ++u) {
        const float s = fmaf(g[i], to_f32(r.v[u]), acc[i][u]);
        acc[i][u] = in ? s : acc[i][u];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMovePacks; ++i) {
    Pack<TO> o;
#pragma unroll
    for (int e = 0; e < kPack; ++e) o.v[e] = from_f32<TO>(acc[i][e]);
    if (m.on[i])
      store_pack(y + m.t[i] * p.D + m.c[i], o, ROWS == kWhole ? kPack : p.D - m.c[i]);
  }
}

struct CombineGradParams {
  const void *rows, *dy;
  void* drows;
  const int32_t* pos;
  const float* gate;
  float* dgate;
  int64_t T;
  int D, k;
};

// drows[pos_j] = gate_j dy_t and dgate_j = <dy_t, rows[pos_j]>, two slots at a
// time: a token per wave (PER = 1), or per workgroup of four where the tokens
// alone would leave most of the device idle (PER = 4).
template <typename TI, typename TY, typename TO, int PER, int ROWS>
__global__ __launch_bounds__(256) void combine_grad_kernel(CombineGradParams p) {
  __shared__ float part[4][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t t = PER == 4 ? wg : wg * 4 + wave;
  if (t >= p.T) return;  // whole waves, and no barrier follows where PER is 1
  const TY* dyb = static_cast<const TY*>(p.dy);
  const TI* rows = static_cast<const TI*>(p.rows);
  TO* drows = static_cast<TO*>(p.drows);
  const int64_t n = p.T * p.k;
  const int first = (PER == 4 ? threadIdx.x : lane) * kPack;
  constexpr int kStride = PER * 64 * kPack;
  for (int j0 = 0; j0 < p.k; j0 += 2) {
    bool in[2];
    float g[2], s[2] = {0.f, 0.f};
    int64_t row[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int32_t at = j0 + j < p.k ? uniform(p.pos[t * p.k + j0 + j]) : -1;
      in[j] = is_row(at, n);
      row[j] = in[j] ? at : 0;
      g[j] = in[j] ? p.gate[t * p.k + j0 + j] : 0.f;
    }
    auto pass = [&](auto* dst, int j, const Pack<TY>& d, const Pack<TI>& r, int c) {
      Pack<TO> o;
#pragma unroll
      for (int i = 0; i < kPack; ++i) {
        const float v = to_f32(d.v[i]);
        s[j] = fmaf(v, to_f32(r.v[i]), s[j]);
        o.v[i] = from_f32<TO>(g[j] * v);
      }
      store_pack(dst + row[j] * p.D + c, o, ROWS == kWhole ? kPack : p.D - c);
    };
    if (in[0] && in[1]) {
#pragma unroll 2
      for (int c = first; c < p.D; c += kStride) {
        RowPack<TY, ROWS> d;
        RowPack<TI, ROWS> a, b;
        d.load(dyb, t, p.T, p.D, c);
        a.load(rows, row[0], n, p.D, c);
        b.load(rows, row[1], n, p.D, c);
        const Pack<TY> dp = d.get(t, p.T, p.D, c);
        pass(drows, 0, dp, a.get(row[0], n, p.D, c), c);
        pass(drows, 1, dp, b.get(row[1], n, p.D, c), c);
      }
    } else if (in[0] || in[1]) {
      const int64_t r = in[0] ? row[0] : row[1];
      for (int c = first; c < p.D; c += kStride) {
        RowPack<TY, ROWS> d;
        RowPack<TI, ROWS> a;
        d.load(dyb, t, p.T, p.D, c);
        a.load(rows, r, n, p.D, c);
        const Pack<TY> dp = d.get(t, p.T, p.D, c);
        const Pack<TI> ap = a.get(r, n, p.D, c);
        if (in[0]) pass(drows, 0, dp, ap, c);
        else pass(drows, 1, dp, ap, c);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) s[j] = wave_sum64(s[j]);
    if (PER == 4) {
      if (lane == 0) {
        part[wave][0] = s[0];
        part[wave][1] = s[1];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j)
        s[j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
      __syncthreads();
    }
    if ((PER == 4 ? (int)threadIdx.x : lane) == 0) {
      p.dgate[t * p.k + j0] = s[0];
      if (j0 + 1 < p.k) p.dgate[t * p.k + j0 + 1] = s[1];
    }
  }
}

int checked() { return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP; }

MoveParams move_params(const void* src, void* dst, const int32_t* pos, const float* gate, int64_t T,
                       int D, int k) {
  MoveParams p;
  p.src = src;
  p.dst = dst;
  p.pos = pos;
  p.gate = gate;
  p.T = T;
  p.D = D;
  p.k = k;
  p.ppr = (D + kPack - 1) / kPack;
  p.packs = T * p.ppr;
  return p;
}

bool move_grid(const MoveParams& p, dim3* grid) {
  const int64_t per = kMoveThreads * kMovePacks;
  const int64_t b = (p.packs + per - 1) / per;
  if (b >= (1 << 24)) return false;  // threads are counted in 32 bits: 2^37 elements
  *grid = dim3((unsigned)b);
  return true;
}

// How rows of width D lie, in the smallest of the tensors read (`least` rows).
int rows_kind(int D, int64_t least) {
  if (D % kPack == 0) return kWhole;
  return least * D >= kPack ? kLoose : kTiny;
}

template <typename TI, typename TY, typename TO, int PER>
int launch_combine_grad_rows(const CombineGradParams& p, hipStream_t s) {
  // threads of a grid's row are counted in 32 bits
  const int64_t wg = (p.T + 4 / PER - 1) / (4 / PER), row = wg < (1 << 22) ? wg : 1 << 22;
  const dim3 grid((unsigned)row, (unsigned)((wg + row - 1) / row)), th(256);
  const int kind = rows_kind(p.D, p.T);
  if (kind == kWhole)
    hipLaunchKernelGGL((combine_grad_kernel<TI, TY, TO, PER, kWhole>), grid, th, 0, s, p);
  else if (kind == kLoose)
    hipLaunchKernelGGL((combine_grad_kernel<TI, TY, TO, PER, kLoose>), grid, th, 0, s, p);
  else
    hipLaunchKernelGGL((combine_grad_kernel<TI, TY, TO, PER, kTiny>), grid, th, 0, s, p);
  return checked();
}

template <typename TI, typename TY, typename TO>
int launch_combine_grad(const CombineGradParams& p, int dev, hipStream_t s) {
  // a workgroup per token where waves alone do not fill every SIMD four times
  return p.T < 16LL * device_cus(dev) ? launch_combine_grad_rows<TI, TY, TO, 4>(p, s)
                                      : launch_combine_grad_rows<TI, TY, TO, 1>(p, s);
}

template <typename T>
int launch_dispatch(const MoveParams& p, dim3 grid, hipStream_t s) {
  const dim3 th(kMoveThreads);
  const int kind = rows_kind(p.D, p.T);
  if (kind == kWhole) hipLaunchKernelGGL((dispatch_kernel<T, kWhole>), grid, th, 0, s, p);
  else if (kind == kLoose) hipLaunchKernelGGL((dispatch_kernel<T, kLoose>), grid, th, 0, s, p);
  else hipLaunchKernelGGL((dispatch_kernel<T, kTiny>), grid, th, 0, s, p);
  return checked();
}

template <typename TI, typename TO>
int launch_combine(const MoveParams& p, dim3 grid, hipStream_t s) {
  const dim3 th(kMoveThreads);
  const int kind = rows_kind(p.D, p.T);
  if (kind == kWhole) hipLaunchKernelGGL((combine_kernel<TI, TO, kWhole>), grid, th, 0, s, p);
  else if (kind == kLoose) hipLaunchKernelGGL((combine_kernel<TI, TO, kLoose>), grid, th, 0, s, p);
  else hipLaunchKernelGGL((combine_kernel<TI, TO, kTiny>), grid, th, 0, s, p);
  return checked();
}

}  // namespace

size_t sort_tokens_bytes(int64_t T, int E, int k) {
  const int b = sort_blocks(T * k);
  return b > 1 ? (size_t)b * E * sizeof(int32_t) : 0;
}

int launch_sort_tokens(const int32_t* idx, int64_t T, int E, int k, int32_t* order, int32_t* pos,
                       int32_t* offsets, void* ws, hipStream_t s) {
  SortParams p;
  p.idx = idx;
  p.order = order;
  p.pos = pos;
  p.offsets = offsets;
  p.n = (int)(T * k);
  p.E = E;
  p.blocks = sort_blocks(T * k);
  if (p.blocks < 1) p.blocks = 1;  // no slots: offsets only
  const int64_t per = ((int64_t)p.n + p.blocks - 1) / p.blocks;
  p.per = (int)((per + kSortThreads - 1) / kSortThreads * kSortThreads);
  if (p.per == 0) p.per = kSortThreads;
  p.blocks = p.n > 0 ? (int)(((int64_t)p.n + p.per - 1) / p.per) : 1;
  p.counts = p.blocks > 1 ? static_cast<int32_t*>(ws) : nullptr;
  if (p.blocks > 1)
    hipLaunchKernelGGL(sort_count_kernel, dim3(p.blocks), dim3(kSortThreads), 0, s, p);
  hipLaunchKernelGGL(sort_place_kernel, dim3(p.blocks), dim3(kSortThreads), 0, s, p);
  return checked();
}

int launch_dispatch_tokens(const void* x, swimba_dtype xd, const int32_t* pos, int64_t T, int D,
                           int k, void* rows, hipStream_t s) {
  const MoveParams p = move_params(x, rows, pos, nullptr, T, D, k);
  dim3 grid;
  if (!move_grid(p, &grid)) return SWIMBA_EUNSUPPORTED;
  if (xd == SWIMBA_BF16) return launch_dispatch<bf16_t>(p, grid, s);
  return launch_dispatch<float>(p, grid, s);
}

int launch_combine_tokens(const void* rows, swimba_dtype rd, const int32_t* pos, const float* gate,
                          int64_t T, int D, int k, void* y, swimba_dtype yd, hipStream_t s) {
  const MoveParams p = move_params(rows, y, pos, gate, T, D, k);
  dim3 grid;
  if (!move_grid(p, &grid)) return SWIMBA_EUNSUPPORTED;
  const bool r = rd == SWIMBA_BF16, o = yd == SWIMBA_BF16;
  if (r && o) return launch_combine<bf16_t, bf16_t>(p, grid, s);
  if (r) return launch_combine<bf16_t, float>(p, grid, s);
  if (o) return launch_combine<float, bf16_t>(p, grid, s);
  return launch_combine<float, float>(p, grid, s);
}

int launch_combine_tokens_backward(const void* rows, swimba_dtype rd, const int32_t* pos,
                                   const float* gate, const void* dy, swimba_dtype dyd, int64_t T,
                                   int D, int k, void* drows, swimba_dtype drd, float* dgate,
                                   int dev, hipStream_t s) {
  CombineGradParams p;
  p.rows = rows;
  p.dy = dy;
  p.drows = drows;
  p.pos = pos;
  p.gate = gate;
  p.dgate = dgate;
  p.T = T;
  p.D = D;
  p.k = k;
  const bool r = rd == SWIMBA_BF16, y = dyd == SWIMBA_BF16, o = drd == SWIMBA_BF16;
  if (r && y && o) return launch_combine_grad<bf16_t, bf16_t, bf16_t>(p, dev, s);
  if (r && y) return launch_combine_grad<bf16_t, bf16_t, float>(p, dev, s);
  if (r && o) return launch_combine_grad<bf16_t, float, bf16_t>(p, dev, s);
  if (r) return launch_combine_grad<bf16_t, float, float>(p, dev, s);
  if (y && o) return launch_combine_grad<float, bf16_t, bf16_t>(p, dev, s);
  if (y) return launch_combine_grad<float, bf16_t, float>(p, dev, s);
  if (o) return launch_combine_grad<float, float, bf16_t>(p, dev, s);
  return launch_combine_grad<float, float, float>(p, dev, s);
}

}  // namespace swimba
