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

// f(token, first element) for the packs of this thread.  Work is laid out over
// packs, not rows, so that every row width fills the workgroups alike.
template <typename F>
__device__ __forceinline__ void each_pack(const MoveParams& p, F f) {
  const int64_t base = (int64_t)blockIdx.x * (kMoveThreads * kMovePacks);
  const int64_t t0 = base / p.ppr;  // uniform
  const uint32_t r0 = (uint32_t)(base - t0 * p.ppr);
#pragma unroll
  for (int i = 0; i < kMovePacks; ++i) {
    const uint32_t r = r0 + i * kMoveThreads + threadIdx.x;
    const uint32_t dt = r / (uint32_t)p.ppr;
    const int64_t t = t0 + dt;
    if (t < p.T) f(t, (int)(r - dt * p.ppr) * kPack);
  }
}

template <typename T>
__global__ __launch_bounds__(kMoveThreads) void dispatch_kernel(MoveParams p) {
  const T* x = static_cast<const T*>(p.src);
  T* rows = static_cast<T*>(p.dst);
  const int64_t n = p.T * p.k;
  each_pack(p, [&](int64_t t, int c) {
    const Pack<T> v = load_pack(x + t * p.D + c, p.D - c);
    for (int j = 0; j < p.k; ++j) {
      const int32_t at = p.pos[t * p.k + j];
      if (is_row(at, n)) store_pack(rows + (int64_t)at * p.D + c, v, p.D - c);
    }
  });
}

// y_t = sum_j gate_j rows[pos_j], in slot order in fp32 (gate null: ones).
template <typename TI, typename TO>
__global__ __launch_bounds__(kMoveThreads) void combine_kernel(MoveParams p) {
  const TI* rows = static_cast<const TI*>(p.src);
  TO* y = static_cast<TO*>(p.dst);
  const int64_t n = p.T * p.k;
  each_pack(p, [&](int64_t t, int c) {
    float acc[kPack] = {};
    for (int j = 0; j < p.k; ++j) {
      const int32_t at = p.pos[t * p.k + j];
      if (!is_row(at, n)) continue;
      const float g = p.gate != nullptr ? p.gate[t * p.k + j] : 1.f;
      const Pack<TI> v = load_pack(rows + (int64_t)at * p.D + c, p.D - c);
#pragma unroll
      for (int i = 0; i < kPack; ++i) acc[i] = fmaf(g, to_f32(v.v[i]), acc[i]);
    }
    Pack<TO> o;
#pragma unroll
    for (int i = 0; i < kPack; ++i) o.v[i] = from_f32<TO>(acc[i]);
    store_pack(y + t * p.D + c, o, p.D - c);
  });
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

// drows[pos_j] = gate_j dy_t and dgate_j = <dy_t, rows[pos_j]>: a workgroup of
// WAVES waves per token and slot pass, sums across its threads.
template <typename TI, typename TY, typename TO, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void combine_grad_kernel(CombineGradParams p) {
  __shared__ float part[WAVES];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const TY* dy = static_cast<const TY*>(p.dy) + t * p.D;
  const int64_t n = p.T * p.k;
  for (int j = 0; j < p.k; ++j) {
    const int32_t at = p.pos[t * p.k + j];  // uniform
    float s = 0.f;
    if (is_row(at, n)) {
      const float g = p.gate[t * p.k + j];
      const TI* row = static_cast<const TI*>(p.rows) + (int64_t)at * p.D;
      TO* drow = static_cast<TO*>(p.drows) + (int64_t)at * p.D;
      for (int c = threadIdx.x * kPack; c < p.D; c += WAVES * 64 * kPack) {
        const Pack<TY> d = load_pack(dy + c, p.D - c);
        const Pack<TI> r = load_pack(row + c, p.D - c);
        Pack<TO> o;
#pragma unroll
        for (int i = 0; i < kPack; ++i) {
          const float v = to_f32(d.v[i]);
          s = fmaf(v, to_f32(r.v[i]), s);
          o.v[i] = from_f32<TO>(g * v);
        }
        store_pack(drow + c, o, p.D - c);
      }
    }
    s = wave_sum64(s);
    if (WAVES > 1) {
      if (lane == 0) part[wave] = s;
      __syncthreads();
      s = 0.f;
      for (int w = 0; w < WAVES; ++w) s += part[w];
      __syncthreads();
    }
    if (threadIdx.x == 0) p.dgate[t * p.k + j] = s;
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
  if (b > 0x7fffffff) return false;
  *grid = dim3((unsigned)b);
  return true;
}

template <typename TI, typename TY, typename TO>
int launch_combine_grad(const CombineGradParams& p, hipStream_t s) {
  if (p.T > 0x7fffffff) return SWIMBA_EUNSUPPORTED;
  hipLaunchKernelGGL((combine_grad_kernel<TI, TY, TO, 4>), dim3((unsigned)p.T), dim3(256), 0, s, p);
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
  if (xd == SWIMBA_BF16)
    hipLaunchKernelGGL((dispatch_kernel<bf16_t>), grid, dim3(kMoveThreads), 0, s, p);
  else
    hipLaunchKernelGGL((dispatch_kernel<float>), grid, dim3(kMoveThreads), 0, s, p);
  return checked();
}

int launch_combine_tokens(const void* rows, swimba_dtype rd, const int32_t* pos, const float* gate,
                          int64_t T, int D, int k, void* y, swimba_dtype yd, hipStream_t s) {
  const MoveParams p = move_params(rows, y, pos, gate, T, D, k);
  dim3 grid;
  if (!move_grid(p, &grid)) return SWIMBA_EUNSUPPORTED;
  const dim3 th(kMoveThreads);
  if (rd == SWIMBA_BF16 && yd == SWIMBA_BF16)
    hipLaunchKernelGGL((combine_kernel<bf16_t, bf16_t>), grid, th, 0, s, p);
  else if (rd == SWIMBA_BF16)
    hipLaunchKernelGGL((combine_kernel<bf16_t, float>), grid, th, 0, s, p);
  else if (yd == SWIMBA_BF16)
    hipLaunchKernelGGL((combine_kernel<float, bf16_t>), grid, th, 0, s, p);
  else
    hipLaunchKernelGGL((combine_kernel<float, float>), grid, th, 0, s, p);
  return checked();
}

int launch_combine_tokens_backward(const void* rows, swimba_dtype rd, const int32_t* pos,
                                   const float* gate, const void* dy, swimba_dtype dyd, int64_t T,
                                   int D, int k, void* drows, swimba_dtype drd, float* dgate,
                                   hipStream_t s) {
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
  if (r && y && o) return launch_combine_grad<bf16_t, bf16_t, bf16_t>(p, s);
  if (r && y) return launch_combine_grad<bf16_t, bf16_t, float>(p, s);
  if (r && o) return launch_combine_grad<bf16_t, float, bf16_t>(p, s);
  if (r) return launch_combine_grad<bf16_t, float, float>(p, s);
  if (y && o) return launch_combine_grad<float, bf16_t, bf16_t>(p, s);
  if (y) return launch_combine_grad<float, bf16_t, float>(p, s);
  if (o) return launch_combine_grad<float, float, bf16_t>(p, s);
  return launch_combine_grad<float, float, float>(p, s);
}

}  // namespace swimba
