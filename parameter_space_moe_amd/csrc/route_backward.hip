// Gradients of the router: softmax over the selected logits, then the product
// x . Wr.  With s_j = gate_j (dgate_j - sum_i gate_i dgate_i) the slope of the
// loss along the token's j-th selected logit,
//   dx_t[d]   = sum_j s_j Wr[d, e_j]          (k terms per element)
//   dWr[d, e] = sum over tokens of s x_t[d]   (a product of s^T and x)
// x is read and dx written once.  A wave owns 64 channels and walks tokens 16
// at a time: lane (q, c) holds channels 4c..4c+3 of token 4i + q, which is the
// B operand of the fp32 matrix instruction 16x16x4 as it comes from memory, so
// dWr accumulates in registers, in fp32, with the slopes of a 64-token tile as
// a dense [token][expert] table in LDS for the A operand (one 64-lane
// instruction per 1024 multiply-adds instead of a read-add-write of an LDS row
// per selected expert).  dx takes the k selected rows of Wr from an LDS copy.
// Bound by the stream of x and dx up to 16 experts: 65536 tokens of 2560 bf16
// channels in 158 us, 4.3 TB/s (421 us with each tile's loads and table waited
// for, 195 us with the rows ahead).  Beyond 32 experts the copy of Wr leaves one
// workgroup per CU and a tile's latency bounds it: 5001 tokens of 1536 fp32
// channels and 64 experts in 38 us, 55 us at 1538, whose rows are unaligned.
#include "pack.hpp"
#include "swimba_internal.hpp"

namespace swimba {
namespace {

constexpr int kThreads = 256;
constexpr int kSlab = 256;        // channels per workgroup, 64 per wave
constexpr int kSlabStride = 260;  // LDS row of Wr^T: 16-byte rows, banks shifted by 4
constexpr int kTile = 64;         // tokens per slope table

typedef float f4 __attribute__((ext_vector_type(4)));

struct RouteGradParams {
  const void* x;
  const float *Wr, *gate, *dgate;
  const int32_t* idx;
  void* dx;
  float* dWr;   // [D][E], written here when there is one split
  float* part;  // [splits][E][D] otherwise
  int64_t T;
  int D, E, k;
  int64_t per;  // tokens per split
  int two;      // LDS holds two slope tables
};

template <typename T>
__device__ __forceinline__ void store4(T* p, int n, const float* v) {
  struct __attribute__((packed, aligned(sizeof(T)))) Loose { T e[4]; };
  if (n >= 4) {
    Loose l;
#pragma unroll
    for (int i = 0; i < 4; ++i) l.e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<Loose*>(p) = l;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// LDS of one tile's slopes: by slot (with the place of the expert's row of Wr^T
// in LDS: the row of zeros behind the last one without an expert), and dense by
// expert.
template <int ET>
struct Slopes {
  static constexpr int kDense = ET * 16 + 1;
  float2* slot;   // [kTile][k] slope, row (an int's bits)
  float* dense;   // [kTile][kDense]
  int32_t* any;   // [kTile] tokens with an expert
  static constexpr size_t words(int k) { return kTile * (kDense + 1 + 2 * (size_t)k); }
  __device__ __forceinline__ Slopes(float* at, int k)
      : slot(reinterpret_cast<float2*>(at)),
        dense(at + 2 * kTile * k),
        any(reinterpret_cast<int32_t*>(dense + kTile * kDense)) {}
};

// Waves per SIMD that the registers have to leave room for: what the LDS of the
// expert count allows, and fewer where a step would spill (its reloads wait for
// the rows on their way).
constexpr int least_waves(size_t elem, int et, int rows) {
  return et == 4 ? 1 : (elem == 4 || et == 2 || rows != kWhole ? 2 : 3);
}

// ET: expert tiles of 16; K: most slots per token that are held in registers
// (0: any number of slots); ROWS: kLoose, kWhole or kTiny.
template <typename TI, typename TO, int ET, int K, int ROWS>
__global__ __launch_bounds__(kThreads, least_waves(sizeof(TI), ET, ROWS))
void route_grad_kernel(RouteGradParams p) {
  using Table = Slopes<ET>;
  constexpr bool WHOLE = ROWS == kWhole;
  constexpr int kDense = Table::kDense;
  extern __shared__ __attribute__((aligned(16))) float smem[];
  const int k = K > 0 ? K : p.k;
  float* sW = smem;  // [E + 1][kSlabStride]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, c = lane & 15;
  const int d0 = blockIdx.x * kSlab, dl = wave * 64 + 4 * c, d = d0 + dl;
  const int left = p.D - d;  // channels of this lane inside the row
  const int64_t tb = (int64_t)blockIdx.y * p.per;
  const int64_t te = tb + p.per < p.T ? tb + p.per : p.T;
  const TI* x = static_cast<const TI*>(p.x);
  TO* dx = static_cast<TO*>(p.dx);

  const int slab = p.D - d0 < kSlab ? p.D - d0 : kSlab;
  // Wr's rows of the slab lie one behind the other; eight loads at a time
  for (int i0 = threadIdx.x; i0 < slab * p.E; i0 += 8 * kThreads) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * kThreads;
      v[u] = p.Wr[(int64_t)d0 * p.E + (i < slab * p.E ? i : 0)];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * kThreads, r = i / p.E;
      if (i < slab * p.E) sW[(i - r * p.E) * kSlabStride + r] = v[u];
    }
  }

  sW[p.E * kSlabStride + threadIdx.x] = 0.f;

  f4 acc[ET][4];
#pragma unroll
  for (int e = 0; e < ET; ++e)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[e][j] = f4{0.f, 0.f, 0.f, 0.f};

  // 32 rows of x are in flight while the 32 before are worked on
  constexpr int kSteps = 8;
  Loose<TI, 4> xr[kSteps];
  auto back = [&](int64_t t) {
    return ROWS == kLoose ? back_of<4>(p.T - 1 - t, p.D, left) : 0;
  };
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t t = t0 + 4 * i + q;
      const bool in = t < te && left > 0;  // others: the first channels of x
      const TI* at = x + (in ? t * p.D + d - back(t) : 0);
      if constexpr (ROWS == kTiny) xr[i].few(at, in ? left : 0);
      else xr[i].whole(at);
    }
  };
  if (tb < te) fetch(tb);  // without tokens x may be null

  // A tile's table is made by one wave, a lane per token, each wave in its turn:
  // from values loaded before the tile ahead of it is worked on.
  constexpr int kHold = K > 0 ? K : 1;
  float pg[kHold], pd[kHold];
  int32_t pe[kHold];
  auto values = [&](int64_t t0) {
    if constexpr (K > 0) {
      const int64_t t = t0 + lane, s = (t < te ? t : tb) * p.k;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int64_t at = s + (j < p.k ? j : 0);
        pg[j] = p.gate[at];
        pd[j] = p.dgate[at];
        pe[j] = p.idx[at];
      }
    }
  };
  auto make = [&](int64_t t0, const Table& tab) {
    float* row = tab.dense + lane * kDense;
    for (int e = 0; e < ET * 16; ++e) row[e] = 0.f;
    int32_t any = 0;
    if (t0 + lane < te) {
      float mean = 0.f;
      if constexpr (K > 0) {
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (j < p.k) mean = fmaf(pg[j], pd[j], mean);
      } else {
        const int64_t s = (t0 + lane) * k;
        for (int j = 0; j < k; ++j) mean = fmaf(p.gate[s + j], p.dgate[s + j], mean);
      }
      auto slot = [&](int j, float g, float dg, int e, bool has) {
        const bool in = has && e >= 0 && e < p.E;
        const float v = g * (dg - mean);
        const int row_at = (in ? e : p.E) * kSlabStride;
        tab.slot[lane * k + j] = make_float2(in ? v : 0.f, __int_as_float(row_at));
        any |= in;
        if (in) row[e] += v;  // an expert listed twice adds twice
      };
      if constexpr (K > 0) {
#pragma unroll
        for (int j = 0; j < K; ++j) slot(j, pg[j], pd[j], pe[j], j < p.k);
      } else {
        const int64_t s = (t0 + lane) * k;
        for (int j = 0; j < k; ++j) slot(j, p.gate[s + j], p.dgate[s + j], p.idx[s + j], true);
      }
    }
    tab.any[lane] = any;
  };
  const Table tab0(smem + (p.E + 1) * kSlabStride, k);
  const Table tab1(smem + (p.E + 1) * kSlabStride + (p.two ? Table::words(k) : 0), k);
  if (wave == 0 && tb < te) {
    values(tb);
    make(tb, tab0);
  }

  for (int64_t t0 = tb; t0 < te; t0 += kTile) {
    const int turn = (int)((t0 - tb) / kTile);
    const int len = te - t0 < kTile ? (int)(te - t0) : kTile;
    const Table& tab = turn & 1 ? tab1 : tab0;
    const bool maker = wave == ((turn + 1) & 3) && t0 + kTile < te;
    __syncthreads();  // this tile's table is made, the one before is done with
    if (maker) values(t0 + kTile);
#pragma unroll 1
    for (int hb = 0; hb < kTile; hb += 4 * kSteps) {
      if (hb >= len) break;
      Loose<TI, 4> xc[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) xc[i] = xr[i];
      fetch(t0 + hb + 4 * kSteps);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int t = hb + 4 * i + q;
        float xv[4];
        // a token without an expert may hold anything: left out
        {
          const int n = t < len && tab.any[t] ? (WHOLE && left > 0 ? 4 : left) : 0;
          TI e[4];
          xc[i].get(back(t0 + t), n, e);
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[j] = to_f32(e[j]);
        }
        float a[ET];
#pragma unroll
        for (int e = 0; e < ET; ++e) a[e] = tab.dense[t * kDense + e * 16 + c];
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[e][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], xv[j], acc[e][j], 0, 0, 0);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        const int ts = t < len ? t : 0;
        for (int j = 0; j < k; ++j) {
          const float2 v = tab.slot[ts * k + j];
          const float4 w = *reinterpret_cast<const float4*>(sW + __float_as_int(v.y) + dl);
          o[0] = fmaf(v.x, w.x, o[0]);
          o[1] = fmaf(v.x, w.y, o[1]);
          o[2] = fmaf(v.x, w.z, o[2]);
          o[3] = fmaf(v.x, w.w, o[3]);
        }
        if (t < len && left > 0)
          store4(dx + t0 * p.D + ((int64_t)t * p.D + d), WHOLE ? 4 : left, o);
        __builtin_amdgcn_sched_barrier(0);  // else every step's operands are held at once
      }
    }
    if (!p.two) __syncthreads();  // one table only: everyone has to be done with it
    if (maker) make(t0 + kTile, turn & 1 ? tab0 : tab1);
  }

  // acc[e][j][i]: expert 16 e + 4 q + i, channel d + j
#pragma unroll
  for (int e = 0; e < ET; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ex = 16 * e + 4 * q + i;
      if (ex >= p.E || left <= 0) continue;
      const float v[4] = {acc[e][0][i], acc[e][1][i], acc[e][2][i], acc[e][3][i]};
      if (p.part != nullptr) {
        store4(p.part + ((int64_t)blockIdx.y * p.E + ex) * p.D + d, left, v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left) p.dWr[(int64_t)(d + j) * p.E + ex] = v[j];
      }
    }
}

// dWr[d][e] = sum over the splits, in order.
__global__ __launch_bounds__(256) void route_grad_sum_kernel(const float* part, float* dWr, int D,
                                                             int E, int splits) {
  const int64_t n = (int64_t)D * E;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
#pragma unroll 8
  for (int r = 0; r < splits; ++r) s += part[(int64_t)r * n + i];
  const int64_t e = i / D;
  dWr[(i - e * D) * E + e] = s;
}

struct RouteGradPlan {
  int slabs = 0, splits = 1;
  int64_t per = 0;
  size_t bytes = 0;
};

// As many workgroups as the device holds at once (by registers and LDS three
// per CU up to 16 experts with bf16 x, two up to 32 and with fp32 x, one
// beyond), splits of whole 64-token tiles, and no more of them than keeps the
// partial sums (8 E bytes per channel and split, out and in) within the stream of
// x and dx: a tile of 64 experts takes a workgroup 7 us, as long as the sums of
// 30 MB.
RouteGradPlan plan(int64_t T, int D, int E, int elem, int dev) {
  RouteGradPlan r;
  r.slabs = (D + kSlab - 1) / kSlab;
  const int64_t tiles = (T + kTile - 1) / kTile;
  const int per_cu = E > 32 ? 1 : (E > 16 || elem == 4 || D % 4 != 0 ? 2 : 3);
  int64_t want = (int64_t)per_cu * device_cus(dev) / r.slabs;
  const int64_t least = (8LL * E / (2 * elem) + kTile - 1) / kTile;  // tiles per split
  if (want > tiles / least) want = tiles / least;
  if (want < 1) want = 1;
  const int64_t per = (tiles + want - 1) / want;
  r.per = per * kTile;
  r.splits = tiles > 0 ? (int)((tiles + per - 1) / per) : 1;
  if (r.splits > 1) r.bytes = (size_t)r.splits * E * D * sizeof(float);
  return r;
}

template <typename TI, typename TO, int ET, int K, int ROWS>
int launch(const RouteGradParams& a, const RouteGradPlan& r, hipStream_t s) {
  RouteGradParams p = a;
  const size_t fixed = (size_t)(p.E + 1) * kSlabStride * sizeof(float);
  const size_t table = Slopes<ET>::words(K > 0 ? K : p.k) * sizeof(float);
  p.two = fixed + 2 * table <= 160 * 1024;  // one table where nearly every expert is selected
  const size_t lds = fixed + (p.two ? 2 : 1) * table;
  allow_dynamic_lds(route_grad_kernel<TI, TO, ET, K, ROWS>, lds);
  hipLaunchKernelGGL((route_grad_kernel<TI, TO, ET, K, ROWS>), dim3(r.slabs, r.splits),
                     dim3(kThreads), lds, s, p);
  if (hipGetLastError() != hipSuccess) return SWIMBA_EHIP;
  if (r.splits > 1) {
    const int64_t n = (int64_t)p.D * p.E;
    hipLaunchKernelGGL(route_grad_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                       p.part, p.dWr, p.D, p.E, r.splits);
  }
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

template <typename TI, typename TO, int ET>
int launch_slots(const RouteGradParams& p, const RouteGradPlan& r, hipStream_t s) {
  const bool whole = p.D % 4 == 0;
  if (p.k == 2)
    return whole ? launch<TI, TO, ET, 2, kWhole>(p, r, s) : launch<TI, TO, ET, 2, kLoose>(p, r, s);
  if (p.k <= 4)
    return whole ? launch<TI, TO, ET, 4, kWhole>(p, r, s) : launch<TI, TO, ET, 4, kLoose>(p, r, s);
  return whole ? launch<TI, TO, ET, 0, kWhole>(p, r, s) : launch<TI, TO, ET, 0, kLoose>(p, r, s);
}

template <typename TI, typename TO>
int launch_types(const RouteGradParams& p, const RouteGradPlan& r, hipStream_t s) {
  if (p.D % 4 != 0 && p.T * p.D < 4) return launch<TI, TO, 4, 0, kTiny>(p, r, s);
  if (p.E <= 16) return launch_slots<TI, TO, 1>(p, r, s);
  if (p.E <= 32) return launch_slots<TI, TO, 2>(p, r, s);
  return launch_slots<TI, TO, 4>(p, r, s);
}

}  // namespace

size_t route_backward_bytes(int64_t T, int D, int E, int dev) {
  // whatever the types are
  const size_t a = plan(T, D, E, 2, dev).bytes, b = plan(T, D, E, 4, dev).bytes;
  return a > b ? a : b;
}

int launch_route_backward(const void* x, swimba_dtype xd, const float* Wr, const int32_t* idx,
                          const float* gate, const float* dgate, int64_t T, int D, int E, int k,
                          void* dx, swimba_dtype dxd, float* dWr, void* ws, int dev,
                          hipStream_t s) {
  const RouteGradPlan r = plan(T, D, E, xd == SWIMBA_BF16 ? 2 : 4, dev);
  RouteGradParams p;
  p.x = x;
  p.Wr = Wr;
  p.idx = idx;
  p.gate = gate;
  p.dgate = dgate;
  p.dx = dx;
  p.dWr = dWr;
  p.part = r.splits > 1 ? static_cast<float*>(ws) : nullptr;
  p.T = T;
  p.D = D;
  p.E = E;
  p.k = k;
  p.per = r.per;
  if (xd == SWIMBA_BF16)
    return dxd == SWIMBA_BF16 ? launch_types<bf16_t, bf16_t>(p, r, s)
                              : launch_types<bf16_t, float>(p, r, s);
  return dxd == SWIMBA_BF16 ? launch_types<float, bf16_t>(p, r, s)
                            : launch_types<float, float>(p, r, s);
}

}  // namespace swimba
