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
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, int n, float* v) {
  struct __attribute__((packed, aligned(sizeof(T)))) Loose { T e[4]; };
  if (n >= 4) {
    const Loose l = *reinterpret_cast<const Loose*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_f32(l.e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

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

// ET: expert tiles of 16.
template <typename TI, typename TO, int ET>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradParams p) {
  constexpr int kDense = ET * 16 + 1;
  extern __shared__ __attribute__((aligned(16))) float smem[];
  float* sW = smem;                               // [E][kSlabStride]
  float* sS = sW + p.E * kSlabStride;             // [kTile][kDense] slopes
  float* sV = sS + kTile * kDense;                // [kTile][k] slopes of the slots
  int32_t* sE = reinterpret_cast<int32_t*>(sV + kTile * p.k);  // [kTile][k] experts
  int32_t* sOk = sE + kTile * p.k;                // [kTile] tokens with an expert
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, c = lane & 15;
  const int d0 = blockIdx.x * kSlab, dl = wave * 64 + 4 * c, d = d0 + dl;
  const int left = p.D - d;  // channels of this lane inside the row
  const int64_t tb = (int64_t)blockIdx.y * p.per;
  const int64_t te = tb + p.per < p.T ? tb + p.per : p.T;
  const TI* x = static_cast<const TI*>(p.x);
  TO* dx = static_cast<TO*>(p.dx);

  const int slab = p.D - d0 < kSlab ? p.D - d0 : kSlab;
  for (int i = threadIdx.x; i < slab * p.E; i += kThreads) {
    const int r = i / p.E;
    sW[(i - r * p.E) * kSlabStride + r] = p.Wr[(int64_t)d0 * p.E + i];
  }

  f4 acc[ET][4];
#pragma unroll
  for (int e = 0; e < ET; ++e)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[e][j] = f4{0.f, 0.f, 0.f, 0.f};

  for (int64_t t0 = tb; t0 < te; t0 += kTile) {
    const int len = te - t0 < kTile ? (int)(te - t0) : kTile;
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kDense; i += kThreads) sS[i] = 0.f;
    __syncthreads();
    if ((int)threadIdx.x < len) {
      const int64_t s = (t0 + threadIdx.x) * p.k;
      float mean = 0.f;
      int32_t any = 0;
      for (int j = 0; j < p.k; ++j) mean = fmaf(p.gate[s + j], p.dgate[s + j], mean);
      for (int j = 0; j < p.k; ++j) {
        const int e = p.idx[s + j];
        const bool in = e >= 0 && e < p.E;
        const float v = p.gate[s + j] * (p.dgate[s + j] - mean);
        sV[threadIdx.x * p.k + j] = v;
        sE[threadIdx.x * p.k + j] = in ? e : -1;
        any |= in;
        if (in) sS[threadIdx.x * kDense + e] += v;  // an expert listed twice adds twice
      }
      sOk[threadIdx.x] = any;
    } else if (threadIdx.x < kTile) {
      sOk[threadIdx.x] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int st = 0; st < kTile / 16; ++st) {
      if (st * 16 >= len) break;
      float xv[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = st * 16 + 4 * i + q;
        // a token without an expert may hold anything: not read
        load4(x + (t0 + t) * p.D + d, sOk[t] ? left : 0, xv[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = st * 16 + 4 * i + q;
        float a[ET];
#pragma unroll
        for (int e = 0; e < ET; ++e) a[e] = sS[t * kDense + e * 16 + c];
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[e][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], xv[i][j], acc[e][j], 0, 0, 0);
        if (t < len && left > 0) {
          float o[4] = {0.f, 0.f, 0.f, 0.f};
          for (int j = 0; j < p.k; ++j) {
            const int e = sE[t * p.k + j];
            if (e < 0) continue;
            const float v = sV[t * p.k + j];
            const float4 w = *reinterpret_cast<const float4*>(sW + e * kSlabStride + dl);
            o[0] = fmaf(v, w.x, o[0]);
            o[1] = fmaf(v, w.y, o[1]);
            o[2] = fmaf(v, w.z, o[2]);
            o[3] = fmaf(v, w.w, o[3]);
          }
          store4(dx + (t0 + t) * p.D + d, left, o);
        }
      }
    }
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

// Four workgroups per CU (the LDS of 16 experts allows more), splits of whole
// 64-token tiles.
RouteGradPlan plan(int64_t T, int D, int E, int dev) {
  RouteGradPlan r;
  r.slabs = (D + kSlab - 1) / kSlab;
  const int64_t tiles = (T + kTile - 1) / kTile;
  int64_t want = (4LL * device_cus(dev) + r.slabs - 1) / r.slabs;
  if (want > tiles) want = tiles;
  if (want < 1) want = 1;
  const int64_t per = (tiles + want - 1) / want;
  r.per = per * kTile;
  r.splits = tiles > 0 ? (int)((tiles + per - 1) / per) : 1;
  if (r.splits > 1) r.bytes = (size_t)r.splits * E * D * sizeof(float);
  return r;
}

template <typename TI, typename TO, int ET>
int launch(const RouteGradParams& p, const RouteGradPlan& r, hipStream_t s) {
  const size_t lds = ((size_t)p.E * kSlabStride + kTile * (ET * 16 + 2) + 2 * (size_t)kTile * p.k) *
                     sizeof(float);
  allow_dynamic_lds(route_grad_kernel<TI, TO, ET>, lds);
  hipLaunchKernelGGL((route_grad_kernel<TI, TO, ET>), dim3(r.slabs, r.splits), dim3(kThreads), lds,
                     s, p);
  if (hipGetLastError() != hipSuccess) return SWIMBA_EHIP;
  if (r.splits > 1) {
    const int64_t n = (int64_t)p.D * p.E;
    hipLaunchKernelGGL(route_grad_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                       p.part, p.dWr, p.D, p.E, r.splits);
  }
  return hipGetLastError() == hipSuccess ? SWIMBA_OK : SWIMBA_EHIP;
}

template <typename TI, typename TO>
int launch_types(const RouteGradParams& p, const RouteGradPlan& r, hipStream_t s) {
  if (p.E <= 16) return launch<TI, TO, 1>(p, r, s);
  if (p.E <= 32) return launch<TI, TO, 2>(p, r, s);
  return launch<TI, TO, 4>(p, r, s);
}

}  // namespace

size_t route_backward_bytes(int64_t T, int D, int E, int dev) { return plan(T, D, E, dev).bytes; }

int launch_route_backward(const void* x, swimba_dtype xd, const float* Wr, const int32_t* idx,
                          const float* gate, const float* dgate, int64_t T, int D, int E, int k,
                          void* dx, swimba_dtype dxd, float* dWr, void* ws, int dev,
                          hipStream_t s) {
  const RouteGradPlan r = plan(T, D, E, dev);
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
