// train.cu - element-wise kernels of the training pass: the combine's gradient and the dense
// product's activation gradient with its column sums.
#include <algorithm>

#include "device.cuh"
#include "epilogue.cuh"
#include "kernels.h"

namespace moe {

namespace {

// ---------------------------------------------------------------------------
// Gradient of the combine: dy[r] = w[t][k] dout[t], dw[t][k] = <dout[t], y[r]>, r the row of (t, k).
// Bound by HBM: K rows read, K rows written and one row of dout read a token.  A token's row is
// taken by WPT warps (a power of two up to 8), each lane holding 16-byte pieces: dout's piece is
// read once for the K rows.  WPT = 1 (no exchange between warps) as soon as the tokens fill the
// GPU's warps, more for few tokens.  Wide rows reach the copy rate (8192 tokens, K 8, H 7168: 344 us, 5.8
// TB/s; 4096 tokens, H 2048: 55 us, 5.2), narrow ones and few of them (K 2) leave lanes or loads idle (8192
// tokens, K 8, H 256: 19 us, 3.8; K 2, H 1032: 38 us, 2.3; 65536 tokens, K 8, H 64: 94 us, 1.6).
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;
constexpr int kCombineRows = 8;  // rows in flight (and partial sums) at a time

__device__ __forceinline__ float dot8(const uint4 a, const uint4 b, float acc) {
  const __nv_bfloat162* pa = reinterpret_cast<const __nv_bfloat162*>(&a);
  const __nv_bfloat162* pb = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __bfloat1622float2(pa[j]), y = __bfloat1622float2(pb[j]);
    acc = fmaf(x.x, y.x, acc);
    acc = fmaf(x.y, y.y, acc);
  }
  return acc;
}

__device__ __forceinline__ uint4 scale8(const uint4 a, float w) {
  const __nv_bfloat162* pa = reinterpret_cast<const __nv_bfloat162*>(&a);
  uint4 o;
  __nv_bfloat162* po = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __bfloat1622float2(pa[j]);
    po[j] = __floats2bfloat162_rn(w * x.x, w * x.y);
  }
  return o;
}

// y and dy may be the same buffer: every piece is read before it is written, by one thread.
template <int WPT>
__global__ void __launch_bounds__(kCombineThreads) combine_bwd_kernel(const uint4* __restrict__ dout, const uint4* y,
                                                                      const int32_t* __restrict__ roa,
                                                                      const float* __restrict__ w, long long T, int vpr,
                                                                      int K, uint4* dy, float* __restrict__ dw) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kTokens = kCombineThreads / 32 / WPT;  // tokens of a block
  __shared__ float s_part[kCombineThreads / 32][kCombineRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = warp / WPT, sub = warp % WPT;
  const long long TK = T * K;
  for (long long t0 = static_cast<long long>(blockIdx.x) * kTokens; t0 < T;
       t0 += static_cast<long long>(gridDim.x) * kTokens) {
    const long long t = t0 + slot;
    const bool live = t < T;
    for (int k0 = 0; k0 < K; k0 += kCombineRows) {
      float acc[kCombineRows], wk[kCombineRows];
      long long base[kCombineRows];  // first piece of the row, or -1
#pragma unroll
      for (int k = 0; k < kCombineRows; ++k) {
        acc[k] = 0.0f;
        wk[k] = 0.0f;
        base[k] = -1;
        if (live && k0 + k < K) {
          const long long row = __ldg(roa + t * K + k0 + k);
          if (row >= 0 && row < TK) base[k] = row * vpr;
          wk[k] = __ldg(w + t * K + k0 + k);
        }
      }
      if (live) {
        for (int v = sub * 32 + lane; v < vpr; v += 32 * WPT) {
          const uint4 d = __ldg(dout + t * vpr + v);
          if (dw) {
            uint4 r[kCombineRows];
#pragma unroll
            for (int k = 0; k < kCombineRows; ++k)
              r[k] = base[k] >= 0 ? y[base[k] + v] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < kCombineRows; ++k)
              if (base[k] >= 0) acc[k] = dot8(d, r[k], acc[k]);
          }
          if (dy) {
#pragma unroll
            for (int k = 0; k < kCombineRows; ++k)
              if (base[k] >= 0) dy[base[k] + v] = scale8(d, wk[k]);
          }
        }
      }
      if (!dw) continue;
#pragma unroll
      for (int k = 0; k < kCombineRows; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
      }
      if constexpr (WPT == 1) {
#pragma unroll
        for (int k = 0; k < kCombineRows; ++k)
          if (lane == k && live && k0 + k < K) dw[t * K + k0 + k] = acc[k];
      } else {
#pragma unroll
        for (int k = 0; k < kCombineRows; ++k)
          if (lane == k) s_part[warp][k] = acc[k];
        __syncthreads();
        if (sub == 0 && lane < kCombineRows && live && k0 + lane < K) {
          float s = 0.0f;
#pragma unroll
          for (int i = 0; i < WPT; ++i) s += s_part[slot * WPT + i][lane];
          dw[t * K + k0 + lane] = s;
        }
        __syncthreads();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Activation gradient: dpre = dout act'(pre), dbias = column sums of dpre (fp32, before dpre is
// rounded).  2 + 4 bytes read and 2 written an element: bound by HBM for ReLU and SiLU where the blocks fill the
// SMs (16384 x 4096, dbias alone: 64 and 67 us, 6.3 and 6.0 TB/s), by the arithmetic for the others (GELU 118,
// tanh-GELU 93).  There are at most 8 ceil(N / 64) blocks, so a layer of fewer than about 1200 columns leaves SMs
// idle whatever its rows (65536 x 512, SiLU: 153 us, 1.3 TB/s).  A block owns 64 columns
// (eight 16-byte pieces) and 32 rows at a time; a cluster of up to 8 blocks shares the columns,
// each with its part of the rows, and adds the parts' column sums over distributed shared memory
// in rank order, so the sums need no workspace, no atomics and one launch.
// ---------------------------------------------------------------------------
constexpr int kActThreads = 256;
constexpr int kActCols = 64;

// sigma(a) and 1 - sigma(a) from e = exp(-|a|).  As a difference the second would carry half a step of 1,
// to one side, which act' then multiplies by up to 35 (gelu_tanh: 2e-6 off at x = 5).
struct Logistic {
  float s, c;
};
__device__ __forceinline__ Logistic logistic(float a) {
  const float e = __expf(-fabsf(a)), r = __fdividef(1.0f, 1.0f + e), q = e * r;
  return a < 0.0f ? Logistic{q, r} : Logistic{r, q};
}

// act'(x).
template <int ACT>
__device__ __forceinline__ float act_grad(float x) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const Logistic l = logistic(x);
    return __fmul_rn(l.s, fmaf(x, l.c, 1.0f));
  }
  if constexpr (ACT == MOE_ACT_GELU) return fmaf(x, __expf(-0.5f * x * x) * 0.3989422804014327f, normal_cdf(x));
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    // x sigma(2 z), z = sqrt(2 / pi) (x + 0.044715 x^3); beyond |x| = 12 sigma is 0 or 1 in fp32
    if (fabsf(x) > 12.0f) return x > 0.0f ? 1.0f : 0.0f;
    const float x2 = x * x;
    const Logistic l = logistic(1.5957691216057308f * fmaf(0.044715f * x2, x, x));
    return fmaf(x * 1.5957691216057308f * fmaf(0.134145f, x2, 1.0f) * l.s, l.c, l.s);
  }
  return 1.0f;
}

// d act'(x), rounded by itself: fused into the column sum in the loop that writes no dpre, it would make dbias
// depend on whether dpre is asked for.  ReLU selects: what it masks is zero, whatever d holds there.
template <int ACT>
__device__ __forceinline__ float act_bwd(float d, float x) {
  if constexpr (ACT == MOE_ACT_NONE) return d;
  if constexpr (ACT == MOE_ACT_RELU) return x <= 0.0f ? 0.0f : d;
  return __fmul_rn(d, act_grad<ACT>(x));
}

__device__ __forceinline__ float ld_shared_cluster(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Rows that a thread loads before it computes: two at 64 registers, four blocks an SM (16384 x 4096, SiLU,
// dbias alone: 67 us; one at a time 89; four at 128 registers 84); four for ReLU's little arithmetic (4096 x
// 2048 with dpre and a 64-column dw 27 us a call, 36 with two).
template <int ACT>
constexpr int kActRows = ACT == MOE_ACT_RELU ? 4 : 2;

template <int ACT>
__global__ void __launch_bounds__(kActThreads, 8 / kActRows<ACT>) act_bwd_kernel(const uint4* __restrict__ dout,
                                                              const float4* __restrict__ pre, long long M, int N,
                                                              int parts, uint4* __restrict__ dpre,
                                                              float* __restrict__ dbias, int accumulate) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRowLanes = kActThreads / 8, R = kActRows<ACT>;
  __shared__ float s_sum[kRowLanes][kActCols + 1];
  __shared__ float s_part[kActCols];
  const int piece = threadIdx.x & 7, rl = threadIdx.x >> 3;
  const int col = blockIdx.x * kActCols + 8 * piece;
  const int part = blockIdx.y;  // the cluster spans the grid's y: rank = blockIdx.y
  const int vpr = N / 8;
  const long long per = (M + parts - 1) / parts;
  const long long lo = part * per, hi = min(M, lo + per);
  float sum[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) sum[c] = 0.0f;
  if (col < N) {
    auto load = [&](long long m, uint4& d, float4 (&p)[2]) {
      const long long o = m * vpr + (col >> 3);
      d = __ldg(dout + o);
      if constexpr (ACT != MOE_ACT_NONE) p[0] = __ldg(pre + 2 * o), p[1] = __ldg(pre + 2 * o + 1);
    };
    auto add = [&](long long m, const uint4& d, const float4 (&p)[2]) {
      const __nv_bfloat162* pd = reinterpret_cast<const __nv_bfloat162*>(&d);
      const float* x = reinterpret_cast<const float*>(p);
      float v[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 f = __bfloat1622float2(pd[c]);
        v[2 * c] = act_bwd<ACT>(f.x, x[2 * c]);
        v[2 * c + 1] = act_bwd<ACT>(f.y, x[2 * c + 1]);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] += v[c];
      if (dpre) {
        uint4 r;
        __nv_bfloat162* pr = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
        for (int c = 0; c < 4; ++c) pr[c] = __floats2bfloat162_rn(v[2 * c], v[2 * c + 1]);
        dpre[m * vpr + (col >> 3)] = r;
      }
    };
    uint4 d[R];
    float4 p[R][2];
    long long m = lo + rl;
    for (; m + (R - 1) * kRowLanes < hi; m += R * kRowLanes) {
#pragma unroll
      for (int r = 0; r < R; ++r) load(m + r * kRowLanes, d[r], p[r]);
#pragma unroll
      for (int r = 0; r < R; ++r) add(m + r * kRowLanes, d[r], p[r]);
    }
    if (m < hi) {  // fewer than R rows are left
#pragma unroll
      for (int r = 0; r < R - 1; ++r)
        if (m + r * kRowLanes < hi) load(m + r * kRowLanes, d[r], p[r]);
#pragma unroll
      for (int r = 0; r < R - 1; ++r)
        if (m + r * kRowLanes < hi) add(m + r * kRowLanes, d[r], p[r]);
    }
  }
  if (!dbias) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) s_sum[rl][8 * piece + c] = sum[c];
  __syncthreads();
  if (threadIdx.x < kActCols) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowLanes; ++i) s += s_sum[i][threadIdx.x];
    s_part[threadIdx.x] = s;
  }
  __syncwarp();
  cluster_sync();
  const int c = blockIdx.x * kActCols + threadIdx.x;
  if (part == 0 && threadIdx.x < kActCols && c < N) {
    const uint32_t mine = smem_u32(&s_part[threadIdx.x]);
    float s = accumulate ? dbias[c] : 0.0f;
    for (int r = 0; r < parts; ++r) s += ld_shared_cluster(mapa_shared(mine, r));
    dbias[c] = s;
  }
  __syncwarp();
  cluster_sync();  // the parts stay in place until they have been read
}

}  // namespace

cudaError_t launch_combine_bwd(const void* dout, const void* y, const int32_t* roa, const float* w, long long T, int H,
                               int K, void* dy, float* dw, cudaStream_t s) {
  if (T == 0 || (!dy && !dw)) return cudaSuccess;
  const int vpr = H / 8;
  // warps a token: enough for 32 warps an SM, but no more than the row has 32-piece steps
  int wpt = 1;
  while (wpt < 8 && T * wpt < 32LL * num_sms() && 32 * wpt < vpr) wpt *= 2;
  const long long tokens = kCombineThreads / 32 / wpt;
  const unsigned blocks = static_cast<unsigned>(std::min<long long>((T + tokens - 1) / tokens, 8LL * num_sms()));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(blocks), dim3(kCombineThreads), 0, s, reinterpret_cast<const uint4*>(dout),
                      reinterpret_cast<const uint4*>(y), roa, w, T, vpr, K, reinterpret_cast<uint4*>(dy), dw);
  };
  if (wpt == 1) return go(combine_bwd_kernel<1>);
  if (wpt == 2) return go(combine_bwd_kernel<2>);
  if (wpt == 4) return go(combine_bwd_kernel<4>);
  return go(combine_bwd_kernel<8>);
}

cudaError_t launch_act_bwd(const void* dout, const float* pre, int act, long long M, int N, void* dpre, float* dbias,
                           int accumulate, cudaStream_t s) {
  if (M == 0 || (!dpre && !dbias)) return cudaSuccess;
  int parts = 1;  // row parts of a cluster, at least 32 rows (one a thread) each
  while (parts < 8 && M > 32LL * parts) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((N + kActCols - 1) / kActCols, parts);
  cfg.blockDim = dim3(kActThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = parts;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  auto go = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, reinterpret_cast<const uint4*>(dout), reinterpret_cast<const float4*>(pre), M,
                              N, parts, reinterpret_cast<uint4*>(dpre), dbias, accumulate);
  };
  switch (act) {
    case MOE_ACT_RELU: return go(act_bwd_kernel<MOE_ACT_RELU>);
    case MOE_ACT_SILU: return go(act_bwd_kernel<MOE_ACT_SILU>);
    case MOE_ACT_GELU: return go(act_bwd_kernel<MOE_ACT_GELU>);
    case MOE_ACT_GELU_TANH: return go(act_bwd_kernel<MOE_ACT_GELU_TANH>);
    default: return go(act_bwd_kernel<MOE_ACT_NONE>);
  }
}

}  // namespace moe
