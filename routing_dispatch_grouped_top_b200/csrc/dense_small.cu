// dense_small.cu - products with few output tiles (a decode step's dense layer, small batches): one
// 128 x NT tile a CTA, its reduction split over the CTAs of a cluster, the partial sums added over
// distributed shared memory, the epilogue of moe_dense_epilogue on the sum.  One launch, no workspace.
//
// With few tiles the persistent CTA-pair kernel leaves most SMs idle and each reduction runs at one
// SM's load rate: 16 tokens x 2048 features, K = 7168, is 4 pair tiles.  Here it is 16 tiles x 8 parts
// of the reduction.  The M side is 128 features of the weight (K-major rows, or columns of a
// [K][features] weight for a gradient with respect to the input), the N side up to NT tokens.
// A cluster's CTA r takes the K steps [r KB / S, (r + 1) KB / S) and then a share of the tile's tokens,
// whose partial sums it reads from the S CTAs in rank order: the result does not depend on timing.
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "epilogue.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxSplit = 8;  // CTAs of a cluster (the portable limit)

template <int NT>
struct Small {
  static constexpr int STAGES = NT == 32 ? 5 : (NT == 64 ? 4 : 3);  // two CTAs fit an SM
  static constexpr int kBBytes = NT * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kThr = 192;                     // producer, MMA, four epilogue warps
  static constexpr uint32_t kTmemCols = NT;
  static constexpr int kPad = kBM + 4;                 // floats of a staged token row
  static constexpr int kRingBytes = STAGES * kStageBytes;
  static_assert(NT * kPad * 4 <= kRingBytes, "partial sums reuse the ring");
  static constexpr int kBarBytes = 8 * (2 * STAGES + 1) + 16;
  static constexpr int kSmemBytes = 1024 + kRingBytes + kBarBytes;
};

struct SmallArgs {
  int M;             // tokens
  int N;             // features
  int Kd;
  int nt;            // tokens of a tile (a multiple of 16, at most NT)
  int a_mn;          // the weight is [Kd][N] (features contiguous)
  const float* bias;
  const void* residual;
  int act;
  void* out;         // [M][N] bf16
  float* pre;        // [M][N] fp32 or nullptr
  int* status;
};

__device__ __forceinline__ float4 ld_shared_cluster4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

template <int NT>
__global__ void __launch_bounds__(Small<NT>::kThr, 2)
    small_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BoxMaps tmB, const SmallArgs args) {
  using L = Small<NT>;
  constexpr int STAGES = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kRingBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = gridDim.x, rank = blockIdx.x;  // the cluster spans the grid's x
  const int n0 = blockIdx.y * kBM, m0 = blockIdx.z * args.nt;
  const int nvalid = min(args.nt, args.M - m0), nround = (nvalid + 15) & ~15;
  const int KB = (args.Kd + kBK - 1) / kBK;
  const int kb_lo = rank * KB / S, kb_hi = (rank + 1) * KB / S;  // the host keeps S <= KB

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) {
    if (lane == 0) tma_prefetch_map(&tmA);
    if (lane >= 1 && lane < kNumBoxes) tma_prefetch_map(&tmB.box[lane]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, pend = 0, pend_phase = 0;
      const uint32_t bytes = kABytes + nround * 128;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, args.status)) {
          ok = false;
          break;
        }
        uint8_t* st = ring + stage * L::kStageBytes;
        mbar_arrive_expect_tx(&full[stage], bytes);
        const int kx = kb * kBK;
        if (args.a_mn) {
          tma_load_3d(st, &tmA, &full[stage], n0, kx, 0);
          tma_load_3d(st + kABytes / 2, &tmA, &full[stage], n0 + 64, kx, 0);
        } else {
          tma_load_3d(st, &tmA, &full[stage], kx, n0, 0);
        }
        int r = 0;
#pragma unroll
        for (int i = 1; i < kNumBoxes; ++i) {
          const int rows = 256 >> i;
          if (nround & rows) {
            tma_load_2d(st + kABytes + r * 128, &tmB.box[i], &full[stage], kx, m0 + r);
            r += rows;
          }
        }
        pend |= 1u << stage;
        pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok)
        for (int s = 0; s < STAGES; ++s)
          if (pend >> s & 1u) mbar_drain(&full[s], pend_phase >> s & 1u, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0;
    const uint32_t idesc = idesc_bf16_f32(kBM, nround) | (args.a_mn ? kIdescAMnMajor : 0u);
    const uint64_t desc_a = args.a_mn ? sw128_mnmajor_desc(0, kABytes / 2) : sw128_kmajor_desc(0);
    const uint32_t step_a = (args.a_mn ? 2048 : 32) >> 4;
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, args.status))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t sa = smem_u32(ring + stage * L::kStageBytes);
      // (masked: the address of a CTA other than the cluster's first has bits above the descriptor's field)
      const uint64_t a = desc_a | ((sa >> 4) & 0x3FFFu), b = sw128_kmajor_desc(sa + kABytes);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_bf16_warp(tmem_base, a + kk * step_a, b + kk * 2, idesc, (kb > kb_lo || kk > 0) ? 1u : 0u);
      umma_commit_warp(&empty[stage]);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    umma_commit_warp(done);
    if (!ok && lane == 0) mbar_drain(done, 0, 200000000ull);
    __syncwarp();
  }
  // Every warp waits for the sums (after an abort: until it is seen), which also ends the ring's use.
  ok = mbar_wait(done, 0, abort_flag, args.status) && ok;
  __syncthreads();
  tc_fence_after();
  float* part = reinterpret_cast<float*>(ring);  // [token][128 features], rows of kPad
  if (warp >= 2) {
    const int q = warp & 3;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    for (int j0 = 0; j0 < nround; j0 += 16) {
      uint32_t r[16];
      tmem_ld_16cols(tbase + j0, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(j0 + j) * L::kPad + q * 32 + lane] = __uint_as_float(r[j]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
  cluster_sync();  // every part is in place

  // This CTA's tokens: one warp a token, a lane holds four consecutive features.
  const int per = (nvalid + S - 1) / S;
  const int j_hi = min(nvalid, (rank + 1) * per);
  const int f = n0 + 4 * lane;
  const uint32_t mine = smem_u32(part) + 16 * lane;
  float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
  if (args.bias && f < args.N)
    bias = make_float4(__ldg(args.bias + f), __ldg(args.bias + f + 1), __ldg(args.bias + f + 2), __ldg(args.bias + f + 3));
  for (int j = rank * per + warp; j < j_hi; j += L::kThr / 32) {
    const long long o = (static_cast<long long>(m0) + j) * args.N + f;
    uint2 rv = make_uint2(0u, 0u);
    if (args.residual && f < args.N)
      rv = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(args.residual) + o);
    float4 p[kMaxSplit];
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r)
      if (r < S) p[r] = ld_shared_cluster4(mapa_shared(mine + j * L::kPad * 4, r));
    float v[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
#pragma unroll
    for (int r = 1; r < kMaxSplit; ++r)
      if (r < S) v[0] += p[r].x, v[1] += p[r].y, v[2] += p[r].z, v[3] += p[r].w;
    v[0] += bias.x, v[1] += bias.y, v[2] += bias.z, v[3] += bias.w;
    if (f < args.N) {
      if (args.pre) *reinterpret_cast<float4*>(args.pre + o) = make_float4(v[0], v[1], v[2], v[3]);
      activate(v, args.act);
      const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&rv.x));
      const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&rv.y));
      if (args.residual) v[0] += lo.x, v[1] += lo.y, v[2] += hi.x, v[3] += hi.y;
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(args.out) + o) =
          make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
  }
  __syncwarp();
  cluster_sync();  // the parts stay in place until every CTA has read them
}

template <int NT>
cudaError_t launch_small(const CUtensorMap& a, const BoxMaps& b, const SmallArgs& args, int S, cudaStream_t stream) {
  using L = Small<NT>;
  static std::atomic<int> attr_done[kMaxDevices] = {};
  const cudaError_t err = smem_attr_once(reinterpret_cast<const void*>(small_kernel<NT>), L::kSmemBytes, attr_done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, (args.N + kBM - 1) / kBM, (args.M + args.nt - 1) / args.nt);
  cfg.blockDim = dim3(L::kThr);
  cfg.dynamicSmemBytes = L::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, small_kernel<NT>, a, b, args);
}

}  // namespace

bool dense_small_fits(long long M, int N) {
  // Pair tiles of 512 features x 256 tokens that would run: below a third of the pairs these kernels
  // are faster (16 tiles, 512 x 4096 x 2048: 16 us against 25 us; 28 to 36 tiles: 3 % slower).
  const long long tiles = ((M + 255) / 256) * ((N + 511) / 512);
  return tiles * 3 < num_sms() / 2;
}

cudaError_t dense_small(const void* a, const void* w, int w_mn, const float* bias, const void* residual, int act,
                        long long M, int N, int Kd, void* out, float* pre, int* status, cudaStream_t stream) {
  CUtensorMap ta;
  BoxMaps tb;
  if (!(w_mn ? map_bf16_3d(&ta, w, N, Kd, 1, kBK) : map_bf16_3d(&ta, w, Kd, N, 1, kBM)) ||
      !map_token_boxes(&tb, a, Kd, M))
    return cudaErrorInvalidValue;
  SmallArgs args{};
  args.M = static_cast<int>(M), args.N = N, args.Kd = Kd, args.a_mn = w_mn, args.bias = bias, args.residual = residual;
  args.act = act, args.out = out, args.pre = pre, args.status = status;
  // Tokens of a tile: 64 rather than 128 while such tiles fit the SMs (the exchange of partial sums is
  // then spread over more CTAs: 256 x 2048 x 2048 11.2 -> 8.8 us; beyond that they only re-read the
  // weights: 1001 x 1544 x 4096 22 -> 28 us).
  const long long ftiles = (N + kBM - 1) / kBM;
  const int most = M <= 32 ? 32 : ((M + 63) / 64 * ftiles <= num_sms() ? 64 : 128);
  const long long chunks = (M + most - 1) / most;
  args.nt = static_cast<int>(((M + chunks - 1) / chunks + 15) / 16 * 16);
  // Parts of the reduction: as many as fill the SMs twice (two CTAs fit one), at least two K steps each
  // (16 x 2048 x 7168: 34 us unsplit, 19, 11 and 7.8 us in 2, 4 and 8 parts).
  const long long tiles = (M + args.nt - 1) / args.nt * ftiles;
  const int KB = (Kd + kBK - 1) / kBK;
  int S = 1;
  while (S < kMaxSplit && tiles * S * 2 <= 2LL * num_sms() && KB >= 4 * S) S *= 2;
  if (most == 32) return launch_small<32>(ta, tb, args, S, stream);
  return most == 64 ? launch_small<64>(ta, tb, args, S, stream) : launch_small<128>(ta, tb, args, S, stream);
}

}  // namespace moe
