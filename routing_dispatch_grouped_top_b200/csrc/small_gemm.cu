// small_gemm.cu - products with few output tiles (a decode step's dense layer, small batches, a few
// experts with few rows): one 128 x NT tile a CTA, its reduction split over the CTAs of a cluster, the
// partial sums added over distributed shared memory, the epilogue on the sum.  One launch, no
// workspace.
//
// With few tiles the persistent CTA-pair kernels leave most SMs idle and each reduction runs at one
// SM's load rate (48 KB a K step, about 0.5 us): 16 tokens x 2048 features, K = 7168, is 4 pair tiles.
// Here it is 16 tiles x 8 parts of the reduction, 7.6 us instead of 56 (graph replays of one call; a call
// among others 8.3).  The M side is 128 features of
// the weight (K-major rows, or columns of a [K][features] weight for a gradient with respect to the
// input), the N side up to NT tokens.  A cluster's CTA r takes the K steps [r KB / S, (r + 1) KB / S)
// and then a share of the tile's tokens, whose partial sums it reads from the S CTAs in rank order:
// the result does not depend on timing.  For grouped rows the grid's z covers the most chunks the rows
// can have; each cluster finds its chunk from the offsets, and those behind the last leave at once.
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "epilogue.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxSplit = 8;  // CTAs of a cluster (the portable limit)

// Boxes of a tile of at most NT token rows, in steps of 16.
template <int NT>
constexpr int kFirstBox = NT == 128 ? 1 : (NT == 64 ? 2 : 3);
constexpr int kLastBox = 4;

// kSmallGrad, a weight gradient dw[n][k] = sum over rows r of a[r][n] b[r][k]: the M side is 128 columns
// of b, the N side 64 columns of a (both MN-major), so that a "token" of the epilogue is a row of dw and
// a "feature" its column.  The reduction is over one group's rows: those behind its last one, which may
// be the next group's and hold anything, are overwritten with zeros up to a multiple of 16 (one MMA's
// K) before the last K step's MMAs.  (Rows behind the tensor's last read as zeros.)
enum SmallMode : int { kSmallDense, kSmallGateUp, kSmallDownBwd, kSmallRows, kSmallGrad };

template <int MODE, int NT>
struct Small {
  static constexpr int NA = MODE == kSmallGateUp ? 2 : 1;  // weight operands, one accumulator each
  static constexpr int STAGES = NA == 2 ? 2 : (NT == 32 ? 5 : (NT == 64 ? 4 : 3));  // two CTAs fit an SM
  static constexpr int kStageA = NA * kABytes;
  static constexpr int kStageBytes = kStageA + NT * 128;
  // producer, MMA, epilogue warps (with 4 of these the 1001 x 1544 x 1032 product takes 16.2 us, with 8
  // 15.7, with 12 15.6)
  static constexpr int kThr = NT == 32 ? 192 : 320;
  static constexpr uint32_t kTmemCols = NA * NT;
  static constexpr int kPad = kBM + 4;                 // floats of a staged token row
  static constexpr int kRingBytes = STAGES * kStageBytes;
  static_assert(NA * NT * kPad * 4 <= kRingBytes, "partial sums reuse the ring");
  static constexpr int kBarBytes = 8 * (2 * STAGES + 1) + 16;
  static constexpr int kSmemBytes = 1024 + kRingBytes + kBarBytes;
};

struct SmallMaps {
  CUtensorMap a[2];  // weights: the two operands (kSmallGateUp) or phases (kSmallRows)
  BoxMaps b[2];      // token rows of the phases (kSmallGrad: b[i].box[0], 64 rows x 64 columns of the i-th a)
};

struct SmallArgs {
  const int32_t* offsets;  // [G + 1] or nullptr: one group of M rows
  int G;
  int M;                   // tokens
  int N;                   // features
  int Kd;                  // reduction length of a phase
  int phases;              // kSmallRows: 1 or 2 (weight, token) pairs summed
  int nt;                  // most tokens of a tile (a multiple of 16, at most NT)
  int a_mn;                // the weights are [Kd][N] (features contiguous)
  const float* bias;
  const void* residual;
  int act;
  void* out;               // [M][N] bf16 (kSmallGateUp: h, kSmallDownBwd: dg)
  void* out2;              // kSmallDownBwd: du; kSmallGrad: the second gradient
  float* pre;              // [M][N] fp32 or nullptr (kSmallGateUp: g)
  float* pre1;             // kSmallGateUp: u
  const float* g;          // kSmallDownBwd
  const float* u;
  int rows_out;            // kSmallGrad: rows of a gradient; N: its columns, out: fp32 or bf16
  int cuts;                // kSmallGrad: cuts of its rows; z = (gradient x G + group) x cuts + cut
  int f32;
  int accumulate;          // kSmallGrad, fp32: added to what it holds
  int late_wait;           // kSmallGrad: no operand is written by the kernel before this one
  int* status;
};

// Chunk `slot` of the groups' rows: s_tile = {group, first row, rows}, group -1 behind the last chunk
// or with bad offsets (reported by the first cluster).  One warp.
__device__ void find_chunk(const SmallArgs& args, int slot, bool first, int* s_tile) {
  const int lane = threadIdx.x & 31;
  if (!args.offsets) {
    const int row0 = slot * args.nt;
    if (lane == 0) s_tile[0] = 0, s_tile[1] = row0, s_tile[2] = min(args.nt, args.M - row0);
    return;
  }
  // Offsets must be non-decreasing inside [0, M].
  bool bad = false;
  for (int g = lane; g <= args.G; g += 32) {
    const int o = __ldg(args.offsets + g);
    bad |= o < (g > 0 ? __ldg(args.offsets + g - 1) : 0) || o > args.M;
  }
  bad = __any_sync(0xffffffffu, bad);
  const int seg = (args.G + 31) / 32, lo = min(args.G, lane * seg), hi = min(args.G, lo + seg);
  int sum = 0;
  for (int g = lo; g < hi; ++g)
    sum += (__ldg(args.offsets + g + 1) - __ldg(args.offsets + g) + args.nt - 1) / args.nt;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  if (bad || slot >= total) {
    if (lane == 0) {
      s_tile[0] = -1;
      if (bad && first) report(args.status, MOE_DEV_BAD_INDEX);
    }
    return;
  }
  int c = slot - (incl - sum);
  if (c >= 0 && c < sum) {  // one lane
    for (int g = lo;; ++g) {
      const int a = __ldg(args.offsets + g), cnt = __ldg(args.offsets + g + 1) - a;
      const int n = (cnt + args.nt - 1) / args.nt;
      if (c < n) {
        const int sz = ((cnt + n - 1) / n + 15) & ~15;
        s_tile[0] = g, s_tile[1] = a + c * sz, s_tile[2] = min(sz, cnt - c * sz);
        break;
      }
      c -= n;
    }
  }
}

// Cut `slot` of the weight gradients: s_tile = {group, first row of the gradient, rows of it, which
// gradient, first row of the reduction, rows of it}, group -1 when there is nothing to do.  One warp.
__device__ void find_cut(const SmallArgs& args, int slot, int nt, bool first, int* s_tile) {
  const int lane = threadIdx.x & 31;
  const int ge = slot / args.cuts, m0 = (slot - ge * args.cuts) * nt, which = ge / args.G, g = ge - which * args.G;
  int lo = 0, cnt = args.M;
  bool bad = false;
  if (args.offsets) {  // must be non-decreasing inside [0, M]
    for (int i = lane; i <= args.G; i += 32) {
      const int o = __ldg(args.offsets + i);
      bad |= o < (i > 0 ? __ldg(args.offsets + i - 1) : 0) || o > args.M;
    }
    bad = __any_sync(0xffffffffu, bad);
    lo = __ldg(args.offsets + g), cnt = __ldg(args.offsets + g + 1) - lo;
  }
  if (lane == 0) {
    s_tile[0] = bad || (cnt == 0 && args.accumulate) ? -1 : g;
    s_tile[1] = m0, s_tile[2] = min(nt, args.rows_out - m0);
    s_tile[3] = which, s_tile[4] = lo, s_tile[5] = cnt;
    if (bad && first) report(args.status, MOE_DEV_BAD_INDEX);
  }
}

__device__ __forceinline__ float4 ld_shared_cluster4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

template <int MODE, int NT, int S>
__global__ void __cluster_dims__(S, 1, 1) __launch_bounds__(Small<MODE, NT>::kThr, 2)
    small_kernel(const __grid_constant__ SmallMaps maps, const SmallArgs args) {
  using L = Small<MODE, NT>;
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
  const int rank = blockIdx.x;  // the cluster of S CTAs spans the grid's x
  __shared__ int s_tile[6];
  const int n0 = blockIdx.y * kBM;
  constexpr bool GRAD = MODE == kSmallGrad;

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
    if (lane == 0 || (lane == 1 && (L::NA == 2 || (MODE == kSmallRows && args.phases == 2))))
      tma_prefetch_map(&maps.a[lane]);
    if (GRAD ? lane == 8 : lane >= 8 + kFirstBox<NT> && lane <= 8 + kLastBox) tma_prefetch_map(&maps.b[0].box[lane - 8]);
    if (GRAD && lane == 16 && args.out2) tma_prefetch_map(&maps.b[1].box[0]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  // With late_wait nothing that this kernel reads comes from the kernel before it, and what comes from
  // the kernels before that one was complete when it let this one start.  It only ends after it.
  if (!(GRAD && args.late_wait)) pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    const bool first = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
    if constexpr (GRAD) find_cut(args, blockIdx.z, NT, first, s_tile);
    else find_chunk(args, blockIdx.z, first, s_tile);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int grp = s_tile[0], m0 = s_tile[1], nvalid = s_tile[2], nround = (nvalid + 15) & ~15;
  const int which = GRAD ? s_tile[3] : 0, row0 = GRAD ? s_tile[4] : 0;
  const int red = GRAD ? s_tile[5] : args.Kd;  // length of the reduction
  const int KB1 = (red + kBK - 1) / kBK, KB = KB1 * (MODE == kSmallRows ? args.phases : 1);
  const int kb_lo = rank * KB / S, kb_hi = (rank + 1) * KB / S;  // weight gradients: may be empty
  if (grp < 0) {  // the whole cluster
    if (warp == 1) tmem_dealloc(tmem_base, L::kTmemCols);
    if (GRAD && args.late_wait) pdl_wait();
    return;
  }
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, pend = 0, pend_phase = 0;
      const uint32_t bytes = L::kStageA + (GRAD ? kBK : nround) * 128;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, args.status)) {
          ok = false;
          break;
        }
        uint8_t* st = ring + stage * L::kStageBytes;
        mbar_arrive_expect_tx(&full[stage], bytes);
        const int ph = MODE == kSmallRows && kb >= KB1 ? 1 : 0, kx = (kb - ph * KB1) * kBK;
        if constexpr (GRAD) {
          tma_load_3d(st, &maps.a[0], &full[stage], n0, row0 + kx, 0);
          tma_load_3d(st + kABytes / 2, &maps.a[0], &full[stage], n0 + 64, row0 + kx, 0);
          tma_load_2d(st + L::kStageA, &maps.b[which].box[0], &full[stage], m0, row0 + kx);
        }
#pragma unroll
        for (int i = 0; i < (GRAD ? 0 : L::NA); ++i) {
          const CUtensorMap* m = &maps.a[L::NA == 2 ? i : ph];
          if (args.a_mn) {
            tma_load_3d(st + i * kABytes, m, &full[stage], n0, kx, grp);
            tma_load_3d(st + i * kABytes + kABytes / 2, m, &full[stage], n0 + 64, kx, grp);
          } else {
            tma_load_3d(st + i * kABytes, m, &full[stage], kx, n0, grp);
          }
        }
        int r = 0;
#pragma unroll
        for (int i = kFirstBox<NT>; i <= kLastBox; ++i) {
          const int rows = 256 >> i;
          if (!GRAD && (nround & rows)) {
            tma_load_2d(st + L::kStageA + r * 128, &maps.b[ph].box[i], &full[stage], kx, m0 + r);
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
    const uint32_t idesc =
        idesc_bf16_f32(kBM, nround) | (args.a_mn ? kIdescAMnMajor : 0u) | (GRAD ? kIdescBMnMajor : 0u);
    constexpr uint64_t kDescB = GRAD ? sw128_mnmajor_desc(0, kBK * 128) : sw128_kmajor_desc(0);
    constexpr uint32_t kStepB = (GRAD ? 2048 : 32) >> 4;
    const uint64_t desc_a = args.a_mn ? sw128_mnmajor_desc(0, kABytes / 2) : sw128_kmajor_desc(0);
    const uint32_t step_a = (args.a_mn ? 2048 : 32) >> 4;
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, args.status))) {
        ok = false;
        break;
      }
      int mmas = 4;
      if constexpr (GRAD) {
        const int v = red - kb * kBK, v16 = (v + 15) & ~15;  // rows of this step
        if (args.offsets && v < kBK) {
          mmas = v16 / 16;
          for (int i = lane; i < 3 * (v16 - v) * 8; i += 32) {  // 16-byte pieces of the chunks of 64 columns
            const int c = i / ((v16 - v) * 8), k = i - c * (v16 - v) * 8;
            *reinterpret_cast<uint4*>(ring + stage * L::kStageBytes + c * (kABytes / 2) + v * 128 + k * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_shared();
          __syncwarp();
        }
      }
      tc_fence_after();
      const uint32_t sa = smem_u32(ring + stage * L::kStageBytes);
      // (masked: the address of a CTA other than the cluster's first has bits above the descriptor's field)
      const uint64_t a = desc_a | ((sa >> 4) & 0x3FFFu), b = kDescB | (((sa + L::kStageA) >> 4) & 0x3FFFu);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (GRAD && kk >= mmas) break;
#pragma unroll
        for (int i = 0; i < L::NA; ++i)
          umma_bf16_warp(tmem_base + i * NT, a + i * (kABytes >> 4) + kk * step_a, b + kk * kStepB, idesc,
                         (kb > kb_lo || kk > 0) ? 1u : 0u);
      }
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
  float* part = reinterpret_cast<float*>(ring);  // [operand][token][128 features], rows of kPad
  if (warp >= 2) {
    const int q = warp & 3;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
    for (int i = 0; i < L::NA; ++i)
      for (int j0 = 32 * ((warp - 2) >> 2); j0 < nround; j0 += (L::kThr - 64) / 4) {  // (columns behind nround: not used)
        uint32_t r[32];
        tmem_ld_32cols(tbase + i * NT + j0, r);
        tmem_wait_ld();
        if (GRAD && kb_lo == kb_hi) {  // nothing was summed
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < 16 || j0 + 16 < nround) part[(i * NT + j0 + j) * L::kPad + q * 32 + lane] = __uint_as_float(r[j]);
      }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
  cluster_sync();  // every part is in place

  // This CTA's tokens: one warp a token, a lane holds four consecutive features.  A warp takes two tokens
  // at a time, so that the parts' and the residual's latencies overlap (1001 x 1544 x 1032 with GELU and a
  // residual: 16.5 us one at a time, 15.7 two, 15.9 four).
  const int per = (nvalid + S - 1) / S;
  const int j_hi = min(nvalid, (rank + 1) * per);
  const int f = n0 + 4 * lane;
  const bool f_ok = f < args.N;
  const uint32_t mine = smem_u32(part) + 16 * lane;
  auto store4 = [](void* out, long long o, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(out) + o) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  };
  float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (MODE == kSmallDense) {
    if (args.bias && f_ok)
      bias = make_float4(__ldg(args.bias + f), __ldg(args.bias + f + 1), __ldg(args.bias + f + 2), __ldg(args.bias + f + 3));
  }
  constexpr int U = S == 8 ? 1 : 2, kWarps = L::kThr / 32;
  for (int j0 = rank * per + warp; j0 < j_hi; j0 += U * kWarps) {
    float4 p[U][L::NA][S];
    uint2 res[U];   // kSmallDense: the residual
    float4 g[U], u[U];  // kSmallDownBwd
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int j = j0 + t * kWarps;
      const bool in = j < j_hi;
      const long long o = (static_cast<long long>(m0) + j) * args.N + f;
      if constexpr (MODE == kSmallDense)
        res[t] = in && f_ok && args.residual
                     ? *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(args.residual) + o)
                     : make_uint2(0u, 0u);
      if constexpr (MODE == kSmallDownBwd) {
        g[t] = u[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in && f_ok) {
          g[t] = __ldg(reinterpret_cast<const float4*>(args.g + o));
          u[t] = __ldg(reinterpret_cast<const float4*>(args.u + o));
        }
      }
      if (in) {
#pragma unroll
        for (int i = 0; i < L::NA; ++i)
#pragma unroll
          for (int r = 0; r < S; ++r)
            p[t][i][r] = S == 1 ? *reinterpret_cast<const float4*>(part + (i * NT + j) * L::kPad + 4 * lane)
                                : ld_shared_cluster4(mapa_shared(mine + (i * NT + j) * L::kPad * 4, r));
      }
    }
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int j = j0 + t * kWarps;
      if (j >= j_hi || !f_ok) continue;
      const long long o = ((GRAD ? static_cast<long long>(grp) * args.rows_out : 0LL) + m0 + j) * args.N + f;
      float v[L::NA][4];  // the sums, in rank order
#pragma unroll
      for (int i = 0; i < L::NA; ++i) {
        v[i][0] = p[t][i][0].x, v[i][1] = p[t][i][0].y, v[i][2] = p[t][i][0].z, v[i][3] = p[t][i][0].w;
#pragma unroll
        for (int r = 1; r < S; ++r)
          v[i][0] += p[t][i][r].x, v[i][1] += p[t][i][r].y, v[i][2] += p[t][i][r].z, v[i][3] += p[t][i][r].w;
      }
      if constexpr (MODE == kSmallDense) {
        v[0][0] += bias.x, v[0][1] += bias.y, v[0][2] += bias.z, v[0][3] += bias.w;
        if (args.pre) *reinterpret_cast<float4*>(args.pre + o) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
        activate(v[0], args.act);
        if (args.residual) {
          const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&res[t].x));
          const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&res[t].y));
          v[0][0] += lo.x, v[0][1] += lo.y, v[0][2] += hi.x, v[0][3] += hi.y;
        }
        store4(args.out, o, v[0]);
      } else if constexpr (MODE == kSmallRows) {
        store4(args.out, o, v[0]);
      } else if constexpr (GRAD) {
        void* out = which ? args.out2 : args.out;
        if (!args.f32) {
          store4(out, o, v[0]);
        } else {
          float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + o);
          float4 n = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
          if (args.accumulate) {
            const float4 old = *d;
            n = make_float4(old.x + n.x, old.y + n.y, old.z + n.z, old.w + n.w);
          }
          *d = n;
        }
      } else if constexpr (MODE == kSmallGateUp) {
        *reinterpret_cast<float4*>(args.pre + o) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
        *reinterpret_cast<float4*>(args.pre1 + o) = make_float4(v[1][0], v[1][1], v[1][2], v[1][3]);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[0][c] = swiglu(v[0][c], v[1][c]);
        store4(args.out, o, v[0]);
      } else {
        const float gv[4] = {g[t].x, g[t].y, g[t].z, g[t].w}, uv[4] = {u[t].x, u[t].y, u[t].z, u[t].w};
        float dg[4], du[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) swiglu_grad(v[0][c], gv[c], uv[c], dg[c], du[c]);
        store4(args.out, o, dg);
        store4(args.out2, o, du);
      }
    }
  }
  __syncwarp();
  cluster_sync();  // the parts stay in place until every CTA has read them
  if (GRAD && args.late_wait) pdl_wait();
}

template <int MODE, int NT, int S>
cudaError_t launch_split(const SmallMaps& maps, const SmallArgs& args, long long chunks, cudaStream_t stream) {
  using L = Small<MODE, NT>;
  static std::atomic<int> attr_done[kMaxDevices] = {};
  const cudaError_t err =
      smem_attr_once(reinterpret_cast<const void*>(small_kernel<MODE, NT, S>), L::kSmemBytes, attr_done);
  if (err != cudaSuccess) return err;
  return launch_pdl(small_kernel<MODE, NT, S>, dim3(S, (args.N + kBM - 1) / kBM, static_cast<unsigned>(chunks)),
                    dim3(L::kThr), L::kSmemBytes, stream, maps, args);
}

// S, a power of two up to kMaxSplit: the parts of the reduction.  128-token tiles are taken where 64-token
// ones would be more than the SMs, which leaves room for two parts at most (split_parts).
template <int MODE, int NT>
cudaError_t launch_small(const SmallMaps& maps, const SmallArgs& args, long long chunks, int S, cudaStream_t stream) {
  if (S == 1) return launch_split<MODE, NT, 1>(maps, args, chunks, stream);
  if constexpr (NT < 128) {
    if (S == 4) return launch_split<MODE, NT, 4>(maps, args, chunks, stream);
    if (S == kMaxSplit) return launch_split<MODE, NT, kMaxSplit>(maps, args, chunks, stream);
  }
  return launch_split<MODE, NT, 2>(maps, args, chunks, stream);
}

// Parts of the reduction for `tiles` tiles of KB K steps: as many as fill the SMs twice (two CTAs fit
// one), at least two K steps each (16 x 2048 x 7168: 34 us unsplit, 19, 11 and 7.8 us in 2, 4 and 8).
int split_parts(long long tiles, int KB) {
  int S = 1;
  for (const long long sms = num_sms(); S < kMaxSplit && tiles * S <= sms && KB >= 4 * S;) S *= 2;
  return S;
}

// Grouped rows: chunks of 64.  The launch covers the most there can be, the split is chosen for the
// fewest (a few large groups, or as many chunks as groups).
template <int MODE>
cudaError_t launch_grouped(const SmallMaps& maps, SmallArgs& args, long long rows, int KB, cudaStream_t stream) {
  args.nt = 64;
  const long long groups = std::min<long long>(args.G, rows), ftiles = (args.N + kBM - 1) / kBM;
  const long long least = std::max((rows + 63) / 64, groups), most = rows / 64 + groups;
  return launch_small<MODE, 64>(maps, args, most, split_parts(least * ftiles, KB), stream);
}

}  // namespace

bool dense_small_fits(long long M, int N) {
  // Pair tiles of 512 features x 256 tokens that would run: below half of the pairs these kernels are
  // faster (2048 x 2048 x 1024, 32 tiles: 13.6 us against 14.4; 2048 x 2560 x 512, 40 tiles: 17.6
  // against 11.7).
  const long long tiles = ((M + 255) / 256) * ((N + 511) / 512);
  return tiles * 2 < num_sms() / 2;
}

// The same for the rows of `groups` experts, below a third of the pairs (chunks of 64 rows re-read the
// weights more often: 1824 rows of one expert, 1728 x 960, 122 us a step, 139 with half); `feat` features
// a pair tile.
bool grouped_small_fits(long long rows, int groups, int N, int feat) {
  const long long tiles = std::max<long long>((rows + 255) / 256, std::min<long long>(groups, rows)) * ((N + feat - 1) / feat);
  // Few rows a group make both kinds read each weight once: then up to one pair tile an SM (136 x 8 rows
  // of 109 experts 230 -> 205 us a training step; with more rows the pair tiles re-read less).
  return tiles * 3 < num_sms() / 2 || (rows <= 48 * std::min<long long>(groups, rows) && tiles < num_sms());
}

cudaError_t dense_small(const void* a, const void* w, int w_mn, const float* bias, const void* residual, int act,
                        long long M, int N, int Kd, void* out, float* pre, int* status, cudaStream_t stream) {
  // Tokens of a tile: 64 rather than 128 while such tiles fit the SMs (the exchange of partial sums is
  // then spread over more CTAs: 256 x 2048 x 2048 11.2 -> 8.8 us; beyond that they only re-read the
  // weights: 1001 x 1544 x 4096 22 -> 28 us).
  const long long ftiles = (N + kBM - 1) / kBM;
  const int most = M <= 32 ? 32 : ((M + 63) / 64 * ftiles <= num_sms() ? 64 : 128);
  SmallMaps m;
  if (!(w_mn ? map_bf16_3d(&m.a[0], w, N, Kd, 1, kBK) : map_bf16_3d(&m.a[0], w, Kd, N, 1, kBM)) ||
      !map_token_boxes(&m.b[0], a, Kd, M, 2, most == 32 ? kFirstBox<32> : (most == 64 ? kFirstBox<64> : kFirstBox<128>),
                       kLastBox))
    return cudaErrorInvalidValue;
  SmallArgs args{};
  args.G = 1, args.M = static_cast<int>(M), args.N = N, args.Kd = Kd, args.phases = 1, args.a_mn = w_mn, args.bias = bias;
  args.residual = residual, args.act = act, args.out = out, args.pre = pre, args.status = status;
  const long long cut = (M + most - 1) / most;
  args.nt = static_cast<int>(((M + cut - 1) / cut + 15) / 16 * 16);
  const long long chunks = (M + args.nt - 1) / args.nt;
  const int S = split_parts(chunks * ftiles, (Kd + kBK - 1) / kBK);
  if (most == 32) return launch_small<kSmallDense, 32>(m, args, chunks, S, stream);
  return most == 64 ? launch_small<kSmallDense, 64>(m, args, chunks, S, stream)
                    : launch_small<kSmallDense, 128>(m, args, chunks, S, stream);
}

cudaError_t small_gate_up_train(const void* xp, const int32_t* offsets, const void* w_gate, const void* w_up, int E,
                                long long rows, int H, int F, float* g, float* u, void* h, int* status,
                                cudaStream_t stream) {
  SmallMaps m;
  if (!map_bf16_3d(&m.a[0], w_gate, H, F, E, kBM) || !map_bf16_3d(&m.a[1], w_up, H, F, E, kBM) ||
      !map_token_boxes(&m.b[0], xp, H, rows, 2, kFirstBox<64>, kLastBox))
    return cudaErrorInvalidValue;
  SmallArgs args{};
  args.offsets = offsets, args.G = E, args.M = static_cast<int>(rows), args.N = F, args.Kd = H, args.phases = 1;
  args.out = h, args.pre = g, args.pre1 = u, args.status = status;
  return launch_grouped<kSmallGateUp>(m, args, rows, (H + kBK - 1) / kBK, stream);
}

cudaError_t small_down_bwd(const void* dy, const float* g, const float* u, const int32_t* offsets, const void* w_down,
                           int E, long long rows, int H, int F, void* dg, void* du, int* status, cudaStream_t stream) {
  SmallMaps m;
  if (!map_bf16_3d(&m.a[0], w_down, F, H, E, kBK) || !map_token_boxes(&m.b[0], dy, H, rows, 2, kFirstBox<64>, kLastBox)) return cudaErrorInvalidValue;
  SmallArgs args{};
  args.offsets = offsets, args.G = E, args.M = static_cast<int>(rows), args.N = F, args.Kd = H, args.phases = 1;
  args.a_mn = 1, args.out = dg, args.out2 = du, args.g = g, args.u = u, args.status = status;
  return launch_grouped<kSmallDownBwd>(m, args, rows, (H + kBK - 1) / kBK, stream);
}

cudaError_t small_rows_bwd(const void* d0, const void* d1, const int32_t* offsets, const void* w0, const void* w1, int G,
                           long long rows, int N, int Kd, void* out, int* status, cudaStream_t stream) {
  SmallMaps m;
  if (!map_bf16_3d(&m.a[0], w0, N, Kd, G, kBK) || !map_token_boxes(&m.b[0], d0, Kd, rows, 2, kFirstBox<64>, kLastBox) ||
      !map_bf16_3d(&m.a[1], w1, N, Kd, G, kBK) || !map_token_boxes(&m.b[1], d1, Kd, rows, 2, kFirstBox<64>, kLastBox))
    return cudaErrorInvalidValue;
  SmallArgs args{};
  args.offsets = offsets, args.G = G, args.M = static_cast<int>(rows), args.N = N, args.Kd = Kd, args.phases = 2;
  args.a_mn = 1, args.out = out, args.status = status;
  return launch_grouped<kSmallRows>(m, args, rows, 2 * ((Kd + kBK - 1) / kBK), stream);
}

// Weight gradients of few pair tiles: those would leave most SMs idle and cannot share an SM with the
// input gradient's CTAs, which these can (a dense layer's whole backward, 3417 x 616 x 880: 70 -> 51 us; 54 x
// 1024 x 1024: 15.2 -> 8.8; 200 x 520 x 776: 19.5 -> 9.8; experts' backward, 8 x 16 rows, 256 x 512: 19.1 ->
// 18.3, 16 x 256 rows, 256 x 256: 33.7 -> 29.2; at half the pairs, 4 x 256 rows, 1024 x 1024: 44.9 -> 47.0).
bool grad_small_fits(int groups, int N, int Kd, int feat) {
  const long long tiles = static_cast<long long>(groups) * ((N + feat - 1) / feat) * ((Kd + 255) / 256);
  return tiles * 3 < num_sms() / 2;
}

cudaError_t small_grad(const void* a0, const void* a1, const void* b, const int32_t* offsets, int G, long long rows,
                       int N, int Kd, void* dw0, void* dw1, int f32, int accumulate, int late_wait, int* status,
                       cudaStream_t stream) {
  SmallMaps m;
  if (!map_bf16_3d(&m.a[0], b, Kd, rows, 1, kBK) || !map_bf16_2d(&m.b[0].box[0], a0, N, rows, kBK) ||
      (a1 && !map_bf16_2d(&m.b[1].box[0], a1, N, rows, kBK)))
    return cudaErrorInvalidValue;
  SmallArgs args{};
  args.offsets = offsets, args.G = G, args.M = static_cast<int>(rows), args.N = Kd, args.phases = 1, args.a_mn = 1;
  args.nt = 64, args.rows_out = N, args.cuts = (N + 63) / 64, args.out = dw0, args.out2 = dw1, args.f32 = f32;
  args.accumulate = accumulate, args.late_wait = late_wait, args.status = status;
  const long long z = static_cast<long long>(a1 ? 2 : 1) * G * args.cuts;
  const int KB = static_cast<int>((rows / G + kBK) / kBK);  // of an average group
  return launch_small<kSmallGrad, 64>(m, args, z, split_parts(z * ((Kd + kBM - 1) / kBM), KB), stream);
}

}  // namespace moe
