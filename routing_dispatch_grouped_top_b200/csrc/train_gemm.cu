// train_gemm.cu - the matrix products of the layer's training pass and of the dense product with a
// fused epilogue: persistent, warp-specialised tcgen05 kernels on CTA pairs (cta_group::2).
//
// With g = xp Wg^T, u = xp Wu^T, h = silu(g) u, y = h Wd^T for the rows of each expert, and dy
// the gradient of y:
//   dh  = dy Wd                   dg = dh u s (1 + g (1 - s)),  du = dh g s,  s = 1 / (1 + e^-g)
//   dxp = dg Wg + du Wu           dWg = dg^T xp,  dWu = du^T xp,  dWd = dy^T h   (per expert)
// Every product reads its operands as they lie in memory, none is transposed first: the tensor
// core takes an operand whose M or N index is contiguous (MN-major) as well as one whose K index
// is (K-major).
//
//   mode          M side (256 or 512 a tile)      N side                 K          epilogue
//   kGateUpTrain  Wg, Wu rows (K-major)           xp rows (K-major)      H          g, u (fp32), h
//   kDownBwd      Wd columns (MN-major)           dy rows (K-major)      H          dg, du from g, u
//   kRowsBwd      Wg, Wu columns (MN-major)       dg, du rows (K-major)  F, twice   dxp
//   kGradGateUp   dg, du columns (MN-major)       xp columns (MN-major)  rows of e  dWg, dWu
//   kGradDown     dy columns (MN-major)           h columns (MN-major)   rows of e  dWd
//   kDense        w rows (K-major)                a rows (K-major)       Kd         bias, act, residual
//
// dg and du are rounded to bf16 (as h is) because they are operands of the next products; all
// sums are fp32 in TMEM.  The pre-activations g and u are kept in fp32: with bf16 copies their
// rounding would add to that of dg and du.
//
// The weight gradients reduce over an expert's rows, whose number is not a multiple of the K step
// (64 rows).  The rows behind the last one belong to the next expert and may hold anything, NaN
// included, so they must be zeros in shared memory and not merely zeros in one operand: the last
// K step is fetched with boxes of 32, 16, 8, 4, 2 and 1 rows that cover exactly the expert's rows,
// then with boxes of 1, 2, 4 and 8 rows that start behind the tensor's last row (TMA fills those
// with zeros) up to a multiple of 16 rows, one MMA's K.  The same two CTAs' producers issue them,
// so no other warp has to touch the stage.
//
// Roles per CTA: warp 0 TMA producer (the leader claims tiles from the workspace's counter),
// warp 1 MMA issuer (leader) and TMEM owner, warps 2-9 epilogue.  Tiles are numbered group-major,
// so that CTAs working at the same time share operand tiles through L2.
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {

namespace {

enum Mode : int { kGateUpTrain, kDownBwd, kRowsBwd, kGradGateUp, kGradDown, kDense };

constexpr int kNumRowBoxes = 7;  // boxes of 64, 32, 16, 8, 4, 2, 1 rows
struct RowMaps {
  CUtensorMap box[kNumRowBoxes];  // box[i] is (64 >> i) rows x 64 columns
};
struct TokenMaps {   // products with a row of tokens on the N side
  CUtensorMap a[2];  // weights
  BoxMaps b[2];      // token rows
  CUtensorMap o;     // output tiles (kRowsBwd)
};
struct GradMaps {    // weight gradients: reduction over an expert's rows
  RowMaps a[2];
  RowMaps b;
  CUtensorMap o[2];
};

template <int MODE>
struct Prod {
  static constexpr bool GRAD = MODE == kGradGateUp || MODE == kGradDown;
  static constexpr bool A_MN = MODE != kGateUpTrain && MODE != kDense;  // M side contiguous in memory
  static constexpr bool TWO_A = MODE == kGateUpTrain || MODE == kGradGateUp;  // two weight operands, one N tile
  using Maps = std::conditional_t<GRAD, GradMaps, TokenMaps>;
  static constexpr int NT = 256;                      // N of a tile
  static constexpr int FEAT = TWO_A ? 256 : 512;      // M of a tile (of each operand)
  static constexpr int STAGES = 4;
  static constexpr int EW = 8;                        // epilogue warps
  static constexpr int kThr = 64 + 32 * EW;
  static constexpr int kStageA = 2 * kABytes;         // this CTA's two 128 x 64 M-side tiles
  static constexpr int kStageB = (NT / 2) * 128;      // this CTA's half of the N side
  static constexpr int kStageBytes = kStageA + kStageB;
  // epilogue staging of a warp: fp32 16 x 32 (rows padded to 36), bf16 32 x 32, or 32 rows of 128 B
  static constexpr int kStgWarp = GRAD ? 4096 : (MODE == kRowsBwd ? 2048 : 16 * 36 * 4);
  static constexpr int kStgBytes = EW * kStgWarp;
  static constexpr int kBarBytes = (8 * (2 * STAGES + 3 + 2 * kRing) + 8 + 4 * kRing + 15) / 16 * 16;
  static constexpr int kTableBytes = GRAD ? 0 : 2 * (kMaxGroups + 1) * 4;
  static constexpr int kSmemBytes = 1024 + STAGES * kStageBytes + kStgBytes + kBarBytes + kTableBytes;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct ProdArgs {
  const int32_t* offsets;  // [G + 1] or nullptr: one group of M rows
  int G;
  int M;                   // rows of the token operands
  int N;                   // output features (token modes), rows of a weight gradient
  int Kd;                  // reduction length of one phase (token modes), columns of a weight gradient
  int phases;              // kRowsBwd: 1 or 2 (weight, token) operand pairs summed
  void* out;               // kRowsBwd, kDense: [M][N] bf16; kGateUpTrain: h; kDownBwd: dg
  void* out2;              // kDownBwd: du
  float* pre0;             // kGateUpTrain: g out; kDense: pre-activation out or nullptr
  float* pre1;             // kGateUpTrain: u out
  const float* g;          // kDownBwd
  const float* u;
  const float* bias;       // kDense: [N] or nullptr
  const void* residual;    // kDense: [M][N] bf16 or nullptr
  int act;                 // kDense: moe_act
  int grad_f32;            // weight gradients in fp32 (else bf16)
  int accumulate;          // added to what the gradients hold
  int* status;
  int* sched;              // two device ints {next tile, finished CTAs}, zero between launches
};

// The K extent of weight-gradient tile g: rows [row0, row0 + cnt).
struct GradTile {
  int g, n0, k0, row0, cnt;
};

template <int FEAT, int NT>
__device__ __forceinline__ GradTile decode_grad(int t, const ProdArgs& a, int nft, int nkt) {
  GradTile r;
  r.g = t / (nft * nkt);
  const int local = t - r.g * nft * nkt;
  r.n0 = (local / nkt) * FEAT;
  r.k0 = (local % nkt) * NT;
  if (a.offsets) {
    r.row0 = __ldg(a.offsets + r.g);
    r.cnt = __ldg(a.offsets + r.g + 1) - r.row0;
  } else {
    r.row0 = 0;
    r.cnt = a.M;
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Logistic function with the fast exponential and divide; the quotient's denominator overflows to
// a result of 0 for g -> -inf.
__device__ __forceinline__ float fast_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case MOE_ACT_RELU: return x < 0.0f ? 0.0f : x;  // NaN stays NaN
    case MOE_ACT_SILU: return __fdividef(x, 1.0f + __expf(-x));
    case MOE_ACT_GELU: return x * normcdff(x);
    case MOE_ACT_GELU_TANH:
      return x * fast_sigmoid(1.5957691216057308f * (x + 0.044715f * x * x * x));
    default: return x;
  }
}

// A warp's accumulator columns [col, col + 16) (16 tokens) of its 32 lanes (features) go through
// its staging tile [16][36] fp32 so that each lane then holds 8 consecutive features of two
// tokens, lane / 4 and lane / 4 + 8 (rows padded to 36 floats: no bank conflicts either way).
__device__ __forceinline__ void stage16(float* stg, int lane, uint32_t taddr) {
  uint32_t r[16];
  __syncwarp();  // the staged values of the previous call have been read
  tmem_ld_16cols(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 16; ++j) stg[j * 36 + lane] = __uint_as_float(r[j]);
  __syncwarp();
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Prod<MODE>::kThr, 1)
    prod_kernel(const __grid_constant__ typename Prod<MODE>::Maps maps, const ProdArgs args) {
  using P = Prod<MODE>;
  constexpr int STAGES = P::STAGES, EW = P::EW, NT = P::NT;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* stg_all = smem + STAGES * P::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + P::kStgBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tempty + 1;
  uint64_t* rfull = drain + 1;
  uint64_t* rempty = rfull + kRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rempty + kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* ring_tile = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* s_off = reinterpret_cast<int*>(stg_all + P::kStgBytes + P::kBarBytes);  // token modes only
  int* s_pre = s_off + (kMaxGroups + 1);
  __shared__ int s_warp_sums[P::kThr / 32];
  __shared__ int s_bad;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int G = args.offsets ? args.G : 1;
  const int NFT = (args.N + P::FEAT - 1) / P::FEAT;
  const int NKT = (args.Kd + NT - 1) / NT;              // weight gradients: column tiles
  const int KB1 = (args.Kd + kBK - 1) / kBK;            // token modes: K steps of a phase

  if (threadIdx.x == 0) {
    s_bad = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * EW);
    mbar_init(drain, 1);
    for (int r = 0; r < kRing; ++r) {
      mbar_init(&rfull[r], 1);
      mbar_init(&rempty[r], 2 + 2 * EW);  // leader MMA, peer producer, both CTAs' epilogue warps
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  pdl_wait();  // offsets and operands come from earlier kernels
  pdl_launch_dependents();
  __syncthreads();
  // Offsets must be non-decreasing inside [0, M]; otherwise no tile runs.
  if constexpr (P::GRAD) {
    if (args.offsets)
      for (int i = threadIdx.x; i <= G; i += P::kThr) {
        const int o = __ldg(args.offsets + i);
        if (o < 0 || o > args.M || (i > 0 && o < __ldg(args.offsets + i - 1))) s_bad = 1;
      }
    __syncthreads();
    if (s_bad && threadIdx.x == 0 && rank == 0) report(args.status, MOE_DEV_BAD_INDEX);
  } else {
    for (int i = threadIdx.x; i <= G; i += P::kThr)
      s_off[i] = args.offsets ? __ldg(args.offsets + i) : (i == 0 ? 0 : args.M);
    __syncthreads();
    for (int i = threadIdx.x; i <= G; i += P::kThr)
      if (s_off[i] < 0 || s_off[i] > args.M || (i > 0 && s_off[i] < s_off[i - 1])) s_bad = 1;
    __syncthreads();
    if (s_bad) {
      if (threadIdx.x == 0 && rank == 0) report(args.status, MOE_DEV_BAD_INDEX);
      for (int i = threadIdx.x; i <= G; i += P::kThr) s_off[i] = 0;
    }
    __syncthreads();
    build_tile_table(s_pre, s_off, G, NT, NFT, s_warp_sums);
  }
  cluster_sync();  // both CTAs' barriers exist before any access over the cluster
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = P::GRAD ? (s_bad ? 0 : G * NFT * NKT) : s_pre[G];
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
  const uint32_t rempty_leader = mapa_shared(smem_u32(rempty), 0);
  const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      const uint32_t rfull_peer = mapa_shared(smem_u32(rfull), 1);
      const uint32_t ring_peer = mapa_shared(smem_u32(const_cast<int*>(ring_tile)), 1);
      uint32_t stage = 0, phase = 0, rs = 0, rphase = 0;
      uint32_t pend = 0, pend_phase = 0;  // one bit a stage
      bool ok = true;
      // Waits for the stage to be free, announces its bytes (both CTAs') and returns its buffer.
      auto acquire = [&](uint32_t bytes) -> uint8_t* {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, args.status)) return nullptr;
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2u * bytes);
        return ring + stage * P::kStageBytes;
      };
      auto advance = [&] {
        pend |= 1u << stage;
        pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      };
      for (;;) {
        int t;
        if (rank == 0) {
          if (!mbar_wait_cluster(&rempty[rs], rphase ^ 1u, abort_flag, args.status)) {
            ok = false;
            break;
          }
          const int claimed = atomicAdd(&args.sched[0], 1);
          t = claimed < total ? claimed : -1;
          ring_tile[rs] = t;
          st_shared_cluster(ring_peer + 4 * rs, t);
          mbar_arrive(&rfull[rs]);
          mbar_arrive_cluster(rfull_peer + 8 * rs);
        } else {
          if (!mbar_wait_cluster(&rfull[rs], rphase, abort_flag, args.status)) {
            ok = false;
            break;
          }
          t = ring_tile[rs];
          mbar_arrive_cluster(rempty_leader + 8 * rs);
        }
        if (++rs == kRing) {
          rs = 0;
          rphase ^= 1u;
        }
        if (t < 0) break;
        if constexpr (P::GRAD) {
          const GradTile tl = decode_grad<P::FEAT, NT>(t, args, NFT, NKT);
          const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          const int half = args.Kd - tl.k0 > 128 ? 128 : 64;  // N columns staged by each CTA
          const int fr = tl.n0 + 128 * static_cast<int>(rank);
          const int kc = tl.k0 + half * static_cast<int>(rank);
          for (int r0 = 0; r0 < tl.cnt; r0 += kBK) {
            const int rows = min(kBK, tl.cnt - r0), rows16 = (rows + 15) & ~15;
            uint8_t* st = acquire(static_cast<uint32_t>(rows16) * (256 * na + 2 * half));
            if (!st) {
              ok = false;
              break;
            }
            const uint32_t bar = full_leader + stage * 8;
            // `n` rows (a power of two) of every operand, from global row `row` to stage row `at`
            auto fetch = [&](int box, int at, int row) {
              for (int i = 0; i < na; ++i) {
                const CUtensorMap* m = &maps.a[P::TWO_A ? i : 0].box[box];
                const int f = fr + (P::TWO_A ? 0 : 256 * i);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  tma_load_2d_pair(st + i * kABytes + c * 8192 + at * 128, m, bar, f + 64 * c, row);
              }
              for (int c = 0; c < half / 64; ++c)
                tma_load_2d_pair(st + P::kStageA + c * 8192 + at * 128, &maps.b.box[box], bar, kc + 64 * c, row);
            };
            int at = 0;
#pragma unroll
            for (int i = 0; i < kNumRowBoxes; ++i) {
              const int n = 64 >> i;
              if (rows & n) {
                fetch(i, at, tl.row0 + r0 + at);
                at += n;
              }
            }
#pragma unroll
            for (int i = kNumRowBoxes - 1; i > 2; --i) {  // zeros: 1, 2, 4, 8 rows
              const int n = 64 >> i;
              if ((rows16 - at) & n) {
                fetch(i, at, args.M);
                at += n;
              }
            }
            advance();
          }
        } else {
          const Tile tl = decode_tile<NT, 16, P::FEAT>(t, s_pre, s_off, G);
          const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          const int half = tl.nround >> 1;  // token rows staged by each CTA
          const int rbase = tl.row0 + static_cast<int>(rank) * half;
          const int fr = tl.n0 + 128 * static_cast<int>(rank);
          for (int kb = 0; kb < KB1 * args.phases; ++kb) {
            uint8_t* st = acquire(static_cast<uint32_t>(na * kABytes + half * 128));
            if (!st) {
              ok = false;
              break;
            }
            const uint32_t bar = full_leader + stage * 8;
            const int ph = (MODE == kRowsBwd && kb >= KB1) ? 1 : 0;
            const int kx = (kb - ph * KB1) * kBK;
            for (int i = 0; i < na; ++i) {
              const CUtensorMap* m = &maps.a[P::TWO_A ? i : ph];
              const int f = fr + (P::TWO_A ? 0 : 256 * i);
              if constexpr (P::A_MN) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  tma_load_3d_pair(st + i * kABytes + c * 8192, m, bar, f + 64 * c, kx, tl.g);
              } else {
                tma_load_3d_pair(st + i * kABytes, m, bar, kx, f, tl.g);
              }
            }
            int r = 0;
#pragma unroll
            for (int i = 1; i < kNumBoxes; ++i) {  // boxes of 128, 64, 32, 16, 8 rows
              const int rows = 256 >> i;
              if (half & rows) {
                tma_load_2d_pair(st + P::kStageA + r * 128, &maps.b[ph].box[i], bar, kx, rbase + r);
                r += rows;
              }
            }
            advance();
          }
        }
        if (!ok) break;
      }
      if (!ok) {  // let the copies already issued land before the CTA exits
        if (rank == 0) {
          for (int s = 0; s < STAGES; ++s)
            if (pend >> s & 1u) mbar_drain(&full[s], pend_phase >> s & 1u, 200000000ull);
        } else {  // the peer's copies complete on the leader's barrier: give them time to land
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < 2000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (lane == 0 && rank == 0) {
      const uint32_t empty_peer = mapa_shared(smem_u32(empty), 1);
      const uint32_t tfull_peer = mapa_shared(smem_u32(tfull), 1);
      uint32_t stage = 0, phase = 0, acc_phase = 0, rs = 0, rphase = 0;
      bool ok = true;
      for (;;) {
        if (!mbar_wait_cluster(&rfull[rs], rphase, abort_flag, args.status)) {
          ok = false;
          break;
        }
        const int t = ring_tile[rs];
        mbar_arrive(&rempty[rs]);
        if (++rs == kRing) {
          rs = 0;
          rphase ^= 1u;
        }
        if (t < 0) break;
        int na, n, steps, last_kk = 4;
        if constexpr (P::GRAD) {
          const GradTile tl = decode_grad<P::FEAT, NT>(t, args, NFT, NKT);
          if (tl.cnt == 0) continue;  // no rows: the epilogue writes zeros
          na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          n = args.Kd - tl.k0 > 128 ? 256 : 128;
          steps = (tl.cnt + kBK - 1) / kBK;
          last_kk = (tl.cnt - (steps - 1) * kBK + 15) / 16;
        } else {
          const Tile tl = decode_tile<NT, 16, P::FEAT>(t, s_pre, s_off, G);
          na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          n = tl.nround;
          steps = KB1 * args.phases;
        }
        if (!mbar_wait(tempty, acc_phase ^ 1u, abort_flag, args.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t idesc = idesc_bf16_f32(256, n) | (P::A_MN ? kIdescAMnMajor : 0u) | (P::GRAD ? kIdescBMnMajor : 0u);
        for (int kb = 0; kb < steps; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, args.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(ring + stage * P::kStageBytes);
          const uint32_t sb = sa + P::kStageA;
          const int nk = kb + 1 == steps ? last_kk : 4;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk >= nk) break;
            const uint64_t bdesc = P::GRAD ? sw128_mnmajor_desc(sb + kk * 2048, 8192) : sw128_kmajor_desc(sb + kk * 32);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i >= na) break;
              const uint32_t ai = sa + i * kABytes;
              const uint64_t adesc = P::A_MN ? sw128_mnmajor_desc(ai + kk * 2048, 8192) : sw128_kmajor_desc(ai + kk * 32);
              umma_bf16_pair(tmem_base + i * NT, adesc, bdesc, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
            }
          }
          umma_commit_pair(smem_u32(&empty[stage]));  // both CTAs' stage buffers are free again
          umma_commit_pair(empty_peer + stage * 8);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(smem_u32(tfull));
        umma_commit_pair(tfull_peer);
        acc_phase ^= 1u;
      }
      if (!ok) {
        umma_commit_pair(smem_u32(drain));
        mbar_drain(drain, 0, 200000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;            // TMEM lanes [32q, 32q + 32)
    const int part = (warp - 2) >> 2;  // two warps per lane quadrant take alternate column chunks
    uint8_t* stg = stg_all + (warp - 2) * P::kStgWarp;
    uint32_t acc_phase = 0, rs = 0, rphase = 0;
    for (;;) {
      if (!mbar_wait_cluster(&rfull[rs], rphase, abort_flag, args.status)) break;
      const int t = ring_tile[rs];
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&rempty[rs]);
        else mbar_arrive_cluster(rempty_leader + 8 * rs);
      }
      if (++rs == kRing) {
        rs = 0;
        rphase ^= 1u;
      }
      if (t < 0) break;
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      if constexpr (P::GRAD) {
        const GradTile tl = decode_grad<P::FEAT, NT>(t, args, NFT, NKT);
        if (tl.cnt == 0 && args.accumulate) continue;
        if (tl.cnt > 0) {
          if (!mbar_wait(tfull, acc_phase, abort_flag, args.status)) break;
          tc_fence_after();
        }
        const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
        const int ncols = min(NT, args.Kd - tl.k0);
        const int step = args.grad_f32 ? 32 : 64;  // columns of a 128-byte staged row
        for (int i = 0; i < na; ++i) {
          // this warp's first row of the gradient
          const int f0 = tl.n0 + 128 * static_cast<int>(rank) + 32 * q + (P::TWO_A ? 0 : 256 * i);
          if (f0 >= args.N) break;
          const CUtensorMap* om = &maps.o[P::TWO_A ? i : 0];
          for (int c0 = step * part; c0 < ncols; c0 += 2 * step) {
            uint32_t r[32], p[32];
            if (tl.cnt == 0) {
#pragma unroll
              for (int j = 0; j < 32; ++j) p[j] = 0u;
            } else if (args.grad_f32) {
              tmem_ld_32cols(tbase + i * NT + c0, p);
              tmem_wait_ld();
            } else {
              uint32_t r2[32];
              tmem_ld_32cols(tbase + i * NT + c0, r);
              tmem_ld_32cols(tbase + i * NT + c0 + 32, r2);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                p[j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                p[16 + j] = pack_bf16(__uint_as_float(r2[2 * j]), __uint_as_float(r2[2 * j + 1]));
              }
            }
            if (lane == 0) bulk_wait_read_all();  // the previous box has left the staging tile
            __syncwarp();
            // row `lane` of the box, 16-byte pieces in the 128-byte swizzle (no bank conflicts)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                  make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (args.accumulate) tma_reduce_add_3d(om, stg, tl.k0 + c0, f0, tl.g);
              else tma_store_3d(om, stg, tl.k0 + c0, f0, tl.g);
              bulk_commit_group();
            }
          }
        }
        if (tl.cnt == 0) continue;  // no accumulator was used
      } else {
        const Tile tl = decode_tile<NT, 16, P::FEAT>(t, s_pre, s_off, G);
        if (!mbar_wait(tfull, acc_phase, abort_flag, args.status)) break;
        tc_fence_after();
        const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
        const int fa = tl.n0 + 128 * static_cast<int>(rank) + 32 * q;  // this warp's first feature
        if constexpr (MODE == kRowsBwd) {
          __nv_bfloat16* outb = reinterpret_cast<__nv_bfloat16*>(args.out);
          for (int j0 = 32 * part; j0 < tl.nvalid; j0 += 64) {
            const int jn = min(32, tl.nvalid - j0);
            for (int i = 0; i < na; ++i) {
              uint32_t r[32];
              tmem_ld_32cols(tbase + i * NT + j0, r);
              tmem_wait_ld();
              float v[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
              store_rows32_tma(reinterpret_cast<__nv_bfloat16*>(stg), lane, v, &maps.o, outb, args.N, args.N,
                               fa + 256 * i, static_cast<long long>(tl.row0) + j0, jn);
            }
          }
        } else {
          float* stf = reinterpret_cast<float*>(stg);
          const int jl = lane >> 2, cl = 8 * (lane & 3);
          for (int j0 = 16 * part; j0 < tl.nvalid; j0 += 32) {
            if constexpr (MODE == kGateUpTrain) {
              float gv[2][8];
              stage16(stf, lane, tbase + j0);
#pragma unroll
              for (int k = 0; k < 2; ++k) load8(stf + (jl + 8 * k) * 36 + cl, gv[k]);
              stage16(stf, lane, tbase + NT + j0);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int j = j0 + jl + 8 * k;
                if (j >= tl.nvalid || fa + cl >= args.N) continue;
                float uv[8], hv[8];
                load8(stf + (jl + 8 * k) * 36 + cl, uv);
                const long long o = (static_cast<long long>(tl.row0) + j) * args.N + fa + cl;
                store8(args.pre0 + o, gv[k]);
                store8(args.pre1 + o, uv);
#pragma unroll
                for (int c = 0; c < 8; ++c) hv[c] = __fdividef(gv[k][c] * uv[c], 1.0f + __expf(-gv[k][c]));
                *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(args.out) + o) = pack8(hv);
              }
            } else {
              for (int i = 0; i < na; ++i) {
                stage16(stf, lane, tbase + i * NT + j0);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int j = j0 + jl + 8 * k, f = fa + 256 * i + cl;
                  if (j >= tl.nvalid || f >= args.N) continue;
                  float v[8];
                  load8(stf + (jl + 8 * k) * 36 + cl, v);
                  const long long o = (static_cast<long long>(tl.row0) + j) * args.N + f;
                  if constexpr (MODE == kDownBwd) {
                    float g[8], u[8], dg[8], du[8];
                    load8(args.g + o, g);
                    load8(args.u + o, u);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                      const float s = fast_sigmoid(g[c]);
                      dg[c] = v[c] * u[c] * s * (1.0f + g[c] * (1.0f - s));
                      du[c] = v[c] * g[c] * s;
                    }
                    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(args.out) + o) = pack8(dg);
                    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(args.out2) + o) = pack8(du);
                  } else {
                    if (args.bias) {
#pragma unroll
                      for (int c = 0; c < 8; ++c) v[c] += __ldg(args.bias + f + c);
                    }
                    if (args.pre0) store8(args.pre0 + o, v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = activate(v[c], args.act);
                    if (args.residual) {
                      // a plain load: the output may be the residual itself
                      const uint4 rv = *reinterpret_cast<const uint4*>(
                          reinterpret_cast<const __nv_bfloat16*>(args.residual) + o);
                      const __nv_bfloat162* rp = reinterpret_cast<const __nv_bfloat162*>(&rv);
#pragma unroll
                      for (int c = 0; c < 4; ++c) {
                        const float2 x = __bfloat1622float2(rp[c]);
                        v[2 * c] += x.x;
                        v[2 * c + 1] += x.y;
                      }
                    }
                    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(args.out) + o) = pack8(v);
                  }
                }
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(tempty);
        else mbar_arrive_cluster(tempty_leader);
      }
      acc_phase ^= 1u;
    }
    if constexpr (P::GRAD || MODE == kRowsBwd) {
      if (lane == 0) bulk_wait_all();  // the tile stores are complete before the CTA exits
    }
  }

  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its barriers or smem
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
  if (threadIdx.x == 0) {  // the last CTA rewinds the schedule for the next launch on this slot
    __threadfence();
    if (atomicAdd(&args.sched[1], 1) == static_cast<int>(gridDim.x) - 1) {
      atomicExch(&args.sched[0], 0);
      atomicExch(&args.sched[1], 0);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Rows [rows][cols] bf16 in boxes of 64 down to 1 rows x 64 columns, 128-byte swizzle.
bool map_row_boxes(RowMaps* m, const void* base, uint64_t cols, uint64_t rows) {
  for (int i = 0; i < kNumRowBoxes; ++i)
    if (!map_bf16_2d(&m->box[i], base, cols, rows, 64u >> i)) return false;
  return true;
}

// Weight gradient [groups][rows][cols] (fp32 or bf16) in boxes of 32 rows x 128 bytes.
bool map_grad_tiles(CUtensorMap* m, void* base, uint64_t cols, uint64_t rows, uint64_t groups, bool f32) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const int elem = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {cols, rows, groups};
  const cuuint64_t strides[2] = {cols * elem, cols * rows * elem};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem), 32, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch_prod(const typename Prod<MODE>::Maps& maps, const ProdArgs& args, long long tiles,
                        cudaStream_t stream) {
  using P = Prod<MODE>;
  static std::atomic<int> attr_done[kMaxDevices] = {};
  const cudaError_t err = smem_attr_once(reinterpret_cast<const void*>(prod_kernel<MODE>), P::kSmemBytes, attr_done);
  if (err != cudaSuccess) return err;
  if (tiles <= 0) return cudaSuccess;
  const int pairs = static_cast<int>(std::min<long long>(num_sms() / 2, tiles));
  return launch_pdl(prod_kernel<MODE>, dim3(2 * pairs), dim3(P::kThr), P::kSmemBytes, stream, maps, args);
}

// Upper bound on the token-mode tiles of `rows` rows in `groups` groups.
long long token_tiles(long long rows, int groups, int N, int feat) {
  return ((rows + 255) / 256 + (groups > 1 ? groups : 0)) * ((N + feat - 1) / feat);
}

// MN-major weights [G][K][N] (N contiguous): boxes of 64 K rows x 64 columns.
bool map_weight_mn(CUtensorMap* m, const void* w, int N, int K, int G) { return map_bf16_3d(m, w, N, K, G, kBK); }

template <int MODE>
cudaError_t weight_grad(const void* a0, const void* a1, const void* b, const int32_t* offsets, int G, long long rows,
                        int N, int Kd, void* dw0, void* dw1, int f32, int accumulate, int* status, int* sched,
                        cudaStream_t stream) {
  GradMaps m;
  if (!map_row_boxes(&m.a[0], a0, N, rows) || !map_row_boxes(&m.b, b, Kd, rows) ||
      !map_grad_tiles(&m.o[0], dw0, Kd, N, G, f32 != 0))
    return cudaErrorInvalidValue;
  m.a[1] = m.a[0];
  m.o[1] = m.o[0];
  if (a1 && (!map_row_boxes(&m.a[1], a1, N, rows) || !map_grad_tiles(&m.o[1], dw1, Kd, N, G, f32 != 0)))
    return cudaErrorInvalidValue;
  ProdArgs args{};
  args.offsets = offsets;
  args.G = G;
  args.M = static_cast<int>(rows);
  args.N = N;
  args.Kd = Kd;
  args.grad_f32 = f32;
  args.accumulate = accumulate;
  args.status = status;
  args.sched = sched;
  const long long tiles = static_cast<long long>(G) * ((N + Prod<MODE>::FEAT - 1) / Prod<MODE>::FEAT) *
                          ((Kd + Prod<MODE>::NT - 1) / Prod<MODE>::NT);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_prod<MODE>(m, args, tiles, stream);
}

}  // namespace

cudaError_t gemm_gate_up_train(const void* xp, const int32_t* offsets, const void* w_gate, const void* w_up, int E,
                               long long rows, int H, int F, float* g, float* u, void* h, int* status, int* sched,
                               cudaStream_t stream) {
  TokenMaps m;
  if (!map_bf16_3d(&m.a[0], w_gate, H, F, E, kBM) || !map_bf16_3d(&m.a[1], w_up, H, F, E, kBM) ||
      !map_token_boxes(&m.b[0], xp, H, rows))
    return cudaErrorInvalidValue;
  m.b[1] = m.b[0];
  m.o = m.a[0];
  ProdArgs args{};
  args.offsets = offsets, args.G = E, args.M = static_cast<int>(rows), args.N = F, args.Kd = H, args.phases = 1;
  args.out = h, args.pre0 = g, args.pre1 = u, args.status = status, args.sched = sched;
  return launch_prod<kGateUpTrain>(m, args, token_tiles(rows, E, F, Prod<kGateUpTrain>::FEAT), stream);
}

cudaError_t gemm_down_bwd(const void* dy, const float* g, const float* u, const int32_t* offsets, const void* w_down,
                          int E, long long rows, int H, int F, void* dg, void* du, int* status, int* sched,
                          cudaStream_t stream) {
  TokenMaps m;
  if (!map_weight_mn(&m.a[0], w_down, F, H, E) || !map_token_boxes(&m.b[0], dy, H, rows)) return cudaErrorInvalidValue;
  m.a[1] = m.a[0];
  m.b[1] = m.b[0];
  m.o = m.a[0];
  ProdArgs args{};
  args.offsets = offsets, args.G = E, args.M = static_cast<int>(rows), args.N = F, args.Kd = H, args.phases = 1;
  args.out = dg, args.out2 = du, args.g = g, args.u = u, args.status = status, args.sched = sched;
  return launch_prod<kDownBwd>(m, args, token_tiles(rows, E, F, Prod<kDownBwd>::FEAT), stream);
}

cudaError_t gemm_rows_bwd(const void* d0, const void* d1, const int32_t* offsets, const void* w0, const void* w1,
                          int G, long long rows, int N, int Kd, void* out, int* status, int* sched,
                          cudaStream_t stream) {
  TokenMaps m;
  if (!map_weight_mn(&m.a[0], w0, N, Kd, G) || !map_token_boxes(&m.b[0], d0, Kd, rows)) return cudaErrorInvalidValue;
  m.a[1] = m.a[0];
  m.b[1] = m.b[0];
  if (d1 && (!map_weight_mn(&m.a[1], w1, N, Kd, G) || !map_token_boxes(&m.b[1], d1, Kd, rows)))
    return cudaErrorInvalidValue;
  GemmArgs shape{};
  shape.M = static_cast<int>(rows), shape.N = N, shape.ldo = N, shape.out = out;
  if (!map_out_tiles(&m.o, shape)) return cudaErrorInvalidValue;
  ProdArgs args{};
  args.offsets = offsets, args.G = G, args.M = static_cast<int>(rows), args.N = N, args.Kd = Kd;
  args.phases = d1 ? 2 : 1, args.out = out, args.status = status, args.sched = sched;
  return launch_prod<kRowsBwd>(m, args, token_tiles(rows, G, N, Prod<kRowsBwd>::FEAT), stream);
}

cudaError_t gemm_grad_gate_up(const void* dg, const void* du, const void* xp, const int32_t* offsets, int E,
                              long long rows, int H, int F, void* dw_gate, void* dw_up, int f32, int accumulate,
                              int* status, int* sched, cudaStream_t stream) {
  return weight_grad<kGradGateUp>(dg, du, xp, offsets, E, rows, F, H, dw_gate, dw_up, f32, accumulate, status, sched,
                                  stream);
}

cudaError_t gemm_grad_down(const void* dy, const void* h, const int32_t* offsets, int G, long long rows, int N, int Kd,
                           void* dw, int f32, int accumulate, int* status, int* sched, cudaStream_t stream) {
  return weight_grad<kGradDown>(dy, nullptr, h, offsets, G, rows, N, Kd, dw, nullptr, f32, accumulate, status, sched,
                                stream);
}

cudaError_t gemm_dense_epilogue(const void* a, const void* w, const float* bias, const void* residual, int act,
                                long long M, int N, int Kd, void* out, float* pre, int* status, int* sched,
                                cudaStream_t stream) {
  TokenMaps m;
  if (!map_bf16_3d(&m.a[0], w, Kd, N, 1, kBM) || !map_token_boxes(&m.b[0], a, Kd, M)) return cudaErrorInvalidValue;
  m.a[1] = m.a[0];
  m.b[1] = m.b[0];
  m.o = m.a[0];
  ProdArgs args{};
  args.G = 1, args.M = static_cast<int>(M), args.N = N, args.Kd = Kd, args.phases = 1;
  args.out = out, args.pre0 = pre, args.bias = bias, args.residual = residual, args.act = act;
  args.status = status, args.sched = sched;
  return launch_prod<kDense>(m, args, token_tiles(M, 1, N, Prod<kDense>::FEAT), stream);
}

}  // namespace moe
