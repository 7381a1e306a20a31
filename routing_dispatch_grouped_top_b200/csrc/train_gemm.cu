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
// Bound: HBM with few rows an expert (weights and weight gradients cross once), the tensor cores with
// many; a tile of 512 x 256 reads its operands from L2 at the rate at which the MMAs need them.  48
// experts x 256 rows, H 2048, F 768, cold caches: kGateUpTrain 100 us, kDownBwd 93, kRowsBwd 87, kGradDown
// 54, kGradGateUp 95 (3.0 to 4.3 TB/s of DRAM traffic, the tensor pipe busy for 20 to 45 %: neither
// is near its peak at 256 rows a tile).  32 experts x 512 rows, H 7168, F 2048: kGateUpTrain 774 us, 1.24
// PFLOP/s.  kDense 4096 x 7168 x 2048 without epilogue: 94 us, 1.28 PFLOP/s (with bias and residual 111,
// keeping pre 129).
//
// The weight gradients reduce over an expert's rows, whose number is not a multiple of the K step
// (64 rows).  The rows behind the last one belong to the next expert and may hold anything, NaN
// included, so they must be zeros in both operands: the K step with the ragged end completes on
// a barrier of its own CTA, whose tail warp overwrites the rows up to a multiple of 16 (one MMA's K)
// with zeros and then reports the stage full; the MMAs behind that are not issued.
//
// Roles per CTA: warp 0 TMA producer, warp 1 MMA issuer (leader) and TMEM owner, then the epilogue
// warps (16, or 8 for the weight gradients, which hold a whole part of a tile in registers), a
// scheduler (the leader claims tiles from the workspace's counter) and the weight gradients' tail
// warp.  With 8 epilogue warps the token modes were 2 to 4 % slower (dg and du of 128 experts x 256
// rows, H 2048, F 768: 201 -> 190 us).  Tiles are numbered group-major, so that CTAs working at the
// same time share operand tiles through L2.
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "epilogue.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {

namespace {

enum Mode : int { kGateUpTrain, kDownBwd, kRowsBwd, kGradGateUp, kGradDown, kDense };

struct ProdMaps {
  CUtensorMap a[2];  // M side: 64 K rows x 64 columns (MN-major), or 128 rows x 64 K columns
  CUtensorMap aw;    // kDense: 256 rows x 64 K columns, both operands of a CTA at once
  CUtensorMap o[2];  // weight gradients: output boxes of 32 rows x 128 bytes
  BoxMaps b[2];      // N side: token rows; weight gradients: b[0].box[0], 64 K rows x 64 columns
};

// A tile as the scheduler publishes it: group, first output feature, first column (weight gradients),
// first row and number of rows (the N side of the token modes, the reduction of the gradients).
struct Entry {
  int g, n0, k0, row0, cnt;  // g < 0: no more tiles
};
constexpr int kEntryInts = 8;

// Tiles in flight from the scheduler to the other warps: enough for the producer to run a tile ahead,
// no more (a claimed tile is not available to other pairs; 3 and 4 were no faster).
constexpr int kTiles = 2;

template <int MODE>
struct Prod {
  static constexpr bool GRAD = MODE == kGradGateUp || MODE == kGradDown;
  static constexpr bool A_MN = MODE != kGateUpTrain && MODE != kDense;  // M side contiguous in memory
  static constexpr bool TWO_A = MODE == kGateUpTrain || MODE == kGradGateUp;  // two weight operands, one N tile
  static constexpr int NT = 256;                      // N of a tile
  static constexpr int FEAT = TWO_A ? 256 : 512;      // M of a tile (of each operand)
  static constexpr int STAGES = 4;
  static constexpr int EW = GRAD ? 8 : 16;            // epilogue warps
  static constexpr int kThr = 64 + 32 * EW + (GRAD ? 64 : 32);
  static constexpr int kStageA = 2 * kABytes;         // this CTA's two 128 x 64 M-side tiles
  static constexpr int kStageB = (NT / 2) * 128;      // this CTA's half of the N side
  static constexpr int kStageBytes = kStageA + kStageB;
  // epilogue staging of a warp: 16 x 32 bf16 as 8 x 36 words, or 32 rows of 128 B
  static constexpr int kStgWarp = GRAD ? 4096 : 8 * 36 * 4;
  static constexpr int kStgBytes = EW * kStgWarp;
  static constexpr int kBarBytes = (8 * (3 * STAGES + 5 + 2 * kTiles) + 8 + 4 * kEntryInts * kTiles + 15) / 16 * 16;
  static constexpr int kTableBytes = GRAD ? 0 : 2 * (kMaxGroups + 1) * 4;  // offsets, first tiles
  static constexpr int kSmemBytes = 1024 + STAGES * kStageBytes + kStgBytes + kBarBytes + kTableBytes;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct ProdArgs {
  const int32_t* offsets;  // [G + 1] or nullptr: one group of M rows
  int G;
  int M;                   // rows of the token operands
  int N;                   // output features (token modes), rows of a weight gradient
  int Kd;                  // reduction length of one phase (token modes), columns of a weight gradient
  int nt;                  // token modes: most rows of a tile (a multiple of 16, at most 256)
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
  int accumulate;          // fp32 weight gradients: added to what they hold
  int late_wait;           // no operand is written by the kernel before this one
  int* status;
  int* sched;              // two device ints {claimed tiles, finished pairs}, zero between launches
};

constexpr int kChunk = kBK * 128;  // bytes of 64 K rows x 64 columns

// First output feature (row of a weight gradient) of CTA `rank` for operand i.  Two operands of one
// tensor lie side by side (256 consecutive features a CTA, one copy), so that CTA 1 starts 256 on;
// with one operand, or one of two tensors, it starts 128 on.
template <bool TWO_A>
__device__ __forceinline__ int first_feature(int n0, int na, uint32_t rank, int i) {
  return TWO_A || na == 1 ? n0 + 128 * static_cast<int>(rank) : n0 + 256 * static_cast<int>(rank) + 128 * i;
}

__device__ __forceinline__ Entry read_entry(const volatile int* ring, uint32_t slot) {
  const volatile int* e = ring + slot * kEntryInts;
  return {e[0], e[1], e[2], e[3], e[4]};
}

// 16 tokens x 32 features between the epilogue's registers (a lane holds one feature of 16 tokens) and
// bf16 rows in global memory (a lane moves 16-byte pieces, 8 features of one token), through a warp's
// staging tile of 8 x 36 words: word (p, l) holds tokens 2p and 2p + 1 of feature l, so that a
// lane writes 8 words and reads back the two tokens' pieces 16 bytes at a time (rows padded to 36
// words: no bank conflicts).
constexpr int kChTok = 16;

struct RowPieces {
  uint4 v[2];  // tokens 2 (lane >> 2) and the next, features 8 (lane & 3) ..
};

__device__ __forceinline__ uint32_t lo_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// Rows `jn` of `src` (row stride ld, `nf` features from here on) into registers; the rest are zeros.
__device__ __forceinline__ void load_pieces(RowPieces& p, const __nv_bfloat16* src, int ld, int lane, int jn, int nf) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = 2 * (lane >> 2) + h, c = 8 * (lane & 3);
    // a plain load: the output may be the residual itself
    p.v[h] = j < jn && c < nf ? *reinterpret_cast<const uint4*>(src + static_cast<long long>(j) * ld + c)
                              : make_uint4(0u, 0u, 0u, 0u);
  }
}

__device__ __forceinline__ void add_pieces(uint32_t* stg, int lane, float (&v)[kChTok], const RowPieces& p) {
  __syncwarp();  // the staged values of the previous call have been read
  const uint4 a = p.v[0], b = p.v[1];
  uint4* dst = reinterpret_cast<uint4*>(stg + (lane >> 2) * 36 + 8 * (lane & 3));
  dst[0] = make_uint4(lo_halves(a.x, b.x), hi_halves(a.x, b.x), lo_halves(a.y, b.y), hi_halves(a.y, b.y));
  dst[1] = make_uint4(lo_halves(a.z, b.z), hi_halves(a.z, b.z), lo_halves(a.w, b.w), hi_halves(a.w, b.w));
  __syncwarp();
#pragma unroll
  for (int t = 0; t < kChTok / 2; ++t) {
    const uint32_t w = stg[t * 36 + lane];
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    v[2 * t] += f.x;
    v[2 * t + 1] += f.y;
  }
}

__device__ __forceinline__ void store_pieces(uint32_t* stg, int lane, const float (&v)[kChTok], __nv_bfloat16* dst,
                                             int ld, int jn, int nf) {
  __syncwarp();
#pragma unroll
  for (int t = 0; t < kChTok / 2; ++t) stg[t * 36 + lane] = pack_bf16(v[2 * t], v[2 * t + 1]);
  __syncwarp();
  const int c = 8 * (lane & 3), t = lane >> 2;
  const uint4* src = reinterpret_cast<const uint4*>(stg + t * 36 + c);
  const uint4 a = src[0], b = src[1];
  __nv_bfloat16* row = dst + static_cast<long long>(2 * t) * ld + c;
  if (c < nf) {
    if (2 * t < jn)
      *reinterpret_cast<uint4*>(row) =
          make_uint4(lo_halves(a.x, a.y), lo_halves(a.z, a.w), lo_halves(b.x, b.y), lo_halves(b.z, b.w));
    if (2 * t + 1 < jn)
      *reinterpret_cast<uint4*>(row + ld) =
          make_uint4(hi_halves(a.x, a.y), hi_halves(a.z, a.w), hi_halves(b.x, b.y), hi_halves(b.z, b.w));
  }
}

// F32: fp32 weight gradients (the other modes: false).
template <int MODE, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Prod<MODE>::kThr, 1)
    prod_kernel(const __grid_constant__ ProdMaps maps, const ProdArgs args) {
  using P = Prod<MODE>;
  constexpr int STAGES = P::STAGES, EW = P::EW, NT = P::NT;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* stg_all = smem + STAGES * P::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + P::kStgBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* rfull = drain + 1;
  uint64_t* rempty = rfull + kTiles;
  uint64_t* tail = rempty + kTiles;  // weight gradients: this CTA's part of a last K step has landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + STAGES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* entries = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* s_off = reinterpret_cast<int*>(stg_all + P::kStgBytes + P::kBarBytes);  // token modes only
  int* s_pre = s_off + (kMaxGroups + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int G = args.offsets ? args.G : 1;
  const int NFT = (args.N + P::FEAT - 1) / P::FEAT;
  const int NKT = (args.Kd + NT - 1) / NT;              // weight gradients: column tiles
  const int KB1 = (args.Kd + kBK - 1) / kBK;            // token modes: K steps of a phase

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 2);  // both CTAs' producers (a last K step: both tail warps)
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * EW);
    }
    mbar_init(drain, 1);
    for (int r = 0; r < kTiles; ++r) {
      mbar_init(&rfull[r], 1);
      // leader MMA, both CTAs' producers, epilogue warps (and tail warps)
      mbar_init(&rempty[r], 3 + 2 * EW + (P::GRAD ? 2 : 0));
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) {  // the maps are parameters: fetched while the previous kernel finishes
    if (lane < 2 && (lane == 0 || P::TWO_A || args.phases == 2)) tma_prefetch_map(&maps.a[lane]);
    if (lane == 2 && MODE == kDense) tma_prefetch_map(&maps.aw);
    if (P::GRAD ? lane == 8 : lane > 8 && lane < 8 + kNumBoxes) tma_prefetch_map(&maps.b[0].box[lane - 8]);
    if (lane > 16 && lane < 16 + kNumBoxes && args.phases == 2) tma_prefetch_map(&maps.b[1].box[lane - 16]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any access over the cluster
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // All of the above may run while the previous kernel finishes.  Offsets and operands come from
  // earlier kernels.  With late_wait they come from kernels before the previous one, and those were
  // complete when the previous one let this one start: the two overlap, and this one only ends after
  // it (below).
  if (!args.late_wait) pdl_wait();
  pdl_launch_dependents();
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
  const uint32_t rempty_leader = mapa_shared(smem_u32(rempty), 0);
  const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, rs = 0, rphase = 0;
      uint32_t pend = 0, pend_phase = 0;  // one bit a stage
      const uint32_t tail_own = mapa_shared(smem_u32(tail), rank);
      bool ok = true;
      // Waits for the stage to be free, announces its bytes (both CTAs' on the leader's barrier) and
      // returns its buffer.
      auto acquire = [&](uint32_t bytes) -> uint8_t* {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, args.status)) return nullptr;
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2u * bytes);
        else mbar_arrive_remote(full_leader + stage * 8);
        return ring + stage * P::kStageBytes;
      };
      // The M side of a K step: `x` is the first row (K-major) or column (MN-major), `k` the first K.
      auto fetch_a = [&](uint8_t* st, uint32_t bar, int ph, int na, int x, int k, int g) {
        if constexpr (!P::A_MN) {
          if (P::TWO_A || na == 1) {
            for (int i = 0; i < na; ++i) tma_load_3d_pair(st + i * kABytes, &maps.a[i], bar, k, x, g);
          } else {
            tma_load_3d_pair(st, &maps.aw, bar, k, x, g);
          }
        } else {
          for (int i = 0; i < na; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              tma_load_3d_pair(st + i * kABytes + c * kChunk, &maps.a[P::TWO_A ? i : ph], bar,
                               x + (P::TWO_A ? 0 : 128 * i) + 64 * c, k, g);
        }
      };
      auto advance = [&] {
        pend |= 1u << stage;
        pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      };
      while (ok) {
        if (!mbar_wait_cluster(&rfull[rs], rphase, abort_flag, args.status)) {
          ok = false;
          break;
        }
        const Entry tl = read_entry(entries, rs);
        if (rank == 0) mbar_arrive(&rempty[rs]);
        else mbar_arrive_remote(rempty_leader + 8 * rs);
        if (++rs == kTiles) {
          rs = 0;
          rphase ^= 1u;
        }
        if (tl.g < 0) break;
        if constexpr (P::GRAD) {
          const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          const int half = args.Kd - tl.k0 > 128 ? 128 : 64;  // N columns staged by each CTA
          const int fr = first_feature<P::TWO_A>(tl.n0, na, rank, 0);
          const int kc = tl.k0 + half * static_cast<int>(rank);
          const uint32_t bytes = static_cast<uint32_t>(na * kABytes + half * 128);
          // The ragged step (the last rows) comes first, where its tail warp's work is hidden by the end
          // of the previous tile; with rows that are no multiple of 16 it completes on this CTA's
          // tail barrier.
          const int steps = (tl.cnt + kBK - 1) / kBK;
          for (int kb = 0; kb < steps; ++kb) {
            const int r0 = (kb == 0 ? steps - 1 : kb - 1) * kBK;
            const bool fix = kb == 0 && (tl.cnt & 15);
            uint8_t* st;
            uint32_t bar = full_leader + stage * 8;
            if (fix) {
              st = mbar_wait(&empty[stage], phase ^ 1u, abort_flag, args.status) ? ring + stage * P::kStageBytes : nullptr;
              if (st) mbar_arrive_expect_tx(&tail[stage], bytes);
              bar = tail_own + stage * 8;
            } else {
              st = acquire(bytes);
            }
            if (!st) {
              ok = false;
              break;
            }
            const int row = tl.row0 + r0;
            fetch_a(st, bar, 0, na, fr, row, 0);
            for (int c = 0; c < half / 64; ++c)
              tma_load_2d_pair(st + P::kStageA + c * kChunk, &maps.b[0].box[0], bar, kc + 64 * c, row);
            advance();
          }
        } else {
          const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          const int half = ((tl.cnt + 15) & ~15) >> 1;  // token rows staged by each CTA
          const int rbase = tl.row0 + static_cast<int>(rank) * half;
          const int fr = first_feature<P::TWO_A>(tl.n0, na, rank, 0);
          for (int kb = 0; kb < KB1 * args.phases; ++kb) {
            uint8_t* st = acquire(static_cast<uint32_t>(na * kABytes + half * 128));
            if (!st) {
              ok = false;
              break;
            }
            const uint32_t bar = full_leader + stage * 8;
            const int ph = (MODE == kRowsBwd && kb >= KB1) ? 1 : 0;
            const int kx = (kb - ph * KB1) * kBK;
            fetch_a(st, bar, ph, na, fr, kx, tl.g);
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
    // The whole warp runs the loop, one elected lane issues.
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, rs = 0, rphase = 0;
      bool ok = true;
      const uint32_t ring_addr = smem_u32(ring), empty_addr = smem_u32(empty), tfull_addr = smem_u32(tfull);
      constexpr uint64_t kDescA = P::A_MN ? sw128_mnmajor_desc(0, kChunk) : sw128_kmajor_desc(0);
      constexpr uint64_t kDescB = P::GRAD ? sw128_mnmajor_desc(0, kChunk) : sw128_kmajor_desc(0);
      constexpr uint32_t kStepA = (P::A_MN ? 2048 : 32) >> 4, kStepB = (P::GRAD ? 2048 : 32) >> 4;  // 16 K elements
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, args.status));
      };
      auto wait_full = [&](uint32_t st, uint32_t ph) -> bool {
        // weight gradients: the peer's tail warp wrote its rows with plain stores
        return P::GRAD ? __all_sync(0xffffffffu, mbar_wait_cluster(&full[st], ph, abort_flag, args.status))
                       : wait(&full[st], ph);
      };
      // Both CTAs' stage buffers are free again / the accumulator buffer's sums are complete.
      auto release = [&](uint32_t st) { umma_commit_both_warp(empty_addr + 8 * st); };
      auto publish = [&](uint32_t buf) { umma_commit_both_warp(tfull_addr + 8 * buf); };
      auto step = [&](uint32_t& st, uint32_t& ph) {
        if (++st == STAGES) {
          st = 0;
          ph ^= 1u;
        }
      };
      for (;;) {
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&rfull[rs], rphase, abort_flag, args.status))) {
          ok = false;
          break;
        }
        const Entry tl = read_entry(entries, rs);
        __syncwarp();
        if (lane == 0) mbar_arrive(&rempty[rs]);
        __syncwarp();
        if (++rs == kTiles) {
          rs = 0;
          rphase ^= 1u;
        }
        if (tl.g < 0) break;
        int na, n, steps, first_kk = 4;
        if constexpr (P::GRAD) {
          if (tl.cnt == 0) continue;  // no rows: the epilogue writes zeros
          na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          n = args.Kd - tl.k0 > 128 ? 256 : 128;
          steps = (tl.cnt + kBK - 1) / kBK;
          first_kk = (tl.cnt - (steps - 1) * kBK + 15) / 16;  // the ragged step comes first
        } else {
          na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
          n = (tl.cnt + 15) & ~15;
          steps = KB1 * args.phases;
        }
        const uint32_t idesc = idesc_bf16_f32(256, n) | (P::A_MN ? kIdescAMnMajor : 0u) | (P::GRAD ? kIdescBMnMajor : 0u);
        // The MMAs of one stage into accumulator buffer `buf` for the M-side operand `i`.
        auto mma = [&](uint32_t st, int i, uint32_t buf, int kb) {
          const uint32_t sa = ((ring_addr + st * P::kStageBytes) >> 4) & 0x3FFFu;
          const uint64_t a = kDescA | (sa + i * (kABytes >> 4)), b = kDescB | (sa + (P::kStageA >> 4));
          const uint32_t d = tmem_base + buf * NT;
          umma_bf16_pair_warp(d, a, b, idesc, kb > 0 ? 1u : 0u);
          if (kb > 0 || first_kk == 4) {
#pragma unroll
            for (int kk = 1; kk < 4; ++kk) umma_bf16_pair_warp(d, a + kk * kStepA, b + kk * kStepB, idesc, 1u);
          } else {
            for (int kk = 1; kk < first_kk; ++kk) umma_bf16_pair_warp(d, a + kk * kStepA, b + kk * kStepB, idesc, 1u);
          }
        };
        // The two accumulator buffers are a ring: a tile takes the next one or two.
        const uint32_t b0 = acc, b1 = acc ^ 1u;
        const uint32_t ph0 = acc_phase, ph1 = acc_phase ^ (acc == 1u ? 1u : 0u);  // phase flips on wrap-around
        if (!wait(&tempty[b0], ph0 ^ 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (na == 1) {
          for (int kb = 0; kb < steps; ++kb) {
            if (!wait_full(stage, phase)) {
              ok = false;
              break;
            }
            tc_fence_after();
            mma(stage, 0, b0, kb);
            release(stage);
            step(stage, phase);
          }
          if (!ok) break;
          publish(b0);
          acc ^= 1u;
          if (acc == 0) acc_phase ^= 1u;
          continue;
        }
        // Two accumulators: operand 0 runs ahead of operand 1 by up to a ring of stages while the second
        // buffer is still being drained, so that this drain overlaps MMAs.  (Running ahead at the end
        // of a tile as well, so that the first buffer is handed over earlier, delays the stages'
        // release: 5 % slower on weight gradients of 256 rows.)
        bool have1 = false;
        int pend = 0;             // stages done for operand 0 only
        uint32_t pst = stage;     // the first of them
        uint32_t pph = 0;
        for (int kb = 0; kb < steps; ++kb) {
          if (!wait_full(stage, phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          mma(stage, 0, b0, kb);
          step(stage, phase);
          ++pend;
          const bool last = kb + 1 == steps, must = last || pend == STAGES;
          if (last) publish(b0);
          if (!have1) {
            have1 = __all_sync(0xffffffffu, mbar_poll(&tempty[b1], ph1 ^ 1u));
            if (!have1 && must) {
              if (!wait(&tempty[b1], ph1 ^ 1u)) {
                ok = false;
                break;
              }
              have1 = true;
            }
            if (have1) tc_fence_after();
          }
          if (have1) {
            for (; pend > 0; --pend) {
              mma(pst, 1, b1, kb + 1 - pend);
              release(pst);
              step(pst, pph);
            }
          }
        }
        if (!ok) break;
        publish(b1);
        acc_phase ^= 1u;  // two buffers on: the same buffer, the other phase
      }
      if (!ok) {
        umma_commit_both_warp(smem_u32(drain));
        if (lane == 0) mbar_drain(drain, 0, 200000000ull);
        __syncwarp();
      }
    }
  } else if (warp < 2 + EW) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;            // TMEM lanes [32q, 32q + 32)
    const int part = (warp - 2) >> 2;  // the warps of a lane quadrant take the column chunks in turn
    uint8_t* stg = stg_all + (warp - 2) * P::kStgWarp;
    uint32_t acc = 0, acc_phase = 0, rs = 0, rphase = 0;
    // Waits for the next accumulator buffer; hands it back.
    auto take = [&]() -> bool {
      if (!mbar_wait(&tfull[acc], acc_phase, abort_flag, args.status)) return false;
      tc_fence_after();
      return true;
    };
    auto give = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&tempty[acc]);
        else mbar_arrive_remote(tempty_leader + 8 * acc);
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    };
    bool ok = true;
    while (ok) {
      if (!mbar_wait_cluster(&rfull[rs], rphase, abort_flag, args.status)) break;
      const Entry tl = read_entry(entries, rs);
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&rempty[rs]);
        else mbar_arrive_remote(rempty_leader + 8 * rs);
      }
      if (++rs == kTiles) {
        rs = 0;
        rphase ^= 1u;
      }
      if (tl.g < 0) break;
      if constexpr (P::GRAD) {
        if (tl.cnt == 0 && args.accumulate) continue;
        const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
        const int ncols = min(NT, args.Kd - tl.k0);
        // Columns of a 128-byte staged row, and how many such chunks of the 256 are this warp's.
        constexpr int kSpan = F32 ? 32 : 64, kSpans = NT / 2 / kSpan;
        for (int i = 0; i < na; ++i) {
          // The whole part goes to registers (bf16 packed) and the buffer back to the MMAs before
          // anything is stored: a tile of 256 or 512 rows has little more MMA work than this drain.
          uint32_t p[kSpans][32];
          if (tl.cnt > 0) {
            if (!take()) {
              ok = false;
              break;
            }
            const uint32_t tbase = tmem_base + acc * NT + (static_cast<uint32_t>(q * 32) << 16) + kSpan * part;
            if constexpr (F32) {
#pragma unroll
              for (int c = 0; c < kSpans; ++c) tmem_ld_32cols(tbase + 2 * kSpan * c, p[c]);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int c = 0; c < kSpans; ++c) {
                uint32_t r0[32], r1[32];
                tmem_ld_32cols(tbase + 2 * kSpan * c, r0);
                tmem_ld_32cols(tbase + 2 * kSpan * c + 32, r1);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  p[c][j] = pack_bf16(__uint_as_float(r0[2 * j]), __uint_as_float(r0[2 * j + 1]));
                  p[c][16 + j] = pack_bf16(__uint_as_float(r1[2 * j]), __uint_as_float(r1[2 * j + 1]));
                }
              }
            }
            give();
          } else {  // an expert without rows: zeros, and no accumulator was used
#pragma unroll
            for (int c = 0; c < kSpans; ++c)
#pragma unroll
              for (int j = 0; j < 32; ++j) p[c][j] = 0u;
          }
          // this warp's first row of the gradient
          const int f0 = first_feature<P::TWO_A>(tl.n0, na, rank, i) + 32 * q;
          const CUtensorMap* om = &maps.o[P::TWO_A ? i : 0];
#pragma unroll
          for (int c = 0; c < kSpans; ++c) {
            const int c0 = kSpan * (part + 2 * c);
            if (f0 >= args.N || c0 >= ncols) break;
            if (lane == 0) bulk_wait_read_all();  // the previous box has left the staging tile
            __syncwarp();
            // row `lane` of the box, 16-byte pieces in the 128-byte swizzle (no bank conflicts)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                  make_uint4(p[c][4 * k], p[c][4 * k + 1], p[c][4 * k + 2], p[c][4 * k + 3]);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (F32 && args.accumulate) tma_reduce_add_3d(om, stg, tl.k0 + c0, f0, tl.g);
              else tma_store_3d(om, stg, tl.k0 + c0, f0, tl.g);
              bulk_commit_group();
            }
            __syncwarp();
          }
          __syncwarp();
        }
      } else {
        const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
        uint32_t* stw = reinterpret_cast<uint32_t*>(stg);
        for (int i = 0; i < na; ++i) {
          // this warp's first feature; a lane holds one feature of 16 tokens at a time
          const int fa = first_feature<P::TWO_A>(tl.n0, na, rank, i) + 32 * q;
          const int nv = fa < args.N ? tl.cnt : 0;
          const bool f_ok = fa + lane < args.N;
          const long long base = static_cast<long long>(tl.row0) * args.N + fa;  // token 0, feature fa
          float bias = 0.0f;
          if constexpr (MODE == kDense) bias = args.bias && f_ok ? __ldg(args.bias + fa + lane) : 0.0f;
          // What the epilogue reads beside the product is fetched ahead: the first tokens' before the
          // wait for the sums, the others' before the tokens before them are stored, and a residual also
          // into L2 right after the wait (earlier, and the weights streaming through L2 would have
          // evicted it).
          float x0[kChTok], x1[kChTok];
          RowPieces res;
          auto fetch = [&](int j0) {
            const long long o = base + static_cast<long long>(j0) * args.N;  // token j0, feature fa
            const int jn = nv - j0;
            if constexpr (MODE == kDownBwd) {
#pragma unroll
              for (int j = 0; j < kChTok; ++j) {
                const bool in = j < jn && f_ok;
                x0[j] = in ? __ldg(args.g + o + static_cast<long long>(j) * args.N + lane) : 0.0f;
                x1[j] = in ? __ldg(args.u + o + static_cast<long long>(j) * args.N + lane) : 0.0f;
              }
            } else if constexpr (MODE == kGateUpTrain) {
              if (i == 1) {  // g, written by this lane for i = 0
#pragma unroll
                for (int j = 0; j < kChTok; ++j)
                  x0[j] = j < jn && f_ok ? args.pre0[o + static_cast<long long>(j) * args.N + lane] : 0.0f;
              }
            } else if constexpr (MODE == kDense) {
              if (args.residual)
                load_pieces(res, reinterpret_cast<const __nv_bfloat16*>(args.residual) + o, args.N, lane, jn, args.N - fa);
            }
          };
          if constexpr (MODE != kGateUpTrain) fetch(kChTok * part);
          if (!take()) {
            ok = false;
            break;
          }
          if constexpr (MODE == kDense) {
            if (args.residual)
              for (int j = kChTok * part + 64 + lane; lane < kChTok && j < nv; j += 64)
                prefetch_l2(reinterpret_cast<const __nv_bfloat16*>(args.residual) + base + static_cast<long long>(j) * args.N);
          }
          const uint32_t tbase = tmem_base + acc * NT + (static_cast<uint32_t>(q * 32) << 16);
          for (int j0 = kChTok * part; j0 < nv; j0 += 64) {
            const int jn = min(kChTok, nv - j0);
            const long long o = base + static_cast<long long>(j0) * args.N;  // token j0, feature fa
            if constexpr (MODE == kGateUpTrain) fetch(j0);  // just written: in L2
            uint32_t r[kChTok];
            __syncwarp();
            tmem_ld_16cols(tbase + j0, r);
            tmem_wait_ld();
            float v[kChTok];
#pragma unroll
            for (int j = 0; j < kChTok; ++j) v[j] = __uint_as_float(r[j]);
            __nv_bfloat16* outb = reinterpret_cast<__nv_bfloat16*>(args.out) + o;
            if constexpr (MODE == kRowsBwd) {
              store_pieces(stw, lane, v, outb, args.N, jn, args.N - fa);
            } else if constexpr (MODE == kGateUpTrain) {
              float* pre = (i == 0 ? args.pre0 : args.pre1) + o + lane;
              if (f_ok) {
#pragma unroll
                for (int j = 0; j < kChTok; ++j)
                  if (j < jn) pre[static_cast<long long>(j) * args.N] = v[j];
              }
              if (i == 1) {  // h = silu(g) u
#pragma unroll
                for (int j = 0; j < kChTok; ++j) v[j] = swiglu(x0[j], v[j]);
                store_pieces(stw, lane, v, outb, args.N, jn, args.N - fa);
              }
            } else if constexpr (MODE == kDownBwd) {
              float du[kChTok];
#pragma unroll
              for (int j = 0; j < kChTok; ++j) swiglu_grad(v[j], x0[j], x1[j], v[j], du[j]);
              if (j0 + 64 < nv) fetch(j0 + 64);
              store_pieces(stw, lane, v, outb, args.N, jn, args.N - fa);
              store_pieces(stw, lane, du, reinterpret_cast<__nv_bfloat16*>(args.out2) + o, args.N, jn, args.N - fa);
            } else {
#pragma unroll
              for (int j = 0; j < kChTok; ++j) v[j] += bias;
              if (args.pre0 && f_ok) {
                float* pre = args.pre0 + o + lane;
#pragma unroll
                for (int j = 0; j < kChTok; ++j)
                  if (j < jn) pre[static_cast<long long>(j) * args.N] = v[j];
              }
              activate(v, args.act);
              if (args.residual) {
                add_pieces(stw, lane, v, res);
                if (j0 + 64 < nv) fetch(j0 + 64);
              }
              store_pieces(stw, lane, v, outb, args.N, jn, args.N - fa);
            }
          }
          give();
        }
      }
    }
    if constexpr (P::GRAD) {
      if (lane == 0) bulk_wait_all();  // the tile stores are complete before the CTA exits
    }
  } else if (warp == 2 + EW) {
    // ------------------------------------------------------------ scheduler (leader only)
    // Reads the offsets, claims tiles and publishes them to both CTAs, in a warp of its own: neither the
    // counter's round trip, the offsets' loads (which queue behind the epilogue's stores) nor the
    // release over the cluster stands between two tiles' loads.  The first tile is the pair's own, the
    // others come from the counter.
    if (rank == 0) {
      // Offsets must be non-decreasing inside [0, M]; otherwise no tile runs.
      bool bad = false;
      for (int i = lane; i <= G; i += 32) {
        const int o = args.offsets ? __ldg(args.offsets + i) : (i == 0 ? 0 : args.M);
        const int before = args.offsets && i > 0 ? __ldg(args.offsets + i - 1) : 0;
        bad |= o < before || o > args.M;
        if constexpr (!P::GRAD) s_off[i] = o;
      }
      __syncwarp();
      bad = __any_sync(0xffffffffu, bad);
      int total = G * NFT * NKT;
      if constexpr (!P::GRAD) {  // s_pre[g]: first tile of group g
        const int seg = (G + 31) / 32, lo = min(G, lane * seg), hi = min(G, lo + seg);
        int sum = 0;
        for (int g = lo; g < hi; ++g) sum += (s_off[g + 1] - s_off[g] + args.nt - 1) / args.nt * NFT;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        int run = incl - sum;
        for (int g = lo; g < hi; ++g) {
          s_pre[g] = run;
          run += (s_off[g + 1] - s_off[g] + args.nt - 1) / args.nt * NFT;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
        if (lane == 0) s_pre[G] = total;
        __syncwarp();
      }
      if (bad) total = 0;
      if (lane == 0) {
        const int pairs = gridDim.x >> 1;
        if (bad && blockIdx.x == 0) report(args.status, MOE_DEV_BAD_INDEX);
        const uint32_t rfull_peer = mapa_shared(smem_u32(rfull), 1);
        const uint32_t entries_peer = mapa_shared(smem_u32(const_cast<int*>(entries)), 1);
        uint32_t rs = 0, rphase = 0;
        for (int t = blockIdx.x >> 1;; t = pairs + atomicAdd(&args.sched[0], 1)) {
          Entry e{-1, 0, 0, 0, 0};
          if (t < total) {
            if constexpr (P::GRAD) {
              e.g = t / (NFT * NKT);
              const int local = t - e.g * NFT * NKT;
              e.n0 = (local / NKT) * P::FEAT;
              e.k0 = (local % NKT) * NT;
              e.row0 = args.offsets ? __ldg(args.offsets + e.g) : 0;
              e.cnt = (args.offsets ? __ldg(args.offsets + e.g + 1) : args.M) - e.row0;
            } else {
              const Tile tl = decode_tile<16, P::FEAT>(t, s_pre, s_off, G, args.nt);
              e = {tl.g, tl.n0, 0, tl.row0, tl.nvalid};
            }
          } else if (atomicAdd(&args.sched[1], 1) == pairs - 1) {
            // every pair has claimed its last tile: the counters are rewound for the next launch
            atomicExch(&args.sched[0], 0);
            atomicExch(&args.sched[1], 0);
          }
          if (!mbar_wait_cluster(&rempty[rs], rphase ^ 1u, abort_flag, args.status)) break;
          const int v[5] = {e.g, e.n0, e.k0, e.row0, e.cnt};
#pragma unroll
          for (int k = 0; k < 5; ++k) {
            entries[rs * kEntryInts + k] = v[k];
            st_shared_cluster(entries_peer + 4 * (rs * kEntryInts + k), v[k]);
          }
          mbar_arrive(&rfull[rs]);
          mbar_arrive_cluster(rfull_peer + 8 * rs);
          if (e.g < 0) break;
          if (++rs == kTiles) {
            rs = 0;
            rphase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if constexpr (P::GRAD) {
    // ------------------------------------------------------------ tail warp (both CTAs)
    // The ragged K step of an expert holds rows of the next one (or zeros behind the tensor) after its
    // own: the rows up to a multiple of 16, one MMA's K, are overwritten with zeros in both operands.
    uint32_t rs = 0, rphase = 0, kstep = 0, tail_phase = 0;  // kstep: this CTA's K steps so far
    for (;;) {
      if (!__all_sync(0xffffffffu, mbar_wait_cluster(&rfull[rs], rphase, abort_flag, args.status))) break;
      const Entry tl = read_entry(entries, rs);
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&rempty[rs]);
        else mbar_arrive_remote(rempty_leader + 8 * rs);
      }
      __syncwarp();
      if (++rs == kTiles) {
        rs = 0;
        rphase ^= 1u;
      }
      if (tl.g < 0) break;
      const int steps = (tl.cnt + kBK - 1) / kBK;
      const uint32_t stage = kstep % STAGES;  // of the ragged step, the tile's first
      kstep += steps;
      if ((tl.cnt & 15) == 0) continue;
      // a stage's tail barrier completes once a use as a tail: its phase is counted per stage
      const uint32_t ph = tail_phase >> stage & 1u;
      tail_phase ^= 1u << stage;
      if (!__all_sync(0xffffffffu, mbar_wait(&tail[stage], ph, abort_flag, args.status))) break;
      const int v = tl.cnt - (steps - 1) * kBK, v16 = (v + 15) & ~15;
      const int na = P::TWO_A || tl.n0 + 256 < args.N ? 2 : 1;
      const int half = args.Kd - tl.k0 > 128 ? 128 : 64;
      uint8_t* st = ring + stage * P::kStageBytes;
      const int chunks = 2 * na + half / 64, per = (v16 - v) * 8;  // 16-byte pieces a chunk
      for (int c = 0; c < chunks; ++c) {
        uint8_t* base = (c < 2 * na ? st + c * kChunk : st + P::kStageA + (c - 2 * na) * kChunk) + v * 128;
        for (int i = lane; i < per; i += 32) *reinterpret_cast<uint4*>(base + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&full[stage]);
        else mbar_arrive_cluster(full_leader + stage * 8);
      }
      __syncwarp();
    }
  }

  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its barriers or smem
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
  if (args.late_wait) pdl_wait();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Rows of a dense product's tiles: the chunk count between ceil(M / 256) and twice that with the
// least (waves of tiles over the pairs) x (rows of a tile + 16 for its start and end).  4096 tokens x
// 7168 features are 224 tiles of 256 rows, two more than three waves; 280 tiles of 208 rows are 3.8.
int dense_rows(long long M, int N) {
  const long long pairs = std::max(1, num_sms() / 2), nft = (N + Prod<kDense>::FEAT - 1) / Prod<kDense>::FEAT;
  const long long least = (M + 255) / 256;
  if (least * nft > 32 * pairs) return 256;  // a last wave in more than 32
  long long best = -1;
  int rows = 256;
  for (long long c = least; c <= 2 * least; ++c) {
    const int r = static_cast<int>(((M + c - 1) / c + 15) / 16 * 16);
    const long long tiles = (M + r - 1) / r * nft, cost = (tiles + pairs - 1) / pairs * (r + 16);
    if (best < 0 || cost < best) best = cost, rows = r;
  }
  return rows;
}

// MN-major operand [G][K][cols] (cols contiguous), boxes of 64 K rows x 64 columns.
bool map_mn(CUtensorMap* m, const void* base, uint64_t cols, uint64_t K, uint64_t G) {
  return map_bf16_3d(m, base, cols, K, G, kBK);
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

template <int MODE, bool F32 = false>
cudaError_t launch_prod(const ProdMaps& maps, const ProdArgs& args, long long tiles,
                        cudaStream_t stream) {
  using P = Prod<MODE>;
  static std::atomic<int> attr_done[kMaxDevices] = {};
  const cudaError_t err = smem_attr_once(reinterpret_cast<const void*>(prod_kernel<MODE, F32>), P::kSmemBytes, attr_done);
  if (err != cudaSuccess) return err;
  if (tiles <= 0) return cudaSuccess;
  const int pairs = static_cast<int>(std::min<long long>(num_sms() / 2, tiles));
  return launch_pdl(prod_kernel<MODE, F32>, dim3(2 * pairs), dim3(P::kThr), P::kSmemBytes, stream, maps, args);
}

// Upper bound on the token-mode tiles of `rows` rows in `groups` groups.
long long token_tiles(long long rows, int groups, int N, int feat) {
  return ((rows + 255) / 256 + (groups > 1 ? groups : 0)) * ((N + feat - 1) / feat);
}

template <int MODE>
cudaError_t weight_grad(const void* a0, const void* a1, const void* b, const int32_t* offsets, int G, long long rows,
                        int N, int Kd, void* dw0, void* dw1, int f32, int accumulate, int late_wait, int* status,
                        int* sched, cudaStream_t stream) {
  ProdMaps m;
  if (!map_mn(&m.a[0], a0, N, rows, 1) || !map_mn(&m.a[1], a1 ? a1 : a0, N, rows, 1) ||
      !map_bf16_2d(&m.b[0].box[0], b, Kd, rows, kBK) || !map_grad_tiles(&m.o[0], dw0, Kd, N, G, f32 != 0) ||
      !map_grad_tiles(&m.o[1], dw1 ? dw1 : dw0, Kd, N, G, f32 != 0))
    return cudaErrorInvalidValue;
  ProdArgs args{};
  args.offsets = offsets;
  args.G = G;
  args.M = static_cast<int>(rows);
  args.N = N;
  args.Kd = Kd;
  args.accumulate = accumulate;
  args.late_wait = late_wait;
  args.status = status;
  args.sched = sched;
  const long long tiles = static_cast<long long>(G) * ((N + Prod<MODE>::FEAT - 1) / Prod<MODE>::FEAT) *
                          ((Kd + Prod<MODE>::NT - 1) / Prod<MODE>::NT);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  return f32 ? launch_prod<MODE, true>(m, args, tiles, stream) : launch_prod<MODE, false>(m, args, tiles, stream);
}

}  // namespace

cudaError_t gemm_gate_up_train(const void* xp, const int32_t* offsets, const void* w_gate, const void* w_up, int E,
                               long long rows, int H, int F, float* g, float* u, void* h, int* status, int* sched,
                               cudaStream_t stream) {
  ProdMaps m;
  if (!map_bf16_3d(&m.a[0], w_gate, H, F, E, kBM) || !map_bf16_3d(&m.a[1], w_up, H, F, E, kBM) ||
      !map_token_boxes(&m.b[0], xp, H, rows, 2, 1))
    return cudaErrorInvalidValue;
  ProdArgs args{};
  args.offsets = offsets, args.G = E, args.M = static_cast<int>(rows), args.N = F, args.Kd = H, args.nt = 256, args.phases = 1;
  args.out = h, args.pre0 = g, args.pre1 = u, args.status = status, args.sched = sched;
  return launch_prod<kGateUpTrain>(m, args, token_tiles(rows, E, F, Prod<kGateUpTrain>::FEAT), stream);
}

cudaError_t gemm_down_bwd(const void* dy, const float* g, const float* u, const int32_t* offsets, const void* w_down,
                          int E, long long rows, int H, int F, void* dg, void* du, int* status, int* sched,
                          cudaStream_t stream) {
  ProdMaps m;
  if (!map_mn(&m.a[0], w_down, F, H, E) || !map_token_boxes(&m.b[0], dy, H, rows, 2, 1)) return cudaErrorInvalidValue;
  ProdArgs args{};
  args.offsets = offsets, args.G = E, args.M = static_cast<int>(rows), args.N = F, args.Kd = H, args.nt = 256, args.phases = 1;
  args.out = dg, args.out2 = du, args.g = g, args.u = u, args.status = status, args.sched = sched;
  return launch_prod<kDownBwd>(m, args, token_tiles(rows, E, F, Prod<kDownBwd>::FEAT), stream);
}

cudaError_t gemm_rows_bwd(const void* d0, const void* d1, const int32_t* offsets, const void* w0, const void* w1,
                          int G, long long rows, int N, int Kd, void* out, int* status, int* sched,
                          cudaStream_t stream) {
  ProdMaps m;
  if (!map_mn(&m.a[0], w0, N, Kd, G) || !map_token_boxes(&m.b[0], d0, Kd, rows, 2, 1)) return cudaErrorInvalidValue;
  if (d1 && (!map_mn(&m.a[1], w1, N, Kd, G) || !map_token_boxes(&m.b[1], d1, Kd, rows, 2, 1))) return cudaErrorInvalidValue;
  ProdArgs args{};
  args.offsets = offsets, args.G = G, args.M = static_cast<int>(rows), args.N = N, args.Kd = Kd;
  args.nt = 256, args.phases = d1 ? 2 : 1, args.out = out, args.status = status, args.sched = sched;
  return launch_prod<kRowsBwd>(m, args, token_tiles(rows, G, N, Prod<kRowsBwd>::FEAT), stream);
}

cudaError_t gemm_grad_gate_up(const void* dg, const void* du, const void* xp, const int32_t* offsets, int E,
                              long long rows, int H, int F, void* dw_gate, void* dw_up, int f32, int accumulate,
                              int late_wait, int* status, int* sched, cudaStream_t stream) {
  return weight_grad<kGradGateUp>(dg, du, xp, offsets, E, rows, F, H, dw_gate, dw_up, f32, accumulate, late_wait,
                                  status, sched, stream);
}

cudaError_t gemm_grad_down(const void* dy, const void* h, const int32_t* offsets, int G, long long rows, int N, int Kd,
                           void* dw, int f32, int accumulate, int late_wait, int* status, int* sched,
                           cudaStream_t stream) {
  return weight_grad<kGradDown>(dy, nullptr, h, offsets, G, rows, N, Kd, dw, nullptr, f32, accumulate, late_wait,
                                status, sched, stream);
}

cudaError_t gemm_dense_epilogue(const void* a, const void* w, const float* bias, const void* residual, int act,
                                long long M, int N, int Kd, void* out, float* pre, int* status, int* sched,
                                cudaStream_t stream) {
  ProdMaps m;
  if (!map_bf16_3d(&m.a[0], w, Kd, N, 1, kBM) || !map_bf16_3d(&m.aw, w, Kd, N, 1, 2 * kBM) ||
      !map_token_boxes(&m.b[0], a, Kd, M, 2, 1))
    return cudaErrorInvalidValue;
  ProdArgs args{};
  args.G = 1, args.M = static_cast<int>(M), args.N = N, args.Kd = Kd, args.nt = dense_rows(M, N), args.phases = 1;
  args.out = out, args.pre0 = pre, args.bias = bias, args.residual = residual, args.act = act;
  args.status = status, args.sched = sched;
  const long long tiles = (M + args.nt - 1) / args.nt * ((N + Prod<kDense>::FEAT - 1) / Prod<kDense>::FEAT);
  return launch_prod<kDense>(m, args, tiles, stream);
}

}  // namespace moe
