// gemm_common.cuh - what the tcgen05 GEMM kernels share: tile sizes, the tile table of a
// grouped launch, row stores through shared memory and the tensor maps.
#pragma once

#include <algorithm>
#include <mutex>

#include "device.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kBM = 128;                  // output features per tile (MMA M)
constexpr int kBK = 64;                   // K per stage: one 128-byte swizzle atom of bf16
constexpr int kABytes = kBM * kBK * 2;    // 16 KB per weight tile
// The token operand of a tile (nround rows, a multiple of 16) is fetched with one TMA box
// per set bit of nround: boxes of 256, 128, 64, 32 and 16 rows (single CTA), or of 128 down to 8
// rows for each CTA's half of a CTA-pair tile.
constexpr int kNumBoxes = 6;
struct BoxMaps {
  CUtensorMap box[kNumBoxes];  // box[i] is (256 >> i) rows x 64 columns
};
constexpr int kMaxGroups = MOE_MAX_E;
constexpr int kRing = 8;                 // tile ids in flight from the producer to the MMA and epilogue warps

struct Tile {
  int g, n0, row0, nvalid, nround;
};

// bf16 outputs leave through a per-warp 32 x 32 transpose in shared memory: the thread of
// feature fbase + lane holds v[j] for tokens row0 + j, a token row wants 32 consecutive
// features, so each lane then writes whole 16-byte pieces of rows (four per 32-token chunk)
// instead of 32 scattered 2-byte values.  Rows j >= jn and features >= N are not written.
__device__ __forceinline__ void store_rows32(__nv_bfloat16* stg, int lane, const float (&v)[32],
                                             __nv_bfloat16* out, long long ldo, int N, int fbase, long long row0,
                                             int jn) {
#pragma unroll
  for (int j = 0; j < 32; ++j) stg[j * 32 + lane] = __float2bfloat16_rn(v[j]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 8 * i + (lane >> 2), c = 8 * (lane & 3);
    if (j < jn && fbase + c < N)
      *reinterpret_cast<uint4*>(out + (row0 + j) * ldo + fbase + c) = *reinterpret_cast<const uint4*>(stg + j * 32 + c);
  }
  __syncwarp();
}

// store_rows32 through a TMA tile store: the 32 x 32 chunk (tokens x features) is staged as 32
// rows of 64 bytes and one lane stores it as one box of `map` (the output, box 32 x 32, no
// swizzle), which completes in the background: the warp goes on (and hands TMEM back) while the
// rows drain.  A chunk with fewer than 32 valid rows takes store_rows32's 16-byte stores, since
// the box would also write the first rows of the next group.  The staging tile is reused only
// after the previous chunk's store has read it.
__device__ __forceinline__ void store_rows32_tma(__nv_bfloat16* stg, int lane, const float (&v)[32],
                                                 const CUtensorMap* map, __nv_bfloat16* out, long long ldo, int N,
                                                 int fbase, long long row0, int jn) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
  if (jn < 32) {
    store_rows32(stg, lane, v, out, ldo, N, fbase, row0, jn);
    return;
  }
  if (fbase >= N) return;
#pragma unroll
  for (int j = 0; j < 32; ++j) stg[j * 32 + lane] = __float2bfloat16_rn(v[j]);
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, stg, fbase, static_cast<int>(row0));
    bulk_commit_group();
  }
}

// Tile t -> (group, weight tile, token chunk).  s_pre[g] = first tile of group g.  A group of
// cnt rows is cut into ceil(cnt / NT) balanced chunks of a multiple of ROUND rows; a weight
// tile covers FEAT output features.
template <int ROUND, int FEAT>
__device__ __forceinline__ Tile decode_tile(int t, const int* s_pre, const int* s_off, int G, int NT) {
  int lo = 0, hi = G;  // s_pre[lo] <= t < s_pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_pre[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int local = t - s_pre[lo];
  const int cnt = s_off[lo + 1] - s_off[lo];
  const int nch = (cnt + NT - 1) / NT;
  const int ft = local / nch;
  const int c = local - ft * nch;
  const int sz = (((cnt + nch - 1) / nch) + ROUND - 1) & ~(ROUND - 1);
  Tile r;
  r.g = lo;
  r.n0 = ft * FEAT;
  r.row0 = s_off[lo] + c * sz;
  r.nvalid = min(sz, cnt - c * sz);
  r.nround = (r.nvalid + ROUND - 1) & ~(ROUND - 1);
  return r;
}

template <int NT, int ROUND, int FEAT>
__device__ __forceinline__ Tile decode_tile(int t, const int* s_pre, const int* s_off, int G) {
  return decode_tile<ROUND, FEAT>(t, s_pre, s_off, G, NT);
}

// s_pre[g] = sum_{g' < g} ceil(cnt_g' / NT) * NFT for g = 0..G (block-wide scan).
__device__ void build_tile_table(int* s_pre, const int* s_off, int G, int NT, int NFT, int* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthreads = blockDim.x;
  const int seg = (G + nthreads - 1) / nthreads;
  const int b = min(G, tid * seg), e = min(G, b + seg);
  int local = 0;
  for (int g = b; g < e; ++g) local += ((s_off[g + 1] - s_off[g] + NT - 1) / NT) * NFT;
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (tid == 0) {
    int run = 0;
    for (int w = 0; w < nthreads / 32; ++w) {
      const int v = s_warp[w];
      s_warp[w] = run;
      run += v;
    }
    s_pre[G] = run;
  }
  __syncthreads();
  int run = s_warp[warp] + incl - local;
  for (int g = b; g < e; ++g) {
    s_pre[g] = run;
    run += ((s_off[g + 1] - s_off[g] + NT - 1) / NT) * NFT;
  }
  __syncthreads();
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Tensor [d2][d1][d0] (d0 contiguous) of bf16 (elem = 2) or 8-bit codes (elem = 1), box
// {128 bytes of d0, box1, 1}, 128-byte swizzle.
bool map_bf16_3d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t box1,
                 int elem = 2) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {d0 * elem, d0 * d1 * elem};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem), box1, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
             const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_bf16_2d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint32_t box1, int elem = 2) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {d0, d1};
  const cuuint64_t strides[1] = {d0 * elem};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), box1};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
             const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `first` to `last`: the boxes that the kernel uses (encoding one takes about 0.1 us of the host's time).
bool map_token_boxes(BoxMaps* m, const void* base, uint64_t d0, uint64_t rows, int elem = 2, int first = 0,
                     int last = kNumBoxes - 1) {
  for (int i = first; i <= last; ++i)
    if (!map_bf16_2d(&m->box[i], base, d0, rows, 256u >> i, elem)) return false;
  return true;
}

// Output map of the pair kernel's tile stores: out [M][N] bf16 (row stride ldo), box 32 x 32.
bool map_out_tiles(CUtensorMap* m, const GemmArgs& args) {
  EncodeTiledFn enc = encoder();
  if (!enc || args.N <= 0 || args.M <= 0) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(args.N), static_cast<cuuint64_t>(args.M)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(args.ldo) * 2};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, args.out, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace moe
