// Grouped products of few rows a group (decode steps, small batches): y = x W[g]^T, 16-bit or with 8-bit
// integers.  Such a product is one read of the weights of the groups that have rows, so the kernel is
// built around that read.  A tile is 128 features of one group and up to 8 or 32 of its rows; one thread
// of a block streams the tiles' W and x as TMA boxes, 128 bytes of every row, into a ring of stages,
// across tile borders, and eight warps multiply 16 features each with mma.sync.  (Register fragments: at
// a few rows a weight the tensor rate is not what counts, and 8-bit codes widen to fp16 on their way
// from shared memory to the fragment.)  The order in which the products of a sum are taken is free, so
// lane (r, c) of a fragment holds 16 consecutive bytes of rows r and r + 8, as one load delivers them.
//
// Where the tiles are fewer than the blocks that fit (one token's 8 experts x 768 features are 48), a
// cluster of 2, 4 or 8 blocks splits the contraction of a tile, and each block adds up its share of the
// tile's partial sums, in the order of the blocks, from the others' shared memory.  A cluster has one tile
// then: the split is chosen so that there is a cluster for every tile that the rows can make.  Rows of a
// group past those of a tile make another tile, whose weights come from L2.
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

namespace moe {

namespace {

enum Type { kBf16, kFp16, kCodes };

constexpr int kWarps = 8;                  // that multiply
constexpr int kFeat = 16 * kWarps;         // features of a tile
constexpr int kCols = 128;                 // bytes of a row in a stage
constexpr int kMaxSplit = 8;               // blocks of a cluster
constexpr int kPairRows = 256;             // rows of a tile of the pairs' kernel
constexpr int kPitch = kFeat + 4;          // floats between the rows of the partial sums

struct StreamParams {
  CUtensorMap W, x;         // bytes: [G, N, row_bytes] in boxes of 128 rows, [rows, row_bytes] in boxes of 8 NT
  const int32_t *begin, *end;
  const float *xs, *ws;     // scales (8-bit integers)
  uint16_t* y;
  int64_t rows, ldy;
  int nst, N, G, nf;        // stages of a tile; feature tiles of a group
  int split;                // blocks of a cluster
  bool fp16;                // y's type
  Hdr* hdr;
};

template <int kType>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (kType == kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d += the products of 16 bytes of two rows of W a lane (16 features) and of one row of x (8 rows).
template <int kType>
__device__ __forceinline__ void step(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& x) {
  mma<kType>(d, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
  mma<kType>(d, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

__device__ __forceinline__ float2 load_peer(const float* p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(cluster_addr(p, rank))
               : "memory");
  return v;
}

// NT: 8-row tiles.
template <int kType, int NT, int kDepth, int kBlocks>
__global__ void __launch_bounds__(32 * (kWarps + 1), kBlocks) stream_kernel(const __grid_constant__ StreamParams p) {
  constexpr int kRows = 8 * NT;
  constexpr uint32_t kWBytes = kFeat * kCols, kStage = kWBytes + kRows * kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(ring + kDepth * kStage);   // partial sums [kRows][kPitch]
  __shared__ GroupTab tab;
  __shared__ uint64_t full[kDepth], empty[kDepth];
  __shared__ uint64_t sums;   // every block's partial sums are in place
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDepth; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    mbar_init(&sums, kWarps * p.split);
    abort_word = 0;
    fence_mbar_init();
    tma_prefetch(&p.W);
    tma_prefetch(&p.x);
  }
  after_previous_kernel();
  const int tiles = load_groups(tab, p.begin, p.end, p.G, p.rows, kRows, p.hdr);   // (a barrier of the block, too)
  if (p.split > 1) cluster_sync();   // all blocks' barriers exist before any remote arrival
  const int ntiles = max(tiles, 0) * p.nf;
  const int rank = p.split > 1 ? (int)cluster_rank() : 0;
  const int first = blockIdx.x / p.split, stride = gridDim.x / p.split;
  const int per = (p.nst + p.split - 1) / p.split;                    // this block's stages of a tile
  const int s0 = min(p.nst, rank * per), s1 = min(p.nst, s0 + per);
  const uint64_t limit = wait_limit_ns(p.hdr);

  struct Tile {
    int g, f0, row0, n;
  };
  // the group of row tile t / nf; within a group the row tiles of a feature tile follow each other
  auto tile_of = [&](int t) {
    const int m = t / p.nf;
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= m) lo = mid; else hi = mid - 1;
    }
    const int mt = tab.first[lo + 1] - tab.first[lo];
    const int local = t - tab.first[lo] * p.nf;
    const int ft = mt == 1 ? local : local / mt;
    Tile j;
    j.g = lo;
    j.f0 = ft * kFeat;
    j.row0 = tab.begin[lo] + (local - ft * mt) * kRows;
    j.n = min(kRows, tab.end[lo] - j.row0);
    return j;
  };

  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  if (warp == kWarps) {
    if (lane == 0) {
      int uses = 0;
      // test hook: the first block skips one fill, so that the wait for it runs out
      const int skip = blockIdx.x == 0 ? *((volatile const int32_t*)&p.hdr->stall_fill_p1) - 1 : -1;
      for (int t = first; ok && t < ntiles; t += stride) {
        const Tile j = tile_of(t);
        for (int s = s0; s < s1; ++s) {
          ok = wait_nap<20>(&empty[slot], phase ^ 1, limit, abort_flag);
          if (!ok) {
            record_error(p.hdr, MOE_ERR_TIMEOUT, kSiteGroupedProducer);
            *abort_flag = 1;
            break;
          }
          if (uses != skip) {
            uint8_t* st = ring + (size_t)slot * kStage;
            mbar_arrive_expect_tx(&full[slot], kStage);
            tma_load_3d(st, &p.W, &full[slot], s * kCols, j.f0, j.g);
            tma_load_2d(st + kWBytes, &p.x, &full[slot], s * kCols, j.row0);
          }
          ++uses;
          if (++slot == kDepth) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      drain_fills(full, kDepth, slot, phase, uses, limit);   // every copy lands before the block exits
    }
  }
  for (int t = first; warp < kWarps && t < ntiles; t += stride) {
    const Tile j = tile_of(t);
    float acc[NT][4];
    {
      const int nt = (j.n + 7) / 8;
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[k][v] = 0.f;
#pragma unroll 1
      for (int s = s0; s < s1 && ok; ++s) {
        ok = __all_sync(0xffffffffu, wait_nap<0>(&full[slot], phase, limit, abort_flag));
        if (!ok) {   // still arrives at the cluster's barrier below, so that no block waits for it in vain
          if (lane == 0) {
            record_error(p.hdr, MOE_ERR_TIMEOUT, kSiteGroupedMma);
            *abort_flag = 1;
          }
          break;
        }
        // chunk 2 c + u of a row: with the 128-byte swizzle eight lanes read distinct banks
        const uint8_t* wst = ring + (size_t)slot * kStage + (warp * 16 + r) * kCols;
        const uint8_t* xst = ring + (size_t)slot * kStage + kWBytes + r * kCols;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = ((2 * c + u) ^ r) << 4;
          const uint4 lo = *reinterpret_cast<const uint4*>(wst + at);
          const uint4 hi = *reinterpret_cast<const uint4*>(wst + 8 * kCols + at);
          if (kType == kCodes) {
            const uint4 lo0 = widen(lo.x, lo.y), lo1 = widen(lo.z, lo.w);
            const uint4 hi0 = widen(hi.x, hi.y), hi1 = widen(hi.z, hi.w);
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              if (k >= nt) break;
              const uint4 x = *reinterpret_cast<const uint4*>(xst + k * 8 * kCols + at);
              step<kFp16>(acc[k], lo0, hi0, widen(x.x, x.y));
              step<kFp16>(acc[k], lo1, hi1, widen(x.z, x.w));
            }
          } else {
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              if (k >= nt) break;
              step<kType>(acc[k], lo, hi, *reinterpret_cast<const uint4*>(xst + k * 8 * kCols + at));
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == kDepth) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    if (p.split == 1) {
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = j.f0 + warp * 16 + r + 8 * h;
        if (f >= p.N) continue;
        const float ws = kType == kCodes ? p.ws[(int64_t)j.g * p.N + f] : 1.f;
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int row = 8 * k + 2 * c + v;
            if (row >= j.n) continue;
            float out = acc[k][2 * h + v];
            if (kType == kCodes) out = out * ws * p.xs[j.row0 + row];
            p.y[(j.row0 + row) * p.ldy + f] = (uint16_t)pack16(out, 0.f, p.fp16);
          }
      }
      continue;
    }
    // the cluster's one tile (its barrier is used once)
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[(8 * k + 2 * c + (v & 1)) * kPitch + warp * 16 + r + 8 * (v >> 1)] = acc[k][v];
    __syncwarp();
    if (lane < p.split) {
      fence_release_smem();
      mbar_arrive_cluster_relaxed(cluster_addr(&sums, lane));
    }
    if (ok) {
      ok = __all_sync(0xffffffffu, wait_nap<0, true>(&sums, 0, limit, abort_flag));
      if (!ok && lane == 0) {
        record_error(p.hdr, MOE_ERR_TIMEOUT, kSiteGroupedEpilogue);
        *abort_flag = 1;
      }
    }
    if (ok) {
      // two features of a row a thread
#pragma unroll 1
      for (int e = rank * 32 * kWarps + threadIdx.x; e < j.n * (kFeat / 2); e += p.split * 32 * kWarps) {
        const int fl = e % (kFeat / 2) * 2, row = e / (kFeat / 2), f = j.f0 + fl;
        if (f >= p.N) continue;   // N is a multiple of 8
        float2 part[kMaxSplit];   // all on their way before the first sum
#pragma unroll
        for (int s = 0; s < kMaxSplit; ++s)
          if (s < p.split) part[s] = load_peer(red + row * kPitch + fl, s);
        float2 v = part[0];
#pragma unroll
        for (int s = 1; s < kMaxSplit; ++s)
          if (s < p.split) v = make_float2(v.x + part[s].x, v.y + part[s].y);
        if (kType == kCodes) {
          const float* ws = p.ws + (int64_t)j.g * p.N + f;   // (aligned as floats are)
          const float xs = p.xs[j.row0 + row];
          v = make_float2(v.x * __ldg(ws) * xs, v.y * __ldg(ws + 1) * xs);
        }
        *reinterpret_cast<uint32_t*>(p.y + (j.row0 + row) * p.ldy + f) = pack16(v.x, v.y, p.fp16);
      }
    }
    break;
  }
  __syncwarp();
  if (p.split > 1) cluster_sync();   // no block ends while another may read its sums or arrive at its barriers
}

template <int kType, int NT, int kDepth, int kBlocks>
cudaError_t launch_stream(const Grouped& c, StreamParams& p, const void* x, const void* W, int size, int id,
                          cudaStream_t s) {
  constexpr int smem = 1024 + kDepth * (kFeat + 8 * NT) * kCols + 8 * NT * kPitch * 4;
  static_assert(smem + sizeof(GroupTab) + 256 <= 232448 / kBlocks - 1024, "shared memory of an SM");
  auto fn = encode_fn();
  const cuuint64_t row = (cuuint64_t)c.K * size;
  const cuuint64_t wdims[3] = {row, (cuuint64_t)c.N, (cuuint64_t)c.G}, wstrides[2] = {row, row * c.N};
  const cuuint64_t xdims[2] = {row, (cuuint64_t)c.rows}, xstrides[1] = {(cuuint64_t)c.ldi * size};
  const cuuint32_t wbox[3] = {kCols, kFeat, 1}, xbox[2] = {kCols, 8 * NT}, es[3] = {1, 1, 1};
  if (!fn ||
      fn(&p.W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(W), wdims, wstrides, wbox, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      fn(&p.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(x), xdims, xstrides, xbox, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  p.nst = (int)((row + kCols - 1) / kCols);
  p.nf = (c.N + kFeat - 1) / kFeat;
  // blocks of a cluster: as many as all fit at once (one token, 8 of 128 experts, 2048 x 768: 7.7 us, 14.3 with
  // one block a tile; 37 rows, 8-bit integers, 4096 x 4096: 16.9 and 35.4).  More tiles than that only lose by the cluster's sums: 64 x 2048 x 1408, one row a group,
  // 62 us with one block a tile, 65 with two.
  const int64_t live = std::min<int64_t>(c.G, c.rows), slots = kBlocks * (int64_t)num_sms();
  const int64_t tiles = (live + (c.rows - live) / (8 * NT)) * p.nf;   // the most that any spread of the rows makes
  p.split = 1;
  while (p.split < kMaxSplit && 2 * p.split * tiles <= slots && 2 * p.split <= p.nst) p.split *= 2;
  const int grid = (int)std::min<int64_t>(p.split * tiles, slots);   // (split > 1: a cluster a tile, see above)
  auto kernel = stream_kernel<kType, NT, kDepth, kBlocks>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  prof_mark(id, s, true);
  e = launch_after(kernel, grid, 32 * (kWarps + 1), smem, p.split, s, p);
  prof_mark(id, s, false);
  return e;
}

template <int kType>
cudaError_t launch_type(const Grouped& c, StreamParams& p, const void* x, const void* W, int id, cudaStream_t s) {
  constexpr int size = kType == kCodes ? 1 : 2;
  // up to 8 rows in all: tiles of 8, whose smaller stages let three blocks of an SM stream (one token as above
  // 7.7 us, 8.4 with tiles of 32; 8-bit integers, 2 of 8 experts of 4096 x 14336, 25.0 and 28.3 us)
  return c.rows <= 8 ? launch_stream<kType, 1, 3, 3>(c, p, x, W, size, id, s)
                     : launch_stream<kType, 4, 4, 2>(c, p, x, W, size, id, s);
}

StreamParams stream_params(const Grouped& c, const int32_t* begin, const int32_t* end, uint16_t* y, Hdr* hdr) {
  StreamParams p{};
  p.begin = begin;
  p.end = end;
  p.y = y;
  p.rows = c.rows;
  p.ldy = c.ldo;
  p.N = c.N;
  p.G = c.G;
  p.fp16 = c.fp16;
  p.hdr = hdr;
  return p;
}

}  // namespace

// Few rows a group: this kernel or the CTA pairs' of the same product.  By device time (graph replays, weights from
// HBM; this kernel : pairs) at one average of rows a group, evenly spread, or in brackets in proportion to
// exponential draws, where a group of more than 32 rows has its weights read again from L2:
//   64 groups of 2048 x 1408   8 rows 62.8 : 73 us (64 : 62)   16 rows 66 : 73 (72 : 63)   32 rows 74 : 75 (90 : 65)
//     8-bit integers           8 rows 39 : 82 (50 : 71)        16 rows 47 : 82 (72 : 73)   32 rows 67 : 82 (90 : 76)
//   8 groups of 4096 x 14336   8 rows 137 : 145 (138 : 146)    16 rows 139 : 146 (148 : 146)
//     8-bit integers           16 rows 98 : 150 (119 : 150)    32 rows 144 : 150 (219 : 154)
// so 8 rows a group on average, 16 with 8-bit integers.  Where the tiles are few, this kernel fills the GPU by its
// split of the contraction and the pairs do not:
//   64 tiles   4096 x 4096, 64 rows 17 : 23 (integers 17 : 30)     768 x 2048, 128 rows 8.2 : 8.8 (8.6 : 12.5)
//   88 tiles   2048 x 1408, 256 rows 17 : 15 (17.5 : 22.6)         44 tiles   the same, 128 rows 11 : 14 (11 : 20)
//   128 tiles  4096 x 4096, 128 rows 28 : 24 (29 : 33)             224 tiles  4096 x 14336, 64 rows 49 : 27 (50 : 32)
// so up to half a tile an SM, one with 8-bit integers, for at most the rows of one tile of the pairs.
// The rule sees the rows of the buffer and the number of groups, not the lengths (they are on the device).  So
// - all rows in one group, as many as the rule takes, are slower here, though faster than the even spread:
//     64 groups of 2048 x 1408   512 rows 26 : 15 us   8-bit integers, 1024 rows 43 : 24
//     8 groups of 4096 x 14336   64 rows 49 : 26 us    8-bit integers, 128 rows 95 : 33
// - rows in a larger buffer, as the layer's dispatch lays them out (up to 255 rows of padding a group), run on the
//   pairs however few they are: 8 rows of 8 of 128 groups, 2048 x 768, 14.7 us (8.0 packed), 8-bit 19.5 (7.9);
//   384 rows of 64 groups, 2048 x 1408, 73 us (63), 8-bit 81 (39).
bool stream_eligible(const Grouped& c, bool codes) {
  if (c.rows <= (codes ? 16 : 8) * (int64_t)c.G) return true;
  if (c.rows > kPairRows) return false;
  const int64_t live = std::min<int64_t>(c.G, c.rows), per = (c.rows + live - 1) / live;   // spread evenly
  return live * ((per + 31) / 32) * ((c.N + kFeat - 1) / kFeat) <= num_sms() / (codes ? 1 : 2);
}

cudaError_t launch_stream_mm(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* x,
                             const uint16_t* W, uint16_t* y, Hdr* hdr, cudaStream_t s) {
  StreamParams p = stream_params(c, begin, end, y, hdr);
  return c.fp16 ? launch_type<kFp16>(c, p, x, W, kKGroupedMm, s) : launch_type<kBf16>(c, p, x, W, kKGroupedMm, s);
}

cudaError_t launch_stream_i8(const Grouped& c, const int32_t* begin, const int32_t* end, const int8_t* q,
                             const float* qs, const int8_t* Wq, const float* Ws, uint16_t* y, Hdr* hdr,
                             cudaStream_t s) {
  StreamParams p = stream_params(c, begin, end, y, hdr);
  p.xs = qs;
  p.ws = Ws;
  return launch_type<kCodes>(c, p, q, Wq, kKGroupedI8, s);
}

}  // namespace moe
