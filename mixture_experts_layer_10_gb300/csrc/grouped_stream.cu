// Grouped products of few rows a group (decode steps, small batches): y = x W[g]^T, 16-bit or with 8-bit
// integers.  Such a product is one read of the weights of the groups that have rows, so the kernel is
// built around that read.  A tile is 32 features of one group and up to 8 or 32 of its rows: small enough
// that one token's 8 experts x 768 features (192 tiles) keep every SM reading, where the 256-feature
// tiles of the tensor-memory kernel occupy 48.  One thread of a block streams the tiles' weights as TMA
// boxes, 512 bytes of every row, into a ring of stages, across tile borders; eight warps multiply with
// mma.sync, each its own 64 bytes of the stage's rows, and add up through shared memory in a fixed order
// at the end of a tile.  (Register fragments: at a few rows a weight the tensor rate is not what counts, and
// 8-bit codes widen to fp16 on their way from shared memory to the fragment.)  The order in which the
// products of a sum are taken is free, so lane (r, c) of a fragment holds 16 consecutive bytes of rows
// r and r + 8, as one load delivers them.  x comes from L2 straight into fragments, on its way while the
// stage is waited for.  Rows of a group past those of a tile make another tile, whose weights come from L2.
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

namespace moe {

namespace {

enum Type { kBf16, kFp16, kCodes };

constexpr int kWarps = 8;                  // that multiply
constexpr int kFeat = 32;                  // features of a tile
constexpr int kBoxCols = 128;              // bytes of a row in a box
constexpr int kBoxes = kWarps / 2;         // boxes of a stage, side by side
constexpr uint32_t kBoxBytes = kFeat * kBoxCols, kStage = kBoxes * kBoxBytes;
constexpr int kCols = kBoxes * kBoxCols;   // bytes of a row in a stage
constexpr int kPitch = kFeat + 4;          // floats between the rows of the partial sums

struct StreamParams {
  CUtensorMap W;            // bytes: [G, N, row_bytes] in boxes of 128 bytes x 32 rows
  const int32_t *begin, *end;
  const uint8_t* x;         // rows ldx bytes apart
  const float *xs, *ws;     // scales (8-bit integers)
  uint16_t* y;
  int64_t rows, ldx, ldy;   // ldx in bytes, ldy in elements
  int row_bytes;            // of a row of W or x
  int N, G, nf;             // nf: feature tiles of a group
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

// 16 bytes of x, zero where not `in`.
__device__ __forceinline__ uint4 load_x(const uint8_t* at, bool in) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(at), "r"((int)in));
  return v;
}

// A barrier of the eight multiplying warps.
__device__ __forceinline__ void bar_warps() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// NT: 8-row tiles.
template <int kType, int NT, int kDepth>
__global__ void __launch_bounds__(32 * (kWarps + 1), 2) stream_kernel(const __grid_constant__ StreamParams p) {
  constexpr int kRows = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(ring + kDepth * kStage);   // partial sums [kWarps][kRows][kPitch]
  __shared__ GroupTab tab;
  __shared__ uint64_t full[kDepth], empty[kDepth];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDepth; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    abort_word = 0;
    fence_mbar_init();
    tma_prefetch(&p.W);
  }
  const int tiles = load_groups(tab, p.begin, p.end, p.G, p.rows, kRows, p.hdr);   // (a barrier of the block, too)
  const int ntiles = max(tiles, 0) * p.nf;
  const int nst = (p.row_bytes + kCols - 1) / kCols;
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
      for (int t = blockIdx.x; ok && t < ntiles; t += gridDim.x) {
        const Tile j = tile_of(t);
        for (int s = 0; s < nst; ++s) {
          ok = mbar_wait(&empty[slot], phase ^ 1, limit, abort_flag);
          if (!ok) {
            record_error(p.hdr, MOE_ERR_TIMEOUT, kSiteGroupedProducer);
            *abort_flag = 1;
            break;
          }
          if (uses != skip) {
            uint8_t* st = ring + (size_t)slot * kStage;
            const int boxes = min(kBoxes, (p.row_bytes - s * kCols + kBoxCols - 1) / kBoxCols);
            mbar_arrive_expect_tx(&full[slot], boxes * kBoxBytes);
            for (int b = 0; b < boxes; ++b)
              tma_load_3d(st + b * kBoxBytes, &p.W, &full[slot], s * kCols + b * kBoxCols, j.f0, j.g);
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
    return;
  }

  // this warp's 64 bytes: the even or odd 16-byte chunks of a box, which in the 128-byte swizzle keep the
  // banks of eight lanes distinct
  const int chunk = 2 * c + (warp & 1), col = warp / 2 * kBoxCols + chunk * 16;
  const uint32_t wat = warp / 2 * kBoxBytes + r * kBoxCols + ((chunk ^ r) << 4);
  for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
    const Tile j = tile_of(t);
    const int nt = (j.n + 7) / 8;
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][k][v] = 0.f;
    const uint8_t* xrow = p.x + j.row0 * p.ldx + col;
#pragma unroll 1
    for (int s = 0; s < nst && ok; ++s) {
      // (rows past the tile's last are read as that: nothing stores their products)
      uint4 x[NT];
#pragma unroll
      for (int k = 0; k < NT; ++k)
        x[k] = load_x(xrow + min(8 * k + r, j.n - 1) * p.ldx + s * kCols, k < nt && s * kCols + col < p.row_bytes);
      ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], phase, limit, abort_flag));
      if (!ok) {   // keeps to the barriers below, so that no warp waits for it in vain
        if (lane == 0) {
          record_error(p.hdr, MOE_ERR_TIMEOUT, kSiteGroupedMma);
          *abort_flag = 1;
        }
        break;
      }
      if (s * kCols + warp / 2 * kBoxCols < p.row_bytes) {   // the stage has this warp's box
        const uint8_t* st = ring + (size_t)slot * kStage + wat;
        uint4 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint4*>(st + e * 8 * kBoxCols);
        if (kType == kCodes) {
          uint4 a[4][2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e][0] = widen(w[e].x, w[e].y);
            a[e][1] = widen(w[e].z, w[e].w);
          }
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            if (k >= nt) break;
            const uint4 x0 = widen(x[k].x, x[k].y), x1 = widen(x[k].z, x[k].w);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              step<kFp16>(acc[i][k], a[2 * i][0], a[2 * i + 1][0], x0);
              step<kFp16>(acc[i][k], a[2 * i][1], a[2 * i + 1][1], x1);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            if (k >= nt) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) step<kType>(acc[i][k], w[2 * i], w[2 * i + 1], x[k]);
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

    bar_warps();   // the previous tile's sums have been read
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[(warp * kRows + 8 * k + 2 * c + (v & 1)) * kPitch + 16 * i + r + 8 * (v >> 1)] = acc[i][k][v];
    bar_warps();
    // two features of a row a thread
    for (int e = threadIdx.x; e < j.n * (kFeat / 2); e += 32 * kWarps) {
      const int fl = e % (kFeat / 2) * 2, row = e / (kFeat / 2), f = j.f0 + fl;
      if (f >= p.N) continue;   // N is a multiple of 8
      const float* from = red + row * kPitch + fl;
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 part = *reinterpret_cast<const float2*>(from + k * kRows * kPitch);
        v0 += part.x;
        v1 += part.y;
      }
      if (kType == kCodes) {
        const float2 ws = __ldg(reinterpret_cast<const float2*>(p.ws + (int64_t)j.g * p.N + f));
        const float xs = p.xs[j.row0 + row];
        v0 = v0 * ws.x * xs;
        v1 = v1 * ws.y * xs;
      }
      *reinterpret_cast<uint32_t*>(p.y + (j.row0 + row) * p.ldy + f) = pack16(v0, v1, p.fp16);
    }
  }
}

template <int kType, int NT, int kDepth>
cudaError_t launch_stream(const Grouped& c, StreamParams& p, const void* W, int id, cudaStream_t s) {
  constexpr int smem = 1024 + kDepth * kStage + kWarps * 8 * NT * kPitch * 4;
  static_assert(smem + sizeof(GroupTab) + 256 <= 232448 / 2 - 1024, "shared memory of an SM");
  auto fn = encode_fn();
  const cuuint64_t row = (cuuint64_t)p.row_bytes;
  const cuuint64_t dims[3] = {row, (cuuint64_t)c.N, (cuuint64_t)c.G}, strides[2] = {row, row * c.N};
  const cuuint32_t box[3] = {kBoxCols, kFeat, 1}, es[3] = {1, 1, 1};
  if (!fn || fn(&p.W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(W), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  p.nf = (c.N + kFeat - 1) / kFeat;
  const int64_t tiles = (std::min<int64_t>(c.G, c.rows) + c.rows / (8 * NT)) * p.nf;   // at most
  auto kernel = stream_kernel<kType, NT, kDepth>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  prof_mark(id, s, true);
  kernel<<<(int)std::min<int64_t>(tiles, 2 * (int64_t)num_sms()), 32 * (kWarps + 1), smem, s>>>(p);
  prof_mark(id, s, false);
  return cudaGetLastError();
}

template <int kType>
cudaError_t launch_type(const Grouped& c, StreamParams& p, const void* W, int id, cudaStream_t s) {
  return c.rows <= 8 ? launch_stream<kType, 1, 5>(c, p, W, id, s) : launch_stream<kType, 4, 3>(c, p, W, id, s);
}

StreamParams stream_params(const Grouped& c, const int32_t* begin, const int32_t* end, const void* x, uint16_t* y,
                           int size, Hdr* hdr) {
  StreamParams p{};
  p.begin = begin;
  p.end = end;
  p.x = static_cast<const uint8_t*>(x);
  p.y = y;
  p.rows = c.rows;
  p.ldx = c.ldi * size;
  p.ldy = c.ldo;
  p.row_bytes = c.K * size;
  p.N = c.N;
  p.G = c.G;
  p.fp16 = c.fp16;
  p.hdr = hdr;
  return p;
}

}  // namespace

bool stream_eligible(const Grouped& c) { return c.rows <= 32 * (int64_t)c.G || c.rows <= 64; }

cudaError_t launch_stream_mm(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* x,
                             const uint16_t* W, uint16_t* y, Hdr* hdr, cudaStream_t s) {
  StreamParams p = stream_params(c, begin, end, x, y, 2, hdr);
  return c.fp16 ? launch_type<kFp16>(c, p, W, kKGroupedMm, s) : launch_type<kBf16>(c, p, W, kKGroupedMm, s);
}

cudaError_t launch_stream_i8(const Grouped& c, const int32_t* begin, const int32_t* end, const int8_t* q,
                             const float* qs, const int8_t* Wq, const float* Ws, uint16_t* y, Hdr* hdr,
                             cudaStream_t s) {
  StreamParams p = stream_params(c, begin, end, q, y, 1, hdr);
  p.xs = qs;
  p.ws = Ws;
  return launch_type<kCodes>(c, p, Wq, kKGroupedI8, s);
}

}  // namespace moe
