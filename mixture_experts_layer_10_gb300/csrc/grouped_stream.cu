// Grouped products of few rows a group (decode steps, small batches): y = x W[g]^T, 16-bit or with 8-bit
// integers.  Such a product is one read of the weights of the groups that have rows, so the kernel is
// built around that read.  A warp takes 16 or 32 features of one group and streams their rows of W from
// global memory straight into the registers of mma.sync fragments: the order in which the products of a
// sum are taken is free, so lane (r, c) of a fragment may hold 16 consecutive bytes of rows r and r + 8,
// as one load delivers them, if the lanes of the x fragment hold the same places of a row of x.  No
// shared memory, barrier or tensor map stands between HBM and the tensor cores, and any number of
// warps can be at work: where the features are few, up to eight warps split K and add up through
// shared memory in a fixed order.  (tcgen05's 128-row tiles leave most SMs without work here: one token's
// 8 experts x 768 features are 48 of them.)  x is read from L1 and L2; rows of a group past the
// 8 NT of a tile make another tile, whose weights come from L2.
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"

namespace moe {

namespace {

enum Type { kBf16, kFp16, kCodes };

constexpr int kWarps = 8;

struct StreamParams {
  const int32_t *begin, *end;
  const uint8_t *x, *W;     // rows ldx bytes apart; weights [G, N, K]
  const float *xs, *ws;     // scales (8-bit integers)
  uint16_t* y;
  int64_t rows, ldx, ldy;   // ldx in bytes, ldy in elements
  int row_bytes;            // of a row of W or x
  int N, G, nf, wk_log2;    // feature tiles of a group; log2 of the warps that split K
  bool fp16;                // y's type
  Hdr* hdr;
};

// 16 bytes under a predicate (else zero): of a weight, which no other block reads, or of x.
__device__ __forceinline__ uint4 load_once(const uint8_t* at, bool in) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@p ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(at), "r"((int)in));
  return v;
}

__device__ __forceinline__ uint4 load_shared(const uint8_t* at, bool in) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(at), "r"((int)in));
  return v;
}

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

// MT: 16-feature tiles of a warp; NT: 8-row tiles; a chunk is 64 KC bytes of every row.  A warp has one
// chunk of W and x in flight, with nothing between the loads that waits; what hides their latency
// is the kBlocks x 8 warps of an SM, each at its own place.
template <int kType, int MT, int NT, int KC, int kBlocks>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) stream_kernel(const __grid_constant__ StreamParams p) {
  __shared__ GroupTab tab;
  extern __shared__ float red[];   // partial sums, [warp][MT][NT][4][32]
  constexpr int kFeat = 16 * MT, kRows = 8 * NT, kVals = MT * NT * 128;
  const int tiles = load_groups(tab, p.begin, p.end, p.G, p.rows, kRows, p.hdr);
  if (tiles < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  const int wk = 1 << p.wk_log2, part = warp & (wk - 1), fw = warp >> p.wk_log2, nfw = kWarps >> p.wk_log2;
  const int nchunk = (p.row_bytes + 64 * KC - 1) / (64 * KC);
  const int ntiles = tiles * p.nf;
  for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
    // the group of row tile t / nf; within a group the row tiles of a feature tile follow each other
    const int m = t / p.nf;
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= m) lo = mid; else hi = mid - 1;
    }
    const int mt = tab.first[lo + 1] - tab.first[lo];
    const int local = t - tab.first[lo] * p.nf;
    const int ft = mt == 1 ? local : local / mt;
    const int row0 = tab.begin[lo] + (local - ft * mt) * kRows;
    const int n = min(kRows, tab.end[lo] - row0);
    const int f0 = (ft * nfw + fw) * kFeat;
    const int nt = (n + 7) / 8;

    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][k][v] = 0.f;

    if (f0 < p.N) {
      // rows past the last feature are read as the last, rows past the group's last as that: nothing
      // stores their products
      const uint8_t* wrow[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wrow[i][h] = p.W + ((int64_t)lo * p.N + min(f0 + 16 * i + 8 * h + r, p.N - 1)) * p.row_bytes + c * 16;
      const uint8_t* xrow = p.x + row0 * p.ldx + c * 16;
#pragma unroll 1
      for (int ch = part; ch < nchunk; ch += wk) {
        uint4 w[KC][MT][2], x[KC][NT];
#pragma unroll
        for (int u = 0; u < KC; ++u) {
          const int at = (ch * KC + u) * 64;
          const bool in = at + c * 16 < p.row_bytes;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[u][i][h] = load_once(wrow[i][h] + at, in);
#pragma unroll
          for (int k = 0; k < NT; ++k) x[u][k] = load_shared(xrow + min(8 * k + r, n - 1) * p.ldx + at, in && k < nt);
        }
#pragma unroll
        for (int u = 0; u < KC; ++u) {
          if (kType == kCodes) {
            uint4 a[MT][2][2];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                a[i][h][0] = widen(w[u][i][h].x, w[u][i][h].y);
                a[i][h][1] = widen(w[u][i][h].z, w[u][i][h].w);
              }
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              if (k >= nt) break;
              const uint4 x0 = widen(x[u][k].x, x[u][k].y), x1 = widen(x[u][k].z, x[u][k].w);
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                step<kFp16>(acc[i][k], a[i][0][0], a[i][1][0], x0);
                step<kFp16>(acc[i][k], a[i][0][1], a[i][1][1], x1);
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              if (k >= nt) break;
#pragma unroll
              for (int i = 0; i < MT; ++i) step<kType>(acc[i][k], w[u][i][0], w[u][i][1], x[u][k]);
            }
          }
        }
      }
    }

    auto put = [&](int f, int row, float v) {
      if (f >= p.N || row >= n) return;
      if (kType == kCodes) v = v * p.ws[(int64_t)lo * p.N + f] * p.xs[row0 + row];
      p.y[(row0 + row) * p.ldy + f] = (uint16_t)pack16(v, 0.f, p.fp16);
    };
    if (wk == 1) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int v = 0; v < 4; ++v) put(f0 + 16 * i + r + 8 * (v >> 1), 8 * k + 2 * c + (v & 1), acc[i][k][v]);
    } else {
      float* mine = red + warp * kVals + lane;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int v = 0; v < 4; ++v) mine[((i * NT + k) * 4 + v) * 32] = acc[i][k][v];
      __syncthreads();
      // feature fastest, so that a warp stores runs of a row; the parts of a sum in their order
      for (int e = threadIdx.x; e < nfw * n * kFeat; e += 32 * kWarps) {
        const int f = e % kFeat, wr = e / kFeat, w0 = nfw == 1 ? 0 : wr / n, row = wr - w0 * n;
        const int at = ((f / 16 * NT + row / 8) * 4 + (f % 16 / 8) * 2 + row % 2) * 32 + f % 8 * 4 + row % 8 / 2;
        const float* from = red + (w0 << p.wk_log2) * kVals + at;
        float v = 0.f;
        for (int k = 0; k < wk; ++k) v += from[k * kVals];
        put((ft * nfw + w0) * kFeat + f, row, v);
      }
      __syncthreads();
    }
  }
}

template <int kType, int MT, int NT, int KC, int kBlocks>
cudaError_t launch_stream(const Grouped& c, StreamParams p, int id, cudaStream_t s) {
  constexpr int smem = kWarps * MT * NT * 128 * 4;
  static_assert(smem + sizeof(GroupTab) <= 232448 / kBlocks - 1024, "shared memory of an SM");
  const int64_t live = std::min<int64_t>(c.G, c.rows);
  const int per = (c.N + 16 * MT - 1) / (16 * MT);   // features of a group, in warps
  // warps that split K: enough for sixteen warps an SM
  p.wk_log2 = 0;
  while (p.wk_log2 < 3 && ((live * per) << p.wk_log2) < (int64_t)num_sms() * 16) ++p.wk_log2;
  p.nf = ((per << p.wk_log2) + kWarps - 1) / kWarps;
  const int64_t tiles = (c.rows / (8 * NT) + live) * p.nf;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(stream_kernel<kType, MT, NT, KC, kBlocks>), smem);
  if (e != cudaSuccess) return e;
  prof_mark(id, s, true);
  stream_kernel<kType, MT, NT, KC, kBlocks>
      <<<(int)std::min<int64_t>(tiles, kBlocks * (int64_t)num_sms()), 32 * kWarps, smem, s>>>(p);
  prof_mark(id, s, false);
  return cudaGetLastError();
}

template <int kType>
cudaError_t launch_type(const Grouped& c, const StreamParams& p, int id, cudaStream_t s) {
  if (c.rows <= 8) return launch_stream<kType, 1, 1, 4, 3>(c, p, id, s);
  if (c.rows <= 16 * (int64_t)c.G) return launch_stream<kType, 2, 4, 1, 2>(c, p, id, s);
  return launch_stream<kType, 2, 8, 1, 1>(c, p, id, s);
}

StreamParams stream_params(const Grouped& c, const int32_t* begin, const int32_t* end, const void* x, const void* W,
                           uint16_t* y, int size, Hdr* hdr) {
  StreamParams p{};
  p.begin = begin;
  p.end = end;
  p.x = static_cast<const uint8_t*>(x);
  p.W = static_cast<const uint8_t*>(W);
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
  const StreamParams p = stream_params(c, begin, end, x, W, y, 2, hdr);
  return c.fp16 ? launch_type<kFp16>(c, p, kKGroupedMm, s) : launch_type<kBf16>(c, p, kKGroupedMm, s);
}

cudaError_t launch_stream_i8(const Grouped& c, const int32_t* begin, const int32_t* end, const int8_t* q,
                             const float* qs, const int8_t* Wq, const float* Ws, uint16_t* y, Hdr* hdr,
                             cudaStream_t s) {
  StreamParams p = stream_params(c, begin, end, q, Wq, y, 1, hdr);
  p.xs = qs;
  p.ws = Ws;
  return launch_type<kCodes>(c, p, kKGroupedI8, s);
}

}  // namespace moe
