// Grouped products: rows of every group times the group's own weight, and the gradients.
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

namespace {

// The groups and the exclusive sum of their row tiles.
struct GroupTab {
  int begin[kMaxGroups];
  int end[kMaxGroups];
  int first[kMaxGroups + 1];   // first tile of every group
  int part[32];
};

// Whole block: read the groups, check them, and number the row tiles of `tile` rows.  Returns the
// number of row tiles, or -1 (recorded in the error word by block 0) when the groups are out of range
// or out of order; every block reads the same values and answers the same.
__device__ int load_groups(GroupTab& t, const int32_t* begin, const int32_t* end, int G, int64_t rows, int tile, Hdr* hdr) {
  const int n = blockDim.x, per = (G + n - 1) / n;
  const int g0 = min(G, (int)threadIdx.x * per), g1 = min(G, g0 + per);
  bool bad = false;
  int sum = 0;
  for (int g = g0; g < g1; ++g) {
    const int b = begin[g], e = end[g];
    const int prev = g == 0 ? 0 : end[g - 1];
    bad |= b < prev || e < b || (int64_t)e > rows;
    t.begin[g] = b;
    t.end[g] = e;
    sum += bad ? 0 : (e - b) / tile + ((e - b) % tile != 0);
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(hdr, MOE_ERR_BAD_INDEX, kSiteGroups);
    return -1;
  }
  // exclusive sum over the threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) t.part[warp] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < warp; ++w) at += t.part[w];
  for (int g = g0; g < g1; ++g) {
    t.first[g] = at;
    const int len = t.end[g] - t.begin[g];
    at += len / tile + (len % tile != 0);
  }
  if (threadIdx.x == 0) {
    int total = 0;
    for (int w = 0; w < n / 32; ++w) total += t.part[w];
    t.first[G] = total;
  }
  __syncthreads();
  return t.first[G];
}

__device__ __forceinline__ float load16(const uint16_t* p, bool fp16) {
  const uint16_t u = *p;
  return fp16 ? __half2float(__ushort_as_half(u)) : __uint_as_float((uint32_t)u << 16);
}

__device__ __forceinline__ uint16_t store16(float v, bool fp16) {
  return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

struct Simple {
  const int32_t *begin, *end;
  const void *a, *b;       // rows operand (or dy), weight (or x)
  void* out;
  const float *as, *bs;    // scales (8-bit integers)
  int64_t rows, ldi, ldo;
  int K, N, G;
  bool fp16, dw_fp32, acc;
  Hdr* hdr;
};

enum { kMm, kDx, kDw, kI8 };

// 64 x 64 tiles of fp32 sums in registers (int32 for 8-bit integers), operands through shared memory.
template <int kOp>
__global__ void __launch_bounds__(256) simple_kernel(const Simple p) {
  __shared__ GroupTab tab;
  __shared__ float sa[16][65], sb[16][65];
  const int tiles = load_groups(tab, p.begin, p.end, p.G, p.rows, 64, p.hdr);
  if (tiles < 0) return;
  const int width = kOp == kDx || kOp == kDw ? p.K : p.N;   // columns of the output
  const int nt = (width + 63) / 64;
  const int mt = kOp == kDw ? p.G * ((p.N + 63) / 64) : tiles;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t t = blockIdx.x; t < (int64_t)mt * nt; t += gridDim.x) {
    const int m = (int)(t / nt), n0 = (int)(t % nt) * 64;
    int g = 0, m0;
    if (kOp == kDw) {
      g = m / ((p.N + 63) / 64);
      m0 = m % ((p.N + 63) / 64) * 64;
    } else {
      while (tab.first[g + 1] <= m) ++g;
      m0 = tab.begin[g] + (m - tab.first[g]) * 64;
    }
    const int mend = kOp == kDw ? p.N : tab.end[g];
    const int k0 = kOp == kDw ? tab.begin[g] : 0, k1 = kOp == kDw ? tab.end[g] : (kOp == kDx ? p.N : p.K);
    float acc[4][4] = {};
    int iacc[4][4] = {};
    for (int k = k0; k < k1; k += 16) {
      for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        const int kk = kOp == kDw ? i / 64 : i % 16, r = kOp == kDw ? i % 64 : i / 16;
        float va = 0.f, vb = 0.f;
        if (k + kk < k1 && m0 + r < mend) {
          if (kOp == kMm) va = load16((const uint16_t*)p.a + (m0 + r) * p.ldi + k + kk, p.fp16);
          if (kOp == kI8) va = (float)((const int8_t*)p.a)[(m0 + r) * p.ldi + k + kk];
          if (kOp == kDx) va = load16((const uint16_t*)p.a + (m0 + r) * p.ldo + k + kk, p.fp16);
          if (kOp == kDw) va = load16((const uint16_t*)p.a + (int64_t)(k + kk) * p.ldo + m0 + r, p.fp16);
        }
        if (k + kk < k1 && n0 + r < width) {
          const int64_t wbase = (int64_t)g * p.N * p.K;
          if (kOp == kMm) vb = load16((const uint16_t*)p.b + wbase + (int64_t)(n0 + r) * p.K + k + kk, p.fp16);
          if (kOp == kI8) vb = (float)((const int8_t*)p.b)[wbase + (int64_t)(n0 + r) * p.K + k + kk];
          if (kOp == kDx) vb = load16((const uint16_t*)p.b + wbase + (int64_t)(k + kk) * p.K + n0 + r, p.fp16);
          if (kOp == kDw) vb = load16((const uint16_t*)p.b + (int64_t)(k + kk) * p.ldi + n0 + r, p.fp16);
        }
        sa[kk][r] = va;
        sb[kk][r] = vb;
      }
      __syncthreads();
      for (int kk = 0; kk < 16; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kOp == kI8) iacc[i][j] += (int)sa[kk][ty + 16 * i] * (int)sb[kk][tx + 16 * j];
            else acc[i][j] = fmaf(sa[kk][ty + 16 * i], sb[kk][tx + 16 * j], acc[i][j]);
          }
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int r = m0 + ty + 16 * i, c = n0 + tx + 16 * j;
        if (r >= mend || c >= width) continue;
        float v = acc[i][j];
        if (kOp == kI8) v = (float)iacc[i][j] * p.bs[(int64_t)g * p.N + c] * p.as[r];
        if (kOp == kDw) {
          const int64_t o = ((int64_t)g * p.N + r) * p.K + c;
          if (p.dw_fp32) ((float*)p.out)[o] = v + (p.acc ? ((float*)p.out)[o] : 0.f);
          else ((uint16_t*)p.out)[o] = store16(v, p.fp16);
        } else {
          ((uint16_t*)p.out)[r * (kOp == kDx ? p.ldi : p.ldo) + c] = store16(v, p.fp16);
        }
      }
  }
}

__global__ void segments_kernel(const Tables* tabs, int G, int32_t* begin, int32_t* end) {
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    begin[g] = tabs->poff[g];
    end[g] = tabs->poff[g] + tabs->kept[g];
  }
}

template <int kOp>
cudaError_t launch_simple(const Grouped& c, const int32_t* begin, const int32_t* end, const void* a, const void* b,
                          void* out, const float* as, const float* bs, Hdr* hdr, int id, cudaStream_t s) {
  const Simple p{begin, end, a, b, out, as, bs, c.rows, c.ldi, c.ldo, c.K, c.N, c.G, c.fp16, c.dw_fp32, c.acc, hdr};
  prof_mark(id, s, true);
  simple_kernel<kOp><<<num_sms() * 4, 256, 0, s>>>(p);
  prof_mark(id, s, false);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_mm(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* x,
                              const uint16_t* W, uint16_t* y, Hdr* hdr, cudaStream_t s) {
  return launch_simple<kMm>(c, begin, end, x, W, y, nullptr, nullptr, hdr, kKGroupedMm, s);
}

cudaError_t launch_grouped_dx(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* dy,
                              const uint16_t* W, uint16_t* dx, Hdr* hdr, cudaStream_t s) {
  return launch_simple<kDx>(c, begin, end, dy, W, dx, nullptr, nullptr, hdr, kKGroupedDx, s);
}

cudaError_t launch_grouped_dw(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* dy,
                              const uint16_t* x, void* dW, Hdr* hdr, cudaStream_t s) {
  return launch_simple<kDw>(c, begin, end, dy, x, dW, nullptr, nullptr, hdr, kKGroupedDw, s);
}

cudaError_t launch_grouped_i8(const Grouped& c, const int32_t* begin, const int32_t* end, const int8_t* q,
                              const float* qs, const int8_t* Wq, const float* Ws, uint16_t* y, Hdr* hdr,
                              cudaStream_t s) {
  return launch_simple<kI8>(c, begin, end, q, Wq, y, qs, Ws, hdr, kKGroupedI8, s);
}

cudaError_t launch_segments(const Tables* tabs, int G, int32_t* begin, int32_t* end, cudaStream_t s) {
  segments_kernel<<<1, 256, 0, s>>>(tabs, G, begin, end);
  return cudaGetLastError();
}

}  // namespace moe
