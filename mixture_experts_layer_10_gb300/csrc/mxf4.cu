// Rows to microscaled 4-bit floating point: for every 32 consecutive values one power of two X and 32 e2m1 codes
// (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), X = 2^(floor(log2(largest)) - 2), code = v / X to the nearest,
// ties to the even code, at most 6 in magnitude.
//
// X is the largest value's exponent field less two, and v / X a product with a power of two, exact but where it is
// below 2^-126 and rounds to 0 anyway; so nothing here rounds but the conversion.  Four lanes share a block, eight
// values each; one pass over the rows, bound by HBM.
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;           // of eight values, a thread

struct MxParams {
  const void* src;
  uint8_t *codes, *scales;
  int64_t vecs;                    // of all rows
  int nvec, blocks, lds;           // of a row: vectors, scales, bytes from one row's scales to the next's
};

template <int kType> struct Raw { uint4 v; };
template <> struct Raw<MOE_FP32> { uint4 v[2]; };

__device__ __forceinline__ void unpack(const Raw<MOE_BF16>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void unpack(const Raw<MOE_FP16>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void unpack(const Raw<MOE_FP32>& r, float (&f)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}

// Eight values to eight codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t encode8(const float (&q)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}

template <int kType>
__global__ void __launch_bounds__(kThreads) quantize_rows_mxf4_kernel(const MxParams p) {
  after_previous_kernel();
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kVecs);
  const int64_t row0 = base / p.nvec;
  const int at0 = (int)(base - row0 * p.nvec);
  const Raw<kType>* src = static_cast<const Raw<kType>*>(p.src) + base;
  const int left = (int)min((int64_t)(kThreads * kVecs), p.vecs - base);   // a multiple of 4: blocks are whole
  Raw<kType> raw[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = threadIdx.x + i * kThreads;
    raw[i] = Raw<kType>{};
    if (v < left) raw[i] = src[v];
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = threadIdx.x + i * kThreads;
    float f[8];
    unpack(raw[i], f);
    uint32_t top = 0;   // of the magnitudes' bits: a NaN's are above infinity's
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int field = (int)(top >> 23);
    const int code = field == 255 ? 255 : max(field - 2, 0);
    const float inv = field == 255 ? 0.f : __uint_as_float((uint32_t)(254 - code) << 23);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = field == 255 ? 0.f : f[j] * inv;
    if (v >= left) continue;
    reinterpret_cast<uint32_t*>(p.codes)[base + v] = encode8(q);
    if ((v & 3) == 0) {
      const int in = at0 + v, dr = in / p.nvec, block = (in - dr * p.nvec) / 4;
      uint8_t* to = p.scales + (row0 + dr) * p.lds + block;
      *to = (uint8_t)code;
      if (block == p.blocks - 1)
        for (int b = p.blocks; b < p.lds; ++b) *++to = 0;
    }
  }
}

}  // namespace

cudaError_t launch_quantize_rows_mxf4(const void* src, int dtype, int64_t rows, int cols, uint8_t* codes,
                                      uint8_t* scales, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  MxParams p{src, codes, scales, rows * (cols / 8), cols / 8, cols / 32, mx_scale_stride(cols)};
  const int64_t per = kThreads * kVecs, blocks = (p.vecs + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  prof_mark(kKQuantMxf4, s, true);
  cudaError_t e;
  if (dtype == MOE_BF16) e = launch_after(quantize_rows_mxf4_kernel<MOE_BF16>, blocks, kThreads, 0, 1, s, p);
  else if (dtype == MOE_FP16) e = launch_after(quantize_rows_mxf4_kernel<MOE_FP16>, blocks, kThreads, 0, 1, s, p);
  else e = launch_after(quantize_rows_mxf4_kernel<MOE_FP32>, blocks, kThreads, 0, 1, s, p);
  prof_mark(kKQuantMxf4, s, false);
  return e;
}

}  // namespace moe
