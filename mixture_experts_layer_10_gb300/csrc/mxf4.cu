// Rows to microscaled 4-bit floating point: for every 32 consecutive values one power of two X and 32 e2m1 codes
// (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), X = 2^(floor(log2(largest)) - 2), code = v / X to the nearest,
// ties to the even code, at most 6 in magnitude.
//
// X is the largest value's exponent field less two, and v / X a product with a power of two, exact but where it is
// below 2^-126 and rounds to 0 anyway; so nothing here rounds but the conversion.  Four lanes share a block, eight
// values each; one pass over the rows, 32 values a thread, all its loads before the first of them is used.
//
// Measured: 16381 rows of 2880, fp16, 18.8 us, 6.4 TB/s of reads and writes (0.95 of a copy's); 24576 rows of 2048 20.2;
// one token's 8 rows 1.7.  (With maxima of single values and a division a vector it was bound by issue: 25.5.)
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
  uint32_t recip;                  // 2^32 / nvec, rounded up: in / nvec is in * recip / 2^32 as long as in * nvec < 2^32
};

template <int kType> struct Raw { uint4 v; };
template <> struct Raw<MOE_FP32> { uint4 v[2]; };

// The largest magnitude's bits as of a float; a NaN's are above infinity's.
__device__ __forceinline__ uint32_t top_of(const Raw<MOE_FP32>& r) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, w[i] & 0x7fffffffu);
  return top;
}
__device__ __forceinline__ uint32_t top16(const uint4& v) {   // (two 16-bit maxima at a time: the order of magnitudes' bits)
  constexpr uint32_t k = 0x7fff7fffu;
  const uint32_t t = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
  return max(t & 0xffffu, t >> 16);
}
__device__ __forceinline__ uint32_t top_of(const Raw<MOE_BF16>& r) { return top16(r.v) << 16; }
__device__ __forceinline__ uint32_t top_of(const Raw<MOE_FP16>& r) {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top16(r.v))));
}

// The values times a power of two.
__device__ __forceinline__ void scaled(const Raw<MOE_BF16>& r, float by, float (&f)[8]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]) * by;
    f[2 * i + 1] = bf16_hi(w[i]) * by;
  }
}
__device__ __forceinline__ void scaled(const Raw<MOE_FP16>& r, float by, float (&f)[8]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = v.x * by;
    f[2 * i + 1] = v.y * by;
  }
}
__device__ __forceinline__ void scaled(const Raw<MOE_FP32>& r, float by, float (&f)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]) * by;
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
    uint32_t top = top_of(raw[i]);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t field = top >> 23, code = field == 255 ? 255u : max(field, 2u) - 2u;
    float f[8];
    scaled(raw[i], __uint_as_float((254u - min(code, 253u)) << 23), f);
    const uint32_t w = encode8(f);
    if (v >= left) continue;
    reinterpret_cast<uint32_t*>(p.codes)[base + v] = code == 255 ? 0u : w;
    if ((v & 3) == 0) {
      const uint32_t in = at0 + v, dr = __umulhi(in, p.recip), block = (in - dr * p.nvec) / 4;
      uint8_t* to = p.scales + (row0 + dr) * p.lds + block;
      *to = (uint8_t)code;
      if ((int)block == p.blocks - 1)
        for (int b = p.blocks; b < p.lds; ++b) *++to = 0;
    }
  }
}

}  // namespace

cudaError_t launch_quantize_rows_mxf4(const void* src, int dtype, int64_t rows, int cols, uint8_t* codes,
                                      uint8_t* scales, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  MxParams p{src, codes, scales, rows * (cols / 8), cols / 8, cols / 32, mx_scale_stride(cols), 0};
  p.recip = (uint32_t)((((uint64_t)1 << 32) + p.nvec - 1) / p.nvec);   // (nvec: 4 .. 8192)
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
