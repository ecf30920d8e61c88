// What the kernels of the grouped products share: the table of the groups and the 16-bit roundings.
#pragma once

#include <atomic>

#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace moe {

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
__device__ __forceinline__ int load_groups(GroupTab& t, const int32_t* begin, const int32_t* end, int G, int64_t rows, int tile,
                           Hdr* hdr) {
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

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  if (!fp16) return pack_bf16(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight codes (two words) to eight fp16 values: a code with its sign bit flipped is u = code + 128, the
// fp16 number with that byte under 0x64 is 1024 + u, and 1152 less is the code, exactly.
__device__ __forceinline__ uint4 widen(uint32_t w0, uint32_t w1) {
  const uint32_t w[2] = {w0, w1};
  uint32_t o[4];
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    o[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A kernel's dynamic shared memory, set once a device rather than at every launch.
struct SmemOnce {
  std::atomic<uint64_t> done{0};
  cudaError_t set(const void* kernel, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// A positive number of a device, found by the first call there (of several threads at once, by each of them:
// the answer is the same).
struct IntOnce {
  std::atomic<int> found[64] = {};
  template <class F>
  cudaError_t get(int* value, F find) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev < 64;
    *value = keep ? found[dev].load(std::memory_order_acquire) : 0;
    if (*value == 0) {
      *value = find();
      if (keep) found[dev].store(*value, std::memory_order_release);
    }
    return cudaSuccess;
  }
};

// The kernels of the grouped products are launched so that a kernel's blocks may start, as those of the
// kernel before it in the stream end, before that one has ended altogether (programmatic dependent launch).
// Each first waits for the kernels before it to have ended and their writes to be visible, so nothing
// but its launch and its barriers' setup overlaps them.  (Blocks that start earlier still, as soon as all
// of the kernel before them are running, take room and slow it: 63.6 -> 66.8 us at 64 tokens, 64 experts.)
__device__ __forceinline__ void after_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), int64_t blocks, int threads, size_t smem, int cluster,
                         cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Releases, at cluster scope, what this thread knows of writes to its CTA's shared memory, to whoever sees a
// relaxed arrival that follows.  (A releasing arrival waits for every other memory operation too: 9% of the
// time of the 8-bit product on CTA pairs.)
__device__ __forceinline__ void fence_release_smem() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}

// Bounded wait with naps of kNap ns between polls.  kCluster acquires at cluster scope: for barriers on
// which the peer CTA's threads arrive after writing shared memory.
template <bool kCluster>
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  if (!kCluster) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

template <int kNap, bool kCluster = false>
__device__ __forceinline__ bool wait_nap(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort) {
  if (try_wait<kCluster>(bar, parity)) return true;
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
      if (kNap > 0) __nanosleep(kNap);
      if (try_wait<kCluster>(bar, parity)) return true;
    }
    const uint64_t t = global_ns();
    if (t0 == 0) t0 = t;
    if (*abort || t - t0 > limit_ns) return false;
  }
}

}  // namespace moe
