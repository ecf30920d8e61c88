// Grouped products: rows of every group times the group's own weight (y = x W[g]^T, dx = dy W[g]), the
// gradient of the weight (dW[g] = dy^T x over the group's rows), and the first of them with 8-bit
// integers.  Groups are given on the device as first and past-the-end rows, of any length and start;
// nothing is padded or copied.
//
// All of them run on the 5th-generation tensor cores in one persistent kernel per product, on CTA pairs
// (a cluster of two, tcgen05.mma.cta_group::2) with a 256 x 256 tile a pair, fp32 accumulators in TMEM
// (two, so that the epilogue of a tile runs under the next one's products):
//
//   warp 0      TMA producer: operand tiles into a ring of shared-memory stages (64 deep in K)
//   warp 1      MMA issuer (the even CTA's one thread)
//   warps 2-5   epilogue: tcgen05.ld of the accumulator, scales, rounding, stores
//   warps 6..   8-bit integers: eight warps that widen the codes to fp16 (below);
//               weight gradient: one warp that clears the rows past the end of a group
//
// Rows times a weight.  The weight's 256 features are the M side of the tile and up to 256 rows of one
// group its N side, so a group's ragged end costs a narrower product (N in steps of 32) rather than
// padded rows: tensor time follows the rows there are.  Rows past the end of the group are loaded (they
// belong to the next group, or lie outside the tensor and read as zero) and fill accumulator columns of
// their own, which nothing stores.  The accumulator holds a feature per TMEM lane and a row per column,
// so a warp stores 32 features of a row at a time.
//
// Weight gradient.  M = 256 columns of dy, N = 256 columns of x, K = the group's rows, both operands
// MN-major.  Here rows past the end of the group would enter the sums, so in a group's last K block
// both CTAs clear those rows of both operands in shared memory before the product.  With dW in fp32 the
// rows go in runs of kRun (an accumulator loses up to one unit of its last place at each step of 16
// rows, which a long contraction would let grow past fp32's own rounding); the runs add up in dW, in
// row order, by reducing bulk stores of the same warp.
//
// 8-bit integers.  sm_103a has no integer product at tensor rates, but every code is exact in fp16 and a
// product of two in fp32, so fp16 tensor products of widened codes are the integer products, and their
// fp32 sums are exact up to 2^24.  Codes travel as bytes; eight warps widen them between the ring that
// TMA fills and the ring that the tensor cores read.
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

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
__device__ int load_groups(GroupTab& t, const int32_t* begin, const int32_t* end, int G, int64_t rows, int tile,
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

enum Op { kMm, kDx, kDw, kI8 };

constexpr int kBM = 128;                     // rows of the M side a CTA holds
constexpr int kTile = 256;                   // pair tile, both sides
constexpr int kBK = 64;                      // K block of a stage (128 bytes a row)
constexpr uint32_t kHalf = kBM * kBK * 2;    // 16 KB: one operand of a stage
constexpr uint32_t kBox = 64 * kBK * 2;      // 8 KB: a 64 x 64 box (MN-major)
constexpr int kBoxes = 3;                    // row-operand boxes: 128, 64 and 32 rows
constexpr int kChunkM = 16;                  // row tiles per L2 reuse chunk of a group
constexpr int kRun = 2048;                   // rows of an fp32 weight-gradient run
constexpr int kTmemCols = 512;
constexpr uint32_t kEpiBox = 32 * 64;        // a staging box: 32 rows of 64 bytes

template <int kOp>
struct Shape {
  static constexpr int kStages = kOp == kI8 ? 4 : 6;       // 16-bit K blocks
  static constexpr int kRaw = kOp == kI8 ? 2 : 0;          // 8-bit blocks, 128 codes deep
  static constexpr int kWiden = 8;                         // warps that widen codes
  static constexpr int kExtra = kOp == kI8 ? kWiden : (kOp == kDw ? 1 : 0);
  static constexpr int kThreads = 32 * (6 + kExtra);
  static constexpr uint32_t kEpi = kOp == kDw ? 4 * 2 * kEpiBox : 0;
  static constexpr size_t kSmem = 1024 + (size_t)(kStages + kRaw) * 2 * kHalf + kEpi + 512 + sizeof(GroupTab);
  static_assert(kSmem <= 232448, "shared memory per block");
};

struct Params {
  CUtensorMap a;              // M side: the weight, or dy (weight gradient)
  CUtensorMap b[kBoxes];      // N side: the rows in boxes of 128, 64, 32; or x in b[0] (weight gradient)
  CUtensorMap out;            // weight gradient: dW in boxes
  const int32_t *begin, *end;
  void* y;
  const float *qs, *ws;       // scales of the rows and of the output channels (8-bit integers)
  int64_t rows, ldy;
  int depth;                  // contraction length (rows times a weight)
  int width;                  // features of the output row; weight gradient: columns of dW (n_in)
  int M;                      // weight gradient: rows of dW (n_out)
  int G, nf, mf;              // tiles across width; weight gradient: tiles across M
  bool fp16, wide_a, wide_b;  // wide: one copy fetches two 64-column boxes (columns a multiple of 64)
  bool dw_fp32, acc;
  uint32_t idesc;             // N and M as of a full tile
  Hdr* hdr;
};

struct Job {
  int g, row, n, f0;   // rows times a weight: first row, rows, first feature
  int m0, kits, run;   // weight gradient: first dW row, K blocks of the run, its number
  int tail;            // rows of the run's last K block that belong to the group (0: all of them)
};

// Rows times a weight: tile t -> group, row tile, feature tile.  Groups in order; within a group,
// chunks of up to 16 row tiles x all feature tiles with the row tile fastest, so that the pairs at work
// share a panel of each operand in L2.
__device__ __forceinline__ Job row_job(const Params& p, const GroupTab& s, int t) {
  const int m = t / p.nf;
  int lo = 0, hi = p.G - 1;   // the last group whose first tile <= m
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.first[mid] <= m) lo = mid; else hi = mid - 1;
  }
  const int first = s.first[lo], mt = s.first[lo + 1] - first;
  const int local = t - first * p.nf;
  const int c = local / (kChunkM * p.nf);
  const int cm = min(kChunkM, mt - c * kChunkM);
  const int r = local - c * kChunkM * p.nf;
  Job j{};
  j.g = lo;
  j.row = s.begin[lo] + (c * kChunkM + r % cm) * kTile;
  j.n = min(kTile, s.end[lo] - j.row);
  j.f0 = r / cm * kTile;
  return j;
}

// Weight gradient: tile t -> group, tile of dW; a tile is one job a run of rows (job_runs).
__device__ __forceinline__ int job_runs(const Params& p, int n) {
  return p.dw_fp32 && n > kRun ? (n + kRun - 1) / kRun : 1;
}

__device__ __forceinline__ Job dw_job(const Params& p, const GroupTab& s, int t, int run) {
  const int per = p.mf * p.nf;
  Job j{};
  j.g = t / per;
  const int r = t - j.g * per;
  j.m0 = r / p.nf * kTile;
  j.f0 = r % p.nf * kTile;
  j.run = run;
  const int n = s.end[j.g] - s.begin[j.g], from = run * kRun;
  j.row = s.begin[j.g] + from;
  j.n = p.dw_fp32 ? min(kRun, n - from) : n;
  j.kits = (j.n + kBK - 1) / kBK;
  j.tail = j.n % kBK;
  return j;
}

// The rows' box for a half of n rows: 0 (128 rows), 1 (64) or 2 (32).
__device__ __forceinline__ int box_of(int half) { return half > 64 ? 0 : (half > 32 ? 1 : 2); }

// 16 codes (four words) to 16 fp16 values: a code with its sign bit flipped is u = code + 128, the fp16
// number with that byte under 0x64 is 1024 + u, and 1152 less is the code, exactly.
__device__ __forceinline__ void widen(const uint4& v, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    o[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// One pair's walk over its tiles, the same in every role of both CTAs: rows times a weight has one job a
// tile, the weight gradient one a run of rows.
template <int kOp>
struct Walk {
  const Params& p;
  const GroupTab& s;
  int t, step, ntiles, run = 0, runs = 0;
  __device__ Walk(const Params& p_, const GroupTab& s_, int first, int step_, int ntiles_)
      : p(p_), s(s_), t(first), step(step_), ntiles(ntiles_) {}
  __device__ bool next(Job& j) {
    if (kOp != kDw) {
      if (t >= ntiles) return false;
      j = row_job(p, s, t);
      j.kits = (p.depth + kBK - 1) / kBK;
      t += step;
      return true;
    }
    if (t >= ntiles) return false;
    if (run == 0) {
      const int g = t / (p.mf * p.nf);
      runs = job_runs(p, s.end[g] - s.begin[g]);
    }
    j = dw_job(p, s, t, run);
    if (++run == runs) {
      run = 0;
      t += step;
    }
    return true;
  }
};

// ---- epilogues -----------------------------------------------------------------------------------

// Rows times a weight: this warp's 32 features (lanes) of the tile's rows (columns).  Lanes exchange
// with their neighbour so that each holds two features of one row: an instruction stores 64 bytes of
// two rows.
template <int kOp>
__device__ __forceinline__ void store_rows(const Params& p, const Job& j, int rank, int q, int lane, uint32_t ta) {
  const int f = j.f0 + kBM * rank + 32 * q + lane;
  const bool odd = lane & 1;
  if (j.f0 + kBM * rank + 32 * q >= p.width) return;   // the whole warp lies past the last feature
  const bool live = f < p.width;                       // a multiple of 8: the same for both lanes of a pair
  const float ws = kOp == kI8 && live ? p.ws[(int64_t)j.g * p.width + f] : 1.f;
  uint16_t* out = static_cast<uint16_t*>(p.y) + (int64_t)(j.row + odd) * p.ldy + (f & ~1);
#pragma unroll 1
  for (int c = 0; c < j.n; c += 32) {
    uint32_t v[32];
    tmem_ld32(ta + c, v);
    float qs = 0.f;
    if (kOp == kI8) qs = c + lane < j.n ? p.qs[j.row + c + lane] : 0.f;
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float a = __uint_as_float(v[i]), b = __uint_as_float(v[i + 1]);
      if (kOp == kI8) {
        a = a * ws * __shfl_sync(0xffffffffu, qs, i);
        b = b * ws * __shfl_sync(0xffffffffu, qs, i + 1);
      }
      const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
      const uint32_t w = odd ? pack16(got, b, p.fp16) : pack16(a, got, p.fp16);
      if (live && c + i + odd < j.n) *reinterpret_cast<uint32_t*>(out + (int64_t)(c + i) * p.ldy) = w;
    }
  }
}

__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, const void* src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Weight gradient: this warp's 32 rows of dW (lanes), 256 columns, through two staging boxes of 32 rows
// x 64 bytes (the layout of the 64-byte swizzle: 16-byte chunk c of row r at c ^ ((r >> 1) & 3)) and
// bulk stores, which clip what lies past dW.  A run after the first adds to what this warp stored
// before, so it first waits for those stores to be performed.
__device__ __forceinline__ void store_dw(const Params& p, const Job& j, int rank, int q, int lane, uint32_t ta,
                                         uint8_t* boxes) {
  const int y = j.m0 + kBM * rank + 32 * q;
  if (y >= p.M) return;
  const bool add = p.acc || j.run > 0;
  if (lane == 0) {
    if (j.run > 0) bulk_wait_all();
    else bulk_wait_read<0>();
  }
  __syncwarp();
  int n = 0;
#pragma unroll 1
  for (int c = 0; c < kTile; c += 32) {
    if (j.f0 + c >= p.width) break;
    uint32_t v[32];
    tmem_ld32(ta + c, v);
    tmem_ld_wait();
    const int parts = p.dw_fp32 ? 2 : 1;   // 32 columns: two fp32 boxes or one 16-bit box
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == parts || j.f0 + c + 16 * h >= p.width) break;
      if (n >= 2) {   // the box of two stores ago has been read
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
      }
      uint8_t* box = boxes + (n & 1) * kEpiBox;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4 w;
        if (p.dw_fp32) {
          w = make_uint4(v[16 * h + 4 * k], v[16 * h + 4 * k + 1], v[16 * h + 4 * k + 2], v[16 * h + 4 * k + 3]);
        } else {
          uint32_t u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            u[i] = pack16(__uint_as_float(v[8 * k + 2 * i]), __uint_as_float(v[8 * k + 2 * i + 1]), p.fp16);
          w = make_uint4(u[0], u[1], u[2], u[3]);
        }
        *reinterpret_cast<uint4*>(box + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = w;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (add) tma_add_3d(&p.out, box, j.f0 + c + 16 * h, y, j.g);
        else tma_store_3d(&p.out, box, j.f0 + c + 16 * h, y, j.g);
        bulk_commit();
      }
      ++n;
    }
  }
}

// A group without rows has a zero gradient (nothing to add to a running one): this warp's 32 rows of
// the tile, a row at a time.
__device__ __forceinline__ void store_zero(const Params& p, const Job& j, int rank, int q, int lane) {
  if (p.acc) return;
  const int size = p.dw_fp32 ? 4 : 2, per = 16 / size;
  const int c1 = min(p.width, j.f0 + kTile);
  for (int i = 0; i < 32; ++i) {
    const int y = j.m0 + kBM * rank + 32 * q + i;
    if (y >= p.M) break;
    char* row = static_cast<char*>(p.y) + (((int64_t)j.g * p.M + y) * p.width) * size;
    for (int c = j.f0 + lane * per; c < c1; c += 32 * per)
      *reinterpret_cast<uint4*>(row + (int64_t)c * size) = make_uint4(0, 0, 0, 0);
  }
}

// Arrive once on the mbarrier at this shared-memory offset in both CTAs when every pair MMA this thread
// issued so far has completed.
__device__ __forceinline__ void umma_commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// True once the phase with parity `parity` has completed; acquires at cluster scope, for barriers on
// which the peer CTA's threads arrive after writing shared memory.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                                  volatile int* abort) {
  const uint64_t t0 = global_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (*abort || global_ns() - t0 > limit_ns) return false;
  }
}

// Barriers (the same offsets in both CTAs; who uses which copy):
//   full[s]     even CTA: the stage's operands of both CTAs are in place (TMA bytes; 8-bit integers: the
//               widening warps of both CTAs; a cleared K block: the clearing warps)
//   empty[s]    stage free: committed to the even CTA, whose producer forwards it to the odd one when it
//               refills the stage (8-bit integers: committed to both, the widening warps wait)
//   tfull[a]    each CTA: accumulator a is complete
//   tempty[a]   even CTA: both CTAs' epilogues have read it
//   raw[s]      own CTA: bytes of a raw stage (8-bit integers), or of a K block that needs clearing
//   rempty[s]   8-bit integers, own CTA: the widening warps have read raw stage s
//   peer[s]     weight gradient, even CTA: the odd CTA has cleared its share of stage s
// Every wait is bounded; whatever happens, both CTAs meet at the last cluster barrier before TMEM is
// freed, with their own copies landed.
template <int kOp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<kOp>::kThreads, 1)
    grouped_kernel(const __grid_constant__ Params p) {
  using S = Shape<kOp>;
  constexpr int kStages = S::kStages, kRaw = S::kRaw;
  constexpr uint32_t kStage = 2 * kHalf;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = smem;
  uint8_t* raws = stages + kStages * kStage;
  uint8_t* boxes = raws + kRaw * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + S::kEpi);
  uint64_t* empty = full + 6;
  uint64_t* raw = empty + 6;
  uint64_t* rempty = raw + 6;
  uint64_t* peer = rempty + 6;
  uint64_t* tfull = peer + 6;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  GroupTab& tab = *reinterpret_cast<GroupTab*>(boxes + S::kEpi + 512);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 6; ++s) {
      mbar_init(&full[s], kOp == kI8 ? S::kWiden : 1);
      mbar_init(&empty[s], 1);
      mbar_init(&raw[s], 1);
      mbar_init(&rempty[s], S::kWiden);
      mbar_init(&peer[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch(&p.a);
    for (int i = 0; i < (kOp == kDw ? 1 : kBoxes); ++i) tma_prefetch(&p.b[i]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  const int rtiles = load_groups(tab, p.begin, p.end, p.G, p.rows, kTile, p.hdr);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t limit = wait_limit_ns(p.hdr);
  const int ntiles = rtiles < 0 ? 0 : (kOp == kDw ? p.G * p.mf * p.nf : rtiles * p.nf);
  Walk<kOp> walk(p, tab, pair, npairs, ntiles);
  Job j;

  auto fail = [&](int site) {
    record_error(p.hdr, MOE_ERR_TIMEOUT, site);
    *abort_flag = 1;
  };

  if (warp == 0) {
    if (lane == 0) {
      int slot = 0, uses = 0;
      uint32_t phase = 0;
      bool ok = true;
      // test hook: the first pair skips one fill, so that the wait for it runs out
      const int skip = pair == 0 ? *((volatile const int32_t*)&p.hdr->stall_fill_p1) - 1 : -1;
      uint32_t raw_used = 0, raw_next = 0;   // weight gradient, a bit per stage: own barrier used, next phase
      if constexpr (kOp == kI8) {
        while (ok && !*abort_flag && walk.next(j)) {
          const int half = ((j.n + 31) / 32 * 32) / 2, bx = box_of(half);
          const uint32_t bytes = kHalf + (128u >> bx) * 128u;
          const int kits = (p.depth + 127) / 128;
          for (int kit = 0; kit < kits; ++kit) {
            if (!mbar_wait(&rempty[slot], phase ^ 1, limit, abort_flag)) {
              fail(kSiteGroupedProducer);
              ok = false;
              break;
            }
            if (uses != skip) {
              uint8_t* st = raws + (size_t)slot * kStage;
              mbar_arrive_expect_tx(&raw[slot], bytes);
              tma_load_3d(st, &p.a, &raw[slot], kit * 128, j.f0 + kBM * rank, j.g);
              tma_load_2d(st + kHalf, &p.b[bx], &raw[slot], kit * 128, j.row + half * rank);
            }
            ++uses;
            if (++slot == kRaw) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        drain_fills(raw, kRaw, slot, phase, uses, limit);
      } else {
        while (ok && !*abort_flag && walk.next(j)) {
          const int half = ((j.n + 31) / 32 * 32) / 2, bx = kOp == kDw ? 0 : box_of(half);
          const uint32_t bytes = kHalf + (kOp == kDw ? kHalf : (128u >> bx) * 128u);
          for (int kit = 0; kit < j.kits; ++kit) {
            if (!mbar_wait(&empty[slot], phase ^ 1, limit, abort_flag)) {
              fail(kSiteGroupedProducer);
              ok = false;
              break;
            }
            if (uses != skip) {
              uint8_t* st = stages + (size_t)slot * kStage;
              if constexpr (kOp == kDw) {
                // a K block that needs clearing lands on this CTA's own barrier, for its clearing warp
                const bool clear = j.tail != 0 && kit == j.kits - 1;
                uint32_t bar = cluster_addr(&full[slot], 0);
                if (clear) {
                  mbar_arrive_expect_tx(&raw[slot], bytes);
                  bar = cluster_addr(&raw[slot], (uint32_t)rank);
                  raw_used |= 1u << slot;
                  raw_next ^= 1u << slot;
                } else if (rank == 0) {
                  mbar_arrive_expect_tx(&full[slot], 2 * bytes);
                }
                const int row = j.row + kit * kBK, ca = j.m0 + kBM * rank, cb = j.f0 + kBM * rank;
                if (p.wide_a) {
                  tma_load_3d_pair(st, &p.a, bar, 0, row, ca / 64);
                } else {
                  tma_load_2d_pair(st, &p.a, bar, ca, row);
                  tma_load_2d_pair(st + kBox, &p.a, bar, ca + 64, row);
                }
                if (p.wide_b) {
                  tma_load_3d_pair(st + kHalf, &p.b[0], bar, 0, row, cb / 64);
                } else {
                  tma_load_2d_pair(st + kHalf, &p.b[0], bar, cb, row);
                  tma_load_2d_pair(st + kHalf + kBox, &p.b[0], bar, cb + 64, row);
                }
              } else {
                if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * bytes);
                const uint32_t bar = cluster_addr(&full[slot], 0);
                const int f = j.f0 + kBM * rank;
                if (kOp == kMm) {
                  tma_load_3d_pair(st, &p.a, bar, kit * kBK, f, j.g);
                } else if (p.wide_a) {
                  tma_load_4d_pair(st, &p.a, bar, 0, kit * kBK, f / 64, j.g);
                } else {
                  tma_load_3d_pair(st, &p.a, bar, f, kit * kBK, j.g);
                  tma_load_3d_pair(st + kBox, &p.a, bar, f + 64, kit * kBK, j.g);
                }
                tma_load_2d_pair(st + kHalf, &p.b[bx], bar, kit * kBK, j.row + half * rank);
              }
            }
            if (rank == 0 && uses >= kStages) mbar_arrive_cluster_relaxed(cluster_addr(&empty[slot], 1));
            ++uses;
            if (++slot == kStages) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        // every load of the pair lands before either CTA's shared memory is released: the even CTA's
        // full barriers complete after both CTAs' bytes, and the odd CTA waits at the cluster barrier
        if (rank == 0) drain_fills(full, kStages, slot, phase, uses, limit);
        for (int s = 0; s < kStages; ++s)
          if ((raw_used >> s) & 1) mbar_wait_drain(&raw[s], ((raw_next >> s) & 1) ^ 1u, limit);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int slot = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, more = walk.next(j);
      while (ok && more && !*abort_flag) {
        const int kits = j.kits;
        const int n = kOp == kDw ? kTile : (j.n + 31) / 32 * 32;
        const uint32_t idesc = (p.idesc & ~(0x3Fu << 17)) | ((uint32_t)(n >> 3) << 17);
        more = walk.next(j);   // the next job, worked out while this one's products run
        if (kits == 0) continue;
        const uint32_t dt = tmem_base + (uint32_t)(acc * kTile);
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1, limit, abort_flag)) {
          fail(kSiteGroupedMma);
          break;
        }
        tc_fence_after();
        for (int kit = 0; kit < kits; ++kit) {
          const bool there = kOp == kI8 || kOp == kDw ? mbar_wait_cluster(&full[slot], phase, limit, abort_flag)
                                                      : mbar_wait(&full[slot], phase, limit, abort_flag);
          if (!there) {
            fail(kSiteGroupedMma);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(stages + (size_t)slot * kStage);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t da = kOp == kMm || kOp == kI8 ? sdesc_kmajor(sa + kk * 32) : sdesc_mnmajor(sa + kk * 2048, kBox);
            const uint64_t db = kOp == kDw ? sdesc_mnmajor(sa + kHalf + kk * 2048, kBox) : sdesc_kmajor(sa + kHalf + kk * 32);
            umma_bf16_pair(dt, da, db, idesc, (kit | kk) != 0);
          }
          if (kOp == kI8) umma_commit_both(&empty[slot]);
          else umma_commit_pair(smem_u32(&empty[slot]));
          if (++slot == kStages) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        umma_commit_both(&tfull[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      // every pair MMA issued has completed, and every arrival on either CTA's barriers, before the
      // TMEM is freed and the CTAs exit (bounded)
      umma_commit_both(drain);
    }
    if (lane == 0) mbar_wait_drain(drain, 0, limit);
  } else if (warp < 6) {
    const int q = warp & 3;   // TMEM lane quarter this warp may access
    int acc = 0;
    uint32_t acc_phase = 0;
    while (walk.next(j)) {
      if (j.kits == 0) {
        store_zero(p, j, rank, q, lane);
        continue;
      }
      if (!mbar_wait_idle(&tfull[acc], acc_phase, limit, abort_flag)) {
        fail(kSiteGroupedEpilogue);
        break;
      }
      tc_fence_after();
      const uint32_t ta = tmem_base + (uint32_t)(acc * kTile) + ((uint32_t)(q * 32) << 16);
      if constexpr (kOp == kDw) store_dw(p, j, rank, q, lane, ta, boxes + (warp - 2) * 2 * kEpiBox);
      else store_rows<kOp>(p, j, rank, q, lane, ta);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[acc], 0));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (kOp == kDw && lane == 0) bulk_wait_all();   // this warp's output stores have landed
  } else if constexpr (kOp == kDw) {
    // the rows past the end of the group in its last K block, in both operands' boxes of this CTA
    int slot = 0;
    uint32_t raw_phase = 0, peer_phase = 0;   // a bit per stage: only cleared blocks use these barriers
    bool ok = true;
    while (ok && walk.next(j)) {
      if (j.tail != 0) {
        const int s = (slot + j.kits - 1) % kStages;
        if (!mbar_wait(&raw[s], (raw_phase >> s) & 1, limit, abort_flag)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) fail(kSiteGroupedStage);
          break;
        }
        raw_phase ^= 1u << s;
        uint8_t* st = stages + (size_t)s * kStage;
#pragma unroll 1
        for (int box = 0; box < 4; ++box)
          for (int o = j.tail * 128 + lane * 16; o < (int)kBox; o += 32 * 16)
            *reinterpret_cast<uint4*>(st + box * kBox + o) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (rank == 1) {
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&peer[s], 0));
        } else {
          if (lane == 0) {
            ok = mbar_wait_cluster(&peer[s], (peer_phase >> s) & 1, limit, abort_flag);
            if (ok) mbar_arrive_cluster(cluster_addr(&full[s], 0));
            else fail(kSiteGroupedStage);
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
          peer_phase ^= 1u << s;
        }
      }
      slot = (slot + j.kits) % kStages;
    }
  } else if constexpr (kOp == kI8) {
    // Widen: an octet of rows at a time, a lane a row and 16 codes -- in the 128-byte swizzle the eight
    // lanes of a phase touch distinct banks on both sides.  A raw stage holds two K blocks; four warps
    // take each, so that the latency of one block's widening runs under the other's.
    constexpr int kTeam = S::kWiden / 2;
    const int team = (warp - 6) / kTeam, w = (warp - 6) % kTeam, r = lane & 7, cq = lane >> 3;
    int block = 0, rblock = 0;   // K blocks and raw stages before this job
    bool ok = true;
    while (ok && walk.next(j)) {
      const int half = ((j.n + 31) / 32 * 32) / 2;
      const int octets = 16 + half / 8;   // of the weight's 128 rows, then of the token rows
      const int kits = j.kits, rkits = (kits + 1) / 2;
      for (int rk = 0; rk < rkits; ++rk) {
        const int rs = (rblock + rk) % kRaw, kit = 2 * rk + team;
        const int at = block + kit, slot = at % kStages;
        // (a team without a block in this raw stage waits for it too, so that its release of the stage
        // counts towards this fill)
        ok = mbar_wait(&raw[rs], (uint32_t)((rblock + rk) / kRaw) & 1u, limit, abort_flag) &&
             (kit >= kits || mbar_wait(&empty[slot], ((uint32_t)(at / kStages) & 1u) ^ 1u, limit, abort_flag));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) fail(kSiteGroupedStage);
          break;
        }
        if (kit < kits) {
          const uint8_t* src = raws + (size_t)rs * kStage + r * 128 + (((team * 4 + cq) ^ r) << 4);
          uint8_t* dst = stages + (size_t)slot * kStage + r * 128;
#pragma unroll 1
          for (int o = w; o < octets; o += 4 * kTeam) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (o + i * kTeam < octets) v[i] = *reinterpret_cast<const uint4*>(src + (o + i * kTeam) * 1024);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (o + i * kTeam >= octets) break;
              uint4 lo, hi;
              widen(v[i], lo, hi);
              uint8_t* d = dst + (o + i * kTeam) * 1024;
              *reinterpret_cast<uint4*>(d + (((2 * cq) ^ r) << 4)) = lo;
              *reinterpret_cast<uint4*>(d + (((2 * cq + 1) ^ r) << 4)) = hi;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&full[slot], 0));
        }
        if (lane == 0) mbar_arrive(&rempty[rs]);
      }
      block += kits;
      rblock += rkits;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

__global__ void segments_kernel(const Tables* tabs, int G, int32_t* begin, int32_t* end) {
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    begin[g] = tabs->poff[g];
    end[g] = tabs->poff[g] + tabs->kept[g];
  }
}

// ---- host side -----------------------------------------------------------------------------------

// A tensor map of up to four dimensions; strides in bytes of dimensions 1...
bool encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn && fn(m, type, rank, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr CUtensorMapDataType k16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, k8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
constexpr CUtensorMapSwizzle kSw128 = CU_TENSOR_MAP_SWIZZLE_128B, kSw64 = CU_TENSOR_MAP_SWIZZLE_64B;

// Rows [rows, width] as K-major boxes of 128 bytes x 128, 64 and 32 rows.
bool map_rows(CUtensorMap* m, const void* base, bool codes, uint64_t rows, uint64_t width, uint64_t ld) {
  const cuuint64_t dims[2] = {width, rows}, strides[1] = {ld * (codes ? 1 : 2)};
  for (int i = 0; i < kBoxes; ++i) {
    const cuuint32_t box[2] = {codes ? 128u : 64u, 128u >> i};
    if (!encode(&m[i], codes ? k8 : k16, 2, base, dims, strides, box, kSw128)) return false;
  }
  return true;
}

// Weights [G, N, K], K-major: boxes of 128 bytes x 128 rows.
bool map_weight(CUtensorMap* m, const void* base, bool codes, uint64_t G, uint64_t N, uint64_t K) {
  const uint64_t size = codes ? 1 : 2;
  const cuuint64_t dims[3] = {K, N, G}, strides[2] = {K * size, K * N * size};
  const cuuint32_t box[3] = {codes ? 128u : 64u, 128, 1};
  return encode(m, codes ? k8 : k16, 3, base, dims, strides, box, kSw128);
}

// Weights [G, N, K] read MN-major (K contiguous): 64 x 64 boxes, two at a time when K allows (the columns
// seen as blocks of 64 would reach past the last row otherwise).
bool map_weight_mn(CUtensorMap* m, const void* base, uint64_t G, uint64_t N, uint64_t K, bool wide) {
  if (wide) return map_mn2_g(m, base, K, N, G);
  const cuuint64_t dims[3] = {K, N, G}, strides[2] = {K * 2, K * N * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  return encode(m, k16, 3, base, dims, strides, box, kSw128);
}

// Rows [rows, width] read MN-major (width contiguous): likewise.
bool map_rows_mn(CUtensorMap* m, const void* base, uint64_t rows, uint64_t width, uint64_t ld, bool wide) {
  if (wide) {
    const cuuint64_t dims[3] = {64, rows, width / 64}, strides[2] = {ld * 2, 128};
    const cuuint32_t box[3] = {64, 64, 2};
    return encode(m, k16, 3, base, dims, strides, box, kSw128);
  }
  const cuuint64_t dims[2] = {width, rows}, strides[1] = {ld * 2};
  const cuuint32_t box[2] = {64, 64};
  return encode(m, k16, 2, base, dims, strides, box, kSw128);
}

// dW [G, N, K] in boxes of 32 rows x 64 bytes.
bool map_dw(CUtensorMap* m, const void* base, uint64_t G, uint64_t N, uint64_t K, bool fp32) {
  const uint64_t size = fp32 ? 4 : 2;
  const cuuint64_t dims[3] = {K, N, G}, strides[2] = {K * size, K * N * size};
  const cuuint32_t box[3] = {(cuuint32_t)(64 / size), 32, 1};
  return encode(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : k16, 3, base, dims, strides, box, kSw64);
}

uint32_t idesc_of(bool fp16, bool a_mn, bool b_mn) {
  const uint32_t fmt = fp16 ? 0u : (1u << 7) | (1u << 10);
  return (idesc_bf16(kTile, kTile, a_mn, b_mn) & ~((7u << 7) | (7u << 10))) | fmt;
}

Params params_of(const Grouped& c, const int32_t* begin, const int32_t* end, Hdr* hdr) {
  Params p{};
  p.begin = begin;
  p.end = end;
  p.rows = c.rows;
  p.G = c.G;
  p.fp16 = c.fp16;
  p.hdr = hdr;
  return p;
}

template <int kOp>
cudaError_t launch(const Params& p, int64_t most_tiles, int id, cudaStream_t s) {
  using S = Shape<kOp>;
  static int most = 0;   // pairs that run at once, per process (all devices here are alike)
  cudaError_t e = cudaFuncSetAttribute(grouped_kernel<kOp>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  if (e != cudaSuccess) return e;
  if (most == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2), 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::kSmem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, grouped_kernel<kOp>, &cfg) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = num_sms() / 2;
    }
    most = std::min(n, num_sms() / 2);
  }
  const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(most, most_tiles));
  prof_mark(id, s, true);
  grouped_kernel<kOp><<<2 * pairs, S::kThreads, S::kSmem, s>>>(p);
  prof_mark(id, s, false);
  return cudaGetLastError();
}

// The most row tiles the rows can make.
int64_t most_row_tiles(const Grouped& c) { return c.rows / kTile + std::min<int64_t>(c.G, c.rows); }

}  // namespace

cudaError_t launch_grouped_mm(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* x,
                              const uint16_t* W, uint16_t* y, Hdr* hdr, cudaStream_t s) {
  if (c.rows == 0) return cudaSuccess;
  Params p = params_of(c, begin, end, hdr);
  if (!map_weight(&p.a, W, false, c.G, c.N, c.K) || !map_rows(p.b, x, false, c.rows, c.K, c.ldi)) return cudaErrorInvalidValue;
  p.y = y;
  p.ldy = c.ldo;
  p.depth = c.K;
  p.width = c.N;
  p.nf = (c.N + kTile - 1) / kTile;
  p.idesc = idesc_of(c.fp16, false, false);
  return launch<kMm>(p, most_row_tiles(c) * p.nf, kKGroupedMm, s);
}

cudaError_t launch_grouped_dx(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* dy,
                              const uint16_t* W, uint16_t* dx, Hdr* hdr, cudaStream_t s) {
  if (c.rows == 0) return cudaSuccess;
  Params p = params_of(c, begin, end, hdr);
  p.wide_a = c.K % 64 == 0;
  if (!map_weight_mn(&p.a, W, c.G, c.N, c.K, p.wide_a) || !map_rows(p.b, dy, false, c.rows, c.N, c.ldo))
    return cudaErrorInvalidValue;
  p.y = dx;
  p.ldy = c.ldi;
  p.depth = c.N;
  p.width = c.K;
  p.nf = (c.K + kTile - 1) / kTile;
  p.idesc = idesc_of(c.fp16, true, false);
  return launch<kDx>(p, most_row_tiles(c) * p.nf, kKGroupedDx, s);
}

cudaError_t launch_grouped_dw(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* dy,
                              const uint16_t* x, void* dW, Hdr* hdr, cudaStream_t s) {
  Params p = params_of(c, begin, end, hdr);
  p.wide_a = c.N % 64 == 0;
  p.wide_b = c.K % 64 == 0;
  if (!map_dw(&p.out, dW, c.G, c.N, c.K, c.dw_fp32)) return cudaErrorInvalidValue;
  // without rows every tile is a zero tile and the operands' maps go unused
  if (c.rows > 0 && (!map_rows_mn(&p.a, dy, c.rows, c.N, c.ldo, p.wide_a) ||
                     !map_rows_mn(&p.b[0], x, c.rows, c.K, c.ldi, p.wide_b)))
    return cudaErrorInvalidValue;
  if (c.rows == 0) p.a = p.b[0] = p.out;
  p.y = dW;
  p.M = c.N;
  p.width = c.K;
  p.mf = (c.N + kTile - 1) / kTile;
  p.nf = (c.K + kTile - 1) / kTile;
  p.dw_fp32 = c.dw_fp32;
  p.acc = c.acc;
  p.idesc = idesc_of(c.fp16, true, true);
  return launch<kDw>(p, (int64_t)c.G * p.mf * p.nf, kKGroupedDw, s);
}

cudaError_t launch_grouped_i8(const Grouped& c, const int32_t* begin, const int32_t* end, const int8_t* q,
                              const float* qs, const int8_t* Wq, const float* Ws, uint16_t* y, Hdr* hdr,
                              cudaStream_t s) {
  if (c.rows == 0) return cudaSuccess;
  Params p = params_of(c, begin, end, hdr);
  if (!map_weight(&p.a, Wq, true, c.G, c.N, c.K) || !map_rows(p.b, q, true, c.rows, c.K, c.ldi)) return cudaErrorInvalidValue;
  p.y = y;
  p.ldy = c.ldo;
  p.qs = qs;
  p.ws = Ws;
  p.depth = c.K;
  p.width = c.N;
  p.nf = (c.N + kTile - 1) / kTile;
  p.idesc = idesc_of(true, false, false);   // widened codes are fp16, whatever y's type
  return launch<kI8>(p, most_row_tiles(c) * p.nf, kKGroupedI8, s);
}

cudaError_t launch_segments(const Tables* tabs, int G, int32_t* begin, int32_t* end, cudaStream_t s) {
  segments_kernel<<<1, 256, 0, s>>>(tabs, G, begin, end);
  return cudaGetLastError();
}

}  // namespace moe
