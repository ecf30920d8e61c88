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
//   warps 6-21  8-bit integers: widen the codes to fp16 (below)
//
// Rows times a weight.  The weight's 256 features are the M side of the tile and up to 256 rows of one
// group its N side, so a group's ragged end costs a narrower product (N in steps of 32) rather than
// padded rows: tensor time follows the rows there are.  Rows past the end of the group are loaded (they
// belong to the next group, or lie outside the tensor and read as zero) and fill accumulator columns of
// their own, which nothing stores.  The accumulator holds a feature per TMEM lane and a row per column,
// so a warp stores 32 features of a row at a time.
//
// Weight gradient.  M = 256 columns of x, N = 256 columns of dy, K = the group's rows, both operands
// MN-major; so here too the accumulator holds a column of dW per TMEM lane and a row per column, and a warp
// stores runs of a row (128 bytes of fp32).  Rows past the end of the group would enter the sums, so
// every group has tensor maps of its own whose rows end where the group does (written by a small kernel
// before: group_maps_kernel), and the copies fill the rest of its last K block with zeros.  The rows
// go in runs of kRun: an accumulator loses up to one unit of its last place at each step of 16 rows, always
// towards zero, and over a whole group the losses would pass the output's own rounding (rows of one sign
// without runs: 4.0e-4 low at 65536 rows, 6.6e-3 at 2^20, where half a step of fp16 is 4.9e-4).  With dW in
// fp32 every run after the first adds to dW what the same threads stored before it; with dW in 16 bits the
// epilogue's threads keep their sums in registers from run to run, and round them once.
//
// 8-bit integers.  sm_103a has no integer product at tensor rates (mma.sync on 8-bit integers: 256 products
// a clock and SM, a quarter of its fp16 rate and a sixteenth of tcgen05's), but every code is exact in
// fp16 and a product of two in fp32, so fp16 tensor products of widened codes are the integer products,
// and their fp32 sums are exact up to 2^24.  TMA brings the codes as bytes to a ring of raw stages, and
// sixteen warps widen them into the ring that the tensor cores read.
//
// Measured (graph replays on inputs larger than L2; 36 launches / after three seconds of them, when the power
// cap has lowered the clock): y of 16384 rows, 8 groups, 4096 x 14336, bf16: 1.14 / 1.19 ms, 1.69 / 1.62
// PFLOP/s, bound by the tensor cores under the power cap; with 8-bit integers 1.38 / 1.39 ms, bound by
// shared memory (the codes' way in, through the widening and out to the products).  dx and dW of 98304 rows,
// 64 groups, 2048 x 1408: 0.35 and 0.37 / 0.41 and 0.43 ms, 1.61 and 1.51 / 1.39 and 1.32 PFLOP/s; the rest is
// the tiles' ends (22 K blocks and fewer a tile).  fp32 dW += of 8192 rows, 128 groups, 2048 x 768: 0.27 ms,
// 5.5 TB/s, bound by reading and writing dW.  The contraction of a tile is one pair's: few tiles of a long one
// leave the other pairs idle (dW of one group, 65536 rows, 128 x 128: one tile, 294 us; y of 300 rows,
// 14336 to 512: four, 67 us).
#include <algorithm>

#include "common.cuh"
#include "grouped.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

namespace moe {

namespace {

enum Op { kMm, kDx, kDw, kI8 };

constexpr int kBM = 128;                     // rows of the M side a CTA holds
constexpr int kTile = 256;                   // pair tile, both sides
constexpr int kBK = 64;                      // K block of a stage (128 bytes a row)
constexpr uint32_t kHalf = kBM * kBK * 2;    // 16 KB: one operand of a stage
constexpr uint32_t kBox = 64 * kBK * 2;      // 8 KB: a 64 x 64 box (MN-major)
constexpr int kBoxes = 3;                    // row-operand boxes: 128, 64 and 32 rows
constexpr int kChunkM = 16;                  // row tiles per L2 reuse chunk of a group
constexpr int kRun = 2048;                   // rows of a run of the weight gradient
constexpr int kTmemCols = 512;
constexpr int kAhead = 4;                    // raw stages of weights fetched to L2 ahead (8-bit integers)

template <int kOp>
struct Shape {
  static constexpr int kStages = kOp == kI8 ? 4 : 6;
  static constexpr int kRaw = kOp == kI8 ? 2 : 0;          // 8-bit integers: stages of codes, two K blocks each,
  static constexpr int kTeams = 4, kTeam = 4;              // and the teams of warps that widen them
  static constexpr int kExtra = kOp == kI8 ? kTeams * kTeam : 0;
  static constexpr int kEpiWarps = kOp == kDw ? 8 : 4;
  static constexpr int kThreads = 32 * (2 + kEpiWarps + kExtra);
  static constexpr size_t kSmem = 1024 + (size_t)(kStages + kRaw) * 2 * kHalf + 512 + sizeof(GroupTab);
  static_assert(kSmem <= 232448, "shared memory per block");
};

struct Params {
  CUtensorMap a;              // M side: the weight
  CUtensorMap b[kBoxes];      // N side: the rows in boxes of 128, 64, 32
  const CUtensorMap* maps;    // weight gradient: every group's x (M side) and dy (N side)
  const int32_t *begin, *end;
  void* y;
  const float *qs, *ws;       // scales of the rows and of the output channels (8-bit integers)
  int64_t rows, ldy;
  int depth;                  // contraction length (rows times a weight)
  int width;                  // features of the output row; weight gradient: columns of dW (n_in)
  int M;                      // weight gradient: rows of a dW (n_out)
  int G, nf, mf;              // whole tiles across width; weight gradient: all tiles across width and M
  bool narrow;                // rows times a weight: there is a last, narrower tile across width
  bool fp16;
  bool wide_a, wide_b;        // weight gradient: one copy fetches two 64-column boxes (columns a multiple of 64)
  bool dw_fp32, acc;
  uint32_t idesc;             // N and M as of a full tile
  Hdr* hdr;
};

struct Job {
  int g, row, n, f0;   // rows times a weight: first row, rows, first feature
  int kits;            // K blocks
  int k0, k;           // weight gradient (row, n, f0: rows and columns of dW): rows of the run,
  int run, runs;       // its number, of how many
};

// Rows times a weight: tile t -> group, row tile, feature tile.  Groups in order; within a group,
// chunks of up to 16 row tiles x all feature tiles with the row tile fastest, so that the pairs at work
// share a panel of each operand in L2.
__device__ __forceinline__ Job row_job(const Params& p, const GroupTab& s, int t) {
  // the tiles of the last, narrower feature tile (if there is one) come after all others: what is
  // left to do while the last pairs finish is then short
  const int full = s.first[p.G] * p.nf;
  const bool narrow = t >= full;
  const int nf = narrow ? 1 : p.nf;
  if (narrow) t -= full;
  const int m = t / nf;
  int lo = 0, hi = p.G - 1;   // the last group whose first tile <= m
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.first[mid] <= m) lo = mid; else hi = mid - 1;
  }
  const int first = s.first[lo], mt = s.first[lo + 1] - first;
  const int local = t - first * nf;
  const int c = local / (kChunkM * nf);
  const int cm = min(kChunkM, mt - c * kChunkM);
  const int r = local - c * kChunkM * nf;
  Job j{};
  j.g = lo;
  j.row = s.begin[lo] + (c * kChunkM + r % cm) * kTile;
  j.n = min(kTile, s.end[lo] - j.row);
  j.f0 = narrow ? p.nf * kTile : r / cm * kTile;
  return j;
}

// Weight gradient: tile t -> group, tile of dW; a tile is one job a run of rows.
__device__ __forceinline__ int job_runs(int n) { return n > kRun ? (n + kRun - 1) / kRun : 1; }

__device__ __forceinline__ Job dw_job(const Params& p, const GroupTab& s, int t, int run) {
  const int per = p.mf * p.nf;
  Job j{};
  j.g = t / per;
  const int r = t - j.g * per;
  j.row = r / p.nf * kTile;
  j.n = min(kTile, p.M - j.row);
  j.f0 = r % p.nf * kTile;
  j.run = run;
  const int n = s.end[j.g] - s.begin[j.g], from = run * kRun;
  j.runs = job_runs(n);
  j.k0 = s.begin[j.g] + from;
  j.k = min(kRun, n - from);
  j.kits = (j.k + kBK - 1) / kBK;
  return j;
}

// The rows' box for a half of n rows: 0 (128 rows), 1 (64) or 2 (32).
__device__ __forceinline__ int box_of(int half) { return half > 64 ? 0 : (half > 32 ? 1 : 2); }

// One pair's walk over its tiles, the same in every role of both CTAs: rows times a weight has one job a
// tile, the weight gradient one a run of rows.
template <int kOp>
struct Walk {
  const Params& p;
  const GroupTab& s;
  int t, step, ntiles, run = 0;
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
    j = dw_job(p, s, t, run);
    if (++run == j.runs) {
      run = 0;
      t += step;
    }
    return true;
  }
};

// A store or an addition under a predicate rather than a branch, so that a run of them needs no reconvergence.
__device__ __forceinline__ void store_if(void* at, uint32_t w, bool yes) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.b32 [%0], %1;\n\t}" ::"l"(at), "r"(w),
               "r"((int)yes)
               : "memory");
}

__device__ __forceinline__ void add_if(float* at, float v, bool yes) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p red.global.add.f32 [%0], %1;\n\t}" ::"l"(at), "f"(v),
               "r"((int)yes)
               : "memory");
}

// ---- epilogues -----------------------------------------------------------------------------------

// 16-bit outputs: 32 rows (from c on) of this warp's 32 features, `out` at this lane's first of them.  Lanes
// exchange with their neighbour so that each holds two features of one row: an instruction stores 64 bytes
// of two rows.
template <int kOp>
__device__ __forceinline__ void emit16(const Params& p, const Job& j, uint16_t* out, int64_t ld, bool live, int lane,
                                       int c, float ws, float qs, const float (&v)[32]) {
  const bool odd = lane & 1;
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
    if (kOp == kI8) {
      a *= ws;
      b *= ws;
    }
    const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    if (kOp == kI8) {   // this lane now has two features of row c + 2 i + odd
      const float s = __shfl_sync(0xffffffffu, qs, 2 * i + odd);
      w[i] = odd ? pack16(got * s, b * s, p.fp16) : pack16(a * s, got * s, p.fp16);
    } else {
      w[i] = odd ? pack16(got, b, p.fp16) : pack16(a, got, p.fp16);
    }
  }
  const int left = live ? j.n - c - odd : 0;   // this lane's rows from c on
#pragma unroll
  for (int i = 0; i < 16; ++i) store_if(out + 2 * i * ld, w[i], 2 * i < left);
}

// This warp's 32 features (lanes) of the tile's rows (columns), the first row at `out`, ld elements apart.
template <int kOp>
__device__ __forceinline__ void store16(const Params& p, const Job& j, uint16_t* out, int64_t ld, int f, int lane,
                                        uint32_t ta, int share) {
  constexpr int kStep = 8 * Shape<kOp>::kEpiWarps;   // rows from one turn of the warp to the next
  const bool live = f < p.width;   // a multiple of 8: the same for both lanes of a pair
  const float ws = kOp == kI8 && live ? p.ws[(int64_t)j.g * p.width + f] : 1.f;
  out += (32 * share + (lane & 1)) * ld + (f & ~1);
#pragma unroll 1
  for (int c = 32 * share; c < j.n; c += kStep, out += kStep * ld) {
    uint32_t u[32];
    tmem_ld32(ta + c, u);
    float qs = 0.f;
    if (kOp == kI8) qs = c + lane < j.n ? p.qs[j.row + c + lane] : 0.f;
    tmem_ld_wait();
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
    emit16<kOp>(p, j, out, ld, live, lane, c, ws, qs, v);
  }
}

// A 16-bit dW whose rows come in runs: the warp's share of the sums stays in its registers from run to run
// and is rounded once, at the end.  (8 groups of 12288 rows, 2048 x 1408: 373 us, 359 with one accumulator
// over each group; groups of up to 2048 rows the same.)
constexpr int kCarry = kTile / 64;   // 32 rows each: two warps share a lane quarter
__device__ __forceinline__ void sum16(const Params& p, const Job& j, int rank, int q, uint32_t ta, int share,
                                      float (&sum)[kCarry][32]) {
  if (j.f0 + kBM * rank + 32 * q >= p.width) return;   // the whole warp lies past the last feature
#pragma unroll
  for (int h = 0; h < kCarry; ++h) {
    const int c = 32 * share + 64 * h;
#pragma unroll
    for (int t = 0; t < 32; t += 16) {
      if (c + t >= j.n) continue;
      uint32_t u[16];
      tmem_ld16(ta + c + t, u);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[h][t + i] += __uint_as_float(u[i]);
    }
  }
}

__device__ __forceinline__ void store_sum16(const Params& p, const Job& j, int rank, int q, int lane, int share,
                                            float (&sum)[kCarry][32]) {
  const int f0 = j.f0 + kBM * rank + 32 * q, f = f0 + lane;
  if (f0 >= p.width) return;
  const int64_t row = (int64_t)j.g * p.M + j.row + 32 * share + (lane & 1);
  uint16_t* out = static_cast<uint16_t*>(p.y) + row * p.width + (f & ~1);
  const int64_t step = 64 * (int64_t)p.width;
#pragma unroll
  for (int h = 0; h < kCarry; ++h, out += step) {
    const int c = 32 * share + 64 * h;
    if (c < j.n) emit16<kDw>(p, j, out, p.width, f < p.width, lane, c, 1.f, 0.f, sum[h]);
  }
}

// fp32 outputs (weight gradient): an instruction stores 128 bytes of a row, or adds them to what is there
// (one addition an element and run, in order: the same sum every time; subnormal values count as zero).
template <int kOp>
__device__ __forceinline__ void store32(const Params& p, const Job& j, float* out, int64_t ld, int f, uint32_t ta,
                                        int share) {
  constexpr int kStep = 8 * Shape<kOp>::kEpiWarps;
  const bool add = p.acc || j.run > 0;
  const int n = f < p.width ? j.n : 0, step = (int)ld;
  out += 32 * share * ld + f;
#pragma unroll 1
  for (int c = 32 * share; c < j.n; c += kStep, out += kStep * ld) {
    uint32_t v[32];
    tmem_ld32(ta + c, v);
    tmem_ld_wait();
    if (add) {
#pragma unroll
      for (int i = 0; i < 32; ++i) add_if(out + i * step, __uint_as_float(v[i]), c + i < n);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) store_if(out + i * step, v[i], c + i < n);
    }
  }
}

// This warp's share of a finished tile.
template <int kOp>
__device__ __forceinline__ void store_tile(const Params& p, const Job& j, int rank, int q, int lane, uint32_t ta, int share) {
  const int f = j.f0 + kBM * rank + 32 * q + lane;
  if (f - lane >= p.width) return;   // the whole warp lies past the last feature
  if (kOp == kDw) {
    const int64_t first = ((int64_t)j.g * p.M + j.row) * p.width;
    if (p.dw_fp32) store32<kOp>(p, j, static_cast<float*>(p.y) + first, p.width, f, ta, share);
    else store16<kOp>(p, j, static_cast<uint16_t*>(p.y) + first, p.width, f, lane, ta, share);
  } else {
    store16<kOp>(p, j, static_cast<uint16_t*>(p.y) + (int64_t)j.row * p.ldy, p.ldy, f, lane, ta, share);
  }
}

// A running gradient's tile that the next epilogue will add to, to L2 ahead of it (a row a thread): without
// it the additions wait in L2 for HBM.
__device__ __forceinline__ void prefetch_dw(const Params& p, const Job& j, int rank, int q, int lane, int share) {
  const int f = j.f0 + kBM * rank, bytes = min(p.width - f, kBM) * 4;
  if (!p.acc || j.kits == 0 || j.run > 0 || bytes <= 0) return;
  const int row = j.row + 128 * share + 32 * q + lane;
  if (row < p.M)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const float*>(p.y) +
                                                                   ((int64_t)j.g * p.M + row) * p.width + f),
                 "r"(bytes)
                 : "memory");
}

// A group without rows has a zero gradient (nothing to add to a running one): this warp's 32 columns of
// the tile.
__device__ __forceinline__ void store_zero(const Params& p, const Job& j, int rank, int q, int lane, int share) {
  const int f = j.f0 + kBM * rank + 32 * q + lane;
  if (p.acc || f >= p.width) return;
  const int64_t first = ((int64_t)j.g * p.M + j.row) * p.width + f;
  for (int i = share; i < j.n; i += 2) {
    if (p.dw_fp32) static_cast<float*>(p.y)[first + (int64_t)i * p.width] = 0.f;
    else static_cast<uint16_t*>(p.y)[first + (int64_t)i * p.width] = 0;
  }
}

// Before the first copy by a tensor map that an earlier kernel wrote.
__device__ __forceinline__ void fence_map(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// A box of a tensor to L2.
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
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

// Barriers (the same offsets in both CTAs; who uses which copy):
//   full[s]     even CTA: the stage's operands of both CTAs are in place (TMA bytes; 8-bit integers: the
//               warps that widened them)
//   empty[s]    stage free: committed to the even CTA, whose producer forwards it to the odd one when it
//               refills the stage (8-bit integers: committed to both, the widening warps wait)
//   tfull[a]    each CTA: accumulator a is complete
//   tempty[a]   even CTA: both CTAs' epilogues have read it
//   raw[s]      8-bit integers, own CTA: the bytes of a raw stage
//   rempty[s]   8-bit integers, own CTA: every widening warp has passed it
// Every wait is bounded; whatever happens, both CTAs meet at the last cluster barrier before TMEM is
// freed, with their own copies landed.
template <int kOp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<kOp>::kThreads, 1)
    grouped_kernel(const __grid_constant__ Params p) {
  using S = Shape<kOp>;
  constexpr int kStages = S::kStages;
  constexpr uint32_t kStage = 2 * kHalf;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = smem;
  uint8_t* raws = stages + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(raws + S::kRaw * kStage);
  uint64_t* empty = full + 6;
  uint64_t* raw = empty + 6;
  uint64_t* rempty = raw + 6;
  uint64_t* tfull = rempty + 6;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  GroupTab& tab = *reinterpret_cast<GroupTab*>(raws + S::kRaw * kStage + 512);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 6; ++s) {
      mbar_init(&full[s], kOp == kI8 ? 2 * S::kTeam : 1);
      mbar_init(&empty[s], 1);
      mbar_init(&raw[s], 1);
      mbar_init(&rempty[s], S::kTeams * S::kTeam);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * S::kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (kOp != kDw) {
      tma_prefetch(&p.a);
      for (int i = 0; i < kBoxes; ++i) tma_prefetch(&p.b[i]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  after_previous_kernel();
  const int rtiles = load_groups(tab, p.begin, p.end, p.G, p.rows, kTile, p.hdr);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t limit = wait_limit_ns(p.hdr);
  const int ntiles = rtiles < 0 ? 0 : (kOp == kDw ? p.G * p.mf * p.nf : rtiles * (p.nf + (int)p.narrow));
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
      int mapped = -1;   // weight gradient: the group whose maps are in use
      bool ok = true;
      // test hook: the first pair skips one fill, so that the wait for it runs out
      const int skip = pair == 0 ? *((volatile const int32_t*)&p.hdr->stall_fill_p1) - 1 : -1;
      if constexpr (kOp == kI8) {
        while (ok && !*abort_flag && walk.next(j)) {
          const int half = ((j.n + 31) / 32 * 32) / 2, bx = box_of(half);
          for (int kit = 0; kit < (j.kits + 1) / 2; ++kit) {
            if (!wait_nap<20>(&rempty[slot], phase ^ 1, limit, abort_flag)) {
              fail(kSiteGroupedProducer);
              ok = false;
              break;
            }
            if (uses != skip) {
              uint8_t* st = raws + (size_t)slot * kStage;
              mbar_arrive_expect_tx(&raw[slot], kHalf + (128u >> bx) * 128u);
              tma_load_3d(st, &p.a, &raw[slot], kit * 2 * kBK, j.f0 + kBM * rank, j.g);
              // two raw stages do not cover the way from HBM: the weight's next ones come to L2 before
              if ((kit + kAhead) * 2 * kBK < p.depth)
                prefetch_3d(&p.a, (kit + kAhead) * 2 * kBK, j.f0 + kBM * rank, j.g);
              tma_load_2d(st + kHalf, &p.b[bx], &raw[slot], kit * 2 * kBK, j.row + half * rank);
            }
            ++uses;
            if (++slot == S::kRaw) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        drain_fills(raw, S::kRaw, slot, phase, uses, limit);
      } else {
        while (ok && !*abort_flag && walk.next(j)) {
          const int half = ((j.n + 31) / 32 * 32) / 2, bx = kOp == kDw ? 0 : box_of(half);
          const uint32_t bytes = kHalf + (kOp == kDw ? kHalf : (128u >> bx) * 128u);
          const CUtensorMap* ma = &p.a;
          const CUtensorMap* mb = &p.b[bx];
          if constexpr (kOp == kDw) {
            ma = p.maps + 2 * j.g;
            mb = ma + 1;
            if (j.g != mapped && j.kits > 0) {
              fence_map(ma);
              fence_map(mb);
              mapped = j.g;
            }
          }
          for (int kit = 0; kit < j.kits; ++kit) {
            if (!wait_nap<20>(&empty[slot], phase ^ 1, limit, abort_flag)) {
              fail(kSiteGroupedProducer);
              ok = false;
              break;
            }
            if (uses != skip) {
              uint8_t* st = stages + (size_t)slot * kStage;
              if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * bytes);
              const uint32_t bar = cluster_addr(&full[slot], 0);
              if constexpr (kOp == kDw) {
                const int row = j.k0 + kit * kBK, ca = j.f0 + kBM * rank, cb = j.row + kBM * rank;
                if (p.wide_a) {
                  tma_load_3d_pair(st, ma, bar, 0, row, ca / 64);
                } else {
                  tma_load_2d_pair(st, ma, bar, ca, row);
                  tma_load_2d_pair(st + kBox, ma, bar, ca + 64, row);
                }
                if (p.wide_b) {
                  tma_load_3d_pair(st + kHalf, mb, bar, 0, row, cb / 64);
                } else {
                  tma_load_2d_pair(st + kHalf, mb, bar, cb, row);
                  tma_load_2d_pair(st + kHalf + kBox, mb, bar, cb + 64, row);
                }
              } else {
                const int f = j.f0 + kBM * rank;
                if (kOp == kMm) {
                  tma_load_3d_pair(st, ma, bar, kit * kBK, f, j.g);
                } else {
                  tma_load_3d_pair(st, ma, bar, f, kit * kBK, j.g);
                  tma_load_3d_pair(st + kBox, ma, bar, f + 64, kit * kBK, j.g);
                }
                tma_load_2d_pair(st + kHalf, mb, bar, kit * kBK, j.row + half * rank);
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
        // full barriers count both CTAs' bytes, and the odd CTA waits at the cluster barrier
        if (rank == 0) drain_fills(full, kStages, slot, phase, uses, limit);
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
        if (!wait_nap<20>(&tempty[acc], acc_phase ^ 1, limit, abort_flag)) {
          fail(kSiteGroupedMma);
          break;
        }
        tc_fence_after();
        for (int kit = 0; kit < kits; ++kit) {
          if (!wait_nap<20, kOp == kI8>(&full[slot], phase, limit, abort_flag)) {
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
  } else if (warp < 2 + S::kEpiWarps) {
    const int q = warp & 3;                      // TMEM lane quarter this warp may access
    const int share = (warp - 2) / 4;            // of two warps of a quarter: every other 32 rows
    int acc = 0;
    uint32_t acc_phase = 0;
    auto wait_acc = [&]() {
      if (!mbar_wait_idle(&tfull[acc], acc_phase, limit, abort_flag)) {
        fail(kSiteGroupedEpilogue);
        return false;
      }
      tc_fence_after();
      return true;
    };
    auto acc_addr = [&]() { return tmem_base + (uint32_t)(acc * kTile) + ((uint32_t)(q * 32) << 16); };
    auto release_acc = [&]() {
      tc_fence_before();
      __syncwarp();
      // (relaxed: the reads of the accumulator have completed, and a release would wait for the tile's stores)
      if (lane == 0) mbar_arrive_cluster_relaxed(cluster_addr(&tempty[acc], 0));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    };
    Job next;
    bool more = walk.next(next);
    if (kOp == kDw && more) prefetch_dw(p, next, rank, q, lane, share);
    while (more) {
      j = next;
      more = walk.next(next);
      if (kOp == kDw && more) prefetch_dw(p, next, rank, q, lane, share);
      if (j.kits == 0) {
        store_zero(p, j, rank, q, lane, share);
        continue;
      }
      if (kOp == kDw && !p.dw_fp32 && j.runs > 1) {
        float sum[kCarry][32] = {};
        bool ok = true;
        while (true) {
          ok = wait_acc();
          if (!ok) break;
          sum16(p, j, rank, q, acc_addr(), share, sum);
          release_acc();
          if (j.run == j.runs - 1) break;
          j = next;   // (the next run)
          more = walk.next(next);
        }
        if (!ok) break;
        store_sum16(p, j, rank, q, lane, share, sum);
        continue;
      }
      if (!wait_acc()) break;
      store_tile<kOp>(p, j, rank, q, lane, acc_addr(), share);
      release_acc();
    }
  } else if constexpr (kOp == kI8) {
    // Widen: the teams take turns at the K blocks (a raw stage holds two), each with a stage of its own; a
    // warp takes every fourth octet of rows (of the weight's 128, then of up to 128 token rows), a lane a
    // row and 16 of its codes: in the 128-byte swizzle the eight lanes of a phase touch distinct banks
    // on both sides.  (Four teams of four warps hide the way of a block through its barriers better than two of
    // eight: 1632 against 1920 us at 16384 rows, 4096 x 14336, when that was tried.)
    static_assert(kStages == S::kTeams, "a stage a team");
    constexpr int kPer = kBM / 8 / S::kTeam;
    const int team = (warp - 2 - S::kEpiWarps) / S::kTeam, w = (warp - 2 - S::kEpiWarps) % S::kTeam, r = lane & 7, cq = lane >> 3;
    const uint32_t to = (w * 8 + r) * 128;
    const uint32_t o0 = ((2 * cq) ^ r) << 4, o1 = ((2 * cq + 1) ^ r) << 4;
    int block = 0, rblock = 0;   // K blocks and raw stages before this job
    bool ok = true;
    while (ok && walk.next(j)) {
      const int half = ((j.n + 31) / 32 * 32) / 2;
      const int kits = j.kits, rkits = (kits + 1) / 2;
      for (int rk = 0; rk < rkits; ++rk) {
        // every warp waits for every raw stage and releases it: a barrier's phase must not pass a waiter by
        const int rs = (rblock + rk) % S::kRaw;
        const int kit = 2 * rk + ((team - block - 2 * rk) & (S::kTeams - 1));   // this team's next block
        const bool mine = kit < min(2 * rk + 2, kits);
        const int at = block + kit;
        ok = __all_sync(0xffffffffu, wait_nap<0>(&raw[rs], (uint32_t)((rblock + rk) / S::kRaw) & 1u, limit, abort_flag));
        if (!ok) {
          if (lane == 0) fail(kSiteGroupedStage);
          break;
        }
        // the codes to registers, and the raw stage free before this warp waits for the stage they go to
        uint4 v[2 * kPer];
        if (mine) {
          const uint8_t* src = raws + (size_t)rs * kStage + to + ((((kit & 1) * 4 + cq) ^ r) << 4);
#pragma unroll
          for (int i = 0; i < 2 * kPer; ++i)
            if (i < kPer || ((i - kPer) * S::kTeam + w) * 8 < half)
              v[i] = *reinterpret_cast<const uint4*>(src + i * S::kTeam * 1024);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rempty[rs]);
        if (!mine) continue;
        ok = __all_sync(0xffffffffu, wait_nap<0>(&empty[team], ((uint32_t)(at / kStages) & 1u) ^ 1u, limit, abort_flag));
        if (!ok) {
          if (lane == 0) fail(kSiteGroupedStage);
          break;
        }
        uint8_t* dst = stages + (size_t)team * kStage + to;
#pragma unroll
        for (int i = 0; i < 2 * kPer; ++i) {
          if (i >= kPer && ((i - kPer) * S::kTeam + w) * 8 >= half) break;
          uint8_t* d = dst + i * S::kTeam * 1024;
          *reinterpret_cast<uint4*>(d + o0) = widen(v[i].x, v[i].y);
          *reinterpret_cast<uint4*>(d + o1) = widen(v[i].z, v[i].w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          fence_release_smem();
          mbar_arrive_cluster_relaxed(cluster_addr(&full[team], 0));
        }
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

// The maps of every group's rows of x and dy for the weight gradient: those of all rows (dimension 1
// counts rows in both forms), ending at the group's end.  A block a group, a warp a map.
__global__ void __launch_bounds__(64) group_maps_kernel(const __grid_constant__ CUtensorMap a,
                                                        const __grid_constant__ CUtensorMap b, const int32_t* end,
                                                        int64_t rows, CUtensorMap* maps) {
  __shared__ __align__(128) CUtensorMap map[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.x;
  reinterpret_cast<uint32_t*>(&map[warp])[lane] = reinterpret_cast<const uint32_t*>(warp == 0 ? &a : &b)[lane];
  __syncwarp();
  after_previous_kernel();
  if (lane == 0) {
    const int64_t to = end[g];   // (whatever it holds, the map stays within the tensor)
    const uint32_t dim = (uint32_t)(to < 1 ? 1 : (to > rows ? rows : to));
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(smem_u32(&map[warp])),
                 "r"(dim)
                 : "memory");
  }
  __syncwarp();
  asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
                   reinterpret_cast<uint64_t>(maps + 2 * g + warp)),
               "r"(smem_u32(&map[warp]))
               : "memory");
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

constexpr CUtensorMapDataType k16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;   // (fp16 values too: bits are copied)
constexpr CUtensorMapDataType k8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
constexpr CUtensorMapSwizzle kSw128 = CU_TENSOR_MAP_SWIZZLE_128B;

// Rows [rows, width], 16-bit or codes, as K-major boxes of 128 bytes x 128, 64 and 32 rows.
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

// Weights [G, N, K] read MN-major (K contiguous): boxes of 64 x 64.
bool map_weight_mn(CUtensorMap* m, const void* base, uint64_t G, uint64_t N, uint64_t K) {
  const cuuint64_t dims[3] = {K, N, G}, strides[2] = {K * 2, K * N * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  return encode(m, k16, 3, base, dims, strides, box, kSw128);
}

// Rows [rows, width] read MN-major (width contiguous): likewise, or two boxes at a time where the width allows (the
// columns seen as blocks of 64 would reach past the last row otherwise).  dW reads both operands so, and is
// the faster by it: 98304 rows, 64 groups of 2048 x 1408, 375 us with a copy for two boxes and 411 with two
// copies.  (dx measured the same either way and has one form.)
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
  static SmemOnce once;
  static IntOnce most;   // pairs that run at once
  cudaError_t e = once.set(reinterpret_cast<const void*>(grouped_kernel<kOp>), S::kSmem);
  if (e != cudaSuccess) return e;
  int fit = 0;
  e = most.get(&fit, [] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2), 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::kSmem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, grouped_kernel<kOp>, &cfg) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = num_sms() / 2;
    }
    return std::min(n, num_sms() / 2);
  });
  if (e != cudaSuccess) return e;
  const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(fit, most_tiles));
  prof_mark(id, s, true);
  e = launch_after(grouped_kernel<kOp>, 2 * pairs, S::kThreads, S::kSmem, 1, s, p);   // (clusters of two: by its attribute)
  prof_mark(id, s, false);
  return e;
}

// The most row tiles the rows can make.
int64_t most_row_tiles(const Grouped& c) { return c.rows / kTile + std::min<int64_t>(c.G, c.rows); }

}  // namespace

cudaError_t launch_grouped_mm(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* x,
                              const uint16_t* W, uint16_t* y, Hdr* hdr, cudaStream_t s) {
  if (c.rows == 0) return cudaSuccess;
  if (stream_eligible(c, false)) return launch_stream_mm(c, begin, end, x, W, y, hdr, s);
  Params p = params_of(c, begin, end, hdr);
  if (!map_weight(&p.a, W, false, c.G, c.N, c.K) || !map_rows(p.b, x, false, c.rows, c.K, c.ldi)) return cudaErrorInvalidValue;
  p.y = y;
  p.ldy = c.ldo;
  p.depth = c.K;
  p.width = c.N;
  p.nf = c.N / kTile;
  p.narrow = c.N % kTile != 0;
  p.idesc = idesc_of(c.fp16, false, false);
  return launch<kMm>(p, most_row_tiles(c) * (p.nf + p.narrow), kKGroupedMm, s);
}

cudaError_t launch_grouped_dx(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* dy,
                              const uint16_t* W, uint16_t* dx, Hdr* hdr, cudaStream_t s) {
  if (c.rows == 0) return cudaSuccess;
  Params p = params_of(c, begin, end, hdr);
  if (!map_weight_mn(&p.a, W, c.G, c.N, c.K) || !map_rows(p.b, dy, false, c.rows, c.N, c.ldo))
    return cudaErrorInvalidValue;
  p.y = dx;
  p.ldy = c.ldi;
  p.depth = c.N;
  p.width = c.K;
  p.nf = c.K / kTile;
  p.narrow = c.K % kTile != 0;
  p.idesc = idesc_of(c.fp16, true, false);
  return launch<kDx>(p, most_row_tiles(c) * (p.nf + p.narrow), kKGroupedDx, s);
}

cudaError_t launch_grouped_dw(const Grouped& c, const int32_t* begin, const int32_t* end, const uint16_t* dy,
                              const uint16_t* x, void* dW, Hdr* hdr, void* maps, cudaStream_t s) {
  Params p = params_of(c, begin, end, hdr);
  p.wide_a = c.K % 64 == 0;
  p.wide_b = c.N % 64 == 0;
  p.maps = static_cast<const CUtensorMap*>(maps);
  if (c.rows > 0) {   // (without rows every tile is a zero tile)
    CUtensorMap mx, mdy;
    if (!map_rows_mn(&mx, x, c.rows, c.K, c.ldi, p.wide_a) || !map_rows_mn(&mdy, dy, c.rows, c.N, c.ldo, p.wide_b))
      return cudaErrorInvalidValue;
    prof_mark(kKGroupMaps, s, true);
    const cudaError_t e = launch_after(group_maps_kernel, c.G, 64, 0, 1, s, mx, mdy, end, c.rows,
                                       static_cast<CUtensorMap*>(maps));
    prof_mark(kKGroupMaps, s, false);
    if (e != cudaSuccess) return e;
  }
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
  if (stream_eligible(c, true)) return launch_stream_i8(c, begin, end, q, qs, Wq, Ws, y, hdr, s);
  Params p = params_of(c, begin, end, hdr);
  if (!map_weight(&p.a, Wq, true, c.G, c.N, c.K) || !map_rows(p.b, q, true, c.rows, c.K, c.ldi)) return cudaErrorInvalidValue;
  p.y = y;
  p.ldy = c.ldo;
  p.qs = qs;
  p.ws = Ws;
  p.depth = c.K;
  p.width = c.N;
  p.nf = c.N / kTile;
  p.narrow = c.N % kTile != 0;
  p.idesc = idesc_of(true, false, false);   // widened codes are fp16, whatever y's type
  return launch<kI8>(p, most_row_tiles(c) * (p.nf + p.narrow), kKGroupedI8, s);
}

cudaError_t launch_segments(const Tables* tabs, int G, int32_t* begin, int32_t* end, cudaStream_t s) {
  prof_mark(kKSegments, s, true);
  segments_kernel<<<1, 256, 0, s>>>(tabs, G, begin, end);
  prof_mark(kKSegments, s, false);
  return cudaGetLastError();
}

}  // namespace moe
