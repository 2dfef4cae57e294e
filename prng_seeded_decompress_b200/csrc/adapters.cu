// adapters.cu -- low-rank adapters of many requests beside a shared
// projection: Y[m] = base[m] + s_a (x_m A_a^T) B_a^T with a the adapter of
// row m, and the plan that sorts a batch's rows by adapter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.cuh"
#include "seedlm_device.cuh"
#include "between_internal.h"
#include "tcgen05.cuh"

namespace seedlm {

SEEDLM_CHECK_FLAG(adapters)

namespace {

// Set when a plan does not belong to the call it is given to, or was written over.
__device__ unsigned int g_plan_mismatch;
// Set when a kernel gave up waiting for its own products.
__device__ unsigned int g_wait_error;

// ---------------------------------------------------------------- the plan
//
// Layout in int32 words: [0, M) order, [M, M + n + 1) offsets, then from the
// next multiple of 4, for tiles of up to 8 rows and for tiles of up to 64, a head
// {M + mark, n, tiles of rows with an adapter, all tiles}; then for each of the two an
// int4 {adapter or -1, first, count, 0} for every tile, in sorted order.  Each
// projection takes the one that suits it.  The mark is larger than any other
// word of a plan, so that no part of another plan looks like a head.

constexpr int kLowRows = 8, kTall = 64;
constexpr int kHeadMark = 0x5e000000;
static_assert(kMaxAdapterRows < 0x02000000 && (kHeadMark & 0x01ffffff) == 0, "M fits below the mark");

__host__ __device__ inline int64_t plan_tail(int64_t M, int64_t n) { return (M + n + 1 + 3) / 4 * 4; }

// Every bin of c rows takes at most c / T + 1 tiles.
__host__ __device__ inline int64_t max_tiles(int64_t M, int64_t n, int T) { return M / T + (M < n + 1 ? M : n + 1); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of all CTAs of the cluster; shared memory written before is
// visible after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A stable counting sort by one cluster: one CTA, or eight for many rows.  Each
// warp takes one contiguous part of the rows and counts its adapters in a
// histogram of its own (match_any groups the lanes of a step, so no two lanes
// touch a bin).  Bin by bin the histograms become starting places: over the
// warps of a CTA, then over the CTAs through distributed shared memory, then
// over the bins.  A second walk over the same rows puts each at its place.
// Latency bound: a few dependent steps, so each lane has 16 of its rows' ids in
// flight at once and keeps them for the second walk where they are all it has
// (64 rows: 3.3 us, 16384 rows of 500 adapters: 10.8 us, 38 us with one CTA and
// the ids read again one by one).
constexpr int kPlanThreads = 1024, kPlanCtas = 8;
constexpr int kPlanSteps = 16;  // ids a lane holds
constexpr int kPlanOneCtaRows = 2048;

__device__ __forceinline__ int load_of_cta(const int* mine, uint32_t cta) {
  uint32_t at;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(cta));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__global__ void __launch_bounds__(kPlanThreads, 1)
adapters_plan_kernel(int M, int n, const int32_t* ids, int32_t* plan) {
  extern __shared__ int32_t sm[];
  const int bins = n + 1, nwarps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = (int)cluster_rank(), ctas = (int)cluster_size();
  int32_t* hist = sm;                             // [nwarps][bins]
  int32_t* total = hist + (size_t)nwarps * bins;  // [bins] rows of each bin in this CTA
  int32_t* base = total + bins;                   // [bins] place of this CTA's first row of each bin
  int32_t* start = base + bins;                   // [bins + 1] of all CTAs
  int32_t* low_start = start + bins + 1;          // [bins + 1] low tiles before each bin
  int32_t* tall_start = low_start + bins + 1;     // [bins + 1] tall ones
  int32_t* warp_sums = tall_start + bins + 1;     // [3][32]
  grid_launch_dependents();
  for (int i = threadIdx.x; i < nwarps * bins; i += blockDim.x) hist[i] = 0;
  grid_wait();
  __syncthreads();
  const int chunk = ((M + ctas * nwarps - 1) / (ctas * nwarps) + 31) / 32 * 32;
  const int64_t first = (int64_t)(cta * nwarps + warp) * chunk;
  const int r0 = (int)(first < M ? first : M), r1 = min(M, r0 + chunk);
  int32_t* mine = hist + (size_t)warp * bins;
  int key[kPlanSteps];  // of row r + 32 i + lane: its bin, -1 for no row
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i) {
      const int row = r + 32 * i + lane;
      key[i] = row < r1 ? ids[row] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i) {
      if (key[i] < 0 || key[i] >= n) key[i] = n;
      if (r + 32 * i + lane >= r1) key[i] = -1;
    }
  };
  for (int r = r0; r < r1; r += 32 * kPlanSteps) {
    load(r);
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i) {
      if (r + 32 * i >= r1) break;
      const unsigned same = __match_any_sync(0xffffffffu, key[i]);
      if (key[i] >= 0 && (same & ((1u << lane) - 1)) == 0) mine[key[i]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += blockDim.x) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < nwarps; ++w) {
      const int t = hist[w * bins + b];
      hist[w * bins + b] = run;
      run += t;
    }
    total[b] = run;
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  // Every CTA scans all bins, each thread taking `per` consecutive ones.
  const int per = (bins + blockDim.x - 1) / blockDim.x;
  const int b0 = min(bins, (int)threadIdx.x * per), b1 = min(bins, b0 + per);
  int mine3[3] = {0, 0, 0};  // rows, low tiles, tall tiles
  for (int b = b0; b < b1; ++b) {
    int before = 0, all = 0;
    if (ctas == 1) {
      all = total[b];
    } else {
#pragma unroll
      for (int c = 0; c < kPlanCtas; ++c) {
        const int v = load_of_cta(total + b, c);
        all += v;
        if (c < cta) before += v;
      }
    }
    start[b] = mine3[0];  // within this thread's bins
    low_start[b] = mine3[1];
    tall_start[b] = mine3[2];
    base[b] = before;
    mine3[0] += all;
    mine3[1] += (all + kLowRows - 1) / kLowRows;
    mine3[2] += (all + kTall - 1) / kTall;
  }
  int before3[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    int incl = mine3[j];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[32 * j + warp] = incl;
    before3[j] = incl - mine3[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 3; ++j) {  // of the warps before this one, a lane each
    int v = lane < warp ? warp_sums[32 * j + lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    before3[j] += v;
  }
  for (int b = b0; b < b1; ++b) {
    start[b] += before3[0];
    low_start[b] += before3[1];
    tall_start[b] += before3[2];
    base[b] += start[b];
    if (cta == 0) plan[M + b] = start[b];
  }
  if (b1 == bins && b0 < bins) {  // the thread of the last bin
    start[bins] = before3[0] + mine3[0];
    low_start[bins] = before3[1] + mine3[1];
    tall_start[bins] = before3[2] + mine3[2];
  }
  __syncthreads();
  for (int r = r0; r < r1; r += 32 * kPlanSteps) {
    if (chunk > 32 * kPlanSteps) load(r);
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i) {
      if (r + 32 * i >= r1) break;
      const unsigned same = __match_any_sync(0xffffffffu, key[i]);
      const int rank = __popc(same & ((1u << lane) - 1));
      int at = 0;
      if (key[i] >= 0) at = base[key[i]] + mine[key[i]] + rank;
      __syncwarp();
      if (key[i] >= 0) {
        if (SEEDLM_IN_BOUNDS(g_check_flag, at, M)) plan[at] = r + 32 * i + lane;
        if (rank == 0) mine[key[i]] += __popc(same);
      }
      __syncwarp();
    }
  }
  int4* tail = reinterpret_cast<int4*>(plan + plan_tail(M, n));
  auto list = [&](int T, const int32_t* first, int4* head, int4* to) {
    const int all = first[bins];
    if (cta == 0 && threadIdx.x == 0) *head = make_int4(kHeadMark + M, n, first[n], all);
    for (int t = cta * blockDim.x + threadIdx.x; t < all; t += ctas * blockDim.x) {
      int lo = 0, hi = bins - 1;  // the last bin that starts at or before tile t
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int at = start[lo] + (t - first[lo]) * T;
      if (SEEDLM_IN_BOUNDS(g_check_flag, t, max_tiles(M, n, T)))
        to[t] = make_int4(lo < n ? lo : -1, at, min(T, start[lo + 1] - at), 0);
    }
  };
  list(kLowRows, low_start, tail, tail + 2);
  list(kTall, tall_start, tail + 1, tail + 2 + max_tiles(M, n, kLowRows));
  if (ctas > 1) cluster_sync();  // no CTA leaves while another reads its totals
}

// ------------------------------------------------------------- the products
//
// Two kernels.  The first takes the sums S = s_a x A_a^T, the second adds
// S B_a^T to the outputs.  Both feed mma.sync with fragments that need no
// shuffling: of a contraction step of 32, the lane in column q of its quad
// takes elements 8q .. 8q + 7 with one 16-byte load and gives words 0, 1 to a
// first m16n8k16 product and words 2, 3 to a second.  The order of the
// contraction does not matter as long as both operands are read alike.  The
// matrix of adapter weights is the operand of 16 rows and the tile's
// activations the one of 8 columns, so a request that is alone with its
// adapter wastes tensor work, of which there is plenty, and no memory traffic,
// which is what bounds both kernels.

constexpr int kLowWarps = 4;   // of the kernels for low tiles
constexpr int kStep = 32;      // contraction elements of one 16-byte load per lane
constexpr int kMaxSplits = 8;  // CTAs of a cluster that share the first contraction

// The parts of a sum that 16-bit operands hold.  bf16 has fp32's range: three
// parts cut off (not rounded, so none overflows) hold all 24 bits.  fp16 parts
// are of the sum times a power of two that brings the largest finite one of
// its block (64 ranks of a row, or all where there are fewer) to [2^14, 2^15):
// two rounded parts leave at most 2^-23 of a sum (half a step of the second, whose
// size is at most 2^-11 of the first's binade), or 2^-39 of the block's largest
// where that is more (half of fp16's smallest step, 2^-25, of 2^14).
template <bool BF16>
constexpr int kParts = BF16 ? 3 : 2;

struct ApplyArgs {
  seedlm_adapters ad;
  const int32_t* plan;
  const int4 *head, *tiles;  // the plan's, of the tiles that are taken
  int room;         // tiles that the plan has room for
  int M;
  const uint16_t* X;
  int64_t ldx;
  const float* base;
  int64_t ldb;
  float* Y;
  int64_t ldy;
  uint16_t* S;      // [M][slices][kParts][slots], rows in sorted order
  float* unscale;   // [M][slices][blocks]: takes fp16 parts back
  int slots;        // ranks of a slice: 32, or rank rounded up to 64
  int blocks;       // slots / 64, or 1
  int split_cols;   // columns of one CTA of the first kernel's clusters
  int groups;       // first kernel: CTAs that share a slice's (tall: all) ranks
  int chunk_first[SEEDLM_MAX_SLICES + 1];  // second kernel: chunks of outputs before each slice
  int chunk_rows;   // outputs of a chunk
  int slice_at[SEEDLM_MAX_SLICES];         // first output of each slice
  // Bytes that every row's address is a multiple of, at most 16.
  int grain_x, grain_a[SEEDLM_MAX_SLICES], grain_b[SEEDLM_MAX_SLICES], grain_y[SEEDLM_MAX_SLICES];
};

// What a plan says is checked before it is followed: memory that holds something
// else is reported and leads to no access outside the arrays.
__device__ __forceinline__ void plan_is_wrong() { atomicOr(&g_plan_mismatch, 1u); }

// The plan's head, with no tiles at all if it does not belong to this call.
__device__ __forceinline__ int4 plan_head(const ApplyArgs& p) {
  int4 head = __ldcg(p.head);
  if (head.x != kHeadMark + p.M || head.y != p.ad.n || (unsigned)head.w > (unsigned)p.room || (unsigned)head.z > (unsigned)head.w) {
    if (threadIdx.x == 0) plan_is_wrong();
    head.z = head.w = 0;
  }
  return head;
}

// Tile t {adapter or -1, first, rows, 0}; t below the plan's room, whether the
// plan has so many or not.
__device__ __forceinline__ int4 plan_tile(const ApplyArgs& p, int64_t t) {
  return __ldcg(p.tiles + t);
}

// Whether it is a tile of at most T rows of this batch, with an adapter from
// `least` on.
__device__ __forceinline__ bool tile_fits(const ApplyArgs& p, const int4& tile, int T, int least) {
  const bool fits = tile.x >= least && tile.x < p.ad.n && tile.z >= 0 && tile.z <= T && tile.y >= 0 && tile.y <= p.M - tile.z;
  if (!fits && threadIdx.x == 0) plan_is_wrong();
  return fits;
}

// A row's number as the plan has it, -1 if there is no such row.
__device__ __forceinline__ int row_of(const ApplyArgs& p, int row) {
  if ((unsigned)row < (unsigned)p.M) return row;
  plan_is_wrong();
  return -1;
}
// The row at place i of the batch in sorted order.
__device__ __forceinline__ int plan_row(const ApplyArgs& p, int i) { return row_of(p, __ldcg(p.plan + i)); }

__device__ __forceinline__ int rank_of(const seedlm_adapters& ad, int a) {
  if (a < 0) return 0;
  return ad.ranks ? max(0, min(__ldcg(ad.ranks + a), ad.rank)) : ad.rank;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Half a step of 32: rows g and g + 8 of the 16-row operand in lo and hi.  The
// halves of several sums are issued in turn, so that no product waits for the
// one before it.
template <bool BF16>
__device__ __forceinline__ void mma_half(int half, float (&d)[4], const uint4& lo, const uint4& hi, const uint4& x) {
  if (half == 0) mma16816<BF16>(d, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
  else mma16816<BF16>(d, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

// Asynchronous copy of 16 bytes to shared memory, all but the first `bytes`
// of them zero (with none, nothing is read).
__device__ __forceinline__ void copy16(void* to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
               "r"(bytes)
               : "memory");
}
// The same where a row's neighbours in its 128-byte line are not wanted: the L2
// then fetches 64 bytes of it, not the line (measured: half the DRAM traffic
// for rows of up to 64 bytes in every 128).
__device__ __forceinline__ void copy16_short(void* to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(bytes)
               : "memory");
}
// The same, or nothing.
__device__ __forceinline__ void copy16_if(bool on, uint32_t to, const void* from, int bytes) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16, %2;\n\t}" ::"r"(to),
               "l"(from), "r"(bytes), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

template <int SIZE>
__device__ __forceinline__ void copy_small(void* to, const void* from, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
               "n"(SIZE), "r"(bytes)
               : "memory");
}

// A matrix's elements, from the first to behind the last: what lies between two
// of its rows may be read (and is not used).
struct Extent {
  const uint16_t* first;
  int64_t size;
};
__device__ __forceinline__ Extent extent_x(const ApplyArgs& p) { return {p.X, (p.M - 1) * p.ldx + p.ad.cols}; }
__device__ __forceinline__ Extent extent_a(const ApplyArgs& p, int s) {
  return {static_cast<const uint16_t*>(p.ad.A[s]),
          (p.ad.n - 1) * p.ad.a_adapter[s] + (p.ad.rank - 1) * p.ad.a_row[s] + p.ad.cols};
}
__device__ __forceinline__ Extent extent_b(const ApplyArgs& p, int s) {
  return {static_cast<const uint16_t*>(p.ad.B[s]),
          (p.ad.n - 1) * p.ad.b_adapter[s] + (p.ad.rows[s] - 1) * p.ad.b_row[s] + p.ad.rank};
}

__device__ __forceinline__ int off_of(const uint16_t* p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15) / 2; }

// Elements off .. off + 7 of the two neighbouring 16-byte words, the first `have`
// of them.
__device__ __forceinline__ uint4 shift_unit(const uint4& lo, const uint4& hi, int off, int have) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = off & 4 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = off & 2 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = have - 2 * i;
    const uint32_t v = __funnelshift_r(w[i], w[i + 1], 16 * (off & 1));
    w[i] = left >= 2 ? v : left == 1 ? v & 0xffffu : 0u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether the two 16-byte words that the 8 elements at `from` lie across are in
// the matrix.
__device__ __forceinline__ bool words_inside(const Extent& m, const uint16_t* from) {
  const int64_t at = from - m.first - off_of(from);
  return at >= 0 && at + 16 <= m.size;
}

// Eight elements of a row, the first `have` of them wanted, on their way to a
// 16-byte unit of shared memory.  A row that is not aligned to 16 bytes comes as
// the two 16-byte words that each of its units lies across, to `to` and `to +
// second`, and is shifted when it is read back (take_raw).  Where a word would
// leave the matrix (at its two ends), the elements come one by one.
__device__ __forceinline__ void copy_raw(const Extent& m, unsigned char* to, const uint16_t* from, int have, int second) {
  if (have <= 0) return;
  const int off = off_of(from);
  if (words_inside(m, from)) {
    copy16(to, from - off, 16);
    copy16(to + second, from - off + 8, 16);
  } else {
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < have ? from[i] : (uint16_t)0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint16_t*>(to + (off + i >= 8 ? second - 16 : 0) + 2 * (off + i)) = e[i];
  }
}

// The same where both words are known to lie in the matrix.
__device__ __forceinline__ void copy_raw_inside(unsigned char* to, const uint16_t* from, int second) {
  const uint16_t* at = from - off_of(from);
  copy16(to, at, 16);
  copy16(to + second, at + 8, 16);
}

__device__ __forceinline__ uint4 take_raw(const unsigned char* at, int second, int off, int have) {
  const uint4 lo = *reinterpret_cast<const uint4*>(at), hi = *reinterpret_cast<const uint4*>(at + second);
  if (have >= 8) return shift_unit(lo, hi, off, 8);
  return shift_unit(lo, hi, off, have);
}

// The same at once, into registers.
__device__ __forceinline__ uint4 load_unit(const Extent& m, const uint16_t* from, int have) {
  if (have <= 0) return make_uint4(0u, 0u, 0u, 0u);
  const int off = off_of(from);
  if (words_inside(m, from)) {
    const uint4* at = reinterpret_cast<const uint4*>(from - off);
    return shift_unit(at[0], at[1], off, have);
  }
  uint16_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < have ? from[i] : (uint16_t)0;
  return make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                    e[6] | (uint32_t)e[7] << 16);
}

// In a checked build: `have` elements from `at` on if they lie in the matrix that
// the call describes, else none and the flag; otherwise `have`.
__device__ __forceinline__ int checked(const Extent& m, const uint16_t* at, int have) {
  SEEDLM_CHECK_ONLY(const int64_t i = at - m.first;
                    if (have > 0 && (i < 0 || !SEEDLM_IN_BOUNDS(g_check_flag, i + have - 1, m.size))) return 0;)
  return have;
}
// Whether outputs at .. at + n - 1 of base or Y lie in it.
__device__ __forceinline__ bool checked_y(const ApplyArgs& p, const float* at, const float* of, int64_t ld, int n) {
  SEEDLM_CHECK_ONLY(const int64_t i = at - of; const int64_t width = p.slice_at[p.ad.slices - 1] + p.ad.rows[p.ad.slices - 1];
                    if (i < 0 || !SEEDLM_IN_BOUNDS(g_check_flag, i + n - 1, (p.M - 1) * ld + width)) return false;)
  return true;
}

// ---- the first kernel's end: the cluster's sums to S

__device__ __forceinline__ float2 load_of_cta(const float* mine, uint32_t cta) {
  uint32_t at;
  float2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(cta));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

template <bool BF16>
__device__ __forceinline__ void split(float v, uint16_t (&part)[3]) {
  if constexpr (BF16) {
    const uint32_t b0 = __float_as_uint(v) & 0xffff0000u;
    const float r1 = finite(v) ? v - __uint_as_float(b0) : 0.f;
    const uint32_t b1 = __float_as_uint(r1) & 0xffff0000u;
    const uint32_t b2 = __float_as_uint(r1 - __uint_as_float(b1));
    part[0] = finite(v) ? (uint16_t)(b0 >> 16) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
    part[1] = (uint16_t)(b1 >> 16);
    part[2] = (uint16_t)(b2 >> 16);
  } else {
    const __half h0 = __float2half_rn(v);
    const float r1 = finite(v) ? v - __half2float(h0) : 0.f;
    part[0] = __half_as_ushort(h0);
    part[1] = __half_as_ushort(__float2half_rn(r1));
    part[2] = 0;
  }
}

// sums[row][stride] of every CTA of the cluster, added in order and scaled, to
// S: slots slot0 .. slot0 + N of the slices laid end to end.  The CTAs take the
// rows in turn, a warp a row, a lane two neighbouring slots.
template <bool BF16, int N>
__device__ __forceinline__ void store_sums(const ApplyArgs& p, const float* sums, int stride, int first, int count,
                                           int rank, int slot0, float scale) {
  constexpr int P = kParts<BF16>;
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32, ctas = (int)cluster_size();
  SEEDLM_CHECK_ONLY(const int64_t extent = (int64_t)p.M * p.ad.slices * P * p.slots;)
  cluster_sync();
  for (int i = (int)cluster_rank() + ctas * (threadIdx.x / 32); i < count; i += ctas * warps)
#pragma unroll
    for (int j0 = 0; j0 < N; j0 += 64) {
      const int j = j0 + 2 * lane;
      const int slot = slot0 + j, s = slot / p.slots, r = slot - s * p.slots;
      const bool in = j < N && s < p.ad.slices;
      float2 v = make_float2(0.f, 0.f), part[kMaxSplits];
#pragma unroll
      for (int c = 0; c < kMaxSplits; ++c)  // all on their way together
        if (in && c < ctas) part[c] = load_of_cta(sums + i * stride + j, c);
#pragma unroll
      for (int c = 0; c < kMaxSplits; ++c)
        if (in && c < ctas) v = make_float2(v.x + part[c].x, v.y + part[c].y);
      // Beyond the adapter's rank rows of zeros met x, which gives NaN where x
      // has infinities.
      v = make_float2(r < rank ? v.x * scale : 0.f, r + 1 < rank ? v.y * scale : 0.f);
      float up = 1.f;
      if constexpr (!BF16) {
        float top = fmaxf(finite(v.x) ? fabsf(v.x) : 0.f, finite(v.y) ? fabsf(v.y) : 0.f);
#pragma unroll
        for (int o = 1; o < 32; o *= 2)
          if (2 * o < p.slots) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^e with e = 14 - floor(log2 top), at most 126 (top below 2^-112).
        const int e = top > 0.f ? min(126, 14 - ((int)(__float_as_uint(top) >> 23) - 127)) : 0;
        up = __uint_as_float((uint32_t)(e + 127) << 23);
        if (in && r % 64 == 0)
          p.unscale[((int64_t)(first + i) * p.ad.slices + s) * p.blocks + r / 64] =
              __uint_as_float((uint32_t)(127 - e) << 23);
      }
      uint16_t lo[3], hi[3];
      split<BF16>(v.x * up, lo);
      split<BF16>(v.y * up, hi);
      const int64_t to = ((int64_t)(first + i) * p.ad.slices + s) * P * p.slots + r;
#pragma unroll
      for (int w = 0; w < P; ++w)
        if (in && SEEDLM_IN_BOUNDS(g_check_flag, to + w * p.slots + 1, extent))
          *reinterpret_cast<uint32_t*>(p.S + to + w * p.slots) = lo[w] | (uint32_t)hi[w] << 16;
    }
  cluster_sync();  // no CTA leaves while another reads its sums
}

// S for low tiles (8 rows): bound by reading A.  A cluster takes one tile and
// 16 RB ranks of one slice, each of its CTAs one part of the columns and each
// warp 32 columns of that at a time.  Each warp keeps a ring of its next steps
// coming into shared memory; a lane copies exactly what it will itself read, so
// the ring needs no barrier.  64 rows with adapters of their own, rank 64, two
// slices of 8192 columns: 135 MB in 31 us (4.4 TB/s).  Rows that are not aligned to
// 16 bytes come raw, two words for each unit: their ring (123 kB for 32 slots, 184
// for 64) leaves one CTA on an SM, and 333 rows of 4099 columns (392 CTAs, four or
// five steps for a warp) take 20 us in three rounds.
template <int RB>
constexpr int kShrinkLowStages = RB == 4 ? 5 : 6;
template <int RB, bool WIDE>
constexpr int kShrinkLowSmem = kLowWarps * kShrinkLowStages<RB> * (2 * RB + 1) * (WIDE ? 512 : 1024);

template <bool BF16, int RB, bool WIDE>
__global__ void __launch_bounds__(32 * kLowWarps)
adapters_shrink_low_kernel(const __grid_constant__ ApplyArgs p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kStages = kShrinkLowStages<RB>, kUnit = WIDE ? 512 : 1024, R = RB * 16;
  constexpr int kStageBytes = (2 * RB + 1) * kUnit;
  grid_wait();
  // After the wait: what ran before this kernel is then complete for the next
  // one too, which reads the plan, B and base before its own wait.
  grid_launch_dependents();
  const int cluster = blockIdx.x / (int)cluster_size();
  const int group = cluster % p.groups, s = cluster / p.groups % p.ad.slices, t = cluster / (p.groups * p.ad.slices);
  const int4 tile = plan_tile(p, t), head = plan_head(p);
  if (t >= head.z) return;
  const int a = tile.x, first = tile.y, count = tile.z;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  // Asked for, at places that there are, before the tile is looked at (37 rows, 20
  // adapters, q, k, v of 4096 columns: 9.0 us, 9.2 after it).
  const int named = __ldcg(p.plan + min((unsigned)first + g, (unsigned)p.M - 1));
  const int some = (int)min((unsigned)a, (unsigned)p.ad.n - 1);
  const int r0 = group * R, rank = rank_of(p.ad, some) - r0;  // of this group
  const float scale = p.ad.scales ? __ldcg(p.ad.scales + some) : 1.f;
  if (!tile_fits(p, tile, kLowRows, 0)) return;  // the same in all CTAs of a cluster
  const int row = g < count ? row_of(p, named) : -1;
  if (rank <= 0 || p.ad.rows[s] == 0) return;
  const int k0 = (int)cluster_rank() * p.split_cols, k1 = min(p.ad.cols, k0 + p.split_cols);
  const int blocks = min(RB, (rank + 15) / 16);

  // Row g of the tile and rows 8 j + g of A, at this lane's place in the part.
  const int64_t a_row = p.ad.a_row[s];
  const bool have_x = row >= 0;
  const int k_first = k0 + warp * kStep + 8 * q;
  const uint16_t* x = p.X + (have_x ? row * p.ldx : 0) + k_first;
  const uint16_t* A = static_cast<const uint16_t*>(p.ad.A[s]) + a * p.ad.a_adapter[s] + r0 * a_row + k_first;
  unsigned char* ring = smem + warp * kStages * kStageBytes + lane * 16;
  if (!SEEDLM_IN_BOUNDS(g_check_flag, (kShrinkLowSmem<RB, WIDE>)-1, seedlm_dynamic_smem_bytes())) return;
  const int steps = k1 > k0 ? max(0, ((k1 - k0 + kStep - 1) / kStep - warp + kLowWarps - 1) / kLowWarps) : 0;
  // Every copy of a step is made, those of rows that are not there with no
  // bytes read and zeros written, so what is multiplied below needs no checks;
  // rows that are not aligned to 16 bytes come raw and are cut to size there.
  int k = k_first, fetched = 0;
  unsigned char* to = ring;
  auto fetch = [&]() {
    if (fetched < steps) {
      const int have = max(0, min(8, k1 - k));
      if (WIDE) {
#pragma unroll
        for (int b = 0; b < RB; ++b)
          if (b < blocks) {
#pragma unroll
            for (int j = 2 * b; j < 2 * b + 2; ++j) {
              const int r = 8 * j + g;
              copy16(to + j * kUnit, A + (r < rank ? r : 0) * a_row, 2 * checked(extent_a(p, s), A + r * a_row, r < rank ? have : 0));
            }
          }
        copy16(to + 2 * RB * kUnit, x, 2 * checked(extent_x(p), x, have_x ? have : 0));
      } else if (k >= 8 && k + 16 <= p.ad.cols) {
#pragma unroll 2
        for (int j = 0; j < 2 * blocks; ++j)
          if (checked(extent_a(p, s), A + (8 * j + g) * a_row, 8 * j + g < rank ? 8 : 0))
            copy_raw_inside(to + j * kUnit, A + (8 * j + g) * a_row, 512);
        if (checked(extent_x(p), x, have_x ? 8 : 0)) copy_raw_inside(to + 2 * RB * kUnit, x, 512);
      } else {
#pragma unroll 1
        for (int j = 0; j < 2 * blocks; ++j) {
          const int r = 8 * j + g;
          copy_raw(extent_a(p, s), to + j * kUnit, A + r * a_row, checked(extent_a(p, s), A + r * a_row, r < rank ? have : 0), 512);
        }
        copy_raw(extent_x(p), to + 2 * RB * kUnit, x, checked(extent_x(p), x, have_x ? have : 0), 512);
      }
      A += kLowWarps * kStep;
      x += kLowWarps * kStep;
      k += kLowWarps * kStep;
      to = to == ring + (kStages - 1) * kStageBytes ? ring : to + kStageBytes;
      ++fetched;
    }
    copies_commit();
  };
  int off[2 * RB + 1], read_k = k_first;
  if (!WIDE) {
#pragma unroll
    for (int j = 0; j < 2 * RB; ++j) off[j] = off_of(A + (8 * j + g) * a_row);
    off[2 * RB] = off_of(x);
  }
  for (int i = 0; i < kStages - 1; ++i) fetch();
  // The tensor cores cut off what an addition leaves below the sum's last bit, so
  // they only add up 8 steps; those sums are added in fp32, rounded.
  float acc[RB][4] = {}, total[RB][4] = {};
  const unsigned char* from = ring;
  for (int step = 0; step < steps; ++step) {
    copies_wait<kStages - 2>();
    const int have = max(0, min(8, k1 - read_k));
    const unsigned char* x_at = from + 2 * RB * kUnit;
    const uint4 v = WIDE ? *reinterpret_cast<const uint4*>(x_at) : take_raw(x_at, 512, off[2 * RB], have_x ? have : 0);
    uint4 w[2 * RB];
#pragma unroll
    for (int b = 0; b < RB; ++b)
      if (b < blocks) {
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j)
          w[j] = WIDE ? *reinterpret_cast<const uint4*>(from + j * kUnit)
                      : take_raw(from + j * kUnit, 512, off[j], 8 * j + g < rank ? have : 0);
      }
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (b < blocks) mma_half<BF16>(half, acc[b], w[2 * b], w[2 * b + 1], v);
    if (step % 8 == 7 || step == steps - 1)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          total[b][e] += acc[b][e];
          acc[b][e] = 0.f;
        }
    read_k += kLowWarps * kStep;
    from = from == ring + (kStages - 1) * kStageBytes ? ring : from + kStageBytes;
    fetch();
  }
  // The warps' sums, [rank][9] (rows of 9 keep the reads off each other's
  // banks), added in order into [row][R], all over the rings.
  float* red = reinterpret_cast<float*>(smem);
  float* sums = red + kLowWarps * R * 9;
  static_assert((kLowWarps * R * 9 + 8 * R) * 4 <= kShrinkLowSmem<RB, WIDE>, "the sums lie over the rings");
  copies_wait<0>();
  __syncthreads();
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[(warp * R + 16 * b + 8 * (e / 2) + g) * 9 + 2 * q + e % 2] = total[b][e];
  __syncthreads();
  for (int e = threadIdx.x; e < R * count; e += 32 * kLowWarps) {
    const int r = e % R, i = e / R;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kLowWarps; ++w) sum += red[(w * R + r) * 9 + i];
    sums[i * R + r] = sum;
  }
  store_sums<BF16, R>(p, sums, R, first, count, r0 + rank, s * p.slots + r0, scale);
}

// S for tall tiles (64 rows) on tcgen05.mma: a cluster takes one tile and 128
// slots of the slices laid end to end (rows of A, the 128-row operand), each of
// its CTAs one part of the columns, 64 at a time through a ring of shared-memory
// stages.  Bound by the traffic from L2 (A again for every tile) and its latency:
// 4096 rows, eight adapters of rank 64, two slices of 8192 columns: 200 MB in 28
// us, 57 with the same products on mma.sync.  The tensor
// cores cut off what an addition leaves below a sum's last bit, so the stages go
// to four sums in turn, which after every 32 stages are added up in fp32, rounded.
// Rows that are not aligned to 16 bytes (not WIDE) come raw, two words for each
// unit of 8 elements, and each thread shifts what it copied into place when it is
// there.
template <bool WIDE>
struct ShrinkTallLayout {
  static constexpr int kThreads = 256, kStages = WIDE ? 4 : 2, kCols = 64, kSlots = 128, kSums = 4, kFlush = 32;
  static constexpr int kStageBytes = (kSlots + kTall) * 128;   // rows of A, then rows of X
  static constexpr int kAhead = 3;                             // stages of copies on their way
  static constexpr int kRawBytes = (kSlots + kTall) * 8 * 32;  // two words for each unit
  static constexpr int kRaw = kStages * kStageBytes;
  static constexpr int kBars = kRaw + (WIDE ? 0 : kAhead * kRawBytes);  // a stage's products are done
  static constexpr int kBytes = kBars + kStages * 8 + 8;       // tensor memory's address, give-up flag
  static constexpr int kColumns = kSums * kTall;
  static constexpr int kSumStride = kSlots + 4;
};
// A product of one tile takes microseconds; a wait this long never ends.
constexpr uint64_t kTallWaitLimit = 2000000000ull;

template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(ShrinkTallLayout<WIDE>::kThreads, WIDE ? 2 : 1)
adapters_shrink_tall_kernel(const __grid_constant__ ApplyArgs p) {
  using L = ShrinkTallLayout<WIDE>;
  static_assert(kTall * L::kSumStride * 4 <= L::kBars, "the sums lie over the stages");
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t bars = tc::smem_u32(smem + L::kBars);
  volatile uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::kBars + L::kStages * 8);
  // Tensor memory before the next kernel may start: one that takes all of it and
  // then waits for this one must not come first.
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(smem + L::kBars + L::kStages * 8), L::kColumns);
  if (tid == 32) {
    for (int i = 0; i < L::kStages; ++i) tc::mbar_init(bars + 8 * i, 1);
    tc::fence_mbar_init();
    slot[1] = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = slot[0];
  grid_wait();
  grid_launch_dependents();  // after the wait, as above
  const int cluster = blockIdx.x / (int)cluster_size();
  const int group = cluster % p.groups, t = cluster / p.groups;
  const int4 tile = plan_tile(p, t), head = plan_head(p);
  bool ok = true;
  if (t < head.z && tile_fits(p, tile, kTall, 0)) {  // the same in all CTAs of a cluster
    const int a = tile.x, first = tile.y, count = tile.z;
    const int rank = rank_of(p.ad, a);
    const int k0 = (int)cluster_rank() * p.split_cols, k1 = min(p.ad.cols, k0 + p.split_cols);
    const int steps = k1 > k0 ? (k1 - k0 + L::kCols - 1) / L::kCols : 0;

    // This thread's rows of every stage: unit `unit` of rows row0, row0 + kApart,
    // ... of A (the first 128) and X (the others).  Rows that are not there are
    // zeroed once in all stages and not copied.
    constexpr int kApart = L::kThreads / 8, kMine = (L::kSlots + kTall) / kApart;
    const int unit = tid % 8, row0 = tid / 8;
    const int place = row0 * 128 + (unit ^ (row0 & 7)) * 16;
    constexpr int kRaw2 = L::kThreads * 32;  // raw words of one of a thread's rows, all threads
    const uint16_t* src[kMine];
    unsigned there = 0;
    // The row's first element; null: no such row.
    auto row_at = [&](int i) -> const uint16_t* {
      const int row = row0 + kApart * i;
      if (row < L::kSlots) {
        const int place_of = group * L::kSlots + row, s = place_of / p.slots, r = place_of - s * p.slots;
        if (s >= p.ad.slices || r >= rank || p.ad.rows[s] == 0) return nullptr;
        return static_cast<const uint16_t*>(p.ad.A[s]) + a * p.ad.a_adapter[s] + r * p.ad.a_row[s];
      }
      const int m = row - L::kSlots < count ? plan_row(p, first + row - L::kSlots) : -1;
      return m >= 0 ? p.X + m * p.ldx : nullptr;
    };
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      src[i] = row_at(i);
      there |= (unsigned)(src[i] != nullptr) << i;
      if (!src[i])
        for (int st = 0; st < L::kStages; ++st)
          *reinterpret_cast<uint4*>(smem + st * L::kStageBytes + i * kApart * 128 + place) = make_uint4(0u, 0u, 0u, 0u);
    }
    auto extent_of = [&](int i) {
      return kApart * i < L::kSlots ? extent_a(p, (group * L::kSlots + row0 + kApart * i) / p.slots) : extent_x(p);
    };
    const uint32_t to_stages = tc::smem_u32(smem) + place;
    auto fetch = [&](int step, int st) {
      if (step < steps) {
        const int k = k0 + step * L::kCols + 8 * unit, have = max(0, min(8, k1 - k));
        if (WIDE) {
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            int wanted = have;
            SEEDLM_CHECK_ONLY(if (there >> i & 1) wanted = checked(extent_of(i), src[i] + k, have);)
            copy16_if(there & 1u << i, to_stages + st * L::kStageBytes + i * kApart * 128, src[i] + k, 2 * wanted);
          }
        } else {
          unsigned char* to = smem + L::kRaw + step % L::kAhead * L::kRawBytes + tid * 16;
          if (k >= 8 && k + 16 <= p.ad.cols) {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
              if ((there >> i & 1) && checked(extent_of(i), src[i] + k, 8)) copy_raw_inside(to + i * kRaw2, src[i] + k, kRaw2 / 2);
          } else {
#pragma unroll 1
            for (int i = 0; i < kMine; ++i)
              if (there >> i & 1) {
                const uint16_t* from = row_at(i) + k;
                copy_raw(extent_of(i), to + i * kRaw2, from, checked(extent_of(i), from, have), kRaw2 / 2);
              }
          }
        }
      }
      copies_commit();
    };
    for (int i = 0; i < L::kAhead; ++i) fetch(i, i);
    const uint32_t idesc = tc::idesc_f16(kTall, BF16 ? 1 : 0);
    auto wait_for = [&](int step) {
      ok = tc::mbar_wait_or_abort(bars + 8 * (step % L::kStages), (step / L::kStages) & 1, kTallWaitLimit, slot + 1) && ok;
    };
    // Of slot tid % 128, rows kHalf (tid / 128) on.
    constexpr int kHalf = kTall * L::kSlots / L::kThreads;
    const int row1 = tid / L::kSlots * kHalf;
    float total[kHalf] = {};
    // The stages are spelled out, so that a copy is an address and a predicate: with
    // few warps to a scheduler the instructions of a step are its time (2750 rows,
    // 14336 columns, four adapters of rank 8, both products: 53.5 us; 62.4 with
    // 128 threads, a branch to a copy and a loop over the stages).
    constexpr int kTurns = WIDE ? L::kStages : 1;
    for (int step0 = 0; step0 < steps; step0 += kTurns) {
#pragma unroll
      for (int u = 0; u < kTurns; ++u) {
        const int step = step0 + u;
        if (step >= steps) break;
        const int st = WIDE ? u : step % L::kStages;
        copies_wait<L::kAhead - 1>();
        if (!WIDE) {
          if (step >= L::kStages) wait_for(step - L::kStages);  // the stage is free
          const int k = k0 + step * L::kCols + 8 * unit, have = max(0, min(8, k1 - k));
          const unsigned char* raw = smem + L::kRaw + step % L::kAhead * L::kRawBytes + tid * 16;
          unsigned char* to = smem + st * L::kStageBytes + place;
#pragma unroll
          for (int i = 0; i < kMine; ++i)
            if (there >> i & 1)
              *reinterpret_cast<uint4*>(to + i * kApart * 128) = take_raw(raw + i * kRaw2, kRaw2 / 2, off_of(src[i]), have);
        }
        tc::fence_proxy_async();
        __syncthreads();
        if (warp == 0) {
          tc::fence_after_sync();
          const int turn = step % L::kFlush;
          const uint64_t w = tc::smem_desc_sw128(tc::smem_u32(smem + st * L::kStageBytes));
          const uint64_t x = w + L::kSlots * 128 / 16;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f16_ss_warp(tmem + turn % L::kSums * kTall, w + 2 * k, x + 2 * k, idesc, turn >= L::kSums || k > 0);
          tc::mma_commit_warp(bars + 8 * st);
        }
        // The stage before this one is read: its place takes the step after next.
        if (WIDE && step > 0) wait_for(step - 1);
        fetch(step + L::kAhead, (u + L::kAhead) % L::kStages);
      }
      const int last = min(steps, step0 + kTurns) - 1;
      if (last % L::kFlush == L::kFlush - 1 || last == steps - 1) {
        wait_for(last);
        tc::fence_after_sync();
#pragma unroll
        for (int j = 0; j < L::kSums; ++j) {
          if (j > last % L::kFlush) break;
#pragma unroll
          for (int c = 0; c < kHalf / 16; ++c) {
            float d[16];
            tc::tmem_ld16(tmem + ((uint32_t)(32 * (warp % 4)) << 16) + j * kTall + row1 + 16 * c, d);
#pragma unroll
            for (int r = 0; r < 16; ++r) total[16 * c + r] += d[r];
          }
        }
        tc::fence_before_sync();
      }
    }
    copies_wait<0>();
    __syncthreads();  // the stages are read by all: the sums go over them
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int r = 0; r < kHalf; ++r) sums[(row1 + r) * L::kSumStride + tid % L::kSlots] = total[r];
    store_sums<BF16, L::kSlots>(p, sums, L::kSumStride, first, count, rank, group * L::kSlots,
                                p.ad.scales ? __ldcg(p.ad.scales + a) : 1.f);
  }
  if (!ok && lane == 0) atomicOr(&g_wait_error, 1u);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kColumns);
  }
}

// ---- the second kernel

// A lane's four outputs of one row: to = from + d.
__device__ __forceinline__ void add4_slow(const ApplyArgs& p, float* to, const float* from, float4 d, int left) {
  if (left <= 0 || !checked_y(p, to, p.Y, p.ldy, min(left, 4)) || !checked_y(p, from, p.base, p.ldb, min(left, 4))) return;
  const float dv[4] = {d.x, d.y, d.z, d.w};
  float b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = j < left ? __ldcg(from + j) : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) to[j] = b[j] + dv[j];
}

// Y = base + S B_a^T.  A CTA takes one tile of rows and a chunk of one slice's
// outputs; a warp takes 32 outputs at a time, of which lane (g, q) holds
// outputs 4g .. 4g + 3 of rows 2q and 2q + 1 of every 8: the rows 4g + j of B
// are dealt to the two 16-row operands so that base and Y are read and written
// 16 bytes a lane, 128 bytes a row.
//
// What a kernel reads besides S does not depend on the first kernel (which let
// this one start only after everything before it had completed), so it is
// requested before the wait for S.

struct ExpandTile {
  int a, first, count, rank, s, c0, c1;
};

// False if this CTA has nothing to do.
__device__ __forceinline__ bool expand_tile(const ApplyArgs& p, int chunks, int in_place, ExpandTile& x) {
  const int t = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int4 tile = plan_tile(p, t), head = plan_head(p);
  if (t >= (in_place ? head.z : head.w) || !tile_fits(p, tile, kLowRows, -1)) return false;
  x.a = tile.x;
  x.first = tile.y;
  x.count = tile.z;
  x.rank = rank_of(p.ad, x.a);
  if (in_place && x.rank == 0) return false;
  x.s = 0;
  while (chunk >= p.chunk_first[x.s + 1]) ++x.s;
  x.c0 = (chunk - p.chunk_first[x.s]) * p.chunk_rows;
  x.c1 = min(p.ad.rows[x.s], x.c0 + p.chunk_rows);
  return true;
}

// Low tiles (8 rows): bound by reading B.  Each warp keeps a ring of its next
// outputs' rows of B and of base coming into shared memory, each lane copying
// what it will itself read, and takes S straight into registers.  An item of
// the ring is 32 outputs and a block of up to 64 ranks (32 KC); the last of an
// output's items brings base.  64 rows with adapters of their own, rank 64,
// 57344 outputs: 500 MB in 87 us (5.7 TB/s).
constexpr int kLowStages = 3;
template <int KC, bool WIDE>
constexpr int kLowItemBytes = 2048 * KC * (WIDE ? 1 : 2) + 1024;
template <int KC, bool WIDE>
constexpr int kExpandLowSmem = kLowWarps * kLowStages * kLowItemBytes<KC, WIDE>;

template <bool BF16, int KC, bool MANY, bool WIDE>
__global__ void __launch_bounds__(32 * kLowWarps)
adapters_expand_low_kernel(const __grid_constant__ ApplyArgs p, int chunks, int in_place) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int P = kParts<BF16>, kItemBytes = kLowItemBytes<KC, WIDE>, kRound = 32 * kLowWarps;
  grid_launch_dependents();
  ExpandTile x;
  if (!expand_tile(p, chunks, in_place, x)) {
    grid_wait();
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  unsigned char* ring = smem + warp * kLowStages * kItemBytes + lane * 16;
  const uint16_t* B = static_cast<const uint16_t*>(p.ad.B[x.s]) + max(x.a, 0) * p.ad.b_adapter[x.s];
  const int64_t b_row = p.ad.b_row[x.s];
  const bool vec_y = p.grain_y[x.s] == 16;
  const bool eights = p.grain_b[x.s] >= 8;  // rows of B that 8-byte copies can fetch
  const float* from[2];
  float* to[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int m = 2 * q + e < x.count ? plan_row(p, x.first + 2 * q + e) : -1;
    const bool ok = m >= 0;
    from[e] = ok ? p.base + m * p.ldb + p.slice_at[x.s] + 4 * g : nullptr;
    to[e] = ok ? p.Y + m * p.ldy + p.slice_at[x.s] + 4 * g : nullptr;
  }
  const int groups = MANY ? max(1, (x.rank + 63) / 64) : 1;
  const int first_n = x.c0 + 32 * warp;
  const int items = first_n < x.c1 ? (x.c1 - first_n + kRound - 1) / kRound * groups : 0;
  // The item to be fetched next: its outputs and its ranks.  As above, every
  // copy of B is made, with no bytes where there is nothing to read.
  const uint16_t* b_next = B + (first_n + 4 * g) * b_row + 8 * q;
  int fetch_n = first_n, fetch_k = 0, fetched = 0;
  unsigned char* into = ring;
  int have[KC];
  auto sizes = [&]() {
#pragma unroll
    for (int c = 0; c < KC; ++c) have[c] = max(0, min(8, x.rank - fetch_k - kStep * c - 8 * q));
  };
  sizes();
  auto fetch = [&]() {
    if (fetched < items) {
      const bool whole = fetch_n + 32 <= x.c1;
      if (MANY) sizes();
      const uint16_t* b = b_next;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = fetch_n + 4 * g + j;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          unsigned char* to = into + (4 * c + j) * 512;
          const uint16_t* from = b + kStep * c;
          const int wanted = checked(extent_b(p, x.s), from, whole || n < x.c1 ? have[c] : 0);
          if (WIDE) {
            copy16_short(to, from, 2 * wanted);
          } else if (eights) {
            copy_small<8>(to, from, max(0, min(8, 2 * wanted)));
            copy_small<8>(to + 8, from + 4, max(0, 2 * wanted - 8));
          } else {
            copy_raw(extent_b(p, x.s), to, from, wanted, 2048 * KC);
          }
        }
        b += b_row;
      }
      b_next += 64;
      fetch_k += 64;
      if (!MANY || fetch_k >= x.rank) {  // the last ranks of these outputs
        if (whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (from[e] && checked_y(p, from[e] + fetch_n, p.base, p.ldb, 4)) {
              unsigned char* to = into + kItemBytes - 1024 + e * 512;
              if (vec_y) {
                copy16(to, from[e] + fetch_n, 16);
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) copy_small<4>(to + 4 * j, from[e] + fetch_n + j, 4);
              }
            }
        }
        b_next += kRound * b_row - 64 * groups;
        fetch_n += kRound;
        fetch_k = 0;
      }
      into = into == ring + (kLowStages - 1) * kItemBytes ? ring : into + kItemBytes;
      ++fetched;
    }
    copies_commit();
  };
  for (int i = 0; i < kLowStages - 1; ++i) fetch();
  grid_wait();
  // Row g of S and its factors; rows that are not there, and rank 0, are zero.
  const int64_t s_row = (int64_t)(x.first + g) * p.ad.slices + x.s;
  const uint16_t* S = p.S + s_row * P * p.slots + 8 * q;
  uint4 v[KC][P];
  auto load_s = [&](int k) {
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int pt = 0; pt < P; ++pt)
        v[c][pt] = g < x.count && k + kStep * c < x.rank
                       ? __ldcg(reinterpret_cast<const uint4*>(S + pt * p.slots + k + kStep * c))
                       : make_uint4(0u, 0u, 0u, 0u);
  };
  float f[2] = {1.f, 1.f};
  auto load_f = [&](int k) {
    if constexpr (!BF16) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * q + e < x.count && k < x.rank)
          f[e] = __ldcg(p.unscale + ((int64_t)(x.first + 2 * q + e) * p.ad.slices + x.s) * p.blocks + k / 64);
    }
  };
  load_s(0);
  load_f(0);
  float total[2][4] = {};
  int n0 = first_n, k = 0;
  const unsigned char* item_at = ring;
  for (int item = 0; item < items; ++item) {
    if (MANY) {
      load_s(k);
      load_f(k);
    }
    copies_wait<kLowStages - 2>();
    float acc[P][2][4] = {};
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      if (k + kStep * c >= x.rank) break;
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned char* at = item_at + (4 * c + j) * 512;
        const int n = n0 + 4 * g + j, r = k + kStep * c + 8 * q;
        w[j] = WIDE || eights ? *reinterpret_cast<const uint4*>(at)
                              : take_raw(at, 2048 * KC, off_of(B + n * b_row + r), n < x.c1 ? max(0, min(8, x.rank - r)) : 0);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int pt = 0; pt < P; ++pt) {
          mma_half<BF16>(half, acc[pt][0], w[0], w[1], v[c][pt]);
          mma_half<BF16>(half, acc[pt][1], w[2], w[3], v[c][pt]);
        }
    }
    // The parts from the smallest on, then the blocks before this one.
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float sum = acc[P - 1][b][e];
#pragma unroll
        for (int pt = P - 2; pt >= 0; --pt) sum += acc[pt][b][e];
        total[b][e] = fmaf(sum, f[e % 2], total[b][e]);
      }
    k += 64;
    if (!MANY || k >= x.rank) {
      const bool whole = n0 + 32 <= x.c1;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (!to[e]) continue;
        const float4 d = make_float4(total[0][e], total[0][2 + e], total[1][e], total[1][2 + e]);
        if (whole) {
          const float4 b = *reinterpret_cast<const float4*>(item_at + kItemBytes - 1024 + e * 512);
          if (!checked_y(p, to[e] + n0, p.Y, p.ldy, 4)) continue;
          if (vec_y) {
            *reinterpret_cast<float4*>(to[e] + n0) = make_float4(b.x + d.x, b.y + d.y, b.z + d.z, b.w + d.w);
          } else {
            to[e][n0] = b.x + d.x;
            to[e][n0 + 1] = b.y + d.y;
            to[e][n0 + 2] = b.z + d.z;
            to[e][n0 + 3] = b.w + d.w;
          }
        } else {
          add4_slow(p, to[e] + n0, from[e] + n0, d, x.c1 - n0 - 4 * g);
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) total[b][e] = 0.f;
      n0 += kRound;
      k = 0;
    }
    item_at = item_at == ring + (kLowStages - 1) * kItemBytes ? ring : item_at + kItemBytes;
    fetch();
  }
}

// Tall tiles (64 rows): bound by reading base and writing Y, so the products are
// left to tcgen05.mma: the tile's 64 rows by 256 outputs, in two of 128 (the even
// and the odd ones), every part of S against the same B, summed in tensor
// memory.  A thread takes two neighbouring outputs of all rows from there, so
// that a warp reads base and writes Y 256 bytes of a row at a time (measured on
// this pattern alone: 6.0 TB/s, against 5.5 with 128 bytes), 16 rows after
// another, and has always asked for the next 16 rows' base before it finishes
// with these.  B for the next 256 outputs arrives meanwhile: its one place is
// free as soon as the products are done.  Each CTA goes through its share of all
// (tile, slice, 256 outputs), in that order, fetching S once for a tile.  4096
// rows, eight adapters of rank 64, 57344 outputs: 338 us for 1.94 GB (5.7 TB/s);
// the products of the same tiles on mma.sync, with the parts of S read from
// shared memory by every warp, took 500.
//
// NB: blocks of 64 ranks; fp16 parts are scaled block by block, so there each
// block has a sum of its own.
constexpr int kTallOutputs = 256, kTallThreads = 128;

template <bool BF16, int NB>
struct TallLayout {
  static constexpr int P = kParts<BF16>;
  static constexpr int kSums = BF16 ? 1 : NB;               // of 2 x 64 columns of tensor memory each
  static constexpr int kColumns = kSums * 2 * kTall;
  static constexpr int kB = P * NB * kTall * 128;           // after S[P][NB][64 rows of 128 bytes]: B[2][NB][128 rows]
  static constexpr int kRows = kB + NB * kTallOutputs * 128;  // from_row, to_row
  static constexpr int kScales = kRows + 2 * kTall * 8;     // fp16: unscale[NB][64]
  static constexpr int kBars = kScales + (BF16 ? 0 : NB * kTall * 4);
  static constexpr int kBytes = kBars + 8 + 8;              // barrier, tensor memory's address, give-up flag
  static constexpr int kCtas = NB == 1 ? 3 : 1;             // on an SM
};
template <bool BF16, int NB, bool WIDE>
__global__ void __launch_bounds__(kTallThreads, NB == 1 ? 3 : 1)
adapters_expand_tall_kernel(const __grid_constant__ ApplyArgs p, int chunks, int in_place) {
  using L = TallLayout<BF16, NB>;
  constexpr int P = L::P, T = kTall, kOut = kTallOutputs, kQ = 16;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int64_t* from_row = reinterpret_cast<int64_t*>(smem + L::kRows);
  int64_t* to_row = from_row + T;
  float* unscale = reinterpret_cast<float*>(smem + L::kScales);
  const uint32_t done = tc::smem_u32(smem + L::kBars);
  volatile uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::kBars + 8);
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(smem + L::kBars + 8), L::kColumns);
  if (tid == 32) {
    tc::mbar_init(done, 1);
    tc::fence_mbar_init();
    slot[1] = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // Only now: a kernel after this one that takes all tensor memory and then
  // waits for this one must not come before this one has its own.
  grid_launch_dependents();
  const uint32_t tmem = slot[0];

  const int4 head = plan_head(p);
  const int64_t total = (int64_t)(in_place ? head.z : head.w) * chunks;
  int64_t item = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  // This thread's units of B and S: 16 bytes `unit` of rows row0, row0 + 16, ...
  const int unit = tid % 8, row0 = tid / 8;
  const int place = row0 * 128 + (unit ^ (row0 & 7)) * 16;
  uint32_t phase = 0;
  bool waited = false, ok = true;
  while (item < end) {
    // The items of one tile and slice.
    const int4 tile = plan_tile(p, item / chunks);
    const int a = tile.x, first = tile.y, count = tile.z;
    const int chunk = (int)(item % chunks);
    int s = 0;
    while (chunk >= p.chunk_first[s + 1]) ++s;
    const int items = (int)min(end - item, (int64_t)(p.chunk_first[s + 1] - chunk));
    item += items;
    if (!tile_fits(p, tile, T, -1)) continue;
    const int rank = rank_of(p.ad, a);
    if (in_place && rank == 0) continue;
    const int rows = p.ad.rows[s], c0 = (chunk - p.chunk_first[s]) * kOut;
    const uint16_t* B = static_cast<const uint16_t*>(p.ad.B[s]) + max(a, 0) * p.ad.b_adapter[s];
    const int64_t b_row = p.ad.b_row[s];
    const bool pairs = p.grain_y[s] >= 8;
    const bool products = rank > 0;
    __syncthreads();  // the tile before is done with shared memory
    bool wrong = false;
    if (tid < T) {
      const int m = tid < count ? plan_row(p, first + tid) : 0;
      wrong = m < 0;
      from_row[tid] = m * p.ldb + p.slice_at[s];
      to_row[tid] = m * p.ldy + p.slice_at[s];
    }
    // B of outputs c0 + 256 i + (0 .. 255): output 2 j + h is row j of half h, or,
    // where base and Y cannot be read in pairs, output 128 h + j.
    const int of_row = pairs ? 2 : 1, of_half = pairs ? 1 : 128;
    auto fetch = [&](int i) {
      const int n = c0 + i * kOut + of_row * row0;
      const uint16_t* src = B + n * b_row + 8 * unit;
      const int64_t b_rows = 16 * of_row * b_row, b_half = of_half * b_row;
      unsigned char* to = smem + L::kB + place;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int have = max(0, min(8, rank - 64 * b - 8 * unit));
        // Unit u: row j of half h, its place and its wanted elements.
        auto unit_of = [&](int u, unsigned char*& place_of, const uint16_t*& from) {
          const int j = u / 2, h = u % 2, at = n + 16 * of_row * j + of_half * h;
          place_of = to + (h * NB + b) * 128 * 128 + j * 16 * 128;
          from = src + 64 * b + j * b_rows + h * b_half;
          return checked(extent_b(p, s), from, at < rows ? have : 0);
        };
        unsigned char* at;
        const uint16_t* from;
        if (WIDE) {
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const int wanted = unit_of(u, at, from);
            copy16_short(at, from, 2 * wanted);
          }
        } else if (p.grain_b[s] >= 8) {
#pragma unroll 2
          for (int u = 0; u < 16; ++u) {
            const int wanted = unit_of(u, at, from);
            copy_small<8>(at, from, max(0, min(8, 2 * wanted)));
            copy_small<8>(at + 8, from + 4, max(0, 2 * wanted - 8));
          }
        } else {
#pragma unroll 1
          for (int u0 = 0; u0 < 16; u0 += 4) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int wanted = unit_of(u0 + u, at, from);
              v[u] = load_unit(extent_b(p, s), from, wanted);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              unit_of(u0 + u, at, from);
              *reinterpret_cast<uint4*>(at) = v[u];
            }
          }
        }
      }
      copies_commit();
    };
    if (products) fetch(0);
    if (!waited) grid_wait();
    waited = true;
    if (products) {
#pragma unroll
      for (int j = 0; j < T / 16; ++j) {
        const int i = row0 + 16 * j;
        const uint16_t* src = p.S + ((int64_t)(first + (i < count ? i : 0)) * p.ad.slices + s) * P * p.slots + 8 * unit;
#pragma unroll
        for (int pt = 0; pt < P; ++pt)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            copy16(smem + (pt * NB + b) * T * 128 + j * 16 * 128 + place, src + pt * p.slots + 64 * b,
                   i < count && 64 * b + 8 * unit < p.slots && 64 * b < rank ? 16 : 0);
      }
      if constexpr (!BF16)
        for (int u = tid; u < NB * T; u += kTallThreads) {
          const int i = u % T, b = u / T;
          unscale[u] = i < count && 64 * b < rank
                           ? __ldcg(p.unscale + ((int64_t)(first + i) * p.ad.slices + s) * p.blocks + b)
                           : 0.f;
        }
      copies_commit();
    }
    // The products of one item, by the first warp.
    auto multiply = [&]() {
      const uint32_t idesc = tc::idesc_f16(T, BF16 ? 1 : 0);
      const uint64_t w = tc::smem_desc_sw128(tc::smem_u32(smem + L::kB));
      const uint64_t v = tc::smem_desc_sw128(tc::smem_u32(smem));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t more = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t d = tmem + ((BF16 ? 0 : b) * 2 + h) * T;
          const int steps = min(4, (rank - 64 * b + 15) / 16);
          if (!BF16) more = 0;
          // The smallest parts first.
#pragma unroll
          for (int pt = P - 1; pt >= 0; --pt)
            for (int k = 0; k < steps; ++k) {
              tc::mma_f16_ss_warp(d, w + (uint64_t)((h * NB + b) * 128 * 128 / 16 + 2 * k),
                                  v + (uint64_t)((pt * NB + b) * T * 128 / 16 + 2 * k), idesc, more);
              more = 1;
            }
        }
      }
      tc::mma_commit_warp(done);
    };
    // Base of rows 16 q .. 16 q + 15 of item i, two outputs of each.  Base and Y
    // pass through L2 as what is first to leave it, so that B stays for the
    // adapter's other tiles (measured without: B came from memory every time).
    float2 ahead[kQ];
    auto ask = [&](int i, int q) {
      const int n = c0 + i * kOut + of_row * tid;
      const float* from = p.base + n;
      if (count >= kQ * (q + 1) && c0 + (i + 1) * kOut <= rows) {
        if (pairs) {
#pragma unroll
          for (int r = 0; r < kQ; ++r)
            if (checked_y(p, from + from_row[kQ * q + r], p.base, p.ldb, 2))
              ahead[r] = __ldcs(reinterpret_cast<const float2*>(from + from_row[kQ * q + r]));
        } else {
#pragma unroll
          for (int r = 0; r < kQ; ++r) {
            const float* at = from + from_row[kQ * q + r];
            if (checked_y(p, at, p.base, p.ldb, of_half + 1)) ahead[r] = make_float2(__ldcs(at), __ldcs(at + of_half));
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < kQ; ++r) {
          const float* at = from + from_row[kQ * q + r];
          const bool in = kQ * q + r < count;
          ahead[r].x = in && n < rows && checked_y(p, at, p.base, p.ldb, 1) ? __ldcg(at) : 0.f;
          ahead[r].y = in && n + of_half < rows && checked_y(p, at + of_half, p.base, p.ldb, 1) ? __ldcg(at + of_half) : 0.f;
        }
      }
    };
    copies_wait<0>();
    tc::fence_proxy_async();
    tc::fence_before_sync();  // of the sums before, read
    if (__syncthreads_or(wrong)) continue;  // (a plan that was written over)
    tc::fence_after_sync();
    if (products && warp == 0) multiply();
    ask(0, 0);
    for (int i = 0; i < items; ++i) {
      if (products) {
        ok = tc::mbar_wait_or_abort(done, phase, kTallWaitLimit, slot + 1) && ok;
        phase ^= 1;
        tc::fence_after_sync();
        if (i + 1 < items) fetch(i + 1);
      }
      const int n = c0 + i * kOut + of_row * tid;
      float* to = p.Y + n;
#pragma unroll
      for (int q = 0; q < T / kQ; ++q) {
        float2 v[kQ];
#pragma unroll
        for (int r = 0; r < kQ; ++r) v[r] = ahead[r];
        if (q + 1 < T / kQ) ask(i, q + 1);
        else if (i + 1 < items) ask(i + 1, 0);
        if (products)
#pragma unroll
          for (int b = 0; b < L::kSums; ++b) {
            float d0[kQ], d1[kQ];
            const uint32_t at = tmem + ((uint32_t)(32 * warp) << 16) + b * 2 * T + kQ * q;
            tc::tmem_ld16(at, d0);
            tc::tmem_ld16(at + T, d1);
            if (BF16 || 64 * b < rank)
#pragma unroll
              for (int r = 0; r < kQ; ++r) {
                const float f = BF16 ? 1.f : unscale[b * T + kQ * q + r];
                v[r] = BF16 ? make_float2(v[r].x + d0[r], v[r].y + d1[r])
                            : make_float2(fmaf(d0[r], f, v[r].x), fmaf(d1[r], f, v[r].y));
              }
          }
        if (!ok) continue;
        if (count >= kQ * (q + 1) && c0 + (i + 1) * kOut <= rows) {
          if (pairs) {
#pragma unroll
            for (int r = 0; r < kQ; ++r)
              if (checked_y(p, to + to_row[kQ * q + r], p.Y, p.ldy, 2))
                __stcs(reinterpret_cast<float2*>(to + to_row[kQ * q + r]), v[r]);
          } else {
#pragma unroll
            for (int r = 0; r < kQ; ++r) {
              float* at = to + to_row[kQ * q + r];
              if (!checked_y(p, at, p.Y, p.ldy, of_half + 1)) continue;
              __stcs(at, v[r].x);
              __stcs(at + of_half, v[r].y);
            }
          }
        } else {
#pragma unroll
          for (int r = 0; r < kQ; ++r) {
            float* at = to + to_row[kQ * q + r];
            const bool in = kQ * q + r < count;
            if (in && n < rows && checked_y(p, at, p.Y, p.ldy, 1)) at[0] = v[r].x;
            if (in && n + of_half < rows && checked_y(p, at + of_half, p.Y, p.ldy, 1)) at[of_half] = v[r].y;
          }
        }
      }
      if (products && i + 1 < items) {
        copies_wait<0>();
        tc::fence_proxy_async();
        tc::fence_before_sync();  // of this item's sums, read
        __syncthreads();
        tc::fence_after_sync();
        if (warp == 0) multiply();
      }
    }
  }
  if (!waited) grid_wait();
  if (!ok && lane == 0) atomicOr(&g_wait_error, 1u);
  copies_wait<0>();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::kColumns);
  }
}

}  // namespace

int64_t adapters_plan_words(int M, int n) {
  return plan_tail(M, n) + 4 * (2 + max_tiles(M, n, kLowRows) + max_tiles(M, n, kTall));
}

int launch_adapters_plan(int M, int n, const int32_t* ids, int32_t* plan, cudaStream_t stream, const DeviceInfo& dev) {
  int rc = allow_max_smem((const void*)adapters_plan_kernel, dev);
  if (rc) return rc;
  // One CTA up to 2048 rows; the cluster's two barriers cost more there than
  // its eight times as many threads save.
  const int ctas = M > kPlanOneCtaRows ? kPlanCtas : 1;
  const int most = M > n + 1 ? M : n + 1;
  const int threads = most >= kPlanThreads ? kPlanThreads : (most + 31) / 32 * 32;
  const int nwarps = threads / 32, bins = n + 1;
  const size_t smem = ((size_t)nwarps * bins + 5 * bins + 3 + 3 * 32) * sizeof(int32_t);
  return launch_pdl_cluster(adapters_plan_kernel, ctas, threads, smem, ctas, stream, M, n, ids, plan);
}

namespace {

// How the first product is shared out: 16 `blocks` ranks of a slice to a cluster
// of the low form, 128 slots of all slices together to one of the tall form; the
// columns in as many parts (CTAs of a cluster) as fill the GPU when there
// are few tiles, none so short that its rings are not filled once.
struct ShrinkShape {
  bool low;
  int64_t tiles;  // at most
  int slots, blocks, groups, splits, split_cols;
};

int slots_of(const seedlm_adapters& ad) { return ad.rank <= 32 ? 32 : (ad.rank + 63) / 64 * 64; }

// Whether a projection takes tiles of 8 rows or of 64.  In units of 57344 outputs
// and inputs a low tile costs about 1 us and 0.03 us a slot (its ranks are read
// and multiplied for eight rows only), a tall one 6 us and 0.05 us a row; the tall
// form's two kernels take 9.5 us more to start.  Fitted to both forms' times at
// 300 places (1 to 64 adapters of rank 8 to 128, 64 to 4096 rows, four shapes of
// projections): the form taken is never more than 17 % behind the other, at any
// of them.  One adapter, rank 8, 4096 inputs and outputs: low 11.1 us at 256 rows
// and 21.9 at 1024, tall 13.6 and 18.8; rank 128, 8192 inputs, two slices of 28672
// outputs, 64 rows: low 48.9, tall 29.7.  Where X or A is not aligned to 16 bytes
// a low tile costs more: 1.3 leaves at most 21 % at 180 places (1: 49 %; four
// adapters, rank 20, 4099 inputs and outputs, 512 rows: 32.0 low, 25.2 tall).
// The tiles are counted as if the rows were dealt evenly to all n adapters, and
// the measurements deal them so: how they are is on the device.  It matters little
// how uneven the rows of the adapters in use are (4096 rows, eight adapters, rank
// 64, two slices of 28672 outputs: 365 us evenly, 355 with nine in ten rows on
// one), much how many are in use at all: 2048 rows on four adapters there take
// 190 us with n = 4, 213 with n = 64 and 445 with n = 1024; 512 rows on one, rank 16,
// q, k, v of 4096 columns 17, 28 and 29.  A batch that uses few of many is better
// served by a description of those alone.
bool takes_low_tiles(const seedlm_adapters& ad, int M, bool wide) {
  const double low_cost = (1 + 0.03 * slots_of(ad)) * (wide ? 1 : 1.3);
  double size = (double)ad.slices * ad.cols;
  for (int s = 0; s < ad.slices; ++s) size += ad.rows[s];
  const int used = std::min(M, ad.n), each = (M + used - 1) / used;
  const double low = (double)used * ((each + kLowRows - 1) / kLowRows), tall = (double)used * ((each + kTall - 1) / kTall);
  return size / 57344 * (low_cost * low - 6 * tall - 0.05 * M) <= 9.5;
}

ShrinkShape shrink_shape(const seedlm_adapters& ad, int M, bool wide, const DeviceInfo& dev) {
  ShrinkShape sh{};
  sh.slots = slots_of(ad);
  sh.low = takes_low_tiles(ad, M, wide);
  sh.tiles = max_tiles(M, ad.n, sh.low ? kLowRows : kTall);
  int64_t clusters = sh.tiles, round;
  if (sh.low) {
    sh.blocks = sh.slots == 32 ? 2 : 4;
    sh.groups = sh.slots / (16 * sh.blocks);
    clusters *= sh.groups * ad.slices;
    round = kLowWarps * 4;
  } else {
    sh.groups = (ad.slices * sh.slots + ShrinkTallLayout<true>::kSlots - 1) / ShrinkTallLayout<true>::kSlots;
    clusters *= sh.groups;
    round = ShrinkTallLayout<true>::kStages * ShrinkTallLayout<true>::kCols / kStep;
  }
  // Low: about one and a half CTAs for each SM, as many again for the last
  // doubling (37 rows, 20 adapters, fused q, k, v of 4096 columns: 9.1 us with 300
  // CTAs, 11.7 with 600).  Tall: no more than the two that fit
  // one (a second round of CTAs costs more than their shorter parts save; 4096
  // rows, 8192 columns: 32 us in one round of 4 parts, 42 in two of 8).
  const int64_t steps = (ad.cols + kStep - 1) / kStep;
  sh.splits = 1;
  while (sh.splits < kMaxSplits && steps >= 2 * sh.splits * round &&
         (sh.low ? 2 * sh.splits * clusters < 3 * dev.num_sms : sh.splits * clusters <= dev.num_sms))
    sh.splits *= 2;
  // Parts begin at whole stages of either form.
  sh.split_cols = (int)(((steps + sh.splits - 1) / sh.splits + 1) / 2 * 2 * kStep);
  return sh;
}

// The largest of 16, 8, 4 .. bytes that the address and the strides are
// multiples of.
int grain_of(const void* p, int64_t stride1, int64_t stride2) {
  const uint64_t all = reinterpret_cast<uintptr_t>(p) | (uint64_t)stride1 | (uint64_t)stride2 | 16;
  return (int)(all & (0 - all));
}

template <class Kernel, class... Args>
int launch_products_kernel(Kernel kernel, int64_t grid, int threads, int smem, int cluster, cudaStream_t stream,
                           const DeviceInfo& dev, const Args&... args) {
  const int rc = allow_max_smem((const void*)kernel, dev);
  return rc ? rc : launch_pdl_cluster(kernel, (unsigned)grid, threads, (size_t)smem, cluster, stream, args...);
}

template <bool BF16, bool WIDE, int RB>
int launch_shrink_low(const ApplyArgs& p, int64_t tiles, int splits, cudaStream_t stream, const DeviceInfo& dev) {
  return launch_products_kernel(adapters_shrink_low_kernel<BF16, RB, WIDE>, tiles * p.ad.slices * p.groups * splits,
                                32 * kLowWarps, kShrinkLowSmem<RB, WIDE>, splits, stream, dev, p);
}

template <bool BF16, bool WIDE>
int launch_shrink_tall(const ApplyArgs& p, int64_t tiles, int splits, cudaStream_t stream, const DeviceInfo& dev) {
  using L = ShrinkTallLayout<WIDE>;
  return launch_products_kernel(adapters_shrink_tall_kernel<BF16, WIDE>, tiles * p.groups * splits, L::kThreads, L::kBytes,
                                splits, stream, dev, p);
}

template <bool BF16, bool WIDE, int KC, bool MANY>
int launch_expand_low(const ApplyArgs& p, int64_t grid, int chunks, cudaStream_t stream, const DeviceInfo& dev) {
  return launch_products_kernel(adapters_expand_low_kernel<BF16, KC, MANY, WIDE>, grid, 32 * kLowWarps, kExpandLowSmem<KC, WIDE>, 1,
                                stream, dev, p, chunks, (int)(p.base == p.Y));
}

template <bool BF16, bool WIDE, int NB>
int launch_expand_tall(const ApplyArgs& p, int64_t items, int chunks, cudaStream_t stream, const DeviceInfo& dev) {
  using L = TallLayout<BF16, NB>;
  return launch_products_kernel(adapters_expand_tall_kernel<BF16, NB, WIDE>,
                                std::min(items, (int64_t)L::kCtas * dev.num_sms), kTallThreads, L::kBytes, 1, stream,
                                dev, p, chunks, (int)(p.base == p.Y));
}

template <bool BF16, bool WIDE, bool WIDE_B>
int launch_products(ApplyArgs& p, const ShrinkShape& sh, int64_t tiles, cudaStream_t stream, const DeviceInfo& dev) {
  const bool low = sh.low;
  int rc;
  if (low)
    rc = sh.blocks == 4 ? launch_shrink_low<BF16, WIDE, 4>(p, tiles, sh.splits, stream, dev)
                        : launch_shrink_low<BF16, WIDE, 2>(p, tiles, sh.splits, stream, dev);
  else
    rc = launch_shrink_tall<BF16, WIDE>(p, tiles, sh.splits, stream, dev);
  if (rc) return rc;
  // Chunks of outputs.  Low tiles, a CTA each: long enough that a CTA's start is
  // paid for, short enough that there are five CTAs for each SM, up to 12 rounds
  // of the CTA's warps (64 rows of their own adapters, rank 64: 187 us on
  // 28672+28672 outputs with one round, 114 with 12, 116 with 16; rank 16 on
  // 8192: 23 with one, 19 with 6, 23 with 16).  Tall tiles: the outputs of one
  // product.
  int64_t total = 0;
  for (int s = 0; s < p.ad.slices; ++s) total += p.ad.rows[s];
  p.chunk_rows = kTallOutputs;
  if (low) {
    const int round = 32 * kLowWarps;
    const int64_t rounds = (total * tiles - 1) / ((int64_t)round * 5 * dev.num_sms) + 1;
    p.chunk_rows = (int)std::min<int64_t>(rounds, 12) * round;
  }
  int64_t chunks = 0;
  int at = 0;
  for (int s = 0; s < p.ad.slices; ++s) {
    p.chunk_first[s] = (int)chunks;
    p.slice_at[s] = at;
    chunks += (p.ad.rows[s] + p.chunk_rows - 1) / p.chunk_rows;
    at += p.ad.rows[s];
  }
  for (int s = p.ad.slices; s <= SEEDLM_MAX_SLICES; ++s) p.chunk_first[s] = (int)chunks;
  const int64_t grid = chunks * tiles;
  if (grid > INT32_MAX) return SEEDLM_EUNSUPPORTED;
  if (low)
    return p.slots == 32   ? launch_expand_low<BF16, WIDE_B, 1, false>(p, grid, (int)chunks, stream, dev)
           : p.slots == 64 ? launch_expand_low<BF16, WIDE_B, 2, false>(p, grid, (int)chunks, stream, dev)
                           : launch_expand_low<BF16, WIDE_B, 2, true>(p, grid, (int)chunks, stream, dev);
  return p.blocks == 1   ? launch_expand_tall<BF16, WIDE_B, 1>(p, grid, (int)chunks, stream, dev)
         : p.blocks == 2 ? launch_expand_tall<BF16, WIDE_B, 2>(p, grid, (int)chunks, stream, dev)
                         : launch_expand_tall<BF16, WIDE_B, 4>(p, grid, (int)chunks, stream, dev);
}

// Bytes of S, then those of its factors.
int64_t sums_bytes(const seedlm_adapters& ad, int M, int slots) {
  const int parts = ad.dtype == SEEDLM_BF16 ? kParts<true> : kParts<false>;
  return (int64_t)M * ad.slices * parts * slots * 2;
}

}  // namespace

int64_t adapters_workspace_bytes(const seedlm_adapters& ad, int M, const DeviceInfo&) {
  const int slots = slots_of(ad);
  const int64_t blocks = std::max(1, slots / 64);
  return sums_bytes(ad, M, slots) + (ad.dtype == SEEDLM_F16 ? (int64_t)M * ad.slices * blocks * 4 : 0);
}

int launch_adapters_apply(const seedlm_adapters& ad, const int32_t* plan, int M, const uint16_t* X, int64_t ldx,
                          const float* base, int64_t ldb, float* Y, int64_t ldy, void* workspace, cudaStream_t stream,
                          const DeviceInfo& dev) {
  ApplyArgs p{};
  p.ad = ad;
  p.plan = plan;
  p.M = M;
  p.X = X;
  p.ldx = ldx;
  p.base = base;
  p.ldb = ldb;
  p.Y = Y;
  p.ldy = ldy;
  int64_t at = 0;
  for (int s = 0; s < ad.slices; ++s) {
    // (A stride that no row is reached by does not count.)
    const int64_t n1 = ad.n > 1, r1 = ad.rank > 1, j1 = ad.rows[s] > 1, m1 = M > 1;
    p.grain_a[s] = ad.rows[s] ? grain_of(ad.A[s], n1 * 2 * ad.a_adapter[s], r1 * 2 * ad.a_row[s]) : 16;
    p.grain_b[s] = grain_of(ad.B[s], n1 * 2 * ad.b_adapter[s], j1 * 2 * ad.b_row[s]);
    p.grain_y[s] = std::min(grain_of(base + at, m1 * 4 * ldb, 0), grain_of(Y + at, m1 * 4 * ldy, 0));
    at += ad.rows[s];
  }
  p.grain_x = grain_of(X, M > 1 ? 2 * ldx : 0, 0);
  bool wide = p.grain_x == 16, wide_b = true;
  for (int s = 0; s < ad.slices; ++s) {
    wide = wide && p.grain_a[s] == 16;
    wide_b = wide_b && p.grain_b[s] == 16;
  }
  const ShrinkShape sh = shrink_shape(ad, M, wide, dev);
  p.S = static_cast<uint16_t*>(workspace);
  p.unscale = reinterpret_cast<float*>(static_cast<char*>(workspace) + sums_bytes(ad, M, sh.slots));
  p.slots = sh.slots;
  p.blocks = std::max(1, sh.slots / 64);
  p.split_cols = sh.split_cols;
  p.groups = sh.groups;
  const int64_t tiles = sh.tiles;
  p.room = (int)tiles;
  p.head = reinterpret_cast<const int4*>(plan + plan_tail(M, ad.n)) + (sh.low ? 0 : 1);
  p.tiles = reinterpret_cast<const int4*>(plan + plan_tail(M, ad.n)) + 2 + (sh.low ? 0 : max_tiles(M, ad.n, kLowRows));
  if (tiles * ad.slices * sh.groups * sh.splits > INT32_MAX) return SEEDLM_EUNSUPPORTED;
  if (ad.dtype == SEEDLM_BF16)
    return wide     ? wide_b ? launch_products<true, true, true>(p, sh, tiles, stream, dev)
                             : launch_products<true, true, false>(p, sh, tiles, stream, dev)
           : wide_b ? launch_products<true, false, true>(p, sh, tiles, stream, dev)
                    : launch_products<true, false, false>(p, sh, tiles, stream, dev);
  return wide     ? wide_b ? launch_products<false, true, true>(p, sh, tiles, stream, dev)
                           : launch_products<false, true, false>(p, sh, tiles, stream, dev)
         : wide_b ? launch_products<false, false, true>(p, sh, tiles, stream, dev)
                  : launch_products<false, false, false>(p, sh, tiles, stream, dev);
}

int read_and_clear_plan_mismatch(unsigned int* out) {
  unsigned int v = 0, zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_plan_mismatch, sizeof(v));
  if (err == cudaSuccess && v) err = cudaMemcpyToSymbol(g_plan_mismatch, &zero, sizeof(zero));
  *out = v;
  return record_cuda_error(err);
}

int read_and_clear_adapters_error(unsigned int* out) {
  unsigned int v = 0, zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_wait_error, sizeof(v));
  if (err == cudaSuccess && v) err = cudaMemcpyToSymbol(g_wait_error, &zero, sizeof(zero));
  *out = v;
  return record_cuda_error(err);
}

}  // namespace seedlm
