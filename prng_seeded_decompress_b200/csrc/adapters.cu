// adapters.cu -- low-rank adapters of many requests beside a shared
// projection: Y[m] = base[m] + s_a (x_m A_a^T) B_a^T with a the adapter of
// row m, and the plan that sorts a batch's rows by adapter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.cuh"
#include "seedlm_device.cuh"
#include "seedlm_internal.h"

namespace seedlm {

SEEDLM_CHECK_FLAG(adapters)

namespace {

// Set when a plan does not belong to the call it is given to.
__device__ unsigned int g_plan_mismatch;

// ---------------------------------------------------------------- the plan
//
// Layout in int32 words: [0, M) order, [M, M + n + 1) offsets, then from the
// next multiple of 4: {M, n, tiles of rows with an adapter, all tiles} and
// one int4 {adapter or -1, first, count, 0} for each tile of up to
// adapter_tile_rows(M) rows of one adapter, in sorted order.

__host__ __device__ inline int64_t plan_tail(int64_t M, int64_t n) { return (M + n + 1 + 3) / 4 * 4; }

// Rows of a tile: short tiles for batches where most requests have their own
// adapter, tall ones where an adapter's rows share its matrices.
__host__ __device__ inline int adapter_tile_rows(int M) { return M <= 256 ? 8 : 64; }

// Every bin of c rows takes at most c / T + 1 tiles.
inline int64_t max_tiles(int64_t M, int64_t n) {
  return M / adapter_tile_rows((int)M) + (M < n + 1 ? M : n + 1);
}

constexpr int kPlanMaxThreads = 1024;

// A stable counting sort by one CTA.  Each warp takes one contiguous part of
// the rows and counts its adapters in a histogram of its own (match_any
// groups the lanes of a step, so no two lanes touch a bin); the histograms
// are turned into starting places bin by bin, and a second walk over the same
// rows puts each at its place.  Latency bound: two passes over 4 M bytes and
// four barriers.
__global__ void __launch_bounds__(kPlanMaxThreads, 1)
adapters_plan_kernel(int M, int n, int T, const int32_t* __restrict__ ids, int32_t* __restrict__ plan,
                     int64_t tail_words) {
  extern __shared__ int32_t sm[];
  const int bins = n + 1, nwarps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int32_t* hist = sm;                            // [nwarps][bins]
  int32_t* start = hist + (size_t)nwarps * bins; // [bins + 1]
  int32_t* tstart = start + bins + 1;            // [bins + 1]
  int32_t* warp_rows = tstart + bins + 1;        // [nwarps]
  int32_t* warp_tiles = warp_rows + nwarps;      // [nwarps]
  grid_launch_dependents();
  for (int i = threadIdx.x; i < nwarps * bins; i += blockDim.x) hist[i] = 0;
  grid_wait();
  __syncthreads();
  const int chunk = ((M + nwarps - 1) / nwarps + 31) / 32 * 32;
  const int r0 = min(M, warp * chunk), r1 = min(M, r0 + chunk);
  int32_t* mine = hist + (size_t)warp * bins;
  for (int r = r0; r < r1; r += 32) {
    const int row = r + lane;
    int key = -1;
    if (row < r1) {
      const int id = ids[row];
      key = id >= 0 && id < n ? id : n;
    }
    const unsigned same = __match_any_sync(0xffffffffu, key);
    if (key >= 0 && (same & ((1u << lane) - 1)) == 0) mine[key] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // Exclusive sums over the warps of each bin; then over the bins, each
  // thread taking `per` consecutive ones.
  const int per = (bins + blockDim.x - 1) / blockDim.x;
  const int b0 = min(bins, (int)threadIdx.x * per), b1 = min(bins, b0 + per);
  int rows = 0, tiles = 0;
  for (int b = b0; b < b1; ++b) {
    int run = 0;
    for (int w = 0; w < nwarps; ++w) {
      const int t = hist[w * bins + b];
      hist[w * bins + b] = run;
      run += t;
    }
    start[b] = rows;  // within this thread's bins
    tstart[b] = tiles;
    rows += run;
    tiles += (run + T - 1) / T;
  }
  int2 incl = make_int2(rows, tiles);
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) incl = make_int2(incl.x + x, incl.y + y);
  }
  if (lane == 31) {
    warp_rows[warp] = incl.x;
    warp_tiles[warp] = incl.y;
  }
  __syncthreads();
  int2 before = make_int2(incl.x - rows, incl.y - tiles);
  for (int w = 0; w < warp; ++w) before = make_int2(before.x + warp_rows[w], before.y + warp_tiles[w]);
  for (int b = b0; b < b1; ++b) {
    start[b] += before.x;
    tstart[b] += before.y;
    plan[M + b] = start[b];
  }
  if (b1 == bins && b0 < bins) {  // the thread of the last bin
    start[bins] = before.x + rows;
    tstart[bins] = before.y + tiles;
  }
  __syncthreads();
  for (int r = r0; r < r1; r += 32) {
    const int row = r + lane;
    int key = -1;
    if (row < r1) {
      const int id = ids[row];
      key = id >= 0 && id < n ? id : n;
    }
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(same & ((1u << lane) - 1));
    int at = 0;
    if (key >= 0) at = start[key] + mine[key] + rank;
    __syncwarp();
    if (key >= 0) {
      if (SEEDLM_IN_BOUNDS(g_check_flag, at, M)) plan[at] = row;
      if (rank == 0) mine[key] += __popc(same);
    }
    __syncwarp();
  }
  int32_t* tail = plan + plan_tail(M, n);
  const int total = tstart[bins];
  if (threadIdx.x == 0) *reinterpret_cast<int4*>(tail) = make_int4(M, n, tstart[n], total);
  for (int t = threadIdx.x; t < total; t += blockDim.x) {
    int lo = 0, hi = bins - 1;  // the last bin that starts at or before tile t
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (tstart[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int first = start[lo] + (t - tstart[lo]) * T;
    if (SEEDLM_IN_BOUNDS(g_check_flag, 4 + 4 * (int64_t)t + 3, tail_words))
      reinterpret_cast<int4*>(tail)[1 + t] = make_int4(lo < n ? lo : -1, first, min(T, start[lo + 1] - first), 0);
  }
}

// ------------------------------------------------------------- the products
//
// Two kernels.  The first takes the sums S = s_a x A_a^T, the second adds
// S B_a^T to the outputs.  Both feed mma.sync with fragments loaded straight
// from memory: of a contraction step of 32, the lane in column q of its quad
// takes elements 8q .. 8q + 7 with one 16-byte load and gives words 0, 1 to a
// first m16n8k16 product and words 2, 3 to a second.  The order of the
// contraction does not matter as long as both operands are read alike, so no
// operand is staged or shuffled.  The matrix of adapter weights is the
// operand of 16 rows and the tile's activations the one of 8 columns, so a
// request that is alone with its adapter wastes tensor work, which is idle
// here, and no memory traffic, which is what bounds both kernels.

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;       // contraction elements of one 16-byte load per lane
constexpr int kMaxSplits = 32;  // parts of the first contraction

struct ApplyArgs {
  seedlm_adapters ad;
  const int32_t* plan;
  int M;
  const uint16_t* X;
  int64_t ldx;
  const float* base;
  int64_t ldb;
  float* Y;
  int64_t ldy;
  float* S;         // [splits][M][width], rows in sorted order
  int splits;       // parts of the columns, one CTA each
  int split_cols;   // columns of a part: a multiple of kStep
  int width;        // slices * rank16
  int rank16;       // rank rounded up to 16
  int groups;       // first kernel: CTAs that share a slice's rank
  int chunk_first[SEEDLM_MAX_SLICES + 1];  // second kernel: chunks of outputs before each slice
  int chunk_rows;   // outputs of a chunk
  int slice_at[SEEDLM_MAX_SLICES];         // first output of each slice
  int vec_a, vec_b, vec_y;  // rows can be read 16 bytes at a time: bit s for slice s
};

__device__ __forceinline__ const int32_t* plan_tail_of(const ApplyArgs& p) { return p.plan + plan_tail(p.M, p.ad.n); }

__device__ __forceinline__ bool plan_fits(const ApplyArgs& p) {
  const int32_t* tail = plan_tail_of(p);
  const bool ok = tail[0] == p.M && tail[1] == p.ad.n;
  if (!ok && threadIdx.x == 0) atomicOr(&g_plan_mismatch, 1u);
  return ok;
}

__device__ __forceinline__ int rank_of(const seedlm_adapters& ad, int a) {
  if (a < 0) return 0;
  return ad.ranks ? max(0, min(ad.ranks[a], ad.rank)) : ad.rank;
}

// Elements k .. k + 7 of a row of `len`, zero beyond its end, one at a time.
__device__ __forceinline__ uint4 load8_slow(const uint16_t* row, int k, int len) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < len) w[i / 2] |= (uint32_t)__ldg(row + k + i) << (16 * (i % 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 load8(const uint16_t* row, int k, int len, bool whole) {
  return whole ? __ldg(reinterpret_cast<const uint4*>(row + k)) : load8_slow(row, k, len);
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

// One step of 32: rows g and g + 8 of the 16-row operand in lo and hi.
template <bool BF16>
__device__ __forceinline__ void mma_step(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& x) {
  mma16816<BF16>(d, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
  mma16816<BF16>(d, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

// S = s_a x A_a^T.  A CTA takes one tile of rows, RB blocks of 16 ranks of one
// slice and one part of the columns; its warps take steps of the part in turn
// (UNROLL at a time, all their loads in flight together) and add their sums
// through shared memory in a fixed order.  The parts are added by the second
// kernel.  NT: the tile's rows / 8.
template <bool BF16, int NT, int RB, int UNROLL>
__global__ void __launch_bounds__(kThreads) adapters_shrink_kernel(const __grid_constant__ ApplyArgs p) {
  extern __shared__ float red[];  // [kWarps][RB * 16][NT * 8]
  grid_wait();
  // After the wait: what ran before this kernel is then complete for the next
  // one too, which reads the plan, B and base before its own wait.
  grid_launch_dependents();
  if (!plan_fits(p)) return;
  const int32_t* tail = plan_tail_of(p);
  const int part = blockIdx.x % p.splits;
  const int group = blockIdx.x / p.splits % p.groups;
  const int s = blockIdx.x / (p.splits * p.groups) % p.ad.slices;
  const int t = blockIdx.x / (p.splits * p.groups * p.ad.slices);
  if (t >= tail[2]) return;
  const int4 tile = reinterpret_cast<const int4*>(tail)[1 + t];
  const int a = tile.x, first = tile.y, count = tile.z;
  const int rank = rank_of(p.ad, a), r0 = group * RB * 16;
  if (r0 >= rank) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int cols = p.ad.cols;
  const uint16_t* A = static_cast<const uint16_t*>(p.ad.A[s]) + a * p.ad.a_adapter[s];
  const int64_t a_row = p.ad.a_row[s];
  const uint16_t* xrow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int at = 8 * i + g;
    const int row = at < count ? p.plan[first + at] : -1;
    xrow[i] = row >= 0 && SEEDLM_IN_BOUNDS(g_check_flag, row, p.M) ? p.X + row * p.ldx : nullptr;
  }
  float acc[RB][NT][4] = {};
  const int k0 = part * p.split_cols, k1 = min(cols, k0 + p.split_cols);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int k = k0 + warp * UNROLL * kStep;
  if ((p.vec_a >> s) & 1) {
    for (; k + UNROLL * kStep <= k1; k += kWarps * UNROLL * kStep) {
      uint4 w[UNROLL][RB][2], x[UNROLL][NT];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int at = k + u * kStep + 8 * q;
        const bool in = SEEDLM_IN_BOUNDS(g_check_flag, at + 7, cols);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          x[u][i] = in && xrow[i] ? __ldg(reinterpret_cast<const uint4*>(xrow[i] + at)) : zero;
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = r0 + 16 * b + 8 * h + g;
            w[u][b][h] = in && r < rank ? ld_stream_u4(A + r * a_row + at) : zero;
          }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int i = 0; i < NT; ++i) mma_step<BF16>(acc[b][i], w[u][b][0], w[u][b][1], x[u][i]);
    }
  }
  // What is left of the part (all of it where rows are not aligned), a step at
  // a time; elements beyond its end count as zero.
  for (; k < k1; k += kWarps * UNROLL * kStep)
    for (int u = 0; u < UNROLL && k + u * kStep < k1; ++u) {
      const int at = k + u * kStep + 8 * q;
      const bool whole = ((p.vec_a >> s) & 1) && k + (u + 1) * kStep <= k1;
      uint4 w[RB][2];
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = r0 + 16 * b + 8 * h + g;
          w[b][h] = r < rank ? load8(A + r * a_row, at, k1, whole) : zero;
        }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 x = xrow[i] ? load8(xrow[i], at, k1, whole) : zero;
#pragma unroll
        for (int b = 0; b < RB; ++b) mma_step<BF16>(acc[b][i], w[b][0], w[b][1], x);
      }
    }
  // Sums of the warps, [rank][row], each warp's in its own place.
  constexpr int T = NT * 8, R = RB * 16;
  float* mine = red + warp * R * T;
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float* d = mine + (16 * b + g) * T + 8 * i + 2 * q;
      *reinterpret_cast<float2*>(d) = make_float2(acc[b][i][0], acc[b][i][1]);
      *reinterpret_cast<float2*>(d + 8 * T) = make_float2(acc[b][i][2], acc[b][i][3]);
    }
  __syncthreads();
  const float scale = p.ad.scales ? p.ad.scales[a] : 1.f;
  float* out = p.S + ((int64_t)part * p.M + first) * p.width + s * p.rank16 + r0;
  SEEDLM_CHECK_ONLY(const int64_t out_extent = (int64_t)(p.splits - part) * p.M * p.width -
                                               (int64_t)first * p.width - s * p.rank16 - r0;)
  for (int e = threadIdx.x; e < R * T; e += kThreads) {
    const int r = e % R, i = e / R;
    if (i >= count || r0 + r >= rank) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[(w * R + r) * T + i];
    if (SEEDLM_IN_BOUNDS(g_check_flag, (int64_t)i * p.width + r, out_extent)) out[(int64_t)i * p.width + r] = scale * sum;
  }
}

// The parts of S that a 16-bit operand holds.  bf16 has fp32's range: three
// parts cut off (not rounded, so none overflows) hold all 24 bits.  fp16 parts
// are of S times a power of two that brings the row's largest finite element
// to [2^14, 2^15): two rounded parts leave at most 2^-24 of an element, or
// 2^-40 of the largest one where that is more.
template <bool BF16>
constexpr int kParts = BF16 ? 3 : 2;

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

// Elements of a row of a part of S in shared memory: an odd multiple of 32, so
// that the 16-byte reads of 8 neighbouring lanes (2 rows x 4) touch every bank
// once.
__host__ __device__ inline int s_stride(int rank) { return ((rank + 31) / 32 | 1) * 32; }

__host__ __device__ inline int expand_smem(int rows, int rank, int parts) {
  return parts * rows * s_stride(rank) * 2 + rows * 4;
}

// Y = base + S B_a^T.  A CTA takes one tile of rows and a chunk of one slice's
// outputs; a warp takes 32 outputs at a time, of which lane (g, q) holds
// outputs 4g .. 4g + 3 of rows 2q and 2q + 1 of every 8: the rows 4g + j of B
// are dealt to the two 16-row operands so that base and Y are read and written
// 16 bytes a lane, 128 bytes a row.
template <bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
adapters_expand_kernel(const __grid_constant__ ApplyArgs p, int chunks, int in_place) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int T = NT * 8, P = kParts<BF16>;
  grid_launch_dependents();
  if (!plan_fits(p)) {
    grid_wait();
    return;
  }
  const int32_t* tail = plan_tail_of(p);
  const int t = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  int4 tile = make_int4(-1, 0, 0, 0);
  if (t < tail[in_place ? 2 : 3]) tile = reinterpret_cast<const int4*>(tail)[1 + t];
  const int a = tile.x, first = tile.y, count = tile.z;
  const int rank = rank_of(p.ad, a);
  if (count == 0 || (in_place && rank == 0)) {
    grid_wait();
    return;
  }
  int s = 0;
  while (chunk >= p.chunk_first[s + 1]) ++s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int stride = s_stride(p.ad.rank);
  uint16_t* sp = reinterpret_cast<uint16_t*>(smem);           // [P][T][stride]
  float* unscale = reinterpret_cast<float*>(sp + P * T * stride);  // [T]
  const int rows = p.ad.rows[s];
  const int c0 = (chunk - p.chunk_first[s]) * p.chunk_rows, c1 = min(rows, c0 + p.chunk_rows);
  const uint16_t* B = static_cast<const uint16_t*>(p.ad.B[s]) + max(a, 0) * p.ad.b_adapter[s];
  const int64_t b_row = p.ad.b_row[s];
  const bool vec_b = (p.vec_b >> s) & 1, vec_y = (p.vec_y >> s) & 1;

  // This lane's rows of base and Y; their numbers come from the plan.
  int yrow[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int at = 8 * i + 2 * q + e;
      yrow[i][e] = at < count ? p.plan[first + at] : -1;
      if (yrow[i][e] >= 0 && !SEEDLM_IN_BOUNDS(g_check_flag, yrow[i][e], p.M)) yrow[i][e] = -1;
    }

  grid_wait();
  // S of the tile, its parts added in order, cut up for the tensor cores: a
  // warp a row, two neighbouring elements a lane.
  for (int i = warp; i < T; i += kWarps) {
    float v[SEEDLM_MAX_RANK / 64][2];
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < SEEDLM_MAX_RANK / 64; ++j) {
      v[j][0] = v[j][1] = 0.f;
      const int r = 64 * j + 2 * lane;
      if (i < count && r < rank) {
        const float* src = p.S + (int64_t)(first + i) * p.width + s * p.rank16 + r;
        for (int part = 0; part < p.splits; ++part) {
          const float2 add = __ldcg(reinterpret_cast<const float2*>(src + (int64_t)part * p.M * p.width));
          v[j][0] += add.x;
          if (r + 1 < rank) v[j][1] += add.y;
        }
        if (finite(v[j][0])) top = fmaxf(top, fabsf(v[j][0]));
        if (finite(v[j][1])) top = fmaxf(top, fabsf(v[j][1]));
      }
    }
    float up = 1.f;
    if constexpr (!BF16) {
#pragma unroll
      for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2^e with e = 14 - floor(log2 top), at most 126 (top below 2^-112).
      const int e = top > 0.f ? min(126, 14 - ((int)(__float_as_uint(top) >> 23) - 127)) : 0;
      up = __uint_as_float((uint32_t)(e + 127) << 23);
      if (lane == 0) unscale[i] = __uint_as_float((uint32_t)(127 - e) << 23);
    }
#pragma unroll
    for (int j = 0; j < SEEDLM_MAX_RANK / 64; ++j) {
      const int r = 64 * j + 2 * lane;
      if (r >= stride) continue;
      uint16_t lo[3], hi[3];
      split<BF16>(v[j][0] * up, lo);
      split<BF16>(v[j][1] * up, hi);
#pragma unroll
      for (int w = 0; w < P; ++w)
        *reinterpret_cast<uint32_t*>(sp + (w * T + i) * stride + r) = lo[w] | (uint32_t)hi[w] << 16;
    }
  }
  __syncthreads();

  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int n0 = c0 + 32 * warp; n0 < c1; n0 += 32 * kWarps) {
    float acc[2][NT][4] = {};
    for (int k = 0; k < rank; k += kStep) {
      uint4 w[4];
      const int at = k + 8 * q;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + 4 * g + j;
        w[j] = zero;
        if (n < c1) {
          if (vec_b && at + 8 <= rank) w[j] = ld_stream_u4(B + n * b_row + at);
          else if (at < rank) w[j] = load8_slow(B + n * b_row, at, rank);
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int pt = 0; pt < P; ++pt) {
          const uint4 x = *reinterpret_cast<const uint4*>(sp + (pt * T + 8 * i + g) * stride + at);
          mma_step<BF16>(acc[0][i], w[0], w[1], x);
          mma_step<BF16>(acc[1][i], w[2], w[3], x);
        }
    }
    const int n = n0 + 4 * g;
    const int64_t col = p.slice_at[s] + n;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (yrow[i][e] < 0 || n >= c1) continue;
        float4 d = make_float4(acc[0][i][e], acc[0][i][2 + e], acc[1][i][e], acc[1][i][2 + e]);
        if constexpr (!BF16) {
          const float f = unscale[8 * i + 2 * q + e];
          d = make_float4(d.x * f, d.y * f, d.z * f, d.w * f);
        }
        const float* from = p.base + yrow[i][e] * p.ldb + col;
        float* to = p.Y + yrow[i][e] * p.ldy + col;
        if (vec_y && n + 4 <= c1) {
          const float4 b = __ldcg(reinterpret_cast<const float4*>(from));
          *reinterpret_cast<float4*>(to) = make_float4(b.x + d.x, b.y + d.y, b.z + d.z, b.w + d.w);
        } else {
          const float dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < c1) to[j] = __ldcg(from + j) + dv[j];
        }
      }
  }
}

}  // namespace

int64_t adapters_plan_words(int M, int n) { return plan_tail(M, n) + 4 + 4 * max_tiles(M, n); }

int launch_adapters_plan(int M, int n, const int32_t* ids, int32_t* plan, cudaStream_t stream, const DeviceInfo& dev) {
  int rc = allow_max_smem((const void*)adapters_plan_kernel, dev);
  if (rc) return rc;
  const int most = M > n + 1 ? M : n + 1;
  const int threads = most >= kPlanMaxThreads ? kPlanMaxThreads : (most + 31) / 32 * 32;
  const int nwarps = threads / 32, bins = n + 1;
  const size_t smem = ((size_t)nwarps * bins + 2 * (bins + 1) + 2 * nwarps) * sizeof(int32_t);
  return launch_pdl(adapters_plan_kernel, 1, threads, smem, stream, M, n, adapter_tile_rows(M), ids, plan,
                    adapters_plan_words(M, n) - plan_tail(M, n));
}

namespace {

// How the first product is shared out: RB blocks of 16 ranks to a CTA, the
// columns in parts so that a few tiles still fill the GPU (about four CTAs an
// SM), no part so short that a warp has less than one load.
struct ShrinkShape {
  int rank16, blocks, groups, splits, split_cols;
};

// Steps of the columns whose loads a warp has in flight together: 12 loads of
// 16 bytes a lane or so.
constexpr int shrink_unroll(int nt, int blocks) { return nt == 1 ? 4 / blocks : 1; }

ShrinkShape shrink_shape(const seedlm_adapters& ad, int M, const DeviceInfo& dev) {
  ShrinkShape sh;
  sh.rank16 = (ad.rank + 15) / 16 * 16;
  const bool low = adapter_tile_rows(M) == 8;
  const int blocks16 = sh.rank16 / 16;
  sh.blocks = blocks16 >= 4 && low ? 4 : blocks16 >= 2 ? 2 : 1;
  sh.groups = (blocks16 + sh.blocks - 1) / sh.blocks;
  const int64_t ctas = max_tiles(M, ad.n) * sh.groups * ad.slices;
  const int64_t steps = (ad.cols + kStep - 1) / kStep;
  const int64_t round = kWarps * shrink_unroll(low ? 1 : 8, sh.blocks);
  int64_t splits = (4 * (int64_t)dev.num_sms + ctas - 1) / ctas;
  if (splits > kMaxSplits) splits = kMaxSplits;
  const int64_t each = std::max<int64_t>(1, ((steps + splits - 1) / splits + round - 1) / round) * round;
  sh.split_cols = (int)(each * kStep);
  sh.splits = (int)std::max<int64_t>(1, (steps + each - 1) / each);
  return sh;
}

bool rows_aligned(const void* p, int64_t ld1, int64_t ld2, int bytes) {
  return aligned(p, 16) && ld1 * bytes % 16 == 0 && ld2 * bytes % 16 == 0;
}

template <bool BF16, int NT, int RB>
int launch_shrink(const ApplyArgs& p, int64_t tiles, cudaStream_t stream, const DeviceInfo& dev) {
  auto kernel = adapters_shrink_kernel<BF16, NT, RB, shrink_unroll(NT, RB)>;
  const size_t smem = (size_t)kWarps * RB * 16 * NT * 8 * sizeof(float);
  int rc = allow_max_smem((const void*)kernel, dev);
  if (rc) return rc;
  return launch_pdl(kernel, (unsigned)(tiles * p.ad.slices * p.groups * p.splits), kThreads, smem, stream, p);
}

template <bool BF16, int NT>
int launch_products(ApplyArgs& p, const ShrinkShape& sh, int64_t tiles, cudaStream_t stream, const DeviceInfo& dev) {
  int rc;
  if (NT == 1 && sh.blocks == 4) rc = launch_shrink<BF16, 1, 4>(p, tiles, stream, dev);
  else if (sh.blocks == 2) rc = launch_shrink<BF16, NT, 2>(p, tiles, stream, dev);
  else rc = launch_shrink<BF16, NT, 1>(p, tiles, stream, dev);
  if (rc) return rc;
  // Chunks of outputs: as long as they can be (a CTA pays for its S once) with
  // some eight CTAs left for each SM, at least one round of its warps.
  int64_t total = 0;
  for (int s = 0; s < p.ad.slices; ++s) total += p.ad.rows[s];
  const int round = 32 * kWarps;
  int64_t rounds = total * tiles / ((int64_t)round * 8 * dev.num_sms);
  rounds = rounds < 1 ? 1 : rounds > 8 ? 8 : rounds;
  p.chunk_rows = (int)rounds * round;
  int chunks = 0, at = 0;
  for (int s = 0; s < p.ad.slices; ++s) {
    p.chunk_first[s] = chunks;
    p.slice_at[s] = at;
    chunks += (p.ad.rows[s] + p.chunk_rows - 1) / p.chunk_rows;
    at += p.ad.rows[s];
  }
  for (int s = p.ad.slices; s <= SEEDLM_MAX_SLICES; ++s) p.chunk_first[s] = chunks;
  if (chunks * tiles > INT32_MAX) return SEEDLM_EUNSUPPORTED;
  auto kernel = adapters_expand_kernel<BF16, NT>;
  if ((rc = allow_max_smem((const void*)kernel, dev))) return rc;
  return launch_pdl(kernel, (unsigned)(chunks * tiles), kThreads, expand_smem(NT * 8, p.ad.rank, kParts<BF16>), stream,
                    p, chunks, (int)(p.base == p.Y));
}

}  // namespace

int64_t adapters_workspace_bytes(const seedlm_adapters& ad, int M, const DeviceInfo& dev) {
  const ShrinkShape sh = shrink_shape(ad, M, dev);
  return (int64_t)sh.splits * M * ad.slices * sh.rank16 * 4;
}

int launch_adapters_apply(const seedlm_adapters& ad, const int32_t* plan, int M, const uint16_t* X, int64_t ldx,
                          const float* base, int64_t ldb, float* Y, int64_t ldy, void* workspace, cudaStream_t stream,
                          const DeviceInfo& dev) {
  const ShrinkShape sh = shrink_shape(ad, M, dev);
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
  p.S = static_cast<float*>(workspace);
  p.splits = sh.splits;
  p.split_cols = sh.split_cols;
  p.rank16 = sh.rank16;
  p.width = ad.slices * sh.rank16;
  p.groups = sh.groups;
  int64_t at = 0;
  for (int s = 0; s < ad.slices; ++s) {
    p.vec_a |= (rows_aligned(ad.A[s], ad.a_adapter[s], ad.a_row[s], 2) && rows_aligned(X, ldx, 0, 2)) << s;
    p.vec_b |= rows_aligned(ad.B[s], ad.b_adapter[s], ad.b_row[s], 2) << s;
    p.vec_y |= (rows_aligned(base, ldb, at, 4) && rows_aligned(Y, ldy, at, 4)) << s;
    at += ad.rows[s];
  }
  const int64_t tiles = max_tiles(M, ad.n);
  if (tiles * ad.slices * sh.groups * sh.splits > INT32_MAX) return SEEDLM_EUNSUPPORTED;
  const bool bf16 = ad.dtype == SEEDLM_BF16;
  if (adapter_tile_rows(M) == 8)
    return bf16 ? launch_products<true, 1>(p, sh, tiles, stream, dev) : launch_products<false, 1>(p, sh, tiles, stream, dev);
  return bf16 ? launch_products<true, 8>(p, sh, tiles, stream, dev) : launch_products<false, 8>(p, sh, tiles, stream, dev);
}

int read_and_clear_plan_mismatch(unsigned int* out) {
  unsigned int v = 0, zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_plan_mismatch, sizeof(v));
  if (err == cudaSuccess && v) err = cudaMemcpyToSymbol(g_plan_mismatch, &zero, sizeof(zero));
  *out = v;
  return record_cuda_error(err);
}

}  // namespace seedlm
