// adapters.cu -- low-rank adapters of many requests beside a shared
// projection: Y[m] = base[m] + s_a (x_m A_a^T) B_a^T with a the adapter of
// row m, and the plan that sorts a batch's rows by adapter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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
  float* S;  // [M][slices * rank], rows in sorted order
};

__device__ __forceinline__ bool plan_fits(const ApplyArgs& p) {
  const int32_t* tail = p.plan + plan_tail(p.M, p.ad.n);
  const bool ok = tail[0] == p.M && tail[1] == p.ad.n;
  if (!ok && threadIdx.x == 0) atomicOr(&g_plan_mismatch, 1u);
  return ok;
}

__device__ __forceinline__ int rank_of(const seedlm_adapters& ad, int a) {
  if (a < 0) return 0;
  return ad.ranks ? max(0, min(ad.ranks[a], ad.rank)) : ad.rank;
}

// S = s_a x A_a^T: one CTA for each sorted row and slice, a warp a dot.
__global__ void __launch_bounds__(256) adapters_shrink_kernel(const ApplyArgs p) {
  grid_wait();
  if (!plan_fits(p)) return;
  const int4* tiles = reinterpret_cast<const int4*>(p.plan + plan_tail(p.M, p.ad.n)) + 1;
  const int T = adapter_tile_rows(p.M), s = blockIdx.y;
  const int t = blockIdx.x / T, i = blockIdx.x % T;
  if (t >= p.plan[plan_tail(p.M, p.ad.n) + 2]) return;
  const int4 tile = tiles[t];
  if (i >= tile.z) return;
  const int pos = tile.y + i, a = tile.x, rank = rank_of(p.ad, a);
  const uint16_t* x = p.X + (int64_t)p.plan[pos] * p.ldx;
  const float scale = p.ad.scales ? p.ad.scales[a] : 1.f;
  const int bf = p.ad.dtype == SEEDLM_BF16, lane = threadIdx.x % 32;
  for (int r = threadIdx.x / 32; r < rank; r += 8) {
    const uint16_t* w = static_cast<const uint16_t*>(p.ad.A[s]) + a * p.ad.a_adapter[s] + r * p.ad.a_row[s];
    float sum = 0.f;
    for (int k = lane; k < p.ad.cols; k += 32) sum = fmaf(act_to_float(x[k], bf), act_to_float(w[k], bf), sum);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) p.S[(int64_t)pos * (p.ad.slices * p.ad.rank) + s * p.ad.rank + r] = scale * sum;
  }
}

// Y = base + S B_a^T: a thread for each output.
__global__ void __launch_bounds__(256) adapters_expand_kernel(const ApplyArgs p, int total_rows, int add_in_place) {
  grid_wait();
  if (!plan_fits(p)) return;
  const int32_t* tail = p.plan + plan_tail(p.M, p.ad.n);
  const int T = adapter_tile_rows(p.M);
  const int t = blockIdx.x / T, i = blockIdx.x % T;
  if (t >= tail[add_in_place ? 2 : 3]) return;
  const int4 tile = reinterpret_cast<const int4*>(tail)[1 + t];
  if (i >= tile.z) return;
  const int pos = tile.y + i, a = tile.x, rank = rank_of(p.ad, a);
  const int64_t row = p.plan[pos];
  const int bf = p.ad.dtype == SEEDLM_BF16;
  const int j = blockIdx.y * 256 + threadIdx.x;
  if (j >= total_rows) return;
  int s = 0, local = j;
  while (local >= p.ad.rows[s]) local -= p.ad.rows[s++];
  const float* S = p.S + (int64_t)pos * (p.ad.slices * p.ad.rank) + s * p.ad.rank;
  const uint16_t* w = static_cast<const uint16_t*>(p.ad.B[s]) + max(a, 0) * p.ad.b_adapter[s] + local * p.ad.b_row[s];
  float sum = 0.f;
  for (int r = 0; r < rank; ++r) sum = fmaf(S[r], act_to_float(w[r], bf), sum);
  p.Y[row * p.ldy + j] = p.base[row * p.ldb + j] + sum;
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

int64_t adapters_workspace_bytes(const seedlm_adapters& ad, int M, const DeviceInfo&) {
  return (int64_t)M * ad.slices * ad.rank * 4;
}

int launch_adapters_apply(const seedlm_adapters& ad, const int32_t* plan, int M, const uint16_t* X, int64_t ldx,
                          const float* base, int64_t ldb, float* Y, int64_t ldy, void* workspace, cudaStream_t stream,
                          const DeviceInfo&) {
  ApplyArgs p{ad, plan, M, X, ldx, base, ldb, Y, ldy, static_cast<float*>(workspace)};
  const unsigned grid = (unsigned)(max_tiles(M, ad.n) * adapter_tile_rows(M));
  int total = 0;
  for (int s = 0; s < ad.slices; ++s) total += ad.rows[s];
  int rc = launch_pdl(adapters_shrink_kernel, dim3(grid, ad.slices), 256, 0, stream, p);
  if (rc) return rc;
  return launch_pdl(adapters_expand_kernel, dim3(grid, (total + 255) / 256), 256, 0, stream, p, total, (int)(base == Y));
}

int read_and_clear_plan_mismatch(unsigned int* out) {
  unsigned int v = 0, zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_plan_mismatch, sizeof(v));
  if (err == cudaSuccess && v) err = cudaMemcpyToSymbol(g_plan_mismatch, &zero, sizeof(zero));
  *out = v;
  return record_cuda_error(err);
}

}  // namespace seedlm
