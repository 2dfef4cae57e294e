// block_norm.cu -- the end of one block and the start of the next:
//   v = norm_post(y);  h' = h_scale h + y_scale gate v;  x = norm_pre(h')
// and the gated activation X = act(G) U between two products.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.cuh"
#include "seedlm_device.cuh"
#include "between_internal.h"

namespace seedlm {

SEEDLM_CHECK_FLAG(block_norm)

namespace {

__device__ __forceinline__ float load_as(const void* p, int64_t i, int dtype) {
  if (dtype == SEEDLM_F32) return static_cast<const float*>(p)[i];
  return act_to_float(static_cast<const uint16_t*>(p)[i], dtype == SEEDLM_BF16);
}

__device__ __forceinline__ void store_as(void* p, int64_t i, int dtype, float v) {
  if (dtype == SEEDLM_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == SEEDLM_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float2 two_of(uint32_t w, bool bf16) {
  return bf16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u))
              : __half22float2(reinterpret_cast<const __half2&>(w));
}

__device__ __forceinline__ uint32_t two_to(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return reinterpret_cast<const uint32_t&>(v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(v);
}

// Sum over the CTA to every thread, in a fixed order; `red` holds a float for
// each warp and is used by one sum at a time.
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < warps ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct NormArgs {
  seedlm_norm nm;
  int M;
  const float* y;
  int64_t ldy;
  const void* gate;
  int64_t ldg;
  const void* h;
  int64_t ldh;
  void* h_out;
  int64_t ldho;
  int h_dtype;
  void* x;
  int64_t ldx;
  int x_dtype;
};

// The 16-bit type of a call: 0 fp16, 1 bf16, 2 only known element by element.
template <int T16>
__device__ __forceinline__ bool is_bf16(int dtype) {
  return T16 == 2 ? dtype == SEEDLM_BF16 : T16 == 1;
}

// A thread's share of a row: NV groups of four elements, neighbouring ones
// (VEC) or, where rows are not aligned for that, ones a CTA's width apart.  The
// type is looked at once for a share, so that all its loads are in flight
// together.
template <int NV, bool VEC, int T16 = 2, bool FULL = false>
struct Share {
  __device__ static int index(int i, int k) {
    return VEC ? 4 * ((int)threadIdx.x + (int)blockDim.x * i) + k : (int)threadIdx.x + (int)blockDim.x * (4 * i + k);
  }
  // Whether the element lies in the row; FULL: the CTA's threads end with it.
  __device__ static bool in(int i, int k, int cols) { return FULL || index(i, k) < cols; }
  // 16-bit elements as they are stored; zeros beyond the row.
  __device__ static void load16(const void* p, int64_t row, int cols, uint2 (&raw)[NV]) {
    const uint16_t* from = static_cast<const uint16_t*>(p) + row;
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        raw[i] = in(i, 0, cols) ? *reinterpret_cast<const uint2*>(from + index(i, 0)) : make_uint2(0u, 0u);
    } else {
      uint16_t e[NV][4];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) e[i][k] = in(i, k, cols) ? from[index(i, k)] : (uint16_t)0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        raw[i] = make_uint2(e[i][0] | (uint32_t)e[i][1] << 16, e[i][2] | (uint32_t)e[i][3] << 16);
    }
  }
  __device__ static void load32(const void* p, int64_t row, int cols, float (&v)[NV][4]) {
    const float* from = static_cast<const float*>(p) + row;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (VEC) {
        const float4 a = in(i, 0, cols) ? *reinterpret_cast<const float4*>(from + index(i, 0)) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = in(i, k, cols) ? from[index(i, k)] : 0.f;
      }
    }
  }
  __device__ static void widen(const uint2 (&raw)[NV], bool bf16, float (&v)[NV][4]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float2 lo = two_of(raw[i].x, bf16), hi = two_of(raw[i].y, bf16);
      v[i][0] = lo.x, v[i][1] = lo.y, v[i][2] = hi.x, v[i][3] = hi.y;
    }
  }
  __device__ static void store(void* p, int64_t row, int cols, int dtype, const float (&v)[NV][4]) {
    if (dtype == SEEDLM_F32) {
      float* to = static_cast<float*>(p) + row;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (VEC) {
          if (in(i, 0, cols))
            *reinterpret_cast<float4*>(to + index(i, 0)) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (in(i, k, cols)) to[index(i, k)] = v[i][k];
        }
    } else {
      uint16_t* to = static_cast<uint16_t*>(p) + row;
      const bool bf16 = is_bf16<T16>(dtype);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint2 a = make_uint2(two_to(v[i][0], v[i][1], bf16), two_to(v[i][2], v[i][3], bf16));
        if (VEC) {
          if (in(i, 0, cols)) *reinterpret_cast<uint2*>(to + index(i, 0)) = a;
        } else {
          const uint32_t w[2] = {a.x, a.y};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (in(i, k, cols)) to[index(i, k)] = (uint16_t)(w[k / 2] >> (16 * (k % 2)));
        }
      }
    }
  }
};

// A share of some type, asked for early and used late: 16-bit elements wait in
// registers as they are; fp32 ones would take too many and are loaded when used.
template <int NV, bool VEC, int T16 = 2, bool FULL = false>
struct Early {
  using S = Share<NV, VEC, T16, FULL>;
  uint2 raw[NV];
  __device__ void ask(const void* p, int64_t row, int cols, int dtype) {
    if (p && dtype != SEEDLM_F32) S::load16(p, row, cols, raw);
  }
  __device__ void use(const void* p, int64_t row, int cols, int dtype, float (&v)[NV][4]) const {
    if (dtype != SEEDLM_F32) S::widen(raw, is_bf16<T16>(dtype), v);
    else S::load32(p, row, cols, v);
  }
};

// v <- norm(v), all but weights and bias; two passes over registers.
template <class S, int NV>
__device__ __forceinline__ void normalise(float (&v)[NV][4], const seedlm_norm& nm, float* red) {
  const float inv = 1.f / nm.cols;
  if (nm.kind == SEEDLM_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s += (v[i][0] + v[i][1]) + (v[i][2] + v[i][3]);
    const float mean = block_sum(s, red) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] = S::in(i, k, nm.cols) ? v[i][k] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    s += fmaf(v[i][0], v[i][0], v[i][1] * v[i][1]) + fmaf(v[i][2], v[i][2], v[i][3] * v[i][3]);
  const float rstd = rsqrtf(block_sum(s, red + 32) * inv + nm.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[i][k] *= rstd;
}

template <class E, int NV>
__device__ __forceinline__ void weigh(float (&v)[NV][4], const seedlm_norm& nm, const void* w, const void* b,
                                      const E& early_w) {
  float t[NV][4];
  if (w) {
    early_w.use(w, 0, nm.cols, nm.dtype, t);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] *= nm.weight_offset + t[i][k];
  }
  if (b) {
    E late;
    late.ask(b, 0, nm.cols, nm.dtype);
    late.use(b, 0, nm.cols, nm.dtype, t);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] += t[i][k];
  }
}

// One CTA a row, which stays in registers: y and h are read once, h' and x
// written once.  For few rows, where latency counts (a row of 8192, 3.3 us), and
// for any number of rows of 8193 to 16384 (2048 of 16384, both norms, bf16: 85 us
// for 336 MB; nothing of the next row is on its way).  Unaligned rows of that
// width spill 236 bytes at 64 registers.
constexpr int kRowThreads = 1024;

template <int NV, bool VEC>
__global__ void __launch_bounds__(kRowThreads) block_norm_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[4][32];  // one place for each sum of a row
  const seedlm_norm& nm = p.nm;
  const int cols = nm.cols;
  const int64_t m = blockIdx.x;
  using S = Share<NV, VEC>;
  if (!SEEDLM_IN_BOUNDS(g_check_flag, m, p.M)) return;
  grid_launch_dependents();
  grid_wait();
  float v[NV][4], h[NV][4];
  Early<NV, VEC> w, stream, gate;
  if (p.y) {
    S::load32(p.y, m * p.ldy, cols, v);
    gate.ask(p.gate, m * p.ldg, cols, nm.dtype);
    if (nm.post) w.ask(nm.w_post, 0, cols, nm.dtype);
  }
  stream.ask(p.h, m * p.ldh, cols, p.h_dtype);
  if (p.y) {
    if (nm.post) {
      normalise<S>(v, nm, red[0]);
      weigh(v, nm, nm.w_post, nm.b_post, w);
    }
    if (p.gate) {
      gate.use(p.gate, m * p.ldg, cols, nm.dtype, h);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] *= h[i][k];
    }
  }
  if (p.h) stream.use(p.h, m * p.ldh, cols, p.h_dtype, h);
  if (p.x && nm.pre) w.ask(nm.w_pre, 0, cols, nm.dtype);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = p.h ? nm.h_scale * h[i][k] : 0.f;
      v[i][k] = p.y ? fmaf(nm.y_scale, v[i][k], a) : a;
    }
  if (p.h_out) S::store(p.h_out, m * p.ldho, cols, p.h_dtype, v);
  if (!p.x) return;
  if (nm.pre) {
    normalise<S>(v, nm, red[2]);
    weigh(v, nm, nm.w_pre, nm.b_pre, w);
  }
  S::store(p.x, m * p.ldx, cols, p.x_dtype, v);
}

// Many rows: each CTA goes through rows a grid apart, with the next row coming
// into shared memory while it sums up this one, so that memory is not left idle.
// A thread copies exactly what it will itself read, as soon as it has taken the
// row before out of the same place, so the copies need no barrier.  256 threads
// hold a row of 8192; the CTAs of an SM wait for their sums in turn.  4096 rows
// of 8192, both norms, bf16: 63 us (5.3 TB/s), 85 with a CTA for each row; bound
// by its instructions (2.4 issued a clock) and the two sums of a row.  Every form
// spills, 24 to 72 bytes at 128 registers.
constexpr int kStreamGroups = 8, kStreamThreads = 256, kStreamSums = 2 * 4 * 32 * 4;

// Asynchronous copy of 8 or 16 bytes to shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
}

template <bool H32, int T16, bool FULL>
__global__ void __launch_bounds__(kStreamThreads, 2)
block_norm_stream_kernel(const __grid_constant__ NormArgs p, int M) {
  constexpr int NV = kStreamGroups, HB = H32 ? 16 : 8;
  extern __shared__ __align__(16) unsigned char shared[];
  float(*red)[4][32] = reinterpret_cast<float(*)[4][32]>(shared);  // [2]: sums of this row and the next
  const seedlm_norm& nm = p.nm;
  const int cols = nm.cols, threads = blockDim.x;
  using S = Share<NV, true, T16, FULL>;
  using E = Early<NV, true, T16, FULL>;
  const bool pre = p.x && nm.pre, post = p.y && nm.post, gates = p.y && p.gate;
  const bool gate_row = gates && p.ldg != 0 && nm.dtype != SEEDLM_F32;  // others are read when used
  // Places of this thread's groups of y, h and gate.
  unsigned char* y_at = shared + kStreamSums + threadIdx.x * 16;
  unsigned char* h_at = shared + kStreamSums + NV * threads * 16 + threadIdx.x * HB;
  unsigned char* g_at = shared + kStreamSums + NV * threads * (16 + HB) + threadIdx.x * 8;
  if (!SEEDLM_IN_BOUNDS(g_check_flag, kStreamSums + NV * threads * (16 + HB + (gate_row ? 8 : 0)) - 1,
                        seedlm_dynamic_smem_bytes()))
    return;
  auto fetch_y = [&](int64_t m) {
    if (p.y && m < M) {
      const float* from = p.y + m * p.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (S::in(i, 0, cols)) copy_async<16>(y_at + i * threads * 16, from + S::index(i, 0));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch_rest = [&](int64_t m) {
    if (p.h && m < M) {
      const unsigned char* from = static_cast<const unsigned char*>(p.h) + m * p.ldh * (HB / 4);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (S::in(i, 0, cols)) copy_async<HB>(h_at + i * threads * HB, from + S::index(i, 0) * (HB / 4));
    }
    if (gate_row && m < M) {
      const uint16_t* from = static_cast<const uint16_t*>(p.gate) + m * p.ldg;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (S::in(i, 0, cols)) copy_async<8>(g_at + i * threads * 8, from + S::index(i, 0));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Takes the 16-bit groups at `at` (zeros beyond the row).
  auto take16 = [&](const unsigned char* at, bool bf16, float (&v)[NV][4]) {
    uint2 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      raw[i] = S::in(i, 0, cols) ? *reinterpret_cast<const uint2*>(at + i * threads * 8) : make_uint2(0u, 0u);
    S::widen(raw, bf16, v);
  };
  auto take32 = [&](const unsigned char* at, float (&v)[NV][4]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float4 a = S::in(i, 0, cols) ? *reinterpret_cast<const float4*>(at + i * threads * 16) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
    }
  };
  grid_launch_dependents();
  grid_wait();
  fetch_y(blockIdx.x);
  fetch_rest(blockIdx.x);
  int parity = 0;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x, parity ^= 1) {
    float v[NV][4], t[NV][4];
    E w;
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (p.y) {
      take32(y_at, v);
      fetch_y(m + gridDim.x);
      if (post) {
        w.ask(nm.w_post, 0, cols, nm.dtype);
        normalise<S>(v, nm, red[parity][0]);
        weigh(v, nm, nm.w_post, nm.b_post, w);
      }
    } else {
      fetch_y(M);
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (gates) {
      if (gate_row) {
        take16(g_at, is_bf16<T16>(nm.dtype), t);
      } else {
        E late;
        late.ask(p.gate, m * p.ldg, cols, nm.dtype);
        late.use(p.gate, m * p.ldg, cols, nm.dtype, t);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] *= t[i][k];
    }
    if (p.h) {
      if (H32) take32(h_at, t);
      else take16(h_at, is_bf16<T16>(p.h_dtype), t);
    }
    fetch_rest(m + gridDim.x);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = p.h ? nm.h_scale * t[i][k] : 0.f;
        v[i][k] = p.y ? fmaf(nm.y_scale, v[i][k], a) : a;
      }
    if (p.h_out) S::store(p.h_out, m * p.ldho, cols, H32 ? SEEDLM_F32 : p.h_dtype, v);
    if (!p.x) continue;
    if (pre) {
      w.ask(nm.w_pre, 0, cols, nm.dtype);
      normalise<S>(v, nm, red[parity][2]);
      weigh(v, nm, nm.w_pre, nm.b_pre, w);
    }
    S::store(p.x, m * p.ldx, cols, p.x_dtype, v);
  }
}

// Many rows that are not aligned for groups of four: each row comes into shared
// memory as the 16-byte words it lies across, and every thread takes E elements a
// CTA's width apart from there.  The copies of the next row go out as soon as all
// threads have taken this one (the barrier inside a sum tells).  The CTA is as
// wide as leaves only a thread's last element to be checked against the row's
// end: threads * (E - 1) < cols <= threads * E.  1000 rows of 5001, layer norms, a
// gate for each row: 33 us, 49 with a CTA a row that reads elements one by one;
// bound by the latency of a row's four sums.
constexpr int kRaggedThreads = 512;

template <bool H32, int E>
__global__ void __launch_bounds__(E >= 16 ? 256 : kRaggedThreads, E >= 16 ? 2 : 1)
block_norm_ragged_kernel(const __grid_constant__ NormArgs p, int M) {
  extern __shared__ __align__(16) unsigned char shared[];
  float(*red)[4][32] = reinterpret_cast<float(*)[4][32]>(shared);  // [2]: sums of this row and the next
  const seedlm_norm& nm = p.nm;
  const int cols = nm.cols, tid = threadIdx.x, threads = blockDim.x;
  constexpr int HB = H32 ? 4 : 2;
  const bool pre = p.x && nm.pre, post = p.y && nm.post, gates = p.y && p.gate;
  const bool gate_row = gates && p.ldg != 0 && nm.dtype != SEEDLM_F32;  // others are read when used
  unsigned char* y_image = shared + kStreamSums;
  unsigned char* h_image = y_image + (cols * 4 + 47) / 16 * 16;
  unsigned char* g_image = h_image + (cols * HB + 47) / 16 * 16;
  if (!SEEDLM_IN_BOUNDS(g_check_flag, g_image - shared + (gate_row ? (cols * 2 + 47) / 16 * 16 : 0) - 1,
                        seedlm_dynamic_smem_bytes()))
    return;
  // Row m of a matrix of M rows, `size` bytes an element.
  auto fetch = [&](unsigned char* image, const void* matrix, int64_t ld, int size, int64_t m) {
    const unsigned char* first = static_cast<const unsigned char*>(matrix);
    const unsigned char* end = first + ((M - 1) * ld + cols) * size;
    const unsigned char* row = first + m * ld * size;
    const int lead = (int)(reinterpret_cast<uintptr_t>(row) & 15), words = (lead + cols * size + 15) / 16;
    const unsigned char* from = row - lead;
    for (int c = tid; c < words; c += threads) {
      if (from + 16 * c >= first && from + 16 * c + 16 <= end) {
        copy_async<16>(image + 16 * c, from + 16 * c);
      } else {  // a word that leaves the matrix: what of it is in the row
        for (int o = 0; o < 16; o += 2)
          if (16 * c + o >= lead && 16 * c + o < lead + cols * size)
            *reinterpret_cast<uint16_t*>(image + 16 * c + o) = *reinterpret_cast<const uint16_t*>(from + 16 * c + o);
      }
    }
  };
  auto image_of = [](unsigned char* image, const void* matrix, int64_t ld, int size, int64_t m) {
    return image + ((reinterpret_cast<uintptr_t>(matrix) + m * ld * size) & 15);
  };
  auto fetch_y = [&](int64_t m) {
    if (p.y && m < M) fetch(y_image, p.y, p.ldy, 4, m);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch_rest = [&](int64_t m) {
    if (p.h && m < M) fetch(h_image, p.h, p.ldh, HB, m);
    if (gate_row && m < M) fetch(g_image, p.gate, p.ldg, 2, m);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto index = [&](int e) { return tid + threads * e; };
  auto in = [&](int e) { return e < E - 1 || index(e) < cols; };
  auto clamped = [&](int e) { return e < E - 1 ? index(e) : min(index(e), cols - 1); };
  const float inv = 1.f / cols;
  // As normalise(), over this mapping; `taken` runs after the first barrier.
  auto normalised = [&](float (&v)[E], float* sums, auto taken) {
    bool told = false;
    if (nm.kind == SEEDLM_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += v[e];
      const float mean = block_sum(s, sums) * inv;
      taken();
      told = true;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = in(e) ? v[e] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(v[e], v[e], s);
    const float rstd = rsqrtf(block_sum(s, sums + 32) * inv + nm.eps);
    if (!told) taken();
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= rstd;
  };
  // v <- f(v, a) with a's elements of this thread; all loads before the first
  // use, the type looked at once.  Beyond the row its last element stands in.
  auto with = [&](float (&v)[E], const void* a, int dtype, auto f) {
    if (dtype == SEEDLM_F32) {
      float t[E];
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = static_cast<const float*>(a)[clamped(e)];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = f(v[e], t[e]);
    } else {
      uint16_t t[E];
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = static_cast<const uint16_t*>(a)[clamped(e)];
      if (dtype == SEEDLM_BF16) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = f(v[e], __uint_as_float((uint32_t)t[e] << 16));
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = f(v[e], __half2float(__ushort_as_half(t[e])));
      }
    }
  };
  auto weighed = [&](float (&v)[E], const void* w, const void* b) {
    if (w) with(v, w, nm.dtype, [&](float v, float w) { return v * (nm.weight_offset + w); });
    if (b) with(v, b, nm.dtype, [](float v, float b) { return v + b; });
  };
  // Beyond the row: zeros, as the sums need them.
  auto cut = [&](float (&v)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (!in(e)) v[e] = 0.f;
  };
  auto put = [&](void* to, int64_t row, int dtype, const float (&v)[E]) {
    if (dtype == SEEDLM_F32) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (in(e)) static_cast<float*>(to)[row + index(e)] = v[e];
    } else if (dtype == SEEDLM_BF16) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (in(e)) static_cast<__nv_bfloat16*>(to)[row + index(e)] = __float2bfloat16_rn(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (in(e)) static_cast<__half*>(to)[row + index(e)] = __float2half_rn(v[e]);
    }
  };
  grid_launch_dependents();
  grid_wait();
  fetch_y(blockIdx.x);
  fetch_rest(blockIdx.x);
  int parity = 0;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x, parity ^= 1) {
    float v[E];
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    if (p.y) {
      const float* y = reinterpret_cast<const float*>(image_of(y_image, p.y, p.ldy, 4, m));
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = in(e) ? y[index(e)] : 0.f;
    }
    auto next_y = [&]() { fetch_y(m + gridDim.x); };
    if (post) {
      normalised(v, red[parity][0], next_y);
      weighed(v, nm.w_post, nm.b_post);
    } else {
      __syncthreads();
      next_y();
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    if (gates) {
      const void* g = gate_row ? image_of(g_image, p.gate, p.ldg, 2, m)
                               : static_cast<const unsigned char*>(p.gate) + m * p.ldg * (nm.dtype == SEEDLM_F32 ? 4 : 2);
      with(v, g, nm.dtype, [](float v, float g) { return v * g; });
    }
    if (p.h) {
      if (!p.y) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
      }
      with(v, image_of(h_image, p.h, p.ldh, HB, m), H32 ? SEEDLM_F32 : p.h_dtype,
           [&](float v, float h) { return fmaf(nm.y_scale, v, nm.h_scale * h); });
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= nm.y_scale;
    }
    cut(v);
    auto next_rest = [&]() { fetch_rest(m + gridDim.x); };
    if (p.h_out) put(p.h_out, m * p.ldho, H32 ? SEEDLM_F32 : p.h_dtype, v);
    if (pre) {
      normalised(v, red[parity][2], next_rest);
      weighed(v, nm.w_pre, nm.b_pre);
    } else {
      __syncthreads();
      next_rest();
    }
    if (p.x) put(p.x, m * p.ldx, p.x_dtype, v);
  }
}

// Rows too wide for the registers of a CTA: the row is read again for every
// step.
constexpr int kWideThreads = 1024;

struct Stats {
  float mean, rstd;
};

template <class F>
__device__ Stats row_stats(F value, const seedlm_norm& nm, float* red) {
  Stats st{0.f, 1.f};
  const float inv = 1.f / nm.cols;
  if (nm.kind == SEEDLM_NORM_LAYER) {
    float s = 0.f;
    for (int j = threadIdx.x; j < nm.cols; j += kWideThreads) s += value(j);
    st.mean = block_sum(s, red) * inv;
  }
  float s = 0.f;
  for (int j = threadIdx.x; j < nm.cols; j += kWideThreads) {
    const float d = value(j) - st.mean;
    s = fmaf(d, d, s);
  }
  st.rstd = rsqrtf(block_sum(s, red + 32) * inv + nm.eps);
  return st;
}

__device__ __forceinline__ float normed(float v, Stats st, const seedlm_norm& nm, const void* w, const void* b, int j) {
  v = (v - st.mean) * st.rstd;
  if (w) v *= nm.weight_offset + load_as(w, j, nm.dtype);
  if (b) v += load_as(b, j, nm.dtype);
  return v;
}

__global__ void __launch_bounds__(kWideThreads) block_norm_wide_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[4][32];
  grid_launch_dependents();
  grid_wait();
  const int64_t m = blockIdx.x;
  if (!SEEDLM_IN_BOUNDS(g_check_flag, m, p.M)) return;
  const seedlm_norm& nm = p.nm;
  Stats post{}, pre{};
  auto y = [&](int j) { return p.y[m * p.ldy + j]; };
  if (p.y && nm.post) post = row_stats(y, nm, red[0]);
  auto hnew = [&](int j) {
    float r = p.h ? nm.h_scale * load_as(p.h, m * p.ldh + j, p.h_dtype) : 0.f;
    if (p.y) {
      float v = y(j);
      if (nm.post) v = normed(v, post, nm, nm.w_post, nm.b_post, j);
      if (p.gate) v *= load_as(p.gate, m * p.ldg + j, nm.dtype);
      r = fmaf(nm.y_scale, v, r);
    }
    return r;
  };
  if (p.x && nm.pre) pre = row_stats(hnew, nm, red[2]);
  for (int j = threadIdx.x; j < nm.cols; j += kWideThreads) {
    const float r = hnew(j);
    if (p.h_out) store_as(p.h_out, m * p.ldho + j, p.h_dtype, r);
    if (p.x) store_as(p.x, m * p.ldx + j, p.x_dtype, nm.pre ? normed(r, pre, nm, nm.w_pre, nm.b_pre, j) : r);
  }
}

// ---------------------------------------------------------------------- glu

// The larger part of erf GELU's work: g/2 (1 + erf(g / sqrt 2)) = max(g, 0) -
// |g| Q(|g|) with Q(m) = erfc(m / sqrt 2) / 2, which keeps the relative accuracy
// of the negative tail, where the sum cancels.  Q(m) = e^(-m^2/2) t P(t), t =
// 1 / (1 + 0.35 m), the form of Hastings' approximations (Abramowitz and Stegun
// 7.1.26); P is a minimax fit of degree 8, made in 64 bits for m up to 13.3 (where
// e^(-m^2/2) leaves fp32), off by 3.2e-8 at most.  With the roundings of fp32, of
// the reciprocal and of the exponential GELU is off by less than (g^2 + 9) 2^-23
// of its value below 0.  2048 x 14336: 43 us, 60 with erfcf, 44 with
// 1 + erff(g / sqrt 2), which is 10 % off at -5.
__device__ __forceinline__ float gelu(float g) {
  const float m = fminf(fabsf(g), 30.f);  // Q is 0 from there on, at infinity too
  const float t = __fdividef(1.f, fmaf(0.35f, m, 1.f));
  float p = -0.029114645f;
  p = fmaf(p, t, 0.143816575f);
  p = fmaf(p, t, -0.255387127f);
  p = fmaf(p, t, 0.158792019f);
  p = fmaf(p, t, -0.0228402093f);
  p = fmaf(p, t, 0.105390742f);
  p = fmaf(p, t, 0.119863458f);
  p = fmaf(p, t, 0.139857516f);
  p = fmaf(p, t, 0.13962166f);
  const float q = t * p * __expf(-0.5f * m * m);
  return fmaf(-m, q, g < 0.f ? 0.f : g);  // (NaN stays)
}

// The sigmoid form of the tanh one: (1 + tanh z) / 2 = 1 / (1 + e^-2z).
template <int ACT>
__device__ __forceinline__ float activate(float g) {
  if (ACT == SEEDLM_SILU) return g / (1.f + __expf(-g));
  if (ACT == SEEDLM_GELU) return gelu(g);
  return g / (1.f + __expf(-1.5957691f * (g + 0.044715f * g * g * g)));
}

// Bound by memory: 2048 x 14336 in 44 us (6.7 TB/s).  Narrow rows share a CTA: a
// CTA costs more to start than they do (3168 rows of 200: 6.6 us, 18.1 with one each).
// Unaligned rows go element by element: 4096 x 1001 takes 18 us for 41 MB.
constexpr int kGluThreads = 256, kGluGroups = 2;  // groups of four outputs a thread

template <int ACT, bool VEC, bool NARROW>
__global__ void __launch_bounds__(kGluThreads)
glu_kernel(int M, int cols, int chunks, const float* GU, int64_t ldgu, void* X, int64_t ldx, int x_dtype) {
  grid_launch_dependents();
  const int64_t m = NARROW ? (int64_t)(blockIdx.x / chunks) * blockDim.y + threadIdx.y : blockIdx.x / chunks;
  const int threads = NARROW ? blockDim.x : kGluThreads, first = (int)(blockIdx.x % chunks) * (4 * threads * kGluGroups);
  const float* G = GU + m * ldgu;
  grid_wait();
  if (NARROW && m >= M) return;
  __align__(16) float g[kGluGroups][4], u[kGluGroups][4];
#pragma unroll
  for (int i = 0; i < kGluGroups; ++i) {
    const int j = first + (VEC ? 4 : 1) * (int)threadIdx.x + 4 * threads * i;
    if (VEC) {
      if (j < cols) {
        *reinterpret_cast<float4*>(g[i]) = *reinterpret_cast<const float4*>(G + j);
        *reinterpret_cast<float4*>(u[i]) = *reinterpret_cast<const float4*>(G + cols + j);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + threads * k < cols) {
          g[i][k] = G[j + threads * k];
          u[i][k] = G[cols + j + threads * k];
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kGluGroups; ++i) {
    const int j = first + (VEC ? 4 : 1) * (int)threadIdx.x + 4 * threads * i;
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = activate<ACT>(g[i][k]) * u[i][k];
    if (VEC) {
      const bool bf16 = x_dtype == SEEDLM_BF16;
      if (j < cols)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(X) + m * ldx + j) =
            make_uint2(two_to(v[0], v[1], bf16), two_to(v[2], v[3], bf16));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + threads * k < cols) store_as(X, m * ldx + j + threads * k, x_dtype, v[k]);
    }
  }
}

// Whether rows can be read or written four elements at a time.
bool rows_of_four(const void* p, int64_t ld, int dtype) {
  return !p || (aligned(p, dtype == SEEDLM_F32 ? 16 : 8) && ld % 4 == 0);
}

template <int NV>
int launch_rows(const NormArgs& p, int M, int threads, bool vec, cudaStream_t stream) {
  return vec ? launch_pdl(block_norm_kernel<NV, true>, M, threads, 0, stream, p)
             : launch_pdl(block_norm_kernel<NV, false>, M, threads, 0, stream, p);
}

template <bool H32, int T16>
int launch_stream(const NormArgs& p, int M, cudaStream_t stream, const DeviceInfo& dev) {
  const int cols = p.nm.cols;
  const int threads = ((cols / 4 + kStreamGroups - 1) / kStreamGroups + 31) / 32 * 32;
  const int smem = kStreamSums + kStreamGroups * threads * (16 + (H32 ? 16 : 8) + (p.y && p.gate && p.ldg != 0 ? 8 : 0));
  auto kernel = cols == 4 * kStreamGroups * threads ? block_norm_stream_kernel<H32, T16, true>
                                                    : block_norm_stream_kernel<H32, T16, false>;
  const int rc = allow_max_smem((const void*)kernel, dev);
  if (rc) return rc;
  // As many CTAs as an SM holds at 128 registers a thread.
  const int ctas = std::max(1, std::min(2 * kStreamThreads / threads, 227 * 1024 / (smem + 1024)));
  return launch_pdl(kernel, std::min<int64_t>(M, (int64_t)ctas * dev.num_sms), threads, (size_t)smem, stream, p, M);
}

template <bool H32, int E>
int launch_ragged(const NormArgs& p, int M, int threads, cudaStream_t stream, const DeviceInfo& dev) {
  const int cols = p.nm.cols;
  const int smem = kStreamSums + (cols * 4 + 47) / 16 * 16 + (cols * (H32 ? 4 : 2) + 47) / 16 * 16 +
                   (p.y && p.gate && p.ldg != 0 ? (cols * 2 + 47) / 16 * 16 : 0);
  auto kernel = block_norm_ragged_kernel<H32, E>;
  const int rc = allow_max_smem((const void*)kernel, dev);
  if (rc) return rc;
  // As many CTAs as an SM holds at 128 registers a thread.
  const int ctas = std::max(1, std::min(512 / threads, 227 * 1024 / (smem + 1024)));
  return launch_pdl(kernel, std::min<int64_t>(M, (int64_t)ctas * dev.num_sms), threads, (size_t)smem, stream, p, M);
}

// Threads for E elements each (see above); 0: there is no such width.
int ragged_threads(int cols, int E, int most) {
  const int threads = ((cols + E - 1) / E + 31) / 32 * 32;
  return threads * (E - 1) < cols && threads <= most ? threads : 0;
}

// SEEDLM_EUNSUPPORTED: no width suits these rows.
template <bool H32>
int launch_ragged_of(const NormArgs& p, int M, cudaStream_t stream, const DeviceInfo& dev) {
  const int cols = p.nm.cols;
  if (const int t = ragged_threads(cols, 32, 256)) return launch_ragged<H32, 32>(p, M, t, stream, dev);
  if (const int t = ragged_threads(cols, 24, 256)) return launch_ragged<H32, 24>(p, M, t, stream, dev);
  if (const int t = ragged_threads(cols, 16, 256)) return launch_ragged<H32, 16>(p, M, t, stream, dev);
  if (const int t = ragged_threads(cols, 12, 512)) return launch_ragged<H32, 12>(p, M, t, stream, dev);
  if (const int t = ragged_threads(cols, 8, 512)) return launch_ragged<H32, 8>(p, M, t, stream, dev);
  if (const int t = ragged_threads(cols, 4, 512)) return launch_ragged<H32, 4>(p, M, t, stream, dev);
  return SEEDLM_EUNSUPPORTED;
}

template <int ACT>
int launch_glu_act(int M, int cols, const float* GU, int64_t ldgu, void* X, int64_t ldx, int x_dtype,
                   cudaStream_t stream) {
  const bool vec = cols % 4 == 0 && rows_of_four(GU, ldgu, SEEDLM_F32) && rows_of_four(X, ldx, x_dtype);
  const int narrow = (cols + 127) / 128 * 32, rows = std::max(1, kGluThreads / narrow);
  const int threads = rows > 1 ? narrow : kGluThreads;
  const int64_t chunks = (cols + 4LL * threads * kGluGroups - 1) / (4 * threads * kGluGroups);
  const int64_t grid = ((int64_t)M + rows - 1) / rows * chunks;
  if (grid > INT32_MAX) return SEEDLM_EUNSUPPORTED;
  auto kernel = rows > 1 ? (vec ? glu_kernel<ACT, true, true> : glu_kernel<ACT, false, true>)
                         : (vec ? glu_kernel<ACT, true, false> : glu_kernel<ACT, false, false>);
  return launch_pdl(kernel, (unsigned)grid, dim3(threads, rows), 0, stream, M, cols, (int)chunks, GU, ldgu, X, ldx, x_dtype);
}

}  // namespace

int launch_block_norm(const seedlm_norm& nm, int M, const float* y, int64_t ldy, const void* gate, int64_t ldg,
                      const void* h, int64_t ldh, void* h_out, int64_t ldho, int h_dtype, void* x, int64_t ldx,
                      int x_dtype, cudaStream_t stream, const DeviceInfo& dev) {
  NormArgs p{nm, M, y, ldy, gate, ldg, h, ldh, h_out, ldho, h_dtype, x, ldx, x_dtype};
  const int cols = nm.cols, groups = (cols + 3) / 4;
  if (groups > 4 * kRowThreads) return launch_pdl(block_norm_wide_kernel, M, kWideThreads, 0, stream, p);
  const int64_t m1 = M > 1;  // the leading dimension of one row does not count
  const bool vec = cols % 4 == 0 && rows_of_four(y, m1 * ldy, SEEDLM_F32) && rows_of_four(gate, m1 * ldg, nm.dtype) &&
                   rows_of_four(h, m1 * ldh, h_dtype) && rows_of_four(h_out, m1 * ldho, h_dtype) &&
                   rows_of_four(x, m1 * ldx, x_dtype) && rows_of_four(nm.w_post, 0, nm.dtype) &&
                   rows_of_four(nm.b_post, 0, nm.dtype) && rows_of_four(nm.w_pre, 0, nm.dtype) &&
                   rows_of_four(nm.b_pre, 0, nm.dtype);
  // Few rows: as many threads as there are, for the latency of one row.  Many:
  // fewer threads with more of a row each, and the next row on its way.
  if (M > 2 * dev.num_sms && groups <= kStreamGroups * kStreamThreads) {
    const bool h32 = (h || h_out) && h_dtype == SEEDLM_F32;
    if (!vec) {
      const int rc = h32 ? launch_ragged_of<true>(p, M, stream, dev) : launch_ragged_of<false>(p, M, stream, dev);
      if (rc != SEEDLM_EUNSUPPORTED) return rc;
    }
    // The one 16-bit type of the call, if it has one.
    int t16 = x ? x_dtype : SEEDLM_F32;
    for (int t : {h || h_out ? h_dtype : SEEDLM_F32, nm.dtype})
      if (t != SEEDLM_F32) t16 = t16 == SEEDLM_F32 || t16 == t ? t : 3;
    if (vec && t16 == SEEDLM_F16)
      return h32 ? launch_stream<true, 0>(p, M, stream, dev) : launch_stream<false, 0>(p, M, stream, dev);
    if (vec && t16 == SEEDLM_BF16)
      return h32 ? launch_stream<true, 1>(p, M, stream, dev) : launch_stream<false, 1>(p, M, stream, dev);
    if (vec) return h32 ? launch_stream<true, 2>(p, M, stream, dev) : launch_stream<false, 2>(p, M, stream, dev);
  }
  int nv = 1;
  while (groups > nv * kRowThreads) nv *= 2;
  const int threads = ((groups + nv - 1) / nv + 31) / 32 * 32;
  return nv == 1   ? launch_rows<1>(p, M, threads, vec, stream)
         : nv == 2 ? launch_rows<2>(p, M, threads, vec, stream)
                   : launch_rows<4>(p, M, threads, vec, stream);
}

int launch_glu(int M, int cols, int act, const float* GU, int64_t ldgu, void* X, int64_t ldx, int x_dtype,
               cudaStream_t stream, const DeviceInfo&) {
  return act == SEEDLM_SILU   ? launch_glu_act<SEEDLM_SILU>(M, cols, GU, ldgu, X, ldx, x_dtype, stream)
         : act == SEEDLM_GELU ? launch_glu_act<SEEDLM_GELU>(M, cols, GU, ldgu, X, ldx, x_dtype, stream)
                              : launch_glu_act<SEEDLM_GELU_TANH>(M, cols, GU, ldgu, X, ldx, x_dtype, stream);
}

}  // namespace seedlm
