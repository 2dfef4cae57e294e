// block_norm.cu -- the end of one block and the start of the next:
//   v = norm_post(y);  h' = h_scale h + y_scale gate v;  x = norm_pre(h')
// and the gated activation X = act(G) U between two products.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "launch.cuh"
#include "seedlm_device.cuh"
#include "seedlm_internal.h"

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

// Sum over the CTA, in a fixed order, to every thread.
__device__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
  return s;
}

struct NormArgs {
  seedlm_norm nm;
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

struct Stats {
  float mean, rstd;
};

template <class F>
__device__ Stats row_stats(F value, const seedlm_norm& nm, float* red) {
  Stats st{0.f, 1.f};
  const float inv = 1.f / nm.cols;
  if (nm.kind == SEEDLM_NORM_LAYER) {
    float s = 0.f;
    for (int j = threadIdx.x; j < nm.cols; j += blockDim.x) s += value(j);
    st.mean = block_sum(s, red) * inv;
  }
  float s = 0.f;
  for (int j = threadIdx.x; j < nm.cols; j += blockDim.x) {
    const float d = value(j) - st.mean;
    s = fmaf(d, d, s);
  }
  st.rstd = rsqrtf(block_sum(s, red) * inv + nm.eps);
  return st;
}

__device__ __forceinline__ float normed(float v, Stats st, const seedlm_norm& nm, const void* w, const void* b, int j) {
  v = (v - st.mean) * st.rstd;
  if (w) v *= nm.weight_offset + load_as(w, j, nm.dtype);
  if (b) v += load_as(b, j, nm.dtype);
  return v;
}

// One CTA a row; the row is read again for every step.
__global__ void __launch_bounds__(256) block_norm_kernel(const NormArgs p) {
  __shared__ float red[32];
  grid_launch_dependents();
  grid_wait();
  const int64_t m = blockIdx.x;
  const seedlm_norm& nm = p.nm;
  Stats post{}, pre{};
  auto y = [&](int j) { return p.y[m * p.ldy + j]; };
  if (p.y && nm.post) post = row_stats(y, nm, red);
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
  if (p.x && nm.pre) pre = row_stats(hnew, nm, red);
  for (int j = threadIdx.x; j < nm.cols; j += blockDim.x) {
    const float r = hnew(j);
    if (p.h_out) store_as(p.h_out, m * p.ldho + j, p.h_dtype, r);
    if (p.x) store_as(p.x, m * p.ldx + j, p.x_dtype, nm.pre ? normed(r, pre, nm, nm.w_pre, nm.b_pre, j) : r);
  }
}

__device__ __forceinline__ float activate(float g, int act) {
  if (act == SEEDLM_SILU) return g / (1.f + expf(-g));
  if (act == SEEDLM_GELU) return 0.5f * g * (1.f + erff(g * 0.70710678f));
  return 0.5f * g * (1.f + tanhf(0.79788456f * (g + 0.044715f * g * g * g)));
}

__global__ void __launch_bounds__(256) glu_kernel(int cols, int act, const float* __restrict__ GU, int64_t ldgu, void* X,
                                                  int64_t ldx, int x_dtype) {
  grid_launch_dependents();
  grid_wait();
  const int64_t m = blockIdx.x;
  for (int j = threadIdx.x; j < cols; j += blockDim.x)
    store_as(X, m * ldx + j, x_dtype, activate(GU[m * ldgu + j], act) * GU[m * ldgu + cols + j]);
}

}  // namespace

int launch_block_norm(const seedlm_norm& nm, int M, const float* y, int64_t ldy, const void* gate, int64_t ldg,
                      const void* h, int64_t ldh, void* h_out, int64_t ldho, int h_dtype, void* x, int64_t ldx,
                      int x_dtype, cudaStream_t stream, const DeviceInfo&) {
  NormArgs p{nm, y, ldy, gate, ldg, h, ldh, h_out, ldho, h_dtype, x, ldx, x_dtype};
  return launch_pdl(block_norm_kernel, M, 256, 0, stream, p);
}

int launch_glu(int M, int cols, int act, const float* GU, int64_t ldgu, void* X, int64_t ldx, int x_dtype,
               cudaStream_t stream, const DeviceInfo&) {
  return launch_pdl(glu_kernel, M, 256, 0, stream, cols, act, GU, ldgu, X, ldx, x_dtype);
}

}  // namespace seedlm
