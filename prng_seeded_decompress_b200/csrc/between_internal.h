// between_internal.h -- host-side declarations of what runs between the
// products of a decoder layer: low-rank adapters, block norms, the gated
// activation.
#pragma once

#include "seedlm_internal.h"

namespace seedlm {

int read_and_clear_check_adapters(unsigned int* out);
int read_and_clear_check_block_norm(unsigned int* out);

// Low-rank adapters (adapters.cu): the plan of a batch, the workspace of one
// projection and its launches; arguments checked by the entry points.
constexpr int kMaxAdapterRows = 1 << 24;
int64_t adapters_plan_words(int M, int n);
int launch_adapters_plan(int M, int n, const int32_t* ids, int32_t* plan, cudaStream_t stream,
                         const DeviceInfo& dev);
int64_t adapters_workspace_bytes(const seedlm_adapters& ad, int M, const DeviceInfo& dev);
int launch_adapters_apply(const seedlm_adapters& ad, const int32_t* plan, int M, const uint16_t* X,
                          int64_t ldx, const float* base, int64_t ldb, float* Y, int64_t ldy,
                          void* workspace, cudaStream_t stream, const DeviceInfo& dev);
int read_and_clear_plan_mismatch(unsigned int* out);
int read_and_clear_adapters_error(unsigned int* out);
// Block boundary and gated activation (block_norm.cu).
int launch_block_norm(const seedlm_norm& nm, int M, const float* y, int64_t ldy, const void* gate,
                      int64_t ldg, const void* h, int64_t ldh, void* h_out, int64_t ldho,
                      int h_dtype, void* x, int64_t ldx, int x_dtype, cudaStream_t stream,
                      const DeviceInfo& dev);
int launch_glu(int M, int cols, int act, const float* GU, int64_t ldgu, void* X, int64_t ldx,
               int x_dtype, cudaStream_t stream, const DeviceInfo& dev);

}  // namespace seedlm
