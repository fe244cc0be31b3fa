// mxq_layer.h -- launch interface between the C-ABI layer (api.cu) and the
// kernels of the attention half of a layer: linear.cu, cache.cu, attention.cu.
// Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mxq.h"

namespace mxq {

// Product of a few tokens with quantized weights; T, N >= 1, K >= 32, K % 32 == 0.
constexpr int64_t kLinearMaxTokens = 2048;
constexpr int64_t kLinearMaxWidth = 65536;     // K
struct LinearArgs {
    const uint16_t *x;
    int64_t T, K, N;
    const uint8_t *codes, *scales;
    const float *s2;
    void *y;
    uint32_t *status;
    uint32_t *xh;               // workspace: f16 rows [T, K] and a factor for each
    float *xf;
};
size_t linear_rows_bytes(int64_t T, int64_t K);     // of xh
size_t linear_workspace_bytes(int64_t T, int64_t K);
cudaError_t launch_linear(const LinearArgs &a, int fmt, int out_f32, cudaStream_t s);

// A cache and a batch of sequences, as the kernels take them.
constexpr int64_t kMaxSeqs = 4096;
struct CacheView {
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const float *k_s2, *v_s2;
    uint32_t pages, heads, page_log;
    const int32_t *cu, *lens, *table;
    uint32_t seqs, width;
    uint32_t *status;
};
cudaError_t launch_cache_write(const CacheView &c, int fmt, int dim, int four_six, const uint16_t *k, int64_t k_stride,
                               const uint16_t *v, int64_t v_stride, uint32_t T, cudaStream_t s);
cudaError_t launch_cache_read(const CacheView &c, int fmt, int dim, uint32_t T, uint16_t *k, uint16_t *v,
                              cudaStream_t s);

struct AttentionCall {
    CacheView c;
    const uint16_t *q;
    int64_t q_stride;
    uint32_t T, heads, max_new;
    float scale;
    uint16_t *o;
    float *lse;
    void *workspace;
};
size_t attention_workspace_bytes(int64_t group, int64_t head_dim, int64_t max_new);
cudaError_t launch_attention(const AttentionCall &a, int fmt, int dim, cudaStream_t s);

} // namespace mxq
