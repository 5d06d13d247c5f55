// Internal launch interfaces of the token mixers (paged attention of one new
// token, gated delta rule) and of the token log probabilities, between the
// C-ABI layer (escha_api.cu) and their kernels. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace escha {

// SMs of the GPU this library is built for: grids and splits go by it, so that
// workspace sizes and the order of sums depend on the sizes of a call alone.
constexpr int kSms = 152;

struct PagedAttnArgs {
    const void* q;         // [B][Hq][d]
    void* k_pool;          // [n_pages][Hkv][page][d]
    void* v_pool;
    const int32_t* table;  // [B][max_pages]
    const int32_t* lens;   // [B]
    const void* k_new;     // [B][Hkv][d] or null
    const void* v_new;
    void* out;   // [B][Hq][d]
    float* lse;  // [B][Hq] or null
    int B, Hq, Hkv, d, page, n_pages, max_pages, max_len;
    float scale;
};
size_t paged_attention_ws_bytes(int B, int Hq, int Hkv, int d, int max_len);
cudaError_t launch_paged_attention(const PagedAttnArgs& a, int dtype, void* ws, cudaStream_t s);

struct DeltaArgs {
    const void* q;      // [T][Hk][dk]
    const void* k;      // [T][Hk][dk]
    const void* v;      // [T][Hv][dv]
    const float* g;     // [T][Hv] log decay
    const float* beta;  // [T][Hv]
    float* state;       // [n][Hv][dk][dv], updated
    const int32_t* at;  // [n + 1] first token of each sequence
    void* out;          // [T][Hv][dv]
    int n, T, Hk, Hv, dk, dv, max_len;
    float scale, eps;
};
size_t delta_rule_ws_bytes(int dtype, int n, int T, int Hk, int Hv, int dk, int dv, int max_len);
cudaError_t launch_delta_rule(const DeltaArgs& a, int dtype, void* ws, cudaStream_t s);

struct LogprobArgs {
    const void* logits;  // [M] rows of V values, ld values apart
    const int32_t* ids;  // [M][n_ids]
    float* logprobs;     // [M][n_ids]
    float* entropy;      // [M] or null
    float* lse;          // [M] or null
    int32_t* top_ids;    // [M][top]
    float* top_logprobs;
    long long ld;
    int M, V, n_ids, top;
};
constexpr int kLogprobMaxTop = 32;
size_t token_logprobs_ws_bytes(int M, int V);
cudaError_t launch_token_logprobs(const LogprobArgs& a, int dtype, void* ws, cudaStream_t s);

}  // namespace escha
