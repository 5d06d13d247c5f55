// Internal launch interfaces of the token mixers (paged attention of one new
// token and of a chunk of tokens, the append that precedes it, gated delta
// rule), of the token log probabilities and the adjusted logits, between the
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

struct RotaryArgs {
    const void* q;  // [T][Hq][d], q_ld values a token, or null
    const void* k;  // [T][Hkv][d]
    const void* v;
    long long q_ld, k_ld, v_ld;
    const uint64_t* turns;     // [rot / 2]: 2^64ths of a turn a position
    const int32_t* positions;  // [T] or null
    void* q_out;               // [T][Hq][d] or null
    void* k_pool;              // [n_pages][Hkv][page][d]
    void* v_pool;
    const int32_t* table;  // [n][max_pages]
    const int32_t* at;     // [n + 1]
    const int32_t* lens;   // [n]
    int n, T, Hq, Hkv, d, rot, interleaved, page, n_pages, max_pages;
    float factor;
};
cudaError_t launch_rotary_append(const RotaryArgs& a, int src_dtype, int dtype, cudaStream_t s);

struct ChunkAttnArgs {
    const void* q;         // [T][Hq][d]
    const void* k_pool;    // [n_pages][Hkv][page][d]
    const void* v_pool;
    const int32_t* table;  // [n][max_pages]
    const int32_t* at;     // [n + 1]
    const int32_t* lens;   // [n]
    void* out;             // [T][Hq][d]
    float* lse;            // [T][Hq] or null
    int n, T, Hq, Hkv, d, page, n_pages, max_pages, max_len;
    float scale;
    int backwards;  // CTA i has the i-th unit from the last one on (tests)
    int polls;      // after which a wait for a tile's work gives up
};
size_t chunk_attention_ws_bytes(int n, int T, int Hq, int Hkv, int d, int max_len);
cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, int dtype, void* ws, cudaStream_t s);

struct AdjustArgs {
    const void* logits;  // [M] rows of V values, ld values apart
    void* out;           // the same, out_ld apart
    const int32_t* ids;  // [n_ids]: row m's are at[m] <= i < at[m + 1], the first prompt[m] of them the prompt's
    const int32_t* at;
    const int32_t* prompt;
    const float* repetition;  // [M] or null
    const float* frequency;
    const float* presence;
    const int32_t* bias_ids;  // [n_bias]
    const float* bias;
    const int32_t* bias_at;  // [M + 1]
    const int32_t* allowed;  // [n_masks][ceil(V / 32)] or null
    const int32_t* allowed_rows;
    long long ld, out_ld;
    int M, V, n_ids, n_bias, n_masks;
};
cudaError_t launch_adjust_logits(const AdjustArgs& a, int dtype, cudaStream_t s);

}  // namespace escha
