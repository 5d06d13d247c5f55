// Attention of one new token a sequence over a paged key-value cache.
//
// Per sequence b and query head h, over the keys j < lens[b] of its key head:
//   x_j = scale q . k_j,  out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
//   lse = m + ln sum_j e^(x_j - m),  m = max_j x_j.
// Parts over different keys join by their (m, sum, weighted values). Scores,
// maxima, sums and weighted values are held in f32; the one rounding is that
// of `out` to its 16-bit type.
//
// First form: one CTA per (sequence, key head, 256 keys); a second kernel joins
// a sequence's parts.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr int kPaThreads = 256;
constexpr int kPaKeys = 256;
constexpr int kPaMaxGroup = 16;

template <int DT>
__device__ __forceinline__ float pa_f32(const void* p, long long i) {
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return DT == 1 ? h2f_bits(b) : bf2f_bits(b);
}
template <int DT>
__device__ __forceinline__ uint16_t pa_bits(float v) {
    return DT == 1 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ int pa_len(const PagedAttnArgs& a, int b) {
    const long long cap = static_cast<long long>(a.max_pages) * a.page;
    const int most = a.max_len < cap ? a.max_len : static_cast<int>(cap);
    return max(0, min(a.lens[b], most));
}

template <int DT>
__global__ void __launch_bounds__(kPaThreads) paged_attention_kernel(PagedAttnArgs a, int splits, int tiles, float* part) {
    __shared__ float qs[kPaMaxGroup][256];
    __shared__ float xs[kPaMaxGroup][kPaKeys];
    __shared__ long long row[kPaKeys];
    __shared__ float ms[kPaMaxGroup], ls[kPaMaxGroup];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int split = blockIdx.x, b = blockIdx.z, kvh = blockIdx.y / tiles, tile = blockIdx.y % tiles;
    const int group = a.Hq / a.Hkv, h0 = kvh * group + tile * kPaMaxGroup, nh = min(kPaMaxGroup, group - tile * kPaMaxGroup);
    const int len = pa_len(a, b), j0 = split * kPaKeys, n = min(kPaKeys, len - j0);
    if (n <= 0) return;
    for (int i = t; i < nh * a.d; i += kPaThreads)
        qs[i / a.d][i % a.d] = pa_f32<DT>(a.q, ((long long)b * a.Hq + h0) * a.d + i) * a.scale;
    for (int i = t; i < n; i += kPaThreads) {
        const int j = j0 + i, pg = a.table[(long long)b * a.max_pages + j / a.page];
        row[i] = pg >= 0 && pg < a.n_pages ? (((long long)pg * a.Hkv + kvh) * a.page + j % a.page) * a.d : -1;
    }
    __syncthreads();
    if (a.k_new && j0 + n == len && row[n - 1] >= 0 && tile == 0) {
        for (int i = t; i < a.d; i += kPaThreads) {
            const long long src = ((long long)b * a.Hkv + kvh) * a.d + i;
            static_cast<uint16_t*>(a.k_pool)[row[n - 1] + i] = static_cast<const uint16_t*>(a.k_new)[src];
            static_cast<uint16_t*>(a.v_pool)[row[n - 1] + i] = static_cast<const uint16_t*>(a.v_new)[src];
        }
    }
    for (int i = warp; i < n; i += kPaThreads / 32) {
        const bool fresh = a.k_new && j0 + i == len - 1;
        const void* src = fresh ? a.k_new : a.k_pool;
        const long long at = fresh ? ((long long)b * a.Hkv + kvh) * a.d : row[i];
        for (int h = 0; h < nh; ++h) {
            float s = 0.f;
            if (row[i] >= 0)
                for (int e = lane; e < a.d; e += 32) s += qs[h][e] * pa_f32<DT>(src, at + e);
            for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            if (lane == 0) xs[h][i] = row[i] >= 0 ? s : -INFINITY;
        }
    }
    __syncthreads();
    for (int h = warp; h < nh; h += kPaThreads / 32) {
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, xs[h][i]);
        for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        for (int i = lane; i < n; i += 32) {
            const float p = m == -INFINITY ? 0.f : expf(xs[h][i] - m);
            xs[h][i] = p;
            l += p;
        }
        for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
        if (lane == 0) ms[h] = m, ls[h] = l;
    }
    __syncthreads();
    for (int e = t; e < a.d; e += kPaThreads) {
        float acc[kPaMaxGroup] = {};
        for (int i = 0; i < n; ++i) {
            if (row[i] < 0) continue;
            const bool fresh = a.k_new && j0 + i == len - 1;
            const float v = fresh ? pa_f32<DT>(a.v_new, ((long long)b * a.Hkv + kvh) * a.d + e) : pa_f32<DT>(a.v_pool, row[i] + e);
            for (int h = 0; h < kPaMaxGroup; ++h)
                if (h < nh) acc[h] += xs[h][i] * v;
        }
        for (int h = 0; h < kPaMaxGroup; ++h)
            if (h < nh) part[(((long long)b * a.Hq + h0 + h) * splits + split) * (a.d + 2) + 2 + e] = acc[h];
    }
    if (t < nh) {
        float* p = part + (((long long)b * a.Hq + h0 + t) * splits + split) * (a.d + 2);
        p[0] = ms[t], p[1] = ls[t];
    }
}

template <int DT>
__global__ void __launch_bounds__(256) paged_attention_join_kernel(PagedAttnArgs a, int splits, const float* part) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y, h = blockIdx.x, e = threadIdx.x;
    const int used = (pa_len(a, b) + kPaKeys - 1) / kPaKeys;
    const float* p = part + ((long long)b * a.Hq + h) * splits * (a.d + 2);
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int i = 0; i < used; ++i) m = fmaxf(m, p[(long long)i * (a.d + 2)]);
    for (int i = 0; i < used; ++i) {
        const float* r = p + (long long)i * (a.d + 2);
        if (r[1] == 0.f) continue;
        const float f = expf(r[0] - m);
        l += f * r[1];
        if (e < a.d) acc += f * r[2 + e];
    }
    if (e < a.d)
        static_cast<uint16_t*>(a.out)[((long long)b * a.Hq + h) * a.d + e] = pa_bits<DT>(l == 0.f ? 0.f : acc / l);
    if (e == 0 && a.lse) a.lse[(long long)b * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

int pa_splits(int max_len) { return (max_len + kPaKeys - 1) / kPaKeys; }

}  // namespace

size_t paged_attention_ws_bytes(int B, int Hq, int Hkv, int d, int max_len) {
    (void)Hkv;
    return static_cast<size_t>(B) * Hq * pa_splits(max_len) * (d + 2) * 4;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, int dtype, void* ws, cudaStream_t s) {
    int splits = pa_splits(a.max_len), tiles = (a.Hq / a.Hkv + kPaMaxGroup - 1) / kPaMaxGroup;
    float* part = static_cast<float*>(ws);
    void* args[] = {const_cast<PagedAttnArgs*>(&a), &splits, &tiles, &part};
    const void* f = dtype == 1 ? reinterpret_cast<const void*>(paged_attention_kernel<1>)
                               : reinterpret_cast<const void*>(paged_attention_kernel<2>);
    cudaError_t e = launch_kernel(f, dim3(splits, a.Hkv * tiles, a.B), dim3(kPaThreads), 0, true, s, args);
    if (e != cudaSuccess) return e;
    void* jargs[] = {const_cast<PagedAttnArgs*>(&a), &splits, &part};
    f = dtype == 1 ? reinterpret_cast<const void*>(paged_attention_join_kernel<1>)
                   : reinterpret_cast<const void*>(paged_attention_join_kernel<2>);
    return launch_kernel(f, dim3(a.Hq, a.B), dim3(256), 0, true, s, jargs);
}

}  // namespace escha
