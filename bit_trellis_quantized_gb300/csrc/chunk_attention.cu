// Attention of a chunk of new tokens over a paged key-value cache.
//
// Token t of sequence s stands at position p = lens[s] - (at[s + 1] - at[s]) +
// t - at[s]; per query head, over the keys j <= p of its key head:
//   x_j = scale q . k_j,  m = max_j x_j,  out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
//   lse = m + ln sum_j e^(x_j - m).
//
// A warp takes one (token, query head), a lane d / 32 values, key by key; 64
// keys are summed by themselves, then added to the rest, so that many small
// weights count beside a large one.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr int kCaWarps = 4;

template <int DT, int D>
__global__ void __launch_bounds__(kCaWarps * 32) chunk_attention_kernel(ChunkAttnArgs a) {
    constexpr int kV = D / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kCaWarps + (threadIdx.x >> 5);
    const int t = static_cast<int>(item / a.Hq), h = static_cast<int>(item % a.Hq);
    if (t >= a.T) return;
    int lo = 0, span = a.n;
    while (span > 1) {
        const int step = (span + 31) / 32, i = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < span && a.at[i] <= t);
        const int k = m ? 31 - __clz(m) : 0;
        span = min(step, span - k * step);
        lo += k * step;
    }
    const int first = max(a.at[lo], 0), end = min(a.at[lo + 1], a.T);
    if (t < first || t >= end) return;  // of no sequence
    const long long pos = (long long)a.lens[lo] - (end - first) + (t - first);
    const long long cap = min((long long)a.max_pages * a.page, (long long)a.max_len);
    const int keys = static_cast<int>(max(0ll, min(pos + 1, cap)));
    const int kvh = h / (a.Hq / a.Hkv);
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((long long)t * a.Hq + h) * D;
    float qv[kV], acc[kV], sum[kV], m = -INFINITY, l = 0.f, part = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) qv[i] = load_act(q, lane + 32 * i, DT), acc[i] = sum[i] = 0.f;
    for (int j = 0; j < keys; ++j) {
        const int p = j / a.page, pg = a.table[(long long)lo * a.max_pages + p];
        if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.n_pages)) continue;
        const long long row = (((long long)pg * a.Hkv + kvh) * a.page + (j - p * a.page)) * D;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) x += qv[i] * load_act(a.k_pool, row + lane + 32 * i, DT);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        x *= a.scale;
        const float top = fmaxf(m, x), base = top == -INFINITY ? 0.f : top;
        const float corr = expf(m - base), w = expf(x - base);
        m = top, l *= corr, part = part * corr + w;
#pragma unroll
        for (int i = 0; i < kV; ++i) sum[i] *= corr, acc[i] = acc[i] * corr + w * load_act(a.v_pool, row + lane + 32 * i, DT);
        if (j % 64 == 63) {
            l += part, part = 0.f;
#pragma unroll
            for (int i = 0; i < kV; ++i) sum[i] += acc[i], acc[i] = 0.f;
        }
    }
    l += part;
    uint16_t* out = static_cast<uint16_t*>(a.out) + ((long long)t * a.Hq + h) * D;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const float y = l == 0.f ? 0.f : (sum[i] + acc[i]) / l;
        out[lane + 32 * i] = DT == 1 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
    }
    if (a.lse && lane == 0) a.lse[(long long)t * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t chunk_attention_ws_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, int dtype, void*, cudaStream_t s) {
    const void* fs[2][3] = {{reinterpret_cast<const void*>(chunk_attention_kernel<1, 64>),
                             reinterpret_cast<const void*>(chunk_attention_kernel<1, 128>),
                             reinterpret_cast<const void*>(chunk_attention_kernel<1, 256>)},
                            {reinterpret_cast<const void*>(chunk_attention_kernel<2, 64>),
                             reinterpret_cast<const void*>(chunk_attention_kernel<2, 128>),
                             reinterpret_cast<const void*>(chunk_attention_kernel<2, 256>)}};
    const long long items = (long long)a.T * a.Hq;
    void* args[] = {const_cast<ChunkAttnArgs*>(&a)};
    return launch_kernel(fs[dtype - 1][a.d / 128], dim3(static_cast<unsigned>((items + kCaWarps - 1) / kCaWarps)),
                         dim3(kCaWarps * 32), 0, true, s, args);
}

}  // namespace escha
