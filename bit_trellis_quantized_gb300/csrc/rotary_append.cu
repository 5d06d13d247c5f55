// Rotation of a step's queries and keys by their positions, and append of its
// keys and values to a paged cache.
//
// A pair (x, y) of frequency f at position p turns by a = p f:
//   (c (x cos a - y sin a), c (x sin a + y cos a)),
// in f32, rounded once. a counts in turns: p times the frequency as a 64-bit
// fraction of a turn, the whole turns dropped by the product's overflow, so
// that an angle at any position is as good as one near 0 (p f in f32 is off by
// 2^-7 at 131072).
//
// Bound: the read of the step's values and the one write. A lane takes 16
// values of a head, 8 pairs or two times 8 values; a warp the heads of a token
// (or a part of them, where tokens are few), so that a lane's cosines and sines
// serve all of them. Measured, 16 heads on 2 key heads of 256, 64 values turned,
// f32 to fp16: one token 3.1 us, 250 tokens 4.9, 32000 tokens 147 us, 6.7 TB/s.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr int kRaWarps = 4;

template <int SRC>
__device__ __forceinline__ void ra_load8(const void* base, long long at, float (&x)[8]) {
    if (SRC == 3) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = p[0], b = p[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = SRC == 1 ? h2f_bits(ws[i] & 0xFFFFu) : bf2f_bits(ws[i] & 0xFFFFu);
            x[2 * i + 1] = SRC == 1 ? h2f_bits(ws[i] >> 16) : bf2f_bits(ws[i] >> 16);
        }
    }
}
template <int DT>
__device__ __forceinline__ void ra_store8(uint16_t* to, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == 1) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp: one token's heads part, part + parts, ... in passes of 32 / (D / 16) heads; the heads are q's, k's, v's.
template <int SRC, int DT, int D>
__global__ void __launch_bounds__(kRaWarps * 32) rotary_append_kernel(RotaryArgs a, int parts) {
    constexpr int kUnits = D / 16, kHeads = 32 / kUnits;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kRaWarps + (threadIdx.x >> 5);
    const int t = static_cast<int>(item / parts), part = static_cast<int>(item % parts);
    if (t >= a.T) return;
    // the token's sequence: the last s with at[s] <= t, in rounds of 32 places
    int lo = 0, span = a.n;  // it is in [lo, lo + span)
    while (span > 1) {
        const int step = (span + 31) / 32, i = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < span && a.at[i] <= t);
        const int k = m ? 31 - __clz(m) : 0;
        span = min(step, span - k * step);
        lo += k * step;
    }
    const int first = a.at[lo], end = a.at[lo + 1];
    if (t < first || t >= end) return;  // of no sequence
    const long long pos = (long long)a.lens[lo] - (min(end, a.T) - max(first, 0)) + (t - max(first, 0));
    long long row = -1;  // of the pools, at key head 0
    if (pos >= 0 && pos < (long long)a.max_pages * a.page) {
        const int p = static_cast<int>(pos / a.page);
        const int pg = a.table[(long long)lo * a.max_pages + p];
        if (static_cast<unsigned>(pg) < static_cast<unsigned>(a.n_pages))
            row = (long long)pg * a.Hkv * a.page + (pos - (long long)p * a.page);
    }
    const int u = lane % kUnits;
    const bool turn = u * 16 < a.rot;
    float c[8], s[8];
    if (turn) {
        const long long at = a.positions ? a.positions[t] : pos;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const long long part_of = static_cast<long long>(static_cast<unsigned long long>(at) * a.turns[u * 8 + i]);
            sincospif(__ll2float_rn(part_of) * 0x1p-63f, &s[i], &c[i]);
            c[i] *= a.factor, s[i] *= a.factor;
        }
    }
    // the lane's two runs of 8 values
    const bool halves = turn && !a.interleaved;
    const int d0 = halves ? u * 8 : u * 16, d1 = halves ? d0 + a.rot / 2 : d0 + 8;
    const int Hq = a.q ? a.Hq : 0, heads = Hq + 2 * a.Hkv;
    for (int h = part * kHeads + lane / kUnits; h < heads; h += parts * kHeads) {
        const void* src;
        uint16_t* dst;
        long long from;
        if (h < Hq) {
            src = a.q, from = (long long)t * a.q_ld + h * D;
            dst = static_cast<uint16_t*>(a.q_out) + ((long long)t * a.Hq + h) * D;
        } else {
            if (row < 0) continue;
            const bool is_k = h < Hq + a.Hkv;
            const int kh = h - Hq - (is_k ? 0 : a.Hkv);
            src = is_k ? a.k : a.v, from = (long long)t * (is_k ? a.k_ld : a.v_ld) + kh * D;
            dst = static_cast<uint16_t*>(is_k ? a.k_pool : a.v_pool) + (row + (long long)kh * a.page) * D;
        }
        float x[8], y[8];
        ra_load8<SRC>(src, from + d0, x);
        ra_load8<SRC>(src, from + d1, y);
        if (turn && h < Hq + a.Hkv) {
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = x[2 * i], y0 = y[2 * i];
                    x[2 * i] = x0 * c[i] - x[2 * i + 1] * s[i], x[2 * i + 1] = x0 * s[i] + x[2 * i + 1] * c[i];
                    y[2 * i] = y0 * c[i + 4] - y[2 * i + 1] * s[i + 4], y[2 * i + 1] = y0 * s[i + 4] + y[2 * i + 1] * c[i + 4];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x0 = x[i];
                    x[i] = x0 * c[i] - y[i] * s[i], y[i] = x0 * s[i] + y[i] * c[i];
                }
            }
        }
        ra_store8<DT>(dst + d0, x);
        ra_store8<DT>(dst + d1, y);
    }
}

template <int SRC, int DT>
cudaError_t ra_launch(const RotaryArgs& a, cudaStream_t s) {
    const void* f = a.d == 64    ? reinterpret_cast<const void*>(rotary_append_kernel<SRC, DT, 64>)
                    : a.d == 128 ? reinterpret_cast<const void*>(rotary_append_kernel<SRC, DT, 128>)
                                 : reinterpret_cast<const void*>(rotary_append_kernel<SRC, DT, 256>);
    const int per = 512 / a.d, passes = ((a.q ? a.Hq : 0) + 2 * a.Hkv + per - 1) / per;
    int parts = 1;
    // Few tokens: a token's heads go to several warps. 16 heads of 256 on 2 key heads, f32: 250 tokens whole 7.0 us, in 10 parts
    // 5.3; 1000 tokens 8.0 and 10.4; 4000 tokens 22 and 30.
    while (parts < passes && (long long)a.T * parts < kSms * 6) parts *= 2;
    parts = parts < passes ? parts : passes;
    const long long items = (long long)a.T * parts;
    void* args[] = {const_cast<RotaryArgs*>(&a), &parts};
    return launch_kernel(f, dim3(static_cast<unsigned>((items + kRaWarps - 1) / kRaWarps)), dim3(kRaWarps * 32), 0, true, s, args);
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryArgs& a, int src_dtype, int dtype, cudaStream_t s) {
    if (dtype == 1) return src_dtype == 3 ? ra_launch<3, 1>(a, s) : ra_launch<1, 1>(a, s);
    return src_dtype == 3 ? ra_launch<3, 2>(a, s) : ra_launch<2, 2>(a, s);
}

}  // namespace escha
