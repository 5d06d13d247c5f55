// Penalties for repeated tokens, biases and grammar masks on logits.
//
// Per row and token i, in this order, in f32, each operation rounded, the
// result rounded once to its type:
//   among the row's ids:             x = x > 0 ? x / repetition : x repetition
//   c > 0 times behind the prompt:   x = x - (frequency c + presence)
//   each bias of i, in list order:   x = x + bias
//   not allowed by the row's mask:   x = -infinity
//
// A CTA takes 8192 tokens of a row and holds a word for each of them in shared
// memory: how often the row's ids name it, and whether they do at all, as
// whole-number sums, which come out alike in any order. Then one pass reads
// what is to be changed (everything, where the result goes to another buffer),
// all a thread's next loads at once, and writes it.
//
// Bound: the write of the banned and the changed logits, and the read of those
// next to them. Slices of 32 KB let five CTAs share a multiprocessor, so that
// one's counting runs beside another's pass.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

#include <limits.h>

namespace escha {

namespace {

constexpr int kAlThreads = 256;
constexpr int kAlSlice = 8192;  // tokens of a CTA at most
constexpr int kAlList = 512;    // biases of a slice in shared memory
constexpr uint32_t kAlPrompt = 1u << 30, kAlBias = 1u << 31;  // the rest counts

template <int DT>
struct AlVec;
template <>
struct AlVec<3> {
    static constexpr int kN = 4;
    using type = float;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct AlVec<1> {
    static constexpr int kN = 8;
    using type = uint16_t;
    static __device__ __forceinline__ float get(uint16_t x) { return h2f_bits(x); }
    static __device__ __forceinline__ uint16_t put(float x) { return __half_as_ushort(__float2half_rn(x)); }
};
template <>
struct AlVec<2> {
    static constexpr int kN = 8;
    using type = uint16_t;
    static __device__ __forceinline__ float get(uint16_t x) { return bf2f_bits(x); }
    static __device__ __forceinline__ uint16_t put(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};

template <int DT>
__global__ void __launch_bounds__(kAlThreads, 5) adjust_logits_kernel(AdjustArgs a, int slices) {
    using A = AlVec<DT>;
    using E = typename A::type;
    constexpr int kN = A::kN, kGroups = 16 / kN;  // of a thread at once
    __shared__ __align__(16) uint32_t words[kAlSlice];
    __shared__ uint32_t masks[kAlSlice / 32 + 2];
    __shared__ int list_n, list_at[kAlList], list_token[kAlList];  // biases: their places and tokens of the slice
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x, row = blockIdx.x / slices;
    const E* x = static_cast<const E*>(a.logits) + row * a.ld;
    E* y = static_cast<E*>(a.out) + row * a.out_ld;
    // Groups of kN values begin where `x` is aligned: group g is [g kN - skew, g kN - skew + kN).
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(E) % kN);
    const bool vec = reinterpret_cast<uintptr_t>(y) / sizeof(E) % kN == static_cast<uintptr_t>(skew);
    const int base = static_cast<int>(blockIdx.x % slices) * kAlSlice - skew;  // token of words[0]
    const int i0 = a.ids ? min(max(a.at[row], 0), a.n_ids) : 0, i1 = a.ids ? min(max(a.at[row + 1], 0), a.n_ids) : 0;
    const int b0 = a.bias_ids ? min(max(a.bias_at[row], 0), a.n_bias) : 0, b1 = a.bias_ids ? min(max(a.bias_at[row + 1], 0), a.n_bias) : 0;
    const int mrow = !a.allowed ? -1 : a.allowed_rows ? a.allowed_rows[row] : row, mwords = (a.V + 31) / 32;
    const bool masked = static_cast<unsigned>(mrow) < static_cast<unsigned>(a.n_masks), copy = a.logits != a.out, counts = i0 < i1 || b0 < b1;
    if (!masked && !copy && !counts) return;
    if (masked) {  // masks[0] holds the token max(base, 0)
        const uint32_t* m = reinterpret_cast<const uint32_t*>(a.allowed) + static_cast<long long>(mrow) * mwords;
        for (int i = t; i < kAlSlice / 32 + 2; i += kAlThreads) masks[i] = max(base, 0) / 32 + i < mwords ? m[max(base, 0) / 32 + i] : 0u;
    }
    if (counts) {
#pragma unroll
        for (int i = 0; i < kAlSlice / (kAlThreads * 4); ++i) *reinterpret_cast<uint4*>(words + (i * kAlThreads + t) * 4) = make_uint4(0, 0, 0, 0);
        if (t == 0) list_n = 0;
        __syncthreads();
        const long long late = static_cast<long long>(i0) + (a.prompt ? max(a.prompt[row], 0) : 0);
#pragma unroll 4
        for (int i = i0 + t; i < i1; i += kAlThreads) {
            const int id = a.ids[i];
            const uint32_t w = static_cast<uint32_t>(id) - static_cast<uint32_t>(base);
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.V) || w >= kAlSlice) continue;
            if (i >= late) atomicAdd(&words[w], 1u);
            else atomicOr(&words[w], kAlPrompt);
        }
        for (int i = b0 + t; i < b1; i += kAlThreads) {
            const int id = a.bias_ids[i];
            const uint32_t w = static_cast<uint32_t>(id) - static_cast<uint32_t>(base);
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.V) || w >= kAlSlice) continue;
            atomicOr(&words[w], kAlBias);
            const int at = atomicAdd(&list_n, 1);
            if (at < kAlList) list_at[at] = i, list_token[at] = static_cast<int>(w);
        }
    }
    __syncthreads();
    const float rep = a.repetition ? a.repetition[row] : 1.f, freq = a.frequency ? a.frequency[row] : 0.f;
    const float pres = a.presence ? a.presence[row] : 0.f;
#pragma unroll 1
    for (int p = 0; p < kAlSlice / (kAlThreads * 16); ++p) {
        if (base + p * 16 * kAlThreads >= a.V) break;
        // of each group: the allowed tokens and the touched ones, a bit each, and its values
        uint32_t open[kGroups], touched[kGroups];
        __align__(16) E v[kGroups][kN];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int w0 = ((p * kGroups + k) * kAlThreads + t) * kN, g0 = base + w0;
            const int lo = g0 < 0 ? -g0 : 0, hi = min(max(a.V - g0, 0), kN);
            const uint32_t all = hi > lo ? ((1u << hi) - 1) & ~((1u << lo) - 1) : 0u;
            open[k] = all, touched[k] = 0;
            if (masked) {
                const int at = g0 + lo - max(base, 0) / 32 * 32;
                open[k] = all & (__funnelshift_r(masks[at / 32], masks[at / 32 + 1], at & 31) << lo);
            }
            if (counts) {
#pragma unroll
                for (int e = 0; e < kN; e += 4) {
                    const uint4 n = *reinterpret_cast<const uint4*>(words + w0 + e);
                    touched[k] |= ((n.x != 0) | (n.y != 0) << 1 | (n.z != 0) << 2 | (n.w != 0) << 3) << e;
                }
                touched[k] &= open[k];
            }
            touched[k] |= (all & ~open[k]) << 16;  // and the banned ones
            if (copy ? all != 0 : touched[k] != 0 && open[k] != 0) {
                if (all == (1u << kN) - 1) *reinterpret_cast<uint4*>(v[k]) = *reinterpret_cast<const uint4*>(x + g0);
                else
#pragma unroll
                    for (int e = 0; e < kN; ++e)
                        if (all >> e & 1) v[k][e] = x[g0 + e];
            }
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int w0 = ((p * kGroups + k) * kAlThreads + t) * kN, g0 = base + w0;
            const uint32_t ban = touched[k] >> 16, all = open[k] | ban;
            if (copy ? all == 0 : touched[k] == 0) continue;
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                if (ban >> e & 1) v[k][e] = A::put(-INFINITY);
                if (!(touched[k] >> e & 1)) continue;
                const uint32_t n = words[w0 + e], c = n & (kAlPrompt - 1);
                float z = A::get(v[k][e]);
                if (n & ~kAlBias) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
                if (c) z = __fsub_rn(z, __fadd_rn(__fmul_rn(freq, static_cast<float>(c)), pres));
                if (n & kAlBias) {
                    if (list_n <= kAlList) {  // in the order of their places
                        for (int last = -1;;) {
                            int next = INT_MAX;
                            for (int i = 0; i < list_n; ++i)
                                if (list_token[i] == w0 + e && list_at[i] > last) next = min(next, list_at[i]);
                            if (next == INT_MAX) break;
                            z = __fadd_rn(z, a.bias[next]);
                            last = next;
                        }
                    } else {
                        for (int b = b0; b < b1; ++b)
                            if (a.bias_ids[b] == g0 + e) z = __fadd_rn(z, a.bias[b]);
                    }
                }
                v[k][e] = A::put(z);
            }
            if (all == (1u << kN) - 1 && vec) *reinterpret_cast<uint4*>(y + g0) = *reinterpret_cast<const uint4*>(v[k]);
            else
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    if (all >> e & 1) y[g0 + e] = v[k][e];
        }
    }
}

template <int DT>
cudaError_t al_launch(const AdjustArgs& a, cudaStream_t s) {
    int slices = static_cast<int>(((long long)a.V + AlVec<DT>::kN - 1 + kAlSlice - 1) / kAlSlice);  // with the skew of a row
    void* args[] = {const_cast<AdjustArgs*>(&a), &slices};
    return launch_kernel(reinterpret_cast<const void*>(adjust_logits_kernel<DT>), dim3(static_cast<unsigned>(a.M) * slices), dim3(kAlThreads), 0, true, s, args);
}

}  // namespace

cudaError_t launch_adjust_logits(const AdjustArgs& a, int dtype, cudaStream_t s) {
    return dtype == 1 ? al_launch<1>(a, s) : dtype == 2 ? al_launch<2>(a, s) : al_launch<3>(a, s);
}

}  // namespace escha
