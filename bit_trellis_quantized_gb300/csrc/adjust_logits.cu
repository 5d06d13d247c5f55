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
// whole-number sums, which come out alike in any order, beside a list of those
// that have one. One pass over the slice bans and copies, then each listed token
// gets what is its own, a thread a token. The biases of a slice are listed, and
// looked through by the tokens that have one; where they are more than 32, after
// the list is put in the order of their places; more than 512 are taken from the
// row's list 512 places at a time, in order. So a list of any length takes a time
// in proportion to it (152064 biases of as many tokens: 0.77 ms).
//
// Bound: the write of the banned and the changed logits, and the read of those
// next to them. Slices of 32 KB let three CTAs share a multiprocessor, so that
// one's counting runs beside another's pass. Measured in f32: 256 rows of 152064,
// all under masks of one token in eight, up to 8000 ids, 65 us (the sectors that
// it cannot do without, 259 MB with those read for their allowed tokens: 38); 61 of
// 248320 copied, 24 us (18); one row in place 4 us. Slices of 4096 to 256 threads: 70 and 25 us.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

#include <limits.h>

namespace escha {

namespace {

constexpr int kAlThreads = 512;
constexpr int kAlSlice = 8192;  // tokens of a CTA at most
constexpr int kAlList = kAlThreads;  // biases that are taken at once, one a thread
constexpr int kAlFew = 32;            // up to so many of a slice, the list is searched as it is
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
__global__ void __launch_bounds__(kAlThreads, 3) adjust_logits_kernel(AdjustArgs a, int slices) {
    using A = AlVec<DT>;
    using E = typename A::type;
    constexpr int kN = A::kN, kEach = kAlSlice / (kAlThreads * kN);  // groups of a thread
    __shared__ __align__(16) uint32_t words[kAlSlice];
    __shared__ uint32_t masks[kAlSlice / 32 + 2];
    __shared__ uint16_t touched[kAlSlice];  // tokens with a word, in any order
    __shared__ int touched_n, list_n[2];
    __shared__ int list_at[kAlList], list_token[kAlList];  // biases of the slice: their places (values, once they are in order) and tokens
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
    constexpr int kFirst = 4;  // of the row's ids: loads that go ahead, with the mask's
    int first[kFirst];
    if (counts) {
#pragma unroll
        for (int k = 0; k < kFirst; ++k) first[k] = i0 + k * kAlThreads + t < i1 ? a.ids[i0 + k * kAlThreads + t] : -1;
#pragma unroll
        for (int i = 0; i < kAlSlice / (kAlThreads * 4); ++i) *reinterpret_cast<uint4*>(words + (i * kAlThreads + t) * 4) = make_uint4(0, 0, 0, 0);
        if (t == 0) list_n[0] = list_n[1] = touched_n = 0;
    }
    __syncthreads();
    // ---- what is banned, and the copy. Where all groups are whole and begin at a multiple of 32 tokens, a word of the mask
    // serves 32 / kN threads as it is, and the values are on their way while the ids are counted.
    constexpr uint32_t kAll = (1u << kN) - 1;
    const bool plain = (masked || copy) && skew == 0 && vec && base + kAlSlice <= a.V;
    __align__(16) E v[kEach][kN];
    uint32_t open[kEach];
    if (plain) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            open[k] = masked ? masks[(k * kAlThreads + t) * kN / 32] >> (t * kN & 31) & kAll : kAll;
            if (open[k] != 0 && (copy || open[k] != kAll)) *reinterpret_cast<uint4*>(v[k]) = *reinterpret_cast<const uint4*>(x + base + (k * kAlThreads + t) * kN);
        }
    }
    if (counts) {
        const long long late = static_cast<long long>(i0) + (a.prompt ? max(a.prompt[row], 0) : 0);
        auto count = [&](int i, int id) {
            const uint32_t w = static_cast<uint32_t>(id) - static_cast<uint32_t>(base);
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.V) || w >= kAlSlice) return;
            if ((i >= late ? atomicAdd(&words[w], 1u) : atomicOr(&words[w], kAlPrompt)) == 0) touched[atomicAdd(&touched_n, 1)] = static_cast<uint16_t>(w);
        };
#pragma unroll
        for (int k = 0; k < kFirst; ++k) count(i0 + k * kAlThreads + t, first[k]);
#pragma unroll 4
        for (int i = i0 + kFirst * kAlThreads + t; i < i1; i += kAlThreads) count(i, a.ids[i]);
        for (int i = b0 + t; i < b1; i += kAlThreads) {
            const int id = a.bias_ids[i];
            const uint32_t w = static_cast<uint32_t>(id) - static_cast<uint32_t>(base);
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.V) || w >= kAlSlice) continue;
            if (atomicOr(&words[w], kAlBias) == 0) touched[atomicAdd(&touched_n, 1)] = static_cast<uint16_t>(w);
            const int at = atomicAdd(&list_n[0], 1);
            if (at < kAlList) list_at[at] = i, list_token[at] = static_cast<int>(w);
        }
    }
    // the n listed biases in the order of their places, a thread each
    auto order = [&](int n) {
        int rank = 0, token = 0;
        float value = 0.f;
        if (t < n) {
            const int at = list_at[t];
            token = list_token[t], value = a.bias[at];
            for (int k = 0; k < n; ++k) rank += list_at[k] < at;
        }
        __syncthreads();
        if (t < n) list_at[rank] = __float_as_int(value), list_token[rank] = token;
        __syncthreads();
    };
    // the allowed ones of a group's tokens, a bit each, and those that there are
    auto bits = [&](int g0) {
        const int lo = g0 < 0 ? -g0 : 0, hi = min(max(a.V - g0, 0), kN);
        return hi > lo ? ((1u << hi) - 1) & ~((1u << lo) - 1) : 0u;
    };
    auto allowed = [&](int g0) {
        if (!masked) return ~0u;
        const int lo = g0 < 0 ? -g0 : 0, at = g0 + lo - max(base, 0) / 32 * 32;
        return __funnelshift_r(masks[at / 32], masks[at / 32 + 1], at & 31) << lo;
    };
    if (plain) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
#pragma unroll
            for (int e = 0; e < kN; ++e)
                if (!(open[k] >> e & 1)) v[k][e] = A::put(-INFINITY);
            if (copy || open[k] != kAll) *reinterpret_cast<uint4*>(y + base + (k * kAlThreads + t) * kN) = *reinterpret_cast<const uint4*>(v[k]);
        }
    } else if (masked || copy) {
        uint32_t all[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int g0 = base + (k * kAlThreads + t) * kN;
            all[k] = bits(g0), open[k] = all[k] ? allowed(g0) & all[k] : 0u;
            if (!copy && open[k] == all[k]) all[k] = 0;  // nothing to write
            if (all[k] == (1u << kN) - 1 && open[k]) *reinterpret_cast<uint4*>(v[k]) = *reinterpret_cast<const uint4*>(x + g0);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int g0 = base + (k * kAlThreads + t) * kN;
            const bool whole = all[k] == (1u << kN) - 1;
            if (whole) {
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    if (!(open[k] >> e & 1)) v[k][e] = A::put(-INFINITY);
            }
            if (whole && vec) {
                *reinterpret_cast<uint4*>(y + g0) = *reinterpret_cast<const uint4*>(v[k]);
            } else if (whole) {
#pragma unroll
                for (int e = 0; e < kN; ++e) y[g0 + e] = v[k][e];
            } else if (all[k]) {
#pragma unroll 1
                for (int e = 0; e < kN; ++e)
                    if (all[k] >> e & 1) y[g0 + e] = open[k] >> e & 1 ? x[g0 + e] : A::put(-INFINITY);
            }
        }
    }
    if (!counts) return;
    __syncthreads();
    // ---- the touched ones. More biases than a list holds are added to the tokens' values, which wait in their words.
    const float rep = a.repetition ? a.repetition[row] : 1.f, freq = a.frequency ? a.frequency[row] : 0.f;
    const float pres = a.presence ? a.presence[row] : 0.f;
    const int biases = list_n[0];
    const bool many = biases > kAlList;
    constexpr uint16_t kWaits = 0x8000;
    static_assert(kAlSlice <= kWaits, "a bit beside the token");
    // As it is, the list is gone through once for each bias of a token: 512 of one token would be 512 x 512 steps of a thread, and are
    // 17 us in order. In order takes barriers more: 256 x 152064, 0 to 50 biases a row, 66.3 us as it is, 68.6 in order.
    if (biases > kAlFew && !many) order(biases);
#pragma unroll 1
    for (int i = t; i < touched_n; i += kAlThreads) {
        const int w = touched[i];
        if (masked) {
            const int at = base + w - max(base, 0) / 32 * 32;
            if (!(masks[at / 32] >> (at & 31) & 1)) continue;
        }
        const uint32_t n = words[w], c = n & (kAlPrompt - 1);
        float z = A::get(x[base + w]);
        if (n & ~kAlBias) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
        if (c) z = __fsub_rn(z, __fadd_rn(__fmul_rn(freq, static_cast<float>(c)), pres));
        if (n & kAlBias) {
            if (many) {
                words[w] = __float_as_uint(z), touched[i] = static_cast<uint16_t>(w | kWaits);
                continue;
            }
            if (biases > kAlFew) {
                for (int k = 0; k < biases; ++k)
                    if (list_token[k] == w) z = __fadd_rn(z, __int_as_float(list_at[k]));
            } else {  // the next place, again and again
                for (int last = -1;;) {
                    int next = INT_MAX;
                    for (int k = 0; k < biases; ++k)
                        if (list_token[k] == w && list_at[k] > last) next = min(next, list_at[k]);
                    if (next == INT_MAX) break;
                    z = __fadd_rn(z, a.bias[next]);
                    last = next;
                }
            }
        }
        y[base + w] = A::put(z);
    }
    if (!many) return;
    // a thread a place, then a thread every kAlThreads-th token
    for (int b = b0, p = 1; b < b1; b += kAlThreads, p ^= 1) {
        const int i = b + t, id = i < b1 ? a.bias_ids[i] : -1;
        const uint32_t w = static_cast<uint32_t>(id) - static_cast<uint32_t>(base);
        if (static_cast<unsigned>(id) < static_cast<unsigned>(a.V) && w < kAlSlice) {
            const int at = atomicAdd(&list_n[p], 1);
            list_at[at] = i, list_token[at] = static_cast<int>(w);
        }
        __syncthreads();
        const int n = list_n[p];
        if (t == 0) list_n[p ^ 1] = 0;  // (of the next places, which are counted behind the next barriers)
        order(n);
        for (int k = 0; k < n; ++k) {
            const int of = list_token[k];
            if (of % kAlThreads == t) words[of] = __float_as_uint(__fadd_rn(__uint_as_float(words[of]), __int_as_float(list_at[k])));
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int i = t; i < touched_n; i += kAlThreads)
        if (touched[i] & kWaits) y[base + (touched[i] & ~kWaits)] = A::put(__uint_as_float(words[touched[i] & ~kWaits]));
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
