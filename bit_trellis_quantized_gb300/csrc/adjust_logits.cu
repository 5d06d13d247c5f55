// Penalties for repeated tokens, biases and grammar masks on logits.
//
// Per row and token i, in this order, in f32, each operation rounded, the
// result rounded once to its type:
//   among the row's ids:             x = x > 0 ? x / repetition : x repetition
//   c > 0 times behind the prompt:   x = x - (frequency c + presence)
//   each bias of i, in list order:   x = x + bias
//   not allowed by the row's mask:   x = -infinity
//
// A CTA takes a slice of a row and holds a word for each of its tokens in
// shared memory: how often the row's ids name it, and whether they do at all,
// as whole-number sums, which come out alike in any order. Then one pass over
// the slice reads what is to be changed (everything, where the result goes to
// another buffer) and writes it.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr int kAlThreads = 512;
constexpr int kAlSlice = 32768;  // tokens of a CTA at most: 128 KB of words
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
__global__ void __launch_bounds__(kAlThreads) adjust_logits_kernel(AdjustArgs a, int slice, int slices) {
    using A = AlVec<DT>;
    using E = typename A::type;
    constexpr int kN = A::kN;
    extern __shared__ __align__(16) uint32_t words[];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x, row = blockIdx.x / slices;
    const E* x = static_cast<const E*>(a.logits) + row * a.ld;
    E* y = static_cast<E*>(a.out) + row * a.out_ld;
    // Groups of kN values begin where `x` is aligned: group g is [g kN - skew, g kN - skew + kN).
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(E) % kN);
    const bool vec = reinterpret_cast<uintptr_t>(y) / sizeof(E) % kN == static_cast<uintptr_t>(skew);
    const long long base = (long long)(blockIdx.x % slices) * slice - skew;  // token of words[0]
    for (int i = t * 4; i < slice; i += kAlThreads * 4) *reinterpret_cast<uint4*>(words + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (a.ids) {
        const int i0 = min(max(a.at[row], 0), a.n_ids), i1 = min(max(a.at[row + 1], 0), a.n_ids);
        const long long late = (long long)i0 + (a.prompt ? max(a.prompt[row], 0) : 0);
        for (int i = i0 + t; i < i1; i += kAlThreads) {
            const long long id = a.ids[i], w = id - base;
            if (id < 0 || id >= a.V || w < 0 || w >= slice) continue;
            if (i >= late) atomicAdd(&words[w], 1u);
            else atomicOr(&words[w], kAlPrompt);
        }
    }
    int b0 = 0, b1 = 0;
    if (a.bias_ids) {
        b0 = min(max(a.bias_at[row], 0), a.n_bias), b1 = min(max(a.bias_at[row + 1], 0), a.n_bias);
        for (int i = b0 + t; i < b1; i += kAlThreads) {
            const long long id = a.bias_ids[i], w = id - base;
            if (id >= 0 && id < a.V && w >= 0 && w < slice) atomicOr(&words[w], kAlBias);
        }
    }
    __syncthreads();
    const float rep = a.repetition ? a.repetition[row] : 1.f, freq = a.frequency ? a.frequency[row] : 0.f;
    const float pres = a.presence ? a.presence[row] : 0.f;
    const int mrow = !a.allowed ? -1 : a.allowed_rows ? a.allowed_rows[row] : row;
    const int mwords = (a.V + 31) / 32;
    const uint32_t* mask = static_cast<unsigned>(mrow) < static_cast<unsigned>(a.n_masks)
                               ? reinterpret_cast<const uint32_t*>(a.allowed) + (long long)mrow * mwords : nullptr;
    const bool copy = a.logits != a.out;
    for (int w0 = t * kN; w0 < slice; w0 += kAlThreads * kN) {
        const long long i0 = base + w0;
        if (i0 >= a.V) break;
        // the group's allowed tokens and the touched ones, a bit each
        const int lo = i0 < 0 ? static_cast<int>(-i0) : 0, hi = static_cast<int>(min((long long)kN, a.V - i0));
        uint32_t open = (1u << kN) - 1;
        if (mask) {
            const int at = static_cast<int>(i0) + lo, wd = at / 32;
            const uint32_t m0 = mask[wd], m1 = wd + 1 < mwords ? mask[wd + 1] : 0;
            open = __funnelshift_r(m0, m1, at & 31) << lo;
        }
        uint32_t n[kN], touched = 0;
#pragma unroll
        for (int e = 0; e < kN; e += 4) *reinterpret_cast<uint4*>(n + e) = *reinterpret_cast<const uint4*>(words + w0 + e);
#pragma unroll
        for (int e = 0; e < kN; ++e) touched |= (n[e] != 0) << e;
        const uint32_t all = ((1u << hi) - 1) & ~((1u << lo) - 1);
        if (!copy && ((touched | ~open) & all) == 0) continue;
        const bool whole = all == (1u << kN) - 1;
        __align__(16) E v[kN];
        if (copy || (open & all)) {
            if (whole) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(x + i0);
            else
                for (int e = lo; e < hi; ++e) v[e] = x[i0 + e];
        }
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            if (!(all >> e & 1)) continue;
            if (!(open >> e & 1)) {
                v[e] = A::put(-INFINITY);
            } else if (n[e]) {
                float z = A::get(v[e]);
                const uint32_t c = n[e] & (kAlPrompt - 1);
                if (n[e] & ~kAlBias) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
                if (c) z = __fsub_rn(z, __fadd_rn(__fmul_rn(freq, static_cast<float>(c)), pres));
                if (n[e] & kAlBias)
                    for (int b = b0; b < b1; ++b)
                        if (a.bias_ids[b] == i0 + e) z = __fadd_rn(z, a.bias[b]);
                v[e] = A::put(z);
            }
        }
        if (whole && vec) *reinterpret_cast<uint4*>(y + i0) = *reinterpret_cast<const uint4*>(v);
        else
#pragma unroll
            for (int e = 0; e < kN; ++e)
                if (all >> e & 1) y[i0 + e] = v[e];
    }
}

template <int DT>
cudaError_t al_launch(const AdjustArgs& a, cudaStream_t s) {
    constexpr int kUnit = 4096;
    const long long whole = (long long)a.V + AlVec<DT>::kN;  // with the skew of a row
    int slice = kAlSlice;
    while (slice > kUnit && a.M * ((whole + slice - 1) / slice) < kSms) slice /= 2;
    int slices = static_cast<int>((whole + slice - 1) / slice);
    const void* f = reinterpret_cast<const void*>(adjust_logits_kernel<DT>);
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlSlice * 4);
    if (e != cudaSuccess) return e;
    void* args[] = {const_cast<AdjustArgs*>(&a), &slice, &slices};
    return launch_kernel(f, dim3(static_cast<unsigned>(a.M) * slices), dim3(kAlThreads), slice * 4, true, s, args);
}

}  // namespace

cudaError_t launch_adjust_logits(const AdjustArgs& a, int dtype, cudaStream_t s) {
    return dtype == 1 ? al_launch<1>(a, s) : dtype == 2 ? al_launch<2>(a, s) : al_launch<3>(a, s);
}

}  // namespace escha
