// Log probabilities of given tokens, the entropy and the top alternatives of
// rows of logits, in one pass over them.
//
// Per row, in units of ln 2: with c = log2 e, m a running maximum, M = c m, and
// z_i = c x_i - M:  s = sum 2^z_i,  t = sum z_i 2^z_i,
//   lse = ln2 (M + log2 s),  logprob(id) = ln2 (z_id - log2 s),
//   entropy = ln2 (log2 s - t / s).
// z is one fma with M rounded; as everything goes by that M, its rounding
// cancels. That holds while the rounding, half a step of M, is a small part of an
// exponent: where |m| is 2^20 or more (a row, or what a lane has seen of it, is
// masked with some -1e9, say), M is c m itself, as z = (x - m) c.
// Two parts join over the larger maximum, f = 2^(M1 - M):
//   s = f s1 + ...,  t = f (t1 + (M1 - M) s1) + ...
// All in f32; m starts at the lowest finite value, so -inf logits (banned
// tokens) add nothing and a row of them alone ends with s = 0.
//
// The top alternatives go by one 64-bit key per logit, (value, lower index
// first). A bound from below for the top-th value comes from the first chunk of
// each warp, out of the lanes' maxima: with q of the 8 warps having p lanes at
// or above a value, p q >= top values are. What reaches it, a few hundred
// values of a row in no order, is collected in shared memory. At the end the
// same bound over what was collected leaves a few more keys than asked for, and
// each of them counts those above it. Where the buffer is full (a row that
// ascends, a row of one value) a warp keeps the best 32 of the rest in order,
// one a lane: right, but slow where most of a row is alike and nothing above it
// raises the bound (all but 10 tokens masked with one value: 2.0 ms for 2048
// rows of 152064, top 8).
//
// Bound: one read of the logits. Each lane loads a chunk ahead; all in all a
// warp issues 13 instructions for 32 values (pairs of f32 where there is an
// instruction for them), half of what the multiprocessors can: 2048 rows of
// 152064 f32 take 202 us, 6.2 TB/s (187 without the top 8). Values of 16 bits
// cost the same instructions and are unpacked besides, for half the bytes: 1000
// such rows of bf16 take 91 us, 3.3 TB/s (66 without the top 8), by the
// arithmetic. How rows are dealt out to warps, CTAs and clusters is at lp_route.
#include <algorithm>

#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kLpValues = 32;  // of a lane's chunk

struct LpPart {
    float m, s, t;
};
struct LpRecord {  // a part of a row
    float m, s, t, pad;
    unsigned long long key[kLogprobMaxTop];
};
// All rows' units cut into ranges, one a CTA: `per` units, one more for the first `rest`.
struct LpCut {
    long long per;
    int units, rest;  // units: of a row
    __device__ __forceinline__ long long begin(int cta) const { return cta * per + min(cta, rest); }
    __device__ __forceinline__ int cta_of(long long unit) const {
        const long long longer = rest * (per + 1);
        return static_cast<int>(unit < longer ? unit / (per + 1) : rest + (unit - longer) / per);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Below this M is rounded, by 2^-4 at most. At 1e9 that would be up to 2^6, and from 1e10 on 2^z could leave the range of f32.
constexpr float kFar = 0x1p20f;

// M of |m| < kFar: always this rounded product (never contracted into a sum), see above.
__device__ __forceinline__ float lp_scaled(float m) { return __fmul_rn(m, kLog2e); }
// M of a less M of m, each as its size has it: c a less M of m, less what c a is above M of a
__device__ __forceinline__ float lp_shift(float a, float m) {
    const bool m_near = fabsf(m) < kFar;
    const float d = fmaf(m_near ? a : a - m, kLog2e, m_near ? -lp_scaled(m) : 0.f);
    return d - (fabsf(a) < kFar ? fmaf(a, kLog2e, -lp_scaled(a)) : 0.f);
}

__device__ __forceinline__ LpPart lp_join(const LpPart& a, const LpPart& b) {
    LpPart r;
    r.m = fmaxf(a.m, b.m);
    const float da = lp_shift(a.m, r.m), db = lp_shift(b.m, r.m);
    const float fa = ex2(da), fb = ex2(db);
    r.s = a.s * fa + b.s * fb;
    // a factor of 0 leaves nothing of t (its difference may be infinite)
    r.t = (fa == 0.f ? 0.f : fa * (a.t + da * a.s)) + (fb == 0.f ? 0.f : fb * (b.t + db * b.s));
    return r;
}

// Whole-number order of f32 values: -0 equals +0, NaN ranks above +inf.
__device__ __forceinline__ unsigned lp_order(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const unsigned b = __float_as_uint(x == 0.f ? 0.f : x);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ unsigned long long lp_key(float x, int i) {
    return (static_cast<unsigned long long>(lp_order(x)) << 32) | static_cast<unsigned>(~i);
}
__device__ __forceinline__ float lp_from_order(unsigned o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ float lp_value(unsigned long long key) {
    const unsigned o = static_cast<unsigned>(key >> 32);
    if (key == 0) return -INFINITY;
    return o == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : lp_from_order(o);
}

// The warp's best 32 keys, best first by lane; `c` is the same in all lanes.
__device__ __forceinline__ void lp_insert(unsigned long long& mine, unsigned long long c, int lane) {
    const int pos = __popc(__ballot_sync(0xffffffffu, mine > c));
    const unsigned long long up = __shfl_up_sync(0xffffffffu, mine, 1);
    if (lane == pos) mine = c;
    if (lane > pos) mine = up;
}

template <int DT>
struct LpVec;
template <>
struct LpVec<3> {
    static constexpr int N = 4;
    static constexpr unsigned kNone = 0xFF800000u;  // -inf
    __device__ static uint4 two(float a, float b) { return make_uint4(__float_as_uint(a), __float_as_uint(b), kNone, kNone); }
    __device__ static void get(const uint4& r, float* x) {
        x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
    }
    __device__ static float one(const void* p, long long i) { return static_cast<const float*>(p)[i]; }
};
template <>
struct LpVec<1> {
    static constexpr int N = 8;
    static constexpr unsigned kNone = 0xFC00FC00u;
    __device__ static uint4 two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);  // exact: both come from this type
        return make_uint4(*reinterpret_cast<const unsigned*>(&h), kNone, kNone, kNone);
    }
    __device__ static void get(const uint4& r, float* x) {
        const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    __device__ static float one(const void* p, long long i) { return h2f_bits(static_cast<const uint16_t*>(p)[i]); }
};
template <>
struct LpVec<2> {
    static constexpr int N = 8;
    static constexpr unsigned kNone = 0xFF80FF80u;
    __device__ static uint4 two(float a, float b) {
        return make_uint4((__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xFFFF0000u), kNone, kNone, kNone);
    }
    __device__ static void get(const uint4& r, float* x) {
        const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    __device__ static float one(const void* p, long long i) { return bf2f_bits(static_cast<const uint16_t*>(p)[i]); }
};

// A warp's state over the values it has seen.
struct LpWarp {
    LpPart p;
    unsigned long long mine;  // by lane: the best of what the buffer had no place for
    float thr;                // values below this are not among the top ones
};

// The n-th largest of the lanes' values, the same in all lanes: by taking the largest away, or out of a sorted warp.
__device__ __forceinline__ unsigned lp_nth(unsigned v, int n, int lane) {
    if (n <= 3) {
        for (;;) {
            const unsigned most = __reduce_max_sync(0xffffffffu, v);
            if (--n == 0) return most;
            if (lane == __ffs(__ballot_sync(0xffffffffu, v == most)) - 1) v = 0u;
        }
    }
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const unsigned o = __shfl_xor_sync(0xffffffffu, v, j);
            // descending within blocks of k whose bit k is 0
            v = ((lane & j) == 0) == ((lane & k) == 0) ? max(v, o) : min(v, o);
        }
    return __shfl_sync(0xffffffffu, v, n - 1);
}

// A value that `top` of the threads' values v (in lp_order) reach: the q-th largest of the warps' p-th largest,
// p q >= top. All threads of the CTA call it; `slots` may be written again after the next __syncthreads.
__device__ __forceinline__ unsigned lp_bound(unsigned v, int top, unsigned* slots, int lane, int warp) {
    const int p = (top + 3) / 4, q = (top + p - 1) / p;  // top <= 32: p <= 8, q <= 4
    v = lp_nth(v, p, lane);
    if (lane == 0) slots[warp] = v;
    __syncthreads();
    v = lane < kLpWarps ? slots[lane] : 0u;
    int above = 0;
#pragma unroll
    for (int j = 0; j < kLpWarps; ++j) {
        const unsigned o = __shfl_sync(0xffffffffu, v, j);
        above += o > v || (o == v && j < lane);
    }
    return __shfl_sync(0xffffffffu, v, __ffs(__ballot_sync(0xffffffffu, lane < kLpWarps && above == q - 1)) - 1);
}

__device__ __forceinline__ unsigned long long pack2(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// max that keeps a NaN of a
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Adds a chunk, kLpValues values of each lane (places past the end hold -inf), to the lane's sums; gives their
// largest.
template <int DT>
__device__ __forceinline__ float lp_sums(LpPart& p, const uint4 (&r)[kLpValues / LpVec<DT>::N]) {
    using V = LpVec<DT>;
    constexpr int N = V::N, kLpLoads = kLpValues / N;
    float b = -INFINITY;
#pragma unroll
    for (int i = 0; i < kLpLoads; ++i) {
        float x[N];
        V::get(r[i], x);
#pragma unroll
        for (int j = 0; j < N; j += 2) b = fmaxf(b, fmaxf(x[j], x[j + 1]));
    }
    if (b > p.m) {
        const float d = lp_shift(p.m, b), f = ex2(d);
        p.t = f == 0.f ? 0.f : f * (p.t + d * p.s);
        p.s *= f;
        p.m = b;
    }
    const bool empty = b == -INFINITY && p.m == kLowest;  // this lane has seen nothing but -inf (or NaN)
    const bool far = !empty && !(fabsf(p.m) < kFar);
    const float M = empty || far ? 0.f : lp_scaled(p.m);
    const unsigned long long c2 = pack2(kLog2e, kLog2e), m2 = pack2(-M, -M);
    unsigned long long s2 = 0ull, t2 = 0ull;
    auto add = [&](auto&& z2) {
#pragma unroll
        for (int i = 0; i < kLpLoads; ++i) {
            float x[N];
            V::get(r[i], x);
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                float z0, z1;
                unpack2(z2(pack2(x[j], x[j + 1])), z0, z1);
                z0 = max_nan(z0, -160.f), z1 = max_nan(z1, -160.f);  // 2^-160 is 0: -inf times it would not be
                const unsigned long long e = pack2(ex2(z0), ex2(z1));
                s2 = add2(s2, e);
                t2 = fma2(pack2(z0, z1), e, t2);
            }
        }
    };
    if (!__any_sync(0xffffffffu, far)) {
        add([&](unsigned long long x) { return fma2(x, c2, m2); });
    } else {
        const float d = far ? -p.m : 0.f;
        const unsigned long long d2 = pack2(d, d);
        add([&](unsigned long long x) { return fma2(add2(x, d2), c2, m2); });
    }
    float s0, s1, t0, t1;
    unpack2(s2, s0, s1);
    unpack2(t2, t0, t1);
    p.s += s0 + s1;
    p.t += t0 + t1;
    return b;
}

// What was collected of a row's part, in no order.
constexpr int kLpKept = 1024;
struct LpKept {
    unsigned long long key[kLpKept + kLpThreads];  // at the end the warps' lists behind it
    int count;  // of all that came, beyond kLpKept too
};

// Collects a chunk's values (`most`: their largest) that reach w.thr, in `kept` (kPlaces of them) or the warp's list. `index(i, j)` is the
// index of value j of the lane's vector i, or -1 for a place past the end.
template <int DT, int kPlaces, typename F>
__device__ __forceinline__ void lp_collect(LpWarp& w, const uint4 (&r)[kLpValues / LpVec<DT>::N],
                                           float most, uint4* buf, LpKept* kept, int top, int lane, F&& index) {
    using V = LpVec<DT>;
    constexpr int N = V::N, kLpLoads = kLpValues / N;
    // a NaN in the sums: a maximum may have passed over one
    const float thr = w.p.s != w.p.s ? -INFINITY : w.thr;
    if (!__any_sync(0xffffffffu, !(most < thr))) return;
    // by lane, which of its values do; those are few, so one short loop takes them, out of shared memory
    unsigned todo = 0, over = 0;  // over: no place for them
#pragma unroll
    for (int i = 0; i < kLpLoads; ++i) {
        float x[N];
        V::get(r[i], x);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (!(x[j] < thr) && index(i, j) >= 0) todo |= 1u << (i * N + j);
        buf[i * 32 + lane] = r[i];
    }
    if (kPlaces == 0) {
        over = todo;
    } else {
#pragma unroll 1
        while (todo) {
            const int k = __ffs(todo) - 1;
            todo &= todo - 1;
            const int at = atomicAdd(&kept->count, 1);
            if (at < kPlaces)
                kept->key[at] = lp_key(V::one(buf + (k / N) * 32 + lane, k % N), index(k / N, k % N));
            else
                over |= 1u << k;
        }
        __syncwarp();
    }
    if (!__any_sync(0xffffffffu, over != 0)) return;
    unsigned long long last = __shfl_sync(0xffffffffu, w.mine, top - 1);
#pragma unroll 1
    for (int k = 0; k < kLpValues; ++k) {
        const bool mine = (over >> k) & 1u;
        if (!__any_sync(0xffffffffu, mine)) continue;
        const float x = V::one(buf + (k / N) * 32 + lane, k % N);
        const unsigned long long key = mine ? lp_key(x, index(k / N, k % N)) : 0ull;
        unsigned more = __ballot_sync(0xffffffffu, key > last);
        while (more) {
            const int src = __ffs(more) - 1;
            more &= more - 1;
            const unsigned long long c = __shfl_sync(0xffffffffu, key, src);
            if (c > last) {
                lp_insert(w.mine, c, lane);
                last = __shfl_sync(0xffffffffu, w.mine, top - 1);
            }
        }
    }
    w.thr = fmaxf(w.thr, lp_value(last));
}

// lp_bound over n keys in shared memory, spread over the warps.
__device__ __forceinline__ unsigned lp_keys_bound(const unsigned long long* keys, int n, int top, unsigned* slots, int lane,
                                                  int warp) {
    unsigned most = 0u;
    for (int i = lane * kLpWarps + warp; i < n; i += kLpThreads) most = max(most, static_cast<unsigned>(keys[i] >> 32));
    return lp_bound(most, top, slots, lane, warp);
}

// So many keys are ranked as they are (160 of them, a row's top 20 in a cluster of 8: 10.8 us, 10.2 with the bound).
constexpr int kLpFew = 96;
// The best `top` of n distinct keys (0: none) in shared memory, in order, to `best`; `work` holds n keys. Each key
// counts those above it; many are first reduced to those that reach a bound. All threads of the CTA call it; `best`
// can be read after it.
__device__ __forceinline__ void lp_select(const unsigned long long* keys, int n, int top, unsigned long long* work,
                                          unsigned long long* best, int lane, int warp) {
    __shared__ unsigned slots[kLpWarps];
    __shared__ int count;
    const int t = threadIdx.x;
    if (t < kLogprobMaxTop) best[t] = 0ull;
    const bool many = n > kLpFew;
    if (many) {
        if (t == 0) count = 0;
        const unsigned bound = lp_keys_bound(keys, n, top, slots, lane, warp);
        for (int i = t; i < n; i += kLpThreads)
            if (keys[i] != 0ull && static_cast<unsigned>(keys[i] >> 32) >= bound) work[atomicAdd(&count, 1)] = keys[i];
        keys = work;
    }
    __syncthreads();
    if (many) n = count;
    for (int i = t; i < n; i += kLpThreads) {
        const unsigned long long mine = keys[i];
        int above = mine == 0ull ? top : 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) above += keys[j] > mine;
        if (above < top) best[above] = mine;
    }
    __syncthreads();
}

// Joins the warp's sums: the maximum, then everybody's parts over it.
__device__ __forceinline__ void lp_join_warp(LpPart& p) {
    float m = p.m;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float d = lp_shift(p.m, m), f = ex2(d);
    p.t = f == 0.f ? 0.f : f * (p.t + d * p.s);
    p.s *= f;
    p.m = m;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) {
        p.s += __shfl_xor_sync(0xffffffffu, p.s, k);
        p.t += __shfl_xor_sync(0xffffffffu, p.t, k);
    }
}
// Joins the sums of the CTA's threads; warp 0 holds the result.
__device__ __forceinline__ void lp_join_sums(LpPart& p, int lane, int warp) {
    __shared__ LpPart parts[kLpWarps];
    lp_join_warp(p);
    if (lane == 0) parts[warp] = p;
    __syncthreads();
    if (warp == 0) {
        p = lane < kLpWarps ? parts[lane] : LpPart{kLowest, 0.f, 0.f};
        lp_join_warp(p);
    }
}

// A given token of a row and its logit, loaded while the row is read.
struct LpGiven {
    int id;
    float x;
};
template <int DT>
__device__ __forceinline__ LpGiven lp_given(const LogprobArgs& a, int row, int i) {
    LpGiven g{-1, 0.f};
    if (i >= a.n_ids) return g;
    g.id = a.ids[(long long)row * a.n_ids + i];
    if (g.id >= 0 && g.id < a.V) g.x = LpVec<DT>::one(static_cast<const char*>(a.logits) + (long long)row * a.ld * (DT == 3 ? 4 : 2), g.id);
    return g;
}

template <int DT>
__device__ __forceinline__ void lp_finish(const LogprobArgs& a, int row, const LpPart& p, unsigned long long mine, const LpGiven& given,
                                          int lane) {
    const float ls = log2f(p.s);
    const bool none = p.s == 0.f;  // every logit is -inf
    auto logprob = [&](float v) {
        if (none) return -INFINITY;
        // (c v of an |v| near the type's end would overflow; there M's rounding is nothing beside v)
        return fabsf(p.m) < kFar && fabsf(v) < 1e37f ? kLn2 * (fmaf(v, kLog2e, -lp_scaled(p.m)) - ls) : (v - p.m) - kLn2 * ls;
    };
    if (lane == 0) {
        if (a.lse) a.lse[row] = none ? -INFINITY : fabsf(p.m) < kFar ? kLn2 * (lp_scaled(p.m) + ls) : p.m + kLn2 * ls;
        if (a.entropy) a.entropy[row] = none ? 0.f : kLn2 * (ls - p.t / p.s);
    }
    for (int i = lane; i < a.n_ids; i += 32) {
        const LpGiven g = i < 32 ? given : lp_given<DT>(a, row, i);
        float r = 0.f;
        if (g.id >= 0 && g.id < a.V)
            r = logprob(g.x);
        else if (g.id != -1)
            r = __uint_as_float(0x7FC00000u);
        a.logprobs[(long long)row * a.n_ids + i] = r;
    }
    if (lane < a.top) {
        a.top_ids[(long long)row * a.top + lane] = static_cast<int32_t>(~static_cast<unsigned>(mine));
        a.top_logprobs[(long long)row * a.top + lane] = logprob(lp_value(mine));
    }
}

__device__ __forceinline__ LpWarp lp_start() {
    LpWarp w;
    w.p = LpPart{kLowest, 0.f, 0.f};
    w.mine = 0ull;
    w.thr = -INFINITY;
    return w;
}

constexpr int kLpCtas = 2;  // a multiprocessor, each lane with two chunks of loads in flight

// The rows are taken in units of 32 vectors; all rows' units, in order, are cut
// into ranges, one a CTA: `per` units, one more for the first `rest` CTAs.
// Values before a row's first 16-byte boundary and behind its last vector go
// with the row's first unit.
// With kCluster > 1 a cluster of CTAs shares a row evenly instead, and its first
// CTA joins the parts.
template <int DT, int kCluster>
__device__ __forceinline__ void lp_ranges(const LogprobArgs& a, const LpCut& cut, LpRecord* rec) {
    using V = LpVec<DT>;
    constexpr int N = V::N, kLpLoads = kLpValues / N;
    constexpr int size = DT == 3 ? 4 : 2;
    __shared__ LpKept kept;
    __shared__ unsigned long long best[kLogprobMaxTop];
    __shared__ uint4 buf[kLpWarps][kLpLoads * 32];  // by warp; for keys once a part's values are collected
    __shared__ unsigned slots[kLpWarps];
    static_assert(sizeof(buf) >= sizeof(kept.key), "the keys of a part");
    __shared__ unsigned long long their_keys[kCluster > 1 ? kCluster * 32 : 1];
    __shared__ LpPart their_sums[kCluster];
    if (kCluster > 1) cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x, rank = kCluster > 1 ? cta % kCluster : 0;
    long long at, end;
    int row, u0;
    const int units = cut.units;
    if (kCluster > 1) {
        row = cta / kCluster;
        u0 = static_cast<int>(static_cast<long long>(rank) * units / kCluster);
        at = 0, end = static_cast<long long>(rank + 1) * units / kCluster - u0;
    } else {
        at = cut.begin(cta), end = cut.begin(cta + 1);
        if (at >> 32) {
            row = static_cast<int>(at / units), u0 = static_cast<int>(at % units);
        } else {
            row = static_cast<int>(static_cast<unsigned>(at) / units), u0 = static_cast<int>(static_cast<unsigned>(at) % units);
        }
    }
    for (bool one = kCluster > 1; one || at < end; ++row, u0 = 0, one = false) {
        const int u1 = static_cast<int>(min(static_cast<long long>(units), u0 + (end - at)));
        const char* x = static_cast<const char*>(a.logits) + (long long)row * a.ld * size;
        const int head = min(a.V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / size));
        const int nv = (a.V - head) / N, tail = head + nv * N;
        const char* base = x + (long long)head * size;
        LpWarp w = lp_start();
        // each warp a run of whole units
        const int mine = (u1 - u0 + kLpWarps - 1) / kLpWarps;
        const int last = min(nv, min(u1, u0 + (warp + 1) * mine) * 32);
        auto load = [&](uint4(&r)[kLpLoads], int v) {
            const char* from = base + (long long)(v + lane) * 16;
            if (v + 32 * kLpLoads <= last) {
#pragma unroll
                for (int i = 0; i < kLpLoads; ++i) r[i] = ldg_stream_v4(from + i * 512);
            } else {
#pragma unroll
                for (int i = 0; i < kLpLoads; ++i) {
                    r[i] = make_uint4(V::kNone, V::kNone, V::kNone, V::kNone);
                    if (v + i * 32 + lane < last) r[i] = ldg_stream_v4(from + i * 512);
                }
            }
        };
        int v = (u0 + warp * mine) * 32;
        uint4 r[kLpLoads];
        load(r, v);
        LpGiven given{-1, 0.f};
        if (warp == 0 && rank == 0 && u0 == 0) given = lp_given<DT>(a, row, lane);
        if (threadIdx.x == 0) kept.count = 0;
        __syncthreads();
        if (a.top > 0) {
            // the bound from every warp's first chunk (-inf where it has none)
            float b = -INFINITY;
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) {
                float h[N];
                V::get(r[i], h);
#pragma unroll
                for (int j = 0; j < N; ++j) b = fmaxf(b, h[j]);
            }
            w.thr = lp_from_order(lp_bound(lp_order(b), a.top, slots, lane, warp));
        }
        const int chunks = (mine + kLpLoads - 1) / kLpLoads;  // the same for all warps
        int again = 2;
        for (int c = 0; c < chunks; ++c, v += 32 * kLpLoads) {
            if (a.top > 0 && c == again) {
                // 2, 8, 32, ... chunks seen: the bound from what they left
                again *= 4;
                __syncthreads();
                const unsigned o = lp_keys_bound(kept.key, min(kept.count, kLpKept), a.top, slots, lane, warp);
                if (o != 0u && o != 0xFFFFFFFFu) w.thr = fmaxf(w.thr, lp_from_order(o));
            }
            if (v >= last) continue;
            uint4 ahead[kLpLoads];
            load(ahead, v + 32 * kLpLoads);
            const float most = lp_sums<DT>(w.p, r);
            if (a.top > 0)
                lp_collect<DT, kLpKept>(w, r, most, buf[warp], &kept, a.top, lane, [&](int i, int j) {
                    const int k = v + i * 32 + lane;
                    return k < last ? head + k * N + j : -1;
                });
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) r[i] = ahead[i];
        }
        if ((kCluster > 1 ? rank == 0 : u0 == 0) && warp == 0 && (head > 0 || tail < a.V)) {
            // fewer than N values at each end: as two values of one vector
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) r[i] = make_uint4(V::kNone, V::kNone, V::kNone, V::kNone);
            r[0] = V::two(lane < head ? V::one(x, lane) : -INFINITY, tail + lane < a.V ? V::one(x, tail + lane) : -INFINITY);
            const float most = lp_sums<DT>(w.p, r);
            if (a.top > 0)
                lp_collect<DT, kLpKept>(w, r, most, buf[0], &kept, a.top, lane, [&](int i, int j) {
                    return i > 0 ? -1 : j == 0 && lane < head ? lane : j == 1 && tail + lane < a.V ? tail + lane : -1;
                });
        }
        lp_join_sums(w.p, lane, warp);  // (a barrier: all is collected)
        if (a.top > 0) {
            const int n = min(kept.count, kLpKept);
            const bool lists = kept.count > kLpKept;
            if (lists) {
                kept.key[kLpKept + threadIdx.x] = w.mine;
                __syncthreads();
            }
            lp_select(kept.key, lists ? kLpKept + kLpThreads : n, a.top, reinterpret_cast<unsigned long long*>(buf), best, lane, warp);
        }
        if (kCluster > 1) {
            cluster_wait();  // all its CTAs run
            if (warp == 0) {
                // to the first CTA's shared memory
                if (lane == 0) {
                    const uint32_t to = cluster_map(smem_u32(&their_sums[rank]), 0);
                    st_cluster_f32(to, w.p.m), st_cluster_f32(to + 4, w.p.s), st_cluster_f32(to + 8, w.p.t);
                }
                if (lane < a.top) st_cluster_u64(cluster_map(smem_u32(&their_keys[rank * a.top + lane]), 0), best[lane]);
            }
            cluster_arrive();
            cluster_wait();
            if (rank != 0) return;
            w.p = threadIdx.x < kCluster ? their_sums[threadIdx.x] : LpPart{kLowest, 0.f, 0.f};
            lp_join_sums(w.p, lane, warp);
            if (a.top > 0) lp_select(their_keys, kCluster * a.top, a.top, reinterpret_cast<unsigned long long*>(buf), best, lane, warp);
            if (warp == 0) lp_finish<DT>(a, row, w.p, a.top > 0 ? best[lane] : 0ull, given, lane);
            return;
        }
        if (warp == 0) {
            const unsigned long long key = a.top > 0 ? best[lane] : 0ull;
            if (u0 == 0 && u1 == units) {
                lp_finish<DT>(a, row, w.p, key, given, lane);
            } else {
                // two records a CTA: of a row that began before its range, and of one that goes on behind it
                LpRecord* to = rec + 2ll * cta + (u0 == 0 ? 1 : 0);
                if (lane == 0) to->m = w.p.m, to->s = w.p.s, to->t = w.p.t;
                to->key[lane] = key;
            }
        }
        at += u1 - u0;
    }
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads, kLpCtas)
    token_logprobs_kernel(LogprobArgs a, LpCut cut, LpRecord* rec) {
    lp_ranges<DT, 1>(a, cut, rec);
}
template <int DT, int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kLpThreads, kLpCtas)
    token_logprobs_cluster_kernel(LogprobArgs a, LpCut cut) {
    lp_ranges<DT, kCluster>(a, cut, nullptr);
}

// Short rows: a warp each, with no barrier among the warps.
template <int DT>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) token_logprobs_rows_kernel(LogprobArgs a) {
    using V = LpVec<DT>;
    constexpr int N = V::N, kLpLoads = kLpValues / N;
    constexpr int size = DT == 3 ? 4 : 2;
    __shared__ uint4 buf[kLpWarps][kLpLoads * 32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (long long at = (long long)blockIdx.x * kLpWarps + warp; at < a.M; at += (long long)gridDim.x * kLpWarps) {
        const int row = static_cast<int>(at);
        const char* x = static_cast<const char*>(a.logits) + row * a.ld * size;
        const int head = min(a.V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / size));
        const int nv = (a.V - head) / N, tail = head + nv * N;
        LpWarp w = lp_start();
        uint4 r[kLpLoads];
        const LpGiven given = lp_given<DT>(a, row, lane);
        // the values at the ends, as two of one vector, after the rest
        for (int v = 0; v < nv; v += 32 * kLpLoads) {
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) {
                r[i] = make_uint4(V::kNone, V::kNone, V::kNone, V::kNone);
                if (v + i * 32 + lane < nv)
                    r[i] = ldg_stream_v4(x + (long long)head * size + (long long)(v + i * 32 + lane) * 16);
            }
            const float b = lp_sums<DT>(w.p, r);
            if (a.top > 0) {
                const unsigned kth = lp_nth(lp_order(b), a.top, lane);
                w.thr = fmaxf(w.thr, lp_from_order(kth));
                lp_collect<DT, 0>(w, r, b, buf[warp], nullptr, a.top, lane, [&](int i, int j) {
                    const int k = v + i * 32 + lane;
                    return k < nv ? head + k * N + j : -1;
                });
            }
        }
        if (head > 0 || tail < a.V) {
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) r[i] = make_uint4(V::kNone, V::kNone, V::kNone, V::kNone);
            r[0] = V::two(lane < head ? V::one(x, lane) : -INFINITY, tail + lane < a.V ? V::one(x, tail + lane) : -INFINITY);
            const float most = lp_sums<DT>(w.p, r);
            if (a.top > 0)
                lp_collect<DT, 0>(w, r, most, buf[warp], nullptr, a.top, lane, [&](int i, int j) {
                    return i > 0 ? -1 : j == 0 && lane < head ? lane : j == 1 && tail + lane < a.V ? tail + lane : -1;
                });
        }
        lp_join_warp(w.p);
        lp_finish<DT>(a, row, w.p, w.mine, given, lane);
    }
}

// Joins the parts of the row that begins in CTA c's range and goes on behind it.
template <int DT>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_join_kernel(LogprobArgs a, LpCut cut, const LpRecord* recs) {
    extern __shared__ unsigned long long lp_smem[];  // two lists of 32 keys a part
    __shared__ unsigned long long best[kLogprobMaxTop];
    pdl_wait();
    pdl_trigger();
    const long long end = cut.begin(blockIdx.x + 1), start = (end - 1) / cut.units * cut.units;
    if (start < cut.begin(blockIdx.x) || start + cut.units == end) return;  // it began before, or it ends here
    const int row = static_cast<int>(start / cut.units), n = cut.cta_of(start + cut.units - 1) - blockIdx.x + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the first CTA's part is its second record
    auto rec = [&](int i) { return recs + 2ll * (blockIdx.x + i) + (i == 0 ? 1 : 0); };
    LpGiven given{-1, 0.f};
    if (warp == 0) given = lp_given<DT>(a, row, lane);
    LpWarp w = lp_start();
    for (int i = threadIdx.x; i < n; i += kLpThreads) w.p = lp_join(w.p, LpPart{rec(i)->m, rec(i)->s, rec(i)->t});
    if (a.top > 0)
#pragma unroll 4
        for (int i = threadIdx.x; i < n * 32; i += kLpThreads) lp_smem[i] = rec(i >> 5)->key[i & 31];
    lp_join_sums(w.p, lane, warp);
    if (a.top > 0) lp_select(lp_smem, n * 32, a.top, lp_smem + n * 32, best, lane, warp);
    if (warp == 0) lp_finish<DT>(a, row, w.p, a.top > 0 ? best[lane] : 0ull, given, lane);
}

// How rows are dealt out: to warps, to clusters of 1 to 8 CTAs (no workspace), or cut over all CTAs with a join
// behind; the launch and the workspace's size both go by this.
//  * A warp is slower at a row than a CTA from about 1000 values on (one row of 3000, top 8: 12 us against 6), but many
//    rows keep all warps busy (4096 rows of 3000: 32 us against 83 cut over CTAs).
//  * The largest cluster that all fit the GPU at once (28 of 8 CTAs, 68 of 4; the next ones wait for a second round:
//    30 rows of 152064 f32 in clusters of 8: 12.4 us, 32: 15.0) and gives each CTA a few thousand values (20000
//    values in 8: 8.0, in 4: 7.5; 5000 in 2: 8.1, in 1: 6.2).
//  * Cut over all CTAs, rows need a second kernel, 5 us and more (61 rows of 152064 f32: 20.6 us against 15.1 in
//    clusters of 4; one: 12.1 against 10.4). That pays where clusters leave most CTAs idle for long (one row of 500000:
//    12.7 against 15.0), by the rates measured: 31 GB/s a CTA, 213 of them fill the memory; and where the last
//    round of many long rows would (1000 of 152064 f32, top 8: 107 against 111; of 16 bits 97 against 91).
constexpr int kLpRows = -1, kLpCut = 0;
int lp_route(int M, int V, int size) {
    if (V <= 1024 || (V <= 4096 && M >= 2 * kLpCtas * kSms)) return kLpRows;
    const int c = M <= 28 && V >= 30000 ? 8 : M <= 68 && V >= 10000 ? 4 : M <= kSms && V >= 30000 ? 2 : 1;
    const double bytes = static_cast<double>(V) * size;
    if (M > kLpCtas * kSms ? bytes > 400e3 : bytes * (1. / c - M / 213.) > 155e3) return kLpCut;
    return c;
}

struct LpPlan {
    LpCut cut;
    int ctas, most_parts;
    bool join;
};
// kLpCtas CTAs a multiprocessor, while each has a row or 2048 values at least; at
// most 74 a row, so that the lists of a row's parts fit the join's shared memory.
LpPlan lp_plan(int M, int V, int dtype) {
    LpPlan p;
    const int per = 32 * 16 / (dtype == 3 ? 4 : 2);
    p.cut.units = (V + per - 1) / per;
    const long long want = std::max<long long>(M, (long long)M * V / 2048), total = (long long)M * p.cut.units;
    p.ctas = static_cast<int>(std::min<long long>(std::min<long long>(kLpCtas * kSms, want), 74ll * M));
    p.cut.per = total / p.ctas;
    p.cut.rest = static_cast<int>(total % p.ctas);
    p.join = p.cut.rest != 0 || p.cut.per % p.cut.units != 0;
    // ranges of `per` units and more that meet a row's units (a row behind the first `rest` ranges meets more than an
    // even share of them): 85 at most, as a range has 8 units or a row and more
    p.most_parts = std::min(p.ctas, std::max(p.cut.units - 2, 0) / static_cast<int>(std::min<long long>(p.cut.per, p.cut.units)) + 2);
    return p;
}

template <int DT>
cudaError_t launch_dt(const LogprobArgs& a, void* ws, cudaStream_t s) {
    const int route = lp_route(a.M, a.V, DT == 3 ? 4 : 2);
    if (route == kLpRows) {
        const int ctas = std::min(kLpCtas * kSms, (a.M + kLpWarps - 1) / kLpWarps);
        void* args[] = {const_cast<LogprobArgs*>(&a)};
        return launch_kernel(reinterpret_cast<const void*>(token_logprobs_rows_kernel<DT>), dim3(ctas), dim3(kLpThreads), 0, true,
                             s, args);
    }
    LpPlan p = lp_plan(a.M, a.V, DT);
    if (route > 1) {
        void* args[] = {const_cast<LogprobArgs*>(&a), &p.cut};
        const void* f = route == 8   ? reinterpret_cast<const void*>(token_logprobs_cluster_kernel<DT, 8>)
                        : route == 4 ? reinterpret_cast<const void*>(token_logprobs_cluster_kernel<DT, 4>)
                                     : reinterpret_cast<const void*>(token_logprobs_cluster_kernel<DT, 2>);
        return launch_kernel(f, dim3(a.M * route), dim3(kLpThreads), 0, true, s, args);
    }
    if (route == 1) {  // ranges of a row each
        p.cut.per = p.cut.units, p.cut.rest = 0;
        p.ctas = a.M;
        p.join = false;
    }
    LpRecord* rec = static_cast<LpRecord*>(ws);
    void* args[] = {const_cast<LogprobArgs*>(&a), &p.cut, &rec};
    cudaError_t e = launch_kernel(reinterpret_cast<const void*>(token_logprobs_kernel<DT>), dim3(p.ctas), dim3(kLpThreads), 0,
                                  true, s, args);
    if (e != cudaSuccess || !p.join) return e;
    return launch_kernel(reinterpret_cast<const void*>(token_logprobs_join_kernel<DT>), dim3(p.ctas), dim3(kLpThreads),
                         a.top > 0 ? p.most_parts * 32 * 2 * 8 : 0, true, s, args);
}

}  // namespace

size_t token_logprobs_ws_bytes(int M, int V) {
    if (lp_route(M, V, 4) != kLpCut) return 0;  // nor do 16-bit rows, half as long, go by it then
    return static_cast<size_t>(lp_plan(M, V, 3).ctas) * 2 * sizeof(LpRecord);
}

cudaError_t launch_token_logprobs(const LogprobArgs& a, int dtype, void* ws, cudaStream_t s) {
    if (dtype == 1) return launch_dt<1>(a, ws, s);
    if (dtype == 2) return launch_dt<2>(a, ws, s);
    return launch_dt<3>(a, ws, s);
}

}  // namespace escha
