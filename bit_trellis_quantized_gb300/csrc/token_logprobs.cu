// Log probabilities of given tokens, the entropy and the top alternatives of
// rows of logits, in one pass over them.
//
// Per row, with m a running maximum, s = sum e^(x - m), t = sum (x - m) e^(x - m):
//   lse = m + ln s,  logprob(id) = (x_id - m) - ln s,  entropy = ln s - t / s.
// Two parts (m1, s1, t1), (m2, s2, t2) join over M = max(m1, m2) with f = e^(m1 - M):
//   s = f s1 + ..., t = f (t1 + (m1 - M) s1) + ...
// All in f32; m starts at the lowest finite value, so -inf logits (banned
// tokens) add nothing and a row of them alone ends with s = 0.
//
// The top alternatives go by one 64-bit key per logit, (value, lower index
// first): each warp keeps the best 32 of what it has seen, one per lane in
// order, and looks closer only at a batch whose largest value reaches the
// top-th best so far.
//
// Bound: one read of the logits. A row is split over CTAs until the grid fills
// the GPU; a second kernel then joins the parts of a row.
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

struct LpPart {
    float m, s, t;
};
struct LpRecord {  // one split of a row
    float m, s, t, pad;
    unsigned long long key[kLogprobMaxTop];
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ LpPart lp_join(const LpPart& a, const LpPart& b) {
    LpPart r;
    r.m = fmaxf(a.m, b.m);
    const float da = a.m - r.m, db = b.m - r.m;
    const float fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);
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
__device__ __forceinline__ float lp_value(unsigned long long key) {
    const unsigned o = static_cast<unsigned>(key >> 32);
    if (key == 0) return -INFINITY;
    return o == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
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
    __device__ static void get(const uint4& r, float* x) {
        x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
    }
    __device__ static float one(const void* p, long long i) { return static_cast<const float*>(p)[i]; }
};
template <>
struct LpVec<1> {
    static constexpr int N = 8;
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
    unsigned long long mine;
    float thr;  // a batch below this holds no top value
};

// N values of consecutive indexes i0.. per lane (those below `ok` count).
template <int N>
__device__ __forceinline__ void lp_batch(LpWarp& w, const float (&x)[N], int i0, int ok, int top, int lane) {
    float b = kLowest;
#pragma unroll
    for (int j = 0; j < N; ++j) b = j < ok ? fmaxf(b, x[j]) : b;
    if (b > w.p.m) {
        const float d = w.p.m - b, f = ex2(d * kLog2e);
        w.p.t = f == 0.f ? 0.f : f * (w.p.t + d * w.p.s);
        w.p.s *= f;
        w.p.m = b;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (j < ok) {
            const float y = x[j] - w.p.m, e = ex2(y * kLog2e);
            w.p.s += e;
            w.p.t += fmaxf(y, kLowest) * e;
        }
    }
    if (top == 0) return;
    // a NaN in s: the maximum may have passed over a NaN
    if (__any_sync(0xffffffffu, ok > 0 && (b >= w.thr || w.p.s != w.p.s))) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned long long key = j < ok ? lp_key(x[j], i0 + j) : 0ull;
            unsigned long long last = __shfl_sync(0xffffffffu, w.mine, top - 1);
            unsigned todo = __ballot_sync(0xffffffffu, key > last);
            while (todo) {
                const int src = __ffs(todo) - 1;
                todo &= todo - 1;
                const unsigned long long c = __shfl_sync(0xffffffffu, key, src);
                if (c > last) {
                    lp_insert(w.mine, c, lane);
                    last = __shfl_sync(0xffffffffu, w.mine, top - 1);
                }
            }
        }
        w.thr = lp_value(__shfl_sync(0xffffffffu, w.mine, top - 1));
    }
}

// Joins the warps' states of a CTA; warp 0 holds the result.
__device__ __forceinline__ void lp_join_cta(LpWarp& w, int top, int lane, int warp) {
    __shared__ LpPart parts[kLpWarps];
    __shared__ unsigned long long keys[kLpWarps][kLogprobMaxTop];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        LpPart o;
        o.m = __shfl_xor_sync(0xffffffffu, w.p.m, m);
        o.s = __shfl_xor_sync(0xffffffffu, w.p.s, m);
        o.t = __shfl_xor_sync(0xffffffffu, w.p.t, m);
        // the same order of the operands in both lanes
        w.p = (lane & m) ? lp_join(o, w.p) : lp_join(w.p, o);
    }
    if (lane == 0) parts[warp] = w.p;
    keys[warp][lane] = w.mine;
    __syncthreads();
    if (warp != 0) return;
    for (int i = 1; i < kLpWarps; ++i) w.p = lp_join(w.p, parts[i]);
    if (top > 0) {
        for (int i = 1; i < kLpWarps; ++i) {
            const unsigned long long theirs = keys[i][lane];
            for (int j = 0; j < top; ++j) {
                const unsigned long long c = __shfl_sync(0xffffffffu, theirs, j);
                if (c <= __shfl_sync(0xffffffffu, w.mine, top - 1)) break;
                lp_insert(w.mine, c, lane);
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void lp_finish(const LogprobArgs& a, int row, const LpWarp& w, int lane) {
    const float ls = logf(w.p.s);
    const bool none = w.p.s == 0.f;  // every logit is -inf
    if (lane == 0) {
        if (a.lse) a.lse[row] = none ? -INFINITY : w.p.m + ls;
        if (a.entropy) a.entropy[row] = none ? 0.f : ls - w.p.t / w.p.s;
    }
    const char* x = static_cast<const char*>(a.logits) + (long long)row * a.ld * (DT == 3 ? 4 : 2);
    for (int i = lane; i < a.n_ids; i += 32) {
        const int id = a.ids[(long long)row * a.n_ids + i];
        float r = 0.f;
        if (id >= 0 && id < a.V)
            r = none ? -INFINITY : (LpVec<DT>::one(x, id) - w.p.m) - ls;
        else if (id != -1)
            r = __uint_as_float(0x7FC00000u);
        a.logprobs[(long long)row * a.n_ids + i] = r;
    }
    if (lane < a.top) {
        a.top_ids[(long long)row * a.top + lane] = static_cast<int32_t>(~static_cast<unsigned>(w.mine));
        a.top_logprobs[(long long)row * a.top + lane] = none ? -INFINITY : (lp_value(w.mine) - w.p.m) - ls;
    }
}

__device__ __forceinline__ LpWarp lp_start() {
    LpWarp w;
    w.p = LpPart{kLowest, 0.f, 0.f};
    w.mine = 0ull;
    w.thr = -INFINITY;
    return w;
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(LogprobArgs a, int splits, LpRecord* rec) {
    using V = LpVec<DT>;
    constexpr int N = V::N;
    constexpr int size = DT == 3 ? 4 : 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.y, split = blockIdx.x;
    const char* x = static_cast<const char*>(a.logits) + (long long)row * a.ld * size;
    // 16-byte vectors of the row, and the values before and behind them
    const int head = min(a.V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / size));
    const int nv = (a.V - head) / N, tail = head + nv * N;
    LpWarp w = lp_start();
    if (split == 0 && warp == 0) {
        // fewer than N values at each end
        float e[2] = {0.f, 0.f};
        const int i0 = lane, i1 = tail + lane;
        if (i0 < head) e[0] = V::one(x, i0);
        if (i1 < a.V) e[1] = V::one(x, i1);
        const float h0[1] = {e[0]}, h1[1] = {e[1]};
        lp_batch(w, h0, i0, i0 < head, a.top, lane);
        lp_batch(w, h1, i1, i1 < a.V, a.top, lane);
    }
    const int per = (nv + splits - 1) / splits;
    const int v0 = min(nv, split * per), v1 = min(nv, v0 + per);
    const char* base = x + (long long)head * size;
    for (int v = v0 + warp * 32; v < v1; v += kLpThreads) {
        const bool ok = v + lane < v1;
        uint4 r = make_uint4(0, 0, 0, 0);
        if (ok) r = ldg_stream_v4(base + (long long)(v + lane) * 16);
        float f[N];
        V::get(r, f);
        lp_batch(w, f, head + (v + lane) * N, ok ? N : 0, a.top, lane);
    }
    lp_join_cta(w, a.top, lane, warp);
    if (warp != 0) return;
    if (splits == 1) {
        lp_finish<DT>(a, row, w, lane);
    } else {
        LpRecord* r = rec + (long long)row * splits + split;
        if (lane == 0) r->m = w.p.m, r->s = w.p.s, r->t = w.p.t;
        r->key[lane] = w.mine;
    }
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_join_kernel(LogprobArgs a, int splits, const LpRecord* rec) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x;
    const LpRecord* r = rec + (long long)row * splits;
    LpWarp w = lp_start();
    // thread i joins the sums of splits i, i + 256, ...
    for (int i = threadIdx.x; i < splits; i += kLpThreads) w.p = lp_join(w.p, LpPart{r[i].m, r[i].s, r[i].t});
    if (a.top > 0) {
        for (int i = warp; i < splits; i += kLpWarps) {
            const unsigned long long theirs = r[i].key[lane];
            for (int j = 0; j < a.top; ++j) {
                const unsigned long long c = __shfl_sync(0xffffffffu, theirs, j);
                if (c <= __shfl_sync(0xffffffffu, w.mine, a.top - 1)) break;
                lp_insert(w.mine, c, lane);
            }
        }
    }
    lp_join_cta(w, a.top, lane, warp);
    if (warp == 0) lp_finish<DT>(a, row, w, lane);
}

// CTAs a row is split over: enough for four a multiprocessor, each with 1024 16-byte vectors at least.
int lp_splits(int M, int V) {
    const long long want = (4ll * kSms + M - 1) / M;
    const long long most = (V + 4095) / 4096;
    return static_cast<int>(want < most ? want : most);
}

template <int DT>
cudaError_t launch_dt(const LogprobArgs& a, LpRecord* rec, cudaStream_t s) {
    int splits = lp_splits(a.M, a.V);
    LogprobArgs b = a;
    void* args[] = {&b, &splits, &rec};
    // rows past 65535 (the grid's y limit) go in further launches
    for (int m0 = 0; m0 < a.M; m0 += 65535) {
        const int m = a.M - m0 < 65535 ? a.M - m0 : 65535;
        b.M = m;
        b.logits = static_cast<const char*>(a.logits) + (long long)m0 * a.ld * (DT == 3 ? 4 : 2);
        b.ids = a.ids ? a.ids + (long long)m0 * a.n_ids : nullptr;
        b.logprobs = a.logprobs ? a.logprobs + (long long)m0 * a.n_ids : nullptr;
        b.entropy = a.entropy ? a.entropy + m0 : nullptr;
        b.lse = a.lse ? a.lse + m0 : nullptr;
        b.top_ids = a.top_ids ? a.top_ids + (long long)m0 * a.top : nullptr;
        b.top_logprobs = a.top_logprobs ? a.top_logprobs + (long long)m0 * a.top : nullptr;
        cudaError_t e = launch_kernel(reinterpret_cast<const void*>(token_logprobs_kernel<DT>), dim3(splits, m),
                                      dim3(kLpThreads), 0, true, s, args);
        if (e != cudaSuccess) return e;
        if (splits > 1) {
            e = launch_kernel(reinterpret_cast<const void*>(token_logprobs_join_kernel<DT>), dim3(m), dim3(kLpThreads),
                              0, true, s, args);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

size_t token_logprobs_ws_bytes(int M, int V) {
    const int splits = lp_splits(M, V);
    return splits > 1 ? static_cast<size_t>(M) * splits * sizeof(LpRecord) : 0;
}

cudaError_t launch_token_logprobs(const LogprobArgs& a, int dtype, void* ws, cudaStream_t s) {
    LpRecord* rec = static_cast<LpRecord*>(ws);
    if (dtype == 1) return launch_dt<1>(a, rec, s);
    if (dtype == 2) return launch_dt<2>(a, rec, s);
    return launch_dt<3>(a, rec, s);
}

}  // namespace escha
