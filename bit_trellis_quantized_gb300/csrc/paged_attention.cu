// Attention of one new token a sequence over a paged key-value cache.
//
// Per sequence b and query head h, over the keys j < lens[b] of its key head:
//   x_j = scale q . k_j,  out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
//   lse = m + ln sum_j e^(x_j - m),  m = max_j x_j.
// Parts over different keys join by their (m, sum, weighted values). Scores,
// maxima, sums and weighted values are held in f32. A weight e^(x - m) enters
// the tensor cores as two 16-bit parts (value, remainder), so that the one
// rounding that shows is that of `out` to its type. fp16 parts are of the
// weight times 2^15: its steps end at 2^-24, and keys at 2^-25 of the largest
// weight, each lost or doubled without it, may be many.
//
// Bound: the one read of K and V (a key is used by Hq / Hkv heads: at most 4 x
// 16 flops a byte). So the layout serves the loads:
//   * A unit is one (sequence, key head, up to 8 NT query heads); its keys are
//     taken in rounds of 64, 16 a warp. A cluster of 1 to 8 CTAs takes a unit,
//     each a run of its rounds, and joins the parts through shared memory. Where
//     the units are few and long, all units' rounds are cut into equal ranges,
//     one a CTA, instead, and the parts joined by a second kernel (pa_route).
//   * Each warp fills its own ring of 16-key stages (cp.async, 16 bytes a lane,
//     rows of the pages wherever they are) and waits for nobody else. Rows that
//     are not there are filled with zeros and masked.
//   * Keys are the M of both products (scores K Q^T, values V^T P^T: m16n8k16),
//     so that 8 query heads fill the instruction's N exactly.
// Measured: 192 sequences of 500 to 16384 keys, 2 key heads of 256: 283 us, 6.6
// TB/s; one of 131071: 49 us, 5.5 TB/s; one of 700: 8.1 us.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
template <int DT>
constexpr float kPaUp = DT == 1 ? 0x1p15f : 1.f;  // of a weight's parts

// A warp's ring holds kHalves halves of stages (16 keys, or their 16 values).
template <int D, int NT>
struct PaCfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRound = 16 * kWarps;  // keys of a round
    static constexpr int kHalves = D == 256 ? 3 : D == 128 ? 4 : 6;
    static constexpr int kCtas = D == 256 ? 2 : D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 4 : 3);  // a multiprocessor
    static constexpr int kRow = D * 2;          // bytes of a row
    static constexpr int kTile = 16 * kRow;     // of a half
    static constexpr int kRing = kWarps * kHalves * kTile;
    static_assert(8 * NT * (D + 4) * 4 <= kHalves * kTile, "a warp's weighted values in its ring");
    static constexpr int kStep = D + 4;         // between heads of a buffer of weighted values: no bank conflicts
    static constexpr int kSmem = kRing + 2 * 8 * NT * kStep * 4;
};

// n / d of n < 2^31 by one multiplication: mul = ceil(2^(31 + l) / d), l = ceil(log2 d).
struct PaDiv {
    uint32_t mul;
    int shift;
};

template <int DT>
__device__ __forceinline__ uint32_t pa_pack(float x, float y) {
    if (DT == 1) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <int DT>
__device__ __forceinline__ float2 pa_unpack(uint32_t w) {
    if (DT == 1) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int DT>
__device__ __forceinline__ void pa_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (DT == 1)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// 16 bytes global -> shared, zeros where `ok` is not set (nothing is read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ int pa_len(const PagedAttnArgs& a, int b) {
    const long long cap = static_cast<long long>(a.max_pages) * a.page;
    const int most = a.max_len < cap ? a.max_len : static_cast<int>(cap);
    return max(0, min(a.lens[b], most));
}

// The new token's position, -1: none, as where its sequence's length was cut to `len`.
__device__ __forceinline__ int pa_new(const PagedAttnArgs& a, int b, int len) { return a.k_new && a.lens[b] == len ? len - 1 : -1; }

// The parts of units cut over CTAs: 8 NT heads' weighted values, then their maxima and sums.
struct PaParts {
    float* acc;  // [2 CTAs][heads][D]: a CTA's first part of a unit begun before its range, its part of one that goes on
    float* ml;   // [2 CTAs][2][heads]
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Up to so many sequences are taken longest first, where they are more than the GPU holds at once (31 of 130 to 8000
// keys, 4 key heads: 41 -> 34 us); finding their order among 192 costs each CTA more than it gives.
constexpr int kPaSort = 64;
// A place in the list of rounds: round r of one (sequence, key head, tile of heads).
struct PaPlace {
    int b, kvh, tile, r, rounds, len, fresh;  // fresh: the new token's position
    template <int kRound>
    __device__ __forceinline__ void next(const PagedAttnArgs& a, int tiles) {
        if (++r < rounds) return;
        r = 0;
        if (++tile < tiles) return;
        tile = 0;
        if (++kvh < a.Hkv) return;
        kvh = 0;
        do {
            if (++b >= a.B) {
                rounds = 0;
                return;
            }
            len = pa_len(a, b);
            fresh = pa_new(a, b, len);
            rounds = (len + kRound - 1) / kRound;
        } while (rounds == 0);
    }
};

// kCluster > 0: a cluster of so many CTAs takes one unit. 0: all units' rounds
// in equal ranges.
template <int DT, int D, int NT, int kCluster>
__device__ __forceinline__ void pa_units(const PagedAttnArgs& a, int tiles, const PaDiv& div, const PaParts& parts) {
    using C = PaCfg<D, NT>;
    constexpr int kHeads = 8 * NT, kHalves = C::kHalves, kTile = C::kTile, kKs = D / 16, kRound = C::kRound;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    extern __shared__ __align__(128) unsigned char smem[];  // (1024 would leave one CTA a multiprocessor at D = 256)
    __shared__ long long scan[kWarps];
    __shared__ int first_s[4];
    __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
    __shared__ float part_m[kHeads], part_l[kHeads];  // of a cluster's CTA
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, g = lane >> 2, q4 = lane & 3;
    constexpr int kShare = kCluster > 0 ? kCluster : 1;
    const int rank = blockIdx.x % kShare;
    const int units = a.Hkv * tiles, group = a.Hq / a.Hkv;

    // ---- this CTA's range of the rounds
    PaPlace cur;
    long long lo = 0, left, total = 0, ctas = 0;
    if (kCluster > 0) {
        const int unit = blockIdx.x / kShare;
        cur.b = unit / units, cur.kvh = unit % units / tiles, cur.tile = unit % tiles;
        if (a.B > 1 && a.B <= kPaSort && gridDim.x > kSms * C::kCtas) {
            int* lens = reinterpret_cast<int*>(smem);  // (the ring is not in use yet)
            const int all = (a.B + 3) & ~3;
            if (t < all) lens[t] = t < a.B ? pa_len(a, t) : -1;
            __syncthreads();
            if (t < a.B) {
                const int n = lens[t];
                int before = 0;
                for (int j = 0; j < all; j += 4) {
                    const int4 o = *reinterpret_cast<const int4*>(&lens[j]);
                    before += (o.x > n || (o.x == n && j < t)) + (o.y > n || (o.y == n && j + 1 < t)) +
                              (o.z > n || (o.z == n && j + 2 < t)) + (o.w > n || (o.w == n && j + 3 < t));
                }
                if (before == cur.b) first_s[0] = t;
            }
            __syncthreads();
            cur.b = first_s[0];
        }
        cur.len = pa_len(a, cur.b);
        cur.fresh = pa_new(a, cur.b, cur.len);
        cur.rounds = (cur.len + kRound - 1) / kRound;
        cur.r = static_cast<int>(static_cast<long long>(cur.rounds) * rank / kShare);
        left = static_cast<long long>(cur.rounds) * (rank + 1) / kShare - cur.r;
    } else {
        const int per = (a.B + kThreads - 1) / kThreads;
        const int b0 = t * per, b1 = min(a.B, b0 + per);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += (long long)((pa_len(a, b) + kRound - 1) / kRound) * units;
        long long incl = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, m);
            if (lane >= m) incl += o;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        long long before = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
        // every CTA that takes part has a round at least (the join counts on it)
        ctas = min(static_cast<long long>(gridDim.x), total);
        // the sequences without keys
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            if (pa_len(a, b) > 0) continue;
            for (int i = t; i < a.Hq * D / 2; i += kThreads) static_cast<uint32_t*>(a.out)[(long long)b * a.Hq * D / 2 + i] = 0u;
            if (a.lse)
                for (int i = t; i < a.Hq; i += kThreads) a.lse[(long long)b * a.Hq + i] = -INFINITY;
        }
        if (blockIdx.x >= ctas) return;
        lo = blockIdx.x * total / ctas;
        left = (blockIdx.x + 1) * total / ctas - lo;
        long long x0 = before + incl - mine;
        if (lo >= x0 && lo < x0 + mine) {
            for (int b = b0; b < b1; ++b) {
                const int len = pa_len(a, b), rounds = (len + kRound - 1) / kRound;
                const long long n = (long long)rounds * units;
                if (lo < x0 + n) {
                    first_s[0] = b, first_s[1] = static_cast<int>((lo - x0) / rounds);
                    first_s[2] = static_cast<int>((lo - x0) % rounds), first_s[3] = len;
                    break;
                }
                x0 += n;
            }
        }
        __syncthreads();
        cur.b = first_s[0], cur.kvh = first_s[1] / tiles, cur.tile = first_s[1] % tiles, cur.r = first_s[2], cur.len = first_s[3];
        cur.fresh = pa_new(a, cur.b, cur.len);
        cur.rounds = (cur.len + kRound - 1) / kRound;
    }

    // ---- the warp's ring
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * kHalves * kTile;
    const char* kp = static_cast<const char*>(a.k_pool);
    const char* vp = static_cast<const char*>(a.v_pool);
    constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks;
    const int c8 = lane % kChunks, rr = lane / kChunks;
    PaPlace ld = cur;  // the next round to load
    // lane r < 16 (and r + 16) holds row r of that round: its number in the pool (-1: not there)
    auto find_row = [&]() -> int {
        const int j = ld.r * kRound + warp * 16 + (lane & 15);
        if (j >= ld.len) return -1;
        const int p = static_cast<int>((static_cast<unsigned long long>(j) * div.mul) >> div.shift);
        const int pg = a.table[(long long)ld.b * a.max_pages + p];
        if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.n_pages)) return -1;
        return (pg * a.Hkv + ld.kvh) * a.page + (j - p * a.page);
    };
    int row = find_row();
    // one half of the round: its keys (pool kp, new rows kn) or values
    auto load = [&](uint32_t to, const char* pool, const void* fresh) {
        const char* base = pool + c8 * 16;
        const int newest = ld.fresh - (ld.r * kRound + warp * 16);  // the new token's row
        if (static_cast<unsigned>(newest) < 16u) {
            const char* nw = static_cast<const char*>(fresh) + ((long long)ld.b * a.Hkv + ld.kvh) * C::kRow + c8 * 16;
            const int there = __shfl_sync(0xffffffffu, row, newest);
            const bool keep = ld.tile == 0 && rr == 0 && there >= 0;
            uint4 w;
            if (keep) w = *reinterpret_cast<const uint4*>(nw);
#pragma unroll
            for (int i = 0; i < 16; i += kAtOnce) {
                const int r = i + rr, n = __shfl_sync(0xffffffffu, row, r);
                cp16(to + r * C::kRow + ((c8 ^ (r & 7)) << 4), r == newest ? nw : base + (long long)max(n, 0) * C::kRow, n >= 0);
            }
            if (keep) *reinterpret_cast<uint4*>(const_cast<char*>(base) + (long long)there * C::kRow) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 16; i += kAtOnce) {
                const int r = i + rr, n = __shfl_sync(0xffffffffu, row, r);
                cp16(to + r * C::kRow + ((c8 ^ (r & 7)) << 4), base + (long long)max(n, 0) * C::kRow, n >= 0);
            }
        }
    };
    // which rows of the rounds in flight hold keys, 16 bits a round, the oldest lowest
    unsigned long long masks = 0;
    long long issued = 0;
    int in_masks = 0;  // rounds in `masks`
    uint32_t to = ring;
    auto issue = [&](bool values) {
        if (issued < 2 * left) {
            if (!values) {
                masks |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu) << (16 * in_masks);
                ++in_masks;
                load(to, kp, a.k_new);
            } else {
                load(to, vp, a.v_new);
                if (issued + 1 < 2 * left) {
                    ld.template next<kRound>(a, tiles);
                    row = find_row();
                }
            }
            ++issued;
            to = to + kTile == ring + kHalves * kTile ? ring : to + kTile;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kHalves - 1; ++i) issue(i & 1);

    uint32_t qf[NT][kKs][2];
    float acc[NT][kKs][4], m[NT][2], l[NT][2];
    bool begin = true;
    int piece_r0 = 0, h0 = 0, nh = 0;
    const float sc = a.scale * kLog2e;
    float* part = reinterpret_cast<float*>(smem + C::kRing);  // of a cluster's CTA
    uint32_t from = ring;
    for (long long i = 0; i < left; ++i) {
        if (begin) {
            begin = false;
            piece_r0 = cur.r;
            h0 = cur.kvh * group + cur.tile * kHeads;
            nh = min(kHeads, group - cur.tile * kHeads);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int h = n * 8 + g;
                const uint16_t* qp = static_cast<const uint16_t*>(a.q) + ((long long)cur.b * a.Hq + h0 + h) * D;
#pragma unroll
                for (int k = 0; k < kKs; ++k) {
                    qf[n][k][0] = h < nh ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + q4 * 2) : 0u;
                    qf[n][k][1] = h < nh ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + q4 * 2 + 8) : 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][k][e] = 0.f;
                }
                m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
            }
        }
        // ---- scores of 16 keys x 8 NT heads
        cp_wait<kHalves - 2>();
        __syncwarp();
        issue((kHalves - 1) & 1);  // into the half that the last values left
        const uint32_t there = static_cast<uint32_t>(masks) & 0xFFFFu;
        masks >>= 16;
        --in_masks;
        constexpr int kWays = NT == 1 ? 4 : 2;
        float x[NT][kWays][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int w = 0; w < kWays; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][w][e] = 0.f;
        {
            const int r = lane & 15, ch = lane >> 4;
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
                uint32_t f[4];
                ldsm4(f, from + r * C::kRow + (((2 * k + ch) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) pa_mma<DT>(x[n][k % kWays], f, qf[n][k][0], qf[n][k][1]);
            }
        }
        from = from + kTile == ring + kHalves * kTile ? ring : from + kTile;
        uint32_t ph[NT][2], pl[NT][2];
        const bool k0 = (there >> g) & 1, k1 = (there >> (g + 8)) & 1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = x[n][0][e] + x[n][1][e];
                if (kWays == 4) v += x[n][kWays - 2][e] + x[n][kWays - 1][e];
                y[e] = (e < 2 ? k0 : k1) ? v * sc : -INFINITY;
            }
            float p[4], corr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = fmaxf(y[e], y[e + 2]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                top = fmaxf(top, m[n][e]);
                const float base = top == -INFINITY ? 0.f : top;
                corr[e] = ex2(m[n][e] - base);
                m[n][e] = top;
                p[e] = ex2(y[e] - base), p[e + 2] = ex2(y[e + 2] - base);
                l[n][e] = l[n][e] * corr[e] + (p[e] + p[e + 2]);
            }
            if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                for (int k = 0; k < kKs; ++k) {
                    acc[n][k][0] *= corr[0], acc[n][k][1] *= corr[1];
                    acc[n][k][2] *= corr[0], acc[n][k][3] *= corr[1];
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float w0 = p[2 * e] * kPaUp<DT>, w1 = p[2 * e + 1] * kPaUp<DT>;
                const uint32_t hi2 = pa_pack<DT>(w0, w1);
                const float2 back = pa_unpack<DT>(hi2);
                ph[n][e] = movm(hi2);
                pl[n][e] = movm(pa_pack<DT>(w0 - back.x, w1 - back.y));
            }
        }
        // ---- weighted values
        cp_wait<kHalves - 2>();
        __syncwarp();
        issue(kHalves & 1);  // into the half that these keys left
        {
            const int r = (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < kKs; k += 2) {
                uint32_t f[2][4];
                ldsm4t(f[0], from + r * C::kRow + (((2 * k + ch) ^ (r & 7)) << 4));
                ldsm4t(f[1], from + r * C::kRow + (((2 * k + 2 + ch) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    pa_mma<DT>(acc[n][k], f[0], ph[n][0], ph[n][1]);
                    pa_mma<DT>(acc[n][k + 1], f[1], ph[n][0], ph[n][1]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    pa_mma<DT>(acc[n][k], f[0], pl[n][0], pl[n][1]);
                    pa_mma<DT>(acc[n][k + 1], f[1], pl[n][0], pl[n][1]);
                }
            }
        }
        from = from + kTile == ring + kHalves * kTile ? ring : from + kTile;

        // ---- the end of a unit, or of this CTA's part of it
        const bool last = cur.r + 1 == cur.rounds;
        if (last || i + 1 == left) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
                    if (g == 0) sm_m[warp][n * 8 + q4 * 2 + e] = m[n][e], sm_l[warp][n * 8 + q4 * 2 + e] = l[n][e];
                }
            __syncthreads();
            float f[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w][n * 8 + q4 * 2 + e]);
                    f[n][e] = ex2(m[n][e] - (top == -INFINITY ? 0.f : top)) * (1.f / kPaUp<DT>);
                }
            // element (head 8 n + 2 q4 + e, value 16 k + g + 8 r). At the end of the range every warp has a buffer,
            // its ring; before, the ring is being filled, and the warps of each parity take turns at one.
            const bool end = i + 1 == left;
            float* bufs = reinterpret_cast<float*>(end ? smem : smem + C::kRing);
            const int n_bufs = end ? kWarps : 2, apart = end ? kHalves * kTile / 4 : kHeads * C::kStep;
            float* mybuf = bufs + (end ? warp : warp & 1) * apart;
#pragma unroll 1
            for (int turn = 0; turn < (end ? 1 : kWarps / 2); ++turn) {
                if (end || warp / 2 == turn) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < kKs; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int at = (n * 8 + q4 * 2 + (e & 1)) * C::kStep + k * 16 + g + (e >> 1) * 8;
                                const float v = acc[n][k][e] * f[n][e & 1];
                                mybuf[at] = turn == 0 ? v : mybuf[at] + v;
                            }
                }
                __syncthreads();
            }
            const bool whole = kCluster == 0 && last && piece_r0 == 0;
            const long long slot = 2ll * blockIdx.x + (piece_r0 == 0 ? 1 : 0);
            for (int at = t * 2; at < nh * D; at += kThreads * 2) {
                const int h = at / D;
                float v0 = 0.f, v1 = 0.f;
                for (int w = 0; w < n_bufs; ++w) {
                    const float2 o = *reinterpret_cast<const float2*>(bufs + w * apart + h * C::kStep + at % D);
                    v0 += o.x, v1 += o.y;
                }
                if (whole) {
                    float top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w][h]);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) sum += sm_l[w][h] * ex2(sm_m[w][h] - (top == -INFINITY ? 0.f : top));
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + ((long long)cur.b * a.Hq + h0) * D + at) =
                        pa_pack<DT>(v0 * inv, v1 * inv);
                } else if (kCluster > 0) {
                    *reinterpret_cast<float2*>(part + at) = make_float2(v0, v1);
                } else {
                    *reinterpret_cast<float2*>(parts.acc + slot * kHeads * D + at) = make_float2(v0, v1);
                }
            }
            if (t < nh) {
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w][t]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sum += sm_l[w][t] * ex2(sm_m[w][t] - (top == -INFINITY ? 0.f : top));
                if (whole) {
                    if (a.lse) a.lse[(long long)cur.b * a.Hq + h0 + t] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
                } else if (kCluster > 0) {
                    part_m[t] = top, part_l[t] = sum;
                } else {
                    parts.ml[(slot * 2) * kHeads + t] = top;
                    parts.ml[(slot * 2 + 1) * kHeads + t] = sum;
                }
            }
            __syncthreads();
            begin = true;
        }
        if (kCluster == 0) cur.template next<kRound>(a, tiles);
        else ++cur.r;
    }
    if (kCluster == 0) return;

    // ---- the unit's parts: each CTA finishes a share of the values
    h0 = cur.kvh * group + cur.tile * kHeads;
    nh = min(kHeads, group - cur.tile * kHeads);
    if (left == 0) {
        for (int i = t; i < nh * D; i += kThreads) part[i] = 0.f;
        if (t < nh) part_m[t] = -INFINITY, part_l[t] = 0.f;
    }
    __syncthreads();
    if (kCluster > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const int each = nh * D / kShare;
    for (int i = t * 2; i < each; i += kThreads * 2) {
        const int at = rank * each + i, h = at / D;
        float pm[kShare], pl[kShare], top = -INFINITY, sum = 0.f, v0 = 0.f, v1 = 0.f;
        float2 pv[kShare];
#pragma unroll
        for (int c = 0; c < kShare; ++c) {
            pm[c] = ld_cluster_f32(cluster_map(smem_u32(&part_m[h]), c));
            pl[c] = ld_cluster_f32(cluster_map(smem_u32(&part_l[h]), c));
            pv[c] = ld_cluster_f32x2(cluster_map(smem_u32(part + at), c));
        }
#pragma unroll
        for (int c = 0; c < kShare; ++c) top = fmaxf(top, pm[c]);
#pragma unroll
        for (int c = 0; c < kShare; ++c) {
            const float f = ex2(pm[c] - (top == -INFINITY ? 0.f : top));
            sum += pl[c] * f, v0 += pv[c].x * f, v1 += pv[c].y * f;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + ((long long)cur.b * a.Hq + h0) * D + at) =
            pa_pack<DT>(v0 * inv, v1 * inv);
        if (a.lse && at % D == 0) a.lse[(long long)cur.b * a.Hq + h0 + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
    if (kCluster > 1) {
        cluster_arrive();  // no CTA leaves while another reads its part
        cluster_wait();
    }
}

template <int DT, int D, int NT>
__global__ void __launch_bounds__(PaCfg<D, NT>::kThreads, PaCfg<D, NT>::kCtas)
    paged_attention_kernel(PagedAttnArgs a, int tiles, PaDiv div, PaParts parts) {
    pa_units<DT, D, NT, 0>(a, tiles, div, parts);
}
template <int DT, int D, int NT, int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(PaCfg<D, NT>::kThreads, PaCfg<D, NT>::kCtas)
    paged_attention_cluster_kernel(PagedAttnArgs a, int tiles, PaDiv div) {
    pa_units<DT, D, NT, kCluster>(a, tiles, div, PaParts{});
}

// Joins the parts of one query head of a unit that lies in several of the
// `grid` CTAs' ranges: CTA (head of the unit, unit, 64 values), kPaSets
// interleaved sets of parts with 16 threads of four values each. Which CTAs
// those are it finds from the lengths, as they did, while they still run; behind
// them all its loads go at once.
constexpr int kPaSets = 32, kPaCols = 16;
constexpr int kPaFew = 38;  // units, and so sequences, that are cut over all CTAs (pa_route), at most
static_assert(16 * (kPaFew + 1) > kSms * 4 && PaCfg<64, 1>::kCtas <= 4 && PaCfg<128, 1>::kCtas <= 4 && PaCfg<256, 1>::kCtas <= 4, "CTAs of a launch");
template <int DT, int D>
__global__ void __launch_bounds__(kPaSets* kPaCols) paged_attention_join_kernel(PagedAttnArgs a, int tiles, int heads, int grid, PaParts parts) {
    constexpr int kCols = kPaCols, kThreads = kPaSets * kCols, kW = kThreads / 32, kHold = kSms * 4;
    __shared__ float4 sums[kPaSets][kCols];
    __shared__ float red[2][kW], factor[kHold];
    __shared__ int rounds[kPaFew];
    const int t = threadIdx.x, col = t % kCols, set = t / kCols, lane = t & 31, warp = t >> 5, d0 = (blockIdx.z * kCols + col) * 4;
    const int units = a.Hkv * tiles, b = blockIdx.y / units, u = blockIdx.y % units;
    const int hh = blockIdx.x, group = a.Hq / a.Hkv, kvh = u / tiles, tile = u % tiles;
    // (lens stands since before the kernel that this one follows)
    if (t < a.B) rounds[t] = (pa_len(a, t) + 63) / 64;
    __syncthreads();
    long long total = 0, first = 0;  // round of the unit
    for (int i = 0; i < a.B; ++i) {
        if (i < b) first += rounds[i];
        total += rounds[i];
    }
    total *= units, first = first * units + (long long)u * rounds[b];
    const long long ctas = min(static_cast<long long>(grid), total);
    int c0 = 0, n = 0;
    if (rounds[b] > 0) {
        // round r is CTA c's, the largest with floor(c total / ctas) <= r
        c0 = static_cast<int>(((first + 1) * ctas - 1) / total);
        n = static_cast<int>(((first + rounds[b]) * ctas - 1) / total) - c0 + 1;
    }
    pdl_wait();
    pdl_trigger();
    if (n <= 1 || tile * heads + hh >= group) return;  // no keys, or finished
    const long long h = (long long)b * a.Hq + kvh * group + tile * heads + hh;
    // the first CTA's part is its second one
    auto slot = [&](int i) { return 2ll * (c0 + i) + (i == 0 ? 1 : 0); };
    auto part = [&](int i) { return *reinterpret_cast<const float4*>(parts.acc + (slot(i) * heads + hh) * D + d0); };
    constexpr int kAhead = 10;
    float4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ahead[k] = set + k * kPaSets < n ? part(set + k * kPaSets) : make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -INFINITY;
    for (int i = t; i < n; i += kThreads) top = fmaxf(top, factor[i] = parts.ml[slot(i) * 2 * heads + hh]);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (lane == 0) red[0][warp] = top;
    float l = t < n ? parts.ml[(slot(t) * 2 + 1) * heads + hh] : 0.f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) top = fmaxf(top, red[0][w]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int i = t; i < n; i += kThreads) {
        const float f = ex2(factor[i] - base);
        if (i >= kThreads) l = parts.ml[(slot(i) * 2 + 1) * heads + hh];
        sum += l * f;
        factor[i] = f;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, const float4& p) {
        const float f = factor[i];
        v.x += f * p.x, v.y += f * p.y, v.z += f * p.z, v.w += f * p.w;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (set + k * kPaSets < n) add(set + k * kPaSets, ahead[k]);
    for (int i = set + kAhead * kPaSets; i < n; i += kPaSets) add(i, part(i));
    sums[set][col] = v;
    __syncthreads();
    if (set != 0) return;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) sum += red[1][w];
#pragma unroll
    for (int s = 1; s < kPaSets; ++s) {
        const float4 o = sums[s][col];
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + h * D + d0) =
        make_uint2(pa_pack<DT>(v.x * inv, v.y * inv), pa_pack<DT>(v.z * inv, v.w * inv));
    if (t == 0 && blockIdx.z == 0 && a.lse) a.lse[h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// CTAs of a unit's cluster, or 0: units are cut over all CTAs and joined by a second kernel. `ctas`: what the GPU holds at
// once. A round takes 0.9 us in a CTA alone on its multiprocessor, a CTA 4 us besides, the second kernel 5.
//  * Few long units cannot fill the GPU by 8 CTAs each: one of 4 key heads of 128 and 12000 keys takes 13 us cut over
//    all, 25 in clusters; of 3000 keys 10 and 9.1; 8 such sequences of 12000 keys 40 and 37.
//  * More CTAs a unit even out ragged lengths and shorten the longest unit; each costs its start (64 sequences of 4 key
//    heads in clusters of 1, 2, 4, 8: up to 700 keys 18, 24, 27, 42 us; up to 3000 55, 40, 41, 57; up to 12000 203,
//    138, 109, 131). Fewer than half the places are worth filling up (16 sequences of 700: 13, 9.7, 8.5, 14).
// `rounds` are those of max_len, as the host does not know the lengths; the figures above had the longest length for it. A
// bound far above the lengths takes more CTAs a unit than they need (the 64 sequences of up to 700, with a bound of 700 and
// of 131072: 16.3 and 21.2 us; up to 3000: 36.5 and 36.7).
int pa_route(long long units, int rounds, int ctas) {
    if (16 * units <= ctas && rounds > 64) return 0;
    const int most = units * 5 <= ctas * 2 ? 8 : units * 2 <= ctas * 3 ? 4 : 2;
    int c = rounds <= 12 ? 1 : rounds <= 40 ? 2 : rounds <= 80 ? 4 : 8;
    while (c < 8 && c < rounds && units * c * 2 < ctas) c *= 2;
    return c < most ? c : most;
}
struct PaPlan {
    int nt, heads, tiles, ctas, cluster;
    long long units;
    size_t acc, ml, total;
};
template <int D>
int pa_ctas(int nt) {
    return kSms * (nt == 1 ? PaCfg<D, 1>::kCtas : PaCfg<D, D == 256 ? 1 : 2>::kCtas);
}
PaPlan pa_plan(int B, int Hq, int Hkv, int d, int max_len) {
    PaPlan p{};
    const int group = Hq / Hkv;
    // 16 heads of 256 values would not fit the registers: at dimension 256 a unit has 8 heads, and a second one reads the
    // keys again
    p.nt = group <= 8 || d == 256 ? 1 : 2;
    p.heads = 8 * p.nt;
    p.tiles = (group + p.heads - 1) / p.heads;
    p.ctas = d == 256 ? pa_ctas<256>(p.nt) : d == 128 ? pa_ctas<128>(p.nt) : pa_ctas<64>(p.nt);
    p.units = (long long)B * Hkv * p.tiles;
    p.cluster = pa_route(p.units, (max_len + 63) / 64, p.ctas);
    if (p.cluster) return p;
    p.acc = 0;
    p.ml = p.acc + static_cast<size_t>(2) * p.ctas * p.heads * d * 4;
    p.total = p.ml + static_cast<size_t>(2) * p.ctas * 2 * p.heads * 4;
    return p;
}
PaDiv pa_div(int d) {
    int l = 0;
    while ((1ll << l) < d) ++l;
    return PaDiv{static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

template <int DT, int D, int NT>
cudaError_t launch_nt(const PagedAttnArgs& a, const PaPlan& p, const PaParts& parts, cudaStream_t s) {
    using C = PaCfg<D, NT>;
    const void* f = p.cluster == 8   ? reinterpret_cast<const void*>(paged_attention_cluster_kernel<DT, D, NT, 8>)
                    : p.cluster == 4 ? reinterpret_cast<const void*>(paged_attention_cluster_kernel<DT, D, NT, 4>)
                    : p.cluster == 2 ? reinterpret_cast<const void*>(paged_attention_cluster_kernel<DT, D, NT, 2>)
                    : p.cluster == 1 ? reinterpret_cast<const void*>(paged_attention_cluster_kernel<DT, D, NT, 1>)
                                     : reinterpret_cast<const void*>(paged_attention_kernel<DT, D, NT>);
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    int tiles = p.tiles, heads = p.heads;
    PaDiv div = pa_div(a.page);
    void* args[] = {const_cast<PagedAttnArgs*>(&a), &tiles, &div, const_cast<PaParts*>(&parts)};
    // 65535 sequences, 1024 key heads, 8 tiles, 2 CTAs (with so many units): below 2^31
    const unsigned grid = static_cast<unsigned>(p.cluster ? p.units * p.cluster : p.ctas);
    e = launch_kernel(f, dim3(grid), dim3(C::kThreads), C::kSmem, true, s, args);
    if (e != cudaSuccess || p.cluster) return e;
    int ctas = p.ctas;
    void* jargs[] = {const_cast<PagedAttnArgs*>(&a), &tiles, &heads, &ctas, const_cast<PaParts*>(&parts)};
    const int group = a.Hq / a.Hkv;
    return launch_kernel(reinterpret_cast<const void*>(paged_attention_join_kernel<DT, D>),
                         dim3(heads < group ? heads : group, static_cast<unsigned>(p.units), D / (4 * kPaCols)), dim3(kPaSets * kPaCols), 0, true, s,
                         jargs);
}

template <int DT>
cudaError_t launch_dt(const PagedAttnArgs& a, const PaPlan& p, const PaParts& parts, cudaStream_t s) {
    if (a.d == 64) return p.nt == 1 ? launch_nt<DT, 64, 1>(a, p, parts, s) : launch_nt<DT, 64, 2>(a, p, parts, s);
    if (a.d == 128) return p.nt == 1 ? launch_nt<DT, 128, 1>(a, p, parts, s) : launch_nt<DT, 128, 2>(a, p, parts, s);
    return launch_nt<DT, 256, 1>(a, p, parts, s);
}

}  // namespace

size_t paged_attention_ws_bytes(int B, int Hq, int Hkv, int d, int max_len) { return pa_plan(B, Hq, Hkv, d, max_len).total; }

cudaError_t launch_paged_attention(const PagedAttnArgs& a, int dtype, void* ws, cudaStream_t s) {
    const PaPlan p = pa_plan(a.B, a.Hq, a.Hkv, a.d, a.max_len);
    char* w = static_cast<char*>(ws);
    const PaParts parts{reinterpret_cast<float*>(w + p.acc), reinterpret_cast<float*>(w + p.ml)};
    return dtype == 1 ? launch_dt<1>(a, p, parts, s) : launch_dt<2>(a, p, parts, s);
}

}  // namespace escha
