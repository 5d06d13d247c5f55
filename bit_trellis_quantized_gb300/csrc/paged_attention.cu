// Attention of one new token a sequence over a paged key-value cache.
//
// Per sequence b and query head h, over the keys j < lens[b] of its key head:
//   x_j = scale q . k_j,  out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
//   lse = m + ln sum_j e^(x_j - m),  m = max_j x_j.
// Parts over different keys join by their (m, sum, weighted values). Scores,
// maxima, sums and weighted values are held in f32. A weight e^(x - m) enters
// the tensor cores as two 16-bit parts (value, remainder), so that the one
// rounding that shows is that of `out` to its type.
//
// Bound: the one read of K and V (a key is used by Hq / Hkv heads: at most 4 x
// 16 flops a byte). So the layout serves the loads:
//   * A unit is one (sequence, key head, up to 8 NT query heads); its keys are
//     taken in rounds of 64, 16 a warp. All units' rounds, in order, are cut
//     into equal ranges, one a CTA: however ragged the lengths, every
//     multiprocessor reads the same number of bytes. A unit that lies in one
//     range is finished by its CTA; the parts of the others go to the
//     workspace, at most two a CTA, and are joined by a second kernel.
//   * Each warp fills its own ring of 16-key stages (cp.async, 16 bytes a lane,
//     rows of the pages wherever they are) and waits for nobody else. Rows that
//     are not there are filled with zeros and masked.
//   * Keys are the M of both products (scores K Q^T, values V^T P^T: m16n8k16),
//     so that 8 query heads fill the instruction's N exactly.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr int kPaWarps = 4;
constexpr int kPaThreads = kPaWarps * 32;
constexpr int kPaRound = 16 * kPaWarps;  // keys of a round
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct PaCfg {
    static constexpr int kStages = D == 64 ? 4 : 3;
    static constexpr int kCtas = D == 256 ? 1 : D == 128 ? 2 : 3;  // a multiprocessor
    static constexpr int kRow = D * 2;                              // bytes of a row
    static constexpr int kTile = 16 * kRow;                         // one stage's keys (and values) of a warp
    static constexpr int kRing = kPaWarps * kStages * 2 * kTile;
};
template <int D, int NT>
constexpr int pa_smem() {
    return PaCfg<D>::kRing + 2 * 8 * NT * D * 4;
}

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

// One part of a unit: 8 NT heads' weighted values, then their maxima and sums.
struct PaParts {
    float* acc;   // [2 G][heads][D]
    float* ml;    // [2 G][2][heads]
    int2* units;  // [B][units a sequence]: first CTA and number of parts (0: finished by its CTA)
};

// A place in the list of rounds: round r of unit u of sequence b.
struct PaPlace {
    int b, u, r, rounds, len;
    __device__ __forceinline__ void next(const PagedAttnArgs& a, int units) {
        if (++r < rounds) return;
        r = 0;
        if (++u < units) return;
        u = 0;
        do {
            if (++b >= a.B) {
                rounds = 0;
                return;
            }
            len = pa_len(a, b);
            rounds = (len + kPaRound - 1) / kPaRound;
        } while (rounds == 0);
    }
};

template <int DT, int D, int NT>
__global__ void __launch_bounds__(kPaThreads) paged_attention_kernel(PagedAttnArgs a, int tiles, PaParts parts) {
    using C = PaCfg<D>;
    constexpr int kHeads = 8 * NT, kStages = C::kStages, kTile = C::kTile, kKs = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ long long scan[kPaWarps];
    __shared__ int first_s[4];
    __shared__ float sm_m[kPaWarps][kHeads], sm_l[kPaWarps][kHeads];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, g = lane >> 2, q4 = lane & 3;
    const int units = a.Hkv * tiles, group = a.Hq / a.Hkv;

    // ---- this CTA's range of the rounds
    const int per = (a.B + kPaThreads - 1) / kPaThreads;
    const int b0 = t * per, b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += (long long)((pa_len(a, b) + kPaRound - 1) / kPaRound) * units;
    long long incl = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    // every CTA that takes part has a round at least (the join counts on it)
    const long long ctas = min(static_cast<long long>(gridDim.x), total);
    if (blockIdx.x >= ctas) return;
    const long long lo = blockIdx.x * total / ctas, hi = (blockIdx.x + 1) * total / ctas;
    long long x0 = before + incl - mine;
    if (lo >= x0 && lo < x0 + mine) {
        for (int b = b0; b < b1; ++b) {
            const int len = pa_len(a, b), rounds = (len + kPaRound - 1) / kPaRound;
            const long long n = (long long)rounds * units;
            if (lo < x0 + n) {
                const int at = static_cast<int>(lo - x0);
                first_s[0] = b, first_s[1] = at / rounds, first_s[2] = at % rounds, first_s[3] = len;
                break;
            }
            x0 += n;
        }
    }
    __syncthreads();
    PaPlace cur;
    cur.b = first_s[0], cur.u = first_s[1], cur.r = first_s[2], cur.len = first_s[3];
    cur.rounds = (cur.len + kPaRound - 1) / kPaRound;

    // ---- the warp's ring
    unsigned char* ring = smem + warp * kStages * 2 * kTile;
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const char* kp = static_cast<const char*>(a.k_pool);
    const char* vp = static_cast<const char*>(a.v_pool);
    PaPlace ld = cur;       // the next round to load
    long long left = hi - lo;
    // lane r < 16 holds row r of the round to load: its offset in values (-1: not there)
    auto find_row = [&](const PaPlace& p) -> long long {
        const int j = p.r * kPaRound + warp * 16 + (lane & 15);
        if (j >= p.len) return -1;
        const int pg = a.table[(long long)p.b * a.max_pages + j / a.page];
        if (pg < 0 || pg >= a.n_pages) return -1;
        return (((long long)pg * a.Hkv + p.u / tiles) * a.page + j % a.page) * D;
    };
    long long row = find_row(ld);
    auto load = [&](int stage) {
        constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks > 0 ? 32 / kChunks : 1;
        const uint32_t ks = ring_s + stage * 2 * kTile, vs = ks + kTile;
        const int newest = a.k_new ? ld.len - 1 - (ld.r * kPaRound + warp * 16) : -1;  // the new token's row
        const long long fresh = ((long long)ld.b * a.Hkv + ld.u / tiles) * D;
#pragma unroll
        for (int i = 0; i < 16; i += kAtOnce) {
            const int r = i + lane / kChunks, c = lane % kChunks;
            const long long off = __shfl_sync(0xffffffffu, row, r);
            const bool ok = off >= 0;
            const char* ksrc = kp;
            const char* vsrc = vp;
            if (ok) {
                ksrc = kp + (off + c * 8) * 2, vsrc = vp + (off + c * 8) * 2;
                if (r == newest) {
                    const char* kn = static_cast<const char*>(a.k_new) + (fresh + c * 8) * 2;
                    const char* vn = static_cast<const char*>(a.v_new) + (fresh + c * 8) * 2;
                    if (ld.u % tiles == 0) {
                        *reinterpret_cast<uint4*>(const_cast<char*>(ksrc)) = *reinterpret_cast<const uint4*>(kn);
                        *reinterpret_cast<uint4*>(const_cast<char*>(vsrc)) = *reinterpret_cast<const uint4*>(vn);
                    }
                    ksrc = kn, vsrc = vn;
                }
            }
            const uint32_t at = r * C::kRow + ((c ^ (r & 7)) << 4);
            cp16(ks + at, ksrc, ok);
            cp16(vs + at, vsrc, ok);
        }
    };
    uint32_t there = 0;  // bit r of a byte pair per stage: which rows hold keys
    uint32_t masks[kStages];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        masks[i] = 0;
        if (i < left) {
            masks[i] = __ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu;
            load(i);
            if (i + 1 < left) {
                ld.next(a, units);
                row = find_row(ld);
            }
        }
        cp_commit();
    }
    masks[kStages - 1] = 0;

    uint32_t qf[NT][kKs][2];
    float acc[NT][kKs][4], m[NT][2], l[NT][2];
    bool begin = true;
    int piece_r0 = 0;
    const float sc = a.scale * kLog2e;
    int stage = 0;
    for (long long i = 0; i < left; ++i) {
        const int kvh = cur.u / tiles, h0 = kvh * group + (cur.u % tiles) * kHeads;
        const int nh = min(kHeads, group - (cur.u % tiles) * kHeads);
        if (begin) {
            begin = false;
            piece_r0 = cur.r;
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
        cp_wait<kStages - 2>();
        __syncwarp();
        {
            // the stage freed in the last iteration takes the round kStages - 1 ahead
            const int to = stage == 0 ? kStages - 1 : stage - 1;
            if (i + kStages - 1 < left) {
                const uint32_t mk = __ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu;
#pragma unroll
                for (int s = 0; s < kStages; ++s)
                    if (s == to) masks[s] = mk;
                load(to);
                if (i + kStages < left) {
                    ld.next(a, units);
                    row = find_row(ld);
                }
            }
            cp_commit();
        }
#pragma unroll
        for (int s = 0; s < kStages; ++s)
            if (s == stage) there = masks[s];
        const uint32_t ks = ring_s + stage * 2 * kTile, vs = ks + kTile;
        // ---- scores of 16 keys x 8 NT heads
        float x[NT][2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][0][e] = x[n][1][e] = 0.f;
        {
            const int r = lane & 15, ch = lane >> 4;
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
                uint32_t f[4];
                ldsm4(f, ks + r * C::kRow + (((2 * k + ch) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) pa_mma<DT>(x[n][k & 1], f, qf[n][k][0], qf[n][k][1]);
            }
        }
        uint32_t ph[NT][2], pl[NT][2];
        const bool k0 = (there >> g) & 1, k1 = (there >> (g + 8)) & 1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = (e < 2 ? k0 : k1) ? (x[n][0][e] + x[n][1][e]) * sc : -INFINITY;
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
                const uint32_t hi2 = pa_pack<DT>(p[2 * e], p[2 * e + 1]);
                const float2 back = pa_unpack<DT>(hi2);
                ph[n][e] = movm(hi2);
                pl[n][e] = movm(pa_pack<DT>(p[2 * e] - back.x, p[2 * e + 1] - back.y));
            }
        }
        // ---- weighted values
        {
            const int r = (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
                uint32_t f[4];
                ldsm4t(f, vs + r * C::kRow + (((2 * k + ch) ^ (r & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    pa_mma<DT>(acc[n][k], f, ph[n][0], ph[n][1]);
                    pa_mma<DT>(acc[n][k], f, pl[n][0], pl[n][1]);
                }
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;

        // ---- the end of a unit, or of this CTA's part of it
        const bool last = cur.r + 1 == cur.rounds;
        if (last || i + 1 == left) {
            float* buf = reinterpret_cast<float*>(smem + C::kRing);  // [2][kHeads][D]
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
                    for (int w = 0; w < kPaWarps; ++w) top = fmaxf(top, sm_m[w][n * 8 + q4 * 2 + e]);
                    f[n][e] = ex2(m[n][e] - (top == -INFINITY ? 0.f : top));
                }
            // element (head 8 n + 2 q4 + e, value 16 k + g + 8 r): warps 2 and 3, then 1, then 0
            auto each = [&](auto&& fn) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < kKs; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            fn(acc[n][k][e] * f[n][e & 1], (n * 8 + q4 * 2 + (e & 1)) * D + k * 16 + g + (e >> 1) * 8);
            };
            if (warp >= 2) each([&](float v, int at) { buf[(warp - 2) * kHeads * D + at] = v; });
            __syncthreads();
            if (warp == 1) each([&](float v, int at) { buf[kHeads * D + at] += v; });
            if (warp == 0) each([&](float v, int at) { buf[at] += v; });
            __syncthreads();
            const bool whole = last && piece_r0 == 0;
            const long long slot = 2ll * blockIdx.x + (piece_r0 == 0 ? 1 : 0);
            for (int at = t * 2; at < nh * D; at += kPaThreads * 2) {
                const int h = at / D;
                const float v0 = buf[at] + buf[kHeads * D + at], v1 = buf[at + 1] + buf[kHeads * D + at + 1];
                if (whole) {
                    float top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kPaWarps; ++w) top = fmaxf(top, sm_m[w][h]);
#pragma unroll
                    for (int w = 0; w < kPaWarps; ++w)
                        sum += sm_l[w][h] * ex2(sm_m[w][h] - (top == -INFINITY ? 0.f : top));
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + ((long long)cur.b * a.Hq + h0) * D + at) =
                        pa_pack<DT>(v0 * inv, v1 * inv);
                } else {
                    *reinterpret_cast<float2*>(parts.acc + slot * kHeads * D + at) = make_float2(v0, v1);
                }
            }
            if (t < nh) {
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kPaWarps; ++w) top = fmaxf(top, sm_m[w][t]);
#pragma unroll
                for (int w = 0; w < kPaWarps; ++w) sum += sm_l[w][t] * ex2(sm_m[w][t] - (top == -INFINITY ? 0.f : top));
                if (whole) {
                    if (a.lse) a.lse[(long long)cur.b * a.Hq + h0 + t] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
                } else {
                    parts.ml[(slot * 2) * kHeads + t] = top;
                    parts.ml[(slot * 2 + 1) * kHeads + t] = sum;
                }
            }
            if (t == 0 && piece_r0 == 0) {
                // the CTA that holds the unit's last round: the largest c with floor(c total / ctas) <= it
                int2 info = make_int2(0, 0);
                if (!last) {
                    const long long end = lo + i + (cur.rounds - 1 - cur.r);
                    info = make_int2(blockIdx.x, static_cast<int>(((end + 1) * ctas - 1) / total) - static_cast<int>(blockIdx.x) + 1);
                }
                parts.units[(long long)cur.b * units + cur.u] = info;
            }
            __syncthreads();
            begin = true;
        }
        cur.next(a, units);
    }
}

// Joins the parts of one (sequence, query head): 64 threads of four values for
// each of four interleaved sets of parts.
template <int DT, int D>
__global__ void __launch_bounds__(D) paged_attention_join_kernel(PagedAttnArgs a, int tiles, int heads, PaParts parts) {
    constexpr int kCols = D / 4, kSets = 4;
    __shared__ float4 sums[kSets][kCols];
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x, col = t % kCols, set = t / kCols;
    const int group = a.Hq / a.Hkv, kvh = h / group, tile = h % group / heads, hh = h % group % heads;
    uint16_t* out = static_cast<uint16_t*>(a.out) + ((long long)b * a.Hq + h) * D;
    if (pa_len(a, b) == 0) {
        if (set == 0) *reinterpret_cast<uint2*>(out + col * 4) = make_uint2(0u, 0u);
        if (t == 0 && a.lse) a.lse[(long long)b * a.Hq + h] = -INFINITY;
        return;
    }
    const int2 info = parts.units[((long long)b * a.Hkv + kvh) * tiles + tile];
    const int n = info.y;
    if (n == 0) return;
    // the first CTA's part is its second one
    auto slot = [&](int i) { return 2ll * (info.x + i) + (i == 0 ? 1 : 0); };
    float top = -INFINITY;
    for (int i = 0; i < n; ++i) top = fmaxf(top, parts.ml[slot(i) * 2 * heads + hh]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int i = 0; i < n; ++i)
        sum += parts.ml[(slot(i) * 2 + 1) * heads + hh] * ex2(parts.ml[slot(i) * 2 * heads + hh] - base);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = set; i < n; i += kSets) {
        const float f = ex2(parts.ml[slot(i) * 2 * heads + hh] - base);
        const float4 p = *reinterpret_cast<const float4*>(parts.acc + (slot(i) * heads + hh) * D + col * 4);
        v.x += f * p.x, v.y += f * p.y, v.z += f * p.z, v.w += f * p.w;
    }
    sums[set][col] = v;
    __syncthreads();
    if (set == 0) {
        for (int s = 1; s < kSets; ++s) {
            const float4 o = sums[s][col];
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2*>(out + col * 4) = make_uint2(pa_pack<DT>(v.x * inv, v.y * inv), pa_pack<DT>(v.z * inv, v.w * inv));
    }
    if (t == 0 && a.lse) a.lse[(long long)b * a.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

struct PaPlan {
    int nt, heads, tiles, ctas;
    size_t acc, ml, units, total;
};
PaPlan pa_plan(int B, int Hq, int Hkv, int d) {
    PaPlan p{};
    const int group = Hq / Hkv;
    p.nt = group <= 8 ? 1 : 2;
    p.heads = 8 * p.nt;
    p.tiles = (group + p.heads - 1) / p.heads;
    p.ctas = kSms * (d == 256 ? PaCfg<256>::kCtas : d == 128 ? PaCfg<128>::kCtas : PaCfg<64>::kCtas);
    p.acc = 0;
    p.ml = p.acc + static_cast<size_t>(2) * p.ctas * p.heads * d * 4;
    p.units = p.ml + static_cast<size_t>(2) * p.ctas * 2 * p.heads * 4;
    p.total = p.units + static_cast<size_t>(B) * Hkv * p.tiles * sizeof(int2);
    return p;
}

template <int DT, int D, int NT>
cudaError_t launch_nt(const PagedAttnArgs& a, const PaPlan& p, const PaParts& parts, cudaStream_t s) {
    const void* f = reinterpret_cast<const void*>(paged_attention_kernel<DT, D, NT>);
    constexpr int smem = pa_smem<D, NT>();
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int tiles = p.tiles, heads = p.heads;
    void* args[] = {const_cast<PagedAttnArgs*>(&a), &tiles, const_cast<PaParts*>(&parts)};
    e = launch_kernel(f, dim3(p.ctas), dim3(kPaThreads), smem, true, s, args);
    if (e != cudaSuccess) return e;
    void* jargs[] = {const_cast<PagedAttnArgs*>(&a), &tiles, &heads, const_cast<PaParts*>(&parts)};
    return launch_kernel(reinterpret_cast<const void*>(paged_attention_join_kernel<DT, D>), dim3(a.Hq, a.B), dim3(D), 0, true, s,
                         jargs);
}

template <int DT>
cudaError_t launch_dt(const PagedAttnArgs& a, const PaPlan& p, const PaParts& parts, cudaStream_t s) {
    if (a.d == 64) return p.nt == 1 ? launch_nt<DT, 64, 1>(a, p, parts, s) : launch_nt<DT, 64, 2>(a, p, parts, s);
    if (a.d == 128) return p.nt == 1 ? launch_nt<DT, 128, 1>(a, p, parts, s) : launch_nt<DT, 128, 2>(a, p, parts, s);
    return p.nt == 1 ? launch_nt<DT, 256, 1>(a, p, parts, s) : launch_nt<DT, 256, 2>(a, p, parts, s);
}

}  // namespace

size_t paged_attention_ws_bytes(int B, int Hq, int Hkv, int d, int max_len) {
    (void)max_len;
    return pa_plan(B, Hq, Hkv, d).total;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, int dtype, void* ws, cudaStream_t s) {
    const PaPlan p = pa_plan(a.B, a.Hq, a.Hkv, a.d);
    char* w = static_cast<char*>(ws);
    const PaParts parts{reinterpret_cast<float*>(w + p.acc), reinterpret_cast<float*>(w + p.ml),
                        reinterpret_cast<int2*>(w + p.units)};
    return dtype == 1 ? launch_dt<1>(a, p, parts, s) : launch_dt<2>(a, p, parts, s);
}

}  // namespace escha
