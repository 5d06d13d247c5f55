// Gated delta rule: per sequence and value head a state S [dk][dv] in f32 that
// each token decays, corrects along its key and reads along its query:
//   S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q,
// k and q divided by sqrt(sum x^2 + eps) first where eps >= 0.
//
// Token by token (delta_step_kernel): a CTA holds [dk][VS] of one state in
// registers. Both products with the old state, S^T k and S^T q, come from one
// pass over it and one reduction, as o = scale (e^g S^T q + (k . q) u). Bound,
// for one token a sequence: the state's read and write (250 states of 32 x 128
// x 128: 154 us, 6.8 TB/s).
// From kChunkFrom tokens on, in chunks of 32 (below): a kernel over all chunks,
// then one that walks them, bound by the latency of that chain.
#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "trellis_core.cuh"

namespace escha {

namespace {

constexpr int kDrThreads = 256;

template <int DT>
__device__ __forceinline__ float dr_f32(const void* p, long long i) {
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return DT == 1 ? h2f_bits(b) : bf2f_bits(b);
}
template <int DT>
__device__ __forceinline__ uint32_t dr_pack(float x, float y) {
    if (DT == 1) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Sequence s's tokens, kept inside [0, T).
__device__ __forceinline__ void dr_tokens(const DeltaArgs& a, int s, int& t0, int& t1) {
    t0 = max(0, min(a.at[s], a.T));
    t1 = max(t0, min(a.at[s + 1], a.T));
}

template <int DT, int DK, int VS>
__global__ void __launch_bounds__(kDrThreads) delta_step_kernel(DeltaArgs a) {
    constexpr int kLanes = VS / 4;              // threads of one row of the state's part
    constexpr int kRows = kDrThreads / kLanes;  // rows held at once
    constexpr int kPer = DK / kRows > 0 ? DK / kRows : 1;
    static_assert(DK % kRows == 0, "rows");
    __shared__ float ks[2][DK], qs[2][DK];
    __shared__ float4 red[kDrThreads / 32][2][kLanes];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid % kLanes, r0 = tid / kLanes;
    const int hv = blockIdx.y, seq = blockIdx.z, hk = hv / (a.Hv / a.Hk), c0 = blockIdx.x * VS + col * 4;
    int t0, t1;
    dr_tokens(a, seq, t0, t1);
    if (t0 == t1) return;
    float* sp = a.state + (((long long)seq * a.Hv + hv) * DK + r0) * a.dv + c0;
    float4 S[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) S[i] = *reinterpret_cast<const float4*>(sp + (long long)i * kRows * a.dv);
    for (int t = t0; t < t1; ++t) {
        const int p = (t - t0) & 1;
        for (int i = tid; i < 2 * DK; i += kDrThreads) {
            if (i < DK)
                ks[p][i] = dr_f32<DT>(a.k, ((long long)t * a.Hk + hk) * DK + i);
            else
                qs[p][i - DK] = dr_f32<DT>(a.q, ((long long)t * a.Hk + hk) * DK + i - DK);
        }
        const float decay = expf(a.g[(long long)t * a.Hv + hv]), beta = a.beta[(long long)t * a.Hv + hv];
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = dr_f32<DT>(a.v, ((long long)t * a.Hv + hv) * a.dv + c0 + j);
        __syncthreads();
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int i = lane; i < DK; i += 32) {
            const float x = ks[p][i], y = qs[p][i];
            kk += x * x, qq += y * y, kq += x * y;
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, m);
            qq += __shfl_xor_sync(0xffffffffu, qq, m);
            kq += __shfl_xor_sync(0xffffffffu, kq, m);
        }
        const float rk = a.eps >= 0.f ? 1.f / sqrtf(kk + a.eps) : 1.f, rq = (a.eps >= 0.f ? 1.f / sqrtf(qq + a.eps) : 1.f) * a.scale;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float k = ks[p][r0 + i * kRows], q = qs[p][r0 + i * kRows];
            x.x += S[i].x * k, x.y += S[i].y * k, x.z += S[i].z * k, x.w += S[i].w * k;
            y.x += S[i].x * q, y.y += S[i].y * q, y.z += S[i].z * q, y.w += S[i].w * q;
        }
#pragma unroll
        for (int m = 16; m >= kLanes; m >>= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, m), x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
            x.z += __shfl_xor_sync(0xffffffffu, x.z, m), x.w += __shfl_xor_sync(0xffffffffu, x.w, m);
            y.x += __shfl_xor_sync(0xffffffffu, y.x, m), y.y += __shfl_xor_sync(0xffffffffu, y.y, m);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, m), y.w += __shfl_xor_sync(0xffffffffu, y.w, m);
        }
        if (lane < kLanes) red[warp][0][col] = x, red[warp][1][col] = y;
        __syncthreads();
        float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kDrThreads / 32; ++w) {
            const float4 e = red[w][0][col], f = red[w][1][col];
            sk[0] += e.x, sk[1] += e.y, sk[2] += e.z, sk[3] += e.w;
            sq[0] += f.x, sq[1] += f.y, sq[2] += f.z, sq[3] += f.w;
        }
        float u[4], o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] = beta * (v[j] - decay * rk * sk[j]);
            o[j] = rq * (decay * sq[j] + rk * kq * u[j]);
        }
        if (r0 == 0) {
            const uint2 w = make_uint2(dr_pack<DT>(o[0], o[1]), dr_pack<DT>(o[2], o[3]));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + ((long long)t * a.Hv + hv) * a.dv + c0) = w;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float k = ks[p][r0 + i * kRows] * rk;
            S[i].x = decay * S[i].x + k * u[0], S[i].y = decay * S[i].y + k * u[1];
            S[i].z = decay * S[i].z + k * u[2], S[i].w = decay * S[i].w + k * u[3];
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) *reinterpret_cast<float4*>(sp + (long long)i * kRows * a.dv) = S[i];
}

// ---- chunks of 32 tokens ------------------------------------------------------
// With G_i = g_1 + ... + g_i inside a chunk and S0 the state before it,
//   (1 + L) U = diag(beta) (V - diag(e^G) K S0),  L_ij = beta_i e^(G_i - G_j) k_i . k_j (j < i)
//   O = diag(e^G) Q S0 + P U,  P_ij = e^(G_i - G_j) q_i . k_j (j <= i)
//   S = e^(G_32) S0 + sum_j e^(G_32 - G_j) k_j u_j^T
// A first kernel makes what does not hang on the state, for all chunks at once:
// T = (1 + L)^-1 diag(beta), P and the factors. The second walks each
// sequence's chunks; its products run on the tensor cores.
//
// Precision: states stay as good as f32 makes them. Keys and queries are fp16
// values (bf16 ones times a power of two a row: exact, but for values below
// 2^-17 of the row's largest, which are 2^-25 of it off at most). Everything
// else enters a product as two fp16 parts of its value times a power of two a
// row (the largest of the row at 2^13): 22 bits and more of the row's largest.
// Sums are f32. What is 2^-38 of a row's largest is lost, and rows of the state
// and of V - ... whose largest is below 2^-60 have fewer bits.
constexpr int kC = 32;  // tokens of a chunk

// What the first kernel leaves for one (chunk, value head).
struct DrChunk {
    uint16_t t_hi[kC][kC], t_lo[kC][kC];  // fp16, row i times 1 / t_inv[i]
    uint16_t p_hi[kC][kC], p_lo[kC][kC];  // fp16, row i times 1 / p_inv[i]; scale and norms in it
    float fall[kC];                       // e^G_j / |k_j|
    float rest[kC];                       // e^(G_32 - G_j) / |k_j|
    float t_inv[kC], p_inv[kC];
    float q_out[kC];  // scale e^G_i / |q_i|
    float decay[kC];  // e^G_32 (all the same)
};
static_assert(sizeof(DrChunk) % 128 == 0, "rows of 16 bytes");

__device__ __forceinline__ void dr_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void dr_ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void dr_ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t dr_movm(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void dr_cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// 2^k that takes values of at most `most` below 2^14 (the largest to 2^13 and more, where k stays in -114..60).
__device__ __forceinline__ float dr_scale(float most) {
    const int k = min(60, max(-114, 140 - static_cast<int>(__float_as_uint(most) >> 23)));
    return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}
// 1 / p of a power of two in 2^-126..2^126
__device__ __forceinline__ float dr_inv(float p) { return __uint_as_float(0x7F000000u - __float_as_uint(p)); }
// The power of two, within 2^-100..2^114, that r is 2^8 and more times
__device__ __forceinline__ float dr_unit(float r) {
    return __uint_as_float(static_cast<uint32_t>(min(241, max(27, static_cast<int>(__float_as_uint(r) >> 23) - 8))) << 23);
}
// x and y as two fp16 parts each: the second is x less the first, by sums of mixed types
__device__ __forceinline__ void dr_split(float x, float y, uint32_t& hi, uint32_t& lo) {
    asm("{\n\t.reg .b16 a, b, m;\n\t.reg .f32 p, q;\n\t"
        "cvt.rn.f16x2.f32 %0, %3, %2;\n\t"
        "mov.b32 {a, b}, %0;\n\t"
        "mov.b16 m, 0xBC00;\n\t"  // -1
        "fma.rn.f32.f16 p, a, m, %2;\n\t"
        "fma.rn.f32.f16 q, b, m, %3;\n\t"
        "cvt.rn.f16x2.f32 %1, q, p;\n\t}"
        : "=&r"(hi), "=r"(lo)
        : "f"(x), "f"(y));
}
__device__ __forceinline__ uint32_t dr_first(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// e^x of a decay, to 2^-22 of it (and x 2^-24)
__device__ __forceinline__ float dr_exp(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
// Place of 16-byte chunk c of row r: rows of 128 bytes and more, or of 64.
template <int kRowBytes>
__device__ __forceinline__ uint32_t dr_at(int r, int c) {
    return r * kRowBytes + ((kRowBytes >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// The chunk data of sequence s begin at slot t0 / kC + s: no two sequences share one.
__host__ __device__ inline long long dr_slots(int T, int n) { return T / kC + static_cast<long long>(n); }

// One CTA of two warps a (chunk, key head): norms, k . k and q . k on the tensor
// cores, then a warp a value head. L and P go row by lane, so that a row's
// largest value and its 16-byte stores are a lane's own; the solve for T goes
// column by lane, its rows of L broadcast from shared memory. Bound: latency of
// that chain of some 1600 instructions a head, hidden by eight CTAs a
// multiprocessor.
template <int DT, int DK>
__global__ void __launch_bounds__(64, 8) delta_prepare_kernel(DeltaArgs a, uint16_t* kf, uint16_t* qf, DrChunk* out) {
    constexpr int kRow = DK * 2, kVec = DK / 16;  // 16-byte pieces of half a row
    constexpr int kDots = 2 * kC * (kC + 4) * 4;
    __shared__ __align__(128) unsigned char kq[2 * kC * kRow > kDots ? 2 * kC * kRow : kDots];  // keys, queries; then their products
    unsigned char *ks = kq, *qs = kq + kC * kRow;
    auto dots = reinterpret_cast<float(*)[kC][kC + 4]>(kq);  // k_i . k_j and q_i . k_j
    __shared__ float inv[2][kC];           // 1 / |k|, 1 / |q| (with the rows' powers of two)
    __shared__ float4 col[2][kC];          // by warp, of token j: its sum of decays (two parts), 1 / |k_j|
    __shared__ __align__(16) float Ls[2][kC][kC + 4];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hk = blockIdx.y;
    // the sequence of this slot: the last whose first slot is not behind it
    int s = 0;
    for (int lo = 0, hi = a.n - 1; lo <= hi;) {
        const int mid = (lo + hi) >> 1;
        if (max(0, min(a.at[mid], a.T)) / kC + static_cast<long long>(mid) <= blockIdx.x)
            s = mid, lo = mid + 1;
        else
            hi = mid - 1;
    }
    int t0, t1;
    dr_tokens(a, s, t0, t1);
    const long long ahead = blockIdx.x - (t0 / kC + static_cast<long long>(s));
    if (ahead < 0 || ahead * kC >= t1 - t0) return;  // a slot that no sequence uses
    t0 += static_cast<int>(ahead) * kC;
    const int n = min(kC, t1 - t0);
    {
        // two threads a row: norms, and for bf16 the power of two that brings the row's largest value to 1..2
        const int r = tid >> 1, part = tid & 1;
        uint4 w[2][kVec];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint16_t* src = static_cast<const uint16_t*>(which ? a.q : a.k) + ((long long)(t0 + r) * a.Hk + hk) * DK + part * (DK / 2);
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[which][i] = r < n ? *reinterpret_cast<const uint4*>(src + i * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float sum0 = 0.f, sum1 = 0.f, most = 0.f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const uint32_t v[4] = {w[which][i].x, w[which][i].y, w[which][i].z, w[which][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 x;
                    if (DT == 1)
                        x = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
                    else
                        x = make_float2(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xFFFF0000u));
                    sum0 += x.x * x.x;
                    sum1 += x.y * x.y;
                    if (DT == 2) most = fmaxf(most, fmaxf(fabsf(x.x), fabsf(x.y)));
                }
            }
            float sum = sum0 + sum1;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            float up = 1.f;
            if (DT == 2) {
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                up = dr_scale(most) * 0x1p-13f;
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    uint32_t v[4] = {w[which][i].x, w[which][i].y, w[which][i].z, w[which][i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = dr_first(__uint_as_float(v[j] << 16) * up, __uint_as_float(v[j] & 0xFFFF0000u) * up);
                    w[which][i] = make_uint4(v[0], v[1], v[2], v[3]);
                    if (r < n)
                        *reinterpret_cast<uint4*>((which ? qf : kf) + ((long long)(t0 + r) * a.Hk + hk) * DK + part * (DK / 2) + i * 8) = w[which][i];
                }
            }
            if (part == 0) inv[which][r] = r >= n ? 0.f : (a.eps >= 0.f ? 1.f / sqrtf(sum + a.eps) : 1.f) / up;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                *reinterpret_cast<uint4*>((which ? qs : ks) + dr_at<kRow>(r, part * kVec + i)) = w[which][i];
        }
    }
    __syncthreads();
    {
        // warp 0: k . k, warp 1: q . k
        const uint32_t A = static_cast<uint32_t>(__cvta_generic_to_shared(warp == 0 ? ks : qs));
        const uint32_t B = static_cast<uint32_t>(__cvta_generic_to_shared(ks));
        float c[2][4][4] = {};
#pragma unroll
        for (int k = 0; k < DK / 16; k += 2) {
            uint32_t b[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) dr_ldsm4(b[i], B + dr_at<kRow>(8 * i + (lane & 7), 2 * k + (lane >> 3)));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t f[4];
                    dr_ldsm4(f, A + dr_at<kRow>(16 * m + (lane & 15), 2 * (k + h) + (lane >> 4)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) dr_mma(c[m][i], f, b[i][2 * h], b[i][2 * h + 1]);
                }
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) dots[warp][16 * m + (lane >> 2) + (e >> 1) * 8][8 * i + (lane & 3) * 2 + (e & 1)] = c[m][i][e];
    }
    __syncthreads();
    const int rep = a.Hv / a.Hk;
    for (int r = warp; r < rep; r += 2) {
        const int hv = hk * rep + r;
        DrChunk* o = out + (long long)blockIdx.x * a.Hv + hv;
        const long long at = (long long)(t0 + lane) * a.Hv + hv;
        float gl = lane < n ? a.g[at] : 0.f;
        const float beta = lane < n ? a.beta[at] : 0.f;
        gl = gl < -1e6f ? -1e6f : gl;  // -infinity has no differences; e^-1e6 is 0 as well
        double G = gl;                 // sums of decays in 64 bits: their differences count
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double p = __shfl_up_sync(0xffffffffu, G, m);
            if (lane >= m) G += p;
        }
        const float g_hi = static_cast<float>(G), g_lo = static_cast<float>(G - g_hi);
        const float all_hi = __shfl_sync(0xffffffffu, g_hi, 31), all_lo = __shfl_sync(0xffffffffu, g_lo, 31);
        const float rk = inv[0][lane], rq = a.scale * inv[1][lane];
        float(&L)[kC][kC + 4] = Ls[warp];
        __syncwarp();
        col[warp][lane] = make_float4(g_hi, g_lo, rk, 0.f);
        __syncwarp();
        // rows of two matrices -> two fp16 parts of each value times `up`, 16 bytes at a time
        auto store = [&](uint16_t(&hi)[kC][kC], uint16_t(&lo)[kC][kC], const float(&v)[kC], float up) {
#pragma unroll
            for (int j = 0; j < kC; j += 8) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) dr_split(v[j + 2 * e] * up, v[j + 2 * e + 1] * up, h[e], l[e]);
                *reinterpret_cast<uint4*>(&hi[lane][j]) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(&lo[lane][j]) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        };
        {
            // row `lane` of L and of P
            float p[kC], most = 0.f;
            const float bk = beta * rk;
#pragma unroll
            for (int j = 0; j < kC; j += 4) {
                float l[4];
                const float4 kk = *reinterpret_cast<const float4*>(&dots[0][lane][j]), qk = *reinterpret_cast<const float4*>(&dots[1][lane][j]);
                const float kk4[4] = {kk.x, kk.y, kk.z, kk.w}, qk4[4] = {qk.x, qk.y, qk.z, qk.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 c = col[warp][j + e];
                    const float d = (g_hi - c.x) + (g_lo - c.y);
                    const float f = j + e <= lane ? dr_exp(d) * c.z : 0.f;
                    l[e] = j + e < lane ? bk * f * kk4[e] : 0.f;
                    p[j + e] = j + e <= lane ? rq * f * qk4[e] : 0.f;
                    most = fmaxf(most, fabsf(p[j + e]));
                }
                *reinterpret_cast<float4*>(&L[lane][j]) = make_float4(l[0], l[1], l[2], l[3]);
            }
            const float up = dr_scale(most);
            store(o->p_hi, o->p_lo, p, up);
            o->p_inv[lane] = dr_inv(up);
        }
        __syncwarp();
        // column `lane` of (1 + L)^-1, row by row
        float x[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float acc[4] = {lane == i ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < i; j += 4) {
                const float4 l = *reinterpret_cast<const float4*>(&L[i][j]);
                acc[0] -= l.x * x[j];
                if (j + 1 < i) acc[1] -= l.y * x[j + 1];
                if (j + 2 < i) acc[2] -= l.z * x[j + 2];
                if (j + 3 < i) acc[3] -= l.w * x[j + 3];
            }
            x[i] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kC; ++i) L[i][lane] = x[i] * beta;
        __syncwarp();
        {
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < kC; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(&L[lane][j]);
                x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
                most = fmaxf(fmaxf(most, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
            }
            const float up = dr_scale(most);
            store(o->t_hi, o->t_lo, x, up);
            o->t_inv[lane] = dr_inv(up);
        }
        const float eg = expf(g_hi + g_lo);
        o->fall[lane] = eg * rk;
        o->rest[lane] = expf((all_hi - g_hi) + (all_lo - g_lo)) * rk;
        o->q_out[lane] = rq * eg;
        o->decay[lane] = expf(all_hi + all_lo);
    }
}

// the same by sums of f32 pairs
__device__ __forceinline__ void dr_split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 b = __half22float2(h);
    unsigned long long xy, nb, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(xy) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(nb) : "f"(-b.x), "f"(-b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(xy), "l"(nb));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = dr_first(x, y);
}
__device__ __forceinline__ unsigned long long dr_pair(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void dr_unpair(unsigned long long xy, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(xy));
}
__device__ __forceinline__ unsigned long long dr_mul2(unsigned long long x, float f) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(dr_pair(f, f)));
    return r;
}

// Walks the chunks of one (sequence, value head, 16 W columns of the state).
// A state warp owns 16 columns, held transposed ([16 columns][dk]) in the tensor
// cores' accumulator layout for the whole walk. In that form each product's
// result is the next one's left operand, register for register: S^T K^T, then
// (V - ...)^T T^T, then U^T K. Nothing of that chain passes through shared
// memory. It hands the operand S^T and U^T to an output warp, which makes
// S^T Q^T + U^T P^T one chunk later; cp.async fetches the next chunks; all warps
// meet once a chunk. The chain bounds a long sequence: at 128 x 128 states a
// chunk takes 1.15 us, some 2400 cycles, of which 152 tensor instructions of 8
// cycles are half: K S 900, the new state 640, V - ... 320, T 210, U's factors
// 300, the meeting 120. The tensor pipes are 39% busy over the multiprocessor.
// Measured and slower: all of it in one warp (2.8 us a chunk); the key
// dimensions halved between two warps, which then meet once more (1.4); 8
// columns a warp as the right operand, which a transpose within the warp has to
// make (2.2); the next chunk's K S from the state before and U, so that only a
// product of 32 x 32 stays in the chain, beside warps that walk the state (1.24:
// those become the chain); S split for the next chunk between the products of
// this one (1.26: an instruction stream of one warp); a long sequence in parts,
// the chunk data of one made beside the walk of the one before (32000 tokens:
// 1512 us against 1420). tcgen05 takes 128 rows at least, all columns of a
// state, and its results would pass through tensor memory between the four
// products of the chain: throughput, which many sequences could use, but not a
// shorter chain.
template <int kThreads>
__device__ __forceinline__ void dr_meet() {  // all warps, each from its own loop
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}
template <int DK, int W>
struct DrWalk {
    static constexpr int kRow = DK * 2, kVRow = W * 32;
    static constexpr int kQ = kC * kRow, kV = 2 * kC * kRow, kD = kV + kC * kVRow;
    static constexpr int kStage = kD + static_cast<int>(sizeof(DrChunk));
    static constexpr int kStages = 4;
    // two warps of each kind: the loading ones share a scheduler with output ones, as two warps before them leave at
    // once. Four state and four output warps: the output warps load (more warps would take registers from all).
    static constexpr int kIdle = W == 2 ? 2 : 0, kLoad = W == 2 ? 2 : 0;
    static constexpr int kThreads = (2 * W + kIdle + kLoad) * 32, kMeet = (2 * W + kLoad) * 32;
    // handed over: S^T, two parts in operand registers; U^T in f32; the columns' factors of S
    static constexpr int kUAt = DK / 16 * 2 * 512, kFAt = kUAt + 4 * 512, kHand = kFAt + 256;
    static constexpr int kHands = kStages * kStage;
    static constexpr int kSmem = kHands + 2 * W * kHand;
};
template <int DT, int DK, int W>
__global__ void __launch_bounds__(DrWalk<DK, W>::kThreads) delta_walk_kernel(DeltaArgs a, const uint16_t* kf, const uint16_t* qf, const DrChunk* data) {
    using C = DrWalk<DK, W>;
    constexpr int kRow = C::kRow, kVRow = C::kVRow, kNt = DK / 8, kStages = C::kStages;
    constexpr int kLoaders = (C::kLoad ? C::kLoad : W) * 32;
    extern __shared__ __align__(1024) unsigned char smem[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warp = wid % W, g = lane >> 2, q4 = lane & 3;
    const int hv = blockIdx.y, hk = hv / (a.Hv / a.Hk), c0 = blockIdx.x * (16 * W);
    int seq = blockIdx.z, t0, t1;
    if (a.n > 1 && a.n <= 64) {
        // the longest sequences first: the first CTAs to run take them
        __shared__ int lens[64], mine;
        if (threadIdx.x < a.n) {
            dr_tokens(a, threadIdx.x, t0, t1);
            lens[threadIdx.x] = t1 - t0;
        }
        __syncthreads();
        if (threadIdx.x < a.n) {
            int before = 0;
            for (int i = 0; i < a.n; ++i) before += lens[i] > lens[threadIdx.x] || (lens[i] == lens[threadIdx.x] && i < threadIdx.x);
            if (before == blockIdx.z) mine = threadIdx.x;
        }
        __syncthreads();
        seq = mine;
    }
    dr_tokens(a, seq, t0, t1);
    const int chunks = (t1 - t0 + kC - 1) / kC;
    if (chunks == 0) return;
    data += (t0 / kC + static_cast<long long>(seq)) * a.Hv + hv;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    auto hand = [&](int c) { return smem + C::kHands + ((c & 1) * W + warp) * C::kHand; };
    auto quad_max = [](float x) {
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    };
    auto parts = [&](const float(&v)[4][4], const float(&up)[2], uint32_t(&hi)[2][4], uint32_t(&lo)[2][4]) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float* w = v[2 * k + (e >> 1)] + (e & 1) * 2;
                float x, y;
                dr_unpair(dr_mul2(dr_pair(w[0], w[1]), up[e & 1]), x, y);
                dr_split(x, y, hi[k][e], lo[k][e]);
            }
    };
    auto row_max = [&](const float(&v)[4][4], float(&m)[2]) {
        m[0] = m[1] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[0] = fmaxf(m[0], fmaxf(fabsf(v[i][0]), fabsf(v[i][1])));
            m[1] = fmaxf(m[1], fmaxf(fabsf(v[i][2]), fabsf(v[i][3])));
        }
        m[0] = quad_max(m[0]), m[1] = quad_max(m[1]);
    };

    // ---- loading
    const int tid = static_cast<int>(threadIdx.x) - (C::kLoad ? 2 * W + C::kIdle : W) * 32;  // of the loading threads
    auto load = [&](int c) {
        const uint32_t to = base + (c % kStages) * C::kStage;
        const int tc = t0 + c * kC, n = min(kC, t1 - tc);
        constexpr int kKc = DK / 8, kVc = W * 2, kStep = kLoaders / kKc, kVStep = kLoaders / kVc;
        {
            const int r0 = tid / kKc, ch = tid % kKc;
            const long long off = ((long long)tc * a.Hk + hk) * DK + ch * 8, step = (long long)a.Hk * DK;
#pragma unroll
            for (int m = 0; m < kC / kStep; ++m) {
                const int r = r0 + m * kStep;
                const long long at = off + (r < n ? r : 0) * step;
                dr_cp16(to + dr_at<kRow>(r, ch), kf + at, r < n);
                dr_cp16(to + C::kQ + dr_at<kRow>(r, ch), qf + at, r < n);
            }
        }
        {
            const int r0 = tid / kVc, ch = tid % kVc;
            const uint16_t* v = static_cast<const uint16_t*>(a.v) + ((long long)tc * a.Hv + hv) * a.dv + c0 + ch * 8;
#pragma unroll
            for (int m = 0; m < kC / kVStep; ++m) {
                const int r = r0 + m * kVStep;
                dr_cp16(to + C::kV + dr_at<kVRow>(r, ch), v + (long long)(r < n ? r : 0) * a.Hv * a.dv, r < n);
            }
        }
        const char* d = reinterpret_cast<const char*>(data + (long long)c * a.Hv) + tid * 16;
#pragma unroll
        for (int m = 0; m < 4 * kC * 4 / kLoaders; ++m) {  // four matrices of 32 rows of 64 bytes
            const int i = tid + m * kLoaders;
            dr_cp16(to + C::kD + (i >> 7) * (kC * 64) + dr_at<64>((i >> 2) & 31, i & 3), d + m * kLoaders * 16, true);
        }
        if (tid < static_cast<int>(sizeof(DrChunk)) / 16 - 4 * kC * 4) dr_cp16(to + C::kD + 4 * kC * 64 + tid * 16, d + 4 * kC * 64, true);
    };
    static_assert(static_cast<int>(sizeof(DrChunk)) / 16 - 4 * kC * 4 <= kLoaders, "the factors in one go");
    auto start = [&]() {
        load(0);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (chunks > 1) load(1);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // chunk `it` is there; the one after the next is on its way
    auto turn = [&](int it) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        dr_meet<C::kMeet>();
        if (it + 2 < chunks) load(it + 2);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (C::kLoad && wid >= 2 * W) {
        if (tid < 0) return;
        start();
        for (int it = 0; it <= chunks; ++it) turn(it);
        return;
    }

    // ---- outputs, one chunk behind
    if (wid >= W) {
        if (!C::kLoad) {
            start();
            turn(0);
        } else {
            dr_meet<C::kMeet>();
        }
        for (int c = 0; c < chunks; ++c) {
            if (!C::kLoad)
                turn(c + 1);
            else
                dr_meet<C::kMeet>();
            const uint32_t st = base + (c % kStages) * C::kStage;
            const DrChunk* cd = reinterpret_cast<const DrChunk*>(smem + (c % kStages) * C::kStage + C::kD);
            const uint4* in = reinterpret_cast<const uint4*>(hand(c)) + lane;
            const float2 f = *reinterpret_cast<const float2*>(hand(c) + C::kFAt + lane * 8);
            float o[4][4] = {}, y[4][4] = {};
#pragma unroll
            for (int k = 0; k < DK / 16; k += 2) {
                uint32_t p[2][2][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint4 w = in[(2 * k + h) * 32];
                    p[h >> 1][h & 1][0] = w.x, p[h >> 1][h & 1][1] = w.y, p[h >> 1][h & 1][2] = w.z, p[h >> 1][h & 1][3] = w.w;
                }
                uint32_t b[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) dr_ldsm4(b[i], st + C::kQ + dr_at<kRow>(8 * i + (lane & 7), 2 * k + (lane >> 3)));
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) dr_mma(o[i], p[h >> 1][h & 1], b[i][(h >> 1) * 2], b[i][(h >> 1) * 2 + 1]);
            }
            uint32_t hi[2][4], lo[2][4];
            float u[4][4], u_inv[2];
            {
                float most[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 w = in[C::kUAt / 16 + i * 32];
                    u[i][0] = __uint_as_float(w.x), u[i][1] = __uint_as_float(w.y), u[i][2] = __uint_as_float(w.z), u[i][3] = __uint_as_float(w.w);
                }
                row_max(u, most);
                const float up[2] = {dr_scale(most[0]), dr_scale(most[1])};
                parts(u, up, hi, lo);
                u_inv[0] = dr_inv(up[0]), u_inv[1] = dr_inv(up[1]);
            }
            uint32_t ph[4][4], pl[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dr_ldsm4(ph[i], st + C::kD + 2 * kC * 64 + dr_at<64>(8 * i + (lane & 7), lane >> 3));
                dr_ldsm4(pl[i], st + C::kD + 3 * kC * 64 + dr_at<64>(8 * i + (lane & 7), lane >> 3));
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // P is lower triangular: the tokens before 16 need its first half only
#pragma unroll
                for (int i = 2 * k; i < 4; ++i) dr_mma(y[i], hi[k], ph[i][2 * k], ph[i][2 * k + 1]);
#pragma unroll
                for (int i = 2 * k; i < 4; ++i) dr_mma(y[i], lo[k], ph[i][2 * k], ph[i][2 * k + 1]);
#pragma unroll
                for (int i = 2 * k; i < 4; ++i) dr_mma(y[i], hi[k], pl[i][2 * k], pl[i][2 * k + 1]);
            }
            const int tc = t0 + c * kC, n = min(kC, t1 - tc);
            uint16_t* to = static_cast<uint16_t*>(a.out) + ((long long)(tc + g) * a.Hv + hv) * a.dv + c0 + warp * 16 + 2 * q4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 fq = *reinterpret_cast<const float2*>(&cd->q_out[8 * i + 2 * q4]);
                const float2 fp = *reinterpret_cast<const float2*>(&cd->p_inv[8 * i + 2 * q4]);
                const float r0 = o[i][0] * f.x * fq.x + y[i][0] * u_inv[0] * fp.x, r1 = o[i][1] * f.x * fq.y + y[i][1] * u_inv[0] * fp.y;
                const float r2 = o[i][2] * f.y * fq.x + y[i][2] * u_inv[1] * fp.x, r3 = o[i][3] * f.y * fq.y + y[i][3] * u_inv[1] * fp.y;
                // [column][token] -> [token][column]
                const uint32_t w0 = dr_movm(dr_pack<DT>(r0, r1)), w1 = dr_movm(dr_pack<DT>(r2, r3));
                if (8 * i + g < n) {
                    uint16_t* at = to + (long long)(8 * i) * a.Hv * a.dv;
                    *reinterpret_cast<uint32_t*>(at) = w0;
                    *reinterpret_cast<uint32_t*>(at + 8) = w1;
                }
            }
        }
        return;
    }

    // ---- the state
    // element e of tile k: column c0 + 16 warp + g + 8 (e / 2), key dimension 8 k + 2 q4 + e % 2
    float S[kNt][4];
    float* sp = a.state + ((long long)seq * a.Hv + hv) * DK * a.dv + c0 + warp * 16 + g;
#pragma unroll
    for (int k = 0; k < kNt; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[k][e] = sp[(long long)(8 * k + 2 * q4 + (e & 1)) * a.dv + (e >> 1) * 8];
    float unit[2] = {1.f, 1.f};  // the state's columns are S unit; powers of two
    for (int c = 0; c < chunks; ++c) {
        dr_meet<C::kMeet>();
        const uint32_t st = base + (c % kStages) * C::kStage;
        const DrChunk* cd = reinterpret_cast<const DrChunk*>(smem + (c % kStages) * C::kStage + C::kD);  // its factors
        uint4* give = reinterpret_cast<uint4*>(hand(c)) + lane;
        // what the next steps need, on its way while the tensor cores work
        uint32_t v0[4], v1[4];
        float2 fall[4], rest[4], t_inv[4];
        dr_ldsm4t(v0, st + C::kV + dr_at<kVRow>(lane, 2 * warp));
        dr_ldsm4t(v1, st + C::kV + dr_at<kVRow>(lane, 2 * warp + 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fall[i] = *reinterpret_cast<const float2*>(&cd->fall[8 * i + 2 * q4]);
            rest[i] = *reinterpret_cast<const float2*>(&cd->rest[8 * i + 2 * q4]);
            t_inv[i] = *reinterpret_cast<const float2*>(&cd->t_inv[8 * i + 2 * q4]);
        }
        const float decay = cd->decay[0];
        float x[4][4], most[2];
        for (int pass = 0;; ++pass) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
            float xl[4][4] = {};
            __half2 big[2] = {__half2{}, __half2{}};
#pragma unroll
            for (int k = 0; k < DK / 16; k += 2) {
                uint32_t hi[2][4], lo[2][4], b[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) dr_ldsm4(b[i], st + dr_at<kRow>(8 * i + (lane & 7), 2 * k + (lane >> 3)));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float* v = S[2 * (k + h) + (e >> 1)] + (e & 1) * 2;
                        if (W == 4)
                            dr_split(v[0], v[1], hi[h][e], lo[h][e]);
                        else  // (the sums of mixed types hold the products up here: 101 us against 94 for 2048 tokens)
                            dr_split2(v[0], v[1], hi[h][e], lo[h][e]);
                        big[e & 1] = __hmax2(big[e & 1], __habs2(*reinterpret_cast<const __half2*>(&hi[h][e])));
                    }
                    give[2 * (k + h) * 32] = make_uint4(hi[h][0], hi[h][1], hi[h][2], hi[h][3]);
                    give[(2 * (k + h) + 1) * 32] = make_uint4(lo[h][0], lo[h][1], lo[h][2], lo[h][3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dr_mma(x[i], hi[h], b[i][2 * h], b[i][2 * h + 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dr_mma(xl[i], lo[h], b[i][2 * h], b[i][2 * h + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] += xl[i][e];
            most[0] = quad_max(fmaxf(__low2float(big[0]), __high2float(big[0])));
            most[1] = quad_max(fmaxf(__low2float(big[1]), __high2float(big[1])));
            // each column's largest has to lie in 1..2^15, where two fp16 parts hold every value to 2^-22 of it (and
            // nothing overflows); else the column changes its unit, once, and it is done again
            const bool out0 = !(most[0] >= 1.f && most[0] < 32768.f), out1 = !(most[1] >= 1.f && most[1] < 32768.f);
            if (pass == 1 || !__any_sync(0xffffffffu, out0 || out1)) break;
            float all[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kNt; ++k) {
                all[0] = fmaxf(all[0], fmaxf(fabsf(S[k][0]), fabsf(S[k][1])));
                all[1] = fmaxf(all[1], fmaxf(fabsf(S[k][2]), fabsf(S[k][3])));
            }
            all[0] = quad_max(all[0]), all[1] = quad_max(all[1]);
            const float f0 = !out0 || all[0] == 0.f ? 1.f : fminf(dr_scale(all[0]), unit[0] * 0x1p100f);
            const float f1 = !out1 || all[1] == 0.f ? 1.f : fminf(dr_scale(all[1]), unit[1] * 0x1p100f);
            // columns of zeros, and those at the end of the units' range, stay
            if (!__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) break;
#pragma unroll
            for (int k = 0; k < kNt; ++k) S[k][0] *= f0, S[k][1] *= f0, S[k][2] *= f1, S[k][3] *= f1;
            unit[0] *= dr_inv(f0), unit[1] *= dr_inv(f1);
        }
        // V - diag(e^G) K S0, transposed, and its two parts
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = fall[i];
            const float2 y0 = DT == 1 ? __half22float2(*reinterpret_cast<const __half2*>(&v0[i]))
                                      : make_float2(__uint_as_float(v0[i] << 16), __uint_as_float(v0[i] & 0xFFFF0000u));
            const float2 y1 = DT == 1 ? __half22float2(*reinterpret_cast<const __half2*>(&v1[i]))
                                      : make_float2(__uint_as_float(v1[i] << 16), __uint_as_float(v1[i] & 0xFFFF0000u));
            x[i][0] = y0.x - f.x * (x[i][0] * unit[0]), x[i][1] = y0.y - f.y * (x[i][1] * unit[0]);
            x[i][2] = y1.x - f.x * (x[i][2] * unit[1]), x[i][3] = y1.y - f.y * (x[i][3] * unit[1]);
        }
        uint32_t hi[2][4], lo[2][4], th[4][4], tl[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dr_ldsm4(th[i], st + C::kD + dr_at<64>(8 * i + (lane & 7), lane >> 3));
            dr_ldsm4(tl[i], st + C::kD + kC * 64 + dr_at<64>(8 * i + (lane & 7), lane >> 3));
        }
        float more[2];
        row_max(x, more);
        float up[2] = {dr_scale(more[0]), dr_scale(more[1])};
        parts(x, up, hi, lo);
        float u[4][4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // T is lower triangular
#pragma unroll
            for (int i = 2 * k; i < 4; ++i) dr_mma(u[i], hi[k], th[i][2 * k], th[i][2 * k + 1]);
#pragma unroll
            for (int i = 2 * k; i < 4; ++i) dr_mma(u[i], lo[k], th[i][2 * k], th[i][2 * k + 1]);
#pragma unroll
            for (int i = 2 * k; i < 4; ++i) dr_mma(u[i], hi[k], tl[i][2 * k], tl[i][2 * k + 1]);
        }
        float w[4][4];
        {
            const float v_inv[2] = {dr_inv(up[0]), dr_inv(up[1])};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = t_inv[i], r = rest[i];
                u[i][0] *= f.x * v_inv[0], u[i][1] *= f.y * v_inv[0];
                u[i][2] *= f.x * v_inv[1], u[i][3] *= f.y * v_inv[1];
                w[i][0] = u[i][0] * r.x, w[i][1] = u[i][1] * r.y, w[i][2] = u[i][2] * r.x, w[i][3] = u[i][3] * r.y;
            }
        }
        // the state after the chunk
        row_max(w, more);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            give[C::kUAt / 16 + i * 32] = make_uint4(__float_as_uint(u[i][0]), __float_as_uint(u[i][1]), __float_as_uint(u[i][2]), __float_as_uint(u[i][3]));
        *reinterpret_cast<float2*>(hand(c) + C::kFAt + lane * 8) = make_float2(unit[0], unit[1]);
        float keep[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // in the state's own unit, while what is left of it or what is added stays well inside that window (sizes
            // as they are, not in units: a quotient of far-apart ones would overflow)
            const float r = fmaxf(decay * most[h] * unit[h], more[h]);
            const float to = r == 0.f || (r >= 4.f * unit[h] && r < 2048.f * unit[h]) ? unit[h] : dr_unit(r);
            keep[h] = decay * unit[h] * dr_inv(to);
            unit[h] = to;
            up[h] = dr_inv(to);
        }
        parts(w, up, hi, lo);
#pragma unroll
        for (int k = 0; k < kNt; k += 8) {
            uint32_t b[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dr_ldsm4t(b[i], st + dr_at<kRow>(lane, k + i));
                dr_unpair(dr_mul2(dr_pair(S[k + i][0], S[k + i][1]), keep[0]), S[k + i][0], S[k + i][1]);
                dr_unpair(dr_mul2(dr_pair(S[k + i][2], S[k + i][3]), keep[1]), S[k + i][2], S[k + i][3]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) dr_mma(S[k + i], hi[0], b[i][0], b[i][1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) dr_mma(S[k + i], hi[1], b[i][2], b[i][3]);
#pragma unroll
            for (int i = 0; i < 8; ++i) dr_mma(S[k + i], lo[0], b[i][0], b[i][1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) dr_mma(S[k + i], lo[1], b[i][2], b[i][3]);
        }
    }
    dr_meet<C::kMeet>();  // the last chunk's hand-over
#pragma unroll
    for (int k = 0; k < kNt; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) sp[(long long)(8 * k + 2 * q4 + (e & 1)) * a.dv + (e >> 1) * 8] = S[k][e] * unit[e >> 1];
}

template <int DT, int DK>
cudaError_t launch_step(const DeltaArgs& a, cudaStream_t s) {
    // 128 columns a CTA where that still fills the GPU
    int vs = a.dv % 128 == 0 && (long long)a.n * a.Hv * (a.dv / 128) >= 2 * kSms ? 128 : a.dv % 64 == 0 && (long long)a.n * a.Hv * (a.dv / 64) >= 2 * kSms ? 64 : 32;
    const void* f = vs == 128 ? reinterpret_cast<const void*>(delta_step_kernel<DT, DK, 128>)
                    : vs == 64 ? reinterpret_cast<const void*>(delta_step_kernel<DT, DK, 64>)
                               : reinterpret_cast<const void*>(delta_step_kernel<DT, DK, 32>);
    void* args[] = {const_cast<DeltaArgs*>(&a)};
    return launch_kernel(f, dim3(a.dv / vs, a.Hv, a.n), dim3(kDrThreads), 0, true, s, args);
}

// Chunks from this length on; below, token by token. One sequence of 8 tokens, 32 heads of 128 x 128: 10.2 us by
// tokens, 12.3 in chunks; of 16: 18.2 and 12.3. 64 sequences of 8: 138 and 161; of 16: 243 and 164.
constexpr int kChunkFrom = 10;

struct DrPlan {
    bool chunks;
    size_t kf, qf, total;  // chunk data first; then, for bf16 alone, the keys and queries in fp16
};
DrPlan dr_plan(int dtype, int n, int T, int Hk, int Hv, int dk, int max_len) {
    DrPlan p{};
    p.chunks = max_len >= kChunkFrom;
    if (!p.chunks) return p;
    p.kf = static_cast<size_t>(dr_slots(T, n)) * Hv * sizeof(DrChunk);
    const size_t each = dtype == 1 ? 0 : static_cast<size_t>(T) * Hk * dk * 2;
    p.qf = p.kf + each;
    p.total = p.qf + each;
    return p;
}

template <int DT, int DK, int W>
cudaError_t launch_walk(const DeltaArgs& a, const uint16_t* kf, const uint16_t* qf, const DrChunk* data, cudaStream_t s) {
    const void* f = reinterpret_cast<const void*>(delta_walk_kernel<DT, DK, W>);
    constexpr int smem = DrWalk<DK, W>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    void* args[] = {const_cast<DeltaArgs*>(&a), &kf, &qf, &data};
    return launch_kernel(f, dim3(a.dv / (16 * W), a.Hv, a.n), dim3(DrWalk<DK, W>::kThreads), smem, true, s, args);
}

template <int DT, int DK>
cudaError_t launch_chunks(const DeltaArgs& a, char* ws, cudaStream_t s) {
    const DrPlan p = dr_plan(DT, a.n, a.T, a.Hk, a.Hv, a.dk, a.max_len);
    DrChunk* data = reinterpret_cast<DrChunk*>(ws);
    uint16_t* kf = reinterpret_cast<uint16_t*>(ws + p.kf);
    uint16_t* qf = reinterpret_cast<uint16_t*>(ws + p.qf);
    void* args[] = {const_cast<DeltaArgs*>(&a), &kf, &qf, &data};
    cudaError_t e = launch_kernel(reinterpret_cast<const void*>(delta_prepare_kernel<DT, DK>), dim3(dr_slots(a.T, a.n), a.Hk), dim3(64), 0,
                                  true, s, args);
    if (e != cudaSuccess) return e;
    const uint16_t* k = DT == 1 ? static_cast<const uint16_t*>(a.k) : kf;
    const uint16_t* q = DT == 1 ? static_cast<const uint16_t*>(a.q) : qf;
    // A multiprocessor holds one CTA of either width, and 64 columns take one and a half times as long as 32 (1024 tokens
    // of 32 heads of 128 x 128: 77 and 57 us; of 40 heads, two rounds of 32 columns: 79 and 94; three sequences of 32
    // heads, two rounds and three: 152 and 145; four: 159 and 190). 64 columns of dk = 128 need more than the 255 registers
    // of a thread: 80 bytes of it are spilled, which these figures have in them.
    const long long rounds2 = ((long long)a.n * a.Hv * (a.dv / 32) + kSms - 1) / kSms;
    const long long rounds4 = ((long long)a.n * a.Hv * (a.dv / 64) + kSms - 1) / kSms;
    if (a.dv % 64 == 0 && 3 * rounds4 < 2 * rounds2) return launch_walk<DT, DK, 4>(a, k, q, data, s);
    return launch_walk<DT, DK, 2>(a, k, q, data, s);
}

template <int DT>
cudaError_t launch_dt(const DeltaArgs& a, char* ws, cudaStream_t s) {
    if (a.max_len >= kChunkFrom) return a.dk == 64 ? launch_chunks<DT, 64>(a, ws, s) : launch_chunks<DT, 128>(a, ws, s);
    return a.dk == 64 ? launch_step<DT, 64>(a, s) : launch_step<DT, 128>(a, s);
}

}  // namespace

size_t delta_rule_ws_bytes(int dtype, int n, int T, int Hk, int Hv, int dk, int dv, int max_len) {
    (void)dv;
    return dr_plan(dtype, n, T, Hk, Hv, dk, max_len).total;
}

cudaError_t launch_delta_rule(const DeltaArgs& a, int dtype, void* ws, cudaStream_t s) {
    return dtype == 1 ? launch_dt<1>(a, static_cast<char*>(ws), s) : launch_dt<2>(a, static_cast<char*>(ws), s);
}

}  // namespace escha
