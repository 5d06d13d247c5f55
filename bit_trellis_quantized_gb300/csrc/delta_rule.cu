// Gated delta rule: per sequence and value head a state S [dk][dv] in f32 that
// each token decays, corrects along its key and reads along its query:
//   S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q,
// k and q divided by sqrt(sum x^2 + eps) first where eps >= 0.
//
// Token by token: a CTA holds [dk][VS] of one state in registers. Both products
// with the old state, S^T k and S^T q, come from one pass over it and one
// reduction, as o = scale (e^g S^T q + (k . q) u). Bound, for one token a
// sequence: the state's read and write.
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

}  // namespace

size_t delta_rule_ws_bytes(int n, int T, int Hk, int Hv, int dk, int dv, int max_len) {
    (void)n, (void)T, (void)Hk, (void)Hv, (void)dk, (void)dv, (void)max_len;
    return 0;
}

cudaError_t launch_delta_rule(const DeltaArgs& a, int dtype, void* ws, cudaStream_t s) {
    (void)ws;
    if (dtype == 1) return a.dk == 64 ? launch_step<1, 64>(a, s) : launch_step<1, 128>(a, s);
    return a.dk == 64 ? launch_step<2, 64>(a, s) : launch_step<2, 128>(a, s);
}

}  // namespace escha
