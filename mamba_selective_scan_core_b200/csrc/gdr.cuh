// The gated delta rule: the Mamba-2 form's state with a decay per head, whose
// update first takes out what the state already answers for the token's key.
// Per sequence and value head h (key head g = h / (H / G)), state S [P][N]:
//
//     a_t = exp(Delta_t A[h]),  Delta_t = softplus(dt_t[h] + dt_bias[h]);   b_t = sigmoid(beta_t[h])
//     S_t = a_t S_{t-1} + b_t (v_t - a_t S_{t-1} k_t) k_t^T                 (v_t: P, k_t: N)
//     y_t = scale S_t q_t
//
// with q_t and k_t divided by sqrt(sum of squares + eps) when the call
// normalises them.
//
// gdr_recurrent_kernel runs that as it stands, token by token: the one-token
// step (decode), short calls and fp32 activations.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "mixer_common.cuh"
#include "proj_gemm.cuh"
#include "ssd.cuh"

namespace mm {

struct GdrParams {
    const void* q;               // [B][L] rows of [G][N], q_stride elements between tokens (act)
    const void* k;               // [B][L] rows of [G][N], k_stride
    const void* v;               // [B][L] rows of [H][P], v_stride
    const void* dt;              // [B][L][H] act
    const void* beta;            // [B][L][H] act
    const float* dt_bias;        // [H] or null
    const float* A;              // [H]
    const float* h0;             // [B][H][P][N] or null (may be h_last: in place)
    void* y;                     // [B][L][H][P] act
    float* h_last;               // [B][H][P][N]
    int64_t L, q_stride, k_stride, v_stride;
    int H, G, P;
    float scale, eps;            // eps > 0: q and k are normalised
    unsigned long long* status;  // [0] (epoch << 8) | code of a failure, [1] the call's epoch; or null
    unsigned long long status_epoch;
};

// four consecutive activations as fp32
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// ---------------------------------------------------------------- token by token
// State rows stay in registers for the whole call.  Eight lanes hold a row,
// lane e its entries 4e + 32m + (0..3), so a warp's load of four rows is whole
// 128-byte lines; a warp holds 4 RPT rows, a CTA of four warps 16 RPT.  Both
// row sums of a token are taken of the state before it,
//     S_t q = a (S_{t-1} q) + b (v - a S_{t-1} k) (k . q),
// so they are reduced together (three shuffles over the eight lanes) and the
// update of the state is off the path from one sum to the next.
constexpr int kGdrRecThreads = 128;

template <typename T, int N, int RPT>
__global__ void __launch_bounds__(kGdrRecThreads)
gdr_recurrent_kernel(const GdrParams p)
{
    constexpr int M = N / 32;                     // float4s of a row per lane
    constexpr int kRows = kGdrRecThreads / 8 * RPT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = lane & 7, sub = lane >> 3;
    const int tiles = p.P / kRows;
    const int h = blockIdx.x / tiles, b = blockIdx.y;
    const int g = h / (p.H / p.G);
    const int row0 = (blockIdx.x - h * tiles) * kRows + warp * 4 * RPT + sub;   // row r of this lane: row0 + 4 r
    if (p.status && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) p.status[1] = p.status_epoch;

    const int64_t srow = (static_cast<int64_t>(b) * p.H + h) * p.P + row0;
    float4 s[RPT][M];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m)
            s[r][m] = p.h0 ? *reinterpret_cast<const float4*>(p.h0 + (srow + 4 * r) * N + 4 * e + 32 * m)
                           : make_float4(0.f, 0.f, 0.f, 0.f);

    const float bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
    const float A = p.A[h];
    const int64_t t_first = static_cast<int64_t>(b) * p.L;
    const T* kp = static_cast<const T*>(p.k) + t_first * p.k_stride + g * N + 4 * e;
    const T* qp = static_cast<const T*>(p.q) + t_first * p.q_stride + g * N + 4 * e;
    const T* vp = static_cast<const T*>(p.v) + t_first * p.v_stride + static_cast<int64_t>(h) * p.P + row0;
    const T* dtp = static_cast<const T*>(p.dt) + t_first * p.H + h;
    const T* bp = static_cast<const T*>(p.beta) + t_first * p.H + h;
    T* yp = static_cast<T*>(p.y) + (t_first * p.H + h) * p.P + row0;

    // the next token's inputs are loaded while the current one is worked on
    float4 kn[M], qn[M];
    float vn[RPT], dtn = 0.0f, bn = 0.0f;
    auto fetch = [&]() {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            kn[m] = load4(kp + 32 * m);
            qn[m] = load4(qp + 32 * m);
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r) vn[r] = Act<T>::load(vp + 4 * r);
        dtn = Act<T>::load(dtp);
        bn = Act<T>::load(bp);
        kp += p.k_stride;
        qp += p.q_stride;
        vp += p.v_stride;
        dtp += p.H;
        bp += p.H;
    };
    if (p.L > 0) fetch();
    for (int64_t t = 0; t < p.L; ++t) {
        float4 k[M], q[M];
        float v[RPT];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            k[m] = kn[m];
            q[m] = qn[m];
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r) v[r] = vn[r];
        const float a = expf(MathExact::step(dtn, bias) * A);
        const float bt = 1.0f / (1.0f + expf(-bn));
        if (t + 1 < p.L) fetch();

        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            kk = dot4(k[m], k[m], kk);
            qq = dot4(q[m], q[m], qq);
            kq = dot4(k[m], q[m], kq);
        }
        float ks[RPT], qs[RPT];
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            ks[r] = qs[r] = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                ks[r] = dot4(s[r][m], k[m], ks[r]);
                qs[r] = dot4(s[r][m], q[m], qs[r]);
            }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            kk += __shfl_xor_sync(kFull, kk, o);
            qq += __shfl_xor_sync(kFull, qq, o);
            kq += __shfl_xor_sync(kFull, kq, o);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                ks[r] += __shfl_xor_sync(kFull, ks[r], o);
                qs[r] += __shfl_xor_sync(kFull, qs[r], o);
            }
        }
        // the norms' factors go into the sums and the update instead of k and q
        const float rk = p.eps > 0.0f ? rsqrtf(kk + p.eps) : 1.0f;
        const float rq = (p.eps > 0.0f ? rsqrtf(qq + p.eps) : 1.0f) * p.scale;
        const float rkq = kq * rk * rq;
        float yv = 0.0f;      // lane e < RPT: row e's output
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const float u = bt * (v[r] - a * (ks[r] * rk));
            const float out = fmaf(a * rq, qs[r], u * rkq);
            if (e == r) yv = out;
            const float uk = u * rk;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                s[r][m].x = fmaf(a, s[r][m].x, uk * k[m].x);
                s[r][m].y = fmaf(a, s[r][m].y, uk * k[m].y);
                s[r][m].z = fmaf(a, s[r][m].z, uk * k[m].z);
                s[r][m].w = fmaf(a, s[r][m].w, uk * k[m].w);
            }
        }
        if (e < RPT) yp[4 * e] = Act<T>::from_f32(yv);
        yp += static_cast<int64_t>(p.H) * p.P;
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m)
            *reinterpret_cast<float4*>(p.h_last + (srow + 4 * r) * N + 4 * e + 32 * m) = s[r][m];
}

}  // namespace mm
