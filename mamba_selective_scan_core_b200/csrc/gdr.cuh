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
// gdr_recurrent_kernel runs that as it stands for one token (decode),
// gdr_tokens_kernel four tokens at a time: short calls and fp32 activations.
// gdr_prep_kernel and gdr_scan_kernel run longer bf16 calls in chunks of 64
// tokens on the tensor cores.
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
    unsigned wait_limit;
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

// One contiguous bulk copy global -> shared (16-byte aligned, a multiple of 16
// bytes), completion on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* gsrc, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n"
                 :: "r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}

// ---------------------------------------------------------------- one token
// Eight lanes hold a state row, lane e its entries 4e + 32m + (0..3), so a
// warp's load of four rows is whole 128-byte lines; a warp holds 4 RPT rows, a
// CTA of four warps 16 RPT.  Both row sums of the token are taken of the state
// before it,
//     S_t q = a (S_{t-1} q) + b (v - a S_{t-1} k) (k . q),
// so they are reduced together (three shuffles over the eight lanes).  No token
// (seqlen 0) copies the state.
//
// The state's traffic bounds it, for few rows a launch's latency: 128 sequences
// of 64 heads (128 x 128) 159 us in bf16, 6.8 TB/s.  At N = 128 the compiler
// gets the registers of three CTAs an SM: in those of four it has fewer of a
// lane's loads in flight (166 us).
constexpr int kGdrRecThreads = 128;

template <typename T, int N, int RPT>
__global__ void __launch_bounds__(kGdrRecThreads, N == 128 ? 3 : 1)
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
    if (p.L > 0) {
        const T* kp = static_cast<const T*>(p.k) + b * p.k_stride + g * N + 4 * e;
        const T* qp = static_cast<const T*>(p.q) + b * p.q_stride + g * N + 4 * e;
        const T* vp = static_cast<const T*>(p.v) + b * p.v_stride + static_cast<int64_t>(h) * p.P + row0;
        const int64_t gate = static_cast<int64_t>(b) * p.H + h;
        float4 k[M], q[M];
        float v[RPT];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            k[m] = load4(kp + 32 * m);
            q[m] = load4(qp + 32 * m);
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r) v[r] = Act<T>::load(vp + 4 * r);
        const float dtn = Act<T>::load(static_cast<const T*>(p.dt) + gate), bn = Act<T>::load(static_cast<const T*>(p.beta) + gate);

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
        const float a = expf(MathExact::step(dtn, bias) * A);
        const float bt = 1.0f / (1.0f + expf(-bn));
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
        if (e < RPT) static_cast<T*>(p.y)[srow + 4 * e] = Act<T>::from_f32(yv);
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m)
            *reinterpret_cast<float4*>(p.h_last + (srow + 4 * r) * N + 4 * e + 32 * m) = s[r][m];
}

// ---------------------------------------------------------------- a few tokens at a time
// The same for calls of several tokens, the state in the same lanes' registers
// for the whole call.  What bounds those is the path from
// one token's sums over the state to the next one's, so four tokens share it:
// with c_i the product of the group's decays up to token i and D_ij that of
// those after j,
//
//     u_i = b_i (v_i - c_i S k_i - sum_{j<i} D_ij (k_i . k_j) u_j)
//     y_i = scale (c_i S q_i + sum_{j<=i} D_ij (q_i . k_j) u_j)
//     S  <- c_3 S + sum_j D_3j u_j k_j^T
//
// needs S once for all eight sums and once for the update.  The coefficients
// are the same for every row: two helper warps, one for each group of a block
// of 8 tokens, work them out a block ahead and keep k, q and v (three tensor
// copies a block; a copy a row takes 90 cycles each to issue) two blocks ahead,
// beside the four warps that hold the state.  All in fp32.  2 x 200 fp32 tokens
// of 16 heads (128 x 64): 90 us with the next token's loads in registers, 68
// a token at a time with a ring that all warps fill, 40 this way, 34 with two
// rows a lane.
constexpr int kGdrBlock = 8;          // tokens of a ring slot: two groups
constexpr int kGdrGroup = 4;
constexpr int kGdrTokThreads = kGdrRecThreads + 64;
template <typename T, int N, int RPT>
struct GdrTokensLayout {
    static constexpr int rows = kGdrRecThreads / 8 * RPT;
    static constexpr int k_off = 0, q_off = k_off + kGdrBlock * N * sizeof(T), v_off = q_off + kGdrBlock * N * sizeof(T);
    static constexpr int stage_bytes = v_off + kGdrBlock * rows * sizeof(T);
    static constexpr int stages = 3;
    static_assert(q_off % 128 == 0 && v_off % 128 == 0 && stage_bytes % 128 == 0, "copies start on 128-byte boundaries");
};
// Of a group of four tokens, with the norms and the scale in them.
struct GdrGroup {
    float alpha[4];     // c_i, of S k_i
    float beta[4];      // scale c_i, of S q_i
    float b[4];         // b_i
    float w[4];         // D_3j, of u_j k_j
    float kk[4][4];     // D_ij (k_i . k_j), j < i; [0][0] is c_3
    float qk[4][4];     // scale D_ij (q_i . k_j), j <= i
};

template <typename T, int N, int RPT>
__global__ void __launch_bounds__(kGdrTokThreads)
gdr_tokens_kernel(const GdrParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v)
{
    using Lay = GdrTokensLayout<T, N, RPT>;
    constexpr int M = N / 32;
    constexpr int kRows = Lay::rows;
    __shared__ __align__(128) unsigned char ring[Lay::stages * Lay::stage_bytes];
    __shared__ __align__(16) GdrGroup coef[2][2];
    __shared__ uint64_t full[Lay::stages];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int e = lane & 7, sub = lane >> 3;
    const int tiles = p.P / kRows;
    const int h = blockIdx.x / tiles, b = blockIdx.y;
    const int g = h / (p.H / p.G);
    const int first = (blockIdx.x - h * tiles) * kRows;
    if (p.status && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) p.status[1] = p.status_epoch;

    const int64_t t_first = static_cast<int64_t>(b) * p.L;
    const int L = static_cast<int>(p.L), blocks = (L + kGdrBlock - 1) / kGdrBlock;
    if (tid == 0) {
        for (int i = 0; i < Lay::stages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto slot = [&](int blk) { return ring + blk % Lay::stages * Lay::stage_bytes; };

    if (warp >= kGdrRecThreads / 32) {
        const int half = warp - kGdrRecThreads / 32;
        // a block: one tensor copy each for k, q and v, zeros past the sequence
        auto request = [&](int blk) {
            if (blk >= blocks || tid != kGdrRecThreads) return;
            unsigned char* st = slot(blk);
            uint64_t* bar = &full[blk % Lay::stages];
            mbar_arrive_expect_tx(bar, Lay::stage_bytes);
            tma_load_3d(st + Lay::k_off, &tm_k, g * N, blk * kGdrBlock, b, bar);
            tma_load_3d(st + Lay::q_off, &tm_q, g * N, blk * kGdrBlock, b, bar);
            tma_load_3d(st + Lay::v_off, &tm_v, h * p.P + first, blk * kGdrBlock, b, bar);
        };
        auto landed = [&](int blk, unsigned limit) {
            return warp_wait(&full[blk % Lay::stages], static_cast<unsigned>((blk / Lay::stages) & 1), limit);
        };
        // lanes 0..3: dt and beta of the group's tokens
        const T* dtp = static_cast<const T*>(p.dt) + (t_first + half * kGdrGroup + lane) * p.H + h;
        const T* bp = static_cast<const T*>(p.beta) + (t_first + half * kGdrGroup + lane) * p.H + h;
        float dtn = 0.0f, bn = 0.0f;
        const float bias = p.dt_bias ? p.dt_bias[h] : 0.0f, A = p.A[h];
        auto fetch_gates = [&](int blk) {
            if (lane < kGdrGroup && blk * kGdrBlock + half * kGdrGroup + lane < L) {
                dtn = Act<T>::load(dtp + static_cast<int64_t>(blk) * kGdrBlock * p.H);
                bn = Act<T>::load(bp + static_cast<int64_t>(blk) * kGdrBlock * p.H);
            }
        };
        auto work_out = [&](int blk) {
            const unsigned char* st = slot(blk);
            const T* kb = reinterpret_cast<const T*>(st + Lay::k_off) + half * kGdrGroup * N + 4 * e;
            const T* qb = reinterpret_cast<const T*>(st + Lay::q_off) + half * kGdrGroup * N + 4 * e;
            float gate = 1.0f, strength = 0.0f;
            if (lane < kGdrGroup && blk * kGdrBlock + half * kGdrGroup + lane < L) {
                gate = expf(MathExact::step(dtn, bias) * A);
                strength = 1.0f / (1.0f + expf(-bn));
            }
            // column j = sub: eight lanes for k_i . k_j, q_i . k_j and q_i . q_i, i = 0..3
            float kk[4] = {}, qk[4] = {}, qq[4] = {};
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float4 kj = load4(kb + sub * N + 32 * m);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 ki = load4(kb + i * N + 32 * m), qi = load4(qb + i * N + 32 * m);
                    kk[i] = dot4(ki, kj, kk[i]);
                    qk[i] = dot4(qi, kj, qk[i]);
                    qq[i] = dot4(qi, qi, qq[i]);
                }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kk[i] += __shfl_xor_sync(kFull, kk[i], o);
                    qk[i] += __shfl_xor_sync(kFull, qk[i], o);
                    qq[i] += __shfl_xor_sync(kFull, qq[i], o);
                }
            // lane (j = sub, i = e) from here on; lanes e >= 4 repeat them
            const int i = e & 3, j = sub;
            const float kij = i == 0 ? kk[0] : i == 1 ? kk[1] : i == 2 ? kk[2] : kk[3];
            const float qij = i == 0 ? qk[0] : i == 1 ? qk[1] : i == 2 ? qk[2] : qk[3];
            const float qii = i == 0 ? qq[0] : i == 1 ? qq[1] : i == 2 ? qq[2] : qq[3];
            const float rq = (p.eps > 0.0f ? rsqrtf(qii + p.eps) : 1.0f) * p.scale;      // of token i
            const float rd = p.eps > 0.0f ? rsqrtf(kij + p.eps) : 1.0f;                  // the norm on the diagonal
            const float rki = __shfl_sync(kFull, rd, 9 * i), rkj = __shfl_sync(kFull, rd, 9 * j);
            float dij = 1.0f, ci = 1.0f, c3 = 1.0f;
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const float al = __shfl_sync(kFull, gate, l);
                dij *= l > j && l <= i ? al : 1.0f;
                ci *= l <= i ? al : 1.0f;
                c3 *= al;
            }
            const float bi = __shfl_sync(kFull, strength, i);
            GdrGroup& out = coef[blk & 1][half];
            if (e < 4) {
                out.kk[i][j] = i == 0 && j == 0 ? c3 : dij * (rki * rkj) * kij;
                out.qk[i][j] = dij * (rq * rkj) * qij;
                if (j == 0) {
                    out.alpha[i] = ci * rki;
                    out.beta[i] = ci * rq;
                    out.b[i] = bi;
                }
                if (i == 3) out.w[j] = dij * rkj;
            }
        };
        request(0);
        request(1);
        fetch_gates(0);
        bool ok = landed(0, p.wait_limit);
        int asked = min(2, blocks);       // blocks requested: no more once a wait has given up
        work_out(0);
        fetch_gates(1);
        for (int blk = 0; blk < blocks; ++blk) {
            if (ok && blk + 1 < blocks) ok = landed(blk + 1, p.wait_limit);
            __syncthreads();      // block blk + 1 is there, blk's coefficients are, blk - 1 is done with
            if (ok && blk + 2 < blocks) {
                request(blk + 2);
                asked = blk + 3;
            }
            if (blk + 1 < blocks) work_out(blk + 1);
            fetch_gates(blk + 2);
        }
        if (!ok) {
            // the copies in flight finish before their shared memory goes away
            if (warp == kGdrRecThreads / 32)
                for (int blk = max(0, asked - Lay::stages); blk < asked; ++blk) landed(blk, 1u << 20);
            if (lane == 0) {
                atomicOr(&g_mm_fault, 1u);
                if (p.status) atomicExch(p.status, (p.status_epoch << 8) | 1ull);
            }
        }
        return;
    }

    const int mine = warp * 4 * RPT + sub;   // row r of this lane: first + mine + 4 r
    const int64_t srow = (static_cast<int64_t>(b) * p.H + h) * p.P + first + mine;
    float4 s[RPT][M];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m)
            s[r][m] = p.h0 ? *reinterpret_cast<const float4*>(p.h0 + (srow + 4 * r) * N + 4 * e + 32 * m)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
    // lane e < 4 writes token e of a group
    const int64_t y_step = static_cast<int64_t>(p.H) * p.P;
    T* yp = static_cast<T*>(p.y) + (t_first * p.H + h) * p.P + first + mine + e * y_step;

    for (int blk = 0; blk < blocks; ++blk) {
        __syncthreads();
        const unsigned char* st = slot(blk);
        const T* kb = reinterpret_cast<const T*>(st + Lay::k_off) + 4 * e;
        const T* qb = reinterpret_cast<const T*>(st + Lay::q_off) + 4 * e;
        const T* vb = reinterpret_cast<const T*>(st + Lay::v_off) + mine;
#pragma unroll 1
        for (int t = 0; t < kGdrBlock; t += kGdrGroup) {
            const GdrGroup& c = coef[blk & 1][t / kGdrGroup];
            float ks[RPT][4], qs[RPT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int r = 0; r < RPT; ++r) ks[r][j] = qs[r][j] = 0.0f;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float4 k = load4(kb + (t + j) * N + 32 * m), q = load4(qb + (t + j) * N + 32 * m);
#pragma unroll
                    for (int r = 0; r < RPT; ++r) {
                        ks[r][j] = dot4(s[r][m], k, ks[r][j]);
                        qs[r][j] = dot4(s[r][m], q, qs[r][j]);
                    }
                }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < RPT; ++r) {
                        ks[r][j] += __shfl_xor_sync(kFull, ks[r][j], o);
                        qs[r][j] += __shfl_xor_sync(kFull, qs[r][j], o);
                    }
            const float4 al = load4(c.alpha), be = load4(c.beta), bt = load4(c.b), w = load4(c.w);
            const float4 k1 = load4(c.kk[1]), k2 = load4(c.kk[2]), k3 = load4(c.kk[3]);
            const float4 q1 = load4(c.qk[1]), q2 = load4(c.qk[2]), q3 = load4(c.qk[3]);
            const float q00 = c.qk[0][0], c3 = c.kk[0][0];
            float u[RPT][4], y[RPT];
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const T* vr = vb + t * kRows + 4 * r;
                u[r][0] = bt.x * fmaf(-al.x, ks[r][0], Act<T>::load(vr));
                u[r][1] = bt.y * fmaf(-k1.x, u[r][0], fmaf(-al.y, ks[r][1], Act<T>::load(vr + kRows)));
                u[r][2] = bt.z * fmaf(-k2.y, u[r][1], fmaf(-k2.x, u[r][0], fmaf(-al.z, ks[r][2], Act<T>::load(vr + 2 * kRows))));
                u[r][3] = bt.w * fmaf(-k3.z, u[r][2], fmaf(-k3.y, u[r][1], fmaf(-k3.x, u[r][0],
                                                                                fmaf(-al.w, ks[r][3], Act<T>::load(vr + 3 * kRows)))));
                const float y0 = fmaf(q00, u[r][0], be.x * qs[r][0]);
                const float y1 = fmaf(q1.y, u[r][1], fmaf(q1.x, u[r][0], be.y * qs[r][1]));
                const float y2 = fmaf(q2.z, u[r][2], fmaf(q2.y, u[r][1], fmaf(q2.x, u[r][0], be.z * qs[r][2])));
                const float y3 = fmaf(q3.w, u[r][3], fmaf(q3.z, u[r][2], fmaf(q3.y, u[r][1], fmaf(q3.x, u[r][0], be.w * qs[r][3]))));
                y[r] = e == 0 ? y0 : e == 1 ? y1 : e == 2 ? y2 : y3;
                u[r][0] *= w.x;
                u[r][1] *= w.y;
                u[r][2] *= w.z;
                u[r][3] *= w.w;
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    s[r][m].x *= c3;
                    s[r][m].y *= c3;
                    s[r][m].z *= c3;
                    s[r][m].w *= c3;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 k = load4(kb + (t + j) * N + 32 * m);
#pragma unroll
                    for (int r = 0; r < RPT; ++r) {
                        s[r][m].x = fmaf(u[r][j], k.x, s[r][m].x);
                        s[r][m].y = fmaf(u[r][j], k.y, s[r][m].y);
                        s[r][m].z = fmaf(u[r][j], k.z, s[r][m].z);
                        s[r][m].w = fmaf(u[r][j], k.w, s[r][m].w);
                    }
                }
            }
            const int at = blk * kGdrBlock + t;
            if (e < 4 && at + e < L)
#pragma unroll
                for (int r = 0; r < RPT; ++r) yp[at * y_step + 4 * r] = Act<T>::from_f32(y[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m)
            *reinterpret_cast<float4*>(p.h_last + (srow + 4 * r) * N + 4 * e + 32 * m) = s[r][m];
}

// ---------------------------------------------------------------- in chunks
// C = 64 tokens at a time.  With cum_i the chunk's inclusive prefix sum of
// Delta A, e_ij = exp(cum_i - cum_j), k and q normalised and S the state
// entering the chunk, the values a token really writes, u_i, solve
//
//     (I + L) u = diag(b) (v - diag(exp cum) k S^T),   L_ij = b_i (k_i . k_j) e_ij  for j < i
//
// so with T = (I + L)^-1 diag(b) and M_ij = scale (q_i . k_j) e_ij (j <= i)
//
//     X = v - diag(exp cum) k S^T            u = T X
//     y = scale diag(exp cum) q S^T + (M T) X
//     S <- exp(cum_C) S + u^T diag(exp(cum_C - cum)) k
//
// gdr_prep_kernel (chunk, head, batch), all chunks at once: the rows [T; M T]
// and each token's factors, into the workspace.  gdr_scan_kernel (64 state
// rows, head, batch), the chunks in order: three tcgen05 products a chunk,
//
//     1. [k; q] S^T       128 x 64 x N     k and q as they arrive (bf16, exact)
//     2. [T; M T] X       128 x 64 x 64
//     3. k^T u'           N x 64 x 64      u' = diag(exp(cum_C - cum)) u
//
// with k's and q's norms in the rows' factors.  Stacking the query's rows
// under the key's makes each product 128 rows tall, so the outputs cost no
// product of their own, and the value of a row of [k; q] S^T or [T; M T] X is
// in one thread's reach: X, u' and y are elementwise.  The state stays in
// registers in fp32 (thread: one n, 16 or 8 of the tile's rows).  Operands that
// the kernels compute (S, T, M, M T, X and u') are the sums of three bf16 parts
// (26 bits), their products taken part by part, so a chunk is as exact as fp32
// sums are: the state after a prefill is off by 1.0 to 1.7e-7 in the norm where
// the same formulas in fp32 are off by 0.9 to 1.6e-7, and y's error before it is
// rounded is as small.  T's diagonal, b, by far its largest entries, stays out
// of the product: b X is added in fp32.  Two parts of S, T, M and M T took 301
// us where this takes 344 (4096 tokens x 64 heads, N = 128) and left 3 to 9e-7
// of the state and 4e-6 of y before its rounding; two parts throughout, the
// diagonal among them, 5e-6 of the state; one bf16 rounding of any of them
// would leave 1e-3.
//
// What bounds them.  The prep kernel: the phases of a chunk's system, most of
// which keep two to four of its eight warps busy (warps wait at barriers 40% of
// their time; 0.46 instructions a cycle and scheduler): 28 ns a chunk of a head
// with four blocks an SM, 10 us for one alone.  The scan: its chain of three
// products a chunk, 3.8 us (N = 128).  With stamps of the clock in it a chunk
// takes 7060 cycles: 2060 are the products' (8 steps of 96 cycles, 4 of 209, 4
// of 113; the tensor pipe is busy 28% of the time), 3260 elementwise (S's parts
// 990, X 1040, u' 1020, the state 210; X and u' on two of the four schedulers,
// which tensor-memory lanes 0..63, the keys' rows, belong to), 1740 go between
// them: barriers, reads of tensor memory, warps that end after one another.
// Longer chunks need more shared memory than there is for [T; M T].
//
// The decays' exponents are differences of the prefix sums, which are taken
// in fp64 and kept as two floats: the sums reach hundreds, the differences of
// neighbours matter.  A token's Delta A is held above -200 (exp(-200) is 0 in
// fp32, so nothing changes) to keep the sums finite.
//
// A product takes whole rows, zeros of T and M among them, and 0 x NaN would
// carry a token that is not finite to those before it.  So the kernels keep
// such values out of T and X (0 in their place), remember the first token from
// which a channel is not finite, and put NaN into its u' and y from there on
// (12 us of 356, 4096 tokens x 64 heads).
constexpr int kGdrC = 64;             // tokens per chunk
constexpr int kGdrTile = 64;          // state rows per CTA of the scan
constexpr int kGdrFac = 5 * kGdrC;    // factors of a chunk
constexpr int kGdrSolved = 6 * kGdrC; // rows of 64 bf16 of its solved system: [T; M T] in three parts
constexpr int kGdrPrepThreads = 256;
constexpr int kGdrWarps = 16;         // elementwise warps of the scan
constexpr int kGdrScanThreads = 32 * (kGdrWarps + 2);

struct GdrChunkParams {
    const __nv_bfloat16* dt;      // [B][L][H]
    const __nv_bfloat16* beta;    // [B][L][H]
    const float* dt_bias;         // [H] or null
    const float* A;               // [H]
    const float* h_in;            // [B][H][P][N] or null
    __nv_bfloat16* y;             // [B][L][H][P]
    float* h_out;                 // [B][H][P][N]
    float* fac;                   // [B][chunks][H] of 64 tokens' {X's, u's, y's factor, the chunk's decay}, then their b
    int64_t L;
    int H, G, P;
    int chunk0, chunks;           // this launch's chunks of the sequence
    int segs, seg_chunks;         // its segments, and their chunks (the last may have fewer)
    float* seg_out;               // [B][segs - 1][H][P + N][N] a segment's last state from zero, then its transition
    float* seg_in;                // [B][segs - 1][H][P][N] the state that enters segment 1, 2, ..
    float scale, eps;
    unsigned wait_limit;
    unsigned long long* status;
    unsigned long long status_epoch;
};

__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) <= 3.402823466e38f; }
__device__ __forceinline__ float nan32() { return __uint_as_float(0x7fffffffu); }

__device__ __forceinline__ void gdr_fail(const GdrChunkParams& p) {
    atomicOr(&g_mm_fault, 1u);
    if (p.status) atomicExch(p.status, (p.status_epoch << 8) | 1ull);
}

// two floats at a time (add, multiply and fma take a pair per instruction)
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
// true in one lane of a converged warp, in a form that keeps the other
// operands of what it guards in uniform registers (a tcgen05.mma takes those:
// 32 to 64 cycles apart then, 46 and more when each operand is moved there
// from one lane's registers first)
__device__ __forceinline__ bool elect_sync() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// v[8] = the sum of three bf16 parts (8 bits each, round to nearest): a 16-byte
// piece of each
__device__ __forceinline__ void split3(const float* v, uint4 (&part)[3]) {
    uint32_t w[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 minus = f2(-1.0f, -1.0f);
        w[0][e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        float2 r = fma2(f2(bf16_lo(w[0][e]), bf16_hi(w[0][e])), minus, f2(v[2 * e], v[2 * e + 1]));
        w[1][e] = pack_bf16x2(r.x, r.y);
        r = fma2(f2(bf16_lo(w[1][e]), bf16_hi(w[1][e])), minus, r);
        w[2][e] = pack_bf16x2(r.x, r.y);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) part[k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}
// the parts `apart` bytes apart
__device__ __forceinline__ void split3_store8(const float* v, unsigned char* p, int apart) {
    uint4 part[3];
    split3(v, part);
#pragma unroll
    for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4*>(p + k * apart) = part[k];
}

template <int N>
struct GdrPrepLayout {
    static constexpr int ld = kGdrC + 4;                          // fp32 rows, 16-byte pieces of 8 rows on different banks
    static constexpr int kq_bytes = 2 * kGdrC * N * 2;            // [k; q]: a [128][64] block per 64 of N
    static constexpr int part = kGdrC * 128;                      // one part of T, of M or of M T
    static constexpr int mat_bytes = kGdrC * ld * 4;
    // L and its inverse (fp32) lie over k and q once [k; q] k^T is taken, T's
    // three parts and M's third over those once T is read; M T's parts take the
    // place of M's
    static constexpr int l_off = 0;
    static constexpr int inv_off = mat_bytes;
    static constexpr int kq_off = 0, t_off = 0;
    static constexpr int m3_off = 3 * part;
    static constexpr int m_off = (2 * mat_bytes + 1023) / 1024 * 1024;
    static_assert(m_off >= kq_bytes && m_off >= m3_off + part, "k and q, T's parts and M's third fit below M");
    // where M's part k lies
    __device__ static constexpr int m_part(int k) { return k < 2 ? m_off + k * part : m3_off; }
    static constexpr int f_off = m_off + 2 * part;
    static constexpr int floats = 5 * kGdrC;
    static constexpr int bar_off = f_off + floats * 4 + 32;
    static constexpr int smem_bytes = 1024 + bar_off + 3 * 8 + 16;
};

// d += a b in fp32 on mma.m16n8k8 with tf32 operands in two parts (tf32 keeps
// 11 bits; the second part's own cut leaves 2^-22)
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void split_tf32(float v, uint32_t& hi, uint32_t& lo) {
    asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(hi) : "f"(v));
    lo = __float_as_uint(v - __uint_as_float(hi));
}
// D [16 MT][8] = A [16 MT][8 KT] B [8 KT][8], fp32 row-major in shared memory
// (lda, ldb floats apart), one warp; lane 4 g + c holds rows g, g + 8 and
// columns 2 c, 2 c + 1 of each 16 x 8 tile
template <int MT, int KT>
__device__ __forceinline__ void warp_matmul(float (&d)[MT][4], const float* A, int lda, const float* B, int ldb, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m) d[m][0] = d[m][1] = d[m][2] = d[m][3] = 0.0f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        uint32_t bh[2], bl[2];
        split_tf32(B[(8 * k + c) * ldb + g], bh[0], bl[0]);
        split_tf32(B[(8 * k + c + 4) * ldb + g], bh[1], bl[1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float* a = A + (16 * m + g) * lda + 8 * k + c;
            uint32_t ah[4], al[4];
            split_tf32(a[0], ah[0], al[0]);
            split_tf32(a[8 * lda], ah[1], al[1]);
            split_tf32(a[4], ah[2], al[2]);
            split_tf32(a[8 * lda + 4], ah[3], al[3]);
            mma_tf32(d[m], ah, bh);
            mma_tf32(d[m], ah, bl);
            mma_tf32(d[m], al, bh);
        }
    }
}
// A 16 x 8 tile to fp32 row-major shared memory, times `sign`
__device__ __forceinline__ void store_tile(float* out, int ld, const float (&d)[4], float sign, int lane) {
    const int g = lane >> 2, c = lane & 3;
    *reinterpret_cast<float2*>(out + g * ld + 2 * c) = f2(sign * d[0], sign * d[1]);
    *reinterpret_cast<float2*>(out + (g + 8) * ld + 2 * c) = f2(sign * d[2], sign * d[3]);
}

// Eight warps.  Warp w reaches the tensor-memory lanes of quarter w % 4: rows
// 32 (w % 4).. of [k; q] [k; q]^T, whose diagonal holds the norms and whose
// columns of k, 32 (w / 4).. for this warp, become L (quarters 0 and 1) and M.
template <int N>
__global__ void __launch_bounds__(kGdrPrepThreads, 4)
gdr_prep_kernel(const GdrChunkParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_t)
{
    using Lay = GdrPrepLayout<N>;
    constexpr int ld = Lay::ld;
    extern __shared__ __align__(1024) unsigned char gdp_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(gdp_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* kq = sm + Lay::kq_off;
    float* Lm = reinterpret_cast<float*>(sm + Lay::l_off);
    float* Tm = reinterpret_cast<float*>(sm + Lay::inv_off);
    unsigned char* tt = sm + Lay::t_off;                 // T's parts, 64 rows each
    float* cum_hi = reinterpret_cast<float*>(sm + Lay::f_off);   // prefix sums times log2(e), hi + lo
    float* cum_lo = cum_hi + kGdrC;
    float* bt = cum_lo + kGdrC;                          // b_t
    float* rk = bt + kGdrC;                              // 1 / |k_t| or 1
    float* rq = rk + kGdrC;                              // scale / |q_t| or scale
    double* half_sum = reinterpret_cast<double*>(rq + kGdrC);
    int* bad = reinterpret_cast<int*>(half_sum + 1);     // the first token whose row of L is not finite
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Lay::bar_off);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3);

    const int c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, half = warp >> 2;
    const int64_t t0 = static_cast<int64_t>(p.chunk0 + c) * kGdrC;
    const int64_t unit = (static_cast<int64_t>(b) * p.chunks + c) * p.H + h;
    const int g = h / (p.H / p.G);
    if (p.status && tid == 0 && c == 0 && h == 0 && b == 0) p.status[1] = p.status_epoch;

    if (tid == 7 * 32) {
        *bad = kGdrC;
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        mbar_init(&bars[2], 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&bars[0], Lay::kq_bytes);
        for (int kb = 0; kb < N / 64; ++kb) {     // rows past the sequence read as zeros
            tma_load_3d(kq + kb * 16384, &tm_k, g * N + kb * 64, static_cast<int>(t0), b, &bars[0]);
            tma_load_3d(kq + kb * 16384 + 8192, &tm_q, g * N + kb * 64, static_cast<int>(t0), b, &bars[0]);
        }
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 128);
        tmem_relinquish();
        tc_fence_before();
    }
    // decays and write strengths; a token past the sequence has a = 1, b = 0
    double cum = 0.0;
    bool fine = true;
    if (tid < kGdrC) {
        float la = 0.0f, be = 0.0f;
        if (t0 + tid < p.L) {
            const int64_t o = (static_cast<int64_t>(b) * p.L + t0 + tid) * p.H + h;
            la = MathExact::step(__bfloat162float(p.dt[o]), p.dt_bias ? p.dt_bias[h] : 0.0f) * p.A[h];
            la = la < -200.0f ? -200.0f : la;         // a NaN stays
            be = 1.0f / (1.0f + expf(-__bfloat162float(p.beta[o])));
        }
        cum = static_cast<double>(la) * 1.4426950408889634;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double n = __shfl_up_sync(kFull, cum, o);
            if (lane >= o) cum += n;
        }
        if (tid == 31) *half_sum = cum;
        fine = is_finite(la) && is_finite(be);
        bt[tid] = is_finite(be) ? be : 0.0f;
    }
    __syncthreads();
    if (!fine) atomicMin(bad, tid);
    if (tid < kGdrC) {
        if (warp == 1) cum += *half_sum;
        const float hi = static_cast<float>(cum);
        cum_hi[tid] = hi;
        cum_lo[tid] = static_cast<float>(cum - static_cast<double>(hi));
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);

    // [k; q] [k; q]^T
    bool loaded = true;
    if (warp == 7) {
        loaded = warp_wait(&bars[0], 0, p.wait_limit);
        if (loaded && elect_sync()) {
            constexpr uint32_t idesc = umma_idesc_bf16(2 * kGdrC, 2 * kGdrC);
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk) {
                const uint64_t d = umma_desc_sw128(smem_addr(kq) + (kk >> 2) * 16384 + (kk & 3) * 32);
                umma_bf16(tmem, d, d, idesc, kk > 0 ? 1u : 0u);
            }
            umma_commit(&bars[1]);
        }
    }
    loaded = __syncthreads_and(loaded);
    bool ok = loaded && warp_wait(&bars[1], 0, p.wait_limit);
    tc_fence_after();
    if (ok && half == 0) {
        float m[32], s = 0.0f;
        tmem_ld32(lane_base + q * 32, m);
#pragma unroll
        for (int e = 0; e < 32; ++e) s = lane == e ? m[e] : s;
        const float r = p.eps > 0.0f ? rsqrtf(s + p.eps) : 1.0f;
        if (q < 2) rk[tid] = r;
        else rq[tid - kGdrC] = r * p.scale;
    }
    const bool ready = __syncthreads_and(ok);

    // row i of L (quarters 0, 1) or of M, 32 columns; the columns past the
    // row's own 32-column block are zero.  M's third part waits in registers
    // until its place is free.
    uint4 m3[4] = {};
    if (ready) {
        const int i = (q & 1) * 32 + lane;
        const bool key = q < 2;
        float m[32];
        if (half <= (q & 1)) {
            tmem_ld32(lane_base + half * 32, m);
            const float ch = cum_hi[i], cl = cum_lo[i];
            const float ri = key ? bt[i] * rk[i] : rq[i];
            const int last = key ? i - 1 : i;             // the row's last column
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
                const int j = half * 32 + 4 * e4;
                const float4 jh = *reinterpret_cast<const float4*>(cum_hi + j), jl = *reinterpret_cast<const float4*>(cum_lo + j),
                             jr = *reinterpret_cast<const float4*>(rk + j);
                m[4 * e4] = j <= last ? m[4 * e4] * (ri * jr.x) * ex2_fast((ch - jh.x) + (cl - jl.x)) : 0.0f;
                m[4 * e4 + 1] = j + 1 <= last ? m[4 * e4 + 1] * (ri * jr.y) * ex2_fast((ch - jh.y) + (cl - jl.y)) : 0.0f;
                m[4 * e4 + 2] = j + 2 <= last ? m[4 * e4 + 2] * (ri * jr.z) * ex2_fast((ch - jh.z) + (cl - jl.z)) : 0.0f;
                m[4 * e4 + 3] = j + 3 <= last ? m[4 * e4 + 3] * (ri * jr.w) * ex2_fast((ch - jh.w) + (cl - jl.w)) : 0.0f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) m[e] = 0.0f;
        }
        if (key) {
            float odd = 0.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e) odd = fmaf(m[e], 0.0f, odd);
            if (odd != 0.0f) {
                atomicMin(bad, i);
#pragma unroll
                for (int e = 0; e < 32; ++e) m[e] = is_finite(m[e]) ? m[e] : 0.0f;
            }
        }
        if (key) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                *reinterpret_cast<float4*>(Lm + i * ld + half * 32 + 4 * e) = make_float4(m[4 * e], m[4 * e + 1], m[4 * e + 2], m[4 * e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t off = sw128_off(i, half * 4 + e);
                uint4 part[3];
                split3(m + 8 * e, part);
                *reinterpret_cast<uint4*>(sm + Lay::m_part(0) + off) = part[0];
                *reinterpret_cast<uint4*>(sm + Lay::m_part(1) + off) = part[1];
                m3[e] = part[2];
            }
        }
    }
    __syncthreads();

    // T = (I + L)^-1 in fp32: the four 16 x 16 diagonal blocks by substitution,
    // then twice [[P, 0], [R, Q]]^-1 = [[P^-1, 0], [-Q^-1 R P^-1, Q^-1]], eight
    // columns a warp
    if (tid < kGdrC) {
        const int d = tid >> 4, col = tid & 15;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float* row = Lm + (16 * d + r) * ld + 16 * d;
            float s[4] = {r == col ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int l = 0; l < r; l += 4) {
                const float4 v = *reinterpret_cast<const float4*>(row + l);
                s[0] = fmaf(-v.x, x[l], s[0]);
                if (l + 1 < r) s[1] = fmaf(-v.y, x[l + 1], s[1]);
                if (l + 2 < r) s[2] = fmaf(-v.z, x[l + 2], s[2]);
                if (l + 3 < r) s[3] = fmaf(-v.w, x[l + 3], s[3]);
            }
            x[r] = (s[0] + s[1]) + (s[2] + s[3]);
            Tm[(16 * d + r) * ld + 16 * d + col] = x[r];
        }
    } else if (tid < 2 * kGdrC) {
        // zeros right of the diagonal blocks
        const int i = tid - kGdrC;
        for (int j = (i / 16 + 1) * 16; j < kGdrC; j += 4) *reinterpret_cast<float4*>(Tm + i * ld + j) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else if (ready && tid < 3 * kGdrC) {
        // the tokens' factors; from the first token whose row of L is not
        // finite on, one that makes X what its u is
        const int t = tid - 2 * kGdrC;
        const float gam = ex2_fast(cum_hi[t] + cum_lo[t]);
        const float end = ex2_fast((cum_hi[kGdrC - 1] - cum_hi[t]) + (cum_lo[kGdrC - 1] - cum_lo[t]));
        float* fac = p.fac + unit * kGdrFac;
        *reinterpret_cast<float4*>(fac + 4 * t) = make_float4(t < *bad ? gam * rk[t] : nan32(), end * rk[t], gam * rq[t],
                                                              ex2_fast(cum_hi[kGdrC - 1] + cum_lo[kGdrC - 1]));
        fac[4 * kGdrC + t] = bt[t];
    }
    __syncthreads();
    // W lies in L's upper right block, which nothing reads
    if (warp < 4) {
        const int o = (warp >> 1) * 32, n = (warp & 1) * 8;
        float* work = Lm + o / 2 * ld + 32 + n;
        float d[1][4];
        warp_matmul<1, 2>(d, Lm + (o + 16) * ld + o, ld, Tm + o * ld + o + n, ld, lane);
        store_tile(work, ld, d[0], 1.0f, lane);
        __syncwarp();
        warp_matmul<1, 2>(d, Tm + (o + 16) * ld + o + 16, ld, work, ld, lane);
        store_tile(Tm + (o + 16) * ld + o + n, ld, d[0], -1.0f, lane);
    }
    __syncthreads();
    {
        const int n = (warp & 3) * 8, m = (warp >> 2) * 16;
        float d[1][4];
        warp_matmul<1, 4>(d, Lm + (32 + m) * ld, ld, Tm + n, ld, lane);
        store_tile(Lm + m * ld + 32 + n, ld, d[0], 1.0f, lane);
        __syncthreads();
        warp_matmul<1, 4>(d, Tm + (32 + m) * ld + 32, ld, Lm + 32 + n, ld, lane);
        store_tile(Tm + (32 + m) * ld + n, ld, d[0], -1.0f, lane);
    }
    __syncthreads();
    // T (diag(b) included) in its parts
    {
        const int i = tid & (kGdrC - 1), part = tid >> 6;     // a quarter of row i
        float t[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = *reinterpret_cast<const float4*>(Tm + i * ld + part * 16 + 4 * e);
            const float4 s = *reinterpret_cast<const float4*>(bt + part * 16 + 4 * e);
            t[4 * e] = v.x * s.x;
            t[4 * e + 1] = v.y * s.y;
            t[4 * e + 2] = v.z * s.z;
            t[4 * e + 3] = v.w * s.w;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t off = sw128_off(i, part * 2 + e);
            split3_store8(t + 8 * e, tt + off, Lay::part);
        }
    }
    if (q >= 2)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(sm + Lay::m_part(2) + sw128_off((q & 1) * 32 + lane, half * 4 + e)) = m3[e];
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // M T: A = the 128 rows that end with M's (the 64 before them are whatever
    // precedes the tile, and their results are not read); B = T [l][j], MN-major
    if (ready && warp == 7 && elect_sync()) {
        constexpr uint32_t idesc = umma_idesc_bf16_mn(2 * kGdrC, kGdrC, false, true);
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int j = 0; i + j < 3; ++j)
#pragma unroll
                for (int kk = 0; kk < kGdrC / 16; ++kk)
                    umma_bf16(tmem, umma_desc_sw128(smem_addr(sm) + Lay::m_part(i) - Lay::part + kk * 32),
                              umma_desc_sw128_mn(smem_addr(tt) + j * Lay::part + kk * 2048, 0), idesc, i + j + kk > 0 ? 1u : 0u);
        umma_commit(&bars[2]);
    }
    const bool done = ready && warp_wait(&bars[2], 0, p.wait_limit);
    tc_fence_after();
    if (done && q >= 2) {
        float m[32];
        tmem_ld32(lane_base + half * 32, m);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t off = sw128_off((q & 1) * 32 + lane, half * 4 + e);
            uint4 part[3];
            split3(m + 8 * e, part);
#pragma unroll
            for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4*>(sm + Lay::m_part(k) + off) = part[k];
        }
        fence_proxy_async_smem();
    }
    if (done && tid < kGdrC) {
        // M T is taken with all of T; the scan adds b X, T's diagonal, itself
        const uint32_t off = sw128_off(tid, tid >> 3) + (tid & 7) * 2;
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<__nv_bfloat16*>(tt + k * Lay::part + off) = __float2bfloat16_rn(0.0f);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    if (__syncthreads_and(done)) {
        if (tid == 0) {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int row = static_cast<int>(unit * kGdrSolved + k * 2 * kGdrC);
                tma_store_2d(&tm_t, tt + k * Lay::part, 0, row);
                tma_store_2d(&tm_t, sm + Lay::m_part(k), 0, row + kGdrC);
            }
            bulk_commit_group();
            bulk_wait_read_all();
        }
        if (warp == 2) {
            tc_fence_after();
            tmem_dealloc(tmem, 128);
        }
    } else {
        if (tid == 0) gdr_fail(p);
        // the copies and products finish before shared and tensor memory go away
        if (warp == 7 && elect_one_lane()) {
            if (!loaded) mbar_wait_bounded(&bars[0], 0, 1u << 20);
            else mbar_wait_bounded(&bars[ready ? 2 : 1], 0, 1u << 20);
        }
        __syncthreads();
        if (warp == 2) tmem_dealloc(tmem, 128);
    }
}

template <int N>
struct GdrScanLayout {
    static constexpr int kq_bytes = 2 * kGdrC * N * 2;          // [k; q]
    static constexpr int v_off = kq_bytes;                      // then v [token][64 rows] and the tokens' factors
    static constexpr int fac_off = v_off + kGdrC * 128;
    static constexpr int in_bytes = (fac_off + kGdrFac * 4 + 1023) / 1024 * 1024;
    static constexpr int t_bytes = 2 * kGdrC * 128;             // one part of [T; M T], of three
    static constexpr int s_bytes = N * 128;                     // one part of S^T [n][64 rows], of three
    static constexpr int x_bytes = kGdrC * 128;                 // one part of X or u' [token][64 rows], of three
    static constexpr int stages = 2;                            // of the inputs; the solved rows have one place
    static constexpr int t_off = stages * in_bytes;
    static constexpr int s_off = t_off + 3 * t_bytes;
    // X and u' lie over S, which product 1 has read by then
    static constexpr int x_off = s_off;
    static_assert(x_bytes <= s_bytes, "X's parts fit S's place");
    static constexpr int bar_off = s_off + 3 * s_bytes;
    static constexpr int bars = 2 * stages + 8;
    static constexpr int odd_off = bar_off + bars * 8 + 16;     // the first token from which each row is not finite, and whether any is not
    static constexpr int smem_bytes = 1024 + odd_off + (kGdrTile + 4) * 4;
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" :: "r"(smem_addr(bar)) : "memory");
}
// 16 consecutive fp32 columns of this thread's row of tensor memory, without
// waiting: the registers are valid after tmem_wait_ld
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// v = the sums of COLS columns at `taddr` and as many 64 (and, of three parts,
// 128) further on: a product's parts
template <int COLS, int PARTS>
__device__ __forceinline__ void tmem_ld_sum(uint32_t taddr, float (&v)[COLS]) {
    uint32_t part[PARTS][COLS];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        if constexpr (COLS == 16) tmem_ld16_async(taddr + 64 * k, part[k]);
        else tmem_ld8_async(taddr + 64 * k, part[k]);
    }
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < COLS; i += 2) {
        float2 r = f2(__uint_as_float(part[PARTS - 1][i]), __uint_as_float(part[PARTS - 1][i + 1]));
#pragma unroll
        for (int k = PARTS - 2; k >= 0; --k) r = add2(r, f2(__uint_as_float(part[k][i]), __uint_as_float(part[k][i + 1])));
        v[i] = r.x;
        v[i + 1] = r.y;
    }
}

// 16 elementwise warps, one that issues the products and one that copies.
// Warp w reaches the tensor-memory lanes of quarter w % 4 and takes columns
// 16 (w / 4).. of its rows: quarters 0 and 1 hold the tokens' keys (X and u'),
// 2 and 3 their queries (y).  With N = 64 product 3 takes the 64 rows of k^T
// twice (both 64-row blocks of the operand at one address), so that all four
// quarters hold the state, 8 columns a thread instead of 16.
//
// STATE: the pass over segments before the one that writes y (see
// gdr_segment_kernel).  A tile of P / 64 or above is one of the transition's:
// its rows start as rows of the identity and its v is zero.
template <int N, bool STATE>
__global__ void __launch_bounds__(kGdrScanThreads, 1)
gdr_scan_kernel(const GdrChunkParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_t)
{
    using Lay = GdrScanLayout<N>;
    constexpr int kStages = Lay::stages;
    constexpr int kCols = N == 128 ? 16 : 8;             // state entries per thread
    constexpr uint32_t kD1 = 0, kD2 = 192, kD3 = 384, kTmemCols = 512;    // 64 columns of each part
    extern __shared__ __align__(1024) unsigned char gds_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(gds_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* kq_full = reinterpret_cast<uint64_t*>(sm + Lay::bar_off);
    uint64_t* kq_free = kq_full + kStages;
    uint64_t* t_full = kq_free + kStages;
    uint64_t* t_free = t_full + 1;
    uint64_t* d_full = t_free + 1;                       // [3] products 1, 2, 3
    uint64_t* in_full = d_full + 3;                      // [3] S, X, u' written
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + 3);
    int* odd_from = reinterpret_cast<int*>(sm + Lay::odd_off);
    volatile int* any_odd = odd_from + kGdrTile;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int segs = STATE ? p.segs - 1 : p.segs;
    const int tile = blockIdx.x, h = blockIdx.y, b = blockIdx.z / segs, seg = blockIdx.z - b * segs;
    const int g = h / (p.H / p.G);
    const int first = seg * p.seg_chunks;
    const int n_chunks = min(p.seg_chunks, p.chunks - first);
    const bool values = tile < p.P / kGdrTile;
    if (STATE && !values && seg == 0) return;      // the first segment's own state is known
    constexpr uint32_t t_rows = STATE ? 64 : 128;  // of [T; M T], and [k; q], that this pass uses

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&kq_full[s], 1);
            mbar_init(&kq_free[s], 1);
        }
        mbar_init(t_full, 1);
        mbar_init(t_free, 1);
        for (int i = 0; i < 3; ++i) mbar_init(&d_full[i], 1);
        mbar_init(&in_full[0], kGdrWarps);
        mbar_init(&in_full[1], kGdrWarps / 2);
        mbar_init(&in_full[2], kGdrWarps);
        fence_mbar_init();
        *any_odd = 0;
    }
    if (tid < kGdrTile) odd_from[tid] = 0x7fffffff;
    // What the kernels before wrote is read from here on.  All of tensor memory
    // is allocated after that, too: a block of theirs that has yet to allocate
    // could otherwise wait for this one, and this one for it.
    grid_dependency_wait();
    if (warp == kGdrWarps) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    int issued = 0;          // the copying lane: chunks requested; the other: products committed

    if (warp == kGdrWarps + 1) {
        if (elect_one_lane()) {
            for (int c = 0; c < n_chunks && ok; ++c) {
                const int s = c % kStages;
                const unsigned par = static_cast<unsigned>(((c / kStages) & 1) ^ 1);
                unsigned char* kq = sm + s * Lay::in_bytes;
                unsigned char* tt = sm + Lay::t_off;
                const int tok = (p.chunk0 + first + c) * kGdrC;
                if (!(ok = mbar_wait_bounded(&kq_free[s], par, p.wait_limit))) break;
                const int64_t unit = (static_cast<int64_t>(b) * p.chunks + first + c) * p.H + h;
                mbar_arrive_expect_tx(&kq_full[s], t_rows * N * 2 + (values ? kGdrC * 128 : 0) + kGdrFac * 4);
                for (int kb = 0; kb < N / 64; ++kb) {
                    tma_load_3d(kq + kb * 16384, &tm_k, g * N + kb * 64, tok, b, &kq_full[s]);
                    if (!STATE) tma_load_3d(kq + kb * 16384 + 8192, &tm_q, g * N + kb * 64, tok, b, &kq_full[s]);
                }
                if (values) tma_load_3d(kq + Lay::v_off, &tm_v, h * p.P + tile * kGdrTile, tok, b, &kq_full[s]);
                bulk_load(kq + Lay::fac_off, p.fac + unit * kGdrFac, kGdrFac * 4, &kq_full[s]);
                ++issued;
                if (!(ok = mbar_wait_bounded(t_free, static_cast<unsigned>(c & 1) ^ 1u, p.wait_limit))) break;
                const int row = static_cast<int>(unit * kGdrSolved);
                mbar_arrive_expect_tx(t_full, 3 * t_rows * 128);
#pragma unroll
                for (int k = 0; k < 6; ++k)
                    if (!STATE || k % 2 == 0) tma_load_2d(tt + k * 8192, &tm_t, 0, row + k * 64, t_full);
                ++issued;
            }
        }
    } else if (warp == kGdrWarps) {
        // A product's second operand has its parts side by side, 192 columns: 32
        // cycles a part and K step of 16, where a product of 64 columns takes 49
        // (bound by the first operand's reads).  Of two operands in parts, the
        // products whose parts' places add up to more than the third's are left
        // out (2^-26).  u's third part goes onto its second one's columns:
        // tensor memory holds 8 parts, not 9.
        constexpr uint32_t id_3 = umma_idesc_bf16_mn(2 * kGdrC, 3 * kGdrTile, false, true);
        constexpr uint32_t id_2 = umma_idesc_bf16_mn(2 * kGdrC, 2 * kGdrTile, false, true);
        constexpr uint32_t id_1 = umma_idesc_bf16_mn(2 * kGdrC, kGdrTile, false, true);
        constexpr uint32_t id_u2 = umma_idesc_bf16_mn(128, 2 * kGdrTile, true, true);
        constexpr uint32_t id_u1 = umma_idesc_bf16_mn(128, kGdrTile, true, true);
        const uint32_t sh = smem_addr(sm + Lay::s_off), xh = smem_addr(sm + Lay::x_off), th = smem_addr(sm + Lay::t_off);
        for (int c = 0; c < n_chunks; ++c) {
            const int s = c % kStages;
            const unsigned par = static_cast<unsigned>(c & 1), spar = static_cast<unsigned>((c / kStages) & 1);
            const uint32_t kq = smem_addr(sm + s * Lay::in_bytes);
            if (!(ok = warp_wait(&kq_full[s], spar, p.wait_limit) && warp_wait(&in_full[0], par, p.wait_limit))) break;
            tc_fence_after();
            if (elect_sync()) {
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk)
                    umma_bf16(tmem + kD1, umma_desc_sw128(kq + (kk >> 2) * 16384 + (kk & 3) * 32),
                              umma_desc_sw128_mn(sh + kk * 2048, Lay::s_bytes), id_3, kk > 0 ? 1u : 0u);
                umma_commit(&d_full[0]);
            }
            ++issued;
            if (!(ok = warp_wait(t_full, par, p.wait_limit) && warp_wait(&in_full[1], par, p.wait_limit))) break;
            tc_fence_after();
            if (elect_sync()) {
#pragma unroll
                for (int kk = 0; kk < kGdrC / 16; ++kk) {
                    umma_bf16(tmem + kD2, umma_desc_sw128(th + kk * 32), umma_desc_sw128_mn(xh + kk * 2048, Lay::x_bytes), id_3,
                              kk > 0 ? 1u : 0u);
                    umma_bf16(tmem + kD2, umma_desc_sw128(th + Lay::t_bytes + kk * 32),
                              umma_desc_sw128_mn(xh + kk * 2048, Lay::x_bytes), id_2, 1u);
                    umma_bf16(tmem + kD2, umma_desc_sw128(th + 2 * Lay::t_bytes + kk * 32), umma_desc_sw128_mn(xh + kk * 2048, 0),
                              id_1, 1u);
                }
                umma_commit(&d_full[1]);
                umma_commit(t_free);
            }
            ++issued;
            if (!(ok = warp_wait(&in_full[2], par, p.wait_limit))) break;
            tc_fence_after();
            if (elect_sync()) {
#pragma unroll
                for (int kk = 0; kk < kGdrC / 16; ++kk) {
                    const uint64_t kt = umma_desc_sw128_mn(kq + kk * 2048, N == 128 ? 16384 : 0);
                    umma_bf16(tmem + kD3, kt, umma_desc_sw128_mn(xh + kk * 2048, Lay::x_bytes), id_u2, kk > 0 ? 1u : 0u);
                    umma_bf16(tmem + kD3 + 64, kt, umma_desc_sw128_mn(xh + 2 * Lay::x_bytes + kk * 2048, 0), id_u1, 1u);
                }
                umma_commit(&d_full[2]);
                umma_commit(&kq_free[s]);
            }
            ++issued;
        }
    } else {
        const int q = warp & 3, wg = warp >> 2;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const int i = (q & 1) * 32 + lane;                                   // this thread's token of a chunk
        const int col0 = wg * 16;                                            // its 16 of the tile's rows
        const int n = N == 128 ? q * 32 + lane : (q & 1) * 32 + lane;        // its state: entry n
        const int srow0 = N == 128 ? wg * 16 : wg * 16 + (q >> 1) * 8;       // of these rows of the tile
        unsigned char* sp = sm + Lay::s_off;
        unsigned char* xp = sm + Lay::x_off;
        float S[kCols];
        const int64_t heads = (static_cast<int64_t>(b) * p.H + h), row = tile * kGdrTile + srow0;
        const int64_t state = (heads * p.P + row) * N + n;
        // segment `seg_` of the P (or P + N) rows of a state of each but one
        auto of_segment = [&](int seg_, int rows) {
            return (((static_cast<int64_t>(b) * (p.segs - 1) + seg_) * p.H + h) * rows + row) * N + n;
        };
        const float* src = seg == 0 ? (p.h_in ? p.h_in + state : nullptr)
                                    : (STATE ? nullptr : p.seg_in + of_segment(seg - 1, p.P));
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            S[j] = src ? src[static_cast<int64_t>(j) * N] : (STATE && row + j == p.P + n ? 1.0f : 0.0f);

        auto wait = [&](uint64_t* bar, unsigned parity) { return ok = warp_wait(bar, parity, p.wait_limit); };
        auto arrive = [&](uint64_t* bar) {
            __syncwarp();
            if (elect_one_lane()) mbar_arrive(bar);
        };
        // whether any value of this chunk or one before it is not finite; the
        // keys' warps have said so before they arrived there
        auto is_odd = [&](unsigned parity) {
            mbar_try_wait(&in_full[1], parity);
            return *any_odd != 0;
        };
        // this thread's part of an operand is written: to the products
        auto hand_over = [&](uint64_t* bar) {
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(bar);
        };
        auto write_state = [&] {
#pragma unroll
            for (int k = 0; k < kCols / 8; ++k) {
                const uint32_t off = sw128_off(n, srow0 / 8 + k);
                split3_store8(S + 8 * k, sp + off, Lay::s_bytes);
            }
            hand_over(&in_full[0]);
        };
        auto add_state = [&](float decay) {
            float add[kCols];
            tmem_ld_sum<kCols, 2>(lane_base + kD3 + srow0, add);
#pragma unroll
            for (int j = 0; j < kCols; j += 2) {
                const float2 r = fma2(f2(decay, decay), f2(S[j], S[j + 1]), f2(add[j], add[j + 1]));
                S[j] = r.x;
                S[j + 1] = r.y;
            }
        };
        if (q < 2) {
            for (int c = 0; c < n_chunks; ++c) {
                const int s = c % kStages;
                const unsigned par = static_cast<unsigned>(c & 1);
                const unsigned char* in = sm + s * Lay::in_bytes;
                write_state();
                if (!wait(&kq_full[s], static_cast<unsigned>((c / kStages) & 1))) break;
                const float4 f = *reinterpret_cast<const float4*>(in + Lay::fac_off + i * 16);
                const float bi = *reinterpret_cast<const float*>(in + Lay::fac_off + kGdrC * 16 + i * 4);
                uint4 v[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    v[k] = values ? *reinterpret_cast<const uint4*>(in + Lay::v_off + sw128_off(i, wg * 2 + k)) : make_uint4(0u, 0u, 0u, 0u);
                if (!wait(&d_full[0], par)) break;
                tc_fence_after();
                float x[16];
                tmem_ld_sum<16, 3>(lane_base + kD1 + col0, x);
                float2 odd = f2(0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 r = fma2(f2(-f.x, -f.x), f2(x[8 * k + 2 * e], x[8 * k + 2 * e + 1]), f2(bf16_lo(w[e]), bf16_hi(w[e])));
                        x[8 * k + 2 * e] = r.x;
                        x[8 * k + 2 * e + 1] = r.y;
                        odd = fma2(r, f2(0.0f, 0.0f), odd);
                    }
                }
                if (odd.x + odd.y != 0.0f) {
                    *any_odd = 1;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (!is_finite(x[e])) {
                            atomicMin(odd_from + col0 + e, c * kGdrC + i);
                            x[e] = 0.0f;
                        }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) split3_store8(x + 8 * k, xp + sw128_off(i, wg * 2 + k), Lay::x_bytes);
                hand_over(&in_full[1]);
                if (!wait(&d_full[1], par)) break;
                tc_fence_after();
                float u[16];
                tmem_ld_sum<16, 3>(lane_base + kD2 + col0, u);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float2 r = mul2(f2(f.y, f.y), fma2(f2(bi, bi), f2(x[8 * k + e], x[8 * k + e + 1]),
                                                                 f2(u[8 * k + e], u[8 * k + e + 1])));
                        u[8 * k + e] = r.x;
                        u[8 * k + e + 1] = r.y;
                    }
                }
                if (is_odd(par))
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = odd_from[col0 + e] <= c * kGdrC + i ? nan32() : u[e];
#pragma unroll
                for (int k = 0; k < 2; ++k) split3_store8(u + 8 * k, xp + sw128_off(i, wg * 2 + k), Lay::x_bytes);
                hand_over(&in_full[2]);
                if (!wait(&d_full[2], par)) break;
                tc_fence_after();
                add_state(f.w);
            }
        } else {
            // y of a chunk, stored once the next chunk's first operand is
            // written: the fence before that waits for the memory operations before it
            uint32_t yw[8] = {};
            auto store_y = [&](int c) {
                const int64_t t = static_cast<int64_t>(p.chunk0 + first + c) * kGdrC + i;
                if (t < p.L) {
                    uint4* dst = reinterpret_cast<uint4*>(p.y + ((static_cast<int64_t>(b) * p.L + t) * p.H + h) * p.P +
                                                          tile * kGdrTile + col0);
                    dst[0] = make_uint4(yw[0], yw[1], yw[2], yw[3]);
                    dst[1] = make_uint4(yw[4], yw[5], yw[6], yw[7]);
                }
            };
            for (int c = 0; c < n_chunks; ++c) {
                const int s = c % kStages;
                const unsigned par = static_cast<unsigned>(c & 1);
                write_state();
                if (!STATE && c > 0) store_y(c - 1);
                if (!wait(&kq_full[s], static_cast<unsigned>((c / kStages) & 1))) break;
                const float4 f = *reinterpret_cast<const float4*>(sm + s * Lay::in_bytes + Lay::fac_off + i * 16);
                // no u' of this warp's: it only must have read its factors
                // before product 3 lets the next chunk but one overwrite them
                arrive(&in_full[2]);
                if (!STATE) {
                    if (!wait(&d_full[1], par)) break;
                    tc_fence_after();
                    float d[16], u[16];
                    tmem_ld_sum<16, 3>(lane_base + kD1 + col0, d);
                    tmem_ld_sum<16, 3>(lane_base + kD2 + col0, u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 r = fma2(f2(f.z, f.z), f2(d[2 * e], d[2 * e + 1]), f2(u[2 * e], u[2 * e + 1]));
                        yw[e] = pack_bf16x2(r.x, r.y);
                    }
                    if (is_odd(par))
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            yw[e] |= (odd_from[col0 + 2 * e] <= c * kGdrC + i ? 0x7fffu : 0u) |
                                     (odd_from[col0 + 2 * e + 1] <= c * kGdrC + i ? 0x7fff0000u : 0u);
                }
                if (!wait(&d_full[2], par)) break;
                tc_fence_after();
                add_state(f.w);
            }
            if (!STATE && ok) store_y(n_chunks - 1);
        }
        if (ok && (STATE || seg == p.segs - 1)) {
            float* dst = STATE ? p.seg_out + of_segment(seg, p.P + N) : p.h_out + state;
#pragma unroll
            for (int j = 0; j < kCols; ++j) dst[static_cast<int64_t>(j) * N] = S[j];
        }
    }
    tc_fence_before();
    if (!__syncthreads_and(ok)) {
        if (tid == 0) gdr_fail(p);
        // the copies and products in flight finish before shared and tensor memory go away
        if (warp == kGdrWarps + 1 && elect_one_lane()) {
            for (int k = max(0, issued - 2 * kStages); k < issued; ++k) {
                const int c = k / 2, s = c % kStages;
                if (k % 2) mbar_wait_bounded(t_full, static_cast<unsigned>(c & 1), 1u << 20);
                else mbar_wait_bounded(&kq_full[s], static_cast<unsigned>((c / kStages) & 1), 1u << 20);
            }
        } else if (warp == kGdrWarps && elect_one_lane() && issued > 0) {
            const int k = issued - 1;
            mbar_wait_bounded(&d_full[k % 3], static_cast<unsigned>((k / 3) & 1), 1u << 20);
        }
        __syncthreads();
    }
    if (warp == kGdrWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- segments of a long sequence
// A chunk's products wait for one another, so a sequence's chunks in order
// leave most SMs idle when there are few heads.  A segment of chunks is affine
// in the state that enters it, S_out = S_in A + S_0, with S_0 its last state
// from zero and row m of A its last state from row m of the identity without
// values.  So: gdr_scan_kernel<N, true> over all segments but the last for
// S_0 and A (N more rows of a state), this kernel for the states entering
// them, in order, and gdr_scan_kernel<N, false> over all segments at once.
// CTA: 16 rows of a head's state; thread: one column; fp32, 128 x 128 x 16 a
// segment from A in shared memory, the next segment's on its way meanwhile
// (read from L2 by each thread, it took 18 us a segment).
constexpr int kGdrSegRows = 16;
template <int N>
struct GdrSegmentLayout {
    static constexpr int a_bytes = N * N * 4;
    static constexpr int cur_off = 2 * a_bytes;
    static constexpr int bar_off = cur_off + N * kGdrSegRows * 4;
    static constexpr int smem_bytes = bar_off + 16;
};
template <int N>
__global__ void __launch_bounds__(N)
gdr_segment_kernel(const GdrChunkParams p)
{
    using Lay = GdrSegmentLayout<N>;
    extern __shared__ __align__(128) unsigned char gdt_sm[];
    float (*cur)[kGdrSegRows] = reinterpret_cast<float (*)[kGdrSegRows]>(gdt_sm + Lay::cur_off);
    uint64_t* full = reinterpret_cast<uint64_t*>(gdt_sm + Lay::bar_off);      // A's two buffers
    const int n = threadIdx.x, row0 = blockIdx.x * kGdrSegRows, h = blockIdx.y, b = blockIdx.z;
    const int rows = p.P + N;
    auto at = [&](int seg) { return (static_cast<int64_t>(b) * (p.segs - 1) + seg) * p.H + h; };
    auto request = [&](int seg) {
        mbar_arrive_expect_tx(&full[seg & 1], Lay::a_bytes);
        bulk_load(gdt_sm + (seg & 1) * Lay::a_bytes, p.seg_out + (at(seg) * rows + p.P) * N, Lay::a_bytes, &full[seg & 1]);
    };
    if (n == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        fence_mbar_init();
    }
    grid_dependency_wait();
    if (n == 0 && p.segs > 2) request(1);
    __syncthreads();
    float s[kGdrSegRows];
    for (int seg = 0; seg + 1 < p.segs; ++seg) {
        const float* from = p.seg_out + (at(seg) * rows + row0) * N + n;
        float next[kGdrSegRows];
#pragma unroll
        for (int r = 0; r < kGdrSegRows; ++r) next[r] = from[r * N];
        if (seg > 0) {
            // the buffer of the segment before is free: every thread is past it
            if (n == 0 && seg + 2 < p.segs) request(seg + 1);
#pragma unroll
            for (int r = 0; r < kGdrSegRows; ++r) cur[n][r] = s[r];
            // buffer seg & 1 is filled for segments 1, 3, .. or 2, 4, ..
            if (!__syncthreads_and(mbar_wait_bounded(&full[seg & 1], static_cast<unsigned>((seg - 1) >> 1) & 1u, p.wait_limit))) {
                if (n == 0) {
                    gdr_fail(p);
                    // the copies in flight finish before their shared memory goes away
                    mbar_wait_bounded(&full[seg & 1], static_cast<unsigned>((seg - 1) >> 1) & 1u, 1u << 20);
                    if (seg + 2 < p.segs)
                        mbar_wait_bounded(&full[(seg + 1) & 1], static_cast<unsigned>(seg >> 1) & 1u, 1u << 20);
                }
                __syncthreads();
                return;
            }
            const float* A = reinterpret_cast<const float*>(gdt_sm + (seg & 1) * Lay::a_bytes) + n;
#pragma unroll 8
            for (int m = 0; m < N; ++m) {
                const float a = A[m * N];
#pragma unroll
                for (int r = 0; r < kGdrSegRows; r += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(&cur[m][r]);
                    next[r] = fmaf(v.x, a, next[r]);
                    next[r + 1] = fmaf(v.y, a, next[r + 1]);
                    next[r + 2] = fmaf(v.z, a, next[r + 2]);
                    next[r + 3] = fmaf(v.w, a, next[r + 3]);
                }
            }
            __syncthreads();
        }
        float* to = p.seg_in + (at(seg) * p.P + row0) * N + n;
#pragma unroll
        for (int r = 0; r < kGdrSegRows; ++r) to[r * N] = s[r] = next[r];
    }
}

}  // namespace mm
