// Projection of a few rows by a weight of 4-bit numbers:
//
//     out[m, n] = sum_k x[m, k] s[n, k / G] (c[n, k] - z[n, k / G])
//
// with c in 0..15, packed two to a byte (even k in the low four bits), a bf16
// scale s and, optionally, a bf16 zero point z (8 without one) per G = 32, 64
// or 128 inputs of a row: the projections of a decoded token, where
// proj_gemm.cuh would pad the rows to 128 and read four times the bytes.
//
// Each weight is used once per row of x, so the weights' HBM traffic bounds
// the product as long as unpacking them keeps up.  A CTA owns 64 outputs; one
// thread streams 64 x 256 tiles of the weight (8 KB: 128 bytes a row, one
// swizzle atom) and the matching columns of x through a shared-memory ring by
// bulk tensor copies, which keeps tens of KB in flight per SM without a
// register held for them.  Eight warps, each with 16 outputs and half of a
// tile's inputs, unpack and multiply on mma.m16n8k16: the outputs are its
// 16 rows, so one row of x costs as much as eight, and no tensor memory or
// operand staging stands between a tile's arrival and its use.  (tcgen05
// takes its operands from shared or tensor memory: the unpacked weights, four
// times the bytes, would have to be written there first.)
//
// c - 8 is exact in bf16, and so is x; products and their sums over a group
// are fp32, and the scale is applied to a group's sum, so nothing is rounded
// to fewer bits before the output.  The zero point's part is
// s (8 - z) sum_k x[m, k], whose sum is one more mma with a matrix of ones; an
// output that is not finite is worked out again term by term.
//
// What bounds it: the instructions around the products.  For 16384 x 16384 with
// one row (52 us) 240 are executed for a warp's 16 x 128 weights, 126 of them
// on the integer pipe at two cycles each: 252 of the 390 cycles that these
// weights have on a scheduler of the SMs with two blocks (of 256 blocks on 148
// SMs; over all, 0.61 instructions a cycle).  Unpacking is 72 of the 126 (32
// mask-and-ors, 24 shifts, 16 byte permutes of x); what the others are has not
// been taken apart.  The copies alone take 29 us, the rest alone 47 (38 without
// the shifts, 44 without the subtractions or the permutes).  16384 x 4096, one
// row: 15.8 us, 2.2 TB/s.
//
// Unpacking: (w >> 4i) & 0x000f000f | 0x43004300 is the bf16 pair
// (128 + c_i, 128 + c_{i+4}) of a word of eight; one packed subtraction of 136
// leaves c - 8.  The pairs (i, i + 4) fix the order of the inputs within a
// word; x is permuted alike as it is read.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "mixer_common.cuh"
#include "proj_gemm.cuh"

namespace mm {

constexpr int kQ4Rows = 64;           // outputs per CTA
constexpr int kQ4K = 256;             // inputs per ring slot: 128 bytes of packed weights a row
constexpr int kQ4Consumers = 8;       // warps: 4 groups of 16 outputs x 2 halves of the slot's inputs
constexpr int kQ4Threads = 32 * (kQ4Consumers + 1);

struct Q4Params {
    const __nv_bfloat16* x;        // [M][K]
    const unsigned char* W;        // [N][K / 2]
    const __nv_bfloat16* scales;   // [N][K / G]
    const __nv_bfloat16* zeros;    // [N][K / G] or null (8)
    void* out;                     // [M][N] fp32 or bf16
    int M, N, K;
    int slots_per_cta;             // ring slots (256 inputs each) of a CTA's share of K
    unsigned wait_limit;
};

template <int MT>
struct Q4Layout {
    static constexpr int w_bytes = kQ4Rows * 128;                // 8 KB
    static constexpr int x_box = MT * 8 * 128;                   // 64 inputs of the rows of x
    static constexpr int stage_bytes = w_bytes + 4 * x_box;
    static constexpr int stages = 4;
    static constexpr int red_ld = kQ4Rows + 1;
    static constexpr int red_bytes = 2 * MT * 8 * red_ld * 4;    // both halves' sums, over the ring once it is drained
    static constexpr int smem_bytes = 1024 + stages * stage_bytes + 2 * stages * 8 + 16;
    static_assert(red_bytes <= stages * stage_bytes, "the sums fit the ring");
};

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the bf16 pair (c_i - 8, c_{i+4} - 8) of a packed word already shifted by 4 i;
// `magic` is 0x43004300 in a register: with both constants immediate the mask
// and the or are two instructions, and these bound the kernel
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, uint32_t magic) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;\n" : "=r"(v) : "r"(w), "r"(magic));
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(136.0f, 136.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void load_pair(const unsigned char* p, uint32_t* v) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = w.x;
    v[1] = w.y;
}

// One output term by term, as the formula has it.
__device__ __noinline__ float q4_formula(const Q4Params& p, int m, int n, int words) {
    const int groups = p.K / (8 * words);
    const __nv_bfloat16* x = p.x + static_cast<int64_t>(m) * p.K;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p.W + static_cast<int64_t>(n) * (p.K / 2));
    const int64_t row = static_cast<int64_t>(n) * groups;
    float sum = 0.0f;
    for (int q = 0; q < groups && sum == sum; ++q) {        // a NaN stays one
        const float z = __bfloat162float(p.zeros[row + q]);
        float part = 0.0f;
        for (int j = 0; j < words; ++j, ++w)
            for (int i = 0; i < 8; ++i, ++x)
                part = fmaf(__bfloat162float(*x), static_cast<float>((*w >> (4 * i)) & 15u) - z, part);
        sum = fmaf(__bfloat162float(p.scales[row + q]), part, sum);
    }
    return sum;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// a float of CTA `rank`'s shared memory, at this CTA's address of it
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

// GB: 32-input blocks of a group (G / 32).  MT: 8-row tiles of x.  The CTAs of
// a cluster share the outputs and split K; their sums are added in rank order.
template <int GB, int MT, bool ZEROS, bool OUT_BF16>
__global__ void __launch_bounds__(kQ4Threads)
proj_q4_kernel(const Q4Params p, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x)
{
    using Lay = Q4Layout<MT>;
    extern __shared__ __align__(1024) unsigned char q4_raw[];
    const uint32_t pad = (1024u - (smem_addr(q4_raw) & 1023u)) & 1023u;
    unsigned char* sm = q4_raw + pad;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + Lay::stages * Lay::stage_bytes);
    uint64_t* empty = full + Lay::stages;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n0 = blockIdx.x * kQ4Rows, m0 = blockIdx.y * MT * 8;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int slots_all = (p.K - 1) / kQ4K + 1;
    const int slot0 = static_cast<int>(rank) * p.slots_per_cta;
    const int slots = max(0, min(p.slots_per_cta, slots_all - slot0));

    if (tid == 0) {
        for (int s = 0; s < Lay::stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kQ4Consumers);
        }
        fence_mbar_init();
    }
    __syncthreads();

    bool ok = true;
    int issued = 0;
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    const int rt = warp & 3, kh = warp >> 2;      // consumers: 16-output group, half of the slot
    const int g = lane >> 2, c = lane & 3;

    if (warp == kQ4Consumers) {
        if (elect_one_lane()) {
            for (int i = 0; i < slots; ++i) {
                const int s = i % Lay::stages;
                if (!mbar_wait_bounded(&empty[s], static_cast<unsigned>(((i / Lay::stages) & 1) ^ 1), p.wait_limit)) {
                    ok = false;
                    break;
                }
                unsigned char* st = sm + s * Lay::stage_bytes;
                mbar_arrive_expect_tx(&full[s], Lay::stage_bytes);
                const int k0 = (slot0 + i) * kQ4K;
                tma_load_2d(st, &tm_w, k0 / 2, n0, &full[s]);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tma_load_2d(st + Lay::w_bytes + q * Lay::x_box, &tm_x, k0 + 64 * q, m0, &full[s]);
                ++issued;
            }
        }
    } else {
        constexpr int kGroups = 4 / GB;               // groups of a warp's 128 inputs
        uint32_t magic = 0x43004300u;
        asm volatile("" : "+r"(magic));               // kept in its register
        const int groups = p.K / (32 * GB);
        // this lane's two outputs; outputs past N read the last one's scales (their sums are not stored)
        const int64_t r0 = static_cast<int64_t>(min(n0 + rt * 16 + g, p.N - 1)) * groups;
        const int64_t r1 = static_cast<int64_t>(min(n0 + rt * 16 + g + 8, p.N - 1)) * groups;
        // Scales and zero points come straight from memory, two slots ahead.
        constexpr int kAhead = 2;
        __nv_bfloat16 sc[kAhead][2][kGroups], zc[kAhead][2][kGroups];
        const __nv_bfloat16 none = __float2bfloat16_rn(0.0f);
        constexpr int kStep = kQ4K / (32 * GB);        // groups of a slot
        const int g0 = slot0 * kStep + kh * kGroups;
        const __nv_bfloat16 *sp0 = p.scales + r0 + g0, *sp1 = p.scales + r1 + g0;
        const __nv_bfloat16 *zp0 = p.zeros + r0 + g0, *zp1 = p.zeros + r1 + g0;
        auto fetch = [&](int i, int d) {
            const int left = i < slots ? groups - g0 - i * kStep : 0;     // groups from this one on
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                const bool in = q < left;
                sc[d][0][q] = in ? sp0[i * kStep + q] : none;
                sc[d][1][q] = in ? sp1[i * kStep + q] : none;
                if constexpr (ZEROS) {
                    zc[d][0][q] = in ? zp0[i * kStep + q] : none;
                    zc[d][1][q] = in ? zp1[i * kStep + q] : none;
                }
            }
        };
#pragma unroll
        for (int d = 0; d < kAhead; ++d) fetch(d, d);
        for (int i0 = 0; i0 < slots && ok; i0 += kAhead)
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
            const int i = i0 + d;
            if (i >= slots) break;
            const int s = i % Lay::stages;
            float s0[kGroups], s1[kGroups], z0[kGroups], z1[kGroups];
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                s0[q] = __bfloat162float(sc[d][0][q]);
                s1[q] = __bfloat162float(sc[d][1][q]);
                z0[q] = ZEROS ? 8.0f - __bfloat162float(zc[d][0][q]) : 0.0f;
                z1[q] = ZEROS ? 8.0f - __bfloat162float(zc[d][1][q]) : 0.0f;
            }
            fetch(i + kAhead, d);
            if (!warp_wait(&full[s], static_cast<unsigned>((i / Lay::stages) & 1), p.wait_limit)) {
                ok = false;
                break;
            }
            // Lane c takes GB consecutive words of a group of a row (one load),
            // eight inputs each: as long as x comes in the same order, a
            // product's inputs may be any of the group's.
            const unsigned char* wrow = sm + s * Lay::stage_bytes + (rt * 16 + g) * 128;
            const unsigned char* xrow = sm + s * Lay::stage_bytes + Lay::w_bytes + g * 128;
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                const int word0 = kh * 16 + q * 4 * GB + c * GB;        // of the row's 32
                const uint32_t woff = ((static_cast<uint32_t>(word0 >> 2) ^ g) << 4) + (word0 & 3) * 4;
                // with four words a lane, lanes 2 and 3 take theirs in the order
                // 2, 3, 0, 1: x's pieces of eight lanes then lie in eight
                // different 16-byte columns
                const int turn = GB == 4 ? c & 2 : 0;
                uint32_t w0[GB], w1[GB];
                if constexpr (GB == 4) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        load_pair(wrow + woff + ((2 * k) ^ turn) * 4, w0 + 2 * k);
                        load_pair(wrow + 8 * 128 + woff + ((2 * k) ^ turn) * 4, w1 + 2 * k);
                    }
                } else if constexpr (GB == 2) {
                    load_pair(wrow + woff, w0);
                    load_pair(wrow + 8 * 128 + woff, w1);
                } else {
                    w0[0] = *reinterpret_cast<const uint32_t*>(wrow + woff);
                    w1[0] = *reinterpret_cast<const uint32_t*>(wrow + 8 * 128 + woff);
                }
                float part[MT][4], xs[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) part[t][k] = xs[t][k] = 0.0f;
#pragma unroll
                for (int j = 0; j < GB; ++j) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        a[u][0] = q4_pair(w0[j] >> (8 * u), magic);
                        a[u][1] = q4_pair(w1[j] >> (8 * u), magic);
                        a[u][2] = q4_pair(w0[j] >> (8 * u + 4), magic);
                        a[u][3] = q4_pair(w1[j] >> (8 * u + 4), magic);
                    }
                    const int word = word0 + (j ^ turn);      // its eight inputs: a 16-byte piece of x
                    const uint32_t xoff = (word >> 3) * Lay::x_box + ((static_cast<uint32_t>(word & 7) ^ g) << 4);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const uint4 x = *reinterpret_cast<const uint4*>(xrow + t * 1024 + xoff);
                        const uint32_t b0 = __byte_perm(x.x, x.z, 0x5410), b1 = __byte_perm(x.x, x.z, 0x7632);
                        const uint32_t b2 = __byte_perm(x.y, x.w, 0x5410), b3 = __byte_perm(x.y, x.w, 0x7632);
                        mma_bf16_16816(part[t], a[0], b0, b1);
                        mma_bf16_16816(part[t], a[1], b2, b3);
                        if constexpr (ZEROS) {
                            constexpr uint32_t one = 0x3f803f80u;
                            const uint32_t ones[4] = {one, one, one, one};
                            mma_bf16_16816(xs[t], ones, b0, b1);
                            mma_bf16_16816(xs[t], ones, b2, b3);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float v0 = ZEROS ? fmaf(z0[q], xs[t][e], part[t][e]) : part[t][e];
                        const float v1 = ZEROS ? fmaf(z1[q], xs[t][e], part[t][2 + e]) : part[t][2 + e];
                        acc[t][e] = fmaf(s0[q], v0, acc[t][e]);
                        acc[t][2 + e] = fmaf(s1[q], v1, acc[t][2 + e]);
                    }
                }
            }
            __syncwarp();
            if (elect_one_lane()) {
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" :: "r"(smem_addr(&empty[s])) : "memory");
            }
        }
    }
    // every copy has landed: the consumers waited for each slot, and a CTA that
    // gave up waits (bounded) for those it issued
    const bool all_ok = __syncthreads_and(ok);
    if (!all_ok) {
        if (tid == 0) atomicOr(&g_mm_fault, 1u);
        if (warp == kQ4Consumers && elect_one_lane())
            for (int i = max(0, issued - Lay::stages); i < issued; ++i)
                mbar_wait_bounded(&full[i % Lay::stages], static_cast<unsigned>((i / Lay::stages) & 1), 1u << 20);
        __syncthreads();
    }
    // sums [half][row of x][output], in the ring's space
    float* red = reinterpret_cast<float*>(sm);
    if (warp < kQ4Consumers) {
        float* r = red + kh * (MT * 8 * Lay::red_ld) + rt * 16 + g;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                r[(t * 8 + 2 * c + e) * Lay::red_ld] = acc[t][e];
                r[(t * 8 + 2 * c + e) * Lay::red_ld + 8] = acc[t][2 + e];
            }
    }
    if (ranks > 1) cluster_sync_all(); else __syncthreads();
    const int rows = min(MT * 8, p.M - m0);
    if (all_ok) {
        for (int i = tid + static_cast<int>(rank) * kQ4Threads; i < rows * kQ4Rows; i += static_cast<int>(ranks) * kQ4Threads) {
            const int m = i / kQ4Rows, n = i % kQ4Rows;
            if (n0 + n >= p.N) continue;
            const float* r = red + m * Lay::red_ld + n;
            float v = 0.0f;
            if (ranks > 1) {
                for (uint32_t k = 0; k < ranks; ++k)
                    v += ld_cluster_f32(smem_addr(r), k) + ld_cluster_f32(smem_addr(r + MT * 8 * Lay::red_ld), k);
            } else {
                v = r[0] + r[MT * 8 * Lay::red_ld];
            }
            // An infinity among x: its part of the two sums may be of either
            // sign, or 0 times it, and they make NaN of what the formula has
            // as an infinity.  Rare enough to be worked out from the start.
            if (ZEROS && !(fabsf(v) <= 3.402823466e38f)) v = q4_formula(p, m0 + m, n0 + n, 4 * GB);
            const int64_t o = static_cast<int64_t>(m0 + m) * p.N + n0 + n;
            if constexpr (OUT_BF16) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
            else static_cast<float*>(p.out)[o] = v;
        }
    }
    // no CTA of the cluster ends while another still reads its sums
    if (ranks > 1) cluster_sync_all();
}

}  // namespace mm
