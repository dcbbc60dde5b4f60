// mx_a4.cuh - tcgen05 product of two MXFP4 operands: y[m, n] = sum_k x[m, k] w[n, k].
//
// The block-scaled tensor-core MMA (kind::mxf4, one power-of-two scale per 32 values) takes both
// operands as they are stored: codes by TMA into 128-byte-swizzled shared memory, scale bytes into
// tensor memory, FP32 sums.  Nothing is expanded, so per K = 256 and CTA only 128 bytes a row move.
//
// A CTA pair computes 256 rows x BN outputs (BN 64, 128 or 192), K = 256 a stage, 4 MMAs of K = 64:
// each CTA holds 128 rows of x and half of the outputs' rows of W.  Scales: tensor memory holds, for
// every 128 rows and K = 128, 32 lanes x 4 columns (row 32 c + l in lane l, column c; its four bytes
// are four blocks, an MMA takes two of them), the same in all four lane quarters; each CTA needs those
// of its own rows of x and of all BN outputs.  Loader warps gather them from the stored rows [rows, K/32],
// 16 bytes a row for two stages, put them into that order in shared memory, and the issuing thread
// copies them with tcgen05.cp just before the stage's MMAs.
//
// Tensor memory: two accumulators of 192 columns (a tile's epilogue runs under the next one's main
// loop, which at K = 2560 takes only about 4000 cycles) and a scale buffer of 24 columns for each of the
// five stages of the ring: a scale buffer is written again only after the barrier that says the stage's
// MMAs are done.
//
// Roles (512 threads): warp 0 codes by TMA, warp 1 MMA issue (leader) and tensor memory, warps 2, 3, 12,
// 14 and 15 scales (with two loader warps their instructions took longer than the MMAs), warps 4-11
// epilogue; warp 13 would share the issuing warp's scheduler and stays idle.
#pragma once

#include "mx_gemm.cuh"

namespace w4a16 {
namespace mx4 {

using mxg::elect_one;
using mxg::Ring;

constexpr int kThreads = 512;
constexpr int kLoaders = 5, kGroups = 10;  // loader warps; groups of 32 rows: four of x, six of W
constexpr int kRows = 128;                // x rows of a CTA
constexpr int kStep = 256;                // K of a stage
constexpr int kStages = 5;
constexpr int kMaxBN = 192;
constexpr int kABytes = kRows * kStep / 2;
constexpr int kBBytes = kMaxBN / 2 * kStep / 2;
constexpr int kChunkBytes = 512;          // scales of 128 rows, K = 128
constexpr int kSBytes = 2 * 3 * kChunkBytes;   // of a stage: [K half][x, W rows 0-127, W rows 128-255]
constexpr int kAccCols = 192, kScaleCol0 = 2 * kAccCols, kScaleCols = 24;
constexpr int kTmemCols = 512;
static_assert(kScaleCol0 + kStages * kScaleCols <= kTmemCols, "tensor memory budget");
constexpr int kEpiWarps = 8;
constexpr int kOffB = kStages * kABytes, kOffS = kOffB + kStages * kBBytes, kOffBar = kOffS + kStages * kSBytes;
constexpr int kSmemBytes = kOffBar + 256 + 1024;   // + barriers, alignment slack
static_assert(kBBytes % 1024 == 0 && kSmemBytes <= 227 * 1024, "shared memory layout");

struct Params {
    mxg::Output o;            // M rows, J = N outputs
    const uint8_t *xs, *ws;   // scales [M, K/32], [N, K/32]
    int K, bn;
    int tiles_m, tiles;
};

// ------------------------------------------------------------------ PTX

// Block-scaled MMA of a CTA pair, both operands E2M1 in shared memory (K-major), E8M0 scales in
// tensor memory, two of them a row.
__device__ __forceinline__ void umma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// 32 rows of 16 bytes in shared memory -> 32 lanes x 4 columns, the same in all four lane quarters;
// in both CTAs of the pair, each from its own shared memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Descriptor of such rows: no swizzle, 16-byte rows, groups of eight 128 bytes apart.
__device__ __forceinline__ uint64_t desc_scales(uint32_t smem_addr) {
    uint64_t d = static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

// Instruction descriptor: E2M1 x E2M1, E8M0 scales, FP32 sums, both K-major; `id` the byte (0 or 2)
// of the scale words at which the MMA's two scales start.
__device__ __forceinline__ uint32_t idesc_mxf4(int m, int n, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(m >> 7) << 27) | (id << 29);
}

// ------------------------------------------------------------------ scale bytes

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// 16 bytes at a 16-byte boundary of an array of scale bytes; behind its end nothing is read.
__device__ __forceinline__ uint4 scale_chunk(const uint8_t *at, const uint8_t *end) {
    if (at + 16 <= end) return ldg_nc_v4(at);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; i < 16; ++i)
        if (at + i < end) w[i >> 2] |= static_cast<uint32_t>(__ldg(at + i)) << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes off .. off + 15 of two neighbouring chunks, the first `valid` of them; 127 for the others.
__device__ __forceinline__ uint4 scale_window(const uint4 &a, const uint4 &b, uint32_t off, int valid) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(w[i], w[i + 1], 8 * (off & 3));
    if (valid < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = valid - 4 * i;
            const uint32_t mask = n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
            v[i] = (v[i] & mask) | (0x7F7F7F7Fu & ~mask);
        }
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// A group of 32 rows, a row a lane: its sixteen bytes of two stages lie in one or two aligned chunks,
// the second of which is the first of the next two stages: one 16-byte load a row for two stages
// whatever the rows' alignment, issued two stages ahead.
struct ScaleGroup {
    const uint8_t *at;                          // the chunk of the row's first byte; null: no such row
    const uint8_t *end;
    uint32_t off;
    uint4 a, b;
    __device__ __forceinline__ void start(const uint8_t *s, int rows, int ks, int row) {
        const long long byte = static_cast<long long>(row) * ks;
        at = row < rows ? s + (byte & ~15ll) : nullptr;
        end = s + static_cast<long long>(rows) * ks;
        off = static_cast<uint32_t>(byte) & 15u;
        a = at ? scale_chunk(at, end) : make_uint4(0u, 0u, 0u, 0u);
        b = at ? scale_chunk(at + 16, end) : make_uint4(0u, 0u, 0u, 0u);
    }
    // the bytes of stages i and i + 1; the chunk for stages i + 2 and i + 3 is asked for
    __device__ __forceinline__ uint4 next(int i, int ks, bool aligned) {
        uint4 v = a;
        if (!aligned || 8 * i + 16 > ks || !at) v = scale_window(a, b, off, at ? ks - 8 * i : 0);
        a = b;
        if (at && 8 * i + 32 < ks + 16) b = scale_chunk(at + 8 * i + 32, end);
        return v;
    }
};

// ------------------------------------------------------------------ the kernel

__global__ void __launch_bounds__(kThreads, 1)
    a4_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *ready = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *empty = ready + kStages, *acc_full = empty + kStages, *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    static_assert((2 * kStages + 4) * 8 + 4 <= 256, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int steps = (p.K + kStep - 1) / kStep;
    const int half = p.bn / 2;
    const int pairs = static_cast<int>(gridDim.x) / 2, first = static_cast<int>(blockIdx.x) / 2;

    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ready[i], 1 + 2 * kLoaders);   // codes of both CTAs, the loader warps of each
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t ready_l = dsmem_addr(smem_u32(ready), 0), acc_empty_l = dsmem_addr(smem_u32(acc_empty), 0);

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------ codes by TMA
            prefetch_tmap(&tm_x);
            prefetch_tmap(&tm_w);
            pdl_wait();
            Ring st;
            long long issued = 0;
            bool ok = true;
            for (int t = first; t < p.tiles && ok; t += pairs) {
                const int row = (t % p.tiles_m) * 2 * kRows + static_cast<int>(rank) * kRows;
                const int out = t / p.tiles_m * p.bn + static_cast<int>(rank) * half;
                for (int i = 0; i < steps; ++i) {
                    if (issued >= kStages && !mbar_wait(&empty[st.slot], st.phase ^ 1u)) { ok = false; break; }
                    if (leader) mbar_arrive_expect_tx(&ready[st.slot], 2 * (kABytes + half * (kStep / 2)));
                    tma_load_2d_pair(smem + st.slot * kABytes, &tm_x, ready_l + 8 * st.slot, i * (kStep / 8), row);
                    tma_load_2d_pair(smem + kOffB + st.slot * kBBytes, &tm_w, ready_l + 8 * st.slot, i * (kStep / 8), out);
                    ++issued;
                    st.advance(kStages);
                }
            }
            // leave no copy in flight: the last stages' MMAs, which consumed them, completed
            for (long long j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
                mbar_wait(&empty[j % kStages], static_cast<uint32_t>((j / kStages) & 1), false);
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------------------ MMA issue (converged warp)
            const bool issuer = elect_one();
            const uint32_t id0 = idesc_mxf4(2 * kRows, p.bn, 0), id2 = idesc_mxf4(2 * kRows, p.bn, 2);
            const bool two_groups = p.bn > 128;
            const uint64_t a_desc0 = umma_desc_sw128(smem_u32(smem)), b_desc0 = umma_desc_sw128(smem_u32(smem + kOffB));
            const uint64_t s_desc0 = desc_scales(smem_u32(smem + kOffS));
            Ring st, acc;
            int done = 0;
            bool ok = true;
            for (int t = first; t < p.tiles && ok; t += pairs, ++done) {
                if (done >= 2 && !mbar_wait_cluster(&acc_empty[acc.slot], acc.phase ^ 1u)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc.slot * kAccCols;
                for (int i = 0; i < steps; ++i) {
                    if (!mbar_wait_spin(&ready[st.slot], st.phase)) { ok = false; break; }
                    if (issuer) {
                        const uint64_t ad = a_desc0 + st.slot * (kABytes >> 4), bd = b_desc0 + st.slot * (kBBytes >> 4);
                        const uint64_t sd = s_desc0 + st.slot * (kSBytes >> 4);
                        const uint32_t sc = tmem + kScaleCol0 + st.slot * kScaleCols;   // x: 2 x 4 columns, W: 2 x 8
#pragma unroll
                        for (int kc = 0; kc < 2; ++kc) {
                            const uint64_t from = sd + kc * (3 * kChunkBytes >> 4);
                            copy_scales_pair(sc + 4 * kc, from);
                            copy_scales_pair(sc + 8 + 8 * kc, from + (kChunkBytes >> 4));
                            if (two_groups) copy_scales_pair(sc + 8 + 8 * kc + 4, from + 2 * (kChunkBytes >> 4));
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_mxf4_pair(d, ad + 2 * kk, bd + 2 * kk, kk & 1 ? id2 : id0, sc + 4 * (kk >> 1),
                                           sc + 8 + 8 * (kk >> 1), kk > 0 || i > 0);
                        umma_commit_pair(&empty[st.slot], 3);
                    }
                    st.advance(kStages);
                }
                if (ok && issuer) umma_commit_pair(&acc_full[acc.slot], 3);
                acc.advance(2);
            }
        }
    } else if (warp < 4 || warp > 11) {
        if (warp != 13) {
            // ------------------------------------------------------------ scales: groups `index` and index + 5
            const int index = warp < 4 ? warp - 2 : (warp == 12 ? 2 : warp - 11);
            const int ks = p.K / mx::kBlock, wgroups = (p.bn + 31) / 32;
            const bool aligned = ks % 16 == 0;
            pdl_wait();
            Ring st;
            long long issued = 0;
            bool ok = true;
            for (int t = first; t < p.tiles && ok; t += pairs) {
                const int row_x = (t % p.tiles_m) * 2 * kRows + static_cast<int>(rank) * kRows, row_w = t / p.tiles_m * p.bn;
                ScaleGroup g[kGroups / kLoaders];
#pragma unroll
                for (int q = 0; q < kGroups / kLoaders; ++q) {
                    const int n = index + q * kLoaders;
                    if (n < 4) g[q].start(p.xs, p.o.M, ks, row_x + 32 * n + lane);
                    else g[q].start(p.ws, n - 4 < wgroups ? p.o.J : 0, ks, row_w + 32 * (n - 4) + lane);
                }
                for (int i = 0; i < steps && ok; i += 2) {
                    uint4 v[kGroups / kLoaders];
#pragma unroll
                    for (int q = 0; q < kGroups / kLoaders; ++q) v[q] = g[q].next(i, ks, aligned);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (i + u >= steps) break;
                        if (issued >= kStages && !mbar_wait(&empty[st.slot], st.phase ^ 1u)) { ok = false; break; }
                        ++issued;
#pragma unroll
                        for (int q = 0; q < kGroups / kLoaders; ++q) {
                            // row 32 c + lane of 128: word c of 16 bytes `lane`
                            const int n = index + q * kLoaders, c = n < 4 ? n : n - 4;
                            const uint32_t dst = smem_u32(smem + kOffS) + st.slot * kSBytes +
                                                 (n < 4 ? 0 : (c < 4 ? kChunkBytes : 2 * kChunkBytes)) + lane * 16 + (c & 3) * 4;
                            sts32(dst, u == 0 ? v[q].x : v[q].z);
                            sts32(dst + 3 * kChunkBytes, u == 0 ? v[q].y : v[q].w);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(ready_l + 8 * st.slot);
                        st.advance(kStages);
                    }
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue: half of the columns a warp
        const int quarter = warp & 3, c0 = (warp - 4) / 4 * half;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        pdl_wait();
        Ring acc;
        for (int t = first; t < p.tiles; t += pairs) {
            const long long m = static_cast<long long>(t % p.tiles_m) * 2 * kRows + rank * kRows + quarter * 32 + lane;
            const int j0 = t / p.tiles_m * p.bn;
            if (!mbar_wait(&acc_full[acc.slot], acc.phase)) break;
            tc_fence_after();
            for (int c = c0; c < c0 + half; c += 32) {
                __syncwarp();                   // the loads are collective
                uint32_t r[32];
                tmem_ld32(tmem + lanes + acc.slot * kAccCols + c, r);
                tmem_ld_wait_regs(r);
                if (m < p.o.M && j0 + c < p.o.J) mxg::write_columns<mxg::kPlain>(p.o, m, j0 + c, r);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_l + 8 * acc.slot);
            acc.advance(2);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while its peer may still signal it
}

}  // namespace mx4
}  // namespace w4a16
