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
// Roles (384 threads): warp 0 codes by TMA, warp 1 MMA issue (leader) and tensor memory, warps 2 and 3
// scales of x and of W, warps 4-11 epilogue.
#pragma once

#include "mx_gemm.cuh"

namespace w4a16 {
namespace mx4 {

using mxg::elect_one;
using mxg::Ring;

constexpr int kThreads = 384;
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

// Bytes first .. first + 15 (blocks of K) of a stored row of ks scale bytes, 127 behind its end and
// for rows outside.  One 16-byte load where rows are 16-byte aligned; else five aligned words, shifted
// into place (the array starts on a 16-byte boundary; its last word may be cut off: read by bytes).
__device__ __forceinline__ uint32_t word_inside(const uint8_t *at, const uint8_t *end) {
    if (at + 4 <= end) return __ldg(reinterpret_cast<const uint32_t *>(at));
    uint32_t v = 0;
    for (int i = 0; i < 3; ++i)
        if (at + i < end) v |= static_cast<uint32_t>(__ldg(at + i)) << (8 * i);
    return v;
}
__device__ __forceinline__ uint4 scale16(const uint8_t *s, int rows, int ks, int row, int first, bool aligned) {
    const uint4 none = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (row >= rows || first >= ks) return none;
    const uint8_t *at = s + static_cast<long long>(row) * ks + first;
    if (aligned) return ldg_nc_v4(at);
    const uint8_t *end = s + static_cast<long long>(rows) * ks;
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 3u);
    uint32_t w[5], v[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = word_inside(at - off + 4 * i, end);
    const int valid = ks - first;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __funnelshift_r(w[i], w[i + 1], 8 * off);
        const int n = valid - 4 * i;                        // valid bytes of this word
        const uint32_t mask = n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
        v[i] = (v[i] & mask) | (0x7F7F7F7Fu & ~mask);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// A loader warp's share of every tile: scales of `groups` x 32 rows from row0(t), two stages at a time.
template <int GROUPS, typename Row0>
__device__ __forceinline__ void load_scales(const uint8_t *s, int rows, int K, int first, int step_t, int tiles, int steps,
                                            uint32_t dst0, uint64_t *empty, uint32_t ready_l, int lane, Row0 row0) {
    const int ks = K / mx::kBlock;
    const bool aligned = ks % 16 == 0;
    Ring st;
    long long issued = 0;
    for (int t = first; t < tiles; t += step_t) {
        const int r0 = row0(t) + lane;
        uint4 v[GROUPS];
#pragma unroll
        for (int c = 0; c < GROUPS; ++c) v[c] = scale16(s, rows, ks, r0 + 32 * c, 0, aligned);
        for (int i = 0; i < steps; i += 2) {
            uint4 cur[GROUPS];
#pragma unroll
            for (int c = 0; c < GROUPS; ++c) cur[c] = v[c];
#pragma unroll
            for (int c = 0; c < GROUPS; ++c) v[c] = scale16(s, rows, ks, r0 + 32 * c, 8 * (i + 2), aligned);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (i + u >= steps) break;
                if (issued >= kStages && !mbar_wait(&empty[st.slot], st.phase ^ 1u)) return;
                ++issued;
                const uint32_t dst = dst0 + st.slot * kSBytes + lane * 16;
#pragma unroll
                for (int kc = 0; kc < 2; ++kc)
#pragma unroll
                    for (int q = 0; q < (GROUPS + 3) / 4; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int g = 4 * q + c;
                            if (g < GROUPS) {
                                const uint4 &x = cur[g < GROUPS ? g : 0];
                                w[c] = u == 0 ? (kc == 0 ? x.x : x.y) : (kc == 0 ? x.z : x.w);
                            } else {
                                w[c] = 0x7F7F7F7Fu;
                            }
                        }
                        sts128(dst + (kc * 3 + q) * kChunkBytes, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(ready_l + 8 * st.slot);
                st.advance(kStages);
            }
        }
    }
}

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
            mbar_init(&ready[i], 1 + 2 * 2);   // codes of both CTAs, two loader warps each
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
            const uint32_t id0 = idesc_mxf4(2 * kRows, p.bn, 0), id2 = idesc_mxf4(2 * kRows, p.bn, 2);
            const int wgroups = p.bn > 128 ? 2 : 1;
            Ring st, acc;
            int done = 0;
            bool ok = true;
            for (int t = first; t < p.tiles && ok; t += pairs, ++done) {
                if (done >= 2 && !mbar_wait_cluster(&acc_empty[acc.slot], acc.phase ^ 1u)) ok = false;
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc.slot * kAccCols;
                for (int i = 0; i < steps; ++i) {
                    if (!mbar_wait_spin(&ready[st.slot], st.phase)) ok = false;
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                    const uint32_t a0 = smem_u32(smem + st.slot * kABytes), b0 = smem_u32(smem + kOffB + st.slot * kBBytes);
                    const uint32_t s0 = smem_u32(smem + kOffS + st.slot * kSBytes);
                    const uint32_t sc = tmem + kScaleCol0 + st.slot * kScaleCols;   // x: 2 x 4 columns, W: 2 x 8
                    if (elect_one()) {
#pragma unroll
                        for (int kc = 0; kc < 2; ++kc) {
                            copy_scales_pair(sc + 4 * kc, desc_scales(s0 + kc * 3 * kChunkBytes));
                            copy_scales_pair(sc + 8 + 8 * kc, desc_scales(s0 + (kc * 3 + 1) * kChunkBytes));
                            if (wgroups > 1)
                                copy_scales_pair(sc + 8 + 8 * kc + 4, desc_scales(s0 + (kc * 3 + 2) * kChunkBytes));
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_mxf4_pair(d, umma_desc_sw128(a0 + 32 * kk), umma_desc_sw128(b0 + 32 * kk), kk & 1 ? id2 : id0,
                                           sc + 4 * (kk >> 1), sc + 8 + 8 * (kk >> 1), i > 0 || kk > 0);
                        umma_commit_pair(&empty[st.slot], 3);
                    }
                    st.advance(kStages);
                }
                if (ok && elect_one()) umma_commit_pair(&acc_full[acc.slot], 3);
                acc.advance(2);
            }
        }
    } else if (warp == 2) {
        pdl_wait();
        load_scales<4>(p.xs, p.o.M, p.K, first, pairs, p.tiles, steps, smem_u32(smem + kOffS), empty, ready_l, lane,
                       [&](int t) { return (t % p.tiles_m) * 2 * kRows + static_cast<int>(rank) * kRows; });
    } else if (warp == 3) {
        pdl_wait();
        const auto row0 = [&](int t) { return t / p.tiles_m * p.bn; };
        const uint32_t dst = smem_u32(smem + kOffS) + kChunkBytes;
        if (p.bn > 128) load_scales<6>(p.ws, p.o.J, p.K, first, pairs, p.tiles, steps, dst, empty, ready_l, lane, row0);
        else load_scales<4>(p.ws, p.o.J, p.K, first, pairs, p.tiles, steps, dst, empty, ready_l, lane, row0);
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
