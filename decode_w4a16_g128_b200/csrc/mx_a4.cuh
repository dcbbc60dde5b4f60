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
// 32 bytes a row for four stages (a barrier's wait and arrival a stage took them longer than the MMAs),
// put them into that order in shared memory, and the issuing thread copies them with tcgen05.cp just
// before a stage's MMAs.
//
// Tensor memory: two accumulators of 192 columns (a tile's epilogue runs under the next one's main
// loop, which at K = 2560 takes only about 4000 cycles) and a scale buffer of 24 columns for each stage of
// the ring: a scale buffer is written again only after the barrier that says the stage's MMAs are done.
//
// Roles (512 threads): warp 0 codes by TMA, warp 1 MMA issue (leader) and tensor memory, warps 2, 3, 12,
// 14 and 15 scales (with two loader warps their instructions took longer than the MMAs), warps 4-11
// epilogue; warp 13 would share the issuing warp's scheduler and stays idle.
//
// Bound, 2048 x 9728 x 2560: 28.0 us (3.64 PFLOP/s; the tensor pipe is active 47 % of the time, no other
// unit more than 35 %); with the quantiser of x in front 32.2 us.  A stage's MMAs take 384 cycles and its turn of the issue loop 525 to 670.
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
constexpr int kSpan = 4, kSpans = 2;      // stages of a scale slot, slots
constexpr int kAccCols = 192, kScaleCol0 = 2 * kAccCols, kScaleCols = 24;
constexpr int kTmemCols = 512;
static_assert(kScaleCol0 + kStages * kScaleCols <= kTmemCols, "tensor memory budget");
constexpr int kEpiWarps = 8;
// Shared memory: stages of A, of B, scale slots, barriers, staging of ragged rows, alignment slack.
// (Keeping all of K of a CTA's rows of x there while it streams W alone was no faster.)
constexpr int kOffB = kStages * kABytes, kOffS = kOffB + kStages * kBBytes, kOffBar = kOffS + kSpans * kSpan * kSBytes;
constexpr int kBarBytes = 1024, kOffStage = kOffBar + kBarBytes;
constexpr int kStageBytes = 2 * 2048;      // of an epilogue warp: two tiles of 32 rows x 64 bytes
static_assert(kStageBytes >= mxg::kStageBytes && kOffStage % 1024 == 0, "staging");
constexpr int kSmemBytes = kOffStage + kEpiWarps * kStageBytes + 1024;
static_assert(kBBytes % 1024 == 0 && kSmemBytes <= 227 * 1024, "shared memory layout");

struct Params {
    mxg::Output o;            // M rows, J = N outputs
    const uint8_t *xs, *ws;   // scales [M, K/32], [N, K/32]
    int K, bn;
    int tiles_n, tiles;
    int x_bytes;              // of a CTA's rows of x in a stage
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

// Wait until at most N bulk stores of this thread still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
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

// 16 bytes of an array of scale bytes; behind its end nothing is read.
__device__ __forceinline__ uint4 scale_chunk(const uint8_t *at, const uint8_t *end) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; i < 16; ++i)
        if (at + i < end) w[i >> 2] |= ldg_u8(at + i) << (8 * (i & 3));
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

// A predicated 16-byte load into registers that hold something else if it is not made: no branch, after
// which the compiler would move the loaded value, and wait for it there.
__device__ __forceinline__ void load_chunk_if(bool p, const uint8_t *at, uint4 &v) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(at), "r"(p ? 1u : 0u));
}

// A row's 32 scale bytes of a span, as the two or three aligned chunks that hold them.
struct ScaleItem {
    uint4 a, b, c;
    const uint8_t *at;                          // of chunk a
    uint32_t off;
    int valid;                                  // bytes inside the row
    __device__ __forceinline__ void fetch(const uint8_t *s, const uint8_t *end, bool live, int ks, int row, int first,
                                          bool aligned) {
        const long long byte = live ? static_cast<long long>(row) * ks + first : 0;
        valid = live ? ks - first : 0;
        at = s + (byte & ~15ll);
        off = static_cast<uint32_t>(byte) & 15u;
        const int need = valid > 0 ? valid + static_cast<int>(off) : 0;
        a = b = c = make_uint4(0u, 0u, 0u, 0u);
        load_chunk_if(need > 0 && at + 16 <= end, at, a);
        load_chunk_if(need > 16 && at + 32 <= end, at + 16, b);
        if (!aligned) load_chunk_if(need > 32 && at + 48 <= end, at + 32, c);
    }
    // The array's last, incomplete chunk was not loaded: its bytes one by one.
    __device__ __forceinline__ void complete(const uint8_t *end) {
        if (valid <= 0 || at + 48 <= end) return;
        if (at + 16 > end) a = scale_chunk(at, end);
        if (at + 32 > end) b = scale_chunk(at + 16, end);
        c = scale_chunk(at + 32, end);
    }
    __device__ __forceinline__ uint4 window(int half, bool aligned) const {
        const uint4 &lo = half ? b : a, &hi = half ? c : b;
        if (aligned && valid >= 32) return lo;
        return scale_window(lo, hi, off, valid - 16 * half);
    }
};

// ------------------------------------------------------------------ the kernel

__global__ void __launch_bounds__(kThreads, 1)
    a4_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
              const __grid_constant__ CUtensorMap tm_y, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sb = smem + kOffB, *ss = smem + kOffS;
    uint64_t *ready = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *empty = ready + kStages, *s_full = empty + kStages, *s_empty = s_full + kSpans;
    uint64_t *acc_full = s_empty + kSpans, *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    static_assert(kSpan == 4, "two turns of the issue loop");
    static_assert((2 * kStages + 2 * kSpans + 4) * 8 + 4 <= kBarBytes, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int steps = (p.K + kStep - 1) / kStep;
    const int half = p.bn / 2;
    // tiles of this pair, neighbours along the outputs: tile t has rows t / tiles_n
    const long long pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int t0 = static_cast<int>(pair * p.tiles / pairs), t1 = static_cast<int>((pair + 1) * p.tiles / pairs);
    const auto row_of = [&](int t) { return t / p.tiles_n * 2 * kRows + static_cast<int>(rank) * kRows; };
    const auto out_of = [&](int t) { return t % p.tiles_n * p.bn; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ready[i], 1);           // codes of both CTAs
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kSpans; ++i) {
            mbar_init(&s_full[i], 2 * kLoaders);   // the loader warps of both CTAs
            mbar_init(&s_empty[i], 1);
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
    if (threadIdx.x == 0) pdl_launch_dependents();   // what starts early cannot take the tensor memory first
    const uint32_t tmem = *tmem_slot;
    const uint32_t ready_l = dsmem_addr(smem_u32(ready), 0), acc_empty_l = dsmem_addr(smem_u32(acc_empty), 0);
    const uint32_t s_full_l = dsmem_addr(smem_u32(s_full), 0);

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------ codes by TMA
            prefetch_tmap(&tm_x);
            prefetch_tmap(&tm_w);
            pdl_wait();
            Ring st;
            long long issued = 0;
            bool ok = true;
            for (int t = t0; t < t1 && ok; ++t) {
                const int row = row_of(t), out = out_of(t) + static_cast<int>(rank) * half;
                for (int i = 0; i < steps; ++i) {
                    if (issued >= kStages && !mbar_wait(&empty[st.slot], st.phase ^ 1u)) { ok = false; break; }
                    // rows of x that there are none of are not loaded: theirs are sums that no one reads
                    if (leader)
                        mbar_arrive_expect_tx(&ready[st.slot], (row + kRows < p.o.M ? 2 : 1) * p.x_bytes + half * kStep);
                    if (row < p.o.M) tma_load_2d_pair(smem + st.slot * kABytes, &tm_x, ready_l + 8 * st.slot, i * (kStep / 8), row);
                    tma_load_2d_pair(sb + st.slot * kBBytes, &tm_w, ready_l + 8 * st.slot, i * (kStep / 8), out);
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
            const uint64_t a_desc0 = umma_desc_sw128(smem_u32(smem)), b_desc0 = umma_desc_sw128(smem_u32(sb));
            const uint64_t s_desc0 = desc_scales(smem_u32(ss));
            // Two stages a turn: what surrounds a stage's MMAs, waits foremost, takes this warp nearly as long
            // as the MMAs take the tensor cores.
            const auto issue = [&](uint32_t d, int slot, int scale_stage, bool first) {
                const uint64_t ad = a_desc0 + slot * (kABytes >> 4), bd = b_desc0 + slot * (kBBytes >> 4);
                const uint64_t sd = s_desc0 + scale_stage * (kSBytes >> 4);
                const uint32_t sc = tmem + kScaleCol0 + slot * kScaleCols;   // x: 2 x 4 columns, W: 2 x 8
#pragma unroll
                for (int kc = 0; kc < 2; ++kc) {
                    const uint64_t from = sd + kc * (3 * kChunkBytes >> 4);
                    copy_scales_pair(sc + 4 * kc, from);
                    copy_scales_pair(sc + 8 + 8 * kc, from + (kChunkBytes >> 4));
                    if (two_groups) copy_scales_pair(sc + 8 + 8 * kc + 4, from + 2 * (kChunkBytes >> 4));
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_mxf4_pair(d, ad + 2 * kk, bd + 2 * kk, kk & 1 ? id2 : id0, sc + 4 * (kk >> 1), sc + 8 + 8 * (kk >> 1),
                                   kk > 0 || !first);
                umma_commit_pair(&empty[slot], 3);
            };
            Ring st, sp, acc;
            int done = 0;
            bool ok = true;
            pdl_wait();
            for (int t = t0; t < t1 && ok; ++t, ++done) {
                if (done >= 2 && !mbar_wait_cluster(&acc_empty[acc.slot], acc.phase ^ 1u)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc.slot * kAccCols;
                for (int i = 0; i < steps; i += 2) {
                    const bool two = i + 1 < steps, last = (i & 2) || i + 2 >= steps;      // of its scale slot
                    Ring st1 = st;
                    st1.advance(kStages);
                    if (!(i & 2) && !mbar_wait_spin(&s_full[sp.slot], sp.phase)) { ok = false; break; }
                    const bool now0 = mbar_test_wait(&ready[st.slot], st.phase), now1 = !two || mbar_test_wait(&ready[st1.slot], st1.phase);
                    if (!now0 && !mbar_wait_spin(&ready[st.slot], st.phase)) { ok = false; break; }
                    if (issuer) issue(d, st.slot, sp.slot * kSpan + (i & 2), i == 0);
                    if (two) {
                        if (!now1 && !mbar_wait_spin(&ready[st1.slot], st1.phase)) { ok = false; break; }
                        if (issuer) issue(d, st1.slot, sp.slot * kSpan + (i & 2) + 1, false);
                        st1.advance(kStages);
                    }
                    st = st1;
                    if (last) {
                        if (issuer) umma_commit_pair(&s_empty[sp.slot], 3);
                        sp.advance(kSpans);
                    }
                }
                if (ok && issuer) umma_commit_pair(&acc_full[acc.slot], 3);
                acc.advance(2);
            }
        }
    } else if (warp < 4 || warp > 11) {
        if (warp != 13) {
            // ------------------------------------------------------------ scales
            // This warp's groups of 32 rows, a row a lane: `index` and index + 5.  An item is a span of
            // four stages of a tile; items are fetched two ahead, over the tiles' borders too.
            const int index = warp < 4 ? warp - 2 : (warp == 12 ? 2 : warp - 11);
            const int ks = p.K / mx::kBlock, wgroups = (p.bn + 31) / 32, spans = (steps + kSpan - 1) / kSpan;
            const bool aligned = ks % 16 == 0;
            constexpr int kOf = kGroups / kLoaders;
            const uint8_t *xs_end = p.xs + static_cast<long long>(p.o.M) * ks, *ws_end = p.ws + static_cast<long long>(p.o.J) * ks;
            const auto fetch = [&](ScaleItem(&v)[kOf], int t, int span) {
                if (t >= t1) return;
#pragma unroll
                for (int q = 0; q < kOf; ++q) {
                    const int n = index + q * kLoaders;
                    const int row = n < 4 ? row_of(t) + 32 * n + lane : out_of(t) + 32 * (n - 4) + lane;
                    v[q].fetch(n < 4 ? p.xs : p.ws, n < 4 ? xs_end : ws_end, n < 4 ? row < p.o.M : n - 4 < wgroups && row < p.o.J, ks,
                               row, 32 * span, aligned);
                }
            };
            const auto put = [&](ScaleItem(&v)[kOf], int slot) {
#pragma unroll
                for (int q = 0; q < kOf; ++q) {
                    v[q].complete(index + q * kLoaders < 4 ? xs_end : ws_end);
                    // row 32 c + lane of 128: word c of 16 bytes `lane`
                    const int n = index + q * kLoaders, c = n < 4 ? n : n - 4;
                    const uint32_t dst = smem_u32(ss) + slot * kSpan * kSBytes +
                                         (n < 4 ? 0 : (c < 4 ? kChunkBytes : 2 * kChunkBytes)) + lane * 16 + (c & 3) * 4;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 w = v[q].window(h, aligned);      // stages 2 h and 2 h + 1
                        sts32(dst + 2 * h * kSBytes, w.x);
                        sts32(dst + 2 * h * kSBytes + 3 * kChunkBytes, w.y);
                        sts32(dst + (2 * h + 1) * kSBytes, w.z);
                        sts32(dst + (2 * h + 1) * kSBytes + 3 * kChunkBytes, w.w);
                    }
                }
            };
            pdl_wait();
            ScaleItem item[2][kOf];
            int t = t0, span = 0;                       // of the item to fetch next
            const auto step = [&]() {
                if (++span == spans) {
                    span = 0;
                    ++t;
                }
            };
            fetch(item[0], t, span);
            step();
            fetch(item[1], t, span);
            step();
            Ring sp;
            const long long items = static_cast<long long>(t1 - t0) * spans;
            bool ok = true;
            for (long long n = 0; n < items && ok; n += 2) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (n + u >= items) break;
                    if (n + u >= kSpans && !mbar_wait_warp(&s_empty[sp.slot], sp.phase ^ 1u)) { ok = false; break; }
                    put(item[u], sp.slot);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(s_full_l + 8 * sp.slot);
                    sp.advance(kSpans);
                    fetch(item[u], t, span);
                    step();
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue: half of the columns a warp
        const int quarter = warp & 3, c0 = (warp - 4) / 4 * half;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        pdl_wait();
        Ring acc;
        // A warp's tile of 32 rows x 32 outputs leaves by TMA from shared memory (two in flight a warp):
        // stores of a row a lane occupy the load/store unit for a cache line a lane, which delayed the
        // issuing warp's barrier tests.  Rows that do not start on 16-byte boundaries: write_ragged.
        uint8_t *tile = smem + kOffStage + (warp - 4) * kStageBytes;
        const bool ragged = p.o.J & 7;
        int buffer = 0;
        for (int t = t0; t < t1; ++t) {
            const int m0 = row_of(t) + quarter * 32, j0 = out_of(t);
            if (!mbar_wait_warp(&acc_full[acc.slot], acc.phase, mxg::tile_limit_ns(steps))) break;
            tc_fence_after();
            for (int c = c0; c < c0 + half; c += 32) {
                __syncwarp();                   // the loads are collective
                uint32_t r[32];
                tmem_ld32(tmem + lanes + acc.slot * kAccCols + c, r);
                tmem_ld_wait_regs(r);
                const int j = j0 + c;
                if (j >= p.o.J || m0 >= p.o.M) break;
                if (ragged) {
                    mxg::write_ragged(p.o, m0, j, r, smem_u32(tile), lane);
                    continue;
                }
                if (lane == 0) bulk_wait_read<1>();       // the copy before the last has read its buffer
                __syncwarp();
                const uint32_t to = smem_u32(tile) + buffer * 2048 + lane * 64;
                float v[32];
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(r[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) sts128(to + ((q ^ ((lane >> 1) & 3)) << 4), mxg::pack8(v + 8 * q));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&tm_y, tile + buffer * 2048, j, m0);
                    bulk_commit_group();
                }
                buffer ^= 1;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_l + 8 * acc.slot);
            acc.advance(2);
        }
        if (lane == 0) bulk_wait_all();         // written, and shared memory released
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
