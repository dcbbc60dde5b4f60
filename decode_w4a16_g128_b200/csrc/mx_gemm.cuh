// mx_gemm.cuh - tcgen05 product of BF16 rows with MXFP4 weights, by rows or by columns of W.
//
//   forward:  D[m, j] = sum_k x[m, k] W[j, k]        (j = n: outputs;  contraction over k)
//   backward: D[m, j] = sum_n dy[m, n] W[n, j]       (j = k: the input's gradient)
//
// Mathematics: a stored value code 2^(e - 127) has two significant bits, so it is exact in BF16 (the
// scale is applied before the product, no factor is left for the accumulator) and the tensor cores'
// products are exact in FP32 (within its normal range); the sum over all of the contraction stays in tensor
// memory.
//
// A CTA pair (cta_group::2) computes 256 rows x BN <= 256 outputs, K = 128 of the contraction a stage:
//   A  128 rows of x per CTA, by TMA, K-major, two tiles of 64 k with the 128-byte swizzle;
//   B  each CTA expands its BN / 2 outputs' codes into BF16 in shared memory.  Forward: [output][64 k]
//      twice, K-major.  Backward: the stored rows run along the outputs, so the tile is kept as stored,
//      [128 n][64 outputs] per group of 64 outputs, MN-major: the transposition is the descriptor's.
// Two accumulators of 256 columns fill tensor memory: the epilogue of a tile runs under the next
// tile's main loop.  The grid is persistent; the host picks BN for the fewest column-rounds (see
// mx_entry.cuh).  Tiles that leave SMs idle, all of them or those after the last whole round, are shared: S
// pairs (or CTAs) of a cluster of up to eight CTAs take a run of a tile's stages each, and their partial sums
// meet in shared memory over the cluster, added in split order.
//
// Roles (768 threads): warp 1 MMA issue (leader) and tensor memory, warps 0, 2-7 and 21 epilogue,
// twelve of warps 8-23 expand codes in three teams, and beside warp 1 on its scheduler one warp that
// copies codes, one that copies x, and the peer's that forwards "expanded" to the leader.  The ring has
// three stages, one a team.  Barriers: ready[s] (leader; x bytes of both CTAs, the leader's four
// expanding warps, the peer's forwarder), empty[s] (both CTAs; the stage's MMAs completed), expd[s] (peer:
// its four expanding warps), w_full[s] / w_empty[s] (codes), acc_full / acc_empty (accumulators).  No
// waiter is a whole ring behind what it waits for: a team's next stage is in the same slot, so it has
// waited for this one's MMAs, and the parities never alias.
//
// Bound, forward, 2048 x 9728 x 2560: 72.2 us (1.41 PFLOP/s; the tensor pipe is active 71 % of the time, the
// integer pipe 43 %, issue slots 47 %, DRAM 4 %).  What is left is the time between two stages' MMAs: with
// stages of K = 64, whose MMAs take less time than the instructions around a stage's waits do in a crowded
// SM, the same product took 84 us.  Backward, 2048 x 9728 x 2560: 73.4 us (1.39 PFLOP/s), of which the shared
// last tiles save 8.  Few rows (33 - 128 x 9728 x 2560): 13.3 us: a stage is as long as its codes take to
// expand, three at a time, each a chain of waits.
#pragma once

#include "mx.cuh"

namespace w4a16 {
namespace mxg {

constexpr int kThreads = 768;
constexpr int kRows = 128;               // x rows of a CTA
constexpr int kStep = 128;               // contraction of a stage
constexpr int kStages = 3;
constexpr int kABytes = kRows * kStep * 2;
constexpr int kEpiWarps = 8;
constexpr int kTeams = kStages, kTeamWarps = 4;   // expanding warps, see there
constexpr int kMaxCluster = 8;           // CTAs that share a tile
// Warps with w % 4 == 1 share the issuing warp's scheduler: light roles.
constexpr int kWarpMma = 1, kWarpCodes = 9, kWarpX = 13, kWarpForward = 17, kWarpEpi = 21;
constexpr int kTmemCols = 512;
constexpr int kMaxBN = 256;              // outputs of a pair
constexpr int kBarBytes = 256;
constexpr int kSmemBudget = 227 * 1024;

// Dynamic shared memory: stages of (A, B, codes), barriers, and slack for 1024-byte alignment.
// `ragged`: with the epilogue's staging (see write_ragged), which leaves room for 224 outputs.
constexpr int kMaxRaggedBN = 224;
__host__ __device__ constexpr int smem_bytes(int b_bytes, int w_bytes, bool ragged) {
    return kStages * (kABytes + b_bytes + w_bytes) + (ragged ? kEpiWarps * 32 * 80 : 0) + kBarBytes + 1024;
}
static_assert(smem_bytes(kMaxBN / 2 * kStep * 2, kMaxBN / 2 * kStep / 2, false) <= kSmemBudget &&
              smem_bytes(kMaxRaggedBN / 2 * kStep * 2, kMaxRaggedBN / 2 * kStep / 2, true) <= kSmemBudget,
              "shared memory budget");
// The S splits' partial sums of a CTA's columns (see there) fit the stages' A and B, S = 1 .. 8.
__host__ __device__ constexpr bool sums_fit(int bn, int ctas, int S) {
    return (S * ((bn / 32 + S - 1) / S)) * 32 * kRows * 4 <= kStages * (kABytes + bn / ctas * kStep * 2);
}
// Two of these kernels, or one and the other tensor-core kernels, never share an SM: each takes all of
// its tensor memory, and a CTA that waited for it might hold what the other needs.
static_assert(2 * smem_bytes(32 * kStep * 2, 32 * kStep / 2, false) > 228 * 1024, "one CTA an SM");

// ------------------------------------------------------------------ PTX

// One lane of a converged warp (the same one each time).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A[smem] . B[smem] of a CTA pair, issued by the leader.
__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Descriptor of an MN-major operand, 128-byte swizzle: rows of 64 contiguous outputs (128 bytes), 8
// rows of the contraction 1024 bytes apart (stride offset), groups of 64 outputs kGroupBytes apart
// (leading offset).
constexpr int kGroupBytes = kStep * 128;
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t smem_addr) {
    uint64_t d = static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(kGroupBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
constexpr uint32_t kIdescBMnMajor = 1u << 16;

// ------------------------------------------------------------------ epilogue helpers

// Eight or sixteen values to BF16 at 16- or 32-byte boundaries.
__device__ __forceinline__ uint4 pack8(const float *v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// Where a product's sums go: BF16 of them [M, J], silu(gate) up [M, J/2], or both gradients [M, J].
enum Epilogue { kPlain = 0, kGated = 1, kGatedBackward = 2 };
struct Output {
    uint16_t *out;
    const uint16_t *dh;       // bf16 [M, J/2] (kGatedBackward)
    int M, J;
    int wide;                 // 32-byte stores: rows and base are multiples of 32 bytes
};

// 32 accumulator columns of one row a lane: outputs j .. j + 31, j a multiple of 32, of row m.
template <int EPILOGUE>
__device__ __forceinline__ void write_columns(const Output &p, long long m, int j, const uint32_t (&r)[32]) {
    if constexpr (EPILOGUE == kPlain) {
        uint16_t *dst = p.out + m * p.J + j;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[16 * q + i]);
            if (j + 16 * q + 8 < p.J) mx::store_pair(dst + 16 * q, pack8(v), pack8(v + 8), p.wide);
            else if (j + 16 * q < p.J) *reinterpret_cast<uint4 *>(dst + 16 * q) = pack8(v);
        }
    } else if constexpr (EPILOGUE == kGated) {    // J is a multiple of 16: 8 gate columns and their 8 up columns
        uint16_t *dst = p.out + m * (p.J / 2) + j / 2;
        uint4 o[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float a[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                a[i] = mx::gated(__uint_as_float(r[16 * q + i]), __uint_as_float(r[16 * q + 8 + i]));
            o[q] = pack8(a);
        }
        if (j + 16 < p.J) mx::store_pair(dst, o[0], o[1], p.wide);
        else *reinterpret_cast<uint4 *>(dst) = o[0];
    } else {
        const uint16_t *src = p.dh + m * (p.J / 2) + j / 2;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (j + 16 * q >= p.J) break;
            const uint4 d = ldg_v4(src + 8 * q);
            const float dh[8] = {bf16_lo_to_f32(d.x), bf16_hi_to_f32(d.x), bf16_lo_to_f32(d.y), bf16_hi_to_f32(d.y),
                                 bf16_lo_to_f32(d.z), bf16_hi_to_f32(d.z), bf16_lo_to_f32(d.w), bf16_hi_to_f32(d.w)};
            float a[8], b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                mx::gated_backward(__uint_as_float(r[16 * q + i]), __uint_as_float(r[16 * q + 8 + i]), dh[i], a[i], b[i]);
            mx::store_pair(p.out + m * p.J + j + 16 * q, pack8(a), pack8(b), p.wide);
        }
    }
}

// The same for rows that do not start on 16-byte boundaries (J not a multiple of 8): the warp's 32 x 32
// values go through shared memory, so that a store writes 64 contiguous bytes of one row instead of
// two bytes of each of 32 rows (a 77 x 1001 product: 14.1 us with the latter).
constexpr int kStagePitch = 80, kStageBytes = 32 * kStagePitch;   // 16-byte rows of chunks on all banks
__device__ __forceinline__ void write_ragged(const Output &p, long long m0, int j, const uint32_t (&r)[32], uint32_t stage,
                                             int lane) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) sts128(stage + lane * kStagePitch + 16 * q, pack8(v + 8 * q));
    __syncwarp();
    const int rows = static_cast<int>(min(32ll, p.M - m0));
    uint16_t *dst = p.out + m0 * p.J + j + lane;
#pragma unroll 8
    for (int i = 0; i < rows; ++i, dst += p.J)
        if (j + lane < p.J) *dst = static_cast<uint16_t>(lds16(stage + i * kStagePitch + 2 * lane));
}

struct Params {
    Output o;                 // M rows, J outputs
    const uint8_t *ws;        // scales [N, K/32]
    int C;                    // contraction
    int ks;                   // scale bytes of a row of W (K / 32)
    int bn;                   // outputs of a pair
    int tiles_m, tiles;
    int full;                 // the first tiles, which one pair (or CTA) computes alone (kLast)
    int b_bytes, w_bytes;     // B tile and codes of a CTA and stage
    int x_bytes;              // of a CTA's rows of x in a stage: all 128, or (alone) the M there are
    int w_pitch;              // bytes of a codes tile row
    int w_swz_shift, w_swz_mask;   // its 16-byte chunks are XORed with (row >> shift) & mask
    int splits;               // pairs that share each of the others (a cluster of them)
};

struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void advance(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Limit of a wait for a whole tile: one of 2^31 values a row takes seconds.
__device__ __forceinline__ unsigned long long tile_limit_ns(int steps) {
    return kWaitTimeoutNs + 4000ull * static_cast<unsigned long long>(steps);
}

// ------------------------------------------------------------------ scale bytes

// Up to four scale bytes of a stored row from block `blk` on: the aligned words that hold them (the
// array starts on a 16-byte boundary), kept as loaded and looked at a stage later, since a look here
// would wait for the load.  The array's last word may be cut off: it is read by bytes then.
__device__ __forceinline__ uint32_t scale_word(const uint8_t *at, const uint8_t *end) {
    if (at + 4 <= end) return ldg_u32(at);
    uint32_t v = 0;
    for (int i = 0; i < 3; ++i)
        if (at + i < end) v |= ldg_u8(at + i) << (8 * i);
    return v;
}
__device__ __forceinline__ uint32_t scale_offset(int row, int blk, int ks) {
    return (static_cast<uint32_t>(row) * static_cast<uint32_t>(ks) + static_cast<uint32_t>(blk)) & 3u;
}
__device__ __forceinline__ uint2 load_scales(const uint8_t *ws, const uint8_t *end, bool live, int row, int blk, int blks,
                                             int ks) {
    uint2 v = make_uint2(0u, 0u);
    if (!live || blk >= ks) return v;
    const int off = static_cast<int>(scale_offset(row, blk, ks));
    const uint8_t *at = ws + (static_cast<long long>(row) * ks + blk - off);
    v.x = scale_word(at, end);
    if (off + blks > 4) v.y = scale_word(at + 4, end);
    return v;
}
// Those bytes; 127 behind the row's end, where the codes are zeros.
__device__ __forceinline__ uint32_t scales_of(uint2 v, int row, int blk, int ks) {
    uint32_t e = __funnelshift_r(v.x, v.y, 8 * scale_offset(row, blk, ks));
    const int left = ks - blk;
    if (left < 4) {
        const uint32_t mask = left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        e = (e & mask) | (0x7F7F7F7Fu & ~mask);
    }
    return e;
}

// A block of 32 codes -> 64 bytes of BF16 at `to`, the first of four swizzled 16-byte chunks.  Codes along
// the contraction keep their order, which is that of x; codes along the outputs (APART) stay in the order
// that costs least, and the epilogue renames the columns (2048 x 9728 x 2560: 83.8 us, 85.0 without).
template <bool APART>
__device__ __forceinline__ void expand_block(const uint4 &c, uint32_t to, uint32_t e) {
    const uint32_t f = mx::factor_of(min(e, mx::kOneFactor));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    if (e <= mx::kOneFactor) {
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            uint32_t v[4];
            if constexpr (APART) mx::expand8_apart(w[jj], f, v);
            else mx::expand8(w[jj], f, v);
            sts128(to ^ (jj << 4), make_uint4(v[0], v[1], v[2], v[3]));
        }
    } else {
        const uint32_t more = mx::second_factor_of(e);
#pragma unroll 1
        for (int jj = 0; jj < 4; ++jj) {
            uint32_t v[4];
            const uint32_t word = jj == 0 ? c.x : (jj == 1 ? c.y : (jj == 2 ? c.z : c.w));
            if constexpr (APART) mx::expand8_apart(word, f, v);
            else mx::expand8(word, f, v);
            sts128(to ^ (jj << 4), make_uint4(mx::mul_bf16x2(v[0], more), mx::mul_bf16x2(v[1], more), mx::mul_bf16x2(v[2], more),
                                              mx::mul_bf16x2(v[3], more)));
        }
    }
}

__device__ __forceinline__ void st_dsmem_v4(uint32_t cluster_addr, uint4 v) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// ------------------------------------------------------------------ the kernel

// Which tiles the pairs (or CTAs) of a cluster share.  (Kernels of their own: with the others' conditions
// in it, each was 1 to 4 % slower.)
enum Share { kNone = 0, kLast = 1, kAll = 2 };

template <bool BACKWARD, int EPILOGUE, bool PAIR, int SHARE>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sa = smem, *sb = sa + kStages * kABytes, *sw = sb + kStages * p.b_bytes;
    uint64_t *ready = reinterpret_cast<uint64_t *>(sw + kStages * p.w_bytes);   // kBarBytes, then the staging
    uint64_t *empty = ready + kStages, *expd = empty + kStages, *w_full = expd + kStages, *w_empty = w_full + kStages;
    uint64_t *acc_full = w_empty + kStages, *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    static_assert((5 * kStages + 4) * 8 + 8 <= kBarBytes, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kCtas = PAIR ? 2 : 1;              // of a tile (and split)
    const uint32_t cluster_rank = cluster_ctarank();       // kCtas split + rank in the pair
    const uint32_t rank = PAIR ? cluster_rank & 1u : 0u, lead = cluster_rank - rank;
    const bool leader = rank == 0;
    const int all_steps = (p.C + kStep - 1) / kStep, split = static_cast<int>(cluster_rank) / kCtas;
    const int half = p.bn / kCtas;                   // outputs that this CTA expands
    constexpr int kTileRows = kCtas * kRows;
    // Work of this pair (or CTA): tiles first, first + pairs, ... of those computed alone, all of their
    // stages, then this split's stages of the cluster's shared tile, if it has one.
    const int pairs = static_cast<int>(gridDim.x) / kCtas, first = static_cast<int>(blockIdx.x) / kCtas;
    constexpr bool SHARED = SHARE != kNone;
    const int full = SHARE == kNone ? p.tiles : (SHARE == kAll ? 0 : p.full);
    const int shared_tile = SHARED ? full + static_cast<int>(blockIdx.x) / (kCtas * p.splits) : p.tiles;
    struct Work {
        int tile, step0, steps;
    };
    const auto work = [&](int t, Work &w) {
        if (SHARE != kAll && t < full) {
            w = {t, 0, all_steps};
            return true;
        }
        if constexpr (!SHARED) return false;
        if (t >= full + pairs || shared_tile >= p.tiles) return false;
        w.tile = shared_tile;
        w.step0 = static_cast<int>(static_cast<long long>(split) * all_steps / p.splits);
        w.steps = static_cast<int>(static_cast<long long>(split + 1) * all_steps / p.splits) - w.step0;
        return true;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ready[i], 1 + kTeamWarps + (PAIR ? 1 : 0));
            mbar_init(&empty[i], 1);
            mbar_init(&expd[i], kTeamWarps);
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], kTeamWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kCtas * kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        if constexpr (PAIR) {
            tmem_alloc_pair(tmem_slot, kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, kTmemCols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (threadIdx.x == 0) pdl_launch_dependents();   // what starts early cannot take the tensor memory first
    const uint32_t tmem = *tmem_slot;
    const uint32_t ready_l = dsmem_addr(smem_u32(ready), lead), acc_empty_l = dsmem_addr(smem_u32(acc_empty), lead);
    const uint16_t pair_mask = static_cast<uint16_t>(3u << lead);

    // two epilogue warps for every quarter of the lanes, 32 columns in turn
    const bool epilogue = (warp < 8 && warp != kWarpMma) || warp == kWarpEpi;
    const int epi_set = warp >= 4 && warp < 8;
    if (warp == kWarpX && lane == 0) {
        // ---------------------------------------------------------------- x by TMA
        prefetch_tmap(&tm_x);
        pdl_wait();
        Ring st;
        long long issued = 0;
        bool ok = true;
        Work w;
        for (int t = first; ok && work(t, w); t += pairs) {
            const int row = (w.tile % p.tiles_m) * kTileRows + static_cast<int>(rank) * kRows;
            for (int i = w.step0; i < w.step0 + w.steps; ++i) {
                if (issued >= kStages && !mbar_wait(&empty[st.slot], st.phase ^ 1u)) { ok = false; break; }
                if (leader) mbar_arrive_expect_tx(&ready[st.slot], kCtas * p.x_bytes);   // both CTAs' rows
                uint8_t *dst = sa + st.slot * kABytes;
                if constexpr (PAIR) {
                    tma_load_2d_pair(dst, &tm_x, ready_l + 8 * st.slot, i * kStep, row);
                    tma_load_2d_pair(dst + kABytes / 2, &tm_x, ready_l + 8 * st.slot, i * kStep + 64, row);
                } else {
                    tma_load_2d(dst, &tm_x, &ready[st.slot], i * kStep, row);
                    tma_load_2d(dst + kABytes / 2, &tm_x, &ready[st.slot], i * kStep + 64, row);
                }
                ++issued;
                st.advance(kStages);
            }
        }
        // leave no copy in flight: the last stages' MMAs, which consumed them, completed
        for (long long j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
            mbar_wait(&empty[j % kStages], static_cast<uint32_t>((j / kStages) & 1), false);
    } else if (warp == kWarpCodes && lane == 0) {
        // ---------------------------------------------------------------- codes by TMA
        prefetch_tmap(&tm_w);
        pdl_wait();
        Ring st;
        long long issued = 0;
        bool ok = true;
        Work w;
        for (int t = first; ok && work(t, w); t += pairs) {
            const int j0 = w.tile / p.tiles_m * p.bn + static_cast<int>(rank) * half;
            for (int i = w.step0; i < w.step0 + w.steps; ++i) {
                if (issued >= kStages && !mbar_wait(&w_empty[st.slot], st.phase ^ 1u)) { ok = false; break; }
                mbar_arrive_expect_tx(&w_full[st.slot], p.w_bytes);
                if constexpr (BACKWARD)
                    tma_load_2d(sw + st.slot * p.w_bytes, &tm_w, &w_full[st.slot], j0 / 8, i * kStep);
                else
                    tma_load_2d(sw + st.slot * p.w_bytes, &tm_w, &w_full[st.slot], i * (kStep / 8), j0);
                ++issued;
                st.advance(kStages);
            }
        }
        for (long long j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
            mbar_wait(&w_full[j % kStages], static_cast<uint32_t>((j / kStages) & 1), false);
    } else if (PAIR && warp == kWarpForward && lane == 0 && !leader) {
        // ---------------------------------------------------------------- "expanded", to the leader
        // The arrival has the default (CTA) scope: the expanding warps' writes reached shared memory before
        // their own arrivals, and a cluster-scope release drains the SM's memory pipeline, about a
        // microsecond a stage.
        Ring st;
        bool ok = true;
        pdl_wait();
        Work w;
        for (int t = first; ok && work(t, w); t += pairs)
            for (int i = 0; i < w.steps && ok; ++i) {
                ok = mbar_wait(&expd[st.slot], st.phase);
                if (ok) mbar_arrive_cluster(ready_l + 8 * st.slot);
                st.advance(kStages);
            }
    } else if (warp == kWarpMma && leader) {
        // ---------------------------------------------------------------- MMA issue
        // The warp stays converged and one elected lane issues: with the loop in one lane's branch
        // the same instructions took 10 to 15 % longer (the descriptors are uniform registers, which
        // divergent code has to move there one lane at a time).  Between two stages' MMAs this warp
        // executes some dozens of instructions, and the tensor pipe idles for as long as they take:
        // no busy warp shares its scheduler.
        const bool issuer = elect_one();
        const uint32_t idesc = umma_idesc_bf16(kTileRows, p.bn) | (BACKWARD ? kIdescBMnMajor : 0u);
        const uint64_t a_desc0 = umma_desc_sw128(smem_u32(sa));
        const uint64_t b_desc0 = BACKWARD ? desc_mn_sw128(smem_u32(sb)) : umma_desc_sw128(smem_u32(sb));
        const int a_hop = kABytes >> 4, b_hop = p.b_bytes >> 4;
        // K = 16 further on, in descriptor units; the second 64 k of a K-major tile are its second half
        constexpr int kBHop = (BACKWARD ? 2048 : 32) >> 4;
        const int b_half = BACKWARD ? 4 * kBHop : p.b_bytes >> 5;
        Ring st, acc;
        int done = 0;
        bool ok = true;
        pdl_wait();
        Work w;
        for (int t = first; ok && work(t, w); t += pairs, ++done) {
            // the accumulator's previous tile has been read
            if (done >= 2 && !mbar_wait_cluster(&acc_empty[acc.slot], acc.phase ^ 1u)) break;
            tc_fence_after();
            const uint32_t d = tmem + acc.slot * 256;
            for (int i = 0; i < w.steps; ++i) {
                if (!mbar_wait_spin(&ready[st.slot], st.phase)) { ok = false; break; }
                if (issuer) {
                    const uint64_t ad = a_desc0 + st.slot * a_hop, bd = b_desc0 + st.slot * b_hop;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint64_t ak = ad + (kk >> 2) * (kABytes >> 5) + 2 * (kk & 3);
                        const uint64_t bk = bd + (kk >> 2) * b_half + kBHop * (kk & 3);
                        if constexpr (PAIR) umma_bf16_pair(d, ak, bk, idesc, kk > 0 || i > 0);
                        else umma_bf16(d, ak, bk, idesc, kk > 0 || i > 0);
                    }
                    if constexpr (PAIR) umma_commit_pair(&empty[st.slot], pair_mask);
                    else umma_commit(&empty[st.slot]);
                }
                st.advance(kStages);
            }
            if (ok && issuer) {
                if constexpr (PAIR) umma_commit_pair(&acc_full[acc.slot], pair_mask);
                else umma_commit(&acc_full[acc.slot]);
            }
            acc.advance(2);
        }
    } else if (warp >= 8 && (warp & 3) != 1) {
        // ---------------------------------------------------------------- codes to BF16
        // Three teams of four warps, one a stage of the ring: expanding one stage is a chain of waits,
        // loads, conversions, stores and a fence, so three stages are under way at once.  The warps on the
        // issuing warp's scheduler (warp % 4 == 1) take no part.
        const int index = (warp - 8) / 4 * 3 + (warp & 3) - ((warp & 3) > 1);    // 0 .. 11
        const int team = index >> 2, id = (index & 3) * 32 + lane;
        // A thread expands blocks of 32 codes of one row of the codes tile, an output's four (forward)
        // or a stored row's half / 32 (backward); forward tiles of 32 or 64 rows a CTA have four or two
        // threads a row, with every fourth or second block each.  Neighbouring lanes have neighbouring
        // rows, whose 16-byte chunks the swizzles of both tiles spread over the banks.
        const int blks = BACKWARD ? half / 32 : 4;
        const int share = BACKWARD ? 1 : (half == 32 ? 4 : (half == 64 ? 2 : 1));
        const int r = share > 1 ? id & (half - 1) : id, b0 = share > 1 ? id / half : 0;
        const bool live = BACKWARD || r < half;
        const uint32_t swz = (r >> p.w_swz_shift) & p.w_swz_mask;
        uint32_t src[4], dst[4];                               // of block b0 + q share; src = 0: none
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int b = b0 + q * share;
            src[q] = live && b < blks ? smem_u32(sw) + team * p.w_bytes + r * p.w_pitch + ((b ^ swz) << 4) : 0u;
            dst[q] = smem_u32(sb) + team * p.b_bytes + (b >> 1) * (BACKWARD ? kGroupBytes : p.b_bytes / 2) + r * 128 +
                     ((((b & 1) * 4) ^ (r & 7)) << 4);
        }
        // The codes' slot is released once they are in registers, so that its next load is under way while
        // they are expanded (us, before / after: alone, 40 rows x 19456 x 2560 24.7 / 23.2; backward, 2048 x
        // 9728 x 2560 82.9 / 81.4), but by forward pairs at the end (512 rows 27.1, early 27.4; 1024 rows
        // 39.0, 39.7).
        constexpr bool kEarly = BACKWARD || !PAIR;
        const int stored = BACKWARD ? p.C : p.o.J;             // rows of W
        const uint8_t *ws_end = p.ws + static_cast<long long>(stored) * p.ks;
        uint32_t phase = 0;
        bool filled = false, ok = true;
        int i = team;                                          // this team's next stage of the tile
        pdl_wait();
        Work w;
        for (int t = first; ok && work(t, w); t += pairs, i -= w.steps) {
            const int j0 = w.tile / p.tiles_m * p.bn + static_cast<int>(rank) * half;
            // row and first block of the scale bytes of stage i
            const auto row = [&](int i) { return BACKWARD ? (w.step0 + i) * kStep + r : j0 + r; };
            const auto blk = [&](int i) { return BACKWARD ? j0 / 32 : 4 * (w.step0 + i); };
            uint2 next = load_scales(p.ws, ws_end, live && row(i) < stored, row(i), blk(i), blks, p.ks);
            for (; i < w.steps; i += kTeams) {
                const uint32_t e = scales_of(next, row(i), blk(i), p.ks);
                next = load_scales(p.ws, ws_end, live && row(i + kTeams) < stored, row(i + kTeams), blk(i + kTeams), blks, p.ks);
                if (!mbar_wait_warp(&w_full[team], phase)) { ok = false; break; }
                uint4 c[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (kEarly) c[q].x = 0u;
                    if (src[q]) c[q] = lds128(src[q]);
                }
                if constexpr (kEarly) {
                    // The next load may overwrite the slot once lane 0 has arrived: behind every lane's loads,
                    // which __syncwarp orders before it (a vote alone orders no memory), and with the values
                    // in registers, for which the vote on a word of each waits.
                    const uint32_t seen = __ballot_sync(0xFFFFFFFFu, (c[0].x ^ c[1].x ^ c[2].x ^ c[3].x) & 1u);
                    __syncwarp();
                    if (lane == (seen == 0xFFFFFFFFu ? 31 : 0)) mbar_arrive(&w_empty[team]);
                }
                if (filled && !mbar_wait_warp(&empty[team], phase ^ 1u)) { ok = false; break; }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (src[q]) expand_block<BACKWARD>(c[q], dst[q], (e >> (8 * (b0 + q * share))) & 255u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (!kEarly) mbar_arrive(&w_empty[team]);
                    if (leader) mbar_arrive(&ready[team]);
                    else mbar_arrive(&expd[team]);
                }
                phase ^= 1u;
                filled = true;
            }
        }
    }

    const int quarter = warp & 3, chunks = p.bn / 32, S = SHARED ? p.splits : 1, own = (chunks + S - 1) / S;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16, row = quarter * 32 + lane;
    // Partial sums of a shared tile: 32 columns belong to split (column / 32) % S.  Every warp takes part
    // (six for each quarter of the rows), after its other work; the others' columns go to their split's
    // shared memory as [source][own columns / 32][4 columns][row] x 16 bytes, idle once the cluster's main
    // loops are over.
    const auto exchange = [&]() {
        __syncwarp();
        tc_fence_before();
        cluster_sync_all();
        tc_fence_after();
        const uint32_t sums = tmem + lanes + (first < full ? ((full - first + pairs - 1) / pairs & 1) * 256 : 0);
        for (int c = warp >> 2; c < chunks; c += kThreads / 128) {
            const int to = c % S;
            if (to == split) continue;
            uint32_t v[32];
            tmem_ld32(sums + 32 * c, v);
            tmem_ld_wait_regs(v);
            const uint32_t base = dsmem_addr(smem_u32(smem), kCtas * to + rank) + ((split * own + c / S) * 8 * kRows + row) * 16;
#pragma unroll
            for (int q = 0; q < 8; ++q) st_dsmem_v4(base + q * kRows * 16, make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
        }
        cluster_sync_all();
    };
    bool to_meet = SHARED && shared_tile < p.tiles;
    if (epilogue) {
        // ---------------------------------------------------------------- epilogue
        const uint32_t stage = smem_u32(ready) + kBarBytes + (epi_set * 4 + quarter) * kStageBytes;
        pdl_wait();
        Ring acc;
        Work w;
        for (int t = first; work(t, w); t += pairs) {
            const long long m = static_cast<long long>(w.tile % p.tiles_m) * kTileRows + rank * kRows + row;
            const int j0 = w.tile / p.tiles_m * p.bn;
            const bool shared = SHARE == kAll || (SHARED && t >= full);
            if (!mbar_wait_warp(&acc_full[acc.slot], acc.phase, tile_limit_ns(w.steps))) break;
            if constexpr (SHARED) {
                if (shared) {
                    exchange();
                    to_meet = false;
                }
            }
            tc_fence_after();
            const int every = shared ? S : 1, own_c = shared ? split : 0;
            for (int c = own_c + every * epi_set; c < chunks; c += 2 * every) {
                __syncwarp();                   // the loads are collective
                uint32_t v[32];
                tmem_ld32(tmem + lanes + acc.slot * 256 + 32 * c, v);
                tmem_ld_wait_regs(v);
                for (int s = 0; s < every; ++s) {   // the other splits' sums, in their order
                    if (s == own_c) continue;
                    const uint32_t from = smem_u32(smem) + ((s * own + c / S) * 8 * kRows + row) * 16;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint4 o = lds128(from + q * kRows * 16);
                        v[4 * q] = __float_as_uint(__uint_as_float(v[4 * q]) + __uint_as_float(o.x));
                        v[4 * q + 1] = __float_as_uint(__uint_as_float(v[4 * q + 1]) + __uint_as_float(o.y));
                        v[4 * q + 2] = __float_as_uint(__uint_as_float(v[4 * q + 2]) + __uint_as_float(o.z));
                        v[4 * q + 3] = __float_as_uint(__uint_as_float(v[4 * q + 3]) + __uint_as_float(o.w));
                    }
                }
                if constexpr (BACKWARD) {       // columns 2 i and 2 i + 1 of eight hold outputs i and i + 4
#pragma unroll
                    for (int g = 0; g < 32; g += 8) {
                        const uint32_t t[8] = {v[g], v[g + 2], v[g + 4], v[g + 6], v[g + 1], v[g + 3], v[g + 5], v[g + 7]};
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[g + i] = t[i];
                    }
                }
                const int j = j0 + 32 * c;
                if (j >= p.o.J) break;
                if (EPILOGUE == kPlain && (p.o.J & 7)) write_ragged(p.o, m - lane, j, v, stage, lane);
                else if (m < p.o.M) write_columns<EPILOGUE>(p.o, m, j, v);
            }
            if (shared) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_l + 8 * acc.slot);
            acc.advance(2);
        }
    }
    if constexpr (SHARED)
        if (to_meet) exchange();

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, kTmemCols);
        else tmem_dealloc(tmem, kTmemCols);
    }
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while its peer may still signal it
}

}  // namespace mxg
}  // namespace w4a16
