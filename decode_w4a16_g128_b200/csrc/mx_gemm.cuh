// mx_gemm.cuh - tcgen05 product of BF16 rows with MXFP4 weights, by rows or by columns of W.
//
//   forward:  D[m, j] = sum_k x[m, k] W[j, k]        (j = n: outputs;  contraction over k)
//   backward: D[m, j] = sum_n dy[m, n] W[n, j]       (j = k: the input's gradient)
//
// Mathematics: a stored value code 2^(e - 127) has two significant bits, so it is exact in BF16 (the
// scale is applied before the product, no factor is left for the accumulator) and the tensor cores'
// products are exact in FP32; the sum over all of the contraction stays in tensor memory.
//
// A CTA pair (cta_group::2) computes 256 rows x BN outputs, K = 64 of the contraction a stage:
//   A  128 rows x 64 of x per CTA, by TMA, K-major, 128-byte swizzle;
//   B  each CTA expands its BN / 2 outputs' codes into BF16 in shared memory.  Forward: [output][64 k],
//      K-major.  Backward: the stored rows run along the outputs, so the tile is kept as stored,
//      [64 n][64 outputs] per group of 64 outputs, MN-major: the transposition is the descriptor's.
//      BN > 256 (backward) is a second MMA over the outputs behind the first 128 of each CTA.
// Accumulators fill tensor memory: two of BN <= 256 columns (the epilogue of a tile runs under the
// next tile's main loop), or one wider.  The grid is persistent; the host picks BN for the fewest
// column-rounds (see mx_entry.cuh).
//
// Roles (512 threads): warp 0 x by TMA, warp 1 MMA issue (leader) and tensor memory, warp 2 codes by
// TMA, warp 3 of the peer forwards "expanded" to the leader, warps 4-7 epilogue, warps 8-15 expand
// codes.  Barriers: ready[s] (leader; x bytes of both CTAs, the leader's two expanding warps, the
// peer's forwarder), empty[s] (both CTAs; the stage's MMAs completed), exp[s] (peer: its two
// expanding warps), w_full / w_empty (codes ring), acc_full / acc_empty (accumulators).
#pragma once

#include "mx.cuh"

namespace w4a16 {
namespace mxg {

constexpr int kThreads = 512;
constexpr int kRows = 128;               // x rows of a CTA
constexpr int kStep = 64;                // contraction of a stage
constexpr int kABytes = kRows * kStep * 2;
constexpr int kMaxStages = 8;
constexpr int kMaxWSlots = 8;
// Stages of a codes copy.  A copy costs the TMA unit time per row, whatever the row's length (a copy
// of 128 rows x 32 bytes a stage, beside x's 128 rows, held the whole pipeline to about 800 cycles
// a stage): forward rows are fetched 128 bytes at a time, K = 256, for the four teams' stages.
template <bool BACKWARD>
constexpr int kWSpan = BACKWARD ? 1 : 4;
constexpr int kDeqWarps = 8, kDeqThreads = 32 * kDeqWarps, kEpiWarps = 4;
constexpr int kTmemCols = 512;
constexpr int kMaxBN = 320;              // outputs of a pair (forward: 256)
constexpr int kBarBytes = 512;
constexpr int kSmemBudget = 227 * 1024;
constexpr int kTeams = 4, kTeamWarps = kDeqWarps / kTeams;   // expanding warps, see there

// Dynamic shared memory: stages x (A, B), codes ring, barriers, and slack for 1024-byte alignment.
__host__ __device__ constexpr int smem_bytes(int stages, int b_bytes, int w_slots, int w_bytes) {
    return stages * (kABytes + b_bytes) + w_slots * w_bytes + kBarBytes + 1024;
}

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
// rows of the contraction 1024 bytes apart (stride offset), groups of 64 outputs 8192 bytes apart
// (leading offset).
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t smem_addr) {
    uint64_t d = static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(8192 >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
constexpr uint32_t kIdescBMnMajor = 1u << 16;

// ------------------------------------------------------------------ codes to BF16

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A scale byte as up to two BF16 factors: a code's three low bits in BF16's lowest exponent bits
// and highest mantissa bit are its magnitude times 2^-126 (code 1 as a subnormal), so the factor is
// 2^(e - 1); above e = 128 that is beyond BF16 and the rest, 2^(e - 128), comes as a second one.
struct Factor {
    uint32_t f, more;          // pairs; more = 0: none
};
__device__ __forceinline__ Factor factor_of(uint32_t e) {
    Factor r;
    r.f = ((e < 128u ? e : 128u) + 126u) * 0x00800080u;
    r.more = 0;
    if (e > 128u) {
        r.more = e == mx::kScaleNan ? 0x7FC07FC0u : (e - 1u) * 0x00800080u;
    }
    return r;
}

// Eight codes, lowest k first -> four BF16 pairs, lowest k first.  Codes 2i and 2i + 1 go to the two
// halves of a register (the selector's sign-replicating bytes are zero there: every byte is below
// 128), one multiplication by 2^12 + 2^6 puts the sign bit to bit 15 and the others to bits 6-8.
__device__ __forceinline__ void expand8(uint32_t v, const Factor &s, uint32_t (&r)[4]) {
    const uint32_t lo = v & 0x0F0F0F0Fu, hi = (v >> 4) & 0x0F0F0F0Fu;
    r[0] = prmt(lo, hi, 0xC480u);
    r[1] = prmt(lo, hi, 0xD591u);
    r[2] = prmt(lo, hi, 0xE6A2u);
    r[3] = prmt(lo, hi, 0xF7B3u);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2((r[i] * 0x1040u) & 0x81C081C0u, s.f);
    if (s.more) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2(r[i], s.more);
    }
}

// ------------------------------------------------------------------ epilogue helpers

// Eight or sixteen values to BF16 at 16- or 32-byte boundaries.
__device__ __forceinline__ uint4 pack8(const float *v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store32(uint16_t *dst, uint4 a, uint4 b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
__device__ __forceinline__ void store_pair(uint16_t *dst, uint4 a, uint4 b, bool wide) {
    if (wide) {
        store32(dst, a, b);
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = a;
        reinterpret_cast<uint4 *>(dst)[1] = b;
    }
}

// Where a product's sums go: BF16 of them [M, J], silu(gate) up [M, J/2], or both gradients [M, J].
enum Epilogue { kPlain = 0, kGated = 1, kGatedBackward = 2 };
struct Output {
    uint16_t *out;
    const uint16_t *dh;       // bf16 [M, J/2] (kGatedBackward)
    int M, J;
    int epilogue;
    int wide;                 // 32-byte stores: rows and base are multiples of 32 bytes
};

// 32 accumulator columns of one row: outputs j .. j + 31 (j a multiple of 32 or, at the start of a
// second MMA's columns, still of 32).
__device__ __forceinline__ void write_columns(const Output &p, long long m, int j, const uint32_t (&r)[32]) {
    if (p.epilogue == kPlain) {
        uint16_t *dst = p.out + m * p.J + j;
        if ((p.J & 7) == 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[16 * q + i]);
                if (j + 16 * q + 8 < p.J) store_pair(dst + 16 * q, pack8(v), pack8(v + 8), p.wide);
                else if (j + 16 * q < p.J) *reinterpret_cast<uint4 *>(dst + 16 * q) = pack8(v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (j + i < p.J) dst[i] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[i])));
        }
        return;
    }
    // J is a multiple of 16: 8 gate columns and their 8 up columns
    const long long h = m * (p.J / 2) + j / 2;
    if (p.epilogue == kGated) {
        uint4 o[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float a[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                a[i] = mx::gated(__uint_as_float(r[16 * q + i]), __uint_as_float(r[16 * q + 8 + i]));
            o[q] = pack8(a);
        }
        if (j + 16 < p.J) store_pair(p.out + h, o[0], o[1], p.wide);
        else *reinterpret_cast<uint4 *>(p.out + h) = o[0];
        return;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (j + 16 * q >= p.J) break;
        const uint4 d = ldg_v4(p.dh + h + 8 * q);
        const float dh[8] = {bf16_lo_to_f32(d.x), bf16_hi_to_f32(d.x), bf16_lo_to_f32(d.y), bf16_hi_to_f32(d.y),
                             bf16_lo_to_f32(d.z), bf16_hi_to_f32(d.z), bf16_lo_to_f32(d.w), bf16_hi_to_f32(d.w)};
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mx::gated_backward(__uint_as_float(r[16 * q + i]), __uint_as_float(r[16 * q + 8 + i]), dh[i], a[i], b[i]);
        store_pair(p.out + m * p.J + j + 16 * q, pack8(a), pack8(b), p.wide);
    }
}

struct Params {
    Output o;                 // M rows, J outputs
    const uint8_t *ws;        // scales [N, K/32]
    int C;                    // contraction
    int ks;                   // scale bytes of a row of W (K / 32)
    int bn;                   // outputs of a pair
    int tiles_m, tiles;
    int stages;
    int b_bytes, w_bytes;     // B tile of a CTA and stage, codes of a copy
    int w_slots;              // codes ring
    int w_pitch;              // bytes of a codes tile row
    int w_swz_shift, w_swz_mask;   // its 16-byte chunks are XORed with (row >> shift) & mask
    int scales16;             // rows of scale bytes start on 16-byte boundaries
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

// ------------------------------------------------------------------ scale bytes of a team's stages

// Forward, stage i of team i % 4 with i % 8 < 4: what scale_bytes needs of row j for stages i and i + 4;
// 127 outside W, where the codes are filled with zeros.  One 16-byte load where rows of scale bytes
// are 16-byte aligned (every lane reads another row, so a load costs a cache line a lane whatever its
// width), else four bytes.  The words are kept as loaded and looked at two stages later: a look here
// would wait for the load.
__device__ __forceinline__ uint4 scale_words(const Params &p, int j, int i, bool live) {
    uint4 v = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (!live || j >= p.o.J) return v;
    const uint8_t *row = p.ws + static_cast<long long>(j) * p.ks;
    const int b = 2 * i;
    if (p.scales16) {
        if ((b & ~15) < p.ks) v = ldg_nc_v4(row + (b & ~15));
    } else {
        if (b < p.ks) v.x = __ldg(row + b);
        if (b + 1 < p.ks) v.y = __ldg(row + b + 1);
        if (b + 8 < p.ks) v.z = __ldg(row + b + 8);
        if (b + 9 < p.ks) v.w = __ldg(row + b + 9);
    }
    return v;
}

// The bytes of blocks 2i, 2i + 1 (stage i, bits 0-15) and 2i + 8, 2i + 9 (stage i + 4, bits 16-31).
__device__ __forceinline__ uint32_t scale_bytes(const Params &p, const uint4 &v, int team) {
    if (p.scales16) {
        const uint32_t lo = team < 2 ? v.x : v.y, hi = team < 2 ? v.z : v.w;
        return team & 1 ? prmt(lo, hi, 0x7632u) : prmt(lo, hi, 0x5410u);
    }
    return prmt(prmt(v.x, v.y, 0x0040u), prmt(v.z, v.w, 0x0040u), 0x5410u);
}

// Backward: the byte of row n, block b.
__device__ __forceinline__ uint32_t scale_by_column(const Params &p, int n, int b, bool live) {
    return live && n < p.C && b < p.ks ? __ldg(p.ws + static_cast<long long>(n) * p.ks + b) : 127u;
}

// ------------------------------------------------------------------ the kernel

template <bool BACKWARD>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int stages = p.stages;
    uint8_t *sa = smem, *sb = sa + stages * kABytes, *sw = sb + stages * p.b_bytes;
    uint64_t *ready = reinterpret_cast<uint64_t *>(sw + p.w_slots * p.w_bytes);
    uint64_t *empty = ready + kMaxStages, *expd = empty + kMaxStages;
    uint64_t *w_full = expd + kMaxStages, *w_empty = w_full + kMaxWSlots;
    uint64_t *acc_full = w_empty + kMaxWSlots, *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    static_assert((3 * kMaxStages + 2 * kMaxWSlots + 4) * 8 + 8 <= kBarBytes, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int steps = (p.C + kStep - 1) / kStep;
    const int half = p.bn / 2;                       // outputs that this CTA expands
    const int nacc = p.bn <= 256 ? 2 : 1;
    const int pairs = static_cast<int>(gridDim.x) / 2, first = static_cast<int>(blockIdx.x) / 2;

    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&ready[i], 1 + kTeamWarps + 1);
            mbar_init(&empty[i], 1);
            mbar_init(&expd[i], kTeamWarps);
        }
        for (int i = 0; i < kMaxWSlots; ++i) {
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], kWSpan<BACKWARD> * kTeamWarps);
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

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------------------- x by TMA
        prefetch_tmap(&tm_x);
        pdl_wait();
        Ring st;
        long long issued = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += pairs) {
            const int row = (t % p.tiles_m) * 2 * kRows + static_cast<int>(rank) * kRows;
            for (int i = 0; i < steps; ++i) {
                if (issued >= stages && !mbar_wait(&empty[st.slot], st.phase ^ 1u)) { ok = false; break; }
                if (leader) mbar_arrive_expect_tx(&ready[st.slot], 2 * kABytes);   // both CTAs' rows
                tma_load_2d_pair(sa + st.slot * kABytes, &tm_x, ready_l + 8 * st.slot, i * kStep, row);
                ++issued;
                st.advance(stages);
            }
        }
        // leave no copy in flight: the last stages' MMAs, which consumed them, completed
        for (long long j = issued > stages ? issued - stages : 0; j < issued; ++j)
            mbar_wait(&empty[j % stages], static_cast<uint32_t>((j / stages) & 1), false);
    } else if (warp == 2 && lane == 0) {
        // ---------------------------------------------------------------- codes by TMA
        prefetch_tmap(&tm_w);
        pdl_wait();
        const int slots = p.w_slots;
        Ring st;
        long long issued = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += pairs) {
            const int j0 = t / p.tiles_m * p.bn + static_cast<int>(rank) * half;
            for (int i = 0; i < steps; i += kWSpan<BACKWARD>) {
                if (issued >= slots && !mbar_wait(&w_empty[st.slot], st.phase ^ 1u)) { ok = false; break; }
                mbar_arrive_expect_tx(&w_full[st.slot], p.w_bytes);
                if constexpr (BACKWARD)
                    tma_load_2d(sw + st.slot * p.w_bytes, &tm_w, &w_full[st.slot], j0 / 8, i * kStep);
                else
                    tma_load_2d(sw + st.slot * p.w_bytes, &tm_w, &w_full[st.slot], i * (kStep / 8), j0);
                ++issued;
                st.advance(slots);
            }
        }
        for (long long j = issued > slots ? issued - slots : 0; j < issued; ++j)
            mbar_wait(&w_full[j % slots], static_cast<uint32_t>((j / slots) & 1), false);
    } else if (warp == 3 && lane == 0 && !leader) {
        // ---------------------------------------------------------------- "expanded", to the leader
        Ring st;
        for (int t = first; t < p.tiles; t += pairs) {
            bool ok = true;
            for (int i = 0; i < steps && ok; ++i) {
                ok = mbar_wait(&expd[st.slot], st.phase);
                if (ok) mbar_arrive_cluster(ready_l + 8 * st.slot);
                st.advance(stages);
            }
            if (!ok) break;
        }
    } else if (warp == 1 && leader) {
        // ---------------------------------------------------------------- MMA issue
        // The warp stays converged and one elected lane issues: with the loop in one lane's branch
        // the same instructions took 10 to 15 % longer (the descriptors are uniform registers, which
        // divergent code has to move there one lane at a time).
        const int n0 = p.bn < 256 ? p.bn : 256, n1 = p.bn - n0;
        const uint32_t major = BACKWARD ? kIdescBMnMajor : 0u;
        const uint32_t idesc0 = umma_idesc_bf16(2 * kRows, n0) | major, idesc1 = umma_idesc_bf16(2 * kRows, n1) | major;
        Ring st, acc;
        int done = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += pairs, ++done) {
            // the accumulator's previous tile has been read
            if (done >= nacc && !mbar_wait_cluster(&acc_empty[acc.slot], acc.phase ^ 1u)) break;
            tc_fence_after();
            const uint32_t d = tmem + acc.slot * 256;
            for (int i = 0; i < steps; ++i) {
                if (!mbar_wait_spin(&ready[st.slot], st.phase)) ok = false;
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                const uint32_t a0 = smem_u32(sa + st.slot * kABytes), b0 = smem_u32(sb + st.slot * p.b_bytes);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kStep / 16; ++kk) {
                        const uint64_t ad = umma_desc_sw128(a0 + 32 * kk);
                        const uint64_t bd = BACKWARD ? desc_mn_sw128(b0 + 2048 * kk) : umma_desc_sw128(b0 + 32 * kk);
                        umma_bf16_pair(d, ad, bd, idesc0, i > 0 || kk > 0);
                        if (BACKWARD && n1)      // the outputs behind this CTA's first 128: the third group of 64
                            umma_bf16_pair(d + 256, ad, desc_mn_sw128(b0 + 16384 + 2048 * kk), idesc1, i > 0 || kk > 0);
                    }
                    umma_commit_pair(&empty[st.slot], 3);
                }
                st.advance(stages);
            }
            if (ok && elect_one()) umma_commit_pair(&acc_full[acc.slot], 3);
            acc.advance(nacc);
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- codes to BF16
        // Four teams of two warps, each every fourth stage: expanding one stage is a chain of waits,
        // loads, conversions, stores and a fence that takes longer than the stage's MMAs, so four
        // stages are under way at once.
        const int team = (warp - 8) >> 1, id = threadIdx.x & 63;
        // Task q of a thread: block of 32 codes (row r, block b) of the codes tile.  Forward: rows of
        // neighbouring lanes, both blocks of a row; backward: the blocks of a row side by side.
        const int rows = BACKWARD ? kStep : half, blks = BACKWARD ? half / 32 : 2;
        const uint32_t sw0 = smem_u32(sw), sb0 = smem_u32(sb);
        constexpr int kMaxTasks = BACKWARD ? kMaxBN / 64 : 4;
        uint32_t src[kMaxTasks], dst[kMaxTasks];
        int trow[kMaxTasks], tblk[kMaxTasks];
#pragma unroll
        for (int q = 0; q < kMaxTasks; ++q) {
            int r, b;
            if constexpr (BACKWARD) {
                r = (id + 64 * q) / blks;
                b = (id + 64 * q) - r * blks;
            } else {
                r = id + 64 * (q >> 1);
                b = q & 1;
            }
            trow[q] = r < rows ? r : -1;
            tblk[q] = b;
            // forward: chunk 2 (i % 4) + b of a 128-byte row, i % 4 the team
            src[q] = sw0 + (BACKWARD ? r * p.w_pitch + ((b ^ ((r >> p.w_swz_shift) & p.w_swz_mask)) << 4)
                                     : r * 128 + (((2 * team + b) ^ (r & 7)) << 4));
            // forward: 64 k of an output, block b the half b; backward: 64 outputs of a row n, group b / 2
            dst[q] = sb0 + (BACKWARD ? (b >> 1) * 8192 + r * 128 : r * 128) + ((((b & 1) * 4) ^ (r & 7)) << 4);
        }
        pdl_wait();
        constexpr int kSpan = kWSpan<BACKWARD>;
        const int slots = p.w_slots;
        const int copies = (steps + kSpan - 1) / kSpan;        // of a tile
        long long base = 0, wbase = 0;                         // stages and copies of the tiles before
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += pairs, base += steps, wbase += copies) {
            const int j0 = t / p.tiles_m * p.bn + static_cast<int>(rank) * half;
            const int i0 = team;                               // this team's stages: team, team + 4, ...
            long long f = base + i0;
            int slot = static_cast<int>(f % stages);
            uint32_t phase = static_cast<uint32_t>(f / stages) & 1u;
            const long long wf = wbase + i0 / kSpan;
            int cslot = static_cast<int>(wf % slots);
            uint32_t cphase = static_cast<uint32_t>(wf / slots) & 1u;
            uint32_t cur[kMaxTasks], nxt[BACKWARD ? kMaxTasks : 1];
            uint4 words[BACKWARD ? 1 : kMaxTasks / 2];
            if constexpr (BACKWARD) {
#pragma unroll
                for (int q = 0; q < kMaxTasks; ++q) nxt[q] = scale_by_column(p, i0 * kStep + trow[q], j0 / 32 + tblk[q], trow[q] >= 0);
            } else {
#pragma unroll
                for (int q = 0; q < kMaxTasks; q += 2) words[q / 2] = scale_words(p, j0 + trow[q], i0, trow[q] >= 0);
            }
            for (int i = i0, it = 0; i < steps; i += 4, ++it, f += 4) {
                if constexpr (BACKWARD) {
#pragma unroll
                    for (int q = 0; q < kMaxTasks; ++q) {
                        cur[q] = nxt[q];
                        nxt[q] = scale_by_column(p, (i + 4) * kStep + trow[q], j0 / 32 + tblk[q], trow[q] >= 0);
                    }
                } else {
                    // four scale bytes of a row: this stage's two and the next one's of this team
#pragma unroll
                    for (int q = 0; q < kMaxTasks; q += 2) {
                        if (it & 1) {
                            cur[q] >>= 16;
                        } else {
                            cur[q] = scale_bytes(p, words[q / 2], team);
                            words[q / 2] = scale_words(p, j0 + trow[q], i + 8, trow[q] >= 0);
                        }
                    }
                }
                if (!mbar_wait(&w_full[cslot], cphase)) { ok = false; break; }
                uint4 c[kMaxTasks];
#pragma unroll
                for (int q = 0; q < kMaxTasks; ++q)
                    if (trow[q] >= 0) c[q] = lds128(src[q] + cslot * p.w_bytes);
                if (f >= stages && !mbar_wait(&empty[slot], phase ^ 1u)) { ok = false; break; }
                const uint32_t to = slot * p.b_bytes;
#pragma unroll
                for (int q = 0; q < kMaxTasks; ++q) {
                    if (trow[q] >= 0) {
                        const Factor fac = factor_of(BACKWARD ? cur[q] : (cur[q & ~1] >> (8 * (q & 1))) & 255u);
                        const uint32_t w[4] = {c[q].x, c[q].y, c[q].z, c[q].w};
#pragma unroll
                        for (int jj = 0; jj < 4; ++jj) {
                            uint32_t r[4];
                            expand8(w[jj], fac, r);
                            sts128((to + dst[q]) ^ (jj << 4), make_uint4(r[0], r[1], r[2], r[3]));
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&w_empty[cslot]);
                    if (leader) mbar_arrive(&ready[slot]);
                    else mbar_arrive(&expd[slot]);
                }
                slot += 4;
                if (slot >= stages) {
                    slot -= stages;
                    phase ^= 1u;
                }
                cslot += 4 / kSpan;
                if (cslot >= slots) {
                    cslot -= slots;
                    cphase ^= 1u;
                }
            }
            // a tile's last copy holds codes of up to four stages: the teams without one release it too
            if (kSpan > 1 && ok && steps % kSpan != 0 && team >= steps % kSpan) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_empty[cslot]);
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        pdl_wait();
        Ring acc;
        for (int t = first; t < p.tiles; t += pairs) {
            const long long m = static_cast<long long>(t % p.tiles_m) * 2 * kRows + rank * kRows + quarter * 32 + lane;
            const int j0 = t / p.tiles_m * p.bn;
            if (!mbar_wait(&acc_full[acc.slot], acc.phase)) break;
            tc_fence_after();
            for (int c = 0; c < p.bn; c += 32) {
                __syncwarp();                   // the loads are collective
                uint32_t r[32];
                tmem_ld32(tmem + lanes + acc.slot * 256 + c, r);
                tmem_ld_wait_regs(r);
                int j = j0 + c;                 // columns in order, but for the second MMA's
                if (BACKWARD && p.bn > 256) {
                    const int w = half - 128, cc = c - 256;
                    j = j0 + (c < 256 ? (c / 128) * half + c % 128 : cc / w * half + 128 + cc % w);
                }
                if (m < p.o.M && j < p.o.J) write_columns(p.o, m, j, r);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_l + 8 * acc.slot);
            acc.advance(nacc);
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

}  // namespace mxg
}  // namespace w4a16
