// mx_matvec.cuh - few rows of x (decode) times MXFP4 weights: y = x W^T, or silu(gate) up over rows
// interleaved in blocks of eight.
//
// Mathematics: the codes become BF16 with their scale applied, exactly, so that mma.sync m16n8k16 (codes
// as A: 16 weight rows x 16 k; x as B: 16 k x 8 rows of x) sums products in FP32 over all of K, each exact
// within FP32's normal range.
//
// Lane (g, t) = (lane / 4, lane % 4) owns block 4 c + t of rows g and g + 8 in the c-th group of 128 k:
// one 16-byte load and one scale byte a row, so a block's factor is one register.  A permutation of k
// that A and B share leaves the sums alone: a word's codes j and j + 4 lie 16 bits apart and become one
// BF16 pair by a mask, a multiplication by 2^12 + 2^6 (sign to bit 15, the others to bits 6-8), a mask
// and the factor; x pairs are matched to that.  x itself may be stored in 4 bits (its values are exact in
// BF16 too): its blocks are expanded like W's.
//
// Split: a CTA owns 16 weight rows and its warps contiguous runs of the groups; the warps' sums join in
// warp order through shared memory, so results repeat.  The codes of D groups are in flight a warp; x, which
// all CTAs of an SM read, is taken from its cache when it is needed (with x fetched ahead too, there are
// registers for two groups: 8 rows x 9728 x 2560 8.2 us, 7.6 so).  Every CTA is resident at once at a decode
// layer's sizes.
// Bound: one row x 9728 x 2560 (13 MB from HBM) takes 8.1 us where its bytes take 2.0: launch, the first
// loads, which wait for the preceding kernel, and the join are half of it, and the expanding keeps the
// integer pipe half busy (tensor pipe 10 %, DRAM 14 %).
#pragma once

#include "mx.cuh"

namespace w4a16 {
namespace mxv {

constexpr int kMaxM = 32;

struct Params {
    const uint16_t *x;        // bf16 [M, K], or
    const uint32_t *xq;       // codes [M, K/8] and
    const uint8_t *xs;        // scales [M, K/32]
    const uint32_t *wq;       // [N, K/8]
    const uint8_t *ws;        // [N, K/32]
    uint16_t *out;            // bf16 [M, N], or [M, N/2] (gated)
    int M, N, K;
    int gated;
};

// Codes j and j + 4 of a word -> BF16 pairs times the factor (`more`: a second one, 0 for none).
__device__ __forceinline__ void expand_pairs(uint32_t v, uint32_t f, uint32_t more, uint32_t (&r)[4]) {
    mx::expand8_apart(v, f, r);
    if (more) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = mx::mul_bf16x2(r[i], more);
    }
}

struct Codes {
    uint4 c[2];               // rows g and g + 8
    uint32_t e[2];
};

__device__ __forceinline__ void load_codes(Codes &st, const Params &p, int group, int row0, int g, int t) {
    const int blk = 4 * group + t, ks = p.K / mx::kBlock;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = row0 + g + 8 * h;
        const bool live = r < p.N && blk < ks;
        const long long at = static_cast<long long>(live ? r : 0) * ks + (live ? blk : 0);
        st.c[h] = make_uint4(0u, 0u, 0u, 0u);
        st.e[h] = 127u;
        if (live) {
            st.c[h] = ldg_v4(p.wq + 4 * at);
            st.e[h] = ldg_u8(p.ws + at);
        }
    }
}

// 32 values of x rows 8 nb + g, in BF16 or (X4) as a block of codes.
template <int NB, bool X4>
struct Rows {
    uint4 v[NB][X4 ? 1 : 4];
    uint32_t e[X4 ? NB : 1];
};
template <int NB, bool X4>
__device__ __forceinline__ void load_rows(Rows<NB, X4> &st, const Params &p, int group, int g, int t) {
    const int blk = 4 * group + t, ks = p.K / mx::kBlock;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int m = 8 * nb + g;
        const bool live = m < p.M && blk < ks;
        const long long at = static_cast<long long>(live ? m : 0) * ks + (live ? blk : 0);
        if constexpr (X4) {
            st.v[nb][0] = live ? ldg_v4(p.xq + 4 * at) : make_uint4(0u, 0u, 0u, 0u);
            st.e[nb] = live ? ldg_u8(p.xs + at) : 127u;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) st.v[nb][q] = live ? ldg_v4(p.x + mx::kBlock * at + 8 * q) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
    return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

template <int NB, bool X4>
__device__ __forceinline__ void multiply(const Codes &st, const Rows<NB, X4> &x, float (&acc)[NB][2][4]) {
    uint32_t f[2], more[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f[h] = mx::factor_of(min(st.e[h], mx::kOneFactor));
        more[h] = st.e[h] > mx::kOneFactor ? mx::second_factor_of(st.e[h]) : 0u;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t b[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if constexpr (X4) {                         // codes come in the same pairs
                const uint32_t e = x.e[nb];
                expand_pairs(word_of(x.v[nb][0], w), mx::factor_of(min(e, mx::kOneFactor)),
                             e > mx::kOneFactor ? mx::second_factor_of(e) : 0u, b[nb]);
            } else {
                const uint4 &v = x.v[nb][w];
                b[nb][0] = prmt(v.x, v.z, 0x5410u);     // k 0 and 4
                b[nb][1] = prmt(v.x, v.z, 0x7632u);     // 1 and 5
                b[nb][2] = prmt(v.y, v.w, 0x5410u);
                b[nb][3] = prmt(v.y, v.w, 0x7632u);
            }
        }
        uint32_t lo[4], hi[4];
        expand_pairs(word_of(st.c[0], w), f[0], more[0], lo);
        expand_pairs(word_of(st.c[1], w), f[1], more[1], hi);
        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            mma_bf16_16816(acc[nb][0], a0, b[nb][0], b[nb][1], acc[nb][0]);
            mma_bf16_16816(acc[nb][1], a1, b[nb][2], b[nb][3], acc[nb][1]);
        }
    }
}

template <int NB, int WARPS, int D, int CTAS, bool X4>
__global__ void __launch_bounds__(32 * WARPS, CTAS) matvec_kernel(const Params p) {
    __shared__ float red[WARPS][16][8 * NB + 1];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int row0 = static_cast<int>(blockIdx.x) * 16;
    const int G = (p.K + 127) / 128;
    const int ga = static_cast<int>(static_cast<long long>(warp) * G / WARPS);
    const int gb = static_cast<int>(static_cast<long long>(warp + 1) * G / WARPS);
    float acc[NB][2][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nb][0][i] = acc[nb][1][i] = 0.f;
    Codes st[D];
    Rows<NB, X4> x;
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (ga + j < gb) load_codes(st[j], p, ga + j, row0, g, t);
    for (int gi = ga; gi < gb; gi += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            const int group = gi + j;
            if (group >= gb) break;
            load_rows<NB, X4>(x, p, group, g, t);
            multiply<NB, X4>(st[j], x, acc);
            if (group + D < gb) load_codes(st[j], p, group + D, row0, g, t);
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float(&a)[2][4] = acc[nb];
        red[warp][g][8 * nb + 2 * t] = a[0][0] + a[1][0];
        red[warp][g][8 * nb + 2 * t + 1] = a[0][1] + a[1][1];
        red[warp][g + 8][8 * nb + 2 * t] = a[0][2] + a[1][2];
        red[warp][g + 8][8 * nb + 2 * t + 1] = a[0][3] + a[1][3];
    }
    __syncthreads();
    if (!p.gated) {
        for (int i = threadIdx.x; i < 16 * p.M; i += 32 * WARPS) {
            const int m = i / 16, r = i % 16, row = row0 + r;
            if (row >= p.N) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += red[w][r][m];
            p.out[static_cast<long long>(m) * p.N + row] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
    } else {
        for (int i = threadIdx.x; i < 8 * p.M; i += 32 * WARPS) {
            const int m = i / 8, r = i % 8, row = row0 / 2 + r;
            if (row >= p.N / 2) continue;
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                gate += red[w][r][m];
                up += red[w][r + 8][m];
            }
            p.out[static_cast<long long>(m) * (p.N / 2) + row] =
                __bfloat16_as_ushort(__float2bfloat16_rn(mx::gated(gate, up)));
        }
    }
}

}  // namespace mxv
}  // namespace w4a16
