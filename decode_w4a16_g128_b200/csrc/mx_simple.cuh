// mx_simple.cuh - every MXFP4 product as one plain tiled kernel on the CUDA cores.
//
// D[m, j] = sum_c A[m, c] B[j, c] in FP32 over tiles of 64 x 64 outputs and 32 values of c, a 4 x 4
// patch of outputs a thread.  A is BF16 or MXFP4 rows; B is the stored weight W[N, K] by rows
// (j = n, c = k) or by columns (j = k, c = n, the input's gradient).  The epilogue writes BF16 sums,
// silu(gate) up over rows interleaved in blocks of eight, or the gradients of both.
#pragma once

#include "mx.cuh"

namespace w4a16 {
namespace mxs {

enum Epilogue { kPlain = 0, kGated = 1, kGatedBackward = 2 };

struct Params {
    const uint16_t *a;         // bf16 [M, C], or
    const uint32_t *aq;        // codes [M, C/8] and
    const uint8_t *as;         // scales [M, C/32]
    const uint32_t *wq;        // codes [N, K/8]
    const uint8_t *ws;         // scales [N, K/32]
    const uint16_t *dh;        // bf16 [M, J/2] (kGatedBackward)
    uint16_t *out;
    int M, J, C, K;            // rows, outputs, contraction, row length of W
    int epilogue;
};

constexpr int kTile = 64, kStep = 32, kThreads = 256;

__device__ __forceinline__ float stored(const uint32_t *wq, const uint8_t *ws, long long row, long long k, long long K) {
    return mx::code_f32(wq[(row * K + k) >> 3] >> (4 * (k & 7))) * mx::scale_f32(ws[(row * K + k) >> 5]);
}

template <bool A4, bool BACKWARD>
__global__ void __launch_bounds__(kThreads) product_kernel(const Params p) {
    __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1], sd[kTile][kTile + 1];
    pdl_launch_dependents();
    pdl_wait();
    const int m0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int c0 = 0; c0 < p.C; c0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int r = i / kStep, c = i % kStep;
            float a = 0.f;
            if (m0 + r < p.M && c0 + c < p.C) {
                if constexpr (A4) a = stored(p.aq, p.as, m0 + r, c0 + c, p.C);
                else a = bf16_to_f32(p.a[static_cast<long long>(m0 + r) * p.C + c0 + c]);
            }
            sa[c][r] = a;
            // by rows: j = r, c = k; by columns: j runs along the row of W
            const int j = BACKWARD ? i % kTile : r, cc = BACKWARD ? i / kTile : c;
            float b = 0.f;
            if (j0 + j < p.J && c0 + cc < p.C)
                b = BACKWARD ? stored(p.wq, p.ws, c0 + cc, j0 + j, p.K) : stored(p.wq, p.ws, j0 + j, c0 + cc, p.K);
            sb[cc][j] = b;
        }
        __syncthreads();
#pragma unroll 8
        for (int c = 0; c < kStep; ++c) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sa[c][4 * ty + i];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = sb[c][4 * tx + i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) sd[4 * ty + i][4 * tx + j] = acc[i][j];
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kTile; i += kThreads) {
        const int r = i / kTile, j = i % kTile, m = m0 + r, jj = j0 + j;
        if (m >= p.M || jj >= p.J) continue;
        if (p.epilogue == kPlain) {
            p.out[static_cast<long long>(m) * p.J + jj] = __bfloat16_as_ushort(__float2bfloat16_rn(sd[r][j]));
        } else if (j & 8) {
            continue;
        } else {
            const float g = sd[r][j], u = sd[r][j + 8];
            const long long h = static_cast<long long>(m) * (p.J / 2) + jj / 16 * 8 + (jj & 7);
            if (p.epilogue == kGated) {
                p.out[h] = __bfloat16_as_ushort(__float2bfloat16_rn(mx::gated(g, u)));
            } else {
                float dg, du;
                mx::gated_backward(g, u, bf16_to_f32(p.dh[h]), dg, du);
                uint16_t *o = p.out + static_cast<long long>(m) * p.J + jj;
                o[0] = __bfloat16_as_ushort(__float2bfloat16_rn(dg));
                o[8] = __bfloat16_as_ushort(__float2bfloat16_rn(du));
            }
        }
    }
}

}  // namespace mxs
}  // namespace w4a16
