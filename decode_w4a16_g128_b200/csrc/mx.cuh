// mx.cuh - the microscaled 4-bit format (MXFP4): conversion helpers, the quantiser and its inverse.
//
// A row of K values is cut into blocks of 32; a block holds one scale byte e (the factor
// 2^(e - 127); 255 marks a block that is not a number) and 32 codes of 4 bits: sign, two exponent
// bits, one mantissa bit, standing for 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.  Eight codes a
// word, the lowest k in the lowest bits, so codes are uint32 [rows, K/8], scales uint8 [rows, K/32].
//
// Codes and scales may come from the quantiser, which releases the next kernel at once: that kernel begins
// before they are written, perhaps on an SM whose cache still holds older ones.  So these kernels read all
// of their inputs behind pdl_wait(), by plain loads or TMA; the non-coherent path would need data that do
// not change from a kernel's beginning on.
#pragma once

#include "ptx.cuh"

namespace w4a16 {
namespace mx {

constexpr int kBlock = 32;              // values of one scale
constexpr uint32_t kScaleNan = 255;     // scale byte of a block that is not a number

// The factor 2^(e - 127) of a scale byte, in FP32 (e = 0 is the subnormal 2^-127).
__device__ __forceinline__ float scale_f32(uint32_t e) {
    const uint32_t b = e == 0 ? 0x00400000u : (e == kScaleNan ? 0x7FC00000u : e << 23);
    return __uint_as_float(b);
}

// Code -> value in FP32: exponent and mantissa bits moved under an exponent that is 126 too low
// (code 1, the format's subnormal, lands on FP32's own subnormals), then times 2^126: exact.
__device__ __forceinline__ float code_f32(uint32_t c) {
    return __uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * __uint_as_float(253u << 23);
}

// ------------------------------------------------------------------ codes to BF16

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A scale byte as BF16 factors: a code's three low bits in BF16's lowest exponent bits and highest
// mantissa bit are its magnitude times 2^-126 (code 1 as a subnormal), so the factor is 2^(e - 1).
// Above e = 128 that is beyond BF16: there the factor is 2^127, and the rest, 2^(e - 128) or NaN, a
// second one.
constexpr uint32_t kOneFactor = 128;       // largest scale byte with one factor
__device__ __forceinline__ uint32_t factor_of(uint32_t e) { return e * 0x00800080u + 126u * 0x00800080u; }
__device__ __forceinline__ uint32_t second_factor_of(uint32_t e) {
    return e == kScaleNan ? 0x7FC07FC0u : (e - 1u) * 0x00800080u;
}

// Eight codes, lowest k first -> four BF16 pairs, lowest k first, times the factor.  Codes 2i and 2i + 1
// go to the two halves of a register (the selector's sign-replicating bytes are zero there: every byte
// is below 128), one multiplication by 2^12 + 2^6 puts the sign bit to bit 15 and the others to bits 6-8.
__device__ __forceinline__ void expand8(uint32_t v, uint32_t f, uint32_t (&r)[4]) {
    const uint32_t lo = v & 0x0F0F0F0Fu, hi = (v >> 4) & 0x0F0F0F0Fu;
    r[0] = prmt(lo, hi, 0xC480u);
    r[1] = prmt(lo, hi, 0xD591u);
    r[2] = prmt(lo, hi, 0xE6A2u);
    r[3] = prmt(lo, hi, 0xF7B3u);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2((r[i] * 0x1040u) & 0x81C081C0u, f);
}

// The same, codes i and i + 4 as pair i: they lie 16 bits apart already, which saves the selections.
__device__ __forceinline__ void expand8_apart(uint32_t v, uint32_t f, uint32_t (&r)[4]) {
    const uint32_t u = v >> 8;
    r[0] = (v & 0x000F000Fu) * 0x1040u;
    r[1] = (v & 0x00F000F0u) * 0x0104u;
    r[2] = (u & 0x000F000Fu) * 0x1040u;
    r[3] = (u & 0x00F000F0u) * 0x0104u;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2(r[i] & 0x81C081C0u, f);
}

// ------------------------------------------------------------------ stores of 32 bytes

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

// ------------------------------------------------------------------ quantiser
//
// Per block: top = the largest magnitude, e = max(0, floor(log2 top) - 2 + 127), so that top lands in
// [4, 8); code = v 2^(127 - e) rounded to the nearest value, ties to even, above 6 down to 6.  The
// factor is a power of two and every input that a code other than 0 can come from stays exact under
// it, so cvt.rn.satfinite.e2m1x2 rounds the true quotient once: the result is the same bit for bit
// as a sequential CPU computation.  A block that holds an infinity or a NaN becomes e = 255, codes 0.
//
// Bound: HBM (4 or 2 bytes read and 0.53 written a value).  Blocks lie back to back over rows, so the
// kernel is one-dimensional: four lanes a block, eight values a lane, the maximum in two shuffles; a
// warp's eight code words of a step leave as 128 contiguous bytes.

constexpr int kQThreads = 256;
constexpr int kQUnroll = 4;

__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *w, long long word, float (&v)[8]) {
    if constexpr (BF16) {
        const uint4 a = ldg_v4(static_cast<const uint4 *>(w) + word);
        v[0] = bf16_lo_to_f32(a.x); v[1] = bf16_hi_to_f32(a.x);
        v[2] = bf16_lo_to_f32(a.y); v[3] = bf16_hi_to_f32(a.y);
        v[4] = bf16_lo_to_f32(a.z); v[5] = bf16_hi_to_f32(a.z);
        v[6] = bf16_lo_to_f32(a.w); v[7] = bf16_hi_to_f32(a.w);
    } else {
        const uint4 *p = static_cast<const uint4 *>(w) + 2 * word;
        const uint4 a = ldg_v4(p), b = ldg_v4(p + 1);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    }
}

// words: code words in all (a multiple of 4).
template <bool BF16>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const void *w, uint32_t *wq, uint8_t *scales,
                                                             long long words) {
    pdl_launch_dependents();
    pdl_wait();
    const long long stride = static_cast<long long>(gridDim.x) * kQThreads * kQUnroll;
    for (long long base = (static_cast<long long>(blockIdx.x) * kQUnroll) * kQThreads + threadIdx.x;
         base - threadIdx.x < words; base += stride) {
        float v[kQUnroll][8];
#pragma unroll
        for (int u = 0; u < kQUnroll; ++u) {
            const long long i = base + u * kQThreads;
            if (i < words) {
                load8<BF16>(w, i, v[u]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kQUnroll; ++u) {
            const long long i = base + u * kQThreads;
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[u][j]) & 0x7FFFFFFFu);
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const uint32_t ex = top >> 23;
            uint32_t e = ex > 2 ? ex - 2 : 0;
            const float f = __uint_as_float((254u - e) << 23);     // 2^(127 - e)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[u][j] *= f;
            uint32_t c = e2m1x8(v[u]);
            if (ex == 255) {
                c = 0;
                e = kScaleNan;
            }
            if (i < words) {
                wq[i] = c;
                if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(e);
            }
        }
    }
}

// ------------------------------------------------------------------ values of stored codes
//
// Every value is exact in BF16 (two significant bits; 2^-128 is one of its subnormals) unless it
// is beyond FP32's range too, where it becomes an infinity.  Bound: HBM.

// Eight codes to 16 bytes of BF16 values.
__device__ __forceinline__ uint4 values_bf16(uint32_t c, uint32_t e) {
    uint32_t r[4];
    expand8(c, factor_of(min(e, kOneFactor)), r);
    if (e > kOneFactor) {
        const uint32_t more = second_factor_of(e);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = mul_bf16x2(r[j], more);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// pairs: pairs of code words in all (blocks have two).  UNROLL of them a thread: two where the work is
// short of CTAs (2048 x 2560: 3.6 us, 4.4 with four), four for the loads in flight (9728 x 2560: 11.5 us,
// 5.5 TB/s; 12.8 with two).  To FP32 the same size takes 39.6 us, 2.9 TB/s: a thread's four stores of 16
// bytes lie 64 bytes from its neighbour's.
template <bool BF16, int UNROLL>
__global__ void __launch_bounds__(kQThreads) dequantize_kernel(const uint2 *wq, const uint8_t *scales, void *w, bool wide,
                                                               long long pairs) {
    pdl_launch_dependents();
    pdl_wait();
    const long long stride = static_cast<long long>(gridDim.x) * kQThreads * UNROLL;
    for (long long base = (static_cast<long long>(blockIdx.x) * UNROLL) * kQThreads + threadIdx.x; base < pairs;
         base += stride) {
        uint2 c[UNROLL];
        uint32_t e[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long long i = base + u * kQThreads;
            c[u] = i < pairs ? __ldcs(wq + i) : make_uint2(0u, 0u);
            e[u] = i < pairs ? scales[i >> 1] : 0u;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long long i = base + u * kQThreads;
            if (i >= pairs) break;
            if constexpr (BF16) {
                store_pair(static_cast<uint16_t *>(w) + 16 * i, values_bf16(c[u].x, e[u]), values_bf16(c[u].y, e[u]), wide);
            } else {
                const float s = scale_f32(e[u]);
                float4 *o = static_cast<float4 *>(w) + 4 * i;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t d = (q < 2 ? c[u].x : c[u].y) >> (16 * (q & 1));
                    o[q] = make_float4(code_f32(d) * s, code_f32(d >> 4) * s, code_f32(d >> 8) * s, code_f32(d >> 12) * s);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ the gated block's scalar parts

// silu(g) u and its derivatives, from FP32 sums: silu(g) = g s, s = 1 / (1 + e^-g), for negative g as
// e^g / (1 + e^g), so that nothing overflows and small s stay.  The fast exponential and division: together
// off by at most (6 + 1.2 |g|) 2^-23 of s, a thousandth of the results' BF16 step at the far end of the
// exponential's range (with the exact functions an epilogue of these outputs took longer than its tile's
// products).  Below 2^-126 s may count as 0.
__device__ __forceinline__ float sigmoid(float g) {
    const float t = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? t : 1.f, 1.f + t);
}
__device__ __forceinline__ float gated(float g, float u) { return g * sigmoid(g) * u; }
__device__ __forceinline__ void gated_backward(float g, float u, float dh, float &dg, float &du) {
    const float s = sigmoid(g);
    dg = dh * u * (s * (1.f + g * (1.f - s)));
    du = dh * (g * s);
}

// Both gradients where the sums are empty, g = u = 0: zeros, but not a number where dh is not finite.
// dh and dgu by eights: dh's block i is followed by dgu's blocks 2 i (gate) and 2 i + 1 (up).
__global__ void __launch_bounds__(kQThreads) empty_gates_kernel(const uint4 *dh, uint4 *dgu, long long blocks) {
    pdl_launch_dependents();
    pdl_wait();
    const long long stride = static_cast<long long>(gridDim.x) * kQThreads;
    for (long long i = static_cast<long long>(blockIdx.x) * kQThreads + threadIdx.x; i < blocks; i += stride) {
        const uint4 d = ldg_v4(dh + i);
        const float v[8] = {bf16_lo_to_f32(d.x), bf16_hi_to_f32(d.x), bf16_lo_to_f32(d.y), bf16_hi_to_f32(d.y),
                            bf16_lo_to_f32(d.z), bf16_hi_to_f32(d.z), bf16_lo_to_f32(d.w), bf16_hi_to_f32(d.w)};
        float a[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) gated_backward(0.f, 0.f, v[j], a[j], b[j]);
        dgu[2 * i] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
        dgu[2 * i + 1] = make_uint4(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]), pack_bf16x2(b[4], b[5]), pack_bf16x2(b[6], b[7]));
    }
}

}  // namespace mx
}  // namespace w4a16
