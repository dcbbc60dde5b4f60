// mx_entry.cuh - host side of the MXFP4 entry points declared in include/w4a16.h: argument checks
// and launches.  Included by w4a16.cu, whose device set-up and helpers it uses.  None of these calls
// allocates or keeps a workspace, so a captured call needs no warm-up and replays share nothing.
#pragma once

#include "mx.cuh"
#include "mx_a4.cuh"
#include "mx_gemm.cuh"
#include "mx_matvec.cuh"

namespace w4a16 {
namespace {

// Row numbers of partial tiles and of stages asked for ahead stay below 2^31.
constexpr int64_t kSizeLimit = (int64_t(1) << 31) - 65536;

struct Span {
    const void *p;
    size_t bytes;
};

// Every buffer present and aligned, no output on top of another buffer.  The first `outputs`
// spans are written.
int check_buffers(const Span *s, int n, int outputs) {
    for (int i = 0; i < n; ++i)
        if (!s[i].p && s[i].bytes) return W4A16_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (s[i].bytes && !aligned16(s[i].p)) return W4A16_ERR_MISALIGNED;
    for (int i = 0; i < outputs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (s[i].bytes && s[j].bytes && overlaps(s[i].p, s[i].bytes, s[j].p, s[j].bytes)) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

int mx_sizes(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0) return W4A16_ERR_INVALID_ARG;
    if (K % mx::kBlock != 0 || M >= kSizeLimit || N >= kSizeLimit || K >= kSizeLimit) return W4A16_ERR_UNSUPPORTED;
    return W4A16_OK;
}

using MxGemm = void(const CUtensorMap, const CUtensorMap, const mxg::Params);
template <bool PAIR, int SHARE>
MxGemm *mx_gemm_of(bool backward, int epilogue) {
    if (backward) return mxg::gemm_kernel<true, mxg::kPlain, PAIR, SHARE>;
    if (epilogue == mxg::kGated) return mxg::gemm_kernel<false, mxg::kGated, PAIR, SHARE>;
    if (epilogue == mxg::kGatedBackward) return mxg::gemm_kernel<false, mxg::kGatedBackward, PAIR, SHARE>;
    return mxg::gemm_kernel<false, mxg::kPlain, PAIR, SHARE>;
}
template <bool PAIR>
MxGemm *mx_gemm_of(bool backward, int epilogue, int share) {
    if (share == mxg::kNone) return mx_gemm_of<PAIR, mxg::kNone>(backward, epilogue);
    if (share == mxg::kLast) return mx_gemm_of<PAIR, mxg::kLast>(backward, epilogue);
    return mx_gemm_of<PAIR, mxg::kAll>(backward, epilogue);
}
MxGemm *mx_gemm_of(bool backward, int epilogue, bool pair, int share) {
    return pair ? mx_gemm_of<true>(backward, epilogue, share) : mx_gemm_of<false>(backward, epilogue, share);
}

cudaLaunchAttribute mx_cluster(int ctas) {
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = ctas;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
    return a;
}

int mx_device(DeviceInfo **d) {
    int dev = 0;
    int rc = current_device(&dev);
    if (!rc) rc = device_setup(dev, d);
    if (rc || (*d)->mx_ready) return rc;
    cudaError_t e = cudaSuccess;
    for (bool pair : {false, true})
        for (int share : {mxg::kNone, mxg::kLast, mxg::kAll})
            for (MxGemm *kernel :
                 {mx_gemm_of(false, mxg::kPlain, pair, share), mx_gemm_of(false, mxg::kGated, pair, share),
                  mx_gemm_of(false, mxg::kGatedBackward, pair, share), mx_gemm_of(true, mxg::kPlain, pair, share)})
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, mxg::kSmemBudget);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(mx4::a4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, mx4::kSmemBytes);
    for (int ctas = 1; ctas <= mxg::kMaxCluster && e == cudaSuccess; ++ctas) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas, 1, 1);
        cfg.blockDim = dim3(mxg::kThreads, 1, 1);
        cfg.dynamicSmemBytes = mxg::kSmemBudget;
        cudaLaunchAttribute cl = mx_cluster(ctas);
        cfg.attrs = &cl;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&(*d)->mx_clusters[ctas], mx_gemm_of(true, mxg::kPlain, false, mxg::kNone), &cfg);
    }
    if (e != cudaSuccess) return cuda_fail(e);
    (*d)->mx_ready = true;
    return W4A16_OK;
}

int zero_fill(void *p, size_t bytes, void *stream) {
    const cudaError_t e = cudaMemsetAsync(p, 0, bytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4A16_OK : cuda_fail(e);
}

// A launch of clusters of `cluster` CTAs with the programmatic-dependent-launch attribute (every
// kernel here waits for the preceding one before its first access).
template <typename... KArgs, typename... Args>
int mx_launch(void (*kernel)(KArgs...), dim3 grid, int cluster, int block, size_t smem, void *stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1] = mx_cluster(cluster);
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? W4A16_OK : cuda_fail(e);
}

// Rows of a tiled load of x, at most a CTA's: where x has fewer, no more than there are, up to eights (the
// swizzle's).  Rows of a load that lie outside a tensor of less than 128 KB cost time: gradients of 24 rows
// x 2560 x 9728 took 25.9 us with loads of 128 rows, 12.5 so; of 1 row x 1024 x 2560 9.2 and 5.8.
int mx_box_rows(int64_t M, int most) { return static_cast<int>(std::min<int64_t>((M + 7) / 8 * 8, most)); }

mxg::Output mx_output(void *out, const void *dh, int64_t M, int64_t J, int epilogue) {
    mxg::Output o;
    o.out = static_cast<uint16_t *>(out);
    o.dh = static_cast<const uint16_t *>(dh);
    o.M = static_cast<int>(M);
    o.J = static_cast<int>(J);
    const int64_t row = epilogue == mxg::kGated ? J / 2 : J;
    o.wide = row % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    return o;
}

// CTAs work in pairs on 256 rows, or alone on 128 where there are no more (64 rows x 9728 x 2560: 14.2 us
// alone, 16.5 in pairs).  The outputs of a tile (bn) and how many pairs or CTAs share a tile's contraction
// (splits) are those of the least estimated time in SM cycles: a stage takes a pair 283 cycles and three an
// output, or either as long as a CTA's codes take to expand, 450 cycles and 3.25 an output of the CTA, and a
// pair about 40 more where a warp of the expanding has rows to spare (all measured: stages of 128, 192 and
// 256 outputs at 2048 x 4096 x 4096 took 0.43, 0.54 and 0.68 us); a persistent grid runs rounds of tiles, and
// the tiles that do not fill a round may be shared, one a cluster of up to eight CTAs, if they then fit the
// device at once, for the price of an exchange of sums.  Backward, 2048 x 9728 x 2560: 80.8 us in two rounds
// of 192 outputs, the second half empty, 72.8 in one of 256 and a shared one; gated block, 40 rows x 2 x
// 9728 x 2560: 23.2 and 21.5; 64 rows, backward of 19456 x 2560, shared by six: 25.6, by four at most: 27.5;
// 2048 x 4096 x 4096 by 256 outputs 49.0, by 160, which a count of MMAs alone would choose, 55.5.
struct MxShape {
    bool pair = true;
    int bn = 0, splits = 1;
    int64_t full = 0, clusters = 0;   // tiles computed by one pair or CTA each; clusters of the grid
};
MxShape mx_gemm_shape(int64_t M, int64_t J, int64_t C, bool backward, bool ragged, const DeviceInfo *d) {
    const int64_t steps = (C + mxg::kStep - 1) / mxg::kStep;
    MxShape best;
    int64_t cost = 0;
    best.pair = M > mxg::kRows;
    const int ctas = best.pair ? 2 : 1;
    const int64_t tm = (M + ctas * mxg::kRows - 1) / (ctas * mxg::kRows);
    const int most = (ragged ? mxg::kMaxRaggedBN : mxg::kMaxBN) * ctas / 2;
    for (int bn = 32 * ctas; bn <= most; bn += backward || ctas == 1 ? 32 * ctas : 32) {
        const int64_t tiles = tm * ((J + bn - 1) / bn);
        const int half = bn / ctas;
        const int64_t stage = best.pair ? std::max(283 + 3 * bn, 450 + 13 * half / 4) + (half % 32 ? 40 : 0) : 450 + 13 * half / 4;
        for (int S = 1; ctas * S <= mxg::kMaxCluster; ++S) {
            const int64_t room = std::max<int64_t>(1, std::min<int64_t>(d->mx_clusters[ctas * S], d->sms / (ctas * S)));
            const int64_t full = S > 1 ? tiles / (room * S) * (room * S) : tiles, rest = tiles - full;
            if (S > 1 && (d->mx_clusters[ctas * S] < 1 || rest == 0 || rest > room || steps < 2 * S || !mxg::sums_fit(bn, ctas, S))) continue;
            const int64_t rounds = (full + room * S - 1) / (room * S);
            const int64_t c = rounds * (steps * stage + 500) +
                              (S > 1 ? (steps + S - 1) / S * stage + 3500 + 500 * S + 4 * bn * (S - 1) : 0);
            if (!best.bn || c <= cost) {
                best.bn = bn;
                best.splits = S;
                best.full = full;
                best.clusters = full ? std::min(room, tiles) : rest;
                cost = c;
            }
        }
    }
    return best;
}

// D = A . W^T (forward) or A . W (backward) on the tensor cores: A bf16 [M, C], J outputs.
int mx_gemm(DeviceInfo *d, const void *a, const uint32_t *wq, const uint8_t *ws, const void *dh, void *out, int64_t M,
            int64_t J, int64_t C, int64_t N, int64_t K, bool backward, int epilogue, void *stream) {
    const bool ragged = epilogue == mxg::kPlain && J % 8 != 0;
    const MxShape shape = mx_gemm_shape(M, J, C, backward, ragged, d);
    mxg::Params p;
    p.o = mx_output(out, dh, M, J, epilogue);
    p.ws = ws;
    p.C = static_cast<int>(C);
    p.ks = static_cast<int>(K / mx::kBlock);
    p.bn = shape.bn;
    p.splits = shape.splits;
    p.full = static_cast<int>(shape.full);
    const int ctas = shape.pair ? 2 : 1;
    const int64_t tm = (M + ctas * mxg::kRows - 1) / (ctas * mxg::kRows), tiles = tm * ((J + p.bn - 1) / p.bn);
    if (tiles >= kSizeLimit) return W4A16_ERR_UNSUPPORTED;
    p.tiles_m = static_cast<int>(tm);
    p.tiles = static_cast<int>(tiles);
    const int half = p.bn / ctas;
    p.b_bytes = backward ? (half + 63) / 64 * mxg::kGroupBytes : half * mxg::kStep * 2;
    p.w_bytes = half * mxg::kStep / 2;
    p.w_pitch = backward ? half / 2 : mxg::kStep / 2;
    // codes tile: rows of 32 and 64 bytes are swizzled by the copy (else neighbouring rows' 16-byte
    // chunks would share banks); chunks at a pitch of 16 or 48 bytes spread by themselves
    CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_NONE;
    p.w_swz_shift = p.w_swz_mask = 0;
    if (p.w_pitch == 32) {
        swz = CU_TENSOR_MAP_SWIZZLE_32B;
        p.w_swz_shift = 2;
        p.w_swz_mask = 1;
    } else if (p.w_pitch == 64) {
        swz = CU_TENSOR_MAP_SWIZZLE_64B;
        p.w_swz_shift = 1;
        p.w_swz_mask = 3;
    }
    const int smem = mxg::smem_bytes(p.b_bytes, p.w_bytes, ragged);

    CUtensorMap tx, tw;
    const int rows = mx_box_rows(M, mxg::kRows);
    p.x_bytes = rows * mxg::kStep * 2;
    int rc = encode_2d(d, &tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a, C, M, C * 2, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    rc = encode_2d(d, &tw, CU_TENSOR_MAP_DATA_TYPE_UINT32, wq, K / 8, N, K / 2, backward ? half / 8 : mxg::kStep / 8,
                   backward ? mxg::kStep : half, swz);
    if (rc) return rc;
    const dim3 grid(static_cast<unsigned>(ctas * p.splits * shape.clusters), 1, 1);
    const int share = shape.splits == 1 ? mxg::kNone : (shape.full ? mxg::kLast : mxg::kAll);
    return mx_launch(mx_gemm_of(backward, epilogue, shape.pair, share), grid, ctas * p.splits, mxg::kThreads, smem, stream, tx, tw, p);
}

// Outputs of a CTA pair of the 4-bit product: the fewest column-rounds of the persistent grid; an MMA
// of 64 columns takes about as long as one of 100.
int mx_a4_width(int64_t M, int64_t N, int pairs) {
    const int64_t tm = (M + 2 * mx4::kRows - 1) / (2 * mx4::kRows);
    int best = 0;
    int64_t cost = 0;
    for (int bn = 64; bn <= mx4::kMaxBN; bn += 64) {
        const int64_t tiles = tm * ((N + bn - 1) / bn), rounds = (tiles + pairs - 1) / pairs;
        const int64_t c = rounds * std::max(bn, 100);
        if (!best || c <= cost) {
            best = bn;
            cost = c;
        }
    }
    return best;
}

int mx_a4(DeviceInfo *d, const uint32_t *xq, const uint8_t *xs, const uint32_t *wq, const uint8_t *ws, void *y, int64_t M,
          int64_t N, int64_t K, void *stream) {
    const int pairs = d->sms / 2;
    mx4::Params p;
    p.o = mx_output(y, nullptr, M, N, mxg::kPlain);
    p.xs = xs;
    p.ws = ws;
    p.K = static_cast<int>(K);
    p.bn = mx_a4_width(M, N, pairs);
    const int64_t tm = (M + 2 * mx4::kRows - 1) / (2 * mx4::kRows), tiles = tm * ((N + p.bn - 1) / p.bn);
    if (tiles >= kSizeLimit) return W4A16_ERR_UNSUPPORTED;
    p.tiles_n = static_cast<int>((N + p.bn - 1) / p.bn);
    p.tiles = static_cast<int>(tiles);
    CUtensorMap tx, tw;
    const int rows = mx_box_rows(M, mx4::kRows);
    p.x_bytes = rows * mx4::kStep / 2;
    int rc = encode_2d(d, &tx, CU_TENSOR_MAP_DATA_TYPE_UINT32, xq, K / 8, M, K / 2, mx4::kStep / 8, rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    rc = encode_2d(d, &tw, CU_TENSOR_MAP_DATA_TYPE_UINT32, wq, K / 8, N, K / 2, mx4::kStep / 8, p.bn / 2,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    CUtensorMap ty;
    std::memset(&ty, 0, sizeof(ty));
    if (N % 8 == 0)
        rc = encode_2d(d, &ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (rc) return rc;
    const dim3 grid(static_cast<unsigned>(2 * std::min<int64_t>(tiles, pairs)), 1, 1);
    return mx_launch(mx4::a4_kernel, grid, 2, mx4::kThreads, mx4::kSmemBytes, stream, tx, tw, ty, p);
}

// Few rows of x take the row kernel: up to 8 always; up to 16 where the weight times the rows beyond 8 is not
// large and K not long, as every CTA of 16 weight rows reads all of x from the cache, group by group, nor long
// for CTAs of four warps that leave SMs half empty; up to 32 where K is short and every CTA of eight warps is
// resident.  Measured, us, row kernel / GEMM, N x K, weights from HBM:
//   M = 8   9728 x 2560 8.6 / 13.0, 151936 x 2560 77.7 / 94.4, 2560 x 19456 20.5 / 22.7; but 16384 x 16384
//           73.8 / 68.6, 5120 x 9728 24.4 / 21.1, 512 x 65536 34.8 / 30.4
//   M = 9   19456 x 2560 16.0 / 21.3, 38912 x 2560 27.8 / 31.6, 9728 x 9728 32.6 / 36.8; but 12800 x 5120
//           24.9 / 21.8, and not taken: 5120 x 9728 29.7 / 21.1, 1024 x 12288 15.2 / 14.0, 512 x 65536 58.3 / 30.5
//   M = 12  9728 x 2560 10.2 / 13.1, 38912 x 2560 30.8 / 31.5, 9728 x 9728 34.1 / 36.8; but 12800 x 2560
//           15.3 / 13.4, and not taken: 151936 x 2560 101.7 / 94.6, 1024 x 16384 20.3 / 15.8
//   M = 16  9728 x 2560 11.6 / 13.1, 4096 x 9728 16.5 / 18.3, 19456 x 2560 21.3 / 21.4; but 12800 x 2560
//           18.4 / 13.3, and not taken: 38912 x 2560 38.0 / 31.7, 151936 x 2560 123.9 / 94.6
//   M = 17  1024 x 2560 6.9 / 9.1, 4096 x 4096 9.9 / 12.8; not taken: 6400 x 2560 12.6 / 11.7, 1024 x 8192
//           16.0 / 12.9
//   M = 32  1024 x 2560 8.5 / 9.1, 4096 x 2560 8.8 / 10.6, 4096 x 4096 13.1 / 12.8; not taken: 2560 x 9728
//           26.9 / 16.3
bool mx_few_rows(int64_t M, int64_t N, int64_t K, int sms) {
    if (M <= 8) return true;
    const int64_t blocks = (N + 15) / 16;
    if (M > 16) return M <= mxv::kMaxM && K <= 4096 && blocks <= 2 * sms;
    if (K > 4096 && blocks > 2 * sms && blocks < 4 * sms) return false;
    return K < 12288 && (M - 8) * N <= (int64_t(3) << 27) / K;
}

template <int NB, int WARPS, int D, int CTAS, bool X4>
int mx_matvec_launch(const mxv::Params &p, void *stream) {
    const dim3 grid(static_cast<unsigned>((int64_t(p.N) + 15) / 16), 1, 1);
    return mx_launch(mxv::matvec_kernel<NB, WARPS, D, CTAS, X4>, grid, 1, 32 * WARPS, 0, stream, p);
}

// Warps of a CTA (they share its rows' K): as many as leave every CTA resident at once, 16 (one
// CTA an SM), 8 (two) or 4 (five).  Measured at M = 1, us, with 16 / 8 / 4 warps: N x K 2560 x 9728
// 10.7 / 9.9 / 13.1, 4096 x 2560 5.8 / 3.9 / 5.4, 9728 x 2560 12.4 / 8.7 / 7.0.  Groups in flight a warp: as
// many as there are registers for (M = 12, 8 warps: 1024 x 2560 4.4 with two, 4.0 with four).
template <bool X4>
int mx_matvec_8(const mxv::Params &p, const DeviceInfo *d, void *stream) {
    const int64_t blocks = (int64_t(p.N) + 15) / 16;
    if (blocks <= d->sms) return mx_matvec_launch<1, 16, 4, 1, X4>(p, stream);
    if (blocks <= 2 * d->sms) return mx_matvec_launch<1, 8, 4, 2, X4>(p, stream);
    return mx_matvec_launch<1, 4, 4, 5, X4>(p, stream);
}

mxv::Params mx_matvec_params(const uint32_t *wq, const uint8_t *ws, void *out, int64_t M, int64_t N, int64_t K) {
    mxv::Params p = {};
    p.wq = wq;
    p.ws = ws;
    p.out = static_cast<uint16_t *>(out);
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    return p;
}

int mx_matvec(DeviceInfo *d, const void *x, const uint32_t *wq, const uint8_t *ws, void *out, int64_t M, int64_t N,
              int64_t K, bool gated, void *stream) {
    mxv::Params p = mx_matvec_params(wq, ws, out, M, N, K);
    p.x = static_cast<const uint16_t *>(x);
    p.gated = gated ? 1 : 0;
    if (M <= 8) return mx_matvec_8<false>(p, d, stream);
    if (M <= 16) {
        if ((N + 15) / 16 <= 2 * d->sms) return mx_matvec_launch<2, 8, 4, 2, false>(p, stream);
        return mx_matvec_launch<2, 4, 2, 5, false>(p, stream);
    }
    return mx_matvec_launch<4, 8, 1, 2, false>(p, stream);
}

// The same with x in 4 bits, for up to 8 rows where every CTA is resident with eight warps or more, or K is
// short: else the FP4 tensor cores are faster, as here x is expanded anew for every 16 weight rows.  Measured,
// us, this / FP4 tensor cores, M = 8, N x K, weights from HBM: 1024 x 2560 3.9 / 6.4, 4736 x 2560 4.9 / 8.4,
// 4096 x 9728 12.7 / 15.2, 512 x 65536 37.4 / 71.5, 9728 x 1024 4.6 / 6.7, 151936 x 512 25.4 / 30.3; not taken:
// 4752 x 2560 8.5 / 7.3, 9728 x 2560 9.2 / 8.8, 5120 x 9728 25.9 / 15.8, 151936 x 2560 84.1 / 52.6.
bool mx_few_a4(int64_t M, int64_t N, int64_t K, int sms) { return M <= 8 && ((N + 15) / 16 <= 2 * sms || K <= 1536); }

int mx_matvec_a4(DeviceInfo *d, const uint32_t *xq, const uint8_t *xs, const uint32_t *wq, const uint8_t *ws, void *out,
                 int64_t M, int64_t N, int64_t K, void *stream) {
    mxv::Params p = mx_matvec_params(wq, ws, out, M, N, K);
    p.xq = xq;
    p.xs = xs;
    return mx_matvec_8<true>(p, d, stream);
}

// CTAs of a streaming kernel whose threads take `unroll` items each at a time.
unsigned stream_grid(int64_t items, int unroll, int sms) {
    const int64_t per = int64_t(mx::kQThreads) * unroll;
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((items + per - 1) / per, int64_t(sms) * 8)));
}

}  // namespace
}  // namespace w4a16

extern "C" {

int w4a16_mx_quantize(const void *w, int32_t w_dtype, uint32_t *wq, uint8_t *scales, int64_t N, int64_t K,
                      void *stream) {
    if (w_dtype != W4A16_DTYPE_F32 && w_dtype != W4A16_DTYPE_BF16) return W4A16_ERR_INVALID_ARG;
    int rc = mx_sizes(0, N, K);
    if (rc || N == 0 || K == 0) return rc;
    const size_t n = size_t(N) * K;
    const Span s[3] = {{wq, n / 2}, {scales, n / 32}, {w, n * (w_dtype == W4A16_DTYPE_F32 ? 4 : 2)}};
    rc = check_buffers(s, 3, 2);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo *d = nullptr;
    rc = mx_device(&d);
    if (rc) return rc;
    const long long words = N * (K / 8);
    const dim3 grid(stream_grid(words, mx::kQUnroll, d->sms), 1, 1);
    if (w_dtype == W4A16_DTYPE_BF16)
        return mx_launch(mx::quantize_kernel<true>, grid, 1, mx::kQThreads, 0, stream, w, wq, scales, words);
    return mx_launch(mx::quantize_kernel<false>, grid, 1, mx::kQThreads, 0, stream, w, wq, scales, words);
}

int w4a16_mx_dequantize(const uint32_t *wq, const uint8_t *scales, void *w, int32_t w_dtype, int64_t N, int64_t K,
                        void *stream) {
    if (w_dtype != W4A16_DTYPE_F32 && w_dtype != W4A16_DTYPE_BF16) return W4A16_ERR_INVALID_ARG;
    int rc = mx_sizes(0, N, K);
    if (rc || N == 0 || K == 0) return rc;
    const size_t n = size_t(N) * K;
    const Span s[3] = {{w, n * (w_dtype == W4A16_DTYPE_F32 ? 4 : 2)}, {wq, n / 2}, {scales, n / 32}};
    rc = check_buffers(s, 3, 1);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo *d = nullptr;
    rc = mx_device(&d);
    if (rc) return rc;
    const long long pairs = N * (K / 16);
    const int unroll = pairs >= (1 << 20) ? 4 : 2;
    const dim3 grid(stream_grid(pairs, unroll, d->sms), 1, 1);
    const auto *codes = reinterpret_cast<const uint2 *>(wq);
    const bool wide = (reinterpret_cast<uintptr_t>(w) & 31u) == 0;
    const auto kernel = w_dtype == W4A16_DTYPE_BF16
                            ? (unroll == 4 ? mx::dequantize_kernel<true, 4> : mx::dequantize_kernel<true, 2>)
                            : (unroll == 4 ? mx::dequantize_kernel<false, 4> : mx::dequantize_kernel<false, 2>);
    return mx_launch(kernel, grid, 1, mx::kQThreads, 0, stream, codes, scales, w, wide, pairs);
}

int w4a16_mx_matmul(const void *x, const uint32_t *wq, const uint8_t *scales, void *y, int64_t M, int64_t N, int64_t K,
                    void *stream) {
    int rc = mx_sizes(M, N, K);
    if (rc || M == 0 || N == 0) return rc;
    const size_t nw = size_t(N) * K;
    const Span s[4] = {{y, size_t(M) * N * 2}, {x, size_t(M) * K * 2}, {wq, nw / 2}, {scales, nw / 32}};
    rc = check_buffers(s, 4, 1);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo *d = nullptr;
    rc = mx_device(&d);
    if (rc) return rc;
    if (K == 0) return zero_fill(y, s[0].bytes, stream);   // an empty sum
    if (mx_few_rows(M, N, K, d->sms)) return mx_matvec(d, x, wq, scales, y, M, N, K, false, stream);
    return mx_gemm(d, x, wq, scales, nullptr, y, M, N, K, N, K, false, mxg::kPlain, stream);
}

int w4a16_mx_matmul_a4(const uint32_t *xq, const uint8_t *xscales, const uint32_t *wq, const uint8_t *scales, void *y,
                       int64_t M, int64_t N, int64_t K, void *stream) {
    int rc = mx_sizes(M, N, K);
    if (rc || M == 0 || N == 0) return rc;
    const size_t nx = size_t(M) * K, nw = size_t(N) * K;
    const Span s[5] = {{y, size_t(M) * N * 2}, {xq, nx / 2}, {xscales, nx / 32}, {wq, nw / 2}, {scales, nw / 32}};
    rc = check_buffers(s, 5, 1);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo *d = nullptr;
    rc = mx_device(&d);
    if (rc) return rc;
    if (K == 0) return zero_fill(y, s[0].bytes, stream);
    if (mx_few_a4(M, N, K, d->sms)) return mx_matvec_a4(d, xq, xscales, wq, scales, y, M, N, K, stream);
    return mx_a4(d, xq, xscales, wq, scales, y, M, N, K, stream);
}

int w4a16_mx_gate_up(const void *x, const uint32_t *wq, const uint8_t *scales, void *h, int64_t M, int64_t N2, int64_t K,
                     void *stream) {
    int rc = mx_sizes(M, N2, K);
    if (rc) return rc;
    if (N2 % 8 != 0 || N2 >= kSizeLimit / 2) return W4A16_ERR_UNSUPPORTED;
    if (M == 0 || N2 == 0) return W4A16_OK;
    const size_t nw = size_t(N2) * 2 * K;
    const Span s[4] = {{h, size_t(M) * N2 * 2}, {x, size_t(M) * K * 2}, {wq, nw / 2}, {scales, nw / 32}};
    rc = check_buffers(s, 4, 1);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo *d = nullptr;
    rc = mx_device(&d);
    if (rc) return rc;
    if (K == 0) return zero_fill(h, s[0].bytes, stream);   // silu(0) 0 = +0
    if (mx_few_rows(M, 2 * N2, K, d->sms)) return mx_matvec(d, x, wq, scales, h, M, 2 * N2, K, true, stream);
    return mx_gemm(d, x, wq, scales, nullptr, h, M, 2 * N2, K, 2 * N2, K, false, mxg::kGated, stream);
}

int w4a16_mx_matmul_backward(const void *dy, const uint32_t *wq, const uint8_t *scales, void *dx, int64_t M, int64_t N,
                             int64_t K, void *stream) {
    int rc = mx_sizes(M, N, K);
    if (rc) return rc;
    if (N % 8 != 0) return W4A16_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return W4A16_OK;
    const size_t nw = size_t(N) * K;
    const Span s[4] = {{dx, size_t(M) * K * 2}, {dy, size_t(M) * N * 2}, {wq, nw / 2}, {scales, nw / 32}};
    rc = check_buffers(s, 4, 1);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo *d = nullptr;
    rc = mx_device(&d);
    if (rc) return rc;
    if (N == 0) return zero_fill(dx, s[0].bytes, stream);
    return mx_gemm(d, dy, wq, scales, nullptr, dx, M, K, N, N, K, true, mxg::kPlain, stream);
}

int w4a16_mx_gate_up_backward(const void *x, const uint32_t *wq, const uint8_t *scales, const void *dh, void *dgu,
                              void *dx, int64_t M, int64_t N2, int64_t K, void *stream) {
    int rc = mx_sizes(M, N2, K);
    if (rc) return rc;
    if (N2 % 8 != 0 || N2 >= kSizeLimit / 2) return W4A16_ERR_UNSUPPORTED;
    if (M == 0) return W4A16_OK;
    const size_t nw = size_t(N2) * 2 * K;
    const Span s[6] = {{dx, size_t(M) * K * 2},  {dgu, size_t(M) * N2 * 4}, {x, size_t(M) * K * 2},
                       {dh, size_t(M) * N2 * 2}, {wq, nw / 2},              {scales, nw / 32}};
    rc = check_buffers(s, 6, 2);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo *d = nullptr;
    rc = mx_device(&d);
    if (rc) return rc;
    if (N2 == 0) return K == 0 ? W4A16_OK : zero_fill(dx, s[0].bytes, stream);
    if (K == 0) {
        const long long blocks = M * (N2 / 8);
        const dim3 grid(stream_grid(blocks, 1, d->sms), 1, 1);
        return mx_launch(mx::empty_gates_kernel, grid, 1, mx::kQThreads, 0, stream, static_cast<const uint4 *>(dh),
                         static_cast<uint4 *>(dgu), blocks);
    }
    rc = mx_gemm(d, x, wq, scales, dh, dgu, M, 2 * N2, K, 2 * N2, K, false, mxg::kGatedBackward, stream);
    if (rc) return rc;
    return mx_gemm(d, dgu, wq, scales, nullptr, dx, M, K, 2 * N2, 2 * N2, K, true, mxg::kPlain, stream);
}

}  // extern "C"
