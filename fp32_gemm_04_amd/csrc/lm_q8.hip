// libsgemm products in 8-bit integers: argument checks, the choice of kernel and launches,
// behind the C ABI declared in include/slm.h.  Nothing here allocates, frees, copies or
// synchronises.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/slm.h"
#include "lm_host.hpp"
#include "lm_kernels.hpp"
#include "lm_q8.hpp"
#include "lm_rule.hpp"

namespace sgemm {
namespace lm {
namespace {

// 2^31 - 1 over 128 * 128: no sum of so many products of bytes overflows.
constexpr int kMostQ8 = 131071;
// Bytes of quantised rows that fit LDS beside the rings of q8_vec_kernel.
constexpr int kVecRows = 104 * 1024;

// An operand that direct loads take: rows at 4-byte addresses, and offsets inside a tile below 2^31.
bool q8_fast(const void *p, int64_t ld, int64_t group_stride)
{
    return aligned(p, 4) && ld % 4 == 0 && group_stride % 4 == 0 && ld < ((int64_t)1 << 22);
}

}  // namespace
}  // namespace lm
}  // namespace sgemm

using namespace sgemm::lm;

extern "C" int sgemm_q8_quantize(int type, int rows, int K, const void *X, int ldx, int k,
                                 const int *place, int out_rows, int8_t *Q, int ldq, float *scales,
                                 hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (rows < 0 || rows > kMostExtent) return -2;
    if (K < 0 || K > kMostExtent) return -3;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = K > 1 ? K : 1;
    const bool work = rows > 0 && out_rows > 0 && (!place || k > 0);
    if ((work && K > 0 && !X) || !aligned(X, size)) return -4;
    if (ldx < least) return -5;
    if (k < 0 || (!place && k != 0) || (rows > 0 && k > kMostExtent / rows)) return -6;
    if (!aligned(place, 4)) return -7;
    if (out_rows < 0 || out_rows > kMostExtent || (!place && out_rows != rows)) return -8;
    if (work && K > 0 && !Q) return -9;
    if (ldq < least) return -10;
    if ((work && !scales) || !aligned(scales, 4)) return -11;
    if (!work) return 0;
    QuantArgs a = {};
    a.X = X, a.Q = Q, a.scales = scales, a.place = place;
    a.ldx = ldx, a.ldq = ldq;
    a.rows = rows, a.K = K, a.k = k, a.out_rows = out_rows;
    // As many waves a row as its first values keep busy.
    const int waves = K <= 1024 ? 1 : K <= 2048 ? 2 : 4;
    const auto fn = [&](auto one, auto two, auto four) {
        return waves == 1 ? one : waves == 2 ? two : four;
    };
    const int64_t blocks = ceil_div(rows, 4 / waves);
    const dim3 grid((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks));
    if (type == SGEMM_TYPE_BF16)
        fn(q8_quantize_kernel<bf16, 1>, q8_quantize_kernel<bf16, 2>,
           q8_quantize_kernel<bf16, 4>)<<<grid, dim3(256), 0, stream>>>(a);
    else
        fn(q8_quantize_kernel<float, 1>, q8_quantize_kernel<float, 2>,
           q8_quantize_kernel<float, 4>)<<<grid, dim3(256), 0, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_q8_gemm(int type, int groups, int rows, int N, int K, const int8_t *X, int ldx,
                             const float *x_scales, const int8_t *W, int ldw, int64_t stride_w,
                             const float *w_scales, void *Y, int ldy, const int *offsets,
                             hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (groups < 0 || (!offsets && groups != 1)) return -2;
    if (rows < 0 || rows > kMostExtent) return -3;
    if (N < 0 || N > kMostExtent) return -4;
    if (K < 0 || K > kMostQ8) return -5;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = K > 1 ? K : 1;
    const bool work = groups > 0 && rows > 0 && N > 0, reads = work && K > 0;
    if (reads && !X) return -6;
    if (ldx < least) return -7;
    if ((work && !x_scales) || !aligned(x_scales, 4)) return -8;
    if (reads && !W) return -9;
    if (ldw < least) return -10;
    if (stride_w < 0) return -11;
    if ((work && !w_scales) || !aligned(w_scales, 4)) return -12;
    if ((work && !Y) || !aligned(Y, size)) return -13;
    if (ldy < (N > 1 ? N : 1)) return -14;
    if (!aligned(offsets, 4)) return -15;
    if (!work) return 0;
    const int used = groups < rows ? groups : rows;  // groups with rows, at most
    if ((rows + (int64_t)used * 15) / 16 * ceil_div(N, 64) > INT_MAX) return -4;

    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    const bool fast = K == 0 || (q8_fast(X, ldx, 0) && q8_fast(W, ldw, stride_w));
    const bool bf16_out = type == SGEMM_TYPE_BF16;
    const int tile = offsets ? rows_tile(1, fast, used, rows, N, ceil_div(K, 2), cus)
                             : plain_tile(1, F_ROWS_T, fast, rows, N, ceil_div(K, 2), cus);
    const TileKernel k = i8_kernel(bf16_out, offsets != nullptr, tile, fast);
    TileArgs a = {};
    a.A = X, a.B = W, a.C = Y;
    a.lda = ldx, a.ldb = ldw, a.ldc = ldy;
    a.group_stride = stride_w;
    a.M = rows, a.N = N, a.K = K;
    a.a_cols = a.b_cols = K;
    a.scale_a = x_scales, a.scale_b = w_scales;
    // How wide the stores to Y may be.
    for (int v = 2; v > 0; --v)
        if (!a.vec_c && aligned(Y, 4 * v * size) && ldy % (4 * v) == 0) a.vec_c = v;
    int64_t most = ceil_div(rows, k.bm);
    if (offsets) {  // every group's last tile may be part full
        most = (rows + (int64_t)used * (k.bm - 1)) / k.bm;
        a.groups = groups, a.offsets = offsets, a.most_tiles = (int)most;
    }
    const int64_t blocks = most * ceil_div(N, k.bn);
    if (blocks > kMostBlocks) return (int)hipErrorInvalidConfiguration;
    k.fn<<<dim3((unsigned)blocks), dim3(k.threads), 0, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_q8_matvec(int type, int groups, int rows, int N, int K, const void *X, int ldx,
                               const int8_t *W, int ldw, int64_t stride_w, const float *w_scales,
                               void *Y, int ldy, const int *offsets, hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (groups < 0 || (!offsets && groups != 1) || groups > 65535) return -2;
    if (rows < 0 || rows > kMostExtent) return -3;
    if (N < 0 || N > kMostExtent) return -4;
    if (K < 0 || K > kVecRows) return -5;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = K > 1 ? K : 1;
    const bool work = groups > 0 && rows > 0 && N > 0, reads = work && K > 0;
    if ((reads && !X) || !aligned(X, size)) return -6;
    if (ldx < least) return -7;
    if (reads && !W) return -8;
    if (ldw < least) return -9;
    if (stride_w < 0) return -10;
    if ((work && !w_scales) || !aligned(w_scales, 4)) return -11;
    if ((work && !Y) || !aligned(Y, size)) return -12;
    if (ldy < (N > 1 ? N : 1)) return -13;
    if (!aligned(offsets, 4)) return -14;
    if (!work) return 0;

    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    VecArgs a = {};
    a.X = X, a.W = W, a.w_scales = w_scales, a.Y = Y, a.offsets = offsets;
    a.ldx = ldx, a.ldw = ldw, a.stride_w = stride_w, a.ldy = ldy;
    a.rows = rows, a.N = N, a.K = K;
    a.slabs = (int)ceil_div(K, 128);
    a.pass = rows < 16 ? rows : 16;
    if (a.slabs > 0 && a.pass > kVecRows / 128 / a.slabs) a.pass = kVecRows / 128 / a.slabs;
    const bool fast = K == 0 || q8_fast(W, ldw, stride_w);
    const int depth = vec_lds(a.pass, a.slabs, 4) <= 160 * 1024 ? 4 : 2;
    const int lds = vec_lds(a.pass, a.slabs, depth);
    const auto fn = [&](auto four, auto two, auto slow) { return !fast ? slow : depth == 4 ? four : two; };
    const VecFn kernel =
        type == SGEMM_TYPE_BF16
            ? fn(q8_vec_kernel<bf16, 4, true>, q8_vec_kernel<bf16, 2, true>, q8_vec_kernel<bf16, 2, false>)
            : fn(q8_vec_kernel<float, 4, true>, q8_vec_kernel<float, 2, true>, q8_vec_kernel<float, 2, false>);
    // Two workgroups a unit where LDS has room, each with its share of the tiles.
    const int64_t tiles = ceil_div(N, 16), used = groups < rows ? groups : rows;
    const int64_t room = (int64_t)cus * (160 * 1024 / lds < 2 ? 1 : 2) / used;
    const int64_t blocks = room < 1 ? 1 : room < tiles ? room : tiles;
    kernel<<<dim3((unsigned)blocks, (unsigned)groups), dim3(kVecWaves * 64), lds, stream>>>(a);
    return (int)hipGetLastError();
}
