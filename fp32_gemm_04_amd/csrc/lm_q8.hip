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

template <typename T, bool PLACED> auto quantize_of(int waves)
{
    return waves == 1   ? q8_quantize_kernel<T, 1, PLACED>
           : waves == 2 ? q8_quantize_kernel<T, 2, PLACED>
           : waves == 4 ? q8_quantize_kernel<T, 4, PLACED>
                        : q8_quantize_kernel<T, 8, PLACED>;
}

template <typename TY, int BM, int BN, int DEPTH, bool FAST> TileKernel split_entry(bool grouped)
{
    return TileKernel{grouped ? (TileFn)q8_split_kernel<TY, BM, BN, DEPTH, true, FAST>
                              : (TileFn)q8_split_kernel<TY, BM, BN, DEPTH, false, FAST>,
                      BM, BN, kSplitWaves * 64};
}
template <typename TY> TileKernel split_of(bool grouped, int split, bool fast)
{
    if (!fast) return split == 0 ? split_entry<TY, 16, 32, 1, false>(grouped) : split_entry<TY, 32, 32, 1, false>(grouped);
    switch (split) {
    case 0: return split_entry<TY, 16, 32, 2, true>(grouped);
    case 1: return split_entry<TY, 32, 32, 2, true>(grouped);
    case 2: return split_entry<TY, 32, 64, 1, true>(grouped);
    default: return split_entry<TY, 64, 64, 1, true>(grouped);
    }
}
TileKernel split_kernel(bool bf16_out, bool grouped, int split, bool fast)
{
    return bf16_out ? split_of<bf16>(grouped, split, fast) : split_of<float>(grouped, split, fast);
}

// A product of few rows: X is int8 with scales, or of the results' type.
int vec_product(VecArgs &a, bool bytes, bool bf16_out, int cus, hipStream_t stream)
{
    a.slabs = (int)ceil_div(a.K, 128);
    a.pass = a.rows < 16 ? a.rows : 16;
    if (a.slabs > 0 && a.pass > kVecRows / 128 / a.slabs) a.pass = kVecRows / 128 / a.slabs;
    const bool fast = a.K == 0 || q8_fast(a.W, a.ldw, a.stride_w);
    const int depth = vec_lds(a.pass, a.slabs, 4) <= 160 * 1024 ? 4 : 2;
    const int lds = vec_lds(a.pass, a.slabs, depth);
    const auto fn = [&](auto four, auto two, auto slow) { return !fast ? slow : depth == 4 ? four : two; };
    const auto of = [&](auto x, auto y) -> VecFn {
        typedef decltype(x) TX;
        typedef decltype(y) TY;
        return fn(q8_vec_kernel<TX, TY, 4, true>, q8_vec_kernel<TX, TY, 2, true>,
                  q8_vec_kernel<TX, TY, 2, false>);
    };
    const VecFn kernel = bytes ? (bf16_out ? of(int8_t(), bf16()) : of(int8_t(), float()))
                         : bf16_out ? of(bf16(), bf16())
                                    : of(float(), float());
    // Two workgroups a unit where LDS has room, each with its share of the tiles.
    const int64_t tiles = ceil_div(a.N, 16), used = a.groups < 1 ? 1 : a.groups < a.rows ? a.groups : a.rows;
    const int64_t room = (int64_t)cus * (160 * 1024 / lds < 2 ? 1 : 2) / used;
    const int64_t blocks = room < 1 ? 1 : room < tiles ? room : tiles;
    kernel<<<dim3((unsigned)blocks, (unsigned)used), dim3(kVecWaves * 64), lds, stream>>>(a);
    return (int)hipGetLastError();
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
    if (K < 0 || K > kMostQ8) return -3;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = K > 1 ? K : 1;
    const bool work = rows > 0 && out_rows > 0 && (!place || k > 0);
    if ((work && K > 0 && !X) || !aligned(X, size)) return -4;
    if (ldx < least) return -5;
    // (Places of no rows may be NULL: then k says that there were some.)
    if (k < 0 || (rows > 0 && (k > kMostExtent / rows || (!place && k > 0)))) return -6;
    if (!aligned(place, 4)) return -7;
    if (out_rows < 0 || out_rows > kMostExtent || (!place && k == 0 && out_rows != rows)) return -8;
    if (work && K > 0 && !Q) return -9;
    if (ldq < least) return -10;
    if ((work && !scales) || !aligned(scales, 4)) return -11;
    if (!work) return 0;
    QuantArgs a = {};
    a.X = X, a.Q = Q, a.scales = scales, a.place = place;
    a.ldx = ldx, a.ldq = ldq;
    a.rows = rows, a.K = K, a.k = k, a.out_rows = out_rows;
    const int64_t pieces = ceil_div(K, 16 / size);
    // As few waves a row as hold it in registers, but more where they would not fill the units.
    int waves = pieces <= 64 * kHeld ? 1 : pieces <= 128 * kHeld ? 2 : pieces <= 256 * kHeld ? 4 : 8;

    // us: 8192 rows of 2048 bf16 11.5 with one, 11.7 with two; 64 rows of 4096 7 with two, 4.3 with four, 3.8
    // with eight; 12 rows of 14336 8.0 with four, 5.3 with eight, 8192 fp32 rows of 8192 70.7 and 61.5 (6.8 TB/s,
    // part of it from the last-level cache), of 5000 36.4 and 36.8.
    while (waves < 8 && (int64_t)rows * waves < 4096 && pieces > 64 * waves) waves *= 2;
    const int threads = quantize_waves(waves) * 64;
    const dim3 grid(launch_blocks(ceil_div(rows, quantize_waves(waves) / waves), threads));
    const auto fn = type == SGEMM_TYPE_BF16
                        ? (place ? quantize_of<bf16, true>(waves) : quantize_of<bf16, false>(waves))
                        : (place ? quantize_of<float, true>(waves) : quantize_of<float, false>(waves));
    fn<<<grid, dim3(threads), 0, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_q8_gemm(int type, int groups, int rows, int N, int K, const int8_t *X, int ldx,
                             const float *x_scales, const int8_t *W, int ldw, int64_t stride_w,
                             const float *w_scales, void *Y, int ldy, const int *offsets,
                             int fill, hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (groups < 0 || (!offsets && groups != 1)) return -2;
    if (rows < 0 || rows > kMostExtent) return -3;
    if (N < 0 || N > kMostExtent) return -4;
    if (K < 0 || K > kMostQ8) return -5;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = K > 1 ? K : 1;
    const bool work = (groups > 0 || fill) && rows > 0 && N > 0, reads = work && groups > 0 && K > 0;
    if (reads && !X) return -6;
    if (ldx < least) return -7;
    if ((work && groups > 0 && !x_scales) || !aligned(x_scales, 4)) return -8;
    if (reads && !W) return -9;
    if (ldw < least) return -10;
    if (stride_w < 0) return -11;
    if ((work && groups > 0 && !w_scales) || !aligned(w_scales, 4)) return -12;
    if ((work && !Y) || !aligned(Y, size)) return -13;
    if (ldy < (N > 1 ? N : 1)) return -14;
    if (!aligned(offsets, 4)) return -15;
    if (fill != 0 && fill != 1) return -16;
    if (!work) return 0;
    const int used = groups < 1 ? 1 : groups < rows ? groups : rows;  // groups with rows, at most
    const bool bf16_out = type == SGEMM_TYPE_BF16;
    const bool fast = K == 0 || (q8_fast(X, ldx, 0) && q8_fast(W, ldw, stride_w));
    const bool few = K <= kVecRows && byte_few_rows(fast, offsets ? groups : 0, used, rows);
    const int side = byte_side(fast);
    if (!few && byte_blocks(offsets ? used : 0, rows, N, side, side) > kMostBlocks) return -4;

    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    if (few) {
        VecArgs v = {};
        v.X = X, v.x_scales = x_scales, v.W = W, v.w_scales = w_scales, v.Y = Y, v.offsets = offsets;
        v.ldx = ldx, v.ldw = ldw, v.stride_w = stride_w, v.ldy = ldy;
        v.rows = rows, v.N = N, v.K = K, v.groups = groups, v.fill = offsets && fill;
        return vec_product(v, true, bf16_out, cus, stream);
    }
    const int tile = byte_rows_tile(fast, offsets ? used : 0, rows, N, K, cus);
    const TileKernel k = tile >= NUM_TILES ? split_kernel(bf16_out, offsets != nullptr, tile - NUM_TILES, fast)
                                           : i8_kernel(bf16_out, offsets != nullptr, tile, fast);
    TileArgs a = {};
    a.A = X, a.B = W, a.C = Y;
    a.lda = ldx, a.ldb = ldw, a.ldc = ldy;
    a.group_stride = stride_w;
    a.M = rows, a.N = N, a.K = K;
    a.a_cols = a.b_cols = K;
    a.scale_a = x_scales, a.scale_b = w_scales;
    const int64_t blocks = byte_blocks(offsets ? used : 0, rows, N, k.bm, k.bn);
    if (offsets)
        a.groups = groups, a.offsets = offsets, a.most_tiles = (int)(blocks / ceil_div(N, k.bn)), a.fill = fill;
    k.fn<<<dim3((unsigned)blocks), dim3(k.threads), 0, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_q8_matvec(int type, int groups, int rows, int N, int K, const void *X, int ldx,
                               const int8_t *W, int ldw, int64_t stride_w, const float *w_scales,
                               void *Y, int ldy, const int *offsets, int fill, hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (groups < 0 || (!offsets && groups != 1) || groups > 65535) return -2;
    if (rows < 0 || rows > kMostExtent) return -3;
    if (N < 0 || N > kMostExtent) return -4;
    if (K < 0 || K > kVecRows) return -5;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = K > 1 ? K : 1;
    const bool work = (groups > 0 || fill) && rows > 0 && N > 0, reads = work && groups > 0 && K > 0;
    if ((reads && !X) || !aligned(X, size)) return -6;
    if (ldx < least) return -7;
    if (reads && !W) return -8;
    if (ldw < least) return -9;
    if (stride_w < 0) return -10;
    if ((work && groups > 0 && !w_scales) || !aligned(w_scales, 4)) return -11;
    if ((work && !Y) || !aligned(Y, size)) return -12;
    if (ldy < (N > 1 ? N : 1)) return -13;
    if (!aligned(offsets, 4)) return -14;
    if (fill != 0 && fill != 1) return -15;
    if (!work) return 0;

    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    VecArgs a = {};
    a.X = X, a.W = W, a.w_scales = w_scales, a.Y = Y, a.offsets = offsets;
    a.ldx = ldx, a.ldw = ldw, a.stride_w = stride_w, a.ldy = ldy;
    a.rows = rows, a.N = N, a.K = K, a.groups = groups, a.fill = offsets && fill;
    return vec_product(a, false, type == SGEMM_TYPE_BF16, cus, stream);
}
