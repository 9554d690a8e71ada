// libsgemm language-model products: argument checks, the choice of tile,
// workspace layout and launches, behind the C ABI declared in include/slm.h.
// Nothing here allocates, frees, copies or synchronises: work is queued on the
// caller's stream.
#include <hip/hip_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "../../include/slm.h"
#include "lm_host.hpp"
#include "lm_kernels.hpp"
#include "lm_rule.hpp"

namespace sgemm {
namespace lm {

int compute_units(int *rc)
{
    static std::atomic<int> cache[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess && dev >= 0 && dev < 64) {
        int n = cache[dev].load(std::memory_order_relaxed);
        if (n > 0) return n;
        e = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
        if (e == hipSuccess && n > 0) {
            cache[dev].store(n, std::memory_order_relaxed);
            return n;
        }
    }
    *rc = e == hipSuccess ? (int)hipErrorInvalidDevice : (int)e;
    return 0;
}

namespace {

// Without a device, sizes are those of a whole MI355X (the call then fails).
constexpr int kNoDeviceUnits = 256;

int elem_size(int type) { return type == SGEMM_TYPE_BF16 ? 2 : 4; }

// An operand the direct loads take: rows at 4-byte addresses, and tile offsets below 2^31.
bool fast_operand(const void *p, int64_t ld, int64_t group_stride, int size)
{
    return aligned(p, 4) && ld * size % 4 == 0 && group_stride * size % 4 == 0 &&
           ld * size < ((int64_t)1 << 22);
}

// How wide the stores to an output may be: TileArgs::vec_c.
int vector_rows(const void *p, int64_t ld, int64_t group_stride, int size)
{
    for (int v = 2; v > 0; --v)
        if (aligned(p, 4 * v * size) && ld % (4 * v) == 0 && group_stride % (4 * v) == 0) return v;
    return 0;
}

TileKernel kernel_for(int type, int form, int tile, bool fast)
{
    return type == SGEMM_TYPE_BF16 ? bf16_kernel(form, tile, fast) : f32_kernel(form, tile, fast);
}

int launch(const TileKernel &k, TileArgs &a, int64_t blocks, int slices, hipStream_t stream)
{
    if (blocks > kMostBlocks) return (int)hipErrorInvalidConfiguration;
    k.fn<<<dim3((unsigned)blocks, 1, (unsigned)slices), dim3(k.threads), 0, stream>>>(a);
    return (int)hipGetLastError();
}

}  // namespace
}  // namespace lm
}  // namespace sgemm

using namespace sgemm::lm;

extern "C" int sgemm_grouped(int type, int trans, int groups, int rows, int N, int K, float alpha,
                             const void *X, int ldx, const void *W, int ldw, int64_t stride_w,
                             float beta, void *Y, int ldy, const int *offsets, hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (trans != 0 && trans != 1) return -2;
    if (groups < 0) return -3;
    if (rows < 0 || rows > kMostExtent) return -4;
    if (N < 0 || N > kMostExtent) return -5;
    if (K < 0 || K > kMostExtent) return -6;
    const int size = elem_size(type);
    const bool work = groups > 0 && rows > 0 && N > 0;
    const bool reads = work && K > 0 && alpha != 0.f;
    if ((reads && !X) || !aligned(X, size)) return -8;
    if (ldx < (K > 1 ? K : 1)) return -9;
    if ((reads && !W) || !aligned(W, size)) return -10;
    const int wcols = trans ? K : N;
    if (ldw < (wcols > 1 ? wcols : 1)) return -11;
    if (stride_w < 0) return -12;
    if ((work && !Y) || !aligned(Y, size)) return -14;
    if (ldy < (N > 1 ? N : 1)) return -15;
    if ((work && !offsets) || !aligned(offsets, 4)) return -16;
    if (!work) return 0;
    const int used = groups < rows ? groups : rows;  // groups with rows, at most
    if ((rows + (int64_t)used * 15) / 16 * ceil_div(N, 64) > INT_MAX) return -5;

    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    const int kk = reads ? K : 0;
    const bool fast = kk == 0 || (fast_operand(X, ldx, 0, size) &&
                                  fast_operand(W, ldw, stride_w, size));
    const int tile = rows_tile(size, fast, used, rows, N, kk, cus);
    const TileKernel k = kernel_for(type, trans ? F_ROWS_T : F_ROWS_N, tile, fast);
    // Every group's last tile may be part full.
    const int64_t most = (rows + (int64_t)used * (k.bm - 1)) / k.bm;
    const int64_t blocks = most * ceil_div(N, k.bn);
    TileArgs a = {};
    a.A = X, a.B = W, a.C = Y;
    a.lda = ldx, a.ldb = ldw, a.ldc = ldy;
    a.group_stride = stride_w;
    a.M = rows, a.N = N, a.K = kk;
    a.a_cols = K, a.b_cols = wcols, a.b_rows = kk;
    a.groups = groups, a.offsets = offsets, a.most_tiles = (int)most;
    a.alpha = alpha, a.beta = beta;
    a.vec_c = vector_rows(Y, ldy, 0, size);
    return launch(k, a, blocks, 1, stream);
}

extern "C" int sgemm_grouped_wgrad(int type, int groups, int rows, int M, int N, float alpha,
                                   const void *X, int ldx, const void *G, int ldg, float beta,
                                   void *D, int ldd, int64_t stride_d, const int *offsets,
                                   hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (groups < 0) return -2;
    if (rows < 0 || rows > kMostExtent) return -3;
    if (M < 0 || M > kMostExtent) return -4;
    if (N < 0 || N > kMostExtent) return -5;
    const int size = elem_size(type);
    const bool work = groups > 0 && M > 0 && N > 0;
    const bool reads = work && rows > 0 && alpha != 0.f;
    if ((reads && !X) || !aligned(X, size)) return -7;
    if (ldx < (M > 1 ? M : 1)) return -8;
    if ((reads && !G) || !aligned(G, size)) return -9;
    if (ldg < (N > 1 ? N : 1)) return -10;
    if ((work && !D) || !aligned(D, size)) return -12;
    if (ldd < (N > 1 ? N : 1)) return -13;
    if (stride_d < 0) return -14;
    // Groups' outputs one after another, or between each other's rows; never shared.
    if (work && groups > 1 && stride_d < (int64_t)(M - 1) * ldd + N &&
        (stride_d < N || stride_d > ((int64_t)ldd - N) / (groups - 1)))
        return -14;
    if ((work && !offsets) || !aligned(offsets, 4)) return -15;
    if (!work) return 0;
    // In parts, so that the product of three extents cannot overflow.
    const int64_t tiles64 = ceil_div(M, 64) * ceil_div(N, 64);
    if (tiles64 > INT_MAX / groups) return -5;

    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    const int kk = reads ? rows : 0;  // 0: every group is empty
    const bool fast = kk == 0 || (fast_operand(X, ldx, 0, size) &&
                                  fast_operand(G, ldg, 0, size));
    const int tile = sum_tile(size, fast, groups, kk, M, N, cus);
    const TileKernel k = kernel_for(type, F_SUM, tile, fast);
    const int64_t blocks = ceil_div(M, k.bm) * ceil_div(N, k.bn) * groups;
    TileArgs a = {};
    a.A = X, a.B = G, a.C = D;
    a.lda = ldx, a.ldb = ldg, a.ldc = ldd;
    a.group_stride = stride_d;
    a.M = M, a.N = N, a.K = kk;
    a.a_cols = M, a.b_cols = N;
    a.groups = groups, a.offsets = offsets;
    a.alpha = alpha, a.beta = beta;
    a.vec_c = vector_rows(D, ldd, stride_d, size);
    return launch(k, a, blocks, 1, stream);
}

// ---------------------------------------------------------------- cross entropy

namespace sgemm {
namespace lm {
namespace {

// Joins the tiles' row statistics, one wave per row: lse = ln 2 (top + log2 sum), top the
// largest of the tiles' and sum theirs, each scaled to top.  The loss takes the target's
// value z off top before log2 sum is added: lse - z would leave lse's own rounding, 2^-24
// of it, which for a confident row is far more than the loss.  Reads the statistics once:
// T 8192, 512 tiles a row: 10 us for 34 MB; with few rows its launch, 4 us.
__global__ void __launch_bounds__(256) xent_join_kernel(int rows, int tiles, int vocab,
                                                        const f32x2 *parts,
                                                        const float *target_value,
                                                        const int64_t *targets, float *loss,
                                                        float *lse)
{
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows;
         row += (int64_t)gridDim.x * 4) {
        const f32x2 *p = parts + row * tiles;
        float top = -INFINITY, sum = 0.f;
        for (int t = lane; t < tiles; t += 64) {
            const f32x2 v = p[t];
            join_sums(top, sum, v[0], v[1]);
        }
#pragma unroll
        for (int d = 32; d; d /= 2) join_sums(top, sum, __shfl_xor(top, d), __shfl_xor(sum, d));
        if (lane == 0) {
            constexpr float ln2 = 0.693147180559945309417f;
            const float more = log2f(sum);
            const float v = ((isfinite(top) ? top : 0.f) + more) * ln2;
            lse[row] = v;
            const int64_t target = targets[row];
            float out = 0.f;
            if (target >= 0 && target < vocab) {
                const float z = target_value[row];
                out = isfinite(top) ? (fmaf(-z, kLog2e, top) + more) * ln2 : v - z;
                out = out < 0.f ? 0.f : out;  // it never is, but for rounding
            }
            loss[row] = out;
        }
    }
}

// dX <- the slices' fp32 sums added in order, each with its remainders' sum low_rows further
// on, rounded once; four columns a thread.  Bound by reading the sums: 8192 x 2048 18 us
// (5.6 TB/s), 28 slices of 384 x 1024 11 us.
template <typename T>
__global__ void __launch_bounds__(256) xent_sum_kernel(int rows, int low_rows, int K, int slices,
                                                       int64_t slice_stride, const float *parts,
                                                       T *dX, int64_t lddx)
{
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
        if (c >= K) continue;
        const float *p = parts + (int64_t)row * K + c;
        const int n = K - c < 4 ? K - c : 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        const int64_t low = (int64_t)low_rows * K;
        for (int s = 0; s < slices; ++s, p += slice_stride) {
            if (K % 4 == 0) {  // 16-byte rows
                f32x4 x = *reinterpret_cast<const f32x4 *>(p);
                if (low_rows) x += *reinterpret_cast<const f32x4 *>(p + low);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += x[q];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < n) v[q] += low_rows ? p[q] + p[q + low] : p[q];
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < n) dX[(int64_t)row * lddx + c + q] = (T)v[q];
    }
}

int check_xent(int type, int rows, int vocab, int K, const void *X, int ldx, const void *W, int ldw,
               const int64_t *targets)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (rows < 0 || rows > kMostExtent) return -2;
    if (vocab < 0 || vocab > kMostExtent || (vocab == 0 && rows > 0)) return -3;
    if (K < 0 || K > kMostExtent) return -4;
    const int size = elem_size(type);
    const bool reads = rows > 0 && K > 0;
    if ((reads && !X) || !aligned(X, size)) return -5;
    if (ldx < (K > 1 ? K : 1)) return -6;
    if ((reads && !W) || !aligned(W, size)) return -7;
    if (ldw < (K > 1 ? K : 1)) return -8;
    if ((rows > 0 && !targets) || !aligned(targets, 8)) return -9;
    if (ceil_div(rows, 16) * ceil_div(vocab, 64) > INT_MAX) return -3;
    return 0;
}

}  // namespace
}  // namespace lm
}  // namespace sgemm

extern "C" int64_t sgemm_xent_workspace(int type, int rows, int vocab, int K, int backward)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (rows < 0 || rows > kMostExtent) return -2;
    if (vocab < 0 || vocab > kMostExtent) return -3;
    if (K < 0 || K > kMostExtent) return -4;
    if (backward != 0 && backward != 1) return -5;
    if (rows == 0 || vocab == 0) return 0;
    int rc = 0;
    int cus = compute_units(&rc);
    if (cus == 0) cus = kNoDeviceUnits;
    const int size = elem_size(type);
    if (!backward) return stats_bytes(size, rows, vocab, K, cus);
    if (K == 0) return 0;  // the gradients have no elements
    // Whichever operands the call gets.
    const int64_t a = xent_plan(size, true, rows, vocab, K, cus).bytes;
    const int64_t b = xent_plan(size, false, rows, vocab, K, cus).bytes;
    return a > b ? a : b;
}

extern "C" int sgemm_xent(int type, int rows, int vocab, int K, const void *X, int ldx,
                          const void *W, int ldw, const int64_t *targets, float *loss, float *lse,
                          void *ws, int64_t ws_bytes, hipStream_t stream)
{
    if (int rc = check_xent(type, rows, vocab, K, X, ldx, W, ldw, targets)) return rc;
    if ((rows > 0 && !loss) || !aligned(loss, 4)) return -10;
    if ((rows > 0 && !lse) || !aligned(lse, 4)) return -11;
    if ((rows > 0 && !ws) || !aligned(ws, 16)) return -12;
    if (rows == 0) return 0;
    int rc = 0;
    const int cus = compute_units(&rc);
    const int size = elem_size(type);
    if (ws_bytes < stats_bytes(size, rows, vocab, K, cus ? cus : kNoDeviceUnits)) return -13;
    if (cus == 0) return rc;
    const bool fast = K == 0 || (fast_operand(X, ldx, 0, size) &&
                                 fast_operand(W, ldw, 0, size));
    const int tile = plain_tile(size, F_STATS, fast, rows, vocab, K, cus);
    const TileKernel k = kernel_for(type, F_STATS, tile, fast);
    float *value = static_cast<float *>(ws);
    float *parts = value + round_up((int64_t)rows * 4, 256) / 4;
    const int tiles = (int)ceil_div(vocab, k.bn);
    TileArgs a = {};
    a.A = X, a.B = W;
    a.lda = ldx, a.ldb = ldw;
    a.M = rows, a.N = vocab, a.K = K;
    a.a_cols = a.b_cols = K;
    a.targets = targets, a.parts = parts, a.target_value = value;
    rc = launch(k, a, ceil_div(rows, k.bm) * tiles, 1, stream);
    if (rc) return rc;
    const int64_t joins = ceil_div(rows, 4);
    xent_join_kernel<<<dim3((unsigned)(joins < kMostBlocks ? joins : kMostBlocks)), dim3(256), 0, stream>>>(
        rows, tiles, vocab, reinterpret_cast<const sgemm::f32x2 *>(parts), value, targets, loss, lse);
    return (int)hipGetLastError();
}

extern "C" int sgemm_xent_backward(int type, int rows, int vocab, int K, const void *X, int ldx,
                                   const void *W, int ldw, const int64_t *targets, const float *lse,
                                   const float *dloss, void *dX, int lddx, void *dW, int lddw,
                                   void *ws, int64_t ws_bytes, hipStream_t stream)
{
    if (int rc = check_xent(type, rows, vocab, K, X, ldx, W, ldw, targets)) return rc;
    const int size = elem_size(type);
    if ((rows > 0 && !lse) || !aligned(lse, 4)) return -10;
    if ((rows > 0 && !dloss) || !aligned(dloss, 4)) return -11;
    if (!aligned(dX, size)) return -12;
    if (lddx < (K > 1 ? K : 1)) return -13;
    if (!aligned(dW, size)) return -14;
    if (lddw < (K > 1 ? K : 1)) return -15;
    if ((rows > 0 && K > 0 && !ws) || !aligned(ws, 16)) return -16;
    if (K == 0 || vocab == 0 || (!dX && !dW) || (rows == 0 && !dW)) return 0;
    int rc = 0;
    const int cus = compute_units(&rc);
    TileArgs a = {};
    if (rows == 0) {  // no row: dW is zero
        a.C = dW, a.ldc = lddw;
        a.M = vocab, a.N = K;
        a.vec_c = vector_rows(dW, lddw, 0, size);
        const TileKernel k = kernel_for(type, F_DW, M64, true);
        return launch(k, a, ceil_div(vocab, k.bm) * ceil_div(K, k.bn), 1, stream);
    }
    const bool fast_x = fast_operand(X, ldx, 0, size), fast_w = fast_operand(W, ldw, 0, size);
    const XentPlan p = xent_plan(size, fast_w, rows, vocab, K, cus ? cus : kNoDeviceUnits);
    if (ws_bytes < p.bytes) return -17;
    if (cus == 0) return rc;
    float *sums = reinterpret_cast<float *>(static_cast<char *>(ws) + p.d_bytes);

    for (int64_t c = 0; c < p.pieces; ++c) {
        const int64_t col0 = c * p.piece;
        const int n = (int)(vocab - col0 < p.piece ? vocab - col0 : p.piece);
        const int n8 = (int)round_up(n, 8);  // columns the derivatives are written for
        const char *Wc = static_cast<const char *>(W) + col0 * ldw * size;
        {
            const bool fast = fast_x && fast_w;
            const int stored = p.low_rows ? p.low_rows : rows;
            const int tile = grad_tile(size, fast, p, rows, n, K, cus);
            const TileKernel k = kernel_for(type, F_GRAD, tile, fast);
            a = TileArgs{};
            a.A = X, a.B = Wc, a.C = ws;
            a.lda = ldx, a.ldb = ldw, a.ldc = p.ld;
            a.M = rows, a.N = n, a.K = K;
            a.a_cols = a.b_cols = K;
            a.targets = targets, a.lse = lse, a.dloss = dloss;
            a.col0 = (int)col0, a.vocab = vocab;
            a.store_rows = stored, a.low_rows = p.low_rows;
            rc = launch(k, a, ceil_div(stored, k.bm) * ceil_div(n, k.bn), 1, stream);
            if (rc) return rc;
        }
        if (dW) {
            const bool fast = fast_x;
            const int tile = plain_tile(size, F_DW, fast, n, K, p.d_rows, cus);
            const TileKernel k = kernel_for(type, F_DW, tile, fast);
            a = TileArgs{};
            a.A = ws, a.B = X, a.C = static_cast<char *>(dW) + col0 * lddw * size;
            a.lda = p.ld, a.ldb = ldx, a.ldc = lddw;
            a.M = n, a.N = K, a.K = p.d_rows;
            a.a_cols = n8, a.b_cols = K, a.b_rows = rows;
            a.wrap = p.low_rows;
            a.alpha = 1.f;
            a.vec_c = vector_rows(dW, lddw, 0, size);
            rc = launch(k, a, ceil_div(n, k.bm) * ceil_div(K, k.bn), 1, stream);
            if (rc) return rc;
        }
        if (dX) {
            const bool fast = fast_w;
            a = TileArgs{};
            a.A = ws, a.B = Wc;
            a.lda = p.ld, a.ldb = ldw;
            a.M = p.d_rows, a.N = K, a.K = n;
            a.a_cols = n8, a.b_cols = K, a.b_rows = n;
            const bool direct = p.dx_form == F_DX;
            const TileKernel k = kernel_for(type, p.dx_form, p.dx_tile, fast);
            if (direct) {
                a.C = dX, a.ldc = lddx, a.alpha = 1.f;
                a.vec_c = vector_rows(dX, lddx, 0, size);
            } else {
                a.C = p.sums ? static_cast<void *>(sums) : dX;
                a.ldc = p.sums ? K : lddx;
                a.vec_c = aligned(a.C, 16) && a.ldc % 4 == 0;
                a.accumulate = c > 0;
                a.split_k = (int)round_up(ceil_div(n, p.slices), 64);
                a.slice_stride = (int64_t)p.d_rows * K;
            }
            rc = launch(k, a, ceil_div(p.d_rows, k.bm) * ceil_div(K, k.bn), direct ? 1 : p.slices,
                        stream);
            if (rc) return rc;
        }
    }
    if (dX && p.sums) {
        const dim3 grid((unsigned)ceil_div(K, 1024), (unsigned)(rows < 65535 ? rows : 65535));
        const int64_t stride = (int64_t)p.d_rows * K;
        if (type == SGEMM_TYPE_BF16)
            xent_sum_kernel<bf16><<<grid, dim3(256), 0, stream>>>(rows, p.low_rows, K, p.slices, stride, sums,
                                                                  static_cast<bf16 *>(dX), lddx);
        else
            xent_sum_kernel<float><<<grid, dim3(256), 0, stream>>>(rows, p.low_rows, K, p.slices, stride, sums,
                                                                   static_cast<float *>(dX), lddx);
        return (int)hipGetLastError();
    }
    return 0;
}
