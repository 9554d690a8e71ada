// libsgemm products with weights held in 4 bits: argument checks, the choice of
// kernel and launches, behind the C ABI declared in include/slm.h.  Nothing
// here allocates, frees, copies or synchronises.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/slm.h"
#include "lm_host.hpp"
#include "q4.hpp"

namespace sgemm {
namespace q4 {
namespace {

using lm::aligned;
using lm::ceil_div;
using lm::compute_units;
using lm::kMostBlocks;
using lm::kMostExtent;

// A workgroup's offsets stay within 32 bits.
constexpr int kMostK = 1 << 27;

struct Form {
    int rt, nt;
};

template <typename T, int BLOCK, bool ALIGNED>
Q4Fn kernel_of(Form f)
{
    if (f.rt == 1) return f.nt == 1 ? q4_kernel<T, BLOCK, 1, 1, ALIGNED>
                                    : q4_kernel<T, BLOCK, 1, 2, ALIGNED>;
    if constexpr (Parts<T>::value == 1)
        if (f.rt == 4) return q4_kernel<T, BLOCK, 4, 2, ALIGNED>;
    return q4_kernel<T, BLOCK, 2, 2, ALIGNED>;
}

template <typename T>
Q4Fn kernel_for(int block, bool al, Form f)
{
    if (block == 32) return al ? kernel_of<T, 32, true>(f) : kernel_of<T, 32, false>(f);
    if (block == 64) return al ? kernel_of<T, 64, true>(f) : kernel_of<T, 64, false>(f);
    return al ? kernel_of<T, 128, true>(f) : kernel_of<T, 128, false>(f);
}

template <typename T>
void quantize(dim3 grid, int N, int K, int block, int nblk, const void *W, int64_t ldw, uint8_t *Q,
              void *S, uint8_t *Z, hipStream_t stream)
{
    auto fn = block == 32 ? (Z ? q4_quantize_kernel<T, 32, true> : q4_quantize_kernel<T, 32, false>)
            : block == 64 ? (Z ? q4_quantize_kernel<T, 64, true> : q4_quantize_kernel<T, 64, false>)
                          : (Z ? q4_quantize_kernel<T, 128, true>
                               : q4_quantize_kernel<T, 128, false>);
    fn<<<grid, dim3(256), 0, stream>>>(N, K, nblk, static_cast<const T *>(W), ldw, Q,
                                       static_cast<T *>(S), Z);
}

}  // namespace
}  // namespace q4
}  // namespace sgemm

using namespace sgemm::q4;

extern "C" int sgemm_q4_matvec(int type, int groups, int rows, int N, int K, int block,
                               const void *X, int ldx, const uint8_t *Q, const void *S,
                               const uint8_t *Z, void *Y, int ldy, const int *offsets,
                               hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (groups < 0 || (!offsets && groups != 1) || groups > 65535) return -2;
    if (rows < 0 || rows > kMostExtent) return -3;
    if (N < 0 || N > kMostExtent) return -4;
    if (K < 0 || K % 2 != 0 || K > kMostK) return -5;
    if (block != 32 && block != 64 && block != 128) return -6;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4;
    const bool work = groups > 0 && rows > 0 && N > 0, reads = work && K > 0;
    if ((reads && !X) || !aligned(X, size)) return -7;
    if (ldx < (K > 1 ? K : 1)) return -8;
    if (reads && !Q) return -9;
    if ((reads && !S) || !aligned(S, size)) return -10;
    if ((work && !Y) || !aligned(Y, size)) return -12;
    if (ldy < (N > 1 ? N : 1)) return -13;
    if (!aligned(offsets, 4)) return -14;
    if (!work) return 0;

    const int parts = type == SGEMM_TYPE_F32 ? 3 : 1;
    const int used = groups < rows ? groups : rows;
    const int64_t mean = ceil_div(rows, used);  // rows of a group
    // Rows per pass: no more than a group is likely to have, so that more of K is staged
    // at once.
    const int64_t likely = offsets ? 2 * mean : rows;
    const int most_pass = parts == 1 ? 64 : 24;
    const int pass = likely < most_pass ? (int)likely : most_pass;
    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    // The more columns a workgroup takes (NT per wave, wn waves), the less often x is
    // staged and read: until four workgroups remain per compute unit, or 1.5 where
    // staging x (two bytes a part, against half a byte a weight) would outweigh the
    // weights.
    Form f = {pass > 32 ? 4 : pass > 16 ? 2 : 1, pass > 16 ? 2 : 1};
    const int64_t tiles = used * ceil_div(N, 16);
    int wn = 1;
    while (wn < kWaves) {
        const int cols = 16 * f.nt * wn;
        const int64_t left = tiles / (f.nt * wn * 2);
        if (left < (cols < 8 * pass * parts ? cus * 3 / 2 : 4 * cus)) break;
        if (f.nt == 1)
            f.nt = 2;
        else
            wn *= 2;
    }
    // What a slab of one chunk per wave needs must fit in 32 KB of LDS beside the rings'
    // 32 KB (two workgroups per compute unit).  With wn = 8 every pass does.
    const auto bytes = [&](int64_t slab, int cols) {
        return type == SGEMM_TYPE_BF16 ? slab_bytes<bf16>((int)slab, block, cols, pass)
                                       : slab_bytes<float>((int)slab, block, cols, pass);
    };
    int room = 32 * 1024;
    const auto fits = [&](int64_t slab) {
        return bytes(slab, wn * f.nt * 16) <= room;
    };
    while (wn < kWaves && !fits(128 * kWaves / wn)) wn *= 2;
    Q4Args a = {};
    a.X = X, a.Q = Q, a.S = S, a.Z = Z, a.Y = Y, a.offsets = offsets;
    a.ldx = ldx, a.ldy = ldy;
    a.q_stride = (int64_t)N * (K / 2);
    a.s_stride = (int64_t)N * ceil_div(K, block);
    a.rows = rows, a.N = N, a.K = K;
    a.wn = wn;
    a.pass = pass;
    const int cols = wn * f.nt * 16;
    const int step = 128 * kWaves / wn;
    if (used * ceil_div(N, cols) <= cus) room = 124 * 1024;
    int64_t slab = step;
    while (slab < K && fits(slab * 2)) slab *= 2;
    a.slab_log2 = __builtin_ctzll((unsigned long long)slab);
    a.vec_x = aligned(X, 16) && (int64_t)ldx * size % 16 == 0;
    // Direct loads: rows at 4-byte addresses, and offsets inside a workgroup below 2^31.
    const bool al = K % 8 == 0 && aligned(Q, 4) && K < (1 << 23);
    const Q4Fn fn = type == SGEMM_TYPE_BF16 ? kernel_for<bf16>(block, al, f)
                                            : kernel_for<float>(block, al, f);
    const int staged = ring_bytes(f.nt) + bytes(slab, cols);
    const int sums = kWaves / wn * pass * cols * 4;
    const int64_t blocks = ceil_div(N, cols);
    fn<<<dim3((unsigned)blocks, (unsigned)groups), dim3(kThreads),
         staged > sums ? staged : sums, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_q4_quantize(int type, int N, int K, int block, const void *W, int ldw,
                                 uint8_t *Q, void *S, uint8_t *Z, hipStream_t stream)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (N < 0 || N > kMostExtent) return -2;
    if (K < 0 || K % 2 != 0 || K > kMostK) return -3;
    if (block != 32 && block != 64 && block != 128) return -4;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4;
    const bool work = N > 0 && K > 0;
    if ((work && !W) || !aligned(W, size)) return -5;
    if (ldw < (K > 1 ? K : 1)) return -6;
    if (work && !Q) return -7;
    if ((work && !S) || !aligned(S, size)) return -8;
    if (!work) return 0;
    const int nblk = (int)ceil_div(K, block);
    const int64_t blocks = ceil_div((int64_t)N * nblk, 16);
    const dim3 grid((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks));
    if (type == SGEMM_TYPE_BF16)
        quantize<bf16>(grid, N, K, block, nblk, W, ldw, Q, S, Z, stream);
    else
        quantize<float>(grid, N, K, block, nblk, W, ldw, Q, S, Z, stream);
    return (int)hipGetLastError();
}
