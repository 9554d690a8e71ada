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

template <typename T, int BLOCK, bool ALIGNED>
Q4Fn kernel_of(const Q4Plan &f)
{
    if (f.rt == 1) return f.nt == 1 ? q4_kernel<T, BLOCK, 1, 1, ALIGNED>
                                    : q4_kernel<T, BLOCK, 1, 2, ALIGNED>;
    if constexpr (Parts<T>::value == 1)
        if (f.rt == 4) return q4_kernel<T, BLOCK, 4, 2, ALIGNED>;
    return q4_kernel<T, BLOCK, 2, 2, ALIGNED>;
}

template <typename T>
Q4Fn kernel_for(int block, bool al, const Q4Plan &f)
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

    int rc = 0;
    const int cus = compute_units(&rc);
    if (cus == 0) return rc;
    const Q4Plan p = q4_plan(size, offsets != nullptr, groups, rows, N, K, block, cus);
    Q4Args a = {};
    a.X = X, a.Q = Q, a.S = S, a.Z = Z, a.Y = Y, a.offsets = offsets;
    a.ldx = ldx, a.ldy = ldy;
    a.q_stride = (int64_t)N * (K / 2);
    a.s_stride = (int64_t)N * ceil_div(K, block);
    a.rows = rows, a.N = N, a.K = K;
    a.wn = p.wn;
    a.pass = p.pass;
    a.slab_log2 = p.slab_log2;
    a.vec_x = aligned(X, 16) && (int64_t)ldx * size % 16 == 0;
    // Direct loads: rows at 4-byte addresses, and offsets inside a workgroup below 2^31.
    const bool al = K % 8 == 0 && aligned(Q, 4) && K < (1 << 23);
    const Q4Fn fn = type == SGEMM_TYPE_BF16 ? kernel_for<bf16>(block, al, p)
                                            : kernel_for<float>(block, al, p);
    const int64_t blocks = ceil_div(N, p.cols);
    fn<<<dim3((unsigned)blocks, (unsigned)groups), dim3(kThreads), p.lds, stream>>>(a);
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
