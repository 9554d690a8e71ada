// Tile kernels of the language-model products (include/slm.h): fp32 or bf16
// operands, fp32 accumulation, three operand layouts, ragged rows or a ragged
// contraction, and the epilogues the products need.
//
// One workgroup computes a BM x BN tile of C = A B^T, where A has BM rows and
// B has BN rows (the columns of C), both walked along the contraction in
// slabs of 128 bytes (BK = 64 bf16 or 32 fp32).  An operand comes in one of
// two layouts in memory:
//   KC  the contraction index is contiguous: a slab row is 128 bytes of it;
//   MC  the row index is contiguous: the slab is BK rows of BM (or BN) values.
//
// A slab travels from memory to an LDS ring of NBUF buffers with
// buffer_load_dwordx4 ... lds (the wave's 64 x 16 bytes land in lane order),
// so no registers hold it.  The buffer descriptor ends where the operand
// ends: a row past the end reads as zero without any per-lane test, and a
// slab issued past the last one touches no memory, so the ring needs no
// special tail.  Only the last slab of a KC operand whose K is not a multiple
// of BK moves single lanes out of the descriptor's range.
// When an operand is not 16-byte aligned throughout (FAST false), the same
// slabs go through registers, each value tested against the operand's ends.
//
// LDS layouts, in 16-byte chunks; the permutation is applied to which chunk a
// lane fetches, since the DMA writes lanes in order:
//   KC: row r holds its 8 chunks at places p = c ^ (r & 7), so the 16 lanes of
//       an operand read (one chunk of each of 16 rows) meet every bank evenly.
//   MC: slab row k holds chunk c at p = c ^ swizzle(k).  bf16 operands are
//       read with ds_read_b64_tr_b16, which hands a lane four consecutive k
//       of one column: 16 lanes read 32 bytes of 4 rows, and swizzle(k) =
//       2 (k & 3) puts those rows in different banks.  fp32 operands need one
//       k per lane and step: four lane groups read 64 bytes of rows 4 apart,
//       and swizzle(k) = k & 12 separates them.
//
// Both operands of a matrix instruction use the same assignment of k to lanes:
// with l = lane, g = l / 16, bf16 16x16x32 takes k = 8 g .. 8 g + 7, and four
// fp32 16x16x4 steps s = 0..3 take k = 4 g + s.  B is the instruction's first
// operand, so a lane holds four consecutive columns of one row of C:
//   row l % 16, columns 4 g .. 4 g + 3 of each 16 x 16 block.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace sgemm {
namespace lm {

typedef __bf16 bf16;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum Layout { KC, MC };
// PLAIN: one product.  ROWS: the rows of A and C fall into groups, each with a
// B of its own.  SUM: the contraction falls into groups, each with a C of its own.
enum Ragged { PLAIN, ROWS, SUM };
// STORE: C <- alpha acc + beta C.  STATS: row maxima and sums of exponentials of
// the tile, and the value at the row's target.  GRAD: the loss's derivative by
// each value.  PART: fp32 C <- acc (+ C), for sums joined later.
enum Epilogue { STORE, STATS, GRAD, PART };

struct TileArgs {
    const void *A, *B;
    void *C;
    int64_t lda, ldb, ldc;       // elements
    int64_t group_stride;        // ROWS: of B; SUM: of C (elements)
    int M, N;                    // extent of C (ROWS: M = all rows)
    int K;                       // contraction (SUM: all rows)
    int a_cols, b_cols;          // readable extent of an operand's contiguous index
    int b_rows;                  // MC, not SUM: rows of B that exist (<= K)
    int groups;
    const int *offsets;          // groups + 1 row numbers (ROWS, SUM)
    int most_tiles;              // ROWS: row tiles that increasing offsets can give
    float alpha, beta;
    int vec_c;                   // C's rows take vector stores
    int accumulate;              // PART: add to what is there
    int split_k;                 // PART: contraction per z-slice (multiple of the slab)
    int64_t slice_stride;        // PART: elements between slices of C
    // Cross entropy: rows are tokens, columns the vocabulary from col0 on.
    const int64_t *targets;
    const float *lse, *dloss;
    float *parts;                // STATS: (maximum, sum) of [row][tile along N]
    float *target_value;
    int col0, vocab;
};

typedef void (*TileFn)(TileArgs);

template <typename T> struct Elem;
template <> struct Elem<bf16> {
    static constexpr int BK = 64, EPC = 8;
    typedef bf16x8 Frag;
};
template <> struct Elem<float> {
    static constexpr int BK = 32, EPC = 4;
    typedef f32x4 Frag;
};

// Lane l's 16 bytes at base + voff go to LDS [lds + 16 l, + 16); zeros where
// voff lies outside the descriptor.  s_nop: an LDS DMA needs a wait state after
// the write of M0, and the descriptor may have been written by the vector unit.
__device__ __forceinline__ void load_slab16(u32x4 rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
                 "buffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(lds)
                 : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_slab_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

constexpr uint32_t kOutside = 0x80000000u;  // beyond every descriptor's range

// A descriptor of the bytes [p, p + left), at most 2^31 of them.
__device__ __forceinline__ u32x4 descriptor(const char *p, int64_t left)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t n = left <= 0 ? 0u : left > (int64_t)kOutside ? kOutside : (uint32_t)left;
    u32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xffffu;
    r[2] = __builtin_amdgcn_readfirstlane(n);
    r[3] = 0x00020000u;
    return r;
}

// One operand's slabs: where this wave's units (64 chunks each) come from.
template <typename T, int B, Layout L>
struct Slab {
    static constexpr int BK = Elem<T>::BK, EPC = Elem<T>::EPC;
    static constexpr int UNITS = B / 8;            // 64-chunk units per slab
    static constexpr int BYTES = B * 128;
    static constexpr int RC = B / EPC;             // MC: chunks per slab row

    __device__ static __forceinline__ int swizzle(int k)
    {
        if constexpr (std::is_same<T, float>::value)
            return (k & 12) & (RC - 1);
        else
            return (2 * (k & 3)) & (RC - 1);
    }
    // Row (KC: of the tile; MC: of the slab) and chunk that slot s fetches.
    __device__ static __forceinline__ void slot(int s, int &row, int &chunk)
    {
        if constexpr (L == KC) {
            row = s >> 3;
            chunk = (s & 7) ^ (row & 7);
        } else {
            row = s / RC;
            chunk = (s % RC) ^ swizzle(row);
        }
    }
    // The operand fragment of 16-row block blk and step (half slab) h.
    __device__ static __forceinline__ typename Elem<T>::Frag frag(const char *buf, int blk, int h,
                                                                  int lane)
    {
        const int l = lane & 15, g = lane >> 4;
        if constexpr (L == KC) {
            const char *p = buf + blk * 2048 + l * 128 + (((4 * h + g) ^ (l & 7)) << 4);
            return *reinterpret_cast<const typename Elem<T>::Frag *>(p);
        } else if constexpr (std::is_same<T, float>::value) {
            f32x4 v;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = 16 * h + 4 * g + s;
                const int c = (4 * blk + (l >> 2)) ^ swizzle(k);
                v[s] = *reinterpret_cast<const float *>(buf + k * (B * 4) + c * 16 + (l & 3) * 4);
            }
            return v;
        } else {
            bf16x8 v;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = 32 * h + 8 * g + 4 * s + (l >> 2);
                const int c = (2 * blk + ((l >> 1) & 1)) ^ swizzle(k);
                const uint32_t at = (uint32_t)(uintptr_t)(const lds_char *)buf + k * (B * 2) +
                                    c * 16 + (l & 1) * 8;
                const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4 *)(uintptr_t)at);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * s + j] = __builtin_bit_cast(bf16, (short)q[j]);
            }
            return v;
        }
    }
};

template <typename T>
__device__ __forceinline__ f32x4 mfma_step(const typename Elem<T>::Frag &b,
                                           const typename Elem<T>::Frag &a, f32x4 c)
{
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
        for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(b[s], a[s], c, 0, 0, 0);
        return c;
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
    }
}

__device__ __forceinline__ int clamp_row(int v, int lo, int hi)
{
    return v < lo ? lo : v > hi ? hi : v;
}

// Rows [begin, end) of group e, whatever the offsets hold: inside [0, rows].
__device__ __forceinline__ void group_rows(const int *offsets, int e, int rows, int &begin, int &end)
{
    begin = clamp_row(offsets[e], 0, rows);
    end = clamp_row(offsets[e + 1], begin, rows);
}

// The row tiles of all groups, counted 64 groups at a time by the wave's lanes.
// 64-bit sums, and the caller's clamp to most_tiles, keep any offsets in range.
__device__ __forceinline__ int64_t scan_tiles(const int *offsets, int groups, int rows, int bm, int g0,
                                              int &begin, int &end, int &tiles)
{
    const int lane = threadIdx.x & 63;
    begin = end = 0;
    if (g0 + lane < groups) group_rows(offsets, g0 + lane, rows, begin, end);
    tiles = (int)(((int64_t)end - begin + bm - 1) / bm);
    int64_t sum = tiles;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t v = __shfl_up((long long)sum, d);
        if (lane >= d) sum += v;
    }
    return sum;  // inclusive
}

template <typename T, int BM, int BN, int WM, int WN, int NBUF, Layout LA, Layout LB, Ragged RG,
          Epilogue EP, bool FAST>
__global__ void __launch_bounds__(WM *WN * 64) tile_kernel(TileArgs g)
{
    using SA = Slab<T, BM, LA>;
    using SB = Slab<T, BN, LB>;
    using Frag = typename Elem<T>::Frag;
    constexpr int BK = Elem<T>::BK, EPC = Elem<T>::EPC, SZ = sizeof(T);
    constexpr int NW = WM * WN;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int U = SA::UNITS + SB::UNITS;
    constexpr int LPW = (U + NW - 1) / NW;  // units a wave loads per slab (some twice, the same data)
    constexpr int STAGE = SA::BYTES + SB::BYTES;
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "wave tiles are 16-aligned");
    static_assert(LPW * (NBUF - 1) <= 63, "loads in flight must fit the vmcnt field");
    static_assert(FAST || NBUF == 2, "the register path alternates two buffers");
    static_assert(EP != STATS || WN * BM * 8 <= NBUF * STAGE, "row statistics fit the ring");
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l15 = lane & 15, lg = lane >> 4;

    // ---- which tile, of which group
    int tm, tn, group = 0, begin = 0, end = 0, m0;
    if constexpr (RG == ROWS) {
        int b, e, n;
        int64_t all = 0;
        for (int g0 = 0; g0 < g.groups; g0 += 64)
            all += __shfl((long long)scan_tiles(g.offsets, g.groups, g.M, BM, g0, b, e, n), 63);
        const int total = (int)(all < g.most_tiles ? all : g.most_tiles);
        const int tiles_n = (g.N + BN - 1) / BN;
        if ((int64_t)blockIdx.x >= (int64_t)total * tiles_n) return;
        tile_of_block(blockIdx.x, total, tiles_n, 8, tm, tn);
        int64_t before = 0;
        for (int g0 = 0; g0 < g.groups; g0 += 64) {
            const int64_t sum = scan_tiles(g.offsets, g.groups, g.M, BM, g0, b, e, n);
            const uint64_t past = __ballot(before + sum > tm);
            if (past) {
                const int at = __builtin_ctzll(past);
                group = g0 + at;
                begin = __shfl(b, at);
                end = __shfl(e, at);
                tm -= (int)(before + __shfl((long long)sum, at) - __shfl(n, at));
                break;
            }
            before += __shfl((long long)sum, 63);
        }
        group = __builtin_amdgcn_readfirstlane(group);
        begin = __builtin_amdgcn_readfirstlane(begin);
        end = __builtin_amdgcn_readfirstlane(end);
        tm = __builtin_amdgcn_readfirstlane(tm);
    } else {
        const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN;
        int bid = blockIdx.x;
        if constexpr (RG == SUM) {
            const int per = tiles_m * tiles_n;
            group = bid / per;
            bid -= group * per;
            group_rows(g.offsets, group, g.K, begin, end);
            begin = __builtin_amdgcn_readfirstlane(begin);
            end = __builtin_amdgcn_readfirstlane(end);
        }
        tile_of_block(bid, tiles_m, tiles_n, 8, tm, tn);
    }
    m0 = tm * BM;
    const int n0 = tn * BN;

    // ---- where the operands start, and how many bytes follow
    int K = g.K, kb = 0;  // contraction of this tile, and where it starts
    if constexpr (RG == SUM) K = end - begin;
    if constexpr (EP == PART) {
        kb = blockIdx.z * g.split_k;
        const int k1 = kb + g.split_k;
        K = (k1 < K ? k1 : K) - kb;
        if (K < 0) K = 0;
    }
    const int row0 = RG == ROWS ? begin : 0;          // of A and C
    const int sum0 = RG == SUM ? begin : kb;          // first contraction index
    const char *pa = static_cast<const char *>(g.A);
    const char *pb = static_cast<const char *>(g.B);
    if constexpr (RG == ROWS) pb += group * g.group_stride * SZ;
    int64_t left_a, left_b;  // bytes from the tile's first value to the operand's end
    // Rows the operands have from there on; the KC ones of A end with the group,
    // whose later rows belong to the next one and are not stored here.
    const int a_rows = LA == KC ? (RG == ROWS ? end - begin - m0 : g.M - m0) : K;
    int b_rows = g.N - n0;
    if constexpr (LB == MC) {
        b_rows = K;
        if constexpr (RG != SUM) b_rows = g.b_rows - kb < K ? g.b_rows - kb : K;
    }
    if constexpr (LA == KC) {
        pa += ((int64_t)(row0 + m0) * g.lda + sum0) * SZ;
        left_a = ((int64_t)(a_rows - 1) * g.lda + (g.a_cols - sum0)) * SZ;
    } else {
        pa += ((int64_t)sum0 * g.lda + m0) * SZ;
        left_a = ((int64_t)(a_rows - 1) * g.lda + (g.a_cols - m0)) * SZ;
        if (a_rows <= 0) left_a = 0;
    }
    if constexpr (LB == KC) {
        pb += ((int64_t)n0 * g.ldb + sum0) * SZ;
        left_b = ((int64_t)(b_rows - 1) * g.ldb + (g.b_cols - sum0)) * SZ;
    } else {
        pb += ((int64_t)sum0 * g.ldb + n0) * SZ;
        left_b = ((int64_t)(b_rows - 1) * g.ldb + (g.b_cols - n0)) * SZ;
        if (b_rows <= 0) left_b = 0;
    }
    const int64_t step_a = LA == KC ? 128 : (int64_t)BK * g.lda * SZ;
    const int64_t step_b = LB == KC ? 128 : (int64_t)BK * g.ldb * SZ;
    const int slabs = (K + BK - 1) / BK;

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int wr = wave / WN, wc = wave % WN;
    auto compute = [&](const char *buf) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Frag a[FM], b[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) b[j] = SB::frag(buf + SA::BYTES, wc * FN + j, h, lane);
#pragma unroll
            for (int i = 0; i < FM; ++i) a[i] = SA::frag(buf, wr * FM + i, h, lane);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma_step<T>(b[j], a[i], acc[i][j]);
        }
    };

    // Unit i of this wave fills chunks 64 u .. 64 u + 63 of the slab, A's first.
    int urow[LPW], uchunk[LPW], uat[LPW];
    bool ua[LPW];
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
        int u = wave + i * NW;
        if ((i + 1) * NW > U && u >= U) u -= U;  // another wave's unit: the same bytes again
        ua[i] = (i + 1) * NW <= SA::UNITS || ((i * NW < SA::UNITS || (i + 1) * NW > U) && u < SA::UNITS);
        uat[i] = u * 1024;
        if (ua[i])
            SA::slot(u * 64 + lane, urow[i], uchunk[i]);
        else
            SB::slot((u - SA::UNITS) * 64 + lane, urow[i], uchunk[i]);
    }

    if constexpr (FAST) {
        uint32_t voff[LPW];
#pragma unroll
        for (int i = 0; i < LPW; ++i)
            voff[i] = (uint32_t)urow[i] * (uint32_t)((ua[i] ? g.lda : g.ldb) * SZ) +
                      (uint32_t)uchunk[i] * 16u;
        const uint32_t base = (uint32_t)(uintptr_t)(lds_char *)lds;
        int kleft = K;  // of the next slab to issue
        auto issue = [&](int buf) {
            const u32x4 ra = descriptor(pa, LA == MC ? left_a : kleft > 0 ? left_a : 0);
            const u32x4 rb = descriptor(pb, LB == MC ? left_b : kleft > 0 ? left_b : 0);
            const uint32_t at = base + (uint32_t)buf * STAGE;
#pragma unroll
            for (int i = 0; i < LPW; ++i) {
                uint32_t v = voff[i];
                if ((ua[i] ? LA : LB) == KC && kleft < BK && uchunk[i] * EPC >= kleft) v = kOutside;
                if (ua[i])
                    load_slab16(ra, v, at + uat[i]);
                else
                    load_slab16(rb, v, at + uat[i]);
            }
            pa += step_a;
            pb += step_b;
            left_a -= step_a;
            left_b -= step_b;
            kleft -= BK;
        };
#pragma unroll
        for (int i = 0; i < NBUF - 1; ++i) issue(i);
        int buf = 0;
        for (int t = 0; t < slabs; ++t) {
            // Slab t has landed; every wave is done with slab t - 1, whose buffer
            // slab t + NBUF - 1 now fills.
            wait_slab_barrier<LPW *(NBUF - 2)>();
            issue(buf == 0 ? NBUF - 1 : buf - 1);
            compute(lds + buf * STAGE);
            buf = buf + 1 == NBUF ? 0 : buf + 1;
        }
        wait_slab_barrier<0>();  // nothing may land in LDS any more
    } else {
        u32x4 hold[LPW];
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < LPW; ++i) {
                const bool kc = (ua[i] ? LA : LB) == KC;
                const int64_t ld = ua[i] ? g.lda : g.ldb;
                const int rows = ua[i] ? a_rows : b_rows;
                const int r = kc ? urow[i] : t * BK + urow[i];
                const int c = kc ? t * BK + uchunk[i] * EPC : uchunk[i] * EPC;
                // First value outside, along the contiguous index.
                const int lim = kc ? K : ua[i] ? g.M - m0 : g.N - n0;
                const T *p = reinterpret_cast<const T *>(ua[i] ? pa : pb) + (int64_t)r * ld + c;
                union {
                    u32x4 v;
                    T e[EPC];
                } x;
                x.v = u32x4{0, 0, 0, 0};
                if (r < rows) {
                    if (c + EPC <= lim) {
                        __builtin_memcpy(&x, p, 16);
                    } else {
#pragma unroll
                        for (int j = 0; j < EPC; ++j)
                            if (c + j < lim) x.e[j] = p[j];
                    }
                }
                hold[i] = x.v;
            }
        };
        auto put = [&](int buf) {
#pragma unroll
            for (int i = 0; i < LPW; ++i)
                *reinterpret_cast<u32x4 *>(lds + buf * STAGE + uat[i] + lane * 16) = hold[i];
        };
        if (slabs > 0) {
            fetch(0);
            put(0);
        }
        __syncthreads();
        for (int t = 0; t < slabs; ++t) {
            if (t + 1 < slabs) fetch(t + 1);
            compute(lds + (t & 1) * STAGE);
            if (t + 1 < slabs) put((t + 1) & 1);
            __syncthreads();
        }
    }

    // ---- epilogue
    const int row_end = RG == ROWS ? end - begin : g.M;
    const int mw = m0 + wr * (BM / WM) + l15;       // row of block 0
    const int nw = n0 + wc * (BN / WN) + 4 * lg;    // first of its four columns in block 0
    if constexpr (EP == STORE) {
        T *C = static_cast<T *>(g.C);
        if constexpr (RG == SUM) C += group * g.group_stride;
        const float alpha = g.alpha, beta = g.beta;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int m = mw + 16 * i;
            if (m >= row_end) continue;
            T *crow = C + (int64_t)(row0 + m) * g.ldc;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n = nw + 16 * j;
                if (n >= g.N) continue;
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = alpha * acc[i][j][q];
                if (g.vec_c && n + 4 <= g.N) {
                    typedef T Vec __attribute__((ext_vector_type(4)));
                    Vec *p = reinterpret_cast<Vec *>(crow + n);
                    if (beta != 0.f) {
                        const Vec old = *p;
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] = fmaf(beta, (float)old[q], v[q]);
                    }
                    Vec out;
#pragma unroll
                    for (int q = 0; q < 4; ++q) out[q] = (T)v[q];
                    *p = out;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (n + q < g.N) {
                            if (beta != 0.f) v[q] = fmaf(beta, (float)crow[n + q], v[q]);
                            crow[n + q] = (T)v[q];
                        }
                }
            }
        }
    } else if constexpr (EP == PART) {
        float *C = static_cast<float *>(g.C) + blockIdx.z * g.slice_stride;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int m = mw + 16 * i;
            if (m >= g.M) continue;
            float *crow = C + (int64_t)m * g.ldc;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n = nw + 16 * j;
                if (n >= g.N) continue;
                if (g.vec_c && n + 4 <= g.N) {
                    f32x4 *p = reinterpret_cast<f32x4 *>(crow + n);
                    *p = g.accumulate ? acc[i][j] + *p : acc[i][j];
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (n + q < g.N)
                            crow[n + q] = g.accumulate ? acc[i][j][q] + crow[n + q] : acc[i][j][q];
                }
            }
        }
    } else if constexpr (EP == GRAD) {
        T *C = static_cast<T *>(g.C);
        // Columns up to the next multiple of 8 are written (as zero past N), so
        // that whole chunks can be read back.
        const int ncols = (g.N + 7) & ~7;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int m = mw + 16 * i;
            if (m >= g.M) continue;
            const int64_t target = g.targets[m];
            const float lse = g.lse[m], w = g.dloss[m];
            const bool counts = target >= 0 && target < g.vocab;
            const int at = counts ? (int)target - g.col0 : -1;  // past the piece: no column's
            T *crow = C + (int64_t)m * g.ldc;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n = nw + 16 * j;
                if (n >= ncols) continue;
                typedef T Vec __attribute__((ext_vector_type(4)));
                Vec out;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float z = acc[i][j][q] - lse;
                    float p;
                    if constexpr (std::is_same<T, float>::value)
                        p = expf(z);
                    else
                        p = __expf(z);
                    if (n + q == at) p -= 1.f;
                    out[q] = (T)(counts && n + q < g.N ? p * w : 0.f);
                }
                *reinterpret_cast<Vec *>(crow + n) = out;
            }
        }
    }
    if constexpr (EP == STATS) {
        // Row maximum and sum over this wave's columns, then over the waves of
        // the tile through LDS.  The sums are of exponentials of the distance to
        // the running maximum, so nothing overflows.
        float *sm = reinterpret_cast<float *>(lds), *ss = sm + WN * BM;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int m = mw + 16 * i;
            const int64_t target = m < g.M ? g.targets[m] : -1;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = nw + 16 * j + q;
                    if (n >= g.N) continue;
                    top = fmaxf(top, acc[i][j][q]);
                    if (target == n) g.target_value[m] = acc[i][j][q];
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            // Without a finite maximum the distance is taken to zero: infinities and
            // NaN then reach the sum as they are.
            const float from = isfinite(top) ? top : 0.f;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = nw + 16 * j + q;
                    if (n < g.N) sum += expf(acc[i][j][q] - from);
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lg == 0) {
                sm[wc * BM + m - m0] = top;
                ss[wc * BM + m - m0] = sum;
            }
        }
        __syncthreads();
        for (int r = threadIdx.x; r < BM; r += NW * 64) {
            if (m0 + r >= g.M) continue;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < WN; ++w) top = fmaxf(top, sm[w * BM + r]);
            const float from = isfinite(top) ? top : 0.f;
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                const float t = sm[w * BM + r];
                sum += ss[w * BM + r] * (t == top || !isfinite(t) ? 1.f : expf(t - from));
            }
            f32x2 *part = reinterpret_cast<f32x2 *>(g.parts) +
                          ((int64_t)(m0 + r) * ((g.N + BN - 1) / BN) + tn);
            *part = f32x2{top, sum};
        }
    }
}

}  // namespace lm
}  // namespace sgemm
