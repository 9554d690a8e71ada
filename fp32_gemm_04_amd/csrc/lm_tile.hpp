// Tile kernels of the language-model products (include/slm.h): fp32 or bf16
// operands with fp32 accumulation, or 8-bit integers with 32-bit sums; three operand
// layouts, ragged rows or a ragged contraction, and the epilogues the products need.
//
// One workgroup computes a BM x BN tile of C = A B^T, where A has BM rows and
// B has BN rows (the columns of C), both walked along the contraction in
// slabs of 128 bytes (BK = 128 integers, 64 bf16 or 32 fp32).  An operand comes in one of
// two layouts in memory:
//   KC  the contraction index is contiguous: a slab row is 128 bytes of it;
//   MC  the row index is contiguous: the slab is BK rows of BM (or BN) values.
//
// A slab travels from memory to an LDS ring of NBUF buffers with
// buffer_load_dwordx4 ... lds (the wave's 64 x 16 bytes land in lane order),
// so no registers hold it.  The addresses need 4-byte alignment only, and the buffer
// descriptor, which checks each 4 bytes, ends where the operand ends: what lies past
// the end reads as zero without any per-lane test, and a slab issued past the last one
// touches no memory, so the ring needs no special tail.  Only in the last slab of a KC
// operand whose K is not a multiple of BK do lanes past K leave the descriptor's range,
// and where K is no multiple of a chunk its values past K are cleared in LDS.
// bf16 operands with rows at odd addresses (FAST false) go through registers, each
// value tested against the operand's ends.
//
// LDS layouts, in 16-byte chunks; the permutation is applied to which chunk a
// lane fetches, since the DMA writes lanes in order:
// LDS has 64 banks of four bytes; a read is conflict-free when the lanes of each
// 256 bytes of it meet all banks:
//   KC: row r holds its 8 chunks at places p = c ^ (r / 2 & 7): the 16 lanes that
//       read one chunk of 16 rows (two rows per 256 bytes) meet 16 places.
//   MC: slab row k holds chunk c at p = c ^ swizzle(k).  bf16 operands are
//       read with ds_read_b64_tr_b16, which hands a lane four consecutive k
//       of one column: 16 lanes read 32 bytes of each of 4 rows.  With BL = 16 the two
//       halves of 32 lanes are 8 rows apart, so 8 rows must differ in their 32-byte
//       place; with BL = 32 they are neighbours, so 4 rows in their 64-byte place.
//       fp32 operands (BL = 16) need one k per lane and step: the lane groups read 64
//       bytes of rows 4 apart.
//
// Both operands of a matrix instruction use the same assignment of k to lanes.
// With blocks of BL = 16 and g = lane / 16, bf16 16x16x32 takes k = 8 g .. 8 g + 7, and
// four fp32 16x16x4 steps s = 0..3 take k = 4 g + s; with BL = 32 and g = lane / 32, two
// bf16 32x32x16 cover the same half slab.  The larger block
// halves the instructions a wave issues, which the largest tile needs: its
// accumulators leave one wave per SIMD.  8-bit integers take 16 bytes of k where bf16 takes
// eight values, so their slabs, addresses and reads of LDS are those of bf16 KC operands.
// B is the instruction's first operand, so
// a lane holds groups of four consecutive columns of one row of C:
//   row lane % BL, columns 4 g .. 4 g + 3 (BL = 32: and 8, 16, 24 further on).
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
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum Layout { KC, MC };
// PLAIN: one product.  ROWS: the rows of A and C fall into groups, each with a
// B of its own.  SUM: the contraction falls into groups, each with a C of its own.
enum Ragged { PLAIN, ROWS, SUM };
// STORE: C <- alpha acc + beta C.  STATS: row maxima and sums of exponentials of
// the tile, and the value at the row's target.  GRAD: the loss's derivative by
// each value.  PART: fp32 C <- acc (+ C), for sums joined later.  SCALE: C <- acc times
// its row's and its column's scale.
enum Epilogue { STORE, STATS, GRAD, PART, SCALE };

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
    int vec_c;                   // C's rows take stores of 4 values (1), or of 8 bf16 (2)
    int accumulate;              // PART: add to what is there
    int split_k;                 // PART: contraction per z-slice (multiple of the slab)
    int64_t slice_stride;        // PART: elements between slices of C
    // Cross entropy: rows are tokens, columns the vocabulary from col0 on.
    const int64_t *targets;
    const float *lse, *dloss;
    float *parts;                // STATS: (maximum, sum) of [row][tile along N]
    float *target_value;
    int col0, vocab;
    // GRAD, split: rows written (those from M on as zeros), and the distance in rows to
    // what rounding each derivative to bf16 leaves over, written as rows of their own (0:
    // not kept).  Sums over both (A MC): B starts over after `wrap` rows, a power of two
    // below a slab's rows or a multiple of them (0: never).
    int store_rows, low_rows;
    int wrap;
    // SCALE: of each row of A, and of each row of B (N of one group after another's).
    const float *scale_a, *scale_b;
    int fill;                    // SCALE, ROWS: rows outside every group are set to zero
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
template <> struct Elem<int8_t> {
    static constexpr int BK = 128, EPC = 16;
    typedef i32x4 Frag;
};

// Lane l's 16 bytes at base + voff go to LDS [lds + 16 l, + 16); zeros where
// voff lies outside the descriptor.  s_nop: an LDS DMA needs a wait state after
// the write of M0.
__device__ __forceinline__ void load_slab16(u32x4 rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\t"
                 "buffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(lds)
                 : "memory", "m0");
}

// voff leaves every descriptor's range unless k < left.  In assembly, like the loads that
// hold voff: compiled code never touches an address register while a load is in flight.
__device__ __forceinline__ void leave_range(uint32_t &voff, int k, int left)
{
    asm volatile("v_cmp_gt_i32_e32 vcc, %2, %1\n\ts_nop 1\n\t"
                 "v_cndmask_b32_e32 %0, %3, %0, vcc"
                 : "+v"(voff)
                 : "v"(k), "s"(left), "v"(0x80000000u)
                 : "vcc");
}

template <int N>
__device__ __forceinline__ void wait_slab_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

constexpr float kLog2e = 1.44269504088896340736f;

// (top, sum) stands for sum * 2^top: (top, sum) += (t, s).  A side whose top is not
// finite has an empty sum (top -inf), or one that is infinite or NaN whatever it is
// scaled by, and is taken as it is.
__device__ __forceinline__ void join_sums(float &top, float &sum, float t, float s)
{
    const float m = fmaxf(top, t);
    const float a = top == m || !isfinite(top) ? 1.f : __builtin_amdgcn_exp2f(top - m);
    const float b = t == m || !isfinite(t) ? 1.f : __builtin_amdgcn_exp2f(t - m);
    sum = sum * a + s * b;
    top = m;
}

constexpr uint32_t kOutside = 0x80000000u;  // beyond every descriptor's range

// A descriptor of the bytes [p, p + left), at most 2^31 of them.
__device__ __forceinline__ u32x4 descriptor(const char *p, int64_t left)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    // Whole words: the last may end past the operand (never past a word it has part of).
    const uint32_t n =
        left <= 0 ? 0u : left > (int64_t)kOutside ? kOutside : ((uint32_t)left + 3u) & ~3u;
    u32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xffffu;
    r[2] = __builtin_amdgcn_readfirstlane(n);
    r[3] = 0x00020000u;
    return r;
}

// One operand's slabs: where this wave's units (64 chunks each) come from.
template <typename T, int B, Layout L, int BL>
struct Slab {
    static constexpr int BK = Elem<T>::BK, EPC = Elem<T>::EPC;
    static constexpr int UNITS = B / 8;            // 64-chunk units per slab
    static constexpr int BYTES = B * 128;
    static constexpr int RC = B / EPC;             // MC: chunks per slab row

    // Rows of a multiple of 256 bytes all start in bank 0; rows of an odd multiple of 128
    // alternate between two halves by themselves, and their chunks stay inside 128 bytes.
    __device__ static __forceinline__ int swizzle(int k)
    {
        static_assert(L == KC || RC % 8 == 0 || RC <= 4, "a slab row is whole 128-byte groups");
        constexpr bool WHOLE = RC % 16 == 0;
        if constexpr (RC <= 4)
            return 0;
        else if constexpr (std::is_same<T, float>::value) {
            static_assert(BL == 16, "fp32 operands are read in blocks of 16");
            // (128-byte rows have room for two places only: reads in pairs.)
            return WHOLE ? 4 * ((k >> 2) & 3) : 4 * ((k >> 2) & 1);
        } else if constexpr (BL == 32) {
            return WHOLE ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
        } else {
            return WHOLE ? 2 * ((k & 3) + ((k >> 1) & 4)) : 2 * (((k >> 1) & 1) + ((k >> 2) & 2));
        }
    }
    // Row (KC: of the tile; MC: of the slab) and chunk that slot s fetches.
    __device__ static __forceinline__ void slot(int s, int &row, int &chunk)
    {
        if constexpr (L == KC) {
            row = s >> 3;
            chunk = (s & 7) ^ ((row >> 1) & 7);
        } else {
            row = s / RC;
            chunk = (s % RC) ^ swizzle(row);
        }
    }
    // The operand fragment of BL-row block blk, step k of 128 / (8 BL) in the slab.
    __device__ static __forceinline__ typename Elem<T>::Frag frag(const char *buf, int blk, int k,
                                                                  int lane)
    {
        constexpr int G = 64 / BL;                    // lane groups: chunks a step takes
        const int l = lane & (BL - 1), g = lane / BL;
        if constexpr (L == KC) {
            const char *p = buf + blk * (BL * 128) + l * 128 + (((G * k + g) ^ ((l >> 1) & 7)) << 4);
            return *reinterpret_cast<const typename Elem<T>::Frag *>(p);
        } else if constexpr (std::is_same<T, float>::value) {
            f32x4 v;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int row = 4 * (G * k + g) + s;
                const int c = (blk * (BL / 4) + (l >> 2)) ^ swizzle(row);
                v[s] = *reinterpret_cast<const float *>(buf + row * (B * 4) + c * 16 + (l & 3) * 4);
            }
            return v;
        } else {
            bf16x8 v;
            const int i = lane & 15;                  // the transposing read works on 16 lanes
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int row = 8 * (G * k + g) + 4 * s + (i >> 2);
                const int c = (blk * (BL / 8) + (l >> 4) * 2 + ((i >> 1) & 1)) ^ swizzle(row);
                const uint32_t at = (uint32_t)(uintptr_t)(const lds_char *)buf + row * (B * 2) +
                                    c * 16 + (i & 1) * 8;
                const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4 *)(uintptr_t)at);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * s + j] = __builtin_bit_cast(bf16, (short)q[j]);
            }
            return v;
        }
    }
};

typedef float f32x16 __attribute__((ext_vector_type(16)));
template <typename T, int BL> struct AccOf { typedef f32x4 Type; };
template <typename T> struct AccOf<T, 32> { typedef f32x16 Type; };
template <> struct AccOf<int8_t, 16> { typedef i32x4 Type; };
template <> struct AccOf<int8_t, 32> { typedef i32x16 Type; };

template <typename T, int BL>
__device__ __forceinline__ typename AccOf<T, BL>::Type mfma_step(const typename Elem<T>::Frag &b,
                                                                 const typename Elem<T>::Frag &a,
                                                                 typename AccOf<T, BL>::Type c)
{
    if constexpr (std::is_same<T, float>::value) {
        static_assert(BL == 16, "fp32 tiles have blocks of 16");
#pragma unroll
        for (int s = 0; s < 4; ++s)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(b[s], a[s], c, 0, 0, 0);
        return c;
    } else if constexpr (std::is_same<T, int8_t>::value) {
        if constexpr (BL == 16)
            return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, c, 0, 0, 0);
    } else if constexpr (BL == 16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
    }
}

// p[i], a scalar load where i is the wave's (no output of these kernels overlaps an input).
template <bool UNIFORM, typename T> __device__ __forceinline__ T read(const T *p, int64_t i)
{
    if constexpr (UNIFORM)
        return ((const __attribute__((address_space(4))) T *)(uintptr_t)p)[i];
    else
        return p[i];
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

// Rows of C outside increasing groups are set to zero, each by one of all workgroups along x.
template <typename TC>
__device__ __forceinline__ void zero_outside(const int *offsets, int groups, int rows, int N, TC *C,
                                             int64_t ldc)
{
    const int low = clamp_row(offsets[0], 0, rows), high = clamp_row(offsets[groups], low, rows);
    for (int64_t i = blockIdx.x; i < (int64_t)low + rows - high; i += gridDim.x) {
        TC *c = C + (i < low ? i : high + i - low) * ldc;
        for (int n = threadIdx.x; n < N; n += blockDim.x) c[n] = (TC)0.f;
    }
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

// The workgroup's tile of its group, and the group's rows; false where there is none for it.
__device__ __forceinline__ bool rows_tile_of_block(const TileArgs &g, int bm, int bn, int band, int &tm,
                                                   int &tn, int &group, int &begin, int &end)
{
    // (Up to 64 groups are counted once: a tile's first loads wait for this.)
    int b, e, n;
    int64_t sum = scan_tiles(g.offsets, g.groups, g.M, bm, 0, b, e, n);
    int64_t all = __shfl((long long)sum, 63);
    for (int g0 = 64; g0 < g.groups; g0 += 64) {
        int b1, e1, n1;
        all += __shfl((long long)scan_tiles(g.offsets, g.groups, g.M, bm, g0, b1, e1, n1), 63);
    }
    const int total = (int)(all < g.most_tiles ? all : g.most_tiles);
    const int tiles_n = (g.N + bn - 1) / bn;
    if ((int64_t)blockIdx.x >= (int64_t)total * tiles_n) return false;
    tile_of_block(blockIdx.x, total, tiles_n, band, tm, tn);
    int64_t before = 0;
    for (int g0 = 0; g0 < g.groups; g0 += 64) {
        if (g0 > 0) sum = scan_tiles(g.offsets, g.groups, g.M, bm, g0, b, e, n);
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
    return true;
}

// Row tiles that an XCD's neighbouring workgroups walk a column of before the next column.  8-bit
// operands: us with 8, 4 and 2, 8192 x 4096 x 14336 451, 447 and 455, 4096 x 4096 x 4096 70.3, 65.8 and
// 66.2; by group with 8, 3 and 1, 16384 rows on 64 experts' 2048 x 1536 101, 99 and 98, 32768 rows 163, 158
// and 161, 8192 rows on eight experts' 4096 x 2048 99, 95 and 95.
constexpr int byte_band(bool grouped)
{
    return grouped ? 3 : 4;
}

// WM x WN waves share the tile, NBUF slabs the ring; WPE waves per SIMD bound the registers.
// What bounds it: the matrix cores where tiles have many rows (256 x 256, T 8192, H 2048, V
// 131072: logits to row statistics 3.70-3.85 ms, 1140-1190 TF/s, the cores 56% busy at 2.0
// GHz; derivatives 503-519 us a piece of 16384 columns, dW and dX 453-468; fp32 128 x 128,
// T 1023, H 1000, V 49999: 794-817 us a product, 126-129 TF/s), memory where they have few
// (16 x 64, 24 rows on 14 experts' 2048 x 1408 weights: 17.4 us, 4.6 TB/s).
// Why this form: slabs of 128 bytes, since 64 with twice the buffers doubled the barriers
// and were slower; operands half a slab ahead, so that reads of LDS hide behind products
// of one wave per SIMD; no workgroup stays for a second tile (no gain, and the 256 tile
// spilled).  Two forms of the 256 tile spill outside their loops: row statistics 32
// registers (written with them: 302 MB instead of 34 at T 8192, V 131072), partial sums 8.
template <typename T, int BM, int BN, int WM, int WN, int NBUF, int BL, int WPE, Layout LA,
          Layout LB, Ragged RG, Epilogue EP, bool FAST, typename TC = T>
__global__ void __launch_bounds__(WM *WN * 64) __attribute__((amdgpu_waves_per_eu(WPE)))
tile_kernel(TileArgs g)
{
    using SA = Slab<T, BM, LA, BL>;
    using SB = Slab<T, BN, LB, BL>;
    using Frag = typename Elem<T>::Frag;
    constexpr int BK = Elem<T>::BK, EPC = Elem<T>::EPC, SZ = sizeof(T);
    constexpr int NW = WM * WN;
    constexpr int FM = BM / WM / BL, FN = BN / WN / BL;  // blocks of a wave
    constexpr int KS = BL / 16;                           // steps per half slab
    constexpr int U = SA::UNITS + SB::UNITS;
    constexpr int LPW = (U + NW - 1) / NW;  // units a wave loads per slab (some twice, the same data)
    constexpr int STAGE = SA::BYTES + SB::BYTES;
    static_assert(BM % (BL * WM) == 0 && BN % (BL * WN) == 0, "wave tiles are whole blocks");
    static_assert(LPW * (NBUF - 1) <= 63, "loads in flight must fit the vmcnt field");
    static_assert(FAST || NBUF == 2, "the register path alternates two buffers");
    static_assert(EP != STATS || WN * BM * 8 <= NBUF * STAGE, "row statistics fit the ring");
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lrow = lane & (BL - 1), lg = lane / BL;

    // ---- which tile, of which group
    constexpr int BAND = std::is_same<T, int8_t>::value ? byte_band(RG == ROWS) : 8;
    int tm, tn, group = 0, begin = 0, end = 0, m0;
    if constexpr (RG == ROWS) {
        if (!rows_tile_of_block(g, BM, BN, BAND, tm, tn, group, begin, end)) {
            if constexpr (EP == SCALE)
                if (g.fill) zero_outside(g.offsets, g.groups, g.M, g.N, static_cast<TC *>(g.C), g.ldc);
            return;
        }
    } else {
        const int tiles_m = ((EP == GRAD ? g.store_rows : g.M) + BM - 1) / BM;
        const int tiles_n = (g.N + BN - 1) / BN;
        int bid = blockIdx.x;
        if constexpr (RG == SUM) {
            const int per = tiles_m * tiles_n;
            group = bid / per;
            bid -= group * per;
            group_rows(g.offsets, group, g.K, begin, end);
            begin = __builtin_amdgcn_readfirstlane(begin);
            end = __builtin_amdgcn_readfirstlane(end);
        }
        tile_of_block(bid, tiles_m, tiles_n, BAND, tm, tn);
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

    typename AccOf<T, BL>::Type acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < BL * BL / 64; ++q) acc[i][j][q] = 0;

    const int wr = wave / WN, wc = wave % WN;
    // Operand read r of half slab h: step by step, the wave's B blocks, then its A blocks.
    constexpr int R1 = FM + FN, R = R1 * KS, M = FM * FN * KS;
    auto read_op = [&](int r, const char *buf, int h, Frag(&a)[KS][FM], Frag(&b)[KS][FN]) {
        const int k = r / R1, i = r % R1;
        if (i < FN)
            b[k][i] = SB::frag(buf + SA::BYTES, wc * FN + i, h * KS + k, lane);
        else
            a[k][i - FN] = SA::frag(buf, wr * FM + i - FN, h * KS + k, lane);
    };
    // The products of one half slab; hook(n) runs before the n-th of the M blocks.
    auto products = [&](const Frag(&a)[KS][FM], const Frag(&b)[KS][FN], auto hook) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    hook((k * FM + i) * FN + j);
                    acc[i][j] = mfma_step<T, BL>(b[k][j], a[k][i], acc[i][j]);
                }
    };

    // Unit i of this wave fills chunks 64 u .. 64 u + 63 of the slab, A's first.
    int uat[LPW];
    bool ua[LPW];
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
        int u = wave + i * NW;
        if ((i + 1) * NW > U && u >= U) u -= U;  // another wave's unit: the same bytes again
        ua[i] = (i + 1) * NW <= SA::UNITS || ((i * NW < SA::UNITS || (i + 1) * NW > U) && u < SA::UNITS);
        uat[i] = u * 1024;
    }
    // Row and chunk that this lane fetches in unit i.
    auto slot = [&](int i, int &row, int &chunk) {
        if (ua[i])
            SA::slot(uat[i] / 16 + lane, row, chunk);
        else
            SB::slot(uat[i] / 16 - SA::UNITS * 64 + lane, row, chunk);
    };

    if constexpr (FAST) {
        uint32_t voff[LPW];
#pragma unroll
        for (int i = 0; i < LPW; ++i) {
            int row, chunk;
            slot(i, row, chunk);
            if (RG == PLAIN && LA == MC && !ua[i] && g.wrap > 0 && g.wrap < BK) row &= g.wrap - 1;
            voff[i] = (uint32_t)row * (uint32_t)((ua[i] ? g.lda : g.ldb) * SZ) + (uint32_t)chunk * 16u;
        }
        const uint32_t base = (uint32_t)(uintptr_t)(lds_char *)lds;
        int kleft = K;  // of the next slab to issue
        int issued = 0;
        u32x4 ra, rb;
        auto next_slab = [&]() {  // descriptors of the slab whose loads come next
            ra = descriptor(pa, LA == MC ? left_a : kleft > 0 ? left_a : 0);
            rb = descriptor(pb, LB == MC ? left_b : kleft > 0 ? left_b : 0);
            if ((LA == KC || LB == KC) && kleft < BK) {
                // The last slab is part full (those after it fetch nothing): lanes whose
                // chunk lies past K leave the range of the descriptor for good.
                asm volatile("; part-full slab");  // a branch, not a select in every slab
#pragma unroll
                for (int i = 0; i < LPW; ++i) {
                    int row, chunk;
                    slot(i, row, chunk);
                    if ((ua[i] ? LA : LB) == KC) leave_range(voff[i], chunk * EPC, kleft);
                }
            }
            // Wait states between a vector unit's write of a descriptor and its use.
            asm volatile("s_nop 4" : "+s"(ra), "+s"(rb));
        };
        auto load = [&](int i, uint32_t at) {
            if (ua[i])
                load_slab16(ra, voff[i], at + uat[i]);
            else
                load_slab16(rb, voff[i], at + uat[i]);
        };
        auto advance = [&]() {
            pa += step_a;
            pb += step_b;
            left_a -= step_a;
            left_b -= step_b;
            kleft -= BK;
            if constexpr (RG == PLAIN && LA == MC) {
                if (++issued * BK == g.wrap) {
                    pb -= issued * step_b;
                    left_b += issued * step_b;
                }
            }
        };
        // Half a slab ahead: while the products of one half run, the operands of the
        // next are read.  In the middle of slab t every wave has read all of it, so
        // one barrier there both frees its buffer for slab t + NBUF and, after the
        // wait for this wave's loads, publishes slab t + 1.
#pragma unroll
        for (int b = 0; b < NBUF; ++b) {
            next_slab();
#pragma unroll
            for (int i = 0; i < LPW; ++i) load(i, base + (uint32_t)b * STAGE);
            advance();
        }
        // Values past K in the last slab's last chunk (KC: row r of an operand, MC: no
        // need, rows past K are past the descriptor).
        const int ragged = K % EPC;
        auto clear_tail = [&](char *slab) {
            auto clear = [&](char *rows, int count) {
                const int chunk = K % BK / EPC;
                for (int r = threadIdx.x; r < count; r += NW * 64) {
                    T *p = reinterpret_cast<T *>(rows + r * 128 + ((chunk ^ ((r >> 1) & 7)) << 4));
                    for (int j = ragged; j < EPC; ++j) p[j] = (T)0.f;
                }
            };
            if constexpr (LA == KC) clear(slab, BM);
            if constexpr (LB == KC) clear(slab + SA::BYTES, BN);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        };
        wait_slab_barrier<LPW *(NBUF - 1)>();
        if ((LA == KC || LB == KC) && ragged && slabs == 1) clear_tail(lds);
        Frag a0[KS][FM], b0[KS][FN], a1[KS][FM], b1[KS][FN];
#pragma unroll
        for (int r = 0; r < R; ++r) read_op(r, lds, 0, a0, b0);
        int buf = 0;
        for (int t = 0; t < slabs; ++t) {
            const char *here = lds + buf * STAGE;
            products(a0, b0, [&](int n) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (n == r * M / (2 * R)) {
                        read_op(r, here, 1, a1, b1);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            });
            __builtin_amdgcn_sched_barrier(0);
            wait_slab_barrier<LPW *(NBUF - 2)>();
            const uint32_t at = base + (uint32_t)buf * STAGE;
            buf = buf + 1 == NBUF ? 0 : buf + 1;
            char *there = lds + buf * STAGE;
            if ((LA == KC || LB == KC) && ragged && t + 2 == slabs) clear_tail(there);
            next_slab();
            products(a1, b1, [&](int n) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (n == r * M / (2 * R)) {
                        read_op(r, there, 0, a0, b0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                for (int i = 0; i < LPW; ++i)
                    if (n == i * M / LPW) {
                        load(i, at);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            });
            __builtin_amdgcn_sched_barrier(0);
            advance();
        }
        wait_slab_barrier<0>();  // nothing may land in LDS any more
    } else if constexpr (std::is_same<T, int8_t>::value) {
        // Rows at any byte: 16-byte loads into registers, two slabs ahead.  They are kept free of
        // branches but at the operand's end: rows past the last repeat it (and are not
        // stored), and values past K meet A's, which are cleared in the last slab.
        static_assert(LA == KC && LB == KC, "bytes are contiguous along the contraction");
        u32x4 hold0[LPW], hold1[LPW];
        const uint8_t *ends[2] = {reinterpret_cast<const uint8_t *>(pa) + left_a,
                                  reinterpret_cast<const uint8_t *>(pb) + left_b};
        const uint8_t *src[LPW];
        int at[LPW];
#pragma unroll
        for (int i = 0; i < LPW; ++i) {
            int row, chunk;
            slot(i, row, chunk);
            const int rows = ua[i] ? a_rows : b_rows;
            at[i] = chunk * EPC;
            src[i] = reinterpret_cast<const uint8_t *>(ua[i] ? pa : pb) +
                     (int64_t)(row < rows ? row : rows - 1) * (ua[i] ? g.lda : g.ldb) + at[i];
        }
        auto fetch = [&](int t, u32x4(&hold)[LPW]) {
            if (t >= slabs) return;
#pragma unroll
            for (int i = 0; i < LPW; ++i) {
                const uint8_t *p = src[i] + (int64_t)t * BK, *end = ends[ua[i] ? 0 : 1];
                if (p + 16 <= end) {
                    __builtin_memcpy(&hold[i], p, 16);
                } else {
                    hold[i] = u32x4{0, 0, 0, 0};
                    for (int j = 0; j < 16; ++j)
                        if (p + j < end) hold[i][j / 4] |= (uint32_t)p[j] << (8 * (j % 4));
                }
            }
        };
        auto put = [&](int t, u32x4(&hold)[LPW]) {
            if (t >= slabs) return;
            const bool last = t + 1 == slabs;
#pragma unroll
            for (int i = 0; i < LPW; ++i) {
                u32x4 v = hold[i];
                if (last && ua[i]) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int keep = K - t * BK - at[i] - 4 * w;  // bytes of this word
                        v[w] = keep >= 4 ? v[w] : keep <= 0 ? 0u : v[w] & ((1u << (8 * keep)) - 1u);
                    }
                }
                *reinterpret_cast<u32x4 *>(lds + (t & 1) * STAGE + uat[i] + lane * 16) = v;
            }
        };
        // Slab t runs; t + 1 is in flight in `next`; t + 2 goes where t was held.
        auto step = [&](int t, u32x4(&free)[LPW], u32x4(&next)[LPW]) {
            if (t >= slabs) return;
            fetch(t + 2, free);
            Frag a[KS][FM], b[KS][FN];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int r = 0; r < R; ++r) read_op(r, lds + (t & 1) * STAGE, h, a, b);
                products(a, b, [](int) {});
            }
            put(t + 1, next);
            __syncthreads();
        };
        fetch(0, hold0);
        fetch(1, hold1);
        put(0, hold0);
        __syncthreads();
        for (int t = 0; t < slabs; t += 2) {
            step(t, hold0, hold1);
            step(t + 1, hold1, hold0);
        }
    } else {
        u32x4 hold[LPW];
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < LPW; ++i) {
                int row, chunk;
                slot(i, row, chunk);
                const bool kc = (ua[i] ? LA : LB) == KC;
                const int64_t ld = ua[i] ? g.lda : g.ldb;
                const int rows = ua[i] ? a_rows : b_rows;
                int r = kc ? row : t * BK + row;
                if (RG == PLAIN && LA == MC && !ua[i] && g.wrap > 0) r %= g.wrap;
                const int c = kc ? t * BK + chunk * EPC : chunk * EPC;
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
            Frag a[KS][FM], b[KS][FN];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int r = 0; r < R; ++r) read_op(r, lds + (t & 1) * STAGE, h, a, b);
                products(a, b, [](int) {});
            }
            if (t + 1 < slabs) put((t + 1) & 1);
            __syncthreads();
        }
    }

    // ---- epilogue
    const int row_end = RG == ROWS ? end - begin : g.M;
    constexpr int GR = BL * BL / 256;               // groups of four columns in a block
    const int mw = m0 + wr * (BM / WM) + lrow;      // row of block 0
    const int nw = n0 + wc * (BN / WN) + 4 * lg;    // first column of group 0, block 0
    // Group u of the wave's FN * GR: its first column, and its values in row block i.
    auto column = [&](int u) { return nw + BL * (u / GR) + 8 * (u % GR); };
    auto value = [&](int i, int u, int q) { return acc[i][u / GR][4 * (u % GR) + q]; };
    typedef TC Vec __attribute__((ext_vector_type(4)));
    // bf16 blocks of 32: two neighbouring groups of a row lie in a lane pair (l, l + 32) as
    // columns 0-3, 8-11 and 4-7, 12-15; exchanged, each lane stores eight in a row, half as
    // many and twice as wide stores.
    constexpr bool PAIRED = BL == 32 && sizeof(TC) == 2;
    auto paired = [&](auto first, auto second) {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        if constexpr (sizeof(first) == sizeof(u32x2)) {
            const u32x2 x = __builtin_bit_cast(u32x2, first), y = __builtin_bit_cast(u32x2, second);
            const auto p = __builtin_amdgcn_permlane32_swap(x[0], y[0], false, false);
            const auto q = __builtin_amdgcn_permlane32_swap(x[1], y[1], false, false);
            return u32x4{p[0], q[0], p[1], q[1]};
        } else {
            return u32x4{};
        }
    };
    auto store_pair = [&](TC *crow, int u, auto first, auto second) {
        *reinterpret_cast<u32x4 *>(crow + column(u) + 4 * lg) = paired(first, second);
    };
    // A tile inside C with vector stores takes copies without per-column tests.
    const bool whole = n0 + BN <= g.N && g.vec_c >= (PAIRED ? 2 : 1);
    if constexpr (EP == STORE) {
        T *C = static_cast<T *>(g.C);
        if constexpr (RG == SUM) C += group * g.group_stride;
        // An empty contraction is 0 whatever alpha holds.
        const float alpha = K > 0 ? g.alpha : 0.f, beta = g.beta;
        auto store = [&](auto inside, auto scaled) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                __builtin_amdgcn_sched_barrier(0);  // one row block at a time: fewer registers
                const int m = mw + BL * i;
                if (m >= row_end) continue;
                T *crow = C + (int64_t)(row0 + m) * g.ldc;
                if constexpr (PAIRED && decltype(inside)::value) {
#pragma unroll
                    for (int u = 0; u < FN * GR; u += 2) {
                        Vec x, y;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            x[q] = (T)(alpha * value(i, u, q));
                            y[q] = (T)(alpha * value(i, u + 1, q));
                        }
                        store_pair(crow, u, x, y);
                    }
                    continue;
                }
#pragma unroll
                for (int u = 0; u < FN * GR; ++u) {
                    const int n = column(u);
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = alpha * value(i, u, q);
                    if (decltype(inside)::value || (g.vec_c && n + 4 <= g.N)) {
                        Vec *p = reinterpret_cast<Vec *>(crow + n);
                        if constexpr (decltype(scaled)::value) {
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
                                if constexpr (decltype(scaled)::value)
                                    v[q] = fmaf(beta, (float)crow[n + q], v[q]);
                                crow[n + q] = (T)v[q];
                            }
                    }
                }
            }
        };
        if (beta != 0.f)
            store(std::false_type{}, std::true_type{});
        else if (whole)
            store(std::true_type{}, std::false_type{});
        else
            store(std::false_type{}, std::false_type{});
    } else if constexpr (EP == SCALE) {
        // Sums below 2^31 become fp32 (half a step of 2^-24 relative), then two products and
        // one rounding to TC.  Vector stores need no more than an element's alignment.
        typedef Vec Loose __attribute__((aligned(sizeof(TC))));
        typedef u32x4 LoosePair __attribute__((aligned(2)));
        TC *C = static_cast<TC *>(g.C);
        const float *sb = g.scale_b + (int64_t)group * g.N;
        auto store = [&](auto inside) {
            f32x4 s[FN * GR];
#pragma unroll
            for (int u = 0; u < FN * GR; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    s[u][q] = decltype(inside)::value || column(u) + q < g.N ? sb[column(u) + q] : 0.f;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                const int m = mw + BL * i;
                if (m >= row_end) continue;
                TC *crow = C + (int64_t)(row0 + m) * g.ldc;
                const float sa = g.scale_a[row0 + m];
                Vec before;
#pragma unroll
                for (int u = 0; u < FN * GR; ++u) {
                    const int n = column(u);
                    Vec out;
#pragma unroll
                    for (int q = 0; q < 4; ++q) out[q] = (TC)((float)value(i, u, q) * sa * s[u][q]);
                    if constexpr (PAIRED && decltype(inside)::value) {
                        if (u % 2 == 0)
                            before = out;
                        else
                            *reinterpret_cast<LoosePair *>(crow + column(u - 1) + 4 * lg) = paired(before, out);
                    } else if (decltype(inside)::value || n + 4 <= g.N) {
                        *reinterpret_cast<Loose *>(crow + n) = out;
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (n + q < g.N) crow[n + q] = out[q];
                    }
                }
            }
        };
        if (n0 + BN <= g.N)
            store(std::true_type{});
        else
            store(std::false_type{});
        if constexpr (RG == ROWS)
            if (g.fill) zero_outside(g.offsets, g.groups, g.M, g.N, C, g.ldc);
    } else if constexpr (EP == PART) {
        float *C = static_cast<float *>(g.C) + blockIdx.z * g.slice_stride;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            const int m = mw + BL * i;
            if (m >= g.M) continue;
            float *crow = C + (int64_t)m * g.ldc;
#pragma unroll
            for (int u = 0; u < FN * GR; ++u) {
                const int n = column(u);
                if (whole || (g.vec_c && n + 4 <= g.N)) {
                    f32x4 *p = reinterpret_cast<f32x4 *>(crow + n);
                    f32x4 v;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = value(i, u, q);
                    *p = g.accumulate ? v + *p : v;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (n + q < g.N)
                            crow[n + q] =
                                g.accumulate ? value(i, u, q) + crow[n + q] : value(i, u, q);
                }
            }
        }
    } else if constexpr (EP == GRAD) {
        // Every value of the tile becomes w exp(z - lse), as 2^(z log2 e - lse log2 e): one
        // fma and one instruction for the power.  For fp32 the rounding of lse log2 e
        // is carried along (low); bf16's own rounding hides it.
        T *C = static_cast<T *>(g.C);
        auto store = [&](auto inside, auto split) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                const int m = mw + BL * i;
                if (m >= g.store_rows) continue;
                const int64_t target = m < g.M ? g.targets[m] : -1;
                const float w = m < g.M ? g.dloss[m] : 0.f, lse = m < g.M ? g.lse[m] : 0.f;
                const float high = lse * kLog2e, low = fmaf(lse, kLog2e, -high);
                const bool counts = target >= 0 && target < g.vocab;
                const int at = counts ? (int)target - g.col0 : -1;  // below every column: none
                T *crow = C + (int64_t)m * g.ldc;
                Vec before;
#pragma unroll
                for (int u = 0; u < FN * GR; ++u) {
                    const int n = column(u);
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float e = fmaf(value(i, u, q), kLog2e, -high);
                        if constexpr (std::is_same<T, float>::value) e -= low;
                        v[q] = __builtin_amdgcn_exp2f(e);
                    }
                    if ((unsigned)(at - n) < 4u)  // one lane of the row, in one tile
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] -= at - n == q ? 1.f : 0.f;
                    Vec out;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[q] = counts && (decltype(inside)::value || n + q < g.N) ? v[q] * w : 0.f;
                        out[q] = (T)v[q];
                    }
                    if constexpr (decltype(split)::value) {
                        Vec low;
#pragma unroll
                        for (int q = 0; q < 4; ++q) low[q] = (T)(v[q] - (float)out[q]);
                        if (n < ((g.N + 7) & ~7))
                            *reinterpret_cast<Vec *>(crow + g.low_rows * g.ldc + n) = low;
                    }
                    if constexpr (PAIRED && decltype(inside)::value) {
                        if (u % 2 == 0)
                            before = out;
                        else
                            store_pair(crow, u - 1, before, out);
                    } else if (decltype(inside)::value || n < ((g.N + 7) & ~7)) {
                        // Columns up to the next multiple of 8 are written, as zero past N,
                        // so that whole chunks can be read back.
                        *reinterpret_cast<Vec *>(crow + n) = out;
                    }
                }
            }
        };
        if constexpr (std::is_same<T, bf16>::value && BM * BN < 256 * 256) {
            if (g.low_rows) {
                store(std::false_type{}, std::true_type{});
                return;
            }
        }
        if (n0 + BN <= g.N)
            store(std::true_type{}, std::false_type{});
        else
            store(std::false_type{}, std::false_type{});
    }
    if constexpr (EP == STATS) {
        // Row maximum and sum over this wave's columns, then over the waves of the
        // tile through LDS, in powers of two: the sum is of 2^(z log2 e - top), top the
        // largest z log2 e of the row rounded, so nothing overflows and the pair (top,
        // sum) stands for top + log2(sum) without the rounding of top.
        float *sm = reinterpret_cast<float *>(lds), *ss = sm + WN * BM;
        if (n0 + BN > g.N) {  // columns past N never count
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int u = 0; u < FN * GR; ++u)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (column(u) + q >= g.N) acc[i][u / GR][4 * (u % GR) + q] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            const int m = mw + BL * i;
            const int64_t target = m < g.M ? g.targets[m] : -1;
            const int at = target >= 0 && target < g.N ? (int)target : -1;  // none
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < FN * GR; ++u) {
#pragma unroll
                for (int q = 0; q < 4; ++q) top = fmaxf(top, value(i, u, q));
                if ((unsigned)(at - column(u)) < 4u)  // one lane of the row, in one tile
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (at - column(u) == q) g.target_value[m] = value(i, u, q);
            }
#pragma unroll
            for (int d = BL; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
            top *= kLog2e;
            // Without a finite maximum the distance is taken to zero: infinities and
            // NaN then reach the sum as they are.
            const float from = isfinite(top) ? top : 0.f;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < FN * GR; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sum += __builtin_amdgcn_exp2f(fmaf(value(i, u, q), kLog2e, -from));
#pragma unroll
            for (int d = BL; d < 64; d *= 2) sum += __shfl_xor(sum, d);
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
            for (int w = 0; w < WN; ++w) join_sums(top, sum, sm[w * BM + r], ss[w * BM + r]);
            f32x2 *part = reinterpret_cast<f32x2 *>(g.parts) +
                          ((int64_t)(m0 + r) * ((g.N + BN - 1) / BN) + tn);
            *part = f32x2{top, sum};
        }
    }
}

}  // namespace lm
}  // namespace sgemm
