// Products with weights held in 4 bits (include/slm.h):
//   y[r][n] = sum_k x[r][k] (q[n][k] - z[n][b]) s[n][b],  b = k / BLOCK,
// for a few rows r: each weight is used once per row, so the time is that of
// reading the weights, and everything else is arranged not to add to it.
//
// The matrix cores do the sums, 16 rows at a time (v_mfma_f32_16x16x32_bf16,
// x as the first operand, 16 weight rows n as the second).  A lane's 16-byte
// load is 32 weights of one n.  Unpacking makes bf16 pairs with one shift and
// one and-or each: nibble i and nibble i + 4 of a 32-bit word, moved to bits 3..6
// of the halves and or'ed into 0x4180 (16.0, whose last four leading mantissa bits
// they are), read 16 + q exactly.  So the accumulator of one block holds
// sum x (16 + q), and with the sums of x over each block, which staging x leaves in LDS,
//   y += s sum x (16 + q) - s (16 + z) sum x,
// whose second part is a product over blocks of its own (v_mfma_f32_16x16x4_f32, a
// chunk's blocks in one instruction), so that the vector unit is left with the
// unpacking and one fma per block and sum.  16 is small beside q, so the
// difference loses about two bits of the fp32 sum.
//
// fp32 rows are split into three bf16 rows that add up to them exactly (8 + 8 +
// 8 leading bits) and go through the matrix cores one after another into the same
// sums; the products by 16 + q are exact in fp32, so an fp32 row loses nothing to bf16.
//
// A chunk is 128 weights along K: lane group g = lane / 16 holds weights
// 32 g .. 32 g + 31 of its n.  With blocks of 128 an instruction may take any 32 of
// them (k = 32 g + 8 j + i in instruction j).  With blocks of 32 or 64 it must stay
// inside one block: a 4 x 4 exchange between lane groups (four permlane swaps)
// gives instruction j the weights k = 32 j + 8 g + i.
//
// A workgroup is 8 waves: WN of them side by side along n, WK = 8 / WN splitting
// the chunks; their sums meet in LDS.  Each wave's weights travel to a ring in LDS of
// its own (buffer_load ... lds), four lanes to the 64 bytes of a row: fetched straight
// into the lanes that use them, neighbouring lanes would ask for different rows, and
// the address unit takes such lanes one by one (measured: twice the time).
// K is walked in slabs: x as bf16 parts in the order the unpacked pairs have, its block
// sums, and each block's and column's scale and zero.
#pragma once

#include "lm_tile.hpp"
#include "q4_rule.hpp"

namespace sgemm {
namespace q4 {

using lm::bf16;
using lm::bf16x8;
using lm::u32x4;

struct Q4Args {
    const void *X;
    const uint8_t *Q;
    const void *S;
    const uint8_t *Z;   // or null: 8 everywhere
    void *Y;
    const int *offsets; // or null: one group of all rows
    int64_t ldx, ldy;
    int64_t q_stride, s_stride;  // per group: bytes of Q; elements of S and Z
    int rows, N, K;
    int wn;             // waves along n (a power of two, at most 8)
    int slab_log2;      // k per slab, at least 128 WK
    int pass;           // rows per pass, at most 16 RT
    int vec_x;          // rows of X take 16-byte loads
};
typedef void (*Q4Fn)(Q4Args);

template <typename T> struct Parts { static constexpr int value = 1; };
template <> struct Parts<float> { static constexpr int value = 3; };

// mask 0x00780078 and sixteen 0x41804180, kept in registers: as literals they would
// cost an instruction more each.
__device__ __forceinline__ bf16x8 unpack(uint32_t u, uint32_t mask, uint32_t sixteen)
{
    u32x4 v;
    v[0] = ((u << 3) & mask) | sixteen;
    v[1] = ((u >> 1) & mask) | sixteen;
    v[2] = ((u >> 5) & mask) | sixteen;
    v[3] = ((u >> 9) & mask) | sixteen;
    return __builtin_bit_cast(bf16x8, v);
}

// The 4 x 4 exchange: lane group g's word j becomes lane group j's word g.
__device__ __forceinline__ u32x4 exchange(u32x4 v)
{
    auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

// Eight values of a row from k on, zero from K on, as they are in memory.
template <typename T> struct Octet {
    static constexpr int E = 16 / sizeof(T);
    union {
        u32x4 v[8 / E];
        T e[8];
    };
};

template <typename T>
__device__ __forceinline__ void load8(const T *row, int k, int K, bool vec, Octet<T> &x)
{
    if (vec && k + 8 <= K) {
#pragma unroll
        for (int h = 0; h < 8 / Octet<T>::E; ++h)
            x.v[h] = *reinterpret_cast<const u32x4 *>(row + k + h * Octet<T>::E);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j < K) x.e[j] = row[k + j];
    }
}

// The sum over the BLOCK / 8 neighbouring lanes that hold a block, in each of them: within
// four lanes, then mirrored eights and sixteens (whose quarters are already equal).
template <int BLOCK>
__device__ __forceinline__ float block_sum(float v)
{
    const auto add = [&](auto ctrl) {
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, v), decltype(ctrl)::value,
                                           0xf, 0xf, true));
    };
    add(std::integral_constant<int, 0xb1>{});                          // lanes 1 0 3 2
    add(std::integral_constant<int, 0x4e>{});                          // lanes 2 3 0 1
    if constexpr (BLOCK >= 64) add(std::integral_constant<int, 0x141>{});   // 7 .. 0
    if constexpr (BLOCK == 128) add(std::integral_constant<int, 0x140>{});  // 15 .. 0
    return v;
}

// A scale and 16 + its zero as LDS holds them: bf16 scales as two bf16 values in a word
// (16 + z is exact), fp32 ones as two floats.
template <typename T> struct Entry {
    uint32_t u;
    __device__ static Entry of(T s, float z)
    {
        return {(__builtin_bit_cast(uint32_t, (float)s) & 0xffff0000u) |
                (__builtin_bit_cast(uint32_t, z) >> 16)};
    }
    __device__ float scale() const { return __builtin_bit_cast(float, u & 0xffff0000u); }
    __device__ float zero() const { return __builtin_bit_cast(float, u << 16); }
};
template <> struct Entry<float> {
    float s, z;
    __device__ static Entry of(float s, float z) { return {s, z}; }
    __device__ float scale() const { return s; }
    __device__ float zero() const { return z; }
};
static_assert(sizeof(Entry<bf16>) == entry_bytes(2) && sizeof(Entry<float>) == entry_bytes(4) &&
                  Parts<bf16>::value == parts_of(2) && Parts<float>::value == parts_of(4),
              "what the rule counts with");

// Every wave's LDS writes are done; global loads stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// RT groups of 16 rows and NT of 16 columns a wave.  What bounds it: one row, 4096 x 4096:
// 7.0 us, a launch and one pass of memory latency; 12 fp32 rows, 8192 x 28001, blocks of 32:
// 63 us for 145 MB (43 without staging x and scales, 56 without products); 48 bf16 rows on
// 23 experts' 2048 x 5632, blocks of 64: 51 us for 146 MB (38 and 49).  fp32 with RT 2 spills 5
// to 29 registers, reloaded in the loop over K: 4096 x 14336, 16 rows 29 us, 17 37, 24 66, and
// 25 rows, two passes, 118.
template <typename T, int BLOCK, int RT, int NT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
__attribute__((amdgpu_waves_per_eu(RT <= 2 ? 4 : 2))) q4_kernel(Q4Args g)
{
    constexpr int D = ring_depth(NT);
    constexpr int P = Parts<T>::value;           // bf16 parts of a value
    constexpr int NB = 128 / BLOCK;              // blocks per chunk
    extern __shared__ __attribute__((aligned(1024))) char lds[];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l15 = lane & 15, lg = lane >> 4;
    const int wk_count = kWaves / g.wn;
    const int wn = wave % g.wn, wk = wave / g.wn;
    const int cols = g.wn * NT * 16;
    const int n_wg = blockIdx.x * cols;
    const int group = blockIdx.y;
    int begin = 0, end = g.rows;
    if (g.offsets) {
        lm::group_rows(g.offsets, group, g.rows, begin, end);
        begin = __builtin_amdgcn_readfirstlane(begin);
        end = __builtin_amdgcn_readfirstlane(end);
    }
    if (begin >= end) return;

    const int nblk = (g.K + BLOCK - 1) / BLOCK;
    const int chunks = (g.K + 127) / 128;
    const int row_bytes = g.K / 2;
    const int ncols = g.N - n_wg < cols ? g.N - n_wg : cols;  // columns that exist
    const uint8_t *Q = g.Q + group * g.q_stride + (int64_t)n_wg * row_bytes;
    const T *S = static_cast<const T *>(g.S) + group * g.s_stride + (int64_t)n_wg * nblk;
    const uint8_t *Z = g.Z ? g.Z + group * g.s_stride + (int64_t)n_wg * nblk : nullptr;
    const T *X = static_cast<const T *>(g.X);

    // LDS: the rings, the parts of x, per block of the slab and row the sum of x, and per
    // block and column its entry (one column more than there are, so that consecutive
    // blocks start in different banks).
    char *ring = lds + wave * (D * NT * 1024);
    const uint32_t ring_at = (uint32_t)(uintptr_t)(lm::lds_char *)ring;
    // All powers of two: a slab's k, octets and blocks.
    const int slab = 1 << g.slab_log2, oct_log2 = g.slab_log2 - 3;
    const int blk_log2 = g.slab_log2 - (BLOCK == 128 ? 7 : BLOCK == 64 ? 6 : 5);
    const int slab_blocks = 1 << blk_log2;
    const int pitch = slab * 2 + 16;  // bytes of a staged row: rows start in different banks
    const int part = g.pass * pitch;  // bytes of a part of x
    char *xs = lds + ring_bytes(NT);
    Entry<T> *entries = reinterpret_cast<Entry<T> *>(xs + P * part);
    float *xsum = reinterpret_cast<float *>(entries + slab_blocks * (cols + 1));

    // The ring: slot (row, place) of a 1 KB tile holds the 16 bytes at piece
    // place ^ (row / 4 & 3) of the row, so that the 16 lanes that later read one piece of
    // 16 rows meet 16 places of 256 bytes.
    const int frow = lane >> 2, fpiece = (lane & 3) ^ ((lane >> 4) & 3);
    uint32_t voff[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        voff[t] = (uint32_t)((wn * NT + t) * 16 + frow) * (uint32_t)row_bytes + fpiece * 16u;
    auto fetch = [&](int c, int d) {  // chunk c into slot d
        if constexpr (ALIGNED) {
            // Rows past N, and chunks past K, are outside the descriptor.
            const int64_t left = c < chunks ? (int64_t)(g.N - n_wg) * row_bytes - c * 64 : 0;
            u32x4 r = lm::descriptor(reinterpret_cast<const char *>(Q) + (int64_t)c * 64, left);
            uint32_t at = __builtin_amdgcn_readfirstlane(ring_at + d * (NT * 1024));
            // Wait states between a vector unit's write of a scalar and a load's use of it.
            asm volatile("s_nop 4" : "+s"(r), "+s"(at));
#pragma unroll
            for (int t = 0; t < NT; ++t) lm::load_slab16(r, voff[t], at + t * 1024);
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int n = (wn * NT + t) * 16 + frow, at = c * 64 + fpiece * 16;
                union {
                    u32x4 v;
                    uint8_t b[16];
                } x;
                x.v = u32x4{0, 0, 0, 0};
                if (n < ncols && at < row_bytes) {
                    const uint8_t *p = Q + (int64_t)n * row_bytes + at;
                    if (at + 16 <= row_bytes) {
                        __builtin_memcpy(&x, p, 16);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (at + j < row_bytes) x.b[j] = p[j];
                    }
                }
                *reinterpret_cast<u32x4 *>(ring + (d * NT + t) * 1024 + lane * 16) = x.v;
            }
        }
    };
    uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
    asm("" : "+s"(mask));
    asm("" : "+v"(sixteen));
    const int per_slab = slab / 128 / wk_count;                    // chunks a wave takes per slab
    const int steps = (chunks + wk_count - 1) / wk_count;          // and in all

    for (int r0 = begin; r0 < end; r0 += g.pass) {
        const int rows = end - r0 < g.pass ? end - r0 : g.pass;
        f32x4 total[RT][NT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) total[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        // The staged row each lane reads (places past the last row: any row; their
        // sums are not stored).
        int my_row[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) my_row[i] = 16 * i + l15 < rows ? 16 * i + l15 : rows - 1;

        auto put = [&](int i, const Octet<T> &x) {
            const int r = i >> oct_log2, o = i & ((1 << oct_log2) - 1);
            float v[8], sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (float)x.e[j];
            // Each part in turn: the leading 16 bits of what is left, and the rest (exact;
            // an infinity leaves a NaN, a NaN stays one).  The block's sum of x is formed
            // part by part, since sums of so few bits hardly round: it is multiplied by up to
            // 31, so its own roundings would outweigh those of the product.
#pragma unroll
            for (int p = 0; p < P; ++p) {
                u32x4 out;
#pragma unroll
                for (int d = 0; d < 4; ++d) {  // values d and d + 4 share a word
                    const uint32_t lo = __builtin_bit_cast(uint32_t, v[d]);
                    const uint32_t hi = __builtin_bit_cast(uint32_t, v[d + 4]);
                    out[d] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
                    if (p + 1 < P) {
                        v[d] -= __builtin_bit_cast(float, lo & 0xffff0000u);
                        v[d + 4] -= __builtin_bit_cast(float, hi & 0xffff0000u);
                    }
                }
                float part_sum = 0.f;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    part_sum += __builtin_bit_cast(float, out[d] << 16) +
                                __builtin_bit_cast(float, out[d] & 0xffff0000u);
                sum += block_sum<BLOCK>(part_sum);
                *reinterpret_cast<u32x4 *>(xs + p * part + r * pitch + o * 16) = out;
            }
            if (o % (BLOCK / 8) == 0) xsum[o / (BLOCK / 8) * g.pass + r] = sum;
        };
        // Scales and zeros kLot at a time, the first lot on its way while x is staged;
        // columns past N and blocks past K (which meet no output, or zeros of x) take the
        // last ones.
        constexpr int kLot = 4;
        T hs[kLot];
        uint8_t hz[kLot];
        const int count_s = cols << blk_log2;
        auto load_lot = [&](int i0, int k0) {
#pragma unroll
            for (int q = 0; q < kLot; ++q) {
                const int i = i0 + lane + q * kThreads;
                int n = i >> blk_log2, b = k0 / BLOCK + (i & (slab_blocks - 1));
                n = n < ncols ? n : ncols - 1;
                b = b < nblk ? b : nblk - 1;
                const uint32_t at = (uint32_t)n * (uint32_t)nblk + (uint32_t)b;
                hs[q] = S[at];
                hz[q] = Z ? Z[at] : 8;
            }
        };
        auto put_lot = [&](int i0) {
#pragma unroll
            for (int q = 0; q < kLot; ++q) {
                const int i = i0 + lane + q * kThreads;
                if (i < count_s)
                    entries[(i & (slab_blocks - 1)) * (cols + 1) + (i >> blk_log2)] =
                        Entry<T>::of(hs[q], 16.f + (float)hz[q]);
            }
        };
        // Rolled loops: values held in registers for the next slab, or unrolled copies
        // with their conditions, cost the main loop its registers (measured: twice the
        // time).
        auto stage = [&](int k0) {
            const int count = rows << oct_log2;
            int i0 = threadIdx.x & ~63;
            load_lot(i0, k0);
            if (g.vec_x && k0 + slab <= g.K) {
                // Four octets' loads at a time; past the end, the last octet again.
#pragma unroll 1
                for (int x0 = threadIdx.x & ~63; x0 < count; x0 += 4 * kThreads) {
                    Octet<T> x[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        int i = x0 + lane + q * kThreads;
                        i = i < count ? i : count - 1;
                        const T *p = X + (int64_t)(r0 + (i >> oct_log2)) * g.ldx + k0 +
                                     8 * (i & ((1 << oct_log2) - 1));
#pragma unroll
                        for (int h = 0; h < 8 / Octet<T>::E; ++h)
                            x[q].v[h] = *reinterpret_cast<const u32x4 *>(p + h * Octet<T>::E);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (x0 + lane + q * kThreads < count) put(x0 + lane + q * kThreads, x[q]);
                }
            } else {
#pragma unroll 1
                for (int i = threadIdx.x; i < count; i += kThreads) {
                    Octet<T> x;
#pragma unroll
                    for (int h = 0; h < 8 / Octet<T>::E; ++h) x.v[h] = u32x4{0, 0, 0, 0};
                    load8(X + (int64_t)(r0 + (i >> oct_log2)) * g.ldx,
                          k0 + 8 * (i & ((1 << oct_log2) - 1)), g.K, g.vec_x, x);
                    put(i, x);
                }
            }
            put_lot(i0);
#pragma unroll 1
            for (i0 += kLot * kThreads; i0 < count_s; i0 += kLot * kThreads) {
                load_lot(i0, k0);
                put_lot(i0);
            }
        };

        lds_barrier();  // the last rows' sums have been read
#pragma unroll
        for (int d = 0; d < D; ++d) fetch(d * wk_count + wk, d);
        int step = 0, slot = 0;
        for (int k0 = 0; k0 < g.K; k0 += slab) {
            lds_barrier();  // the slab before has been read
            stage(k0);
            lds_barrier();
            const int last = step + per_slab < steps ? step + per_slab : steps;
            for (; step < last; ++step) {
                const int c = step * wk_count + wk;
                asm volatile("s_waitcnt vmcnt(%0)" : : "n"((D - 1) * NT) : "memory");
                u32x4 w[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    w[t] = *reinterpret_cast<const u32x4 *>(
                        ring + (slot * NT + t) * 1024 + l15 * 64 + ((lg ^ (l15 >> 2)) << 4));
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before refilled
                fetch(c + D * wk_count, slot);
                slot = slot + 1 == D ? 0 : slot + 1;
                if (c >= chunks) continue;  // of the last step
                if constexpr (BLOCK != 128) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) w[t] = exchange(w[t]);
                }
                const int cs = c - k0 / 128;  // in the slab
                const char *xc = xs + cs * 256;
                const Entry<T> *sc = entries + cs * NB * (cols + 1) + wn * NT * 16 + l15;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    __builtin_amdgcn_sched_barrier(0);  // one block's operands at a time
                    f32x4 acc[RT][NT];
#pragma unroll
                    for (int i = 0; i < RT; ++i)
#pragma unroll
                        for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = b * 4 / NB; j < (b + 1) * 4 / NB; ++j) {
                        const int k = BLOCK == 128 ? 32 * lg + 8 * j : 32 * j + 8 * lg;
                        bf16x8 x[RT][P];
#pragma unroll
                        for (int i = 0; i < RT; ++i)
#pragma unroll
                            for (int p = 0; p < P; ++p)
                                x[i][p] = *reinterpret_cast<const bf16x8 *>(
                                    xc + p * part + my_row[i] * pitch + k * 2);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const bf16x8 q = unpack(w[t][j], mask, sixteen);
#pragma unroll
                            for (int p = 0; p < P; ++p)
#pragma unroll
                                for (int i = 0; i < RT; ++i)
                                    acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                        x[i][p], q, acc[i][t], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float s = sc[b * (cols + 1) + t * 16].scale();
#pragma unroll
                        for (int i = 0; i < RT; ++i)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                total[i][t][q] = fmaf(s, acc[i][t][q], total[i][t][q]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                // Lane group g adds block g's - s (16 + z) sum x; groups past the chunk's
                // blocks add nothing.
                const int mine = lg < NB ? lg : 0;
                float sums[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) sums[i] = xsum[(cs * NB + mine) * g.pass + my_row[i]];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Entry<T> e = sc[mine * (cols + 1) + t * 16];
                    const float sz = lg < NB ? -e.scale() * e.zero() : 0.f;
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        total[i][t] =
                            __builtin_amdgcn_mfma_f32_16x16x4f32(sums[i], sz, total[i][t], 0, 0, 0);
                }
            }
        }

        // Sums of the waves that share columns, through LDS: [wk][row][column of the
        // workgroup], where the rings were.
        float *join = reinterpret_cast<float *>(lds);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing lands in the rings any more
        lds_barrier();
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int r = 16 * i + 4 * lg + q;
                    if (r < rows)
                        join[(wk * g.pass + r) * cols + (wn * NT + t) * 16 + l15] = total[i][t][q];
                }
        lds_barrier();
        for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
            const int r = i / cols, c = i % cols;
            if (c >= ncols) continue;
            float v = 0.f;
            for (int w = 0; w < wk_count; ++w) v += join[(w * g.pass + r) * cols + c];
            static_cast<T *>(g.Y)[(int64_t)(r0 + r) * g.ldy + n_wg + c] = (T)v;
        }
    }
}

// Quantisation: 16 lanes per block of BLOCK weights, BLOCK / 16 each; one pass over W, done
// once per weight, so nothing beyond coalesced reads is arranged.
template <typename T, int BLOCK, bool ZEROS>
__global__ void __launch_bounds__(256) q4_quantize_kernel(int N, int K, int nblk, const T *W,
                                                          int64_t ldw, uint8_t *Q, T *S, uint8_t *Z)
{
    constexpr int E = BLOCK / 16;
    const int l = threadIdx.x & 15;
    // The 16 lanes of an item together.
    for (int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4; item < (int64_t)N * nblk;
         item += (int64_t)gridDim.x * 16) {
        const int n = (int)(item / nblk), b = (int)(item % nblk);
        const int k0 = b * BLOCK + l * E;
        float w[E], lo = 0.f, hi = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            w[j] = k0 + j < K ? (float)W[(int64_t)n * ldw + k0 + j] : 0.f;
            lo = fminf(lo, w[j]);
            hi = fmaxf(hi, w[j]);
        }
#pragma unroll
        for (int d = 1; d < 16; d *= 2) {
            lo = fminf(lo, __shfl_xor(lo, d));
            hi = fmaxf(hi, __shfl_xor(hi, d));
        }
        // The scale as it will be read back; a block of zeros keeps scale 0.
        const T scale = (T)(ZEROS ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f);
        const float s = (float)scale;
        float zero = 8.f;
        if (ZEROS) zero = s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            uint32_t byte = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float q = s > 0.f ? fminf(fmaxf(rintf(w[j + h] / s) + zero, 0.f), 15.f) : zero;
                byte |= (uint32_t)q << (4 * h);
            }
            if (k0 + j < K) Q[(int64_t)n * (K / 2) + (k0 + j) / 2] = (uint8_t)byte;
        }
        if (l == 0) {
            S[item] = scale;
            if (ZEROS) Z[item] = (uint8_t)zero;
        }
    }
}

}  // namespace q4
}  // namespace sgemm
