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
// the chunks; their sums meet in LDS.  x is staged in LDS as bf16, up to
// kSlab bytes at a time, in the order the unpacked pairs have.
#pragma once

#include "lm_tile.hpp"

namespace sgemm {
namespace q4 {

using lm::bf16;
using lm::bf16x8;
using lm::u32x4;

constexpr int kWaves = 8;
constexpr int kSlab = 64 * 1024;  // bytes of staged x: two workgroups per CU

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
    int slab;           // k per slab, a multiple of 128
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

// Eight values of a row from k on, zero from K on.
template <typename T>
__device__ __forceinline__ void load8(const T *row, int k, int K, bool vec, float *v)
{
    constexpr int E = 16 / sizeof(T);
    if (vec && k + 8 <= K) {
        typedef T Vec __attribute__((ext_vector_type(E)));
#pragma unroll
        for (int h = 0; h < 8 / E; ++h) {
            const Vec x = *reinterpret_cast<const Vec *>(row + k + h * E);
#pragma unroll
            for (int j = 0; j < E; ++j) v[h * E + j] = (float)x[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = k + j < K ? (float)row[k + j] : 0.f;
    }
}

// Chunks of weights a wave keeps in flight: 4 KB, which with 16 waves on a compute
// unit covers the latency of memory at its full rate.
constexpr int ring_depth(int nt) { return nt == 1 ? 4 : 2; }

template <typename T, int BLOCK, int RT, int NT, bool ALIGNED>
__global__ void __launch_bounds__(kWaves * 64)
__attribute__((amdgpu_waves_per_eu(RT * NT <= 4 ? 4 : 2))) q4_kernel(Q4Args g)
{
    constexpr int D = ring_depth(NT);
    constexpr int P = Parts<T>::value;           // bf16 parts of a value
    constexpr int NB = 128 / BLOCK;              // blocks per chunk
    extern __shared__ __attribute__((aligned(16))) char lds[];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l15 = lane & 15, lg = lane >> 4;
    const int wk_count = kWaves / g.wn;
    const int wn = wave % g.wn, wk = wave / g.wn;
    const int n_wg = blockIdx.x * (g.wn * NT * 16);
    const int group = blockIdx.y;
    int begin = 0, end = g.rows;
    if (g.offsets) lm::group_rows(g.offsets, group, g.rows, begin, end);
    if (begin >= end) return;

    const int nblk = (g.K + BLOCK - 1) / BLOCK;
    const int chunks = (g.K + 127) / 128;
    const int row_bytes = g.K / 2;
    // This lane's weight rows (past N: the last one, whose outputs are not stored), as
    // offsets from the workgroup's first row: bytes of Q, blocks of S and Z.
    const uint8_t *Q = g.Q + group * g.q_stride + (int64_t)n_wg * row_bytes;
    const T *S = static_cast<const T *>(g.S) + group * g.s_stride + (int64_t)n_wg * nblk;
    const uint8_t *Z = g.Z ? g.Z + group * g.s_stride + (int64_t)n_wg * nblk : nullptr;
    uint32_t qoff[NT], soff[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        int n = (wn * NT + t) * 16 + l15;
        n = n_wg + n < g.N ? n : g.N - 1 - n_wg;
        qoff[t] = (uint32_t)n * (uint32_t)row_bytes + (uint32_t)lg * 16u;
        soff[t] = (uint32_t)n * (uint32_t)nblk;
    }

    typedef T Scales __attribute__((ext_vector_type(NB)));
    typedef uint8_t Zeros __attribute__((ext_vector_type(NB)));
    struct Chunk {
        u32x4 q[NT];
        Scales s[NT];
        Zeros z[NT];
    };
    auto fetch = [&](int c, Chunk &h) {
        const uint8_t *qc = Q + (int64_t)c * 64;
        const T *sc = S + (int64_t)c * NB;
        const uint8_t *zc = Z + (Z ? (int64_t)c * NB : 0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (ALIGNED) {  // K a multiple of 128: whole chunks, whole vectors of scales
                h.q[t] = *reinterpret_cast<const u32x4 *>(qc + qoff[t]);
                h.s[t] = *reinterpret_cast<const Scales *>(sc + soff[t]);
                if (Z) h.z[t] = *reinterpret_cast<const Zeros *>(zc + soff[t]);
            } else {
                const int at = c * 64 + lg * 16;  // byte of the row
                if (at + 16 <= row_bytes) {
                    __builtin_memcpy(&h.q[t], qc + qoff[t], 16);
                } else {
                    union {
                        u32x4 v;
                        uint8_t b[16];
                    } x;
                    x.v = u32x4{0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (at + j < row_bytes) x.b[j] = qc[qoff[t] + j];
                    h.q[t] = x.v;
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    // A block past the last holds only zeros of x: any scale will do.
                    int blk = c * NB + b;
                    blk = blk < nblk ? blk : nblk - 1;
                    h.s[t][b] = S[soff[t] + blk];
                    if (Z) h.z[t][b] = Z[soff[t] + blk];
                }
            }
        }
    };

    const int pitch = g.slab * 2 + 16;  // bytes of a staged row: rows start in different banks
    const int part = g.pass * pitch;    // bytes of a part of x
    float *xsum = reinterpret_cast<float *>(lds + P * part);  // [block of the slab][row]
    uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
    asm("" : "+s"(mask));
    asm("" : "+v"(sixteen));
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

        for (int k0 = 0; k0 < g.K; k0 += g.slab) {
            const int kn = g.K - k0 < g.slab ? g.K - k0 : g.slab;
            const int c0 = k0 / 128, c1 = c0 + (kn + 127) / 128;
            Chunk ring[D];
            const int first = c0 + wk;
#pragma unroll
            for (int d = 0; d < D; ++d)
                if (first + d * wk_count < c1) fetch(first + d * wk_count, ring[d]);
            __syncthreads();  // the slab (or the sums) before this one have been read
            const int octets = (c1 - c0) * 16;
            for (int i = threadIdx.x; i < rows * octets; i += kWaves * 64) {
                const int r = i / octets, o = i % octets;
                float v[8];
                load8(static_cast<const T *>(g.X) + (int64_t)(r0 + r) * g.ldx, k0 + 8 * o, g.K,
                      g.vec_x, v);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += v[j];
                // Each part in turn: the leading 16 bits of what is left, and the rest
                // (exact; an infinity leaves a NaN, a NaN stays one).
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
                    *reinterpret_cast<u32x4 *>(lds + p * part + r * pitch + o * 16) = out;
                }
                // The BLOCK / 8 lanes of a block are neighbours, all of them here.
#pragma unroll
                for (int d = 1; d < BLOCK / 8; d *= 2) sum += __shfl_xor(sum, d);
                if (o % (BLOCK / 8) == 0) xsum[o / (BLOCK / 8) * g.pass + r] = sum;
            }
            __syncthreads();

            auto chunk = [&](int c, const Chunk &h) {
                const char *xs = lds + (c - c0) * 256;
                u32x4 w[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) w[t] = BLOCK == 128 ? h.q[t] : exchange(h.q[t]);
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
                                    xs + p * part + my_row[i] * pitch + k * 2);
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
                        const float s = (float)h.s[t][b];
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
                for (int i = 0; i < RT; ++i)
                    sums[i] = xsum[((c - c0) * NB + mine) * g.pass + my_row[i]];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float s = (float)h.s[t][0], z = Z ? (float)h.z[t][0] : 8.f;
#pragma unroll
                    for (int b = 1; b < NB; ++b) {
                        s = lg == b ? (float)h.s[t][b] : s;
                        if (Z) z = lg == b ? (float)h.z[t][b] : z;
                    }
                    const float sz = lg < NB ? -s * (16.f + z) : 0.f;
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        total[i][t] =
                            __builtin_amdgcn_mfma_f32_16x16x4f32(sums[i], sz, total[i][t], 0, 0, 0);
                }
            };
            for (int c = first; c < c1; c += D * wk_count) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    const int cd = c + d * wk_count;
                    if (cd >= c1) break;
                    chunk(cd, ring[d]);
                    if (cd + D * wk_count < c1) fetch(cd + D * wk_count, ring[d]);
                }
            }
        }

        // Sums of the waves that share columns, through LDS: [wk][row][column of the
        // workgroup].
        const int cols = g.wn * NT * 16;
        float *join = reinterpret_cast<float *>(lds);
        __syncthreads();
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
        __syncthreads();
        for (int i = threadIdx.x; i < rows * cols; i += kWaves * 64) {
            const int r = i / cols, c = i % cols;
            if (n_wg + c >= g.N) continue;
            float v = 0.f;
            for (int w = 0; w < wk_count; ++w) v += join[(w * g.pass + r) * cols + c];
            static_cast<T *>(g.Y)[(int64_t)(r0 + r) * g.ldy + n_wg + c] = (T)v;
        }
    }
}

// Quantisation: 16 lanes per block of BLOCK weights, BLOCK / 16 each.
template <typename T, int BLOCK, bool ZEROS>
__global__ void __launch_bounds__(256) q4_quantize_kernel(int N, int K, int nblk, const T *W,
                                                          int64_t ldw, uint8_t *Q, T *S, uint8_t *Z)
{
    constexpr int E = BLOCK / 16;
    const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;
    const int l = threadIdx.x & 15;
    if (item >= (int64_t)N * nblk) return;  // the 16 lanes of an item together
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

}  // namespace q4
}  // namespace sgemm
