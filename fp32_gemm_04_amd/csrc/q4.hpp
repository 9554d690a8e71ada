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
// sum x (16 + q), and one more product by a vector of ones holds sum x:
//   y += s (sum x (16 + q) - (16 + z) sum x).
// The constant is small beside q, so the difference loses about two bits of
// the fp32 sum.
//
// fp32 rows are split into three bf16 rows that add up to them exactly (8 + 8 +
// 8 leading bits), which take three of the 16 places; the products by 16 + q
// are exact in fp32, so an fp32 row loses nothing to bf16.
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
    int pass;           // rows per pass, at most pass_rows<T>(RT)
    int vec_x;          // rows of X take 16-byte loads
};
typedef void (*Q4Fn)(Q4Args);

template <typename T> struct Parts { static constexpr int value = 1; };
template <> struct Parts<float> { static constexpr int value = 3; };

// Rows that RT tiles of 16 places hold.
template <typename T> constexpr int pass_rows(int rt) { return rt * 16 / Parts<T>::value; }

__device__ __forceinline__ bf16x8 unpack(uint32_t u)
{
    u32x4 v;
    v[0] = ((u << 3) & 0x00780078u) | 0x41804180u;
    v[1] = ((u >> 1) & 0x00780078u) | 0x41804180u;
    v[2] = ((u >> 5) & 0x00780078u) | 0x41804180u;
    v[3] = ((u >> 9) & 0x00780078u) | 0x41804180u;
    return __builtin_bit_cast(bf16x8, v);
}

// Place of value i of eight in the order of the unpacked pairs: 0 4 1 5 2 6 3 7.
__device__ __forceinline__ constexpr int place(int i) { return i < 4 ? 2 * i : 2 * (i - 4) + 1; }

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

__device__ __forceinline__ uint16_t top_half(float v)
{
    return (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16);
}

template <typename T, int BLOCK, int RT, int NT, bool ALIGNED>
__global__ void __launch_bounds__(kWaves * 64) q4_kernel(Q4Args g)
{
    constexpr int P = Parts<T>::value;
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
    const uint8_t *Q = g.Q + group * g.q_stride;
    const T *S = static_cast<const T *>(g.S) + group * g.s_stride;
    const uint8_t *Z = g.Z ? g.Z + group * g.s_stride : nullptr;

    // This lane's weight rows (past N: the last one, whose outputs are not stored).
    const uint8_t *qrow[NT];
    const T *srow[NT];
    const uint8_t *zrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        int n = n_wg + (wn * NT + t) * 16 + l15;
        n = n < g.N ? n : g.N - 1;
        qrow[t] = Q + (int64_t)n * row_bytes;
        srow[t] = S + (int64_t)n * nblk;
        zrow[t] = Z ? Z + (int64_t)n * nblk : nullptr;
    }

    struct Chunk {
        u32x4 q[NT];
        float s[NT][NB], z[NT][NB];
    };
    auto fetch = [&](int c, Chunk &h) {
        const int at = c * 64 + lg * 16;  // byte of the row
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint8_t *p = qrow[t] + at;
            if (at + 16 <= row_bytes) {
                if constexpr (ALIGNED)
                    h.q[t] = *reinterpret_cast<const u32x4 *>(p);
                else
                    __builtin_memcpy(&h.q[t], p, 16);
            } else {
                union {
                    u32x4 v;
                    uint8_t b[16];
                } x;
                x.v = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (at + j < row_bytes) x.b[j] = p[j];
                h.q[t] = x.v;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                // A block past the last holds only zeros of x: any scale will do.
                int blk = c * NB + b;
                blk = blk < nblk ? blk : nblk - 1;
                h.s[t][b] = (float)srow[t][blk];
                h.z[t][b] = zrow[t] ? (float)zrow[t][blk] : 8.f;
            }
        }
    };

    const int pitch = g.slab * 2 + 16;  // bytes of a staged row: rows start in different banks
    for (int r0 = begin; r0 < end; r0 += g.pass) {
        const int rows = end - r0 < g.pass ? end - r0 : g.pass;
        f32x4 total[RT][NT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) total[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        // The staged row each lane reads (places past the last row: any row; their
        // sums are not stored).
        int place_row[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int p = 16 * i + l15;
            place_row[i] = p < rows * P ? p : rows * P - 1;
        }

        for (int k0 = 0; k0 < g.K; k0 += g.slab) {
            const int kn = g.K - k0 < g.slab ? g.K - k0 : g.slab;
            const int c0 = k0 / 128, c1 = c0 + (kn + 127) / 128;
            Chunk cur, nxt;
            const int first = c0 + wk;
            if (first < c1) fetch(first, cur);
            __syncthreads();  // the slab (or the sums) before this one have been read
            const int octets = (c1 - c0) * 16;
            for (int i = threadIdx.x; i < rows * octets; i += kWaves * 64) {
                const int r = i / octets, o = i % octets;
                float v[8];
                load8(static_cast<const T *>(g.X) + (int64_t)(r0 + r) * g.ldx, k0 + 8 * o, g.K,
                      g.vec_x, v);
                union {
                    u32x4 v;
                    uint16_t h[8];
                } x[P];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (P == 1) {
                        x[0].h[place(j)] = top_half(v[j]);
                    } else {
                        // Leading 8 bits, the next 8 and the rest, each exact; an infinity
                        // or NaN stays whole in the first.
                        float a = v[j];
                        const bool fin = isfinite(a);
                        if (!fin) a = isinf(a) ? a : __builtin_nanf("");
                        const uint16_t h0 = top_half(a);
                        const float r1 =
                            fin ? a - __builtin_bit_cast(float, (uint32_t)h0 << 16) : 0.f;
                        const uint16_t h1 = top_half(r1);
                        const float r2 = r1 - __builtin_bit_cast(float, (uint32_t)h1 << 16);
                        x[0].h[place(j)] = h0;
                        x[1].h[place(j)] = h1;
                        x[2].h[place(j)] = top_half(r2);
                    }
                }
#pragma unroll
                for (int p = 0; p < P; ++p)
                    *reinterpret_cast<u32x4 *>(lds + (r * P + p) * pitch + o * 16) = x[p].v;
            }
            __syncthreads();

            for (int c = first; c < c1; c += wk_count) {
                if (c + wk_count < c1) fetch(c + wk_count, nxt);
                u32x4 w[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) w[t] = BLOCK == 128 ? cur.q[t] : exchange(cur.q[t]);
                const u32x4 one_bits = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
                const bf16x8 ones = __builtin_bit_cast(bf16x8, one_bits);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    f32x4 sum[RT], acc[RT][NT];
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
                    }
#pragma unroll
                    for (int j = b * 4 / NB; j < (b + 1) * 4 / NB; ++j) {
                        const int k = BLOCK == 128 ? 32 * lg + 8 * j : 32 * j + 8 * lg;
                        bf16x8 x[RT];
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            x[i] = *reinterpret_cast<const bf16x8 *>(
                                lds + place_row[i] * pitch + ((c - c0) * 128 + k) * 2);
                            sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], ones, sum[i], 0,
                                                                             0, 0);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const bf16x8 q = unpack(w[t][j]);
#pragma unroll
                            for (int i = 0; i < RT; ++i)
                                acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    x[i], q, acc[i][t], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float s = cur.s[t][b], z = 16.f + cur.z[t][b];
#pragma unroll
                        for (int i = 0; i < RT; ++i)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                total[i][t][q] = fmaf(s, fmaf(-z, sum[i][q], acc[i][t][q]),
                                                      total[i][t][q]);
                    }
                }
                cur = nxt;
            }
        }

        // Sums of the waves that share columns, and of the parts of a row, through
        // LDS: [wk][place][column of the workgroup].
        const int cols = g.wn * NT * 16;
        float *sums = reinterpret_cast<float *>(lds);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int p = 16 * i + 4 * lg + q;
                    if (p < rows * P)
                        sums[(wk * (RT * 16) + p) * cols + (wn * NT + t) * 16 + l15] =
                            total[i][t][q];
                }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * cols; i += kWaves * 64) {
            const int r = i / cols, c = i % cols;
            if (n_wg + c >= g.N) continue;
            float v = 0.f;
            for (int w = 0; w < wk_count; ++w)
#pragma unroll
                for (int p = 0; p < P; ++p) v += sums[(w * (RT * 16) + r * P + p) * cols + c];
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
