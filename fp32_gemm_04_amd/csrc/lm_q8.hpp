// Rows in 8-bit integers, and products of a few such rows with 8-bit weights (include/slm.h).
//
// Quantisation.  scale = m * fl(1/127) with m the row's largest magnitude, which is what torch
// makes of a division by 127 on the device (m / 127 or its neighbour); q is x / scale rounded to
// the nearest integer, ties to even, of the exact quotient.  One fma with the reciprocal of scale
// and 1.5 * 2^23 rounds x / scale to an integer, in the last bits of its result, and a second gives
// how far from it the quotient was.  The reciprocal's rounding moves the quotient by less than
// 2^-17 (127 * 2^-24), so only where that distance is within 2^-16 of a half may q be one off
// (values of a wave: some 3% of the time); there the remainder x - q scale, exact in one fma (a
// multiple of the smaller operand's last bit, below 2 scale), is compared with half of scale.
#pragma once

#include "lm_tile.hpp"

namespace sgemm {
namespace lm {

__device__ __forceinline__ uint32_t magnitude(float x)
{
    return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

// What a row's values are divided by, scaled by a power of two so that its reciprocal is
// finite and normal where the scale is tiny.
struct Quantum {
    float scale;    // as stored
    float by;       // power of two
    float step, inverse;
    // m: the largest magnitude's bits, in which an infinity or a NaN lies above every number.
    __device__ __forceinline__ explicit Quantum(uint32_t m)
    {
        constexpr float kPart = 1.f / 127.f;
        scale = __builtin_bit_cast(float, m) * kPart;
        by = scale < 0x1p-60f ? 0x1p80f : 1.f;
        step = scale * by;
        inverse = step > 0.f ? 1.f / step : 0.f;
        if (m >= 0x7f800000u) {
            scale = __builtin_nanf("");
            step = inverse = 0.f;
        }
    }
    // One value, whatever the scale; without branches.
    __device__ __forceinline__ int exact(float x) const
    {
        const float v = x * by, q = rintf(v * inverse);
        const float left = fmaf(-q, step, v), twice = 2.f * fabsf(left);
        int i = inverse > 0.f ? (int)q : 0;
        // On a tie the even neighbour stays.
        const bool move = twice > step || (twice == step && (i & 1));
        i += move ? (left > 0.f ? 1 : -1) : 0;
        i = i > 127 ? 127 : i < -127 ? -127 : i;
        return inverse > 0.f ? i : 0;
    }
    // N values (a multiple of 4) as bytes, the first in the lowest.
    template <int N> __device__ __forceinline__ void bytes(const float (&x)[N], uint32_t (&q)[N / 4]) const
    {
        constexpr float kWhole = 12582912.f;  // 1.5 * 2^23
        float far = 0.f;
#pragma unroll
        for (int w = 0; w < N / 4; ++w) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = x[4 * w + i], whole = fmaf(v, inverse, kWhole);
                far = fmaxf(far, fabsf(fmaf(v, inverse, kWhole - whole)));
                u[i] = __builtin_bit_cast(uint32_t, whole);
            }
            // The low byte of each.
            q[w] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400u),
                                         __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u), 0x05040100u);
        }
        if (by != 1.f || !(inverse > 0.f) || far > 0.5f - 0x1p-16f) {
#pragma unroll
            for (int w = 0; w < N / 4; ++w) {
                q[w] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) q[w] |= ((uint32_t)exact(x[4 * w + i]) & 0xffu) << (8 * i);
            }
        }
    }
};

// The wave's largest value: within rows of 16 lanes, then from row to row; lane 63 has it.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    const auto join = [&](auto ctrl, auto rows) {
        const uint32_t u = __builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value,
                                                       decltype(rows)::value, 0xf, false);
        v = u > v ? u : v;
    };
    typedef std::integral_constant<int, 0xf> All;
    join(std::integral_constant<int, 0x111>{}, All{});                               // from the lane below
    join(std::integral_constant<int, 0x112>{}, All{});                               // two below
    join(std::integral_constant<int, 0x114>{}, All{});                               // four
    join(std::integral_constant<int, 0x118>{}, All{});                               // eight
    join(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // rows 0, 2 to 1, 3
    join(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // row 1 to 2, 3
    return __builtin_amdgcn_readlane(v, 63);
}

// N values of a row from k on as fp32, zeros from K on.
template <int N, typename T>
__device__ __forceinline__ void load_values(const T *row, int k, int K, float (&v)[N])
{
    if (k + N <= K) {
        typedef T Vec __attribute__((ext_vector_type(N)));
        typedef Vec Loose __attribute__((aligned(sizeof(T))));
        const Vec x = *reinterpret_cast<const Loose *>(row + k);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (float)x[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = K > 0 ? (float)row[k + i < K ? k + i : K - 1] : 0.f;
            v[i] = k + i < K ? x : 0.f;
        }
    }
}

// The first `left` of 16 bytes, zeros after them.  (Each byte of a part is a load of its own, all in
// flight at once: past the last the last is read again.)
template <typename B> __device__ __forceinline__ u32x4 load_bytes(const B *p, int left)
{
    u32x4 q = {0, 0, 0, 0};
    if (left >= 16) {
        __builtin_memcpy(&q, p, 16);
    } else if (left > 0) {
        uint32_t b[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = (uint8_t)p[i < left ? i : left - 1];
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i / 4] |= (i < left ? b[i] : 0u) << (8 * (i % 4));
    }
    return q;
}

template <int N> __device__ __forceinline__ uint32_t max_of(const float (&v)[N], uint32_t m)
{
#pragma unroll
    for (int i = 0; i < N; ++i) m = magnitude(v[i]) > m ? magnitude(v[i]) : m;
    return m;
}

struct QuantArgs {
    const void *X;
    int8_t *Q;
    float *scales;
    const int *place;  // or null: row r to row r
    int64_t ldx, ldq;
    int rows, K, k, out_rows;
};

// WAVES waves share a row of X, 16 bytes a lane at a time; each lane keeps its first kHeld pieces,
// and reads what follows again.  All loads of the kept pieces are in flight at once: none is
// behind a branch, since a piece that would end past the row is moved back to end with it (its
// values meet another piece's, and so do the bytes that both write).
constexpr int kHeld = 4;

constexpr int quantize_waves(int waves)  // of a workgroup
{
    return waves < 4 ? 4 : waves;
}

template <typename T, int WAVES, bool PLACED>
__global__ void __launch_bounds__(quantize_waves(WAVES) * 64) q8_quantize_kernel(QuantArgs a)
{
    constexpr int ROWS = quantize_waves(WAVES) / WAVES, E = 16 / sizeof(T), step = WAVES * 64 * E;
    typedef T Vec __attribute__((ext_vector_type(E)));
    typedef Vec Loose __attribute__((aligned(sizeof(T))));
    // Magnitudes order like their bits, as integers of the value's size.
    typedef typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type U;
    typedef U Bits __attribute__((ext_vector_type(E)));
    __shared__ uint32_t part[quantize_waves(WAVES)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k0 = ((wave % WAVES) * 64 + lane) * E;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t r = r0 + wave / WAVES;
        const bool here = r < a.rows;
        const T *row = static_cast<const T *>(a.X) + (here ? r : a.rows - 1) * a.ldx;
        // f(row of Q, whether it is a dropped choice's) for every row that this one goes to.
        const auto each_row = [&](auto f) {
            if constexpr (!PLACED) {
                f(r, false);
            } else {
                for (int j = 0; j < a.k; ++j) {
                    const int p = read<true>(a.place, r * a.k + j), out = p <= -2 ? -2 - p : p;
                    if ((uint32_t)out < (uint32_t)a.out_rows) f((int64_t)out, p <= -2);
                }
            }
        };
        const auto put_scale = [&](float scale) {
            if (wave % WAVES == 0 && lane == 0)
                each_row([&](int64_t out, bool dropped) { a.scales[out] = dropped ? 0.f : scale; });
        };
        if (a.K < E) {  // no whole piece (one wave a row)
            const float x = lane < a.K ? (float)row[lane] : 0.f;
            const Quantum s(wave_max(magnitude(x)));
            if (!here) continue;
            each_row([&](int64_t out, bool dropped) {
                if (lane < a.K) a.Q[out * a.ldq + lane] = dropped ? 0 : (int8_t)s.exact(x);
            });
            put_scale(s.scale);
            continue;
        }
        const auto start = [&](int k) { return k + E <= a.K ? k : a.K - E; };
        const auto load = [&](int k) { return (Vec) * reinterpret_cast<const Loose *>(row + start(k)); };
        Bits top = 0;
        const auto max_in = [&](Vec x) {
            top = __builtin_elementwise_max(top, __builtin_bit_cast(Bits, x) & (U)((U)~(U)0 >> 1));
        };
        // (A row past the last reads the last, and a lane past the row's end its last piece.)
        Vec held[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) held[i] = load(k0 + i * step);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) max_in(held[i]);
        for (int k = k0 + kHeld * step; k < a.K; k += step) max_in(load(k));
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) m = top[i] > m ? top[i] : m;
        m = wave_max(m << (32 - 8 * sizeof(T)));
        if constexpr (WAVES > 1) {
            if (lane == 0) part[wave] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const uint32_t u = part[wave / WAVES * WAVES + w];
                m = u > m ? u : m;
            }
            __syncthreads();
        }
        if (!here) continue;
        const Quantum s(m);
        const auto put = [&](Vec x, int k) {
            if (k >= a.K) return;
            float v[E];
            uint32_t q[E / 4];
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = (float)x[i];
            s.bytes(v, q);
            each_row([&](int64_t out, bool dropped) {
                uint32_t z[E / 4];
#pragma unroll
                for (int w = 0; w < E / 4; ++w) z[w] = dropped ? 0 : q[w];
                __builtin_memcpy(a.Q + out * a.ldq + start(k), z, E);
            });
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // one piece at a time: fewer registers
            if (i * step < a.K) put(held[i], k0 + i * step);
        }
        for (int k = k0 + kHeld * step; k < a.K; k += step) put(load(k), k);
        put_scale(s.scale);
    }
}

// ------------------------------------------------------------- a few rows

// Y[r][n] for a few rows that are quantised on the way, have weights at odd bytes or more than 64
// groups: every weight is used once a row, so the time is that of reading the weights.  A workgroup
// of eight waves puts its rows into LDS once, quantising them where TX is not int8, then takes tiles
// of 16 columns; the waves split the contraction, slab by slab of 128 bytes, and their integer sums
// meet in LDS.  Weights travel through a ring of LDS of each wave's own by direct loads, which ask
// for whole 128-byte rows; fetched straight into the lanes that the matrix instruction wants them
// in, neighbouring lanes would ask for different rows.  The ring runs on from tile to tile, and is
// filled before the rows are quantised.  us in a graph: 1 row, 4096 x 4096 7.9 (of 8-bit rows 5.4),
// 4096 x 14336 13.8, 8192 x 28001 41.4 (5.5 TB/s).
struct VecArgs {
    const void *X;
    const float *x_scales;  // of 8-bit rows
    const int8_t *W;
    const float *w_scales;
    void *Y;
    const int *offsets;  // or null: one group of all rows
    int64_t ldx, ldw, stride_w, ldy;
    int rows, N, K, groups;
    int fill;            // rows outside every group are set to zero
    int pass;            // rows in LDS at once, at most 16
    int slabs;           // of 128 bytes
};
typedef void (*VecFn)(VecArgs);

constexpr int kVecWaves = 8;
constexpr int kVecSlab = 16 * 128;
constexpr int kVecTiles = 32;  // tiles whose column scales are fetched at once
// Bytes of LDS: the rows, the rings, two tiles' sums, two sets of column scales, and the rows'
// maxima and scales.
inline int vec_lds(int pass, int slabs, int depth)
{
    return pass * slabs * 128 + kVecWaves * depth * kVecSlab + 2 * kVecWaves * 1024 +
           2 * kVecTiles * 64 + 16 * kVecWaves * 4 + 64;
}

template <typename TX, typename TY, int DEPTH, bool FAST>
__global__ void __launch_bounds__(kVecWaves * 64) q8_vec_kernel(VecArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) char vec_shared[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char *ring = vec_shared + wave * (DEPTH * kVecSlab);
    int *sums = reinterpret_cast<int *>(vec_shared + kVecWaves * DEPTH * kVecSlab);
    float *columns = reinterpret_cast<float *>(sums + 2 * kVecWaves * 256);
    uint32_t *maxima = reinterpret_cast<uint32_t *>(columns + 2 * kVecTiles * 16);
    float *scales = reinterpret_cast<float *>(maxima + 16 * kVecWaves);
    char *rows_lds = reinterpret_cast<char *>(scales + 16);

    if (a.fill && blockIdx.y == 0)
        zero_outside(a.offsets, a.groups, a.rows, a.N, static_cast<TY *>(a.Y), a.ldy);
    int group = blockIdx.y, begin = 0, end = a.rows;
    if ((int)gridDim.y < a.groups) {
        // More groups than rows: the blockIdx.y-th of those that have rows.
        int before = blockIdx.y, at = -1;
        for (int g0 = 0; g0 < a.groups && at < 0; g0 += 64) {
            int b = 0, e = 0;
            if (g0 + lane < a.groups) group_rows(a.offsets, g0 + lane, a.rows, b, e);
            uint64_t some = __ballot(e > b);
            const int n = __popcll(some);
            if (before >= n) {
                before -= n;
                continue;
            }
            for (; before > 0; --before) some &= some - 1;
            at = g0 + __builtin_ctzll(some);
        }
        group = at;
    }
    if (group < 0 || group >= a.groups) return;
    if (a.offsets) group_rows(a.offsets, group, a.rows, begin, end);
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(end);
    const int tiles_n = (a.N + 15) / 16;
    const int8_t *W = a.W + group * a.stride_w;
    const float *ws = a.w_scales + (int64_t)group * a.N;
    // This wave's slabs of a tile, and this workgroup's tiles.
    const int ns = wave < a.slabs ? (a.slabs - wave + kVecWaves - 1) / kVecWaves : 0;
    const int tiles = (int)blockIdx.x < tiles_n ? (tiles_n - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;

    for (int first = begin; first < end; first += a.pass) {
        const int R = end - first < a.pass ? end - first : a.pass;
        // ---- the ring: the next slab to fetch, and where to
        int f_tile = blockIdx.x, f_slab = 0, f_buf = 0;
        const int frow = lane >> 3, fchunk = (lane & 7) ^ ((frow >> 1) & 7);
        const int frow2 = frow + 8, fchunk2 = (lane & 7) ^ ((frow2 >> 1) & 7);
        const uint32_t voff = (uint32_t)frow * (uint32_t)a.ldw + fchunk * 16u;
        const uint32_t voff2 = (uint32_t)frow2 * (uint32_t)a.ldw + fchunk2 * 16u;
        u32x4 hold[2];
        auto fetch = [&]() {
            const int k = (wave + kVecWaves * f_slab) * 128;
            const bool more = f_slab < ns && f_tile < tiles_n;
            const int64_t n0 = (int64_t)f_tile * 16;
            const char *p = reinterpret_cast<const char *>(W) + n0 * a.ldw + k;
            const int64_t left = more ? (a.N - 1 - n0) * a.ldw + a.K - k : 0;
            if constexpr (FAST) {
                u32x4 rs = descriptor(p, left);
                uint32_t at = (uint32_t)(uintptr_t)(lds_char *)ring + f_buf * kVecSlab;
                // Wait states between a vector unit's write of these and their use.
                asm volatile("s_nop 4" : "+s"(rs), "+s"(at));
                load_slab16(rs, voff, at);
                load_slab16(rs, voff2, at + 1024);
                f_buf = f_buf + 1 == DEPTH ? 0 : f_buf + 1;
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = h ? frow2 : frow, c = (h ? fchunk2 : fchunk) * 16;
                    const char *q = p + row * a.ldw + c;
                    const int room = more && n0 + row < a.N ? a.K - k - c : 0;
                    hold[h] = load_bytes(q, room);
                }
            }
            if (++f_slab >= ns) f_slab = 0, f_tile += gridDim.x;
        };
        const TX *X = static_cast<const TX *>(a.X) + (int64_t)first * a.ldx;
        // Rows to be quantised: `per` waves a row.  One row a wave and one chunk of 16 values a lane stay in
        // registers between the two passes, and come before the weights: a wait for them, which is
        // one for all loads before them, then leaves the weights in flight.
        int per = 1;
        while (per < kVecWaves && per * 2 * R <= kVecWaves) per *= 2;
        const int stride = kVecWaves / per, part = wave % per, chunks = a.slabs * 8;
        const bool stays = !std::is_same<TX, int8_t>::value && R <= stride && chunks <= per * 64;
        float v[16];
        uint32_t top = 0;
        if constexpr (!std::is_same<TX, int8_t>::value) {
            if (stays && wave / per < R && part * 64 + lane < chunks) {
                load_values<16>(X + wave / per * a.ldx, (part * 64 + lane) * 16, a.K, v);
                top = max_of(v, top);
            }
            asm volatile("" : "+v"(top));
        }
        if (ns > 0) {
            if constexpr (FAST) {
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) fetch();
            } else {
                fetch();
            }
        }
        // ---- the rows, in the slabs' order: chunk c of row r of a slab at place c ^ (r / 2)
        const auto chunk_of = [&](int r, int c) {
            return reinterpret_cast<u32x4 *>(rows_lds + ((c >> 3) * R + r) * 128 +
                                             (((c & 7) ^ ((r >> 1) & 7)) << 4));
        };
        if constexpr (std::is_same<TX, int8_t>::value) {
            if (threadIdx.x < R) scales[threadIdx.x] = a.x_scales[first + threadIdx.x];
            for (int i = threadIdx.x; i < R * a.slabs * 8; i += kVecWaves * 64) {
                const int r = i / (a.slabs * 8), c = i - r * (a.slabs * 8), left = a.K - c * 16;
                *chunk_of(r, c) = load_bytes(X + r * a.ldx + c * 16, left);
            }
        } else {
            for (int r = wave / per; r < R; r += stride) {
                uint32_t m = top;
                for (int c = part * 64 + lane; !stays && c < chunks; c += per * 64) {
                    load_values<16>(X + r * a.ldx, c * 16, a.K, v);
                    m = max_of(v, m);
                }
                m = wave_max(m);
                if (lane == 0) maxima[r * kVecWaves + part] = m;
            }
            __syncthreads();
            for (int r = wave / per; r < R; r += stride) {
                uint32_t m = 0;
#pragma unroll
                for (int p = 0; p < kVecWaves; ++p) {  // (all of them read at once)
                    const uint32_t u = maxima[r * kVecWaves + p];
                    m = p < per && u > m ? u : m;
                }
                const Quantum s(m);
                if (part == 0 && lane == 0) scales[r] = s.scale;
                for (int c = part * 64 + lane; c < chunks; c += per * 64) {
                    if (!stays) load_values<16>(X + r * a.ldx, c * 16, a.K, v);
                    uint32_t q[4];
                    s.bytes(v, q);
                    *chunk_of(r, c) = u32x4{q[0], q[1], q[2], q[3]};
                }
            }
        }
        __syncthreads();
        // ---- tiles
        const int l16 = lane & 15, g = lane >> 4;
        const int xr = l16 < R ? l16 : R - 1;  // rows past the last repeat it, and are not stored
        int buf = 0;
        for (int i = 0; i < tiles; ++i) {
            const int n0 = (blockIdx.x + i * gridDim.x) * 16;
            if (i % kVecTiles == 0) {
                // A thread for each column of the next tiles: a wait for them, which is one for
                // the ring's loads too, is rare.  Read after the tile's barrier.
                const int64_t n = (blockIdx.x + (int64_t)(i + (threadIdx.x >> 4)) * gridDim.x) * 16 +
                                  (threadIdx.x & 15);
                columns[(i / kVecTiles & 1) * (kVecTiles * 16) + threadIdx.x] = n < a.N ? ws[n] : 0.f;
            }
            i32x4 acc = {0, 0, 0, 0};
            for (int t = 0; t < ns; ++t) {
                if constexpr (FAST) {
                    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(2 * (DEPTH - 1)) : "memory");
                } else {
                    *reinterpret_cast<u32x4 *>(ring + lane * 16) = hold[0];
                    *reinterpret_cast<u32x4 *>(ring + 1024 + lane * 16) = hold[1];
                    fetch();
                    __builtin_amdgcn_wave_barrier();
                }
                const char *slab = ring + buf * kVecSlab;
                const char *x = rows_lds + ((wave + kVecWaves * t) * R + xr) * 128;
                i32x4 wf[2], xf[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    wf[k] = *reinterpret_cast<const i32x4 *>(
                        slab + l16 * 128 + (((4 * k + g) ^ ((l16 >> 1) & 7)) << 4));
                    xf[k] = *reinterpret_cast<const i32x4 *>(x + (((4 * k + g) ^ ((xr >> 1) & 7)) << 4));
                }
                if constexpr (FAST) {
                    // Read before the buffer is filled again.
                    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(wf[0]), "+v"(wf[1]) : : "memory");
                    fetch();
                    buf = buf + 1 == DEPTH ? 0 : buf + 1;
                } else {
                    __builtin_amdgcn_wave_barrier();
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[k], xf[k], acc, 0, 0, 0);
            }
            // Two sets of sums in turn, so that one barrier a tile is enough.
            int *tile = sums + (i & 1) * (kVecWaves * 256);
            *reinterpret_cast<i32x4 *>(tile + wave * 256 + l16 * 16 + 4 * g) = acc;
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const int row = threadIdx.x >> 4, n = n0 + (threadIdx.x & 15);
            if (row < R && n < a.N) {
                const float w = columns[i % (2 * kVecTiles) * 16 + (threadIdx.x & 15)];
                int sum = 0;
#pragma unroll
                for (int v = 0; v < kVecWaves; ++v) sum += tile[v * 256 + threadIdx.x];
                static_cast<TY *>(a.Y)[(int64_t)(first + row) * a.ldy + n] =
                    (TY)((float)sum * scales[row] * w);
            }
        }
        if constexpr (FAST) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();  // the rows and the rings may be written again
    }
}

// ------------------------------------------------------ tens of rows

// A tile of BM x BN whose contraction the workgroup's waves split, slab by slab of 128 bytes.  With tens
// to hundreds of rows the operands come from L2, and the tiles have to be small for every unit to have
// some; waves that split such a tile among them wait for each other at every slab and read LDS several times
// over.  Here each wave has a ring of its own, no barrier before the end of the contraction, and
// reads each byte of LDS once; the sums, exact in any order, meet in LDS.  Rings are short, so that a unit
// has two or three workgroups.  us in a graph, K = N = 4096, with this and with the best of the tile
// kernels: 16 rows 5.6 and 13.0, 64 rows 7.0 and 13.4, 128 rows 9.4 and 13.7, 256 rows 12.0 and 13.9, 512 rows
// 17.2 and 17.5 (17.1-19.0 over several runs); 64 rows with K 14336 13.8 and 35.0.  64 rows in tiles of 32 x 32 with eight waves took 7.5
// where this took 6.6, with rings of three slabs 6.9, in tiles of 64 x 16 7.5, of 64 x 32 8.6.  A tile of
// 128 x 128 for each wave, which reads the least LDS of all, was slower or (1024 rows) within 3% of the
// tile kernels: its waves read their slabs and multiply in step.
constexpr int kSplitWaves = 4;

// Workgroups a unit's LDS has room for, of which three are enough.
constexpr int split_room(int ring)
{
    return 160 * 1024 / ring < 3 ? 160 * 1024 / ring : 3;
}

template <typename TY, int BM, int BN, int DEPTH, bool GROUPED, bool FAST>
__global__ void __launch_bounds__(kSplitWaves * 64)
    __attribute__((amdgpu_waves_per_eu(split_room(kSplitWaves * DEPTH * (BM + BN) * 128))))
q8_split_kernel(TileArgs g)
{
    constexpr int WAVES = kSplitWaves;
    constexpr int STAGE = (BM + BN) * 128, LPW = STAGE / 1024, FM = BM / 16, FN = BN / 16;
    constexpr int RING = WAVES * DEPTH * STAGE;
    // Columns whose sums of all waves fit the rings at once.
    constexpr int BLOCK = WAVES * BM * 16 * 4, FIT = RING / BLOCK, COLS = FIT >= FN ? FN : FN % FIT == 0 ? FIT : 1;
    static_assert(FIT >= 1 && FN % COLS == 0, "whole blocks of columns");
    static_assert(LPW * (DEPTH - 1) <= 63, "loads in flight must fit the vmcnt field");
    static_assert(FAST || DEPTH == 1, "the register path has one buffer");
    __shared__ __attribute__((aligned(1024))) char lds[RING];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    TY *C = static_cast<TY *>(g.C);

    int tm, tn, group = 0, begin = 0, end = g.M;
    if constexpr (GROUPED) {
        if (!rows_tile_of_block(g, BM, BN, byte_band(true), tm, tn, group, begin, end)) {
            if (g.fill) zero_outside(g.offsets, g.groups, g.M, g.N, C, g.ldc);
            return;
        }
    } else {
        tile_of_block(blockIdx.x, (g.M + BM - 1) / BM, (g.N + BN - 1) / BN, byte_band(false), tm, tn);
    }
    const int first = begin + tm * BM, n0 = tn * BN;
    const int rows = end - first < BM ? end - first : BM;
    const char *pa = static_cast<const char *>(g.A) + first * g.lda;
    const char *pb = static_cast<const char *>(g.B) + group * g.group_stride + n0 * g.ldb;
    const int64_t left_a = (int64_t)(rows - 1) * g.lda + g.K;
    const int64_t left_b = (int64_t)(g.N - 1 - n0) * g.ldb + g.K;
    const int slabs = (g.K + 127) / 128;

    // The results' columns and rows of this thread, and their scales, long before they are used.
    constexpr int QUADS = COLS * 4, THREADS = WAVES * 64, ITEMS = (BM * QUADS + THREADS - 1) / THREADS;
    static_assert(THREADS % QUADS == 0, "a thread's items are in one column");
    const int out_col = threadIdx.x % QUADS * 4, out_row = threadIdx.x / QUADS;
    const float *sb = g.scale_b + (int64_t)group * g.N;
    float row_scale[ITEMS];
    f32x4 col_scale[FN / COLS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int r = out_row + i * (THREADS / QUADS);
        row_scale[i] = g.scale_a[first + (r < rows ? r : rows - 1)];
    }
#pragma unroll
    for (int c = 0; c < FN / COLS; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = n0 + c * (COLS * 16) + out_col + q;
            col_scale[c][q] = sb[n < g.N ? n : g.N - 1];
        }

    // Load i: eight rows of A or B, 16 bytes a lane.
    uint32_t voff[FAST ? LPW : 1];
    const uint8_t *src[FAST ? 1 : LPW];
    u32x4 hold[FAST ? 1 : LPW];
    const uint8_t *ends[2] = {reinterpret_cast<const uint8_t *>(pa) + left_a,
                              reinterpret_cast<const uint8_t *>(pb) + left_b};
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
        const bool of_a = i < BM / 8;
        const int row = (of_a ? i : i - BM / 8) * 8 + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
        if constexpr (FAST) {
            voff[i] = (uint32_t)row * (uint32_t)(of_a ? g.lda : g.ldb) + chunk * 16u;
        } else {  // (Rows past the last repeat it, and are not stored.)
            const int last = of_a ? rows - 1 : g.N - 1 - n0;
            src[i] = reinterpret_cast<const uint8_t *>(of_a ? pa : pb) +
                     (row < last ? row : last) * (of_a ? g.lda : g.ldb) + chunk * 16;
        }
    }
    char *ring = lds + wave * (DEPTH * STAGE);
    u32x4 ra, rb;
    uint32_t at;
    const auto aim = [&](int t, int buf) {  // at slab t's bytes and where they go
        // (Past the last slab: nothing is in range, and zeros are written.)
        ra = descriptor(pa + t * (int64_t)128, t < slabs ? left_a - t * (int64_t)128 : 0);
        rb = descriptor(pb + t * (int64_t)128, t < slabs ? left_b - t * (int64_t)128 : 0);
        at = (uint32_t)(uintptr_t)(lds_char *)ring + buf * STAGE;
        // Wait states between a vector unit's write of these and their use.
        asm volatile("s_nop 4" : "+s"(ra), "+s"(rb), "+s"(at));
    };
    const auto load = [&](int i) { load_slab16(i < BM / 8 ? ra : rb, voff[i], at + i * 1024); };
    // Rows at any byte: slab t into registers, while the one before it is multiplied.
    const auto take = [&](int t) {
        if (t >= slabs) return;
#pragma unroll
        for (int i = 0; i < LPW; ++i) {
            const uint8_t *p = src[i] + t * (int64_t)128, *end = ends[i < BM / 8 ? 0 : 1];
            if (p + 16 <= end) {
                __builtin_memcpy(&hold[i], p, 16);
            } else {
                hold[i] = u32x4{0, 0, 0, 0};
                for (int j = 0; j < 16; ++j)
                    if (p + j < end) hold[i][j / 4] |= (uint32_t)p[j] << (8 * (j % 4));
            }
        }
    };
    if constexpr (FAST) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            aim(wave + d * WAVES, d);
#pragma unroll
            for (int i = 0; i < LPW; ++i) load(i);
        }
    } else {
        take(wave);
    }
    i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int l16 = lane & 15, lg = lane >> 4;
    int buf = 0;
    for (int t = wave; t < slabs; t += WAVES) {
        if constexpr (FAST) {
            asm volatile("s_waitcnt vmcnt(%0)" : : "n"(LPW * (DEPTH - 1)) : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < LPW; ++i) *reinterpret_cast<u32x4 *>(ring + i * 1024 + lane * 16) = hold[i];
            __builtin_amdgcn_wave_barrier();  // a wave's writes and reads of LDS stay in order
            take(t + WAVES);
        }
        const char *slab = ring + buf * STAGE + l16 * 128;
        i32x4 a[2][FM], b[2][FN];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = ((4 * k + lg) ^ ((l16 >> 1) & 7)) << 4;
#pragma unroll
            for (int i = 0; i < FM; ++i) a[k][i] = *reinterpret_cast<const i32x4 *>(slab + i * 2048 + c);
#pragma unroll
            for (int j = 0; j < FN; ++j) b[k][j] = *reinterpret_cast<const i32x4 *>(slab + BM * 128 + j * 2048 + c);
        }
        if constexpr (FAST) {
            // Read before the buffer is filled again.
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            aim(t + DEPTH * WAVES, buf);
            buf = buf + 1 == DEPTH ? 0 : buf + 1;
        } else {
            __builtin_amdgcn_wave_barrier();
        }
        if (t == slabs - 1 && g.K % 128) {
            // What lies past K is anything: it meets zeros.
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int keep = g.K - t * 128 - (4 * k + lg) * 16 - 4 * w;  // bytes of this word
                    const uint32_t mask = keep >= 4 ? ~0u : keep <= 0 ? 0u : (1u << (8 * keep)) - 1u;
#pragma unroll
                    for (int i = 0; i < FM; ++i) a[k][i][w] &= (int)mask;
                }
        }
        // The next slab's loads: between the products where these are many, since all at once they would
        // keep them waiting.
        constexpr int M = 2 * FM * FN;
        if constexpr (FAST && M < 32) {
#pragma unroll
            for (int i = 0; i < LPW; ++i) load(i);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if constexpr (FAST && M >= 32) {
                        static_assert(M < 32 || LPW <= M, "a load at a product at most");
                        const int n = (k * FM + i) * FN + j;
                        if (n * LPW % M < LPW) {
                            load(n * LPW / M);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[k][j], a[k][i], acc[i][j], 0, 0, 0);
                }
    }
    // ---- the waves' sums meet in LDS: blocks of 16 x 16, a lane's four columns in one piece
#pragma unroll
    for (int c = 0; c < FN / COLS; ++c) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int j = 0; j < COLS; ++j)
#pragma unroll
            for (int i = 0; i < FM; ++i)
                *reinterpret_cast<i32x4 *>(lds + ((wave * COLS + j) * FM + i) * 1024 + (l16 * 4 + lg) * 16) =
                    acc[i][c * COLS + j];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int r = out_row + i * (THREADS / QUADS), n = n0 + c * (COLS * 16) + out_col;
            if (r >= rows || n >= g.N) continue;
            const char *p = lds + ((out_col >> 4) * FM + (r >> 4)) * 1024 + ((r & 15) * 4 + (out_col >> 2 & 3)) * 16;
            i32x4 sum = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < WAVES; ++w) sum += *reinterpret_cast<const i32x4 *>(p + w * (COLS * FM * 1024));
            typedef TY Vec __attribute__((ext_vector_type(4)));
            typedef Vec Loose __attribute__((aligned(sizeof(TY))));
            Vec y;
#pragma unroll
            for (int q = 0; q < 4; ++q) y[q] = (TY)((float)sum[q] * row_scale[i] * col_scale[c][q]);
            TY *out = C + (int64_t)(first + r) * g.ldc + n;
            if (n + 4 <= g.N) {
                *reinterpret_cast<Loose *>(out) = y;
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (n + q < g.N) out[q] = y[q];
            }
        }
    }
    if constexpr (GROUPED)
        if (g.fill) zero_outside(g.offsets, g.groups, g.M, g.N, C, g.ldc);
}

}  // namespace lm
}  // namespace sgemm
