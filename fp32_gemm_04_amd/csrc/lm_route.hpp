// Tokens on their way to experts and back (include/slm.h): a stable counting sort of the
// experts' numbers, and copies between tokens' rows and experts' rows.
//
// Everything is addressed from the token's side by place, the row of each of its k choices:
// the way in reads a token once and writes k rows, the way back reads k rows and writes a
// token once, so neither direction needs atomics, and sums have one order.
#pragma once

#include <climits>
#include <type_traits>

#include "lm_tile.hpp"

namespace sgemm {
namespace lm {

// ------------------------------------------------------------------- sorting

struct SortArgs {
    const int64_t *experts;
    int *offsets, *order, *place;
    int *counts;    // of each expert and segment, or null: counted by every workgroup itself
    int slots, groups;
    int segment;    // slots of a workgroup, a multiple of a chunk
    int segments;
    int pitch;      // counts of one expert: segments, rounded up to 4
};

// The place of an expert's number among the counters: those outside come last.
__device__ __forceinline__ int sort_key(const int64_t *experts, int64_t slot, int groups)
{
    const int64_t e = experts[slot];
    return e >= 0 && e < groups ? (int)e : groups;
}

// Counts of each segment's slots by expert, for the sort of many slots.
__global__ void __launch_bounds__(1024) sort_count_kernel(SortArgs a)
{
    extern __shared__ int hist[];
    const int n = a.groups + 1;
    for (int e = threadIdx.x; e < n; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * a.segment;
    const int64_t s1 = s0 + a.segment < a.slots ? s0 + a.segment : a.slots;
#pragma unroll 4
    for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x)
        atomicAdd(&hist[sort_key(a.experts, s, a.groups)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += blockDim.x)
        a.counts[(int64_t)e * a.pitch + blockIdx.x] = hist[e];
}

// One segment's slots to their rows.  A slot's row is the number of slots with a lower
// expert, of earlier segments' with its own, and of earlier ones in its segment.  The last is
// found 64 slots at a time: the lanes with one expert are the and, over the bits of its
// number, of the ballots of that bit (or their complements); the first of them advances
// the wave's counter of the expert.  Integer counts: any order of the atomics gives the same.
// A chunk is ITEMS slots of each lane, in registers.
template <int ITEMS>
__global__ void __launch_bounds__(1024) sort_place_kernel(SortArgs a)
{
    extern __shared__ int shared[];
    __shared__ int wave_sum[16];
    const int n = a.groups + 1, waves = blockDim.x >> 6, chunk = blockDim.x * ITEMS;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int *base = shared;                                            // n: next row of each expert
    int *total = shared + n;                                       // n
    uint16_t *cnt = reinterpret_cast<uint16_t *>(shared + 2 * n);  // waves x n
    uint16_t *own = cnt + wave * n;
    const int64_t s0 = (int64_t)blockIdx.x * a.segment;
    const int64_t s1 = s0 + a.segment < a.slots ? s0 + a.segment : a.slots;
    int key[ITEMS], rank[ITEMS];
    const auto load = [&](int64_t c0) {
        const int64_t w0 = c0 + wave * (64 * ITEMS) + lane;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            key[i] = w0 + i * 64 < s1 ? sort_key(a.experts, w0 + i * 64, a.groups) : n;
    };
    load(s0);
    // All slots by expert, and those of earlier segments.  (One chunk counts itself below.)
    const bool alone = a.slots <= chunk;
    // Without counts: some sets of counters in cnt's place, of earlier slots and of the others, so that
    // neighbouring lanes with one expert wait less for each other.
    const int sets = waves / 4;
    int *part = shared + 2 * n;
    for (int e = threadIdx.x; e < (a.counts || alone ? 2 : 2 + 2 * sets) * n; e += blockDim.x) shared[e] = 0;
    __syncthreads();
    if (a.counts) {
        // Some threads for each expert, 16 bytes of its counts at a time.
        const int quads = a.pitch / 4;
        const int share = (int)blockDim.x / n < 1 ? 1 : (int)blockDim.x / n;
        const int mine = threadIdx.x / n;
        for (int e = threadIdx.x - mine * n; e < n && mine < share; e += blockDim.x) {
            const i32x4 *c = reinterpret_cast<const i32x4 *>(a.counts + (int64_t)e * a.pitch);
            int all = 0, earlier = 0;
#pragma unroll 8
            for (int q = mine; q < quads; q += share) {
                const i32x4 v = c[q];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s = 4 * q + i;
                    all += s < a.segments ? v[i] : 0;
                    earlier += s < (int)blockIdx.x ? v[i] : 0;
                }
            }
            atomicAdd(&total[e], all);
            atomicAdd(&base[e], earlier);
        }
    } else if (!alone) {
        // Pairs of slots, four loads in flight; past the last pair it is read again and not counted.
        // (4096 slots 5.8 us, 12297 6.7; single slots and one set of counters took 1.0 and 1.2 more.)
        typedef int64_t Pair __attribute__((ext_vector_type(2)));
        typedef Pair LoosePair __attribute__((aligned(8)));
        const auto count = [&](int64_t expert, int at) {
            const int e = expert >= 0 && expert < a.groups ? (int)expert : a.groups;
            if (at < a.slots) atomicAdd(&part[((at < s0 ? sets : 0) + (lane & (sets - 1))) * n + e], 1);
        };
        for (int s = 2 * threadIdx.x; s < a.slots; s += 8 * blockDim.x) {
            Pair e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = s + 2 * i * (int)blockDim.x;
                e[i] = *reinterpret_cast<const LoosePair *>(a.experts + (at < a.slots - 1 ? at : a.slots - 2));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = s + 2 * i * (int)blockDim.x;
                count(at < a.slots - 1 ? e[i][0] : e[i][1], at);
                count(e[i][1], at + 1);
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < n; e += blockDim.x) {
            int earlier = 0, others = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int s = c < sets ? c : 0;
                const int o = part[s * n + e], b = part[(sets + s) * n + e];
                others += c < sets ? o : 0;
                earlier += c < sets ? b : 0;
            }
            base[e] = earlier;
            total[e] = earlier + others;
        }
        __syncthreads();  // cnt's place is free
    }
    const int bits = 32 - __builtin_clz(n);  // n itself marks lanes without a slot
    for (int64_t c0 = s0; c0 < s1 || c0 == s0; c0 += chunk) {
        for (int e = lane; e < n; e += 64) own[e] = 0;
        if (c0 > s0) load(c0);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            uint64_t same = ~0ull;
            for (int b = 0; b < bits; ++b) {
                const uint64_t set = __ballot(key[i] >> b & 1);
                same &= key[i] >> b & 1 ? set : ~set;
            }
            const int lower = __popcll(same & ((1ull << lane) - 1));
            rank[i] = 0;
            __builtin_amdgcn_wave_barrier();  // a wave's reads and writes of LDS stay in order
            if (key[i] < n) rank[i] = *(volatile uint16_t *)(own + key[i]) + lower;
            __builtin_amdgcn_wave_barrier();
            if (key[i] < n && lower == 0)
                *(volatile uint16_t *)(own + key[i]) = (uint16_t)(rank[i] + __popcll(same));
        }
        __syncthreads();
        // The waves' counts to rows before each wave's; a chunk that is all there is: the totals.
        for (int e = threadIdx.x; e < n; e += blockDim.x) {
            int sum = 0;
            for (int w = 0; w < waves; w += 8) {  // eight or sixteen: read at once
                int v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = cnt[(w + i) * n + e];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cnt[(w + i) * n + e] = (uint16_t)sum;
                    sum += v[i];
                }
            }
            if (alone) total[e] = sum;
        }
        __syncthreads();
        if (c0 == s0) {
            // Rows before each expert: every thread sums `per` neighbouring experts.
            const int per = (n + blockDim.x - 1) / blockDim.x, e0 = threadIdx.x * per;
            int mine = 0;
            for (int e = e0; e < e0 + per && e < n; ++e) mine += total[e];
            int before = mine;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(before, d);
                if (lane >= d) before += v;
            }
            if (lane == 63) wave_sum[wave] = before;
            __syncthreads();
            for (int w = 0; w < wave; ++w) before += wave_sum[w];
            before -= mine;
            for (int e = e0; e < e0 + per && e < n; ++e) {
                if (blockIdx.x == 0) a.offsets[e] = before;
                base[e] += before;
                before += total[e];
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (key[i] >= n) continue;
            const int slot = (int)(c0 + wave * (64 * ITEMS) + i * 64 + lane);
            const int row = base[key[i]] + own[key[i]] + rank[i];
            a.place[slot] = key[i] < a.groups ? row : -2 - row;
            if (a.order) a.order[row] = slot;
        }
        if (c0 + chunk >= s1) break;
        __syncthreads();
        // The next chunk's rows follow.
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (key[i] < n) atomicAdd(&base[key[i]], 1);
        __syncthreads();
    }
}

// ------------------------------------------------------------------- copies

struct RouteArgs {
    const void *X;         // tokens' rows (gather: X; backward: dout)
    const void *R;         // experts' rows that are read
    void *out;             // gather, backward: experts' rows; combine: tokens' rows
    const int *place;
    const float *weights;  // or null: 1
    float *dweights;       // or null
    int64_t ldx, ldr, ldo;
    int tokens, k, H, rows;
    int fill;
    float beta;
    int cols_log2;         // threads of a workgroup along a row (of 256)
};

// Sixteen bytes of a row (E values); addresses need the element's alignment only.
template <typename T> struct Piece {
    static constexpr int E = 16 / sizeof(T);
    typedef T Vec __attribute__((ext_vector_type(E)));
    typedef Vec Loose __attribute__((aligned(sizeof(T))));
    Vec v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const Loose *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Loose *>(p) = v; }
    __device__ __forceinline__ void zero() { v = (T)0.f; }
};
// One value, for what is left of a row after its whole pieces.
template <typename T> struct Single {
    static constexpr int E = 1;
    T v[1];
    __device__ __forceinline__ void load(const T *p) { v[0] = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v[0]; }
    __device__ __forceinline__ void zero() { v[0] = (T)0.f; }
};

// Up to N choices of a token from j0 on: their places and weights.  The kernels handle KT at a
// time, whose rows are all in flight at once.
template <bool UNIFORM, int N> struct Choices {
    int p[N];
    float w[N];
    uint32_t rows;
    __device__ __forceinline__ Choices(const RouteArgs &a, int t, int j0, bool weighted) : rows(a.rows)
    {
        // (Past the last choice the last is read again: loads without branches.)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t slot = (int64_t)t * a.k + (j0 + j < a.k ? j0 + j : a.k - 1);
            p[j] = read<UNIFORM>(a.place, slot);
            if (j0 + j >= a.k) p[j] = -1;
            w[j] = 1.f;
            if (weighted) w[j] = read<UNIFORM>(a.weights, slot);
        }
    }
    // Choice j has row p[j]; or it is dropped, and row -2 - p[j] is one that no expert has.
    __device__ __forceinline__ bool held(int j) const { return (uint32_t)p[j] < rows; }
    __device__ __forceinline__ bool dropped(int j) const { return (uint32_t)(-2 - p[j]) < rows; }
};

// Turns of workgroups over the tokens' rows: `parts` of a row's whole pieces, each a thread.
template <int E> struct Turns {
    int cols, per, parts;
    int64_t count;
    __device__ __forceinline__ explicit Turns(const RouteArgs &a)
        : cols(1 << a.cols_log2), per(256 >> a.cols_log2)
    {
        parts = (a.H / E + cols - 1) >> a.cols_log2;
        if (parts == 0) parts = 1;
        count = ((int64_t)a.tokens + per - 1) / per * parts;
    }
    // Turn b: which `per` tokens, and which part of their rows.
    __device__ __forceinline__ int64_t tokens(int64_t b, int &part) const
    {
        part = 0;
        if (parts == 1) return b;
        if (b <= INT_MAX) {  // 32 bits: a division of 64 is a hundred instructions
            const uint32_t q = (uint32_t)b / (uint32_t)parts;
            part = (int)((uint32_t)b - q * parts);
            return q;
        }
        part = (int)(b % parts);
        return b / parts;
    }
};

// f(piece, column) for what this thread has of a row in a part of it: a whole piece, and, in the
// first part, the values after the last whole piece, one each for as many threads.
template <typename T, typename F>
__device__ __forceinline__ void row_pieces(const RouteArgs &a, int cols, int col, int part, F f)
{
    constexpr int E = Piece<T>::E;
    const uint32_t h = ((uint32_t)part * cols + col) * E, whole = (uint32_t)a.H / E * E;
    if (h < whole) f(Piece<T>(), (int)h);
    if (part == 0)
        for (uint32_t at = whole + col; at < (uint32_t)a.H; at += cols) f(Single<T>(), (int)at);
}

// The token of a workgroup's turn.  UNIFORM: a wave has one, and the compiler is told so: its
// places and weights then are scalar loads, and its rows' addresses a scalar base each, where
// vector loads of them would be two more for each of a row.
template <bool UNIFORM>
__device__ __forceinline__ int64_t token_of(const RouteArgs &a, int64_t turn, int per)
{
    int sub = threadIdx.x >> a.cols_log2;
    if constexpr (UNIFORM) sub = __builtin_amdgcn_readfirstlane(sub);
    return turn * per + sub;
}

// R[place] <- w X[t], a thread per 16 bytes of a token.
template <typename T, int KT, bool WEIGHTED, bool UNIFORM>
__global__ void __launch_bounds__(256) gather_kernel(RouteArgs a)
{
    const Turns<Piece<T>::E> turns(a);
    for (int64_t b = blockIdx.x; b < turns.count; b += gridDim.x) {
        int part;
        const int64_t at_token = token_of<UNIFORM>(a, turns.tokens(b, part), turns.per);
        if (at_token >= a.tokens) continue;
        const int t = (int)at_token;
        const auto copy = [&](auto x, int at) {
            x.load(static_cast<const T *>(a.X) + t * a.ldx + at);
            for (int j0 = 0; j0 < a.k; j0 += KT) {
                const Choices<UNIFORM, KT> c(a, t, j0, WEIGHTED);
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    auto y = x;
                    if (c.held(j)) {
                        if constexpr (WEIGHTED) {
#pragma unroll
                            for (int i = 0; i < x.E; ++i) y.v[i] = (T)(c.w[j] * (float)x.v[i]);
                        }
                        y.store(static_cast<T *>(a.out) + c.p[j] * a.ldo + at);
                    } else if (a.fill && c.dropped(j)) {
                        y.zero();
                        y.store(static_cast<T *>(a.out) + (-2 - c.p[j]) * a.ldo + at);
                    }
                }
            }
        };
        row_pieces<T>(a, turns.cols, threadIdx.x & (turns.cols - 1), part, copy);
    }
}

// out[t] <- beta out[t] + sum_j w R[place], a thread per 16 bytes of a token.
template <typename T, int KT, bool UNIFORM>
__global__ void __launch_bounds__(256) combine_kernel(RouteArgs a)
{
    const Turns<Piece<T>::E> turns(a);
    for (int64_t b = blockIdx.x; b < turns.count; b += gridDim.x) {
        int part;
        const int64_t at_token = token_of<UNIFORM>(a, turns.tokens(b, part), turns.per);
        if (at_token >= a.tokens) continue;
        const int t = (int)at_token;
        const auto sum_up = [&](auto y, int at) {
            float sum[y.E];
#pragma unroll
            for (int i = 0; i < y.E; ++i) sum[i] = 0.f;
            for (int j0 = 0; j0 < a.k; j0 += KT) {
                const Choices<UNIFORM, KT> c(a, t, j0, a.weights != nullptr);
                decltype(y) x[KT];
#pragma unroll
                for (int j = 0; j < KT; ++j)
                    if (c.held(j)) x[j].load(static_cast<const T *>(a.R) + c.p[j] * a.ldr + at);
#pragma unroll
                for (int j = 0; j < KT; ++j)
                    if (c.held(j))
#pragma unroll
                        for (int i = 0; i < y.E; ++i) sum[i] = fmaf(c.w[j], (float)x[j].v[i], sum[i]);
            }
            T *out = static_cast<T *>(a.out) + t * a.ldo + at;
            if (a.beta != 0.f) {
                y.load(out);
#pragma unroll
                for (int i = 0; i < y.E; ++i) sum[i] = fmaf(a.beta, (float)y.v[i], sum[i]);
            }
#pragma unroll
            for (int i = 0; i < y.E; ++i) y.v[i] = (T)sum[i];
            y.store(out);
        };
        row_pieces<T>(a, turns.cols, threadIdx.x & (turns.cols - 1), part, sum_up);
    }
}

// p, in a way that keeps what is computed from it where it is used: the addresses of eight rows of
// two operands, taken out of a loop, would not fit the scalar registers.
__device__ __forceinline__ int here_only(int p)
{
    asm("" : "+s"(p));
    return p;
}

// dR[place] <- w dout[t] and dw = <dout[t], R[place]>: WAVES waves share a token, KT of its
// choices at a time.
template <typename T, int WAVES, int KT>
__global__ void __launch_bounds__(256) combine_backward_kernel(RouteArgs a)
{
    constexpr int E = Piece<T>::E, TOKENS = 4 / WAVES;
    __shared__ float parts[4][KT];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < a.tokens; t0 += (int64_t)gridDim.x * TOKENS) {
        const bool here = t0 + wave / WAVES < a.tokens;
        const int t = (int)(here ? t0 + wave / WAVES : a.tokens - 1);
        for (int j0 = 0; j0 < a.k; j0 += KT) {
            float dot[KT];
#pragma unroll
            for (int j = 0; j < KT; ++j) dot[j] = 0.f;
            if (here && a.rows > 0) {
                const Choices<true, KT> c(a, t, j0, a.weights != nullptr);
                const auto both = [&](auto d, int at) {
                    decltype(d) x[KT];
                    if (a.dweights) {
#pragma unroll
                        for (int j = 0; j < KT; ++j)
                            if (c.held(j)) x[j].load(static_cast<const T *>(a.R) + here_only(c.p[j]) * a.ldr + at);
                    }
                    d.load(static_cast<const T *>(a.X) + t * a.ldx + at);
                    if (a.out) {
#pragma unroll
                        for (int j = 0; j < KT; ++j) {
                            auto y = d;
                            if (c.held(j)) {
#pragma unroll
                                for (int i = 0; i < d.E; ++i) y.v[i] = (T)(c.w[j] * (float)d.v[i]);
                                y.store(static_cast<T *>(a.out) + here_only(c.p[j]) * a.ldo + at);
                            } else if (a.fill && c.dropped(j)) {
                                y.zero();
                                y.store(static_cast<T *>(a.out) + here_only(-2 - c.p[j]) * a.ldo + at);
                            }
                        }
                    }
                    if (a.dweights) {
#pragma unroll
                        for (int j = 0; j < KT; ++j)
                            if (c.held(j))
#pragma unroll
                                for (int i = 0; i < d.E; ++i)
                                    dot[j] = fmaf((float)d.v[i], (float)x[j].v[i], dot[j]);
                    }
                };
                constexpr int THREADS = WAVES * 64;
                const uint32_t thread = (wave % WAVES) * 64 + lane, whole = (uint32_t)a.H / E * E;
                for (uint32_t h = thread * E; h < whole; h += THREADS * E) both(Piece<T>(), (int)h);
                if (whole + thread < (uint32_t)a.H) both(Single<T>(), (int)(whole + thread));
            }
            if (!a.dweights) continue;
            // While several sums are left a lane exchanges half of them for its neighbour's other
            // half: lane l ends with the sum of choice l % KT.
#pragma unroll
            for (int n = KT / 2, d = 1; d < 64; n /= 2, d *= 2) {
                if (n > 0) {
                    const bool odd = lane & d;
#pragma unroll
                    for (int j = 0; j < n; ++j) {
                        const float keep = odd ? dot[2 * j + 1] : dot[2 * j];
                        dot[j] = keep + __shfl_xor(odd ? dot[2 * j] : dot[2 * j + 1], d);
                    }
                } else {
                    dot[0] += __shfl_xor(dot[0], d);
                }
            }
            if constexpr (WAVES > 1) {
                if (lane < KT) parts[wave][lane] = dot[0];
                __syncthreads();
                dot[0] = 0.f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) dot[0] += parts[wave / WAVES * WAVES + w][lane % KT];
                __syncthreads();
            }
            if (here && wave % WAVES == 0 && lane < KT && j0 + lane < a.k)
                a.dweights[(int64_t)t * a.k + j0 + lane] = dot[0];
        }
    }
}

}  // namespace lm
}  // namespace sgemm
