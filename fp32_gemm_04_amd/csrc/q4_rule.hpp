// Which kernel a product with weights held in 4 bits runs with, and what it stages in LDS: a
// rule on sizes alone, in plain C++.
#pragma once

#include <cstdint>

#include "lm_host.hpp"

namespace sgemm {
namespace q4 {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;

// Chunks of weights a wave keeps in flight: 4 KB, which with 16 waves on a compute
// unit covers the latency of memory at its full rate.
constexpr int ring_depth(int nt) { return nt == 1 ? 4 : 2; }
constexpr int ring_bytes(int nt) { return kWaves * ring_depth(nt) * nt * 1024; }

// bf16 parts of a value, and bytes of a staged scale with its zero, by the size of an element.
constexpr int parts_of(int size) { return size == 2 ? 1 : 3; }
constexpr int entry_bytes(int size) { return size == 2 ? 4 : 8; }

// Bytes of LDS after the ring.
inline int64_t slab_bytes(int size, int64_t slab, int block, int cols, int pass)
{
    return slab / block * ((cols + 1) * entry_bytes(size) + pass * 4) +
           parts_of(size) * pass * (slab * 2 + 16) + 16;
}

struct Q4Plan {
    int rt, nt;     // groups of 16 rows, and of 16 columns, a wave
    int wn;         // waves along n
    int cols;       // columns of a workgroup
    int pass;       // rows per pass
    int slab_log2;  // k per slab
    int lds;        // bytes
};

inline Q4Plan q4_plan(int size, bool offsets, int groups, int rows, int64_t N, int64_t K, int block,
                      int cus)
{
    using lm::ceil_div;
    Q4Plan p;
    const int parts = parts_of(size);
    const int used = groups < rows ? groups : rows;
    const int64_t mean = ceil_div(rows, used);  // rows of a group
    // Rows per pass: no more than a group is likely to have, so that more of K is staged
    // at once.
    const int64_t likely = offsets ? 2 * mean : rows;
    const int most_pass = parts == 1 ? 64 : 24;
    p.pass = likely < most_pass ? (int)likely : most_pass;
    p.rt = p.pass > 32 ? 4 : p.pass > 16 ? 2 : 1;
    p.nt = p.pass > 16 ? 2 : 1;
    // The more columns a workgroup takes (NT per wave, wn waves), the less often x is
    // staged and read: until four workgroups remain per compute unit, or 1.5 where
    // staging x (two bytes a part, against half a byte a weight) would outweigh the
    // weights.
    const int64_t tiles = used * ceil_div(N, 16);
    p.wn = 1;
    while (p.wn < kWaves) {
        const int cols = 16 * p.nt * p.wn;
        const int64_t left = tiles / (p.nt * p.wn * 2);
        if (left < (cols < 8 * p.pass * parts ? cus * 3 / 2 : 4 * cus)) break;
        if (p.nt == 1)
            p.nt = 2;
        else
            p.wn *= 2;
    }
    // What a slab of one chunk per wave needs must fit in 32 KB of LDS beside the rings'
    // 32 KB (two workgroups per compute unit).  With wn = 8 every pass does.
    int64_t room = 32 * 1024;
    const auto fits = [&](int64_t slab) {
        return slab_bytes(size, slab, block, p.wn * p.nt * 16, p.pass) <= room;
    };
    while (p.wn < kWaves && !fits(128 * kWaves / p.wn)) p.wn *= 2;
    p.cols = p.wn * p.nt * 16;
    if (used * ceil_div(N, p.cols) <= cus) room = 124 * 1024;
    int64_t slab = 128 * kWaves / p.wn;
    while (slab < K && fits(slab * 2)) slab *= 2;
    p.slab_log2 = __builtin_ctzll((unsigned long long)slab);
    const int64_t staged = ring_bytes(p.nt) + slab_bytes(size, slab, block, p.cols, p.pass);
    const int64_t sums = kWaves / p.wn * p.pass * p.cols * 4;
    p.lds = (int)(staged > sums ? staged : sums);
    return p;
}

}  // namespace q4
}  // namespace sgemm
