// libsgemm rows sorted by expert: argument checks, launch shapes and launches, behind the C
// ABI declared in include/slm.h.  Nothing here allocates, frees, copies or synchronises.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/slm.h"
#include "lm_host.hpp"
#include "lm_route.hpp"

namespace sgemm {
namespace lm {
namespace {

constexpr int kMostGroups = 4096;
constexpr int kMostSegments = 256;

// How a sort is cut into segments of whole chunks, one a workgroup.  Few slots are counted by
// every workgroup for itself, in one launch; for more, a launch before counts each segment's.
struct SortPlan {
    int waves, items, segment, segments, pitch;
    int64_t bytes;  // of counts; 0: one launch
};

// us in a graph.  One launch and two: 4096 slots, 64 experts 5.8 and 7.5, 16384, 32 experts 7.1 and
// 7.4 (a call of Python's: 9.9 and 14.5), 32768, 128 experts 9.9 and 8.5.  Chunks of one and two slots a
// lane: 128 slots, 64 experts 4.0 and 4.7, 16384, 32 experts 7.1 and 8.3, 65536, 64 experts 8.2 and 9.1,
// 262144, 64 experts 10.6 both, 256 experts 19.8 and 15.0 (every workgroup reads all counts).
SortPlan sort_plan(int slots, int groups)
{
    SortPlan p;
    p.waves = groups <= 2048 ? 16 : 8;  // whose counters fit LDS
    const int most = slots > 0 ? slots : 1;
    p.items = slots <= 16384 || ceil_div(slots, p.waves * 64) * (groups + 1) <= 16384 ? 1 : 2;
    const int chunk = p.waves * 64 * p.items;
    const int64_t chunks = ceil_div(most, chunk);
    p.segments = (int)(chunks < kMostSegments ? chunks : kMostSegments);
    // The last segments may be empty.
    p.segment = (int)(ceil_div(chunks, p.segments) * chunk);
    p.pitch = (int)round_up(p.segments, 4);
    p.bytes = slots > 16384 ? (int64_t)p.pitch * (groups + 1) * 4 : 0;
    return p;
}

// The shape of a launch over tokens' rows: threads along a row, and workgroups.
int cols_log2(int pieces)
{
    int n = 0;
    while (n < 8 && (1 << n) < pieces) ++n;
    return n;
}

dim3 copy_grid(int tokens, int pieces, int log2)
{
    const int64_t work = ceil_div(tokens, 256 >> log2) * ceil_div(pieces, 1 << log2);
    return dim3((unsigned)(work < kMostBlocks ? work : kMostBlocks));
}

typedef void (*RouteFn)(RouteArgs);

// Two, four or eight choices at a time; from 64 threads a row on a wave has one token.  us with
// as many as k needs and with eight: gather of 4096 x 1 fp32 rows of 2048 12.4 and 17.4, weighted
// gather of 8192 x 2 bf16 rows of 4096 37.7 and 43.2, combine 38.2 and 41.7, its gradients 69.9 and 73.7.
template <typename T, int KT> RouteFn gather_of_choices(bool weighted, bool uniform)
{
    if (weighted) return uniform ? gather_kernel<T, KT, true, true> : gather_kernel<T, KT, true, false>;
    return uniform ? gather_kernel<T, KT, false, true> : gather_kernel<T, KT, false, false>;
}
template <typename T> RouteFn gather_of(int k, bool weighted, int cols_log2)
{
    const bool uniform = cols_log2 >= 6;
    return k <= 2   ? gather_of_choices<T, 2>(weighted, uniform)
           : k <= 4 ? gather_of_choices<T, 4>(weighted, uniform)
                    : gather_of_choices<T, 8>(weighted, uniform);
}
template <typename T> RouteFn combine_of(int k, int cols_log2)
{
    const bool uniform = cols_log2 >= 6;
    if (k <= 2) return uniform ? combine_kernel<T, 2, true> : combine_kernel<T, 2, false>;
    if (k <= 4) return uniform ? combine_kernel<T, 4, true> : combine_kernel<T, 4, false>;
    return uniform ? combine_kernel<T, 8, true> : combine_kernel<T, 8, false>;
}
template <typename T, int KT> RouteFn backward_of_choices(int waves)
{
    return waves == 1   ? combine_backward_kernel<T, 1, KT>
           : waves == 2 ? combine_backward_kernel<T, 2, KT>
                        : combine_backward_kernel<T, 4, KT>;
}
template <typename T> RouteFn backward_of(int k, int waves)
{
    return k <= 2   ? backward_of_choices<T, 2>(waves)
           : k <= 4 ? backward_of_choices<T, 4>(waves)
                    : backward_of_choices<T, 8>(waves);
}

// The checks that the copies share, of sizes; `type` is parameter 1, tokens 2, k 3, H 4.
int check_sizes(int type, int tokens, int k, int H)
{
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return -1;
    if (tokens < 0 || tokens > kMostExtent) return -2;
    if (k < 0 || (tokens > 0 && k > kMostExtent / tokens)) return -3;
    if (H < 0 || H > kMostExtent) return -4;
    return 0;
}

}  // namespace
}  // namespace lm
}  // namespace sgemm

using namespace sgemm::lm;

extern "C" int64_t sgemm_expert_sort_workspace(int slots, int groups)
{
    if (slots < 0 || slots > kMostExtent) return -1;
    if (groups < 0 || groups > kMostGroups) return -2;
    return sort_plan(slots, groups).bytes;
}

extern "C" int sgemm_expert_sort(int slots, int groups, const int64_t *experts, int *offsets,
                                 int *order, int *place, void *ws, int64_t ws_bytes,
                                 hipStream_t stream)
{
    if (slots < 0 || slots > kMostExtent) return -1;
    if (groups < 0 || groups > kMostGroups) return -2;
    if ((slots > 0 && !experts) || !aligned(experts, 8)) return -3;
    if (!offsets || !aligned(offsets, 4)) return -4;
    if (!aligned(order, 4)) return -5;
    if ((slots > 0 && !place) || !aligned(place, 4)) return -6;
    const SortPlan p = sort_plan(slots, groups);
    if ((p.bytes > 0 && !ws) || !aligned(ws, 16)) return -7;
    if (ws_bytes < p.bytes) return -8;
    SortArgs a = {};
    a.experts = experts, a.offsets = offsets, a.order = order, a.place = place;
    a.counts = p.bytes > 0 ? static_cast<int *>(ws) : nullptr;
    a.slots = slots, a.groups = groups;
    a.segment = p.segment, a.segments = p.segments, a.pitch = p.pitch;
    const int n = groups + 1;
    if (a.counts) {
        sort_count_kernel<<<dim3(p.segments), dim3(p.waves * 64), n * 4, stream>>>(a);
        if (int rc = (int)hipGetLastError()) return rc;
    }
    const int lds = 2 * n * 4 + p.waves * n * 2;
    (p.items == 1 ? sort_place_kernel<1> : sort_place_kernel<2>)<<<dim3(p.segments), dim3(p.waves * 64), lds, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_expert_gather(int type, int tokens, int k, int H, const void *X, int ldx,
                                   const int *place, const float *weights, int rows, void *R,
                                   int ldr, int fill, hipStream_t stream)
{
    if (int rc = check_sizes(type, tokens, k, H)) return rc;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = H > 1 ? H : 1;
    const bool work = tokens > 0 && k > 0 && H > 0 && rows > 0;
    if ((work && !X) || !aligned(X, size)) return -5;
    if (ldx < least) return -6;
    if ((work && !place) || !aligned(place, 4)) return -7;
    if (!aligned(weights, 4)) return -8;
    if (rows < 0 || rows > kMostExtent) return -9;
    if ((work && !R) || !aligned(R, size)) return -10;
    if (ldr < least) return -11;
    if (fill != 0 && fill != 1) return -12;
    if (!work) return 0;
    RouteArgs a = {};
    a.X = X, a.out = R, a.place = place, a.weights = weights;
    a.ldx = ldx, a.ldo = ldr;
    a.tokens = tokens, a.k = k, a.H = H, a.rows = rows, a.fill = fill;
    const int pieces = H / (16 / size) > 1 ? H / (16 / size) : 1;  // whole ones; the rest is theirs
    a.cols_log2 = cols_log2(pieces);
    const auto fn = type == SGEMM_TYPE_BF16 ? gather_of<bf16>(k, weights != nullptr, a.cols_log2)
                                            : gather_of<float>(k, weights != nullptr, a.cols_log2);
    fn<<<copy_grid(tokens, pieces, a.cols_log2), dim3(256), 0, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_expert_combine(int type, int tokens, int k, int H, int rows, const void *R,
                                    int ldr, const int *place, const float *weights, float beta,
                                    void *out, int ldo, hipStream_t stream)
{
    if (int rc = check_sizes(type, tokens, k, H)) return rc;
    if (rows < 0 || rows > kMostExtent) return -5;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = H > 1 ? H : 1;
    const bool work = tokens > 0 && H > 0, reads = work && k > 0 && rows > 0;
    if ((reads && !R) || !aligned(R, size)) return -6;
    if (ldr < least) return -7;
    if ((reads && !place) || !aligned(place, 4)) return -8;
    if (!aligned(weights, 4)) return -9;
    if ((work && !out) || !aligned(out, size)) return -11;
    if (ldo < least) return -12;
    if (!work) return 0;
    RouteArgs a = {};
    a.R = R, a.out = out, a.place = place, a.weights = weights;
    a.ldr = ldr, a.ldo = ldo, a.beta = beta;
    a.tokens = tokens, a.k = reads ? k : 0, a.H = H, a.rows = rows;
    const int pieces = H / (16 / size) > 1 ? H / (16 / size) : 1;  // whole ones; the rest is theirs
    a.cols_log2 = cols_log2(pieces);
    const auto fn = type == SGEMM_TYPE_BF16 ? combine_of<bf16>(a.k, a.cols_log2)
                                            : combine_of<float>(a.k, a.cols_log2);
    fn<<<copy_grid(tokens, pieces, a.cols_log2), dim3(256), 0, stream>>>(a);
    return (int)hipGetLastError();
}

extern "C" int sgemm_expert_combine_backward(int type, int tokens, int k, int H, int rows,
                                             const void *dout, int lddo, const void *R, int ldr,
                                             const int *place, const float *weights, void *dR,
                                             int lddr, int fill, float *dweights, hipStream_t stream)
{
    if (int rc = check_sizes(type, tokens, k, H)) return rc;
    if (rows < 0 || rows > kMostExtent) return -5;
    const int size = type == SGEMM_TYPE_BF16 ? 2 : 4, least = H > 1 ? H : 1;
    const bool slots = tokens > 0 && k > 0;
    const bool work = slots && H > 0 && rows > 0 && (dR || dweights);
    if ((work && !dout) || !aligned(dout, size)) return -6;
    if (lddo < least) return -7;
    if ((work && dweights && !R) || !aligned(R, size)) return -8;
    if (ldr < least) return -9;
    if ((work && !place) || !aligned(place, 4)) return -10;
    if (!aligned(weights, 4)) return -11;
    if (!aligned(dR, size)) return -12;
    if (lddr < least) return -13;
    if (fill != 0 && fill != 1) return -14;
    if (!aligned(dweights, 4)) return -15;
    // Without columns or rows the dot products are empty: zeros are still written.
    if (!slots || (!dR && !dweights) || (!work && !dweights)) return 0;
    RouteArgs a = {};
    a.X = dout, a.R = R, a.out = work ? dR : nullptr, a.place = place, a.weights = weights;
    a.dweights = dweights;
    a.ldx = lddo, a.ldr = ldr, a.ldo = lddr;
    a.tokens = tokens, a.k = k, a.H = H, a.rows = work ? rows : 0, a.fill = fill;
    // As many waves a token as its row has 16-byte pieces for.  us with 1, 2 and 4 waves: 32768 x 8
    // choices, 64 pieces 122, 132, 180; 128 pieces 232, 232, 242; 16384 x 4, 256 pieces 139, 135, 122;
    // 8192 x 2, 512 pieces 81, 73, 72.
    const int64_t pieces = ceil_div(H, 16 / size);
    const int waves = pieces <= 64 ? 1 : pieces <= 128 ? 2 : 4;
    const auto fn = type == SGEMM_TYPE_BF16 ? backward_of<bf16>(k, waves) : backward_of<float>(k, waves);
    const int64_t blocks = ceil_div(tokens, 4 / waves);
    fn<<<dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3(256), 0, stream>>>(a);
    return (int)hipGetLastError();
}
