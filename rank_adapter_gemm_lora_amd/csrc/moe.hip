// moe.hip -- a mixture layer's router and the grouping of its (row, choice)
// pairs by expert, and the weighted sum that brings the pairs' results back to
// their rows.
//
// Router.  A row's experts are its top_k largest logits, the lowest number
// first among equal ones.  G neighbouring lanes hold a row, V logits each, as
// integers that order like the floats; each choice is one maximum over the
// lanes' own values and a butterfly of register moves over the G lanes.  Of
// bf16 logits the key holds the expert's number in its lower half, so the
// maximum settles ties too; of fp32 logits a minimum over the numbers does.
//
// Grouping.  A stable counting sort, as for adapters: positions of equal keys
// inside a wavefront by ballots over the key's bits, wavefronts and steps by
// counts in LDS.  Batches of at most kMoeSmallPairs pairs take one workgroup
// and one launch, others two: rows in chunks, each with its histogram; then
// every workgroup sums the histograms of all chunks (and of those ahead of its
// own) and places its chunk.
#include "mx_device.h"
#include "moe.h"

namespace lora {

namespace {

constexpr int kMaxBuckets = LORA_MAX_EXPERTS + 1;   // the last: pairs without an expert
constexpr int kPlaceThreads = 1024;
constexpr int kPlaceWaves = kPlaceThreads / 64;
constexpr int kCountThreads = 1024;

template <int CTRL> __device__ __forceinline__ uint32_t lane_move(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// op over G lanes (16: a row of lanes; 64: the wavefront), the same result in all.
template <int G, class OP> __device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, OP op)
{
    v = op(v, lane_move<0xB1>(v));    // neighbours
    v = op(v, lane_move<0x4E>(v));    // pairs
    v = op(v, lane_move<0x141>(v));   // halves of a row of 16, mirrored
    v = op(v, lane_move<0x140>(v));   // rows, mirrored
    if constexpr (G == 64) {
        uint32_t r = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
        r = op(r, (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
        r = op(r, (uint32_t)__builtin_amdgcn_readlane((int)v, 32));
        v = op(r, (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
    }
    return v;
}
template <int G> __device__ __forceinline__ float lanes_sum(float v)
{
    return __uint_as_float(lanes_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// A logit as an integer that orders like it; 0, below every other, for -inf and
// NaN (experts that are switched off).  Both zeros are one.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);
    const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return x > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Choices of one row; lane j of the row's G lanes gets choice j (id -1, weight
// 0 where fewer experts are left).  `in`: the row exists; the lanes of one that
// does not go through the same steps.
template <int DT, int G, int V>
__device__ __forceinline__ void route_row(const MoeRouteArgs &a, int64_t row, bool in, int lane, int &id, float &weight)
{
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * G + lane;
        float x = -INFINITY;
        if (in && e < a.experts) {
            if constexpr (DT == DT_F32)
                x = static_cast<const float *>(a.logits)[row * a.ldl + e];
            else
                x = __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.logits)[row * a.ldl + e] << 16);
        }
        key[v] = logit_key(x);
        if constexpr (DT == DT_BF16)
            key[v] = key[v] ? (key[v] & 0xffff0000u) | (0xffffu - e) : 0u;
    }
    auto value = [](uint32_t k) {
        // the lower half of a negative bf16's key is all ones
        return logit_of(DT == DT_BF16 ? (k & 0x80000000u ? k & 0xffff0000u : k | 0xffffu) : k);
    };
    float top = 0.f, all = 0.f, mine = 0.f;
    id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            m = max(m, key[v]);
        m = lanes_reduce<G>(m, [](uint32_t p, uint32_t q) { return max(p, q); });
        if (j == 0) {
            top = m ? value(m) : 0.f;
            if (a.score == LORA_MOE_SOFTMAX && !a.renorm) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    all += key[v] == 0u ? 0.f : value(key[v]) == top ? 1.f : expf(value(key[v]) - top);
                all = lanes_sum<G>(all);
            }
        }
        int e;
        if constexpr (DT == DT_BF16) {
            e = 0xffff - (int)(m & 0xffffu);
#pragma unroll
            for (int v = 0; v < V; ++v)
                key[v] = key[v] == m ? 0u : key[v];
        } else {
            uint32_t least = 0xffffffffu;
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                least = key[v] == m ? (uint32_t)(v * G + lane) : least;
            e = (int)lanes_reduce<G>(least, [](uint32_t p, uint32_t q) { return min(p, q); });
#pragma unroll
            for (int v = 0; v < V; ++v)
                key[v] = v * G + lane == e ? 0u : key[v];
        }
        if (lane == j && m) {
            id = e;
            mine = value(m);
        }
    }
    float p = 0.f;
    if (id >= 0) {
        if (a.score == LORA_MOE_SOFTMAX) {
            p = mine == top ? 1.f : expf(mine - top);   // infinite logits are equal, not NaN apart
        } else {
            // normalised, all over e^min(top, 0): far negative logits keep their ratio
            const float rel = a.renorm ? fminf(top, 0.f) : 0.f, low = fminf(mine, 0.f);
            p = (low == rel ? 1.f : expf(low - rel)) / (1.f + expf(-fabsf(mine)));
        }
    }
    const float sum = a.renorm ? lanes_sum<G>(p) : a.score == LORA_MOE_SOFTMAX ? all : 1.f;
    weight = id >= 0 ? p / sum * a.scale : 0.f;
}

// Inclusive sum over a wavefront.
__device__ __forceinline__ int wave_scan(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);   // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);   // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);   // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast:15 -> rows 1, 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast:31 -> rows 2, 3
    return x;
}

struct PlaceLds {
    int count[kMaxBuckets];                    // pairs of a bucket, in the whole batch
    int next[kMaxBuckets];                     // where this workgroup's next pair of a bucket goes
    int step[kMaxBuckets];                     // of which the current step takes so many
    int tile0[kMoeHeights][LORA_MAX_EXPERTS + 1];
    int waves[kMoeHeights + 1][kPlaceWaves];
    uint16_t wave_count[kPlaceWaves * kMaxBuckets];   // [wavefront][experts + 1]
};

// From l.count: the groups' offsets (added to l.next) and first tiles, and this
// workgroup's share of what everybody reads of them.
__device__ __forceinline__ void place_scan(const MoeRouteArgs &a, PlaceLds &l)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), E = a.experts;
    const int count = tid < E ? l.count[tid] : 0;
    int in[kMoeHeights + 1], own[kMoeHeights + 1];
#pragma unroll
    for (int i = 0; i <= kMoeHeights; ++i) {
        own[i] = i == 0 ? count : (count + (1 << moe_height_shift(i - 1)) - 1) >> moe_height_shift(i - 1);
        in[i] = wave_scan(own[i]);
        if (lane == 63)
            l.waves[i][wave] = in[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i <= kMoeHeights; ++i) {
        const int ahead = wave_scan(lane < kPlaceWaves ? l.waves[i][lane & (kPlaceWaves - 1)] : 0);
        in[i] += wave > 0 ? __builtin_amdgcn_readlane(ahead, wave - 1) : 0;
    }
    int *offsets = l.step;   // not in use yet
    if (tid < E) {
        offsets[tid] = in[0] - count;
        l.next[tid] += in[0] - count;
#pragma unroll
        for (int i = 0; i < kMoeHeights; ++i)
            l.tile0[i][tid] = in[i + 1] - own[i + 1];
        if (tid == E - 1) {
            offsets[E] = in[0];
            l.next[E] += in[0];
#pragma unroll
            for (int i = 0; i < kMoeHeights; ++i)
                l.tile0[i][E] = in[i + 1];
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int e = tid; e <= E; e += kPlaceThreads) {
            a.l.offsets[e] = offsets[e];
            if (a.offsets)
                a.offsets[e] = offsets[e];
        }
        if (tid < kMoeHeights)
            a.l.n_tiles[tid] = l.tile0[tid][E];
    }
    // the tiles of all heights, one height after the other
    int ends[kMoeHeights];
#pragma unroll
    for (int i = 0; i < kMoeHeights; ++i)
        ends[i] = (i > 0 ? ends[i - 1] : 0) + l.tile0[i][E];
    for (int t = (int)blockIdx.x * kPlaceThreads + tid; t < ends[kMoeHeights - 1]; t += (int)gridDim.x * kPlaceThreads) {
        int h = 0, at = t;
        MoeTile *tiles = a.l.tiles[0];
#pragma unroll
        for (int i = 1; i < kMoeHeights; ++i) {
            if (t >= ends[i - 1]) {
                h = i;
                at = t - ends[i - 1];
                tiles = a.l.tiles[i];
            }
        }
        const int *tile0 = l.tile0[h], shift = moe_height_shift(h);
        int lo = 0, hi = E;   // the last expert whose first tile is at most `at`: it has tiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile0[mid] <= at)
                lo = mid;
            else
                hi = mid;
        }
        const int first = offsets[lo] + ((at - tile0[lo]) << shift);
        tiles[at] = MoeTile{lo, first, min(first + (1 << shift), offsets[lo] + l.count[lo]), 0};
    }
    __syncthreads();   // the offsets' place is the steps' again
}

// Pairs [begin, end) to their positions; id(pair): its expert, or anything
// outside [0, experts).
template <class F>
__device__ __forceinline__ void place_pairs(const MoeRouteArgs &a, PlaceLds &l, int64_t begin, int64_t end, F id)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.experts;
    const int bits = 32 - __clz(E), B = E + 1;
    for (int64_t p0 = begin; p0 < end; p0 += kPlaceThreads) {
        const int64_t p = p0 + tid;
        const bool in = p < end;
        int key = in ? id(p) : E;
        key = (uint32_t)key < (uint32_t)E ? key : E;
        if (p0 > begin) {   // the first step finds them zero
            for (int i = tid; i < kPlaceWaves * B; i += kPlaceThreads)
                l.wave_count[i] = 0;
            __syncthreads();
        }
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((key >> b) & 1);
            same &= (key >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (in && rank == 0)
            l.wave_count[wave * B + key] = (uint16_t)__popcll(same);
        __syncthreads();
        for (int b = tid; b < B; b += kPlaceThreads) {
            int sum = 0, c[kPlaceWaves];
#pragma unroll
            for (int w = 0; w < kPlaceWaves; ++w)
                c[w] = l.wave_count[w * B + b];
#pragma unroll
            for (int w = 0; w < kPlaceWaves; ++w) {
                l.wave_count[w * B + b] = (uint16_t)sum;
                sum += c[w];
            }
            l.step[b] = sum;
        }
        __syncthreads();
        if (in) {
            const int at = l.next[key] + l.wave_count[wave * B + key] + rank;
            a.l.order[at] = (int)p;
            a.l.row[at] = (int)mx_div_of((uint32_t)p, a.by_top_k);
            a.l.place[p] = key < E ? at : -1;
            if (a.order)
                a.order[at] = (int)p;
        }
        if (p0 + kPlaceThreads < end) {
            __syncthreads();
            for (int b = tid; b < B; b += kPlaceThreads)
                l.next[b] += l.step[b];
        }
    }
}

// Counts to zero, ahead of the first use of any.
__device__ __forceinline__ void place_clear(PlaceLds &l, int B)
{
    for (int i = threadIdx.x; i < B; i += kPlaceThreads)
        l.count[i] = l.next[i] = 0;
    for (int i = threadIdx.x; i < kPlaceWaves * B; i += kPlaceThreads)
        l.wave_count[i] = 0;
    __syncthreads();
}

// One workgroup: a whole batch.
template <int DT, int G, int V>
__global__ __launch_bounds__(kPlaceThreads) void moe_small_kernel(MoeRouteArgs a)
{
    __shared__ PlaceLds l;
    __shared__ int ids[kMoeSmallPairs];
    const int tid = threadIdx.x, E = a.experts, pairs = (int)a.n_rows * a.top_k;
    place_clear(l, E + 1);
    if (a.logits) {
        const int lane = tid % G;
        for (int r0 = 0; r0 < a.n_rows; r0 += kPlaceThreads / G) {
            const int row = r0 + tid / G;
            const bool in = row < a.n_rows;
            int id;
            float weight;
            route_row<DT, G, V>(a, row, in, lane, id, weight);
            if (in && lane < a.top_k) {
                const int p = row * a.top_k + lane;
                a.ids[p] = id;
                a.weights[p] = weight;
                ids[p] = id;
                atomicAdd(&l.count[id < 0 ? E : id], 1);
            }
        }
    } else {
        for (int p = tid; p < pairs; p += kPlaceThreads) {
            const int id = a.ids_in[p];
            ids[p] = id;
            atomicAdd(&l.count[(uint32_t)id < (uint32_t)E ? id : E], 1);
        }
    }
    __syncthreads();
    place_scan(a, l);
    place_pairs(a, l, 0, pairs, [&](int64_t p) { return ids[p]; });
}

// One chunk of rows: its choices, and its histogram.
template <int DT, int G, int V>
__global__ __launch_bounds__(kCountThreads) void moe_count_kernel(MoeRouteArgs a)
{
    __shared__ int hist[kMaxBuckets];
    const int tid = threadIdx.x, E = a.experts;
    const int64_t begin = blockIdx.x * a.chunk_rows, end = min(begin + a.chunk_rows, a.n_rows);
    for (int e = tid; e <= E; e += kCountThreads)
        hist[e] = 0;
    __syncthreads();
    if (a.logits) {
        const int lane = tid % G;
        for (int64_t r0 = begin; r0 < end; r0 += kCountThreads / G) {
            const int64_t row = r0 + tid / G;
            const bool in = row < end;
            int id;
            float weight;
            route_row<DT, G, V>(a, row, in, lane, id, weight);
            if (in && lane < a.top_k) {
                a.ids[row * a.top_k + lane] = id;
                a.weights[row * a.top_k + lane] = weight;
                atomicAdd(&hist[id < 0 ? E : id], 1);
            }
        }
    } else {
        for (int64_t p = begin * a.top_k + tid; p < end * a.top_k; p += kCountThreads) {
            const int id = a.ids_in[p];
            atomicAdd(&hist[(uint32_t)id < (uint32_t)E ? id : E], 1);
        }
    }
    __syncthreads();
    for (int e = tid; e <= E; e += kCountThreads)
        a.hist[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

// One chunk of rows: its pairs' positions.
__global__ __launch_bounds__(kPlaceThreads) void moe_place_kernel(MoeRouteArgs a)
{
    __shared__ PlaceLds l;
    const int tid = threadIdx.x, B = a.experts + 1;
    place_clear(l, B);
    // a bucket a thread, as often as the workgroup has room; each takes every
    // `per`-th chunk, kAtOnce loads in flight
    constexpr int kAtOnce = 16;
    const int per = max(1, kPlaceThreads / B);
    for (int b0 = 0; b0 < B; b0 += kPlaceThreads) {
        const int b = per > 1 ? tid % B : b0 + tid, first = per > 1 ? tid / B : 0;
        if (b < B && first < per) {
            int all = 0, ahead = 0;
            for (int c0 = first; c0 < a.n_chunks; c0 += per * kAtOnce) {
                int n[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
                    n[j] = a.hist[(int64_t)min(c0 + j * per, a.n_chunks - 1) * B + b];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const int c = c0 + j * per;
                    all += c < a.n_chunks ? n[j] : 0;
                    ahead += c < (int)blockIdx.x ? n[j] : 0;
                }
            }
            atomicAdd(&l.count[b], all);
            atomicAdd(&l.next[b], ahead);
        }
    }
    __syncthreads();
    place_scan(a, l);
    const int32_t *ids = a.logits ? a.ids : a.ids_in;
    const int64_t begin = blockIdx.x * a.chunk_rows, end = min(begin + a.chunk_rows, a.n_rows);
    place_pairs(a, l, begin * a.top_k, end * a.top_k, [&](int64_t p) { return ids[p]; });
}

// out[i] = residual[i] + sum_j weight[i][j] y[place(i, j)], summed in the
// choices' order in fp32, rounded once.  A wavefront takes 64 units of 8 columns
// of one row, so places and weights are the same in all of its lanes; all
// choices' loads are issued before the first is used, eight at a time.  Bound by
// the read of y.
constexpr int kCombineThreads = 256;
template <int DT, int YDT>
__global__ __launch_bounds__(kCombineThreads) void moe_combine_kernel(MoeCombineArgs a, int waves_a_row, MxDiv by_waves)
{
    const uint32_t w = blockIdx.x * (kCombineThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = mx_div_of(w, by_waves);
    const int64_t row = a.row0 + r;
    const int64_t c = ((int64_t)(w - r * waves_a_row) * 64 + (threadIdx.x & 63)) * 8;
    if (r >= a.rows || c >= a.d)
        return;
    float sum[8];
    Vec8<DT> v;
    v.zero();
    if (a.res)
        v.load(a.res, row * a.ldr + c);
    v.to_f32(sum);
    constexpr int kAtOnce = 8;
    for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
        Vec8<YDT> y[kAtOnce];
        float weight[kAtOnce];
        int at[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t p = row * a.top_k + min(j0 + j, a.top_k - 1);
            at[j] = j0 + j < a.top_k ? a.place[p] : -1;
            weight[j] = a.weights[p];
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (at[j] >= 0)
                y[j].load(a.y, at[j] * a.ldy + c);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (at[j] >= 0) {
                float f[8];
                y[j].to_f32(f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] = fmaf(weight[j], f[e], sum[e]);
            }
        }
    }
    Vec8<DT>::store(a.out, row * a.ldo + c, sum);
}

template <int DT, int G, int V> void route_go(const MoeRouteArgs &a, hipStream_t s)
{
    if (a.n_rows * a.top_k <= kMoeSmallPairs) {
        moe_small_kernel<DT, G, V><<<1, kPlaceThreads, 0, s>>>(a);
        return;
    }
    moe_count_kernel<DT, G, V><<<a.n_chunks, kCountThreads, 0, s>>>(a);
    moe_place_kernel<<<a.n_chunks, kPlaceThreads, 0, s>>>(a);
}

template <int DT> void route_pick(const MoeRouteArgs &a, hipStream_t s)
{
    if (!a.logits || a.experts <= 64)
        route_go<DT, 16, 4>(a, s);
    else if (a.experts <= 128)
        route_go<DT, 16, 8>(a, s);
    else if (a.experts <= 256)
        route_go<DT, 16, 16>(a, s);
    else
        route_go<DT, 64, 16>(a, s);
}

}  // namespace

hipError_t launch_moe_route(int dtype, const MoeRouteArgs &a, hipStream_t s)
{
    if (dtype == DT_F32)
        route_pick<DT_F32>(a, s);
    else
        route_pick<DT_BF16>(a, s);
    return hipGetLastError();
}

hipError_t launch_moe_combine(int dtype, const MoeCombineArgs &a, hipStream_t s)
{
    const int64_t waves = (a.d + 511) / 512;
    const MxDiv by = mx_div((uint32_t)waves);
    // a launch's wavefronts fit 25 bits (2^32 threads and 31 bits of mx_div both hold)
    for_slabs(a.n_rows, ((int64_t)1 << 25) / waves, [&](int64_t row0, int64_t rows) {
        MoeCombineArgs b = a;
        b.row0 = row0;
        b.rows = rows;
        const uint32_t grid = (uint32_t)((rows * waves + kCombineThreads / 64 - 1) / (kCombineThreads / 64));
        if (dtype == DT_F32 && a.y_dtype == DT_F32)
            moe_combine_kernel<DT_F32, DT_F32><<<grid, kCombineThreads, 0, s>>>(b, (int)waves, by);
        else if (dtype == DT_F32)
            moe_combine_kernel<DT_F32, DT_BF16><<<grid, kCombineThreads, 0, s>>>(b, (int)waves, by);
        else if (a.y_dtype == DT_F32)
            moe_combine_kernel<DT_BF16, DT_F32><<<grid, kCombineThreads, 0, s>>>(b, (int)waves, by);
        else
            moe_combine_kernel<DT_BF16, DT_BF16><<<grid, kCombineThreads, 0, s>>>(b, (int)waves, by);
    });
    return hipGetLastError();
}

}  // namespace lora
