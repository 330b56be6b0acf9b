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
// and one launch (64 rows of 64 experts, top 8: 7.2 us, a chain of dependent
// steps); others three: rows in chunks, each with its histogram; the
// histograms' sums over the chunks ahead; the chunks' pairs to their places.
// 35422 rows of 128 experts, top 8, bf16: 9.8 + 3.7 + 9.2 us, the first bound by its
// instructions (19 us with the maximum over unsorted keys), the last by scattered
// writes of 4 bytes (the order, twice where the caller wants it too; the pairs' places
// are written in their own order).  Given ids, a call among others: 64 rows top 8 of
// 64 4.4 us (with order and offsets 4.9), 256 rows 5.6, 35422 of 128 13.2 (15.6).
#include "mx_device.h"
#include "moe.h"

namespace lora {

namespace {

constexpr int kMaxBuckets = LORA_MAX_EXPERTS + 1;   // the last: pairs without an expert
constexpr int kSmallThreads = 1024, kSmallSteps = kMoeSmallPairs / kSmallThreads;
constexpr int kCountThreads = 1024;                      // at most
constexpr int kScanBuckets = 16, kScanThreads = 256;     // of one workgroup of the sums over chunks
constexpr int kScanChunks = kMoeMaxChunks / (kScanThreads / kScanBuckets);   // of one thread
constexpr int kPlaceThreads = 256, kPlaceSteps = 8;

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
__device__ __forceinline__ uint32_t logit_key(uint32_t bits)
{
    constexpr int kOff = 0x007;   // the classes NaN (two) and -inf
    const float x = __uint_as_float(bits);
    const uint32_t b = __float_as_uint(x + 0.f), k = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
    return __builtin_amdgcn_classf(x, kOff) ? 0u : k;
}
// The same of a bf16 logit, with the expert's number in the lower half, so that
// no two keys of a row are equal and the lower of two numbers orders higher.
__device__ __forceinline__ uint32_t logit_key(uint32_t bits, int e)
{
    constexpr int kOff = 0x007;
    const float x = __uint_as_float(bits);
    const uint32_t b = __float_as_uint(x + 0.f), k = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
    return __builtin_amdgcn_classf(x, kOff) ? 0u : (k & 0xffff0000u) | (0xffffu - e);
}
template <int DT> __device__ __forceinline__ float logit_of(uint32_t key)
{
    if (DT == DT_BF16)   // the lower half of a negative bf16's key is all ones
        key = key & 0x80000000u ? key & 0xffff0000u : key | 0xffffu;
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Largest first, by Batcher's merges of odd and even places (V a power of two).
template <int V> __device__ __forceinline__ void sort_down(uint32_t (&key)[V])
{
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = key[i + j], y = key[i + j + k];
                        key[i + j] = max(x, y);
                        key[i + j + k] = min(x, y);
                    }
}

// Choices of one row; lane j of the row's G lanes gets choice j (id -1, weight
// 0 where fewer experts are left).  A row past the last is the last once more.
// FULL: there are G * V experts.
template <int DT, int G, int V, bool FULL>
__device__ __forceinline__ void route_row(const MoeRouteArgs &a, int row, int lane, int &id, float &weight)
{
    // all loads without a branch, from addresses inside the row
    constexpr int kSize = DT == DT_F32 ? 4 : 2;
    const char *at = static_cast<const char *>(a.logits) + min((int64_t)row, a.n_rows - 1) * a.ldl * kSize;
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = FULL ? v * G + lane : min(v * G + lane, a.experts - 1);
        if constexpr (DT == DT_F32)
            key[v] = *reinterpret_cast<const uint32_t *>(at + (uint32_t)(e * kSize));
        else
            key[v] = *reinterpret_cast<const uint16_t *>(at + (uint32_t)(e * kSize));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * G + lane;
        key[v] = DT == DT_F32 ? logit_key(key[v]) : logit_key(key[v] << 16, e);
        if (!FULL)
            key[v] &= e < a.experts ? 0xffffffffu : 0u;
    }
    if constexpr (DT == DT_BF16)
        sort_down(key);   // each lane's largest is then its first
    float top = 0.f, all = 0.f;
    uint32_t mine = 0;
    int which = 0;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t m = key[0];
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int v = 1; v < V; ++v)
                m = max(m, key[v]);
        }
        m = lanes_reduce<G>(m, [](uint32_t p, uint32_t q) { return max(p, q); });
        if (j == 0) {
            top = m ? logit_of<DT>(m) : 0.f;
            if (a.score == LORA_MOE_SOFTMAX && !a.renorm) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float x = logit_of<DT>(key[v]);
                    all += key[v] == 0u ? 0.f : x == top ? 1.f : expf(x - top);
                }
                all = lanes_sum<G>(all);
            }
        }
        if constexpr (DT == DT_BF16) {
            // one lane's, as keys are different, or zeros are left everywhere; by bits,
            // as a choice of two elements would be compiled as one of their index
            const uint32_t take = key[0] == m ? 0xffffffffu : 0u;
#pragma unroll
            for (int v = 0; v + 1 < V; ++v)
                key[v] = (key[v + 1] & take) | (key[v] & ~take);
            key[V - 1] &= ~take;
        } else {
            uint32_t least = 0xffffffffu;
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                least = key[v] == m ? (uint32_t)(v * G + lane) : least;
            const int e = (int)lanes_reduce<G>(least, [](uint32_t p, uint32_t q) { return min(p, q); });
#pragma unroll
            for (int v = 0; v < V; ++v)
                key[v] = v * G + lane == e ? 0u : key[v];
            which = lane == j ? e : which;
        }
        mine = lane == j ? m : mine;
    }
    const bool some = mine != 0;
    id = !some ? -1 : DT == DT_F32 ? which : 0xffff - (int)(mine & 0xffffu);
    const float x = logit_of<DT>(mine);
    float p;
    if (a.score == LORA_MOE_SOFTMAX) {
        p = x == top ? 1.f : expf(x - top);   // infinite logits are equal, not NaN apart
    } else {
        // normalised, all over e^min(top, 0): far negative logits keep their ratio
        const float rel = a.renorm ? fminf(top, 0.f) : 0.f, low = fminf(x, 0.f);
        p = (low == rel ? 1.f : expf(low - rel)) / (1.f + expf(-fabsf(x)));
    }
    p = some ? p : 0.f;
    const float sum = a.renorm ? lanes_sum<G>(p) : a.score == LORA_MOE_SOFTMAX ? all : 1.f;
    weight = some ? p / sum * a.scale : 0.f;
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

template <int T> struct PlaceLds {
    int count[kMaxBuckets];                    // pairs of a bucket, in the whole batch
    int next[kMaxBuckets];                     // where this workgroup's next pair of a bucket goes
    int step[kMaxBuckets];                     // of which the current step takes so many
    int offsets[kMaxBuckets];
    int tile0[kMoeHeights][kMaxBuckets];
    int waves[kMoeHeights + 1][T / 64];
    uint16_t wave_count[T / 64 * kMaxBuckets]; // [wavefront][experts + 1]
};

// From l.count: the groups' offsets (added to l.next) and first tiles, and this
// workgroup's share of what the plan keeps of them.
template <int T> __device__ __forceinline__ void place_scan(const MoeRouteArgs &a, PlaceLds<T> &l)
{
    constexpr int kPer = (LORA_MAX_EXPERTS + T - 1) / T;   // experts of a thread, at most
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), E = a.experts;
    const int per = (E + T - 1) / T;
    int own[kPer][kMoeHeights + 1], in[kMoeHeights + 1];
#pragma unroll
    for (int i = 0; i <= kMoeHeights; ++i)
        in[i] = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = tid * per + j;
        const int n = j < per && e < E ? l.count[e] : 0;
#pragma unroll
        for (int i = 0; i <= kMoeHeights; ++i) {
            own[j][i] = i == 0 ? n : (n + (1 << moe_height_shift(i - 1)) - 1) >> moe_height_shift(i - 1);
            in[i] += own[j][i];
        }
    }
    int mine[kMoeHeights + 1];
#pragma unroll
    for (int i = 0; i <= kMoeHeights; ++i) {
        mine[i] = in[i];
        in[i] = wave_scan(in[i]);
        if (lane == 63)
            l.waves[i][wave] = in[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i <= kMoeHeights; ++i) {
        const int ahead = wave_scan(lane < T / 64 ? l.waves[i][lane % (T / 64)] : 0);
        in[i] += (wave > 0 ? __builtin_amdgcn_readlane(ahead, wave - 1) : 0) - mine[i];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = tid * per + j;
        if (j < per && e < E) {
            l.offsets[e] = in[0];
            l.next[e] += in[0];
#pragma unroll
            for (int i = 0; i < kMoeHeights; ++i)
                l.tile0[i][e] = in[i + 1];
#pragma unroll
            for (int i = 0; i <= kMoeHeights; ++i)
                in[i] += own[j][i];
            if (e == E - 1) {
                l.offsets[E] = in[0];
                l.next[E] += in[0];
#pragma unroll
                for (int i = 0; i < kMoeHeights; ++i)
                    l.tile0[i][E] = in[i + 1];
            }
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (a.offsets)
            for (int e = tid; e <= E; e += T)
                a.offsets[e] = l.offsets[e];
        if (tid < kMoeHeights)
            a.l.n_tiles[tid] = l.tile0[tid][E];
    }
    // the tiles of all heights, one height after the other
    int ends[kMoeHeights];
#pragma unroll
    for (int i = 0; i < kMoeHeights; ++i)
        ends[i] = (i > 0 ? ends[i - 1] : 0) + l.tile0[i][E];
    for (int t = (int)blockIdx.x * T + tid; t < ends[kMoeHeights - 1]; t += (int)gridDim.x * T) {
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
        const int first = l.offsets[lo] + ((at - tile0[lo]) << shift);
        tiles[at] = MoeTile{lo, first, min(first + (1 << shift), l.offsets[lo] + l.count[lo]), 0};
    }
}

// Pairs [begin, end) to their positions, up to T * STEPS at a time; a wavefront
// takes neighbouring ones.  first: the ids of this thread's pairs of the first
// time; id(pair): an id of a later one.  Anything outside [0, experts) is no
// expert.  l.wave_count comes in zero.
template <int T, int STEPS> __device__ __forceinline__ int place_steps(int begin, int end)
{
    return min(STEPS, (end - begin + T - 1) / T);
}
template <int T, int STEPS, class F>
__device__ __forceinline__ void place_pairs(const MoeRouteArgs &a, PlaceLds<T> &l, int begin, int end, const int (&first)[STEPS], F id)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.experts;
    const int bits = 32 - __clz(E), B = E + 1;
    uint16_t *counts = l.wave_count + wave * B;
    for (int p0 = begin; p0 < end; p0 += T * STEPS) {
        const int steps = place_steps<T, STEPS>(p0, end);
        const int mine = p0 + wave * 64 * steps + lane;
        int key[STEPS], rank[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int p = mine + 64 * i;
            key[i] = p0 == begin ? first[i] : i < steps && p < end ? id(p) : E;
            key[i] = (uint32_t)key[i] < (uint32_t)E ? key[i] : E;
        }
        if (p0 > begin) {
            for (int i = tid; i < T / 64 * B; i += T)
                l.wave_count[i] = 0;
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (i < steps) {
                const bool in = mine + 64 * i < end;
                uint64_t same = __ballot(in);
                for (int b = 0; b < bits; ++b) {
                    const uint64_t set = __ballot((key[i] >> b) & 1);
                    same &= (key[i] >> b) & 1 ? set : ~set;
                }
                const int before = counts[key[i]], ahead = __popcll(same & ((1ull << lane) - 1));
                rank[i] = before + ahead;
                if (in && ahead == 0)
                    counts[key[i]] = (uint16_t)(before + __popcll(same));
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
            }
        }
        __syncthreads();
        for (int b = tid; b < B; b += T) {
            int sum = 0, c[T / 64];
#pragma unroll
            for (int w = 0; w < T / 64; ++w)
                c[w] = l.wave_count[w * B + b];
#pragma unroll
            for (int w = 0; w < T / 64; ++w) {
                l.wave_count[w * B + b] = (uint16_t)sum;
                sum += c[w];
            }
            l.step[b] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int p = mine + 64 * i;
            if (i < steps && p < end) {
                const int at = l.next[key[i]] + counts[key[i]] + rank[i];
                a.l.order[at] = p;
                a.l.place[p] = key[i] < E ? at : -1;
                if (a.order)
                    a.order[at] = p;
            }
        }
        if (p0 + T * STEPS < end) {
            __syncthreads();
            for (int b = tid; b < B; b += T)
                l.next[b] += l.step[b];
        }
    }
}

// One workgroup: a whole batch.
template <int DT, int G, int V, bool FULL>
__global__ __launch_bounds__(kSmallThreads) void moe_small_kernel(MoeRouteArgs a)
{
    constexpr int T = kSmallThreads;
    __shared__ PlaceLds<T> l;
    __shared__ int ids[kMoeSmallPairs];
    const int tid = threadIdx.x, E = a.experts, B = E + 1, pairs = (int)a.n_rows * a.top_k;
    for (int i = tid; i < B; i += T)
        l.count[i] = l.next[i] = 0;
    for (int i = tid; i < T / 64 * B; i += T)
        l.wave_count[i] = 0;
    __syncthreads();
    if (a.logits) {
        const int lane = tid % G;
        for (int r0 = 0; r0 < a.n_rows; r0 += T / G) {
            const int row = r0 + tid / G;
            const bool in = row < a.n_rows;
            int id;
            float weight;
            route_row<DT, G, V, FULL>(a, row, lane, id, weight);
            if (in && lane < a.top_k) {
                const int p = row * a.top_k + lane;
                a.ids[p] = id;
                a.weights[p] = weight;
                ids[p] = id;
                atomicAdd(&l.count[id < 0 ? E : id], 1);
            }
        }
    } else {
        for (int p = tid; p < pairs; p += T) {
            const int id = a.ids_in[p];
            ids[p] = id;
            atomicAdd(&l.count[(uint32_t)id < (uint32_t)E ? id : E], 1);
        }
    }
    __syncthreads();
    place_scan<T>(a, l);
    int first[kSmallSteps];
    const int steps = place_steps<T, kSmallSteps>(0, pairs);
#pragma unroll
    for (int i = 0; i < kSmallSteps; ++i) {
        const int p = (tid >> 6) * 64 * steps + (tid & 63) + 64 * i;
        first[i] = i < steps && p < pairs ? ids[p] : E;
    }
    place_pairs<T, kSmallSteps>(a, l, 0, pairs, first, [&](int p) { return ids[p]; });
}

// One chunk of rows: its choices, and its histogram.
template <int DT, int G, int V, bool FULL>
__global__ __launch_bounds__(kCountThreads) void moe_count_kernel(MoeRouteArgs a)
{
    __shared__ int hist[kMaxBuckets];
    const int tid = threadIdx.x, T = blockDim.x, E = a.experts;
    const int begin = (int)(blockIdx.x * a.chunk_rows), end = (int)min(begin + a.chunk_rows, a.n_rows);
    for (int e = tid; e <= E; e += T)
        hist[e] = 0;
    __syncthreads();
    if (a.logits) {
        const int lane = tid % G;
        for (int r0 = begin; r0 < end; r0 += T / G) {
            const int row = r0 + tid / G;
            const bool in = row < end;
            int id;
            float weight;
            route_row<DT, G, V, FULL>(a, row, lane, id, weight);
            if (in && lane < a.top_k) {
                a.ids[row * a.top_k + lane] = id;
                a.weights[row * a.top_k + lane] = weight;
                atomicAdd(&hist[id < 0 ? E : id], 1);
            }
        }
    } else {
        for (int p = begin * a.top_k + tid; p < end * a.top_k; p += T) {
            const int id = a.ids_in[p];
            atomicAdd(&hist[(uint32_t)id < (uint32_t)E ? id : E], 1);
        }
    }
    __syncthreads();
    for (int e = tid; e <= E; e += T)
        a.hist[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

// Histograms to their sums over the chunks ahead, and the batch's totals behind
// the last chunk.  16 buckets a workgroup; 16 threads a bucket, neighbouring
// chunks each, all of them loaded before the first is used.
__global__ __launch_bounds__(kScanThreads) void moe_scan_kernel(MoeRouteArgs a)
{
    constexpr int kParts = kScanThreads / kScanBuckets;
    __shared__ int part[kParts][kScanBuckets];
    const int B = a.experts + 1, in = threadIdx.x % kScanBuckets, g = threadIdx.x / kScanBuckets;
    const int b = min((int)blockIdx.x * kScanBuckets + in, B - 1);   // past the last: its work again
    const int per = (a.n_chunks + kParts - 1) / kParts;
    int n[kScanChunks], sum = 0;
#pragma unroll
    for (int j = 0; j < kScanChunks; ++j)
        n[j] = a.hist[(int64_t)min(g * per + j, a.n_chunks - 1) * B + b];
#pragma unroll
    for (int j = 0; j < kScanChunks; ++j) {
        n[j] = j < per && g * per + j < a.n_chunks ? n[j] : 0;
        sum += n[j];
    }
    part[g][in] = sum;
    __syncthreads();
    int ahead = 0;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        ahead += i < g ? part[i][in] : 0;
    if ((int)blockIdx.x * kScanBuckets + in >= B)
        return;
#pragma unroll
    for (int j = 0; j < kScanChunks; ++j) {
        const int c = g * per + j;
        if (j < per && c < a.n_chunks)
            a.hist[(int64_t)c * B + b] = ahead;
        ahead += n[j];
    }
    if (g == kParts - 1)
        a.hist[(int64_t)a.n_chunks * B + b] = ahead;
}

// One chunk of rows: its pairs' positions.
__global__ __launch_bounds__(kPlaceThreads) void moe_place_kernel(MoeRouteArgs a)
{
    constexpr int T = kPlaceThreads;
    __shared__ PlaceLds<T> l;
    const int tid = threadIdx.x, B = a.experts + 1;
    const int32_t *ids = a.logits ? a.ids : a.ids_in;
    const int begin = (int)(blockIdx.x * a.chunk_rows) * a.top_k;
    const int end = (int)min((int64_t)begin + a.chunk_rows * a.top_k, a.n_rows * a.top_k);
    const int steps = place_steps<T, kPlaceSteps>(begin, end);
    int first[kPlaceSteps];   // on their way during the scan
#pragma unroll
    for (int i = 0; i < kPlaceSteps; ++i)
        first[i] = ids[min(begin + (tid >> 6) * 64 * steps + (tid & 63) + 64 * i, end - 1)];
    for (int b = tid; b < B; b += T) {
        l.next[b] = a.hist[(int64_t)blockIdx.x * B + b];
        l.count[b] = a.hist[(int64_t)a.n_chunks * B + b];
    }
    for (int i = tid; i < T / 64 * B; i += T)
        l.wave_count[i] = 0;
    __syncthreads();
    place_scan<T>(a, l);
    place_pairs<T, kPlaceSteps>(a, l, begin, end, first, [&](int p) { return ids[p]; });
}

// out[i] = residual[i] + sum_j weight[i][j] y[place(i, j)], summed in the
// choices' order in fp32, rounded once.  A wavefront takes 64 units of 8 columns
// of one row, so places and weights are the same in all of its lanes; all
// choices' loads are issued before the first is used, eight at a time.  Bound by
// the read of y: 8192 rows of 8 x 4096 fp32, 1.34 GB in 247 - 281 us (4.8 - 5.4 TB/s).
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
    const int64_t pairs = a.n_rows * a.top_k;
    for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
        Vec8<YDT> y[kAtOnce];
        float weight[kAtOnce];
        int at[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t p = row * a.top_k + min(j0 + j, a.top_k - 1);
            at[j] = j0 + j < a.top_k ? a.place[p] : -1;
            at[j] = at[j] < pairs ? at[j] : -1;   // y has no more rows, whatever grouping the plan holds by now
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

template <int DT, int G, int V, bool FULL> void route_go(const MoeRouteArgs &a, hipStream_t s)
{
    if (a.n_rows * a.top_k <= kMoeSmallPairs) {
        moe_small_kernel<DT, G, V, FULL><<<1, kSmallThreads, 0, s>>>(a);
        return;
    }
    // a chunk's rows in as few passes as a workgroup can, of equal sizes
    const int64_t at_once = kCountThreads / G, passes = (a.chunk_rows + at_once - 1) / at_once;
    const int64_t threads = ((a.chunk_rows + passes - 1) / passes * G + 63) / 64 * 64;
    moe_count_kernel<DT, G, V, FULL><<<a.n_chunks, (uint32_t)threads, 0, s>>>(a);
    moe_scan_kernel<<<(a.experts + kScanBuckets) / kScanBuckets, kScanThreads, 0, s>>>(a);
    moe_place_kernel<<<a.n_chunks, kPlaceThreads, 0, s>>>(a);
}

// 16 lanes a row up to 256 experts, 64 beyond; without the bounds of a last,
// shorter set of experts where there is none.
template <int DT, int G, int V> void route_full(const MoeRouteArgs &a, hipStream_t s)
{
    if (a.experts == G * V)
        route_go<DT, G, V, true>(a, s);
    else
        route_go<DT, G, V, false>(a, s);
}
template <int DT> void route_pick(const MoeRouteArgs &a, hipStream_t s)
{
    if (!a.logits)
        route_go<DT, 16, 4, false>(a, s);
    else if (a.experts <= 64)
        route_full<DT, 16, 4>(a, s);
    else if (a.experts <= 128)
        route_full<DT, 16, 8>(a, s);
    else if (a.experts <= 256)
        route_full<DT, 16, 16>(a, s);
    else
        route_full<DT, 64, 16>(a, s);
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
