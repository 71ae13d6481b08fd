// Vectors sorted by list and back: a stable sort of (vector, list) pairs by
// list, rows gathered in that order, and rows in that order summed back to
// their vectors with weights; and the gradients of both.
//
// Slot u = t k + j is pair j of vector t.  The sort gives every kept slot a
// position p; order[p] is the slot at p (-1 past the kept ones) and pos[u] the
// position of slot u (-1 for a slot without a list).
#include "common.hpp"
#include "rows.hpp"
#include "rows_internal.hpp"

namespace ivfpq {

// ---------------------------------------------------------------------------
// stable sort by list
// ---------------------------------------------------------------------------

// Eight waves a workgroup against four, 320,000 slots of 1024 lists: count 4.9
// against 6.3 us, scatter 9.1 against 12.2 us.
constexpr int kSortWaves = 8;
constexpr int kSortChunk = 2048; // slots of one workgroup
constexpr int kSortBits = 11;    // bits of one pass
constexpr int kSortBins = 1 << kSortBits;

// Up to this many slots and lists the sort is one workgroup of 16 waves: 512
// slots of 64 lists 3.6 us (5.3 us a call, three launches 10.6).  At 8192 slots a
// call takes 9.3 us of 64 lists and 12.6 of 1024; 16,384 slots in three launches
// 10.6 and 12.8.
constexpr int kSoloSlots = 8192;
constexpr int kSoloBins = 1088;

// The sort key of a slot: its list, or nlist when it has none.
__device__ __forceinline__ uint32_t list_key(const int32_t *lists, uint32_t u, uint32_t nlist)
{
    const uint32_t l = (uint32_t)lists[u];
    return l < nlist ? l : nlist;
}

struct SortPass {
    const int32_t *lists;   // first pass: the lists themselves
    const uint32_t *key_in; // later passes: keys and slots of the pass before
    const uint32_t *slot_in;
    uint32_t n, nlist, shift, bins, blocks;
    uint32_t *hist;  // [blocks][bins], then the exclusive sums along a bin
    uint32_t *total; // [bins]
    uint32_t *key_out, *slot_out; // nullptr in the last pass of a single-pass sort
    int32_t *offsets, *order, *pos; // of the last pass (offsets: single-pass sort only)

    __device__ __forceinline__ uint32_t key(uint32_t i) const
    {
        return key_in ? key_in[i] : list_key(lists, i, nlist);
    }
    __device__ __forceinline__ uint32_t bin(uint32_t k) const
    {
        return (k >> shift) & (kSortBins - 1);
    }
};

// Counts of one workgroup's chunk by bin.
__global__ __launch_bounds__(64 * kSortWaves) void route_count_kernel(SortPass s)
{
    __shared__ uint32_t count[kSortBins];
    for (uint32_t b = threadIdx.x; b < s.bins; b += blockDim.x)
        count[b] = 0;
    __syncthreads();
    const uint32_t first = blockIdx.x * (uint32_t)kSortChunk;
    const uint32_t end = min(first + (uint32_t)kSortChunk, s.n);
    constexpr int ROUNDS = kSortChunk / (64 * kSortWaves);
    uint32_t key[ROUNDS]; // all under way at once
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const uint32_t i = first + r * 64 * kSortWaves + threadIdx.x;
        key[r] = i < end ? s.key(i) : 0;
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
        if (first + r * 64 * kSortWaves + threadIdx.x < end)
            atomicAdd(&count[s.bin(key[r])], 1u);
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < s.bins; b += blockDim.x)
        s.hist[(size_t)blockIdx.x * s.bins + b] = count[b];
}

// Exclusive sums of the bins' counts along the workgroups: 64 bins a workgroup,
// a lane each, its 16 waves sharing the rows of counts out between them (a
// lane's reads are far apart, a wave's side by side).
__global__ __launch_bounds__(1024) void route_scan_kernel(SortPass s)
{
    __shared__ uint32_t part[16][64];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t b = blockIdx.x * 64 + lane;
    const bool live = b < s.bins;
    const uint32_t rows = (s.blocks + 15) / 16;
    const uint32_t first = min(wave * rows, s.blocks), end = min(first + rows, s.blocks);
    uint32_t sum = 0;
#pragma unroll 4
    for (uint32_t i = first; i < end; ++i)
        sum += live ? s.hist[(size_t)i * s.bins + b] : 0;
    part[wave][lane] = sum;
    __syncthreads();
    uint32_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        base += w < wave ? part[w][lane] : 0;
        all += part[w][lane];
    }
    if (!live)
        return;
    if (wave == 0)
        s.total[b] = all;
#pragma unroll 4
    for (uint32_t i = first; i < end; ++i) {
        const uint32_t v = s.hist[(size_t)i * s.bins + b];
        s.hist[(size_t)i * s.bins + b] = base;
        base += v;
    }
}

// Every slot to its place.  Ranks come from ballots, a bit of the bin each, so
// that equal bins keep their order and no atomic decides it.  320,000 slots of
// 1024 lists: 8.5 us here, 4.7 us for the counts and 5.2 us for their sums.
//
// The place: the start of its bin, plus the bin's slots of earlier
// workgroups, of earlier waves of this one (each wave has a contiguous part of
// the chunk) and of earlier lanes.  SOLO: the one workgroup of a small sort,
// which has all counts itself, and so is the whole sort in one launch.
template <int WAVES, int BINS, bool SOLO>
__global__ __launch_bounds__(64 * WAVES) void route_scatter_kernel(SortPass s)
{
    __shared__ uint32_t at[WAVES][BINS];
    __shared__ uint32_t sums[WAVES];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    constexpr int ROUNDS = (SOLO ? kSoloSlots : kSortChunk) / (64 * WAVES);
    const uint32_t part = SOLO ? (s.n + WAVES - 1) / WAVES : kSortChunk / WAVES;
    const uint32_t first = min(blockIdx.x * (uint32_t)kSortChunk + wave * part, s.n);
    const uint32_t end = min(first + part, s.n);
    const int rounds = (int)((end - first + 63) / 64);
    uint32_t key[ROUNDS]; // all of the wave's keys under way at once
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
        key[r] = first + r * 64 + lane < end ? s.key(first + r * 64 + lane) : 0;
    for (uint32_t b = threadIdx.x; b < s.bins; b += 64 * WAVES)
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            at[w][b] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
        if (first + r * 64 + lane < end)
            atomicAdd(&at[wave][s.bin(key[r])], 1u);
    __syncthreads();
    // a thread has `each` bins in a row: exclusive sums of the totals
    const uint32_t each = (s.bins + 64 * WAVES - 1) / (64 * WAVES);
    const uint32_t b0 = min(threadIdx.x * each, s.bins), b1 = min(b0 + each, s.bins);
    uint32_t mine = 0;
    for (uint32_t b = b0; b < b1; ++b) {
        if constexpr (SOLO) {
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                mine += at[w][b];
        } else {
            mine += s.total[b];
        }
    }
    const uint32_t upto = wave_inclusive_sum(mine);
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    uint32_t start = upto - mine;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        start += w < wave ? sums[w] : 0;
    for (uint32_t b = b0; b < b1; ++b) {
        if (s.offsets && blockIdx.x == 0)
            s.offsets[b] = (int32_t)start;
        uint32_t p = start;
        if constexpr (!SOLO) {
            start += s.total[b];
            p += s.hist[(size_t)blockIdx.x * s.bins + b];
        }
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const uint32_t c = at[w][b];
            at[w][b] = p;
            p += c;
        }
        if constexpr (SOLO)
            start = p;
    }
    __syncthreads();
    int bits = 0;
    while ((1u << bits) < s.bins)
        ++bits;
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r < rounds) {
            const uint32_t i = first + r * 64 + lane;
            const bool live = i < end;
            const uint32_t bin = s.bin(key[r]);
            uint64_t same = __ballot(live);
            for (int q = 0; q < bits; ++q) {
                const uint64_t m = __ballot((bin >> q) & 1);
                same &= (bin >> q) & 1 ? m : ~m;
            }
            if (live) {
                const uint32_t before = (uint32_t)__popcll(same & ((1ull << lane) - 1));
                const uint32_t p = at[wave][bin] + before;
                const uint32_t u = s.slot_in ? s.slot_in[i] : i;
                if (s.slot_out)
                    s.slot_out[p] = u;
                if (s.key_out)
                    s.key_out[p] = key[r];
                if (s.order) {
                    s.order[p] = key[r] < s.nlist ? (int32_t)u : -1;
                    s.pos[u] = key[r] < s.nlist ? (int32_t)p : -1;
                }
                if ((same >> lane) == 1) // the bin's last lane moves its cursor on
                    at[wave][bin] = p + 1;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); // the cursors, for the next 64
        }
    }
}

// The same sort of up to kSoloSlots slots of any number of lists: one workgroup, as many
// passes of 8 bits as the lists' numbers have, keys and slots in LDS between them.
// 1000 slots of 5003 lists: 6.7 us and 3.6 for the offsets (seven launches: 27 us).
constexpr int kDigitBins = 256;

__global__ __launch_bounds__(1024) void route_solo_kernel(SortPass s)
{
    constexpr int WAVES = 16, ROUNDS = kSoloSlots / (64 * WAVES);
    __shared__ uint32_t keys[kSoloSlots];
    __shared__ uint16_t slots[kSoloSlots];
    __shared__ uint32_t at[WAVES][kDigitBins];
    __shared__ uint32_t sums[kDigitBins / 64];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t part = (s.n + WAVES - 1) / WAVES;
    const uint32_t first = min(wave * part, s.n), end = min(first + part, s.n);
    const int rounds = (int)((end - first + 63) / 64);
    uint32_t key[ROUNDS], slot[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        slot[r] = first + r * 64 + lane;
        key[r] = slot[r] < end ? list_key(s.lists, slot[r], s.nlist) : 0;
    }
    for (uint32_t shift = 0; s.nlist >> shift; shift += 8) {
        for (uint32_t b = threadIdx.x; b < WAVES * kDigitBins; b += 1024)
            (&at[0][0])[b] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            if (first + r * 64 + lane < end)
                atomicAdd(&at[wave][(key[r] >> shift) & (kDigitBins - 1)], 1u);
        __syncthreads();
        // a thread a digit: exclusive sums over the digits, then over the waves
        uint32_t mine = 0, upto = 0;
        if (threadIdx.x < kDigitBins) {
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                mine += at[w][threadIdx.x];
            upto = wave_inclusive_sum(mine);
            if (lane == 63)
                sums[wave] = upto;
        }
        __syncthreads();
        if (threadIdx.x < kDigitBins) {
            uint32_t p = upto - mine;
            for (int w = 0; w < wave; ++w)
                p += sums[w];
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const uint32_t c = at[w][threadIdx.x];
                at[w][threadIdx.x] = p;
                p += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if (r < rounds) {
                const bool live = first + r * 64 + lane < end;
                const uint32_t bin = (key[r] >> shift) & (kDigitBins - 1);
                uint64_t same = __ballot(live);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint64_t m = __ballot((bin >> q) & 1);
                    same &= (bin >> q) & 1 ? m : ~m;
                }
                if (live) {
                    const uint32_t p =
                        at[wave][bin] + (uint32_t)__popcll(same & ((1ull << lane) - 1));
                    keys[p] = key[r];
                    slots[p] = (uint16_t)slot[r];
                    if ((same >> lane) == 1)
                        at[wave][bin] = p + 1;
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); // the cursors
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const uint32_t i = first + r * 64 + lane;
            key[r] = i < end ? keys[i] : 0;
            slot[r] = i < end ? slots[i] : 0;
        }
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const uint32_t p = first + r * 64 + lane;
        if (p < end) {
            const bool kept = key[r] < s.nlist;
            s.key_out[p] = key[r];
            s.order[p] = kept ? (int32_t)slot[r] : -1;
            s.pos[slot[r]] = kept ? (int32_t)p : -1;
        }
    }
}

// List starts of a sort of more than one pass: offsets[l] = keys below l.
__global__ __launch_bounds__(256) void route_bounds_kernel(const uint32_t *__restrict__ keys,
                                                           uint32_t n, uint32_t nlist,
                                                           int32_t *__restrict__ offsets)
{
    const uint32_t l = blockIdx.x * 256u + threadIdx.x;
    if (l > nlist)
        return;
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < l)
            lo = mid + 1;
        else
            hi = mid;
    }
    offsets[l] = (int32_t)lo;
}

static bool sort_solo(int64_t n, int nlist) { return n <= kSoloSlots && nlist < kSoloBins; }

static uint32_t sort_blocks(int64_t n)
{
    return (uint32_t)((n + kSortChunk - 1) / kSortChunk);
}

size_t route_sort_bytes(int64_t n, int nlist)
{
    if (sort_solo(n, nlist))
        return 0;
    const size_t blocks = sort_blocks(n);
    const size_t bins = nlist < kSortBins ? (size_t)nlist + 1 : (size_t)kSortBins;
    size_t b = (bins * blocks + bins) * 4;
    if (nlist >= kSortBins || n <= kSoloSlots)
        b += (size_t)n * 4 * 3; // keys and slots after the first pass, keys after the second
    return b;
}

hipError_t launch_route_sort(const int32_t *lists, int64_t n, int nlist, void *ws, int32_t *offsets,
                             int32_t *order, int32_t *pos, hipStream_t stream)
{
    SortPass s{};
    s.lists = lists;
    s.n = (uint32_t)n;
    s.nlist = (uint32_t)nlist;
    s.blocks = sort_blocks(n);
    const bool two = nlist >= kSortBins;
    s.bins = two ? kSortBins : (uint32_t)nlist + 1;
    s.hist = static_cast<uint32_t *>(ws);
    s.total = s.hist + (size_t)s.bins * s.blocks;
    uint32_t *keys = s.total + s.bins, *slots = keys + n, *sorted = slots + n;
    if (n == 0) { // every list is empty
        hipLaunchKernelGGL(route_bounds_kernel, dim3((unsigned)nlist / 256 + 1), dim3(256), 0,
                           stream, nullptr, 0u, (uint32_t)nlist, offsets);
        return hipGetLastError();
    }
    if (sort_solo(n, nlist)) {
        s.order = order;
        s.pos = pos;
        s.offsets = offsets;
        hipLaunchKernelGGL((route_scatter_kernel<16, kSoloBins, true>), dim3(1), dim3(1024), 0,
                           stream, s);
        return hipGetLastError();
    }
    if (n <= kSoloSlots) { // more lists than the one-launch sort has counters for
        s.order = order;
        s.pos = pos;
        s.key_out = sorted;
        hipLaunchKernelGGL(route_solo_kernel, dim3(1), dim3(1024), 0, stream, s);
        hipLaunchKernelGGL(route_bounds_kernel, dim3((unsigned)nlist / 256 + 1), dim3(256), 0,
                           stream, sorted, (uint32_t)n, (uint32_t)nlist, offsets);
        return hipGetLastError();
    }
    for (int pass = 0; pass < (two ? 2 : 1); ++pass) {
        if (pass == 1) {
            s.shift = kSortBits;
            s.bins = ((uint32_t)nlist >> kSortBits) + 1;
            s.key_in = keys;
            s.slot_in = slots;
        }
        const bool last = pass == (two ? 1 : 0);
        s.key_out = !two ? nullptr : last ? sorted : keys;
        s.slot_out = last ? nullptr : slots;
        s.order = last ? order : nullptr;
        s.pos = last ? pos : nullptr;
        s.offsets = two ? nullptr : offsets;
        hipLaunchKernelGGL(route_count_kernel, dim3(s.blocks), dim3(64 * kSortWaves), 0, stream, s);
        hipLaunchKernelGGL(route_scan_kernel, dim3((s.bins + 63) / 64), dim3(1024), 0, stream, s);
        hipLaunchKernelGGL((route_scatter_kernel<kSortWaves, kSortBins, false>), dim3(s.blocks),
                           dim3(64 * kSortWaves), 0, stream, s);
    }
    if (two)
        hipLaunchKernelGGL(route_bounds_kernel, dim3((unsigned)nlist / 256 + 1), dim3(256), 0,
                           stream, sorted, (uint32_t)n, (uint32_t)nlist, offsets);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// rows there and back
// ---------------------------------------------------------------------------

// Lanes that share a row: enough for one 16-byte piece each, at most a wave.
template <typename T>
static int row_lanes(int d)
{
    const int pieces = (d + Piece<T>::N - 1) / Piece<T>::N;
    int l = 1;
    while (l < pieces && l < 64)
        l *= 2;
    return l;
}

// rows[p] = w x[t] of the slot at p (rounded once), zero where no slot is.  A
// thread has one piece of kRowsAtOnce rows that lie `step` apart, so that as many
// loads are under way: they wait for their slot numbers, and the stores for them.
// Bound by the rows written: 320,000 of 128 float32 35 us, 4.7 TB/s.
constexpr int kRowsAtOnce = 4;

template <typename T, bool NT>
__global__ __launch_bounds__(256) void route_gather_kernel(const T *__restrict__ x, int64_t n,
                                                           int64_t step, int d, FastDiv pieces,
                                                           FastDiv k,
                                                           const int32_t *__restrict__ order,
                                                           const float *__restrict__ weights,
                                                           T *__restrict__ rows, int64_t row0)
{
    constexpr int N = Piece<T>::N;
    const uint32_t g = blockIdx.x * 256u + threadIdx.x;
    const int64_t p0 = row0 + pieces.div(g);
    if (p0 >= step)
        return;
    const int c = (int)(g - (uint32_t)(p0 - row0) * pieces.c) * N;
    uint32_t u[kRowsAtOnce];
    Piece<T> v[kRowsAtOnce];
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i)
        u[i] = p0 + i * step < n ? (uint32_t)order[p0 + i * step] : ~0u;
    if (d - c >= N) {
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            v[i].load(x + (int64_t)k.div(u[i] < (uint64_t)n ? u[i] : 0) * d + c, N);
    } else {
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
            v[i].load(x + (int64_t)k.div(u[i] < (uint64_t)n ? u[i] : 0) * d + c, d - c);
    }
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const int64_t p = p0 + i * step;
        if (p >= n)
            break;
        if (u[i] >= (uint64_t)n) {
            v[i].zero();
        } else if (weights) {
            const float w = weights[u[i]];
#pragma unroll
            for (int e = 0; e < N; ++e)
                v[i].v[e] *= w;
        }
        v[i].template store<NT>(rows + p * d + c, d - c);
    }
}

// y[t] = sum over j of w[t][j] rows[pos[t][j]], j ascending in float32,
// rounded once; slots without a position add nothing (row 0 is read in their
// place and dropped, so that a batch of loads has no branch in it).  A thread
// has one piece of a vector, kSlotsAtOnce of its rows under way together.  Bound
// by the rows read: 10,000 vectors of 32 rows of 128 float32 33 us, 5.2 TB/s;
// 16,384 of 8 rows of 2048 bfloat16 133 us, 4.5 TB/s.
constexpr int kSlotsAtOnce = 8;

template <typename T>
__global__ __launch_bounds__(256) void route_combine_kernel(const T *__restrict__ rows,
                                                            int64_t nvec, int d, FastDiv pieces,
                                                            int k,
                                                            const int32_t *__restrict__ pos,
                                                            const float *__restrict__ weights,
                                                            T *__restrict__ out, int64_t row0)
{
    constexpr int N = Piece<T>::N;
    const uint32_t g = blockIdx.x * 256u + threadIdx.x;
    const int64_t t = row0 + pieces.div(g);
    if (t >= nvec)
        return;
    const int c = (int)(g - (uint32_t)(t - row0) * pieces.c) * N;
    const int64_t n = nvec * k;
    const bool whole = d - c >= N;
    Piece<T> sum;
    sum.zero();
    for (int j0 = 0; j0 < k; j0 += kSlotsAtOnce) {
        int64_t p[kSlotsAtOnce];
        float w[kSlotsAtOnce];
        Piece<T> v[kSlotsAtOnce];
        if (j0 + kSlotsAtOnce <= k) { // eight numbers in two loads, at any alignment
            typedef int32_t I8 __attribute__((ext_vector_type(8), aligned(4)));
            typedef float F8 __attribute__((ext_vector_type(8), aligned(4)));
            const I8 pv = *reinterpret_cast<const I8 *>(pos + t * k + j0);
            F8 wv = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            if (weights)
                wv = *reinterpret_cast<const F8 *>(weights + t * k + j0);
#pragma unroll
            for (int j = 0; j < kSlotsAtOnce; ++j) {
                p[j] = pv[j];
                w[j] = wv[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSlotsAtOnce; ++j) {
                const int at = min(j0 + j, k - 1);
                p[j] = j0 + j < k ? pos[t * k + at] : -1;
                w[j] = weights ? weights[t * k + at] : 1.f;
            }
        }
        if (whole) {
#pragma unroll
            for (int j = 0; j < kSlotsAtOnce; ++j)
                v[j].load(rows + ((uint64_t)p[j] < (uint64_t)n ? p[j] : 0) * d + c, N);
        } else {
#pragma unroll
            for (int j = 0; j < kSlotsAtOnce; ++j)
                v[j].load(rows + ((uint64_t)p[j] < (uint64_t)n ? p[j] : 0) * d + c, d - c);
        }
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
            const bool kept = (uint64_t)p[j] < (uint64_t)n;
#pragma unroll
            for (int e = 0; e < N; ++e)
                sum.v[e] = kept ? fmaf(w[j], v[j].v[e], sum.v[e]) : sum.v[e];
        }
    }
    sum.store(out + t * d + c, d - c);
}

// Gradient of the weighted sum, a group of lanes a slot: d_rows[p] = w dy[t]
// and d_weights[slot] = <dy[t], rows[p]>, summed in float32 in an order that
// depends on d alone.  The same group also clears row number slot when no slot
// sits there.  Bound by the rows read and written: 131,072 of 2048 bfloat16 223
// us, 5.1 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void route_combine_grad_kernel(
    const T *__restrict__ grad, const T *__restrict__ rows, int64_t n, int d, int lanes, FastDiv k,
    const int32_t *__restrict__ order, const int32_t *__restrict__ pos,
    const float *__restrict__ weights, T *__restrict__ d_rows, float *__restrict__ d_weights,
    int64_t block0)
{
    constexpr int N = Piece<T>::N;
    const int64_t u = (block0 + blockIdx.x) * (256 / lanes) + threadIdx.x / lanes;
    const int sub = threadIdx.x & (lanes - 1);
    const int64_t p = u < n ? pos[u] : -1;
    const bool kept = p >= 0 && p < n;
    const bool clear = u < n && (uint32_t)order[u] >= (uint64_t)n;
    const T *dy = grad + (u < n ? (int64_t)k.div((uint32_t)u) : 0) * d;
    const float w = kept ? weights[u] : 0.f;
    float dot = 0.f;
    for (int c = sub * N; c < d; c += lanes * N) {
        if (kept) {
            Piece<T> g, r;
            g.load(dy + c, d - c);
            r.load(rows + p * d + c, d - c);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                dot = fmaf(g.v[i], r.v[i], dot);
                g.v[i] *= w;
            }
            g.store(d_rows + p * d + c, d - c);
        }
        if (clear) {
            Piece<T> z;
            z.zero();
            z.store(d_rows + u * d + c, d - c);
        }
    }
    for (int s = 1; s < lanes; s <<= 1)
        dot += __uint_as_float((uint32_t)__builtin_amdgcn_ds_bpermute(
            (lane_id() ^ s) << 2, (int)__float_as_uint(dot)));
    if (sub == 0 && u < n)
        d_weights[u] = dot;
}

template <typename T>
static hipError_t gather_as(const void *x, int64_t nvec, int d, const int32_t *order,
                            const float *weights, int k, void *rows, hipStream_t stream)
{
    const int64_t pieces = (d + Piece<T>::N - 1) / Piece<T>::N, n = nvec * k;
    const int64_t step = (n + kRowsAtOnce - 1) / kRowsAtOnce;
    const int64_t most = 0x7FFFFF00ll / pieces; // rows of one launch: 32-bit piece numbers
    // Rows that would fill half of the last-level cache (256 MB) go past it:
    // 164 MB of them 42 -> 35 us, and what lay in the cache stays.  Fewer rows
    // are better kept for their reader.
    const bool past = n * d * (int64_t)sizeof(T) >= (int64_t)128 << 20;
    for (int64_t r = 0; r < step; r += most) {
        const int64_t now = (step - r < most ? step - r : most) * pieces;
        const auto kernel = past ? route_gather_kernel<T, true> : route_gather_kernel<T, false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)((now + 255) / 256)), dim3(256), 0, stream,
                           static_cast<const T *>(x), n, step, d, FastDiv((uint32_t)pieces),
                           FastDiv((uint32_t)k), order, weights, static_cast<T *>(rows), r);
    }
    return hipGetLastError();
}

template <typename T>
static hipError_t combine_as(const void *rows, int64_t nvec, int d, const int32_t *pos,
                             const float *weights, int k, void *out, hipStream_t stream)
{
    const int64_t pieces = (d + Piece<T>::N - 1) / Piece<T>::N;
    const int64_t most = 0x7FFFFF00ll / pieces;
    for (int64_t r = 0; r < nvec; r += most) {
        const int64_t now = (nvec - r < most ? nvec - r : most) * pieces;
        hipLaunchKernelGGL(route_combine_kernel<T>, dim3((unsigned)((now + 255) / 256)), dim3(256),
                           0, stream, static_cast<const T *>(rows), nvec, d,
                           FastDiv((uint32_t)pieces), k, pos, weights, static_cast<T *>(out), r);
    }
    return hipGetLastError();
}

template <typename T>
static hipError_t combine_grad_as(const void *grad, const void *rows, int64_t nvec, int d,
                                  const int32_t *order, const int32_t *pos, const float *weights,
                                  int k, void *d_rows, float *d_weights, hipStream_t stream)
{
    const int lanes = row_lanes<T>(d);
    const int64_t n = nvec * k, blocks = (n + 256 / lanes - 1) / (256 / lanes);
    const int64_t most = most_blocks(256);
    for (int64_t b = 0; b < blocks; b += most)
        hipLaunchKernelGGL(route_combine_grad_kernel<T>,
                           dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(256), 0,
                           stream, static_cast<const T *>(grad), static_cast<const T *>(rows), n, d,
                           lanes, FastDiv((uint32_t)k), order, pos, weights,
                           static_cast<T *>(d_rows), d_weights, b);
    return hipGetLastError();
}

hipError_t launch_route_gather(const void *x, int type, int64_t nvec, int d, const int32_t *order,
                               const float *weights, int k, void *rows, hipStream_t stream)
{
    switch (type) {
    case kF32: return gather_as<float>(x, nvec, d, order, weights, k, rows, stream);
    case kBF16: return gather_as<__bf16>(x, nvec, d, order, weights, k, rows, stream);
    default: return gather_as<_Float16>(x, nvec, d, order, weights, k, rows, stream);
    }
}

hipError_t launch_route_combine(const void *rows, int type, int64_t nvec, int d, const int32_t *pos,
                                const float *weights, int k, void *out, hipStream_t stream)
{
    switch (type) {
    case kF32: return combine_as<float>(rows, nvec, d, pos, weights, k, out, stream);
    case kBF16: return combine_as<__bf16>(rows, nvec, d, pos, weights, k, out, stream);
    default: return combine_as<_Float16>(rows, nvec, d, pos, weights, k, out, stream);
    }
}

hipError_t launch_route_combine_grad(const void *grad, const void *rows, int type, int64_t nvec,
                                     int d, const int32_t *order, const int32_t *pos,
                                     const float *weights, int k, void *d_rows, float *d_weights,
                                     hipStream_t stream)
{
    switch (type) {
    case kF32:
        return combine_grad_as<float>(grad, rows, nvec, d, order, pos, weights, k, d_rows,
                                      d_weights, stream);
    case kBF16:
        return combine_grad_as<__bf16>(grad, rows, nvec, d, order, pos, weights, k, d_rows,
                                       d_weights, stream);
    default:
        return combine_grad_as<_Float16>(grad, rows, nvec, d, order, pos, weights, k, d_rows,
                                         d_weights, stream);
    }
}

} // namespace ivfpq
