// Tokens sorted by expert: the rows of all (token, k) pairs grouped by expert, in pair order inside a group.
//
// A stable counting sort.  Up to kSortOnce pairs one workgroup does all of it; more are cut into parts, one
// launch counts each part's pairs by expert, and in a second one each part adds the counts of the parts
// before it to where each expert begins.  Inside a part a wave owns consecutive pairs, its own counts by
// expert, and ranks 64 pairs at a time: lanes with the same id find each other by one ballot for each
// bit of the id.  No order depends on atomics: those only count.
// What bounds it is latency, two launches and a few dependent loads: 262144 pairs are 3 MB.
#include "sort.h"

namespace moonep {

constexpr int kKept = 4;             // rounds of 64 pairs: a wave's share of kSortPart

// Lanes of the wave with this lane's id; ids below 2^bits.
__device__ __forceinline__ unsigned long long same_id(int id, bool valid, int bits) {
    unsigned long long m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const unsigned long long one = __ballot((id >> b) & 1);
        m &= (id >> b) & 1 ? one : ~one;
    }
    return m;
}

__global__ __launch_bounds__(64 * kSortWaves) void sort_count_kernel(SortArgs a) {
    __shared__ int count[kMaxE];
    for (int e = threadIdx.x; e < a.E; e += 64 * kSortWaves) count[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * a.part, last = min(a.P - first, a.part);
    for (int i = threadIdx.x; i < last; i += 64 * kSortWaves) {
        const int id = a.topk[first + i];
        if ((unsigned)id < (unsigned)a.E) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    const int even = (a.E + 1) & ~1;
    for (int e = threadIdx.x; e < even; e += 64 * kSortWaves) a.hist[(size_t)blockIdx.x * even + e] = e < a.E ? count[e] : 0;
}

// Exclusive prefix sums over the experts of up to two counts each, for threads that hold two experts in a row.
__device__ __forceinline__ int wave_scan_sum(int v) {
    const int lane = threadIdx.x & 63;
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}
__device__ __forceinline__ int block_before(int v, int* sums) {
    const int s = wave_scan_sum(v), wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sums[wave] = s;
    __syncthreads();
    int before = s - v;
    for (int w = 0; w < wave; ++w) before += sums[w];
    return before;
}

template <bool ONCE>
__global__ __launch_bounds__(64 * kSortWaves) void sort_place_kernel(SortArgs a) {
    constexpr int NT = 64 * kSortWaves, PER = kMaxE / NT;
    __shared__ int at[kSortWaves][kMaxE];        // a wave's counts, then where its next pair of an expert goes
    __shared__ int sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < a.E; e += NT)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) at[w][e] = 0;
    __syncthreads();
    const int begin = blockIdx.x * a.part, n = min(a.P - begin, a.part);
    const int rounds = (n + NT - 1) / NT;        // of 64 pairs a wave
    const int first = begin + wave * rounds * 64, last = min(begin + n, first + rounds * 64);
    // the first kKept rounds' ids stay in registers for the second time that they are needed
    int kept[kKept];
#pragma unroll
    for (int r = 0; r < kKept; ++r) {
        const int p = first + r * 64 + lane;
        kept[r] = p < last ? a.topk[p] : -1;
    }
#pragma unroll
    for (int r = 0; r < kKept; ++r)
        if ((unsigned)kept[r] < (unsigned)a.E) atomicAdd(&at[wave][kept[r]], 1);
    for (int p = first + kKept * 64 + lane; p < last; p += 64) {
        const int id = a.topk[p];
        if ((unsigned)id < (unsigned)a.E) atomicAdd(&at[wave][id], 1);
    }
    // pairs of each expert in all parts, and in the parts before this one
    int total[PER], before[PER], mine[PER];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        total[i] = before[i] = mine[i] = 0;
        if (e >= a.E) continue;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) mine[i] += at[w][e];
        if constexpr (ONCE) total[i] = mine[i];
    }
    if constexpr (!ONCE) {
        // two experts a thread; where that is not all threads, several groups of them share the parts
        __shared__ int2 sums_of[2][NT];
        const int pairs = (a.E + 1) / 2, groups = min(NT / pairs, 16), g = tid / pairs;
        int2 all = make_int2(0, 0), earlier = make_int2(0, 0);
        if (g < groups) {
            const int2* h = reinterpret_cast<const int2*>(a.hist) + tid % pairs;
#pragma unroll 8
            for (int b = g; b < a.parts; b += groups) {
                const int2 c = h[(size_t)b * pairs];
                const bool before_this = b < (int)blockIdx.x;
                all.x += c.x;
                all.y += c.y;
                earlier.x += before_this ? c.x : 0;
                earlier.y += before_this ? c.y : 0;
            }
        }
        sums_of[0][tid] = all;
        sums_of[1][tid] = earlier;
        __syncthreads();
        static_assert(PER == 2, "a thread's experts are one pair");
        if (tid < pairs)
            for (int i = 0; i < groups; ++i) {
                const int2 c = sums_of[0][i * pairs + tid], b = sums_of[1][i * pairs + tid];
                total[0] += c.x;
                total[1] += c.y;
                before[0] += b.x;
                before[1] += b.y;
            }
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += total[i];
    int start = block_before(sum, sums);
    if (blockIdx.x == 0 && tid == NT - 1) a.offsets[a.E] = start + sum;
    int runs = 0, start0 = start;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        if (e < a.E) {
            if (blockIdx.x == 0) a.offsets[e] = start;
            int next = start + before[i];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const int c = at[w][e];
                at[w][e] = next;
                next += c;
            }
        }
        start += total[i];
        if (a.run_rows) runs += (total[i] + a.run_rows - 1) / a.run_rows;
    }
    if (a.run_rows && blockIdx.x == 0) {
        int r = block_before(runs, sums);
        if (tid == NT - 1) a.nruns[0] = r + runs;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            for (int o = 0; o < total[i]; o += a.run_rows)
                a.runs[r++] = Run{tid * PER + i, start0 + o, min(a.run_rows, total[i] - o)};
            start0 += total[i];
        }
    }
    __syncthreads();
    const int bits = 32 - __clz(a.E);
    auto place = [&](int p, int id, bool valid, unsigned long long same) {
        int row = -1;
        if (valid) {
            row = at[wave][id] + __popcll(same & ((1ull << lane) - 1));
            if (a.pair) a.pair[row] = p;
        }
        if (p < last) a.dest[p] = row;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (valid && lane == 63 - __clzll(same)) at[wave][id] = row + 1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    unsigned long long same[kKept];
#pragma unroll
    for (int r = 0; r < kKept; ++r) same[r] = same_id(kept[r], (unsigned)kept[r] < (unsigned)a.E, bits);
#pragma unroll
    for (int r = 0; r < kKept; ++r) place(first + r * 64 + lane, kept[r], (unsigned)kept[r] < (unsigned)a.E, same[r]);
    for (int p0 = first + kKept * 64; p0 < last; p0 += 64) {
        const int p = p0 + lane;
        const int id = p < last ? a.topk[p] : -1;
        const bool valid = (unsigned)id < (unsigned)a.E;
        place(p, id, valid, same_id(id, valid, bits));
    }
}

int launch_sort(const SortArgs& a, hipStream_t s) {
    if (a.parts == 1) {
        hipLaunchKernelGGL(sort_place_kernel<true>, dim3(1), dim3(64 * kSortWaves), 0, s, a);
        MOONEP_LAUNCH_CHECK();
        return MOONEP_OK;
    }
    hipLaunchKernelGGL(sort_count_kernel, dim3(a.parts), dim3(64 * kSortWaves), 0, s, a);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(sort_place_kernel<false>, dim3(a.parts), dim3(64 * kSortWaves), 0, s, a);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

static int check_sort(const moonep_dims_t* d) {
    if (!d || check_flags(d) != MOONEP_OK) return MOONEP_EINVAL;
    if (d->R < 1 || d->R > kMaxR || d->S < 1 || d->E < 1 || d->E > kMaxE) return MOONEP_EINVAL;
    if (d->K < 1 || d->K > kMaxK) return MOONEP_EINVAL;
    if ((int64_t)d->R * d->S * d->K > (int64_t)1 << 30) return MOONEP_EINVAL;
    return MOONEP_OK;
}

}  // namespace moonep

using namespace moonep;

extern "C" size_t moonep_sort_workspace_bytes(const moonep_dims_t* dims) {
    if (check_sort(dims) != MOONEP_OK) return 0;
    return align_up(std::max<size_t>(sort_hist_bytes(sort_args(dims->R * dims->S * dims->K, dims->E)), 1), 256);
}

extern "C" int moonep_sort(const moonep_dims_t* dims, const int32_t* topk, void* ws, int32_t* offsets, int32_t* dest,
                           int32_t* pair, void* stream) {
    const int rc = check_sort(dims);
    if (rc != MOONEP_OK) return rc;
    MOONEP_CHECK_PTR(topk);
    MOONEP_CHECK_PTR(ws);
    MOONEP_CHECK_PTR(offsets);
    MOONEP_CHECK_PTR(dest);
    if (pair && !aligned16(pair)) return MOONEP_EALIGN;
    SortArgs a = sort_args(dims->R * dims->S * dims->K, dims->E);
    const size_t pairs = (size_t)a.P * 4;
    const Span spans[] = {{ws, moonep_sort_workspace_bytes(dims)}, {offsets, (a.E + 1) * 4u}, {dest, pairs}, {pair, pairs},
                          {topk, pairs}};
    if (outputs_overlap(spans, 4, 5)) return MOONEP_EINVAL;
    a.topk = topk, a.hist = static_cast<int32_t*>(ws), a.offsets = offsets, a.dest = dest, a.pair = pair;
    return launch_sort(a, static_cast<hipStream_t>(stream));
}
