// Pairs (token, k) sorted by expert: shared by moonep_sort and the 8-bit experts.
//
// A stable counting sort.  Up to kSortOnce pairs one workgroup does all of it; more are cut into parts, one
// launch counts each part's pairs by expert, and in a second one each part adds the counts of the parts
// before it to where each expert begins.  Inside a part a wave owns consecutive pairs, its own counts by
// expert, and ranks 64 pairs at a time: lanes with the same id find each other by one ballot for each
// bit of the id.  No order depends on atomics: those only count.
#pragma once

#include "common.h"

namespace moonep {

constexpr int kSortWaves = 8;
constexpr int kSortOnce = 2048;      // pairs that one workgroup sorts in one launch (5.1 us; 4096 8.8, two launches 6.9)
constexpr int kSortParts = 256;      // workgroups of a larger sort, at most
// Pairs of one of them, at least: each reads the counts of all.  Parts of 1024 / 2048 pairs (us, 256 experts): 8192 pairs
// 7.2 / 8.1, 32768 7.5 / 9.1, 65536 8.2 / 8.9, 262144 12.4 / 11.3, and of 1024 experts 25 / 18.
constexpr int kSortPart = 1024, kSortLargePart = 2048, kSortLarge = 1 << 16;

// Runs of an expert's rows for the workgroups of a product: run i covers rows first .. first + n of expert e.
struct Run {
    int32_t expert, first, n;
};

struct SortArgs {
    const int32_t* topk;             // [P]
    int32_t P, E;
    int32_t part, parts;             // pairs a workgroup, workgroups
    int32_t* hist;                   // [parts][E, even], with more than one workgroup: each part's counts
    int32_t* offsets;                // [E + 1]
    int32_t* dest;                   // [P]: row of the pair, -1 without an expert
    int32_t* pair;                   // [P]: pair of the row, or NULL
    int32_t run_rows;                // > 0: also cut into runs of so many rows
    Run* runs;
    int32_t* nruns;                  // [1]
};

inline SortArgs sort_args(int P, int E) {
    SortArgs a{};
    a.P = P, a.E = E;
    if (P <= kSortOnce) {
        a.part = P, a.parts = 1;
    } else {
        // whole rounds of the workgroup's waves
        constexpr int round = kSortWaves * 64;
        a.part = std::max(P <= kSortLarge ? kSortPart : kSortLargePart, (P + kSortParts - 1) / kSortParts);
        a.part = (a.part + round - 1) / round * round;
        a.parts = (P + a.part - 1) / a.part;
    }
    return a;
}
// What a sort of up to P pairs takes, at most.
inline size_t sort_hist_most(int64_t P, int E) {
    const int64_t small = (std::min<int64_t>(P, kSortLarge) + kSortPart - 1) / kSortPart;
    const int64_t parts = std::max(small, std::min<int64_t>((P + kSortLargePart - 1) / kSortLargePart, kSortParts));
    return P > kSortOnce ? (size_t)parts * ((E + 1) / 2) * 8 : 0;
}
int launch_sort(const SortArgs& a, hipStream_t s);

constexpr int kKept = 4;             // rounds of 64 pairs: a wave's share of kSortLargePart

// Lanes of the wave with this lane's id; ids below 2^bits.
__device__ __forceinline__ unsigned long long same_id(int id, bool valid, int bits) {
    unsigned long long m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const unsigned long long one = __ballot((id >> b) & 1);
        m &= (id >> b) & 1 ? one : ~one;
    }
    return m;
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

// Places part `part` of the pairs: a workgroup's work.  ONCE: there is no other part.
template <bool ONCE>
__device__ __forceinline__ void sort_place(const SortArgs& a, int part) {
    constexpr int NT = 64 * kSortWaves, PER = kMaxE / NT;
    __shared__ int at[kSortWaves][kMaxE];        // a wave's counts, then where its next pair of an expert goes
    __shared__ int sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < a.E; e += NT)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) at[w][e] = 0;
    const int begin = part * a.part, n = min(a.P - begin, a.part);
    const int rounds = (n + NT - 1) / NT;        // of 64 pairs a wave
    const int first = begin + wave * rounds * 64, last = min(begin + n, first + rounds * 64);
    // the first kKept rounds' ids stay in registers for the second time that they are needed
    int kept[kKept];
#pragma unroll
    for (int r = 0; r < kKept; ++r) {
        const int p = first + r * 64 + lane;
        kept[r] = p < last ? a.topk[p] : -1;
    }
    // the other parts' counts, on their way with the ids: two experts a thread; where that is not all threads, several
    // groups of them share the parts
    __shared__ int2 sums_of[2][ONCE ? 1 : NT];
    const int pairs = (a.E + 1) / 2, groups = min(NT / pairs, 16);
    if constexpr (!ONCE) {
        int2 all = make_int2(0, 0), earlier = make_int2(0, 0);
        if (tid / pairs < groups) {
            const int2* h = reinterpret_cast<const int2*>(a.hist) + tid % pairs;
#pragma unroll 8
            for (int b = tid / pairs; b < a.parts; b += groups) {
                const int2 c = h[(size_t)b * pairs];
                const bool before_this = b < part;
                all.x += c.x;
                all.y += c.y;
                earlier.x += before_this ? c.x : 0;
                earlier.y += before_this ? c.y : 0;
            }
        }
        sums_of[0][tid] = all;
        sums_of[1][tid] = earlier;
    }
    __syncthreads();
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
    if (part == 0 && tid == NT - 1) a.offsets[a.E] = start + sum;
    int runs = 0, start0 = start;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        if (e < a.E) {
            if (part == 0) a.offsets[e] = start;
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
    if (a.run_rows && part == 0) {
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
    for (int r = 0; r < kKept; ++r)
        if (r < rounds) same[r] = same_id(kept[r], (unsigned)kept[r] < (unsigned)a.E, bits);
#pragma unroll
    for (int r = 0; r < kKept; ++r)
        if (r < rounds) place(first + r * 64 + lane, kept[r], (unsigned)kept[r] < (unsigned)a.E, same[r]);
    for (int p0 = first + kKept * 64; p0 < last; p0 += 64) {
        const int p = p0 + lane;
        const int id = p < last ? a.topk[p] : -1;
        const bool valid = (unsigned)id < (unsigned)a.E;
        place(p, id, valid, same_id(id, valid, bits));
    }
}

}  // namespace moonep
