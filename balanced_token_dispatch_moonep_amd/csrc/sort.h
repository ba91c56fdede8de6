// Pairs (token, k) sorted by expert: shared by moonep_sort and the 8-bit experts.
#pragma once

#include "common.h"

namespace moonep {

constexpr int kSortWaves = 8;
constexpr int kSortOnce = 8192;      // pairs that one workgroup sorts in one launch
constexpr int kSortParts = 256;      // workgroups of a larger sort, at most
constexpr int kSortPart = 2048;      // pairs of one of them, at least

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
        a.part = std::max(kSortPart, (P + kSortParts - 1) / kSortParts);
        a.part = (a.part + round - 1) / round * round;
        a.parts = (P + a.part - 1) / a.part;
    }
    return a;
}
// The most that a sort of up to P pairs takes.
inline size_t sort_hist_most(int64_t P, int E) {
    return P > kSortOnce ? (size_t)std::min<int64_t>((P + kSortPart - 1) / kSortPart, kSortParts) * ((E + 1) / 2) * 8 : 0;
}
inline size_t sort_hist_bytes(const SortArgs& a) { return a.parts > 1 ? (size_t)a.parts * ((a.E + 1) / 2) * 8 : 0; }
int launch_sort(const SortArgs& a, hipStream_t s);

}  // namespace moonep
