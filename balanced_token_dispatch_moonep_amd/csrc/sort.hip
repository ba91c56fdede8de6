// Tokens sorted by expert: the rows of all (token, k) pairs grouped by expert, in pair order inside a group.
//
// What bounds it is latency, two launches and a few dependent loads: 262144 pairs over 256 experts are 3 MB and
// take 12 us, 2.8 to count and 9.5 to place (9.9 where the other parts' counts are asked for after the part's own are
// made); 1024 pairs, one launch, 3.8 us.  With parts of 4096 pairs it took 20, with counts read by a thread an expert 17.
#include "sort.h"

namespace moonep {

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

template <bool ONCE>
__global__ __launch_bounds__(64 * kSortWaves) void sort_place_kernel(SortArgs a) {
    sort_place<ONCE>(a, blockIdx.x);
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
    return align_up(std::max<size_t>(sort_hist_most(dims->R * dims->S * dims->K, dims->E), 1), 256);
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
