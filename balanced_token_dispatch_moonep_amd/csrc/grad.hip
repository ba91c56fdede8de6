// The global norm of many gradients, and clipping by it.
//
// Both are streams over memory: the norm reads every gradient once, clipping reads and writes it
// once (or leaves it alone where the norm is small enough).  The gradients' addresses travel in the
// kernel arguments, kTable of them a launch, so a call needs no device table and can be captured.
// On one MI355X, 1409 MB of float32 gradients: norm 208 us (6.8 TB/s), clipping 528 us (5.3 TB/s); the
// float64 sums cost nothing beside the loads (loads of 4 bytes and one accumulator: 1556 us for both).
#include "common.h"

#include <cfloat>
#include <cmath>
#include <vector>

namespace moonep {

constexpr int kTable = 160;          // gradients a launch: 20 bytes each, within 4 KiB of arguments
constexpr int kSpan = 16384;         // elements a workgroup takes at a time
constexpr int kNormBlocks = 2048;    // workgroups (and partial sums) a launch, at most

struct GradTable {
    uint64_t at[kTable];             // address; bit 0: the type
    int64_t numel[kTable];
    int32_t first[kTable + 1];       // spans before gradient i
    int32_t n;
};
static_assert(sizeof(GradTable) <= 3584, "kernel arguments");

// The gradient that span c is of.
__device__ __forceinline__ int find_grad(const GradTable& t, int c) {
    int lo = 0, hi = t.n;            // first[lo] <= c < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double lds[4];
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// A float32 has 24 bits, so a float64 holds its square exactly; two accumulators a lane keep the
// chains of dependent additions short.
__device__ __forceinline__ void add_square(double& s, float f) { s += (double)f * (double)f; }

template <bool BF16>
__device__ __forceinline__ void add_squares(double& s, double& t, uint4 v) {
    if constexpr (BF16) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            add_square(s, bf16_lo(w[i]));
            add_square(t, bf16_hi(w[i]));
        }
    } else {
        add_square(s, __uint_as_float(v.x));
        add_square(t, __uint_as_float(v.y));
        add_square(s, __uint_as_float(v.z));
        add_square(t, __uint_as_float(v.w));
    }
}

template <bool BF16>
__device__ __forceinline__ float one(const void* g, int j) {
    if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(g)[j] << 16);
    else return static_cast<const float*>(g)[j];
}

constexpr int kUnroll = 4;           // 16-byte loads a lane has in flight

// Gradients that the caches cannot hold are loaded and stored past them (non-temporal): norm and
// clipping of 1409 MB took 742 us so and 814 us otherwise, of 128 MB 73 and 79 us.  Where the last
// pass has left them in the caches that would be the slower way: 38 MB took 29 us so and 25 us otherwise.
constexpr int64_t kStreamBytes = 100 << 20;

template <bool STREAM>
__device__ __forceinline__ uint4 load(const uint4* p) {
    if constexpr (STREAM) return ld_nt(p);
    else return *p;
}
template <bool STREAM>
__device__ __forceinline__ void store(uint4 v, uint4* p) {
    if constexpr (STREAM) st_nt(v, p);
    else *p = v;
}

// Squares of n elements from g (16-byte aligned), by the workgroup.
template <bool BF16, bool STREAM>
__device__ __forceinline__ void span_squares(const void* g, int n, double& s, double& t) {
    constexpr int N = BF16 ? 8 : 4;
    const uint4* p = static_cast<const uint4*>(g);
    const int nv = n / N;
    int v = threadIdx.x;
    for (; v + 256 * (kUnroll - 1) < nv; v += 256 * kUnroll) {
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u] = load<STREAM>(p + v + 256 * u);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) add_squares<BF16>(s, t, x[u]);
    }
    for (; v < nv; v += 256) add_squares<BF16>(s, t, p[v]);
    const int j = nv * N + threadIdx.x;
    if (j < n) add_square(s, one<BF16>(g, j));
}

// A float32 times the factor, rounded to float32 once.  The factor is a float64, which costs nothing beside
// the loads and stores: max_norm / norm may lie where float32 has few bits left or none, with a product
// that does not.
__device__ __forceinline__ float scaled(float g, double f) { return (float)((double)g * f); }

template <bool BF16>
__device__ __forceinline__ uint4 times(uint4 v, double f) {
    if constexpr (BF16)
        return make_uint4(pack_bf16(scaled(bf16_lo(v.x), f), scaled(bf16_hi(v.x), f)),
                          pack_bf16(scaled(bf16_lo(v.y), f), scaled(bf16_hi(v.y), f)),
                          pack_bf16(scaled(bf16_lo(v.z), f), scaled(bf16_hi(v.z), f)),
                          pack_bf16(scaled(bf16_lo(v.w), f), scaled(bf16_hi(v.w), f)));
    else
        return make_uint4(__float_as_uint(scaled(__uint_as_float(v.x), f)), __float_as_uint(scaled(__uint_as_float(v.y), f)),
                          __float_as_uint(scaled(__uint_as_float(v.z), f)), __float_as_uint(scaled(__uint_as_float(v.w), f)));
}

template <bool BF16, bool STREAM>
__device__ __forceinline__ void span_times(void* g, int n, double f) {
    constexpr int N = BF16 ? 8 : 4;
    uint4* p = static_cast<uint4*>(g);
    const int nv = n / N;
    int v = threadIdx.x;
    for (; v + 256 * (kUnroll - 1) < nv; v += 256 * kUnroll) {
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u] = load<STREAM>(p + v + 256 * u);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) store<STREAM>(times<BF16>(x[u], f), p + v + 256 * u);
    }
    for (; v < nv; v += 256) p[v] = times<BF16>(p[v], f);
    const int j = nv * N + threadIdx.x;
    if (j < n) {
        const float r = scaled(one<BF16>(g, j), f);
        if constexpr (BF16) static_cast<uint16_t*>(g)[j] = (uint16_t)pack_bf16(r, 0.0f);
        else static_cast<float*>(g)[j] = r;
    }
}

// part[block] = sum of squares of the block's spans, in float64.
template <bool STREAM>
__global__ __launch_bounds__(256) void grad_squares_kernel(GradTable t, double* __restrict__ part) {
    double s0 = 0.0, s1 = 0.0;
    const int spans = t.first[t.n];
    for (int c = blockIdx.x; c < spans; c += gridDim.x) {
        const int i = find_grad(t, c);
        const int64_t lo = (int64_t)(c - t.first[i]) * kSpan;
        const int n = (int)std::min<int64_t>(kSpan, t.numel[i] - lo);
        const uint64_t at = t.at[i];
        if (at & MOONEP_GRAD_BF16) span_squares<true, STREAM>(reinterpret_cast<const char*>(at & ~1ull) + lo * 2, n, s0, s1);
        else span_squares<false, STREAM>(reinterpret_cast<const char*>(at) + lo * 4, n, s0, s1);
    }
    const double s = block_sum(s0 + s1);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void grad_join_kernel(const double* __restrict__ part, int n,
                                                        float* __restrict__ norm) {
    double s = 0.0;
#pragma unroll 8
    for (int j = threadIdx.x; j < n; j += 256) s += part[j];
    s = block_sum(s);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
}

template <bool STREAM>
__global__ __launch_bounds__(256) void grad_clip_kernel(GradTable t, const float* __restrict__ norm, float most) {
    const float s = norm[0];
    if (s <= most) return;
    const float q = most / s;        // NaN for a NaN norm, 0 for an infinite one
    const double f = q < FLT_MIN ? (double)most / (double)s : (double)q;
    const int spans = t.first[t.n];
    for (int c = blockIdx.x; c < spans; c += gridDim.x) {
        const int i = find_grad(t, c);
        const int64_t lo = (int64_t)(c - t.first[i]) * kSpan;
        const int n = (int)std::min<int64_t>(kSpan, t.numel[i] - lo);
        const uint64_t at = t.at[i];
        if (at & MOONEP_GRAD_BF16) span_times<true, STREAM>(reinterpret_cast<char*>(at & ~1ull) + lo * 2, n, f);
        else span_times<false, STREAM>(reinterpret_cast<char*>(at) + lo * 4, n, f);
    }
}

static int check_grads(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* dtype) {
    if (n < 0 || (n > 0 && (!grads || !numel || !dtype))) return MOONEP_EINVAL;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        if (numel[i] < 0 || numel[i] > (int64_t)1 << 40) return MOONEP_EINVAL;
        if (dtype[i] != MOONEP_GRAD_F32 && dtype[i] != MOONEP_GRAD_BF16) return MOONEP_EINVAL;
        if (numel[i] == 0) continue;
        MOONEP_CHECK_PTR(grads[i]);
        total += (numel[i] + kSpan - 1) / kSpan;
    }
    return total > 0x7fffffff ? MOONEP_EINVAL : MOONEP_OK;
}

static bool streams(int32_t n, const int64_t* numel, const int32_t* dtype) {
    int64_t bytes = 0;
    for (int i = 0; i < n; ++i) bytes += numel[i] * (dtype[i] == MOONEP_GRAD_BF16 ? 2 : 4);
    return bytes > kStreamBytes;
}

// Calls launch(table, workgroups) for every kTable gradients that hold something.
template <class F>
static int for_tables(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* dtype, F launch) {
    for (int i = 0; i < n;) {
        GradTable t{};
        for (; i < n && t.n < kTable; ++i) {
            if (numel[i] == 0) continue;
            t.at[t.n] = reinterpret_cast<uint64_t>(grads[i]) | (uint64_t)dtype[i];
            t.numel[t.n] = numel[i];
            t.first[t.n + 1] = t.first[t.n] + (int32_t)((numel[i] + kSpan - 1) / kSpan);
            ++t.n;
        }
        if (t.n == 0) break;
        launch(t, std::min(t.first[t.n], kNormBlocks));
        if (hipGetLastError() != hipSuccess) return MOONEP_EHIP;
    }
    return MOONEP_OK;
}

// Whether two of the gradients share memory.
static bool overlap(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* dtype) {
    auto begin = [&](int i) { return reinterpret_cast<uintptr_t>(grads[i]); };
    auto end = [&](int i) { return begin(i) + (uintptr_t)numel[i] * (dtype[i] == MOONEP_GRAD_BF16 ? 2 : 4); };
    std::vector<int32_t> order;
    order.reserve(n);
    bool sorted = true;
    for (int i = 0; i < n; ++i) {
        if (numel[i] == 0) continue;
        sorted = sorted && (order.empty() || begin(order.back()) <= begin(i));
        order.push_back(i);
    }
    if (!sorted) std::sort(order.begin(), order.end(), [&](int a, int b) { return begin(a) < begin(b); });
    for (size_t j = 1; j < order.size(); ++j)
        if (end(order[j - 1]) > begin(order[j])) return true;
    return false;
}

// Whether a gradient and the `bytes` at p share memory.
static bool touches(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* dtype, const void* p,
                    size_t bytes) {
    for (int i = 0; i < n; ++i) {
        if (numel[i] == 0) continue;
        const Span both[] = {{p, bytes}, {grads[i], (size_t)numel[i] * (dtype[i] == MOONEP_GRAD_BF16 ? 2 : 4)}};
        if (outputs_overlap(both, 1, 2)) return true;
    }
    return false;
}

}  // namespace moonep

using namespace moonep;

extern "C" size_t moonep_grad_norm_workspace_bytes(int32_t n) {
    if (n < 0) return 0;
    return (size_t)((n + (int64_t)kTable - 1) / kTable + (n == 0)) * kNormBlocks * sizeof(double);
}

extern "C" int moonep_grad_norm(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* dtype,
                                void* ws, float* norm, void* stream) {
    int rc = check_grads(n, grads, numel, dtype);
    if (rc != MOONEP_OK) return rc;
    MOONEP_CHECK_PTR(ws);
    MOONEP_CHECK_PTR(norm);
    if (touches(n, grads, numel, dtype, ws, moonep_grad_norm_workspace_bytes(n)) ||
        touches(n, grads, numel, dtype, norm, sizeof(float)))
        return MOONEP_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    double* part = static_cast<double*>(ws);
    const bool stream_past = streams(n, numel, dtype);
    int parts = 0;
    rc = for_tables(n, grads, numel, dtype, [&](const GradTable& t, int blocks) {
        if (stream_past) hipLaunchKernelGGL(grad_squares_kernel<true>, dim3(blocks), dim3(256), 0, s, t, part + parts);
        else hipLaunchKernelGGL(grad_squares_kernel<false>, dim3(blocks), dim3(256), 0, s, t, part + parts);
        parts += blocks;
    });
    if (rc != MOONEP_OK) return rc;
    hipLaunchKernelGGL(grad_join_kernel, dim3(1), dim3(256), 0, s, part, parts, norm);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

extern "C" int moonep_grad_clip(int32_t n, void* const* grads, const int64_t* numel, const int32_t* dtype,
                                const float* norm, float max_norm, void* stream) {
    const int rc = check_grads(n, grads, numel, dtype);
    if (rc != MOONEP_OK) return rc;
    if (!(max_norm >= 0.0f)) return MOONEP_EINVAL;
    MOONEP_CHECK_PTR(norm);
    if (touches(n, grads, numel, dtype, norm, sizeof(float))) return MOONEP_EINVAL;   // read by all, written by one
    try {
        if (overlap(n, grads, numel, dtype)) return MOONEP_EINVAL;
    } catch (...) {                  // no memory for the list of a host that has none left
        return MOONEP_EINVAL;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool stream_past = streams(n, numel, dtype);
    return for_tables(n, grads, numel, dtype, [&](const GradTable& t, int blocks) {
        if (stream_past) hipLaunchKernelGGL(grad_clip_kernel<true>, dim3(blocks), dim3(256), 0, s, t, norm, max_norm);
        else hipLaunchKernelGGL(grad_clip_kernel<false>, dim3(blocks), dim3(256), 0, s, t, norm, max_norm);
    });
}
