// The router's top K and its gates, forward and backward.
//
// A row is one token's logits over E experts.  Ranked by a key (the logit, or with a bias the logit or its
// sigmoid plus the bias in float64), the K largest are its experts, equal keys to the lower id.  With p a
// softmax over the picked logits (of their log-sigmoids in sigmoid mode), or over the row:
//   gates g_k = scale * p_k;
//   dlogit of a pick = scale * p_k * (dg_k - sum_i p_i dg_i)          times (1 - sigmoid) in sigmoid mode;
//   over the whole row: dlogit_e = scale * ([e picked] p_e dg_e - p_e sum_i p_i dg_i).
// A sum of sigmoids that underflows is no division by zero this way: s_k / sum s = softmax(log s)_k.
//
// Sixteen lanes share a row, so that four rows go through a wave and every step across lanes is a rotation
// inside 16 lanes, an operand modifier instead of an instruction through LDS.  Where rows are too few to fill the
// chip, all 64 lanes share one: a quarter of the elements to rank for two more steps (one token over 256 experts,
// with a bias: 10.5 us, with 64 lanes 7.6, which is what the host needs for a call).  A lane's elements are groups of
// VEC side by side, the lanes' groups next to each other, so that a load of the lanes is one piece of the row.
#include <type_traits>

#include "common.h"

namespace moonep {

constexpr int kRouteThreads = 256;
constexpr int kWideRows = 4096;      // up to here a row gets 64 lanes

struct RouteArgs {
    const void* logits;              // [T, E]
    const float* bias;               // [E] or NULL
    int32_t* topk;                   // [T, K]
    float* gates;                    // [T, K]
    const float* dgates;             // [T, K]
    void* dlogits;                   // [T, E]
    int T, E, K, mode;
    float scale;
};

// v of the lane N places further round in its 16
template <int N>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, true);
}
template <int N>
__device__ __forceinline__ float turned(float v) {
    return __uint_as_float(turned<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ uint64_t turned(uint64_t v) {
    return (uint64_t)turned<N>((uint32_t)(v >> 32)) << 32 | turned<N>((uint32_t)v);
}

// a of the lanes of a row with a's lane STEP places away (16 and 32 lanes: halves and quarters of the wave change places)
template <class T, class F>
__device__ __forceinline__ T with_quarters(T v, F f) {
    union {
        T t;
        uint32_t u[sizeof(T) / 4];
    } a, b;
    a.t = b.t = v;
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 4; ++i) {
        const auto r = __builtin_amdgcn_permlane16_swap(a.u[i], b.u[i], false, false);
        a.u[i] = r[0];
        b.u[i] = r[1];
    }
    v = f(a.t, b.t);
    a.t = b.t = v;
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 4; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(a.u[i], b.u[i], false, false);
        a.u[i] = r[0];
        b.u[i] = r[1];
    }
    return f(a.t, b.t);
}

// f over the lanes of a row, in each of them.  Each step joins the same pairs in every lane, and f is
// commutative, so that all lanes agree where f rounds, too.
template <int LANES, class T, class F>
__device__ __forceinline__ T over_row(T v, F f) {
    v = f(v, turned<8>(v));
    v = f(v, turned<4>(v));
    v = f(v, turned<2>(v));
    v = f(v, turned<1>(v));
    if constexpr (LANES == 64) v = with_quarters(v, f);
    return v;
}
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
    return over_row<LANES>(v, [](float a, float b) { return a + b; });
}
template <int LANES>
__device__ __forceinline__ float row_max(float v) {
    return over_row<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}

__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ float element(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// A lane's elements of a row: element VEC * v + i is number (v * LANES + lane) * VEC + i of the row;
// -inf past its end.
template <int LANES, int NE, int VEC, class T>
__device__ __forceinline__ void load_row(float (&x)[NE], const T* row, int E, int lane) {
#pragma unroll
    for (int v = 0; v < NE / VEC; ++v) {
        const int e = (v * LANES + lane) * VEC;
        if constexpr (VEC == 4 && sizeof(T) == 4) {
            const float inf = -__builtin_inff();
            const float4 f = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(inf, inf, inf, inf);
            x[v * 4] = f.x, x[v * 4 + 1] = f.y, x[v * 4 + 2] = f.z, x[v * 4 + 3] = f.w;
        } else if constexpr (VEC == 4) {
            const uint2 u = e < E ? *reinterpret_cast<const uint2*>(row + e) : make_uint2(0xff80ff80u, 0xff80ff80u);
            x[v * 4] = bf16_lo(u.x), x[v * 4 + 1] = bf16_hi(u.x), x[v * 4 + 2] = bf16_lo(u.y), x[v * 4 + 3] = bf16_hi(u.y);
        } else {
            x[v] = e < E ? element(row + e) : -__builtin_inff();
        }
    }
}
template <int LANES, int VEC>
__device__ __forceinline__ int index_of(int i, int lane) {
    return (i / VEC * LANES + lane) * VEC + i % VEC;
}

// Order-preserving keys: larger for larger values, largest for NaN of either sign, 0 for -inf (no expert).
// Zeros of both signs are one value.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    if (v != v) return 0xffffffffu;
    if (v == -__builtin_inff()) return 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t u = __double_as_longlong(v + 0.0);
    if (v != v) return ~0ull;
    if (v == -__builtin_inf()) return 0;
    return u >> 63 ? ~u : u | 1ull << 63;
}

// log(sigmoid(v)): no underflow for v far below zero
__device__ __forceinline__ float log_sigmoid(float v) { return fminf(v, 0.0f) - log1pf(expf(-fabsf(v))); }

// p of a row's picks, lane k that of pick k (0 where `here` is false); w is the picked logit or what stands
// for it.  `top` and `total` are over the whole row in SOFTMAX_ALL.
template <int LANES>
__device__ __forceinline__ float picked_share(float w, bool here, bool all, float top, float total) {
    if (!all) {
        top = row_max<LANES>(here ? w : -__builtin_inff());
        total = row_sum<LANES>(here ? expf(w - top) : 0.0f);
    }
    return here ? expf(w - top) / total : 0.0f;
}

// Row maximum and sum of exp(x - maximum) over all of the row's elements.
template <int LANES, int NE>
__device__ __forceinline__ void row_softmax(const float (&x)[NE], float& top, float& total) {
    top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NE; ++i) top = fmaxf(top, x[i]);
    top = row_max<LANES>(top);
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) total += x[i] == -__builtin_inff() ? 0.0f : expf(x[i] - top);
    total = row_sum<LANES>(total);
}

template <class T, int LANES, int NE, int VEC, bool BIAS>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    using Key = std::conditional_t<BIAS, uint64_t, uint32_t>;
    const int lane = threadIdx.x % LANES, row = blockIdx.x * (kRouteThreads / LANES) + threadIdx.x / LANES;
    if (row >= a.T) return;
    const T* logits = static_cast<const T*>(a.logits) + (size_t)row * a.E;
    float x[NE];
    load_row<LANES, NE, VEC>(x, logits, a.E, lane);
    Key key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        if constexpr (BIAS) {
            const int e = index_of<LANES, VEC>(i, lane);
            const double b = e < a.E ? a.bias[e] : 0.0f;
            const double v = a.mode == MOONEP_ROUTE_SIGMOID ? 1.0 / (1.0 + exp(-(double)x[i])) : (double)x[i];
            key[i] = x[i] == -__builtin_inff() ? 0 : key_of(v + b);
        } else {
            key[i] = key_of(x[i]);
        }
    }
    int mine = -1;                   // the expert of pick `lane`
    for (int k = 0; k < a.K; ++k) {
        Key best = 0;                // first the largest key, then the lowest of the ids that have it
#pragma unroll
        for (int i = 0; i < NE; ++i) best = key[i] > best ? key[i] : best;
        const Key top = over_row<LANES>(best, [](Key p, Key q) { return p > q ? p : q; });
        uint32_t at = 0x7fffffffu;
#pragma unroll
        for (int i = NE - 1; i >= 0; --i)
            if (key[i] == top) at = index_of<LANES, VEC>(i, lane);
        const uint32_t id = over_row<LANES>(at, [](uint32_t p, uint32_t q) { return p < q ? p : q; });
        if (lane == k && top != 0) mine = (int)id;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (index_of<LANES, VEC>(i, lane) == (int)id) key[i] = 0;
    }
    const bool here = mine >= 0, all = a.mode == MOONEP_ROUTE_SOFTMAX_ALL;
    float w = here ? element(logits + mine) : 0.0f, top = 0.0f, total = 0.0f;
    if (a.mode == MOONEP_ROUTE_SIGMOID) w = log_sigmoid(w);
    if (all) row_softmax<LANES>(x, top, total);
    const float p = picked_share<LANES>(w, here, all, top, total);
    if (lane < a.K) {
        a.topk[(size_t)row * a.K + lane] = mine;
        a.gates[(size_t)row * a.K + lane] = here ? a.scale * p : 0.0f;
    }
}

template <class T, int LANES, int NE, int VEC>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a) {
    const int lane = threadIdx.x % LANES, row = blockIdx.x * (kRouteThreads / LANES) + threadIdx.x / LANES;
    if (row >= a.T) return;
    const T* logits = static_cast<const T*>(a.logits) + (size_t)row * a.E;
    const bool all = a.mode == MOONEP_ROUTE_SOFTMAX_ALL;
    int id = -1;
    float dg = 0.0f;
    if (lane < a.K) {
        id = a.topk[(size_t)row * a.K + lane];
        dg = a.dgates[(size_t)row * a.K + lane];
    }
    const bool here = (unsigned)id < (unsigned)a.E;
    if (!here) id = -1, dg = 0.0f;
    const float l = here ? element(logits + id) : 0.0f;
    float x[NE], top = 0.0f, total = 0.0f;
    if (all) {
        load_row<LANES, NE, VEC>(x, logits, a.E, lane);
        row_softmax<LANES>(x, top, total);
    }
    const float p = picked_share<LANES>(a.mode == MOONEP_ROUTE_SIGMOID ? log_sigmoid(l) : l, here, all, top, total);
    const float dot = row_sum<LANES>(here ? p * dg : 0.0f);
    // the picks' own part
    float d = all ? p * dg : p * (dg - dot);
    if (a.mode == MOONEP_ROUTE_SIGMOID) d *= 1.0f / (1.0f + expf(l));
    if (!here) d = 0.0f;
    const bool any = row_max<LANES>(here ? 1.0f : 0.0f) > 0.0f;
    float g[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i)
        g[i] = all && any && x[i] != -__builtin_inff() ? -(expf(x[i] - top) / total) * dot : 0.0f;
    for (int k = 0; k < a.K; ++k) {  // an id that is named twice gets both, in this order
        const int to = __shfl(id, k, LANES);
        const float v = __shfl(d, k, LANES);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (index_of<LANES, VEC>(i, lane) == to) g[i] += v;
    }
    T* out = static_cast<T*>(a.dlogits) + (size_t)row * a.E;
#pragma unroll
    for (int v = 0; v < NE / VEC; ++v) {
        const int e = (v * LANES + lane) * VEC;
        if (e >= a.E) continue;
        if constexpr (VEC == 4 && sizeof(T) == 4) {
            *reinterpret_cast<float4*>(out + e) =
                make_float4(a.scale * g[v * 4], a.scale * g[v * 4 + 1], a.scale * g[v * 4 + 2], a.scale * g[v * 4 + 3]);
        } else if constexpr (VEC == 4) {
            *reinterpret_cast<uint2*>(out + e) = make_uint2(pack_bf16(a.scale * g[v * 4], a.scale * g[v * 4 + 1]),
                                                            pack_bf16(a.scale * g[v * 4 + 2], a.scale * g[v * 4 + 3]));
        } else if constexpr (sizeof(T) == 4) {
            out[e] = a.scale * g[v];
        } else {
            out[e] = (uint16_t)pack_bf16(a.scale * g[v], 0.0f);
        }
    }
}

constexpr uint32_t kRouteModes = 3, kRouteBits = kRouteModes | MOONEP_ROUTE_BF16;

static int check_route(const moonep_dims_t* d, uint32_t mode, float scale) {
    if (!d || (mode & ~kRouteBits) || (mode & kRouteModes) > MOONEP_ROUTE_SIGMOID) return MOONEP_EINVAL;
    if (check_flags(d) != MOONEP_OK) return MOONEP_EINVAL;
    if (d->R < 1 || d->R > kMaxR || d->S < 1 || d->E < 1 || d->E > kMaxE) return MOONEP_EINVAL;
    if (d->K < 1 || d->K > kMaxK || d->K > d->E) return MOONEP_EINVAL;
    if ((int64_t)d->R * d->S * d->K > (int64_t)1 << 30) return MOONEP_EINVAL;
    if (!(scale > -__builtin_inff() && scale < __builtin_inff())) return MOONEP_EINVAL;
    return MOONEP_OK;
}

template <class T, int LANES, int NE, int VEC, bool BACK>
static void launch_route(const RouteArgs& a, hipStream_t s) {
    constexpr int rows = kRouteThreads / LANES;
    const dim3 grid((a.T + rows - 1) / rows);
    if constexpr (BACK)
        hipLaunchKernelGGL((route_backward_kernel<T, LANES, NE, VEC>), grid, dim3(kRouteThreads), 0, s, a);
    else if (a.bias)
        hipLaunchKernelGGL((route_kernel<T, LANES, NE, VEC, true>), grid, dim3(kRouteThreads), 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<T, LANES, NE, VEC, false>), grid, dim3(kRouteThreads), 0, s, a);
}

template <class T, int VEC, bool BACK>
static void route_sizes(const RouteArgs& a, hipStream_t s) {
    if (a.T <= kWideRows) {
        if (a.E <= 4 * 64) launch_route<T, 64, 4, VEC, BACK>(a, s);
        else if (a.E <= 8 * 64) launch_route<T, 64, 8, VEC, BACK>(a, s);
        else launch_route<T, 64, 16, VEC, BACK>(a, s);
    } else {
        if (a.E <= 4 * 16) launch_route<T, 16, 4, VEC, BACK>(a, s);
        else if (a.E <= 8 * 16) launch_route<T, 16, 8, VEC, BACK>(a, s);
        else if (a.E <= 16 * 16) launch_route<T, 16, 16, VEC, BACK>(a, s);
        else if (a.E <= 32 * 16) launch_route<T, 16, 32, VEC, BACK>(a, s);
        else launch_route<T, 16, 64, VEC, BACK>(a, s);
    }
}

// Rows of a multiple of four logits start where a load of four does.
template <bool BACK>
static void route_types(const RouteArgs& a, bool bf16, hipStream_t s) {
    if (bf16) {
        if (a.E % 4 == 0) route_sizes<uint16_t, 4, BACK>(a, s);
        else route_sizes<uint16_t, 1, BACK>(a, s);
    } else {
        if (a.E % 4 == 0) route_sizes<float, 4, BACK>(a, s);
        else route_sizes<float, 1, BACK>(a, s);
    }
}

}  // namespace moonep

using namespace moonep;

extern "C" int moonep_route(const moonep_dims_t* dims, uint32_t mode, float scale, const void* logits,
                            const float* bias, int32_t* topk, float* gates, void* stream) {
    const int rc = check_route(dims, mode, scale);
    if (rc != MOONEP_OK) return rc;
    MOONEP_CHECK_PTR(logits);
    if (bias && !aligned16(bias)) return MOONEP_EALIGN;
    MOONEP_CHECK_PTR(topk);
    MOONEP_CHECK_PTR(gates);
    const size_t rows = (size_t)dims->R * dims->S, picks = rows * dims->K * 4;
    const bool bf16 = mode & MOONEP_ROUTE_BF16;
    const Span spans[] = {{topk, picks}, {gates, picks}, {logits, rows * dims->E * (bf16 ? 2 : 4)}, {bias, dims->E * 4u}};
    if (outputs_overlap(spans, 2, 4)) return MOONEP_EINVAL;
    RouteArgs a{};
    a.logits = logits, a.bias = bias, a.topk = topk, a.gates = gates;
    a.T = (int)rows, a.E = dims->E, a.K = dims->K, a.mode = mode & kRouteModes, a.scale = scale;
    route_types<false>(a, bf16, static_cast<hipStream_t>(stream));
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

extern "C" int moonep_route_backward(const moonep_dims_t* dims, uint32_t mode, float scale, const float* dgates,
                                     const void* logits, const int32_t* topk, void* dlogits, void* stream) {
    const int rc = check_route(dims, mode, scale);
    if (rc != MOONEP_OK) return rc;
    MOONEP_CHECK_PTR(dgates);
    MOONEP_CHECK_PTR(logits);
    MOONEP_CHECK_PTR(topk);
    MOONEP_CHECK_PTR(dlogits);
    const size_t rows = (size_t)dims->R * dims->S, picks = rows * dims->K * 4;
    const bool bf16 = mode & MOONEP_ROUTE_BF16;
    const size_t all = rows * dims->E * (bf16 ? 2 : 4);
    const Span spans[] = {{dlogits, all}, {dgates, picks}, {logits, all}, {topk, picks}};
    if (outputs_overlap(spans, 1, 4)) return MOONEP_EINVAL;
    RouteArgs a{};
    a.logits = logits, a.topk = const_cast<int32_t*>(topk), a.dgates = dgates, a.dlogits = dlogits;
    a.T = (int)rows, a.E = dims->E, a.K = dims->K, a.mode = mode & kRouteModes, a.scale = scale;
    route_types<true>(a, bf16, static_cast<hipStream_t>(stream));
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}
