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
// What bounds it is ranking.  Without a bias each lane sorts its best K and the K heads are compared across lanes:
// 32768 rows of 256 float32 take 11.5 us for K 8 and 16.0 for K 16 in a graph with logits from memory, of which reading
// them is 5 to 6 (9.7 and 13.3 where the last-level cache holds them); K times a maximum over all elements took 17.1
// and 25.5.  With a bias keys are doubles and are ranked that way, and a sigmoid in float64 comes before it: 33 to 37 us.
//
// Sixteen lanes share a row, so that four rows go through a wave and every step across lanes is a rotation
// inside 16 lanes, an operand modifier instead of an instruction through LDS.  Where rows are too few to fill the
// chip, all 64 lanes share one: a quarter of the elements to rank for two more steps (one token over 256 experts,
// with a bias: 10.5 us a call, with 64 lanes 7.0, which is what the host needs for it).  A lane's elements are groups of
// VEC side by side, the lanes' groups next to each other, so that a load of the lanes is one piece of the row.
#include "common.h"

namespace moonep {

constexpr int kRouteThreads = 256;
// Up to so many rows get 64 lanes each (16 lanes / 64, us, E 256, K 8): 1024 rows 3.4 / 3.3 and 2048 3.4 / 3.8; with a
// bias 1024 rows 10.3 / 5.5 and 4096 11.5 / 10.0, backward 4.0 / 3.3 and 4.9 / 4.9.
constexpr int kWideRows = 1024, kWideSlowRows = 4096;

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
template <int N>
__device__ __forceinline__ double turned(double v) {
    return __longlong_as_double(turned<N>((uint64_t)__double_as_longlong(v)));
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

// Without a bias a logit and its id make one number, so that one comparison ranks both: a double from 1 up to 2
// with the logit's 32 bits in order and then kMaxE - 1 - id in the 52 bits of its fraction, which the maximum of two doubles
// orders as it does integers.  (Doubles because one instruction takes the larger of two, and none does of 64-bit
// integers.)
constexpr double kNoPick = 1.0, kNoKey = -0x1p200;
static_assert(kMaxE == 1 << 10, "32 bits of a logit and 10 of its id");
__device__ __forceinline__ double ranked(float v, int id) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t key = v != v ? 0xffffffffu : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    const uint32_t hi = __builtin_amdgcn_alignbit(0x3ffu, key, 12), lo = (key << 20) + (kMaxE - 1 - id);
    return __longlong_as_double((uint64_t)hi << 32 | lo);
}
// -1 for what is no pick: -inf and less
__device__ __forceinline__ int ranked_id(double v) {
    const uint64_t u = __double_as_longlong(v);
    return (u >> 43 & 0x1ff) != 0 ? kMaxE - 1 - (int)(u & (kMaxE - 1)) : -1;
}
// No operand is NaN.  (fmax and fmin quiet NaN in an instruction of their own, for most operands here.)
__device__ __forceinline__ double larger(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double smaller(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
// The same for results that move to other lanes: two wait states before that.
__device__ __forceinline__ double larger_to_move(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2\n\ts_nop 1" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ void larger_first(double& a, double& b) {
    const double m = larger(a, b);
    b = smaller(a, b);
    a = m;
}

// Comparisons that sort N values (Batcher's odd-even merges).
template <int N>
struct Network {
    int n = 0, a[N * 4] = {}, b[N * 4] = {};
    constexpr Network() {
        for (int p = 1; p < N; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < N; j += 2 * k)
                    for (int i = 0; i < k && i + j + k < N; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            a[n] = i + j;
                            b[n++] = i + j + k;
                        }
    }
};

// The D best of a lane's NE elements, best first: D at a time sorted, and joined with the best so far, of which
// the element-wise larger ones against the others backwards are the D best, in an order that log D steps sort.
template <int LANES, int NE, int VEC, int D>
__device__ __forceinline__ void lane_best(double (&best)[D], const float (&x)[NE], int lane) {
    constexpr Network<D> net;
#pragma unroll
    for (int c = 0; c < NE; c += D) {
        double v[D];
#pragma unroll
        for (int i = 0; i < D; ++i) v[i] = ranked(x[c + i], index_of<LANES, VEC>(c + i, lane));
#pragma unroll
        for (int i = 0; i < net.n; ++i) larger_first(v[net.a[i]], v[net.b[i]]);
        if (c == 0) {
#pragma unroll
            for (int i = 0; i < D; ++i) best[i] = v[i];
            continue;
        }
#pragma unroll
        for (int i = 0; i < D; ++i) best[i] = larger(best[i], v[D - 1 - i]);
#pragma unroll
        for (int step = D / 2; step > 0; step /= 2)
#pragma unroll
            for (int i = 0; i < D; ++i)
                if ((i & step) == 0) larger_first(best[i], best[i + step]);
    }
}

// Pick k, and the MOVES first of the lane's others if it was its own.
template <int LANES, int MOVES, int D>
__device__ __forceinline__ void next_pick(double (&best)[D], double& pick, int k, int lane) {
    const double top = over_row<LANES>(best[0], larger_to_move);
    if (lane == k) pick = top;
    const bool own = best[0] == top;
#pragma unroll
    for (int i = 0; i < MOVES; ++i)
        best[i] = own ? i + 1 < D ? best[i + 1] : kNoPick : best[i];
}
// Picks k .. K of up to KM, each moving what later ones can need.
template <int LANES, int KM, int k, int D>
__device__ __forceinline__ void next_picks(double (&best)[D], double& pick, int K, int lane) {
    if (k >= K) return;
    next_pick<LANES, KM - 1 - k < D ? KM - 1 - k : D>(best, pick, k, lane);
    if constexpr (k + 1 < KM) next_picks<LANES, KM, k + 1>(best, pick, K, lane);
}

// KM: without a bias, K at most; 0 with one.
template <class T, int LANES, int NE, int VEC, int KM>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x % LANES, row = blockIdx.x * (kRouteThreads / LANES) + threadIdx.x / LANES;
    if (row >= a.T) return;
    const T* logits = static_cast<const T*>(a.logits) + (size_t)row * a.E;
    float x[NE];
    load_row<LANES, NE, VEC>(x, logits, a.E, lane);
    int mine = -1;                   // the expert of pick `lane`
    if constexpr (KM > 0) {
        constexpr int D = NE < KM ? NE : KM;
        double best[D];
        lane_best<LANES, NE, VEC, D>(best, x, lane);
        asm("s_nop 1" : "+v"(best[0]));
        double pick = kNoPick;
        next_picks<LANES, KM, 0>(best, pick, a.K, lane);
        mine = ranked_id(pick);
    } else {
        // finite keys are below 2^130: infinity and NaN are larger ones, so that all are numbers.  What either -inf takes
        // out is none of these, though the sum with a logit that is not finite is NaN.
        double key[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = index_of<LANES, VEC>(i, lane);
            const float b = e < a.E ? a.bias[e] : 0.0f;
            const bool out = x[i] == -__builtin_inff() || b == -__builtin_inff();
            const double v = (a.mode == MOONEP_ROUTE_SIGMOID ? 1.0 / (1.0 + exp(-(double)x[i])) : (double)x[i]) + b;
            key[i] = out ? kNoKey : v != v ? 0x1p201 : fmin(fmax(v, kNoKey), 0x1p200);
        }
        for (int k = 0; k < a.K; ++k) {      // first the largest key, then the lowest of the ids that have it
            double best = key[0];
#pragma unroll
            for (int i = 1; i < NE; ++i) best = larger(best, key[i]);
            asm("s_nop 1" : "+v"(best));
            const double top = over_row<LANES>(best, larger_to_move);
            uint32_t at = 0x7fffffffu;
#pragma unroll
            for (int i = NE - 1; i >= 0; --i)
                if (key[i] == top) at = index_of<LANES, VEC>(i, lane);
            const uint32_t id = over_row<LANES>(at, [](uint32_t p, uint32_t q) { return p < q ? p : q; });
            if (lane == k && top != kNoKey) mine = (int)id;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (index_of<LANES, VEC>(i, lane) == (int)id) key[i] = kNoKey;
        }
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
    if ((int64_t)d->R * d->S > 1 << 27) return MOONEP_ENOTSUP;      // 16 lanes a row: fewer than 2^32 in a launch
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
        hipLaunchKernelGGL((route_kernel<T, LANES, NE, VEC, 0>), grid, dim3(kRouteThreads), 0, s, a);
    else if (a.K <= 8)
        hipLaunchKernelGGL((route_kernel<T, LANES, NE, VEC, 8>), grid, dim3(kRouteThreads), 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<T, LANES, NE, VEC, 16>), grid, dim3(kRouteThreads), 0, s, a);
}

template <class T, int VEC, bool BACK>
static void route_sizes(const RouteArgs& a, hipStream_t s) {
    if (a.T <= (BACK || a.bias ? kWideSlowRows : kWideRows)) {
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
