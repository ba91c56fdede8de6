// Layer norm in front of the MoE layer, forward and backward.
//
//   forward   m = avg(x), v = avg((x - m)^2), rstd = 1 / sqrt(v + eps), y = (x - m) rstd w + b
//   backward  n = (x - m) rstd, g = dy w:  dx = rstd (g - avg(g) - n avg(g n));
//             dw = sum over rows of dy n, db = sum over rows of dy
#include "common.h"

#include <cmath>

namespace moonep {

// ---------------------------------------------------------------------------
// 16-byte vectors of a row as float32
// ---------------------------------------------------------------------------

template <bool F32>
struct RowVec {
    static constexpr int N = F32 ? 4 : 8;   // elements in 16 bytes
};

template <bool F32>
__device__ __forceinline__ void unpack_row(uint4 v, float* f) {
    if constexpr (F32) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    } else {
        f[0] = bf16_lo(v.x);
        f[1] = bf16_hi(v.x);
        f[2] = bf16_lo(v.y);
        f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z);
        f[5] = bf16_hi(v.z);
        f[6] = bf16_lo(v.w);
        f[7] = bf16_hi(v.w);
    }
}

template <bool F32>
__device__ __forceinline__ uint4 pack_row(const float* f) {
    if constexpr (F32)
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
        return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// f[0..N) = p[v * N ..), or `none` where p is NULL
template <int N>
__device__ __forceinline__ void load_param(const float* p, int v, float none, float* f) {
    const float4* q = reinterpret_cast<const float4*>(p) + (size_t)v * (N / 4);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 a = p ? q[i / 4] : make_float4(none, none, none, none);
        f[i] = a.x;
        f[i + 1] = a.y;
        f[i + 2] = a.z;
        f[i + 3] = a.w;
    }
}

// Sum over a workgroup of 256, in every thread.
__device__ __forceinline__ float block_sum(float v, float* lds) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// One workgroup per row; the row is read three times (from L2 after the first).
template <bool F32>
__global__ __launch_bounds__(256) void norm_rows_kernel(const uint4* __restrict__ x, const float* __restrict__ w,
                                                        const float* __restrict__ b, uint4* __restrict__ y,
                                                        float* __restrict__ mean, float* __restrict__ rstd, int nv,
                                                        float eps) {
    constexpr int N = RowVec<F32>::N;
    __shared__ float lds[4];
    const uint4* xr = x + (size_t)blockIdx.x * nv;
    const float n = (float)nv * N;     // divided by, so that a constant row has its value as the mean
    float f[N], s = 0.0f;
    for (int v = threadIdx.x; v < nv; v += 256) {
        unpack_row<F32>(xr[v], f);
#pragma unroll
        for (int i = 0; i < N; ++i) s += f[i];
    }
    const float m = block_sum(s, lds) / n;
    s = 0.0f;
    for (int v = threadIdx.x; v < nv; v += 256) {
        unpack_row<F32>(xr[v], f);
#pragma unroll
        for (int i = 0; i < N; ++i) s += (f[i] - m) * (f[i] - m);
    }
    const float r = 1.0f / sqrtf(block_sum(s, lds) / n + eps);
    for (int v = threadIdx.x; v < nv; v += 256) {
        float wf[N], bf[N];
        unpack_row<F32>(xr[v], f);
        load_param<N>(w, v, 1.0f, wf);
        load_param<N>(b, v, 0.0f, bf);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = (f[i] - m) * r * wf[i] + bf[i];
        y[(size_t)blockIdx.x * nv + v] = pack_row<F32>(f);
    }
    if (mean && threadIdx.x == 0) {
        mean[blockIdx.x] = m;
        rstd[blockIdx.x] = r;
    }
}

// dx of one row per workgroup; both rows are read twice.
template <bool F32>
__global__ __launch_bounds__(256) void norm_dx_rows_kernel(const uint4* __restrict__ dy, const uint4* __restrict__ x,
                                                           const float* __restrict__ w, const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, uint4* __restrict__ dx,
                                                           int nv) {
    constexpr int N = RowVec<F32>::N;
    __shared__ float lds[4];
    const size_t row = (size_t)blockIdx.x * nv;
    const float n = (float)nv * N;     // divided by, so that a constant row has its value as the mean
    const float m = mean[blockIdx.x], r = rstd[blockIdx.x];
    float sg = 0.0f, sgn = 0.0f, f[N], d[N], wf[N];
    for (int v = threadIdx.x; v < nv; v += 256) {
        unpack_row<F32>(x[row + v], f);
        unpack_row<F32>(dy[row + v], d);
        load_param<N>(w, v, 1.0f, wf);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float g = d[i] * wf[i];
            sg += g;
            sgn += g * ((f[i] - m) * r);
        }
    }
    const float c1 = block_sum(sg, lds) / n;
    const float c2 = block_sum(sgn, lds) / n;
    for (int v = threadIdx.x; v < nv; v += 256) {
        unpack_row<F32>(x[row + v], f);
        unpack_row<F32>(dy[row + v], d);
        load_param<N>(w, v, 1.0f, wf);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = r * (d[i] * wf[i] - c1 - (f[i] - m) * r * c2);
        dx[row + v] = pack_row<F32>(f);
    }
}

// Partial sums over a share of the rows: ws[split][0] = sum dy n, ws[split][1] = sum dy, per column.
template <bool F32>
__global__ __launch_bounds__(256) void norm_dw_cols_kernel(const uint4* __restrict__ dy, const uint4* __restrict__ x,
                                                           const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, float* __restrict__ ws,
                                                           int rows, int nv) {
    constexpr int N = RowVec<F32>::N;
    const int v = blockIdx.x * 256 + threadIdx.x;
    if (v >= nv) return;
    float aw[N] = {}, ab[N] = {}, f[N], d[N];
    for (int t = blockIdx.y; t < rows; t += gridDim.y) {
        unpack_row<F32>(x[(size_t)t * nv + v], f);
        unpack_row<F32>(dy[(size_t)t * nv + v], d);
        const float m = mean[t], r = rstd[t];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            aw[i] += d[i] * ((f[i] - m) * r);
            ab[i] += d[i];
        }
    }
    const size_t H = (size_t)nv * N;
    float* o = ws + (size_t)blockIdx.y * 2 * H + (size_t)v * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        o[i] = aw[i];
        o[H + i] = ab[i];
    }
}

// Joins the partial sums of `splits` shares, one column per thread.
__global__ __launch_bounds__(256) void norm_dw_join_kernel(const float* __restrict__ ws, float* __restrict__ dw,
                                                           float* __restrict__ db, int splits, int H, int accum) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    float* out = blockIdx.y == 0 ? dw : db;
    if (c >= H || !out) return;
    const float* p = ws + (size_t)blockIdx.y * H + c;
    float s = 0.0f;
    for (int i = 0; i < splits; ++i) s += p[(size_t)i * 2 * H];
    out[c] = accum ? out[c] + s : s;
}

// Shares of the rows whose sums the backward joins.
static int norm_splits(const moonep_dims_t* d) { return std::min(d->R * d->S, 512); }

}  // namespace moonep

using namespace moonep;

extern "C" int moonep_layer_norm(const moonep_dims_t* dims, const void* x, const float* weight, const float* bias,
                                 float eps, void* y, float* mean, float* rstd, void* stream) {
    const int rc = check_dims(dims, false);
    if (rc != MOONEP_OK) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps) || !mean != !rstd) return MOONEP_EINVAL;
    MOONEP_CHECK_PTR(x);
    MOONEP_CHECK_PTR(y);
    if (!aligned16(weight) || !aligned16(bias) || !aligned16(mean) || !aligned16(rstd)) return MOONEP_EALIGN;
    const bool f32 = (dims->flags & MOONEP_F32_ROWS) != 0;
    const int nv = dims->H / (f32 ? 4 : 8);
    const dim3 grid(dims->R * dims->S);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint4* xv = static_cast<const uint4*>(x);
    uint4* yv = static_cast<uint4*>(y);
    if (f32) hipLaunchKernelGGL(norm_rows_kernel<true>, grid, dim3(256), 0, s, xv, weight, bias, yv, mean, rstd, nv, eps);
    else hipLaunchKernelGGL(norm_rows_kernel<false>, grid, dim3(256), 0, s, xv, weight, bias, yv, mean, rstd, nv, eps);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

extern "C" size_t moonep_layer_norm_workspace_bytes(const moonep_dims_t* dims) {
    if (check_dims(dims, false) != MOONEP_OK) return 0;
    return (size_t)norm_splits(dims) * 2 * dims->H * sizeof(float);
}

extern "C" int moonep_layer_norm_backward(const moonep_dims_t* dims, const void* dy, const void* x,
                                          const float* weight, const float* mean, const float* rstd, void* dx,
                                          float* dweight, float* dbias, void* ws, void* stream) {
    const int rc = check_dims(dims, false);
    if (rc != MOONEP_OK) return rc;
    MOONEP_CHECK_PTR(dy);
    MOONEP_CHECK_PTR(x);
    MOONEP_CHECK_PTR(mean);
    MOONEP_CHECK_PTR(rstd);
    MOONEP_CHECK_PTR(dx);
    if (!aligned16(weight) || !aligned16(dweight) || !aligned16(dbias)) return MOONEP_EALIGN;
    const bool sums = dweight || dbias;
    if (sums) MOONEP_CHECK_PTR(ws);
    const bool f32 = (dims->flags & MOONEP_F32_ROWS) != 0;
    const int rows = dims->R * dims->S, nv = dims->H / (f32 ? 4 : 8);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint4 *dv = static_cast<const uint4*>(dy), *xv = static_cast<const uint4*>(x);
    uint4* ov = static_cast<uint4*>(dx);
    if (f32) hipLaunchKernelGGL(norm_dx_rows_kernel<true>, dim3(rows), dim3(256), 0, s, dv, xv, weight, mean, rstd, ov, nv);
    else hipLaunchKernelGGL(norm_dx_rows_kernel<false>, dim3(rows), dim3(256), 0, s, dv, xv, weight, mean, rstd, ov, nv);
    MOONEP_LAUNCH_CHECK();
    if (!sums) return MOONEP_OK;
    const int splits = norm_splits(dims);
    const dim3 grid((nv + 255) / 256, splits);
    float* wsf = static_cast<float*>(ws);
    if (f32) hipLaunchKernelGGL(norm_dw_cols_kernel<true>, grid, dim3(256), 0, s, dv, xv, mean, rstd, wsf, rows, nv);
    else hipLaunchKernelGGL(norm_dw_cols_kernel<false>, grid, dim3(256), 0, s, dv, xv, mean, rstd, wsf, rows, nv);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(norm_dw_join_kernel, dim3((dims->H + 255) / 256, 2), dim3(256), 0, s, wsf, dweight, dbias,
                       splits, dims->H, (dims->flags & MOONEP_GRAD_ACCUM) != 0);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}
