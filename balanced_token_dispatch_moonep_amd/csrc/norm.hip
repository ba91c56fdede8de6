// Layer norm in front of the MoE layer, forward and backward.
//
//   forward   m = avg(x), v = avg((x - m)^2), rstd = 1 / sqrt(v + eps), y = (x - m) rstd w + b
//   backward  n = (x - m) rstd, g = dy w:  dx = rstd (g - avg(g) - n avg(g n));
//             dw = sum over rows of dy n, db = sum over rows of dy
//
// Bound by memory: the forward reads and writes a row once, the backward reads two rows and writes
// one.  Rows of up to 32768 bf16 elements (backward: 16384) stay in registers between their statistics and
// their results; workgroups walk over the rows with the parameters in registers, the next row on its
// way, and for the backward with their sums over rows.  At 32768 rows of 7168 bf16 on one MI355X:
// forward 160 us (5.9 TB/s), backward 242 us (5.8 TB/s); three-pass kernels that re-read each row
// took 275 and 705.
#include "common.h"

#include <cmath>
#include <type_traits>

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

// ---------------------------------------------------------------------------
// rows that fit a wave's or a workgroup's registers
// ---------------------------------------------------------------------------

// LPR lanes hold a row (a wave 64 / LPR rows), or with LPR = 0 a whole workgroup does.  Lane l of a
// row holds its vectors l, l + lanes, ...: NV of them, so its columns are the same for every row, and
// the parameters and the sums over rows stay in registers while the workgroup walks over its rows.

template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Sum over the row.  For workgroups, `lds` is 16 words that no wave still reads: one barrier a sum.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
    if constexpr (LPR > 0) {
        return lanes_sum<LPR>(v);
    } else {
        v = lanes_sum<64>(v);
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        float s = 0.0f;
        for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += lds[i];
        return s;
    }
}

template <bool F32, int LPR, int NV>
__global__ __launch_bounds__(LPR > 0 ? 256 : 1024) void norm_kernel(const uint4* __restrict__ x,
                                                                    const float* __restrict__ w,
                                                                    const float* __restrict__ b,
                                                                    uint4* __restrict__ y, float* __restrict__ mean,
                                                                    float* __restrict__ rstd, int rows, int nv,
                                                                    float eps) {
    constexpr int N = RowVec<F32>::N;
    __shared__ float lds[2][16];
    const int lanes = LPR > 0 ? LPR : blockDim.x;
    const int lane = LPR > 0 ? threadIdx.x & (LPR - 1) : threadIdx.x;
    const int at_once = LPR > 0 ? 256 / LPR : 1;
    const int stride = gridDim.x * at_once;
    const float n = (float)nv * N;     // divided by, so that a constant row has its value as the mean
    int row = blockIdx.x * at_once + (LPR > 0 ? threadIdx.x / LPR : 0);
    if (row >= rows) return;           // whole rows only: a row's lanes leave together
    float wf[NV][N], bf[NV][N];
    uint4 next[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int v = lane + u * lanes;
        if (v >= nv) continue;
        load_param<N>(w, v, 1.0f, wf[u]);
        load_param<N>(b, v, 0.0f, bf[u]);
        next[u] = x[(size_t)row * nv + v];
    }
    for (; row < rows; row += stride) {
        float f[NV][N], s = 0.0f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = lane + u * lanes;
            if (v < nv) unpack_row<F32>(next[u], f[u]);
            else
#pragma unroll
                for (int i = 0; i < N; ++i) f[u][i] = 0.0f;
        }
        if (row + stride < rows) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int v = lane + u * lanes;
                if (v < nv) next[u] = x[(size_t)(row + stride) * nv + v];
            }
        }
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) s += f[u][i];
        const float m = row_sum<LPR>(s, lds[0]) / n;
        s = 0.0f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (lane + u * lanes >= nv) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f[u][i] -= m;
                s += f[u][i] * f[u][i];
            }
        }
        const float r = 1.0f / sqrtf(row_sum<LPR>(s, lds[1]) / n + eps);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = lane + u * lanes;
            if (v >= nv) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) f[u][i] = f[u][i] * r * wf[u][i] + bf[u][i];
            st_nt(pack_row<F32>(f[u]), y + (size_t)row * nv + v);
        }
        if (mean && lane == 0) {
            mean[row] = m;
            rstd[row] = r;
        }
    }
}

// One pass over dy and x: dx, and the workgroup's share of the sums over rows in
// ws[workgroup][0] = sum dy n, ws[workgroup][1] = sum dy (ws NULL: not wanted).
// LONG, for rows of more than 8 waves, whose lanes have half the registers: the weights are read again for
// each row (from the caches) and the next row is asked for at the end of a row, not at its start.  At 8192
// rows of 16384 bf16 178 us, of 8200 105; with four vectors a lane and 8 waves, which spills, 203 and 165,
// with the next row held across the sums 180 and 119.  At 4096 rows of 16384 fp32 155 us, where the kernels
// for longer rows take 337.
template <bool F32, int LPR, int NV, bool LONG>
__global__ __launch_bounds__(LPR > 0 ? 256 : LONG ? 1024 : 512) void norm_backward_kernel(
    const uint4* __restrict__ dy, const uint4* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ mean, const float* __restrict__ rstd, uint4* __restrict__ dx, float* __restrict__ ws,
    int rows, int nv) {
    constexpr int N = RowVec<F32>::N;
    // Lanes past the row read its last vector instead of none: no branches, 13 registers fewer and so
    // nothing spilled (fp32, 16384 wide: 263 -> 161 us).  Elsewhere the branches are as fast or faster
    // (7168 bf16: 245 us, without 250; 8200 bf16: 104, without 112).
    constexpr bool CLAMP = F32 && LONG;
    __shared__ float lds[4][16];
    const int lanes = LPR > 0 ? LPR : blockDim.x;
    const int lane = LPR > 0 ? threadIdx.x & (LPR - 1) : threadIdx.x;
    const int at_once = LPR > 0 ? 256 / LPR : 1;
    const int stride = gridDim.x * at_once;
    const float n = (float)nv * N;
    int row = blockIdx.x * at_once + (LPR > 0 ? threadIdx.x / LPR : 0);
    float wf[LONG ? 1 : NV][N], aw[NV][N], ab[NV][N];
    uint4 nx[NV], nd[NV];
    float nm = 0.0f, nr = 0.0f;
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            int v = lane + u * lanes;
            if (CLAMP) v = min(v, nv - 1);
            else if (v >= nv) continue;
            nx[u] = x[(size_t)t * nv + v];
            nd[u] = dy[(size_t)t * nv + v];
        }
        nm = mean[t];
        nr = rstd[t];
    };
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int v = lane + u * lanes;
        if (!LONG && v < nv) load_param<N>(w, v, 1.0f, wf[u]);
#pragma unroll
        for (int i = 0; i < N; ++i) aw[u][i] = ab[u][i] = 0.0f;
    }
    if (row < rows) fetch(row);
    for (int turn = 0; row < rows; row += stride, turn ^= 2) {
        float f[NV][N], d[NV][N], sg = 0.0f, sn = 0.0f;
        const float m = nm, r = nr;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (lane + u * lanes < nv) {
                unpack_row<F32>(nx[u], f[u]);
                unpack_row<F32>(nd[u], d[u]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) f[u][i] = d[u][i] = wf[LONG ? 0 : u][i] = 0.0f;
            }
        }
        if (!LONG && row + stride < rows) fetch(row + stride);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float* wu = wf[LONG ? 0 : u];
            if (LONG) {
                const bool in = lane + u * lanes < nv;
                int at = in ? lane + u * lanes : nv - 1;
                asm volatile("" : "+v"(at));     // not the same for each row: else the compiler keeps the weights
                load_param<N>(w, at, 1.0f, wu);
#pragma unroll
                for (int i = 0; i < N; ++i) wu[i] = in ? wu[i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f[u][i] = (f[u][i] - m) * r;
                aw[u][i] += d[u][i] * f[u][i];
                ab[u][i] += d[u][i];
                d[u][i] *= wu[i];
                sg += d[u][i];
                sn += d[u][i] * f[u][i];
            }
        }
        float c1, c2;
        if constexpr (LPR > 0) {
            c1 = lanes_sum<LPR>(sg) / n;
            c2 = lanes_sum<LPR>(sn) / n;
        } else {
            // the sums of two rows in a row use different words: one barrier a row
            sg = lanes_sum<64>(sg);
            sn = lanes_sum<64>(sn);
            if ((threadIdx.x & 63) == 0) {
                lds[turn][threadIdx.x >> 6] = sg;
                lds[turn + 1][threadIdx.x >> 6] = sn;
            }
            __syncthreads();
            sg = sn = 0.0f;
            for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
                sg += lds[turn][i];
                sn += lds[turn + 1][i];
            }
            c1 = sg / n;
            c2 = sn / n;
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = lane + u * lanes;
            if (v >= nv) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) f[u][i] = r * (d[u][i] - c1 - f[u][i] * c2);
            st_nt(pack_row<F32>(f[u]), dx + (size_t)row * nv + v);
        }
        if (LONG && row + stride < rows) fetch(row + stride);
    }
    if (!ws) return;
    const size_t H = (size_t)nv * N;
    float* o = ws + (size_t)blockIdx.x * 2 * H;
    if constexpr (LPR > 0) {
        // the rows of a wave, then those of the four waves
        __shared__ float part[4][LPR * N];
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float s = k == 0 ? aw[u][i] : ab[u][i];
#pragma unroll
                    for (int off = LPR; off < 64; off <<= 1) s += __shfl_xor(s, off, 64);
                    if ((threadIdx.x & 63) < LPR) part[threadIdx.x >> 6][lane * N + i] = s;
                }
                __syncthreads();
                const int c0 = u * LPR * N;
                for (int c = threadIdx.x; c < LPR * N && c0 + c < (int)H; c += 256)
                    o[k * H + c0 + c] = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
            }
    } else {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = lane + u * lanes;
            if (v >= nv) continue;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                *reinterpret_cast<float4*>(o + (size_t)v * N + i) = make_float4(aw[u][i], aw[u][i + 1], aw[u][i + 2], aw[u][i + 3]);
                *reinterpret_cast<float4*>(o + H + (size_t)v * N + i) = make_float4(ab[u][i], ab[u][i + 1], ab[u][i + 2], ab[u][i + 3]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// longer rows
// ---------------------------------------------------------------------------

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

// Joins the partial sums of `splits` shares: 64 columns a workgroup, the shares dealt to its 16 waves.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* __restrict__ ws, float* __restrict__ dw,
                                                         float* __restrict__ db, int splits, int H, int accum) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    float* out = blockIdx.y == 0 ? dw : db;
    if (!out) return;
    const float* p = ws + (size_t)blockIdx.y * H + c;
    float s = 0.0f;
    if (c < H) {
#pragma unroll 8
        for (int i = wave; i < splits; i += 16) s += p[(size_t)i * 2 * H];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || c >= H) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += part[i][lane];
    out[c] = accum ? out[c] + s : s;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr int kCUs = 256;

// How a row of nv vectors is spread: over `lpr` lanes of a wave, or (0) over `waves` waves, `per`
// vectors a lane; per == 0: it does not fit, the kernels for longer rows take it.
struct RowShape {
    int lpr, waves, per;
};

static RowShape row_shape(int nv, int max_waves) {
    if (nv <= 8) return {8, 4, 1};
    if (nv <= 16) return {16, 4, 1};
    if (nv <= 32) return {32, 4, 1};
    if (nv <= 64) return {64, 4, 1};
    if (nv <= 128) return {64, 4, 2};
    for (int per = 2; per <= 4; per *= 2) {
        const int waves = (nv + 64 * per - 1) / (64 * per);
        if (waves <= max_waves) return {0, waves, per};
    }
    return {0, 4, 0};
}

static RowShape forward_shape(const moonep_dims_t* d) {
    return row_shape(d->H / (d->flags & MOONEP_F32_ROWS ? 4 : 8), 16);
}

// The backward holds a row or two and its sums, 16 elements of each a lane: up to 8 waves with the weights
// in registers too, up to 16 without them (LONG).
static RowShape backward_shape(const moonep_dims_t* d) {
    const bool f32 = (d->flags & MOONEP_F32_ROWS) != 0;
    const int nv = d->H / (f32 ? 4 : 8), per = f32 ? 4 : 2, waves = (nv + 64 * per - 1) / (64 * per);
    if (waves <= 8) return row_shape(nv, 8);
    return waves <= 16 ? RowShape{0, waves, per} : RowShape{0, 4, 0};
}

// Workgroups of the backward, each with its share of the rows.  Eight waves a CU, or nine, 16 bytes of each
// row a lane ahead: 244 us at 32768 x 7168 (16 waves 252, 24 waves 259), 43 us at 16384 x 2048 (16 waves
// 57): fewer shares to write and join.  Workgroups of three waves: 52 us at 16384 x 2560 with three of them
// a CU, 62 with two.  Of five: one a CU (105 us at 16384 x 5120, two 109), but two where a lane has 8
// elements instead of 16 (16384 x 2056 fp32: 76 us, one 88).
static int norm_splits(const moonep_dims_t* d) {
    const int rows = d->R * d->S;
    const RowShape s = backward_shape(d);
    if (s.per == 0) return std::min(rows, 2 * kCUs);
    const int at_once = s.lpr > 0 ? 256 / s.lpr : 1;
    const int waves = s.per == 2 && d->flags & MOONEP_F32_ROWS ? 8 + s.waves / 2 : 9;
    const int most = kCUs * (s.lpr > 0 ? 2 : std::max(1, waves / s.waves));
    return std::min((rows + at_once - 1) / at_once, most);
}

template <class F>
static void with_shape(const RowShape& s, F f) {
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I4 = std::integral_constant<int, 4>;
    if (s.lpr == 8) f(std::integral_constant<int, 8>{}, I1{});
    else if (s.lpr == 16) f(std::integral_constant<int, 16>{}, I1{});
    else if (s.lpr == 32) f(std::integral_constant<int, 32>{}, I1{});
    else if (s.lpr == 64 && s.per == 1) f(std::integral_constant<int, 64>{}, I1{});
    else if (s.lpr == 64) f(std::integral_constant<int, 64>{}, I2{});
    else if (s.per == 2) f(I0{}, I2{});
    else f(I0{}, I4{});
}

template <bool F32>
static void launch_norm(const moonep_dims_t* d, hipStream_t s, const uint4* x, const float* w, const float* b,
                        uint4* y, float* mean, float* rstd, float eps) {
    const int rows = d->R * d->S, nv = d->H / RowVec<F32>::N;
    const RowShape sh = forward_shape(d);
    if (sh.per == 0) {
        hipLaunchKernelGGL(norm_rows_kernel<F32>, dim3(rows), dim3(256), 0, s, x, w, b, y, mean, rstd, nv, eps);
        return;
    }
    const int at_once = sh.lpr > 0 ? 256 / sh.lpr : 1;
    // as many workgroups as are resident: up to 24 waves a CU in whole workgroups (32768 x 7168 bf16, 7 waves a
    // row: 161 us with 21 waves a CU; 16 asked for 194, 32 asked for 206, one round of resident ones and part
    // of another), so one workgroup of 13 to 16 (32768 x 7168 float32: 348 us, 5.4 TB/s; 16384 x 16384 bf16:
    // 224 us, 4.8 TB/s); rows within a wave 20 (200000 x 512: 74 us; 24 waves 83)
    const int most = kCUs * (sh.lpr > 0 ? 5 : std::max(1, 24 / sh.waves));
    const dim3 grid(std::min((rows + at_once - 1) / at_once, most));
    with_shape(sh, [&](auto lpr, auto per) {
        hipLaunchKernelGGL((norm_kernel<F32, lpr.value, per.value>), grid, dim3(64 * sh.waves), 0, s, x, w, b, y,
                           mean, rstd, rows, nv, eps);
    });
}

template <bool F32>
static void launch_norm_backward(const moonep_dims_t* d, hipStream_t s, const uint4* dy, const uint4* x,
                                 const float* w, const float* mean, const float* rstd, uint4* dx, float* ws) {
    const int rows = d->R * d->S, nv = d->H / RowVec<F32>::N, splits = norm_splits(d);
    const RowShape sh = backward_shape(d);
    if (sh.per == 0) {
        hipLaunchKernelGGL(norm_dx_rows_kernel<F32>, dim3(rows), dim3(256), 0, s, dy, x, w, mean, rstd, dx, nv);
        if (ws)
            hipLaunchKernelGGL(norm_dw_cols_kernel<F32>, dim3((nv + 255) / 256, splits), dim3(256), 0, s, dy, x, mean,
                               rstd, ws, rows, nv);
        return;
    }
    const dim3 grid(splits), block(64 * sh.waves);
    if (sh.waves > 8) {
        hipLaunchKernelGGL((norm_backward_kernel<F32, 0, F32 ? 4 : 2, true>), grid, block, 0, s, dy, x, w, mean, rstd,
                           dx, ws, rows, nv);
        return;
    }
    with_shape(sh, [&](auto lpr, auto per) {
        if constexpr (F32 || per.value <= 2)
            hipLaunchKernelGGL((norm_backward_kernel<F32, lpr.value, per.value, false>), grid, block, 0, s, dy, x, w,
                               mean, rstd, dx, ws, rows, nv);
    });
}

// The dims that a norm has: the rows (2^30 at most), their length and type.
static int check_rows(const moonep_dims_t* d) {
    if (!d) return MOONEP_EINVAL;
    if (d->R < 1 || d->R > kMaxR || d->S < 1 || d->H < 8 || d->H % 8 != 0) return MOONEP_EINVAL;
    if ((int64_t)d->R * d->S > (int64_t)1 << 30) return MOONEP_EINVAL;
    if (d->flags & ~(MOONEP_TRAINING | MOONEP_F32_ROWS | MOONEP_GRAD_ACCUM | MOONEP_PLAN_LOWMIG | kPhaseBits))
        return MOONEP_EINVAL;
    return MOONEP_OK;
}

static size_t row_bytes(const moonep_dims_t* d) {
    return (size_t)d->R * d->S * d->H * (d->flags & MOONEP_F32_ROWS ? 4 : 2);
}
static size_t stat_bytes(const moonep_dims_t* d) { return (size_t)d->R * d->S * sizeof(float); }
static size_t param_bytes(const moonep_dims_t* d) { return (size_t)d->H * sizeof(float); }

}  // namespace moonep

using namespace moonep;

extern "C" int moonep_layer_norm(const moonep_dims_t* dims, const void* x, const float* weight, const float* bias,
                                 float eps, void* y, float* mean, float* rstd, void* stream) {
    const int rc = check_rows(dims);
    if (rc != MOONEP_OK) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps) || !mean != !rstd) return MOONEP_EINVAL;
    MOONEP_CHECK_PTR(x);
    MOONEP_CHECK_PTR(y);
    if (!aligned16(weight) || !aligned16(bias) || !aligned16(mean) || !aligned16(rstd)) return MOONEP_EALIGN;
    const bool f32 = (dims->flags & MOONEP_F32_ROWS) != 0;
    // workgroups read their next row while they write one
    const size_t rows = row_bytes(dims), stats = stat_bytes(dims), params = param_bytes(dims);
    const Span all[] = {{y, rows}, {mean, stats}, {rstd, stats}, {x, rows}, {weight, params}, {bias, params}};
    if (outputs_overlap(all, 3, 6)) return MOONEP_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint4* xv = static_cast<const uint4*>(x);
    uint4* yv = static_cast<uint4*>(y);
    if (f32) launch_norm<true>(dims, s, xv, weight, bias, yv, mean, rstd, eps);
    else launch_norm<false>(dims, s, xv, weight, bias, yv, mean, rstd, eps);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

extern "C" size_t moonep_layer_norm_workspace_bytes(const moonep_dims_t* dims) {
    if (check_rows(dims) != MOONEP_OK) return 0;
    return (size_t)norm_splits(dims) * 2 * dims->H * sizeof(float);
}

extern "C" int moonep_layer_norm_backward(const moonep_dims_t* dims, const void* dy, const void* x,
                                          const float* weight, const float* mean, const float* rstd, void* dx,
                                          float* dweight, float* dbias, void* ws, void* stream) {
    const int rc = check_rows(dims);
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
    const size_t rows = row_bytes(dims), stats = stat_bytes(dims), params = param_bytes(dims);
    const Span all[] = {{dx, rows}, {dweight, params}, {dbias, params},
                        {sums ? ws : nullptr, moonep_layer_norm_workspace_bytes(dims)},
                        {dy, rows}, {x, rows}, {weight, params}, {mean, stats}, {rstd, stats}};
    if (outputs_overlap(all, 4, 9)) return MOONEP_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint4 *dv = static_cast<const uint4*>(dy), *xv = static_cast<const uint4*>(x);
    uint4* ov = static_cast<uint4*>(dx);
    float* wsf = sums ? static_cast<float*>(ws) : nullptr;
    if (f32) launch_norm_backward<true>(dims, s, dv, xv, weight, mean, rstd, ov, wsf);
    else launch_norm_backward<false>(dims, s, dv, xv, weight, mean, rstd, ov, wsf);
    MOONEP_LAUNCH_CHECK();
    if (!sums) return MOONEP_OK;
    hipLaunchKernelGGL(norm_join_kernel, dim3((dims->H + 63) / 64, 2), dim3(1024), 0, s, wsf, dweight, dbias,
                       norm_splits(dims), dims->H, (dims->flags & MOONEP_GRAD_ACCUM) != 0);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}
