// The experts' FFN for decoded tokens, with weights in 4 bits.
//
//   out[t] = sum_k gate[t,k] * ((silu(x_t G_e) * (x_t U_e)) D_e),  e = topk[t,k]
//
// A weight is an e2m1 code times a power of two shared by 32 values along the input direction (the
// OCP Microscaling FP4 format).  v_cvt_scalef32_pk_bf16_fp4 turns two codes and their scale into two
// bf16 values, exactly, in one instruction; matrix instructions multiply them by the tokens' rows.
//
// Pairs (token, k) are grouped by expert first, so that an expert's weights are read once for all
// its tokens.  A lane (column c = lane % 16, group q = lane / 16) of a wave loads 16 bytes: the 32
// codes of group q of column c in a block of 128 input values.  The matrix instruction of step m
// multiplies values q * 32 + m * 8 .. + 8 of each group, which is an order of the input direction
// that both operands share.
#include "common.h"

namespace moonep {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kGroup = 32;           // values a scale
constexpr int kBlock = 128;          // input values of one wave's load
constexpr int kRowsUp = 16;          // rows a matrix instruction takes

struct W4Dims {
    int T, K, E, H, I;
};

// A matrix in the 4-bit layout.
struct W4Mat {
    const uint4* codes;              // [E][N/16][kb][64]
    const uint32_t* scales;          // [E][N/16][sb][64]
    int kin, kb, sb, nb;
};

// A run of an expert's pairs: at most kRowsUp of them.
struct Chunk {
    int32_t expert, first, rows, pad;
};

struct W4Ws {
    int32_t* nchunk;                 // [1]
    Chunk* chunks;                   // [max chunks]
    int32_t* pair;                   // [T*K] pairs t * K + k by expert
    uint16_t* act;                   // [T*K][2][I] bf16: leading and trailing term, by place in `pair`
    float* y;                        // [T*K][H] by pair
    int max_chunks;
};

static size_t w4_ws_layout(const W4Dims& d, void* base, W4Ws* ws) {
    const size_t pairs = (size_t)d.T * d.K;
    W4Ws w{};
    w.max_chunks = (int)(std::min<size_t>(pairs, d.E) + pairs / kRowsUp);
    size_t off = 0;
    auto take = [&](size_t bytes) -> void* {
        void* p = base ? static_cast<char*>(base) + off : nullptr;
        off = align_up(off + bytes, 256);
        return p;
    };
    w.nchunk = (int32_t*)take(4);
    w.chunks = (Chunk*)take(w.max_chunks * sizeof(Chunk));
    w.pair = (int32_t*)take(pairs * 4);
    w.act = (uint16_t*)take(pairs * 2 * d.I * 2);
    w.y = (float*)take(pairs * d.H * 4);
    if (ws) *ws = w;
    return off;
}

// ---------------------------------------------------------------------------
// Groups the pairs by expert: one workgroup, a thread an expert.  The order of an expert's pairs
// depends on which thread's atomic comes first; a row's result does not depend on its place.
// ---------------------------------------------------------------------------

__device__ __forceinline__ int wave_scan(int v) {    // inclusive prefix sum over the wave
    const int lane = threadIdx.x & 63;
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}

__global__ __launch_bounds__(1024) void w4_group_kernel(const int32_t* __restrict__ topk, W4Ws w, int pairs, int E) {
    __shared__ int count[1024], place[1024];
    __shared__ int wave_rows[16], wave_chunks[16];
    const int e = threadIdx.x, lane = e & 63, wv = e >> 6;
    count[e] = 0;
    __syncthreads();
    for (int p = e; p < pairs; p += 1024) {
        const int id = topk[p];
        if ((unsigned)id < (unsigned)E) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    const int rows = count[e], chunks = (rows + kRowsUp - 1) / kRowsUp;
    const int rs = wave_scan(rows), cs = wave_scan(chunks);
    if (lane == 63) {
        wave_rows[wv] = rs;
        wave_chunks[wv] = cs;
    }
    __syncthreads();
    int row0 = rs - rows, chunk0 = cs - chunks;
    for (int i = 0; i < wv; ++i) {
        row0 += wave_rows[i];
        chunk0 += wave_chunks[i];
    }
    place[e] = row0;
    for (int i = 0; i < chunks; ++i)
        w.chunks[chunk0 + i] = Chunk{e, row0 + i * kRowsUp, min(kRowsUp, rows - i * kRowsUp), 0};
    if (e == 1023) w.nchunk[0] = chunk0 + chunks;
    __syncthreads();
    for (int p = e; p < pairs; p += 1024) {
        const int id = topk[p];
        if ((unsigned)id < (unsigned)E) w.pair[atomicAdd(&place[id], 1)] = p;
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

// The scale of a lane's group in block j of four, as the float the conversion takes (255: NaN).
__device__ __forceinline__ float scale_of(uint32_t four, int j) {
    const uint32_t s = (four >> (8 * j)) & 255u;
    return __uint_as_float(s == 255u ? 0x7fc00000u : s << 23);
}

// Eight codes times their scale as bf16: exact.
__device__ __forceinline__ bf16x8_t widen(uint32_t codes, float scale) {
    union {
        bf16x2_t two[4];
        bf16x8_t all;
    } r;
    r.two[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    r.two[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    r.two[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    r.two[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return r.all;
}

// acc += rows (each lane's own, bf16, its group's first value in the first block) times one column tile.
__device__ __forceinline__ f32x4_t w4_tile(const uint16_t* __restrict__ row, const W4Mat& m, size_t tile) {
    const int lane = threadIdx.x & 63, q = lane >> 4;
    const uint4* codes = m.codes + tile * m.kb * 64 + lane;
    const uint32_t* scales = m.scales + tile * m.sb * 64 + lane;
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = 0; kb < m.kb; ++kb) {
        const uint4 c = codes[(size_t)kb * 64];
        const float s = scale_of(scales[(size_t)(kb >> 2) * 64], kb & 3);
        const bool in = kb * kBlock + q * kGroup < m.kin;
        const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 a = make_uint4(0, 0, 0, 0);
            if (in) a = *reinterpret_cast<const uint4*>(row + kb * kBlock + i * 8);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), widen(cs[i], s), acc, 0, 0, 0);
        }
    }
    return acc;
}

// act = silu(x G) * (x U) for one chunk and 16 columns, as two bf16 terms.
__global__ __launch_bounds__(64) void w4_up_kernel(const uint16_t* __restrict__ x, W4Mat m, W4Ws w, W4Dims d) {
    if ((int)blockIdx.y >= w.nchunk[0]) return;
    const Chunk ch = w.chunks[blockIdx.y];
    const int lane = threadIdx.x, c = lane & 15, q = lane >> 4;
    // rows past the chunk's compute with its last one; nothing of them is stored
    const int token = w.pair[ch.first + min(c, ch.rows - 1)] / d.K;
    const uint16_t* row = x + (size_t)token * d.H + q * kGroup;
    const size_t tile = (size_t)ch.expert * m.nb + blockIdx.x;
    const f32x4_t g = w4_tile(row, m, tile);
    const f32x4_t u = w4_tile(row, m, tile + m.nb / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = q * 4 + i;
        if (r >= ch.rows) continue;
        const float a = g[i] / (1.0f + expf(-g[i])) * u[i];
        // leading term cut, not rounded, so that it cannot overflow; the rest is exact before its rounding
        const uint32_t hi = __float_as_uint(a) & 0xffff0000u;
        const float lo = (hi & 0x7f800000u) == 0x7f800000u ? 0.0f : a - __uint_as_float(hi);
        uint16_t* o = w.act + (size_t)(ch.first + r) * 2 * d.I + blockIdx.x * 16 + c;
        o[0] = (uint16_t)(hi >> 16);
        o[d.I] = (uint16_t)pack_bf16(lo, 0.0f);
    }
}

// y = act D for one chunk and 16 columns: the rows of the matrix instruction are the two terms of 8 pairs.
__global__ __launch_bounds__(64) void w4_down_kernel(W4Mat m, W4Ws w, W4Dims d) {
    if ((int)blockIdx.y >= w.nchunk[0]) return;
    const Chunk ch = w.chunks[blockIdx.y];
    const int lane = threadIdx.x, c = lane & 15, q = lane >> 4;
    const size_t tile = (size_t)ch.expert * m.nb + blockIdx.x;
    for (int r0 = 0; r0 < ch.rows; r0 += 8) {
        const int term = min(r0 * 2 + c, ch.rows * 2 - 1);
        const f32x4_t v = w4_tile(w.act + ((size_t)ch.first * 2 + term) * d.I + q * kGroup, m, tile);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r0 + q * 2 + i;
            if (r < ch.rows) w.y[(size_t)w.pair[ch.first + r] * d.H + blockIdx.x * 16 + c] = v[2 * i] + v[2 * i + 1];
        }
    }
}

// out = sum over k of gate * y, in k order, skipping ids that name no expert.
__global__ __launch_bounds__(256) void w4_join_kernel(const int32_t* __restrict__ topk, const float* __restrict__ gates,
                                                      W4Ws w, uint16_t* __restrict__ out, W4Dims d) {
    const int h = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (h >= d.H) return;
    float s = 0.0f;
    for (int k = 0; k < d.K; ++k) {
        const int p = t * d.K + k;
        if ((unsigned)topk[p] < (unsigned)d.E) s += gates[p] * w.y[(size_t)p * d.H + h];
    }
    out[(size_t)t * d.H + h] = (uint16_t)pack_bf16(s, 0.0f);
}

// ---------------------------------------------------------------------------
// quantisation
// ---------------------------------------------------------------------------

// A thread a group of 32 values of one column: 16 columns side by side read 32 bytes of each row.
__global__ __launch_bounds__(256) void w4_quantize_kernel(const uint16_t* __restrict__ w, uint4* __restrict__ codes,
                                                          uint8_t* __restrict__ scales, int kin, int N, int kb, int sb) {
    const int n = blockIdx.x * 256 + threadIdx.x, g = blockIdx.y, e = blockIdx.z;
    if (n >= N) return;
    const int b = g >> 2, q = g & 3, lane = q * 16 + (n & 15);
    const size_t tile = (size_t)e * (N / 16) + n / 16;
    uint4 code = make_uint4(0, 0, 0, 0);
    uint32_t s = 127;
    if (g * kGroup < kin) {
        const uint16_t* p = w + ((size_t)e * kin + (size_t)g * kGroup) * N + n;
        uint16_t v[kGroup];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            v[i] = p[(size_t)i * N];
            top = max(top, (uint32_t)(v[i] & 0x7fff));
        }
        top >>= 7;                               // the largest exponent field: floor(log2) + 127
        s = top == 255u ? 255u : max((int)top - 2, 1);
        if (s != 255u) {
            const float f = __uint_as_float(s << 23);
            uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = __uint_as_float((uint32_t)v[i * 8 + j * 2] << 16);
                    const float z = __uint_as_float((uint32_t)v[i * 8 + j * 2 + 1] << 16);
                    uint32_t r;
                    if (j == 0) r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, z, f, 0);
                    else if (j == 1) r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], a, z, f, 1);
                    else if (j == 2) r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], a, z, f, 2);
                    else r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], a, z, f, 3);
                    c[i] = r;
                }
            }
            code = make_uint4(c[0], c[1], c[2], c[3]);
        }
    }
    if (b < kb) codes[(tile * kb + b) * 64 + lane] = code;
    scales[((tile * sb + (b >> 2)) * 64 + lane) * 4 + (b & 3)] = (uint8_t)s;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static int blocks_of(int kin) { return (kin + kBlock - 1) / kBlock; }
static int fours_of(int kin) { return (blocks_of(kin) + 3) / 4; }

static W4Mat w4_mat(const void* codes, const void* scales, int kin, int n) {
    return W4Mat{static_cast<const uint4*>(codes), static_cast<const uint32_t*>(scales), kin, blocks_of(kin),
                 fours_of(kin), n / 16};
}

static bool w4_size(int32_t kin, int32_t n) {
    return kin >= kGroup && kin % kGroup == 0 && n >= kGroup && n % kGroup == 0 && kin <= 1 << 20 && n <= 1 << 21;
}

static int check_w4(const moonep_dims_t* d) {
    if (!d) return MOONEP_EINVAL;
    if (d->R < 1 || d->R > kMaxR || d->S < 1 || d->E < 1 || d->E > kMaxE) return MOONEP_EINVAL;
    if (d->K < 1 || d->K > kMaxK || d->K > d->E || d->H < 8 || d->I < 8) return MOONEP_EINVAL;
    if (d->flags & ~(MOONEP_TRAINING | MOONEP_F32_ROWS | MOONEP_GRAD_ACCUM | MOONEP_PLAN_LOWMIG | kPhaseBits))
        return MOONEP_EINVAL;
    if (d->flags & MOONEP_F32_ROWS) return MOONEP_ENOTSUP;
    if (!w4_size(d->H, d->I) || !w4_size(d->I, d->H)) return MOONEP_ENOTSUP;
    if ((int64_t)d->R * d->S * d->K > MOONEP_W4_MAX_PAIRS) return MOONEP_ENOTSUP;
    return MOONEP_OK;
}

}  // namespace moonep

using namespace moonep;

extern "C" size_t moonep_w4_code_bytes(int32_t Kin, int32_t N) {
    return w4_size(Kin, N) ? (size_t)N * blocks_of(Kin) * 64 : 0;
}

extern "C" size_t moonep_w4_scale_bytes(int32_t Kin, int32_t N) {
    return w4_size(Kin, N) ? (size_t)N * fours_of(Kin) * 16 : 0;
}

extern "C" int moonep_quantize_w4(int32_t E, int32_t Kin, int32_t N, const void* w, void* codes, void* scales,
                                  void* stream) {
    if (E < 1 || E > kMaxE || Kin < 1 || N < 1) return MOONEP_EINVAL;
    if (!w4_size(Kin, N)) return MOONEP_ENOTSUP;
    MOONEP_CHECK_PTR(w);
    MOONEP_CHECK_PTR(codes);
    MOONEP_CHECK_PTR(scales);
    const dim3 grid((N + 255) / 256, fours_of(Kin) * 16, E);
    hipLaunchKernelGGL(w4_quantize_kernel, grid, dim3(256), 0, static_cast<hipStream_t>(stream),
                       static_cast<const uint16_t*>(w), static_cast<uint4*>(codes), static_cast<uint8_t*>(scales), Kin,
                       N, blocks_of(Kin), fours_of(Kin));
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

extern "C" size_t moonep_w4_ffn_workspace_bytes(const moonep_dims_t* dims) {
    if (check_w4(dims) != MOONEP_OK) return 0;
    return w4_ws_layout(W4Dims{dims->R * dims->S, dims->K, dims->E, dims->H, dims->I}, nullptr, nullptr);
}

extern "C" int moonep_w4_ffn(const moonep_dims_t* dims, const int32_t* topk, const float* gates, const void* x,
                             const void* w13_codes, const void* w13_scales, const void* w2_codes,
                             const void* w2_scales, void* ws, void* out, void* stream) {
    const int rc = check_w4(dims);
    if (rc != MOONEP_OK) return rc;
    MOONEP_CHECK_PTR(topk);
    MOONEP_CHECK_PTR(gates);
    MOONEP_CHECK_PTR(x);
    MOONEP_CHECK_PTR(w13_codes);
    MOONEP_CHECK_PTR(w13_scales);
    MOONEP_CHECK_PTR(w2_codes);
    MOONEP_CHECK_PTR(w2_scales);
    MOONEP_CHECK_PTR(ws);
    MOONEP_CHECK_PTR(out);
    const W4Dims d{dims->R * dims->S, dims->K, dims->E, dims->H, dims->I};
    W4Ws w;
    w4_ws_layout(d, ws, &w);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const W4Mat up = w4_mat(w13_codes, w13_scales, d.H, 2 * d.I), down = w4_mat(w2_codes, w2_scales, d.I, d.H);
    hipLaunchKernelGGL(w4_group_kernel, dim3(1), dim3(1024), 0, s, topk, w, d.T * d.K, d.E);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_up_kernel, dim3(d.I / 16, w.max_chunks), dim3(64), 0, s, static_cast<const uint16_t*>(x), up,
                       w, d);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_down_kernel, dim3(d.H / 16, w.max_chunks), dim3(64), 0, s, down, w, d);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_join_kernel, dim3((d.H + 255) / 256, d.T), dim3(256), 0, s, topk, gates, w,
                       static_cast<uint16_t*>(out), d);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}
