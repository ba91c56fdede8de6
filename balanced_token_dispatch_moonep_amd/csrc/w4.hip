// The experts' FFN for decoded tokens, with weights in 4 bits.
//
//   out[t] = sum_k gate[t,k] * ((silu(x_t G_e) * (x_t U_e)) D_e),  e = topk[t,k]
//
// A weight is an e2m1 code times a power of two shared by 32 values along the input direction (the
// OCP Microscaling FP4 format).  v_cvt_scalef32_pk_bf16_fp4 turns two codes and their scale into two
// bf16 values, exactly, in one instruction; matrix instructions multiply them by the tokens' rows.
//
// Pairs (token, k) are grouped by expert, so that an expert's weights are read once for all its
// tokens.  A lane (column c = lane % 16, group q = lane / 16) of a wave loads 16 bytes: the 32 codes
// of group q of column c in a block of 128 input values.  The matrix instruction of step m
// multiplies values q * 32 + m * 8 .. + 8 of each group, which is an order of the input direction
// that both operands share.
//
// Up to 64 pairs, one wave can look at all ids at once: each workgroup finds its own group, and rows
// are read where they lie.  Beyond, a first kernel groups the pairs and lays their rows out in the
// order in which the matrix instruction's operand reads them.
#include "common.h"

namespace moonep {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kGroup = 32;           // values a scale
constexpr int kBlock = 128;          // input values of one wave's load
constexpr int kTile = 16;            // rows a matrix instruction takes, columns of a tile
constexpr int kRowTiles = 4;         // row tiles of a chunk
constexpr int kChunk4 = kTile * kRowTiles;
constexpr int kFewPairs = 64;

struct W4Dims {
    int T, K, E, H, I;
};

// A matrix in the 4-bit layout.
struct W4Mat {
    const uint4* codes;              // [E][N/16][kb][64]
    const uint32_t* scales;          // [E][N/16][sb][64]
    int kin, kb, sb, nb;
};

// A run of an expert's pairs, at most kChunk4 of them, in row tiles of their own.
struct Chunk {
    int32_t expert, tile, rows, pad;
};

// Scratch.  Few pairs use act alone, as [T*K][2][I]; otherwise
struct W4Ws {
    int32_t* nchunk;                 // [1]
    Chunk* chunks;                   // [max_chunks]
    int32_t* pair;                   // [max_tiles][16] the pair of each row
    uint4* rows;                     // [max_tiles][H/128][4 steps][64 lanes] x, as operands
    uint16_t* act;                   // [max_tiles * 2][I/128][4 steps][64 lanes][8]: a row tile's 16
                                     // activations in two bf16 terms, a pair's terms next to each other
    float* y;                        // [T*K][H] by pair
    int max_chunks;
};

static int blocks_of(int kin) { return (kin + kBlock - 1) / kBlock; }
static int fours_of(int kin) { return (blocks_of(kin) + 3) / 4; }

static size_t w4_ws_layout(const W4Dims& d, void* base, W4Ws* ws) {
    const size_t pairs = (size_t)d.T * d.K, experts = std::min<size_t>(pairs, d.E);
    const bool few = pairs <= kFewPairs;
    // an expert leaves less than one tile, and less than one chunk, partly empty
    const size_t tiles = few ? 0 : experts + pairs / kTile;
    W4Ws w{};
    w.max_chunks = (int)(experts + pairs / kChunk4);
    size_t off = 0;
    auto take = [&](size_t bytes) -> void* {
        void* p = base ? static_cast<char*>(base) + off : nullptr;
        off = align_up(off + bytes, 256);
        return p;
    };
    w.nchunk = (int32_t*)take(4);
    w.chunks = (Chunk*)take(w.max_chunks * sizeof(Chunk));
    w.pair = (int32_t*)take(tiles * kTile * 4);
    w.rows = (uint4*)take(tiles * blocks_of(d.H) * 4096);
    // one tile more: the second product takes an expert's last tiles by two, and reads (without using
    // it) the tile after an odd one
    w.act = (uint16_t*)take(few ? pairs * 2 * d.I * 2 : (tiles + 1) * 2 * blocks_of(d.I) * 4096);
    w.y = (float*)take(few ? 0 : pairs * d.H * 4);
    if (ws) *ws = w;
    return off;
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

__device__ __forceinline__ uint32_t dword(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// A lane's codes and scales of four blocks of NT column tiles.
template <int NT>
struct Four {
    uint4 codes[NT][4];
    uint32_t scales[NT];
};

template <int NT>
__device__ __forceinline__ void load_four(Four<NT>& f, const W4Mat& m, const size_t* tile, int four) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint4* c = m.codes + (tile[t] * m.kb + four * 4) * 64 + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (four * 4 + j < m.kb) f.codes[t][j] = ld_nt(c + j * 64);
        f.scales[t] = m.scales[(tile[t] * m.sb + four) * 64 + lane];
    }
}

// acc[r][t] += rows * weights of four blocks; a(r, kb, i, in) is the row operand of row tile r, block
// kb and step i, of which lanes with `in` false are past the end of the input direction.
template <int RT, int NT, class A>
__device__ __forceinline__ void multiply_four(f32x4_t (&acc)[RT][NT], const Four<NT>& f, const W4Mat& m, int four, A a) {
    auto block = [&](int j, bool in) {
        const int kb = four * 4 + j;
        float s[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t] = scale_of(f.scales[t], j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bf16x8_t b[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) b[t] = widen(dword(f.codes[t][j], i), s[t]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const bf16x8_t v = __builtin_bit_cast(bf16x8_t, a(r, kb, i, in));
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, b[t], acc[r][t], 0, 0, 0);
            }
        }
    };
    if ((four + 1) * 4 * kBlock <= m.kin) {
#pragma unroll
        for (int j = 0; j < 4; ++j) block(j, true);
    } else {
        const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (four * 4 + j < m.kb) block(j, (four * 4 + j) * kBlock + q * kGroup < m.kin);
    }
}

// acc = rows times NT column tiles over fours first, first + step, ...; the next four's loads are in
// flight while one is multiplied.
template <int RT, int NT, class A>
__device__ __forceinline__ void multiply(f32x4_t (&acc)[RT][NT], const W4Mat& m, const size_t* tile, int first,
                                         int step, A a) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (first >= m.sb) return;
    Four<NT> next;
    load_four(next, m, tile, first);
    for (int four = first; four < m.sb; four += step) {
        const Four<NT> now = next;
        if (four + step < m.sb) load_four(next, m, tile, four + step);
        multiply_four<RT, NT>(acc, now, m, four, a);
    }
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// a as two bf16 terms, at least 16 bits together.  The leading one is cut, not rounded, so that it
// cannot overflow; the rest is exact before its own rounding.
__device__ __forceinline__ void two_terms(float a, uint16_t& lead, uint16_t& rest) {
    const uint32_t hi = __float_as_uint(a) & 0xffff0000u;
    const float lo = (hi & 0x7f800000u) == 0x7f800000u ? 0.0f : a - __uint_as_float(hi);
    lead = (uint16_t)(hi >> 16);
    rest = (uint16_t)pack_bf16(lo, 0.0f);
}

// ---------------------------------------------------------------------------
// few pairs
// ---------------------------------------------------------------------------

// A wave's view of all pairs: the expert of pair `lane`, -1 for none.
__device__ __forceinline__ int pair_expert(const int32_t* topk, int pairs, int E) {
    const int lane = threadIdx.x & 63;
    const int id = lane < pairs ? topk[lane] : -1;
    return (unsigned)id < (unsigned)E ? id : -1;
}

// Lane r's pair of the r-th member of `members`, r < popcount.
__device__ __forceinline__ int member_pair(unsigned long long members) {
    const int lane = threadIdx.x & 63;
    const unsigned long long below = (1ull << lane) - 1;
    const int n = __popcll(members);
    const int to = (members >> lane) & 1 ? __popcll(members & below) : n + __popcll(~members & below);
    return __builtin_amdgcn_ds_permute(to * 4, lane);
}

// act = silu(x G) * (x U) for one expert and 16 columns.  The waves deal out the input direction and
// join their sums in order.  blockIdx.y: a pair, that leads its expert's group if it is the first of
// it, or an expert where there are fewer experts than pairs.
constexpr int kUpWaves = 7;

__global__ __launch_bounds__(64 * kUpWaves) void w4_few_up_kernel(const int32_t* __restrict__ topk,
                                                                  const uint16_t* __restrict__ x, W4Mat m,
                                                                  uint16_t* __restrict__ act, W4Dims d) {
    __shared__ float4 part[kUpWaves][2][64];
    const int pairs = d.T * d.K, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
    const int id = pair_expert(topk, pairs, d.E);
    const int e = pairs <= d.E ? __builtin_amdgcn_readlane(id, blockIdx.y) : blockIdx.y;
    const unsigned long long members = __ballot(id == e);
    if (e < 0 || members == 0) return;
    if (pairs <= d.E && __ffsll(members) - 1 != (int)blockIdx.y) return;
    const int n = __popcll(members), pair = member_pair(members);
    const size_t g = (size_t)e * m.nb + blockIdx.x, tile[2] = {g, g + m.nb / 2};
    for (int r0 = 0; r0 < n; r0 += kTile) {
        // rows past the group's compute with its last one; nothing of them is stored
        const int token = __shfl(pair, min(r0 + c, n - 1), 64) / d.K;
        const uint16_t* row = x + (size_t)token * d.H + q * kGroup;
        f32x4_t acc[1][2];
        multiply<1, 2>(acc, m, tile, wave, kUpWaves, [&](int, int kb, int i, bool in) {
            return in ? *reinterpret_cast<const uint4*>(row + kb * kBlock + i * 8) : make_uint4(0, 0, 0, 0);
        });
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t)
            part[wave][t][lane] = make_float4(acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3]);
        __syncthreads();
        const int r = threadIdx.x >> 4, to = __shfl(pair, min(r0 + r, n - 1), 64);
        if (r < min(kTile, n - r0)) {
            const int at = (r / 4 * 16 + c) * 4 + r % 4;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kUpWaves; ++w) {
                gate += reinterpret_cast<const float*>(part[w][0])[at];
                up += reinterpret_cast<const float*>(part[w][1])[at];
            }
            uint16_t lead, rest;
            two_terms(swiglu(gate, up), lead, rest);
            uint16_t* o = act + (size_t)to * 2 * d.I + blockIdx.x * kTile + c;
            o[0] = lead;
            o[d.I] = rest;
        }
    }
}

// out for 16 columns and all tokens: the waves take the experts in turn, each group's rows go to LDS,
// and a token's are joined in k order.  The rows of a matrix instruction are the two terms of 8 pairs.
constexpr int kDownWaves = 8;

__global__ __launch_bounds__(64 * kDownWaves) void w4_few_down_kernel(const int32_t* __restrict__ topk,
                                                                      const float* __restrict__ gates,
                                                                      const uint16_t* __restrict__ act, W4Mat m,
                                                                      uint16_t* __restrict__ out, W4Dims d) {
    __shared__ float y[kFewPairs][kTile];
    const int pairs = d.T * d.K, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
    const int id = pair_expert(topk, pairs, d.E);
    unsigned long long left = __ballot(id >= 0);
    for (int turn = 0; left; ++turn) {
        const int e = __builtin_amdgcn_readlane(id, __ffsll(left) - 1);
        const unsigned long long members = __ballot(id == e);
        left &= ~members;
        if (turn % kDownWaves != wave) continue;
        const int n = __popcll(members), pair = member_pair(members);
        const size_t tile[1] = {(size_t)e * m.nb + blockIdx.x};
        for (int r0 = 0; r0 < n; r0 += kTile / 2) {
            const int term = min(r0 * 2 + c, n * 2 - 1);
            const uint16_t* row = act + ((size_t)__shfl(pair, term / 2, 64) * 2 + term % 2) * d.I + q * kGroup;
            f32x4_t acc[1][1];
            multiply<1, 1>(acc, m, tile, 0, 1, [&](int, int kb, int i, bool in) {
                return in ? *reinterpret_cast<const uint4*>(row + kb * kBlock + i * 8) : make_uint4(0, 0, 0, 0);
            });
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = r0 + q * 2 + i, p = __shfl(pair, min(r, n - 1), 64);
                if (r < n) y[p][c] = acc[0][0][2 * i] + acc[0][0][2 * i + 1];
            }
        }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < d.T * kTile; v += 64 * kDownWaves) {
        const int t = v / kTile, col = v % kTile;
        float s = 0.0f;
        for (int p = t * d.K; p < (t + 1) * d.K; ++p)
            if ((unsigned)topk[p] < (unsigned)d.E) s += gates[p] * y[p][col];
        out[(size_t)t * d.H + blockIdx.x * kTile + col] = (uint16_t)pack_bf16(s, 0.0f);
    }
}

// ---------------------------------------------------------------------------
// many pairs
// ---------------------------------------------------------------------------

__device__ __forceinline__ int block_sum(int v, int* lds) {   // workgroup of 256
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Expert blockIdx.y's pairs in order, and four blocks of their rows as operands.  Every workgroup
// counts all pairs itself, so that one launch does.
__global__ __launch_bounds__(256) void w4_gather_kernel(const int32_t* __restrict__ topk,
                                                        const uint16_t* __restrict__ x, W4Ws w, W4Dims d) {
    __shared__ int count[kMaxE];
    __shared__ uint16_t member[MOONEP_W4_MAX_PAIRS];
    __shared__ int lds[4];
    const int pairs = d.T * d.K, e = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < d.E; i += 256) count[i] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += 256) {
        const int id = topk[p];
        if ((unsigned)id < (unsigned)d.E) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    const int n = count[e];
    int tiles = 0, chunks = 0;
    for (int i = tid; i < e; i += 256) {
        tiles += (count[i] + kTile - 1) / kTile;
        chunks += (count[i] + kChunk4 - 1) / kChunk4;
    }
    tiles = block_sum(tiles, lds);
    chunks = block_sum(chunks, lds);
    if (e == d.E - 1 && blockIdx.x == 0 && tid == 0) w.nchunk[0] = chunks + (n + kChunk4 - 1) / kChunk4;
    if (n == 0) return;
    for (int p0 = 0, got = 0; p0 < pairs && got < n; p0 += 256) {
        const int p = p0 + tid;
        const bool hit = p < pairs && topk[p] == e;
        const unsigned long long hits = __ballot(hit);
        __syncthreads();
        if (lane == 0) lds[wave] = __popcll(hits);
        __syncthreads();
        int at = got + __popcll(hits & ((1ull << lane) - 1));
        for (int i = 0; i < wave; ++i) at += lds[i];
        if (hit) member[at] = (uint16_t)p;
        got += (lds[0] + lds[1]) + (lds[2] + lds[3]);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int r = tid; r < n; r += 256) w.pair[tiles * kTile + r] = member[r];
        for (int i = tid; i * kChunk4 < n; i += 256)
            w.chunks[chunks + i] = Chunk{e, tiles + i * kRowTiles, min(kChunk4, n - i * kChunk4), 0};
    }
    const int kb_all = (d.H + kBlock - 1) / kBlock, kb0 = blockIdx.x * 4;
    const int per_tile = min(4, kb_all - kb0) * 256, tiles_here = (n + kTile - 1) / kTile;
    for (int v = tid; v < tiles_here * per_tile; v += 256) {
        const int rt = v / per_tile, s = v % per_tile, l = s & 63, i = (s >> 6) & 3, kb = kb0 + (s >> 8);
        const int r = rt * kTile + (l & 15), k = kb * kBlock + (l >> 4) * kGroup + i * 8;
        if (r >= n || k >= d.H) continue;
        const int token = member[r] / d.K;
        w.rows[((size_t)(tiles + rt) * kb_all + kb) * 256 + (s & 255)] =
            *reinterpret_cast<const uint4*>(x + (size_t)token * d.H + k);
    }
}

// acc over the whole input direction for RT row tiles whose operands start at `rows`.
template <int RT, int NT>
__device__ __forceinline__ void multiply_rows(f32x4_t (&acc)[RT][NT], const W4Mat& m, const size_t* tile, const uint4* rows) {
    const uint4* mine = rows + (threadIdx.x & 63);
    multiply<RT, NT>(acc, m, tile, 0, 1, [&](int r, int kb, int i, bool in) {
        const uint4 v = mine[((size_t)r * m.kb + kb) * 256 + i * 64];
        return in ? v : make_uint4(0, 0, 0, 0);
    });
}

// act for one chunk; a wave takes 16 columns.
template <int RT>
__device__ __forceinline__ void up_tiles(const W4Mat& m, const W4Ws& w, const W4Dims& d, const Chunk& ch, int col) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const size_t g = (size_t)ch.expert * m.nb + col, tile[2] = {g, g + m.nb / 2};
    f32x4_t acc[RT][2];
    multiply_rows<RT, 2>(acc, m, tile, w.rows + (size_t)ch.tile * m.kb * 256);
    const int kb_all = (d.I + kBlock - 1) / kBlock, k = col * kTile + c;
    const int kb = k / kBlock, lane0 = k % kBlock / kGroup * 16, step = k % kGroup / 8, j = k % 8;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = r * kTile + q * 4 + i;
            if (row >= ch.rows) continue;
            uint16_t lead, rest;
            two_terms(swiglu(acc[r][0][i], acc[r][1][i]), lead, rest);
            const size_t half = (size_t)ch.tile * 2 + row / 8;
            uint16_t* o = w.act + (((half * kb_all + kb) * 4 + step) * 64 + lane0 + row % 8 * 2) * 8 + j;
            o[0] = lead;
            o[8] = rest;
        }
}

__global__ __launch_bounds__(256) void w4_up_kernel(W4Mat m, W4Ws w, W4Dims d) {
    if ((int)blockIdx.y >= w.nchunk[0]) return;
    const Chunk ch = w.chunks[blockIdx.y];
    const int col = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (col >= d.I / kTile) return;
    const int rt = (ch.rows + kTile - 1) / kTile;
    if (rt == 1) up_tiles<1>(m, w, d, ch, col);
    else if (rt == 2) up_tiles<2>(m, w, d, ch, col);
    else if (rt == 3) up_tiles<3>(m, w, d, ch, col);
    else up_tiles<4>(m, w, d, ch, col);
}

// y for one chunk; a wave takes 32 columns.
template <int RT>
__device__ __forceinline__ void down_tiles(const W4Mat& m, const W4Ws& w, const W4Dims& d, const Chunk& ch, int col) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const size_t g = (size_t)ch.expert * m.nb + col, tile[2] = {g, g + 1};
    f32x4_t acc[RT][2];
    multiply_rows<RT, 2>(acc, m, tile, reinterpret_cast<const uint4*>(w.act) + (size_t)ch.tile * 2 * m.kb * 256);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = r * 8 + q * 2 + i;
            if (row >= ch.rows) continue;
            float* o = w.y + (size_t)w.pair[ch.tile * kTile + row] * d.H + col * kTile + c;
            o[0] = acc[r][0][2 * i] + acc[r][0][2 * i + 1];
            o[kTile] = acc[r][1][2 * i] + acc[r][1][2 * i + 1];
        }
}

__global__ __launch_bounds__(256) void w4_down_kernel(W4Mat m, W4Ws w, W4Dims d) {
    if ((int)blockIdx.y >= w.nchunk[0]) return;
    const Chunk ch = w.chunks[blockIdx.y];
    const int col = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 2;
    if (col >= d.H / kTile) return;
    const int rt = (ch.rows + kTile / 2 - 1) / (kTile / 2);
    if (rt == 1) down_tiles<1>(m, w, d, ch, col);
    else if (rt == 2) down_tiles<2>(m, w, d, ch, col);
    else if (rt <= 4) down_tiles<4>(m, w, d, ch, col);
    else down_tiles<8>(m, w, d, ch, col);
}

// out = sum over k of gate * y, in k order, skipping ids that name no expert.
__global__ __launch_bounds__(256) void w4_join_kernel(const int32_t* __restrict__ topk, const float* __restrict__ gates,
                                                      const float4* __restrict__ y, uint2* __restrict__ out, W4Dims d) {
    const int h = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (h >= d.H / 4) return;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p = t * d.K; p < (t + 1) * d.K; ++p) {
        if ((unsigned)topk[p] >= (unsigned)d.E) continue;
        const float4 v = y[(size_t)p * (d.H / 4) + h];
        const float g = gates[p];
        s.x += g * v.x;
        s.y += g * v.y;
        s.z += g * v.z;
        s.w += g * v.w;
    }
    out[(size_t)t * (d.H / 4) + h] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
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
    const uint16_t* xr = static_cast<const uint16_t*>(x);
    if (d.T * d.K <= kFewPairs) {
        hipLaunchKernelGGL(w4_few_up_kernel, dim3(d.I / kTile, std::min(d.T * d.K, d.E)), dim3(64 * kUpWaves), 0, s,
                           topk, xr, up, w.act, d);
        MOONEP_LAUNCH_CHECK();
        hipLaunchKernelGGL(w4_few_down_kernel, dim3(d.H / kTile), dim3(64 * kDownWaves), 0, s, topk, gates, w.act,
                           down, static_cast<uint16_t*>(out), d);
        MOONEP_LAUNCH_CHECK();
        return MOONEP_OK;
    }
    hipLaunchKernelGGL(w4_gather_kernel, dim3(fours_of(d.H), d.E), dim3(256), 0, s, topk, xr, w, d);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_up_kernel, dim3((d.I / kTile + 3) / 4, w.max_chunks), dim3(256), 0, s, up, w, d);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_down_kernel, dim3((d.H / kTile + 7) / 8, w.max_chunks), dim3(256), 0, s, down, w, d);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_join_kernel, dim3((d.H / 4 + 255) / 256, d.T), dim3(256), 0, s, topk, gates,
                       reinterpret_cast<const float4*>(w.y), static_cast<uint2*>(out), d);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}
