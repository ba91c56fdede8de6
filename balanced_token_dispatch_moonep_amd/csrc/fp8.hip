// The experts' FFN in 8-bit floating point.
//
//   out[t] = sum_k gate[t,k] * (q((silu(q(x_t) G_e) * (q(x_t) U_e))) D_e),  e = topk[t,k]
//
// G, U, D are e4m3 codes times a power of two for each block of 128 x 128; q() rounds a row the same way, a
// power of two for each 128 values along it.  The matrix instruction v_mfma_scale_f32_32x32x64_f8f6f4 multiplies
// such codes and applies both powers itself, so a product needs no arithmetic beside it; that is why the scales
// are powers of two and not floats (which would cost a multiply-add for every accumulator and block).
//
// What bounds it (32 experts of H 7168 and I 2048, 8 a token; a call, inputs changing):
//   1 token       70 us   reading 352 MB of weights, 5.0 TB/s: the first product has 128 workgroups
//   64 tokens    260 us   reading 1409 MB, 5.7 TB/s in the products; 17 us to sort, round and join
//   512 tokens   350 us   the same weights, in whole rounds of tiles (3.1 of the first product): 4.2 TB/s
//   8192 tokens 2770 us   matrix instructions: 2.1 PFLOP/s in all, 2.3 to 2.5 in the first product, where the matrix
//                         cores are busy 67 to 71 % of the time at the 1.8 GHz that power leaves; the second stores its
//                         results for 180 us of its 1000, as the registers that hold them are those of the next tile
#include "dma.h"
#include "sort.h"

#include <type_traits>

namespace moonep {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBlk = 128;            // values a scale, along both directions of a weight
constexpr int kCols = 32;            // columns of a tile of the layout
constexpr int kTileBytes = kCols * kBlk;

struct F8Dims {
    int T, K, E, H, I;
};

// A matrix in the 8-bit layout.
struct F8Mat {
    const uint4* codes;              // [E][N/32][kb][8 pieces][32 columns]
    const uint8_t* scales;           // [E][nb][kbp]
    int kin, n, kb, kbp, nb;
};

// Rows in 8 bits: codes [rows][kb * 128], scale bytes [rows][sp].
struct F8Rows {
    uint8_t* codes;
    uint8_t* scales;
    int pitch, sp;
};

// A tile of a product of many rows: `rows` rows from row0 on, of one expert, and column tile nt.
struct alignas(16) Tile {
    int32_t expert, row0, rows, nt;
};

struct F8Ws {
    int32_t *hist, *offsets, *dest, *pair, *nruns;
    Run* runs;
    Tile *up_tiles, *down_tiles;
    int32_t* token;                  // [P]: of each row
    int max_runs, run_rows;
    F8Rows x, act;                   // [T], [P]
    uint16_t* y16;                   // [P][H]: float16 times
    uint8_t* y16_exp;                // [P][H/64] a power of two for each 64
    int y16_sp;
};

__host__ __device__ static constexpr int blks(int n) { return (n + kBlk - 1) / kBlk; }

// column tiles of 128 pairs of gate and up columns, and of 256 columns
__host__ __device__ static constexpr int up_columns(const F8Dims& d) { return (d.I + 127) / 128; }
__host__ __device__ static constexpr int down_columns(const F8Dims& d) { return (d.H + 255) / 256; }

// Whether two launches for few pairs take a call: 8 tokens of up to 64 pairs, whose rounded rows fit LDS.  Against tiles
// of 64 rows (us, experts as above): 1 token 71 / 90, 2 tokens 101 / 126, 4 tokens 170 / 207, 8 tokens 210 / 241; 256
// such experts, 8 tokens 408 / 454.
constexpr int kFewRows = 8, kFewPitch = 8192;
static bool f8_few(const F8Dims& d) {
    return d.T <= kFewRows && d.T * d.K <= kFewPairs && blks(d.H) * kBlk <= kFewPitch;
}

// Rows of a tile otherwise: by the pairs that an expert has on average, with which more rows that are not there meet
// fewer reads of a weight.  Tiles of 64 / 128 / 256 rows (us, experts as above): 16 pairs an expert 262 / 262 / 315, 32 272
// / 267 / -, 40 315 / 272 / -, 64 335 / 282 / 335, 128 - / 360 / 381, 192 - / 483 / 470, 512 - / 913 / 839; 8 experts of
// H 4096 and I 1024: 128 - / 55 / 74, 512 - / 115 / 108.  (Tiles of 64 rows are the exact ones, below.)
static int f8_rows(const F8Dims& d) {
    const int64_t pairs = (int64_t)d.T * d.K;
    return pairs < 36ll * d.E ? 64 : pairs < 192ll * d.E ? 128 : 256;
}

static size_t f8_ws_layout(const F8Dims& d, void* base, F8Ws* ws) {
    const size_t pairs = (size_t)d.T * d.K, experts = std::min<size_t>(pairs, d.E);
    F8Ws w{};
    size_t off = 0;
    auto take = [&](size_t bytes) -> uint8_t* {
        uint8_t* p = base ? static_cast<uint8_t*>(base) + off : nullptr;
        off = align_up(off + bytes, 256);
        return p;
    };
    auto rows = [&](size_t n, int k) {
        F8Rows r{};
        r.pitch = blks(k) * kBlk;
        r.sp = (blks(k) + 31) / 32 * 32;
        r.codes = take(n * r.pitch);
        r.scales = take(n * r.sp);
        return r;
    };
    // the same parts for every way of a call, so that the scratch of a larger call serves smaller ones
    w.run_rows = f8_rows(d);
    w.act = rows(pairs, d.I);
    if (!f8_few(d)) {
        const size_t most = experts + pairs / 64;        // runs
        w.max_runs = (int)(experts + pairs / w.run_rows);
        w.hist = (int32_t*)take(sort_hist_most(pairs, d.E));
        w.offsets = (int32_t*)take((size_t)(d.E + 1) * 4);
        w.dest = (int32_t*)take(pairs * 4);
        w.pair = (int32_t*)take(pairs * 4);
        w.token = (int32_t*)take(pairs * 4);
        w.nruns = (int32_t*)take(4);
        w.runs = (Run*)take(most * sizeof(Run));
        w.up_tiles = (Tile*)take(most * up_columns(d) * sizeof(Tile));
        w.down_tiles = (Tile*)take(most * down_columns(d) * sizeof(Tile));
        w.x = rows(d.T, d.H);
        w.y16_sp = (d.H + 63) / 64;
        w.y16 = (uint16_t*)take(pairs * d.H * 2);
        w.y16_exp = take(pairs * w.y16_sp);
    }
    if (ws) *ws = w;
    return off;
}

// ---------------------------------------------------------------------------
// rounding
// ---------------------------------------------------------------------------

// The scale byte of a block whose largest magnitude has the bits `top`: the smallest power of two that 448
// of hold it, at least 2^-126.  A block that is not finite: 127, and codes that are NaN.
__device__ __forceinline__ int scale_byte(uint32_t top) {
    const int e = (int)(top >> 23);
    if (e == 255) return 127;
    return max(e - 8 + ((top & 0x7fffffu) > 0x600000u), 1);
}
// What values of that block are multiplied by: exact.
__device__ __forceinline__ float to_codes(uint32_t top) {
    return (top >> 23) == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(254 - scale_byte(top)) << 23);
}
// Four values as codes, to nearest even.
__device__ __forceinline__ uint32_t four_codes(float a, float b, float c, float d, float m) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * m, b * m, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * m, d * m, r, true);
}

template <int N>
__device__ __forceinline__ uint32_t max_turned(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, true));
}
// Largest of 16 lanes, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max_turned<8>(v);
    v = max_turned<4>(v);
    v = max_turned<2>(v);
    return max_turned<1>(v);
}

// Eight values of a row by each of 16 lanes that hold one block: rounds them and writes codes and scale.
__device__ __forceinline__ void put_block(const float (&v)[8], const F8Rows& r, size_t row, int block, int lane16) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = max16(top);
    const float m = to_codes(top);
    *reinterpret_cast<uint2*>(r.codes + row * r.pitch + block * kBlk + lane16 * 8) =
        make_uint2(four_codes(v[0], v[1], v[2], v[3], m), four_codes(v[4], v[5], v[6], v[7], m));
    if (lane16 == 0) r.scales[row * r.sp + block] = (uint8_t)scale_byte(top);
}

// Tile t of the list: expert by expert, column tile by column tile, run by run, so that neighbours share rows and
// weights; the tiles of the first product, then those of the second.
__device__ __forceinline__ void list_tile(const F8Ws& w, const F8Dims& d, int nruns, int t) {
    int NT = up_columns(d);
    Tile* tiles = w.up_tiles;
    if (t >= nruns * NT) {
        t -= nruns * NT;
        NT = down_columns(d);
        tiles = w.down_tiles;
        if (t >= nruns * NT) return;
    }
    const Run run = w.runs[t / NT];
    const int begin = w.offsets[run.expert], rows = w.offsets[run.expert + 1] - begin;
    const int mtiles = (rows + w.run_rows - 1) / w.run_rows;
    const int local = t - (t / NT - (run.first - begin) / w.run_rows) * NT, row0 = local % mtiles * w.run_rows;
    tiles[t] = Tile{run.expert, begin + row0, min(w.run_rows, rows - row0), local / mtiles};
}

// Rounds blocks of a row of x, 16 lanes each.
__device__ __forceinline__ void round_row(const uint16_t* x, const F8Ws& w, const F8Dims& d, size_t row, int block) {
    const int lane16 = threadIdx.x % 16, k = block * kBlk + lane16 * 8;
    if (block >= blks(d.H)) return;
    const uint4 u = k < d.H ? *reinterpret_cast<const uint4*>(x + row * d.H + k) : make_uint4(0, 0, 0, 0);
    const float v[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                        bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
    put_block(v, w.x, row, block, lane16);
}

// All that comes before the products, up to kSortOnce pairs: one workgroup sorts and lists, and the others round x
// meanwhile (512 pairs 8.5 us; 4096 pairs 20, three launches 17).
__global__ __launch_bounds__(64 * kSortWaves) void fp8_begin_kernel(const uint16_t* __restrict__ x, SortArgs a, F8Ws w,
                                                                    F8Dims d) {
    constexpr int NT = 64 * kSortWaves;
    if (blockIdx.x > 0) {
        round_row(x, w, d, blockIdx.x - 1, blockIdx.y * (NT / 16) + threadIdx.x / 16);
        return;
    }
    if (blockIdx.y > 0) return;
    sort_place<true>(a, 0);
    __syncthreads();
    const int nruns = w.nruns[0], rows = w.offsets[d.E];
    for (int i = threadIdx.x; i < rows; i += NT) w.token[i] = w.pair[i] / d.K;
    for (int t = threadIdx.x; t < nruns * (up_columns(d) + down_columns(d)); t += NT) list_tile(w, d, nruns, t);
}

// The same after a sort: the workgroups past the rows of x list tiles and tokens.
__global__ __launch_bounds__(256) void fp8_rows_kernel(const uint16_t* __restrict__ x, F8Ws w, F8Dims d) {
    if ((int)blockIdx.x < d.T) {
        round_row(x, w, d, blockIdx.x, blockIdx.y * 16 + threadIdx.x / 16);
        return;
    }
    if (blockIdx.y > 0) return;
    const int t = (blockIdx.x - d.T) * 256 + threadIdx.x;
    if (t < w.offsets[d.E]) w.token[t] = w.pair[t] / d.K;
    list_tile(w, d, w.nruns[0], t);
}

// A workgroup a block of 128 x 128.  A thread reads eight columns of eight rows; the codes are turned in
// LDS so that 16 along the input direction lie together.
__global__ __launch_bounds__(256) void fp8_quantize_kernel(const uint16_t* __restrict__ w, uint4* __restrict__ codes,
                                                           uint8_t* __restrict__ scales, int kin, int N, int kb,
                                                           int kbp) {
    __shared__ __attribute__((aligned(16))) uint8_t turn[kBlk][kBlk + 16];   // [column][k]
    __shared__ uint32_t tops[4];
    const int tid = threadIdx.x, b = blockIdx.x, nblk = blockIdx.y;
    const size_t e = blockIdx.z;
    const int c8 = tid % 16 * 8, n = nblk * kBlk + c8, k0 = b * kBlk + tid / 16 * 8;
    uint8_t* scale = scales + (e * gridDim.y + nblk) * kbp;
    if (b >= kb) {                   // scales past the matrix
        if (tid == 0 && b < kbp) scale[b] = 127;
        return;
    }
    uint4 v[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = k0 + i < kin && n < N ? *reinterpret_cast<const uint4*>(w + (e * kin + k0 + i) * N + n)
                                     : make_uint4(0, 0, 0, 0);
        for (uint32_t u : {v[i].x, v[i].y, v[i].z, v[i].w}) top = max(top, max(u << 16 & 0x7fff0000u, u & 0x7fff0000u));
    }
    for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    if (tid % 64 == 0) tops[tid / 64] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const float m = to_codes(top);
    auto value = [&](int i, int j) {
        const uint32_t u = j / 2 == 0 ? v[i].x : j / 2 == 1 ? v[i].y : j / 2 == 2 ? v[i].z : v[i].w;
        return j % 2 ? bf16_hi(u) : bf16_lo(u);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint2*>(&turn[c8 + j][tid / 16 * 8]) =
            make_uint2(four_codes(value(0, j), value(1, j), value(2, j), value(3, j), m),
                       four_codes(value(4, j), value(5, j), value(6, j), value(7, j), m));
    if (tid == 0) scale[b] = (uint8_t)scale_byte(top);
    __syncthreads();
    // 4 tiles of 32 columns, 8 pieces, 32 columns
    for (int i = tid; i < 4 * 256; i += 256) {
        const int tile = i / 256, piece = i / 32 % 8, c = i % 32;
        if (nblk * kBlk + tile * kCols >= N) continue;
        codes[((e * (N / kCols) + nblk * 4 + tile) * kb + b) * 256 + piece * 32 + c] =
            *reinterpret_cast<const uint4*>(&turn[tile * kCols + c][piece * 16]);
    }
}

// ---------------------------------------------------------------------------
// few pairs
// ---------------------------------------------------------------------------

// Eight codes times their scale as bf16: exact (down to 2^-133).
__device__ __forceinline__ bf16x8_t widen(uint32_t lo, uint32_t hi, float scale) {
    union {
        bf16x2_t two[4];
        bf16x8_t all;
    } r;
    r.two[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    r.two[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    r.two[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    r.two[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return r.all;
}
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float((uint32_t)byte << 23); }
// The row of a 32 x 32 result that a lane's register r holds; the column is lane % 32.
__device__ __forceinline__ int result_row(int r, int lane) { return r / 4 * 8 + (lane >> 5) * 4 + r % 4; }

// acc = 32 rows times NT column tiles, over all blocks of the input direction.
// A lane holds row lane % 32 and, of each 32 input values, the 16 of its half of the wave; so does it of
// the columns, whose layout makes a wave's load one KiB in a row.  D blocks of weights are on their way while one is
// multiplied; past the last one they are asked for again instead of branching around the load.  start() runs
// after the first of them have been asked for; rows(k, p) and row_scale(k) give piece p and the scale of block k,
// from LDS or, with AHEAD, from memory, when they are asked for with the weights: loads return in order.
// The codes are widened to bf16: the 8-bit matrix instructions keep a sum of products to about 16 bits only
// (measured: relative error 1.3e-5, with 32x32x64, 16x16x128 and 32x32x16 alike), which moves values of act over
// the border between two codes; with bf16 operands it is exact to float32.  Half the rate costs nothing where
// reading the weights is what takes the time.
template <int NT, int D, bool AHEAD, class Start, class Rows, class Scale>
__device__ __forceinline__ void multiply_few(f32x16_t (&acc)[NT], const F8Mat& m, const size_t* tile,
                                             const uint8_t* const* scale, Start start, Rows rows, Scale row_scale) {
    const int lane = threadIdx.x & 63, n = m.kb;
    uint4 a[D][4], b[D][NT][4];
    int sa[D], sb[D][NT];
    const uint4* base[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        base[t] = m.codes + tile[t] * m.kb * 256;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] = 0.0f;
    }
    auto load = [&](int j, int s) {
        const int k = min(s, n - 1);
        if constexpr (AHEAD) {
            sa[j] = row_scale(k);
#pragma unroll
            for (int p = 0; p < 4; ++p) a[j][p] = rows(k, p);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sb[j][t] = scale[t][k];
#pragma unroll
            for (int p = 0; p < 4; ++p) b[j][t][p] = ld_nt(base[t] + (size_t)k * 256 + p * 64 + lane);
        }
    };
#pragma unroll
    for (int j = 0; j < D; ++j) load(j, j);
    start();
    for (int s = 0; s < n; s += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (s + j < n) {
                const int k = s + j;
                const float fa = scale_of(AHEAD ? sa[j] : row_scale(k));
                float fb[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) fb[t] = scale_of(sb[j][t]);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const uint4 r = AHEAD ? a[j][p] : rows(k, p);
                    const bf16x8_t a0 = widen(r.x, r.y, fa), a1 = widen(r.z, r.w, fa);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 c = b[j][t][p];
                        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0, widen(c.x, c.y, fb[t]), acc[t], 0, 0, 0);
                        acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a1, widen(c.z, c.w, fb[t]), acc[t], 0, 0, 0);
                    }
                }
            }
            load(j, s + j + D);
        }
    }
}

__device__ __forceinline__ float silu_times(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// act = q(silu(q(x) G) * (q(x) U)) of one expert's pairs and 128 columns: a block of act, which the workgroup rounds
// itself.  A wave has a pair of gate and up tiles and all of the input direction: with two or four waves a pair, which then
// join their sums, the kernel took 47 .. 55 us for one token of H 7168 instead of 46.5.
// blockIdx.y: a pair, that leads its expert's group if it is the first of it, or an expert where there are
// fewer experts than pairs.  The workgroup rounds the rows of x itself, while the first weights arrive.
__global__ __launch_bounds__(256) void fp8_few_up_kernel(const int32_t* __restrict__ topk,
                                                         const uint16_t* __restrict__ x, F8Mat m, F8Rows act, F8Dims d) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int pairs = d.T * d.K, tid = threadIdx.x, lane = tid & 63, wave = wave_of();
    const int id = pair_expert(topk, pairs, d.E);
    const int e = pairs <= d.E ? __builtin_amdgcn_readlane(id, blockIdx.y) : blockIdx.y;
    const unsigned long long members = __ballot(id == e);
    if (e < 0 || members == 0) return;
    if (pairs <= d.E && __ffsll(members) - 1 != (int)blockIdx.y) return;
    const int n = __popcll(members), pair = member_pair(members), block = blockIdx.x;
    const int gate = min(block * 4 + wave, d.I / kCols - 1), up = d.I / kCols + gate;
    const size_t tiles = (size_t)e * (m.n / kCols), tile[2] = {tiles + gate, tiles + up};
    const uint8_t* scales = m.scales + (size_t)e * m.nb * m.kbp;
    const uint8_t* scale[2] = {scales + (size_t)(gate / 4) * m.kbp, scales + (size_t)(up / 4) * m.kbp};
    // rows of x in LDS, 16 bytes apart from multiples of 128 so that eight rows meet eight groups of banks;
    // the waves' sums take their place
    const int pitch = m.kb * kBlk + 16;
    uint8_t* rows = reinterpret_cast<uint8_t*>(smem);
    uint8_t* row_scales = rows + kFewRows * pitch;
    float(*part)[2][4][64] = reinterpret_cast<float(*)[2][4][64]>(smem);
    for (int r0 = 0; r0 < n; r0 += kFewRows) {
        const int count = min(kFewRows, n - r0), mine = min(lane & 31, count - 1);
        __syncthreads();
        f32x16_t acc[2];
        multiply_few<2, 4, false>(
            acc, m, tile, scale,
            [&] {
                // 16 lanes a block
                for (int i0 = 0; i0 < count * m.kb; i0 += 16) {
                    const int i = i0 + tid / 16, r = min(i / m.kb, count - 1), b = i % m.kb, k = b * kBlk + tid % 16 * 8;
                    const size_t token = __shfl(pair, r0 + r, 64) / d.K;
                    if (i >= count * m.kb) continue;
                    const uint4 u = k < d.H ? *reinterpret_cast<const uint4*>(x + token * d.H + k) : make_uint4(0, 0, 0, 0);
                    const float v[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                                        bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
                    put_block(v, F8Rows{rows, row_scales, pitch, m.kb}, r, b, tid % 16);
                }
                wait_lgkm0();
                block_sync();
            },
            [&](int k, int p) {
                return *reinterpret_cast<const uint4*>(rows + mine * pitch + k * kBlk + p * 32 + (lane >> 5) * 16);
            },
            [&](int k) { return (int)row_scales[mine * m.kb + k]; });
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[wave][t][r][lane] = acc[t][r];      // rows 0 .. 7
        __syncthreads();
        // 16 lanes a row, eight columns each
        const int i = tid / 16;
        const size_t to = __shfl(pair, min(r0 + i, n - 1), 64);
        if (i < count) {
            const int c8 = tid % 16 * 8, t = c8 / kCols, l = i / 4 * 32 + c8 % kCols;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float g = part[t][0][i % 4][l + j], u = part[t][1][i % 4][l + j];
                v[j] = block * kBlk + c8 < d.I ? silu_times(g, u) : 0.0f;
            }
            put_block(v, act, to, block, tid % 16);
        }
    }
}

// out for 32 columns and all tokens: the waves take the experts in turn, and a token's pairs are joined in k order.
constexpr int kDownWaves = 8;
__global__ __launch_bounds__(64 * kDownWaves) void fp8_few_down_kernel(const int32_t* __restrict__ topk,
                                                                       const float* __restrict__ gates, F8Mat m,
                                                                       F8Rows act, uint16_t* __restrict__ out,
                                                                       F8Dims d) {
    __shared__ float y[kFewPairs][kCols];
    const int pairs = d.T * d.K, lane = threadIdx.x & 63, wave = wave_of(), col = blockIdx.x;
    const int id = pair_expert(topk, pairs, d.E);
    unsigned long long left = __ballot(id >= 0);
    for (int turn = 0; left; ++turn) {
        const int e = __builtin_amdgcn_readlane(id, __ffsll(left) - 1);
        const unsigned long long members = __ballot(id == e);
        left &= ~members;
        if (turn % kDownWaves != wave) continue;
        const int n = __popcll(members), pair = member_pair(members);
        const size_t tile[1] = {(size_t)e * (m.n / kCols) + col};
        const uint8_t* scale[1] = {m.scales + ((size_t)e * m.nb + col / 4) * m.kbp};
        for (int r0 = 0; r0 < n; r0 += 32) {
            const size_t row = __shfl(pair, min(r0 + (lane & 31), n - 1), 64);
            const uint8_t *codes = act.codes + row * act.pitch + (lane >> 5) * 16, *scales = act.scales + row * act.sp;
            f32x16_t acc[1];
            multiply_few<1, 2, true>(
                acc, m, tile, scale, [] {},
                [&](int k, int p) { return *reinterpret_cast<const uint4*>(codes + (size_t)k * kBlk + p * 32); },
                [&](int k) { return (int)scales[k]; });
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = r0 + result_row(r, lane), p = __shfl(pair, min(i, n - 1), 64);
                if (i < n) y[p][lane & 31] = acc[0][r];
            }
        }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < d.T * kCols; v += 64 * kDownWaves) {
        const int t = v / kCols, c = v % kCols;
        float s = 0.0f;
        for (int p = t * d.K; p < (t + 1) * d.K; ++p)
            if ((unsigned)topk[p] < (unsigned)d.E) s += gates[p] * y[p][c];
        out[(size_t)t * d.H + col * kCols + c] = (uint16_t)pack_bf16(s, 0.0f);
    }
}

// The same with the hardware's exponential and reciprocal, each off by up to 2^-23 of its value.  2^t has the rounding of t
// in it, |g| 2^-24 of the value; exp(-g) is 2^t (1 + d), where d is what t log(2) leaves of -g, with log(2) in two parts.
// In all 8 roundings of 2^-24 at most: exponential and its correction 3, sum 1, reciprocal 2, products 2.  (h keeps t finite
// for large g; t is held below 128, so that for g below -89, whose d is large then, the exponential is infinite.  From -87
// on the reciprocal may be 0, and the result with it, which is less than 2^-119 |u| there.  Without d, off by up to 66 roundings,
// 8192 tokens take 2809 instead of 2819 us.)
__device__ __forceinline__ float silu_fast(float g, float u) {
    const float h = fminf(g, 126.0f), t = fminf(h * -1.44269504089f, 127.99f);
    const float d = fmaf(t, 0x1.05c61p-29f, fmaf(t, -0x1.62e43p-1f, -h)), e = __builtin_amdgcn_exp2f(t);
    return g * __builtin_amdgcn_rcpf(1.0f + fmaf(e, d, e)) * u;
}

// ---------------------------------------------------------------------------
// products of many rows
// ---------------------------------------------------------------------------

// Tiles of BM rows x 256 columns (UP: 128 gate and the 128 up columns that belong to them); eight waves
// of BM / 2 x 64, two on a SIMD, whose results take half of its registers.  A stage is one block of 128 input values:
// BM rows of A and eight column tiles of B, copied straight into LDS, NS stages in turn, as many as fit.
// 8192 tokens, first product / second (us; 1570 / 1000 as it is): A in more and smaller units that are asked for earlier
// 1716 / 1160, B straight to registers 1807 / 1228; four waves of 128 x 128, operands read a row block earlier, or waves
// that start staggered, no faster: what waits less runs at a lower clock (all codes zero: 1370 / 920).
template <int BM>
struct F8Tile {
    static constexpr int MT = BM / 64;           // 32-row blocks of a wave
    static constexpr int NS = BM == 256 ? 2 : 3;
    static constexpr int ABYTES = BM * kBlk, STAGE = ABYTES + 256 * kBlk;
    static constexpr int PER = MT + 4;           // copies of a wave and stage
    static constexpr int SCALES_AT = NS * STAGE; // scale bytes of the rows: [2][BM][16], 16 stages each
    static constexpr int TOPS_AT = SCALES_AT + 2 * BM * 16;    // UP: largest of a row in each of four waves
    static constexpr int SMEM = TOPS_AT + 4 * BM * 4;
    static_assert(SMEM <= 160 * 1024, "one workgroup a CU");
    // stores of a wave for a tile without rows or columns past the end, at least
    static constexpr int stores(bool up) { return up ? MT : 5 * MT; }
};

__device__ __forceinline__ i32x8_t operand(uint4 a, uint4 b) {
    return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// After it the lower half of the wave holds a of both halves, a the lower's and b the upper's; the upper half b's.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ float max_halves(float v) {
    uint32_t a = __float_as_uint(v), b = a;
    swap_halves(a, b);
    return fmaxf(__uint_as_float(a), __uint_as_float(b));
}

// The 64 columns of y that a wave has of 32 rows, of which `valid` are there: float16 with one power of two that brings
// the largest of them to 2^14 .. 2^15, half the bytes of float32 and off by at most 2^-11 of a value, or 2^-39 of the
// largest (bf16 would be by 2^-8, as much as the output's own rounding).  The stored byte is the largest one's exponent field; infinities and NaN, which
// have none, stay what they are.  A lane has 16 columns of each tile of one row, in fours, and the lane in the
// other half of the wave the fours between: two of them make 16 bytes.
__device__ __forceinline__ void put_y(const f32x16_t (&v)[2], const F8Ws& w, const F8Dims& d, size_t row0, int col,
                                      int valid) {
    const int half = (threadIdx.x >> 5) & 1;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(v[j][r]));
    top = max_halves(top);
    if (__any(top == __builtin_inff())) {
        float fine = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) fine = fmaxf(fine, fabsf(v[j][r]) == __builtin_inff() ? 0.0f : fabsf(v[j][r]));
        top = max_halves(fine);
    }
    const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
    const float m = __uint_as_float((268u - e) << 23);
    // piece k: columns 16 k .. + 8 in the lower half of the wave, + 8 .. + 16 in the upper one
    uint32_t h[4][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
            f16x2_t t;
            t.x = (_Float16)(v[j][2 * i] * m);
            t.y = (_Float16)(v[j][2 * i + 1] * m);
            h[j * 2 + i / 4][i % 4] = __builtin_bit_cast(uint32_t, t);
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        swap_halves(h[k][0], h[k][2]);
        swap_halves(h[k][1], h[k][3]);
    }
    // 16 lanes of a piece change places with 16 of the next one: a store then covers 64 bytes of 16 rows, and
    // not 32 of 32 (128 bytes of 8 rows are no faster than 64)
    const int lane = threadIdx.x & 63, group = lane >> 4;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto r = __builtin_amdgcn_permlane16_swap(h[k][i], h[k + 1][i], false, false);
            h[k][i] = r[0];
            h[k + 1][i] = r[1];
        }
        const int c = col + k * 16 + (group & 1) * 16 + (group >> 1) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (lane & 15) + i * 16;
            if (r < valid && c < d.H)
                *reinterpret_cast<uint4*>(w.y16 + (row0 + r) * d.H + c) =
                    make_uint4(h[k + i][0], h[k + i][1], h[k + i][2], h[k + i][3]);
        }
    }
    if ((lane & 31) < valid && half == 0 && col < d.H) w.y16_exp[(row0 + lane) * w.y16_sp + col / 64] = (uint8_t)e;
}

template <int MT>
struct F8Frags {
    i32x8_t a[MT], b[2];
};

// What a tile's copies and products read.
template <int MT>
struct F8TileIn {
    const uint4* B;                  // the column tile that this wave copies
    const int32_t* sb[2];            // scales of the two that it multiplies, four stages a word
    const uint8_t *A, *S;
    uint32_t ao[MT];                 // the lane's pieces of A, from there
    uint32_t so;                     // scales of the row whose scales the lane copies, from S
    int nt, row0, rows;
};

template <int BM, bool UP>
__global__ __launch_bounds__(512, 1) void fp8_tile_kernel(F8Mat m, F8Ws w, F8Dims d) {
    using L = F8Tile<BM>;
    constexpr int MT = L::MT, NS = L::NS, PER = L::PER;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / 4, wn = wave % 4;
    const F8Rows in = UP ? w.x : w.act;
    const int ncol = m.n / kCols, nst = m.kb;
    const int total = sload(w.nruns) * (UP ? up_columns(d) : down_columns(d));
    // each XCD (blockIdx % 8) takes a contiguous range of tiles, whose neighbours share rows and weights
    const int chunk = (total + 7) / 8, first = blockIdx.x % 8 * chunk, end = min(total, first + chunk);
    const uint32_t lds = lds_addr(smem);
    const uint32_t a_to = __builtin_amdgcn_readfirstlane(lds + wave * 1024);
    const uint32_t b_to = __builtin_amdgcn_readfirstlane(lds + L::ABYTES + wave * 4096);
    const uint32_t s_to = __builtin_amdgcn_readfirstlane(lds + L::SCALES_AT + wave * (BM / 8) * 16);
    // where a lane reads 16 bytes of its row of a 32-row block: piece p of the block of 128
    const int r32 = lane & 31, half = lane >> 5;
    int a_at[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) a_at[p] = (wm * (BM / 2) + r32) * 128 + ((2 * p + half) ^ (r32 >> 1 & 7)) * 16;

    auto tile_of = [&](int t) {
        const int32_t* p = reinterpret_cast<const int32_t*>((UP ? w.up_tiles : w.down_tiles) + t);
        return Tile{sload(p), sload(p + 1), sload(p + 2), sload(p + 3)};
    };
    // the rows that this lane copies, within the tile: eight a copy, eight lanes a row; and one for its scales
    auto copied = [&](int u) { return u < MT ? u * 64 + wave * 8 + (lane >> 3) : wave * (BM / 8) + min(lane, BM / 8 - 1); };
    // those rows of A
    struct Sources {
        int row[MT + 1];
    };
    auto sources = [&](const Tile& c) {
        Sources r;
#pragma unroll
        for (int u = 0; u <= MT; ++u) {
            const int i = c.row0 + min(copied(u), c.rows - 1);
            r.row[u] = UP ? w.token[i] : i;
        }
        return r;
    };
    auto tile_in = [&](const Tile& c, const Sources& from) {
        F8TileIn<MT> q;
        q.nt = c.nt, q.row0 = c.row0, q.rows = c.rows;
        // column tiles that this wave copies and multiplies, past the last one the last one
        int copy, cols[2];
        if (UP) {
            const int g = d.I / kCols;
            cols[0] = min(q.nt * 4 + wn, g - 1);
            cols[1] = g + cols[0];
            copy = cols[wave / 4];
        } else {
            copy = min(q.nt * 8 + wave, ncol - 1);
            cols[0] = min(q.nt * 8 + 2 * wn, ncol - 1);
            cols[1] = min(q.nt * 8 + 2 * wn + 1, ncol - 1);
        }
        q.B = m.codes + ((size_t)c.expert * ncol + copy) * nst * 256;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            q.sb[j] = reinterpret_cast<const int32_t*>(m.scales + ((size_t)c.expert * m.nb + cols[j] / 4) * m.kbp);
        // pieces of 16 bytes are swapped by row, so that sixteen rows side by side meet sixteen different groups of
        // banks when they are read; act is addressed from the tile's first row
        q.A = UP ? in.codes : in.codes + (size_t)q.row0 * in.pitch;
        q.S = UP ? in.scales : in.scales + (size_t)q.row0 * in.sp;
        const int base = UP ? 0 : q.row0;
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int r = copied(u), p = (lane & 7) ^ (r >> 1 & 7);
            q.ao[u] = r < q.rows ? (uint32_t)(from.row[u] - base) * (uint32_t)in.pitch + p * 16 : kZeroOff;
        }
        q.so = (uint32_t)(from.row[MT] - base) * (uint32_t)in.sp;
        return q;
    };
    auto copy_scales = [&](const F8TileIn<MT>& q, int piece) {
        if (lane < BM / 8)
            dma16s(reinterpret_cast<const uint16_t*>(q.S + piece * 16), q.so, s_to + (piece & 1) * BM * 16);
    };
    auto copy_part = [&](const F8TileIn<MT>& q, int s, int buf, int i) {     // copy i of stage s
        const uint32_t to = buf * L::STAGE;
        if (i < MT)
            dma16b(rsrc_of(q.A + (size_t)s * kBlk), q.ao[i], __builtin_amdgcn_readfirstlane(a_to + to + i * 8192));
        else
            dma16s(reinterpret_cast<const uint16_t*>(q.B + (size_t)s * 256 + (i - MT) * 64), lane * 16,
                   __builtin_amdgcn_readfirstlane(b_to + to + (i - MT) * 1024));
    };
    auto copy_stage = [&](const F8TileIn<MT>& q, int s) {
        if (s < nst)
#pragma unroll
            for (int i = 0; i < PER; ++i) copy_part(q, s, s, i);
    };

    int t = first + blockIdx.x / 8;
    if (t >= end) return;
    Tile c = tile_of(t);
    F8TileIn<MT> q = tile_in(c, sources(c));
    copy_scales(q, 0);
    copy_stage(q, 0);
    copy_stage(q, 1);
    bool counted = false;            // whether the stores since those copies are as many as stores() says
    while (true) {
        if constexpr (NS == 3) copy_stage(q, 2);
        // stage 0 is there; newer copies and the last tile's stores may be on their way
        constexpr int newer = L::stores(UP) + (NS - 1) * PER;
        if (counted && nst > NS) wait_vm<newer>();
        else wait_vm<0>();
        block_sync();
        // what the next tile begins with is on its way during this one
        t += gridDim.x / 8;
        c = tile_of(min(t, end - 1));
        const Sources next = sources(c);

        f32x16_t acc[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

        F8Frags<MT> f0, f1;
        int sa0[MT], sa1[MT];        // scales of this stage's rows and the next one's
        auto read_a = [&](F8Frags<MT>& f, const char* st, int kk, int i) {
            f.a[i] = operand(*reinterpret_cast<const uint4*>(st + a_at[2 * kk] + i * 4096),
                             *reinterpret_cast<const uint4*>(st + a_at[2 * kk + 1] + i * 4096));
        };
        auto read_b = [&](F8Frags<MT>& f, const char* st, int kk) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const char* p = st + L::ABYTES + (UP ? wn + 4 * j : 2 * wn + j) * 4096 + kk * 2048 + lane * 16;
                f.b[j] = operand(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 1024));
            }
        };
        auto read_sa = [&](int (&sa)[MT], int s) {
            const char* p = smem + L::SCALES_AT + ((s >> 4) & 1) * BM * 16 + (wm * (BM / 2) + r32) * 16 + (s & 15);
#pragma unroll
            for (int i = 0; i < MT; ++i) sa[i] = *reinterpret_cast<const uint8_t*>(p + i * 512);
        };
        read_sa(sa0, 0);
        read_b(f0, smem, 0);
#pragma unroll
        for (int i = 0; i < MT; ++i) read_a(f0, smem, 0, i);
        // The products so far are asked for before what follows: they have no effect that keeps their place, and
        // moved behind a branch they hold the operands' registers.  (No instruction reads them here.)
        // acc += rows times one column tile, one slice.  Tiles of 64 rows, which few rows an expert fill, take the time that
        // reading their weights takes, and widen their operands as multiply_few does (64 tokens 262 us, with the 8-bit
        // instructions 258, and 128 rows a tile 262; with weights that the caches hold 46, 38 and 44 for 64 tokens of 8 experts
        // of H 4096 and I 1024: but then the output is off by 0.0019 to 0.0024 instead of 0.0017, unevenly where it
        // has few values, as some 4 in 10000 of act take another code).
        // None of the wave's rows is there: in tiles of 64 rows it multiplies nothing (64 tokens 268 -> 262 us; where tiles
        // are fuller 1 to 4 % slower).
        const bool idle = wm * (BM / 2) >= q.rows;
        auto product = [&](f32x16_t& sum, const i32x8_t& a, const i32x8_t& b, int sa, int sb) {
            if constexpr (BM == 64) {
                if (idle) return;
#pragma unroll
                for (int h = 0; h < 8; h += 2)
                    sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(b[h], b[h + 1], scale_of(sb)),
                                                                  widen(a[h], a[h + 1], scale_of(sa)), sum, 0, 0, 0);
            } else {
                sum = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, sum, 0, 0, 0, sb, 0, sa);
            }
        };
        auto settle = [&] {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(acc[i][j]));
        };
        // One stage: two slices of 64 input values.  After the first one every wave has read all of the
        // stage and, behind the barrier, the next stage is there for all; this stage's buffer then takes
        // stage s + NS.  A row block's operand is read where the one before has been used, so one set of
        // registers serves.  STEADY: stage s + NS exists; FIRST: stage 0 of those, whose next stage was asked for
        // before the last tile's stores; MORE: stage s + 1 exists.
        enum { LAST, MORE, STEADY, FIRST };
        int cur = 0;
        auto stage = [&](int s, auto kind_c) {
            constexpr int kind = decltype(kind_c)::value;
            const char* st = smem + cur * L::STAGE;
            const int nxt = cur + 1 == NS ? 0 : cur + 1;
            const int shift = 8 * (s & 3);
            const int w0 = sload(q.sb[0] + (s >> 2)) >> shift & 255, w1 = sload(q.sb[1] + (s >> 2)) >> shift & 255;
            read_b(f1, st, 1);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                product(acc[i][0], f0.a[i], f0.b[0], sa0[i], w0);
                product(acc[i][1], f0.a[i], f0.b[1], sa0[i], w1);
                __builtin_amdgcn_sched_barrier(0);
                read_a(f1, st, 1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            wait_lgkm0();
            if constexpr (kind == FIRST) {
                settle();
                if (counted) wait_vm<newer - PER>();
                else wait_vm<0>();
            } else if constexpr (NS == 3 && kind == STEADY) {
                wait_vm<PER>();
            } else {
                wait_vm<0>();
            }
            block_sync();
            if constexpr (kind != LAST) {
                read_sa(sa1, s + 1);
                read_b(f0, smem + nxt * L::STAGE, 0);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                product(acc[i][0], f1.a[i], f1.b[0], sa0[i], w0);
                product(acc[i][1], f1.a[i], f1.b[1], sa0[i], w1);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (kind != LAST) read_a(f0, smem + nxt * L::STAGE, 0, i);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (kind >= STEADY) {
#pragma unroll
                    for (int p = PER * i / MT; p < PER * (i + 1) / MT; ++p) copy_part(q, s + NS, cur, p);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) sa0[i] = sa1[i];
            cur = nxt;
        };
        int s = 0;
        if (nst > NS) {
            if (nst > 16) copy_scales(q, 1);
            stage(s++, std::integral_constant<int, FIRST>{});
        }
        while (s + NS < nst) {       // the scales of the next 16 stages, then those stages: no branch among these
            if ((s & 15) == 0 && s + 16 < nst) copy_scales(q, (s >> 4) + 1);
            const int stop = min(nst - NS, (s & ~15) + 16);
            for (; s < stop; ++s) stage(s, std::integral_constant<int, STEADY>{});
        }
        for (; s + 1 < nst; ++s) stage(s, std::integral_constant<int, MORE>{});
        stage(s, std::integral_constant<int, LAST>{});
        settle();

        // the next tile's first two stages are on their way while this one's results go out
        const int nt = q.nt, row0 = q.row0, rows = q.rows;
        counted = rows == BM && (UP || nt * 256 + 256 <= d.H);
        if (t < end) {
            q = tile_in(c, next);
            copy_scales(q, 0);
            copy_stage(q, 0);
            copy_stage(q, 1);
        }
        // A column of a result is a row of the tile: lane % 32 is its row, register r its column result_row(r).
        if constexpr (UP) {
            float* tops = reinterpret_cast<float*>(smem + L::TOPS_AT);
            const bool real = nt * 4 + wn < d.I / kCols;     // columns past the last one are zeros
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t top = 0;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float g = acc[i][0][r], u = acc[i][1][r];
                    const float v = !real ? 0.0f : BM == 64 ? silu_times(g, u) : silu_fast(g, u);
                    top = max(top, __float_as_uint(v) & 0x7fffffffu);
                    acc[i][0][r] = v;
                }
                uint32_t a = top, b = top;
                swap_halves(a, b);
                if (half == 0) tops[wn * BM + wm * (BM / 2) + i * 32 + r32] = __uint_as_float(max(a, b));
            }
            wait_lgkm0();
            block_sync();
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = wm * (BM / 2) + i * 32 + r32;
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(tops[k * BM + r]));
                const float f = to_codes(top);
                uint32_t c[4];
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    c[g] = four_codes(acc[i][0][4 * g], acc[i][0][4 * g + 1], acc[i][0][4 * g + 2], acc[i][0][4 * g + 3], f);
                swap_halves(c[0], c[2]);             // the lower half's columns 0 .. 15, the upper one's 16 .. 31
                swap_halves(c[1], c[3]);
                const size_t row = (size_t)row0 + r;
                if (r < rows) {
                    *reinterpret_cast<uint4*>(w.act.codes + row * w.act.pitch + nt * 128 + wn * 32 + half * 16) =
                        make_uint4(c[0], c[2], c[1], c[3]);
                    if (wn == 0 && half == 0) w.act.scales[row * w.act.sp + nt] = (uint8_t)scale_byte(top);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = wm * (BM / 2) + i * 32;
                put_y(acc[i], w, d, (size_t)row0 + r, nt * 256 + wn * 64, rows - r);
            }
        }
        if (t >= end) break;
        wait_lgkm0();
        block_sync();                // the third stage's place is free
    }
}

// out = sum over k of gate * y, in k order, skipping pairs without a row; a wave a token and VB pieces of 512 columns, KU
// of its rows read together.  Bound by memory: 8192 tokens of 8 rows of 7168 (1.06 GB) take 221 us with 7 pieces,
// 4.8 TB/s.  Fewer tokens need more waves, a piece each, and loads in flight (1 / 4 / 8 rows): 64 tokens 10.2 / 8.3 / 8.8
// us, 512 tokens 16.6 / 15.2 / 19.2, with 7 pieces a wave 64.
template <int VB, int KU>
__global__ __launch_bounds__(256) void fp8_join_kernel(const float* __restrict__ gates, F8Ws w, uint4* __restrict__ out,
                                                       F8Dims d) {
    const int tok = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63, vecs = d.H / 8;
    if (tok >= d.T) return;
    const int32_t* dest = w.dest + (size_t)tok * d.K;
    const uint4* y16 = reinterpret_cast<const uint4*>(w.y16);
    const int v0 = blockIdx.y * 64 * VB;
    float acc[VB][8] = {};
#pragma unroll 1
    for (int k0 = 0; k0 < d.K; k0 += KU) {
        int row[KU];
        float g[KU];
        uint4 y[KU][VB];
        int ex[KU][VB];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            const bool there = k0 + j < d.K;
            row[j] = there ? dest[k0 + j] : -1;
            g[j] = there ? gates[(size_t)tok * d.K + k0 + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < KU; ++j)
#pragma unroll
            for (int u = 0; u < VB; ++u) {
                const int v = v0 + u * 64 + lane;
                const bool there = row[j] >= 0 && v < vecs;
                y[j][u] = there ? ld_nt(y16 + (size_t)row[j] * vecs + v) : make_uint4(0, 0, 0, 0);
                ex[j][u] = there ? w.y16_exp[(size_t)row[j] * w.y16_sp + v / 8] : 15;
            }
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            if (row[j] < 0) continue;
#pragma unroll
            for (int u = 0; u < VB; ++u) {
                union {
                    uint4 u;
                    _Float16 h[8];
                } r;
                r.u = y[j][u];
                const float s = __uint_as_float((uint32_t)(ex[j][u] - 14) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[u][i] += g[j] * ((float)r.h[i] * s);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < VB; ++u) {
        const int v = v0 + u * 64 + lane;
        if (v < vecs)
            st_nt(make_uint4(pack_bf16(acc[u][0], acc[u][1]), pack_bf16(acc[u][2], acc[u][3]),
                             pack_bf16(acc[u][4], acc[u][5]), pack_bf16(acc[u][6], acc[u][7])),
                  out + (size_t)tok * vecs + v);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

template <int BM, bool UP>
static int launch_tiles(const F8Mat& m, const F8Ws& w, const F8Dims& d, hipStream_t s) {
    const auto kernel = fp8_tile_kernel<BM, UP>;
    constexpr int smem = F8Tile<BM>::SMEM;
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        hipSuccess)
        return MOONEP_EHIP;
    hipLaunchKernelGGL(kernel, dim3(256), dim3(512), smem, s, m, w, d);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

template <int BM>
static int launch_both(const F8Mat& up, const F8Mat& down, const F8Ws& w, const F8Dims& d, hipStream_t s) {
    const int rc = launch_tiles<BM, true>(up, w, d, s);
    return rc != MOONEP_OK ? rc : launch_tiles<BM, false>(down, w, d, s);
}

static bool f8_size(int32_t kin, int32_t n) {
    return kin >= kCols && kin % kCols == 0 && n >= kCols && n % kCols == 0 && kin <= 1 << 20 && n <= 1 << 21;
}
static size_t f8_code_bytes(int kin, int n) { return (size_t)(n / kCols) * blks(kin) * kTileBytes; }
static int f8_scale_pitch(int kin) { return (blks(kin) + 3) / 4 * 4; }

static F8Mat f8_mat(const void* codes, const void* scales, int kin, int n) {
    return F8Mat{static_cast<const uint4*>(codes), static_cast<const uint8_t*>(scales), kin, n, blks(kin),
                 f8_scale_pitch(kin), blks(n)};
}

static int check_f8(const moonep_dims_t* d) {
    if (!d || check_flags(d) != MOONEP_OK) return MOONEP_EINVAL;
    if (d->R < 1 || d->R > kMaxR || d->S < 1 || d->E < 1 || d->E > kMaxE) return MOONEP_EINVAL;
    if (d->K < 1 || d->K > kMaxK || d->K > d->E || d->H < 8 || d->I < 8) return MOONEP_EINVAL;
    if (d->flags & MOONEP_F32_ROWS) return MOONEP_ENOTSUP;
    if (!f8_size(d->H, d->I) || !f8_size(d->I, d->H)) return MOONEP_ENOTSUP;
    if ((int64_t)d->R * d->S * d->K > MOONEP_FP8_MAX_PAIRS) return MOONEP_ENOTSUP;
    // rows of x are found by 32-bit offsets
    if ((int64_t)d->R * d->S * blks(d->H) * kBlk > 0xffff0000ll) return MOONEP_ENOTSUP;
    return MOONEP_OK;
}

}  // namespace moonep

using namespace moonep;

extern "C" size_t moonep_fp8_code_bytes(int32_t Kin, int32_t N) { return f8_size(Kin, N) ? f8_code_bytes(Kin, N) : 0; }

extern "C" size_t moonep_fp8_scale_bytes(int32_t Kin, int32_t N) {
    return f8_size(Kin, N) ? (size_t)blks(N) * f8_scale_pitch(Kin) : 0;
}

extern "C" int moonep_quantize_fp8(int32_t E, int32_t Kin, int32_t N, const void* w, void* codes, void* scales,
                                   void* stream) {
    if (E < 1 || E > kMaxE || Kin < 1 || N < 1) return MOONEP_EINVAL;
    if (!f8_size(Kin, N)) return MOONEP_ENOTSUP;
    MOONEP_CHECK_PTR(w);
    MOONEP_CHECK_PTR(codes);
    MOONEP_CHECK_PTR(scales);
    const Span spans[] = {{codes, E * moonep_fp8_code_bytes(Kin, N)}, {scales, E * moonep_fp8_scale_bytes(Kin, N)},
                          {w, (size_t)E * Kin * N * 2}};
    if (outputs_overlap(spans, 2, 3)) return MOONEP_EINVAL;
    const dim3 grid(f8_scale_pitch(Kin), blks(N), E);
    hipLaunchKernelGGL(fp8_quantize_kernel, grid, dim3(256), 0, static_cast<hipStream_t>(stream),
                       static_cast<const uint16_t*>(w), static_cast<uint4*>(codes), static_cast<uint8_t*>(scales), Kin, N,
                       blks(Kin), f8_scale_pitch(Kin));
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}

extern "C" size_t moonep_fp8_ffn_workspace_bytes(const moonep_dims_t* dims) {
    if (check_f8(dims) != MOONEP_OK) return 0;
    return f8_ws_layout(F8Dims{dims->R * dims->S, dims->K, dims->E, dims->H, dims->I}, nullptr, nullptr);
}

extern "C" int moonep_fp8_ffn(const moonep_dims_t* dims, const int32_t* topk, const float* gates, const void* x,
                              const void* w13_codes, const void* w13_scales, const void* w2_codes,
                              const void* w2_scales, void* ws, void* out, void* stream) {
    const int rc = check_f8(dims);
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
    const F8Dims d{dims->R * dims->S, dims->K, dims->E, dims->H, dims->I};
    const size_t E = d.E, pairs = (size_t)d.T * d.K, rows = (size_t)d.T * d.H * 2;
    F8Ws w;
    const size_t ws_bytes = f8_ws_layout(d, ws, &w);
    const Span spans[] = {{ws, ws_bytes}, {out, rows}, {topk, pairs * 4}, {gates, pairs * 4}, {x, rows},
                          {w13_codes, E * moonep_fp8_code_bytes(d.H, 2 * d.I)},
                          {w13_scales, E * moonep_fp8_scale_bytes(d.H, 2 * d.I)},
                          {w2_codes, E * moonep_fp8_code_bytes(d.I, d.H)},
                          {w2_scales, E * moonep_fp8_scale_bytes(d.I, d.H)}};
    if (outputs_overlap(spans, 2, 9)) return MOONEP_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const F8Mat up = f8_mat(w13_codes, w13_scales, d.H, 2 * d.I), down = f8_mat(w2_codes, w2_scales, d.I, d.H);
    if (f8_few(d)) {
        const int smem = std::max(kFewRows * (up.kb * kBlk + 16 + up.kb), 4 * 2 * 4 * 64 * 4);
        if (smem > 64 * 1024 && hipFuncSetAttribute(reinterpret_cast<const void*>(fp8_few_up_kernel),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, smem) != hipSuccess)
            return MOONEP_EHIP;
        hipLaunchKernelGGL(fp8_few_up_kernel, dim3(blks(d.I), std::min(d.T * d.K, d.E)), dim3(256), smem, s, topk,
                           static_cast<const uint16_t*>(x), up, w.act, d);
        MOONEP_LAUNCH_CHECK();
        hipLaunchKernelGGL(fp8_few_down_kernel, dim3(d.H / kCols), dim3(64 * kDownWaves), 0, s, topk, gates, down, w.act,
                           static_cast<uint16_t*>(out), d);
        MOONEP_LAUNCH_CHECK();
        return MOONEP_OK;
    }
    SortArgs a = sort_args((int)pairs, d.E);
    a.topk = topk, a.hist = w.hist, a.offsets = w.offsets, a.dest = w.dest, a.pair = w.pair;
    a.run_rows = w.run_rows, a.runs = w.runs, a.nruns = w.nruns;
    if (pairs <= kSortOnce) {
        hipLaunchKernelGGL(fp8_begin_kernel, dim3(d.T + 1, (up.kb + 31) / 32), dim3(64 * kSortWaves), 0, s,
                           static_cast<const uint16_t*>(x), a, w, d);
    } else {
        if (launch_sort(a, s) != MOONEP_OK) return MOONEP_EHIP;
        const size_t listed = std::max(pairs, (size_t)w.max_runs * (up_columns(d) + down_columns(d)));
        hipLaunchKernelGGL(fp8_rows_kernel, dim3(d.T + (unsigned)((listed + 255) / 256), (up.kb + 15) / 16), dim3(256), 0,
                           s, static_cast<const uint16_t*>(x), w, d);
    }
    MOONEP_LAUNCH_CHECK();
    const int rc2 = w.run_rows == 64 ? launch_both<64>(up, down, w, d, s)
                    : w.run_rows == 128 ? launch_both<128>(up, down, w, d, s)
                                        : launch_both<256>(up, down, w, d, s);
    if (rc2 != MOONEP_OK) return rc2;
    uint4* o = static_cast<uint4*>(out);
    const int quads = (d.T + 3) / 4, vecs = d.H / 8;
    if (d.T >= 4096)
        hipLaunchKernelGGL((fp8_join_kernel<7, 1>), dim3(quads, (vecs + 447) / 448), dim3(256), 0, s, gates, w, o, d);
    else
        hipLaunchKernelGGL((fp8_join_kernel<1, 4>), dim3(quads, (vecs + 63) / 64), dim3(256), 0, s, gates, w, o, d);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}
