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
// of group q of column c in a block of 128 input values.  The matrix instruction of step i multiplies
// values q * 32 + i * 8 .. + 8 of each group, which is an order of the input direction that both
// operands share.
//
// What bounds it is reading the weights: 0.53 bytes each, against about 6 TB/s.  Measured over 32
// experts of H 7168, I 2048, 8 a token (one pass among others, weights not in the caches):
//     tokens   experts read   us     TB/s of weights
//        1           8        36       5.2
//        8          28       110       6.0
//       64          32       147       5.1
//      128          32       206       3.6, 438 TFLOP/s
// The loads skip the caches' keeping (ld_nt): with plain ones 16 tokens took 141 us instead of 125.
// From about 16 rows an expert on, feeding the matrix instructions adds to that: at 128 tokens, with two
// terms of the activation and tiles of 16 rows in part empty, they do 1.6 times the 90 GFLOP of the
// products themselves.  They are busy for 28 and 31 % of the two products, and LDS as much; without the
// weights' loads it took 193 us, without the operands' LDS reads as well 115 to 132: the waits for operands
// are most of it, on two waves a SIMD.  The second product also reads its weights 1.46 times.  Operands read
// and widened a step ahead gave 202 us instead of 206, the 32 x 32 x 16 instruction in place of the
// 16 x 16 x 32 one (as fast for each product) 224 to 270.
// From about 7000 pairs on the bf16 layer (moonep_grouped_ffn) takes less time: 8192 pairs 1170 us and 1020,
// 6144 pairs 901 and 962.
//
// Rows go through LDS, and not from global memory to the operand: loads return in order, so a wait
// for rows would be a wait for the weights that were asked for before them.  This and a loop in which
// no load is waited for early (over_fours) brought one token from 53 us to 38.
#include "common.h"

#include <type_traits>

namespace moonep {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kGroup = 32;           // values a scale
constexpr int kBlock = 128;          // input values of one wave's load
constexpr int kFour = 4 * kBlock;    // input values of four blocks, whose scales come in one load
constexpr int kTile = 16;            // rows a matrix instruction takes, columns of a tile
constexpr int kFewPairs = 64;        // one wave can look at all their ids
constexpr int kCUs = 256;

struct W4Dims {
    int T, K, E, H, I;
};

// A matrix in the 4-bit layout.
struct W4Mat {
    const uint4* codes;              // [E][N/16][kb][64]
    const uint32_t* scales;          // [E][N/16][sb][64]
    int kin, kb, sb, nb;
};

// A run of an expert's pairs.
struct Chunk {
    int32_t expert, first, n;        // its pairs are pair[first] .. pair[first + n)
};

// Most pairs a chunk of the first product, and of the second, whose rows are two a pair.  Halves of these
// took 237 us at 128 tokens instead of 208 (weights are read again for each chunk), three quarters 220,
// twice 205 with registers spilled.
constexpr int kUpRows = 64;
constexpr int kDownPairs = 32;

// Pairs a chunk of the first product.  Where a chunk of each expert is less than a round of workgroups (two
// a CU), weights read again cost less than CUs without work: 256 pairs over 4 experts of H 7168, I 2048
// 54 us with chunks of 32 and 67 of 64, 800 over 16 of H 4096, I 1024 58 and 67, 200 over 8 of H 4096, I 512 28
// and 33; with a round or more, 1024 pairs over 32 of H 7168, I 2048 229 and 207.  Less than a round but not
// much, 256 pairs over 8 of H 4096, I 2048 52 and 49, 512 pairs 71 and 74.
static int w4_up_rows(const W4Dims& d) { return d.E * ((d.I + 63) / 64) < 2 * kCUs ? kUpRows / 2 : kUpRows; }

// Scratch; few pairs need only act.
struct W4Ws {
    uint16_t* act;                   // [T*K][2][I] bf16: leading and trailing term
    float* y;                        // [T*K][H]
    int32_t* pair;                   // [T*K] by expert
    int32_t* chunks;                 // how many of each
    Chunk *up, *down;
    int max_up, max_down;
    int up_rows;
};

// Whether the kernels for few pairs take a call.  They are two launches instead of four and split an
// expert's weights finer, but a workgroup of the second product goes through all pairs, I values each,
// one after the other, and an expert's weights are read again for each eight of its pairs (four in the
// second product).  us there and with the others: 32 pairs over 8 experts of H 4096, I 1024 17 and 23,
// 64 pairs 25 and 23; 16 pairs over 7 of H 2048, I 2048 17 and 21, 64 pairs 32 and 23; 64 pairs over 28 of
// H 4096, I 512 25 and 28.  Where reading the weights takes longer than that, some more pairs: 32 over 23
// of 32 experts of H 7168, I 2048 89 and 93, over 12 of 16 experts 53 and 59, but over 4 of 4 39 and 31;
// 48 over 24 of 32 100 and 97.
static bool w4_few(const W4Dims& d) {
    const int pairs = d.T * d.K;
    if (pairs > kFewPairs) return false;
    return (int64_t)pairs * d.I <= 24 * 2048 || (d.H > 4096 && pairs <= std::min(32, 2 * d.E));
}

static int blocks_of(int kin) { return (kin + kBlock - 1) / kBlock; }
static int fours_of(int kin) { return (blocks_of(kin) + 3) / 4; }

static size_t w4_ws_layout(const W4Dims& d, void* base, W4Ws* ws) {
    const size_t pairs = (size_t)d.T * d.K, experts = std::min<size_t>(pairs, d.E);
    W4Ws w{};
    size_t off = 0;
    auto take = [&](size_t bytes) -> void* {
        void* p = base ? static_cast<char*>(base) + off : nullptr;
        off = align_up(off + bytes, 256);
        return p;
    };
    w.act = (uint16_t*)take(pairs * 2 * d.I * 2);
    if (!w4_few(d)) {
        // an expert leaves less than one chunk partly empty
        w.up_rows = w4_up_rows(d);
        w.max_up = (int)(experts + pairs / w.up_rows);
        w.max_down = (int)(experts + pairs / kDownPairs);
        w.y = (float*)take(pairs * d.H * 4);
        w.pair = (int32_t*)take(pairs * 4);
        w.chunks = (int32_t*)take(2 * 4);
        w.up = (Chunk*)take(w.max_up * sizeof(Chunk));
        w.down = (Chunk*)take(w.max_down * sizeof(Chunk));
    }
    if (ws) *ws = w;
    return off;
}

// The wave's number, known to be the same for all its lanes: what follows from it stays in scalar registers.
__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

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

// The order of a product over fours first, first + step, ...  fetch(four, whole) asks for the rows of
// four blocks, place() puts them into LDS.  load(four, n) asks for the weights of its n blocks,
// scales(then, more) takes over the present scales and asks for those of four `then`.  blocks(more, n,
// then) multiplies n blocks and lets each block's codes make room for the same block's of four `then`.
// So rows, then weights, of the next four are on their way while one is multiplied.  The loop has no
// branches: a load whose register meets another value at a join of two paths would be waited for there.
template <class Fetch, class Place, class Load, class Scales, class Blocks>
__device__ __forceinline__ void over_fours(const W4Mat& m, int first, int step, Fetch fetch, Place place, Load load,
                                           Scales scales, Blocks blocks) {
    const int whole = m.kin / kFour;
    int four = first;
    if (four < whole) {
        fetch(four, true);
        load(four, 4);
        for (; four + step < whole; four += step) {
            const int then = four + step;
            place();
            fetch(then, true);
            scales(then, std::true_type{});
            blocks(std::true_type{}, 4, then);
        }
        place();
        scales(0, std::false_type{});
        blocks(std::false_type{}, 4, 0);
        four += step;
    }
    if (four < m.sb) {               // the end of the input direction, in part
        const int n = m.kb - four * 4;
        fetch(four, false);
        load(four, n);
        place();
        scales(0, std::false_type{});
        blocks(std::false_type{}, n, 0);
    }
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// a as two bf16 terms, at least 16 bits together: the matrix instruction takes bf16, one term of 8 bits would
// show in the output (1.4 times the error that its own rounding to bf16 has), two do not (1.6e-3, as with a
// float32 activation), a third would be half as many matrix instructions more for nothing.  The leading one
// is cut, not rounded, so that it cannot overflow; the rest is exact before its own rounding.
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

// acc = up to eight rows times NT column tiles, over fours first, first + step, ...  The wave keeps
// RN rows of four blocks in `lds` (RN KiB of its own), 16-byte pieces swapped by row so that equal
// pieces of different rows lie in different banks.  Rows past RN repeat the last.
template <int RN, int NT, class Row>
__device__ __forceinline__ void multiply_few(f32x4_t (&acc)[NT], const W4Mat& m, const size_t* tile, int first,
                                             int step, uint4* lds, Row row) {
    const int lane = threadIdx.x & 63, q = lane >> 4, mine = min(lane & 15, RN - 1);
    const uint4* base[NT];           // of the tiles, the lane is added at each load: these stay scalar
    const uint32_t* sbase[NT];
    uint4 a[RN], codes[NT][4];
    uint32_t next[NT], now[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        base[t] = m.codes + tile[t] * m.kb * 64;
        sbase[t] = m.scales + tile[t] * m.sb * 64;
        acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto load_codes = [&](int four, int j) {
#pragma unroll
        for (int t = 0; t < NT; ++t) codes[t][j] = ld_nt(base[t] + (four * 4 + j) * 64 + lane);
    };
    auto load_scales = [&](int four) {
#pragma unroll
        for (int t = 0; t < NT; ++t) next[t] = (sbase[t] + four * 64)[lane];
    };
    over_fours(
        m, first, step,
        [&](int four, bool whole) {
            const int k = four * kFour + lane * 8;
#pragma unroll
            for (int r = 0; r < RN; ++r)
                a[r] = whole || k < m.kin ? *reinterpret_cast<const uint4*>(row(r) + k) : make_uint4(0, 0, 0, 0);
        },
        [&] {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int r = 0; r < RN; ++r) lds[r * 64 + (lane ^ r)] = a[r];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        },
        [&](int four, int n) {
            load_scales(four);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) load_codes(four, j);
        },
        [&](int then, auto more) {
#pragma unroll
            for (int t = 0; t < NT; ++t) now[t] = next[t];
            if constexpr (more.value) load_scales(then);
        },
        [&](auto more, int n, int then) {
            auto read = [&](int step) {
                return __builtin_bit_cast(bf16x8_t, lds[mine * 64 + ((step / 4 * 16 + q * 4 + step % 4) ^ mine)]);
            };
            bf16x8_t rows[2];        // of this step and the next
            rows[0] = read(0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= n) break;
                float s[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) s[t] = scale_of(now[t], j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (j * 4 + i < 15) rows[(i + 1) & 1] = read(j * 4 + i + 1);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(rows[i & 1], widen(dword(codes[t][j], i), s[t]),
                                                                         acc[t], 0, 0, 0);
                    // without it more steps' operands are read ahead, into registers that spill
                    __builtin_amdgcn_sched_barrier(0);
                }
                if constexpr (more.value) load_codes(then, j);
            }
        });
}

// Calls f with the number of rows, 1, 2, 4 or 8, that n rows at most eight are computed as.
template <class F>
__device__ __forceinline__ void with_rows(int n, F f) {
    if (n <= 1) f(std::integral_constant<int, 1>{});
    else if (n <= 2) f(std::integral_constant<int, 2>{});
    else if (n <= 4) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 8>{});
}

// act = silu(x G) * (x U) for one expert and 16 columns.  The waves deal out the input direction and
// join their sums in order.  blockIdx.y: a pair, that leads its expert's group if it is the first of
// it, or an expert where there are fewer experts than pairs.
// WAVES: four, three to a SIMD (168 registers): 65 us at 2 tokens; five waves 73; four to a SIMD (128
// registers, spilled) 97.  Two where H has no more than two fours, and more waves would only wait (H 1024,
// I 2048, 16 pairs over 14 experts: 19.9 us, four 22.1).
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES, 3) void w4_few_up_kernel(const int32_t* __restrict__ topk,
                                                                  const uint16_t* __restrict__ x, W4Mat m,
                                                                  uint16_t* __restrict__ act, W4Dims d) {
    __shared__ uint4 lds[WAVES][8 * 64];
    const int pairs = d.T * d.K, lane = threadIdx.x & 63, wave = wave_of(), c = lane & 15;
    const int id = pair_expert(topk, pairs, d.E);
    const int e = pairs <= d.E ? __builtin_amdgcn_readlane(id, blockIdx.y) : blockIdx.y;
    const unsigned long long members = __ballot(id == e);
    if (e < 0 || members == 0) return;
    if (pairs <= d.E && __ffsll(members) - 1 != (int)blockIdx.y) return;
    const int n = __popcll(members), pair = member_pair(members);
    const size_t g = (size_t)e * m.nb + blockIdx.x, tile[2] = {g, g + m.nb / 2};
    for (int r0 = 0; r0 < n; r0 += 8) {
        const int rows = min(8, n - r0);
        f32x4_t acc[2];
        __syncthreads();
        with_rows(rows, [&](auto rn) {
            multiply_few<rn.value, 2>(acc, m, tile, wave, WAVES, lds[wave], [&](int r) {
                return x + (size_t)(__builtin_amdgcn_readlane(pair, min(r0 + r, n - 1)) / d.K) * d.H;
            });
        });
        // the sums take the place of the wave's rows
        float4* part = reinterpret_cast<float4*>(lds[wave]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            part[t * 64 + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        __syncthreads();
        const int r = threadIdx.x >> 4, to = __shfl(pair, min(r0 + r, n - 1), 64);
        if (r < rows) {
            const int at = (r / 4 * 16 + c) * 4 + r % 4;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                gate += reinterpret_cast<const float*>(lds[w])[at];
                up += reinterpret_cast<const float*>(lds[w])[256 + at];
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
// and a token's are joined in k order.  The rows of a matrix instruction are the two terms of 4 pairs.
// WAVES: four where there are more workgroups than CUs (H 7168: 35.6 us at one token, 89 at four; eight
// 37.5 and 91, as a CU holds one workgroup of them, six 41), else eight (H 4096, I 512, 64 pairs over 28
// experts: 24 us, four 28).
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void w4_few_down_kernel(const int32_t* __restrict__ topk,
                                                                    const float* __restrict__ gates,
                                                                    const uint16_t* __restrict__ act, W4Mat m,
                                                                    uint16_t* __restrict__ out, W4Dims d) {
    __shared__ uint4 lds[WAVES][8 * 64];
    __shared__ float y[kFewPairs][kTile];
    const int pairs = d.T * d.K, lane = threadIdx.x & 63, wave = wave_of(), c = lane & 15, q = lane >> 4;
    const int id = pair_expert(topk, pairs, d.E);
    unsigned long long left = __ballot(id >= 0);
    for (int turn = 0; left; ++turn) {
        const int e = __builtin_amdgcn_readlane(id, __ffsll(left) - 1);
        const unsigned long long members = __ballot(id == e);
        left &= ~members;
        if (turn % WAVES != wave) continue;
        const int n = __popcll(members), pair = member_pair(members);
        const size_t tile[1] = {(size_t)e * m.nb + blockIdx.x};
        for (int r0 = 0; r0 < n; r0 += 4) {
            f32x4_t acc[1];
            with_rows(min(8, (n - r0) * 2), [&](auto rn) {
                multiply_few<rn.value, 1>(acc, m, tile, 0, 1, lds[wave], [&](int r) {
                    const int p = __builtin_amdgcn_readlane(pair, min(r0 + r / 2, n - 1));
                    return act + ((size_t)p * 2 + r % 2) * d.I;
                });
            });
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = r0 + q * 2 + i, p = __shfl(pair, min(r, n - 1), 64);
                if (q < 2 && r < n) y[p][c] = acc[0][2 * i] + acc[0][2 * i + 1];
            }
        }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < d.T * kTile; v += 64 * WAVES) {
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

__device__ __forceinline__ int wave_scan(int v) {    // inclusive prefix sum over the wave
    const int lane = threadIdx.x & 63;
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}

// Sorts the pairs by expert and cuts them into chunks for the two products: one workgroup, a thread an
// expert.  The order of an expert's pairs depends on which thread's atomic comes first; a row's result
// does not depend on its place.
__global__ __launch_bounds__(1024) void w4_group_kernel(const int32_t* __restrict__ topk, W4Ws w, int pairs, int E) {
    __shared__ int count[kMaxE], place[kMaxE];
    __shared__ int sums[3][16];
    const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
    count[e] = 0;
    __syncthreads();
    for (int p = e; p < pairs; p += 1024) {
        const int id = topk[p];
        if ((unsigned)id < (unsigned)E) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    const int n = count[e], up = (n + w.up_rows - 1) / w.up_rows, down = (n + kDownPairs - 1) / kDownPairs;
    const int s0 = wave_scan(n), s1 = wave_scan(up), s2 = wave_scan(down);
    if (lane == 63) {
        sums[0][wave] = s0;
        sums[1][wave] = s1;
        sums[2][wave] = s2;
    }
    __syncthreads();
    int first = s0 - n, u0 = s1 - up, d0 = s2 - down;
    for (int i = 0; i < wave; ++i) {
        first += sums[0][i];
        u0 += sums[1][i];
        d0 += sums[2][i];
    }
    place[e] = first;
    for (int i = 0; i < up; ++i) w.up[u0 + i] = Chunk{e, first + i * w.up_rows, min(w.up_rows, n - i * w.up_rows)};
    for (int i = 0; i < down; ++i) w.down[d0 + i] = Chunk{e, first + i * kDownPairs, min(kDownPairs, n - i * kDownPairs)};
    if (e == 1023) {
        w.chunks[0] = u0 + up;
        w.chunks[1] = d0 + down;
    }
    __syncthreads();
    for (int p = e; p < pairs; p += 1024) {
        const int id = topk[p];
        if ((unsigned)id < (unsigned)E) w.pair[atomicAdd(&place[id], 1)] = p;
    }
}

// acc = RT row tiles times NT column tiles, a wave's own.  The workgroup's 256 threads bring the rows
// of four blocks to LDS, 16 bytes of a row each at a time: rows(t) is the thread's row of tile t at its
// piece.  Where a piece lies in LDS is swapped by row, so that 16 lanes side by side meet 16 different
// groups of four banks; a quarter of LDS's active cycles are counted as conflicts all the same.
template <int RT, int NT, class Rows>
__device__ __forceinline__ void multiply_many(f32x4_t (&acc)[RT][NT], const W4Mat& m, const size_t* tile, uint4* lds,
                                              Rows rows) {
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
    const int piece = tid & 15, swapped = piece % 4 * 64 + piece / 4 * 16 + ((tid >> 4) ^ (piece % 4 * 4 + piece / 4));
    const uint4* base[NT];           // of the tiles, the lane is added at each load: these stay scalar
    const uint32_t* sbase[NT];
    const uint16_t* row[RT];
    uint4 a[RT][4], codes[NT][4];
    uint32_t next[NT], now[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        base[t] = m.codes + tile[t] * m.kb * 64;
        sbase[t] = m.scales + tile[t] * m.sb * 64;
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) row[r] = rows(r);
    auto load_codes = [&](int four, int j) {
#pragma unroll
        for (int t = 0; t < NT; ++t) codes[t][j] = ld_nt(base[t] + (four * 4 + j) * 64 + lane);
    };
    auto load_scales = [&](int four) {
#pragma unroll
        for (int t = 0; t < NT; ++t) next[t] = (sbase[t] + four * 64)[lane];
    };
    over_fours(
        m, 0, 1,
        [&](int four, bool whole) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = four * kFour + j * kBlock;
                    a[r][j] = whole || k + piece * 8 < m.kin ? *reinterpret_cast<const uint4*>(row[r] + k)
                                                             : make_uint4(0, 0, 0, 0);
                }
        },
        [&] {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) lds[(r * 4 + j) * 256 + swapped] = a[r][j];
            __syncthreads();
        },
        [&](int four, int n) {
            load_scales(four);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) load_codes(four, j);
        },
        [&](int then, auto more) {
#pragma unroll
            for (int t = 0; t < NT; ++t) now[t] = next[t];
            if constexpr (more.value) load_scales(then);
        },
        [&](auto more, int n, int then) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= n) break;
                float s[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) s[t] = scale_of(now[t], j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bf16x8_t b[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) b[t] = widen(dword(codes[t][j], i), s[t]);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const bf16x8_t v = __builtin_bit_cast(
                            bf16x8_t, lds[(r * 4 + j) * 256 + i * 64 + q * 16 + (c ^ (i * 4 + q))]);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, b[t], acc[r][t], 0, 0, 0);
                    }
                }
                if constexpr (more.value) load_codes(then, j);
                // without it all blocks' operands are read ahead, into registers that spill
                __builtin_amdgcn_sched_barrier(0);
            }
        });
}

// act for one chunk; a wave takes 16 columns.
template <int RT>
__device__ __forceinline__ void up_tiles(const uint16_t* x, const W4Mat& m, const W4Ws& w, const W4Dims& d,
                                         const Chunk& ch, uint4* lds) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4, last = d.I / kTile - 1;
    const int col = blockIdx.x * 4 + wave_of();
    const int* member = w.pair + ch.first;
    const size_t g = (size_t)ch.expert * m.nb + min(col, last), tile[2] = {g, g + m.nb / 2};
    f32x4_t acc[RT][2];
    multiply_many<RT, 2>(acc, m, tile, lds, [&](int t) {
        // rows past the chunk's compute with its last one; nothing of them is stored
        const int r = min(t * kTile + (int)(threadIdx.x >> 4), ch.n - 1);
        return x + (size_t)(member[r] / d.K) * d.H + (threadIdx.x & 15) * 8;
    });
    if (col > last) return;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = t * kTile + q * 4 + i;
            if (r >= ch.n) continue;
            uint16_t lead, rest;
            two_terms(swiglu(acc[t][0][i], acc[t][1][i]), lead, rest);
            uint16_t* o = w.act + (size_t)member[r] * 2 * d.I + col * kTile + c;
            o[0] = lead;
            o[d.I] = rest;
        }
}

__global__ __launch_bounds__(256, 2) void w4_up_kernel(const uint16_t* __restrict__ x, W4Mat m, W4Ws w, W4Dims d) {
    __shared__ uint4 lds[kUpRows / kTile * 1024];
    if ((int)blockIdx.y >= w.chunks[0]) return;
    const Chunk ch = w.up[blockIdx.y];
    if (ch.n > 48) up_tiles<4>(x, m, w, d, ch, lds);
    else if (ch.n > 32) up_tiles<3>(x, m, w, d, ch, lds);
    else if (ch.n > 16) up_tiles<2>(x, m, w, d, ch, lds);
    else up_tiles<1>(x, m, w, d, ch, lds);
}

// y for one chunk; a wave takes 32 columns.  The rows are the two terms of 8 pairs a row tile.
template <int RT>
__device__ __forceinline__ void down_tiles(const W4Mat& m, const W4Ws& w, const W4Dims& d, const Chunk& ch, uint4* lds) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4, last = d.H / kTile - 2;
    const int col = (blockIdx.x * 4 + wave_of()) * 2;
    const int* member = w.pair + ch.first;
    const size_t g = (size_t)ch.expert * m.nb + min(col, last), tile[2] = {g, g + 1};
    f32x4_t acc[RT][2];
    multiply_many<RT, 2>(acc, m, tile, lds, [&](int t) {
        const int term = t * kTile + (threadIdx.x >> 4);
        return w.act + ((size_t)member[min(term / 2, ch.n - 1)] * 2 + term % 2) * d.I + (threadIdx.x & 15) * 8;
    });
    if (col > last) return;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = t * 8 + q * 2 + i;
            if (r >= ch.n) continue;
            float* o = w.y + (size_t)member[r] * d.H + col * kTile + c;
            o[0] = acc[t][0][2 * i] + acc[t][0][2 * i + 1];
            o[kTile] = acc[t][1][2 * i] + acc[t][1][2 * i + 1];
        }
}

__global__ __launch_bounds__(256, 2) void w4_down_kernel(W4Mat m, W4Ws w, W4Dims d) {
    __shared__ uint4 lds[kDownPairs / 8 * 1024];
    if ((int)blockIdx.y >= w.chunks[1]) return;
    const Chunk ch = w.down[blockIdx.y];
    if (ch.n > 24) down_tiles<4>(m, w, d, ch, lds);
    else if (ch.n > 16) down_tiles<3>(m, w, d, ch, lds);
    else if (ch.n > 8) down_tiles<2>(m, w, d, ch, lds);
    else down_tiles<1>(m, w, d, ch, lds);
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
    if (w4_few(d)) {
        const dim3 up_grid(d.I / kTile, std::min(d.T * d.K, d.E));
        if (d.H > 2 * kFour)
            hipLaunchKernelGGL(w4_few_up_kernel<4>, up_grid, dim3(64 * 4), 0, s, topk, xr, up, w.act, d);
        else
            hipLaunchKernelGGL(w4_few_up_kernel<2>, up_grid, dim3(64 * 2), 0, s, topk, xr, up, w.act, d);
        MOONEP_LAUNCH_CHECK();
        uint16_t* o = static_cast<uint16_t*>(out);
        const dim3 grid(d.H / kTile);
        if (grid.x > kCUs)
            hipLaunchKernelGGL(w4_few_down_kernel<4>, grid, dim3(64 * 4), 0, s, topk, gates, w.act, down, o, d);
        else
            hipLaunchKernelGGL(w4_few_down_kernel<8>, grid, dim3(64 * 8), 0, s, topk, gates, w.act, down, o, d);
        MOONEP_LAUNCH_CHECK();
        return MOONEP_OK;
    }
    hipLaunchKernelGGL(w4_group_kernel, dim3(1), dim3(1024), 0, s, topk, w, d.T * d.K, d.E);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_up_kernel, dim3((d.I + 63) / 64, w.max_up), dim3(256), 0, s, xr, up, w, d);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_down_kernel, dim3((d.H + 127) / 128, w.max_down), dim3(256), 0, s, down, w, d);
    MOONEP_LAUNCH_CHECK();
    hipLaunchKernelGGL(w4_join_kernel, dim3((d.H / 4 + 255) / 256, d.T), dim3(256), 0, s, topk, gates,
                       reinterpret_cast<const float4*>(w.y), static_cast<uint2*>(out), d);
    MOONEP_LAUNCH_CHECK();
    return MOONEP_OK;
}
