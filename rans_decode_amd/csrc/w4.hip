// w4.hip -- products of a few tokens with 4-bit weights that carry a scale
// (and a zero point) per group of 32, 64 or 128 columns: eq_w4_matvec, and
// the load-time layout eq_w4_pack.
//
// Mathematics: y[t, r] = sum_g scale[r, g] * (sum_{c in g} q[r, c] x[t, c]
//   - zero[r, g] * sum_{c in g} x[t, c]). The inner sums run on the matrix
// cores: tokens are the rows of A, weight rows the columns of B, so a lane's
// accumulators all belong to one weight row (lane & 15) and a group's scale
// is one value per lane. By kind of weight and activation:
//   INT4 x bf16: a code's 4 bits go to mantissa bits 3..6 under the exponent
//     of 16, the exact bf16 16 + u with u = q + 8 (signed codes) or q (with
//     zeros): one shift and one three-input logic instruction per two weights.
//     The 16 + zero is taken off with sum(x), which one more matrix product
//     with a B of ones gives in the same registers.
//   INT4 x int8: signed codes in the upper half of a byte are the int8 16 q
//     (the 1/16 goes into the scale, exactly): three instructions per eight
//     weights, exact int32 sums within a group. With zeros the codes stay
//     unsigned and a B of ones gives sum(x).
//   E2M1 x bf16: v_cvt_scalef32_pk_bf16_fp4, one instruction per two weights.
//   E2M1 x E4M3: both sides widen to bf16, where they are exact. (The fp8 x
//     fp4 matrix instruction takes them as they are, but adds its 128 products
//     with fewer than 32 bits: 1.0e-5 off in 2-norm over a row of 28672, where
//     fp32 sums are 1e-7 off.)
// What bounds it: HBM reads of the codes (see k_w4).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/eq.h"
#include "device_util.hpp"

namespace {

using namespace eqdev;

constexpr uint32_t kTileRows = 16, kTileCols = 128, kTileBytes = 1024;
constexpr uint32_t kWaves = 8;            // waves of a workgroup
constexpr uint32_t kMaxTokens = 64;       // tokens of one pass over the weights

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

struct W4Args {
    const u32x4 *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
    const void *x;
    const float *x_scale;
    void *y;
    uint64_t ldx, ldy;
    uint32_t rows, cols;
    uint32_t wg_begin;  // first workgroup of this tensor
    uint32_t k_waves;   // waves that share out the columns of one row of tiles (1, 2, 4, 8)
    uint32_t group;
};

struct W4Launch {
    W4Args t[EQ_MAX_BLOCK_TENSORS];
    uint32_t n_tensors;
    uint32_t tokens;
    uint32_t y_f32;
};

// Column within a tile of the first of the 8 weights in word j of a lane:
// of every group (of `span` columns) a quarter wave holds span / 4
// consecutive ones, so that a lane's activations are as contiguous as the
// groups allow.
__host__ __device__ constexpr uint32_t word_col(uint32_t span, uint32_t quarter, uint32_t j) {
    const uint32_t words = span / 32;  // words of a lane per group
    return j / words * span + quarter * (span / 4) + j % words * 8;
}

// Activations of one lane for a tile: word j's 8 values at w[j * N].
template <uint32_t X>
struct XFrag {
    static constexpr uint32_t N = X == EQ_DTYPE_BF16 ? 4 : 2;
    uint32_t w[4 * N];
};

// `row` points at the tile's first column. left: columns that exist from
// there on (FULL: at least 128).
template <uint32_t X, uint32_t S, bool FULL>
__device__ __forceinline__ XFrag<X> load_x(const void *row, uint32_t quarter, uint32_t left) {
    XFrag<X> f;
    if constexpr (X == EQ_DTYPE_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(row);
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t at = word_col(S, quarter, j);
            u32x4 v = {0, 0, 0, 0};
            if (FULL || at + 8 <= left) {
                v = *reinterpret_cast<const u32x4_a2 *>(p + at);
            } else {
                for (uint32_t i = 0; i < 8; ++i)
                    if (at + i < left) v[i / 2] |= (uint32_t)p[at + i] << (16 * (i & 1));
            }
            for (int i = 0; i < 4; ++i) f.w[4 * j + i] = v[i];
        }
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(row);
        if constexpr (FULL && S >= 64) {
#pragma unroll
            for (uint32_t j = 0; j < 4; j += 2) {
                const u32x4 v = *reinterpret_cast<const u32x4_a1 *>(p + word_col(S, quarter, j));
                for (int i = 0; i < 4; ++i) f.w[2 * j + i] = v[i];
            }
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint32_t at = word_col(S, quarter, j);
                u32x2 v = {0, 0};
                if (FULL || at + 8 <= left) {
                    v = *reinterpret_cast<const u32x2_a1 *>(p + at);
                } else {
                    for (uint32_t i = 0; i < 8; ++i)
                        if (at + i < left) v[i / 4] |= (uint32_t)p[at + i] << (8 * (i & 3));
                }
                f.w[2 * j] = v[0];
                f.w[2 * j + 1] = v[1];
            }
        }
    }
    return f;
}

// One word of codes (8 weights of one row) as bf16.
template <uint32_t W, bool Z>
__device__ __forceinline__ u32x4 decode8(uint32_t w) {
    u32x4 r;
    if constexpr (W == EQ_DTYPE_INT4) {
        constexpr uint32_t bias = Z ? 0x41804180u : 0x41C041C0u;  // signed codes: the sign bit is flipped
        r[0] = ((w << 3) & 0x00780078u) ^ bias;
        r[1] = ((w >> 1) & 0x00780078u) ^ bias;
        r[2] = ((w >> 5) & 0x00780078u) ^ bias;
        r[3] = ((w >> 9) & 0x00780078u) ^ bias;
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
    }
    return r;
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ i32x4 mfma_i8x64(u32x4 a, u32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mfma_i8x32(u32x2 a, u32x2 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0, 0, 0);
}

// What a wave reads of one column of tiles: R rows of tiles, NT token tiles.
template <uint32_t X, uint32_t S, bool Z, int NT, int R>
struct Stage {
    u32x4 c[R];
    uint32_t s[R][2];  // bf16 scales of the lane's row: 128 / S of them
    uint32_t z[R];     // zeros, a byte each
    XFrag<X> x[NT];
};

template <uint32_t X, uint32_t S, bool Z, int NT, int R, bool FULL>
__device__ __forceinline__ void load_stage(Stage<X, S, Z, NT, R> &st, const W4Args &T, const u32x4 *codes,
                                           const uint16_t *scales, const uint8_t *zeros, const char *const *x_row,
                                           uint32_t kt, uint32_t k_tiles, uint32_t quarter) {
    constexpr uint32_t P = kTileCols / S;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint64_t tile = (uint64_t)r * k_tiles + kt;
        st.c[r] = __builtin_nontemporal_load(codes + tile * 64);
        const uint16_t *sp = scales + tile * 16 * P;
        if constexpr (P == 1) st.s[r][0] = *sp;
        else if constexpr (P == 2) st.s[r][0] = *reinterpret_cast<const uint32_t *>(sp);
        else {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(sp);
            st.s[r][0] = v[0];
            st.s[r][1] = v[1];
        }
        if constexpr (Z) {
            const uint8_t *zp = zeros + tile * 16 * P;
            if constexpr (P == 1) st.z[r] = *zp;
            else if constexpr (P == 2) st.z[r] = *reinterpret_cast<const uint16_t *>(zp);
            else st.z[r] = *reinterpret_cast<const uint32_t *>(zp);
        }
    }
    constexpr size_t XB = X == EQ_DTYPE_BF16 ? 2 : 1;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        st.x[n] = load_x<X, S, FULL>(x_row[n] + (uint64_t)kt * kTileCols * XB, quarter, T.cols - kt * kTileCols);
}

// acc += the stage's products.
template <uint32_t W, uint32_t X, uint32_t S, bool Z, int NT, int R>
__device__ __forceinline__ void compute(const Stage<X, S, Z, NT, R> &st, f32x4 (&acc)[NT][R]) {
    constexpr uint32_t P = kTileCols / S, J = 4 / P;  // groups of a tile, words of a lane per group
    auto scale = [&](int r, uint32_t g) {
        const uint32_t w = st.s[r][g / 2];
        return g & 1 ? bf16_hi(w) : bf16_lo(w);
    };
    auto zero = [&](int r, uint32_t g) { return (float)(st.z[r] >> (8 * g) & 255u); };
    if constexpr (X == EQ_DTYPE_INT8) {
#pragma unroll
        for (uint32_t g = 0; g < P; ++g) {
            u32x4 a[NT][(J + 1) / 2];  // a group's activations in the order of the code bytes (J = 1: half used)
            i32x4 sx[NT] = {};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                for (uint32_t j = 0; j < J; ++j) {
                    const uint32_t lo = st.x[n].w[2 * (g * J + j)], hi = st.x[n].w[2 * (g * J + j) + 1];
                    a[n][j / 2][2 * (j & 1)] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);      // columns 0 4 1 5
                    a[n][j / 2][2 * (j & 1) + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);  // columns 2 6 3 7
                }
                if constexpr (Z) {
                    constexpr uint32_t one = 0x01010101u;
                    if constexpr (J == 1) sx[n] = mfma_i8x32(u32x2{a[n][0][0], a[n][0][1]}, u32x2{one, one}, sx[n]);
                    else
                        for (uint32_t m = 0; m < J / 2; ++m) sx[n] = mfma_i8x64(a[n][m], u32x4{one, one, one, one}, sx[n]);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint32_t b[2 * J];
                for (uint32_t j = 0; j < J; ++j) {
                    const uint32_t w = st.c[r][g * J + j];
                    b[2 * j] = Z ? w & 0x0F0F0F0Fu : (w << 4) & 0xF0F0F0F0u;
                    b[2 * j + 1] = Z ? (w >> 4) & 0x0F0F0F0Fu : w & 0xF0F0F0F0u;
                }
                const float s = Z ? scale(r, g) : scale(r, g) * 0.0625f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    i32x4 d = {};
                    if constexpr (J == 1) d = mfma_i8x32(u32x2{a[n][0][0], a[n][0][1]}, u32x2{b[0], b[1]}, d);
                    else
                        for (uint32_t m = 0; m < J / 2; ++m)
                            d = mfma_i8x64(a[n][m], u32x4{b[4 * m], b[4 * m + 1], b[4 * m + 2], b[4 * m + 3]}, d);
                    for (int i = 0; i < 4; ++i) {
                        float v = (float)d[i];  // below 2^24: exact, as is the zeros' part
                        if constexpr (Z) v = fmaf(-zero(r, g), (float)sx[n][i], v);
                        acc[n][r][i] = fmaf(s, v, acc[n][r][i]);
                    }
                }
            }
        }
    } else {
        const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
        for (uint32_t g = 0; g < P; ++g) {
            f32x4 d[NT][R] = {}, sx[NT] = {};
#pragma unroll
            for (uint32_t j = g * J; j < (g + 1) * J; ++j) {
                u32x4 xa[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (X == EQ_DTYPE_BF16) {
                        for (int i = 0; i < 4; ++i) xa[n][i] = st.x[n].w[4 * j + i];
                    } else {
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t v = st.x[n].w[2 * j + i / 2];
                            xa[n][i] = __builtin_bit_cast(
                                uint32_t, i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true)
                                                : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
                        }
                    }
                    if constexpr (W == EQ_DTYPE_INT4) sx[n] = mfma_bf16(xa[n], ones, sx[n]);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const u32x4 b = decode8<W, Z>(st.c[r][j]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) d[n][r] = mfma_bf16(xa[n], b, d[n][r]);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float s = scale(r, g);
                float off = 24.0f;  // 16 + 8
                if constexpr (Z) off = 16.0f + zero(r, g);
                for (int n = 0; n < NT; ++n)
                    for (int i = 0; i < 4; ++i) {
                        const float v = W == EQ_DTYPE_INT4 ? fmaf(-off, sx[n][i], d[n][r][i]) : d[n][r][i];
                        acc[n][r][i] = fmaf(s, v, acc[n][r][i]);
                    }
            }
        }
    }
}

// A workgroup's 8 waves are (8 / k_waves) x k_waves: wave (rw, kw) owns R rows
// of tiles and every k_waves-th column of tiles, reads the next column's data
// while it computes one, and the k_waves partial sums are joined in LDS in
// wave order. Up to 16 * NT tokens.
template <uint32_t W, uint32_t X, uint32_t S, bool Z, int NT, int R>
__global__ void __launch_bounds__(64 * kWaves) k_w4(W4Launch a) {
    __shared__ f32x4 part[kWaves][R][64];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t i16 = lane & 15u, quarter = lane >> 4;
    uint32_t ti = 0;
    while (ti + 1 < a.n_tensors && blockIdx.x >= a.t[ti + 1].wg_begin) ++ti;
    const W4Args &T = a.t[ti];
    const uint32_t kw_n = T.k_waves, rw_n = kWaves / kw_n;
    const uint32_t rw = wave / kw_n, kw = wave % kw_n;
    const uint32_t row_tiles = (T.rows + kTileRows - 1) / kTileRows;
    const uint32_t k_tiles = (T.cols + kTileCols - 1) / kTileCols, k_full = T.cols / kTileCols;
    const uint32_t wg_tile = (blockIdx.x - T.wg_begin) * rw_n * R;
    const uint32_t token0 = blockIdx.y * kMaxTokens;
    constexpr size_t XB = X == EQ_DTYPE_BF16 ? 2 : 1;
    constexpr uint32_t P = kTileCols / S;

    const char *x_row[NT];
    for (int n = 0; n < NT; ++n) {
        // token rows past the end repeat the last one; their sums are not stored
        uint32_t t = token0 + n * 16 + i16;
        t = t < a.tokens ? t : a.tokens - 1;
        x_row[n] = static_cast<const char *>(T.x) + (uint64_t)t * T.ldx * XB;
    }
    // rows of tiles past the end: the wave computes its R rows from the last
    // R that exist (R <= row_tiles, see the launcher), stores skip them
    uint32_t tile0 = wg_tile + rw * R;
    tile0 = tile0 + R <= row_tiles ? tile0 : row_tiles - R;
    const uint64_t base = (uint64_t)tile0 * k_tiles;
    const u32x4 *codes = T.codes + base * 64 + lane;
    const uint16_t *scales = T.scales + (base * 16 + i16) * P;
    const uint8_t *zeros = Z ? T.zeros + (base * 16 + i16) * P : nullptr;

    f32x4 acc[NT][R] = {};
    using St = Stage<X, S, Z, NT, R>;
    auto load = [&](St &st, uint32_t kt) {
        load_stage<X, S, Z, NT, R, true>(st, T, codes, scales, zeros, x_row, kt, k_tiles, quarter);
    };
    uint32_t left = k_full > kw ? (k_full - kw + kw_n - 1) / kw_n : 0;  // whole tiles of this wave
    uint32_t kt = kw;
    if (left) {
        St st0, st1;
        load(st0, kt);
        while (left > 2) {
            load(st1, kt + kw_n);
            compute<W>(st0, acc);
            load(st0, kt + 2 * kw_n);
            compute<W>(st1, acc);
            kt += 2 * kw_n;
            left -= 2;
        }
        if (left == 2) {
            load(st1, kt + kw_n);
            compute<W>(st0, acc);
            compute<W>(st1, acc);
        } else {
            compute<W>(st0, acc);
        }
    }
    if (k_full < k_tiles && k_full % kw_n == kw) {  // the ragged last tile
        St st;
        load_stage<X, S, Z, NT, R, false>(st, T, codes, scales, zeros, x_row, k_full, k_tiles, quarter);
        compute<W>(st, acc);
    }

#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n) __syncthreads();
        for (int r = 0; r < R; ++r) part[wave][r][lane] = acc[n][r];
        __syncthreads();
        for (uint32_t o = wave; o < rw_n * R; o += kWaves) {
            const uint32_t orw = o / R, r = o % R;
            f32x4 s = part[orw * kw_n][r][lane];
            for (uint32_t w = 1; w < kw_n; ++w) s += part[orw * kw_n + w][r][lane];
            uint32_t t0 = wg_tile + orw * R;
            const bool moved = t0 + R > row_tiles;
            if (moved && (t0 >= row_tiles || row_tiles - R + r < t0)) continue;  // another wave's row of tiles
            if (moved) t0 = row_tiles - R;
            const uint32_t row = (t0 + r) * kTileRows + i16;
            for (int i = 0; i < 4; ++i) {
                const uint32_t t = token0 + n * 16 + quarter * 4 + i;
                if (t < a.tokens && row < T.rows) {
                    float v = s[i];
                    if constexpr (X != EQ_DTYPE_BF16) v *= T.x_scale[t];
                    if (a.y_f32) static_cast<float *>(T.y)[t * T.ldy + row] = v;
                    else static_cast<uint16_t *>(T.y)[t * T.ldy + row] = (uint16_t)pack_bf16(v, 0.0f);
                }
            }
        }
    }
}

typedef void (*W4Fn)(W4Launch);

template <uint32_t W, uint32_t X, bool Z, uint32_t S>
W4Fn pick_shape(uint32_t nt, uint32_t r) {
    if (nt == 1) return r == 1 ? k_w4<W, X, S, Z, 1, 1> : k_w4<W, X, S, Z, 1, 2>;
    if (nt == 2) return r == 1 ? k_w4<W, X, S, Z, 2, 1> : k_w4<W, X, S, Z, 2, 2>;
    return r == 1 ? k_w4<W, X, S, Z, 4, 1> : k_w4<W, X, S, Z, 4, 2>;
}
template <uint32_t W, uint32_t X, bool Z>
W4Fn pick_group(uint32_t group, uint32_t nt, uint32_t r) {
    if (group == 32) return pick_shape<W, X, Z, 32>(nt, r);
    if (group == 64) return pick_shape<W, X, Z, 64>(nt, r);
    return pick_shape<W, X, Z, 128>(nt, r);
}
W4Fn pick(uint32_t w, uint32_t x, bool z, uint32_t group, uint32_t nt, uint32_t r) {
    if (w == EQ_DTYPE_E2M1)
        return x == EQ_DTYPE_BF16 ? pick_group<EQ_DTYPE_E2M1, EQ_DTYPE_BF16, false>(group, nt, r)
                                  : pick_group<EQ_DTYPE_E2M1, EQ_DTYPE_E4M3, false>(group, nt, r);
    if (x == EQ_DTYPE_BF16)
        return z ? pick_group<EQ_DTYPE_INT4, EQ_DTYPE_BF16, true>(group, nt, r)
                 : pick_group<EQ_DTYPE_INT4, EQ_DTYPE_BF16, false>(group, nt, r);
    return z ? pick_group<EQ_DTYPE_INT4, EQ_DTYPE_INT8, true>(group, nt, r)
             : pick_group<EQ_DTYPE_INT4, EQ_DTYPE_INT8, false>(group, nt, r);
}

// Row-major codes, scales and zeros to tiles: one thread per 4-byte word of
// codes; the first 16 * (groups per tile) threads of a tile also place its
// scales and zeros.
__global__ void __launch_bounds__(256)
k_w4_pack(W4Args t, uint32_t e2m1, const uint8_t *__restrict__ src, const uint16_t *__restrict__ src_scales,
          const uint8_t *__restrict__ src_zeros, u32x4 *codes, uint16_t *scales, uint8_t *zeros) {
    const uint32_t k_tiles = (t.cols + kTileCols - 1) / kTileCols;
    const uint64_t tile = blockIdx.x;
    const uint32_t row_tile = (uint32_t)(tile / k_tiles), kt = (uint32_t)(tile % k_tiles);
    const uint64_t pitch = (t.cols + 1ull) / 2;
    const uint32_t lane = threadIdx.x >> 2, j = threadIdx.x & 3u;
    const uint32_t row = row_tile * kTileRows + (lane & 15u);
    const uint32_t k = kt * kTileCols + word_col(t.group, lane >> 4, j);
    uint32_t w = 0;
    for (uint32_t p = 0; p < 8; ++p) {
        const uint32_t c = k + (e2m1 ? p : p < 4 ? 2 * p : 2 * p - 7);
        if (row < t.rows && c < t.cols) w |= (uint32_t)((src[row * pitch + c / 2] >> (4 * (c & 1))) & 15u) << (4 * p);
    }
    reinterpret_cast<uint32_t *>(codes)[tile * 256 + threadIdx.x] = w;
    const uint32_t per_tile = kTileCols / t.group;
    if (threadIdx.x < 16 * per_tile) {
        const uint32_t r = row_tile * kTileRows + threadIdx.x / per_tile;
        const uint64_t g = (uint64_t)kt * per_tile + threadIdx.x % per_tile;
        const uint64_t groups = (t.cols + t.group - 1) / t.group;
        const bool there = r < t.rows && g < groups;
        const uint64_t at = tile * 16 * per_tile + threadIdx.x;
        scales[at] = there ? src_scales[r * groups + g] : (uint16_t)0;
        if (zeros) zeros[at] = there ? src_zeros[r * groups + g] : (uint8_t)0;
    }
}

constexpr uint64_t kMaxSide = 0x7FFFFFFFull;
constexpr uint64_t kMaxThreads = 0xFFFFFFFFull;  // of one grid dimension

uint64_t tiles(uint64_t rows, uint64_t cols) {
    return ((rows + kTileRows - 1) / kTileRows) * ((cols + kTileCols - 1) / kTileCols);
}
bool shape_ok(uint64_t rows, uint64_t cols) { return rows && cols && rows <= kMaxSide && cols <= kMaxSide; }
bool group_ok(uint32_t group) { return group == 32 || group == 64 || group == 128; }
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool tensor_ok(const eq_w4_tensor &t) {
    if (t.dtype != EQ_DTYPE_INT4 && t.dtype != EQ_DTYPE_E2M1) return false;
    if (!group_ok(t.group) || !shape_ok(t.rows, t.cols)) return false;
    if (!t.d_codes || !t.d_scales || (t.d_zeros && t.dtype == EQ_DTYPE_E2M1)) return false;
    return aligned(t.d_codes, 16) && aligned(t.d_scales, 8) && aligned(t.d_zeros, 4);
}

struct Shape {
    uint32_t nt, r;  // token tiles of 16 and rows of tiles per wave
};

// R: rows of tiles that share a wave's activations.
Shape shape(uint64_t tokens, uint64_t row_tiles, uint64_t fewest) {
    const uint32_t nt = tokens <= 16 ? 1 : tokens <= 32 ? 2 : 4;
    uint32_t r = tokens > 4 ? 2 : 1;
    while (r > 1 && (row_tiles < 512 * r || fewest < r)) r /= 2;
    return {nt, r};
}

// Waves that share out the columns: as many as have two tiles each.
uint32_t k_waves(uint64_t cols) {
    const uint64_t k_tiles = (cols + kTileCols - 1) / kTileCols;
    uint32_t n = kWaves;
    while (n > 1 && k_tiles < 2 * n) n /= 2;
    return n;
}

W4Args tensor_args(const eq_w4_tensor &t) {
    W4Args a{};
    a.codes = static_cast<const u32x4 *>(t.d_codes);
    a.scales = t.d_scales;
    a.zeros = t.d_zeros;
    a.rows = (uint32_t)t.rows;
    a.cols = (uint32_t)t.cols;
    a.group = t.group;
    return a;
}

}  // namespace

extern "C" {

uint64_t eq_w4_codes_bytes(uint64_t rows, uint64_t cols) {
    return shape_ok(rows, cols) ? tiles(rows, cols) * kTileBytes : 0;
}

uint64_t eq_w4_groups(uint64_t rows, uint64_t cols, uint32_t group) {
    return shape_ok(rows, cols) && group_ok(group) ? tiles(rows, cols) * kTileRows * (kTileCols / group) : 0;
}

eq_status eq_w4_pack(const eq_w4_tensor *t, const uint8_t *d_codes, const uint16_t *d_scales, const uint8_t *d_zeros,
                     void *stream) {
    if (!t || !tensor_ok(*t) || !d_codes || !d_scales || !aligned(d_scales, 2)) return EQ_EINVAL;
    if ((t->d_zeros == nullptr) != (d_zeros == nullptr)) return EQ_EINVAL;
    const uint64_t n = tiles(t->rows, t->cols);
    if (n > kMaxThreads / 256) return EQ_EINVAL;
    hipLaunchKernelGGL(k_w4_pack, dim3((uint32_t)n), dim3(256), 0, static_cast<hipStream_t>(stream), tensor_args(*t),
                       t->dtype == EQ_DTYPE_E2M1 ? 1u : 0u, d_codes, d_scales, d_zeros,
                       static_cast<u32x4 *>(t->d_codes), t->d_scales, t->d_zeros);
    return hipGetLastError() == hipSuccess ? EQ_OK : EQ_EHIP;
}

eq_status eq_w4_matvec(const eq_w4_tensor *tensors, uint32_t n_tensors, const eq_matrix *x, const eq_matrix *y,
                       uint64_t tokens, void *stream) {
    if (n_tensors == 0) return EQ_OK;
    if (!tensors || !x || !y || tokens > 65535ull * kMaxTokens) return EQ_EINVAL;
    for (uint32_t i = 0; i < n_tensors; ++i) {
        const eq_w4_tensor &t = tensors[i];
        if (!tensor_ok(t) || x[i].reserved || y[i].reserved) return EQ_EINVAL;
        if (y[i].dtype != EQ_DTYPE_F32 && y[i].dtype != EQ_DTYPE_BF16) return EQ_EINVAL;
        if (x[i].dtype != EQ_DTYPE_BF16 && x[i].dtype != EQ_DTYPE_INT8 && x[i].dtype != EQ_DTYPE_E4M3) return EQ_EINVAL;
        if (x[i].dtype != EQ_DTYPE_BF16 && x[i].dtype != (t.dtype == EQ_DTYPE_INT4 ? EQ_DTYPE_INT8 : EQ_DTYPE_E4M3))
            return EQ_EUNSUPPORTED;
        if (x[i].stride < t.cols || y[i].stride < t.rows || x[i].stride > (1ull << 40) || y[i].stride > (1ull << 40))
            return EQ_EINVAL;
        if (tokens == 0) continue;
        if (!x[i].d || !y[i].d || !aligned(y[i].d, y[i].dtype == EQ_DTYPE_F32 ? 4 : 2)) return EQ_EINVAL;
        if (x[i].dtype == EQ_DTYPE_BF16 ? !aligned(x[i].d, 2) : (!x[i].d_scale || !aligned(x[i].d_scale, 4)))
            return EQ_EINVAL;
    }
    if (tokens == 0) return EQ_OK;
    // one launch per kind (type, group, zeros, x and y types) and
    // EQ_MAX_BLOCK_TENSORS tensors; a tensor is launched with the first of its kind
    auto kind = [&](uint32_t i) {
        return tensors[i].dtype | x[i].dtype << 4 | y[i].dtype << 8 | (tensors[i].d_zeros ? 1u : 0u) << 12 |
               tensors[i].group << 16;
    };
    for (uint32_t first = 0; first < n_tensors; ++first) {
        uint32_t before = 0;  // tensors of this kind ahead of this one
        for (uint32_t i = 0; i < first; ++i) before += kind(i) == kind(first);
        if (before % EQ_MAX_BLOCK_TENSORS) continue;
        uint32_t which[EQ_MAX_BLOCK_TENSORS], n = 0;
        uint64_t total = 0, fewest = ~0ull;  // rows of tiles
        for (uint32_t i = first; i < n_tensors && n < EQ_MAX_BLOCK_TENSORS; ++i) {
            if (kind(i) != kind(first)) continue;
            which[n++] = i;
            const uint64_t rt = (tensors[i].rows + kTileRows - 1) / kTileRows;
            total += rt;
            fewest = rt < fewest ? rt : fewest;
        }
        const Shape sh = shape(tokens, total, fewest);
        W4Launch a{};
        uint64_t wgs = 0;
        for (; a.n_tensors < n; ++a.n_tensors) {
            const uint32_t i = which[a.n_tensors];
            W4Args &t = a.t[a.n_tensors];
            t = tensor_args(tensors[i]);
            t.x = x[i].d;
            t.x_scale = x[i].d_scale;
            t.y = y[i].d;
            t.ldx = x[i].stride;
            t.ldy = y[i].stride;
            t.wg_begin = (uint32_t)wgs;
            t.k_waves = k_waves(tensors[i].cols);
            const uint64_t per_wg = kWaves / t.k_waves * sh.r * kTileRows;
            wgs += (tensors[i].rows + per_wg - 1) / per_wg;
        }
        const uint64_t passes = (tokens + kMaxTokens - 1) / kMaxTokens;
        if (wgs > kMaxThreads / (64 * kWaves)) return EQ_EINVAL;
        a.tokens = (uint32_t)tokens;
        a.y_f32 = y[first].dtype == EQ_DTYPE_F32;
        hipLaunchKernelGGL(pick(tensors[first].dtype, x[first].dtype, tensors[first].d_zeros != nullptr,
                                tensors[first].group, sh.nt, sh.r),
                           dim3((uint32_t)wgs, (uint32_t)passes), dim3(64 * kWaves), 0,
                           static_cast<hipStream_t>(stream), a);
        if (hipGetLastError() != hipSuccess) return EQ_EHIP;
    }
    return EQ_OK;
}

}  // extern "C"
