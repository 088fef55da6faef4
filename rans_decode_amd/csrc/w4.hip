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
// What bounds it (graph replays over several copies of the weights): at one
// token HBM reads of the codes (two 28672 x 8192 INT4 matrices, int8 activations:
// 36.4 us, 6.6 TB/s; bf16: 37.8); at 16 tokens over few rows the activations,
// re-read from L2 by every workgroup (8192 x 28672 E2M1, E4M3: 24.3 us, 5.0 TB/s
// of codes); at 64 tokens reading the codes and computing alike, which hide each
// other only in part (the two matrices, int8: 56 us, 4.3 TB/s; see k_w4_wide);
// small matrices a launch and one memory latency (4096 x 4096, one token: 4.1 us).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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
    uint32_t k_tiles, row_tiles;  // columns and rows of tiles
    uint32_t kw_log2;             // 1 << kw_log2 waves share out the columns (k_w4)
    // a wave's rows of tiles: the kernel's R, or 1 where there are fewer than R (it
    // then computes that one R times and stores it once), and the step from one
    // to the next in tiles
    uint32_t wave_tiles, r_step;
    uint32_t group;
};

struct W4Launch {
    uint32_t wg_begin[EQ_MAX_BLOCK_TENSORS];  // first workgroup of each tensor, 2^32 - 1 past the last
    uint32_t tokens;
    uint32_t per_pass;  // tokens of a pass over the weights (grid y)
    uint32_t y_f32;
    W4Args t[EQ_MAX_BLOCK_TENSORS];
};

// The tensor of a workgroup. (One load of all the starts: walking them took a
// dependent load per tensor.)
__device__ __forceinline__ uint32_t tensor_of(const W4Launch &a, uint32_t wg) {
    uint32_t ti = 0;
#pragma unroll
    for (uint32_t i = 1; i < EQ_MAX_BLOCK_TENSORS; ++i) ti += wg >= a.wg_begin[i];
    return ti;
}

// Column within a tile of the first of the 8 weights in word j of a lane:
// word pairs hold 16 consecutive columns of a block of 64 (one 16-byte load of
// 8-bit activations), so that no matrix instruction mixes groups of 64; with
// groups of 32, words hold 8 of a block of 32.
__host__ __device__ constexpr uint32_t word_col(uint32_t group, uint32_t quarter, uint32_t j) {
    return group == 32 ? j * 32 + quarter * 8 : j / 2 * 64 + quarter * 16 + j % 2 * 8;
}

// One word of codes (8 weights of one row) as bf16.
template <uint32_t W, bool Z>
__device__ __forceinline__ u32x4 decode8(uint32_t w) {
    u32x4 r;
    if constexpr (W == EQ_DTYPE_INT4) {
        constexpr uint32_t mask = 0x00780078u;
        constexpr uint32_t bias = Z ? 0x41804180u : 0x41C041C0u;  // signed codes: the sign bit is flipped
        constexpr int kAndXor = (0xF0 & 0xCC) ^ 0xAA;             // (a & b) ^ c
        r[0] = __builtin_amdgcn_bitop3_b32(w << 3, mask, bias, kAndXor);
        r[1] = __builtin_amdgcn_bitop3_b32(w >> 1, mask, bias, kAndXor);
        r[2] = __builtin_amdgcn_bitop3_b32(w >> 5, mask, bias, kAndXor);
        r[3] = __builtin_amdgcn_bitop3_b32(w >> 9, mask, bias, kAndXor);
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
    }
    return r;
}

// 8 E4M3 values as bf16 (exact).
__device__ __forceinline__ u32x4 widen_e4m3(u32x2 v) {
    u32x4 o;
    for (int i = 0; i < 4; ++i)
        o[i] = __builtin_bit_cast(uint32_t, i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i / 2], 1.0f, true)
                                                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i / 2], 1.0f, false));
    return o;
}

// A kind of weight and activation: a lane's codes of a tile are Q pieces, one
// per matrix instruction; a group is PG pieces.
//   Raw: a lane's activations of a piece as loaded; Op: a matrix operand.
template <uint32_t W, uint32_t X, uint32_t S, bool Z>
struct Kind {  // bf16 products
    static constexpr uint32_t Q = 4, PG = S / 32;
    static constexpr bool kSumX = W == EQ_DTYPE_INT4;  // sum(x) is needed
    static constexpr float kScale = 1.0f;
    typedef typename std::conditional<X == EQ_DTYPE_BF16, u32x4, u32x2>::type Raw;
    typedef u32x4 Op;
    typedef f32x4 Sum;
    static __device__ __forceinline__ uint32_t col(uint32_t quarter, uint32_t p) { return word_col(S, quarter, p); }
    static __device__ __forceinline__ Op acts(Raw r) {
        if constexpr (X == EQ_DTYPE_BF16) {
            return r;
        } else {
            return widen_e4m3(r);
        }
    }
    static __device__ __forceinline__ Op codes(u32x4 c, uint32_t p) { return decode8<W, Z>(c[p]); }
    static __device__ __forceinline__ Op ones() { return Op{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}; }
    static __device__ __forceinline__ Sum mma(Op a, Op b, Sum c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    }
    static __device__ __forceinline__ float value(float d, float sum_x, float zero) {
        return kSumX ? fmaf(-(Z ? 16.0f + zero : 24.0f), sum_x, d) : d;
    }
};

template <uint32_t W, uint32_t S, bool Z>
struct KindE4M3x64 {  // E4M3 in groups of 64 or 128: 64 columns a piece, two instructions
    typedef Kind<W, EQ_DTYPE_BF16, S, Z> B;
    static constexpr uint32_t Q = 2, PG = S / 64;
    static constexpr bool kSumX = false;
    static constexpr float kScale = 1.0f;
    typedef u32x4 Raw;
    struct Op { u32x4 h[2]; };
    typedef f32x4 Sum;
    static __device__ __forceinline__ uint32_t col(uint32_t quarter, uint32_t p) { return word_col(S, quarter, 2 * p); }
    static __device__ __forceinline__ Op acts(Raw r) {
        return Op{{widen_e4m3(u32x2{r[0], r[1]}), widen_e4m3(u32x2{r[2], r[3]})}};
    }
    static __device__ __forceinline__ Op codes(u32x4 c, uint32_t p) { return Op{{B::codes(c, 2 * p), B::codes(c, 2 * p + 1)}}; }
    static __device__ __forceinline__ Op ones() { return Op{}; }
    static __device__ __forceinline__ Sum mma(Op a, Op b, Sum c) { return B::mma(a.h[1], b.h[1], B::mma(a.h[0], b.h[0], c)); }
    static __device__ __forceinline__ float value(float d, float, float) { return d; }
};
template <>
struct Kind<EQ_DTYPE_E2M1, EQ_DTYPE_E4M3, 64, false> : KindE4M3x64<EQ_DTYPE_E2M1, 64, false> {};
template <>
struct Kind<EQ_DTYPE_E2M1, EQ_DTYPE_E4M3, 128, false> : KindE4M3x64<EQ_DTYPE_E2M1, 128, false> {};

// int8 products. The bytes of a word's lower halves are columns 0 4 1 5 of its
// eight, those of its upper halves 2 6 3 7; activations are put in that order.
__device__ __forceinline__ u32x2 int8_order(uint32_t lo, uint32_t hi) {
    return u32x2{__builtin_amdgcn_perm(hi, lo, 0x05010400u), __builtin_amdgcn_perm(hi, lo, 0x07030602u)};
}
template <bool Z>
__device__ __forceinline__ u32x2 int8_codes(uint32_t w) {
    if (Z) return u32x2{w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu};
    return u32x2{(w << 4) & 0xF0F0F0F0u, w & 0xF0F0F0F0u};  // 16 q
}
template <bool Z>
__device__ __forceinline__ float int8_value(int32_t d, int32_t sum_x, float zero) {
    // |d| and |zero * sum_x| stay below 2^24: exact
    return Z ? fmaf(-zero, (float)sum_x, (float)d) : (float)d;
}

template <uint32_t S, bool Z>
struct Kind<EQ_DTYPE_INT4, EQ_DTYPE_INT8, S, Z> {  // 64 columns an instruction
    static constexpr uint32_t Q = 2, PG = S / 64;
    static constexpr bool kSumX = Z;
    static constexpr float kScale = Z ? 1.0f : 0.0625f;
    typedef u32x4 Raw;
    typedef u32x4 Op;
    typedef i32x4 Sum;
    static __device__ __forceinline__ uint32_t col(uint32_t quarter, uint32_t p) { return word_col(S, quarter, 2 * p); }
    static __device__ __forceinline__ Op acts(Raw r) {
        const u32x2 a = int8_order(r[0], r[1]), b = int8_order(r[2], r[3]);
        return Op{a[0], a[1], b[0], b[1]};
    }
    static __device__ __forceinline__ Op codes(u32x4 c, uint32_t p) {
        const u32x2 a = int8_codes<Z>(c[2 * p]), b = int8_codes<Z>(c[2 * p + 1]);
        return Op{a[0], a[1], b[0], b[1]};
    }
    static __device__ __forceinline__ Op ones() { return Op{0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u}; }
    static __device__ __forceinline__ Sum mma(Op a, Op b, Sum c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0,
                                                     0);
    }
    static __device__ __forceinline__ float value(int32_t d, int32_t sum_x, float zero) { return int8_value<Z>(d, sum_x, zero); }
};

template <bool Z>
struct Kind<EQ_DTYPE_INT4, EQ_DTYPE_INT8, 32, Z> {  // groups of 32: 32 columns an instruction
    static constexpr uint32_t Q = 4, PG = 1;
    static constexpr bool kSumX = Z;
    static constexpr float kScale = Z ? 1.0f : 0.0625f;
    typedef u32x2 Raw;
    typedef u32x2 Op;
    typedef i32x4 Sum;
    static __device__ __forceinline__ uint32_t col(uint32_t quarter, uint32_t p) { return word_col(32, quarter, p); }
    static __device__ __forceinline__ Op acts(Raw r) { return int8_order(r[0], r[1]); }
    static __device__ __forceinline__ Op codes(u32x4 c, uint32_t p) { return int8_codes<Z>(c[p]); }
    static __device__ __forceinline__ Op ones() { return Op{0x01010101u, 0x01010101u}; }
    static __device__ __forceinline__ Sum mma(Op a, Op b, Sum c) {
        return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float value(int32_t d, int32_t sum_x, float zero) { return int8_value<Z>(d, sum_x, zero); }
};

// Activations at p.
template <uint32_t X, typename Raw>
__device__ __forceinline__ Raw load_raw(const char *p) {
    if constexpr (X == EQ_DTYPE_BF16) return *reinterpret_cast<const u32x4_a2 *>(p);
    else if constexpr (sizeof(Raw) == 16) return *reinterpret_cast<const u32x4_a1 *>(p);
    else return *reinterpret_cast<const u32x2_a1 *>(p);
}

// The same from column `at` of a row of `cols`; what lies past its end reads
// as zero: the row's last values are loaded as one piece and shifted down.
// (Loaded value by value, each piece was waited for: 36 tokens of 91 columns
// took 13.5 us, so 12.7.)
template <uint32_t X, typename Raw>
__device__ __forceinline__ Raw load_raw_tail(const char *row, uint32_t at, uint32_t cols) {
    constexpr uint32_t XB = X == EQ_DTYPE_BF16 ? 2 : 1, N = sizeof(Raw) / XB, B = sizeof(Raw);
    if (cols < N) {  // rows shorter than a piece
        Raw r = {};
        for (uint32_t i = 0; i < N; ++i)
            if (at + i < cols) {
                const uint32_t v = XB == 2 ? reinterpret_cast<const uint16_t *>(row)[at + i]
                                           : reinterpret_cast<const uint8_t *>(row)[at + i];
                r[i * XB / 4] |= v << (8 * (i * XB % 4));
            }
        return r;
    }
    const uint32_t from = at < cols - N ? at : cols - N;
    const Raw v = load_raw<X, Raw>(row + (uint64_t)from * XB);
    const uint32_t by = (at - from) * XB;  // bytes to shift down; B or more: nothing is left
    uint64_t lo = (uint64_t)v[1] << 32 | v[0];
    if constexpr (B == 8) {
        lo = by < 8 ? lo >> (8 * by) : 0;
        return Raw{(uint32_t)lo, (uint32_t)(lo >> 32)};
    } else {
        uint64_t hi = (uint64_t)v[3] << 32 | v[2];
        if (by >= 8) {
            lo = by < 16 ? hi >> (8 * (by - 8)) : 0;
            hi = 0;
        } else if (by) {
            lo = lo >> (8 * by) | hi << (64 - 8 * by);
            hi >>= 8 * by;
        }
        return Raw{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
}

// What a wave reads of the weights of one column of tiles: R rows of tiles.
template <uint32_t S, bool Z, int R>
struct Weights {
    static constexpr uint32_t P = kTileCols / S;  // groups of a tile
    u32x4 c[R];
    uint32_t s[R][2];  // bf16 scales of the lane's row, one per group of the tile
    uint32_t z[R];     // zeros, a byte each

    // tile0: the first of the wave's rows of tiles, lane offsets apart from it
    // (a uniform base in scalar registers and one 32-bit offset per lane)
    __device__ __forceinline__ void load(const W4Args &T, uint64_t tile0, uint32_t kt, uint32_t r_step, uint32_t lane) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t tile = tile0 + (uint64_t)r * r_step + kt;
            c[r] = __builtin_nontemporal_load(T.codes + tile * 64 + lane);  // read once: plain loads took 8% longer
            const uint16_t *sp = T.scales + tile * 16 * P + (lane & 15u) * P;
            if constexpr (P == 1) s[r][0] = *sp;
            else if constexpr (P == 2) s[r][0] = *reinterpret_cast<const uint32_t *>(sp);
            else {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(sp);
                s[r][0] = v[0];
                s[r][1] = v[1];
            }
            if constexpr (Z) {
                const uint8_t *zp = T.zeros + tile * 16 * P + (lane & 15u) * P;
                if constexpr (P == 1) z[r] = *zp;
                else if constexpr (P == 2) z[r] = *reinterpret_cast<const uint16_t *>(zp);
                else z[r] = *reinterpret_cast<const uint32_t *>(zp);
            }
        }
    }
    __device__ __forceinline__ float scale(int r, uint32_t g) const {
        const uint32_t w = P == 4 ? (g & 2 ? s[r][1] : s[r][0]) : s[r][0];
        return P == 1 || !(g & 1) ? bf16_lo(w) : bf16_hi(w);
    }
    __device__ __forceinline__ float zero(int r, uint32_t g) const {
        return Z ? (float)(P == 1 ? z[r] : z[r] >> (8 * g) & 255u) : 0.0f;
    }
};

__device__ __forceinline__ bool not_finite(float v) { return !(fabsf(v) < __builtin_inff()); }

__device__ __forceinline__ void store_y(const W4Args &T, bool f32, uint32_t t, uint32_t row, float v) {
    if (f32) static_cast<float *>(T.y)[t * T.ldy + row] = v;
    else static_cast<uint16_t *>(T.y)[t * T.ldy + row] = (uint16_t)pack_bf16(v, 0.0f);
}

// bf16 activations reach to 2^128, so the sums of a group, taken before its
// scale and with a code's bias, can overflow (from |x| of 2^116 on, with zeros
// from 2^112; E2M1 2^118) or meet an infinity in x that the bias turns into
// inf - inf, although W x is a number or one infinity. A wave whose outputs are
// not all finite therefore looks at them again (y[t, its rows of one tile])
// and sums those with W = (q - zero) * scale itself, which fp32 holds exactly:
// lane (row, quarter) takes the words that it loads in the products, and the
// four quarters join in order. A NaN in x's row leaves nothing to look for.
// The check, one comparison per output, costs up to 2% (64 tokens x 11008 x
// 4096, group 32: 33.3 us, 32.6 without; one token within noise). One token
// through 57344 x 8192: 36 us, with an infinity in x 231, with a NaN 50.
template <uint32_t W, uint32_t S, bool Z>
__device__ __forceinline__ void sum_again(const W4Args &T, bool f32, uint32_t t, uint32_t row_tile) {
    constexpr uint32_t P = kTileCols / S;
    // counted anew, and another value to the compiler than the products' lane:
    // what the two shared was kept in registers all through the products
    uint32_t lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
    asm volatile("" : "+v"(lane));
    const uint32_t i16 = lane & 15u, quarter = lane >> 4, row = row_tile * kTileRows + i16;
    bool bad = false;
    if (row < T.rows) {
        const uint64_t at = t * T.ldy + row;
        bad = not_finite(f32 ? static_cast<const float *>(T.y)[at] : bf16_lo(static_cast<const uint16_t *>(T.y)[at]));
    }
    if (!__any(bad)) return;
    const char *x = static_cast<const char *>(T.x) + (uint64_t)t * T.ldx * 2;
    bool nan = false;
    for (uint64_t c = lane; c < T.cols; c += 64) nan |= (reinterpret_cast<const uint16_t *>(x)[c] & 0x7FFFu) > 0x7F80u;
    if (__any(nan)) return;
    float sum = 0.0f;
#pragma unroll 1
    for (uint32_t kt = 0; kt < T.k_tiles; ++kt) {
        const uint64_t tile = (uint64_t)row_tile * T.k_tiles + kt;
        float tile_sum = 0.0f;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {  // (unrolled it took more registers than the products)
            const uint32_t word = reinterpret_cast<const uint32_t *>(T.codes + tile * 64 + lane)[j];
            const uint32_t col = word_col(S, quarter, j);
            const uint64_t g = (tile * kTileRows + i16) * P + col / S;
            const float scale = bf16_lo(T.scales[g]);
            const int32_t zero = Z ? T.zeros[g] : 0;
            const u32x4 v = load_raw_tail<EQ_DTYPE_BF16, u32x4>(x, kt * kTileCols + col, T.cols);
            const u32x4 floats = decode8<W, Z>(word);  // E2M1's values
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                float q;
                if constexpr (W == EQ_DTYPE_INT4) {
                    const uint32_t up = word << (28 - 4 * (k % 2 * 4 + k / 2));  // the code in the upper 4 bits
                    q = (float)(Z ? (int32_t)(up >> 28) - zero : (int32_t)up >> 28);
                } else {
                    q = k % 2 ? bf16_hi(floats[k / 2]) : bf16_lo(floats[k / 2]);
                }
                const float xv = k % 2 ? bf16_hi(v[k / 2]) : bf16_lo(v[k / 2]);
                // columns past the end have x = 0 and, in whole groups, scale 0
                tile_sum = fmaf(q * scale, xv, tile_sum);
            }
        }
        sum += tile_sum;
    }
    float total = 0.0f;
    for (uint32_t k = 0; k < 4; ++k) total += __shfl(sum, (int)(k * 16 + i16));
    if (bad && quarter == 0) store_y(T, f32, t, row, total);
}

// A wave's LDS accesses are performed in program order; this keeps the compiler
// from changing that order where lanes exchange values.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// A workgroup's 8 waves are (8 / k_waves) x k_waves: wave (rw, kw) owns R rows
// of tiles and every k_waves-th column of tiles; D columns of its data are on
// their way while it computes, and the k_waves partial sums are joined in LDS
// in wave order.
//
// TP tokens share a matrix instruction's 16 rows of A: with TP < 16 row
// m = LJ t + jj holds token t and piece jj of every LJ = 16 / TP pieces, so that
// one load brings several pieces and few tokens cost few loads (one token of
// bf16 took 4 loads a tile, each as large as the codes' own, and bounded the
// kernel). Every piece's instruction then computes all rows; those of its own
// piece are, with rows 4 quarter + i in registers i of a quarter wave, the
// registers i = jj mod LJ, which alone are scaled and added up. TP = 4 keeps one
// token per lane, TP = 8 two, TP = 16 four. NT > 1 (TP = 16): up to 16 * NT
// tokens.
//
// TP = 16: a load whose neighbouring lanes read 16 different rows takes the
// cache 64 look-ups, one whose 4 neighbours read 64 consecutive bytes 16; so
// lanes load in that order, lane = 4 row + quarter, and swap through LDS (a
// wave's own slots: no barrier). The slots are rotated by 4 per quarter; with
// 16-byte pieces that does not free both sides of bank conflicts (counted: 1.4e6
// cycles, 2.2 us a compute unit, in the 24.3 us of 16 tokens E4M3 x 8192 x 28672).
template <uint32_t W, uint32_t X, uint32_t S, bool Z, int TP, int NT, int R, int D>
__global__ void __launch_bounds__(64 * kWaves) k_w4(W4Launch a) {
    typedef Kind<W, X, S, Z> K;
    constexpr uint32_t XB = X == EQ_DTYPE_BF16 ? 2 : 1;
    constexpr uint32_t LJ = 16 / TP;                      // pieces per load
    constexpr uint32_t NL = K::Q / LJ;                    // loads per tile
    constexpr uint32_t F = K::PG > LJ ? K::PG / LJ : 1;   // loads that share a lane's group
    static_assert(NL >= 1 && NL % F == 0 && (NT == 1 || TP == 16), "tokens, pieces and groups fit");
    constexpr uint32_t NI = 4 / LJ;                       // tokens a lane keeps sums of, per token tile
    typedef float Acc __attribute__((ext_vector_type(NI)));
    __shared__ Acc part[kWaves][R][64];
    __shared__ typename K::Raw swap[TP == 16 ? kWaves : 1][TP == 16 ? NL : 1][64];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t i16 = lane & 15u, quarter = lane >> 4;
    // where this lane's loads come from, and its slots for swapping them
    const uint32_t load_row = TP == 16 ? lane >> 2 : i16, load_quarter = TP == 16 ? lane & 3u : quarter;
    const uint32_t put = load_quarter * 16 + ((load_row + 4 * load_quarter) & 15u);
    const uint32_t get = quarter * 16 + ((i16 + 4 * quarter) & 15u);
    const uint32_t ti = tensor_of(a, blockIdx.x);
    const W4Args &T = a.t[ti];
    const uint32_t kw_n = 1u << T.kw_log2, rw_n = kWaves >> T.kw_log2;
    const uint32_t rw = wave >> T.kw_log2, kw = wave & (kw_n - 1);
    const uint32_t row_tiles = T.row_tiles, k_tiles = T.k_tiles, k_full = T.cols / kTileCols;
    const uint32_t wave_tiles = T.wave_tiles, r_step = T.r_step;
    const uint32_t wg_tile = (blockIdx.x - a.wg_begin[ti]) * rw_n * wave_tiles;
    const uint32_t token0 = blockIdx.y * a.per_pass;

    const char *x_row[NT];
    for (int n = 0; n < NT; ++n) {
        // token rows past the end repeat the last one; their sums are not stored
        uint32_t t = token0 + n * 16 + load_row / LJ;
        t = t < a.tokens ? t : a.tokens - 1;
        x_row[n] = static_cast<const char *>(T.x) + (uint64_t)t * T.ldx * XB;
    }
    uint32_t x_col[NL];
    for (uint32_t l = 0; l < NL; ++l) x_col[l] = K::col(load_quarter, l * LJ + load_row % LJ);
    // rows of tiles past the end: the wave computes its rows from the last ones
    // that exist (wave_tiles <= row_tiles, see the launcher), stores skip them
    uint32_t tile0 = wg_tile + rw * wave_tiles;
    tile0 = tile0 + wave_tiles <= row_tiles ? tile0 : row_tiles - wave_tiles;
    const uint64_t base = (uint64_t)tile0 * k_tiles;

    struct St {  // what the wave reads of one column of tiles
        Weights<S, Z, R> w;
        typename K::Raw x[NT][NL];
    };
    auto load = [&](St &st, uint32_t kt) {
        st.w.load(T, base, kt, r_step, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            for (uint32_t l = 0; l < NL; ++l)
                st.x[n][l] = load_raw<X, typename K::Raw>(x_row[n] + ((uint64_t)kt * kTileCols + x_col[l]) * XB);
    };
    auto load_tail = [&](St &st, uint32_t kt) {
        st.w.load(T, base, kt, r_step, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            for (uint32_t l = 0; l < NL; ++l)
                st.x[n][l] = load_raw_tail<X, typename K::Raw>(x_row[n], kt * kTileCols + x_col[l], T.cols);
    };

    Acc acc[NT][R] = {};
    auto compute = [&](const St &st) {
#pragma unroll
        for (uint32_t f = 0; f < NL / F; ++f) {
            typename K::Sum d[NT][R][LJ] = {}, sx[NT] = {};
#pragma unroll
            for (uint32_t l = f * F; l < (f + 1) * F; ++l) {
                typename K::Op xa[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (TP == 16) {
                        swap[wave][l][put] = st.x[n][l];
                        wave_order();
                        xa[n] = K::acts(swap[wave][l][get]);
                        wave_order();
                    } else {
                        xa[n] = K::acts(st.x[n][l]);
                    }
                    if constexpr (K::kSumX) sx[n] = K::mma(xa[n], K::ones(), sx[n]);
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (uint32_t jj = 0; jj < LJ; ++jj) {
                        const typename K::Op b = K::codes(st.w.c[r], l * LJ + jj);
#pragma unroll
                        for (int n = 0; n < NT; ++n) d[n][r][jj] = K::mma(xa[n], b, d[n][r][jj]);
                    }
            }
#pragma unroll
            for (uint32_t jj = 0; jj < LJ; ++jj) {
                const uint32_t g = (f * F * LJ + jj) / K::PG;  // the group of this piece (of all F loads)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float s = st.w.scale(r, g) * K::kScale, zero = st.w.zero(r, g);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        for (uint32_t i = 0; i < NI; ++i) {
                            const uint32_t at = i * LJ + jj;
                            acc[n][r][i] = fmaf(s, K::value(d[n][r][jj][at], sx[n][at], zero), acc[n][r][i]);
                        }
                }
            }
        }
    };

    const uint32_t n_tiles = k_full > kw ? (k_full - kw + kw_n - 1) >> T.kw_log2 : 0;  // whole tiles of this wave
    if (n_tiles) {
        St st[D];
        // a tile past the last is the last again: it is not computed
        auto column = [&](uint32_t i) { return kw + ((i < n_tiles ? i : n_tiles - 1) << T.kw_log2); };
#pragma unroll
        for (uint32_t d = 0; d < D; ++d) load(st[d], column(d));
        uint32_t i = 0;
        for (; i + D < n_tiles; i += D) {
#pragma unroll
            for (uint32_t d = 0; d < D; ++d) {
                compute(st[d]);
                __builtin_amdgcn_sched_barrier(0);
                load(st[d], column(i + D + d));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (uint32_t d = 0; d < D; ++d)
            if (i + d < n_tiles) compute(st[d]);
    }
    if (k_full < k_tiles && (k_full & (kw_n - 1)) == kw) {  // the ragged last tile
        St st;
        load_tail(st, k_full);
        compute(st);
    }

    // the row of tiles of the workgroup's o-th output, none where it is another's
    constexpr uint32_t kNone = ~0u;
    auto row_tile_of = [&](uint32_t o) -> uint32_t {
        const uint32_t r = o % R, t0 = wg_tile + o / R * wave_tiles;
        if (r >= wave_tiles || t0 >= row_tiles) return kNone;
        if (t0 + wave_tiles <= row_tiles) return t0 + r;
        return row_tiles - wave_tiles + r < t0 ? kNone : row_tiles - wave_tiles + r;
    };
    bool bad = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n) __syncthreads();
        for (int r = 0; r < R; ++r) part[wave][r][lane] = acc[n][r];
        __syncthreads();
        for (uint32_t o = wave; o < rw_n * R; o += kWaves) {
            const uint32_t row_tile = row_tile_of(o);
            if (row_tile == kNone) continue;
            Acc s = {};
            for (uint32_t w = 0; w < kw_n; ++w) s += part[o / R * kw_n + w][o % R][lane];
            const uint32_t row = row_tile * kTileRows + i16;
            for (uint32_t i = 0; i < NI; ++i) {
                const uint32_t t = token0 + n * 16 + quarter * NI + i;
                if (t < a.tokens && row < T.rows) {
                    float v = s[i];
                    if constexpr (X != EQ_DTYPE_BF16) v *= T.x_scale[t];
                    store_y(T, a.y_f32, t, row, v);
                    bad |= not_finite(v);
                }
            }
        }
    }
    if constexpr (X == EQ_DTYPE_BF16) {
        if (__any(bad)) {
            __threadfence_block();  // lanes read what others of the wave stored
            const uint32_t end = token0 + TP * NT < a.tokens ? token0 + TP * NT : a.tokens;
#pragma unroll 1
            for (uint32_t o = wave; o < rw_n * R; o += kWaves) {
                const uint32_t row_tile = row_tile_of(o);
                if (row_tile == kNone) continue;
#pragma unroll 1
                for (uint32_t t = token0; t < end; ++t) sum_again<W, S, Z>(T, a.y_f32, t, row_tile);
            }
        }
    }
}

// Many rows and more than a few tokens: the activations, read by every row of
// tiles, outweigh the codes (64 tokens of int8 are 8 KiB a column of tiles
// against R KiB of codes), so the 8 waves of a workgroup, R rows of tiles
// each, share them: a chunk of kChunkTiles columns of tiles is put in LDS as
// matrix operands while the chunk before it is computed (two buffers, one
// barrier a chunk), and the codes of a whole chunk are on their way.
// Measured, two 28672 x 8192 INT4 matrices, group 128, 64 tokens int8: 55 to 58
// us (k_w4 114). With the rest of the loop left out: loads of codes and scales 51
// (with those of the activations 49), products and activations 48, products
// alone 43. Each is most of the whole, and the one workgroup that a compute unit
// holds by its registers (224 for 256 units) overlaps them only in part. Per chunk
// and wave 64 matrix instructions and about 440 vector ones (a conversion and a
// multiply-add per sum and group), of which a matrix instruction hides only about
// two; the swap's bank conflicts are 4.6e6 cycles, 7.6 us a unit.
constexpr uint32_t kChunkTiles = 4;

// (E2M1 x bf16 with two token tiles fits twice on a compute unit with 128
// registers; left alone the compiler takes 128 or 130.)
template <uint32_t W, uint32_t X, uint32_t S, bool Z, int NT, int R>
__global__ void __launch_bounds__(64 * kWaves, W == EQ_DTYPE_E2M1 && X == EQ_DTYPE_BF16 && NT == 2 ? 4 : 2)
k_w4_wide(W4Launch a) {
    // KS: how a lane loads activations; K: how it multiplies
    typedef Kind<W, X, S, Z> KS;
    typedef Kind<W, X == EQ_DTYPE_E4M3 ? EQ_DTYPE_BF16 : X, S, Z> K;
    constexpr uint32_t XB = X == EQ_DTYPE_BF16 ? 2 : 1;
    constexpr uint32_t P = kTileCols / S, C = kChunkTiles;
    constexpr uint32_t kOps = K::Q / KS::Q;            // operands from one load (1, or 2 for E4M3 x 64)
    constexpr uint32_t kLoads = C * NT * KS::Q / kWaves;  // a wave's loads for a chunk
    static_assert(kLoads >= 1 && C * NT * KS::Q % kWaves == 0, "waves share out a chunk's loads evenly");
    // sum(x) of every token and group, by the wave that stages it (where one
    // wave stages whole token tiles); one matrix instruction per piece and wave
    // otherwise
    constexpr bool kSums = K::kSumX && kLoads % KS::Q == 0;
    __shared__ typename K::Op xs[2][C][NT][K::Q][64];
    __shared__ typename K::Sum xsum[2][C][NT][P][kSums ? 4 : 1];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t i16 = lane & 15u, quarter = lane >> 4;
    const uint32_t ti = tensor_of(a, blockIdx.x);
    const W4Args &T = a.t[ti];
    const uint32_t row_tiles = T.row_tiles, k_tiles = T.k_tiles;
    const uint32_t chunks = T.cols / (C * kTileCols);  // whole ones
    const uint32_t token0 = blockIdx.y * a.per_pass;
    const uint32_t wave_tiles = T.wave_tiles, r_step = T.r_step;
    const uint32_t want = ((blockIdx.x - a.wg_begin[ti]) * kWaves + wave) * wave_tiles;  // as in k_w4
    const uint32_t tile0 = want + wave_tiles <= row_tiles ? want : row_tiles - wave_tiles;
    const uint64_t base = (uint64_t)tile0 * k_tiles;

    // the wave's loads of a chunk: (tile, token tile, piece) triples, in the
    // lane order of k_w4's TP = 16 (not where the sums are taken from the
    // registers, which want operand order); operands lie in its slots
    const uint32_t load_row = kSums ? i16 : lane >> 2, load_quarter = kSums ? quarter : lane & 3u;
    const uint32_t put = load_quarter * 16 + ((load_row + 4 * load_quarter) & 15u);
    const uint32_t get = quarter * 16 + ((i16 + 4 * quarter) & 15u);
    const char *x_at[kLoads];
    uint32_t x_col[kLoads], x_to[kLoads];
    for (uint32_t i = 0; i < kLoads; ++i) {
        const uint32_t k = wave * kLoads + i, p = k % KS::Q, n = k / KS::Q % NT, tile = k / KS::Q / NT;
        uint32_t t = token0 + n * 16 + load_row;
        t = t < a.tokens ? t : a.tokens - 1;
        x_col[i] = tile * kTileCols + KS::col(load_quarter, p);
        x_at[i] = static_cast<const char *>(T.x) + ((uint64_t)t * T.ldx + x_col[i]) * XB;
        x_to[i] = (tile * NT + n) * K::Q + p * kOps;
    }
    typename KS::Raw raw[kLoads];
    auto load_x = [&](uint32_t chunk) {
        for (uint32_t i = 0; i < kLoads; ++i)
            raw[i] = load_raw<X, typename KS::Raw>(x_at[i] + (uint64_t)chunk * (C * kTileCols * XB));
    };
    auto put_x = [&](uint32_t buf) {
        typename K::Op(*to)[64] = &xs[buf][0][0][0];
        [[maybe_unused]] typename K::Sum sx = {};
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i) {
            const auto o = KS::acts(raw[i]);
            if constexpr (kOps == 2) {
                to[x_to[i]][put] = o.h[0];
                to[x_to[i] + 1][put] = o.h[1];
            } else {
                to[x_to[i]][put] = o;
                if constexpr (kSums) {
                    sx = i % K::PG ? K::mma(o, K::ones(), sx) : K::mma(o, K::ones(), typename K::Sum{});
                    // every column of the result is the sums; column 0 stores them
                    if (i % K::PG == K::PG - 1 && i16 == 0) (&xsum[buf][0][0][0][0])[(x_to[i] / K::PG) * 4 + quarter] = sx;
                }
            }
        }
    };

    f32x4 acc[NT][R] = {};
    auto compute = [&](const Weights<S, Z, R> &w, uint32_t buf, uint32_t tile) {
#pragma unroll
        for (uint32_t g = 0; g < P; ++g) {
            typename K::Op b[K::PG][R], xa[2][K::PG];
            float s[R], zero[R];
            [[maybe_unused]] typename K::Sum sn[3];
            auto fetch = [&](int n) {
                for (uint32_t p = 0; p < K::PG; ++p) xa[n & 1][p] = xs[buf][tile][n][g * K::PG + p][get];
                if constexpr (kSums) sn[n % 3] = xsum[buf][tile][n][g][quarter];
            };
            fetch(0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                for (uint32_t p = 0; p < K::PG; ++p) b[p][r] = K::codes(w.c[r], g * K::PG + p);
                s[r] = w.scale(r, g) * K::kScale;
                zero[r] = w.zero(r, g);
            }
            // one token tile's sums are scaled while the next one's products run
            typename K::Sum d[2][R], sx[2];
#pragma unroll
            for (int n = 0; n <= NT; ++n) {
                if (n + 1 < NT) fetch(n + 1);
                if (n < NT) {
                    sx[n & 1] = typename K::Sum{};
                    if constexpr (kSums) sx[n & 1] = sn[n % 3];
                    for (int r = 0; r < R; ++r) d[n & 1][r] = typename K::Sum{};
                    for (uint32_t p = 0; p < K::PG; ++p) {
                        if constexpr (K::kSumX && !kSums) sx[n & 1] = K::mma(xa[n & 1][p], K::ones(), sx[n & 1]);
                        for (int r = 0; r < R; ++r) d[n & 1][r] = K::mma(xa[n & 1][p], b[p][r], d[n & 1][r]);
                    }
                }
                if (n > 0)
                    for (int r = 0; r < R; ++r)
                        for (int i = 0; i < 4; ++i)
                            acc[n - 1][r][i] = fmaf(s[r], K::value(d[~n & 1][r][i], sx[~n & 1][i], zero[r]), acc[n - 1][r][i]);
            }
        }
    };

    Weights<S, Z, R> w[C];
    const uint32_t ragged = chunks * C;  // first column of tiles of the last, short chunk
    auto load_w = [&](Weights<S, Z, R> &d, uint32_t kt) { d.load(T, base, kt < k_tiles ? kt : k_tiles - 1, r_step, lane); };
#pragma unroll
    for (uint32_t d = 0; d < C; ++d) load_w(w[d], d);
    if (chunks) {
        load_x(0);
        put_x(0);
    }
    __syncthreads();
    // All workgroups walk the columns in the same order: the activations of a
    // chunk are then in L2 for all of them (started at different chunks, they
    // took 15% longer). The fences keep loads where they are issued: moved
    // down to the end of a chunk they were waited for at the start of the next.
    for (uint32_t ch = 0; ch < chunks; ++ch) {
        load_x(ch + 1 < chunks ? ch + 1 : ch);  // the last one again: not used
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (uint32_t d = 0; d < C; ++d) {
            compute(w[d], ch & 1, d);
            for (int n = 0; n < NT; ++n)
                for (int r = 0; r < R; ++r) asm volatile("" : "+v"(acc[n][r]));
            __builtin_amdgcn_sched_barrier(0);
            load_w(w[d], (ch + 1) * C + d);
            __builtin_amdgcn_sched_barrier(0);
        }
        put_x(~ch & 1);
        __syncthreads();
    }
    if (ragged < k_tiles) {
        for (uint32_t i = 0; i < kLoads; ++i)
            raw[i] = load_raw_tail<X, typename KS::Raw>(x_at[i] - (uint64_t)x_col[i] * XB, ragged * kTileCols + x_col[i], T.cols);
        put_x(0);
        __syncthreads();
#pragma unroll
        for (uint32_t d = 0; d < C; ++d)
            if (ragged + d < k_tiles) compute(w[d], 0, d);
    }
    bool bad = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t row = (tile0 + r) * kTileRows + i16;
        if (r >= (int)wave_tiles || tile0 + r < want || row >= T.rows) continue;  // another wave's row of tiles, or none
#pragma unroll
        for (int n = 0; n < NT; ++n)
            for (int i = 0; i < 4; ++i) {
                const uint32_t t = token0 + n * 16 + quarter * 4 + i;
                if (t < a.tokens) {
                    const float v = X == EQ_DTYPE_BF16 ? acc[n][r][i] : acc[n][r][i] * T.x_scale[t];
                    store_y(T, a.y_f32, t, row, v);
                    bad |= not_finite(v);
                }
            }
    }
    if constexpr (X == EQ_DTYPE_BF16) {
        if (__any(bad)) {
            __threadfence_block();  // lanes read what others of the wave stored
            const uint32_t end = token0 + 16 * NT < a.tokens ? token0 + 16 * NT : a.tokens;
#pragma unroll 1
            for (uint32_t r = 0; r < wave_tiles; ++r) {
                if (tile0 + r < want) continue;
#pragma unroll 1
                for (uint32_t t = token0; t < end; ++t) sum_again<W, S, Z>(T, a.y_f32, t, tile0 + r);
            }
        }
    }
}

typedef void (*W4Fn)(W4Launch);

template <uint32_t W, uint32_t X, bool Z, uint32_t S>
W4Fn pick_shape(uint32_t nt, uint32_t tp, uint32_t r, bool wide) {
    if (wide) {
        if (nt == 1) return k_w4_wide<W, X, S, Z, 1, 2>;
        if (nt == 2) return r == 1 ? k_w4_wide<W, X, S, Z, 2, 1> : k_w4_wide<W, X, S, Z, 2, 2>;
        return r == 1 ? k_w4_wide<W, X, S, Z, 4, 1> : k_w4_wide<W, X, S, Z, 4, 2>;
    }
    if (tp == 4) {
        if constexpr (Kind<W, X, S, Z>::Q == 4) return r == 1 ? k_w4<W, X, S, Z, 4, 1, 1, 4> : k_w4<W, X, S, Z, 4, 1, 2, 2>;
        tp = 8;  // 64 columns a piece: two pieces a load
    }
    if (tp == 8) return r == 1 ? k_w4<W, X, S, Z, 8, 1, 1, 4> : k_w4<W, X, S, Z, 8, 1, 2, 2>;
    if (nt == 1) return r == 1 ? k_w4<W, X, S, Z, 16, 1, 1, 2> : r == 2 ? k_w4<W, X, S, Z, 16, 1, 2, 2> : k_w4<W, X, S, Z, 16, 1, 4, 2>;
    if (nt == 2) return r == 1 ? k_w4<W, X, S, Z, 16, 2, 1, 2> : r == 2 ? k_w4<W, X, S, Z, 16, 2, 2, 2> : k_w4<W, X, S, Z, 16, 2, 4, 2>;
    return r == 1 ? k_w4<W, X, S, Z, 16, 4, 1, 2> : k_w4<W, X, S, Z, 16, 4, 2, 2>;
}
template <uint32_t W, uint32_t X, bool Z>
W4Fn pick_group(uint32_t group, uint32_t nt, uint32_t tp, uint32_t r, bool wide) {
    if (group == 32) return pick_shape<W, X, Z, 32>(nt, tp, r, wide);
    if (group == 64) return pick_shape<W, X, Z, 64>(nt, tp, r, wide);
    return pick_shape<W, X, Z, 128>(nt, tp, r, wide);
}
W4Fn pick(uint32_t w, uint32_t x, bool z, uint32_t group, uint32_t nt, uint32_t tp, uint32_t r, bool wide) {
    if (w == EQ_DTYPE_E2M1)
        return x == EQ_DTYPE_BF16 ? pick_group<EQ_DTYPE_E2M1, EQ_DTYPE_BF16, false>(group, nt, tp, r, wide)
                                  : pick_group<EQ_DTYPE_E2M1, EQ_DTYPE_E4M3, false>(group, nt, tp, r, wide);
    if (x == EQ_DTYPE_BF16)
        return z ? pick_group<EQ_DTYPE_INT4, EQ_DTYPE_BF16, true>(group, nt, tp, r, wide)
                 : pick_group<EQ_DTYPE_INT4, EQ_DTYPE_BF16, false>(group, nt, tp, r, wide);
    return z ? pick_group<EQ_DTYPE_INT4, EQ_DTYPE_INT8, true>(group, nt, tp, r, wide)
             : pick_group<EQ_DTYPE_INT4, EQ_DTYPE_INT8, false>(group, nt, tp, r, wide);
}

// Row-major codes, scales and zeros to tiles: a workgroup per tile, a thread
// per word, reading its 8 columns as they lie (one u32 where rows are 4-byte
// aligned); the first 16 * (groups per tile) threads also place the tile's
// scales and zeros.
__global__ void __launch_bounds__(256)
k_w4_pack(W4Args t, uint32_t e2m1, const uint8_t *__restrict__ src, const uint16_t *__restrict__ src_scales,
          const uint8_t *__restrict__ src_zeros, uint32_t *codes, uint16_t *scales, uint8_t *zeros) {
    const uint32_t k_tiles = t.k_tiles;
    const uint64_t tile = blockIdx.x;
    const uint32_t row_tile = (uint32_t)(tile / k_tiles), kt = (uint32_t)(tile % k_tiles);
    const uint64_t pitch = (t.cols + 1ull) / 2;
    const uint32_t i = threadIdx.x & 15u, r16 = threadIdx.x >> 4;  // columns 8 i .. 8 i + 7 of row r16
    const uint32_t row = row_tile * kTileRows + r16, c0 = kt * kTileCols + i * 8;
    const bool words = ((reinterpret_cast<uintptr_t>(src) | pitch) & 3u) == 0;
    uint32_t w = 0;
    if (row < t.rows) {
        const uint8_t *p = src + row * pitch + c0 / 2;
        if (words && c0 + 8 <= t.cols) {
            w = *reinterpret_cast<const uint32_t *>(p);
        } else {
            for (uint32_t k = 0; k < 8; ++k)
                if (c0 + k < t.cols) w |= (uint32_t)((p[k / 2] >> (4 * (k & 1))) & 15u) << (4 * k);
        }
    }
    if (!e2m1) {  // 0 1 2 3 4 5 6 7 -> 0 2 4 6 1 3 5 7
        uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
        even = (even | even >> 4) & 0x00FF00FFu;
        odd = (odd | odd >> 4) & 0x00FF00FFu;
        w = ((even | even >> 8) & 0xFFFFu) | (odd | odd >> 8) << 16;
    }
    // the word's place: word_col turned round
    const uint32_t quarter = t.group == 32 ? i & 3u : i >> 1 & 3u;
    const uint32_t j = t.group == 32 ? i >> 2 : i >> 3 << 1 | (i & 1u);
    codes[tile * 256 + (quarter * 16 + r16) * 4 + j] = w;
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
// rows of eq_w4_matvec's tensors: EQ_MAX_BLOCK_TENSORS of them stay below
// kMaxThreads with a workgroup per row of tiles
constexpr uint64_t kMaxRows = kTileRows * (kMaxThreads / (64 * kWaves) / EQ_MAX_BLOCK_TENSORS);

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

// Waves that share out the columns (log2): as many as have two tiles each.
uint32_t kw_log2(uint32_t k_tiles) {
    uint32_t n = 3;
    while (n > 0 && k_tiles < (2u << n)) --n;
    return n;
}

struct Shape {
    uint32_t nt, tp, r;  // token tiles of tp (4, 8 or 16) tokens and rows of tiles per wave
    bool wide;           // k_w4_wide
};

// Measured on MI355X (graph replays, us; rows of tiles of 16 rows), the rule's
// choice first:
//  * rows of tiles a wave takes (r), whose activations are loaded once: one
//    token 1 (its activations are small: 4096 x 4096 4.2, two 5.0); 2 to 8
//    tokens 2 (gate + up 57344 x 8192, four tokens bf16 38.2, one 43.0; eight
//    tokens 43.0, one 58.6; 5001 x 4133 with zeros, seven tokens 7.0, one 8.6); 9 to 32
//    tokens 4 where 160 workgroups remain (11008 x 4096, 16 tokens bf16 9.0, two
//    10.2) and 2 below (8192 x 28672 E4M3 24.3, four 32.4); 33 to 64 tokens 2
//    (registers: four would spill; INT4 with zeros in groups of 32 spills 6 at two
//    and is still ahead, 11008 x 4096 36.9, one 42.2). Halved while fewer than 128
//    workgroups would remain.
//  * k_w4_wide where its workgroups of 8 r rows of tiles still fill the chip:
//    16 tokens from 2560 rows of tiles (3584: bf16 44.0, k_w4 55.8; 1792: int8
//    25.2, wide 29.1), 32 from 1536 (3584: int8 47.8, k_w4 57.8), 64 from 1024
//    (3584: int8 55.3, k_w4 114; 688: bf16 30.2, wide 32.3); there r = 2 from 2560
//    (3584, 64 tokens int8: 55.3, one 60.2; 1792: 36.0, two 47.6).
//  * with fewer than 512 workgroups of one row of tiles a wave, the tokens are
//    spread over passes of 32 or 16 (64 tokens int8 x 1024 x 8192: 6.4, one pass
//    14.7; bf16 x 4096 x 4096: 9.9, 15.9).
// Where the rule takes the slower side: 4 tokens with r = 2 at 256 and 640 rows of
// tiles (4096 x 4096 5.0, one 4.5; 10240 x 8192 E2M1 12.4, one 11.5); 32 tokens of
// 8 bits at 1280 (28.9, wide 23.5); 64 tokens int8 x 8192 x 28672 in one pass
// (47.3; two passes of r = 4 40.5).
Shape shape(uint64_t tokens, uint64_t row_tiles, uint32_t kw_log2) {
    uint32_t nt = tokens <= 16 ? 1 : tokens <= 32 ? 2 : 4;
    const uint32_t tp = tokens <= 4 ? 4 : tokens <= 8 ? 8 : 16;
    if (tokens > 8 && row_tiles >= (nt == 1 ? 2560 : nt == 2 ? 1536 : 1024))
        return {nt, tp, row_tiles >= 2560 ? 2u : 1u, true};
    const uint64_t wgs = ((row_tiles << kw_log2) + kWaves - 1) / kWaves;  // with one row of tiles a wave
    while (nt > 1 && wgs * ((tokens + 16 * nt - 1) / (16 * nt)) < 512) nt /= 2;
    uint32_t r = tokens == 1 ? 1 : tokens <= 8 || nt == 4 || wgs < 640 ? 2 : 4;
    while (r > 1 && wgs < 128 * r) r /= 2;
    return {nt, tp, r, false};
}

W4Args tensor_args(const eq_w4_tensor &t) {
    W4Args a{};
    a.codes = static_cast<const u32x4 *>(t.d_codes);
    a.scales = t.d_scales;
    a.zeros = t.d_zeros;
    a.rows = (uint32_t)t.rows;
    a.cols = (uint32_t)t.cols;
    a.k_tiles = (uint32_t)((t.cols + kTileCols - 1) / kTileCols);
    a.row_tiles = (uint32_t)((t.rows + kTileRows - 1) / kTileRows);
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
                       static_cast<uint32_t *>(t->d_codes), t->d_scales, t->d_zeros);
    return hipGetLastError() == hipSuccess ? EQ_OK : EQ_EHIP;
}

eq_status eq_w4_matvec(const eq_w4_tensor *tensors, uint32_t n_tensors, const eq_matrix *x, const eq_matrix *y,
                       uint64_t tokens, void *stream) {
    if (n_tensors == 0) return EQ_OK;
    if (!tensors || !x || !y || tokens > 65535ull * kMaxTokens) return EQ_EINVAL;
    for (uint32_t i = 0; i < n_tensors; ++i) {
        const eq_w4_tensor &t = tensors[i];
        if (!tensor_ok(t) || t.rows > kMaxRows || x[i].reserved || y[i].reserved) return EQ_EINVAL;
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
        uint64_t total = 0;  // rows of tiles
        uint32_t kw = 0;
        for (uint32_t i = first; i < n_tensors && n < EQ_MAX_BLOCK_TENSORS; ++i) {
            if (kind(i) != kind(first)) continue;
            which[n++] = i;
            total += (tensors[i].rows + kTileRows - 1) / kTileRows;
            const uint32_t k = kw_log2((uint32_t)((tensors[i].cols + kTileCols - 1) / kTileCols));
            kw = k > kw ? k : kw;
        }
        const Shape sh = shape(tokens, total, kw);
        W4Launch a{};
        uint64_t wgs = 0;
        for (uint32_t k = 0; k < EQ_MAX_BLOCK_TENSORS; ++k) a.wg_begin[k] = ~0u;
        for (uint32_t k = 0; k < n; ++k) {
            const uint32_t i = which[k];
            W4Args &t = a.t[k];
            t = tensor_args(tensors[i]);
            t.x = x[i].d;
            t.x_scale = x[i].d_scale;
            t.y = y[i].d;
            t.ldx = x[i].stride;
            t.ldy = y[i].stride;
            a.wg_begin[k] = (uint32_t)wgs;
            t.kw_log2 = sh.wide ? 0 : kw_log2(t.k_tiles);
            t.wave_tiles = t.row_tiles < sh.r ? 1 : sh.r;
            t.r_step = t.wave_tiles == 1 ? 0 : t.k_tiles;
            const uint64_t per_wg = (kWaves >> t.kw_log2) * t.wave_tiles;
            wgs += (t.row_tiles + per_wg - 1) / per_wg;
        }
        a.per_pass = sh.tp < 16 ? kMaxTokens : 16 * sh.nt;
        const uint64_t passes = (tokens + a.per_pass - 1) / a.per_pass;
        a.tokens = (uint32_t)tokens;
        a.y_f32 = y[first].dtype == EQ_DTYPE_F32;
        hipLaunchKernelGGL(pick(tensors[first].dtype, x[first].dtype, tensors[first].d_zeros != nullptr,
                                tensors[first].group, sh.nt, sh.tp, sh.r, sh.wide),
                           dim3((uint32_t)wgs, (uint32_t)passes), dim3(64 * kWaves), 0,
                           static_cast<hipStream_t>(stream), a);
        if (hipGetLastError() != hipSuccess) return EQ_EHIP;
    }
    return EQ_OK;
}

}  // extern "C"
