// w4.hip -- products of a few tokens with 4-bit weights that carry a scale
// (and a zero point) per group of 32, 64 or 128 columns: eq_w4_matvec, and
// the load-time layout eq_w4_pack.
//
// Mathematics: y[t, r] = sum_g scale[r, g] * (sum_{c in g} q[r, c] x[t, c]
//   - zero[r, g] * sum_{c in g} x[t, c]). The inner sums run on the matrix
// cores: tokens are the rows of A, weight rows the columns of B, so a lane's
// accumulators all belong to one weight row (lane & 15) and a group's scale
// is one value per lane. Codes become exact bf16 values:
//   INT4: the 4 bits go to mantissa bits 3..6 under the exponent of 16:
//     16 + u with u = q + 8 (signed codes) or q (with zeros), one shift and
//     one three-input logic instruction per two weights; the 16 + zero is
//     taken off with sum(x), which one more matrix product with a B of ones
//     gives in the same registers.
//   E2M1: v_cvt_scalef32_pk_bf16_fp4, one instruction per two weights.
// What bounds it: HBM reads of the codes at few tokens.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/eq.h"
#include "device_util.hpp"

namespace {

using namespace eqdev;

constexpr uint32_t kTileRows = 16, kTileCols = 128, kTileBytes = 1024;
constexpr uint32_t kWaves = 8;            // waves of a workgroup; they share out the columns
constexpr uint32_t kMaxTokens = 64;       // tokens of one pass over the weights

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct W4Args {
    const u32x4 *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
    const void *x;
    const float *x_scale;
    void *y;
    uint64_t ldx, ldy;
    uint32_t rows, cols;
    uint32_t tile_begin;  // first workgroup of this tensor
    uint32_t group;
};

struct W4Launch {
    W4Args t[EQ_MAX_BLOCK_TENSORS];
    uint32_t n_tensors;
    uint32_t tokens;
    uint32_t y_f32;
};

// 8 consecutive activations as bf16, of which `left` exist (the rest zero).
// int8 and E4M3 values are exact in bf16.
template <uint32_t X>
__device__ __forceinline__ u32x4 load_x8(const void *row, uint32_t at, int32_t left) {
    u32x4 r = {0, 0, 0, 0};
    if (left <= 0) return r;
    if constexpr (X == EQ_DTYPE_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(row) + at;
        if (left >= 8) return *reinterpret_cast<const u32x4_a2 *>(p);
        for (int32_t i = 0; i < 8; ++i)
            if (i < left) r[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(row) + at;
        u32x2 b = {0, 0};
        if (left >= 8) {
            b = *reinterpret_cast<const u32x2_a1 *>(p);
        } else {
            for (int32_t i = 0; i < 8; ++i)
                if (i < left) b[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
        }
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = b[i / 2] >> (16 * (i & 1));
            if constexpr (X == EQ_DTYPE_INT8) r[i] = pack_bf16((float)(int8_t)h, (float)(int8_t)(h >> 8));
            else r[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h, 1.0f, false));
        }
    }
    return r;
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

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// Workgroup: 16 weight rows (one row of tiles), all columns, up to 16 * NT
// tokens; wave w takes tiles w, w + kWaves, ... and the waves' sums are joined
// in LDS in wave order.
template <uint32_t W, uint32_t X, bool Z, int NT>
__global__ void __launch_bounds__(64 * kWaves) k_w4(W4Launch a) {
    __shared__ f32x4 part[kWaves][NT][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    const uint32_t i16 = lane & 15u, quarter = lane >> 4;
    uint32_t ti = 0;
    while (ti + 1 < a.n_tensors && blockIdx.x >= a.t[ti + 1].tile_begin) ++ti;
    const W4Args &T = a.t[ti];
    const uint32_t row_tile = blockIdx.x - T.tile_begin;
    const uint32_t k_tiles = (T.cols + kTileCols - 1) / kTileCols;
    const uint32_t per_tile = kTileCols / T.group;  // groups of one row in a tile: 1, 2 or 4
    const uint32_t per_group = 4 / per_tile;        // 32-column steps per group
    const uint32_t token0 = blockIdx.y * kMaxTokens;
    constexpr size_t XB = X == EQ_DTYPE_BF16 ? 2 : 1;

    const char *x_row[NT];
    for (int n = 0; n < NT; ++n) {
        // token rows past the end repeat the last one; their sums are not stored
        uint32_t t = token0 + n * 16 + i16;
        t = t < a.tokens ? t : a.tokens - 1;
        x_row[n] = static_cast<const char *>(T.x) + (uint64_t)t * T.ldx * XB;
    }
    f32x4 acc[NT] = {};
    const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    for (uint32_t kt = wave; kt < k_tiles; kt += kWaves) {
        const uint64_t tile = (uint64_t)row_tile * k_tiles + kt;
        const u32x4 c = __builtin_nontemporal_load(T.codes + tile * 64 + lane);
        const uint64_t g0 = (tile * 16 + i16) * per_tile;
        f32x4 d[NT] = {}, sx[NT] = {};
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t k = kt * kTileCols + j * 32 + quarter * 8;
            const u32x4 b = decode8<W, Z>(c[j]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const u32x4 xa = load_x8<X>(x_row[n], k, (int32_t)(T.cols - k));
                d[n] = mfma(xa, b, d[n]);
                if constexpr (W == EQ_DTYPE_INT4) sx[n] = mfma(xa, ones, sx[n]);
            }
            if ((j + 1) % per_group == 0) {
                const uint64_t g = g0 + j / per_group;
                const float s = bf16_val(T.scales[g]);
                float off = 24.0f;
                if constexpr (Z) off = 16.0f + (float)T.zeros[g];
                for (int n = 0; n < NT; ++n) {
                    for (int i = 0; i < 4; ++i) {
                        const float v = W == EQ_DTYPE_INT4 ? fmaf(-off, sx[n][i], d[n][i]) : d[n][i];
                        acc[n][i] = fmaf(s, v, acc[n][i]);
                    }
                    d[n] = f32x4{};
                    sx[n] = f32x4{};
                }
            }
        }
    }
    for (int n = 0; n < NT; ++n) part[wave][n][lane] = acc[n];
    __syncthreads();
    if (wave < NT) {
        f32x4 s = {};
        for (uint32_t w = 0; w < kWaves; ++w) s += part[w][wave][lane];
        const uint32_t row = row_tile * kTileRows + i16;
        for (int i = 0; i < 4; ++i) {
            const uint32_t t = token0 + wave * 16 + quarter * 4 + i;
            if (t < a.tokens && row < T.rows) {
                float v = s[i];
                if constexpr (X != EQ_DTYPE_BF16) v *= T.x_scale[t];
                if (a.y_f32) static_cast<float *>(T.y)[t * T.ldy + row] = v;
                else static_cast<uint16_t *>(T.y)[t * T.ldy + row] = (uint16_t)pack_bf16(v, 0.0f);
            }
        }
    }
}

typedef void (*W4Fn)(W4Launch);

template <uint32_t W, uint32_t X, bool Z>
W4Fn pick_nt(uint64_t tokens) {
    if (tokens <= 16) return k_w4<W, X, Z, 1>;
    if (tokens <= 32) return k_w4<W, X, Z, 2>;
    return k_w4<W, X, Z, 4>;
}

W4Fn pick(uint32_t w, uint32_t x, bool z, uint64_t tokens) {
    if (w == EQ_DTYPE_E2M1)
        return x == EQ_DTYPE_BF16 ? pick_nt<EQ_DTYPE_E2M1, EQ_DTYPE_BF16, false>(tokens)
                                  : pick_nt<EQ_DTYPE_E2M1, EQ_DTYPE_E4M3, false>(tokens);
    if (x == EQ_DTYPE_BF16)
        return z ? pick_nt<EQ_DTYPE_INT4, EQ_DTYPE_BF16, true>(tokens) : pick_nt<EQ_DTYPE_INT4, EQ_DTYPE_BF16, false>(tokens);
    return z ? pick_nt<EQ_DTYPE_INT4, EQ_DTYPE_INT8, true>(tokens) : pick_nt<EQ_DTYPE_INT4, EQ_DTYPE_INT8, false>(tokens);
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
    const uint32_t k = kt * kTileCols + j * 32 + (lane >> 4) * 8;
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
    // one launch per kind (type, group does not matter, zeros, x and y types)
    // and EQ_MAX_BLOCK_TENSORS tensors; a tensor is launched with the first of its kind
    auto kind = [&](uint32_t i) {
        return tensors[i].dtype | x[i].dtype << 4 | y[i].dtype << 8 | (tensors[i].d_zeros ? 1u : 0u) << 12;
    };
    for (uint32_t first = 0; first < n_tensors; ++first) {
        uint32_t before = 0;  // tensors of this kind ahead of this one
        for (uint32_t i = 0; i < first; ++i) before += kind(i) == kind(first);
        if (before % EQ_MAX_BLOCK_TENSORS) continue;
        W4Launch a{};
        uint64_t wgs = 0;
        for (uint32_t i = first; i < n_tensors && a.n_tensors < EQ_MAX_BLOCK_TENSORS; ++i) {
            if (kind(i) != kind(first)) continue;
            W4Args &t = a.t[a.n_tensors++];
            t = tensor_args(tensors[i]);
            t.x = x[i].d;
            t.x_scale = x[i].d_scale;
            t.y = y[i].d;
            t.ldx = x[i].stride;
            t.ldy = y[i].stride;
            t.tile_begin = (uint32_t)wgs;
            wgs += (tensors[i].rows + kTileRows - 1) / kTileRows;
        }
        const uint64_t passes = (tokens + kMaxTokens - 1) / kMaxTokens;
        if (wgs > kMaxThreads / (64 * kWaves)) return EQ_EINVAL;
        a.tokens = (uint32_t)tokens;
        a.y_f32 = y[first].dtype == EQ_DTYPE_F32;
        hipLaunchKernelGGL(pick(tensors[first].dtype, x[first].dtype, tensors[first].d_zeros != nullptr, tokens),
                           dim3((uint32_t)wgs, (uint32_t)passes), dim3(64 * kWaves), 0,
                           static_cast<hipStream_t>(stream), a);
        if (hipGetLastError() != hipSuccess) return EQ_EHIP;
    }
    return EQ_OK;
}

}  // extern "C"
