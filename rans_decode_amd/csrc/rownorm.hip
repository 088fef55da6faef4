// rownorm.hip -- the row-wise steps around a block's weight products: residual
// addition + root-mean-square norm (eq_add_rmsnorm) and silu(gate) * up
// (eq_silu_mul), each with bf16, int8 or E4M3 outputs.
//
// Mathematics, per row of n values:
//   norm: s = x + r; y = (s * w) * R, R = 1 / sqrt(mean(s^2) + eps).
//     R > 0 scales the whole row, so max|y| = max|s * w| * R (rounding is
//     monotone): the sum of squares and the 8-bit scale's maximum come out of
//     ONE reduction, and a row is read once.
//   silu: y = g * (1 / (1 + exp(-g))) * u, with the hardware's exp2 and
//     reciprocal (1 ulp each; the exponent's product with log2 e adds at most
//     |g| 2^-24 relative, and 1 / (1 + exp(-g)) is insensitive to it for
//     g > 0): far below the 2^-9 of a bf16 output, and a correctly rounded
//     exp and division would make the kernel compute-bound.
//   8 bits: a = max(max|y|, 2^-96), scale = a / L, code = round(y * (L / a)).
//     The floor keeps L / a finite; a row of zeros gets codes 0. Maxima are
//     taken over the bit patterns of |y| as integers: the order is that of
//     the values, and a NaN (the largest patterns) is kept, which a
//     floating-point maximum would drop.
// What bounds both: HBM. One workgroup per row holds the row in registers in
// chunks of 8 values per thread (16-byte loads of bf16), so nothing is read
// twice.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/eq.h"
#include "device_util.hpp"

namespace {

using namespace eqdev;

constexpr uint32_t kChunk = 8;            // values per thread and step
constexpr float kAmaxFloor = 0x1p-96f;    // smallest row maximum of an 8-bit scale
constexpr uint32_t kMaxThreads = 1024;
constexpr uint32_t kGridX = 1u << 20;     // rows along grid x (x * threads stays below 2^32)

struct RowArgs {
    const void *x, *r;      // norm: x, residual; silu: gate, up
    void *r_out;            // norm: where s goes
    const void *w;          // norm: weight (bf16 or fp32) or NULL
    void *out;
    float *scale;
    uint64_t ldx, ldr, ldro, ldo;
    uint32_t tokens, cols, w_f32;
    float eps;
};

// 8 consecutive values of a row of bf16 or fp32, of which `left` exist (the
// rest read as zero).
template <bool F32>
__device__ __forceinline__ void load8(const void *row, uint32_t at, uint32_t left, float (&v)[kChunk]) {
    if constexpr (F32) {
        const float *p = static_cast<const float *>(row) + at;
        if (left >= kChunk) {
            const f32x4 a = *reinterpret_cast<const f32x4_a4 *>(p), b = *reinterpret_cast<const f32x4_a4 *>(p + 4);
            for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
        } else {
            for (uint32_t i = 0; i < kChunk; ++i) v[i] = i < left ? p[i] : 0.0f;
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(row) + at;
        if (left >= kChunk) {
            const u32x4 a = *reinterpret_cast<const u32x4_a2 *>(p);
            for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(a[i]), v[2 * i + 1] = bf16_hi(a[i]);
        } else {
            for (uint32_t i = 0; i < kChunk; ++i) v[i] = i < left ? bf16_val(p[i]) : 0.0f;
        }
    }
}

__device__ __forceinline__ void store_bf16(void *row, uint32_t at, uint32_t left, const float (&v)[kChunk]) {
    uint16_t *p = static_cast<uint16_t *>(row) + at;
    u32x4 a;
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (left >= kChunk) {
        *reinterpret_cast<u32x4_a2 *>(p) = a;
    } else {
        for (uint32_t i = 0; i < kChunk; ++i)
            if (i < left) p[i] = (uint16_t)(a[i / 2] >> (16 * (i & 1)));
    }
}

__device__ __forceinline__ void store_f32(void *row, uint32_t at, uint32_t left, const float (&v)[kChunk]) {
    float *p = static_cast<float *>(row) + at;
    if (left >= kChunk) {
        *reinterpret_cast<f32x4_a4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4_a4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        for (uint32_t i = 0; i < kChunk; ++i)
            if (i < left) p[i] = v[i];
    }
}

// 8-bit codes of v * inv. |v * inv| <= L * (1 + 2^-23), which rounds to L.
template <uint32_t OUT>
__device__ __forceinline__ void store_8bit(void *row, uint32_t at, uint32_t left, const float (&v)[kChunk], float inv) {
    uint8_t *p = static_cast<uint8_t *>(row) + at;
    uint32_t a[2];
    for (int h = 0; h < 2; ++h) {
        const float *t = v + 4 * h;
        if constexpr (OUT == EQ_DTYPE_INT8) {
            a[h] = 0;
            for (int i = 0; i < 4; ++i) a[h] |= ((uint32_t)(int32_t)rintf(t[i] * inv) & 255u) << (8 * i);
        } else {
            a[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[0] * inv, t[1] * inv, 0, false);
            a[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[2] * inv, t[3] * inv, (int)a[h], true);
        }
    }
    if (left >= kChunk) {
        *reinterpret_cast<u32x2_a1 *>(p) = u32x2{a[0], a[1]};
    } else {
        for (uint32_t i = 0; i < kChunk; ++i)
            if (i < left) p[i] = (uint8_t)(a[i / 4] >> (8 * (i & 3)));
    }
}

// One step of a wave reduction: every lane joins the value of its partner.
template <int CTRL>
__device__ __forceinline__ void join(float &sum, uint32_t &top) {
    sum += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(sum), CTRL, 0xF, 0xF, true));
    const uint32_t o = __builtin_amdgcn_update_dpp(0, top, CTRL, 0xF, 0xF, true);
    top = top > o ? top : o;
}

// Sum and maximum over the workgroup, in a fixed order; every thread gets
// both. `lds` holds one pair per wave.
__device__ __forceinline__ void reduce(float &sum, uint32_t &top, float *lds_sum, uint32_t *lds_top) {
    join<0xB1>(sum, top);   // quad_perm 1 0 3 2
    join<0x4E>(sum, top);   // quad_perm 2 3 0 1
    join<0x141>(sum, top);  // row_half_mirror
    join<0x140>(sum, top);  // row_mirror: each row of 16 lanes holds its own total
    float s = 0.0f;
    uint32_t t = 0;
    for (int i = 0; i < 4; ++i) {
        s += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sum), 16 * i));
        const uint32_t o = __builtin_amdgcn_readlane(top, 16 * i);
        t = t > o ? t : o;
    }
    const uint32_t waves = blockDim.x >> 6;
    if (waves > 1) {
        if ((threadIdx.x & 63u) == 0) {
            lds_sum[threadIdx.x >> 6] = s;
            lds_top[threadIdx.x >> 6] = t;
        }
        __syncthreads();
        s = 0.0f;
        t = 0;
        for (uint32_t i = 0; i < waves; ++i) {
            s += lds_sum[i];
            t = t > lds_top[i] ? t : lds_top[i];
        }
    }
    sum = s;
    top = t;
}

enum Op : uint32_t { NORM, SILU };

// The row's values before its common factor: s * w (norm, squares of s added
// to sum) or the finished y (silu); top joins the patterns of their |value|.
template <uint32_t OP, bool XF32, uint32_t RES>  // RES: 0 none, else EQ_DTYPE_BF16 / EQ_DTYPE_F32
__device__ __forceinline__ void values8(const RowArgs &a, uint64_t row, uint32_t at, float (&v)[kChunk],
                                        float &sum, uint32_t &top) {
    const uint32_t left = a.cols - at;
    constexpr size_t XB = XF32 ? 4 : 2;
    load8<XF32>(static_cast<const char *>(a.x) + row * a.ldx * XB, at, left, v);
    if constexpr (OP == SILU) {
        float u[kChunk];
        load8<XF32>(static_cast<const char *>(a.r) + row * a.ldr * XB, at, left, u);
        for (uint32_t i = 0; i < kChunk; ++i) v[i] = v[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-v[i])) * u[i];
    } else {
        if constexpr (RES != 0) {
            constexpr bool RF32 = RES == EQ_DTYPE_F32;
            float r[kChunk];
            load8<RF32>(static_cast<const char *>(a.r) + row * a.ldr * (RF32 ? 4 : 2), at, left, r);
            for (uint32_t i = 0; i < kChunk; ++i) v[i] += r[i];
            if constexpr (RF32) {
                store_f32(static_cast<char *>(a.r_out) + row * a.ldro * 4, at, left, v);
            } else {
                store_bf16(static_cast<char *>(a.r_out) + row * a.ldro * 2, at, left, v);
                // the norm is of the residual as it is stored
                for (uint32_t i = 0; i < kChunk; i += 2) {
                    const uint32_t p = pack_bf16(v[i], v[i + 1]);
                    v[i] = bf16_lo(p);
                    v[i + 1] = bf16_hi(p);
                }
            }
        }
        for (uint32_t i = 0; i < kChunk; ++i) sum = fmaf(v[i], v[i], sum);
        if (a.w) {
            float w[kChunk];
            if (a.w_f32) load8<true>(a.w, at, left, w);
            else load8<false>(a.w, at, left, w);
            for (uint32_t i = 0; i < kChunk; ++i) v[i] *= w[i];
        }
    }
    for (uint32_t i = 0; i < kChunk; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        top = top > b ? top : b;
    }
}

// NV chunks per thread in registers; NV = 0: rows of any length, whose values
// are computed a second time for the output (norm: from the stored sum where
// there is one, else from x).
template <uint32_t OP, bool XF32, uint32_t RES, uint32_t OUT, int NV>
__global__ void __launch_bounds__(kMaxThreads) k_row(RowArgs a) {
    __shared__ float lds_sum[kMaxThreads / 64];
    __shared__ uint32_t lds_top[kMaxThreads / 64];
    const uint64_t row = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.tokens) return;
    const uint32_t step = blockDim.x * kChunk;
    const uint32_t first = threadIdx.x * kChunk;
    float v[NV ? NV : 1][kChunk];
    float sum = 0.0f;
    uint32_t top = 0;
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t at = first + i * step;
            if (at < a.cols) values8<OP, XF32, RES>(a, row, at, v[i], sum, top);
        }
    } else {
        for (uint64_t at = first; at < a.cols; at += step) values8<OP, XF32, RES>(a, row, (uint32_t)at, v[0], sum, top);
    }
    float factor = 1.0f, inv = 1.0f;
    if constexpr (OP == NORM || OUT != EQ_DTYPE_BF16) {
        reduce(sum, top, lds_sum, lds_top);
        if constexpr (OP == NORM) factor = rsqrtf(sum / (float)a.cols + a.eps);
        if constexpr (OUT != EQ_DTYPE_BF16) {
            constexpr float L = OUT == EQ_DTYPE_INT8 ? 127.0f : 448.0f;
            float amax = __uint_as_float(top) * factor;
            amax = amax < kAmaxFloor ? kAmaxFloor : amax;  // a NaN stays
            inv = L / amax;
            if (threadIdx.x == 0) a.scale[row] = amax / L;
        }
    }
    constexpr size_t OB = OUT == EQ_DTYPE_BF16 ? 2 : 1;
    void *out = static_cast<char *>(a.out) + row * a.ldo * OB;
    auto finish = [&](uint32_t at, float(&t)[kChunk]) {
        if constexpr (OP == NORM)
            for (uint32_t i = 0; i < kChunk; ++i) t[i] *= factor;
        if constexpr (OUT == EQ_DTYPE_BF16) store_bf16(out, at, a.cols - at, t);
        else store_8bit<OUT>(out, at, a.cols - at, t, inv);
    };
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t at = first + i * step;
            if (at < a.cols) finish(at, v[i]);
        }
    } else {
        RowArgs again = a;
        if constexpr (RES != 0) {  // each thread reads back what it wrote itself
            again.x = a.r_out;
            again.ldx = a.ldro;
        }
        constexpr bool XF = RES ? RES == EQ_DTYPE_F32 : XF32;
        for (uint64_t at = first; at < a.cols; at += step) {
            values8<OP, XF, 0>(again, row, (uint32_t)at, v[0], sum, top);
            finish((uint32_t)at, v[0]);
        }
    }
}

typedef void (*RowFn)(RowArgs);

template <uint32_t OP, bool XF32, uint32_t RES, uint32_t OUT>
RowFn pick_nv(int nv) {
    switch (nv) {
        case 1: return k_row<OP, XF32, RES, OUT, 1>;
        case 2: return k_row<OP, XF32, RES, OUT, 2>;
        case 4: return k_row<OP, XF32, RES, OUT, 4>;
        default: return k_row<OP, XF32, RES, OUT, 0>;
    }
}
template <uint32_t OP, bool XF32, uint32_t RES>
RowFn pick_out(uint32_t out, int nv) {
    if (out == EQ_DTYPE_BF16) return pick_nv<OP, XF32, RES, EQ_DTYPE_BF16>(nv);
    if (out == EQ_DTYPE_INT8) return pick_nv<OP, XF32, RES, EQ_DTYPE_INT8>(nv);
    return pick_nv<OP, XF32, RES, EQ_DTYPE_E4M3>(nv);
}
template <bool XF32>
RowFn pick_res(uint32_t res, uint32_t out, int nv) {
    if (res == 0) return pick_out<NORM, XF32, 0>(out, nv);
    if (res == EQ_DTYPE_BF16) return pick_out<NORM, XF32, EQ_DTYPE_BF16>(out, nv);
    return pick_out<NORM, XF32, EQ_DTYPE_F32>(out, nv);
}

bool is_real(uint32_t dtype) { return dtype == EQ_DTYPE_BF16 || dtype == EQ_DTYPE_F32; }
bool is_8bit(uint32_t dtype) { return dtype == EQ_DTYPE_INT8 || dtype == EQ_DTYPE_E4M3; }

bool matrix_ok(const eq_matrix *m, uint64_t cols) {
    if (!m || !m->d || m->reserved || m->stride < cols || m->stride > (1ull << 40)) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(m->d);
    if (m->dtype == EQ_DTYPE_F32) return a % 4 == 0;
    if (m->dtype == EQ_DTYPE_BF16) return a % 2 == 0;
    return is_8bit(m->dtype) && m->d_scale && reinterpret_cast<uintptr_t>(m->d_scale) % 4 == 0;
}

bool sizes_ok(uint64_t tokens, uint64_t cols) { return cols && cols <= 0x7FFFFFFFull && tokens <= 0x7FFFFFFFull; }

eq_status launch_rows(RowFn fn, const RowArgs &a, uint64_t tokens, uint32_t threads, void *stream) {
    const uint32_t gx = tokens < kGridX ? (uint32_t)tokens : kGridX;
    hipLaunchKernelGGL(fn, dim3(gx, (uint32_t)((tokens + gx - 1) / gx)), dim3(threads), 0,
                       static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? EQ_OK : EQ_EHIP;
}

// Threads per row and chunks per thread.
void shape(uint64_t cols, uint32_t *threads, int *nv) {
    const uint64_t chunks = (cols + kChunk - 1) / kChunk;
    uint32_t t = 64;
    while (t < kMaxThreads && t < chunks) t *= 2;
    const uint64_t per = (chunks + t - 1) / t;
    *threads = t;
    *nv = per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 0;
}

}  // namespace

extern "C" {

eq_status eq_add_rmsnorm(const eq_matrix *x, const eq_matrix *residual, const eq_matrix *residual_out,
                         const void *d_weight, uint32_t weight_dtype, float eps, uint64_t tokens,
                         uint64_t cols, const eq_matrix *out, void *stream) {
    if (!sizes_ok(tokens, cols) || !(eps >= 0.0f)) return EQ_EINVAL;
    if (!x || !out || !is_real(x->dtype) || !(out->dtype == EQ_DTYPE_BF16 || is_8bit(out->dtype))) return EQ_EINVAL;
    if ((residual == nullptr) != (residual_out == nullptr)) return EQ_EINVAL;
    if (residual && (!is_real(residual->dtype) || residual->dtype != residual_out->dtype)) return EQ_EINVAL;
    if (d_weight && (!is_real(weight_dtype) ||
                     reinterpret_cast<uintptr_t>(d_weight) % (weight_dtype == EQ_DTYPE_F32 ? 4 : 2)))
        return EQ_EINVAL;
    if (tokens == 0) return EQ_OK;
    if (!matrix_ok(x, cols) || !matrix_ok(out, cols)) return EQ_EINVAL;
    if (residual && (!matrix_ok(residual, cols) || !matrix_ok(residual_out, cols))) return EQ_EINVAL;
    RowArgs a{};
    a.x = x->d;
    a.ldx = x->stride;
    if (residual) {
        a.r = residual->d;
        a.ldr = residual->stride;
        a.r_out = residual_out->d;
        a.ldro = residual_out->stride;
    }
    a.w = d_weight;
    a.w_f32 = weight_dtype == EQ_DTYPE_F32;
    a.out = out->d;
    a.ldo = out->stride;
    a.scale = out->d_scale;
    a.cols = (uint32_t)cols;
    a.tokens = (uint32_t)tokens;
    a.eps = eps;
    uint32_t threads;
    int nv;
    shape(cols, &threads, &nv);
    const uint32_t res = residual ? residual->dtype : 0;
    RowFn fn = x->dtype == EQ_DTYPE_F32 ? pick_res<true>(res, out->dtype, nv) : pick_res<false>(res, out->dtype, nv);
    return launch_rows(fn, a, tokens, threads, stream);
}

eq_status eq_silu_mul(const eq_matrix *gate, const eq_matrix *up, uint64_t tokens, uint64_t cols,
                      const eq_matrix *out, void *stream) {
    if (!sizes_ok(tokens, cols)) return EQ_EINVAL;
    if (!gate || !up || !out || !is_real(gate->dtype) || gate->dtype != up->dtype ||
        !(out->dtype == EQ_DTYPE_BF16 || is_8bit(out->dtype)))
        return EQ_EINVAL;
    if (tokens == 0) return EQ_OK;
    if (!matrix_ok(gate, cols) || !matrix_ok(up, cols) || !matrix_ok(out, cols)) return EQ_EINVAL;
    RowArgs a{};
    a.x = gate->d;
    a.ldx = gate->stride;
    a.r = up->d;
    a.ldr = up->stride;
    a.out = out->d;
    a.ldo = out->stride;
    a.scale = out->d_scale;
    a.cols = (uint32_t)cols;
    a.tokens = (uint32_t)tokens;
    uint32_t threads;
    int nv;
    shape(cols, &threads, &nv);
    RowFn fn = gate->dtype == EQ_DTYPE_F32 ? pick_out<SILU, true, 0>(out->dtype, nv)
                                           : pick_out<SILU, false, 0>(out->dtype, nv);
    return launch_rows(fn, a, tokens, threads, stream);
}

}  // extern "C"
