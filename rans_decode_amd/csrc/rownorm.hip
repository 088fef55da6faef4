// rownorm.hip -- the row-wise steps around a block's weight products: residual
// addition + root-mean-square norm (eq_add_rmsnorm) and silu(gate) * up
// (eq_silu_mul), each with bf16, int8 or E4M3 outputs.
//
// Mathematics, per row of n values:
//   norm: s = x + r; y = (s * w) * R, R = 1 / sqrt(mean(s^2) + eps).
//     R > 0 scales the whole row, so max|y| = max|s * w| * R (rounding is
//     monotone): the sum of squares and the 8-bit scale's maximum come out of
//     ONE reduction, and a row is read once. Where mean(s^2) + eps or s * w
//     leaves fp32's range the row is read again (see in_range); its output is
//     of ordinary size all the same.
//   silu: y = g / (1 + exp(-g)) * u, see silu_near.
//   8 bits: a = max(max|y|, 2^-96), scale = a / L, code = round(y * (L / a)).
//     The floor keeps L / a finite; a row of zeros gets codes 0. Maxima are
//     taken over the bit patterns of |y| as integers: the order is that of
//     the values, and a NaN (the largest patterns) is kept, which a
//     floating-point maximum would drop.
// What bounds both: HBM. One workgroup per row holds the row in registers in
// chunks of 8 values per thread (16-byte loads of bf16), so nothing is read
// twice. Measured (graph replays): norm of 8192 x 8192 bf16 with a bf16 residual
// to E4M3 85.8 us, 5.5 TB/s (a device copy: 5.1); silu of 4096 x 11008 bf16 to
// E4M3 44.6 us, 5.1 TB/s; one row of 4096 2.6 us, a launch and the latency of one
// load, reduction and store; one row of 28672 (silu, fp32 to int8) 5.3, the
// arithmetic of a row on one compute unit.
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

// 8 consecutive values of a row of bf16 or fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void *row, uint32_t at, float (&v)[kChunk]) {
    if constexpr (F32) {
        const float *p = static_cast<const float *>(row) + at;
        const f32x4 a = *reinterpret_cast<const f32x4_a4 *>(p), b = *reinterpret_cast<const f32x4_a4 *>(p + 4);
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
        const u32x4 a = *reinterpret_cast<const u32x4_a2 *>(static_cast<const uint16_t *>(row) + at);
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(a[i]), v[2 * i + 1] = bf16_hi(a[i]);
    }
}

// One value as stored, and as a number.
template <bool F32>
__device__ __forceinline__ uint32_t load_bits(const void *row, uint32_t at) {
    return F32 ? static_cast<const uint32_t *>(row)[at] : static_cast<const uint16_t *>(row)[at];
}
template <bool F32>
__device__ __forceinline__ float from_bits(uint32_t b) {
    return __uint_as_float(F32 ? b : b << 16);
}

__device__ __forceinline__ uint32_t bf16_bits(float v) { return pack_bf16(v, 0.0f) & 0xFFFFu; }

__device__ __forceinline__ void store8_bf16(void *row, uint32_t at, const float (&v)[kChunk]) {
    u32x4 a;
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4_a2 *>(static_cast<uint16_t *>(row) + at) = a;
}

__device__ __forceinline__ void store8_f32(void *row, uint32_t at, const float (&v)[kChunk]) {
    float *p = static_cast<float *>(row) + at;
    *reinterpret_cast<f32x4_a4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_a4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

// The nearest integer, ties to even. The clamp changes no finite value (see
// codes4); it gives a NaN an integer, which the conversion alone would not.
__device__ __forceinline__ uint32_t int8_bits(float t) {
    return (uint32_t)(int32_t)rintf(__builtin_amdgcn_fmed3f(t, -127.0f, 127.0f)) & 255u;
}

// Four 8-bit codes. |t| <= L * (1 + 2^-23), which rounds to L.
template <uint32_t OUT>
__device__ __forceinline__ uint32_t codes4(float t0, float t1, float t2, float t3) {
    if constexpr (OUT == EQ_DTYPE_INT8) {
        return int8_bits(t0) | int8_bits(t1) << 8 | int8_bits(t2) << 16 | int8_bits(t3) << 24;
    } else {
        const int a = __builtin_amdgcn_cvt_pk_fp8_f32(t0, t1, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t2, t3, a, true);
    }
}

// v * inv as codes (8-bit types) or v as bf16.
template <uint32_t OUT>
__device__ __forceinline__ void store8(void *row, uint32_t at, const float (&v)[kChunk], float inv) {
    if constexpr (OUT == EQ_DTYPE_BF16) {
        store8_bf16(row, at, v);
    } else {
        const u32x2 a = {codes4<OUT>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                         codes4<OUT>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
        *reinterpret_cast<u32x2_a1 *>(static_cast<uint8_t *>(row) + at) = a;
    }
}
template <uint32_t OUT>
__device__ __forceinline__ void store1(void *row, uint32_t at, float v, float inv) {
    if constexpr (OUT == EQ_DTYPE_BF16) static_cast<uint16_t *>(row)[at] = (uint16_t)bf16_bits(v);
    else static_cast<uint8_t *>(row)[at] = (uint8_t)codes4<OUT>(v * inv, 0.0f, 0.0f, 0.0f);
}

// One step of a wave reduction: every lane joins the value of its partner.
template <int CTRL>
__device__ __forceinline__ void join(float &sum, uint32_t &top) {
    sum += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(sum), CTRL, 0xF, 0xF, true));
    const uint32_t o = __builtin_amdgcn_update_dpp(0, top, CTRL, 0xF, 0xF, true);
    top = top > o ? top : o;
}

// Sum and maximum over the workgroup, in a fixed order; every thread gets
// both (what is not used is not computed). `lds` holds one pair per wave.
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

// g / (1 + exp(-g)) where exp(g) is a normal number. exp(-g) = 2^t exp(-d): t =
// -g log2 e as rounded, d = g + t ln 2 what that left out (ln 2 as rounded adds
// |g| 2^-29, 2 ulp at most), to first order; without d the error would grow as
// |g| 2^-24. The hardware's exp2 and reciprocal are within 1 ulp. (A Newton step
// on the reciprocal gained nothing: root mean square error for |g| < 20 0.53 2^-23
// with and without, one token x 28672 fp32 to int8 5.70 us, so 5.35; without d, 4.93.)
constexpr float kNear = 87.0f;
__device__ __forceinline__ float silu_near(float g) {
    const float t = g * -0x1.715476p+0f;
    const float e = __builtin_amdgcn_exp2f(t), d = fmaf(t, 0x1.62e430p-1f, g);
    const float den = fmaf(-e, d, e) + 1.0f;
    const float r = __builtin_amdgcn_rcpf(den);
    return g * r;
}
// The rest: 1 + exp(-|g|) is 1, and g exp(g) = (g h) h, h = exp(g / 2), vanishes
// through all of fp32's range before h does. The residual belongs to one h, with
// ln 2 in two parts.
__device__ __forceinline__ float silu_far(float g) {
    const float t = g * 0x1.715476p-1f;
    const float h = __builtin_amdgcn_exp2f(t), d = fmaf(t, -0x1.05c610p-28f, fmaf(t, 0x1.62e430p+0f, -g));
    return g < 0.0f ? g * h * fmaf(-h, d, h) : g;
}
__device__ __forceinline__ float silu(float g) { return fabsf(g) < kNear ? silu_near(g) : silu_far(g); }

// Whether a norm's sums can be used: squares overflow from |s| of 2^64 on, below
// 2^-63 they lose bits (which matters where eps does not cover them), and s * w
// may overflow although s * R * w does not. A row whose mean is out of range is
// summed again times k = 2^-80 or 2^80, which R takes back: with 2^-80 up to 2^31
// squares of the largest s stay below 2^128. (Infinities and NaN come out the
// same.) The outputs of such a row, and of one where s * w overflowed, are (s * R) * w,
// and so is what their 8-bit scale's maximum is taken of. bf16 outputs need no
// maximum over the row: there a thread that stored an infinity looks again by itself.
// (Looked for ahead of the reduction it cost 18 registers and 1777 rows of 5003
// 29%.)
constexpr float kMeanLow = 0x1p-90f, kMeanHigh = 0x1p126f, kRescale = 0x1p80f;
constexpr uint32_t kInf = 0x7F800000u;

__device__ __forceinline__ void join_top(uint32_t &top, float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    top = top > b ? top : b;
}

// The row's values before its common factor: s * w (norm, squares of s added
// to sum) or the finished y (silu); top joins the patterns of their |value|.
// RES: 0 none, else EQ_DTYPE_BF16 / EQ_DTYPE_F32. A second reading of a norm's
// row: SCALED takes s times k, FINAL (s * k * f) * w.
enum Scales : uint32_t { UNSCALED, SCALED, FINAL };
template <uint32_t OP, bool XF32, uint32_t RES, uint32_t SCALES = UNSCALED>
struct Row {
    static constexpr bool RF32 = OP == SILU ? XF32 : RES == EQ_DTYPE_F32;
    static constexpr size_t XB = XF32 ? 4 : 2, RB = RF32 ? 4 : 2;
    const char *x, *r;
    char *r_out;
    const void *w;
    bool w_f32;
    float k, f;

    __device__ __forceinline__ Row(const RowArgs &a, uint64_t row, float scale = 1.0f, float factor = 1.0f)
        : x(static_cast<const char *>(a.x) + row * a.ldx * XB), r(static_cast<const char *>(a.r) + row * a.ldr * RB),
          r_out(static_cast<char *>(a.r_out) + row * a.ldro * RB), w(a.w), w_f32(a.w_f32), k(scale), f(factor) {}

    __device__ __forceinline__ float scaled(float s) const {
        return SCALES == FINAL ? s * k * f : SCALES == SCALED ? s * k : s;
    }

    __device__ __forceinline__ void values8(uint32_t at, float (&v)[kChunk], float &sum, uint32_t &top) const {
        load8<XF32>(x, at, v);
        if constexpr (OP == SILU) {
            float u[kChunk];
            load8<XF32>(r, at, u);
            float most = 0.0f;
            for (uint32_t i = 0; i < kChunk; ++i) most = fmaxf(most, fabsf(v[i]));
            if (most < kNear)  // the same values, without the rest's instructions
                for (uint32_t i = 0; i < kChunk; ++i) v[i] = silu_near(v[i]) * u[i];
            else
                for (uint32_t i = 0; i < kChunk; ++i) v[i] = silu(v[i]) * u[i];
        } else {
            if constexpr (RES != 0) {
                float t[kChunk];
                load8<RF32>(r, at, t);
                for (uint32_t i = 0; i < kChunk; ++i) v[i] += t[i];
                if constexpr (RF32) {
                    store8_f32(r_out, at, v);
                } else {
                    store8_bf16(r_out, at, v);
                    // the norm is of the residual as it is stored
                    for (uint32_t i = 0; i < kChunk; ++i) v[i] = from_bits<false>(bf16_bits(v[i]));
                }
            }
            for (uint32_t i = 0; i < kChunk; ++i) v[i] = scaled(v[i]);
            for (uint32_t i = 0; i < kChunk; ++i) sum = fmaf(v[i], v[i], sum);
            if (w) {
                float t[kChunk];
                if (w_f32) load8<true>(w, at, t);
                else load8<false>(w, at, t);
                for (uint32_t i = 0; i < kChunk; ++i) v[i] *= t[i];
            }
        }
        for (uint32_t i = 0; i < kChunk; ++i) join_top(top, v[i]);
    }

    // One value of the last, short chunk: its loads, and what is made of them.
    struct Bits { uint32_t x, r, w; };
    __device__ __forceinline__ Bits load1(uint32_t at) const {
        Bits b = {load_bits<XF32>(x, at), 0, 0};
        if constexpr (OP == SILU || RES != 0) b.r = load_bits<RF32>(r, at);
        if constexpr (OP == NORM)
            if (w) b.w = w_f32 ? load_bits<true>(w, at) : load_bits<false>(w, at) << 16;
        return b;
    }
    __device__ __forceinline__ float value1(uint32_t at, Bits b, float &sum, uint32_t &top) const {
        float v = from_bits<XF32>(b.x);
        if constexpr (OP == SILU) {
            v = silu(v) * from_bits<RF32>(b.r);
        } else {
            if constexpr (RES != 0) {
                v += from_bits<RF32>(b.r);
                if constexpr (RF32) {
                    reinterpret_cast<float *>(r_out)[at] = v;
                } else {
                    const uint32_t h = bf16_bits(v);
                    reinterpret_cast<uint16_t *>(r_out)[at] = (uint16_t)h;
                    v = from_bits<false>(h);
                }
            }
            v = scaled(v);
            sum = fmaf(v, v, sum);
            if (w) v *= __uint_as_float(b.w);
        }
        join_top(top, v);
        return v;
    }
};

// NV chunks per thread in registers; NV = 0: rows of any length, whose values
// are computed a second time for the output (norm: from the stored sum where
// there is one, else from x). The last cols % 8 values go to one thread each,
// their loads ahead of the chunks' (a chunk of its own for them, filled value
// by value, cost rows of 5003 bf16 20%).
// At least 7 waves a SIMD are asked for where a norm to bf16 without a residual
// holds three chunks: by itself the compiler takes 73 registers, one more than 7
// waves have, and with the request 48 (1777 rows of 5003: 15.1 us, 11.3 with it).
template <uint32_t OP, bool XF32, uint32_t RES, uint32_t OUT, int NV>
__global__ void __launch_bounds__(kMaxThreads, OP == NORM && RES == 0 && OUT == EQ_DTYPE_BF16 && NV == 3 ? 7 : 4)
k_row(RowArgs a) {
    typedef Row<OP, XF32, RES> In;
    __shared__ float lds_sum[kMaxThreads / 64];
    __shared__ uint32_t lds_top[kMaxThreads / 64];
    const uint64_t row = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.tokens) return;
    const In in(a, row);
    const uint32_t whole = a.cols / kChunk * kChunk;  // values in whole chunks
    const uint32_t step = blockDim.x * kChunk;
    const uint32_t first = threadIdx.x * kChunk, last = whole + threadIdx.x;
    const bool extra = last < a.cols;
    float v[NV ? NV : 1][kChunk], v1 = 0.0f;
    float sum = 0.0f;
    uint32_t top = 0;
    typename In::Bits bits = {};
    if (extra) bits = in.load1(last);
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * step < whole) in.values8(first + i * step, v[i], sum, top);
    } else {
        for (uint64_t at = first; at < whole; at += step) in.values8((uint32_t)at, v[0], sum, top);
    }
    if (extra) v1 = in.value1(last, bits, sum, top);

    // A second reading (take(at, 8 values) and take1(at, value) for all of this
    // thread's): a norm's reads the stored sum, where there is one, which is what
    // this thread itself stored.
    auto read_again = [&](auto scales, float k, float f, float &sum2, uint32_t &top2, auto take, auto take1) {
        typedef Row<OP, RES ? RES == EQ_DTYPE_F32 : XF32, 0, OP == NORM ? (uint32_t)scales() : UNSCALED> Again;
        RowArgs b = a;
        if constexpr (RES != 0) {
            b.x = a.r_out;
            b.ldx = a.ldro;
        }
        const Again again(b, row, k, f);
        uint32_t from = first;
        // or the first reading's addresses are kept for it, at the cost of a workgroup a unit
        asm volatile("" : "+v"(from));
        const uint32_t from1 = whole + from / kChunk;
#pragma unroll 1
        for (uint64_t at = from; at < whole; at += step) {
            float t[kChunk];
            again.values8((uint32_t)at, t, sum2, top2);
            take((uint32_t)at, t);
        }
        if (from1 < a.cols) take1(from1, again.value1(from1, again.load1(from1), sum2, top2));
    };

    float factor = 1.0f, inv = 1.0f, k = 1.0f;
    bool again = false;  // the outputs are (s * k * factor) * w, read a second time
    if constexpr (OP == NORM || OUT != EQ_DTYPE_BF16) {
        reduce(sum, top, lds_sum, lds_top);
        if constexpr (OP == NORM) {
            float mean = sum / (float)a.cols + a.eps;
            const bool usable = mean >= kMeanLow && mean <= kMeanHigh;
            factor = rsqrtf(mean);
            again = __builtin_amdgcn_readfirstlane(!usable || (OUT != EQ_DTYPE_BF16 && top >= kInf));  // the same in all threads
            if (again) {
                auto none = [](uint32_t, float(&)[kChunk]) {};
                auto none1 = [](uint32_t, float) {};
                if (!usable) {
                    k = mean < kMeanLow ? kRescale : 1.0f / kRescale;
                    sum = 0.0f;
                    uint32_t unused = 0;
                    read_again([] { return SCALED; }, k, 1.0f, sum, unused, none, none1);
                    __syncthreads();  // the sums before have been read
                    reduce(sum, unused, lds_sum, lds_top);
                    mean = sum / (float)a.cols + a.eps * k * k;
                    factor = rsqrtf(mean);
                }
                if constexpr (OUT != EQ_DTYPE_BF16) {
                    top = 0;
                    read_again([] { return FINAL; }, k, factor, sum, top, none, none1);
                    __syncthreads();
                    reduce(sum, top, lds_sum, lds_top);
                }
            }
        }
        if constexpr (OUT != EQ_DTYPE_BF16) {
            constexpr float L = OUT == EQ_DTYPE_INT8 ? 127.0f : 448.0f;
            float amax = again ? __uint_as_float(top) : __uint_as_float(top) * factor;
            amax = amax < kAmaxFloor ? kAmaxFloor : amax;  // a NaN stays
            inv = L / amax;
            if (threadIdx.x == 0) a.scale[row] = amax / L;
        }
    }
    constexpr size_t OB = OUT == EQ_DTYPE_BF16 ? 2 : 1;
    void *out = static_cast<char *>(a.out) + row * a.ldo * OB;
    bool overflow = false;  // an output of this thread is not finite
    auto finish = [&](uint32_t at, float(&t)[kChunk]) {
        if constexpr (OP == NORM)
            for (uint32_t i = 0; i < kChunk; ++i) {
                t[i] *= factor;
                if constexpr (OUT == EQ_DTYPE_BF16) overflow |= !(fabsf(t[i]) < __builtin_inff());
            }
        store8<OUT>(out, at, t, inv);
    };
    auto finish1 = [&](uint32_t at, float t) {
        if constexpr (OP == NORM) {
            t *= factor;
            if constexpr (OUT == EQ_DTYPE_BF16) overflow |= !(fabsf(t) < __builtin_inff());
        }
        store1<OUT>(out, at, t, inv);
    };
    float sum2 = 0.0f;
    uint32_t top2 = 0;
    if (!again) {
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step < whole) finish(first + i * step, v[i]);
            if (extra) finish1(last, v1);
        } else {
            read_again([] { return UNSCALED; }, 1.0f, 1.0f, sum2, top2, finish, finish1);
        }
        again = overflow;
    }
    if constexpr (OP == NORM)
        if (again)
            read_again([] { return FINAL; }, k, factor, sum2, top2,
                       [&](uint32_t at, float(&t)[kChunk]) { store8<OUT>(out, at, t, inv); },
                       [&](uint32_t at, float t) { store1<OUT>(out, at, t, inv); });
}

typedef void (*RowFn)(RowArgs);

template <uint32_t OP, bool XF32, uint32_t RES, uint32_t OUT>
RowFn pick_nv(int nv) {
    switch (nv) {
        case 1: return k_row<OP, XF32, RES, OUT, 1>;
        case 2: return k_row<OP, XF32, RES, OUT, 2>;
        case 3: return k_row<OP, XF32, RES, OUT, 3>;
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

// Threads per row and chunks per thread. Few rows: a thread per chunk (512 rows
// of 4096: 5.3 us, with three chunks a thread 5.8); many: up to three, so that
// more rows are on their way at once (1777 rows of 5003 bf16: 11.3 us, one chunk
// 14.9, two 13.8; of 5000 9.5, 12.1; 8192 rows of 8192 with residual to E4M3: 85.8,
// one 84.7, four 88.8).
void shape(uint64_t tokens, uint64_t cols, uint32_t *threads, int *nv) {
    const uint64_t chunks = (cols + kChunk - 1) / kChunk, most = tokens < 1024 ? 1 : 3;
    uint32_t t = 64;
    while (t < kMaxThreads && t * most < chunks) t *= 2;
    const uint64_t per = (chunks + t - 1) / t;
    *threads = t;
    *nv = per <= 4 ? (int)per : 0;
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
    shape(tokens, cols, &threads, &nv);
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
    shape(tokens, cols, &threads, &nv);
    RowFn fn = gate->dtype == EQ_DTYPE_F32 ? pick_out<SILU, true, 0>(out->dtype, nv)
                                           : pick_out<SILU, false, 0>(out->dtype, nv);
    return launch_rows(fn, a, tokens, threads, stream);
}

}  // extern "C"
