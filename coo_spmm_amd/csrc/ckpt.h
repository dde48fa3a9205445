// ckpt.h -- the 8-bit block format of the activation checkpoints, on the device.
//
// A block is 32 consecutive features of one row (the last block of a row may
// hold fewer; its missing codes are 0).  It is kept as 32 one-byte codes c_i and
// one exponent byte s, and stands for c_i * 2^(s - 127), c_i a signed integer
// (SNACK_INT8) or an e4m3 number (SNACK_E4M3).  s is the smallest value >= 1
// that brings the block's largest |x| to at most 127 or 448, so the codes never
// saturate.  A block that holds a NaN or an infinity is stored as s = 255 with
// codes 0, which decodes to 0 * inf = NaN throughout: the loss of the block is
// visible to whoever reads it.
#pragma once

#include "internal.h"

namespace snack {

constexpr int kCkptBlock = 32;   // features of a row that share one exponent

// Vector types whose loads and stores need only the element's alignment: a row
// of odd length starts anywhere, and gfx950's global accesses of 8 and 16 bytes
// do not ask for more.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));

// round to nearest even; NaN stays a quiet NaN
__device__ inline uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ inline float bf16_value(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// the exponent byte of a block whose largest |x| has these bits (as integers,
// the bits of |x| are ordered like |x|, infinities and NaN last)
template <int FMT>
__device__ inline uint32_t ckpt_exponent(uint32_t amax)
{
    // amax = 1.f * 2^(e - 127); 1.f * 2^(e - s) <= 127 = 1.984375 * 2^6 or 448 = 1.75 * 2^8
    const int e = (int)(amax >> 23);
    const uint32_t f = amax & 0x7FFFFFu;
    int s = FMT == SNACK_INT8 ? e - 6 + (f > 0x7E0000u ? 1 : 0) : e - 8 + (f > 0x600000u ? 1 : 0);
    s = s < 1 ? 1 : s;
    return e == 255 ? 255u : (uint32_t)s;
}

// 2^(127 - s) for an exponent byte made by ckpt_exponent (1..249; 255 gives a value that is not used)
__device__ inline float ckpt_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// 2^(s - 127) for any byte: 2^-127 at 0, infinity at 255
__device__ inline float ckpt_scale(uint32_t s) { return __builtin_amdgcn_ldexpf(1.0f, (int)s - 127); }

// four values' codes, nearest even (x * inv is exact, so each is rounded once)
template <int FMT>
__device__ inline uint32_t ckpt_encode4(f32x4 x, uint32_t s)
{
    const float inv = ckpt_inverse(s);
    uint32_t w;
    if constexpr (FMT == SNACK_INT8) {
        // 1.5 * 2^23 + v rounds v to an integer whose two's complement is the sum's low byte
        const float big = 12582912.0f;
        const uint32_t a = __float_as_uint(fmaf(x.x, inv, big)), b = __float_as_uint(fmaf(x.y, inv, big));
        const uint32_t c = __float_as_uint(fmaf(x.z, inv, big)), d = __float_as_uint(fmaf(x.w, inv, big));
        const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
        w = lo | hi;
    } else {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(x.x * inv, x.y * inv, 0, false);
        w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x.z * inv, x.w * inv, p, true);
    }
    return s == 255u ? 0u : w;
}

// the four codes of a word as numbers (without the block's scale)
template <int FMT>
__device__ inline f32x4 ckpt_codes4(uint32_t w)
{
    f32x4 v;
    if constexpr (FMT == SNACK_INT8) {
        v.x = (float)(int8_t)(w & 0xFFu);
        v.y = (float)(int8_t)((w >> 8) & 0xFFu);
        v.z = (float)(int8_t)((w >> 16) & 0xFFu);
        v.w = (float)(int8_t)(w >> 24);
    } else {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        v.x = lo[0];
        v.y = lo[1];
        v.z = hi[0];
        v.w = hi[1];
    }
    return v;
}

// the largest of x over the eight lanes that share a block (all eight active):
// lanes 1 and 2 apart within the quad, then the half row mirrored
__device__ inline uint32_t octet_max(uint32_t x)
{
    uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true);
    x = x > y ? x : y;
    y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true);
    x = x > y ? x : y;
    y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, true);
    return x > y ? x : y;
}

__device__ inline uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ inline uint32_t abs_max4(f32x4 x)
{
    const uint32_t a = abs_bits(x.x), b = abs_bits(x.y), c = abs_bits(x.z), d = abs_bits(x.w);
    const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
    return ab > cd ? ab : cd;
}

// The block of eight lanes, each holding four of its values in order: codes to
// q (the lane's word) and the exponent byte to *s (by lane 0 of the eight).
template <int FMT>
__device__ inline void ckpt_store(f32x4 x, uint32_t* q, uint8_t* s, int lane8)
{
    const uint32_t e = ckpt_exponent<FMT>(octet_max(abs_max4(x)));
    *q = ckpt_encode4<FMT>(x, e);
    if (lane8 == 0) *s = (uint8_t)e;
}

// row = id / d for 0 <= id < 2^31 by one high multiplication (see fast_div)
struct FastDiv {
    uint32_t mul;   // 0: the divisor is 1
    uint32_t shift;
    uint32_t d;
};
__device__ inline uint32_t fast_quot(const FastDiv& f, uint32_t id)
{
    return f.mul ? __umulhi(id, f.mul) >> f.shift : id;
}
// With l = ceil(log2 d) and mul = ceil(2^(31 + l) / d) <= 2^32 - 1, the error
// mul * d - 2^(31 + l) is below d <= 2^l, so id * error < 2^(31 + l) and the
// quotient's floor is exact.
inline FastDiv fast_div(uint32_t d)
{
    FastDiv f{0, 0, d};
    if (d <= 1) return f;
    int l = 0;
    while ((1ull << l) < d) ++l;
    f.mul = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
    f.shift = (uint32_t)(l - 1);
    return f;
}

inline bool ckpt_format(int32_t fmt) { return fmt == SNACK_INT8 || fmt == SNACK_E4M3; }

}  // namespace snack
