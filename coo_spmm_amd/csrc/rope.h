// rope.h -- one head of one token on a group of lanes: its norm and its rotation.
//
// LPR lanes a head, eight features each (16 or 32 bytes of memory), in one of two
// ways.  Eight in a row: a block of 32 features is four neighbouring lanes, as the
// cache takes keys and values.  Whole pairs of the rotation (find_spot8): nothing is
// read twice; for what is written as it is, and for keys where eight neighbouring
// lanes then hold a block.
#pragma once

#include "ckpt.h"

namespace snack {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef double f64x8 __attribute__((ext_vector_type(8)));

// heads of tokens as a kernel takes them: rows = tokens * heads, the heads of a token side by side
struct Heads {
    const void* p;
    int64_t row, head;   // elements from token to token, from head to head
    FastDiv heads;
    uint32_t rows;
};

struct Rotation {
    const float* table;   // null: none
    uint32_t positions;
    int r;                // rotated pairs
    int layout;
};

// x of the lane that the DPP control names (every lane active)
template <int CTRL>
__device__ inline float dpp(float x)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ inline double dpp(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// x added over LPR neighbouring lanes: one and two apart within the quad, then mirrored halves and rows of
// lanes, then the neighbouring row; the same tree in each of them
template <int LPR, typename T>
__device__ inline T lanes_sum(T x)
{
    x += dpp<0xB1>(x);
    x += dpp<0x4E>(x);
    if constexpr (LPR >= 8) x += dpp<0x141>(x);
    if constexpr (LPR >= 16) x += dpp<0x140>(x);
    if constexpr (LPR >= 32) x += __shfl_xor(x, 16, kWave);
    if constexpr (LPR >= 64) x += __shfl_xor(x, 32, kWave);
    return x;
}

// eight features from p, of which the first `left` exist (the others are 0)
__device__ inline f32x8 load8(const float* __restrict__ p, int left)
{
    f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (left >= 8) {
        const f32x4 a = *reinterpret_cast<const f32x4u*>(p), b = *reinterpret_cast<const f32x4u*>(p + 4);
        v = f32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) v[i] = p[i];
    }
    return v;
}
__device__ inline f32x8 load8(const uint16_t* __restrict__ p, int left)
{
    f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (left >= 8) {
        const u16x8u h = *reinterpret_cast<const u16x8u*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bf16_value(h[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) v[i] = bf16_value(p[i]);
    }
    return v;
}
__device__ inline float load1(const float* p) { return *p; }
__device__ inline float load1(const uint16_t* p) { return bf16_value(*p); }

__device__ inline void store8(float* __restrict__ p, f32x8 v, int left)
{
    if (left >= 8) {
        *reinterpret_cast<f32x4u*>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4u*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) p[i] = v[i];
    }
}
__device__ inline void store8(uint16_t* __restrict__ p, f32x8 v, int left)
{
    u16x8u h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = bf16_bits(v[i]);
    if (left >= 8) {
        *reinterpret_cast<u16x8u*>(p) = h;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) p[i] = h[i];
    }
}

// What turns a lane's features f0..f0+7: feature i becomes c[i] x[i] + s[i] x[partner], sin with its sign; cos is 1
// and sin 0 past the rotated features.
struct Turn {
    f32x8 c, s;
};
__device__ inline Turn load_turn(const Rotation& ro, int pos, int f0)
{
    Turn t;
    const bool ok = (uint32_t)pos < ro.positions;
    const float* row = ro.table + (int64_t)(ok ? pos : 0) * (2 * ro.r);
    if (ro.layout == SNACK_ROPE_PAIRS) {
        const int i0 = f0 >> 1;
        f32x4 c, s;
        if (i0 + 4 <= ro.r) {
            c = *reinterpret_cast<const f32x4u*>(row + i0);
            s = *reinterpret_cast<const f32x4u*>(row + ro.r + i0);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = i0 + i < ro.r ? row[i0 + i] : 1.0f;
                s[i] = i0 + i < ro.r ? row[ro.r + i0 + i] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.c[2 * i] = t.c[2 * i + 1] = c[i];
            t.s[2 * i] = -s[i];
            t.s[2 * i + 1] = s[i];
        }
    } else if (f0 + 8 <= ro.r || (f0 >= ro.r && f0 + 8 <= 2 * ro.r)) {
        const bool second = f0 >= ro.r;
        const int i0 = second ? f0 - ro.r : f0;
        t.c = load8(row + i0, 8);
        t.s = load8(row + ro.r + i0, 8);
        if (!second) t.s = -t.s;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int f = f0 + i, j = f >= ro.r ? f - ro.r : f;
            const bool in = f < 2 * ro.r;
            t.c[i] = in ? row[j] : 1.0f;
            const float s = in ? row[ro.r + j] : 0.0f;
            t.s[i] = f < ro.r ? -s : s;
        }
    }
    if (!ok) {
        const float nan = __builtin_nanf("");
        t.c = f32x8{nan, nan, nan, nan, nan, nan, nan, nan};
    }
    return t;
}
// the partners of features f0..f0+7 in the array p (0 past the rotated ones)
template <typename X>
__device__ inline f32x8 load_partners(const Rotation& ro, const X* __restrict__ p, int f0)
{
    f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (f0 + 8 <= ro.r) return load8(p + f0 + ro.r, 8);
    if (f0 >= ro.r && f0 + 8 <= 2 * ro.r) return load8(p + f0 - ro.r, 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int f = f0 + i;
        if (f < 2 * ro.r) v[i] = load1(p + (f < ro.r ? f + ro.r : f - ro.r));
    }
    return v;
}
template <typename V>
__device__ inline V swap_pairs(V v)
{
    return __builtin_shufflevector(v, v, 1, 0, 3, 2, 5, 4, 7, 6);
}

// The same head with a lane holding whole pairs: four pairs (half layout: features 4 l..4 l + 3 and their partners r
// further; pairs layout: eight in a row) on the first ceil(r / 4) lanes, eight of the other features on the lanes behind
// them.  Nothing is read for a partner's sake, and a lane takes four angles for its eight features.
struct Eight {
    f32x4 a, b;
};
struct Spot8 {
    int a, b;     // first features of the two fours
    int na, nb;   // how many of each exist
    bool turned;
};
__device__ inline Spot8 find_spot8(int lane, int d, int r, int layout)
{
    const int turning = (r + 3) >> 2;
    Spot8 s;
    s.turned = lane < turning;
    if (s.turned && layout == SNACK_ROPE_HALF) {
        s.a = 4 * lane;
        s.b = r + s.a;
        s.na = s.nb = min(4, r - s.a);
    } else {
        const int end = s.turned ? 2 * r : d;
        s.a = s.turned ? 8 * lane : 2 * r + 8 * (lane - turning);
        s.b = s.a + 4;
        s.na = max(0, min(4, end - s.a));
        s.nb = max(0, min(4, end - s.b));
        if (s.na == 0) s.a = s.b = 0;    // a lane without features: its loads stay within the head
    }
    return s;
}
// whether every lane has eight features or none (EVEN below): no four that lacks some, none to move into place
inline bool even_lanes(int d, int r) { return r % 4 == 0 && (d - 2 * r) % 8 == 0; }
inline int pair_lanes(int d, int r)
{
    const int n = (r + 3) / 4 + (d - 2 * r + 7) / 8;
    return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64;
}
// Four of n numbers from i on, without a branch round the load where n >= 4: the last four where fewer are left, moved
// into place.  Those past the m-th are 0.
__device__ inline f32x4 raw4(const float* p) { return *reinterpret_cast<const f32x4u*>(p); }
__device__ inline f32x4 raw4(const uint16_t* p)
{
    const u16x4u h = *reinterpret_cast<const u16x4u*>(p);
    return f32x4{bf16_value(h.x), bf16_value(h.y), bf16_value(h.z), bf16_value(h.w)};
}
template <bool EVEN, typename X>
__device__ inline f32x4 take4(const X* __restrict__ p, int i, int n, int m)
{
    f32x4 v = {0, 0, 0, 0};
    if constexpr (EVEN) {
        v = raw4(p + i);
        return m > 0 ? v : f32x4{0, 0, 0, 0};
    }
    if (n < 4) {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < m) v[k] = load1(p + i + k);
        return v;
    }
    const int over = i - (n - 4);
    v = raw4(p + (over > 0 ? n - 4 : i));
    if (over > 0) v = f32x4{over == 1 ? v.y : over == 2 ? v.z : v.w, over == 1 ? v.z : v.w, v.w, 0.0f};
    return f32x4{m > 0 ? v.x : 0.0f, m > 1 ? v.y : 0.0f, m > 2 ? v.z : 0.0f, m > 3 ? v.w : 0.0f};
}
template <bool EVEN, typename X>
__device__ inline Eight take8(const X* __restrict__ p, const Spot8& s, int d)
{
    return Eight{take4<EVEN>(p, s.a, d, s.na), take4<EVEN>(p, s.b, d, s.nb)};
}
__device__ inline void put4(float* __restrict__ p, f32x4 v, int m)
{
    if (m >= 4) *reinterpret_cast<f32x4u*>(p) = v;
    else
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < m) p[i] = v[i];
}
__device__ inline void put4(uint16_t* __restrict__ p, f32x4 v, int m)
{
    if (m >= 4) *reinterpret_cast<u16x4u*>(p) = u16x4u{bf16_bits(v.x), bf16_bits(v.y), bf16_bits(v.z), bf16_bits(v.w)};
    else
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < m) p[i] = bf16_bits(v[i]);
}
// cos and sin of the lane's four pairs (1 and 0 where it has none); NaN for a position outside the table
struct Angles {
    f32x4 c, s;
};
template <bool EVEN>
__device__ inline Angles take_angles(const Rotation& ro, int pos, int lane, bool turned)
{
    const bool ok = (uint32_t)pos < ro.positions;
    const float* row = ro.table + (int64_t)(ok ? pos : 0) * (2 * ro.r);
    const int i = turned ? 4 * lane : 0, m = turned ? min(4, ro.r - i) : 0;
    Angles t{take4<EVEN>(row, i, ro.r, m), take4<EVEN>(row + ro.r, i, ro.r, m)};
    const float one = ok ? 1.0f : __builtin_nanf("");
    if (!turned || !ok) t.c = f32x4{one, one, one, one};
    return t;
}

// 1 / sqrt(a): the instruction's 2^-14 or better brought to 64 bits by three Newton steps
__device__ inline double rsqrt64(double a)
{
    double y = __builtin_amdgcn_rsq(a);
    const double h = 0.5 * a;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const double e = fma(-h * y, y, 0.5);
        y = fma(y, e, y);
    }
    return y;
}

// y of features f0..f0+7 of the head at p, in 64 bits
template <int LPR, typename X>
__device__ inline f64x8 qk_value(const X* __restrict__ p, int f0, int d, const float* __restrict__ gain, double eps,
                                 double inv_d, const Rotation& ro, int pos)
{
    const f32x8 xf = load8(p + f0, d - f0);
    f64x8 y = __builtin_convertvector(xf, f64x8);
    double rstd = 1.0;
    if (gain) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma(y[i], y[i], ss);
        const double a = fma(lanes_sum<LPR>(ss), inv_d, eps);
        // an infinity among the features: their quotients are 0, and NaN where they are infinite
        rstd = a < __builtin_inf() ? rsqrt64(a) : a == a ? 0.0 : a;
        y *= __builtin_convertvector(load8(gain + f0, d - f0), f64x8) * rstd;
    }
    if (!ro.table || f0 >= 2 * ro.r) {
        if (ro.table && (uint32_t)pos >= ro.positions) y *= __builtin_nan("");
        return y;
    }
    const Turn t = load_turn(ro, pos, f0);
    f64x8 o;
    if (ro.layout == SNACK_ROPE_PAIRS) {
        o = swap_pairs(y);
    } else {
        // the turning sin is 0 past the rotated features, whose partner is read as 0
        o = __builtin_convertvector(load_partners(ro, p, f0), f64x8);
        if (gain) o *= __builtin_convertvector(load_partners(ro, gain, f0), f64x8) * rstd;
    }
    // each product is exact in 64 bits where y is not normed, else within 2^-53 of it
    f64x8 z;
    const f64x8 c = __builtin_convertvector(t.c, f64x8), s = __builtin_convertvector(t.s, f64x8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // a feature that is not rotated keeps its own value, whatever its neighbours hold
        const bool in = f0 + i < 2 * ro.r;
        z[i] = in ? fma(o[i], s[i], y[i] * c[i]) : y[i] * c[i];
    }
    return z;
}

// The same on lanes that hold whole pairs (find_spot8): everything is loaded before the first of it is waited for.
struct Eight64 {
    double a[4], b[4];
};
template <int LPR, bool EVEN, typename X>
__device__ inline Eight qk_pairs(const X* __restrict__ p, const Spot8& at, int lane, int d, const float* __restrict__ gain,
                                 double eps, double inv_d, const Rotation& ro, int pos)
{
    const Eight x = take8<EVEN>(p, at, d);
    Eight g{{1, 1, 1, 1}, {1, 1, 1, 1}};
    if (gain) g = take8<EVEN>(gain, at, d);
    Angles t{{1, 1, 1, 1}, {0, 0, 0, 0}};
    if (ro.table) t = take_angles<EVEN>(ro, pos, lane, at.turned);
    Eight64 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y.a[i] = x.a[i];
        y.b[i] = x.b[i];
    }
    if (gain) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma(y.b[i], y.b[i], fma(y.a[i], y.a[i], ss));
        const double v = fma(lanes_sum<LPR>(ss), inv_d, eps);
        // an infinity among the features: their quotients are 0, and NaN where they are infinite
        const double rstd = v < __builtin_inf() ? rsqrt64(v) : v == v ? 0.0 : v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y.a[i] *= rstd * g.a[i];
            y.b[i] *= rstd * g.b[i];
        }
    }
    Eight z;
    if (at.turned && ro.layout == SNACK_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z.a[i] = (float)fma(-y.b[i], (double)t.s[i], y.a[i] * t.c[i]);
            z.b[i] = (float)fma(y.a[i], (double)t.s[i], y.b[i] * t.c[i]);
        }
    } else if (at.turned) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            z.a[2 * i] = (float)fma(-y.a[2 * i + 1], (double)t.s[i], y.a[2 * i] * t.c[i]);
            z.a[2 * i + 1] = (float)fma(y.a[2 * i], (double)t.s[i], y.a[2 * i + 1] * t.c[i]);
            z.b[2 * i] = (float)fma(-y.b[2 * i + 1], (double)t.s[2 + i], y.b[2 * i] * t.c[2 + i]);
            z.b[2 * i + 1] = (float)fma(y.b[2 * i], (double)t.s[2 + i], y.b[2 * i + 1] * t.c[2 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z.a[i] = (float)(y.a[i] * t.c[i]);
            z.b[i] = (float)(y.b[i] * t.c[i]);
        }
    }
    return z;
}

// lanes of a head of d features
inline int head_lanes(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// checks of the arguments that the calls share, and their form for the kernels
snack_status make_heads(const void* p, int64_t row, int64_t head, int32_t heads, int64_t tokens, int32_t d, int32_t fmt,
                        Heads* out);
snack_status make_rotation(const snack_rope* rope, int32_t d, const int32_t* pos, int64_t tokens, Rotation* out);

inline bool float_format(int32_t f) { return f == SNACK_F32 || f == SNACK_BF16; }
inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// One launch of norm, rotation and cache writes (cache.hip): the queries to yq, the keys to yk or into the cache, the
// values into the cache; each part may be empty (rows = 0).
struct CacheView;
struct QkPass {
    Heads q, k, v;
    int32_t d;
    const int32_t* pos;
    const int64_t* slot;
    Rotation ro;
    const float *q_gain, *k_gain;
    double eps, inv_d;
    void *yq, *yk;
    bool key_pairs;     // set by qk_pass
};
snack_status qk_pass(const QkPass& a, const CacheView* cache, int cache_fmt, int x_fmt, int y_fmt, int kclass,
                     hipStream_t s);

}  // namespace snack
