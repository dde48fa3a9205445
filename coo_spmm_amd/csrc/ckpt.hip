// ckpt.hip -- 8-bit activation checkpoints: pack, unpack, and the exact GELU that
// leaves checkpoints of its input and output, with its gradient from them.
//
// All of them are one pass over [rows, n] arrays and bound by HBM.  The eight
// lanes of an octet share a 32-feature block, four consecutive features each:
// values move as 16 bytes a lane (whole kilobytes a wavefront), codes as four
// bytes a lane, and the block's largest |x| is three DPP steps away.  Blocks of
// all rows are numbered through, so ragged widths cost one multiplication per
// block instead of idle lanes.  4096 x 10000: pack 33 us (206 MB), read back in
// fp32 32 us (206 MB) and in bf16 20 us (124 MB).
#include "ckpt.h"

namespace snack {
namespace {

constexpr int kThreads = 256;

struct Shape {
    int64_t n;        // features of a row
    uint32_t total;   // blocks of all rows
    FastDiv per_row;  // blocks of a row
};

// four values from p, of which the first `left` exist (the others read as 0)
__device__ inline f32x4 load4(const float* __restrict__ p, int left)
{
    if (left >= 4) return *reinterpret_cast<const f32x4u*>(p);
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (left > 0) v.x = p[0];
    if (left > 1) v.y = p[1];
    if (left > 2) v.z = p[2];
    return v;
}
__device__ inline void store4(float* __restrict__ p, f32x4 v, int left)
{
    if (left >= 4) {
        *reinterpret_cast<f32x4u*>(p) = v;
        return;
    }
    if (left > 0) p[0] = v.x;
    if (left > 1) p[1] = v.y;
    if (left > 2) p[2] = v.z;
}

// block `id`: the offset of this lane's features in a [rows, n] array and how many of them exist
__device__ inline int64_t place(const Shape& sh, uint32_t id, int first, int& left)
{
    const uint32_t row = fast_quot(sh.per_row, id);
    const int64_t f = (int64_t)(id - row * sh.per_row.d) * kCkptBlock + first;
    const int64_t l = sh.n - f;
    left = l > 32 ? 32 : (int)l;
    return (int64_t)row * sh.n + f;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) pack_kernel(const float* __restrict__ X, uint32_t* __restrict__ Q,
                                                        uint8_t* __restrict__ S, Shape sh)
{
    const int lane8 = (int)threadIdx.x & 7;
    const uint32_t step = gridDim.x * (kThreads / 8);
    for (uint32_t id = (blockIdx.x * kThreads + threadIdx.x) >> 3; id < sh.total; id += step) {
        int left;
        const int64_t at = place(sh, id, 4 * lane8, left);
        ckpt_store<FMT>(load4(X + at, left), Q + (int64_t)id * 8 + lane8, S + id, lane8);
    }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) unpack_f32_kernel(const uint32_t* __restrict__ Q,
                                                              const uint8_t* __restrict__ S, float* __restrict__ Y,
                                                              Shape sh)
{
    const int lane8 = (int)threadIdx.x & 7;
    const uint32_t step = gridDim.x * (kThreads / 8);
    for (uint32_t id = (blockIdx.x * kThreads + threadIdx.x) >> 3; id < sh.total; id += step) {
        int left;
        const int64_t at = place(sh, id, 4 * lane8, left);
        const float sc = ckpt_scale(S[id]);
        store4(Y + at, ckpt_codes4<FMT>(Q[(int64_t)id * 8 + lane8]) * sc, left);
    }
}

// four lanes a block, eight features each: 16-byte stores of bf16
template <int FMT>
__global__ void __launch_bounds__(kThreads) unpack_bf16_kernel(const uint2* __restrict__ Q,
                                                               const uint8_t* __restrict__ S,
                                                               uint16_t* __restrict__ Y, Shape sh)
{
    const int lane4 = (int)threadIdx.x & 3;
    const uint32_t step = gridDim.x * (kThreads / 4);
    for (uint32_t id = (blockIdx.x * kThreads + threadIdx.x) >> 2; id < sh.total; id += step) {
        int left;
        const int64_t at = place(sh, id, 8 * lane4, left);
        const uint2 w = Q[(int64_t)id * 4 + lane4];
        const float sc = ckpt_scale(S[id]);
        const f32x4 a = ckpt_codes4<FMT>(w.x) * sc, b = ckpt_codes4<FMT>(w.y) * sc;
        u16x8u o;
        o[0] = bf16_bits(a.x); o[1] = bf16_bits(a.y); o[2] = bf16_bits(a.z); o[3] = bf16_bits(a.w);
        o[4] = bf16_bits(b.x); o[5] = bf16_bits(b.y); o[6] = bf16_bits(b.z); o[7] = bf16_bits(b.w);
        if (left >= 8) {
            *reinterpret_cast<u16x8u*>(Y + at) = o;
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) Y[at + i] = o[i];
        }
    }
}

// Phi(-a) = exp(-a^2 / 2) R(a) for a = |x|, R(a) = erfcx(a / sqrt 2) / 2.  R is
// t P(t) with t = 1 / (1 + 0.35 a), P the degree-8 polynomial of least relative
// error on 0 <= a <= 13.5 (3.2e-8; fitted by reweighted least squares); past
// that Phi(-a) is below 2^-126 and the exponential ends it.  One reciprocal, one
// exponential and a dozen multiply-adds, no branch, and the tail of negative x
// keeps its relative accuracy.  Measured in fp32 over |x| <= 8: cdf within
// 1.9e-7, as 1 + erf within 0.6e-7 at 60 to 90 instructions.  Over normal x of
// scale 1.5 (rms of the error over rms of the value, here : through erff): the
// GELU 2.7e-8 : 3.7e-8, its slope 4.7e-8 : 3.7e-8, where x itself was rounded
// to eight bits before.
struct GeluTerms {
    float e;   // exp(-a^2 / 2)
    float r;   // R(a)
    float a;   // |x|, at most 16
};
__device__ inline GeluTerms gelu_terms(float x)
{
    GeluTerms g;
    g.a = fminf(fabsf(x), 16.0f);
    const float u = fmaf(g.a, 0.35f, 1.0f);
    float t = __builtin_amdgcn_rcpf(u);
    t = fmaf(fmaf(-u, t, 1.0f), t, t);
    float p = -0.02912587672472f;
    p = fmaf(p, t, 0.14387229084968567f);
    p = fmaf(p, t, -0.25550466775894165f);
    p = fmaf(p, t, 0.15892940759658813f);
    p = fmaf(p, t, -0.022937219589948654f);
    p = fmaf(p, t, 0.10543297231197357f);
    p = fmaf(p, t, 0.11985243111848831f);
    p = fmaf(p, t, 0.13985908031463623f);
    p = fmaf(p, t, 0.1396215707063675f);
    g.r = p * t;
    // exp(-a^2/2) = 2^(c a^2), c = -log2(e) / 2, with the roundings of a^2, of c and of the product put back
    const float c = -0.72134752044448170f, c_lo = -0.72134752044448170 - (double)-0.72134752044448170f;
    const float h = g.a * g.a, h_lo = fmaf(g.a, g.a, -h);
    const float m = h * c;
    const float m_lo = fmaf(h_lo, c, fmaf(h, c_lo, fmaf(h, c, -m)));
    const float e = __builtin_amdgcn_exp2f(m);
    g.e = fmaf(e * 0.69314718055994531f, m_lo, e);
    return g;
}
// x Phi(x)
__device__ inline float gelu_fwd_value(float x)
{
    const GeluTerms g = gelu_terms(x);
    const float q = g.e * g.r;
    // -|x| q, and x - |x| q past 0, rounded once; |x| stays finite where x is not (0 and x at the infinities)
    return fmaf(-g.a, q, x < 0.0f ? 0.0f : x);
}
// Phi(x) + x phi(x); 0 and 1 at the infinities
__device__ inline float gelu_slope_value(float x)
{
    const GeluTerms g = gelu_terms(x);
    const float d = g.e * fmaf(g.a, -0.39894228040143268f, g.r);
    const float v = x < 0.0f ? d : 1.0f - d;
    return x != x ? x : v;
}
__device__ inline f32x4 gelu_fwd4(f32x4 x)
{
    f32x4 y;
    y.x = gelu_fwd_value(x.x);
    y.y = gelu_fwd_value(x.y);
    y.z = gelu_fwd_value(x.z);
    y.w = gelu_fwd_value(x.w);
    return y;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads)
gelu_ckpt_fwd_kernel(const float* __restrict__ X, float* __restrict__ Y, uint32_t* __restrict__ QX,
                     uint8_t* __restrict__ SX, uint32_t* __restrict__ QY, uint8_t* __restrict__ SY, Shape sh)
{
    const int lane8 = (int)threadIdx.x & 7;
    const uint32_t step = gridDim.x * (kThreads / 8);
    for (uint32_t id = (blockIdx.x * kThreads + threadIdx.x) >> 3; id < sh.total; id += step) {
        int left;
        const int64_t at = place(sh, id, 4 * lane8, left);
        const f32x4 x = load4(X + at, left);
        const f32x4 y = gelu_fwd4(x);
        if (QX) ckpt_store<FMT>(x, QX + (int64_t)id * 8 + lane8, SX + id, lane8);
        if (QY) ckpt_store<FMT>(y, QY + (int64_t)id * 8 + lane8, SY + id, lane8);
        if (Y) store4(Y + at, y, left);
    }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads)
gelu_ckpt_bwd_kernel(const uint32_t* __restrict__ QX, const uint8_t* __restrict__ SX, const float* __restrict__ dY,
                     float* __restrict__ dX, Shape sh)
{
    const int lane8 = (int)threadIdx.x & 7;
    const uint32_t step = gridDim.x * (kThreads / 8);
    for (uint32_t id = (blockIdx.x * kThreads + threadIdx.x) >> 3; id < sh.total; id += step) {
        int left;
        const int64_t at = place(sh, id, 4 * lane8, left);
        const f32x4 d = load4(dY + at, left);
        const float sc = ckpt_scale(SX[id]);
        const f32x4 x = ckpt_codes4<FMT>(QX[(int64_t)id * 8 + lane8]) * sc;
        f32x4 o;
        o.x = d.x * gelu_slope_value(x.x);
        o.y = d.y * gelu_slope_value(x.y);
        o.z = d.z * gelu_slope_value(x.z);
        o.w = d.w * gelu_slope_value(x.w);
        store4(dX + at, o, left);
    }
}

// rows x n as numbered blocks; false where they number 2^31 or more
bool make_shape(int64_t rows, int64_t n, Shape* sh)
{
    const int64_t per = (n + kCkptBlock - 1) / kCkptBlock;
    if (per >= (1ll << 31) || rows >= (1ll << 31) || rows * per >= (1ll << 31)) return false;
    sh->n = n;
    sh->total = (uint32_t)(rows * per);
    sh->per_row = fast_div((uint32_t)per);
    return true;
}

// workgroups for `lanes` lanes a block: one block a lane group, at most
// 8192 workgroups (32 a CU), which then stride
unsigned grid_for(const Shape& sh, int lanes)
{
    const int64_t g = ((int64_t)sh.total * lanes + kThreads - 1) / kThreads;
    return (unsigned)(g > 8192 ? 8192 : g);
}

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// checks common to the entry points; 1: nothing to do
snack_status common(int64_t rows, int64_t n, int32_t fmt, Shape* sh)
{
    if (rows < 0 || n < 1 || !ckpt_format(fmt)) return SNACK_ERR_INVALID_ARG;
    if (!make_shape(rows, n, sh)) return SNACK_ERR_UNSUPPORTED;
    return SNACK_OK;
}

}  // namespace

}  // namespace snack

using namespace snack;

extern "C" snack_status snack_ckpt_pack(const float* X, int64_t rows, int64_t n, int32_t fmt, uint8_t* Q, uint8_t* S,
                                        snack_stream stream)
{
    Shape sh;
    SNACK_CHECK(common(rows, n, fmt, &sh));
    if (rows == 0) return SNACK_OK;
    if (!X || !Q || !S || misaligned(X, 4) || misaligned(Q, 16)) return SNACK_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_CKPT, s);
    const auto k = fmt == SNACK_INT8 ? pack_kernel<SNACK_INT8> : pack_kernel<SNACK_E4M3>;
    hipLaunchKernelGGL(k, dim3(grid_for(sh, 8)), dim3(kThreads), 0, s, X, (uint32_t*)Q, S, sh);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

extern "C" snack_status snack_ckpt_unpack(const uint8_t* Q, const uint8_t* S, int64_t rows, int64_t n, int32_t fmt,
                                          void* Y, int32_t y_fmt, snack_stream stream)
{
    Shape sh;
    SNACK_CHECK(common(rows, n, fmt, &sh));
    if (y_fmt != SNACK_F32 && y_fmt != SNACK_BF16) return SNACK_ERR_INVALID_ARG;
    if (rows == 0) return SNACK_OK;
    if (!Q || !S || !Y || misaligned(Q, 16) || misaligned(Y, y_fmt == SNACK_F32 ? 4 : 2)) return SNACK_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_CKPT, s);
    if (y_fmt == SNACK_F32) {
        const auto k = fmt == SNACK_INT8 ? unpack_f32_kernel<SNACK_INT8> : unpack_f32_kernel<SNACK_E4M3>;
        hipLaunchKernelGGL(k, dim3(grid_for(sh, 8)), dim3(kThreads), 0, s, (const uint32_t*)Q, S, (float*)Y, sh);
    } else {
        const auto k = fmt == SNACK_INT8 ? unpack_bf16_kernel<SNACK_INT8> : unpack_bf16_kernel<SNACK_E4M3>;
        hipLaunchKernelGGL(k, dim3(grid_for(sh, 4)), dim3(kThreads), 0, s, (const uint2*)Q, S, (uint16_t*)Y, sh);
    }
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

extern "C" snack_status snack_gelu_ckpt_fwd(const float* X, int64_t rows, int64_t n, int32_t fmt, float* Y,
                                            uint8_t* QX, uint8_t* SX, uint8_t* QY, uint8_t* SY, snack_stream stream)
{
    Shape sh;
    SNACK_CHECK(common(rows, n, fmt, &sh));
    if (rows == 0) return SNACK_OK;
    if (!X || misaligned(X, 4) || misaligned(Y, 4) || (!Y && !QX && !QY)) return SNACK_ERR_INVALID_ARG;
    if (!QX != !SX || !QY != !SY || misaligned(QX, 16) || misaligned(QY, 16)) return SNACK_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_CKPT, s);
    const auto k = fmt == SNACK_INT8 ? gelu_ckpt_fwd_kernel<SNACK_INT8> : gelu_ckpt_fwd_kernel<SNACK_E4M3>;
    hipLaunchKernelGGL(k, dim3(grid_for(sh, 8)), dim3(kThreads), 0, s, X, Y, (uint32_t*)QX, SX, (uint32_t*)QY, SY, sh);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

extern "C" snack_status snack_gelu_ckpt_bwd(const uint8_t* QX, const uint8_t* SX, const float* dY, int64_t rows,
                                            int64_t n, int32_t fmt, float* dX, snack_stream stream)
{
    Shape sh;
    SNACK_CHECK(common(rows, n, fmt, &sh));
    if (rows == 0) return SNACK_OK;
    if (!QX || !SX || !dY || !dX || misaligned(QX, 16) || misaligned(dY, 4) || misaligned(dX, 4))
        return SNACK_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_CKPT, s);
    const auto k = fmt == SNACK_INT8 ? gelu_ckpt_bwd_kernel<SNACK_INT8> : gelu_ckpt_bwd_kernel<SNACK_E4M3>;
    hipLaunchKernelGGL(k, dim3(grid_for(sh, 8)), dim3(kThreads), 0, s, (const uint32_t*)QX, SX, dY, dX, sh);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}
