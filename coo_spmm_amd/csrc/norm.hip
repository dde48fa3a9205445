// norm.hip -- root-mean-square norm over rows with the residual's addition, its
// output's 8-bit checkpoint, and its gradient from a hidden state held in fp32,
// bf16 or as a checkpoint.
//
//   h = x + residual (rounded to the residual stream's type)
//   y = h rstd gain,  rstd = 1 / sqrt(mean(h^2) + eps)
//   dx = rstd (w - xh mean(w xh)) + dR,  xh = h rstd,  w = dY gain
//   dgain = sum over rows of dY xh
//
// Both directions are one pass over HBM, which bounds them: a row stays in
// registers between its sum and its outputs.  Rows of up to 1024 features take one
// wavefront each (the sum never leaves it), longer ones a workgroup of as many
// wavefronts as give every thread at most four groups of four features; rows past
// 16384 features, which no longer fit, and rows of less than four are read twice.
// Features are dealt to threads so that eight neighbouring lanes always hold one
// 32-feature block.  All of a row's loads are in flight before the first is used
// (read4).  dgain: every workgroup adds up its own rows' terms in registers, in row
// order, and writes one row of partial sums; a second kernel adds the partial rows
// in a fixed tree (for few rows, workgroups of their own add up columns in the same
// launch).  No atomics, so the result does not depend on timing.
//
// Measured (a copy of 1 GiB runs at 5.2 TB/s): forward 8192 x 5000, bf16 residual,
// e4m3 checkpoint, 534 MB in 109 us (4.9 TB/s); 1 x 768 in 2.7 us (a launch).
// Gradient 3333 x 4999, fp32 h, 266 MB in 44 us and 4.9 us for the partial rows;
// 10000 x 1500 from an int8 checkpoint, 195 MB in 40 us with both.  Rows read twice: 2000 x 20000, bf16 residual, int8
// checkpoint, 520 MB in 127 us, gradient from bf16 h 128 us; 200000 x 3, a workgroup a row of three values, 1.2 and
// 0.9 ms.
#include "ckpt.h"

#include <float.h>

namespace snack {
namespace {

constexpr int kChunks = 4;                       // groups of four features a thread holds
constexpr int kWaveRow = kWave * 4 * kChunks;    // longest row of one wavefront
constexpr int kRowMax = 1024 * 4 * kChunks;      // longest row of one workgroup
constexpr int kLongThreads = 1024;               // workgroup of the rows past it
constexpr int kCus = 256;                        // compute units
constexpr int kBwdWaves = 10;                    // wavefronts a unit of the gradient, and most workgroups
constexpr int kBwdPerCu = 4;
constexpr int kGainLanes = 4;                    // lanes of a row in the sum of dgain beside the rows
constexpr int kColThreads = 256;                 // column pass of rows past kRowMax
// Outputs of a forward call past this many bytes, the size of the last-level cache, are stored past the caches:
// nothing of them would still be there for whoever reads them.  Measured (us, cached : past them): 8192 x 5000,
// 288 MB, 115 : 105 alone; with a reader of y behind it 32768 x 2000, 459 MB, 231 : 221, but 16384 x 2000,
// 229 MB, 107 : 113 and 4096 x 2000, 57 MB, 26.0 : 28.2.
constexpr int64_t kStreamBytes = 256ll << 20;
constexpr int kSumCols = 32, kSumRows = 32;      // final sum: columns and row strides of a workgroup
// Threads of a launch at most (HIP takes fewer than 2^32 of them) and its blocks in y: what needs more, from 2^21
// rows of a workgroup each on, is launched in pieces.
constexpr int64_t kLaunchThreads = 1ll << 31;
constexpr int64_t kLaunchY = 1 << 15;

// x added over the lanes of a wavefront, the same tree in every lane
template <typename T>
__device__ inline T wave_sum(T x)
{
#pragma unroll
    for (int m = kWave / 2; m >= 1; m >>= 1) x += __shfl_xor(x, m, kWave);
    return x;
}

// the same over a workgroup; part holds 16 numbers.  Every thread gets the sum;
// safe to call again at once with the other half of a doubled buffer
template <typename T>
__device__ inline T group_sum(T x, T* part)
{
    x = wave_sum(x);
    const int w = (int)threadIdx.x / kWave, nw = (int)blockDim.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) part[w] = x;
    __syncthreads();
    T s = 0;
#pragma unroll 4
    for (int i = 0; i < nw; ++i) s += part[i];
    return s;
}

template <int HF>
struct HType { using T = float; };
template <>
struct HType<SNACK_BF16> { using T = uint16_t; };

// Four features from p, of which the first `left` exist (the others are 0).
__device__ inline f32x4 load4(const float* __restrict__ p, int left)
{
    if (left >= 4) return *reinterpret_cast<const f32x4u*>(p);
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (left > 0) v.x = p[0];
    if (left > 1) v.y = p[1];
    if (left > 2) v.z = p[2];
    return v;
}
__device__ inline f32x4 value4(f32x4 v) { return v; }
__device__ inline f32x4 value4(u16x4u h)
{
    return f32x4{bf16_value(h.x), bf16_value(h.y), bf16_value(h.z), bf16_value(h.w)};
}
__device__ inline f32x4 load4(const uint16_t* __restrict__ p, int left)
{
    u16x4u h = {0, 0, 0, 0};
    if (left >= 4) {
        h = *reinterpret_cast<const u16x4u*>(p);
    } else {
        if (left > 0) h.x = p[0];
        if (left > 1) h.y = p[1];
        if (left > 2) h.z = p[2];
    }
    return value4(h);
}

// The same from a row of n >= 4 features, in two steps without a branch round the load: read4 takes the last four
// of the row where fewer are left, kept4 brings them in place.  A thread's loads are then all issued before the
// first is waited for (with a branch round each, its conversion holds the next load back: a row of 1100 features
// of a checkpoint took 3.7 us in place of 1.7).
// The row's address is a scalar and a lane's offset in it 32 unsigned bits: one register an access.
__device__ inline const char* at_bytes(const void* row, uint32_t bytes) { return (const char*)row + bytes; }
__device__ inline char* at_bytes(void* row, uint32_t bytes) { return (char*)row + bytes; }
__device__ inline f32x4 read4(const float* __restrict__ row, int f, int n)
{
    return *reinterpret_cast<const f32x4u*>(at_bytes(row, 4u * (uint32_t)min(f, n - 4)));
}
__device__ inline u16x4u read4(const uint16_t* __restrict__ row, int f, int n)
{
    return *reinterpret_cast<const u16x4u*>(at_bytes(row, 2u * (uint32_t)min(f, n - 4)));
}
__device__ inline f32x4 kept4(f32x4 v, int left)
{
    if (left >= 4) return v;
    return f32x4{left > 2 ? v.y : left > 1 ? v.z : left > 0 ? v.w : 0.0f, left > 2 ? v.z : left > 1 ? v.w : 0.0f,
                 left > 2 ? v.w : 0.0f, 0.0f};
}
__device__ inline f32x4 kept4(u16x4u h, int left) { return kept4(value4(h), left); }

// stream: past the caches (a value that is the same for the whole launch)
__device__ inline void store4(float* __restrict__ p, f32x4 v, int left, bool stream = false)
{
    if (left >= 4) {
        if (stream) __builtin_nontemporal_store(v, reinterpret_cast<f32x4u*>(p));
        else *reinterpret_cast<f32x4u*>(p) = v;
        return;
    }
    if (left > 0) p[0] = v.x;
    if (left > 1) p[1] = v.y;
    if (left > 2) p[2] = v.z;
}
__device__ inline void store4(uint16_t* __restrict__ p, f32x4 v, int left, bool stream = false)
{
    const u16x4u h = {bf16_bits(v.x), bf16_bits(v.y), bf16_bits(v.z), bf16_bits(v.w)};
    if (left >= 4) {
        if (stream) __builtin_nontemporal_store(h, reinterpret_cast<u16x4u*>(p));
        else *reinterpret_cast<u16x4u*>(p) = h;
        return;
    }
    if (left > 0) p[0] = h.x;
    if (left > 1) p[1] = h.y;
    if (left > 2) p[2] = h.z;
}
__device__ inline float dot4(f32x4 a, f32x4 b) { return fmaf(a.x, b.x, a.y * b.y) + fmaf(a.z, b.z, a.w * b.w); }

struct FwdArgs {
    const float* X;
    const void* R;       // residual, or null
    const float* gain;
    void* H;             // h, or null (no residual: h is X)
    float* Y;            // or null
    float* rstd;
    uint8_t* Q;          // checkpoint of y, or null
    uint8_t* S;
    int64_t rows, n, per_row;   // per_row: blocks of a row
    float eps;
    bool stream;                // h and y past the caches
};

// h of four features: x + residual, rounded to the stream's type
template <int HF>
__device__ inline f32x4 hidden4(f32x4 x, f32x4 res)
{
    const f32x4 h = x + res;
    if constexpr (HF != SNACK_BF16) return h;
    return f32x4{bf16_value(bf16_bits(h.x)), bf16_value(bf16_bits(h.y)), bf16_value(bf16_bits(h.z)),
                 bf16_value(bf16_bits(h.w))};
}
template <int HF>
__device__ inline f32x4 hidden4(const FwdArgs& A, int64_t at, int left)
{
    const f32x4 x = load4(A.X + at, left);
    return A.R ? hidden4<HF>(x, load4((const typename HType<HF>::T*)A.R + at, left)) : x;
}

// h^2 of four features added in 64 bits: squares of fp32 numbers neither round nor overflow there
__device__ inline double add_squares(double s, f32x4 h)
{
    s = fma((double)h.x, (double)h.x, s);
    s = fma((double)h.y, (double)h.y, s);
    s = fma((double)h.z, (double)h.z, s);
    return fma((double)h.w, (double)h.w, s);
}

// rstd as an fp32 number and what is left of it.  y = h rstd gain is then rounded once (to within a few 2^-48): a
// value next to a border of the 8-bit grid goes to the wrong side half as often as with a rounding a product (37
// against 68 of 25 million normal values, int8), and no error of rstd moves a whole row one way.
struct Rstd {
    float hi, lo;
};
__device__ inline Rstd rstd_of(double ss, const FwdArgs& A)
{
    const double r = 1.0 / sqrt(ss / (double)A.n + (double)A.eps);
    const float hi = (float)r;
    return {hi, (float)(r - (double)hi)};
}
__device__ inline float scaled(float h, float g, Rstd r)
{
    const float u = h * r.hi;
    const float e = fmaf(h, r.lo, fmaf(h, r.hi, -u));
    const float y = fmaf(u, g, e * g);
    return fabsf(y) <= FLT_MAX ? y : u * g;   // an infinite gain: e g may be a NaN or the other infinity
}

// y of four features and what is kept of it
template <int QF>
__device__ inline void finish4(const FwdArgs& A, int64_t row, int64_t f, int64_t at, int left, f32x4 h, f32x4 g, Rstd r)
{
    const f32x4 y = {scaled(h.x, g.x, r), scaled(h.y, g.y, r), scaled(h.z, g.z, r), scaled(h.w, g.w, r)};
    if (A.Y) store4(A.Y + at, y, left, A.stream);
    if constexpr (QF != SNACK_F32) {
        const int64_t blk = row * A.per_row + f / kCkptBlock;
        ckpt_store<QF>(y, (uint32_t*)(A.Q + blk * kCkptBlock) + ((f / 4) & 7), A.S + blk, (int)((f / 4) & 7));
    }
}

// WG: a workgroup a row; else a wavefront a row
template <int HF, int QF, bool WG>
__global__ void __launch_bounds__(WG ? 1024 : 256) norm_fwd_kernel(FwdArgs A)
{
    __shared__ double part[16];
    using T = typename HType<HF>::T;
    const int64_t row = WG ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
    if (row >= A.rows) return;   // never with WG
    const int t = WG ? (int)threadIdx.x : (int)threadIdx.x & (kWave - 1);
    const int nt = WG ? (int)blockDim.x : kWave;
    const int n = (int)A.n;
    const int64_t base = row * A.n;
    f32x4 h[kChunks], g[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) h[i] = read4(A.X + base, 4 * (t + i * nt), n);
    if (A.R) {
        decltype(read4((const T*)nullptr, 0, 0)) res[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) res[i] = read4((const T*)A.R + base, 4 * (t + i * nt), n);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) g[i] = read4(A.gain, 4 * (t + i * nt), n);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) h[i] = hidden4<HF>(h[i], value4(res[i]));
    } else {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) g[i] = read4(A.gain, 4 * (t + i * nt), n);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        h[i] = kept4(h[i], n - 4 * (t + i * nt));
        g[i] = kept4(g[i], n - 4 * (t + i * nt));
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int f = 4 * (t + i * nt);
        if (A.H) store4((T*)A.H + base + f, h[i], n - f, A.stream);
        ss = add_squares(ss, h[i]);
    }
    ss = WG ? group_sum(ss, part) : wave_sum(ss);
    const Rstd r = rstd_of(ss, A);
    if (t == 0) A.rstd[row] = r.hi;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int f = 4 * (t + i * nt);
        // whole blocks: the eight lanes of a row's last block stay together
        if ((f & ~(kCkptBlock - 1)) < n) finish4<QF>(A, row, f, base + f, n - f, h[i], g[i], r);
    }
}

// rows past kRowMax: h made twice
template <int HF, int QF>
__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(FwdArgs A)
{
    __shared__ double part[16];
    using T = typename HType<HF>::T;
    const int64_t row = blockIdx.x, base = row * A.n;
    double ss = 0.0;
    for (int64_t f = 4 * (int64_t)threadIdx.x; f < A.n; f += 4 * kLongThreads) {
        const f32x4 h = hidden4<HF>(A, base + f, A.n - f);
        if (A.H) store4(reinterpret_cast<T*>(A.H) + base + f, h, A.n - f, A.stream);
        ss = add_squares(ss, h);
    }
    ss = group_sum(ss, part);
    const Rstd r = rstd_of(ss, A);
    if (threadIdx.x == 0) A.rstd[row] = r.hi;
    for (int64_t f = 4 * (int64_t)threadIdx.x; (f & ~(int64_t)(kCkptBlock - 1)) < A.n; f += 4 * kLongThreads)
        finish4<QF>(A, row, f, base + f, A.n - f, hidden4<HF>(A, base + f, A.n - f), load4(A.gain + f, A.n - f), r);
}

struct BwdArgs {
    const void* H;        // h: fp32, bf16, or the codes of a checkpoint
    const uint8_t* HS;    // the checkpoint's exponent bytes
    const float* gain;
    const float* rstd;
    const float* dY;
    const float* dR;      // gradient that reaches h directly, or null
    float* dX;
    float* part;          // [gridDim.x][n] partial sums of dgain, or null
    float* mean;          // [rows] mean(w xh) (long_rows)
    int64_t rows, n, per_row;
    float* dgain;         // written here by the workgroups past `groups`, or null
    int groups;           // workgroups that take rows
    int64_t col0;         // first column of this launch (norm_bwd_cols_kernel)
};

// Four features of one row of h, from feature f, in the same two steps: h and hs are the row's (its codes and
// exponent bytes for a checkpoint, whose codes past the n-th are bytes, but no values).
template <int HF>
struct Kept {
    decltype(read4((const typename HType<HF>::T*)nullptr, 0, 0)) v;
    __device__ inline void read(const void* __restrict__ h, const uint8_t* __restrict__, int f, int n)
    {
        v = read4((const typename HType<HF>::T*)h, f, n);
    }
    __device__ inline f32x4 value(int left) const { return kept4(v, left); }
};
template <int HF>
struct KeptCodes {
    uint32_t w, s;
    __device__ inline void read(const void* __restrict__ h, const uint8_t* __restrict__ hs, int f, int n)
    {
        const uint32_t at = (uint32_t)min(f, (n - 1) & ~3);
        w = *reinterpret_cast<const uint32_t*>(at_bytes(h, at));
        s = *(const uint8_t*)at_bytes(hs, at / kCkptBlock);
    }
    __device__ inline f32x4 value(int left) const
    {
        f32x4 v = ckpt_codes4<HF>(w) * ckpt_scale(s);
        if (left >= 4) return v;
        return f32x4{left > 0 ? v.x : 0.0f, left > 1 ? v.y : 0.0f, left > 2 ? v.z : 0.0f, 0.0f};
    }
};
template <>
struct Kept<SNACK_INT8> : KeptCodes<SNACK_INT8> {};
template <>
struct Kept<SNACK_E4M3> : KeptCodes<SNACK_E4M3> {};

// the same for rows of any length
template <int HF>
__device__ inline f32x4 hidden_row4(const void* __restrict__ h, const uint8_t* __restrict__ hs, int f, int n)
{
    if constexpr (HF == SNACK_INT8 || HF == SNACK_E4M3) {
        Kept<HF> k;
        k.read(h, hs, f, n);
        return k.value(n - f);
    } else {
        return load4((const typename HType<HF>::T*)h + f, n - f);
    }
}
template <int HF>
__host__ __device__ inline const void* kept_row(const BwdArgs& A, int64_t row)
{
    if constexpr (HF == SNACK_INT8 || HF == SNACK_E4M3) return (const uint8_t*)A.H + row * A.per_row * kCkptBlock;
    else return (const typename HType<HF>::T*)A.H + row * A.n;
}

// dgain of 4 kGainLanes features by one workgroup: kGainLanes lanes a row, then the rows' sums in a fixed tree.  It
// needs no row's mean, so it runs beside the rows' workgroups.
template <int HF>
__device__ inline void gain_block(const BwdArgs& A, int block)
{
    constexpr int kDeep = 8;                     // rows a lane has in flight
    __shared__ f32x4 sums[16][kGainLanes];
    const int n = (int)A.n, f = 4 * (block * kGainLanes + (int)threadIdx.x % kGainLanes), left = n - f;
    const int r0 = (int)threadIdx.x / kGainLanes, step = (int)blockDim.x / kGainLanes;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t row = r0; row < A.rows; row += (int64_t)kDeep * step) {
        Kept<HF> kept[kDeep];
        f32x4 d[kDeep];
        float r[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int64_t at = row + (int64_t)k * step < A.rows ? row + (int64_t)k * step : A.rows - 1;
            kept[k].read(kept_row<HF>(A, at), A.HS + at * A.per_row, f, n);
            d[k] = read4(A.dY + at * A.n, f, n);
            r[k] = A.rstd[at];
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (row + (int64_t)k * step < A.rows) acc += kept4(d[k], left) * (kept[k].value(left) * r[k]);
    }
#pragma unroll
    for (int m = kGainLanes; m < kWave; m <<= 1) {
        acc.x += __shfl_xor(acc.x, m, kWave);
        acc.y += __shfl_xor(acc.y, m, kWave);
        acc.z += __shfl_xor(acc.z, m, kWave);
        acc.w += __shfl_xor(acc.w, m, kWave);
    }
    const int lane = (int)threadIdx.x & (kWave - 1), nw = (int)blockDim.x / kWave;
    if (lane < kGainLanes) sums[(int)threadIdx.x / kWave][lane] = acc;
    __syncthreads();
    if (threadIdx.x >= kGainLanes) return;
    acc = sums[0][lane];
    for (int w = 1; w < nw; ++w) acc += sums[w][lane];
    store4(A.dgain + f, acc, left);
}

// T: most threads of a workgroup: 256 for a wavefront a row, else of the workgroup that takes one.  With 1024
// there are 128 registers a thread, and the gain lies in LDS.
template <int HF, int T>
__global__ void __launch_bounds__(T) norm_bwd_kernel(BwdArgs A)
{
    constexpr bool WG = T > 256, GAIN_LDS = T > 512;
    if ((int)blockIdx.x >= A.groups) {
        gain_block<HF>(A, (int)blockIdx.x - A.groups);
        return;
    }
    __shared__ f32x4 gain[GAIN_LDS ? kChunks * T : 1];
    __shared__ float part[32];
    __shared__ float gsum[WG ? 1 : 3 * kWaveRow];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int t = WG ? (int)threadIdx.x : (int)threadIdx.x & (kWave - 1);
    const int nt = WG ? (int)blockDim.x : kWave;
    const int n = (int)A.n;
    const int64_t step = WG ? (int64_t)A.groups : (int64_t)A.groups * 4;
    const float inv_n = 1.0f / (float)A.n;
    f32x4 g[kChunks], acc[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int f = 4 * (t + i * nt);
        g[i] = kept4(read4(A.gain, f, n), n - f);
        if constexpr (GAIN_LDS) gain[t + i * T] = g[i];   // read by the thread that wrote it
        acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    int flip = 0;
    for (int64_t row = WG ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave; row < A.rows; row += step) {
        const float r = A.rstd[row];
        const void* h = kept_row<HF>(A, row);
        const uint8_t* hs = A.HS + row * A.per_row;
        const float* dy = A.dY + row * A.n;
        const float* dr = A.dR ? A.dR + row * A.n : nullptr;
        float* dx = A.dX + row * A.n;
        int n = (int)A.n;
        asm volatile("" : "+s"(n));   // keeps the offsets and tails of the row from being held across rows
        Kept<HF> kept[kChunks];
        f32x4 xh[kChunks], w[kChunks], e[kChunks];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int f = 4 * (t + i * nt);
            kept[i].read(h, hs, f, n);
            w[i] = read4(dy, f, n);
        }
        if (dr) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) e[i] = read4(dr, 4 * (t + i * nt), n);
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int left = n - 4 * (t + i * nt);
            xh[i] = kept[i].value(left) * r;
            w[i] = kept4(w[i], left);
            acc[i] += w[i] * xh[i];
            w[i] *= GAIN_LDS ? gain[t + i * T] : g[i];
            dot += dot4(w[i], xh[i]);
        }
        dot = WG ? group_sum(dot, part + 16 * flip) : wave_sum(dot);
        flip ^= 1;   // the next row's sums go to the other half, so one barrier a row is enough
        const float c = dot * inv_n;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int f = 4 * (t + i * nt);
            f32x4 o = (w[i] - xh[i] * c) * r;
            if (dr) o += kept4(e[i], n - f);
            store4((float*)at_bytes(dx, 4u * (uint32_t)f), o, n - f);
        }
    }
    if (!A.part) return;
    if constexpr (!WG) {
        // the workgroup's four wavefronts hold the same features: added in wavefront order
        if (wave > 0) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                *reinterpret_cast<f32x4*>(&gsum[(wave - 1) * kWaveRow + 4 * (t + i * kWave)]) = acc[i];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            for (int v = 0; v < 3; ++v)
                acc[i] += *reinterpret_cast<const f32x4*>(&gsum[v * kWaveRow + 4 * (t + i * kWave)]);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int f = 4 * (t + i * nt);
        store4(A.part + (int64_t)blockIdx.x * A.n + f, acc[i], n - f);
    }
}

// rows past kRowMax, first pass: mean(w xh) of each row
template <int HF>
__global__ void __launch_bounds__(kLongThreads) norm_bwd_mean_kernel(BwdArgs A)
{
    __shared__ float part[16];
    const int64_t row = blockIdx.x, base = row * A.n;
    const void* h = kept_row<HF>(A, row);
    const uint8_t* hs = A.HS + row * A.per_row;
    const float r = A.rstd[row];
    float dot = 0.0f;
    for (int64_t f = 4 * (int64_t)threadIdx.x; f < A.n; f += 4 * kLongThreads) {
        const int left = (int)(A.n - f);
        dot += dot4(load4(A.dY + base + f, left) * load4(A.gain + f, left), hidden_row4<HF>(h, hs, (int)f, (int)A.n) * r);
    }
    dot = group_sum(dot, part);
    if (threadIdx.x == 0) A.mean[row] = dot / (float)A.n;
}

// second pass: a workgroup takes 1024 columns (col0 and blockIdx.y) of rows blockIdx.x, + gridDim.x, ...
template <int HF>
__global__ void __launch_bounds__(kColThreads) norm_bwd_cols_kernel(BwdArgs A)
{
    const int64_t at0 = A.col0 + 4 * ((int64_t)blockIdx.y * kColThreads + threadIdx.x);
    if (at0 >= A.n) return;
    const int f = (int)at0, left = (int)(A.n - at0);
    const f32x4 g = load4(A.gain + f, left);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const float r = A.rstd[row], c = A.mean[row];
        const int64_t at = row * A.n + f;
        const f32x4 xh = hidden_row4<HF>(kept_row<HF>(A, row), A.HS + row * A.per_row, f, (int)A.n) * r;
        const f32x4 d = load4(A.dY + at, left);
        acc += d * xh;
        f32x4 o = (d * g - xh * c) * r;
        if (A.dR) o += load4(A.dR + at, left);
        store4(A.dX + at, o, left);
    }
    if (A.part) store4(A.part + (int64_t)blockIdx.x * A.n + f, acc, left);
}

// out[c] = sum of part[g][c], from column c0 on: 32 strided runs of rows, then the runs in order
__global__ void __launch_bounds__(kSumCols * kSumRows) part_sum_kernel(const float* __restrict__ part, int groups,
                                                                       int64_t n, int64_t c0, float* __restrict__ out)
{
    __shared__ float sh[kSumRows][kSumCols + 1];
    const int tx = (int)threadIdx.x % kSumCols, ty = (int)threadIdx.x / kSumCols;
    const int64_t c = c0 + (int64_t)blockIdx.x * kSumCols + tx;
    float a = 0.0f;
    if (c < n) {
#pragma unroll 8
        for (int g = ty; g < groups; g += kSumRows) a += part[(int64_t)g * n + c];
    }
    sh[ty][tx] = a;
    __syncthreads();
    if (ty == 0 && c < n) {
        for (int i = 1; i < kSumRows; ++i) a += sh[i][tx];
        out[c] = a;
    }
}

// rows that do not stay in registers, and those too short for read4
bool long_rows(int64_t n) { return n < 4 || n > kRowMax; }

// threads of a workgroup that takes a row of n features (kWaveRow < n <= kRowMax)
int row_threads(int64_t n) { return kWave * (int)((n + kWaveRow - 1) / kWaveRow); }

// Workgroups of the gradient, one partial row of dgain each: a fixed number of them rather than one a row (at
// 3333 x 4999 the partial rows are then a seventh of dY's bytes instead of all of them), the same number on every
// compute unit, of about ten wavefronts.  Measured with 1, 2, 3 and 4 a unit (us, int8 h): 1500 features (2
// wavefronts) 86, 50, 41, 40; 3000 (3) 52, 40, 41, 42; 4999 (5) 52, 44.5, 50, 53; 9000 (9) 52, 57, 61, 67;
// 16000 (16) 49, 55, 62, 68.
int bwd_groups(int64_t rows, int64_t n)
{
    int64_t most = kCus, g = rows;
    if (n <= kWaveRow) {
        g = (rows + 3) / 4;
        most *= n > kWaveRow / 2 ? kBwdWaves / 4 : kBwdPerCu;   // 20000 x 200: 25.8 us with two, 20.9 with four
    } else if (n <= kRowMax) {
        const int per_cu = kBwdWaves / (row_threads(n) / kWave);
        most *= per_cu < 1 ? 1 : per_cu > kBwdPerCu ? kBwdPerCu : per_cu;
    }
    return (int)(g < most ? g : most);
}

// Whether dgain is summed beside the rows in the same launch, which reads dY and h twice and walks all rows in every
// workgroup, instead of from partial rows.  Measured (us a call replayed from a graph, partial rows : beside, int8 h):
// 256 x 768 6.4 : 3.7, 1024 x 768 6.8 : 5.9 (called in turn, where the host's second launch counts, 13.2 : 10.5),
// 1024 x 200 7.0 : 5.8, 1024 x 1500 12.7 : 10.7, 256 x 4999 10.5 : 8.2, 100 x 15000 12.9 : 14.2; past the rule (us on
// the GPU) 1536 x 768 9.9 : 10.3, 2048 x 1500 15.8 : 18.9, 512 x 4999 15.6 : 17.7.
bool gain_beside(int64_t rows, int64_t n) { return rows > 0 && rows <= 1024 && !long_rows(n) && rows * n <= 3 << 19; }

bool bad_size(int64_t rows, int64_t n) { return n >= (1ll << 31) - kCkptBlock || rows >= (1ll << 31); }
inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// a pointer moved by so many elements; null stays null
template <typename T>
T* moved(T* p, int64_t by) { return p ? p + by : nullptr; }

// the call's rows from r0 on, at most `rows` of them
template <int HF>
FwdArgs rows_from(FwdArgs A, int64_t r0, int64_t rows)
{
    using T = typename HType<HF>::T;
    A.X += r0 * A.n;
    A.R = moved((const T*)A.R, r0 * A.n);
    A.H = moved((T*)A.H, r0 * A.n);
    A.Y = moved(A.Y, r0 * A.n);
    A.rstd += r0;
    A.Q = moved(A.Q, r0 * A.per_row * kCkptBlock);
    A.S = moved(A.S, r0 * A.per_row);
    A.rows = A.rows - r0 < rows ? A.rows - r0 : rows;
    return A;
}

template <int HF, int QF>
void launch_fwd(const FwdArgs& all, hipStream_t s)
{
    const int threads = long_rows(all.n) ? kLongThreads : all.n <= kWaveRow ? kWave : row_threads(all.n);   // a row
    const int64_t most = kLaunchThreads / threads;
    for (int64_t r0 = 0; r0 < all.rows; r0 += most) {
        const FwdArgs A = rows_from<HF>(all, r0, most);
        if (long_rows(A.n))
            hipLaunchKernelGGL((norm_fwd_long_kernel<HF, QF>), dim3((unsigned)A.rows), dim3(threads), 0, s, A);
        else if (A.n <= kWaveRow)
            hipLaunchKernelGGL((norm_fwd_kernel<HF, QF, false>), dim3((unsigned)((A.rows + 3) / 4)), dim3(256), 0, s, A);
        else
            hipLaunchKernelGGL((norm_fwd_kernel<HF, QF, true>), dim3((unsigned)A.rows), dim3(threads), 0, s, A);
    }
}
template <int HF>
void launch_fwd(const FwdArgs& A, int q_fmt, hipStream_t s)
{
    if (q_fmt == SNACK_INT8) launch_fwd<HF, SNACK_INT8>(A, s);
    else if (q_fmt == SNACK_E4M3) launch_fwd<HF, SNACK_E4M3>(A, s);
    else launch_fwd<HF, SNACK_F32>(A, s);
}

template <int HF>
void launch_bwd(const BwdArgs& A, hipStream_t s)
{
    const unsigned grid = (unsigned)A.groups + (A.dgain ? (unsigned)((A.n + 4 * kGainLanes - 1) / (4 * kGainLanes)) : 0u);
    if (long_rows(A.n)) {
        constexpr int64_t most = kLaunchThreads / kLongThreads;
        for (int64_t r0 = 0; r0 < A.rows; r0 += most) {
            BwdArgs P = A;
            P.H = kept_row<HF>(A, r0);
            P.HS = moved(A.HS, r0 * A.per_row);
            P.rstd += r0;
            P.dY += r0 * A.n;
            P.mean += r0;
            const int64_t rows = A.rows - r0 < most ? A.rows - r0 : most;
            hipLaunchKernelGGL(norm_bwd_mean_kernel<HF>, dim3((unsigned)rows), dim3(kLongThreads), 0, s, P);
        }
        const int64_t cols = (A.n + 4 * kColThreads - 1) / (4 * kColThreads);
        for (int64_t c = 0; c < cols; c += kLaunchY) {
            BwdArgs P = A;
            P.col0 = c * 4 * kColThreads;
            const unsigned y = (unsigned)(cols - c < kLaunchY ? cols - c : kLaunchY);
            hipLaunchKernelGGL(norm_bwd_cols_kernel<HF>, dim3((unsigned)A.groups, y), dim3(kColThreads), 0, s, P);
        }
    } else if (A.n <= kWaveRow) {
        hipLaunchKernelGGL((norm_bwd_kernel<HF, 256>), dim3(grid), dim3(256), 0, s, A);
    } else {
        const int threads = row_threads(A.n);
        const auto k = threads <= 512 ? norm_bwd_kernel<HF, 512> : norm_bwd_kernel<HF, 1024>;
        hipLaunchKernelGGL(k, dim3(grid), dim3(threads), 0, s, A);
    }
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" snack_status snack_rmsnorm_fwd(const float* X, const void* R, int32_t h_fmt, const float* gain, float eps,
                                          int64_t rows, int64_t n, void* H, float* Y, float* rstd, int32_t q_fmt,
                                          uint8_t* Q, uint8_t* S, snack_stream stream)
{
    if (rows < 0 || n < 1 || !(eps >= 0.0f) || (h_fmt != SNACK_F32 && h_fmt != SNACK_BF16)) return SNACK_ERR_INVALID_ARG;
    if (bad_size(rows, n)) return SNACK_ERR_UNSUPPORTED;
    if (rows == 0) return SNACK_OK;
    if (!X || !gain || !rstd || !R != !H || !Q != !S || (Q && !ckpt_format(q_fmt)) || (!Y && !Q))
        return SNACK_ERR_INVALID_ARG;
    const uintptr_t ha = h_fmt == SNACK_BF16 ? 2 : 4;
    if (misaligned(X, 4) || misaligned(gain, 4) || misaligned(rstd, 4) || misaligned(Y, 4) || misaligned(R, ha) ||
        misaligned(H, ha) || misaligned(Q, 16))
        return SNACK_ERR_INVALID_ARG;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_NORM, s);
    const int64_t out = rows * n * ((H ? (int64_t)ha : 0) + (Y ? 4 : 0) + (Q ? 1 : 0));
    const FwdArgs A{X, R, gain, H, Y, rstd, Q, S, rows, n, (n + kCkptBlock - 1) / kCkptBlock, eps, out > kStreamBytes};
    const int qf = Q ? q_fmt : (int)SNACK_F32;
    if (h_fmt == SNACK_BF16 && R) launch_fwd<SNACK_BF16>(A, qf, s);
    else launch_fwd<SNACK_F32>(A, qf, s);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

extern "C" snack_status snack_rmsnorm_bwd_work(int64_t rows, int64_t n, int64_t* bytes)
{
    if (!bytes || rows < 0 || n < 1) return SNACK_ERR_INVALID_ARG;
    if (bad_size(rows, n)) return SNACK_ERR_UNSUPPORTED;
    *bytes = 4 * ((int64_t)bwd_groups(rows, n) * n + (long_rows(n) ? rows : 0));
    return SNACK_OK;
}

extern "C" snack_status snack_rmsnorm_bwd(const void* H, const uint8_t* HS, int32_t h_fmt, const float* gain,
                                          const float* rstd, const float* dY, const float* dR, int64_t rows, int64_t n,
                                          float* dX, float* dgain, void* work, int64_t work_bytes, snack_stream stream)
{
    if (rows < 0 || n < 1) return SNACK_ERR_INVALID_ARG;
    if (h_fmt != SNACK_F32 && h_fmt != SNACK_BF16 && !ckpt_format(h_fmt)) return SNACK_ERR_INVALID_ARG;
    if (bad_size(rows, n)) return SNACK_ERR_UNSUPPORTED;
    int64_t need = 0;
    SNACK_CHECK(snack_rmsnorm_bwd_work(rows, n, &need));
    if (rows > 0) {
        if (!H || (ckpt_format(h_fmt) && !HS) || !gain || !rstd || !dY || !dX) return SNACK_ERR_INVALID_ARG;
        const uintptr_t ha = ckpt_format(h_fmt) ? 16 : h_fmt == SNACK_BF16 ? 2 : 4;
        if (misaligned(H, ha) || misaligned(gain, 4) || misaligned(rstd, 4) || misaligned(dY, 4) ||
            misaligned(dR, 4) || misaligned(dX, 4))
            return SNACK_ERR_INVALID_ARG;
        if (dgain || long_rows(n)) {
            if (!work || misaligned(work, 4)) return SNACK_ERR_INVALID_ARG;
            if (work_bytes < need) return SNACK_ERR_WORKSPACE;
        }
    }
    if (misaligned(dgain, 4)) return SNACK_ERR_INVALID_ARG;
    if (rows == 0 && !dgain) return SNACK_OK;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    ProfScope prof(KC_NORM, s);
    const int groups = bwd_groups(rows, n);
    const bool beside = gain_beside(rows, n);
    float* mean = (float*)work;
    float* part = (float*)work + (long_rows(n) ? rows : 0);
    if (rows > 0) {
        const BwdArgs A{H, HS, gain, rstd, dY, dR, dX, dgain && !beside ? part : nullptr, mean, rows, n,
                        (n + kCkptBlock - 1) / kCkptBlock, beside ? dgain : nullptr, groups, 0};
        switch (h_fmt) {
        case SNACK_F32: launch_bwd<SNACK_F32>(A, s); break;
        case SNACK_BF16: launch_bwd<SNACK_BF16>(A, s); break;
        case SNACK_INT8: launch_bwd<SNACK_INT8>(A, s); break;
        default: launch_bwd<SNACK_E4M3>(A, s); break;
        }
        SNACK_HIP(hipGetLastError());
    }
    if (dgain && !beside) {
        // no rows: no partial rows, and the sum over none of them is 0
        constexpr int64_t most = kLaunchThreads / kSumRows;   // columns
        for (int64_t c0 = 0; c0 < n; c0 += most) {
            const int64_t cols = n - c0 < most ? n - c0 : most;
            hipLaunchKernelGGL(part_sum_kernel, dim3((unsigned)((cols + kSumCols - 1) / kSumCols)),
                               dim3(kSumCols * kSumRows), 0, s, part, groups, n, c0, dgain);
        }
        SNACK_HIP(hipGetLastError());
    }
    return SNACK_OK;
}
