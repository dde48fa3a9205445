// operands.hip -- what a layer's gradient passes read, made from the batch-major dY
// [B][M] and the checkpoint of x [B][K] in one launch.
//
//   feature-major copies   f[c * bp + b], 0 for B <= b < bp: the passes over the
//                          stored positions
//   instruction operands   32 features x 16 batch rows, a kilobyte, 16 bytes a lane
//                          (lane l: feature l % 32, batch rows 8 (l / 32) ...), in bf16:
//                          dY as three exact parts, x as it is: the tiles of sample.hip
//
// Bound by HBM.  A workgroup takes 64 features of 64 batch rows through LDS, so both
// sides move in whole lines: rows of 256 (dY) or 64 bytes (codes, 16 a lane) in, runs
// of 256 bytes of a feature or kilobytes of an operand out.  One launch for all of it:
// 12.4 us at 3072 x 768 and 1024 rows (46 MB; 17.2 us as two launches that each read
// dY), 10.4 us at 768 x 3072 and 1000 rows (22 MB; 15.8 us as two).
#include "ckpt.h"

namespace snack {
namespace {

constexpr int kTile = 64;
constexpr int kStep = kSampleStep;

// the three bf16 parts of x (hi + mid + lo = x, exactly for |x| >= 2^-109, below which lo ends at
// bf16's smallest step of 2^-133); an infinity or NaN is all in the first
__device__ inline void split3(float x, uint16_t& hi, uint16_t& mid, uint16_t& lo)
{
    const uint32_t b = __float_as_uint(x);
    const bool fin = (b & 0x7F800000u) != 0x7F800000u;
    const float r1 = x - __uint_as_float(b & 0xFFFF0000u);
    const uint32_t b1 = fin ? __float_as_uint(r1) : 0u;
    const float r2 = __uint_as_float(b1) - __uint_as_float(b1 & 0xFFFF0000u);
    const uint32_t nan = (b & 0x7FFFFFFFu) > 0x7F800000u ? 0x40u : 0u;
    hi = (uint16_t)((b >> 16) | nan);
    mid = (uint16_t)(b1 >> 16);
    lo = (uint16_t)(__float_as_uint(r2) >> 16);
}

__device__ inline uint4 pack8(const uint16_t* v)
{
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

struct OperandArgs {
    const float* dY;      // [B][M]
    const uint8_t* Q;     // [B][32 per_row]
    const uint8_t* S;     // [B][per_row]
    float* dyt;           // [M][bp], or null
    float* xt;            // [K][bp], or null
    uint4* A;             // [32-row blocks][steps][3][64], or null
    uint4* X;             // [32-column blocks][steps][64], or null
    int M, K, B, bp, per_row, steps, mtiles;
};

template <int FMT>
__global__ void __launch_bounds__(256) layer_operands_kernel(OperandArgs P)
{
    __shared__ float tile[kTile][kTile + 1];   // [batch row][feature]
    const int tid = (int)threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const bool of_dy = (int)blockIdx.x < P.mtiles;
    const int c0 = (of_dy ? (int)blockIdx.x : (int)blockIdx.x - P.mtiles) * kTile, b0 = (int)blockIdx.y * kTile;
    if (of_dy) {
        const int c = c0 + 4 * (tid & 15), left = P.M - c;
        f32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int b = b0 + (tid >> 4) + 16 * k;
            v[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const float* p = P.dY + (int64_t)b * P.M + c;
            if (b < P.B) {
                if (left >= 4) {
                    v[k] = *reinterpret_cast<const f32x4u*>(p);
                } else {
                    if (left > 0) v[k].x = p[0];
                    if (left > 1) v[k].y = p[1];
                    if (left > 2) v[k].z = p[2];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float* t = &tile[(tid >> 4) + 16 * k][4 * (tid & 15)];
            t[0] = v[k].x;
            t[1] = v[k].y;
            t[2] = v[k].z;
            t[3] = v[k].w;
        }
    } else {
        const int b = b0 + (tid >> 2), part = tid & 3, blk = c0 / kCkptBlock + (part >> 1);
        uint4 w = make_uint4(0, 0, 0, 0);
        float sc = 0.0f;
        if (b < P.B && blk < P.per_row) {
            const int64_t at = (int64_t)b * P.per_row + blk;
            w = reinterpret_cast<const uint4*>(P.Q)[at * 2 + (part & 1)];
            sc = ckpt_scale(P.S[at]);
        }
        float* t = &tile[tid >> 2][16 * part];
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 v = ckpt_codes4<FMT>(q[i]) * sc;
            t[4 * i] = v.x;
            t[4 * i + 1] = v.y;
            t[4 * i + 2] = v.z;
            t[4 * i + 3] = v.w;
        }
    }
    __syncthreads();

    float* const ft = of_dy ? P.dyt : P.xt;
    if (ft) {
        const int n = of_dy ? P.M : P.K;
        if ((P.bp & 3) == 0) {   // four batch rows a lane, four features a wavefront
            const int b = 4 * (lane & 15);
            if (b0 + b < P.bp) {
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i) {
                    const int cc = 16 * i + 4 * wave + (lane >> 4);
                    const f32x4 v = {tile[b][cc], tile[b + 1][cc], tile[b + 2][cc], tile[b + 3][cc]};
                    if (c0 + cc < n) *reinterpret_cast<f32x4*>(ft + (int64_t)(c0 + cc) * P.bp + b0 + b) = v;
                }
            }
        } else if (b0 + lane < P.bp) {   // two batch rows
            for (int cc = wave; cc < kTile; cc += 4)
                if (c0 + cc < n) ft[(int64_t)(c0 + cc) * P.bp + b0 + lane] = tile[lane][cc];
        }
    }
    if (!(of_dy ? P.A : P.X)) return;
    const int blocks = ((of_dy ? P.M : P.K) + 31) / 32;
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // wavefront w: step w of the tile, both blocks of 32 features
        const int blk = c0 / 32 + i, step = (int)blockIdx.y * (kTile / kStep) + wave;
        if (blk >= blocks || step >= P.steps) continue;
        const float* t = &tile[wave * kStep + 8 * (lane >> 5)][32 * i + (lane & 31)];
        const int64_t at = (int64_t)blk * P.steps + step;
        uint16_t hi[8];
        if (of_dy) {
            uint16_t mid[8], lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(t[j * (kTile + 1)], hi[j], mid[j], lo[j]);
            uint4* out = P.A + at * 3 * kWave + lane;
            out[0] = pack8(hi);
            out[kWave] = pack8(mid);
            out[2 * kWave] = pack8(lo);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) hi[j] = bf16_bits(t[j * (kTile + 1)]);   // exact: eight significant bits
            P.X[at * kWave + lane] = pack8(hi);
        }
    }
}

}  // namespace

snack_status layer_operands(const snack_layer* L, const uint8_t* Q, const uint8_t* S, int fmt, const float* dY, int B,
                            int bp, const LayerOperands& out, hipStream_t s)
{
    ProfScope prof(KC_TRANSPOSE, s);
    OperandArgs a;
    a.dY = dY;
    a.Q = Q;
    a.S = S;
    a.dyt = out.dyt;
    a.xt = out.xt;
    a.A = (uint4*)out.a;
    a.X = (uint4*)out.x;
    a.M = L->M;
    a.K = L->K;
    a.B = B;
    a.bp = bp;
    a.per_row = (L->K + kCkptBlock - 1) / kCkptBlock;
    a.steps = (B + kStep - 1) / kStep;
    a.mtiles = (L->M + kTile - 1) / kTile;
    const dim3 grid((unsigned)(a.mtiles + (L->K + kTile - 1) / kTile), (unsigned)((bp + kTile - 1) / kTile));
    const auto k = fmt == SNACK_INT8 ? layer_operands_kernel<SNACK_INT8> : layer_operands_kernel<SNACK_E4M3>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

}  // namespace snack
