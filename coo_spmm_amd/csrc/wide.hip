// wide.hip -- the passes of wide batches (more than one 64-column batch tile)
// over views whose keys hold few entries: the 99 %-sparse layers of a
// transformer MLP at a thousand tokens, where a key's handful of entries
// gives the slice-tiled and key-major kernels too little to share per load.
//
// wide_spmm_kernel (forward over the row view, dX over the column view):
//   out[b, j] = sum over the entries e of key j of v_e * ft[idx_e, b]
// with ft the feature-major operand [nidx][bp] (zero past the batch).  A
// workgroup takes 64 batch columns (one per lane) and a block of keys, a
// wavefront a run of 1-4 consecutive keys, whose entries it streams as one
// run: the indices and values are uniform (scalar loads), every entry is one
// coalesced 256-byte row segment of ft from L2 and one fused multiply-add per
// lane, in entry order.  The key x column tile goes through LDS so that the
// batch-major stores are whole rows.
//
// wide_sddmm_kernel (dW over the canonical entries):
//   dW[e] = sum over b of dyt[r_e, b] * xt[c_e, b]
// lane l of a wavefront sums the columns l, l + 64, ... of an entry in order,
// then a fixed butterfly adds the 64 lane sums.  A wavefront takes one entry, or
// four consecutive ones, which share the row of dyt where they lie in one row
// (five operand rows from L2 for four entries instead of eight).
#include "internal.h"
#include <type_traits>

namespace snack {
namespace {

constexpr int kWideThreads = 256;              // the dW pass
constexpr int kWideWaves = kWideThreads / kWave;
constexpr int kWideSpmmThreads = 1024;         // the SpMM pass: 16 wavefronts, 1 to 4 keys each
constexpr int kWideSpmmWaves = kWideSpmmThreads / kWave;
constexpr int kWideU = 8;            // entries whose operand rows are loaded together
constexpr int kWideShortKey = 40;    // most entries per key (on average) for these passes

template <int R>
__global__ void __launch_bounds__(kWideSpmmThreads)
wide_spmm_kernel(const int32_t* __restrict__ ptr, const int32_t* __restrict__ idx, const float* __restrict__ vals,
                 int32_t nkeys, const float* __restrict__ ft, int32_t bp, int32_t B, float* __restrict__ out)
{
    constexpr int KPW = R / kWideSpmmWaves;   // consecutive keys of one wavefront
    __shared__ float tile[R][kWave + 1];
    const int32_t j0 = (int32_t)blockIdx.x * R;
    const int32_t t0 = (int32_t)blockIdx.y * kWave;
    const int lane = (int)(threadIdx.x & (kWave - 1));
    // the wavefront index is uniform: said so, every key index and address below is too (scalar loads)
    const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const float* __restrict__ col = ft + t0 + lane;
    const int32_t jw = j0 + wv * KPW;                            // the wavefront's first key
    int kl = 0;                                                  // its key being summed
    float acc = 0.0f;
    if (jw < nkeys) {
        const int32_t jn = jw + KPW < nkeys ? jw + KPW : nkeys;
        // the keys' entries are one run: taken in groups whose loads are all issued first, a key's
        // sum going to LDS where the next key's entries begin
        const int32_t P1 = ptr[jn];
        int32_t kend = ptr[jw + 1];
        for (int32_t e0 = ptr[jw]; e0 < P1; e0 += kWideU) {
            const int32_t n = P1 - e0;
            // the arrays are padded past nnz, so the loads of a short last group stay in bounds;
            // their lanes' sums are not changed (a zero product of a non-finite operand would be NaN)
            int32_t c[kWideU];
            float v[kWideU], x[kWideU];
#pragma unroll
            for (int u = 0; u < kWideU; ++u) {
                c[u] = u < n ? idx[e0 + u] : 0;
                v[u] = vals[e0 + u];
            }
#pragma unroll
            for (int u = 0; u < kWideU; ++u) x[u] = col[(int64_t)c[u] * bp];
#pragma unroll
            for (int u = 0; u < kWideU; ++u) {
                if (u >= n) break;
                while (e0 + u >= kend) {   // the next key (empty keys pass straight through)
                    tile[wv * KPW + kl][lane] = acc;
                    acc = 0.0f;
                    ++kl;
                    kend = ptr[jw + kl + 1];
                }
                acc = fmaf(v[u], x[u], acc);
            }
        }
    }
    for (; kl < KPW; ++kl) {   // the last key summed, and keys with no entries after it
        tile[wv * KPW + kl][lane] = acc;
        acc = 0.0f;
    }
    __syncthreads();
    // the tile's rows of out: column t0 + tt, keys j0 .. j0 + R - 1
    for (int q = (int)threadIdx.x; q < kWave * R; q += kWideSpmmThreads) {
        const int tt = q / R, jj = q % R;
        const int32_t b = t0 + tt, j = j0 + jj;
        if (b < B && j < nkeys) out[(int64_t)b * nkeys + j] = tile[jj][tt];
    }
}

template <int E>
__global__ void __launch_bounds__(kWideThreads)
wide_sddmm_kernel(const int32_t* __restrict__ rows, const int32_t* __restrict__ cols, int64_t nnz,
                  const float* __restrict__ xt, const float* __restrict__ dyt, int32_t bp, float* __restrict__ dW)
{
    const int lane = (int)(threadIdx.x & (kWave - 1));
    const int64_t wave0 = (int64_t)blockIdx.x * kWideWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int64_t nwaves = (int64_t)gridDim.x * kWideWaves;
    // the sums of n consecutive entries of one row (their columns' copies: the arrays are padded past nnz)
    auto entries = [&](int64_t e, auto count, int n) {
        constexpr int N = decltype(count)::value;
        const float* __restrict__ y = dyt + (int64_t)rows[e] * bp + lane;
        const float* __restrict__ x[N];
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = xt + (int64_t)cols[i < n ? e + i : e] * bp + lane;
            acc[i] = 0.0f;
        }
        int32_t b = 0;
        for (; b + 4 * kWave <= bp; b += 4 * kWave) {
            float yy[4], xx[N][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) yy[u] = y[b + u * kWave];
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) xx[i][u] = x[i][b + u * kWave];
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[i] = fmaf(yy[u], xx[i][u], acc[i]);
        }
        for (; b < bp; b += kWave) {
            const float yy = y[b];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(yy, x[i][b], acc[i]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int d = kWave / 2; d >= 1; d >>= 1) acc[i] += __shfl_xor(acc[i], d, kWave);
            if (lane == 0 && i < n) dW[e + i] = acc[i];
        }
    };
    for (int64_t e = wave0 * E; e < nnz; e += nwaves * E) {
        const int n = nnz - e < E ? (int)(nnz - e) : E;
        if (E == 1 || rows[e] == rows[e + n - 1]) {   // rows ascend
            entries(e, std::integral_constant<int, E>(), n);
        } else {
            for (int i = 0; i < n; ++i) entries(e + i, std::integral_constant<int, 1>(), 1);
        }
    }
}

}  // namespace

bool wide_short(const snack_layer* L, const View& v, const BatchPlan& p)
{
    return p.ntiles > 1 && p.bp % kWave == 0 && L->nnz > 0 && v.nkeys > 0 &&
           L->nnz <= (int64_t)kWideShortKey * v.nkeys;
}

snack_status wide_spmm(const snack_layer* L, const View& v, const float* ft, const BatchPlan& p, int B, float* out,
                       hipStream_t s)
{
    if (!wide_short(L, v, p)) return SNACK_ERR_INVALID_ARG;
    const unsigned ty = (unsigned)(p.bp / kWave);
    // keys per workgroup: the largest of 64, 32, 16 that still gives about eight wavefronts per SIMD
    auto kblocks = [&](int R) { return (int64_t)(v.nkeys + R - 1) / R; };
    if (kblocks(64) * ty * kWideSpmmWaves >= 8192)
        hipLaunchKernelGGL(wide_spmm_kernel<64>, dim3((unsigned)kblocks(64), ty), dim3(kWideSpmmThreads), 0, s, v.ptr,
                           v.idx, v.vals, v.nkeys, ft, p.bp, B, out);
    else if (kblocks(32) * ty * kWideSpmmWaves >= 8192)
        hipLaunchKernelGGL(wide_spmm_kernel<32>, dim3((unsigned)kblocks(32), ty), dim3(kWideSpmmThreads), 0, s, v.ptr,
                           v.idx, v.vals, v.nkeys, ft, p.bp, B, out);
    else
        hipLaunchKernelGGL(wide_spmm_kernel<16>, dim3((unsigned)kblocks(16), ty), dim3(kWideSpmmThreads), 0, s, v.ptr,
                           v.idx, v.vals, v.nkeys, ft, p.bp, B, out);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

snack_status wide_sddmm(const snack_layer* L, const float* xt, const float* dyt, const BatchPlan& p, float* dW,
                        hipStream_t s)
{
    if (!wide_short(L, L->fwd, p)) return SNACK_ERR_INVALID_ARG;
    auto go = [&](auto kern, int per_wave) {
        int64_t blocks = (L->nnz + kWideWaves * per_wave - 1) / (kWideWaves * per_wave);
        if (blocks > 65536) blocks = 65536;
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kWideThreads), 0, s, L->rows, L->cols, L->nnz, xt, dyt,
                           p.bp, dW);
    };
    // The bits are the same.  Four entries a wavefront save launches of wavefronts in narrow batches and reads of dyt
    // where rows are long enough to be shared; in wide batches over short rows neither counts, and a group that
    // crosses a row runs its entries one after the other.  Measured (us, a call for dW, one : four), 3000 columns:
    //   8000 entries,  2048 batch rows 27.0 : 31.4;  23592 entries, 1000 batch rows 27.0 : 26.9
    //   100000 entries, 1 a row:  256 batch rows 61 : 55, 384 92 : 89, 768 177 : 185, 2048 504 : 540
    //                   2 a row:  384 batch rows 66 : 60, 512 76 : 76, 768 115 : 126, 2048 317 : 374
    //                   4 a row:  512 batch rows 56 : 52, 768 82 : 89;    8 a row: 768 65 : 63, 1024 87 : 91
    //                  16 a row: 1024 batch rows 115 : 112, 2048 218 : 221;  30 a row: 2048 189 : 183
    if (L->nnz >= 32768 && p.bp <= 384 + 56 * (L->nnz / L->M)) go(wide_sddmm_kernel<4>, 4);
    else go(wide_sddmm_kernel<1>, 1);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

}  // namespace snack
