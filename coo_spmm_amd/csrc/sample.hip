// sample.hip -- dW on the support from a checkpointed input, by matrix instructions.
//
//   dW[k] = sum_b dY[b, r_k] x[b, c_k]
//
// Walking the stored positions costs every entry two operand rows of B values, so
// past about one position in 64 it is cheaper to compute whole tiles of dY^T X on
// the matrix cores and keep only the stored positions.  A wavefront's registers
// hold 32 x 128 cells; they go to LDS 16 rows at a time, from where the stored
// ones are read and written to dW.  (Tiles of 64 x 128, half the operand reads a
// cell but two wavefronts a SIMD instead of four: no faster anywhere, 61.7 us
// against 55.7 at 10000 x 10000, 90 %, 64 batch rows.)  The dense product itself
// never leaves the CU.
//
// Which cells are stored comes from a list in tile order (32 rows x 128 columns a
// tile, row-major within it), made once after every change of the index: 4 bytes
// a position, read in whole lines and known before the product starts.  (Reading
// each row's run of column indices instead, eight lanes a row, left a dependent
// load behind every run longer than eight: 65 us against 42 at 10000 x 10000,
// 95 %, 64 batch rows.)
//
// fp32 accuracy from bf16 instructions: an fp32 number is the exact sum of three
// bf16 numbers (its 24 significant bits in three runs of eight, taken by
// truncation, so nothing overflows), and a checkpoint's value has at most eight
// significant bits, so it is one bf16 number.  Three products, each exact, are
// added in fp32: what is rounded is the sums alone, as in a chain of fp32
// multiply-adds.  Against a checkpoint this costs half of what two fp32
// operands would (six products).
//
// Both operands come in the order in which the matrix instruction takes them (32
// rows or columns x 16 batch rows, a kilobyte, 16 bytes a lane; operands.hip), so
// the product's loads are whole kilobytes from L2 into registers, without LDS and
// without barriers.
#include "ckpt.h"

namespace snack {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kStep = kSampleStep;
constexpr int kCols = 128;            // columns of a tile
constexpr int kCB = kCols / 32;
constexpr int kCellBits = 12;         // a cell of a tile: 32 x 128
constexpr int kSampleMaxK = 32640;    // columns at most: a slot of a 32-row panel then fits the other 20 bits,
                                      // and the list kernel's tables 64 KB
constexpr int kAhead = 4;             // list words a lane holds
constexpr int kStage = 16 * kCols;    // cells a wavefront stages at once: half a tile
constexpr int kListThreads = 1024;    // workgroup of a panel's list
constexpr int kXcd = 8;
constexpr int kFragBytes = kWave * 16;   // one instruction's operand

// The tile list of one panel of 32 rows by one workgroup.  A panel's positions are
// one run of the canonical order; the list holds the same run in tile order:
// list[i] = (slot - panel's first slot) << 12 | row in panel * 128 + column in tile, and
// tile_ptr[panel * tiles + t] the place of tile t's first.  Every entry's place follows from
// where its row enters its tile, so nothing is counted by atomics.  Bound by the latency of a row's
// loads: two rows a wavefront (10000 x 10000, 95 %: 38 us; 66 with eight).
__global__ void __launch_bounds__(kListThreads) sample_list_kernel(const int32_t* __restrict__ ptr,
                                                          const int32_t* __restrict__ cols, int M, int tiles,
                                                          uint32_t* __restrict__ list, int32_t* __restrict__ tile_ptr)
{
    extern __shared__ int32_t at[];   // [32][tiles + 1]: a row's first entry in tile t or later; then [32][tiles] places
    const int lane = (int)threadIdx.x & (kWave - 1), wave = (int)threadIdx.x / kWave;
    const int r0 = (int)blockIdx.x * 32, nr = min(32, M - r0);
    const int w = tiles + 1;
    int32_t* place = at + 32 * w;
    const int32_t base = ptr[r0];
    for (int r = wave; r < 32; r += kListThreads / kWave) {
        const int32_t lo = r < nr ? ptr[r0 + r] : ptr[M], hi = r < nr ? ptr[r0 + r + 1] : ptr[M];
        for (int32_t e = lo + lane; e < hi; e += kWave) {
            const int t = cols[e] / kCols, before = e > lo ? cols[e - 1] / kCols : -1;
            for (int s = before + 1; s <= t; ++s) at[r * w + s] = e;
        }
        const int last = hi > lo ? cols[hi - 1] / kCols : -1;
        for (int s = last + 1 + lane; s <= tiles; s += kWave) at[r * w + s] = hi;
    }
    __syncthreads();
    // a tile's entries before each row, then (one wavefront) the tiles' places
    for (int t = (int)threadIdx.x; t < tiles; t += kListThreads) {
        int32_t n = 0;
        for (int r = 0; r < 32; ++r) {
            place[r * tiles + t] = n;
            n += at[r * w + t + 1] - at[r * w + t];
        }
    }
    __syncthreads();
    if (wave == 0) {
        int32_t carry = base;
        for (int t0 = 0; t0 < tiles; t0 += kWave) {
            const int t = t0 + lane;
            const int32_t n = t < tiles ? place[31 * tiles + t] + at[31 * w + t + 1] - at[31 * w + t] : 0;
            int32_t x = n;
            for (int d = 1; d < kWave; d <<= 1) {
                const int32_t y = __shfl_up(x, d, kWave);
                if (lane >= d) x += y;
            }
            const int32_t first = carry + x - n;
            if (t < tiles) {
                tile_ptr[(int64_t)blockIdx.x * tiles + t] = first;
                for (int r = 0; r < 32; ++r) place[r * tiles + t] += first;
            }
            carry += __shfl(x, kWave - 1, kWave);
        }
        if (lane == 0 && blockIdx.x == gridDim.x - 1) tile_ptr[(int64_t)gridDim.x * tiles] = carry;
    }
    __syncthreads();
    for (int r = wave; r < nr; r += kListThreads / kWave) {
        for (int32_t e = ptr[r0 + r] + lane; e < ptr[r0 + r + 1]; e += kWave) {
            const int c = cols[e], t = c / kCols;
            list[place[r * tiles + t] + e - at[r * w + t]] =
                (uint32_t)(e - base) << kCellBits | (uint32_t)(r * kCols + c % kCols);
        }
    }
}

struct SampleArgs {
    const uint4* A;
    const uint4* X;
    const uint32_t* list;
    const int32_t* tile_ptr;
    const int32_t* row_ptr;
    float* dW;
    int steps, rblocks, cblocks;
    int tiles;             // across; rblocks of them down
    int per_xcd;           // workgroups an XCD takes
    uint32_t a_bytes, x_bytes;
};

// KS: wavefronts of the workgroup that share a tile, each a KS-th of the batch rows;
// their sums are added, in wavefront order, where the positions are read.
template <int KS>
__global__ void __launch_bounds__(256, 4) sample_kernel(SampleArgs P)
{
    __shared__ float stage[4][kStage];
    const int lane = (int)threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int ks = wave % KS;
    // an XCD takes a contiguous run of tiles, column tiles first: a panel's rows stay in its L2, and
    // the pieces of a row's dW that neighbouring tiles write meet there
    const int64_t unit = (int64_t)(blockIdx.x % kXcd) * P.per_xcd + blockIdx.x / kXcd;
    const int64_t tile = unit * (4 / KS) + wave / KS;
    const bool live = tile < (int64_t)P.rblocks * P.tiles;
    if (KS == 1 && !live) return;
    // with KS > 1 the workgroup's wavefronts meet at barriers: one past the end repeats the last tile and stores nothing
    const int64_t id = live ? tile : (int64_t)P.rblocks * P.tiles - 1;
    const int panel = (int)((uint32_t)id / (uint32_t)P.tiles);
    const int ct = (int)((uint32_t)id - (uint32_t)panel * (uint32_t)P.tiles);

    // the first positions this wavefront stores: the words ks * 64 + lane, + 64 KS, ... of the tile's list
    const int32_t pos = P.tile_ptr[id] + ks * kWave + lane;
    const int32_t p1 = live ? P.tile_ptr[id + 1] : 0;
    uint32_t word[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)   // the list is padded: reads past the tile's end stay in bounds
        word[k] = P.list[pos + k * KS * kWave];

    f32x16 acc[kCB];
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[cb][i] = 0.0f;

    if (ks < P.steps) {
        // Loads through buffer descriptors: the block's offset is a scalar, the lane's a constant, and a
        // load stays where it is written (an ordinary load that is carried round the loop gets moved to
        // its use).  Blocks past the matrix repeat the last one (their cells hold no position).
        const auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)P.A, 0, P.a_bytes, 0x00027000);
        const auto rx = __builtin_amdgcn_make_buffer_rsrc((void*)P.X, 0, P.x_bytes, 0x00027000);
        const int at = lane * 16;
        auto frag_a = [&](uint32_t blk) {
            return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(ra, at, (int)(blk * kFragBytes), 0));
        };
        auto frag_x = [&](uint32_t blk) {
            return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rx, at, (int)(blk * kFragBytes), 0));
        };
        const uint32_t a = (uint32_t)panel * P.steps * 3;
        uint32_t x[kCB];
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb) x[cb] = (uint32_t)min(ct * kCB + cb, P.cblocks - 1) * P.steps;
        // one set of A registers, each refilled for the next step as soon as its products are issued, and
        // two of X: with the sums that is what fits at four wavefronts a SIMD
        bf16x8 fa[3], fx[kCB], nx[kCB];
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb) fx[cb] = frag_x(x[cb] + ks);
#pragma unroll
        for (int q = 2; q >= 0; --q) {   // in the loop's order, so that its waits need not be wider
            __builtin_amdgcn_sched_barrier(0);
            fa[q] = frag_a(a + ks * 3 + q);
        }
#pragma unroll 1
        for (int s = ks; s < P.steps; s += KS) {
            const int next = min(s + KS, P.steps - 1);   // past the last step the loads repeat it
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) nx[cb] = frag_x(x[cb] + next);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 2; q >= 0; --q) {   // the smallest part first
#pragma unroll
                for (int cb = 0; cb < kCB; ++cb)
                    acc[cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[q], fx[cb], acc[cb], 0, 0, 0);
                fa[q] = frag_a(a + next * 3 + q);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) fx[cb] = nx[cb];
        }
    }

    float* mine = stage[wave];
    const float* group = stage[wave - ks];
    // half a tile at a time goes through LDS, so that four workgroups fit on a CU
    auto settle = [&] {
        if constexpr (KS > 1) {
            __syncthreads();
        } else {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
    };
    float* out = P.dW + P.row_ptr[panel * 32];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half > 0) settle();
        // lane l holds column l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4 of each 32 x 32 block
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                mine[(8 * (i / 4) + 4 * (lane >> 5) + (i & 3)) * kCols + cb * 32 + (lane & 31)] = acc[cb][8 * half + i];
        settle();
        auto put = [&](uint32_t w, int32_t e) {
            const int cell = (int)(w & ((1u << kCellBits) - 1)) - half * kStage;
            if (e < p1 && (uint32_t)cell < (uint32_t)kStage) {
                float v = group[cell];
#pragma unroll
                for (int j = 1; j < KS; ++j) v += group[cell + j * kStage];
                out[w >> kCellBits] = v;
            }
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) put(word[k], pos + k * KS * kWave);
        for (int32_t e = pos + kAhead * KS * kWave; e < p1; e += kAhead * KS * kWave) {
            uint32_t more[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) more[k] = P.list[e + k * KS * kWave];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) put(more[k], e + k * KS * kWave);
        }
    }
}

inline int blocks32(int n) { return (n + 31) / 32; }

}  // namespace

// Where the tiles beat the walk over the positions, which gets its dX nearly free beside dW at up to 64
// batch rows (so there only large layers gain).  Measured (us a call, walk : tiles), int8:
//   dW alone     8 rows,  10000 x 10000: 95 % 28.8 : 25.0, 98 % 14.6 : 21.7;  6000 x 1500, 95 %: 9.5 : 7.4
//               64 rows,  10000 x 10000: 95 % 83.7 : 46.0, 98 % 39.4 : 43.6;  2500 x 2500, 98 %: 13.0 : 8.6
//             1024 rows,  2500 x 2500, 98 %: 46.4 : 46.8;  768 x 3072: 98 % 37.7 : 27.9, 99 % 31.8 : 28.3
//   dX and dW   16 rows,  10000 x 10000: 90 % 65.3 : 58.8, 95 % 43.1 : 45.5;  2500 x 2500, 95 %: 14.4 : 15.4
//               64 rows,  10000 x 10000: 95 % 105.9 : 91.3, 98 % 69.3 : 80.7;  2500 x 2500, 95 %: 27.1 : 23.8;
//                         6000 x 1500: 90 % 41.4 : 38.3, 95 % 33.2 : 34.1;  3072 x 768: 90 % 19.9 : 21.8
//              128 rows,  3072 x 768: 90 % 23.6 : 20.1, 98 % 20.4 : 19.3;  2500 x 2500: 90 % 49.4 : 35.8, 98 % 21.0 : 22.4
// What one count of positions and one density cannot tell apart goes the slower way: dW alone at 10000 x 10000, 98 %,
// 32 rows (22.3 : 28.0, tiles taken) and 64 (above); dX and dW at 64 rows, 768 x 3072, 90 % (25.6 : 20.2, walk taken),
// where the transposed shape's walk is faster.
// Operands stay below 4 GB (buffer offsets).
constexpr int64_t kSampleBesideDx = 300000;   // positions at least, at up to 64 rows
bool sample_layer(int64_t M, int64_t K, int64_t nnz) { return nnz > 0 && K <= kSampleMaxK && nnz >= M * K / 64; }
bool sample_applies(const snack_layer* L, const BatchPlan& p, bool want_dx)
{
    if (!L->sample_list) return false;
    const bool dense = L->nnz >= (int64_t)L->M * L->K / 32;
    if (want_dx ? p.bp <= (dense && L->nnz >= kSampleBesideDx ? 16 : 64) : p.bp < (dense ? 8 : 32)) return false;
    const int64_t steps = (p.bp + kStep - 1) / kStep;
    return steps * 3 * blocks32(L->M) < (1ll << 32) / kFragBytes && steps * blocks32(L->K) < (1ll << 32) / kFragBytes;
}

size_t sample_ptr_bytes(const snack_layer* L)
{
    return ((size_t)((L->K + kCols - 1) / kCols) * blocks32(L->M) + 1) * sizeof(int32_t);
}

size_t sample_ws_bytes(const snack_layer* L, const BatchPlan& p, size_t* a_bytes)
{
    if (!sample_applies(L, p, false)) return 0;   // where it applies beside dX, it applies alone
    const size_t step = (size_t)((p.bp + kStep - 1) / kStep) * kFragBytes, a = 3 * step * blocks32(L->M);
    if (a_bytes) *a_bytes = a;
    return a + step * blocks32(L->K);
}

snack_status sample_index(const snack_layer* L, hipStream_t s)
{
    const int tiles = (L->K + kCols - 1) / kCols;
    hipLaunchKernelGGL(sample_list_kernel, dim3((unsigned)blocks32(L->M)), dim3(kListThreads),
                       (size_t)32 * (2 * tiles + 1) * sizeof(int32_t), s, L->row_ptr, L->cols, L->M, tiles,
                       L->sample_list, L->sample_ptr);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

snack_status sample_dw(const snack_layer* L, const void* a, const void* x, int B, float* dW, hipStream_t s)
{
    ProfScope prof(KC_SDDMM_DW, s);
    if (!L->sample_valid) {
        SNACK_CHECK(sample_index(L, s));
        L->sample_valid = !stream_capturing(s);
        L->sample_used = true;
    }
    SampleArgs t;
    t.A = (const uint4*)a;
    t.X = (const uint4*)x;
    t.list = L->sample_list;
    t.tile_ptr = L->sample_ptr;
    t.row_ptr = L->row_ptr;
    t.dW = dW;
    t.steps = (B + kStep - 1) / kStep;
    t.rblocks = blocks32(L->M);
    t.cblocks = blocks32(L->K);
    t.a_bytes = (uint32_t)t.rblocks * t.steps * 3 * kFragBytes;
    t.x_bytes = (uint32_t)t.cblocks * t.steps * kFragBytes;
    t.tiles = (L->K + kCols - 1) / kCols;
    auto go = [&](auto kern, int ks) {
        const int64_t units = ((int64_t)t.rblocks * t.tiles + 4 / ks - 1) / (4 / ks);
        t.per_xcd = (int)((units + kXcd - 1) / kXcd);
        hipLaunchKernelGGL(kern, dim3((unsigned)(t.per_xcd * kXcd)), dim3(256), 0, s, t);
    };
    // Wavefronts a tile: one where the tiles alone give every SIMD more than one, else two or four.  Measured
    // with 1, 2 and 4 (us, 1024 rows, with the operands' launch): 64 tiles (500 x 500) 29.6, 18.8, 13.8;
    // 576 tiles (3072 x 768) 36.6, 31.2, 28.7; 1008 tiles (2000 x 2000) 37.7, 32.5, 34.0;
    // 1580 tiles (2500 x 2500) 47.6, 51.9, 52.6.
    const int64_t all = (int64_t)t.rblocks * t.tiles;
    if (all >= 5 * (int64_t)L->cus) go(sample_kernel<1>, 1);
    else if (all >= 3 * (int64_t)L->cus) go(sample_kernel<2>, 2);
    else go(sample_kernel<4>, 4);
    SNACK_HIP(hipGetLastError());
    return SNACK_OK;
}

}  // namespace snack
