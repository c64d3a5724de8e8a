// Low-rank adapters of many requests beside one shared KS projection
// (ks_adapter_matmul) and their gradients (ks_adapter_backward):
//
//     H[n] = scale[s] X[n] A[s]^T,   Y[n] = act(X[n] K^T + bias + H[n] B[s]^T),   s = ids[n],
//     G[n] = scale[s] dY[n] B[s],    dX[n] = dY[n] K + G[n] A[s],
//     dA[s] = sum_{n: ids[n] = s} G[n]^T X[n],   dB[s] = sum_{n: ids[n] = s} dY[n]^T H[n],
//
// A[s] rank x in_features, B[s] out_features x rank.  A row whose id is negative
// takes no adapter; one whose id is n_adapters or more takes none either and
// raises kDevBadIndex in the device status word.  Every sum is fp32 in an order that
// depends on the sizes, the ids and the alignment alone, and every result is rounded once; in
// bf16, H and G are rounded as well where they are operands of the tensor cores.
//
// Which kernels a forward call takes (the first that fits):
//   few rows               ks_adapter_rows.cu, one launch (or two);
//   bf16, a pattern of the tcgen05 kernel
//                          H as operand planes (shrink_mma_kernel), then the product with
//                          the adapters and the bias as further K steps (ks_tc.cu);
//   fp32, d a multiple of 8, 2^30 flop and more
//                          H (shrink_fp32_kernel), then the product with the adapters as
//                          further stages (ks_fma32.cu);
//   anything else          H, the product (of a tiled kernel, or tile_product_kernel), and a second
//                          pass over it (expand_kernel); in bf16 the product is held in fp32 for
//                          that pass, some rows at a time, so that the result is rounded once.
// A backward call: one launch that lays out what the others read (prepare_kernel),
// one for G and H, the product for dX as above (few rows of a GPT-2-shaped bf16 layer: 41 us
// for all gradients of 32 rows where the tensor-core product takes 64), one for the partial
// sums of dA and dB, one that adds them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "ks_adapter.cuh"
#include "ks_epilogue.cuh"
#include "ks_internal.h"

namespace ks {
namespace {

// ---------------------------------------------------------------- H = scale X W^T
//
// W[s] is rank x F with F contiguous (A, or B transposed).  H[n][r], r < ldh, is
// scale[s] sum_f X[n][f] W[s][r][f], zero for ranks past R and rows without an
// adapter; fp32, or bf16 (rounded once) where it becomes a tensor-core operand:
// its rounding, 2^-9 of each term of the low-rank sum on average, stays below
// the rounding of a bf16 result (error against 64 bits of a prompt, relative: 1.9e-3 to 2.0e-3
// where the rounding of the result alone gives 1.7e-3; gradients 2.3e-3).

// The smallest id above `last` among the warp's (INT_MAX: none left).
__device__ __forceinline__ int next_id(int id, int last) {
    return (int)__reduce_min_sync(0xFFFFFFFFu, (unsigned)(id > last ? id : INT_MAX));
}

// Sums over the lanes of 64 values of a lane: a lane keeps the half of its values that
// its bit picks, so 62 exchanges leave sums 2 lane and 2 lane + 1 in v[0] and v[1].
__device__ __forceinline__ void sum_lanes(float (&v)[64], int lane) {
#pragma unroll
    for (int half = 32; half >= 2; half >>= 1) {
        const int bit = half >> 1;  // lane bits 16, 8, 4, 2, 1
        const bool up = lane & bit;
#pragma unroll
        for (int q = 0; q < half; ++q) {
            const float send = up ? v[q] : v[q + half], keep = up ? v[q + half] : v[q];
            v[q] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, bit);
        }
    }
}

// Any size, type and alignment: a warp takes eight rows and eight ranks, its lanes the
// features, and loads the rows of one adapter in each pass.  12057 x 588 bf16, rank 64:
// 98 us, where a warp for each row, reading all of W[s] for it, took 270.
template <typename T, typename O>
__global__ void __launch_bounds__(128) shrink_any_kernel(const __grid_constant__ ShrinkArgs p) {
    const ShrinkJob &job = p.job[blockIdx.z];
    const T *const X = static_cast<const T *>(job.X), *const W = static_cast<const T *>(job.W);
    O *const H = static_cast<O *>(job.H);
    const int F = job.F, R = p.R, ldh = p.ldh, r0 = blockIdx.y * 8;
    const int lane = threadIdx.x & 31;
    const long long n0 = ((long long)blockIdx.x * 4 + (threadIdx.x >> 5)) * 8;
    if (n0 >= p.N) return;
    const int id = lane < 8 ? row_adapter(p.ids, n0 + lane, p.N, p.S, p.status) : -1;
    const int row = lane >> 2, r = r0 + 2 * (lane & 3);  // whose sums end in this lane (ranks r and r + 1)
    const long long n = n0 + row;
    const int row_id = __shfl_sync(0xFFFFFFFFu, id, row);
    if (row_id < 0 && n < p.N) {
        if (r < ldh) put(H + n * ldh + r, 0.f);
        if (r + 1 < ldh) put(H + n * ldh + r + 1, 0.f);
    }
    for (int s = next_id(id, -1); s != INT_MAX; s = next_id(id, s)) {
        const unsigned take = __ballot_sync(0xFFFFFFFFu, id == s);
        const T *w = W + ((long long)s * R + r0) * F, *x = X + n0 * F;
        const int ranks = min(8, R - r0);  // (none of a padded octet)
        float acc[64];
#pragma unroll
        for (int q = 0; q < 64; ++q) acc[q] = 0.f;
#pragma unroll 2
        for (int f = lane; f < F; f += 32) {
            float xv[8], wv[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) xv[m] = take >> m & 1 ? to_f(x[(long long)m * F + f]) : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) wv[e] = e < ranks ? to_f(w[(long long)e * F + f]) : 0.f;
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[m * 8 + e] = fmaf(xv[m], wv[e], acc[m * 8 + e]);
        }
        sum_lanes(acc, lane);
        const float sc = p.scales ? p.scales[s] : 1.f;
        if (row_id == s) {
            if (r < ldh) put(H + n * ldh + r, r < R ? sc * acc[0] : 0.f);
            if (r + 1 < ldh) put(H + n * ldh + r + 1, r + 1 < R ? sc * acc[1] : 0.f);
        }
    }
}

// The adapters among each 128 rows and their rows, for the products that take them
// as further stages (TcAdapters::lists): one warp per 128 rows.
__device__ void tile_list(const int *__restrict__ ids, int *__restrict__ lists, int list_stride, long long N, int S,
                          long long tile, int lane) {
    int id[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const long long n = tile * 128 + 32 * q + lane;
        id[q] = n < N ? (ids ? ids[n] : 0) : -1;
        if (id[q] >= S) id[q] = -1;
    }
    int *list = lists + tile * list_stride;
    int count = 0, last = -1;
    while (true) {
        int best = INT_MAX;
#pragma unroll
        for (int q = 0; q < 4; ++q) best = id[q] > last ? min(best, id[q]) : best;
        last = (int)__reduce_min_sync(0xFFFFFFFFu, (unsigned)best);
        if (last == INT_MAX) break;
        unsigned off[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) off[q] = ~__ballot_sync(0xFFFFFFFFu, id[q] == last);
        if (lane == 0) {
            int *e = list + 8 + 8 * count;
            e[0] = last;
            if (count == 0) list[1] = last;
            *reinterpret_cast<uint4 *>(e + 4) = make_uint4(off[0], off[1], off[2], off[3]);
        }
        ++count;
    }
    if (lane == 0) list[0] = count;
}

// fp32, F a multiple of 4 and 16-byte aligned: a warp takes eight rows and eight
// ranks, its lanes the features (four each), and adds the lanes up at the end.  An
// adapter's pass runs over all eight rows and keeps those that take it.  X runs
// two steps ahead in shared memory (cp.async; a lane copies what it reads itself, so
// nothing is synchronised): at 160 registers the loads of 12 warps an SM alone did
// not cover X's latency.  25216 x 384, rank 8: 15 us; with 25216 x 1536 beside it 40 us,
// 4.8 TB/s.  SPLIT warps share eight rows where there are few: their features are
// dealt in turn and their sums meet in shared memory.
// Blocks past the rows' build the lists of the product that follows.
template <int SPLIT>
__global__ void __launch_bounds__(128)
    shrink_fp32_kernel(const __grid_constant__ ShrinkArgs p, int row_blocks, int *__restrict__ lists, int list_stride) {
    constexpr int STAGES = 3, STEP = 128 * SPLIT;
    __shared__ float4 xs[4][STAGES][8][32];
    const ShrinkJob &job = p.job[blockIdx.z];
    const float *__restrict__ const X = static_cast<const float *>(job.X);
    const float *__restrict__ const W = static_cast<const float *>(job.W);
    float *__restrict__ const H = static_cast<float *>(job.H);
    const float *const scales = p.scales;
    const long long N = p.N;
    const int F = job.F, R = p.R, ldh = p.ldh, r0 = blockIdx.y * 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % SPLIT;
    if ((int)blockIdx.x >= row_blocks) {
        const long long tile = (long long)(blockIdx.x - row_blocks) * 4 + warp;
        if (blockIdx.y == 0 && blockIdx.z == 0 && tile * 128 < N)
            tile_list(p.ids, lists, list_stride, N, p.S, tile, lane);
        return;
    }
    const long long n0 = ((long long)blockIdx.x * (4 / SPLIT) + warp / SPLIT) * 8;
    if (n0 >= N) return;
    const int id = lane < 8 ? row_adapter(p.ids, n0 + lane, N, p.S, p.status) : -1;
    const int row = lane >> 2, r = r0 + 2 * (lane & 3);  // whose sums end in this lane (ranks r and r + 1)
    const long long n = n0 + row;
    const int row_id = __shfl_sync(0xFFFFFFFFu, id, row);
    if (row_id < 0 && n < N && part == 0) {
        if (r < ldh) H[n * ldh + r] = 0.f;
        if (r + 1 < ldh) H[n * ldh + r + 1] = 0.f;
    }
    int found = 0;
    for (int s = next_id(id, -1); s != INT_MAX; s = next_id(id, s)) ++found;
    if (found > 2) {  // each pass computes all eight rows: more than two cost more than row by row
        for (int m = part; m < 8; m += SPLIT) {
            const int s = __shfl_sync(0xFFFFFFFFu, id, m);
            if (s < 0) continue;
            for (int q = r0; q < r0 + 8; q += 4) {
                float h[4] = {0.f, 0.f, 0.f, 0.f};
                if (q < R) dot4(X + (n0 + m) * F, W + ((long long)s * R + q) * F, F, R - q, lane, h);
                const float v = lane == 0 ? h[0] : lane == 1 ? h[1] : lane == 2 ? h[2] : h[3];
                if (lane < 4 && q + lane < ldh)
                    H[(n0 + m) * ldh + q + lane] = q + lane < R ? (scales ? scales[s] : 1.f) * v : 0.f;
            }
        }
        return;
    }
    const auto issue = [&](int f, int stage) {  // (rows past the last are read as the last one)
        if (f < F) {
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const float *src = X + (n0 + m < N ? n0 + m : N - 1) * F + f;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 (unsigned)__cvta_generic_to_shared(&xs[warp][stage][m][lane])),
                             "l"(src)
                             : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int s = next_id(id, -1); s != INT_MAX; s = next_id(id, s)) {
        const float sc = scales ? scales[s] : 1.f;
        const float *w = W + ((long long)s * R + (r0 < R ? r0 : 0)) * F;
        float acc[64];
#pragma unroll
        for (int q = 0; q < 64; ++q) acc[q] = 0.f;
        const int f0 = part * 128 + lane * 4;
        issue(f0, 0);
        issue(f0 + STEP, 1);
        int stage = 0;
        for (int f = f0; f - lane * 4 < F; f += STEP) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            float4 x[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) x[m] = xs[warp][stage][m][lane];
            issue(f + 2 * STEP, stage == 0 ? 2 : stage - 1);
            stage = stage == 2 ? 0 : stage + 1;
            if (f >= F) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int rr = r0 + e < R ? e : 0;
                const float4 v = __ldg(reinterpret_cast<const float4 *>(w + (long long)rr * F + f));
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    float a = acc[m * 8 + e];
                    a = fmaf(x[m].x, v.x, a);
                    a = fmaf(x[m].y, v.y, a);
                    a = fmaf(x[m].z, v.z, a);
                    acc[m * 8 + e] = fmaf(x[m].w, v.w, a);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        sum_lanes(acc, lane);
        if constexpr (SPLIT > 1) {
            // (the warp's stages are free by now)
            if (part) xs[warp][0][0][lane] = make_float4(acc[0], acc[1], 0.f, 0.f);
            __syncthreads();
            if (!part) {
#pragma unroll
                for (int q = 1; q < SPLIT; ++q) acc[0] += xs[warp + q][0][0][lane].x, acc[1] += xs[warp + q][0][0][lane].y;
            }
            __syncthreads();
        }
        if (row_id == s && part == 0) {
            if (r < ldh) H[n * ldh + r] = r < R ? sc * acc[0] : 0.f;
            if (r + 1 < ldh) H[n * ldh + r + 1] = r + 1 < R ? sc * acc[1] : 0.f;
        }
    }
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8) of bf16 fragments in registers.
__device__ __forceinline__ void mma16816(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                         unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The bias as the tensor-core product takes it (TcAdapters): a thread for each
// output, and the plane of ones by the first block.
struct BiasPack {
    const unsigned short *bias;
    uint4 *packed, *ones;
    int n, blocks;
};
__device__ __forceinline__ void pack_bias(const BiasPack &b, int block) {
    const int at = block * 256 + (int)threadIdx.x;
    if (at < b.n) b.packed[at] = make_uint4(b.bias[at], 0u, 0u, 0u);
    // 16-byte lines (rank octet, row group, rank): rank 0 is ones, eight rows of 1.0 in bf16
    if (block == 0) {
        const unsigned one = threadIdx.x < 128 && threadIdx.x % 8 == 0 ? 0x3F803F80u : 0u;
        b.ones[threadIdx.x] = make_uint4(one, one, one, one);
    }
}

// bf16, F a multiple of 8 and 16-byte aligned, on the tensor cores (mma.sync: the
// operands of so narrow a product are read once each, straight into registers,
// and a tcgen05 tile would first have to pass through shared memory).  A block
// takes 16 MT rows and NT * 8 ranks, its eight warps every eighth 32 features.  Both
// operands have the features contiguous, and a sum does not care which of them an
// MMA calls its k: lane (g, t) loads the eight features 8 t .. 8 t + 7 of rows g
// (X, and W) as one 16-byte vector, which is its share of two MMA steps.  The
// warps' sums meet in shared memory in a fixed order.  Bound by the latency of X
// and by W, which each block reads again from L2: rank 16, 8192 x 1024: 6 us; G and H
// of 8192 rows (4096 and 1024 wide) 22 us, 3.8 TB/s; rank 64, 8192 x 4096: 48 us.  Blocks past the rows'
// build the lists of the tensor-core product that follows, whose operand planes
// (TcAdapters::planes) take H instead of, or beside, the rows of H.
__device__ __forceinline__ unsigned short *plane_at(unsigned short *planes, long long n, int r, int plane_r) {
    return planes + n / 128 * (plane_r * 128) + (r >> 3) * 1024 + (int)(n % 128 >> 3) * 64 + (r & 7) * 8 + (int)(n & 7);
}

// Blocks of rows with more adapters than this go row by row: a pass takes about
// as long as six rows' dot products.
constexpr int kMixed = 6;

template <int MT, int NT, typename O>
__global__ void __launch_bounds__(256)
    shrink_mma_kernel(const __grid_constant__ ShrinkArgs p, int row_blocks, int *__restrict__ lists, int list_stride,
                      const __grid_constant__ BiasPack bias) {
    const ShrinkJob &job = p.job[blockIdx.z];
    const __nv_bfloat16 *__restrict__ const X = static_cast<const __nv_bfloat16 *>(job.X);
    const __nv_bfloat16 *__restrict__ const W = static_cast<const __nv_bfloat16 *>(job.W);
    O *__restrict__ const H = static_cast<O *>(job.H);
    unsigned short *__restrict__ const planes = job.planes;
    const float *const scales = p.scales;
    const long long N = p.N;
    const int F = job.F, R = p.R, ldh = p.ldh, plane_r = p.plane_r;
    constexpr int ROWS = 16 * MT, RC = 8 * NT, LD = RC + 1;
    __shared__ float red[4][ROWS][LD];
    __shared__ int row_id[ROWS], found[ROWS], n_found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= row_blocks) {
        if (bias.packed && (int)blockIdx.x - row_blocks < bias.blocks) {
            pack_bias(bias, (int)blockIdx.x - row_blocks);
            return;
        }
        const long long tile = (long long)(blockIdx.x - row_blocks - bias.blocks) * 8 + warp;
        if (blockIdx.y == 0 && blockIdx.z == 0 && tile * 128 < N)
            tile_list(p.ids, lists, list_stride, N, p.S, tile, lane);
        return;
    }
    const long long n0 = (long long)blockIdx.x * ROWS;
    const int r0 = blockIdx.y * RC;
    if (warp == 0) {
        const int id = lane < ROWS ? row_adapter(p.ids, n0 + lane, N, p.S, p.status) : -1;
        if (lane < ROWS) row_id[lane] = id;
        int count = 0;
        for (int s = next_id(id, -1); s != INT_MAX; s = next_id(id, s)) {
            if (lane == 0) found[count] = s;
            ++count;
        }
        if (lane == 0) n_found = count;
    }
    __syncthreads();
    const int g = lane >> 2, t = lane & 3;
    for (int q = threadIdx.x; q < ROWS * RC; q += 256) {
        const int m = q / RC, r = r0 + q % RC;
        if (H && row_id[m] < 0 && n0 + m < N && r < ldh) put(H + (n0 + m) * ldh + r, 0.f);
    }
    const int n_s = n_found;
    if (n_s > kMixed) {  // too many passes: row by row
        for (int q = warp; q < ROWS * RC / 4; q += 8) {
            const int m = q / (RC / 4), r = r0 + q % (RC / 4) * 4, s = row_id[m];
            if (s < 0) continue;
            float h[4] = {0.f, 0.f, 0.f, 0.f};
            if (r < R) dot4(X + (n0 + m) * F, W + ((long long)s * R + r) * F, F, R - r, lane, h);
            if (lane < 4) {
                const float v = (lane == 0 ? h[0] : lane == 1 ? h[1] : lane == 2 ? h[2] : h[3]);
                const float hv = r + lane < R ? (scales ? scales[s] : 1.f) * v : 0.f;
                if (H && r + lane < ldh) put(H + (n0 + m) * ldh + r + lane, hv);
                if (planes && r + lane < plane_r)
                    *plane_at(planes, n0 + m, r + lane, plane_r) = __bfloat16_as_ushort(__float2bfloat16_rn(hv));
            }
        }
        return;
    }
    const uint4 *x[2 * MT];
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m) {  // rows past the last are read as the last one
        const long long n = n0 + 8 * m + g < N ? n0 + 8 * m + g : N - 1;
        x[m] = reinterpret_cast<const uint4 *>(X + n * F);
    }
    for (int k = 0; k < n_s; ++k) {
        const int s = found[k];
        const uint4 *w[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {  // ranks past R are read as the last one
            const int r = min(r0 + 8 * j + g, R - 1);
            w[j] = reinterpret_cast<const uint4 *>(W + ((long long)s * R + r) * F);
        }
        float acc[MT][NT][4] = {};
        // U steps' loads in flight together
        constexpr int U = NT <= 2 ? 4 : 1;
        for (int f0 = warp * 32 + 8 * t; f0 - 8 * t < F; f0 += 256 * U) {
            uint4 xv[U][2 * MT], wv[U][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int f = f0 + 256 * u;
                const bool in = f < F;
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m) xv[u][m] = in ? __ldg(x[m] + (f >> 3)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int j = 0; j < NT; ++j) wv[u][j] = in ? __ldg(w[j] + (f >> 3)) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 &p0 = xv[u][2 * m], &p1 = xv[u][2 * m + 1], &v = wv[u][j];
                        mma16816(acc[m][j], p0.x, p1.x, p0.y, p1.y, v.x, v.y);
                        mma16816(acc[m][j], p0.z, p1.z, p0.w, p1.w, v.z, v.w);
                    }
        }
        // warps 4..7 hand their sums to warps 0..3, which add theirs
        if (warp >= 4) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        red[warp - 4][16 * m + g + 8 * (e >> 1)][8 * j + 2 * t + (e & 1)] = acc[m][j][e];
        }
        __syncthreads();
        if (warp < 4) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        red[warp][16 * m + g + 8 * (e >> 1)][8 * j + 2 * t + (e & 1)] += acc[m][j][e];
        }
        __syncthreads();
        const float sc = scales ? scales[s] : 1.f;
        for (int q = threadIdx.x; q < ROWS * RC; q += 256) {
            const int m = q / RC, c = q % RC, r = r0 + c;
            if (row_id[m] == s) {
                const float h = r < R ? sc * ((red[0][m][c] + red[1][m][c]) + (red[2][m][c] + red[3][m][c])) : 0.f;
                if (H && r < ldh) put(H + (n0 + m) * ldh + r, h);
                if (planes && r < plane_r)
                    *plane_at(planes, n0 + m, r, plane_r) = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- Y = act(P + bias + H W)

constexpr int kExpandRows = 8;

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
}

// F a multiple of 4 and vectors of four aligned (25216 x 384 fp32, rank 8: 17 us, 4.5
// TB/s; 16 rows a thread took 23): a thread owns four outputs of eight
// rows and passes once over the weights of each adapter among them, four ranks at
// a time; H is read from shared memory (the same address in a warp), P before the
// products, so that its latency is theirs.  P is the KS product in fp32: Y itself, or in
// bf16 a workspace.
// RC: the ranks are contiguous in W (B) and come in whole fours; otherwise the
// features are (A).
template <typename T, bool RC, int ACT>
__global__ void __launch_bounds__(128, 6)
    expand_kernel(T *Y, const float *P, const T *__restrict__ W, const int *__restrict__ ids,
                  const float *__restrict__ H, long long N, int F, int R, int ldh, int S,
                  const T *__restrict__ bias) {
    constexpr int ROWS = kExpandRows;
    extern __shared__ float4 hs[];  // [rank / 4][row]
    __shared__ int row_id[ROWS];
    const long long n0 = (long long)blockIdx.x * ROWS;
    const int rows = (int)min((long long)ROWS, N - n0);
    if (threadIdx.x < ROWS) {
        const int s = (int)threadIdx.x < rows ? (ids ? ids[n0 + threadIdx.x] : 0) : -1;
        row_id[threadIdx.x] = s < S ? s : -1;
    }
    const int rq = ldh / 4;
    for (int q = threadIdx.x; q < rows * rq; q += 128)
        hs[(q % rq) * ROWS + q / rq] = *reinterpret_cast<const float4 *>(H + n0 * ldh + (long long)q * 4);
    __syncthreads();
    const int f = (blockIdx.y * 128 + threadIdx.x) * 4;
    const bool in = f < F;
    T *y = Y + n0 * F + f;
    const float *product = P + n0 * F + f;
    float4 acc[ROWS];
    {
        const float4 b = bias && in ? load4(bias + f) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
            acc[m] = b;
            if (in && m < rows) {
                const float4 v = load4(product + (long long)m * F);
                acc[m] = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
            }
        }
    }
    const int lane = threadIdx.x & 31;
    const int id = lane < ROWS ? row_id[lane] : -1;
    for (int s = next_id(id, -1); s != INT_MAX; s = next_id(id, s)) {
        const unsigned take = __ballot_sync(0xFFFFFFFFu, id == s);
        if (!in) continue;
        const T *w = W + (long long)s * R * F;
        for (int r = 0; r < R; r += 4) {
            // v[c]: ranks r .. r + 3 of output f + c
            float4 v[4];
            if constexpr (RC) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = load4(w + (long long)(f + c) * R + r);
            } else {
                float4 u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    u[e] = r + e < R ? load4(w + (long long)(r + e) * F + f) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[0] = make_float4(u[0].x, u[1].x, u[2].x, u[3].x);
                v[1] = make_float4(u[0].y, u[1].y, u[2].y, u[3].y);
                v[2] = make_float4(u[0].z, u[1].z, u[2].z, u[3].z);
                v[3] = make_float4(u[0].w, u[1].w, u[2].w, u[3].w);
            }
            const float4 *h = hs + (r >> 2) * ROWS;
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                if (take >> m & 1) {
                    const float4 x = h[m];
                    float4 a = acc[m];
                    a.x = fmaf(x.w, v[0].w, fmaf(x.z, v[0].z, fmaf(x.y, v[0].y, fmaf(x.x, v[0].x, a.x))));
                    a.y = fmaf(x.w, v[1].w, fmaf(x.z, v[1].z, fmaf(x.y, v[1].y, fmaf(x.x, v[1].x, a.y))));
                    a.z = fmaf(x.w, v[2].w, fmaf(x.z, v[2].z, fmaf(x.y, v[2].y, fmaf(x.x, v[2].x, a.z))));
                    a.w = fmaf(x.w, v[3].w, fmaf(x.z, v[3].z, fmaf(x.y, v[3].y, fmaf(x.x, v[3].x, a.w))));
                    acc[m] = a;
                }
            }
        }
    }
    if (!in) return;
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
        if (m < rows) {
            float4 v = acc[m];
            if constexpr (ACT == KS_ACT_GELU_ERF) {
                const float2 a = gelu_erf_f2(make_float2(v.x, v.y)), b = gelu_erf_f2(make_float2(v.z, v.w));
                v = make_float4(a.x, a.y, b.x, b.y);
            } else if constexpr (ACT != KS_ACT_NONE) {
                v.x = ep_act_fn(v.x, ACT);
                v.y = ep_act_fn(v.y, ACT);
                v.z = ep_act_fn(v.z, ACT);
                v.w = ep_act_fn(v.w, ACT);
            }
            store4(y + (long long)m * F, v);
        }
    }
}

// The same for any size and alignment: a thread's four outputs are as far apart as the
// block is wide.  RV: the ranks come in whole aligned fours (3535 x 570 fp32, rank 64: 34 us,
// where a thread for each output took 346).
template <typename T, bool RC, bool RV>
__global__ void __launch_bounds__(128)
    expand_any_kernel(T *Y, const float *P, const T *__restrict__ W, const int *__restrict__ ids,
                      const float *__restrict__ H, long long N, int F, int R, int ldh, int S,
                      const T *__restrict__ bias, int act) {
    constexpr int ROWS = kExpandRows;
    extern __shared__ float4 hs[];  // [rank / 4][row]
    const int threads = blockDim.x;
    const unsigned col_blocks = (unsigned)((F + 4LL * threads - 1) / (4 * threads));
    const long long n0 = (long long)(blockIdx.x / col_blocks) * ROWS, f0 = (long long)(blockIdx.x % col_blocks) * (4 * threads);
    const int rows = (int)min((long long)ROWS, N - n0), lane = threadIdx.x & 31;
    int id = lane < rows ? (ids ? ids[n0 + lane] : 0) : -1;
    if (id >= S) id = -1;
    const int rq = ldh / 4;
    for (int q = threadIdx.x; q < rows * rq; q += threads)
        hs[(q % rq) * ROWS + q / rq] = *reinterpret_cast<const float4 *>(H + n0 * ldh + (long long)q * 4);
    __syncthreads();
    int f[4];
    bool in[4];
    float acc[ROWS][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const long long at = f0 + c * threads + threadIdx.x;
        in[c] = at < F;
        f[c] = in[c] ? (int)at : 0;
#pragma unroll
        for (int m = 0; m < ROWS; ++m) acc[m][c] = in[c] && m < rows ? P[(n0 + m) * F + f[c]] : 0.f;
    }
    for (int s = next_id(id, -1); s != INT_MAX; s = next_id(id, s)) {
        const unsigned take = __ballot_sync(0xFFFFFFFFu, id == s);
        const T *w = W + (long long)s * R * F;
        for (int r = 0; r < R; r += 4) {
            float v[4][4];  // ranks r .. r + 3 of output f[c]
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (RV) {
                    const float4 u = load4(w + (long long)f[c] * R + r);
                    v[c][0] = u.x, v[c][1] = u.y, v[c][2] = u.z, v[c][3] = u.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[c][e] = r + e < R ? to_f(RC ? w[(long long)f[c] * R + r + e] : w[(long long)(r + e) * F + f[c]])
                                            : 0.f;
                }
            }
            const float4 *h = hs + (r >> 2) * ROWS;
#pragma unroll
            for (int m = 0; m < ROWS; ++m)
                if (take >> m & 1) {
                    const float4 x = h[m];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[m][c] = fmaf(x.w, v[c][3],
                                         fmaf(x.z, v[c][2], fmaf(x.y, v[c][1], fmaf(x.x, v[c][0], acc[m][c]))));
                }
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
            if (in[c] && m < rows) put(Y + (n0 + m) * F + f[c], ep_apply(acc[m][c], bias, f[c], act));
}

// ---------------------------------------------------------------- Y = X K^T of odd and small layers

// For patterns that no tiled kernel of the library takes (its streaming kernels read X
// again for every output), and few rows in fp32: the blocks (i, l) one by one as 64 x 64
// tiles of rows and outputs, 16 products deep, through shared memory; a thread holds 4 x 4
// sums.  X and Y have stride d here; the blocks of all l run side by side, so that the
// lines they share are read from L2.  Bound by shared memory's reads, eight bytes for
// each four FMAs, and by the scattered loads.  10577 rows of (5, 117, 108, 3) in fp32: 204 us, 20
// TFLOP/s (streaming: 3000 us); 675 rows of (1, 104, 171, 4) in bf16: 17 us (76).
constexpr int kProductTile = 64, kProductDepth = 16;
template <typename T>
__global__ void __launch_bounds__(256)
    tile_product_kernel(const T *__restrict__ X, const T *__restrict__ V, float *__restrict__ Y, long long N, int a,
                       int b, int c, int d) {
    constexpr int TILE = kProductTile, DEPTH = kProductDepth, LD = TILE + 4;
    __shared__ __align__(16) float xs[DEPTH][LD], vs[DEPTH][LD];
    const int k_tiles = (b + TILE - 1) / TILE;
    const int l = blockIdx.x % d, k0 = blockIdx.x / d % k_tiles * TILE, i = blockIdx.x / d / k_tiles;
    const long long n0 = (long long)blockIdx.y * TILE;
    const long long in_f = (long long)a * c * d, out_f = (long long)a * b * d;
    const int j = threadIdx.x % DEPTH, m = threadIdx.x / DEPTH;  // loads: rows (outputs) m, m + 16, ..
    const T *const x = X + n0 * in_f + (long long)i * c * d + l;
    const T *const v = V + ((long long)(i * (long long)d + l) * b + k0) * c;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;  // outputs 4 tx .., rows 4 ty ..
    float acc[4][4] = {};
    float xr[4], vr[4];
    const auto load = [&](int j0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int at = m + 16 * q;
            xr[q] = j0 + j < c && n0 + at < N ? to_f(x[at * in_f + (long long)(j0 + j) * d]) : 0.f;
            vr[q] = j0 + j < c && k0 + at < b ? to_f(v[(long long)at * c + j0 + j]) : 0.f;
        }
    };
    load(0);
    for (int j0 = 0; j0 < c; j0 += DEPTH) {
#pragma unroll
        for (int q = 0; q < 4; ++q) xs[j][m + 16 * q] = xr[q], vs[j][m + 16 * q] = vr[q];
        __syncthreads();
        load(j0 + DEPTH);  // (in flight during the products)
#pragma unroll
        for (int e = 0; e < DEPTH; ++e) {
            const float4 p = load4(&xs[e][4 * ty]), w = load4(&vs[e][4 * tx]);
            const float pa[4] = {p.x, p.y, p.z, p.w}, wa[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[r][k] = fmaf(pa[r], wa[k], acc[r][k]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + 4 * ty + r < N && k0 + 4 * tx + k < b)
                Y[(n0 + 4 * ty + r) * out_f + ((long long)i * b + k0 + 4 * tx + k) * d + l] = acc[r][k];
}

// ---------------------------------------------------------------- dA and dB

constexpr int kPrepareThreads = 256;

// The rows of each adapter in order: perm[offsets[s] .. offsets[s + 1]) holds the
// rows with id s.  The block counts the rows of smaller ids, then writes the rows of
// its own, 4096 ids at a time, 16 neighbouring ones a thread: the loads of a step are in
// flight together, and their latency is what this costs.
__device__ void order_rows(const int *__restrict__ ids, int *__restrict__ perm, int *__restrict__ offsets, int N, int S,
                           int s) {
    constexpr int WARPS = kPrepareThreads / 32, EACH = 16, STEP = EACH * kPrepareThreads;
    __shared__ int warp_n[2][WARPS];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int less = 0;
    for (int n0 = 0; n0 < N; n0 += STEP) {
        int id[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int n = n0 + e * kPrepareThreads + t;
            id[e] = n < N ? ids[n] : -1;
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e) less += id[e] >= 0 && id[e] < s;
    }
    less = __reduce_add_sync(0xFFFFFFFFu, less);
    if (lane == 0) warp_n[0][warp] = less;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) base += warp_n[0][w];
    if (t == 0) offsets[s] = base;
    int buf = 1;
    for (int n0 = 0; n0 < N; n0 += STEP, buf ^= 1) {
        const int first = n0 + EACH * t;
        unsigned mine = 0;
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            if (first + e < N && ids[first + e] == s) mine |= 1u << e;
        const int c = __popc(mine);
        int sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += u;
        }
        if (lane == 31) warp_n[buf][warp] = sum;
        __syncthreads();  // (the next step writes the other buffer, the one after that is past a barrier)
        int at = base + sum - c;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const int u = warp_n[buf][w];
            if (w < warp) at += u;
            base += u;
        }
        for (; mine; mine &= mine - 1) perm[at++] = first + __ffs(mine) - 1;
    }
    if (s == S - 1 && t == 0) offsets[S] = base;
}

// What a backward pass has to lay out first, in one launch:
// transposed copies out[q][c][r] = in[q][r][c] of `blocks` blocks of rows x cols (32 x
// 32 tiles; out's rows are ld long, zeros past `rows`), and the rows of each adapter.
struct Transpose {
    const void *in;
    void *out;
    long long blocks;
    int rows, cols, ld, tr, tc;  // tr, tc: tiles along ld and cols
    long long tiles;
};
struct PrepareArgs {
    Transpose job[3];
    const int *ids;
    int *perm, *offsets;
    int N, S;
    int sorted;  // blocks that order rows (S or 0), before the tiles
};
template <typename T>
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(const __grid_constant__ PrepareArgs p) {
    if ((int)blockIdx.x < p.sorted) {
        order_rows(p.ids, p.perm, p.offsets, p.N, p.S, (int)blockIdx.x);
        return;
    }
    __shared__ T tile[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const long long step = gridDim.x - p.sorted;
    long long at = blockIdx.x - p.sorted;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const Transpose &q = p.job[j];
        for (; at < q.tiles; at += step) {
            const unsigned per = (unsigned)(q.tr * q.tc);
            const long long blk = q.tiles >> 32 ? at / per : (unsigned)at / per;
            const int rest = (int)(at - blk * per), r0 = rest / q.tc * 32, c0 = rest % q.tc * 32;
            const T *in = static_cast<const T *>(q.in) + blk * q.rows * q.cols;
#pragma unroll
            for (int e = 0; e < 32; e += kPrepareThreads / 32) {
                T v{};
                if (r0 + y + e < q.rows && c0 + x < q.cols) v = in[(long long)(r0 + y + e) * q.cols + c0 + x];
                tile[y + e][x] = v;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 32; e += kPrepareThreads / 32)
                if (c0 + y + e < q.cols && r0 + x < q.ld)
                    static_cast<T *>(q.out)[(blk * q.cols + c0 + y + e) * q.ld + r0 + x] = tile[x][y + e];
            __syncthreads();
        }
        at -= q.tiles;
    }
}

// A gradient is out[s][f][r] = sum over the rows n of adapter s of P[n][f] Q[n][r]
// (dA: P = X, Q = G; dB: P = dY, Q = H).  The rows in the adapters' order are cut
// into chunks of `chunk` positions; a block takes some features of one chunk and
// writes, for each adapter s with rows in chunk z, a partial sum to slot z + s.
// (A step from one piece (z, s) to the next raises z or s, so z + s is a piece's
// own, and chunks + S slots are enough, however the rows spread.)  reduce_kernel
// adds an adapter's slots in order.

// The first adapter whose rows end after position p.
__device__ __forceinline__ int adapter_at(const int *offsets, int S, int p) {
    int a = 0, b = S;  // offsets[a] <= p < offsets[b] where such exist
    while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (offsets[mid] <= p)
            a = mid;
        else
            b = mid;
    }
    return a;
}

// One or two gradients (dA, dB) of a launch: the features of both, one after the
// other, are dealt to blockIdx.x.
struct GradJob {
    const void *P, *V;  // V: batch x ldh
    float *W;           // partial sums: (chunks + S) x R x F
    void *out;          // entry (r, f) of out[s] at r * rs + f * fs
    int F, rs, fs;
};
struct GradArgs {
    GradJob job[2];
    const int *perm, *offsets;
    int N, R, ldh, S, chunk;
    int first;  // blocks of job[0]
};

// fp32: a warp takes 128 features (four a lane) and every fourth row of the chunk,
// RC ranks of each; Q's row is the same address in a warp.  64 FMAs (RC = 16) for
// each 16 bytes of P a lane loads.  Bound by P's latency: what costs warps an SM (rows
// of P a step ahead in registers, Q's rows in shared memory and eight rows in
// flight: 106 and 98 us where this takes 59, 25216 x (1536 + 384) rank 8) loses more than it hides.  Types and alignment: any (VEC: vectors of four).
template <typename T, int RC, bool VEC>
__global__ void __launch_bounds__(128) grad_kernel(const __grid_constant__ GradArgs a) {
    const GradJob &job = a.job[(int)blockIdx.x >= a.first];
    const int bx = (int)blockIdx.x >= a.first ? (int)blockIdx.x - a.first : (int)blockIdx.x;
    const T *__restrict__ const P = static_cast<const T *>(job.P);
    const float *__restrict__ const V = static_cast<const float *>(job.V);
    const int *__restrict__ const perm = a.perm, *__restrict__ const offsets = a.offsets;
    float *__restrict__ const W = job.W;
    const int N = a.N, F = job.F, R = a.R, ldh = a.ldh, S = a.S, chunk = a.chunk;
    __shared__ float4 red[3][RC][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int f = (bx * 32 + lane) * 4, r0 = blockIdx.z * RC;
    const int total = offsets ? offsets[S] : N;
    const int begin = blockIdx.y * chunk, end = min(begin + chunk, total);
    if (begin >= end) return;
    int s = offsets ? adapter_at(offsets, S, begin) : 0;
    for (int lo = begin; lo < end; ++s) {
        const int hi = offsets ? min(end, offsets[s + 1]) : end;
        if (hi <= lo) continue;
        float4 acc[RC];
#pragma unroll
        for (int r = 0; r < RC; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = lo + warp; k < hi; k += 4) {
            const long long n = perm ? perm[k] : k;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            const T *p = P + n * F + f;
            if constexpr (VEC) {
                if (f < F) x = load4(p);
            } else {
                if (f < F) x.x = to_f(p[0]);
                if (f + 1 < F) x.y = to_f(p[1]);
                if (f + 2 < F) x.z = to_f(p[2]);
                if (f + 3 < F) x.w = to_f(p[3]);
            }
            const float *v = V + n * ldh + r0;
#pragma unroll
            for (int r = 0; r < RC; r += 4) {
                if (r0 + r >= ldh) break;
                const float4 q = load4(v + r);
                const float qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[r + e].x = fmaf(x.x, qq[e], acc[r + e].x);
                    acc[r + e].y = fmaf(x.y, qq[e], acc[r + e].y);
                    acc[r + e].z = fmaf(x.z, qq[e], acc[r + e].z);
                    acc[r + e].w = fmaf(x.w, qq[e], acc[r + e].w);
                }
            }
        }
        if (warp) {
#pragma unroll
            for (int r = 0; r < RC; ++r) red[warp - 1][r][lane] = acc[r];
        }
        __syncthreads();
        if (!warp) {
            float *w = W + (long long)(blockIdx.y + s) * R * F;
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                if (r0 + r >= R) break;
                float4 v = acc[r];
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const float4 b = red[q][r][lane];
                    v.x += b.x, v.y += b.y, v.z += b.z, v.w += b.w;
                }
                float *d = w + (long long)(r0 + r) * F + f;
                if (f + 3 < F && F % 4 == 0) {
                    store4(d, v);
                } else {
                    if (f < F) d[0] = v.x;
                    if (f + 1 < F) d[1] = v.y;
                    if (f + 2 < F) d[2] = v.z;
                    if (f + 3 < F) d[3] = v.w;
                }
            }
        }
        __syncthreads();
        lo = hi;
    }
}

__device__ __forceinline__ uint4 load8_bf16(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ uint4 load8_bf16(const float *p) {
    const float4 a = load4(p), b = load4(p + 4);
    uint4 v;
    const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w),
                                 __floats2bfloat162_rn(b.x, b.y), __floats2bfloat162_rn(b.z, b.w)};
    v.x = *reinterpret_cast<const unsigned *>(&h[0]), v.y = *reinterpret_cast<const unsigned *>(&h[1]);
    v.z = *reinterpret_cast<const unsigned *>(&h[2]), v.w = *reinterpret_cast<const unsigned *>(&h[3]);
    return v;
}

// bf16, F a multiple of 8 and 16-byte aligned: out^T = Q^T P on the tensor cores, m
// the ranks (MT * 16 of them), n the features, k the rows.  A warp takes 64
// features: lane (g, t) loads features 8 g .. 8 g + 7 of rows 4 t .. 4 t + 3 as four
// 16-byte vectors, and pairs rows with byte permutes, which gives its share of
// eight MMAs whose columns are features 8 g + j, j = 0 .. 7 (the order of the rows
// within a sum and of the features across columns is free).  P goes straight
// to registers, four whole 128-byte lines for each warp load; Q, R/512 of P's bytes
// or so, is staged transposed in shared memory, 128 positions at a time.  Bound by
// the latency of P (8192 x (1024 + 4096), rank 16: 25 us, 3.3 TB/s).  Q is rounded to
// bf16 where it is fp32.
template <int MT, typename Q>
__global__ void __launch_bounds__(256) grad_mma_kernel(const __grid_constant__ GradArgs a) {
    const GradJob &job = a.job[(int)blockIdx.x >= a.first];
    const int bx = (int)blockIdx.x >= a.first ? (int)blockIdx.x - a.first : (int)blockIdx.x;
    const __nv_bfloat16 *__restrict__ const P = static_cast<const __nv_bfloat16 *>(job.P);
    const Q *__restrict__ const V = static_cast<const Q *>(job.V);
    const int *__restrict__ const perm = a.perm, *__restrict__ const offsets = a.offsets;
    float *__restrict__ const W = job.W;
    const int N = a.N, F = job.F, R = a.R, ldh = a.ldh, S = a.S, chunk = a.chunk;
    constexpr int RC = 16 * MT, POS = 128, LD = POS + 16;  // 72 words a row: 8-byte reads of four rows hit all banks
    __shared__ __align__(16) unsigned short qs[RC][LD];
    __shared__ int rows[POS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int f0 = (bx * (blockDim.x >> 5) + warp) * 64, r0 = blockIdx.z * RC;
    const int total = offsets ? offsets[S] : N;
    const int begin = blockIdx.y * chunk, end = min(begin + chunk, total);
    if (begin >= end) return;
    const bool in = f0 + 8 * g < F;
    const __nv_bfloat16 *p = P + f0 + 8 * g;
    int s = offsets ? adapter_at(offsets, S, begin) : 0;
    for (int lo = begin; lo < end; ++s) {
        const int hi = offsets ? min(end, offsets[s + 1]) : end;
        if (hi <= lo) continue;
        float acc[MT][8][4] = {};
        for (int k0 = lo; k0 < hi; k0 += POS) {
            const int here = min(POS, hi - k0);
            __syncthreads();
            for (int q = threadIdx.x; q < POS * 2 * MT; q += blockDim.x) {
                const int k = q / (2 * MT), r = (q % (2 * MT)) * 8;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (k < here && r0 + r < ldh) {
                    const long long n = perm ? perm[k0 + k] : k0 + k;
                    v = load8_bf16(V + n * ldh + r0 + r);
                    if (r == 0) rows[k] = (int)n;
                }
                const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) qs[r + e][k] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
            }
            __syncthreads();
#pragma unroll MT == 1 ? 4 : 2
            for (int k = 0; k < here; k += 16) {
                uint4 x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = make_uint4(0u, 0u, 0u, 0u);
                    const int kk = k + 4 * t + e;
                    if (in && kk < here) x[e] = *reinterpret_cast<const uint4 *>(p + (long long)rows[kk] * F);
                }
                const unsigned xw[4][4] = {{x[0].x, x[0].y, x[0].z, x[0].w},
                                           {x[1].x, x[1].y, x[1].z, x[1].w},
                                           {x[2].x, x[2].y, x[2].z, x[2].w},
                                           {x[3].x, x[3].y, x[3].z, x[3].w}};
                uint2 qa[MT][2];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    qa[m][0] = *reinterpret_cast<const uint2 *>(&qs[16 * m + g][k + 4 * t]);
                    qa[m][1] = *reinterpret_cast<const uint2 *>(&qs[16 * m + g + 8][k + 4 * t]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const unsigned sel = j & 1 ? 0x7632u : 0x5410u;
                    const unsigned b0 = __byte_perm(xw[0][j >> 1], xw[1][j >> 1], sel);
                    const unsigned b1 = __byte_perm(xw[2][j >> 1], xw[3][j >> 1], sel);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        mma16816(acc[m][j], qa[m][0].x, qa[m][1].x, qa[m][0].y, qa[m][1].y, b0, b1);
                }
            }
        }
        // acc[m][j]: ranks 16 m + g (+ 8), features f0 + 16 t + j (+ 8)
        float *w = W + (long long)(blockIdx.y + s) * R * F;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + 16 * m + g + 8 * h;
                if (r >= R) continue;
                float *d = w + (long long)r * F + f0 + 16 * t;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (f0 + 16 * t + 8 * c >= F) continue;
                    store4(d + 8 * c, make_float4(acc[m][0][2 * h + c], acc[m][1][2 * h + c], acc[m][2][2 * h + c],
                                                  acc[m][3][2 * h + c]));
                    store4(d + 8 * c + 4, make_float4(acc[m][4][2 * h + c], acc[m][5][2 * h + c],
                                                      acc[m][6][2 * h + c], acc[m][7][2 * h + c]));
                }
            }
        lo = hi;
    }
}

// out = the sums of the slots of each adapter.  A block takes 32 features and eight
// ranks of one adapter; its eight warps every eighth chunk, and their sums are
// added in order.  r * rs + f * fs is an entry's place in out[s].
template <typename T>
__global__ void __launch_bounds__(256) reduce_kernel(const __grid_constant__ GradArgs a) {
    __shared__ float part[8][8][33];
    const GradJob &job = a.job[(int)blockIdx.x >= a.first];
    const float *__restrict__ const W = job.W;
    const int *__restrict__ const offsets = a.offsets;
    const int F = job.F, R = a.R, rs = job.rs, fs = job.fs, chunk = a.chunk;
    const int s = blockIdx.y, r0 = blockIdx.z * 8;
    const int f0 = ((int)blockIdx.x >= a.first ? (int)blockIdx.x - a.first : (int)blockIdx.x) * 32;
    const int lo = offsets ? offsets[s] : 0, hi = offsets ? offsets[s + 1] : s == 0 ? a.N : 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float sum[8] = {};
    if (lo < hi && f0 + lane < F) {
        const float *w = W + ((long long)s * R + r0) * F + f0 + lane;
        const int last = (hi - 1) / chunk;
#pragma unroll 4
        for (int z = lo / chunk + warp; z <= last; z += 8)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (r0 + e < R) sum[e] += w[((long long)z * R + e) * F];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][e][lane] = sum[e];
    __syncthreads();
    // neighbouring threads take neighbouring entries of out
    const int r = rs == 1 ? threadIdx.x & 7 : threadIdx.x >> 5, f = rs == 1 ? threadIdx.x >> 3 : threadIdx.x & 31;
    if (r0 + r < R && f0 + f < F) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v += part[q][r][f];
        put(static_cast<T *>(job.out) + (long long)s * R * F + (long long)(r0 + r) * rs + (long long)(f0 + f) * fs, v);
    }
}

// The same where an adapter has few chunks: one thread for a feature and eight ranks
// (256 adapters of 32 rows, rank 16: blocks of reduce_kernel spend their time in
// starting and meeting).
template <typename T>
__global__ void __launch_bounds__(256) reduce_few_kernel(const __grid_constant__ GradArgs a) {
    const GradJob &job = a.job[(int)blockIdx.x >= a.first];
    const int *__restrict__ const offsets = a.offsets;
    const int F = job.F, R = a.R, rs = job.rs, fs = job.fs, chunk = a.chunk;
    const int s = blockIdx.y, r0 = blockIdx.z * 8;
    const int f = ((int)blockIdx.x >= a.first ? (int)blockIdx.x - a.first : (int)blockIdx.x) * 256 + (int)threadIdx.x;
    if (f >= F) return;
    const int lo = offsets ? offsets[s] : 0, hi = offsets ? offsets[s + 1] : s == 0 ? a.N : 0;
    float sum[8] = {};
    if (lo < hi) {
        const float *__restrict__ const w = job.W + ((long long)s * R + r0) * F + f;
        for (int z = lo / chunk; z <= (hi - 1) / chunk; ++z)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (r0 + e < R) sum[e] += w[((long long)z * R + e) * F];
    }
    T *o = static_cast<T *>(job.out) + (long long)s * R * F + (long long)r0 * rs + (long long)f * fs;
    if (sizeof(T) == 2 && rs == 1 && R % 8 == 0 && reinterpret_cast<uintptr_t>(job.out) % 16 == 0) {
        unsigned v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(sum[2 * e], sum[2 * e + 1]);
            v[e] = *reinterpret_cast<const unsigned *>(&h);
        }
        *reinterpret_cast<uint4 *>(o) = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (r0 + e < R) put(o + (long long)e * rs, sum[e]);
    }
}

// B as the tensor-core product reads it: out[s][f][r], r < Rp (a multiple of 8), zeros past R.
__global__ void __launch_bounds__(256)
    pack_kernel(const unsigned short *__restrict__ W, unsigned short *__restrict__ out, int S, int F, int R, int Rp) {
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    const int octets = Rp / 8;
    if (at >= (long long)S * octets * F) return;
    const long long row = at / octets;
    const int o = (int)(at - row * octets);
    const unsigned short *w = W + row * R;
    unsigned v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (8 * o + e < R) v[e >> 1] |= (unsigned)w[8 * o + e] << (16 * (e & 1));
    *reinterpret_cast<uint4 *>(out + row * Rp + 8 * o) = make_uint4(v[0], v[1], v[2], v[3]);
}

// ---------------------------------------------------------------- host side
struct Adapters {
    const float *scales;
    const int *ids;
    int S, R;
    bool bf16;
    cudaStream_t st;
};

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int round_up(int x, int m) { return (x + m - 1) / m * m; }

// Words of a tile's list (TcAdapters::lists), and tiles.
int list_stride(int S) { return 8 + 8 * std::min(S, 128); }
long long list_tiles(long long N) { return (N + 127) / 128; }

// Bytes of H as operand planes (TcAdapters::planes).
size_t plane_bytes(long long N, int R) { return (size_t)list_tiles(N) * round_up(R, 16) * 256; }

// Whether X and W (S x R x F) can take the vector kernels.
bool shrink_vec(const Adapters &q, const void *X, const void *W, int F) {
    return aligned(X, 16) && aligned(W, 16) && F % (q.bf16 ? 8 : 4) == 0;
}

// One warp for four ranks of a row, W[s] read again for each row, while that is at
// most 16 MB (fp32: 64 MB, its tiles are slower) from L2: more warps than the
// tiles have.
bool by_rows(const Adapters &q, long long N, int F) {
    return (double)N * q.R * F * (q.bf16 ? 2 : 4) <= (q.bf16 ? 16e6 : 64e6);
}

// H = scale X W^T of one or two jobs.  h_bf16: their H are bf16; lists: null, or the
// lists of the product that takes the adapters as stages, to be built (a tensor-core
// product's planes are job[0]'s; the caller has made sure of vectors); its bias to
// be packed; few: row by row (by_rows); widest: F of the widest job that the call can have.
cudaError_t shrink(const Adapters &q, const ShrinkJob *job, int jobs, bool h_bf16, long long N, int ldh, int *lists,
                   bool few, int widest, const BiasPack &bias = BiasPack{}) {
    ShrinkArgs p{};
    bool vec = true;
    for (int j = 0; j < jobs; ++j) {
        p.job[j] = job[j];
        vec = vec && shrink_vec(q, job[j].X, job[j].W, job[j].F);
    }
    p.scales = q.scales, p.ids = q.ids, p.N = N, p.R = q.R, p.ldh = ldh, p.S = q.S;
    p.plane_r = round_up(q.R, 16);
    p.status = device_status_ptr();
    const unsigned z = (unsigned)jobs;
    if (!vec && jobs == 2) {  // each as it can
        const cudaError_t e = shrink(q, job, 1, h_bf16, N, ldh, lists, few, widest);
        return e == cudaSuccess ? shrink(q, job + 1, 1, h_bf16, N, ldh, nullptr, few, widest) : e;
    }
    if (few) return launch_shrink_rows(p, jobs, q.bf16, vec, q.st);
    if (!vec) {
        const dim3 grid((unsigned)((N + 31) / 32), (unsigned)((ldh + 7) / 8), z);
        if (!q.bf16)
            shrink_any_kernel<float, float><<<grid, 128, 0, q.st>>>(p);
        else if (h_bf16)
            shrink_any_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 128, 0, q.st>>>(p);
        else
            shrink_any_kernel<__nv_bfloat16, float><<<grid, 128, 0, q.st>>>(p);
        return cudaGetLastError();
    }
    if (!q.bf16) {
        const int octets = (ldh + 7) / 8, list_blocks = lists ? (int)((list_tiles(N) + 3) / 4) : 0;
        // A block's four warps share eight rows where there are few blocks (841 x 12288, rank 3: 114
        // and 34 us), or where the features are many, W's being read by neighbours then (25216 x 12288,
        // rank 8: 329 and 248 us; 25216 x 384: 17 and 25).
        const bool split = (N + 31) / 32 * octets < 4 * sm_count() || widest >= 2048;
        const int row_blocks = (int)(split ? (N + 7) / 8 : (N + 31) / 32);
        const dim3 grid((unsigned)(row_blocks + list_blocks), (unsigned)octets, z);
        if (split)
            shrink_fp32_kernel<4><<<grid, 128, 0, q.st>>>(p, row_blocks, lists, list_stride(q.S));
        else
            shrink_fp32_kernel<1><<<grid, 128, 0, q.st>>>(p, row_blocks, lists, list_stride(q.S));
        return cudaGetLastError();
    }
    const int cols = lists ? std::max(ldh, p.plane_r) : ldh;
    const int nt = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
    // 16 rows a block for few ranks (more warps for X's latency), 32 for many (W is read half as often)
    const int rows = nt <= 2 ? 16 : 32;
    const int row_blocks = (int)((N + rows - 1) / rows), list_blocks = lists ? (int)((list_tiles(N) + 7) / 8) : 0;
    const dim3 grid((unsigned)(row_blocks + bias.blocks + list_blocks), (unsigned)((cols + 8 * nt - 1) / (8 * nt)), z);
    const auto go = [&](auto kernel) {
        kernel<<<grid, 256, 0, q.st>>>(p, row_blocks, lists, list_stride(q.S), bias);
        return cudaGetLastError();
    };
    const auto ranks = [&](auto h) {
        using O = decltype(h);
        return nt == 1   ? go(shrink_mma_kernel<1, 1, O>)
               : nt == 2 ? go(shrink_mma_kernel<1, 2, O>)
                         : go(shrink_mma_kernel<2, 4, O>);
    };
    return h_bf16 ? ranks(__nv_bfloat16{}) : ranks(float{});
}

// Y = act(P + bias + H W), P in fp32 (Y itself, or a workspace); with_a: W is A (rank x F), else B (F x rank).
template <typename T>
cudaError_t expand(const Adapters &q, void *Y, const float *P, const void *W, bool with_a, long long N, int F,
                   const float *H, int ldh, const void *bias, int act) {
    T *y = static_cast<T *>(Y);
    const T *w = static_cast<const T *>(W), *b = static_cast<const T *>(bias);
    const size_t smem = (size_t)ldh * kExpandRows * 4;
    if (F % 4 == 0 && aligned(Y, 4 * sizeof(T)) && aligned(P, 16) && aligned(W, 4 * sizeof(T)) &&
        aligned(bias, 4 * sizeof(T)) && (with_a || q.R % 4 == 0) && (F + 511LL) / 512 <= 65535) {
        const dim3 grid((unsigned)((N + kExpandRows - 1) / kExpandRows), (unsigned)((F + 511) / 512));
        const auto go = [&](auto kernel) {
            kernel<<<grid, 128, smem, q.st>>>(y, P, w, q.ids, H, N, F, q.R, ldh, q.S, b);
            return cudaGetLastError();
        };
        if (with_a) return go(expand_kernel<T, false, KS_ACT_NONE>);
        switch (act) {
            case KS_ACT_NONE: return go(expand_kernel<T, true, KS_ACT_NONE>);
            case KS_ACT_RELU: return go(expand_kernel<T, true, KS_ACT_RELU>);
            case KS_ACT_GELU_TANH: return go(expand_kernel<T, true, KS_ACT_GELU_TANH>);
            default: return go(expand_kernel<T, true, KS_ACT_GELU_ERF>);
        }
    }
    const int threads = F >= 512 ? 128 : round_up((F + 3) / 4, 32);
    const long long blocks = (N + kExpandRows - 1) / kExpandRows * ((F + 4LL * threads - 1) / (4 * threads));
    if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
    const auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, threads, smem, q.st>>>(y, P, w, q.ids, H, N, F, q.R, ldh, q.S, b, act);
        return cudaGetLastError();
    };
    if (with_a) return go(expand_any_kernel<T, false, false>);
    return q.R % 4 == 0 && aligned(W, 4 * sizeof(T)) ? go(expand_any_kernel<T, true, true>)
                                                     : go(expand_any_kernel<T, true, false>);
}

// The product of a call that does not take the adapters along (bf16: with y_f32), in small tiles where the
// library would stream, and in fp32 where they are at most two for each SM (300 rows of (1, 256, 256,
// 4): 18 us, 62 of the fp32 kernel, whose CTAs are fewer and longer; from 600 tiles on, 2400
// rows, it catches up).
ks_status product(const Problem &p) {
    Plan plan;
    const char *why = "";
    const long long blocks = p.a * p.d * ((p.b + kProductTile - 1) / kProductTile);
    const long long tiles = (p.batch + kProductTile - 1) / kProductTile;
    // (smaller blocks leave most of a tile empty: 20000 rows of (2, 16, 8, 3) take 19 us of either kind)
    if (p.dtype == KS_TF32 || p.b < 16 || p.c < 4 || tiles > 65535 || blocks > INT_MAX ||
        !make_plan(p, KS_VARIANT_AUTO, &plan, &why) ||
        (plan.variant != KS_VARIANT_STREAM && (p.dtype != KS_F32 || blocks * tiles > 2 * sm_count())))
        return run(p, KS_VARIANT_AUTO);
    const dim3 grid((unsigned)blocks, (unsigned)tiles);
    const auto go = [&](auto t) {
        using T = decltype(t);
        tile_product_kernel<T><<<grid, 256, 0, p.stream>>>(static_cast<const T *>(p.X), static_cast<const T *>(p.V),
                                                          static_cast<float *>(p.Y), p.batch, (int)p.a, (int)p.b,
                                                          (int)p.c, (int)p.d);
        return cudaGetLastError();
    };
    const cudaError_t e = p.dtype == KS_BF16 ? go(__nv_bfloat16{}) : go(float{});
    return e == cudaSuccess ? KS_OK : cuda_fail(e, "adapter product launch");
}

// The product and the second pass over it: p.Y = act(X K^T + bias + H W).  In bf16 the product goes
// to `sums` in fp32, product_rows() rows at a time (p's bias and act are the second pass's).  Twice
// the bytes of a product in bf16 between the two passes: (1, 96, 24, 8) 58 us either way, (8, 2, 2,
// 256) 181 us for 156, 8000 rows each.  Pieces of 64 MB do not gain by L2 what they lose at their
// ends (195 us, 24 MB: 234), so the limit is one on memory.
constexpr long long kSumsBytes = 256 << 20;
long long product_rows(const Problem &p) {
    const long long rows = kSumsBytes / (4 * p.out_features()) / 128 * 128;
    return p.dtype == KS_BF16 ? std::min<long long>(p.batch, std::max<long long>(128, rows)) : p.batch;
}
size_t sums_bytes(const Problem &p) {
    return p.dtype == KS_BF16 ? (size_t)(product_rows(p) * p.out_features() * 4) : 0;
}
ks_status product_and_expand(Adapters q, const Problem &p, char *sums, const void *W, bool with_a, const float *H,
                             int ldh) {
    const int F = (int)p.out_features(), es = p.elem_bytes();
    const long long step = product_rows(p);
    for (long long n0 = 0; n0 < p.batch; n0 += step) {
        Problem part = p;
        part.X = static_cast<const char *>(p.X) + n0 * p.in_features() * es;
        part.batch = std::min<long long>(step, p.batch - n0);
        void *const Y = static_cast<char *>(p.Y) + n0 * F * es;
        part.Y = q.bf16 ? sums : Y;
        part.y_f32 = q.bf16;
        part.bias = nullptr, part.act = KS_ACT_NONE;
        const ks_status s = product(part);
        if (s != KS_OK) return s;
        const auto *P = static_cast<const float *>(part.Y);
        const cudaError_t e =
            q.bf16 ? expand<__nv_bfloat16>(q, Y, P, W, with_a, part.batch, F, H + n0 * ldh, ldh, p.bias, p.act)
                   : expand<float>(q, Y, P, W, with_a, part.batch, F, H + n0 * ldh, ldh, p.bias, p.act);
        if (e != cudaSuccess) return cuda_fail(e, "adapter launch");
        if (q.ids) q.ids += step;
    }
    return KS_OK;
}

// How the gradients (dA, dB; out null: not wanted) are cut: feature blocks of each,
// `bz` blocks of ranks, chunks of `chunk` of the N rows, for about 16 warps an SM
// (tensor cores) or 32.
struct GradPlan {
    bool mma, vec;
    int warps, bx[2], bz, rc, chunk, chunks;
    size_t at[2], bytes;  // partial sums of each, and of both
};
GradPlan grad_plan(const Adapters &q, const GradJob (&job)[2], long long N) {
    GradPlan g{};
    const int widest = std::max(job[0].F, job[1].F);
    const auto vectors = [&](int v) {
        return job[0].F % v == 0 && job[1].F % v == 0 && aligned(job[0].P, 16) && aligned(job[1].P, 16);
    };
    g.mma = q.bf16 && vectors(8);
    g.vec = !q.bf16 && vectors(4);
    g.warps = g.mma ? std::min(8, (widest + 63) / 64) : 4;
    const int features = g.mma ? 64 * g.warps : 128;
    g.rc = g.mma ? (q.R <= 16 ? 16 : q.R <= 32 ? 32 : 64) : q.R <= 8 ? 8 : 16;
    g.bz = (q.R + g.rc - 1) / g.rc;
    long long blocks = 0;
    for (int j = 0; j < 2; ++j) blocks += g.bx[j] = (job[j].F + features - 1) / features;
    const long long wanted = std::max<long long>(1, (g.mma ? 16LL : 32LL) * sm_count() / g.warps / (blocks * g.bz));
    long long chunk = std::max<long long>(64, (N + wanted - 1) / wanted);
    chunk = std::min<long long>((chunk + 15) / 16 * 16, (N + 15) / 16 * 16);
    chunk = std::max<long long>(chunk, (N + 65534) / 65535);  // grid limit
    g.chunk = (int)chunk;
    g.chunks = (int)((N + chunk - 1) / chunk);
    for (int j = 0; j < 2; ++j) {
        if (!job[j].out) {
            g.bx[j] = 0;
            continue;
        }
        g.at[j] = g.bytes;
        g.bytes += ((size_t)(g.chunks + q.S) * (size_t)q.R * (size_t)job[j].F * 4 + 255) / 256 * 256;
    }
    return g;
}

cudaError_t grads(const Adapters &q, const GradPlan &g, const GradJob (&job)[2], bool v_bf16, int ldh,
                  const int *perm, const int *offsets, long long N, char *W) {
    GradArgs p{};
    const bool few = g.chunks <= 3 * q.S;  // chunks of an adapter, were the rows spread evenly
    int reduce_blocks[2] = {};
    for (int j = 0; j < 2; ++j) {
        p.job[j] = job[j];
        p.job[j].W = reinterpret_cast<float *>(W + g.at[j]);
        if (job[j].out) reduce_blocks[j] = few ? (job[j].F + 255) / 256 : (job[j].F + 31) / 32;
    }
    p.perm = perm, p.offsets = offsets, p.N = (int)N, p.R = q.R, p.ldh = ldh, p.S = q.S, p.chunk = g.chunk;
    p.first = g.bx[0];
    const dim3 grid((unsigned)(g.bx[0] + g.bx[1]), (unsigned)g.chunks, (unsigned)g.bz);
    const auto go = [&](auto kernel) {
        kernel<<<grid, 32 * g.warps, 0, q.st>>>(p);
        return cudaGetLastError();
    };
    const auto mma = [&](auto v) {
        using V = decltype(v);
        return g.rc == 16   ? go(grad_mma_kernel<1, V>)
               : g.rc == 32 ? go(grad_mma_kernel<2, V>)
                            : go(grad_mma_kernel<4, V>);
    };
    cudaError_t e;
    if (g.mma)
        e = v_bf16 ? mma(__nv_bfloat16{}) : mma(float{});
    else if (q.bf16)
        e = g.rc == 8 ? go(grad_kernel<__nv_bfloat16, 8, false>) : go(grad_kernel<__nv_bfloat16, 16, false>);
    else if (g.vec)
        e = g.rc == 8 ? go(grad_kernel<float, 8, true>) : go(grad_kernel<float, 16, true>);
    else
        e = g.rc == 8 ? go(grad_kernel<float, 8, false>) : go(grad_kernel<float, 16, false>);
    if (e != cudaSuccess) return e;
    p.first = reduce_blocks[0];
    const dim3 rgrid((unsigned)(reduce_blocks[0] + reduce_blocks[1]), (unsigned)q.S, (unsigned)((q.R + 7) / 8));
    const auto sum = [&](auto kernel) {
        kernel<<<rgrid, 256, 0, q.st>>>(p);
        return cudaGetLastError();
    };
    if (q.bf16) return few ? sum(reduce_few_kernel<__nv_bfloat16>) : sum(reduce_kernel<__nv_bfloat16>);
    return few ? sum(reduce_few_kernel<float>) : sum(reduce_kernel<float>);
}

// (each adapter's rows are found by a scan of all ids: prepare_kernel)
constexpr int kMaxAdapters = 4096, kMaxRank = 1024;

struct Checked {
    int64_t in_f, out_f, nvals, abytes, bbytes;
    int elem;
};

ks_status check(int64_t a, int64_t b, int64_t c, int64_t d, int64_t batch, int dtype, const void *A, const void *B,
                const float *scales, const int32_t *ids, int64_t n_adapters, int64_t rank, Checked *o) {
    ks_status s = check_dtype(dtype);
    if (s != KS_OK) return s;
    if ((s = check_sizes(a, b, c, d, batch, &o->in_f, &o->out_f, &o->nvals)) != KS_OK) return s;
    if (n_adapters < 1 || n_adapters > kMaxAdapters)
        return record_error(KS_ERR_INVALID_ARG, "n_adapters must be in 1..%d (got %lld)", kMaxAdapters,
                            (long long)n_adapters);
    if (rank < 1 || rank > kMaxRank)
        return record_error(KS_ERR_INVALID_ARG, "rank must be in 1..%d (got %lld)", kMaxRank, (long long)rank);
    // rows are indexed with 32 bits (ids and their order), one thread per output in places
    if (batch > (int64_t{1} << 30)) return record_error(KS_ERR_INVALID_ARG, "adapters take at most 2^30 rows");
    o->elem = dtype == KS_BF16 ? 2 : 4;
    o->abytes = n_adapters * rank * o->in_f * o->elem;
    o->bbytes = n_adapters * rank * o->out_f * o->elem;
    if (batch > 0 && (!A || !B)) return record_error(KS_ERR_INVALID_ARG, "A and B must be non-null");
    if ((s = check_align(A, o->elem, "A")) != KS_OK || (s = check_align(B, o->elem, "B")) != KS_OK ||
        (s = check_align(scales, 4, "scales")) != KS_OK || (s = check_align(ids, 4, "ids")) != KS_OK)
        return s;
    return KS_OK;
}

// `out` must not share bytes with any of the adapters' inputs.
ks_status check_apart(const void *out, int64_t bytes, const char *name, const void *A, const void *B,
                      const float *scales, const int32_t *ids, int64_t n_adapters, int64_t batch, const Checked &o) {
    if (ranges_overlap(out, bytes, A, o.abytes)) return record_error(KS_ERR_INVALID_ARG, "%s overlaps A", name);
    if (ranges_overlap(out, bytes, B, o.bbytes)) return record_error(KS_ERR_INVALID_ARG, "%s overlaps B", name);
    if (ranges_overlap(out, bytes, scales, n_adapters * 4))
        return record_error(KS_ERR_INVALID_ARG, "%s overlaps scales", name);
    if (ranges_overlap(out, bytes, ids, batch * 4)) return record_error(KS_ERR_INVALID_ARG, "%s overlaps ids", name);
    return KS_OK;
}

// Offsets of the parts of one workspace, 256-byte aligned.
struct Layout {
    size_t bytes = 0;
    size_t add(size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    }
};

// Whether the tensor-core kernel can take the product with adapters beside it:
// bf16, and a pattern that AUTO gives to it.  The product's V may be null: a workspace's.
bool fuses(const Adapters &q, Problem p, int F) {
    if (!q.bf16) return false;
    static const char dummy[16] __attribute__((aligned(256))) = {};
    if (!p.V) p.V = dummy;
    Plan plan;
    const char *why = "";
    const int ldh = round_up(q.R, 8);
    const TcAdapters tc{dummy, dummy, nullptr, q.S, ldh, 0};
    p.ad = &tc;
    return make_plan(p, KS_VARIANT_AUTO, &plan, &why) && plan.variant == KS_VARIANT_TC &&
           tc_adapters_supported(p, tc) && shrink_vec(q, p.X, nullptr, F);
}

// The same for the fp32 kernel, with A's vectors aligned (null: a workspace's).
bool fuses_fp32(const Adapters &q, Problem p, const void *A, int F) {
    static const char dummy[16] __attribute__((aligned(256))) = {};
    if (!p.V) p.V = dummy;
    return !q.bf16 && p.dtype == KS_F32 && shrink_vec(q, p.X, A, F) && fma32_adapters_supported(p);
}

cudaError_t pack(const Adapters &q, const void *W, void *out, int F, int Rp) {
    const long long n = (long long)q.S * F * (Rp / 8);
    if ((n + 255) / 256 > INT_MAX) return cudaErrorInvalidConfiguration;
    pack_kernel<<<(unsigned)((n + 255) / 256), 256, 0, q.st>>>(static_cast<const unsigned short *>(W),
                                                               static_cast<unsigned short *>(out), q.S, F, q.R, Rp);
    return cudaGetLastError();
}

// A transpose of prepare_kernel: out[q][c][r] = in[q][r][c], rows of out ld long.
Transpose transpose(const void *in, void *out, long long blocks, long long rows, long long cols, long long ld) {
    Transpose t{in, out, blocks, (int)rows, (int)cols, (int)ld, (int)((ld + 31) / 32), (int)((cols + 31) / 32), 0};
    t.tiles = blocks * t.tr * t.tc;
    return t;
}

cudaError_t prepare(const Adapters &q, PrepareArgs &p, long long N) {
    long long tiles = 0;
    for (const Transpose &t : p.job) tiles += t.tiles;
    const long long blocks = p.sorted + std::min<long long>(tiles, 16LL * sm_count());
    if (blocks == 0) return cudaSuccess;
    p.ids = q.ids, p.N = (int)N, p.S = q.S;
    if (q.bf16)
        prepare_kernel<unsigned short><<<(unsigned)blocks, kPrepareThreads, 0, q.st>>>(p);
    else
        prepare_kernel<float><<<(unsigned)blocks, kPrepareThreads, 0, q.st>>>(p);
    return cudaGetLastError();
}

ks_status alloc(char **p, size_t bytes, cudaStream_t st) {
    const cudaError_t e = pool_alloc(reinterpret_cast<void **>(p), bytes, st);
    if (e == cudaSuccess) return KS_OK;
    (void)cudaGetLastError();
    return record_error(KS_ERR_ALLOC, "workspace allocation of %zu bytes failed: %s", bytes, cudaGetErrorString(e));
}

}  // namespace
}  // namespace ks

using namespace ks;

extern "C" {

ks_status ks_adapter_matmul(const void *X, const void *values, int64_t a, int64_t b, int64_t c, int64_t d,
                            int64_t batch, void *Y, int dtype, const void *bias, int activation, const void *A,
                            const void *B, const float *scales, const int32_t *ids, int64_t n_adapters, int64_t rank,
                            void *stream) {
    Checked o;
    ks_status s = check(a, b, c, d, batch, dtype, A, B, scales, ids, n_adapters, rank, &o);
    if (s != KS_OK) return s;
    if (activation < KS_ACT_NONE || activation > KS_ACT_GELU_ERF)
        return record_error(KS_ERR_INVALID_ARG, "unknown activation %d", activation);
    if (batch == 0) return KS_OK;
    if ((s = check_apart(Y, batch * o.out_f * o.elem, "Y", A, B, scales, ids, n_adapters, batch, o)) != KS_OK) return s;
    Problem p;
    bool noop = false;
    if ((s = make_problem(X, values, a, b, c, d, batch, Y, dtype, stream, &p, &noop)) != KS_OK) return s;
    if ((s = check_align(bias, o.elem, "bias")) != KS_OK) return s;
    if (bias && ranges_overlap(Y, batch * o.out_f * o.elem, bias, o.out_f * o.elem))
        return record_error(KS_ERR_INVALID_ARG, "Y overlaps bias");
    const Adapters q{scales, ids, (int)n_adapters, (int)rank, dtype == KS_BF16, p.stream};
    const int in_f = (int)o.in_f, out_f = (int)o.out_f;
    cudaError_t e;
    char *w = nullptr;
    const int row_ldh = round_up(q.R, 4);
    if (adapter_rows_supported(p, row_ldh)) {
        // few rows: one launch, or two where A[s] is more than a block should read for itself, which
        // takes four rows from 16 on (32 rows in fp32, A[s] of 64 KB: 25 us in one, 19 in two)
        const bool apart = (size_t)q.R * in_f * o.elem > (batch < 16 ? 64 : 32) * 1024;
        p.bias = bias;
        p.act = activation;
        if (!apart) {
            e = launch_adapter_rows(p, A, B, scales, ids, q.S, q.R, nullptr, row_ldh);
            return e == cudaSuccess ? KS_OK : cuda_fail(e, "adapter launch");
        }
        if ((s = alloc(&w, (size_t)batch * row_ldh * 4, q.st)) != KS_OK) return s;
        float *H = reinterpret_cast<float *>(w);
        const ShrinkJob job{X, A, H, nullptr, in_f};
        e = shrink(q, &job, 1, false, batch, row_ldh, nullptr, true, in_f);
        if (e == cudaSuccess) e = launch_adapter_rows(p, A, B, scales, ids, q.S, q.R, H, row_ldh);
    } else if (fuses(q, p, in_f)) {
        // the adapters as K steps of the tensor-core product, with its bias and activation
        Layout m;
        const int ldh = round_up(q.R, 8);
        const size_t h = m.add(plane_bytes(batch, q.R)), l = m.add((size_t)list_tiles(batch) * list_stride(q.S) * 4);
        const bool packed = q.R != ldh || !aligned(B, 16);
        const size_t b_at = packed ? m.add((size_t)q.S * out_f * ldh * 2) : 0;
        const size_t a_at = aligned(A, 16) ? 0 : m.add((size_t)o.abytes);  // a copy that H's vectors can read
        const size_t bias_at = bias ? m.add((size_t)out_f * 16) : 0, ones_at = bias ? m.add(4096) : 0;
        if ((s = alloc(&w, m.bytes, q.st)) != KS_OK) return s;
        TcAdapters tc{packed ? w + b_at : B, w + h, reinterpret_cast<int *>(w + l), q.S, ldh, list_stride(q.S)};
        BiasPack pack_b{};
        if (bias) {
            tc.bias = w + bias_at, tc.ones = w + ones_at;
            pack_b = BiasPack{static_cast<const unsigned short *>(bias), reinterpret_cast<uint4 *>(w + bias_at),
                              reinterpret_cast<uint4 *>(w + ones_at), out_f, (out_f + 255) / 256};
        }
        e = packed ? pack(q, B, w + b_at, out_f, ldh) : cudaSuccess;
        const void *vectors = A;
        if (!aligned(A, 16)) {
            vectors = w + a_at;
            if (e == cudaSuccess) e = cudaMemcpyAsync(w + a_at, A, (size_t)o.abytes, cudaMemcpyDeviceToDevice, q.st);
        }
        const ShrinkJob job{X, vectors, nullptr, reinterpret_cast<unsigned short *>(w + h), in_f};
        if (e == cudaSuccess) e = shrink(q, &job, 1, true, batch, ldh, reinterpret_cast<int *>(w + l), false, in_f, pack_b);
        if (e == cudaSuccess) {
            p.act = activation;
            p.ad = &tc;
            s = run(p, KS_VARIANT_TC);
        }
    } else if (fuses_fp32(q, p, A, in_f)) {
        // the adapters as stages of the fp32 product, with its bias and activation
        Layout m;
        const int ldh = round_up(q.R, 4);
        const size_t h = m.add((size_t)batch * ldh * 4), l = m.add((size_t)list_tiles(batch) * list_stride(q.S) * 4);
        const size_t v = m.add((size_t)o.nvals * 4);
        if ((s = alloc(&w, m.bytes, q.st)) != KS_OK) return s;
        const auto *vt = reinterpret_cast<const float *>(w + v);
        const ShrinkJob job{X, A, w + h, nullptr, in_f};
        e = launch_transpose_blocks(values, w + v, a * d, b, c, dtype, q.st);
        if (e == cudaSuccess) e = shrink(q, &job, 1, false, batch, ldh, reinterpret_cast<int *>(w + l), false, in_f);
        p.bias = bias;
        p.act = activation;
        const Fma32Adapters ad{reinterpret_cast<const float *>(w + h), static_cast<const float *>(B),
                               reinterpret_cast<const int *>(w + l), q.R, ldh, q.R, list_stride(q.S)};
        if (e == cudaSuccess) e = launch_fma32_adapters(p, vt, ad);
    } else {
        // H, then the product and one pass that adds the adapters, the bias and the activation
        Layout m;
        const int ldh = round_up(q.R, 4);
        const size_t h = m.add((size_t)batch * ldh * 4), sums = m.add(sums_bytes(p));
        if ((s = alloc(&w, m.bytes, q.st)) != KS_OK) return s;
        const ShrinkJob job{X, A, w + h, nullptr, in_f};
        e = shrink(q, &job, 1, false, batch, ldh, nullptr, by_rows(q, batch, in_f), in_f);
        p.bias = bias;
        p.act = activation;
        if (e == cudaSuccess)
            s = product_and_expand(q, p, w + sums, B, false, reinterpret_cast<const float *>(w + h), ldh);
    }
    if (e != cudaSuccess && s == KS_OK) s = cuda_fail(e, "adapter launch");
    e = cudaFreeAsync(w, q.st);
    if (e != cudaSuccess && s == KS_OK) s = cuda_fail(e, "workspace free");
    return s;
}

ks_status ks_adapter_backward(const void *dY, const void *X, const void *values, int64_t a, int64_t b, int64_t c,
                              int64_t d, int64_t batch, int dtype, const void *A, const void *B, const float *scales,
                              const int32_t *ids, int64_t n_adapters, int64_t rank, void *dX, void *dA, void *dB,
                              void *stream) {
    Checked o;
    ks_status s = check(a, b, c, d, batch, dtype, A, B, scales, ids, n_adapters, rank, &o);
    if (s != KS_OK) return s;
    const int64_t xb = batch * o.in_f * o.elem, yb = batch * o.out_f * o.elem;
    struct { void *p; int64_t bytes; const char *name; } outs[3] = {{dX, xb, "dX"}, {dA, o.abytes, "dA"}, {dB, o.bbytes, "dB"}};
    for (int k = 0; k < 3; ++k) {
        if (!outs[k].p) continue;
        if ((s = check_align(outs[k].p, o.elem, outs[k].name)) != KS_OK ||
            (s = check_apart(outs[k].p, outs[k].bytes, outs[k].name, A, B, scales, ids, n_adapters, batch, o)) != KS_OK)
            return s;
        if (ranges_overlap(outs[k].p, outs[k].bytes, dY, yb) || ranges_overlap(outs[k].p, outs[k].bytes, X, xb) ||
            ranges_overlap(outs[k].p, outs[k].bytes, values, o.nvals * o.elem))
            return record_error(KS_ERR_INVALID_ARG, "%s overlaps dY, X or values", outs[k].name);
        for (int j = 0; j < k; ++j)
            if (ranges_overlap(outs[k].p, outs[k].bytes, outs[j].p, outs[j].bytes))
                return record_error(KS_ERR_INVALID_ARG, "%s overlaps %s", outs[k].name, outs[j].name);
    }
    const Adapters q{scales, ids, (int)n_adapters, (int)rank, dtype == KS_BF16, static_cast<cudaStream_t>(stream)};
    if (batch == 0) {  // empty sums
        cudaError_t e = cudaSuccess;
        if (dA) e = cudaMemsetAsync(dA, 0, (size_t)o.abytes, q.st);
        if (e == cudaSuccess && dB) e = cudaMemsetAsync(dB, 0, (size_t)o.bbytes, q.st);
        return e == cudaSuccess ? KS_OK : cuda_fail(e, "gradient clear");
    }
    if (!dY || ((dA || dB) && !X) || (dX && !values))
        return record_error(KS_ERR_INVALID_ARG, "dY, X (for dA and dB) and values (for dX) must be non-null");
    if ((s = check_align(dY, o.elem, "dY")) != KS_OK || (s = check_align(X, o.elem, "X")) != KS_OK ||
        (s = check_align(values, o.elem, "values")) != KS_OK)
        return s;
    if (!dX && !dA && !dB) return KS_OK;
    const int in_f = (int)o.in_f, out_f = (int)o.out_f;
    // Workspace: G and H, B transposed to rank x out (what G contracts over), the
    // rows' order, the partial sums, for dX the transposed values and, fused, A
    // packed to in x rank, the lists and G's planes.
    Layout m;
    const int ldh = round_up(q.R, 8);
    const bool want_g = dX || dA;
    const size_t bt = want_g ? m.add((size_t)o.bbytes) : 0;
    // dX = dY K: the product of pattern (a, c, b, d) with the transposed blocks.  What
    // is wanted, and the alignment of what dX alone reads and writes (values, dX), do not decide
    // how G, H and the sums are computed: a gradient asked for alone has the bits it has beside the others.
    static const char dummy[16] __attribute__((aligned(256))) = {};
    Problem p{dY, nullptr, const_cast<char *>(dummy), a, c, b, d, batch, dtype, q.st};
    // Few rows: the kernel of few rows, G for H and A transposed for B.
    const bool rowable = adapter_rows_supported(p, ldh), rows_x = rowable && dX;
    const bool fusable = !rowable && fuses(q, p, out_f), fused = fusable && dX && aligned(dX, 16);
    // fp32: the transposed blocks, transposed for the kernel, are the values as they are
    const bool fusable32 = !rowable && fuses_fp32(q, p, nullptr, out_f);
    const bool fused32 = fusable32 && dX && aligned(dX, 16) && aligned(values, 16);
    p.Y = dX;
    GradJob grad[2] = {{X, nullptr, nullptr, dA, in_f, in_f, 1}, {dY, nullptr, nullptr, dB, out_f, 1, q.R}};
    const GradPlan plan = grad_plan(q, grad, batch);
    // rows of G and H in bf16 where no kernel sees more of them: those of the tensor cores round them themselves
    const bool v_bf16 = fused && plan.mma;
    const size_t vt = dX && !fused32 ? m.add((size_t)(o.nvals * o.elem)) : 0;
    const bool rows_g = dA || !fused;  // G also as rows
    const size_t h_bytes = (size_t)batch * ldh * (v_bf16 ? 2 : 4);
    const size_t g_at = want_g && rows_g ? m.add(h_bytes) : 0, h_at = dB ? m.add(h_bytes) : 0;
    const size_t p_at = fused ? m.add(plane_bytes(batch, q.R)) : 0;
    const size_t l_at = fused || fused32 ? m.add((size_t)list_tiles(batch) * list_stride(q.S) * 4) : 0;
    const size_t ap = fused || fused32 || rows_x ? m.add((size_t)q.S * in_f * ldh * o.elem) : 0;
    const size_t sums = dX && !fused && !fused32 && !rows_x ? m.add(sums_bytes(p)) : 0;
    const bool sorted = ids && (dA || dB);
    const size_t perm_at = sorted ? m.add((size_t)batch * 4) : 0, off_at = sorted ? m.add((size_t)(q.S + 1) * 4) : 0;
    const size_t w_at = dA || dB ? m.add(plan.bytes) : 0;
    char *w = nullptr;
    if ((s = alloc(&w, m.bytes, q.st)) != KS_OK) return s;
    int *perm = sorted ? reinterpret_cast<int *>(w + perm_at) : nullptr;
    int *offsets = sorted ? reinterpret_cast<int *>(w + off_at) : nullptr;
    int *lists = fused || fused32 ? reinterpret_cast<int *>(w + l_at) : nullptr;

    PrepareArgs prep{};
    prep.perm = perm, prep.offsets = offsets, prep.sorted = sorted ? q.S : 0;
    if (want_g) prep.job[0] = transpose(B, w + bt, q.S, o.out_f, q.R, o.out_f);
    if (dX && !fused32) prep.job[1] = transpose(values, w + vt, a * d, b, c, b);
    if (fused || fused32 || rows_x) prep.job[2] = transpose(A, w + ap, q.S, q.R, o.in_f, ldh);
    cudaError_t e = prepare(q, prep, batch);
    ShrinkJob job[2];
    int n_jobs = 0;
    if (want_g)
        job[n_jobs++] = ShrinkJob{dY, w + bt, rows_g ? w + g_at : nullptr,
                                  fused ? reinterpret_cast<unsigned short *>(w + p_at) : nullptr, out_f};
    if (dB) job[n_jobs++] = ShrinkJob{X, A, w + h_at, nullptr, in_f};
    if (e == cudaSuccess)
        e = shrink(q, job, n_jobs, v_bf16, batch, ldh, lists,
                   !fusable && !fusable32 && by_rows(q, batch, std::max(in_f, out_f)), std::max(in_f, out_f));
    if (fused32 && e == cudaSuccess) {
        const Fma32Adapters ad{reinterpret_cast<const float *>(w + g_at), reinterpret_cast<const float *>(w + ap), lists,
                               q.R, ldh, ldh, list_stride(q.S)};
        e = launch_fma32_adapters(p, static_cast<const float *>(values), ad);
    } else if (rows_x && e == cudaSuccess) {
        p.V = w + vt;
        e = launch_adapter_rows(p, nullptr, w + ap, nullptr, ids, q.S, ldh, reinterpret_cast<const float *>(w + g_at), ldh);
    } else if (dX && e == cudaSuccess) {
        p.V = w + vt;
        const TcAdapters tc{w + ap, w + p_at, lists, q.S, ldh, list_stride(q.S)};
        if (fused) p.ad = &tc;
        s = fused ? run(p, KS_VARIANT_TC)
                  : product_and_expand(q, p, w + sums, A, true, reinterpret_cast<const float *>(w + g_at), ldh);
    }
    if ((dA || dB) && e == cudaSuccess && s == KS_OK) {
        grad[0].V = w + g_at;
        grad[1].V = w + h_at;
        e = grads(q, plan, grad, v_bf16, ldh, perm, offsets, batch, w + w_at);
    }
    if (e != cudaSuccess && s == KS_OK) s = cuda_fail(e, "adapter gradient launch");
    e = cudaFreeAsync(w, q.st);
    if (e != cudaSuccess && s == KS_OK) s = cuda_fail(e, "workspace free");
    return s;
}

}  // extern "C"
