// Adapters beside a KS product for few rows (single tokens of some requests): one
// launch computes, for a few rows and a range of output columns a block,
//
//     h[r] = scale sum_f A[s][r][f] x[f],    y = act(sum_j values[i,l,k,j] x[i,j,l] + bias + sum_r B[s][col][r] h[r]).
//
// Such a call is bound by latency and by reading the weights once, so there are no
// tiles to fill: the blocks are as many as the SMs can hold, every one computes
// the h that it needs by itself (A[s] is read again by each block of a row, from
// L2) instead of waiting for another launch, and a values row is read by
// neighbouring lanes as 16-byte vectors for all rows of the block.  fp32 sums, one
// rounding.  GPT-2-shaped bf16 layer, rank 16, bias and GELU: 6.1 us for one row, 14 us for 32 rows
// of 32 adapters, against 28 and 81 us of the tile kernels.
//
// h can also come from memory (shrink_rows_kernel, one warp for four ranks of a
// row): where A[s] is large, reading it in every block costs more than a launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ks_adapter.cuh"
#include "ks_epilogue.cuh"
#include "ks_internal.h"

namespace ks {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSmem = 96 * 1024;       // dynamic shared memory of a block at most
constexpr int kDefaultSmem = 48 * 1024;   // without opting in, rows_kernel's own `sid` included

// H[n][r] = scale[s] sum_f X[n][f] W[s][r][f], r < ldh (zeros past R and for rows without an adapter).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) shrink_rows_kernel(const __grid_constant__ ShrinkArgs p) {
    const ShrinkJob &job = p.job[blockIdx.z];
    const T *__restrict__ const X = static_cast<const T *>(job.X);
    const T *__restrict__ const W = static_cast<const T *>(job.W);
    float *__restrict__ const H = static_cast<float *>(job.H);
    const float *const scales = p.scales;
    const int F = job.F, R = p.R, ldh = p.ldh;
    const int lane = threadIdx.x & 31, quads = (ldh + 3) / 4;
    const long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long n = task / quads;
    if (n >= p.N) return;
    const int r0 = (int)(task - n * quads) * 4;
    const int s = row_adapter(p.ids, n, p.N, p.S, p.status);
    float h[4] = {0.f, 0.f, 0.f, 0.f};
    if (s >= 0 && r0 < R) {
        const T *x = X + n * F, *w = W + ((long long)s * R + r0) * F;
        if constexpr (VEC)
            dot4(x, w, F, R - r0, lane, h);
        else
            dot4_any(x, w, F, R - r0, lane, h);
        const float sc = scales ? scales[s] : 1.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = r0 + r < R ? h[r] * sc : 0.f;
    }
    if (lane < 4 && r0 + lane < ldh) {
        const float v = lane == 0 ? h[0] : lane == 1 ? h[1] : lane == 2 ? h[2] : h[3];
        H[n * ldh + r0 + lane] = v;
    }
}

struct RowsParams {
    const void *X, *V, *bias, *A, *B;
    const float *scales, *H;  // H: null, or batch x ldh
    const int *ids;
    void *Y;
    long long N;
    int a, b, c, d, in_f, out_f, R, ldh, S, act;
    int cols;          // of a block
    int lanes_log2;    // lanes of a values row: 1 << lanes_log2
    int pitch;         // elements of a row of x in shared memory, [i][l][j]
    int x_rows;        // rows (i, l) of x in shared memory
    int x_bytes;       // of all rows of x there
    int a_vec, b_vec;  // rows of x and A, of B are whole aligned vectors
    unsigned *status;
};

// RB rows of a block; blockIdx.x: columns, blockIdx.y: rows.  VEC: rows of the values are
// whole aligned vectors.
template <typename T, int RB, bool VEC>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowsParams p) {
    constexpr int V = kVec<T>;
    extern __shared__ __align__(16) uint8_t smem[];
    T *const xs = reinterpret_cast<T *>(smem);  // [RB][x_rows][pitch]
    float *const ys = reinterpret_cast<float *>(smem + p.x_bytes);  // [RB][cols]
    float *const hs = ys + RB * p.cols;                                                              // [RB][ldh]
    __shared__ int sid[RB];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long n0 = (long long)blockIdx.y * RB;
    const int col0 = blockIdx.x * p.cols, cols = min(p.cols, p.out_f - col0);
    const T *const X = static_cast<const T *>(p.X), *const A = static_cast<const T *>(p.A);
    if (tid < RB) sid[tid] = row_adapter(p.ids, n0 + tid, p.N, p.S, p.status);
    // x of the blocks i that the columns belong to, [i][j][l] -> [i][l][j]
    const int bd = p.b * p.d, cd = p.c * p.d;
    const int i0 = col0 / bd, ni = (col0 + cols - 1) / bd - i0 + 1;
#pragma unroll
    for (int m = 0; m < RB; ++m) {
        if (n0 + m >= p.N) break;
        const T *src = X + (n0 + m) * p.in_f + (long long)i0 * cd;
        T *dst = xs + (size_t)m * p.x_rows * p.pitch;
        if (VEC && p.d % V == 0) {
            for (int e = tid * V; e < ni * cd; e += kThreads * V) {
                const int i = e / cd, j = (e - i * cd) / p.d, l = (e - i * cd) - j * p.d;
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src + e));
                const T *v = reinterpret_cast<const T *>(&w);
#pragma unroll
                for (int q = 0; q < V; ++q) dst[(i * p.d + l + q) * p.pitch + j] = v[q];
            }
        } else {
            for (int e = tid; e < ni * cd; e += kThreads) {
                const int i = e / cd, j = (e - i * cd) / p.d, l = (e - i * cd) - j * p.d;
                dst[(i * p.d + l) * p.pitch + j] = src[e];
            }
        }
    }
    __syncthreads();
    // h
    if (p.H) {
        for (int q = tid; q < RB * p.ldh; q += kThreads) {
            const long long n = n0 + q / p.ldh;
            if (n < p.N) hs[q] = p.H[n * p.ldh + q % p.ldh];
        }
    } else {
        const int quads = p.ldh / 4;
        for (int q = warp; q < RB * quads; q += kThreads / 32) {
            const int m = q / quads, r0 = (q - m * quads) * 4, s = sid[m];
            if (s < 0) continue;
            float h[4];
            const T *x = X + (n0 + m) * p.in_f, *w = A + ((long long)s * p.R + r0) * p.in_f;
            if (p.a_vec)
                dot4(x, w, p.in_f, p.R - r0, lane, h);
            else
                dot4_any(x, w, p.in_f, p.R - r0, lane, h);
            const float sc = p.scales ? p.scales[s] : 1.f;
            if (lane < 4) {
                const float v = lane == 0 ? h[0] : lane == 1 ? h[1] : lane == 2 ? h[2] : h[3];
                hs[m * p.ldh + r0 + lane] = v * sc;
            }
        }
    }
    // the KS product: 1 << lanes_log2 lanes a column
    {
        const int lanes = 1 << p.lanes_log2, sub = lane & (lanes - 1), per_warp = 32 >> p.lanes_log2;
        const T *const Vp = static_cast<const T *>(p.V);
        for (int e0 = warp * per_warp; e0 < cols; e0 += kThreads / 32 * per_warp) {
            const int e = e0 + (lane >> p.lanes_log2);
            const int col = col0 + min(e, cols - 1);
            const int i = col / bd, k = (col - i * bd) / p.d, l = (col - i * bd) - k * p.d;
            const T *v = Vp + ((long long)(i * p.d + l) * p.b + k) * p.c;
            const T *x = xs + ((i - i0) * p.d + l) * p.pitch;
            float acc[RB];
#pragma unroll
            for (int m = 0; m < RB; ++m) acc[m] = 0.f;
            if constexpr (VEC) {
#pragma unroll 2
                for (int j = sub * V; j < p.c; j += lanes * V) {
                    float vf[V];
                    unpack(__ldg(reinterpret_cast<const uint4 *>(v + j)), vf);
#pragma unroll
                    for (int m = 0; m < RB; ++m) {
                        float xf[V];
                        unpack(*reinterpret_cast<const uint4 *>(x + (size_t)m * p.x_rows * p.pitch + j), xf);
#pragma unroll
                        for (int q = 0; q < V; ++q) acc[m] = fmaf(vf[q], xf[q], acc[m]);
                    }
                }
            } else {
#pragma unroll 4
                for (int j = sub; j < p.c; j += lanes) {
                    const float vf = to_f(v[j]);
#pragma unroll
                    for (int m = 0; m < RB; ++m)
                        acc[m] = fmaf(vf, to_f(x[(size_t)m * p.x_rows * p.pitch + j]), acc[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < RB; ++m) {
                for (int o = lanes >> 1; o; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
                if (sub == 0 && e < cols) ys[m * p.cols + e] = acc[m];
            }
        }
    }
    __syncthreads();
    const T *const B = static_cast<const T *>(p.B), *const bias = static_cast<const T *>(p.bias);
    for (int q = tid; q < RB * cols; q += kThreads) {
        const int m = q / cols, e = q - m * cols, s = sid[m];
        const long long n = n0 + m;
        if (n >= p.N) break;
        float y = ys[m * p.cols + e];
        if (s >= 0) {
            const T *w = B + ((long long)s * p.out_f + col0 + e) * p.R;
            const float *h = hs + m * p.ldh;
            float acc = 0.f;
            if (p.b_vec) {
                for (int r = 0; r < p.R; r += V) {
                    float wf[V];
                    unpack(__ldg(reinterpret_cast<const uint4 *>(w + r)), wf);
#pragma unroll
                    for (int z = 0; z < V; ++z) acc = fmaf(wf[z], h[r + z], acc);
                }
            } else {
                for (int r = 0; r < p.R; ++r) acc = fmaf(to_f(w[r]), h[r], acc);
            }
            y += acc;
        }
        put(static_cast<T *>(p.Y) + n * p.out_f + col0 + e, ep_apply(y, bias, col0 + e, p.act));
    }
}

struct RowsPlan {
    bool vec;
    int rb, cols, lanes_log2, pitch, x_rows, tiles;
    size_t x_bytes, smem;
};

// Blocks for about two a SM (at least 32 columns each: one values row for each
// warp's group of lanes), more rows of a block as the batch grows.
bool rows_plan(const Problem &p, int ldh, RowsPlan *o) {
    const int es = p.elem_bytes();
    const uintptr_t al = reinterpret_cast<uintptr_t>(p.X) | reinterpret_cast<uintptr_t>(p.V);
    o->vec = p.c % (16 / es) == 0 && al % 16 == 0;
    const int vec = o->vec ? 16 / es : 1;
    const int out_f = (int)p.out_features();
    for (o->rb = p.batch >= 16 ? 4 : p.batch >= 4 ? 2 : 1; o->rb >= 1; o->rb /= 2) {
        const long long groups = (p.batch + o->rb - 1) / o->rb;
        const long long want = std::max<long long>(1, 2LL * sm_count() / groups);
        o->cols = (int)std::min<long long>(1024, std::max<long long>(32, ((out_f + want - 1) / want + 31) / 32 * 32));
        o->tiles = (out_f + o->cols - 1) / o->cols;
        int lanes = 0;
        while ((vec << lanes) < p.c && lanes < 5) ++lanes;
        o->lanes_log2 = lanes;
        // rows of 16-byte units, an odd number of them for c a power of two
        o->pitch = o->vec ? (int)p.c + vec : (int)p.c | 1;
        const long long i_n = std::min<long long>(p.a, (o->cols - 1) / (p.b * p.d) + 2);
        o->x_rows = (int)std::min<long long>(i_n * p.d, 1 << 20);
        o->x_bytes = (o->rb * (size_t)o->x_rows * o->pitch * es + 15) / 16 * 16;
        const double smem = (double)o->x_bytes + (double)o->rb * (o->cols + ldh) * 4;
        if (smem <= kMaxSmem) {
            o->smem = (size_t)smem;
            return true;
        }
    }
    return false;
}

}  // namespace

bool adapter_rows_supported(const Problem &p, int ldh) {
    // About 5 us and 1 us for each 1.9M products in bf16, 0.5M in fp32, 0.2M without vectors,
    // against 38 to 48 us of the bf16 tiles, 20 to 30 of the fp32 ones and 18 to 25 of odd layers'
    // (GPT-2-shaped bf16, rank 16: 128 rows 29 and 48 us, 256 rows 53 and 47; fp32, rank 8: 16 rows
    // 14 and 19, 64 rows 29 and 22).
    const long long work = p.batch * p.out_features() * (p.c + ldh);
    if (p.dtype == KS_TF32 || p.batch > 256 || work > (p.dtype == KS_BF16 ? 50LL : 11LL) * 1000000) return false;
    RowsPlan o;
    return rows_plan(p, ldh, &o) && (o.vec || work <= 4000000);
}

cudaError_t launch_shrink_rows(const ShrinkArgs &p, int jobs, bool bf16, bool vec, cudaStream_t st) {
    const dim3 grid((unsigned)((p.N * ((p.ldh + 3) / 4) + 7) / 8), 1, (unsigned)jobs);
    const auto go = [&](auto kernel) {
        kernel<<<grid, 256, 0, st>>>(p);
        return cudaGetLastError();
    };
    if (!bf16) return vec ? go(shrink_rows_kernel<float, true>) : go(shrink_rows_kernel<float, false>);
    return vec ? go(shrink_rows_kernel<__nv_bfloat16, true>) : go(shrink_rows_kernel<__nv_bfloat16, false>);
}

cudaError_t launch_adapter_rows(const Problem &pr, const void *A, const void *B, const float *scales, const int *ids,
                                int S, int R, const float *H, int ldh) {
    RowsPlan o;
    if (!rows_plan(pr, ldh, &o)) return cudaErrorInvalidConfiguration;
    RowsParams p{};
    p.X = pr.X, p.V = pr.V, p.bias = pr.bias, p.A = A, p.B = B, p.scales = scales, p.H = H, p.ids = ids, p.Y = pr.Y;
    p.N = pr.batch, p.act = pr.act;
    p.a = (int)pr.a, p.b = (int)pr.b, p.c = (int)pr.c, p.d = (int)pr.d;
    p.in_f = (int)pr.in_features(), p.out_f = (int)pr.out_features();
    p.R = R, p.ldh = ldh, p.S = S;
    p.cols = o.cols, p.lanes_log2 = o.lanes_log2, p.pitch = o.pitch, p.x_rows = o.x_rows;
    p.x_bytes = (int)o.x_bytes;
    p.a_vec = (reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(pr.X)) % 16 == 0 &&
              p.in_f * pr.elem_bytes() % 16 == 0;
    p.b_vec = reinterpret_cast<uintptr_t>(B) % 16 == 0 && R * pr.elem_bytes() % 16 == 0;
    p.status = device_status_ptr();
    const dim3 grid((unsigned)o.tiles, (unsigned)((pr.batch + o.rb - 1) / o.rb));
    const auto go = [&](auto kernel) {
        // (the limit is the function's, for all host threads: one that every call sets to the same value)
        if (o.smem + 4 * sizeof(int) > kDefaultSmem) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
            if (e != cudaSuccess) return e;
        }
        kernel<<<grid, kThreads, o.smem, pr.stream>>>(p);
        return cudaGetLastError();
    };
    const auto typed = [&](auto t) {
        using T = decltype(t);
        if (o.vec)
            return o.rb == 4   ? go(rows_kernel<T, 4, true>)
                   : o.rb == 2 ? go(rows_kernel<T, 2, true>)
                               : go(rows_kernel<T, 1, true>);
        return o.rb == 4   ? go(rows_kernel<T, 4, false>)
               : o.rb == 2 ? go(rows_kernel<T, 2, false>)
                           : go(rows_kernel<T, 1, false>);
    };
    return pr.dtype == KS_BF16 ? typed(__nv_bfloat16{}) : typed(float{});
}

}  // namespace ks
