// Low-rank adapters of many requests beside one shared KS projection
// (ks_adapter_matmul) and their gradients (ks_adapter_backward):
//
//     H[n] = scale[s] X[n] A[s]^T,   Y[n] = act(X[n] K^T + bias + H[n] B[s]^T),   s = ids[n],
//     G[n] = scale[s] dY[n] B[s],    dX[n] = dY[n] K + G[n] A[s],
//     dA[s] = sum_{n: ids[n] = s} G[n]^T X[n],   dB[s] = sum_{n: ids[n] = s} dY[n]^T H[n],
//
// A[s] rank x in_features, B[s] out_features x rank.  A row whose id is negative
// takes no adapter; one whose id is n_adapters or more takes none either and
// raises kDevBadIndex in the device status word.  H and G are fp32; every sum is
// fp32 in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "ks_epilogue.cuh"
#include "ks_internal.h"

namespace ks {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ int adapter_of(const int *ids, long long n, int adapters, unsigned *status) {
    const int s = ids ? ids[n] : 0;
    if (s >= adapters) {
        atomicOr(status, kDevBadIndex);
        return -1;
    }
    return s < 0 ? -1 : s;
}

// H[n][r] = scale[s] sum_f X[n][f] W[s][r * rs + f * fs]; one warp per row.
template <typename T>
__global__ void __launch_bounds__(256)
    shrink_kernel(const T *__restrict__ X, const T *__restrict__ W, const float *__restrict__ scales,
                  const int *__restrict__ ids, float *__restrict__ H, long long N, int F, int R, int ldh, int S,
                  int rs, int fs, unsigned *status) {
    const int lane = threadIdx.x & 31;
    const long long n = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= N) return;
    const int s = adapter_of(ids, n, S, status);
    float *h = H + n * ldh;
    if (s < 0) {
        for (int r = lane; r < ldh; r += 32) h[r] = 0.f;
        return;
    }
    const T *x = X + n * F, *w = W + (long long)s * R * F;
    const float sc = scales ? scales[s] : 1.f;
    for (int r0 = 0; r0 < R; r0 += 8) {
        float acc[8] = {};
        for (int f = lane; f < F; f += 32) {
            const float xv = to_f(x[f]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (r0 + e < R) acc[e] = fmaf(xv, to_f(w[(long long)(r0 + e) * rs + (long long)f * fs]), acc[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int o = 16; o; o >>= 1) acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], o);
            if (lane == e && r0 + e < ldh) h[r0 + e] = r0 + e < R ? sc * acc[e] : 0.f;
        }
    }
}

// Y[n][f] = act(Y[n][f] + bias[f] + sum_r H[n][r] W[s][r * rs + f * fs]).
template <typename T>
__global__ void __launch_bounds__(256)
    expand_kernel(T *__restrict__ Y, const T *__restrict__ W, const int *__restrict__ ids, const float *__restrict__ H,
                  long long N, int F, int R, int ldh, int S, int rs, int fs, const T *__restrict__ bias, int act) {
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long n = at / F;
    if (n >= N) return;
    const int f = (int)(at - n * F);
    const int s = ids ? ids[n] : 0;
    float y = to_f(Y[at]);
    if (s >= 0 && s < S) {
        const T *w = W + (long long)s * R * F + (long long)f * fs;
        const float *h = H + n * ldh;
        float acc = 0.f;
        for (int r = 0; r < R; ++r) acc = fmaf(h[r], to_f(w[(long long)r * rs]), acc);
        y += acc;
    }
    put(Y + at, ep_apply(y, bias, f, act));
}

// The rows of each adapter in order: perm[offsets[s] .. offsets[s + 1]) holds the
// rows with id s.  Block s counts the rows of smaller ids and of its own, then
// writes its own in row order.
__global__ void __launch_bounds__(1024)
    order_kernel(const int *__restrict__ ids, int *__restrict__ perm, int *__restrict__ offsets, int N, int S) {
    __shared__ int warp_n[32];
    __shared__ int base_sh, total_sh;
    const int s = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int less = 0;
    for (int n = t; n < N; n += 1024) {
        const int id = ids[n];
        less += id >= 0 && id < s;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) less += __shfl_xor_sync(0xFFFFFFFFu, less, o);
    if (lane == 0) warp_n[warp] = less;
    __syncthreads();
    if (t == 0) {
        int b = 0;
        for (int w = 0; w < 32; ++w) b += warp_n[w];
        offsets[s] = b;
        base_sh = b;
    }
    __syncthreads();
    int base = base_sh;
    for (int n0 = 0; n0 < N; n0 += 1024) {
        const int n = n0 + t;
        const bool mine = n < N && ids[n] == s;
        const unsigned b = __ballot_sync(0xFFFFFFFFu, mine);
        if (lane == 0) warp_n[warp] = __popc(b);
        __syncthreads();
        if (warp == 0) {
            const int v = warp_n[lane];
            int sum = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += u;
            }
            warp_n[lane] = sum - v;
            if (lane == 31) total_sh = sum;
        }
        __syncthreads();
        if (mine) perm[base + warp_n[warp] + __popc(b & ((1u << lane) - 1))] = n;
        base += total_sh;
        __syncthreads();
    }
    if (s == S - 1 && t == 0) offsets[S] = base;
}

// out[s][r * rs + f * fs] = sum over the rows n of adapter s of P[n][f] Q[n][r].
template <typename T>
__global__ void __launch_bounds__(128)
    grad_kernel(const T *__restrict__ P, const float *__restrict__ Q, const int *__restrict__ perm,
                const int *__restrict__ offsets, T *__restrict__ out, int N, int F, int R, int ldh, int rs, int fs) {
    const int f = blockIdx.x * 128 + threadIdx.x, s = blockIdx.y, r0 = blockIdx.z * 8;
    if (f >= F) return;
    const int begin = offsets ? offsets[s] : 0, end = offsets ? offsets[s + 1] : N;
    float acc[8] = {};
    for (int k = begin; k < end; ++k) {
        const long long n = perm ? perm[k] : k;
        const float x = to_f(P[n * F + f]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (r0 + e < R) acc[e] = fmaf(x, Q[n * ldh + r0 + e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (r0 + e < R) put(out + (long long)s * R * F + (long long)(r0 + e) * rs + (long long)f * fs, acc[e]);
}

struct Adapters {
    const void *A, *B;
    const float *scales;
    const int *ids;
    int S, R, ldh;
    bool bf16;
    cudaStream_t st;
};

// W[s][r][f] at r * rs + f * fs: A is rank x in, B is out x rank
cudaError_t shrink(const Adapters &q, const void *X, bool with_a, long long N, int F, float *H) {
    const int rs = with_a ? F : 1, fs = with_a ? 1 : q.R;
    const unsigned grid = (unsigned)((N + 7) / 8);
    if (q.bf16)
        shrink_kernel<__nv_bfloat16><<<grid, 256, 0, q.st>>>(
            static_cast<const __nv_bfloat16 *>(X), static_cast<const __nv_bfloat16 *>(with_a ? q.A : q.B), q.scales,
            q.ids, H, N, F, q.R, q.ldh, q.S, rs, fs, device_status_ptr());
    else
        shrink_kernel<float><<<grid, 256, 0, q.st>>>(static_cast<const float *>(X),
                                                     static_cast<const float *>(with_a ? q.A : q.B), q.scales, q.ids,
                                                     H, N, F, q.R, q.ldh, q.S, rs, fs, device_status_ptr());
    return cudaGetLastError();
}

cudaError_t expand(const Adapters &q, void *Y, bool with_a, long long N, int F, const float *H, const void *bias,
                   int act) {
    const int rs = with_a ? F : 1, fs = with_a ? 1 : q.R;
    const unsigned grid = (unsigned)((N * F + 255) / 256);
    if (q.bf16)
        expand_kernel<__nv_bfloat16><<<grid, 256, 0, q.st>>>(
            static_cast<__nv_bfloat16 *>(Y), static_cast<const __nv_bfloat16 *>(with_a ? q.A : q.B), q.ids, H, N, F,
            q.R, q.ldh, q.S, rs, fs, static_cast<const __nv_bfloat16 *>(bias), act);
    else
        expand_kernel<float><<<grid, 256, 0, q.st>>>(static_cast<float *>(Y),
                                                     static_cast<const float *>(with_a ? q.A : q.B), q.ids, H, N, F,
                                                     q.R, q.ldh, q.S, rs, fs, static_cast<const float *>(bias), act);
    return cudaGetLastError();
}

cudaError_t grad(const Adapters &q, const void *P, const float *Q, const int *perm, const int *offsets, void *out,
                 bool with_a, long long N, int F) {
    const int rs = with_a ? F : 1, fs = with_a ? 1 : q.R;
    const dim3 grid((unsigned)((F + 127) / 128), (unsigned)q.S, (unsigned)((q.R + 7) / 8));
    if (q.bf16)
        grad_kernel<__nv_bfloat16><<<grid, 128, 0, q.st>>>(static_cast<const __nv_bfloat16 *>(P), Q, perm, offsets,
                                                           static_cast<__nv_bfloat16 *>(out), (int)N, F, q.R, q.ldh,
                                                           rs, fs);
    else
        grad_kernel<float><<<grid, 128, 0, q.st>>>(static_cast<const float *>(P), Q, perm, offsets,
                                                   static_cast<float *>(out), (int)N, F, q.R, q.ldh, rs, fs);
    return cudaGetLastError();
}

constexpr int kMaxAdapters = 65535, kMaxRank = 1024;

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
    if (batch > INT32_MAX / 2) return record_error(KS_ERR_INVALID_ARG, "adapters take at most 2^30 rows");
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

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

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
    if ((s = check_align(bias, o.elem, "bias")) != KS_OK) return s;
    if (bias && ranges_overlap(Y, batch * o.out_f * o.elem, bias, o.out_f * o.elem))
        return record_error(KS_ERR_INVALID_ARG, "Y overlaps bias");
    // The product checks X, values and Y; the adapters, the bias and the
    // activation are added to it.  In bf16 the product is rounded before they are.
    if ((s = ks_matmul(X, values, a, b, c, d, batch, Y, dtype, stream)) != KS_OK) return s;
    const Adapters q{A, B, scales, ids, (int)n_adapters, (int)rank, (int)(rank + 3) / 4 * 4, dtype == KS_BF16,
                     static_cast<cudaStream_t>(stream)};
    char *w = nullptr;
    if ((s = alloc(&w, (size_t)batch * q.ldh * 4, q.st)) != KS_OK) return s;
    float *H = reinterpret_cast<float *>(w);
    cudaError_t e = shrink(q, X, true, batch, (int)o.in_f, H);
    if (e == cudaSuccess) e = expand(q, Y, false, batch, (int)o.out_f, H, bias, activation);
    if (e != cudaSuccess) s = cuda_fail(e, "adapter launch");
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
    const Adapters q{A, B, scales, ids, (int)n_adapters, (int)rank, (int)(rank + 3) / 4 * 4, dtype == KS_BF16,
                     static_cast<cudaStream_t>(stream)};
    if (batch == 0) {  // empty sums
        cudaError_t e = cudaSuccess;
        if (dA) e = cudaMemsetAsync(dA, 0, (size_t)o.abytes, q.st);
        if (e == cudaSuccess && dB) e = cudaMemsetAsync(dB, 0, (size_t)o.bbytes, q.st);
        return e == cudaSuccess ? KS_OK : cuda_fail(e, "gradient clear");
    }
    if (!dY || ((dA || dB) && !X) || (dX && !values))
        return record_error(KS_ERR_INVALID_ARG, "dY, X (for dA and dB) and values (for dX) must be non-null");
    if ((s = check_align(dY, o.elem, "dY")) != KS_OK || (s = check_align(X, o.elem, "X")) != KS_OK) return s;
    if (dX && (s = ks_matmul_dx(dY, values, a, b, c, d, batch, dX, dtype, stream)) != KS_OK) return s;
    if (!dX && !dA && !dB) return KS_OK;
    const size_t hb = up256((size_t)batch * q.ldh * 4);
    const size_t pb = up256((size_t)batch * 4), ob = up256((size_t)(q.S + 1) * 4);
    char *w = nullptr;
    if ((s = alloc(&w, 2 * hb + pb + ob, q.st)) != KS_OK) return s;
    float *G = reinterpret_cast<float *>(w), *H = reinterpret_cast<float *>(w + hb);
    int *perm = reinterpret_cast<int *>(w + 2 * hb), *offsets = reinterpret_cast<int *>(w + 2 * hb + pb);
    cudaError_t e = cudaSuccess;
    const auto then = [&](cudaError_t r) { if (e == cudaSuccess) e = r; };
    if (dX || dA) then(shrink(q, dY, false, batch, (int)o.out_f, G));
    if (dX && e == cudaSuccess) then(expand(q, dX, true, batch, (int)o.in_f, G, nullptr, KS_ACT_NONE));
    if ((dA || dB) && ids && e == cudaSuccess) {
        order_kernel<<<(unsigned)q.S, 1024, 0, q.st>>>(ids, perm, offsets, (int)batch, q.S);
        then(cudaGetLastError());
    }
    if (!ids) perm = offsets = nullptr;
    if (dA && e == cudaSuccess) then(grad(q, X, G, perm, offsets, dA, true, batch, (int)o.in_f));
    if (dB && e == cudaSuccess) {
        then(shrink(q, X, true, batch, (int)o.in_f, H));
        if (e == cudaSuccess) then(grad(q, dY, H, perm, offsets, dB, false, batch, (int)o.out_f));
    }
    if (e != cudaSuccess) s = cuda_fail(e, "adapter gradient launch");
    e = cudaFreeAsync(w, q.st);
    if (e != cudaSuccess && s == KS_OK) s = cuda_fail(e, "workspace free");
    return s;
}

}  // extern "C"
