// Device code shared by the kernels of the low-rank adapters (ks_adapter.cu,
// ks_adapter_rows.cu): element conversions, a row's adapter, and dot products of
// one row by a warp.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ks_internal.h"

namespace ks {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Elements of a 16-byte vector, as fp32.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[2 * q] = __uint_as_float(w[q] << 16);
        f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}

// The adapter of row n, -1 for none; an id past the adapters is reported.
__device__ __forceinline__ int row_adapter(const int *ids, long long n, long long N, int S, unsigned *status) {
    if (n >= N) return -1;
    const int s = ids ? ids[n] : 0;
    if (s >= S) {
        atomicOr(status, kDevBadIndex);
        return -1;
    }
    return s < 0 ? -1 : s;
}

// One or two products H = scale X W^T of the same rows (blockIdx.z picks one): W[s] is
// R x F; H, batch x ldh, and planes (TcAdapters::planes, plane_r ranks) may each be null.
struct ShrinkJob {
    const void *X, *W;
    void *H;
    unsigned short *planes;
    int F;
};
struct ShrinkArgs {
    ShrinkJob job[2];
    const float *scales;
    const int *ids;
    long long N;
    int R, ldh, S, plane_r;
    unsigned *status;
};

// Sums over F of x[f] w[r][f] for four ranks (w: F elements apart) by one warp;
// every lane gets them.  F a multiple of the vector, rows past `ranks` not read.
template <typename T>
__device__ __forceinline__ void dot4(const T *x, const T *w, int F, int ranks, int lane, float (&out)[4]) {
    constexpr int V = kVec<T>;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int f = lane * V; f < F; f += 32 * V) {
        float xf[V];
        unpack(__ldg(reinterpret_cast<const uint4 *>(x + f)), xf);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r < ranks) {
                float wf[V];
                unpack(__ldg(reinterpret_cast<const uint4 *>(w + (long long)r * F + f)), wf);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[r] = fmaf(xf[e], wf[e], acc[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[r] += __shfl_xor_sync(0xFFFFFFFFu, acc[r], o);
        out[r] = acc[r];
    }
}

// The same for any F and alignment.
template <typename T>
__device__ __forceinline__ void dot4_any(const T *x, const T *w, int F, int ranks, int lane, float (&out)[4]) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int f = lane; f < F; f += 32) {
        const float xf = to_f(x[f]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < ranks) acc[r] = fmaf(xf, to_f(w[(long long)r * F + f]), acc[r]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[r] += __shfl_xor_sync(0xFFFFFFFFu, acc[r], o);
        out[r] = acc[r];
    }
}

}  // namespace ks
