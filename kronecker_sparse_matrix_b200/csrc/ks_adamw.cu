// AdamW over many tensors in one launch (ks_adamw_step): with decoupled weight
// decay, for each element of each tensor
//
//     m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2,
//     p = p (1 - lr wd) - (lr / (1 - beta1^t)) m / (sqrt(v) / sqrt(1 - beta2^t) + eps),
//
// the states m and v in fp32, or in 8 bits: m and sqrt(v) as e4m3 numbers times
// one fp32 scale for each 256 consecutive elements of a tensor (the largest
// magnitude of the 256 is 448, e4m3's largest number).  Holding sqrt(v) instead
// of v squares the range that a block can span: an element is kept down to
// 2^-9/448 of the block's largest sqrt(v).  A positive sqrt(v) is never held as
// zero (the smallest e4m3 number stands for it), so no step divides by eps
// alone because of the format.  A block whose largest magnitude is below 2^-100
// is held as zeros (448 / top would leave the fp32 range).  One whose largest magnitude
// is infinite (in v: also that of a gradient whose square leaves the fp32 range) is held as NaN.
//
// The step needs p, g, m and v read and p, m and v written once: 28 bytes per
// fp32 element with fp32 states, 10.06 bytes per bf16 element with 8-bit ones.
//
// One block of 256 threads takes 2048 consecutive elements of one tensor at a time,
// a warp 256 of them (one scale's worth), a lane eight.  The tensors of a launch
// and the prefix sums of their blocks travel in the kernel's parameters, so a step
// over many tensors is one launch, with no table to copy to the device; a block
// finds its tensor by bisection.  Arithmetic runs on pairs (fp32x2).
//
// Roundings: m and v are each two products and a sum, every one rounded to
// nearest.  The square root of an 8-bit state and the reciprocal in the update are the
// hardware's approximations (a few units in the last place of fp32), far inside
// half a step of e4m3 and the rounding of p.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "ks_internal.h"

namespace ks {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 256;                  // elements of a scale: one warp's
constexpr int kChunk = kThreads / 32 * kBlock;  // elements that a thread block takes at a time
// units of a warp in a large step (142M bf16 parameters with 8-bit states, before blend: 286
// us with 4, 276 us with 8; 49M with masters and fp32 states: 218 and 221 us)
constexpr int kIters8 = 8, kIters32 = 4;
constexpr float kTop = 448.f;                // largest e4m3 number
constexpr float kLow = 0.001953125f;         // 2^-9, the smallest positive one
constexpr float kNone = 7.888609052210118e-31f;  // 2^-100

struct Hyper {
    float lr, beta1, omb1, beta2, omb2, eps, wd, one;
    float bc1, inv_root_bc2;  // 1 - beta1^t and 1 / sqrt(1 - beta2^t), when step is null
    double log_beta1, log_beta2;
    const long long *step;    // device step number, or null
    const float *lr_dev;      // device learning rate, or null
    const float *grad_scale;  // device factor of the gradients, or null
};

template <int NT>
struct Table {
    void *p[NT];
    const void *g[NT];
    void *m[NT];
    void *v[NT];
    float *master[NT];
    float *ms[NT];
    float *vs[NT];
    long long n[NT];
    int first[NT + 1];  // first thread block of each tensor
    unsigned char aligned[NT];
    int count, iters;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float *o) { *o = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(x); }

__device__ __forceinline__ float code_value(unsigned char c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
__device__ __forceinline__ unsigned char value_code(float x) {
    return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// Eight elements of a lane: consecutive (vectors), or 32 apart.
__device__ __forceinline__ void load8(const float *s, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(s)[0], b = reinterpret_cast<const float4 *>(s)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *s, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(s);
    const unsigned w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(w[q] << 16);
        v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const unsigned char *s, float (&v)[8]) {
    const uint2 a = *reinterpret_cast<const uint2 *>(s);
    const unsigned w[2] = {a.x, a.y};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[q >> 1] >> (16 * (q & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * q] = f.x;
        v[2 * q + 1] = f.y;
    }
}
__device__ __forceinline__ void store8(float *d, const float (&v)[8]) {
    reinterpret_cast<float4 *>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *d, const float (&v)[8]) {
    unsigned w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
        w[q] = *reinterpret_cast<const unsigned *>(&h);
    }
    *reinterpret_cast<uint4 *>(d) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(unsigned char *d, const float (&v)[8]) {
    unsigned w[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q >> 1] |= (unsigned)__nv_cvt_float2_to_fp8x2(make_float2(v[2 * q], v[2 * q + 1]), __NV_SATFINITE,
                                                        __NV_E4M3)
                     << (16 * (q & 1));
    *reinterpret_cast<uint2 *>(d) = make_uint2(w[0], w[1]);
}
template <typename S>
__device__ __forceinline__ float load1(const S *s) {
    if constexpr (sizeof(S) == 1)
        return code_value(*s);
    else
        return to_f(*s);
}
template <typename S>
__device__ __forceinline__ void store1(S *d, float x) {
    if constexpr (sizeof(S) == 1)
        *d = value_code(x);
    else
        from_f(x, d);
}
// `left` elements remain from s on: fewer than 256, or unaligned buffers
template <typename S>
__device__ __forceinline__ void load8(const S *s, float (&v)[8], bool vec, int lane, long long left) {
    if (vec) {
        load8(s + lane * 8, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = lane + 32 * e < left ? load1(s + lane + 32 * e) : 0.f;
    }
}
template <typename S>
__device__ __forceinline__ void store8(S *d, const float (&v)[8], bool vec, int lane, long long left) {
    if (vec) {
        store8(d + lane * 8, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (lane + 32 * e < left) store1(d + lane + 32 * e, v[e]);
    }
}

// Largest magnitude of the warp's 256 elements (NaN elements do not count:
// each keeps its own NaN code), zero below 2^-100.  The bits of floats that are
// not negative are ordered like the floats.
__device__ __forceinline__ float warp_top(const float (&v)[8]) {
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = fmaxf(t, fabsf(v[e]));
    t = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(t)));
    return t < kNone ? 0.f : t;
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 448 / top: the reciprocal to within one rounding by a Newton step, its residual exact
// by the FMA.  (With the bare approximation more elements fell to the other side of a tie
// between two codes than rounding alone puts there.)  NaN for an infinite top.  `top` is
// below 2^126 or infinite: the reciprocal of a larger number is subnormal, which the
// approximation flushes.
__device__ __forceinline__ float codes_per(float top) {
    const float r = rcp_approx(top);
    return fmaf(fmaf(-r, top, 1.f), r, r) * kTop;
}

// x a + y b of pairs, both products and the sum rounded.  The sum is an FMA by a one that
// the compiler does not know: it contracts a product and a sum of pairs into one FMA, and
// codes of m near a tie then differ from those of the formula as written.  142M bf16
// parameters with 8-bit states: 302 us, contracted 257; fp32 states: no difference.
__device__ __forceinline__ float2 blend(float2 x, float2 a, float2 y, float2 b, float2 one) {
    return __ffma2_rn(__fmul2_rn(x, a), one, __fmul2_rn(y, b));
}

// T: type of p and g; S: type of the states (float, or unsigned char: e4m3).
template <typename T, typename S, bool MASTER, int NT>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<NT> t, const Hyper h) {
    constexpr bool S8 = sizeof(S) == 1;
    const int block = (int)blockIdx.x;
    int lo = 0, hi = t.count;  // first[lo] <= block < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= block)
            lo = mid;
        else
            hi = mid;
    }
    const int lane = threadIdx.x & 31;
    float lr = h.lr, bc1 = h.bc1, ib2 = h.inv_root_bc2;
    if (h.lr_dev) lr = *h.lr_dev;
    if (h.step) {
        const double s = (double)*h.step;
        bc1 = -expm1f((float)(s * h.log_beta1));
        ib2 = rsqrtf(-expm1f((float)(s * h.log_beta2)));
    }
    const float gs = h.grad_scale ? *h.grad_scale : 1.f;
    const float2 keep = make_float2(1.f - lr * h.wd, 1.f - lr * h.wd), rate = make_float2(-lr / bc1, -lr / bc1);
    const float2 b1 = make_float2(h.beta1, h.beta1), o1 = make_float2(h.omb1, h.omb1);
    const float2 b2 = make_float2(h.beta2, h.beta2), o2 = make_float2(h.omb2, h.omb2);
    const float2 one = make_float2(h.one, h.one);
    const float2 gs2 = make_float2(gs, gs), ib = make_float2(ib2, ib2), eps = make_float2(h.eps, h.eps);
    const long long n = t.n[lo];
    const bool vectors = t.aligned[lo];
    // Units of the block: its warps side by side, iters times over.  Their scales
    // are read and written as one piece: stores of single scales, 4 bytes of a
    // sector that other warps are reading, made the step up to 1.5x slower.
    constexpr int kWarps = kThreads / 32;
    __shared__ float scales[S8 ? 2 : 1][S8 ? kWarps * kIters8 : 1];
    const long long unit0 = (long long)(block - t.first[lo]) * (kWarps * t.iters);
    const int units = (int)min((long long)kWarps * t.iters, (n + kBlock - 1) / kBlock - unit0);
    if constexpr (S8) {
        if ((int)threadIdx.x < units) {
            scales[0][threadIdx.x] = t.ms[lo][unit0 + threadIdx.x];
            scales[1][threadIdx.x] = t.vs[lo][unit0 + threadIdx.x];
        }
        __syncthreads();
    }
    for (int u = threadIdx.x >> 5; u < units; u += kWarps) {
        const long long at = (unit0 + u) * kBlock;
        const long long left = n - at;
        const bool vec = vectors && left >= kBlock;
        T *p = static_cast<T *>(t.p[lo]) + at;
        const T *g = static_cast<const T *>(t.g[lo]) + at;
        S *m = static_cast<S *>(t.m[lo]) + at;
        S *v = static_cast<S *>(t.v[lo]) + at;
        float *w = MASTER ? t.master[lo] + at : nullptr;

        float pe[8], ge[8], me[8], ve[8];
        load8(g, ge, vec, lane, left);
        load8(m, me, vec, lane, left);
        load8(v, ve, vec, lane, left);
        if constexpr (MASTER)
            load8(w, pe, vec, lane, left);
        else
            load8(p, pe, vec, lane, left);
        float2 m_scale, v_scale;
        if constexpr (S8) {
            m_scale.x = m_scale.y = scales[0][u];
            v_scale.x = v_scale.y = scales[1][u];
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 gr = __fmul2_rn(make_float2(ge[e], ge[e + 1]), gs2);
            float2 m0 = make_float2(me[e], me[e + 1]), v0 = make_float2(ve[e], ve[e + 1]);
            if constexpr (S8) {
                m0 = __fmul2_rn(m0, m_scale);
                v0 = __fmul2_rn(v0, v_scale);
                v0 = __fmul2_rn(v0, v0);
            }
            const float2 m1 = blend(m0, b1, gr, o1, one);
            const float2 v1 = blend(v0, b2, __fmul2_rn(gr, gr), o2, one);
            float2 root;
            if constexpr (S8)
                root = make_float2(sqrt_approx(v1.x), sqrt_approx(v1.y));
            else
                root = make_float2(__fsqrt_rn(v1.x), __fsqrt_rn(v1.y));
            const float2 den = __ffma2_rn(root, ib, eps);
            const float2 change = __fmul2_rn(m1, make_float2(rcp_approx(den.x), rcp_approx(den.y)));
            const float2 p1 = __ffma2_rn(rate, change, __fmul2_rn(make_float2(pe[e], pe[e + 1]), keep));
            pe[e] = p1.x, pe[e + 1] = p1.y;
            me[e] = m1.x, me[e + 1] = m1.y;
            ve[e] = S8 ? root.x : v1.x, ve[e + 1] = S8 ? root.y : v1.y;
        }
        if constexpr (MASTER) store8(w, pe, vec, lane, left);
        store8(p, pe, vec, lane, left);
        if constexpr (S8) {
            const float m_top = warp_top(me), v_top = warp_top(ve);
            // (m can be as large as a gradient: 448 / m_top as 28 / (m_top / 16))
            const float m_inv = m_top == 0.f ? 0.f : codes_per(m_top * (1.f / 16.f)) * (1.f / 16.f);
            const float v_inv = v_top == 0.f ? 0.f : codes_per(v_top);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                me[e] *= m_inv;
                const float y = ve[e] * v_inv;
                ve[e] = ve[e] > 0.f ? fmaxf(y, kLow) : y;
            }
            if (lane == 0) {  // (the warp's reductions above come after every lane's reads)
                scales[0][u] = m_top * (1.f / kTop);
                scales[1][u] = fmaf(v_inv, 0.f, v_top * (1.f / kTop));  // NaN with v_inv, for codes that fmaxf made kLow
            }
        }
        store8(m, me, vec, lane, left);
        store8(v, ve, vec, lane, left);
    }
    if constexpr (S8) {
        __syncthreads();
        if ((int)threadIdx.x < units) {
            t.ms[lo][unit0 + threadIdx.x] = scales[0][threadIdx.x];
            t.vs[lo][unit0 + threadIdx.x] = scales[1][threadIdx.x];
        }
    }
}

bool is_aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename T, typename S, bool MASTER, int NT>
cudaError_t launch_table(const ks_adamw_tensor *ts, int count, int iters, const Hyper &h, cudaStream_t st) {
    Table<NT> t;
    t.count = count;
    t.iters = iters;
    long long blocks = 0;
    for (int k = 0; k < count; ++k) {
        const ks_adamw_tensor &q = ts[k];
        t.p[k] = q.param, t.g[k] = q.grad, t.m[k] = q.exp_avg, t.v[k] = q.exp_avg_sq;
        t.master[k] = q.master, t.ms[k] = q.exp_avg_scale, t.vs[k] = q.exp_avg_sq_scale, t.n[k] = q.n;
        t.first[k] = (int)blocks;
        // eight elements of a lane as 16-byte (fp32: two) or 8-byte (e4m3) vectors
        t.aligned[k] = is_aligned(q.param, 16) && is_aligned(q.grad, 16) && is_aligned(q.exp_avg, 16) &&
                       is_aligned(q.exp_avg_sq, 16) && is_aligned(q.master, 16);
        blocks += (q.n + (long long)kChunk * iters - 1) / ((long long)kChunk * iters);
    }
    t.first[count] = (int)blocks;
    adamw_kernel<T, S, MASTER, NT><<<(unsigned)blocks, kThreads, 0, st>>>(t, h);
    return cudaGetLastError();
}

// Launches of at most kMany tensors and 2^31 - 1 blocks.  The parameter block of
// a launch is copied with it, so few tensors take a small one.
constexpr int kFew = 16, kSome = 96, kMany = 400;
constexpr long long kMaxBlocks = 0x7FFFFFFFll;

template <typename T, typename S, bool MASTER>
cudaError_t launch_all(const std::vector<ks_adamw_tensor> &ts, const Hyper &h, cudaStream_t st) {
    size_t k = 0;
    while (k < ts.size()) {
        long long blocks = 0;
        size_t e = k;
        while (e < ts.size() && e - k < (size_t)kMany) {
            const long long b = (ts[e].n + kChunk - 1) / kChunk;
            if (e > k && blocks + b > kMaxBlocks) break;
            blocks += b;
            ++e;
        }
        const int count = (int)(e - k);
        // several units a warp where that leaves eight blocks and more for each SM:
        // finding the tensor and the step's numbers are then paid once for them
        constexpr int many = sizeof(S) == 1 ? kIters8 : kIters32;
        const int iters = blocks >= 8LL * many * sm_count() ? many : 1;
        const cudaError_t err = count <= kFew    ? launch_table<T, S, MASTER, kFew>(&ts[k], count, iters, h, st)
                                : count <= kSome ? launch_table<T, S, MASTER, kSome>(&ts[k], count, iters, h, st)
                                                 : launch_table<T, S, MASTER, kMany>(&ts[k], count, iters, h, st);
        if (err != cudaSuccess) return err;
        k = e;
    }
    return cudaSuccess;
}

struct Range {
    uintptr_t begin, end;
    bool written;
};

// Whether a written buffer shares bytes with any other of the step's buffers.  The
// buffers come in columns (all params, all grads, ..), which are mostly in the order
// of their addresses already: each is sorted if need be, and they are merged.
constexpr int kColumns = 8;
bool any_overlap(std::vector<Range> (&col)[kColumns]) {
    const auto before = [](const Range &x, const Range &y) { return x.begin < y.begin; };
    size_t at[kColumns] = {};
    for (auto &c : col)
        if (!std::is_sorted(c.begin(), c.end(), before)) std::sort(c.begin(), c.end(), before);
    uintptr_t end_read = 0, end_written = 0;
    while (true) {
        int k = -1;
        uintptr_t least = UINTPTR_MAX;
        for (int j = 0; j < kColumns; ++j)
            if (at[j] < col[j].size() && col[j][at[j]].begin < least) {
                least = col[j][at[j]].begin;
                k = j;
            }
        if (k < 0) return false;
        const Range &q = col[k][at[k]++];
        if (q.begin < end_written || (q.written && q.begin < end_read)) return true;
        (q.written ? end_written : end_read) = std::max(q.written ? end_written : end_read, q.end);
    }
}

ks_status adamw_step(const ks_adamw_tensor *tensors, int64_t n_tensors, int dtype, int state_bits,
                     const ks_adamw_options *opt, void *stream) {
    if (dtype != KS_F32 && dtype != KS_BF16)
        return record_error(KS_ERR_INVALID_ARG, "parameters are fp32 or bf16 (dtype %d)", dtype);
    if (state_bits != 8 && state_bits != 32)
        return record_error(KS_ERR_INVALID_ARG, "state_bits must be 8 or 32 (got %d)", state_bits);
    if (!opt) return record_error(KS_ERR_INVALID_ARG, "options must be non-null");
    if (n_tensors < 0 || (n_tensors > 0 && !tensors))
        return record_error(KS_ERR_INVALID_ARG, "need n_tensors >= 0 and non-null tensors");
    const auto unit = [](double b) { return b >= 0.0 && b < 1.0; };  // false for NaN
    if (!unit(opt->beta1) || !unit(opt->beta2))
        return record_error(KS_ERR_INVALID_ARG, "betas must be in [0, 1) (got %g, %g)", opt->beta1, opt->beta2);
    if (!(opt->eps >= 0.0) || !std::isfinite(opt->eps) || !(opt->weight_decay >= 0.0) ||
        !std::isfinite(opt->weight_decay))
        return record_error(KS_ERR_INVALID_ARG, "eps and weight_decay must be finite and not negative");
    if (!opt->lr_ptr && (!(opt->lr >= 0.0) || !std::isfinite(opt->lr)))
        return record_error(KS_ERR_INVALID_ARG, "lr must be finite and not negative (got %g)", opt->lr);
    if (!opt->step_ptr && opt->step < 1)
        return record_error(KS_ERR_INVALID_ARG, "step counts from 1 (got %lld)", (long long)opt->step);
    if (!is_aligned(opt->lr_ptr, 4) || !is_aligned(opt->grad_scale, 4) || !is_aligned(opt->step_ptr, 8))
        return record_error(KS_ERR_MISALIGNED, "lr_ptr, grad_scale or step_ptr is not aligned to its element");
    const uintptr_t elem = dtype == KS_BF16 ? 2 : 4, selem = state_bits == 8 ? 1 : 4;
    std::vector<ks_adamw_tensor> ts;
    std::vector<Range> ranges[kColumns];
    ts.reserve((size_t)n_tensors);
    for (auto &c : ranges) c.reserve((size_t)n_tensors + 3);
    bool masters = false;
    for (int64_t k = 0; k < n_tensors; ++k) {
        const ks_adamw_tensor &q = tensors[k];
        if (q.n < 0 || q.n > (int64_t)kMaxBlocks * 16)
            return record_error(KS_ERR_INVALID_ARG, "tensor %lld: bad element count %lld", (long long)k,
                                (long long)q.n);
        if (q.n == 0) continue;
        if (!q.param || !q.grad || !q.exp_avg || !q.exp_avg_sq)
            return record_error(KS_ERR_INVALID_ARG, "tensor %lld: param, grad and states must be non-null",
                                (long long)k);
        if (state_bits == 8 && (!q.exp_avg_scale || !q.exp_avg_sq_scale))
            return record_error(KS_ERR_INVALID_ARG, "tensor %lld: 8-bit states need their scales", (long long)k);
        if (ts.empty()) {
            masters = q.master != nullptr;
        } else if (masters != (q.master != nullptr)) {
            return record_error(KS_ERR_INVALID_ARG, "tensor %lld: masters for all tensors or for none", (long long)k);
        }
        if (q.master && dtype != KS_BF16)
            return record_error(KS_ERR_INVALID_ARG, "tensor %lld: masters are for bf16 parameters", (long long)k);
        if (!is_aligned(q.param, elem) || !is_aligned(q.grad, elem) || !is_aligned(q.exp_avg, selem) ||
            !is_aligned(q.exp_avg_sq, selem) || !is_aligned(q.master, 4) || !is_aligned(q.exp_avg_scale, 4) ||
            !is_aligned(q.exp_avg_sq_scale, 4))
            return record_error(KS_ERR_MISALIGNED, "tensor %lld: a buffer is not aligned to its element",
                                (long long)k);
        const auto add = [&](int column, const void *p, uintptr_t bytes, bool written) {
            if (p) ranges[column].push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, written});
        };
        const uintptr_t n = (uintptr_t)q.n, blocks = (n + kBlock - 1) / kBlock;
        add(0, q.param, n * elem, true);
        add(1, q.grad, n * elem, false);
        add(2, q.exp_avg, n * selem, true);
        add(3, q.exp_avg_sq, n * selem, true);
        add(4, q.master, n * 4, true);
        if (state_bits == 8) {
            add(5, q.exp_avg_scale, blocks * 4, true);
            add(6, q.exp_avg_sq_scale, blocks * 4, true);
        }
        ts.push_back(q);
    }
    if (ts.empty()) return KS_OK;
    const auto scalar = [&](const void *p, uintptr_t bytes) {
        if (p) ranges[7].push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, false});
    };
    scalar(opt->lr_ptr, 4);
    scalar(opt->grad_scale, 4);
    scalar(opt->step_ptr, 8);
    if (any_overlap(ranges))
        return record_error(KS_ERR_INVALID_ARG, "a parameter or state overlaps another buffer of the step");
    Hyper h{};
    h.lr = (float)opt->lr;
    h.beta1 = (float)opt->beta1, h.omb1 = (float)(1.0 - opt->beta1);
    h.beta2 = (float)opt->beta2, h.omb2 = (float)(1.0 - opt->beta2);
    h.eps = (float)opt->eps, h.wd = (float)opt->weight_decay, h.one = 1.f;
    h.bc1 = (float)(1.0 - std::pow(opt->beta1, (double)opt->step));
    h.inv_root_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(opt->beta2, (double)opt->step)));
    h.log_beta1 = std::log(opt->beta1), h.log_beta2 = std::log(opt->beta2);  // -inf for 0: 1 - 0^t = 1
    h.step = reinterpret_cast<const long long *>(opt->step_ptr);
    h.lr_dev = opt->lr_ptr;
    h.grad_scale = opt->grad_scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (state_bits == 32)
        e = dtype == KS_F32 ? launch_all<float, float, false>(ts, h, st)
            : masters       ? launch_all<__nv_bfloat16, float, true>(ts, h, st)
                            : launch_all<__nv_bfloat16, float, false>(ts, h, st);
    else
        e = dtype == KS_F32 ? launch_all<float, unsigned char, false>(ts, h, st)
            : masters       ? launch_all<__nv_bfloat16, unsigned char, true>(ts, h, st)
                            : launch_all<__nv_bfloat16, unsigned char, false>(ts, h, st);
    if (e != cudaSuccess)
        return record_error(KS_ERR_CUDA, "AdamW launch: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return KS_OK;
}

}  // namespace
}  // namespace ks

extern "C" ks_status ks_adamw_step(const ks_adamw_tensor *tensors, int64_t n_tensors, int dtype, int state_bits,
                                   const ks_adamw_options *options, void *stream) {
    try {
        return ks::adamw_step(tensors, n_tensors, dtype, state_bits, options, stream);
    } catch (...) {  // host memory for the tables
        return ks::record_error(KS_ERR_ALLOC, "host memory for %lld tensors", (long long)n_tensors);
    }
}
