// Shared by the operators around the scan (ssd_norm.hip, ssd_conv.hip,
// ssd_step.hip, ssd_selscan.hip): row vectors of any alignment, wave sums,
// launch and argument checks, and the column sum that ends every weight
// gradient.  Internal.
#pragma once

#include "ssd_device.h"
#include "ssd.h"

namespace ssd {

// out0 | out1 | out2 (c0, c1 and the remaining columns) = sum over the rows of
// part [rows, cols], float32, in a fixed order.  Any out may be null.
struct ColSum {
    const float* part;
    int64_t rows, cols;
    float* out0;
    int64_t c0;
    float* out1;
    int64_t c1;
    float* out2;
};
int launch_colsum(const ColSum& p, hipStream_t s);

// With SSD_CHECK=1 in the environment: true, with the status, where cu_seqlens
// is not 0..T and non-decreasing (copies it to the host).  Else false.
bool check_cu_env(const int32_t* cu, int32_t nseq, int64_t T, hipStream_t s, int* status);

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 24;
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1;

constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;  // of a launch

inline size_t elem_size(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }
inline bool elem_aligned(const void* p, size_t e) { return ((uintptr_t)p & (e - 1)) == 0; }
inline int64_t imax(int64_t a, int64_t b) { return a > b ? a : b; }
__host__ __device__ inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// [a, a + na) and [b, b + nb) share bytes (NULL shares none).
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || !na || !nb) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

inline int launched() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

// V consecutive elements from an address aligned to one element, the first n
// of them valid (the rest read as 0).  A whole vector is one load of up to
// 16 bytes: the hardware takes it at any element alignment, so odd widths and
// strided views need no second path.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* __restrict__ p, int n, float (&o)[V]) {
    if (n >= V) {
        T t[V];
        __builtin_memcpy(t, p, sizeof(T) * V);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = (float)t[j];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = j < n ? (float)p[j] : 0.f;
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* __restrict__ p, int n, const float (&v)[V]) {
    if (n >= V) {
        T t[V];
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = (T)v[j];
        __builtin_memcpy(p, t, sizeof(T) * V);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < n) p[j] = (T)v[j];
    }
}

// The same in two steps: the bits first (a load in flight holds no more than
// them), their values later.
template <typename T, int V>
struct RawVec {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_raw(const T* __restrict__ p, int n, RawVec<T, V>& r) {
    if (n >= V) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) r.v[j] = j < n ? p[j] : (T)0.f;
    }
}

// Sum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float v) { return lane_value(wave_prefix_sum(v), 63); }

// 1 / (1 + e^-v), by the hardware exp2 and reciprocal (each within about one
// unit in the last place).  e^-v past the float range gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + fexp2(-v * kLog2e));
}

// softplus(z) = max(z, 0) + log(1 + v), v = e^-|z|.  A layer's steps are small, and
// their relative error is that of every u = d x and of the gradients: with
// s = v / (1 + v / 2), log(1 + v) = 2 atanh(s / 2) = s (1 + s^2 R(s^2)), where 1 + v,
// which drops v's low bits, is never formed.  R is a least-maximum fit for s <= 2/3
// (4.5e-9 of the whole; its first terms tend to 1/12, 1/80).  Steps of 0.016 to 0.03
// came 4e-6 off from the logarithm of 1 + v and come 4e-7 off here, for as many
// instructions.
__device__ __forceinline__ float step_softplus(float z) {
    const float v = fexp2(-fabsf(z) * kLog2e);
    const float s = v * __builtin_amdgcn_rcpf(fmaf(v, 0.5f, 1.f));
    const float q = s * s;
    const float r = fmaf(q, fmaf(q, fmaf(q, 5.471051e-4f, 2.187644e-3f), 1.2506727e-2f), 8.333302e-2f);
    return fmaxf(z, 0.f) + fmaf(s, q * r, s);
}

// A rate with -inf kept finite: times a step of 0 it would be NaN.  A comparison,
// not a maximum, which would give the number where the rate is NaN.
__device__ __forceinline__ float finite_rate(float a) { return a < -3e38f ? -3e38f : a; }

// d/dv of v sigmoid(v)
__device__ __forceinline__ float silu_slope(float v, float s) { return s * (1.f + v * (1.f - s)); }

// n % d, and n / d into *q; 32-bit where n allows.
__device__ __forceinline__ int64_t divide(int64_t n, int32_t d, int64_t* q) {
    if ((uint64_t)n >> 32 == 0) {
        const uint32_t k = (uint32_t)n / (uint32_t)d;
        *q = k;
        return (uint32_t)n - k * (uint32_t)d;
    }
    *q = n / d;
    return n % d;
}

// First index i in [0, n) with cu[i + 1] > t; n - 1 if there is none.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int n, int64_t t) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// Sequence i's tokens [first, last), kept inside [0, T) whatever cu holds.
__device__ __forceinline__ void sequence_span(const int32_t* cu, int i, int64_t L, int64_t T,
                                              int64_t* first, int64_t* last) {
    if (!cu) {
        *first = i * L;
        *last = *first + L;
        return;
    }
    const int64_t a = cu[i], b = cu[i + 1];
    *first = a < 0 ? 0 : (a > T ? T : a);
    *last = b < *first ? *first : (b > T ? T : b);
}

}  // namespace
}  // namespace ssd
