// Layer norm, forward and backward, and the column sum behind every weight
// gradient of the library.
//
//   mean = sum x / W, rstd = 1 / sqrt(sum (x - mean)^2 / W + eps)
//   y = (x - mean) rstd w + b
// and with xh = (x - mean) rstd, q = dy w:
//   dx = rstd (q - mean(q) - xh mean(q xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// Both directions are bound by HBM: one pass, the row held in registers
// between the sums and the output (but for the widths named at kMostFwd), so x
// (and dy) is read once.  A row belongs to one wave where it fits (no barrier),
// else to one workgroup.
#include "ssd_layer.h"

namespace ssd {
namespace {

constexpr int kMaxWaves = 16;   // per row
constexpr int64_t kMaxGrid = ((int64_t)1 << 22) - 1;  // of 1024 threads
constexpr int kWavesPerWg = 4;  // rows of a workgroup where a row is one wave's

struct NormParams {
    const void* x;
    const void* dy;
    void* out;  // y or dx
    const float* weight;
    const float* bias;
    float* mean;
    float* rstd;
    const float* mean_in;
    const float* rstd_in;
    float* part;  // [slots][2][width]
    int64_t rows, x_row, out_row, dy_row;
    int32_t width;
    int32_t slots;  // row walkers (waves or workgroups) of the backward launch
    float eps;
};

// Sums over the row's lanes of two values; `waves` waves share a row (1: no
// barrier).  The exchange is double-buffered by `turn`, so one barrier a call
// is enough: a wave can be at most one call ahead.
__device__ __forceinline__ void row_sums(float& a, float& b, int waves, float (*ex)[kMaxWaves][2],
                                         int& turn) {
    a = wave_sum(a);
    b = wave_sum(b);
    if (waves == 1) return;
    float (*e)[2] = ex[turn];
    turn ^= 1;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        e[w][0] = a;
        e[w][1] = b;
    }
    __syncthreads();
    a = b = 0.f;
    for (int i = 0; i < waves; ++i) {
        a += e[i][0];
        b += e[i][1];
    }
}

// Vector i of a row's thread: V elements from c, of which the first `skip`
// belong to another vector too (the last one is moved back to end with the row,
// a thread without elements takes the last vector and skips all of it).  They
// are left out of the row's sums; what is written for them is the same twice.
template <int V>
struct Piece {
    int c, skip;
    __device__ __forceinline__ Piece(int i, int lanes, int lane, int width) {
        const int at = (i * lanes + lane) * V;
        c = min(at, width - V);
        skip = min(at - c, V);
    }
    __device__ __forceinline__ bool any() const { return skip < V; }
};

// V elements a load, NV loads a thread.
template <typename T, int V, int NV>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormParams p, int waves) {
    __shared__ float ex[2][kMaxWaves][2];
    const int lanes = waves * 64;
    const int per = waves == 1 ? kWavesPerWg : 1;
    int64_t row = (int64_t)blockIdx.x * per + (waves == 1 ? threadIdx.x >> 6 : 0);
    const int lane = waves == 1 ? threadIdx.x & 63 : threadIdx.x;
    int turn = 0;
    // one row, but for more rows than a launch may have threads
    for (; row < p.rows; row += (int64_t)gridDim.x * per) {
        const T* x = (const T*)p.x + row * p.x_row;
        T* y = (T*)p.out + row * p.out_row;
        RawVec<T, V> raw[NV];
        float v[NV][V];
        float s = 0.f, zero = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            load_raw<T, V>(x + Piece<V>(i, lanes, lane, p.width).c, V, raw[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Piece<V> q(i, lanes, lane, p.width);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] = (float)raw[i].v[j];
                s += j >= q.skip ? v[i][j] : 0.f;
            }
        }
        row_sums(s, zero, waves, ex, turn);
        const float mean = s / (float)p.width;
        float sq = 0.f;
        zero = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Piece<V> q(i, lanes, lane, p.width);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] -= mean;
                sq += j >= q.skip ? v[i][j] * v[i][j] : 0.f;
            }
        }
        row_sums(sq, zero, waves, ex, turn);
        const float rstd = 1.f / sqrtf(sq / (float)p.width + p.eps);
        if (lane == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Piece<V> q(i, lanes, lane, p.width);
            float w[V], b[V], o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                w[j] = 1.f;
                b[j] = 0.f;
            }
            if (p.weight) load_vec<float, V>(p.weight + q.c, V, w);
            if (p.bias) load_vec<float, V>(p.bias + q.c, V, b);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = v[i][j] * rstd * w[j] + b[j];
            if (q.any()) store_vec<T, V>(y + q.c, V, o);
        }
    }
}

// Each walker (wave or workgroup) takes the rows slot, slot + slots, ... and
// keeps its share of dw and db in registers until its last row.
template <typename T, int V, int NV>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormParams p, int waves) {
    __shared__ float ex[2][kMaxWaves][2];
    const int lanes = waves * 64;
    const int slot = waves == 1 ? blockIdx.x * kWavesPerWg + (threadIdx.x >> 6) : blockIdx.x;
    if (slot >= p.slots) return;  // only where a row is one wave's: no barrier below
    const int lane = waves == 1 ? threadIdx.x & 63 : threadIdx.x;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Piece<V> q(i, lanes, lane, p.width);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = 1.f;
            dw[i][j] = db[i][j] = 0.f;
        }
        if (p.weight) load_vec<float, V>(p.weight + q.c, V, w[i]);
    }
    int turn = 0;
    const float inv = 1.f / (float)p.width;
    // the next row is on its way while this one's sums are formed, where the
    // registers of 16 waves hold both
    constexpr bool kAhead = V * NV <= 8;
    RawVec<T, V> xr[NV], gr[NV];
    float mean_r = 0.f, rstd_r = 0.f;
    auto fetch = [&](int64_t row) {
        const T* x = (const T*)p.x + row * p.x_row;
        const T* dy = (const T*)p.dy + row * p.dy_row;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Piece<V> q(i, lanes, lane, p.width);
            load_raw<T, V>(x + q.c, V, xr[i]);
            load_raw<T, V>(dy + q.c, V, gr[i]);
        }
        mean_r = p.mean_in[row];
        rstd_r = p.rstd_in[row];
    };
    if (kAhead && slot < p.rows) fetch(slot);
    for (int64_t row = slot; row < p.rows; row += p.slots) {
        if (!kAhead) fetch(row);
        const float mean = mean_r, rstd = rstd_r;
        float v[NV][V], g[NV][V];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] = (float)xr[i].v[j];
                g[i][j] = (float)gr[i].v[j];
            }
        if (kAhead) fetch(row + p.slots < p.rows ? row + p.slots : row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Piece<V> q(i, lanes, lane, p.width);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] = (v[i][j] - mean) * rstd;
                dw[i][j] += g[i][j] * v[i][j];
                db[i][j] += g[i][j];
                g[i][j] *= w[i][j];
                s0 += j >= q.skip ? g[i][j] : 0.f;
                s1 += j >= q.skip ? g[i][j] * v[i][j] : 0.f;
            }
        }
        row_sums(s0, s1, waves, ex, turn);
        s0 *= inv;
        s1 *= inv;
        T* dx = (T*)p.out + row * p.out_row;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Piece<V> q(i, lanes, lane, p.width);
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = rstd * (g[i][j] - s0 - v[i][j] * s1);
            if (q.any()) store_vec<T, V>(dx + q.c, V, o);
        }
    }
    float* pw = p.part + (int64_t)slot * 2 * p.width;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Piece<V> q(i, lanes, lane, p.width);
        if (q.any()) {
            store_vec<float, V>(pw + q.c, V, dw[i]);
            store_vec<float, V>(pw + p.width + q.c, V, db[i]);
        }
    }
}

// Sixteen waves a workgroup, each adding every sixteenth row of 64 columns;
// the waves' sums are joined in LDS.
__global__ __launch_bounds__(1024) void colsum_kernel(ColSum p) {
    __shared__ float ex[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < p.cols) {
        const float* q = p.part + c;
        int64_t r = w;
        for (; r + 7 * 16 < p.rows; r += 8 * 16) {
            float t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = q[(r + k * 16) * p.cols];
#pragma unroll
            for (int k = 0; k < 8; ++k) s += t[k];
        }
        for (; r < p.rows; r += 16) s += q[r * p.cols];
    }
    ex[w][lane] = s;
    __syncthreads();
    if (w || c >= p.cols) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += ex[k][lane];
    if (c < p.c0) {
        if (p.out0) p.out0[c] = s;
    } else if (c < p.c0 + p.c1) {
        if (p.out1) p.out1[c - p.c0] = s;
    } else if (p.out2) {
        p.out2[c - p.c0 - p.c1] = s;
    }
}

// Waves a row and loads a thread: the fewest waves that hold the row with at
// most `most` loads a thread.
struct NormPlan {
    int waves, nv;
};
// Elements a load: 16 bytes, or one where a row is shorter.
int norm_vec(const ssd_norm_dims& d) {
    const int V = d.dtype == SSD_BF16 ? 8 : 4;
    return d.width >= V ? V : 1;
}
NormPlan norm_plan(const ssd_norm_dims& d, int most) {
    const int64_t vecs = cdiv(d.width, norm_vec(d));
    NormPlan pl;
    const int64_t w = cdiv(vecs, 64 * most);
    pl.waves = (int)w;
    pl.nv = (int)cdiv(vecs, 64 * w);
    return pl;
}
// Forward, at most 8 loads a lane against at most 4, us for 6e7 elements (at 5.0 TB/s
// bf16 takes 48, float32 96):
//   width            2560  3328  4096  6144  8192 12288 16384
//   bf16, 8            47    62    81    50    83    85    84
//   bf16, 4            53    54    52    51    51    57    57
//   float32, 8         92    91    90    92    93    98    96
//   float32, 4         88    88    86    88    88    94   110
// The kernel is compiled for 1024 threads, 128 registers; 7 or 8 loads of 8 bf16 elements
// do not fit, and 40 and 100 bytes a lane go through scratch memory.
constexpr int kMostFwd = 8;
// backward: one load of 8 or two of 4 elements of x and dy (then the next row is
// loaded ahead); more where 16 waves do not span the row
inline int most_bwd(const ssd_norm_dims& d) {
    const int V = norm_vec(d), least = 8 / V;
    const int64_t need = cdiv(d.width, (int64_t)V * 64 * kMaxWaves);
    return need > least ? (int)need : least;
}

int32_t norm_slots(const ssd_norm_dims& d) {
    // Ten waves a CU.  Fewer walkers leave loads unhidden, more only write
    // more shares (8192 x 2560 bf16, 5 waves: 256 walkers 38 us, 512 to 768
    // 32, 1024 38; 2400 x 16384 float32, 16 waves: 256 walkers 114, 512 126,
    // 1024 141); and none takes fewer than four rows.
    const NormPlan pl = norm_plan(d, most_bwd(d));
    const int64_t by_waves = imax(256, 2560 / pl.waves), most = by_waves < 2048 ? by_waves : 2048;
    const int64_t s = imax(1, cdiv(d.rows, 4));
    return (int32_t)(s < most ? s : most);
}

int norm_check(const ssd_norm_dims* d) {
    if (!d) return SSD_ERR_NULL_ARG;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->rows < 0 || d->rows > kMaxTokens || d->width < 1) return SSD_ERR_SHAPE;
    if (d->width > SSD_NORM_MAX_WIDTH) return SSD_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f)) return SSD_ERR_SHAPE;
    for (int64_t s : {d->x_row, d->y_row, d->dy_row})
        if (s < d->width || s > kMaxStride) return SSD_ERR_SHAPE;
    return SSD_OK;
}

template <typename T, int V, bool BWD>
void launch_norm(const NormParams& p, NormPlan pl, hipStream_t s) {
    const int64_t walkers = BWD ? p.slots : p.rows;
    const int64_t wgs = pl.waves == 1 ? cdiv(walkers, kWavesPerWg) : walkers;
    const dim3 grid((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid));
    const dim3 block(pl.waves == 1 ? 64 * kWavesPerWg : 64 * pl.waves);
    if constexpr (V == 1) {  // rows of fewer elements than a vector: one load
        if constexpr (BWD) norm_bwd_kernel<T, 1, 1><<<grid, block, 0, s>>>(p, pl.waves);
        else norm_fwd_kernel<T, 1, 1><<<grid, block, 0, s>>>(p, pl.waves);
    } else {
#define SSD_NORM_CASE(NV)                                                       \
    case NV:                                                                    \
        if constexpr (!BWD) norm_fwd_kernel<T, V, NV><<<grid, block, 0, s>>>(p, pl.waves); \
        else if constexpr (NV * V <= 16) norm_bwd_kernel<T, V, NV><<<grid, block, 0, s>>>(p, pl.waves); \
        break
    switch (pl.nv) {
        SSD_NORM_CASE(1);
        SSD_NORM_CASE(2);
        SSD_NORM_CASE(3);
        SSD_NORM_CASE(4);
        SSD_NORM_CASE(5);
        SSD_NORM_CASE(6);
        SSD_NORM_CASE(7);
        SSD_NORM_CASE(8);
    }
    }
#undef SSD_NORM_CASE
}
template <bool BWD>
void launch_norm(const ssd_norm_dims& d, const NormParams& p, NormPlan pl, hipStream_t s) {
    if (d.dtype == SSD_BF16) {
        if (norm_vec(d) == 1) launch_norm<bf16, 1, BWD>(p, pl, s);
        else launch_norm<bf16, 8, BWD>(p, pl, s);
    } else {
        if (norm_vec(d) == 1) launch_norm<float, 1, BWD>(p, pl, s);
        else launch_norm<float, 4, BWD>(p, pl, s);
    }
}

}  // namespace

int launch_colsum(const ColSum& p, hipStream_t s) {
    if (p.cols <= 0) return SSD_OK;
    colsum_kernel<<<dim3((unsigned)cdiv(p.cols, 64)), dim3(1024), 0, s>>>(p);
    return launched();
}

}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_norm_fwd(const ssd_norm_dims* dims, const void* x, const float* weight, const float* bias,
                 void* y, float* mean, float* rstd, void* stream) {
    const int st = norm_check(dims);
    if (st != SSD_OK) return st;
    if (dims->rows == 0) return SSD_OK;
    if (!x || !y) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(dims->dtype);
    if (!elem_aligned(x, e) || !elem_aligned(y, e) || !elem_aligned(weight, 4) ||
        !elem_aligned(bias, 4) || !elem_aligned(mean, 4) || !elem_aligned(rstd, 4))
        return SSD_ERR_ALIGN;
    NormParams p = {};
    p.x = x;
    p.out = y;
    p.weight = weight;
    p.bias = bias;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = dims->rows;
    p.x_row = dims->x_row;
    p.out_row = dims->y_row;
    p.width = dims->width;
    p.eps = dims->eps;
    const NormPlan pl = norm_plan(*dims, kMostFwd);
    launch_norm<false>(*dims, p, pl, (hipStream_t)stream);
    return launched();
}

size_t ssd_norm_bwd_workspace_bytes(const ssd_norm_dims* dims) {
    if (norm_check(dims) != SSD_OK) return 0;
    return up256((size_t)norm_slots(*dims) * 2 * dims->width * sizeof(float));
}

int ssd_norm_bwd(const ssd_norm_dims* dims, const void* x, const float* weight, const float* mean,
                 const float* rstd, const void* dy, void* dx, float* dweight, float* dbias,
                 void* workspace, size_t workspace_bytes, void* stream) {
    const int st = norm_check(dims);
    if (st != SSD_OK) return st;
    if (dims->rows > 0 && (!x || !mean || !rstd || !dy || !dx)) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(dims->dtype);
    if (!elem_aligned(x, e) || !elem_aligned(dy, e) || !elem_aligned(dx, e) ||
        !elem_aligned(weight, 4) || !elem_aligned(mean, 4) || !elem_aligned(rstd, 4) ||
        !elem_aligned(dweight, 4) || !elem_aligned(dbias, 4) || ((uintptr_t)workspace & 255))
        return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < ssd_norm_bwd_workspace_bytes(dims))
        return SSD_ERR_WORKSPACE;
    NormParams p = {};
    p.x = x;
    p.dy = dy;
    p.out = dx;
    p.weight = weight;
    p.mean_in = mean;
    p.rstd_in = rstd;
    p.part = (float*)workspace;
    p.rows = dims->rows;
    p.x_row = dims->x_row;
    p.out_row = dims->x_row;
    p.dy_row = dims->dy_row;
    p.width = dims->width;
    p.slots = norm_slots(*dims);  // with no rows one walker, which writes zeros
    const NormPlan pl = norm_plan(*dims, most_bwd(*dims));
    launch_norm<true>(*dims, p, pl, (hipStream_t)stream);
    const int rc = launched();
    if (rc != SSD_OK || (!dweight && !dbias)) return rc;
    ColSum c = {};
    c.part = p.part;
    c.rows = p.slots;
    c.cols = 2 * (int64_t)dims->width;
    c.out0 = dweight;
    c.c0 = dims->width;
    c.out1 = dbias;
    c.c1 = dims->width;
    return launch_colsum(c, (hipStream_t)stream);
}

}  // extern "C"
