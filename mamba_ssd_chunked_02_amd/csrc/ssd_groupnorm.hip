// Group norm, channels last, with an activation; forward and backward.
//
// x [n, P, C]: a sample's statistics run over its P positions and the D = C / G channels of
// each group (P = 1: every row's groups on their own, the norm of a layer's heads):
//   mean = sum x / (P D),  rstd = 1 / sqrt(sum (x - mean)^2 / (P D) + eps)
//   xh = (x - mean) rstd,  u = xh w + b,  y = u | silu(u) | u silu(z)
// and with du = dL/du (from dy through the activation), g = du w:
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum du xh,  db = sum du,  dz = dy u silu'(z).
//
// Both are bound by memory.  P = 1: a group is D consecutive elements, LG lanes take it (64 /
// LG groups a wave) and hold it in registers between the sums and the output: one pass.
// P > 1: statistics of runs of positions (one pass over x), and a second pass for the output,
// which joins them first and which the caches serve as far as they hold x.
//
// Reached (what a copy of 1 GiB reaches is 5.16 TB/s): 8192 x 16 groups of 128, gated, gradients
// (168 MB) 34 us, 4.9 TB/s; 4096 x 12 groups of 128, gated (38 MB) 10 us in the kernel, 3.8 TB/s;
// 8 maps of 4096 x 320 (42 MB) 23 us in two launches, the second of which joins the runs behind a
// cold read of what other XCDs wrote, a third of its time.  A group that one wave cannot hold (over
// 2048 channels in bf16, 1024 in float32) takes the launches of P > 1 with P = 1: 4096 x 4096 in one
// group, bf16, 121 us, six times what its bytes take.
#include "ssd_layer.h"

namespace ssd {
namespace {

enum { PLAIN = SSD_ACT_NONE, SILU = SSD_ACT_SILU, GATE = SSD_ACT_GATE };

struct GnParams {
    const void* x;
    const void* z;
    const void* dy;
    void* out;  // y or dx
    void* dz;
    const float* weight;
    const float* bias;
    float* mean;
    float* rstd;
    const float* mean_in;
    const float* rstd_in;
    float* part;  // columns' sums of the runs [n][runs][2][C]
    float* of_runs;  // groups' sums of the runs [n][runs][2][G], where a workgroup spans the channels
    float* sums;  // groups' sums over their runs [n][G][2], where it does not
    int64_t n, P;
    int64_t x_n, x_p, z_n, z_p, y_n, y_p, dy_n, dy_p;  // strides of samples and positions
    int64_t runlen;
    int32_t C, G, D, runs, walkers;
    float eps;
};

// A launch's units of work lie along x, and along z where there are more than kAlong.
constexpr int64_t kAlong = (int64_t)1 << 20;
__device__ __forceinline__ int64_t unit() { return (int64_t)blockIdx.z * gridDim.x + blockIdx.x; }
dim3 units(int64_t n, int64_t y = 1) {
    const int64_t x = n < kAlong ? n : kAlong;
    return dim3((unsigned)x, (unsigned)y, (unsigned)cdiv(n, x));
}

// u's value through the activation, z where it has a gate
template <int ACT>
__device__ __forceinline__ float activate(float u, float z) {
    if (ACT == SILU) return u * sigmoid(u);
    if (ACT == GATE) return u * (z * sigmoid(z));
    return u;
}
// dL/du from dy, and dL/dz
template <int ACT>
__device__ __forceinline__ float slope(float dy, float u, float z, float& dz) {
    if (ACT == SILU) return dy * silu_slope(u, sigmoid(u));
    if (ACT == GATE) {
        const float s = sigmoid(z);
        dz = dy * u * silu_slope(z, s);
        return dy * (z * s);
    }
    return dy;
}

// Sum over LG consecutive lanes (a power of two), in each of them.
template <int LG>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < LG; o *= 2) v += __shfl_xor(v, o);
    return v;
}

// ---- P = 1 ---------------------------------------------------------------------------------

// LG lanes x NV vectors of V elements hold one group of a row.  The last vector is moved back
// to end with the group; the elements it shares (`skip`) are left out of the sums and stored
// twice with the same value.
template <int V>
struct Cell {
    int c, skip;
    __device__ __forceinline__ Cell(int i, int lanes, int lane, int D) {
        const int at = (i * lanes + lane) * V;
        c = min(at, D - V);
        skip = min(at - c, V);
    }
};

template <typename T, int V, int NV, int LG, int ACT>
__global__ __launch_bounds__(256) void gn_row_fwd(GnParams p) {
    const int64_t id = (unit() * 256 + threadIdx.x) / LG;
    const int lane = threadIdx.x % LG;
    if (id >= p.n * p.G) return;  // whole groups of lanes
    int64_t row;
    const int g = (int)divide(id, p.G, &row);
    const int c0 = g * p.D;
    const T* x = (const T*)p.x + row * p.x_n + c0;
    const T* z = (const T*)p.z + row * p.z_n + c0;
    T* y = (T*)p.out + row * p.y_n + c0;
    RawVec<T, V> xr[NV], zr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Cell<V> q(i, LG, lane, p.D);
        load_raw<T, V>(x + q.c, V, xr[i]);
        if (ACT == GATE) load_raw<T, V>(z + q.c, V, zr[i]);
    }
    float v[NV][V], s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Cell<V> q(i, LG, lane, p.D);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[i][j] = (float)xr[i].v[j];
            s += j >= q.skip ? v[i][j] : 0.f;
        }
    }
    const float mean = lanes_sum<LG>(s) / (float)p.D;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Cell<V> q(i, LG, lane, p.D);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[i][j] -= mean;
            s += j >= q.skip ? v[i][j] * v[i][j] : 0.f;
        }
    }
    const float rstd = 1.f / sqrtf(lanes_sum<LG>(s) / (float)p.D + p.eps);
    if (lane == 0) {
        if (p.mean) p.mean[id] = mean;
        if (p.rstd) p.rstd[id] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Cell<V> q(i, LG, lane, p.D);
        float w[V], b[V], o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[j] = 1.f;
            b[j] = 0.f;
        }
        if (p.weight) load_vec<float, V>(p.weight + c0 + q.c, V, w);
        if (p.bias) load_vec<float, V>(p.bias + c0 + q.c, V, b);
#pragma unroll
        for (int j = 0; j < V; ++j)
            o[j] = activate<ACT>(v[i][j] * rstd * w[j] + b[j], ACT == GATE ? (float)zr[i].v[j] : 0.f);
        if (q.skip < V) store_vec<T, V>(y + q.c, V, o);
    }
}

// A walker (LG lanes) keeps one group of channels and takes the rows walker, walker +
// walkers, ...; its share of dw and db stays in registers until its last row.
template <typename T, int V, int NV, int LG, int ACT>
__global__ __launch_bounds__(256) void gn_row_bwd(GnParams p) {
    const int64_t id = (unit() * 256 + threadIdx.x) / LG;
    const int lane = threadIdx.x % LG;
    if (id >= (int64_t)p.walkers * p.G) return;
    int64_t walker;
    const int g = (int)divide(id, p.G, &walker);
    const int c0 = g * p.D;
    float w[NV][V], b[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Cell<V> q(i, LG, lane, p.D);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = 1.f;
            b[i][j] = dw[i][j] = db[i][j] = 0.f;
        }
        if (p.weight) load_vec<float, V>(p.weight + c0 + q.c, V, w[i]);
        if (ACT != PLAIN && p.bias) load_vec<float, V>(p.bias + c0 + q.c, V, b[i]);
    }
    const float inv = 1.f / (float)p.D;
    for (int64_t row = walker; row < p.n; row += p.walkers) {
        const T* x = (const T*)p.x + row * p.x_n + c0;
        const T* z = (const T*)p.z + row * p.z_n + c0;
        const T* dy = (const T*)p.dy + row * p.dy_n + c0;
        T* dx = (T*)p.out + row * p.y_n + c0;
        T* dz = (T*)p.dz + row * p.z_n + c0;
        RawVec<T, V> xr[NV], zr[NV], gr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Cell<V> q(i, LG, lane, p.D);
            load_raw<T, V>(x + q.c, V, xr[i]);
            load_raw<T, V>(dy + q.c, V, gr[i]);
            if (ACT == GATE) load_raw<T, V>(z + q.c, V, zr[i]);
        }
        const float mean = p.mean_in[row * p.G + g], rstd = p.rstd_in[row * p.G + g];
        float xh[NV][V], gw[NV][V], s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Cell<V> q(i, LG, lane, p.D);
            float zo[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[i][j] = ((float)xr[i].v[j] - mean) * rstd;
                const float du = slope<ACT>((float)gr[i].v[j], xh[i][j] * w[i][j] + b[i][j],
                                            ACT == GATE ? (float)zr[i].v[j] : 0.f, zo[j]);
                dw[i][j] += du * xh[i][j];
                db[i][j] += du;
                gw[i][j] = du * w[i][j];
                s0 += j >= q.skip ? gw[i][j] : 0.f;
                s1 += j >= q.skip ? gw[i][j] * xh[i][j] : 0.f;
            }
            if (ACT == GATE && q.skip < V) store_vec<T, V>(dz + q.c, V, zo);
        }
        s0 = lanes_sum<LG>(s0) * inv;
        s1 = lanes_sum<LG>(s1) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Cell<V> q(i, LG, lane, p.D);
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = rstd * (gw[i][j] - s0 - xh[i][j] * s1);
            if (q.skip < V) store_vec<T, V>(dx + q.c, V, o);
        }
    }
    float* part = p.part + walker * 2 * p.C + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Cell<V> q(i, LG, lane, p.D);
        if (q.skip < V) {
            store_vec<float, V>(part + q.c, V, dw[i]);
            store_vec<float, V>(part + p.C + q.c, V, db[i]);
        }
    }
}

// ---- P > 1 ---------------------------------------------------------------------------------

// Threads of a workgroup: across CV vectors of V channels, down R rows.  The workgroup takes
// one run of positions of one sample; R threads of a column are joined in LDS.
template <int V>
struct Grid {
    int cl, r, R;  // this thread's vector and row, rows of the workgroup
    int64_t c;     // first channel (moved back to end with the row), and those it shares
    int skip;
    __device__ __forceinline__ Grid(const GnParams& p, int across) {
        cl = threadIdx.x % across;
        r = threadIdx.x / across;
        R = blockDim.x / across;
        const int64_t at = ((int64_t)blockIdx.y * across + cl) * V;
        c = at < p.C - V ? at : p.C - V;
        skip = (int)(at - c < V ? at - c : V);
    }
};

constexpr int kWide = 2048;  // channels that a workgroup spans at most (256 vectors)

// Calls f(g, lane, lanes) once for each of G groups with `lanes` neighbouring lanes (a power of
// two up to 64: as many as the workgroup has for each group, so that one round does).  With g = G
// there is nothing to do but take part in the lanes' sums.
template <typename F>
__device__ __forceinline__ void each_group(int G, F f) {
    int lanes = 64;
    while (lanes > 1 && lanes * G > (int)blockDim.x) lanes /= 2;
    const int at = threadIdx.x / lanes, step = blockDim.x / lanes;
    // threads behind the last whole set of lanes take no group
    for (int g0 = 0; g0 < G; g0 += step)
        f(at < step && g0 + at < G ? g0 + at : G, threadIdx.x % lanes, lanes);
}
__device__ __forceinline__ float some_sum(float v, int lanes) {
    for (int o = 1; o < lanes; o *= 2) v += __shfl_xor(v, o);
    return v;
}

// Columns' means and squared deviations of a run.  A thread takes blocks of UN positions: sums of
// their distances from the first of them, which is one of them, so that the mean's share of the
// squares is at most UN times the deviations, wherever the values lie; then joins the block to
// what it has by counts, means and deviations,
//   n = na + nb, d = mb - ma:  m = ma + d nb / n,  s = sa + sb + d^2 na nb / n,
// whose terms are all positive: one rounding of the whole a block.  (With one origin for a run
// of 16384 positions, its first of 1000 among unit normals, the variance was 2e-3 off; it is
// 2e-7 off so, and 8 maps of 4096 x 320 in bf16 take 22.6 us where they took 21.7.)
template <typename T, int V>
__global__ __launch_bounds__(256) void gn_stats(GnParams p, int across) {
    constexpr int UN = 8;
    __shared__ float ex[2][256][V], counts[256];
    const Grid<V> t(p, across);
    int64_t n;
    const int64_t run = divide(unit(), p.runs, &n);
    if (n >= p.n) return;
    const int64_t p0 = run * p.runlen, p1 = p0 + p.runlen < p.P ? p0 + p.runlen : p.P;
    const T* x = (const T*)p.x + n * p.x_n + t.c;
    float mean[V], m2[V], count = 0.f;
    load_vec<T, V>(x + (p0 + t.r < p1 ? p0 + t.r : p0) * p.x_p, V, mean);
#pragma unroll
    for (int j = 0; j < V; ++j) m2[j] = 0.f;
    for (int64_t q = p0 + t.r; q < p1; q += UN * t.R) {
        RawVec<T, V> raw[UN];
        float rows = 0.f;
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            // rows past the run's end are the block's first: no distance
            const int64_t at = q + i * t.R;
            load_raw<T, V>(x + (at < p1 ? at : q) * p.x_p, V, raw[i]);
            rows += at < p1 ? 1.f : 0.f;
        }
        const float per = __builtin_amdgcn_rcpf(rows), total = count + rows;
        const float f = rows * __builtin_amdgcn_rcpf(total), cf = count * f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float first = (float)raw[0].v[j];
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 1; i < UN; ++i) {
                const float d = (float)raw[i].v[j] - first;
                s1 += d;
                s2 = fmaf(d, d, s2);
            }
            const float e = s1 * per, sq = fmaf(-e, s1, s2), d = (first - mean[j]) + e;
            mean[j] = fmaf(d, f, mean[j]);
            m2[j] += fmaf(d * cf, d, sq < 0.f ? 0.f : sq);  // a NaN stays
        }
        count = total;
    }
    // the threads of a column: the lower half joins the upper, until one is left (one thread after the
    // other took 53 us for 64 maps of 4096 x 8 in bf16, 256 threads a column; halves take 16)
    int half = 0;  // none to join with one
    if (t.R > 1)
        for (half = 1; 2 * half < t.R;) half *= 2;
    for (int top = t.R; half > 0; top = half, half /= 2) {
        if (t.r >= half && t.r < top) {
            counts[threadIdx.x] = count;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                ex[0][threadIdx.x][j] = mean[j];
                ex[1][threadIdx.x][j] = m2[j];
            }
        }
        __syncthreads();
        if (t.r < half && t.r + half < top) {
            const int other = threadIdx.x + half * across;
            const float rows = counts[other], total = count + rows;
            const float f = total > 0.f ? rows * __builtin_amdgcn_rcpf(total) : 0.f, cf = count * f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = ex[0][other][j] - mean[j];
                mean[j] = fmaf(d, f, mean[j]);
                m2[j] += fmaf(d * cf, d, ex[1][other][j]);
            }
            count = total;
        }
        __syncthreads();
    }
    if (t.r && !p.of_runs) return;
    const float len = (float)(p1 - p0);
    if (!p.of_runs) {
        if (t.skip < V) {
            float* part = p.part + (n * p.runs + run) * 2 * p.C + t.c;
            store_vec<float, V>(part, V, mean);
            store_vec<float, V>(part + p.C, V, m2);
        }
        return;
    }
    // the run's groups: columns of equal counts
    __syncthreads();
    float* const cm = &ex[0][0][0];
    float* const cs = &ex[1][0][0];
    if (t.r == 0)
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= t.skip) {
                cm[t.c + j] = mean[j];
                cs[t.c + j] = m2[j];
            }
    __syncthreads();
    each_group(p.G, [&](int g, int lane, int lanes) {
        const int d0 = g < p.G ? g * p.D : 0, D = g < p.G ? p.D : 0;
        float a = 0.f, b = 0.f;
        for (int d = lane; d < D; d += lanes) a += cm[d0 + d];
        a = some_sum(a, lanes) / (float)p.D;
        for (int d = lane; d < D; d += lanes) {
            const float e = cm[d0 + d] - a;
            b += cs[d0 + d] + len * e * e;
        }
        b = some_sum(b, lanes);
        if (D && lane == 0) {
            float* o = p.of_runs + (n * p.runs + run) * 2 * p.G + g;
            o[0] = a;
            o[p.G] = b;
        }
    });
}

// Sum over a workgroup of 256, in every thread.
__device__ __forceinline__ float group_sum(float v, float* ex) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) ex[threadIdx.x >> 6] = v;
    __syncthreads();
    return ex[0] + ex[1] + ex[2] + ex[3];
}

// Where a workgroup does not span the channels, one for each sample and group: mean and rstd
// from its columns' of every run.
__global__ __launch_bounds__(256) void gn_stats_join(GnParams p) {
    __shared__ float ex[4];
    const int64_t id = unit();
    if (id >= p.n * p.G) return;
    int64_t n;
    const int g = (int)divide(id, p.G, &n);
    const float* part = p.part + n * p.runs * 2 * p.C + g * p.D;
    const int64_t items = (int64_t)p.runs * p.D;
    const float total = (float)p.P * (float)p.D;
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < items; i += 256) {
        int64_t run;
        const int d = (int)divide(i, p.D, &run);
        const int64_t len = run + 1 < p.runs ? p.runlen : p.P - run * p.runlen;
        s += (float)len / (float)p.P * part[run * 2 * p.C + d];
    }
    const float mean = group_sum(s, ex) / (float)p.D;
    s = 0.f;
    for (int64_t i = threadIdx.x; i < items; i += 256) {
        int64_t run;
        const int d = (int)divide(i, p.D, &run);
        const int64_t len = run + 1 < p.runs ? p.runlen : p.P - run * p.runlen;
        const float e = part[run * 2 * p.C + d] - mean;
        s += part[(run * 2 + 1) * p.C + d] + (float)len * e * e;
    }
    const float rstd = 1.f / sqrtf(group_sum(s, ex) / total + p.eps);
    if (threadIdx.x == 0) {
        p.mean[id] = mean;
        p.rstd[id] = rstd;
    }
}

// The output's pass.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(256) void gn_apply(GnParams p, int across) {
    constexpr int UN = 4;
    __shared__ float stats[2][kWide];
    const Grid<V> t(p, across);
    int64_t n;
    const int64_t run = divide(unit(), p.runs, &n);
    if (n >= p.n) return;
    const int64_t p0 = run * p.runlen, p1 = p0 + p.runlen < p.P ? p0 + p.runlen : p.P;
    const T* x = (const T*)p.x + n * p.x_n + t.c;
    const T* z = (const T*)p.z + n * p.z_n + t.c;
    T* y = (T*)p.out + n * p.y_n + t.c;
    // the first rows are on their way while the statistics are joined, and each time the next
    RawVec<T, V> xr[UN], zr[UN];
    auto fetch = [&](int64_t q) {
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t at = q + i * t.R < p1 ? q + i * t.R : p0;
            load_raw<T, V>(x + at * p.x_p, V, xr[i]);
            if (ACT == GATE) load_raw<T, V>(z + at * p.z_p, V, zr[i]);
        }
    };
    fetch(p0 + t.r);
    float a[V], m[V], b[V], w[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        w[j] = 1.f;
        b[j] = 0.f;
    }
    if (p.weight) load_vec<float, V>(p.weight + t.c, V, w);
    if (p.bias) load_vec<float, V>(p.bias + t.c, V, b);
    if (p.of_runs) {
        // runs joined as gn_stats joins blocks, one after the other in a lane, then the lanes
        each_group(p.G, [&](int g, int lane, int lanes) {
            const float* q = p.of_runs + n * p.runs * 2 * p.G + (g < p.G ? g : 0);
            float count = 0.f, mean = q[0], m2 = 0.f;
            const float D = (float)p.D;
            auto join = [&](float c, float m, float s) {
                const float total = count + c, f = total > 0.f ? c * __builtin_amdgcn_rcpf(total) : 0.f;
                const float d = m - mean;
                m2 += fmaf(D * (d * (count * f)), d, s);
                mean = fmaf(d, f, mean);
                count = total;
            };
#pragma unroll 8
            for (int i = lane; i < p.runs; i += lanes)
                join((float)(i + 1 < p.runs ? p.runlen : p.P - i * p.runlen), q[(int64_t)i * 2 * p.G],
                     q[((int64_t)i * 2 + 1) * p.G]);
            for (int o = 1; o < lanes; o *= 2)
                join(__shfl_xor(count, o), __shfl_xor(mean, o), __shfl_xor(m2, o));
            const float rstd = 1.f / sqrtf(m2 / ((float)p.P * D) + p.eps);
            if (g < p.G && lane == 0) {
                stats[0][g] = mean;
                stats[1][g] = rstd;
                if (run == 0) {
                    if (p.mean) p.mean[n * p.G + g] = mean;
                    if (p.rstd) p.rstd[n * p.G + g] = rstd;
                }
            }
        });
        __syncthreads();
    }
    int g = (int)t.c / p.D, at0 = (int)t.c % p.D;  // a group, and the channel in it
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j && ++at0 == p.D) at0 = 0, ++g;
        m[j] = p.of_runs ? stats[0][g] : p.mean[n * p.G + g];
        a[j] = p.of_runs ? stats[1][g] : p.rstd[n * p.G + g];
    }
    for (int64_t q = p0 + t.r; q < p1; q += UN * t.R) {
        float v[UN][V], u[UN][V];
#pragma unroll
        for (int i = 0; i < UN; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] = (float)xr[i].v[j];
                u[i][j] = ACT == GATE ? (float)zr[i].v[j] : 0.f;
            }
        if (q + UN * t.R < p1) fetch(q + UN * t.R);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t at = q + i * t.R;
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = activate<ACT>((v[i][j] - m[j]) * a[j] * w[j] + b[j], u[i][j]);
            if (at < p1) store_own<T, V>(y + at * p.y_p, t.skip, o);
        }
    }
}

// Backward.  DX false: columns' sums of du xh and du of a run (and dz); true: dx.
template <typename T, int V, int ACT, bool DX>
__global__ __launch_bounds__(256) void gn_bwd(GnParams p, int across) {
    constexpr int UN = 2;
    __shared__ float ex[2][256][V];  // DX: mean(g) and mean(g xh) of the groups
    const Grid<V> t(p, across);
    int64_t n;
    const int64_t run = divide(unit(), p.runs, &n);
    if (n >= p.n) return;
    const int64_t p0 = run * p.runlen, p1 = p0 + p.runlen < p.P ? p0 + p.runlen : p.P;
    const T* x = (const T*)p.x + n * p.x_n + t.c;
    const T* z = (const T*)p.z + n * p.z_n + t.c;
    const T* dy = (const T*)p.dy + n * p.dy_n + t.c;
    T* dx = (T*)p.out + n * p.y_n + t.c;
    T* dz = (T*)p.dz + n * p.z_n + t.c;
    // the first rows are on their way while the groups' sums are joined, and each time the next
    RawVec<T, V> xr[UN], zr[UN], gr[UN];
    auto fetch = [&](int64_t q) {
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t at = q + i * t.R < p1 ? q + i * t.R : p0;
            load_raw<T, V>(x + at * p.x_p, V, xr[i]);
            load_raw<T, V>(dy + at * p.dy_p, V, gr[i]);
            if (ACT == GATE) load_raw<T, V>(z + at * p.z_p, V, zr[i]);
        }
    };
    fetch(p0 + t.r);
    float m[V], a[V], b[V], w[V], s0[V], s1[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        w[j] = 1.f;
        b[j] = 0.f;
    }
    if (p.weight) load_vec<float, V>(p.weight + t.c, V, w);
    if (ACT != PLAIN && p.bias) load_vec<float, V>(p.bias + t.c, V, b);
    int64_t g = n * p.G + (int)t.c / p.D;  // a group, and the channel in it
    int at0 = (int)t.c % p.D;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j && ++at0 == p.D) at0 = 0, ++g;
        m[j] = p.mean_in[g];
        a[j] = p.rstd_in[g];
        s0[j] = DX && !p.of_runs ? p.sums[2 * g] : 0.f;
        s1[j] = DX && !p.of_runs ? p.sums[2 * g + 1] : 0.f;
    }
    if (DX && p.of_runs) {
        float* const sums = &ex[0][0][0];  // [2][G], G <= 256 V
        each_group(p.G, [&](int g, int lane, int lanes) {
            const float* q = p.of_runs + n * p.runs * 2 * p.G + (g < p.G ? g : 0);
            float x = 0.f, y = 0.f;
#pragma unroll 8
            for (int i = lane; i < p.runs; i += lanes) {
                x += q[(int64_t)i * 2 * p.G];
                y += q[((int64_t)i * 2 + 1) * p.G];
            }
            const float inv = 1.f / ((float)p.P * (float)p.D);
            x = some_sum(x, lanes) * inv;
            y = some_sum(y, lanes) * inv;
            if (g < p.G && lane == 0) {
                sums[g] = x;
                sums[p.G + g] = y;
            }
        });
        __syncthreads();
        int g = (int)t.c / p.D, at0 = (int)t.c % p.D;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j && ++at0 == p.D) at0 = 0, ++g;
            s0[j] = sums[g];
            s1[j] = sums[p.G + g];
        }
    }
    for (int64_t q = p0 + t.r; q < p1; q += UN * t.R) {
        float xv[UN][V], zv[UN][V], gv[UN][V];
#pragma unroll
        for (int i = 0; i < UN; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xv[i][j] = (float)xr[i].v[j];
                zv[i][j] = ACT == GATE ? (float)zr[i].v[j] : 0.f;
                gv[i][j] = (float)gr[i].v[j];
            }
        if (q + UN * t.R < p1) fetch(q + UN * t.R);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t at = q + i * t.R;
            float o[V], zo[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (xv[i][j] - m[j]) * a[j];
                const float du = slope<ACT>(gv[i][j], xh * w[j] + b[j], zv[i][j], zo[j]);
                if (DX) {
                    o[j] = a[j] * (du * w[j] - s0[j] - xh * s1[j]);
                } else if (at < p1) {
                    s0[j] += du * xh;
                    s1[j] += du;
                }
            }
            if (at < p1) {
                if (DX) store_own<T, V>(dx + at * p.y_p, t.skip, o);
                else if (ACT == GATE) store_own<T, V>(dz + at * p.z_p, t.skip, zo);
            }
        }
    }
    if constexpr (!DX) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            ex[0][threadIdx.x][j] = s0[j];
            ex[1][threadIdx.x][j] = s1[j];
        }
        __syncthreads();
        if (t.r || t.skip >= V) {
            if (!p.of_runs) return;
        } else for (int r = 1; r < t.R; ++r)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s0[j] += ex[0][r * across + t.cl][j];
                s1[j] += ex[1][r * across + t.cl][j];
            }
        if (t.r == 0 && t.skip < V) {
            float* part = p.part + (n * p.runs + run) * 2 * p.C + t.c;
            store_vec<float, V>(part, V, s0);
            store_vec<float, V>(part + p.C, V, s1);
        }
        if (!p.of_runs) return;
        // the run's groups: sums of g = du w and of g xh
        __syncthreads();
        float* const cx = &ex[0][0][0];
        float* const cd = &ex[1][0][0];
        if (t.r == 0)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j >= t.skip) {
                    cx[t.c + j] = s0[j] * w[j];
                    cd[t.c + j] = s1[j] * w[j];
                }
        __syncthreads();
        each_group(p.G, [&](int g, int lane, int lanes) {
            const int d0 = g < p.G ? g * p.D : 0, D = g < p.G ? p.D : 0;
            float x = 0.f, y = 0.f;
            for (int d = lane; d < D; d += lanes) {
                x += cd[d0 + d];
                y += cx[d0 + d];
            }
            x = some_sum(x, lanes);
            y = some_sum(y, lanes);
            if (D && lane == 0) {
                float* o = p.of_runs + (n * p.runs + run) * 2 * p.G + g;
                o[0] = x;
                o[p.G] = y;
            }
        });
    }
}

// Likewise mean(g) and mean(g xh) from the columns' sums.
__global__ __launch_bounds__(256) void gn_bwd_join(GnParams p) {
    __shared__ float ex[4];
    const int64_t id = unit();
    if (id >= p.n * p.G) return;
    int64_t n;
    const int g = (int)divide(id, p.G, &n);
    const float* part = p.part + n * p.runs * 2 * p.C + g * p.D;
    const float* w = p.weight ? p.weight + g * p.D : nullptr;
    float s0 = 0.f, s1 = 0.f;
    for (int64_t i = threadIdx.x; i < (int64_t)p.runs * p.D; i += 256) {
        int64_t run;
        const int d = (int)divide(i, p.D, &run);
        const float f = w ? w[d] : 1.f;
        s1 += f * part[run * 2 * p.C + d];
        s0 += f * part[(run * 2 + 1) * p.C + d];
    }
    const float total = (float)p.P * (float)p.D;
    s0 = group_sum(s0, ex) / total;
    s1 = group_sum(s1, ex) / total;
    if (threadIdx.x == 0) {
        p.sums[2 * id] = s0;
        p.sums[2 * id + 1] = s1;
    }
}

// ---- host ----------------------------------------------------------------------------------

int gn_vec(const ssd_groupnorm_dims& d, int64_t width) {
    const int V = d.dtype == SSD_BF16 ? 8 : 4;
    return width >= V ? V : 1;
}

// P = 1: lanes of a group and vectors of a lane
struct RowPlan {
    int V, LG, NV;
};
RowPlan row_plan(const ssd_groupnorm_dims& d) {
    const int64_t D = d.channels / d.groups;
    RowPlan r;
    r.V = gn_vec(d, D);
    const int64_t vecs = cdiv(D, r.V);
    r.LG = 8;
    while (r.LG < 64 && r.LG < vecs) r.LG *= 2;
    r.NV = 1;
    while (r.NV * r.LG < vecs) r.NV *= 2;
    return r;
}
constexpr int kRowMost = 4;  // vectors of a lane: groups of up to 2048 (bf16) or 1024 channels

// P > 1: runs of positions; threads across the channels
struct RunPlan {
    int V, across;
    int64_t runlen;
    int32_t runs, blocks;
};
RunPlan run_plan(const ssd_groupnorm_dims& d) {
    RunPlan r;
    r.V = gn_vec(d, d.channels);
    const int64_t vecs = cdiv(d.channels, r.V);
    r.blocks = (int)cdiv(vecs, 256);
    r.across = (int)cdiv(vecs, r.blocks);
    const int64_t R = 256 / r.across;
    // Two workgroups a CU, but no fewer than 4 rows a thread: more runs leave more to join (8 x
    // 4096 x 320 bf16, one call behind the other, us: 256 workgroups 24, 512 24, 768 26, 1024 31).
    const int64_t want = cdiv(512, imax(1, d.samples) * r.blocks);
    r.runlen = imax(cdiv(d.positions, want), 4 * R);
    r.runs = (int)cdiv(d.positions, r.runlen);
    return r;
}

bool by_rows(const ssd_groupnorm_dims& d) {
    return d.positions == 1 && row_plan(d).NV <= kRowMost;
}

int32_t row_walkers(const ssd_groupnorm_dims& d) {
    const RowPlan r = row_plan(d);
    // 768 workgroups' worth of lanes (three a CU) at most, and no fewer than four rows each: each
    // walker writes a row of sums that is read again (8192 x 16 groups of 128 bf16 with a gate,
    // us: 512 workgroups 34, 768 34, 1024 36, 2048 42).
    const int64_t per = cdiv((int64_t)d.groups * r.LG, 256);
    int64_t w = imax(1, 768 / per);
    const int64_t most = imax(1, cdiv(d.samples, 4));
    return (int32_t)(w < most ? w : most);
}

int gn_check(const ssd_groupnorm_dims* d) {
    if (!d) return SSD_ERR_NULL_ARG;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->samples < 0 || d->positions < 1 || d->groups < 1 || d->channels < 1 ||
        d->channels % d->groups || d->channels > kMaxStride ||
        d->samples > kMaxTokens / d->positions || !(d->eps >= 0.f) || d->reserved != 0)
        return SSD_ERR_SHAPE;
    if (d->activation < SSD_ACT_NONE || d->activation > SSD_ACT_GATE) return SSD_ERR_UNSUPPORTED;
    if (d->samples * d->groups > kMaxTokens) return SSD_ERR_SHAPE;
    for (int64_t s : {d->x_row, d->y_row, d->z_row, d->dy_row})
        if (s < d->channels || s > kMaxStride) return SSD_ERR_SHAPE;
    for (int64_t s : {d->x_sample, d->y_sample, d->z_sample, d->dy_sample})
        if (s < 0 || s > (int64_t)1 << 40) return SSD_ERR_SHAPE;
    return SSD_OK;
}

GnParams gn_params(const ssd_groupnorm_dims& d) {
    GnParams p = {};
    p.n = d.samples;
    p.P = d.positions;
    p.C = d.channels;
    p.G = d.groups;
    p.D = d.channels / d.groups;
    p.eps = d.eps;
    p.x_n = d.x_sample, p.x_p = d.x_row;
    p.z_n = d.z_sample, p.z_p = d.z_row;
    p.y_n = d.y_sample, p.y_p = d.y_row;
    p.dy_n = d.dy_sample, p.dy_p = d.dy_row;
    return p;
}

template <typename T, int V, int NV, int LG, bool BWD>
void launch_row(const ssd_groupnorm_dims& d, const GnParams& p, hipStream_t s) {
    const int64_t groups = BWD ? (int64_t)p.walkers * p.G : p.n * p.G;
    const dim3 grid = units(cdiv(groups * LG, 256));
#define SSD_GN_ACT(A)                                                        \
    case A:                                                                  \
        if constexpr (BWD) gn_row_bwd<T, V, NV, LG, A><<<grid, 256, 0, s>>>(p); \
        else gn_row_fwd<T, V, NV, LG, A><<<grid, 256, 0, s>>>(p);            \
        break
    switch (d.activation) {
        SSD_GN_ACT(PLAIN);
        SSD_GN_ACT(SILU);
        SSD_GN_ACT(GATE);
    }
#undef SSD_GN_ACT
}
template <typename T, int V, bool BWD>
void launch_row(const ssd_groupnorm_dims& d, const GnParams& p, RowPlan r, hipStream_t s) {
    if (r.V == 1) return launch_row<T, 1, 1, 8, BWD>(d, p, s);  // fewer channels than a vector
    switch (r.NV * 64 + r.LG) {
        case 64 + 8: return launch_row<T, V, 1, 8, BWD>(d, p, s);
        case 64 + 16: return launch_row<T, V, 1, 16, BWD>(d, p, s);
        case 64 + 32: return launch_row<T, V, 1, 32, BWD>(d, p, s);
        case 128: return launch_row<T, V, 1, 64, BWD>(d, p, s);
        case 192: return launch_row<T, V, 2, 64, BWD>(d, p, s);
        default: return launch_row<T, V, 4, 64, BWD>(d, p, s);
    }
}

template <typename T, int V>
void launch_runs_fwd(const ssd_groupnorm_dims& d, const GnParams& p, RunPlan r, hipStream_t s) {
    const dim3 grid = units(p.n * r.runs, r.blocks);
    const dim3 block((unsigned)(256 / r.across * r.across));
    gn_stats<T, V><<<grid, block, 0, s>>>(p, r.across);
    if (!p.of_runs) gn_stats_join<<<units(p.n * p.G), 256, 0, s>>>(p);
    if (d.activation == PLAIN) gn_apply<T, V, PLAIN><<<grid, block, 0, s>>>(p, r.across);
    else if (d.activation == SILU) gn_apply<T, V, SILU><<<grid, block, 0, s>>>(p, r.across);
    else gn_apply<T, V, GATE><<<grid, block, 0, s>>>(p, r.across);
}
template <typename T, int V, int ACT>
void launch_runs_bwd(const GnParams& p, RunPlan r, hipStream_t s) {
    const dim3 grid = units(p.n * r.runs, r.blocks);
    const dim3 block((unsigned)(256 / r.across * r.across));
    gn_bwd<T, V, ACT, false><<<grid, block, 0, s>>>(p, r.across);
    if (!p.of_runs) gn_bwd_join<<<units(p.n * p.G), 256, 0, s>>>(p);
    gn_bwd<T, V, ACT, true><<<grid, block, 0, s>>>(p, r.across);
}
template <typename T, int V>
void launch_runs_bwd(const ssd_groupnorm_dims& d, const GnParams& p, RunPlan r, hipStream_t s) {
    if (d.activation == PLAIN) launch_runs_bwd<T, V, PLAIN>(p, r, s);
    else if (d.activation == SILU) launch_runs_bwd<T, V, SILU>(p, r, s);
    else launch_runs_bwd<T, V, GATE>(p, r, s);
}

// Workspace: columns' sums of the runs, and groups' (of the runs, or where a workgroup does not
// span the channels joined; in the forward the statistics then, if the caller does not take
// them).  The forward needs no columns' sums but in that case.
struct GnSpace {
    size_t part, sums;
};
GnSpace gn_space(const ssd_groupnorm_dims& d, bool bwd) {
    GnSpace w = {};
    if (by_rows(d)) {
        w.part = bwd ? up256((size_t)row_walkers(d) * 2 * d.channels * 4) : 0;
        return w;
    }
    const RunPlan r = run_plan(d);
    const size_t runs = (size_t)imax(1, d.samples * r.runs), one = r.blocks == 1;
    w.part = bwd || !one ? up256(runs * 2 * d.channels * 4) : 0;
    w.sums = up256((one ? runs : (size_t)imax(1, d.samples)) * 2 * d.groups * 4);
    return w;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_groupnorm_fwd_workspace_bytes(const ssd_groupnorm_dims* dims) {
    if (gn_check(dims) != SSD_OK) return 0;
    const GnSpace w = gn_space(*dims, false);
    return w.part + w.sums;
}

int ssd_groupnorm_fwd(const ssd_groupnorm_dims* dims, const void* x, const float* weight,
                      const float* bias, const void* z, void* y, float* mean, float* rstd,
                      void* workspace, size_t workspace_bytes, void* stream) {
    const int st = gn_check(dims);
    if (st != SSD_OK) return st;
    const ssd_groupnorm_dims& d = *dims;
    if (d.samples == 0) return SSD_OK;
    if (!x || !y || (d.activation == SSD_ACT_GATE && !z)) return SSD_ERR_NULL_ARG;
    if (!rows_apart(d.samples, d.y_sample, d.positions, d.y_row, d.channels)) return SSD_ERR_SHAPE;
    const size_t e = elem_size(d.dtype);
    if (!elem_aligned(x, e) || !elem_aligned(y, e) || !elem_aligned(z, e) || !elem_aligned(weight, 4) ||
        !elem_aligned(bias, 4) || !elem_aligned(mean, 4) || !elem_aligned(rstd, 4) ||
        ((uintptr_t)workspace & 255))
        return SSD_ERR_ALIGN;
    const GnSpace w = gn_space(d, false);
    if (w.part + w.sums && (!workspace || workspace_bytes < w.part + w.sums)) return SSD_ERR_WORKSPACE;
    GnParams p = gn_params(d);
    p.x = x;
    p.z = z;
    p.out = y;
    p.weight = weight;
    p.bias = bias;
    p.mean = mean;
    p.rstd = rstd;
    const hipStream_t s = (hipStream_t)stream;
    if (by_rows(d)) {
        const RowPlan r = row_plan(d);
        if (d.dtype == SSD_BF16) launch_row<bf16, 8, false>(d, p, r, s);
        else launch_row<float, 4, false>(d, p, r, s);
        return launched();
    }
    const RunPlan r = run_plan(d);
    p.part = (float*)workspace;
    p.runs = r.runs;
    p.runlen = r.runlen;
    float* const sums = (float*)((char*)workspace + w.part);
    if (r.blocks == 1) {
        p.of_runs = sums;
    } else {
        if (!p.mean) p.mean = sums;
        if (!p.rstd) p.rstd = sums + d.samples * d.groups;
    }
    if (d.dtype == SSD_BF16) {
        if (r.V == 1) launch_runs_fwd<bf16, 1>(d, p, r, s);
        else launch_runs_fwd<bf16, 8>(d, p, r, s);
    } else {
        if (r.V == 1) launch_runs_fwd<float, 1>(d, p, r, s);
        else launch_runs_fwd<float, 4>(d, p, r, s);
    }
    return launched();
}

size_t ssd_groupnorm_bwd_workspace_bytes(const ssd_groupnorm_dims* dims) {
    if (gn_check(dims) != SSD_OK) return 0;
    const GnSpace w = gn_space(*dims, true);
    return w.part + w.sums;
}

int ssd_groupnorm_bwd(const ssd_groupnorm_dims* dims, const void* x, const float* weight,
                      const float* bias, const void* z, const float* mean, const float* rstd,
                      const void* dy, void* dx, void* dz, float* dweight, float* dbias,
                      void* workspace, size_t workspace_bytes, void* stream) {
    const int st = gn_check(dims);
    if (st != SSD_OK) return st;
    const ssd_groupnorm_dims& d = *dims;
    const bool gate = d.activation == SSD_ACT_GATE;
    if (d.samples > 0 && (!x || !mean || !rstd || !dy || !dx || (gate && (!z || !dz)))) return SSD_ERR_NULL_ARG;
    if (d.samples > 0 && (!rows_apart(d.samples, d.y_sample, d.positions, d.y_row, d.channels) ||
                          (gate && !rows_apart(d.samples, d.z_sample, d.positions, d.z_row, d.channels))))
        return SSD_ERR_SHAPE;
    const size_t e = elem_size(d.dtype);
    for (const void* a : {x, z, dy, (const void*)dx, (const void*)dz})
        if (!elem_aligned(a, e)) return SSD_ERR_ALIGN;
    for (const void* a : {(const void*)weight, (const void*)bias, (const void*)mean, (const void*)rstd,
                          (const void*)dweight, (const void*)dbias})
        if (!elem_aligned(a, 4)) return SSD_ERR_ALIGN;
    if ((uintptr_t)workspace & 255) return SSD_ERR_ALIGN;
    const GnSpace w = gn_space(d, true);
    if (!workspace || workspace_bytes < w.part + w.sums) return SSD_ERR_WORKSPACE;
    GnParams p = gn_params(d);
    p.x = x;
    p.z = z;
    p.dy = dy;
    p.out = dx;
    p.dz = dz;
    p.weight = weight;
    p.bias = bias;
    p.mean_in = mean;
    p.rstd_in = rstd;
    p.part = (float*)workspace;
    const hipStream_t s = (hipStream_t)stream;
    ColSum c = {};
    c.part = p.part;
    c.cols = 2 * (int64_t)d.channels;
    c.out0 = dweight;
    c.c0 = d.channels;
    c.out1 = dbias;
    c.c1 = d.channels;
    if (d.samples == 0) {
        // no rows: sums of nothing
        c.rows = 0;
    } else if (by_rows(d)) {
        const RowPlan r = row_plan(d);
        c.rows = p.walkers = row_walkers(d);
        if (d.dtype == SSD_BF16) launch_row<bf16, 8, true>(d, p, r, s);
        else launch_row<float, 4, true>(d, p, r, s);
    } else {
        const RunPlan r = run_plan(d);
        p.runs = r.runs;
        p.runlen = r.runlen;
        (r.blocks == 1 ? p.of_runs : p.sums) = (float*)((char*)workspace + w.part);
        c.rows = d.samples * r.runs;
        if (d.dtype == SSD_BF16) {
            if (r.V == 1) launch_runs_bwd<bf16, 1>(d, p, r, s);
            else launch_runs_bwd<bf16, 8>(d, p, r, s);
        } else {
            if (r.V == 1) launch_runs_bwd<float, 1>(d, p, r, s);
            else launch_runs_bwd<float, 4>(d, p, r, s);
        }
    }
    const int rc = launched();
    if (rc != SSD_OK || (!dweight && !dbias)) return rc;
    return launch_colsum(c, s);
}

}  // extern "C"
