// Short causal convolution with bias and SiLU over packed sequences, forward
// and backward.
//
//   v_t = b + sum_k w[k] x_{t-W+1+k},  y_t = v_t s_t,  s_t = 1 / (1 + e^-v_t)
//   dv_t = dy_t s_t (1 + v_t (1 - s_t))
//   dx_t = sum_j w[W-1-j] dv_{t+j},  dw[k] = sum_t dv_t x_{t-W+1+k},  db = sum_t dv_t
//
// Bound by HBM.  A thread takes a vector of channels over a run of tokens,
// every row of which it loads once and keeps in registers: the W - 1 rows
// before the run (and, backwards, after it) are the only re-reads, and they
// come from cache.  Threads of a wave lie along the channels, so every load
// is a contiguous piece of a row; where the channels are no multiple of the
// vector, the last one is moved back to end with them (the channels it shares
// with its neighbour are formed twice, to the same bits), so there is no
// partial vector.  Runs that lie whole inside one sequence take an unrolled
// path with all loads issued first; the others walk token by token.  The states (final_state, dinit_state)
// come from work items of their own behind the tokens'.
#include "ssd_layer.h"

namespace ssd {
namespace {

struct ConvParams {
    const void* x;
    const void* init;
    const void* dy;
    const void* d_final;
    void* out;        // y or dx
    void* state_out;  // final_state or dinit_state, or null
    const float* weight;
    const float* bias;
    float* part;  // backward: [blocks][W + 1][E]
    const int32_t* cu;
    int64_t xs, os, gs;  // token strides of x, out, dy
    int64_t L, T;
    int64_t main_blocks;  // workgroups of the tokens' items
    int64_t state_items;
    int32_t E, S, nseq, nvec;
    int64_t tiles;          // backward: token tiles in all
    int32_t tiles_per_row;  // token tiles of a batch row (of the packed tokens)
    int32_t iters;          // backward: tiles a wave walks
};

// What a token walk needs of the sequence it is in.
struct Walk {
    int seq;
    int64_t first, last;
};

// At token t of batch row brow (of the packed tokens).
__device__ __forceinline__ Walk walk_at(const ConvParams& p, int64_t t, int64_t brow) {
    Walk w;
    w.seq = p.cu ? sequence_of(p.cu, p.nseq, t) : (int)brow;
    sequence_span(p.cu, w.seq, p.L, p.T, &w.first, &w.last);
    return w;
}

// First channel of vector i.
template <int V>
__device__ __forceinline__ int channel_of(const ConvParams& p, int i) {
    return V == 1 ? i : min(i * V, p.E - V);
}

template <typename T, int V>
__device__ __forceinline__ void load(const T* __restrict__ p, float (&o)[V]) {
    load_vec<T, V>(p, V, o);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* __restrict__ p, const float (&v)[V]) {
    store_vec<T, V>(p, V, v);
}

// Row `row` of sequence seq's initial state (W - 2: the input before its first token).
template <typename T, int W, int V>
__device__ __forceinline__ void load_init(const ConvParams& p, int seq, int row, int e, float (&o)[V]) {
    if (p.init) {
        load<T, V>((const T*)p.init + ((int64_t)seq * (W - 1) + row) * p.E + e, o);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = 0.f;
    }
}

// x at token t of the walk's sequence, or the state's row where t lies before it.
template <typename T, int W, int V>
__device__ __forceinline__ void load_line(const ConvParams& p, const Walk& w, int64_t t, int e,
                                          float (&o)[V]) {
    if (t >= w.first) {
        load<T, V>((const T*)p.x + t * p.xs + e, o);
    } else {
        const int64_t row = t - w.first + W - 1;  // < 0 only where cu_seqlens is not sorted
        load_init<T, W, V>(p, w.seq, row < 0 ? 0 : (int)row, e, o);
    }
}

template <typename T, int V>
using Raw = RawVec<T, V>;
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* __restrict__ p) {
    Raw<T, V> r;
    load_raw<T, V>(p, V, r);
    return r;
}

template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvParams& p, int e, float (&w)[W][V], float (&b)[V]) {
#pragma unroll
    for (int k = 0; k < W; ++k) load<float, V>(p.weight + (int64_t)k * p.E + e, w[k]);
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = 0.f;
    if (p.bias) load<float, V>(p.bias + e, b);
}

template <int W, int V>
__device__ __forceinline__ void filter(const float (&win)[W][V], const float (&w)[W][V],
                                       const float (&b)[V], float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        v[j] = b[j];
#pragma unroll
        for (int k = 0; k < W; ++k) v[j] += win[k][j] * w[k][j];
    }
}
template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W][V]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) win[k][j] = win[k + 1][j];
}

// ---- forward ------------------------------------------------------------------------------

template <typename T, int W, int V, int TT>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p) {
    const T* x = (const T*)p.x;
    if (blockIdx.x >= p.main_blocks) {
        // final_state: row r of sequence s is input last - (W - 1) + r
        const int64_t id = ((int64_t)blockIdx.x - p.main_blocks) * 256 + threadIdx.x;
        if (id >= p.state_items) return;
        int64_t sr;
        const int e = channel_of<V>(p, (int)divide(id, p.nvec, &sr));
        Walk w;
        w.seq = (int)(sr / (W - 1));
        const int r = (int)(sr % (W - 1));
        sequence_span(p.cu, w.seq, p.L, p.T, &w.first, &w.last);
        float o[V];
        load_line<T, W, V>(p, w, w.last - (W - 1) + r, e, o);
        store<T, V>((T*)p.state_out + sr * p.E + e, o);
        return;
    }
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int64_t tile, brow;
    const int e = channel_of<V>(p, (int)divide(id, p.nvec, &tile));
    const int64_t len = p.cu ? p.T : p.L;
    const int64_t at0 = divide(tile, p.tiles_per_row, &brow) * TT;
    const int64_t t0 = brow * len + at0, t1 = imin(t0 + TT, (brow + 1) * len);
    if (t0 >= p.T || t0 >= t1) return;
    Walk at = walk_at(p, t0, brow);
    float w[W][V], b[V], win[W][V], v[V];
    const T* px = x + t0 * p.xs + e;
    T* py = (T*)p.out + t0 * p.os + e;
    if (t0 + TT <= t1 && t1 <= at.last) {
        Raw<T, V> rows[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) rows[i] = load_raw<T, V>(px + i * p.xs);
        load_taps<W, V>(p, e, w, b);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load_line<T, W, V>(p, at, t0 - (W - 1) + k, e, win[k]);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) win[W - 1][j] = (float)rows[i].v[j];
            filter<W, V>(win, w, b, v);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= sigmoid(v[j]);
            store<T, V>(py + i * p.os, v);
            shift<W, V>(win);
        }
        return;
    }
    load_taps<W, V>(p, e, w, b);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_line<T, W, V>(p, at, t0 - (W - 1) + k, e, win[k]);
    Raw<T, V> next = load_raw<T, V>(px);
#pragma unroll 1
    for (int64_t t = t0; t < t1; ++t, px += p.xs, py += p.os) {
        const Raw<T, V> now = next;
        if (t + 1 < t1) next = load_raw<T, V>(px + p.xs);
        if (p.cu && t >= at.last && at.seq + 1 < p.nseq) {  // the next sequence that has tokens
            at = walk_at(p, t, 0);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) load_init<T, W, V>(p, at.seq, k, e, win[k]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) win[W - 1][j] = (float)now.v[j];
        filter<W, V>(win, w, b, v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= sigmoid(v[j]);
        store<T, V>(py, v);
        shift<W, V>(win);
    }
}

// ---- backward -----------------------------------------------------------------------------

// A workgroup takes 64 vectors of channels; its four waves walk `iters` token
// tiles each and join their shares of dw and db in LDS, so one row of partial
// sums is written for 4 * iters * TT tokens.
template <typename T, int W, int V, int TT>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvParams p) {
    const T* x = (const T*)p.x;
    const T* dy = (const T*)p.dy;
    const T* df = (const T*)p.d_final;
    if (blockIdx.x >= p.main_blocks) {
        // dinit_state row r of sequence s: token p <= r meets it with tap r - p,
        // and final_state holds it at row r - len where the sequence is short
        const int64_t id = ((int64_t)blockIdx.x - p.main_blocks) * 256 + threadIdx.x;
        if (id >= p.state_items) return;
        int64_t sr;
        const int e = channel_of<V>(p, (int)divide(id, p.nvec, &sr));
        Walk at;
        at.seq = (int)(sr / (W - 1));
        const int r = (int)(sr % (W - 1));
        sequence_span(p.cu, at.seq, p.L, p.T, &at.first, &at.last);
        const int64_t len = at.last - at.first;
        float acc[V], w[W][V], b[V];
        load_taps<W, V>(p, e, w, b);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
#pragma unroll
        for (int q = 0; q < W - 1; ++q) {
            if (q > r || q >= len) break;
            float v[V], g[V], win[W][V];
#pragma unroll
            for (int k = 0; k < W; ++k) load_line<T, W, V>(p, at, at.first + q - (W - 1) + k, e, win[k]);
            filter<W, V>(win, w, b, v);
            load<T, V>(dy + (at.first + q) * p.gs + e, g);
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (k == r - q) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        acc[j] += g[j] * silu_slope(v[j], sigmoid(v[j])) * w[k][j];
                }
        }
        if (df && r >= len) {
            float g[V];
            load<T, V>(df + ((int64_t)at.seq * (W - 1) + r - len) * p.E + e, g);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += g[j];
        }
        store<T, V>((T*)p.state_out + sr * p.E + e, acc);
        return;
    }
    __shared__ float ex[3][W + 1][V][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint32_t groups = (uint32_t)(p.nvec + 63) / 64;
    const int64_t strip = blockIdx.x / groups;
    const int vec = (int)(blockIdx.x % groups) * 64 + lane;
    const bool live = vec < p.nvec;
    const int e = channel_of<V>(p, live ? vec : 0);
    float w[W][V], b[V], dw[W][V], db[V];
    load_taps<W, V>(p, e, w, b);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        db[j] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][j] = 0.f;
    }
    T* dx = (T*)p.out;
    const int64_t len = p.cu ? p.T : p.L;
    for (int it = 0; it < p.iters; ++it) {
        const int64_t tile = (strip * 4 + wave) * p.iters + it;
        if (tile >= p.tiles || !live) break;
        int64_t brow;
        const int64_t at0 = divide(tile, p.tiles_per_row, &brow) * TT;
        const int64_t t0 = brow * len + at0;
        const int64_t t1 = imin(t0 + TT, (brow + 1) * len);
        Walk at = walk_at(p, t0, brow);
        float win[W][V], acc[W][V], v[V], dv[V];  // acc[j]: dx of token t - (W - 1) + j
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[k][j] = 0.f;
        const T* px = x + t0 * p.xs + e;
        const T* pg = dy + t0 * p.gs + e;
        T* po = dx + t0 * p.xs + e;
        if (t0 + TT <= t1 && t1 + W - 1 <= at.last) {
            // every token whose dv reaches the run is of its sequence, and none
            // of the run is a row of final_state
            Raw<T, V> xr[TT + W - 1], gr[TT + W - 1];
#pragma unroll
            for (int i = 0; i < TT + W - 1; ++i) {
                xr[i] = load_raw<T, V>(px + i * p.xs);
                gr[i] = load_raw<T, V>(pg + i * p.gs);
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k) load_line<T, W, V>(p, at, t0 - (W - 1) + k, e, win[k]);
#pragma unroll
            for (int i = 0; i < TT + W - 1; ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) win[W - 1][j] = (float)xr[i].v[j];
                filter<W, V>(win, w, b, v);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dv[j] = (float)gr[i].v[j] * silu_slope(v[j], sigmoid(v[j]));
                    if (i < TT) {
                        db[j] += dv[j];
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[k][j] += dv[j] * win[k][j];
                    }
                    // of the accumulators only those of the run's tokens count
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        if (i - (W - 1) + k >= 0 && i - (W - 1) + k < TT) acc[k][j] += dv[j] * w[k][j];
                }
                shift<W, V>(win);
                if (i >= W - 1) store<T, V>(po + (i - (W - 1)) * p.xs, acc[0]);
                shift<W, V>(acc);
#pragma unroll
                for (int j = 0; j < V; ++j) acc[W - 1][j] = 0.f;
            }
            continue;
        }
        const int64_t te = imin(t1 + W - 1, (brow + 1) * len);  // tokens whose dv is formed
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load_line<T, W, V>(p, at, t0 - (W - 1) + k, e, win[k]);
        Raw<T, V> xn = load_raw<T, V>(px), gn = load_raw<T, V>(pg);
#pragma unroll 1
        for (int64_t t = t0; t < t1 + W - 1; ++t) {
            if (t < te) {
                const Raw<T, V> xt = xn, gt = gn;
                if (t + 1 < te) {
                    xn = load_raw<T, V>(x + (t + 1) * p.xs + e);
                    gn = load_raw<T, V>(dy + (t + 1) * p.gs + e);
                }
                if (p.cu && t >= at.last && at.seq + 1 < p.nseq) {
                    at = walk_at(p, t, 0);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) load_init<T, W, V>(p, at.seq, k, e, win[k]);
                }
                const int64_t pos = t - at.first;
#pragma unroll
                for (int j = 0; j < V; ++j) win[W - 1][j] = (float)xt.v[j];
                filter<W, V>(win, w, b, v);
#pragma unroll
                for (int j = 0; j < V; ++j) dv[j] = (float)gt.v[j] * silu_slope(v[j], sigmoid(v[j]));
                if (t < t1) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        db[j] += dv[j];
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[k][j] += dv[j] * win[k][j];
                    }
                    if (df && at.last > t && at.last - t <= W - 1) {  // a row of final_state
                        float g[V];
                        load<T, V>(df + ((int64_t)at.seq * (W - 1) + (W - 1) - (at.last - t)) * p.E + e, g);
#pragma unroll
                        for (int j = 0; j < V; ++j) acc[W - 1][j] += g[j];
                    }
                }
                // dv_t reaches the tokens of its own sequence only
#pragma unroll
                for (int k = 0; k < W; ++k)
                    if (pos >= W - 1 - k) {
#pragma unroll
                        for (int j = 0; j < V; ++j) acc[k][j] += dv[j] * w[k][j];
                    }
                shift<W, V>(win);
            }
            const int64_t done = t - (W - 1);
            if (done >= t0 && done < t1) store<T, V>(dx + done * p.xs + e, acc[0]);
            shift<W, V>(acc);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[W - 1][j] = 0.f;
        }
    }
    if (wave) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int k = 0; k < W; ++k) ex[wave - 1][k][j][lane] = dw[k][j];
            ex[wave - 1][W][j][lane] = db[j];
        }
    }
    __syncthreads();
    if (wave || !live) return;
#pragma unroll
    for (int o = 0; o < 3; ++o)
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][j] += ex[o][k][j][lane];
            db[j] += ex[o][W][j][lane];
        }
    float* q = p.part + strip * (W + 1) * p.E + e;
#pragma unroll
    for (int k = 0; k < W; ++k) store<float, V>(q + (int64_t)k * p.E, dw[k]);
    store<float, V>(q + (int64_t)W * p.E, db);
}

// ---- host ---------------------------------------------------------------------------------

// 65536 packed tokens x 1792 channels, bf16: runs of 16 tokens by vectors of 4
// channels 98 us; 8 by 4 104, 32 by 4 106, 16 by 8 115, 8 by 8 117 (fewer waves
// per SIMD to hide the loads).  As it stands now: 92 us, 5.1 TB/s.
constexpr int kFwdTile = 16, kShortTile = 4;
constexpr int kFwdVec = 4;
constexpr int kBwdTile = 16, kBwdShortTile = 8;
constexpr int kBwdVec = 4, kBwdShortVec = 2;

// Channels a thread: fewer than a vector's are taken one by one.
int vec_of(int32_t channels, int vec) { return channels >= vec ? vec : 1; }

struct ConvBwdPlan {
    int64_t tiles, strips;
    int32_t tile, vec, tiles_per_row, iters;
};

ConvBwdPlan conv_bwd_plan(const ssd_conv_dims& d) {
    ConvBwdPlan pl;
    const int64_t len = d.seqlen, rows = d.batch;  // packed: one row
    // Runs of 16 tokens by 4 channels re-read 2 (W - 1) / 16 of their rows, those
    // of 8 twice that (32768 tokens x 1792 channels: 95 us against 110, bf16; 155
    // against 165, float32).  Where tokens are few, runs of 8 by 2 channels give
    // enough waves to hide the loads (4096 tokens, float32: 25.7 us, by 4 channels
    // 29.4, 16 by 4 30.0).
    const bool many = rows * cdiv(len, kBwdTile) * cdiv(d.channels, 64 * kBwdVec) >= 4 * 1024;
    pl.vec = vec_of(d.channels, many ? kBwdVec : kBwdShortVec);
    pl.tile = pl.vec == kBwdVec ? kBwdTile : kBwdShortTile;
    const int64_t groups = cdiv(cdiv(d.channels, pl.vec), 64);
    pl.tiles_per_row = (int32_t)imax(1, cdiv(len, pl.tile));
    pl.tiles = len == 0 ? 0 : rows * pl.tiles_per_row;
    // more tiles a wave (fewer partial rows) only while every CU keeps eight
    // workgroups
    const int64_t it = pl.tiles * groups / (4 * 256 * 8);
    pl.iters = (int32_t)(it < 1 ? 1 : (it > 8 ? 8 : it));
    pl.strips = imax(1, cdiv(pl.tiles, 4 * pl.iters));
    return pl;
}

int conv_check(const ssd_conv_dims* d) {
    if (!d) return SSD_ERR_NULL_ARG;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->batch < 1 || d->seqlen < 0 || d->seqlen > kMaxTokens || d->channels < 1 ||
        d->channels > kMaxStride || d->nseq < 0 || (d->nseq > 0 && d->batch != 1) ||
        (int64_t)d->batch * d->seqlen > kMaxTokens)
        return SSD_ERR_SHAPE;
    if (d->width < 2 || d->width > 4) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int conv_layout(const ssd_conv_dims& d, const ssd_conv_layout* lay, bool bwd, ssd_conv_layout* l) {
    const int64_t E = d.channels;
    *l = {E, E, E};
    if (lay) *l = *lay;
    if (l->x_token < E || l->x_token > kMaxStride) return SSD_ERR_SHAPE;
    const int64_t o = bwd ? l->dy_token : l->y_token;
    if (o < E || o > kMaxStride) return SSD_ERR_SHAPE;
    return SSD_OK;
}

size_t conv_state_bytes(const ssd_conv_dims& d) {
    const int64_t S = d.nseq > 0 ? d.nseq : d.batch;
    return (size_t)S * (d.width - 1) * d.channels * elem_size(d.dtype);
}

ConvParams conv_params(const ssd_conv_dims& d, const ssd_conv_layout& l, const int32_t* cu, int V) {
    ConvParams p = {};
    p.cu = cu;
    p.xs = l.x_token;
    p.L = d.seqlen;
    p.T = (int64_t)d.batch * d.seqlen;
    p.E = d.channels;
    p.nseq = d.nseq;
    p.S = d.nseq > 0 ? d.nseq : d.batch;
    p.nvec = (int32_t)cdiv(d.channels, V);
    return p;
}

template <typename T, int V, int TT>
void launch_conv_fwd(const ConvParams& p, int W, dim3 grid, hipStream_t s) {
    if (W == 2) conv_fwd_kernel<T, 2, V, TT><<<grid, dim3(256), 0, s>>>(p);
    else if (W == 3) conv_fwd_kernel<T, 3, V, TT><<<grid, dim3(256), 0, s>>>(p);
    else conv_fwd_kernel<T, 4, V, TT><<<grid, dim3(256), 0, s>>>(p);
}
template <typename T>
void launch_conv_fwd(const ConvParams& p, int W, int V, int tt, dim3 grid, hipStream_t s) {
    if (V == 1) launch_conv_fwd<T, 1, kShortTile>(p, W, grid, s);
    else if (tt == kFwdTile) launch_conv_fwd<T, kFwdVec, kFwdTile>(p, W, grid, s);
    else launch_conv_fwd<T, kFwdVec, kShortTile>(p, W, grid, s);
}

template <typename T, int V, int TT>
void launch_conv_bwd(const ConvParams& p, int W, dim3 grid, hipStream_t s) {
    if (W == 2) conv_bwd_kernel<T, 2, V, TT><<<grid, dim3(256), 0, s>>>(p);
    else if (W == 3) conv_bwd_kernel<T, 3, V, TT><<<grid, dim3(256), 0, s>>>(p);
    else conv_bwd_kernel<T, 4, V, TT><<<grid, dim3(256), 0, s>>>(p);
}
template <typename T>
void launch_conv_bwd(const ConvParams& p, int W, int V, dim3 grid, hipStream_t s) {
    if (V == 1) launch_conv_bwd<T, 1, kBwdShortTile>(p, W, grid, s);
    else if (V == kBwdVec) launch_conv_bwd<T, kBwdVec, kBwdTile>(p, W, grid, s);
    else launch_conv_bwd<T, kBwdShortVec, kBwdShortTile>(p, W, grid, s);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_conv_fwd(const ssd_conv_dims* dims, const ssd_conv_layout* layout, const void* x,
                 const float* weight, const float* bias, const void* init_state,
                 const int32_t* cu_seqlens, void* y, void* final_state, void* stream) {
    int st = conv_check(dims);
    if (st != SSD_OK) return st;
    const ssd_conv_dims& d = *dims;
    ssd_conv_layout l;
    if ((st = conv_layout(d, layout, false, &l)) != SSD_OK) return st;
    if ((d.nseq > 0) != (cu_seqlens != nullptr)) return cu_seqlens ? SSD_ERR_SHAPE : SSD_ERR_NULL_ARG;
    const int64_t T = (int64_t)d.batch * d.seqlen;
    if (!weight || (T > 0 && (!x || !y))) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(d.dtype);
    for (const void* q : {x, (const void*)y, init_state, (const void*)final_state})
        if (!elem_aligned(q, e)) return SSD_ERR_ALIGN;
    for (const void* q : {(const void*)weight, (const void*)bias, (const void*)cu_seqlens})
        if (!elem_aligned(q, 4)) return SSD_ERR_ALIGN;
    const size_t sb = conv_state_bytes(d);
    if (overlaps(init_state, sb, final_state, sb)) return SSD_ERR_OVERLAP;
    hipStream_t s = (hipStream_t)stream;
    if (cu_seqlens && check_cu_env(cu_seqlens, d.nseq, T, s, &st)) return st;
    const int V = vec_of(d.channels, kFwdVec);
    ConvParams p = conv_params(d, l, cu_seqlens, V);
    p.x = x;
    p.weight = weight;
    p.bias = bias;
    p.init = init_state;
    p.out = y;
    p.os = l.y_token;
    p.state_out = final_state;
    // runs of 16 tokens where that still gives every SIMD a wave, else of 4
    const int64_t len = d.seqlen;
    const int tt = V > 1 && (int64_t)d.batch * cdiv(len, kFwdTile) * p.nvec >= 4 * 256 * 64
                       ? kFwdTile : kShortTile;
    p.tiles_per_row = (int32_t)imax(1, cdiv(len, tt));
    p.main_blocks = len == 0 ? 0 : cdiv((int64_t)d.batch * p.tiles_per_row * p.nvec, 256);
    p.state_items = final_state ? (int64_t)p.S * (d.width - 1) * p.nvec : 0;
    const int64_t grid = p.main_blocks + cdiv(p.state_items, 256);
    if (grid == 0) return SSD_OK;
    if (grid * 256 > kMaxThreads) return SSD_ERR_SHAPE;
    const dim3 gd((unsigned)grid);
    if (d.dtype == SSD_BF16) launch_conv_fwd<bf16>(p, d.width, V, tt, gd, s);
    else launch_conv_fwd<float>(p, d.width, V, tt, gd, s);
    return launched();
}

size_t ssd_conv_bwd_workspace_bytes(const ssd_conv_dims* dims) {
    if (conv_check(dims) != SSD_OK) return 0;
    const ConvBwdPlan pl = conv_bwd_plan(*dims);
    return up256((size_t)pl.strips * (dims->width + 1) * dims->channels * sizeof(float));
}

int ssd_conv_bwd(const ssd_conv_dims* dims, const ssd_conv_layout* layout, const void* x,
                 const float* weight, const float* bias, const void* init_state,
                 const int32_t* cu_seqlens, const void* dy, const void* d_final, void* dx,
                 float* dweight, float* dbias, void* dinit_state, void* workspace,
                 size_t workspace_bytes, void* stream) {
    int st = conv_check(dims);
    if (st != SSD_OK) return st;
    const ssd_conv_dims& d = *dims;
    ssd_conv_layout l;
    if ((st = conv_layout(d, layout, true, &l)) != SSD_OK) return st;
    if ((d.nseq > 0) != (cu_seqlens != nullptr)) return cu_seqlens ? SSD_ERR_SHAPE : SSD_ERR_NULL_ARG;
    const int64_t T = (int64_t)d.batch * d.seqlen;
    if (!weight || (T > 0 && (!x || !dy || !dx))) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(d.dtype);
    for (const void* q : {x, dy, (const void*)dx, init_state, d_final, (const void*)dinit_state})
        if (!elem_aligned(q, e)) return SSD_ERR_ALIGN;
    for (const void* q : {(const void*)weight, (const void*)bias, (const void*)cu_seqlens,
                          (const void*)dweight, (const void*)dbias})
        if (!elem_aligned(q, 4)) return SSD_ERR_ALIGN;
    if ((uintptr_t)workspace & 255) return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < ssd_conv_bwd_workspace_bytes(dims)) return SSD_ERR_WORKSPACE;
    const size_t sb = conv_state_bytes(d);
    if (overlaps(d_final, sb, dinit_state, sb)) return SSD_ERR_OVERLAP;
    hipStream_t s = (hipStream_t)stream;
    if (cu_seqlens && check_cu_env(cu_seqlens, d.nseq, T, s, &st)) return st;
    const ConvBwdPlan pl = conv_bwd_plan(d);
    ConvParams p = conv_params(d, l, cu_seqlens, pl.vec);
    p.x = x;
    p.weight = weight;
    p.bias = bias;
    p.init = init_state;
    p.dy = dy;
    p.gs = l.dy_token;
    p.d_final = d_final;
    p.out = dx;
    p.os = l.x_token;
    p.state_out = dinit_state;
    p.part = (float*)workspace;
    p.tiles_per_row = pl.tiles_per_row;
    p.iters = pl.iters;
    p.tiles = pl.tiles;
    // with no tokens one strip of workgroups still writes the sums' zeros
    p.main_blocks = pl.strips * cdiv(p.nvec, 64);
    p.state_items = dinit_state ? (int64_t)p.S * (d.width - 1) * p.nvec : 0;
    const int64_t grid = p.main_blocks + cdiv(p.state_items, 256);
    if (grid * 256 > kMaxThreads) return SSD_ERR_SHAPE;
    if (d.dtype == SSD_BF16) launch_conv_bwd<bf16>(p, d.width, pl.vec, dim3((unsigned)grid), s);
    else launch_conv_bwd<float>(p, d.width, pl.vec, dim3((unsigned)grid), s);
    if ((st = launched()) != SSD_OK || (!dweight && !dbias)) return st;
    ColSum c = {};
    c.part = p.part;
    c.rows = pl.strips;
    c.cols = (int64_t)(d.width + 1) * d.channels;
    c.out0 = dweight;
    c.c0 = (int64_t)d.width * d.channels;
    c.out1 = dbias;
    c.c1 = d.channels;
    return launch_colsum(c, s);
}

}  // extern "C"
