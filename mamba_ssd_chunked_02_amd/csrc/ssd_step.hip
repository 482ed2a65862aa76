// Single-token forms: one new token for each of b sequences whose states lie
// in a pool of nslots rows (slots[i] is sequence i's row).
//
//   ssd_step          h = e^-d h + d B x^T,  y = C h        (h: N x P per head)
//   ssd_selscan_step  h_n = e^(d A_n) h_n + d B_n x,  y = (C h + D x) silu(z)
//   ssd_conv_step     y = silu(b + w . [state, x]), state shifted by one
//   ssd_linattn_step  S = e^decay S + k v^T,  y = scale q S   (S: K x V per head)
//
// All are bound by the state, read once and written once; every thread
// holds its part of it in registers between the two, so the same buffer may
// be updated in place.
#include "ssd_layer.h"

namespace ssd {
namespace {

// The pool row of batch entry i, or -1 for a padding row.
__device__ __forceinline__ int64_t pool_row(const int32_t* slots, int32_t nslots, int64_t i) {
    const int64_t s = slots ? slots[i] : i;
    return s >= 0 && s < nslots ? s : -1;
}

// ---- SSD ----------------------------------------------------------------------------------

struct StepParams {
    const void* x;
    const void* d_raw;
    const void* B;
    const void* C;
    void* y;
    const float* state;
    float* new_state;
    const int32_t* slots;
    int64_t xs_t, xs_h, ds_t, ds_h, bs_t, bs_g, cs_t, cs_g, ys_t, ys_h;
    float d_init;
    int32_t nslots, H, P, N, hpg, pieces;
};

// 64 sequences x 80 heads x 64 x 128 states: 65.9 us, 5.1 TB/s, what a copy of
// this size reaches (75 with loads predicated by row).  With 64 states (128
// sequences) 63.3 us, 5.3 TB/s; with 32 (256) 91.7, 3.7, and with 16 (512) 151, 2.3:
// there 6 and 7 of a thread's 8 loads repeat the state's last row.
// A workgroup takes CP headdim columns of one head: CP / 4 lanes across, the
// other threads down the state rows, at most UN rows each at a time (all
// their loads in flight together).
template <typename T, int CP>
__global__ __launch_bounds__(256) void step_kernel(StepParams p) {
    constexpr int PL = CP / 4, ROWS = 256 / PL, UN = 8;
    __shared__ float ex[4][CP];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    uint32_t id = blockIdx.x;
    const int piece = id % (uint32_t)p.pieces;
    id /= (uint32_t)p.pieces;
    const int h = id % (uint32_t)p.H;
    const int64_t b = id / (uint32_t)p.H;
    const int g = h / p.hpg;
    const int n0 = tid / PL;
    int c = piece * CP + (tid % PL) * 4;
    const bool own = c < p.P;  // P is a multiple of 16
    c = own ? c : p.P - 4;
    const int64_t row = pool_row(p.slots, p.nslots, b);
    T* y = (T*)p.y + b * p.ys_t + h * p.ys_h;
    if (row < 0) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        if (n0 == 0 && own) store_vec<T, 4>(y + c, 4, zero);
        return;
    }
    const int64_t at = (row * p.H + h) * (int64_t)p.N * p.P + c;
    const float* in = p.state + at;
    float* out = p.new_state + at;
    const T* B = (const T*)p.B + b * p.bs_t + g * p.bs_g;
    const T* C = (const T*)p.C + b * p.cs_t + g * p.cs_g;
    const float d = step_softplus((float)((const T*)p.d_raw)[b * p.ds_t + h * p.ds_h] + p.d_init);
    const float decay = fexp2(-d * kLog2e);
    float u[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
    load_vec<T, 4>((const T*)p.x + b * p.xs_t + h * p.xs_h + c, 4, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] *= d;
    for (int nb = 0; nb < p.N; nb += ROWS * UN) {
        float s[UN][4], bv[UN], cv[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int n = min(nb + i * ROWS + n0, p.N - 1);
            load_vec<float, 4>(in + (int64_t)n * p.P, 4, s[i]);
            bv[i] = (float)B[n];
            cv[i] = (float)C[n];
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int n = nb + i * ROWS + n0;
            if (n >= p.N) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = decay * s[i][j] + bv[i] * u[j];
                acc[j] += cv[i] * s[i][j];
            }
            if (own) store_vec<float, 4>(out + (int64_t)n * p.P, 4, s[i]);
        }
    }
    // rows of one wave, then the four waves
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int o = PL; o < 64; o *= 2) acc[j] += __shfl_xor(acc[j], o);
    if (lane < PL) {
#pragma unroll
        for (int j = 0; j < 4; ++j) ex[wave][lane * 4 + j] = acc[j];
    }
    __syncthreads();
    if (tid < CP && piece * CP + tid < p.P)
        y[piece * CP + tid] = (T)(ex[0][tid] + ex[1][tid] + ex[2][tid] + ex[3][tid]);
}

// ---- selective scan -----------------------------------------------------------------------

struct SelStepParams {
    const void* x;
    const void* d_raw;
    const void* B;
    const void* C;
    const void* z;
    void* y;
    const float* d_init;
    const float* A;
    const float* D;
    const float* state;
    float* new_state;
    const int32_t* slots;
    int64_t xs, ds, zs, ys, bs_t, bs_g, cs_t, cs_g, items;
    int32_t nslots, E, N, epg, vpg, G;
};

// A thread takes V channels of one sequence, all their state entries.  Small
// workgroups even out over the CUs: 128 sequences x 5120 channels x 16 states 26.1
// us with 64 or 128 threads, 27.3 with 256, 32.4 with 512; two channels a thread or
// all 16 entries at once are no faster (27.5 to 34).  As it stands now: 20.2 us,
// 4.4 TB/s.
constexpr int kSelThreads = 128;

template <typename T, int V>
__global__ __launch_bounds__(kSelThreads) void selscan_step_kernel(SelStepParams p) {
    constexpr int UN = 8;
    const int64_t id = (int64_t)blockIdx.x * kSelThreads + threadIdx.x;
    if (id >= p.items) return;
    const uint32_t per = (uint32_t)(p.vpg * p.G);
    const int64_t b = (uint32_t)id / per;
    const uint32_t v = (uint32_t)id % per;
    const int g = v / (uint32_t)p.vpg, at = (v % (uint32_t)p.vpg) * V;
    const int off = min(at, p.epg - V), skip = at - off, e = g * p.epg + off;
    T* y = (T*)p.y + b * p.ys + e;
    const int64_t row = pool_row(p.slots, p.nslots, b);
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    if (row < 0) {
        store_own<T, V>(y, skip, acc);
        return;
    }
    const float* in = p.state + row * (int64_t)p.N * p.E + e;
    float* out = p.new_state + row * (int64_t)p.N * p.E + e;
    const float* A = p.A + e;
    const T* B = (const T*)p.B + b * p.bs_t + g * p.bs_g;
    const T* C = (const T*)p.C + b * p.cs_t + g * p.cs_g;
    float x[V], d[V], u[V], r[V];
    load_vec<T, V>((const T*)p.x + b * p.xs + e, V, x);
    load_vec<T, V>((const T*)p.d_raw + b * p.ds + e, V, d);
    load_vec<float, V>(p.d_init + e, V, r);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        d[j] = step_softplus(d[j] + r[j]);
        u[j] = d[j] * x[j];
        d[j] *= kLog2e;
    }
    for (int n0 = 0; n0 < p.N; n0 += UN) {
        float s[UN][V], a[UN][V];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int n = min(n0 + i, p.N - 1);
            load_vec<float, V>(in + (int64_t)n * p.E, V, s[i]);
            load_vec<float, V>(A + (int64_t)n * p.E, V, a[i]);
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int n = n0 + i;
            if (n >= p.N) break;
            const float bn = (float)B[n], cn = (float)C[n];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[i][j] = fexp2(d[j] * finite_rate(a[i][j])) * s[i][j] + bn * u[j];
                acc[j] += cn * s[i][j];
            }
            store_own<float, V>(out + (int64_t)n * p.E, skip, s[i]);
        }
    }
    if (p.D) {
        load_vec<float, V>(p.D + e, V, r);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += r[j] * x[j];
    }
    if (p.z) {
        load_vec<T, V>((const T*)p.z + b * p.zs + e, V, r);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] *= r[j] * sigmoid(r[j]);
    }
    store_own<T, V>(y, skip, acc);
}

// ---- convolution --------------------------------------------------------------------------

struct ConvStepParams {
    const void* x;
    const void* state;
    void* y;
    void* new_state;
    const float* weight;
    const float* bias;
    const int32_t* slots;
    int64_t xs, ys, items;
    int32_t nslots, E, nvec;
};

template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepParams p) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= p.items) return;
    const int64_t b = (uint32_t)id / (uint32_t)p.nvec;
    const int at = (uint32_t)id % (uint32_t)p.nvec * V, e = min(at, p.E - V), skip = at - e;
    T* y = (T*)p.y + b * p.ys + e;
    const int64_t row = pool_row(p.slots, p.nslots, b);
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.f;
    if (row < 0) {
        store_own<T, V>(y, skip, v);
        return;
    }
    const T* in = (const T*)p.state + row * (int64_t)(W - 1) * p.E + e;
    T* out = (T*)p.new_state + row * (int64_t)(W - 1) * p.E + e;
    float t[W][V], w[W][V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_vec<T, V>(in + (int64_t)k * p.E, V, t[k]);
    load_vec<T, V>((const T*)p.x + b * p.xs + e, V, t[W - 1]);
#pragma unroll
    for (int k = 0; k < W; ++k) load_vec<float, V>(p.weight + (int64_t)k * p.E + e, V, w[k]);
    if (p.bias) load_vec<float, V>(p.bias + e, V, v);
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += t[k][j] * w[k][j];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_own<T, V>(out + (int64_t)k * p.E, skip, t[k + 1]);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= sigmoid(v[j]);
    store_own<T, V>(y, skip, v);
}

// ---- linear attention ---------------------------------------------------------------------

struct LinStepParams {
    const void* q;
    const void* k;
    const void* v;
    void* y;
    const float* decay;
    const float* state;
    float* new_state;
    const int32_t* slots;
    int64_t qs_t, qs_h, ks_t, ks_g, vs_t, vs_g, ys_t, ys_h;
    float scale;
    int32_t nslots, H, K, V, hpg, pieces;
};

// A workgroup takes CP value columns of one head: CP / VW lanes across (VW columns each,
// the last vector moved back to end with the row), the other threads down the state's
// rows, UN rows in flight each.  Bound by memory: 64 sequences x 32 heads of 128 x 128 (270 MB) 46
// us where the states are in the 256 MB cache in part, 58 where they are not (4.7 TB/s).
template <typename T, int CP, int VW>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinStepParams p) {
    constexpr int PL = CP / VW, ROWS = 256 / PL, UN = 8;
    __shared__ float ex[4][CP];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    uint32_t id = blockIdx.x;
    const int piece = id % (uint32_t)p.pieces;
    id /= (uint32_t)p.pieces;
    const int h = id % (uint32_t)p.H;
    const int64_t b = id / (uint32_t)p.H;
    const int g = h / p.hpg, k0 = tid / PL, at = piece * CP + (tid % PL) * VW;
    const bool own = at < p.V;
    const int c = min(at, p.V - VW), skip = min(at - c, VW);
    const int64_t row = pool_row(p.slots, p.nslots, b);
    T* y = (T*)p.y + b * p.ys_t + h * p.ys_h;
    float acc[VW];
#pragma unroll
    for (int j = 0; j < VW; ++j) acc[j] = 0.f;
    if (row < 0) {
        if (k0 == 0 && own) store_own<T, VW>(y + c, skip, acc);
        return;
    }
    const int64_t base = (row * p.H + h) * ((int64_t)p.K * p.V) + c;
    const float* in = p.state + base;
    float* out = p.new_state + base;
    const T* q = (const T*)p.q + b * p.qs_t + h * p.qs_h;
    const T* k = (const T*)p.k + b * p.ks_t + g * p.ks_g;
    const float rate = expf(p.decay[h]);
    float v[VW];
    load_vec<T, VW>((const T*)p.v + b * p.vs_t + g * p.vs_g + c, VW, v);
    for (int kb = 0; kb < p.K; kb += ROWS * UN) {
        float s[UN][VW], qv[UN], kv[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int n = min(kb + i * ROWS + k0, p.K - 1);
            load_vec<float, VW>(in + n * p.V, VW, s[i]);
            qv[i] = (float)q[n];
            kv[i] = (float)k[n];
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int n = kb + i * ROWS + k0;
            if (n >= p.K) break;
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                s[i][j] = rate * s[i][j] + kv[i] * v[j];
                acc[j] += qv[i] * s[i][j];
            }
            if (own) store_own<float, VW>(out + n * p.V, skip, s[i]);
        }
    }
    // rows of one wave, then the four waves
#pragma unroll
    for (int j = 0; j < VW; ++j)
#pragma unroll
        for (int o = PL; o < 64; o *= 2) acc[j] += __shfl_xor(acc[j], o);
    if (lane < PL) {
#pragma unroll
        for (int j = 0; j < VW; ++j) ex[wave][lane * VW + j] = acc[j];
    }
    __syncthreads();
    if (tid < PL && own) {
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            const int x = tid * VW + j;
            acc[j] = p.scale * (ex[0][x] + ex[1][x] + ex[2][x] + ex[3][x]);
        }
        store_own<T, VW>(y + c, skip, acc);
    }
}

// in place, or two pools that share nothing
bool pools_ok(const void* a, const void* b, size_t bytes) {
    return a == b || !overlaps(a, bytes, b, bytes);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_step(const ssd_dims* dims, const ssd_layout* layout, const void* x, const void* d_raw,
             float d_init, const void* B, const void* C, const float* state, const int32_t* slots,
             int32_t nslots, void* y, float* new_state, void* stream) {
    if (!dims) return SSD_ERR_NULL_ARG;
    const ssd_dims& d = *dims;
    if (d.dtype != SSD_F32 && d.dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d.batch < 0 || d.seqlen != 1 || d.nseq != 0 || d.nheads < 1 || d.headdim < 16 ||
        d.headdim > 512 || d.headdim % 16 || d.ngroups < 1 || d.nheads % d.ngroups || nslots < 0 ||
        (!slots && nslots < d.batch))
        return SSD_ERR_SHAPE;
    if (d.d_state != 16 && d.d_state != 32 && d.d_state != 64 && d.d_state != 128 &&
        d.d_state != 256)
        return SSD_ERR_UNSUPPORTED;
    const int64_t HP = (int64_t)d.nheads * d.headdim, GN = (int64_t)d.ngroups * d.d_state;
    if (HP > kMaxStride || GN > kMaxStride) return SSD_ERR_SHAPE;
    ssd_layout l;
    if (layout) {
        l = *layout;
    } else {
        l.x_token = l.y_token = HP;
        l.x_head = l.y_head = d.headdim;
        l.d_raw_token = d.nheads;
        l.d_raw_head = 1;
        l.B_token = l.C_token = GN;
        l.B_group = l.C_group = d.d_state;
    }
    for (int64_t s : {l.x_token, l.x_head, l.d_raw_token, l.d_raw_head, l.B_token, l.B_group,
                      l.C_token, l.C_group, l.y_token, l.y_head})
        if (s < 0 || s > kMaxStride) return SSD_ERR_SHAPE;
    if (d.batch == 0) return SSD_OK;
    if (!rows_apart(d.batch, l.y_token, d.nheads, l.y_head, d.headdim)) return SSD_ERR_SHAPE;
    if (!x || !d_raw || !B || !C || !y) return SSD_ERR_NULL_ARG;
    if (nslots > 0 && (!state || !new_state)) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(d.dtype);
    for (const void* q : {x, d_raw, B, C, (const void*)y})
        if (!elem_aligned(q, e)) return SSD_ERR_ALIGN;
    if (!elem_aligned(state, 4) || !elem_aligned(new_state, 4) || !elem_aligned(slots, 4))
        return SSD_ERR_ALIGN;
    if (!pools_ok(state, new_state, (size_t)nslots * HP * d.d_state * 4)) return SSD_ERR_OVERLAP;
    // 64 columns a workgroup; 16 where that leaves CUs without one
    const int64_t heads = (int64_t)d.batch * d.nheads;
    const int cp = heads * cdiv(d.headdim, 64) >= 256 && d.headdim > 16 ? 64 : 16;
    StepParams p = {};
    p.x = x;
    p.d_raw = d_raw;
    p.B = B;
    p.C = C;
    p.y = y;
    p.state = state;
    p.new_state = new_state;
    p.slots = slots;
    p.xs_t = l.x_token;
    p.xs_h = l.x_head;
    p.ds_t = l.d_raw_token;
    p.ds_h = l.d_raw_head;
    p.bs_t = l.B_token;
    p.bs_g = l.B_group;
    p.cs_t = l.C_token;
    p.cs_g = l.C_group;
    p.ys_t = l.y_token;
    p.ys_h = l.y_head;
    p.d_init = d_init;
    p.nslots = nslots;
    p.H = d.nheads;
    p.P = d.headdim;
    p.N = d.d_state;
    p.hpg = d.nheads / d.ngroups;
    p.pieces = (int32_t)cdiv(d.headdim, cp);
    const int64_t grid = heads * p.pieces;
    if (grid * 256 > kMaxThreads) return SSD_ERR_SHAPE;
    const dim3 gd((unsigned)grid), bd(256);
    hipStream_t s = (hipStream_t)stream;
    if (d.dtype == SSD_BF16) {
        if (cp == 64) step_kernel<bf16, 64><<<gd, bd, 0, s>>>(p);
        else step_kernel<bf16, 16><<<gd, bd, 0, s>>>(p);
    } else {
        if (cp == 64) step_kernel<float, 64><<<gd, bd, 0, s>>>(p);
        else step_kernel<float, 16><<<gd, bd, 0, s>>>(p);
    }
    return launched();
}

int ssd_selscan_step(const ssd_selscan_dims* dims, const ssd_selscan_layout* layout, const void* x,
                     const void* d_raw, const float* d_init, const float* A, const void* B,
                     const void* C, const float* D, const void* z, const float* state,
                     const int32_t* slots, int32_t nslots, void* y, float* new_state,
                     void* stream) {
    if (!dims) return SSD_ERR_NULL_ARG;
    const ssd_selscan_dims& d = *dims;
    if (d.dtype != SSD_F32 && d.dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d.batch < 0 || d.seqlen != 1 || d.nseq != 0 || d.channels < 1 ||
        d.channels > SSD_SELSCAN_MAX_CHANNELS || d.ngroups < 1 || d.channels % d.ngroups ||
        d.d_state < 1 || nslots < 0 || (!slots && nslots < d.batch))
        return SSD_ERR_SHAPE;
    if (d.d_state > SSD_SELSCAN_MAX_STATE) return SSD_ERR_UNSUPPORTED;
    const int64_t E = d.channels, N = d.d_state, G = d.ngroups;
    ssd_selscan_layout l = {E, E, E, G * N, N, G * N, N, E, E};
    if (layout) l = *layout;
    if (!z) l.z_token = E;
    for (int64_t s : {l.x_token, l.d_raw_token, l.z_token, l.y_token})
        if (s < E || s > kMaxStride) return SSD_ERR_SHAPE;
    for (int64_t s : {l.B_token, l.B_group, l.C_token, l.C_group})
        if (s < 0 || s > kMaxStride) return SSD_ERR_SHAPE;
    if (d.batch == 0) return SSD_OK;
    if (!x || !d_raw || !d_init || !A || !B || !C || !y) return SSD_ERR_NULL_ARG;
    if (nslots > 0 && (!state || !new_state)) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(d.dtype);
    for (const void* q : {x, d_raw, B, C, z, (const void*)y})
        if (!elem_aligned(q, e)) return SSD_ERR_ALIGN;
    for (const void* q : {(const void*)d_init, (const void*)A, (const void*)D, (const void*)state,
                          (const void*)new_state, (const void*)slots})
        if (!elem_aligned(q, 4)) return SSD_ERR_ALIGN;
    if (!pools_ok(state, new_state, (size_t)nslots * N * E * 4)) return SSD_ERR_OVERLAP;
    SelStepParams p = {};
    p.x = x;
    p.d_raw = d_raw;
    p.B = B;
    p.C = C;
    p.z = z;
    p.y = y;
    p.d_init = d_init;
    p.A = A;
    p.D = D;
    p.state = state;
    p.new_state = new_state;
    p.slots = slots;
    p.xs = l.x_token;
    p.ds = l.d_raw_token;
    p.zs = l.z_token;
    p.ys = l.y_token;
    p.bs_t = l.B_token;
    p.bs_g = l.B_group;
    p.cs_t = l.C_token;
    p.cs_g = l.C_group;
    p.nslots = nslots;
    p.E = d.channels;
    p.N = d.d_state;
    p.G = d.ngroups;
    p.epg = d.channels / d.ngroups;
    // four channels a thread (16-byte state rows) where that still gives every
    // CU a workgroup
    const bool wide = (int64_t)d.batch * E >= (int64_t)4 * 256 * 256 && p.epg >= 4;
    p.vpg = (int32_t)cdiv(p.epg, wide ? 4 : 1);
    p.items = (int64_t)d.batch * p.vpg * G;
    if (p.items > INT32_MAX) return SSD_ERR_SHAPE;
    const dim3 gd((unsigned)cdiv(p.items, kSelThreads)), bd(kSelThreads);
    hipStream_t s = (hipStream_t)stream;
    if (d.dtype == SSD_BF16) {
        if (wide) selscan_step_kernel<bf16, 4><<<gd, bd, 0, s>>>(p);
        else selscan_step_kernel<bf16, 1><<<gd, bd, 0, s>>>(p);
    } else {
        if (wide) selscan_step_kernel<float, 4><<<gd, bd, 0, s>>>(p);
        else selscan_step_kernel<float, 1><<<gd, bd, 0, s>>>(p);
    }
    return launched();
}

int ssd_conv_step(const ssd_conv_dims* dims, const ssd_conv_layout* layout, const void* x,
                  const float* weight, const float* bias, const void* state, const int32_t* slots,
                  int32_t nslots, void* y, void* new_state, void* stream) {
    if (!dims) return SSD_ERR_NULL_ARG;
    const ssd_conv_dims& d = *dims;
    if (d.dtype != SSD_F32 && d.dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d.batch < 0 || d.seqlen != 1 || d.nseq != 0 || d.channels < 1 || d.channels > kMaxStride ||
        nslots < 0 || (!slots && nslots < d.batch))
        return SSD_ERR_SHAPE;
    if (d.width < 2 || d.width > 4) return SSD_ERR_UNSUPPORTED;
    const int64_t E = d.channels;
    ssd_conv_layout l = {E, E, E};
    if (layout) l = *layout;
    if (l.x_token < E || l.x_token > kMaxStride || l.y_token < E || l.y_token > kMaxStride)
        return SSD_ERR_SHAPE;
    if (d.batch == 0) return SSD_OK;
    if (!x || !weight || !y) return SSD_ERR_NULL_ARG;
    if (nslots > 0 && (!state || !new_state)) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(d.dtype);
    for (const void* q : {x, (const void*)y, state, (const void*)new_state})
        if (!elem_aligned(q, e)) return SSD_ERR_ALIGN;
    for (const void* q : {(const void*)weight, (const void*)bias, (const void*)slots})
        if (!elem_aligned(q, 4)) return SSD_ERR_ALIGN;
    if (!pools_ok(state, new_state, (size_t)nslots * (d.width - 1) * E * e)) return SSD_ERR_OVERLAP;
    ConvStepParams p = {};
    p.x = x;
    p.state = state;
    p.y = y;
    p.new_state = new_state;
    p.weight = weight;
    p.bias = bias;
    p.slots = slots;
    p.xs = l.x_token;
    p.ys = l.y_token;
    p.nslots = nslots;
    p.E = d.channels;
    const int V = E >= 4 ? 4 : 1;
    p.nvec = (int32_t)cdiv(E, V);
    p.items = (int64_t)d.batch * p.nvec;
    if (p.items > INT32_MAX) return SSD_ERR_SHAPE;
    const dim3 gd((unsigned)cdiv(p.items, 256)), bd(256);
    hipStream_t s = (hipStream_t)stream;
#define SSD_CONV_STEP(T, V)                                               \
    do {                                                                  \
        if (d.width == 2) conv_step_kernel<T, 2, V><<<gd, bd, 0, s>>>(p);      \
        else if (d.width == 3) conv_step_kernel<T, 3, V><<<gd, bd, 0, s>>>(p); \
        else conv_step_kernel<T, 4, V><<<gd, bd, 0, s>>>(p);                   \
    } while (0)
    if (d.dtype == SSD_BF16) {
        if (V == 4) SSD_CONV_STEP(bf16, 4);
        else SSD_CONV_STEP(bf16, 1);
    } else {
        if (V == 4) SSD_CONV_STEP(float, 4);
        else SSD_CONV_STEP(float, 1);
    }
#undef SSD_CONV_STEP
    return launched();
}

int ssd_linattn_step(const ssd_linattn_dims* dims, const ssd_linattn_layout* layout, const void* q,
                     const void* k, const void* v, const float* decay, const float* state,
                     const int32_t* slots, int32_t nslots, void* y, float* new_state, void* stream) {
    if (!dims) return SSD_ERR_NULL_ARG;
    const ssd_linattn_dims& d = *dims;
    if (d.dtype != SSD_F32 && d.dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d.batch < 0 || d.seqlen != 1 || d.nseq != 0 || d.nheads < 1 || d.ngroups < 1 ||
        d.nheads % d.ngroups || d.keydim < 1 || d.valuedim < 1 || d.reserved != 0 || nslots < 0 ||
        (!slots && nslots < d.batch) || !(d.scale == d.scale) ||
        (int64_t)d.batch * d.nheads > (int64_t)1 << 21)
        return SSD_ERR_SHAPE;
    if (d.keydim > SSD_LINATTN_MAX_DIM || d.valuedim > SSD_LINATTN_MAX_DIM) return SSD_ERR_UNSUPPORTED;
    const int64_t H = d.nheads, G = d.ngroups, K = d.keydim, V = d.valuedim;
    ssd_linattn_layout l = {H * K, K, G * K, K, G * V, V, H * V, V};
    if (layout) l = *layout;
    for (int64_t s : {l.q_token, l.q_head, l.k_token, l.k_group, l.v_token, l.v_group, l.y_token, l.y_head})
        if (s < 0 || s > kMaxStride) return SSD_ERR_SHAPE;
    if (d.batch == 0) return SSD_OK;
    if (!rows_apart(d.batch, l.y_token, H, l.y_head, V)) return SSD_ERR_SHAPE;
    if (!q || !k || !v || !decay || !y) return SSD_ERR_NULL_ARG;
    if (nslots > 0 && (!state || !new_state)) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(d.dtype);
    for (const void* a : {q, k, v, (const void*)y})
        if (!elem_aligned(a, e)) return SSD_ERR_ALIGN;
    for (const void* a : {(const void*)decay, (const void*)state, (const void*)new_state, (const void*)slots})
        if (!elem_aligned(a, 4)) return SSD_ERR_ALIGN;
    if (!pools_ok(state, new_state, (size_t)nslots * H * K * V * 4)) return SSD_ERR_OVERLAP;
    LinStepParams p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.y = y;
    p.decay = decay;
    p.state = state;
    p.new_state = new_state;
    p.slots = slots;
    p.qs_t = l.q_token;
    p.qs_h = l.q_head;
    p.ks_t = l.k_token;
    p.ks_g = l.k_group;
    p.vs_t = l.v_token;
    p.vs_g = l.v_group;
    p.ys_t = l.y_token;
    p.ys_h = l.y_head;
    p.scale = d.scale;
    p.nslots = nslots;
    p.H = d.nheads;
    p.K = d.keydim;
    p.V = d.valuedim;
    p.hpg = d.nheads / d.ngroups;
    // 64 columns a workgroup; 16 where that leaves CUs without one
    const bool wide = d.batch * H * cdiv(V, 64) >= 256 && V > 16;
    p.pieces = (int)cdiv(V, wide ? 64 : 16);
    const dim3 gd((unsigned)(d.batch * H * p.pieces));
    hipStream_t s = (hipStream_t)stream;
#define SSD_LINATTN_STEP(T)                                              \
    do {                                                                 \
        if (V < 4) linattn_step_kernel<T, 16, 1><<<gd, 256, 0, s>>>(p);  \
        else if (wide) linattn_step_kernel<T, 64, 4><<<gd, 256, 0, s>>>(p); \
        else linattn_step_kernel<T, 16, 4><<<gd, 256, 0, s>>>(p);        \
    } while (0)
    if (d.dtype == SSD_BF16) SSD_LINATTN_STEP(bf16);
    else SSD_LINATTN_STEP(float);
#undef SSD_LINATTN_STEP
    return launched();
}

}  // extern "C"
