// Selective scan, forward, the sum that ends the backward pass's dB and dC, and
// the entry points (see ssd_selscan.h).
#include "ssd_selscan.h"

namespace ssd {
namespace {

// ---- what a span does to a state ------------------------------------------------------------

// The wave takes a run of the span's chunks and keeps its state in registers;
// the waves' are joined once at the end.
template <typename T, int NR>
__global__ __launch_bounds__(512) void selscan_span_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kFwdTokens, NP = S::NP, MW = 8, Q = TW / 4;
    __shared__ __align__(16) float bc[MW][TW][2][NP];
    __shared__ __align__(16) float exD[MW][64], exH[MW][64][NR];
    Place o;
    if (!place_of(p, o) || o.k >= o.nspan) return;
    if (o.k == o.nspan - 1) return;  // nothing comes after it
    float A2[NR], h[NR];
    load_rates<NR>(p, o, A2);
    const float dinit = o.live ? p.d_init[o.ch] : 0.f;
    const int chunks = (o.last - o.first + TW - 1) / TW, run = (chunks + MW - 1) / MW;
    const int c0 = min(o.wave * run, chunks), c1 = min(c0 + run, chunks);
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) h[r] = 0.f;
    uint32_t xr[Q], dr[Q];
    Rows<T, NR, TW> Br;
    auto fetch = [&](int t) {
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->x, k->xs, o, t, xr);
        load_tokens<T, TW>(k->d_raw, k->ds, o, t, dr);
        load_rows<T, NR, TW>(k->B, k->bs_t, k->bs_g, k->N, o, t, Br);
    };
    int tb = o.first + c0 * TW;
    if (c0 < c1) fetch(tb);
    for (int c = c0; c < c1; ++c, tb += TW) {
        const int have = min(o.last - tb, TW);
        float d[Q], u[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            d[i] = step_of(value_of<T>(dr[i]) + dinit, 4 * i + o.nl < have);
            u[i] = d[i] * value_of<T>(xr[i]);
            sum += d[i];  // the lane's; the quad's at the end
        }
        wave_lds_fence();
        put_rows<T, NR, TW>(&bc[o.wave][0][0][0], o, Br);
        wave_lds_fence();
        if (c + 1 < c1) fetch(tb + TW);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            float b[NR];
            lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
            const float dt = quad_lane(d[t / 4], t % 4), ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                h[r] = fexp2(dt * A2[r]) * h[r] + b[r] * ut;
            }
            if (t & 1) keep_order();
        }
    }
    sum = quad_total(sum);
    exD[o.wave][o.lane] = sum;
    lds_put<NR>(exH[o.wave][o.lane], h);
    __syncthreads();
    if (o.wave) return;
    for (int j = 1; j < MW; ++j) {
        const float dj = exD[j][o.lane];
        float hj[NR];
        lds_get<NR>(exH[j][o.lane], hj);
#pragma unroll
        for (int r = 0; r < NR; ++r) h[r] = fexp2(dj * A2[r]) * h[r] + hj[r];
        sum += dj;
    }
    const int64_t at = ((int64_t)o.slot * p.nblk + o.blk) * 64 + o.lane;
    p.span_d[at] = sum;
    __builtin_memcpy(p.span_h + at * NR, h, sizeof(h));
}

// ---- forward ------------------------------------------------------------------------------

template <typename T, int NR, int MW>
__global__ __launch_bounds__(64 * MW, Shape<NR>::kFwdPerSimd) void selscan_fwd_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kFwdTokens, NP = S::NP, Q = TW / 4, waves = MW;
    __shared__ __align__(16) float bc[MW][TW][2][NP];
    __shared__ __align__(16) float exP[2][MW][64][NR], exH[2][MW][64][NR];
    __shared__ __align__(16) float enter[2][64][NR];  // the state entering a segment
    Place o;
    if (!place_of(p, o)) return;
    const int seg = waves * TW;
    const bool b0 = o.nl & 1, b1 = o.nl & 2;
    float A2[NR], h[NR];
    load_rates<NR>(p, o, A2);
    const float dinit = o.live ? p.d_init[o.ch] : 0.f;
    const float Dv = o.live && p.D ? p.D[o.ch] : 0.f;
    const uint32_t yoff = o.live ? (uint32_t)(o.nl * p.ys + o.e) * (uint32_t)sizeof(T) : kNowhere;
    const bool gated = p.z != nullptr;
    if (o.k >= o.nspan) return;
    if (o.wave == 0) {
        load_state<NR>(p.init, p, o, h);
        if (p.span) fold_spans<NR>(p, o, A2, h);
        lds_put<NR>(enter[0][o.lane], h);
        if (o.first >= o.last) store_state<NR>(p.final_state, p, o, h);
    }
    const bool ends = o.k == o.nspan - 1;  // the span's last state is the sequence's

    uint32_t xr[Q], dr[Q], zr[Q];
    Rows<T, NR, TW> Br, Cr;
    int tb = o.first + o.wave * TW;
    auto fetch = [&](int t) {
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->x, k->xs, o, t, xr);
        load_tokens<T, TW>(k->d_raw, k->ds, o, t, dr);
        load_rows<T, NR, TW>(k->B, k->bs_t, k->bs_g, k->N, o, t, Br);
        load_rows<T, NR, TW>(k->C, k->cs_t, k->cs_g, k->N, o, t, Cr);
    };
    fetch(tb);
    int turn = 0;
    for (int base = o.first; base < o.last; base += seg, tb += seg, turn ^= 1) {
        if (tb >= o.last) {  // in the last segment, and nothing waits for this wave
            __syncthreads();
            break;
        }
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->z, k->zs, o, tb, zr);
        float d[Q], u[Q], x[Q];
        float sumd = 0.f;
        // tokens of this chunk that the sequence has (where fewer: the rest take
        // d = 0, which passes the state on unchanged)
        const int have = min(o.last - tb, TW);
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            x[i] = value_of<T>(xr[i]);
            d[i] = step_of(value_of<T>(dr[i]) + dinit, 4 * i + o.nl < have);
            u[i] = d[i] * x[i];
            sumd += d[i];
        }
        sumd = quad_total(sumd);
        put_rows<T, NR, TW>(&bc[o.wave][0][0][0], o, Br);
        put_rows<T, NR, TW>(&bc[o.wave][0][1][0], o, Cr);
        wave_lds_fence();

        float a[TW][NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) h[r] = fexp2(sumd * A2[r]);
        lds_put<NR>(exP[turn][o.wave][o.lane], h);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            float b[NR];
            lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
            const float dt = quad_lane(d[t / 4], t % 4), ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                a[t][r] = fexp2(dt * A2[r]);
                h[r] = t ? a[t][r] * h[r] + b[r] * ut : b[r] * ut;
            }
            if (t & 1) keep_order();
        }
        lds_put<NR>(exH[turn][o.wave][o.lane], h);
        // the exchange is double-buffered: a wave is at most one barrier ahead
        __syncthreads();
        // the state entering this chunk
        lds_get<NR>(enter[turn][o.lane], h);
        for (int j = 0; j < o.wave; ++j) {
            float Pj[NR], hj[NR];
            lds_get<NR>(exP[turn][j][o.lane], Pj);
            lds_get<NR>(exH[turn][j][o.lane], hj);
#pragma unroll
            for (int r = 0; r < NR; ++r) h[r] = Pj[r] * h[r] + hj[r];
        }
        keep_order();
        const RowBuf<T> y = row_buf<T>(k->y, k->ys, o.ch0, tb, have, o.width);
        const uint32_t yat = fresh(yoff);
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            // the next segment's rows, once half of a is used up
            if (i == Q / 2) fetch(tb + seg);
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 4 * i + k;
                float b[NR], c[NR];
                lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
                lds_get<NR>(&bc[o.wave][t][1][o.nl * NR], c);
                const float ut = quad_lane(u[i], k);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    h[r] = a[t][r] * h[r] + b[r] * ut;
                    v[k] = r ? v[k] + c[r] * h[r] : c[r] * h[r];
                }
                if (k & 1) keep_order();
            }
            float out = quad_sums(v[0], v[1], v[2], v[3], b0, b1) + Dv * x[i];
            const float zf = value_of<T>(zr[i]);
            out *= gated ? zf * sigmoid(zf) : 1.f;
            y.put(yat + i * (uint32_t)(4 * k->ys * sizeof(T)), out);
            keep_order();
        }
        // the segment's last chunk leaves the state that enters the next one;
        // its slot was last read before the barrier that this wave has passed
        if (o.last - base <= seg) {
            if (ends && o.last - tb <= TW) store_state<NR>(p.final_state, p, o, h);
        } else if (o.wave == waves - 1) {
            lds_put<NR>(enter[turn ^ 1][o.lane], h);
        }
        wave_lds_fence();  // the next segment's rows go where these were read
    }
}

// dB and dC: the sum over a group's channel blocks, in order.
template <typename T>
__global__ __launch_bounds__(256) void selscan_bc_kernel(SelParams p, void* dB, void* dC, int NP) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row = 2 * NP;
    const int64_t tg = id / row;
    const int j = (int)(id % row), n = j % NP;
    const int64_t t = tg / p.G;
    const int g = (int)(tg % p.G);
    if (t >= p.T || n >= p.N) return;
    const float* q = p.part_bc + ((int64_t)g * p.bpg * p.T + t) * row + j;
    const int64_t step = p.T * row;
    float s = 0.f;
    int b = 0;
    for (; b + 8 <= p.bpg; b += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = q[(b + k) * step];
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
    }
    for (; b < p.bpg; ++b) s += q[b * step];
    if (j < NP) ((T*)dB)[t * p.bs_t + g * p.bs_g + n] = (T)s;
    else ((T*)dC)[t * p.cs_t + g * p.cs_g + n] = (T)s;
}

// ---- host ---------------------------------------------------------------------------------

int32_t entries_per_lane(int32_t N) { return N <= 8 ? 2 : (N <= 16 ? 4 : (N <= 32 ? 8 : 16)); }

int sel_check(const ssd_selscan_dims* d) {
    if (!d) return SSD_ERR_NULL_ARG;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->batch < 1 || d->seqlen < 0 || d->seqlen > kMaxTokens || d->channels < 1 ||
        d->channels > SSD_SELSCAN_MAX_CHANNELS || d->ngroups < 1 || d->channels % d->ngroups ||
        d->d_state < 1 || d->nseq < 0 || (d->nseq > 0 && d->batch != 1) ||
        (int64_t)d->batch * d->seqlen > kMaxTokens - 65536)  // token sums stay in 32 bits
        return SSD_ERR_SHAPE;
    if (d->d_state > SSD_SELSCAN_MAX_STATE) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

struct SelPlan {
    int32_t NR, S, bpg, nblk, upr;
    int32_t waves;      // forward: of a workgroup
    int64_t runs;       // backward: of a sequence
    int32_t span, per;  // tokens of a span (0: sequences are not cut), spans a sequence
    int64_t slots, units, grid, T;
    size_t off_h, off_q, off_d, off_ch, off_cd, off_w, off_bc, total;
};

template <typename F>
auto with_shape(int NR, F f) {
    if (NR == 2) return f(Shape<2>{});
    if (NR == 4) return f(Shape<4>{});
    if (NR == 8) return f(Shape<8>{});
    return f(Shape<16>{});
}

// Waves of a forward workgroup.  One workgroup of all the waves that a CU holds
// scans a channel block's tokens the widest; where there are enough workgroups,
// smaller ones do better, because several share a CU without waiting for each
// other and because fewer waves stand idle in a sequence's last segment.
// Measured with 16 states (us at 16 / 8 / 4 / 2 waves):
//   192 workgroups, 2048 tokens:        51 / 60 / 89 / 177
//   576 workgroups, 2048 tokens:       156 / 151 / 157 / 223
//   1536 workgroups, 256..8192 tokens: 640 / 576 / 550 / 687
//   24576 workgroups, 20 tokens:       479 / 248 / 137 / 86
// With 8, 32 and 64 states there are all the waves or a quarter of them (us, all /
// a quarter; 1536 channels, so 96 workgroups a sequence):
//                                    8 states    32 states    64 states
//   192 workgroups, 2048 tokens:      38 / 61    122 / 323     332 / 630
//   576 workgroups, 2048 tokens:     111 / 104   344 / 388     946 / 800
//   960 workgroups, 2048 tokens:     173 / 150   462 / 406    1268 / 1399
//   1536 workgroups, 2048 tokens:    265 / 218   691 / 517    1902 / 1661
//   6144 workgroups, 130 tokens:     160 / 70    273 / 147     606 / 448
//   24576 workgroups, 20 tokens:     514 / 118   492 / 144     748 / 388
int32_t forward_waves(int NR, int64_t workgroups, int64_t chunks) {
    const int32_t full = with_shape(NR, [](auto s) { return s.kFwdWaves; });
    if (NR != 4) return workgroups >= 1024 || chunks <= full / 4 ? full / 4 : full;
    int32_t w = workgroups >= 1024 ? 4 : workgroups >= 512 ? 8 : 16;
    while (w > 2 && w / 2 >= chunks) w /= 2;
    return w;
}

int sel_plan(const ssd_selscan_dims& d, bool bwd, SelPlan* pl) {
    *pl = {};
    pl->NR = entries_per_lane(d.d_state);
    pl->T = (int64_t)d.batch * d.seqlen;
    pl->S = d.nseq > 0 ? d.nseq : d.batch;
    pl->bpg = (int32_t)cdiv(d.channels / d.ngroups, kChan);
    const int64_t nblk = (int64_t)pl->bpg * d.ngroups;
    pl->nblk = (int32_t)nblk;
    pl->upr = (int32_t)cdiv(nblk, kRun);
    // packed sequences are taken as equally long
    const int64_t len = cdiv(pl->T, pl->S), whole = (int64_t)pl->S * nblk;
    if (bwd) {
        pl->span = with_shape(pl->NR, [](auto s) { return s.kRunTokens; });
        pl->runs = cdiv(len, pl->span);
        pl->per = (int32_t)imax(1, cdiv(d.seqlen, pl->span));
    } else {
        const int64_t tokens = with_shape(pl->NR, [](auto s) { return s.kFwdTokens; });
        pl->waves = forward_waves(pl->NR, whole, cdiv(len, tokens));
        // Cut sequences into spans where that shortens the longest chain of
        // segments on a CU by more than the second launch costs.  A segment's
        // cost is 1; with spans its tokens are walked once more for the spans'
        // states (0.6 of a segment).  Set for 16 states and applied to all.
        const int64_t seg = pl->waves * tokens, nseg = cdiv(len, seg);
        double best = (double)cdiv(whole, 256) * nseg;
        int64_t segs = 0;
        for (int64_t k = 2; k <= 64 && k <= nseg; ++k) {
            const int64_t each = cdiv(nseg, k), spans = cdiv(nseg, each);
            const double cost = (double)cdiv(whole * spans, 256) * each * 1.6 + 1.5 + 0.05 * spans;
            if (cost < best) {
                best = cost;
                segs = each;
            }
        }
        pl->span = (int32_t)(segs * seg);
        pl->per = segs ? (int32_t)cdiv(nseg, segs) : 1;
    }
    pl->slots = d.nseq > 0 && pl->span ? pl->T / pl->span + pl->S : (int64_t)pl->S * pl->per;
    pl->units = pl->slots * pl->upr;
    pl->grid = cdiv(pl->units, kXcds) * kXcds * kRun;
    const int64_t threads = bwd ? 64 : imax(512, 64 * pl->waves);
    if (pl->grid * threads > kMaxThreads || whole * 512 > kMaxThreads) return SSD_ERR_SHAPE;
    size_t off = 0;
    const auto take = [&off](int64_t floats) {
        const size_t at = off;
        off = up256(off + (size_t)floats * sizeof(float));
        return at;
    };
    const int64_t lanes = nblk * 64;
    if (bwd) {
        const int64_t chunks = pl->T / with_shape(pl->NR, [](auto s) { return s.kBwdTokens; }) + pl->slots;
        pl->off_h = take(pl->slots * lanes * pl->NR);
        pl->off_q = take(pl->slots * lanes * pl->NR);
        pl->off_d = take(pl->slots * lanes);
        pl->off_ch = take(chunks * lanes * pl->NR);
        pl->off_cd = take(chunks * lanes);
        pl->off_w = take(pl->slots * (d.d_state + 2) * d.channels);
        pl->off_bc = take(nblk * pl->T * 8 * pl->NR);
    } else if (pl->span) {
        pl->off_h = take(pl->slots * lanes * pl->NR);
        pl->off_d = take(pl->slots * lanes);
    }
    pl->total = off;
    return SSD_OK;
}

// Shared checks and parameters of both directions.
int sel_setup(const ssd_selscan_dims* dims, const ssd_selscan_layout* layout, const void* x,
              const void* d_raw, const float* d_init, const float* A, const void* B, const void* C,
              const float* D, const void* z, const float* init, const int32_t* cu, bool bwd,
              SelParams* p, SelPlan* pl) {
    int st = sel_check(dims);
    if (st != SSD_OK) return st;
    const ssd_selscan_dims& d = *dims;
    const int64_t E = d.channels, N = d.d_state, G = d.ngroups;
    ssd_selscan_layout l = {E, E, E, G * N, N, G * N, N, E, E};
    if (layout) l = *layout;
    if (!z) l.z_token = E;
    for (int64_t s : {l.x_token, l.d_raw_token, l.z_token, bwd ? l.dy_token : l.y_token})
        if (s < E || s > kMaxStride) return SSD_ERR_SHAPE;
    for (int64_t s : {l.B_token, l.B_group, l.C_token, l.C_group})
        if (s < 0 || s > kMaxStride) return SSD_ERR_SHAPE;
    if ((d.nseq > 0) != (cu != nullptr)) return cu ? SSD_ERR_SHAPE : SSD_ERR_NULL_ARG;
    if ((st = sel_plan(d, bwd, pl)) != SSD_OK) return st;
    if (!d_init || !A || (pl->T > 0 && (!x || !d_raw || !B || !C))) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(d.dtype);
    for (const void* q : {x, d_raw, B, C, z})
        if (!elem_aligned(q, e)) return SSD_ERR_ALIGN;
    for (const void* q : {(const void*)d_init, (const void*)A, (const void*)D, (const void*)init,
                          (const void*)cu})
        if (!elem_aligned(q, 4)) return SSD_ERR_ALIGN;
    *p = {};
    p->x = x;
    p->d_raw = d_raw;
    p->z = z;
    p->B = B;
    p->C = C;
    p->d_init = d_init;
    p->A = A;
    p->D = D;
    p->init = init;
    p->cu = cu;
    p->xs = l.x_token;
    p->ds = l.d_raw_token;
    p->zs = l.z_token;
    p->bs_t = l.B_token;
    p->bs_g = l.B_group;
    p->cs_t = l.C_token;
    p->cs_g = l.C_group;
    p->ys = l.y_token;
    p->gs = l.dy_token;
    p->L = d.seqlen;
    p->T = pl->T;
    p->E = d.channels;
    p->N = d.d_state;
    p->G = d.ngroups;
    p->epg = d.channels / d.ngroups;
    p->S = pl->S;
    p->nblk = pl->nblk;
    p->bpg = pl->bpg;
    p->units = (int32_t)pl->units;
    p->upr = pl->upr;
    p->span = pl->span;
    p->per = pl->per;
    return SSD_OK;
}

template <typename T, int NR, int MW>
void launch(const SelParams& p, unsigned grid, hipStream_t s) {
    if (p.span) selscan_span_kernel<T, NR><<<dim3(grid), dim3(512), 0, s>>>(p);
    selscan_fwd_kernel<T, NR, MW><<<dim3(grid), dim3(64 * MW), 0, s>>>(p);
}

template <typename T>
void launch(const SelParams& p, int NR, int waves, unsigned grid, hipStream_t s) {
    if (NR == 2) {
        if (waves == 16) launch<T, 2, 16>(p, grid, s);
        else launch<T, 2, 4>(p, grid, s);
    } else if (NR == 4) {
        if (waves == 16) launch<T, 4, 16>(p, grid, s);
        else if (waves == 8) launch<T, 4, 8>(p, grid, s);
        else if (waves == 4) launch<T, 4, 4>(p, grid, s);
        else launch<T, 4, 2>(p, grid, s);
    } else if (NR == 8) {
        if (waves == 8) launch<T, 8, 8>(p, grid, s);
        else launch<T, 8, 2>(p, grid, s);
    } else {
        if (waves == 8) launch<T, 16, 8>(p, grid, s);
        else launch<T, 16, 2>(p, grid, s);
    }
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_selscan_fwd_workspace_bytes(const ssd_selscan_dims* dims) {
    SelPlan pl;
    if (sel_check(dims) != SSD_OK || sel_plan(*dims, false, &pl) != SSD_OK) return 0;
    return pl.total;
}

int ssd_selscan_fwd(const ssd_selscan_dims* dims, const ssd_selscan_layout* layout, const void* x,
                    const void* d_raw, const float* d_init, const float* A, const void* B,
                    const void* C, const float* D, const void* z, const float* init_state,
                    const int32_t* cu_seqlens, void* y, float* final_state, void* workspace,
                    size_t workspace_bytes, void* stream) {
    SelParams p;
    SelPlan pl;
    int st = sel_setup(dims, layout, x, d_raw, d_init, A, B, C, D, z, init_state, cu_seqlens, false,
                       &p, &pl);
    if (st != SSD_OK) return st;
    if (pl.T > 0 && !y) return SSD_ERR_NULL_ARG;
    if (!elem_aligned(y, elem_size(dims->dtype)) || !elem_aligned(final_state, 4))
        return SSD_ERR_ALIGN;
    if (pl.total > 0) {
        if ((uintptr_t)workspace & 255) return SSD_ERR_ALIGN;
        if (!workspace || workspace_bytes < pl.total) return SSD_ERR_WORKSPACE;
    }
    const size_t sb = (size_t)pl.S * dims->d_state * dims->channels * sizeof(float);
    if (overlaps(init_state, sb, final_state, sb)) return SSD_ERR_OVERLAP;
    hipStream_t s = (hipStream_t)stream;
    if (cu_seqlens && check_cu_env(cu_seqlens, dims->nseq, pl.T, s, &st)) return st;
    if (pl.T == 0 && !final_state) return SSD_OK;
    p.y = y;
    p.final_state = final_state;
    p.span_h = (float*)((char*)workspace + pl.off_h);
    p.span_d = (float*)((char*)workspace + pl.off_d);
    if (dims->dtype == SSD_BF16) launch<bf16>(p, pl.NR, pl.waves, (unsigned)pl.grid, s);
    else launch<float>(p, pl.NR, pl.waves, (unsigned)pl.grid, s);
    return launched();
}

size_t ssd_selscan_bwd_workspace_bytes(const ssd_selscan_dims* dims) {
    SelPlan pl;
    if (sel_check(dims) != SSD_OK || sel_plan(*dims, true, &pl) != SSD_OK) return 0;
    return pl.total;
}

int ssd_selscan_bwd(const ssd_selscan_dims* dims, const ssd_selscan_layout* layout, const void* x,
                    const void* d_raw, const float* d_init, const float* A, const void* B,
                    const void* C, const float* D, const void* z, const float* init_state,
                    const int32_t* cu_seqlens, const void* dy, const float* d_final, void* dx,
                    void* dd_raw, void* dB, void* dC, void* dz, float* dA, float* dD,
                    float* dd_init, float* dinit_state, void* workspace, size_t workspace_bytes,
                    void* stream) {
    SelParams p;
    SelPlan pl;
    int st = sel_setup(dims, layout, x, d_raw, d_init, A, B, C, D, z, init_state, cu_seqlens, true,
                       &p, &pl);
    if (st != SSD_OK) return st;
    if (pl.T * dims->ngroups * 8 * pl.NR + 256 > kMaxThreads) return SSD_ERR_SHAPE;
    // dB and dC take the places of B and C: no two of their rows may share one
    if (pl.T > 0 && (!rows_apart(pl.T, p.bs_t, p.G, p.bs_g, p.N) ||
                     !rows_apart(pl.T, p.cs_t, p.G, p.cs_g, p.N)))
        return SSD_ERR_SHAPE;
    if (pl.T > 0 && (!dy || !dx || !dd_raw || !dB || !dC || (z && !dz))) return SSD_ERR_NULL_ARG;
    const size_t e = elem_size(dims->dtype);
    for (const void* q : {dy, (const void*)dx, (const void*)dd_raw, (const void*)dB,
                          (const void*)dC, (const void*)dz})
        if (!elem_aligned(q, e)) return SSD_ERR_ALIGN;
    for (const void* q : {(const void*)d_final, (const void*)dA, (const void*)dD,
                          (const void*)dd_init, (const void*)dinit_state})
        if (!elem_aligned(q, 4)) return SSD_ERR_ALIGN;
    if ((uintptr_t)workspace & 255) return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < pl.total) return SSD_ERR_WORKSPACE;
    const size_t sb = (size_t)pl.S * dims->d_state * dims->channels * sizeof(float);
    if (overlaps(d_final, sb, dinit_state, sb)) return SSD_ERR_OVERLAP;
    hipStream_t s = (hipStream_t)stream;
    if (cu_seqlens && check_cu_env(cu_seqlens, dims->nseq, pl.T, s, &st)) return st;
    char* ws = (char*)workspace;
    p.dy = dy;
    p.d_final = d_final;
    p.y = dx;
    p.dd_raw = dd_raw;
    p.dz = dz;
    p.final_state = dinit_state;
    p.run_h = (float*)(ws + pl.off_h);
    p.run_q = (float*)(ws + pl.off_q);
    p.run_d = (float*)(ws + pl.off_d);
    p.chunk_h = (float*)(ws + pl.off_ch);
    p.chunk_d = (float*)(ws + pl.off_cd);
    p.part_w = (float*)(ws + pl.off_w);
    p.part_bc = (float*)(ws + pl.off_bc);
    if ((st = launch_selscan_bwd(p, dims->dtype, pl.NR, pl.runs, (unsigned)pl.grid, s)) != SSD_OK)
        return st;
    const int NP = 4 * pl.NR;
    const int64_t items = pl.T * dims->ngroups * 2 * NP;
    if (items > 0) {
        const int64_t grid = cdiv(items, 256);
        const dim3 gd((unsigned)grid), bd(256);
        if (dims->dtype == SSD_BF16) selscan_bc_kernel<bf16><<<gd, bd, 0, s>>>(p, dB, dC, NP);
        else selscan_bc_kernel<float><<<gd, bd, 0, s>>>(p, dB, dC, NP);
        if ((st = launched()) != SSD_OK) return st;
    }
    ColSum c = {};
    c.part = p.part_w;
    c.rows = pl.slots;
    c.cols = (int64_t)(dims->d_state + 2) * dims->channels;
    c.out0 = dA;
    c.c0 = (int64_t)dims->d_state * dims->channels;
    c.out1 = dD;
    c.c1 = dims->channels;
    c.out2 = dd_init;
    return launch_colsum(c, s);
}

}  // extern "C"
