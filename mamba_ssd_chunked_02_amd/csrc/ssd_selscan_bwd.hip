// Selective scan, backward (see ssd_selscan.h).
#include "ssd_selscan.h"

namespace ssd {
namespace {

// First the segments forward, only to find the state that enters each chunk
// (kept in chunk_states); then backward, where each wave holds a and h of its
// chunk in registers.  What enters the last segment's chunks is found there,
// so a sequence of one segment is walked once.
template <typename T, int NR, int MW>
__global__ __launch_bounds__(64 * MW, Shape<NR>::kBwdPerSimd) void selscan_bwd_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kBwdTokens, NP = S::NP, Q = TW / 4, waves = MW;
    __shared__ __align__(16) float bc[MW][TW][2][NP];
    __shared__ __align__(16) float exP[2][MW][64][NR], exH[2][MW][64][NR], exQ[2][MW][64][NR];
    __shared__ __align__(16) float enter[3][64][NR];  // h or q entering a segment
    Place o;
    if (!place_of(p, o)) return;
    const int seg = waves * TW;
    const bool b0 = o.nl & 1, b1 = o.nl & 2;
    float A2[NR], dA[NR], h[NR], q[NR];
    load_rates<NR>(p, o, A2);
    const float dinit = o.live ? p.d_init[o.ch] : 0.f;
    const float Dv = o.live && p.D ? p.D[o.ch] : 0.f;
    const bool gated = p.z != nullptr;
    // (a slot without a span has no tokens and still writes its share: zeros)
    const int nseg = o.k < o.nspan ? (o.last - o.first + seg - 1) / seg : 0;
    // sequences' segments follow one another: this one's start at a slot that
    // no earlier sequence reaches
    float* states = p.chunk_states +
                    ((((int64_t)(o.first / seg + o.seq) * waves + o.wave) * p.nblk + o.blk) * 64 + o.lane) * NR;
    const int64_t states_step = (int64_t)waves * p.nblk * 64 * NR;

    uint32_t xr[Q], dr[Q], zr[Q], gr[Q];
    Rows<T, NR, TW> Br, Cr;
    int turn = 0;
    // -- forward over all segments but the last
    int tb = o.first + o.wave * TW;
    if (o.wave == 0) {
        load_state<NR>(p.init, p, o, h);
        if (p.span && nseg > 0) fold_spans<NR>(p.span_h, p, o, A2, 0, o.k, 1, h);
        lds_put<NR>(enter[0][o.lane], h);
    }
    auto fetch_forward = [&](int t) {
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->x, k->xs, o, t, xr);
        load_tokens<T, TW>(k->d_raw, k->ds, o, t, dr);
        load_rows<T, NR, TW>(k->B, k->bs_t, k->bs_g, k->N, o, t, Br);
    };
    if (nseg > 1) fetch_forward(tb);
    for (int k = 1; k < nseg; ++k, turn ^= 1) {
        float d[Q], u[Q], P[NR];
        float sumd = 0.f;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            d[i] = softplus(value_of<T>(dr[i]) + dinit);
            u[i] = d[i] * value_of<T>(xr[i]);
            sumd += d[i];
        }
        sumd = quad_total(sumd);
        wave_lds_fence();
        put_rows<T, NR, TW>(&bc[o.wave][0][0][0], o, Br);
        wave_lds_fence();
        tb += seg;
        if (k + 1 < nseg) fetch_forward(tb);
#pragma unroll
        for (int r = 0; r < NR; ++r) P[r] = fexp2(sumd * A2[r]);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            float b[NR];
            lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
            const float dt = quad_lane(d[t / 4], t % 4), ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                h[r] = t ? fexp2(dt * A2[r]) * h[r] + b[r] * ut : b[r] * ut;
        }
        lds_put<NR>(exP[turn][o.wave][o.lane], P);
        lds_put<NR>(exH[turn][o.wave][o.lane], h);
        __syncthreads();
        float hin[NR];
        lds_get<NR>(enter[turn][o.lane], hin);
        for (int j = 0; j < o.wave; ++j) {
            float Pj[NR], hj[NR];
            lds_get<NR>(exP[turn][j][o.lane], Pj);
            lds_get<NR>(exH[turn][j][o.lane], hj);
#pragma unroll
            for (int r = 0; r < NR; ++r) hin[r] = Pj[r] * hin[r] + hj[r];
        }
        __builtin_memcpy(states + (k - 1) * states_step, hin, sizeof(hin));
        if (o.wave == waves - 1) {
#pragma unroll
            for (int r = 0; r < NR; ++r) hin[r] = P[r] * hin[r] + h[r];
            lds_put<NR>(enter[turn ^ 1][o.lane], hin);
        }
    }
    // -- backward.  enter[turn] holds the state entering the last segment; q goes
    // through the other two slots in turn, first through the one that no wave
    // can still be reading.
    const int last_slot = turn;
    int q_slot = 2, q_next = turn ^ 1;
    if (o.wave == 0) {
        load_state<NR>(p.d_final, p, o, q);
        if (p.span) fold_spans<NR>(p.span_q, p, o, A2, o.nspan - 1, o.nspan - 1 - o.k, -1, q);
        lds_put<NR>(enter[q_slot][o.lane], q);
    }
    float dD = 0.f, dI = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) dA[r] = 0.f;
    // where the lane's sums over channels go: see the reduction below
    const int r_of = (o.lane & 16 ? NR / 2 : 0) + (NR > 2 && (o.lane & 8) ? NR / 4 : 0);
    const uint32_t sum_off = !(o.lane & 4) && (NR > 2 || !(o.lane & 8))
                                 ? (uint32_t)((o.lane & 32 ? NP : 0) + o.nl * NR + r_of) * 4u
                                 : kNowhere;
    auto fetch = [&](int t) {
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->x, k->xs, o, t, xr);
        load_tokens<T, TW>(k->d_raw, k->ds, o, t, dr);
        load_tokens<T, TW>(k->dy, k->gs, o, t, gr);
        load_tokens<T, TW>(k->z, k->zs, o, t, zr);
        load_rows<T, NR, TW>(k->B, k->bs_t, k->bs_g, k->N, o, t, Br);
        load_rows<T, NR, TW>(k->C, k->cs_t, k->cs_g, k->N, o, t, Cr);
    };
    tb = o.first + (nseg - 1) * seg + o.wave * TW;
    if (nseg > 0) fetch(tb);
    for (int k = nseg - 1; k >= 0; --k, tb -= seg, turn ^= 1) {
        if (tb >= o.last) {  // in the last segment, behind the sequence
            __syncthreads();
            if (k > 0) fetch(tb - seg);
            q_slot = q_next;
            q_next = 2;
            continue;
        }
        const int have = min(o.last - tb, TW);
        float hin[NR];
        if (k < nseg - 1) __builtin_memcpy(hin, states + k * states_step, sizeof(hin));
        // past the sequence and in lanes without a channel x and dy are 0
        float d[Q], u[Q], w[Q], x[Q], raw[Q], gz[Q];  // gz: what dz multiplies v by
        float sumd = 0.f;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            x[i] = value_of<T>(xr[i]);
            raw[i] = value_of<T>(dr[i]) + dinit;
            d[i] = step_of(raw[i], 4 * i + o.nl < have);
            u[i] = d[i] * x[i];
            sumd += d[i];
            w[i] = gz[i] = value_of<T>(gr[i]);
            if (gated) {
                const float zf = value_of<T>(zr[i]), sz = sigmoid(zf);
                w[i] *= zf * sz;
                gz[i] *= silu_slope(zf, sz);
            }
            dD += w[i] * x[i];
        }
        sumd = quad_total(sumd);
        wave_lds_fence();
        put_rows<T, NR, TW>(&bc[o.wave][0][0][0], o, Br);
        put_rows<T, NR, TW>(&bc[o.wave][0][1][0], o, Cr);
        wave_lds_fence();
        // (1) every decay of the chunk, and q through it from zero
        float a[TW][NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) h[r] = fexp2(sumd * A2[r]);
        lds_put<NR>(exP[turn][o.wave][o.lane], h);
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            const float dt = quad_lane(d[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r) a[t][r] = fexp2(dt * A2[r]);
        }
        if (k == nseg - 1) {
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                float b[NR];
                lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
                const float ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
                for (int r = 0; r < NR; ++r) h[r] = t ? a[t][r] * h[r] + b[r] * ut : b[r] * ut;
                if (t & 1) keep_order();
            }
            lds_put<NR>(exH[turn][o.wave][o.lane], h);
        }
#pragma unroll
        for (int t = TW - 1; t >= 0; --t) {
            float c[NR];
            lds_get<NR>(&bc[o.wave][t][1][o.nl * NR], c);
            const float wt = quad_lane(w[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                q[r] = t < TW - 1 ? a[t][r] * (c[r] * wt + q[r]) : a[t][r] * (c[r] * wt);
            if (!(t & 1)) keep_order();
        }
        lds_put<NR>(exQ[turn][o.wave][o.lane], q);
        // (2) fold the chunks behind this one (q), and in the last segment those
        // before it (h)
        __syncthreads();
        if (k == nseg - 1) {
            lds_get<NR>(enter[last_slot][o.lane], hin);
            for (int j = 0; j < o.wave; ++j) {
                float Pj[NR], hj[NR];
                lds_get<NR>(exP[turn][j][o.lane], Pj);
                lds_get<NR>(exH[turn][j][o.lane], hj);
#pragma unroll
                for (int r = 0; r < NR; ++r) hin[r] = Pj[r] * hin[r] + hj[r];
            }
        }
        lds_get<NR>(enter[q_slot][o.lane], q);
        // the waves behind the sequence have left nothing
        for (int j = min(waves, (o.last - o.first - k * seg + TW - 1) / TW) - 1; j > o.wave; --j) {
            float Pj[NR], qj[NR];
            lds_get<NR>(exP[turn][j][o.lane], Pj);
            lds_get<NR>(exQ[turn][j][o.lane], qj);
#pragma unroll
            for (int r = 0; r < NR; ++r) q[r] = Pj[r] * q[r] + qj[r];
        }
        // (3) h of every token, then the gradients from the last token back
        float hs[TW][NR];
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            float b[NR];
            lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
            const float ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                hs[t][r] = a[t][r] * (t ? hs[t - 1][r] : hin[r]) + b[r] * ut;
            if (t & 1) keep_order();
        }
        const ArgPtr out = fresh_args();
        const RowBuf<float> sums = row_buf<float>(out->part_bc + (int64_t)o.blk * out->T * (2 * NP),
                                                  2 * NP, 0, tb, have, 2 * NP);
        const RowBuf<T> dx = row_buf<T>(out->y, out->xs, o.ch0, tb, have, o.width);
        const RowBuf<T> ddr = row_buf<T>(out->dd_raw, out->ds, o.ch0, tb, have, o.width);
        const RowBuf<T> dz = row_buf<T>(out->dz, out->zs, o.ch0, tb, gated ? have : 0, o.width);
        const auto lane_off = [&](int64_t stride) {
            return fresh(o.live ? (uint32_t)(o.nl * stride + o.e) * (uint32_t)sizeof(T) : kNowhere);
        };
        const uint32_t xoff = lane_off(out->xs), doff = lane_off(out->ds), zoff = lane_off(out->zs);
#pragma unroll
        for (int i = Q - 1; i >= 0; --i) {
            // the next segment's rows, once half of a and hs is used up
            if (i == (Q - 1) / 2 && k > 0) fetch(tb - seg);
            float gB[4], sA[4], v[4];
#pragma unroll
            for (int kk = 3; kk >= 0; --kk) {
                const int t = 4 * i + kk;
                float b[NR], c[NR], db[NR], dc[NR];
                lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
                lds_get<NR>(&bc[o.wave][t][1][o.nl * NR], c);
                const float dt = quad_lane(d[i], kk), ut = quad_lane(u[i], kk);
                const float wt = quad_lane(w[i], kk);
                gB[kk] = sA[kk] = v[kk] = 0.f;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float g = c[r] * wt + q[r];
                    q[r] = a[t][r] * g;
                    const float s = q[r] * (t ? hs[t - 1][r] : hin[r]);
                    gB[kk] += g * b[r];
                    sA[kk] += A2[r] * s;
                    dA[r] += dt * s;
                    v[kk] += c[r] * hs[t][r];
                    db[r] = g * ut;
                    dc[r] = hs[t][r] * wt;
                }
                // sums over the wave's 16 channels: lane bit 5 picks dB or dC,
                // bits 4 and 3 the entry, bits 1 and 0 the quad's lane
                constexpr int M = NR >= 4 ? NR / 4 : 1;
                float f[M];
                if constexpr (NR == 2) {
                    f[0] = ring_sum(row_sums16(half_sums(db[0], dc[0]), half_sums(db[1], dc[1])));
                } else {
                    const bool b3 = o.lane & 8;
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const float f0 = ring_sum(row_sums16(half_sums(db[m], dc[m]),
                                                             half_sums(db[m + NR / 2], dc[m + NR / 2])));
                        const float f1 = ring_sum(
                            row_sums16(half_sums(db[m + NR / 4], dc[m + NR / 4]),
                                       half_sums(db[m + 3 * NR / 4], dc[m + 3 * NR / 4])));
                        f[m] = b3 ? f1 : f0;
                    }
                }
#pragma unroll
                for (int m = 0; m < M; ++m) sums.put(sum_off + (uint32_t)(t * 2 * NP + m) * 4u, f[m]);
                keep_order();
            }
            const float gBt = quad_sums(gB[0], gB[1], gB[2], gB[3], b0, b1);
            // A2 is A log2(e)
            const float sAt = quad_sums(sA[0], sA[1], sA[2], sA[3], b0, b1) * 0.69314718055994531f;
            const float dd = 4 * i + o.nl < have && o.live ? (x[i] * gBt + sAt) * sigmoid(raw[i]) : 0.f;
            dI += dd;
            dx.put(xoff + i * (uint32_t)(4 * out->xs * sizeof(T)), w[i] * Dv + d[i] * gBt);
            ddr.put(doff + i * (uint32_t)(4 * out->ds * sizeof(T)), dd);
            if (gated) {
                const float vt = quad_sums(v[0], v[1], v[2], v[3], b0, b1) + Dv * x[i];
                dz.put(zoff + i * (uint32_t)(4 * out->zs * sizeof(T)), gz[i] * vt);
            }
            keep_order();
        }
        // q leaving the segment's first chunk enters the segment before it; its
        // slot was last read before the barrier that this wave has passed
        if (o.wave == 0) lds_put<NR>(enter[q_next][o.lane], q);
        const int used = q_slot;
        q_slot = q_next;
        q_next = used;
        wave_lds_fence();
    }
    if (o.wave == 0 && o.k == 0) store_state<NR>(p.final_state, p, o, q);
    // the waves' shares of dA, dD and dd_init
    dD = quad_total(dD);
    dI = quad_total(dI);
    __syncthreads();
    lds_put<NR>(exP[0][o.wave][o.lane], dA);
    exH[0][o.wave][o.lane][0] = dD;
    exH[0][o.wave][o.lane][1] = dI;
    __syncthreads();
    if (o.wave || !o.live) return;
    for (int j = 1; j < waves; ++j) {
        float t[NR];
        lds_get<NR>(exP[0][j][o.lane], t);
#pragma unroll
        for (int r = 0; r < NR; ++r) dA[r] += t[r];
        dD += exH[0][j][o.lane][0];
        dI += exH[0][j][o.lane][1];
    }
    float* pw = p.part_w + (int64_t)o.slot * (p.N + 2) * p.E + o.ch;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int n = o.nl * NR + r;
        if (n < p.N) pw[(int64_t)n * p.E] = dA[r];
    }
    if (o.nl == 0) {
        pw[(int64_t)p.N * p.E] = dD;
        pw[(int64_t)(p.N + 1) * p.E] = dI;
    }
}


template <typename T, int NR, int MW>
void launch(const SelParams& p, unsigned grid, hipStream_t s) {
    if (p.span) selscan_span_kernel<T, NR, true><<<dim3(grid), dim3(512), 0, s>>>(p);
    selscan_bwd_kernel<T, NR, MW><<<dim3(grid), dim3(64 * MW), 0, s>>>(p);
}

template <typename T>
void launch(const SelParams& p, int NR, int waves, unsigned grid, hipStream_t s) {
    if (NR == 2) {
        if (waves == 8) launch<T, 2, 8>(p, grid, s);
        else launch<T, 2, 2>(p, grid, s);
    } else if (NR == 4) {
        if (waves == 8) launch<T, 4, 8>(p, grid, s);
        else if (waves == 4) launch<T, 4, 4>(p, grid, s);
        else launch<T, 4, 2>(p, grid, s);
    } else if (NR == 8) {
        if (waves == 8) launch<T, 8, 8>(p, grid, s);
        else launch<T, 8, 2>(p, grid, s);
    } else {
        if (waves == 4) launch<T, 16, 4>(p, grid, s);
        else launch<T, 16, 1>(p, grid, s);
    }
}

}  // namespace

int launch_selscan_bwd(const SelParams& p, int32_t dtype, int NR, int waves, unsigned grid,
                       hipStream_t s) {
    if (dtype == SSD_BF16) launch<bf16>(p, NR, waves, grid, s);
    else launch<float>(p, NR, waves, grid, s);
    return launched();
}

}  // namespace ssd
