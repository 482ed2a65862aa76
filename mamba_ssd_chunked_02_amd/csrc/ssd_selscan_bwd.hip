// Selective scan, backward (see ssd_selscan.h).
//
// Three launches.  A wave owns a run of 64 tokens of its 16 channels:
//   runs   every run from zero, forward in time: its state, what it does to a q
//          that enters from behind (q before = P q + Q, composed chunk by chunk),
//          its sum of d, and the state before each of its chunks;
//   links  along each sequence: the h that enters every run and the q that enters
//          it from behind, in place;
//   grads  every run again, its chunks from the last to the first, a and h of a
//          chunk in registers.
// The runs are independent of each other in both large launches: they fill the
// chip whatever the number of sequences and channels, and no wave waits for
// another.  (One launch that walked a sequence's segments forward and back, its
// waves exchanging states in LDS, needed a workgroup per sequence and channel
// block: 2 x 2048 tokens x 1536 channels kept 192 of 256 CUs busy, 193 us.)
#include "ssd_selscan.h"

namespace ssd {
namespace {

// A workgroup is one wave and its slot's span is one run.  (Workgroups of four
// waves took as long where the runs were many, and kept the registers of idle
// waves where they were few: 24 sequences of 170 tokens 230 us instead of 188.)
// Where a run's and its chunks' records lie: chunk c of the run in slot i, which
// starts at token f, has record f / TW + i + c, so no two runs meet.
struct Run {
    int first, chunks;
    int64_t rec;     // of the run: [slot][blk][lane]
    int64_t chunk0;  // of its first chunk
};
template <int NR>
__device__ __forceinline__ Run run_of(const SelParams& p, const Place& o) {
    using S = Shape<NR>;
    Run r;
    r.first = o.first;
    r.chunks = o.k < o.nspan ? (o.last - o.first + S::kBwdTokens - 1) / S::kBwdTokens : 0;
    r.rec = ((int64_t)o.slot * p.nblk + o.blk) * 64 + o.lane;
    r.chunk0 = ((int64_t)(r.first / S::kBwdTokens + o.slot) * p.nblk + o.blk) * 64 + o.lane;
    return r;
}

// A token's decay.  The product takes 0 times anything as 0: behind the sequence,
// where d is 0, the decay is 1 also for a rate that is NaN, and q reaches the last
// token unchanged.
__device__ __forceinline__ float decay_of(float d, float A2) {
    float p;
    asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(p) : "v"(d), "v"(A2));
    return fexp2(p);
}

template <typename T, int NR>
__global__ __launch_bounds__(64, NR <= 8 ? 4 : 2) void selscan_runs_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kBwdTokens, NP = S::NP, Q = TW / 4;
    __shared__ __align__(16) float bc[TW][2][NP];
    Place o;
    if (!place_of(p, o)) return;
    const Run run = run_of<NR>(p, o);
    if (run.chunks == 0) return;
    float A2[NR], h[NR], q[NR];
    load_rates<NR>(p, o, A2);
    const float dinit = o.live ? p.d_init[o.ch] : 0.f;
    const bool gated = p.z != nullptr;
    uint32_t xr[Q], dr[Q], gr[Q], zr[Q];
    Rows<T, NR, TW> Br, Cr;
    auto fetch = [&](int t) {
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->x, k->xs, o, t, xr);
        load_tokens<T, TW>(k->d_raw, k->ds, o, t, dr);
        load_tokens<T, TW>(k->dy, k->gs, o, t, gr);
        load_tokens<T, TW>(k->z, k->zs, o, t, zr);
        load_rows<T, NR, TW>(k->B, k->bs_t, k->bs_g, k->N, o, t, Br);
        load_rows<T, NR, TW>(k->C, k->cs_t, k->cs_g, k->N, o, t, Cr);
    };
#pragma unroll
    for (int r = 0; r < NR; ++r) h[r] = q[r] = 0.f;
    float sum = 0.f;
    int tb = run.first;
    fetch(tb);
    for (int c = 0; c < run.chunks; ++c, tb += TW) {
        if (c > 0) {  // before the first chunk both are 0
            const int64_t rec = run.chunk0 + (int64_t)c * p.nblk * 64;
            p.chunk_d[rec] = sum;
            __builtin_memcpy(p.chunk_h + rec * NR, h, sizeof(h));
        }
        const int have = min(o.last - tb, TW);
        float d[Q], u[Q], w[Q], chunk_d = 0.f;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            d[i] = step_of(value_of<T>(dr[i]) + dinit, 4 * i + o.nl < have);
            u[i] = d[i] * value_of<T>(xr[i]);
            chunk_d += d[i];
            const float zf = value_of<T>(zr[i]);
            w[i] = value_of<T>(gr[i]) * (gated ? zf * sigmoid(zf) : 1.f);
        }
        wave_lds_fence();
        put_rows<T, NR, TW>(&bc[0][0][0], o, Br);
        put_rows<T, NR, TW>(&bc[0][1][0], o, Cr);
        wave_lds_fence();
        if (c + 1 < run.chunks) fetch(tb + TW);
        float a[TW][NR], ql[NR];
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            float b[NR];
            lds_get<NR>(&bc[t][0][o.nl * NR], b);
            const float dt = quad_lane(d[t / 4], t % 4), ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                a[t][r] = decay_of(dt, A2[r]);
                h[r] = a[t][r] * h[r] + b[r] * ut;
            }
            if (t & 1) keep_order();
        }
#pragma unroll
        for (int t = TW - 1; t >= 0; --t) {
            float cc[NR];
            lds_get<NR>(&bc[t][1][o.nl * NR], cc);
            const float wt = quad_lane(w[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                ql[r] = t < TW - 1 ? a[t][r] * (cc[r] * wt + ql[r]) : a[t][r] * (cc[r] * wt);
            if (!(t & 1)) keep_order();
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) q[r] += fexp2(sum * A2[r]) * ql[r];
        sum += quad_total(chunk_d);
    }
    p.run_d[run.rec] = sum;
    __builtin_memcpy(p.run_h + run.rec * NR, h, sizeof(h));
    __builtin_memcpy(p.run_q + run.rec * NR, q, sizeof(q));
}

// LW waves walk a sequence's runs forward (h), LW backward (q), each a piece of
// them: first from zero, then, after the pieces before it are folded, from what
// enters it.  Eight runs' records are loaded at a time.
template <int NR, int LW>
__global__ __launch_bounds__(128 * LW) void selscan_links_kernel(SelParams p) {
    constexpr int AHEAD = 8;
    __shared__ __align__(16) float exV[2][LW][64][NR], exD[2][LW][64];
    Place o = {};
    o.seq = blockIdx.x / (uint32_t)p.nblk;
    o.blk = blockIdx.x % (uint32_t)p.nblk;
    o.group = o.blk / p.bpg;
    o.lane = threadIdx.x & 63;
    o.nl = o.lane & 3;
    const int off = (o.blk % p.bpg) * kChan + (o.lane >> 2);
    o.live = off < p.epg;
    o.ch = o.group * p.epg + off;
    int64_t first, last;
    sequence_span(p.cu, o.seq, p.L, p.T, &first, &last);
    const int slot = p.cu ? (int)first / p.span + o.seq : o.seq * p.per;
    const int runs = (int)((last - first + Shape<NR>::kRunTokens - 1) / Shape<NR>::kRunTokens);
    const int back = wave_id() / LW, piece = wave_id() % LW;
    const int each = (runs + LW - 1) / LW, j0 = min(piece * each, runs), j1 = min(j0 + each, runs);
    float A2[NR], v[NR];
    load_rates<NR>(p, o, A2);
    const int64_t step = (int64_t)p.nblk * 64 * (back ? -1 : 1);
    const int64_t at0 = ((int64_t)(slot + (back ? runs - 1 - j0 : j0)) * p.nblk + o.blk) * 64 + o.lane;
    float* state = back ? p.run_q : p.run_h;
    float sum = 0.f;
    const auto walk = [&](bool write) {
        int64_t at = at0;
        for (int j = j0; j < j1; j += AHEAD, at += AHEAD * step) {
            float d[AHEAD], s[AHEAD][NR];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (j + i < j1) {
                    d[i] = p.run_d[at + i * step];
                    __builtin_memcpy(s[i], state + (at + i * step) * NR, sizeof(s[i]));
                }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (j + i < j1) {
                    if (write) __builtin_memcpy(state + (at + i * step) * NR, v, sizeof(v));
                    sum += d[i];
#pragma unroll
                    for (int r = 0; r < NR; ++r) v[r] = fexp2(d[i] * A2[r]) * v[r] + s[i][r];
                }
        }
    };
    if constexpr (LW > 1) {
#pragma unroll
        for (int r = 0; r < NR; ++r) v[r] = 0.f;
        walk(false);
        exD[back][piece][o.lane] = sum;
        lds_put<NR>(exV[back][piece][o.lane], v);
        __syncthreads();
    }
    load_state<NR>(back ? p.d_final : p.init, p, o, v);
    if constexpr (LW > 1)
        for (int i = 0; i < piece; ++i) {
            const float d = exD[back][i][o.lane];
            float s[NR];
            lds_get<NR>(exV[back][i][o.lane], s);
#pragma unroll
            for (int r = 0; r < NR; ++r) v[r] = fexp2(d * A2[r]) * v[r] + s[r];
        }
    walk(true);
    if (back && piece == LW - 1) store_state<NR>(p.final_state, p, o, v);
}

template <typename T, int NR>
__global__ __launch_bounds__(64, Shape<NR>::kBwdPerSimd) void selscan_grads_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kBwdTokens, NP = S::NP, Q = TW / 4;
    __shared__ __align__(16) float bc[TW][2][NP];
    Place o;
    if (!place_of(p, o)) return;
    const Run run = run_of<NR>(p, o);
    const bool b0 = o.nl & 1, b1 = o.nl & 2;
    float A2[NR], dA[NR], q[NR], hrun[NR];
    load_rates<NR>(p, o, A2);
    const float dinit = o.live ? p.d_init[o.ch] : 0.f;
    const float Dv = o.live && p.D ? p.D[o.ch] : 0.f;
    const bool gated = p.z != nullptr;
    uint32_t xr[Q], dr[Q], zr[Q], gr[Q];
    Rows<T, NR, TW> Br, Cr;
    float cd = 0.f, ch[NR];  // of the chunk's record
    auto fetch = [&](int c) {
        const ArgPtr k = fresh_args();
        const int t = run.first + c * TW;
        load_tokens<T, TW>(k->x, k->xs, o, t, xr);
        load_tokens<T, TW>(k->d_raw, k->ds, o, t, dr);
        load_tokens<T, TW>(k->dy, k->gs, o, t, gr);
        load_tokens<T, TW>(k->z, k->zs, o, t, zr);
        load_rows<T, NR, TW>(k->B, k->bs_t, k->bs_g, k->N, o, t, Br);
        load_rows<T, NR, TW>(k->C, k->cs_t, k->cs_g, k->N, o, t, Cr);
        if (c > 0) {
            const int64_t rec = run.chunk0 + (int64_t)c * k->nblk * 64;
            cd = k->chunk_d[rec];
            __builtin_memcpy(ch, k->chunk_h + rec * NR, sizeof(ch));
        } else {
            cd = 0.f;
#pragma unroll
            for (int r = 0; r < NR; ++r) ch[r] = 0.f;
        }
    };
    float dD = 0.f, dI = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) dA[r] = 0.f;
    // where the lane's sums over channels go: see the reduction below
    const int r_of = (o.lane & 16 ? NR / 2 : 0) + (NR > 2 && (o.lane & 8) ? NR / 4 : 0);
    const uint32_t sum_off = !(o.lane & 4) && (NR > 2 || !(o.lane & 8))
                                 ? (uint32_t)((o.lane & 32 ? NP : 0) + o.nl * NR + r_of) * 4u
                                 : kNowhere;
    if (run.chunks > 0) {
        fetch(run.chunks - 1);
        __builtin_memcpy(q, p.run_q + run.rec * NR, sizeof(q));
        __builtin_memcpy(hrun, p.run_h + run.rec * NR, sizeof(hrun));
    }
    for (int c = run.chunks - 1; c >= 0; --c) {
        const int tb = run.first + c * TW;
        const int have = min(o.last - tb, TW);
        float hin[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) hin[r] = ch[r] + fexp2(cd * A2[r]) * hrun[r];
        // past the sequence and in lanes without a channel x and dy are 0
        float d[Q], u[Q], w[Q], x[Q], raw[Q], gz[Q];  // gz: what dz multiplies v by
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            x[i] = value_of<T>(xr[i]);
            raw[i] = value_of<T>(dr[i]) + dinit;
            d[i] = step_of(raw[i], 4 * i + o.nl < have);
            u[i] = d[i] * x[i];
            w[i] = gz[i] = value_of<T>(gr[i]);
            if (gated) {
                const float zf = value_of<T>(zr[i]), sz = sigmoid(zf);
                w[i] *= zf * sz;
                gz[i] *= silu_slope(zf, sz);
            }
            dD += w[i] * x[i];
        }
        wave_lds_fence();
        put_rows<T, NR, TW>(&bc[0][0][0], o, Br);
        put_rows<T, NR, TW>(&bc[0][1][0], o, Cr);
        wave_lds_fence();
        // h of every token, then the gradients from the last token back
        float a[TW][NR], hs[TW][NR];
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            float b[NR];
            lds_get<NR>(&bc[t][0][o.nl * NR], b);
            const float dt = quad_lane(d[t / 4], t % 4), ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                a[t][r] = decay_of(dt, A2[r]);
                hs[t][r] = a[t][r] * (t ? hs[t - 1][r] : hin[r]) + b[r] * ut;
            }
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
            // the chunk before, once half of a and hs is used up
            if (i == (Q - 1) / 2 && c > 0) fetch(c - 1);
            float gB[4], sA[4], v[4];
#pragma unroll
            for (int kk = 3; kk >= 0; --kk) {
                const int t = 4 * i + kk;
                float b[NR], cc[NR], db[NR], dc[NR];
                lds_get<NR>(&bc[t][0][o.nl * NR], b);
                lds_get<NR>(&bc[t][1][o.nl * NR], cc);
                const float dt = quad_lane(d[i], kk), ut = quad_lane(u[i], kk);
                const float wt = quad_lane(w[i], kk);
                gB[kk] = sA[kk] = v[kk] = 0.f;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float g = cc[r] * wt + q[r];
                    q[r] = a[t][r] * g;
                    const float s = q[r] * (t ? hs[t - 1][r] : hin[r]);
                    gB[kk] += g * b[r];
                    sA[kk] += A2[r] * s;
                    dA[r] += dt * s;
                    v[kk] += cc[r] * hs[t][r];
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
    }
    // the run's share of dA, dD and dd_init
    dD = quad_total(dD);
    dI = quad_total(dI);
    if (!o.live) return;
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


template <typename T, int NR>
void launch(const SelParams& p, int64_t runs, unsigned grid, hipStream_t s) {
    const dim3 links((unsigned)p.S * (unsigned)p.nblk);
    selscan_runs_kernel<T, NR><<<dim3(grid), dim3(64), 0, s>>>(p);
    if (runs <= 16) selscan_links_kernel<NR, 1><<<links, dim3(128), 0, s>>>(p);
    else selscan_links_kernel<NR, 4><<<links, dim3(512), 0, s>>>(p);
    selscan_grads_kernel<T, NR><<<dim3(grid), dim3(64), 0, s>>>(p);
}

template <typename T>
void launch(const SelParams& p, int NR, int64_t runs, unsigned grid, hipStream_t s) {
    if (NR == 2) launch<T, 2>(p, runs, grid, s);
    else if (NR == 4) launch<T, 4>(p, runs, grid, s);
    else if (NR == 8) launch<T, 8>(p, runs, grid, s);
    else launch<T, 16>(p, runs, grid, s);
}

}  // namespace

int launch_selscan_bwd(const SelParams& p, int32_t dtype, int NR, int64_t runs, unsigned grid,
                       hipStream_t s) {
    if (dtype == SSD_BF16) launch<bf16>(p, NR, runs, grid, s);
    else launch<float>(p, NR, runs, grid, s);
    return launched();
}

}  // namespace ssd
