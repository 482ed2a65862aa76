// Selective scan with a decay per channel and state entry, forward and backward.
//
//   d_t = softplus(d_raw_t + d_init),  u_t = d_t x_t,  a_t,n = exp(d_t A_n)
//   h_t,n = a_t,n h_{t-1},n + B_t,n u_t,   v_t = sum_n C_t,n h_t,n + D x_t,  y_t = v_t silu(z_t)
// and with w_t = dy_t silu(z_t), q_t = a_{t+1} g_{t+1} (q after the last token: d_final):
//   g_t,n = C_t,n w_t + q_t,n,                  dz_t = dy_t v_t silu'(z_t)
//   dx_t = D w_t + d_t sum_n g_t,n B_t,n,       dB_t,n = sum_e g u,   dC_t,n = sum_e h w
//   dd_t = x_t sum_n g B + sum_n A_n (a g h_{t-1}),   dd_raw_t = dd_t sigmoid(d_raw_t + d_init)
//   dA_n = sum_t d_t (a g h_{t-1}),  dD = sum w x,  dd_init = sum dd_raw,  dinit_state = a_0 g_0
//
// Every token of every channel costs N exponentials and about 4 N products, so
// both directions are bound by the vector units, not by memory; nothing here
// has the shape of a matrix product (the decay differs in every lane).
//
// Mapping.  Four lanes of a wave hold one channel (a quad; N / 4 state entries
// each), a wave 16 channels.  A workgroup owns 16 channels of one sequence;
// its waves take consecutive chunks of TW tokens.  A segment of waves x TW
// tokens goes: (1) every wave scans its chunk from a zero state, keeping all
// a_t,n in registers; (2) the waves exchange (decay product, state) in LDS and
// fold those before them; (3) every wave scans its chunk again from the state
// that enters it, without forming an exponential.  The state that leaves the
// segment enters the next one, so a sequence needs no other launch and no
// global scratch.  Per-token values (d, u, y) live in the quad's lanes, token
// 4 i + k in lane k, and reach the other three as DPP operands.
#include "ssd_layer.h"

namespace ssd {
namespace {

struct SelParams {
    const void* x;
    const void* d_raw;
    const void* z;
    const void* B;
    const void* C;
    const void* dy;
    void* y;  // or dx
    void* dd_raw;
    void* dz;
    const float* d_init;
    const float* A;
    const float* D;
    const float* init;
    const float* d_final;
    const int32_t* cu;
    float* final_state;  // or dinit_state
    float* span_h;       // spans' states from zero [slots][blocks][64][NR]
    float* span_q;       // backward: what their tokens pass on to the span before
    float* span_d;       // their sums of d [slots][blocks][64]
    float* chunk_states; // backward: states entering the chunks [segments][waves][blocks][64][NR]
    float* part_w;       // backward: [slots][(N + 2) E] shares of dA, dD, dd_init
    float* part_bc;      // backward: [blocks][T][2 NP] shares of dB, dC
    int64_t xs, ds, zs, bs_t, bs_g, cs_t, cs_g, ys, gs;
    int64_t L, T;
    int32_t E, N, G, epg, S;
    int32_t nblk;   // channel blocks in all
    int32_t bpg;    // of one group
    int32_t units;  // runs of kRun adjacent channel blocks, over all slots
    int32_t upr;    // of one slot
    int32_t span;   // tokens of a span (whole segments; 0: a sequence is one span)
    int32_t per;    // without cu_seqlens: spans of a sequence
};

// The kernel's argument block, read anew: what is loaded through the returned
// pointer is not kept in scalar registers across the loops around it.  (Kept,
// the pointers and strides of ten tensors did not fit and went through vector
// lanes, 500 instructions a segment of the backward kernel.)
typedef const __attribute__((address_space(4))) SelParams* ArgPtr;
__device__ __forceinline__ ArgPtr fresh_args() {
    ArgPtr k = (ArgPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(k));
    return k;
}

constexpr int kChan = 16;  // channels of a wave
constexpr int kRun = 8;    // adjacent channel blocks kept on one XCD

template <int NR>
struct Shape {
    static constexpr int NP = 4 * NR;           // state entries held
    static constexpr int kFwdTokens = 64 / NR;  // of a wave's chunk
    static constexpr int kFwdWaves = NR <= 4 ? 16 : 8;
    static constexpr int kBwdTokens = NR == 2 ? 16 : 64 / NR;
    static constexpr int kBwdWaves = NR <= 8 ? 8 : 4;
    static constexpr int kBwdSegment = kBwdTokens * kBwdWaves;
};

// Bounds what the scheduler moves together, so that the unrolled token loops
// stay within the registers; LDS reads may still be started early.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x100); }

// ---- lane helpers -------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// The value of the quad's lane k (constant once unrolled).
__device__ __forceinline__ float quad_lane(float v, int k) {
    switch (k) {
        case 0: return dpp<0x00>(v);
        case 1: return dpp<0x55>(v);
        case 2: return dpp<0xaa>(v);
        default: return dpp<0xff>(v);
    }
}
// Lane k of each quad gets the quad's sum of v_k.
__device__ __forceinline__ float quad_sums(float v0, float v1, float v2, float v3, bool b0, bool b1) {
    const float r01 = (b0 ? v1 : v0) + dpp<0xb1>(b0 ? v0 : v1);
    const float r23 = (b0 ? v3 : v2) + dpp<0xb1>(b0 ? v2 : v3);
    return (b1 ? r23 : r01) + dpp<0x4e>(b1 ? r01 : r23);
}
__device__ __forceinline__ float quad_total(float v) {
    v += dpp<0xb1>(v);
    return v + dpp<0x4e>(v);
}
// Lower half: sum of a over lanes l and l + 32; upper half: of b.
__device__ __forceinline__ float half_sums(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Even rows of 16 lanes: sum of a over the row and the next; odd rows: of b.
__device__ __forceinline__ float row_sums16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the four lanes of a row of 16 that share bits 0 and 1.
__device__ __forceinline__ float ring_sum(float v) {
    v += dpp<0x128>(v);  // row_ror:8
    return v + dpp<0x124>(v);  // row_ror:4
}

// Orders a wave's own LDS writes before its later reads of other lanes' data.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int NR>
__device__ __forceinline__ void lds_get(const float* p, float (&o)[NR]) {
    if constexpr (NR == 2) {
        const f32x2 t = *(const f32x2*)p;
        o[0] = t[0];
        o[1] = t[1];
    } else {
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
            const f32x4 t = *(const f32x4*)(p + r);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[r + j] = t[j];
        }
    }
}
template <int NR>
__device__ __forceinline__ void lds_put(float* p, const float (&v)[NR]) {
    if constexpr (NR == 2) {
        *(f32x2*)p = f32x2{v[0], v[1]};
    } else {
#pragma unroll
        for (int r = 0; r < NR; r += 4) *(f32x4*)(p + r) = f32x4{v[r], v[r + 1], v[r + 2], v[r + 3]};
    }
}

// d of a token, 0 where it does not count.  The softplus is formed either way:
// a branch around it costs more than its 20 operations.
__device__ __forceinline__ float step_of(float raw, bool counts) {
    float d = softplus(raw);
    asm volatile("" : "+v"(d));
    return counts ? d : 0.f;
}

// ---- the parts of a chunk -----------------------------------------------------------------

// What a workgroup works on: a channel block of one span.  Long sequences may
// be cut into spans of whole segments so that few channels still fill the chip;
// a first launch then forms what every span does to a state, and the scan of a
// span begins by folding those before it.
struct Place {
    int seq, group, blk;     // blk counts over all groups
    int slot, k, nspan;      // the span's slot; it is span k of nspan (k >= nspan: nothing)
    int lane, wave, nl, e;   // nl: lane of the quad; e: channel of the wave
    int ch0, ch;             // the workgroup's first channel; the lane's
    int width;               // channels of the workgroup
    bool live;               // ch is one of them
    int first, last;         // the span's tokens
};

// The sequence with the slot-th most tokens of at most 64 (equal ones in
// order): the longest start first, so that none is left running alone.
__device__ __forceinline__ int by_length(const int32_t* cu, int S, int slot) {
    const int lane = threadIdx.x & 63;
    const int len = lane < S ? cu[lane + 1] - cu[lane] : INT32_MIN;
    int rank = 0;
    for (int j = 0; j < S; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane);
    }
    const uint64_t hit = __ballot(lane < S && rank == slot);
    return __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
}

// False where the grid's rounding left the workgroup without a channel block.
// Runs of kRun adjacent channel blocks, which share the cache lines of x and
// the rows of B and C, go to one XCD (workgroups are dealt to the eight XCDs
// in turn).
//
// Slots of packed sequences: span k of sequence i, which starts at token f, has
// slot f / span + i + k.  A sequence of n tokens takes at most
// (f + n) / span - f / span + 1 of them, so no two sequences meet, some slots
// stay empty, and the sequence of a slot is found by bisection.
__device__ __forceinline__ bool place_of(const SelParams& p, Place& o) {
    const uint32_t id = blockIdx.x;
    const uint32_t unit = id / (kXcds * kRun) * kXcds + id % kXcds;
    if (unit >= (uint32_t)p.units) return false;
    o.slot = (int)(unit / (uint32_t)p.upr);
    o.blk = (int)(unit % (uint32_t)p.upr) * kRun + (int)(id / kXcds % kRun);
    if (o.blk >= p.nblk) return false;
    o.group = o.blk / p.bpg;
    o.lane = threadIdx.x & 63;
    o.wave = wave_id();
    o.nl = o.lane & 3;
    o.e = o.lane >> 2;
    const int off = (o.blk % p.bpg) * kChan + o.e;
    o.live = off < p.epg;
    o.ch0 = o.group * p.epg + (o.blk % p.bpg) * kChan;
    o.ch = o.ch0 + o.e;
    o.width = min(kChan, p.epg - (o.blk % p.bpg) * kChan);
    o.seq = o.slot;
    o.k = 0;
    int64_t first, last;
    if (!p.cu) {
        o.seq = o.slot / p.per;
        o.k = o.slot % p.per;
    } else if (p.span) {
        int lo = 0, hi = p.S - 1;  // the last sequence whose slots start at or before this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            sequence_span(p.cu, mid, p.L, p.T, &first, &last);
            if ((int)first / p.span + mid <= o.slot) lo = mid; else hi = mid - 1;
        }
        o.seq = __builtin_amdgcn_readfirstlane(lo);
    } else if (p.S <= 64) {
        o.seq = by_length(p.cu, p.S, o.slot);
    }
    sequence_span(p.cu, o.seq, p.L, p.T, &first, &last);
    o.first = __builtin_amdgcn_readfirstlane((int)first);
    o.last = __builtin_amdgcn_readfirstlane((int)last);
    o.nspan = 1;
    if (p.span) {
        if (p.cu) o.k = o.slot - (o.first / p.span + o.seq);
        o.nspan = max(1, (o.last - o.first + p.span - 1) / p.span);
        if (o.k < 0) o.k = o.nspan;  // only where cu_seqlens is not sorted
        if (o.k < o.nspan) {
            o.first += o.k * p.span;
            if (o.last - o.first > p.span) o.last = o.first + p.span;
        }
    }
    return true;
}

// The rows [tb, tb + have) of a per-token tensor as a buffer resource: lanes
// give byte offsets from row tb, and an offset past the last row reads 0 and
// stores nothing, so no access is predicated.  Everything in it is uniform.
template <typename T>
__device__ __forceinline__ float value_of(uint32_t bits) {
    return __uint_as_float(sizeof(T) == 2 ? bits << 16 : bits);
}

template <typename T>
struct RowBuf {
    __amdgpu_buffer_rsrc_t r;
    // The element's bits, one register each: prefetched elements of 16 bits are
    // not paired up (which would wait for them at once).
    __device__ __forceinline__ uint32_t get(uint32_t off) const {
        if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
    }
    __device__ __forceinline__ void put(uint32_t off, float v) const {
        if constexpr (sizeof(T) == 2)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (T)v), r, off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), r, off, 0, 0);
    }
};
// An offset past every row of a chunk (at most 32 rows of 2^24 4-byte
// elements): added to the largest row offset it still does not wrap.
constexpr uint32_t kNowhere = 0x80000000u;
// A value the compiler does not carry sums of across loop iterations: the
// offsets off + i * step are formed anew in each segment (one add each) rather
// than kept, which took 30 registers and spilled.
__device__ __forceinline__ uint32_t fresh(uint32_t off) {
    asm volatile("" : "+v"(off));
    return off;
}

// width: elements of the last row that count.
template <typename T>
__device__ __forceinline__ RowBuf<T> row_buf(const void* src, int64_t stride, int64_t col, int tb,
                                             int have, int width) {
    const T* q = (const T*)src + (int64_t)tb * stride + col;
    const uint32_t n = src && have > 0
                           ? (uint32_t)(((have - 1) * stride + width) * (int64_t)sizeof(T)) : 0u;
    return {__builtin_amdgcn_make_buffer_rsrc((void*)q, (short)0, (int)n, 0x00020000)};
}

// The chunk's rows of one per-token tensor: lane nl of a quad loads token
// 4 i + nl from the lane's offset `off` (kNowhere in a lane without a channel).
template <typename T, int TW>
__device__ __forceinline__ void load_tokens(const void* src, int64_t stride, const Place& o, int tb,
                                            uint32_t (&r)[TW / 4]) {
    const RowBuf<T> q = row_buf<T>(src, stride, o.ch0, tb, min(o.last - tb, TW), o.width);
    const uint32_t step = (uint32_t)(4 * stride) * (uint32_t)sizeof(T);
    const uint32_t off =
        fresh(o.live ? (uint32_t)(o.nl * stride + o.e) * (uint32_t)sizeof(T) : kNowhere);
#pragma unroll
    for (int i = 0; i < TW / 4; ++i) r[i] = q.get(off + i * step);
}

// The chunk's B or C rows, NP entries a token (0 past N and past the sequence).
template <typename T, int NR, int TW>
struct Rows {
    static constexpr int K = TW * 4 * NR / 64;
    uint32_t v[K];
};
template <typename T, int NR, int TW>
__device__ __forceinline__ void load_rows(const void* src, int64_t stride, int64_t gstride, int N,
                                          const Place& o, int tb, Rows<T, NR, TW>& r) {
    constexpr int NP = 4 * NR, TK = 64 / NP;  // tokens a load
    const RowBuf<T> q = row_buf<T>(src, stride, o.group * gstride, tb, min(o.last - tb, TW), N);
    const int n = o.lane % NP, t0 = o.lane / NP;
    const uint32_t step = (uint32_t)(TK * stride) * (uint32_t)sizeof(T);
    const uint32_t off =
        fresh(n < N ? (uint32_t)(t0 * stride + n) * (uint32_t)sizeof(T) : kNowhere);
#pragma unroll
    for (int k = 0; k < r.K; ++k) r.v[k] = q.get(off + k * step);
}
// Into LDS as float32: token row t at dst + t * 2 NP.
template <typename T, int NR, int TW>
__device__ __forceinline__ void put_rows(float* dst, const Place& o, const Rows<T, NR, TW>& r) {
    constexpr int NP = 4 * NR, TK = 64 / NP;
    float* q = dst + o.lane / NP * 2 * NP + o.lane % NP;
#pragma unroll
    for (int k = 0; k < r.K; ++k) q[k * TK * 2 * NP] = value_of<T>(r.v[k]);
}

// A[n] log2(e) of the lane's channel and entries (0 where it has none).  A rate
// of -inf is kept finite: times a step of 0 it would be NaN.
template <int NR>
__device__ __forceinline__ void load_rates(const SelParams& p, const Place& o, float (&A2)[NR]) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int n = o.nl * NR + r;
        A2[r] = o.live && n < p.N ? fmaxf(p.A[(int64_t)n * p.E + o.ch] * kLog2e, -3e38f) : 0.f;
    }
}
// The lane's entries of its sequence's row of [S, N, E] (null reads 0, stores nothing).
template <int NR>
__device__ __forceinline__ void load_state(const float* src, const SelParams& p, const Place& o,
                                           float (&h)[NR]) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int n = o.nl * NR + r;
        h[r] = src && o.live && n < p.N ? src[((int64_t)o.seq * p.N + n) * p.E + o.ch] : 0.f;
    }
}
template <int NR>
__device__ __forceinline__ void store_state(float* dst, const SelParams& p, const Place& o,
                                            const float (&h)[NR]) {
    if (!dst || !o.live) return;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int n = o.nl * NR + r;
        if (n < p.N) dst[((int64_t)o.seq * p.N + n) * p.E + o.ch] = h[r];
    }
}

// h = P h + (state of the span), over n spans of the sequence from span `from`
// on (by = 1) or back (by = -1); P = exp of the span's sum of d times A.
template <int NR>
__device__ __forceinline__ void fold_spans(const float* states, const SelParams& p, const Place& o,
                                           const float (&A2)[NR], int from, int n, int by,
                                           float (&h)[NR]) {
    const int64_t step = (int64_t)p.nblk * 64 * by;
    int64_t at = ((int64_t)(o.slot - o.k + from) * p.nblk + o.blk) * 64 + o.lane;
#pragma unroll 4
    for (int j = 0; j < n; ++j, at += step) {
        const float d = p.span_d[at];
        float v[NR];
        __builtin_memcpy(v, states + at * NR, sizeof(v));
#pragma unroll
        for (int r = 0; r < NR; ++r) h[r] = fexp2(d * A2[r]) * h[r] + v[r];
    }
}

// ---- what a span does to a state ------------------------------------------------------------

// The wave takes a run of the span's chunks and keeps its state (and, for the
// backward pass, Q and P: q before = P q behind + Q) in registers; the waves'
// are joined once at the end.
template <typename T, int NR, bool BWD>
__global__ __launch_bounds__(512) void selscan_span_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kBwdTokens, NP = S::NP, MW = 8, Q = TW / 4;
    __shared__ __align__(16) float bc[MW][TW][2][NP];
    __shared__ __align__(16) float exD[MW][64], exH[MW][64][NR], exQ[BWD ? MW : 1][64][NR];
    Place o;
    if (!place_of(p, o) || o.k >= o.nspan) return;
    // nothing comes after a sequence's last span, and nothing before its first
    if (!BWD && o.k == o.nspan - 1) return;
    float A2[NR], h[NR], q[NR];
    load_rates<NR>(p, o, A2);
    const float dinit = o.live ? p.d_init[o.ch] : 0.f;
    const bool gated = p.z != nullptr;
    const int chunks = (o.last - o.first + TW - 1) / TW, run = (chunks + MW - 1) / MW;
    const int c0 = min(o.wave * run, chunks), c1 = min(c0 + run, chunks);
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) h[r] = q[r] = 0.f;
    uint32_t xr[Q], dr[Q], gr[Q], zr[Q];
    Rows<T, NR, TW> Br, Cr;
    auto fetch = [&](int t) {
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->x, k->xs, o, t, xr);
        load_tokens<T, TW>(k->d_raw, k->ds, o, t, dr);
        load_rows<T, NR, TW>(k->B, k->bs_t, k->bs_g, k->N, o, t, Br);
        if constexpr (BWD) {
            load_tokens<T, TW>(k->dy, k->gs, o, t, gr);
            load_tokens<T, TW>(k->z, k->zs, o, t, zr);
            load_rows<T, NR, TW>(k->C, k->cs_t, k->cs_g, k->N, o, t, Cr);
        }
    };
    int tb = o.first + c0 * TW;
    if (c0 < c1) fetch(tb);
    for (int c = c0; c < c1; ++c, tb += TW) {
        const int have = min(o.last - tb, TW);
        float d[Q], u[Q], w[Q], chunk_d = 0.f;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            d[i] = step_of(value_of<T>(dr[i]) + dinit, 4 * i + o.nl < have);
            u[i] = d[i] * value_of<T>(xr[i]);
            chunk_d += d[i];
            if constexpr (BWD) {
                const float zf = value_of<T>(zr[i]);
                w[i] = value_of<T>(gr[i]) * (gated ? zf * sigmoid(zf) : 1.f);
            }
        }
        wave_lds_fence();
        put_rows<T, NR, TW>(&bc[o.wave][0][0][0], o, Br);
        if constexpr (BWD) put_rows<T, NR, TW>(&bc[o.wave][0][1][0], o, Cr);
        wave_lds_fence();
        if (c + 1 < c1) fetch(tb + TW);
        float a[BWD ? TW : 1][NR];
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            float b[NR];
            lds_get<NR>(&bc[o.wave][t][0][o.nl * NR], b);
            const float dt = quad_lane(d[t / 4], t % 4), ut = quad_lane(u[t / 4], t % 4);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float at = fexp2(dt * A2[r]);
                h[r] = at * h[r] + b[r] * ut;
                if constexpr (BWD) a[t][r] = at;
            }
            if (t & 1) keep_order();
        }
        if constexpr (BWD) {
            float ql[NR];
#pragma unroll
            for (int t = TW - 1; t >= 0; --t) {
                float cc[NR];
                lds_get<NR>(&bc[o.wave][t][1][o.nl * NR], cc);
                const float wt = quad_lane(w[t / 4], t % 4);
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    ql[r] = t < TW - 1 ? a[t][r] * (cc[r] * wt + ql[r]) : a[t][r] * (cc[r] * wt);
                if (!(t & 1)) keep_order();
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) q[r] += fexp2(sum * A2[r]) * ql[r];
        }
        sum += quad_total(chunk_d);
    }
    exD[o.wave][o.lane] = sum;
    lds_put<NR>(exH[o.wave][o.lane], h);
    if constexpr (BWD) lds_put<NR>(exQ[o.wave][o.lane], q);
    __syncthreads();
    if (o.wave) return;
    for (int j = 1; j < MW; ++j) {
        const float dj = exD[j][o.lane];
        float hj[NR], qj[NR];
        lds_get<NR>(exH[j][o.lane], hj);
        if constexpr (BWD) lds_get<NR>(exQ[j][o.lane], qj);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            h[r] = fexp2(dj * A2[r]) * h[r] + hj[r];
            if constexpr (BWD) q[r] += fexp2(sum * A2[r]) * qj[r];
        }
        sum += dj;
    }
    const int64_t at = ((int64_t)o.slot * p.nblk + o.blk) * 64 + o.lane;
    p.span_d[at] = sum;
    __builtin_memcpy(p.span_h + at * NR, h, sizeof(h));
    if constexpr (BWD) __builtin_memcpy(p.span_q + at * NR, q, sizeof(q));
}

// ---- forward ------------------------------------------------------------------------------

template <typename T, int NR>
__global__ __launch_bounds__(64 * Shape<NR>::kFwdWaves) void selscan_fwd_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kFwdTokens, NP = S::NP, MW = S::kFwdWaves, Q = TW / 4;
    __shared__ __align__(16) float bc[MW][TW][2][NP];
    __shared__ __align__(16) float exP[2][MW][64][NR], exH[2][MW][64][NR];
    __shared__ __align__(16) float enter[2][64][NR];  // the state entering a segment
    Place o;
    if (!place_of(p, o)) return;
    const int waves = blockDim.x >> 6;
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
        if (p.span) fold_spans<NR>(p.span_h, p, o, A2, 0, o.k, 1, h);
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
        const ArgPtr k = fresh_args();
        load_tokens<T, TW>(k->z, k->zs, o, tb, zr);
        float d[Q], u[Q], x[Q];
        float sumd = 0.f;
        // tokens of this chunk that the sequence has (none or fewer: the rest
        // take d = 0, which passes the state on unchanged)
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
            if (ends && have > 0 && o.last - tb <= TW) store_state<NR>(p.final_state, p, o, h);
        } else if (o.wave == waves - 1) {
            lds_put<NR>(enter[turn ^ 1][o.lane], h);
        }
        wave_lds_fence();  // the next segment's rows go where these were read
    }
}

// ---- backward -----------------------------------------------------------------------------

// First the segments forward, only to find the state that enters each chunk
// (kept in chunk_states); then backward, where each wave holds a and h of its
// chunk in registers.  What enters the last segment's chunks is found there,
// so a sequence of one segment is walked once.
template <typename T, int NR>
__global__ __launch_bounds__(64 * Shape<NR>::kBwdWaves) void selscan_bwd_kernel(SelParams p) {
    using S = Shape<NR>;
    constexpr int TW = S::kBwdTokens, NP = S::NP, MW = S::kBwdWaves, Q = TW / 4;
    __shared__ __align__(16) float bc[MW][TW][2][NP];
    __shared__ __align__(16) float exP[2][MW][64][NR], exH[2][MW][64][NR], exQ[2][MW][64][NR];
    __shared__ __align__(16) float enter[3][64][NR];  // h or q entering a segment
    Place o;
    if (!place_of(p, o)) return;
    const int waves = blockDim.x >> 6;
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
        for (int j = waves - 1; j > o.wave; --j) {
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
        (int64_t)d->batch * d->seqlen > kMaxTokens)
        return SSD_ERR_SHAPE;
    if (d->d_state > SSD_SELSCAN_MAX_STATE) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

struct SelPlan {
    int32_t NR, S, bpg, nblk, upr;
    int32_t span, per;  // tokens of a span (0: sequences are not cut), spans a sequence
    int64_t slots, units, grid, T;
    size_t off_h, off_q, off_d, off_seg, off_w, off_bc, total;
};

template <typename F>
auto with_shape(int NR, F f) {
    if (NR == 2) return f(Shape<2>{});
    if (NR == 4) return f(Shape<4>{});
    if (NR == 8) return f(Shape<8>{});
    return f(Shape<16>{});
}

int sel_plan(const ssd_selscan_dims& d, bool bwd, SelPlan* pl) {
    pl->NR = entries_per_lane(d.d_state);
    pl->T = (int64_t)d.batch * d.seqlen;
    pl->S = d.nseq > 0 ? d.nseq : d.batch;
    pl->bpg = (int32_t)cdiv(d.channels / d.ngroups, kChan);
    const int64_t nblk = (int64_t)pl->bpg * d.ngroups;
    pl->nblk = (int32_t)nblk;
    pl->upr = (int32_t)cdiv(nblk, kRun);
    const int64_t seg = with_shape(pl->NR, [bwd](auto s) {
        return bwd ? s.kBwdSegment : s.kFwdTokens * s.kFwdWaves;
    });
    // Cut sequences into spans where that shortens the longest chain of
    // segments on a CU by more than the second launch costs.  A segment's cost
    // is 1; with spans its tokens are walked once more for the spans' states
    // (kAgain of a segment).  Packed sequences are taken as equally long.
    const double kAgain = bwd ? 0.35 : 0.6, kLaunch = 1.5, kFold = 0.05;
    const int64_t len = pl->S ? cdiv(pl->T, pl->S) : 0, nseg = cdiv(len, seg);
    const int64_t whole = (int64_t)pl->S * nblk;
    double best = (double)cdiv(whole, 256) * nseg;
    int64_t best_segs = 0;
    for (int64_t k = 2; k <= 64 && k <= nseg; ++k) {
        const int64_t segs = cdiv(nseg, k), kk = cdiv(nseg, segs);
        const double cost = (double)cdiv(whole * kk, 256) * segs * (1 + kAgain) + kLaunch + kFold * kk;
        if (cost < best) {
            best = cost;
            best_segs = segs;
        }
    }
    pl->span = (int32_t)(best_segs * seg);
    pl->per = best_segs ? (int32_t)cdiv(nseg, best_segs) : 1;
    pl->slots = d.nseq > 0 && pl->span ? pl->T / pl->span + pl->S : (int64_t)pl->S * pl->per;
    pl->units = pl->slots * pl->upr;
    pl->grid = cdiv(pl->units, kXcds) * kXcds * kRun;
    if (pl->grid > INT32_MAX) return SSD_ERR_SHAPE;
    size_t off = 0;
    pl->off_h = pl->off_q = pl->off_d = 0;
    if (pl->span) {
        const size_t states = (size_t)pl->slots * nblk * 64 * pl->NR * sizeof(float);
        pl->off_h = off;
        off = up256(off + states);
        pl->off_d = off;
        off = up256(off + (size_t)pl->slots * nblk * 64 * sizeof(float));
        pl->off_q = off;
        if (bwd) off = up256(off + states);
    }
    pl->off_seg = pl->off_w = pl->off_bc = off;
    if (bwd) {
        const int64_t waves = with_shape(pl->NR, [](auto s) { return s.kBwdWaves; });
        off = up256(off + (size_t)(pl->T / seg + pl->S + 1) * waves * nblk * 64 * pl->NR * sizeof(float));
        pl->off_w = off;
        off = up256(off + (size_t)pl->slots * (d.d_state + 2) * d.channels * sizeof(float));
        pl->off_bc = off;
        off = up256(off + (size_t)nblk * pl->T * 8 * pl->NR * sizeof(float));
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

template <typename T, int NR>
void launch_sel(const SelParams& p, unsigned grid, bool bwd, hipStream_t s) {
    if (bwd) {
        if (p.span) selscan_span_kernel<T, NR, true><<<dim3(grid), dim3(512), 0, s>>>(p);
        selscan_bwd_kernel<T, NR><<<dim3(grid), dim3(64 * Shape<NR>::kBwdWaves), 0, s>>>(p);
    } else {
        if (p.span) selscan_span_kernel<T, NR, false><<<dim3(grid), dim3(512), 0, s>>>(p);
        selscan_fwd_kernel<T, NR><<<dim3(grid), dim3(64 * Shape<NR>::kFwdWaves), 0, s>>>(p);
    }
}
template <typename T>
void launch_sel(const SelParams& p, int NR, unsigned grid, bool bwd, hipStream_t s) {
    if (NR == 2) launch_sel<T, 2>(p, grid, bwd, s);
    else if (NR == 4) launch_sel<T, 4>(p, grid, bwd, s);
    else if (NR == 8) launch_sel<T, 8>(p, grid, bwd, s);
    else launch_sel<T, 16>(p, grid, bwd, s);
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
    if (dims->dtype == SSD_BF16) launch_sel<bf16>(p, pl.NR, (unsigned)pl.grid, false, s);
    else launch_sel<float>(p, pl.NR, (unsigned)pl.grid, false, s);
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
    p.span_h = (float*)(ws + pl.off_h);
    p.span_q = (float*)(ws + pl.off_q);
    p.span_d = (float*)(ws + pl.off_d);
    p.chunk_states = (float*)(ws + pl.off_seg);
    p.part_w = (float*)(ws + pl.off_w);
    p.part_bc = (float*)(ws + pl.off_bc);
    if (dims->dtype == SSD_BF16) launch_sel<bf16>(p, pl.NR, (unsigned)pl.grid, true, s);
    else launch_sel<float>(p, pl.NR, (unsigned)pl.grid, true, s);
    if ((st = launched()) != SSD_OK) return st;
    const int NP = 4 * pl.NR;
    const int64_t items = pl.T * dims->ngroups * 2 * NP;
    if (items > 0) {
        const int64_t grid = cdiv(items, 256);
        if (grid > INT32_MAX) return SSD_ERR_SHAPE;
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
