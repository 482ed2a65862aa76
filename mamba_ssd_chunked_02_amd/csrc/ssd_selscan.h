// Shared by the selective scan's forward (ssd_selscan.hip) and backward
// (ssd_selscan_bwd.hip) kernels: the mathematics, the mapping, and the parts of a
// chunk both walk.  Internal.
//
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
// Every token of every channel costs N exponentials and about 4 N products
// (backward three times that), so both directions are bound by the vector units,
// not by memory; nothing here has the shape of a matrix product (the decay
// differs in every lane).
//
// Mapping.  Four lanes of a wave hold one channel (a quad; N / 4 state entries
// each), a wave 16 channels; chunks are TW tokens.  Forward, a workgroup owns 16
// channels of one sequence and its waves take consecutive chunks.  A segment of
// waves x TW tokens goes: (1) every wave scans its chunk from a zero state, keeping all
// a_t,n in registers; (2) the waves exchange (decay product, state) in LDS and
// fold those before them; (3) every wave scans its chunk again from the state
// that enters it, without forming an exponential.  The state that leaves the
// segment enters the next one, so a sequence needs no other launch and no
// global scratch (scanning twice costs 8 issues a state entry and token where a
// scan in order costs 6, but only this fills the chip).  The vector units bound
// it: 2 x 2048 tokens x 1536 channels x 16 states 47 us on 192 of the 256 CUs,
// 65536 packed tokens 538 to 566 us; their issue slots take 45 and 505 us at 2.4 GHz.
// Per-token values (d, u, y) live in the quad's lanes, token
// 4 i + k in lane k, and reach the other three as DPP operands.
#pragma once

#include "ssd_layer.h"

namespace ssd {

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
    float* span_h;       // forward: spans' states from zero [slots][blocks][64][NR]
    float* span_d;       // their sums of d [slots][blocks][64]
    float* run_h;        // backward: runs' states from zero, then entering them
    float* run_q;        // q before them from zero, then q entering from behind
                         // [runs][blocks][64][NR]
    float* run_d;        // their sums of d [runs][blocks][64]
    float* chunk_h;      // h before a run's chunks, from zero [chunks][blocks][64][NR]
    float* chunk_d;      // the sum of d there [chunks][blocks][64]
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

// The launches of the backward scan up to the sums over channel blocks and
// sequences (its own translation unit); runs: of a sequence.
int launch_selscan_bwd(const SelParams& p, int32_t dtype, int NR, int64_t runs, unsigned grid,
                       hipStream_t s);

namespace {

// The kernel's argument block, read anew: what is loaded through the returned
// pointer is not kept in scalar registers across the loops around it.  (Kept,
// the pointers and strides of ten tensors did not fit and went through vector
// lanes: 528 lane reads in the backward loop.)
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
    static constexpr int kFwdWaves = NR <= 4 ? 16 : 8;  // of a workgroup, at most
    static constexpr int kFwdPerSimd = kFwdWaves / 4;  // smaller workgroups as many
    static constexpr int kBwdTokens = NR == 2 ? 16 : NR == 4 ? 8 : 4;
    static constexpr int kRunTokens = 64;              // backward: of a wave
    static constexpr int kBwdPerSimd = NR <= 4 ? 3 : NR == 8 ? 2 : 1;
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
    float d = step_softplus(raw);
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

// A[n] log2(e) of the lane's channel and entries (0 where it has none).
template <int NR>
__device__ __forceinline__ void load_rates(const SelParams& p, const Place& o, float (&A2)[NR]) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int n = o.nl * NR + r;
        A2[r] = o.live && n < p.N ? finite_rate(p.A[(int64_t)n * p.E + o.ch] * kLog2e) : 0.f;
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

// h through the n spans of the sequence before this one: h = P h + (state of the
// span from zero), P = exp of the span's sum of d times A.
template <int NR>
__device__ __forceinline__ void fold_spans(const SelParams& p, const Place& o, const float (&A2)[NR],
                                           float (&h)[NR]) {
    int64_t at = ((int64_t)(o.slot - o.k) * p.nblk + o.blk) * 64 + o.lane;
#pragma unroll 4
    for (int j = 0; j < o.k; ++j, at += (int64_t)p.nblk * 64) {
        const float d = p.span_d[at];
        float v[NR];
        __builtin_memcpy(v, p.span_h + at * NR, sizeof(v));
#pragma unroll
        for (int r = 0; r < NR; ++r) h[r] = fexp2(d * A2[r]) * h[r] + v[r];
    }
}

}  // namespace
}  // namespace ssd
