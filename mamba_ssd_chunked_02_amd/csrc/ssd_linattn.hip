// Linear attention with a constant decay per head, forward and backward.
//
//   S_t = l S_{t-1} + k_t^T v_t,  y_t = scale q_t S_t        (l = exp(decay[h]); S: K x V)
//
// in chunks of C tokens.  With E the state that enters a chunk, decayed to its first token
// (E = l S_{-1}), and i, j the tokens of the chunk:
//   y_i = scale (l^i q_i E + sum_{j <= i} l^{i-j} (q_i . k_j) v_j)
//   E'  = l^C E + sum_j l^{C-j} k_j^T v_j
// The gradients are scans of the same form with other roles:
//   dq = scan(q: dy, k: v,  v: k)           in the forward's order,   state S^T
//   dk = scan(q: v,  k: dy, v: scale q)     in the opposite order,    state R^T
//   dv = scan(q: k,  k: scale q, v: dy)     in the opposite order,    state R
// with R_t = scale q_t^T dy_t + l R_{t+1} (R_{L-1} adds d_final, which therefore enters
// undecayed) and dinit = l R_0: one kernel serves all four (LinPass::init_pow, final_pow).
//
// (C = 32.)  A workgroup walks the chunks of one span of a sequence for one head and VT columns of V,
// the state in registers: each of its four waves holds all K rows of VT / 4 columns, so no
// product needs a sum across waves.  Where sequences x heads do not fill the chip a
// sequence is cut into spans: their states are formed first (STATE), joined along the
// sequence (linattn_join) and then every span is walked from its own incoming state.
//
// What bounds it, and figures (one MI355X, whole calls).  65536 packed tokens x 16 heads of 128 x
// 128, bf16 (1.1 GB): 452 us, where its bytes take 215: the spans' states read k and v a second
// time, near the memory's rate, and in the scan the two waves of a SIMD do not cover each other's
// chain of a chunk (load, LDS, products, barrier): matrix units are busy 33 % of the time, LDS 28,
// vector units 35 to 44.
// 32768 x 8 heads of 256 (0.54 GB): 358 us, with one wave a SIMD; forming its states reads 1.9
// TB/s.  4096 tokens x 12 heads of 64 x 128 34 us and their gradients 78: three and six launches of 8
// to 26 us, of which 4 are before the first chunk.  Float32 runs at the matrix units' float32 rate.
// More waves of fewer columns wait for LDS (each reads every key and query), a third wave a SIMD
// spills, and a third buffer of tiles gained nothing.
#include <type_traits>

#include "ssd_layer.h"

namespace ssd {
namespace {

struct LinPass {
    const void* q;
    const void* k;
    const void* v;
    void* o;
    int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
    const float* decay;
    const float* init;  // [S][H] states of K * V entries, entry (k, v) at k s_k + v s_v
    float* final;
    float* spans;       // [slots][H][vtiles] span states in register order
    const int32_t* cu;
    int64_t L, T, span; // tokens of a sequence without cu, of all, of a span
    int32_t S, H, K, V, s_k, s_v;
    int32_t qdiv, kdiv, vdiv;  // head h reads head h / div
    int32_t slots, per;        // span slots; spans of a sequence without cu
    int32_t vtiles, together, reverse, init_pow, final_pow;
    float in_scale, out_scale;
};

// Passes of one launch: blockIdx.y's is its own.
struct LinPasses {
    LinPass p[3];
};

// Sequence and span of a slot.  With cu sequence i owns the slots from cu[i] / span + i on:
// one for every span it can have, and at least one.
struct Span {
    int64_t first, len;  // the sequence's tokens
    int64_t t0;          // of the span, in processing order
    int32_t seq, at;
};
__device__ __forceinline__ int64_t slot_base(const LinPass& p, int i) {
    const int64_t c = p.cu[i];
    return (c < 0 ? 0 : (c > p.T ? p.T : c)) / p.span + i;
}
__device__ __forceinline__ Span span_of(const LinPass& p, int slot) {
    Span s;
    if (!p.cu) {
        s.seq = slot / p.per;
        s.at = slot - s.seq * p.per;
        s.first = s.seq * p.L;
        s.len = p.L;
    } else {
        int lo = 0, hi = p.S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (slot_base(p, mid) <= slot) lo = mid; else hi = mid - 1;
        }
        s.seq = lo;
        s.at = slot - (int)slot_base(p, lo);
        int64_t last;
        sequence_span(p.cu, lo, 0, p.T, &s.first, &last);
        s.len = last - s.first;
    }
    s.t0 = s.at * p.span;
    return s;
}

// l^n in double (0^0 = 1): products of many chunks keep the rate's low bits.
__device__ __forceinline__ double power(float decay, int64_t n) {
    return n == 0 ? 1.0 : exp((double)n * (double)decay);
}

// Factors l^n, one for each of many steps of n tokens, as floats whose product stays the
// power: what a float leaves out of l^n (`low`, relative) is gathered and put back whenever
// it has grown to a unit of the last place.  Over 1000 steps of 32 tokens a fixed factor is
// up to 3e-5 off.  A power below 2^-126 has fewer bits than that, and 1 over it may be infinite:
// what is left out of it, of a state that is gone in two steps, is not gathered.
struct Rate {
    float rate, low, unrate, owed;
    __device__ __forceinline__ explicit Rate(double exact) {
        rate = (float)exact;
        const bool normal = rate >= 1.17549435e-38f;
        low = normal ? (float)((exact - (double)rate) / (double)rate) : 0.f;
        unrate = normal ? 1.f / rate : 0.f;
        owed = 0.f;
    }
    __device__ __forceinline__ float next() {
        owed += low;
        const float f = fmaf(rate, owed, rate);
        owed -= (f - rate) * unrate;
        return f;
    }
};

// An LDS tile of C tokens, row-major in 16-byte units, unit u of row r at place u ^ swap(r): a
// tile is then filled by loads straight from memory, which put 64 lanes' units next to each
// other, and every read below touches all banks evenly (16 rows of one half unit, 4 rows of
// two or four units).
constexpr int C = 32;  // tokens of a chunk
template <typename T, int COLS>
struct Tile {
    static constexpr int EPU = 16 / sizeof(T), UPR = COLS / EPU, ROW = COLS * (int)sizeof(T);  // ROW: bytes
    __device__ static __forceinline__ int swap(int r) {
        return UPR == 8 ? ((r >> 1) & 3) << 1 | ((r >> 3) & 1) : (r & 7) << 1 | ((r >> 3) & 1);
    }
    // byte address of column c of row r
    __device__ static __forceinline__ int at(int r, int c) {
        return r * ROW + (((c / EPU) ^ swap(r)) * 16) + c % EPU * (int)sizeof(T);
    }
};

// Rows and columns of two result tiles side by side are dealt out so that a lane's 4 entries of
// each are 8 neighbours in memory: entry m of tile `half` is 8 (m / 4) + 4 half + m % 4 of 32.
template <int TILES>
__device__ __forceinline__ int dealt(int half, int m) {
    return TILES == 2 ? 8 * (m >> 2) + 4 * half + (m & 3) : m;
}

// MFMA operands.  Over 32 keys a lane of group g has keys 8g..8g+7, over 32 tokens tokens
// 4g..4g+3 and 16+4g..16+4g+3: the orders in which a pair of result tiles holds them (the
// state's with its keys dealt out, the scores' as they come).  Multiples of 16 rows and columns
// move an address by a constant: + r0 ROW, ^ c0 sizeof(T).
template <typename T, int COLS>
__device__ __forceinline__ int row_base(int lane) {
    return Tile<T, COLS>::at(lane & 15, 8 * (lane >> 4));
}
// tile[r0 + l16][c0 ..]
template <int COLS>
__device__ __forceinline__ bf16x8 row_frag(const bf16*, const char* t, int base, int r0, int c0) {
    return *(const bf16x8*)(t + (base ^ c0 * 2) + r0 * Tile<bf16, COLS>::ROW);
}
template <int COLS>
__device__ __forceinline__ f32x8 row_frag(const float*, const char* t, int base, int r0, int c0) {
    return cat<f32x8, f32x4>(*(const f32x4*)(t + (base ^ c0 * 4) + r0 * Tile<float, COLS>::ROW),
                             *(const f32x4*)(t + (base ^ c0 * 4 ^ 16) + r0 * Tile<float, COLS>::ROW));
}
// tile[0 ..][c0 + the lane's column], the first of TILES side by side; ^ 4 sizeof(T) is the second
template <typename T, int COLS, int TILES>
__device__ __forceinline__ int col_base(int lane) {
    const int j = lane & 15, r = 4 * (lane >> 4);
    if (sizeof(T) == 2) return Tile<T, COLS>::at(r + (j >> 2), dealt<TILES>(0, 4 * (j & 3)));
    return Tile<T, COLS>::at(r, dealt<TILES>(0, j));
}
template <int COLS>
__device__ __forceinline__ bf16x8 col_frag(const bf16*, const char* t, int base, int c0) {
    const bf16* const q = (const bf16*)(t + (base ^ c0 * 2));
    return cat<bf16x8, bf16x4>(ldtr(q), ldtr(q + 16 * COLS));
}
template <int COLS>
__device__ __forceinline__ f32x8 col_frag(const float*, const char* t, int base, int c0) {
    f32x8 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // swap(4g + k) = swap(4g) ^ 2k
        const float* const q = (const float*)(t + (base ^ (c0 * 4) ^ (32 * k))) + k * COLS;
        v[k] = q[0];
        v[4 + k] = q[16 * COLS];
    }
    return v;
}

// x less the first (I = 0) or second value of a pair: exact where that is x rounded.  One instruction
// on the pair as it is packed, where unpacking and subtracting are two.  The constant is kept in a
// register: an inline -1 would be the float32 one, which is -1 in the pair's second place.
template <int I>
__device__ __forceinline__ float less(float x, bf16 a, bf16 b) {
    typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
    uint32_t one = I == 0 ? 0x0000bf80u : 0xbf800000u;
    asm("" : "+s"(one));
    return __builtin_amdgcn_fdot2_f32_bf16(bf16x2{a, b}, __builtin_bit_cast(bf16x2, one), x, false);
}
// c + a (v w), v w in full: a float32 state that takes bfloat16 inputs would lose 16 bits
// to one rounded product, so it is split into three bfloat16 values, whose sum is exact.
__device__ __forceinline__ f32x4 mma_weighted(const bf16x8& a, const bf16x8 (&vw)[3], f32x4 c) {
    c = mma(a, vw[2], c);
    c = mma(a, vw[1], c);
    return mma(a, vw[0], c);
}
__device__ __forceinline__ f32x4 mma_weighted(const f32x8& a, const f32x8 (&vw)[1], f32x4 c) {
    return mma(a, vw[0], c);
}
__device__ __forceinline__ void weigh(const bf16x8& v, const f32x8& w, bf16x8 (&o)[3]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float x = (float)v[j] * w[j], y = (float)v[j + 1] * w[j + 1];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            o[i][j] = (bf16)x;
            o[i][j + 1] = (bf16)y;
            x = less<0>(x, o[i][j], o[i][j + 1]);
            y = less<1>(y, o[i][j], o[i][j + 1]);
        }
    }
}
__device__ __forceinline__ void weigh(const f32x8& v, const f32x8& w, f32x8 (&o)[1]) { o[0] = v * w; }

// The rows of a chunk of one per-token tensor as a buffer resource: offsets are in bytes from
// the chunk's lowest address, and one outside its rows reads 0 and stores nothing, so nothing
// is predicated.  A chunk's rows span less than 2^31 bytes (32 rows of 2^24 elements),
// which kNowhere is past.
constexpr uint32_t kNowhere = 0x80000000u;
struct Rows {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __amdgpu_buffer_rsrc_t r;
    u32x4 words;  // the same
    // `low`: the lowest row; have rows, `step` bytes apart, of `width` bytes
    __device__ __forceinline__ Rows(const void* low, uint32_t step, int have, uint32_t width)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(low), (short)0,
                                              (int)((uint32_t)(have - 1) * step + width), 0x00020000)),
          words{word((uint32_t)(uintptr_t)low), word((uint32_t)((uintptr_t)low >> 32) & 0xffff),
                word((uint32_t)(have - 1) * step + width), 0x00020000u} {}
    __device__ static __forceinline__ uint32_t word(uint32_t v) {
        return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
    }
};

// Scores, and the state where queries meet it, as bfloat16 operands in two parts, 16 bits.  In one
// part their rounding is as large as the output's own, and where few of them are summed nothing
// averages it out.  With the state in one part outputs are 2.25e-3 off (root of the mean square),
// with two 1.66e-3, which is the output's own rounding.  It costs two matrix instructions for 32 keys and
// 16 columns: 65536 tokens x 16 heads of 128 x 128 452 us where one part takes 437, 32768 x 8 of
// 256 x 256 358 and 328, 4096 x 12 of 64 x 128 34.0 and 33.6, their gradients 78.0 and 75.9.
template <typename T> constexpr int kSplit = sizeof(T) == 2 ? 2 : 1;
__device__ __forceinline__ void in_parts(const f32x8& s, bf16x8 (&o)[2]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        o[0][j] = (bf16)s[j];
        o[0][j + 1] = (bf16)s[j + 1];
        o[1][j] = (bf16)less<0>(s[j], o[0][j], o[0][j + 1]);
        o[1][j + 1] = (bf16)less<1>(s[j + 1], o[0][j], o[0][j + 1]);
    }
}
__device__ __forceinline__ void in_parts(const f32x8& s, f32x8 (&o)[1]) { o[0] = s; }

// N neighbours of a row at byte offset `off`, of which `left` lie in the row: whole units of 16
// bytes (or the one run of 8) lie in it or not, each for itself, since a row of float32 may end
// between the two units of a run.
template <typename OT, int N, bool SINGLY>
__device__ __forceinline__ void store_run(const Rows& b, uint32_t off, int left, const float (&x)[N]) {
    typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    OT o[N];
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = (OT)x[j];
    if constexpr (!SINGLY) {
        if constexpr (sizeof(o) == 8) {
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, o), b.r, left >= N ? off : kNowhere,
                                                  0, 0);
        } else {
            constexpr int U = 16 / sizeof(OT);
#pragma unroll
            for (int j = 0; j < (int)sizeof(o) / 16; ++j) {
                u32x4 v;
                __builtin_memcpy(&v, (const char*)o + 16 * j, 16);
                __builtin_amdgcn_raw_buffer_store_b128(v, b.r, left >= (j + 1) * U ? off + 16 * j : kNowhere, 0, 0);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t at = j < left ? off + j * (uint32_t)sizeof(OT) : kNowhere;
            if constexpr (sizeof(OT) == 2)
                __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, o[j]), b.r, at, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, o[j]), b.r, at, 0, 0);
        }
    }
}

// Waves a SIMD that the kernel is compiled for: two workgroups a CU.
constexpr int lin_waves(int KD, int VT, int size) { return 2 * (2 * KD + VT) * C * size > 80 * 1024 - 1024 ? 1 : 2; }

template <typename T> constexpr int kParts = sizeof(T) == 2 ? 3 : 1;

// 16 bytes of each lane, to 1 KB of LDS from `to` on.  In assembly, since the compiler has every
// transposing read of LDS wait for all such loads that it knows of, the next chunk's among them;
// vm_wait is theirs.  The wait states are those of a scalar register that a vector instruction
// wrote (5) and of m0 (1), which the compiler does not see to in here.
__device__ __forceinline__ void load_unit(const Rows& b, char* to, uint32_t off) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)to);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 ::"s"(at), "v"(off), "s"(b.words) : "memory", "m0");
}

// What a kernel is built for: FULL, K is KD and rows are whole units; PADDED, K is less, and
// products over nothing but padding are skipped; RAGGED, rows need not be whole units either.
enum { FULL, PADDED, RAGGED };

// The chunks of one per-token tensor on their way into LDS tiles.  Row r of a tile is the
// chunk's r-th token in processing order (with `back` the chunks lie in memory from the last
// to the first, and so do their rows); rows past the chunk's end are zeros, or values of the
// chunk where its rows lie closer than they are wide, and columns past `cols` zeros.  Each of
// four waves issues every fourth load of 64 units straight into LDS: nothing passes through
// registers and nothing is waited for.  RAGGED: element by element, waiting.
template <typename T, int COLS, int MODE>
struct Stream {
    using L = Tile<T, COLS>;
    static constexpr int N = C * L::UPR / 256;
    const char* low;   // lowest row of the next chunk, were it full
    uint32_t step, width, off[N];
    int32_t cols;
    bool back;
    // `first`: the first token's row
    __device__ __forceinline__ Stream(const T* first, int64_t stride, int cols_, bool back_)
        : step((uint32_t)stride * (uint32_t)sizeof(T)), width(cols_ * (uint32_t)sizeof(T)), cols(cols_), back(back_) {
        low = (const char*)first - (back ? (int64_t)(C - 1) * step : 0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int place = (i * 4 + wave_id()) * 64 + (threadIdx.x & 63), r = place / L::UPR;
            const int c = (place % L::UPR ^ L::swap(r)) * L::EPU;
            off[i] = (uint32_t)(back ? C - 1 - r : r) * step + (uint32_t)(c * sizeof(T));
            if (MODE != RAGGED && c >= cols) off[i] = kNowhere;
        }
    }
    // the next chunk, of `have` tokens
    __device__ __forceinline__ void fill(char* tile, int have) {
        const uint32_t gap = back ? (uint32_t)(C - have) * step : 0;  // kNowhere - gap stays past the rows
        const Rows b(low + gap, step, have, width);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int load = i * 4 + wave_id();
            if constexpr (MODE != RAGGED) {
                load_unit(b, tile + load * 1024, off[i] - gap);
            } else {
                const int place = load * 64 + (threadIdx.x & 63);
                const int c = (place % L::UPR ^ L::swap(place / L::UPR)) * L::EPU;
                T u[L::EPU];
#pragma unroll
                for (int j = 0; j < L::EPU; ++j) {
                    const uint32_t at = c + j < cols ? off[i] - gap + j * (uint32_t)sizeof(T) : kNowhere;
                    if constexpr (sizeof(T) == 2)
                        u[j] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(b.r, at, 0, 0));
                    else
                        u[j] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(b.r, at, 0, 0));
                }
                __builtin_memcpy(__builtin_assume_aligned(tile + place * 16, 16), u, 16);
            }
        }
        low += back ? -(int64_t)C * step : (int64_t)C * step;
    }
};

// The chunk being worked on and the next one.
template <typename T, int KD, int VT, bool STATE>
struct __attribute__((aligned(1024))) Shared {
    char q[STATE ? 0 : 2][C * Tile<T, KD>::ROW];
    char k[2][C * Tile<T, KD>::ROW];
    char v[2][C * Tile<T, VT>::ROW];
    double pc;        // l^C
    float pw[C + 4];  // l^n
    float w[2][C];    // the tokens' weights in the state behind their chunk; behind the last
};

// Workgroups that read the same rows (the V tiles of a head, the heads of a group) follow each
// other on one XCD, whose L2 then serves all but the first: workgroups go to the 8 XCDs in turn.
__device__ __forceinline__ uint32_t same_xcd(uint32_t id, uint32_t together, uint32_t n) {
    const uint32_t whole = n / (8 * together) * (8 * together);
    if (id >= whole) return id;
    const uint32_t x = id % 8, i = id / 8;
    return (i / together * 8 + x) * together + i % together;
}

// One span (or, STATE, only its state).  OT: the output's type.
template <typename T, typename OT, int KD, int VT, int MODE, bool STATE>
__global__ __launch_bounds__(256, lin_waves(KD, VT, sizeof(T))) void linattn_kernel(LinPasses ps) {
    const LinPass& p = ps.p[blockIdx.y];
    touch_args(p);
    using X8 = typename Vec<T>::x8;
    constexpr int CB = VT / 64, KB = KD / 16, KS = KD / 32;
    __shared__ Shared<T, KD, VT, STATE> sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), l16 = lane & 15, g = lane >> 4;
    uint32_t id = same_xcd(blockIdx.x, p.together, gridDim.x);
    const int vt = id % (uint32_t)p.vtiles;
    id /= (uint32_t)p.vtiles;
    const int h = id % (uint32_t)p.H, slot = id / (uint32_t)p.H;
    const Span sp = span_of(p, slot);
    if (sp.at < 0 || (sp.at > 0 && sp.t0 >= sp.len)) return;
    const int64_t n = imin(p.span, sp.len - sp.t0);
    const bool last = sp.t0 + n >= sp.len;
    if (STATE && last) return;  // no span behind it
    const int64_t block = ((int64_t)sp.seq * p.H + h) * ((int64_t)p.K * p.V);
    const int v0 = vt * VT, vcols = min(VT, p.V - v0), c0 = wave * (16 * CB);
    float* const mine = p.spans + (((int64_t)slot * p.H + h) * p.vtiles + vt) * (KD * VT) +
                        wave * (CB * KB * 256) + lane * 4;

    if (!STATE && n == 0) {  // an empty sequence hands on what came in
        if (p.final)
            for (int i = tid; i < p.K * vcols; i += 256) {
                const int64_t e = block + (int64_t)(i / vcols) * p.s_k + (int64_t)(v0 + i % vcols) * p.s_v;
                p.final[e] = p.init ? p.init[e] : 0.f;
            }
        return;
    }

    const bool back = p.reverse != 0;
    const int64_t tok0 = back ? sp.first + sp.len - 1 - sp.t0 : sp.first + sp.t0;
    Stream<T, KD, MODE> ks((const T*)p.k + tok0 * p.k_t + (h / p.kdiv) * p.k_h, p.k_t, p.K, back);
    Stream<T, KD, MODE> qs((const T*)p.q + tok0 * p.q_t + (h / p.qdiv) * p.q_h, p.q_t, p.K, back);
    Stream<T, VT, MODE> vs((const T*)p.v + tok0 * p.v_t + (h / p.vdiv) * p.v_h + v0, p.v_t, vcols, back);
    auto fetch = [&](int have, int to) {
        if constexpr (!STATE) qs.fill(sh.q[to], have);
        ks.fill(sh.k[to], have);
        vs.fill(sh.v[to], have);
    };
    fetch((int)imin(C, n), 0);

    // One exponential a thread: l^0 .. l^C.
    if (tid <= C) {
        const double x = power(p.decay[h], tid);
        sh.pw[tid] = (float)x;
        if (tid == C) sh.pc = x;
    }

    // the state that comes in, in flight while the powers are formed: from the workspace where
    // the sequence is in spans
    f32x4 st[KB][CB];
    const bool split = p.per != 1, come = !STATE && !split && p.init;
    const Rows sb(come ? (const void*)(p.init + block) : (const void*)p.decay, 0, 1,
                  come ? (uint32_t)(p.K * p.V) * 4 : 0);
    // this lane's first entry of each column block; its rows are s_k apart
    uint32_t s0[CB];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const int vc = c0 + dealt<CB>(cb, l16);
        s0[cb] = vc < vcols ? (uint32_t)(8 * g * p.s_k + (v0 + vc) * p.s_v) * 4 : kNowhere;
    }
    auto entry = [&](int kb, int cb, int r) {
        const int k = 32 * (kb / 2) + 4 * (kb % 2) + r;  // and 8 g
        return 8 * g + k < p.K ? s0[cb] + (uint32_t)(k * p.s_k * 4) : kNowhere;
    };
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            if (STATE) {
                st[kb][cb] = f32x4{0.f, 0.f, 0.f, 0.f};
            } else if (split) {
                st[kb][cb] = *(const f32x4*)(mine + (cb * KB + kb) * 256);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    st[kb][cb][r] = __uint_as_float(
                        __builtin_amdgcn_raw_buffer_load_b32(sb.r, entry(kb, cb, r), 0, 0));
            }
        }
    vm_wait<0>();
    block_sync();
    Rate rate(sh.pc);
    // weights of a score: within a block of 16 tokens, and of rows 16-31 with columns 0-15
    f32x4 tw[2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int d = l16 - 4 * g - r;
        const float x = p.in_scale * p.out_scale * sh.pw[max(d, 0)];
        tw[0][r] = d >= 0 ? x : 0.f;
        tw[1][r] = p.in_scale * p.out_scale * sh.pw[16 + d];
    }
    // the sequence's last chunk, of `tail` tokens, is followed by no decay, or by final_pow
    const int tail = (int)((n - 1) % C) + 1, top = tail - 1 + p.final_pow;
    if (tid < C) {
        sh.w[0][tid] = p.in_scale * sh.pw[C - tid];
        sh.w[1][tid] = tid < tail ? p.in_scale * sh.pw[max(top - tid, 0)] : 0.f;
    }
    const float closing = sh.pw[top], out_scale = p.out_scale;
    block_sync();
    // The state is st * held: a chunk's factor goes into `held`, and into the entries only once
    // that has left [1/256, 256] (every sixth chunk at l = 31/32).
    float held = !STATE && !split && p.init_pow ? sh.pw[1] : 1.f;

    const int rb = row_base<T, KD>(lane), kc = col_base<T, KD, 2>(lane), vb = col_base<T, VT, CB>(lane);
    // outputs: this lane's 4 CB columns of tokens l16 and 16 + l16
    const uint32_t os = (uint32_t)p.o_t * (uint32_t)sizeof(OT);
    const int oc = c0 + dealt<CB>(0, 4 * g);
    const char* op = (const char*)((OT*)p.o + tok0 * p.o_t + h * p.o_h + v0) - (back ? (int64_t)(C - 1) * os : 0);
    const uint32_t ooff = (uint32_t)(back ? C - 1 - l16 : l16) * os + (uint32_t)(oc * sizeof(OT));
    const uint32_t onext = back ? 0u - 16 * os : 16 * os, owidth = vcols * (uint32_t)sizeof(OT);
    const int keys = p.K;
    const bool final = p.final != nullptr;
    const int chunks = (int)cdiv(n, C);
    for (int i = 0; i < chunks; ++i) {
        const int buf = i & 1;
        const bool end = i + 1 == chunks, close = last && end;  // of the span, of the sequence
        const int cl = end ? tail : C;
        // Tables are read ahead of the loads of the next chunk: the compiler would have a read of
        // them wait for those loads.
        const float* const wt = sh.w[close ? 1 : 0] + 4 * g;
        f32x8 w = cat<f32x8, f32x4>(*(const f32x4*)wt, *(const f32x4*)(wt + 16));
        float f0 = sh.pw[l16], f1 = sh.pw[16 + l16];
        asm volatile("" : "+v"(w), "+v"(f0), "+v"(f1));
        if (!end) fetch(i + 2 == chunks ? tail : C, buf ^ 1);
        const char* const tq = sh.q[STATE ? 0 : buf];
        const char* const tk = sh.k[buf];
        const char* const tv = sh.v[buf];
        const float come_in = held, now = held * (close ? closing : rate.next());
        const bool drop = !(now >= 0.00390625f && now <= 256.f);
        held = drop ? 1.f : now;
        // v, plain and weighted for the state behind the chunk
        X8 vf[CB], vw[CB][kParts<T>];
        w *= __builtin_amdgcn_rcpf(held);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            vf[cb] = col_frag<VT>((const T*)nullptr, tv, vb ^ cb * 4 * (int)sizeof(T), c0);
            weigh(vf[cb], w, vw[cb]);
        }
        // Results are transposed: a lane has 4 columns of token 16 ib + l16, and of the scores 4
        // tokens j of one row i, which is the order in which they meet the values.
        f32x4 acc[2][CB];
        if constexpr (!STATE) {
            f32x4 s00 = {0.f, 0.f, 0.f, 0.f}, s01 = s00, s11 = s00;
#pragma unroll
            for (int ib = 0; ib < 2; ++ib)
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) acc[ib][cb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                if (MODE != FULL && kk && 32 * kk >= keys) break;
                const X8 q0 = row_frag<KD>((const T*)nullptr, tq, rb, 0, 32 * kk);
                const X8 q1 = row_frag<KD>((const T*)nullptr, tq, rb, 16, 32 * kk);
                const X8 k0 = row_frag<KD>((const T*)nullptr, tk, rb, 0, 32 * kk);
                const X8 k1 = row_frag<KD>((const T*)nullptr, tk, rb, 16, 32 * kk);
                s00 = mma(k0, q0, s00);
                s01 = mma(k0, q1, s01);
                s11 = mma(k1, q1, s11);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    X8 e[kSplit<T>];
                    in_parts(cat<f32x8, f32x4>(st[2 * kk][cb], st[2 * kk + 1][cb]), e);
#pragma unroll
                    for (int j = 0; j < kSplit<T>; ++j) {
                        acc[0][cb] = mma(e[j], q0, acc[0][cb]);
                        acc[1][cb] = mma(e[j], q1, acc[1][cb]);
                    }
                }
            }
            f0 *= come_in * out_scale;
            f1 *= come_in * out_scale;
            // above the diagonal a weight of 0 is not enough: a score there may be infinite
            f32x8 sf[2];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = l16 >= 4 * g + r;
                sf[0][r] = in ? s00[r] * tw[0][r] : 0.f;
                sf[0][4 + r] = 0.f;
                sf[1][r] = s01[r] * tw[1][r];
                sf[1][4 + r] = in ? s11[r] * tw[0][r] : 0.f;
            }
            X8 sc[2][kSplit<T>];
            in_parts(sf[0], sc[0]);
            in_parts(sf[1], sc[1]);
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                acc[0][cb] *= f0;
                acc[1][cb] *= f1;
#pragma unroll
                for (int j = 0; j < kSplit<T>; ++j) {
                    acc[0][cb] = mma(vf[cb], sc[0][j], acc[0][cb]);
                    acc[1][cb] = mma(vf[cb], sc[1][j], acc[1][cb]);
                }
            }
        }
        // formed here, among the products above, and not behind the branch
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int j = 0; j < kParts<T>; ++j) asm volatile("" : "+v"(vw[cb][j]));
        if (drop) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) st[kb][cb] *= now;
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if (MODE != FULL && kb >= 2 && 32 * (kb / 2) >= keys) break;
            const X8 a = col_frag<KD>((const T*)nullptr, tk, kc ^ kb % 2 * 4 * (int)sizeof(T), 32 * (kb / 2));
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) st[kb][cb] = mma_weighted(a, vw[cb], st[kb][cb]);
        }
        // The next chunk's loads are waited for ahead of this one's stores, which need not be.
        if (!end) vm_wait<0>();
        if constexpr (!STATE) {
            const uint32_t gap = back ? (uint32_t)(C - cl) * os : 0;
            const Rows ob(op + gap, os, cl, owidth);
            op += back ? -(int64_t)C * os : (int64_t)C * os;
#pragma unroll
            for (int ib = 0; ib < 2; ++ib) {
                float x[4 * CB];
#pragma unroll
                for (int j = 0; j < 4 * CB; ++j) x[j] = acc[ib][j / 4][j % 4];
                store_run<OT, 4 * CB, MODE == RAGGED>(ob, ooff + ib * onext - gap,
                                                      16 * ib + l16 < cl ? vcols - oc : 0, x);
            }
        }
        block_sync();
    }

    const Rows fb(last && p.final ? (const void*)(p.final + block) : (const void*)p.decay, 0, 1,
                  last && p.final ? (uint32_t)(p.K * p.V) * 4 : 0);
    if (STATE || (last && final))
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                if (STATE) {
                    *(f32x4*)(mine + (cb * KB + kb) * 256) = st[kb][cb] * held;
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(st[kb][cb][r] * held), fb.r,
                                                              entry(kb, cb, r), 0, 0);
                }
            }
}

// Joins the span states of every sequence: slot s gets the state that enters span s.
// A thread takes 4 entries (one lane's part of a result tile).
__global__ __launch_bounds__(256) void linattn_join(LinPasses ps, int KD, int VT) {
    const LinPass& p = ps.p[blockIdx.z];
    touch_args(p);
    uint32_t id = blockIdx.x;
    const int vt = id % (uint32_t)p.vtiles;
    id /= (uint32_t)p.vtiles;
    const int h = id % (uint32_t)p.H, seq = id / (uint32_t)p.H;
    // The sequence's own bounds, not those of whom the first slot would be looked up for: with
    // cu out of order that may be another, whose spans from here on would leave the workspace.
    const int slot0 = p.cu ? (int)slot_base(p, seq) : seq * p.per;
    int64_t first, end;
    sequence_span(p.cu, seq, p.L, p.T, &first, &end);
    const int64_t spans = cdiv(end - first, p.span);
    const int e = blockIdx.y * 256 + threadIdx.x, lane = e & 63, tile = e >> 6;
    const int kb = tile % (KD / 16), vb = tile / (KD / 16);
    const int kr = 32 * (kb / 2) + 4 * (kb % 2) + 8 * (lane >> 4);
    const int vc = vt * VT + (VT == 64 ? 16 * vb + (lane & 15)
                                       : vb / 2 * 32 + dealt<2>(vb % 2, lane & 15));
    float* at = p.spans + (((int64_t)slot0 * p.H + h) * p.vtiles + vt) * (KD * VT) + e * 4;
    const int64_t step = (int64_t)p.H * p.vtiles * (KD * VT);
    constexpr int UN = 16;  // spans in flight
    f32x4 x[UN], s = {0.f, 0.f, 0.f, 0.f};
    auto load = [&](int64_t i) {
#pragma unroll
        for (int j = 0; j < UN; ++j)
            if (i + j + 1 < spans) x[j] = *(const f32x4*)(at + j * step);
    };
    load(0);
    if (p.init)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (kr + r < p.K && vc < p.V)
                s[r] = p.init[((int64_t)seq * p.H + h) * ((int64_t)p.K * p.V) +
                              (int64_t)(kr + r) * p.s_k + (int64_t)vc * p.s_v];
    const float decay = p.decay[h];
    Rate rate(power(decay, p.span));
    if (p.init_pow) s *= (float)power(decay, 1);
    for (int64_t i = 0; i < spans; i += UN, at += UN * step) {
        if (i) load(i);
#pragma unroll
        for (int j = 0; j < UN; ++j)
            if (i + j < spans) {
                *(f32x4*)(at + j * step) = s;
                if (i + j + 1 < spans) s = s * rate.next() + x[j];
            }
    }
}

// out[t][g] = the sum of part[t][g * R .. g * R + R - 1] (rows of D entries): gradients of
// keys and values that R heads share.  Tokens outside the sequences have no shares and stay as
// they are.
template <typename T>
__global__ __launch_bounds__(256) void linattn_heads_sum(const float* part, T* out, const int32_t* cu, int S,
                                                         int64_t items, int D, int G, int R, int64_t o_t,
                                                         int64_t o_g) {
    const int64_t first = cu ? cu[0] : 0, end = cu ? cu[S] : (int64_t)1 << 40;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        int64_t tg, t;
        const int d = (int)divide(i, D, &tg);
        const int g = (int)divide(tg, G, &t);
        if (t < first || t >= end) continue;
        const float* q = part + (tg * R) * D + d;
        float s = 0.f;
        for (int r = 0; r < R; ++r) s += q[(int64_t)r * D];
        out[t * o_t + g * o_g + d] = (T)s;
    }
}

// ---- host ----------------------------------------------------------------------------------

struct LinTiles {
    int KD, VT;
};
// K is padded to 64, 128 or 256, V cut into tiles of 128 columns, or 64 where there are no more
// (and for 256 float32 keys, whose tiles with 128 columns would not fit LDS twice).
LinTiles lin_tiles(int K, int V, int32_t dtype) {
    LinTiles t;
    t.KD = K <= 64 ? 64 : (K <= 128 ? 128 : 256);
    t.VT = V <= 64 || (t.KD == 256 && dtype == SSD_F32) ? 64 : 128;
    return t;
}

struct LinPlan {
    LinTiles t;
    int64_t span;
    int32_t slots, per, vtiles;
    size_t bytes;  // of the span states (0: whole sequences)
};

// Workgroups that are resident at once: two a CU, or one where the tiles take more than half of
// its LDS (lin_waves).
int64_t lin_resident(const LinTiles& t, int32_t dtype) {
    return 256 * lin_waves(t.KD, t.VT, (int)elem_size(dtype));
}

// Spans.  A workgroup takes 1.2 us a chunk by itself (64 x 128 bf16; 3.5 128 x 128 float32), and
// cutting a sequence takes two more launches and a state written and read for every span:
// enough spans that every resident workgroup has one, two in a packed batch, whose spans are
// uneven (in the mean of some draws of the lengths: 65536 tokens x 16 heads in 16 sequences, bf16,
// one for each 498 us, 1.5 475, two 459, three 476; gradients of 3001 x 8 heads of 96 and 72 in 7
// sequences, float32, 176, 160, 155 and 157.  32768 x 8 heads of 256, one workgroup a CU: 128
// workgroups 635 us, 256 368, 512 386).
// Short sequences stay whole: 2 x 256 tokens x 12 heads of 64 x 128, bf16, 19 us, cut 20; 2 x 512 30
// and 22; float32 2 x 128 23 and 26, 2 x 256 39 and 27.
LinPlan lin_plan(const ssd_linattn_dims& d, int K, int V, int passes = 1) {
    LinPlan pl;
    pl.t = lin_tiles(K, V, d.dtype);
    pl.vtiles = (int)cdiv(V, pl.t.VT);
    const int64_t S = d.nseq > 0 ? d.nseq : d.batch, T = (int64_t)d.batch * d.seqlen;
    const int64_t rows = (int64_t)d.nheads * pl.vtiles * passes;  // workgroups of a sequence in one span
    const int64_t fill = lin_resident(pl.t, d.dtype) * (d.nseq > 0 ? 2 : 1);
    // packed sequences are of any length: cut as if they were one
    const int64_t tokens = d.nseq > 0 ? T : d.seqlen, want = cdiv(fill, d.nseq > 0 ? rows : S * rows);
    pl.span = imax(cdiv(cdiv(tokens, want), C), 2) * C;
    const int64_t least = (d.dtype == SSD_BF16 ? 8 : 4) * C;
    if (pl.span >= tokens || T <= S * least) {
        pl.span = (int64_t)1 << 40;  // whole sequences
        pl.per = 1;
        pl.slots = (int)S;
        pl.bytes = 0;
        return pl;
    }
    pl.per = d.nseq > 0 ? 0 : (int)cdiv(d.seqlen, pl.span);
    pl.slots = (int)(d.nseq > 0 ? T / pl.span + S : S * pl.per);
    pl.bytes = up256((size_t)pl.slots * d.nheads * pl.vtiles * pl.t.KD * pl.t.VT * 4);
    return pl;
}

template <typename T, typename OT, int KD, int VT, int MODE>
void launch_tiles(const LinPasses& ps, int passes, const LinPlan& pl, hipStream_t s) {
    const LinPass& p = ps.p[0];
    const dim3 grid((unsigned)((int64_t)pl.slots * p.H * pl.vtiles), passes);
    if (pl.bytes) {
        linattn_kernel<T, OT, KD, VT, MODE, true><<<grid, 256, 0, s>>>(ps);
        const dim3 joins((unsigned)((int64_t)p.S * p.H * pl.vtiles), KD * VT / 1024, passes);
        linattn_join<<<joins, 256, 0, s>>>(ps, KD, VT);
    }
    linattn_kernel<T, OT, KD, VT, MODE, false><<<grid, 256, 0, s>>>(ps);
}
template <typename T, typename OT, int KD, int VT>
void launch_tiles(const LinPasses& ps, int passes, const LinPlan& pl, hipStream_t s) {
    constexpr int EPU = 16 / sizeof(T);
    bool full = true;  // the passes' K and V are the same two numbers
    for (int i = 0; i < passes; ++i) full = full && ps.p[i].K == KD;
    if (ps.p[0].K % EPU || ps.p[0].V % EPU) launch_tiles<T, OT, KD, VT, RAGGED>(ps, passes, pl, s);
    else if (!full) launch_tiles<T, OT, KD, VT, PADDED>(ps, passes, pl, s);
    else launch_tiles<T, OT, KD, VT, FULL>(ps, passes, pl, s);
}
// Passes of one plan, side by side in each launch: their span states lie behind each other in
// the workspace (pl.bytes each).
template <typename T, typename OT>
void launch_passes(LinPasses& ps, int passes, const LinPlan& pl, hipStream_t s) {
    for (int i = 0; i < passes; ++i) {
        LinPass& p = ps.p[i];
        p.span = pl.span;
        p.slots = pl.slots;
        p.per = pl.per;
        p.vtiles = pl.vtiles;
        p.together = pl.vtiles * (p.qdiv > p.kdiv ? p.qdiv : p.kdiv);
        p.spans = (float*)((char*)p.spans + i * pl.bytes);
    }
    if (pl.t.KD == 64) {
        if (pl.t.VT == 64) launch_tiles<T, OT, 64, 64>(ps, passes, pl, s);
        else launch_tiles<T, OT, 64, 128>(ps, passes, pl, s);
    } else if (pl.t.KD == 128) {
        if (pl.t.VT == 64) launch_tiles<T, OT, 128, 64>(ps, passes, pl, s);
        else launch_tiles<T, OT, 128, 128>(ps, passes, pl, s);
    } else if constexpr (sizeof(T) == 4) {  // two tiles of 256 x 128 would not fit LDS
        launch_tiles<T, OT, 256, 64>(ps, passes, pl, s);
    } else {
        if (pl.t.VT == 64) launch_tiles<T, OT, 256, 64>(ps, passes, pl, s);
        else launch_tiles<T, OT, 256, 128>(ps, passes, pl, s);
    }
}

int lin_check(const ssd_linattn_dims* d, const ssd_linattn_layout* l) {
    if (!d) return SSD_ERR_NULL_ARG;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->batch < 1 || d->seqlen < 0 || d->nheads < 1 || d->ngroups < 1 || d->nseq < 0 ||
        d->nheads % d->ngroups != 0 || d->keydim < 1 ||
        d->valuedim < 1 || d->reserved != 0 || d->seqlen > kMaxTokens / d->batch)
        return SSD_ERR_SHAPE;
    if (d->nseq > 0 && d->batch != 1) return SSD_ERR_SHAPE;
    if (d->keydim > SSD_LINATTN_MAX_DIM || d->valuedim > SSD_LINATTN_MAX_DIM) return SSD_ERR_UNSUPPORTED;
    if (!(d->scale == d->scale)) return SSD_ERR_SHAPE;
    // workgroups of a launch; a sequence has at least one span
    const int64_t S = d->nseq > 0 ? d->nseq : d->batch;
    if (S * d->nheads > (int64_t)1 << 21) return SSD_ERR_SHAPE;
    if (l)
        for (int64_t s : {l->q_token, l->q_head, l->k_token, l->k_group, l->v_token, l->v_group,
                          l->y_token, l->y_head, l->dy_token, l->dy_head, l->dq_token, l->dq_head,
                          l->dk_token, l->dk_group, l->dv_token, l->dv_group})
            if (s < 0 || s > kMaxStride) return SSD_ERR_SHAPE;
    return SSD_OK;
}

ssd_linattn_layout lin_layout(const ssd_linattn_dims& d, const ssd_linattn_layout* l) {
    if (l) return *l;
    const int64_t H = d.nheads, G = d.ngroups, K = d.keydim, V = d.valuedim;
    return ssd_linattn_layout{H * K, K, G * K, K, G * V, V, H * V, V, H * V, V, H * K, K, G * K, K, G * V, V};
}

LinPass lin_common(const ssd_linattn_dims& d, const float* decay, const int32_t* cu) {
    LinPass p = {};
    p.decay = decay;
    p.cu = cu;
    p.L = d.seqlen;
    p.T = (int64_t)d.batch * d.seqlen;
    p.S = d.nseq > 0 ? d.nseq : d.batch;
    p.H = d.nheads;
    p.qdiv = p.kdiv = p.vdiv = 1;
    return p;
}

size_t state_bytes(const ssd_linattn_dims& d) {
    return (size_t)(d.nseq > 0 ? d.nseq : d.batch) * d.nheads * d.keydim * d.valuedim * 4;
}

// The backward's plan.  The passes for dq and dk have the same sizes, and where K and V take the
// same tiles that for dv too: they share their launches, if their outputs have one type (where
// heads share keys and values, their shares of dk and dv are float32, and added up afterwards).
// 3001 tokens x 8 heads of 96 and 72, float32: one launch for each pass 203 us, one for two 172,
// one for all three 155.
struct LinBwdPlan {
    LinPlan qk, v;  // dq and dk, dv
    int together;   // passes of a launch: 1, 2 (dq and dk) or 3
    size_t spans, dk_shares, dv_shares;
};
LinBwdPlan lin_bwd_plan(const ssd_linattn_dims& d) {
    LinBwdPlan b;
    const int K = d.keydim, V = d.valuedim;
    const LinTiles x = lin_tiles(V, K, d.dtype), y = lin_tiles(K, V, d.dtype);
    const bool same = x.KD == y.KD && x.VT == y.VT && cdiv(K, x.VT) == cdiv(V, y.VT);
    b.together = d.nheads != d.ngroups && d.dtype != SSD_F32 ? 1 : (same ? 3 : 2);
    b.qk = lin_plan(d, V, K, b.together);
    b.v = b.together == 3 ? b.qk : lin_plan(d, K, V);
    b.spans = (size_t)imax(b.together * b.qk.bytes, b.v.bytes);
    const size_t rows = d.nheads == d.ngroups ? 0 : (size_t)d.batch * d.seqlen * d.nheads;
    b.dk_shares = up256(rows * K * 4);
    b.dv_shares = up256(rows * V * 4);
    return b;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_linattn_fwd_workspace_bytes(const ssd_linattn_dims* dims) {
    if (lin_check(dims, nullptr) != SSD_OK) return 0;
    return lin_plan(*dims, dims->keydim, dims->valuedim).bytes;
}

int ssd_linattn_fwd(const ssd_linattn_dims* dims, const ssd_linattn_layout* layout, const void* q,
                    const void* k, const void* v, const float* decay, const float* init_state,
                    const int32_t* cu_seqlens, int32_t reverse, void* y, float* final_state,
                    void* workspace, size_t workspace_bytes, void* stream) {
    int st = lin_check(dims, layout);
    if (st != SSD_OK) return st;
    const ssd_linattn_dims& d = *dims;
    if ((d.nseq > 0) != (cu_seqlens != nullptr)) return cu_seqlens ? SSD_ERR_SHAPE : SSD_ERR_NULL_ARG;
    const ssd_linattn_layout l = lin_layout(d, layout);
    const int64_t T = (int64_t)d.batch * d.seqlen;
    if (!decay || (T > 0 && (!q || !k || !v || !y))) return SSD_ERR_NULL_ARG;
    if (!rows_apart(T, l.y_token, d.nheads, l.y_head, d.valuedim)) return SSD_ERR_SHAPE;
    const size_t e = elem_size(d.dtype);
    if (!elem_aligned(q, e) || !elem_aligned(k, e) || !elem_aligned(v, e) || !elem_aligned(y, e) ||
        !elem_aligned(decay, 4) || !elem_aligned(init_state, 4) || !elem_aligned(final_state, 4) ||
        !elem_aligned(cu_seqlens, 4) || ((uintptr_t)workspace & 255))
        return SSD_ERR_ALIGN;
    if (init_state != final_state && overlaps(init_state, state_bytes(d), final_state, state_bytes(d)))
        return SSD_ERR_OVERLAP;
    const LinPlan pl = lin_plan(d, d.keydim, d.valuedim);
    if (pl.bytes && (!workspace || workspace_bytes < pl.bytes)) return SSD_ERR_WORKSPACE;
    if (cu_seqlens && check_cu_env(cu_seqlens, d.nseq, T, (hipStream_t)stream, &st)) return st;
    LinPasses ps = {};
    LinPass& p = ps.p[0] = lin_common(d, decay, cu_seqlens);
    p.q = q, p.q_t = l.q_token, p.q_h = l.q_head;
    p.k = k, p.k_t = l.k_token, p.k_h = l.k_group;
    p.v = v, p.v_t = l.v_token, p.v_h = l.v_group;
    p.o = y, p.o_t = l.y_token, p.o_h = l.y_head;
    p.kdiv = p.vdiv = d.nheads / d.ngroups;
    p.K = d.keydim, p.V = d.valuedim, p.s_k = d.valuedim, p.s_v = 1;
    p.init = init_state, p.final = final_state, p.spans = (float*)workspace;
    p.reverse = reverse != 0, p.init_pow = 1, p.final_pow = 0;
    p.in_scale = 1.f, p.out_scale = d.scale;
    if (d.dtype == SSD_BF16) launch_passes<bf16, bf16>(ps, 1, pl, (hipStream_t)stream);
    else launch_passes<float, float>(ps, 1, pl, (hipStream_t)stream);
    return launched();
}

size_t ssd_linattn_bwd_workspace_bytes(const ssd_linattn_dims* dims) {
    if (lin_check(dims, nullptr) != SSD_OK) return 0;
    const LinBwdPlan b = lin_bwd_plan(*dims);
    return b.spans + b.dk_shares + b.dv_shares;
}

int ssd_linattn_bwd(const ssd_linattn_dims* dims, const ssd_linattn_layout* layout, const void* q,
                    const void* k, const void* v, const float* decay, const float* init_state,
                    const int32_t* cu_seqlens, int32_t reverse, const void* dy,
                    const float* d_final, void* dq, void* dk, void* dv, float* dinit_state,
                    void* workspace, size_t workspace_bytes, void* stream) {
    int st = lin_check(dims, layout);
    if (st != SSD_OK) return st;
    const ssd_linattn_dims& d = *dims;
    if ((d.nseq > 0) != (cu_seqlens != nullptr)) return cu_seqlens ? SSD_ERR_SHAPE : SSD_ERR_NULL_ARG;
    const ssd_linattn_layout l = lin_layout(d, layout);
    const int64_t T = (int64_t)d.batch * d.seqlen;
    if (!decay || (T > 0 && (!q || !k || !v || !dy || !dq || !dk || !dv))) return SSD_ERR_NULL_ARG;
    if (!rows_apart(T, l.dq_token, d.nheads, l.dq_head, d.keydim) ||
        !rows_apart(T, l.dk_token, d.ngroups, l.dk_group, d.keydim) ||
        !rows_apart(T, l.dv_token, d.ngroups, l.dv_group, d.valuedim))
        return SSD_ERR_SHAPE;
    const size_t e = elem_size(d.dtype);
    for (const void* a : {q, k, v, dy, (const void*)dq, (const void*)dk, (const void*)dv})
        if (!elem_aligned(a, e)) return SSD_ERR_ALIGN;
    if (!elem_aligned(decay, 4) || !elem_aligned(init_state, 4) || !elem_aligned(d_final, 4) ||
        !elem_aligned(dinit_state, 4) || !elem_aligned(cu_seqlens, 4) || ((uintptr_t)workspace & 255))
        return SSD_ERR_ALIGN;
    if (d_final != dinit_state && overlaps(d_final, state_bytes(d), dinit_state, state_bytes(d)))
        return SSD_ERR_OVERLAP;
    if (overlaps(init_state, state_bytes(d), dinit_state, state_bytes(d))) return SSD_ERR_OVERLAP;
    const LinBwdPlan b = lin_bwd_plan(d);
    const size_t need = b.spans + b.dk_shares + b.dv_shares;
    if (need && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    if (cu_seqlens && check_cu_env(cu_seqlens, d.nseq, T, (hipStream_t)stream, &st)) return st;
    const hipStream_t s = (hipStream_t)stream;
    const int R = d.nheads / d.ngroups;
    float* const dk_shares = (float*)((char*)workspace + b.spans);
    float* const dv_shares = (float*)((char*)dk_shares + b.dk_shares);
    const bool half = d.dtype == SSD_BF16;

    LinPass q_ = lin_common(d, decay, cu_seqlens);
    q_.spans = (float*)workspace;
    LinPass k_ = q_, v_ = q_;
    q_.q = dy, q_.q_t = l.dy_token, q_.q_h = l.dy_head;
    q_.k = v, q_.k_t = l.v_token, q_.k_h = l.v_group, q_.kdiv = R;
    q_.v = k, q_.v_t = l.k_token, q_.v_h = l.k_group, q_.vdiv = R;
    q_.o = dq, q_.o_t = l.dq_token, q_.o_h = l.dq_head;
    q_.K = d.valuedim, q_.V = d.keydim, q_.s_k = 1, q_.s_v = d.valuedim;
    q_.init = init_state;
    q_.reverse = reverse != 0, q_.init_pow = 1, q_.final_pow = 0;
    q_.in_scale = 1.f, q_.out_scale = d.scale;

    k_.q = v, k_.q_t = l.v_token, k_.q_h = l.v_group, k_.qdiv = R;
    k_.k = dy, k_.k_t = l.dy_token, k_.k_h = l.dy_head;
    k_.v = q, k_.v_t = l.q_token, k_.v_h = l.q_head;
    k_.o = R == 1 ? dk : dk_shares;
    k_.o_t = R == 1 ? l.dk_token : (int64_t)d.nheads * d.keydim;
    k_.o_h = R == 1 ? l.dk_group : d.keydim;
    k_.K = d.valuedim, k_.V = d.keydim, k_.s_k = 1, k_.s_v = d.valuedim;

    v_.q = k, v_.q_t = l.k_token, v_.q_h = l.k_group, v_.qdiv = R;
    v_.k = q, v_.k_t = l.q_token, v_.k_h = l.q_head;
    v_.v = dy, v_.v_t = l.dy_token, v_.v_h = l.dy_head;
    v_.o = R == 1 ? dv : dv_shares;
    v_.o_t = R == 1 ? l.dv_token : (int64_t)d.nheads * d.valuedim;
    v_.o_h = R == 1 ? l.dv_group : d.valuedim;
    v_.K = d.keydim, v_.V = d.valuedim, v_.s_k = d.valuedim, v_.s_v = 1;
    v_.final = dinit_state;
    for (LinPass* p : {&k_, &v_}) {
        p->init = d_final;
        p->reverse = reverse == 0;
        p->init_pow = 0, p->final_pow = 1;
        p->in_scale = d.scale, p->out_scale = 1.f;
    }
    auto run = [&](const LinPass& p, bool share, const LinPlan& pl) {
        LinPasses ps = {{p}};
        if (!half) launch_passes<float, float>(ps, 1, pl, s);
        else if (share) launch_passes<bf16, float>(ps, 1, pl, s);
        else launch_passes<bf16, bf16>(ps, 1, pl, s);
    };
    auto join = [&](const float* shares, void* out, int64_t o_t, int64_t o_g, int D) {
        const int64_t items = T * d.ngroups * D;
        const dim3 grid((unsigned)(items < (1 << 28) ? cdiv(items, 256) : 1 << 20));
        if (half)
            linattn_heads_sum<bf16><<<grid, 256, 0, s>>>(shares, (bf16*)out, cu_seqlens, d.nseq, items, D,
                                                         d.ngroups, R, o_t, o_g);
        else
            linattn_heads_sum<float><<<grid, 256, 0, s>>>(shares, (float*)out, cu_seqlens, d.nseq, items, D,
                                                          d.ngroups, R, o_t, o_g);
    };
    // dinit may be d_final's buffer, which the pass for dk reads: dv's is behind it then
    const bool apart = dinit_state && dinit_state == d_final;
    const bool all = b.together == 3 && !apart;
    if (T > 0) {
        if (b.together > 1) {
            LinPasses ps = {{q_, k_, v_}};
            if (half) launch_passes<bf16, bf16>(ps, all ? 3 : 2, b.qk, s);
            else launch_passes<float, float>(ps, all ? 3 : 2, b.qk, s);
        } else {
            run(q_, false, b.qk);
            run(k_, true, b.qk);
        }
    }
    if ((T > 0 && !all) || (T == 0 && dinit_state)) run(v_, R > 1, b.v);
    if (T > 0 && R > 1) {
        join(dk_shares, dk, l.dk_token, l.dk_group, d.keydim);
        join(dv_shares, dv, l.dv_token, l.dv_group, d.valuedim);
    }
    return launched();
}

}  // extern "C"
