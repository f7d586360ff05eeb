// Linear attention with a decay (include/tm_layer.h): the memory of one
// matrix,  S_t = e^{g_t} S_{t-1} + k_t v_t^T,  y_t = scale S_t^T q_t,  and
// its gradients.
//
// Over a chunk of C tokens, with G the running sum of g in it (fp64) and S_0
// the state before it:
//   y_i = scale (sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j + e^{G_i} S_0^T q_i)
//   S_C = e^{G_C} S_0 + sum_j e^{G_C - G_j} k_j v_j^T
// No factor ever exceeds what the formula has (differences are taken before
// the exponential), and none is divided by, so a decay of -inf is a value
// like another: it is held as -1000, whose exponential is zero in any type.
//
// The gradients are three more runs of the same form.  With R_t the gradient
// of S_t (R goes over the tokens backwards) and y' = scale dy:
//   dq_i = sum_{j <= i} e^{G_i - G_j} (y'_i . v_j) k_j + e^{G_i} S_0 y'_i
//   dk_j = sum_{i >= j} e^{G_i - G_j} (v_j . y'_i) q_i + e^{G_C - G_j} R_C v_j
//   dv_j = sum_{i >= j} e^{G_i - G_j} (k_j . q_i) y'_i + e^{G_C - G_j} R_C^T k_j
//   R_0  = e^{G_C} R_C + sum_i e^{G_i} q_i y'_i^T
// so one kernel serves all: (query, key, value, state) is (q, k, v, S),
// (dy, v, k, S^T), (v, dy, q, R^T) or (k, q, dy, R).  The gradient of g_t is
// all that flows over the border before t, from tokens j < t to tokens i >= t:
//   dg_t = sum_{i >= t > j} X_ij + sum_{i >= t} fq_i + sum_{j < t} fk_j + through,
// the sums over the chunk, X_ij = e^{G_i - G_j} (q_i . k_j) (y'_i . v_j),
// fq_i = q_i . (the state's part of dq_i) what tokens before the chunk give
// to i, fk_j = k_j . (the state's part of dk_j) what j gives to tokens behind
// the chunk, and `through` what passes the chunk: <R_C, S_C> - sum fk at its
// end, <R_0, S_0> - sum fq at its start.  Taken as a running difference of
// what enters and leaves (q_i . dq_i - k_i . dk_i, the shorter formula), a
// decay's sum over n tokens would lose n^1.5 roundings.
#include <math.h>

#include <algorithm>

#include "../../include/tm_layer.h"
#include "tm_device.h"

namespace tmk {

constexpr double LOG2E = 1.4426950408889634074;
// Calls of up to as many tokens go token by token: us by tokens / by chunks
// (widths of 128, 64 and 512 heads' states; widths of 64, 8 states), bf16
// 2 tokens 7.3 / 12.3, 8 tokens 10.8 / 12.3, 28.4 / 22.3 and 8.4 / 7.9, 16
// tokens 17.5 / 12.2, 44.4 / 22.3 and 12.8 / 7.8; fp32 8 tokens 9.8 / 14.0,
// 27.3 / 27.0 and 7.5 / 7.4, 16 tokens 15.1 / 14.2, 43.6 / 27.0 and 11.3 / 7.4.
template <class T> constexpr int lin_few() { return sizeof(T) == 4 ? 8 : 5; }
// Tokens of a segment in the backward, at most. All gradients, segments of 128 /
// 256 / 512 tokens: 2 x 4096 tokens of 16 heads of 128 335 / 266 / 242 us (64:
// 484), 2 x 2048 in fp32 317 / 293 / 284, 4 x 2048 tokens of 16 heads of 64 147 /
// 124 / 124; but at 512 the gates' gradients, whose roundings grow with a segment,
// are 1.05e-6 of their size from 64 bits instead of 7.4e-7.
constexpr int LIN_BACK_SEG = 256;

// What a chunk run does (see the table of roles above).
enum { LIN_OUT, LIN_STATE, LIN_STATE_BACK, LIN_DQ, LIN_DK, LIN_DV };

struct LinArgs {
    const void *q, *k, *v, *z;           // z: rows that the far part is multiplied with (LIN_DQ: q, LIN_DK: k)
    long qb, qt, kb, kt, vb, vt, zb, zt; // elements between batch entries and between tokens
    int dk, dv;                          // width of queries and keys, width of values
    const float* ld;                     // log_decay
    const int* counts;
    const float* s_in;                   // [batch * key heads][s_seg][...]; null: zeros
    float* s_out;                        // null: not wanted
    long s_in_bh, s_in_seg, s_out_bh, s_out_seg;   // elements between heads' and between segments' states
    void* out;
    float* dot;                          // [slabs][batch * key heads][T]
    double* gsum;                        // [batch * key heads][nseg]: log2 of what a segment keeps
    float pair_scale, far_scale, state_scale;
    int per_token, B, T, Hk, G, nseg, L, slabs;
};

__device__ __forceinline__ int lin_tokens(const LinArgs& a, int b) {
    return a.counts ? min(max(a.counts[b], 0), a.T) : a.T;
}
// log2 of what a token keeps: -inf as -1000 (NaN stays NaN)
constexpr float LIN_DROPS = -1000.f;
__device__ __forceinline__ double lin_gate(float g) {
    return (double)(g < LIN_DROPS ? LIN_DROPS : g) * LOG2E;
}

// Rows in LDS, D elements long without gaps: the piece of 4 elements at column
// 4 u of row r stands at piece u ^ g(r), so that the reads of a wave are spread
// over the 32 banks: 16 rows at one column (8 bytes a lane for bf16, 16 lanes a
// cycle), 4 rows of 16 columns (transposing reads), for fp32 8 rows of 16
// bytes and 2 rows of 16 columns.  Padded rows had served one kind of read or
// the other (2300 of a chunk's 26000 cycles were conflicts).
template <class T> __device__ __forceinline__ int lin_turn(int r) {
    return sizeof(T) == 2 ? (r & 3) * 4 + (r >> 2 & 3) : (r & 7) ^ (r >> 1 & 4);
}

// 8 values of row `row` from column c on (a multiple of 32), in the order in
// which two stacked accumulator tiles hold 32 rows: lane group g has 4 g ..
// and 16 + 4 g ..
template <int D> __device__ __forceinline__ bf16x8 lin_split8(const bf16* m, int row, int c, int g) {
    typedef bf16 V4 __attribute__((ext_vector_type(4)));
    const bf16* p = m + row * D;
    const int t = lin_turn<bf16>(row), u = c / 4 + g;
    const V4 a = *reinterpret_cast<const V4*>(p + 4 * (u ^ t)), b = *reinterpret_cast<const V4*>(p + 4 * (u ^ t ^ 4));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int D> __device__ __forceinline__ f32x8 lin_split8(const float* m, int row, int c, int g) {
    const float* p = m + row * D;
    const int t = lin_turn<float>(row), u = c / 4 + g;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + 4 * (u ^ t)), b = *reinterpret_cast<const f32x4*>(p + 4 * (u ^ t ^ 4));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x8 lin_f32(f32x8 x) { return x; }
__device__ __forceinline__ f32x8 lin_f32(bf16x8 x) {   // a bf16's bits are an fp32's upper ones
    typedef unsigned U4 __attribute__((ext_vector_type(4)));
    const U4 u = __builtin_bit_cast(U4, x);
    f32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = __builtin_bit_cast(float, u[i] << 16);
        r[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xffff0000u);
    }
    return r;
}

// fp32 values as operands: one for fp32, N of 8 bits each for bf16.  A pair's
// weight and the state before a chunk take two: 16 bits of each, so that what
// an output is off by is its own rounding to 8 (with weights of 8 bits outputs
// were 0.0023 of their size from 64 bits, 0.0017 of it their own; the second
// operand costs 1 to 3% of a call, 8% at widths of 64).
template <class T, int N> struct Parts {
    typename Frag<T>::T p[N];
    __device__ __forceinline__ void set(f32x8 x) {
        if constexpr (sizeof(T) == 4) {
            p[0] = x;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                p[i] = __builtin_convertvector(x, bf16x8);
                if (i + 1 < N) x -= lin_f32(p[i]);
            }
        }
    }
};
template <class T> constexpr int lin_parts(int n) { return sizeof(T) == 4 ? 1 : n; }

// Tokens of a chunk: 64, for fp32 32 (with its four times slower matrix
// instructions the pairs of a chunk cost more than the state it saves).
template <class T> constexpr int lin_chunk() { return sizeof(T) == 4 ? 32 : 64; }

// A run's LDS.  STATE: one that forms states alone, without queries and pairs.
template <class T, int DK, int CW, bool STATE> struct LinLds {
    static constexpr int C = lin_chunk<T>(), VD = 64 * CW, PP = C + 16 / sizeof(T), PARTS = lin_parts<T>(2);
    // tokens whose decays are summed at a time (half as many where two workgroups would not fit a compute unit)
    static constexpr int GATES = sizeof(T) == 2 && DK == 192 ? 256 : 512;
    static constexpr size_t q = 0, k = q + (STATE ? 0 : sizeof(T) * C * DK), v = k + sizeof(T) * C * DK,
                            p = v + sizeof(T) * C * VD, g = p + (STATE ? 0 : sizeof(T) * C * PP * PARTS),
                            head = g + 8 * GATES, tail = head + 4 * GATES, dot = tail + 4 * GATES,
                            bad = dot + 4 * 4 * 64, bytes = bad + 16;
};

// Whether 16 bytes hold a non-finite value: an exponent of ones.
__device__ __forceinline__ bool lin_lost(f32x4 x) {
    const f32x4 zero = x * 0.f;   // NaN where x is not finite
    return !((zero[0] + zero[1]) + (zero[2] + zero[3]) == 0.f);
}
__device__ __forceinline__ bool lin_lost(bf16x8 x) {
    typedef unsigned short H8 __attribute__((ext_vector_type(8)));
    const H8 h = __builtin_bit_cast(H8, x) & (unsigned short)0x7fff;
    typedef unsigned short H4 __attribute__((ext_vector_type(4)));
    typedef unsigned short H2 __attribute__((ext_vector_type(2)));
    const H4 a = __builtin_elementwise_max(__builtin_shufflevector(h, h, 0, 1, 2, 3), __builtin_shufflevector(h, h, 4, 5, 6, 7));
    const H2 b = __builtin_elementwise_max(__builtin_shufflevector(a, a, 0, 1), __builtin_shufflevector(a, a, 2, 3));
    return b[0] >= 0x7f80 || b[1] >= 0x7f80;
}

// A tile [C][D] of a token array on its way from memory to LDS, 16 bytes at a
// time.  Rows behind the last and columns behind the array's are read as ones
// that are there and taken as zeros when they are put down.  x: the tile's
// first row; step: elements between rows (64 rows are less than 2^31 bytes
// apart: an offset is 32 bits beside an address of the whole workgroup).
template <class T, int D, int C> struct LinTile {
    // rows of PER by N cover C; where they are more, or 256 threads are no whole
    // rows (D 192), some rows are read and put down twice
    static constexpr int VE = 16 / sizeof(T), UNITS = D / VE, PER = 256 / UNITS, N = (C + PER - 1) / PER;
    static constexpr bool WHOLE = 256 % UNITS == 0 && C % PER == 0;
    typedef T Vec __attribute__((ext_vector_type(VE)));
    Vec v[N];
    __device__ __forceinline__ void load(const T* x, unsigned step, int rows, int c0, int cols) {
        const unsigned u = threadIdx.x % UNITS, c = c0 + u * VE < (unsigned)cols ? c0 + u * VE : 0u, r0 = threadIdx.x / UNITS;
        const char* at = reinterpret_cast<const char*>(x);
        if (WHOLE && rows == C) {
            const unsigned off = (r0 * step + c) * (unsigned)sizeof(T);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = *reinterpret_cast<const Vec*>(at + (unsigned long)(i * PER) * step * sizeof(T) + off);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = *reinterpret_cast<const Vec*>(at + (min(r0 + i * PER, rows - 1u) * step + c) * (unsigned)sizeof(T));
        }
    }
    // TURN: pieces permuted (lin_turn).  bad: the first row with a non-finite
    // element, which is taken as zero
    template <bool CHECK, bool TURN>
    __device__ __forceinline__ void store(T* to, int row, int rows, int c0, int cols, int* bad) {
        const int u = threadIdx.x % UNITS, r0 = threadIdx.x / UNITS;
        if (rows < C || c0 + D > cols) {
            const bool there = c0 + u * VE < cols;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = keep_if(v[i], there && r0 + i * PER < rows);
        }
        if constexpr (CHECK) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < N; ++i) any |= lin_lost(v[i]);
            if (any)
#pragma unroll 1
                for (int i = 0; i < N; ++i) {
                    bool here = false;
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j == i && lin_lost(v[j])) {
                            here = true;
#pragma unroll
                            for (int e = 0; e < VE; ++e)
                                if (!__builtin_isfinite((float)v[j][e])) v[j][e] = (T)0.f;
                        }
                    if (here) atomicMin(bad, r0 + i * PER);
                }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (WHOLE || r0 + i * PER < C) {
                const int r = r0 + i * PER;
                if constexpr (!TURN) {
                    *reinterpret_cast<Vec*>(to + r * row + u * VE) = v[i];
                } else if constexpr (VE == 4) {
                    *reinterpret_cast<Vec*>(to + r * row + 4 * (u ^ lin_turn<T>(r))) = v[i];
                } else {
                    typedef T V4 __attribute__((ext_vector_type(4)));
                    *reinterpret_cast<V4*>(to + r * row + 4 * (2 * u ^ lin_turn<T>(r))) = __builtin_shufflevector(v[i], v[i], 0, 1, 2, 3);
                    *reinterpret_cast<V4*>(to + r * row + 4 * ((2 * u + 1) ^ lin_turn<T>(r))) = __builtin_shufflevector(v[i], v[i], 4, 5, 6, 7);
                }
            }
    }
};

// 8 rows from r0 on (a multiple of 32; lane group g has rows r0 + 8 g ..) of
// column c + (lane % 16), c a multiple of 16.  l: the lane.
template <int D> __device__ __forceinline__ bf16x8 lin_column8(const bf16* m, int r0, int c, int l) {
    typedef short S4 __attribute__((ext_vector_type(4)));
    typedef short S8 __attribute__((ext_vector_type(8)));
    const int i = l & 15;
    // the transposing read: a lane names 4 columns of a row, and gets 4 rows of its column
    const int r = 8 * (l >> 4) + (i >> 2), u = c / 4 + (i & 3);
    const bf16* p = m + (r0 + r) * D;
    const bf16* a = p + 4 * (u ^ lin_turn<bf16>(r));
    const bf16* b = p + 4 * D + 4 * (u ^ lin_turn<bf16>(r + 4));
    const S4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) S4*)(a));
    const S4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) S4*)(b));
    return __builtin_bit_cast(bf16x8, (S8)__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int D> __device__ __forceinline__ f32x8 lin_column8(const float* m, int r0, int c, int l) {
    const int r = 8 * (l >> 4), col = c + (l & 15);
    f32x8 x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = m[(r0 + r + e) * D + 4 * ((col / 4) ^ lin_turn<float>(r + e)) + col % 4];
    return x;
}

// The lane.  ANEW: what is computed from it is not kept in registers from one
// part of a chunk's work (or from one chunk) to the next.  The large kernels
// have none left for it (spilling, widths of 128 took 1.4 times as long); the
// others are better off with the addresses kept (widths of 64: 57 us against
// 62 for 1024 tokens of 256 heads).
template <bool ANEW> __device__ __forceinline__ int lin_lane() {
    int l = threadIdx.x & 63;
    if constexpr (ANEW) asm volatile("" : "+v"(l));
    return l;
}

// One workgroup of 4 waves takes one key head of one entry, one segment of its
// tokens, and 64 CW columns of the values (16 CW a wave), whose slice of the
// state its waves hold in accumulators.  The next chunk's rows are read while
// a chunk is computed.
template <class T, int DK, int CW, int KIND> __device__ __forceinline__ void lin_body(const LinArgs& a, int block) {
    constexpr bool STATE = KIND == LIN_STATE || KIND == LIN_STATE_BACK;
    constexpr bool REV = KIND == LIN_STATE_BACK || KIND == LIN_DK || KIND == LIN_DV;
    constexpr bool SUM = REV;   // the group's heads are summed (else each has an output of its own)
    constexpr bool DOT = KIND == LIN_DQ || KIND == LIN_DK;
    constexpr int C = lin_chunk<T>(), NT = C / 16, NS = DK / 32, NM = DK / 16, KS = C / 32;
    // the state as an operand keeps 16 bits, 24 where its products enter the gradients of the decays
    constexpr int SP = lin_parts<T>(DOT ? 3 : 2), VP3 = lin_parts<T>(3);   // what is added to the state: 24
    typedef typename Frag<T>::T F;
    typedef LinLds<T, DK, CW, STATE> S_;
    constexpr int VD = S_::VD, PP = S_::PP, BATCH = S_::GATES / C;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    T* qs = reinterpret_cast<T*>(lds + S_::q);
    T* ks = reinterpret_cast<T*>(lds + S_::k);
    T* vs = reinterpret_cast<T*>(lds + S_::v);
    T* ps = reinterpret_cast<T*>(lds + S_::p);
    double* gs = reinterpret_cast<double*>(lds + S_::g);
    float* head = reinterpret_cast<float*>(lds + S_::head);
    float* tail = reinterpret_cast<float*>(lds + S_::tail);
    float* dots = reinterpret_cast<float*>(lds + S_::dot);
    int* bads = reinterpret_cast<int*>(lds + S_::bad);

    const int slab = block % a.slabs, rest = block / a.slabs;
    const int seg = rest % a.nseg, bh = rest / a.nseg, b = bh / a.Hk, h = bh % a.Hk;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
    const int col0 = slab * 64 * CW, wcol = 16 * CW * wave;   // the workgroup's first column, the wave's in it
    const int n = lin_tokens(a, b), first = seg * a.L, last = (int)min((long)n, (long)first + a.L);
    const int chunks = last > first ? (last - first + C - 1) / C : 0, steps = chunks * a.G;

    const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb;
    const T* k = reinterpret_cast<const T*>(a.k) + b * a.kb;
    const T* v = reinterpret_cast<const T*>(a.v) + b * a.vb;
    const T* z = reinterpret_cast<const T*>(a.z) + b * a.zb;

    f32x4 S[NM][CW];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int w = 0; w < CW; ++w) S[m][w] = f32x4{0.f, 0.f, 0.f, 0.f};
    // a row of the state is a row of the array, or (where queries and keys are the values) a column
    constexpr bool TURNED = KIND == LIN_DQ || KIND == LIN_DK;
    auto cell = [&](int i, int c) { return TURNED ? c * a.dk + i : i * a.dv + c; };
    if (!STATE && a.s_in) {
        const float* s = a.s_in + bh * a.s_in_bh + seg * a.s_in_seg;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int w = 0; w < CW; ++w) {
                const int i = 16 * m + 4 * lg, c = col0 + wcol + 16 * w + l16;   // dk: a multiple of 8
                const bool there = i < a.dk && c < a.dv;
                if constexpr (TURNED) {
                    S[m][w] = *reinterpret_cast<const f32x4*>(s + (there ? cell(i, c) : 0));
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[m][w][r] = s[there ? cell(i + r, c) : 0];
                }
            }
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int w = 0; w < CW; ++w)
                S[m][w] = keep_if(S[m][w], 16 * m + 4 * lg < a.dk && col0 + wcol + 16 * w + l16 < a.dv);
    }
    double kept = 0.0;

    LinTile<T, DK, C> qv, kv;
    LinTile<T, 64 * CW, C> vv;
    auto start = [&](int ci) { return first + (REV ? chunks - 1 - ci : ci) * C; };
    auto fetch = [&](int ci, int g) {
        const int t0 = start(ci), many = h * a.G + g, rows = min(C, last - t0);
        if constexpr (!STATE)
            if (!SUM || g == 0) qv.load(q + t0 * a.qt + (long)(SUM ? h : many) * a.dk, (unsigned)a.qt, rows, 0, a.dk);
        if (SUM || g == 0) {
            const int kh = SUM ? many : h;
            kv.load(k + t0 * a.kt + (long)kh * a.dk, (unsigned)a.kt, rows, 0, a.dk);
            vv.load(v + t0 * a.vt + (long)kh * a.dv, (unsigned)a.vt, rows, col0, a.dv);
        }
    };
    f32x4 O[NT][CW];
    float far_dot[NT];
    auto put_dots = [&](int t0) {   // over the workgroup's columns
        const int i = threadIdx.x;
        if (i < min(C, last - t0))
            a.dot[((long)slab * a.B * a.Hk + bh) * a.T + t0 + i] = (dots[i] + dots[64 + i]) + (dots[128 + i] + dots[192 + i]);
    };
    // the state is there: seen as still under way, its first use in every chunk would wait for the rows read ahead
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    if (steps) fetch(0, 0);
    if (KIND == LIN_OUT && threadIdx.x < 2) bads[threadIdx.x] = C;
    int ci = 0, g = 0;
#pragma unroll 1
    for (int st = 0; st < steps; ++st) {
        const int t0 = start(ci), many = h * a.G + g, gate0 = ci % BATCH * C, rows = min(C, last - t0);
        int* bad = bads + (ci & 1);
        __syncthreads();   // the step before is done with what stands in LDS
        if constexpr (!STATE)
            if (!SUM || g == 0) qv.template store<false, true>(qs, DK, rows, 0, a.dk, nullptr);
        if (SUM || g == 0) {
            kv.template store<false, true>(ks, DK, rows, 0, a.dk, nullptr);
            vv.template store<KIND == LIN_OUT, true>(vs, VD, rows, col0, a.dv, bad);
        }
        if constexpr (DOT)
            if (g == 0 && ci > 0) put_dots(start(ci - 1));
        const int next_g = g + 1 < a.G ? g + 1 : 0, next_ci = next_g ? ci : ci + 1;
        if (st + 1 < steps) fetch(next_ci, next_g);
        if (g == 0 && gate0 == 0) {   // the decays of the next 512 tokens, C lanes a chunk
#pragma unroll
            for (int it = 0; it < S_::GATES / 256; ++it) {
                const int slot = it * 256 + threadIdx.x, c = ci + slot / C, i = slot % C;
                double x = 0.0;
                if (c < chunks && start(c) + i < last)
                    x = lin_gate(a.ld[a.per_token ? ((long)b * a.T + start(c) + i) * a.Hk + h : h]);
#pragma unroll
                for (int m = 1; m < C; m <<= 1) {
                    const double o = __shfl_up(x, m, C);
                    if (i >= m) x += o;
                }
                const double end = __shfl(x, C - 1, C);
                gs[slot] = x;
                const float before = __builtin_amdgcn_exp2f((float)x), after = __builtin_amdgcn_exp2f((float)(end - x));
                head[slot] = (REV ? after : before) * a.far_scale;
                tail[slot] = (REV ? before : after) * a.state_scale;
            }
        }
        __syncthreads();
        if constexpr (!STATE) {
            if (KIND == LIN_OUT && g == 0 && threadIdx.x == 0) bads[(ci + 1) & 1] = C;
            // the pairs' weights: tiles of 16 queries by 16 keys, those that a step of 32 keys reads
#pragma unroll
            for (int pi = 0; pi < (NT == 4 ? 3 : 1); ++pi) {
                const int l = lin_lane<DK * CW >= 192>(), l16 = l & 15, lg = l >> 4;
                const int p = wave + 4 * pi;
                int qt = p < 4 ? p >> 1 : 2 + ((p - 4) >> 2), kt = p < 4 ? p & 1 : (p - 4) & 3;
                if (REV) {
                    qt = NT - 1 - qt;
                    kt = NT - 1 - kt;
                }
                const int i = 16 * qt + l16, j0 = 16 * kt + 4 * lg;
                f32x4 w = f32x4{0.f, 0.f, 0.f, 0.f}, by;
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    mma(w, lin_split8<DK>(ks, 16 * kt + l16, 32 * s, lg), lin_split8<DK>(qs, i, 32 * s, lg));
                const double gi = gs[gate0 + i];
                const double* gj = gs + gate0 + j0;
#pragma unroll
                for (int r = 0; r < 4; ++r)   // pairs of the other order: their weight is not used
                    by[r] = __builtin_amdgcn_exp2f((float)(REV ? gj[r] - gi : gi - gj[r])) * a.pair_scale;
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r] = (REV ? j0 + r >= i : j0 + r <= i) ? w[r] * by[r] : 0.f;
                typedef T V4 __attribute__((ext_vector_type(4)));
                V4 o;
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] = (T)w[r];
                *reinterpret_cast<V4*>(ps + i * PP + 16 * kt + 4 * lg) = o;
                if constexpr (S_::PARTS == 2) {   // what 8 bits leave of a weight, 8 bits of it
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[r] = (T)(w[r] - (float)o[r]);
                    *reinterpret_cast<V4*>(ps + C * PP + i * PP + 16 * kt + 4 * lg) = o;
                }
            }
            // the far part, out of the state before the chunk
            if (!SUM || g == 0) {
                const int l = lin_lane<DK * CW >= 192>(), l16 = l & 15, lg = l >> 4;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int w = 0; w < CW; ++w) O[i][w] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    Parts<T, SP> sp[CW];
#pragma unroll
                    for (int w = 0; w < CW; ++w)
                        sp[w].set(__builtin_shufflevector(S[2 * s][w], S[2 * s + 1][w], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const F qf = lin_split8<DK>(qs, 16 * i + l16, 32 * s, lg);
#pragma unroll
                        for (int p = SP - 1; p >= 0; --p)
#pragma unroll
                            for (int w = 0; w < CW; ++w) {
                                if constexpr (sizeof(T) == 4) {   // sums of 32, then of those
                                    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
                                    mma(sum, sp[w].p[p], qf);
                                    O[i][w] += sum;
                                } else {
                                    mma(O[i][w], sp[w].p[p], qf);
                                }
                            }
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float by = head[gate0 + 16 * i + l16];
                    if (DOT && g == 0) far_dot[i] = 0.f;
#pragma unroll
                    for (int w = 0; w < CW; ++w) {
                        O[i][w] *= by;
                        if constexpr (DOT) {
                            const int t = t0 + 16 * i + l16, c = col0 + wcol + 16 * w + 4 * lg;
                            if (t < last && c < a.dv) {
                                typedef T V4 __attribute__((ext_vector_type(4)));
                                const V4 zr = *reinterpret_cast<const V4*>(z + (long)t * a.zt + (long)(SUM ? h : many) * a.dv + c);
#pragma unroll
                                for (int r = 0; r < 4; ++r) far_dot[i] += O[i][w][r] * (float)zr[r];
                            }
                        }
                    }
                }
            }
            __syncthreads();
            // the chunk's own
            const int l = lin_lane<DK * CW >= 192>(), l16 = l & 15, lg = l >> 4;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                F vf[CW];
#pragma unroll
                for (int w = 0; w < CW; ++w) vf[w] = lin_column8<VD>(vs, 32 * s, wcol + 16 * w, l);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (REV ? s < i / 2 : s > i / 2) continue;
                    if constexpr (S_::PARTS == 2) {
                        const F rest = ld8(ps + C * PP + (16 * i + l16) * PP + 32 * s + 8 * lg);
#pragma unroll
                        for (int w = 0; w < CW; ++w) mma(O[i][w], vf[w], rest);
                    }
                    const F pf = ld8(ps + (16 * i + l16) * PP + 32 * s + 8 * lg);
#pragma unroll
                    for (int w = 0; w < CW; ++w) mma(O[i][w], vf[w], pf);
                }
            }
            if (!SUM || g == a.G - 1) {
                const int heads = SUM ? a.Hk : a.Hk * a.G, oh = SUM ? h : many;
                const unsigned step = (unsigned)(heads * a.dv);
                char* to = reinterpret_cast<char*>(reinterpret_cast<T*>(a.out) + ((long)b * a.T + t0) * step + (long)oh * a.dv + col0);
                const unsigned off = (l16 * step + wcol + 4 * lg) * (unsigned)sizeof(T);
                typedef T V4 __attribute__((ext_vector_type(4)));
                auto put = [&](bool all) {
                    // a non-finite value is zero in vs: its products with the weights of earlier tokens, which are
                    // zero, would not be
                    const int from = KIND == LIN_OUT && !all ? *bad : C;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const bool lost = KIND == LIN_OUT && !all && 16 * i + l16 >= from;
#pragma unroll
                        for (int w = 0; w < CW; ++w)
                            if (all || (16 * i + l16 < rows && col0 + wcol + 16 * w + 4 * lg < a.dv)) {
                                V4 o;
#pragma unroll
                                for (int r = 0; r < 4; ++r) o[r] = (T)(lost ? __builtin_nanf("") : O[i][w][r]);
                                *reinterpret_cast<V4*>(to + (unsigned long)(16 * i) * step * sizeof(T) + 16 * w * sizeof(T) + off) = o;
                            }
                    }
                };
                if (rows == C && col0 + 64 * CW <= a.dv && (KIND != LIN_OUT || *bad == C)) put(true);
                else put(false);
                if constexpr (DOT)
                    if (g == a.G - 1)
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            float d = far_dot[i];
                            d += __shfl_xor(d, 16, 64);
                            d += __shfl_xor(d, 32, 64);
                            if (lg == 0) dots[wave * 64 + 16 * i + l16] = d;
                        }
            }
        }
        // the state behind the chunk: the values take the decays (and are split), the keys go in as they are
        if (SUM || g == a.G - 1) {
            const int l = lin_lane<DK * CW >= 192>(), lg = l >> 4;
            float keep = 1.f;
            if (!SUM || g == 0) {
                const double end = gs[gate0 + C - 1];
                keep = __builtin_amdgcn_exp2f((float)end);
                kept += end;
            }
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int w = 0; w < CW; ++w) S[m][w] *= keep;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    Parts<T, VP3> vp[CW];
                    const f32x8 by = ld8(tail + gate0 + 32 * s + 8 * lg);
#pragma unroll
                    for (int w = 0; w < CW; ++w)
                        vp[w].set(lin_f32(lin_column8<VD>(vs, 32 * s, wcol + 16 * w, l)) * by);
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        const F kf = lin_column8<DK>(ks, 32 * s, 16 * m, l);
#pragma unroll
                        for (int p = VP3 - 1; p >= 0; --p)
#pragma unroll
                            for (int w = 0; w < CW; ++w) mma(S[m][w], kf, vp[w].p[p]);
                    }
                }
            } else {   // a chunk's sum is formed by itself: the state takes one rounding a chunk, not one a product of 4 tokens
                static_assert(sizeof(T) == 2 || KS == 1, "a chunk of 32 tokens");
                const f32x8 by = ld8(tail + gate0 + 8 * lg);
                F vf[CW];
#pragma unroll
                for (int w = 0; w < CW; ++w) vf[w] = lin_column8<VD>(vs, 0, wcol + 16 * w, l) * by;
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const F kf = lin_column8<DK>(ks, 0, 16 * m, l);
#pragma unroll
                    for (int w = 0; w < CW; ++w) {
                        f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
                        mma(sum, kf, vf[w]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) S[m][w][r] = fmaf(keep, S[m][w][r], sum[r]);
                    }
                }
            }
            if (KIND == LIN_OUT && *bad < C) {
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int w = 0; w < CW; ++w) S[m][w] += __builtin_nanf("");
            }
        }
        g = next_g;
        ci = next_ci;
    }
    if constexpr (DOT)
        if (chunks) {
            __syncthreads();
            put_dots(start(chunks - 1));
        }
    if (!TURNED && a.s_out) {
        float* s = a.s_out + bh * a.s_out_bh + seg * a.s_out_seg;
#pragma unroll
        for (int w = 0; w < CW; ++w) {
            const int c = col0 + wcol + 16 * w + l16;
            if (c < a.dv)
#pragma unroll
                for (int m = 0; m < NM; ++m)
                    if (16 * m + 4 * lg < a.dk)
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[cell(16 * m + 4 * lg + r, c)] = S[m][w][r];
        }
    }
    if (STATE && a.gsum && slab == 0 && threadIdx.x == 0) a.gsum[(long)bh * a.nseg + seg] = kept;
}

template <class T, int DK, int CW, int KIND> __global__ __launch_bounds__(256, 2) void lin_kernel(LinArgs a) {
    lin_body<T, DK, CW, KIND>(a, blockIdx.x);
}
// The backward's runs that do not need each other, in one launch each: what
// the segments add to the state and to its gradient, then the three gradients.
struct LinMany {
    LinArgs a[3];
    int blocks[3];
};
template <class T, int DK, int CW> __global__ __launch_bounds__(256, 2) void lin_states_kernel(LinMany m) {
    const int i = blockIdx.x;
    if (i < m.blocks[0]) lin_body<T, DK, CW, LIN_STATE_BACK>(m.a[0], i);
    else lin_body<T, DK, CW, LIN_STATE>(m.a[1], i - m.blocks[0]);
}
template <class T, int DK, int CW> __global__ __launch_bounds__(256, 2) void lin_gradients_kernel(LinMany m) {
    const int i = blockIdx.x;
    if (i < m.blocks[0]) lin_body<T, DK, CW, LIN_DK>(m.a[0], i);
    else if (i < m.blocks[0] + m.blocks[1]) lin_body<T, DK, CW, LIN_DQ>(m.a[1], i - m.blocks[0]);
    else lin_body<T, DK, CW, LIN_DV>(m.a[2], i - m.blocks[0] - m.blocks[1]);
}

// Single tokens and short drafts, token by token: 32 columns of a head's
// state a workgroup, in its registers (4 columns and DK / 32 rows a thread).
// Bound by reading and writing the state once; the tokens' rows are brought
// into LDS together, and the waves' shares of the outputs meet there once for
// all of them, so a draft pays the way to memory and the barriers once.
template <class T> struct LinToken {   // LDS bytes of one token
    static constexpr size_t bytes(int G, int dk) { return (size_t)(G + 1) * dk * sizeof(T) + 32 * 4 + 16 + (size_t)G * 512; }
};
template <class T, int DK>
__global__ __launch_bounds__(256) void lin_token_kernel(LinArgs a, int batch) {   // batch: tokens in LDS at a time
    constexpr int R = DK / 32, VE = 16 / sizeof(T);
    typedef T Vec __attribute__((ext_vector_type(VE)));
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int rows = (a.G + 1) * a.dk;                                   // queries, then the key
    float* red = reinterpret_cast<float*>(lds);                          // [batch][G][4 waves][32]
    float* vs = red + batch * a.G * 128;                                 // [batch][32]
    float* keeps = vs + batch * 32;                                      // [batch], in 16 bytes each
    T* qk = reinterpret_cast<T*>(keeps + 4 * batch);                     // [batch][rows]
    const int slab = blockIdx.x % a.slabs, bh = blockIdx.x / a.slabs, b = bh / a.Hk, h = bh % a.Hk;
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3, wave = threadIdx.x >> 6, c0 = slab * 32, c = c0 + 4 * cg;
    const bool on = c < a.dv;
    const int n = lin_tokens(a, b);
    f32x4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int row = rg + 32 * i;
        if (a.s_in && on && row < a.dk)
            S[i] = *reinterpret_cast<const f32x4*>(a.s_in + bh * a.s_in_bh + (long)row * a.dv + c);
    }
    for (int t0 = 0; t0 < n; t0 += batch) {
        const int m = min(batch, n - t0), units = a.dk / VE;
        if (t0 > 0) __syncthreads();
        const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb + t0 * a.qt + (long)h * a.G * a.dk;
        const T* k = reinterpret_cast<const T*>(a.k) + b * a.kb + t0 * a.kt + (long)h * a.dk;
        const T* v = reinterpret_cast<const T*>(a.v) + b * a.vb + t0 * a.vt + (long)h * a.dv + c0;
        const int per = (a.G + 1) * units;
        for (int i = threadIdx.x; i < m * per; i += 256) {
            const int t = i / per, u = i % per;
            const T* x = u < a.G * units ? q + t * a.qt + u * VE : k + t * a.kt + (u - a.G * units) * VE;
            *reinterpret_cast<Vec*>(qk + t * rows + u * VE) = *reinterpret_cast<const Vec*>(x);
        }
        for (int i = threadIdx.x; i < m * 32; i += 256) {
            const int t = i >> 5, e = i & 31;
            vs[i] = c0 + e < a.dv ? (float)v[t * a.vt + e] : 0.f;
        }
        for (int t = threadIdx.x; t < m; t += 256)
            keeps[4 * t] = expf(a.ld[a.per_token ? ((long)b * a.T + t0 + t) * a.Hk + h : h]);
        __syncthreads();
        for (int t = 0; t < m; ++t) {
            const T* qr = qk + t * rows;
            const T* kr = qr + a.G * a.dk;
            const f32x4 vv = *reinterpret_cast<const f32x4*>(vs + t * 32 + 4 * cg);
            const float keep = keeps[4 * t];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int row = rg + 32 * i;
                const float kv = row < a.dk ? (float)kr[row] : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][e] = fmaf(keep, S[i][e], kv * vv[e]);
            }
            for (int g = 0; g < a.G; ++g) {
                f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int row = rg + 32 * i;
                    const float qv = row < a.dk ? (float)qr[g * a.dk + row] : 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = row < a.dk ? fmaf(qv, S[i][e], y[e]) : y[e];
                }
#pragma unroll
                for (int s = 8; s < 64; s <<= 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] += __shfl_xor(y[e], s, 64);
                if ((threadIdx.x & 63) < 8) *reinterpret_cast<f32x4*>(red + ((t * a.G + g) * 4 + wave) * 32 + 4 * cg) = y;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < m * a.G * 32; i += 256) {
            const int tg = i >> 5, col = i & 31, t = t0 + tg / a.G, g = tg % a.G;
            const float* p = red + tg * 128 + col;
            const float y = ((p[0] + p[32]) + (p[64] + p[96])) * a.far_scale;
            if (c0 + col < a.dv)
                reinterpret_cast<T*>(a.out)[(((long)b * a.T + t) * a.Hk * a.G + (long)h * a.G + g) * a.dv + c0 + col] = (T)y;
        }
    }
    if (a.s_out && on)
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = rg + 32 * i;
            if (row < a.dk) *reinterpret_cast<f32x4*>(a.s_out + bh * a.s_out_bh + (long)row * a.dv + c) = S[i];
        }
}

// The states at the segments' borders from what each segment adds by itself:
// slot s becomes the state before segment s (BACK: the gradient of the state
// behind it), and what comes out at the far end goes to `end` (null: not
// wanted) and, with slots = nseg + 1, to the last slot.
struct LinScan {
    float* part;         // [batch * key heads][slots][cells]
    const float* begin;  // [batch * key heads][cells]; null: zeros
    float* end;
    const double* gsum;
    int nseg, slots, cells;
};
template <bool BACK> __device__ __forceinline__ void lin_scan(const LinScan& s) {
    constexpr int AHEAD = 8;   // segments read at a time
    const int i = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (i >= s.cells) return;
    const long bh = blockIdx.x;
    f32x4 run = f32x4{0.f, 0.f, 0.f, 0.f};
    if (s.begin) run = *reinterpret_cast<const f32x4*>(s.begin + bh * s.cells + i);
    for (int n0 = 0; n0 < s.nseg; n0 += AHEAD) {
        f32x4 own[AHEAD];
        float keep[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            const int n = min(n0 + e, s.nseg - 1), seg = BACK ? s.nseg - 1 - n : n;
            own[e] = *reinterpret_cast<const f32x4*>(s.part + (bh * s.slots + seg) * s.cells + i);
            keep[e] = __builtin_amdgcn_exp2f((float)s.gsum[bh * s.nseg + seg]);
        }
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            const int n = n0 + e, seg = BACK ? s.nseg - 1 - n : n;
            if (n < s.nseg) {
                *reinterpret_cast<f32x4*>(s.part + (bh * s.slots + seg) * s.cells + i) = run;
#pragma unroll
                for (int c = 0; c < 4; ++c) run[c] = fmaf(keep[e], run[c], own[e][c]);
            }
        }
    }
    if (s.slots > s.nseg) *reinterpret_cast<f32x4*>(s.part + (bh * s.slots + s.nseg) * s.cells + i) = run;
    if (s.end) *reinterpret_cast<f32x4*>(s.end + bh * s.cells + i) = run;
}
// forward: the states (blockIdx.z 0), and their gradients (1)
__global__ __launch_bounds__(256) void lin_scan_kernel(LinScan states, LinScan grads) {
    if (blockIdx.z == 0) lin_scan<false>(states);
    else lin_scan<true>(grads);
}

// <R, S> at the end of a segment.
struct LinFlow {
    const float *S, *R;   // the borders' states and their gradients
    double* flow;         // [batch * key heads][nseg]
    int nseg, slots, cells;
};
__device__ __forceinline__ void lin_flow(const LinFlow& f, int block) {
    __shared__ double red[4];
    const long bh = block / f.nseg;
    const int seg = block % f.nseg;
    const float* s = f.S + (bh * f.slots + seg + 1) * f.cells;
    const float* r = f.R + (bh * f.slots + seg) * f.cells;
    double d = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x * 4; i < f.cells; i += 1024) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(s + i), y = *reinterpret_cast<const f32x4*>(r + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) d = fma((double)x[e], (double)y[e], d);
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) d += __shfl_xor(d, m, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = d;
    __syncthreads();
    if (threadIdx.x == 0) f.flow[bh * f.nseg + seg] = (red[0] + red[1]) + (red[2] + red[3]);
}

// dg of a chunk's tokens but for what passes the chunk, and the sums of fq
// and fk that this follows from.
struct LinPairs {
    const void *q, *k, *v, *dy;
    long qb, qt, kb, kt, vb, vt, gb, gt;
    const float* ld;
    const int* counts;
    const float *dotq, *dotk;   // fq, fk: [slabs][batch * key heads][T]
    float* h;                   // [batch * key heads][T]
    double* sums;               // [batch * key heads][chunks][2]
    float scale;
    int per_token, B, T, Hk, G, dk, dv, chunks, slabs;
};
// All rows are read at once; queries and keys stand in LDS first, then
// gradients and values in their place: 36 KB at widths of 128, so that three
// workgroups share a compute unit (their registers allow no fourth) and hide each
// other's way to memory. 47 us for 2 x 4096 tokens of 16 heads of 128, bf16, with
// the borders' flows; operands straight from memory, in rows of 64 bytes, 57 us.
template <class T, int D, int C>
__global__ __launch_bounds__(256) void lin_pairs_kernel(LinPairs a, LinFlow f, int flows) {
    if ((int)blockIdx.x < flows) return lin_flow(f, blockIdx.x);   // a whole workgroup
    constexpr int PAD = 16 / sizeof(T), RP = D + PAD, NT = C / 16, NS = D / 32, XP = C + 1;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    T* left = reinterpret_cast<T*>(lds);                // queries, then gradients
    T* right = left + C * RP;                           // keys, then values
    double* gs = reinterpret_cast<double*>(right + C * RP);
    float* cross = reinterpret_cast<float*>(gs + 64);   // [64]
    float* X = reinterpret_cast<float*>(lds);           // [C][XP], in the operands' place once they are read
    static_assert(4 * C * XP <= 2 * (int)sizeof(T) * C * RP, "X fits in the operands' place");
    const int block = blockIdx.x - flows, chunk = block % a.chunks, bh = block / a.chunks, b = bh / a.Hk, h = bh % a.Hk;
    const int n = a.counts ? min(max(a.counts[b], 0), a.T) : a.T, t0 = chunk * C;
    if (t0 >= n) return;
    const int rows = min(C, n - t0);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
    if (wave == 0) {
        double g = 0.0;
        if (lane < rows) g = lin_gate(a.ld[a.per_token ? ((long)b * a.T + t0 + lane) * a.Hk + h : h]);
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double o = __shfl_up(g, m, 64);
            if (lane >= m) g += o;
        }
        gs[lane] = g;
    }
    const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb + t0 * a.qt + (long)h * a.G * a.dk;
    const T* k = reinterpret_cast<const T*>(a.k) + b * a.kb + t0 * a.kt + (long)h * a.dk;
    const T* v = reinterpret_cast<const T*>(a.v) + b * a.vb + t0 * a.vt + (long)h * a.dv;
    const T* y = reinterpret_cast<const T*>(a.dy) + b * a.gb + t0 * a.gt + (long)h * a.G * a.dv;
    float x[NT][4];
#pragma unroll
    for (int kt = 0; kt < NT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[kt][r] = 0.f;
    const int i = 16 * wave + l16;
    LinTile<T, D, C> tq, tk, ty, tv;
    for (int g = 0; g < a.G; ++g) {
        tq.load(q + (long)g * a.dk, (unsigned)a.qt, rows, 0, a.dk);
        tk.load(k, (unsigned)a.kt, rows, 0, a.dk);
        ty.load(y + (long)g * a.dv, (unsigned)a.gt, rows, 0, a.dv);
        tv.load(v, (unsigned)a.vt, rows, 0, a.dv);
        f32x4 s[NT], p[NT];
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            __syncthreads();   // what stands in LDS is read
            if (part == 0) {
                tq.template store<false, false>(left, RP, rows, 0, a.dk, nullptr);
                tk.template store<false, false>(right, RP, rows, 0, a.dk, nullptr);
            } else {
                ty.template store<false, false>(left, RP, rows, 0, a.dv, nullptr);
                tv.template store<false, false>(right, RP, rows, 0, a.dv, nullptr);
            }
            __syncthreads();
            f32x4* to = part ? p : s;
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) {
                to[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (kt <= wave && wave < NT)
#pragma unroll
                    for (int u = 0; u < NS; ++u)
                        mma(to[kt], ld8(right + (16 * kt + l16) * RP + 32 * u + 8 * lg), ld8(left + i * RP + 32 * u + 8 * lg));
            }
        }
        if (wave < NT) {
            const double gi = gs[i];
#pragma unroll
            for (int kt = 0; kt < NT; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * kt + 4 * lg + r;
                    const float by = __builtin_amdgcn_exp2f((float)(gi - gs[j])) * a.scale;
                    x[kt][r] += j < i ? s[kt][r] * p[kt][r] * by : 0.f;
                }
        }
    }
    __syncthreads();
    if (wave < NT)
#pragma unroll
        for (int kt = 0; kt < NT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) X[i * XP + 16 * kt + 4 * lg + r] = x[kt][r];
    __syncthreads();
    // sums over j < t of every row, then of those over i >= t: four threads a row, then four a column
    const int at = threadIdx.x >> 2, quarter = threadIdx.x & 3, E = C / 4;
    if (at < C) {
        float* row = X + at * XP + quarter * E;
        float run = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float v0 = row[e];
            row[e] = run;
            run += v0;
        }
        float before = 0.f;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const float o = __shfl(run, (lane & ~3) + p, 64);
            if (p < quarter) before += o;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) row[e] += before;
    }
    __syncthreads();
    if (at < C) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (quarter * E + e >= at) s += X[(quarter * E + e) * XP + at];
        s += __shfl_xor(s, 1, 64);
        s += __shfl_xor(s, 2, 64);
        if (quarter == 0) cross[at] = s;
    }
    __syncthreads();
    if (wave == 0) {
        // 64 bits: what passes a chunk is the small difference of such sums, over all chunks of a segment
        double fq = 0.0, fk = 0.0;
        const long to = (long)bh * a.T + t0 + lane, step = (long)a.B * a.Hk * a.T;
        if (lane < rows)
            for (int z = 0; z < a.slabs; ++z) {
                fq += (double)a.dotq[z * step + to];
                fk += (double)a.dotk[z * step + to];
            }
        double from = fq, upto = fk;   // sums from this token on, and up to it
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double o = __shfl_down(from, m, 64), p = __shfl_up(upto, m, 64);
            if (lane + m < 64) from += o;
            if (lane >= m) upto += p;
        }
        if (lane < rows) a.h[to] = (float)((double)cross[lane] + from + (upto - fk));
        const double all_k = __shfl(upto, 63, 64);
        if (lane == 0) {
            double* s = a.sums + ((long)bh * a.chunks + chunk) * 2;
            s[0] = from;
            s[1] = all_k;
        }
    }
}

// dg of a segment's tokens (per token), or their sum (into part): from the
// segment's last chunk to its first, with what passes each.  Nothing passes a
// chunk with a token that drops what came before, and that token's dg is 0:
// both are set, where the difference would leave a rounding of the flow.
__global__ __launch_bounds__(64) void lin_gates_kernel(const float* h, const double* sums, const double* flow,
                                                       const float* ld, const int* counts, float* dg, double* part,
                                                       int per_token, int T, int Hk, int nseg, int L, int C) {
    const int seg = blockIdx.x % nseg, bh = blockIdx.x / nseg, b = bh / Hk, kh = bh % Hk, lane = threadIdx.x;
    const int n = counts ? min(max(counts[b], 0), T) : T, chunks = (T + C - 1) / C;
    const int first = seg * L, last = (int)min((long)n, (long)first + L);
    double border = flow[(long)bh * nseg + seg], sum = 0.0;
    for (int c = (last - first + C - 1) / C - 1; c >= 0; --c) {
        const int t = first + c * C + lane;
        const double* s = sums + ((long)bh * chunks + first / C + c) * 2;
        const bool on = lane < C && t < last;
        const long at = ((long)b * T + t) * Hk + kh;
        const bool drops = on && ld[per_token ? at : kh] <= LIN_DROPS;
        const double through = __any(drops) ? 0.0 : border - s[1];
        border = through + s[0];
        if (on) {
            const double g = drops ? 0.0 : through + (double)h[(long)bh * T + t];
            if (per_token) dg[at] = (float)g;
            sum += g;
        }
    }
    if (!per_token) {
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m, 64);
        if (lane == 0) part[(long)bh * nseg + seg] = sum;
    }
}
__global__ __launch_bounds__(64) void lin_gate_sum_kernel(const double* part, float* dg, int B, int Hk, int nseg) {
    const int h = blockIdx.x, lane = threadIdx.x;
    double s = 0.0;
    for (long i = lane; i < (long)B * nseg; i += 64) s += part[(i / nseg * Hk + h) * nseg + i % nseg];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m, 64);
    if (lane == 0) dg[h] = (float)s;
}

// to = from (null: zeros), n a multiple of 4
__global__ __launch_bounds__(256) void lin_copy_kernel(const float* from, float* to, long n) {
    for (long i = ((long)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (long)gridDim.x * 1024) {
        f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
        if (from) x = *reinterpret_cast<const f32x4*>(from + i);
        *reinterpret_cast<f32x4*>(to + i) = x;
    }
}
__global__ void lin_zero_kernel(float* p, int n) {
    for (int i = threadIdx.x; i < n; i += 256) p[i] = 0.f;
}

// ---------------------------------------------------------------------------
// launches

#define LIN_TRY(x) do { const hipError_t e_ = (x); if (e_ != hipSuccess) return e_; } while (0)

static int lin_width(int d) { return (d + 63) / 64 * 64; }

template <class T, int DK, int CW, int KIND>
static hipError_t lin_run(LinArgs a, hipStream_t st) {
    a.slabs = (a.dv + 64 * CW - 1) / (64 * CW);
    const long blocks = (long)a.B * a.Hk * a.nseg * a.slabs;
    if (blocks >= 1L << 24) return hipErrorInvalidValue;   // a launch has fewer than 2^32 threads along an axis
    constexpr size_t bytes = LinLds<T, DK, CW, KIND == LIN_STATE>::bytes;
    static_assert(bytes <= 156 * 1024, "LDS of a compute unit");
    static std::atomic<unsigned long long> done{0};
    LIN_TRY(lds_limit((const void*)lin_kernel<T, DK, CW, KIND>, bytes, done));
    return timed_layer(st, [&] {
        launch_k((lin_kernel<T, DK, CW, KIND>), dim3((unsigned)blocks), dim3(256), bytes, st, a);
        return hipGetLastError();
    });
}
// 128 columns a workgroup where its registers hold them (the queries' and
// keys' rows are then read once), 64 for narrow values or wide keys.
static int lin_columns(int dk, int dv) { return dv > 64 && dk <= 128 ? 128 : 64; }
template <class T, int KIND> static hipError_t lin_launch(const LinArgs& a, hipStream_t st) {
    const int w = lin_width(a.dk);
    if (w == 256) return lin_run<T, 256, 1, KIND>(a, st);
    if (w == 192) return lin_run<T, 192, 1, KIND>(a, st);
    if (lin_columns(a.dk, a.dv) == 128)
        return w == 128 ? lin_run<T, 128, 2, KIND>(a, st) : lin_run<T, 64, 2, KIND>(a, st);
    return w == 128 ? lin_run<T, 128, 1, KIND>(a, st) : lin_run<T, 64, 1, KIND>(a, st);
}

// a launch of several runs: the wider of keys and values decides for all
template <class T, int DK, int CW, bool STATES> static hipError_t lin_many_run(LinMany m, hipStream_t st) {
    long blocks = 0;
    for (int i = 0; i < (STATES ? 2 : 3); ++i) {
        m.a[i].slabs = (m.a[i].dv + 64 * CW - 1) / (64 * CW);
        const long own = (long)m.a[i].B * m.a[i].Hk * m.a[i].nseg * m.a[i].slabs;
        m.blocks[i] = (int)own;   // refused below where it does not fit
        blocks += own;
    }
    if (blocks >= 1L << 24) return hipErrorInvalidValue;
    constexpr size_t bytes = LinLds<T, DK, CW, STATES>::bytes;
    auto go = [&](auto kernel) {
        static std::atomic<unsigned long long> done{0};   // an instance of this function has one kernel
        LIN_TRY(lds_limit((const void*)kernel, bytes, done));
        return timed_layer(st, [&] {
            launch_k(kernel, dim3((unsigned)blocks), dim3(256), bytes, st, m);
            return hipGetLastError();
        });
    };
    if constexpr (STATES) return go(lin_states_kernel<T, DK, CW>);
    else return go(lin_gradients_kernel<T, DK, CW>);
}
template <class T, bool STATES> static hipError_t lin_many(const LinMany& m, int wide, hipStream_t st) {
    const int w = lin_width(wide);
    return w == 256   ? lin_many_run<T, 256, 1, STATES>(m, st)
           : w == 192 ? lin_many_run<T, 192, 1, STATES>(m, st)
           : w == 128 ? lin_many_run<T, 128, 2, STATES>(m, st)
                      : lin_many_run<T, 64, 1, STATES>(m, st);
}
static int lin_many_columns(int wide) { return lin_width(wide) == 128 ? 128 : 64; }

template <class T, int D, int C> static hipError_t lin_pairs_run(LinPairs a, const LinFlow& f, hipStream_t st) {
    a.chunks = (a.T + C - 1) / C;
    const long flows = (long)a.B * a.Hk * f.nseg, blocks = flows + (long)a.B * a.Hk * a.chunks;
    if (blocks >= 1L << 24) return hipErrorInvalidValue;
    constexpr size_t bytes = 2 * sizeof(T) * C * (D + 16 / sizeof(T)) + 8 * 64 + 4 * 64;
    static_assert(bytes <= 156 * 1024, "LDS of a compute unit");
    static std::atomic<unsigned long long> done{0};
    LIN_TRY(lds_limit((const void*)lin_pairs_kernel<T, D, C>, bytes, done));
    return timed_layer(st, [&] {
        launch_k((lin_pairs_kernel<T, D, C>), dim3((unsigned)blocks), dim3(256), bytes, st, a, f, (int)flows);
        return hipGetLastError();
    });
}
template <class T> static hipError_t lin_pairs(const LinPairs& a, const LinFlow& f, hipStream_t st) {
    const int w = lin_width(a.dk > a.dv ? a.dk : a.dv);
    constexpr int C = lin_chunk<T>();
    return w >= 192 ? lin_pairs_run<T, 256, C>(a, f, st) : w == 128 ? lin_pairs_run<T, 128, C>(a, f, st) : lin_pairs_run<T, 64, C>(a, f, st);
}

template <class T, int DK> static hipError_t lin_token_run(LinArgs a, hipStream_t st) {
    a.slabs = (a.dv + 31) / 32;
    const long blocks = (long)a.B * a.Hk * a.slabs;
    if (blocks >= 1L << 24) return hipErrorInvalidValue;
    const size_t one = LinToken<T>::bytes(a.G, a.dk);
    static_assert(LinToken<float>::bytes(64, 256) <= 156 * 1024, "LDS of a compute unit");
    const int batch = (int)std::max<size_t>(1, std::min<size_t>(a.T, 40 * 1024 / one));
    static std::atomic<unsigned long long> done{0};
    LIN_TRY(lds_limit((const void*)lin_token_kernel<T, DK>, one * batch, done));
    return timed_layer(st, [&] {
        launch_k((lin_token_kernel<T, DK>), dim3((unsigned)blocks), dim3(256), one * batch, st, a, batch);
        return hipGetLastError();
    });
}
template <class T> static hipError_t lin_tokens_run(const LinArgs& a, hipStream_t st) {
    return a.dk <= 64 ? lin_token_run<T, 64>(a, st) : a.dk <= 128 ? lin_token_run<T, 128>(a, st) : lin_token_run<T, 256>(a, st);
}

// How a call is divided, and where its workspace holds what.
struct LinPlan {
    int nseg, L;
    size_t states, grads, gsum, flow, dotq, dotk, h, sums, part, bytes;
};
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

static LinPlan lin_plan(int B, int T, int Hk, int dk, int dv, bool back) {
    LinPlan p{};
    if (B == 0 || T == 0) return p;
    const size_t bh = (size_t)B * Hk, cells = (size_t)dk * dv;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += up256(n);
        return o;
    };
    if (back) {
        // Halved while there are fewer segments than compute units: a segment is a
        // workgroup's walk, one chunk after another.
        p.L = LIN_BACK_SEG;
        while (p.L > 64 && (long)bh * ((T + p.L - 1) / p.L) < 256) p.L /= 2;
        p.nseg = (T + p.L - 1) / p.L;
        p.states = take(bh * (p.nseg + 1) * cells * 4);
        p.grads = take(bh * (p.nseg + 1) * cells * 4);
        p.gsum = take(bh * p.nseg * 8);
        p.flow = take(bh * p.nseg * 8);
        p.dotq = take(bh * T * 4 * ((dk + 63) / 64));
        p.dotk = take(bh * T * 4 * ((dk + 63) / 64));
        p.h = take(bh * T * 4);
        p.sums = take(bh * ((T + 31) / 32) * 16);   // chunks of 32 tokens, or 64
        p.part = take(bh * p.nseg * 8);
    } else {
        // The sequence is divided where its heads alone do not fill the chip, into
        // segments of 64 tokens while those are few, else of 128 at least (us
        // undivided / 256 / 128 / 64 tokens at least, bf16: 8 heads of 128, 512
        // tokens 48 / 42 / 28 / 23, 4096 tokens 350 / 49 / 40 / 47; 64 heads of 128,
        // 512 tokens 51 / 48 / 39 / 44; 2 heads of 64, 2048 tokens 98 / 26 / 19 / 18;
        // fp32: 8 heads of 128, 1024 tokens 239 / 97 / 57 / 41).  Undivided: 256
        // heads of 64, 2048 tokens 103 against 107 (512 tokens 30 against 41, fp32
        // 2048 tokens 180 against 217); 8 heads of 128, 128 tokens 17.
        const long cols = lin_columns(dk, dv), wgs = (long)bh * ((dv + cols - 1) / cols);
        const long least = wgs * ((T + 63) / 64) <= 256 ? 64 : 128;
        long seg = wgs >= 256 || T <= 192 ? 1 : (512 + wgs - 1) / wgs;
        seg = seg < (T + least - 1) / least ? seg : (T + least - 1) / least;
        p.L = (int)(((T + seg - 1) / seg + 63) / 64 * 64);
        p.nseg = (T + p.L - 1) / p.L;
        if (p.nseg > 1) {
            p.states = take(bh * p.nseg * cells * 4);
            p.gsum = take(bh * p.nseg * 8);
        }
    }
    p.bytes = at;
    return p;
}

static hipError_t lin_scan_run(const LinScan& s, const LinScan* grads, long bh, hipStream_t st) {
    return timed_layer(st, [&] {
        launch_k(lin_scan_kernel, dim3((unsigned)bh, (s.cells + 1023) / 1024, grads ? 2 : 1), dim3(256), 0, st, s,
                 grads ? *grads : LinScan{});
        return hipGetLastError();
    });
}

static hipError_t lin_copy(const float* from, float* to, long n, hipStream_t st) {
    const long blocks = (n + 1023) / 1024;
    return timed_layer(st, [&] {
        launch_k(lin_copy_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, from, to, n);
        return hipGetLastError();
    });
}

template <class T> static hipError_t lin_forward(LinArgs a, float* state_out, char* ws, hipStream_t st) {
    const long cells = (long)a.dk * a.dv;
    a.s_in_bh = a.s_out_bh = cells;
    if (a.T <= lin_few<T>()) {
        a.s_out = state_out;
        return lin_tokens_run<T>(a, st);
    }
    const LinPlan p = lin_plan(a.B, a.T, a.Hk, a.dk, a.dv, false);
    a.nseg = p.nseg;
    a.L = p.L;
    if (p.nseg == 1) {
        a.s_out = state_out;
        return lin_launch<T, LIN_OUT>(a, st);
    }
    float* parts = reinterpret_cast<float*>(ws + p.states);
    double* gsum = reinterpret_cast<double*>(ws + p.gsum);
    LinArgs b = a;
    b.G = 1;
    b.s_out = parts;
    b.s_out_bh = p.nseg * cells;
    b.s_out_seg = cells;
    b.gsum = gsum;
    LIN_TRY((lin_launch<T, LIN_STATE>(b, st)));
    LIN_TRY(lin_scan_run(LinScan{parts, a.s_in, state_out, gsum, p.nseg, p.nseg, (int)cells}, nullptr, (long)a.B * a.Hk, st));
    a.s_in = parts;
    a.s_in_bh = p.nseg * cells;
    a.s_in_seg = cells;
    return lin_launch<T, LIN_OUT>(a, st);
}

struct LinBack {
    const void* dy;
    long gb, gt;
    const float* dstate_out;
    void *dq, *dk, *dv;
    float *dld, *dstate_in;
};

template <class T> static hipError_t lin_backward(LinArgs a, const LinBack& g, char* ws, hipStream_t st) {
    const int dk = a.dk, dv = a.dv;
    const long cells = (long)dk * dv, bh = (long)a.B * a.Hk;
    const LinPlan p = lin_plan(a.B, a.T, a.Hk, dk, dv, true);
    const int slots = p.nseg + 1, wide = dk > dv ? dk : dv;
    // the largest launches (three runs of up to four slabs, a chunk of 32 tokens or a segment each): before the first
    if (bh * p.nseg * 12 >= 1L << 24 || bh * ((a.T + 31) / 32 + (long)p.nseg) >= 1L << 24) return hipErrorInvalidValue;
    a.nseg = p.nseg;
    a.L = p.L;
    float* S = reinterpret_cast<float*>(ws + p.states);
    float* R = reinterpret_cast<float*>(ws + p.grads);
    double* gsum = reinterpret_cast<double*>(ws + p.gsum);
    double* flow = reinterpret_cast<double*>(ws + p.flow);
    float* dotq = reinterpret_cast<float*>(ws + p.dotq);
    float* dotk = reinterpret_cast<float*>(ws + p.dotk);
    const float scale = a.far_scale;
    // what each segment adds to the state and to its gradient, then the borders
    LinArgs s = a;
    s.G = 1;
    s.s_out = S;
    s.s_out_bh = slots * cells;
    s.s_out_seg = cells;
    s.gsum = gsum;
    LinArgs r = s;
    r.G = a.G;
    r.k = a.q; r.kb = a.qb; r.kt = a.qt;
    r.v = g.dy; r.vb = g.gb; r.vt = g.gt;
    r.s_out = R;
    r.state_scale = scale;
    r.gsum = nullptr;
    LIN_TRY((lin_many<T, true>(LinMany{{r, s}, {}}, wide, st)));
    const LinScan back{R, g.dstate_out, g.dstate_in, gsum, p.nseg, slots, (int)cells};
    LIN_TRY(lin_scan_run(LinScan{S, a.s_in, nullptr, gsum, p.nseg, slots, (int)cells}, &back, bh, st));
    // the three gradients of token arrays
    LinArgs x = a;
    x.s_in_bh = slots * cells;
    x.s_in_seg = cells;
    x.s_out = nullptr;
    x.gsum = nullptr;
    LinArgs y = x;
    y.q = g.dy; y.qb = g.gb; y.qt = g.gt; y.k = a.v; y.kb = a.vb; y.kt = a.vt; y.v = a.k; y.vb = a.kb; y.vt = a.kt;
    y.z = a.q; y.zb = a.qb; y.zt = a.qt;
    y.dk = dv; y.dv = dk; y.s_in = S; y.out = g.dq; y.dot = dotq;
    LinArgs w = x;
    w.q = a.v; w.qb = a.vb; w.qt = a.vt; w.k = g.dy; w.kb = g.gb; w.kt = g.gt; w.v = a.q; w.vb = a.qb; w.vt = a.qt;
    w.z = a.k; w.zb = a.kb; w.zt = a.kt;
    w.dk = dv; w.dv = dk; w.s_in = R; w.out = g.dk; w.dot = dotk;
    w.far_scale = 1.f; w.state_scale = scale;
    x.q = a.k; x.qb = a.kb; x.qt = a.kt; x.k = a.q; x.kb = a.qb; x.kt = a.qt; x.v = g.dy; x.vb = g.gb; x.vt = g.gt;
    x.s_in = R; x.out = g.dv;
    x.far_scale = 1.f; x.state_scale = scale;
    LIN_TRY((lin_many<T, false>(LinMany{{w, y, x}, {}}, wide, st)));
    if (!g.dld) return hipSuccess;
    // the decays
    float* h = reinterpret_cast<float*>(ws + p.h);
    double* part = reinterpret_cast<double*>(ws + p.part);
    double* sums = reinterpret_cast<double*>(ws + p.sums);
    LinPairs pairs{a.q, a.k, a.v, g.dy, a.qb, a.qt, a.kb, a.kt, a.vb, a.vt, g.gb, g.gt, a.ld, a.counts, dotq, dotk, h, sums,
               scale, a.per_token, a.B, a.T, a.Hk, a.G, dk, dv, 0, (dk + lin_many_columns(wide) - 1) / lin_many_columns(wide)};
    LIN_TRY(lin_pairs<T>(pairs, LinFlow{S, R, flow, p.nseg, slots, (int)cells}, st));
    LIN_TRY(timed_layer(st, [&] {
        launch_k(lin_gates_kernel, dim3((unsigned)(bh * p.nseg)), dim3(64), 0, st, h, sums, flow, a.ld, a.counts,
                 g.dld, part, a.per_token, a.T, a.Hk, p.nseg, p.L, lin_chunk<T>());
        return hipGetLastError();
    }));
    if (a.per_token) return hipSuccess;
    return timed_layer(st, [&] {
        launch_k(lin_gate_sum_kernel, dim3(a.Hk), dim3(64), 0, st, part, g.dld, a.B, a.Hk, p.nseg);
        return hipGetLastError();
    });
}

static bool lin_sizes_ok(int B, int T, int H, int Hk, int dk, int dv) {
    return B >= 0 && T >= 0 && T <= 1 << 30 && H > 0 && Hk > 0 && H % Hk == 0 && H / Hk <= 64 && H <= 32768 && dk >= 8 && dk <= 256 &&
           dk % 8 == 0 && dv >= 8 && dv <= 256 && dv % 8 == 0 && (long)B * Hk < 1L << 24 &&
           (B == 0 || T <= (1L << 40) / ((long)B * H * 256));
}
static bool lin_tokens_ok(const void* p, long batch, long token, int B, int T) {
    const long lim = 1L << 40;   // 64 rows within 2^31 bytes
    return p && (uintptr_t)p % 16 == 0 && batch >= 0 && token >= 0 && batch <= lim && token < 1L << 23 && batch % 8 == 0 &&
           token % 8 == 0 && (double)B * (double)batch < 4e18 && (double)T * (double)token < 4e18;
}
static tm_status lin_status(hipError_t e) {
    return e == hipSuccess ? TM_OK : e == hipErrorInvalidValue ? TM_ERR_INVALID : TM_ERR_HIP;
}

}  // namespace tmk

using namespace tmk;

extern "C" {

size_t tm_linear_workspace_bytes(int batch, int n_tokens, int heads, int kv_heads, int key_dim, int value_dim,
                                 int backward) {
    if (!lin_sizes_ok(batch, n_tokens, heads, kv_heads, key_dim, value_dim)) return 0;
    return lin_plan(batch, n_tokens, kv_heads, key_dim, value_dim, backward != 0).bytes;
}

tm_status tm_linear_attention(const void* q, long q_batch, long q_token, const void* k, long k_batch, long k_token,
                              const void* v, long v_batch, long v_token, const float* log_decay, int per_token,
                              const int* counts, const float* state_in, float* state_out, void* out, double scale,
                              int batch, int n_tokens, int heads, int kv_heads, int key_dim, int value_dim,
                              tm_dtype dtype, void* workspace, void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (!lin_sizes_ok(batch, n_tokens, heads, kv_heads, key_dim, value_dim) || !isfinite((float)scale) ||
        (uintptr_t)state_in % 16 || (uintptr_t)state_out % 16)
        return TM_ERR_INVALID;
    if (batch == 0) return TM_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (n_tokens == 0) {
        if (!state_out || state_out == state_in) return TM_OK;
        return lin_status(lin_copy(state_in, state_out, (long)batch * kv_heads * key_dim * value_dim, st));
    }
    if (!lin_tokens_ok(q, q_batch, q_token, batch, n_tokens) || !lin_tokens_ok(k, k_batch, k_token, batch, n_tokens) ||
        !lin_tokens_ok(v, v_batch, v_token, batch, n_tokens) || !out || (uintptr_t)out % 16 || !log_decay ||
        (uintptr_t)log_decay % 4 || (uintptr_t)counts % 4 || (uintptr_t)workspace % 256 ||
        (!workspace && lin_plan(batch, n_tokens, kv_heads, key_dim, value_dim, false).bytes))
        return TM_ERR_INVALID;
    LinArgs a{};
    a.q = q; a.qb = q_batch; a.qt = q_token; a.k = k; a.kb = k_batch; a.kt = k_token; a.v = v; a.vb = v_batch; a.vt = v_token;
    a.ld = log_decay; a.per_token = per_token != 0; a.counts = counts; a.s_in = state_in; a.out = out;
    a.pair_scale = a.far_scale = (float)scale; a.state_scale = 1.f;
    a.B = batch; a.T = n_tokens; a.Hk = kv_heads; a.G = heads / kv_heads; a.dk = key_dim; a.dv = value_dim;
    char* ws = static_cast<char*>(workspace);
    return lin_status(dtype == TM_F32 ? lin_forward<float>(a, state_out, ws, st) : lin_forward<bf16>(a, state_out, ws, st));
}

tm_status tm_linear_attention_backward(const void* q, long q_batch, long q_token, const void* k, long k_batch,
                                       long k_token, const void* v, long v_batch, long v_token,
                                       const float* log_decay, int per_token, const int* counts,
                                       const float* state_in, const void* dout, long dout_batch, long dout_token,
                                       const float* dstate_out, void* dq, void* dk, void* dv, float* dlog_decay,
                                       float* dstate_in, double scale, int batch, int n_tokens, int heads,
                                       int kv_heads, int key_dim, int value_dim, tm_dtype dtype, void* workspace,
                                       void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (!lin_sizes_ok(batch, n_tokens, heads, kv_heads, key_dim, value_dim) || !isfinite((float)scale) ||
        (uintptr_t)state_in % 16 || (uintptr_t)dstate_out % 16 || (uintptr_t)dstate_in % 16 || (uintptr_t)dlog_decay % 4)
        return TM_ERR_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (batch == 0 || n_tokens == 0) {
        if (dlog_decay && !per_token) {
            const hipError_t e = timed_layer(st, [&] {
                launch_k(lin_zero_kernel, dim3(1), dim3(256), 0, st, dlog_decay, kv_heads);
                return hipGetLastError();
            });
            if (e != hipSuccess) return lin_status(e);
        }
        if (batch == 0 || !dstate_in || dstate_in == dstate_out) return TM_OK;
        return lin_status(lin_copy(dstate_out, dstate_in, (long)batch * kv_heads * key_dim * value_dim, st));
    }
    if (!lin_tokens_ok(q, q_batch, q_token, batch, n_tokens) || !lin_tokens_ok(k, k_batch, k_token, batch, n_tokens) ||
        !lin_tokens_ok(v, v_batch, v_token, batch, n_tokens) ||
        !lin_tokens_ok(dout, dout_batch, dout_token, batch, n_tokens) || !dq || (uintptr_t)dq % 16 || !dk ||
        (uintptr_t)dk % 16 || !dv || (uintptr_t)dv % 16 || !log_decay || (uintptr_t)log_decay % 4 ||
        (uintptr_t)counts % 4 || !workspace || (uintptr_t)workspace % 256)
        return TM_ERR_INVALID;
    LinArgs a{};
    a.q = q; a.qb = q_batch; a.qt = q_token; a.k = k; a.kb = k_batch; a.kt = k_token; a.v = v; a.vb = v_batch; a.vt = v_token;
    a.ld = log_decay; a.per_token = per_token != 0; a.counts = counts; a.s_in = state_in;
    a.pair_scale = a.far_scale = (float)scale; a.state_scale = 1.f;
    a.B = batch; a.T = n_tokens; a.Hk = kv_heads; a.G = heads / kv_heads; a.dk = key_dim; a.dv = value_dim;
    const LinBack g{dout, dout_batch, dout_token, dstate_out, dq, dk, dv, dlog_decay, dstate_in};
    char* ws = static_cast<char*>(workspace);
    return lin_status(dtype == TM_F32 ? lin_backward<float>(a, g, ws, st) : lin_backward<bf16>(a, g, ws, st));
}

}  // extern "C"
