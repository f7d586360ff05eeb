// Products with 8-bit integers (include/tm_layer.h): rows as codes with a
// scale each, and the matrix product of codes with a scale for each row of
// either side,  y[m][n] = (sum_k a[m][k] w[n][k]) a_scale[m] w_scale[n].
// The sums are exact in 32 bits (at most 131072 products of 127 * 127).
#include <math.h>

#include "../../include/tm_layer.h"
#include "tm_device.h"

namespace tmk {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// codes = rint((127 x) / m) in fp32.  The product comes first: it is exact for
// bf16, so that a quotient halfway between two codes is one in fp32 too, and
// (127 x and m have 15 and 8 bits) no other is; a row whose 127 m would
// overflow is divided by 2^10 beforehand (exactly).  Products with 127 / m
// give the quotients to 2.3e-5 (127 times two roundings and the quotient's
// own), so only where one is within 1e-4 of a half are four of them divided.
struct Int8Scale {
    float scale, down, top, by;   // the row's scale; its factors
    bool any;                     // false: all codes are 0
};
__device__ __forceinline__ Int8Scale int8_scale(float m) {   // m: infinity where an element is not finite
    Int8Scale s;
    const bool lost = m == __builtin_inff();
    s.any = m > 0.f && !lost;
    s.down = m > 1e36f ? 0x1p-10f : 1.f;
    s.top = m * s.down;
    s.by = 127.f / m;   // infinite for the smallest m: all are divided then
    s.scale = lost ? __builtin_nanf("") : m / 127.f;
    return s;
}
// max |x| of a row's share, infinity where an element is not finite: as bits
// without their sign, which are in the order of the values (bf16: two at a
// time).
template <class T> struct Int8Max;
template <> struct Int8Max<float> {
    unsigned m = 0;
    __device__ __forceinline__ void add(float x) { m = max(m, __builtin_bit_cast(unsigned, x) & 0x7fffffffu); }
    __device__ __forceinline__ void add(f32x4 v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) add(v[e]);
    }
    __device__ __forceinline__ float get() const { return __builtin_bit_cast(float, min(m, 0x7f800000u)); }
};
template <> struct Int8Max<bf16> {
    typedef unsigned short H2 __attribute__((ext_vector_type(2)));
    typedef unsigned U4 __attribute__((ext_vector_type(4)));
    H2 m = {0, 0};
    __device__ __forceinline__ void two(unsigned w) { m = __builtin_elementwise_max(m, __builtin_bit_cast(H2, w & 0x7fff7fffu)); }
    __device__ __forceinline__ void add(bf16 x) { two(__builtin_bit_cast(unsigned short, x)); }
    __device__ __forceinline__ void add(bf16x8 v) {
        const U4 u = __builtin_bit_cast(U4, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) two(u[e]);
    }
    __device__ __forceinline__ float get() const {
        const unsigned h = max(m[0], m[1]);
        return __builtin_bit_cast(float, min(h, 0x7f80u) << 16);
    }
};
template <class T> struct Int8Vec;
template <> struct Int8Vec<float> { typedef f32x4 V; };
template <> struct Int8Vec<bf16> { typedef bf16x8 V; };

// 4 values as the bytes of a word.  Added to 1.5 * 2^23 a quotient is rounded
// to a whole number, to even at a half, which stands in the low bits.
__device__ __forceinline__ unsigned int8_pack(const float* x, const Int8Scale& s) {
    constexpr float ONES = 12582912.f;
    float v[4], off[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = fmaf(x[e], s.by, ONES);
        off[e] = fabsf(fmaf(x[e], s.by, -(v[e] - ONES)));   // from the whole number
    }
    // next to a half; an infinite factor makes all of these infinite or NaN
    if (!(fmaxf(fmaxf(off[0], off[1]), fmaxf(off[2], off[3])) < 0.4999f) || s.by == __builtin_inff())
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = 127.f * (x[e] * s.down) / s.top + ONES;
    const unsigned a = __builtin_bit_cast(unsigned, v[0]), b = __builtin_bit_cast(unsigned, v[1]),
                   c = __builtin_bit_cast(unsigned, v[2]), d = __builtin_bit_cast(unsigned, v[3]);
    // the low bytes: of a and b, then of c and d, then both pairs
    const unsigned ab = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), cd = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
    return s.any ? (ab | cd << 16) : 0u;
}
// the codes of 16 bytes of a row
__device__ __forceinline__ void int8_put_codes(signed char* c, f32x4 v, const Int8Scale& s) {
    const float f[4] = {v[0], v[1], v[2], v[3]};
    *reinterpret_cast<unsigned*>(c) = int8_pack(f, s);
}
__device__ __forceinline__ void int8_put_codes(signed char* c, bf16x8 v, const Int8Scale& s) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
    const uint2 w = {int8_pack(f, s), int8_pack(f + 4, s)};
    *reinterpret_cast<uint2*>(c) = w;
}

// One row a workgroup.  VEC: rows allow loads of 16 bytes; up to 32 elements a
// thread stay in registers between the maximum and the codes.
template <class T, bool VEC>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const T* x, long x_row, signed char* codes, long code_row,
                                                            float* scales, int cols) {
    typedef typename Int8Vec<T>::V Vec;
    constexpr int VE = 16 / sizeof(T), KEEP = 32 / VE;
    __shared__ float red[4];
    const long row = blockIdx.x;
    const T* p = x + row * x_row;
    signed char* c = codes + row * code_row;
    Int8Max<T> top;
    Vec kept[KEEP];
    const int units = VEC ? cols / VE : 0;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int u = threadIdx.x + 256 * i;
            if (u < units) kept[i] = *reinterpret_cast<const Vec*>(p + (long)u * VE);
        }
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if ((int)threadIdx.x + 256 * i < units) top.add(kept[i]);
        for (int u = threadIdx.x + 256 * KEEP; u < units; u += 256) top.add(*reinterpret_cast<const Vec*>(p + (long)u * VE));
    }
    for (int i = units * VE + threadIdx.x; i < cols; i += 256) top.add(p[i]);
    float m = top.get();
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    const Int8Scale s = int8_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    if (threadIdx.x == 0) scales[row] = s.scale;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if ((int)threadIdx.x + 256 * i < units) int8_put_codes(c + (long)(threadIdx.x + 256 * i) * VE, kept[i], s);
        for (int u = threadIdx.x + 256 * KEEP; u < units; u += 256)
            int8_put_codes(c + (long)u * VE, *reinterpret_cast<const Vec*>(p + (long)u * VE), s);
    }
    // the rest of the row, and the zeros behind it, 4 columns at a time
    for (long i = units * VE + 4 * threadIdx.x; i < code_row; i += 1024) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = i + e < cols ? (float)p[i + e] : 0.f;
        *reinterpret_cast<unsigned*>(c + i) = int8_pack(f, s);
    }
}

struct Int8Args {
    const signed char* a;
    const float* as;
    const signed char* w;
    const float* wsc;
    void* y;
    long code_row, y_row, M;
    int N, mtiles, ntiles, vec;   // vec: rows of y allow stores of 4 values
    const void* x;                // the fused call's rows
    long x_row;
    int cols, xvec;
};

// 4 neighbouring outputs of one row, in 64 bits: neither product overflows
// where the result does not.
template <class T>
__device__ __forceinline__ void int8_put(const Int8Args& g, long m, int n, const int* sum, double s) {
    T* y = reinterpret_cast<T*>(g.y) + m * g.y_row;
    struct __align__(4 * sizeof(T)) V4 { T e[4]; } o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o.e[r] = (T)((double)sum[r] * s * (double)(n + r < g.N ? g.wsc[n + r] : 0.f));
    if (g.vec && n + 3 < g.N) {
        *reinterpret_cast<V4*>(y + n) = o;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < g.N) y[n + r] = o.e[r];
    }
}

// BM rows of x by BN rows of w a workgroup, WM x WN waves.  128 bytes of each
// row go through one of two LDS buffers by loads that write it directly, while
// the other is multiplied.  A row's 16-byte pieces are permuted by its number
// (piece p of row r stands at p ^ (r & 7)), so that 16 rows are read at
// different banks; the loads permute on the memory's side.  The rows of w are
// the matrix instruction's first operand, so a lane ends up with 4
// neighbouring outputs of one row of y.
template <class T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void int8_tile_kernel(Int8Args g) {
    constexpr int KT = 128, NWV = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int PIECES = (BM + BN) / 8 / NWV;   // 8 rows a load of a wave
    static_assert((BM + BN) % (8 * NWV) == 0, "whole loads");
    extern __shared__ __attribute__((aligned(16))) signed char lds[];   // [2][BM + BN][KT]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, lg = lane >> 4;
    // neighbouring tiles on one XCD (workgroups go to the 8 of them in turn):
    // 8 tiles of x's rows by consecutive ones of w's
    const long tiles = (long)g.mtiles * g.ntiles;
    long tile = blockIdx.x;
    {
        const long per = tiles / 8, more = tiles % 8, xcd = tile % 8, at = tile / 8;
        tile = xcd * per + min(xcd, more) + at;
    }
    const long band = tile / (8L * g.ntiles), in_band = tile - band * 8 * g.ntiles;
    const int high = (int)min(8L, g.mtiles - band * 8);
    const long m0 = (band * 8 + in_band % high) * BM;
    const int n0 = (int)(in_band / high) * BN;
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);

    // this lane's pieces: row (of the stacked tiles) 8 piece + lane / 8, 16 bytes (lane & 7) ^ (row & 7)
    const signed char* src[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int r = 8 * (wave + NWV * i) + (lane >> 3);
        const long c = (((lane & 7) ^ (r & 7)) * 16);
        // rows behind the last are read as the last (their products are not stored)
        src[i] = (r < BM ? g.a + min(m0 + r, g.M - 1) * g.code_row : g.w + min(n0 + r - BM, g.N - 1) * g.code_row) + c;
    }
    const int steps = (int)((g.code_row + KT - 1) / KT), full = (int)(g.code_row / KT);
    auto fetch = [&](int k) {
        signed char* to = lds + (k & 1) * (BM + BN) * KT;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            signed char* at = to + 8 * (wave + NWV * i) * KT;   // one for the wave
            if (k < full) {
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src[i] + (long)k * KT),
                                                 (__attribute__((address_space(3))) void*)at, 16, 0, 0);
            } else {   // the last columns: zeros behind them
                const int r = 8 * (wave + NWV * i) + (lane >> 3);
                const long c = (long)k * KT + (((lane & 7) ^ (r & 7)) * 16);
                i32x4 v = i32x4{0, 0, 0, 0};
                if (c < g.code_row) v = *reinterpret_cast<const i32x4*>(src[i] + (long)k * KT);
                *reinterpret_cast<i32x4*>(at + lane * 16) = v;
            }
        }
    };
    i32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    fetch(0);
    for (int k = 0; k < steps; ++k) {
        // buffer k is there (a barrier by itself does not wait for loads into LDS), the other one is read
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (k + 1 < steps) fetch(k + 1);
        const signed char* at = lds + (k & 1) * (BM + BN) * KT;
        const signed char* wt = at + BM * KT;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int off = ((4 * s + lg) ^ (l16 & 7)) * 16;
            i32x4 x[TM], y[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) y[j] = *reinterpret_cast<const i32x4*>(wt + (wn + 16 * j + l16) * KT + off);
#pragma unroll
            for (int i = 0; i < TM; ++i) x[i] = *reinterpret_cast<const i32x4*>(at + (wm + 16 * i + l16) * KT + off);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(y[j], x[i], acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const long m = m0 + wm + 16 * i + l16;
        if (m >= g.M) continue;
        const double s = g.as[m];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = n0 + wn + 16 * j + 4 * lg;
            if (n < g.N) {
                const int sum[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                int8_put<T>(g, m, n, sum, s);
            }
        }
    }
}

// Few rows of x: 16 NR rows of w by 16 MT rows of x a workgroup, the columns
// divided among its 8 waves, whose sums meet in LDS.  Bound by reading w once.
// FUSED (MT 1): the workgroup makes the rows' codes itself, in LDS, while its
// first loads of w are under way: one launch, and the rows come from the L2.
// Every workgroup repeats that, so NR is 2 where 16 rows of w would make more
// workgroups than there are compute units.
template <class T, int MT, int NR, bool FUSED>
__global__ __launch_bounds__(512, NR == 1 ? 4 : 2) void int8_thin_kernel(Int8Args g) {
    constexpr int AHEAD = 8;   // blocks of 64 columns in flight for a wave
    extern __shared__ __attribute__((aligned(16))) signed char lds[];   // codes [M][stride] (FUSED); sums [8][MT][NR][16][17]
    __shared__ float sc[16];
    __shared__ float top[8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16 * NR;
    const long m0 = (long)blockIdx.y * 16 * MT;
    const int blocks = (int)((g.code_row + 63) / 64), per = (blocks + 7) / 8;
    const int b0 = wave * per, b1 = min(blocks, b0 + per);
    const int stride = blocks * 64 + 16;
    const signed char* w[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) w[r] = g.w + (long)min(n0 + 16 * r + l16, g.N - 1) * g.code_row + 16 * lg;
    auto load_w = [&](int r, int b) {
        i32x4 v = i32x4{0, 0, 0, 0};
        if (b < b1 && 64L * b + 16 * lg < g.code_row) v = *reinterpret_cast<const i32x4*>(w[r] + 64L * b);
        return v;
    };
    i32x4 wv[NR][AHEAD];
    auto first_w = [&] {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int r = 0; r < NR; ++r) wv[r][i] = load_w(r, b0 + i);
    };
    if constexpr (!FUSED) first_w();
    if constexpr (FUSED) {
        // threads of a row: all 512 for one row, 32 for 16
        const int M = (int)g.M;
        int lanes = 512;
        while (lanes * M > 512) lanes >>= 1;
        const int row = threadIdx.x / lanes, at = threadIdx.x % lanes;
        const bool on = row < M;
        const T* x = reinterpret_cast<const T*>(g.x) + (on ? row : 0) * g.x_row;
        typedef typename Int8Vec<T>::V Vec;
        constexpr int VE = 16 / sizeof(T), KEEP = 64 / VE;
        const int units = g.xvec ? g.cols / VE : 0;
        Int8Max<T> most;
        Vec kept[KEEP];
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (on && at + i * lanes < units) kept[i] = *reinterpret_cast<const Vec*>(x + (long)(at + i * lanes) * VE);
        first_w();   // behind the rows' loads, which are waited for first: loads come back in order
        if (on) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (at + i * lanes < units) most.add(kept[i]);
            for (int u = at + KEEP * lanes; u < units; u += lanes) most.add(*reinterpret_cast<const Vec*>(x + (long)u * VE));
            for (int i = units * VE + at; i < g.cols; i += lanes) most.add(x[i]);
        }
        float m = most.get();
        for (int s = min(lanes, 64) >> 1; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
        if (lanes > 64) {   // a row's waves
            if (lane == 0) top[wave] = m;
            __syncthreads();
            const int first = row * (lanes / 64);
            if (on)
                for (int i = 0; i < lanes / 64; ++i) m = fmaxf(m, top[first + i]);
        }
        const Int8Scale s = int8_scale(m);
        if (on) {
            if (at == 0) sc[row] = s.scale;
            signed char* c = lds + row * stride;
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (at + i * lanes < units) int8_put_codes(c + (at + i * lanes) * VE, kept[i], s);
            for (int u = at + KEEP * lanes; u < units; u += lanes)
                int8_put_codes(c + u * VE, *reinterpret_cast<const Vec*>(x + (long)u * VE), s);
            for (int i = units * VE + 4 * at; i < blocks * 64; i += 4 * lanes) {
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = i + e < g.cols ? (float)x[i + e] : 0.f;
                *reinterpret_cast<unsigned*>(c + i) = int8_pack(f, s);
            }
        }
        __syncthreads();
    }
    i32x4 acc[MT][NR];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[i][r] = i32x4{0, 0, 0, 0};
    for (int b = b0; b < b1; b += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            i32x4 cur[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                cur[r] = wv[r][i];
                wv[r][i] = load_w(r, b + AHEAD + i);
            }
            if (b + i < b1)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    i32x4 x = i32x4{0, 0, 0, 0};
                    if constexpr (FUSED) {
                        x = *reinterpret_cast<const i32x4*>(lds + min(l16, (int)g.M - 1) * stride + 64 * (b + i) + 16 * lg);
                    } else {
                        const long c = 64L * (b + i) + 16 * lg;
                        if (c < g.code_row)
                            x = *reinterpret_cast<const i32x4*>(g.a + min(m0 + 16 * t + l16, g.M - 1) * g.code_row + c);
                    }
#pragma unroll
                    for (int r = 0; r < NR; ++r) acc[t][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(cur[r], x, acc[t][r], 0, 0, 0);
                }
        }
    }
    __syncthreads();   // the codes are read
    int* sums = reinterpret_cast<int*>(lds);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int z = 0; z < NR; ++z)
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[(((wave * MT + t) * NR + z) * 16 + l16) * 17 + 4 * lg + r] = acc[t][z][r];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * NR * 256; i += 512) {
        const int tz = i >> 8, t = tz / NR, m = (i >> 4) & 15, n = n0 + 16 * (tz % NR) + (i & 15);
        const long row = m0 + 16 * t + m;
        int s = 0;
#pragma unroll
        for (int z = 0; z < 8; ++z) s += sums[((z * MT * NR + tz) * 16 + m) * 17 + (i & 15)];
        if (row < g.M && n < g.N)
            reinterpret_cast<T*>(g.y)[row * g.y_row + n] =
                (T)((double)s * (double)(FUSED ? sc[m] : g.as[row]) * (double)g.wsc[n]);
    }
}

static hipError_t int8_quantize(const void* x, long x_row, signed char* codes, long code_row, float* scales, long rows,
                                int cols, tm_dtype dtype, hipStream_t st) {
    if (rows >= 1L << 24) return hipErrorInvalidValue;   // a launch has fewer than 2^32 threads along an axis
    const bool vec = (uintptr_t)x % 16 == 0 && x_row % (dtype == TM_F32 ? 4 : 8) == 0;
    auto go = [&](auto t, auto v) {
        typedef decltype(t) T;
        launch_k((int8_quantize_kernel<T, decltype(v)::value>), dim3((unsigned)rows), dim3(256), 0, st,
                 static_cast<const T*>(x), x_row, codes, code_row, scales, cols);
        return hipGetLastError();
    };
    return timed_layer(st, [&] {
        if (dtype == TM_F32) return vec ? go(0.f, std::true_type{}) : go(0.f, std::false_type{});
        return vec ? go((bf16)0.f, std::true_type{}) : go((bf16)0.f, std::false_type{});
    });
}

template <class T, int BM, int BN, int WM, int WN> static hipError_t int8_tile(Int8Args g, hipStream_t st) {
    const long mt = (g.M + BM - 1) / BM, nt = (g.N + BN - 1L) / BN;
    if (mt * nt * (WM * WN) >= 1L << 26) return hipErrorInvalidValue;   // a launch has fewer than 2^32 threads
    g.mtiles = (int)mt;
    g.ntiles = (int)nt;
    const size_t bytes = 2 * (BM + BN) * 128;
    static std::atomic<unsigned long long> done{0};
    const hipError_t e = lds_limit((const void*)int8_tile_kernel<T, BM, BN, WM, WN>, bytes, done);
    if (e != hipSuccess) return e;
    return timed_layer(st, [&] {
        launch_k((int8_tile_kernel<T, BM, BN, WM, WN>), dim3((unsigned)(mt * nt)), dim3(WM * WN * 64), bytes, st, g);
        return hipGetLastError();
    });
}

template <class T, int MT, int NR, bool FUSED> static hipError_t int8_thin_run(const Int8Args& g, hipStream_t st) {
    const long nb = (g.N + 16L * NR - 1) / (16 * NR), mb = (g.M + 16 * MT - 1) / (16 * MT);
    if (nb >= 1L << 23 || mb > 65535) return hipErrorInvalidValue;
    const size_t sums = 8 * MT * NR * 16 * 17 * 4, codes = FUSED ? (size_t)g.M * ((g.code_row + 63) / 64 * 64 + 16) : 0;
    const size_t bytes = sums > codes ? sums : codes;
    static std::atomic<unsigned long long> done{0};
    const hipError_t e = lds_limit((const void*)int8_thin_kernel<T, MT, NR, FUSED>, bytes, done);
    if (e != hipSuccess) return e;
    return timed_layer(st, [&] {
        launch_k((int8_thin_kernel<T, MT, NR, FUSED>), dim3((unsigned)nb, (unsigned)mb), dim3(512), bytes, st, g);
        return hipGetLastError();
    });
}
template <class T, int MT, bool FUSED> static hipError_t int8_thin(const Int8Args& g, hipStream_t st) {
    if constexpr (FUSED)
        if (g.N > 16 * 256) return int8_thin_run<T, MT, 2, FUSED>(g, st);
    return int8_thin_run<T, MT, 1, FUSED>(g, st);
}

// A call whose workgroups make the codes themselves: as many rows as an
// instruction takes, in half a compute unit's LDS (8 rows of 4096 to 6144: 11 us
// a pass against 14 with the codes from a launch of their own).
static bool int8_fused(long rows, long code_row) { return rows <= 16 && rows * ((code_row + 63) / 64 * 64 + 16) <= 72 * 1024; }

template <class T> static hipError_t int8_matmul_t(const Int8Args& g, hipStream_t st) {
    // Large tiles where they fill the chip, us by tiles of 256 / 128 / 64 / few rows:
    //   4096 x 4096 -> 4096: 81 / 89 / 114 / 592;  2048 x 4096 -> 4096: 76 / 47 / 56 / 299;
    //   4096 x 1024 -> 2048: 38 / 24 / 24 / 100;   1024 x 4096 -> 4096: 73 / 38 / 30 / 152;
    //   256 x 4096 -> 4096: 70 / 34 / 17 / 41;     64 x 4096 -> 4096: 57 / 33 / 16 / 15;
    //   300 x 1024 -> 1024: 36 / 18 / 8 / 8;       100 x 8192 -> 300: 106 / 54 / 25 / 21.
    auto tiles = [&](long b) { return (g.M + b - 1) / b * ((g.N + b - 1) / b); };
    if (tiles(256) >= 200) return int8_tile<T, 256, 256, 2, 4>(g, st);
    if (tiles(128) >= 400) return int8_tile<T, 128, 128, 2, 2>(g, st);
    if (g.M > 64 && tiles(64) >= 128) return int8_tile<T, 64, 64, 2, 2>(g, st);
    if (g.M <= 16) return int8_thin<T, 1, false>(g, st);
    if (g.M <= 32) return int8_thin<T, 2, false>(g, st);
    return int8_thin<T, 4, false>(g, st);
}

static hipError_t int8_matmul(Int8Args g, tm_dtype dtype, hipStream_t st) {
    const size_t es = dtype == TM_F32 ? 4 : 2;
    g.vec = (uintptr_t)g.y % (4 * es) == 0 && g.y_row % 4 == 0;
    return dtype == TM_F32 ? int8_matmul_t<float>(g, st) : int8_matmul_t<bf16>(g, st);
}

static tm_status int8_status(hipError_t e) {
    return e == hipSuccess ? TM_OK : e == hipErrorInvalidValue ? TM_ERR_INVALID : TM_ERR_HIP;
}

constexpr int INT8_COLS = 131072;
constexpr long INT8_LIM = 1L << 40;

static bool int8_codes_ok(const void* codes, long code_row, int cols) {
    return codes && (uintptr_t)codes % 16 == 0 && code_row % 16 == 0 && code_row >= cols && code_row <= INT8_COLS;
}
static bool int8_rows_ok(const void* x, long row, long rows, long width, size_t es, bool apart) {
    return x && (uintptr_t)x % es == 0 && row >= 0 && row <= INT8_LIM && (double)rows * (double)row < 4e18 &&
           (!apart || rows <= 1 || row >= width);
}

}  // namespace tmk

using namespace tmk;

extern "C" {

tm_status tm_int8_quantize(const void* x, long x_row, signed char* codes, long code_row, float* scales, long rows,
                           int cols, tm_dtype dtype, void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (rows < 0 || cols < 1 || cols > INT8_COLS) return TM_ERR_INVALID;
    if (rows == 0) return TM_OK;
    if (rows >= 1L << 31 || !int8_rows_ok(x, x_row, rows, cols, dtype == TM_F32 ? 4 : 2, false) ||
        !int8_codes_ok(codes, code_row, cols) || !scales || (uintptr_t)scales % 4)
        return TM_ERR_INVALID;
    return int8_status(int8_quantize(x, x_row, codes, code_row, scales, rows, cols, dtype, static_cast<hipStream_t>(stream)));
}

tm_status tm_int8_matmul(const signed char* a, const float* a_scales, const signed char* w, const float* w_scales,
                         long code_row, void* y, long y_row, long rows, int outs, int cols, tm_dtype dtype,
                         void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (rows < 0 || rows >= 1L << 31 || outs < 0 || cols < 1 || cols > INT8_COLS) return TM_ERR_INVALID;
    if (rows == 0 || outs == 0) return TM_OK;
    if (!int8_codes_ok(a, code_row, cols) || !int8_codes_ok(w, code_row, cols) || !a_scales || (uintptr_t)a_scales % 4 ||
        !w_scales || (uintptr_t)w_scales % 4 || !int8_rows_ok(y, y_row, rows, outs, dtype == TM_F32 ? 4 : 2, true))
        return TM_ERR_INVALID;
    return int8_status(int8_matmul(Int8Args{a, a_scales, w, w_scales, y, code_row, y_row, rows, outs}, dtype,
                                   static_cast<hipStream_t>(stream)));
}

size_t tm_int8_workspace_bytes(long rows, int cols) {
    if (rows < 0 || rows >= 1L << 31 || cols < 1 || cols > INT8_COLS) return 0;
    const size_t wide = (size_t)(cols + 15) / 16 * 16;
    const size_t bytes = ((size_t)rows * wide + 255) / 256 * 256 + ((size_t)rows * 4 + 255) / 256 * 256;
    return bytes < 256 ? 256 : bytes;
}

tm_status tm_int8_linear(const void* x, long x_row, const signed char* w, const float* w_scales, long code_row,
                         void* y, long y_row, long rows, int outs, int cols, tm_dtype dtype, void* workspace,
                         void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (rows < 0 || rows >= 1L << 31 || outs < 0 || cols < 1 || cols > INT8_COLS) return TM_ERR_INVALID;
    if (rows == 0 || outs == 0) return TM_OK;
    const size_t es = dtype == TM_F32 ? 4 : 2;
    // the rows' codes are as wide as w's
    if (code_row != (cols + 15L) / 16 * 16 || !int8_rows_ok(x, x_row, rows, cols, es, false) ||
        !int8_codes_ok(w, code_row, cols) || !w_scales || (uintptr_t)w_scales % 4 ||
        !int8_rows_ok(y, y_row, rows, outs, es, true) || !workspace || (uintptr_t)workspace % 256)
        return TM_ERR_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (int8_fused(rows, code_row)) {
        Int8Args g{nullptr, nullptr, w, w_scales, y, code_row, y_row, rows, outs};
        g.x = x;
        g.x_row = x_row;
        g.cols = cols;
        g.xvec = (uintptr_t)x % 16 == 0 && x_row % (16 / (long)es) == 0;
        return int8_status(dtype == TM_F32 ? int8_thin<float, 1, true>(g, st) : int8_thin<bf16, 1, true>(g, st));
    }
    signed char* codes = static_cast<signed char*>(workspace);
    float* scales = reinterpret_cast<float*>(codes + ((size_t)rows * code_row + 255) / 256 * 256);
    const hipError_t e = int8_quantize(x, x_row, codes, code_row, scales, rows, cols, dtype, st);
    if (e != hipSuccess) return int8_status(e);
    return int8_status(int8_matmul(Int8Args{codes, scales, w, w_scales, y, code_row, y_row, rows, outs}, dtype, st));
}

}  // extern "C"
