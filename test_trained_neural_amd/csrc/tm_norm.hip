// Norms of queries and keys for each head with their rotary positions, and
// the gradients of both (include/tm_layer.h, tm_head_norm).
//
//   y  = R(p) (w * u),  u = x r,  r = 1 / sqrt(mean x^2 + eps)
//   dn = R(-p) dy,  dw = sum dn * u,  dx = r (e - u mean(e * u)),  e = w * dn
//
// A head vector belongs to a group of lanes of one wave and stays in their
// registers between the sum over its elements and the rotation, so x is read
// once and y written once.  As in the rotation by itself, a lane forms the
// sines and cosines of its pairs once for a token (fp64 angle, reduced to
// half turns) and takes several heads through them.
#include <math.h>

#include "../../include/tm_layer.h"
#include "tm_device.h"

namespace tmk {

struct NormArgs {
    const void* x;
    void* y;               // y; dx in the backward
    const void* dy;
    long xb, xt, yb, yt, gb, gt;   // elements between batch entries and between tokens (g: dy)
    const float* wq;
    const float* wk;
    float* part;           // backward: [groups of tokens][2][d] partial sums of dw
    const int* pos;
    const double* freq;
    float scale, eps;
    int per_token;
    int B, T, H, K, d, r;  // heads, key heads, head width, rotated width
    int units, rot_units;  // work units of a head vector, those of them that are rotated
    int hgroup;            // heads per thread
    int tokens;            // backward: tokens (of all entries) per group of lanes
};

template <bool STREAM, class V> __device__ __forceinline__ V nget(const V* p) {
    if constexpr (STREAM) {
        typedef unsigned U __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(V, __builtin_nontemporal_load(reinterpret_cast<const U*>(p)));
    } else {
        return *p;
    }
}
template <bool STREAM, class V> __device__ __forceinline__ void nput(V* p, V v) {
    if constexpr (STREAM) {
        typedef unsigned U __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(__builtin_bit_cast(U, v), reinterpret_cast<U*>(p));
    } else {
        *p = v;
    }
}

// Workgroups from which a call's heads are divided no further: the sines and
// cosines of a token are formed again for every division.  us with half as
// many / these / twice as many.  Forward: 2048 tokens of 40 heads of 128 15.3 /
// 15.5 / 16.7, of 20 heads of 96 in fp32 11.4 / 9.5 / 10.  Past the caches: 2 x
// 8192 tokens of 40 heads of 128, interleaved pairs 80 / 77 / 89, half layout
// 74 / 90 / 99, not rotated 86 / 83 / 94, 2 x 4096 in fp32 109 / 120 / 130.
// Gradients: 4 x 2047 tokens of 20 heads of 96 47 / 36 / 45, 4 x 2048 in fp32
// 92 / 92 / 129, of 20 heads of 128, interleaved, 41 / 41 / 37, 2 x 2048 tokens
// of 10 heads of 256 33 / 31 / 45.
constexpr int NORM_WGS = 1024, NORM_STREAM_WGS = 4096, NORM_BACK_WGS = 512;

// A unit of a head vector.  Half layout: V pairs, elements c .. c + V - 1 and
// r / 2 further on; interleaved: V / 2 pairs (one where V is 1); behind the
// rotated elements V elements.
template <int V, bool HALF> struct Unit {
    static constexpr int E = HALF ? 2 * V : (V > 1 ? V : 2);   // elements
    static constexpr int NP = E / 2;                            // pairs
};

template <class T, int V, bool HALF, bool STREAM>
__device__ __forceinline__ void load_unit(const T* x, int u, const NormArgs& a, float* e) {
    constexpr int E = Unit<V, HALF>::E;
    struct __align__(sizeof(T) * V) Vec { T e[V]; };
    if (u < a.rot_units) {
        if constexpr (HALF) {
            const Vec lo = nget<STREAM>(reinterpret_cast<const Vec*>(x + u * V));
            const Vec hi = nget<STREAM>(reinterpret_cast<const Vec*>(x + a.r / 2 + u * V));
#pragma unroll
            for (int j = 0; j < V; ++j) {
                e[j] = (float)lo.e[j];
                e[V + j] = (float)hi.e[j];
            }
        } else if constexpr (V > 1) {
            const Vec v = nget<STREAM>(reinterpret_cast<const Vec*>(x + u * V));
#pragma unroll
            for (int j = 0; j < V; ++j) e[j] = (float)v.e[j];
        } else {
            e[0] = (float)x[2 * u];
            e[1] = (float)x[2 * u + 1];
        }
    } else {
        const Vec v = nget<STREAM>(reinterpret_cast<const Vec*>(x + a.r + (u - a.rot_units) * V));
#pragma unroll
        for (int j = 0; j < E; ++j) e[j] = j < V ? (float)v.e[j < V ? j : 0] : 0.f;
    }
}
template <class T, int V, bool HALF, bool STREAM>
__device__ __forceinline__ void store_unit(T* y, int u, const NormArgs& a, const float* e) {
    struct __align__(sizeof(T) * V) Vec { T e[V]; };
    if (u < a.rot_units) {
        if constexpr (HALF) {
            Vec lo, hi;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                lo.e[j] = (T)e[j];
                hi.e[j] = (T)e[V + j];
            }
            nput<STREAM>(reinterpret_cast<Vec*>(y + u * V), lo);
            nput<STREAM>(reinterpret_cast<Vec*>(y + a.r / 2 + u * V), hi);
        } else if constexpr (V > 1) {
            Vec v;
#pragma unroll
            for (int j = 0; j < V; ++j) v.e[j] = (T)e[j];
            nput<STREAM>(reinterpret_cast<Vec*>(y + u * V), v);
        } else {
            y[2 * u] = (T)e[0];
            y[2 * u + 1] = (T)e[1];
        }
    } else {
        Vec v;
#pragma unroll
        for (int j = 0; j < V; ++j) v.e[j] = (T)e[j];
        nput<STREAM>(reinterpret_cast<Vec*>(y + a.r + (u - a.rot_units) * V), v);
    }
}

// Element e of unit u, and whether it stands for one (a unit behind the
// rotated elements holds V of E).
template <int V, bool HALF> __device__ __forceinline__ int element(int u, int e, const NormArgs& a) {
    if (u >= a.rot_units) return e < V ? a.r + (u - a.rot_units) * V + e : -1;
    if constexpr (HALF) return e < V ? u * V + e : a.r / 2 + u * V + e - V;
    return u * Unit<V, HALF>::E + e;
}

// Sines and cosines of a unit's pairs at a token, in the order of the pairs.
template <int V, bool HALF>
__device__ __forceinline__ void angles(int u, double p, const NormArgs& a, float* cs, float* sn) {
    constexpr int NP = Unit<V, HALF>::NP;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        cs[j] = 1.f;
        sn[j] = 0.f;
        if (u < a.rot_units) {
            // in half turns: angle / pi, minus the nearest even whole number
            double w = p * a.freq[u * NP + j] * 0.31830988618379067154;
            w -= 2.0 * rint(0.5 * w);
            float s, c;
            sincospif((float)w, &s, &c);
            cs[j] = c * a.scale;
            sn[j] = s * a.scale;
        }
    }
}

// Turns a unit's pairs; back: by the negative angle.
template <int V, bool HALF, bool BACK>
__device__ __forceinline__ void turn(float* e, const float* cs, const float* sn) {
    constexpr int NP = Unit<V, HALF>::NP;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        float& a = e[HALF ? j : 2 * j];
        float& b = e[HALF ? NP + j : 2 * j + 1];
        const float s = BACK ? -sn[j] : sn[j], a0 = a, b0 = b;
        if constexpr (BACK && V >= 4) {   // the units whose kernel has a second form, past the caches
            a = fmaf(a0, cs[j], -(b0 * s));
            b = fmaf(a0, s, b0 * cs[j]);
        } else {
            a = a0 * cs[j] - b0 * s;
            b = a0 * s + b0 * cs[j];
        }
    }
}

template <int LG> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = LG / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// U units a lane, LG lanes a head vector.
template <class T, int V, bool HALF, int U, bool STREAM>
__global__ __launch_bounds__(256) void head_norm_kernel(NormArgs a, int lg) {
    constexpr int E = Unit<V, HALF>::E, NP = Unit<V, HALF>::NP, AHEAD = U == 1 ? 2 : 1;
    const int lane = threadIdx.x & (lg - 1);
    const long bt = (long)blockIdx.x * (256 / lg) + threadIdx.x / lg;
    if (bt >= (long)a.B * a.T) return;   // a whole group of lanes
    const int t = (int)(bt % a.T), b = (int)(bt / a.T);
    const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb + t * a.xt;
    T* y = reinterpret_cast<T*>(a.y) + b * a.yb + t * a.yt;
    const double p = a.rot_units ? (double)a.pos[a.per_token ? bt : b] + (a.per_token ? 0 : t) : 0.0;
    float cs[U][NP], sn[U][NP], w[U][E];
#pragma unroll
    for (int i = 0; i < U; ++i) angles<V, HALF>(lane + i * lg, p, a, cs[i], sn[i]);
    const int h0 = blockIdx.y * a.hgroup, h1 = min(a.H + a.K, h0 + a.hgroup);
    const float inv_d = 1.f / (float)a.d;
    for (int part = 0; part < 2; ++part) {   // queries, keys
        const int from = part ? max(h0, a.H) : h0, to = part ? h1 : min(h1, a.H);
        if (from >= to) continue;
        const float* wp = part ? a.wk : a.wq;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int u = lane + i * lg, c = u < a.units ? element<V, HALF>(u, j, a) : -1;
                w[i][j] = wp && c >= 0 ? wp[c] : 1.f;
            }
        for (int h = from; h < to; h += AHEAD) {   // AHEAD heads at a time: their loads are under way together
            float e[AHEAD][U][E], sum[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int u = lane + i * lg;
                    if (u < a.units) load_unit<T, V, HALF, STREAM>(x + (long)min(h + k, to - 1) * a.d, u, a, e[k][i]);
                }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                sum[k] = 0.f;
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (lane + i * lg < a.units)
#pragma unroll
                        for (int j = 0; j < E; ++j) sum[k] += e[k][i][j] * e[k][i][j];
            }
            for (int m = lg >> 1; m > 0; m >>= 1)
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) sum[k] += __shfl_xor(sum[k], m, 64);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float r = 1.f / sqrtf(sum[k] * inv_d + a.eps);
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int u = lane + i * lg;
                    if (u < a.units && h + k < to) {
#pragma unroll
                        for (int j = 0; j < E; ++j) e[k][i][j] *= r * w[i][j];
                        if (u < a.rot_units) turn<V, HALF, false>(e[k][i], cs[i], sn[i]);
                        store_unit<T, V, HALF, STREAM>(y + (long)(h + k) * a.d, u, a, e[k][i]);
                    }
                }
            }
        }
    }
}

// The backward: a group of lanes takes some heads (blockIdx.y) of a.tokens
// tokens, so that the sums of dw stay in its registers; a workgroup adds its
// groups' sums through LDS in their order and writes one partial sum.  Its
// sums of products are written as the multiply-adds they are: left to the
// compiler, which of two products is rounded by itself differed between the
// forms of one kernel, and with it a token's bits by the size of its call.
template <class T, int V, bool HALF, int U, bool STREAM>
__global__ __launch_bounds__(256) void head_norm_backward_kernel(NormArgs a, int lg) {
    constexpr int E = Unit<V, HALF>::E, NP = Unit<V, HALF>::NP, AHEAD = U == 1 ? 2 : 1;
    extern __shared__ float red[];   // [groups][d]
    const int lane = threadIdx.x & (lg - 1), group = threadIdx.x / lg, groups = 256 / lg;
    const long first = ((long)blockIdx.x * groups + group) * a.tokens, total = (long)a.B * a.T;
    const long last = min(total, first + a.tokens);
    const float inv_d = 1.f / (float)a.d;
    for (int part = 0; part < (a.K ? 2 : 1); ++part) {   // queries, keys
        const int h0 = blockIdx.y * a.hgroup, h1 = min(a.H + a.K, h0 + a.hgroup);
        const int from = part ? max(h0, a.H) : h0, to = part ? h1 : min(h1, a.H);
        const float* wp = part ? a.wk : a.wq;
        float w[U][E], dw[U][E];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int u = lane + i * lg, c = u < a.units ? element<V, HALF>(u, j, a) : -1;
                w[i][j] = wp && c >= 0 ? wp[c] : 1.f;
                dw[i][j] = 0.f;
            }
        for (long bt = first; bt < last && from < to; ++bt) {
            const int t = (int)(bt % a.T), b = (int)(bt / a.T);
            const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb + t * a.xt;
            const T* g = reinterpret_cast<const T*>(a.dy) + b * a.gb + t * a.gt;
            T* dx = reinterpret_cast<T*>(a.y) + b * a.yb + t * a.yt;
            const double p = a.rot_units ? (double)a.pos[a.per_token ? bt : b] + (a.per_token ? 0 : t) : 0.0;
            float cs[U][NP], sn[U][NP];
#pragma unroll
            for (int i = 0; i < U; ++i) angles<V, HALF>(lane + i * lg, p, a, cs[i], sn[i]);
            for (int h = from; h < to; h += AHEAD) {
                float e[AHEAD][U][E], n[AHEAD][U][E], sum[AHEAD], dot[AHEAD];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k)
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int u = lane + i * lg;
                        const long at = (long)min(h + k, to - 1) * a.d;
                        if (u < a.units) {
                            load_unit<T, V, HALF, STREAM>(x + at, u, a, e[k][i]);
                            load_unit<T, V, HALF, STREAM>(g + at, u, a, n[k][i]);
                        }
                    }
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    sum[k] = dot[k] = 0.f;
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int u = lane + i * lg;
                        if (u < a.units) {
                            if (u < a.rot_units) turn<V, HALF, true>(n[k][i], cs[i], sn[i]);
#pragma unroll
                            for (int j = 0; j < E; ++j) {
                                sum[k] = fmaf(e[k][i][j], e[k][i][j], sum[k]);
                                dot[k] = fmaf(e[k][i][j] * n[k][i][j], w[i][j], dot[k]);
                            }
                        }
                    }
                }
                for (int m = lg >> 1; m > 0; m >>= 1)
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k) {
                        sum[k] += __shfl_xor(sum[k], m, 64);
                        dot[k] += __shfl_xor(dot[k], m, 64);
                    }
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const float r = 1.f / sqrtf(fmaf(sum[k], inv_d, a.eps)), mean = dot[k] * r * inv_d;
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int u = lane + i * lg;
                        if (u < a.units && h + k < to) {
#pragma unroll
                            for (int j = 0; j < E; ++j) {
                                const float unit = e[k][i][j] * r;
                                dw[i][j] = fmaf(n[k][i][j], unit, dw[i][j]);
                                e[k][i][j] = r * fmaf(n[k][i][j], w[i][j], -(unit * mean));
                            }
                            store_unit<T, V, HALF, STREAM>(dx + (long)(h + k) * a.d, u, a, e[k][i]);
                        }
                    }
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int u = lane + i * lg, c = u < a.units ? element<V, HALF>(u, j, a) : -1;
                if (c >= 0) red[group * a.d + c] = dw[i][j];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += 256) {
            float s = 0.f;
            for (int k = 0; k < groups; ++k) s += red[k * a.d + c];
            a.part[(((long)blockIdx.y * gridDim.x + blockIdx.x) * 2 + part) * a.d + c] = s;
        }
    }
}

// dw of queries (blockIdx.y 0) and keys (1): the workgroups' partial sums in
// a fixed order, 8 elements a workgroup, 128 sums of each side by side.
__global__ __launch_bounds__(1024) void head_norm_dw_kernel(const float* part, int n, int d, float* dwq, float* dwk) {
    __shared__ float red[1024];
    const int c = blockIdx.x * 8 + (threadIdx.x & 7), k = threadIdx.x >> 3;
    float* dw = blockIdx.y ? dwk : dwq;
    float s = 0.f;
    if (c < d && dw)
#pragma unroll 4
        for (int i = k; i < n; i += 128) s += part[((long)i * 2 + blockIdx.y) * d + c];
    red[threadIdx.x] = s;
#pragma unroll
    for (int m = 64; m > 0; m >>= 1) {
        __syncthreads();
        if (k < m) red[threadIdx.x] += red[threadIdx.x + 8 * m];
    }
    if (k == 0 && c < d && dw) dw[c] = red[threadIdx.x];
}

__global__ void head_norm_zero_kernel(int d, float* dwq, float* dwk) {
    for (int c = threadIdx.x; c < d; c += 256) {
        if (dwq) dwq[c] = 0.f;
        if (dwk) dwk[c] = 0.f;
    }
}

static int pow2_up(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// Workgroups of the backward at most, each with a partial sum.
constexpr int NORM_PARTS = 2048;

template <class T, int V, bool HALF, int U>
static hipError_t norm_launch(NormArgs a, int lg, bool back, int* parts, hipStream_t st) {
    const long tokens = (long)a.B * a.T;
    const int per = 256 / lg;
    const bool stream = V * sizeof(T) == 16 &&
                        tokens * (a.H + a.K) * a.d * (long)sizeof(T) * (back ? 3 : 2) > 256L << 20;
    if (back) {
        const long groups = (tokens + per - 1) / per;
        a.tokens = (int)((groups + 1023) / 1024);
        const long blocks = (tokens + (long)per * a.tokens - 1) / ((long)per * a.tokens);
        int parts_y = 1;
        while (parts_y < a.H + a.K && blocks * parts_y < NORM_BACK_WGS) parts_y *= 2;   // at most NORM_PARTS with the last doubling
        a.hgroup = (a.H + a.K + parts_y - 1) / parts_y;
        parts_y = (a.H + a.K + a.hgroup - 1) / a.hgroup;
        const dim3 grid((unsigned)blocks, (unsigned)parts_y);
        *parts = (int)(blocks * parts_y);
        const size_t lds = (size_t)per * a.d * sizeof(float);
        if constexpr (V * sizeof(T) == 16) {
            if (stream) {
                launch_k(head_norm_backward_kernel<T, V, HALF, U, true>, grid, dim3(256), lds, st, a, lg);
                return hipGetLastError();
            }
        }
        launch_k(head_norm_backward_kernel<T, V, HALF, U, false>, grid, dim3(256), lds, st, a, lg);
        return hipGetLastError();
    }
    const long blocks = (tokens + per - 1) / per;
    if (blocks >= 1L << 24) return hipErrorInvalidValue;   // a launch has fewer than 2^32 threads along an axis
    const int heads = a.H + a.K;
    int groups = 1;
    while (groups < heads && blocks * groups < (stream ? NORM_STREAM_WGS : NORM_WGS)) groups *= 2;
    a.hgroup = (heads + groups - 1) / groups;
    const dim3 grid((unsigned)blocks, (unsigned)((heads + a.hgroup - 1) / a.hgroup));
    if constexpr (V * sizeof(T) == 16) {
        if (stream) {
            launch_k(head_norm_kernel<T, V, HALF, U, true>, grid, dim3(256), 0, st, a, lg);
            return hipGetLastError();
        }
    }
    launch_k(head_norm_kernel<T, V, HALF, U, false>, grid, dim3(256), 0, st, a, lg);
    return hipGetLastError();
}

template <class T, int V, bool HALF>
static hipError_t norm_units(NormArgs a, bool back, int* parts, hipStream_t st) {
    a.rot_units = HALF || V == 1 ? a.r / 2 / V : a.r / V;
    a.units = a.rot_units + (a.d - a.r) / V;
    const int lg = a.units >= 64 ? 64 : pow2_up(a.units), u = (a.units + lg - 1) / lg;
    if (u == 1) return norm_launch<T, V, HALF, 1>(a, lg, back, parts, st);
    if (u <= 4) return norm_launch<T, V, HALF, 4>(a, lg, back, parts, st);
    if constexpr (V <= 2) return norm_launch<T, V, HALF, 16>(a, lg, back, parts, st);
    return hipErrorInvalidValue;   // not reached: 1024 elements are 4 units of 4 a lane
}

template <class T>
static hipError_t norm_dispatch(const NormArgs& a, bool half, bool back, int* parts, hipStream_t st) {
    // the widest unit that the widths, distances and addresses allow
    auto fits = [&](int v) {
        const size_t al = v * sizeof(T);
        return (uintptr_t)a.x % al == 0 && (uintptr_t)a.y % al == 0 && (!back || (uintptr_t)a.dy % al == 0) &&
               a.xb % v == 0 && a.xt % v == 0 && a.yb % v == 0 && a.yt % v == 0 && a.gb % v == 0 && a.gt % v == 0 &&
               a.d % v == 0 && a.r % v == 0 && (!half || a.r / 2 % v == 0);
    };
    auto go = [&](auto v) {
        constexpr int V = decltype(v)::value;
        return half ? norm_units<T, V, true>(a, back, parts, st) : norm_units<T, V, false>(a, back, parts, st);
    };
    if constexpr (sizeof(T) == 2)
        if (fits(8)) return go(std::integral_constant<int, 8>{});
    if (fits(4)) return go(std::integral_constant<int, 4>{});
    if (fits(2)) return go(std::integral_constant<int, 2>{});
    return go(std::integral_constant<int, 1>{});
}

// The rows of one array must not run into each other.
static bool rows_apart(long batch_d, long token_d, int batch, int n_tokens, long row) {
    const long yb = batch > 1 ? batch_d : 0, yt = n_tokens > 1 ? token_d : 0;
    const bool apart = (batch <= 1 || yb >= (n_tokens - 1) * yt + row) && (n_tokens <= 1 || yt >= row);
    const bool swapped = (n_tokens <= 1 || yt >= (batch - 1) * yb + row) && (batch <= 1 || yb >= row);
    return apart || swapped;
}

static tm_status norm_check(const NormArgs& a, bool back, double eps, double result_scale, tm_rope_layout layout,
                            tm_dtype dtype) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (layout != TM_ROPE_HALF && layout != TM_ROPE_INTERLEAVED) return TM_ERR_INVALID;
    if (a.B < 0 || a.T < 0 || a.H <= 0 || a.K < 0 || a.H > 65535 - a.K || a.d <= 0 || a.d > 1024 || a.r < 0 ||
        a.r % 2 != 0 || a.r > a.d || !isfinite(result_scale) || !(eps >= 0.0) || !isfinite((float)eps))
        return TM_ERR_INVALID;
    if (a.B == 0 || a.T == 0) return TM_OK;
    const long row = (long)(a.H + a.K) * a.d, lim = 1L << 40;
    const size_t es = dtype == TM_F32 ? 4 : 2;
    if ((long)a.B * a.T > lim / row) return TM_ERR_INVALID;
    if (!a.x || !a.y || (uintptr_t)a.x % es || (uintptr_t)a.y % es || (uintptr_t)a.wq % 4 || (uintptr_t)a.wk % 4 ||
        (back && (!a.dy || (uintptr_t)a.dy % es)))
        return TM_ERR_INVALID;
    if (a.r && (!a.pos || !a.freq || (uintptr_t)a.pos % 4 || (uintptr_t)a.freq % 8)) return TM_ERR_INVALID;
    const long dist[6] = {a.xb, a.xt, a.yb, a.yt, a.gb, a.gt};
    for (int i = 0; i < 6; ++i)
        if (dist[i] < 0 || dist[i] > lim || (double)(i % 2 ? a.T : a.B) * (double)dist[i] > 4e18) return TM_ERR_INVALID;
    if (!rows_apart(a.yb, a.yt, a.B, a.T, row)) return TM_ERR_INVALID;
    if (a.x == a.y && (a.xb != a.yb || a.xt != a.yt)) return TM_ERR_INVALID;
    if (back && a.dy == a.y && (a.gb != a.yb || a.gt != a.yt)) return TM_ERR_INVALID;
    return TM_OK;
}

static tm_status norm_status(hipError_t e) {
    return e == hipSuccess ? TM_OK : e == hipErrorInvalidValue ? TM_ERR_INVALID : TM_ERR_HIP;
}

}  // namespace tmk

using namespace tmk;

extern "C" {

tm_status tm_head_norm(const void* x, long x_batch, long x_token, void* y, long y_batch, long y_token,
                       const float* w_q, const float* w_k, double eps, const int* positions, int per_token,
                       const double* freq, double result_scale, int batch, int n_tokens, int heads, int kv_heads,
                       int head_dim, int rot_dim, tm_rope_layout layout, tm_dtype dtype, void* stream) {
    NormArgs a{};
    a.x = x; a.y = y; a.xb = x_batch; a.xt = x_token; a.yb = y_batch; a.yt = y_token;
    a.wq = w_q; a.wk = w_k; a.pos = positions; a.freq = freq; a.per_token = per_token != 0;
    a.scale = (float)result_scale; a.eps = (float)eps;
    a.B = batch; a.T = n_tokens; a.H = heads; a.K = kv_heads; a.d = head_dim; a.r = rot_dim;
    const tm_status s = norm_check(a, false, eps, result_scale, layout, dtype);
    if (s != TM_OK || batch == 0 || n_tokens == 0) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool half = layout == TM_ROPE_HALF;
    return norm_status(timed_layer(st, [&] {
        return dtype == TM_F32 ? norm_dispatch<float>(a, half, false, nullptr, st)
                               : norm_dispatch<bf16>(a, half, false, nullptr, st);
    }));
}

size_t tm_head_norm_workspace_bytes(int batch, int n_tokens, int heads, int kv_heads, int head_dim) {
    if (batch < 0 || n_tokens < 0 || heads <= 0 || kv_heads < 0 || head_dim <= 0 || head_dim > 1024) return 0;
    return (size_t)NORM_PARTS * 2 * head_dim * sizeof(float);
}

tm_status tm_head_norm_backward(const void* x, long x_batch, long x_token, const void* dy, long dy_batch,
                                long dy_token, void* dx, long dx_batch, long dx_token, const float* w_q,
                                const float* w_k, float* dw_q, float* dw_k, double eps, const int* positions,
                                int per_token, const double* freq, double result_scale, int batch, int n_tokens,
                                int heads, int kv_heads, int head_dim, int rot_dim, tm_rope_layout layout,
                                tm_dtype dtype, void* workspace, void* stream) {
    NormArgs a{};
    a.x = x; a.y = dx; a.dy = dy;
    a.xb = x_batch; a.xt = x_token; a.yb = dx_batch; a.yt = dx_token; a.gb = dy_batch; a.gt = dy_token;
    a.wq = w_q; a.wk = w_k; a.pos = positions; a.freq = freq; a.per_token = per_token != 0;
    a.scale = (float)result_scale; a.eps = (float)eps;
    a.B = batch; a.T = n_tokens; a.H = heads; a.K = kv_heads; a.d = head_dim; a.r = rot_dim;
    const tm_status s = norm_check(a, true, eps, result_scale, layout, dtype);
    if (s != TM_OK) return s;
    if ((uintptr_t)dw_q % 4 || (uintptr_t)dw_k % 4) return TM_ERR_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    float* dwk = kv_heads ? dw_k : nullptr;
    if (batch == 0 || n_tokens == 0) {
        if (!dw_q && !dwk) return TM_OK;
        return norm_status(timed_layer(st, [&] {
            launch_k(head_norm_zero_kernel, dim3(1), dim3(256), 0, st, head_dim, dw_q, dwk);
            return hipGetLastError();
        }));
    }
    if (!workspace || (uintptr_t)workspace % 256) return TM_ERR_INVALID;
    a.part = static_cast<float*>(workspace);
    int parts = 0;
    const bool half = layout == TM_ROPE_HALF;
    hipError_t e = timed_layer(st, [&] {
        return dtype == TM_F32 ? norm_dispatch<float>(a, half, true, &parts, st)
                               : norm_dispatch<bf16>(a, half, true, &parts, st);
    });
    if (e == hipSuccess && (dw_q || dwk))
        e = timed_layer(st, [&] {
            launch_k(head_norm_dw_kernel, dim3((head_dim + 7) / 8, kv_heads ? 2 : 1), dim3(1024), 0, st, a.part, parts,
                     head_dim, dw_q, dwk);
            return hipGetLastError();
        });
    return norm_status(e);
}

}  // extern "C"
