// Rotary positions (include/tm_attention.h, tm_rotary): each pair of a head
// vector turns by the angle position * freq[pair].
//
// The angle is one fp64 product, reduced to half turns in fp64 (position and
// frequency keep 53 bits: an fp32 product is off by a radian's sixteenth at
// position 10^6), and its sine and cosine are taken in fp32 of the reduced
// angle.  They belong to the token, not to the head, so a thread forms those
// of its pairs once and takes the pairs of several heads through them: the
// call is bound by reading x and writing y once (2 x 16384 tokens of 40 heads
// of 128, bf16: 130 us, 5.2 TB/s).
#include <math.h>

#include "../../include/tm_attention.h"
#include "tm_device.h"

namespace tmk {

struct RopeArgs {
    const void* x;
    void* y;
    long xb, xt, yb, yt;   // elements between batch entries and between tokens
    const int* pos;
    const double* freq;
    float scale;           // negative angles: `inverse`
    int per_token, inverse;
    int B, T, H, d, r;     // heads, head width, rotated width
    int units, hgroup;     // work units of a head vector; heads per thread
};

// 16-byte loads and stores past the caches (STREAM) or through them.
template <bool STREAM, class V> __device__ __forceinline__ V get(const V* p) {
    if constexpr (STREAM) {
        typedef unsigned U __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(V, __builtin_nontemporal_load(reinterpret_cast<const U*>(p)));
    } else {
        return *p;
    }
}
template <bool STREAM, class V> __device__ __forceinline__ void put(V* p, V v) {
    if constexpr (STREAM) {
        typedef unsigned U __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(__builtin_bit_cast(U, v), reinterpret_cast<U*>(p));
    } else {
        *p = v;
    }
}

// One unit is V consecutive elements (16 bytes at most).  Half layout: V
// pairs (V elements of each half); interleaved: V / 2 pairs (one where V is
// 1); the elements behind the rotated ones are units of their own, copied.
template <class T, int V, bool HALF, bool STREAM>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
    struct __align__(sizeof(T) * V) Vec { T e[V]; };
    constexpr int NP = HALF ? V : (V > 1 ? V / 2 : 1);
    const int rot_units = HALF || V == 1 ? a.r / 2 / V : a.r / V;
    const long total = (long)a.B * a.T * a.units;
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int u = (int)(i % a.units);
    const long bt = i / a.units;
    const int t = (int)(bt % a.T), b = (int)(bt / a.T);
    const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb + t * a.xt;
    T* y = reinterpret_cast<T*>(a.y) + b * a.yb + t * a.yt;
    const int h0 = blockIdx.y * a.hgroup, h1 = min(a.H, h0 + a.hgroup);
    if (u >= rot_units) {   // not rotated
        if (x == y) return;
        const int c = a.r + (u - rot_units) * V;
        for (int h = h0; h < h1; ++h)
            *reinterpret_cast<Vec*>(y + (long)h * a.d + c) = get<STREAM>(reinterpret_cast<const Vec*>(x + (long)h * a.d + c));
        return;
    }
    const double p = (double)a.pos[a.per_token ? bt : b] + (a.per_token ? 0 : t);
    float cs[NP], sn[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        // in half turns: angle / pi, minus the nearest even whole number
        double w = p * a.freq[HALF ? u * V + j : u * NP + j] * 0.31830988618379067154;
        w -= 2.0 * rint(0.5 * w);
        float s, c;
        sincospif((float)w, &s, &c);
        cs[j] = c * a.scale;
        sn[j] = (a.inverse ? -s : s) * a.scale;
    }
    if constexpr (HALF) {
        const int c = u * V;
#pragma unroll 4
        for (int h = h0; h < h1; ++h) {
            const Vec lo = get<STREAM>(reinterpret_cast<const Vec*>(x + (long)h * a.d + c));
            const Vec hi = get<STREAM>(reinterpret_cast<const Vec*>(x + (long)h * a.d + a.r / 2 + c));
            Vec ol, oh;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float p0 = (float)lo.e[j], p1 = (float)hi.e[j];
                ol.e[j] = (T)(p0 * cs[j] - p1 * sn[j]);
                oh.e[j] = (T)(p0 * sn[j] + p1 * cs[j]);
            }
            put<STREAM>(reinterpret_cast<Vec*>(y + (long)h * a.d + c), ol);
            put<STREAM>(reinterpret_cast<Vec*>(y + (long)h * a.d + a.r / 2 + c), oh);
        }
    } else {
        struct __align__(sizeof(T) * V) Pairs { T e[2 * NP]; };
        const int c = u * 2 * NP;
#pragma unroll 4
        for (int h = h0; h < h1; ++h) {
            const Pairs v = get<STREAM>(reinterpret_cast<const Pairs*>(x + (long)h * a.d + c));
            Pairs o;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const float p0 = (float)v.e[2 * j], p1 = (float)v.e[2 * j + 1];
                o.e[2 * j] = (T)(p0 * cs[j] - p1 * sn[j]);
                o.e[2 * j + 1] = (T)(p0 * sn[j] + p1 * cs[j]);
            }
            put<STREAM>(reinterpret_cast<Pairs*>(y + (long)h * a.d + c), o);
        }
    }
}

template <class T, int V>
static hipError_t launch_v(RopeArgs a, bool half, hipStream_t st) {
    a.units = (half || V == 1 ? a.r / 2 / V : a.r / V) + (a.d - a.r) / V;
    const long threads = (long)a.B * a.T * a.units;
    const long blocks = (threads + 255) / 256;
    if (blocks >= 1L << 24) return hipErrorInvalidValue;   // a launch has fewer than 2^32 threads along an axis
    // What does not fit the 256 MB of the last-level cache goes past the
    // caches, with more workgroups (2 x 16384 tokens of 40 heads of 128 in
    // bf16, 671 MB: 131 us against 138; 4 x 8192 of 10 heads of 64, 84 MB:
    // through the caches 17 us, past them 24).
    const bool stream = (long)a.B * a.T * a.H * a.d * (long)sizeof(T) * 2 > 256L << 20;
    // heads per thread: all of them where the tokens alone fill the chip,
    // fewer until about 4 workgroups (64 in a stream) stand on each of 256
    // compute units
    int groups = 1;
    while (groups < a.H && blocks * groups < (stream ? 16384 : 1024)) groups *= 2;
    a.hgroup = (a.H + groups - 1) / groups;
    const dim3 grid((unsigned)blocks, (unsigned)((a.H + a.hgroup - 1) / a.hgroup));
    if constexpr (V * sizeof(T) == 16) {
        if (stream) {
            if (half) launch_k(rope_kernel<T, V, true, true>, grid, dim3(256), 0, st, a);
            else launch_k(rope_kernel<T, V, false, true>, grid, dim3(256), 0, st, a);
            return hipGetLastError();
        }
    }
    if (half) launch_k(rope_kernel<T, V, true, false>, grid, dim3(256), 0, st, a);
    else launch_k(rope_kernel<T, V, false, false>, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <class T>
static hipError_t launch_t(const RopeArgs& a, bool half, hipStream_t st) {
    // the widest unit that the widths, distances and addresses allow
    auto fits = [&](int v) {
        const size_t al = v * sizeof(T);
        return (uintptr_t)a.x % al == 0 && (uintptr_t)a.y % al == 0 && a.xb % v == 0 && a.xt % v == 0 && a.yb % v == 0 &&
               a.yt % v == 0 && a.d % v == 0 && a.r % v == 0 && (!half || a.r / 2 % v == 0);
    };
    if constexpr (sizeof(T) == 2)
        if (fits(8)) return launch_v<T, 8>(a, half, st);
    if (fits(4)) return launch_v<T, 4>(a, half, st);
    if (fits(2)) return launch_v<T, 2>(a, half, st);
    return launch_v<T, 1>(a, half, st);
}

}  // namespace tmk

using namespace tmk;

extern "C" {

tm_status tm_rotary_frequencies(int rot_dim, double base, tm_rope_scaling scaling, double factor,
                                double original_len, double beta_fast, double beta_slow, double* freq,
                                double* result_scale) {
    if (!freq || !result_scale || rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0 || !(base > 1.0) ||
        !isfinite(base))
        return TM_ERR_INVALID;
    if (scaling != TM_ROPE_NONE && scaling != TM_ROPE_LINEAR && scaling != TM_ROPE_BASE && scaling != TM_ROPE_PARTS)
        return TM_ERR_INVALID;
    if (scaling != TM_ROPE_NONE && (!(factor > 0.0) || !isfinite(factor))) return TM_ERR_INVALID;
    if (scaling == TM_ROPE_BASE && rot_dim <= 2) return TM_ERR_INVALID;
    if (scaling == TM_ROPE_PARTS &&
        (!(original_len > 0.0) || !isfinite(original_len) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
         !isfinite(beta_fast)))
        return TM_ERR_INVALID;
    const int n = rot_dim / 2;
    const double r = rot_dim, pi = 3.14159265358979323846;
    if (scaling == TM_ROPE_BASE) {
        base *= pow(factor, r / (r - 2.0));
        if (!(base > 0.0) || !isfinite(base)) return TM_ERR_INVALID;
    }
    *result_scale = 1.0;
    double lo = 0.0, hi = 0.0;
    if (scaling == TM_ROPE_PARTS) {
        // pair index at which a pair turns `beta` times within original_len;
        // the ramp's ends may lie before the first pair and behind the last
        // (drawn in to them, it would divide a last pair that still turns
        // several times by the whole factor)
        auto at = [&](double beta) { return r * log(original_len / (beta * 2.0 * pi)) / (2.0 * log(base)); };
        lo = floor(at(beta_fast));
        hi = ceil(at(beta_slow));   // above lo: beta_fast > beta_slow
        if (factor > 1.0) *result_scale = 0.1 * log(factor) + 1.0;
    }
    for (int i = 0; i < n; ++i) {
        const double f = pow(base, -2.0 * i / r);
        if (scaling == TM_ROPE_LINEAR) {
            freq[i] = f / factor;
        } else if (scaling == TM_ROPE_PARTS) {
            const double share = fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
            freq[i] = f * (1.0 - share) + f / factor * share;
        } else {
            freq[i] = f;
        }
        if (!isfinite(freq[i])) return TM_ERR_INVALID;
    }
    return TM_OK;
}

tm_status tm_rotary(const void* x, long x_batch, long x_token, void* y, long y_batch, long y_token,
                    const int* positions, int per_token, const double* freq, double result_scale, int batch,
                    int n_tokens, int heads, int head_dim, int rot_dim, tm_rope_layout layout, int inverse,
                    tm_dtype dtype, void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (layout != TM_ROPE_HALF && layout != TM_ROPE_INTERLEAVED) return TM_ERR_INVALID;
    if (batch < 0 || n_tokens < 0 || heads <= 0 || heads > 65535 || head_dim <= 0 || head_dim > 1024 || rot_dim < 2 ||
        rot_dim % 2 != 0 || rot_dim > head_dim || !isfinite(result_scale))
        return TM_ERR_INVALID;
    if (batch == 0 || n_tokens == 0) return TM_OK;
    const long row = (long)heads * head_dim, lim = 1L << 40;
    const size_t es = dtype == TM_F32 ? 4 : 2;
    if ((long)batch * n_tokens > lim / row) return TM_ERR_INVALID;
    if (!x || !y || !positions || !freq || (uintptr_t)x % es || (uintptr_t)y % es || (uintptr_t)positions % 4 ||
        (uintptr_t)freq % 8)
        return TM_ERR_INVALID;
    // y's rows must not run into each other
    if (x_batch < 0 || x_token < 0 || y_batch < 0 || y_token < 0 || x_batch > lim || x_token > lim || y_batch > lim ||
        y_token > lim || (double)batch * (double)y_batch > 4e18 || (double)n_tokens * (double)y_token > 4e18)
        return TM_ERR_INVALID;
    const long yb = batch > 1 ? y_batch : 0, yt = n_tokens > 1 ? y_token : 0;
    const bool apart = (batch <= 1 || yb >= (n_tokens - 1) * yt + row) && (n_tokens <= 1 || yt >= row);
    const bool swapped = (n_tokens <= 1 || yt >= (batch - 1) * yb + row) && (batch <= 1 || yb >= row);
    if (!apart && !swapped) return TM_ERR_INVALID;
    if (x == y && (x_batch != y_batch || x_token != y_token)) return TM_ERR_INVALID;
    RopeArgs a{x, y, x_batch, x_token, y_batch, y_token, positions, freq, (float)result_scale, per_token != 0,
               inverse != 0, batch, n_tokens, heads, head_dim, rot_dim, 0, 0};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool half = layout == TM_ROPE_HALF;
    const hipError_t e = timed_attn(st, [&] {
        return dtype == TM_F32 ? launch_t<float>(a, half, st) : launch_t<bf16>(a, half, st);
    });
    return e == hipSuccess ? TM_OK : e == hipErrorInvalidValue ? TM_ERR_INVALID : TM_ERR_HIP;
}

}  // extern "C"
