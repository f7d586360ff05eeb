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
// (127 x and m have 15 and 8 bits) no other is; a row whose 127 m
// would overflow is divided by 2^10 beforehand (exactly).
template <class T>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const T* x, long x_row, signed char* codes, long code_row,
                                                            float* scales, int cols) {
    __shared__ float red[4];
    const long row = blockIdx.x;
    const T* p = x + row * x_row;
    signed char* c = codes + row * code_row;
    float m = 0.f;
    bool fine = true;
    for (int i = threadIdx.x; i < cols; i += 256) {
        const float v = fabsf((float)p[i]);
        fine &= v <= 3.402823466e38f;   // not for NaN and infinity
        m = fmaxf(m, v);
    }
    if (!fine) m = __builtin_inff();
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const bool lost = m == __builtin_inff(), any = m > 0.f && !lost;
    const float down = m > 1e36f ? 0x1p-10f : 1.f, top = m * down;
    if (threadIdx.x == 0) scales[row] = lost ? __builtin_nanf("") : m / 127.f;
    for (long i = threadIdx.x; i < code_row; i += 256) {
        int v = 0;
        if (any && i < cols) v = (int)rintf(127.f * ((float)p[i] * down) / top);
        c[i] = (signed char)v;
    }
}

struct Int8Args {
    const signed char* a;
    const float* as;
    const signed char* w;
    const float* wsc;
    void* y;
    long code_row, y_row, M;
    int N, mtiles, vec;   // vec: rows of y allow stores of 4 values
};

// 128 rows of x by 128 rows of w a workgroup, 64 by 64 a wave.  The rows of w
// are the matrix instruction's first operand, so a lane ends up with 4
// neighbouring outputs of one row of y.
template <class T> __global__ __launch_bounds__(256) void int8_matmul_kernel(Int8Args g) {
    constexpr int KT = 64, ROW = KT + 16;
    __shared__ __attribute__((aligned(16))) signed char at[128 * ROW], wt[128 * ROW];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
    const long m0 = (long)(blockIdx.x % g.mtiles) * 128;
    const int n0 = blockIdx.x / g.mtiles * 128;
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    i32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    for (long k0 = 0; k0 < g.code_row; k0 += KT) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = threadIdx.x + 256 * i, r = u >> 2, c = (u & 3) * 16;
            i32x4 x = i32x4{0, 0, 0, 0}, y = x;
            if (k0 + c < g.code_row) {
                if (m0 + r < g.M) x = *reinterpret_cast<const i32x4*>(g.a + (m0 + r) * g.code_row + k0 + c);
                if (n0 + r < g.N) y = *reinterpret_cast<const i32x4*>(g.w + (long)(n0 + r) * g.code_row + k0 + c);
            }
            *reinterpret_cast<i32x4*>(at + r * ROW + c) = x;
            *reinterpret_cast<i32x4*>(wt + r * ROW + c) = y;
        }
        __syncthreads();
        i32x4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const i32x4*>(at + (wm + 16 * i + l16) * ROW + 16 * lg);
            y[i] = *reinterpret_cast<const i32x4*>(wt + (wn + 16 * i + l16) * ROW + 16 * lg);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(y[j], x[i], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long m = m0 + wm + 16 * i + l16;
        if (m >= g.M) continue;
        const double s = g.as[m];   // 64 bits: neither product overflows where the result does not
        T* y = reinterpret_cast<T*>(g.y) + m * g.y_row;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + wn + 16 * j + 4 * lg;
            struct __align__(4 * sizeof(T)) V4 { T e[4]; } o;
#pragma unroll
            for (int r = 0; r < 4; ++r) o.e[r] = (T)((double)acc[i][j][r] * s * (double)(n + r < g.N ? g.wsc[n + r] : 0.f));
            if (g.vec && n + 3 < g.N) {
                *reinterpret_cast<V4*>(y + n) = o;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n + r < g.N) y[n + r] = o.e[r];
            }
        }
    }
}

static hipError_t int8_quantize(const void* x, long x_row, signed char* codes, long code_row, float* scales, long rows,
                                int cols, tm_dtype dtype, hipStream_t st) {
    if (rows >= 1L << 24) return hipErrorInvalidValue;   // a launch has fewer than 2^32 threads along an axis
    return timed_layer(st, [&] {
        if (dtype == TM_F32)
            launch_k(int8_quantize_kernel<float>, dim3((unsigned)rows), dim3(256), 0, st, static_cast<const float*>(x),
                     x_row, codes, code_row, scales, cols);
        else
            launch_k(int8_quantize_kernel<bf16>, dim3((unsigned)rows), dim3(256), 0, st, static_cast<const bf16*>(x),
                     x_row, codes, code_row, scales, cols);
        return hipGetLastError();
    });
}

static hipError_t int8_matmul(Int8Args g, tm_dtype dtype, hipStream_t st) {
    const size_t es = dtype == TM_F32 ? 4 : 2;
    g.vec = (uintptr_t)g.y % (4 * es) == 0 && g.y_row % 4 == 0;
    const long mt = (g.M + 127) / 128, blocks = mt * ((g.N + 127L) / 128);
    if (blocks >= 1L << 24) return hipErrorInvalidValue;
    g.mtiles = (int)mt;
    return timed_layer(st, [&] {
        if (dtype == TM_F32) launch_k(int8_matmul_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, st, g);
        else launch_k(int8_matmul_kernel<bf16>, dim3((unsigned)blocks), dim3(256), 0, st, g);
        return hipGetLastError();
    });
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
    return int8_status(int8_matmul(Int8Args{a, a_scales, w, w_scales, y, code_row, y_row, rows, outs, 0, 0}, dtype,
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
    signed char* codes = static_cast<signed char*>(workspace);
    float* scales = reinterpret_cast<float*>(codes + ((size_t)rows * code_row + 255) / 256 * 256);
    const hipError_t e = int8_quantize(x, x_row, codes, code_row, scales, rows, cols, dtype, st);
    if (e != hipSuccess) return int8_status(e);
    return int8_status(int8_matmul(Int8Args{codes, scales, w, w_scales, y, code_row, y_row, rows, outs, 0, 0}, dtype, st));
}

}  // extern "C"
