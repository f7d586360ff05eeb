// Attention over the paged 8-bit cache (include/tm_attention.h,
// tm_cache_attend).
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c (q . k_j) - m),
//   c = score_scale log2(e), m the row's running maximum of c (q . k_j)
//
// One pass over the keys and values: a wave takes a page of 64 tokens at a
// time, keeps each row's maximum and sum in fp32, and rescales what it has
// accumulated when a maximum grows.  Both products run on the matrix cores
// in bf16: a code times its power-of-two scale is exact in bf16, and the
// hardware conversion applies the scale.  In fp32 calls the other operand
// (the queries, then the weights) is split into three bf16 parts whose sum
// holds 24 bits, each with a product of its own.
//
// The scores are computed transposed (S^T = K Q^T, then O^T = V^T P^T), so
// that a lane's scores of one row are, without any exchange, the operand of
// the second product: the rows of K are fed to the matrix core in the order
// that leaves lane group g (of 4) with the tokens 16 g .. 16 g + 15 of the
// page, one block of one scale, and the values, stored tokens innermost, give
// the same lane the same 16 tokens of a dim in one 16-byte load.  Nothing of
// the cache goes through LDS.
#include <math.h>

#include <type_traits>

#include "tm_cache.h"

namespace tmk {

struct AttendArgs {
    CacheView c;
    const int* seqs;
    const int* counts;
    const void* q;
    long qb, qt;
    void* out;
    int B, T, G;         // entries, query tokens, query heads per kv head
    float scale2;        // score_scale log2(e)
    int window, sink;
    int splits;          // key ranges that the sequence is divided into
    float* part;         // [B][H][splits][rows][D]: accumulators
    float* ml;           // [B][H][splits][rows][2]: maximum and sum
};

constexpr float NEG_INF = -__builtin_inff();

// What the row r = i G + g of entry b sees: tokens lo .. pos and 0 .. sink-1.
struct RowSpan {
    int pos, lo;
};

// The pages a range of rows sees: `first` pages of the sequence's beginning
// (the sink), then lo_page ..; n in all.
struct PageSpan {
    int first, lo_page, n;
    __device__ int at(int i) const { return i < first ? i : lo_page + i - first; }
};
__device__ __forceinline__ PageSpan page_span(const AttendArgs& a, int pos_min, int pos_max) {
    if (pos_max < 0) return PageSpan{0, 0, 0};
    int lo = 0;
    if (a.window > 0) lo = max(0, max(pos_min, 0) - a.window + 1);
    const int lo_page = lo / PAGE;
    const int first = a.window > 0 ? min((a.sink + PAGE - 1) / PAGE, lo_page) : 0;
    return PageSpan{first, lo_page, first + pos_max / PAGE + 1 - lo_page};
}

// Three bf16 values whose sum is x to 24 bits (NP parts of it).
template <int NP> __device__ __forceinline__ void split_bf16(float x, bf16 (&out)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        out[i] = (bf16)x;
        if (i + 1 < NP) x -= (float)out[i];
    }
}

typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
// 8 codes times 2^e, as a matrix operand
__device__ __forceinline__ bf16x8 operand8(unsigned lo, unsigned hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The codes of one page and head that a lane holds: per 16-token tile its
// row's pieces of the keys; per 16-dim tile 16 tokens of its dim.
template <int D> struct KeyRegs {
    uint4 w[4][D / 64 + 1];   // the last: 8 bytes, where D is an odd multiple of 32
};
template <int D> struct ValueRegs {
    uint4 w[D / 16];
};

template <int D> __device__ __forceinline__ void load_keys(KeyRegs<D>& r, const unsigned char* k, int lane) {
    const int m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const unsigned char* row = k + (16 * (m >> 2) + 4 * t + (m & 3)) * D;
#pragma unroll
        for (int n = 0; n < D / 64; ++n) r.w[t][n] = *reinterpret_cast<const uint4*>(row + 64 * n + 16 * g);
        if constexpr (D % 64) {
            const uint2 x = *reinterpret_cast<const uint2*>(row + D / 64 * 64 + 8 * g);
            r.w[t][D / 64] = uint4{x.x, x.y, 0, 0};
        }
    }
}
template <int D> __device__ __forceinline__ void load_values(ValueRegs<D>& r, const unsigned char* v, int lane) {
    const int m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < D / 16; ++u) r.w[u] = *reinterpret_cast<const uint4*>(v + (16 * u + m) * PAGE + 16 * g);
}
// the head dim that slot (step, lane group, j) of the first product's K axis
// stands for, less j
template <int D> __device__ __forceinline__ int key_dim(int step, int g) {
    return step / 2 < D / 64 ? 64 * (step / 2) + 16 * g + 8 * (step & 1) : D / 64 * 64 + 8 * g;
}

// max over the four lane groups (lanes 16 apart)
__device__ __forceinline__ float group_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16, 64));
    return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float group_sum(float x) {
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// Rows of one kv head against its sequence, RT tiles of 16 rows per
// workgroup (row r = i G + g: query token i, head g of the group).  The four
// waves take every fourth page of the workgroup's range; their accumulators
// are joined in LDS at the end.  With one range the workgroup writes the
// output, otherwise its accumulators, maxima and sums for combine_kernel.
template <class T, int D, int RT>
__global__ __launch_bounds__(256) void attend_rows_kernel(AttendArgs a) {
    constexpr int NP = sizeof(T) == 4 ? 3 : 1;
    constexpr int WAVES = 4;
    const CacheView& c = a.c;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits, h = blockIdx.y, b = blockIdx.z;
    const int s = a.seqs ? a.seqs[b] : b;
    const int count = a.counts ? min(max(a.counts[b], 0), a.T) : a.T;
    const int rows = count * a.G, row0 = tile * 16 * RT;
    if (row0 >= rows) return;
    const bool known = (unsigned)s < (unsigned)c.n_seqs;
    const int len = known ? c.length(s) : 0;
    const int i_min = row0 / a.G, i_max = (min(rows, row0 + 16 * RT) - 1) / a.G;
    const int pos_min = len - count + i_min, pos_max = len - count + i_max;
    const PageSpan span = page_span(a, pos_min, pos_max);
    const int per = (span.n + a.splits - 1) / a.splits;
    const int p_begin = min(split * per, span.n), p_end = min(p_begin + per, span.n);

    // this lane's row of each tile: its queries as matrix operands, its span
    bf16x8 qf[RT][D / 32][NP];
    int pos[RT];
    const int HG = c.H * a.G;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = row0 + rt * 16 + m, i = r / a.G, hg = h * a.G + r % a.G;
        pos[rt] = r < rows ? len - count + i : -1;
        const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb + i * a.qt + (long)hg * D;
#pragma unroll
        for (int st = 0; st < D / 32; ++st) {
            if (r < rows) {
                const auto x = ld8(q + key_dim<D>(st, g));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    bf16 parts[NP];
                    split_bf16<NP>((float)x[j], parts);
#pragma unroll
                    for (int p = 0; p < NP; ++p) qf[rt][st][p][j] = parts[p];
                }
            } else {
#pragma unroll
                for (int p = 0; p < NP; ++p) qf[rt][st][p] = zero_frag<bf16>();
            }
        }
    }

    f32x4 o[RT][D / 16];
    float mx[RT], sum[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        mx[rt] = NEG_INF;
        sum[rt] = 0.f;
#pragma unroll
        for (int u = 0; u < D / 16; ++u) o[rt][u] = f32x4{0, 0, 0, 0};
    }

    auto page_of = [&](int i) {   // table entry of the range's page i, or -1
        const int page = i < p_end ? c.page_at(s, span.at(i)) : -1;
        return c.page_ok(page) ? page : -1;
    };
    KeyRegs<D> kr;
    ValueRegs<D> vr;
    float ks, vs;
    auto base = [&](int page) { return c.head_at(max(page, 0), h); };
    int page = page_of(p_begin + w), next = page_of(p_begin + w + WAVES);
    if (p_begin + w < p_end) {
        load_keys<D>(kr, c.k + base(page) * PAGE * D, lane);
        ks = scale_of(c.scales[base(page) * 8 + (m >> 2)]);
    }
    for (int i = p_begin + w; i < p_end; i += WAVES) {
        load_values<D>(vr, c.v + base(page) * PAGE * D, lane);
        vs = scale_of(c.scales[base(page) * 8 + 4 + g]);
        // scores, transposed: lane's row m, tokens 16 g + 4 t + e
        f32x4 sc[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int t = 0; t < 4; ++t) sc[rt][t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int st = 0; st < D / 32; ++st) {
                const uint4 x = kr.w[t][st / 2];
                const bf16x8 kf = st & 1 ? operand8(x.z, x.w, ks) : operand8(x.x, x.y, ks);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int p = 0; p < NP; ++p) mma(sc[rt][t], kf, qf[rt][st][p]);
            }
        }
        const int tok = span.at(i) * PAGE;
        const int here = page;
        page = next;
        if (i + WAVES < p_end) {   // the next page's keys, in flight over what follows
            load_keys<D>(kr, c.k + base(page) * PAGE * D, lane);
            ks = scale_of(c.scales[base(page) * 8 + (m >> 2)]);
            next = page_of(i + 2 * WAVES);
        }
        // a page that every row of the workgroup sees whole needs no mask
        const bool whole = here >= 0 && tok + PAGE - 1 <= pos_min &&
                           (a.window == 0 || tok > pos_max - a.window || tok + PAGE <= a.sink) && row0 + 16 * RT <= rows;
        bf16x8 pf[RT][2][NP];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float top = NEG_INF;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = sc[rt][t][e] * a.scale2;
                    if (!whole) {
                        const int j = tok + 16 * g + 4 * t + e;
                        const bool see = here >= 0 && j <= pos[rt] &&
                                         (a.window == 0 || j > pos[rt] - a.window || j < a.sink);
                        x = see ? x : NEG_INF;
                    }
                    sc[rt][t][e] = x;
                    top = fmaxf(top, x);
                }
            top = fmaxf(mx[rt], group_max(top));
            if (__any(top > mx[rt])) {
                const float by = top == NEG_INF ? 1.f : __builtin_amdgcn_exp2f(mx[rt] - top);
                sum[rt] *= by;
#pragma unroll
                for (int u = 0; u < D / 16; ++u) o[rt][u] *= by;
                mx[rt] = top;
            }
            const float ref = top == NEG_INF ? 0.f : top;   // nothing seen yet: every weight 2^-inf = 0
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = __builtin_amdgcn_exp2f(sc[rt][t][e] - ref);
                    sum[rt] += p;
                    bf16 parts[NP];
                    split_bf16<NP>(p, parts);
#pragma unroll
                    for (int z = 0; z < NP; ++z) pf[rt][t >> 1][z][(t & 1) * 4 + e] = parts[z];
                }
        }
        // behind the sequence's end the page holds anything, NaN codes too
        const int live = len - tok - 16 * g;   // tokens of this lane's block
        const bool cut = tok + PAGE > len;
        if (cut && live <= 0) vs = 1.f;
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {
            uint4 x = vr.w[u];
            if (cut) {
                unsigned* xw = reinterpret_cast<unsigned*>(&x);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int n = min(max(live - 4 * z, 0), 4);
                    xw[z] &= n == 4 ? ~0u : (1u << (8 * n)) - 1;
                }
            }
            const bf16x8 v0 = operand8(x.x, x.y, vs), v1 = operand8(x.z, x.w, vs);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int z = 0; z < NP; ++z) {
                    mma(o[rt][u], v0, pf[rt][0][z]);
                    mma(o[rt][u], v1, pf[rt][1][z]);
                }
        }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sum[rt] = group_sum(sum[rt]);

    // join the waves: common maximum, then sums in a tree
    __shared__ float ml[WAVES][RT * 16][2];
    __shared__ float acc[WAVES / 2][RT * 16][D + 4];
    if (g == 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            ml[w][rt * 16 + m][0] = mx[rt];
            ml[w][rt * 16 + m][1] = sum[rt];
        }
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        float top = NEG_INF, total = 0.f;
#pragma unroll
        for (int z = 0; z < WAVES; ++z) top = fmaxf(top, ml[z][rt * 16 + m][0]);
        const float ref = top == NEG_INF ? 0.f : top;
#pragma unroll
        for (int z = 0; z < WAVES; ++z)
            total += ml[z][rt * 16 + m][1] * __builtin_amdgcn_exp2f(ml[z][rt * 16 + m][0] - ref);
        const float by = __builtin_amdgcn_exp2f(mx[rt] - ref);
#pragma unroll
        for (int u = 0; u < D / 16; ++u) o[rt][u] *= by;
        mx[rt] = top;
        sum[rt] = total;
    }
#pragma unroll
    for (int half = WAVES / 2; half >= 1; half /= 2) {
        if (w >= half && w < 2 * half) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int u = 0; u < D / 16; ++u)
                    *reinterpret_cast<f32x4*>(&acc[w - half][rt * 16 + m][16 * u + 4 * g]) = o[rt][u];
        }
        __syncthreads();
        if (w < half) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int u = 0; u < D / 16; ++u)
                    o[rt][u] += *reinterpret_cast<const f32x4*>(&acc[w][rt * 16 + m][16 * u + 4 * g]);
        }
        __syncthreads();
    }
    if (w != 0) return;
    typedef T Four __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = row0 + rt * 16 + m;
        if (r >= rows) continue;
        if (a.splits == 1) {
            const float by = sum[rt] > 0.f ? 1.f / sum[rt] : (sum[rt] == 0.f ? 0.f : sum[rt]);
            T* out = reinterpret_cast<T*>(a.out) + (((long)b * a.T + r / a.G) * HG + h * a.G + r % a.G) * D;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {
                Four y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (T)(o[rt][u][e] * by);
                *reinterpret_cast<Four*>(out + 16 * u + 4 * g) = y;
            }
        } else {
            const size_t at = (((size_t)b * c.H + h) * a.splits + split) * ((size_t)a.T * a.G) + r;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) *reinterpret_cast<f32x4*>(a.part + at * D + 16 * u + 4 * g) = o[rt][u];
            if (g == 0) {
                a.ml[2 * at] = mx[rt];
                a.ml[2 * at + 1] = sum[rt];
            }
        }
    }
}

// Joins the ranges of a row: a wave per row.
template <class T, int D>
__global__ __launch_bounds__(256) void combine_kernel(AttendArgs a) {
    const CacheView& c = a.c;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, h = blockIdx.y, b = blockIdx.z;
    const int count = a.counts ? min(max(a.counts[b], 0), a.T) : a.T;
    const int r = blockIdx.x * 4 + w;
    if (r >= count * a.G) return;
    const size_t rows = (size_t)a.T * a.G, at0 = ((size_t)b * c.H + h) * a.splits * rows + r;
    float top = NEG_INF;
    for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, a.ml[2 * (at0 + s * rows)]);
#pragma unroll
    for (int x = 32; x > 0; x /= 2) top = fmaxf(top, __shfl_xor(top, x, 64));
    const float ref = top == NEG_INF ? 0.f : top;
    constexpr int IT = (D + 127) / 128;
    float o[IT][2], total = 0.f;
#pragma unroll
    for (int it = 0; it < IT; ++it) o[it][0] = o[it][1] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const size_t at = at0 + s * rows;
        const float by = __builtin_amdgcn_exp2f(a.ml[2 * at] - ref);
        total += a.ml[2 * at + 1] * by;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int dim = it * 128 + 2 * lane;
            if (dim < D) {
                const float2 x = *reinterpret_cast<const float2*>(a.part + at * D + dim);
                o[it][0] += x.x * by;
                o[it][1] += x.y * by;
            }
        }
    }
    const float by = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
    typedef T Two __attribute__((ext_vector_type(2)));
    T* out = reinterpret_cast<T*>(a.out) + (((long)b * a.T + r / a.G) * c.H * a.G + h * a.G + r % a.G) * D;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int dim = it * 128 + 2 * lane;
        if (dim < D) *reinterpret_cast<Two*>(out + dim) = Two{(T)(o[it][0] * by), (T)(o[it][1] * by)};
    }
}

// How a call is launched: tiles of 16 or 32 rows, and into how many ranges
// the sequences are divided.
struct AttendPlan {
    int rt, tiles, splits;
};
static AttendPlan attend_plan(const tm_cache* c, int batch, int n_tokens, int heads, long max_len) {
    AttendPlan p;
    const long rows = (long)n_tokens * (heads / c->H);
    p.rt = rows > 16 ? 2 : 1;
    p.tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
    const long pages = (max_len + PAGE - 1) / PAGE, groups = (long)batch * c->H * p.tiles;
    long s = 1024 / groups;
    const long most = (pages + 7) / 8;   // two pages a wave at least
    if (s > most) s = most;
    if (s > 256) s = 256;
    p.splits = s < 1 ? 1 : (int)s;
    return p;
}

size_t attend_workspace(const tm_cache* c, int batch, int n_tokens, int heads) {
    if (heads % c->H != 0 || batch == 0 || n_tokens == 0) return 0;
    // the most ranges that any max_len leads to
    const AttendPlan p = attend_plan(c, batch, n_tokens, heads, (long)c->seq_pages * PAGE);
    if (p.splits == 1) return 0;
    const size_t rows = (size_t)batch * c->H * p.splits * n_tokens * (heads / c->H);
    return (rows * (c->d + 2) * 4 + 511) / 256 * 256;
}

template <class T>
static hipError_t launch_attend(const tm_cache* c, const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
    hipError_t e = timed_attn(st, [&] {
        return for_head_dim(c->d, [&](auto D) {
            const dim3 grid((unsigned)(p.tiles * p.splits), (unsigned)c->H, (unsigned)a.B);
            if (p.rt == 1) launch_k(attend_rows_kernel<T, D(), 1>, grid, dim3(256), 0, st, a);
            else launch_k(attend_rows_kernel<T, D(), 2>, grid, dim3(256), 0, st, a);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || p.splits == 1) return e;
    return timed_attn(st, [&] {
        return for_head_dim(c->d, [&](auto D) {
            const dim3 grid((unsigned)(((long)a.T * a.G + 3) / 4), (unsigned)c->H, (unsigned)a.B);
            launch_k(combine_kernel<T, D()>, grid, dim3(256), 0, st, a);
            return hipGetLastError();
        });
    });
}

}  // namespace tmk

using namespace tmk;

extern "C" tm_status tm_cache_attend(const tm_cache* c, const void* blob, const int* seqs, const int* counts,
                                     const void* q, long q_batch, long q_token, void* out, int batch, int n_tokens,
                                     int heads, float score_scale, int window, int sink, int max_len, tm_dtype dtype,
                                     void* workspace, void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (!c || !ptr_ok(blob, 256) || batch < 0 || n_tokens < 0 || heads < 1 || heads % c->H != 0 || heads / c->H > 64 ||
        !isfinite(score_scale) || window < 0 || sink < 0 || max_len < 0)
        return TM_ERR_INVALID;
    if (batch == 0 || n_tokens == 0) return TM_OK;
    const long most = (long)c->seq_pages * PAGE;
    if (batch > 65535 || (!seqs && batch > c->n_seqs) || n_tokens > 1 << 24 || (uintptr_t)seqs % 4 || (uintptr_t)counts % 4 ||
        !ptr_ok(q, 16) || !ptr_ok(out, 16) || !strides_ok(q_batch, q_token))
        return TM_ERR_INVALID;
    const AttendPlan p = attend_plan(c, batch, n_tokens, heads, max_len > 0 && max_len < most ? max_len : most);
    if (p.splits > 1 && !ptr_ok(workspace, 256)) return TM_ERR_INVALID;
    const int G = heads / c->H;
    const size_t rows = (size_t)batch * c->H * p.splits * n_tokens * G;
    float* part = static_cast<float*>(workspace);
    AttendArgs a{cache_view(c, const_cast<void*>(blob)), seqs, counts, q, q_batch, q_token, out, batch, n_tokens, G,
                 score_scale * 1.44269504088896340736f, window, sink < most ? sink : (int)most, p.splits, part, part + rows * c->d};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == TM_F32 ? launch_attend<float>(c, a, p, st) : launch_attend<bf16>(c, a, p, st);
    return e == hipSuccess ? TM_OK : TM_ERR_HIP;
}
