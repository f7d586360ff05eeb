// Attention over the paged 8-bit cache (include/tm_attention.h,
// tm_cache_attend).
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c s_j - m),   s_j = +-q . k_j,
//   c = |score_scale| log2(e), m the row's running maximum of c s_j
//
// (the sign of score_scale goes into q, so that the largest s_j has the
// largest weight and c is applied in the exponent's fused multiply-add).
//
// One pass over the keys and values: a wave takes a page of 64 tokens at a
// time, keeps each row's maximum and sum in fp32, and rescales what it has
// accumulated when a maximum grows.  Both products run on the matrix cores
// in bf16: a code times its power-of-two scale is exact in bf16, and the
// hardware conversion applies the scale.  In fp32 calls the other operand
// (the queries, then the weights) is split into three bf16 parts whose sum
// holds 24 bits, each with a product of its own.  In bf16 calls the queries
// are bf16 already; the weights are split into two parts (16 bits) for few
// rows and rounded to one for many (the kernels say why).
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
    float scale2, sign;  // |score_scale| log2(e), above 0 (a masked score is -inf times it), and score_scale's sign
    int window, sink;
    int splits;          // the most key ranges that a tile's pages are divided into
    int least;           // pages of a range, at least
    int tile_rows;       // rows of a workgroup
    float* part;         // [B][H][splits][rows][D]: accumulators
    float* ml;           // [B][H][splits][rows][2]: maximum and sum
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

constexpr float NEG_INF = -__builtin_inff();
// A row's running maximum moves when it grows by more than this: weights up
// to 2^8 are as exact, and the accumulators are rarely rescaled.
constexpr float SLACK = 8.f;

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

// One workgroup's part of a call: a tile of rows of entry b.  Wave-uniform.
struct Tile {
    int len, rows;          // tokens of the sequence; rows of the entry
    int first;              // position of query 0
    int pos_min, pos_max;   // positions of the tile's first and last row
    PageSpan span;          // the pages its rows see
    int ranges, per;        // how many ranges they are divided into, pages of each
};
__device__ __forceinline__ Tile tile_of(const AttendArgs& a, int b, int s, int tile) {
    Tile t;
    const int count = uniform(a.counts ? min(max(a.counts[b], 0), a.T) : a.T);
    t.len = uniform((unsigned)s < (unsigned)a.c.n_seqs ? a.c.length(s) : 0);
    t.rows = count * a.G;
    t.first = t.len - count;
    t.pos_min = t.first + tile * a.tile_rows / a.G;
    t.pos_max = t.first + (min(t.rows, (tile + 1) * a.tile_rows) - 1) / a.G;
    t.span = page_span(a, t.pos_min, t.pos_max);
    t.ranges = min(a.splits, max(1, (t.span.n + a.least - 1) / a.least));
    t.per = (t.span.n + t.ranges - 1) / t.ranges;
    return t;
}

// What a row at `pos` sees: the tokens lo .. lo + n - 1 (one unsigned
// comparison a token) and those below `sink`; nothing before the sequence's
// start.
struct Sight {
    int lo, sink;
    unsigned n;
    __device__ bool sees(int j) const { return ((unsigned)(j - lo) < n) | (j < sink); }
};
__device__ __forceinline__ Sight sight_of(const AttendArgs& a, int pos) {
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    return Sight{lo, a.window > 0 ? min(a.sink, pos + 1) : 0, pos < 0 ? 0u : (unsigned)(pos - lo + 1)};
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

// Over the lanes 32 apart, and 16 and 32 apart: row swaps of the vector
// units, no trip through LDS.  Each of the two results holds one side (taken
// out before it is reinterpreted: a bit cast of a vector's element in place
// reads the first).
__device__ __forceinline__ float pair_max(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned lo = r[0], hi = r[1];
    return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}
__device__ __forceinline__ float group_max(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const unsigned lo = r[0], hi = r[1];
    return pair_max(fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)));
}
__device__ __forceinline__ float group_sum(float x) {
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// Few rows of one kv head against its sequence (single tokens, drafts): RT
// tiles of 16 rows per wave (row r = i G + g: query token i, head g of the
// group), which share the codes' conversion; WR such groups per workgroup.
// Wave w takes row group w % WR and every (WAVES / WR)-th page of the
// workgroup's range; the waves of a group are joined in LDS at the end.  With
// one range the workgroup writes the output, otherwise its accumulators,
// maxima and sums for combine_kernel.  Bound by reading the pages: a wave's
// next keys and present values are in flight while it computes.  That leaves
// room for the weights' second part in bf16 calls: with it results differ from
// 64 bits by their own rounding (0.0017 of their size; with one part 0.0023).
// One part against two: 48 sequences as below 285 us each; 16 of 2000 to 20000
// tokens with 4 key heads, single tokens of 16 heads, then 4 tokens of 64: width
// 64 22.8 against 23.8 and 46 against 50 us, 128 40.6 against 40.8 and 114 each,
// 256 96 against 97 and 178 against 190; width 32, bound by the vector units,
// 16.7 against 18.4 and 38 against 47.
// 48 sequences of 2000 to 30000 tokens, 32 heads on 8 of 128, bf16: 288 us, 5.4 TB/s; 4
// fp32 tokens of one of 10^6, 16 heads on 2 of 256: 232 us, 4.4 TB/s.
template <class T, int D, int WR, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D * RT * (sizeof(T) == 4 ? 3 : 1) <= 192 ? 2 : 1) void attend_rows_kernel(AttendArgs a) {
    constexpr int NP = sizeof(T) == 4 ? 3 : 1, NW = sizeof(T) == 4 ? 3 : 2;   // parts of a query, of a weight
    constexpr int WP = WAVES / WR;   // waves that share a row group
    const CacheView& c = a.c;
    const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6), m = lane & 15, g = lane >> 4;
    const int wr = w % WR, wp = w / WR;
    const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits, h = blockIdx.y, b = blockIdx.z;
    const int s = uniform(a.seqs ? a.seqs[b] : b), row0 = (tile * WR + wr) * 16 * RT;
    const Tile tl = tile_of(a, b, s, tile);
    const int rows = tl.rows, len = tl.len, pos_min = tl.pos_min, pos_max = tl.pos_max;
    if (tile * WR * RT * 16 >= rows || split >= tl.ranges) return;
    const PageSpan span = tl.span;
    const int p_begin = min(split * tl.per, span.n), p_end = min(p_begin + tl.per, span.n);

    // this lane's rows: their queries as matrix operands, their positions
    // (too many for the registers in three parts or with wide heads: in LDS)
    constexpr bool Q_LDS = NP > 1 || RT * D > 256;
    constexpr int QL = Q_LDS ? WR * RT * (D / 32) * NP * 64 * 16 : 0;                   // their bytes
    constexpr int ACC = WP > 1 ? WAVES / 2 * RT * 16 * (D + 4) * 4 : 0;                 // the join's, in their place
    __shared__ __align__(16) unsigned char lds[QL > ACC ? QL : ACC > 16 ? ACC : 16];
    bf16x8* ql = reinterpret_cast<bf16x8*>(lds);
    bf16x8 qf[RT][Q_LDS ? 1 : D / 32];
    const int HG = c.H * a.G;
    Sight sight[RT];
    auto row_of = [&](int rt) { return row0 + 16 * rt + m; };
    auto head_of = [&](int rt) { return h * a.G + row_of(rt) % a.G; };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = row_of(rt);
        sight[rt] = sight_of(a, tl.first + r / a.G);   // (rows behind the last see as if there: dropped)
        const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb + (long)(r / a.G) * a.qt + (long)head_of(rt) * D;
#pragma unroll
        for (int st = 0; st < D / 32; ++st) {
            bf16x8 f[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) f[p] = zero_frag<bf16>();
            if (r < rows) {
                const auto x = ld8(q + key_dim<D>(st, g));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    bf16 parts[NP];
                    split_bf16<NP>((float)x[j] * a.sign, parts);
#pragma unroll
                    for (int p = 0; p < NP; ++p) f[p][j] = parts[p];
                }
            }
            if constexpr (Q_LDS) {
                if (wp == 0) {
#pragma unroll
                    for (int p = 0; p < NP; ++p) ql[((wr * RT + rt) * (D / 32) * NP + st * NP + p) * 64 + lane] = f[p];
                }
            } else {
                qf[rt][st] = f[0];
            }
        }
    }
    if constexpr (Q_LDS) __syncthreads();

    f32x4 o[RT][D / 16];
    float mx[RT], sum[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        mx[rt] = NEG_INF;
        sum[rt] = 0.f;
#pragma unroll
        for (int u = 0; u < D / 16; ++u) o[rt][u] = f32x4{0, 0, 0, 0};
    }

    // Table entries of this wave's next 64 pages, one a lane, read ahead of the
    // codes: a load behind them would be waited for together with them.
    const int i0 = p_begin + wp;
    int ids = -1;
    auto page_of = [&](int n) {   // the wave's n-th page, or -1; called in order
        if ((n & 63) == 0) {
            const int i = i0 + (n + lane) * WP;
            ids = i < p_end ? c.page_at(s, span.at(i)) : -1;
        }
        const int page = __builtin_amdgcn_readlane(ids, n & 63);
        return c.page_ok(page) ? page : -1;
    };
    struct Codes {
        KeyRegs<D> k;
        ValueRegs<D> v;
        unsigned char ks, vs;   // the scales of the lane's rows, as stored: made numbers where they are used, not
                                // where they are loaded, which would wait for the codes loaded before them
    };
    auto base = [&](int page) { return c.head_at(max(page, 0), h); };
    auto load_k = [&](Codes& x, int page) {
        load_keys<D>(x.k, c.k + base(page) * PAGE * D, lane);
        x.ks = c.scales[base(page) * 8 + (m >> 2)];
    };
    auto load_v = [&](Codes& x, int page) {
        load_values<D>(x.v, c.v + base(page) * PAGE * D, lane);
        x.vs = c.scales[base(page) * 8 + 4 + g];
    };
    // one page's step; `then` starts loads as soon as the keys are used up
    auto step = [&](Codes& x, int i, int here, auto&& then) {
        // scores, transposed: lane's row m, tokens 16 g + 4 t + e
        f32x4 sc[RT][4];
        const float ks = scale_of(x.ks);
        int ql_lane = lane;   // hidden from the optimizer, which would lift the queries' reads into registers
        if constexpr (Q_LDS) asm volatile("" : "+v"(ql_lane));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int t = 0; t < 4; ++t) sc[rt][t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int st = 0; st < D / 32; ++st) {
            bf16x8 kf[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint4 y = x.k.w[t][st / 2];
                kf[t] = st & 1 ? operand8(y.z, y.w, ks) : operand8(y.x, y.y, ks);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    bf16x8 f;
                    if constexpr (Q_LDS) f = ql[((wr * RT + rt) * (D / 32) * NP + st * NP + p) * 64 + ql_lane];
                    else f = qf[rt][st];
#pragma unroll
                    for (int t = 0; t < 4; ++t) mma(sc[rt][t], kf[t], f);
                }
        }
        then();
        const int tok = span.at(i) * PAGE;
        // a page that every row sees whole needs no mask
        const bool whole = here >= 0 && tok + PAGE - 1 <= pos_min &&
                           (a.window == 0 || tok > pos_max - a.window || tok + PAGE <= a.sink);
        bf16x8 pf[RT][2][NW];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            if (!whole) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = tok + 16 * g + 4 * t + e;
                        const bool see = (here >= 0) & sight[rt].sees(j);
                        sc[rt][t][e] = see ? sc[rt][t][e] : NEG_INF;
                    }
            }
            float top = NEG_INF;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[rt][t][e]);
            top = group_max(top) * a.scale2;
            const bool grown = top > mx[rt] + SLACK;
            if (__any(grown)) {   // a row's steps follow from the row alone: the others' factor is 1
                top = grown ? top : mx[rt];
                const float by = grown ? __builtin_amdgcn_exp2f(mx[rt] - top) : 1.f;
                sum[rt] *= by;
#pragma unroll
                for (int u = 0; u < D / 16; ++u) o[rt][u] *= by;
                mx[rt] = top;
            }
            const float ref = mx[rt] == NEG_INF ? 0.f : mx[rt];   // nothing seen yet: every weight 2^-inf = 0
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(sc[rt][t][e], a.scale2, -ref));
                    sum[rt] += p;
                    bf16 parts[NW];
                    split_bf16<NW>(p, parts);
#pragma unroll
                    for (int z = 0; z < NW; ++z) pf[rt][t >> 1][z][(t & 1) * 4 + e] = parts[z];
                }
        }
        float vs = scale_of(x.vs);
        // behind the sequence's end the page holds anything, NaN codes too, and
        // so does the page that was loaded for an entry out of range
        if (tok + PAGE > len || here < 0) {
            const int live = here < 0 ? 0 : len - tok - 16 * g;   // tokens of this lane's block
            if (live <= 0) vs = 1.f;
            unsigned keep[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int n = min(max(live - 4 * z, 0), 4);
                keep[z] = n == 4 ? ~0u : (1u << (8 * n)) - 1;
            }
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {
                x.v.w[u].x &= keep[0];
                x.v.w[u].y &= keep[1];
                x.v.w[u].z &= keep[2];
                x.v.w[u].w &= keep[3];
            }
        }
        // two dim tiles at a time: products that do not wait for each other
#pragma unroll
        for (int u = 0; u < D / 16; u += 2) {
            bf16x8 vf[2][2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                vf[y][0] = operand8(x.v.w[u + y].x, x.v.w[u + y].y, vs);
                vf[y][1] = operand8(x.v.w[u + y].z, x.v.w[u + y].w, vs);
            }
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                for (int z = 0; z < NW; ++z)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) mma(o[rt][u + y], vf[y][k2], pf[rt][k2][z]);
        }
    };
    const int pages = i0 < p_end ? (p_end - i0 + WP - 1) / WP : 0;
    // A page's values are loaded over its first product, the next page's keys
    // over the rest.  The loads of what comes next are issued on every path
    // (the last page's keys again behind the end): behind a branch, every wait
    // would have to be for all that may be in flight.  (Loading both a whole
    // page ahead, with twice the registers, measured no faster: 2-3% slower
    // for 48 sequences of 2000 to 30000 tokens.)
    if (pages > 0) {
        Codes x;
        int page = page_of(0);
        load_k(x, page);
        for (int n = 0; n < pages; ++n) {
            const int here = page;
            load_v(x, here);
            step(x, i0 + n * WP, here, [&] {
                if (n + 1 < pages) page = page_of(n + 1);
                load_k(x, page);
            });
        }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sum[rt] = group_sum(sum[rt]);

    // join the waves of a row group: common maximum, then sums in a tree
    __shared__ float ml[WAVES][RT * 16][2];
    if constexpr (WP > 1) {
        float(*acc)[RT * 16][D + 4] = reinterpret_cast<float(*)[RT * 16][D + 4]>(lds);
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
            const int at = rt * 16 + m;
            float top = NEG_INF, total = 0.f;
#pragma unroll
            for (int z = 0; z < WP; ++z) top = fmaxf(top, ml[z * WR + wr][at][0]);
            const float ref = top == NEG_INF ? 0.f : top;
#pragma unroll
            for (int z = 0; z < WP; ++z)
                total += ml[z * WR + wr][at][1] * __builtin_amdgcn_exp2f(ml[z * WR + wr][at][0] - ref);
            const float by = __builtin_amdgcn_exp2f(mx[rt] - ref);
#pragma unroll
            for (int u = 0; u < D / 16; ++u) o[rt][u] *= by;
            mx[rt] = top;
            sum[rt] = total;
        }
#pragma unroll
        for (int half = WP / 2; half >= 1; half /= 2) {
            if (wp >= half && wp < 2 * half) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int u = 0; u < D / 16; ++u)
                        *reinterpret_cast<f32x4*>(&acc[w - half * WR][rt * 16 + m][16 * u + 4 * g]) = o[rt][u];
            }
            __syncthreads();
            if (wp < half) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int u = 0; u < D / 16; ++u)
                        o[rt][u] += *reinterpret_cast<const f32x4*>(&acc[w][rt * 16 + m][16 * u + 4 * g]);
            }
            __syncthreads();
        }
    }
    if (wp != 0) return;
    typedef T Four __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = row_of(rt);
        if (r >= rows) continue;
        if (tl.ranges == 1) {
            const float by = sum[rt] > 0.f ? 1.f / sum[rt] : (sum[rt] == 0.f ? 0.f : sum[rt]);
            T* out = reinterpret_cast<T*>(a.out) + (((long)b * a.T + r / a.G) * HG + head_of(rt)) * D;
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

// Many rows of one kv head against its sequence (a segment or a prompt): 32
// rows per wave, on the 32x32x16 matrix instruction.  Every row tile needs
// every page, so the pages' codes are converted to bf16 once per workgroup,
// into LDS (two buffers: the next pages are loaded over the present ones'
// products and stored into the other buffer, one barrier per step); rows of
// D + 8 and 64 + 8 elements keep the 16-byte operand reads off each other's
// banks.  Bound by the matrix and vector units in turn: 2 x 2048 ragged
// queries over 7000 tokens in a window of 4096, 32 heads on 8 of 128, bf16:
// 240 to 250 us, 830 to 860 TFLOP/s; 2 x 1024 over 2064, 6 heads of 64: 24 us,
// 208 TFLOP/s; the prompt at widths 64, 160, 192, 224, 256: 140, 478, 538, 684,
// 670 us (above 128 a wave is alone on its SIMD).  In fp32, with three products
// for each: the prompt at 64, 128, 256 345, 562, 1480 us, the segment 35 us; the
// queries' three parts do not all fit the registers at widths 224 and 256 and for
// eight waves of width 128 (232, 336 and 108 bytes a lane go to memory).
// (The next page's scores computed beside the present one's weights: 252 and
// 27 us, since two waves a SIMD overlap already.)  bf16 calls round a weight
// to bf16 once, and results differ from 64 bits by 0.0023 of their size
// instead of 0.0017: a second part, as single tokens take it, is half as many
// matrix instructions again where those bound the kernel (323 us against 250
// and 28.6 against 24.5, at best), and the sum of the rounded weights in place
// of the exact ones' gains next to nothing (0.00226; 3% slower).  The same call
// in fp32 keeps 24 bits.
// The transposed scores' layout (lane group h of 2 holds rows 8 a + 4 h + b) is
// again made the second product's operand by the order in which rows of K are
// fed: row 8 a + 4 h + b of a 32-token tile is token 16 (a / 2) + 8 h + 4 (a % 2) + b,
// so a lane ends up with runs of 8 tokens.
//
// KW waves share a row tile and take a page each of the KW that a step holds;
// they are joined in LDS at the end.  Large calls take KW = 1 (128 rows of
// four waves; the sequence in several ranges where the tiles do not fill the
// chip); a window's few tiles take eight waves and KW = 2 or 4, which walks
// the sequence in fewer steps without a second launch.
typedef float f32x16 __attribute__((ext_vector_type(16)));
template <class T, int D, int WAVES, int KW>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 2 && D <= 128 ? 2 : 1) void attend_tiles_kernel(AttendArgs a) {
    constexpr int NP = sizeof(T) == 4 ? 3 : 1;
    constexpr int THREADS = 64 * WAVES, TILE_ROWS = 32 * WAVES / KW;
    constexpr int KS = D + 8, VS = PAGE + 8, KB = PAGE * KS, VB = D * VS;   // LDS row and page distances
    constexpr int PP = 4 * D, PIECES = KW * PP, NK = (PIECES + THREADS - 1) / THREADS;   // 16-byte pieces of the keys
    __shared__ __align__(16) bf16 kv[2][KW * (KB + VB)];
    const CacheView& c = a.c;
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 31, g = lane >> 5;
    const int w = uniform(tid >> 6), kw = w % KW;
    // heads innermost: with a multiple of 8 of them, the workgroups that read
    // the same pages stand on one XCD and share its L2
    const int h = blockIdx.x % c.H, x = blockIdx.x / c.H, b = blockIdx.z;
    const int s = uniform(a.seqs ? a.seqs[b] : b);
    // the last rows first: they see the most
    const int split = x % a.splits, tile = (a.T * a.G + TILE_ROWS - 1) / TILE_ROWS - 1 - x / a.splits;
    const Tile tl = tile_of(a, b, s, tile);
    const int rows = tl.rows, len = tl.len, first = tl.first, row0 = tile * TILE_ROWS;
    if (row0 >= rows || split >= tl.ranges) return;
    const PageSpan span = tl.span;
    const int p_begin = min(split * tl.per, span.n), p_end = min(p_begin + tl.per, span.n);

    // this wave's rows, and what all of them and any of them see
    const int wr0 = row0 + 32 * (w / KW), r = wr0 + m, HG = c.H * a.G;
    const bool live_row = r < rows;
    const Sight sight = sight_of(a, first + r / a.G);   // (rows behind the last see as if there: dropped)
    const int w_min = first + wr0 / a.G, w_max = wr0 < rows ? first + (min(rows, wr0 + 32) - 1) / a.G : -1;

    bf16x8 qf[D / 16][NP];
    {
        const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb + (long)(r / a.G) * a.qt + (long)(h * a.G + r % a.G) * D;
#pragma unroll
        for (int st = 0; st < D / 16; ++st) {
            if (live_row) {
                const auto x = ld8(q + 16 * st + 8 * g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    bf16 parts[NP];
                    split_bf16<NP>((float)x[j] * a.sign, parts);
#pragma unroll
                    for (int z = 0; z < NP; ++z) qf[st][z][j] = parts[z];
                }
            } else {
#pragma unroll
                for (int z = 0; z < NP; ++z) qf[st][z] = zero_frag<bf16>();
            }
        }
    }
    f32x16 o[D / 32];
#pragma unroll
    for (int u = 0; u < D / 32; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[u][e] = 0.f;
    float mx = NEG_INF, sum = 0.f;

    uint4 kr[NK], vr[NK];
    uint2 scales[NK];
    int ids = -1;   // table entries of 64 of the range's pages, one a lane
    auto turn = [&](int n) {   // to the 64 entries that hold the range's page n, a multiple of KW
        if ((n & 63) == 0) {
            const int i = p_begin + n + lane;
            const int page = i < p_end ? c.page_at(s, span.at(i)) : -1;
            ids = c.page_ok(page) ? page : -1;
        }
    };
    auto load = [&](int n) {
#pragma unroll
        for (int z = 0; z < NK; ++z) {
            const int q = tid + THREADS * z, pk = q / PP, p = q % PP;
            if (PIECES % THREADS != 0 && q >= PIECES) continue;
            const int page = KW == 1 ? __builtin_amdgcn_readlane(ids, n & 63) : __shfl(ids, (n + pk) & 63, 64);
            if (page < 0) continue;
            const size_t at = c.head_at(page, h);
            kr[z] = reinterpret_cast<const uint4*>(c.k + at * PAGE * D)[p];
            vr[z] = reinterpret_cast<const uint4*>(c.v + at * PAGE * D)[p];
            scales[z] = *reinterpret_cast<const uint2*>(c.scales + at * 8);
        }
    };
    auto stage = [&](int buf, int n) {
#pragma unroll
        for (int z = 0; z < NK; ++z) {
            const int q = tid + THREADS * z, pk = q / PP, p = q % PP;
            if (PIECES % THREADS != 0 && q >= PIECES) continue;
            const int tok = span.at(p_begin + n + pk) * PAGE;
            const int t = p / (D / 16), col = p % (D / 16) * 16;
            const float ks = scale_of((unsigned char)(scales[z].x >> (8 * (t >> 4))));
            bf16* kd = &kv[buf][pk * KB + t * KS + col];
            *reinterpret_cast<bf16x8*>(kd) = operand8(kr[z].x, kr[z].y, ks);
            *reinterpret_cast<bf16x8*>(kd + 8) = operand8(kr[z].z, kr[z].w, ks);
            const int dim = p >> 2, quarter = p & 3;
            const int live = len - tok - 16 * quarter;   // tokens of the piece within the sequence
            float vs = scale_of((unsigned char)(scales[z].y >> (8 * quarter)));
            uint4 x = vr[z];
            if (live < 16) {   // behind the end the page holds anything, NaN codes too
                unsigned* xw = reinterpret_cast<unsigned*>(&x);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int k4 = min(max(live - 4 * y, 0), 4);
                    xw[y] &= k4 == 4 ? ~0u : (1u << (8 * k4)) - 1;
                }
                if (live <= 0) vs = 1.f;
            }
            bf16* vd = &kv[buf][KW * KB + pk * VB + dim * VS + quarter * 16];
            *reinterpret_cast<bf16x8*>(vd) = operand8(x.x, x.y, vs);
            *reinterpret_cast<bf16x8*>(vd + 8) = operand8(x.z, x.w, vs);
        }
    };
    const int tau = 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3);   // token of row m of a tile

    turn(0);
    load(0);
    stage(0, 0);
    __syncthreads();
    for (int n = 0; n < p_end - p_begin; n += KW) {
        const int buf = (n / KW) & 1, tok = span.at(p_begin + n + kw) * PAGE;
        const int page = __builtin_amdgcn_readlane(ids, (n + kw) & 63);
        const bool more = n + KW < p_end - p_begin;
        if (more) {
            turn(n + KW);
            load(n + KW);
        }
        const bf16* kb = &kv[buf][kw * KB];
        const bf16* vb = &kv[buf][KW * KB + kw * VB];
        // nothing of the page in sight of the wave's rows: its products are skipped
        const bool seen = page >= 0 && tok <= w_max &&
                          (a.window == 0 || tok + PAGE - 1 > w_min - a.window || tok < a.sink);
        if (seen) {
            f32x16 sc[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) sc[t][e] = 0.f;
#pragma unroll
            for (int st = 0; st < D / 16; ++st)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const bf16x8 kf = *reinterpret_cast<const bf16x8*>(&kb[(t * 32 + tau) * KS + 16 * st + 8 * g]);
#pragma unroll
                    for (int z = 0; z < NP; ++z)
                        sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[st][z], sc[t], 0, 0, 0);
                }
            const bool whole = tok + PAGE - 1 <= w_min &&
                               (a.window == 0 || tok > w_max - a.window || tok + PAGE <= a.sink);
            float top = NEG_INF;
            if (!whole) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = tok + 32 * t + 16 * (e >> 3) + 8 * g + (e & 7);
                        sc[t][e] = sight.sees(j) ? sc[t][e] : NEG_INF;
                    }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[t][e]);
            top = pair_max(top) * a.scale2;
            const bool grown = top > mx + SLACK;
            if (__any(grown)) {   // a row's steps follow from the row alone: the others' factor is 1
                top = grown ? top : mx;
                const float by = grown ? __builtin_amdgcn_exp2f(mx - top) : 1.f;
                sum *= by;
#pragma unroll
                for (int u = 0; u < D / 32; ++u) o[u] *= by;
                mx = top;
            }
            const float ref = mx == NEG_INF ? 0.f : mx;
            bf16x8 pf[4][NP];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(sc[t][e], a.scale2, -ref));
                    sum += p;
                    bf16 parts[NP];
                    split_bf16<NP>(p, parts);
#pragma unroll
                    for (int z = 0; z < NP; ++z) pf[2 * t + (e >> 3)][z][e & 7] = parts[z];
                }
#pragma unroll
            for (int u = 0; u < D / 32; ++u)
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4) {
                    const bf16x8 vf = *reinterpret_cast<const bf16x8*>(&vb[(32 * u + m) * VS + 16 * k4 + 8 * g]);
#pragma unroll
                    for (int z = 0; z < NP; ++z)
                        o[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[k4][z], o[u], 0, 0, 0);
                }
        }
        if (more) stage(buf ^ 1, n + KW);
        __syncthreads();
    }
    sum += __shfl_xor(sum, 32, 64);
    if constexpr (KW > 1) {   // join the waves of a row tile, in the pages' place
        float* ml = reinterpret_cast<float*>(kv);            // [WAVES][32][2]
        float* acc = ml + WAVES * 64;                        // [WAVES / 2][32][D + 4]
        static_assert(sizeof(kv) >= 4 * (WAVES * 64 + WAVES / 2 * 32 * (D + 4)), "the join fits the pages' place");
        if (g == 0) {
            ml[(w * 32 + m) * 2] = mx;
            ml[(w * 32 + m) * 2 + 1] = sum;
        }
        __syncthreads();
        const int w0 = w / KW * KW;
        float top = NEG_INF, total = 0.f;
#pragma unroll
        for (int z = 0; z < KW; ++z) top = fmaxf(top, ml[((w0 + z) * 32 + m) * 2]);
        const float ref = top == NEG_INF ? 0.f : top;
#pragma unroll
        for (int z = 0; z < KW; ++z)
            total += ml[((w0 + z) * 32 + m) * 2 + 1] * __builtin_amdgcn_exp2f(ml[((w0 + z) * 32 + m) * 2] - ref);
        const float by = __builtin_amdgcn_exp2f(mx - ref);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) o[u] *= by;
        mx = top;
        sum = total;
#pragma unroll
        for (int half = KW / 2; half >= 1; half /= 2) {
            float* at = acc + ((w / KW * (KW / 2) + kw % half) * 32 + m) * (D + 4) + 4 * g;
            if (kw >= half && kw < 2 * half) {
#pragma unroll
                for (int u = 0; u < D / 32; ++u)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        *reinterpret_cast<f32x4*>(at + 32 * u + 8 * z) =
                            f32x4{o[u][4 * z], o[u][4 * z + 1], o[u][4 * z + 2], o[u][4 * z + 3]};
            }
            __syncthreads();
            if (kw < half) {
#pragma unroll
                for (int u = 0; u < D / 32; ++u)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const f32x4 y = *reinterpret_cast<const f32x4*>(at + 32 * u + 8 * z);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[u][4 * z + e] += y[e];
                    }
            }
            __syncthreads();
        }
    }
    if (!live_row || kw != 0) return;
    if (tl.ranges == 1) {
        const float by = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        typedef T Four __attribute__((ext_vector_type(4)));
        T* out = reinterpret_cast<T*>(a.out) + (((long)b * a.T + r / a.G) * HG + h * a.G + r % a.G) * D + 4 * g;
#pragma unroll
        for (int u = 0; u < D / 32; ++u)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                Four y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (T)(o[u][4 * z + e] * by);
                *reinterpret_cast<Four*>(out + 32 * u + 8 * z) = y;
            }
    } else {
        const size_t at = (((size_t)b * c.H + h) * a.splits + split) * ((size_t)a.T * a.G) + r;
#pragma unroll
        for (int u = 0; u < D / 32; ++u)
#pragma unroll
            for (int z = 0; z < 4; ++z)
                *reinterpret_cast<f32x4*>(a.part + at * D + 32 * u + 8 * z + 4 * g) =
                    f32x4{o[u][4 * z], o[u][4 * z + 1], o[u][4 * z + 2], o[u][4 * z + 3]};
        if (g == 0) {
            a.ml[2 * at] = mx;
            a.ml[2 * at + 1] = sum;
        }
    }
}

// One launch instead of ranges: head widths up to which calls take it, and
// pages up to which single tokens do (ONE_PAGES_MID: 65 to 256 workgroups).
constexpr int ONE_DIM = 128, ONE_PAGES = 24, ONE_PAGES_MID = 40;

// Joins the ranges of a row, a few lanes per range so that several are read
// at a time: a wave per row (ONE), or where there are many ranges a workgroup
// per row and slice of its dims (2 x 32 rows of 256 dims in 256 ranges,
// 17 MB: 9 us against 16 with a workgroup a row).
template <class T, int D, bool ONE>
__global__ __launch_bounds__(256) void combine_kernel(AttendArgs a) {
    constexpr int SL = ONE ? D : D % 64 ? 32 : 64;                        // dims of a slice
    constexpr int LP = SL / 4, GW = 64 / LP, GROUPS = ONE ? GW : 4 * GW;   // lanes of a range, ranges at a time
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, h = blockIdx.y, b = blockIdx.z;
    const int r = ONE ? blockIdx.x * 4 + w : blockIdx.x / (D / SL), d0 = ONE ? 0 : blockIdx.x % (D / SL) * SL;
    const Tile tl = tile_of(a, b, uniform(a.seqs ? a.seqs[b] : b), r / a.tile_rows);
    const bool out_of = r >= tl.rows || tl.ranges == 1;
    if (!ONE && out_of) return;
    const int ranges = out_of ? 0 : tl.ranges;
    const size_t rows = (size_t)a.T * a.G, at0 = ((size_t)b * a.c.H + h) * a.splits * rows + r;
    __shared__ __align__(16) float acc[4 * GW][SL + 4];
    __shared__ float sums[4 * GW];
    float top = NEG_INF;
    for (int s = lane; s < ranges; s += 64) top = fmaxf(top, a.ml[2 * (at0 + s * rows)]);
#pragma unroll
    for (int x = 32; x > 0; x /= 2) top = fmaxf(top, __shfl_xor(top, x, 64));
    const float ref = top == NEG_INF ? 0.f : top;
    const int grp = (ONE ? 0 : w * GW) + lane / LP, col = lane % LP * 4;
    if (lane < GW * LP) {
        f32x4 o = {0, 0, 0, 0};
        float total = 0.f;
#pragma unroll 4
        for (int s = grp; s < ranges; s += GROUPS) {
            const size_t at = at0 + s * rows;
            const float by = __builtin_amdgcn_exp2f(a.ml[2 * at] - ref);
            total += a.ml[2 * at + 1] * by;
            o += *reinterpret_cast<const f32x4*>(a.part + at * D + d0 + col) * by;
        }
        *reinterpret_cast<f32x4*>(&acc[w * GW + lane / LP][col]) = o;
        if (col == 0) sums[w * GW + lane / LP] = total;
    }
    __syncthreads();
    if (out_of) return;
    T* out = reinterpret_cast<T*>(a.out) + (((long)b * a.T + r / a.G) * a.c.H * a.G + h * a.G + r % a.G) * D + d0;
    const int z0 = ONE ? w * GW : 0;
    for (int dim = ONE ? lane : threadIdx.x; dim < SL; dim += ONE ? 64 : 256) {
        float y = 0.f, total = 0.f;
#pragma unroll
        for (int z = 0; z < GROUPS; ++z) {
            y += acc[z0 + z][dim];
            total += sums[z0 + z];
        }
        out[dim] = (T)(y * (total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total)));
    }
}

// How a call is launched: which kernel, how many tiles of rows, and into how
// many ranges the sequences are divided.
struct AttendPlan {
    bool wide;       // attend_tiles_kernel, else attend_rows_kernel
    int kw;          // its KW
    int waves, tile_rows, tiles, splits, least;
};
// Ranges, at most: as many workgroups as the compute units take at a time in
// bf16 (tiles; in fp32 a unit takes one from width 96 on, so two rounds), or
// several rounds of them, which even out ragged lengths (rows: 48 sequences of
// 2000 to 30000 tokens, 32 heads on 8 of 128, 336 us with 1024 workgroups, 289
// us with 8192), and at least TILE_PAGES or ROW_PAGES pages a range.  Grows with `pages`, so the workspace is that of the longest sequence
// whatever max_len a call names.
constexpr int TILE_PAGES = 4, ROW_PAGES = 8;
static int most_ranges(const tm_cache* c, bool wide, long groups, long pages) {
    long s = (wide ? (c->d <= 128 ? 512 : 256) : 8192) / groups;
    const long most = wide ? (pages + TILE_PAGES - 1) / TILE_PAGES : (pages + ROW_PAGES - 1) / ROW_PAGES;
    if (s > most) s = most;
    if (s > 256) s = 256;
    return s < 1 ? 1 : (int)s;
}
static AttendPlan attend_plan(const tm_cache* c, int batch, int n_tokens, int heads, long max_len, bool f32) {
    AttendPlan p;
    const long rows = (long)n_tokens * (heads / c->H), pages = (max_len + PAGE - 1) / PAGE;
    p.wide = rows > 64;
    p.kw = 1;
    p.waves = 4;
    p.tile_rows = p.wide ? 128 : rows > 32 ? 64 : rows > 16 ? 32 : 16;
    p.tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
    const long groups = (long)batch * c->H * p.tiles;
    // Rows: two pages a wave while the chip is not full, more as soon as it is,
    // since every range costs a start and a place in the join.
    const long eights = groups * ((pages + 7) / 8);
    p.least = p.wide ? TILE_PAGES : eights <= 1024 ? ROW_PAGES : eights <= 4096 ? 2 * ROW_PAGES : 4 * ROW_PAGES;
    p.splits = most_ranges(c, p.wide, groups, pages);
    const long fit = (pages + p.least - 1) / p.least;
    if (p.splits > fit) p.splits = fit < 1 ? 1 : (int)fit;
    // One launch of eight waves, which share the sequence among them, instead
    // of ranges and their join (registers and LDS allow it up to width 128).
    // Rows: where there would be ranges (more than 8 pages) but few of them.
    // Eight waves against four with ranges, us on the GPU, single tokens in bf16:
    //   key heads x
    //   entries          width   200       1000       1500       2064       4000 tokens
    //   12               64      5.6/5.5   7.7/9.4    8.8/9.4    10.2/9.5   15.0/9.6
    //                    128     7.6/7.4   12.6/11.9  15.4/12.1  18.1/12.3  28/12
    //   128              64      5.8/5.5   7.9/9.8    9.7/11.7   12.0/14.1  17.5/18.6
    //                    128     7.8/7.3   13.9/13.6  17.1/18.9  19.8/24.2  31/31
    //   384              64      7.2/6.5   13.5/16.8  17.6/20.4  22.2/25.6  37/38
    //                    128     14/10     28/27      35/33      43/43      90/83
    // fp32 is 10 to 40% longer and turns at the same sizes, but for 12 and 64
    // key heads of width 64 and 96, from 1500 tokens on (11.1 against 10.4).
    // Tiles: by the time that 256 workgroups take for a page, that as many of
    // eight waves take for KW pages, and of the ranges' join (its launch and the
    // partial results' way out and in), fitted to 480 calls measured in both
    // forms; the choice is 2% slower than the better one on average, 1.5 times
    // at most.  us on the GPU, eight waves against four:
    //   heads x entries  queries, of   width 64: bf16, fp32   width 128: bf16, fp32
    //   6 x 2            512, 1040     16/19      24/24      29/26      54/35
    //   6 x 2            1024, 2064    24/31      37/42      48/38      96/70
    //   6 x 2            2048, 2048    27/42      40/60      45/51      93/83
    //   8 x 2 (2 key)    512, 4096     36/32      60/47      77/43      163/85
    //   8 x 2 (2 key)    2048, 2048    29/50      44/75      45/61      93/100
    //   8 x 8            128, 128      8.7/8.8    11/12      11/11      18/17
    //   8 x 8            128, 4096     36/30      58/46      78/41      170/86
    //   32 x 8 (8 key)   1024, 2064    277/150    433/345    299/249    660/757
    if (c->d > ONE_DIM) return p;
    if (!p.wide) {
        const int most = groups > 64 && groups <= 256 ? ONE_PAGES_MID : c->d < ONE_DIM ? ONE_PAGES : 0;
        if (rows > 16 || pages <= ROW_PAGES || pages > most) return p;
        p.waves = 8;
    } else {
        const int kw = c->d <= 64 ? 4 : 2, tile = 256 / kw;
        const long tiles = (rows + tile - 1) / tile, rounds = ((long)batch * c->H * tiles + 255) / 256;
        const double page = (0.3 + c->d * 0.0043) * (f32 ? 2.6 : 1.0);   // us
        const double step = page * (c->d <= 64 ? (f32 ? 2.2 : 3.0) : (f32 ? 1.6 : 2.3));
        const double part = (double)groups * p.tile_rows * p.splits * (c->d + 2) * 8;   // bytes, written and read
        const double here = (double)(rounds * ((pages + kw - 1) / kw)) * step;
        const double there = (double)((groups * p.splits + 255) / 256 * ((pages + p.splits - 1) / p.splits)) * page +
                             (p.splits > 1 ? 3.3 + part * 0.35e-6 : 0.0);
        if (here > there) return p;
        p.waves = 8;
        p.kw = kw;
        p.tile_rows = tile;
        p.tiles = (int)tiles;
    }
    p.splits = 1;
    p.least = 1 << 20;
    return p;
}

size_t attend_workspace(const tm_cache* c, int batch, int n_tokens, int heads) {
    if (heads % c->H != 0 || batch == 0 || n_tokens == 0) return 0;
    // the most ranges that any max_len leads to
    const long rows = (long)n_tokens * (heads / c->H), tile = rows > 64 ? 128 : rows > 32 ? 64 : rows > 16 ? 32 : 16;
    const int splits = most_ranges(c, rows > 64, (long)batch * c->H * ((rows + tile - 1) / tile), c->seq_pages);
    if (splits == 1) return 0;
    return ((size_t)batch * c->H * splits * rows * (c->d + 2) * 4 + 511) / 256 * 256;
}

template <class T>
static hipError_t launch_attend(const tm_cache* c, const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
    hipError_t e = timed_attn(st, [&] {
        return for_head_dim(c->d, [&](auto D) {
            if (p.wide) {
                const dim3 grid((unsigned)(p.tiles * p.splits * c->H), 1, (unsigned)a.B);
                if constexpr (D() <= 128) {
                    if (p.kw > 1) {
                        launch_k(attend_tiles_kernel<T, D(), 8, D() <= 64 ? 4 : 2>, grid, dim3(512), 0, st, a);
                        return hipGetLastError();
                    }
                }
                launch_k(attend_tiles_kernel<T, D(), 4, 1>, grid, dim3(256), 0, st, a);
                return hipGetLastError();
            }
            const dim3 grid((unsigned)(p.tiles * p.splits), (unsigned)c->H, (unsigned)a.B);
            if constexpr (D() <= ONE_DIM) {
                if (p.waves == 8) {
                    launch_k(attend_rows_kernel<T, D(), 1, 1, 8>, grid, dim3(512), 0, st, a);
                    return hipGetLastError();
                }
            }
            // more rows: tiles of other waves, which read the same pages from L2, or
            // at width 256, where a wave is alone on its SIMD anyway, two tiles a
            // wave (8 x 60000 tokens, 24 rows on 8 heads, bf16: width 128 250 us
            // against 260, width 256 496 against 443)
            constexpr int RT = D() < 256 ? 1 : 2;
            if (p.tile_rows == 16) launch_k(attend_rows_kernel<T, D(), 1, 1, 4>, grid, dim3(256), 0, st, a);
            else if (p.tile_rows == 32) launch_k(attend_rows_kernel<T, D(), 2 / RT, RT, 4>, grid, dim3(256), 0, st, a);
            else launch_k(attend_rows_kernel<T, D(), 4 / RT, RT, 4>, grid, dim3(256), 0, st, a);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || p.splits == 1) return e;
    return timed_attn(st, [&] {
        return for_head_dim(c->d, [&](auto D) {
            const int rows = a.T * a.G;
            if (p.splits > 16)
                launch_k(combine_kernel<T, D(), false>, dim3((unsigned)(rows * (D() / (D() % 64 ? 32 : 64))), (unsigned)c->H, (unsigned)a.B),
                         dim3(256), 0, st, a);
            else
                launch_k(combine_kernel<T, D(), true>, dim3((unsigned)((rows + 3) / 4), (unsigned)c->H, (unsigned)a.B), dim3(256),
                         0, st, a);
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
    const AttendPlan p = attend_plan(c, batch, n_tokens, heads, max_len > 0 && max_len < most ? max_len : most,
                                     dtype == TM_F32);
    // a launch has fewer than 2^32 threads along an axis
    if ((long)p.tiles * p.splits * c->H * 64 * p.waves >= 1L << 32) return TM_ERR_INVALID;
    if (p.splits > 1 && !ptr_ok(workspace, 256)) return TM_ERR_INVALID;
    const int G = heads / c->H;
    const size_t rows = (size_t)batch * c->H * p.splits * n_tokens * G;
    float* part = static_cast<float*>(workspace);
    AttendArgs a{cache_view(c, const_cast<void*>(blob)), seqs, counts, q, q_batch, q_token, out, batch, n_tokens, G,
                 fmaxf(fabsf(score_scale) * 1.44269504088896340736f, 1.2e-38f), score_scale < 0 ? -1.f : 1.f,
                 window < most ? window : (int)most, sink < most ? sink : (int)most, p.splits, p.least, p.tile_rows,
                 part, part + rows * c->d};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == TM_F32 ? launch_attend<float>(c, a, p, st) : launch_attend<bf16>(c, a, p, st);
    return e == hipSuccess ? TM_OK : TM_ERR_HIP;
}
