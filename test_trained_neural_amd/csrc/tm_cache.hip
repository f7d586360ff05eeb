// The paged 8-bit key/value cache (include/tm_attention.h): writing tokens,
// reading them back, and the bookkeeping of pages (fork, free, compact).
//
// Everything that decides which page a token goes to runs on the device, in
// one workgroup per call (append, compact), one per entry (fork, free) or all
// of them alike (an append of a few tokens), so no call waits for the host
// and every call can be captured into a graph.
// Pages are found by a scan of the reference counts from a lower bound on the
// first free one, in ascending order: which page an entry gets follows from
// the bookkeeping alone, and no result depends on the order of atomics.
#include <new>
#include <type_traits>

#include "tm_cache.h"

namespace tmk {

constexpr int PLAN_THREADS = 1024;
constexpr int MAX_SEQS = 8192;

// What the append's plan leaves for its write, per entry of the call.
struct AppendPlan {
    int old, n;      // tokens held before, tokens to write
    int copy_from;   // the shared page that the entry's last page is a copy of, or -1
    int page;        // the page of token `old`
};

struct AppendArgs {
    CacheView c;
    const int* seqs;
    const int* counts;
    const void* k;
    const void* v;
    long kb, kt, vb, vt;
    int B, T;
    AppendPlan* plan;
};

// Inclusive sum over the workgroup; every thread gets the total too.
template <int THREADS> __device__ __forceinline__ int block_scan(int x, int* wave_sums, int& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int s = x;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const int y = __shfl_up(s, o, 64);
        if (lane >= o) s += y;
    }
    __syncthreads();   // the sums of an earlier scan have been read
    if (lane == 63) wave_sums[w] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
        const int y = wave_sums[i];
        if (i < w) before += y;
        all += y;
    }
    total = all;
    return s + before;
}

// One workgroup decides the whole append: which entries are served, which
// pages they get, and the lengths and reference counts after it.
//   1. equal entries: the first one's index wins its sequence (atomicMin in
//      LDS: the least index, whatever the order);
//   2. each entry's pages: those its tokens begin, and one for a copy of a
//      shared last page ("shared" as before the call); an inclusive sum over
//      the entries gives each its ranks among the free pages;
//   3. a scan over the reference counts finds the free pages in order; page
//      of rank r goes to the entry whose ranks hold r (binary search);
//   4. entries within the free pages take effect.
// Bound by the latency of its dependent reads (list, length, last page, its
// references); the first reference counts of the scan are read beside them
// (8 or 64 entries: 5.5 us).  The write that follows has the bytes.
template <int THREADS, int ENTRIES>
__global__ __launch_bounds__(THREADS) void append_plan_kernel(AppendArgs a) {
    const CacheView& c = a.c;
    constexpr int PER = ENTRIES / THREADS, STEP = THREADS * 4;
    __shared__ int ranks[MAX_SEQS];   // first the winners of 1, then the inclusive sums of 2
    __shared__ short copies[ENTRIES]; // 1: the entry's first page is a copy; 2: its first page is new
    __shared__ int olds[ENTRIES <= 256 ? ENTRIES : 1];
    __shared__ int wave_sums[THREADS / 64];
    __shared__ int flags, hint;
    const int tid = threadIdx.x;
    const int from = min(max(c.status[1], 0), c.n_pages) / 4 * 4;
    auto free_of = [&](int p) {   // bit e: page p + e is free
        int r[4], f = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = p + e < c.n_pages ? c.refs[p + e] : 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) f |= (r[e] <= 0) << e;
        return f;
    };
    int free4 = free_of(from + tid * 4);
    if (tid == 0) {
        flags = 0;
        hint = 0x7fffffff;
    }
    auto seq_of = [&](int i) { return a.seqs ? a.seqs[i] : i; };
    int seq[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = tid + j * THREADS;
        seq[j] = i < a.B ? seq_of(i) : -1;
        if ((unsigned)seq[j] < (unsigned)c.n_seqs) ranks[seq[j]] = 0x7fffffff;
        else seq[j] = -1;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (seq[j] >= 0) atomicMin(&ranks[seq[j]], tid + j * THREADS);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = tid + j * THREADS;
        if (i < a.B && (seq[j] < 0 || ranks[seq[j]] != i)) {
            atomicOr(&flags, TM_CACHE_BAD_ENTRY);
            seq[j] = -1;
        }
    }
    __syncthreads();
    int base = 0;
    AppendPlan plan[PER];
    int before[PER], incl[PER];   // an entry's ranks: before .. incl - 1
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = tid + j * THREADS, s = seq[j];
        AppendPlan p{0, 0, -1, -1};
        int need = 0;
        if (s >= 0) {
            p.old = c.length(s);
            p.n = a.counts ? min(max(a.counts[i], 0), a.T) : a.T;
            if (p.n > c.seq_pages * PAGE - p.old) {
                atomicOr(&flags, TM_CACHE_FULL);
                p.n = 0;
            }
            if (p.n > 0 && p.old % PAGE) {
                p.page = c.page_at(s, p.old / PAGE);
                if (!c.page_ok(p.page)) {
                    atomicOr(&flags, TM_CACHE_BAD_ENTRY);
                    p.n = 0;
                } else if (c.refs[p.page] > 1) {
                    p.copy_from = p.page;
                }
            }
            if (p.n > 0) need = (p.old + p.n + PAGE - 1) / PAGE - (p.old + PAGE - 1) / PAGE + (p.copy_from >= 0);
        }
        int total;
        incl[j] = base + block_scan<THREADS>(need, wave_sums, total);
        before[j] = incl[j] - need;
        base += total;
        plan[j] = p;
        if (i < a.B) {
            ranks[i] = incl[j];
            copies[i] = p.copy_from >= 0 ? 1 : p.n > 0 && p.old % PAGE == 0 ? 2 : 0;
            if constexpr (ENTRIES <= 256) olds[i] = p.old;
            a.plan[i] = p;
        }
    }
    const int want = base;   // pages of the whole call
    __syncthreads();
    int found = 0;           // free pages seen
    if (want > 0) {
        for (int p0 = from; p0 < c.n_pages && found < want; p0 += STEP) {
            const int p = p0 + tid * 4;
            if (p0 != from) free4 = free_of(p);
            int total;
            const int n4 = __popc(free4);
            int r = found + block_scan<THREADS>(n4, wave_sums, total) - n4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!(free4 >> e & 1)) continue;
                if (r < want) {
                    int lo = 0, hi = a.B - 1;   // the first entry whose inclusive sum is above r
                    while (lo < hi) {
                        const int mid = (lo + hi) / 2;
                        if (ranks[mid] > r) hi = mid;
                        else lo = mid + 1;
                    }
                    int old;
                    if constexpr (ENTRIES <= 256) old = olds[lo];
                    else old = a.plan[lo].old;
                    const int nth = r - (lo ? ranks[lo - 1] : 0), kind = copies[lo];
                    const int slot = (kind == 1 ? old / PAGE : (old + PAGE - 1) / PAGE) + nth;
                    c.table[(size_t)seq_of(lo) * c.seq_pages + slot] = p + e;
                    c.refs[p + e] = 1;
                    if (kind && nth == 0) a.plan[lo].page = p + e;
                    if (r == want - 1) hint = p + e + 1;
                }
                ++r;
            }
            found += total;
        }
        __threadfence_block();
    }
    __syncthreads();
    const int have = min(found, want);
    if (tid == 0 && have < want) hint = c.n_pages;   // every free page was taken (or is given back below)
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = tid + j * THREADS, s = seq[j];
        AppendPlan& p = plan[j];
        if (i >= a.B || p.n == 0) continue;
        if (incl[j] > before[j] && incl[j] > have) {   // not enough pages: those taken so far go back
            atomicOr(&flags, TM_CACHE_NO_PAGES);
            const int first = p.copy_from >= 0 ? p.old / PAGE : (p.old + PAGE - 1) / PAGE;
            for (int r = before[j]; r < have; ++r) {
                const int page = c.table[(size_t)s * c.seq_pages + first + r - before[j]];
                c.refs[page] = 0;
                atomicMin(&hint, page);
            }
            if (p.copy_from >= 0 && have > before[j]) c.table[(size_t)s * c.seq_pages + first] = p.copy_from;
            a.plan[i].n = 0;
            continue;
        }
        c.lengths[s] = p.old + p.n;
        if (p.copy_from >= 0 && atomicSub(&c.refs[p.copy_from], 1) == 1) atomicMin(&hint, p.copy_from);
    }
    __syncthreads();
    if (tid == 0) {
        if (want > 0) c.status[1] = min(hint, c.n_pages);
        if (flags) c.status[0] |= flags;
    }
}

__device__ __forceinline__ float finite_or_zero(float x, bool& bad) {
    if (!(fabsf(x) < __builtin_inff())) {
        bad = true;
        return 0.f;
    }
    return x;
}

// The least e with amax <= 448 2^e (448 = 1.75 * 2^8), in the stored range.
__device__ __forceinline__ int block_exponent(float amax) {
    const unsigned u = __builtin_bit_cast(unsigned, amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0);
    return min(max(e, CACHE_E_MIN), CACHE_E_MAX);
}
__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (unsigned)(e + 127) << 23); }

__device__ __forceinline__ float to_range(float x) { return fminf(fmaxf(x, -448.f), 448.f); }
// four e4m3 codes of values already divided by their scale
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(to_range(a), to_range(b), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(to_range(c), to_range(d), w, true);
    return (unsigned)w;
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f32x4 values4(unsigned w) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return f32x4{a[0], a[1], b[0], b[1]};
}
// codes of a grown block: times 2^(old exponent - new one), rounded again
__device__ __forceinline__ unsigned shift4(unsigned w, float by) {
    const f32x4 x = values4(w);
    return codes4(x[0] * by, x[1] * by, x[2] * by, x[3] * by);
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int o = 32; o > 0; o /= 2) x = fmaxf(x, __shfl_xor(x, o, 64));
    return x;
}

// A wave writes what a call has for block w of page `page` (the entry's
// slot-th) and head h: the block's new tokens, and, where the page is a copy,
// what the shared page holds.  Keys: a lane takes 8 consecutive elements of a
// token.  Values, whose tokens are innermost: a lane takes two neighbouring
// dims of all 16 tokens (4 or 8 bytes a lane and token, so a token's row is
// read whole) and stores the block's 16 codes of a dim at once; the page's
// 64-byte row of a dim is made of four waves' pieces.  All tokens are read up
// front, once, and stay as they are in registers through the wave's reduction
// to the block's largest magnitude.
template <class T, int D>
__device__ __forceinline__ void write_block(const AppendArgs& a, const AppendPlan& p, int b, int h, int slot, int page,
                                            int w, bool copied) {
    const CacheView& c = a.c;
    const int lane = threadIdx.x & 63;
    const int b0 = slot * PAGE + w * BLOCK, end = p.old + p.n;   // the block's first token
    const int lo = max(p.old, b0), hi = min(end, b0 + BLOCK);    // the new tokens in it
    if (lo >= hi && !copied) return;
    const T* kx = reinterpret_cast<const T*>(a.k) + b * a.kb + (long)h * D;
    const T* vx = reinterpret_cast<const T*>(a.v) + b * a.vb + (long)h * D;

    typedef T Two __attribute__((ext_vector_type(2)));
    constexpr int KI = BLOCK * D / 8 / 64, VI = (D / 2 + 63) / 64;
    // bf16 tokens are read past the caches: nothing reads them again here (8
    // prompts of up to 4096: 36.6 us against 38.5; of 512, which the caches
    // hold: the same; fp32's 32 bytes a lane: 15.6 against 14.4 for 3 of 2048)
    auto get2 = [](const T* x) {
        const auto* p = reinterpret_cast<const Two*>(x);
        if constexpr (sizeof(T) == 2) return __builtin_nontemporal_load(p);
        else return *p;
    };
    auto get8 = [](const T* x) {
        if constexpr (sizeof(T) == 2) return __builtin_nontemporal_load(reinterpret_cast<const bf16x8*>(x));
        else return ld8(x);
    };
    decltype(ld8(kx)) kr[KI];
    Two vr[VI][BLOCK];
#pragma unroll
    for (int it = 0; it < KI; ++it) {
        const int u = it * 64 + lane, t = u / (D / 8), col = u % (D / 8) * 8;
        kr[it] = {};
        if (b0 + t >= lo && b0 + t < hi) kr[it] = get8(kx + (long)(b0 + t - p.old) * a.kt + col);
    }
#pragma unroll
    for (int it = 0; it < VI; ++it) {
        const int dim = (it * 64 + lane) * 2;
#pragma unroll
        for (int t = 0; t < BLOCK; ++t) {
            vr[it][t] = Two{(T)0.f, (T)0.f};
            if (dim < D && b0 + t >= lo && b0 + t < hi)
                vr[it][t] = get2(vx + (long)(b0 + t - p.old) * a.vt + dim);
        }
    }
    const int from = copied ? p.copy_from : page;   // where the block's present codes are
    const bool begun = lo > b0 && lo < hi;          // it holds earlier tokens, and gets new ones
    const size_t at = c.head_at(page, h), at0 = c.head_at(from, h);
    const bool use = begun || lo >= hi;             // the present scales matter
    const int had_k = use ? (int)c.scales[at0 * 8 + w] - 127 : 0, had_v = use ? (int)c.scales[at0 * 8 + 4 + w] - 127 : 0;
    // bytes of the block's 16 that take new codes; around them the present ones
    // stay, so a block that is not written whole is read first
    const unsigned fresh = lo < hi ? ((1u << (hi - b0)) - 1) & ~((1u << (lo - b0)) - 1) : 0;
    const bool whole = fresh == 0xffffu;
    uint4 was[VI][2];
    if (!whole) {
#pragma unroll
        for (int it = 0; it < VI; ++it)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int dim = (it * 64 + lane) * 2 + z;
                if (dim < D) was[it][z] = *reinterpret_cast<const uint4*>(c.v + (at0 * D + dim) * PAGE + w * BLOCK);
            }
    }
    bool bad = false;
    // the block's new exponent, and what its present codes are multiplied by
    auto settle = [&](float top, int had, float& by, float& shift) {
        int e = had;
        if (lo < hi) {
            e = block_exponent(wave_max(top));
            if (begun) e = max(e, had);
        }
        by = pow2(-e);
        shift = begun && e > had ? pow2(max(had - e, -126)) : 1.f;
        return (unsigned char)(e + 127);
    };

    // ---- keys ----
    {
        const unsigned char* src = c.k + (at0 * PAGE + w * BLOCK) * D;
        unsigned char* dst = c.k + (at * PAGE + w * BLOCK) * D;
        float top = 0.f;
#pragma unroll
        for (int it = 0; it < KI; ++it)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(finite_or_zero((float)kr[it][e], bad)));
        float by, shift;
        const unsigned char scale = settle(top, had_k, by, shift);
#pragma unroll
        for (int it = 0; it < KI; ++it) {
            const int u = it * 64 + lane, t = u / (D / 8), col = u % (D / 8) * 8;
            uint2 o;
            if (b0 + t >= lo && b0 + t < hi) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = finite_or_zero((float)kr[it][e], bad) * by;
                o.x = codes4(x[0], x[1], x[2], x[3]);
                o.y = codes4(x[4], x[5], x[6], x[7]);
                *reinterpret_cast<uint2*>(dst + t * D + col) = o;
            } else if (copied || (shift != 1.f && b0 + t < lo)) {
                o = *reinterpret_cast<const uint2*>(src + t * D + col);
                if (shift != 1.f && b0 + t < lo) {
                    o.x = shift4(o.x, shift);
                    o.y = shift4(o.y, shift);
                }
                *reinterpret_cast<uint2*>(dst + t * D + col) = o;
            }
        }
        if (lane == 0) c.scales[at * 8 + w] = scale;
    }
    // ---- values ----
    {
        float top = 0.f;
#pragma unroll
        for (int it = 0; it < VI; ++it)
#pragma unroll
            for (int t = 0; t < BLOCK; ++t)
#pragma unroll
                for (int z = 0; z < 2; ++z) top = fmaxf(top, fabsf(finite_or_zero((float)vr[it][t][z], bad)));
        float by, shift;
        const unsigned char scale = settle(top, had_v, by, shift);
#pragma unroll
        for (int it = 0; it < VI; ++it) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int dim = (it * 64 + lane) * 2 + z;
                if (dim >= D) continue;
                unsigned o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = finite_or_zero((float)vr[it][4 * q + e][z], bad) * by;
                    o[q] = codes4(x[0], x[1], x[2], x[3]);
                }
                if (!whole) {
                    const unsigned old4[4] = {was[it][z].x, was[it][z].y, was[it][z].z, was[it][z].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const unsigned n4 = fresh >> (4 * q) & 15;   // spread to bytes
                        const unsigned m = (n4 & 1 ? 0xffu : 0u) | (n4 & 2 ? 0xff00u : 0u) | (n4 & 4 ? 0xff0000u : 0u) |
                                           (n4 & 8 ? 0xff000000u : 0u);
                        unsigned keep = old4[q];
                        if (shift != 1.f) {   // the earlier tokens only: bytes below lo
                            const int n = min(max(lo - b0 - 4 * q, 0), 4);
                            const unsigned below = n == 4 ? ~0u : (1u << (8 * n)) - 1;
                            keep = (shift4(keep, shift) & below) | (keep & ~below);
                        }
                        o[q] = (o[q] & m) | (keep & ~m);
                    }
                }
                *reinterpret_cast<uint4*>(c.v + (at * D + dim) * PAGE + w * BLOCK) = uint4{o[0], o[1], o[2], o[3]};
            }
        }
        if (lane == 0) c.scales[at * 8 + 4 + w] = scale;
    }
    if (__any(bad) && lane == 0) atomicOr(&c.status[0], TM_CACHE_NONFINITE);
}

// One workgroup per page and head, a wave per block.  Bound by the tokens' way
// in: 8 prompts of up to 4096 tokens, 8 heads of 128, bf16, 151 MB in all: 37
// us, 4.1 TB/s.
template <class T, int D>
__global__ __launch_bounds__(256) void append_write_kernel(AppendArgs a) {
    const int b = blockIdx.z, w = threadIdx.x >> 6;
    const AppendPlan p = a.plan[b];
    const int slot = p.old / PAGE + blockIdx.x;
    if (p.n == 0 || slot * PAGE >= p.old + p.n) return;
    const int page = blockIdx.x == 0 ? p.page : a.c.page_at(a.seqs ? a.seqs[b] : b, slot);
    if (a.c.page_ok(page))
        write_block<T, D>(a, p, b, blockIdx.y, slot, page, w, blockIdx.x == 0 && p.copy_from >= 0);
}

// One token of an entry into head h of a page of its own, by a wave.  Where
// the block's scales stay, that is a byte a dim in keys and values each; a
// scale that grows goes the way above.  kr, vr: the token's elements, dims
// lane, lane + 64, ...
template <class T, int D>
__device__ __forceinline__ void write_token(const AppendArgs& a, const AppendPlan& p, int b, int h,
                                            const T (&kr)[(D + 63) / 64], const T (&vr)[(D + 63) / 64]) {
    const CacheView& c = a.c;
    const int lane = threadIdx.x & 63;
    constexpr int IT = (D + 63) / 64;
    const int tok = p.old % PAGE, w = tok / BLOCK;
    const size_t at = c.head_at(p.page, h);
    bool bad = false;
    float topk = 0.f, topv = 0.f;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        topk = fmaxf(topk, fabsf(finite_or_zero((float)kr[it], bad)));
        topv = fmaxf(topv, fabsf(finite_or_zero((float)vr[it], bad)));
    }
    int ek = block_exponent(wave_max(topk)), ev = block_exponent(wave_max(topv));
    if (tok % BLOCK) {   // the block holds earlier tokens: its scales stay, or grow
        const int had_k = (int)c.scales[at * 8 + w] - 127, had_v = (int)c.scales[at * 8 + 4 + w] - 127;
        if (ek > had_k || ev > had_v) {
            write_block<T, D>(a, p, b, h, p.old / PAGE, p.page, w, false);
            return;
        }
        ek = had_k;
        ev = had_v;
    } else if (lane == 0) {
        c.scales[at * 8 + w] = (unsigned char)(ek + 127);
        c.scales[at * 8 + 4 + w] = (unsigned char)(ev + 127);
    }
    const float bk = pow2(-ek), bv = pow2(-ev);
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int dim = it * 64 + lane;
        if (dim >= D) continue;
        const unsigned o = codes4(finite_or_zero((float)kr[it], bad) * bk, finite_or_zero((float)vr[it], bad) * bv, 0.f, 0.f);
        c.k[(at * PAGE + tok) * D + dim] = (unsigned char)o;
        c.v[(at * D + dim) * PAGE + tok] = (unsigned char)(o >> 8);
    }
    if (__any(bad) && lane == 0) atomicOr(&c.status[0], TM_CACHE_NONFINITE);
}
template <class T, int D>
__device__ __forceinline__ void load_token(const AppendArgs& a, int b, int h, T (&kr)[(D + 63) / 64],
                                           T (&vr)[(D + 63) / 64]) {
#pragma unroll
    for (int it = 0; it < (D + 63) / 64; ++it) {
        const int dim = it * 64 + (threadIdx.x & 63);
        kr[it] = vr[it] = (T)0.f;
        if (dim < D) {
            kr[it] = reinterpret_cast<const T*>(a.k)[b * a.kb + (long)h * D + dim];
            vr[it] = reinterpret_cast<const T*>(a.v)[b * a.vb + (long)h * D + dim];
        }
    }
}

// Calls of one token an entry behind the plan's launch: a workgroup per head.
template <class T, int D>
__global__ __launch_bounds__(256) void append_token_kernel(AppendArgs a) {
    const int b = blockIdx.y, h = blockIdx.x;
    T kr[(D + 63) / 64], vr[(D + 63) / 64];
    load_token<T, D>(a, b, h, kr, vr);
    const AppendPlan p = a.plan[b];
    if (p.n == 0 || !a.c.page_ok(p.page)) return;
    const int wave = threadIdx.x >> 6;
    if (p.copy_from >= 0) write_block<T, D>(a, p, b, h, p.old / PAGE, p.page, wave, true);   // a block a wave
    else if (wave == 0) write_token<T, D>(a, p, b, h, kr, vr);
}

// Calls of a few tokens an entry with the plan, in one launch (a decode step,
// drafts): every workgroup works out the entries' needs (at most two pages
// each) and its own entry's pages for itself, from bookkeeping that no
// workgroup changes; the last of them to be done, by a count in status[2] that
// it sets back, makes the plan's changes.  A wave writes a head's token (ONE:
// one token an entry at most), two its even and odd blocks.  64 entries of 8
// heads, one token: 8 us against 5.5 and 4 in two launches, a call from the
// host 2 to 3 us shorter (with two waves a head as well 10 us: twice the workgroups).
constexpr int STEP_ENTRIES = 256, STEP_TOKENS = 16;
template <class T, int D, bool ONE>
__global__ __launch_bounds__(STEP_ENTRIES) void append_step_kernel(AppendArgs a) {
    static_assert(STEP_TOKENS <= PAGE, "two pages an entry");
    const CacheView& c = a.c;
    const int b = blockIdx.y, i = threadIdx.x, w = threadIdx.x >> 6;
    constexpr int WAVES = ONE ? 1 : 2;   // of a head
    const int h = blockIdx.x * (4 / WAVES) + w / WAVES;
    __shared__ int seqs[STEP_ENTRIES], page_of[2 * STEP_ENTRIES], wave_sums[STEP_ENTRIES / 64];
    __shared__ unsigned listed[MAX_SEQS / 32];   // bit s: sequence s is in the list
    __shared__ int flags, hint, last, doubles, own_rank, own_need;
    __shared__ AppendPlan own;
    const int from = min(max(c.status[1], 0), c.n_pages);
    constexpr int STEP = STEP_ENTRIES * 4;
    auto free_of = [&](int p) {   // bit e: page p + e is free
        int r[4], f = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = p + e < c.n_pages ? c.refs[p + e] : 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) f |= (r[e] <= 0) << e;
        return f;
    };
    const int free4 = free_of(from + i * 4);
    T kr[(D + 63) / 64], vr[(D + 63) / 64];
    if constexpr (ONE)
        if (h < c.H) load_token<T, D>(a, b, h, kr, vr);
    if (i == 0) {
        flags = doubles = 0;
        hint = 0x7fffffff;
    }
    static_assert(MAX_SEQS / 32 == STEP_ENTRIES, "a word a thread");
    listed[i] = 0;
    int s = i < a.B ? (a.seqs ? a.seqs[i] : i) : -1;
    if ((unsigned)s >= (unsigned)c.n_seqs) s = -1;
    seqs[i] = s;
    __syncthreads();
    if (a.seqs) {
        if (s >= 0 && (atomicOr(&listed[s / 32], 1u << (s % 32)) >> (s % 32) & 1)) doubles = 1;
        __syncthreads();
    }
    AppendPlan p{0, 0, -1, -1};
    int flag = i < a.B && s < 0 ? TM_CACHE_BAD_ENTRY : 0, need = 0;
    if (s >= 0) {
        bool twice = false;
        if (doubles)
            for (int j = 0; j < i; ++j) twice |= seqs[j] == s;
        if (twice) flag = TM_CACHE_BAD_ENTRY;
        else {
            p.old = c.length(s);
            p.n = a.counts ? min(max(a.counts[i], 0), a.T) : a.T;
            if (p.n > c.seq_pages * PAGE - p.old) {
                flag = TM_CACHE_FULL;
                p.n = 0;
            }
            if (p.n > 0 && p.old % PAGE) {
                p.page = c.page_at(s, p.old / PAGE);
                if (!c.page_ok(p.page)) {
                    flag = TM_CACHE_BAD_ENTRY;
                    p.n = 0;
                } else if (c.refs[p.page] > 1) {
                    p.copy_from = p.page;
                }
            }
            if (p.n > 0) need = (p.old + p.n + PAGE - 1) / PAGE - (p.old + PAGE - 1) / PAGE + (p.copy_from >= 0);
        }
    }
    int want;
    const int rank = block_scan<STEP_ENTRIES>(need, wave_sums, want) - need;
    if (i == b) {
        own = p;
        own_rank = rank;
        own_need = need;
    }
    __syncthreads();
    // page_of: the first free pages in order, `upto` of them at least, where
    // there are so many; how many there are, `upto` at most.  A thread reads
    // four references, and the last workgroup's second call goes on where its
    // first stopped: behind one low hole and 30000 used pages an append takes
    // 38 us, as the plan of its own launch does (a reference a thread and the
    // whole scan twice: 145).
    int found = 0, next = from;
    auto scan_free = [&](int upto) {
        while (found < upto && next < c.n_pages) {
            const int p = next + i * 4, now4 = next == from ? free4 : free_of(p);
            next += STEP;
            int total;
            const int n4 = __popc(now4);
            int r = found + block_scan<STEP_ENTRIES>(n4, wave_sums, total) - n4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!(now4 >> e & 1)) continue;
                if (r < 2 * STEP_ENTRIES) page_of[r] = p + e;
                ++r;
            }
            found += total;
        }
        __syncthreads();
        return min(found, upto);
    };
    const int upto = own_need > 0 ? own_rank + own_need : 0;
    if (upto == 0 || scan_free(upto) == upto) {
        const int at = upto - own_need;   // rank of the entry's first new page
        const bool begins = own.copy_from >= 0 || own.old % PAGE == 0;   // its tokens' first page is new
        const AppendPlan mine{own.old, own.n, own.copy_from, begins && upto ? page_of[at] : own.page};
        if (h < c.H && mine.n > 0) {
            const bool copied = mine.copy_from >= 0;
            const int first = mine.old / PAGE, after = begins ? at + 1 : at;
            if constexpr (ONE) {
                if (!copied) write_token<T, D>(a, mine, b, h, kr, vr);
                else
                    for (int x = 0; x < PAGE / BLOCK; ++x) write_block<T, D>(a, mine, b, h, first, mine.page, x, true);
            } else {
                int x = mine.old / BLOCK, x1 = (mine.old + mine.n - 1) / BLOCK;
                if (copied) {   // all of the page
                    x = first * (PAGE / BLOCK);
                    x1 = max(x1, x + PAGE / BLOCK - 1);
                }
                for (x += w % WAVES; x <= x1; x += WAVES) {
                    const int slot = x / (PAGE / BLOCK);
                    write_block<T, D>(a, mine, b, h, slot, slot == first ? mine.page : page_of[after], x % (PAGE / BLOCK),
                                      copied && slot == first);
                }
            }
        }
    }

    // What this workgroup needs of the bookkeeping is in its registers (the
    // barrier is behind their use), and it has written none of it: the count
    // orders nothing else, so it needs no fence (with one, a write-back
    // of the L2 each, a launch of 512 workgroups took 22 us instead of 13).
    __syncthreads();
    if (i == 0) {
        const unsigned n = gridDim.x * gridDim.y, before = (unsigned)atomicAdd(&c.status[2], 1);
        last = before == n - 1;
        if (before >= n) atomicOr(&c.status[0], TM_CACHE_BAD_ENTRY);   // the count did not begin at 0
    }
    __syncthreads();
    if (!last) return;
    const int have = want > 0 ? scan_free(want) : 0;
    if (i == 0 && want > 0) hint = have < want ? c.n_pages : page_of[want - 1] + 1;
    __syncthreads();
    if (p.n > 0) {
        const int slot = p.copy_from >= 0 ? p.old / PAGE : (p.old + PAGE - 1) / PAGE;   // of the first new page
        if (rank + need > have && need > 0) {
            flag = TM_CACHE_NO_PAGES;
            if (rank < have) atomicMin(&hint, page_of[rank]);   // not taken
        } else {
            for (int r = 0; r < need; ++r) {
                c.table[(size_t)s * c.seq_pages + slot + r] = page_of[rank + r];
                c.refs[page_of[rank + r]] = 1;
            }
            c.lengths[s] = p.old + p.n;
            if (p.copy_from >= 0 && atomicSub(&c.refs[p.copy_from], 1) == 1) atomicMin(&hint, p.copy_from);
        }
    }
    if (flag) atomicOr(&flags, flag);
    __syncthreads();
    if (i == 0) {
        if (want > 0) c.status[1] = min(hint, c.n_pages);
        if (flags) atomicOr(&c.status[0], flags);
        c.status[2] = 0;
    }
}

struct ReadArgs {
    CacheView c;
    const int* seqs;
    void* k;
    void* v;
    int start, B, T;
};

// The append's mapping backwards: one workgroup per page and head, a wave
// per block.  Bound by its writes: 8 sequences of 4096 tokens, 8 heads of 128,
// bf16, 202 MB in all: 32 us, 6.3 TB/s.
template <class T, int D>
__global__ __launch_bounds__(256) void cache_read_kernel(ReadArgs a) {
    const CacheView& c = a.c;
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int s = a.seqs ? a.seqs[b] : b;
    if ((unsigned)s >= (unsigned)c.n_seqs) return;
    const int slot = a.start / PAGE + blockIdx.x;
    const int b0 = slot * PAGE + w * BLOCK;
    const int lo = max(a.start, b0), hi = (int)min((long)min(c.length(s), b0 + BLOCK), (long)a.start + a.T);
    if (lo >= hi) return;
    const int page = c.page_at(s, slot);
    if (!c.page_ok(page)) return;
    const size_t at = c.head_at(page, h);
    const long row = (long)c.H * D;   // elements between tokens
    T* ko = reinterpret_cast<T*>(a.k) + ((long)b * a.T - a.start) * row + (long)h * D;
    T* vo = reinterpret_cast<T*>(a.v) + ((long)b * a.T - a.start) * row + (long)h * D;
    const float sk = scale_of(c.scales[at * 8 + w]), sv = scale_of(c.scales[at * 8 + 4 + w]);
    typedef T Four __attribute__((ext_vector_type(4)));
    constexpr int IT = BLOCK * D / 4 / 64;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int u = it * 64 + lane, t = u / (D / 4), col = u % (D / 4) * 4;
        if (b0 + t < lo || b0 + t >= hi) continue;
        const f32x4 x = values4(*reinterpret_cast<const unsigned*>(c.k + (at * PAGE + w * BLOCK + t) * D + col));
        Four o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (T)(x[e] * sk);
        *reinterpret_cast<Four*>(ko + (b0 + t) * row + col) = o;
    }
    typedef T Two __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int it = 0; it < (D / 2 + 63) / 64; ++it) {
        const int dim = (it * 64 + lane) * 2;
        if (dim >= D) continue;
        const uint4 x0 = *reinterpret_cast<const uint4*>(c.v + (at * D + dim) * PAGE + w * BLOCK);
        const uint4 x1 = *reinterpret_cast<const uint4*>(c.v + (at * D + dim + 1) * PAGE + w * BLOCK);
        const unsigned w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4 f0 = values4(w0[q]), f1 = values4(w1[q]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = b0 + 4 * q + e;
                if (t < lo || t >= hi) continue;
                *reinterpret_cast<Two*>(vo + t * row + dim) = Two{(T)(f0[e] * sv), (T)(f1[e] * sv)};
            }
        }
    }
}

struct ForkArgs {
    CacheView c;
    const int* src;
    const int* dst;
    int n;
};

// One workgroup per fork.  Which forks are served follows from the lists and
// the lengths before the call alone: a destination must be empty, not listed
// before, and no source; then no workgroup writes what another reads.
// Latency: 4 us for 128 forks.
__global__ __launch_bounds__(256) void fork_kernel(ForkArgs a) {
    const CacheView& c = a.c;
    const int i = blockIdx.x, tid = threadIdx.x;
    __shared__ int refused;
    if (tid == 0) refused = 0;
    __syncthreads();
    const int src = a.src[i], dst = a.dst[i];
    if ((unsigned)src >= (unsigned)c.n_seqs || (unsigned)dst >= (unsigned)c.n_seqs) {
        if (tid == 0) atomicOr(&c.status[0], TM_CACHE_BAD_ENTRY);
        return;
    }
    bool no = false;
    for (int j = tid; j < a.n; j += 256) {
        const int d = a.dst[j];
        no |= (j < i && d == dst) || d == src;
    }
    if (tid == 0) no |= c.lengths[dst] != 0;
    if (no) refused = 1;
    __syncthreads();
    if (refused) {
        if (tid == 0) atomicOr(&c.status[0], TM_CACHE_BAD_ENTRY);
        return;
    }
    const int len = c.length(src), held = (len + PAGE - 1) / PAGE;
    for (int p = tid; p < held; p += 256) {
        const int page = c.page_at(src, p);
        c.table[(size_t)dst * c.seq_pages + p] = page;
        if (c.page_ok(page)) atomicAdd(&c.refs[page], 1);
    }
    if (tid == 0) c.lengths[dst] = len;
}

struct FreeArgs {
    CacheView c;
    const int* seqs;
    const int* keep;
    int n;
};

// One workgroup per entry; an entry whose sequence stands earlier in the list
// is refused, so each sequence's length has one reader and writer.  Latency:
// 4 us for 64 to 128 entries.
__global__ __launch_bounds__(256) void free_kernel(FreeArgs a) {
    const CacheView& c = a.c;
    const int i = blockIdx.x, tid = threadIdx.x;
    const int s = a.seqs ? a.seqs[i] : i;
    __shared__ int twice;
    if (tid == 0) twice = 0;
    __syncthreads();
    bool no = (unsigned)s >= (unsigned)c.n_seqs;
    if (a.seqs)
        for (int j = tid; j < i; j += 256) no |= a.seqs[j] == s;
    if (no) twice = 1;
    __syncthreads();
    if (twice) {
        if (tid == 0) atomicOr(&c.status[0], TM_CACHE_BAD_ENTRY);
        return;
    }
    const int old = c.length(s), keep = a.keep ? min(max(a.keep[i], 0), old) : 0;
    __syncthreads();   // every thread has read the length
    if (tid == 0) c.lengths[s] = keep;
    for (int p = (keep + PAGE - 1) / PAGE + tid; p < (old + PAGE - 1) / PAGE; p += 256) {
        const int page = c.page_at(s, p);
        if (c.page_ok(page) && atomicSub(&c.refs[page], 1) == 1) atomicMin(&c.status[1], page);
    }
}

struct CompactArgs {
    CacheView c;
    int* count;   // [0] pages to move, [1] pages in use
    int* from;    // the i-th used page at or above [1]
    int* to;      // the i-th free page below [1]
    int* map;     // page -> where it goes (used pages at or above [1])
    int d;
};

// One workgroup: the number of pages in use, then the lists of those that
// move and of the holes they move to, both ascending.  Latency of its passes
// over the reference counts: 11 us for 9000 pages.
__global__ __launch_bounds__(PLAN_THREADS) void compact_plan_kernel(CompactArgs a) {
    const CacheView& c = a.c;
    __shared__ int wave_sums[PLAN_THREADS / 64];
    const int tid = threadIdx.x;
    int mine = 0, used;
    for (int p = tid; p < c.n_pages; p += PLAN_THREADS) mine += c.refs[p] > 0;
    block_scan<PLAN_THREADS>(mine, wave_sums, used);
    int moved = 0, holes = 0;
    for (int p0 = 0; p0 < c.n_pages; p0 += PLAN_THREADS * 4) {
        const int p = p0 + tid * 4;
        int pick4 = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (p + e < c.n_pages && (c.refs[p + e] > 0) == (p + e >= used)) pick4 |= 1 << e;
        // free pages below `used` and used pages above it: a group of four may
        // hold both, so both are counted in one sum (16 bits each: at most
        // 4096 in a pass)
        int nh = 0, nm = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            nh += (pick4 >> e & 1) && p + e < used;
            nm += (pick4 >> e & 1) && p + e >= used;
        }
        int total;
        const int sum = block_scan<PLAN_THREADS>(nh | nm << 16, wave_sums, total);
        int rh = holes + (sum & 0xffff) - nh, rm = moved + (sum >> 16) - nm;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!(pick4 >> e & 1)) continue;
            if (p + e < used) a.to[rh++] = p + e;
            else a.from[rm++] = p + e;
        }
        holes += total & 0xffff;
        moved += total >> 16;
    }
    __threadfence_block();
    __syncthreads();
    for (int i = tid; i < moved; i += PLAN_THREADS) a.map[a.from[i]] = a.to[i];
    if (tid == 0) {
        a.count[0] = moved;
        a.count[1] = used;
        c.status[1] = used;
    }
}

// Workgroups below `seq_blocks` rewrite the tables, the others copy pages (a
// page's keys, values and scales; eight 16-byte pieces a thread and step, past
// the caches: 256 sequences' third of 1.2 GB moved in 112 us against 120 with
// ordinary loads and stores).
typedef unsigned U __attribute__((ext_vector_type(4)));
__global__ __launch_bounds__(256) void compact_move_kernel(CompactArgs a, int seq_blocks) {
    const CacheView& c = a.c;
    const int tid = threadIdx.x, moved = a.count[0], used = a.count[1];
    if ((int)blockIdx.x < seq_blocks) {
        for (int s = blockIdx.x; s < c.n_seqs; s += seq_blocks) {
            const int held = (c.length(s) + PAGE - 1) / PAGE;
            for (int p = tid; p < held; p += 256) {
                int* at = c.table + (size_t)s * c.seq_pages + p;
                const int page = *at;
                if (page < used || !c.page_ok(page)) continue;
                const int to = a.map[page];
                if (c.page_ok(to)) *at = to;
            }
        }
        return;
    }
    const long half = (long)c.H * PAGE * c.d;   // bytes of a page's keys
    const int pieces = (int)(half / 16);        // and as many of its values
    for (int i = blockIdx.x - seq_blocks; i < moved; i += gridDim.x - seq_blocks) {
        const int from = a.from[i], to = a.to[i];
        const U* ks = reinterpret_cast<const U*>(c.k + from * half);
        const U* vs = reinterpret_cast<const U*>(c.v + from * half);
        U* kd = reinterpret_cast<U*>(c.k + to * half);
        U* vd = reinterpret_cast<U*>(c.v + to * half);
        for (int p = tid; p < pieces; p += 256 * 4) {
            U kk[4], vv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (p + 256 * e >= pieces) continue;
                kk[e] = __builtin_nontemporal_load(ks + p + 256 * e);
                vv[e] = __builtin_nontemporal_load(vs + p + 256 * e);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (p + 256 * e >= pieces) continue;
                __builtin_nontemporal_store(kk[e], kd + p + 256 * e);
                __builtin_nontemporal_store(vv[e], vd + p + 256 * e);
            }
        }
        const uint2* ss = reinterpret_cast<const uint2*>(c.scales + (size_t)from * c.H * 8);
        uint2* sd = reinterpret_cast<uint2*>(c.scales + (size_t)to * c.H * 8);
        for (int p = tid; p < c.H; p += 256) sd[p] = ss[p];
        if (tid == 0) {
            c.refs[to] = c.refs[from];
            c.refs[from] = 0;
        }
    }
}

__global__ __launch_bounds__(256) void cache_init_kernel(CacheView c) {
    const long n = 64L + c.n_seqs + c.n_pages;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) c.status[i] = 0;
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

static tm_status status_of(hipError_t e) { return e == hipSuccess ? TM_OK : TM_ERR_HIP; }

static bool blob_ok(const tm_cache* c, const void* blob) { return c && ptr_ok(blob, 256); }
static bool list_ok(const int* p) { return (uintptr_t)p % 4 == 0; }

}  // namespace tmk

using namespace tmk;

extern "C" {

tm_status tm_cache_create(int kv_heads, int head_dim, int n_pages, int n_seqs, int seq_pages, tm_cache** out) {
    if (!out) return TM_ERR_INVALID;
    *out = nullptr;
    if (kv_heads < 1 || kv_heads > 1024 || head_dim < 32 || head_dim > 256 || head_dim % 32 != 0 || n_pages < 1 ||
        n_pages > 1 << 24 || n_seqs < 1 || n_seqs > MAX_SEQS || seq_pages < 1 || seq_pages > 1 << 20 ||
        (long)n_seqs * seq_pages > 1L << 30)
        return TM_ERR_INVALID;
    tm_cache* c = new (std::nothrow) tm_cache;
    if (!c) return TM_ERR_INVALID;
    c->H = kv_heads;
    c->d = head_dim;
    c->n_pages = n_pages;
    c->n_seqs = n_seqs;
    c->seq_pages = seq_pages;
    const size_t cells = (size_t)n_pages * kv_heads * PAGE * head_dim;
    c->off[0] = 0;
    c->off[1] = up256(4 * (64 + (size_t)n_seqs + n_pages + (size_t)n_seqs * seq_pages));
    c->off[2] = c->off[1] + up256((size_t)n_pages * kv_heads * 8);
    c->off[3] = c->off[2] + up256(cells);
    c->bytes = c->off[3] + up256(cells);
    *out = c;
    return TM_OK;
}

void tm_cache_destroy(tm_cache* c) { delete c; }

size_t tm_cache_bytes(const tm_cache* c) { return c ? c->bytes : 0; }

tm_status tm_cache_layout(const tm_cache* c, size_t offsets[4]) {
    if (!c || !offsets) return TM_ERR_INVALID;
    for (int i = 0; i < 4; ++i) offsets[i] = c->off[i];
    return TM_OK;
}

size_t tm_cache_workspace_bytes(const tm_cache* c, int batch, int n_tokens, int heads) {
    if (!c || batch < 0 || n_tokens < 0 || heads < 0) return 0;
    size_t n = up256((size_t)batch * sizeof(AppendPlan));
    const size_t compact = 256 + up256((size_t)c->n_pages * 12);
    if (compact > n) n = compact;
    if (heads > 0) {
        const size_t at = attend_workspace(c, batch, n_tokens, heads);
        if (at > n) n = at;
    }
    return n;
}

tm_status tm_cache_init(const tm_cache* c, void* blob, void* stream) {
    if (!blob_ok(c, blob)) return TM_ERR_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const long n = 64L + c->n_seqs + c->n_pages;
    const unsigned blocks = (unsigned)((n + 255) / 256 < 1024 ? (n + 255) / 256 : 1024);
    return status_of(timed_attn(st, [&] {
        launch_k(cache_init_kernel, dim3(blocks), dim3(256), 0, st, cache_view(c, blob));
        return hipGetLastError();
    }));
}

tm_status tm_cache_append(const tm_cache* c, void* blob, const int* seqs, const int* counts, const void* k,
                          long k_batch, long k_token, const void* v, long v_batch, long v_token, int batch,
                          int n_tokens, tm_dtype dtype, void* workspace, void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (!blob_ok(c, blob) || batch < 0 || n_tokens < 0) return TM_ERR_INVALID;
    if (batch == 0 || n_tokens == 0) return TM_OK;
    if (batch > c->n_seqs || !list_ok(seqs) || !list_ok(counts) || !ptr_ok(k, 16) || !ptr_ok(v, 16) ||
        !ptr_ok(workspace, 256) || !strides_ok(k_batch, k_token) || !strides_ok(v_batch, v_token))
        return TM_ERR_INVALID;
    // a longer call could not be served by any sequence
    const long most = (long)c->seq_pages * PAGE;
    if (n_tokens > most && !counts) return TM_ERR_INVALID;
    AppendArgs a{cache_view(c, blob), seqs, counts, k, v, k_batch, k_token, v_batch, v_token, batch, n_tokens,
                 static_cast<AppendPlan*>(workspace)};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 each((unsigned)c->H, (unsigned)batch);
    // One launch while its workgroups are few: it saves the host a launch, and
    // takes the GPU longer than the two, the more the more workgroups go to the
    // count that ends it; a shared page's head is copied by one or two waves
    // where the write has four.  8 heads of 128, a call from the host (with a
    // small copy beside it) / on the GPU alone (in a graph), us, one launch against two; tokens into begun
    // blocks, then into copies of shared pages:
    //   one token, 16 entries   14.5/5.9 against 16.9/5.0    20.2/18.1 against 17.1/11.1
    //              64           14.6/7.5 against 16.8/5.9    21.7/19.5 against 17.0/13.4
    //              128          14.6/9.6 against 16.8/7.2    25.0/22.9 against 19.6/17.6
    //   4 tokens,  16           14.6/8.9 against 16.9/8.1    16.1/14.2 against 17.0/12.0
    //              64           14.6/11.5 against 16.9/9.6   19.2/17.1 against 19.8/17.8
    //              128          17.8/15.7 against 16.8/12.0  25.5/23.3 against 27.8/25.7
    // So: 4 tokens up to 64 entries of these; one token, whose copies lose by
    // it, too, though other single tokens would gain up to 256 entries.
    const int heads = n_tokens == 1 ? 4 : 2;
    const dim3 step((unsigned)((c->H + heads - 1) / heads), (unsigned)batch);
    if (n_tokens <= STEP_TOKENS && batch <= STEP_ENTRIES && (long)batch * step.x <= (n_tokens == 1 ? 128 : 256)) {
        return status_of(timed_attn(st, [&] {
            return for_head_dim(c->d, [&](auto D) {
                if (dtype == TM_F32) {
                    if (n_tokens == 1) launch_k(append_step_kernel<float, D(), true>, step, dim3(STEP_ENTRIES), 0, st, a);
                    else launch_k(append_step_kernel<float, D(), false>, step, dim3(STEP_ENTRIES), 0, st, a);
                } else {
                    if (n_tokens == 1) launch_k(append_step_kernel<bf16, D(), true>, step, dim3(STEP_ENTRIES), 0, st, a);
                    else launch_k(append_step_kernel<bf16, D(), false>, step, dim3(STEP_ENTRIES), 0, st, a);
                }
                return hipGetLastError();
            });
        }));
    }
    hipError_t e = timed_attn(st, [&] {
        if (batch <= 256) launch_k(append_plan_kernel<256, 256>, dim3(1), dim3(256), 0, st, a);
        else launch_k(append_plan_kernel<PLAN_THREADS, MAX_SEQS>, dim3(1), dim3(PLAN_THREADS), 0, st, a);
        return hipGetLastError();
    });
    if (e != hipSuccess) return TM_ERR_HIP;
    const long tokens = n_tokens < most ? n_tokens : most;
    const dim3 grid((unsigned)((tokens + PAGE - 2) / PAGE + 1), (unsigned)c->H, (unsigned)batch);
    return status_of(timed_attn(st, [&] {
        return for_head_dim(c->d, [&](auto D) {
            if (n_tokens == 1) {
                if (dtype == TM_F32) launch_k(append_token_kernel<float, D()>, each, dim3(256), 0, st, a);
                else launch_k(append_token_kernel<bf16, D()>, each, dim3(256), 0, st, a);
                return hipGetLastError();
            }
            if (dtype == TM_F32) launch_k(append_write_kernel<float, D()>, grid, dim3(256), 0, st, a);
            else launch_k(append_write_kernel<bf16, D()>, grid, dim3(256), 0, st, a);
            return hipGetLastError();
        });
    }));
}

tm_status tm_cache_read(const tm_cache* c, const void* blob, const int* seqs, int start, void* k, void* v, int batch,
                        int n_tokens, tm_dtype dtype, void* stream) {
    if (dtype != TM_F32 && dtype != TM_BF16) return TM_ERR_DTYPE;
    if (!blob_ok(c, blob) || batch < 0 || n_tokens < 0 || start < 0) return TM_ERR_INVALID;
    if (batch == 0 || n_tokens == 0) return TM_OK;
    const long most = (long)c->seq_pages * PAGE;
    if (batch > 65535 || (!seqs && batch > c->n_seqs) || !list_ok(seqs) || !ptr_ok(k, 16) || !ptr_ok(v, 16))
        return TM_ERR_INVALID;
    if (start >= most) return TM_OK;
    ReadArgs a{cache_view(c, const_cast<void*>(blob)), seqs, k, v, start, batch, n_tokens};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const long last = (long)start + n_tokens < most ? (long)start + n_tokens : most;
    const dim3 grid((unsigned)((last + PAGE - 1) / PAGE - start / PAGE), (unsigned)c->H, (unsigned)batch);
    return status_of(timed_attn(st, [&] {
        return for_head_dim(c->d, [&](auto D) {
            if (dtype == TM_F32) launch_k(cache_read_kernel<float, D()>, grid, dim3(256), 0, st, a);
            else launch_k(cache_read_kernel<bf16, D()>, grid, dim3(256), 0, st, a);
            return hipGetLastError();
        });
    }));
}

tm_status tm_cache_fork(const tm_cache* c, void* blob, const int* src, const int* dst, int n, void* stream) {
    if (!blob_ok(c, blob) || n < 0) return TM_ERR_INVALID;
    if (n == 0) return TM_OK;
    if (n > c->n_seqs || !ptr_ok(src, 4) || !ptr_ok(dst, 4)) return TM_ERR_INVALID;
    ForkArgs a{cache_view(c, blob), src, dst, n};
    hipStream_t st = static_cast<hipStream_t>(stream);
    return status_of(timed_attn(st, [&] {
        launch_k(fork_kernel, dim3((unsigned)n), dim3(256), 0, st, a);
        return hipGetLastError();
    }));
}

tm_status tm_cache_free(const tm_cache* c, void* blob, const int* seqs, const int* keep, int n, void* stream) {
    if (!blob_ok(c, blob) || n < 0) return TM_ERR_INVALID;
    if (n == 0) return TM_OK;
    if (n > c->n_seqs || !list_ok(seqs) || !list_ok(keep)) return TM_ERR_INVALID;
    FreeArgs a{cache_view(c, blob), seqs, keep, n};
    hipStream_t st = static_cast<hipStream_t>(stream);
    return status_of(timed_attn(st, [&] {
        launch_k(free_kernel, dim3((unsigned)n), dim3(256), 0, st, a);
        return hipGetLastError();
    }));
}

tm_status tm_cache_compact(const tm_cache* c, void* blob, void* workspace, void* stream) {
    if (!blob_ok(c, blob) || !ptr_ok(workspace, 256)) return TM_ERR_INVALID;
    int* ws = static_cast<int*>(workspace);
    CompactArgs a{cache_view(c, blob), ws, ws + 64, ws + 64 + (size_t)c->n_pages, ws + 64 + 2 * (size_t)c->n_pages, c->d};
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = timed_attn(st, [&] {
        launch_k(compact_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, st, a);
        return hipGetLastError();
    });
    if (e != hipSuccess) return TM_ERR_HIP;
    const int seq_blocks = c->n_seqs < 256 ? c->n_seqs : 256;
    const int movers = c->n_pages < 4096 ? c->n_pages : 4096;
    return status_of(timed_attn(st, [&] {
        launch_k(compact_move_kernel, dim3((unsigned)(seq_blocks + movers)), dim3(256), 0, st, a, seq_blocks);
        return hipGetLastError();
    }));
}

tm_status tm_cache_check(const tm_cache* c, const void* blob, int* flags, int* pages_used, void* stream) {
    if (!blob_ok(c, blob)) return TM_ERR_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const CacheView v = cache_view(c, const_cast<void*>(blob));
    int f = 0;
    if (hipMemcpyAsync(&f, v.status, 4, hipMemcpyDeviceToHost, st) != hipSuccess) return TM_ERR_HIP;
    int* refs = nullptr;
    if (pages_used) {
        refs = new (std::nothrow) int[c->n_pages];
        if (!refs) return TM_ERR_HIP;
        if (hipMemcpyAsync(refs, v.refs, 4 * (size_t)c->n_pages, hipMemcpyDeviceToHost, st) != hipSuccess) {
            (void)hipStreamSynchronize(st);
            delete[] refs;
            return TM_ERR_HIP;
        }
    }
    const bool ok = hipStreamSynchronize(st) == hipSuccess;
    if (ok && flags) *flags = f;
    if (ok && pages_used) {
        int n = 0;
        for (int i = 0; i < c->n_pages; ++i) n += refs[i] > 0;
        *pages_used = n;
    }
    delete[] refs;
    return ok ? TM_OK : TM_ERR_HIP;
}

}  // extern "C"
