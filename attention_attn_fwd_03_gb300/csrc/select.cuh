// select.cuh -- which pages of a long context a query token attends to: the
// device functions that the selection kernels (select.cu) and the fused
// page-sparse kernel (sparse.cu) share.
//
// Score.  The sketch of a page holds, per channel, the largest and smallest
// key value in 8 bits; with the query in 8-bit codes c,
//   I = sum_c max(c, 0) max8_c + min(c, 0) min8_c
// is an integer dot product of length 2 d: [max(c, 0), min(c, 0)] against
// [max8, min8].  |I| < 2 d 127^2 < 2^23, so I is exact in fp32 and in any
// order; the score max_h(|q_h|max I_h) amp is two further roundings.  The
// products run on the matrix units in fp16 with fp32 sums: a sketch byte b
// enters as (b + 128) 2^-24, two byte permutations for four of them, and
// 128 sum c comes off at the end; sums below 2^23 units are exact.  (Four-byte
// integer dot products and the int8 form of the matrix instruction give the
// same sums, but are slow on this GPU.)
//
// Selection.  Counting in equal intervals of the order-preserving integer
// image of the scores finds the smallest score that still belongs, then one
// ordered pass compacts the chosen pages in the order of their keys, ties from
// the front.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

// The request of token t: the last one that starts at or before it.  cu is
// bisected 32 ways at a time by the whole warp.
__device__ __forceinline__ int request_of(const int32_t* cu, int B, int t, int lane) {
    int lo = 0, n = B;  // candidates [lo, lo + n): the first starts at or before t
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool starts = i < n && __ldg(cu + lo + i) <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, starts));
        const int skip = c > 0 ? (c - 1) * step : 0;
        lo += skip;
        n = min(step, n - skip);
    }
    return lo;
}

struct Token {
    int r;          // its request
    long long pos;  // its position; -1: it sees no key
    bool owned;     // false: behind the last request
};

// Position of token t (whole warp).  Offsets that do not hold t, or a length
// out of range, set bad.
__device__ __forceinline__ Token token_of(const SelectParams& p, int t, int lane, bool& bad) {
    Token k;
    k.owned = true;
    long long behind = 1;  // keys of the request from this token on
    if (p.cu == nullptr) {
        k.r = t;
    } else {
        k.r = 0;
        k.pos = -1;
        const int end = __ldg(p.cu + p.B);
        if (end < 0 || end > p.total_q) bad = true;
        if (t >= end) {
            k.owned = false;
            return k;
        }
        k.r = request_of(p.cu, p.B, t, lane);
        const int a = __ldg(p.cu + k.r), b = __ldg(p.cu + k.r + 1);
        if (a < 0 || t < a || t >= b || b > p.total_q) {
            bad = true;
            return k;
        }
        behind = (long long)b - t;
    }
    long long len = __ldg(p.seq_lens + k.r);
    const long long cap = (long long)p.max_pages << p.page_shift;
    if (len < 0 || len > cap) {
        bad = true;
        len = len < 0 ? 0 : cap;
    }
    k.pos = len - behind;
    if (k.pos < 0) k.pos = -1;
    return k;
}

// fp32 -> uint32 with the same order; -0 counts as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// 16-byte pieces of a page's sketch, and of a head's codes.
template <int D>
constexpr int kPieces = 2 * D / 16;

// Sketches of 8 STEPS pages on their way to a warp's registers.  Four lanes
// take a page, so that a 16-byte load of the warp covers eight pages, 64 bytes
// of each; round s covers pages first + 8 s .. + 7.
template <int D, int STEPS>
struct SketchLoads {
    static constexpr int PL = kPieces<D> / 4;
    uint4 x[STEPS][PL];
    float amp[STEPS];
    int id[STEPS];  // -1: not a page

    // Ids of the pages first .. that lie below end; then their sketches.
    __device__ __forceinline__ void look_up(const int32_t* table, int first, int end, int lane) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int page = first + s * 8 + (lane >> 2);
            id[s] = page < end ? __ldg(table + page) : -1;
        }
    }
    // Pages from first on that lie below end and do not exist set bad, and read the first page's sketch.
    __device__ __forceinline__ void fetch(const SelectParams& p, int kvh, int first, int end, int lane, bool& bad) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (id[s] < 0 || id[s] >= p.num_pages) {
                bad |= first + s * 8 + (lane >> 2) < end;
                id[s] = -1;
            }
            const long long rec = (long long)(id[s] < 0 ? 0 : id[s]) * p.H_kv + kvh;
            const uint4* src = reinterpret_cast<const uint4*>(p.sketch + rec * (2 * D));
#pragma unroll
            for (int i = 0; i < PL; ++i) x[s][i] = __ldg(src + i * 4 + (lane & 3));
            amp[s] = __ldg(p.amp + rec);
        }
    }

    // Ordered scores of the pages, key[s] that of page first + 8 s + lane / 4.  A pair of rounds is
    // the 16 rows of the warp-level matrix instruction, TB tiles of 8 query heads its columns; the
    // channels enter in the order in which the lanes hold them, which is the same for both operands.
    template <int TB>
    __device__ __forceinline__ void keys(const uint4* codes, const float2* heads, int G, int lane, uint32_t* key) const {
        static_assert(STEPS % 2 == 0, "two rounds make 16 rows");
        const int sub = lane & 3;
        float best[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) best[s] = -INFINITY;
        for (int h0 = 0; h0 < G; h0 += 8 * TB) {
            float acc[TB][STEPS / 2][4];
#pragma unroll
            for (int n = 0; n < TB; ++n)
#pragma unroll
                for (int g = 0; g < STEPS / 2; ++g) acc[n][g][0] = acc[n][g][1] = acc[n][g][2] = acc[n][g][3] = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                uint4 c[TB];
#pragma unroll
                for (int n = 0; n < TB; ++n) {
                    const int h = h0 + n * 8 + (lane >> 2);
                    c[n] = codes[(h < G ? h : 0) * kPieces<D> + i * 4 + sub];
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a[STEPS][2];
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) fractions(word(x[s][i], w), a[s]);
#pragma unroll
                    for (int n = 0; n < TB; ++n) {
                        uint32_t bw[2];
                        integers(word(c[n], w), bw);
#pragma unroll
                        for (int g = 0; g < STEPS / 2; ++g)
                            asm volatile(
                                "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                                "{%8, %9}, {%0, %1, %2, %3};"
                                : "+f"(acc[n][g][0]), "+f"(acc[n][g][1]), "+f"(acc[n][g][2]), "+f"(acc[n][g][3])
                                : "r"(a[2 * g][0]), "r"(a[2 * g + 1][0]), "r"(a[2 * g][1]), "r"(a[2 * g + 1][1]),
                                  "r"(bw[0]), "r"(bw[1]));
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < TB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = h0 + n * 8 + sub * 2 + e;
                    const float2 q = h < G ? heads[h] : make_float2(0.f, 0.f);
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
                        const float I = fmaf(acc[n][s / 2][(s & 1) * 2 + e], 16777216.f, -q.y);  // exact
                        const float v = q.x == INFINITY ? INFINITY : __fmul_rn(q.x, I);
                        best[s] = h < G ? fmaxf(best[s], v) : best[s];
                    }
                }
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            best[s] = fmaxf(best[s], __shfl_xor_sync(0xffffffffu, best[s], 1));
            best[s] = fmaxf(best[s], __shfl_xor_sync(0xffffffffu, best[s], 2));
            float score = __fmul_rn(best[s], amp[s]);
            if (score != score || amp[s] == INFINITY) score = INFINITY;
            if (id[s] < 0) score = -INFINITY;  // not a page: the last to be taken
            key[s] = ordered(score);
        }
    }

    static __device__ __forceinline__ uint32_t word(const uint4& v, int w) {
        return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
    }
    // Four int8 b to two packed pairs of fp16: (b + 128) 2^-24, the bytes with their sign bits flipped
    // as subnormal fp16 numbers, which the matrix units take as they are.
    static __device__ __forceinline__ void fractions(uint32_t bytes, uint32_t* h) {
        const uint32_t u = bytes ^ 0x80808080u;
        // volatile: converted where they are used, not all at once into registers
        asm volatile("prmt.b32 %0, %1, 0, 0x4140;" : "=r"(h[0]) : "r"(u));
        asm volatile("prmt.b32 %0, %1, 0, 0x4342;" : "=r"(h[1]) : "r"(u));
    }
    // Four int8 to two packed pairs of fp16, exactly: with its sign bit flipped a byte b is the
    // fraction of the fp16 number 1024 + 128 + b.
    static __device__ __forceinline__ void integers(uint32_t bytes, uint32_t* h) {
        const uint32_t u = bytes ^ 0x80808080u;
        const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
        asm volatile("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[0]) : "r"(lo), "r"(0x64806480u));
        asm volatile("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[1]) : "r"(hi), "r"(0x64806480u));
    }
};

// 8-bit codes of the group's query heads, with each head's largest magnitude
// and 128 times the sum of its codes; a warp per head, D / 32 channels per lane.
template <int D>
__device__ __forceinline__ void make_codes(const uint16_t* group, int G, uint4* s_codes, float2* s_heads, int warp,
                                           int n_warps, int lane) {
    constexpr int C = D / 32;
    for (int h = warp; h < G; h += n_warps) {
        const uint16_t* q = group + (long long)h * D + lane * C;
        uint32_t w[C / 2];
        if (C == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(q);
            w[0] = v.x;
            w[C / 2 - 1] = v.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(q);
        }
        uint32_t top = 0;  // largest magnitude as bf16 bits; infinities and NaN above every number
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            const uint32_t a = w[i] & 0x7fff7fffu;
            top = max(top, max(a & 0xffffu, a >> 16));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const bool usable = top < 0x7f80u && top != 0u;
        const float qmax = __uint_as_float(top << 16);
        uint32_t up = 0, down = 0;
        int total = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float v = (i & 1) ? bf16hi_to_f32(w[i / 2]) : bf16lo_to_f32(w[i / 2]);
            const int c = usable ? __float2int_rn(__fmul_rn(__fdiv_rn(v, qmax), 127.f)) : 0;
            total += c;
            up |= ((uint32_t)max(c, 0) & 0xffu) << (8 * i);
            down |= ((uint32_t)min(c, 0) & 0xffu) << (8 * i);
        }
        uint8_t* dst = reinterpret_cast<uint8_t*>(s_codes + h * kPieces<D>) + lane * C;
        if (C == 4) {
            *reinterpret_cast<uint32_t*>(dst) = up;
            *reinterpret_cast<uint32_t*>(dst + D) = down;
        } else {
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)up;
            *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)down;
        }
        total = __reduce_add_sync(0xffffffffu, total);
        if (lane == 0) s_heads[h] = make_float2(top < 0x7f80u ? qmax : INFINITY, 128.f * (float)total);
    }
}

// Shared memory of a selection by NTHREADS threads.
constexpr int kBins = 1024;
constexpr int kFew = 128;  // contenders that are ranked against one another

template <int NTHREADS>
struct SelectScratch {
    int a[NTHREADS / 32], b[NTHREADS / 32];
    uint32_t lo, hi;
    int bin, above, inside, few;
    uint32_t value;
    int left;
    uint32_t key[kFew];
    int index[kFew];
};

// Exclusive sums of (x, y) over the CTA's threads.
template <int NTHREADS>
__device__ __forceinline__ void block_sums(int& x, int& y, SelectScratch<NTHREADS>& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, ix, o), v = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += u;
            iy += v;
        }
    }
    if (lane == 31) {
        s.a[warp] = ix;
        s.b[warp] = iy;
    }
    __syncthreads();
    x = ix - x;
    y = iy - y;
#pragma unroll
    for (int w = 0; w < NTHREADS / 32; ++w) {
        x += w < warp ? s.a[w] : 0;
        y += w < warp ? s.b[w] : 0;
    }
}

// f(key, i) for every key of the CTA, kBatch loads at a time.
constexpr int kBatch = 8;
template <int NTHREADS, class F>
__device__ __forceinline__ void for_keys(const uint32_t* keys, int n, F f) {
    for (int i0 = threadIdx.x; i0 < n; i0 += NTHREADS * kBatch) {
        uint32_t key[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) key[x] = i0 + x * NTHREADS < n ? keys[i0 + x * NTHREADS] : 0u;
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
            if (i0 + x * NTHREADS < n) f(key[x], i0 + x * NTHREADS);
    }
}

// Calls emit(place, i) for the `need` (1 <= need < n) best of keys[0 .. n - 1],
// ties to the smaller i, place = 0 .. need - 1 in the order of i, and returns the
// smallest key among them.  bins: kBins words of shared memory.  All NTHREADS
// threads call it.
//
// The keys between the smallest and the largest are counted in up to kBins
// equal intervals, which leaves a few contenders in the interval where the
// count from above passes `need`; they are ranked against one another.  An
// interval with more of them (outliers had stretched the range, or scores tie)
// is divided again, ten bits of the range at a time, until it holds one value.
template <int NTHREADS, class Emit>
__device__ __forceinline__ uint32_t select_best(const uint32_t* keys, int n, int need, int* bins,
                                            SelectScratch<NTHREADS>& s, Emit emit) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t lo = 0xffffffffu, hi = 0u;
    if (tid == 0) {
        s.lo = 0xffffffffu;
        s.hi = 0u;
    }
    for_keys<NTHREADS>(keys, n, [&](uint32_t key, int) {
        lo = min(lo, key);
        hi = max(hi, key);
    });
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        atomicMin(&s.lo, lo);
        atomicMax(&s.hi, hi);
    }
    __syncthreads();
    lo = s.lo;
    hi = s.hi;
    int left = need;  // to take among the keys of [lo, hi]; those above hi are taken
    uint32_t value = lo;
    while (lo < hi) {
        const int bits = 32 - __clz(hi - lo);  // hi - lo < 2^bits
        const int shift = bits > 10 ? bits - 10 : 0;
        for (int i = tid; i < kBins; i += NTHREADS) bins[i] = 0;
        if (tid == 0) s.few = 0;
        __syncthreads();
        for_keys<NTHREADS>(keys, n, [&](uint32_t key, int) {
            if (key >= lo && key <= hi) atomicAdd(&bins[(key - lo) >> shift], 1);
        });
        __syncthreads();
        // from the highest interval down, a run per thread
        constexpr int RUN = kBins / NTHREADS;
        int c[RUN], above = 0, none = 0;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            c[i] = bins[kBins - 1 - (tid * RUN + i)];
            above += c[i];
        }
        const int sum = above;
        block_sums(above, none, s);
        if (above < left && left <= above + sum) {  // one thread: the interval is in its run
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                if (above < left && left <= above + c[i]) {
                    s.bin = kBins - 1 - (tid * RUN + i);
                    s.above = above;
                    s.inside = c[i];
                }
                above += c[i];
            }
        }
        __syncthreads();
        const int inside = s.inside;
        left -= s.above;
        lo += (uint32_t)s.bin << shift;
        const uint32_t width = (1u << shift) - 1u;
        hi = hi - lo > width ? lo + width : hi;
        value = lo;
        if (inside <= kFew && lo < hi) {
            for_keys<NTHREADS>(keys, n, [&](uint32_t key, int i) {
                if (key >= lo && key <= hi) {
                    const int at = atomicAdd(&s.few, 1);
                    s.key[at] = key;
                    s.index[at] = i;
                }
            });
            __syncthreads();
            if (tid < inside) {
                const uint32_t key = s.key[tid];
                const int at = s.index[tid];
                int before = 0, greater = 0;
                for (int i = 0; i < inside; ++i) {
                    const uint32_t k = s.key[i];
                    greater += k > key ? 1 : 0;
                    before += k > key || (k == key && s.index[i] < at) ? 1 : 0;
                }
                if (before == left - 1) {  // the last one taken
                    s.value = key;
                    s.left = left - greater;
                }
            }
            __syncthreads();
            value = s.value;
            left = s.left;
            break;
        }
        __syncthreads();  // the bins are written again
    }
    // taken: every key above `value`, and the first `left` of those equal to it.  A warp walks its own
    // run of keys, 32 at a time, so the order of the keys is the order of the lanes and the warps.
    constexpr int WARPS = NTHREADS / 32;
    const int run = ((n + WARPS - 1) / WARPS + 31) / 32 * 32;
    const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
    int more = 0, equal = 0;  // of the lane's own keys
    for (int i = i0; i < i1; i += 32 * kBatch) {
        uint32_t key[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) key[x] = i + x * 32 + lane < i1 ? keys[i + x * 32 + lane] : 0u;
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const bool in = i + x * 32 + lane < i1;
            more += in && key[x] > value ? 1 : 0;
            equal += in && key[x] == value ? 1 : 0;
        }
    }
    more = __reduce_add_sync(0xffffffffu, more);
    equal = __reduce_add_sync(0xffffffffu, equal);
    __syncthreads();  // s.a and s.b are free
    if (lane == 0) {
        s.a[warp] = more;
        s.b[warp] = equal;
    }
    __syncthreads();
    more = equal = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        more += w < warp ? s.a[w] : 0;
        equal += w < warp ? s.b[w] : 0;
    }
    const unsigned below = (1u << lane) - 1u;
    for (int i = i0; i < i1; i += 32 * kBatch) {
        uint32_t key[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) key[x] = i + x * 32 + lane < i1 ? keys[i + x * 32 + lane] : 0u;
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const bool in = i + x * 32 + lane < i1;
            const unsigned gt = __ballot_sync(0xffffffffu, in && key[x] > value);
            const unsigned eq = __ballot_sync(0xffffffffu, in && key[x] == value);
            const int ties = equal + __popc(eq & below);  // equal keys before this one
            const bool taken = in && (key[x] > value || (key[x] == value && ties < left));
            if (taken) emit(more + __popc(gt & below) + min(ties, left), i + x * 32 + lane);
            more += __popc(gt);
            equal += __popc(eq);
        }
    }
    return value;
}

}  // namespace

}  // namespace attn
