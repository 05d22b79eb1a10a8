// select.cuh -- which pages of a long context a query token attends to: the
// device functions that the selection kernels (select.cu) and the fused
// page-sparse kernel (sparse.cu) share.
//
// Score.  The sketch of a page holds, per channel, the largest and smallest
// key value in 8 bits; with the query in 8-bit codes c,
//   I = sum_c max(c, 0) max8_c + min(c, 0) min8_c
// is an integer dot product of length 2 d: [max(c, 0), min(c, 0)] against
// [max8, min8].  |I| < 2 d 127^2 < 2^24, so I is exact in fp32 and in any
// order; the score max_h(|q_h|max I_h) amp is two further roundings.
//
// Selection.  A radix search of four 8-bit digits over the order-preserving
// integer image of the scores finds the smallest score that still belongs,
// then one ordered pass compacts the chosen pages in the order of their keys,
// ties from the front.
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

    __device__ __forceinline__ void fetch(const SelectParams& p, const int32_t* table, int kvh, int first, int end,
                                          int lane, bool& bad) {
        const int sub = lane & 3;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int page = first + s * 8 + (lane >> 2);
            id[s] = -1;
            if (page < end) {
                id[s] = __ldg(table + page);
                if (id[s] < 0 || id[s] >= p.num_pages) {
                    bad = true;
                    id[s] = -1;
                }
            }
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const long long rec = (long long)(id[s] < 0 ? 0 : id[s]) * p.H_kv + kvh;
            const uint4* src = reinterpret_cast<const uint4*>(p.sketch + rec * (2 * D));
#pragma unroll
            for (int i = 0; i < PL; ++i) x[s][i] = __ldg(src + i * 4 + sub);
            amp[s] = __ldg(p.amp + rec);
        }
    }

    // Ordered score of the lane's page, round lane & 3: page first + 8 (lane & 3) + lane / 4 (STEPS = 4).
    __device__ __forceinline__ void keys(const uint4* codes, const float* qmax, int G, int lane, uint32_t* key) const {
        const int sub = lane & 3;
        float best[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) best[s] = -INFINITY;
        for (int h = 0; h < G; ++h) {
            int acc[STEPS];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) acc[s] = 0;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const uint4 c = codes[h * kPieces<D> + i * 4 + sub];
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    acc[s] = __dp4a((int)x[s][i].x, (int)c.x, acc[s]);
                    acc[s] = __dp4a((int)x[s][i].y, (int)c.y, acc[s]);
                    acc[s] = __dp4a((int)x[s][i].z, (int)c.z, acc[s]);
                    acc[s] = __dp4a((int)x[s][i].w, (int)c.w, acc[s]);
                }
            }
            const float qm = qmax[h];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                acc[s] += __shfl_xor_sync(0xffffffffu, acc[s], 1);
                acc[s] += __shfl_xor_sync(0xffffffffu, acc[s], 2);
                best[s] = fmaxf(best[s], qm == INFINITY ? INFINITY : __fmul_rn(qm, (float)acc[s]));
            }
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            float score = __fmul_rn(best[s], amp[s]);
            if (score != score || amp[s] == INFINITY) score = INFINITY;
            if (id[s] < 0) score = -INFINITY;  // not a page: the last to be taken
            key[s] = ordered(score);
        }
    }
};

// 8-bit codes and largest magnitudes of the group's query heads, a warp per
// head, D / 32 channels per lane.
template <int D>
__device__ __forceinline__ void make_codes(const uint16_t* group, int G, uint4* s_codes, float* s_qmax, int warp,
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
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float v = (i & 1) ? bf16hi_to_f32(w[i / 2]) : bf16lo_to_f32(w[i / 2]);
            const int c = usable ? __float2int_rn(__fmul_rn(__fdiv_rn(v, qmax), 127.f)) : 0;
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
        if (lane == 0) s_qmax[h] = top < 0x7f80u ? qmax : INFINITY;
    }
}

// Shared memory of a selection by NTHREADS threads.
template <int NTHREADS>
struct SelectScratch {
    int hist[256];
    int a[NTHREADS / 32], b[NTHREADS / 32];
    int digit, above;
};

// Calls emit(place, i) for the `need` (1 <= need < n) best of keys[0 .. n - 1],
// place = 0 .. need - 1 in the order of i.  All NTHREADS threads call it.
template <int NTHREADS, class Emit>
__device__ __forceinline__ void select_best(const uint32_t* keys, int n, int need, SelectScratch<NTHREADS>& s, Emit emit) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t value = 0, mask = 0;  // the digits found so far
    int left = need;               // still to take among those that match them
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += NTHREADS) s.hist[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < n; i0 += NTHREADS) {
            const int i = i0 + tid;
            const uint32_t key = i < n ? keys[i] : 0u;
            const bool in = i < n && (key & mask) == value;
            const int digit = in ? (int)((key >> shift) & 255u) : 256;
            // scores crowd into a few digits: lanes that share one add once
            const unsigned peers = __match_any_sync(0xffffffffu, digit);
            if (in && lane == __ffs(peers) - 1) atomicAdd(&s.hist[digit], __popc(peers));
        }
        __syncthreads();
        if (tid < 32) {  // from the highest digit down: lane l holds digits 255 - 8 l .. 248 - 8 l
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = s.hist[255 - 8 * lane - i];
                sum += c[i];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int above = incl - sum;
            if (above < left && left <= incl) {  // one lane: the digit is among its eight
                for (int i = 0; i < 8; ++i) {
                    if (left <= above + c[i]) {
                        s.digit = 255 - 8 * lane - i;
                        s.above = above;
                        break;
                    }
                    above += c[i];
                }
            }
        }
        __syncthreads();
        value |= (uint32_t)s.digit << shift;
        mask |= 255u << shift;
        left -= s.above;
        __syncthreads();
    }
    // taken: every key above `value`, and the first `left` of those equal to it.  Each thread walks
    // its own run, so the order of the keys is the order of the threads.
    const int run = (n + NTHREADS - 1) / NTHREADS | 1;  // odd: no two lanes of a bank
    const int i0 = min(n, tid * run), i1 = min(n, i0 + run);
    int more = 0, equal = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = keys[i];
        more += key > value ? 1 : 0;
        equal += key == value ? 1 : 0;
    }
    int sa = more, sb = equal;  // sums over the threads before this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sa, o), y = __shfl_up_sync(0xffffffffu, sb, o);
        if (lane >= o) {
            sa += x;
            sb += y;
        }
    }
    if (lane == 31) {
        s.a[warp] = sa;
        s.b[warp] = sb;
    }
    __syncthreads();
    sa -= more;
    sb -= equal;
    for (int w = 0; w < warp; ++w) {
        sa += s.a[w];
        sb += s.b[w];
    }
    int at = sa + min(sb, left);
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = keys[i];
        const bool tie = key == value;
        if (key > value || (tie && sb < left)) emit(at++, i);
        sb += tie ? 1 : 0;
    }
}

}  // namespace

}  // namespace attn
