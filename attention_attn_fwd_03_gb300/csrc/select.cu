// select.cu -- which pages of a long context a query token attends to.
//
// Score.  The sketch of a page holds, per channel, the largest and smallest
// key value in 8 bits; with the query in 8-bit codes c,
//   I = sum_c max(c, 0) max8_c + min(c, 0) min8_c
// is an integer dot product of length 2 d: [max(c, 0), min(c, 0)] against
// [max8, min8].  |I| < 2 d 127^2 < 2^24, so I is exact in fp32 and in any
// order; the score max_h(|q_h|max I_h) amp is two further roundings.
//
// The score kernel is bound by reading 2 d + 4 bytes per page and KV head,
// 1/64 of a 64-row page's keys: four lanes take a page (so a 16-byte load of a
// warp covers eight pages, 64 bytes of each), up to sixteen loads in flight
// per lane, and the four-byte integer dot products of all G query heads run
// from registers against codes in shared memory.
//
// The selection kernel takes one (token, KV head) per CTA: a radix search of
// four 8-bit digits over the order-preserving integer image of the scores
// finds the smallest score that still belongs, then one ordered pass compacts
// the chosen pages in the order of their keys, ties from the front.  It works
// from shared memory (or through L2 above kCached pages) and is
// latency-bound.
#include <cmath>
#include <cstring>

#include "attn_kv.h"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr int kScoreWarps = 4;
constexpr int kSelectThreads = 512;
constexpr int kCached = 11264;  // scores a selection keeps in shared memory (44 KB: no opt-in size)

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
    int r;        // its request
    long long pos;  // its position; -1: it sees no key
    bool owned;   // false: behind the last request
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

// PAGES pages per warp: STEPS rounds of eight.
template <int D, int STEPS>
__global__ void __launch_bounds__(kScoreWarps * 32) page_score_kernel(const __grid_constant__ SelectParams p) {
    constexpr int PIECES = 2 * D / 16;   // 16-byte pieces of a sketch
    constexpr int PL = PIECES / 4;       // pieces per lane
    constexpr int PAGES = kScoreWarps * STEPS * 8;
    extern __shared__ uint4 s_codes[];   // [G][PIECES]
    float* s_qmax = reinterpret_cast<float*>(s_codes + p.G * PIECES);
    griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    long long u = blockIdx.x;
    const int chunk = (int)(u % p.n_chunks);
    u /= p.n_chunks;
    const int kvh = (int)(u % p.H_kv);
    const int t = (int)(u / p.H_kv);
    bool bad = false;
    const Token k = token_of(p, t, lane, bad);
    const int n_vis = k.pos < 0 ? 0 : (int)(k.pos >> p.page_shift) + 1;
    const int page0 = chunk * PAGES;
    if (n_vis <= p.budget || page0 >= n_vis) return;  // everything is taken, or nothing is here

    // the pages' ids and sketches are on their way while the codes are made
    const int sub = lane & 3;
    int page[STEPS], id[STEPS];
    uint4 x[STEPS][PL];
    float amp[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        page[s] = page0 + (s * kScoreWarps + warp) * 8 + (lane >> 2);
        id[s] = -1;
        if (page[s] < n_vis) {
            id[s] = __ldg(p.table + (long long)k.r * p.max_pages + page[s]);
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

    // codes of the group's query heads: a warp per head, D / 32 channels per lane
    constexpr int C = D / 32;
    for (int h = warp; h < p.G; h += kScoreWarps) {
        const uint16_t* q = p.q + ((long long)t * p.H + kvh * p.G + h) * D + lane * C;
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
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
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
        uint8_t* dst = reinterpret_cast<uint8_t*>(s_codes + h * PIECES) + lane * C;
        if (C == 4) {
            *reinterpret_cast<uint32_t*>(dst) = up;
            *reinterpret_cast<uint32_t*>(dst + D) = down;
        } else {
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)up;
            *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)down;
        }
        if (lane == 0) s_qmax[h] = top < 0x7f80u ? qmax : INFINITY;
    }
    __syncthreads();

    float best[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) best[s] = -INFINITY;
    for (int h = 0; h < p.G; ++h) {
        int acc[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) acc[s] = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const uint4 c = s_codes[h * PIECES + i * 4 + sub];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                acc[s] = __dp4a((int)x[s][i].x, (int)c.x, acc[s]);
                acc[s] = __dp4a((int)x[s][i].y, (int)c.y, acc[s]);
                acc[s] = __dp4a((int)x[s][i].z, (int)c.z, acc[s]);
                acc[s] = __dp4a((int)x[s][i].w, (int)c.w, acc[s]);
            }
        }
        const float qmax = s_qmax[h];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            acc[s] += __shfl_xor_sync(0xffffffffu, acc[s], 1);
            acc[s] += __shfl_xor_sync(0xffffffffu, acc[s], 2);
            best[s] = fmaxf(best[s], qmax == INFINITY ? INFINITY : __fmul_rn(qmax, (float)acc[s]));
        }
    }
    uint32_t* keys = p.keys + ((long long)t * p.H_kv + kvh) * p.max_pages;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        float score = __fmul_rn(best[s], amp[s]);
        if (score != score || amp[s] == INFINITY) score = INFINITY;
        if (id[s] < 0) score = -INFINITY;  // not a page: the last to be taken
        if (sub == 0 && page[s] < n_vis) keys[page[s]] = ordered(score);
    }
    if (bad) atomicOr(p.status, 1u << kStatusDeviceData);
}

// Exclusive sums of (a, b) over the CTA's threads; all threads call it.
__device__ __forceinline__ void block_sums(int& a, int& b, int* s_a, int* s_b, int tid) {
    const int lane = tid & 31, warp = tid >> 5;
    const int a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        s_a[warp] = a;
        s_b[warp] = b;
    }
    __syncthreads();
    int ba = 0, bb = 0;
    for (int w = 0; w < warp; ++w) {
        ba += s_a[w];
        bb += s_b[w];
    }
    a += ba - a0;
    b += bb - b0;
}

__global__ void __launch_bounds__(kSelectThreads) page_select_kernel(const __grid_constant__ SelectParams p) {
    extern __shared__ uint32_t s_keys[];  // [kCached] or less
    __shared__ int s_hist[256];
    __shared__ int s_a[kSelectThreads / 32], s_b[kSelectThreads / 32];
    __shared__ int s_digit, s_above;
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    const int kvh = (int)(blockIdx.x % p.H_kv);
    const int t = (int)(blockIdx.x / p.H_kv);
    bool bad = false;
    const Token k = token_of(p, t, lane, bad);
    const int ps = 1 << p.page_shift;
    const int n_vis = k.pos < 0 ? 0 : (int)(k.pos >> p.page_shift) + 1;
    const int n_sel = min(n_vis, p.budget);
    const int sel_len = n_vis == 0 ? 0 : (n_sel - 1) * ps + (int)(k.pos & (ps - 1)) + 1;
    const int32_t* table = p.table + (long long)k.r * p.max_pages;
    int32_t* out = p.tables + ((long long)t * p.H_kv + kvh) * p.budget;
    griddep_wait();  // the scores are complete; an earlier call's readers of these outputs too
    if (tid == 0) {
        if (kvh == 0) {
            p.sel_lens[t] = sel_len;
            if (bad) atomicOr(p.status, 1u << kStatusDeviceData);
        }
        if (p.cu_out != nullptr && kvh == 0) {
            // each owned token is a request of its own to the attention kernel, the others are empty ones
            const int end = p.cu == nullptr ? p.total_q : max(0, min(p.total_q, __ldg(p.cu + p.B)));
            p.cu_out[t] = min(t, end);
            if (t == p.total_q - 1) p.cu_out[p.total_q] = end;
        }
        if (p.sched != nullptr && blockIdx.x == 0) {
            p.sched[0] = 0;
            p.sched[1] = p.total_q * p.H_kv * p.n_splits;
        }
    }
    // the attention kernel's work list: every split of this (token, KV head)
    if (p.sched != nullptr) {
        for (int s = tid; s < p.n_splits; s += kSelectThreads) {
            const int unit = (s * p.total_q + t) * p.H_kv + kvh;
            p.sched_list[unit] = make_int4(unit, t, k.owned ? 1 : 0, sel_len);
        }
    }
    for (int i = n_sel + tid; i < p.budget; i += kSelectThreads) out[i] = -1;
    if (n_vis <= p.budget) {
        for (int i = tid; i < n_vis; i += kSelectThreads) out[i] = __ldg(table + i);
        return;
    }

    // more pages than the budget: `first` in front, `last` behind, the best of [first, n_vis - last)
    const int need = p.budget - p.first - p.last;
    const int n = n_vis - p.first - p.last;  // > need
    for (int i = tid; i < p.first; i += kSelectThreads) out[i] = __ldg(table + i);
    for (int i = tid; i < p.last; i += kSelectThreads) out[p.budget - p.last + i] = __ldg(table + n_vis - p.last + i);
    if (need == 0) return;
    const uint32_t* keys = p.keys + ((long long)t * p.H_kv + kvh) * p.max_pages + p.first;
    if (n <= kCached) {
        for (int i = tid; i < n; i += kSelectThreads) s_keys[i] = keys[i];
        keys = s_keys;
    }
    uint32_t value = 0, mask = 0;  // the digits found so far
    int left = need;               // pages still to take among those that match them
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) s_hist[tid] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
            const int i = i0 + tid;
            const uint32_t key = i < n ? keys[i] : 0u;
            const bool in = i < n && (key & mask) == value;
            const int digit = in ? (int)((key >> shift) & 255u) : 256;
            // scores crowd into a few digits: lanes that share one add once
            const unsigned peers = __match_any_sync(0xffffffffu, digit);
            if (in && lane == __ffs(peers) - 1) atomicAdd(&s_hist[digit], __popc(peers));
        }
        __syncthreads();
        if (tid < 32) {  // from the highest digit down: lane l holds digits 255 - 8 l .. 248 - 8 l
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = s_hist[255 - 8 * lane - i];
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
                        s_digit = 255 - 8 * lane - i;
                        s_above = above;
                        break;
                    }
                    above += c[i];
                }
            }
        }
        __syncthreads();
        value |= (uint32_t)s_digit << shift;
        mask |= 255u << shift;
        left -= s_above;
        __syncthreads();
    }
    // taken: every score above `value`, and the first `left` of those equal to it.  Each thread
    // walks its own run of pages, so the order of the keys is the order of the threads.
    const int run = (n + kSelectThreads - 1) / kSelectThreads | 1;  // odd: no two lanes of a bank
    const int i0 = min(n, tid * run), i1 = min(n, i0 + run);
    int more = 0, equal = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = keys[i];
        more += key > value ? 1 : 0;
        equal += key == value ? 1 : 0;
    }
    block_sums(more, equal, s_a, s_b, tid);
    int at = p.first + more + min(equal, left);
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = keys[i];
        const bool tie = key == value;
        if (key > value || (tie && equal < left)) out[at++] = __ldg(table + p.first + i);
        equal += tie ? 1 : 0;
    }
}

// Below this many CTAs of 128 pages the score kernel takes 32 pages per CTA.
constexpr long long kFewChunks = 608;  // four per SM

template <int D>
cudaError_t launch_d(SelectParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.total_q * p.H_kv;
    const int smem = p.G * (2 * D + 4);
    if (p.max_pages > p.budget) {
        const int wide = kScoreWarps * 32, narrow = kScoreWarps * 8;
        const long long chunks = (p.max_pages + wide - 1) / wide;
        if (rows * chunks >= kFewChunks) {
            p.n_chunks = (int)chunks;
            page_score_kernel<D, 4><<<(unsigned)(rows * chunks), kScoreWarps * 32, smem, stream>>>(p);
        } else {
            p.n_chunks = (p.max_pages + narrow - 1) / narrow;
            page_score_kernel<D, 1><<<(unsigned)(rows * p.n_chunks), kScoreWarps * 32, smem, stream>>>(p);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const int n = p.max_pages < kCached ? p.max_pages : kCached;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = p.max_pages > p.budget ? (size_t)n * 4 : 0;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.max_pages > p.budget ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, page_select_kernel, p);
}

}  // namespace

size_t select_keys_bytes(int total_q, int H_kv, int max_pages, int budget) {
    if (max_pages <= budget) return 256;
    return ((size_t)total_q * H_kv * max_pages * sizeof(uint32_t) + 255) / 256 * 256;
}

cudaError_t launch_select(int d, SelectParams p, cudaStream_t stream) {
    if (d == 128) return launch_d<128>(p, stream);
    if (d == 64) return launch_d<64>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
