// append8.cu -- the append that quantises, and the read that undoes it, for a
// paged cache of e4m3 codes with a scale for each block of rows and KV head.
//
// A block's scale is a power of two, 2^e with amax <= 448 2^e: e4m3 keeps its 4
// significant bits wherever in its range a number lies, so rounding the scale up
// costs no accuracy, x 2^-e is exact, and when a later token needs a larger scale
// the older codes move by whole binades: exactly, but for those that become
// subnormal.
//
// Work.  Tokens of one block follow one another in the call (a run).  A CTA owns
// the runs that begin among its 64 tokens, for K or for V, and up to eight heads; the
// last run may reach past them.  A thread holds 16 dims of a row (8 pairs of the
// rotation, whose cosines and sines serve all heads); 64 rows from the first run's
// first token on go side by side, which is all of them unless blocks are larger.
// First pass: the rows are rotated and each run's largest magnitude found (lanes of a
// row by shuffles, rows by an atomic maximum in shared memory, whose order does not
// matter).  Then the scales; second pass: the rows again, mostly from L1 and L2,
// rotated and stored as codes.  Rows that a block held before are requantised by
// the whole CTA where the scale grew.  The same launch rotates q, in CTAs of their own.
//
// Measured.  16,300 tokens of 8 requests, 32 + 8 heads, d = 128, blocks of 64 rows: 71 us, 5.2 TB/s of what has to move (a
// copy: 6.8); loads are waited for more than anything, and 64 registers a thread leave 0.43 of the warps and spill 82 bytes;
// 16,384 tokens with blocks of 256, 512, 1024 rows: 93, 162, 295 us, since only windows in which a run begins have work.  64
// tokens: 5.4 us, 16 x 1 .. 8 tokens with d = 64: 4.3 us: latency (slot, rows, angles, then the block's scale).
// 64 tokens of as many requests, all of whose scales grow: 35 us; 16: 12 us; 256: 36 us.  A CTA goes over its runs in turn then.
#include <cmath>
#include <cstring>

#include "attn_kv8.h"
#include "kernels.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace attn {

namespace {

constexpr int kWindow = 64;    // tokens whose runs a K or V CTA owns, rows side by side in a CTA
constexpr int kHeads = 2;      // heads whose loads a thread has in flight
constexpr int kMaxHeads = 8;   // heads of a K or V CTA: their rows' angles are computed once
constexpr int kReadThreads = 256;
constexpr long long kStreamBytes = 128LL << 20;  // L2: a q_out above it is stored evict-first, as in rope.cu

struct Append8Params {
    const char* in[2];       // k, v: bf16 through byte strides
    long long it[2], ih[2];  // token, head
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* slots;
    const int32_t* positions;
    const void* freq;
    unsigned* status;
    long long n_slots;
    int freq64, T, H_kv, d, rot;
    int page_shift, block_shift;
    int hpc, splits;         // heads per CTA, CTAs that share a window's heads
    unsigned kv_ctas;        // CTAs of K, as many of V; those of q follow
    const char* q;           // bf16 through byte strides, or nullptr
    char* q_out;
    long long qt, qh, qot, qoh;
    int H, q_hpc, q_splits, q_stream;
    float amplitude;
};

// Eight fp32 -> eight e4m3 bytes.  The magnitudes are at most 448 by the choice of the scale.
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
    return make_uint2(pack_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      pack_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}
// The same by division, for a scale that is no power of two (another writer's), and with the code of NaN for an
// infinity or NaN (x - x is NaN for both, 0 otherwise).
__device__ uint2 codes8_careful(const float* x, float s) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] / s + (x[e] - x[e]);
    return codes8(y, 1.f);
}

// Two e4m3 bytes -> two fp32 (exact).
__device__ __forceinline__ float2 values2(uint16_t x) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(x));
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

// The smallest power of two s >= 2^-126 with amax <= 448 s, for a finite amax >= 0: 448 = 1.75 2^8,
// so a significand above 1.75 (the carry) takes one binade more.
__device__ __forceinline__ float scale_for(float amax) {
    const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;  // biased by 127
    return __uint_as_float((unsigned)max(e, 1) << 23);
}

// A power of two from 2^-126 to 2^126.
__device__ __forceinline__ bool is_pow2(float s) {
    return (__float_as_uint(s) & 0x807fffffu) == 0u && s > 0.f && s <= 0x1p126f;
}

__device__ __forceinline__ uint4 ld16(const char* p) { return *reinterpret_cast<const uint4*>(p); }

// The slot of token t, -1 where there is none.
__device__ __forceinline__ int slot_of(const Append8Params& p, int t) {
    const int s = __ldg(p.slots + t);
    return s < 0 || s >= p.n_slots ? -1 : s;
}

template <bool INTERLEAVED>
struct Turn {  // 8 pairs of one row
    float cs[8], sn[8];
    __device__ __forceinline__ void rotate(float* a, float* c) const {
        if (INTERLEAVED) {  // pieces hold pairs (0, 1), (2, 3), ..
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float x0 = a[e], x1 = a[e + 1], y0 = c[e], y1 = c[e + 1];
                a[e] = x0 * cs[e / 2] - x1 * sn[e / 2];
                a[e + 1] = x0 * sn[e / 2] + x1 * cs[e / 2];
                c[e] = y0 * cs[4 + e / 2] - y1 * sn[4 + e / 2];
                c[e + 1] = y0 * sn[4 + e / 2] + y1 * cs[4 + e / 2];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = a[e], y = c[e];
                a[e] = x * cs[e] - y * sn[e];
                c[e] = x * sn[e] + y * cs[e];
            }
        }
    }
};

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
    x[0] = bf16lo_to_f32(v.x); x[1] = bf16hi_to_f32(v.x);
    x[2] = bf16lo_to_f32(v.y); x[3] = bf16hi_to_f32(v.y);
    x[4] = bf16lo_to_f32(v.z); x[5] = bf16hi_to_f32(v.z);
    x[6] = bf16lo_to_f32(v.w); x[7] = bf16hi_to_f32(v.w);
}

__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr unsigned kInfBits = 0x7f800000u;

// What a thread knows of its place in a row: 16 dims in two pieces, that turn where the rotation reaches them.
template <int D, bool INTERLEAVED>
struct Place {
    static constexpr int UPR = D / 16;                 // threads of a row
    static constexpr int THREADS = kWindow * UPR;
    int j, row, off_a, off_b;                     // pieces in elements
    bool turns;
    __device__ __forceinline__ Place(int rot) {
        j = threadIdx.x % UPR;
        row = threadIdx.x / UPR;
        turns = j * 16 < rot;
        if (turns) {
            off_a = INTERLEAVED ? j * 16 : j * 8;
            off_b = INTERLEAVED ? j * 16 + 8 : rot / 2 + j * 8;
        } else {  // the dims that pass through, in two halves
            off_a = rot + (j - rot / 16) * 8;
            off_b = off_a + (D - rot) / 2;
        }
    }
    __device__ __forceinline__ void angles(const Append8Params& p, const unsigned long long* s_turn, int t, Turn<INTERLEAVED>& w) const {
        if (!turns) return;
        const int pos = __ldg(p.positions + t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float c, s;
            turned_cos_sin(s_turn[j * 8 + e], pos, &c, &s);
            w.cs[e] = c * p.amplitude;
            w.sn[e] = s * p.amplitude;
        }
    }
};

__device__ __forceinline__ void load_turns(const Append8Params& p, unsigned long long* s_turn) {
    const int i = threadIdx.x;
    if (i < p.rot / 2)
        s_turn[i] = p.freq64 ? turn_fraction(static_cast<const double*>(p.freq)[i])
                             : turn_fraction(static_cast<const float*>(p.freq)[i]);
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void st16(char* p, const uint4& v, bool stream) {
    if (stream)
        __stcs(reinterpret_cast<uint4*>(p), v);
    else
        *reinterpret_cast<uint4*>(p) = v;
}

// q of a CTA's tokens and heads, rotated into q_out.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void query_part(const Append8Params& p, int cta, unsigned long long* s_turn) {
    const Place<D, INTERLEAVED> at(p.rot);
    const int t = cta / p.q_splits * kWindow + at.row;
    const int h0 = cta % p.q_splits * p.q_hpc, h1 = min(p.H, h0 + p.q_hpc);
    load_turns(p, s_turn);
    __syncthreads();
    if (t >= p.T || slot_of(p, t) < 0) return;
    Turn<INTERLEAVED> w;
    const char* src = p.q + t * p.qt;
    char* dst = p.q_out + t * p.qot;
    for (int h = h0; h < h1; h += kHeads) {
        uint4 x[kHeads], y[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h + i < h1) {
                x[i] = ld16(src + (h + i) * p.qh + at.off_a * 2);
                y[i] = ld16(src + (h + i) * p.qh + at.off_b * 2);
            }
        if (h == h0) at.angles(p, s_turn, t, w);
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h + i < h1) {
                if (at.turns) {
                    float a[8], c[8];
                    unpack8(x[i], a);
                    unpack8(y[i], c);
                    w.rotate(a, c);
                    x[i] = pack8(a);
                    y[i] = pack8(c);
                }
                st16(dst + (h + i) * p.qoh + at.off_a * 2, x[i], p.q_stream != 0);
                st16(dst + (h + i) * p.qoh + at.off_b * 2, y[i], p.q_stream != 0);
            }
    }
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(4 * D, 1024 / (4 * D)) append8_kernel(const __grid_constant__ Append8Params p) {
    using P = Place<D, INTERLEAVED>;
    constexpr int UPR = P::UPR, THREADS = P::THREADS;
    static_assert(THREADS == 4 * D && THREADS >= 4 * kWindow, "a thread for each slot that is looked at first");
    __shared__ unsigned long long s_turn[D / 2];
    __shared__ int s_amax[kMaxHeads][kWindow];     // by run, named by its first token's place in the window
    __shared__ float s_scale[kMaxHeads][kWindow];
    __shared__ float s_ratio[kMaxHeads][kWindow];  // before / now of the rows already there, 1: as they are
    __shared__ int s_slot[2 * kWindow];         // of the window's tokens and as many behind it, -1: none
    __shared__ unsigned s_lead[2];              // the window's tokens that begin runs
    __shared__ int s_end;
    if (blockIdx.x >= 2 * p.kv_ctas) {
        query_part<D, INTERLEAVED>(p, (int)(blockIdx.x - 2 * p.kv_ctas), s_turn);
        return;
    }
    const int tid = threadIdx.x;
    const int side = blockIdx.x >= p.kv_ctas;  // 0: K, 1: V
    const unsigned cta = blockIdx.x - (side ? p.kv_ctas : 0u);
    const int window = (int)(cta / (unsigned)p.splits), split = (int)(cta % (unsigned)p.splits);
    const int t0 = window * kWindow;
    const int h0 = split * p.hpc, nh = min(p.hpc, p.H_kv - h0);
    const int bmask = (1 << p.block_shift) - 1;
    const P at(side == 0 ? p.rot : 0);

    if (tid < 2 * kWindow) {
        const int t = t0 + tid;
        int s = -1;
        bool lead = false;
        if (t < p.T) {
            s = __ldg(p.slots + t);
            const int before = t > 0 ? __ldg(p.slots + t - 1) : -2;
            if (s >= p.n_slots) {
                if (side == 0 && split == 0 && tid < kWindow) atomicOr(p.status, 1u << kStatusDeviceData);
                s = -1;
            }
            lead = s >= 0 && ((s & bmask) == 0 || before != s - 1 || t == 0);
        }
        s_slot[tid] = s;
        const unsigned m = __ballot_sync(0xffffffffu, lead);
        if ((tid & 31) == 0 && tid < kWindow) s_lead[tid / 32] = m;
    }
    for (int i = tid; i < kMaxHeads * kWindow; i += THREADS) (&s_amax[0][0])[i] = 0;
    if (tid == 0) s_end = p.T;
    if (side == 0 && p.rot > 0) load_turns(p, s_turn);
    __syncthreads();
    const unsigned long long lead = s_lead[0] | (unsigned long long)s_lead[1] << 32;
    if (lead == 0ull) return;  // the tokens here belong to a run that began before, or to none
    const int first = t0 + __ffsll((long long)lead) - 1, last_lead = t0 + 63 - __clzll((long long)lead);

    // token t's row of heads h, h + 1, .., unless it is skipped
    uint4 x[kHeads], y[kHeads];
    auto fetch = [&](int t, int h, bool there) {
        const char* src = p.in[side] + t * p.it[side] + (h0 + h) * p.ih[side];
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h + i < nh && there) {
                x[i] = ld16(src + i * p.ih[side] + at.off_a * 2);
                y[i] = ld16(src + i * p.ih[side] + at.off_b * 2);
            }
    };
    fetch(first + at.row, 0, s_slot[first - t0 + at.row] >= 0);  // (its place is below 2 kWindow; past T there is no slot)
    int end = last_lead + 1;
    {  // the end of the last run: its first token that does not follow on
        const int s0 = s_slot[last_lead - t0];
        const int room = bmask + 1 - (s0 & bmask);  // rows of the block from the run's first on
        if (room > 1) {
            for (int i = 1 + tid; i <= room; i += THREADS) {
                const int t = last_lead + i;
                if (t >= p.T) break;
                const int s = t - t0 < 2 * kWindow ? s_slot[t - t0] : __ldg(p.slots + t);
                if (i == room || s != s0 + i) {
                    atomicMin(&s_end, t);
                    break;
                }
            }
            __syncthreads();
            end = s_end;
        }
    }
    // the run of token t: the last of the window's runs to begin at or before it
    auto run_of = [&](int t) {
        const int i = min(t - t0, 63);
        return 63 - __clzll((long long)(lead & (~0ull >> (63 - i))));
    };
    // whether token t belongs to one of the window's runs
    auto in_run = [&](int t) { return t < end && (t - t0 >= kWindow || s_slot[t - t0] >= 0); };

    Turn<INTERLEAVED> w;
    bool bad = false;  // an infinity or NaN among the values
    const int passes = (end - first + kWindow - 1) / kWindow;
    for (int pass = 0; pass < passes; ++pass) {  // the largest magnitudes
        const int t = first + pass * kWindow + at.row;
        const bool in = in_run(t);
        const int run = run_of(t);
        if (in) at.angles(p, s_turn, t, w);
#pragma unroll 1
        for (int h = 0; h < nh; h += kHeads) {
            if (pass + h > 0) fetch(t, h, in);
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                unsigned top = 0u;  // of the bits: as numbers, in the same order
                if (in && h + i < nh) {
                    float a[8], c[8];
                    unpack8(x[i], a);
                    unpack8(y[i], c);
                    if (at.turns) w.rotate(a, c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, max(abs_bits(a[e]), abs_bits(c[e])));
                    if (top >= kInfBits) {
                        bad = true;
                        top = 0u;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (abs_bits(a[e]) < kInfBits) top = max(top, abs_bits(a[e]));
                            if (abs_bits(c[e]) < kInfBits) top = max(top, abs_bits(c[e]));
                        }
                    }
                }
#pragma unroll
                for (int o = UPR / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (in && at.j == 0 && h + i < nh) atomicMax(&s_amax[h + i][run], (int)top);
            }
        }
    }
    const bool any_bad = __syncthreads_or(bad) != 0;
    bool grew = false;
    for (int k = tid; k < nh * kWindow; k += THREADS) {  // the scales
        const int h = k / kWindow, i = k % kWindow;
        if (!(lead >> i & 1ull)) continue;
        const int s = s_slot[i];
        const int per_page = 1 << (p.page_shift - p.block_shift);
        float* scale = p.scale[side] + ((long long)(s >> p.page_shift) * p.H_kv + h0 + h) * per_page +
                       ((s & ((1 << p.page_shift) - 1)) >> p.block_shift);
        const float need = scale_for(__int_as_float(s_amax[h][i]));
        float now = need, ratio = 1.f;
        if ((s & bmask) != 0) {
            const float before = *scale;
            now = fmaxf(before, need);
            if (!(before >= now)) {
                ratio = before / now;
                grew = true;
            }
        }
        s_scale[h][i] = now;
        s_ratio[h][i] = ratio;
        *scale = now;
    }
    const bool any_grew = __syncthreads_or(grew) != 0;
    for (int pass = passes - 1; pass >= 0; --pass) {  // the codes; the last pass's angles and last heads are at hand
        const int t = first + pass * kWindow + at.row;
        if (!in_run(t)) continue;
        if (pass != passes - 1) at.angles(p, s_turn, t, w);
        const int run = run_of(t);
        const int s = s_slot[run] + (t - t0 - run);  // a run's slots follow one another
#pragma unroll 1
        for (int h = (nh - 1) / kHeads * kHeads; h >= 0; h -= kHeads) {
            if (pass != passes - 1 || h + kHeads < nh) fetch(t, h, true);
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (h + i < nh) {
                    float a[8], c[8];
                    unpack8(x[i], a);
                    unpack8(y[i], c);
                    if (at.turns) w.rotate(a, c);
                    const float now = s_scale[h + i][run];
                    uint2 ca, cc;
                    if (!any_bad && is_pow2(now)) {
                        // 1 / now: its exponent negated (now is 2^-126 to 2^126; above, the quotient would be subnormal)
                        const float inv = __uint_as_float(0x7f000000u - __float_as_uint(now));
                        ca = codes8(a, inv);
                        cc = codes8(c, inv);
                    } else {
                        ca = codes8_careful(a, now);
                        cc = codes8_careful(c, now);
                    }
                    uint8_t* dst = p.codes[side] + ((long long)s * p.H_kv + h0 + h + i) * D;
                    *reinterpret_cast<uint2*>(dst + at.off_a) = ca;
                    *reinterpret_cast<uint2*>(dst + at.off_b) = cc;
                }
        }
    }
    if (!any_grew) return;
    for (unsigned long long left = lead; left != 0ull; left &= left - 1) {  // rows that were there, under a larger scale now
        const int i = __ffsll((long long)left) - 1;
        const int s = s_slot[i], held = s & bmask;
        if (held == 0) continue;
        for (int h = 0; h < nh; ++h) {
            const float ratio = s_ratio[h][i];
            if (ratio == 1.f) continue;
            for (int r = at.row; r < held; r += kWindow) {
                uint4* word4 = reinterpret_cast<uint4*>(p.codes[side] + ((long long)(s - held + r) * p.H_kv + h0 + h) * D + at.j * 16);
                uint4 old = *word4;
                uint32_t* word = reinterpret_cast<uint32_t*>(&old);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 lo = values2((uint16_t)word[e]), hi = values2((uint16_t)(word[e] >> 16));
                    word[e] = pack_e4m3x4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
                }
                *word4 = old;
            }
        }
    }
}

// ---------------------------------------------------------------- reading back

struct Read8Params {
    const uint8_t* codes[2];
    const float* scale[2];
    char* out[2];
    const int32_t* table;
    const int32_t* cu;
    unsigned* status;
    int B, total, H_kv, d, page_shift, block_shift, max_pages, num_pages;
    int sides;               // 2: K and V; 1: one of them, in place 0
};

constexpr int kReadRows = 8;  // rows of a CTA

// Offsets a, b of a request that are in order, in range, and not of more keys than its table holds.
__device__ __forceinline__ bool read_ok(const Read8Params& p, int a, int b) {
    return a >= 0 && b >= a && b <= p.total && (long long)b - a <= ((long long)p.max_pages << p.page_shift);
}

// Bound by memory: a code is read, two bytes (or four) written.  A CTA takes 8 rows of K and V: their
// requests and cache rows are looked up once, then each thread moves 16 codes at a time.  Measured: 57 thousand keys of 8
// heads, d = 128, 57 us, 0.91 of a copy; 777 keys of 2 heads 2.4 us.
template <int EB>
__global__ void __launch_bounds__(kReadThreads) read8_kernel(const __grid_constant__ Read8Params p) {
    __shared__ int s_row[kReadRows];  // cache row, -1: left as it is, -2: zeros
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * kReadRows;
    // the offsets are looked through by warps that wait for the first one's search: a bad pair need not have a row that finds it
    constexpr int kLookers = kReadThreads - 32;
    if (tid >= 32)
        for (long long r = (long long)blockIdx.x * kLookers + tid - 32; r < p.B; r += (long long)gridDim.x * kLookers)
            if (!read_ok(p, __ldg(p.cu + r), __ldg(p.cu + r + 1))) atomicOr(p.status, 1u << kStatusDeviceData);
    if (tid < kReadRows) {
        const int t = t0 + tid;
        int row = -1;
        if (t < p.total) {
            int lo = 0, hi = p.B - 1;  // the last request that begins at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldg(p.cu + mid) <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int a = __ldg(p.cu + lo), b = __ldg(p.cu + lo + 1);
            if (t >= a && t < b && read_ok(p, a, b)) {
                const int key = t - a;
                const int id = __ldg(p.table + (long long)lo * p.max_pages + (key >> p.page_shift));
                if (id >= 0 && id < p.num_pages) {
                    row = (id << p.page_shift) + (key & ((1 << p.page_shift) - 1));
                } else {
                    row = -2;
                    atomicOr(p.status, 1u << kStatusDeviceData);
                }
            }
        }
        s_row[tid] = row;
    }
    __syncthreads();
    const int units = p.H_kv * (p.d / 16);  // pieces of 16 codes in a row
    const int per_page = 1 << (p.page_shift - p.block_shift);
    for (int x = tid; x < kReadRows * units; x += kReadThreads) {
        const int i = x / units, u = x - i * units;
        const int row = s_row[i];
        if (row == -1) continue;
        const int h = u / (p.d / 16);
        for (int side = 0; side < p.sides; ++side) {
            uint4 c = make_uint4(0u, 0u, 0u, 0u);
            float s = 0.f;
            if (row >= 0) {
                c = __ldcs(reinterpret_cast<const uint4*>(p.codes[side] + (long long)row * units * 16 + u * 16));
                s = __ldg(p.scale[side] + ((long long)(row >> p.page_shift) * p.H_kv + h) * per_page +
                          ((row & ((1 << p.page_shift) - 1)) >> p.block_shift));
            }
            const uint32_t* word = reinterpret_cast<const uint32_t*>(&c);
            char* dst = p.out[side] + ((long long)(t0 + i) * units + u) * 16 * EB;
            float f[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = values2((uint16_t)word[e]), hi = values2((uint16_t)(word[e] >> 16));
                f[4 * e] = lo.x * s;
                f[4 * e + 1] = lo.y * s;
                f[4 * e + 2] = hi.x * s;
                f[4 * e + 3] = hi.y * s;
            }
            if (EB == 2) {
#pragma unroll
                for (int e = 0; e < 16; e += 8)
                    *reinterpret_cast<uint4*>(dst + e * 2) = make_uint4(pack_bf16(f[e], f[e + 1]), pack_bf16(f[e + 2], f[e + 3]),
                                                                        pack_bf16(f[e + 4], f[e + 5]), pack_bf16(f[e + 6], f[e + 7]));
            } else {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4*>(dst + e * 4) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
        }
    }
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
int shift_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

attn_status_t blocks_ok(int page_size, int block, int num_pages) {
    if (num_pages < 1 || page_size < 1 || block < 1 || block > page_size) return ATTN_ERR_INVALID_ARG;
    if (!pow2(page_size) || page_size < 8 || page_size > 1024 || !pow2(block)) return ATTN_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

}  // namespace attn

using namespace attn;

extern "C" {

attn_status_t attn_paged_append_fp8(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                                    void* v_cache, float* k_scale, float* v_scale, const int32_t* slots,
                                    const int32_t* positions, const void* inv_freq, int freq_bits, int T, int H,
                                    int H_kv, int d, int rot, int page_size, int block, int num_pages,
                                    const long long* strides, int interleaved, float amplitude, void* stream) {
    attn_status_t st = append_args_ok(q, q_out, k, v, k_cache, v_cache, slots, positions, inv_freq, freq_bits, T, H, H_kv,
                                      d, rot, page_size, num_pages, strides, interleaved, amplitude);
    if (st != ATTN_OK) return st;
    st = blocks_ok(page_size, block, num_pages);
    if (st != ATTN_OK) return st;
    if (T > 0x7fffffff - 2048) return ATTN_ERR_INVALID_ARG;  // a run reaches at most 1024 tokens past its window
    if (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)) return ATTN_ERR_INVALID_ARG;
    unsigned* status = nullptr;
    int sm_count = 0;
    st = status_word_address(&status, &sm_count);
    if (st != ATTN_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);

    Append8Params p;
    std::memset(&p, 0, sizeof p);
    const void* in[2] = {k, v};
    void* out[2] = {k_cache, v_cache};
    float* scale[2] = {k_scale, v_scale};
    for (int i = 0; i < 2; ++i) {
        p.in[i] = static_cast<const char*>(in[i]);
        p.it[i] = strides[4 + 2 * i] * 2;
        p.ih[i] = strides[5 + 2 * i] * 2;
        p.codes[i] = static_cast<uint8_t*>(out[i]);
        p.scale[i] = scale[i];
    }
    p.slots = slots;
    p.positions = positions;
    p.freq = inv_freq;
    p.status = status;
    p.n_slots = (long long)num_pages * page_size;
    p.freq64 = freq_bits == 64;
    p.T = T;
    p.H_kv = H_kv;
    p.d = d;
    p.rot = rot;
    p.page_shift = shift_of(page_size);
    p.block_shift = shift_of(block);
    p.amplitude = amplitude;
    // CTAs: as many heads to each, up to 8 (q: 64), as leave one of K or V, and two of q, to every SM
    const int want = 2 * sm_count;
    const long long windows = ((long long)T + kWindow - 1) / kWindow;
    p.hpc = H_kv < kMaxHeads ? H_kv : kMaxHeads;
    while (p.hpc > 1 && 2 * windows * ((H_kv + p.hpc - 1) / p.hpc) < sm_count) p.hpc = (p.hpc + 1) / 2;
    p.splits = (H_kv + p.hpc - 1) / p.hpc;
    long long ctas = 2 * windows * p.splits, q_ctas = 0;
    if (ctas > 0x3fffffffLL) return ATTN_ERR_INVALID_ARG;
    p.kv_ctas = (unsigned)(windows * p.splits);
    if (q) {
        const long long tiles = windows;
        p.q = static_cast<const char*>(q);
        p.q_out = static_cast<char*>(q_out);
        p.qt = strides[0] * 2;
        p.qh = strides[1] * 2;
        p.qot = strides[2] * 2;
        p.qoh = strides[3] * 2;
        p.H = H;
        p.q_hpc = H < 64 ? H : 64;
        while (p.q_hpc > 1 && tiles * ((H + p.q_hpc - 1) / p.q_hpc) < want) p.q_hpc = (p.q_hpc + 1) / 2;
        p.q_splits = (H + p.q_hpc - 1) / p.q_hpc;
        p.q_stream = (long long)T * H * d * 2 > kStreamBytes;
        q_ctas = tiles * p.q_splits;
    }
    if (ctas + q_ctas > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    const unsigned grid = (unsigned)(ctas + q_ctas);
    if (d == 128) {
        if (interleaved)
            append8_kernel<128, true><<<grid, 4 * d, 0, cs>>>(p);
        else
            append8_kernel<128, false><<<grid, 4 * d, 0, cs>>>(p);
    } else {
        if (interleaved)
            append8_kernel<64, true><<<grid, 4 * d, 0, cs>>>(p);
        else
            append8_kernel<64, false><<<grid, 4 * d, 0, cs>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_paged_read_fp8(const void* k_cache, const void* v_cache, const float* k_scale,
                                  const float* v_scale, const int32_t* block_table, const int32_t* cu_seqlens_k,
                                  int B, int total_k, int H_kv, int d, int page_size, int block, int max_pages,
                                  int num_pages, void* k, void* v, int elem_bytes, void* stream) {
    if (!block_table || !cu_seqlens_k || (!k && !v)) return ATTN_ERR_INVALID_ARG;
    if ((k && (!k_cache || !k_scale)) || (v && (!v_cache || !v_scale))) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || total_k < 1 || total_k > 0x7fffffff - kReadRows || H_kv < 1 || H_kv > 65535 || max_pages < 1)
        return ATTN_ERR_INVALID_ARG;
    attn_status_t st = blocks_ok(page_size, block, num_pages);
    if (st != ATTN_OK) return st;
    if ((d != 64 && d != 128) || (elem_bytes != 2 && elem_bytes != 4)) return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size > 0x7fffffffLL || (long long)B * max_pages > 0x7fffffffLL)
        return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {static_cast<const void*>(k), static_cast<const void*>(v), k ? k_cache : nullptr,
                            v ? v_cache : nullptr})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(cu_seqlens_k, 4) || (k && !aligned(k_scale, 4)) || (v && !aligned(v_scale, 4)))
        return ATTN_ERR_INVALID_ARG;
    Read8Params p;
    std::memset(&p, 0, sizeof p);
    st = status_word_address(&p.status);
    if (st != ATTN_OK) return st;
    auto add = [&](const void* codes, const float* scale, void* out) {
        p.codes[p.sides] = static_cast<const uint8_t*>(codes);
        p.scale[p.sides] = scale;
        p.out[p.sides++] = static_cast<char*>(out);
    };
    if (k) add(k_cache, k_scale, k);
    if (v) add(v_cache, v_scale, v);
    p.table = block_table;
    p.cu = cu_seqlens_k;
    p.B = B;
    p.total = total_k;
    p.H_kv = H_kv;
    p.d = d;
    p.page_shift = shift_of(page_size);
    p.block_shift = shift_of(block);
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    const unsigned blocks = (unsigned)((total_k + kReadRows - 1) / kReadRows);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (elem_bytes == 2)
        read8_kernel<2><<<blocks, kReadThreads, 0, cs>>>(p);
    else
        read8_kernel<4><<<blocks, kReadThreads, 0, cs>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
