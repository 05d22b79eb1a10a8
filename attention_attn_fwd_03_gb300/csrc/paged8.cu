// paged8.cu -- attention over a paged cache of e4m3 codes with block scales.
//
//   s_j = scale ks_j (q . kc_j),  p_j = e^(s_j),  O = sum p_j vs_j vc_j / sum p_j,  LSE = ln sum p_j
//
// (kc, vc: codes; ks, vs: the scales of key j's block), by the one-pass online
// softmax (running maximum, sum and unnormalised O, one final division).
//
// What bounds it.  A decode step reads every code once and computes 4 G d flops for
// 2 d bytes (G query heads to a KV head): HBM.  At its rate an SM gets some 23 bytes a
// cycle, too many to convert to 16 bits on the way: so the codes go from the cache to the
// matrix units as they are, by TMA into swizzled shared memory and from there as e4m3
// operands of tcgen05.mma (kind::f8f6f4).  The other operands have few rows, so their
// precision is bought with more rows:
//   q = 2^x (hi + lo / 16): a bf16 number has 8 significant bits, two e4m3 numbers hold
//       them; x by the head vector's largest element.
//   P vs / 2^(running maximum) = hi + mid + (lo + end) / 64: an fp16 number's 11 bits in four e5m2 numbers of 3.
//       These have the range that small probabilities need: a long tail of them may be all of O, where the large
//       ones' values are near zero.  (Three e4m3 numbers hold 11 bits down to 2^-13 of the row's largest only, and
//       nothing below 2^-24; the matrix unit takes e4m3 by e5m2.)
// Both products are transposed, so that keys (or channels) fill the 128 rows of the
// matrix instruction and query rows its columns:
//   S^T [128 keys, 2 R] = Kc [128, d] Q^T,    O^T [d, 2 R or 4 R] += Vc^T [d, 128 keys] P^T,
// R = 8, 16 or 32 query rows (tokens times the heads of a group; those of two KV heads, if a
// unit has two: each head's rows meet that head's codes only).  A thread of the softmax
// then has one key and 8 rows: no thread is idle.  It takes 32 / R tiles of 128 keys (a step) at a time:
// one test per step, over all threads, whether a row's maximum grew by more than kTau.
//
// Work split.  Requests, KV heads (or pairs of them: paged8_plan), row tiles and key tiles in a row, cut into equal shares,
// one for each CTA (two to an SM, so that one's softmax runs during the other's loads).  Each
// CTA computes the cut from the lengths.  A unit (request, head or pair, row tile) that lies in one
// CTA is finished there; pieces of others leave (m, l, O), merged by a second kernel.
//
// A CTA, 384 threads:
//   warp 0    TMA producer: the units, their pages, K and V tiles into a ring, in the order
//             K of step n + 1, V of step n.
//   warp 1    MMA issuer (one lane); the warp clears rows past the request's keys.
//   warps 2-9 softmax and epilogue: thread = key, then thread = channel.
//   warp 10   query rows as e4m3 pairs.
//   warp 11   the scales of the steps' keys.
//
// Measured (inputs from HBM, d = 128, 32 heads over 8 unless said).  4 requests of 200 to 262 thousand keys: 287 to 319 us
// on different GPUs, 5.9 to 6.6 TB/s (a copy: 6.8); 64 of 512 to 8192: 99 to 108 us, 5.3 to 5.8 TB/s; 33 of 0 to 4096 with
// 16 heads over 16: 58 us; one of 32 thousand (which stays in L2): 22 us; 1 to 8 tokens of 16 requests, d = 64, 16 heads over 2,
// a scale to every token: 53 us, 0.9 of it in the softmax.  16 requests of 8192, by query rows (tokens times heads of a
// group) to each of 8 KV heads: 4 to 8 57 to 60 us, 16 68 to 70, 32 117, 64 210, 128 394, where reading the codes back and attn_varlen_fwd
// take 244 for 64 and 269 for 128.  A call of one tile takes 11 us: 4 until the first page is asked
// for, 4 for the tile, 2 to 3 for the merge; a unit's start and end, and the last CTAs' lead over the mean, take most of what
// is not streaming in the others.
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

// How far a row's maximum may lag behind, in log2 units, and the scale of P, which is 2^(kTau + kBase) = 2^15 at most: e5m2
// numbers reach 1.75 2^15, fp16 numbers as far.  hi leaves 2^-3 of a number, mid 2^-3 of that: 64 times what is left then
// is 2^15 at most again.  The smallest step is 2^-16 / 64: with fp16's own, 2^-24, P is off by less than 2^-33 of the
// row's largest, and by 2^-11 of itself where that is more.
constexpr float kTau = 4.f;
constexpr float kBase = 11.f;
// log2 of how much smaller the values' scales may be than 1 before P gets smaller than kBase says: so far P's factor,
// 2^(kVMin + kBase), and its inverse at the unit's end are normal numbers.
constexpr float kVMin = 112.f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kThreads8 = 384;
constexpr float kHuge = 3e38f;
constexpr int kQN = 4;            // unit queue between the producer and the other warps
constexpr int kUnitInts = 10;
constexpr int kMiscFirst = 30;   // place in the misc words of the first request's extent
constexpr int kMinShare = 1;      // tiles
// What a unit's start and end take, in tiles of 128 keys (33 requests of up to 4096 keys, 16 heads: 63 us with 1, 57 with
// 2, 59 with 3).
constexpr int kUnitCost = 2;

template <int D, int R, int NH>
struct Cfg {
    static constexpr int SB = 32 / R;                  // key tiles of a step
    static constexpr int RH = R / NH;                  // rows of a head
    static constexpr bool WIDE = NH == 2 && D == 64;   // a tile holds the codes of two heads, side by side
    static constexpr int TPK = NH == 2 && D == 128 ? 2 : 1;  // tiles to 128 keys: one for each head
    static constexpr int W = WIDE ? 128 : D;           // bytes of a tile's row
    static constexpr int PH = TPK == 2 ? RH : R;       // rows of a P operand
    // hi and mid may share O's columns, as lo and end may: half as many to rescale, for twice as many instructions.  Drafted
    // tokens in units of 32 rows take 53.2 us so, 57.0 with columns for each; with 8 rows to an operand one request of 32 thousand keys
    // takes 22.9 and 22.2, 33 requests with 16 heads 59.3 and 57.8, four long ones 314 and 317.
    static constexpr bool FOLD = R == 32;
    static constexpr int NPV = (FOLD ? 2 : 4) * PH;    // columns of O^T
    static constexpr int TILE = 128 * W;               // bytes of a K or V tile
    static constexpr int NST = (SB * NH == 4 ? 5 : 4) * 128 / W;  // ring stages
    static constexpr int QBYTES = 2 * R * D;
    // A tile of P: keys as its rows and hi, lo, mid, end of the query rows side by side in each (a thread's eight rows are then
    // eight bytes: 53.5 us instead of 55.4 for 1 to 8 tokens of 16 requests); for 8 rows hi, lo, mid and end as its rows.
    static constexpr bool KEYS = PH >= 16;
    static constexpr int WP = PH == 32 ? 128 : PH == 16 ? 64 : 128;  // bytes of a row of P, and its swizzle
    static constexpr int PTILE = KEYS ? 128 * WP : 4 * PH * 128;
    static constexpr int PBUF = SB * NH == 4 || TPK == 2 || R == 32 ? 1 : 2;  // steps' P held at once
    // Steps' scales held at once: they are read at a step's start, and the next ones' come during the rest of it.  Two heads'
    // tiles of P leave room for one step only.
    static constexpr int SCB = TPK == 2 && R == 16 ? 1 : 2;
    static constexpr uint32_t TM_O = 128;              // S: two buffers of 64 columns
    static constexpr uint32_t TM_COLS = 256;
    static constexpr int OFF_KV = 0;
    static constexpr int OFF_P = OFF_KV + NST * TILE;
    static constexpr int OFF_Q = OFF_P + PBUF * SB * TPK * PTILE;
    static constexpr int OFF_SC = OFF_Q + 2 * QBYTES;                 // float2 [SCB][NH][SB * 128]: ks, vs of 1 .. 16 keys
    static constexpr int OFF_ROW = OFF_SC + SCB * NH * SB * 128 * 8;    // int4 [2][R]: factor, last visible key, output row
    static constexpr int OFF_STAT = OFF_ROW + 2 * R * 16;             // float2 [R]: running maxima of s and of s + log2 vs
    static constexpr int OFF_PAR = OFF_STAT + R * 8;                  // float2 [R]: the maximum, and P's factor
    static constexpr int OFF_ALPHA = OFF_PAR + R * 8;                 // float2 [R]
    static constexpr int OFF_EXCH = OFF_ALPHA + R * 8;                // float2 [8][R]
    static constexpr int OFF_SUM = OFF_EXCH + 8 * R * 8;              // float [8][R]
    static constexpr int OFF_NAN = OFF_SUM + 8 * R * 4;               // int [NH * D]: first row that sees a NaN in this channel
    static constexpr int OFF_BAR = OFF_NAN + NH * D * 4;
    static constexpr int N_BARS = 2 * NST + 15 + 2 * kQN;
    static constexpr int OFF_UQ = OFF_BAR + 8 * N_BARS;
    static constexpr int OFF_MISC = OFF_UQ + 4 * kQN * kUnitInts;
    static constexpr int SMEM_BYTES = OFF_MISC + 144 + 1024;
    static_assert(SMEM_BYTES <= 115712, "two CTAs to an SM");
    static_assert(TPK * NPV <= 128, "columns of O^T");
    static_assert(OFF_P % 1024 == 0 && PTILE % 1024 == 0 && OFF_Q % 1024 == 0 && QBYTES % 1024 == 0, "swizzle atoms");
};

struct Bars {
    uint64_t* kv_full;   // [NST]
    uint64_t* kv_empty;  // [NST]
    uint64_t* q_full;    // [2] query rows prepared
    uint64_t* q_empty;   // [2] the unit's last S product, and the eight softmax warps
    uint64_t* sc_full;   // [SCB] scales of a step: 32 lanes' copies
    uint64_t* sc_empty;  // [SCB] eight softmax warps
    uint64_t* s_full;    // [2]
    uint64_t* p_full;    // [2] 256 arrivals per step
    uint64_t* o_full;    // [2] PV products of a step, and the issuing lane
    uint64_t* done;
    uint64_t* uq_full;   // [kQN]
    uint64_t* uq_empty;  // [kQN] eleven readers
};

// A piece of a unit: key tiles [tile0, tile0 + nt) for rows [row0, row0 + nr) of request r and NH KV heads from
// kvh * NH.  A head's row x is query token x / G of the request, head x % G of the group.
struct Unit {
    int r;  // -1: no more
    int kvh, q_start, q_len, kv_len, row0, nr, tile0, nt;
    int slot;  // partial record, -1: the whole unit
};

struct Extent {
    int q_start, q_len, kv_len;
    bool bad;
};

// A request's numbers as they are in memory, and what they say.
struct Raw {
    int q0, q1, len;
};
__device__ __forceinline__ Raw raw_extent(const Paged8Params& p, int r) {
    Raw x;
    x.q0 = r;
    x.q1 = r + 1;
    if (p.cu_q != nullptr) {
        x.q0 = __ldg(p.cu_q + r);
        x.q1 = __ldg(p.cu_q + r + 1);
    }
    x.len = __ldg(p.seq_lens + r);
    return x;
}
__device__ __forceinline__ Extent extent_of(const Paged8Params& p, const Raw& x) {
    Extent e;
    e.bad = false;
    e.q_start = x.q0;
    e.q_len = 1;
    if (p.cu_q != nullptr) {
        const int a = x.q0, b = x.q1;
        e.q_start = a;
        e.q_len = b - a;
        if (a < 0 || b < a || b > p.total_q || e.q_len > p.max_q_len) {
            e.bad = true;
            e.q_start = 0;
            e.q_len = 0;
        }
    }
    e.kv_len = x.len;
    const int cap = p.max_pages << p.page_shift;
    if (e.kv_len < 0 || e.kv_len > cap) {
        e.bad = true;
        e.kv_len = e.kv_len < 0 ? 0 : cap;
    }
    return e;
}

__device__ __forceinline__ Extent extent(const Paged8Params& p, int r) { return extent_of(p, raw_extent(p, r)); }

// Key tiles of every unit of a request (one at least, so that its rows are written), its row tiles, and its
// size in the cut, where each unit counts kUnitCost tiles more: what its start and end take.
__device__ __forceinline__ int key_tiles(const Extent& e) { return max(1, (int)(((long long)e.kv_len + 127) / 128)); }
template <int RH>
__device__ __forceinline__ int row_tiles(const Paged8Params& p, const Extent& e) { return (e.q_len * p.G + RH - 1) / RH; }
template <int RH>
__device__ __forceinline__ long long work_of(const Paged8Params& p, const Extent& e) {
    return (long long)p.kv_units * row_tiles<RH>(p, e) * (key_tiles(e) + kUnitCost);
}

// a / b (both positive, the quotient an int), by a 32-bit division where that will do: the 64-bit one takes a noticeable
// part of a short call.
__device__ __noinline__ long long long_quotient(long long a, long long b) { return a / b; }
__device__ __forceinline__ int quotient(long long a, long long b) {
    return a < 0x7fffffffLL && b < 0x7fffffffLL ? (int)((unsigned)a / (unsigned)b) : (int)long_quotient(a, b);
}

__device__ __forceinline__ void publish(volatile int* q, const Unit& u) {
    q[0] = u.r; q[1] = u.kvh; q[2] = u.q_start; q[3] = u.q_len; q[4] = u.kv_len;
    q[5] = u.row0; q[6] = u.nr; q[7] = u.tile0; q[8] = u.nt; q[9] = u.slot;
}
__device__ __forceinline__ Unit read_unit(const volatile int* q) {
    Unit u;
    u.r = q[0]; u.kvh = q[1]; u.q_start = q[2]; u.q_len = q[3]; u.kv_len = q[4];
    u.row0 = q[5]; u.nr = q[6]; u.tile0 = q[7]; u.nt = q[8]; u.slot = q[9];
    return u;
}

// Position of row x of a unit's request in the request, and with the causal mask its last visible key.
__device__ __forceinline__ int last_key(const Paged8Params& p, const Unit& u, int x) {
    if (!p.causal || u.q_len == 1) return u.kv_len - 1;
    return (int)min((long long)u.kv_len - 1, (long long)u.kv_len - u.q_len + x / p.G);
}

// wait_bar (ptx.cuh) with all but its first look out of line: this kernel waits in many places, and what is executed
// has to fit the instruction cache.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
    return wait_bar(bar, parity, abort_flag, status);
}
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
    return bar_try_wait(bar, parity) || wait_on(bar, parity, abort_flag, status);
}
// A whole warp's wait: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
    return __all_sync(0xffffffffu, wait_short(bar, parity, abort_flag, status));
}

__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void st_u8(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_v2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

// 16 or 4 bytes from global to shared memory, or zeros; and the wait for a thread's own.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {  // this thread's arrival, once its copies are there
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Two fp16 numbers -> two e5m2 numbers (nearest, saturating; NaN stays NaN), and back: an e5m2 number is an fp16
// number's upper byte.
__device__ __forceinline__ uint32_t e5m2_of(uint32_t h2) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
    return r;
}
__device__ __forceinline__ uint32_t half2_of_e5m2(uint32_t e) { return __byte_perm(e, 0u, 0x1404); }
// Two e4m3 numbers -> two fp16 numbers.
__device__ __forceinline__ uint32_t half2_of(uint32_t e) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)e));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_mul64(uint32_t a) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x54005400u));  // 64
    return r;
}

// Shared-memory descriptor of an operand tile: rows of W bytes with a swizzle of W bytes, 8-row groups 8 W bytes
// apart.  The same bytes serve as a K-major operand (rows are M or N) and as an MN-major one (rows are K).
template <int W>
__device__ __forceinline__ uint64_t desc(uint32_t addr) {
    uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)1u << 16;
    d |= (uint64_t)((8 * W) >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)(W == 128 ? 2u : 4u) << 61;
    return d;
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (a finite amax).
__device__ __forceinline__ float scale_for(float amax) {
    const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;
    return __uint_as_float((unsigned)max(e, 1) << 23);
}

// ---------------------------------------------------------------- producer (whole warp)

template <int D, int R, int NH>
__device__ void producer_role(const Paged8Params& p, uint8_t* smem, const Bars& b, volatile int* uq, volatile int* abort_flag,
                              int lane, int r, long long w, long long w1, long long start, Extent e,
                              long long share) {
    using C = Cfg<D, R, NH>;
    if (lane == 0) {
        tma_prefetch_map(&p.tm_k);
        tma_prefetch_map(&p.tm_v);
    }
    const int rows = p.rows_per_box, per_tile = 128 / rows;  // boxes of a tile: 1 .. 16
    const long long w0 = w;
    int kv_idx = 0, pub = 0;
    bool ok = true;
    // lane i: request base + i (the first one's extent is known: the loads are not waited for)
    int base = r;
    Raw mine = raw_extent(p, min(base + lane, p.B - 1));
    int prev_rows[2] = {0, 0}, prev_nt = 0, prev_kvh = 0;  // the step whose V tiles are due
    Unit u{};
    int s = 0, id[2] = {-1, -1};
    auto page_ids = [&](int from, int* ids) {  // of the boxes of a step (box x in lane x % 32, register x / 32)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int x = k * 32 + lane;
            const long long key = (long long)(u.tile0 + from) * 128 + (long long)x * rows;
            ids[k] = -1;
            if (x < min(C::SB, u.nt - from) * per_tile && key < u.kv_len)
                ids[k] = __ldg(p.block_table + (size_t)u.r * p.max_pages + (key >> p.page_shift));
        }
    };
    while (ok) {
        if (s >= u.nt) {  // the next unit of the cut
            long long past = -1;  // its last place, if it begins here and goes on in the CTAs after this one
            s = 0;
            u.r = -1;
            u.nt = 0;
            while (w < w1) {
                const long long work = work_of<C::RH>(p, e);
                if (w - start >= work) {
                    start += work;
                    if (++r >= base + 32) {
                        base = r;
                        mine = raw_extent(p, min(base + lane, p.B - 1));
                    }
                    e = extent_of(p, Raw{__shfl_sync(0xffffffffu, mine.q0, r - base), __shfl_sync(0xffffffffu, mine.q1, r - base),
                                         __shfl_sync(0xffffffffu, mine.len, r - base)});
                    continue;
                }
                const int nb = key_tiles(e), nqt = row_tiles<C::RH>(p, e), size = nb + kUnitCost;
                const long long off = w - start;
                const int unit = quotient(off, size);
                int at = (int)(off - (long long)unit * size);  // place in the unit: kUnitCost, then its tiles
                if (at < kUnitCost) {
                    w += kUnitCost - at;
                    at = kUnitCost;
                    if (w >= w1) break;
                }
                const int tile = at - kUnitCost;
                const int n = (int)min((long long)(nb - tile), w1 - w);
                u.r = r;
                u.kvh = nqt == 1 ? unit : unit / nqt;
                u.q_start = e.q_start;
                u.q_len = e.q_len;
                u.kv_len = e.kv_len;
                u.row0 = (unit - u.kvh * nqt) * C::RH;
                u.nr = min(C::RH, e.q_len * p.G - u.row0);
                u.tile0 = tile;
                const long long seen = (last_key(p, u, u.row0 + u.nr - 1) + 128LL) / 128;  // tiles that the last row sees
                u.nt = (int)max(0LL, min((long long)n, seen - tile));
                u.slot = n == nb ? -1 : 2 * (int)blockIdx.x + (w - tile <= w0 ? 0 : 1);
                if (tile == 0 && n < nb) past = w + nb - 1;
                w += n;
                break;
            }
            page_ids(0, id);
            if (lane == 0) {
                const int slot = pub % kQN;
                if (pub >= kQN) ok = wait_short(&b.uq_empty[slot], (uint32_t)((pub / kQN - 1) & 1), abort_flag, p.status);
                if (ok) {
                    publish(uq + slot * kUnitInts, u);
                    bar_arrive(&b.uq_full[slot]);
                    if (past >= 0) {  // for the merge
                        int4* cut = p.cuts + 2 * blockIdx.x;
                        cut[0] = make_int4(quotient(past, share), u.slot, u.nr, u.kvh);
                        cut[1] = make_int4(u.q_start, u.row0, 0, 0);
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ++pub;
        }
        const int nt = min(C::SB, u.nt - s);  // 0: a unit without visible keys, or the end: only V tiles may be due
        int row_of[2], next_id[2];
        page_ids(s + nt, next_id);            // loaded a step before they are used
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int x = k * 32 + lane;
            const long long key = (long long)(u.tile0 + s) * 128 + (long long)x * rows;
            row_of[k] = p.kv_rows;
            if (id[k] >= 0 && id[k] < p.num_pages)
                row_of[k] = (id[k] << p.page_shift) + (int)(key & ((1 << p.page_shift) - 1));
            else if (x < nt * per_tile && key < u.kv_len)
                atomicOr(p.status, 1u << kStatusDeviceData);
            id[k] = next_id[k];
        }
        // K of this step, then V of the one before
#pragma unroll 1
        for (int t = 0; t < (nt + prev_nt) * C::TPK; ++t) {
            const bool is_k = t < nt * C::TPK;
            const int slot = kv_idx % C::NST, round = kv_idx / C::NST;
            if (lane == 0) {
                if (round > 0) ok = wait_short(&b.kv_empty[slot], (uint32_t)((round - 1) & 1), abort_flag, p.status);
                if (ok) bar_arrive_expect_tx(&b.kv_full[slot], C::TILE);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            const int x = is_k ? t : t - nt * C::TPK;
            const int first = x / C::TPK * per_tile;  // per_tile divides 32: the tile's boxes lie in one register
            const int i = lane - (first & 31);
            const int* from = is_k ? row_of : prev_rows;
            if (i >= 0 && i < per_tile)
                tma_load_3d(smem + C::OFF_KV + slot * C::TILE + i * rows * C::W, is_k ? &p.tm_k : &p.tm_v, &b.kv_full[slot], 0,
                            (is_k ? u.kvh : prev_kvh) * C::TPK + x % C::TPK, first < 32 ? from[0] : from[1]);
            ++kv_idx;
        }
        prev_rows[0] = row_of[0];
        prev_rows[1] = row_of[1];
        prev_nt = nt;
        prev_kvh = u.kvh;
        s += nt;
        if (u.r < 0) break;
    }
    // every copy that this warp started must land before the CTA exits
    if (lane == 0)
#pragma unroll 1
        for (int idx = kv_idx - C::NST > 0 ? kv_idx - C::NST : 0; idx < kv_idx; ++idx)
            drain_wait(&b.kv_full[idx % C::NST], (uint32_t)((idx / C::NST) & 1), p.status);
    __syncwarp();
}

// ---------------------------------------------------------------- MMA issuer (whole warp, lane 0 issues)

// Rows of a tile past the request's keys may hold anything: cleared, since a NaN there would reach every row of the
// second product (as 0 * NaN), and the softmax masks scores by adding -inf to them.
template <int D>
__device__ __forceinline__ void clear_rows(uint32_t tile, int left, int lane) {
#pragma unroll 1
    for (int x = left * (D / 16) + lane; x < 128 * (D / 16); x += 32) st_zero16(tile + (uint32_t)x * 16u);
    fence_async_smem();
    __syncwarp();
}

// The scores of one tile.
template <int D, int R, int NH>
__device__ __forceinline__ void product_s(uint32_t d, uint64_t k, uint64_t q) {
    constexpr int N = 2 * Cfg<D, R, NH>::RH;
    constexpr uint32_t ID = idesc_make(128, N, 0u, false, false);
    if (Cfg<D, R, NH>::WIDE) {  // each head's half of the row
        mma_f8_ss(d, k, q, ID, 0u);
        mma_f8_ss(d, k + 2, q + 2, ID, 1u);
        mma_f8_ss(d + N, k + 4, q + 4, ID, 0u);
        mma_f8_ss(d + N, k + 6, q + 6, ID, 1u);
    } else if (D == 128) {
        mma4_ss<2, 4, 6, 2, 4, 6, true>(d, k, q, ID, 0u);
    } else {
        mma_f8_ss(d, k, q, ID, 0u);
        mma_f8_ss(d, k + 2, q + 2, ID, 1u);
    }
}

// One tile's part of O^T: four blocks of 32 keys.
template <int D, int R, int NH>
__device__ __forceinline__ void product_pv(uint32_t o, uint64_t v, uint64_t p, bool accumulate) {
    constexpr uint32_t ID = idesc_make(Cfg<D, R, NH>::W, Cfg<D, R, NH>::NPV, 0u, true, Cfg<D, R, NH>::KEYS) |
                            1u << 10;  // B's format: e5m2
    constexpr int VS = (32 * Cfg<D, R, NH>::W) >> 4;  // 32 rows of V in descriptor units
    constexpr int PS = Cfg<D, R, NH>::KEYS ? (32 * Cfg<D, R, NH>::WP) >> 4 : 2;
    mma4_ss<VS, 2 * VS, 3 * VS, PS, 2 * PS, 3 * PS, true>(o, v, p, ID, accumulate ? 1u : 0u);
    if (Cfg<D, R, NH>::FOLD) {  // mid and end behind hi and lo in each row of P
        static_assert(!Cfg<D, R, NH>::FOLD || Cfg<D, R, NH>::KEYS, "by keys");
        mma4_ss<VS, 2 * VS, 3 * VS, PS, 2 * PS, 3 * PS, true>(o, v, p + (2 * Cfg<D, R, NH>::PH >> 4), ID, 1u);
    }
}

// S^T of step n + 1, then O^T += V^T P^T of step n: the order of the ring.  (Two issuers, one for each product, were
// slower: which tile of the ring is whose is known only in this order, and the waits for one another cost more than the
// 300 to 500 cycles that a tile's few instructions, wait and commit take here.)
template <int D, int R, int NH>
__device__ void mma_role(const Paged8Params& p, uint8_t* smem, const Bars& b, volatile int* uq, volatile int* abort_flag,
                         uint32_t tmem, int lane) {
    using C = Cfg<D, R, NH>;
    const uint32_t sbase = smem_u32(smem), o = tmem + C::TM_O;
    constexpr int W = C::W, TPK = C::TPK;
    const uint64_t kv_desc = desc<W>(sbase + C::OFF_KV), p_desc = desc<C::WP>(sbase + C::OFF_P);
    int* s_nan = reinterpret_cast<int*>(smem + C::OFF_NAN);
    int stage = 0, phase = 0, units = 0;
    uint32_t n = 0;  // steps issued
    // the step whose second product is due: tiles, whether it is its unit's first, and what masks need of the unit
    int prev_nt = 0, prev_first = 0, prev_tile0 = 0, prev_kv_len = 0, prev_q_len = 0, prev_row0 = 0, prev_last = 0;

    // Tiles [0, count) of the ring from here on, by one lane: issue(t, tile in descriptor units) for each.
    auto tiles = [&](int count, auto issue) -> bool {
        bool ok = true;
        if (lane == 0) {
#pragma unroll 1
            for (int t = 0; t < count; ++t) {
                ok = wait_short(&b.kv_full[stage], (uint32_t)phase, abort_flag, p.status);
                if (!ok) break;
                tc_fence_after();
                issue(t, (uint64_t)(stage * (C::TILE >> 4)));
                tc_commit(&b.kv_empty[stage]);
                if (++stage == C::NST) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        stage = __shfl_sync(0xffffffffu, stage, 0);
        phase = __shfl_sync(0xffffffffu, phase, 0);
        return __shfl_sync(0xffffffffu, ok, 0);
    };
    auto next_stage = [&]() {
        if (++stage == C::NST) {
            stage = 0;
            phase ^= 1;
        }
    };
    auto second = [&](uint32_t step) -> bool {  // of the pending step, number `step`
        const int nt = prev_nt;
        const long long key0 = (long long)prev_tile0 * 128;
        const int keys = (int)min((long long)nt * 128, prev_kv_len - key0);
        // tiles without rows to clear (all but the request's last) and without keys that only some of the unit's rows see
        const int whole = prev_last < prev_kv_len - 1 && key0 + keys - 1 > prev_last ? 0 : keys / 128;
        const uint64_t p_step = p_desc + (uint64_t)((C::PBUF == 2 ? step & 1u : 0u) * (C::SB * TPK * C::PTILE >> 4));
        if (!warp_wait(&b.p_full[step & 1u], (step >> 1) & 1u, abort_flag, p.status)) return false;
        auto product = [&](int t, uint64_t tile) {
            product_pv<D, R, NH>(o + (uint32_t)(t % TPK * C::NPV), kv_desc + tile, p_step + (uint64_t)(t * (C::PTILE >> 4)),
                                 !prev_first || t >= TPK);
        };
        if (!tiles(whole * TPK, product)) return false;
#pragma unroll 1
        for (int x = whole * TPK; x < nt * TPK; ++x) {
            const int t = x / TPK;
            if (!warp_wait(&b.kv_full[stage], (uint32_t)phase, abort_flag, p.status)) return false;
            const int left = min(128, keys - t * 128);
            const uint32_t v = sbase + C::OFF_KV + (uint32_t)(stage * C::TILE);
            if (left < 128) clear_rows<W>(v, left, lane);
            if (key0 + t * 128 + left - 1 > prev_last) {
                // Keys that only some of the rows see: a NaN among their values must not reach the others
                // through 0 * NaN.  It is taken out and noted, by channel, for the rows from the first that sees it.
                const int from = (int)max(0LL, min(128LL, prev_last + 1LL - key0 - t * 128));
#pragma unroll 1
                for (int i = from * (W / 4) + lane; i < left * (W / 4); i += 32) {
                    const int key = i / (W / 4), word = i % (W / 4);  // stored word of the row, swizzled
                    const int chunk = (word >> 2) ^ (W == 128 ? key & 7 : (key >> 1) & 3);
                    const uint32_t at = v + (uint32_t)(key * W + word * 4);
                    uint32_t c;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(c) : "r"(at) : "memory");
                    uint32_t keep = c;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (((c >> (8 * k)) & 0x7fu) == 0x7fu) {
                            keep &= ~(0xffu << (8 * k));
                            // token of the first row that sees the key
                            const long long tok = key0 + t * 128 + key - ((long long)prev_kv_len - prev_q_len);
                            const int row = (int)max(0LL, tok * p.G - prev_row0);
                            atomicMin(s_nan + x % TPK * D + chunk * 16 + (word & 3) * 4 + k, row);
                        }
                    if (keep != c) st_u32(at, keep);
                }
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) {
                tc_fence_after();
                product(x, (uint64_t)(stage * (C::TILE >> 4)));
                tc_commit(&b.kv_empty[stage]);
            }
            next_stage();
        }
        __syncwarp();
        if (lane == 0) {
            tc_commit(&b.o_full[step & 1u]);
            bar_arrive(&b.o_full[step & 1u]);  // what the warp noted of NaNs
        }
        return true;
    };

    Unit u{};
    int s = 0, qb = 0, first_last = 0;  // next step of the unit; its query buffer; the last key that its first row sees
    uint64_t q_desc = 0;
    for (int k = 0;;) {
        if (s >= u.nt) {
            const int slot = k % kQN;
            if (!warp_wait(&b.uq_full[slot], (uint32_t)((k / kQN) & 1), abort_flag, p.status)) return;
            u = read_unit(uq + slot * kUnitInts);
            __syncwarp();
            if (lane == 0) bar_arrive(&b.uq_empty[slot]);
            ++k;
            s = 0;
            qb = units & 1;
            if (u.nt > 0) {
                if (!warp_wait(&b.q_full[qb], (uint32_t)((units >> 1) & 1), abort_flag, p.status)) return;
                ++units;
                q_desc = desc<W>(sbase + C::OFF_Q + (uint32_t)(qb * C::QBYTES));
                first_last = last_key(p, u, u.row0);
            }
        }
        const int nt = min(C::SB, u.nt - s);  // 0: a unit without visible keys, or the end
        if (nt > 0) {
            // (S's buffer is free: the softmax read step n - 2 before it let that step's second product go)
            const uint32_t d = tmem + (n & 1u) * 64u;
            const int keys = (int)min((long long)nt * 128, (long long)u.kv_len - (long long)(u.tile0 + s) * 128);
            const int whole = keys / 128;  // tiles without rows to clear: all but the request's last
            auto product = [&](int t, uint64_t tile) {
                product_s<D, R, NH>(d + (uint32_t)(t * (2 * R / TPK)), kv_desc + tile, q_desc + (uint64_t)(t % TPK * (C::QBYTES / TPK >> 4)));
            };
            if (!tiles(whole * TPK, product)) return;
#pragma unroll 1
            for (int t = whole * TPK; t < nt * TPK; ++t) {
                if (!warp_wait(&b.kv_full[stage], (uint32_t)phase, abort_flag, p.status)) return;
                clear_rows<W>(sbase + C::OFF_KV + (uint32_t)(stage * C::TILE), keys - whole * 128, lane);
                if (lane == 0) {
                    tc_fence_after();
                    product(t, (uint64_t)(stage * (C::TILE >> 4)));
                    tc_commit(&b.kv_empty[stage]);
                }
                next_stage();
            }
            if (lane == 0) {
                tc_commit(&b.s_full[n & 1u]);
                if (s + nt == u.nt) tc_commit(&b.q_empty[qb]);
            }
            __syncwarp();
        }
        if (prev_nt > 0 && !second(n - 1u)) return;
        if (u.r < 0) return;
        if (nt == 0) {
            // (after the products of the step before, which must not wait for this unit: its query rows wait for the
            // buffer that the unit of that step may still hold)
            if (!warp_wait(&b.q_full[qb], (uint32_t)((units >> 1) & 1), abort_flag, p.status)) return;
            ++units;
            if (lane == 0) bar_arrive(&b.q_empty[qb]);
        } else {
            ++n;
        }
        prev_nt = nt;
        prev_first = s == 0;
        prev_tile0 = u.tile0 + s;
        prev_kv_len = u.kv_len;
        prev_q_len = u.q_len;
        prev_row0 = u.row0;
        prev_last = first_last;
        s += nt;
    }
}

// ---------------------------------------------------------------- query rows (one warp)

template <int D, int R, int NH>
__device__ void query_role(const Paged8Params& p, uint8_t* smem, const Bars& b, volatile int* uq, volatile int* abort_flag,
                         int lane) {
    using C = Cfg<D, R, NH>;
    constexpr int LPR = D / 8;         // lanes of a query row, 8 elements each
    constexpr int PASS = R * LPR / 32;
    const uint32_t sbase = smem_u32(smem);
    int units = 0;
    for (int k = 0;; ++k) {
        const int slot = k % kQN;
        if (!warp_wait(&b.uq_full[slot], (uint32_t)((k / kQN) & 1), abort_flag, p.status)) return;
        const Unit u = read_unit(uq + slot * kUnitInts);
        __syncwarp();
        if (lane == 0) bar_arrive(&b.uq_empty[slot]);
        if (u.r < 0) return;
        const int qb = units & 1;
        if (units >= 2 && !warp_wait(&b.q_empty[qb], (uint32_t)(((units >> 1) - 1) & 1), abort_flag, p.status)) return;
        ++units;
        const uint32_t q_at = sbase + C::OFF_Q + (uint32_t)(qb * C::QBYTES);
        int4* s_row = reinterpret_cast<int4*>(smem + C::OFF_ROW) + qb * R;
        if (lane < R) {
            const int row = u.row0 + min(lane % C::RH, u.nr - 1), tok = row / p.G;
            s_row[lane] = make_int4(0, max(last_key(p, u, row), -1),
                                    (u.q_start + tok) * p.H + (u.kvh * NH + lane / C::RH) * p.G + (row - tok * p.G), 0);
        }
        __syncwarp();
        // A row goes as it is to the place of its codes, the first half where hi will be, the second where lo will be, and
        // is taken from there: a rolled loop without loads' latency in it.  (Unrolled over registers, its first run waits
        // for instructions.)  A lane's row in pass i and its 8 elements; two heads that share operand rows go together.
        auto row_at = [&](int i) {
            const int x = (i * 32 + lane) / LPR;
            return C::WIDE ? (x & 1) * C::RH + (x >> 1) : x;
        };
        auto place = [&](int r, int half) {  // of a row's hi (0) or lo (1)
            return q_at + (uint32_t)(((C::WIDE ? 0 : r / C::RH * 2 * C::RH) + half * C::RH + r % C::RH) * C::W + (C::WIDE ? r / C::RH * D : 0));
        };
        const int part = lane % LPR;
#pragma unroll 1
        for (int i = 0; i < PASS; ++i) {
            const int r = row_at(i);
            const bool there = r % C::RH < u.nr;
            copy16(place(r, part / (LPR / 2)) + (uint32_t)(part % (LPR / 2) * 16),
                   p.q + (there ? (size_t)(unsigned)s_row[r].z * D + part * 8 : 0), there);
        }
        copies_wait();
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < PASS; ++i) {
            const int r = row_at(i);
            uint32_t word[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3])
                         : "r"(place(r, part / (LPR / 2)) + (uint32_t)(part % (LPR / 2) * 16)) : "memory");
            __syncwarp();  // the pass's rows have been read
            float f[8], top = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                f[c] = c & 1 ? bf16hi_to_f32(word[c / 2]) : bf16lo_to_f32(word[c / 2]);
                const float a = fabsf(f[c]);
                top = fmaxf(top, a < INFINITY ? a : 0.f);
            }
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float qs = scale_for(top), inv = 1.f / qs;
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                // an infinity or NaN: x - x makes a NaN of it
                const float a = fmaf(f[c], inv, f[c] - f[c]), d = fmaf(f[c + 1], inv, f[c + 1] - f[c + 1]);
                uint16_t e, e2;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e) : "f"(d), "f"(a));
                const uint32_t back = half2_of(e);
                const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&back));
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e2) : "f"((d - w.y) * 16.f), "f"((a - w.x) * 16.f));
                hi[c / 4] = c & 2 ? hi[c / 4] | (uint32_t)e << 16 : (uint32_t)e;
                lo[c / 4] = c & 2 ? lo[c / 4] | (uint32_t)e2 << 16 : (uint32_t)e2;
            }
            // a head's rows: hi, lo; its operand is a tile of its own, or its half of the rows of the common one
            const int byte = lane % LPR * 8 + (C::WIDE ? r / C::RH * D : 0), head = C::WIDE ? 0 : r / C::RH;
            auto at = [&](int row) {
                const int chunk = (byte >> 4) ^ (C::W == 128 ? row & 7 : (row >> 1) & 3);
                return q_at + (uint32_t)((head * 2 * C::RH + row) * C::W + chunk * 16 + (byte & 15));
            };
            st_v2(at(r % C::RH), hi[0], hi[1]);
            st_v2(at(C::RH + r % C::RH), lo[0], lo[1]);
            if (lane % LPR == 0) s_row[r].x = __float_as_int(qs * p.c_scale);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&b.q_full[qb]);
    }
}

// ---------------------------------------------------------------- scales of the steps' keys (one warp)

template <int D, int R, int NH>
__device__ void scale_role(const Paged8Params& p, uint8_t* smem, const Bars& b, volatile int* uq, volatile int* abort_flag,
                           int lane) {
    using C = Cfg<D, R, NH>;
    const int per_page = p.page_shift - p.block_shift;
    const int gshift = min(p.block_shift, 4);  // keys that share an entry of s_scale: 1 to 16
    const uint32_t at0 = smem_u32(smem + C::OFF_SC);
    uint32_t n = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int slot = k % kQN;
        if (!warp_wait(&b.uq_full[slot], (uint32_t)((k / kQN) & 1), abort_flag, p.status)) break;
        const Unit u = read_unit(uq + slot * kUnitInts);
        __syncwarp();
        if (lane == 0) bar_arrive(&b.uq_empty[slot]);
        if (u.r < 0) break;
#pragma unroll 1
        for (int s = 0; s < u.nt; s += C::SB, ++n) {
            const uint32_t buf = n % C::SCB;
            const int groups = (min(C::SB, u.nt - s) * 128) >> gshift;
            const long long key0 = (long long)(u.tile0 + s) * 128;
            // pages of the step (64 at most): x in lane x % 32, register x / 32
            const long long page0 = key0 >> p.page_shift;
            int id[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const long long page = page0 + i * 32 + lane, key = page << p.page_shift;
                id[i] = -1;
                if (key < key0 + C::SB * 128 && key < u.kv_len) id[i] = __ldg(p.block_table + (size_t)u.r * p.max_pages + page);
            }
            if (n >= C::SCB && !(ok = warp_wait(&b.sc_empty[buf], (n / C::SCB - 1u) & 1u, abort_flag, p.status))) break;
#pragma unroll 1
            for (int x0 = 0; x0 < NH * groups; x0 += 32) {
                const int x = x0 + lane, head = NH == 2 && x >= groups, g = x - head * groups;
                const long long key = key0 + ((long long)g << gshift);
                const int page = (int)((key >> p.page_shift) - page0);
                const int id0 = __shfl_sync(0xffffffffu, id[0], page & 31), id1 = __shfl_sync(0xffffffffu, id[1], page & 31);
                const int of = page < 32 ? id0 : id1;
                const bool there = key < u.kv_len && of >= 0 && of < p.num_pages;
                const size_t at = there ? (((size_t)(unsigned)of * p.H_kv + u.kvh * NH + head) << per_page) +
                                              (((int)key & ((1 << p.page_shift) - 1)) >> p.block_shift)
                                        : 0;
                const uint32_t to = at0 + (uint32_t)(((buf * NH + head) * C::SB * 128 + g) * 8);
                if (x < NH * groups) {
                    copy4(to, p.k_scale + at, there);
                    copy4(to + 4, p.v_scale + at, there);
                }
            }
            copies_arrive(&b.sc_full[buf]);
        }
    }
    copies_wait();
}

// ---------------------------------------------------------------- softmax + epilogue (eight warps)

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Sums of eight values over the warp: lane i gets that of value 4 (i >> 4 & 1) + 2 (i >> 3 & 1) + (i >> 2 & 1).
__device__ __forceinline__ float warp_sum8(const float* v, int lane) {
    float a[4], c[2], x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        c[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 8);
    }
    x = (lane & 4 ? c[1] : c[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? c[0] : c[1], 4);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x + __shfl_xor_sync(0xffffffffu, x, 1);
}

// A step's 32 / R x R / 8 blocks of 128 keys x 8 rows go to two groups of four warps: two blocks to a thread, whose 16
// scores stay in registers.  Few instructions, each used often: the two blocks are two turns of a rolled loop that shifts
// their scores along.  Warps wait for instructions before they wait for data, once the loop does not fit the cache.
template <int D, int R, int NH>
__device__ void softmax_role(const Paged8Params& p, uint8_t* smem, const Bars& b, volatile int* uq, volatile int* abort_flag,
                             uint32_t tmem, int warp8, int wq, int lane) {
    using C = Cfg<D, R, NH>;
    constexpr int SB = C::SB, RH = C::RH, PH = C::PH;
    constexpr int SETS = R == 32 ? 2 : 1;        // sets of 8 rows that a thread sees
    const int grp = warp8 >> 2;
    const int tid = wq * 32 + lane;              // key within a tile, TMEM lane
    const int gtid = warp8 * 32 + lane;          // 0 .. 255
    // block k of this thread: tile tile_of(k), rows row_of(k) ..
    auto tile_of = [&](int k) { return R == 8 ? grp + 2 * k : R == 16 ? k : 0; };
    auto row_of = [&](int k) { return R == 8 ? 0 : R == 16 ? 8 * grp : 8 * grp + 16 * k; };
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off, tO = tmem + lane_off + C::TM_O;
    // this key's row of P, or its byte of row 0 before the swizzle
    const uint32_t p_at = smem_u32(smem + C::OFF_P) + (uint32_t)(C::KEYS ? tid * C::WP : tid);
    const float2* s_scale = reinterpret_cast<const float2*>(smem + C::OFF_SC);
    float2* s_stat = reinterpret_cast<float2*>(smem + C::OFF_STAT);
    float2* s_par = reinterpret_cast<float2*>(smem + C::OFF_PAR);
    float2* s_alpha = reinterpret_cast<float2*>(smem + C::OFF_ALPHA);
    float2* s_exch = reinterpret_cast<float2*>(smem + C::OFF_EXCH);
    float* s_sum = reinterpret_cast<float*>(smem + C::OFF_SUM);
    int* s_nan = reinterpret_cast<int*>(smem + C::OFF_NAN);
    const int gshift = min(p.block_shift, 4);
    uint32_t n = 0;  // step
    // A failed wait leaves this warp on the common path, so that no barrier lacks a warp; all leave together where
    // they next agree on it.
    bool fail = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!fail) fail = !warp_wait(bar, parity, abort_flag, p.status);
    };

    auto wait_products = [&](uint32_t step) { wait(&b.o_full[step & 1u], (step >> 1) & 1u); };

    for (int k = 0;; ++k) {
        const int slot = k % kQN, qb = k & 1;
        wait(&b.uq_full[slot], (uint32_t)((k / kQN) & 1));
        if (softmax_any(fail)) return;
        const Unit u = read_unit(uq + slot * kUnitInts);
        __syncwarp();
        if (lane == 0) bar_arrive(&b.uq_empty[slot]);
        if (u.r < 0) return;
        wait(&b.q_full[qb], (uint32_t)((k >> 1) & 1));
        const int4* s_row = reinterpret_cast<const int4*>(smem + C::OFF_ROW) + qb * R;
        const int first_last = last_key(p, u, u.row0);  // the last key that the unit's first row sees

        for (int s = 0; s < u.nt; s += SB, ++n) {
            const int nt = min(SB, u.nt - s);
            const uint32_t buf = n & 1u, sc_buf = n % C::SCB;
            const int key0 = (u.tile0 + s) * 128;  // below kv_len
            const bool diagonal = first_last < u.kv_len - 1 && (long long)key0 + nt * 128 - 1 > first_last;
            wait(&b.sc_full[sc_buf], (n / C::SCB) & 1u);
            wait(&b.s_full[buf], (n >> 1) & 1u);
            tc_fence_after();
            // ---- scores in log2 units, -inf where masked; the rows' maxima over the warp
            float e0[8], e1[8], vk0 = 0.f, vk1 = 0.f;  // of the thread's two blocks; their values' scales
            bool grew = s == 0;
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
                const int t = tile_of(j), rb = row_of(j);
#pragma unroll
                for (int i = 0; i < 8; ++i) e0[i] = e1[i];
                vk0 = vk1;
                if (t < nt && rb % RH < u.nr) {
                    uint32_t x[16];
                    const uint32_t col = buf * 64u + (uint32_t)(t * 2 * R + rb / RH * 2 * RH + rb % RH);
                    tmem_ld8(tS + col, x);
                    tmem_ld8(tS + col + (uint32_t)RH, x + 8);
                    const float2 sc = s_scale[(sc_buf * NH + rb / RH) * SB * 128 + ((t * 128 + tid) >> gshift)];
                    // the rows of keys past the request's end are zeros
                    const float mask = (unsigned)key0 + (unsigned)(t * 128 + tid) < (unsigned)u.kv_len ? 0.f : -INFINITY;
                    vk1 = fminf(sc.y, kHuge);  // (a masked key's may be an infinity or NaN)
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = __int_as_float(s_row[rb + i].x) * sc.x;
                    tmem_ld_wait();
                    reg_after_wait<16>(x);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        e1[i] = fmaf(fmaf(__uint_as_float(x[8 + i]), 0.0625f, __uint_as_float(x[i])), f[i], mask);
                    if (diagonal) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if ((long long)key0 + t * 128 + tid > s_row[rb + i].y) e1[i] = -INFINITY;
                    }
                } else {
                    vk1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) e1[i] = -INFINITY;
                }
                if (SETS == 2 || j == 1) {
                    float a = 0.f, c = 0.f;
                    const float lv0 = lg2(vk0), lv1 = lg2(vk1);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float top = warp_max(SETS == 2 ? e1[i] : fmaxf(e0[i], e1[i]));
                        const float top_v = warp_max(SETS == 2 ? e1[i] + lv1 : fmaxf(e0[i] + lv0, e1[i] + lv1));
                        if (lane == i) {
                            a = top;
                            c = top_v;
                        }
                    }
                    if (lane < 8) {
                        const float2 stat = s_stat[rb + lane];
                        grew = grew || a > stat.x + kTau || c > stat.y + kTau;
                        s_exch[warp8 * R + rb + lane] = make_float2(a, c);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&b.sc_empty[sc_buf]);
            if (softmax_any(grew || fail)) {
                if (softmax_any(fail)) return;
                if (gtid < R) {
                    const float2 old = s == 0 ? make_float2(-INFINITY, -INFINITY) : s_stat[gtid];
                    float2 now = old;
                    // the warps that saw the row: of both groups, or of the one that has its eight
                    const int from = R == 8 ? 0 : (gtid >> 3 & 1) * 4;
#pragma unroll
                    for (int w = 0; w < (R == 8 ? 8 : 4); ++w) {
                        const float2 x = s_exch[(from + w) * R + gtid];
                        now.x = fmaxf(now.x, x.x);
                        now.y = fmaxf(now.y, x.y);
                    }
                    // (scales of V are 2^-126 at least: P of a row whose own are all below 2^-kVMin is smaller than it might be, by
                    // up to 2^14)
                    now.y = fmaxf(now.y, now.x - kVMin);
                    const float m = now.x == -INFINITY ? 0.f : now.x;
                    s_stat[gtid] = now;
                    s_par[gtid] = make_float2(m, now.y == -INFINITY ? 0.f : ex2(m - now.y + kBase));
                    s_alpha[gtid] = make_float2(old.x == -INFINITY ? 1.f : ex2(old.x - now.x),
                                                old.y == -INFINITY ? 1.f : ex2(old.y - now.y));
                }
                softmax_sync();
                if (s > 0) {
                    wait_products(n - 1u);
                    tc_fence_after();
                    if (lane < R) s_sum[warp8 * R + lane] *= s_alpha[lane].x;
                    __syncwarp();
#pragma unroll 1
                    for (int c = 8 * grp; c < R / PH * C::NPV; c += 16) {
                        uint32_t x[8];
                        const uint32_t col = tO + (uint32_t)c;
                        const int r = c / C::NPV * PH + c % PH;
                        tmem_ld8(col, x);
                        tmem_ld_wait();
                        reg_after_wait<8>(x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * s_alpha[r + i].y);
                        tmem_st8(col, x);
                    }
                    tmem_st_wait();
                }
            }
            // the products that read this buffer of P before (those of the unit before are complete)
            if (s >= C::PBUF * SB) wait_products(n - C::PBUF);
            // ---- probabilities
            float l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = 0.f;
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
                const int t = tile_of(j), rb = row_of(j);
                if (t < nt && rb % RH < u.nr) {
                    uint32_t h[4], hi[4], mid[4], lo[4], end[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {  // two rows share the conversions
                        const float2 par0 = s_par[rb + i], par1 = s_par[rb + i + 1];
                        const float p0 = ex2(e0[i] - par0.x), p1 = ex2(e0[i + 1] - par1.x);
                        l[i] += p0;
                        l[i + 1] += p1;
                        // (the factor first: times the scale it may overflow, where the scales of a row are far apart)
                        h[i / 2] = pack_half(p0 * par0.y * vk0, p1 * par1.y * vk0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) hi[i] = e5m2_of(h[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = h2_sub(h[i], half2_of_e5m2(hi[i]));
#pragma unroll
                    for (int i = 0; i < 4; ++i) mid[i] = e5m2_of(h[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = h2_mul64(h2_sub(h[i], half2_of_e5m2(mid[i])));
#pragma unroll
                    for (int i = 0; i < 4; ++i) lo[i] = e5m2_of(h[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) end[i] = e5m2_of(h2_sub(h[i], half2_of_e5m2(lo[i])));
                    const uint32_t tile = p_at + (uint32_t)((((C::PBUF == 2 ? buf : 0u) * SB + t) * C::TPK + rb / PH) * C::PTILE);
                    if (C::KEYS) {
                        const uint32_t turn = (uint32_t)(C::WP == 128 ? tid & 7 : (tid >> 1) & 3) << 4;
                        auto put = [&](int col, const uint32_t* x) {
                            st_v2(tile + ((uint32_t)col ^ turn), x[0] | x[1] << 16, x[2] | x[3] << 16);
                        };
                        put(rb % PH, hi);
                        put(PH + rb % PH, lo);
                        put(2 * PH + rb % PH, mid);
                        put(3 * PH + rb % PH, end);
                    } else {
                        const uint32_t at = tile + (uint32_t)(rb % PH * 128);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a0 = (at ^ (uint32_t)(2 * i << 4)) + (uint32_t)(2 * i * 128);
                            const uint32_t a1 = (at ^ (uint32_t)((2 * i + 1) << 4)) + (uint32_t)((2 * i + 1) * 128);
                            st_u8(a0, hi[i]);
                            st_u8(a1, hi[i] >> 8);
                            st_u8(a0 + PH * 128, lo[i]);
                            st_u8(a1 + PH * 128, lo[i] >> 8);
                            st_u8(a0 + 2 * PH * 128, mid[i]);
                            st_u8(a1 + 2 * PH * 128, mid[i] >> 8);
                            st_u8(a0 + 3 * PH * 128, end[i]);
                            st_u8(a1 + 3 * PH * 128, end[i] >> 8);
                        }
                    }
                }
                if (SETS == 2 || j == 1) {  // the rows' sums, one lane each
                    const float x = warp_sum8(l, lane);
                    float* sum = s_sum + warp8 * R + rb + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
                    if ((lane & 3) == 0) *sum = x + (s > 0 ? *sum : 0.f);
                    if (SETS == 2) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) l[i] = 0.f;
                    }
                }
                vk0 = vk1;
#pragma unroll
                for (int i = 0; i < 8; ++i) e0[i] = e1[i];
            }
            fence_async_smem();
            tc_fence_before();
            bar_arrive(&b.p_full[buf]);
        }

        // ---- the unit's end: O by channel, every other row by each group
        softmax_sync();  // every warp's sums
        if (u.nt > 0) wait_products(n - 1u);
        const int lane_chan = C::W == 128 ? tid : wq * 16 + (lane & 15), chan = lane_chan % D;
        const bool mine = !fail && (C::W == 128 || lane < 16);
        tc_fence_after();
#pragma unroll 1
        for (int x = grp; x < u.nr * C::TPK; x += 2) {  // (a wide tile's heads: half of the channels each)
            const int head = C::WIDE ? tid / D : x >= u.nr, y = C::WIDE ? x : x - head * u.nr, r = head * RH + y;
            float v = 0.f, m = 0.f, sum = 0.f;
            if (u.nt > 0) {
                uint32_t x[4] = {0u, 0u, 0u, 0u};
                const uint32_t col = tO + (uint32_t)(r / PH * C::NPV + r % PH);
                tmem_ld1(col, x);
                tmem_ld1(col + (uint32_t)PH, x + 1);
                if (!C::FOLD) {
                    tmem_ld1(col + (uint32_t)(2 * PH), x + 2);
                    tmem_ld1(col + (uint32_t)(3 * PH), x + 3);
                }
                const int from = R == 8 ? 0 : (r >> 3 & 1) * 4;
#pragma unroll
                for (int w = 0; w < (R == 8 ? 8 : 4); ++w) sum += s_sum[(from + w) * R + r];
                const float2 st = s_stat[r];
                m = st.x == -INFINITY ? 0.f : st.x;
                const float f = st.y == -INFINITY ? 0.f : ex2(st.y - kBase - m);
                tmem_ld_wait();
                reg_after_wait<4>(x);
                v = fmaf(__uint_as_float(x[1]) + __uint_as_float(x[3]), 0x1p-6f, __uint_as_float(x[0]) + __uint_as_float(x[2])) * f;
                if (y >= s_nan[head * D + chan]) v = __int_as_float(0x7fffffff);
            }
            if (u.slot < 0) {
                const size_t out = (size_t)(unsigned)s_row[r].z;
                const float o = sum == 0.f ? 0.f : v * (1.f / sum);
                if (mine) p.o[out * D + chan] = (uint16_t)pack_bf16(o, o);
                if (!fail && chan == y && p.lse != nullptr) p.lse[out] = sum == 0.f ? -INFINITY : (m + lg2(sum)) * kLn2;
            } else {
                const size_t rec = (size_t)u.slot * R + r;
                if (mine) p.part_o[rec * D + chan] = v;
                if (!fail && chan == y) *reinterpret_cast<float2*>(p.part_ml + rec * 2) = make_float2(sum == 0.f ? -INFINITY : m, sum);
            }
        }
        tc_fence_before();
        softmax_sync();  // s_stat, s_sum, s_nan and the rows have been read
        if (gtid < NH * D) s_nan[gtid] = 0x7fffffff;
        if (lane == 0) bar_arrive(&b.q_empty[qb]);
    }
}

// ---------------------------------------------------------------- kernels

template <int D, int R, int NH>
__global__ void __launch_bounds__(kThreads8, 2) paged8_kernel(const __grid_constant__ Paged8Params p) {
    using C = Cfg<D, R, NH>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    Bars b;
    b.kv_full = bars;
    b.kv_empty = b.kv_full + C::NST;
    b.q_full = b.kv_empty + C::NST;
    b.q_empty = b.q_full + 2;
    b.sc_full = b.q_empty + 2;
    b.sc_empty = b.sc_full + 2;
    b.s_full = b.sc_empty + 2;
    b.p_full = b.s_full + 2;
    b.o_full = b.p_full + 2;
    b.done = b.o_full + 2;
    b.uq_full = b.done + 1;
    b.uq_empty = b.uq_full + kQN;
    volatile int* uq = reinterpret_cast<volatile int*>(smem + C::OFF_UQ);
    int* misc = reinterpret_cast<int*>(smem + C::OFF_MISC);  // tmem, abort, skip, r0; then the words below
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc);
    volatile int* abort_flag = misc + 1;
    long long* wide = reinterpret_cast<long long*>(misc + 4);  // [0] start of request r0, [1 .. 12] sums of the warps

    griddep_launch_dependents();  // the merge may be scheduled; it waits for this grid
    // ---- the cut: tiles of all requests, in order, in shares of equal size.  Warp 0, which needs it, makes it for up to 64
    // requests, without a barrier; all threads do for more.
    const bool few = p.B <= 64, cutter = !few || warp == 0;
    const int per = few ? (p.B + 31) >> 5 : (p.B + kThreads8 - 1) / kThreads8;
    const int ra = min(p.B, tid * per), rb = min(p.B, ra + per);
    Extent e{}, e2{};
    if (cutter) {  // the loads are under way during the set-up
        e = extent(p, min(ra, p.B - 1));
        if (few) e2 = extent(p, min(ra + 1, p.B - 1));
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, C::TM_COLS);
        tmem_relinquish();
    }
    if (tid >= 64 && tid - 64 < C::N_BARS) {
        uint64_t* x = bars + tid - 64;
        int count = 1;
        if (x >= b.uq_empty) count = 11;
        else if (x >= b.o_full) count = x < b.done ? 2 : 1;
        else if (x >= b.p_full) count = 256;
        else if (x >= b.s_full) count = 1;
        else if (x >= b.sc_empty) count = 8;
        else if (x >= b.sc_full) count = 32;
        else if (x >= b.q_empty) count = 9;
        bar_init(x, count);
        bar_init_fence();
    }
    if (tid == kThreads8 - 1) {
        *abort_flag = 0;
        misc[2] = timeout_recorded(p.status) ? 1 : 0;  // an earlier launch gave up
    }
    for (int i = kThreads8 - 1 - tid; i < NH * D; i += kThreads8) reinterpret_cast<int*>(smem + C::OFF_NAN)[i] = 0x7fffffff;
    long long share = 0, w0 = 0, w1 = 0;
    if (cutter) {
        long long sum = 0, total;
        bool bad = false;
#pragma unroll 1
        for (int r = ra; r < rb; ++r) {
            const Extent x = r == ra ? e : few ? e2 : extent(p, r);
            bad |= x.bad;
            sum += work_of<C::RH>(p, x);
        }
        if (bad && blockIdx.x == 0) atomicOr(p.status, 1u << kStatusDeviceData);
        long long before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        total = __shfl_sync(0xffffffffu, before, 31);
        before -= sum;
        if (!few) {
            if (lane == 31) wide[1 + warp] = total;
            __syncthreads();
            total = 0;
#pragma unroll 1
            for (int w = 0; w < kThreads8 / 32; ++w) {
                if (w < warp) before += wide[1 + w];
                total += wide[1 + w];
            }
        }
        share = total < 0x7fff0000LL ? max((unsigned)kMinShare, ((unsigned)total + gridDim.x - 1) / gridDim.x)
                                     : long_quotient(total + gridDim.x - 1, gridDim.x);
        w0 = (long long)blockIdx.x * share;
        w1 = min(total, w0 + share);
        if (w0 >= before && w0 < before + sum) {  // this thread's requests hold the CTA's first tile
            long long at = before;
#pragma unroll 1
            for (int r = ra; r < rb; ++r) {
                const Extent x = r == ra ? e : few ? e2 : extent(p, r);
                const long long work = work_of<C::RH>(p, x);
                if (w0 < at + work) {
                    misc[3] = r;
                    wide[0] = at;
                    int* first = misc + kMiscFirst;
                    first[0] = x.q_start;
                    first[1] = x.q_len;
                    first[2] = x.kv_len;
                    break;
                }
                at += work;
            }
        }
        if (tid == 0) p.cuts[2 * blockIdx.x].x = -1;  // the producer (this thread) may put a cut in its place
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    if (misc[2] == 0) {
        if (warp >= 2 && warp < 10) {
            softmax_role<D, R, NH>(p, smem, b, uq, abort_flag, tmem, warp - 2, warp & 3, lane);
        } else if (warp == 0) {
            const bool any = w0 < w1;  // otherwise its first unit is the end
            const int* first = misc + kMiscFirst;
            producer_role<D, R, NH>(p, smem, b, uq, abort_flag, lane, any ? misc[3] : 0, w0, w1, any ? wide[0] : 0,
                                    Extent{first[0], first[1], first[2], false}, share);
        } else if (warp == 10) {
            query_role<D, R, NH>(p, smem, b, uq, abort_flag, lane);
        } else if (warp == 11) {
            scale_role<D, R, NH>(p, smem, b, uq, abort_flag, lane);
        } else {
            mma_role<D, R, NH>(p, smem, b, uq, abort_flag, tmem, lane);
            __syncwarp();
            if (lane == 0) {
                tc_commit(b.done);  // every issued MMA finishes before tensor memory is released
                drain_wait(b.done, 0, p.status);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TM_COLS);
    }
}

// The units that were cut, gridDim.y CTAs to each, which take two of its rows at a time: a row's pieces to kMergeWarps
// warps in turn,
//   m = max m_i,  l = sum l_i 2^(m_i - m),  O = sum 2^(m_i - m) O_i / l.
// The pieces are one unit's last of CTA c0 and first of the CTAs up to c1.  Their (m, l) and O are asked for at once.  (More
// CTAs to a unit cost more, since most have nothing to do, than they save: 32 thousand keys of one request 21.9 us with 2,
// 22.4 with 4; with 32 rows 58 and 55.)
constexpr int kMergeWarps = 4;
constexpr int kMergeRows = 2;   // of a CTA
template <int D>
__global__ void __launch_bounds__(kMergeRows * kMergeWarps * 32) paged8_merge_kernel(const __grid_constant__ Paged8Params p) {
    constexpr int PER = D / 32;
    using Vec = typename std::conditional<PER == 4, float4, float2>::type;
    __shared__ float s_o[kMergeRows][kMergeWarps][D], s_ml[kMergeRows][kMergeWarps][2];
    const int lane = threadIdx.x & 31, c0 = blockIdx.x;
    const int sub = threadIdx.x / (kMergeWarps * 32), tid = threadIdx.x % (kMergeWarps * 32), warp = tid >> 5;
    griddep_wait();
    const int4 cut = __ldcg(p.cuts + 2 * c0), unit = __ldcg(p.cuts + 2 * c0 + 1);
    if (timeout_recorded(p.status) || cut.x < 0) return;
    for (int x0 = blockIdx.y * kMergeRows; x0 < cut.z * p.NH; x0 += gridDim.y * kMergeRows) {
        const int x = min(x0 + sub, cut.z * p.NH - 1);  // (the last row twice, if they are odd)
        const int head = x / cut.z, y = x - head * cut.z, r = head * p.RH + y;
        float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
        for (int c = c0 + warp; c <= cut.x; c += 4 * kMergeWarps) {  // four pieces in flight
            Vec v[4];
            float2 ml[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int ck = c + k * kMergeWarps;
                ml[k] = make_float2(-INFINITY, 0.f);
                if (ck <= cut.x) {
                    const size_t rec = (size_t)(ck == c0 ? cut.y : 2 * ck) * p.R + r;
                    ml[k] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + rec);
                    v[k] = __ldcg(reinterpret_cast<const Vec*>(p.part_o + rec * D) + lane);
                }
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
            const float old = m == -INFINITY ? 0.f : ex2(m - top);
            m = top;
            l *= old;
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] *= old;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (ml[k].x == -INFINITY) continue;  // no such piece, or one without a visible key: it has no O
                const float w = ex2(ml[k].x - m);
                const float* f = reinterpret_cast<const float*>(&v[k]);
                l = fmaf(ml[k].y, w, l);
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[i] = fmaf(f[i], w, acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) s_o[sub][warp][lane * PER + i] = acc[i];
        if (lane == 0) {
            s_ml[sub][warp][0] = m;
            s_ml[sub][warp][1] = l;
        }
        __syncthreads();
        if (tid < D / 2) {
            float top = -INFINITY, sum = 0.f, f2[2] = {0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, s_ml[sub][w][0]);
#pragma unroll
            for (int w = 0; w < kMergeWarps; ++w) {
                const float f = s_ml[sub][w][0] == -INFINITY ? 0.f : ex2(s_ml[sub][w][0] - top);
                sum = fmaf(s_ml[sub][w][1], f, sum);
                f2[0] = fmaf(s_o[sub][w][2 * tid], f, f2[0]);
                f2[1] = fmaf(s_o[sub][w][2 * tid + 1], f, f2[1]);
            }
            const int at = unit.y + y, tok = at / p.G;
            const size_t row = (size_t)(unit.x + tok) * p.H + (cut.w * p.NH + head) * p.G + (at - tok * p.G);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            reinterpret_cast<uint32_t*>(p.o + row * D)[tid] = pack_bf16(f2[0] * inv, f2[1] * inv);
            if (tid == 0 && p.lse != nullptr) p.lse[row] = sum == 0.f ? -INFINITY : (top + lg2(sum)) * kLn2;
        }
        __syncthreads();
    }
}

template <int D, int R, int NH>
cudaError_t launch(const Paged8Params& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> opted{0};
    cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(paged8_kernel<D, R, NH>), Cfg<D, R, NH>::SMEM_BYTES, opted);
    if (e != cudaSuccess) return e;
    paged8_kernel<D, R, NH><<<p.n_ctas, kThreads8, Cfg<D, R, NH>::SMEM_BYTES, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.n_ctas, p.R > 16 ? 4u : 2u);
    cfg.blockDim = dim3(kMergeRows * kMergeWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged8_merge_kernel<D>, p);
}

}  // namespace

// Two KV heads to a unit halve the number of units, and read rows of the cache that lie side by side together: 128 bytes
// for two heads of d = 64, where rows of 64 bytes come at 3.2 TB/s, those of 128 at 6.2; tiles in turn with d = 128.  Single
// heads and pairs, d = 128: 33 requests of 0 to 4096 keys, 16 heads 64 and 56 us; 64 of 256, 8 heads 18.0 and 16.4, of 512 to
// 8192 98 and 100 (on a GPU with slower memory 113 and 109); 4 of 200 to 262 thousand 298 and 289 (343 and 313).  d = 64: 64
// of 256 17.1 and 12.9, 8 of 32 thousand 71 and 54.  One unit takes longer, though: what does not fill the CTAs, or leaves
// each a few tiles only, is faster by single heads (one request of 1024 keys 11.6 and 14.9 us with d = 128, 11.3 and 12.2
// with d = 64; of 32 thousand 20 and 25, 19 and 20; of 131 thousand 50 and 55, 41 and 39).  The lengths are not known here,
// but how long they can be.  More rows than 16 to a head share their tiles well enough with d = 128.
Paged8Plan paged8_plan(int B, int max_q_len, int H, int H_kv, int d, int page_size, int max_pages) {
    Paged8Plan pl;
    const long long rows = (long long)max_q_len * (H / H_kv);
    const long long units = (long long)B * H_kv, tiles = units * (((long long)page_size * max_pages + 127) / 128);
    const bool large = units > kPaged8Ctas || tiles > kPaged8Ctas * (d == 128 ? 32LL : 8LL);
    pl.NH = H_kv % 2 == 0 && large && (d == 64 || rows <= 16) ? 2 : 1;
    pl.R = rows <= 8 ? 8 * pl.NH : rows * pl.NH <= 16 ? 16 : 32;
    pl.part_ml = kPaged8Ctas * 2 * sizeof(int4);
    pl.part_o = pl.part_ml + (size_t)2 * kPaged8Ctas * pl.R * 2 * sizeof(float);
    pl.bytes = pl.part_o + (size_t)2 * kPaged8Ctas * pl.R * d * sizeof(float);
    return pl;
}

cudaError_t launch_paged8(int d, const Paged8Params& p, cudaStream_t stream) {
    if (d == 128) {
        if (p.NH == 2) return p.R == 16 ? launch<128, 16, 2>(p, stream) : launch<128, 32, 2>(p, stream);
        return p.R == 8 ? launch<128, 8, 1>(p, stream) : p.R == 16 ? launch<128, 16, 1>(p, stream) : launch<128, 32, 1>(p, stream);
    }
    if (p.NH == 2) return p.R == 16 ? launch<64, 16, 2>(p, stream) : launch<64, 32, 2>(p, stream);
    return p.R == 8 ? launch<64, 8, 1>(p, stream) : p.R == 16 ? launch<64, 16, 1>(p, stream) : launch<64, 32, 1>(p, stream);
}

}  // namespace attn
