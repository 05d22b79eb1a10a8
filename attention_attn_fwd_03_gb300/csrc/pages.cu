// pages.cu -- the bookkeeping of a paged cache on the GPU: page plans (table
// rows, slots and positions from request lengths) and page sketches (8-bit
// channel extremes of each page's keys, which page selection scores).
#include <cooperative_groups.h>

#include <cmath>
#include <cstring>

#include "attn_kv.h"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------- page plan
//
// Two prefix sums over the requests, new tokens and new pages, place
// everything: token t belongs to the last request r with cu[r] <= t, and the
// i-th new page of request r is the (before[r] + i)-th taken from the stack.
//
// Every CTA computes both sums for itself into shared memory (a few words per
// request, read through L2), then the tokens are dealt to all threads, each
// finding its request by bisection in shared memory.  A token that starts a
// page enters it in the table, so table writes are as balanced as the tokens.
// A call whose outputs replace inputs runs in one cluster: its barrier lets
// every CTA read the lengths and the free count before CTA 0 writes seq_lens
// and free_left; any other call uses as many CTAs as it has tokens for.
// Latency-bound: the largest calls write 8 bytes per token, the smallest a few
// hundred bytes.

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxB = 16384;
constexpr int kPlanMaxCluster = 8;

struct PlanParams {
    const int32_t* ctx;
    const int32_t* fresh;  // new tokens per request, or nullptr: one each
    int32_t* table;
    const int32_t* free_pages;
    const int32_t* free_count;
    int32_t *cu, *seq_lens, *positions, *slots, *free_left;
    unsigned* status;
    int B, total_q, page_size, max_pages, num_pages, n_free;
    int in_place;  // an output replaces an input: the grid is one cluster
};

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanParams p) {
    extern __shared__ int s_plan[];
    int* s_cu = s_plan;              // [B + 1], clamped to INT_MAX
    int* s_ctx = s_cu + p.B + 1;     // [B]
    int* s_before = s_ctx + p.B;     // [B]
    __shared__ long long s_tok[32], s_pg[32];
    __shared__ int s_count;
    __shared__ long long s_demand;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)blockIdx.x, n_ctas = (int)gridDim.x;
    const int ps = p.page_size;
    const long long cap = (long long)p.max_pages * ps;
    bool bad = false;

    if (tid == 0) {
        const int c = *p.free_count;
        s_count = c < 0 ? 0 : c > p.n_free ? p.n_free : c;
        bad = s_count != c;
    }
    // each thread sums a run of consecutive requests
    const int run = (p.B + kPlanThreads - 1) / kPlanThreads;
    const int r0 = tid * run, r1 = min(p.B, r0 + run);
    auto lengths = [&](int r, long long& ctx, long long& len) {
        ctx = p.ctx[r];
        long long add = p.fresh != nullptr ? p.fresh[r] : 1;
        if (ctx < 0 || ctx > cap) {
            bad = true;
            ctx = ctx < 0 ? 0 : cap;
        }
        if (add < 0 || ctx + add > cap) {
            bad = true;
            add = add < 0 ? 0 : cap - ctx;
        }
        len = ctx + add;
    };
    auto pages = [&](long long n) { return (n + ps - 1) / ps; };
    long long tok = 0, pg = 0;
    for (int r = r0; r < r1; ++r) {
        long long ctx, len;
        lengths(r, ctx, len);
        tok += len - ctx;
        pg += pages(len) - pages(ctx);
    }
    long long it = tok, ip = pg;  // inclusive sums over the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ip, o);
        if (lane >= o) {
            it += a;
            ip += b;
        }
    }
    if (lane == 31) {
        s_tok[warp] = it;
        s_pg[warp] = ip;
    }
    __syncthreads();
    if (warp == 0) {
        long long a = s_tok[lane], b = s_pg[lane];
        const long long a0 = a, b0 = b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) {
                a += x;
                b += y;
            }
        }
        s_tok[lane] = a - a0;
        s_pg[lane] = b - b0;
        if (lane == 31) s_demand = b;
    }
    __syncthreads();
    tok = s_tok[warp] + it - tok;
    pg = s_pg[warp] + ip - pg;
    auto clip = [](long long x) { return (int)(x < 0x7fffffffLL ? x : 0x7fffffffLL); };
    for (int r = r0; r < r1; ++r) {
        long long ctx, len;
        lengths(r, ctx, len);
        s_cu[r] = clip(tok);
        s_ctx[r] = (int)ctx;
        s_before[r] = clip(pg);
        tok += len - ctx;
        pg += pages(len) - pages(ctx);
        if (r == p.B - 1) {
            s_cu[p.B] = clip(tok);
            bad |= tok > p.total_q;
        }
    }
    if (p.in_place)  // all inputs that an output may replace have been read, by every CTA
        cg::this_cluster().sync();
    else
        __syncthreads();
    const int count = s_count;
    const int owned = s_cu[p.B];
    if (rank == 0) {
        for (int r = tid; r < p.B; r += kPlanThreads) p.seq_lens[r] = s_ctx[r] + (s_cu[r + 1] - s_cu[r]);
        for (int r = tid; r <= p.B; r += kPlanThreads) p.cu[r] = s_cu[r];
        if (tid == 0) *p.free_left = s_demand < count ? count - (int)s_demand : 0;
    }
    for (long long t64 = (long long)rank * kPlanThreads + tid; t64 < p.total_q; t64 += (long long)n_ctas * kPlanThreads) {
        const int t = (int)t64;
        int pos = 0, slot = -1;
        if (t < owned) {
            int lo = 0, hi = p.B - 1;  // the last request that starts at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_cu[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int ctx = s_ctx[lo];
            pos = ctx + (t - s_cu[lo]);
            const int pi = pos / ps, at = pos - pi * ps;
            const int held = (int)pages(ctx);
            int32_t* entry = p.table + (long long)lo * p.max_pages + pi;
            int id = -1;
            if (pi < held) {
                id = *entry;
            } else {
                const long long top = (long long)count - 1 - s_before[lo] - (pi - held);  // its place in the stack
                if (top >= 0) id = p.free_pages[top];
                if (id >= p.num_pages) id = -1;
                if (at == 0) *entry = id < 0 ? -1 : id;
            }
            if (id >= 0 && id < p.num_pages)
                slot = id * ps + at;
            else
                bad = true;
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
    if (bad) atomicOr(p.status, 1u << kStatusDeviceData);
}

// ---------------------------------------------------------------- page sketch
//
// Per page and KV head the channel extremes over the valid rows, scaled by
// their largest magnitude to 8 bits.  Extremes are exact in bf16 and do not
// depend on the order of the rows, and the codes are two fp32 roundings
// (divide, multiply) and one to an integer, so a page's sketch is a function
// of its keys alone.
//
// Bound by reading the keys once.  A CTA takes one page, or a block of its
// channels: a thread owns 8 channels and every RG-th row, 16 bytes per load;
// row groups combine through shared memory.  With many pages a CTA takes up to
// LANES = 128 pieces of a row (1024 channels), so that the page is read in
// whole rows, in batches of U = 12 per thread; with few pages (a decode
// step) LANES = 16 spreads a page over many CTAs and puts eight rows side by
// side, so that no thread waits for memory more than once or twice.
// The loads of a batch keep their order, but the extremes between them move up:
// for U = 8, 12 and 24 alike 47 registers are used, room for about eight loads in
// flight.  120 MB of keys, us with U = 8, 12, 24: 8 requests of 6144 - 8192 in
// 64-row pages 20.0, 19.4, 21.1; of 7168 19.2, 18.4, 17.5, in 16-row pages 24.0,
// 22.7, 29.4, in 128-row pages 25.5 each; 64 requests (940 MB) 137, 138, 143.
// Measured, 120 MB of keys: 19.4 us with 128 lanes (6.1 TB/s), 28 with 16; the
// last pages of 64 requests 6.4 and 3.9 us, of 256 9.5 and 8.0, of 512 12.5 and 14.7.
// Many small pages of narrow rows (up to 32 pieces a row, 512 a page) take a
// warp each: 2 KB pages of 16 x 8192 keys 23.5 -> 8.2 us, 8 KB pages 14.3 ->
// 8.8, while 16 KB ones are equal and 32 KB ones slower (9.0 -> 16.0).

constexpr int kSketchThreads = 128;
constexpr long long kManyPages = 512;
constexpr long long kNarrowPieces = 512;

struct SketchParams {
    const uint16_t* k;
    const int32_t* table;
    const int32_t* cu;
    const int32_t* seq_lens;
    int8_t* sketch;
    float* amp;
    unsigned* status;
    int B, max_q_len, H_kv, d, page_size, max_pages, num_pages;
    int per_req, col_blocks;  // pages per request and channel blocks that the grid covers
};

// Largest / smallest of two packed bf16 pairs; a NaN in either operand stays.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t code4(uint32_t a, uint32_t b, float amp) {
    uint32_t r = 0;
    const float x[4] = {bf16lo_to_f32(a), bf16hi_to_f32(a), bf16lo_to_f32(b), bf16hi_to_f32(b)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r |= ((uint32_t)__float2int_rn(__fmul_rn(__fdiv_rn(x[i], amp), 127.f)) & 0xffu) << (8 * i);
    return r;
}

// The page of unit u (request, its nth page from the first new key on); id -1: nothing to do.
struct SketchPage {
    int id, rows;
};
__device__ __forceinline__ SketchPage sketch_page(const SketchParams& p, long long u, bool report) {
    SketchPage g = {-1, 0};
    const int nth = (int)(u % p.per_req);
    const int r = (int)(u / p.per_req);
    const long long cap = (long long)p.max_pages * p.page_size;
    long long len = __ldg(p.seq_lens + r);
    long long fresh = p.max_q_len;
    bool bad = len < 0 || len > cap;
    len = len < 0 ? 0 : len > cap ? cap : len;
    if (p.cu != nullptr) {
        fresh = (long long)__ldg(p.cu + r + 1) - __ldg(p.cu + r);
        if (fresh < 0 || fresh > p.max_q_len || fresh > len) {
            bad = true;
            fresh = fresh < 0 ? 0 : fresh > p.max_q_len ? p.max_q_len : fresh;
        }
    }
    if (fresh > len) fresh = len;
    if (bad && report && nth == 0) atomicOr(p.status, 1u << kStatusDeviceData);
    if (fresh <= 0) return g;
    const long long page = (len - fresh) / p.page_size + nth;
    if (page * p.page_size >= len) return g;
    const int id = __ldg(p.table + (long long)r * p.max_pages + page);
    if (id < 0 || id >= p.num_pages) {
        if (report) atomicOr(p.status, 1u << kStatusDeviceData);
        return g;
    }
    g.id = id;
    g.rows = (int)min((long long)p.page_size, len - page * p.page_size);
    return g;
}

// Extremes of 8 channels of one thread, as packed bf16 pairs.
struct Extremes {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ Extremes() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = 0xff80ff80u;  // -inf
            lo[i] = 0x7f807f80u;  // +inf
        }
    }
    __device__ __forceinline__ void add(const uint4& a, const uint4& b) {  // a for the largest, b for the smallest
        hi[0] = max2(hi[0], a.x); lo[0] = min2(lo[0], b.x);
        hi[1] = max2(hi[1], a.y); lo[1] = min2(lo[1], b.y);
        hi[2] = max2(hi[2], a.z); lo[2] = min2(lo[2], b.z);
        hi[3] = max2(hi[3], a.w); lo[3] = min2(lo[3], b.w);
    }
};

// 16 bytes that nobody reads again; volatile, so that the loads are issued in the order of the rows.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Rows row0, row0 + step, .. below rows of one 16-byte column: with ONCE in batches of U loads while they
// are whole, the rest (else all) in eights.
template <int U, bool ONCE>
__device__ __forceinline__ void scan_rows(const uint4* src, int cols, int row0, int step, int rows, Extremes& e) {
    for (; ONCE && row0 + step * (U - 1) < rows; row0 += step * U) {
        uint4 x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] = ld_once(src + (long long)(row0 + i * step) * cols);
#pragma unroll
        for (int i = 0; i < U; ++i) e.add(x[i], x[i]);
    }
    constexpr int V = 8;
    for (; row0 < rows; row0 += step * V) {
        uint4 x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // past the last row the first one is read again: extremes do not change
            const int row = row0 + i * step < rows ? row0 + i * step : row0;
            x[i] = __ldg(src + (long long)row * cols);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) e.add(x[i], x[i]);
    }
}

// The largest magnitude over the head's channels, then the codes (whole warps call it; `write`: this thread's are stored).
__device__ __forceinline__ void store_sketch(const SketchParams& p, const Extremes& e, int id, int col, bool write) {
    // as bf16 bits without the sign: the order of the integers is that of the magnitudes, infinities and
    // NaN above every number
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = e.hi[i] & 0x7fff7fffu, b = e.lo[i] & 0x7fff7fffu;
        top = max(top, max(max(a & 0xffffu, a >> 16), max(b & 0xffffu, b >> 16)));
    }
    const int lanes_per_head = p.d / 8;  // 8 or 16 neighbouring lanes of a warp
    for (int o = 1; o < lanes_per_head; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!write) return;
    const bool finite = top < 0x7f80u;
    const float amp = finite ? __uint_as_float(top << 16) : INFINITY;
    uint2 ch = make_uint2(0u, 0u), cl = make_uint2(0u, 0u);
    if (finite && top != 0u) {
        ch = make_uint2(code4(e.hi[0], e.hi[1], amp), code4(e.hi[2], e.hi[3], amp));
        cl = make_uint2(code4(e.lo[0], e.lo[1], amp), code4(e.lo[2], e.lo[3], amp));
    }
    const int head = col / lanes_per_head, c0 = (col % lanes_per_head) * 8;
    const long long rec = (long long)id * p.H_kv + head;
    *reinterpret_cast<uint2*>(p.sketch + rec * (2 * p.d) + c0) = ch;
    *reinterpret_cast<uint2*>(p.sketch + rec * (2 * p.d) + p.d + c0) = cl;
    if (c0 == 0) p.amp[rec] = amp;
}

template <int LANES, int U>
__global__ void __launch_bounds__(kSketchThreads) page_sketch_kernel(const __grid_constant__ SketchParams p) {
    __shared__ uint4 s_hi[kSketchThreads], s_lo[kSketchThreads];
    const int cols = p.H_kv * p.d / 8;  // 16-byte pieces of a row
    const int L = cols < LANES ? cols : LANES;
    const int RG = kSketchThreads / L;
    const int cb = (int)(blockIdx.x % p.col_blocks);
    const SketchPage g = sketch_page(p, blockIdx.x / p.col_blocks, threadIdx.x == 0 && cb == 0);
    if (g.id < 0) return;
    const int lane = threadIdx.x % L, rg = threadIdx.x / L;
    const int col = cb * LANES + lane;
    Extremes e;
    if (rg < RG && col < cols)
        scan_rows<U, (LANES > 16)>(reinterpret_cast<const uint4*>(p.k) + (long long)g.id * p.page_size * cols + col, cols, rg, RG, g.rows, e);
    s_hi[threadIdx.x] = make_uint4(e.hi[0], e.hi[1], e.hi[2], e.hi[3]);
    s_lo[threadIdx.x] = make_uint4(e.lo[0], e.lo[1], e.lo[2], e.lo[3]);
    __syncthreads();
    if (rg == 0) {
        const int groups = RG < g.rows ? RG : g.rows;  // groups that read a row
        for (int x = 1; x < groups; ++x) e.add(s_hi[x * L + lane], s_lo[x * L + lane]);
    }
    store_sketch(p, e, g.id, col, rg == 0 && col < cols);
}

// Rows of at most 32 pieces: a warp takes a page, L lanes across a row, and
// combines its 32 / L row groups by shuffles.  L is the power of two at or
// above the pieces of a row.
template <int U>
__global__ void __launch_bounds__(kSketchThreads) page_sketch_warp_kernel(const __grid_constant__ SketchParams p) {
    const int lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.x * (kSketchThreads / 32) + (threadIdx.x >> 5);
    if (u >= (long long)p.B * p.per_req) return;
    const SketchPage g = sketch_page(p, u, lane == 0);
    if (g.id < 0) return;
    const int cols = p.H_kv * p.d / 8;
    int L = 8;
    while (L < cols) L <<= 1;
    const int RG = 32 / L, rg = lane / L, col = lane % L;
    Extremes e;
    if (col < cols)
        scan_rows<U, false>(reinterpret_cast<const uint4*>(p.k) + (long long)g.id * p.page_size * cols + col, cols, rg, RG, g.rows, e);
    for (int o = L; o < 32; o <<= 1) {
        uint4 a, b;
        a.x = __shfl_xor_sync(0xffffffffu, e.hi[0], o); b.x = __shfl_xor_sync(0xffffffffu, e.lo[0], o);
        a.y = __shfl_xor_sync(0xffffffffu, e.hi[1], o); b.y = __shfl_xor_sync(0xffffffffu, e.lo[1], o);
        a.z = __shfl_xor_sync(0xffffffffu, e.hi[2], o); b.z = __shfl_xor_sync(0xffffffffu, e.lo[2], o);
        a.w = __shfl_xor_sync(0xffffffffu, e.hi[3], o); b.w = __shfl_xor_sync(0xffffffffu, e.lo[3], o);
        e.add(a, b);
    }
    store_sketch(p, e, g.id, col, rg == 0 && col < cols);
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace attn

using namespace attn;

extern "C" {

attn_status_t attn_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int32_t* block_table,
                              const int32_t* free_pages, const int32_t* free_count, int B, int total_q,
                              int page_size, int max_pages, int num_pages, int n_free, int32_t* cu_seqlens_q,
                              int32_t* seq_lens, int32_t* positions, int32_t* slots, int32_t* free_left,
                              void* stream) {
    if (!ctx_lens || !block_table || !free_pages || !free_count || !cu_seqlens_q || !seq_lens || !positions ||
        !slots || !free_left)
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || total_q < 1 || page_size < 1 || max_pages < 1 || num_pages < 1 || n_free < 1)
        return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens),
                            static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                            static_cast<const void*>(free_count), static_cast<const void*>(cu_seqlens_q),
                            static_cast<const void*>(seq_lens), static_cast<const void*>(positions),
                            static_cast<const void*>(slots), static_cast<const void*>(free_left)})
        if (!aligned(ptr, 4)) return ATTN_ERR_INVALID_ARG;
    if (B > kPlanMaxB || page_size < 8 || page_size > 1024 || page_size % 8 != 0) return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size > 0x7fffffffLL || (long long)num_pages * page_size > 0x7fffffffLL)
        return ATTN_ERR_INVALID_ARG;

    PlanParams p;
    std::memset(&p, 0, sizeof p);
    int sm_count = 0;
    attn_status_t st = status_word_address(&p.status, &sm_count);
    if (st != ATTN_OK) return st;
    p.ctx = ctx_lens;
    p.fresh = new_lens;
    p.table = block_table;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.cu = cu_seqlens_q;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.slots = slots;
    p.free_left = free_left;
    p.B = B;
    p.total_q = total_q;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.n_free = n_free;
    const int smem = (3 * B + 1) * (int)sizeof(int);
    static std::atomic<unsigned long long> opted{0};
    if (opt_in_smem(reinterpret_cast<const void*>(paged_plan_kernel), (3 * kPlanMaxB + 1) * (int)sizeof(int), opted) !=
        cudaSuccess)
        return ATTN_ERR_CUDA;
    int ctas = (total_q + kPlanThreads - 1) / kPlanThreads;
    p.in_place = seq_lens == ctx_lens || seq_lens == new_lens || free_left == free_count;
    if (p.in_place)
        ctas = ctas >= kPlanMaxCluster ? kPlanMaxCluster : ctas > 2 ? 4 : ctas;
    else
        ctas = ctas > sm_count ? sm_count : ctas;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.in_place ? (unsigned)ctas : 1u;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_page_sketch(const void* k_cache, const int32_t* block_table, const int32_t* cu_seqlens_q,
                               const int32_t* seq_lens, int B, int max_q_len, int H_kv, int d, int page_size,
                               int max_pages, int num_pages, int8_t* sketch, float* amp, void* stream) {
    if (!k_cache || !block_table || !seq_lens || !sketch || !amp) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || max_q_len < 1 || H_kv < 1 || H_kv > 65535 || page_size < 1 || max_pages < 1 || num_pages < 1)
        return ATTN_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(sketch, 16) || !aligned(amp, 16) || !aligned(block_table, 4) ||
        !aligned(cu_seqlens_q, 4) || !aligned(seq_lens, 4))
        return ATTN_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
        return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size > 0x7fffffffLL || (long long)num_pages * page_size > 0x7fffffffLL)
        return ATTN_ERR_INVALID_ARG;

    SketchParams p;
    std::memset(&p, 0, sizeof p);
    // max_q_len tokens touch at most this many pages, wherever they start
    long long per_req = ((long long)max_q_len - 1 + page_size - 1) / page_size + 1;
    if (per_req > max_pages) per_req = max_pages;
    p.per_req = (int)per_req;
    const int cols = H_kv * d / 8;
    const bool many = (long long)B * per_req >= kManyPages;
    const bool narrow = many && cols <= 32 && (long long)page_size * cols <= kNarrowPieces;
    const int lanes = many ? 128 : 16;
    p.col_blocks = narrow ? 1 : (cols + lanes - 1) / lanes;
    const int pages_per_cta = narrow ? kSketchThreads / 32 : 1;
    const long long blocks = ((long long)B * per_req * p.col_blocks + pages_per_cta - 1) / pages_per_cta;
    if (blocks > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = status_word_address(&p.status);
    if (st != ATTN_OK) return st;
    p.k = static_cast<const uint16_t*>(k_cache);
    p.table = block_table;
    p.cu = cu_seqlens_q;
    p.seq_lens = seq_lens;
    p.sketch = sketch;
    p.amp = amp;
    p.B = B;
    p.max_q_len = max_q_len;
    p.H_kv = H_kv;
    p.d = d;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (narrow)
        page_sketch_warp_kernel<8><<<(unsigned)blocks, kSketchThreads, 0, cs>>>(p);
    else if (many)
        page_sketch_kernel<128, 12><<<(unsigned)blocks, kSketchThreads, 0, cs>>>(p);
    else
        page_sketch_kernel<16, 8><<<(unsigned)blocks, kSketchThreads, 0, cs>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
