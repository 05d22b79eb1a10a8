// select.cu -- page selection as a call of its own (select.cuh holds the
// mathematics and the device functions).
//
// The score kernel is bound by reading 2 d + 4 bytes per page and KV head,
// 1/64 of a 64-row page's keys: four lanes take a page, up to sixteen 16-byte
// loads in flight per lane, and go to the matrix units from registers.
//
// The selection kernel takes one (token, KV head) per CTA and is latency-bound.
// It reads the scores through L1, a few times each: a copy in shared memory
// first was no faster.  Score CTAs of 64 pages instead of 128 gained 0.5 us at
// 512 pages of one token and lost 3 to 20% elsewhere.  Both kernels, 8 KV heads:
// one token of 512 pages 10.0 us, of 4096 17.0, 64 tokens of 1024 44.2 (20 of
// them for the bytes); selection by 512 threads 10.9, 15.7, 53.7, by 128 9.9,
// 27.9, 45.9.
#include <cmath>
#include <cstring>

#include "attn_kv.h"
#include "kernels.h"
#include "ptx.cuh"
#include "select.cuh"

namespace attn {

namespace {

constexpr int kScoreWarps = 4;
constexpr int kSelectThreads = 256;

constexpr int kSteps = 4;  // 32 pages per warp

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) page_score_kernel(const __grid_constant__ SelectParams p) {
    constexpr int PAGES = kScoreWarps * kSteps * 8;
    extern __shared__ uint4 s_codes[];  // [G][pieces], then the heads' scalars [G]
    float2* s_heads = reinterpret_cast<float2*>(s_codes + p.G * kPieces<D>);
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
    if (n_vis <= p.budget || chunk * PAGES >= n_vis) return;  // everything is taken, or nothing is here

    // the sketches are on their way while the codes are made
    const int first = chunk * PAGES + warp * kSteps * 8;
    SketchLoads<D, kSteps> loads;
    loads.look_up(p.table + (long long)k.r * p.max_pages, first, n_vis, lane);
    loads.fetch(p, kvh, first, n_vis, lane, bad);
    make_codes<D>(p.q + ((long long)t * p.H + kvh * p.G) * D, p.G, s_codes, s_heads, warp, kScoreWarps, lane);
    __syncthreads();
    uint32_t key[kSteps];
    loads.template keys<2>(s_codes, s_heads, p.G, lane, key);
    uint32_t* keys = p.keys + ((long long)t * p.H_kv + kvh) * p.max_pages;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int page = first + s * 8 + (lane >> 2);
        if ((lane & 3) == 0 && page < n_vis) keys[page] = key[s];
    }
    if (bad) atomicOr(p.status, 1u << kStatusDeviceData);
}

__global__ void __launch_bounds__(kSelectThreads) page_select_kernel(const __grid_constant__ SelectParams p) {
    __shared__ SelectScratch<kSelectThreads> scratch;
    __shared__ int s_bins[kBins];
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
    auto page_id = [&](int i) {  // of the request's page i; -1 and reported where the table names none
        const int id = __ldg(table + i);
        if (id >= 0 && id < p.num_pages) return id;
        atomicOr(p.status, 1u << kStatusDeviceData);
        return -1;
    };
    for (int i = n_sel + tid; i < p.budget; i += kSelectThreads) out[i] = -1;
    if (n_vis <= p.budget) {
        for (int i = tid; i < n_vis; i += kSelectThreads) out[i] = page_id(i);
        return;
    }

    // more pages than the budget: `first` in front, `last` behind, the best of [first, n_vis - last)
    const int need = p.budget - p.first - p.last;
    const int n = n_vis - p.first - p.last;  // > need
    for (int i = tid; i < p.first; i += kSelectThreads) out[i] = page_id(i);
    for (int i = tid; i < p.last; i += kSelectThreads) out[p.budget - p.last + i] = page_id(n_vis - p.last + i);
    if (need == 0) return;
    const uint32_t* keys = p.keys + ((long long)t * p.H_kv + kvh) * p.max_pages + p.first;
    const uint32_t lowest = select_best<kSelectThreads>(
        keys, n, need, s_bins, scratch, [&](int place, int i) { out[p.first + place] = __ldg(table + p.first + i); });
    if (lowest == ordered(-INFINITY)) {  // rare: pages that do not exist may be among the chosen (the scores reported them)
        __syncthreads();
        for (int i = p.first + tid; i < p.budget - p.last; i += kSelectThreads)
            if (out[i] < 0 || out[i] >= p.num_pages) out[i] = -1;
    }
}

template <int D>
cudaError_t launch_d(SelectParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.total_q * p.H_kv;
    const int smem = p.G * (2 * D + 8);
    if (p.max_pages > p.budget) {
        const int pages = kScoreWarps * kSteps * 8;
        p.n_chunks = (p.max_pages + pages - 1) / pages;
        page_score_kernel<D><<<(unsigned)(rows * p.n_chunks), kScoreWarps * 32, smem, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.max_pages > p.budget ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, page_select_kernel, p);
}

}  // namespace

size_t select_keys_bytes(int total_q, int H_kv, int max_pages, int budget) {
    if (max_pages <= budget) return 256;  // none needed
    const size_t n = ((size_t)total_q * H_kv * max_pages * sizeof(uint32_t) + 255) / 256 * 256;
    return n < 512 ? 512 : n;
}

cudaError_t launch_select(int d, SelectParams p, cudaStream_t stream) {
    if (d == 128) return launch_d<128>(p, stream);
    if (d == 64) return launch_d<64>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
