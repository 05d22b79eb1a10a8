// sparse.cu -- page-sparse attention of single query tokens in one kernel:
// scores, selection and attention of one (token, KV head) at a time, the
// G <= 24 (d = 64: 32) query heads of the group against the chosen pages.
//
// Bound by memory: 4 d bytes of K and V per key serve 4 d G flops, and the
// sketches are 1/64 of a 64-row page's keys, so the kernel has to keep loads in
// flight on every SM and little else; for few tokens it is bound by the chain
// length -> table -> sketches -> selection -> keys, which one launch keeps
// short.  A cluster of CTAs takes a (token, KV head):
//   1. its warps score the pages, 16 at a time (select.cuh), and put each score
//      into the shared memory of every CTA of the cluster (eight warps per CTA:
//      the sketches are small and their loads latency-bound);
//   2. every CTA selects for itself from the whole list (the scores are the
//      same bits everywhere, so are the choices);
//   3. the chosen keys are cut into chunks of 16 (d = 64: 32) and dealt to four
//      warps of each CTA.  Each warp is its own pipeline, with no barrier between
//      warps: one lane keeps STAGES chunks of 8 KB in flight into the warp's own
//      shared-memory ring (one TMA box per page and panel of a chunk), and the
//      warp runs the online softmax on the chunk that has landed;
//   4. the warps' partials (O, m, l) meet in shared memory, across the cluster
//      through distributed shared memory, in one merge.
// So a token occupies up to eight SMs without scores, tables or partials in
// device memory, and a CTA is small enough that two share an SM and cover each
// other's phases.
//
// The products run transposed, S^T = K Q^T and O^T = V^T P^T: 16 keys (or 16
// dims of V) fill the 16 rows of the warp-level matrix instruction and the
// query heads are its 8 columns, so a group of up to 8 heads wastes nothing
// that 128 rows of a whole-CTA tile would.  In this orientation a thread holds
// the same two heads in S^T and in O^T: the running maximum and the rescaling
// stay in its registers.  P^T becomes the second product's operand by a
// register transpose within the warp.
//
//   m' = max(m, max_k s_k)  (raised lazily, by more than kTau at a time)
//   l  = l 2^(m - m') + sum_k 2^(s_k - m'),  O = O 2^(m - m') + sum_k 2^(s_k - m') V_k
// in log2 units, and at the end the (m, l, O) merge over the warps.
//
// Measured, d = 128, 32 query heads over 8, 64-row pages: one token of 32000
// keys, 32 pages chosen: 13.7 us (1.3 to the token's position, 2.8 scores, 2.3
// selection, 3.6 attention, 2.6 merge, the rest launch and barriers); 32 tokens
// of up to 65536 keys, 64 pages chosen: 101 us, 0.83 of what its bytes take at
// the copy rate (14 scores, 3 selection, 66 - 90 attention, 3 merge); 4 tokens
// of 200000 - 262144 keys, 128 pages chosen: 47 us.
#include <cooperative_groups.h>

#include <cmath>

#include "kernels.h"
#include "ptx.cuh"
#include "select.cuh"

namespace attn {

namespace {

namespace cg = cooperative_groups;

constexpr float kTau = 8.0f;  // log2 units
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kWarps = 4;       // warps that attend
constexpr int kAllWarps = 8;    // and all of a CTA's: scores, selection and merge
constexpr int kThreads = kAllWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxG = 32;       // query heads per KV head: four column tiles
constexpr int kMaxBudget = 1024;  // pages in a CTA's list

template <int D>
struct SCfg {
    static constexpr int KEYS = sparse_chunk_keys(D); // keys per chunk
    static constexpr int KT = KEYS / 16;              // row tiles of a chunk
    static constexpr int NPANEL = D / 64;             // 128-byte panels of the head dim
    static constexpr int PANEL_BYTES = KEYS * 128;    // KEYS rows x 128 B, 128-byte swizzle
    static constexpr int TILE_BYTES = NPANEL * PANEL_BYTES;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K and V
    static constexpr int STAGES = 3;
    static constexpr int RING_BYTES = STAGES * STAGE_BYTES;  // per warp
    static constexpr int O_ROW = D + 4;               // floats per head of a warp's partial O: no bank conflicts
    // before the first load the rings hold the query codes and the scores
    static constexpr int OFF_CODES = 0;
    static constexpr int OFF_HEADS = OFF_CODES + kMaxG * 2 * D;
    static constexpr int OFF_KEYS = OFF_HEADS + kMaxG * 8;
    static constexpr int AHEAD = D == 128 ? 2 : 4;                   // groups of 16 sketches in a warp's registers
    static constexpr int MAX_PAGES = (kWarps * RING_BYTES - OFF_KEYS) / 4;
    static constexpr int OFF_LIST = kWarps * RING_BYTES;             // the chosen pages [kMaxBudget]
    static constexpr int OFF_ML = OFF_LIST + kMaxBudget * 4;         // (m, l) [kWarps][kMaxG]
    static constexpr int OFF_W = OFF_ML + kWarps * kMaxG * 8;        // merge weights [kMaxG][kMaxCluster * kWarps]
    static constexpr int OFF_BAR = OFF_W + kMaxG * kMaxCluster * kWarps * 4;
    static constexpr int OFF_SCRATCH = OFF_BAR + kWarps * STAGES * 8;
    static constexpr int OFF_MISC = OFF_SCRATCH + (int)sizeof(SelectScratch<kThreads>);
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;  // + alignment of the ring to 1024
    static_assert(kBins * 4 <= kMaxG * 2 * D, "the selection's bins take the codes' place");
    static_assert(kMaxG * O_ROW * 4 <= RING_BYTES, "a warp's partial O overlays its ring");
    static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8 x 8 matrix of 16-bit elements across the warp
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NT column tiles of 8 query heads.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT * D <= 128 ? 2 : 1) sparse_kernel(const __grid_constant__ SparseParams p) {
    using C = SCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    cg::cluster_group cluster = cg::this_cluster();
    const SelectParams& sp = p.sel;
    const int n_ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = (int)(blockIdx.x / n_ctas);  // (token, KV head)
    const int t = row / sp.H_kv, kvh = row % sp.H_kv;
    const int W = n_ctas * kWarps, gw = rank * kWarps + warp;  // attending warps of the cluster, and this one
    const int SW = n_ctas * kAllWarps, gs = rank * kAllWarps + warp;  // the same of all warps
    // the ring starts on 1024 bytes of the shared window, in every CTA alike: a peer's address is this CTA's
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t ring = base + (warp % kWarps) * C::RING_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + (warp % kWarps) * C::STAGES;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    volatile int* s_skip = abort_flag + 1;  // an earlier launch gave up
    float2* s_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    int* s_list = reinterpret_cast<int*>(smem + C::OFF_LIST);
    auto sync_all = [&]() {
        if (n_ctas > 1)
            cluster.sync();
        else
            __syncthreads();
    };

    if (lane == 0 && warp < kWarps) {
        for (int s = 0; s < C::STAGES; ++s) bar_init(&bars[s], 1);
        bar_init_fence();
        if (warp == 0) {
            tma_prefetch_map(&p.tm_k);
            tma_prefetch_map(&p.tm_v);
        }
    }
    if (tid == 0) {
        *abort_flag = 0;
        *s_skip = timeout_recorded(sp.status) ? 1 : 0;
    }
    bool bad = false;
    const Token tok = token_of(sp, t, lane, bad);
    const int ps = 1 << sp.page_shift;
    const int n_vis = tok.pos < 0 ? 0 : (int)(tok.pos >> sp.page_shift) + 1;
    const int n_sel = min(n_vis, sp.budget);
    const int sel_len = n_vis == 0 ? 0 : (n_sel - 1) * ps + (int)(tok.pos & (ps - 1)) + 1;
    const int32_t* table = sp.table + (long long)tok.r * sp.max_pages;
    const uint16_t* q_group = sp.q + ((long long)t * sp.H + kvh * sp.G) * D;

    // Q^T as the second operand: head lane / 4 of each column tile, dims 16 kk + 2 (lane % 4) and + 8;
    // loaded ahead of the selection where the registers allow it
    uint32_t qf[NT][D / 16][2];
    auto load_q = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = n * 8 + (lane >> 2);
            const uint32_t* q = reinterpret_cast<const uint32_t*>(q_group + (long long)(h < sp.G ? h : 0) * D) + (lane & 3);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t a = __ldg(q + kk * 8), b = __ldg(q + kk * 8 + 4);
                qf[n][kk][0] = h < sp.G ? a : 0u;
                qf[n][kk][1] = h < sp.G ? b : 0u;
            }
        }
    };
    if (NT <= 2) load_q();

    // ---- 1, 2: the page list (every CTA of the cluster takes the same branches: they depend on the token alone)
    if (n_vis <= sp.budget) {
        for (int i = tid; i < n_vis; i += kThreads) s_list[i] = __ldg(table + i);
    } else {
        const int need = sp.budget - sp.first - sp.last;
        const int n = n_vis - sp.first - sp.last;
        for (int i = tid; i < sp.first; i += kThreads) s_list[i] = __ldg(table + i);
        for (int i = tid; i < sp.last; i += kThreads)
            s_list[sp.budget - sp.last + i] = __ldg(table + n_vis - sp.last + i);
        if (need > 0) {
            uint4* s_codes = reinterpret_cast<uint4*>(smem + C::OFF_CODES);
            float2* s_heads = reinterpret_cast<float2*>(smem + C::OFF_HEADS);
            uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem + C::OFF_KEYS);
            // a warp's candidates come in groups of 16, the sketches of kAhead groups on their way to registers
            const int32_t* from = table + sp.first;  // candidate c is page first + c
            const int groups = (n + 15) / 16;
            // the warp's page ids first, all at once, to where their scores will be
            for (int g = gs + (lane >> 4) * SW; g < groups; g += 2 * SW) {
                const int c = g * 16 + (lane & 15);
                if (c < n) s_keys[c] = (uint32_t)__ldg(from + c);
            }
            __syncwarp();
            constexpr int kAhead = C::AHEAD;
            SketchLoads<D, 2> loads[kAhead];
            auto fetch = [&](SketchLoads<D, 2>& to, int g) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int c = g * 16 + s * 8 + (lane >> 2);
                    to.id[s] = c < n ? (int)s_keys[c] : -1;
                }
                to.fetch(sp, kvh, g * 16, n, lane, bad);
            };
#pragma unroll
            for (int x = 0; x < kAhead; ++x)
                if (gs + x * SW < groups) fetch(loads[x], gs + x * SW);
            make_codes<D>(q_group, sp.G, s_codes, s_heads, warp, kAllWarps, lane);
            sync_all();  // the codes are there, and every CTA of the cluster runs
            for (int g0 = gs; g0 < groups; g0 += kAhead * SW)
#pragma unroll
                for (int x = 0; x < kAhead; ++x) {
                    const int g = g0 + x * SW;
                    if (g >= groups) break;
                    uint32_t key[2];
                    loads[x].template keys<NT>(s_codes, s_heads, sp.G, lane, key);
                    if (g + kAhead * SW < groups) fetch(loads[x], g + kAhead * SW);
                    const int s = lane & 1, c = g * 16 + s * 8 + (lane >> 2);
                    if ((lane & 2) == 0 && c < n) {
                        const uint32_t mine = s ? key[1] : key[0];
                        if (n_ctas > 1)
                            for (int r = 0; r < n_ctas; ++r) *cluster.map_shared_rank(s_keys + c, r) = mine;
                        else
                            s_keys[c] = mine;
                    }
                }
            sync_all();
            select_best<kThreads>(s_keys, n, need, reinterpret_cast<int*>(smem + C::OFF_CODES),
                                     *reinterpret_cast<SelectScratch<kThreads>*>(smem + C::OFF_SCRATCH),
                                     [&](int place, int i) { s_list[sp.first + place] = __ldg(table + sp.first + i); });
        }
    }
    if (bad) atomicOr(sp.status, 1u << kStatusDeviceData);

    if (NT > 2) load_q();
    fence_async_smem();  // what the rings held gives way to TMA writes
    __syncthreads();
    const bool skip = *s_skip != 0;
    const int n_keys = skip ? 0 : sel_len;
    if (sp.tables != nullptr && rank == 0) {
        int32_t* out = sp.tables + (long long)row * sp.budget;
        for (int i = tid; i < sp.budget; i += kThreads) {  // an id out of range becomes -1 (its loads report it)
            const int id = i < n_sel ? s_list[i] : -1;
            out[i] = id < sp.num_pages ? max(id, -1) : -1;
        }
        if (tid == 0 && kvh == 0) sp.sel_lens[t] = sel_len;
    }

    // ---- 3: this warp's chunks: gw, gw + W, gw + 2 W, ..
    const int chunks = (n_keys + C::KEYS - 1) / C::KEYS;
    const int mine = warp < kWarps && chunks > gw ? (chunks - gw + W - 1) / W : 0;
    const int boxes = ps < C::KEYS ? C::KEYS / ps : 1;  // boxes per panel of a chunk

    // cache row of box x of the warp's chunk i: a box past the last page, or of a page that does not exist,
    // starts behind the cache and reads zeros
    auto cache_row = [&](int i, int x) {
        const int k = (gw + i * W) * C::KEYS + x * ps;
        if (k >= n_keys) return p.kv_rows;
        const int id = s_list[k >> sp.page_shift];
        if (id >= 0 && id < sp.num_pages) return (id << sp.page_shift) + (k & (ps - 1));
        atomicOr(sp.status, 1u << kStatusDeviceData);
        return p.kv_rows;
    };
    auto load = [&](int i) {  // the warp's chunk i into its stage (one lane)
        const int s = i % C::STAGES;
        uint8_t* dst = smem + warp * C::RING_BYTES + s * C::STAGE_BYTES;
        bar_arrive_expect_tx(&bars[s], C::STAGE_BYTES);
        for (int x = 0; x < boxes; ++x) {
            const int r = cache_row(i, x);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
#pragma unroll
                for (int pn = 0; pn < C::NPANEL; ++pn)
                    tma_load_3d(dst + kv * C::TILE_BYTES + pn * C::PANEL_BYTES + x * ps * 128, kv ? &p.tm_v : &p.tm_k, &bars[s],
                                pn * 64, kvh, r);
        }
    };
    int loaded = min(C::STAGES, mine);
    if (lane == 0)
        for (int i = 0; i < loaded; ++i) load(i);

    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];  // heads 2 (lane % 4) and + 1 of each column tile; l: this thread's keys only
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }
    // row of this lane in the four 8 x 8 matrices of one ldmatrix: K by (keys, dims), V by (dims, keys) transposed
    const int k_key = (lane & 7) + ((lane >> 3) & 1) * 8, k_chunk = lane >> 4;
    const int v_key = (lane & 7) + (lane >> 4) * 8, v_chunk = (lane >> 3) & 1;

    bool ok = true;
    int i = 0;
    for (; i < mine; ++i) {
        const int s = i % C::STAGES;
        ok = __all_sync(0xffffffffu, wait_bar(&bars[s], (uint32_t)((i / C::STAGES) & 1), abort_flag, sp.status));
        if (!ok) break;
        const uint32_t kt = ring + s * C::STAGE_BYTES, vt = kt + C::TILE_BYTES;
        const int key0 = (gw + i * W) * C::KEYS;
        if (key0 + C::KEYS > n_keys) {
            // cache rows behind the token's last key may hold anything, and 0 times NaN would reach O
            for (int z = n_keys - key0 + (lane >> 3); z < C::KEYS; z += 4)
#pragma unroll
                for (int pn = 0; pn < C::NPANEL; ++pn)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + pn * C::PANEL_BYTES + z * 128 +
                                                                                  (lane & 7) * 16),
                                 "r"(0u)
                                 : "memory");
            __syncwarp();
        }
        float sc[C::KT][NT][4];
#pragma unroll
        for (int y = 0; y < C::KT; ++y)
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[y][n][0] = sc[y][n][1] = sc[y][n][2] = sc[y][n][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int y = 0; y < C::KT; ++y) {
                uint32_t a[4];
                const int c = kk * 2 + k_chunk;
                ldsm4(a, kt + (c >> 3) * C::PANEL_BYTES + (y * 16 + k_key) * 128 + (((c & 7) ^ (k_key & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(sc[y][n], a, qf[n][kk][0], qf[n][kk][1]);
            }
        // sc[y][n][0..1]: key 16 y + lane / 4, heads 2 (lane % 4), + 1; [2..3]: key + 8
        uint32_t pt[C::KT][NT][2], pr[C::KT][NT][2];  // P^T in bf16, and what that rounding left out
        bool moved = false;
        float alpha[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY;
#pragma unroll
                for (int y = 0; y < C::KT; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const bool in = key0 + y * 16 + x * 8 + (lane >> 2) < n_keys;
                        float& v = sc[y][n][2 * x + e];
                        v = in ? v * p.c_scale : -INFINITY;
                        top = fmaxf(top, v);
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                alpha[n][e] = 1.f;
                if (top > m[n][e] + kTau) {
                    alpha[n][e] = ex2(m[n][e] - top);  // m = -inf: 0
                    m[n][e] = top;
                    l[n][e] *= alpha[n][e];
                    moved = true;
                }
                const float mu = m[n][e] == -INFINITY ? 0.f : m[n][e];
#pragma unroll
                for (int y = 0; y < C::KT; ++y) {
                    sc[y][n][e] = ex2(sc[y][n][e] - mu);
                    sc[y][n][2 + e] = ex2(sc[y][n][2 + e] - mu);
                    l[n][e] += sc[y][n][e] + sc[y][n][2 + e];
                }
            }
#pragma unroll
            for (int y = 0; y < C::KT; ++y)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p0 = sc[y][n][2 * x], p1 = sc[y][n][2 * x + 1];
                    const uint32_t w = pack_bf16(p0, p1);
                    pt[y][n][x] = transpose8(w);
                    pr[y][n][x] = transpose8(pack_bf16(p0 - bf16lo_to_f32(w), p1 - bf16hi_to_f32(w)));
                }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    o[n][x][0] *= alpha[n][0];
                    o[n][x][1] *= alpha[n][1];
                    o[n][x][2] *= alpha[n][0];
                    o[n][x][3] *= alpha[n][1];
                }
        }
#pragma unroll
        for (int y = 0; y < C::KT; ++y)
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                uint32_t a[4];
                const int c = x * 2 + v_chunk;
                ldsm4_t(a, vt + (c >> 3) * C::PANEL_BYTES + (y * 16 + v_key) * 128 + (((c & 7) ^ (v_key & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816(o[n][x], a, pt[y][n][0], pt[y][n][1]);
                    mma16816(o[n][x], a, pr[y][n][0], pr[y][n][1]);
                }
            }
        __syncwarp();  // every lane has read the stage
        if (loaded < mine) {
            if (lane == 0) load(loaded);
            ++loaded;
        }
    }
    if (!ok && lane == 0)  // copies in flight land before the ring is reused or released
        for (int x = i; x < loaded; ++x) drain_wait(&bars[x % C::STAGES], (uint32_t)((x / C::STAGES) & 1), sp.status);
    __syncwarp();

    // ---- 4: this warp's partial: O over its ring, (m, l) beside
    float* po = reinterpret_cast<float*>(smem + (warp % kWarps) * C::RING_BYTES);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[n][e];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int h = n * 8 + (lane & 3) * 2 + e;
            if (warp < kWarps && lane < 4) s_ml[warp * kMaxG + h] = make_float2(m[n][e], sum);
            if (warp < kWarps && h < sp.G) {
                float* to = po + h * C::O_ROW + (lane >> 2);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    to[x * 16] = o[n][x][e];
                    to[x * 16 + 8] = o[n][x][2 + e];
                }
            }
        }
    sync_all();
    // This CTA's share of the outputs: whole 16-byte pieces of O, E of them in the group.  First the
    // weights 2^(m_j - m) / l of the W partials of each head in the share, then the pieces, `ways`
    // neighbouring threads to a piece, each summing every ways-th partial.
    constexpr int PIECES = D / 4;  // fp32 pieces of a head
    const int E = sp.G * PIECES;
    const int share = (E + n_ctas - 1) / n_ctas;
    const int e0 = min(E, rank * share), e1 = min(E, e0 + share);
    float* s_w = reinterpret_cast<float*>(smem + C::OFF_W);
    const bool write = !skip && tok.owned && e0 < e1;
    if (write) {
        for (int h = e0 / PIECES + warp; h <= (e1 - 1) / PIECES; h += kAllWarps) {
            float mj = -INFINITY, lj = 0.f;
            if (lane < W) {
                const float2* src = s_ml + (lane % kWarps) * kMaxG + h;
                const float2 ml = n_ctas > 1 ? *cluster.map_shared_rank(src, lane / kWarps) : *src;
                mj = ml.x;
                lj = ml.y;
            }
            float top = mj;
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float wj = mj == -INFINITY ? 0.f : ex2(mj - top);
            float sum = lj * wj;
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // NaN stays
            if (lane < W) s_w[h * (kMaxCluster * kWarps) + lane] = wj * inv;
            if (lane == 0 && p.lse != nullptr && h * PIECES >= e0)
                p.lse[(long long)t * sp.H + kvh * sp.G + h] = sum == 0.f ? -INFINITY : (top + lg2(sum)) * kLn2;
        }
    }
    __syncthreads();
    if (write) {
        int ways = 1;
        while (ways * 2 <= W && (e1 - e0) * ways * 2 <= kThreads) ways *= 2;
        const int per = kThreads / ways;  // pieces at a time
        for (int e = e0 + tid / ways; e < e1 + per; e += per) {  // whole warps, for the shuffles
            if (e - tid / ways >= e1) break;
            const bool in = e < e1;
            const int h = in ? e / PIECES : e0 / PIECES, c = in ? e % PIECES : 0;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int j = tid % ways; j < W; j += ways) {
                const float w = s_w[h * (kMaxCluster * kWarps) + j];
                const float* src = reinterpret_cast<const float*>(smem + (j % kWarps) * C::RING_BYTES) + h * C::O_ROW + c * 4;
                if (n_ctas > 1) src = cluster.map_shared_rank(src, j / kWarps);
                const float4 v = *reinterpret_cast<const float4*>(src);
                acc.x = fmaf(w, v.x, acc.x);
                acc.y = fmaf(w, v.y, acc.y);
                acc.z = fmaf(w, v.z, acc.z);
                acc.w = fmaf(w, v.w, acc.w);
            }
            for (int x = 1; x < ways; x <<= 1) {
                acc.x += __shfl_xor_sync(0xffffffffu, acc.x, x);
                acc.y += __shfl_xor_sync(0xffffffffu, acc.y, x);
                acc.z += __shfl_xor_sync(0xffffffffu, acc.z, x);
                acc.w += __shfl_xor_sync(0xffffffffu, acc.w, x);
            }
            if (in && tid % ways == 0)
                *reinterpret_cast<uint2*>(p.o + ((long long)t * sp.H + kvh * sp.G + h) * D + c * 4) =
                    make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
        }
    }
    if (n_ctas > 1) cluster.sync();  // peers may still be reading this CTA's partials
}

template <int D, int NT>
cudaLaunchConfig_t launch_config(int cluster, cudaLaunchAttribute* attr) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SCfg<D>::SMEM_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of 2^log2 CTAs that the device holds at once, asked once per device: a cluster stays within a
// group of SMs, so these are fewer than the SMs' CTAs make up (groups of 18 SMs hold two clusters of
// eight with one CTA to an SM).
template <int D, int NT>
cudaError_t resident_clusters(int log2, int* n) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][4];  // the number + 1; 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    std::atomic<int>& k = known[dev][log2];
    *n = k.load(std::memory_order_acquire) - 1;
    if (*n >= 0) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = launch_config<D, NT>(1 << log2, attr);
    e = cudaOccupancyMaxActiveClusters(n, sparse_kernel<D, NT>, &cfg);
    if (e == cudaSuccess) k.store(*n + 1, std::memory_order_release);
    return e;
}

// CTAs per (token, KV head): no more than let the whole launch reside on the GPU at once, and no more than there
// is work for.  Up to one CTA per SM that is a chunk of keys for each attending warp, or a group of pages for
// each scoring warp; beyond, where CTAs begin to share SMs, four chunks.  Measured (d = 128, us, CTAs per row
// 1, 2, 4, 8; 32 heads over 8): one token, 4 of 500 64-row pages 13.4, 12.5, 11.4, 11.4; 8 of 2000 16-row pages
// 19.7, 15.9, 13.9, 12.6; 4 tokens, 16 of 500 64-row pages 22.7, 17.0, 13.8, 14.3; 128 of 4000: 146, 82, 49, 48;
// more than fit: 16 tokens, 32 of 500 pages 38.4, 37.3, 47.7, 69.3.
// Pages are counted by the table's width, since the lengths are on the device: one token of 2000 keys in 16-row
// pages, 8 of them, takes 10.3, 11.0, 11.7, 11.8 and 11.0 by the rule in a table of its own 125 pages, 11.8 in
// one of 1024 to 16384.
template <int D, int NT>
cudaError_t launch_t(const SparseParams& p, int sm_count, cudaStream_t stream) {
    static std::atomic<unsigned long long> opted{0};
    cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(sparse_kernel<D, NT>), SCfg<D>::SMEM_BYTES, opted);
    if (e != cudaSuccess) return e;
    const SelectParams& s = p.sel;
    const long long rows = (long long)s.total_q * s.H_kv;
    const long long keys = (long long)(s.budget < s.max_pages ? s.budget : s.max_pages) << s.page_shift;
    const long long chunks = (keys + SCfg<D>::KEYS - 1) / SCfg<D>::KEYS;
    const long long groups = s.budget < s.max_pages ? (s.max_pages + 15) / 16 : 0;  // of pages to score
    int log2 = 0;
    while ((1 << log2) < kMaxCluster) {
        const int next = 1 << (log2 + 1);
        if (rows * next <= sm_count ? chunks < (long long)next * kWarps && groups < (long long)next * kAllWarps
                                    : chunks < (long long)next * 4 * kWarps)
            break;
        int fit = 0;
        e = resident_clusters<D, NT>(log2 + 1, &fit);
        if (e != cudaSuccess) return e;
        if (rows > fit) break;
        ++log2;
    }
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = launch_config<D, NT>(1 << log2, attr);
    cfg.gridDim = dim3((unsigned)(rows << log2));
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, sparse_kernel<D, NT>, p);
}

template <int D>
cudaError_t launch_d(const SparseParams& p, int sm_count, cudaStream_t stream) {
    switch ((p.sel.G + 7) / 8) {
    case 1: return launch_t<D, 1>(p, sm_count, stream);
    case 2: return launch_t<D, 2>(p, sm_count, stream);
    case 3: return launch_t<D, 3>(p, sm_count, stream);
    case 4:
        if constexpr (D == 64) return launch_t<D, 4>(p, sm_count, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// Larger groups run on the paged kernel's tiles of 128 rows, whose cost does
// not grow with the group.  Measured there and here, us, tokens of 4 KV heads
// over 4096 of 16384 - 32768 keys: d = 128, 32 tokens, G = 8: 79 and 60, 12: 80
// and 73, 16: 82 and 74, 24: 89 and 86, 32: 91 and 117 (four column tiles need all
// registers); 4 tokens, G = 16: 31 and 29, 24: 33 and 35; d = 64, 32 tokens, G = 16:
// 66 and 48 (two column tiles at 128 registers spill 56 bytes), 24: 68 and 50,
// 32: 69 and 57; 4 tokens, G = 32: 30 and 26.
bool sparse_fused_ok(int d, int G, int max_pages, int budget) {
    return G <= (d == 128 ? 24 : kMaxG) && budget <= kMaxBudget && max_pages <= (d == 128 ? SCfg<128>::MAX_PAGES : SCfg<64>::MAX_PAGES);
}

cudaError_t launch_sparse(int d, const SparseParams& p, int sm_count, cudaStream_t stream) {
    if (d == 128) return launch_d<128>(p, sm_count, stream);
    if (d == 64) return launch_d<64>(p, sm_count, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
