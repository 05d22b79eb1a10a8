// paged8.cu -- attention over a paged cache of e4m3 codes with block scales.
//
// A CTA per (query token, query head); a warp per key: its lanes hold d / 32 dims each.  Online
// softmax per warp (running max m, sum l, unnormalised O), the warps merged at the end.
#include <cmath>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float value(uint8_t x) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) paged8_simple_kernel(const __grid_constant__ Paged8Params p) {
    constexpr int PER = D / 32;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
    const int tok = blockIdx.x, head = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int r = tok, q_start = tok, q_len = 1;
    bool bad = false;
    if (p.cu_q != nullptr) {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(p.cu_q + mid) <= tok)
                lo = mid;
            else
                hi = mid - 1;
        }
        r = lo;
        const int a = __ldg(p.cu_q + r), b = __ldg(p.cu_q + r + 1);
        bad = a < 0 || b < a || b > p.total_q || b - a > p.max_q_len;
        if (!bad && (tok < a || tok >= b)) return;
        q_start = a;
        q_len = b - a;
    }
    int len = __ldg(p.seq_lens + r);
    const int cap = p.max_pages << p.page_shift;
    if (len < 0 || len > cap) {
        bad = true;
        len = len < 0 ? 0 : cap;
    }
    if (bad && threadIdx.x == 0) atomicOr(p.status, 1u << kStatusDeviceData);
    const long long limit = p.causal ? (long long)len - q_len + (tok - q_start) + 1 : len;
    const int n = (int)(limit < len ? limit : len);
    const int kvh = head / p.G;
    const int per_page = 1 << (p.page_shift - p.block_shift);
    const size_t row = (size_t)tok * p.H + head;
    float q[PER], o[PER], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        q[c] = __uint_as_float((uint32_t)p.q[row * D + lane * PER + c] << 16);
        o[c] = 0.f;
    }
    for (int k = warp; k < n; k += kWarps) {
        const int id = __ldg(p.block_table + (size_t)r * p.max_pages + (k >> p.page_shift));
        const int in_page = k & ((1 << p.page_shift) - 1);
        float s = 0.f, ks = 0.f, vs = 0.f;
        const size_t at = ((((size_t)(unsigned)id << p.page_shift) + in_page) * p.H_kv + kvh) * D + lane * PER;
        const bool ok = id >= 0 && id < p.num_pages;
        if (ok) {
            const size_t sc = ((size_t)id * p.H_kv + kvh) * per_page + (in_page >> p.block_shift);
            ks = __ldg(p.k_scale + sc);
            vs = __ldg(p.v_scale + sc);
#pragma unroll
            for (int c = 0; c < PER; ++c) s = fmaf(q[c], value(p.k_cache[at + c]), s);
        } else if (lane == 0) {
            atomicOr(p.status, 1u << kStatusDeviceData);
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= ks * p.c_scale;
        const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
        const float alpha = exp2f(m - base), w = exp2f(s - base);
        m = top;
        l = l * alpha + w;
#pragma unroll
        for (int c = 0; c < PER; ++c) o[c] = o[c] * alpha + (ok ? w * (vs * value(p.v_cache[at + c])) : 0.f);
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int c = 0; c < PER; ++c) s_o[warp][lane * PER + c] = o[c];
    __syncthreads();
    if (threadIdx.x >= D) return;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float base = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(s_m[w] - base);
        sum += s_l[w] * f;
        acc += s_o[w][threadIdx.x] * f;
    }
    const float out = sum == 0.f ? 0.f : acc / sum;
    p.o[row * D + threadIdx.x] = (uint16_t)pack_bf16(out, out);
    if (threadIdx.x == 0 && p.lse != nullptr)
        p.lse[row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.69314718055994530942f;
}

}  // namespace

cudaError_t launch_paged8(int d, const Paged8Params& p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.total_q, (unsigned)p.H);
    if (d == 128)
        paged8_simple_kernel<128><<<grid, kWarps * 32, 0, stream>>>(p);
    else
        paged8_simple_kernel<64><<<grid, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
