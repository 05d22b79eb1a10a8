// rope.cu -- rotary positions, and the cache append that rotates on its way.
//
// A pair (a, b) of a head vector at position P turns by t = P f_i:
//   a' = s (a cos t - b sin t),  b' = s (a sin t + b cos t).
//
// The angle.  In units of a whole turn it is P f_i / 2 pi, of which only the
// fraction matters.  f_i / 2 pi is held as a 64-bit binary fraction, so that the
// integer product with P, taken modulo 2^64, is that fraction to |P| 2^-63 turns
// for any 32-bit P and either sign, without float64 arithmetic.  Its first 24
// bits, as fp32 half turns in [-1, 1), feed sincospif; the angle e of the next
// 32 (below 2^-23 half turns) turns the result once more: (cos - e sin, sin + e
// cos), off by e^2 / 2 < 2^-43 of either.  So the cosine and sine are those
// functions' own (1 ulp) and one more rounding, however far the position, and
// small ones keep their relative accuracy.
//
// Work.  Bound by memory: each element is read and written once, 3 flops
// each.  A CTA takes TOK consecutive tokens and all (or a share) of their
// heads: the TOK * rot / 2 angles are computed once, by all threads, into
// shared memory; each thread then keeps the cosines and sines of its few
// pairs in registers and walks over the heads, 32 bytes of a head vector at a
// time (two 16-byte loads), three heads in flight.  Outputs of more than L2
// holds are stored evict-first, so that they do not push out lines that loads
// share.  Measured, [1, 32 + 8, 32768, 128] bf16: 100 us, 6.7 TB/s, 0.98 of a
// copy (2, 4, 5 heads in flight: 105, 110, 117 us; plain stores: 114; 8 tokens
// per CTA instead of 4: 102, but 48 for 44 us on fp32).  With a reader of q
// behind it: 80 MB out 51.8 us evict-first and 49.2 plain, 160 MB 95.4 and 94.6.
// Few tokens take a CTA or more each: 64 tokens of 40 heads 2.8 us (four to a
// CTA: 4.1), 512 both 4.4, 1024 7.0 (5.4), 4096 23 (17).
#include <cmath>
#include <cstring>

#include "attn_kv.h"
#include "kernels.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 3;  // heads whose loads a thread issues before it uses the first
constexpr long long kStreamBytes = 128LL << 20;  // L2
constexpr int kManyTokens = 512;
constexpr int kFewCtas = 304;  // for fewer tokens: two CTAs to each of the chip's 152 SMs

struct RopeSide {
    const char* in;
    char* out;
    long long ib, ih, it;  // input strides in bytes: batch, head, token
    long long ob, oh, ot;  // output strides in bytes (paged sides: oh only)
};

struct RopeParams {
    RopeSide q, k, v;        // v: append only
    const int32_t* positions;
    long long pos_b;
    const void* freq;
    int freq64;
    const int32_t* slots;    // append only
    long long n_slots;
    unsigned* status;
    int n_tokens, N;         // n_tokens = B * N
    int H, H_k, n_heads;     // n_heads = H + H_k (+ H_k for v)
    int d, rot;
    int tok, splits;         // tokens per CTA; CTAs that share a token's heads
    int stream;              // outputs too large to be found in L2 by who reads them next
    float amplitude, sign;
};

__device__ __forceinline__ uint4 ld16(const char* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ void st16(char* p, const uint4& v, bool stream) {
    if (stream)
        asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
    else
        asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
}

template <int EB>
struct Vec;  // the elements of 16 bytes
template <>
struct Vec<2> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
        x[0] = bf16lo_to_f32(v.x); x[1] = bf16hi_to_f32(v.x);
        x[2] = bf16lo_to_f32(v.y); x[3] = bf16hi_to_f32(v.y);
        x[4] = bf16lo_to_f32(v.z); x[5] = bf16hi_to_f32(v.z);
        x[6] = bf16lo_to_f32(v.w); x[7] = bf16hi_to_f32(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
};
template <>
struct Vec<4> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// Unit j of a head vector is two 16-byte pieces holding the VN pairs
// j VN .. j VN + VN - 1 (rotated units, j < rot / 2 VN) or 2 VN dims that pass
// through.
template <int EB, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = Vec<EB>;
    constexpr int VN = V::N;
    extern __shared__ unsigned long long smem_rope[];
    const int half = p.rot >> 1;
    unsigned long long* s_turn = smem_rope;                     // [rot / 2]
    float* s_cos = reinterpret_cast<float*>(s_turn + half);     // [tok][rot / 2]
    float* s_sin = s_cos + p.tok * half;
    const int tid = threadIdx.x;
    const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int t0 = tile * p.tok;  // within n_tokens < 2^31 by the grid

    for (int i = tid; i < half; i += kThreads)
        s_turn[i] = p.freq64 ? turn_fraction(static_cast<const double*>(p.freq)[i])
                             : turn_fraction(static_cast<const float*>(p.freq)[i]);
    const int units = p.d / (2 * VN);        // units of a head vector: 4, 8 or 16
    const int r_units = p.rot / (2 * VN);    // of which this many rotate
    __syncthreads();
    // pair i of token k at [k][i / 4 % (VN / 4)][i / VN][i % 4]: the threads of
    // neighbouring units then read neighbouring 16-byte pieces
    for (int x = tid; x < p.tok * half; x += kThreads) {
        const int k = x / half, i = x - k * half;
        const int t = t0 + k;
        if (t >= p.n_tokens) break;
        int pos;
        if (p.positions != nullptr) {
            const int b = t / p.N;
            pos = __ldg(p.positions + (long long)b * p.pos_b + (t - b * p.N));
        } else {
            pos = t % p.N;
        }
        float cs, sn;
        turned_cos_sin(s_turn[i], pos, &cs, &sn);
        const int at = k * half + (VN == 8 ? ((i >> 2) & 1) * (half >> 1) : 0) + (i / VN) * 4 + (i & 3);
        s_cos[at] = cs * p.amplitude;
        s_sin[at] = sn * p.sign * p.amplitude;
    }
    __syncthreads();

    const int j = tid % units;
    const int rest = tid / units;
    const int k = rest % p.tok;
    const int t = t0 + k;
    const int lanes = kThreads / (units * p.tok);  // heads side by side (at least 1)
    const int hl = rest / p.tok;
    if (t >= p.n_tokens || hl >= lanes) return;
    long long slot = 0;
    if (APPEND) {
        slot = __ldg(p.slots + t);
        if (slot >= p.n_slots) {
            if (j == 0 && hl == 0) atomicOr(p.status, 1u << kStatusDeviceData);
            return;
        }
        if (slot < 0) return;
    }
    const bool turns = j < r_units;
    float cs[VN], sn[VN];
    if (turns) {
#pragma unroll
        for (int e = 0; e < VN; e += 4) {
            const int at = k * half + (e >> 2) * (half >> 1) + j * 4;
            const float4 c4 = *reinterpret_cast<const float4*>(s_cos + at);
            const float4 s4 = *reinterpret_cast<const float4*>(s_sin + at);
            cs[e] = c4.x; cs[e + 1] = c4.y; cs[e + 2] = c4.z; cs[e + 3] = c4.w;
            sn[e] = s4.x; sn[e + 1] = s4.y; sn[e + 2] = s4.z; sn[e + 3] = s4.w;
        }
    }
    // byte offsets of the unit's two pieces; for a v vector nothing turns, so
    // the same pieces serve as a plain copy
    const bool split_halves = turns && !INTERLEAVED;
    const int off_a = split_halves ? j * 16 : j * 32;
    const int off_b = split_halves ? half * EB + j * 16 : j * 32 + 16;
    const int b = t / p.N;
    const long long n = t - b * p.N;

    const int step = lanes * p.splits;
    for (int h0 = split * lanes + hl; h0 < p.n_heads; h0 += step * kInFlight) {
        uint4 xa[kInFlight], xb[kInFlight];
        char* dst[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int h = h0 + u * step;
            dst[u] = nullptr;
            if (h < p.n_heads) {
                const bool is_q = h < p.H, is_v = APPEND && h >= p.H + p.H_k;
                const RopeSide& s = is_q ? p.q : is_v ? p.v : p.k;
                const int hh = is_q ? h : is_v ? h - p.H - p.H_k : h - p.H;
                const char* src = s.in + b * s.ib + hh * s.ih + n * s.it;
                if (APPEND && !is_q)
                    dst[u] = s.out + slot * s.ot + hh * s.oh;
                else
                    dst[u] = s.out + b * s.ob + hh * s.oh + n * s.ot;
                xa[u] = ld16(src + off_a);
                xb[u] = ld16(src + off_b);
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            if (dst[u] == nullptr) break;
            const bool is_v = APPEND && h0 + u * step >= p.H + p.H_k;
            if (turns && !is_v) {
                float a[VN], c[VN];
                V::unpack(xa[u], a);
                V::unpack(xb[u], c);
                if (INTERLEAVED) {  // pieces hold pairs (0, 1), (2, 3), ..
#pragma unroll
                    for (int e = 0; e < VN; e += 2) {
                        const float x0 = a[e], x1 = a[e + 1], y0 = c[e], y1 = c[e + 1];
                        a[e] = x0 * cs[e / 2] - x1 * sn[e / 2];
                        a[e + 1] = x0 * sn[e / 2] + x1 * cs[e / 2];
                        c[e] = y0 * cs[VN / 2 + e / 2] - y1 * sn[VN / 2 + e / 2];
                        c[e + 1] = y0 * sn[VN / 2 + e / 2] + y1 * cs[VN / 2 + e / 2];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VN; ++e) {
                        const float x = a[e], y = c[e];
                        a[e] = x * cs[e] - y * sn[e];
                        c[e] = x * sn[e] + y * cs[e];
                    }
                }
                xa[u] = V::pack(a);
                xb[u] = V::pack(c);
            }
            st16(dst[u] + off_a, xa[u], p.stream != 0);
            st16(dst[u] + off_b, xb[u], p.stream != 0);
        }
    }
}

template <int EB, bool IL, bool APPEND>
cudaError_t launch(const RopeParams& p, long long blocks, int smem, cudaStream_t stream) {
    rope_kernel<EB, IL, APPEND><<<(unsigned)blocks, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

// Tokens per CTA and CTAs per token tile.  A CTA of 256 threads covers
// 256 / units head vectors at a time.
void plan(RopeParams& p, int elem_bytes, long long* blocks) {
    const int units = p.d / (32 / elem_bytes);
    const int rows = kThreads / units;  // head vectors side by side in a CTA
    p.tok = p.n_tokens >= kManyTokens ? 4 : 1;
    if (p.tok > rows) p.tok = rows;
    const int lanes = rows / p.tok;
    p.splits = 1;
    if (p.tok == 1) {
        const int most = (p.n_heads + lanes - 1) / lanes;  // more would leave CTAs without a head
        const int want = (kFewCtas + p.n_tokens - 1) / p.n_tokens;
        p.splits = want < most ? want : most;
        if (p.splits < 1) p.splits = 1;
    }
    *blocks = (((long long)p.n_tokens + p.tok - 1) / p.tok) * p.splits;
}

cudaError_t run(RopeParams& p, int elem_bytes, bool interleaved, bool append, cudaStream_t stream) {
    long long blocks = 0;
    plan(p, elem_bytes, &blocks);
    p.stream = (long long)p.n_tokens * p.n_heads * p.d * elem_bytes > kStreamBytes;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int half = p.rot / 2;
    const int smem = half * 8 + p.tok * half * 8;
    if (append)
        return interleaved ? launch<2, true, true>(p, blocks, smem, stream)
                           : launch<2, false, true>(p, blocks, smem, stream);
    if (elem_bytes == 2)
        return interleaved ? launch<2, true, false>(p, blocks, smem, stream)
                           : launch<2, false, false>(p, blocks, smem, stream);
    return interleaved ? launch<4, true, false>(p, blocks, smem, stream)
                       : launch<4, false, false>(p, blocks, smem, stream);
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The strides of a tensor in the dims longer than 1: multiples of a 16-byte
// piece, not negative, an output's at least one head vector.
bool strides_ok(const long long* s, const long long* sizes, int n, int d, int elem_bytes, bool out) {
    for (int i = 0; i < n; ++i) {
        if (sizes[i] <= 1) continue;
        if (s[i] < 0 || s[i] % (16 / elem_bytes) != 0 || s[i] > (1LL << 60) / (sizes[i] + 1)) return false;
        if (out && s[i] < d) return false;
    }
    return true;
}

void set_side(RopeSide& s, const void* in, void* out, const long long* si, const long long* so, int eb) {
    s.in = static_cast<const char*>(in);
    s.out = static_cast<char*>(out);
    s.ib = si[0] * eb;
    s.ih = si[1] * eb;
    s.it = si[2] * eb;
    s.ob = so[0] * eb;
    s.oh = so[1] * eb;
    s.ot = so[2] * eb;
}

}  // namespace

attn_status_t append_args_ok(const void* q, const void* q_out, const void* k, const void* v, const void* k_cache,
                             const void* v_cache, const int32_t* slots, const int32_t* positions,
                             const void* inv_freq, int freq_bits, int T, int H, int H_kv, int d, int rot,
                             int page_size, int num_pages, const long long* strides, int interleaved,
                             float amplitude) {
    if (!k || !v || !k_cache || !v_cache || !slots || !strides || (q == nullptr) != (q_out == nullptr))
        return ATTN_ERR_INVALID_ARG;
    if (!q) H = 0;
    if (T < 1 || T > 0x7fffffff - 8 || H < 0 || H > 65535 || H_kv < 1 || H_kv > 65535 || (q && H < 1) || num_pages < 1 ||
        page_size < 1)
        return ATTN_ERR_INVALID_ARG;
    if (rot != 0 && (!positions || !inv_freq || (freq_bits != 32 && freq_bits != 64))) return ATTN_ERR_INVALID_ARG;
    if ((interleaved & ~1) || !std::isfinite(amplitude)) return ATTN_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || rot < 0 || rot > d || rot % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    if (page_size < 8 || page_size > 1024 || page_size % 8 != 0) return ATTN_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {q, static_cast<const void*>(q_out), k, v, static_cast<const void*>(k_cache),
                            static_cast<const void*>(v_cache)})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned(positions, 4) || (rot != 0 && !aligned(inv_freq, freq_bits / 8)))
        return ATTN_ERR_INVALID_ARG;
    const long long nq[2] = {T, H}, nk[2] = {T, H_kv};
    if (q && (!strides_ok(strides, nq, 2, d, 2, false) || !strides_ok(strides + 2, nq, 2, d, 2, true)))
        return ATTN_ERR_INVALID_ARG;
    if (!strides_ok(strides + 4, nk, 2, d, 2, false) || !strides_ok(strides + 6, nk, 2, d, 2, false))
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

}  // namespace attn

using namespace attn;

extern "C" {

attn_status_t attn_rope_inv_freq(double* inv_freq, double* amplitude, int rot, double base, int scaling,
                                 double factor, int orig_len, double low, double high) {
    if (!inv_freq || rot < 2 || rot > 1024 || rot % 2 != 0 || !(std::isfinite(base) && base > 1.0))
        return ATTN_ERR_INVALID_ARG;
    if (scaling < ATTN_ROPE_PLAIN || scaling > ATTN_ROPE_YARN) return ATTN_ERR_INVALID_ARG;
    if (scaling != ATTN_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return ATTN_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    if (scaling == ATTN_ROPE_BANDS || scaling == ATTN_ROPE_YARN) {
        if (orig_len < 1 || !(std::isfinite(high) && low > 0.0 && low < high)) return ATTN_ERR_INVALID_ARG;
    }
    if (scaling == ATTN_ROPE_NTK && rot > 2) base *= std::pow(factor, (double)rot / (rot - 2));
    double ramp0 = 0.0, ramp1 = 1.0;
    if (scaling == ATTN_ROPE_YARN) {
        auto at = [&](double turns) { return rot * std::log(orig_len / (two_pi * turns)) / (2.0 * std::log(base)); };
        auto clamp = [&](double x) { return x < 0.0 ? 0.0 : x > rot - 1.0 ? rot - 1.0 : x; };
        ramp0 = clamp(std::floor(at(high)));
        ramp1 = clamp(std::ceil(at(low)));
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == ATTN_ROPE_LINEAR) f /= factor;
        if (scaling == ATTN_ROPE_BANDS || scaling == ATTN_ROPE_YARN) {
            double keep;
            if (scaling == ATTN_ROPE_BANDS) {
                keep = (orig_len * f / two_pi - low) / (high - low);
            } else {
                const double width = ramp1 - ramp0 > 1e-3 ? ramp1 - ramp0 : 1e-3;
                keep = 1.0 - (i - ramp0) / width;
            }
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = keep * f + (1.0 - keep) * (f / factor);
        }
        inv_freq[i] = f;
    }
    if (amplitude) *amplitude = scaling == ATTN_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return ATTN_OK;
}

attn_status_t attn_rope(const void* q, void* q_out, const void* k, void* k_out, const int32_t* positions,
                        long long pos_stride_b, const void* inv_freq, int freq_bits, int elem_bytes, int B, int H,
                        int H_k, int N, int d, int rot, const long long* strides, int interleaved, int inverse,
                        float amplitude, void* stream) {
    if (!q || !q_out || !inv_freq || !strides || (k == nullptr) != (k_out == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (!k) H_k = 0;
    if (B < 1 || N < 1 || H < 1 || H > 65535 || H_k < 0 || H_k > 65535 || (k && H_k < 1)) return ATTN_ERR_INVALID_ARG;
    if ((long long)B * N > 0x7fffffffLL - 8) return ATTN_ERR_INVALID_ARG;
    if ((interleaved | inverse) & ~1) return ATTN_ERR_INVALID_ARG;
    if ((freq_bits != 32 && freq_bits != 64) || !std::isfinite(amplitude)) return ATTN_ERR_INVALID_ARG;
    if (elem_bytes != 2 && elem_bytes != 4) return ATTN_ERR_UNSUPPORTED;
    if ((d != 64 && d != 128) || rot < 16 || rot > d || rot % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(inv_freq, freq_bits / 8) || !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
    if (positions && (pos_stride_b < 0 || pos_stride_b > (1LL << 40))) return ATTN_ERR_INVALID_ARG;
    const long long nq[3] = {B, H, N}, nk[3] = {B, H_k, N};
    if (!strides_ok(strides, nq, 3, d, elem_bytes, false) || !strides_ok(strides + 3, nq, 3, d, elem_bytes, true))
        return ATTN_ERR_INVALID_ARG;
    if (k && (!strides_ok(strides + 6, nk, 3, d, elem_bytes, false) ||
              !strides_ok(strides + 9, nk, 3, d, elem_bytes, true)))
        return ATTN_ERR_INVALID_ARG;

    RopeParams p;
    std::memset(&p, 0, sizeof p);
    set_side(p.q, q, q_out, strides, strides + 3, elem_bytes);
    if (k) set_side(p.k, k, k_out, strides + 6, strides + 9, elem_bytes);
    p.positions = positions;
    p.pos_b = pos_stride_b;
    p.freq = inv_freq;
    p.freq64 = freq_bits == 64;
    p.n_tokens = B * N;
    p.N = N;
    p.H = H;
    p.H_k = H_k;
    p.n_heads = H + H_k;
    p.d = d;
    p.rot = rot;
    p.amplitude = amplitude;
    p.sign = inverse ? -1.f : 1.f;
    return run(p, elem_bytes, interleaved != 0, false, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

attn_status_t attn_paged_append(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                                void* v_cache, const int32_t* slots, const int32_t* positions,
                                const void* inv_freq, int freq_bits, int T, int H, int H_kv, int d, int rot,
                                int page_size, int num_pages, const long long* strides, int interleaved,
                                float amplitude, void* stream) {
    attn_status_t st = append_args_ok(q, q_out, k, v, k_cache, v_cache, slots, positions, inv_freq, freq_bits, T, H, H_kv,
                                      d, rot, page_size, num_pages, strides, interleaved, amplitude);
    if (st != ATTN_OK) return st;
    if (!q) H = 0;
    unsigned* status = nullptr;
    st = status_word_address(&status);
    if (st != ATTN_OK) return st;

    RopeParams p;
    std::memset(&p, 0, sizeof p);
    auto side = [&](RopeSide& s, const void* in, void* out, const long long* si, long long out_t, long long out_h) {
        const long long i3[3] = {0, si[1], si[0]}, o3[3] = {0, out_h, out_t};
        set_side(s, in, out, i3, o3, 2);
    };
    if (q) side(p.q, q, q_out, strides, strides[2], strides[3]);
    side(p.k, k, k_cache, strides + 4, (long long)H_kv * d, d);
    side(p.v, v, v_cache, strides + 6, (long long)H_kv * d, d);
    p.positions = positions;
    p.freq = inv_freq;
    p.freq64 = freq_bits == 64;
    p.slots = slots;
    p.n_slots = (long long)num_pages * page_size;
    p.status = status;
    p.n_tokens = T;
    p.N = T;
    p.H = H;
    p.H_k = H_kv;
    p.n_heads = H + 2 * H_kv;
    p.d = d;
    p.rot = rot;
    p.amplitude = amplitude;
    p.sign = 1.f;
    return run(p, 2, interleaved != 0, true, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                                              : ATTN_ERR_CUDA;
}

}  // extern "C"
