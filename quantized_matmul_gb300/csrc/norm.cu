// Root-mean-square norm with the residual's addition and an 8-bit output,
// ready for the quantized products: one launch takes the place of the
// addition, the norm and the activation quantizer.
//
//   h = x + r                          (f32; h = x without a residual)
//   y = (h * rsqrt(mean(h^2) + eps)) * w
//   Q8_0:   per 32-element block of y the recipe of qmm_quantize_act_q8_0
//   BitNet: per row of y the recipe of qmm_quantize_act_bitnet
//
// The sum of squares is f32 in a fixed order (thread, warp, CTA), so a row's
// bits do not depend on the other rows; division, square root and the codes'
// rounding are IEEE (the codes' rounding to 8 bits is the format's).
#include <cuda_fp16.h>

#include <cfloat>

#include "qmm_internal.h"

namespace qmm {
namespace {

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The code of y under a scale: round half away from zero, clamped.
__device__ __forceinline__ int code(float v) {
    return (int)fminf(fmaxf(roundf(v), -127.0f), 127.0f);
}

// 1 / sqrt(mean + eps); 0 for a row of zeros without eps, whose y is 0.
__device__ __forceinline__ float inverse_rms(float sum, const NormArgs &a) {
    const float mean = __fdiv_rn(sum, (float)a.k) + a.eps;
    return mean > 0.0f ? __fdiv_rn(1.0f, __fsqrt_rn(mean)) : 0.0f;
}

constexpr int kRowThreads = 256;

// Any k: the row is read again after the sum of squares (h is read back from
// where this thread wrote it, so h may be x or r itself).
template <bool BITNET>
__global__ void __launch_bounds__(kRowThreads)
rms_norm_rows_kernel(const NormArgs a, bool pdl) {
    __shared__ float s_part[kRowThreads / 32];
    __shared__ int s_sum[kRowThreads / 32];
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = blockIdx.x;
    const float *x = a.x + i * a.ldx;
    const float *r = a.r ? a.r + i * a.ldr : nullptr;
    float *h = a.h ? a.h + i * a.ldh : nullptr;
    float ss = 0.0f;
    for (int64_t j = threadIdx.x; j < a.k; j += kRowThreads) {
        const float v = r ? x[j] + r[j] : x[j];
        if (h) h[j] = v;
        ss = fmaf(v, v, ss);
    }
    ss = warp_sum(ss);
    if (lane == 0) s_part[warp] = ss;
    __syncthreads();
    float tot = 0.0f;
    for (int w = 0; w < kRowThreads / 32; ++w) tot += s_part[w];
    const float inv = inverse_rms(tot, a);
    auto normed = [&](int64_t j) {
        const float v = h ? h[j] : (r ? x[j] + r[j] : x[j]);
        return (v * inv) * a.w[j];
    };
    if (!BITNET) {
        for (int64_t j = threadIdx.x; j < a.k; j += kRowThreads) {  // a warp holds one block
            const float y = normed(j);
            const float d = __fdiv_rn(warp_max(fabsf(y)), 127.0f);
            a.aq[i * a.k + j] = (int8_t)(d != 0.0f ? code(__fdiv_rn(y, d)) : 0);
            if (lane == 0)
                a.ad[i * (a.k / kQK) + j / kQK] = __half_as_ushort(__float2half_rn(d));
        }
        return;
    }
    float amax = 0.0f;
    for (int64_t j = threadIdx.x; j < a.k; j += kRowThreads) amax = fmaxf(amax, fabsf(normed(j)));
    amax = warp_max(amax);
    __syncthreads();
    if (lane == 0) s_part[warp] = amax;
    __syncthreads();
    for (int w = 0; w < kRowThreads / 32; ++w) amax = fmaxf(amax, s_part[w]);
    const float scale = amax != 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
    int sum = 0;
    for (int64_t j = threadIdx.x; j < a.k; j += kRowThreads) {
        const int q = scale != 0.0f ? code(__fmul_rn(normed(j), scale)) : 0;
        a.aq[i * a.k + j] = (int8_t)q;
        sum += q;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kRowThreads / 32; ++w) sum += s_sum[w];
        a.scale[i] = scale;
        a.sum[i] = sum;
    }
}

// Four codes as bytes, lowest first: the numbers (at most 127 and a rounding)
// rounded to whole ones by adding 1.5 * 2^23, whose low byte is then the code.
// `off`: the largest distance to a whole number among them; halves, which the
// sum rounds to even and the format away from zero, have 0.5.
__device__ __forceinline__ uint32_t codes4(const float4 &t, float &off) {
    constexpr float kWhole = 12582912.0f;
    const float a = t.x + kWhole, b = t.y + kWhole, c = t.z + kWhole, d = t.w + kWhole;
    off = fmaxf(fmaxf(fabsf(t.x - (a - kWhole)), fabsf(t.y - (b - kWhole))),
                fmaxf(fabsf(t.z - (c - kWhole)), fabsf(t.w - (d - kWhole))));
    return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                       __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

// The same with halves away from zero, and clamped.
__device__ __forceinline__ uint32_t codes4_exact(const float4 &t) {
    return (uint32_t)(code(t.x) & 255) | (uint32_t)(code(t.y) & 255) << 8 |
           (uint32_t)(code(t.z) & 255) << 16 | (uint32_t)(code(t.w) & 255) << 24;
}

// Rows of up to 4 * T * V elements, 16-byte aligned: one CTA a row, which
// stays in registers from its one read to its codes.  Thread j holds float4
// j, j + T, ..., so 8 neighbouring threads hold a block and its maximum takes
// three shuffles.  What bounds it: the bytes for many rows (2048 x 4096 with a
// residual, 110 MB: 5.7 TB/s of the 6.8 a copy reaches), the launch and one
// row's chain of latencies for few (2.6 us for one).
template <int T, int V, bool BITNET>
__global__ void __launch_bounds__(T, V <= 2 ? 2048 / T : V == 6 ? 2 : 1)  // V <= 2: a full SM, at 32 registers
rms_norm_kernel(const NormArgs a, bool pdl) {
    __shared__ float s_part[2][T / 32];
    __shared__ int s_sum[T / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = blockIdx.x;
    const int k = (int)a.k;
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    auto at = [&](int e) { return 4 * (e * T + (int)threadIdx.x); };
    float4 h[V], w[V];
    const float *x = a.x + i * a.ldx;
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e)
        h[e] = at(e) < k ? *reinterpret_cast<const float4 *>(x + at(e)) : make_float4(0, 0, 0, 0);
    if (a.r) {
        const float *r = a.r + i * a.ldr;
        float4 q[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            q[e] = at(e) < k ? *reinterpret_cast<const float4 *>(r + at(e)) : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < V; ++e)
            h[e].x += q[e].x, h[e].y += q[e].y, h[e].z += q[e].z, h[e].w += q[e].w;
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        w[e] = at(e) < k ? __ldg(reinterpret_cast<const float4 *>(a.w + at(e))) : make_float4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        ss = fmaf(h[e].x, h[e].x, ss);
        ss = fmaf(h[e].y, h[e].y, ss);
        ss = fmaf(h[e].z, h[e].z, ss);
        ss = fmaf(h[e].w, h[e].w, ss);
    }
    ss = warp_sum(ss);
    if (lane == 0) s_part[0][warp] = ss;
    if (a.h) {
        float *out = a.h + i * a.ldh;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (at(e) < k) *reinterpret_cast<float4 *>(out + at(e)) = h[e];
    }
    __syncthreads();
    // every warp adds the warps' sums up in the same order
    const float inv = inverse_rms(warp_sum(lane < T / 32 ? s_part[0][lane] : 0.0f), a);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        h[e].x = (h[e].x * inv) * w[e].x;
        h[e].y = (h[e].y * inv) * w[e].y;
        h[e].z = (h[e].z * inv) * w[e].z;
        h[e].w = (h[e].w * inv) * w[e].w;
    }
    uint32_t *codes = reinterpret_cast<uint32_t *>(a.aq + i * a.k);
    if constexpr (!BITNET) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float m = fmaxf(fmaxf(fabsf(h[e].x), fabsf(h[e].y)), fmaxf(fabsf(h[e].z), fabsf(h[e].w)));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float d = __fdiv_rn(m, 127.0f);
            // The quotients by d's reciprocal differ from the IEEE ones by less
            // than 2^-15 (three roundings of a number up to 127), so they round
            // as those do unless one is that near to a half; only then (within
            // 2^-14), and for a d whose reciprocal leaves f32's normal range,
            // divide.
            uint32_t q = 0;
            float off = 1.0f;
            if (d >= 1e-37f) {
                const float r = __frcp_rn(d);
                q = codes4(make_float4(h[e].x * r, h[e].y * r, h[e].z * r, h[e].w * r), off);
            }
            if (off > 0.5f - 1.0f / 16384.0f)
                q = d != 0.0f ? codes4_exact(make_float4(__fdiv_rn(h[e].x, d), __fdiv_rn(h[e].y, d),
                                                         __fdiv_rn(h[e].z, d), __fdiv_rn(h[e].w, d)))
                              : 0;
            if (at(e) < k) {
                codes[at(e) / 4] = q;
                if (threadIdx.x % 8 == 0)
                    a.ad[i * (a.k / kQK) + at(e) / kQK] = __half_as_ushort(__float2half_rn(d));
            }
        }
    } else {
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e)
            amax = fmaxf(amax, fmaxf(fmaxf(fabsf(h[e].x), fabsf(h[e].y)), fmaxf(fabsf(h[e].z), fabsf(h[e].w))));
        amax = warp_max(amax);
        if (lane == 0) s_part[1][warp] = amax;
        __syncthreads();
        amax = warp_max(lane < T / 32 ? s_part[1][lane] : 0.0f);
        const float scale = amax != 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
        int sum = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            // a row of zeros has scale 0 and needs no case of its own
            const float4 t = make_float4(__fmul_rn(h[e].x, scale), __fmul_rn(h[e].y, scale),
                                         __fmul_rn(h[e].z, scale), __fmul_rn(h[e].w, scale));
            float off;
            uint32_t q = codes4(t, off);
            // 127 / amax overflows below 3.7e-37: the products are infinite
            // (NaN where y is 0), which only the exact codes clamp
            if (off >= 0.5f || scale > FLT_MAX) q = codes4_exact(t);
            if (at(e) < k) {
                codes[at(e) / 4] = q;
                sum = __dp4a((int)q, 0x01010101, sum);
            }
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w2 = 1; w2 < T / 32; ++w2) sum += s_sum[w2];
            a.scale[i] = scale;
            a.sum[i] = sum;
        }
    }
}

template <int T, int V>
cudaError_t launch_rows(const NormArgs &a, cudaStream_t s, bool pdl) {
    return launch_kernel(a.ad ? rms_norm_kernel<T, V, false> : rms_norm_kernel<T, V, true>,
                         dim3((unsigned)a.m), dim3(T), 0, s, pdl, a, pdl);
}

bool vectors(const void *p, int64_t ld) {
    return ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs &a, cudaStream_t s, bool pdl) {
    if (a.k <= 16384 && vectors(a.x, a.ldx) && (!a.r || vectors(a.r, a.ldr)) &&
        (!a.h || vectors(a.h, a.ldh)) && vectors(a.w, 0) && reinterpret_cast<uintptr_t>(a.aq) % 4 == 0) {
        // Short rows want few idle threads (16384 rows of 256: 11.6 us with 64
        // threads, 21.4 with 128), others as many CTAs a SM as the loads of a
        // row's two streams need to overlap the rows' barriers: 2048 rows of
        // 4096 take 19.3 us with 512 threads of two float4, 20.5 with 256 of
        // four, 24.2 with 128 of eight; 1024 rows of 8192 19.3 with 512 of four
        // (1024 of two: 21.6); 1024 of 11008 28.5 with 512 of six (1024 of
        // four: 34.4).
        if (a.k <= 256) return launch_rows<64, 1>(a, s, pdl);
        if (a.k <= 1024) return launch_rows<128, 2>(a, s, pdl);
        if (a.k <= 4096) return launch_rows<512, 2>(a, s, pdl);
        if (a.k <= 8192) return launch_rows<512, 4>(a, s, pdl);
        if (a.k <= 12288) return launch_rows<512, 6>(a, s, pdl);
        return launch_rows<1024, 4>(a, s, pdl);
    }
    return launch_kernel(a.ad ? rms_norm_rows_kernel<false> : rms_norm_rows_kernel<true>,
                         dim3((unsigned)a.m), dim3(kRowThreads), 0, s, pdl, a, pdl);
}

}  // namespace qmm
