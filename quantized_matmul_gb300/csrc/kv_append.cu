// Writes new tokens' keys and values into the paged cache, rounding each to
// the cache's type: fp16 to nearest even, or the Q8_0 recipe of
// qmm_quantize_act_q8_0 per 32 elements.
//
// One CTA a token (and a group of heads): x threads hold a head's row, four
// elements each, so eight threads hold a block and its maximum takes three
// shuffles; a thread has its key's and its value's loads in flight together.
// Bound by the bytes (8 read, 4 or 2.125 written an element pair) for many
// tokens (2048 tokens of 8 heads of 128, f16: 3.8 us with rows that L2 still
// holds, as behind the projection that wrote them; 5.9 us, 4.3 TB/s, from HBM;
// Q8_0 7.6 us from HBM) and by the launch for a few (16 tokens, Q8_0: 2.0 us).
// With the key and the value one after the other and divisions it took 8.0 us
// for the 2048 of L2.
#include "kvcache.cuh"

namespace qmm {
namespace {

constexpr int kAppendThreads = 256;

template <bool Q8, bool VEC>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const KvAppendArgs a) {
    pdl_launch_dependents();
    pdl_wait();  // nothing is read or written before the predecessor's end
    const int64_t i = blockIdx.x;
    const int64_t head = (int64_t)blockIdx.y * blockDim.y + threadIdx.y;
    if (head >= a.kv_heads) return;  // rows of threads, whole groups of 8
    const int64_t slot = a.slots[i];
    if (slot < 0 || slot >= a.num_pages * a.page_size) return;
    // slot / page_size by its reciprocal rounded up in 64 bits: both are below 2^32
    const int64_t page = a.page_size > 1 ? (int64_t)__umul64hi((uint64_t)slot, a.page_mul) : slot;
    const int64_t row = (page * a.kv_heads + head) * a.page_size + (slot - page * a.page_size);
    const int j = 4 * threadIdx.x;
    const float *from[2] = {a.k + i * a.ldk + head * a.d + j, a.v + i * a.ldv + head * a.d + j};
    float4 x[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
        x[c] = VEC ? *reinterpret_cast<const float4 *>(from[c])
                   : make_float4(from[c][0], from[c][1], from[c][2], from[c][3]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float4 f = x[c];
        void *plane = c ? a.vc : a.kc;
        if constexpr (!Q8) {
            const __half2 lo = __floats2half2_rn(f.x, f.y), hi = __floats2half2_rn(f.z, f.w);
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(plane) + row * a.d + j) = make_uint2(
                reinterpret_cast<const uint32_t &>(lo), reinterpret_cast<const uint32_t &>(hi));
        } else {
            float amax = fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w)));
            const unsigned thread = threadIdx.y * blockDim.x + threadIdx.x;
            const unsigned group = 0xffu << (thread & 24);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
            const float d = __fdiv_rn(amax, 127.0f);
            auto code = [&](float v) {
                return d != 0.0f ? (int)fminf(fmaxf(roundf(__fdiv_rn(v, d)), -127.0f), 127.0f) : 0;
            };
            *reinterpret_cast<char4 *>(static_cast<int8_t *>(plane) + row * a.d + j) =
                make_char4((signed char)code(f.x), (signed char)code(f.y), (signed char)code(f.z),
                           (signed char)code(f.w));
            if ((threadIdx.x & 7) == 0)
                (c ? a.vd : a.kd)[row * (a.d / kQK) + j / kQK] = __half_as_ushort(__float2half_rn(d));
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &args, cudaStream_t s) {
    KvAppendArgs a = args;
    a.page_mul = ~(uint64_t)0 / (uint64_t)a.page_size + 1;
    const int across = (int)a.d / 4;  // 8 .. 64
    const int64_t fit = kAppendThreads / across, rows = a.kv_heads < fit ? a.kv_heads : fit;
    const dim3 block((unsigned)across, (unsigned)rows);
    const dim3 grid((unsigned)a.m, (unsigned)((a.kv_heads + rows - 1) / rows));
    const bool vec = a.ldk % 4 == 0 && a.ldv % 4 == 0 && reinterpret_cast<uintptr_t>(a.k) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.v) % 16 == 0;
    auto *kernel = a.kd ? (vec ? kv_append_kernel<true, true> : kv_append_kernel<true, false>)
                        : (vec ? kv_append_kernel<false, true> : kv_append_kernel<false, false>);
    return launch_kernel(kernel, grid, block, 0, s, true, a);
}

}  // namespace qmm
