// Exchange of partial results between the CTAs of a cluster, through their
// shared memory: asynchronous stores that an mbarrier of the receiver counts.
// The receiver waits for one store's way; with plain stores and a cluster
// barrier the senders wait for their stores' acknowledgements first (attention
// of 577 tokens: 4.8 us, 4.3 this way).
//
// The receiver opens its barrier with the bytes that it will get before the
// cluster's first barrier (arrive, and wait before the first store), and
// leaves only after they came, so no store finds its memory gone; a sender may
// leave at once.  The wait is bounded: after the limit of polls, each of which
// suspends for 20 us at most, it sets an error word (qmm_check_device_error)
// and, after waiting as long again for what is on its way, gives up.
#pragma once

#include <atomic>

#include "qmm_internal.h"

namespace qmm {
namespace {

__device__ unsigned int g_exchange_error = 0;  // of this translation unit's kernels
// Whether any of them was launched (or captured) with an exchange: else their
// error word is not read, which takes about 10 us of qmm_check_device_error.
std::atomic<bool> g_exchange_used{false};

__device__ __forceinline__ uint32_t shared_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ int cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return (int)r;
}

// One thread, before it arrives at the cluster's barrier.
__device__ __forceinline__ void exchange_open(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_addr(bar)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_addr(bar)), "r"(bytes)
                 : "memory");
}

// Shared memory of the cluster's CTA `rank` at the place of this CTA's `p`.
__device__ __forceinline__ uint32_t exchange_addr(const void *p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(shared_addr(p)), "r"(rank));
    return r;
}

// Stores of 8 and 16 bytes, `bar` of the same CTA as `dst`.
__device__ __forceinline__ void exchange_store(uint32_t dst, float x, float y, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(dst),
                 "f"(x), "f"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void exchange_store(uint32_t dst, uint64_t x, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(dst), "l"(x),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void exchange_store(uint32_t dst, float x, float y, float z, float w, uint32_t bar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
        "f"(x), "f"(y), "f"(z), "f"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ bool exchange_done(uint64_t *bar) {
    uint32_t done;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0, 20000;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done)
        : "r"(shared_addr(bar))
        : "memory");
    return done != 0;
}

// True once all bytes are in.
__device__ __forceinline__ bool exchange_wait(uint64_t *bar, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i)
        if (exchange_done(bar)) return true;
    atomicOr(&g_exchange_error, 1u);
    for (uint32_t i = 0; i < limit && !exchange_done(bar); ++i) {
    }
    return false;
}

cudaError_t exchange_read_and_clear_error(unsigned int *word, cudaStream_t s) {
    const unsigned int zero = 0;
    *word = 0;
    if (!g_exchange_used.load(std::memory_order_relaxed)) return cudaSuccess;
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_exchange_error, sizeof zero, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || !*word) return e;
    e = cudaMemcpyToSymbolAsync(g_exchange_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace
}  // namespace qmm
