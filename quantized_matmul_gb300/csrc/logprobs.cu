// Log probabilities of given words, the entropy and the most probable words
// of each row of logits, in one pass over the row.
//
// With M = max_j x_j and z_j = x_j - M (z <= 0), Z = sum_j exp(z_j):
//   log p_j = z_j - log Z,   H = log Z - (sum_j exp(z_j) z_j) / Z.
// The running state of any part of a row is (m, s, t): its maximum, the sum
// of exp(x - m), and the sum of exp(x - m) (x - m) log2(e).  It is taken to a
// larger maximum m' by d = (m - m') log2(e), f = 2^d: (m', s f, t f + s f d).
// Parts join in a fixed order, so the results do not vary between runs.  A NaN
// anywhere makes s NaN.
//
// Z is 1 + r, r the sum without one element that attains the maximum, and
// log Z = log1p(r): so both terms of H are >= 0 and nothing cancels.  Where a
// word is nearly certain (Z < 1 + 2^-6), s - 1 would have lost r's digits:
// then r is summed again without that element (the other threads' sums are
// exact enough; the one thread that has it looks at its elements again), so a
// log probability near 0 keeps its relative precision.
//
// Many rows are bound by the bytes (512 rows of 128256 logits, f32, 8
// alternatives: 47 us, 5.6 TB/s): all 512 CTAs are resident at once, three or
// four a SM, and reach their tails together.  Two, four and eight CTAs a row
// would spread them evenly, but their tails cost more than that gives (1.04,
// 1.1 and 1.4 times as long).  Few rows are bound by latency: one row takes 6.4
// us with 20 alternatives, most of it the chain of barriers, shuffles and the
// cluster's exchange behind a read of 1.3 us.  Code that runs once counts
// there, so loops that are rarely taken stay rolled.
//
// Packed f32 pairs halve the sums' instructions.
//
// The alternatives are ordered by a 64-bit key: the value's bits mapped to an
// ordered integer (NaN above +inf, -0 equal to +0), then the lower index.
// Keys are unique, so ranks are too: a key's rank is the number of larger
// ones, counted by eight lanes.  They cost the pass over the row nothing: a
// thread knows its own maximum at the end, the top_k-th largest of the maxima
// of 64 groups of threads bounds the top_k-th largest element from below, and
// only threads that reach that bound look at elements again (about top_k of
// them): at those of the chunk that gave the maximum, or where a second chunk
// reaches the bound at all of them, a warp for each such thread.  What passes goes to a
// list, which is ranked.  Where more elements reach the bound than the list
// holds, as under a mask that leaves fewer than top_k words, only those above
// it are ranked, and of those that equal it the first are taken in the row's
// order.  (Should even those above it be too many, which takes a row laid out
// for it, the keys are taken one after the other.)
//
// Each thread copies what it will read itself, asynchronously, two chunks
// ahead, so the copies need no barrier.
#include <climits>

#include "exchange.cuh"

namespace qmm {
namespace {

constexpr int T = 256;       // threads
constexpr int kE = 16;       // elements a thread holds of a chunk
constexpr int kTop = 32;     // the most alternatives
constexpr int kList = 512;   // elements that may reach the bound
constexpr int kGroups = 64;  // groups of threads whose maxima give it
constexpr int kCrowd = 128;  // threads that reach the bound: more is taken as crowded
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct State {
    float m, s, t;  // s: r once a CTA's part is complete
};

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Signed-integer order of floats; -0 counts as +0, every NaN as the largest.
__device__ __forceinline__ int ordered(float v) {
    const int b = __float_as_int(v + 0.0f);
    if (v != v) return 0x7fffffff;
    return b ^ ((b >> 31) & 0x7fffffff);
}

__device__ __forceinline__ float from_ordered(int o) {
    return __int_as_float(o ^ ((o >> 31) & 0x7fffffff));
}

// Larger key = earlier alternative; 0 is below every key of an element.
__device__ __forceinline__ uint64_t make_key(int ord, uint32_t index) {
    return ((uint64_t)((uint32_t)ord ^ 0x80000000u) << 32) | (uint32_t)~index;
}

// The first k of `count` keys, in order, to `out`; zeros are no keys, and
// follow the last one to a multiple of 32.  Eight lanes count the larger ones
// of a key.  Whole CTA, no barrier inside.
__device__ __forceinline__ void rank_keys(const uint64_t *keys, int count, uint64_t *out, int k) {
    for (int i = threadIdx.x >> 3; i < (count + 31) / 32 * 32; i += T / 8) {
        const uint64_t key = keys[i];
        int larger = 0;
        for (int j = threadIdx.x & 7; j < count; j += 32)
#pragma unroll
            for (int u = 0; u < 32; u += 8) larger += keys[j + u] > key;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) larger += __shfl_xor_sync(0xffffffffu, larger, o);
        if (key != 0 && larger < k && (threadIdx.x & 7) == 0) out[larger] = key;
    }
}

// The states of each N lanes of a warp, joined (all lanes hold the same N):
// every lane is taken to the largest maximum at once, then two sums.  REST: s
// is r, and one of the lanes at the maximum keeps standing for it.
template <bool REST, int N>
__device__ __forceinline__ State join_warp(const State &st) {
    const float m = from_ordered(__reduce_max_sync(0xffffffffu, ordered(st.m)));
    const bool top = st.m == m;
    // 2^-300 is 0 in f32, so the clamp only keeps 0 * inf out
    const float d = top ? 0.0f : fmaxf((st.m - m) * kLog2e, -300.0f), f = exp2_approx(d);
    float s = (REST ? 1.0f + st.s : st.s) * f;
    float t = fmaf(s, d, f * st.t);
    if (REST && top) s = st.s;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if (REST) {
        const int tops = __popc(__ballot_sync(0xffffffffu, top) & (N < 32 ? (1u << N % 32) - 1 : 0xffffffffu));
        if (m != -INFINITY) s += (float)(tops - 1);
    }
    return {m, s, t};
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Packed f32 pairs.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <bool VEC>
__device__ __forceinline__ void copy_async(uint32_t dst, const float *src) {
    if (VEC)
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int kStages, bool VEC>
__global__ void __launch_bounds__(T, 4)
log_probs_kernel(const LogProbsArgs a, int64_t slice) {
    constexpr int kChunk = T * kE, kGroup = T / kGroups;
    __shared__ uint64_t s_list[kList];
    __shared__ __align__(16) int s_group[kGroups];
    __shared__ uint64_t s_best[kTop];
    __shared__ uint64_t s_all[kMaxCluster * kTop];  // every CTA's best, in the first CTA
    __shared__ float4 s_parts[kMaxCluster];         // and state
    __shared__ uint64_t s_arrived;                  // counts both
    __shared__ State s_state[T / 32], s_row;
    __shared__ uint64_t s_key[T / 32];
    __shared__ float s_rest[T / 32];
    __shared__ uint16_t s_pass[T];
    __shared__ int s_count, s_passing, s_bound;
    // (aligned to 16 alone it may be filled slower: 512 x 128256: 51 us for 47)
    extern __shared__ __align__(128) float4 s_chunk[];  // [stage][kE / 4][T], each thread's own

    const int rank = cluster_rank(), ranks = cluster_size();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / ranks;
    const float *x = a.logits + row * a.ldl;
    const int k = a.top_k;
    // this CTA's slice; indices below are relative to it
    const int64_t lo = rank * slice;
    const int size = (int)(lo >= a.n ? 0 : lo + slice < a.n ? slice : a.n - lo);
    const float *xs = x + lo;

    auto place = [&](int base, int e) {
        return VEC ? base + (e / 4) * (T * 4) + (int)threadIdx.x * 4 + e % 4
                   : base + e * T + (int)threadIdx.x;
    };
    // a stage's bytes, and where this thread's own begin
    constexpr int kStage = kChunk * 4;
    const uint32_t mine_at = (uint32_t)__cvta_generic_to_shared(s_chunk + threadIdx.x);
    const float *mine_from = xs + place(0, 0);
    auto fetch = [&](int base, int stage) {
        const uint32_t to = mine_at + stage * kStage;
        const float *from = mine_from + base;
        if (size - base >= kChunk) {
#pragma unroll
            for (int e = 0; e < kE; e += VEC ? 4 : 1)
                copy_async<VEC>(to + e / 4 * T * 16 + e % 4 * 4, from + e * T);
        } else {
#pragma unroll
            for (int e = 0; e < kE; e += VEC ? 4 : 1)
                if (place(base, e) + (VEC ? 3 : 0) < size)
                    copy_async<VEC>(to + e / 4 * T * 16 + e % 4 * 4, from + e * T);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (ranks > 1) {
        if (rank == 0 && threadIdx.x == 0) exchange_open(&s_arrived, (uint32_t)(ranks * (16 + 8 * k)));
        cluster_arrive_relaxed();  // waited for before the first store to another CTA
    }
    // The next grid may take its SMs early only where this one leaves most of
    // them: its CTAs would crowd on what is free (64 rows: 14 us against 11).
    if (kStages > 3) pdl_launch_dependents();
    pdl_wait();  // nothing is read or written before the predecessor's end
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i * kChunk, i);

    // the given words' logits, early
    int32_t word = -1;
    float word_x = 0.0f;
    if (rank == 0 && threadIdx.x < a.n_tokens) {
        word = a.tokens[row * a.n_tokens + threadIdx.x];
        if (word >= 0 && word < a.n) word_x = x[word];
    }
    if (threadIdx.x < kTop) s_best[threadIdx.x] = 0;
    if (k > 0)
        for (int i = threadIdx.x; i < kList; i += T) s_list[i] = 0;
    if (threadIdx.x == 0) s_count = s_passing = 0, s_bound = INT_MAX;
    int stage = 0;
    State st{-INFINITY, 0.0f, 0.0f};

    float v[kE];
    // waits for the thread's own copies of this chunk and asks for a later one
    auto load = [&](int base) {
        fetch(base <= size - (kStages - 1) * kChunk ? base + (kStages - 1) * kChunk : size,
              stage == 0 ? kStages - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        const float4 *from = s_chunk + stage * (kE / 4) * T + threadIdx.x;
#pragma unroll
        for (int e = 0; e < kE; e += 4) {
            const float4 q = from[e / 4 * T];
            v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
        }
        if (size - base < kChunk) {
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                if (place(base, e) >= size) v[e] = -INFINITY;
                // a vector that the slice ends in was not copied
                else if (VEC && place(base, e) - e % 4 + 3 >= size) v[e] = xs[place(base, e)];
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    };
    constexpr int kWide = VEC ? 4 : 1, kLoads = kE / kWide;  // elements of a load, loads of a chunk
    auto key_at = [&](float value, int at) { return make_key(ordered(value), (uint32_t)(lo + at)); };

    // the thread's j-th load: four neighbours, or one element
    auto again = [&](int thread, int j, float (&q)[4]) {
        const int at = (j * T + thread) * (VEC ? 4 : 1);
        if (VEC && at + 3 < size) {
            const float4 w = size <= kStages * kChunk  // every chunk is still in shared memory
                                 ? s_chunk[j * T + thread]
                                 : *reinterpret_cast<const float4 *>(xs + at);
            q[0] = w.x, q[1] = w.y, q[2] = w.z, q[3] = w.w;
        } else {
#pragma unroll
            for (int e = 0; e < (VEC ? 4 : 1); ++e) q[e] = at + e < size ? xs[at + e] : 0.0f;
        }
        return at;
    };

    const State none{-INFINITY, 0.0f, 0.0f};
    // the chunk that has the thread's maximum, and the largest of the others'
    int top_chunk = 0;
    float second = -INFINITY;
    uint64_t s2 = 0, t2 = 0;
    for (int base = 0; base < size; base += kChunk) {
        load(base);
        float mc = v[0];
#pragma unroll
        for (int e = 1; e < kE; ++e) mc = fmaxf(mc, v[e]);  // a NaN does not pass, but stays in v
        second = fmaxf(second, fminf(mc, st.m));
        if (mc > st.m) {
            top_chunk = base;
            if (st.m != -INFINITY) {
                const float d = fmaxf((st.m - mc) * kLog2e, -300.0f), f = exp2_approx(d);
                s2 = mul2(s2, pair(f, f));
                t2 = fma2(s2, pair(d, d), mul2(t2, pair(f, f)));
            }
            st.m = mc;
        }
        const float from = st.m == -INFINITY ? 0.0f : -st.m;
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
            const uint64_t z2 = mul2(add2(pair(v[e], v[e + 1]), pair(from, from)), pair(kLog2e, kLog2e));
            const float2 z = split(z2);
            const uint64_t p2 = pair(exp2_approx(z.x), exp2_approx(z.y));
            s2 = add2(s2, p2);
            t2 = fma2(p2, pair(fmaxf(z.x, -300.0f), fmaxf(z.y, -300.0f)), t2);
        }
    }
    st.s = split(s2).x + split(s2).y;
    st.t = split(t2).x + split(t2).y;

    const State mine = st;
    st = join_warp<false, 32>(st);
    if (lane == 0) s_state[warp] = st;
    int own = 0, next = 0, most = 0;
    if (k > 0) {
        // the thread's largest element; a NaN above all (s is NaN for +inf too)
        bool nan = false;
        if (mine.s != mine.s)
            for (int j = 0; (j * T + (int)threadIdx.x) * (VEC ? 4 : 1) < size; ++j) {
                float q[4];
                again(threadIdx.x, j, q);
#pragma unroll
                for (int e = 0; e < (VEC ? 4 : 1); ++e) nan |= q[e] != q[e];
            }
        own = nan ? INT_MAX : ordered(mine.m);
        next = nan ? INT_MAX : ordered(second);
        most = own;
#pragma unroll
        for (int o = 1; o < kGroup; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (threadIdx.x % kGroup == 0) s_group[threadIdx.x / kGroup] = most;
    }
    __syncthreads();
    st = join_warp<false, T / 32>(s_state[lane % (T / 32)]);
    if (k > 0) {
        // the smallest of the k largest group maxima: a group's threads count
        // a part of the larger ones each
        int larger = 0;
        constexpr int kPart = kGroups / kGroup;
#pragma unroll
        for (int j = 0; j < kPart; j += 4) {
            const int4 q = *reinterpret_cast<const int4 *>(s_group + threadIdx.x % kGroup * kPart + j);
            larger += (q.x > most) + (q.y > most) + (q.z > most) + (q.w > most);
        }
#pragma unroll
        for (int o = 1; o < kGroup; o <<= 1) larger += __shfl_xor_sync(0xffffffffu, larger, o);
        const int least = __reduce_min_sync(0xffffffffu, larger < k ? most : INT_MAX);
        if (lane == 0) atomicMin(&s_bound, least);
        __syncthreads();
        const int bound = s_bound;
        // Lists the elements of at least `least` and returns their number
        // (more than the list holds where the threads alone are a crowd).
        auto collect = [&](int least, int crowd) {
            if (__syncthreads_count(own >= least) > crowd) return kList + 1;
            const float floor = from_ordered(least);  // NaN where only NaN reaches it
            // of the elements that start at `first`, kWide neighbours in each
            // load of the CTA's, those of a mask
            auto list = [&](unsigned passes, int first) {
                for (; passes; passes &= passes - 1) {
                    const int e = __ffs(passes) - 1, at = first + e / kWide * (T * kWide) + e % kWide;
                    if (at >= size) break;
                    const float value = VEC && size <= kStages * kChunk && (at | 3) < size
                                            ? reinterpret_cast<const float *>(s_chunk)[at]
                                            : xs[at];
                    const int c = atomicAdd(&s_count, 1);
                    if (c < kList) s_list[c] = key_at(value, at);
                }
            };
            // (a thread with a NaN is none of the first kind)
            const bool one = own >= least && next < least, all = own >= least && next >= least;
            if (one) {
                float q[kLoads][4];
                unsigned passes = 0;
#pragma unroll
                for (int e = 0; e < kLoads; ++e) again(threadIdx.x, top_chunk / kChunk * kLoads + e, q[e]);
#pragma unroll
                for (int e = 0; e < kE; ++e) passes |= q[e / kWide][e % kWide] >= floor ? 1u << e : 0u;
                list(passes, place(top_chunk, 0));
            } else if (all) {
                s_pass[atomicAdd(&s_passing, 1)] = (uint16_t)threadIdx.x;
            }
            if (__syncthreads_or(all)) {
                const int passing = s_passing;
                for (int i = warp; i < passing; i += T / 32) {
                    const int thread = s_pass[i];
                    for (int j = lane; (j * T + thread) * kWide < size; j += 32) {
                        float q[4];
                        const int at = again(thread, j, q);
                        unsigned passes = 0;
#pragma unroll
                        for (int f = 0; f < kWide; ++f)
                            passes |= q[f] >= floor || q[f] != q[f] ? 1u << f : 0u;
                        list(passes, at);
                    }
                }
                __syncthreads();
            }
            return s_count;
        };
        int found = collect(bound, kCrowd);
        const bool crowded = found > kList;
        if (crowded) {
            __syncthreads();
            if (threadIdx.x == 0) s_count = s_passing = 0;
            for (int i = threadIdx.x; i < kList; i += T) s_list[i] = 0;
            __syncthreads();
            found = bound != INT_MAX ? collect(bound + 1, T) : 0;
        }
        if (found <= kList) {
            rank_keys(s_list, found, s_best, k);
            // in the row's order, those that equal the bound
            for (int at = (int)threadIdx.x; crowded && found < k; at += T) {
                const bool equal = at < size && ordered(xs[at]) == bound;
                const unsigned lanes = __ballot_sync(0xffffffffu, equal);
                if (lane == 0) s_key[warp] = __popc(lanes);
                __syncthreads();
                int before = found;
                for (int w = 0; w < T / 32; ++w) {
                    if (w == warp) before = found + __popc(lanes & ((1u << lane) - 1));
                    found += (int)s_key[w];
                }
                if (equal && before < k) s_best[before] = key_at(xs[at], at);
                __syncthreads();
            }
        } else {
            // one key after the other: each thread offers its largest below the last
            uint64_t last = ~(uint64_t)0;
            for (int i = 0; i < k; ++i) {
                uint64_t key = 0;
                if (own >= bound)
                    for (int at = (int)threadIdx.x * (VEC ? 4 : 1); at < size;
                         at += VEC && at % 4 != 3 ? 1 : VEC ? 4 * T - 3 : T) {
                        const uint64_t other = key_at(xs[at], at);
                        if (other < last && other > key) key = other;
                    }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
                    key = other > key ? other : key;
                }
                if (lane == 0) s_key[warp] = key;
                __syncthreads();
                for (int w = 0; w < T / 32; ++w) key = s_key[w] > key ? s_key[w] : key;
                last = key;
                if (threadIdx.x == 0) s_best[i] = key;
                if (key == 0) break;
                __syncthreads();
            }
        }
    }

    if (st.s >= 0.5f && st.s < 1.0f + 1.0f / 64.0f) {
        // a nearly certain word: the sum without it (the one thread at the
        // maximum has it, else the sum would be 2 at least)
        float rest = mine.m == st.m ? 0.0f : mine.s * exp2_approx((mine.m - st.m) * kLog2e);
        const unsigned tops = __ballot_sync(0xffffffffu, mine.m == st.m);
        if (tops) {
            const int thread = 32 * warp + __ffs(tops) - 1;
            for (int j = lane; (j * T + thread) * (VEC ? 4 : 1) < size; j += 32) {
                float q[4];
                const int at = again(thread, j, q);
#pragma unroll
                for (int e = 0; e < (VEC ? 4 : 1); ++e)
                    if (at + e < size && q[e] != st.m) rest += exp2_approx((q[e] - st.m) * kLog2e);
            }
        }
        rest = warp_sum(rest);
        if (lane == 0) s_rest[warp] = rest;
        __syncthreads();
        st.s = warp_sum(lane < T / 32 ? s_rest[lane] : 0.0f);
    } else if (st.m != -INFINITY) {
        st.s -= 1.0f;
    }
    if (threadIdx.x == 0 && ranks == 1) s_row = st;
    if (ranks > 1) {
        __syncthreads();  // s_best is complete, s_list read
        s_list[threadIdx.x] = 0;
        if (threadIdx.x == 0) s_count = 0;
        cluster_wait();
        if (!a.withhold) {
            const uint32_t arrived = exchange_addr(&s_arrived, 0);
            if (threadIdx.x == T - 1) exchange_store(exchange_addr(&s_parts[rank], 0), st.m, st.s, st.t, 0.0f, arrived);
            if (threadIdx.x < k)
                exchange_store(exchange_addr(&s_all[rank * kTop + threadIdx.x], 0), s_best[threadIdx.x], arrived);
        }
        if (kStages <= 3) pdl_launch_dependents();
        if (rank != 0) return;
        // The list and its count are empty before any warp adds to them: the
        // bytes that end the wait may come while a warp is still before its
        // reset.  (The barrier's time passes beside the exchange's.)
        __syncthreads();
        if (!exchange_wait(&s_arrived, a.wait_limit)) return;
        if (warp == 0) {
            const float4 part = s_parts[lane % kMaxCluster];
            st = join_warp<true, kMaxCluster>(lane % kMaxCluster < ranks ? State{part.x, part.y, part.z} : none);
            if (lane == 0) s_row = st;
        }
        if (k > 0) {
            // every CTA's list is sorted: what `ranks` lists have at place
            // ceil(k / ranks) - 1 or before is k keys at least
            const int place = (k + ranks - 1) / ranks - 1;
            uint64_t bound = ~(uint64_t)0;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) {
                const uint64_t key = s_all[min(c, ranks - 1) * kTop + place];
                bound = key < bound ? key : bound;
            }
            if (warp < ranks && lane < k) {
                const uint64_t key = s_all[warp * kTop + lane];
                if (key >= bound) s_list[atomicAdd(&s_count, 1)] = key;
            }
            __syncthreads();
            rank_keys(s_list, s_count, s_best, k);
        }
    }
    __syncthreads();
    st = s_row;
    // A row that has an infinite or NaN logit has no distribution (NaN); a row
    // of -inf alone has none to give either: every log probability is -inf
    // there and the entropy 0.
    const bool bad = st.m == INFINITY || st.s != st.s, empty = st.m == -INFINITY;
    const float log_z = log1pf(st.s);
    auto log_prob = [&](float v) {
        return bad ? NAN : empty ? -INFINITY : (v - st.m) - log_z;
    };
    if (threadIdx.x == 0 && a.entropy)
        a.entropy[row] = bad ? NAN : empty ? 0.0f : log_z - __fdiv_rn(st.t * (1.0f / kLog2e), 1.0f + st.s);
    if (threadIdx.x < k) {
        const uint64_t key = s_best[threadIdx.x];
        a.top_ids[row * k + threadIdx.x] = (int32_t)~(uint32_t)key;
        a.top_lp[row * k + threadIdx.x] =
            log_prob(from_ordered((int)((uint32_t)(key >> 32) ^ 0x80000000u)));
    }
    for (int64_t j = threadIdx.x; j < a.n_tokens; j += T) {
        if (j >= T) {
            word = a.tokens[row * a.n_tokens + j];
            if (word >= 0 && word < a.n) word_x = x[word];
        }
        a.token_lp[row * a.n_tokens + j] = word >= 0 && word < a.n ? log_prob(word_x) : -INFINITY;
    }
}

template <int kStages, bool VEC>
cudaError_t launch(const LogProbsArgs &a, int ranks, cudaStream_t s) {
    constexpr int kBytes = kStages * T * kE * 4;
    static std::atomic<uint64_t> opted_in;  // devices whose shared-memory limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!(opted_in.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(log_probs_kernel<kStages, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kBytes);
        if (e != cudaSuccess) return e;
        opted_in.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
    }
    const int64_t slice = ((a.n + ranks - 1) / ranks + 3) / 4 * 4;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ranks, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.m * ranks));
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    if (ranks > 1) g_exchange_used.store(true, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, log_probs_kernel<kStages, VEC>, a, slice);
}

}  // namespace

cudaError_t launch_log_probs(const LogProbsArgs &a, cudaStream_t s) {
    const bool vec = a.ldl % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    // as many CTAs a row as give every SM work, each with a chunk at least;
    // few rows: every chunk of a slice on its way at once
    const int64_t sms = device_sm_count();
    const int64_t chunks = (a.n + T * kE - 1) / (T * kE);
    int ranks = 1;
    while (ranks < kMaxCluster && ranks * 2 <= chunks && a.m * ranks < sms) ranks *= 2;
    if (a.m * ranks <= sms) return vec ? launch<5, true>(a, ranks, s) : launch<5, false>(a, ranks, s);
    return vec ? launch<3, true>(a, ranks, s) : launch<3, false>(a, ranks, s);
}

cudaError_t log_probs_read_and_clear_error(unsigned int *word, cudaStream_t s) {
    return exchange_read_and_clear_error(word, s);
}

}  // namespace qmm
