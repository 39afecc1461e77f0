// Attention of one new token over the paged key-value cache (attend_f16.cu
// and attend_q8.cu instantiate it for the two cache types).
//
//   s_j = scale * q . k_j,  out = sum_j exp(s_j - M) v_j / sum_j exp(s_j - M),
//   lse = M + log(sum_j exp(s_j - M)),  j over the sequence's attended tokens.
//
// The bytes bound it: every key and value is read once for all the query
// heads that share it (4 or 8 in one tile), and 4 operations a value and head
// are far below what the tensor cores take.  So each warp streams tiles of
// tokens through a ring of its own in shared memory, filled by 16-byte
// asynchronous copies and drained by the warp-level MMA (m16n8k16, f16
// operands, f32 accumulators), with no barrier between warps.  A copy of a
// token that is not attended to reads nothing and fills in zeros, so what the
// cache holds there never enters the arithmetic.
//
// Measured (32 query and 8 key heads of 128): 131067 tokens f16 in 88 us (6.1
// TB/s; the copies alone take as long), 64 ragged sequences of up to 4096
// tokens Q8_0 in 63 us (4.7 TB/s; the copies alone take 54; issue is at 61% and
// DRAM at 60%: half of the CTAs are empty, and 16 warps a SM hide neither the
// loads nor the chain from codes to f16 to products), 577 tokens f16 in 4.2 us.
// Copying each row in bulk, one instruction a row counted by an mbarrier, in
// place of 16 bytes a lane took 101 us, and 6.1 for the 577.
//
// Precision: q and the softmax weights are f32, the cache's values are exact
// in f16 (int8 codes too).  Each f32 factor enters the MMA as two f16 numbers
// hi + lo, hi = f16(f), lo = f16(f - hi), which keep 22 bits (of a weight at
// least 2^-36 of the largest); a third part would take columns of B from other
// heads, and the outputs' errors are 3e-7 to 9e-7 of 64 bits as it is, a plain
// f32 form's 4e-7 to 1.8e-6.  The cache is the MMA's A operand (16 tokens for
// the scores, 16 elements of the values for the output); the 8 columns of B are
// 4 heads' hi and lo in turn, so a lane's two neighbouring accumulators add up
// to a head's product.  The MMA sums one tile's tokens, f32 additions the tiles.
// Powers of two keep both in f16's range: a head's q is scaled to its largest
// element, the weights by 2^11.
//
// The softmax's base need not be the running maximum: weights up to 2^4 fit,
// so the base (and with it the outputs so far) moves only when a score passes
// it by more than 4 binary orders, which costs a warp one vote a tile.
//
// Q8_0: a score takes a block's product times the key's scale, block after
// block.  A value's scale d multiplies the weight's halves: hi = f16(w_hi d),
// lo = f16(w_lo d + (w_hi d - hi)), the bracket exact by a fused multiply-add.
// That takes scales of 2^-14 to 1 (or, times 2^10, up to 2^-10); tiles with
// others form the product in f32 and give each block and head a power of two of
// its own (64 ragged sequences with scales of 0.02 and 60 in a token: 72 us
// against 63).
#pragma once

#include <type_traits>

#include "exchange.cuh"
#include "kvcache.cuh"

namespace qmm {
namespace {

constexpr int kMaxCluster = 8;

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint4 &a, const uint2 &b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y));
}

// the same on accumulators of zero
__device__ __forceinline__ void mma_16816_first(float (&c)[4], const uint4 &a, const uint2 &b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "f"(0.0f));
}

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float exp2i(int e) {  // -126 .. 127
    return __int_as_float((127 + e) << 23);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(h);
}

// {a, b} as two f16 pairs: hi, and the rest of each
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 back = __half22float2(h);
    hi = reinterpret_cast<const uint32_t &>(h);
    lo = pack_half2(a - back.x, b - back.y);
}

// On f16 pairs: a weight's lo half, lo = w_lo d + (w_hi d - f16(w_hi d)); with
// (0, w_hi) in place of (w_hi, w_lo) its hi half.
__device__ __forceinline__ uint32_t scale_half(uint32_t w_hi, uint32_t w_lo, uint32_t d) {
    const __half2 h = reinterpret_cast<const __half2 &>(w_hi), f = reinterpret_cast<const __half2 &>(d);
    const __half2 rest = __hfma2(h, f, __hneg2(__hmul2(h, f)));
    const __half2 out = __hfma2(reinterpret_cast<const __half2 &>(w_lo), f, rest);
    return reinterpret_cast<const uint32_t &>(out);
}

// element b (mod 2) of an f16 pair
__device__ __forceinline__ float half_of(uint32_t pair, int b) {
    return __half2float(__ushort_as_half((unsigned short)(b & 1 ? pair >> 16 : pair)));
}

// f16 pairs of biased bytes: 0x6400 | u is 1024 + u, u = code + 128
__device__ __forceinline__ uint32_t bytes_to_half2(uint32_t bytes, uint32_t selector) {
    const uint32_t w = __byte_perm(bytes, 0x64646464u, selector);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 h = __hsub2(reinterpret_cast<const __half2 &>(w), bias);
    return reinterpret_cast<const uint32_t &>(h);
}

// Asynchronous copies of N bytes; `bytes` of them are read, the rest is zeros.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int bytes) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                     "r"(bytes)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes),
                     "n"(N)
                     : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool TRANS>
__device__ __forceinline__ uint4 load_matrices(uint32_t addr) {
    uint4 v;
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(addr)
                     : "memory");
    return v;
}

// One stage of a warp's ring: a tile of kTokens tokens' keys, values, scales
// and row numbers.
template <int NB, bool Q8, int NT>
struct Tile {
    static constexpr int kD = NB * 32;
    static constexpr int kWarps = 4;
    static constexpr int kSub = kD <= 64 ? 2 : 1;               // 16-token steps of a tile
    static constexpr int kTokens = 16 * kSub;
    static constexpr int kHeads = 4 * NT;                       // query heads, 4 for each B tile
    static constexpr int kRowsOut = kD / 16;                    // 16-element tiles of the output
    static constexpr float kLift = 2048.0f;                     // weights up to 2^4 stay below 2^15
    static constexpr int kRowBytes = kD * (Q8 ? 1 : 2);
    // Row strides: f16 rows are an odd number of 16-byte units apart, which
    // keeps the fragment loads free of bank conflicts; Q8_0 rows an odd number
    // of 32-byte blocks, which does so for the keys (the values' loads of 4
    // bytes a lane take two turns; permuting the blocks by row instead takes
    // more address arithmetic than that costs).
    static constexpr int kStride = Q8 ? 32 * (NB | 1) : kRowBytes + 16;
    static constexpr int kPlane = kTokens * kStride;
    // NB scales of 2 bytes, copied in words that cover them
    static constexpr int kScaleWords = Q8 ? (NB + 1) / 2 : 0;
    static constexpr int kScales = kTokens * kScaleWords * 4;
    static constexpr int kRows = 2 * kPlane + 2 * kScales;
    static constexpr int kBytes = kRows + kTokens * 4;
    // CTAs a SM: as many as registers allow where each ring has two stages at
    // least (of the SM's 228 KB, 1 KB a CTA is reserved)
    static constexpr int kQuery = 2 * NB * NT * 256;
    static constexpr int stages(int ctas) {
        return (228 * 1024 / ctas - 1024 - 512 - kQuery) / (kWarps * kBytes);
    }
    static constexpr int kCtas = Q8 && kD <= 128 ? (NT == 1 ? 4 : 3) : stages(2) >= 2 ? 2 : 1;
    static constexpr int kStages = stages(kCtas) < 4 ? stages(kCtas) : 4;
    static constexpr int kRing = kWarps * kStages * kBytes;
    static_assert(kBytes % 16 == 0 && kStages >= 2, "");
    static_assert(kRing >= kWarps * kHeads * kD * 4, "the outputs are joined in the ring");
    static constexpr int kClusterParts = (kHeads * kD + 4 * kMaxCluster) * 4;  // behind the ring, in a cluster

    // offset of 16-byte unit `unit` of a row
    static __device__ __forceinline__ int offset(int row, int unit) {
        return row * kStride + unit * 16;
    }

    // token i (0, 1) of step s of this lane's scores, and token i (0..3) of its weights
    static __device__ __forceinline__ int score_token(int s, int i, int g) { return 16 * s + 8 * i + g; }
    static __device__ __forceinline__ int weight_token(int s, int i, int t) {
        return 16 * s + 2 * t + (i & 1) + 8 * (i >> 1);
    }

    // the element of step i's fragment that lane quad t holds at place u
    static __device__ __forceinline__ int query_element(int i, int u, int t) {
        return Q8 ? 32 * (i / 2) + 8 * t + 4 * (i % 2) + u : 16 * i + 2 * t + (u & 1) + 8 * (u >> 1);
    }

    // lane i holds the row of the tile's token i (mod their number)
    static __device__ __forceinline__ void issue(const AttendArgs &a, uint32_t stage, uint32_t rows,
                                                 int lane) {
        constexpr int kUnits = kRowBytes / 16;
        // the first token's row of each 16-token step
        const uint32_t own = __shfl_sync(0xffffffffu, rows, kSub == 1 ? 0 : lane & 16);
        if (__all_sync(0xffffffffu, rows == own + lane % 16 && rows != kNoRow)) {
            // each step is one run of bytes (as where 16 divides the page)
            const char *k[kSub], *v[kSub];
#pragma unroll
            for (int s = 0; s < kSub; ++s) {
                const uint32_t first = kSub == 1 ? own : __shfl_sync(0xffffffffu, rows, 16 * s);
                const uint64_t at = (uint64_t)first * kRowBytes + 16 * lane;
                k[s] = static_cast<const char *>(a.kc) + at, v[s] = static_cast<const char *>(a.vc) + at;
            }
            constexpr int kTurns = kUnits / 2;  // of a step
#pragma unroll
            for (int i = 0; i < kSub * kTurns; ++i) {
                const int c = lane + 32 * i, s = i / kTurns;
                const uint32_t dst = stage + offset(c / kUnits, c % kUnits);
                copy_async<16>(dst, k[s] + 512 * (i % kTurns), 16);
                copy_async<16>(dst + kPlane, v[s] + 512 * (i % kTurns), 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kTokens * kUnits / 32; ++i) {
                const int c = lane + 32 * i, token = c / kUnits, unit = c % kUnits;
                uint32_t row = __shfl_sync(0xffffffffu, rows, token);
                const int bytes = row != kNoRow ? 16 : 0;
                row = row != kNoRow ? row : 0;
                const uint32_t dst = stage + offset(token, unit);
                const char *k = static_cast<const char *>(a.kc) + 16 * unit;
                const char *v = static_cast<const char *>(a.vc) + 16 * unit;
                copy_async<16>(dst, k + (uint64_t)row * kRowBytes, bytes);
                copy_async<16>(dst + kPlane, v + (uint64_t)row * kRowBytes, bytes);
            }
        }
        if (lane < kTokens) {
            if constexpr (Q8) {
                const bool ok = rows != kNoRow;
                const uint64_t first = (uint64_t)(ok ? rows : 0) * NB;
                const uint32_t dst = stage + 2 * kPlane + lane * kScaleWords * 4;
                const uint16_t *kd = a.kd + (first & ~(uint64_t)1), *vd = a.vd + (first & ~(uint64_t)1);
                if constexpr (NB == 8 || NB == 4) {
                    copy_async<2 * NB>(dst, kd, ok ? 2 * NB : 0);
                    copy_async<2 * NB>(dst + kScales, vd, ok ? 2 * NB : 0);
                } else {
#pragma unroll
                    for (int w = 0; w < kScaleWords; ++w) {
                        // an odd number of scales that starts on a word ends in half of one
                        const bool half = NB % 2 && w == kScaleWords - 1 && first % 2 == 0;
                        copy_async<4>(dst + 4 * w, kd + 2 * w, !ok ? 0 : half ? 2 : 4);
                        copy_async<4>(dst + kScales + 4 * w, vd + 2 * w, !ok ? 0 : half ? 2 : 4);
                    }
                }
            }
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + kRows + 4 * lane), "r"(rows) : "memory");
        }
    }

    // a token's scales as f16 pairs (`row`: its row number, whose parity places odd numbers of scales)
    static constexpr int kPairs = (NB + 1) / 2;
    static __device__ __forceinline__ void load_scales(const char *scales, int token, uint32_t row,
                                                       uint32_t (&w)[kPairs]) {
        const char *p = scales + token * kScaleWords * 4;
        if constexpr (NB % 8 == 0) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (NB % 4 == 0) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (NB % 2 == 0) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p) + (row & 1);
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                w[i] = h[2 * i] | (2 * i + 1 < NB ? (uint32_t)h[2 * i + 1] << 16 : 0u);
        }
    }

    // raw scores of the lane's tokens and heads t + 4 n: out[step][token][n]
    static __device__ __forceinline__ void scores(const char *stage, const uint4 (*q)[NT][32],
                                                  const uint32_t (&rows)[kSub][2], int lane,
                                                  float (&out)[kSub][2][NT]) {
        const int g = lane >> 2, t = lane & 3;
        if constexpr (!Q8) {
            float c[kSub][NT][4] = {};
            const uint32_t from = shared_addr(stage) + (lane & 15) * kStride + (lane >> 4) * 16;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                uint4 y[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) y[n] = q[i][n][lane];
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    const uint4 k0 = load_matrices<false>(from + 16 * s * kStride + 64 * i);
                    const uint4 k1 = load_matrices<false>(from + 16 * s * kStride + 64 * i + 32);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_16816(c[s][n], k0, {y[n].x, y[n].y});
                        mma_16816(c[s][n], k1, {y[n].z, y[n].w});
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < kSub; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) out[s][i][n] = c[s][n][2 * i] + c[s][n][2 * i + 1];
        } else {
            uint32_t d[kSub][2][kPairs];
#pragma unroll
            for (int s = 0; s < kSub; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    load_scales(stage + 2 * kPlane, score_token(s, i, g), rows[s][i], d[s][i]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) out[s][i][n] = 0.0f;
                }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    uint32_t x[2], y[2];  // 8 codes of each token
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint2 k = *reinterpret_cast<const uint2 *>(
                            stage + offset(score_token(s, i, g), 2 * b) + 8 * t);
                        x[i] = k.x ^ 0x80808080u, y[i] = k.y ^ 0x80808080u;
                    }
                    const uint4 k0 = {bytes_to_half2(x[0], 0x4140), bytes_to_half2(x[1], 0x4140),
                                      bytes_to_half2(x[0], 0x4342), bytes_to_half2(x[1], 0x4342)};
                    const uint4 k1 = {bytes_to_half2(y[0], 0x4140), bytes_to_half2(y[1], 0x4140),
                                      bytes_to_half2(y[0], 0x4342), bytes_to_half2(y[1], 0x4342)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float c[4];
                        const uint4 f = q[b][n][lane];
                        mma_16816_first(c, k0, {f.x, f.y});
                        mma_16816(c, k1, {f.z, f.w});
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            out[s][i][n] = fmaf(c[2 * i] + c[2 * i + 1], half_of(d[s][i][b / 2], b), out[s][i][n]);
                    }
                }
        }
    }

    // Q8_0: block b's codes of 16 tokens as the MMA's A operands, elements 4 (lane / 4) + {0, 1}
    // (v0) and + {2, 3} (v1)
    static __device__ __forceinline__ void values(const char *stage, int lane, int s, int b, uint4 &v0, uint4 &v1) {
        const int g = lane >> 2, t = lane & 3;
        uint32_t lo[2], hi[2];  // bytes of a token pair, interleaved
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t x[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                x[j] = *reinterpret_cast<const uint32_t *>(
                           stage + kPlane + offset(weight_token(s, 2 * i + j, t), 2 * b + (g >> 2)) + 4 * (g & 3)) ^
                       0x80808080u;
            lo[i] = __byte_perm(x[0], x[1], 0x5140);
            hi[i] = __byte_perm(x[0], x[1], 0x7362);
        }
        v0 = {bytes_to_half2(lo[0], 0x4140), bytes_to_half2(lo[0], 0x4342), bytes_to_half2(lo[1], 0x4140),
              bytes_to_half2(lo[1], 0x4342)};
        v1 = {bytes_to_half2(hi[0], 0x4140), bytes_to_half2(hi[0], 0x4342), bytes_to_half2(hi[1], 0x4140),
              bytes_to_half2(hi[1], 0x4342)};
    }

    // o += weight times value over the tile.  Q8_0: d holds the value scales
    // times 2^up, none of them above 1.
    static __device__ __forceinline__ void weigh(const char *stage, int lane, const float (&p)[kSub][2][NT],
                                                 const uint32_t (&d)[Q8 ? kSub : 1][4][kPairs], int up,
                                                 float (&o)[kRowsOut][NT][2]) {
        const int g = lane >> 2, t = lane & 3;
        // From the scores' layout (tokens g, g + 8 of head t) to the weights'
        // (tokens 2t, 2t + 1, 2t + 8, 2t + 9 of head g / 2, hi where g is even):
        // a weight travels as its two halves.
        const uint32_t low = g & 1 ? 0xffffffffu : 0u, pick = g & 1 ? 0x7632u : 0x5410u;
        const int source = 8 * t + (g >> 1);
        uint2 w[kSub][NT], w_lo[kSub][NT];
#pragma unroll
        for (int s = 0; s < kSub; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t hi, lo;
                split_pair(p[s][0][n] * kLift, p[s][1][n] * kLift, hi, lo);
                uint32_t both[2][2];  // [token g or g + 8][source lane]
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t mine = __byte_perm(hi, lo, i ? 0x7632 : 0x5410);
                    both[i][0] = __shfl_sync(0xffffffffu, mine, source);
                    both[i][1] = __shfl_sync(0xffffffffu, mine, source + 4);
                }
                if constexpr (!Q8) {
                    w[s][n] = {__byte_perm(both[0][0], both[0][1], pick), __byte_perm(both[1][0], both[1][1], pick)};
                } else {
                    w[s][n] = {__byte_perm(both[0][0], both[0][1], 0x5410) & low,
                               __byte_perm(both[1][0], both[1][1], 0x5410) & low};
                    w_lo[s][n] = {__byte_perm(both[0][0], both[0][1], pick), __byte_perm(both[1][0], both[1][1], pick)};
                }
            }
        const float down = 1.0f / kLift * (Q8 ? exp2i(-up) : 1.0f);
        if constexpr (!Q8) {
            const uint32_t from = shared_addr(stage) + kPlane + ((lane >> 4) * 8 + (lane & 7)) * kStride +
                                  ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int c = 0; c < kRowsOut; ++c) {
                float x[NT][4];
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    const uint4 v = load_matrices<true>(from + 16 * s * kStride + 32 * c);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (s == 0) mma_16816_first(x[n], v, w[s][n]);
                        else mma_16816(x[n], v, w[s][n]);
                }
                add(x, down, o[c]);
            }
        } else {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float x0[NT][4], x1[NT][4];
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    const uint32_t d0 = __byte_perm(d[s][0][b / 2], d[s][1][b / 2], b & 1 ? 0x7632 : 0x5410);
                    const uint32_t d1 = __byte_perm(d[s][2][b / 2], d[s][3][b / 2], b & 1 ? 0x7632 : 0x5410);
                    uint4 v0, v1;
                    values(stage, lane, s, b, v0, v1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 wd = {scale_half(w[s][n].x, w_lo[s][n].x, d0),
                                          scale_half(w[s][n].y, w_lo[s][n].y, d1)};
                        if (s == 0) {
                            mma_16816_first(x0[n], v0, wd);
                            mma_16816_first(x1[n], v1, wd);
                        } else {
                            mma_16816(x0[n], v0, wd);
                            mma_16816(x1[n], v1, wd);
                        }
                    }
                }
                add(x0, down, o[2 * b]);
                add(x1, down, o[2 * b + 1]);
            }
        }
    }

    // The same for value scales d of any size: a weight's product with its
    // scale is taken in f32 and then halved, each block and head of a tile
    // under a power of two of its own, which takes the largest product to
    // [2^14, 2^15).
    static __device__ __forceinline__ void weigh_any(const char *stage, int lane, const float (&p)[kSub][2][NT],
                                                     const uint32_t (&d)[Q8 ? kSub : 1][4][kPairs],
                                                     float (&o)[kRowsOut][NT][2]) {
        const int g = lane >> 2, t = lane & 3, source = 8 * t + (g >> 1);
        float w[kSub][NT][4];  // the weights' layout, as in weigh
#pragma unroll
        for (int s = 0; s < kSub; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[s][n][j] = __shfl_sync(0xffffffffu, p[s][j >> 1][n], source + 4 * (j & 1));
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float x0[NT][4], x1[NT][4], up[NT], down[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float most = 0.0f;
#pragma unroll
                for (int s = 0; s < kSub; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        most = fmaxf(most, fabsf(w[s][n][j] * half_of(d[s][j][b / 2], b)));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const int e = max(__float_as_int(most) >> 23, 15);  // most is below 2^(e - 126), 2^20
                up[n] = exp2i(141 - e);
                down[n] = __shfl_sync(0xffffffffu, exp2i(e - 141), 8 * t);  // the products' head is t, not g / 2
            }
#pragma unroll
            for (int s = 0; s < kSub; ++s) {
                uint4 v0, v1;
                values(stage, lane, s, b, v0, v1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = w[s][n][j] * half_of(d[s][j][b / 2], b) * up[n];
                    uint2 hi, lo;
                    split_pair(x[0], x[1], hi.x, lo.x);
                    split_pair(x[2], x[3], hi.y, lo.y);
                    const uint2 wd = g & 1 ? lo : hi;
                    if (s == 0) {
                        mma_16816_first(x0[n], v0, wd);
                        mma_16816_first(x1[n], v1, wd);
                    } else {
                        mma_16816(x0[n], v0, wd);
                        mma_16816(x1[n], v1, wd);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    o[2 * b][n][i] = fmaf(x0[n][2 * i] + x0[n][2 * i + 1], down[n], o[2 * b][n][i]);
                    o[2 * b + 1][n][i] = fmaf(x1[n][2 * i] + x1[n][2 * i + 1], down[n], o[2 * b + 1][n][i]);
                }
        }
    }

    // A tile's products, the weights' halves joined, times `down` to the outputs.  The MMA
    // truncates what it adds to its accumulators, and always towards zero: over
    // a long sequence's tiles that would add up (32768 tokens of one split: 9e-6
    // of the output with f16, 4e-5 with Q8_0; a sum rounded to nearest 2e-7), so
    // only the products of one tile are summed there.
    static __device__ __forceinline__ void add(const float (&x)[NT][4], float down, float (&o)[NT][2]) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) o[n][i] = fmaf(x[n][2 * i] + x[n][2 * i + 1], down, o[n][i]);
    }

    // the element that row g (i = 0) or g + 8 (i = 1) of output tile c stands for
    static __device__ __forceinline__ int element(int c, int i, int g) {
        return Q8 ? 32 * (c / 2) + 4 * g + 2 * (c % 2) + i : 16 * c + 8 * i + g;
    }
};

// CTA (head tile and split, key head, sequence): its warps take the split's
// tiles of tokens in turn, each with its own ring, running maximum, sum and
// output; they are joined in shared memory at the end.
template <int NB, bool Q8, int NT>
__global__ void __launch_bounds__(Tile<NB, Q8, NT>::kWarps * 32, Tile<NB, Q8, NT>::kCtas)
attend_kernel(const AttendArgs a) {
    using T = Tile<NB, Q8, NT>;
    constexpr int D = NB * 32, H = T::kHeads;
    // (at 16 off a multiple of 32, Q8_0 rows were filled slower: 66 us for 62)
    extern __shared__ __align__(128) char s_ring[];
    __shared__ uint4 s_q[NB][NT][32];  // two steps of 16 elements
    __shared__ float s_m[T::kWarps][H], s_l[T::kWarps][H];
    __shared__ float s_scale[NT > 1 ? H : 1];
    __shared__ float2 s_tops[kMaxCluster][H];  // bases and sums of a cluster's CTAs
    __shared__ uint64_t s_arrived;             // counts what they send

    pdl_launch_dependents();  // the next grid waits for this one's end itself
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    // A cluster's CTAs are the splits of one head tile.  Otherwise the head
    // tiles that read the same keys are neighbours, then the key heads, which
    // share pages (splits before them: 0 to 14% longer over 40 shapes), then
    // the splits.
    const int tile = a.cluster ? blockIdx.x / a.splits : blockIdx.x % a.head_tiles;
    const int split = a.cluster ? blockIdx.x % a.splits : blockIdx.y;
    const int kv_head = a.cluster ? blockIdx.y : blockIdx.x / a.head_tiles;
    const int64_t b = blockIdx.z;
    const int first_head = kv_head * a.group + tile * H;
    const int tile_heads = min(H, a.group - tile * H);
    if (a.cluster) {
        if (threadIdx.x == 0) {
            const int part = (H * D / 4 + a.splits - 1) / a.splits * 4;
            const int mine = max(0, min(part, tile_heads * D - split * part));
            exchange_open(&s_arrived, (uint32_t)(a.splits * (4 * mine + 8 * tile_heads)));
        }
        cluster_arrive_relaxed();  // waited for before the first store to another CTA
    }
    pdl_wait();  // for the predecessor's end, before anything is read or written

    // The query's fragments: column g is head g / 2's hi (g even) or lo; a warp
    // takes 4 heads, or a part of 4 heads' steps.  Loaded first: the length,
    // the page table and these come in one latency.
    static_assert(NT <= T::kWarps, "");
    const int n_own = NT == 1 ? 0 : warp, own_head = 4 * n_own + (g >> 1);
    const bool any = own_head < tile_heads;
    float x[2 * NB][4];
    if (NT == 1 || n_own < NT) {
        const float *q = a.q + b * a.ldq + (int64_t)(first_head + (any ? own_head : 0)) * D;
        if (((reinterpret_cast<uintptr_t>(a.q) | (uintptr_t)a.ldq * 4) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
                for (int u = 0; u < 4; u += 2) {  // pairs are neighbours
                    const float2 y = *reinterpret_cast<const float2 *>(q + T::query_element(i, u, t));
                    x[i][u] = y.x, x[i][u + 1] = y.y;
                }
        } else {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) x[i][u] = q[T::query_element(i, u, t)];
        }
    }

    const int len = a.lens[b];
    const int all = min(max(len, 0), a.max_tokens);
    const int start = a.window > 0 ? max(0, all - a.window) : 0;
    const int64_t from = start + (int64_t)split * a.span;  // below 2^30 + a span
    const int begin = (int)from;  // at or behind `end` where the split is empty
    const int end = a.span < all - from ? begin + a.span : all;

    const int32_t *table = a.table + b * a.table_ld;
    // The table is read whether or not the length covers the token (it has an
    // entry), so that a CTA's first read does not wait for the length's.
    auto row_of = [&](int token) {
        const uint32_t p = (uint32_t)(((uint64_t)(uint32_t)token * a.page_mul) >> a.page_shift);
        const uint32_t page = p < (uint32_t)a.table_ld ? (uint32_t)table[p] : 0xffffffffu;
        const uint32_t row = (page * (uint32_t)a.kv_heads + kv_head) * (uint32_t)a.page_size +
                             ((uint32_t)token - p * (uint32_t)a.page_size);
        return token < end && page < (uint32_t)a.num_pages ? row : kNoRow;
    };
    // tile i of this warp starts at token begin + (warp + T::kWarps i) kTokens
    constexpr int kStep = T::kWarps * T::kTokens;
    const int first = begin + warp * T::kTokens;
    const int tiles = first < end ? (end - first + kStep - 1) / kStep : 0;
    char *ring = s_ring + warp * T::kStages * T::kBytes;
    const uint32_t ring_addr = shared_addr(ring);
    const int token = first + lane % T::kTokens;
    uint32_t ahead[T::kStages], full = 0;  // full: a bit for each stage
#pragma unroll
    for (int i = 0; i < T::kStages; ++i) ahead[i] = row_of(token + i * kStep);
    if (begin >= end && a.splits > 1 && !a.cluster) return;  // the join counts the same splits
#pragma unroll
    for (int i = 0; i < T::kStages - 1; ++i) {
        if (i < tiles) T::issue(a, ring_addr + i * T::kBytes, ahead[i], lane);
        full |= (uint32_t)__all_sync(0xffffffffu, ahead[i] != kNoRow) << i;
        copies_commit();
    }
    uint32_t next_rows = ahead[T::kStages - 1];

    float scale[NT];
    if (NT == 1 || n_own < NT) {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[i][u] = any ? x[i][u] : 0.0f;
                most = fmaxf(most, fabsf(x[i][u]));
            }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // most is in [2^(E - 127), 2^(E - 126)): times 2^(134 - E) it is in [128, 256)
        int e = min(max(__float_as_int(most) >> 23, 8), 254);
        if (most == 0.0f) e = 134;
        const float up = exp2i(134 - e);
        const float mine = a.scale * 1.4426950408889634f * exp2i(e - 134);
        if constexpr (NT == 1)
            scale[0] = __shfl_sync(0xffffffffu, mine, 8 * t);  // the scores' head is t, not g / 2
        else if (t == 0 && g % 2 == 0)
            s_scale[own_head] = mine;
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
            if (NT == 1 && i % T::kWarps != warp) continue;
            uint2 hi, lo;
            split_pair(x[i][0] * up, x[i][1] * up, hi.x, lo.x);
            split_pair(x[i][2] * up, x[i][3] * up, hi.y, lo.y);
            reinterpret_cast<uint2 *>(&s_q[i / 2][n_own][lane])[i % 2] = g & 1 ? lo : hi;
        }
    }
    __syncthreads();
    if constexpr (NT > 1)
#pragma unroll
        for (int n = 0; n < NT; ++n) scale[n] = s_scale[4 * n + t];

    // o: elements g and g + 8 of each tile of 16, of head t; l: the sum of this
    // lane's weights, both relative to 2^base
    float o[T::kRowsOut][NT][2] = {}, base[NT], l[NT] = {};
#pragma unroll
    for (int n = 0; n < NT; ++n) base[n] = -INFINITY;
    // Q8_0: the value scales are taken times 2^up, 0 or 10, which fits tiles
    // whose scales other than 0 lie in [least_d, most_d]; -1: each block has a
    // power of its own (weigh_any), and every tile is looked at again
    int up = -1;
    __half2 least_d = __half2half2(__ushort_as_half(0)), most_d = __half2half2(__float2half_rn(-1.0f));
    int slot = 0, fill = T::kStages - 1;
    for (int i = 0; i < tiles; ++i) {
        copies_wait<T::kStages - 2>();
        __syncwarp();  // every lane's copies are in, and the last tile is read by all
        if (i + T::kStages - 1 < tiles) T::issue(a, ring_addr + fill * T::kBytes, next_rows, lane);
        copies_commit();
        // whether every token of the tile that will be in this slot is attended to
        full = (full & ~(1u << fill)) | ((uint32_t)__all_sync(0xffffffffu, next_rows != kNoRow) << fill);
        fill = fill + 1 == T::kStages ? 0 : fill + 1;
        next_rows = i + T::kStages < tiles ? row_of(token + (i + T::kStages) * kStep) : kNoRow;

        const char *stage = ring + slot * T::kBytes;
        const bool whole = full >> slot & 1;
        slot = slot + 1 == T::kStages ? 0 : slot + 1;
        const uint32_t *s_rows = reinterpret_cast<const uint32_t *>(stage + T::kRows);
        uint32_t rows[T::kSub][2] = {};
        if (!whole || (Q8 && NB % 2))
#pragma unroll
            for (int s = 0; s < T::kSub; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) rows[s][j] = s_rows[T::score_token(s, j, g)];
        float raw[T::kSub][2][NT], p[T::kSub][2][NT];
        T::scores(stage, s_q, rows, lane, raw);
        uint32_t d[Q8 ? T::kSub : 1][4][T::kPairs];
        __half2 largest = __half2half2(__ushort_as_half(0)), smallest = __half2half2(__ushort_as_half(0x3c00));
        auto look = [&](const __half2 &scales) {
            const __half2 size = __habs2(scales);
            largest = __hmax2(largest, size);
            smallest = __hmin2(smallest, __hadd2(size, __heq2(size, __half2half2(__ushort_as_half(0)))));
        };
        if constexpr (Q8) {
#pragma unroll
            for (int s = 0; s < T::kSub; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = T::weight_token(s, j, t);
                    T::load_scales(stage + 2 * T::kPlane + T::kScales, at, NB % 2 ? s_rows[at] : 0u, d[s][j]);
                    if constexpr (NB % 2)
#pragma unroll
                        for (int c = 0; c < T::kPairs; ++c) look(reinterpret_cast<const __half2 &>(d[s][j][c]));
                }
            if constexpr (NB % 2 == 0) {  // the words hold scales alone: a lane looks at a part of them
                constexpr int kWords = T::kTokens * T::kScaleWords;  // 48 where d is 192; row numbers lie behind
                const __half2 *words = reinterpret_cast<const __half2 *>(stage + 2 * T::kPlane + T::kScales);
#pragma unroll
                for (int c = 0; c < kWords; c += 32)
                    if (kWords % 32 == 0 || c + lane < kWords) look(words[c + lane]);
            }
        }
        bool move = Q8 && !(__hble2(largest, most_d) && __hbge2(smallest, least_d));
#pragma unroll
        for (int s = 0; s < T::kSub; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (!whole && rows[s][j] == kNoRow) raw[s][j][n] = -INFINITY;
                    p[s][j][n] = fmaf(raw[s][j][n], scale[n], -base[n]);
                    move |= p[s][j][n] > 4.0f;
                }
        if (__any_sync(0xffffffffu, move)) {
            if constexpr (Q8) {
                // The largest weight so far is 1 to 2^4: times kLift and a scale
                // of 2^-14 to 1 it keeps 22 bits and stays below 2^15.
                auto halves = [](const __half2 &x) { return reinterpret_cast<const uint32_t &>(x); };
                const uint32_t most = __reduce_max_sync(0xffffffffu, max(halves(largest) & 0xffffu, halves(largest) >> 16));
                const uint32_t least =
                    __reduce_min_sync(0xffffffffu, min(halves(smallest) & 0xffffu, halves(smallest) >> 16));
                // f16: 0x3c00 is 1, 0x1400 is 2^-10, 0x0400 is 2^-14, and none above 0 is below 2^-24
                up = most <= 0x1400u ? 10 : most <= 0x3c00u && least >= 0x0400u ? 0 : -1;
                most_d = up < 0 ? __half2half2(__float2half_rn(-1.0f)) : __half2half2(__ushort_as_half(up ? 0x1400 : 0x3c00));
                least_d = __half2half2(__ushort_as_half(up ? 0 : 0x0400));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top = base[n];
#pragma unroll
                for (int s = 0; s < T::kSub; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) top = fmaxf(top, raw[s][j][n] * scale[n]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float alpha = top == base[n] ? 1.0f : exp2_approx(base[n] - top);
                base[n] = top;
                l[n] *= alpha;
#pragma unroll
                for (int c = 0; c < T::kRowsOut; ++c)
#pragma unroll
                    for (int j = 0; j < 2; ++j) o[c][n][j] *= alpha;
#pragma unroll
                for (int s = 0; s < T::kSub; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) p[s][j][n] = fmaf(raw[s][j][n], scale[n], -top);
            }
        }
#pragma unroll
        for (int s = 0; s < T::kSub; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    p[s][j][n] = exp2_approx(p[s][j][n]);
                    if (!whole && rows[s][j] == kNoRow) p[s][j][n] = 0.0f;
                    l[n] += p[s][j][n];
                }
        if (Q8 && up > 0) {
            const __half2 f = __half2half2(__float2half_rn(1024.0f));
#pragma unroll
            for (int s = 0; s < (Q8 ? T::kSub : 1); ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < T::kPairs; ++c) {
                        const __half2 h = __hmul2(reinterpret_cast<const __half2 &>(d[s][j][c]), f);
                        d[s][j][c] = reinterpret_cast<const uint32_t &>(h);
                    }
        }
        if (Q8 && up < 0)
            T::weigh_any(stage, lane, p, d, o);
        else
            T::weigh(stage, lane, p, d, up, o);
    }

#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n] += __shfl_xor_sync(0xffffffffu, l[n], x);
        if (g == 0) s_m[warp][4 * n + t] = base[n], s_l[warp][4 * n + t] = l[n];
    }
    __syncthreads();  // the ring is read: it takes the outputs [warp][head][element]
    float *s_o = reinterpret_cast<float *>(s_ring);
#pragma unroll
    for (int c = 0; c < T::kRowsOut; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s_o[(warp * H + 4 * n + t) * D + T::element(c, i, g)] = o[c][n][i];
    __syncthreads();
    const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)a.ldo * 4) & 15) == 0;
    auto finish = [&](int h, int e, float top, float sum, const float (&acc)[4]) {
        const float inverse = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
        float *to = a.out + b * a.ldo + (int64_t)(first_head + h) * D + e;
        if (wide) {
            *reinterpret_cast<float4 *>(to) =
                make_float4(acc[0] * inverse, acc[1] * inverse, acc[2] * inverse, acc[3] * inverse);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) to[u] = acc[u] * inverse;
        }
        if (e == 0 && a.lse)
            a.lse[b * a.heads + first_head + h] =
                sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    // `count` parts of four elements, each relative to a base of its own
    auto join = [&](int count, auto base_of, auto sum_of, auto part_of, float &top, float &sum, float (&acc)[4]) {
        constexpr int kMost = kMaxCluster;
        float4 p[kMost];
        float m[kMost], l[kMost];
#pragma unroll
        for (int c = 0; c < kMost; ++c) {
            m[c] = -INFINITY, l[c] = 0.0f, p[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c < count) m[c] = base_of(c), l[c] = sum_of(c), p[c] = *reinterpret_cast<const float4 *>(part_of(c));
        }
        top = m[0];
#pragma unroll
        for (int c = 1; c < kMost; ++c) top = fmaxf(top, m[c]);
        const float base = top == -INFINITY ? 0.0f : top;
        sum = acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
#pragma unroll
        for (int c = 0; c < kMost; ++c) {
            const float f = exp2_approx(m[c] - base);
            sum = fmaf(f, l[c], sum);
            acc[0] = fmaf(f, p[c].x, acc[0]), acc[1] = fmaf(f, p[c].y, acc[1]);
            acc[2] = fmaf(f, p[c].z, acc[2]), acc[3] = fmaf(f, p[c].w, acc[3]);
        }
    };
    // Of a cluster's CTA: the elements that it finishes, 2^22 / part rounded up
    // (j / part for j < 2^11).
    const int part = (H * D / 4 + a.splits - 1) / a.splits * 4;
    const uint32_t part_mul = (1u << 22) / (uint32_t)part + 1;
    static_assert(H * D <= 2048, "");
    // In a cluster each CTA finishes `part` elements: it gets them, and every
    // head's base and sum, from all CTAs into shared memory of its own.
    float *s_parts = reinterpret_cast<float *>(s_ring + T::kRing);  // [split][part]
    if (a.cluster) cluster_wait();
    float top, sum, acc[4];
#pragma unroll 1
    for (int j = 4 * threadIdx.x; j < tile_heads * D; j += T::kWarps * 128) {
        const int h = j / D, e = j % D;
        join(T::kWarps, [&](int w) { return s_m[w][h]; }, [&](int w) { return s_l[w][h]; },
             [&](int w) { return s_o + (w * H + h) * D + e; }, top, sum, acc);
        if (a.cluster) {
            if (a.withhold) continue;
            const int to = (uint32_t)j * part_mul >> 22, rank = e / 4;
            exchange_store(exchange_addr(s_parts + split * part + j - to * part, to), acc[0], acc[1], acc[2], acc[3],
                           exchange_addr(&s_arrived, to));
            if (rank < a.splits)
                exchange_store(exchange_addr(&s_tops[split][h], rank), top, sum, exchange_addr(&s_arrived, rank));
        } else if (a.splits == 1) {
            finish(h, e, top, sum, acc);
        } else {
            const int64_t place = (b * a.heads + first_head + h) * a.splits + split;
            *reinterpret_cast<float4 *>(a.part + place * D + e) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (e == 0) a.part_ml[place] = make_float2(top, sum);
        }
    }
    if (!a.cluster || !exchange_wait(&s_arrived, a.wait_limit)) return;
#pragma unroll 1
    for (int i = 4 * threadIdx.x; i < part && split * part + i < tile_heads * D; i += T::kWarps * 128) {
        const int j = split * part + i, h = j / D;
        join(a.splits, [&](int c) { return s_tops[c][h].x; }, [&](int c) { return s_tops[c][h].y; },
             [&](int c) { return s_parts + c * part + i; }, top, sum, acc);
        finish(h, j % D, top, sum, acc);
    }
}

// Joins the splits of a head: warp w takes splits w, w + kJoinWarps, ... in
// order, then the warps' sums are added in order.  A warp reads a partial
// output 4 elements a lane (128 a turn), all of its loads before their use:
// one warp a head going through the splits one by one took 5 us of a
// 38-split join.
template <int NB, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendArgs a) {
    constexpr int D = NB * 32, kTurns = (D + 127) / 128, kAhead = 4;
    __shared__ float s_o[kJoinWarps][D];
    __shared__ float s_l[kJoinWarps];
    // The next grid is not let in before this one's CTAs leave: where it is one
    // wave, as the next attention is, its CTAs would crowd on what is free (1
    // sequence of 65536 tokens, Q8_0, 64 heads: 47 us against 39).
    pdl_wait();
    const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.y, head = b * a.heads + h;
    const int all = min(max(a.lens[b], 0), a.max_tokens);
    const int start = a.window > 0 ? max(0, all - a.window) : 0;
    const int splits = (int)(((int64_t)(all - start) + a.span - 1) / a.span);
    const float2 *ml = a.part_ml + head * a.splits;
    const float *part = a.part + head * a.splits * D;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, ml[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.0f : top;
    float4 acc[kTurns] = {};
    float sum = 0.0f;
    for (int s0 = warp; s0 < splits; s0 += kJoinWarps * kAhead) {
        float4 x[kAhead][kTurns];
        float2 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int s = s0 + i * kJoinWarps;
            w[i] = s < splits ? ml[s] : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int j = 0; j < kTurns; ++j) {
                const int e = 128 * j + 4 * lane;
                x[i][j] = s < splits && e < D ? *reinterpret_cast<const float4 *>(part + (int64_t)s * D + e)
                                              : make_float4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float f = exp2_approx(w[i].x - base);
            sum = fmaf(f, w[i].y, sum);
#pragma unroll
            for (int j = 0; j < kTurns; ++j) {
                acc[j].x = fmaf(f, x[i][j].x, acc[j].x);
                acc[j].y = fmaf(f, x[i][j].y, acc[j].y);
                acc[j].z = fmaf(f, x[i][j].z, acc[j].z);
                acc[j].w = fmaf(f, x[i][j].w, acc[j].w);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kTurns; ++j)
        if (128 * j + 4 * lane < D) *reinterpret_cast<float4 *>(&s_o[warp][128 * j + 4 * lane]) = acc[j];
    if (lane == 0) s_l[warp] = sum;
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kJoinWarps * 32) {
        float total = 0.0f, out = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) total += s_l[w], out += s_o[w][e];
        a.out[b * a.ldo + (int64_t)h * D + e] = total == 0.0f ? 0.0f : __fdiv_rn(out, total);
        if (e == 0 && a.lse)
            a.lse[head] = total == 0.0f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
    }
}

template <int NB, bool Q8, int NT>
cudaError_t launch_attend_nb(const AttendArgs &a, cudaStream_t s) {
    using T = Tile<NB, Q8, NT>;
    const dim3 grid = a.cluster ? dim3((unsigned)(a.splits * a.head_tiles), (unsigned)a.kv_heads, (unsigned)a.batch)
                                : dim3((unsigned)(a.head_tiles * a.kv_heads), (unsigned)a.splits, (unsigned)a.batch);
    static std::atomic<uint64_t> opted_in;  // devices whose limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!(opted_in.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(attend_kernel<NB, Q8, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 T::kRing + T::kClusterParts);
        if (e != cudaSuccess) return e;
        opted_in.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)a.splits, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(T::kWarps * 32);
    cfg.dynamicSmemBytes = T::kRing + (a.cluster ? T::kClusterParts : 0);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster ? 2 : 1;
    if (a.cluster) g_exchange_used.store(true, std::memory_order_relaxed);
    e = cudaLaunchKernelEx(&cfg, attend_kernel<NB, Q8, NT>, a);
    if (e != cudaSuccess || a.splits == 1 || a.cluster) return e;
    const dim3 join((unsigned)a.heads, (unsigned)a.batch);
    if (a.splits <= 8) return launch_kernel(attend_join_kernel<NB, 4>, join, dim3(4 * 32), 0, s, true, a);
    return launch_kernel(attend_join_kernel<NB, 16>, join, dim3(16 * 32), 0, s, true, a);
}

// f(std::integral_constant<int, NB>) for d = 32 NB
template <typename F>
auto with_blocks(int d, F f) {
    switch (d / 32) {
        case 1: return f(std::integral_constant<int, 1>());
        case 2: return f(std::integral_constant<int, 2>());
        case 3: return f(std::integral_constant<int, 3>());
        case 4: return f(std::integral_constant<int, 4>());
        case 5: return f(std::integral_constant<int, 5>());
        case 6: return f(std::integral_constant<int, 6>());
        case 7: return f(std::integral_constant<int, 7>());
        default: return f(std::integral_constant<int, 8>());
    }
}

// f(std::integral_constant<int, NT>): B tiles of 4 heads a CTA takes, for
// `group` query heads to a key head.  More than 8 heads take several CTAs,
// which read the keys one from HBM and the others from L2: 16 heads in one
// (NT = 4) took as long for 16 sequences and 10 us instead of 7 for one.
template <typename F>
auto with_heads(int group, F f) {
    if (group <= 4) return f(std::integral_constant<int, 1>());
    return f(std::integral_constant<int, 2>());
}

template <bool Q8>
AttendShape attend_shape(int d, int group) {
    return with_blocks(d, [&](auto nb) {
        return with_heads(group, [](auto nt) {
            using T = Tile<decltype(nb)::value, Q8, decltype(nt)::value>;
            return AttendShape{T::kCtas, T::kHeads};
        });
    });
}

template <bool Q8>
cudaError_t launch_attend(const AttendArgs &a, cudaStream_t s) {
    return with_blocks(a.d, [&](auto nb) {
        return with_heads(a.group, [&](auto nt) {
            return launch_attend_nb<decltype(nb)::value, Q8, decltype(nt)::value>(a, s);
        });
    });
}

}  // namespace
}  // namespace qmm
