// Beam search's selection (sm_103a): the n best of score + log-softmax over
// beams x vocabulary, in one pass over the logits, and the gather that gives
// the new beams their parents' states.
//
//   score(r, x) = scores[r] + logits[r][x] - log sum_y exp(logits[r][y])
//
// beam_part_kernel: a CTA per (row, chunk of the row).  A chunk's logits are
// read once into registers; its maximum, its sum of exponentials and its n
// best logits go to the workspace.  Within a row scores order like logits, so
// a row's n best scores are among its chunks' n best logits.  The n best of a
// chunk: each warp sorts its lanes' maxima; all eight warps' ceil(n / 8)-th, and
// four warps' ceil(n / 4)-th, are bounds that at least n logits reach, and few
// more do (about 30 for n = 16); those are ranked against one another.  (More
// reach it where many are equal, or the large ones lie in few threads: then one
// after the other is taken.)
// beam_join_kernel: a CTA per request joins the sums, scores the candidates and
// ranks them the same way, taking the best of every chunk first.
// What decides between beams has to be finer than fp32, and the FP64 pipe is
// slow here (a join that compared doubles took 47 us, one that added and took
// exponentials in them 15): scores, and sums beyond a thread's 32 exponentials
// (which are added in fp32: 2^-22 of the sum, as the exponentials themselves),
// are pairs of fp32 numbers, value and rest (48 bits, by error-free sums),
// compared as 64-bit whole numbers of the same order.
// 32 requests of 8 beams over 131072 fp32 tokens, n = 16 (a fifth of the beams
// finished): parts 29 us (107 MB, 3.7 TB/s; 668 instructions a warp and chunk at
// 55% of the issue slots), join 6; as bf16 or fp16, half the bytes at the same
// instructions, 34 us in place of 36.  One request of 4 beams over 32000: 8.8 us
// with the states' gather, the two kernels' latencies.  32 logits a thread and
// four CTAs per SM were best: 64 logits 63 us, 16 logits 52, a persistent grid
// that copies the next chunk ahead 69 (of 40 for all three kernels).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/kvp.h"
#include "kvp_internal.h"
#include "launch.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 32;                       // logits per thread
constexpr int kChunk = kThreads * kPer;
constexpr int kUneven = kChunk - 8;            // chunk of a row off 16-byte boundaries (8 logits at most in 16 bytes)
constexpr int kMaxOut = 128, kMaxBeams = 128;
constexpr int kCap = 1024;                     // candidates ranked at once

// A chunk's part of its row.
struct alignas(16) PartHead {
    float sum, rest;   // of exp(logit - top)
    float top;         // largest logit; +inf where the row is not to be used
    float pad;
};

struct BeamArgs {
    const void *logits;
    int64_t row_stride;
    const float *scores;
    const uint8_t *finished;
    int32_t pad, groups, beams, vocab, n, chunks;
    int32_t step;                 // logits of a chunk
    int32_t early;                // the join may start beside the parts' CTAs
    uint32_t div;                 // 2^32 / (chunks * beams), rounded up; 0: too large for that
    float *out_scores;
    int32_t *out_rows, *out_tokens;
    PartHead *heads;              // [rows][chunks]
    float *cand;                  // [rows][chunks][n], descending, then -inf
    int32_t *cand_at;
};

// An fp32 number as a whole number of the same order (-0 as 0), and back from
// the upper half of a 64-bit one.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t k = (uint32_t)(key >> 32);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// The fourth largest of eight.
template <class T>
__device__ __forceinline__ T fourth_of_8(const T *from) {
    T a[4], b[4];
    auto least = [](T x, T y) { return x < y ? x : y; };
    auto most = [](T x, T y) { return x < y ? y : x; };
    auto order = [&](T &x, T &y) {
        const T t = most(x, y);
        y = least(x, y);
        x = t;
    };
    auto sort4 = [&](T (&v)[4], const T *from) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = from[i];
        order(v[0], v[1]);
        order(v[2], v[3]);
        order(v[0], v[2]);
        order(v[1], v[3]);
        order(v[1], v[2]);
    };
    sort4(a, from);
    sort4(b, from + 4);
    return most(most(most(a[3], b[3]), least(a[1], b[1])), most(least(a[0], b[2]), least(a[2], b[0])));
}

__device__ __forceinline__ bool bigger(float x, float y) { return x > y; }
__device__ __forceinline__ bool bigger(uint64_t x, uint64_t y) { return x > y; }
// A warp's values in descending order.
template <class T>
__device__ __forceinline__ T sort_warp(T x, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {
            const T y = __shfl_xor_sync(0xffffffffu, x, j);
            const bool large = ((lane & j) == 0) == ((lane & k) == 0);     // this lane takes the larger
            x = bigger(y, x) == large ? y : x;
        }
    return x;
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

// Thread i's k-th logit of a chunk sits at (k / V) * V * kThreads + i * V + k % V.
template <class T> constexpr int kVec = 16 / sizeof(T);
template <class T>
__device__ __forceinline__ int place(int tid, int k) { return (k / kVec<T>) * kVec<T> * kThreads + tid * kVec<T> + k % kVec<T>; }

__device__ __forceinline__ float exp2_sfu(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// (x, xr) += (y, yr): the error of the fp32 sum goes into the rest.
__device__ __forceinline__ void add2(float &x, float &xr, float y, float yr) {
    const float s = __fadd_rn(x, y), b = __fsub_rn(s, x);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(x, __fsub_rn(s, b)), __fsub_rn(y, b)), __fadd_rn(xr, yr));
    x = __fadd_rn(s, e);
    xr = __fsub_rn(e, __fsub_rn(x, s));
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) beam_part_kernel(const BeamArgs a) {
    __shared__ float2 s_sum[kWarps];
    __shared__ __align__(16) float s_max[kWarps], s_eighth[kWarps], s_fourth[kWarps];
    __shared__ uint64_t s_key[kCap];
    __shared__ int s_count, s_best[kWarps];
    __shared__ float s_bestv[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
    griddep_wait();
    if (a.early) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (a.finished && a.finished[row]) return;
    // logits x0 .. x0 + len - 1, the thread's k-th at place(tid, k) - shift: rows
    // may begin anywhere, their 16-byte pieces are read whole all the same, and
    // only the ends one by one
    const int x0 = chunk * a.step, len = min(a.step, a.vocab - x0);
    const T *src = static_cast<const T *>(a.logits) + row * a.row_stride + x0;
    const int shift = (int)((uintptr_t)src % 16 / sizeof(T));
    const bool full = len == kChunk && shift == 0;
    float v[kPer];
    {
        uint4 raw[kPer / kVec<T>];
#pragma unroll
        for (int i = 0; i < kPer / kVec<T>; ++i) {
            const int at = place<T>(tid, i * kVec<T>) - shift;
            if (full || (at >= 0 && at + kVec<T> <= len)) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(src + at));
        }
#pragma unroll
        for (int i = 0; i < kPer / kVec<T>; ++i) {
            const int at = place<T>(tid, i * kVec<T>) - shift;
            const T *e = reinterpret_cast<const T *>(&raw[i]);
            if (full || (at >= 0 && at + kVec<T> <= len)) {
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) v[i * kVec<T> + k] = as_float(e[k]);
            } else {
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k)
                    v[i * kVec<T> + k] = (unsigned)(at + k) < (unsigned)len ? as_float(src[at + k]) : -INFINITY;
            }
        }
    }
    constexpr int GROUP = 4;             // maxima of 4 logits: most reach no candidate
    float part_top[kPer / GROUP], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer / GROUP; ++i) {
        part_top[i] = v[i * GROUP];
#pragma unroll
        for (int k = 1; k < GROUP; ++k) part_top[i] = fmaxf(part_top[i], v[i * GROUP + k]);
        top = fmaxf(top, part_top[i]);
    }
    if (top == -INFINITY) {              // (a thread of NaNs alone; others show in its sum)
        bool nan = false;
#pragma unroll
        for (int k = 0; k < kPer; ++k) nan |= v[k] != v[k];
        if (nan) top = INFINITY;         // as +inf does: the row has no log-sum-exp
    }
    top = sort_warp(top, lane);
    if (lane == 0) s_max[warp] = top;
    if (lane == (a.n + 7) / 8 - 1) s_eighth[warp] = top;
    if (lane == (a.n + 3) / 4 - 1) s_fourth[warp] = top;
    if (tid == 0) s_count = 0;
    __syncthreads();
    static_assert(kWarps == 8, "eight warps");
    float all = s_max[0], bound = s_eighth[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        all = fmaxf(all, s_max[w]);
        bound = fminf(bound, s_eighth[w]);
    }
    bound = fmaxf(bound, fourth_of_8(s_fourth));
    bound = fmaxf(bound, -FLT_MAX);      // -inf is no candidate
    PartHead *head = a.heads + (int64_t)row * a.chunks + chunk;
    float *cand = a.cand + ((int64_t)row * a.chunks + chunk) * a.n;
    int32_t *cand_at = a.cand_at + ((int64_t)row * a.chunks + chunk) * a.n;
    if (!(all < INFINITY) || all == -INFINITY) {       // nothing here, or nothing in the row
        if (tid == 0) *head = PartHead{0.f, 0.f, all, 0.f};
        if (tid < a.n) cand[tid] = -INFINITY;
        return;
    }
    // 2^(v log2 e - c), c = all log2 e rounded: one rounding of each exponent
    // (2^-24 of it) and the power's 2^-22, both ways alike; c's own rounding,
    // known exactly, is one factor of the sum.  (expf: 10 instructions a logit
    // instead of 3)
    constexpr float kLog2e = 1.4426950408889634f;
    const bool near = fabsf(all) < 256.f;     // (c's rounding is below 2^-15)
    const float c = __fmul_rn(all, kLog2e);
    float part = 0.f, rest = 0.f;
    if (near) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) part += exp2_sfu(__fmaf_rn(v[k], kLog2e, -c));
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) part += exp2_sfu((v[k] - all) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        add2(part, rest, __shfl_xor_sync(0xffffffffu, part, o), __shfl_xor_sync(0xffffffffu, rest, o));
    if (lane == 0) s_sum[warp] = make_float2(part, rest);
#pragma unroll
    for (int i = 0; i < kPer / GROUP; ++i) {
        if (!(part_top[i] >= bound)) continue;
#pragma unroll
        for (int k = i * GROUP; k < (i + 1) * GROUP; ++k)
            if (v[k] >= bound) {
                const int j = atomicAdd(&s_count, 1);
                // (larger first, then the lower token)
                if (j < kCap) s_key[j] = (uint64_t)order_key(v[k]) << 32 | (uint32_t)~(place<T>(tid, k) - shift);
            }
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) add2(part, rest, s_sum[w].x, s_sum[w].y);
        // times 2^(c - all log2 e) = 1 - d log 2 and terms below 2^-30
        const float d = near ? __fmaf_rn(all, kLog2e, -c) * 0.69314718f : 0.f;
        add2(part, rest, -d * part, 0.f);
        *head = PartHead{part, rest, part == part ? all : INFINITY, 0.f};
    }
    const int found = s_count;
    if (found <= kCap) {
        for (int i = tid; i < found; i += kThreads) {
            const uint64_t x = s_key[i];
            int r = 0;
#pragma unroll 4
            for (int j = 0; j < found; ++j) r += s_key[j] > x;
            if (r < a.n) {
                cand[r] = key_value(x);
                cand_at[r] = x0 + (int)~(uint32_t)x;
            }
        }
        if (tid >= found && tid < a.n) cand[tid] = -INFINITY;
        return;
    }
    // one after the other: the largest logit behind the last one taken
    float last = INFINITY;
    int last_at = -1;
    for (int r = 0; r < a.n; ++r) {
        float best = -INFINITY;
        int at = INT_MAX;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int p = place<T>(tid, k) - shift;
            const bool open = v[k] < last || (v[k] == last && p > last_at);
            if (open && (v[k] > best || (v[k] == best && p < at)) && v[k] > -INFINITY) {
                best = v[k];
                at = p;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, best, o);
            const int p = __shfl_xor_sync(0xffffffffu, at, o);
            if (y > best || (y == best && p < at)) {
                best = y;
                at = p;
            }
        }
        __syncthreads();
        if (lane == 0) {
            s_bestv[warp] = best;
            s_best[warp] = at;
        }
        __syncthreads();
        best = s_bestv[0];
        at = s_best[0];
        for (int w = 1; w < kWarps; ++w)
            if (s_bestv[w] > best || (s_bestv[w] == best && s_best[w] < at)) {
                best = s_bestv[w];
                at = s_best[w];
            }
        last = best;
        last_at = at;
        if (tid == 0) {
            cand[r] = best;
            cand_at[r] = x0 + at;
        }
    }
}

// A candidate's place in the order: its score (value and rest) as a whole number
// of the same order, 0 for none; then the lower row, the higher logit, the lower
// token.
struct Place {
    uint64_t score, tie;
};
__device__ __forceinline__ bool before(const Place &x, const Place &y) {
    return x.score > y.score || (x.score == y.score && x.tie > y.tie);
}

constexpr int kHeld = 8;       // candidates a thread keeps in registers

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamArgs a) {
    __shared__ float2 s_add[kMaxBeams];     // score - log-sum-exp; -inf: no candidates
    __shared__ uint8_t s_done[kMaxBeams];
    __shared__ Place s_place[kCap];
    __shared__ int s_token[kCap];
    __shared__ uint64_t s_rank[4][kWarps];  // each warp's ceil(n / 8)-th, n / 4, n / 2 and n-th largest maximum
    __shared__ int s_count;
    __shared__ Place s_best[kWarps];
    __shared__ int s_best_token[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.x;
    griddep_wait();
    const int lists = a.chunks * a.beams, per_beam = a.chunks * a.n, total = lists * a.n;
    const float *cand = a.cand + (int64_t)g * total;
    const int32_t *cand_at = a.cand_at + (int64_t)g * total;
    // candidate x in the order in which threads take them: the best of every
    // chunk first, then all second ones, and so on, so that the first few are
    // most of what is looked for; where it lies
    auto lies = [&](int x) {
        const int rank = a.div ? (int)__umulhi(x, a.div) : x / lists;
        return (x - rank * lists) * a.n + rank;
    };
    float held[kHeld];
    int held_at[kHeld], held_in[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int x = tid + k * kThreads;
        held_in[k] = x < total ? lies(x) : 0;
        held[k] = x < total ? cand[held_in[k]] : -INFINITY;
        held_at[k] = x < total ? cand_at[held_in[k]] : 0;
    }
    for (int b = warp; b < a.beams; b += kWarps) {
        const int row = g * a.beams + b;
        const float cum = a.scores[row];
        const bool done = a.finished && a.finished[row];
        float2 add = make_float2(-INFINITY, 0.f);
        if (isfinite(cum)) {
            if (done) {
                add.x = cum;
            } else {
                const PartHead *h = a.heads + (int64_t)row * a.chunks;
                const PartHead mine = lane < a.chunks ? h[lane] : PartHead{0.f, 0.f, -INFINITY, 0.f};
                float top = mine.top;
                for (int c = lane + 32; c < a.chunks; c += 32) top = fmaxf(top, h[c].top);
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (top < INFINITY && top > -INFINITY) {
                    float sum = 0.f, rest = 0.f;
                    for (int c = lane; c < a.chunks; c += 32) {
                        const PartHead x = c == lane ? mine : h[c];
                        const float w = expf(x.top - top);
                        const float y = __fmul_rn(x.sum, w);
                        add2(sum, rest, y, __fmaf_rn(x.sum, w, -y) + x.rest * w);
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1)
                        add2(sum, rest, __shfl_xor_sync(0xffffffffu, sum, o), __shfl_xor_sync(0xffffffffu, rest, o));
                    // log(sum) = k log 2 + log(m), m in [0.75, 1.5): log(m) is
                    // small, and its fp32 rounding with it
                    int k;
                    float m = frexpf(sum, &k);          // [0.5, 1)
                    if (m < 0.75f) {
                        m *= 2.f;
                        --k;
                    }
                    const double z = (double)cum - (double)top - k * 0.693147180559945309417 -
                                     ((double)logf(m) + (double)(rest / sum));
                    add.x = (float)z;
                    add.y = (float)(z - (double)add.x);
                }
            }
        }
        if (lane == 0) {
            s_add[b] = isfinite(add.x) ? add : make_float2(-INFINITY, 0.f);
            s_done[b] = done;
        }
    }
    if (tid < 4 * kWarps) s_rank[tid / kWarps][tid % kWarps] = 0;
    if (tid == 0) s_count = 0;
    __syncthreads();
    // the place of the candidate that lies at i; a finished beam's one is its
    // first
    auto place_of = [&](int i, float logit) -> Place {
        const int b = i / per_beam;
        float2 add = s_add[b];
        if (s_done[b]) {
            if (i != b * per_beam) return Place{0, 0};
            logit = 0.f;
        } else {
            if (!(logit > -INFINITY)) return Place{0, 0};
            add2(add.x, add.y, logit, 0.f);
        }
        // (a beam without candidates, or a score below fp32's range)
        if (!(add.x > -INFINITY)) return Place{0, 0};
        // (of equal logits of a beam, the one that lies first has the lower
        // token; per_beam is below 2^25)
        return Place{(uint64_t)order_key(add.x) << 32 | order_key(add.y),
                     (uint64_t)(kMaxBeams - 1 - b) << 57 | (uint64_t)order_key(logit) << 25 | (0x1ffffff - (i - b * per_beam))};
    };
    Place place[kHeld];
    uint64_t top = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        place[k] = tid + k * kThreads < total ? place_of(held_in[k], held[k]) : Place{0, 0};
        top = max(top, place[k].score);
    }
    // (the chunks' best ones are among those held)
    top = sort_warp(top, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane == (a.n + (8 >> i) - 1) / (8 >> i) - 1) s_rank[i][warp] = top;
    __syncthreads();
    // a score that 8, 4, 2 or 1 of the warps reach with an eighth, a fourth, ...
    // of n maxima each: the largest of those bounds
    uint64_t bound = s_rank[0][0], first = 0, second = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        bound = min(bound, s_rank[0][w]);
        second = max(second, min(first, s_rank[2][w]));
        first = max(first, s_rank[2][w]);
    }
    bound = max(max(bound, fourth_of_8(s_rank[1])), max(second, (uint64_t)1));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) bound = max(bound, s_rank[3][w]);
    auto collect = [&](const Place &x, int i, int at) {
        const int k = atomicAdd(&s_count, 1);
        if (k < kCap) {
            s_place[k] = x;
            s_token[k] = s_done[i / per_beam] ? a.pad : at;
        }
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
        if (place[k].score >= bound) collect(place[k], held_in[k], held_at[k]);
#pragma unroll 1
    for (int x = tid + kHeld * kThreads; x < total; x += kThreads) {
        const int i = lies(x);
        const Place p = place_of(i, cand[i]);
        if (p.score >= bound) collect(p, i, cand_at[i]);
    }
    __syncthreads();
    const int found = s_count;
    float *os = a.out_scores + (int64_t)g * a.n;
    int32_t *orow = a.out_rows + (int64_t)g * a.n, *ot = a.out_tokens + (int64_t)g * a.n;
    auto put = [&](int r, const Place &x, int token) {
        os[r] = key_value(x.score);
        orow[r] = g * a.beams + kMaxBeams - 1 - (int)(x.tie >> 57);
        ot[r] = token;
    };
    if (found <= kCap) {
        for (int i = tid; i < found; i += kThreads) {
            const Place x = s_place[i];
            int r = 0;
#pragma unroll 4
            for (int j = 0; j < found; ++j) r += before(s_place[j], x);
            if (r < a.n) put(r, x, s_token[i]);
        }
        for (int r = found + tid; r < a.n; r += kThreads) {
            os[r] = -INFINITY;
            orow[r] = ot[r] = -1;
        }
        return;
    }
    // one after the other, each the best behind the last one
    Place last{~0ull, ~0ull};
    for (int r = 0; r < a.n; ++r) {
        Place best{0, 0};
        int token = -1;
#pragma unroll 1
        for (int i = tid; i < total; i += kThreads) {
            const Place p = place_of(i, cand[i]);
            if (before(last, p) && before(p, best)) {
                best = p;
                token = s_done[i / per_beam] ? a.pad : cand_at[i];
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            Place y;
            y.score = __shfl_xor_sync(0xffffffffu, best.score, o);
            y.tie = __shfl_xor_sync(0xffffffffu, best.tie, o);
            const int t = __shfl_xor_sync(0xffffffffu, token, o);
            if (before(y, best)) {
                best = y;
                token = t;
            }
        }
        __syncthreads();
        if (lane == 0) {
            s_best[warp] = best;
            s_best_token[warp] = token;
        }
        __syncthreads();
        best = s_best[0];
        token = s_best_token[0];
        for (int w = 1; w < kWarps; ++w)
            if (before(s_best[w], best)) {
                best = s_best[w];
                token = s_best_token[w];
            }
        last = best;
        if (tid == 0) put(r, best, token);
    }
}

// ------------------------------------------------------------------ states

constexpr int kCopyThreads = 256, kInFlight = 8;

// dst[o][i] = src[o][index[i]], V bytes a chunk: a CTA takes a stretch of one
// row, eight chunks in flight a thread.
template <class V>
__global__ void __launch_bounds__(kCopyThreads)
    state_reorder_kernel(const V *src, V *dst, const int32_t *index, int32_t n_src, int32_t n_dst, int64_t chunks,
                         int64_t tiles) {
    const int64_t row = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int64_t o = row / n_dst;
    griddep_wait();
    const int from = index[row % n_dst];
    if ((unsigned)from >= (unsigned)n_src) return;
    const V *s = src + (o * n_src + from) * chunks;
    V *d = dst + row * chunks;
    const int64_t x0 = tile * kCopyThreads * kInFlight + threadIdx.x;
    V v[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
        if (x0 + u * kCopyThreads < chunks) v[u] = s[x0 + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
        if (x0 + u * kCopyThreads < chunks) d[x0 + u * kCopyThreads] = v[u];
}

template <class V>
cudaError_t launch_reorder(const void *src, void *dst, const int32_t *index, int64_t outer, int32_t n_src, int32_t n_dst,
                           int64_t row_bytes, cudaStream_t stream) {
    const int64_t chunks = row_bytes / sizeof(V), tiles = (chunks + kCopyThreads * kInFlight - 1) / (kCopyThreads * kInFlight);
    if (tiles > INT32_MAX || outer * n_dst > INT32_MAX / tiles) return cudaErrorInvalidValue;
    return launch_behind(state_reorder_kernel<V>, dim3((unsigned)(outer * n_dst * tiles)), kCopyThreads, 0, 1, stream, static_cast<const V *>(src),
                         static_cast<V *>(dst), index, n_src, n_dst, chunks, tiles);
}

bool bad(const void *p, uintptr_t align) { return !p || ((uintptr_t)p & (align - 1)); }

bool overlap(const void *x, size_t nx, const void *y, size_t ny) {
    const uintptr_t a = (uintptr_t)x, b = (uintptr_t)y;
    return a < b + ny && b < a + nx;
}

bool beam_shape_ok(int32_t groups, int32_t beams, int32_t vocab, int32_t n_out) {
    if (groups <= 0 || beams <= 0 || beams > kMaxBeams || vocab <= 0 || vocab > (1 << 30) || n_out <= 0 || n_out > kMaxOut)
        return false;
    const int64_t chunks = (vocab + kUneven - 1) / kUneven;
    return (int64_t)groups * beams * chunks <= INT32_MAX && beams * chunks * n_out <= INT32_MAX / 2;
}

template <class T>
cudaError_t launch_beam(BeamArgs a, cudaStream_t stream) {
    // (several waves: the joins' CTAs would only take the parts' places, 113
    // instead of 73 us for 4096 of them)
    a.early = a.groups * a.beams * a.chunks <= 2 * device_sm_count();
    const int64_t lists = (int64_t)a.chunks * a.beams;
    a.div = lists > 1 && lists * lists * a.n < (INT64_C(1) << 32) ? (uint32_t)(((INT64_C(1) << 32) + lists - 1) / lists) : 0;
    const cudaError_t e =
        launch_behind(beam_part_kernel<T>, dim3((unsigned)(a.groups * a.beams * a.chunks)), kThreads, 0, 1, stream, a);
    if (e != cudaSuccess) return e;
    return launch_behind(beam_join_kernel, dim3((unsigned)a.groups), kThreads, 0, 1, stream, a);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" {

size_t kvp_beam_workspace_size(int32_t groups, int32_t beams, int32_t vocab, int32_t n_out) {
    if (!beam_shape_ok(groups, beams, vocab, n_out)) return 0;
    const size_t parts = (size_t)groups * beams * ((vocab + kUneven - 1) / kUneven);
    return parts * (sizeof(PartHead) + (size_t)n_out * 8);
}

int kvp_beam_select(const void *logits, int32_t logits_type, int64_t row_stride, const float *scores,
                    const uint8_t *finished, int32_t pad_token, int32_t groups, int32_t beams, int32_t vocab,
                    int32_t n_out, float *out_scores, int32_t *out_rows, int32_t *out_tokens, void *workspace,
                    size_t ws_bytes, void *stream) {
    if (!beam_shape_ok(groups, beams, vocab, n_out) || row_stride < 0 || logits_type < KVP_F32 || logits_type > KVP_F16)
        return KVP_ERR_INVALID;
    const int size = logits_type == KVP_F32 ? 4 : 2;
    if (bad(logits, size) || bad(scores, 4) || bad(out_scores, 4) || bad(out_rows, 4) || bad(out_tokens, 4) ||
        bad(workspace, 16) || ws_bytes < kvp_beam_workspace_size(groups, beams, vocab, n_out))
        return KVP_ERR_INVALID;
    // a request's results are written while others' scores are still read; its own
    // are read by then, so that new scores may take the old ones' places
    const size_t rows = (size_t)groups * beams, results = (size_t)groups * n_out * 4;
    const bool in_place = out_scores == scores && n_out == beams;
    if (!in_place && overlap(out_scores, results, scores, rows * 4)) return KVP_ERR_INVALID;
    if (overlap(out_rows, results, scores, rows * 4) || overlap(out_tokens, results, scores, rows * 4)) return KVP_ERR_INVALID;
    if (finished && (overlap(out_scores, results, finished, rows) || overlap(out_rows, results, finished, rows) ||
                     overlap(out_tokens, results, finished, rows)))
        return KVP_ERR_INVALID;
    if (!stream && stream_capturing(nullptr)) return KVP_ERR_STATE;
    BeamArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.scores = scores;
    a.finished = finished;
    a.pad = pad_token; a.groups = groups; a.beams = beams; a.vocab = vocab; a.n = n_out;
    // (rows off 16-byte boundaries: the pieces of a chunk reach over its ends)
    const bool even = ((uintptr_t)logits & 15) == 0 && row_stride * size % 16 == 0;
    a.step = even ? kChunk : kUneven;
    a.chunks = (vocab + a.step - 1) / a.step;
    a.out_scores = out_scores; a.out_rows = out_rows; a.out_tokens = out_tokens;
    const size_t parts = (size_t)groups * beams * a.chunks;
    a.heads = static_cast<PartHead *>(workspace);
    a.cand = reinterpret_cast<float *>(a.heads + parts);
    a.cand_at = reinterpret_cast<int32_t *>(a.cand + parts * n_out);
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = logits_type == KVP_F32    ? launch_beam<float>(a, st)
                          : logits_type == KVP_BF16 ? launch_beam<__nv_bfloat16>(a, st)
                                                    : launch_beam<__half>(a, st);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

int kvp_state_reorder(const void *src, void *dst, const int32_t *index, int64_t outer, int32_t n_src, int32_t n_dst,
                      int64_t row_bytes, void *stream) {
    if (outer < 0 || n_src < 0 || n_dst < 0 || row_bytes < 0) return KVP_ERR_INVALID;
    if (outer == 0 || n_dst == 0 || row_bytes == 0) return KVP_OK;
    if (n_src == 0) return KVP_OK;              // no index is inside
    if (!src || !dst || bad(index, 4) || outer > INT64_MAX / std::max(n_src, n_dst) / row_bytes) return KVP_ERR_INVALID;
    const uintptr_t s = (uintptr_t)src, d = (uintptr_t)dst;
    if (s < d + (uint64_t)outer * n_dst * row_bytes && d < s + (uint64_t)outer * n_src * row_bytes) return KVP_ERR_INVALID;
    if (!stream && stream_capturing(nullptr)) return KVP_ERR_STATE;
    const uintptr_t all = s | d | (uintptr_t)row_bytes;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (all % 16 == 0)
        e = launch_reorder<uint4>(src, dst, index, outer, n_src, n_dst, row_bytes, st);
    else if (all % 4 == 0)
        e = launch_reorder<uint32_t>(src, dst, index, outer, n_src, n_dst, row_bytes, st);
    else
        e = launch_reorder<unsigned char>(src, dst, index, outer, n_src, n_dst, row_bytes, st);
    return e == cudaSuccess ? KVP_OK : e == cudaErrorInvalidValue ? KVP_ERR_INVALID : KVP_ERR_CUDA;
}

}  // extern "C"
