// Which pages of a paged sequence a query should read (sm_103a): bounds of
// each page's keys, a score of each page from them, and the selection.
//
//   bounds   lo_i = min, hi_i = max over the page's keys of dim i;
//   score    scale * sum over the group's query heads and the dims of
//            max(q_i lo_i, q_i hi_i)
//          = scale * ((sum_h min(q_h, 0)) . lo + (sum_h max(q_h, 0)) . hi),
//            as lo <= hi: one dot product of length 2 d a page, whatever the
//            group's size;
//   select   the sinks, the last pages, and the best of the others.
//
// All three take tables and lengths from device memory, so a captured call
// follows them as they change.
//
// Measured on one GB300: scores of 64 sequences of about 1900 pages (8 kv heads,
// d 128) 79 us with their newest page's bounds, 6.1 TB/s of 485 MB, 90% of the
// copy peak; selection of 128 out of about 6100 pages for 2048 rows 21.9 us
// (50 MB; 926 instructions a warp at half of the issue slots, and barriers),
// one sequence's 64 of 2063 4.8 us; 128 out of about 50000 for 128 rows, in
// several passes over each row, 205 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/kvp.h"
#include "kvp_internal.h"
#include "launch.cuh"
#include "query_rows.cuh"

namespace kvp {
namespace {

// ------------------------------------------------------------------ bounds

constexpr int kBoundWarps = 4;

struct BoundsArgs {
    const uint4 *k;         // 16-byte chunks
    uint4 *bounds;
    const int32_t *tables, *lens;
    int32_t S, MB, L, Hkv, NB, bs, n_new, pages;
};

template <bool MAX>
__device__ __forceinline__ uint32_t pick2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&a), y = *reinterpret_cast<const __nv_bfloat162 *>(&b);
    const __nv_bfloat162 r = MAX ? __hmax2_nan(x, y) : __hmin2_nan(x, y);
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <bool MAX>
__device__ __forceinline__ uint4 pick(uint4 a, uint4 b) {
    return make_uint4(pick2<MAX>(a.x, b.x), pick2<MAX>(a.y, b.y), pick2<MAX>(a.z, b.z), pick2<MAX>(a.w, b.w));
}
template <bool MAX>
__device__ __forceinline__ uint4 pick_across(uint4 a, int step) {
    uint4 b;
    b.x = __shfl_xor_sync(0xffffffffu, a.x, step);
    b.y = __shfl_xor_sync(0xffffffffu, a.y, step);
    b.z = __shfl_xor_sync(0xffffffffu, a.z, step);
    b.w = __shfl_xor_sync(0xffffffffu, a.w, step);
    return pick<MAX>(a, b);
}

// A warp per (page, kv head, layer): its rows are one contiguous run, read 512
// bytes an instruction, 16 bytes a lane, each lane keeping its 8 dims.
template <int D>
__global__ void __launch_bounds__(32 * kBoundWarps) page_bounds_kernel(const BoundsArgs a) {
    constexpr int CH = D / 8, RPI = 32 / CH;     // chunks per row, rows per instruction
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.y;
    const int64_t unit = (int64_t)blockIdx.x * kBoundWarps + warp;      // page-major over (layer, kv head)
    const int LH = a.L * a.Hkv;
    const int jj = (int)(unit / LH), lh = (int)(unit % LH);
    if (jj >= a.pages) return;
    const int n = (int)min((int64_t)max(a.lens[s], 0), (int64_t)a.MB * a.bs);
    const int j = max(0, n - a.n_new) / a.bs + jj;
    if ((int64_t)j * a.bs >= n) return;
    const int blk = a.tables[(int64_t)s * a.MB + j];
    if ((unsigned)blk >= (unsigned)a.NB) return;
    const int l = lh / a.Hkv, h = lh % a.Hkv;
    const int64_t page = ((int64_t)l * a.NB + blk) * a.Hkv + h;
    const int rows = min(a.bs, n - j * a.bs);
    const uint4 *src = a.k + page * a.bs * CH + lane;
    const int r0 = lane / CH;
    uint4 lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);    // +inf
    uint4 hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    constexpr int U = 8;
    for (int r = r0; r < rows; r += RPI * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // a row past the end: the first one again
            const int q = r + u * RPI;
            v[u] = src[(int64_t)((q < rows ? q : r) - r0) * CH];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            lo = pick<false>(lo, v[u]);
            hi = pick<true>(hi, v[u]);
        }
    }
#pragma unroll
    for (int step = 16; step >= CH; step >>= 1) {
        lo = pick_across<false>(lo, step);
        hi = pick_across<true>(hi, step);
    }
    if (lane < CH) {
        a.bounds[page * 2 * CH + lane] = lo;
        a.bounds[(page * 2 + 1) * CH + lane] = hi;
    }
}

// ------------------------------------------------------------------ scores

constexpr int kScoreWarps = 4;
constexpr int kScoreSteps = 4;      // groups of 16 pages per warp
constexpr int kScorePages = 16 * kScoreWarps * kScoreSteps;

struct ScoreArgs {
    QueryRows rows;
    const __nv_bfloat16 *q;
    const uint4 *bounds;
    float *scores;
    int64_t stride;
    int32_t L, Hq, Hkv, G, NB, chunks;
    float scale;
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x as the sum of three bf16 numbers (24 bits, all of an fp32's); what is not
// finite stands whole in the first
__device__ __forceinline__ void split3(float x, __nv_bfloat16 &a, __nv_bfloat16 &b, __nv_bfloat16 &c) {
    a = __float2bfloat16_rn(x);
    float r = x - __bfloat162float(a);
    if (!isfinite(r)) r = 0.f;
    b = __float2bfloat16_rn(r);
    c = __float2bfloat16_rn(r - __bfloat162float(b));
}

// A warp scores 16 pages at a time for up to QT query rows of one sequence:
// pages are the rows of mma.sync's A operand, read straight from global memory
// (the contraction may run over the dims in any order, so a lane's operand is
// 16 contiguous bytes of its page, four lanes to 64), and the queries' summed
// parts the columns of B.  Each fp32 part is three bf16 numbers, so that the
// products carry all of its bits; the three are columns of their own, added up
// at the end.  QT = 1 has its three columns in one B tile, QT = 8 in three.
template <int D, int QT>
__global__ void __launch_bounds__(32 * kScoreWarps) page_score_kernel(const ScoreArgs a) {
    constexpr int K = 2 * D, C = K / 32;      // 32-value chunks of a page's bounds
    constexpr int ROW = K + 32;               // shared-memory row: two rows never meet in a bank
    constexpr int NT = QT == 1 ? 1 : 3;
    __shared__ __align__(16) __nv_bfloat16 s_part[3 * QT][ROW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int lh = blockIdx.y, l = lh / a.Hkv, h = lh % a.Hkv;
    griddep_wait();
    // which query rows, which pages
    int r0, nr, seq;
    const int chunk = (int)(blockIdx.x % a.chunks);
    if (!a.rows.tile(QT, blockIdx.x / a.chunks, r0, nr, seq)) return;
    const int last = a.rows.pages(seq, r0 + nr - 1);       // pages that the last row sees
    const int p_begin = chunk * kScorePages;
    if (p_begin >= last) return;
    // the warp's first pages and their bounds while the queries come in
    const int32_t *table = a.rows.tables + (int64_t)seq * a.rows.MB;
    int ba, bb;              // blocks of pages p0 + g and p0 + g + 8
    auto find = [&](int p0) {
        ba = p0 + g < last ? table[p0 + g] : -1;
        bb = p0 + g + 8 < last ? table[p0 + g + 8] : -1;
    };
    int p0 = p_begin + warp * 16;
    find(p0);
    uint4 va[C], vb[C];
    auto fetch = [&]() {
        const bool oka = (unsigned)ba < (unsigned)a.NB, okb = (unsigned)bb < (unsigned)a.NB;
        const uint4 *xa = a.bounds + (((int64_t)l * a.NB + (oka ? ba : 0)) * a.Hkv + h) * (K / 8) + t;
        const uint4 *xb = a.bounds + (((int64_t)l * a.NB + (okb ? bb : 0)) * a.Hkv + h) * (K / 8) + t;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            va[c] = oka ? __ldg(xa + 4 * c) : make_uint4(0, 0, 0, 0);
            vb[c] = okb ? __ldg(xb + 4 * c) : make_uint4(0, 0, 0, 0);
        }
    };
    fetch();
    // E dims of a row per thread: one, so that all threads have work, or eight
    constexpr int E = QT == 1 ? 1 : 8, U = 4;         // heads in flight
    using Dims = typename std::conditional<QT == 1, unsigned short, uint4>::type;
    for (int i = threadIdx.x; i < QT * D / E; i += blockDim.x) {
        const int r = i / (D / E), e0 = i % (D / E) * E;
        float neg[E] = {}, pos[E] = {};
        if (r < nr) {
            const __nv_bfloat16 *q = a.q + (((int64_t)l * a.rows.T + r0 + r) * a.Hq + h * a.G) * D + e0;
            for (int x = 0; x < a.G; x += U) {
                Dims v[U];
#pragma unroll
                for (int y = 0; y < U; ++y)
                    v[y] = x + y < a.G ? *reinterpret_cast<const Dims *>(q + (int64_t)(x + y) * D) : Dims();
#pragma unroll
                for (int y = 0; y < U; ++y)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float f = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(&v[y])[e]);
                        neg[e] += f > 0.f ? 0.f : f;      // (a NaN goes into both)
                        pos[e] += f < 0.f ? 0.f : f;
                    }
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            split3(neg[e], s_part[r][e0 + e], s_part[QT + r][e0 + e], s_part[2 * QT + r][e0 + e]);
            split3(pos[e], s_part[r][D + e0 + e], s_part[QT + r][D + e0 + e], s_part[2 * QT + r][D + e0 + e]);
        }
    }
    __syncthreads();
    uint4 b1[QT == 1 ? C : 1];
    if constexpr (QT == 1) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            b1[c] = g < 3 ? *reinterpret_cast<const uint4 *>(&s_part[g < 3 ? g : 0][32 * c + 8 * t]) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll 1
    for (int step = 0; step < kScoreSteps; ++step) {
        if (p0 >= last) return;
        const int pa = p0 + g, pb = pa + 8;
        const bool oka = (unsigned)ba < (unsigned)a.NB, okb = (unsigned)bb < (unsigned)a.NB;
        p0 += 16 * kScoreWarps;
        if (step + 1 < kScoreSteps) find(p0);
        float acc[NT][4] = {};
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint4 b;
                if constexpr (QT == 1)
                    b = b1[c];
                else
                    b = *reinterpret_cast<const uint4 *>(&s_part[n * QT + g][32 * c + 8 * t]);
                mma(acc[n], va[c].x, vb[c].x, va[c].y, vb[c].y, b.x, b.y);
                mma(acc[n], va[c].z, vb[c].z, va[c].w, vb[c].w, b.z, b.w);
            }
        }
        if constexpr (QT == 1) {
            // columns 0, 1 are lane t = 0's, column 2 lane t = 1's
            const float la = __shfl_down_sync(0xffffffffu, acc[0][0], 1), lb = __shfl_down_sync(0xffffffffu, acc[0][2], 1);
            if (t == 0) {
                float *out = a.scores + (((int64_t)l * a.rows.T + r0) * a.Hkv + h) * a.stride;
                if (pa < last) out[pa] = oka ? (acc[0][0] + (acc[0][1] + la)) * a.scale : -INFINITY;
                if (pb < last) out[pb] = okb ? (acc[0][2] + (acc[0][3] + lb)) * a.scale : -INFINITY;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {       // query columns 2 t, 2 t + 1
                const int r = 2 * t + e;
                if (r >= nr) continue;
                const int seen = a.rows.pages(seq, r0 + r);
                float *out = a.scores + (((int64_t)l * a.rows.T + r0 + r) * a.Hkv + h) * a.stride;
                if (pa < seen) out[pa] = oka ? (acc[0][e] + (acc[1][e] + acc[2][e])) * a.scale : -INFINITY;
                if (pb < seen) out[pb] = okb ? (acc[0][2 + e] + (acc[1][2 + e] + acc[2][2 + e])) * a.scale : -INFINITY;
            }
        }
        if (step + 1 < kScoreSteps) fetch();
    }
}

// --------------------------------------------------------------- selection

constexpr int kSelThreads = 256;
constexpr int kSelCap = 128;         // keys above the bound that a warp lists

struct SelectArgs {
    QueryRows rows;
    const float *scores;
    int64_t stride;
    int32_t *selected;
    int32_t Hkv, budget, sink, recent;
};

// Scores as unsigned keys of the same order: NaN above everything (a sum that
// is NaN is the one positive NaN 0x7fffffff), -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kStays = 0xffffffffu;    // sinks and the last pages: above every score

// The larger of two lanes' keys to the lower lane, down to a descending warp.
__device__ __forceinline__ uint32_t sort_warp(uint32_t x, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {
            const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
            const bool up = ((lane & j) == 0) == ((lane & k) == 0);     // this lane takes the larger
            x = up ? max(x, y) : min(x, y);
        }
    return x;
}

// The k-th largest key, of which all but the lowest `bits` bits are in `cut`,
// from the number of keys >= t; above: how many are larger.  It ends early at a
// t that exactly k keys reach (after about half of the bits where keys do not
// repeat): those are then all above `cut`, and none of the equal ones is due.
template <class Count>
__device__ __forceinline__ void find_cut(int bits, int k, uint32_t &cut, int &above, Count count) {
    for (int b = bits - 1; b >= 0; --b) {
        const uint32_t t = cut | 1u << b;
        const int c = count(t);
        if (c == k) {
            cut = t - 1;
            above = k;
            return;
        }
        if (c > k) cut = t;
    }
    above = cut == 0xffffffffu ? 0 : count(cut + 1);
}

// A CTA per (layer, query row, kv head) of at most W * 32 * E pages: k = budget
// - sinks - last pages of those in between are to be found.  Page sink + W * 32
// e + thread is the thread's e-th.
//   1. The scores, rounded to bf16 and packed in pairs (rounding keeps the
//      order, if not strictly), which is what most of them are looked at as:
//      half of the registers and of the instructions.
//   2. A bound that at least k of them reach, from the threads' maxima (of four
//      parts each where k is above W * 32): each warp's ceil(k / W)-th largest
//      maximum, the smallest of those.
//   3. The pages that reach it (a NaN always does), few more than k, go on the
//      warps' lists with their scores as they are, and one warp (short lists: 22
//      us for 2048 rows, all warps 24) or all of them (k above W * 32: 300 pages
//      31 us, one warp 55) find the k-th largest of those.  Where the lists do
//      not hold them (many equal scores, k above W * 70 or so), all warps look
//      through all keys instead.
//   4. Keys above it, and those equal to it, as two bit maps by page; counts
//      up to a word give every chosen page its place.
template <int W, int E>
__global__ void __launch_bounds__(32 * W, W <= 8 ? 48 / W : 1) page_select_kernel(const SelectArgs a) {
    constexpr int WORDS = W * E, PER = (WORDS + 32 * W - 1) / (32 * W), STEP = 32 * W;
    __shared__ uint32_t s_key[W][kSelCap];
    __shared__ uint16_t s_at[W][kSelCap];
    __shared__ uint32_t s_up[WORDS], s_eq[WORDS];
    __shared__ uint32_t s_warp[W], s_hits[W];
    __shared__ uint32_t s_cut;
    __shared__ int s_above, s_count[34];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x;
    griddep_wait();
    const int r = (int)(row / a.Hkv % a.rows.T);
    const int seq = a.rows.sequence(r);
    if (seq < 0) return;
    const int n = a.rows.pages(seq, r);
    const int lo = a.sink, len = n - a.recent - lo, k = a.budget - a.sink - a.recent;
    const float *score = a.scores + row * a.stride + lo;
    int32_t *out = a.selected + row * a.budget;
    if (n <= a.budget) {
        for (int j = tid; j < a.budget; j += STEP) out[j] = j < n ? j : -1;
        return;
    }
    // pair i: pages 2 i (low half) and 2 i + 1 of the thread
    __nv_bfloat162 pair[E / 2];
    {
        float x[E];
        if (len == STEP * E) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = __ldg(score + e * STEP + tid);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = e * STEP + tid < len ? __ldg(score + e * STEP + tid) : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) pair[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    }
    for (int j = tid; j < lo; j += STEP) out[j] = j;
    for (int j = tid; j < a.recent; j += STEP) out[a.budget - a.recent + j] = n - a.recent + j;
    if (k == 0) return;
    out += lo;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (tid + i * STEP < WORDS) s_up[tid + i * STEP] = s_eq[tid + i * STEP] = 0;
    if (tid < 34) s_count[tid] = 0;
    // maxima to bound it by: the threads', or of four parts of each one's pages
    constexpr int PARTS = E >= 8 ? 4 : 1;
    const bool few = k <= STEP * PARTS;
    uint32_t bound = 0;
    if (few && k > STEP) {
        // the warp's ceil(k / W)-th largest of 32 PARTS, by the 16 bits that a
        // bf16's key has
        const int rank = (k + W - 1) / W;
        uint32_t top[PARTS], at_least = 0;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            __nv_bfloat162 most = __floats2bfloat162_rn(-INFINITY, -INFINITY);
#pragma unroll
            for (int i = 0; i < E / 2 / PARTS; ++i) most = __hmax2(most, pair[q * (E / 2 / PARTS) + i]);
            top[q] = score_key(fmaxf(__low2float(most), __high2float(most))) >> 16;
        }
#pragma unroll 1
        for (uint32_t b = 0x8000; b; b >>= 1) {
            int c = 0;
#pragma unroll
            for (int q = 0; q < PARTS; ++q) c += __popc(__ballot_sync(0xffffffffu, top[q] >= (at_least | b)));
            if (c >= rank) at_least |= b;
        }
        // (the low half of a negative bf16's key is ones)
        if (lane == 0) s_warp[warp] = at_least << 16 | (at_least & 0x8000 ? 0u : 0xffffu);
    } else if (few) {
        __nv_bfloat162 most = __floats2bfloat162_rn(-INFINITY, -INFINITY);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) most = __hmax2(most, pair[i]);      // (a NaN is not taken)
        const uint32_t top = sort_warp(score_key(fmaxf(__low2float(most), __high2float(most))), lane);
        if (lane == (k + W - 1) / W - 1) s_warp[warp] = top;
    }
    __syncthreads();
    uint32_t mine = 0;               // the thread's pages that reach the bound, even ones in the low half
    if (few) {
        bound = s_warp[0];
#pragma unroll
        for (int w = 1; w < W; ++w) bound = min(bound, s_warp[w]);
        const __nv_bfloat162 least = __float2bfloat162_rn(key_score(bound));
#pragma unroll
        for (int i = 0; i < E / 2; ++i) mine |= __hgeu2_mask(pair[i], least) & (0x10001u << i);
        const int have = max(0, min(E, (len - tid + STEP - 1) / STEP));
        mine &= ((1u << (have + 1) / 2) - 1u) | ((1u << have / 2) - 1u) << 16;
    }
    int at = __popc(mine);
    int hits = at;                   // up to this lane, then all of the warp's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, hits, o);
        if (lane >= o) hits += y;
    }
    at = hits - at;
    hits = __shfl_sync(0xffffffffu, hits, 31);
    while (mine) {
        const int b = __ffs(mine) - 1;
        mine &= mine - 1;
        if (at < kSelCap) s_at[warp][at] = (uint16_t)((2 * (b & 15) + (b >> 4)) * STEP + tid);
        ++at;
    }
    __syncwarp();
    if (hits <= kSelCap)
        for (int i = lane; i < hits; i += 32) s_key[warp][i] = score_key(score[s_at[warp][i]]);
    if (lane == 0) s_hits[warp] = few ? hits : kSelCap + 1;
    __syncthreads();
    int most = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) most = max(most, (int)s_hits[w]);
    uint32_t cut = 0;                // the k-th largest key
    int above = 0;                   // keys larger than it
    int step = 0;                    // (counts of all warps, each with a word of its own)
    auto total = [&](int c) {
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) atomicAdd(&s_count[step], c);
        __syncthreads();
        return s_count[step++];
    };
    if (most <= kSelCap) {
        if (k > STEP) {
            uint32_t held[kSelCap / 32];
#pragma unroll
            for (int i = 0; i < kSelCap / 32; ++i) held[i] = 32 * i + lane < hits ? s_key[warp][32 * i + lane] : 0u;
            find_cut(32, k, cut, above, [&](uint32_t t) {      // keys of at least t
                int c = 0;
#pragma unroll
                for (int i = 0; i < kSelCap / 32; ++i) c += held[i] >= t;
                return total(c);
            });
        } else if (warp == 0) {
            constexpr int H = W <= 8 ? 2 : 1;        // 32 * H keys of each list in registers
            uint32_t x[W * H];
            uint32_t any = 0, all = 0xffffffffu;
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int j = 32 * i + lane;
                    x[w * H + i] = j < (int)s_hits[w] ? s_key[w][j] : 0u;
                    if (j < (int)s_hits[w]) {
                        any |= x[w * H + i];
                        all &= x[w * H + i];
                    }
                }
            if (most > 32 * H)
                for (int w = 0; w < W; ++w)
                    for (int j = 32 * H + lane; j < (int)s_hits[w]; j += 32) {
                        any |= s_key[w][j];
                        all &= s_key[w][j];
                    }
            auto count = [&](uint32_t t) {           // keys of at least t
                int c = 0;
#pragma unroll
                for (int i = 0; i < W * H; ++i) c += x[i] >= t;
                if (most > 32 * H)
                    for (int w = 0; w < W; ++w)
                        for (int j = 32 * H + lane; j < (int)s_hits[w]; j += 32) c += s_key[w][j] >= t;
                return (int)__reduce_add_sync(0xffffffffu, c);
            };
            // the leading bits that all keys share need no test
            any = __reduce_or_sync(0xffffffffu, any);
            all = __reduce_and_sync(0xffffffffu, all);
            const int bits = any != all ? 32 - __clz(any ^ all) : 0;
            cut = bits == 32 ? 0u : all >> bits << bits;
            find_cut(bits, k, cut, above, count);
            if (lane == 0) {
                s_cut = cut;
                s_above = above;
            }
        }
        if (k <= STEP) {
            __syncthreads();
            cut = s_cut;
            above = s_above;
        }
        for (int i = lane; i < hits; i += 32) {
            const uint32_t x = s_key[warp][i];
            const int j = s_at[warp][i];
            if (x > cut) atomicOr(&s_up[j >> 5], 1u << (j & 31));
            if (x == cut) atomicOr(&s_eq[j >> 5], 1u << (j & 31));
        }
    } else {
        // (steps past the end are as low as -inf, and behind every page of that score)
        uint32_t key[E];
#pragma unroll
        for (int e = 0; e < E; ++e) key[e] = score_key(e * STEP + tid < len ? score[e * STEP + tid] : -INFINITY);
        find_cut(32, k, cut, above, [&](uint32_t t) {
            int c = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) c += key[e] >= t;
            return total(c);
        });
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t up = __ballot_sync(0xffffffffu, key[e] > cut), eq = __ballot_sync(0xffffffffu, key[e] == cut);
            if (lane == 0) {
                s_up[e * W + warp] = up;
                s_eq[e * W + warp] = eq;
            }
        }
    }
    __syncthreads();
    // places: words in page order, PER to a thread; counts of both maps in the
    // halves of one word
    static_assert(STEP * E <= 32768, "two 16-bit counts");
    uint32_t up[PER], eq[PER], here = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int w = tid * PER + i;
        up[i] = w < WORDS ? s_up[w] : 0u;
        eq[i] = w < WORDS ? s_eq[w] : 0u;
        here += __popc(up[i]) + (__popc(eq[i]) << 16);
    }
    uint32_t before = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) s_warp[warp] = before;
    __syncthreads();
    before -= here;
#pragma unroll
    for (int w = 0; w < W; ++w)
        if (w < warp) before += s_warp[w];
    int n_up = before & 0xffff, n_eq = before >> 16;
    const int left = k - above;                 // of the equal ones, the first
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        uint32_t any = up[i] | eq[i];
        while (any) {
            const int b = __ffs(any) - 1;
            any &= any - 1;
            const bool is_up = up[i] >> b & 1;
            if (is_up || n_eq < left) out[n_up + min(n_eq, left)] = lo + (tid * PER + i) * 32 + b;
            n_up += is_up;
            n_eq += !is_up;
        }
    }
}

// Longer rows: the budget-th largest key by a radix select over the row in
// global memory, 8 bits a pass, then the pages in order.
__global__ void __launch_bounds__(kSelThreads) page_select_long_kernel(const SelectArgs a) {
    __shared__ int s_bin[256];
    __shared__ int s_up[kSelThreads / 32], s_eq[kSelThreads / 32];
    __shared__ int s_digit, s_left;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x;
    griddep_wait();
    const int r = (int)(row / a.Hkv % a.rows.T);
    const int seq = a.rows.sequence(r);
    if (seq < 0) return;
    const int n = a.rows.pages(seq, r);
    const float *score = a.scores + row * a.stride;
    int32_t *out = a.selected + row * a.budget;
    if (n <= a.budget) {
        for (int j = tid; j < a.budget; j += kSelThreads) out[j] = j < n ? j : -1;
        return;
    }
    const int lo = a.sink, hi = n - a.recent;
    auto key_at = [&](int j) { return j < lo || j >= hi ? kStays : min(score_key(score[j]), kStays - 1); };
    uint32_t prefix = 0;
    int left = a.budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
        s_bin[tid] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += kSelThreads) {
            const uint32_t key = key_at(j);
            if (shift == 24 || ((key ^ prefix) >> (shift + 8)) == 0) atomicAdd(&s_bin[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int d = 255, m = left;
            while (s_bin[d] < m) m -= s_bin[d--];
            s_digit = d;
            s_left = m;
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        left = s_left;
        __syncthreads();
    }
    // keys above `prefix` and the first `left` of those equal to it, in order
    int base = 0, eq_base = 0;
    for (int j0 = 0; j0 < n; j0 += kSelThreads) {
        const int j = j0 + tid;
        const uint32_t key = j < n ? key_at(j) : 0u;
        const bool up = j < n && key > prefix, eq = j < n && key == prefix;
        const uint32_t mu = __ballot_sync(0xffffffffu, up), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            s_up[warp] = __popc(mu);
            s_eq[warp] = __popc(me);
        }
        __syncthreads();
        int bu = base, be = eq_base;
        for (int w = 0; w < kSelThreads / 32; ++w) {
            if (w < warp) {
                bu += s_up[w];
                be += s_eq[w];
            }
            base += s_up[w];
            eq_base += s_eq[w];
        }
        const uint32_t below = (1u << lane) - 1u;
        const int eq_before = be + __popc(me & below);
        if (up || (eq && eq_before < left)) out[bu + __popc(mu & below) + min(eq_before, left)] = j;
        __syncthreads();
    }
}

bool bad(const void *p, uintptr_t align) { return !p || ((uintptr_t)p & (align - 1)); }

// What the batch's arguments have to satisfy in every call.
bool batch_ok(const kvp_attn_desc *d, const int32_t *tables, const int32_t *lens, int32_t S, int32_t MB) {
    return attn_desc_ok(d) && d->kv_format == KVP_KV_BF16 && (int64_t)d->num_layers * d->num_kv_heads <= 65535 &&
           S > 0 && MB > 0 && (int64_t)MB * d->block_size <= INT32_MAX / 2 && !bad(tables, 4) && !bad(lens, 4);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" {

int kvp_page_bounds(const void *k_pool, const int32_t *block_tables, const int32_t *seq_lens, int32_t num_seqs,
                    int32_t max_blocks, int32_t n_new, const kvp_attn_desc *desc, void *bounds, void *stream) {
    if (!batch_ok(desc, block_tables, seq_lens, num_seqs, max_blocks) || bad(k_pool, 16) || bad(bounds, 16) || n_new < 0 ||
        num_seqs > 65535)
        return KVP_ERR_INVALID;
    if (!stream && stream_capturing(nullptr)) return KVP_ERR_STATE;
    if (n_new == 0) return KVP_OK;
    BoundsArgs a{};
    a.k = static_cast<const uint4 *>(k_pool);
    a.bounds = static_cast<uint4 *>(bounds);
    a.tables = block_tables;
    a.lens = seq_lens;
    a.S = num_seqs; a.MB = max_blocks; a.L = desc->num_layers; a.Hkv = desc->num_kv_heads;
    a.NB = desc->num_blocks; a.bs = desc->block_size; a.n_new = n_new;
    a.pages = (int32_t)std::min<int64_t>(max_blocks, ((int64_t)n_new + a.bs - 2) / a.bs + 1);
    const int64_t grid = ((int64_t)a.pages * a.L * a.Hkv + kBoundWarps - 1) / kBoundWarps;
    if (grid > INT32_MAX) return KVP_ERR_INVALID;
    const dim3 g((unsigned)grid, (unsigned)num_seqs);
    cudaError_t e;
    if (desc->head_dim == 64)
        e = launch_behind(page_bounds_kernel<64>, g, 32 * kBoundWarps, 0, 1, (cudaStream_t)stream, a);
    else
        e = launch_behind(page_bounds_kernel<128>, g, 32 * kBoundWarps, 0, 1, (cudaStream_t)stream, a);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

int kvp_page_scores(const void *q, const int32_t *q_start, int32_t num_q, const void *bounds,
                    const int32_t *block_tables, const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks,
                    const kvp_attn_desc *desc, float *scores, int64_t score_stride, void *stream) {
    if (!batch_ok(desc, block_tables, seq_lens, num_seqs, max_blocks) || bad(bounds, 16) || score_stride < max_blocks ||
        num_q < 0 || ((uintptr_t)q_start & 3) || (!q_start && num_q != num_seqs))
        return KVP_ERR_INVALID;
    if (num_q == 0) return KVP_OK;
    if (bad(q, 16) || bad(scores, 4)) return KVP_ERR_INVALID;
    if (!stream && stream_capturing(nullptr)) return KVP_ERR_STATE;
    ScoreArgs a{};
    a.rows = QueryRows{q_start, block_tables, seq_lens, num_seqs, num_q, max_blocks, desc->block_size};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.bounds = static_cast<const uint4 *>(bounds);
    a.scores = scores;
    a.stride = score_stride;
    a.L = desc->num_layers; a.Hq = desc->num_q_heads; a.Hkv = desc->num_kv_heads; a.G = a.Hq / a.Hkv;
    a.NB = desc->num_blocks;
    a.scale = desc->scale > 0.f ? desc->scale : 1.f / sqrtf((float)desc->head_dim);
    a.chunks = (max_blocks + kScorePages - 1) / kScorePages;
    const int64_t tiles = q_start ? QueryRows::tiles(num_q, num_seqs, 8) : num_q;
    if (tiles * a.chunks > INT32_MAX) return KVP_ERR_INVALID;
    const dim3 g((unsigned)(tiles * a.chunks), (unsigned)(a.L * a.Hkv));
    cudaStream_t st = (cudaStream_t)stream;
    const int threads = 32 * kScoreWarps;
    cudaError_t e;
    if (desc->head_dim == 64) {
        if (q_start)
            e = launch_behind(page_score_kernel<64, 8>, g, threads, 0, 1, st, a);
        else
            e = launch_behind(page_score_kernel<64, 1>, g, threads, 0, 1, st, a);
    } else {
        if (q_start)
            e = launch_behind(page_score_kernel<128, 8>, g, threads, 0, 1, st, a);
        else
            e = launch_behind(page_score_kernel<128, 1>, g, threads, 0, 1, st, a);
    }
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

int kvp_page_select(const float *scores, int64_t score_stride, const int32_t *q_start, int32_t num_q,
                    const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks, const kvp_attn_desc *desc,
                    int32_t budget, int32_t n_sink, int32_t n_recent, int32_t *selected, void *stream) {
    if (!batch_ok(desc, seq_lens, seq_lens, num_seqs, max_blocks) || score_stride < max_blocks || num_q < 0 ||
        ((uintptr_t)q_start & 3) || (!q_start && num_q != num_seqs) || budget <= 0 || n_sink < 0 || n_recent < 0 ||
        (int64_t)n_sink + n_recent > budget)
        return KVP_ERR_INVALID;
    if (num_q == 0) return KVP_OK;
    if (bad(scores, 4) || bad(selected, 4)) return KVP_ERR_INVALID;
    const int64_t grid = (int64_t)desc->num_layers * num_q * desc->num_kv_heads;
    if (grid > INT32_MAX) return KVP_ERR_INVALID;
    if (!stream && stream_capturing(nullptr)) return KVP_ERR_STATE;
    SelectArgs a{};
    a.rows = QueryRows{q_start, nullptr, seq_lens, num_seqs, num_q, max_blocks, desc->block_size};
    a.scores = scores;
    a.stride = score_stride;
    a.selected = selected;
    a.Hkv = desc->num_kv_heads; a.budget = budget; a.sink = n_sink; a.recent = n_recent;
    // the smallest kernel whose registers hold the longest row that the tables
    // allow; 1024 threads for rows that 256 do not hold
    const dim3 ctas((unsigned)grid);
    cudaError_t e;
    cudaStream_t st = (cudaStream_t)stream;
    if (max_blocks <= 256)
        e = launch_behind(page_select_kernel<4, 2>, ctas, 128, 0, 1, st, a);
    else if (max_blocks <= 1024)
        e = launch_behind(page_select_kernel<4, 8>, ctas, 128, 0, 1, st, a);
    else if (max_blocks <= 2048)
        e = launch_behind(page_select_kernel<8, 8>, ctas, 256, 0, 1, st, a);
    else if (max_blocks <= 4096)
        e = launch_behind(page_select_kernel<8, 16>, ctas, 256, 0, 1, st, a);
    else if (max_blocks <= 8192)
        e = launch_behind(page_select_kernel<8, 32>, ctas, 256, 0, 1, st, a);
    else if (max_blocks <= 32768)
        e = launch_behind(page_select_kernel<32, 32>, ctas, 1024, 0, 1, st, a);
    else
        e = launch_behind(page_select_long_kernel, ctas, kSelThreads, 0, 1, st, a);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

}  // extern "C"
