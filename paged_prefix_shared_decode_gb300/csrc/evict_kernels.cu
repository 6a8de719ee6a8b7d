// Eviction from the paged cache by accumulated attention weight (sm_103a):
// which tokens of a sequence stay, and the compaction of its pages.
//
// Selection, one CTA per (layer, sequence, kv head): the first `sink` and the
// last `recent` tokens stay, and of the rest the k = budget - sink - recent
// with the largest weight, equal weights by lowest position.  The k-th
// largest is found by a radix select over the weights as ordered 32-bit keys
// (11, 11 and 10 bits a pass, a histogram in shared memory), which reads the
// row three times from L2 and compares nothing; a sort would move it.  Then
// each warp takes a contiguous stretch of the row, so that one scan over the
// 16 warps' counts gives every kept token its place in position order.
//
// Compaction: kept token j of a (layer, kv head) moves to slot j of the
// sequence.  A row of K or V is d * 2 contiguous bytes and moves in 16-byte
// chunks.
//   - Sequences whose pages are all shared get fresh pages, sources and
//     destinations are disjoint, and every row moves on its own
//     (evict_copy_kernel): bound by HBM, with eight loads in flight a thread.
//   - Pages that the sequence alone holds are filled in place
//     (evict_pack_kernel).  The j-th kept token sits at a slot >= j, so one
//     CTA that takes its rows in ascending runs, reading a run before any of
//     it is written, never overwrites a row still to be read.  Columns are
//     independent, so a 64-byte column slice per CTA keeps the GPU full.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kvp_internal.h"

namespace kvp {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kRowTile = 64;      // rows of K and of V per copy CTA
constexpr int kMoveThreads = 256;
constexpr int kInFlight = 8;      // 16-byte loads in flight per thread

// Order of weights as unsigned keys: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);   // -0 + 0 = +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int scan_warp(int x, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictLaunch a) {
    __shared__ int s_bin[kBins];
    __shared__ int s_sum[kSelWarps], s_eq[kSelWarps];
    __shared__ int s_digit, s_left;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % a.Hkv, ls = blockIdx.x / a.Hkv;
    const int s = ls % a.S;
    const EvictSeq sq = a.seqs[s];
    const float *m = a.mass + (size_t)blockIdx.x * a.stride;
    float *mo = a.mass_out ? a.mass_out + (size_t)blockIdx.x * a.stride : nullptr;
    int32_t *kept = a.kept + (size_t)blockIdx.x * a.budget;
    (void)h;
    if (sq.len <= a.budget) {   // everything stays where it is
        for (int j = tid; j < a.budget; j += kSelThreads) kept[j] = j < sq.len ? j : -1;
        if (mo && mo != m)
            for (int j = tid; j < sq.len; j += kSelThreads) mo[j] = m[j];
        return;
    }
    // positions [lo, hi) compete for k places
    const int lo = a.sink, hi = sq.len - a.recent;
    const int k = a.budget - a.sink - a.recent;
    uint32_t prefix = 0;   // the leading bits of the k-th largest key
    int left = k;          // places left among the keys that share them
    if (k > 0) {
#pragma unroll 1
        for (int p = 0; p < 3; ++p) {
            const int shift = p == 0 ? 21 : p == 1 ? 10 : 0, bits = p == 2 ? 10 : 11;
            for (int i = tid; i < kBins; i += kSelThreads) s_bin[i] = 0;
            __syncthreads();
#pragma unroll 8
            for (int i = lo + tid; i < hi; i += kSelThreads) {
                const uint32_t key = order_key(m[i]);
                // (the shift by 32 of the first pass is split in two)
                if ((key >> shift >> bits) == (p == 0 ? 0u : prefix >> shift >> bits))
                    atomicAdd(&s_bin[(key >> shift) & ((1 << bits) - 1)], 1);
            }
            __syncthreads();
            // from the largest digit down: thread i has digits 2047 - 4 i - {0..3}
            int n[4], sum = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += n[e] = s_bin[kBins - 1 - 4 * tid - e];
            const int inc = scan_warp(sum, lane);
            if (lane == 31) s_sum[warp] = inc;
            __syncthreads();
            int before = inc - sum;
            for (int w = 0; w < warp; ++w) before += s_sum[w];
            if (before < left && before + sum >= left) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (before < left && before + n[e] >= left) {
                        s_digit = kBins - 1 - 4 * tid - e;
                        s_left = left - before;
                        break;
                    }
                    before += n[e];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_digit << shift;
            left = s_left;
            __syncthreads();
        }
    }
    // stretch of this warp; its tokens above the k-th largest (and the sinks
    // and recent ones), and those equal to it
    const int per = ((sq.len + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int b0 = min(warp * per, sq.len), b1 = min(b0 + per, sq.len);
    auto kind = [&](int i) -> int {   // 2: stays, 1: equal, 0: goes
        if (i < lo || i >= hi) return 2;
        if (k == 0) return 0;
        const uint32_t key = order_key(m[i]);
        return key > prefix ? 2 : key == prefix ? 1 : 0;
    };
    int above = 0, equal = 0;
#pragma unroll 4
    for (int i = b0 + lane; i < b1; i += 32) {
        const int c = kind(i);
        above += c == 2;
        equal += c == 1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        above += __shfl_xor_sync(0xffffffffu, above, o);
        equal += __shfl_xor_sync(0xffffffffu, equal, o);
    }
    if (lane == 0) {
        s_sum[warp] = above;
        s_eq[warp] = equal;
    }
    __syncthreads();
    int n_above = 0, n_equal = 0;
    for (int w = 0; w < warp; ++w) {
        n_above += s_sum[w];
        n_equal += s_eq[w];
    }
    for (int i0 = b0; i0 < b1; i0 += 32) {
        const int i = i0 + lane;
        const int c = i < b1 ? kind(i) : 0;
        const uint32_t up = __ballot_sync(0xffffffffu, c == 2), eq = __ballot_sync(0xffffffffu, c == 1);
        const uint32_t mask = (1u << lane) - 1u;
        const int eq_before = n_equal + __popc(eq & mask);
        // (k == 0: nothing is equal)
        if (c == 2 || (c == 1 && eq_before < left))
            kept[n_above + __popc(up & mask) + min(eq_before, left)] = i;
        n_above += __popc(up);
        n_equal += __popc(eq);
    }
    if (!mo) return;
    // the kept weights, in place if need be: a run is read before any of it
    // is written, and later runs lie at or behind their places
    __syncthreads();
    constexpr int U = 4;
    for (int j0 = 0; j0 < a.budget; j0 += kSelThreads * U) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kSelThreads + tid;
            v[u] = j < a.budget ? m[kept[j]] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kSelThreads + tid;
            if (j < a.budget) mo[j] = v[u];
        }
    }
}

// 16-byte chunk c of the row of token `pos` in a table's pages
__device__ __forceinline__ int64_t chunk_at(const EvictLaunch &a, const int32_t *table, int pos, int l, int h, int c) {
    const int blk = table[pos / a.bs];
    return ((((int64_t)l * a.NB + blk) * a.Hkv + h) * a.bs + pos % a.bs) * a.CH + c;
}

__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const EvictLaunch a, int row_tiles) {
    const int s = blockIdx.x / row_tiles, r0 = (blockIdx.x % row_tiles) * kRowTile;
    const EvictSeq sq = a.seqs[s];
    if (sq.how != kEvictCopy) return;
    const int h = blockIdx.y % a.Hkv, l = blockIdx.y / a.Hkv;
    const int32_t *src = a.tables + sq.src, *dst = a.tables + sq.dst;
    const int32_t *kept = a.kept + (((size_t)l * a.S + s) * a.Hkv + h) * a.budget;
    const uint4 *kp = static_cast<const uint4 *>(a.k_pool), *vp = static_cast<const uint4 *>(a.v_pool);
    uint4 *ko = static_cast<uint4 *>(a.k_pool), *vo = static_cast<uint4 *>(a.v_pool);
    const int total = min(kRowTile, a.budget - r0) * a.CH;
    for (int x0 = threadIdx.x; x0 < total; x0 += kMoveThreads * (kInFlight / 2)) {
        uint4 kv[kInFlight / 2], vv[kInFlight / 2];
        int64_t to[kInFlight / 2];
#pragma unroll
        for (int u = 0; u < kInFlight / 2; ++u) {
            const int x = x0 + u * kMoveThreads;
            to[u] = -1;
            if (x < total) {
                const int j = r0 + x / a.CH, c = x % a.CH;
                const int64_t from = chunk_at(a, src, kept[j], l, h, c), t = chunk_at(a, dst, j, l, h, c);
                if (from != t) {   // (a page of sink tokens stays as it is)
                    to[u] = t;
                    kv[u] = kp[from];
                    vv[u] = vp[from];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight / 2; ++u)
            if (to[u] >= 0) {
                ko[to[u]] = kv[u];
                vo[to[u]] = vv[u];
            }
    }
}

// One CTA per (in-place sequence, layer, kv head, K or V, column slice of
// `width` chunks).
__global__ void __launch_bounds__(kMoveThreads) evict_pack_kernel(const EvictLaunch a, int width) {
    const int slices = a.CH / width;
    int x = blockIdx.x;
    const int slice = x % slices;
    x /= slices;
    uint4 *pool = static_cast<uint4 *>(x % 2 ? a.v_pool : a.k_pool);
    const int s = x / 2;
    const EvictSeq sq = a.seqs[s];
    if (sq.how != kEvictPack) return;
    const int h = blockIdx.y % a.Hkv, l = blockIdx.y / a.Hkv;
    const int32_t *src = a.tables + sq.src, *dst = a.tables + sq.dst;
    const int32_t *kept = a.kept + (((size_t)l * a.S + s) * a.Hkv + h) * a.budget;
    const int per = kMoveThreads / width;   // rows per step of the CTA
    const int row = threadIdx.x / width, c = slice * width + threadIdx.x % width;
    for (int j0 = 0; j0 < a.budget; j0 += per * kInFlight) {
        uint4 v[kInFlight];
        int64_t to[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int j = j0 + u * per + row;
            to[u] = -1;
            if (row < per && j < a.budget) {
                const int64_t from = chunk_at(a, src, kept[j], l, h, c), t = chunk_at(a, dst, j, l, h, c);
                if (from != t) {
                    to[u] = t;
                    v[u] = pool[from];
                }
            }
        }
        __syncthreads();   // the whole run is read; the runs behind it lie at or behind their places
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (to[u] >= 0) pool[to[u]] = v[u];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch &a, bool copies, bool packs, cudaStream_t stream) {
    evict_select_kernel<<<(unsigned)(a.L * a.S * a.Hkv), kSelThreads, 0, stream>>>(a);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const unsigned lh = (unsigned)(a.L * a.Hkv);
    if (copies) {
        const int tiles = (a.budget + kRowTile - 1) / kRowTile;
        evict_copy_kernel<<<dim3((unsigned)(tiles * a.S), lh), kMoveThreads, 0, stream>>>(a, tiles);
        count_launch();
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (packs) {
        const int width = a.CH % 4 == 0 ? 4 : 1;
        evict_pack_kernel<<<dim3((unsigned)(2 * a.S * (a.CH / width)), lh), kMoveThreads, 0, stream>>>(a, width);
        count_launch();
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace kvp
