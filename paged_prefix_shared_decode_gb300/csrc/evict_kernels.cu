// Eviction from the paged cache by accumulated attention weight (sm_103a):
// which tokens of a sequence stay, and the compaction of its pages.
//
// Selection, one CTA per (layer, sequence, kv head): the first `sink` and the
// last `recent` tokens stay, and of the rest the k = budget - sink - recent
// with the largest weight, equal weights by lowest position.  The k-th
// largest is found by a radix select over the weights as ordered 32-bit keys
// (11, 11 and 10 bits a pass, a histogram in shared memory).  Each warp holds
// a contiguous stretch of the row, so that one scan over the 16 warps' counts
// gives every kept token its place in position order.  Rows are read once and
// stay in shared memory as keys (which also makes the weights' compaction safe
// in place) as far as it reaches; longer ones are read again in every pass,
// from L2.  (Keys in registers, 32 to a lane, needed every loop unrolled:
// straight-line code that each CTA runs once waits for instruction fetches,
// 27 to 35 us where this takes 23 us for rows of up to 16000.)
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
#include <cstring>
#include <mutex>

#include "kvp_internal.h"

namespace kvp {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kHoldKeys = 48 * 1024;   // keys of a row that fit in shared memory
constexpr int kRowTile = 64;      // rows of K and of V per copy CTA
constexpr int kMoveThreads = 256;
constexpr int kInFlight = 8;      // 16-byte loads in flight per thread

// Weights as unsigned keys of the same order: NaN below everything, -0 as 0
// (a kept weight written from its key is 0 and one NaN for all of those).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x == x ? x + 0.f : __uint_as_float(0xffffffffu));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_weight(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kStays = 0xffffffffu;   // sinks and recent tokens: above every weight's key

__device__ __forceinline__ int scan_warp(int x, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The sequences and the tables: from the workspace, or from the image in the
// kernel's parameters.
template <class Image>
__device__ __forceinline__ const EvictSeq *seqs_of(const EvictLaunch &a, const Image &image) {
    return std::is_same<Image, InlineImage>::value ? reinterpret_cast<const EvictSeq *>(&image) : a.seqs;
}
template <class Image>
__device__ __forceinline__ const int32_t *tables_of(const EvictLaunch &a, const Image &image) {
    return std::is_same<Image, InlineImage>::value
               ? reinterpret_cast<const int32_t *>(reinterpret_cast<const unsigned char *>(&image) + a.tables_at)
               : a.tables;
}

// HOLD: the row's keys are kept in (dynamic) shared memory.
template <bool HOLD, class Image>
__global__ void __launch_bounds__(kSelThreads, 3)
    evict_select_kernel(const EvictLaunch a, const __grid_constant__ Image image) {
    __shared__ __align__(16) int s_bin[kBins];
    __shared__ int s_sum[kSelWarps], s_eq[kSelWarps];
    __shared__ int s_digit, s_left;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && tid == 0) *a.err = 0;
    const EvictSeq sq = seqs_of(a, image)[blockIdx.x / a.Hkv % a.S];
    const float *m = a.mass + (size_t)blockIdx.x * a.stride;
    float *mo = a.mass_out ? a.mass_out + (size_t)blockIdx.x * a.stride : nullptr;
    int32_t *kept = a.kept + (size_t)blockIdx.x * a.budget;
    if (sq.len <= a.budget) {   // everything stays where it is
        for (int j = tid; j < a.budget; j += kSelThreads) kept[j] = j < sq.len ? j : -1;
        if (mo && mo != m)
            for (int j = tid; j < sq.len; j += kSelThreads) mo[j] = m[j];
        return;
    }
    // this warp's stretch: tokens b0 + lane + 32 k below b1.  A token that
    // stays by its position has the highest key, and one past the end the
    // lowest (a NaN's, but behind it), so the `budget` first keys by (key,
    // position) are the kept tokens and nothing below looks at positions.
    const int per = ((sq.len + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int b0 = min(warp * per, sq.len), b1 = min(b0 + per, sq.len);
    const int lo = a.sink, hi = sq.len - a.recent;
    auto key_at = [&](int i, float x) -> uint32_t {
        return i >= b1 ? 0u : (unsigned)(i - lo) < (unsigned)(hi - lo) ? order_key(x) : kStays;
    };
    extern __shared__ uint32_t s_key[];
    if (HOLD) {   // (each lane reads back its own)
#pragma unroll 8
        for (int i = b0 + lane; i < b1; i += 32) s_key[i] = key_at(i, m[i]);
    }
    // f(i, key) for the lane's tokens in ascending order, the whole warp at
    // every step
    auto each = [&](auto f) {
#pragma unroll 4
        for (int i = b0 + lane; i - lane < b1; i += 32)
            f(i, i >= b1 ? 0u : HOLD ? s_key[i] : key_at(i, m[i]));
    };
    uint32_t prefix = 0;      // the leading bits of the last kept key
    int left = a.budget;      // places left among the keys that share them
#pragma unroll 1
    for (int p = 0; p < 3; ++p) {
        const int shift = p == 0 ? 21 : p == 1 ? 10 : 0, bits = p == 2 ? 10 : 11;
        for (int i = tid; i < kBins / 4; i += kSelThreads) reinterpret_cast<int4 *>(s_bin)[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
        if (p == 0) {
            each([&](int, uint32_t key) { atomicAdd(&s_bin[key >> 21], 1); });
        } else {
            const uint32_t mask = ~0u << (shift + bits);
            each([&](int, uint32_t key) {
                if (((key ^ prefix) & mask) == 0) atomicAdd(&s_bin[(key >> shift) & ((1 << bits) - 1)], 1);
            });
        }
        __syncthreads();
        // from the largest digit down: thread i has digits 2047 - 4 i - {0..3}
        int4 q = make_int4(0, 0, 0, 0);
        if (tid < kBins / 4) q = reinterpret_cast<const int4 *>(s_bin)[kBins / 4 - 1 - tid];
        const int n[4] = {q.w, q.z, q.y, q.x};
        const int sum = n[0] + n[1] + n[2] + n[3];
        const int inc = scan_warp(sum, lane);
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        int before = inc - sum + (int)__reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
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
    }
    // keys above the last kept one stay, of those equal to it the first
    // `left`: how many of each lie before this warp's stretch
    int above = 0, equal = 0;
    each([&](int i, uint32_t key) {
        above += key > prefix;
        equal += key == prefix;
    });
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        s_sum[warp] = above;
        s_eq[warp] = equal;
    }
    __syncthreads();
    int n_above = __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
    int n_equal = __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
    const uint32_t mask = (1u << lane) - 1u;
    // (with the keys held, no weight is read again but those of tokens that
    // stay by position: sinks keep their place, recent ones are moved below)
    const bool write = HOLD && mo;
    if (equal == 0 || n_equal >= left) {   // no key of the stretch is kept as an equal
        int j0 = n_above + min(n_equal, left);
        each([&](int i, uint32_t key) {
            const uint32_t up = __ballot_sync(0xffffffffu, key > prefix);
            const int j = j0 + __popc(up & mask);
            if (key > prefix) {
                kept[j] = i;
                if (write && key != kStays) mo[j] = key_weight(key);
            }
            j0 += __popc(up);
        });
    } else {
        each([&](int i, uint32_t key) {
            const uint32_t up = __ballot_sync(0xffffffffu, key > prefix), eq = __ballot_sync(0xffffffffu, key == prefix);
            const int eq_before = n_equal + __popc(eq & mask);
            if (key > prefix || (key == prefix && eq_before < left)) {
                const int j = n_above + __popc(up & mask) + min(eq_before, left);
                kept[j] = i;
                if (write && key != kStays) mo[j] = key_weight(key);
            }
            n_above += __popc(up);
            n_equal += __popc(eq);
        });
    }
    if (!mo) return;
    // the weights not yet in place: all of them, or the recent tokens' (whose
    // sources lie behind every place written so far).  In place if need be: a
    // run is read before any of it is written, and later runs lie at or
    // behind their places
    __syncthreads();
    if (HOLD && mo != m)
        for (int j = tid; j < lo; j += kSelThreads) mo[j] = m[j];
    constexpr int U = 4;
    for (int j0 = HOLD ? a.budget - a.recent : 0; j0 < a.budget; j0 += kSelThreads * U) {
        float w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kSelThreads + tid;
            w[u] = j < a.budget ? m[kept[j]] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kSelThreads + tid;
            if (j < a.budget) mo[j] = w[u];
        }
    }
}

// 16-byte chunk c of the row of token `pos` in a table's pages
__device__ __forceinline__ int64_t chunk_at(const EvictLaunch &a, const int32_t *table, int pos, int l, int h, int c) {
    const int blk = table[pos / a.bs];
    return ((((int64_t)l * a.NB + blk) * a.Hkv + h) * a.bs + pos % a.bs) * a.CH + c;
}

template <class Image>
__global__ void __launch_bounds__(kMoveThreads)
    evict_copy_kernel(const EvictLaunch a, int row_tiles, const __grid_constant__ Image image) {
    const int s = blockIdx.x / row_tiles, r0 = (blockIdx.x % row_tiles) * kRowTile;
    const EvictSeq sq = seqs_of(a, image)[s];
    if (sq.how != kEvictCopy) return;
    const int h = blockIdx.y % a.Hkv, l = blockIdx.y / a.Hkv;
    const int32_t *src = tables_of(a, image) + sq.src, *dst = tables_of(a, image) + sq.dst;
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
template <class Image>
__global__ void __launch_bounds__(kMoveThreads)
    evict_pack_kernel(const EvictLaunch a, int width, const __grid_constant__ Image image) {
    const int slices = a.CH / width;
    int x = blockIdx.x;
    const int slice = x % slices;
    x /= slices;
    uint4 *pool = static_cast<uint4 *>(x % 2 ? a.v_pool : a.k_pool);
    const int s = x / 2;
    const EvictSeq sq = seqs_of(a, image)[s];
    if (sq.how != kEvictPack) return;
    const int h = blockIdx.y % a.Hkv, l = blockIdx.y / a.Hkv;
    const int32_t *src = tables_of(a, image) + sq.src, *dst = tables_of(a, image) + sq.dst;
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

// Per device: the selection kernels' shared-memory limit is raised once.
bool select_ready() {
    static bool ok[kMaxDevices];
    static std::once_flag once[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return false;
    std::call_once(once[dev], [dev] {
        const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
        ok[dev] = cudaFuncSetAttribute(evict_select_kernel<true, NoImage>, attr, kHoldKeys * 4) == cudaSuccess &&
                  cudaFuncSetAttribute(evict_select_kernel<true, InlineImage>, attr, kHoldKeys * 4) == cudaSuccess;
    });
    return ok[dev];
}

template <class Image>
cudaError_t launch_evict_with(const EvictLaunch &a, int max_len, bool copies, bool packs, const Image &image,
                              cudaStream_t stream) {
    const unsigned rows = (unsigned)(a.L * a.S * a.Hkv);
    if (max_len <= kHoldKeys) {
        if (!select_ready()) return cudaErrorInvalidDevice;
        evict_select_kernel<true><<<rows, kSelThreads, (size_t)max_len * 4, stream>>>(a, image);
    } else {
        evict_select_kernel<false><<<rows, kSelThreads, 0, stream>>>(a, image);
    }
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const unsigned lh = (unsigned)(a.L * a.Hkv);
    if (copies) {
        const int tiles = (a.budget + kRowTile - 1) / kRowTile;
        evict_copy_kernel<<<dim3((unsigned)(tiles * a.S), lh), kMoveThreads, 0, stream>>>(a, tiles, image);
        count_launch();
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (packs) {
        const int width = a.CH % 4 == 0 ? 4 : 1;
        evict_pack_kernel<<<dim3((unsigned)(2 * a.S * (a.CH / width)), lh), kMoveThreads, 0, stream>>>(a, width, image);
        count_launch();
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch &a0, int max_len, bool copies, bool packs, const unsigned char *image,
                         size_t bytes, size_t tables_at, cudaStream_t stream) {
    EvictLaunch a = a0;
    if (!image) return launch_evict_with(a, max_len, copies, packs, NoImage{}, stream);
    if (bytes > kInlineMax) return cudaErrorInvalidValue;
    a.tables_at = (int32_t)tables_at;
    InlineImage in;
    std::memcpy(in.b, image, bytes);
    return launch_evict_with(a, max_len, copies, packs, in, stream);
}

}  // namespace kvp
