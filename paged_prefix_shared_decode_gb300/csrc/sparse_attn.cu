// Attention over selected pages of a paged sequence (sm_103a): each query row
// and kv head with its own list of pages, decode steps and short chunks.
//
// Two products per 16 tokens of a page and the group's query heads, both with
// the tokens or dims on mma.sync's 16 rows and up to 8 heads on its columns
// (S^T = K Q^T, O^T += V^T P^T), so that nothing is padded to 16 heads.  K and
// V go from global memory straight into the operands' registers: Q K^T may
// run over the dims in any order, so a lane's part of K is 16 contiguous
// bytes; of V a lane reads 16 bytes of each of its four tokens and pairs the
// tokens up with byte permutes.  P^T turns from accumulator to operand by
// movmatrix.  Softmax in one pass: a reference maximum per head that is
// raised only when a score passes it by more than 8 (in powers of two).
//
// A weight P enters P V as two bf16 numbers (its rounding and the rest), which
// keeps 16 bits of it; V is bf16 as cached.
//
// The tiles of a row are dealt out to the warps of one or several CTAs of a
// cluster (several when there are few rows), whose partial sums are joined
// through distributed shared memory: one launch, no workspace.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/kvp.h"
#include "kvp_internal.h"
#include "launch.cuh"
#include "query_rows.cuh"

namespace kvp {
namespace {

constexpr int kWarps = 4;
constexpr int kList = 512;       // selected pages looked up at a time
constexpr int kMaxCtas = 8;      // CTAs of a cluster

struct SparseArgs {
    QueryRows rows;
    const __nv_bfloat16 *q, *k, *v;
    const int32_t *selected;
    __nv_bfloat16 *out;
    float *lse;
    int32_t L, Hq, Hkv, G, NB, bs_log2, budget, parts, ctas;   // parts: slices of 8 * NT heads of a group
    int32_t qt;                // rows of a tile
    float scale_log2;
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float exp2_sfu(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p) {
    return __ldg(reinterpret_cast<const uint4 *>(p));
}
__device__ __forceinline__ uint32_t word(const uint4 &x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }
__device__ __forceinline__ uint32_t mapa(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// What a part with reference m and sum l counts for beside the largest
// reference `top`: nothing if it saw no key (a NaN among its keys goes on).
__device__ __forceinline__ float share(float m, float l, float top) { return l == 0.f ? 0.f : exp2_sfu(m - top); }

// One value of out, and the row's lse (at >= 0) with its first.
__device__ __forceinline__ void put(const SparseArgs &a, int64_t o, int64_t at, float sum, float z, float top) {
    a.out[o] = __float2bfloat16_rn(z == 0.f ? 0.f : sum / z);
    if (at >= 0 && a.lse) a.lse[at] = z == 0.f ? -INFINITY : (top + log2f(z)) * 0.69314718055994531f;
}

// Partial results of a warp, then (in warp 0's place) of the CTA.
template <int D, int NT>
struct Partial {
    float o[8 * NT][D + 4];
    float m[8 * NT], l[8 * NT];
};

// A warp's state: columns 8 n + 2 t + e of a lane are (query, head) pairs.
template <int D, int NT>
struct Warp {
    uint4 q[NT][D / 32];            // B operand: column 8 n + g, 8 dims in a row
    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];       // reference, and the sum over this lane's tokens

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
        }
    }

    // 16 tokens at k and v (rows of D), of which the first `valid` are read;
    // column (n, e) sees those up to last(n, e).
    template <class Last>
    __device__ __forceinline__ void step(const __nv_bfloat16 *k, const __nv_bfloat16 *v, int valid, int lane, Last last) {
        constexpr int KC = D / 32, VC = D / 64;
        const int g = lane >> 2, t = lane & 3;
        uint4 kv[2][KC], vv[4][VC];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c = 0; c < KC; ++c)
                kv[e][c] = g + 8 * e < valid ? load16(k + (g + 8 * e) * D + 32 * c + 8 * t) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                const int tok = 2 * t + (e & 1) + 8 * (e >> 1);
                vv[e][c] = tok < valid ? load16(v + tok * D + 64 * c + 8 * g) : make_uint4(0, 0, 0, 0);
            }
        float s[NT][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma(s[n], kv[0][c].x, kv[1][c].x, kv[0][c].y, kv[1][c].y, q[n][c].x, q[n][c].y);
                mma(s[n], kv[0][c].z, kv[1][c].z, kv[0][c].w, kv[1][c].w, q[n][c].z, q[n][c].w);
            }
        // s[n][0..1]: token g, columns 2 t, 2 t + 1; s[n][2..3]: token g + 8
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[n][e] = g + 8 * (e >> 1) <= last(n, e & 1) ? s[n][e] * scale_log2 : -INFINITY;
                raise |= !(s[n][e] <= m[n][e & 1] + 8.f);    // (a NaN too)
            }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
                    for (int i = 4; i < 32; i <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, i));
                    x = fmaxf(x, m[n][e]);
                    const float f = m[n][e] == -INFINITY ? 0.f : exp2_sfu(m[n][e] - x);
                    m[n][e] = x;
                    l[n][e] *= f;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        o[n][j][e] *= f;
                        o[n][j][2 + e] *= f;
                    }
                }
        }
        uint32_t p_hi[NT][2], p_lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x[2], y[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float z = s[n][2 * e + i];
                    x[i] = z == -INFINITY ? 0.f : exp2_sfu(z - m[n][i]);
                    l[n][i] += x[i];
                    y[i] = x[i] - __bfloat162float(__float2bfloat16_rn(x[i]));
                }
                const __nv_bfloat162 hi = __floats2bfloat162_rn(x[0], x[1]), lo = __floats2bfloat162_rn(y[0], y[1]);
                p_hi[n][e] = transpose8(*reinterpret_cast<const uint32_t *>(&hi));
                p_lo[n][e] = transpose8(*reinterpret_cast<const uint32_t *>(&lo));
            }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            // rows g and g + 8 of V^T tile j: dims 8 g + j and 64 + 8 g + j
            // (head dim 64: 8 g + j and 8 g + 4 + j)
            const int c1 = VC - 1, j1 = VC == 2 ? j : j + 4;
            const uint32_t sel0 = j & 1 ? 0x7632 : 0x5410, sel1 = j1 & 1 ? 0x7632 : 0x5410;
            const uint32_t a0 = __byte_perm(word(vv[0][0], j >> 1), word(vv[1][0], j >> 1), sel0);
            const uint32_t a1 = __byte_perm(word(vv[0][c1], j1 >> 1), word(vv[1][c1], j1 >> 1), sel1);
            const uint32_t a2 = __byte_perm(word(vv[2][0], j >> 1), word(vv[3][0], j >> 1), sel0);
            const uint32_t a3 = __byte_perm(word(vv[2][c1], j1 >> 1), word(vv[3][c1], j1 >> 1), sel1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma(o[n][j], a0, a1, a2, a3, p_hi[n][0], p_hi[n][1]);
                mma(o[n][j], a0, a1, a2, a3, p_lo[n][0], p_lo[n][1]);
            }
        }
    }

    // The sums into shared memory.
    __device__ __forceinline__ void leave(Partial<D, NT> &part, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = 8 * n + 2 * t + e;
                float x = l[n][e];
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
                if (g == 0) {
                    part.m[c] = m[n][e];
                    part.l[c] = x;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    part.o[c][8 * g + j] = o[n][j][e];
                    part.o[c][D == 128 ? 64 + 8 * g + j : 8 * g + 4 + j] = o[n][j][2 + e];
                }
            }
    }

    float scale_log2;
};

// Value e of column c joined over the CTA's warps.
template <int D, int NT>
__device__ __forceinline__ void join_warps(const Partial<D, NT> *part, int c, int e, float &sum, float &z, float &top) {
    top = part[0].m[c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, part[w].m[c]);
    sum = z = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = share(part[w].m[c], part[w].l[c], top);
        sum += f * part[w].o[c][e];
        z += f * part[w].l[c];
    }
}

// One query row (and up to 8 NT heads of a group) per cluster of CTAs.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 3 : 2) sparse_attn_kernel(const SparseArgs a) {
    constexpr int H = 8 * NT;
    extern __shared__ __align__(16) unsigned char smem[];
    Partial<D, NT> *part = reinterpret_cast<Partial<D, NT> *>(smem);
    __shared__ int32_t s_page[kList], s_blk[kList];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    griddep_wait();
    const int rank = blockIdx.x % a.ctas;
    int64_t unit = blockIdx.x / a.ctas;
    const int slice = (int)(unit % a.parts);
    unit /= a.parts;
    const int h = (int)(unit % a.Hkv);
    const int64_t lr = unit / a.Hkv;                     // layer * T + row
    const int r = (int)(lr % a.rows.T), l = (int)(lr / a.rows.T);
    const int seq = a.rows.sequence(r);
    if (seq < 0) return;                                 // (the whole cluster's row)
    const int pos = a.rows.position(seq, r);
    const int seen = a.rows.pages(seq, r);
    const int heads = min(H, a.G - slice * H);           // query heads of this slice
    const int hq0 = h * a.G + slice * H;

    Warp<D, NT> w;
    w.scale_log2 = a.scale_log2;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            w.q[n][c] = 8 * n + g < heads ? load16(a.q + (lr * a.Hq + hq0 + 8 * n + g) * D + 32 * c + 8 * t)
                                          : make_uint4(0, 0, 0, 0);
    w.clear();

    const int sub_log2 = a.bs_log2 - 4;                  // 16-token tiles per page
    const int64_t head = (int64_t)l * a.NB * a.Hkv + h;
    const int32_t *sel = a.selected + (lr * a.Hkv + h) * a.budget;
    const int32_t *table = a.rows.tables + (int64_t)seq * a.rows.MB;
    for (int s0 = 0; s0 < a.budget; s0 += kList) {
        const int ns = min(kList, a.budget - s0);
        __syncthreads();
        for (int i = tid; i < ns; i += 32 * kWarps) {
            const int page = sel[s0 + i];
            int blk = -1;
            if (page >= 0 && page < seen) blk = table[page];
            const bool ok = (unsigned)blk < (unsigned)a.NB;
            s_page[i] = ok ? page : 0;
            s_blk[i] = ok ? blk : -1;
        }
        __syncthreads();
        const int tiles = ns << sub_log2, step = kWarps * a.ctas;
        for (int x = rank * kWarps + warp; x < tiles; x += step) {
            const int i = x >> sub_log2, sub = x & ((1 << sub_log2) - 1);
            const int blk = s_blk[i];
            const int first = (s_page[i] << a.bs_log2) + 16 * sub;       // position of the tile's first token
            if (blk < 0 || first > pos) continue;
            const int valid = min(16, pos - first + 1);
            const int64_t at = (((head + (int64_t)blk * a.Hkv) << a.bs_log2) + 16 * sub) * D;
            w.step(a.k + at, a.v + at, valid, lane, [&](int, int) { return valid - 1; });
        }
    }
    w.leave(part[warp], lane);
    __syncthreads();
    // joined over the CTA's warps (into warp 0's place when there is a
    // cluster), then over the cluster's CTAs
    const bool alone = a.ctas == 1;
    constexpr int PER = H * D / (32 * kWarps);          // values per thread
    float val[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = tid + i * 32 * kWarps, hd = x / D, e = x % D;
        float z, top;
        join_warps(part, hd, e, val[i], z, top);
        if (alone && hd < heads)
            put(a, (lr * a.Hq + hq0 + hd) * D + e, e == 0 ? lr * a.Hq + hq0 + hd : -1, val[i], z, top);
    }
    if (alone) return;
    float my_m = 0.f, my_l = 0.f;
    if (tid < H) {
        my_m = part[0].m[tid];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) my_m = fmaxf(my_m, part[w].m[tid]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            my_l += share(part[w].m[tid], part[w].l[tid], my_m) * part[w].l[tid];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = tid + i * 32 * kWarps;
        part[0].o[x / D][x % D] = val[i];
    }
    if (tid < H) {
        part[0].m[tid] = my_m;
        part[0].l[tid] = my_l;
    }
    cluster_sync();
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(part);
    constexpr uint32_t m_at = H * (D + 4) * 4, l_at = m_at + H * 4;     // as Partial lays them out
    // each CTA takes every ctas-th run of values
    for (int x = rank * 32 * kWarps + tid; x < heads * D; x += a.ctas * 32 * kWarps) {
        const int hd = x / D, e = x % D;
        float top = -INFINITY, mm[kMaxCtas];
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c) {
            mm[c] = c < a.ctas ? load_cluster(mapa(base + m_at + 4 * hd, c)) : -INFINITY;
            top = fmaxf(top, mm[c]);
        }
        float sum = 0.f, z = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c)
            if (c < a.ctas) {
                const float lc = load_cluster(mapa(base + l_at + 4 * hd, c)), f = share(mm[c], lc, top);
                sum += f * load_cluster(mapa(base + 4 * (hd * (D + 4) + e), c));
                z += f * lc;
            }
        put(a, (lr * a.Hq + hq0 + hd) * D + e, e == 0 ? lr * a.Hq + hq0 + hd : -1, sum, z, top);
    }
    cluster_sync();      // no CTA ends while another reads its sums
}


constexpr int kTilePages = 16384;    // pages of a sequence that a tile's map covers
constexpr int kTileList = 1024;      // pages listed at a time
constexpr int kTileBytes = kTilePages + kTileList * 8;

// Several consecutive query rows of a sequence (as many as fill 16 columns with
// their groups' heads): neighbours choose much the same pages, so a page is
// read once for all the rows that named it.  Which rows name a page is a byte
// per page in shared memory, and the pages are taken in ascending order.
//
// A value that is not finite in a page that only some of the rows see would
// reach the others as 0 * inf; then (and when a row names a page twice) the
// rows are done one after the other instead, each by its own list.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, 2) sparse_tile_kernel(const SparseArgs a) {
    constexpr int THREADS = 32 * kWarps;
    extern __shared__ __align__(16) unsigned char smem[];
    Partial<D, NT> *part = reinterpret_cast<Partial<D, NT> *>(smem);     // after the pages are done
    uint32_t *s_rows = reinterpret_cast<uint32_t *>(smem);               // a byte per page
    int32_t *s_blk = reinterpret_cast<int32_t *>(smem + kTilePages);
    int32_t *s_page = s_blk + kTileList;                                 // page << 8 | rows
    __shared__ int s_scan[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    griddep_wait();
    const int h = blockIdx.y % a.Hkv, l = blockIdx.y / a.Hkv;
    int r0, nr, seq;
    if (!a.rows.tile(a.qt, blockIdx.x, r0, nr, seq)) return;
    const int pos0 = a.rows.position(seq, r0);
    const int seen = a.rows.pages(seq, r0 + nr - 1);
    const int cols = nr * a.G;
    const int64_t lr0 = (int64_t)l * a.rows.T + r0;
    auto q_row = [&](int c) { return (lr0 + c / a.G) * a.Hq + h * a.G + c % a.G; };   // row of q, out, lse

    Warp<D, NT> w;
    w.scale_log2 = a.scale_log2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = 8 * n + g;
        const __nv_bfloat16 *q = a.q + (c < cols ? q_row(c) : 0) * D + 8 * t;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w.q[n][i] = c < cols ? load16(q + 32 * i) : make_uint4(0, 0, 0, 0);
    }
    w.clear();
    int row[NT][2];                                      // row of each of the lane's columns; 31: none
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) row[n][e] = 8 * n + 2 * t + e < cols ? (8 * n + 2 * t + e) / a.G : 31;

    const int sub_log2 = a.bs_log2 - 4;
    const int64_t head = (int64_t)l * a.NB * a.Hkv + h;
    const int32_t *table = a.rows.tables + (int64_t)seq * a.rows.MB;
    const int32_t *sel = a.selected + (lr0 * a.Hkv + h) * a.budget;
    const int64_t sel_row = (int64_t)a.Hkv * a.budget;
    auto page_of = [&](int q, int i) {                   // entry i of row q; -1: none that it sees
        const int page = sel[q * sel_row + i];
        return page >= 0 && pos0 + q >= 0 && page <= (pos0 + q) >> a.bs_log2 ? page : -1;
    };
    auto attend = [&](int n_list) {
        const int tiles = n_list << sub_log2;
        for (int x = warp; x < tiles; x += kWarps) {
            const int i = x >> sub_log2, sub = x & ((1 << sub_log2) - 1);
            const int blk = s_blk[i], page = s_page[i] >> 8, rows = s_page[i] & 255;
            const int first = (page << a.bs_log2) + 16 * sub;
            // the tokens that the last of the rows naming the page sees
            const int valid = min(16, pos0 + (31 - __clz(rows | 1)) - first + 1);
            if (blk < 0 || valid <= 0) continue;
            const int64_t at = (((head + (int64_t)blk * a.Hkv) << a.bs_log2) + 16 * sub) * D;
            w.step(a.k + at, a.v + at, valid, lane,
                   [&](int n, int e) { return rows >> row[n][e] & 1 ? pos0 + row[n][e] - first : -1; });
        }
    };
    auto block_of = [&](int page) {
        const int blk = table[page];
        return (unsigned)blk < (unsigned)a.NB ? blk : -1;
    };

    for (int i = tid; i < (seen + 15) / 16; i += THREADS) reinterpret_cast<uint4 *>(s_rows)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    bool twice = false;
    for (int64_t x = tid; x < (int64_t)nr * a.budget; x += THREADS) {
        const int q = (int)(x / a.budget), page = page_of(q, (int)(x % a.budget));
        if (page < 0) continue;
        const uint32_t bit = 1u << ((page & 3) * 8 + q);
        twice |= (atomicOr(&s_rows[page >> 2], bit) & bit) != 0;
    }
    bool single = __syncthreads_or(twice);
    if (!single) {
        const uint8_t *rows_of = reinterpret_cast<const uint8_t *>(s_rows);
        for (int p0 = 0; p0 < seen; p0 += kTileList) {
            // pages that some row names, in order: eight in a row per thread
            constexpr int PER = kTileList / THREADS;
            const int p = p0 + tid * PER;
            int mine = 0;
            uint32_t two[PER / 4];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) {
                two[i] = p + 4 * i < seen ? s_rows[(p >> 2) + i] : 0u;
                mine += __popc(__vcmpne4(two[i], 0u)) >> 3;
            }
            int before = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += y;
            }
            if (lane == 31) s_scan[warp] = before;
            __syncthreads();
            int all = 0;
            before -= mine;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                before += i < warp ? s_scan[i] : 0;
                all += s_scan[i];
            }
            if (mine)
                for (int i = 0; i < PER; ++i)
                    if (p + i < seen && rows_of[p + i]) {
                        s_page[before] = (p + i) << 8 | rows_of[p + i];
                        s_blk[before++] = block_of(p + i);
                    }
            __syncthreads();
            attend(all);
            __syncthreads();
        }
        bool bad = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bad |= !isfinite(w.l[n][e & 1]);
#pragma unroll
                for (int j = 0; j < D / 16; ++j) bad |= !isfinite(w.o[n][j][e]);
            }
        single = __syncthreads_or(bad);
    }
    // the sums of columns c0 .. c1 - 1 joined and written (part takes the
    // lists' place)
    auto finish = [&](int c0, int c1) {
        __syncthreads();
        w.leave(part[warp], lane);
        __syncthreads();
        for (int x = c0 * D + tid; x < c1 * D; x += THREADS) {
            const int c = x / D, e = x % D;
            float sum, z, top;
            join_warps(part, c, e, sum, z, top);
            put(a, q_row(c) * D + e, e == 0 ? q_row(c) : -1, sum, z, top);
        }
    };
    if (!single) {
        finish(0, cols);
        return;
    }
    for (int q = 0; q < nr; ++q) {
        w.clear();
        for (int i0 = 0; i0 < a.budget; i0 += kTileList) {
            const int n = min(kTileList, a.budget - i0);
            __syncthreads();
            for (int i = tid; i < n; i += THREADS) {
                const int page = page_of(q, i0 + i);
                s_page[i] = page < 0 ? 0 : page << 8 | 1 << q;
                s_blk[i] = page < 0 ? -1 : block_of(page);
            }
            __syncthreads();
            attend(n);
        }
        finish(q * a.G, (q + 1) * a.G);
    }
}

template <int D, int NT>
cudaError_t launch_sparse(SparseArgs a, cudaStream_t stream) {
    a.parts = (a.G + 8 * NT - 1) / (8 * NT);
    const int64_t units = (int64_t)a.L * a.rows.T * a.Hkv * a.parts;
    // few rows: several CTAs to each, as long as all of them run at once and
    // each warp has a tile or two
    a.ctas = 1;
    const int64_t tiles = (int64_t)a.budget << (a.bs_log2 - 4);
    while (a.ctas < kMaxCtas && units * a.ctas * 2 <= 2LL * device_sm_count() && tiles >= 2LL * kWarps * a.ctas * 2)
        a.ctas *= 2;
    if (units * a.ctas > INT32_MAX) return cudaErrorInvalidValue;
    return launch_behind(sparse_attn_kernel<D, NT>, dim3((unsigned)(units * a.ctas)), 32 * kWarps,
                         sizeof(Partial<D, NT>) * kWarps, a.ctas, stream, a);
}

template <int D, int NT>
cudaError_t launch_tile(const SparseArgs &a, int64_t tiles, cudaStream_t stream) {
    const size_t bytes = std::max<size_t>(sizeof(Partial<D, NT>) * kWarps, kTileBytes);
    return launch_behind(sparse_tile_kernel<D, NT>, dim3((unsigned)tiles, (unsigned)(a.L * a.Hkv)), 32 * kWarps, bytes, 1,
                         stream, a);
}

template <int D>
cudaError_t launch_for(SparseArgs a, cudaStream_t stream) {
    // rows of a chunk by tiles, where a tile holds two or more of them and
    // there is a CTA for every place on the GPU (two per SM); single rows
    // spread over clusters otherwise
    a.qt = std::min(8, 16 / a.G);
    if (a.rows.start && a.qt > 1 && a.rows.MB <= kTilePages && a.L * a.Hkv <= 65535 &&
        (int64_t)(a.rows.T / a.qt) * a.L * a.Hkv >= 2LL * device_sm_count())
        return a.qt * a.G <= 8 ? launch_tile<D, 1>(a, QueryRows::tiles(a.rows.T, a.rows.S, a.qt), stream)
                               : launch_tile<D, 2>(a, QueryRows::tiles(a.rows.T, a.rows.S, a.qt), stream);
    return a.G <= 8 ? launch_sparse<D, 1>(a, stream) : launch_sparse<D, 2>(a, stream);
}

bool bad(const void *p, uintptr_t align) { return !p || ((uintptr_t)p & (align - 1)); }

}  // namespace
}  // namespace kvp

extern "C" int paged_sparse_attention(const void *q, const int32_t *q_start, int32_t num_q, const void *k_pool,
                                      const void *v_pool, const int32_t *block_tables, const int32_t *seq_lens,
                                      int32_t num_seqs, int32_t max_blocks, const int32_t *selected, int32_t budget,
                                      const kvp_attn_desc *desc, void *out, float *lse, void *stream) {
    using namespace kvp;
    if (!attn_desc_ok(desc) || desc->kv_format != KVP_KV_BF16 || num_seqs <= 0 || max_blocks <= 0 ||
        (int64_t)max_blocks * desc->block_size > INT32_MAX / 2 || bad(block_tables, 4) || bad(seq_lens, 4) || num_q < 0 ||
        ((uintptr_t)q_start & 3) || (!q_start && num_q != num_seqs) || budget <= 0 || budget > (1 << 24) ||
        ((uintptr_t)lse & 3))
        return KVP_ERR_INVALID;
    if (num_q == 0) return KVP_OK;
    if (bad(q, 16) || bad(k_pool, 16) || bad(v_pool, 16) || bad(selected, 4) || bad(out, 16)) return KVP_ERR_INVALID;
    if (!stream && stream_capturing(nullptr)) return KVP_ERR_STATE;
    SparseArgs a{};
    a.rows = QueryRows{q_start, block_tables, seq_lens, num_seqs, num_q, max_blocks, desc->block_size};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k_pool);
    a.v = static_cast<const __nv_bfloat16 *>(v_pool);
    a.selected = selected;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.L = desc->num_layers; a.Hq = desc->num_q_heads; a.Hkv = desc->num_kv_heads; a.G = a.Hq / a.Hkv;
    a.NB = desc->num_blocks; a.budget = budget;
    while ((1 << a.bs_log2) < desc->block_size) ++a.bs_log2;
    const float scale = desc->scale > 0.f ? desc->scale : 1.f / sqrtf((float)desc->head_dim);
    a.scale_log2 = scale * 1.4426950408889634f;
    if ((int64_t)a.L * num_q * a.Hkv * ((a.G + 7) / 8) > INT32_MAX / kMaxCtas) return KVP_ERR_INVALID;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = desc->head_dim == 64 ? launch_for<64>(a, st) : launch_for<128>(a, st);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}
