// Attention over selected pages of a paged sequence (sm_103a): each query row
// and kv head with its own list of pages: decode steps, a few rows each of many
// sequences, and the calls.  (Chunks of prompts: sparse_tc.cuh.)
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
//
// Bound by HBM: 64 sequences of 128 pages, 2 layers, 8 kv heads at d 128 173 us,
// 6.2 TB/s of 1.08 GB, 92% of the copy peak.  One sequence of 64 pages 6.2 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/kvp.h"
#include "kvp_internal.h"
#include "launch.cuh"
#include "query_rows.cuh"
#include "tc_ops.cuh"

namespace kvp {
namespace {

constexpr int kWarps = 4;
constexpr int kList = 512;       // selected pages looked up at a time
constexpr int kMaxCtas = 8;      // CTAs of a cluster
// Largest reference m, in powers of two, for 2^(s scale - m) in one fused
// instruction: m = s scale rounded is off by 2^-24 m, a factor that every weight
// of the row carries; it stays far from fp32's ends.
constexpr float kLargestScore = 0x1p28f;

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

// Where a row's 16-byte chunk lies in shared memory: the four lanes of two
// neighbouring rows (K), and of four even or odd ones (V), meet in no bank.
__device__ __forceinline__ int swizzle(int row, int chunk) { return chunk ^ (row & 6) ^ (row & 1) << 2; }

// 16 bytes into shared memory, or zeros.
__device__ __forceinline__ void copy16(const uint4 *to, const void *from, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(real ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

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

    // 16 tokens at k and v (rows of D), of which the first `valid` are read and
    // seen by every column.
    __device__ __forceinline__ void step(const __nv_bfloat16 *k, const __nv_bfloat16 *v, int valid, int lane) {
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
        float s[NT][4] = {}, s2[NT][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) scores(s, s2, kv[0][c], kv[1][c], c);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
        uint32_t p_hi[NT][2], p_lo[NT][2];
        weigh(s, lane, valid, p_hi, p_lo);
        values(vv, p_hi, p_lo);
    }

    // S^T += K Q^T over chunk c of the dims, in two sums (one chain of products
    // waits for every result): rows g and g + 8 are tokens.
    __device__ __forceinline__ void scores(float (&s)[NT][4], float (&s2)[NT][4], const uint4 &ka, const uint4 &kb, int c) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma(s[n], ka.x, kb.x, ka.y, kb.y, q[n][c].x, q[n][c].y);
            mma(s2[n], ka.z, kb.z, ka.w, kb.w, q[n][c].z, q[n][c].w);
        }
    }

    // Scores (s[n][0..1]: token g, columns 2 t, 2 t + 1; s[n][2..3]: token g + 8)
    // to weights as B operands.
    __device__ __forceinline__ void weigh(float (&s)[NT][4], int lane, int valid, uint32_t (&p_hi)[NT][2],
                                          uint32_t (&p_lo)[NT][2]) {
        const int g = lane >> 2;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = g + 8 * (e >> 1) < valid ? s[n][e] * scale_log2 : -INFINITY;
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) raise |= !(s[n][e] <= m[n][e & 1] + 8.f);    // (a NaN too)
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
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // (2^(-inf - 0) = 0 for a column that has seen nothing yet)
            const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x0 = exp2_sfu(s[n][2 * e] - m0), x1 = exp2_sfu(s[n][2 * e + 1] - m1);
                l[n][0] += x0;
                l[n][1] += x1;
                const __nv_bfloat162 hi = __floats2bfloat162_rn(x0, x1);
                const uint32_t h = *reinterpret_cast<const uint32_t *>(&hi);
                const __nv_bfloat162 lo =
                    __floats2bfloat162_rn(x0 - __uint_as_float(h << 16), x1 - __uint_as_float(h & 0xffff0000u));
                p_hi[n][e] = transpose8(h);
                p_lo[n][e] = transpose8(*reinterpret_cast<const uint32_t *>(&lo));
            }
        }
    }

    // O^T += V^T P^T.  Rows g and g + 8 of V^T tile j are dims 8 g + j and 64 +
    // 8 g + j (head dim 64: 8 g + j and 8 g + 4 + j).
    __device__ __forceinline__ void values(const uint4 (&vv)[4][D / 64], const uint32_t (&p_hi)[NT][2],
                                           const uint32_t (&p_lo)[NT][2]) {
        constexpr int VC = D / 64, J = 4;
#pragma unroll
        for (int j0 = 0; j0 < D / 16; j0 += J) {
            uint32_t a[J][4];
#pragma unroll
            for (int i = 0; i < J; ++i) {
                const int j = j0 + i, c1 = VC - 1, j1 = VC == 2 ? j : j + 4;
                const uint32_t sel0 = j & 1 ? 0x7632 : 0x5410, sel1 = j1 & 1 ? 0x7632 : 0x5410;
                a[i][0] = __byte_perm(word(vv[0][0], j >> 1), word(vv[1][0], j >> 1), sel0);
                a[i][1] = __byte_perm(word(vv[0][c1], j1 >> 1), word(vv[1][c1], j1 >> 1), sel1);
                a[i][2] = __byte_perm(word(vv[2][0], j >> 1), word(vv[3][0], j >> 1), sel0);
                a[i][3] = __byte_perm(word(vv[2][c1], j1 >> 1), word(vv[3][c1], j1 >> 1), sel1);
            }
#pragma unroll
            for (int i = 0; i < J; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma(o[n][j0 + i], a[i][0], a[i][1], a[i][2], a[i][3], p_hi[n][0], p_hi[n][1]);
#pragma unroll
            for (int i = 0; i < J; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma(o[n][j0 + i], a[i][0], a[i][1], a[i][2], a[i][3], p_lo[n][0], p_lo[n][1]);
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
// OCC: CTAs per SM that the registers are cut for.
template <int D, int NT, int OCC>
__global__ void __launch_bounds__(32 * kWarps, OCC) sparse_attn_kernel(const SparseArgs a) {
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
            w.step(a.k + at, a.v + at, valid, lane);
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


// A warp's state for 16 (query, head) rows: rows g and g + 8 of a lane.  With
// that many the queries are the 16 rows and K the columns of S = Q K^T, whose
// fragments are those of P in O += P V, and K's operand is two registers of
// one load in a row (as rows, tokens g and g + 8 interleave: a quarter of the
// kernel's instructions were moves).
template <int D>
struct Rows16 {
    uint32_t q[D / 16][4];
    float o[D / 8][4];              // tile 8 c + j: dims 64 c + 8 (2 t) + j and 64 c + 8 (2 t + 1) + j
    float m[2], l[2];
    float scale_log2;

    __device__ __forceinline__ void clear() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    }
    // 8 dims of rows g and g + 8, from 32 c + 8 t on
    __device__ __forceinline__ void load_q(int c, uint4 a, uint4 b) {
        q[2 * c][0] = a.x; q[2 * c][1] = b.x; q[2 * c][2] = a.y; q[2 * c][3] = b.y;
        q[2 * c + 1][0] = a.z; q[2 * c + 1][1] = b.z; q[2 * c + 1][2] = a.w; q[2 * c + 1][3] = b.w;
    }

    // 16 tokens in shared memory: K, then V, rows of D with their 16-byte
    // chunks at swizzle(row, chunk).  Row g + 8 e sees those up to last[e].
    __device__ __forceinline__ void step(const uint4 *kv, int lane, bool full, const int (&last)[2]) {
        constexpr int CH = D / 8, VC = D / 64;
        const int g = lane >> 2, t = lane & 3;
        // (two chains of products for each tile of tokens: one after the other
        // they wait for one another's results)
        float s[2][4] = {}, s2[2][4] = {};
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const int at = g * CH + swizzle(g, 4 * c + t);           // (tokens g and g + 8 alike)
            const uint4 k0 = kv[at], k1 = kv[at + 8 * CH];
            mma(s[0], q[2 * c][0], q[2 * c][1], q[2 * c][2], q[2 * c][3], k0.x, k0.y);
            mma(s[1], q[2 * c][0], q[2 * c][1], q[2 * c][2], q[2 * c][3], k1.x, k1.y);
            mma(s2[0], q[2 * c + 1][0], q[2 * c + 1][1], q[2 * c + 1][2], q[2 * c + 1][3], k0.z, k0.w);
            mma(s2[1], q[2 * c + 1][0], q[2 * c + 1][1], q[2 * c + 1][2], q[2 * c + 1][3], k1.z, k1.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[0][i] += s2[0][i];
            s[1][i] += s2[1][i];
        }
        // s[n][0..1]: row g, tokens 8 n + 2 t, + 1; s[n][2..3]: row g + 8
        if (!full) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (8 * n + 2 * t + (i & 1) > last[i >> 1]) s[n][i] = -INFINITY;
        }
        // the reference is in units of unscaled scores: 2^((s - m) scale).  (slack is
        // finite: the first reference is -inf)
        bool raise = false;
        const float slack = fminf(8.f / scale_log2, 1e30f);
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
            raise |= top[e] > m[e] + slack;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = top[e];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                x = fmaxf(x, m[e]);
                const float f = m[e] == -INFINITY ? 0.f : exp2_sfu((m[e] - x) * scale_log2);
                m[e] = x;
                l[e] *= f;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][2 * e] *= f;
                    o[j][2 * e + 1] *= f;
                }
            }
        }
        uint32_t p_hi[4], p_lo[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // (2^-inf = 0 for a row that has seen nothing yet)
            float shift = m[e] == -INFINITY ? 0.f : -m[e] * scale_log2;
            if (fabsf(shift) > kLargestScore) {      // the difference first
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    s[n][2 * e] -= m[e];
                    s[n][2 * e + 1] -= m[e];
                }
                shift = 0.f;
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float x0 = exp2_sfu(fmaf(s[n][2 * e], scale_log2, shift));
                const float x1 = exp2_sfu(fmaf(s[n][2 * e + 1], scale_log2, shift));
                l[e] += x0 + x1;
                const __nv_bfloat162 hi = __floats2bfloat162_rn(x0, x1);
                const uint32_t h = *reinterpret_cast<const uint32_t *>(&hi);
                const __nv_bfloat162 lo =
                    __floats2bfloat162_rn(x0 - __uint_as_float(h << 16), x1 - __uint_as_float(h & 0xffff0000u));
                p_hi[2 * n + e] = h;
                p_lo[2 * n + e] = *reinterpret_cast<const uint32_t *>(&lo);
            }
        }
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
                v[i] = kv[(16 + tok) * CH + swizzle(tok, 8 * c + g)];
            }
            uint32_t b[8][2];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t pick = j & 1 ? 0x7632 : 0x5410;
                b[j][0] = __byte_perm(word(v[0], j >> 1), word(v[1], j >> 1), pick);
                b[j][1] = __byte_perm(word(v[2], j >> 1), word(v[3], j >> 1), pick);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) mma(o[8 * c + j], p_hi[0], p_hi[1], p_hi[2], p_hi[3], b[j][0], b[j][1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) mma(o[8 * c + j], p_lo[0], p_lo[1], p_lo[2], p_lo[3], b[j][0], b[j][1]);
        }
    }

    __device__ __forceinline__ void leave(Partial<D, 2> &part, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = g + 8 * e;
            float x = l[e];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (t == 0) {
                part.m[r] = m[e] * scale_log2;
                part.l[r] = x;
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                part.o[r][64 * (j / 8) + 16 * t + j % 8] = o[j][2 * e];
                part.o[r][64 * (j / 8) + 16 * t + 8 + j % 8] = o[j][2 * e + 1];
            }
        }
    }
};

constexpr int kTilePages = 4096;     // pages of a sequence that a tile's map covers
constexpr int kTileList = 256;       // pages listed at a time
constexpr int kTileSteps = 8;        // 16-token steps in a CTA's rings
constexpr int kTileMap = kTilePages + kTileList * 16;

// Several consecutive query rows of a sequence (as many as fill 16 MT rows with
// their groups' heads, at most 8): neighbours choose much the same pages, so a
// page is read once for all the rows that named it.  Which rows name a page is
// a byte per page in shared memory, and the pages are taken in ascending order.
// For batches of a few rows each (64 sequences of 2.4 rows on average, 32 pages of
// 32 tokens, d 128: 86 us; tiles of 128 rows, which suit chunks, 100).  Bound by
// what L2 delivers, 10 to 11 TB/s.
//
// A value that is not finite in a page that only some of the rows see would
// reach the others as 0 * inf; then (and when a row names a page twice) the
// rows are done one after the other instead, each by its own list.
//
// MT warps, with 16 rows each, go through the same 16-token steps, which they
// copy (cp.async) into a ring in shared memory some steps ahead; 4 / MT rings
// of a CTA share the list.  (Straight from global memory, as single rows do it,
// the 8 warps of two CTAs that 230 registers leave waited for every load.)
struct alignas(16) Page {
    int64_t at;          // where its rows of K and V start
    int32_t first;       // position of its first token
    int32_t count_rows;  // tokens that the last of the rows naming it sees << 8 | those rows
};
template <int D, int MT>
__global__ void __launch_bounds__(32 * kWarps, D == 64 ? 4 : 3) sparse_tile_kernel(const SparseArgs a) {
    constexpr int THREADS = 32 * kWarps, SPLITS = kWarps / MT, STAGES = kTileSteps / SPLITS;
    extern __shared__ __align__(16) unsigned char smem[];
    uint32_t *s_rows = reinterpret_cast<uint32_t *>(smem);               // a byte per page
    Page *s_list = reinterpret_cast<Page *>(smem + kTilePages);
    constexpr int CH = D / 8, STEP = 32 * CH;                            // 16-byte chunks of a row, of a step
    uint4 *s_ring = reinterpret_cast<uint4 *>(smem + kTileMap);
    Partial<D, 2> *part = reinterpret_cast<Partial<D, 2> *>(s_ring);   // after the pages are done
    __shared__ int s_scan[kWarps];
    __shared__ float s_share[SPLITS][16 * MT];
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

    const int mt = warp % MT, split = warp / MT, col0 = 16 * mt;         // this warp's rows and steps
    Rows16<D> w;
    w.scale_log2 = a.scale_log2;
    int row[2];                                          // query row of rows g and g + 8; 31: none
#pragma unroll
    for (int e = 0; e < 2; ++e) row[e] = col0 + g + 8 * e < cols ? (col0 + g + 8 * e) / a.G : 31;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        uint4 x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            x[e] = row[e] < 31 ? load16(a.q + q_row(col0 + g + 8 * e) * D + 32 * c + 8 * t) : make_uint4(0, 0, 0, 0);
        w.load_q(c, x[0], x[1]);
    }
    w.clear();
    // its query rows, as bits (none: a tile with fewer rows than it has room for)
    const int q_lo = col0 / a.G, q_hi = min(col0 + 15, cols - 1) / a.G;
    const int own = col0 < cols ? (2 << q_hi) - (1 << q_lo) : 0;

    const int sub_log2 = a.bs_log2 - 4;
    const int64_t head = (int64_t)l * a.NB * a.Hkv + h;
    const int32_t *table = a.rows.tables + (int64_t)seq * a.rows.MB;
    const int32_t *sel = a.selected + (lr0 * a.Hkv + h) * a.budget;
    const int64_t sel_row = (int64_t)a.Hkv * a.budget;
    auto page_of = [&](int q, int i) {                   // entry i of row q; -1: none that it sees
        const int page = sel[q * sel_row + i];
        return page >= 0 && pos0 + q >= 0 && page <= (pos0 + q) >> a.bs_log2 ? page : -1;
    };
    uint4 *ring = s_ring + split * STAGES * STEP;
    // the warps of a ring, of which each has waited for its own copies
    auto meet = [&] {
        if constexpr (MT == 1)
            __syncwarp();
        else if (split == 0)
            asm volatile("bar.sync 1, %0;\n" ::"n"(32 * MT) : "memory");
        else
            asm volatile("bar.sync 2, %0;\n" ::"n"(32 * MT) : "memory");
    };
    auto attend = [&](int n_list) {
        const int tiles = n_list << sub_log2;
        const int sub_mask = (1 << sub_log2) - 1;
        auto fetch = [&](int x, int stage) {
            if (x >= tiles) {
                copies_commit();
                return;
            }
            const Page p = s_list[x >> sub_log2];
            const int sub = 16 * (x & sub_mask), valid = min(16, (p.count_rows >> 8) - sub);
            if (valid > 0) {
                const uint4 *k = reinterpret_cast<const uint4 *>(a.k + p.at + sub * D);
                const uint4 *v = reinterpret_cast<const uint4 *>(a.v + p.at + sub * D);
                // token RPI i + lane / CH, chunk lane % CH, i = 0, 1, ...: of the
                // swizzle's terms one is the lane's and one the step's
                constexpr int RPI = 32 / CH;
                const int tok = lane / CH, c = lane % CH ^ (tok & 6) ^ (tok & 1) << 2;
                uint4 *to = ring + stage * STEP + tok * CH;
                auto rows16 = [&](const uint4 *from, uint4 *to) {
                    if (valid == 16) {
#pragma unroll
                        for (int i = 0; i < 16 / RPI; ++i)
                            copy16(to + RPI * i * CH + (c ^ (RPI * i & 6)), from + lane + 32 * i, true);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16 / RPI; ++i) {
                            const bool real = tok + RPI * i < valid;
                            copy16(to + RPI * i * CH + (c ^ (RPI * i & 6)), from + (real ? lane + 32 * i : 0), real);
                        }
                    }
                };
                if (MT == 1 || mt == 0) rows16(k, to);
                if (MT == 1 || mt == 1) rows16(v, to + 16 * CH);
            }
            copies_commit();
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) fetch(split + i * SPLITS, i);
        int stage = 0;
        for (int x = split; x < tiles; x += SPLITS) {
            copies_wait<STAGES - 2>();
            meet();                // the step is there, and the one before it done with
            fetch(x + (STAGES - 1) * SPLITS, stage == 0 ? STAGES - 1 : stage - 1);
            const Page p = s_list[x >> sub_log2];
            const int sub = 16 * (x & sub_mask), rows = p.count_rows & 255, mine = rows & own;
            if (mine && (p.count_rows >> 8) > sub) {
                // how far behind the step's first token row 0 is
                const int ahead = pos0 - p.first - sub;
                const int last[2] = {mine >> row[0] & 1 ? ahead + row[0] : -1, mine >> row[1] & 1 ? ahead + row[1] : -1};
                w.step(ring + stage * STEP, lane, mine == own && ahead + q_lo >= 15, last);
            }
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }
        copies_wait<0>();
        meet();
    };
    auto entry = [&](int page, int rows) {
        const int blk = table[page], first = page << a.bs_log2;
        // (an entry without a block is passed over)
        const int count = (unsigned)blk < (unsigned)a.NB ? min(1 << a.bs_log2, pos0 + 31 - __clz(rows) - first + 1) : 0;
        return Page{((head + (int64_t)max(blk, 0) * a.Hkv) << a.bs_log2) * D, first, max(count, 0) << 8 | rows};
    };

    for (int i = tid; i < (seen + 15) / 16; i += THREADS) reinterpret_cast<uint4 *>(s_rows)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    bool twice = false;
    // (a row's entries by a quarter of the threads or more, so that no thread
    // divides by the budget)
    for (int q = warp; q < nr; q += kWarps)
        for (int i = lane; i < a.budget; i += 32) {
            const int page = page_of(q, i);
            if (page < 0) continue;
            const uint32_t bit = 1u << ((page & 3) * 8 + q);
            twice |= (atomicOr(&s_rows[page >> 2], bit) & bit) != 0;
        }
    bool single = __syncthreads_or(twice);
    if (!single) {
        const uint8_t *rows_of = reinterpret_cast<const uint8_t *>(s_rows);
        for (int p0 = 0; p0 < seen; p0 += kTileList) {
            // pages that some row names, in order: a few in a row per thread
            constexpr int PER = kTileList / THREADS;
            const int p = p0 + tid * PER;
            int mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) mine += p + i < seen && rows_of[p + i];
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
                    if (p + i < seen && rows_of[p + i]) s_list[before++] = entry(p + i, rows_of[p + i]);
            __syncthreads();
            attend(all);
            __syncthreads();
        }
        bool bad = !isfinite(w.l[0]) || !isfinite(w.l[1]);
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) bad |= !isfinite(w.o[j][i]);
        single = __syncthreads_or(bad);
    }
    // the sums of columns c0 .. c1 - 1 joined and written (part takes the
    // lists' place)
    auto finish = [&](int c0, int c1) {
        __syncthreads();
        w.leave(part[warp], lane);
        __syncthreads();
        // what each warp counts for in a row's sum, then 8 dims at a time
        if (tid < 16 * MT) {
            const Partial<D, 2> *p = part + tid / 16;          // part[split * MT + mt]
            const int c = tid % 16;
            float top = -INFINITY, z = 0.f, f[SPLITS];
#pragma unroll
            for (int i = 0; i < SPLITS; ++i) top = fmaxf(top, p[i * MT].m[c]);
#pragma unroll
            for (int i = 0; i < SPLITS; ++i) {
                f[i] = share(p[i * MT].m[c], p[i * MT].l[c], top);
                z += f[i] * p[i * MT].l[c];
            }
#pragma unroll
            for (int i = 0; i < SPLITS; ++i) s_share[i][tid] = z == 0.f ? 0.f : f[i] / z;
            if (tid >= c0 && tid < c1 && a.lse)
                a.lse[q_row(tid)] = z == 0.f ? -INFINITY : (top + log2f(z)) * 0.69314718055994531f;
        }
        __syncthreads();
        for (int x = c0 * CH + tid; x < c1 * CH; x += THREADS) {
            const int c = x / CH, e = x % CH * 8;
            float sum[8] = {};
#pragma unroll
            for (int i = 0; i < SPLITS; ++i) {
                const float f = s_share[i][c];
                const float *p = &part[i * MT + c / 16].o[c % 16][e];
                const float4 u = *reinterpret_cast<const float4 *>(p), v = *reinterpret_cast<const float4 *>(p + 4);
                // (a warp that saw no key counts for nothing, whatever it holds)
                if (f != 0.f) {
                    sum[0] += f * u.x; sum[1] += f * u.y; sum[2] += f * u.z; sum[3] += f * u.w;
                    sum[4] += f * v.x; sum[5] += f * v.y; sum[6] += f * v.z; sum[7] += f * v.w;
                }
            }
            uint4 out;
            uint32_t *o = &out.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(sum[2 * i], sum[2 * i + 1]);
                o[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *reinterpret_cast<uint4 *>(a.out + q_row(c) * D + e) = out;
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
                s_list[i] = page < 0 ? Page{0, 0, 0} : entry(page, 1 << q);
            }
            __syncthreads();
            attend(n);
        }
        finish(q * a.G, (q + 1) * a.G);
    }
}

template <int D, int NT, int OCC>
cudaError_t launch_sparse(SparseArgs a, cudaStream_t stream) {
    a.parts = (a.G + 8 * NT - 1) / (8 * NT);
    const int64_t units = (int64_t)a.L * a.rows.T * a.Hkv * a.parts;
    // few rows: several CTAs to each, as long as all of them run at once (three
    // fit on an SM, four at head dim 64) and each warp has a tile or two.  (24
    // sequences of 128 pages at head dim 128: two each 38 us, one 46; 32 four
    // each, which do not fit, 66 against 50.)
    a.ctas = 1;
    const int64_t tiles = (int64_t)a.budget << (a.bs_log2 - 4), places = (D == 64 ? 4LL : 3LL) * device_sm_count();
    while (a.ctas < kMaxCtas && units * a.ctas * 2 <= places && tiles >= 2LL * kWarps * a.ctas * 2) a.ctas *= 2;
    if (units * a.ctas > INT32_MAX) return cudaErrorInvalidValue;
    return launch_behind(sparse_attn_kernel<D, NT, OCC>, dim3((unsigned)(units * a.ctas)), 32 * kWarps,
                         sizeof(Partial<D, NT>) * kWarps, a.ctas, stream, a);
}

template <int D, int MT>
cudaError_t launch_tile(const SparseArgs &a, cudaStream_t stream) {
    constexpr size_t ring = (size_t)kTileSteps * 64 * D, parts = sizeof(Partial<D, 2>) * kWarps;
    constexpr size_t bytes = kTileMap + (ring > parts ? ring : parts);
    static std::once_flag once[kMaxDevices];
    static bool ok[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(sparse_tile_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)bytes) == cudaSuccess;
    });
    if (!ok[dev]) return cudaErrorInvalidDevice;
    const dim3 grid((unsigned)QueryRows::tiles(a.rows.T, a.rows.S, a.qt), (unsigned)(a.L * a.Hkv));
    return launch_behind(sparse_tile_kernel<D, MT>, grid, 32 * kWarps, bytes, 1, stream, a);
}

}  // namespace
}  // namespace kvp

#include "sparse_tc.cuh"

namespace kvp {
namespace {

template <int D>
cudaError_t launch_for(SparseArgs a, cudaStream_t stream) {
    // chunks by tiles of 128 (query, head) rows on the tensor cores, which cost 12
    // us before their first page (of 8 kv heads at head dim 128, 53 queries 33 us
    // where single rows take 29, 105 queries 33 against 62; at head dim 64 with 4
    // heads 300 queries 29 against 28) and read a page for all their rows whatever
    // part of a tile these fill (64 sequences of 5.4 rows on average 112 us against
    // 126, of 2.4 100 against 86).  Both kinds of tile have a place in shared memory
    // for each page that the table can name; chunks in wider tables are done by
    // single rows (643 queries over 32 pages of 32 tokens 275 us in place of 63)
    const int64_t units = (int64_t)a.rows.T * a.L * a.Hkv;
    if (a.rows.start && a.rows.MB <= kTcPages && a.L * a.Hkv <= 65535 && a.G <= kTcRows / 2 &&
        units * D >= 512LL * device_sm_count() && a.rows.T >= 5LL * a.rows.S &&
        tc_path_supported(a.L, a.NB, a.Hkv, 1 << a.bs_log2)) {
        a.qt = std::min(32, kTcRows / a.G);
        return launch_tc<D>(a, stream);
    }
    // a few rows each of many sequences by tiles of 32 (query, head) rows where
    // that gives a CTA for two places of every SM, by tiles of 16 where those do;
    // single rows, spread over clusters when they are few, otherwise
    if (a.rows.start && a.rows.MB <= kTilePages && a.L * a.Hkv <= 65535) {
        auto many = [&](int qt) { return (int64_t)(a.rows.T / qt) * a.L * a.Hkv >= 2LL * device_sm_count(); };
        a.qt = std::min(8, 32 / a.G);
        if (a.qt > 1 && a.qt * a.G > 16 && many(a.qt)) return launch_tile<D, 2>(a, stream);
        a.qt = std::min(8, 16 / a.G);
        if (a.qt > 1 && many(a.qt)) return launch_tile<D, 1>(a, stream);
    }
    if (a.G > 8) return launch_sparse<D, 2, 2>(a, stream);
    // three CTAs per SM have the registers to load faster (256 of 128 pages at
    // head dim 128: 50 us, with four 64), four come in fewer rounds where three
    // do not hold all rows (512: 89 us against 112, 1024: 173 against 183)
    const bool all = (int64_t)a.L * a.rows.T * a.Hkv <= 3LL * device_sm_count();
    return all ? launch_sparse<D, 1, 3>(a, stream) : launch_sparse<D, 1, 4>(a, stream);
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
