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

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 3 : 2) sparse_attn_kernel(const SparseArgs a) {
    constexpr int H = 8 * NT, KC = D / 32, VC = D / 64;
    extern __shared__ __align__(16) unsigned char smem[];
    Partial<D, NT> *part = reinterpret_cast<Partial<D, NT> *>(smem);
    __shared__ int32_t s_page[kList], s_blk[kList];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
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

    // Q as the B operand: column g is a head, the dims of a lane 8 in a row
    uint4 qf[NT][KC];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < KC; ++c)
            qf[n][c] = 8 * n + g < heads ? load16(a.q + (lr * a.Hq + hq0 + 8 * n + g) * D + 32 * c + 8 * t)
                                         : make_uint4(0, 0, 0, 0);
    float o[NT][D / 16][4] = {};
    float m[NT][2], lsum[NT][2];     // of heads 2 t, 2 t + 1; lsum: this lane's tokens only
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, lsum[n][0] = lsum[n][1] = 0.f;

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
            const int64_t row0 = ((head + (int64_t)blk * a.Hkv) << a.bs_log2) + 16 * sub;
            // tokens behind the query's are not read (their slots may hold anything)
            uint4 kv[2][KC], vv[4][VC];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    kv[e][c] = g + 8 * e < valid ? load16(a.k + (row0 + g + 8 * e) * D + 32 * c + 8 * t) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    const int tok = 2 * t + (e & 1) + 8 * (e >> 1);
                    vv[e][c] = tok < valid ? load16(a.v + (row0 + tok) * D + 64 * c + 8 * g) : make_uint4(0, 0, 0, 0);
                }
            float s[NT][4] = {};
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma(s[n], kv[0][c].x, kv[1][c].x, kv[0][c].y, kv[1][c].y, qf[n][c].x, qf[n][c].y);
                    mma(s[n], kv[0][c].z, kv[1][c].z, kv[0][c].w, kv[1][c].w, qf[n][c].z, qf[n][c].w);
                }
            // s[n][0..1]: token g, heads 2 t, 2 t + 1; s[n][2..3]: token g + 8
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = g + 8 * (e >> 1) < valid ? s[n][e] * a.scale_log2 : -INFINITY;
                    raise |= !(s[n][e] <= m[n][e & 1] + 8.f);    // (a NaN too)
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
                        for (int o_ = 4; o_ < 32; o_ <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o_));
                        x = fmaxf(x, m[n][e]);
                        const float f = m[n][e] == -INFINITY ? 0.f : exp2_sfu(m[n][e] - x);
                        m[n][e] = x;
                        lsum[n][e] *= f;
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
                    for (int i2 = 0; i2 < 2; ++i2) {
                        const float z = s[n][2 * e + i2];
                        x[i2] = z == -INFINITY ? 0.f : exp2_sfu(z - m[n][i2]);
                        lsum[n][i2] += x[i2];
                        y[i2] = x[i2] - __bfloat162float(__float2bfloat16_rn(x[i2]));
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
    }
    // the warp's sums into shared memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = lsum[n][e];
#pragma unroll
            for (int o_ = 4; o_ < 32; o_ <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o_);
            if (g == 0) {
                part[warp].m[8 * n + 2 * t + e] = m[n][e];
                part[warp].l[8 * n + 2 * t + e] = x;
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                part[warp].o[8 * n + 2 * t + e][8 * g + j] = o[n][j][e];
                part[warp].o[8 * n + 2 * t + e][VC == 2 ? 64 + 8 * g + j : 8 * g + 4 + j] = o[n][j][2 + e];
            }
        }
    __syncthreads();
    // joined over the CTA's warps (into warp 0's place when there is a
    // cluster), then over the cluster's CTAs
    const bool alone = a.ctas == 1;
    constexpr int PER = H * D / (32 * kWarps);          // values per thread
    float val[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int x = tid + i * 32 * kWarps, hd = x / D, e = x % D;
        float top = part[0].m[hd];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, part[w].m[hd]);
        float sum = 0.f, z = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = share(part[w].m[hd], part[w].l[hd], top);
            sum += f * part[w].o[hd][e];
            z += f * part[w].l[hd];
        }
        val[i] = sum;
        if (alone && hd < heads) put(a, (lr * a.Hq + hq0 + hd) * D + e, e == 0 ? lr * a.Hq + hq0 + hd : -1, sum, z, top);
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
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * a.ctas));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = sizeof(Partial<D, NT>) * kWarps;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, sparse_attn_kernel<D, NT>, a);
    count_launch();
    return e;
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
    cudaError_t e;
    if (desc->head_dim == 64)
        e = a.G <= 8 ? launch_sparse<64, 1>(a, st) : launch_sparse<64, 2>(a, st);
    else
        e = a.G <= 8 ? launch_sparse<128, 1>(a, st) : launch_sparse<128, 2>(a, st);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}
