// Accumulated attention weight per cached token (sm_103a):
//   out[l][s][h][t] = decay * in[l][s][h][t]
//                   + sum over queries i of s at positions >= t, and over the
//                     query heads of kv head h, of exp(scale q.k_t - lse),
// lse being the natural log-sum-exp that the attention call left for that
// query row.  K is read once and V never: a softmax row needs no second pass
// when its log-sum-exp is at hand.
//
// A warp takes 32 consecutive tokens of one (layer, kv head, sequence) and
// keeps their K rows in registers as mma.sync B operands, loaded straight
// from global memory: the contraction may run over the head dimension in any
// order, so lane (t, j) of an 8-token group reads 16 contiguous bytes (dims
// 32 c + 8 j .. + 7 of token t) and Q's fragments are gathered to match.
// That is 64 contiguous bytes per token and instruction, no shared memory,
// and (d / 8) 16-byte loads in flight per lane, which is what a kernel bound
// by HBM needs.  Every row of scores is turned into weights and added up in
// registers; the sum over the rows ends in a transposing reduction that
// leaves lane x with token x, so the store is one 128-byte line.
// This kernel takes at most 16 query rows a sequence (a decode step), whose
// fragments stay in registers while the warp walks `tiles` groups of 32
// tokens; more rows go to the tcgen05 kernel (mass_tc.cu).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/kvp.h"
#include "kvp_internal.h"

namespace kvp {
namespace {

constexpr int kMassWarps = 4;
constexpr int kMassTok = 32;    // tokens per warp and step

// (volatile: products in program order leave the tile's loads ahead of them;
// reordered ones measured 255 instead of 219 us over 32 x about 9000 tokens)
__device__ __forceinline__ void mass_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float mass_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// K rows of 32 tokens: group g (8 tokens), chunk c (32 dims) of lane (t, j).
template <int D>
struct KTile {
    uint4 k[4][D / 32];
};

// Blocks of a warp's 32 tokens from pos0 (a multiple of 32) on, one per
// 16 tokens (bs >= 16, so a group of 8 tokens never crosses a block).
template <int D>
__device__ __forceinline__ void load_k(KTile<D> &kt, const MassLaunch &a, const int32_t *table, int pos0, int len,
                                       size_t head_base, int lane) {
    const __nv_bfloat16 *pool = static_cast<const __nv_bfloat16 *>(a.k_pool);
    const int t = lane >> 2, j = lane & 3;
    const size_t block_stride = ((size_t)a.Hkv << a.bs_log2) * D;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int pos = pos0 + 8 * g + t;
        const bool in = pos < len;
        const int blk = in ? table[pos >> a.bs_log2] : 0;   // (may lie in the kernel's parameters)
        const __nv_bfloat16 *src =
            pool + head_base + (size_t)blk * block_stride + (size_t)(pos & ((1 << a.bs_log2) - 1)) * D + 8 * j;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            kt.k[g][c] = make_uint4(0u, 0u, 0u, 0u);
            if (in) kt.k[g][c] = __ldg(reinterpret_cast<const uint4 *>(src + 32 * c));
        }
    }
}

// One 16-row tile of queries: fragments in load_k's order of dims.
// Words x of lane (t, j): rows t and t + 8, dims 32 c + 8 j .. + 7.
template <int D>
__device__ __forceinline__ void q_frags(uint32_t (&qf)[D / 16][4], const uint4 (&x0)[D / 32],
                                        const uint4 (&x1)[D / 32]) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        qf[2 * c][0] = x0[c].x;      qf[2 * c][1] = x1[c].x;
        qf[2 * c][2] = x0[c].y;      qf[2 * c][3] = x1[c].y;
        qf[2 * c + 1][0] = x0[c].z;  qf[2 * c + 1][1] = x1[c].z;
        qf[2 * c + 1][2] = x0[c].w;  qf[2 * c + 1][3] = x1[c].w;
    }
}

// Adds the weights that one 16-row tile gives the warp's 32 tokens: acc[2 g
// + e] is token 8 g + 2 j + e.  n0, n1: tokens from pos0 on that rows t and
// t + 8 see (<= 0: none).  l0, l1: their log2-sum-exp.
template <int D>
__device__ __forceinline__ void add_tile(float (&acc)[8], const KTile<D> &kt, const uint32_t (&qf)[D / 16][4],
                                         float sc, float l0, float l1, int n0, int n1, int lane) {
    const int j2 = 2 * (lane & 3);
    // warps whose every row sees all 32 tokens skip the selects
    const bool whole = __all_sync(0xffffffffu, n0 >= kMassTok && n1 >= kMassTok);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            mass_mma(s, qf[2 * c], kt.k[g][c].x, kt.k[g][c].y);
            mass_mma(s, qf[2 * c + 1], kt.k[g][c].z, kt.k[g][c].w);
        }
        float e[4] = {mass_exp2(fmaf(s[0], sc, -l0)), mass_exp2(fmaf(s[1], sc, -l0)), mass_exp2(fmaf(s[2], sc, -l1)),
                      mass_exp2(fmaf(s[3], sc, -l1))};
        if (!whole) {   // selects: a masked score may be anything
            e[0] = 8 * g + j2 < n0 ? e[0] : 0.f;
            e[1] = 8 * g + j2 + 1 < n0 ? e[1] : 0.f;
            e[2] = 8 * g + j2 < n1 ? e[2] : 0.f;
            e[3] = 8 * g + j2 + 1 < n1 ? e[3] : 0.f;
        }
        acc[2 * g] += e[0] + e[2];
        acc[2 * g + 1] += e[1] + e[3];
    }
}

// Sums acc over the 8 row lanes t and leaves lane x with token x's sum.
// Three halving steps over t: after them lane (t, j) holds acc index
// b = (t & 1) * 4 + (t & 2) + (t >> 2), i.e. token 8 (b >> 1) + 2 j + (b & 1).
__device__ __forceinline__ float spread(const float (&acc)[8], int lane) {
    const int t = lane >> 2;
    float a4[4], a2[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float keep = (t & 1) ? acc[4 + i] : acc[i], give = (t & 1) ? acc[i] : acc[4 + i];
        a4[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float keep = (t & 2) ? a4[2 + i] : a4[i], give = (t & 2) ? a4[i] : a4[2 + i];
        a2[i] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
    }
    const float keep = (t & 4) ? a2[1] : a2[0], give = (t & 4) ? a2[0] : a2[1];
    const float v = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    // token x = lane's own: held by the lane with b >> 1 = x / 8, j = (x % 8) / 2, b & 1 = x % 2
    const int b = 2 * (lane >> 3) + (lane & 1);
    const int ts = (b >> 2) | (b & 2) | ((b & 1) << 2);
    return __shfl_sync(0xffffffffu, v, ts * 4 + ((lane & 7) >> 1));
}

__device__ __forceinline__ void store_mass(const MassLaunch &a, size_t row, int pos, int len, int prev, float add) {
    if (pos >= len) return;
    float v = add;
    if (a.mass_in && pos < prev) v = fmaf(a.decay, a.mass_in[row + pos], add);
    a.mass_out[row + pos] = v;
}

template <int D, class Image>
__global__ void __launch_bounds__(32 * kMassWarps)
    mass_kernel(const MassLaunch a, const __grid_constant__ Image image) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
    const int kvh = blockIdx.y % a.Hkv, l = blockIdx.y / a.Hkv;
    constexpr bool INLINE = std::is_same<Image, InlineImage>::value;
    const unsigned char *img = reinterpret_cast<const unsigned char *>(&image);
    if (INLINE && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.err = 0;
    const MassSeq sq = INLINE ? reinterpret_cast<const MassSeq *>(img)[s] : a.seqs[s];
    const int first = chunk * a.tiles * kMassWarps * kMassTok;
    if (first >= sq.len) return;
    const int32_t *table = (INLINE ? reinterpret_cast<const int32_t *>(img + a.tables_at) : a.tables) + sq.table;
    const size_t head_base = (((size_t)l * a.NB * a.Hkv + kvh) << a.bs_log2) * D;
    const size_t out_row = (((size_t)l * a.S + s) * a.Hkv + kvh) * (size_t)a.stride;
    const int G = a.G, rows = sq.nq * G;
    const int t = lane >> 2, j = lane & 3;
    const float sc = a.scale_log2;
    const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(a.q);
    // row r: query r / G at position len - nq + r / G, head kvh * G + r % G
    auto row_of = [&](int r) -> size_t {
        return ((size_t)l * a.T + sq.q0 + r / G) * a.Hq + (size_t)kvh * G + r % G;
    };
    // a row without keys (lse -inf) gives nothing; a row past the last one too
    auto lse2 = [&](int r) -> float {
        const float v = r < rows ? a.lse[row_of(r)] : INFINITY;
        return v == -INFINITY ? INFINITY : v * 1.4426950408889634f;
    };
    uint4 x0[D / 32], x1[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        x0[c] = x1[c] = make_uint4(0u, 0u, 0u, 0u);
        if (t < rows) x0[c] = __ldg(reinterpret_cast<const uint4 *>(qb + row_of(t) * D + 32 * c + 8 * j));
        if (t + 8 < rows) x1[c] = __ldg(reinterpret_cast<const uint4 *>(qb + row_of(t + 8) * D + 32 * c + 8 * j));
    }
    uint32_t qf[D / 16][4];
    q_frags<D>(qf, x0, x1);
    const float l0 = lse2(t), l1 = lse2(t + 8);
    const int see0 = t < rows ? sq.len - sq.nq + t / G + 1 : 0;
    const int see1 = t + 8 < rows ? sq.len - sq.nq + (t + 8) / G + 1 : 0;
    for (int i = 0; i < a.tiles; ++i) {
        const int pos0 = first + (i * kMassWarps + warp) * kMassTok;
        if (pos0 >= sq.len) break;
        KTile<D> kt;
        load_k<D>(kt, a, table, pos0, sq.len, head_base, lane);
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        add_tile<D>(acc, kt, qf, sc, l0, l1, see0 - pos0, see1 - pos0, lane);
        store_mass(a, out_row, pos0 + lane, sq.len, sq.prev, spread(acc, lane));
    }
}

template <int D>
cudaError_t launch_mass_d(MassLaunch a, int max_len, const unsigned char *image, size_t bytes, cudaStream_t stream) {
    const int step = kMassWarps * kMassTok;
    const int64_t tiles = ((int64_t)max_len + step - 1) / step;
    // a CTA walks several tiles of tokens once there are CTAs enough to fill
    // the GPU eight times over (one each measured 313 instead of 255 us)
    const int64_t ctas = tiles * a.S * a.L * a.Hkv;
    a.tiles = (int)std::max<int64_t>(1, std::min<int64_t>(8, ctas / (8LL * 8 * device_sm_count())));
    a.chunks = (int)((tiles + a.tiles - 1) / a.tiles);
    if ((int64_t)a.chunks * a.S > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(a.chunks * a.S), (unsigned)(a.L * a.Hkv));
    if (image) {
        InlineImage in;
        std::memcpy(in.b, image, bytes);
        mass_kernel<D, InlineImage><<<grid, 32 * kMassWarps, 0, stream>>>(a, in);
    } else {
        mass_kernel<D, NoImage><<<grid, 32 * kMassWarps, 0, stream>>>(a, NoImage{});
    }
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mass(const MassLaunch &a0, int max_len, const unsigned char *image, size_t bytes, size_t tables_at,
                        cudaStream_t stream) {
    MassLaunch a = a0;
    a.tables_at = (int32_t)tables_at;
    if (image && bytes > kInlineMax) return cudaErrorInvalidValue;
    if (a.D == 64) return launch_mass_d<64>(a, max_len, image, bytes, stream);
    if (a.D == 128) return launch_mass_d<128>(a, max_len, image, bytes, stream);
    return cudaErrorInvalidValue;
}

}  // namespace kvp

using namespace kvp;

namespace {

struct MassLayout {
    size_t seqs, starts, tables, total;
};

// Checks the batch and lays out its image: a zero header (the error word),
// the sequences, a start per SM, then the sequences' block tables.
bool mass_layout(const kvp_attn_desc &d, const int32_t *tables, const int32_t *lens, const int32_t *q_lens, int32_t S,
                 int32_t MB, MassLayout &w) {
    int64_t blocks = 0, rows = 0;
    for (int32_t s = 0; s < S; ++s) {
        const int32_t nq = q_lens ? q_lens[s] : 1;
        if (lens[s] < 0 || nq < 0 || nq > lens[s]) return false;
        const int64_t nb = ((int64_t)lens[s] + d.block_size - 1) / d.block_size;
        if (nb > MB) return false;
        for (int64_t j = 0; j < nb; ++j) {
            const int32_t id = tables[(size_t)s * MB + j];
            if (id < 0 || id >= d.num_blocks) return false;
        }
        blocks += nb;
        rows += nq;
    }
    // (query rows of one kv head, and 128-token tiles over all of them, are
    // counted in 32 bits)
    if (rows * d.num_q_heads > INT32_MAX / 2 ||
        (blocks + S) * (d.block_size / 16) * d.num_layers * d.num_kv_heads > INT32_MAX)
        return false;
    w.seqs = 256;
    w.starts = (w.seqs + sizeof(MassSeq) * (size_t)S + 255) & ~(size_t)255;
    w.tables = (w.starts + sizeof(int4) * (size_t)device_sm_count() + 255) & ~(size_t)255;
    w.total = (w.tables + sizeof(int32_t) * (size_t)blocks + 255) & ~(size_t)255;
    return true;
}

// More than 16 query rows go to the tcgen05 kernel (256 rows over 2 x about
// 7000 tokens: 19 us; the same rows as 16-row tiles on mma.sync took 62 us).
// Up to 16 the register kernel is faster (4 rows over 32 x about 9000 tokens:
// 219 us against 260 us) and starts sooner.
bool use_tc(const MassLaunch &a, int32_t max_q) { return (int64_t)max_q * a.G > 16; }

bool mass_args_ok(const kvp_attn_desc *d, const int32_t *tables, const int32_t *lens, int32_t S, int32_t MB) {
    return attn_desc_ok(d) && d->kv_format == KVP_KV_BF16 && (int64_t)d->num_layers * d->num_kv_heads <= 65535 &&
           S > 0 && MB > 0 && tables && lens;
}

}  // namespace

extern "C" {

size_t kvp_mass_workspace_size(const kvp_attn_desc *desc, const int32_t *block_tables, const int32_t *seq_lens,
                               const int32_t *q_lens, int32_t num_seqs, int32_t max_blocks) {
    MassLayout w{};
    if (!mass_args_ok(desc, block_tables, seq_lens, num_seqs, max_blocks) ||
        !mass_layout(*desc, block_tables, seq_lens, q_lens, num_seqs, max_blocks, w))
        return 0;
    return w.total;
}

int kvp_attention_mass(const void *q, const int32_t *q_lens, const float *lse, const void *k_pool,
                       const int32_t *block_tables, const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks,
                       const kvp_attn_desc *desc, float decay, const float *mass_in, const int32_t *prev_lens,
                       float *mass_out, int64_t mass_stride, void *workspace, size_t ws_bytes, void *stream) {
    MassLayout w{};
    if (!mass_args_ok(desc, block_tables, seq_lens, num_seqs, max_blocks) ||
        !mass_layout(*desc, block_tables, seq_lens, q_lens, num_seqs, max_blocks, w))
        return KVP_ERR_INVALID;
    if (!k_pool || !mass_out || !workspace || ((uintptr_t)workspace & 255) || ws_bytes < w.total)
        return KVP_ERR_INVALID;
    if ((((uintptr_t)q | (uintptr_t)k_pool) & 15) ||
        (((uintptr_t)lse | (uintptr_t)mass_in | (uintptr_t)mass_out) & 3))
        return KVP_ERR_INVALID;
    if (!(decay - decay == 0.f)) return KVP_ERR_INVALID;   // inf or NaN
    const int32_t bs = desc->block_size, S = num_seqs;
    int32_t max_len = 0, max_q = 0;
    int64_t T = 0;
    for (int32_t s = 0; s < S; ++s) {
        const int32_t nq = q_lens ? q_lens[s] : 1;
        if (prev_lens && (prev_lens[s] < 0 || prev_lens[s] > seq_lens[s])) return KVP_ERR_INVALID;
        max_len = std::max(max_len, seq_lens[s]);
        max_q = std::max(max_q, nq);
        T += nq;
    }
    if (mass_stride < max_len || (T > 0 && (!q || !lse))) return KVP_ERR_INVALID;
    if (mass_in && mass_in != mass_out) {   // in place, or apart
        const uintptr_t x = (uintptr_t)mass_in, y = (uintptr_t)mass_out;
        const uintptr_t n = (uintptr_t)desc->num_layers * desc->num_kv_heads * S * (uintptr_t)mass_stride * 4;
        if (x < y + n && y < x + n) return KVP_ERR_INVALID;
    }
    cudaStream_t st = (cudaStream_t)stream;
    if (stream_capturing(st)) return KVP_ERR_STATE;
    if (max_len == 0) return KVP_OK;
    const unsigned char *base = static_cast<const unsigned char *>(workspace);
    MassLaunch a{};
    a.q = q;
    a.k_pool = k_pool;
    a.lse = lse;
    a.mass_in = mass_in;
    a.mass_out = mass_out;
    a.seqs = reinterpret_cast<const MassSeq *>(base + w.seqs);
    a.starts = reinterpret_cast<const int4 *>(base + w.starts);
    a.tables = reinterpret_cast<const int32_t *>(base + w.tables);
    a.err = reinterpret_cast<int32_t *>(workspace);
    a.stride = mass_stride;
    a.L = desc->num_layers; a.S = S; a.T = (int32_t)T;
    a.Hq = desc->num_q_heads; a.Hkv = desc->num_kv_heads; a.G = desc->num_q_heads / desc->num_kv_heads;
    a.D = desc->head_dim; a.NB = desc->num_blocks;
    while ((1 << a.bs_log2) < bs) ++a.bs_log2;
    const float scale = desc->scale > 0.f ? desc->scale : 1.0f / std::sqrt((float)desc->head_dim);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.decay = decay;
    const bool tc = use_tc(a, max_q);
    if (tc && !mass_tc_fits(a)) return KVP_ERR_INVALID;
    int ctas = 0;
    try {
        thread_local std::vector<unsigned char> image;
        image.assign(w.total, 0);
        MassSeq *seqs = reinterpret_cast<MassSeq *>(image.data() + w.seqs);
        int32_t *tabs = reinterpret_cast<int32_t *>(image.data() + w.tables);
        int64_t at = 0;
        int32_t q0 = 0;
        for (int32_t s = 0; s < S; ++s) {
            const int32_t nq = q_lens ? q_lens[s] : 1;
            seqs[s] = MassSeq{seq_lens[s], nq, q0, prev_lens ? prev_lens[s] : seq_lens[s] - nq, at};
            const int64_t nb = ((int64_t)seq_lens[s] + bs - 1) / bs;
            std::copy(block_tables + (size_t)s * max_blocks, block_tables + (size_t)s * max_blocks + nb, tabs + at);
            at += nb;
            q0 += nq;
        }
        if (tc) {
            thread_local std::vector<int4> starts;
            ctas = mass_tc_starts(a, seqs, device_sm_count(), starts);
            std::copy(starts.begin(), starts.end(), reinterpret_cast<int4 *>(image.data() + w.starts));
        }
        // sequences and tables, without the header and the starts
        const size_t head = w.starts - w.seqs, need = head + sizeof(int32_t) * (size_t)at;
        if (!tc && need <= kInlineMax) {
            std::copy(tabs, tabs + at, reinterpret_cast<int32_t *>(image.data() + w.starts));
            a.seqs = nullptr;
            a.tables = nullptr;
            return launch_mass(a, max_len, image.data() + w.seqs, need, head, st) == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
        }
        // pageable source: the copy is staged before the call returns
        if (cudaMemcpyAsync(workspace, image.data(), w.total, cudaMemcpyHostToDevice, st) != cudaSuccess)
            return KVP_ERR_CUDA;
    } catch (const std::bad_alloc &) {
        return KVP_ERR_OOM;
    }
    const cudaError_t e = tc ? launch_mass_tc(a, ctas, st) : launch_mass(a, max_len, nullptr, 0, 0, st);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

}  // extern "C"
