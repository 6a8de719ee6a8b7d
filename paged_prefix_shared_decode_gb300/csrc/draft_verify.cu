// Verification of drafted tokens against the target's probabilities
// (sm_103a): which draft node is accepted, and which token follows it.
//
// At a node whose children were drawn one after the other from the draft
// distribution q, with the target's distribution p, the k-th child x is
// accepted with probability min(1, r_k(x) / q(x)), and a rejection leaves
// r_{k+1} = max(r_k - q, 0) normalised, r_0 = p.  Unnormalised, every r_k is
// max(p - c_k q, 0) for one number c_k: with Z_k = sum max(p - c_k q, 0),
// r_k - q is proportional to (p - c_k q) - Z_k q on the support, so
//   c_0 = 0, Z_0 = 1;   c_{k+1} = c_k + Z_k;
//   accept x when u q(x) Z_k < p(x) - c_k q(x).
// A rejection therefore costs one sum over the vocabulary and nothing is
// stored; an accepted child costs two numbers.  The token after the walk is
// the first at which the running sum of max(p - c q, 0) exceeds v times the
// whole.  Without q (a draft that was certain of its tokens) a rejection
// takes p(x) away from p and from Z, so the walk needs no sums at all.
//
// What is decided here is a token, so a sum may not depend on how it was
// split: weights are added as 64-bit fixed point (2^-60), in which addition
// is exact and any order gives the same bits.  An fp32 value from 2^-37 up is
// represented exactly, a smaller one is cut at 2^-60.  (Sums in fp32 picked
// another token wherever v fell within 1e-6 of a boundary; fp64 has one
// unit for 64 lanes on this part, and converting and adding there would take
// ten times as long as reading the row.)
//
// One cluster of kCtas CTAs per sequence: a row of the vocabulary is cut into
// kCtas * kWarps contiguous runs, one per warp, whose sums meet through
// distributed shared memory.  Warp 0 of every CTA walks the tree redundantly
// on the same numbers (all nodes' p(x) and q(x) are gathered at the start), so
// the walk needs no communication but the sums.  The last sum's runs tell
// which warp holds the sampled token: only that run is read again.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/kvp.h"
#include "kvp_internal.h"

namespace kvp {
namespace {

constexpr int kCtas = 8;        // portable cluster size
constexpr int kWarps = 16;
constexpr int kRuns = kCtas * kWarps;
constexpr int kOne = 60;        // fixed-point fraction bits of a weight

struct DraftVerifyArgs {
    const float *target, *draft;
    int64_t t_batch, t_row, d_batch, d_row;   // strides in elements
    const int32_t *parent, *token;
    const float *u, *u_next;
    int32_t n, vocab, run;                    // run: tokens per warp, a multiple of 32
    int32_t *accepted, *count, *next;
};

// p as fixed point with `bits` fraction bits, cut below; p in [0, 1]
__device__ __forceinline__ uint64_t to_fixed(float p, int bits) {
    const uint32_t b = __float_as_uint(p);
    const int sh = (int)(b >> 23) - 150 + bits;
    const uint64_t m = (b & 0x7fffffu) | 0x800000u;
    return b < 0x00800000u ? 0u : sh >= 0 ? m << sh : sh > -24 ? m >> -sh : 0u;
}
// a probability: NaN and negative values count as 0, values above 1 as 1
__device__ __forceinline__ float prob(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

// The weight max(p - c q, 0) of one token: MODE 0 takes c = 0, 1 takes c = 1,
// 2 any c as a 57-bit fraction.
template <int MODE>
__device__ __forceinline__ uint64_t weight(float p, float q, uint64_t c) {
    const uint64_t a = to_fixed(prob(p), kOne);
    if (MODE == 0) return a;
    uint64_t b;
    if (MODE == 1) {
        b = to_fixed(prob(q), kOne);
    } else {   // 57 + 63 fraction bits, 60 of them kept
        const uint64_t f = to_fixed(prob(q), 63);
        b = (__umul64hi(c, f) << 4) | ((c * f) >> 60);
    }
    return a > b ? a - b : 0u;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t x, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Sum of the weights of tokens [lo, hi) of one row, this lane's share.  VEC:
// the rows are 16-byte aligned (lo always is a multiple of 32).
template <int MODE, bool VEC>
__device__ __forceinline__ uint64_t run_sum(const float *p, const float *q, uint64_t c, int lo, int hi, int lane) {
    uint64_t s = 0;
    int x = lo;
    if (VEC) {
#pragma unroll 4
        for (x = lo + 4 * lane; x + 4 <= hi; x += 128) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p + x));
            float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
            if (MODE) b = __ldg(reinterpret_cast<const float4 *>(q + x));
            s += weight<MODE>(a.x, b.x, c) + weight<MODE>(a.y, b.y, c) + weight<MODE>(a.z, b.z, c) +
                 weight<MODE>(a.w, b.w, c);
        }
        for (; x < hi; ++x) s += weight<MODE>(__ldg(p + x), MODE ? __ldg(q + x) : 0.f, c);
    } else {
#pragma unroll 8
        for (x = lo + lane; x < hi; x += 32) s += weight<MODE>(__ldg(p + x), MODE ? __ldg(q + x) : 0.f, c);
    }
    return s;
}

struct Walk {              // what warp 0 tells its CTA
    const float *p, *q;    // the row last summed, or to sum
    uint64_t c;            // 57-bit fraction
    int mode;              // weight()'s
    int n_cut;             // without q: rejected tokens, in s_cut
    bool done;             // the sums at hand are the last
    uint64_t before, at;   // sum of the CTAs before this one; the sampled token's place (~0: none)
};

template <bool VEC>
__global__ void __launch_bounds__(32 * kWarps) draft_verify_kernel(const DraftVerifyArgs a) {
    __shared__ int s_par[kMaxDraft], s_tok[kMaxDraft], s_cut[kMaxDraft];
    __shared__ float s_p[kMaxDraft], s_q[kMaxDraft], s_u[kMaxDraft];
    __shared__ uint64_t s_run[kWarps], s_cta[2];
    __shared__ Walk s_walk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
    const int b = blockIdx.x / kCtas;
    const float *tb = a.target + b * a.t_batch;
    const float *db = a.draft ? a.draft + b * a.d_batch : nullptr;
    if (tid < a.n) {
        const size_t i = (size_t)b * a.n + tid;
        int par = a.parent[i];
        if (par < -1 || par >= tid) par = -1;   // a root, as in tree verify
        const int x = a.token[i];
        const bool ok = x >= 0 && x < a.vocab;
        s_par[tid] = par;
        s_tok[tid] = ok ? x : -1;               // -1: the node does not exist
        s_u[tid] = a.u[i];
        s_p[tid] = ok ? prob(tb[(par + 1) * a.t_row + x]) : 0.f;
        s_q[tid] = ok && db ? prob(db[(par + 1) * a.d_row + x]) : 0.f;
    }
    __syncthreads();

    // warp 0's walk, the same in every CTA.  rest: children of cur still to
    // be tried; summed: the sums at hand are those of cur's row and c
    int cur = -1, cnt = 0, n_cut = 0;
    double c = 0., Z = 1.;
    bool summed = false, plain = false;   // plain: sample from p itself
    int par0 = -2, par1 = -2;
    if (warp == 0) {
        if (lane < a.n && s_tok[lane] >= 0) par0 = s_par[lane];
        if (lane + 32 < a.n && s_tok[lane + 32] >= 0) par1 = s_par[lane + 32];
    }
    auto children = [&](int node) -> uint64_t {
        return (uint64_t)__ballot_sync(0xffffffffu, par0 == node) |
               (uint64_t)__ballot_sync(0xffffffffu, par1 == node) << 32;
    };
    uint64_t rest = warp == 0 ? children(-1) : 0;
    // this warp's run of every row
    const long long begin = (long long)(rank * kWarps + warp) * a.run;
    const int lo = (int)(begin < a.vocab ? begin : a.vocab);
    const int hi = (int)(begin + a.run < a.vocab ? begin + a.run : a.vocab);

    for (int pass = 0;; ++pass) {
        if (warp == 0) {
            bool need = false;   // the walk waits for a sum
            while (rest != 0 && !need) {
                const int i = __ffsll((long long)rest) - 1;
                rest &= rest - 1;
                const double u = s_u[i], p = s_p[i];
                bool yes;
                if (db) {
                    const double q = s_q[i];
                    yes = u * q * Z < p - c * q;
                } else {
                    bool cut = false;
                    for (int k = 0; k < n_cut; ++k) cut |= s_cut[k] == s_tok[i];
                    yes = u * Z < (cut ? 0. : p);
                    if (!yes && !cut) {
                        Z = fmax(Z - p, 0.);
                        if (lane == 0) s_cut[n_cut] = s_tok[i];
                        __syncwarp();
                        ++n_cut;
                    }
                }
                if (yes) {
                    cur = i;
                    ++cnt;
                    c = 0.;
                    Z = 1.;
                    n_cut = 0;
                    summed = false;
                    rest = children(cur);
                } else if (db) {
                    c = fmin(c + Z, 127.);
                    need = true;
                }
            }
            const bool done = !need && summed;
            if (lane == 0) {
                s_walk.done = done;
                if (!done) {
                    s_walk.mode = c == 0. || plain ? 0 : c == 1. ? 1 : 2;
                    s_walk.p = tb + (cur + 1) * a.t_row;
                    s_walk.q = s_walk.mode ? db + (cur + 1) * a.d_row : nullptr;
                    s_walk.c = (uint64_t)(c * 0x1p57);
                    s_walk.n_cut = plain ? 0 : n_cut;
                }
            }
        }
        __syncthreads();
        if (s_walk.done) break;
        const Walk w = s_walk;
        uint64_t s = w.mode == 0   ? run_sum<0, VEC>(w.p, w.q, w.c, lo, hi, lane)
                     : w.mode == 1 ? run_sum<1, VEC>(w.p, w.q, w.c, lo, hi, lane)
                                   : run_sum<2, VEC>(w.p, w.q, w.c, lo, hi, lane);
        s = warp_sum(s);
        // (the rejected tokens of a certain draft are distinct)
        for (int k = 0; k < w.n_cut; ++k) {
            const int x = s_cut[k];
            if (x >= lo && x < hi) s -= weight<0>(__ldg(w.p + x), 0.f, 0);
        }
        if (lane == 0) s_run[warp] = s;
        __syncthreads();
        if (warp == 0) {
            const uint64_t mine = warp_sum(lane < kWarps ? s_run[lane] : 0);
            if (lane == 0) s_cta[pass & 1] = mine;
        }
        // the CTAs' sums meet.  The next pass writes the other word, and the
        // one after it this word again, when every CTA has been through the
        // next pass's barrier and so has read it
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
        if (warp == 0) {
            uint64_t v = 0;
            if (lane < kCtas) {
                uint32_t addr = (uint32_t)__cvta_generic_to_shared(&s_cta[pass & 1]);
                asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n" : "+r"(addr) : "r"(lane));
                asm volatile("ld.shared::cluster.u64 %0, [%1];\n" : "=l"(v) : "r"(addr) : "memory");
            }
            const uint64_t sc = warp_scan(v, lane);
            const uint64_t total = __shfl_sync(0xffffffffu, sc, 31);
            if (lane == (int)rank) {
                float v1 = a.u_next[b];
                v1 = v1 > 0.f ? fminf(v1, 1.f - 0x1p-24f) : 0.f;
                s_walk.before = sc - v;
                s_walk.at = total ? __umul64hi(to_fixed(v1, 64), total) : ~0ull;
            }
            Z = (double)total * 0x1p-60;
            summed = true;
            if (rest == 0 && total == 0 && !plain) {
                // nothing is left of p once its rejected part is taken off:
                // sample from p itself
                plain = true;
                summed = false;
            }
        }
    }

    // the sampled token is the first whose running sum exceeds `at`
    const Walk w = s_walk;
    if (rank == 0 && tid == 0) {
        a.accepted[b] = cur;
        a.count[b] = cnt;
        if (w.at == ~0ull) a.next[b] = -1;   // p is zero everywhere
    }
    const uint64_t mine = lane < kWarps ? s_run[lane] : 0;
    const uint64_t upto = warp_scan(mine, lane);
    const uint64_t end = w.before + __shfl_sync(0xffffffffu, upto, warp);
    const uint64_t start = end - s_run[warp];
    if (w.at != ~0ull && w.at >= start && w.at < end) {
        const uint64_t t = w.at - start;
        auto token_weight = [&](int x) -> uint64_t {
            for (int k = 0; k < w.n_cut; ++k)
                if (s_cut[k] == x) return 0;
            const float p = __ldg(w.p + x);
            return w.mode == 0 ? weight<0>(p, 0.f, 0)
                               : w.mode == 1 ? weight<1>(p, __ldg(w.q + x), 0) : weight<2>(p, __ldg(w.q + x), w.c);
        };
        // which lane's share of the run, then which of its tokens
        const int share = a.run / 32;
        uint64_t s = 0;
#pragma unroll 4
        for (int k = 0; k < share; ++k) {
            const int x = lo + lane * share + k;
            if (x < hi) s += token_weight(x);
        }
        uint64_t inc = warp_scan(s, lane);
        const int f = __ffs(__ballot_sync(0xffffffffu, inc > t)) - 1;
        uint64_t base = __shfl_sync(0xffffffffu, inc - s, f);
        for (int k = 0; k < share; k += 32) {
            const int x = lo + f * share + k + lane;
            inc = base + warp_scan(k + lane < share && x < hi ? token_weight(x) : 0, lane);
            const uint32_t hit = __ballot_sync(0xffffffffu, inc > t);
            if (hit) {
                if (lane == 0) a.next[b] = lo + f * share + k + __ffs(hit) - 1;
                break;
            }
            base = __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    // every CTA's sum has been read before any CTA ends
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

template <bool VEC>
cudaError_t launch_draft_verify(const DraftVerifyArgs &a, int32_t batch, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)batch * kCtas);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, draft_verify_kernel<VEC>, a);
    count_launch();
    return e;
}

}  // namespace
}  // namespace kvp

extern "C" int kvp_draft_verify(const float *target, int64_t target_batch_stride, int64_t target_row_stride,
                                const float *draft, int64_t draft_batch_stride, int64_t draft_row_stride,
                                const int32_t *tree_parent, const int32_t *draft_tokens, const float *u_accept,
                                const float *u_next, int32_t batch, int32_t n_draft, int32_t vocab,
                                int32_t *accepted, int32_t *n_accepted, int32_t *next_token, void *stream) {
    using namespace kvp;
    if (!target || !u_next || !accepted || !n_accepted || !next_token || batch <= 0 || batch > INT32_MAX / kCtas ||
        n_draft < 0 || n_draft > kMaxDraft || vocab <= 0 || vocab > (1 << 30))
        return KVP_ERR_INVALID;
    if (n_draft > 0 && (!tree_parent || !draft_tokens || !u_accept)) return KVP_ERR_INVALID;
    if (target_batch_stride < 0 || target_row_stride < 0) return KVP_ERR_INVALID;
    if (draft && (draft_batch_stride < 0 || draft_row_stride < 0)) return KVP_ERR_INVALID;
    const uintptr_t words = (uintptr_t)target | (uintptr_t)draft | (uintptr_t)tree_parent | (uintptr_t)draft_tokens |
                            (uintptr_t)u_accept | (uintptr_t)u_next | (uintptr_t)accepted | (uintptr_t)n_accepted |
                            (uintptr_t)next_token;
    if (words & 3) return KVP_ERR_INVALID;
    DraftVerifyArgs a{};
    a.target = target;
    a.draft = draft;
    a.t_batch = target_batch_stride;
    a.t_row = target_row_stride;
    a.d_batch = draft_batch_stride;
    a.d_row = draft_row_stride;
    a.parent = tree_parent;
    a.token = draft_tokens;
    a.u = u_accept;
    a.u_next = u_next;
    a.n = n_draft;
    a.vocab = vocab;
    a.run = (int32_t)(((int64_t)vocab + 32 * kRuns - 1) / (32 * kRuns)) * 32;
    a.accepted = accepted;
    a.count = n_accepted;
    a.next = next_token;
    auto vec = [](const float *p, int64_t batch_stride, int64_t row_stride) {
        return ((uintptr_t)p & 15) == 0 && batch_stride % 4 == 0 && row_stride % 4 == 0;
    };
    const bool v4 = vec(target, target_batch_stride, target_row_stride) &&
                    (!draft || vec(draft, draft_batch_stride, draft_row_stride));
    const cudaError_t e = v4 ? launch_draft_verify<true>(a, batch, (cudaStream_t)stream)
                             : launch_draft_verify<false>(a, batch, (cudaStream_t)stream);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}
