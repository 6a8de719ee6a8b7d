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
// represented exactly, a smaller one is cut at 2^-60.  (fp32 sums would pick
// another token wherever v falls within about 1e-6 of a boundary, and fp64
// arithmetic runs at a small fraction of the integer rate on this part.)
//
// One cluster of up to 8 CTAs per sequence: a row of the vocabulary is cut
// into contiguous runs, one per warp of the cluster, and every warp stores its
// run's sum into every CTA's shared memory, so that one cluster barrier ends a
// pass.  Warp 0 of every CTA walks the tree redundantly on the same numbers
// (all nodes' p(x) and q(x), and the tests of first children, are made ready
// by one lane per node at the start), so the walk needs no communication but
// the sums.  The last pass's run sums tell which run holds the sampled token:
// its CTA's warps read that run alone once more.
//
// Measured: 6.6 us for one chain of 5 over 32000 tokens (launch, the gather,
// one pass and the search, each a memory latency or two), 18.3 us for 8 trees
// of 64 nodes over 32003 (up to 7 passes of about 2 us, one per rejection:
// two barriers, reductions and an L2 latency each), 22.5 us for 64 chains
// over 131072 (67 MB, 3.0 TB/s: load latency and barriers, 7.5 and 4.2 warps
// waiting per issue, and 256 CTAs that put two on 104 SMs and one on 48; the
// passes' issue slots, about 30 instructions a token, make 6 us of it).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/kvp.h"
#include "kvp_internal.h"

namespace kvp {
namespace {

constexpr int kMaxCtas = 8;     // portable cluster size
constexpr int kWarps = 16;
constexpr int kMaxRuns = kMaxCtas * kWarps;
constexpr int kOne = 60;        // fixed-point fraction bits of a weight

struct DraftVerifyArgs {
    const float *target, *draft;
    int64_t t_batch, t_row, d_batch, d_row;   // strides in elements
    const int32_t *parent, *token;
    const float *u, *u_next;
    int32_t n, vocab, run;                    // run: tokens per warp, a multiple of 32
    int32_t *accepted, *count, *next;
};

// p in [0, 1] as fixed point with kOne (60) or 63 fraction bits, cut below:
// the significand, its first bit at p = 1's place, shifted right by 127 minus
// the exponent (PTX shifts clamp, so zeros and subnormals come out as 0).
template <int BITS>
__device__ __forceinline__ uint64_t to_fixed(float p) {
    const uint32_t b = __float_as_uint(p);
    const uint32_t m = b << 8 | 0x80000000u, r = 127u - (b >> 23);
    const uint32_t hi = m >> (63 - BITS), lo = BITS == 63 ? 0u : m << (BITS - 31);
    uint32_t h, l, far;
    asm("shr.u32 %0, %1, %2;" : "=r"(h) : "r"(hi), "r"(r));
    asm("shf.r.clamp.b32 %0, %1, %2, %3;" : "=r"(l) : "r"(lo), "r"(hi), "r"(r));
    asm("shr.u32 %0, %1, %2;" : "=r"(far) : "r"(hi), "r"(r - 32u));
    return (uint64_t)h << 32 | (r > 32u ? far : l);
}
// a probability: NaN and negative values count as 0, values above 1 as 1
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// The weight max(p - c q, 0) of one token: MODE 0 takes c = 0, 1 takes c = 1,
// 2 any c as a 57-bit fraction.
template <int MODE>
__device__ __forceinline__ uint64_t weight(float p, float q, uint64_t c) {
    const uint64_t a = to_fixed<kOne>(prob(p));
    if (MODE == 0) return a;
    uint64_t b;
    if (MODE == 1) {
        b = to_fixed<kOne>(prob(q));
    } else {   // 57 + 63 fraction bits, 60 of them kept
        const uint64_t f = to_fixed<63>(prob(q)), hi = __umul64hi(c, f);
        if (hi >> 56) return 0u;   // c q >= 1 >= p (c reaches 127, and from c q = 16 on 64 bits would not hold it)
        b = hi << 4 | (c * f) >> 60;
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

// How a warp reads its run of a row: element by element; as 16-byte vectors
// (aligned rows); or, for runs of at most 32 * kHeld tokens, once into
// registers, where the passes after a node's second and later rejections find
// the row again.
enum { kScalar = 0, kVector = 1, kHold = 2 };
constexpr int kHeld = 8;

// Sum of the weights of tokens [lo, hi) of one row, this lane's share (lo is
// a multiple of 32).
template <int MODE, int READ>
__device__ __forceinline__ uint64_t run_sum(const float *p, const float *q, uint64_t c, int lo, int hi, int lane,
                                            const float (&hp)[kHeld], const float (&hq)[kHeld]) {
    uint64_t s = 0;
    int x = lo;
    if (READ == kHold) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) s += weight<MODE>(hp[k], hq[k], c);
    } else if (READ == kVector) {
#pragma unroll 4
        for (x = lo + 4 * lane; x + 4 <= hi; x += 128) {
            const float4 u = __ldg(reinterpret_cast<const float4 *>(p + x));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (MODE) v = __ldg(reinterpret_cast<const float4 *>(q + x));
            s += weight<MODE>(u.x, v.x, c) + weight<MODE>(u.y, v.y, c) + weight<MODE>(u.z, v.z, c) +
                 weight<MODE>(u.w, v.w, c);
        }
        for (; x < hi; ++x) s += weight<MODE>(__ldg(p + x), MODE ? __ldg(q + x) : 0.f, c);
    } else {
#pragma unroll 8
        for (x = lo + lane; x < hi; x += 32) s += weight<MODE>(__ldg(p + x), MODE ? __ldg(q + x) : 0.f, c);
    }
    return s;
}

constexpr uint64_t kOneZ = 1ull << 60, kOneC = 1ull << 57, kMaxC = 127ull << 57;

// u q Z < p - c q, in 32 bits where that is beyond doubt (each side's error
// is below 2^-20 of the terms, which are far from underflow), else in 64: fp64 is slow here and every
// later sibling's test is on the walk's critical path.
__device__ __forceinline__ bool accepts(float u, float p, float q, uint64_t c, uint64_t Z) {
    const float cq = __ull2float_rn(c) * 0x1p-57f * q, uqz = u * q * (__ull2float_rn(Z) * 0x1p-60f);
    const float gap = p - cq - uqz;
    const float terms = p + cq + uqz;
    if (terms > 1e-30f && fabsf(gap) > 0x1p-20f * terms) return gap > 0.f;
    return (double)u * q * ((double)Z * 0x1p-60) < p - (double)c * 0x1p-57 * q;
}

struct Walk {              // what warp 0 tells its CTA
    const float *p, *q;    // the row last summed, or to sum
    uint64_t c;            // 57-bit fraction
    int mode;              // weight()'s
    int n_cut;             // without q: rejected tokens, in s_cut
    bool done;             // the sums at hand are the last
    uint64_t at;           // the sampled token's place in the running sum (~0: none)
};

// Inclusive scan over the cluster's run sums, four runs to a lane.
__device__ __forceinline__ uint64_t scan_runs(const uint64_t *run, int lane, uint64_t (&v)[4]) {
    uint64_t s = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) s += v[k] = run[4 * lane + k];
    return warp_scan(s, lane);
}

template <int READ>
__global__ void __launch_bounds__(32 * kWarps, 2) draft_verify_kernel(const DraftVerifyArgs a) {
    __shared__ int s_par[kMaxDraft], s_tok[kMaxDraft], s_cut[kMaxDraft];
    __shared__ float s_p[kMaxDraft], s_q[kMaxDraft], s_u[kMaxDraft];
    __shared__ uint64_t s_run[2][kMaxRuns], s_part[kWarps];
    __shared__ Walk s_walk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(ctas));
    const int b = blockIdx.x / ctas;
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
    if (tid < 2 * kMaxRuns) s_run[0][tid] = 0;  // (runs that a smaller cluster lacks)
    const float u_next = tid == 0 ? a.u_next[b] : 0.f;
    __syncthreads();
    // every CTA has cleared its sums before another stores into them
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");

    // warp 0's walk, the same in every CTA.  rest: children of cur still to
    // be tried; first: nodes that are accepted when tried first (c = 0, Z =
    // 1; a first rejection makes c 1); summed: the sums at hand are those of cur's row and c
    int cur = -1, cnt = 0, n_cut = 0;
    uint64_t c = 0, Z = kOneZ;   // 57 and 60 fraction bits
    bool summed = false, plain = false;   // plain: sample from p itself
    int par0 = -2, par1 = -2;
    uint64_t first = 0;
    if (warp == 0) {
        auto test = [&](int i, int &par) -> bool {
            if (i >= a.n || s_tok[i] < 0) return false;
            par = s_par[i];
            return db ? (double)s_u[i] * s_q[i] < s_p[i] : s_u[i] < s_p[i];
        };
        const bool t0 = test(lane, par0), t1 = test(lane + 32, par1);
        first = (uint64_t)__ballot_sync(0xffffffffu, t0) | (uint64_t)__ballot_sync(0xffffffffu, t1) << 32;
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
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");

    float hp[kHeld], hq[kHeld];
    int pass = 0;
    for (;; ++pass) {
        if (warp == 0) {
            bool need = false;   // the walk waits for a sum
            while (rest != 0 && !need) {
                const int i = __ffsll((long long)rest) - 1;
                rest &= rest - 1;
                bool yes = (first >> i) & 1;
                if (db) {
                    if (c != 0) yes = accepts(s_u[i], s_p[i], s_q[i], c, Z);
                } else {
                    bool cut = false;
                    for (int k = 0; k < n_cut; ++k) cut |= s_cut[k] == s_tok[i];
                    if (n_cut > 0) yes = (double)s_u[i] * ((double)Z * 0x1p-60) < (cut ? 0. : (double)s_p[i]);
                    if (!yes && !cut) {
                        const uint64_t p = to_fixed<kOne>(s_p[i]);
                        Z = Z > p ? Z - p : 0;
                        if (lane == 0) s_cut[n_cut] = s_tok[i];
                        __syncwarp();
                        ++n_cut;
                    }
                }
                if (yes) {
                    cur = i;
                    ++cnt;
                    c = 0;
                    Z = kOneZ;
                    n_cut = 0;
                    summed = false;
                    rest = children(cur);
                } else if (db) {
                    c = min(c + (Z >> 3), kMaxC);
                    need = true;
                }
            }
            const bool done = !need && summed;
            if (lane == 0) {
                s_walk.done = done;
                if (!done) {
                    s_walk.mode = c == 0 || plain ? 0 : c == kOneC ? 1 : 2;
                    s_walk.p = tb + (cur + 1) * a.t_row;
                    s_walk.q = s_walk.mode ? db + (cur + 1) * a.d_row : nullptr;
                    s_walk.c = c;
                    s_walk.n_cut = plain ? 0 : n_cut;
                }
            }
        }
        __syncthreads();
        if (s_walk.done) break;
        const Walk w = s_walk;
        if (READ == kHold && w.mode < 2) {   // (a third pass over a row finds it held)
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                const int x = lo + 32 * k + lane;
                hp[k] = x < hi ? __ldg(w.p + x) : 0.f;
                hq[k] = x < hi && w.mode ? __ldg(w.q + x) : 0.f;
            }
        }
        uint64_t s = w.mode == 0   ? run_sum<0, READ>(w.p, w.q, w.c, lo, hi, lane, hp, hq)
                     : w.mode == 1 ? run_sum<1, READ>(w.p, w.q, w.c, lo, hi, lane, hp, hq)
                                   : run_sum<2, READ>(w.p, w.q, w.c, lo, hi, lane, hp, hq);
        s = warp_sum(s);
        // (the rejected tokens of a certain draft are distinct)
        for (int k = 0; k < w.n_cut; ++k) {
            const int x = s_cut[k];
            if (x >= lo && x < hi) s -= weight<0>(__ldg(w.p + x), 0.f, 0);
        }
        // lane r stores the sum into CTA r.  The next pass stores into the
        // other array, and the one after it here again, when every CTA has
        // been through the next pass's barrier and so has read this one
        if (lane < ctas) {
            uint32_t addr = (uint32_t)__cvta_generic_to_shared(&s_run[pass & 1][rank * kWarps + warp]);
            asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n" : "+r"(addr) : "r"(lane));
            asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(addr), "l"(s) : "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
        if (warp == 0) {
            uint64_t v[4];
            const uint64_t total = __shfl_sync(0xffffffffu, scan_runs(s_run[pass & 1], lane, v), 31);
            Z = total;
            summed = true;
            if (rest == 0 && total == 0 && !plain) {
                // nothing is left of p once its rejected part is taken off:
                // sample from p itself
                plain = true;
                summed = false;
            }
            if (lane == 0) {
                const float v1 = u_next > 0.f ? fminf(u_next, 1.f - 0x1p-24f) : 0.f;
                // (v1 < 1, so 64 fraction bits fit)
                s_walk.at = total ? __umul64hi(to_fixed<63>(v1) << 1, total) : ~0ull;
            }
        }
    }

    // the sampled token is the first whose running sum exceeds `at`: which
    // run, then which part of it (one per warp of its CTA), lane and token
    const Walk w = s_walk;
    if (rank == 0 && tid == 0) {
        a.accepted[b] = cur;
        a.count[b] = cnt;
        if (w.at == ~0ull) a.next[b] = -1;   // p is zero everywhere
    }
    if (w.at != ~0ull) {
        uint64_t v[4];
        const uint64_t inc = scan_runs(s_run[(pass - 1) & 1], lane, v);
        const int f = __ffs(__ballot_sync(0xffffffffu, inc > w.at)) - 1;
        uint64_t start = inc - (v[0] + v[1] + v[2] + v[3]);
        int run = 4 * lane;
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (run == 4 * lane + k && start + v[k] <= w.at) {
                start += v[k];
                ++run;
            }
        start = __shfl_sync(0xffffffffu, start, f);
        run = __shfl_sync(0xffffffffu, run, f);
        if (run / kWarps == (int)rank) {   // (the same for the whole CTA)
            auto token_weight = [&](int x) -> uint64_t {
                for (int k = 0; k < w.n_cut; ++k)
                    if (s_cut[k] == x) return 0;
                const float p = __ldg(w.p + x);
                return w.mode == 0   ? weight<0>(p, 0.f, 0)
                       : w.mode == 1 ? weight<1>(p, __ldg(w.q + x), 0)
                                     : weight<2>(p, __ldg(w.q + x), w.c);
            };
            const int part = a.run / kWarps, share = (part + 31) / 32;
            const int x0 = run * a.run + warp * part;
            const int xl = min(x0 + lane * share, a.vocab);
            const int xe = min(min(xl + share, x0 + part), a.vocab);
            uint64_t s = 0;
#pragma unroll 4
            for (int x = xl; x < xe; ++x) s += token_weight(x);
            const uint64_t in_warp = warp_scan(s, lane);
            if (lane == 31) s_part[warp] = in_warp;
            __syncthreads();
            for (int k = 0; k < warp; ++k) start += s_part[k];
            uint64_t upto = start + in_warp - s;
            if (w.at >= upto && w.at < upto + s) {   // one lane of the CTA
                int x = xl;
                for (; x < xe - 1; ++x) {
                    upto += token_weight(x);
                    if (upto > w.at) break;
                }
                a.next[b] = x;
            }
        }
    }
    // no CTA ends while another may still store into it
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

template <int READ>
cudaError_t launch_draft_verify(const DraftVerifyArgs &a, int32_t batch, int ctas, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)batch * ctas);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, draft_verify_kernel<READ>, a);
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
    if (!target || !u_next || !accepted || !n_accepted || !next_token || batch <= 0 || batch > INT32_MAX / kMaxCtas ||
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
    // the largest cluster with which the batch still runs at once (two CTAs
    // fit on an SM)
    int ctas = kMaxCtas;
    while (ctas > 1 && (int64_t)batch * ctas > 2LL * device_sm_count()) ctas /= 2;
    const int64_t step = 32LL * kWarps * ctas;
    a.run = (int32_t)((vocab + step - 1) / step) * 32;
    a.accepted = accepted;
    a.count = n_accepted;
    a.next = next_token;
    auto vec = [](const float *p, int64_t batch_stride, int64_t row_stride) {
        return ((uintptr_t)p & 15) == 0 && batch_stride % 4 == 0 && row_stride % 4 == 0;
    };
    const bool v4 = vec(target, target_batch_stride, target_row_stride) &&
                    (!draft || vec(draft, draft_batch_stride, draft_row_stride));
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = a.run <= 32 * kHeld ? launch_draft_verify<kHold>(a, batch, ctas, st)
                          : v4                ? launch_draft_verify<kVector>(a, batch, ctas, st)
                                              : launch_draft_verify<kScalar>(a, batch, ctas, st);
    return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}
