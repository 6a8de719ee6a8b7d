// Append with the rotation of K and Q by position (sm_103a): new keys into
// their pages rotated, new values as they are, queries rotated beside them,
// and the copy-on-write copies of shared last pages, in one launch.
//
// Pair (x, y) at position p becomes (x cos a - y sin a, y cos a + x sin a),
// a = p * freq.  In turns, a / 2 pi = p * f with only f modulo 1 of account,
// as p is a whole number: f is held as 64-bit fixed point, p * f wraps modulo
// 2^64, and its top 32 bits are the angle to 2^-33 of a turn, beside p times the
// rounding of f (a double's quotient: 2^-56 of a turn for a frequency of 1, so
// 2^-33 at position 2^23 and 2^-25 at 2^31; fp32 p * freq loses 2^-24 p of it).
// The rotation runs in fp32, the result is rounded to bf16 once.
//
// One CTA takes a few tokens of a layer.  Its threads work out the tokens'
// cos and sin once (every head of K and Q uses them) while their first loads
// are in flight.  A unit of work is 2 x W values of a head: W pairs, or a
// plain copy of V or of the dims behind rot_dim; W = 8 makes each a 16-byte
// access, W = 1 serves rot_dim that are no multiple of 16.  Bound by HBM for
// prompts (4 bytes per value moved): 26800 tokens in 2 layers, 48 heads of 128
// in all, 190 us, 6.9 TB/s of 1.32 GB, the rate of a plain copy.  By latency for
// decode steps: 64 beams in 8 layers, of which 59 copy their last page, 8.9 us
// (39 MB), one token in 22 layers 2.8 us.  4-bit pages have a CTA per token and a
// warp per row with accesses of 2 to 8 bytes: 27700 prompt tokens in 2 layers 910
// us, 1.3 TB/s; 64 beams in 8 layers 15 us.
//
// The host describes tokens by runs (a sequence's consecutive slots) and
// their blocks, in the kernel's parameters: 4 bytes per page instead of per
// token, so a prompt of 65536 tokens on 16-token pages is one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "kv4_quant.cuh"
#include "kvp_internal.h"
#include "launch.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;          // units in flight per thread (4: 119 registers, half the warps)
constexpr int kCopies = 8;         // 16-byte copies in flight per thread
constexpr int kMaxTok = 4;         // tokens per CTA
constexpr int kTokMax = 1 << 19;   // tokens per launch

struct Run {
    int32_t tok0;    // first token of the run in this launch
    int32_t pos0;    // its slot in the sequence
    int32_t blk;     // where the run's blocks start (block of pos0 first)
};

template <int NR, int NB_, int NC>
struct RopeArgs {
    void *k_pool, *v_pool;
    int8_t *k_exp, *v_exp;
    const __nv_bfloat16 *k, *v, *q;
    __nv_bfloat16 *q_out;
    const int32_t *positions;
    int32_t L, NB, Hkv, Hq, bs, d;
    int32_t ntok_total, tok_begin, ntok, per_cta;
    int32_t rot, adjacent;
    int32_t nrun, ncow;
    uint32_t div_unit, div_token;      // 2^32 / units of a head and of a token, rounded up
    float scale;
    uint64_t freq[kMaxRot / 2];
    Run run[NR];
    int32_t blk[NB_];
    int32_t cow[3 * NC];
};
// Decode batches pass a small parameter block, prompts a full one.
using SmallArgs = RopeArgs<64, 128, 64>;
using LargeArgs = RopeArgs<512, 4096, 512>;
static_assert(sizeof(LargeArgs) <= 32764, "kernel parameters");

// Where this CTA's tokens go, and their angles.
struct Tokens {
    int64_t row[kMaxTok];      // (block * Hkv) * bs + slot: the row of kv head 0 in layer 0
    float2 turn[kMaxTok][kMaxRot / 2];   // scale * (cos, sin)
};

template <class Args>
__device__ __forceinline__ int32_t place_token(const Args &a, int t, int64_t &row) {
    int lo = 0, hi = a.nrun - 1;       // the run that holds token t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.run[mid].tok0 <= t) lo = mid; else hi = mid - 1;
    }
    const int32_t pos0 = a.run[lo].pos0, pos = pos0 + (t - a.run[lo].tok0);
    const int32_t b = a.blk[a.run[lo].blk + pos / a.bs - pos0 / a.bs];
    row = (int64_t)b * a.Hkv * a.bs + pos % a.bs;
    return pos;
}

template <class Args>
__device__ __forceinline__ void fill_tokens(const Args &a, Tokens &s, int t0, int nt) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int t = i / half, p = i % half;
        int64_t row;
        int32_t pos = place_token(a, t0 + t, row);
        if (p == 0) s.row[t] = row;
        if (a.positions) pos = a.positions[a.tok_begin + t0 + t];
        const uint64_t turns = a.freq[p] * (uint64_t)(int64_t)pos;
        float sn, cs;
        // half turns in [-1, 1)
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn, &cs);
        s.turn[t][p] = make_float2(cs * a.scale, sn * a.scale);
    }
}

__device__ __forceinline__ void rotate(float &x, float &y, float2 w) {
    const float u = __fmaf_rn(x, w.x, -__fmul_rn(y, w.y));
    y = __fmaf_rn(y, w.x, __fmul_rn(x, w.y));
    x = u;
}

template <int W> struct Vec;
template <> struct Vec<8> { using type = uint4; };
template <> struct Vec<1> { using type = unsigned short; };

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// W pairs in two vectors: (x_i, y_i) across them, or adjacent in each.
__device__ __forceinline__ void turn_vec(uint4 &x, uint4 &y, const float2 *w, bool adjacent) {
    uint32_t *xs = &x.x, *ys = &y.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a0 = lo_f(xs[i]), a1 = hi_f(xs[i]), b0 = lo_f(ys[i]), b1 = hi_f(ys[i]);
        if (adjacent) {
            rotate(a0, a1, w[i]);
            rotate(b0, b1, w[4 + i]);
        } else {
            rotate(a0, b0, w[2 * i]);
            rotate(a1, b1, w[2 * i + 1]);
        }
        xs[i] = pack2(a0, a1);
        ys[i] = pack2(b0, b1);
    }
}
__device__ __forceinline__ void turn_vec(unsigned short &x, unsigned short &y, const float2 *w, bool) {
    float a = bf16_bits_to_float(x), b = bf16_bits_to_float(y);
    rotate(a, b, w[0]);
    x = __bfloat16_as_ushort(__float2bfloat16_rn(a));
    y = __bfloat16_as_ushort(__float2bfloat16_rn(b));
}

// Copy-on-write: CTA x of ncow * L copies the used slots of one triple in one
// layer, K and V, one contiguous run per head.
template <class Args>
__device__ __forceinline__ void copy_cow(const Args &a, int x) {
    const int i = x % a.ncow, l = x / a.ncow;
    const int src = a.cow[3 * i], dst = a.cow[3 * i + 1], used = a.cow[3 * i + 2];
    const int64_t run = (int64_t)used * (a.d / 8), tile = (int64_t)a.bs * (a.d / 8);     // 16-byte chunks
    const int64_t step = (int64_t)(dst - src) * a.Hkv * tile, head = ((int64_t)l * a.NB + src) * a.Hkv;
    uint4 *kp = static_cast<uint4 *>(a.k_pool), *vp = static_cast<uint4 *>(a.v_pool);
    if (tile * a.Hkv * 2 <= INT32_MAX) {
        // (a divisor per thread and batch: the loads are what takes time)
        const int total = (int)run * a.Hkv * 2, r = (int)run;
        for (int y0 = threadIdx.x; y0 < total; y0 += kThreads * kCopies) {
            uint4 v[kCopies];
            int at[kCopies];             // chunk behind the source block's first
#pragma unroll
            for (int u = 0; u < kCopies; ++u) {
                const int z = (y0 + u * kThreads) >> 1, h = z / r;
                at[u] = h * (int)tile + (z - h * r);
                if (y0 + u * kThreads < total) v[u] = (y0 & 1 ? vp : kp)[head * tile + at[u]];
            }
#pragma unroll
            for (int u = 0; u < kCopies; ++u)
                if (y0 + u * kThreads < total) (y0 & 1 ? vp : kp)[head * tile + at[u] + step] = v[u];
        }
    } else {
        for (int h = 0; h < a.Hkv; ++h)
            for (int64_t c = threadIdx.x; c < run; c += kThreads) {
                const int64_t at = (head + h) * tile + c;
                kp[at + step] = kp[at];
                vp[at + step] = vp[at];
            }
    }
}

template <int W, class Args>
__global__ void __launch_bounds__(kThreads, 4) rope_append_kernel(const __grid_constant__ Args a) {
    using V = typename Vec<W>::type;
    __shared__ Tokens s;
    griddep_wait();
    const int cow_ctas = a.ncow * a.L;
    if ((int)blockIdx.x < cow_ctas) {
        copy_cow(a, blockIdx.x);
        return;
    }
    const int groups = (a.ntok + a.per_cta - 1) / a.per_cta;
    const int x0 = blockIdx.x - cow_ctas;
    const int l = x0 / groups, t0 = (x0 % groups) * a.per_cta;
    const int nt = min(a.per_cta, a.ntok - t0);
    // units of a token: heads of K, of Q, of V; a head's U units, of which the
    // first R of K and Q are pairs (in halves: W values of each half), the
    // others 2 W values in a row
    const int R = a.rot / 2 / W, U = (a.d + 2 * W - 1) / (2 * W), per_tok = (2 * a.Hkv + a.Hq) * U;
    const int total = nt * per_tok;
    const int64_t tok = l * (int64_t)a.ntok_total + a.tok_begin + t0;
    const int64_t layer = (int64_t)l * a.NB * a.Hkv * a.bs;
    bool ready = false;
    for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < total; i0 += kThreads * kBatch) {
        V x[kBatch], y[kBatch];
        int tt[kBatch], hh[kBatch], uu[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = min(i0 + b * kThreads, total - 1);      // (past the end: the last unit again, not stored)
            const int t = a.per_cta == 1 ? 0 : (int)__umulhi(i, a.div_token), r = i - t * per_tok;
            const int h = U == 1 ? r : (int)__umulhi(r, a.div_unit), u = r - h * U;
            const __nv_bfloat16 *p = h < a.Hkv          ? a.k + ((tok + t) * a.Hkv + h) * a.d
                                     : h < a.Hkv + a.Hq ? a.q + ((tok + t) * a.Hq + h - a.Hkv) * a.d
                                                        : a.v + ((tok + t) * a.Hkv + h - a.Hkv - a.Hq) * a.d;
            const bool halves = u < R && h < a.Hkv + a.Hq && !a.adjacent;
            const int ea = halves ? u * W : 2 * u * W, eb = halves ? ea + a.rot / 2 : ea + W;
            x[b] = *reinterpret_cast<const V *>(p + ea);
            if (eb < a.d) y[b] = *reinterpret_cast<const V *>(p + eb);
            tt[b] = t; hh[b] = h; uu[b] = u;
        }
        if (!ready) {
            fill_tokens(a, s, t0, nt);
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (i0 + b * kThreads >= total) break;
            const int t = tt[b], h = hh[b], u = uu[b];
            const bool is_v = h >= a.Hkv + a.Hq, turned = u < R && !is_v, halves = turned && !a.adjacent;
            const int ea = halves ? u * W : 2 * u * W, eb = halves ? ea + a.rot / 2 : ea + W;
            const int64_t row = layer + s.row[t];
            __nv_bfloat16 *p = h < a.Hkv ? static_cast<__nv_bfloat16 *>(a.k_pool) + (row + (int64_t)h * a.bs) * a.d
                               : !is_v   ? a.q_out + ((tok + t) * a.Hq + h - a.Hkv) * a.d
                                         : static_cast<__nv_bfloat16 *>(a.v_pool) +
                                               (row + (int64_t)(h - a.Hkv - a.Hq) * a.bs) * a.d;
            if (turned) turn_vec(x[b], y[b], s.turn[t] + u * W, a.adjacent);
            *reinterpret_cast<V *>(p + ea) = x[b];
            if (eb < a.d) *reinterpret_cast<V *>(p + eb) = y[b];
        }
    }
}

// 4-bit pages: a CTA per (layer, token), a warp per row.  A row is rotated in
// shared memory and rounded to bf16 (the keys that a bf16 pool would hold),
// then quantised as seq_append does.
template <class Args>
__global__ void __launch_bounds__(kThreads) rope_append4_kernel(const __grid_constant__ Args a) {
    __shared__ Tokens s;
    __shared__ float s_row[kThreads / 32][128];
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, vpl = a.d / 32;
    const int cow_ctas = a.ncow * a.L;
    if ((int)blockIdx.x < cow_ctas) {
        const int i = blockIdx.x % a.ncow, l = blockIdx.x / a.ncow;
        const int src = a.cow[3 * i], dst = a.cow[3 * i + 1], used = a.cow[3 * i + 2];
        const int ch = a.d / 32;       // 16-byte chunks of codes per row
        const int64_t tile = (int64_t)a.bs * ch;
        for (int64_t y = threadIdx.x; y < 2LL * a.Hkv * used * (ch + 1); y += blockDim.x) {
            const int64_t h = y / (2 * used * (ch + 1)), r = y % (2 * used * (ch + 1));
            const bool is_v = r >= used * (ch + 1);
            const int64_t c = is_v ? r - used * (ch + 1) : r;
            const int64_t from = (int64_t)(l * (int64_t)a.NB + src) * a.Hkv + h, to = (l * (int64_t)a.NB + dst) * a.Hkv + h;
            if (c < used * ch) {
                uint4 *pool = static_cast<uint4 *>(is_v ? a.v_pool : a.k_pool);
                pool[to * tile + c] = pool[from * tile + c];
            } else {
                int8_t *pool = is_v ? a.v_exp : a.k_exp;
                pool[to * a.bs + c - used * ch] = pool[from * a.bs + c - used * ch];
            }
        }
        return;
    }
    const int x0 = blockIdx.x - cow_ctas;
    const int l = x0 / a.ntok, t = x0 % a.ntok;
    const int64_t tok = l * (int64_t)a.ntok_total + a.tok_begin + t;
    fill_tokens(a, s, t, 1);
    __syncthreads();
    const int half = a.rot / 2;
    for (int r = warp; r < 2 * a.Hkv + a.Hq; r += kThreads / 32) {
        const int h = r < a.Hkv ? r : r < 2 * a.Hkv ? r - a.Hkv : r - 2 * a.Hkv;
        const bool is_v = r >= a.Hkv && r < 2 * a.Hkv, is_q = r >= 2 * a.Hkv;
        const __nv_bfloat16 *src = (is_q ? a.q + (tok * a.Hq + h) * a.d : (is_v ? a.v : a.k) + (tok * a.Hkv + h) * a.d);
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < vpl; ++j) {
            x[j] = __bfloat162float(src[lane * vpl + j]);
            s_row[warp][lane * vpl + j] = x[j];
        }
        __syncwarp();
        if (!is_v) {
            for (int j = 0; j < vpl; ++j) {
                const int e = lane * vpl + j;
                if (e >= a.rot) continue;
                const int p = a.adjacent ? e / 2 : e % half;
                float u = s_row[warp][a.adjacent ? 2 * p : p], w = s_row[warp][a.adjacent ? 2 * p + 1 : p + half];
                rotate(u, w, s.turn[0][p]);
                const bool second = a.adjacent ? e & 1 : e >= half;
                x[j] = __bfloat162float(__float2bfloat16_rn(second ? w : u));
            }
        }
        if (is_q) {
            for (int j = 0; j < vpl; ++j) a.q_out[(tok * a.Hq + h) * a.d + lane * vpl + j] = __float2bfloat16_rn(x[j]);
        } else {
            const int64_t row = (int64_t)l * a.NB * a.Hkv * a.bs + s.row[0] + (int64_t)h * a.bs;
            store_row4(x, vpl, static_cast<uint8_t *>(is_v ? a.v_pool : a.k_pool) + row * (a.d / 2),
                       (is_v ? a.v_exp : a.k_exp) + row, lane);
        }
        __syncwarp();
    }
}

// One launch over tokens [tok, tok + ntok) given as runs and blocks.
template <class Args>
cudaError_t launch_part(const RopeAppend &r, const Run *run, int nrun, const int32_t *blk, int nblk, int cow0,
                        int ncow, int tok, int ntok, cudaStream_t stream) {
    Args a;   // on the stack: parameters are copied at launch
    a.k_pool = r.k_pool; a.v_pool = r.v_pool;
    a.k_exp = static_cast<int8_t *>(r.k_exp); a.v_exp = static_cast<int8_t *>(r.v_exp);
    a.k = static_cast<const __nv_bfloat16 *>(r.k); a.v = static_cast<const __nv_bfloat16 *>(r.v);
    a.q = static_cast<const __nv_bfloat16 *>(r.q); a.q_out = static_cast<__nv_bfloat16 *>(r.q_out);
    a.positions = r.positions;
    a.L = r.L; a.NB = r.NB; a.Hkv = r.Hkv; a.Hq = r.q ? r.Hq : 0; a.bs = r.bs; a.d = r.d;
    a.ntok_total = r.ntok; a.tok_begin = tok; a.ntok = ntok;
    a.rot = r.rot; a.adjacent = r.adjacent;
    a.nrun = nrun; a.ncow = ncow;
    a.scale = r.scale;
    std::memcpy(a.freq, r.freq, sizeof a.freq);
    std::memcpy(a.run, run, sizeof(Run) * nrun);
    std::memcpy(a.blk, blk, sizeof(int32_t) * nblk);
    std::memcpy(a.cow, r.cow + 3 * cow0, sizeof(int32_t) * 3 * ncow);
    a.per_cta = 1;
    if (r.k_exp) {
        return launch_behind(rope_append4_kernel<Args>, dim3((unsigned)((ncow + ntok) * r.L)), kThreads, 0, 1, stream, a);
    } else {
        // several tokens to a CTA once one each would be many per SM
        const int W = r.rot % 16 == 0 ? 8 : 1, U = (r.d + 2 * W - 1) / (2 * W);
        const int64_t per_tok = (2LL * r.Hkv + a.Hq) * U;
        // x / n as the high word of x * ceil(2^32 / n): exact while x * n < 2^32
        auto magic = [](int64_t n) { return (uint32_t)(((1LL << 32) + n - 1) / n); };
        a.div_unit = U > 1 ? magic(U) : 0;
        a.div_token = magic(per_tok);
        while (a.per_cta < kMaxTok && (int64_t)ntok * r.L > 16LL * a.per_cta * device_sm_count() && per_tok < 16384)
            a.per_cta *= 2;
        const unsigned grid = (unsigned)((ncow + (ntok + a.per_cta - 1) / a.per_cta) * r.L);
        return launch_behind(W == 8 ? rope_append_kernel<8, Args> : rope_append_kernel<1, Args>, dim3(grid), kThreads, 0, 1,
                             stream, a);
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppend &r, cudaStream_t stream) {
    if (r.copies_first) {
        RopeAppend copies = r, tokens = r;
        copies.copies_first = tokens.copies_first = false;
        copies.nseq = tokens.ncow = 0;
        const cudaError_t e = launch_rope_append(copies, stream);
        return e == cudaSuccess ? launch_rope_append(tokens, stream) : e;
    }
    constexpr int NR = 512, NBk = 4096, NC = 512;
    Run run[NR];
    int32_t blk[NBk];
    int nrun = 0, nblk = 0, tok = 0, ntok = 0, cow = 0;
    // what is gathered, as a launch
    auto flush = [&]() -> cudaError_t {
        const int ncow = std::min(NC, r.ncow - cow);
        if (ntok == 0 && ncow == 0) return cudaSuccess;
        const bool small = nrun <= 64 && nblk <= 128 && ncow <= 64;
        const cudaError_t e = small ? launch_part<SmallArgs>(r, run, nrun, blk, nblk, cow, ncow, tok, ntok, stream)
                                    : launch_part<LargeArgs>(r, run, nrun, blk, nblk, cow, ncow, tok, ntok, stream);
        cow += ncow;
        tok += ntok;
        nrun = nblk = ntok = 0;
        return e;
    };
    for (int i = 0; i < r.nseq; ++i) {
        int32_t left = r.seqs[i].ntok, pos = r.seqs[i].pos0;
        const int32_t *b = r.seqs[i].blocks;
        while (left > 0) {
            if (nrun == NR || nblk == NBk || ntok == kTokMax) {
                const cudaError_t e = flush();
                if (e != cudaSuccess) return e;
            }
            const int32_t off = pos % r.bs;
            const int64_t room = (int64_t)(NBk - nblk) * r.bs - off;
            const int32_t take = (int32_t)std::min<int64_t>(std::min<int64_t>(left, kTokMax - ntok), room);
            run[nrun++] = Run{ntok, pos, nblk};
            const int32_t nb = (int32_t)(((int64_t)off + take + r.bs - 1) / r.bs);
            for (int32_t j = 0; j < nb; ++j) blk[nblk++] = b[j];
            ntok += take;
            left -= take;
            pos += take;
            b += ((int64_t)off + take) / r.bs;
        }
    }
    cudaError_t e = flush();
    while (e == cudaSuccess && cow < r.ncow) e = flush();   // copies beyond a launch's share
    return e;
}

}  // namespace kvp
