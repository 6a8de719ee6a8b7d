// Accumulated attention weight on the 5th-generation tensor cores (tcgen05 +
// TMA, sm_103a).  (The operator: mass_kernels.cu, whose kernel keeps short
// calls with few query rows.)
//
// S = K Q^T with the tokens as rows: M = 128 cached tokens of one sequence
// and kv head, N = up to 128 query rows, K = d, one tcgen05.mma chain per
// (token tile, query chunk) into TMEM.  A token's weights are then the columns
// of one TMEM lane, so one thread sums them without talking to another, and
// a row of K that is no token (past the end, or an unwritten slot) spoils
// only its own lane, which is not written.
//
// One persistent CTA of 11 warps per SM over a contiguous run of token tiles
// (so that a sequence's queries are loaded once), the runs cut by weight:
//   warp 0      K producer: one TMA box per block and 64-column slab into a
//               ring of 128-token tiles (128 KB in flight per SM)
//   warp 1      MMA issuer (one thread)
//   warp 2      query loader: chunk c of the query rows into buffer c mod 2
//               when it is not there already, by TMA boxes of whole rows (by
//               cp.async for GQA groups that do not tile 128 rows: 3 us longer
//               a chunk), with the rows' log-sum-exps; it clears every step
//               for the MMA issuer
//   warps 3-10  epilogue, two groups of four warps that take turns with the
//               tiles, one thread per token: w = 2^(s * scale - lse) over the
//               chunk's columns, masked by position, added up in fp32 (the
//               chunks with compensation); after the last out = decay * in + sum
// Each group has two S buffers in TMEM (all 512 columns), so the tensor cores
// work ahead of both.  Every wait is bounded, as in the attention kernel.
//
// What bounds it: on long runs the exponentials, 128 x 128 a step at 32 a clock
// and SM.  256 rows over 2 x about 7000 tokens, 8 kv heads of 128 (936 tiles,
// 6.2 a CTA; 32 MB, 7 GFLOP) take 19 us, of which the exponentials need 3 and
// the loads 5; where the rest goes has not been taken apart (the first tile
// waits for the plan's copy and three dependent loads).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>
#include <vector>

#include "../../include/kvp.h"
#include "kvp_internal.h"
#include "tc_ops.cuh"

namespace kvp {
namespace {

constexpr int kTok = 128;           // tokens per tile (rows of S)
constexpr int kChunk = 128;         // query rows per step (columns of S)
constexpr int kMtThreads = 11 * 32;
constexpr int kEpiThreads = 128;    // of one group
constexpr int kMtTmemCols = 512;
constexpr uint32_t kMtWaitLimit = 1u << 22;

template <int D>
struct MtCfg {
    static constexpr int SLABS = D / 64;
    static constexpr int CH = D / 8;                 // 16-byte chunks per row
    static constexpr int SLAB = kTok * 128;          // 64 columns of 128 rows
    static constexpr int OPER = SLABS * SLAB;
    static constexpr int NK = D == 64 ? 8 : 4;       // K ring depth
    static constexpr int Q_OFF = NK * OPER;          // two query buffers
    static constexpr int L_OFF = Q_OFF + 2 * OPER;   // [2][kChunk] negated lse, base 2
    static constexpr int BAR_OFF = L_OFF + 2 * kChunk * 4;
    static constexpr int B_K_FULL = 0, B_K_EMPTY = NK, B_Q_FULL = 2 * NK, B_S_FULL = B_Q_FULL + 4,
                         B_S_EMPTY = B_S_FULL + 4, B_DRAIN = B_S_EMPTY + 4, N_BARS = B_DRAIN + 1;
    static constexpr int MISC_OFF = BAR_OFF + N_BARS * 8;
    static constexpr int SMEM = MISC_OFF + 16 + 1024;
};
static_assert(MtCfg<64>::SMEM <= 227 * 1024 && MtCfg<128>::SMEM <= 227 * 1024, "shared memory");

// (d0, d1) = (a0, a1) * b + (c0, c1) in one packed instruction
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n.reg .b64 ra, rb, rc, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\nmov.b64 rc, {%5, %6};\n"
        "fma.rn.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
// The CTA's tiles in order, and the query chunks of each: every role walks
// them with its own copy.
struct TileWalk {
    const MassLaunch &a;
    int lh, s, pos0, left;
    MassSeq sq;
    int rows, c0, c1;   // query rows, chunks [c0, c1) that some token of the tile is seen by

    __device__ TileWalk(const MassLaunch &l, const int4 &st) : a(l), lh(st.x), s(st.y), pos0(st.z), left(st.w) {
        if (left > 0) {
            sq = a.seqs[s];
            set();
        }
    }
    __device__ void set() {
        rows = sq.nq * a.G;
        const int first = pos0 - (sq.len - sq.nq);   // query that sees the tile's first token
        c0 = first > 0 ? first * a.G / kChunk : 0;
        c1 = rows > kChunk ? (rows + kChunk - 1) / kChunk : 1;
    }
    __device__ void next() {
        if (--left <= 0) return;
        pos0 += kTok;
        while (pos0 >= sq.len) {   // (some sequence holds the tiles that are left)
            pos0 = 0;
            if (++s == a.S) s = 0, ++lh;
            sq = a.seqs[s];
        }
        set();
    }
    __device__ long long group() const { return (long long)lh * a.S + s; }
};

template <int D>
__global__ void __launch_bounds__(kMtThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap,
                   const MassLaunch a, const int box_rows, const int q_tma) {
    using C = MtCfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float *s_l = reinterpret_cast<float *>(smem + C::L_OFF);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    const uint32_t bar0 = saddr(smem + C::BAR_OFF);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < C::NK; ++i) {
            mbar_init(bar(C::B_K_FULL + i), 1);
            mbar_init(bar(C::B_K_EMPTY + i), 1);
        }
        // S buffer i = 2 * group + (the group's step mod 2), cleared by Q_FULL
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(C::B_Q_FULL + i), 64);   // 32 lanes' copies, and their stores of lse
            mbar_init(bar(C::B_S_FULL + i), 1);
            mbar_init(bar(C::B_S_EMPTY + i), kEpiThreads);
        }
        mbar_init(bar(C::B_DRAIN), 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(saddr(s_tmem)),
                     "r"(kMtTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *s_tmem;

    // bounded wait; on a timeout the whole CTA aborts
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        if (mbar_test_wait(b, parity)) return true;
        for (uint32_t i = 0; i < kMtWaitLimit; ++i) {
            if (mbar_try_wait(b, parity)) return true;
            if ((i & 1023) == 1023 && *s_abort) return false;
        }
        *s_abort = 1;
        atomicOr(a.err, KVP_DEVERR_WAIT_TIMEOUT);
        return false;
    };
    // lane 0 waits and the warp follows it
    auto wait_warp = [&](uint32_t b, uint32_t parity) -> bool {
        int ok = 1;
        if (lane == 0) ok = wait(b, parity) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        __syncwarp();
        return ok != 0;
    };
    // bounded wait that records nothing: lets copies and MMAs in flight land
    auto settle = [&](uint32_t b, uint32_t parity) {
        for (uint32_t i = 0; i < kMtWaitLimit && !mbar_try_wait(b, parity); ++i) {
        }
    };
    const uint32_t k_smem = saddr(smem), q_smem = saddr(smem + C::Q_OFF);
    TileWalk w(a, a.starts[blockIdx.x]);

    if (warp == 0) {
        // ------------------------------------------------------------ K
        if (lane == 0) asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        const int bs = 1 << a.bs_log2;
        const int per_tile = kTok / box_rows;        // boxes per slab
        const int k = lane / C::SLABS, slab = lane % C::SLABS;
        uint32_t i = 0;
        // each lane's block id is fetched a tile ahead: its latency would
        // leave a freed ring slot empty
        auto boxes = [&](const TileWalk &t) { return min(per_tile, (t.sq.len - t.pos0 + box_rows - 1) / box_rows); };
        auto block = [&](const TileWalk &t) -> int {
            return t.left > 0 && k < boxes(t) ? __ldg(a.tables + t.sq.table + ((t.pos0 + k * box_rows) >> a.bs_log2)) : 0;
        };
        TileWalk ahead = w;
        int blk_next = block(ahead);
        for (; w.left > 0; w.next(), ++i) {
            const int st = i % C::NK;
            const int nbox = boxes(w), blk = blk_next;
            ahead.next();
            blk_next = block(ahead);
            if (!wait_warp(bar(C::B_K_EMPTY + st), ((i / C::NK) & 1) ^ 1)) break;
            const uint32_t fb = bar(C::B_K_FULL + st);
            if (lane == 0) mbar_expect_tx(fb, (uint32_t)(nbox * C::SLABS * box_rows * 128));
            __syncwarp();
            if (k < nbox) {
                const int kvh = w.lh % a.Hkv, l = w.lh / a.Hkv;
                const int y = ((l * a.NB + blk) * a.Hkv + kvh) * bs + (bs > box_rows ? w.pos0 & (bs - 1) : 0);
                tma_load_2d(k_smem + st * C::OPER + slab * C::SLAB + k * box_rows * 128, &kmap, slab * 64, y, fb);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(fb);
        }
        if (lane == 0)
            for (uint32_t x = i > (uint32_t)C::NK ? i - C::NK : 0u; x < i; ++x)
                settle(bar(C::B_K_FULL + x % C::NK), (x / C::NK) & 1);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        // the whole warp, converged; one elected lane issues
        const bool lead = elect_one();
        const uint32_t tm = uniform(tmem), ks0 = uniform(k_smem), qs0 = uniform(q_smem);
        auto wait_all = [&](uint32_t b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(b, parity)); };
        uint32_t i = 0, steps[2] = {0, 0};
        bool ok = true;
        for (; ok && w.left > 0; w.next(), ++i) {
            const int st = i % C::NK;
            ok = wait_all(bar(C::B_K_FULL + st), (i / C::NK) & 1);
            uint32_t step = i & 1 ? steps[1] : steps[0];
            const int c1 = uniform(w.c1), rows = uniform(w.rows);
            for (int c = uniform(w.c0); ok && c < c1; ++c, ++step) {
                const int b = c & 1, sb = 2 * (i & 1) + (step & 1);
                ok = wait_all(bar(C::B_Q_FULL + sb), (step >> 1) & 1);
                if (ok) ok = wait_all(bar(C::B_S_EMPTY + sb), ((step >> 1) & 1) ^ 1);
                if (!ok) break;
                fence_async_smem();   // Q came through the generic proxy (cp.async)
                tc_after();
                const int n = min(kChunk, rows - c * kChunk);
                const uint32_t idesc = idesc_bf16(kTok, max(16, (n + 15) & ~15), false);
                const uint64_t kd = sdesc(ks0 + st * C::OPER, 16, 1024), qd = sdesc(qs0 + b * C::OPER, 16, 1024);
                const uint32_t d_tm = tm + sb * kChunk;
                if (lead) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t o = ((uint32_t)(x >> 2) * C::SLAB + (uint32_t)(x & 3) * 32) >> 4;
                        umma_ss(d_tm, kd + o, qd + o, idesc, x > 0 ? 1u : 0u);
                    }
                    umma_commit(bar(C::B_S_FULL + sb));
                }
            }
            (i & 1 ? steps[1] : steps[0]) = step;
            if (lead) umma_commit(bar(C::B_K_EMPTY + st));
        }
        if (lead) umma_commit(bar(C::B_DRAIN));
        settle(bar(C::B_DRAIN), 0);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ queries
        const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(a.q);
        if (q_tma && lane == 0)
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
        uint32_t next[2] = {0, 0};        // each group's next step
        // each group's last step that reads buffer 0, 1 (+ 1; 0: none)
        uint32_t used0[2] = {0, 0}, used1[2] = {0, 0};
        long long held[2] = {-1, -1};     // the chunk in it
        // S_EMPTY of a group's step.  Only steps whose successor on the same
        // S buffer this warp has not cleared are waited for, so the barriers'
        // phases are unambiguous
        auto over = [&](uint32_t step, int grp) {
            return wait_warp(bar(C::B_S_EMPTY + 2 * grp + (step & 1)), (step >> 1) & 1);
        };
        bool ok = true;
        for (int grp = 0; ok && w.left > 0; w.next(), grp ^= 1) {
            for (int c = w.c0; c < w.c1; ++c) {
                const int b = c & 1;
                const uint32_t step = next[grp];
                if (step >= 2) ok = over(step - 2, grp);
                const long long tag = (w.group() << 24) + c;   // (rows fit 31 bits, so chunks fit 24)
                if (ok && held[b] != tag) {
                    held[b] = tag;
                    // the buffer's readers are over: this is known of the
                    // group's steps up to two before this one, and up to three
                    // before the other group's next
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint32_t u = b ? used1[g] : used0[g];
                        if (ok && u > 0 && u + (g == grp ? 0 : 1) >= next[g]) ok = over(u - 1, g);
                    }
                    if (!ok) break;
                    const int kvh = w.lh % a.Hkv, l = w.lh / a.Hkv;
                    const int r0 = c * kChunk, n = min(kChunk, w.rows - r0), np = max(16, (n + 15) & ~15);
                    // row r of the chunk: query (r0 + r) / G, head (r0 + r) % G of the group
                    const size_t q_row = ((size_t)l * a.T + w.sq.q0) * a.Hq + (size_t)kvh * a.G;
                    float v[kChunk / 32];
#pragma unroll
                    for (int x = 0; x < kChunk / 32; ++x) {
                        const int r = r0 + lane + 32 * x;
                        v[x] = lane + 32 * x < n ? __ldg(a.lse + q_row + (size_t)(r / a.G) * a.Hq + r % a.G) : -INFINITY;
                    }
                    if (q_tma) {
                        // a box: the kv head's G query heads of max(1, 8 / G)
                        // consecutive tokens, one 64-column slab; boxes past
                        // the last row are read out of range (zero fill)
                        const int tpb = a.G < 8 ? 8 / a.G : 1, rpb = tpb * a.G;
                        const int nbox = (np + rpb - 1) / rpb, box = lane / C::SLABS, slab = lane % C::SLABS;
                        const uint32_t fb = bar(C::B_Q_FULL + 2 * grp + (step & 1));
                        if (lane == 0) mbar_expect_tx(fb, (uint32_t)(nbox * C::SLABS * rpb * 128));
                        __syncwarp();
                        if (box < nbox)
                            tma_load_3d(q_smem + b * C::OPER + slab * C::SLAB + box * rpb * 128, &qmap, slab * 64,
                                        kvh * a.G,
                                        box * rpb < n ? l * a.T + w.sq.q0 + r0 / a.G + box * tpb : a.L * a.T, fb);
                    } else {
                        for (int r = lane; r < np; r += 32) {
                            const bool in = r < n;
                            const __nv_bfloat16 *src = in ? qb + (q_row + (size_t)((r0 + r) / a.G) * a.Hq + (r0 + r) % a.G) * D
                                                          : static_cast<const __nv_bfloat16 *>(a.k_pool);
                            const uint32_t dst = q_smem + b * C::OPER + r * 128;
#pragma unroll
                            for (int ch = 0; ch < C::CH; ++ch)
                                cp_async16(dst + (ch >> 3) * C::SLAB + (((ch & 7) ^ (r & 7)) << 4),
                                           src + (in ? ch * 8 : 0), in ? 16 : 0);
                        }
                    }
                    // a row without keys (lse -inf), or past the last one, gives nothing
#pragma unroll
                    for (int x = 0; x < kChunk / 32; ++x)
                        s_l[b * kChunk + lane + 32 * x] = v[x] == -INFINITY ? -INFINITY : v[x] * -1.4426950408889634f;
                }
                if (!ok) break;
                (b ? used1 : used0)[grp] = step + 1;
                next[grp] = step + 1;
                cp_async_arrive(bar(C::B_Q_FULL + 2 * grp + (step & 1)));
                mbar_arrive(bar(C::B_Q_FULL + 2 * grp + (step & 1)));
            }
        }
        // this warp's copies land before the CTA ends (the boxes of the last
        // two steps that it cleared for each group)
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        if (lane == 0)
            for (int grp = 0; grp < 2; ++grp)
                for (uint32_t x = next[grp] > 2 ? next[grp] - 2 : 0u; x < next[grp]; ++x)
                    settle(bar(C::B_Q_FULL + 2 * grp + (x & 1)), (x >> 1) & 1);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ weights
        const int quarter = warp & 3;          // TMEM lanes this warp may read
        const int grp = warp >= 7 ? 1 : 0;     // warps 3-6, 7-10: each has all four quarters
        const int row = quarter * 32 + lane;   // token of the tile
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        uint32_t step = 0;
        bool ok = true;
        if (grp == 1) w.next();
        for (; ok && w.left > 0; w.next(), w.next()) {
            const int pos = w.pos0 + row;
            const bool in = pos < w.sq.len;
            const size_t at = ((((size_t)(w.lh / a.Hkv) * a.S + w.s) * a.Hkv + w.lh % a.Hkv)) * (size_t)a.stride + pos;
            float old = 0.f;
            if (in && a.mass_in && pos < w.sq.prev) old = a.mass_in[at];
            // the chunks' sums are added up with their roundings carried along
            // (one running sum over 131072 equal weights was off by 3e-4)
            float sum = 0.f, rest = 0.f;
            for (int c = w.c0; c < w.c1; ++c, ++step) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                const int b = c & 1, sb = 2 * grp + (step & 1);
                ok = wait(bar(C::B_Q_FULL + sb), (step >> 1) & 1) && ok;   // (the rows' lse)
                ok = wait(bar(C::B_S_FULL + sb), (step >> 1) & 1) && ok;
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_after();
                const int n = min(kChunk, w.rows - c * kChunk);
                // columns below `from` are queries before the token
                const int from = max(pos - (w.sq.len - w.sq.nq), 0) * a.G - c * kChunk;
                const bool all = __all_sync(0xffffffffu, from <= 0);
                const float *nl = s_l + b * kChunk;
                const uint32_t st = tmem + lanes + sb * kChunk;
                for (int j0 = 0; j0 < n; j0 += 32) {
                    uint32_t x[32];
                    tmem_ld32(st + j0, x);
                    tmem_wait_ld();
                    if (all && j0 + 32 <= n) {
#pragma unroll
                        for (int v = 0; v < 32; v += 4) {
                            const float4 m = *reinterpret_cast<const float4 *>(nl + j0 + v);
                            float y0, y1, y2, y3;
                            fma2(y0, y1, __uint_as_float(x[v]), __uint_as_float(x[v + 1]), a.scale_log2, m.x, m.y);
                            fma2(y2, y3, __uint_as_float(x[v + 2]), __uint_as_float(x[v + 3]), a.scale_log2, m.z, m.w);
                            acc[0] += exp2_sfu(y0);
                            acc[1] += exp2_sfu(y1);
                            acc[2] += exp2_sfu(y2);
                            acc[3] += exp2_sfu(y3);
                        }
                    } else {   // (columns past n hold whatever the query boxes did)
#pragma unroll
                        for (int v = 0; v < 32; ++v) {
                            const int j = j0 + v;
                            const float e = exp2_sfu(fmaf(__uint_as_float(x[v]), a.scale_log2, nl[j]));
                            acc[v & 3] += j >= from && j < n ? e : 0.f;
                        }
                    }
                }
                tc_before();
                mbar_arrive(bar(C::B_S_EMPTY + sb));
                const float x = (acc[0] + acc[1]) + (acc[2] + acc[3]), up = sum + x;
                rest += sum < x ? (x - up) + sum : (sum - up) + x;   // (both are positive)
                sum = up;
            }
            if (ok && in) a.mass_out[at] = fmaf(a.decay, old, isfinite(sum) ? sum + rest : sum);
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kMtTmemCols)
                     : "memory");
}

template <int D>
bool mass_tc_ready() {
    static bool ok[kMaxDevices];
    static std::once_flag once[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return false;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(mass_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       MtCfg<D>::SMEM) == cudaSuccess;
    });
    return ok[dev];
}

template <int D>
cudaError_t launch_mass_tc_d(const MassLaunch &a, int ctas, cudaStream_t stream) {
    if (!mass_tc_ready<D>()) return cudaErrorInvalidDevice;
    const int bs = 1 << a.bs_log2;
    const int box_rows = bs < kTok ? bs : kTok;
    alignas(64) CUtensorMap map;
    std::memset(&map, 0, sizeof map);
    if (!make_pool_map(&map, a.k_pool, D, (long long)a.L * a.NB * a.Hkv * bs, box_rows)) return cudaErrorInvalidValue;
    // query boxes of max(8, G) rows must tile a chunk
    alignas(64) CUtensorMap qmap;
    const bool q_tma = (a.G <= 8 ? 8 % a.G == 0 : kChunk % a.G == 0) && a.T > 0 &&
                       make_q_map(&qmap, a.q, D, a.Hq, (long long)a.L * a.T, a.G);
    if (!q_tma) std::memset(&qmap, 0, sizeof qmap);
    mass_tc_kernel<D><<<ctas, kMtThreads, MtCfg<D>::SMEM, stream>>>(map, qmap, a, box_rows, q_tma ? 1 : 0);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

// Cuts the tiles of all (layer, kv head)s, in order, into `ctas` runs of
// about equal cost: a tile costs its load, or its steps where they take
// longer (a 128-row step measured about half a 32 KB tile's load).
int mass_tc_starts(const MassLaunch &a, const MassSeq *seqs, int32_t ctas_max, std::vector<int4> &starts) {
    std::vector<int64_t> cost((size_t)a.S + 1, 0), tiles((size_t)a.S + 1, 0), w((size_t)a.S, 0);
    for (int32_t s = 0; s < a.S; ++s) {
        const int64_t n = ((int64_t)seqs[s].len + kTok - 1) / kTok;
        const int64_t steps = ((int64_t)seqs[s].nq * a.G + kChunk - 1) / kChunk;
        w[s] = steps > 2 ? steps : 2;
        tiles[s + 1] = tiles[s] + n;
        cost[s + 1] = cost[s] + n * w[s];
    }
    const int64_t lh = (int64_t)a.L * a.Hkv, total = cost[a.S] * lh, all = tiles[a.S] * lh;
    const int ctas = (int)(all < ctas_max ? all : ctas_max);
    starts.assign((size_t)ctas, int4{0, 0, 0, 0});
    int64_t before = 0;
    for (int i = 0; i <= ctas; ++i) {
        int64_t at = all;
        int4 st{0, 0, 0, 0};
        if (i < ctas) {
            const int64_t t = total / ctas * i + total % ctas * i / ctas;
            const int64_t h = t / cost[a.S], rem = t % cost[a.S];
            int32_t lo = 0, hi = a.S - 1;   // the sequence with cost[s] <= rem < cost[s + 1]
            while (lo < hi) {
                const int32_t mid = (lo + hi) / 2;
                if (cost[mid + 1] > rem) hi = mid;
                else lo = mid + 1;
            }
            const int64_t tile = (rem - cost[lo]) / w[lo];
            at = h * tiles[a.S] + tiles[lo] + tile;
            st = int4{(int)h, lo, (int)(tile * kTok), 0};
        }
        if (i > 0) starts[i - 1].w = (int)(at - before);
        if (i < ctas) starts[i] = st;
        before = at;
    }
    return ctas;
}

bool mass_tc_fits(const MassLaunch &a) { return tc_path_supported(a.L, a.NB, a.Hkv, 1 << a.bs_log2); }

cudaError_t launch_mass_tc(const MassLaunch &a, int ctas, cudaStream_t stream) {
    if (ctas <= 0) return cudaSuccess;
    if (a.D == 64) return launch_mass_tc_d<64>(a, ctas, stream);
    if (a.D == 128) return launch_mass_tc_d<128>(a, ctas, stream);
    return cudaErrorInvalidValue;
}

}  // namespace kvp
