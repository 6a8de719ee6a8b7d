// Attention of prompt chunks over selected pages on the 5th-generation tensor
// cores (tcgen05, sm_103a): up to 32 consecutive query rows of a sequence with
// their group's heads, 128 (query, head) rows, share a tile that reads each
// page that any of them names once.  (The operator, and the kernels for single
// rows, few rows and small groups: sparse_attn.cu.)
//
// Which rows name a page is a word per page in shared memory.  Its pages, in
// ascending order, are cut into groups of 16 tokens, and eight groups are a
// step: S = Q K^T (M = 128 rows, N = 128 tokens) into TMEM, two threads per row
// turn their halves of it into weights, and O += P V with P read from TMEM.  P
// stands in S's place, as two bf16 numbers a weight: for 32 tokens 16 columns of
// their roundings and 16 of the rest.
//
// A step is a chain of S, maximum, exponentials and P V in which each part
// waits for the one before, and an SM holds one CTA (TMEM).  So the even and the
// odd steps are two chains side by side, each with its places for K, V and S /
// P, its warps, its O, reference and sum; the two are joined at the end.  S of
// both and both O are all 512 columns of TMEM at head dim 128.
//
//   warps 0-15   softmax: warp w has the steps of parity w / 8, rows 32 (w mod 4)
//                .. + 31, tokens 64 (w / 4 mod 2) .. + 63; at the end they write
//                out and lse
//   warp 16, 17  producers of K, V: a TMA box per run of 16 to 128 tokens and
//                64-column slab, cp.async for a page's ragged end; warp 16 also
//                leaves what the groups are
//   warp 18, 19  MMA issuers of the even, odd steps (one elected lane)
//
// A token that no row of the tile sees (past the last one's position) is read as
// zeros, whatever the page holds.  A NaN or an infinity in a page that some rows
// name reaches the others too, as 0 times that, and a row that names a page
// twice counts it twice: both are found, and such a tile's rows are then done
// one after the other, each by its own list, in slow_row().  So are those of a
// tile with scores beyond kLargestScore.
//
// Every wait is bounded; should one run out, the tile's results are NaN.
//
// Bound by the chain of a step, 2300 cycles for 128 tokens of which the products
// are 1536, and by 12 us before a tile's first page and after its last (Q, the
// lists and the table in sequence, the join).  643 queries over 32 pages of 32
// tokens, 8 kv heads of four query heads at d 128: 65 us (176 tiles of about 70
// pages on 152 SMs, two rounds; tiles of 32 rows on mma.sync 144 us), 194
// queries 37 us.  One chain with one MMA issuer and steps of 64 tokens took 78
// us, a TMA box per 16 tokens with the groups worked out one by one 87, cp.async
// for everything 92.
#pragma once
#include "tc_ops.cuh"

namespace kvp {
namespace {

constexpr int kTcThreads = 20 * 32;
constexpr int kTcRows = 128;         // (query, head) rows of a tile
constexpr int kTcPages = 4096;       // pages of a sequence that a tile's map covers
constexpr int kTcStep = 128;         // tokens of a step
constexpr int kTcGroups = kTcStep / 16;
constexpr int kTcCols = 512;         // TMEM columns: S / P of two steps, both O
constexpr int kTcSlots = 8;          // steps whose groups are kept
constexpr uint32_t kTcWaitLimit = 1u << 22;

struct Group {                       // 16 tokens of a page
    int32_t first;                   // position of its first token
    uint32_t rows;                   // query rows that name the page
};

template <int D>
struct TcCfg {
    static constexpr int SLABS = D / 64, CH = D / 8;
    static constexpr int Q_SLAB = kTcRows * 128, SLAB = kTcStep * 128, OPER = SLABS * SLAB;
    static constexpr int K_OFF = SLABS * Q_SLAB, V_OFF = K_OFF + 2 * OPER, MAP_OFF = V_OFF + 2 * OPER;
    // [kTcSlots][kTcGroups] groups.  Those of step i are written after K of steps
    // i - 1 and i - 2 had its place, so after S of steps i - 3 and i - 4 and P of
    // steps i - 5 and i - 6: the slot's readers are done
    static constexpr int LIST_OFF = MAP_OFF + kTcPages * 4, GROUP_OFF = LIST_OFF + kTcPages * 2;
    static_assert(kTcSlots >= 5);
    // [S buffer][half][row] largest score; [parity][half][row] sum, [parity][row] reference
    static constexpr int TOP_OFF = GROUP_OFF + kTcSlots * kTcGroups * 8;
    static constexpr int SUM_OFF = TOP_OFF + 4 * kTcRows * 4;
    static constexpr int BAR_OFF = SUM_OFF + 6 * kTcRows * 4;
    // (S of a step frees its K's place, P V its V's)
    static constexpr int B_K_FULL = 0, B_V_FULL = 2, B_S_FULL = 4, B_P_FULL = 6, B_PV_DONE = 8, B_TOP = 10,
                         B_SUM = B_TOP + 8, B_DRAIN = B_SUM + 4, B_G_FULL = B_DRAIN + 1, N_BARS = B_G_FULL + kTcSlots;
    static constexpr int MISC_OFF = BAR_OFF + N_BARS * 8;
    static constexpr int SMEM = MISC_OFF + 96 + 1024;            // (the base is aligned to 1024)
};
static_assert(TcCfg<128>::SMEM <= 227 * 1024 && TcCfg<64>::SMEM <= 227 * 1024, "shared memory");

// (d0, d1) = (a0, a1) * b + (c0, c1), (a0, a1) + (c0, c1) in one packed instruction
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n.reg .b64 ra, rb, rc, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\nmov.b64 rc, {%5, %6};\n"
        "fma.rn.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1, float c0, float c1) {
    asm("{\n.reg .b64 ra, rc, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rc, {%4, %5};\nadd.rn.f32x2 rd, ra, rc;\n"
        "mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(c0), "f"(c1));
}

// One (query, head) row by a warp, from its own list: a token per lane for the
// scores, D / 32 dims per lane for the output.
template <int D>
__device__ void slow_row(const SparseArgs &a, int64_t row, int pos, const int32_t *table, const int32_t *sel,
                         int64_t head, int lane) {
    constexpr int PER = D / 32;
    const __nv_bfloat16 *q = a.q + row * D;
    float o[PER] = {}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < a.budget; ++i) {
        const int page = sel[i];
        if (page < 0 || pos < 0 || page > pos >> a.bs_log2) continue;
        const int blk = table[page];
        if ((unsigned)blk >= (unsigned)a.NB) continue;
        const int64_t at = ((head + (int64_t)blk * a.Hkv) << a.bs_log2) * D;
        const int n = min(1 << a.bs_log2, pos - (page << a.bs_log2) + 1);
        for (int t0 = 0; t0 < n; t0 += 32) {
            float s = -INFINITY;
            if (t0 + lane < n) {
                const uint4 *k = reinterpret_cast<const uint4 *>(a.k + at + (int64_t)(t0 + lane) * D);
                s = 0.f;
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = k[c], y = load16(q + 8 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u = word(x, e), v = word(y, e);
                        s = fmaf(__uint_as_float(u << 16), __uint_as_float(v << 16), s);
                        s = fmaf(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u), s);
                    }
                }
                s *= a.scale_log2;
            }
            float top = fmaxf(s, m);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float f = m == top ? 1.f : exp2_sfu(m - top);
            m = top;
            const float p = s == -INFINITY ? 0.f : exp2_sfu(s - m);
            l = fmaf(l, f, p);
#pragma unroll
            for (int e = 0; e < PER; ++e) o[e] *= f;
            for (int t = 0; t < min(32, n - t0); ++t) {
                const float w = __shfl_sync(0xffffffffu, p, t);
                const __nv_bfloat16 *v = a.v + at + (int64_t)(t0 + t) * D + PER * lane;
#pragma unroll
                for (int e = 0; e < PER; ++e) o[e] = fmaf(w, __bfloat162float(v[e]), o[e]);
            }
        }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
    for (int e = 0; e < PER; ++e) put(a, row * D + PER * lane + e, e == 0 && lane == 0 ? row : -1, o[e], l, m);
}

// The 16-token groups of a tile's pages in order, 32 at a time, a group per
// lane; the blocks of the next 32 are on their way while these are used.
struct GroupWalk {
    const uint32_t *map;             // rows per page
    const uint16_t *list;            // pages
    const int32_t *table;
    int n, sub_log2, page_next, blk_next;

    __device__ __forceinline__ void peek(int j) {
        page_next = j < n ? list[j >> sub_log2] : 0;
        blk_next = j < n ? __ldg(table + page_next) : 0;
    }
    // group j of this lane (of n); tokens that no row sees: valid 0
    __device__ __forceinline__ void take(const SparseArgs &a, int j, int64_t head, int pos0, Group &x, int &at, int &valid) {
        x.first = 0;
        x.rows = 0;
        at = valid = 0;
        if (j < n) {
            const int sub = 16 * (j & ((1 << sub_log2) - 1));
            x.first = (page_next << a.bs_log2) + sub;
            x.rows = map[page_next];
            at = (int)((head + (int64_t)blk_next * a.Hkv) << a.bs_log2) + sub;
            valid = max(min(16, pos0 + 31 - __clz(x.rows) - x.first + 1), 0);
        }
        peek(j + 32);
    }
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    sparse_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const SparseArgs a, const int box_rows) {
    using C = TcCfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint32_t *s_map = reinterpret_cast<uint32_t *>(smem + C::MAP_OFF);
    float *s_top = reinterpret_cast<float *>(smem + C::TOP_OFF);
    float *s_sum = reinterpret_cast<float *>(smem + C::SUM_OFF);
    Group *s_group = reinterpret_cast<Group *>(smem + C::GROUP_OFF);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    int *s_scan = reinterpret_cast<int *>(smem + C::MISC_OFF + 8);
    uint16_t *s_list = reinterpret_cast<uint16_t *>(smem + C::LIST_OFF);
    const uint32_t bar0 = saddr(smem + C::BAR_OFF);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_wait();
    if (warp == 0 && lane < a.rows.S) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(a.rows.lens + lane));
    const int h = blockIdx.y % a.Hkv, l = blockIdx.y / a.Hkv;
    int r0, nr, seq;
    if (!a.rows.tile(a.qt, blockIdx.x, r0, nr, seq)) return;
    const int cols = nr * a.G;
    const int64_t lr0 = (int64_t)l * a.rows.T + r0;
    // the entries of a warp's rows are on their way before anything waits
    constexpr int WARPS = kTcThreads / 32, PER = (32 + WARPS - 1) / WARPS;
    const int32_t *sel = a.selected + (lr0 * a.Hkv + h) * a.budget;
    const int64_t sel_row = (int64_t)a.Hkv * a.budget;
    int page[PER];
    auto entries = [&](int i) {
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            const int q = warp + x * WARPS;
            page[x] = q < nr && i < a.budget ? __ldg(sel + q * sel_row + i) : -1;
        }
    };
    entries(lane);
    const int pos0 = a.rows.position(seq, r0);
    const int seen = min(a.rows.pages(seq, r0 + nr - 1), kTcPages);
    auto q_row = [&](int c) { return (lr0 + c / a.G) * a.Hq + h * a.G + c % a.G; };   // row of q, out, lse
    const int64_t head = (int64_t)l * a.NB * a.Hkv + h;
    const int32_t *table = a.rows.tables + (int64_t)seq * a.rows.MB;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::B_K_FULL + i), 32);
            mbar_init(bar(C::B_V_FULL + i), 32);
            mbar_init(bar(C::B_S_FULL + i), 1);
            mbar_init(bar(C::B_P_FULL + i), 8);          // warps
            mbar_init(bar(C::B_PV_DONE + i), 1);
        }
        for (int i = 0; i < 8; ++i) mbar_init(bar(C::B_TOP + i), 2);    // [parity][quarter]
        for (int i = 0; i < 4; ++i) mbar_init(bar(C::B_SUM + i), 4);
        for (int i = 0; i < kTcSlots; ++i) mbar_init(bar(C::B_G_FULL + i), 1);
        mbar_init(bar(C::B_DRAIN), 2);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 18) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(saddr(s_tmem)),
                     "r"(kTcCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    // Q, and zeros behind the last row
    const uint32_t q_smem = saddr(smem), k_smem = saddr(smem + C::K_OFF), v_smem = saddr(smem + C::V_OFF);
    {
        // a thread's rows are a multiple of 8 apart, so that their swizzle is one;
        // r / G by a product (exact for r < 128)
        constexpr int EACH = kTcThreads / C::CH;
        static_assert(EACH % 8 == 0 && kTcThreads % C::CH == 0);
        const int c = tid % C::CH, first = tid / C::CH, inv = (65535 + a.G) / a.G;
        const uint32_t to = q_smem + (c >> 3) * C::Q_SLAB + (((c & 7) ^ (first & 7)) << 4);
        const __nv_bfloat16 *from = a.q + (lr0 * a.Hq + h * a.G) * D + 8 * c;
        for (int r = first; r < kTcRows; r += EACH) {
            const int q = r * inv >> 16;
            cp_async16(to + r * 128, r < cols ? from + (int64_t)(q * (a.Hq - a.G) + r) * D : a.q, r < cols ? 16 : 0);
        }
    }
    for (int i = tid; i < (seen + 3) / 4; i += kTcThreads) reinterpret_cast<uint4 *>(s_map)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (tid * 32 < seen) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(table + tid * 32));
    bool twice = false;
    for (int i = lane; i < a.budget; i += 32) {
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            const int q = warp + x * WARPS, pos = pos0 + q;
            if (page[x] >= 0 && pos >= 0 && page[x] <= pos >> a.bs_log2 && page[x] < seen)
                twice |= (atomicOr(&s_map[page[x]], 1u << q) >> q & 1) != 0;
        }
        entries(i + 32);
    }
    const bool again = __syncthreads_or(twice);
    // the pages in order, those without a block passed over: a few per thread
    constexpr int MOST = (kTcPages + kTcThreads - 1) / kTcThreads;
    const int each = (seen + kTcThreads - 1) / kTcThreads, p0 = tid * each;
    uint32_t named = 0;
    if (!again) {
#pragma unroll
        for (int x = 0; x < MOST; ++x)
            if (x < each && p0 + x < seen && s_map[p0 + x] && (unsigned)__ldg(table + p0 + x) < (unsigned)a.NB) named |= 1u << x;
    }
    int before = __popc(named);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) s_scan[warp] = before;
    __syncthreads();
    before -= __popc(named);
    int pages = 0;
#pragma unroll
    for (int x = 0; x < WARPS; ++x) {
        before += x < warp ? s_scan[x] : 0;
        pages += s_scan[x];
    }
    for (; named; named &= named - 1) s_list[before++] = (uint16_t)(p0 + __ffs(named) - 1);
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    fence_async_smem();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *s_tmem;
    const int sub_log2 = a.bs_log2 - 4, groups = pages << sub_log2, steps = (groups + kTcGroups - 1) / kTcGroups;

    // bounded wait; on a timeout the whole CTA gives up
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        if (mbar_test_wait(b, parity)) return true;
        for (uint32_t i = 0; i < kTcWaitLimit; ++i) {
            if (mbar_try_wait(b, parity)) return true;
            if ((i & 1023) == 1023 && *s_abort) return false;
        }
        *s_abort = 1;
        return false;
    };
    auto wait_all = [&](uint32_t b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(b, parity)); };
    bool bad = false;                // a row of this thread that is not finite
    float m = -INFINITY, sum = 0.f;
    // this thread's row of the tile, half of a step, and where O's half is in TMEM
    const int r = (warp & 3) * 32 + lane, half = warp >> 2 & 1, par = warp >> 3 & 1;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) * 32 << 16), o_half = lanes + 2 * kTcStep + half * (D / 2);
    // bounded wait that records nothing: lets copies and products in flight land
    auto settle = [&](uint32_t b, uint32_t parity) {
        for (uint32_t i = 0; i < kTcWaitLimit && !mbar_try_wait(b, parity); ++i) {
        }
    };

    if (warp < 16) {
        // ------------------------------------------------------------ softmax
        // a row past the last one sees nothing
        const int q = r < cols ? r / a.G : 0, pos = r < cols ? pos0 + q : -1;
        const uint32_t o_tm = o_half + par * D;
        for (int i = par; i < steps; i += 2) {
            const int slot = i % kTcSlots;
            const uint32_t phase = (i >> 1) & 1;
            if (!wait_all(bar(C::B_G_FULL + slot), (i / kTcSlots) & 1)) break;
            int n[4], parts = 0;     // tokens of each group that the row sees
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const Group x = s_group[kTcGroups * slot + 4 * half + g];
                n[g] = x.rows >> q & 1 ? min(max(pos - x.first + 1, 0), 16) : 0;
                parts |= n[g];
            }
            // (groups behind the last one have no S)
            const bool whole = __all_sync(0xffffffffu, !(parts & 15)) && (i + 1) * kTcGroups <= groups;
            if (!wait_all(bar(C::B_S_FULL + par), phase)) break;
            tc_after();
            const uint32_t s_tm = lanes + par * kTcStep + 64 * half;
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u) {            // 32 tokens at a time
                uint32_t x[32];
                tmem_ld32(s_tm + 32 * u, x);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int seen = n[2 * u + g];
                    float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (whole) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) y[c % 4] = fmaxf(y[c % 4], __uint_as_float(x[16 * g + c]));
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            y[c % 4] = fmaxf(y[c % 4], c < seen ? __uint_as_float(x[16 * g + c]) : -INFINITY);
                    }
                    if (seen) top = fmaxf(top, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
                }
            }
            s_top[(2 * par + half) * kTcRows + r] = top;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_TOP + 4 * par + (warp & 3)));
            if (!wait_all(bar(C::B_TOP + 4 * par + (warp & 3)), phase)) break;
            top = fmaxf(top, s_top[(2 * par + (half ^ 1)) * kTcRows + r]) * a.scale_log2;
            // the reference is raised only by more than 8 (in powers of two)
            const float before = m;
            if (top > m + 8.f) m = top;
            if (i > 1 && __any_sync(0xffffffffu, m != before && before != -INFINITY)) {
                // (this S came after P V of this parity's step before)
                const float f = m != before ? exp2_sfu(before - m) : 1.f;
                sum *= f;
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t y[32];
                    tmem_ld32(o_tm + c, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                    tmem_st32(o_tm + c, y);
                }
            }
            float part[2] = {};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // (S is read again: 64 of it and of P are more than the registers)
                uint32_t x[32], out[32];
                tmem_ld32(s_tm + 32 * u, x);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    // (a group that the row does not see: exp2(-inf))
                    const int seen = n[2 * u + g];
                    const float ref = seen ? -m : -INFINITY;
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const uint32_t *y = x + 16 * g + c;
                        float p0, p1, l0, l1;
                        fma2(p0, p1, __uint_as_float(y[0]), __uint_as_float(y[1]), a.scale_log2, ref, ref);
                        p0 = exp2_sfu(p0);
                        p1 = exp2_sfu(p1);
                        if (!whole) {
                            p0 = c < seen ? p0 : 0.f;
                            p1 = c + 1 < seen ? p1 : 0.f;
                        }
                        add2(part[0], part[1], part[0], part[1], p0, p1);
                        const uint32_t w = pack_bf16x2(p0, p1);
                        add2(l0, l1, p0, p1, -__uint_as_float(w << 16), -__uint_as_float(w & 0xffff0000u));
                        out[8 * g + c / 2] = w;
                        out[16 + 8 * g + c / 2] = pack_bf16x2(l0, l1);
                    }
                }
                tmem_st32(s_tm + 32 * u, out);
            }
            sum += part[0] + part[1];
            tmem_wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_P_FULL + par));
        }
        // the row's sums and references, of both parities
        s_sum[(2 * par + half) * kTcRows + r] = sum;
        if (half == 0) s_sum[(4 + par) * kTcRows + r] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_SUM + (warp & 3)));
        wait_all(bar(C::B_SUM + (warp & 3)), 0);
        const float z0 = s_sum[r] + s_sum[kTcRows + r], z1 = s_sum[2 * kTcRows + r] + s_sum[3 * kTcRows + r];
        const float m0 = s_sum[4 * kTcRows + r], m1 = s_sum[5 * kTcRows + r], top = fmaxf(m0, m1);
        float f0 = share(m0, z0, top), f1 = share(m1, z1, top);
        const float z = f0 * z0 + f1 * z1;
        wait_all(bar(C::B_DRAIN), 0);
        tc_after();
        const bool lost = *s_abort != 0;
        f0 = lost ? NAN : z == 0.f ? 0.f : f0 / z;
        f1 = z == 0.f ? 0.f : f1 / z;
        const int64_t row = r < cols ? q_row(r) : 0;
        if (par == 0 && half == 0 && r < cols && a.lse)
            a.lse[row] = lost ? NAN : z == 0.f ? -INFINITY : (top + log2f(z)) * 0.69314718055994531f;
        bad = !isfinite(z) || (fabsf(m0) > kLargestScore && m0 > -INFINITY) ||
              (fabsf(m1) > kLargestScore && m1 > -INFINITY);
        for (int c = 32 * par; c < D / 2; c += 64) {
            uint32_t y0[32] = {}, y1[32] = {};
            if (steps > 0) tmem_ld32(o_half + c, y0);
            if (steps > 1) tmem_ld32(o_half + D + c, y1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint4 v;
                uint32_t *o = &v.x;
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float u0 = f0 * __uint_as_float(y0[e + j]) + f1 * __uint_as_float(y1[e + j]);
                    const float u1 = f0 * __uint_as_float(y0[e + j + 1]) + f1 * __uint_as_float(y1[e + j + 1]);
                    bad |= !isfinite(u0) || !isfinite(u1);
                    o[j / 2] = pack_bf16x2(u0, u1);
                }
                if (r < cols) *reinterpret_cast<uint4 *>(a.out + row * D + half * (D / 2) + c + e) = v;
            }
            __syncwarp();
        }
        bad = bad && !lost && r < cols;
    } else if (warp < 18) {
        // ------------------------------------------------------------ K, V
        const bool is_v = warp == 17;
        const __nv_bfloat16 *from = is_v ? a.v : a.k;
        const CUtensorMap *map = is_v ? &vmap : &kmap;
        if (lane == 0) asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
        const uint32_t to = is_v ? v_smem : k_smem;
        const int full = is_v ? C::B_V_FULL : C::B_K_FULL, empty = is_v ? C::B_PV_DONE : C::B_S_FULL;
        // token RPI i + lane / CH of a group, chunk lane % CH, i = 0, 1, ...
        constexpr int RPI = 32 / C::CH;
        const int tok = lane / C::CH, c = lane % C::CH;
        const uint32_t slab = (uint32_t)(c >> 3) * C::SLAB;
        GroupWalk w{s_map, s_list, table, groups, sub_log2, 0, 0};
        w.peek(lane);
        // a box of box_rows rows (1, 2, 4 or 8 groups) and 64 columns: this lane's
        const int per = box_rows >> 4, box_at = lane / C::SLABS * per, my_slab = lane % C::SLABS;
        Group x;
        int at = 0, valid = 0;               // group 32 (i / 4) + lane
        int i = 0;
        for (; i < steps; ++i) {
            const int st = i & 1, g0 = kTcGroups * (i & 3), count = min(kTcGroups, groups - kTcGroups * i);
            if (g0 == 0) w.take(a, kTcGroups * i + lane, head, pos0, x, at, valid);
            if (!is_v && (lane & ~(kTcGroups - 1)) == g0) s_group[i % kTcSlots * kTcGroups + lane % kTcGroups] = x;
            // the step's groups with all their tokens, as bits; boxes of such groups
            uint32_t boxed = __ballot_sync(0xffffffffu, valid == 16) >> g0 & 255;
            const int box = __shfl_sync(0xffffffffu, at, g0 + box_at % kTcGroups);
            if (per > 1) boxed &= boxed >> 1 & 0x55, boxed |= boxed << 1;
            if (per > 2) boxed &= boxed >> 2 & 0x33, boxed |= boxed << 2;
            if (per > 4) boxed = boxed == 255 ? 255 : 0;
            __syncwarp();
            if (!is_v && lane == 0) mbar_arrive(bar(C::B_G_FULL + i % kTcSlots));
            if (!wait_all(bar(empty + st), (i >> 1 & 1) ^ 1)) break;
            const uint32_t fb = bar(full + st);
            if (lane == 0) mbar_expect_tx(fb, (uint32_t)(__popc(boxed) * C::SLABS * 16 * 128));
            __syncwarp();
            if (box_at < kTcGroups && boxed >> box_at & 1)
                tma_load_2d(to + st * C::OPER + my_slab * C::SLAB + box_at * 16 * 128, map, my_slab * 64, box, fb);
            __syncwarp();
            for (int g = 0; boxed != 255 && g < count; ++g) {
                const int g_at = __shfl_sync(0xffffffffu, at, g0 + g), n = __shfl_sync(0xffffffffu, valid, g0 + g);
                if (boxed >> g & 1) continue;
                const __nv_bfloat16 *src = from + (int64_t)g_at * D + 8 * lane;
                const uint32_t dst = to + st * C::OPER + slab + (16 * g + tok) * 128;
#pragma unroll
                for (int e = 0; e < 16 / RPI; ++e) {
                    const int t = tok + RPI * e;         // (16 g does not change it mod 8)
                    cp_async16(dst + RPI * e * 128 + (((c & 7) ^ (t & 7)) << 4), t < n ? src + 32 * 8 * e : from,
                               t < n ? 16 : 0);
                }
            }
            cp_async_arrive(fb);
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        if (lane == 0)
            for (int x = max(i - 2, 0); x < i; ++x) settle(bar(full + (x & 1)), x >> 1 & 1);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ MMA
        // the whole warp, converged; one elected lane issues
        constexpr uint32_t IDESC_PV = idesc_bf16(kTcRows, D, true);
        const bool lead = elect_one();
        const int odd = uniform(warp - 18), all = uniform(groups);
        const uint32_t s_tm = uniform(tmem) + odd * kTcStep, o_tm = uniform(tmem) + 2 * kTcStep + odd * D;
        const uint64_t qd = sdesc(uniform(q_smem), 16, 1024), kd = sdesc(uniform(k_smem) + odd * C::OPER, 16, 1024),
                       vd = sdesc(uniform(v_smem) + odd * C::OPER, C::SLAB, 1024);
        auto score = [&](int i) {
            const uint32_t idesc = idesc_bf16(kTcRows, 16 * min(kTcGroups, all - kTcGroups * i), false);
            if (lead) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_ss(s_tm, qd + (((k >> 2) * C::Q_SLAB + (k & 3) * 32) >> 4),
                            kd + (((k >> 2) * C::SLAB + (k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
                umma_commit(bar(C::B_S_FULL + odd));
            }
        };
        // (copies by cp.async came through the generic proxy)
        bool ok = odd < steps && wait_all(bar(C::B_K_FULL + odd), 0);
        if (ok) {
            fence_async_smem();
            tc_after();
            score(odd);
        }
        for (int i = odd; ok && i < steps; i += 2) {
            const uint32_t phase = i >> 1 & 1;
            // what the step needs besides P first
            ok = wait_all(bar(C::B_V_FULL + odd), phase) &&
                 (i + 2 >= steps || wait_all(bar(C::B_K_FULL + odd), phase ^ 1));
            fence_async_smem();
            ok = ok && wait_all(bar(C::B_P_FULL + odd), phase);
            if (!ok) break;
            tc_after();
            // the weights' roundings and the rest of 16 tokens
            auto product = [&](int k, int rest) {
                umma_ts(o_tm, s_tm + 32 * (k >> 1) + 16 * rest + 8 * (k & 1), vd + k * (2048 >> 4), IDESC_PV,
                        i > 1 || k > 0 || rest ? 1u : 0u);
            };
            const int count = min(kTcGroups, all - kTcGroups * i);
            if (lead) {
                if (count == kTcGroups) {
#pragma unroll
                    for (int k = 0; k < kTcGroups; ++k) {
                        product(k, 0);
                        product(k, 1);
                    }
                } else {
                    for (int k = 0; k < count; ++k) {
                        product(k, 0);
                        product(k, 1);
                    }
                }
                umma_commit(bar(C::B_PV_DONE + odd));
            }
            if (i + 2 < steps) score(i + 2);
        }
        // every product has ended before the CTA does
        if (lead) umma_commit(bar(C::B_DRAIN));
        settle(bar(C::B_DRAIN), 0);
        __syncwarp();
    }
    // (what was written is written again)
    if (__syncthreads_or(bad) || again)
        for (int c = warp; c < cols; c += WARPS)
            slow_row<D>(a, q_row(c), pos0 + c / a.G, table, sel + c / a.G * sel_row, head, lane);
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 18)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTcCols) : "memory");
}

template <int D>
cudaError_t launch_tc(const SparseArgs &a, cudaStream_t stream) {
    static std::once_flag once[kMaxDevices];
    static bool ok[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        ok[dev] = cudaFuncSetAttribute(sparse_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       TcCfg<D>::SMEM) == cudaSuccess;
    });
    if (!ok[dev]) return cudaErrorInvalidDevice;
    alignas(64) CUtensorMap kmap, vmap;
    const int64_t rows = (int64_t)a.L * a.NB * a.Hkv << a.bs_log2;
    const int box = std::min(1 << a.bs_log2, kTcStep);
    if (!make_pool_map(&kmap, a.k, D, rows, box) || !make_pool_map(&vmap, a.v, D, rows, box)) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)QueryRows::tiles(a.rows.T, a.rows.S, a.qt), (unsigned)(a.L * a.Hkv));
    return launch_behind(sparse_tc_kernel<D>, grid, kTcThreads, TcCfg<D>::SMEM, 1, stream, kmap, vmap, a, box);
}

}  // namespace
}  // namespace kvp
