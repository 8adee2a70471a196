// Attention over the 4-bit cache for sequences with more than 16 query rows to
// a KV head (windows of several rows, prompts), on tcgen05: a tile of 128 * NT
// query rows, and of every 64-key block one widened copy of K and V in shared
// memory that all of the tile's rows share.
//
//   S_t = Q_t K^T   M = 128 rows, N = 64 keys, K = 128 dims  (A = Q_t in TMEM, B = K)
//   O_t += P_t V    M = 128 rows, N = 128 dims, K = 64 keys  (A = P_t in TMEM, B = V)
// Operands are fp16: a code times its scale is exact in it, Q is scaled per row
// by a power of two and P is relative to a lazily raised maximum, as in kv4.cu.
// Q in TMEM rather than in shared memory: with N = 64 an A operand from shared
// memory would ask for more than its bandwidth beside the widening's traffic.
//
// Persistent CTAs (NT = 1: two to an SM, 256 TMEM columns each; NT = 2: one, 512
// columns), one tile's softmax running while the other tile's (or CTA's)
// products do.  Warps:
//   4 NT  softmax: thread i of tile t owns query row 128 t + i (a TMEM lane):
//         writes Q, turns S into P in place, rescales O when its maximum grows
//         by more than 2^8, and at an item's end reads O out,
//   4     widen: warp w takes page w of every block from the ring of raw pages
//         to the fp16 K and V blocks (128-byte swizzle; V dims contiguous,
//         used as an MN-major operand),
//   1     a thread issues the MMAs (and the warp allocates TMEM),
//   1     bulk copies of the raw pages.
// Bounds at a 32-row window of 7 heads a KV head: matrix pipe 1024 cycles a
// 64-key block and tile pair, exp2 unit the same, widening and softmax issue
// slots about 850.  All waits are bounded; a timeout sets the device error word.
#include <algorithm>

#include "kv4.cuh"

namespace wedlm {
namespace {

using namespace kv4;

constexpr int KBLK = 64;                      // keys of a block
constexpr int PPB = KBLK / kPage;             // pages of a block
constexpr int RAW_BYTES = PPB * kHeadPage;    // a block's raw pages
constexpr int HALF_BYTES = KBLK * 128;        // 64 keys x 64 dims of fp16
constexpr int BLK_BYTES = 2 * HALF_BYTES;     // a widened K or V block
constexpr int FLAGS = 16;                     // ring of per-block flags (more than any run-ahead)

template <int NT>
struct Cfg {
    static constexpr int CTAS_PER_SM = NT == 1 ? 2 : 1;
    static constexpr int NRAW = NT == 1 ? 3 : 6;  // raw blocks in flight
    static constexpr int NKV = NT == 1 ? 2 : 3;   // widened K and V blocks
    static constexpr int WARP_WIDEN = 4 * NT, WARP_MMA = WARP_WIDEN + 4, WARP_LOAD = WARP_MMA + 1;
    static constexpr int THREADS = 32 * (WARP_LOAD + 1);
    static constexpr uint32_t TM_COLS = NT == 1 ? 256 : 512;
    static constexpr uint32_t tm_s(int t) { return t * 64; }
    static constexpr uint32_t tm_q(int t) { return NT * 64 + t * 64; }
    static constexpr uint32_t tm_o(int t) { return NT * 128 + t * 128; }
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + NKV * BLK_BYTES;
    static constexpr int OFF_RAW = OFF_V + NKV * BLK_BYTES;
    static constexpr int OFF_ITEMS = OFF_RAW + NRAW * RAW_BYTES;
    static constexpr int OFF_BAR = OFF_ITEMS + (int)sizeof(ItemTable);
    static constexpr int NBARS = 2 * NRAW + 4 * NKV + 4 * NT + 1;
    static constexpr int OFF_FLAGS = OFF_BAR + NBARS * 8;
    static constexpr int SMEM = OFF_FLAGS + FLAGS * 4 + 16 + 1024 /* alignment */;
    static_assert(CTAS_PER_SM * (SMEM + 1024) <= 228 * 1024, "shared memory");
    static_assert(NRAW + NKV + 2 < FLAGS, "flag ring");
    static_assert(TM_COLS >= (uint32_t)(NT * 256), "TMEM");
};

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// K-major tile with the 128-byte swizzle (128-byte rows, 8-row atoms 1024 B apart).
__device__ __forceinline__ uint64_t sdesc(uint32_t addr) {
    uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// MN-major tile with the 128-byte swizzle: 128-byte rows along K (one key
// each, 64 dims), 8-row atoms 1024 B apart, the next 64 dims HALF_BYTES on.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t addr) {
    uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(HALF_BYTES >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// fp16 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The whole warp waits; false for all of it if a lane gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(bar), parity, err));
}

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::THREADS, Cfg<NT>::CTAS_PER_SM) attn_kv4_tc_kernel(const AttnKv4Params p) {
    using C = Cfg<NT>;
    constexpr int NRAW = C::NRAW, NKV = C::NKV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = smem + C::OFF_K;
    uint8_t* sV = smem + C::OFF_V;
    uint8_t* raw = smem + C::OFF_RAW;
    ItemTable& items = *reinterpret_cast<ItemTable*>(smem + C::OFF_ITEMS);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [NRAW] a block's pages are there
    uint64_t* raw_empty = raw_full + NRAW;                                // [NRAW] widened (4 warps)
    uint64_t* k_full = raw_empty + NRAW;                                  // [NKV] K block widened (4 warps)
    uint64_t* k_empty = k_full + NKV;                                     // [NKV] its products done
    uint64_t* v_full = k_empty + NKV;
    uint64_t* v_empty = v_full + NKV;
    uint64_t* q_full = v_empty + NKV;  // [NT] an item's Q is in TMEM (4 warps)
    uint64_t* s_full = q_full + NT;    // [NT] S of a block done
    uint64_t* p_full = s_full + NT;    // [NT] P written (4 warps)
    uint64_t* pv_done = p_full + NT;   // [NT] P V of a block done: S / P free, O settled
    uint64_t* drain = pv_done + NT;
    volatile int* flags = reinterpret_cast<volatile int*>(smem + C::OFF_FLAGS);  // bit x: page x of the block is not there
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAGS + FLAGS * 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NRAW; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], 4);
        }
        for (int s = 0; s < NKV; ++s) {
            mbar_init(&k_full[s], 4);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_full[s], 4);
            mbar_init(&v_empty[s], 1);
        }
        for (int t = 0; t < NT; ++t) {
            mbar_init(&q_full[t], 4);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&pv_done[t], 1);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == C::WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(C::TM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    items_build(p, items);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch();
    const uint32_t tmem = *tmem_slot;
    int* err = p.err;
    const int g = p.hq / p.hkv;
    const int workers = gridDim.x;
    ItemIter it;
    it.next = blockIdx.x;
    Item item;

    if (warp == C::WARP_LOAD) {
        // ----------------------------------------------------------- loader
        // Lane l holds the ids of pages l, l + 32, ... of the item, 32 at a time.
        uint32_t gb = 0;
        bool ok = true;
        while (ok && item_next(it, p, items, workers, item)) {
            const int32_t* table = p.table + (int64_t)item.b * p.pages_per_seq;
            const int page0 = item.ks / kPage, npages = (item.ke + kPage - 1) / kPage - page0;
            const int nblk = (npages + PPB - 1) / PPB;
            int ids = -1;
            for (int j = 0; j < nblk; ++j, ++gb) {
                const int k0 = j * PPB;
                if ((k0 & 31) == 0) {
                    const int idx = page0 + k0 + lane;
                    ids = k0 + lane < npages && idx < p.pages_per_seq ? __ldcg(table + idx) : -1;
                }
                const int page = __shfl_sync(0xffffffffu, ids, (k0 + (lane & (PPB - 1))) & 31);
                const bool wanted = k0 + (lane & (PPB - 1)) < npages;
                const bool there = wanted && page >= 0 && page < p.num_pages;
                const uint32_t have = __ballot_sync(0xffffffffu, there && lane < PPB);
                if (wanted && !there) set_error(err, kErrBounds);
                const int s = gb % NRAW;
                if (!(ok = warp_wait(&raw_empty[s], ((gb / NRAW) & 1) ^ 1, err))) break;
                if (lane == 0) {
                    flags[gb % FLAGS] = (int)(~have & ((1u << PPB) - 1));
                    bar_expect(&raw_full[s], __popc(have) * kHeadPage);
                }
                __syncwarp();
                if (there && lane < PPB)
                    load_page(raw + s * RAW_BYTES + lane * kHeadPage,
                              p.pool + ((int64_t)page * p.hkv + item.h) * kHeadPage, &raw_full[s]);
            }
        }
        // copies still in flight (only after an error) land before the CTA exits
        if (lane == 0)
            for (uint32_t j = gb > (uint32_t)NRAW ? gb - NRAW : 0u; j < gb; ++j)
                mbar_wait_bounded(smem_u32(&raw_full[j % NRAW]), (j / NRAW) & 1, nullptr, 200000000LL);
    } else if (warp >= C::WARP_WIDEN && warp < C::WARP_MMA) {
        // ------------------------------------------------------------ widen
        // Lane: 16-dim block `blk` of tokens 4 i + tok0 of the warp's page.
        const int w = warp - C::WARP_WIDEN, blk = lane & 7, tok0 = lane >> 3;
        const int half = (blk >> 2) * HALF_BYTES;
        // a block's two 16-byte chunks; lanes of the upper dims write theirs in the
        // other order, so that eight lanes never meet in a bank
        const int ch0 = (blk & 3) * 2 + (blk >> 2), ch1 = ch0 ^ 1;
        uint32_t gb = 0;
        bool ok = true;
        while (ok && item_next(it, p, items, workers, item)) {
            const int page0 = item.ks / kPage, npages = (item.ke + kPage - 1) / kPage - page0;
            const int nblk = (npages + PPB - 1) / PPB;
            for (int j = 0; j < nblk; ++j, ++gb) {
                const int s = gb % NRAW, d = gb % NKV;
                if (!(ok = warp_wait(&raw_full[s], (gb / NRAW) & 1, err))) break;
                const uint8_t* src = raw + s * RAW_BYTES + w * kHeadPage;
                const int key0 = item.ks + j * KBLK + w * kPage;
                // keys behind the last row's, or of a page that is not there, add nothing
                const int live = (flags[gb % FLAGS] >> w) & 1 ? 0 : item.ke - key0;
                uint2 code[4];
                uint32_t scale[4];
                auto fetch = [&](const uint8_t* half_page) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = 4 * i + tok0;
                        code[i] = *reinterpret_cast<const uint2*>(half_page + tok * 64 + blk * 8);
                        scale[i] = half_page[kCodes + tok * 8 + blk];
                    }
                };
                auto widen = [&](uint8_t* dst) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = w * kPage + 4 * i + tok0;
                        const uint32_t sc = e4m3x2_to_f16x2(scale[i] * 0x101u);
                        uint32_t f[8];
                        e2m1x8_to_f16x2(code[i].x, *reinterpret_cast<uint32_t(*)[4]>(&f[0]));
                        e2m1x8_to_f16x2(code[i].y, *reinterpret_cast<uint32_t(*)[4]>(&f[4]));
#pragma unroll
                        for (int x = 0; x < 8; ++x) f[x] = hmul2(f[x], sc);
                        uint8_t* row = dst + half + r * 128;
                        const bool up = blk >> 2;
                        *reinterpret_cast<uint4*>(row + ((ch0 ^ (r & 7)) << 4)) =
                            make_uint4(up ? f[4] : f[0], up ? f[5] : f[1], up ? f[6] : f[2], up ? f[7] : f[3]);
                        *reinterpret_cast<uint4*>(row + ((ch1 ^ (r & 7)) << 4)) =
                            make_uint4(up ? f[0] : f[4], up ? f[1] : f[5], up ? f[2] : f[6], up ? f[3] : f[7]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                };
                fetch(src);
                if (!(ok = warp_wait(&k_empty[d], ((gb / NKV) & 1) ^ 1, err))) break;
                widen(sK + d * BLK_BYTES);
                if (lane == 0) bar_arrive(&k_full[d]);
                fetch(src + kHalfPage);
                if (live < kPage) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * i + tok0 >= live) scale[i] = 0;
                }
                __syncwarp();
                if (lane == 0) bar_arrive(&raw_empty[s]);
                if (!(ok = warp_wait(&v_empty[d], ((gb / NKV) & 1) ^ 1, err))) break;
                widen(sV + d * BLK_BYTES);
                if (lane == 0) bar_arrive(&v_full[d]);
            }
        }
    } else if (warp == C::WARP_MMA) {
        // -------------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t idS = idesc_f16(128, KBLK);
            constexpr uint32_t idO = idesc_f16(128, HD) | (1u << 16);  // B (V) MN-major
            uint32_t gb = 0;
            int li = 0;
            bool ok = true;
            while (ok && item_next(it, p, items, workers, item)) {
                const int nblk = (item.ke - item.ks + KBLK - 1) / KBLK;
                for (int j = 0; j < nblk && ok; ++j, ++gb) {
                    const int d = gb % NKV;
                    const uint32_t kvpar = (gb / NKV) & 1;
                    if (!(ok = mbar_wait_bounded(smem_u32(&k_full[d]), kvpar, err))) break;
                    const uint32_t kb = smem_u32(sK + d * BLK_BYTES), vb = smem_u32(sV + d * BLK_BYTES);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        ok = ok && (j == 0 ? mbar_wait_bounded(smem_u32(&q_full[t]), li & 1, err)
                                           : mbar_wait_bounded(smem_u32(&pv_done[t]), (gb - 1) & 1, err));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            mma_ts(tmem + C::tm_s(t), tmem + C::tm_q(t) + kk * 8,
                                   sdesc(kb + (kk >> 2) * HALF_BYTES + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                        umma_commit(&s_full[t]);
                    }
                    if (!ok) break;
                    umma_commit(&k_empty[d]);
                    if (!(ok = mbar_wait_bounded(smem_u32(&v_full[d]), kvpar, err))) break;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (!(ok = ok && mbar_wait_bounded(smem_u32(&p_full[t]), gb & 1, err))) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < KBLK / 16; ++kk)
                            mma_ts(tmem + C::tm_o(t), tmem + C::tm_s(t) + kk * 8, sdesc_mn(vb + kk * 2048), idO,
                                   (j > 0 || kk > 0) ? 1u : 0u);
                        umma_commit(&pv_done[t]);
                    }
                    if (ok) umma_commit(&v_empty[d]);
                }
                ++li;
            }
            // every MMA issued has completed before TMEM may be released
            umma_commit(drain);
            mbar_wait_bounded(smem_u32(drain), 0, nullptr, 200000000LL);
        }
    } else {
        // ---------------------------------------------------------- softmax
        const int t = warp >> 2;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + C::tm_s(t), tQ = tmem + lane_base + C::tm_q(t),
                       tO = tmem + lane_base + C::tm_o(t);
        const int row = threadIdx.x;  // of the tile
        uint32_t gb = 0;
        bool ok = true;
        while (ok && item_next(it, p, items, workers, item)) {
            const int qr = item.q0 + row;
            const bool live = qr < item.rows;
            const int qc = min(qr, item.rows - 1);
            const int64_t at = ((int64_t)item.b * p.stride + qc / g) * p.hq + item.h * g + qc % g;
            // Q of the row to TMEM, scaled by a power of two
            int ex = 0;
            {
                uint32_t w[64];
                const uint4* q = reinterpret_cast<const uint4*>(p.q + at * HD);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const uint4 u = live ? __ldcg(q + x) : make_uint4(0, 0, 0, 0);
                    w[4 * x] = u.x;
                    w[4 * x + 1] = u.y;
                    w[4 * x + 2] = u.z;
                    w[4 * x + 3] = u.w;
                }
                uint32_t mx = 0;
#pragma unroll
                for (int x = 0; x < 64; ++x) mx = max(mx, max(w[x] & 0x7FFFu, (w[x] >> 16) & 0x7FFFu));
                ex = mx ? min(100, 14 + 127 - (int)(mx >> 7)) : 0;
                const float f = __int_as_float((ex + 127) << 23);
#pragma unroll
                for (int x = 0; x < 64; ++x)
                    w[x] = pack_half2(__uint_as_float(w[x] << 16) * f, __uint_as_float(w[x] & 0xFFFF0000u) * f);
                tmem_st32(tQ, &w[0]);
                tmem_st32(tQ + 32, &w[32]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&q_full[t]);
            }
            const float sl = 1.4426950408889634f / sqrtf((float)HD) * p.k_scale * __int_as_float((127 - ex) << 23);
            const int lim = min(item.S + qc / g, item.ke - 1);              // last key the row sees
            const int all = min(item.S + item.q0 / g, item.ke - 1);         // last key every row of the tile sees
            const int nblk = (item.ke - item.ks + KBLK - 1) / KBLK;
            float m = -INFINITY, z = 1e30f, l = 0.f;
            for (int j = 0; j < nblk; ++j, ++gb) {
                if (!(ok = warp_wait(&s_full[t], gb & 1, err))) break;
                tc_fence_after();
                const int key0 = item.ks + j * KBLK;
                float e[64];
                tmem_ld32(tS, reinterpret_cast<uint32_t*>(&e[0]));
                tmem_ld32(tS + 32, reinterpret_cast<uint32_t*>(&e[32]));
                const int gone = flags[gb % FLAGS];
                tmem_wait_ld();
                if (key0 + KBLK - 1 > all || gone) {
#pragma unroll
                    for (int x = 0; x < 64; ++x)
                        if (key0 + x > lim || ((gone >> (x / kPage)) & 1)) e[x] = -INFINITY;
                }
                float top = -INFINITY;
#pragma unroll
                for (int x = 0; x < 64; ++x) top = fmaxf(top, e[x]);
                const float v = top * sl;
                const bool grew = fmaf(top, sl, z) > kWeightLog2 + kLazyLog2;
                if (__any_sync(0xffffffffu, grew)) {
                    const float f = grew ? exp2_fast(m - v) : 1.f;
                    if (grew) {
                        m = v;
                        z = kWeightLog2 - v;
                        l *= f;
                    }
                    if (j > 0) {
#pragma unroll 1
                        for (int x = 0; x < HD; x += 32) {
                            uint32_t r[32];
                            tmem_ld32(tO + x, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 32; ++y) r[y] = __float_as_uint(__uint_as_float(r[y]) * f);
                            tmem_st32(tO + x, r);
                        }
                    }
                }
                uint32_t pk[32];
                float sum[4] = {};
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    const float a = exp2_fast(fmaf(e[2 * x], sl, z)), b = exp2_fast(fmaf(e[2 * x + 1], sl, z));
                    sum[x & 3] += a + b;
                    pk[x] = pack_half2(a, b);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st32(tS, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&p_full[t]);
            }
            if (!ok) break;
            // O of the item
            if (!(ok = warp_wait(&pv_done[t], (gb - 1) & 1, err))) break;
            tc_fence_after();
            const float f = out_factor(p.v_scale, l);
#pragma unroll 1
            for (int x = 0; x < HD; x += 32) {
                uint32_t r[32];
                tmem_ld32(tO + x, r);
                tmem_wait_ld();
                if (!live) continue;
                if (item.nsplit == 1) {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + at * HD + x);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 h2 =
                                __floats2bfloat162_rn(__uint_as_float(r[8 * y + 2 * k]) * f, __uint_as_float(r[8 * y + 2 * k + 1]) * f);
                            o[k] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        dst[y] = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(p.part_o + (at * p.max_splits + item.sp) * HD + x);
#pragma unroll
                    for (int y = 0; y < 8; ++y) dst[y] = make_uint4(r[4 * y], r[4 * y + 1], r[4 * y + 2], r[4 * y + 3]);
                }
            }
            if (live && item.nsplit > 1) p.part_ml[at * p.max_splits + item.sp] = make_float2(m, l);
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TM_COLS) : "memory");
    }
}

template <int NT>
cudaError_t launch(const AttnKv4Params& p, int num_sms, cudaStream_t st) {
    using C = Cfg<NT>;
    // (cheap, and needed once per device)
    cudaError_t e = cudaFuncSetAttribute(attn_kv4_tc_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)p.n_seq * p.hkv * p.tiles * p.max_splits;
    const int grid = (int)std::min<int64_t>(most, (int64_t)C::CTAS_PER_SM * num_sms);
    return launch_pdl(attn_kv4_tc_kernel<NT>, dim3(grid), dim3(C::THREADS), C::SMEM, st, p);
}

}  // namespace

namespace kv4 {

cudaError_t launch_attn_kv4_tc(const AttnKv4Params& p, int num_sms, cudaStream_t st) {
    return p.tile_rows <= 128 ? launch<1>(p, num_sms, st) : launch<2>(p, num_sms, st);
}

}  // namespace kv4
}  // namespace wedlm
