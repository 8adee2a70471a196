// Attention over the 4-bit cache for sequences with more than 16 query rows to
// a KV head (windows of several rows, prompts), on tcgen05: of every 128-key
// block one widened copy of K and V in shared memory, fp16, and two products
//   S_t = Q_t K^T   M = 128 rows, N = 128 keys, K = 128 dims  (A = Q_t, B = K: shared memory)
//   O_t += P_t V    M = 128 rows, N = 128 dims, K = 128 keys  (A = P_t in TMEM over S_t, B = V)
// for the CTA's two tiles t.  ROWS: the tiles are the two halves of 256 query
// rows and every block serves both.  Otherwise (at most 128 query rows) the
// tiles hold the same rows and take the blocks in turn, each with its own
// maximum, sum and O, joined at the item's end; with at most 64 rows they are
// repeated on lanes 64 .. 127, which weigh the second half of a block's keys as
// the lower lanes do the first, so that all warps share the softmax.  Operands are fp16: a code
// times its scale is exact in it, Q is scaled per row by a power of two and P is
// relative to a lazily raised maximum, as in kv4.cu.
//
// Why these shapes (measured, cycles): an MMA of N = 32 or 64 takes 45 whatever
// its A operand, of N = 128 65, the full rate; a commit is seen by a waiting
// thread after 220, so few and large steps.  Two tiles, because one's softmax
// (at least 1024 cycles of the exp2 unit a block) then runs under the other's
// products (1040).  A block and tile pair costs the tensor pipe 2080 cycles
// (ROWS), the shared memory's bandwidth about 2300, and takes 4300: a tile's
// chain of S (810 until a softmax warp sees it), softmax (2580) and P V (890 until
// the next S may start, which overwrites P) is what bounds it.  With the softmax
// left out it took 3500, with the widening's stores left out too 3400 (the MMA
// thread's own chain of products and commits); 16 softmax warps, which share the
// same schedulers, were no faster, an MMA thread for each tile slower (456 us:
// products of both tiles alternate in the pipe).
//   64 sequences at 8.2k to 8.7k, windows of 32, 7 heads to a KV head: 323 us,
//   600 TFLOP/s (mma.sync items of 16 rows: 1180); 16 sequences of 128 to 2047,
//   windows of 16, 4 heads: 31 us (51), of which the start takes 5 and the end 3;
//   16 prompts of 512 rows 99 us, 64 of 1024 1.04 ms (32 and 8 heads).
//
// Persistent, one CTA to an SM.  Warps:
//   8  softmax: thread i of tile t owns lane i of TMEM, a query row: Q to shared
//      memory, S to P in place, O rescaled when its maximum grows by more than
//      2^8, O read out at an item's end,
//   8  widen: warp w takes page w of every block from the ring of raw pages to
//      the fp16 blocks (128-byte swizzle; V dims contiguous, used as an MN-major
//      operand),
//   1  a thread issues the MMAs (and the warp allocates TMEM),
//   1  bulk copies of the raw pages.
// All waits are bounded; a timeout sets the device error word.
#include <algorithm>
#include <type_traits>

#include "kv4.cuh"

namespace wedlm {
namespace {

using namespace kv4;

constexpr int KBLK = 128;                     // keys of a block
constexpr int PPB = KBLK / kPage;             // pages of a block
constexpr int RPP = 4;                        // pages of a raw stage (half a block)
constexpr int RAW_BYTES = RPP * kHeadPage;
constexpr int HALF_BYTES = KBLK * 128;        // 128 keys (or rows) x 64 dims of fp16
constexpr int BUF_BYTES = 2 * HALF_BYTES;     // a widened K or V block, or a tile's Q
constexpr int NRAW = 3;                       // raw stages: half block r lies in stage r % NRAW
// Its barriers are numbers r % NRAWBAR.  An even number, so that a barrier belongs to
// either the lower or the upper halves of blocks and the four warps that wait on it see
// every one of its phases: with one to a stage they would see every other one, and a
// parity cannot tell a phase from the one before last.
constexpr int NRAWBAR = 4;
constexpr int NBUF = 4;                       // widened K, V, K, V blocks
constexpr int FLAGS = 8;                      // ring of per-block flags (more than any run-ahead)
constexpr int NITEM = 4;                      // ring of items
constexpr int WARP_WIDEN = 8, WARP_MMA = 16, WARP_LOAD = 17;
constexpr int THREADS = 20 * 32;               // (two warps idle: register shares go by groups of four)
// Registers a thread: launched with 96, then shared out by what the roles need.
constexpr int REGS_SOFTMAX = 144, REGS_WIDEN = 56, REGS_REST = 80;
static_assert(8 * REGS_SOFTMAX + 8 * REGS_WIDEN + 4 * REGS_REST <= 20 * 96, "more registers than the block was launched with");
constexpr uint32_t TM_COLS = 512;             // S_t at 128 t, O_t at 256 + 128 t
constexpr int OFF_BUF = 0;
constexpr int OFF_Q = OFF_BUF + NBUF * BUF_BYTES;  // ROWS: a Q per tile; else one Q and the exchange of the parts' O
constexpr int OFF_RAW = OFF_Q + 2 * BUF_BYTES;
constexpr int OFF_ITEMS = OFF_RAW + NRAW * RAW_BYTES;
constexpr int OFF_ML = OFF_ITEMS + (int)sizeof(ItemTable);  // !ROWS: every softmax thread's (m, l)
constexpr int OFF_EX = OFF_ML + 256 * 8;                    // !ROWS: the exponents added to Q's rows
constexpr int OFF_BAR = OFF_EX + 128 * 4;
constexpr int NBARS = 2 * NRAWBAR + 2 * NBUF + 2 * NITEM + 8 + 1;
constexpr int OFF_FLAGS = OFF_BAR + NBARS * 8;
constexpr int OFF_RING = OFF_FLAGS + FLAGS * 4;
constexpr int SMEM = OFF_RING + NITEM * (int)sizeof(Item) + 16 + 1024 /* alignment */;
static_assert(SMEM <= 227 * 1024, "shared memory");
static_assert(NRAW / 2 + 4 < FLAGS, "flag ring");
static_assert(NRAWBAR % 2 == 0 && NRAWBAR > NRAW, "raw barriers");
static_assert(sizeof(ItemTable) % 8 == 0, "alignment of what follows");

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
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Waits for the loads issued so far; r: registers that one of them fills (tied, so
// that no use of them moves ahead of the wait).
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]) : : "memory");
    asm volatile("" : "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// mbar_wait_bounded without its long suspension: these waits are short and on
// the critical path (a woken thread went on 300 cycles sooner).
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity, int* err) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(a, parity)) return true;
        if ((it & 255u) == 0) {
            if (stalled(err)) return false;
            if (clock64() - t0 > 2000000000LL) {
                set_error(err, kErrTimeout);
                return false;
            }
        }
    }
}
// The whole warp waits; false for all of it if a lane gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
    return __all_sync(0xffffffffu, wait_short(bar, parity, err));
}

// 32 dims from c on of a row's O: the output (times f), or the chunk's partial.
__device__ __forceinline__ void store_row(const AttnKv4Params& p, int nsplit, int sp, int64_t at, int c, uint32_t (&r)[32],
                                          float f) {
    if (nsplit == 1) {
#pragma unroll
        for (int y = 0; y < 16; ++y) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[2 * y]) * f, __uint_as_float(r[2 * y + 1]) * f);
            r[y] = *reinterpret_cast<const uint32_t*>(&h);
        }
        st_global8(p.out + at * HD + c, r);
        st_global8(p.out + at * HD + c + 16, r + 8);
    } else {
        float* dst = p.part_o + (at * p.max_splits + sp) * HD + c;
#pragma unroll
        for (int y = 0; y < 32; y += 8) st_global8(dst + y, r + y);
    }
}

// 8 dims from c on.
__device__ __forceinline__ void store8(const AttnKv4Params& p, int nsplit, int sp, int64_t at, int c, const float (&v)[8],
                                       float f) {
    uint32_t r[8];
    if (nsplit == 1) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * y] * f, v[2 * y + 1] * f);
            r[y] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p.out + at * HD + c) = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
#pragma unroll
        for (int y = 0; y < 8; ++y) r[y] = __float_as_uint(v[y]);
        st_global8(p.part_o + (at * p.max_splits + sp) * HD + c, r);
    }
}

// Barrier among the 256 softmax threads, returning whether `v` holds in all of
// them: steps that synchronise the tiles are entered by all or by none, also
// when a bounded wait gave up in one warp only.
__device__ __forceinline__ bool softmax_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"((uint32_t)v) : "memory");
    return r != 0;
}

template <bool ROWS>
__global__ void __launch_bounds__(THREADS, 1) attn_kv4_tc_kernel(const AttnKv4Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset: the compiler still knows that it is shared memory)
    uint8_t* bufs = smem + OFF_BUF;
    uint8_t* sQ = smem + OFF_Q;
    float* xch = reinterpret_cast<float*>(smem + OFF_Q + BUF_BYTES);  // !ROWS: 32 dims x 256 threads
    uint8_t* raw = smem + OFF_RAW;
    ItemTable& items = *reinterpret_cast<ItemTable*>(smem + OFF_ITEMS);
    float2* s_ml = reinterpret_cast<float2*>(smem + OFF_ML);
    int* s_ex = reinterpret_cast<int*>(smem + OFF_EX);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);  // [NRAWBAR] half a block's pages are there
    uint64_t* raw_empty = raw_full + NRAWBAR;                          // [NRAWBAR] read (a warp a page)
    uint64_t* buf_full = raw_empty + NRAWBAR;                          // [NBUF] K or V widened (8 warps)
    uint64_t* buf_empty = buf_full + NBUF;                             // [NBUF] its products done (of both tiles that it serves)
    uint64_t* q_full = buf_empty + NBUF;                               // [2] an item's Q is there (4 warps)
    uint64_t* s_full = q_full + 2;                                     // [2] S of a tile's block done
    uint64_t* p_full = s_full + 2;                                     // [2] P written (4 warps)
    uint64_t* pv_done = p_full + 2;                                    // [2] P V done: S / P free, O settled
    uint64_t* item_full = pv_done + 2;                                 // [NITEM] an item is in the ring
    uint64_t* item_empty = item_full + NITEM;                          // [NITEM] every role is past it
    uint64_t* drain = item_empty + NITEM;
    volatile int* flags = reinterpret_cast<volatile int*>(smem + OFF_FLAGS);  // bit x: page x of the block is not there
    // The CTA's items in order, an item with ke <= ks ending them
    volatile Item* ring = reinterpret_cast<volatile Item*>(smem + OFF_RING);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_RING + NITEM * sizeof(Item));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NRAWBAR; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], RPP);
        }
        for (int s = 0; s < NBUF; ++s) {
            mbar_init(&buf_full[s], PPB);
            mbar_init(&buf_empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 4);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&pv_done[t], 1);
        }
        for (int s = 0; s < NITEM; ++s) {
            mbar_init(&item_full[s], 1);
            mbar_init(&item_empty[s], 8 + PPB + 1);  // softmax and widening warps, the MMA thread
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TM_COLS) : "memory");
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
    auto blocks_of = [](const volatile Item& o) { return (o.ke - o.ks + KBLK - 1) / KBLK; };

    if (warp >= WARP_MMA) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
    if (warp == WARP_LOAD) {
        // ----------------------------------------------------------- loader
        // Lane l holds the ids of pages l, l + 32, ... of the item, 32 at a time;
        // lanes 0 .. 7 load the pages of a block.
        uint32_t gb = 0, gr = 0;
        bool ok = true;
        ItemIter it;
        it.next = blockIdx.x;
        Item item;
        for (uint32_t li = 0; ok; ++li) {
            const bool has = item_next(it, p, items, gridDim.x, item);
            if (!(ok = warp_wait(&item_empty[li % NITEM], ((li / NITEM) & 1) ^ 1, err))) break;
            if (lane == 0) {
                if (!has) item.ke = item.ks = 0;
                volatile Item& o = ring[li % NITEM];
                o.b = item.b;
                o.h = item.h;
                o.sp = item.sp;
                o.q0 = item.q0;
                o.S = item.S;
                o.rows = item.rows;
                o.ks = item.ks;
                o.ke = item.ke;
                o.nsplit = item.nsplit;
                bar_arrive(&item_full[li % NITEM]);
            }
            __syncwarp();
            if (!has) break;
            const int32_t* table = p.table + (int64_t)item.b * p.pages_per_seq;
            const int page0 = item.ks / kPage, npages = (item.ke - 1) / kPage + 1 - page0;
            const int nblk = blocks_of(item);
            int ids = -1;
            for (int j = 0; j < nblk && ok; ++j, ++gb) {
                const int k0 = j * PPB, mine = k0 + (lane & (PPB - 1));
                if ((k0 & 31) == 0) {
                    const int idx = page0 + k0 + lane;
                    ids = k0 + lane < npages && idx < p.pages_per_seq ? __ldcg(table + idx) : -1;
                }
                const int page = __shfl_sync(0xffffffffu, ids, mine & 31);
                const bool wanted = mine < npages, there = wanted && page >= 0 && page < p.num_pages;
                const uint32_t have = __ballot_sync(0xffffffffu, there && lane < PPB);
                if (wanted && !there) set_error(err, kErrBounds);
                if (lane == 0) flags[gb % FLAGS] = (int)(~have & ((1u << PPB) - 1));
#pragma unroll
                for (int x = 0; x < 2; ++x, ++gr) {  // two stages to a block
                    const int s = gr % NRAW;
                    uint64_t* full = &raw_full[gr % NRAWBAR];
                    const uint32_t old = gr - NRAW;  // the stage's last half block
                    if (gr >= NRAW && !(ok = warp_wait(&raw_empty[old % NRAWBAR], (old / NRAWBAR) & 1, err))) break;
                    const uint32_t part = (have >> (RPP * x)) & ((1u << RPP) - 1);
                    if (lane == 0) bar_expect(full, __popc(part) * kHeadPage);
                    __syncwarp();
                    if (there && lane < PPB && lane / RPP == x)
                        load_page(raw + s * RAW_BYTES + (lane % RPP) * kHeadPage,
                                  p.pool + ((int64_t)page * p.hkv + item.h) * kHeadPage, full);
                }
            }
        }
        // copies still in flight (only after an error) land before the CTA exits
        if (lane == 0)
            for (uint32_t j = gr > (uint32_t)NRAW ? gr - NRAW : 0u; j < gr; ++j)
                mbar_wait_bounded(smem_u32(&raw_full[j % NRAWBAR]), (j / NRAWBAR) & 1, nullptr, 200000000LL);
    } else if (warp == WARP_MMA) {
        // -------------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t idS = idesc_f16(128, KBLK);
            constexpr uint32_t idO = idesc_f16(128, HD) | (1u << 16);  // B (V) MN-major
            // The tiles in turn, P V of a block and then S of the tile's next one: while
            // one tile's products run, the other's softmax does.
            // (Rolled over the tiles and with descriptors that only add constants: this
            // thread's code competes with the other roles' for the instruction cache,
            // and a miss delays every product.)
            uint32_t base = 0;  // the CTA's number of the item's first block
            uint32_t xs = 0;    // bit t: parity of the tile's blocks so far
            bool ok = true;
            const uint64_t dq = sdesc(smem_u32(sQ)), dk = sdesc(smem_u32(bufs)), dv = sdesc_mn(smem_u32(bufs));
            constexpr uint64_t BUF16 = BUF_BYTES >> 4, HALF16 = HALF_BYTES >> 4;
            auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && wait_short(bar, parity, err); };
            // (A look at a barrier takes over a hundred cycles beside the widening's
            // stores: a widened block is waited for before what it waits for anyway, and
            // ROWS by tile 0 alone; tile 1, whose products come later, lets it go.)
            auto issue_s = [&](int t, uint32_t b, uint64_t* after, uint32_t after_parity) {
                const uint32_t kx = 2 * b;
                if ((!ROWS || t == 0) && !wait(&buf_full[kx % NBUF], (kx / NBUF) & 1)) return;
                if (!wait(after, after_parity)) return;
                tc_fence_after();
                const uint64_t q = dq + (ROWS ? t : 0) * BUF16, k = dk + (kx % NBUF) * BUF16;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    mma_ss(tmem + 128 * t, q + (kk >> 2) * HALF16 + (kk & 3) * 2, k + (kk >> 2) * HALF16 + (kk & 3) * 2, idS,
                           kk > 0 ? 1u : 0u);
                umma_commit(&s_full[t]);
                if (!ROWS || t == 1) umma_commit(&buf_empty[kx % NBUF]);
            };
            auto issue_pv = [&](int t, uint32_t b, bool first) {
                const uint32_t vx = 2 * b + 1;
                if ((!ROWS || t == 0) && !wait(&buf_full[vx % NBUF], (vx / NBUF) & 1)) return;
                if (!wait(&p_full[t], (xs >> t) & 1)) return;
                tc_fence_after();
                const uint64_t v = dv + (vx % NBUF) * BUF16;
#pragma unroll
                for (int kk = 0; kk < KBLK / 16; ++kk)
                    mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + (kk >> 1) * 32 + (kk & 1) * 8, v + kk * 128, idO,
                           (!first || kk > 0) ? 1u : 0u);
                umma_commit(&pv_done[t]);
                if (!ROWS || t == 1) umma_commit(&buf_empty[vx % NBUF]);
            };
            for (uint32_t li = 0; ok; ++li) {
                if (!wait(&item_full[li % NITEM], (li / NITEM) & 1)) break;
                const int nblk = blocks_of(ring[li % NITEM]);
                bar_arrive(&item_empty[li % NITEM]);
                if (nblk <= 0) break;
                constexpr int STEP = ROWS ? 1 : 2;  // from one block of a tile to its next
                // The tiles in turn: P V of a block (from the tile's second turn on), then S
                // of its next one.
#pragma unroll 1
                for (int j0 = -STEP; ok && j0 < nblk; j0 += STEP) {
#pragma unroll 1
                    for (int t = 0; t < 2 && ok; ++t) {
                        const int j = j0 + (ROWS ? 0 : t);
                        if (j0 < 0) {
                            if (j + STEP < nblk) issue_s(t, base + j + STEP, &q_full[ROWS ? t : 0], li & 1);
                            else if (!ROWS) wait(&q_full[0], li & 1);  // (every phase is looked at)
                        } else if (j < nblk) {
                            issue_pv(t, base + j, j0 == 0);
                            if (ok && j + STEP < nblk) issue_s(t, base + j + STEP, &pv_done[t], (xs >> t) & 1);
                            xs ^= 1u << t;
                        }
                    }
                }
                base += nblk;
            }
            // every MMA issued has completed before TMEM may be released
            umma_commit(drain);
            mbar_wait_bounded(smem_u32(drain), 0, nullptr, 200000000LL);
        }
    }
    } else if (warp >= WARP_WIDEN) {
        // ------------------------------------------------------------ widen
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_WIDEN));
        // Lane: 16-dim block `blk` of tokens 4 i + tok of the warp's page.  Lanes of
        // the upper dims take the token beside the others': the swizzle then sends
        // the eight lanes of a 16-byte store to eight different places.
        const int w = warp - WARP_WIDEN, blk = lane & 7, tok = (lane >> 3) ^ (blk >> 2);
        // place of the first of the block's two 16-byte chunks in token tok's row (the
        // second's differs in bit 4, those of token tok + 4 in bit 6)
        const uint32_t place = smem_u32(bufs) + (blk >> 2) * HALF_BYTES + (w * kPage + tok) * 128 + (((2 * (blk & 3)) ^ tok) << 4);
        uint32_t gb = 0;
        bool ok = true;
        for (uint32_t li = 0; ok; ++li) {
            if (!(ok = warp_wait(&item_full[li % NITEM], (li / NITEM) & 1, err))) break;
            const int ks = ring[li % NITEM].ks, ke = ring[li % NITEM].ke, nblk = (ke - ks + KBLK - 1) / KBLK;
            __syncwarp();
            if (lane == 0) bar_arrive(&item_empty[li % NITEM]);
            if (nblk <= 0) break;
            for (int j = 0; j < nblk && ok; ++j, ++gb) {
                // K and then V of the warp's page
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t x = 2 * gb + kv;
                    const uint32_t dst = place + (x % NBUF) * BUF_BYTES;
                    if (!(ok = warp_wait(&buf_empty[x % NBUF], ((x / NBUF) & 1) ^ 1, err))) break;
                    const uint32_t r = 2 * gb + w / RPP;
                    if (kv == 0 && !(ok = warp_wait(&raw_full[r % NRAWBAR], (r / NRAWBAR) & 1, err))) break;
                    const uint8_t* src = raw + (r % NRAW) * RAW_BYTES + (w % RPP) * kHeadPage + kv * kHalfPage;
                    uint2 code[4];
                    uint32_t scale[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        code[i] = *reinterpret_cast<const uint2*>(src + (4 * i + tok) * 64 + blk * 8);
                        scale[i] = src[kCodes + (4 * i + tok) * 8 + blk];
                    }
                    if (kv) {
                        // V of keys behind the last row's, or of a page that is not there, is zero
                        const int gone = flags[gb % FLAGS];
                        const int live = (gone >> w) & 1 ? 0 : ke - (ks + j * KBLK + w * kPage);
                        if (live < kPage) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (4 * i + tok >= live) scale[i] = 0;
                        }
                        __syncwarp();
                        if (lane == 0) bar_arrive(&raw_empty[r % NRAWBAR]);  // (K and V of the page have been read)
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t sc = e4m3x2_to_f16x2(scale[i] * 0x101u);
                        uint32_t lo[4], hi[4];
                        e2m1x8_to_f16x2(code[i].x, lo);
                        e2m1x8_to_f16x2(code[i].y, hi);
                        const uint32_t at = (i & 1 ? dst ^ 64u : dst) + 512 * i;
                        st_shared16(at, hmul2(lo[0], sc), hmul2(lo[1], sc), hmul2(lo[2], sc), hmul2(lo[3], sc));
                        st_shared16(at ^ 16u, hmul2(hi[0], sc), hmul2(hi[1], sc), hmul2(hi[2], sc), hmul2(hi[3], sc));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) bar_arrive(&buf_full[x % NBUF]);
                }
            }
        }
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        const int t = warp >> 2;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + 128 * t, tO = tmem + lane_base + 256 + 128 * t;
        const int lane_row = threadIdx.x & 127;
        uint32_t x = 0, base = 0;  // the tile's and the CTA's blocks so far
        bool ok = true;
        for (uint32_t li = 0;; ++li) {
            ok = warp_wait(&item_full[li % NITEM], (li / NITEM) & 1, err);
            if (!ROWS) ok = softmax_all(ok);  // (and Q and the exchange have been read)
            if (!ok) break;
            const volatile Item& item = ring[li % NITEM];
            const int nblk = blocks_of(item);
            if (nblk <= 0) break;
            const int tile_rows = min(item.rows - item.q0, ROWS ? 256 : 128);
            const bool twice = !ROWS && tile_rows <= 64;  // rows repeated on lanes 64 .. 127
            const int row = ROWS ? (int)threadIdx.x : twice ? lane_row & 63 : lane_row;
            const bool live = row < tile_rows;
            // the keys of a block this thread works on: with `twice` the lower lanes the first half
            const int cb = twice ? lane_row & 64 : 0, ce = twice ? cb + 64 : KBLK;
            const int qr = item.q0 + min(row, tile_rows - 1);
            const int64_t at = ((int64_t)item.b * p.stride + qr / g) * p.hq + item.h * g + qr % g;
            // Q by the tile that owns it: each thread brings its row to the row's place in
            // shared memory, finds its largest magnitude and scales it there.  (Rolled:
            // at a kernel's start every instruction comes from far away.)
            int ex;
            if (ROWS || t == 0) {
                uint8_t* dst = sQ + (ROWS ? t : 0) * BUF_BYTES + lane_row * 128;
                const uint8_t* src = reinterpret_cast<const uint8_t*>(p.q + at * HD);
                const uint32_t bytes = row < tile_rows ? 16 : 0;  // 0: zeros
#pragma unroll 4
                for (int y = 0; y < 16; ++y)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                                 ::"r"(smem_u32(dst + (y >> 3) * HALF_BYTES + (((y & 7) ^ (lane_row & 7)) << 4))),
                                 "l"(src + 16 * y), "r"(bytes) : "memory");
                asm volatile("cp.async.wait_all;" ::: "memory");
                // (chunks in an order that keeps eight threads in different banks)
                auto chunk = [&](int y) {
                    return reinterpret_cast<uint4*>(dst + (y >> 3) * HALF_BYTES + (((y & 7) ^ (lane_row & 7)) << 4));
                };
                uint32_t mx = 0;
#pragma unroll 4
                for (int y = 0; y < 16; ++y) {
                    const uint4 u = *chunk(y);
                    mx = max(mx, max(max(u.x & 0x7FFFu, (u.x >> 16) & 0x7FFFu), max(u.y & 0x7FFFu, (u.y >> 16) & 0x7FFFu)));
                    mx = max(mx, max(max(u.z & 0x7FFFu, (u.z >> 16) & 0x7FFFu), max(u.w & 0x7FFFu, (u.w >> 16) & 0x7FFFu)));
                }
                ex = min(100, 14 + 127 - (int)(mx >> 7));
                const float f = __int_as_float((ex + 127) << 23);
                auto scaled = [&](uint32_t w) {
                    return pack_half2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
                };
#pragma unroll 2
                for (int y = 0; y < 16; ++y) {
                    const uint4 u = *chunk(y);
                    *chunk(y) = make_uint4(scaled(u.x), scaled(u.y), scaled(u.z), scaled(u.w));
                }
                if (!ROWS) s_ex[lane_row] = ex;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(&q_full[t]);
            } else {
                ok = warp_wait(&q_full[0], li & 1, err);
                ex = s_ex[lane_row];
            }
            const float sl = score_factor(p.k_scale, ex);
            const int lim = min(item.S + qr / g, item.ke - 1);               // last key the row sees
            const int all = min(item.S + item.q0 / g, item.ke - 1);          // last key every row of the tile sees
            const int ks = item.ks, nsplit = item.nsplit, sp = item.sp;
            __syncwarp();
            if (lane == 0) bar_arrive(&item_empty[li % NITEM]);
            // The running maximum m in units of log2 and the weights' sum l.  A weight is
            // 2^(sl product + off), off = 6 - m, in one fma: m and off may be wrong by half a unit
            // in their last place, so scores must stay below 2^23.4, as they do with a factor up
            // to kNearFactor.  A row with a larger one has weights of 2^(sl (product + off) + 6),
            // -off the largest product; a warp with such a row takes the loop with that sum (its
            // other rows add 0 there).  That loop for all: 344 us for 326 at 64 windows of 32
            // over 8k.
            const bool far = sl > kNearFactor;
            float m = -INFINITY, off = kNoMax, l = 0.f;
            bool any = false;  // O holds something
            auto weigh_blocks = [&](auto far_rows) {  // the item's blocks of the tile
            constexpr bool FAR = decltype(far_rows)::value;
            for (int j = ROWS ? 0 : t; j < nblk; j += ROWS ? 1 : 2, ++x) {
                if (!(ok = warp_wait(&s_full[t], x & 1, err))) break;
                tc_fence_after();
                {
                    const int key0 = ks + j * KBLK;
                    const int gone = flags[(base + j) % FLAGS];  // (written before the block's K was)
                    // (Loops are kept rolled: four roles share the instruction cache.)
                    if (key0 + KBLK - 1 > all || gone) {
                        // scores of keys that are not visible to -inf, in place
#pragma unroll 1
                        for (int c = cb; c < ce; c += 32) {
                            uint32_t r[32];
                            tmem_ld32(tS + c, r);
                            tmem_wait_ld(r);
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (key0 + c + y > lim || ((gone >> ((c + y) / kPage)) & 1)) r[y] = 0xFF800000u;
                            tmem_st32(tS + c, r);
                        }
                        tmem_wait_st();
                    }
                    uint32_t ra[32], rb[32];  // scores of 32 keys each, one set loaded while the other is used
                    float mx[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) mx[y] = -INFINITY;
                    auto take_max = [&](const uint32_t (&r)[32]) {
#pragma unroll
                        for (int y = 0; y < 32; y += 2)
                            mx[(y >> 1) & 3] = max3(mx[(y >> 1) & 3], __uint_as_float(r[y]), __uint_as_float(r[y + 1]));
                    };
                    tmem_ld32(tS + cb, ra);
#pragma unroll 1
                    for (int c = cb; c < ce; c += 64) {
                        tmem_wait_ld(ra);
                        tmem_ld32(tS + c + 32, rb);
                        take_max(ra);
                        tmem_wait_ld(rb);
                        tmem_ld32(tS + (c + 64 < ce ? c + 64 : cb), ra);  // (at last the first ones again, for the weights)
                        take_max(rb);
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool grew = FAR && far ? top > -off : fmaf(top, sl, off) > kWeightLog2 + kLazyLog2;
                    if (__any_sync(0xffffffffu, grew)) {
                        const float v = top * sl, f = grew ? exp2_fast(m - v) : 1.f;
                        if (grew) {
                            m = v;
                            off = FAR && far ? -top : kWeightLog2 - v;
                            l *= f;
                        }
                        if (any) {
                            // (the tile's last P V was done before this S was issued)
#pragma unroll 1
                            for (int c = 0; c < HD; c += 32) {
                                tmem_ld32(tO + c, rb);
                                tmem_wait_ld(rb);
#pragma unroll
                                for (int y = 0; y < 32; ++y) rb[y] = __float_as_uint(__uint_as_float(rb[y]) * f);
                                tmem_st32(tO + c, rb);
                            }
                        }
                    }
                    uint64_t sum[2] = {0, 0};
                    const float z = FAR && far ? kWeightLog2 : off, shift = FAR && far ? off : 0.f;
                    const uint64_t sl2 = pair(sl, sl), z2 = pair(z, z), shift2 = pair(shift, shift);
                    // P of 32 keys over the first half of their own S: the arguments, then the
                    // exponentials, then the sums, so that the exp2 unit is fed without a pause
                    auto weigh = [&](int c, const uint32_t (&r)[32]) {
                        uint32_t pk[16];
                        float2 v[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const uint64_t s2 = pair(r[2 * y], r[2 * y + 1]);
                            v[y] = unpair(fma2(FAR ? add2(s2, shift2) : s2, sl2, z2));
                        }
#pragma unroll
                        for (int y = 0; y < 16; ++y) v[y] = make_float2(exp2_fast(v[y].x), exp2_fast(v[y].y));
#pragma unroll
                        for (int y = 0; y < 16; ++y) pk[y] = pack_half2(v[y].x, v[y].y);
#pragma unroll
                        for (int y = 0; y < 16; ++y) sum[y & 1] = add2(sum[y & 1], pair(v[y].x, v[y].y));
                        tmem_st16(tS + c, pk);
                    };
#pragma unroll 1
                    for (int c = cb; c < ce; c += 64) {
                        tmem_wait_ld(ra);
                        tmem_ld32(tS + c + 32, rb);
                        weigh(c, ra);
                        tmem_wait_ld(rb);
                        if (c + 64 < ce) tmem_ld32(tS + c + 64, ra);
                        weigh(c + 32, rb);
                    }
                    if (!ROWS && twice) {  // the other half's keys weigh nothing in this row of P
                        uint32_t zero[16] = {};
                        tmem_st16(tS + 64 - cb, zero);
                        tmem_st16(tS + 96 - cb, zero);
                    }
                    const float2 both = unpair(add2(sum[0], sum[1]));
                    l += both.x + both.y;
                    tmem_wait_st();
                }
                any = true;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&p_full[t]);
            }
            };
            if (__any_sync(0xffffffffu, far)) weigh_blocks(std::true_type{});
            else weigh_blocks(std::false_type{});
            base += nblk;
            if (ok && any) {
                ok = warp_wait(&pv_done[t], (x - 1) & 1, err);
                tc_fence_after();
            }
            if (ROWS) {
                if (!ok) break;
                const float f = out_factor(p.v_scale, l);
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(tO + c, r);
                    tmem_wait_ld(r);
                    if (live) store_row(p, nsplit, sp, at, c, r, f);
                }
                if (live && nsplit > 1) p.part_ml[at * p.max_splits + sp] = make_float2(m, l);
            } else {
                // A row's 2 (`twice`: 4) parts, of the threads that lie `step` apart, joined:
                // O = sum of 2^(m_i - M) O_i, M the largest m_i.  Of every 32 dims each of
                // those threads adds up and stores its share.
                const int step = twice ? 64 : 128, mine = (int)threadIdx.x & (step - 1);
                s_ml[threadIdx.x] = make_float2(m, l);
                if (!(ok = softmax_all(ok))) break;
                float M = -INFINITY, L = 0.f;
                for (int x = mine; x < 256; x += step) M = fmaxf(M, s_ml[x].x);
                for (int x = mine; x < 256; x += step) {
                    const float2 o = s_ml[x];
                    L += (o.x == -INFINITY ? 0.f : exp2_fast(o.x - M)) * o.y;  // (NaN stays NaN)
                }
                const float f = any && m > -INFINITY ? exp2_fast(m - M) : 0.f, inv = out_factor(p.v_scale, L);
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    uint32_t r[32];
                    if (any) {
                        tmem_ld32(tO + c, r);
                        tmem_wait_ld(r);
                    }
#pragma unroll
                    for (int y = 0; y < 32; ++y) xch[y * 256 + threadIdx.x] = f > 0.f ? f * __uint_as_float(r[y]) : 0.f;
                    if (!(ok = softmax_all(ok))) break;
                    const int share = step / 8, d0 = ((int)threadIdx.x / step) * share;  // 32 dims / (256 / step) threads
#pragma unroll 1
                    for (int d = d0; live && d < d0 + share; d += 8) {
                        float v[8] = {};
#pragma unroll 2
                        for (int x = mine; x < 256; x += step)
#pragma unroll
                            for (int y = 0; y < 8; ++y) v[y] += xch[(d + y) * 256 + x];
                        store8(p, nsplit, sp, at, c + d, v, inv);
                    }
                    if (!(ok = softmax_all(ok))) break;
                }
                if (!ok) break;
                if ((int)threadIdx.x < step && live && nsplit > 1) p.part_ml[at * p.max_splits + sp] = make_float2(M, L);
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
    }
}

template <bool ROWS>
cudaError_t launch(const AttnKv4Params& p, int num_sms, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(attn_kv4_tc_kernel<ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)p.n_seq * p.hkv * p.tiles * p.max_splits;
    const int grid = (int)std::min<int64_t>(most, num_sms);
    return launch_pdl(attn_kv4_tc_kernel<ROWS>, dim3(grid), dim3(THREADS), SMEM, st, p);
}

}  // namespace

namespace kv4 {

cudaError_t launch_attn_kv4_tc(const AttnKv4Params& p, int num_sms, cudaStream_t st) {
    return p.tile_rows <= 128 ? launch<false>(p, num_sms, st) : launch<true>(p, num_sms, st);
}

}  // namespace kv4
}  // namespace wedlm
