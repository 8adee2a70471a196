// What the kernels of the 4-bit KV cache share: its format, conversions, the
// attention's arguments and the division of its work.
//
// Format.  A row of 128 dims (one token's K or V of one head) is 8 blocks of
// 16 dims; a block is one scale s (e4m3) and 16 codes (e2m1: +-{0, .5, 1, 1.5,
// 2, 3, 4, 6}), and stands for code * s * k_scale (or v_scale), the latter a
// power of two the caller chooses.  4.5 bits per value, against 16.
//   s = e4m3(max|x| / 6),  code = e2m1(x / s),  both rounded to nearest even.
// A code has 2 and a scale 4 significant bits, so code * s is exact in fp16
// (at most 6 * 448, at least 2^-10): the attention multiplies them in fp16 and
// feeds the tensor cores without any rounding.
//
// A page of one head is 2304 contiguous bytes: [K, V][codes: 16 tokens x 64
// bytes (dim 2i in the low, 2i + 1 in the high nibble of byte i)][scales: 16
// tokens x 8 bytes], brought in by one bulk copy.
#pragma once

#include <cuda_fp16.h>

#include "kernels.cuh"

namespace wedlm {
namespace kv4 {

constexpr int HD = 128;
constexpr int kHalfPage = WEDLM_KV4_HALF_PAGE;  // K or V of one head's page
constexpr int kHeadPage = 2 * kHalfPage;        // both
constexpr int kCodes = kPage * HD / 2;          // bytes of codes in a half page

// ---------------------------------------------------------------------------
// Conversions between fp32 / fp16 and the 4- and 8-bit formats (one
// instruction each on sm_100a).
// The four bytes of a word: eight values.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// Eight values, the first in the lowest nibble.
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xFFu;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 half2_floats(uint32_t a) { return __half22float2(*reinterpret_cast<__half2*>(&a)); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Two fp32 values as one operand, and two operations in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void st_global8(void* p, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

// ---------------------------------------------------------------------------
// The attention.
constexpr int kMaxSplits = 128;       // key chunks of a row tile
constexpr float kLazyLog2 = 8.0f;     // growth of the maximum tolerated before O is rescaled
constexpr float kWeightLog2 = 6.0f;   // weights are held times 2^6
// In place of what a row adds to its scores before it has seen a key: any visible one (at
// least -2^124, see score_factor) raises the maximum, a masked one (-inf) does not.
constexpr float kNoMax = 0x1.8p127f;
constexpr float kNearFactor = 0x1p-10f;  // score factor up to which scores are below 2^23.4 (q rows up to 128 at k_scale 1)

struct AttnKv4Params {
    const bf16* q;
    const uint8_t* pool;
    const int32_t* table;
    const int32_t* S;
    const int32_t* n;
    bf16* out;
    float* part_o;       // [rows][hq][max_splits][128]
    float2* part_ml;     // [rows][hq][max_splits]
    unsigned* tickets;   // [n_seq][hkv] (one tile a sequence), zero between calls; nullptr: a second kernel joins the chunks
    int* err;
    int num_pages, hq, hkv, pages_per_seq, n_seq, stride, max_ctx, chunk, max_splits;
    int tile_rows, tiles;  // query rows (window rows x heads of a KV head) of a tile, tiles of a sequence
    float k_scale, v_scale;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void bar_init(uint64_t* bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// One head's page into shared memory; completes on `bar`.
__device__ __forceinline__ void load_page(void* dst, const uint8_t* src, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(kHeadPage), "r"(smem_u32(bar)) : "memory");
}

// Division of the work among persistent workers.  An item is one chunk of keys
// of (sequence, row tile, KV head); the items of all sequences that have rows
// are numbered full chunks first, every tile's last (shorter) chunk after them,
// and worker w of W takes items w, w + W, ...  A tile's place in the numbering
// comes from prefix sums over the (sequence, tile) groups, which a CTA builds
// once in shared memory; with more than kGroupCap groups they are walked, 32 at a
// time (64 prompts of 1024 rows, 32/8 heads: 1.04 ms, one at a time 1.25).
constexpr int kGroupCap = 256;

struct Item {
    int b, h, sp, q0, S, rows, ks, ke, nsplit;
};

struct ItemTable {
    int2 group[kGroupCap];  // (S, live query rows) of a group's sequence
    int full[kGroupCap];    // full-chunk items of the groups up to this one
    int last[kGroupCap];    // last-chunk items
};

// S, live query rows and key chunks of group grp (chunks 0: nothing to do).
__device__ __forceinline__ int group_load(const AttnKv4Params& p, int grp, int& S, int& rows) {
    const int b = grp / p.tiles, q0 = (grp - b * p.tiles) * p.tile_rows, g = p.hq / p.hkv;
    S = __ldcg(p.S + b);
    const int n = min(__ldcg(p.n + b), p.stride);
    rows = max(n, 0) * g;
    if (q0 >= rows) return 0;
    if (S < 0 || (int64_t)S + n > p.max_ctx) {
        set_error(p.err, kErrBounds);
        return 0;
    }
    return (S + (min(q0 + p.tile_rows, rows) - 1) / g) / p.chunk + 1;
}

__device__ __forceinline__ void item_fill(const AttnKv4Params& p, int grp, int h, int sp, int S, int rows, Item& o) {
    o.b = grp / p.tiles;
    o.q0 = (grp - o.b * p.tiles) * p.tile_rows;
    o.h = h;
    o.sp = sp;
    o.S = S;
    o.rows = rows;
    const int kend = S + (min(o.q0 + p.tile_rows, rows) - 1) / (p.hq / p.hkv) + 1;
    o.nsplit = (kend - 1) / p.chunk + 1;  // (positions, and ends of pages and blocks less one, fit 32 bits; sums past them may not)
    o.ks = sp * p.chunk;
    o.ke = o.ks + min(kend - o.ks, p.chunk);
}

// Called by all threads of the CTA; synchronises it.
__device__ __forceinline__ void items_build(const AttnKv4Params& p, ItemTable& t) {
    const int G = p.n_seq * p.tiles;
    if (G > kGroupCap) return;
    for (int i = threadIdx.x; i < G; i += blockDim.x) {
        int S, rows;
        const int ns = group_load(p, i, S, rows);
        t.group[i] = make_int2(S, rows);
        t.full[i] = ns > 0 ? p.hkv * (ns - 1) : 0;
        t.last[i] = ns > 0 ? p.hkv : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int carry = 0, carry2 = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            int v = g0 + lane < G ? t.full[g0 + lane] : 0, v2 = g0 + lane < G ? t.last[g0 + lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o), u2 = __shfl_up_sync(0xffffffffu, v2, o);
                if (lane >= o) {
                    v += u;
                    v2 += u2;
                }
            }
            if (g0 + lane < G) {
                t.full[g0 + lane] = carry + v;
                t.last[g0 + lane] = carry2 + v2;
            }
            carry += __shfl_sync(0xffffffffu, v, 31);
            carry2 += __shfl_sync(0xffffffffu, v2, 31);
        }
    }
    __syncthreads();
}

struct ItemIter {
    int64_t next;                      // number of the next item
    int g1 = 0, g2 = 0;                // where the searches start
    // walking: 32 groups from grp on, one to a lane; base: number of their first item
    int64_t base = 0;
    int grp = 0, S = 0, rows = 0, ns = 0, upto = -1;  // upto: items of the groups up to the lane's, -1: not loaded
};

// First g in [lo, G) with a[g] > x (a non-decreasing, a[G - 1] > x).
__device__ __forceinline__ int item_search(const int* a, int lo, int G, int x) {
    int hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Called by a whole warp.
__device__ __forceinline__ bool item_next(ItemIter& it, const AttnKv4Params& p, const ItemTable& t, int workers,
                                          Item& o) {
    const int G = p.n_seq * p.tiles;
    if (G <= kGroupCap) {
        const int nfull = t.full[G - 1];
        if (it.next >= nfull + t.last[G - 1]) return false;
        const bool in_full = it.next < nfull;
        const int x = (int)it.next - (in_full ? 0 : nfull);
        const int* a = in_full ? t.full : t.last;
        const int g = item_search(a, in_full ? it.g1 : it.g2, G, x);
        (in_full ? it.g1 : it.g2) = g;
        const int local = x - (g ? a[g - 1] : 0), of = a[g] - (g ? a[g - 1] : 0);
        const int2 v = t.group[g];
        const int per = of / p.hkv;  // full chunks of a head (1 among the last ones)
        item_fill(p, g, local / per, local % per, v.x, v.y, o);
        if (!in_full) {
            o.sp = o.nsplit - 1;
            o.ks = o.sp * p.chunk;
            o.ke = o.S + (min(o.q0 + p.tile_rows, o.rows) - 1) / (p.hq / p.hkv) + 1;
        }
        it.next += workers;
        return true;
    }
    const int lane = threadIdx.x & 31;
    while (it.grp < G) {
        if (__any_sync(0xffffffffu, it.upto < 0)) {
            it.ns = it.grp + lane < G ? group_load(p, it.grp + lane, it.S, it.rows) : 0;
            it.upto = p.hkv * it.ns;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, it.upto, d);
                if (lane >= d) it.upto += u;
            }
        }
        const int all = __shfl_sync(0xffffffffu, it.upto, 31);
        if (it.next < it.base + all) {
            const int x = (int)(it.next - it.base);
            const int g = __ffs(__ballot_sync(0xffffffffu, it.upto > x)) - 1;
            const int ns = __shfl_sync(0xffffffffu, it.ns, g), S = __shfl_sync(0xffffffffu, it.S, g),
                      rows = __shfl_sync(0xffffffffu, it.rows, g);
            const int local = x - (__shfl_sync(0xffffffffu, it.upto, g) - p.hkv * ns);
            item_fill(p, it.grp + g, local / ns, local % ns, S, rows, o);
            it.next += workers;
            return true;
        }
        it.base += all;
        it.upto = -1;
        it.grp += 32;
    }
    return false;
}

// What turns the product of a q row that was scaled by 2^e and a key without its scale into a
// score in units of log2: kept inside fp32's normal range whatever the scale and e (a factor of
// zero would turn a masked score, -inf, into NaN, an infinite one a score of zero).  Products
// are below 2^34 and above 2^-34: with a factor of 2^-126 every score is as good as zero, and
// with one of 2^89 two scores are equal or far apart, as with the true factors beyond.
// A row with an infinity or a NaN (its e) has NaN: the softmax of its scores is that, also
// where all of them are -inf, which are not to be taken for masked ones.
constexpr int kNotFinite = 14 + 127 - 255;
__device__ __forceinline__ float score_factor(float k_scale, int e) {
    if (e == kNotFinite) return __int_as_float(0x7FC00000);
    const float f = 1.4426950408889634f / sqrtf((float)HD) * k_scale * __int_as_float((127 - e) << 23);
    return fminf(fmaxf(f, 0x1p-126f), 0x1p89f);
}

// What the outputs are multiplied by, given the weights' sum: 0 for a row that
// saw no key (every page of it outside the pool), NaN where the sum is.
__device__ __forceinline__ float out_factor(float v_scale, float l) { return l > 0.f || l != l ? v_scale / l : 0.f; }

// The kernel for tiles of more than 16 query rows (kv4_tc.cu): p.tile_rows
// query rows a tile, 128 or 256.
cudaError_t launch_attn_kv4_tc(const AttnKv4Params& p, int num_sms, cudaStream_t st);

}  // namespace kv4
}  // namespace wedlm
