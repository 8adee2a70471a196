// A KV cache held in 4 bits and the attention that reads it.
#include <algorithm>
#include <cmath>

#include "kv4.cuh"

namespace wedlm {
namespace {

using namespace kv4;

// ---------------------------------------------------------------------------
// Rows in and out of the cache.
struct RowsParams {
    uint8_t* pool;
    const int32_t* table;
    const int32_t* S;
    const int32_t* n;
    int* err;
    int64_t rows;
    int64_t k_stride, v_stride;
    int num_pages, hkv, pages_per_seq, stride;
    float k_scale, v_scale;
    uint32_t by, shift;  // x / stride = x * by >> shift, for x below 2^31
    int wide;            // every row starts on a 32-byte boundary
};

constexpr int kRowWarps = 4;  // rows of a CTA

// Where a row's token lies in its page (all lanes alike): the page, or -1 for a
// row that is not live or has no place.
__device__ __forceinline__ int locate_row(const RowsParams& p, uint32_t row, int& tok) {
    const uint32_t b = (uint32_t)((uint64_t)row * p.by >> p.shift);
    const int r = (int)(row - b * (uint32_t)p.stride);
    const int n = __ldcg(p.n + b), S = __ldcg(p.S + b);
    if (r >= n) return -1;
    const int64_t pos = (int64_t)S + r;
    if (S < 0 || pos >= (int64_t)p.pages_per_seq * kPage) {
        set_error(p.err, kErrBounds);
        return -1;
    }
    const int page = __ldcg(p.table + (int64_t)b * p.pages_per_seq + pos / kPage);
    if (page < 0 || page >= p.num_pages) {
        set_error(p.err, kErrBounds);
        return -1;
    }
    tok = (int)(pos % kPage);
    return page;
}

// Block u of a row: K's heads, then V's, eight 16-dim blocks each.
struct RowBlock {
    int which, head, blk;
};
__device__ __forceinline__ RowBlock row_block(const RowsParams& p, int u) {
    RowBlock o;
    o.blk = u & 7;
    o.which = u >= p.hkv * 8;
    o.head = (u >> 3) - o.which * p.hkv;
    return o;
}
__device__ __forceinline__ uint8_t* half_page(const RowsParams& p, int page, const RowBlock& o) {
    return p.pool + (((int64_t)page * p.hkv + o.head) * 2 + o.which) * kHalfPage;
}

// 32 bytes of a row, a whole memory sector: in one access where the rows allow it
// (two of 16 bytes ask for the sector twice: 5 us more of 41 at 16 x 1024 rows of
// 8 heads, in and back out).
__device__ __forceinline__ void load32(uint4* w, const void* x, int wide) {
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x), "=r"(w[1].y), "=r"(w[1].z),
                       "=r"(w[1].w)
                     : "l"(x)
                     : "memory");
    } else {
        w[0] = __ldcg(static_cast<const uint4*>(x));
        w[1] = __ldcg(static_cast<const uint4*>(x) + 1);
    }
}
__device__ __forceinline__ void store32(void* x, const uint32_t (&w)[8], int wide) {
    if (wide) {
        st_global8(x, w);
    } else {
        static_cast<uint4*>(x)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(x)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// 16 values as they lie in memory, their largest magnitude (as fp32 bits: 0x7F800000
// or more where one is not finite) and their fp32 form.
template <typename T>
struct Raw16;
template <>
struct Raw16<float> {
    uint4 w[4];
    __device__ __forceinline__ void load(const float* x, int wide) {
        load32(w, x, wide);
        load32(w + 2, x + 8, wide);
    }
    __device__ __forceinline__ uint32_t word(int j) const {
        const uint4 u = w[j >> 2];
        return (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, word(j) & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ float get(int j) const { return __uint_as_float(word(j)); }
};
template <>
struct Raw16<bf16> {
    uint4 w[2];
    __device__ __forceinline__ void load(const bf16* x, int wide) { load32(w, x, wide); }
    __device__ __forceinline__ uint32_t word(int j) const {
        const uint4 u = w[j >> 2];
        return (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;  // two 16-bit maxima
#pragma unroll
        for (int j = 0; j < 8; ++j) m = __vmaxu2(m, word(j) & 0x7FFF7FFFu);
        return max(m >> 16, m & 0xFFFFu) << 16;
    }
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float(j & 1 ? word(j >> 1) & 0xFFFF0000u : word(j >> 1) << 16);
    }
};
__device__ __forceinline__ void store16(float* x, const float (&v)[16], int wide) {
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[h + j]);
        store32(x + h, w, wide);
    }
}
__device__ __forceinline__ void store16(bf16* x, const float (&v)[16], int wide) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&t);
    }
    store32(x, w, wide);
}

// The scale's and the codes' quotients.  One halfway between two e4m3 or e2m1 values
// must be met exactly, one that is not must stay on its side.  fp32 rows: a
// correctly rounded division does both.  bf16 rows: x has 8 significant bits, s has
// 4, the halfway points 5 and 3 and 6 has 2, so that a quotient that is no halfway
// point is at least 2^-10 of itself away from one: a product with an approximate
// reciprocal (off by less than 2^-21 with its own rounding) does, once it is
// rounded to 12 bits.  (On the bits: a half added, the rest cleared.  An infinity
// that comes of it saturates like the value itself.)
__device__ __forceinline__ float round12(float x) {
    return __uint_as_float((__float_as_uint(x) + 0x800u) & 0xFFFFF000u);
}
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <typename T>
__device__ __forceinline__ float sixth(float x) {
    if constexpr (sizeof(T) == 4) return __fdiv_rn(x, 6.0f);
    return round12(x * (1.0f / 6.0f));
}
__device__ __forceinline__ uint32_t codes8(const Raw16<float>& x, int at, float s, float inv_g) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __fdiv_rn(x.get(at + j) * inv_g, s);
    return f32_to_e2m1x8(q);
}
__device__ __forceinline__ uint32_t codes8(const Raw16<bf16>& x, int at, float s, float inv_g) {
    const float d = reciprocal(s) * inv_g;
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = round12(x.get(at + j) * d);
    return f32_to_e2m1x8(q);
}

// A warp per row, a lane per block of 16 dims, U blocks of a lane in flight (the
// second grid axis takes the rest of a row): the row's place in the cache is
// looked up once, beside the first loads.  A block with a NaN or an infinity is
// stored as zeros and recorded in the error word: the cache only ever holds
// finite values.
template <typename T, int U>
__global__ void __launch_bounds__(32 * kRowWarps) kv4_append_kernel(const T* k, const T* v, RowsParams p) {
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, u0 = blockIdx.y * (32 * U) + lane, units = p.hkv * 16;
    const uint32_t row = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (row >= (uint32_t)p.rows) return;
    Raw16<T> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (u0 + 32 * i >= units) continue;
        const RowBlock o = row_block(p, u0 + 32 * i);
        x[i].load((o.which ? v + row * p.v_stride : k + row * p.k_stride) + o.head * HD + o.blk * 16, p.wide);
    }
    int tok = 0;
    const int page = locate_row(p, row, tok);
    if (page < 0) return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (u0 + 32 * i >= units) continue;
        const RowBlock o = row_block(p, u0 + 32 * i);
        const float inv_g = 1.0f / (o.which ? p.v_scale : p.k_scale);  // powers of two: exact
        const uint32_t top = x[i].top();
        uint32_t lo = 0, hi = 0, sc = 0;
        if (top >= 0x7F800000u) {
            set_error(p.err, kErrNonFinite);
        } else {
            sc = f32_to_e4m3(sixth<T>(fminf(__uint_as_float(top) * inv_g, 3.0e38f)));
            if (sc) {
                const float s = half2_floats(e4m3x2_to_f16x2(sc)).x;
                lo = codes8(x[i], 0, s, inv_g);
                hi = codes8(x[i], 8, s, inv_g);
            }
        }
        uint8_t* half = half_page(p, page, o);
        *reinterpret_cast<uint2*>(half + tok * 64 + o.blk * 8) = make_uint2(lo, hi);
        half[kCodes + tok * 8 + o.blk] = (uint8_t)sc;
    }
}

// The kernel after this one does not start early: the rows may have been written
// straight into pages of a bf16 cache, and the attention over those reads them before
// its dependency wait.
template <typename T, int U>
__global__ void __launch_bounds__(32 * kRowWarps) kv4_read_kernel(T* k, T* v, RowsParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31, u0 = blockIdx.y * (32 * U) + lane, units = p.hkv * 16;
    const uint32_t row = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (row >= (uint32_t)p.rows) return;
    int tok = 0;
    const int page = locate_row(p, row, tok);
    if (page < 0) return;
    uint2 c[U];
    uint32_t sc[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (u0 + 32 * i >= units) continue;
        const RowBlock o = row_block(p, u0 + 32 * i);
        const uint8_t* half = half_page(p, page, o);
        c[i] = __ldcg(reinterpret_cast<const uint2*>(half + tok * 64 + o.blk * 8));
        sc[i] = __ldcg(half + kCodes + tok * 8 + o.blk);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (u0 + 32 * i >= units) continue;
        const RowBlock o = row_block(p, u0 + 32 * i);
        const float s = half2_floats(e4m3x2_to_f16x2(sc[i])).x * (o.which ? p.v_scale : p.k_scale);
        float x[16];
        uint32_t h[4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            e2m1x8_to_f16x2(w ? c[i].y : c[i].x, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = half2_floats(h[j]);
                x[8 * w + 2 * j] = f.x * s;
                x[8 * w + 2 * j + 1] = f.y * s;
            }
        }
        store16((o.which ? v + row * p.v_stride : k + row * p.k_stride) + o.head * HD + o.blk * 16, x, p.wide);
    }
    settle_writes();
}

// Four blocks of a lane (more loads in flight, one look-up for all) where a launch
// has rows enough to fill the GPU with that, else one (more warps).  In and back
// out, 8 heads: 16 x 1024 bf16 rows 43 us with four, 66 with one (158 MB at 6.5 TB/s:
// 24 us; bound by the instructions of the conversions and by the latency of the
// look-up), fp32 rows 71 and 76 (306 MB, 47 us; append alone 42 and 38); with one head
// 15.5 and 14.9.  16 x 16 fp32 rows 5.7 us with one, 7.9 with four (latency alone).
template <typename T>
cudaError_t launch_append(const RowsParams& p, const void* k, const void* v, cudaStream_t st) {
    const unsigned ctas = (unsigned)((p.rows + kRowWarps - 1) / kRowWarps), per = (unsigned)(p.hkv + 1) / 2;
    if (p.rows < 4096)
        return launch_pdl(kv4_append_kernel<T, 1>, dim3(ctas, per), dim3(32 * kRowWarps), 0, st, (const T*)k, (const T*)v, p);
    return launch_pdl(kv4_append_kernel<T, 4>, dim3(ctas, (per + 3) / 4), dim3(32 * kRowWarps), 0, st, (const T*)k,
                      (const T*)v, p);
}
template <typename T>
cudaError_t launch_read(const RowsParams& p, void* k, void* v, cudaStream_t st) {
    const unsigned ctas = (unsigned)((p.rows + kRowWarps - 1) / kRowWarps), per = (unsigned)(p.hkv + 1) / 2;
    if (p.rows < 4096)
        return launch_pdl(kv4_read_kernel<T, 1>, dim3(ctas, per), dim3(32 * kRowWarps), 0, st, (T*)k, (T*)v, p);
    return launch_pdl(kv4_read_kernel<T, 4>, dim3(ctas, (per + 3) / 4), dim3(32 * kRowWarps), 0, st, (T*)k, (T*)v, p);
}

// ---------------------------------------------------------------------------
// Attention over the 4-bit cache: out = softmax(q K^T / sqrt(128)) V of window
// rows r over cache positions 0 .. S + r, as wedlm_attention_bf16.
//
// Work item (a CTA of one warp): all of a sequence's query rows of one KV head
// (window rows x the g heads that share it, at most NT * 8), one chunk of keys, two
// pages at a time through a ring of page buffers filled by bulk copies.  Codes go
// from shared memory to registers, are widened and scaled there and feed mma.sync
// directly: no widened copy of K or V is ever written anywhere.  The cache is the M side of
// both products (S^T = K Q^T, O^T = V^T P^T), so that a token's 4 to 8 query
// rows fill the 8-wide N side; P^T is S^T transposed in registers.  The dims
// are permuted inside the products (which changes no sum): in K Q^T the lanes
// of a quad own 32 consecutive dims each, so a lane's operands of a key are 16
// consecutive bytes; in V^T P^T a lane owns the 16 dims of one scale block.
// Warps share nothing, so the SM's schedulers always have others to run while
// one of them starts, waits or writes its result.
//
// Q is held in fp16 scaled per row by a power of two (its largest element in
// [2^14, 2^15)), which keeps every bit of a bf16 q that is within 2^-28 of the
// row's largest; the factor is undone in the fp32 scores.  P is fp16, relative
// to a running maximum that is only raised when a score exceeds it by 2^8, and
// times 2^6, so weights down to 2^-30 of the largest are kept; sums and
// outputs are fp32.
//
// Measured: 64 sequences of 1k to 8.2k keys, one row of 32 heads over 8 KV heads:
// 92.6 us, 3.6 TB/s, with the join's 9 (four warps to a CTA that joined their parts in
// shared memory: 132).  Bound by instructions, 373 a page, with the issue slots 67 %
// busy: of the 20 warps that an SM's registers allow 15 are there on average, the
// others end, start, or have no item left.  1 sequence of 256: 7.9 us, latency (the
// four warps of a CTA, which joined through shared memory, 6.2; they lost at length).
constexpr int kStep = 2;              // pages of a stage
constexpr int kStages = 2;            // (three, at 16 warps an SM: slower)
constexpr int kItemsPerSm = 48;       // (36 and 64: no faster)
// Up to this many chunks the one that finishes last joins them, 8 lanes a row; more are
// left to a second kernel (1 sequence of 2000, 32 chunks: 9.5 us, by the last one 13.5).
constexpr int kTicketSplits = 8;
// Tickets count from call to call, so they have a place in the workspace that no call, of
// whatever sizes, uses for anything else: room for this many in front of the partial results,
// 64 KB.  Calls with more (sequence, KV head) pairs take the second kernel (1024 sequences of
// 1000 keys and 8 KV heads, two chunks each: 241 us with tickets, 264 with the kernel).
constexpr int kTickets = 16384;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values (lane 4 i + c holds row i, columns 2c, 2c + 1) transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// A lane's 32 dims of one query row (32 c .. 32 c + 31), scaled to fp16: the
// operands of the 8 k-steps (two registers per step); returns the exponent
// that was added.
__device__ __forceinline__ int load_q(const bf16* q, bool live, uint32_t (&a)[16]) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 u = live ? __ldcg(reinterpret_cast<const uint4*>(q) + j) : make_uint4(0, 0, 0, 0);
        w[4 * j] = u.x;
        w[4 * j + 1] = u.y;
        w[4 * j + 2] = u.z;
        w[4 * j + 3] = u.w;
    }
    uint32_t m = 0;  // the largest magnitude's bits
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = min(100, 14 + 127 - (int)(m >> 7));
    const float f = __int_as_float((e + 127) << 23);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        a[j] = pack_half2(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xFFFF0000u) * f);
    return e;
}

__device__ __forceinline__ void store_out(const AttnKv4Params& p, int64_t at, int lane, float4 v, float f) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * f, v.y * f), hi = __floats2bfloat162_rn(v.z * f, v.w * f);
    *reinterpret_cast<uint2*>(p.out + at * HD + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Chunks s0 .. s0 + 31 of one (row, head), those below `end`: weights relative
// to their common maximum m, in lane s - s0; the weighted sum of the outputs'
// dims 4 lane .. + 3 in acc and of the l's in l.
__device__ __forceinline__ void join_range(const AttnKv4Params& p, int64_t at, int s0, int end, int lane, float& m,
                                           float& l, float4& acc) {
    const int count = min(32, end - s0);
    const float2 ml = lane < count ? __ldcg(p.part_ml + at * p.max_splits + s0 + lane) : make_float2(-INFINITY, 0.f);
    const float4* po = reinterpret_cast<const float4*>(p.part_o + (at * p.max_splits + s0) * HD) + lane;
    float4 v[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] = x < count ? __ldcg(po + x * (HD / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
    m = warp_max(ml.x);
    const float w = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - m);
    l = warp_sum(w * ml.y);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < count; x0 += 8) {
        if (x0 > 0) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                v[x] = x0 + x < count ? __ldcg(po + (x0 + x) * (HD / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float f = __shfl_sync(0xffffffffu, w, (x0 + x) & 31);
            acc.x += f * v[x].x;
            acc.y += f * v[x].y;
            acc.z += f * v[x].z;
            acc.w += f * v[x].w;
        }
    }
}

template <int NT>
__global__ void __launch_bounds__(32, NT == 1 ? 20 : 10) attn_kv4_kernel(const AttnKv4Params p) {
    __shared__ __align__(128) uint8_t ring[kStages][kStep][kHeadPage];
    __shared__ __align__(8) uint64_t bars[kStages];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x, c = lane & 3, j8 = lane >> 2;
    const int g = p.hq / p.hkv;
    // All sequences' first chunks, then their second ones, ...: items beyond a
    // sequence's end come last (chunks of a sequence in a row: 97 us for 94).
    const unsigned pair = blockIdx.x / p.hkv;
    const int h = (int)(blockIdx.x - pair * p.hkv), b = (int)(pair % p.n_seq), sp = (int)(pair / p.n_seq);
    const int S = __ldcg(p.S + b), n = min(__ldcg(p.n + b), p.stride);
    const int32_t* table = p.table + (int64_t)b * p.pages_per_seq;
    const int ks = sp * p.chunk, page0 = ks / kPage;
    // Page ids, 32 at a time, one per lane; the first ones are read together with S and n.
    auto raw_id = [&](int k) { return page0 + k < p.pages_per_seq && k * kPage < p.chunk ? __ldcg(table + page0 + k) : -1; };
    int ids = raw_id(lane);
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) bar_init(&bars[s]);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    const int rows = n * g;  // at most 8 NT
    if (n <= 0) return;
    if (S < 0 || (int64_t)S + n > p.max_ctx) {
        set_error(p.err, kErrBounds);
        return;
    }
    const int kend = S + n;
    const int nsplit = (kend - 1) / p.chunk + 1;
    if (sp >= nsplit) return;
    const int ke = ks + min(kend - ks, p.chunk);
    const int npages = (ke - 1) / kPage + 1 - page0, steps = (npages + kStep - 1) / kStep;
    // Step k's pages into its stage; a page outside the pool is not loaded and
    // its keys count as masked.
    uint32_t gone = 0;  // bit kStep * s + x: page x of stage s is not there
    int issued = 0;
    auto issue = [&]() {
        const int k0 = issued * kStep, s = issued % kStages;
        if ((k0 & 31) == 0 && k0 > 0) ids = raw_id(k0 + lane);
        int page[kStep];
        uint32_t bytes = 0;
        gone &= ~(((1u << kStep) - 1) << (kStep * s));
#pragma unroll
        for (int x = 0; x < kStep; ++x) {
            page[x] = __shfl_sync(0xffffffffu, ids, (k0 + x) & 31);
            const bool wanted = k0 + x < npages;
            if (wanted && page[x] >= 0 && page[x] < p.num_pages) {
                bytes += kHeadPage;
            } else {
                if (wanted && lane == 0) set_error(p.err, kErrBounds);
                gone |= 1u << (kStep * s + x);
                page[x] = -1;
            }
        }
        if (lane == 0) {
            bar_expect(&bars[s], bytes);
#pragma unroll
            for (int x = 0; x < kStep; ++x)
                if (page[x] >= 0)
                    load_page(ring[s][x], p.pool + ((int64_t)page[x] * p.hkv + h) * kHeadPage, &bars[s]);
        }
        ++issued;
    };
    while (issued < min(steps, kStages)) issue();

    // Q of row j8 of every n-tile (operand B) and, for the lane's own columns
    // (queries 2c and 2c + 1 of every n-tile), score factors and last keys
    uint32_t qf[NT][16];
    float sl[NT][2];
    int lim[NT][2], lim_min = ke - 1;
    const int64_t row0 = (int64_t)b * p.stride;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = 8 * t + j8, rc = min(r, rows - 1);
        const int e = load_q(p.q + ((row0 + rc / g) * p.hq + h * g + rc % g) * HD + 32 * c, r < rows, qf[t]);
        const float f = score_factor(p.k_scale, e);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            sl[t][x] = __shfl_sync(0xffffffffu, f, (2 * c + x) * 4);
            lim[t][x] = min(S + min(8 * t + 2 * c + x, rows - 1) / g, ke - 1);
            lim_min = min(lim_min, lim[t][x]);
        }
    }
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));

    float o[8][NT][4] = {};
    // Per own column: the running maximum m of the scores in the exp2 domain and
    // the weights' sum; a weight is exp2(score + z), z = 6 - m (before the first key
    // kNoMax).  The score is rounded before z is added, as m was: of a fused product and
    // sum the part that m lost would remain, more than any exponent at scores past 2^28.
    float m[NT][2], z[NT][2], l[NT][2] = {};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t][0] = m[t][1] = -INFINITY;
        z[t][0] = z[t][1] = kNoMax;
    }
    // A page's 16 keys.  (One body, its masks under a branch: the loop stays small
    // enough for the instruction cache.)
    auto step = [&](const uint8_t* K, int key0) {
        const uint8_t* V = K + kHalfPage;
        const bool edge = key0 + kPage - 1 > lim_min;
        // S^T: lane's rows are keys j8 and j8 + 8
        float sc[NT][4] = {}, sd[NT][4] = {};  // (two sums, so that half as many products wait for one another)
        {
            const uint4 u0 = *reinterpret_cast<const uint4*>(K + j8 * 64 + c * 16);
            const uint4 u1 = *reinterpret_cast<const uint4*>(K + j8 * 64 + 512 + c * 16);
            const uint32_t s0 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(K + kCodes + j8 * 8 + c * 2));
            const uint32_t s1 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(K + kCodes + j8 * 8 + 64 + c * 2));
            const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
            const uint32_t f0[2] = {__byte_perm(s0, s0, 0x1010), __byte_perm(s0, s0, 0x3232)};
            const uint32_t f1[2] = {__byte_perm(s1, s1, 0x1010), __byte_perm(s1, s1, 0x3232)};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t a[4], d[4];
                e2m1x8_to_f16x2(w0[x], a);
                e2m1x8_to_f16x2(w1[x], d);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t a0 = hmul2(a[2 * y], f0[x >> 1]), a1 = hmul2(d[2 * y], f1[x >> 1]);
                    const uint32_t a2 = hmul2(a[2 * y + 1], f0[x >> 1]), a3 = hmul2(d[2 * y + 1], f1[x >> 1]);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        mma_f16(y ? sd[t] : sc[t], a0, a1, a2, a3, qf[t][4 * x + 2 * y], qf[t][4 * x + 2 * y + 1]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[t][x] += sd[t][x];
        }
        // V^T: lane's rows are dims 16 j8 .. + 15, its columns keys 2c, 2c + 1, 8 + 2c, 9 + 2c
        uint2 u[4];
        uint32_t vs[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = t * 8 + 2 * c;
            u[2 * t] = *reinterpret_cast<const uint2*>(V + tok * 64 + j8 * 8);
            u[2 * t + 1] = *reinterpret_cast<const uint2*>(V + tok * 64 + 64 + j8 * 8);
            vs[2 * t] = V[kCodes + tok * 8 + j8];
            vs[2 * t + 1] = V[kCodes + tok * 8 + 8 + j8];
        }
        if (edge) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (key0 + j8 + 8 * (x >> 1) > lim[t][x & 1]) sc[t][x] = -INFINITY;
            // V of keys past the last row's: whatever their bytes say, they add nothing
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (key0 + 8 * (x >> 1) + 2 * c + (x & 1) >= ke) vs[x] = 0;
        }
        float top = -INFINITY;
        float e[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                e[t][x] = __fadd_rn(__fmul_rn(sc[t][x], sl[t][x & 1]), z[t][x & 1]);
                top = fmaxf(top, e[t][x]);
            }
        if (__any_sync(0xffffffffu, top > kWeightLog2 + kLazyLog2)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float s0 = __fmul_rn(sc[t][x], sl[t][x]), s1 = __fmul_rn(sc[t][2 + x], sl[t][x]);
                    float v = fmaxf(s0, s1);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                    // (by this row's own scores alone: no result depends on the rows beside it)
                    if (__fadd_rn(v, z[t][x]) > kWeightLog2 + kLazyLog2) {
                        const float f = exp2_fast(m[t][x] - v);
                        m[t][x] = v;
                        z[t][x] = kWeightLog2 - v;
                        l[t][x] *= f;
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            o[y][t][x] *= f;
                            o[y][t][2 + x] *= f;
                        }
                    }
                    e[t][x] = __fadd_rn(s0, z[t][x]);
                    e[t][2 + x] = __fadd_rn(s1, z[t][x]);
                }
        }
        uint32_t bt[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                e[t][x] = exp2_fast(e[t][x]);
                l[t][x & 1] += e[t][x];
            }
            bt[t][0] = transpose8x8(pack_half2(e[t][0], e[t][1]));
            bt[t][1] = transpose8x8(pack_half2(e[t][2], e[t][3]));
        }
        const uint32_t s2[2] = {e4m3x2_to_f16x2(vs[0] | vs[1] << 8), e4m3x2_to_f16x2(vs[2] | vs[3] << 8)};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            // bytes of (key, key + 1) codes: even dims, then odd dims, of 8 dims
            uint32_t ev[2][4], od[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t w0 = x ? u[2 * t].y : u[2 * t].x, w1 = x ? u[2 * t + 1].y : u[2 * t + 1].x;
                e2m1x8_to_f16x2((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), ev[t]);
                e2m1x8_to_f16x2(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), od[t]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t a0 = hmul2(ev[0][y], s2[0]), a1 = hmul2(od[0][y], s2[0]);
                const uint32_t a2 = hmul2(ev[1][y], s2[1]), a3 = hmul2(od[1][y], s2[1]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(o[4 * x + y][t], a0, a1, a2, a3, bt[t][0], bt[t][1]);
            }
        }
    };
    bool ok = true;  // after a wait that gave up the rest is computed from whatever is there: the error word tells
    for (int k = 0, s = 0, par = 0; k < steps; ++k) {
        const int key0 = (page0 + k * kStep) * kPage;
        ok = mbar_wait_bounded(smem_u32(&bars[s]), par, p.err) && ok;
        __syncwarp();
#pragma unroll 1
        for (int pg = 0; pg < kStep; ++pg)
            if (!((gone >> (kStep * s + pg)) & 1)) step(ring[s][pg], key0 + pg * kPage);
        __syncwarp();  // every lane has read the stage
        if (issued < steps) issue();
        if (++s == kStages) {
            s = 0;
            par ^= 1;
        }
    }
    if (__any_sync(0xffffffffu, !ok)) {  // copies still in flight land before the CTA's memory is given up
        for (int k = max(0, steps - kStages); k < steps; ++k)
            mbar_wait_bounded(smem_u32(&bars[k % kStages]), (k / kStages) & 1, nullptr, 200000000LL);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[t][x] += __shfl_xor_sync(0xffffffffu, l[t][x], d);
            // dims 16 j8 .. + 15 of the column's row
            const int qr = 8 * t + 2 * c + x;
            if (qr >= rows) continue;
            const int64_t at = (row0 + qr / g) * p.hq + h * g + qr % g;
            if (nsplit == 1) {
                const float f = out_factor(p.v_scale, l[t][x]);
#pragma unroll
                for (int u = 0; u < 8; u += 2)
                    store_out(p, at, 4 * j8 + u / 2,
                              make_float4(o[u][t][x], o[u][t][2 + x], o[u + 1][t][x], o[u + 1][t][2 + x]), f);
            } else {
                float4* dst = reinterpret_cast<float4*>(p.part_o + (at * p.max_splits + sp) * HD + 16 * j8);
#pragma unroll
                for (int u = 0; u < 8; u += 2)
                    dst[u / 2] = make_float4(o[u][t][x], o[u][t][2 + x], o[u + 1][t][x], o[u + 1][t][2 + x]);
                if (j8 == 0) p.part_ml[at * p.max_splits + sp] = make_float2(m[t][x], l[t][x]);
            }
        }
    if (nsplit == 1 || !p.tickets) return;
    // The chunk that finishes last joins them all.  The ticket counts to nsplit
    // and wraps to zero, so the workspace is as it was.
    __threadfence();
    __syncwarp();
    unsigned last = 0;
    if (lane == 0)
        last = atomicInc(p.tickets + (int64_t)b * p.hkv + h, nsplit - 1) == (unsigned)nsplit - 1;
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __threadfence();
    // Eight lanes a row, four rows at a time: lane x of the eight holds chunk x's
    // (m, l) and 16 of the dims.
    const int x8 = lane & 7;
    for (int r0 = 0; r0 < rows; r0 += 4) {
        const int r = min(r0 + (lane >> 3), rows - 1);
        const int64_t at = (row0 + r / g) * p.hq + h * g + r % g;
        const float2 ml = x8 < nsplit ? __ldcg(p.part_ml + at * p.max_splits + x8) : make_float2(-INFINITY, 0.f);
        const float4* po = reinterpret_cast<const float4*>(p.part_o + at * p.max_splits * HD) + x8;
        float mm = ml.x;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
        const float w = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - mm);
        float ll = w * ml.y;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
        float4 acc[4] = {};
#pragma unroll 2
        for (int s = 0; s < nsplit; ++s) {
            const float f = __shfl_sync(0xffffffffu, w, (lane & 24) + s);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float4 v = __ldcg(po + s * (HD / 4) + 8 * d);
                acc[d].x += f * v.x;
                acc[d].y += f * v.y;
                acc[d].z += f * v.z;
                acc[d].w += f * v.w;
            }
        }
        if (r0 + (lane >> 3) < rows) {
#pragma unroll
            for (int d = 0; d < 4; ++d) store_out(p, at, x8 + 8 * d, acc[d], out_factor(p.v_scale, ll));
        }
    }
}

// The key chunks of a (row, query head) joined, where they are many: a CTA
// each, a warp for every 32 chunks.
__global__ void __launch_bounds__(kMaxSplits) attn_kv4_join_kernel(const AttnKv4Params p) {
    __shared__ float4 s_acc[kMaxSplits / 32][32];
    __shared__ float2 s_ml[kMaxSplits / 32];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t at = blockIdx.x;
    const int64_t row = at / p.hq;
    const int head = (int)(at - row * p.hq), b = (int)(row / p.stride), r = (int)(row - (int64_t)b * p.stride);
    const int S = __ldcg(p.S + b), n = min(__ldcg(p.n + b), p.stride), g = p.hq / p.hkv;
    if (r >= n || S < 0 || (int64_t)S + n > p.max_ctx) return;
    const int q_end = min(((r * g + head % g) / p.tile_rows + 1) * p.tile_rows, n * g);
    const int nsplit = (S + (q_end - 1) / g) / p.chunk + 1;
    if (nsplit <= 1) return;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (32 * warp < nsplit) join_range(p, at, 32 * warp, nsplit, lane, m, l, acc);
    s_acc[warp][lane] = acc;
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp > 0) return;
    const int parts = blockDim.x >> 5;
    for (int w = 0; w < parts; ++w) m = fmaxf(m, s_ml[w].x);
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < parts; ++w) {
        const float f = s_ml[w].x == -INFINITY ? 0.f : exp2_fast(s_ml[w].x - m);
        const float4 v = s_acc[w][lane];
        l += f * s_ml[w].y;
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
    }
    store_out(p, at, lane, acc, out_factor(p.v_scale, l));
}

// ---------------------------------------------------------------------------
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

struct AttnKv4Plan {
    int tile_rows, chunk, max_splits, tiles, sms;
    bool ticketed;  // chunks are joined by the one that finishes last
    size_t off_ticket, off_ml, off_o, bytes;
};

bool plan_attn_kv4(int n_seq, int stride, int hq, int hkv, int max_ctx, AttnKv4Plan* w) {
    if (n_seq < 1 || stride < 1 || stride > 1024 || hq < 1 || hkv < 1 || hq % hkv || hq / hkv > 128 || max_ctx < 1)
        return false;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    w->sms = sms;
    // Tiles of 8 or 16 query rows (kv4.cu), of 128 or 256 (kv4_tc.cu): the
    // smallest that holds a sequence's.
    const int rows = stride * (hq / hkv);
    w->tile_rows = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 128 ? 128 : 256;
    w->tiles = (rows + w->tile_rows - 1) / w->tile_rows;
    const bool tc = w->tile_rows > 16;
    // Chunks by the call's capacity alone (a sequence's result does not depend on
    // its neighbours' lengths).
    const int64_t pairs = (int64_t)n_seq * hkv * w->tiles;
    int64_t chunk;
    if (tc) {
        // The number of chunks whose rounds of items (one CTA an SM) cost the least,
        // averaged over sequences at the capacity and at half of it: an item costs
        // its 128-key blocks and about two more to start and end, the chunks' joining
        // about half a block for every 64 MB of partial results.
        double best = 0.;
        chunk = 0;
        for (int s = 1; s <= kMaxSplits; ++s) {
            const int64_t c = ((int64_t)max_ctx + 128LL * s - 1) / (128LL * s) * 128;
            double cost = s > 1 ? 2. + (double)pairs * std::min(rows, w->tile_rows) * s * 512. / (128 << 20) : 0.;
            for (int half = 0; half < 2; ++half) {
                const int64_t len = std::max(1, half ? max_ctx / 2 : max_ctx);
                const int64_t items = pairs * ((len + c - 1) / c);
                cost += (double)((items + sms - 1) / sms) * (double)((std::min(c, len) + 127) / 128 + 2);
            }
            if (chunk == 0 || cost < best) {
                best = cost;
                chunk = c;
            }
            if (c <= 256) break;
        }
    } else {
        // Some items (warps) for every SM when the sequences are at half the capacity, 64 to 1024 keys.
        const int64_t keys = pairs * std::max(1, max_ctx / 2), items = (int64_t)kItemsPerSm * sms;
        chunk = std::max<int64_t>(64, std::min<int64_t>(1024, ((keys + items - 1) / items + 63) / 64 * 64));
        chunk = std::max<int64_t>(chunk, ((int64_t)max_ctx + 64LL * kMaxSplits - 1) / (64LL * kMaxSplits) * 64);
    }
    w->chunk = (int)std::min<int64_t>(chunk, 1 << 30);
    w->max_splits = (int)(((int64_t)max_ctx + w->chunk - 1) / w->chunk);
    const size_t parts = w->max_splits > 1 ? (size_t)n_seq * stride * hq * w->max_splits : 0;
    w->off_ticket = 256;
    w->ticketed = !tc && w->max_splits > 1 && w->max_splits <= kTicketSplits && pairs <= kTickets;
    w->off_ml = w->off_ticket + kTickets * sizeof(unsigned);
    w->off_o = w->off_ml + round256(parts * sizeof(float2));
    w->bytes = w->off_o + round256(parts * HD * sizeof(float));
    return pairs * w->max_splits <= INT32_MAX && (int64_t)n_seq * stride * hq <= INT32_MAX;
}

bool valid_scale(float x) {
    int e;
    return std::isfinite(x) && x > 0.f && std::frexp(x, &e) == 0.5f && e >= -58 && e <= 59;  // 2^-59 to 2^58
}

wedlm_status rows_params(RowsParams* p, const void* k, const void* v, int32_t dtype, int64_t k_stride,
                         int64_t v_stride, void* pool, int32_t num_pages, int32_t hkv, const int32_t* table,
                         int32_t pages_per_seq, const int32_t* S, const int32_t* n, int32_t n_seq, int32_t stride,
                         float k_scale, float v_scale, void* err) {
    if (n_seq < 0 || stride < 1 || hkv < 1 || num_pages < 1 || pages_per_seq < 1) return WEDLM_ERR_INVALID_ARG;
    if (dtype != WEDLM_DTYPE_F32 && dtype != WEDLM_DTYPE_BF16) return WEDLM_ERR_UNSUPPORTED;
    if (!valid_scale(k_scale) || !valid_scale(v_scale)) return WEDLM_ERR_INVALID_ARG;
    const int vec = dtype == WEDLM_DTYPE_F32 ? 4 : 8;
    if (k_stride < (int64_t)hkv * HD || v_stride < (int64_t)hkv * HD || k_stride % vec || v_stride % vec)
        return WEDLM_ERR_INVALID_ARG;
    if (n_seq > 0 && (!k || !v || !pool || !table || !S || !n || !err)) return WEDLM_ERR_INVALID_ARG;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)pool) & 15) return WEDLM_ERR_INVALID_ARG;
    if (((uintptr_t)table | (uintptr_t)S | (uintptr_t)n | (uintptr_t)err) & 3) return WEDLM_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)n_seq * stride;
    if (rows > INT32_MAX || hkv > 65535) return WEDLM_ERR_INVALID_ARG;
    *p = RowsParams{static_cast<uint8_t*>(pool), table, S, n, static_cast<int*>(err), rows, k_stride,
                    v_stride, num_pages, hkv, pages_per_seq, stride, k_scale, v_scale};
    // by = ceil(2^shift / stride), 2^(shift - 32) < stride <= 2^(shift - 31): by < 2^32, and x (by stride - 2^shift) < 2^shift
    p->shift = 31;
    while ((1ll << (p->shift - 31)) < stride) ++p->shift;
    p->by = (uint32_t)(((1ull << p->shift) + (uint64_t)stride - 1) / (uint64_t)stride);
    p->wide = !(((uintptr_t)k | (uintptr_t)v) & 31) && k_stride % (2 * vec) == 0 && v_stride % (2 * vec) == 0;
    return WEDLM_OK;
}

}  // namespace
}  // namespace wedlm

using namespace wedlm;

extern "C" {

wedlm_status wedlm_kv4_append(const void* k, const void* v, int32_t dtype, int64_t k_stride, int64_t v_stride,
                              void* kv4_pool, int32_t num_pages, int32_t n_kv_heads, const int32_t* page_table,
                              int32_t pages_per_seq, const int32_t* S, const int32_t* n, int32_t n_seq,
                              int32_t stride, float k_scale, float v_scale, void* error_word, void* stream) {
    RowsParams p;
    const wedlm_status s = rows_params(&p, k, v, dtype, k_stride, v_stride, kv4_pool, num_pages, n_kv_heads, page_table,
                                       pages_per_seq, S, n, n_seq, stride, k_scale, v_scale, error_word);
    if (s || p.rows == 0) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == WEDLM_DTYPE_F32 ? launch_append<float>(p, k, v, st) : launch_append<bf16>(p, k, v, st);
    return e == cudaSuccess ? WEDLM_OK : WEDLM_ERR_CUDA;
}

wedlm_status wedlm_kv4_read(const void* kv4_pool, int32_t num_pages, int32_t n_kv_heads, const int32_t* page_table,
                            int32_t pages_per_seq, const int32_t* S, const int32_t* n, int32_t n_seq, int32_t stride,
                            float k_scale, float v_scale, void* k, void* v, int32_t dtype, int64_t k_stride,
                            int64_t v_stride, void* error_word, void* stream) {
    RowsParams p;
    const wedlm_status s = rows_params(&p, k, v, dtype, k_stride, v_stride, const_cast<void*>(kv4_pool), num_pages,
                                       n_kv_heads, page_table, pages_per_seq, S, n, n_seq, stride, k_scale, v_scale,
                                       error_word);
    if (s || p.rows == 0) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == WEDLM_DTYPE_F32 ? launch_read<float>(p, k, v, st) : launch_read<bf16>(p, k, v, st);
    return e == cudaSuccess ? WEDLM_OK : WEDLM_ERR_CUDA;
}

wedlm_status wedlm_attention_kv4_workspace_bytes(int32_t n_seq, int32_t stride, int32_t n_heads, int32_t n_kv_heads,
                                                 int32_t max_ctx, int64_t* bytes) {
    AttnKv4Plan w;
    if (!bytes || !plan_attn_kv4(n_seq, stride, n_heads, n_kv_heads, max_ctx, &w)) return WEDLM_ERR_INVALID_ARG;
    *bytes = (int64_t)w.bytes;
    return WEDLM_OK;
}

wedlm_status wedlm_attention_kv4(const void* q, const void* kv4_pool, int32_t num_pages, int32_t n_heads,
                                 int32_t n_kv_heads, const int32_t* page_table, int32_t pages_per_seq,
                                 const int32_t* S, const int32_t* n, int32_t n_seq, int32_t stride, int32_t max_ctx,
                                 float k_scale, float v_scale, void* out, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
    AttnKv4Plan w;
    if (!plan_attn_kv4(n_seq, stride, n_heads, n_kv_heads, max_ctx, &w)) return WEDLM_ERR_INVALID_ARG;
    if (!q || !kv4_pool || !page_table || !S || !n || !out || !workspace || num_pages < 1 || pages_per_seq < 1)
        return WEDLM_ERR_INVALID_ARG;
    if (!valid_scale(k_scale) || !valid_scale(v_scale)) return WEDLM_ERR_INVALID_ARG;
    if (workspace_bytes < (int64_t)w.bytes || ((uintptr_t)workspace & 255)) return WEDLM_ERR_INVALID_ARG;
    if ((((uintptr_t)q | (uintptr_t)kv4_pool) & 15) || ((uintptr_t)out & 31)) return WEDLM_ERR_INVALID_ARG;
    if (((uintptr_t)page_table | (uintptr_t)S | (uintptr_t)n) & 3) return WEDLM_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    cudaStream_t st = (cudaStream_t)stream;
    const AttnKv4Params p{(const bf16*)q, (const uint8_t*)kv4_pool, page_table, S, n, (bf16*)out,
                          (float*)(ws + w.off_o), (float2*)(ws + w.off_ml),
                          w.ticketed ? (unsigned*)(ws + w.off_ticket) : nullptr, (int*)ws, num_pages, n_heads,
                          n_kv_heads, pages_per_seq, n_seq, stride, max_ctx, w.chunk, w.max_splits, w.tile_rows,
                          w.tiles, k_scale, v_scale};
    const bool tc = w.tile_rows > 16;
    const dim3 grid((unsigned)((int64_t)n_seq * n_kv_heads * w.tiles * w.max_splits));
    cudaError_t e = tc                  ? launch_attn_kv4_tc(p, w.sms, st)
                    : w.tile_rows == 8 ? launch_pdl(attn_kv4_kernel<1>, grid, dim3(32), 0, st, p)
                                       : launch_pdl(attn_kv4_kernel<2>, grid, dim3(32), 0, st, p);
    if (e == cudaSuccess && w.max_splits > 1 && !w.ticketed)
        e = launch_pdl(attn_kv4_join_kernel, dim3((unsigned)((int64_t)n_seq * stride * n_heads)),
                       dim3((w.max_splits + 31) / 32 * 32), 0, st, p);
    return e == cudaSuccess ? WEDLM_OK : WEDLM_ERR_CUDA;
}

}  // extern "C"
