// Page operations of a paged KV cache: copy, reserve, fork, free and compact,
// for pages of any format (the engine's bf16 or fp32 pages, the 4-bit pages of
// kv4.cu).  Page tables, committed lengths and reference counts live on the
// device, and every decision (which pages are free, which move where) is taken
// there, so the calls need no host round trip and can be captured in a graph.
//
// A call is a plan by one CTA (free: a CTA for each sequence), whose work is a few
// integers per listed sequence plus a scan of the reference counts that stops
// once enough free pages are found, and where pages are copied a kernel that does
// it with the whole GPU.  All results are integers or copied bytes and do not
// depend on the order in which threads run: free pages are taken in ascending
// order and handed out in list order.
//
// The kernels wait for the kernel before them before they read anything and
// never let the kernel after them start early: kernels of the decode step read
// page tables, lengths and cached keys (by TMA) before their own dependency wait
// (settle_writes in common.cuh).
//
// A plan is a chain of dependent reads, each a trip to L2 (some 0.7 us) whatever
// its size: its lists lie in shared memory where they fit, the first reference
// counts are read at the start, and what needs no decision (the table rows of a
// fork) is left to the copy.  Freeing 64 branches, forking 8 sequences eightfold
// (28 layers, 57 MB copied) and reserving for them: 30.6 us in a graph, with every
// list in global memory 47; three branches of a small cache: 12.4, and 17.4.
#include <algorithm>

#include "kernels.cuh"

namespace wedlm {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanShared = 2048;  // entries of a list that a plan keeps in shared memory
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 4;  // 16-byte vectors per thread in flight
constexpr int kShareRun = 128;  // pages that a warp shares at a time
constexpr int64_t kAloneBytes = 64 << 10;  // what the plan of a copy moves by itself

// Workspace: [0] the error word, [1] the number of planned copies, then the
// copies (source, destination), one int per page (free pages, marks or the
// map of a compaction) and three ints per sequence (marks, offsets, a value).
struct PagesWs {
    int* err;
    int* count;
    int2* pairs;
    int* list;
    int* mark;
    int* off;
    int* val;
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

size_t pages_ws_bytes(int32_t num_pages, int32_t n_seq) {
    return 256 + round256((size_t)num_pages * sizeof(int2)) + round256((size_t)num_pages * 4) +
           3 * round256((size_t)n_seq * 4);
}

PagesWs pages_ws(void* ws, int32_t num_pages, int32_t n_seq) {
    char* c = static_cast<char*>(ws);
    PagesWs w;
    w.err = reinterpret_cast<int*>(c);
    w.count = w.err + 1;
    c += 256;
    w.pairs = reinterpret_cast<int2*>(c);
    c += round256((size_t)num_pages * sizeof(int2));
    w.list = reinterpret_cast<int*>(c);
    c += round256((size_t)num_pages * 4);
    w.mark = reinterpret_cast<int*>(c);
    c += round256((size_t)n_seq * 4);
    w.off = reinterpret_cast<int*>(c);
    c += round256((size_t)n_seq * 4);
    w.val = reinterpret_cast<int*>(c);
    return w;
}

// Exclusive prefix sum over the CTA's threads; *total receives the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
    __shared__ int part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    __syncthreads();  // part[] of the call before has been read
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int p = lane < nw ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p += u;
    }
    *total = __shfl_sync(0xffffffffu, p, 31);
    const int before = __shfl_sync(0xffffffffu, p, (warp + 31) & 31);
    return x - v + (warp ? before : 0);
}

// Four consecutive reference counts from page i on; pages past the end read `past`.
__device__ __forceinline__ void load_refs(const int32_t* refs, int64_t i, int num_pages, int past, int (&r)[4]) {
    if (i + 4 <= num_pages) {
        const int4 v = __ldcg(reinterpret_cast<const int4*>(refs + i));
        r[0] = v.x;
        r[1] = v.y;
        r[2] = v.z;
        r[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = i + k < num_pages ? __ldcg(refs + i + k) : past;
    }
}

// The `want` lowest pages without a reference, ascending, into list[]; returns
// how many there are (at most want).  Stops scanning once it has them.
// `r` holds the thread's counts of the first 4 kPlanThreads pages.
__device__ int find_free(const int32_t* refs, int num_pages, int want, int* list, int (&r)[4]) {
    int have = 0;
    for (int64_t i0 = 0; i0 < num_pages && have < want; i0 += 4 * kPlanThreads) {
        const int64_t i = i0 + 4 * threadIdx.x;
        if (i0 > 0) load_refs(refs, i, num_pages, 1, r);
        int c = 0, total;
#pragma unroll
        for (int k = 0; k < 4; ++k) c += r[k] == 0;
        int at = have + block_scan(c, &total);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r[k] == 0) {
                if (at < want) list[at] = (int)(i + k);
                ++at;
            }
        have += total;
    }
    return min(have, want);
}

// off[i] (the pages entry i asks for) to exclusive prefix sums; returns the total.
__device__ int scan_needs(int* off, int n) {
    int64_t base = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const int v = i < n ? off[i] : 0;
        int total;
        const int at = block_scan(v, &total);
        if (i < n) off[i] = (int)min((int64_t)INT32_MAX, base + at);
        base += total;
    }
    return (int)min((int64_t)INT32_MAX, base);
}

// What a plan leaves to be done.
struct MoveArgs {
    const int2* pairs;
    const int* count;
    int* err;
    const int32_t* map;                 // a compaction: new ids, or nullptr
    const int32_t *parents, *children;  // a fork of n entries (n = 0: none)
    const int* full;                    // the pages each of them shares, -1: none
    int n;
};

// A compaction's page tables renamed, or a fork's full pages shared, by CTA `cta` of `ctas`.
__device__ void move_tables(const wedlm_kv_pages& p, const MoveArgs& w, int cta, int ctas) {
    if (w.map) {
        const int64_t entries = (int64_t)p.n_seq * p.pages_per_seq;
        for (int64_t e = (int64_t)cta * blockDim.x + threadIdx.x; e < entries; e += (int64_t)ctas * blockDim.x) {
            const int page = __ldcg(p.page_table + e);
            if (page == -1) continue;
            const int to = page >= 0 && page < p.num_pages ? __ldcg(w.map + page) : -1;
            if (to < 0) set_error(w.err, kErrBounds);  // not a page in use: left as it is
            else if (to != page) p.page_table[e] = to;
        }
    }
    // (a warp for every kShareRun pages of an entry)
    const int64_t warps = blockDim.x / 32, runs = (p.pages_per_seq + kShareRun - 1) / kShareRun;
    for (int64_t u = cta * warps + (threadIdx.x >> 5); u < w.n * runs; u += ctas * warps) {
        const int i = (int)(u / runs), j0 = (int)(u - i * runs) * kShareRun + (threadIdx.x & 31);
        const int full = __ldcg(w.full + i), a = __ldcg(w.parents + i), c = __ldcg(w.children + i);
        if (j0 >= full) continue;
        const int32_t* from = p.page_table + (int64_t)a * p.pages_per_seq;
        int32_t* to = p.page_table + (int64_t)c * p.pages_per_seq;
        int page[kShareRun / 32];
#pragma unroll
        for (int k = 0; k < kShareRun / 32; ++k) page[k] = j0 + 32 * k < full ? __ldcg(from + j0 + 32 * k) : -1;
#pragma unroll
        for (int k = 0; k < kShareRun / 32; ++k)
            if (page[k] >= 0) {
                to[j0 + 32 * k] = page[k];
                atomicAdd(p.refs + page[k], 1);
            }
    }
}

// The planned copies in every layer, 16 KB of a page at a time, after the tables.
// Bound by HBM: each byte is read and written once.
__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(wedlm_kv_pages p, MoveArgs w) {
    griddep_wait();
    move_tables(p, w, blockIdx.x, gridDim.x);
    const int64_t nvec = p.page_bytes / 16;
    const int64_t chunks = (nvec + kCopyThreads * kCopyVec - 1) / (kCopyThreads * kCopyVec);
    const int64_t per_pair = chunks * p.n_layers, units = per_pair * __ldcg(w.count);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t k = u / per_pair, rest = u - k * per_pair;
        const int64_t layer = rest / chunks, v0 = (rest - layer * chunks) * (kCopyThreads * kCopyVec) + threadIdx.x;
        const int2 m = __ldcg(w.pairs + k);
        char* base = static_cast<char*>(p.pool) + layer * p.layer_stride;
        const int4* from = reinterpret_cast<const int4*>(base + (int64_t)m.x * p.page_bytes);
        int4* to = reinterpret_cast<int4*>(base + (int64_t)m.y * p.page_bytes);
        int4 v[kCopyVec];
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (v0 + j * kCopyThreads < nvec) v[j] = __ldcg(from + v0 + j * kCopyThreads);
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (v0 + j * kCopyThreads < nvec) to[v0 + j * kCopyThreads] = v[j];
    }
    settle_writes();
}

// The copies by the plan's own CTA: the vectors of all pages in one row, so that
// small pages keep every thread busy.  All threads call it.
__device__ void move_alone(const wedlm_kv_pages& p, const PagesWs& w) {
    __syncthreads();
    const uint32_t nvec = (uint32_t)(p.page_bytes / 16), per_pair = nvec * p.n_layers, all = per_pair * __ldcg(w.count);
    for (uint32_t i0 = threadIdx.x; i0 < all; i0 += kPlanThreads * kCopyVec) {
        int4 v[kCopyVec];
        int4* to[kCopyVec];
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j) {
            const uint32_t i = i0 + j * kPlanThreads;
            to[j] = nullptr;
            if (i >= all) continue;
            const uint32_t k = i / per_pair, rest = i - k * per_pair, layer = rest / nvec, at = rest - layer * nvec;
            const int2 m = __ldcg(w.pairs + k);
            int4* base = reinterpret_cast<int4*>(static_cast<char*>(p.pool) + layer * p.layer_stride) + at;
            v[j] = __ldcg(base + (int64_t)m.x * nvec);
            to[j] = base + (int64_t)m.y * nvec;
        }
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (to[j]) *to[j] = v[j];
    }
    settle_writes();
}

__global__ void __launch_bounds__(kPlanThreads) pages_copy_plan_kernel(const int32_t* src, const int32_t* dst, int n,
                                                                       wedlm_kv_pages p, bool alone, PagesWs w) {
    griddep_wait();
    const int num_pages = p.num_pages;
    __shared__ int cnt;
    if (threadIdx.x == 0) cnt = 0;
    auto ok = [&](int i, int& s, int& d) {
        s = __ldcg(src + i);
        d = __ldcg(dst + i);
        return s >= 0 && s < num_pages && d >= 0 && d < num_pages;
    };
    // Marks of the listed pages: low bits count the entries that write a page,
    // bit 30 says that one reads it.
    int s, d;
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (ok(i, s, d)) w.list[s] = w.list[d] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (ok(i, s, d)) {
            atomicOr(&w.list[s], 1 << 30);
            atomicAdd(&w.list[d], 1);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        if (ok(i, s, d) && __ldcg(&w.list[d]) == 1)
            w.pairs[atomicAdd(&cnt, 1)] = make_int2(s, d);
        else
            set_error(w.err, kErrBounds);
    }
    __syncthreads();
    if (threadIdx.x == 0) *w.count = cnt;
    if (alone) move_alone(p, w);
}

// Lists of a plan with n entries over n_seq sequences: two values an entry, what
// it asks for, marks of the sequences.
struct PlanLists {
    int val[2][kPlanShared], off[kPlanShared], mark[kPlanShared];
};

__global__ void __launch_bounds__(kPlanThreads) pages_reserve_kernel(const int32_t* seqs, const int32_t* tokens, int n,
                                                                     wedlm_kv_pages p, PagesWs w) {
    griddep_wait();
    extern __shared__ __align__(16) char smem[];
    PlanLists& t = *reinterpret_cast<PlanLists*>(smem);
    const bool small = p.n_seq <= kPlanShared;  // (n <= n_seq)
    int* mark = small ? t.mark : w.mark;
    int* off = small ? t.off : w.off;
    int* held_by = small ? t.val[0] : w.val;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int refs[4];
    load_refs(p.refs, 4 * threadIdx.x, p.num_pages, 1, refs);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int q = __ldcg(seqs + i);
        if (q >= 0 && q < p.n_seq) mark[q] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int q = __ldcg(seqs + i);
        if (q >= 0 && q < p.n_seq) atomicAdd(&mark[q], 1);
    }
    __syncthreads();
    // The pages each entry asks for.
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int q = __ldcg(seqs + i), tok = __ldcg(tokens + i);
        bool ok = q >= 0 && q < p.n_seq && tok >= 0 && (int64_t)tok <= (int64_t)p.pages_per_seq * kPage;
        if (ok) ok = mark[q] == 1;
        int need = 0, held = 0;
        if (ok) {
            const int32_t* row = p.page_table + (int64_t)q * p.pages_per_seq;
            int first = p.pages_per_seq;
#pragma unroll 4
            for (int j = lane; j < p.pages_per_seq; j += 32) {
                if (__ldcg(row + j) >= 0) ++held;
                else first = min(first, j);
            }
            held = __reduce_add_sync(0xffffffffu, held);
            first = __reduce_min_sync(0xffffffffu, first);
            ok = held == first;  // no place empty before one that is taken
            need = max(0, (tok + kPage - 1) / kPage - held);
        }
        if (lane == 0) {
            if (!ok) set_error(w.err, kErrBounds);
            off[i] = ok ? need : 0;
            held_by[i] = held;
        }
    }
    __syncthreads();
    const int total = scan_needs(off, n);
    int* list = total <= kPlanShared ? t.val[1] : w.list;
    const int have = find_free(p.refs, p.num_pages, total, list, refs);
    __syncthreads();
    if (have < total) {
        if (threadIdx.x == 0) set_error(w.err, kErrPages);
        return;
    }
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int at = off[i], need = (i + 1 < n ? off[i + 1] : total) - at;
        if (need == 0) continue;
        int32_t* row = p.page_table + (int64_t)__ldcg(seqs + i) * p.pages_per_seq + held_by[i];
        for (int j = lane; j < need; j += 32) {
            const int page = list[at + j];
            row[j] = page;
            p.refs[page] = 1;
        }
    }
    settle_writes();
}

// Leaves in w.val[i] the full pages that child i is to share with its parent,
// or -1 for an entry that is not served: the copy kernel fills those in.
__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(const int32_t* parents, const int32_t* children,
                                                                       int n, wedlm_kv_pages p, PagesWs w) {
    griddep_wait();
    extern __shared__ __align__(16) char smem[];
    PlanLists& t = *reinterpret_cast<PlanLists*>(smem);
    const bool small = p.n_seq <= kPlanShared;  // (n <= n_seq)
    int* mark = small ? t.mark : w.mark;
    int* off = small ? t.off : w.off;
    int* len = small ? t.val[0] : w.val;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int refs[4];
    load_refs(p.refs, 4 * threadIdx.x, p.num_pages, 1, refs);
    auto in = [&](int q) { return q >= 0 && q < p.n_seq; };
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int a = __ldcg(parents + i), c = __ldcg(children + i);
        if (in(a)) mark[a] = 0;
        if (in(c)) mark[c] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int a = __ldcg(parents + i), c = __ldcg(children + i);
        len[i] = in(a) ? __ldcg(p.S + a) : -1;
        if (in(a)) atomicOr(&mark[a], 1 << 30);
        if (in(c)) atomicAdd(&mark[c], 1);
    }
    __syncthreads();
    // len[i]: the tokens entry i shares, -1 when it cannot be served; off[i]: 1 when
    // it needs a page of its own, for the parent's last page that is not full.
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int a = __ldcg(parents + i), c = __ldcg(children + i), L = len[i];
        bool ok = in(a) && in(c) && L >= 0 && (int64_t)L <= (int64_t)p.pages_per_seq * kPage;
        if (ok) ok = mark[c] == 1;
        if (ok) {
            const int32_t* row = p.page_table + (int64_t)a * p.pages_per_seq;
            const int32_t* own = p.page_table + (int64_t)c * p.pages_per_seq;
            const int pages = (L + kPage - 1) / kPage;
            for (int j0 = lane; j0 < p.pages_per_seq; j0 += 128) {
                int page[4], count[4], mine[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = j0 + 32 * k;
                    page[k] = j < pages ? __ldcg(row + j) : 0;
                    mine[k] = j < p.pages_per_seq ? __ldcg(own + j) : -1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    ok = ok && page[k] >= 0 && page[k] < p.num_pages && mine[k] < 0;
                    count[k] = ok && j0 + 32 * k < pages ? __ldcg(p.refs + page[k]) : 1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) ok = ok && count[k] > 0;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) {
            if (!ok) {
                set_error(w.err, kErrBounds);
                len[i] = -1;
            }
            off[i] = ok ? (L % kPage != 0) : 0;
        }
    }
    __syncthreads();
    const int total = scan_needs(off, n);
    int* list = total <= kPlanShared ? t.val[1] : w.list;
    const int have = find_free(p.refs, p.num_pages, total, list, refs);
    __syncthreads();
    if (threadIdx.x == 0) {
        *w.count = have < total ? 0 : total;
        if (have < total) set_error(w.err, kErrPages);
    }
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int L = have < total ? -1 : len[i];
        w.val[i] = L < 0 ? -1 : L / kPage;
        if (L < 0) continue;
        const int a = __ldcg(parents + i), c = __ldcg(children + i);
        p.S[c] = L;
        if (L % kPage) {
            const int at = off[i], page = list[at];
            const int64_t place = L / kPage;
            w.pairs[at] = make_int2(__ldcg(p.page_table + (int64_t)a * p.pages_per_seq + place), page);
            p.page_table[(int64_t)c * p.pages_per_seq + place] = page;
            p.refs[page] = 1;
        }
    }
}

// One CTA per listed sequence.  A sequence listed twice is freed once: each
// place of its table row is taken by one exchange.
__global__ void __launch_bounds__(128) pages_free_kernel(const int32_t* seqs, wedlm_kv_pages p, int* err) {
    griddep_wait();
    const int q = __ldcg(seqs + blockIdx.x);
    if (q < 0 || q >= p.n_seq) {
        if (threadIdx.x == 0) set_error(err, kErrBounds);
        return;
    }
    int32_t* row = p.page_table + (int64_t)q * p.pages_per_seq;
    for (int j = threadIdx.x; j < p.pages_per_seq; j += 128) {
        if (__ldcg(row + j) == -1) continue;
        const int page = atomicExch(row + j, -1);
        if (page == -1) continue;
        if (page < 0 || page >= p.num_pages) {
            set_error(err, kErrBounds);
        } else if (atomicSub(p.refs + page, 1) <= 0) {  // held by nobody
            atomicAdd(p.refs + page, 1);
            set_error(err, kErrBounds);
        }
    }
    if (threadIdx.x == 0) p.S[q] = 0;
    settle_writes();
}

// Used pages move to the lowest ids: with u pages in use, the k-th used page at
// or past u moves into the k-th unused one below u (there are as many of both).
__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(wedlm_kv_pages p, int32_t* map, PagesWs w) {
    griddep_wait();
    int used = 0, total;
    for (int64_t i = 4 * threadIdx.x; i < p.num_pages; i += 4 * kPlanThreads) {
        int r[4];
        load_refs(p.refs, i, p.num_pages, 0, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) used += r[k] > 0;
    }
    block_scan(used, &total);
    const int u = total;
    // Holes below u and movers from u on are counted by one running number:
    // every hole comes before every mover.
    int below = 0;
    for (int64_t i = 4 * threadIdx.x; i < u; i += 4 * kPlanThreads) {
        int r[4];
        load_refs(p.refs, i, p.num_pages, 0, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) below += r[k] <= 0 && i + k < u;
    }
    block_scan(below, &total);
    const int moves = total;
    int base = 0;
    for (int64_t i0 = 0; i0 < p.num_pages; i0 += 4 * kPlanThreads) {
        const int64_t i = i0 + 4 * threadIdx.x;
        int r[4], c = 0;
        load_refs(p.refs, i, p.num_pages, 0, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) c += (i + k < u) != (r[k] > 0);
        int at = base + block_scan(c, &total);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (i + k >= p.num_pages) break;
            if ((i + k < u) != (r[k] > 0)) {
                if (at < moves) w.pairs[at].y = (int)(i + k);
                else w.pairs[at - moves].x = (int)(i + k);
                ++at;
            }
            map[i + k] = r[k] > 0 ? (int)(i + k) : -1;
        }
        base += total;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < moves; k += kPlanThreads) {
        const int2 m = w.pairs[k];
        map[m.x] = m.y;
        p.refs[m.y] = __ldcg(p.refs + m.x);
        p.refs[m.x] = 0;
    }
    if (threadIdx.x == 0) *w.count = moves;
}

// most: how many copies there can be.
cudaError_t launch_move(const wedlm_kv_pages& p, const MoveArgs& a, int64_t most, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t chunks = (p.page_bytes / 16 + kCopyThreads * kCopyVec - 1) / (kCopyThreads * kCopyVec);
    int64_t units = most * p.n_layers * chunks;
    if (a.map) units = std::max(units, ((int64_t)p.n_seq * p.pages_per_seq + kCopyThreads - 1) / kCopyThreads);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(units, (int64_t)sms * 8));
    return launch_pdl(pages_move_kernel, dim3((unsigned)grid), dim3(kCopyThreads), 0, st, p, a);
}

// A description that the kernels can follow without leaving its buffers.
bool pages_ok(const wedlm_kv_pages* p, const void* ws, int64_t ws_bytes) {
    if (!p || !ws || !p->pool || !p->page_table || !p->S || !p->refs) return false;
    if (p->n_layers < 1 || p->num_pages < 1 || p->n_seq < 1 || p->pages_per_seq < 1) return false;
    // positions and the table's entries (so the pages that one call can ask for, too) fit 32 bits
    if (p->pages_per_seq > INT32_MAX / kPage || p->n_seq > INT32_MAX / p->pages_per_seq) return false;
    if (p->page_bytes < 16 || p->page_bytes % 16 || p->layer_stride % 16) return false;
    if (p->page_bytes > (INT64_MAX / 2) / p->num_pages) return false;
    if (p->n_layers > 1 && p->layer_stride < p->page_bytes * p->num_pages) return false;
    if (((uintptr_t)p->pool | (uintptr_t)p->refs) & 15) return false;
    if (((uintptr_t)p->page_table | (uintptr_t)p->S) & 3) return false;
    return !((uintptr_t)ws & 255) && ws_bytes >= (int64_t)pages_ws_bytes(p->num_pages, p->n_seq);
}

wedlm_status done(cudaError_t e) { return e == cudaSuccess ? WEDLM_OK : WEDLM_ERR_CUDA; }

}  // namespace
}  // namespace wedlm

using namespace wedlm;

extern "C" {

wedlm_status wedlm_kv_pages_workspace_bytes(int32_t num_pages, int32_t n_seq, int64_t* bytes) {
    if (!bytes || num_pages < 1 || n_seq < 1) return WEDLM_ERR_INVALID_ARG;
    *bytes = (int64_t)pages_ws_bytes(num_pages, n_seq);
    return WEDLM_OK;
}

wedlm_status wedlm_kv_pages_copy(const wedlm_kv_pages* pages, const int32_t* src, const int32_t* dst, int32_t n,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes) || n < 0 || n > pages->num_pages) return WEDLM_ERR_INVALID_ARG;
    if (n == 0) return WEDLM_OK;
    if (!src || !dst) return WEDLM_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const PagesWs w = pages_ws(workspace, pages->num_pages, pages->n_seq);
    // Little is copied by the plan itself, which saves a launch: us eagerly (in a captured
    // graph) for 16 KB 4.9 (4.1), with a second kernel 7.1 (4.9); 48 KB 5.1 (4.9) and 7.3
    // (4.5); 64 KB 6.0 (5.9) and 7.1 (4.7); 128 KB 8.0 (7.9) and 7.2 (4.8).
    const bool alone = pages->page_bytes <= kAloneBytes && n <= kAloneBytes / pages->page_bytes / pages->n_layers;
    cudaError_t e = launch_pdl(pages_copy_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, src, dst, n, *pages, alone, w);
    if (e == cudaSuccess && !alone)
        e = launch_move(*pages, {w.pairs, w.count, w.err, nullptr, nullptr, nullptr, nullptr, 0}, n, st);
    return done(e);
}

wedlm_status wedlm_kv_pages_reserve(const wedlm_kv_pages* pages, const int32_t* seqs, const int32_t* tokens, int32_t n,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes) || n < 0 || n > pages->n_seq) return WEDLM_ERR_INVALID_ARG;
    if (n == 0) return WEDLM_OK;
    if (!seqs || !tokens) return WEDLM_ERR_INVALID_ARG;
    const PagesWs w = pages_ws(workspace, pages->num_pages, pages->n_seq);
    return done(launch_pdl(pages_reserve_kernel, dim3(1), dim3(kPlanThreads), sizeof(PlanLists), (cudaStream_t)stream, seqs,
                           tokens, n, *pages, w));
}

wedlm_status wedlm_kv_pages_fork(const wedlm_kv_pages* pages, const int32_t* parents, const int32_t* children,
                                 int32_t n, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes) || n < 0 || n > pages->n_seq) return WEDLM_ERR_INVALID_ARG;
    if (n == 0) return WEDLM_OK;
    if (!parents || !children) return WEDLM_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const PagesWs w = pages_ws(workspace, pages->num_pages, pages->n_seq);
    cudaError_t e = launch_pdl(pages_fork_plan_kernel, dim3(1), dim3(kPlanThreads), sizeof(PlanLists), st, parents,
                               children, n, *pages, w);
    if (e == cudaSuccess) e = launch_move(*pages, {w.pairs, w.count, w.err, nullptr, parents, children, w.val, n}, n, st);
    return done(e);
}

wedlm_status wedlm_kv_pages_free(const wedlm_kv_pages* pages, const int32_t* seqs, int32_t n, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes) || n < 0 || n > pages->n_seq) return WEDLM_ERR_INVALID_ARG;
    if (n == 0) return WEDLM_OK;
    if (!seqs) return WEDLM_ERR_INVALID_ARG;
    return done(launch_pdl(pages_free_kernel, dim3((unsigned)n), dim3(128), 0, (cudaStream_t)stream, seqs, *pages,
                           static_cast<int*>(workspace)));
}

wedlm_status wedlm_kv_pages_compact(const wedlm_kv_pages* pages, int32_t* map, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes)) return WEDLM_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const PagesWs w = pages_ws(workspace, pages->num_pages, pages->n_seq);
    int32_t* m = map ? map : w.list;
    cudaError_t e = launch_pdl(pages_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, *pages, m, w);
    if (e == cudaSuccess)
        e = launch_move(*pages, {w.pairs, w.count, w.err, m, nullptr, nullptr, nullptr, 0}, pages->num_pages / 2, st);
    return done(e);
}

}  // extern "C"
