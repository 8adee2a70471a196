// Page operations of a paged KV cache: copy, reserve, fork, free and compact,
// for pages of any format (the engine's bf16 or fp32 pages, the 4-bit pages of
// kv4.cu).  Page tables, committed lengths and reference counts live on the
// device, and every decision (which pages are free, which move where) is taken
// there, so the calls need no host round trip and can be captured in a graph.
//
// Each call but free is two kernels: a plan by one CTA, whose work is a few
// integers per listed sequence plus a scan of the reference counts that stops
// once enough free pages are found, and a copy of the planned pages by the
// whole GPU.  All results are integers or copied bytes and do not depend on
// the order in which threads run: free pages are taken in ascending order and
// handed out in list order.
//
// The kernels wait for the kernel before them before they read anything and
// never let the kernel after them start early: kernels of the decode step read
// page tables, lengths and cached keys before their own dependency wait.
#include <algorithm>

#include "kernels.cuh"

namespace wedlm {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 4;  // 16-byte vectors per thread in flight

// Workspace: [0] the error word, [1] the number of planned copies, then the
// copies (source, destination), one int per page (free pages, marks or the
// map of a compaction) and two ints per sequence (marks, offsets).
struct PagesWs {
    int* err;
    int* count;
    int2* pairs;
    int* list;
    int* mark;
    int* off;
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

size_t pages_ws_bytes(int32_t num_pages, int32_t n_seq) {
    return 256 + round256((size_t)num_pages * sizeof(int2)) + round256((size_t)num_pages * 4) +
           2 * round256((size_t)n_seq * 4);
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
__device__ int find_free(const int32_t* refs, int num_pages, int want, int* list) {
    int have = 0;
    for (int64_t i0 = 0; i0 < num_pages && have < want; i0 += 4 * kPlanThreads) {
        const int64_t i = i0 + 4 * threadIdx.x;
        int r[4];
        load_refs(refs, i, num_pages, 1, r);
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

__global__ void __launch_bounds__(kPlanThreads) pages_copy_plan_kernel(const int32_t* src, const int32_t* dst, int n,
                                                                       int num_pages, PagesWs w) {
    griddep_wait();
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
}

__global__ void __launch_bounds__(kPlanThreads) pages_reserve_kernel(const int32_t* seqs, const int32_t* tokens, int n,
                                                                     wedlm_kv_pages p, PagesWs w) {
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int q = __ldcg(seqs + i);
        if (q >= 0 && q < p.n_seq) w.mark[q] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int q = __ldcg(seqs + i);
        if (q >= 0 && q < p.n_seq) atomicAdd(&w.mark[q], 1);
    }
    __syncthreads();
    // The pages each entry asks for.
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int q = __ldcg(seqs + i), t = __ldcg(tokens + i);
        bool ok = q >= 0 && q < p.n_seq && t >= 0 && (int64_t)t <= (int64_t)p.pages_per_seq * kPage;
        if (ok) ok = __ldcg(&w.mark[q]) == 1;
        int need = 0;
        if (ok) {
            const int32_t* row = p.page_table + (int64_t)q * p.pages_per_seq;
            int held = 0, first = p.pages_per_seq;
            for (int j = lane; j < p.pages_per_seq; j += 32) {
                if (__ldcg(row + j) >= 0) ++held;
                else first = min(first, j);
            }
            held = __reduce_add_sync(0xffffffffu, held);
            first = __reduce_min_sync(0xffffffffu, first);
            ok = held == first;  // no place empty before one that is taken
            need = max(0, (t + kPage - 1) / kPage - held);
        }
        if (lane == 0) {
            if (!ok) set_error(w.err, kErrBounds);
            w.off[i] = ok ? need : 0;
        }
    }
    __syncthreads();
    const int total = scan_needs(w.off, n);
    const int have = find_free(p.refs, p.num_pages, total, w.list);
    __syncthreads();
    if (have < total) {
        if (threadIdx.x == 0) set_error(w.err, kErrPages);
        return;
    }
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int at = w.off[i], need = (i + 1 < n ? w.off[i + 1] : total) - at;
        if (need == 0) continue;
        int32_t* row = p.page_table + (int64_t)__ldcg(seqs + i) * p.pages_per_seq;
        int held = 0;
        for (int j = lane; j < p.pages_per_seq; j += 32) held += __ldcg(row + j) >= 0;
        held = __reduce_add_sync(0xffffffffu, held);
        for (int j = lane; j < need; j += 32) {
            const int page = w.list[at + j];
            row[held + j] = page;
            p.refs[page] = 1;
        }
    }
    __threadfence();
}

__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(const int32_t* parents, const int32_t* children,
                                                                       int n, wedlm_kv_pages p, PagesWs w) {
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto in = [&](int q) { return q >= 0 && q < p.n_seq; };
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int a = __ldcg(parents + i), c = __ldcg(children + i);
        if (in(a)) w.mark[a] = 0;
        if (in(c)) w.mark[c] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int a = __ldcg(parents + i), c = __ldcg(children + i);
        if (in(a)) atomicOr(&w.mark[a], 1 << 30);
        if (in(c)) atomicAdd(&w.mark[c], 1);
    }
    __syncthreads();
    // off[i]: 1 when entry i needs a page of its own, for the parent's last page
    // that is not full; -1 for an entry that cannot be served.
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int a = __ldcg(parents + i), c = __ldcg(children + i);
        bool ok = in(a) && in(c);
        int L = 0;
        if (ok) {
            L = __ldcg(p.S + a);
            ok = __ldcg(&w.mark[c]) == 1 && L >= 0 && (int64_t)L <= (int64_t)p.pages_per_seq * kPage;
        }
        if (ok) {
            const int32_t* row = p.page_table + (int64_t)a * p.pages_per_seq;
            for (int j = lane; j < (L + kPage - 1) / kPage; j += 32) {
                const int page = __ldcg(row + j);
                if (page < 0 || page >= p.num_pages || __ldcg(p.refs + page) <= 0) ok = false;
            }
            const int32_t* own = p.page_table + (int64_t)c * p.pages_per_seq;
            for (int j = lane; j < p.pages_per_seq; j += 32) ok = ok && __ldcg(own + j) < 0;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) {
            if (!ok) set_error(w.err, kErrBounds);
            if (in(c)) w.mark[c] = ok ? 1 : 2;  // 2: this entry's child is left alone
            w.off[i] = ok ? (L % kPage != 0) : 0;
        }
    }
    __syncthreads();
    const int total = scan_needs(w.off, n);
    const int have = find_free(p.refs, p.num_pages, total, w.list);
    __syncthreads();
    if (threadIdx.x == 0) *w.count = have < total ? 0 : total;
    if (have < total) {
        if (threadIdx.x == 0) set_error(w.err, kErrPages);
        return;
    }
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int a = __ldcg(parents + i), c = __ldcg(children + i);
        if (!in(a) || !in(c) || __ldcg(&w.mark[c]) != 1) continue;
        const int32_t* from = p.page_table + (int64_t)a * p.pages_per_seq;
        int32_t* to = p.page_table + (int64_t)c * p.pages_per_seq;
        const int L = __ldcg(p.S + a), full = L / kPage;
        for (int j = lane; j < full; j += 32) {
            const int page = __ldcg(from + j);
            to[j] = page;
            atomicAdd(p.refs + page, 1);
        }
        if (lane == 0) {
            p.S[c] = L;
            if (L % kPage) {
                const int at = w.off[i], page = w.list[at];
                to[full] = page;
                p.refs[page] = 1;
                w.pairs[at] = make_int2(__ldcg(from + full), page);
            }
        }
    }
}

// One warp per listed sequence.  A sequence listed twice is freed once: each
// place of its table row is taken by one exchange.
__global__ void __launch_bounds__(128) pages_free_kernel(const int32_t* seqs, int n, wedlm_kv_pages p, int* err) {
    griddep_wait();
    const int lane = threadIdx.x & 31, i = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (i >= n) return;
    const int q = __ldcg(seqs + i);
    if (q < 0 || q >= p.n_seq) {
        if (lane == 0) set_error(err, kErrBounds);
        return;
    }
    int32_t* row = p.page_table + (int64_t)q * p.pages_per_seq;
    for (int j = lane; j < p.pages_per_seq; j += 32) {
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
    if (lane == 0) p.S[q] = 0;
    __threadfence();
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

// The planned copies in every layer, 16 KB of a page at a time, and (map !=
// nullptr) the page tables renamed.  Bound by HBM: each byte is read and
// written once.
__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(wedlm_kv_pages p, const int2* pairs, const int* count,
                                                                  const int32_t* map, int* err) {
    griddep_wait();
    if (map) {
        const int64_t entries = (int64_t)p.n_seq * p.pages_per_seq;
        for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < entries;
             e += (int64_t)gridDim.x * kCopyThreads) {
            const int page = __ldcg(p.page_table + e);
            if (page == -1) continue;
            const int to = page >= 0 && page < p.num_pages ? __ldcg(map + page) : -1;
            if (to < 0) set_error(err, kErrBounds);  // not a page in use: left as it is
            else if (to != page) p.page_table[e] = to;
        }
    }
    const int64_t nvec = p.page_bytes / 16;
    const int64_t chunks = (nvec + kCopyThreads * kCopyVec - 1) / (kCopyThreads * kCopyVec);
    const int64_t per_pair = chunks * p.n_layers, units = per_pair * __ldcg(count);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t k = u / per_pair, rest = u - k * per_pair;
        const int64_t layer = rest / chunks, v0 = (rest - layer * chunks) * (kCopyThreads * kCopyVec) + threadIdx.x;
        const int2 m = __ldcg(pairs + k);
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
    __threadfence();
}

cudaError_t launch_move(const wedlm_kv_pages& p, const PagesWs& w, int64_t most, const int32_t* map, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t chunks = (p.page_bytes / 16 + kCopyThreads * kCopyVec - 1) / (kCopyThreads * kCopyVec);
    int64_t units = most * p.n_layers * chunks;
    if (map) units = std::max(units, ((int64_t)p.n_seq * p.pages_per_seq + kCopyThreads - 1) / kCopyThreads);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(units, (int64_t)sms * 8));
    return launch_pdl(pages_move_kernel, dim3((unsigned)grid), dim3(kCopyThreads), 0, st, p, (const int2*)w.pairs,
                      (const int*)w.count, map, w.err);
}

// A description that the kernels can follow without leaving its buffers.
bool pages_ok(const wedlm_kv_pages* p, const void* ws, int64_t ws_bytes) {
    if (!p || !ws || !p->pool || !p->page_table || !p->S || !p->refs) return false;
    if (p->n_layers < 1 || p->num_pages < 1 || p->n_seq < 1 || p->pages_per_seq < 1) return false;
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
    cudaError_t e = launch_pdl(pages_copy_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, src, dst, n,
                               pages->num_pages, w);
    if (e == cudaSuccess) e = launch_move(*pages, w, n, nullptr, st);
    return done(e);
}

wedlm_status wedlm_kv_pages_reserve(const wedlm_kv_pages* pages, const int32_t* seqs, const int32_t* tokens, int32_t n,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes) || n < 0 || n > pages->n_seq) return WEDLM_ERR_INVALID_ARG;
    if (n == 0) return WEDLM_OK;
    if (!seqs || !tokens) return WEDLM_ERR_INVALID_ARG;
    const PagesWs w = pages_ws(workspace, pages->num_pages, pages->n_seq);
    return done(launch_pdl(pages_reserve_kernel, dim3(1), dim3(kPlanThreads), 0, (cudaStream_t)stream, seqs, tokens, n,
                           *pages, w));
}

wedlm_status wedlm_kv_pages_fork(const wedlm_kv_pages* pages, const int32_t* parents, const int32_t* children,
                                 int32_t n, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes) || n < 0 || n > pages->n_seq) return WEDLM_ERR_INVALID_ARG;
    if (n == 0) return WEDLM_OK;
    if (!parents || !children) return WEDLM_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const PagesWs w = pages_ws(workspace, pages->num_pages, pages->n_seq);
    cudaError_t e = launch_pdl(pages_fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, parents, children, n,
                               *pages, w);
    if (e == cudaSuccess) e = launch_move(*pages, w, n, nullptr, st);
    return done(e);
}

wedlm_status wedlm_kv_pages_free(const wedlm_kv_pages* pages, const int32_t* seqs, int32_t n, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes) || n < 0 || n > pages->n_seq) return WEDLM_ERR_INVALID_ARG;
    if (n == 0) return WEDLM_OK;
    if (!seqs) return WEDLM_ERR_INVALID_ARG;
    return done(launch_pdl(pages_free_kernel, dim3((unsigned)((n + 3) / 4)), dim3(128), 0, (cudaStream_t)stream, seqs,
                           n, *pages, static_cast<int*>(workspace)));
}

wedlm_status wedlm_kv_pages_compact(const wedlm_kv_pages* pages, int32_t* map, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    if (!pages_ok(pages, workspace, workspace_bytes)) return WEDLM_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const PagesWs w = pages_ws(workspace, pages->num_pages, pages->n_seq);
    int32_t* m = map ? map : w.list;
    cudaError_t e = launch_pdl(pages_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, *pages, m, w);
    if (e == cudaSuccess) e = launch_move(*pages, w, pages->num_pages / 2, (const int32_t*)m, st);
    return done(e);
}

}  // extern "C"
