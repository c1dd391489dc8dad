// kvl_pages.cu -- who owns the pages of a cache: extend, fork, free, compact, copy.
//
// The reference counts are the whole allocator: a page is free when its count is zero, and
// a batch that needs k pages takes the k lowest free numbers in batch order, so the result
// is a function of the state and not of which thread came first.  extend and compact are
// one CTA that walks the counts in tiles of kTile pages with block-wide prefix sums
// (bound by latency: a few microseconds); fork and free are one CTA a sequence (atomic adds,
// whose order does not show); copy moves whole pages with bulk copies through a ring of
// shared-memory stages, small ones a warp each (bound by HBM, as the copy kernels of kvl_copy.cu are).
#include "kvl_pages.cuh"

namespace kvl {
namespace {

// What batch entry i of an extend asks for.
struct Need {
    int32_t slot, len, count;
    int32_t first;  // first table entry that receives a page
    int32_t pages;
    int32_t shared; // the page that is replaced by a copy, or -1
    int32_t error;
};

__device__ Need need_of(const kvl_pages &p, const int32_t *slots, const int32_t *counts, int i)
{
    Need n = {slots[i], 0, counts[i], 0, 0, -1, KVL_OK};
    if (n.slot < 0 || n.slot >= p.n_slots || n.count < 0) {
        n.error = KVL_EINVAL;
        return n;
    }
    n.len = p.lens[n.slot];
    const int32_t B = p.block_tokens;
    const int64_t hi = ceil_div64(int64_t(n.len) + n.count, B);
    if (n.len < 0 || hi > p.table_stride || int64_t(n.len) + n.count > INT32_MAX) {
        n.error = KVL_ERANGE;
        return n;
    }
    n.first = int32_t(ceil_div64(n.len, B));
    if (n.count > 0 && n.len % B) {
        const int32_t last = p.tables[n.slot * p.table_stride + n.first - 1];
        if (last < 0 || last >= p.pool_blocks) {
            n.error = KVL_ERANGE;
            return n;
        }
        if (p.refs[last] > 1) {
            n.shared = last;
            --n.first;
        }
    }
    n.pages = int32_t(hi) - n.first;
    if (n.pages > (1 << 20)) n.error = KVL_ERANGE;  // keeps a chunk's sum within an int
    return n;
}

__global__ void __launch_bounds__(kThreads) extend_kernel(kvl_pages p, int32_t n, const int32_t *slots,
                                                          const int32_t *counts, void *rep)
{
    extern __shared__ uint32_t named[];  // one bit a slot
    __shared__ int scan_a[32], scan_b[32];
    __shared__ long long scan_need[32];
    __shared__ int s_prefix[kThreads], s_first[kThreads], s_slot[kThreads];
    __shared__ int s_bad;
    const int tid = threadIdx.x;
    for (int w = tid; w < (p.n_slots + 31) / 32; w += kThreads) named[w] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();

    // 1. what the batch needs (pages in the low half of a sum, copies in the high one), and whether it
    // may have it
    const Need nothing = {0, 0, 0, 0, 0, -1, KVL_OK};
    Need q = nothing;
    long long prefix = 0, want = 0;  // of the (last) chunk of entries
    int64_t need = 0;
    for (int base = 0; base < n; base += kThreads) {
        const int i = base + tid;
        q = nothing;
        if (i < n) {
            q = need_of(p, slots, counts, i);
            if (q.error == KVL_OK && (atomicOr(&named[q.slot >> 5], 1u << (q.slot & 31)) >> (q.slot & 31) & 1u))
                q.error = KVL_EDUP;
            if (q.error) {
                report(rep, q.error, i);
                s_bad = 1;
            }
        }
        if (base) __syncthreads();  // readers of the chunk before
        prefix = block_scan<long long>(q.error ? 0 : q.pages | (long long)(q.shared >= 0) << 32, scan_need, want);
        need += want & 0xffffffffll;
    }
    __syncthreads();
    bool ok = s_bad == 0 && need <= p.pool_blocks;
    if (s_bad == 0 && need > p.pool_blocks && tid == 0) report(rep, KVL_ERANGE, n);
    // the free pages: of a pool of one tile, their ranks stay for the second part
    int r[kPerThread], mine = 0, rank = 0;
    const bool one_tile = p.pool_blocks <= kTile;
    if (ok) {
        int64_t free_pages = 0;
        for (int64_t base = 0; base < p.pool_blocks && free_pages < need; base += kTile) {
            int total;
            mine = 0;
            load_refs(p.refs, base, p.pool_blocks, r);
#pragma unroll
            for (int k = 0; k < kPerThread; ++k) mine += r[k] == 0;
            if (base) __syncthreads();
            rank = block_scan<int>(mine, scan_a, total);
            free_pages += total;
        }
        if (free_pages < need) {
            ok = false;
            if (tid == 0) report(rep, KVL_ERANGE, n);
        }
    }
    if (!ok) {
        if (tid == 0) *p.n_pairs = 0;
        return;
    }

    // 2. hand the pages out: batch order meets page order
    int64_t tile = 0;
    int n_pairs = 0;
    for (int base = 0; base < n; base += kThreads) {
        const int i = base + tid;
        if (n > kThreads) {
            q = i < n ? need_of(p, slots, counts, i) : nothing;
            __syncthreads();
            prefix = block_scan<long long>(q.pages | (long long)(q.shared >= 0) << 32, scan_need, want);
        }
        const int pages = int(want & 0xffffffffll), copies = int(want >> 32), pair = int(prefix >> 32);
        s_prefix[tid] = int(prefix & 0xffffffffll);
        s_first[tid] = q.first;
        s_slot[tid] = q.slot;
        __syncthreads();
        int given = 0;
        while (given < pages && tile < p.pool_blocks) {
            int total = pages;
            if (!one_tile || base) {
                mine = 0;
                load_refs(p.refs, tile, p.pool_blocks, r);
#pragma unroll
                for (int k = 0; k < kPerThread; ++k) mine += r[k] == 0;
                rank = block_scan<int>(mine, scan_b, total);
                __syncthreads();
            }
            int at = given + rank;
#pragma unroll
            for (int k = 0; k < kPerThread; ++k) {
                if (r[k] != 0) continue;
                if (at < pages) {
                    // the last entry whose prefix is at most `at` (entries without need share the prefix
                    // of the next one, so the last of equals is the one that needs)
                    int lo = 0, hi = kThreads;
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) >> 1;
                        if (s_prefix[mid] <= at) lo = mid; else hi = mid;
                    }
                    const int64_t id = tile + int64_t(tid) * kPerThread + k;
                    p.tables[s_slot[lo] * p.table_stride + s_first[lo] + (at - s_prefix[lo])] = int32_t(id);
                    p.refs[id] = 1;
                }
                ++at;
            }
            given += total;
            if (given < pages) tile += kTile;  // otherwise the next entries go on in this tile
        }
        __syncthreads();  // the tables and counts written above
        if (i < n) {
            if (q.shared >= 0)
                reinterpret_cast<int2 *>(p.pairs)[n_pairs + pair] = make_int2(q.shared, p.tables[q.slot * p.table_stride + q.first]);
            p.lens[q.slot] = q.len + q.count;
        }
        n_pairs += copies;
    }
    __syncthreads();
    // 3. the replaced pages lose a reference (only now: the calls of need_of saw the counts
    // as they were when the call began)
    for (int k = tid; k < n_pairs; k += kThreads) atomicSub(&p.refs[reinterpret_cast<const int2 *>(p.pairs)[k].x], 1);
    if (tid == 0) *p.n_pairs = n_pairs;
}

__global__ void __launch_bounds__(128) fork_kernel(kvl_pages p, const int32_t *parents, const int32_t *children,
                                                   void *rep)
{
    __shared__ int s_len;
    const int i = blockIdx.x;
    const int32_t a = parents[i], c = children[i];
    if (a < 0 || a >= p.n_slots || c < 0 || c >= p.n_slots || a == c) {
        if (threadIdx.x == 0) report(rep, KVL_EINVAL, i);
        return;
    }
    if (threadIdx.x == 0) {
        int len = p.lens[a];
        if (len < 0 || ceil_div64(len, p.block_tokens) > p.table_stride) {
            report(rep, KVL_ERANGE, i);
            len = 0;
        } else if (atomicCAS(&p.lens[c], 0, len) != 0) {
            report(rep, KVL_EINVAL, i);
            len = 0;
        }
        s_len = len;
    }
    __syncthreads();
    const int n = int(ceil_div64(s_len, p.block_tokens));
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
        const int32_t id = p.tables[a * p.table_stride + k];
        p.tables[c * p.table_stride + k] = id;
        if (id >= 0 && id < p.pool_blocks)
            atomicAdd(&p.refs[id], 1);
        else
            report(rep, KVL_ERANGE, i);
    }
}

__global__ void __launch_bounds__(128) free_kernel(kvl_pages p, const int32_t *slots, void *rep)
{
    __shared__ int s_len;
    const int i = blockIdx.x;
    const int32_t s = slots[i];
    if (s < 0 || s >= p.n_slots) {
        if (threadIdx.x == 0) report(rep, KVL_EINVAL, i);
        return;
    }
    if (threadIdx.x == 0) {
        int len = atomicExch(&p.lens[s], 0);  // a slot named twice is empty the second time
        if (len < 0 || ceil_div64(len, p.block_tokens) > p.table_stride) {
            report(rep, KVL_ERANGE, i);
            len = 0;
        }
        s_len = len;
    }
    __syncthreads();
    const int n = int(ceil_div64(s_len, p.block_tokens));
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
        const int32_t id = p.tables[s * p.table_stride + k];
        if (id < 0 || id >= p.pool_blocks) {
            report(rep, KVL_ERANGE, i);
        } else if (atomicSub(&p.refs[id], 1) <= 0) {
            atomicAdd(&p.refs[id], 1);
            report(rep, KVL_EINVAL, i);
        }
    }
}

__global__ void __launch_bounds__(kThreads) compact_kernel(kvl_pages p)
{
    __shared__ int scan_a[32];
    __shared__ long long scan_b[32];
    int64_t live = 0;
    for (int64_t base = 0; base < p.pool_blocks; base += kTile) {
        int r[kPerThread], mine = 0, total;
        load_refs(p.refs, base, p.pool_blocks, r);
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) mine += base + int64_t(threadIdx.x) * kPerThread + k < p.pool_blocks && r[k] > 0;
        if (base) __syncthreads();
        block_scan<int>(mine, scan_a, total);
        live += total;
    }
    // free numbers below `live` and live pages from it on are equally many: both lists go
    // straight into the pairs, each at its rank
    int2 *pairs = reinterpret_cast<int2 *>(p.pairs);
    int holes = 0, movers = 0;
    for (int64_t base = 0; base < p.pool_blocks; base += kTile) {
        int r[kPerThread], h = 0, m = 0;
        long long both;
        load_refs(p.refs, base, p.pool_blocks, r);
        const int64_t at = base + int64_t(threadIdx.x) * kPerThread;
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            h += at + k < live && r[k] <= 0;
            m += at + k >= live && at + k < p.pool_blocks && r[k] > 0;
        }
        if (base) __syncthreads();
        const long long before = block_scan<long long>(h | (long long)m << 32, scan_b, both);
        int hr = holes + int(before & 0xffffffffll), mr = movers + int(before >> 32);
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            if (at + k < live && r[k] <= 0) pairs[hr++].y = int32_t(at + k);
            if (at + k >= live && at + k < p.pool_blocks && r[k] > 0) pairs[mr++].x = int32_t(at + k);
        }
        holes += int(both & 0xffffffffll);
        movers += int(both >> 32);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kThreads) {
        const int2 q = pairs[k];
        p.refs[q.y] = p.refs[q.x];
        p.refs[q.x] = 0;
    }
    if (threadIdx.x == 0) *p.n_pairs = movers;
}

// Table entries that name a moved page follow it: the pairs are sorted by old number, and searched in
// shared memory where they fit (a search in memory is a dozen loads one after another).
constexpr int kNamesHeld = 8192;

__global__ void __launch_bounds__(256) rename_kernel(kvl_pages p, void *rep)
{
    __shared__ int32_t held[kNamesHeld];
    const int n = *p.n_pairs;
    if (n == 0) return;
    const int2 *pairs = reinterpret_cast<const int2 *>(p.pairs);
    const bool in_shared = n <= kNamesHeld;
    if (in_shared)
        for (int k = threadIdx.x; k < n; k += 256) held[k] = pairs[k].x;
    const int32_t lowest = pairs[0].x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int s = blockIdx.x * 8 + int(threadIdx.x >> 5); s < p.n_slots; s += gridDim.x * 8) {
        const int32_t len = p.lens[s];
        int64_t used = ceil_div64(len, p.block_tokens);
        if (len < 0 || used > p.table_stride) {
            if (lane == 0) report(rep, KVL_ERANGE, s);
            used = 0;
        }
        for (int64_t k = lane; k < used; k += 32) {
            int32_t *e = p.tables + s * p.table_stride + k;
            const int32_t id = *e;
            if (id < lowest) continue;
            int lo = 0, hi = n;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if ((in_shared ? held[mid] : pairs[mid].x) <= id) lo = mid; else hi = mid;
            }
            const int2 q = pairs[lo];
            if (q.x == id) *e = q.y;
        }
    }
}

// ---- copies ------------------------------------------------------------------------------

constexpr int kCopyStages = 6;
constexpr int kCopyThreads = 64;  // warp 0: bulk copies of codes; warp 1: scales

struct CopyPagesArgs {
    kvl_cache c;
    const int32_t *pairs;
    const int32_t *n_pairs;
    int64_t max_pairs;
    int64_t page_bytes;   // B*H*d
    int32_t chunks;       // stages' worth of bytes per plane of a page
    void *report;
};

__device__ __forceinline__ bool pair_of(const CopyPagesArgs &a, int64_t k, int2 &q)
{
    q = reinterpret_cast<const int2 *>(a.pairs)[k];
    return q.x >= 0 && q.x < a.c.pool_blocks && q.y >= 0 && q.y < a.c.pool_blocks;
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a)
{
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ __align__(8) unsigned long long bars[kCopyStages];
    int64_t n = *a.n_pairs;
    if (n < 0 || n > a.max_pairs) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(a.report, KVL_ERANGE, n);
        n = n < 0 ? 0 : a.max_pairs;
    }
    const int64_t planes = int64_t(a.c.n_layers) * 2, N = a.c.pool_blocks;
    if (threadIdx.x >= 32) {
        // scales: H floats a (pair, layer, plane)
        const int H = a.c.n_kv_heads, lane = threadIdx.x - 32;
        for (int64_t u = blockIdx.x; u < n * planes; u += gridDim.x) {
            const int64_t k = u / planes, lp = u - k * planes;
            int2 q;
            if (!pair_of(a, k, q)) {
                if (lane == 0) report(a.report, KVL_ERANGE, k);
                continue;
            }
            const float *src = a.c.scales + (lp * N + q.x) * H;
            float *dst = a.c.scales + (lp * N + q.y) * H;
            for (int h = lane; h < H; h += 32) dst[h] = src[h];
        }
        return;
    }
    if (threadIdx.x != 0) return;
    const uint32_t bar0 = smem_u32(bars), buf0 = smem_u32(stages);
    for (int s = 0; s < kCopyStages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
    const int64_t units = n * planes * a.chunks;
    uint8_t *codes = static_cast<uint8_t *>(a.c.codes);
    auto locate = [&](int64_t u, uint8_t *&src, uint8_t *&dst, uint32_t &bytes) {
        const int64_t kp = u / a.chunks, at = (u - kp * a.chunks) * kStageBytes;
        const int64_t k = kp / planes, lp = kp - k * planes;
        int2 q;
        if (!pair_of(a, k, q)) return false;
        src = codes + (lp * N + q.x) * a.page_bytes + at;
        dst = codes + (lp * N + q.y) * a.page_bytes + at;
        bytes = uint32_t(min(int64_t(kStageBytes), a.page_bytes - at));
        return true;
    };
    // loads run kCopyStages - 1 units ahead of the stores; a stage is loaded again once the
    // store that read it has (all store groups but the newest are waited for)
    const int64_t first = blockIdx.x, step = gridDim.x;
    int64_t issued = 0, done = 0;
    bool timed_out = false;
    const int64_t mine = first < units ? (units - first + step - 1) / step : 0;
    while (done < mine && !timed_out) {
        while (issued < mine && issued < done + kCopyStages - 1) {
            const int s = int(issued % kCopyStages);
            uint8_t *src, *dst;
            uint32_t bytes;
            if (locate(first + issued * step, src, dst, bytes)) {
                mbar_arrive_expect_tx(bar0 + 8 * s, bytes);
                bulk_load(buf0 + s * kStageBytes, src, bytes, bar0 + 8 * s);
            } else {
                mbar_arrive(bar0 + 8 * s);  // keeps the stage's phases in step
            }
            ++issued;
        }
        const int s = int(done % kCopyStages);
        if (!mbar_wait_bounded(bar0 + 8 * s, uint32_t((done / kCopyStages) & 1))) {
            report(a.report, KVL_ETIMEOUT, blockIdx.x);
            timed_out = true;
            break;
        }
        uint8_t *src, *dst;
        uint32_t bytes;
        if (locate(first + done * step, src, dst, bytes)) bulk_store(dst, buf0 + s * kStageBytes, bytes);
        bulk_commit();
        bulk_wait_read_all_but_one();
        ++done;
    }
    if (timed_out)
        for (int64_t k = done; k < issued; ++k)
            mbar_wait_bounded(bar0 + 8 * int(k % kCopyStages), uint32_t((k / kCopyStages) & 1));
    bulk_wait_all();
}

// Small pages: a warp a page and plane, 16 bytes a lane, as one thread that issues bulk copies takes 0.8 us a
// unit, however small.  Measured (us, lanes / bulk copies; bytes of a page's plane of one layer): 1 KB x
// 128,000 68 / 663, 4 KB x 128,000 211 / 660, 8 KB x 38,400 125 / 198; 16 KB x 32,000 192 / 177, 32 KB x
// 4,800 61 / 51.
constexpr int kSmallThreads = 256, kSmallCtasPerSm = 8;
constexpr int64_t kSmallPage = 8192;

__global__ void __launch_bounds__(kSmallThreads, kSmallCtasPerSm) copy_small_pages_kernel(const __grid_constant__ CopyPagesArgs a)
{
    int64_t n = *a.n_pairs;
    if (n < 0 || n > a.max_pairs) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(a.report, KVL_ERANGE, n);
        n = n < 0 ? 0 : a.max_pairs;
    }
    const int64_t planes = int64_t(a.c.n_layers) * 2, N = a.c.pool_blocks;
    const int H = a.c.n_kv_heads, lane = threadIdx.x & 31, page_bytes = int(a.page_bytes);
    // unit u: pair u / planes, layer and plane u % planes
    const int64_t u = int64_t(blockIdx.x) * (kSmallThreads / 32) + (threadIdx.x >> 5);
    const int64_t step = int64_t(gridDim.x) * (kSmallThreads / 32), dk = step / planes, dlp = step - dk * planes;
    int64_t k = u / planes, lp = u - k * planes;
    while (k < n) {
        int2 q;
        if (pair_of(a, k, q)) {
            const uint8_t *src = static_cast<const uint8_t *>(a.c.codes) + (lp * N + q.x) * a.page_bytes;
            uint8_t *dst = static_cast<uint8_t *>(a.c.codes) + (lp * N + q.y) * a.page_bytes;
            const float *from = a.c.scales + (lp * N + q.x) * H;
            float *to = a.c.scales + (lp * N + q.y) * H;
            const float first = lane < H ? from[lane] : 0.f;  // on its way with the codes
            for (int at = lane * 16; at < page_bytes; at += 4 * 512) {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + 512 * i < page_bytes) v[i] = *reinterpret_cast<const uint4 *>(src + at + 512 * i);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + 512 * i < page_bytes) *reinterpret_cast<uint4 *>(dst + at + 512 * i) = v[i];
            }
            if (lane < H) to[lane] = first;
            for (int h = lane + 32; h < H; h += 32) to[h] = from[h];
        } else if (lane == 0) {
            report(a.report, KVL_ERANGE, k);
        }
        k += dk;
        lp += dlp;
        if (lp >= planes) {
            lp -= planes;
            ++k;
        }
    }
}

}  // namespace
}  // namespace kvl

using namespace kvl;

extern "C" kvl_status kvl_pages_extend(const kvl_pages *pages, int32_t n, const int32_t *slots,
                                       const int32_t *counts, void *d_report, void *stream)
{
    const kvl_status s = check_batch(pages, n, slots, counts, d_report);
    if (s) return s;
    static std::atomic<unsigned long long> ready[kMaxDevices];
    const int smem = (pages->n_slots + 31) / 32 * 4;
    if (smem > 32 * 1024 && !allow_smem(extend_kernel, ready, (1 << 20) / 8)) return KVL_ECUDA;
    extend_kernel<<<1, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(*pages, n, slots, counts, d_report);
    return launch_status();
}

extern "C" kvl_status kvl_pages_fork(const kvl_pages *pages, int32_t n, const int32_t *parents,
                                     const int32_t *children, void *d_report, void *stream)
{
    const kvl_status s = check_batch(pages, n, parents, children, d_report);
    if (s || n == 0) return s;
    fork_kernel<<<n, 128, 0, static_cast<cudaStream_t>(stream)>>>(*pages, parents, children, d_report);
    return launch_status();
}

extern "C" kvl_status kvl_pages_free(const kvl_pages *pages, int32_t n, const int32_t *slots,
                                     void *d_report, void *stream)
{
    const kvl_status s = check_batch(pages, n, slots, slots, d_report);
    if (s || n == 0) return s;
    free_kernel<<<n, 128, 0, static_cast<cudaStream_t>(stream)>>>(*pages, slots, d_report);
    return launch_status();
}

extern "C" kvl_status kvl_pages_compact(const kvl_pages *pages, void *d_report, void *stream)
{
    const kvl_status s = check_pages(pages);
    if (s) return s;
    if (bad_report(d_report)) return KVL_EALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    compact_kernel<<<1, kThreads, 0, st>>>(*pages);
    if (launch_status()) return KVL_ECUDA;
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    const int ctas = (pages->n_slots + 7) / 8;
    rename_kernel<<<ctas < 4 * sms ? ctas : 4 * sms, 256, 0, st>>>(*pages, d_report);
    return launch_status();
}

extern "C" kvl_status kvl_pages_copy(const kvl_cache *cache, const int32_t *pairs, const int32_t *d_n_pairs,
                                     int64_t max_pairs, void *d_report, void *stream)
{
    const kvl_status s = check_cache(cache);
    if (s) return s;
    if (max_pairs < 0 || max_pairs > INT32_MAX) return KVL_EINVAL;
    if (max_pairs == 0) return KVL_OK;
    if (!pairs || !d_n_pairs) return KVL_EINVAL;
    if ((reinterpret_cast<uintptr_t>(pairs) & 7u) || misaligned4(d_n_pairs) || bad_report(d_report)) return KVL_EALIGN;
    CopyPagesArgs a;
    a.c = *cache;
    a.pairs = pairs;
    a.n_pairs = d_n_pairs;
    a.max_pairs = max_pairs;
    a.page_bytes = int64_t(cache->block_tokens) * cache->n_kv_heads * cache->head_dim;
    const int64_t chunks = ceil_div64(a.page_bytes, kStageBytes);
    if (chunks > INT32_MAX) return KVL_EINVAL;
    a.chunks = int32_t(chunks);
    a.report = d_report;
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    if (a.page_bytes <= kSmallPage) {
        copy_small_pages_kernel<<<sms * kSmallCtasPerSm, kSmallThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
        return launch_status();
    }
    static std::atomic<unsigned long long> ready[kMaxDevices];
    if (!allow_smem(copy_pages_kernel, ready, kCopyStages * kStageBytes)) return KVL_ECUDA;
    copy_pages_kernel<<<sms, kCopyThreads, kCopyStages * kStageBytes, static_cast<cudaStream_t>(stream)>>>(a);
    return launch_status();
}
