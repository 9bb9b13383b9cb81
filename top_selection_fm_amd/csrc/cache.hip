// cache.hip -- the pages of a cache: forking, growing, compacting and freeing requests.
//
// All state lives on the device: block tables, lengths, a reference count a page and a stack of
// free pages.  Every call is one or two launches and needs nothing from the host, so a step that
// forks, grows or compacts can sit in a captured graph.
//
// Bookkeeping (cache_plan_kernel, cache_release_kernel) is one workgroup: the work is a scan over
// the call's entries and a pass over the table cells that change, bound by latency; one workgroup
// needs no counters cleared between launches and gives the same stacks in every run.  Entry i's
// pages come from the stack by a prefix sum over the entries; pages that nobody refers to any
// more are collected in a bitmap in LDS and pushed in page order.  Moving data
// (cache_copy_kernel, cache_move_kernel) is spread over the chip and bound by memory.  Measured
// (eight pools of 8 heads of 256-byte rows): 12 of 16 requests of 8,000 entries freed and forked
// again 19 us (release 4 to 6, plan 5, copy 7: 25 MB); 32 requests grown by 64 entries and
// compacted 24 us (plan 6, copy 1 to 2, move 8, release 6).  The rest is four launches.
#include <algorithm>

#include "fm_internal.h"

namespace fm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kPlanNT = 1024;

__device__ __forceinline__ int pages_of(int entries) { return (int)(((int64_t)entries + kPage - 1) / kPage); }

// Exclusive prefix sum over the workgroup's threads; total receives the sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *sh, int64_t &total) {
    const int ln = __lane_id(), w = threadIdx.x >> 6;
    int64_t inc = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t y = __shfl_up(inc, o);
        if (ln >= o) inc += y;
    }
    if (ln == 63) sh[w] = inc;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kPlanNT / 64; ++i) {
        if (i < w) before += sh[i];
        total += sh[i];
    }
    __syncthreads();
    return before + inc - x;
}

// First entry of the call naming each request: later ones with the same request are refused.
__device__ __forceinline__ void claim(const CacheArgs &A, const int32_t *req, int32_t *claims) {
    const int mine = threadIdx.x < A.n ? req[threadIdx.x] : -1;      // on its way meanwhile
    for (int b = threadIdx.x; b < A.B; b += kPlanNT) claims[b] = INT32_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < A.n; i += kPlanNT) {
        const int r = i < kPlanNT ? mine : req[i];
        if (r >= 0 && r < A.B) atomicMin(&claims[r], i);
    }
    __syncthreads();
}

__device__ __forceinline__ int length_of(const CacheArgs &A, int r) {
    return (int)max((int64_t)0, min((int64_t)A.seq_lens[r], A.bt_ld * kPage));
}

// One reference less; the page goes into the bitmap when it was the last, and any is set.
__device__ __forceinline__ void drop(const CacheArgs &A, int page, uint32_t *freed, int *any) {
    const int before = atomicSub(&A.ref[page], 1);
    if (before == 1) {
        atomicOr(&freed[page >> 5], 1u << (page & 31));
        *any = 1;
    } else if (before <= 0) {
        atomicAdd(&A.ref[page], 1);                       // was free already: left as it was
    }
}

// The bitmap's pages onto the stack, which holds `held` of them, in page order.
__device__ __forceinline__ void push(const CacheArgs &A, const uint32_t *freed, int any, int64_t held, int64_t *sh) {
    if (!any) {
        if (threadIdx.x == 0) *A.n_free = (int32_t)held;
        return;
    }
    const int words = (int)((A.n_phys + 31) / 32), per = (words + kPlanNT - 1) / kPlanNT;
    const int w0 = min(words, (int)threadIdx.x * per), w1 = min(words, w0 + per);
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(freed[w]);
    int64_t total;
    int64_t at = held + block_scan(mine, sh, total);
    for (int w = w0; w < w1; ++w)
        for (uint32_t x = freed[w]; x; x &= x - 1) {
            if (at < A.n_phys) A.free_list[at] = 32 * w + __builtin_ctz(x);
            ++at;
        }
    if (threadIdx.x == 0) *A.n_free = (int32_t)min(held + total, A.n_phys);
}

__device__ __forceinline__ void clear_freed(const CacheArgs &A, uint32_t *freed) {
    for (int w = threadIdx.x; w < (A.n_phys + 31) / 32; w += kPlanNT) freed[w] = 0;
}

// Threads per entry when the workgroup's threads are shared among n entries: a power of two.
__device__ __forceinline__ int team_size(int n) {
    int t = 16;
    while (t < kPlanNT && (int64_t)t * 2 * n <= kPlanNT) t *= 2;
    return t;
}

// Entry i of a compaction: where it starts, how many entries it keeps, and of those the thread's
// first and the one before, read without waiting for each other.
struct Kept {
    int start, k, s, prev;
};
__device__ __forceinline__ Kept read_kept(const CacheArgs &A, int i, int lane) {
    const int32_t *keep = A.keep + (int64_t)i * A.keep_ld;
    return {A.start[i], A.n_keep[i], lane < A.keep_ld ? keep[lane] : -1, lane && lane < A.keep_ld ? keep[lane - 1] : -1};
}
// Whether it may be carried out, as far as thread `lane` of `lanes` checks it: the kept entries
// ascending within [start, len), and every page that receives or gives a moved entry mapped, the
// receiving ones held by this request alone.  The pages are read while len is on its way.
__device__ __forceinline__ bool keep_is_good(const CacheArgs &A, int i, int r, int len, const Kept &e, int lane, int lanes) {
    const int32_t *keep = A.keep + (int64_t)i * A.keep_ld;
    const int32_t *row = A.block_table + (int64_t)r * A.bt_ld;
    const int64_t cells = A.bt_ld * kPage;
    bool good = e.start >= 0 && e.k >= 0 && e.k <= A.keep_ld;
    const int k = good ? e.k : 0;
    for (int j = lane; j < k && good; j += lanes) {
        const int s = j == lane ? e.s : keep[j], prev = j == 0 ? e.start - 1 : j == lane ? e.prev : keep[j - 1];
        const int64_t d = (int64_t)e.start + j;
        if (s <= prev || s < d || s >= cells) {            // so d < cells too
            good = false;
        } else if (s != d) {
            const int from = row[s / kPage], to = row[d / kPage];
            const bool live = to >= 0 && to < A.n_phys;
            good = from >= 0 && from < A.n_phys && live && A.ref[live ? to : 0] == 1;
        }
        good = good && s < len;
    }
    return good && e.start <= len && e.k <= len - e.start;
}

// Requests cut to a new length: freeing (COMPACT false; new_len[i], or 0) and the end of a
// compaction (start[i] + n_keep[i], after its entries have moved).  Every entry is judged before
// any reference is dropped: what one entry gives up must not change another's verdict.
template <bool COMPACT>
__global__ __launch_bounds__(kPlanNT) void cache_release_kernel(CacheArgs A) {
    __shared__ uint32_t freed[kCacheMaxPages / 32];
    __shared__ int32_t claims[kCacheMaxRequests];
    __shared__ uint8_t bad[kCacheMaxRequests];
    __shared__ int64_t sh[kPlanNT / 64];
    __shared__ int any;
    const int64_t held = max((int64_t)0, min((int64_t)*A.n_free, A.n_phys));
    const int team = team_size(A.n), lane = threadIdx.x % team, first = threadIdx.x / team, teams = kPlanNT / team;
    // entry i's request, its length and where it is cut; with an entry a team they stay in
    // registers from the verdict to the release
    int r = -1, len = 0, cut = 0;
    Kept kept = {};
    auto look = [&](int i) {
        r = A.req[i];
        if constexpr (COMPACT) kept = read_kept(A, i, lane);
        cut = COMPACT ? kept.start + kept.k : A.new_len ? A.new_len[i] : 0;
        len = r >= 0 && r < A.B ? length_of(A, r) : -1;
    };
    if (first < A.n) look(first);
    clear_freed(A, freed);
    if (threadIdx.x == 0) any = 0;
    for (int i = threadIdx.x; i < A.n; i += kPlanNT) bad[i] = 0;
    claim(A, A.req, claims);
    for (int i = first; i < A.n; i += teams) {
        if (i != first) look(i);
        bool good = len >= 0 && claims[r] == i;
        if (good) {
            if constexpr (COMPACT) good = keep_is_good(A, i, r, len, kept, lane, team);
            else good = cut >= 0 && cut <= len;
        }
        if (!good) bad[i] = 1;
    }
    __syncthreads();
    for (int i = first; i < A.n; i += teams) {
        const bool good = !bad[i];
        if (lane == 0 && A.ok) A.ok[i] = good;
        if (!good) continue;
        if (teams < A.n) look(i);
        int32_t *row = A.block_table + (int64_t)r * A.bt_ld;
        const int c1 = pages_of(len);
        for (int c = pages_of(cut) + lane; c < c1; c += team) {
            const int page = row[c];
            row[c] = -1;
            if (page >= 0 && page < A.n_phys) drop(A, page, freed, &any);
        }
        if (lane == 0) A.seq_lens[r] = cut;               // read by this team alone
    }
    __syncthreads();
    push(A, freed, any, held, sh);
}

// Pages for forks (FORK) and for growth.  plan[i] receives what the copy needs: a fork's length
// (or -1: refused); a growth's page to copy and its copy (or -1).
template <bool FORK>
__global__ __launch_bounds__(kPlanNT) void cache_plan_kernel(CacheArgs A) {
    __shared__ uint32_t freed[FORK ? 1 : kCacheMaxPages / 32];
    __shared__ int32_t claims[kCacheMaxRequests];
    __shared__ int64_t sh[kPlanNT / 64];
    __shared__ int4 plans[kPlanNT];                       // of the call's entries, where they fit
    __shared__ int any, taken;
    const bool fits = A.n <= kPlanNT;
    const int32_t *req = FORK ? A.dst : A.req;
    const int64_t have = max((int64_t)0, min((int64_t)*A.n_free, A.n_phys));
    if constexpr (!FORK) clear_freed(A, freed);
    if (threadIdx.x == 0) any = taken = 0;
    claim(A, req, claims);
    // what each entry needs, before anything is changed; its first page's rank goes to plan[i].w
    int64_t base = 0;
    for (int i0 = 0; i0 < A.n; i0 += kPlanNT) {
        const int i = i0 + threadIdx.x;
        bool good = false;
        int need = 0, len = 0, cow = -1, r = -1, old = 0;
        if (i < A.n) {
            r = req[i];
            if (r >= 0 && r < A.B) {
                if constexpr (FORK) {
                    const int s = A.src[i];
                    if (s >= 0 && s < A.B && s != r) {
                        len = length_of(A, s);
                        need = A.deep ? pages_of(len) : len % kPage != 0;
                        good = A.seq_lens[r] == 0 && claims[r] == i;
                    }
                } else {
                    old = length_of(A, r);
                    len = A.new_len[i];
                    if (claims[r] == i && len >= old && pages_of(len) <= A.bt_ld) {
                        good = true;
                        need = pages_of(len) - pages_of(old);
                        if (old % kPage && len > old) {
                            const int page = A.block_table[(int64_t)r * A.bt_ld + old / kPage];
                            if (page >= 0 && page < A.n_phys && A.ref[page] > 1) cow = page;
                        }
                        need += cow >= 0;
                    }
                }
            }
        }
        int64_t total;
        const int64_t mine = base + block_scan(good ? need : 0, sh, total);
        good = good && mine + need <= have;
        base += total;
        // granted entries are a prefix of the valid ones: the last one's end is what is taken
        if (good) atomicMax(&taken, (int)(mine + need));
        if (i < A.n) {
            const int4 p = make_int4(good ? len : -1, cow, -1, good ? (int)mine : 0);
            if (fits) plans[i] = p;
            A.plan[i] = p;
            if (A.ok) A.ok[i] = good;
        }
    }
    __syncthreads();
    const int team = team_size(A.n), lane = threadIdx.x % team;
    for (int i = threadIdx.x / team; i < A.n; i += kPlanNT / team) {
        const int4 p = fits ? plans[i] : A.plan[i];
        if (p.x < 0) continue;
        const int r = req[i];
        int32_t *row = A.block_table + (int64_t)r * A.bt_ld;
        const int old = FORK ? 0 : length_of(A, r);
        // fresh pages go to cells c0 .. c1 - 1; a copied one to the cell before, from the first rank
        const int c0 = FORK ? (A.deep ? 0 : p.x / kPage) : pages_of(old), c1 = pages_of(p.x);
        const int cow = !FORK && p.y >= 0;
        for (int c = c0 - cow + lane; c < c1; c += team) {
            const int page = A.free_list[have - 1 - (p.w + (c - (c0 - cow)))];
            const bool fine = page >= 0 && page < A.n_phys;
            row[c] = fine ? page : -1;
            if (fine) A.ref[page] = 1;
            if (cow && c == c0 - 1) {
                A.plan[i].z = fine ? page : -1;
                drop(A, p.y, freed, &any);
            }
        }
    }
    __syncthreads();                                       // the lengths are read
    for (int i = threadIdx.x; i < A.n; i += kPlanNT) {
        const int len = fits ? plans[i].x : A.plan[i].x;
        if (len >= 0) A.seq_lens[req[i]] = len;
    }
    if constexpr (FORK) {
        if (threadIdx.x == 0) *A.n_free = (int32_t)(have - taken);
    } else {
        push(A, freed, any, have - taken, sh);
    }
}

__device__ __forceinline__ int64_t page_bytes(const CacheArgs &A, int pool) {
    return (int64_t)A.heads[pool] * kPage * A.row_bytes[pool];
}

// A part of a page, 16 bytes a thread and turn.
__device__ __forceinline__ void copy_part(const CacheArgs &A, int pool, int from, int to, int part, int parts) {
    const int64_t bytes = page_bytes(A, pool), n = bytes / 16;
    const u32x4 *src = (const u32x4 *)(A.pool[pool] + from * bytes);
    u32x4 *dst = (u32x4 *)(A.pool[pool] + to * bytes);
    constexpr int U = 8;                                   // loads in flight a thread
    for (int64_t x = part * 256 + threadIdx.x; x < n; x += (int64_t)U * parts * 256) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (x + u * parts * 256 < n) v[u] = src[x + u * parts * 256];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (x + u * parts * 256 < n) dst[x + u * parts * 256] = v[u];
    }
}

// The data of forks and growths: workgroup (part of a page, entry, pool).
constexpr int kCopyParts = 4;
template <bool FORK>
__global__ __launch_bounds__(256) void cache_copy_kernel(CacheArgs A) {
    const int i = blockIdx.y, pool = blockIdx.z;
    const int4 p = A.plan[i];
    if (p.x < 0) return;
    if constexpr (!FORK) {
        if (p.y >= 0 && p.z >= 0) copy_part(A, pool, p.y, p.z, blockIdx.x, gridDim.x);
        return;
    }
    const int32_t *from = A.block_table + (int64_t)A.src[i] * A.bt_ld;
    int32_t *to = A.block_table + (int64_t)A.dst[i] * A.bt_ld;
    const int full = A.deep ? 0 : p.x / kPage;
    if (pool == 0)                                         // shared pages
        for (int c = blockIdx.x * 256 + threadIdx.x; c < full; c += gridDim.x * 256) {
            const int page = from[c];
            to[c] = page;
            if (page >= 0 && page < A.n_phys) atomicAdd(&A.ref[page], 1);
        }
    for (int c = full + blockIdx.x / kCopyParts; c < pages_of(p.x); c += gridDim.x / kCopyParts) {
        const int a = from[c], b = to[c];
        if (a >= 0 && a < A.n_phys && b >= 0 && b < A.n_phys)
            copy_part(A, pool, a, b, blockIdx.x % kCopyParts, kCopyParts);
    }
}

// The kept entries of a compaction to the front, in place: workgroup (head, entry, pool).  Entries
// go in ascending chunks, a chunk read whole before it is written; entry j moves down to start + j
// <= keep[j] < keep[j + 1], so a write never meets a later chunk's source.
template <class T>
__device__ __forceinline__ void move_rows(const CacheArgs &A, int r, int pool, int head, int start, const int32_t *keep,
                                          int first, int k) {
    constexpr int U = 4, STEP = 256 * U;
    const int row_bytes = A.row_bytes[pool], per = row_bytes / (int)sizeof(T);
    const int64_t bytes = page_bytes(A, pool), at = (int64_t)head * kPage * row_bytes;
    const int32_t *row = A.block_table + (int64_t)r * A.bt_ld;
    auto place = [&](int s, int e) {
        return (T *)(A.pool[pool] + row[s / kPage] * bytes + at + (int64_t)(s % kPage) * row_bytes) + e;
    };
    // columns e0 .. e0 + w - 1 of a row at a time (all of it, but for rows past STEP pieces)
    for (int e0 = 0; e0 < per; e0 += STEP) {
        const int w = min(per - e0, STEP), rows = STEP / w;
        for (int j0 = first; j0 < k; j0 += rows) {
            const int total = min(rows, k - j0) * w;
            T v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int x = 256 * u + threadIdx.x;
                if (x < total) v[u] = *place(keep[j0 + x / w], e0 + x % w);
            }
            __builtin_amdgcn_s_waitcnt(0);                 // every wave's reads before any write
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int x = 256 * u + threadIdx.x;
                if (x < total) *place(start + j0 + x / w, e0 + x % w) = v[u];
            }
        }
    }
}

__global__ __launch_bounds__(256) void cache_move_kernel(CacheArgs A) {
    __shared__ int bad, moved;
    const int head = blockIdx.x, i = blockIdx.y, pool = blockIdx.z, tid = threadIdx.x;
    if (head >= A.heads[pool]) return;
    const Kept kept = read_kept(A, i, tid);
    const int r = A.req[i];
    if (r < 0 || r >= A.B) return;
    if (tid == 0) bad = 0, moved = INT32_MAX;
    __syncthreads();
    const int len = length_of(A, r);
    bool good = true;
    for (int j = tid; j < i; j += 256) good = good && A.req[j] != r;
    good = keep_is_good(A, i, r, len, kept, tid, 256) && good;
    if (!good) bad = 1;
    __syncthreads();
    if (bad) return;
    const int32_t *keep = A.keep + (int64_t)i * A.keep_ld;
    const int start = kept.start, k = kept.k;
    // entries from the first that moves on all move
    for (int j = tid; j < k; j += 256)
        if ((j == tid ? kept.s : keep[j]) != start + j) {
            atomicMin(&moved, j);
            break;
        }
    __syncthreads();
    if (moved >= k) return;
    if (A.row_bytes[pool] % 16 == 0) move_rows<u32x4>(A, r, pool, head, start, keep, moved, k);
    else move_rows<uint32_t>(A, r, pool, head, start, keep, moved, k);
}

}  // namespace

hipError_t launch_cache_release(const CacheArgs &a, bool compact, hipStream_t s) {
    if (compact) {
        int heads = 0;
        for (int l = 0; l < a.n_pools; ++l) heads = a.heads[l] > heads ? a.heads[l] : heads;
        cache_move_kernel<<<dim3((unsigned)heads, (unsigned)a.n, (unsigned)a.n_pools), 256, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        cache_release_kernel<true><<<1, kPlanNT, 0, s>>>(a);
    } else {
        cache_release_kernel<false><<<1, kPlanNT, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_cache_plan(const CacheArgs &a, bool fork, hipStream_t s) {
    if (fork) cache_plan_kernel<true><<<1, kPlanNT, 0, s>>>(a);
    else cache_plan_kernel<false><<<1, kPlanNT, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (fork) {
        // deep: a request's pages spread over as many workgroups as 2^16 in all allow
        const int64_t share = 65536 / ((int64_t)kCopyParts * a.n * a.n_pools);
        const unsigned pages = a.deep ? (unsigned)std::max<int64_t>(1, std::min(a.bt_ld, share)) : 1u;
        cache_copy_kernel<true><<<dim3(kCopyParts * pages, (unsigned)a.n, (unsigned)a.n_pools), 256, 0, s>>>(a);
    } else {
        cache_copy_kernel<false><<<dim3(kCopyParts, (unsigned)a.n, (unsigned)a.n_pools), 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace fm
