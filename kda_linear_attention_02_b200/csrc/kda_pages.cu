// kda_pages.cu -- pages of a cache on the device: copying, forking, freeing and compacting.
//
// The bookkeeping (references, tables, counts) is integer work of one block or less; what costs is the
// pages' bytes, read once and written once.  A call that moves pages is therefore at most two launches: one
// block that validates the call and lists the moves, and a grid that carries them out, 16 bytes per thread
// and load, several loads in flight.
//
// 48 states of 2 MB copied: 33.5 us = 6.0 TB/s.  12 states forked to 48 and freed again: 34 us, the plan 8, the moves 22
// (126 MB), the freeing 4; 200 states compacted: 22 us, the plan 6, the moves 13 (88 MB).  Calls on small pages take what
// their launches take on the host: 300 pages of 8 KB copied 7.0 us.
#include <algorithm>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kNt = 256;
constexpr int kUnroll = 8;                         // 16-byte loads in flight per thread
constexpr size_t kSlice = 16 * kNt * kUnroll;      // bytes one block moves between two looks at its list (32 KB)
constexpr int kMaxGroup = 64;                      // copies one block checks together
constexpr int kSms = 148;

// n16 16-byte words from src to dst (they do not overlap), by the whole block
__device__ __forceinline__ void move_words(uint4* __restrict__ dst, const uint4* __restrict__ src, int n16) {
    for (int b = threadIdx.x; b < n16; b += kNt * kUnroll) {
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (b + u * kNt < n16) x[u] = src[b + u * kNt];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (b + u * kNt < n16) dst[b + u * kNt] = x[u];
    }
}

// ---------------------------------------------------------------------------------------------- copy
//
// Which copies depend on each other is found without a sort: a block hashes the pages its own copies name
// (at most 2 x kMaxGroup), and counts over the whole list how often each of those is written and read.  The
// outcome for a copy does not depend on which block looks.
constexpr int kHash = 4 * kMaxGroup;

struct CopyArgs {
    char* dst;
    const char* src;
    long long n_dst, n_src;
    const int32_t* dst_pages;
    const int32_t* src_pages;
    int n, group, slices;        // copies per block, blocks per copy (one of the two is 1)
    size_t page_bytes;
    bool same, check;            // one pool; whether copies can depend on each other
    int* status;
};

__device__ __forceinline__ int page_of(const int32_t* tab, int i) { return tab ? tab[i] : i; }

// 0: nothing to do, 1: a copy, -1: out of range
__device__ __forceinline__ int copy_kind(const CopyArgs& a, int d, int s) {
    if (d < 0 || s < 0) return 0;
    if (d >= a.n_dst || s >= a.n_src) return -1;
    return a.same && d == s ? 0 : 1;
}

__device__ __forceinline__ uint32_t hash_at(int page) { return (static_cast<uint32_t>(page) * 2654435761u) >> 24; }
static_assert(kHash == 256, "hash_at gives 8 bits");

__device__ __forceinline__ int hash_find(const int* key, int page) {
    for (uint32_t p = hash_at(page);; p = (p + 1) & (kHash - 1)) {
        const int x = key[p];
        if (x == page) return static_cast<int>(p);
        if (x < 0) return -1;   // the table is at most half full
    }
}

__global__ void __launch_bounds__(kNt) pages_copy_kernel(const CopyArgs a) {
    __shared__ int s_d[kMaxGroup], s_s[kMaxGroup], key[kHash], writes[kHash], reads[kHash];
    grid_launch_dependents();
    grid_dependency_wait();
    const int t = threadIdx.x, i0 = blockIdx.x / a.slices * a.group, slice = blockIdx.x % a.slices;
    const int m = min(a.group, a.n - i0);
    if (t < m) {
        int d = page_of(a.dst_pages, i0 + t), s = page_of(a.src_pages, i0 + t);
        const int kind = copy_kind(a, d, s);
        if (kind < 0) set_status(a.status, KDA_ERR_DEVICE_INPUT);
        s_d[t] = kind > 0 ? d : -1;
        s_s[t] = s;
    }
    if (a.check) {
        key[t] = -1;
        writes[t] = reads[t] = 0;
        __syncthreads();
        auto insert = [&](int page) {
            for (uint32_t p = hash_at(page);; p = (p + 1) & (kHash - 1)) {
                const int was = atomicCAS(&key[p], -1, page);
                if (was == -1 || was == page) return;
            }
        };
        if (t < m && s_d[t] >= 0) {
            insert(s_d[t]);
            if (a.same) insert(s_s[t]);
        }
        __syncthreads();
        for (int j = t; j < a.n; j += kNt) {
            const int d = page_of(a.dst_pages, j), s = page_of(a.src_pages, j);
            if (copy_kind(a, d, s) <= 0) continue;
            const int x = hash_find(key, d);
            if (x >= 0) atomicAdd(&writes[x], 1);
            if (a.same) {
                const int y = hash_find(key, s);
                if (y >= 0) atomicAdd(&reads[y], 1);
            }
        }
        __syncthreads();
        if (t < m && s_d[t] >= 0) {
            const int x = hash_find(key, s_d[t]);
            bool bad = writes[x] > 1;
            if (a.same) bad |= reads[x] > 0 || writes[hash_find(key, s_s[t])] > 0;
            if (bad) {
                s_d[t] = -1;
                set_status(a.status, KDA_ERR_DEVICE_INPUT);
            }
        }
    }
    __syncthreads();
    const size_t per = a.slices > 1 ? ((a.page_bytes / 16 + a.slices - 1) / a.slices) * 16 : a.page_bytes;
    const size_t lo = slice * per, hi = min(a.page_bytes, lo + per);
    if (lo >= hi) return;
    for (int i = 0; i < m; ++i) {
        if (s_d[i] < 0) continue;
        move_words(reinterpret_cast<uint4*>(a.dst + s_d[i] * a.page_bytes + lo),
                   reinterpret_cast<const uint4*>(a.src + s_s[i] * a.page_bytes + lo), static_cast<int>((hi - lo) / 16));
    }
}

// ------------------------------------------------------------------------------------ moves of a plan

struct PlanHead {
    int n_moves;
    int pad[3];
};

// Carries out the moves (to, from; from < 0: zeros when `zero`, else nothing) in every plane of the pool.
// Work is handed out in slices of kSlice bytes, round robin over the blocks.
__device__ __forceinline__ void carry_out(char* pool, int n_planes, int n_pages, size_t page_bytes, const int2* moves,
                                          int n_moves, bool zero) {
    const long long slices = (page_bytes + kSlice - 1) / kSlice;
    const long long work = slices * n_planes * n_moves;
    for (long long x = blockIdx.x; x < work; x += gridDim.x) {
        const long long mv = x / (slices * n_planes), rest = x % (slices * n_planes);
        const int2 move = moves[mv];
        const size_t plane = static_cast<size_t>(rest / slices) * n_pages * page_bytes;
        const size_t lo = static_cast<size_t>(rest % slices) * kSlice, hi = min(page_bytes, lo + kSlice);
        uint4* dst = reinterpret_cast<uint4*>(pool + plane + move.x * page_bytes + lo);
        const int n16 = static_cast<int>((hi - lo) / 16);
        if (move.y >= 0) {
            move_words(dst, reinterpret_cast<const uint4*>(pool + plane + move.y * page_bytes + lo), n16);
        } else if (zero) {
            for (int b = threadIdx.x; b < n16; b += kNt) dst[b] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

__global__ void __launch_bounds__(kNt) pages_move_kernel(char* pool, int n_planes, int n_pages, size_t page_bytes,
                                                         const PlanHead* head,
                                                         const int2* moves, bool zero) {
    grid_launch_dependents();
    grid_dependency_wait();
    carry_out(pool, n_planes, n_pages, page_bytes, moves, head->n_moves, zero);
}

// Sum of x over the threads of the block ahead of this one, and over all of them (1024 threads).
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) y += z;
    }
    __syncthreads();   // the sums of the call before have been read
    if (lane == 31) warp_sums[w] = y;
    __syncthreads();
    if (w == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += z;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    return y - x + (w ? warp_sums[w - 1] : 0);
}

// ---------------------------------------------------------------------------------------------- fork

struct ForkEntry {
    int have, keep, first, count;   // pages of the parent, those shared, rank of the first new page, new pages
};

// Validates the call, finds the free pages, and writes the bookkeeping and the list of moves; nothing but the
// workspace is written before the whole call is known to be good.  `opened` (dynamic shared memory) has a bit
// for each row.
__global__ void __launch_bounds__(1024) pages_fork_plan_kernel(int32_t* refs, int n_pages, int32_t* table, int32_t* counts,
                                                               int n_rows, int max_pages, const int32_t* parents,
                                                               const int32_t* children, const int32_t* n_shared,
                                                               const int32_t* n_fresh, int n, PlanHead* head,
                                                               ForkEntry* entries, int2* moves, int* status) {
    extern __shared__ uint32_t opened[];
    __shared__ int warp_sums[32];
    __shared__ ForkEntry near_entries[1024];   // the entries of a call that has no more
    grid_launch_dependents();
    grid_dependency_wait();
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    if (n <= 1024) entries = near_entries;
    // references of the first pages, which are looked at last: the block's steps each wait for a load
    int ahead[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) ahead[u] = 4 * t + u < n_pages ? refs[4 * t + u] : 1;
    for (int i = t; i < (n_rows + 31) / 32; i += 1024) opened[i] = 0u;
    __syncthreads();
    bool bad = false;
    int needed = 0;   // at most n max_pages, which the host keeps below 2^30
    for (int base = 0; base < n; base += 1024) {
        const int i = base + t;
        ForkEntry e{0, 0, 0, 0};
        if (i < n) {
            const int p = parents[i], c = children[i], fresh = n_fresh ? n_fresh[i] : 0;
            bool ok = c >= 0 && c < n_rows && p >= -1 && p < n_rows && fresh >= 0 && fresh <= max_pages;
            if (ok) {
                e.have = p >= 0 ? counts[p] : 0;
                e.keep = p == c ? e.have : p >= 0 && n_shared ? n_shared[i] : 0;
                ok = e.have >= 0 && e.have <= max_pages && e.keep >= 0 && e.keep <= e.have && fresh <= max_pages - e.have &&
                     (p == c || counts[c] == 0) && !(atomicOr(&opened[c >> 5], 1u << (c & 31)) >> (c & 31) & 1u);
            }
            e.count = ok ? e.have - e.keep + fresh : 0;
            if (!ok) e.have = 0;
            bad |= !ok;
        }
        int total;
        e.first = needed + block_scan(e.count, warp_sums, total);
        if (i < n) entries[i] = e;
        needed += total;
    }
    __syncthreads();
    // no row that the call opens or extends is another entry's parent, and the parents' pages are in use
    for (int i = w; i < n; i += 32) {
        const int p = parents[i], have = entries[i].have;
        if (p >= 0 && p < n_rows && p != children[i]) bad |= (opened[p >> 5] >> (p & 31)) & 1u;
        for (int j = lane; j < have; j += 32) {
            const int page = table[static_cast<size_t>(p) * max_pages + j];
            bad |= page < 0 || page >= n_pages || refs[page] <= 0;
        }
    }
    if (__syncthreads_or(bad)) {
        if (t == 0) {
            head->n_moves = 0;
            set_status(status, KDA_ERR_DEVICE_INPUT);
        }
        return;
    }
    // the lowest free pages, as many as needed
    int found = 0;
    for (int base = 0; base < n_pages && found < needed; base += 4096) {
        int f[4], k = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int p = base + 4 * t + u;
            f[u] = base == 0 ? ahead[u] == 0 : p < n_pages && refs[p] == 0;
            k += f[u];
        }
        int total, at = found + block_scan(k, warp_sums, total);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (f[u]) {
                if (at < needed) moves[at].x = base + 4 * t + u;
                ++at;
            }
        found += total;
    }
    if (found < needed) {
        if (t == 0) {
            head->n_moves = 0;
            set_status(status, KDA_ERR_NO_PAGES);
        }
        return;
    }
    __syncthreads();   // the free pages are listed, and no reference changes before all have been read
    for (int i = w; i < n; i += 32) {
        const ForkEntry e = entries[i];
        const int p = parents[i], c = children[i];
        for (int j = (p == c ? e.keep : 0) + lane; j < e.keep + e.count; j += 32) {
            const int theirs = j < e.have ? table[static_cast<size_t>(p) * max_pages + j] : -1;
            int page = theirs;
            if (j < e.keep) {
                atomicAdd(&refs[page], 1);
            } else {
                int2* mv = &moves[e.first + j - e.keep];
                page = mv->x;
                mv->y = theirs;
                refs[page] = 1;
            }
            table[static_cast<size_t>(c) * max_pages + j] = page;
        }
        if (lane == 0) counts[c] = e.keep + e.count;
    }
    if (t == 0) head->n_moves = needed;
}

// ---------------------------------------------------------------------------------------------- free

// A warp per row.  The count is taken by an exchange, so that a row named twice is freed once.
__global__ void __launch_bounds__(kNt) pages_free_kernel(int32_t* refs, int n_pages, const int32_t* table,
                                                         int32_t* counts, int n_rows, int max_pages,
                                                         const int32_t* rows, int n, int* status) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int i = blockIdx.x * (kNt / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= n) return;
    const int r = rows[i];
    bool bad = r < 0 || r >= n_rows;
    // A count that no row can have stays, with the row's pages and their references.  (Counts change here by becoming 0
    // alone, so that one which passed may at most be 0 by the time it is taken.)
    int c = 0;
    if (!bad && lane == 0) {
        c = atomicAdd(&counts[r], 0);
        if (c > 0 && c <= max_pages) c = atomicExch(&counts[r], 0);
    }
    c = __shfl_sync(0xffffffffu, c, 0);
    if (c < 0 || c > max_pages) {
        bad = true;
        c = 0;
    }
    for (int j = lane; j < c; j += 32) {
        const int page = table[static_cast<size_t>(r) * max_pages + j];
        if (page < 0 || page >= n_pages) {
            bad = true;
        } else if (atomicSub(&refs[page], 1) <= 0) {
            atomicAdd(&refs[page], 1);
            bad = true;
        }
    }
    if (bad) set_status(status, KDA_ERR_DEVICE_INPUT);
}

// ------------------------------------------------------------------------------------------- compact

// Lists the moves (hole, page) and writes remap; refs follow once all of them have been read.
__global__ void __launch_bounds__(1024) pages_compact_plan_kernel(int32_t* refs, int n_pages, int32_t* __restrict__ remap,
                                                                  int32_t* n_live_out, PlanHead* head, int2* moves) {
    __shared__ int warp_sums[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int t = threadIdx.x;
    int mine = 0, n_live;
    for (int p = t; p < n_pages; p += 1024) mine += refs[p] > 0;
    block_scan(mine, warp_sums, n_live);
    int holes = 0, movers = 0;
    for (int base = 0; base < n_pages; base += 4096) {
        int r[4], k = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int p = base + 4 * t + u;
            r[u] = p < n_pages ? refs[p] : 0;
            k += p < n_live ? r[u] <= 0 : r[u] > 0;   // a page is a hole or a mover by its place
        }
        // holes come before movers in page order: one running count serves both, split where it passes n_live
        int total, at = holes + movers + block_scan(k, warp_sums, total);
        int holes_here = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int p = base + 4 * t + u;
            if (p >= n_pages) continue;
            if (p < n_live) {
                if (r[u] > 0) {
                    remap[p] = p;
                } else {
                    moves[at++].x = p;
                    ++holes_here;
                }
            } else if (r[u] > 0) {
                remap[p] = at++;   // its rank behind all holes, for now
            } else {
                remap[p] = -1;
            }
        }
        int holes_total;
        block_scan(holes_here, warp_sums, holes_total);
        holes += holes_total;
        movers += total - holes_total;
    }
    __syncthreads();
    // as many holes among the first n_live pages as pages in use behind them
    for (int p = n_live + t; p < n_pages; p += 1024)
        if (refs[p] > 0) moves[remap[p] - holes].y = p;
    __syncthreads();
    for (int m = t; m < holes; m += 1024) {
        const int2 mv = moves[m];
        refs[mv.x] = refs[mv.y];
        refs[mv.y] = 0;
        remap[mv.x] = -1;
        remap[mv.y] = mv.x;
    }
    if (t == 0) {
        head->n_moves = holes;
        if (n_live_out) *n_live_out = n_live;
    }
}

__global__ void __launch_bounds__(kNt) pages_compact_kernel(char* pool, int n_planes, int n_pages, size_t page_bytes,
                                                            const PlanHead* head,
                                                            const int2* moves, int32_t* __restrict__ table,
                                                            const int32_t* counts, int n_rows, int max_pages,
                                                            const int32_t* remap, int* status) {
    grid_launch_dependents();
    grid_dependency_wait();
    const long long entries = static_cast<long long>(n_rows) * max_pages;
    bool bad = false;
    for (long long x = static_cast<long long>(blockIdx.x) * kNt + threadIdx.x; x < entries;
         x += static_cast<long long>(gridDim.x) * kNt) {
        const int r = static_cast<int>(x / max_pages), j = static_cast<int>(x % max_pages);
        if (j >= counts[r]) continue;
        const int page = table[x];
        const int to = page >= 0 && page < n_pages ? remap[page] : -1;
        if (to >= 0) table[x] = to;
        else bad = true;
    }
    if (bad) set_status(status, KDA_ERR_DEVICE_INPUT);
    carry_out(pool, n_planes, n_pages, page_bytes, moves, head->n_moves, false);
}

// A launch that may start while the kernel before it, which lets it, still writes: the kernels launched so wait before
// they read, and declare nothing const and __restrict__ (which would let them read by the non-coherent path).
template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr size_t kHeadBytes = 256;
constexpr int kMaxRows = 1 << 20;   // a bit for each row in one block's shared memory (128 KB)
constexpr long long kMaxMoves = 1ll << 30;
constexpr int kMaxList = 1 << 30;   // pages of a pool, entries of a list: what the kernels' 32-bit loops can step over

size_t fork_bytes(int n, int max_pages) {
    return kHeadBytes + round256(sizeof(ForkEntry) * static_cast<size_t>(n)) +
           round256(sizeof(int2) * static_cast<size_t>(n) * max_pages);
}
size_t compact_bytes(int n_pages) { return kHeadBytes + round256(sizeof(int2) * (static_cast<size_t>(n_pages) / 2 + 1)); }

// Blocks that carry out up to `moves` moves: every slice its own, at most eight blocks per SM.
unsigned move_blocks(size_t page_bytes, int n_planes, long long moves) {
    const long long slices = static_cast<long long>((page_bytes + kSlice - 1) / kSlice);
    const long long work = moves > 0x7fffffffLL / (slices * n_planes) ? 0x7fffffffLL : slices * n_planes * moves;
    return static_cast<unsigned>(std::max(1LL, std::min(work, 8LL * kSms)));
}

bool pool_ok(int n_planes, int n_pages, size_t page_bytes) {
    // every byte offset fits 63 bits
    return n_planes > 0 && n_pages >= 0 && n_pages <= kMaxList && page_bytes > 0 && page_bytes % 16 == 0 && page_bytes <= (size_t{1} << 30) &&
           static_cast<double>(page_bytes) * n_pages * n_planes < 9e18;
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_pages_copy(void* dst, int64_t n_dst, const void* src, int64_t n_src, const int32_t* dst_pages,
                            const int32_t* src_pages, int n, size_t page_bytes, kda_stream_t stream) {
    if (n < 0 || n > kMaxList || n_dst < 0 || n_src < 0 || n_dst > 0x7fffffffLL || n_src > 0x7fffffffLL) return KDA_ERR_ARG;
    if (page_bytes == 0 || page_bytes % 16 != 0 || page_bytes > (size_t{1} << 30)) return KDA_ERR_ARG;
    if ((!dst_pages && n > n_dst) || (!src_pages && n > n_src)) return KDA_ERR_ARG;
    if (n == 0) return KDA_OK;
    if ((!dst && n_dst > 0) || (!src && n_src > 0)) return KDA_ERR_ARG;
    if (!aligned(dst, 16) || !aligned(src, 16) || (dst_pages && !aligned(dst_pages, 4)) ||
        (src_pages && !aligned(src_pages, 4)))
        return KDA_ERR_ALIGN;
    const uintptr_t d0 = reinterpret_cast<uintptr_t>(dst), s0 = reinterpret_cast<uintptr_t>(src);
    if (d0 != s0 && d0 < s0 + n_src * page_bytes && s0 < d0 + n_dst * page_bytes) return KDA_ERR_ARG;
    CopyArgs a{};
    a.dst = static_cast<char*>(dst); a.src = static_cast<const char*>(src); a.n_dst = n_dst; a.n_src = n_src;
    a.dst_pages = dst_pages; a.src_pages = src_pages; a.n = n; a.page_bytes = page_bytes;
    a.same = d0 == s0;
    a.check = dst_pages || a.same;
    // large pages are split over blocks, small ones grouped: a block moves up to about kSlice bytes, and there
    // are enough blocks for the SMs before copies share one
    const size_t slices = (page_bytes + kSlice - 1) / kSlice;
    a.slices = static_cast<int>(std::min<size_t>(slices, 65536));
    const int by_bytes = static_cast<int>(std::max<size_t>(1, kSlice / page_bytes));
    a.group = std::max(1, std::min({by_bytes, kMaxGroup, n / (4 * kSms)}));
    const long long blocks = static_cast<long long>((n + a.group - 1) / a.group) * a.slices;
    if (blocks > 0x7fffffffLL) return KDA_ERR_ARG;
    a.status = status_ptr();
    if (!a.status) return KDA_ERR_CUDA;
    return launch_chained(pages_copy_kernel, static_cast<unsigned>(blocks), kNt, 0, reinterpret_cast<cudaStream_t>(stream),
                          a) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_pages_fork_workspace_bytes(int n, int max_pages) {
    if (n < 0 || max_pages <= 0 || static_cast<long long>(n) * max_pages > kMaxMoves) return 0;
    return fork_bytes(n, max_pages);
}

kda_status_t kda_pages_fork(void* pool, int n_planes, int n_pages, size_t page_bytes, int32_t* refs, int32_t* table,
                            int32_t* counts, int n_rows, int max_pages, const int32_t* parents,
                            const int32_t* children, const int32_t* n_shared, const int32_t* n_fresh, int n,
                            int zero_fresh, void* workspace, size_t ws_bytes, kda_stream_t stream) {
    if (n < 0 || !pool_ok(n_planes, n_pages, page_bytes) || n_rows < 0 || n_rows > kMaxRows || max_pages <= 0 ||
        static_cast<long long>(n) * max_pages > kMaxMoves || (zero_fresh != 0 && zero_fresh != 1))
        return KDA_ERR_ARG;
    if (n == 0) return KDA_OK;
    if ((!pool && n_pages > 0) || (!refs && n_pages > 0) || !table || !counts || !parents || !children || !workspace)
        return KDA_ERR_ARG;
    const void* ints[] = {refs, table, counts, parents, children, n_shared, n_fresh};
    for (const void* p : ints)
        if (!aligned(p, 4)) return KDA_ERR_ALIGN;
    if (!aligned(pool, 16) || !aligned(workspace, 256)) return KDA_ERR_ALIGN;
    if (ws_bytes < fork_bytes(n, max_pages)) return KDA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    PlanHead* head = reinterpret_cast<PlanHead*>(ws);
    ForkEntry* entries = reinterpret_cast<ForkEntry*>(ws + kHeadBytes);
    int2* moves = reinterpret_cast<int2*>(ws + kHeadBytes + round256(sizeof(ForkEntry) * static_cast<size_t>(n)));
    int* st = status_ptr();
    if (!st) return KDA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = (static_cast<size_t>(n_rows) + 31) / 32 * 4;
    static SmemLimit limit;
    if (smem > 24576 && limit.raise(reinterpret_cast<const void*>(&pages_fork_plan_kernel), kMaxRows / 8) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (launch_chained(pages_fork_plan_kernel, 1, 1024, smem, s, refs, n_pages, table, counts, n_rows, max_pages, parents,
                       children, n_shared, n_fresh, n, head, entries, moves, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    return launch_chained(pages_move_kernel, move_blocks(page_bytes, n_planes, static_cast<long long>(n) * max_pages), kNt, 0,
                          s, static_cast<char*>(pool), n_planes, n_pages, page_bytes, head, moves, zero_fresh != 0) ==
                   cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_pages_free(int32_t* refs, int n_pages, const int32_t* table, int32_t* counts, int n_rows, int max_pages,
                            const int32_t* rows, int n, kda_stream_t stream) {
    if (n < 0 || n > kMaxList || n_pages < 0 || n_pages > kMaxList || n_rows < 0 || max_pages <= 0) return KDA_ERR_ARG;
    if (n == 0) return KDA_OK;
    if ((!refs && n_pages > 0) || !rows || (n_rows > 0 && (!table || !counts))) return KDA_ERR_ARG;
    if (!aligned(refs, 4) || !aligned(table, 4) || !aligned(counts, 4) || !aligned(rows, 4)) return KDA_ERR_ALIGN;
    int* st = status_ptr();
    if (!st) return KDA_ERR_CUDA;
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(n) + kNt / 32 - 1) / (kNt / 32));
    return launch_chained(pages_free_kernel, blocks, kNt, 0, reinterpret_cast<cudaStream_t>(stream), refs, n_pages, table,
                          counts, n_rows, max_pages, rows, n, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_pages_compact_workspace_bytes(int n_pages) {
    return n_pages < 0 || n_pages > kMaxList ? 0 : compact_bytes(n_pages);
}

kda_status_t kda_pages_compact(void* pool, int n_planes, int n_pages, size_t page_bytes, int32_t* refs, int32_t* table,
                               const int32_t* counts, int n_rows, int max_pages, int32_t* remap, int32_t* n_live,
                               void* workspace, size_t ws_bytes, kda_stream_t stream) {
    if (!pool_ok(n_planes, n_pages, page_bytes) || n_rows < 0 || max_pages <= 0) return KDA_ERR_ARG;
    if (n_pages > 0 && (!pool || !refs || !remap)) return KDA_ERR_ARG;
    if ((n_rows > 0 && (!table || !counts)) || !workspace) return KDA_ERR_ARG;
    if (!aligned(pool, 16) || !aligned(workspace, 256)) return KDA_ERR_ALIGN;
    const void* ints[] = {refs, table, counts, remap, n_live};
    for (const void* p : ints)
        if (!aligned(p, 4)) return KDA_ERR_ALIGN;
    if (ws_bytes < compact_bytes(n_pages)) return KDA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    PlanHead* head = reinterpret_cast<PlanHead*>(ws);
    int2* moves = reinterpret_cast<int2*>(ws + kHeadBytes);
    int* st = status_ptr();
    if (!st) return KDA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch_chained(pages_compact_plan_kernel, 1, 1024, 0, s, refs, n_pages, remap, n_live, head, moves) != cudaSuccess)
        return KDA_ERR_CUDA;
    return launch_chained(pages_compact_kernel, move_blocks(page_bytes, n_planes, n_pages / 2 + 1), kNt, 0, s,
                          static_cast<char*>(pool), n_planes, n_pages, page_bytes, head, moves, table, counts, n_rows,
                          max_pages, remap, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
