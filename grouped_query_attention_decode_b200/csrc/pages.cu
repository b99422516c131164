// Pages of a paged cache held by several sequences: forking, freeing, reserving (with copy on
// write), compacting and copying.
//
// The state is the block tables, the lengths and one count per page, the number of table entries
// that hold it; a page is free when its count is zero, so there is no list to keep in step.  All
// of it is integers: counts change by atomic additions, whose sum does not depend on their order,
// and free pages are taken lowest number first by a scan, so every call has one result.  The
// calls on tables are bound by their latency (a few dependent reads): fork, reserve and copy of 64
// beams of 4096 rows take 14 us together.  The copy is bound by HBM: 771 MB in 131 us, 5.9 TB/s.
#include <cuda_runtime_api.h>

#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "launch.h"

namespace gqa {

namespace {

__device__ __forceinline__ void flag(int32_t *status, int bits) {
    if (status != nullptr) atomicOr(status, bits);
}

// A table entry as a page, -1 for none.
__device__ __forceinline__ int entry_page(int e, int n_pages, int32_t *status) {
    if (e >= 0 && e < n_pages) return e;
    if (e != -1) flag(status, GQA_STATUS_PAGE_RANGE);
    return -1;
}

__device__ __forceinline__ void add_holders(int32_t *refs, int page, int delta, int32_t *status) {
    if (atomicAdd(refs + page, delta) + delta < 0) flag(status, GQA_STATUS_PAGE_REFS);
}

// ---------------------------------------------------------------------------------- fork, free
// Blocks [0, B_out) copy rows, blocks [B_out, B_out + B_in) count: a row with c children adds
// c - 1 to each of its pages, so a row that has one child costs no atomics.
__global__ void __launch_bounds__(256)
pages_fork_kernel(const int32_t *__restrict__ parents, const int32_t *__restrict__ table_in,
                  const int32_t *__restrict__ lens_in, int B_in, int32_t *__restrict__ table_out,
                  int32_t *__restrict__ lens_out, int B_out, int max_pages, int32_t *refs, int n_pages,
                  int32_t *status) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x;
    if (static_cast<int>(blockIdx.x) < B_out) {
        const int i = blockIdx.x, par = parents[i];
        const bool some = par >= 0 && par < B_in;
        if (tid == 0) {
            if (!some && par != -1) flag(status, GQA_STATUS_INDEX_RANGE);
            lens_out[i] = some ? lens_in[par] : 0;
        }
        const int32_t *src = table_in + static_cast<long long>(some ? par : 0) * max_pages;
        int32_t *dst = table_out + static_cast<long long>(i) * max_pages;
        for (int j = tid; j < max_pages; j += 256) dst[j] = some ? src[j] : -1;
        return;
    }
    const int i = blockIdx.x - B_out;
    int c = 0;
    for (int j0 = 0; j0 < B_out; j0 += 256) {
        const int j = j0 + tid;
        c += __syncthreads_count(j < B_out && parents[j] == i);
    }
    if (c == 1) return;
    const int32_t *row = table_in + static_cast<long long>(i) * max_pages;
    for (int j = tid; j < max_pages; j += 256) {
        const int page = entry_page(row[j], n_pages, status);
        if (page >= 0) add_holders(refs, page, c - 1, status);
    }
}

// One block per listed sequence.  Entries are taken by exchange, so a sequence that is listed
// twice is freed once.
__global__ void __launch_bounds__(256)
pages_free_kernel(const int32_t *__restrict__ seqs, int32_t *table, int32_t *lens, int B, int max_pages,
                  int32_t *refs, int n_pages, int32_t *status) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int s = seqs[blockIdx.x];
    if (s < 0 || s >= B) {
        if (threadIdx.x == 0) flag(status, GQA_STATUS_INDEX_RANGE);
        return;
    }
    int32_t *row = table + static_cast<long long>(s) * max_pages;
    for (int j = threadIdx.x; j < max_pages; j += 256) {
        if (row[j] == -1) continue;
        const int page = entry_page(atomicExch(row + j, -1), n_pages, status);
        if (page >= 0) add_holders(refs, page, -1, status);
    }
    if (threadIdx.x == 0) lens[s] = 0;
}

// ---------------------------------------------------------------------------------- reserve
// What one block needs of a page that a sequence is about to write: how many of the sequences in
// this call would write it, the last of them, and its holders on entry.
struct PageUse {
    int writers, last, holders, pad;
};

struct ReserveParams {
    int32_t *table;
    const int32_t *lens;
    int32_t *refs, *copies, *status;
    PageUse *use;   // [n_pages], only the entries of pages in question
    int32_t *free;  // [n_pages] the free pages found, in ascending order
    int B, max_pages, page_size, rows, n_pages, lanes;  // lanes: threads per sequence, 1 or 32
};

constexpr int kReserveThreads = 1024;

// Inclusive scan over the block of one value per thread; `total` gets the sum.
template <class T>
__device__ T block_scan(T v, T *warp_sums, T &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(kFullMask, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // warp_sums of a scan before has been read
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    T w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(kFullMask, w, o);
        if (lane >= o) w += u;
    }
    total = __shfl_sync(kFullMask, w, 31);
    const T before = __shfl_sync(kFullMask, w, (warp + 31) & 31);
    return warp > 0 ? v + before : v;
}

// The table slots that sequence b's next rows fall into, none when they do not fit.
__device__ __forceinline__ void slots_of(const ReserveParams &p, int b, int &first, int &last, int &len) {
    len = p.lens[b];
    first = 0;
    last = -1;
    if (len >= 0 && static_cast<long long>(len) + p.rows <= static_cast<long long>(p.max_pages) * p.page_size) {
        first = len / p.page_size;
        last = (len + p.rows - 1) / p.page_size;
    }
}

// Does slot (page, -1 for none) of sequence b need a new page?  A page with other holders does --
// but when everyone who holds it is about to write, the last of them keeps it.
__device__ __forceinline__ bool needs_page(const ReserveParams &p, int page, int b) {
    if (page < 0) return true;
    const PageUse u = p.use[page];
    return u.holders > 1 && !(u.writers >= u.holders && u.last == b);
}

// One block.  Sequences are served in order while free pages last.
__global__ void __launch_bounds__(kReserveThreads) pages_reserve_kernel(const ReserveParams p) {
    __shared__ long long sums[32];
    __shared__ int s_found;
    const int tid = threadIdx.x, W = p.lanes, lane = tid & (W - 1);
    const int per_round = kReserveThreads / W;
    grid_dependency_wait();
    grid_launch_dependents();
    // A sequence's threads take its slots W at a time; a round takes per_round sequences.
    auto for_slots = [&](auto fn) {
        for (int b0 = 0; b0 < p.B; b0 += per_round) {
            const int b = b0 + tid / W;
            if (b >= p.B) continue;
            int first, last, len;
            slots_of(p, b, first, last, len);
            for (int j = first + lane; j <= last; j += W) fn(b, p.table[static_cast<long long>(b) * p.max_pages + j]);
        }
    };
    for_slots([&](int b, int e) {
        const int page = entry_page(e, p.n_pages, p.status);
        if (page < 0) return;
        const int holders = p.refs[page];
        if (holders < 1) flag(p.status, GQA_STATUS_PAGE_REFS);
        p.use[page] = PageUse{0, -1, holders, 0};  // everyone writes the same
    });
    __syncthreads();
    for_slots([&](int b, int e) {
        const int page = entry_page(e, p.n_pages, nullptr);
        if (page < 0 || p.use[page].holders < 2) return;
        atomicAdd(&p.use[page].writers, 1);
        atomicMax(&p.use[page].last, b);
    });
    __syncthreads();
    // pages needed in all
    long long mine = 0, demand;
    for_slots([&](int b, int e) { mine += needs_page(p, entry_page(e, p.n_pages, nullptr), b); });
    block_scan(mine, sums, demand);
    // the lowest free pages, 16 to a thread and round: four runs of 4 * 1024 pages, whose counts
    // share one scan (16 bits each)
    int found = 0;
    const int4 *refs4 = reinterpret_cast<const int4 *>(p.refs);
    for (int base = 0; base < p.n_pages && found < demand; base += 16 * kReserveThreads) {
        unsigned char is_free[4];
        long long packed = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int at = base + (r * kReserveThreads + tid) * 4;
            int4 v = make_int4(1, 1, 1, 1);
            if (at + 3 < p.n_pages) {
                v = refs4[at / 4];
            } else {
                if (at < p.n_pages) v.x = p.refs[at];
                if (at + 1 < p.n_pages) v.y = p.refs[at + 1];
                if (at + 2 < p.n_pages) v.z = p.refs[at + 2];
            }
            is_free[r] = (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
            packed |= static_cast<long long>(__popc(is_free[r])) << (16 * r);
        }
        long long total;
        const long long incl = block_scan(packed, sums, total);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            int rank = found + static_cast<int>((incl >> (16 * r)) & 0xffff) - __popc(is_free[r]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (is_free[r] >> k & 1) {
                    if (rank < demand) p.free[rank] = base + (r * kReserveThreads + tid) * 4 + k;
                    ++rank;
                }
            found += static_cast<int>((total >> (16 * r)) & 0xffff);
        }
    }
    if (tid == 0) s_found = found;
    __syncthreads();
    found = s_found;
    // hand them out
    long long before = 0;  // pages needed by the sequences of earlier rounds
    for (int b0 = 0; b0 < p.B; b0 += per_round) {
        const int b = b0 + tid / W;
        int first = 0, last = -1, len = 0;
        if (b < p.B) slots_of(p, b, first, last, len);
        int32_t *row = p.table + static_cast<long long>(b < p.B ? b : 0) * p.max_pages;
        int count = 0;
        for (int j = first + lane; j <= last; j += W) count += needs_page(p, entry_page(row[j], p.n_pages, nullptr), b);
        if (W == 32) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(kFullMask, count, o);
        }
        long long round;  // every thread of a sequence gets the same `upto`: its first one adds the count
        const long long upto = before + block_scan(static_cast<long long>(lane == 0 ? count : 0), sums, round);
        before += round;
        const bool refused = b < p.B && last < 0;
        const bool served = upto <= found;
        if (b < p.B && lane == 0) {
            if (refused) flag(p.status, GQA_STATUS_APPEND_OVERFLOW);
            else if (!served) flag(p.status, GQA_STATUS_POOL_FULL);
        }
        if (b >= p.B) continue;  // whole groups of W threads; no barrier below
        int2 pair = make_int2(-1, -1);
        int next = static_cast<int>(upto) - count;
        for (int j0 = first; served && !refused && j0 <= last; j0 += W) {
            const int j = j0 + lane;
            const int page = j <= last ? entry_page(row[j], p.n_pages, nullptr) : -1;
            const bool need = j <= last && needs_page(p, page, b);
            int at = next;
            if (W == 32) {
                const uint32_t m = __ballot_sync(kFullMask, need);
                at += __popc(m & ((1u << lane) - 1u));
                next += __popc(m);
            } else {
                next += need;
            }
            if (!need) continue;
            const int fresh = p.free[at];
            row[j] = fresh;
            p.refs[fresh] = 1;
            if (page >= 0) {
                atomicSub(p.refs + page, 1);
                if (j == first && len % p.page_size != 0) pair = make_int2(page, fresh);
            }
        }
        if (lane == 0) reinterpret_cast<int2 *>(p.copies)[b] = pair;  // slot `first` is lane 0's
    }
}

// ---------------------------------------------------------------------------------- compact
// With n live pages, the live ones numbered n and up go, in ascending order, to the free ones
// below n.  Three launches: live pages per block of pages; the ranks of what moves; the moves.
constexpr int kCompactBlock = 4096;  // pages per block, four to a thread

struct CompactParams {
    int32_t *table, *refs, *copies, *n_live, *status;
    int32_t *count;  // [blocks] live pages
    int32_t *rank;   // [n_pages] of a live page past the end: its place among those
    long long entries;
    int n_pages, blocks, most;  // most: pairs in `copies`
};

__device__ __forceinline__ int4 load_refs(const CompactParams &p, int at) {
    int4 v = make_int4(0, 0, 0, 0);
    if (at + 3 < p.n_pages) return *reinterpret_cast<const int4 *>(p.refs + at);
    if (at < p.n_pages) v.x = p.refs[at];
    if (at + 1 < p.n_pages) v.y = p.refs[at + 1];
    if (at + 2 < p.n_pages) v.z = p.refs[at + 2];
    return v;
}

__global__ void __launch_bounds__(1024) compact_count_kernel(const CompactParams p) {
    __shared__ int sums[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int4 v = load_refs(p, blockIdx.x * kCompactBlock + threadIdx.x * 4);
    int total;
    block_scan((v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0), sums, total);
    if (threadIdx.x == 0) p.count[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) compact_rank_kernel(const CompactParams p) {
    __shared__ int sums[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x;
    int all = 0, before = 0;
    for (int i = tid; i < p.blocks; i += 1024) {
        const int c = __ldcg(p.count + i);
        all += c;
        if (i < static_cast<int>(blockIdx.x)) before += c;
    }
    int n, first;
    block_scan(all, sums, n);
    block_scan(before, sums, first);
    // live pages numbered below n: those of whole blocks and of the block that n falls into
    const int edge = n / kCompactBlock;
    int low = 0, below;
    for (int i = tid; i < edge; i += 1024) low += __ldcg(p.count + i);
    {
        const int at = edge * kCompactBlock + tid * 4;
        const int4 v = load_refs(p, at);
        low += (at < n && v.x > 0) + (at + 1 < n && v.y > 0) + (at + 2 < n && v.z > 0) + (at + 3 < n && v.w > 0);
    }
    block_scan(low, sums, below);
    const int moves = n - below;
    const int at = blockIdx.x * kCompactBlock + tid * 4;
    const int4 v = load_refs(p, at);
    const int live[4] = {v.x > 0, v.y > 0, v.z > 0, v.w > 0};
    const int c = live[0] + live[1] + live[2] + live[3];
    int total;
    int seen = first + block_scan(c, sums, total) - c;  // live pages before this thread's
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int page = at + k;
        if (page >= p.n_pages) break;
        if (page >= n) {
            p.rank[page] = live[k] ? seen - below : -1;
            if (live[k] && seen - below < p.most) p.copies[2 * (seen - below)] = page;
        } else if (!live[k] && page - seen < p.most) {
            p.copies[2 * (page - seen) + 1] = page;
        }
        seen += live[k];
    }
    for (int i = blockIdx.x * 1024 + tid; i < p.most; i += gridDim.x * 1024)
        if (i >= moves) reinterpret_cast<int2 *>(p.copies)[i] = make_int2(-1, -1);
    if (blockIdx.x == 0 && tid == 0) *p.n_live = n;
}

__global__ void __launch_bounds__(256) compact_move_kernel(const CompactParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long t0 = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<long long>(gridDim.x) * 256;
    const int n = __ldcg(p.n_live);
    for (long long i = t0; i < p.most; i += step) {
        const int2 m = __ldcg(reinterpret_cast<const int2 *>(p.copies) + i);
        if (m.x < 0) break;  // the moves stand at the front
        p.refs[m.y] = p.refs[m.x];
        p.refs[m.x] = 0;
    }
    for (long long i = t0; i < p.entries; i += step) {
        const int page = entry_page(p.table[i], p.n_pages, p.status);
        if (page < n) continue;  // also -1
        const int rank = __ldcg(p.rank + page);
        if (rank < 0 || rank >= p.most) flag(p.status, GQA_STATUS_PAGE_REFS);  // held, but counted as free
        else p.table[i] = __ldcg(p.copies + 2 * rank + 1);
    }
}

// ---------------------------------------------------------------------------------- copy
constexpr int kCopyThreads = 256, kCopyVecs = 4;  // 16-byte vectors per thread and item: 16 KB items

__global__ void __launch_bounds__(kCopyThreads)
pages_copy_kernel(uint4 *k_pool, uint4 *v_pool, const int2 *__restrict__ pairs, int n, long long page_vecs, int n_pages,
                  int32_t *status) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int ITEM = kCopyThreads * kCopyVecs;
    const int items = static_cast<int>((page_vecs + ITEM - 1) / ITEM);  // per page and pool
    const long long all = 2ll * n * items;
    for (long long w = blockIdx.x; w < all; w += gridDim.x) {
        const int pair = static_cast<int>(w / (2 * items)), rest = static_cast<int>(w - 2ll * pair * items);
        const int2 m = __ldg(pairs + pair);
        if (m.x == -1 && m.y == -1) continue;
        if (m.x < 0 || m.y < 0 || m.x >= n_pages || m.y >= n_pages) {
            if (threadIdx.x == 0) flag(status, GQA_STATUS_INDEX_RANGE);
            continue;
        }
        uint4 *pool = rest < items ? k_pool : v_pool;
        const long long at = static_cast<long long>(rest < items ? rest : rest - items) * ITEM + threadIdx.x;
        const uint4 *src = pool + m.x * page_vecs;
        uint4 *dst = pool + m.y * page_vecs;
        uint4 v[kCopyVecs];
#pragma unroll
        for (int u = 0; u < kCopyVecs; ++u)
            if (at + u * kCopyThreads < page_vecs) v[u] = __ldcs(src + at + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kCopyVecs; ++u)
            if (at + u * kCopyThreads < page_vecs) __stcs(dst + at + u * kCopyThreads, v[u]);
    }
}

// ---------------------------------------------------------------------------------- host
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// The sizes of a table: entries have to be countable in 32 bits.
bool table_fits(int B, int max_pages) { return B > 0 && max_pages > 0 && static_cast<long long>(B) * max_pages <= (1ll << 30); }

template <class... K, class... A>
int launch(void (*kern)(K...), int grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<K>(args)...) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" int gqa_pages_fork(const int32_t *parents, const int32_t *table_in, const int32_t *lens_in, int B_in,
                              int32_t *table_out, int32_t *lens_out, int B_out, int max_pages, int32_t *ref_counts,
                              int n_pages, int32_t *status, cudaStream_t stream) {
    if (!parents || !table_in || !lens_in || !table_out || !lens_out || !ref_counts) return GQA_ERR_NULL;
    if (!table_fits(B_in, max_pages) || !table_fits(B_out, max_pages) || n_pages <= 0 || static_cast<long long>(B_in) + B_out > (1ll << 30))
        return GQA_ERR_SHAPE;
    for (const int32_t *p : {parents, table_in, lens_in, static_cast<const int32_t *>(table_out), static_cast<const int32_t *>(lens_out),
                             static_cast<const int32_t *>(ref_counts), static_cast<const int32_t *>(status)})
        if (!aligned(p, 4)) return GQA_ERR_ALIGNMENT;
    if (overlap(table_in, 4ull * B_in * max_pages, table_out, 4ull * B_out * max_pages) || overlap(lens_in, 4ull * B_in, lens_out, 4ull * B_out))
        return GQA_ERR_OVERLAP;
    int dev = 0;
    if (device_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    return launch(pages_fork_kernel, B_out + B_in, 256, stream, parents, table_in, lens_in, B_in, table_out, lens_out, B_out,
                  max_pages, ref_counts, n_pages, status);
}

extern "C" int gqa_pages_free(const int32_t *seqs, int n, int32_t *block_table, int32_t *seq_lens, int B, int max_pages,
                              int32_t *ref_counts, int n_pages, int32_t *status, cudaStream_t stream) {
    if (!seqs || !block_table || !seq_lens || !ref_counts) return GQA_ERR_NULL;
    if (n <= 0 || !table_fits(B, max_pages) || n_pages <= 0) return GQA_ERR_SHAPE;
    for (const int32_t *p : {seqs, static_cast<const int32_t *>(block_table), static_cast<const int32_t *>(seq_lens),
                             static_cast<const int32_t *>(ref_counts), static_cast<const int32_t *>(status)})
        if (!aligned(p, 4)) return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (device_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    return launch(pages_free_kernel, n, 256, stream, seqs, block_table, seq_lens, B, max_pages, ref_counts, n_pages, status);
}

extern "C" size_t gqa_pages_workspace_size(int n_pages) {
    return n_pages > 0 ? static_cast<size_t>(n_pages) * (sizeof(PageUse) + 4) + 256 : 0;
}

extern "C" int gqa_pages_reserve(int32_t *block_table, const int32_t *seq_lens, int B, int max_pages, int page_size,
                                 int rows, int32_t *ref_counts, int n_pages, int32_t *copies, void *workspace,
                                 size_t workspace_bytes, int32_t *status, cudaStream_t stream) {
    if (!block_table || !seq_lens || !ref_counts || !copies) return GQA_ERR_NULL;
    if (!table_fits(B, max_pages) || page_size <= 0 || rows <= 0 || n_pages <= 0 ||
        static_cast<long long>(max_pages) * page_size > (1ll << 30))
        return GQA_ERR_SHAPE;
    if (!workspace || workspace_bytes < gqa_pages_workspace_size(n_pages)) return GQA_ERR_WORKSPACE;
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(ref_counts, 16) || !aligned(copies, 8) ||
        !aligned(workspace, 256) || !aligned(status, 4))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (device_sm_count(&dev) <= 0) return GQA_ERR_NO_DEVICE;
    ReserveParams p;
    p.table = block_table;
    p.lens = seq_lens;
    p.refs = ref_counts;
    p.copies = copies;
    p.status = status;
    p.use = static_cast<PageUse *>(workspace);
    p.free = reinterpret_cast<int32_t *>(p.use + n_pages);
    p.B = B;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.rows = rows;
    p.n_pages = n_pages;
    // A decoding step touches a page or two of each sequence: a thread each, all at once.  Rows
    // for a prompt touch many: a warp each.
    p.lanes = (rows - 1) / page_size + 2 <= 4 ? 1 : 32;
    return launch(pages_reserve_kernel, 1, kReserveThreads, stream, p);
}

extern "C" int gqa_pages_compact(int32_t *block_table, int B, int max_pages, int32_t *ref_counts, int n_pages,
                                 int32_t *copies, int32_t *n_live, void *workspace, size_t workspace_bytes,
                                 int32_t *status, cudaStream_t stream) {
    if (!block_table || !ref_counts || !copies || !n_live) return GQA_ERR_NULL;
    if (!table_fits(B, max_pages) || n_pages <= 0 || n_pages > (1 << 30)) return GQA_ERR_SHAPE;
    if (!workspace || workspace_bytes < gqa_pages_workspace_size(n_pages)) return GQA_ERR_WORKSPACE;
    if (!aligned(block_table, 4) || !aligned(ref_counts, 16) || !aligned(copies, 8) || !aligned(n_live, 4) ||
        !aligned(workspace, 256) || !aligned(status, 4))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    const int sms = device_sm_count(&dev);
    if (sms <= 0) return GQA_ERR_NO_DEVICE;
    CompactParams p;
    p.table = block_table;
    p.refs = ref_counts;
    p.copies = copies;
    p.n_live = n_live;
    p.status = status;
    p.rank = static_cast<int32_t *>(workspace);
    p.count = p.rank + n_pages;
    p.entries = static_cast<long long>(B) * max_pages;
    p.n_pages = n_pages;
    p.blocks = (n_pages + kCompactBlock - 1) / kCompactBlock;
    p.most = n_pages / 2 > 0 ? n_pages / 2 : 1;
    int rc = launch(compact_count_kernel, p.blocks, 1024, stream, p);
    if (rc == GQA_OK) rc = launch(compact_rank_kernel, p.blocks, 1024, stream, p);
    const long long work = p.entries > p.most ? p.entries : p.most;
    const long long grid = (work + 1023) / 1024;  // four to a thread
    if (rc == GQA_OK) rc = launch(compact_move_kernel, static_cast<int>(grid < 8 * sms ? grid : 8 * sms), 256, stream, p);
    return rc;
}

extern "C" int gqa_pages_copy(void *k_pool, void *v_pool, const int32_t *copies, int n, int page_size, int n_pages,
                              int H_kv, int d, gqa_dtype_t dtype, int32_t *status, cudaStream_t stream) {
    if (!k_pool || !v_pool || !copies) return GQA_ERR_NULL;
    if (dtype != GQA_DTYPE_F32 && dtype != GQA_DTYPE_BF16 && dtype != GQA_DTYPE_E4M3) return GQA_ERR_UNSUPPORTED_DTYPE;
    if (n <= 0 || page_size <= 0 || n_pages <= 0 || H_kv <= 0) return GQA_ERR_SHAPE;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED_DIM;
    const int elem = dtype == GQA_DTYPE_F32 ? 4 : dtype == GQA_DTYPE_BF16 ? 2 : 1;
    const long long rows = static_cast<long long>(page_size) * H_kv;  // of d elements, whole 16-byte vectors
    if (rows > (1ll << 24)) return GQA_ERR_SHAPE;
    const long long page_vecs = rows * d * elem / 16;
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(copies, 8) || !aligned(status, 4)) return GQA_ERR_ALIGNMENT;
    int dev = 0;
    const int sms = device_sm_count(&dev);
    if (sms <= 0) return GQA_ERR_NO_DEVICE;
    const long long items = 2ll * n * ((page_vecs + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs));
    const long long grid = items < 8ll * sms ? items : 8ll * sms;
    return launch(pages_copy_kernel, static_cast<int>(grid), kCopyThreads, stream, static_cast<uint4 *>(k_pool),
                  static_cast<uint4 *>(v_pool), reinterpret_cast<const int2 *>(copies), n, page_vecs, n_pages, status);
}
