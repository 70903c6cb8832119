// Block table, slots and positions of a step's new tokens, from the
// sequences' lengths: integers only, one launch.
//
// Sequence b holds len_b positions and gets n_b new ones.  Their rows follow
// sequence after sequence (row_starts, the running sum of n).  The pages it
// lacks, ceil((len + n) / page) - ceil(len / page), come off the top of the
// stack of free pages in the order of the sequences (the running sum of what
// each needs), so every row's page is known from two prefix sums:
//   page = block_table[b][j] if j is a page that b holds already,
//          free_pages[count - 1 - (pages taken before b) - (j - held)] if not.
//
// Bound by latency: a few KB in, 8 bytes out for each row.  One thread-block
// cluster does it all: every block of it computes the prefix sums for itself
// (they fit its shared memory), the barrier of the cluster stands between
// the reading of the lengths and their update in place, and rows and pages
// are then written by all its threads, each finding its sequence by bisection.
// 10 us for the 256 rows of a decode step, 16 for 131072 rows of chunks, of
// which 9 are the launch, the prefix sums and the barrier (kernel alone, cold).
// Rows past max_rows are always those of the last sequences, so one scan could
// give both sums, and a single block does without the cluster: not done.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "gda.h"
#include "gda_internal.h"

namespace cg = cooperative_groups;

namespace gda {
namespace {

constexpr int kThreads = 1024;

// Pages that n positions fill.
__device__ __forceinline__ int pages_of(int n, int page_size) { return n > 0 ? (n - 1) / page_size + 1 : 0; }

// Exclusive prefix of x over the block's threads; *total is the sum.
__device__ long long block_prefix(long long x, long long *scratch, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        long long w = scratch[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    *total = scratch[31];
    return incl - x + (warp ? scratch[warp - 1] : 0);
}

// The last index i in [0, n) with key[i] <= x (key[0] <= x, keys not falling).
__device__ __forceinline__ int last_at_most(const int *key, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (key[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) gda_block_tables_kernel(const BlockTablesArgs a) {
    __shared__ long long scratch[32];
    __shared__ int last_page;
    extern __shared__ int seq[];
    int *start = seq, *first = seq + a.B, *len = seq + 2 * a.B;    // first row, first page taken, length (-1: refused)
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
    const int t = threadIdx.x;
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
    const int each = (a.B + kThreads - 1) / kThreads;              // sequences of a thread: consecutive ones
    const int b0 = min(t * each, a.B), b1 = min(b0 + each, a.B);
    int count = *a.free_count;
    unsigned err = 0;
    if (count < 0 || count > a.free_capacity) {
        err |= GDA_DEVERR_BAD_PAGE;
        count = count < 0 ? 0 : a.free_capacity;
    }

    // lengths and additions of the thread's sequences: read once (both at the same time), kept in shared memory
    long long mine = 0, rows = 0;
    for (int b = b0; b < b1; ++b) {
        const int have = a.cache_lens[b], add = a.new_lens[b];
        len[b] = have;
        first[b] = add;
        mine += max(add, 0);
    }
    long long at = block_prefix(mine, scratch, &rows);
    mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int have = len[b], add = first[b];
        const long long n = max(add, 0);
        const bool ok = have >= 0 && add >= 0 && have + n <= cap && at + n <= a.max_rows;
        if (!ok) err |= GDA_DEVERR_BAD_LENGTH;
        start[b] = static_cast<int>(min(at, 0x7fffffffLL));
        len[b] = ok ? have : -1;
        const int need = ok ? pages_of(have + add, a.page_size) - pages_of(have, a.page_size) : 0;
        first[b] = need;
        at += n;
        mine += need;
    }
    long long wanted = 0;
    at = block_prefix(mine, scratch, &wanted);
    if (t == 0) last_page = 0;
    __syncthreads();
    int taken = 0;
    for (int b = b0; b < b1; ++b) {
        const int need = first[b];
        first[b] = static_cast<int>(min(at, 0x7fffffffLL));
        at += need;
        if (need > 0) {
            if (at > count) {
                len[b] = -1;
                err |= GDA_DEVERR_NO_PAGES;
            } else {
                taken = static_cast<int>(at);
            }
        }
    }
    if (taken > 0) atomicMax(&last_page, taken);
    cluster.sync();                                                // all blocks have read the lengths and the count
    const int pages = last_page;

    if (rank == 0) {
        for (int b = b0; b < b1; ++b) {
            a.row_starts[b] = start[b];
            a.lens_out[b] = len[b] >= 0 ? len[b] + a.new_lens[b] : a.cache_lens[b];
        }
        if (t == 0) {
            a.row_starts[a.B] = static_cast<int>(min(rows, 0x7fffffffLL));
            *a.free_out = count - pages;
        }
    }
    const int gt = rank * kThreads + t, gn = blocks * kThreads;
    // the pages that were taken
    for (int q = gt; q < pages; q += gn) {
        const int b = last_at_most(first, a.B, q);
        const int held = pages_of(len[b], a.page_size);
        const int id = a.free_pages[count - 1 - q];
        if (id < 0 || id >= a.num_pages) err |= GDA_DEVERR_BAD_PAGE;
        a.block_table[static_cast<size_t>(b) * a.max_pages + held + (q - first[b])] = id;
    }
    // the rows, four in a row to a thread: one bisection for them, a division where a sequence begins and a page looked
    // up where it changes (the integer work of a row, not its 8 bytes, is what the blocks' SMs spend their time on)
    const bool vector = ((reinterpret_cast<uintptr_t>(a.slot_map) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
    for (long long q = gt; 4 * q < a.max_rows; q += gn) {
        const int r0 = static_cast<int>(4 * q), n = min(4, a.max_rows - r0);
        int slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0};
        if (r0 < rows) {
            int b = last_at_most(start, a.B, r0);
            int have = 0, page = 0, at = 0, off = a.page_size, base = -1;   // of the row before: page, position, place in the page
            bool begin = true;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k;
                if (k >= n || r >= rows) break;
                while (b + 1 < a.B && start[b + 1] <= r) ++b, begin = true;
                if (begin) {
                    have = len[b];
                    at = have + (r - start[b]);
                    page = at / a.page_size;
                    off = at - page * a.page_size;
                } else {
                    ++at, ++off;
                    if (off == a.page_size) off = 0, ++page;
                }
                if (have < 0) {
                    begin = true;
                    continue;
                }
                if (begin || off == 0) {
                    int id;
                    if (static_cast<long long>(page) * a.page_size < have) {
                        id = a.block_table[static_cast<size_t>(b) * a.max_pages + page];
                    } else {
                        id = a.free_pages[count - 1 - (first[b] + page - pages_of(have, a.page_size))];
                    }
                    base = id >= 0 && id < a.num_pages ? id * a.page_size : -1;
                    if (base < 0) err |= GDA_DEVERR_BAD_PAGE;
                }
                begin = false;
                if (base >= 0) slot[k] = base + off, pos[k] = at;
            }
        }
        if (n == 4 && vector) {
            reinterpret_cast<int4 *>(a.slot_map)[q] = make_int4(slot[0], slot[1], slot[2], slot[3]);
            reinterpret_cast<int4 *>(a.positions)[q] = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < n) a.slot_map[r0 + k] = slot[k], a.positions[r0 + k] = pos[k];
        }
    }
    if (err) atomicOr(a.dev_err, err);
}

}  // namespace

int launch_block_tables(const BlockTablesArgs &a, cudaStream_t stream) {
    // One block for a decode step, up to eight (the portable cluster) for many rows.  us with 1 / 4 / 8 blocks: 4096 rows
    // 10.4 / 10.2 / 10.2, 8192 13.0 / 9.4 / 9.7, 16384 18.0 / 9.7 / 9.6, 131072 82 / 25.7 / 16.7; 256 rows 10.5 with any.
    const int blocks = a.max_rows <= 4 * kThreads ? 1 : (a.max_rows <= 16 * kThreads ? 4 : 8);
    const size_t smem = static_cast<size_t>(a.B) * 3 * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(gda_block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kBlockTablesMaxB * 3 * sizeof(int)));
    if (e != cudaSuccess) return record_cuda_error(e);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gda_block_tables_kernel, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? GDA_OK : record_cuda_error(e);
}

}  // namespace gda
