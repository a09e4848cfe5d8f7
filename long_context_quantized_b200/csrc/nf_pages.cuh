// nf_pages.cuh -- the pages of the segmented KV pool: reserving them for new
// tokens, releasing them behind a window or a finished sequence, forking a
// sequence, compacting the pool and copying pages (nf_kv_reserve, _release,
// _fork, _compact, _copy_blocks).
//
// State: the block table [rows][max_blocks] (entry -1: no page) and one count
// per block of the pool, refs[id] = the number of table entries that hold it,
// 0 for a free block.  Everything is decided on the device, from the lengths
// there, so that a captured decode loop turns its pages without the host.
//
// Results never depend on timing: fresh blocks are the lowest free ids, handed
// out in row order (by prefix sums in one CTA, whose work is a pass over the
// counts: 4 bytes per block), and what runs on many CTAs only adds to and
// subtracts from integer counts.
//
// The bytes are in the copies: a page of 4 kv-heads of K8/V4 is 207 KB per
// layer.  copy_pages spreads (pair, layer, 16 KB piece) units evenly over the
// grid; a thread has four 16-byte loads in flight before it stores.  Measured:
// compacting 180 pages x 16 layers (1.19 GB read and written) 207 us, 5.75 TB/s
// (0.89 of the measured copy rate); forking 32 rows with their cut pages (212 MB)
// 36 us, 5.85 TB/s.  Eight loads in flight: 202 and 37 us; default caching
// instead of streaming loads and stores: 210 and 35.  A step's reserve and
// release of 64 rows take 3 us each, chains of dependent loads of one CTA.
#pragma once

#include "nf_common.cuh"

namespace nf {

constexpr int kMaxLayers = 128;
constexpr int kPlanThreads = 1024;
constexpr int kMaxForks = 1024;     // pairs of one fork call
constexpr int kFreeList = 8192;     // fresh blocks handed out per round of reserve
constexpr int kCopyThreads = 256;
constexpr int kCopyPiece = kCopyThreads * 16 * 4;  // bytes of one copy unit

// One thread's view of a block-wide exclusive prefix sum of v over
// kPlanThreads threads; total returned to all.  warp_sum: kPlanThreads / 32 + 1
// ints of shared memory, free again on return.
__device__ __forceinline__ int block_scan(int v, int *warp_sum, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = lane < kPlanThreads / 32 ? warp_sum[lane] : 0;
    int winc = before;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, winc, d);
        if (lane >= d) winc += o;
    }
    total = __shfl_sync(0xffffffffu, winc, 31);
    const int base = __shfl_sync(0xffffffffu, winc - before, warp);
    __syncthreads();
    return base + inc - v;
}

// Four counts from refs[id0 ..], 1 where there is no block.
__device__ __forceinline__ int4 load_refs4(const int32_t *refs, int id0, int num_blocks) {
    if (id0 + 3 < num_blocks && (reinterpret_cast<uintptr_t>(refs) & 15) == 0)
        return __ldcg(reinterpret_cast<const int4 *>(refs + id0));
    int4 r;
    r.x = id0 < num_blocks ? __ldcg(refs + id0) : 1;
    r.y = id0 + 1 < num_blocks ? __ldcg(refs + id0 + 1) : 1;
    r.z = id0 + 2 < num_blocks ? __ldcg(refs + id0 + 2) : 1;
    r.w = id0 + 3 < num_blocks ? __ldcg(refs + id0 + 3) : 1;
    return r;
}

// The lowest `want` free blocks with id >= cursor into list (whole CTA);
// returns how many there were.  cursor: moved behind the last one taken.
__device__ __forceinline__ int take_free(const int32_t *refs, int num_blocks, int &cursor, int want, int *list,
                                         int *warp_sum, int *next) {
    int got = 0;
    while (got < want && cursor < num_blocks) {
        const int id0 = cursor + 4 * (int)threadIdx.x;  // cursor + 4095 stays far below 2^31: num_blocks is checked
        const int base = cursor;
        const int4 r = cursor % 4 == 0 ? load_refs4(refs, id0, num_blocks)
                                       : make_int4(id0 < num_blocks ? refs[id0] : 1, id0 + 1 < num_blocks ? refs[id0 + 1] : 1,
                                                   id0 + 2 < num_blocks ? refs[id0 + 2] : 1,
                                                   id0 + 3 < num_blocks ? refs[id0 + 3] : 1);
        const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
        int total;
        int rank = got + block_scan(f[0] + f[1] + f[2] + f[3], warp_sum, total);
        if (threadIdx.x == 0) *next = base + 4 * kPlanThreads;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (f[e]) {
                if (rank < want) list[rank] = id0 + e;
                if (rank == want - 1) *next = id0 + e + 1;
                ++rank;
            }
        __syncthreads();
        got = min(want, got + total);
        cursor = *next;
        __syncthreads();
    }
    return got;
}

// refs[id] - 1; a count that is not positive stays as it was and is reported.
__device__ __forceinline__ void release_block(int32_t *refs, int num_blocks, int id) {
    if (id < 0 || id >= num_blocks) {
        report(NF_DEVERR_BLOCK_ID);
        return;
    }
    if (atomicSub(&refs[id], 1) <= 0) {
        atomicAdd(&refs[id], 1);
        report(NF_DEVERR_REFS);
    }
}

// ---------------------------------------------------------------- reserve
struct ReserveParams {
    int32_t *refs;
    int num_blocks;
    int32_t *table;
    int rows, max_blocks;
    const int32_t *from, *to;
};

// One CTA.  A row's missing pages are counted by one warp; the rows' counts
// are summed in row order, the lowest free blocks listed, and each warp deals
// its rows' pages out of the list.
__global__ void __launch_bounds__(kPlanThreads) pages_reserve_kernel(const ReserveParams p) {
    __shared__ int warp_sum[kPlanThreads / 32 + 1], next, list[kFreeList], base_of[kPlanThreads];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int cursor = 0;
    auto range = [&](int row, int &e0, int &e1) {
        const int f = p.from[row], t = p.to[row];
        e0 = f >> 8;
        e1 = t > f ? (int)(((long long)t + kBlock - 1) >> 8) : e0;
        if (f < 0 || e1 > p.max_blocks) {
            if (t > f && lane == 0) report(NF_DEVERR_TABLE);
            if (f < 0) e1 = e0;
            e1 = min(e1, p.max_blocks);
        }
    };
    // rows of one pass: their pages, at most 2^23 a row, are counted in 32 bits
    const int pass = min(kPlanThreads, 0x7fffffff / p.max_blocks);
    for (int row0 = 0; row0 < p.rows; row0 += pass) {
        const int nrow = min(pass, p.rows - row0);
        for (int r = warp; r < nrow; r += kPlanThreads / 32) {
            int e0, e1, n = 0;
            range(row0 + r, e0, e1);
            const int32_t *t = p.table + (size_t)(row0 + r) * p.max_blocks;
            for (int e = e0; e < e1; e += 32)
                n += __popc(__ballot_sync(0xffffffffu, e + lane < e1 && t[e + lane] < 0));
            if (lane == 0) base_of[r] = n;
        }
        __syncthreads();
        int total;
        const int mine = (int)threadIdx.x < nrow ? base_of[threadIdx.x] : 0;
        const int base = block_scan(mine, warp_sum, total);
        base_of[threadIdx.x] = base;
        __syncthreads();
        for (int done = 0; done < total; done += kFreeList) {
            const int want = min(kFreeList, total - done);
            const int got = take_free(p.refs, p.num_blocks, cursor, want, list, warp_sum, &next);
            if (got < want && threadIdx.x == 0) report(NF_DEVERR_POOL);
            for (int r = warp; r < nrow; r += kPlanThreads / 32) {
                int rank = base_of[r] - done;
                const int end = (r + 1 < nrow ? base_of[r + 1] : total) - done;
                if (rank == end || end <= 0 || rank >= got) continue;
                int e0, e1;
                range(row0 + r, e0, e1);
                int32_t *t = p.table + (size_t)(row0 + r) * p.max_blocks;
                // a row whose pages spread over two rounds: those of the first
                // round are in the table by now, so its count starts where it stopped
                if (rank < 0) rank = 0;
                for (int e = e0; e < e1 && rank < got; e += 32) {
                    const unsigned need = __ballot_sync(0xffffffffu, e + lane < e1 && t[e + lane] < 0);
                    const int k = rank + __popc(need & ((1u << lane) - 1u));
                    if ((need >> lane & 1u) && k < got) {
                        const int id = list[k];
                        t[e + lane] = id;
                        p.refs[id] = 1;
                    }
                    rank += __popc(need);
                }
            }
            __syncthreads();
            if (got < want) return;
        }
    }
}

// ---------------------------------------------------------------- release
struct ReleaseParams {
    int32_t *refs;
    int num_blocks;
    int32_t *table;
    int rows, max_blocks;
    const int32_t *from, *to;
};

// One CTA per row; only whole pages inside [from, to) are touched.
__global__ void __launch_bounds__(128) pages_release_kernel(const ReleaseParams p) {
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x;
    const int f = p.from[row], t = p.to[row];
    if (f >= t) return;
    if (f < 0) {
        if (threadIdx.x == 0) report(NF_DEVERR_TABLE);
        return;
    }
    const int e0 = (int)(((long long)f + kBlock - 1) >> 8), e1 = min(t >> 8, p.max_blocks);
    int32_t *row_t = p.table + (size_t)row * p.max_blocks;
    for (int e = e0 + (int)threadIdx.x; e < e1; e += blockDim.x) {
        const int id = row_t[e];
        if (id == -1) continue;
        row_t[e] = -1;
        release_block(p.refs, p.num_blocks, id);
    }
}

// ---------------------------------------------------------------- copies
struct PoolView {
    char *plane[kMaxLayers][4];
    int plane_bytes[4];  // bytes of one block in each plane (0: no such plane)
    int n_layers, num_blocks;
};

// Units of one (pair, layer): the planes' pieces one after the other.
__device__ __forceinline__ int pieces_of(int bytes) { return (bytes + kCopyPiece - 1) / kCopyPiece; }

// Copies the pairs' blocks src[i] -> dst[i] in every layer and plane, this
// CTA's even share of the units.  check(i): whether pair i is to be copied,
// asked by all threads once for each pair of the share.
template <typename Check>
__device__ __forceinline__ void copy_pages(const PoolView &v, const int32_t *src, const int32_t *dst, int n, Check check) {
    int first[5];
    first[0] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) first[k + 1] = first[k] + pieces_of(v.plane_bytes[k]);
    const int per_layer = first[4], per_pair = per_layer * v.n_layers;
    const long long W = (long long)n * per_pair;
    const long long u1 = W * (blockIdx.x + 1) / gridDim.x;
    int pair = -1, s = 0, d = 0;
    bool good = false;
    for (long long u = W * blockIdx.x / gridDim.x; u < u1; ++u) {
        const int i = (int)(u / per_pair), rest = (int)(u % per_pair);
        if (i != pair) {
            pair = i;
            good = check(i);
            s = src[i];
            d = dst[i];
        }
        if (!good) {
            u = (long long)(i + 1) * per_pair - 1;  // the next pair
            continue;
        }
        const int layer = rest / per_layer, piece = rest % per_layer;
        const int k = piece < first[1] ? 0 : piece < first[2] ? 1 : piece < first[3] ? 2 : 3;
        const int bytes = v.plane_bytes[k];
        const int at = (piece - first[k]) * kCopyPiece;
        const char *from = v.plane[layer][k] + (size_t)s * bytes;
        char *to = v.plane[layer][k] + (size_t)d * bytes;
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int o = at + (j * kCopyThreads + (int)threadIdx.x) * 16;
            if (o < bytes) x[j] = __ldcs(reinterpret_cast<const uint4 *>(from + o));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int o = at + (j * kCopyThreads + (int)threadIdx.x) * 16;
            if (o < bytes) __stcs(reinterpret_cast<uint4 *>(to + o), x[j]);
        }
    }
}

struct CopyBlocksParams {
    PoolView v;
    const int32_t *src, *dst;
    int n;
};

// The caller's own list.  A pair whose destination is also another pair's
// destination or source is not copied (and reported): the others then read
// blocks that nothing writes, so the result does not depend on the order.
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyBlocksParams p) {
    pdl_trigger();
    pdl_wait();
    copy_pages(p.v, p.src, p.dst, p.n, [&](int i) {
        const int s = p.src[i], d = p.dst[i];
        if (s < 0 || (s == d && s < p.v.num_blocks)) return false;  // unused, or nothing to do
        if (s >= p.v.num_blocks || d < 0 || d >= p.v.num_blocks) {
            if (threadIdx.x == 0) report(NF_DEVERR_BLOCK_ID);
            return false;
        }
        int clash = 0;
        for (int j = threadIdx.x; j < p.n; j += kCopyThreads)
            clash |= j != i && p.src[j] >= 0 && (p.dst[j] == d || p.src[j] == d);
        clash = __syncthreads_or(clash);
        if (clash && threadIdx.x == 0) report(NF_DEVERR_CONFLICT);
        return clash == 0;
    });
}

// ---------------------------------------------------------------- fork
// Workspace of fork: n entries of each array.
struct ForkPlan {
    int32_t *src_row;   // -1: pair not carried out
    int32_t *dst_row;
    int32_t *full;      // pages shared
    int32_t *cut_src;   // the partly filled page (-1: none) ...
    int32_t *cut_dst;   // ... and its fresh copy
};
struct ForkParams {
    PoolView v;
    ForkPlan plan;
    int32_t *refs;
    int32_t *table;
    int rows, max_blocks;
    const int32_t *src, *dst;
    int n;
    int32_t *seqlens;
};

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const __grid_constant__ ForkParams p) {
    __shared__ int warp_sum[kPlanThreads / 32 + 1], next, list[kMaxForks], ssrc[kMaxForks], sdst[kMaxForks];
    pdl_trigger();
    pdl_wait();
    const int i = threadIdx.x;
    const bool mine = i < p.n;
    const int s = mine ? p.src[i] : -1, d = mine ? p.dst[i] : -1;
    ssrc[i] = s;
    sdst[i] = d;
    __syncthreads();
    bool ok = mine && s >= 0;
    if (ok && (s >= p.rows || d < 0 || d >= p.rows)) {
        report(NF_DEVERR_TABLE);
        ok = false;
    }
    if (ok) {
        bool clash = s == d;
        for (int j = 0; j < p.n; ++j) clash |= j != i && ssrc[j] >= 0 && (sdst[j] == d || ssrc[j] == d);
        if (clash) {
            report(NF_DEVERR_CONFLICT);
            ok = false;
        }
    }
    const int len = ok ? p.seqlens[s] : 0;
    if (ok && (len < 0 || (len + (long long)kBlock - 1) / kBlock > p.max_blocks)) {
        report(NF_DEVERR_SEQLEN);
        ok = false;
    }
    const int full = len >> 8;
    int tail = -1;
    if (ok && (len & (kBlock - 1))) {
        tail = p.table[(size_t)s * p.max_blocks + full];
        if (tail < 0 || tail >= p.v.num_blocks) {
            report(NF_DEVERR_BLOCK_ID);
            ok = false;
            tail = -1;
        }
    }
    int total, cursor = 0;
    const int rank = block_scan(tail >= 0, warp_sum, total);
    const int got = take_free(p.refs, p.v.num_blocks, cursor, total, list, warp_sum, &next);
    if (tail >= 0 && rank >= got) {
        report(NF_DEVERR_POOL);
        ok = false;
        tail = -1;
    }
    if (!mine) return;
    p.plan.src_row[i] = ok ? s : -1;
    p.plan.dst_row[i] = d;
    p.plan.full[i] = full;
    p.plan.cut_src[i] = tail;
    p.plan.cut_dst[i] = tail >= 0 ? list[rank] : -1;
    if (tail >= 0) p.refs[list[rank]] = 1;
    if (ok) p.seqlens[d] = len;
}

__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const __grid_constant__ ForkParams p) {
    pdl_trigger();
    pdl_wait();
    // the children's rows: no destination row is another pair's source, so a
    // row is read as it was
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int s = p.plan.src_row[i];
        if (s < 0) continue;
        const int full = p.plan.full[i], fresh = p.plan.cut_dst[i];
        const int32_t *from = p.table + (size_t)s * p.max_blocks;
        int32_t *to = p.table + (size_t)p.plan.dst_row[i] * p.max_blocks;
        for (int e = threadIdx.x; e < p.max_blocks; e += kCopyThreads) {
            int id = e < full ? from[e] : e == full ? fresh : -1;
            const int old = to[e];
            if (e < full && id != -1) {
                if (id < 0 || id >= p.v.num_blocks) {
                    report(NF_DEVERR_BLOCK_ID);
                    id = -1;
                } else {
                    atomicAdd(&p.refs[id], 1);
                }
            }
            if (old != -1) release_block(p.refs, p.v.num_blocks, old);
            if (old != id) to[e] = id;
        }
    }
    copy_pages(p.v, p.plan.cut_src, p.plan.cut_dst, p.n, [&](int i) { return p.plan.cut_src[i] >= 0; });
}

// ---------------------------------------------------------------- compact
struct CompactParams {
    PoolView v;
    int32_t *refs;
    int32_t *table;
    int rows, max_blocks;
    int32_t *head;  // [0] blocks in use, [1] moves
    int32_t *src, *dst;  // the moves
    int32_t *to;    // [num_blocks] new id of each block behind the first head[0]; -1: not in use
};

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int warp_sum[kPlanThreads / 32 + 1];
    pdl_trigger();
    pdl_wait();
    const int nb = p.v.num_blocks;
    constexpr int kTile = 4 * kPlanThreads;
    int used = 0;
    for (int id0 = 4 * (int)threadIdx.x; id0 < nb; id0 += kTile) {
        const int4 r = load_refs4(p.refs, id0, nb);
        used += (r.x != 0) + (id0 + 1 < nb && r.y != 0) + (id0 + 2 < nb && r.z != 0) + (id0 + 3 < nb && r.w != 0);
    }
    int live;
    block_scan(used, warp_sum, live);
    // the i-th block in use behind the first `live` ids goes to the i-th free one among them
    int ns = 0, nd = 0;
    for (int t0 = 0; t0 < nb; t0 += kTile) {
        const int id0 = t0 + 4 * (int)threadIdx.x;
        const int4 r4 = load_refs4(p.refs, id0, nb);
        const int r[4] = {r4.x, r4.y, r4.z, r4.w};
        int cs = 0, cd = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int id = id0 + e;
            cs += id < nb && id >= live && r[e] != 0;
            cd += id < live && r[e] == 0;
        }
        // both sums in one scan: a tile has at most 4096 of each
        int total;
        const int at = block_scan(cs | (cd << 16), warp_sum, total);
        int ks = ns + (at & 0xFFFF), kd = nd + (at >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int id = id0 + e;
            if (id < nb && id >= live && r[e] != 0) p.src[ks++] = id;
            if (id < live && r[e] == 0) p.dst[kd++] = id;
            if (id < nb && id >= live && r[e] == 0) p.to[id] = -1;
        }
        ns += total & 0xFFFF;
        nd += total >> 16;
    }
    __syncthreads();  // ns == nd: blocks in use behind `live` are as many as free ones before it
    for (int k = threadIdx.x; k < ns; k += kPlanThreads) {
        const int s = p.src[k], d = p.dst[k];
        p.to[s] = d;
        p.refs[d] = p.refs[s];
        p.refs[s] = 0;
    }
    if (threadIdx.x == 0) {
        p.head[0] = live;
        p.head[1] = ns;
    }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const __grid_constant__ CompactParams p) {
    pdl_trigger();
    pdl_wait();
    const int live = p.head[0], n = p.head[1];
    const long long entries = (long long)p.rows * p.max_blocks;
    for (long long e = (long long)blockIdx.x * kCopyThreads + threadIdx.x; e < entries;
         e += (long long)gridDim.x * kCopyThreads) {
        const int id = p.table[e];
        if (id < live) continue;
        if (id >= p.v.num_blocks) {
            report(NF_DEVERR_BLOCK_ID);
            continue;
        }
        const int to = p.to[id];
        if (to < 0) report(NF_DEVERR_REFS);  // an entry that no count stands for
        p.table[e] = to;
    }
    copy_pages(p.v, p.src, p.dst, n, [](int) { return true; });
}

}  // namespace nf
