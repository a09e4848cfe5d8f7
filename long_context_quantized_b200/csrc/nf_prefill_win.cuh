// nf_prefill_win.cuh -- chunked-prefill attention with a sliding window and
// sinks over the segmented K8/V4 pool (nf_prefill_attn_window), on the
// 5th-generation tensor cores.
//
// Mathematics: a query at position P sees the keys t <= P with t > P - window or
// t < n_sink; softmax in one pass over the 64-key tiles with a running max m
// per row that is only raised (and O rescaled) when a tile exceeds it by more
// than 2^8, weights 2^(x - m) in fp16, O and the row sums in fp32.
//
// Work: one CTA per 256 query rows of a kv-head (two MMA tiles a, b of 128 rows,
//   the G heads of a position side by side), which reads the sinks' key tiles
//   and those from its first row's window to its last row's position.  Only tiles
//   on an edge of the window are masked.
// Roles:
//   warps 0-15  softmax: eight warps per MMA tile, two threads per row, each with 32
//              of a key tile's 64 scores.  They stage the query rows (scaled by a
//              power of two to max |q| in [1, 2), fp16) once.  Per key tile a thread reads its scores from
//              tensor memory into registers at once and frees them for the next S;
//              the two threads of a row agree on whether its max rises (a barrier
//              with an OR over the two warps), then write their weights as the fp16
//              A operand of P . V, in tensor memory too;
//   warps 16-23 converters: two threads per key's K row (64 channels each), two per
//              V row, loaded a tile ahead in registers, dequantised to fp16 into
//              rings of four key tiles;
//   warps 24, 25 S = Q . K^T of MMA tile a, b: of key tile j + 1 as soon as the softmax
//              has read S of tile j, so that the next scores are ready when the softmax
//              of this tile ends;
//   warps 26, 27 O += P . V of MMA tile a, b once the tile's weights are written.
// Tensor memory (512 columns x 128 lanes): S of tile x at columns 64x, its P (two
// fp16 a column) at 128 + 32x, its O at 256 + 128x.
// Shared memory: Q [2 tiles][2 blocks of 64 channels][128 rows][128 B], K and V
// [4 stages][2 blocks][64 keys][128 B] each, 128-byte swizzle as in
// nf_prefill.cuh.
// What bounds it: a softmax thread's chain per 64-key tile, about 1.1 us -- the wait
// for S, its load, the pair's barrier, the exponentials (four warps share a
// sub-partition's MUFU: 1024 cycles of the 2100) and the store of P -- against
// 0.73 us of MMA work for the two tiles (8.4 MFLOP at an SM's share of the measured
// 1692 TFLOP/s), so the MMAs are not far behind the chain.  Without the
// exponentials a launch takes 0.90, without the barrier 0.92, without the
// converters 0.99 of its time.  Measured (32 / 4 heads, one B200, launches back to
// back): a chunk of 1024 queries at 180224 keys, window 4096, 82 us (0.50 of the
// 1692 TFLOP/s); a prompt of 8192 with window 2048, 309 us (0.46; a CTA's start
// and end are 15% of its 45 us).
// Choices measured on the same two cases:
//   P in tensor memory, S freed as soon as it is in registers, 16 softmax warps
//     with 32 columns each: 82 / 307 us.  8 warps with 64 columns: 96 / 384.
//     P through shared memory, S double-buffered, 8 warps (nf_prefill.cuh's
//     roles): 123 / 437.  128-key tiles with P over S: 126 / 441.
//   Waits that sleep until the phase completes: 82; in a try_wait loop 93, which
//     takes issue slots from the warps that work (issue is 64% busy).
//   Two threads per converted row: 82; one (four converter warps): 115, its K
//     conversion takes 1.5 us a tile.
//   The MMA operands in uniform registers (a whole warp runs the issue loop): 96
//     instead of 115 before the changes above.
// Every mbarrier wait is bounded; a time-out records NF_DEVERR_TIMEOUT and every
// role leaves its loop.
#pragma once

#include "nf_prefill.cuh"

namespace nf {

constexpr int kPwThreads = 896;
constexpr int kPwRows = 256;
constexpr int kPwKeys = 64;
constexpr int kPwStages = 4;
constexpr uint32_t kPwIdescQK = umma_idesc_f16(128, 64, false);
constexpr uint32_t kPwIdescPV = umma_idesc_f16(128, 128, true);

struct PrefillWinParams : PrefillParams {
    int window, n_sink;
    int out_bf16;  // out holds bf16 (o rounded once) instead of fp32
};

struct PwSmem {
    static constexpr int kQ = 0;
    static constexpr int kK = 65536;                        // [stages][16384]
    static constexpr int kV = kK + kPwStages * 16384;       // [stages][16384]
    static constexpr int kBars = kV + kPwStages * 16384;
    static constexpr int kQf = kBars + 256;    // float [256]: the rows' factors
    static constexpr int kRed = kQf + 1024;    // float [2][2 halves][256]: the halves' row maxima; their sums
    static constexpr int kLeave = kRed + 4096; // int [16]: a softmax warp's wait gave up
    static constexpr int kMisc = kLeave + 64;  // tensor memory address, abort flag
    static constexpr int kBytes = kMisc + 16;
    static_assert(kBytes <= 232448, "shared memory per CTA");
};
enum { kPwQ = 0, kPwKFull = 1, kPwKFree = 5, kPwVFull = 9, kPwVFree = 13, kPwS = 17, kPwSFree = 19, kPwP = 21, kPwPv = 23,
       kPwO = 25, kPwDrain = 26, kPwNumBars = 27 };
static_assert(kPwNumBars * 8 <= 256 && kPwStages == 4, "mbarrier slots");

// The keys [0, n_sink) and [lo, end) a CTA's rows see between them.  Tile j of
// the CTA's list holds the 64 keys of key tile j + (j >= sinks ? skip : 0).
struct PwKeys {
    int n_sink, lo, end, sinks, skip;
    __device__ __forceinline__ bool seen(int pos) const { return pos < end && (pos >= lo || pos < n_sink); }
    __device__ __forceinline__ int first(int j) const { return (j + (j >= sinks ? skip : 0)) * kPwKeys; }
};

// Half a key's K row: 64 channels' codes and the key's scale, all 0 for a key
// that no row sees.
struct PwHalfK {
    uint4 k[4];
    uint32_t ks;  // fp16 bits
    // dequantised to fp16 (code x scale) into block `part` of a [2][64 keys][128 B] tile
    __device__ __forceinline__ void store(int key, int part, unsigned char *tile) const {
        if ((ks & 0x7FFFu) > kTcMaxKScaleBits) report(NF_DEVERR_RANGE);
        const __half2 sk = u32_h2(ks * 0x10001u);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t w[4] = {k[u].x, k[u].y, k[u].z, k[u].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                i8x4_to_f16(w[e], o[2 * e], o[2 * e + 1]);
                o[2 * e] = h2_u32(__hmul2(u32_h2(o[2 * e]), sk));
                o[2 * e + 1] = h2_u32(__hmul2(u32_h2(o[2 * e + 1]), sk));
            }
            *reinterpret_cast<uint4 *>(tile + tc_swz(key, 8 * part + 2 * u, 8192u)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(tile + tc_swz(key, 8 * part + 2 * u + 1, 8192u)) =
                make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
};
// Half a key's V row: 64 channels' nibbles and their two scales.
struct PwHalfV {
    uint4 v[2];
    uint32_t vs;
    __device__ __forceinline__ void store(int key, int part, unsigned char *tile) const {
        if (max(vs & 0x7FFFu, (vs >> 16) & 0x7FFFu) > kTcMaxVScaleBits) report(NF_DEVERR_RANGE);
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // 32 channels
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            const __half2 sv = u32_h2(prmt(vs, 0, u == 0 ? 0x1010 : 0x3232));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint4 o;
                o.x = h2_u32(__hmul2(nib_even(w[e]), sv));
                o.y = h2_u32(__hmul2(nib_odd(w[e]), sv));
                o.z = h2_u32(__hmul2(nib_even(w[e] >> 8), sv));
                o.w = h2_u32(__hmul2(nib_odd(w[e] >> 8), sv));
                *reinterpret_cast<uint4 *>(tile + tc_swz(key, 8 * part + 4 * u + e, 8192u)) = o;
            }
        }
    }
};

// (x0, x1) = (s0, s1) * (f, f) + (c, c)
__device__ __forceinline__ void fma_pair(uint32_t s0, uint32_t s1, uint64_t ff, uint64_t cc, float &x0, float &x1) {
    uint64_t s, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(s) : "r"(s0), "r"(s1));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(s), "l"(ff), "l"(cc));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(d));
}
// (a0, a1) += (x0, x1)
__device__ __forceinline__ void add_pair(uint64_t &a, float x0, float x1) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(x));
}
__device__ __forceinline__ float pair_sum(uint64_t a) {
    float x0, x1;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(a));
    return x0 + x1;
}
__device__ __forceinline__ uint64_t pair_of(float x) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(x));
    return d;
}

__global__ void __launch_bounds__(kPwThreads, 1) prefill_win_kernel(const __grid_constant__ PrefillWinParams p) {
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + PwSmem::kBars);
    uint64_t *q_full = bars + kPwQ, *k_full = bars + kPwKFull, *k_free = bars + kPwKFree, *v_full = bars + kPwVFull,
             *v_free = bars + kPwVFree, *s_full = bars + kPwS, *s_free = bars + kPwSFree, *p_full = bars + kPwP,
             *pv_done = bars + kPwPv, *o_full = bars + kPwO, *drain = bars + kPwDrain;
    float *qfs = reinterpret_cast<float *>(smem + PwSmem::kQf), *red = reinterpret_cast<float *>(smem + PwSmem::kRed);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + PwSmem::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + PwSmem::kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, h = blockIdx.y;
    const int rt = p.row_tiles - 1 - (int)blockIdx.x;  // late positions first
    const int r0 = rt * kPwRows;
    const int G = p.group;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 512);
        for (int i = 0; i < kPwStages; ++i) {
            mbar_init(&k_full[i], 128);
            mbar_init(&k_free[i], 2);  // the two tiles' S
            mbar_init(&v_full[i], 128);
            mbar_init(&v_free[i], 2);  // the two tiles' P . V
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 256);
            mbar_init(&p_full[i], 8);  // the tile's warps
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(o_full, 2);
        mbar_init(drain, 4);
        *abort_flag = 0;
        for (int i = 0; i < 16; ++i) reinterpret_cast<volatile int *>(smem + PwSmem::kLeave)[i] = 0;
        // the swizzled operands need 1024-byte alignment of the window
        if (smem_addr(smem) & 1023u) {
            if (blockIdx.x == 0 && h == 0 && b == 0) report(NF_DEVERR_INTERNAL);
            *abort_flag = 1;
        }
        fence_mbar_init();
    }
    if (warp == 24) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    pdl_wait();
    pdl_trigger();
    const int L = p.seqlens[b];
    // row r0 + i (i < 256): position pos0 + d, head g of the group, with d = (g0 + i) / G
    // worked out in fp32 (exact: g0 + i < 2^20)
    const int pos0 = r0 / G, g0 = r0 - pos0 * G;
    const float inv_g = 1.0f / (float)G;
    auto row_pos = [&](int i) { return pos0 + (int)(((float)(g0 + i) + 0.5f) * inv_g); };
    auto out_row = [&](int i) {
        const int j = row_pos(i), gq = r0 + i - j * G;
        return ((size_t)b * p.n_q + j) * p.num_q_heads + (size_t)h * G + gq;
    };
    uint4 qw[8];
    if (warp < 16) {
        // the query rows this warp stages, on their way before the length is known
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = 16 * warp + 2 * u + (lane >> 4);
            qw[u] = r0 + i < p.rows ? __ldg(reinterpret_cast<const uint4 *>(p.q + out_row(i) * kHeadDim) + (lane & 15))
                                    : make_uint4(0, 0, 0, 0);
        }
    }
    const bool bad_len = L < p.n_q || L > p.max_seqlen;
    const int last_row = min(r0 + kPwRows, p.rows) - 1;
    const int32_t *bt = p.block_table + (size_t)b * p.max_blocks;
    PwKeys keys{p.n_sink, 0, 0, 0, 0};
    if (!bad_len) {
        keys.end = L - p.n_q + row_pos(last_row - r0) + 1;
        keys.lo = max(0, L - p.n_q + pos0 - p.window + 1);
        const int first = keys.lo / kPwKeys, s = (p.n_sink + kPwKeys - 1) / kPwKeys;
        if (p.n_sink < keys.lo && s < first) {
            keys.sinks = s;
            keys.skip = first - s;
        }
    }
    const int T = (keys.end + kPwKeys - 1) / kPwKeys - keys.skip;

    if (bad_len) {
        if (threadIdx.x == 0 && rt == p.row_tiles - 1 && h == 0 && L != 0) report(NF_DEVERR_SEQLEN);
        for (int idx = threadIdx.x; idx < kPwRows * kHeadDim; idx += kPwThreads) {
            const int i = idx / kHeadDim, ch = idx % kHeadDim;
            if (r0 + i >= p.rows) continue;
            store_out1<true>(p.out, p.out_bf16, out_row(i) * kHeadDim + ch, 0.f);
            if (ch == 0 && p.out_lse) p.out_lse[out_row(i)] = -INFINITY;
        }
    } else if (warp < 16 && !*abort_flag) {
        // ================================================== softmax of tile x, row r, half hf of the keys
        const int x = warp >> 3, hf = (warp >> 2) & 1, r = threadIdx.x & 127;
        const uint32_t pair_bar = 1 + 4 * x + (warp & 3);  // the two warps of these rows
        float *red_row = red + 128 * x + r;                // + 256: the other half's
        volatile int *leave = reinterpret_cast<volatile int *>(smem + PwSmem::kLeave);
        const int row = r0 + 128 * x + r;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        // this half's scores and weights, and its half of O's columns
        const uint32_t t_s = t_lane + 64u * x + 32u * hf, t_p = t_lane + 128u + 32u * x + 16u * hf;
        const uint32_t t_o = t_lane + 256u + 128u * x + 64u * hf;
        {
            // 16 of the tile's query rows, two at a time: half a warp per row, lane m
            // channels 8m .. 8m + 7.  A row is scaled by a power of two to max |q| in [1, 2)
            // (its bf16 values are then fp16 values, exact down to 2^-17)
            const int m = lane & 15, w0 = 16 * (warp & 7) + (lane >> 4);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int tr = w0 + 2 * u;  // row of the tile
                const uint32_t ww[4] = {qw[u].x, qw[u].y, qw[u].z, qw[u].w};
                // max |q| straight from the bf16 bits (sign cleared)
                uint32_t am = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) am = max(am, max((ww[e] << 16) & 0x7FFFFFFFu, ww[e] & 0x7FFF0000u));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
                const uint32_t ex = min(max(am >> 23, 1u), 253u);
                const float up = __uint_as_float((254u - ex) << 23);  // 2^-(ex - 127)
                uint32_t o4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o4[e] = pack_f16(__uint_as_float(ww[e] << 16) * up, __uint_as_float(ww[e] & 0xFFFF0000u) * up);
                *reinterpret_cast<uint4 *>(smem + PwSmem::kQ + x * 32768 + tc_swz(tr, m, 16384u)) =
                    make_uint4(o4[0], o4[1], o4[2], o4[3]);
                // the row's factor stays positive, so that a hidden key's -inf times it is -inf
                if (m == 0) qfs[128 * x + tr] = fmaxf(__uint_as_float(ex << 23) * p.scale_log2, FLT_MIN);
            }
            fence_async_smem();
            mbar_arrive(q_full);
        }
        bool ok = __all_sync(0xffffffffu, tc_wait(q_full, 0, abort_flag));
        const float qf = ok ? qfs[128 * x + r] : 1.f;
        const int lim = row < p.rows ? L - p.n_q + row_pos(row - r0) : -1;
        // positions of the tile's first and last row: a key tile between the last
        // row's window and the first row's position, or inside the sinks, is not masked
        const int pos_lo = L - p.n_q + row_pos(128 * x);
        const int pos_hi = L - p.n_q + row_pos(min(128 * x + 127, p.rows - 1 - r0));
        const uint64_t ff = pair_of(qf);
        float m_run = -INFINITY, l_run = 0.f;
        // Every wait's outcome is made warp-uniform: the tensor-memory loads and stores
        // below are warp-collective.  A warp whose wait gave up still comes to the next
        // barriers of its pair and says so there, and the two leave together: neither is
        // left waiting at one.
        bool left = false, leaves = !ok;
        for (int j = 0; ok && j < T; ++j) {
            if (!__all_sync(0xffffffffu, tc_wait(&s_full[x], j & 1, abort_flag))) { ok = false; leaves = true; break; }
            tc_fence_after();
            uint32_t s[32];
            tmem_ld32(t_s, s);
            const int k0 = keys.first(j), key0 = k0 + 32 * hf;
            tmem_wait_ld_tied<32>(s);
            tc_fence_before();
            mbar_arrive(&s_free[x]);
            if (k0 + kPwKeys - 1 > pos_lo || (k0 <= pos_hi - p.window && k0 + kPwKeys > p.n_sink)) {
                // hidden: keys behind the row, and those before its window that are no sinks
                const int nvis = lim - key0 + 1, first = lim - p.window + 1 - key0, sink = max(0, p.n_sink - key0);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i >= nvis || (i >= sink && i < first)) s[i] = 0xFF800000u;
            }
            float m4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 4]));
#pragma unroll
            for (int i = 8; i < 32; i += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m4[e] = fmaxf(fmaxf(m4[e], __uint_as_float(s[i + e])), __uint_as_float(s[i + e + 4]));
            float tmax = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * qf;
            const bool rise = bar_red_or(pair_bar, 64, tmax > m_run + kTcLazy);
            float alpha = 1.f;
            if (rise) {
                // some row's max rises, in one of the halves, or one of the warps leaves
                red_row[256 * hf] = tmax;
                named_sync(pair_bar, 64);
                if (leave[warp ^ 4]) { ok = false; left = true; break; }
                tmax = fmaxf(tmax, red_row[256 * (hf ^ 1)]);
                if (tmax > m_run + kTcLazy) {
                    alpha = ex2(m_run - tmax);  // 0 when m_run was -inf
                    l_run *= alpha;
                    m_run = tmax;
                }
            }
            // weights 2^(s qf - m) and their sum in fp32; rounded to fp16 for P . V
            const uint64_t cc = pair_of(m_run == -INFINITY ? 0.f : -m_run);
            uint32_t w[16];
            uint64_t sum2 = 0ull, sum3 = 0ull;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x0, x1;
                fma_pair(s[2 * i], s[2 * i + 1], ff, cc, x0, x1);
                x0 = ex2(x0);
                x1 = ex2(x1);
                w[i] = pack_f16(x0, x1);
                if (i & 1)
                    add_pair(sum3, x0, x1);
                else
                    add_pair(sum2, x0, x1);
            }
            l_run += pair_sum(sum2) + pair_sum(sum3);
            // P's columns and O are free once P . V of the last tile is done
            if (j > 0) {
                // (after the last tile the pair meets at the barrier below)
                if (!__all_sync(0xffffffffu, tc_wait(&pv_done[x], (j - 1) & 1, abort_flag))) {
                    ok = false;
                    leaves = j + 1 < T;
                    break;
                }
                tc_fence_after();  // the stores below come after the MMA's reads of P and O
                if (rise) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[16];
                        tmem_ld16(t_o + 16u * c, o);
                        tmem_wait_ld_tied<16>(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st16(t_o + 16u * c, o);
                    }
                }
            }
            tmem_st16(t_p, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();  // every lane has stored and fenced its weights
            if (lane == 0) mbar_arrive(&p_full[x]);
        }
        if (leaves) {
            (void)bar_red_or(pair_bar, 64, true);
            if (lane == 0) leave[warp] = 1;
            named_sync(pair_bar, 64);
            left = true;
        }
        if (!left) {
            red_row[512 + 256 * hf] = l_run;
            named_sync(pair_bar, 64);
            l_run = red_row[512] + red_row[512 + 256];
        }
        if (ok && !left && __all_sync(0xffffffffu, tc_wait(o_full, 0, abort_flag))) {
            tc_fence_after();
            const float inv = l_run > 0.f ? 1.0f / l_run : 0.f;
            const size_t at = row < p.rows ? out_row(row - r0) * kHeadDim : 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 16 of this half's 64 channels
                uint32_t o[16];
                __syncwarp();
                tmem_ld16(t_o + 16u * c, o);
                tmem_wait_ld_tied<16>(o);
                // column 8g + e holds channel 8g + (0, 4, 1, 5, 2, 6, 3, 7)[e]
#pragma unroll
                for (int g = 0; g < 2 && row < p.rows; ++g) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[(e >> 1) + 4 * (e & 1)] = __uint_as_float(o[8 * g + e]) * inv;
                    const size_t to = at + 64 * hf + 16 * c + 8 * g;
                    if (p.out_bf16) {
                        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + to) =
                            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                       pack_bf16(v[6], v[7]));
                    } else {
                        float4 *d = reinterpret_cast<float4 *>(p.out + to);
                        d[0] = make_float4(v[0], v[1], v[2], v[3]);
                        d[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
            if (m_run != -INFINITY && fabsf(m_run) > kTcMaxScore) report(NF_DEVERR_RANGE);
            if (row < p.rows && p.out_lse && hf == 0)
                p.out_lse[out_row(row - r0)] = l_run > 0.f ? (m_run + log2f(l_run)) * 0.69314718055994531f : -INFINITY;
        }
    } else if (warp < 24 && !*abort_flag) {
        // ================================================== converters: key t of each tile
        // (thread 2t or 2t + 1 of its row kind: the key's first or second 64 channels)
        const int t = (threadIdx.x & 127) >> 1, part = threadIdx.x & 1;
        const bool is_k = threadIdx.x < 512 + 128;
        // A key tile lies in one 256-key block and holds a key < L.  The table entry
        // is read a tile before the rows.
        auto entry = [&](int j) { return j < T ? __ldg(bt + (keys.first(j) >> 8)) : 0; };
        auto slot = [&](int j, int blk, bool &ok) -> size_t {
            const int pos = keys.first(j) + t;
            ok = blk >= 0 && blk < p.num_blocks;
            if (!ok) {
                if (t == 0 && part == 0) report(NF_DEVERR_BLOCK_ID);
                return 0;
            }
            ok = keys.seen(pos);
            return ((size_t)blk * p.num_kv_heads + h) * kBlock + (pos & (kBlock - 1));
        };
        auto ring = [&](auto &cur, auto &nxt, auto load, auto convert, int region, uint64_t *full, uint64_t *free_) {
            int blk = entry(1);
            load(0, entry(0), cur);
            auto stage_tile = [&](int j, auto &c, auto &n) -> bool {
                const int st = j % kPwStages;
                if (j + 1 < T) load(j + 1, blk, n);
                blk = entry(j + 2);
                if (j >= kPwStages && !tc_wait(&free_[st], (j / kPwStages - 1) & 1, abort_flag)) return false;
                convert(c, smem + region + st * 16384);
                fence_async_smem();
                mbar_arrive(&full[st]);
                return true;
            };
            for (int j = 0; j < T; j += 2) {
                if (!stage_tile(j, cur, nxt)) break;
                if (j + 1 < T && !stage_tile(j + 1, nxt, cur)) break;
            }
        };
        if (is_k) {
            PwHalfK ra, rb;
            ring(ra, rb,
                 [&](int j, int blk, PwHalfK &r) {
                     bool ok;
                     const size_t si = slot(j, blk, ok);
                     const uint4 *kp = reinterpret_cast<const uint4 *>(p.k_codes + si * kHeadDim) + 4 * part;
#pragma unroll
                     for (int u = 0; u < 4; ++u) r.k[u] = ok ? __ldg(kp + u) : make_uint4(0, 0, 0, 0);
                     r.ks = ok ? __ldg(reinterpret_cast<const unsigned short *>(p.k_scales + si)) : 0u;
                 },
                 [&](const PwHalfK &r, unsigned char *dst) { r.store(t, part, dst); }, PwSmem::kK, k_full, k_free);
        } else {
            PwHalfV ra, rb;
            ring(ra, rb,
                 [&](int j, int blk, PwHalfV &r) {
                     bool ok;
                     const size_t si = slot(j, blk, ok);
                     const uint4 *vp = reinterpret_cast<const uint4 *>(p.v_codes + si * (kHeadDim / 2)) + 2 * part;
#pragma unroll
                     for (int u = 0; u < 2; ++u) r.v[u] = ok ? __ldg(vp + u) : make_uint4(0, 0, 0, 0);
                     r.vs = ok ? __ldg(reinterpret_cast<const uint32_t *>(p.v_scales + si * (kHeadDim / kVGroup)) + part) : 0u;
                 },
                 [&](const PwHalfV &r, unsigned char *dst) { r.store(t, part, dst); }, PwSmem::kV, v_full, v_free);
        }
    } else if (warp >= 24 && !*abort_flag) {
        // ================================================== the MMAs of tile x
        // The whole warp runs this loop, one lane issues; the broadcasts tell the
        // compiler that the operands are the same in every lane, so that they stay in
        // uniform registers (moving them there for each MMA costs more than the MMA).
        const int role = __shfl_sync(0xffffffffu, warp - 24, 0), x = role & 1;
        const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t mine = lane == 0;
        const uint32_t sQ = smem_addr(smem + PwSmem::kQ) + x * 32768, sK = smem_addr(smem + PwSmem::kK);
        const uint32_t sV = smem_addr(smem + PwSmem::kV);
        const uint32_t t_s = tmem_u + 64u * x, t_p = tmem_u + 128u + 32u * x, t_o = tmem_u + 256u + 128u * x;
        // descriptors of the first k-step, stage 0; the address field counts 16 bytes
        const uint64_t dq = umma_desc_sw128(sQ, 16, 1024), dk = umma_desc_sw128(sK, 16, 1024);
        const uint64_t dv = umma_desc_sw128(sV, 8192, 1024);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag)) != 0;
        };
        bool ok = true;
        if (role < 2) {
            // S of key tile j, once its K is staged and the softmax has read S of tile j - 1
            ok = wait(q_full, 0);
            for (int j = 0; ok && j < T; ++j) {
                const int st = j % kPwStages;
                ok = wait(&k_full[st], (j / kPwStages) & 1) && (j == 0 || wait(&s_free[x], (j - 1) & 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_f16_if(mine, t_s, dq + (ks >> 2) * 1024u + (ks & 3) * 2u,
                                dk + st * 1024u + (ks >> 2) * 512u + (ks & 3) * 2u, kPwIdescQK, ks > 0 ? 1u : 0u);
                umma_commit_if(mine, &s_full[x]);
                umma_commit_if(mine, &k_free[st]);
            }
        } else {
            // O += P . V of key tile j, once its V is staged and its weights are written
            for (int j = 0; ok && j < T; ++j) {
                const int st = j % kPwStages;
                ok = wait(&v_full[st], (j / kPwStages) & 1) && wait(&p_full[x], j & 1);
                if (!ok) break;
                tc_fence_after();
                // P of keys 16 kk ..: two fp16 a column
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_f16_ta_if(mine, t_o, t_p + 8u * kk, dv + st * 1024u + kk * 128u, kPwIdescPV,
                                   (j > 0 || kk > 0) ? 1u : 0u);
                umma_commit_if(mine, &pv_done[x]);
                umma_commit_if(mine, &v_free[st]);
            }
            if (ok) umma_commit_if(mine, o_full);
        }
        umma_commit_if(mine, drain);  // arrives once every MMA this thread issued has completed
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 24) {
        // every MMA has completed before tensor memory is freed (a sequence without
        // valid keys, or a launch that gave up at once, issued none)
        if (lane == 0 && !bad_len) {
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait_sleep(drain, 0, 20000u))
                if (global_ns() - t0 > kWaitLimitNs) {
                    report(NF_DEVERR_TIMEOUT);
                    break;
                }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace nf
