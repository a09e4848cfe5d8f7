// nf_rope.cuh -- rotary positions with several axes on a step's queries and
// keys, fused with the quantised append (nf_rope_append_quant).
//
// Mathematics: frequency i of rot / 2 turns one pair of channels by the angle
//   a_i = position[axis(i)] * inv_freq[i]:  (x, y) -> (x cos - y sin, y cos + x sin).
// Positions of a long context put a_i at 10^5 radians and more, where an fp32
// product is off by hundredths of a radian.  So the angle is taken in turns in
// fp64: position * inv_freq as an exact sum of two doubles (a product and, by an
// FMA, what its rounding left), and its turns, a / 2 pi, as a sum of two doubles
// again (the product with the leading double of 1 / 2 pi split by an FMA, plus
// the products with the trailing one); the whole turns are dropped exactly and
// what is left, at most half a turn, goes to sincospi.  cos and sin are then good to
// a few units of 2^-53 whatever the position.
//   Queries are turned in fp32 (cos and sin rounded to fp32 once) and rounded
// once to their type.  Keys are turned in fp64 and rounded to fp32 once before
// they are quantised: a code is a rounding of x / scale, so a key value that is
// off by an fp32 step now and then lands on another code, and the codes would
// depend on the order of the kernel's operations.  In fp64 that has a chance of
// about 2^-40 per value, so the pool's bytes are those of the definition.  The
// fp64 work is 4 products and sums per key channel pair and one sincospi per
// frequency and CTA, small beside the bytes moved.
//
// Work: one CTA of four warps per token (per slice of a token's rows when there
// are few tokens).  Every warp first issues the loads of its first query rows
// and of its first key or value row; meanwhile 64 threads work out the token's
// cos and sin into shared memory.
//   Queries: half a warp per row, lane m of 16 holding two pieces of 4 channels
// that turn with each other -- 4m.. and rot / 2 + 4m.. (halves) or 8m.. and 8m
// + 4.. (pairs) -- so a turn needs no exchange between lanes, and in both
// layouts the lane's frequencies are 4m .. 4m + 3, kept in registers for all its
// rows.  Lanes from rot / 8 on hold the channels that are not turned.
//   Keys: the same half-warp layout, two heads per warp, each quantised within its
// 16 lanes (RK4V4-E8 keys, whose scale groups of 32 channels cut across the
// pieces, take a warp per row, lane l channels 4l .. 4l + 3, the partner channels
// coming from the lane rot / 8 away).  Values: half a warp per row, lane m
// channels 8m .. 8m + 7.
//
// What bounds it: many tokens, the bytes and the instructions about equally
// (16384 tokens, 40 + 2 x 8 heads, int8 cache: 84 us, 437 MB, 0.80 of the measured
// copy rate; issue 76% busy); a chunk of 1024 tokens (32 + 2 x 4 heads) 6.2 us,
// half of it the latency of one CTA; a step's tokens 2.8 us, a launch.  With one
// lane per 4 channels and shuffled partners for every row, and IEEE quotients,
// the 16384 tokens took 207 us.
#pragma once

#include "nf_append.cuh"
#include "nf_common.cuh"

namespace nf {

constexpr int kRopeWarps = 4;

struct RopeParams {
    AppendParams a;  // pool, table, lengths; k_new / v_new with the strides below
    const void *q;
    void *q_out;     // [batch][n_new][H_q][128]
    long long q_bs, q_ts, k_bs, k_ts, v_bs, v_ts;  // batch and token strides, elements
    int num_q_heads;
    const int32_t *positions;  // [batch][n_new][n_axes]
    int n_axes;
    const int32_t *n_valid;    // [batch] or null
    const float *inv_freq;     // [rot / 2]
    int rot, pairs;
    int slices;                // CTAs per token
    uint32_t axis[4];          // axis of frequency f: bits 2 (f % 16) of word f / 16
};

// cos and sin of position * f, see above.
__device__ __forceinline__ void rope_angle(int position, float f, double &c, double &s) {
    constexpr double kInv2PiHi = 0x1.45f306dc9c883p-3, kInv2PiLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi) as hi + lo
    const double a = (double)position * (double)f, a_lo = fma((double)position, (double)f, -a);
    const double hi = a * kInv2PiHi;
    const double lo = fma(a, kInv2PiHi, -hi) + fma(a, kInv2PiLo, a_lo * kInv2PiHi);
    const double turn = (hi - rint(hi)) + lo;
    sincospi(2.0 * turn, &s, &c);
}

// Four consecutive channels as they lie in memory.
template <bool F32>
struct Quad {
    float4 v;
    __device__ __forceinline__ void load(const void *base, long long elem) {
        // (an ordinary load: q_out may be q's memory, which this launch then writes)
        v = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + elem);
    }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
    static __device__ __forceinline__ void put(void *base, long long elem, const float (&x)[4]) {
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + elem) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <>
struct Quad<false> {
    uint2 v;
    __device__ __forceinline__ void load(const void *base, long long elem) {
        v = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(base) + elem);
    }
    __device__ __forceinline__ void get(float (&x)[4]) const {
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    static __device__ __forceinline__ void put(void *base, long long elem, const float (&x)[4]) {
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(base) + elem) =
            make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    }
};

// Largest magnitude over the lane's channels and over lanes m ^ (w - 1) .. of its
// group of w lanes.
template <int W>
__device__ __forceinline__ float group_absmax(const float (&x)[4], const float (&y)[4]) {
    float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    a = fmaxf(a, fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3]))));
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// One row held by half a warp as two pieces of 4 channels at c0 and c1, into the
// row's place of a plane with one scale per row (int8, e4m3) or of a bf16
// plane.  All lanes take part; only those with `store` write.
template <int FMT>
__device__ __forceinline__ void store_row16(const float (&x)[4], const float (&y)[4], int m, int c0, int c1, bool store,
                                            void *codes, __half *scales, size_t si) {
    if (FMT == NF_KV_BF16) {
        if (store) {
            Quad<false>::put(codes, (long long)si * kHeadDim + c0, x);
            Quad<false>::put(codes, (long long)si * kHeadDim + c1, y);
        }
        return;
    }
    float sigma;
    const __half h = make_scale(group_absmax<16>(x, y), FMT == NF_KV_F8 ? 448.0f : 127.0f, sigma);
    const uint32_t w0 = FMT == NF_KV_F8 ? pack_codes_f8<true>(x, sigma) : pack_codes8<true>(x, sigma);
    const uint32_t w1 = FMT == NF_KV_F8 ? pack_codes_f8<true>(y, sigma) : pack_codes8<true>(y, sigma);
    if (store) {
        uint8_t *row = static_cast<uint8_t *>(codes) + si * kHeadDim;
        *reinterpret_cast<uint32_t *>(row + c0) = w0;
        *reinterpret_cast<uint32_t *>(row + c1) = w1;
        if (m == 0) scales[si] = h;
    }
}

// One value row, lane m holding channels 8m .. 8m + 7.
template <int FMT>
__device__ __forceinline__ void store_v16(const AppendParams &a, const float (&x)[4], const float (&y)[4], int m, bool store,
                                          size_t si) {
    if (FMT == NF_KV_K8V4) {  // a scale per 32 channels = 4 lanes
        float sigma;
        const __half h = make_scale(group_absmax<4>(x, y), 7.0f, sigma);
        int lo[4], hi[4];
        make_codes<true>(x, sigma, 7, lo);
        make_codes<true>(y, sigma, 7, hi);
        if (store) {
            reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.v_codes) + si * (kHeadDim / 2))[m] =
                pack_codes4(lo) | (pack_codes4(hi) << 16);
            if ((m & 3) == 0) a.v_scales[si * (kHeadDim / kVGroup) + (m >> 2)] = h;
        }
    } else if (FMT == NF_KV_K4V4) {
        float inv;
        const int e = e8_exponent(group_absmax<4>(x, y), inv);
        const uint32_t w = pack_codes_e8(x, inv) | (pack_codes_e8(y, inv) << 16);
        if (store) {
            reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.v_codes) + si * (kHeadDim / 2))[m] = w;
            if ((m & 3) == 0) reinterpret_cast<uint8_t *>(a.v_scales)[si * 4 + (m >> 2)] = (uint8_t)(e + 127);
        }
    } else {
        store_row16<FMT>(x, y, m, 8 * m, 8 * m + 4, store, a.v_codes, a.v_scales, si);
    }
}

template <bool F32, bool PAIRS, int FMT>
__global__ void __launch_bounds__(kRopeWarps * 32, F32 ? 6 : 8) rope_append_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kAhead = F32 ? 2 : 4;  // query rows a half-warp has in flight (64 bytes a lane)
    constexpr int kHalfWarps = 2 * kRopeWarps;
    __shared__ double c64[kHeadDim / 2], s64[kHeadDim / 2];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const AppendParams &a = p.a;
    const int i = blockIdx.x, b = blockIdx.z;  // token i of sequence b
    const long long token = (long long)b * a.n_new + i;
    if (p.n_valid && i >= p.n_valid[b]) return;  // the whole CTA: padding token
    const int half = p.rot >> 1, H = a.num_kv_heads, n_q = p.num_q_heads;

    // this CTA's query rows [q0, q1) and pairs of key or value rows [k0, k1):
    // pair t < T is the keys of heads 2t and 2t + 1, pair T + t their values
    const int T = (H + 1) >> 1;
    int q0 = 0, q1 = n_q, k0 = 0, k1 = 2 * T;
    if (p.slices > 1) {
        const int s = blockIdx.y;
        q0 = n_q * s / p.slices;
        q1 = n_q * (s + 1) / p.slices;
        k0 = 2 * T * s / p.slices;
        k1 = 2 * T * (s + 1) / p.slices;
    }

    // ---- loads in flight while the angles are worked out
    const int m = lane & 15, hw = 2 * warp + (lane >> 4);
    const bool lane_turns = 8 * m < p.rot;
    int c0, c1;  // first channels of the lane's two pieces
    if (PAIRS) {
        c0 = 8 * m;
        c1 = c0 + 4;
    } else if (lane_turns) {
        c0 = 4 * m;
        c1 = half + c0;
    } else {  // the channels behind rot, split the same way
        c0 = p.rot + 4 * (m - (p.rot >> 3));
        c1 = c0 + ((kHeadDim - p.rot) >> 1);
    }
    const long long q_at = b * p.q_bs + i * p.q_ts;
    Quad<F32> x0[kAhead], x1[kAhead];
    auto load_q = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + kHalfWarps * u;
            if (r < q1) {
                x0[u].load(p.q, q_at + r * kHeadDim + c0);
                x1[u].load(p.q, q_at + r * kHeadDim + c1);
            }
        }
    };
    Quad<F32> kv0, kv1;
    auto load_kv = [&](int t) {
        const bool is_k = t < T;
        const int h = 2 * (is_k ? t : t - T) + (lane >> 4);
        if (h >= H || (FMT == NF_KV_K4V4 && is_k)) return;
        if (is_k) {
            const long long at = b * p.k_bs + i * p.k_ts + h * kHeadDim;
            kv0.load(a.k_new, at + c0);
            kv1.load(a.k_new, at + c1);
        } else {
            const long long at = b * p.v_bs + i * p.v_ts + h * kHeadDim + 8 * m;
            kv0.load(a.v_new, at);
            kv1.load(a.v_new, at + 4);
        }
    };
    int qr = q0 + hw, t = k0 + warp;
    load_q(qr);
    if (t < k1) load_kv(t);

    if (threadIdx.x < half) {
        const int f = threadIdx.x;
        const uint32_t w = f < 16 ? p.axis[0] : f < 32 ? p.axis[1] : f < 48 ? p.axis[2] : p.axis[3];
        const int axis = (int)(w >> (2 * (f & 15))) & 3;
        double c, s;
        rope_angle(p.positions[token * p.n_axes + axis],
                   __ldg(p.inv_freq + threadIdx.x), c, s);
        c64[threadIdx.x] = c;
        s64[threadIdx.x] = s;
    }
    // where the new token's K and V go
    const int pos = a.seqlens_before[b] + i;
    const int blk_i = pos >> 8;
    int blk = -1;
    if (pos < 0 || blk_i >= a.max_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0) report(NF_DEVERR_TABLE);
    } else {
        blk = a.block_table[(size_t)b * a.max_blocks + blk_i];
        if (blk < 0 || blk >= a.num_blocks) {
            if (threadIdx.x == 0 && blockIdx.y == 0) report(NF_DEVERR_BLOCK_ID);
            blk = -1;
        }
    }
    __syncthreads();

    // ---- queries
    if (q0 < q1) {
        float c[4], s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c[e] = lane_turns ? (float)c64[4 * m + e] : 1.f;
            s[e] = lane_turns ? (float)s64[4 * m + e] : 0.f;
        }
        const long long out_at = token * n_q * kHeadDim;
        while (qr < q1) {
            const int r0 = qr;
            qr += kHalfWarps * kAhead;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int r = r0 + kHalfWarps * u;
                if (r >= q1) break;
                float x[4], y[4];
                x0[u].get(x);
                x1[u].get(y);
                if (qr + kHalfWarps * u < q1) {  // the row that takes this one's registers
                    x0[u].load(p.q, q_at + (qr + kHalfWarps * u) * kHeadDim + c0);
                    x1[u].load(p.q, q_at + (qr + kHalfWarps * u) * kHeadDim + c1);
                }
                if (lane_turns) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &v = PAIRS ? (e < 2 ? x[2 * e] : y[2 * e - 4]) : x[e];
                        float &w = PAIRS ? (e < 2 ? x[2 * e + 1] : y[2 * e - 3]) : y[e];
                        const float z = fmaf(v, c[e], -(w * s[e]));
                        w = fmaf(w, c[e], v * s[e]);
                        v = z;
                    }
                }
                Quad<F32>::put(p.q_out, out_at + r * kHeadDim + c0, x);
                Quad<F32>::put(p.q_out, out_at + r * kHeadDim + c1, y);
            }
        }
    }

    // ---- keys and values
    if (blk < 0) return;
    for (; t < k1; t += kRopeWarps) {
        const bool is_k = t < T;
        const int h0 = 2 * (is_k ? t : t - T), h = h0 + (lane >> 4);
        const size_t s0 = ((size_t)blk * H + h0) * kBlock + (pos & (kBlock - 1)), si = s0 + (size_t)(lane >> 4) * kBlock;
        if (FMT == NF_KV_K4V4 && is_k) {
            // channel 4 lane + e: x cos - x' sin in the first of a pair, x cos + x' sin in the second
            const bool turned = 4 * lane < p.rot;
            const bool second = !PAIRS && 4 * lane >= half;  // the second half of the turned channels
            const int f0 = !turned ? 0 : PAIRS ? 2 * lane : 4 * lane - (second ? half : 0);  // frequency of channel 4 lane
            const int partner = !turned || PAIRS ? lane : second ? lane - (half >> 2) : lane + (half >> 2);
            for (int j = 0; j < 2 && h0 + j < H; ++j) {
                Quad<F32> k4;
                k4.load(a.k_new, b * p.k_bs + i * p.k_ts + (h0 + j) * kHeadDim + 4 * lane);
                float x[4], xp[4];
                k4.get(x);
#pragma unroll
                for (int e = 0; e < 4; ++e) xp[e] = PAIRS ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], partner);
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int f = PAIRS ? f0 + (e >> 1) : f0 + e;
                        const double z = (double)xp[e] * s64[f];
                        x[e] = (float)fma((double)x[e], c64[f], (PAIRS ? (e & 1) != 0 : second) ? z : -z);
                    }
                }
                store_k_row<FMT>(a, x, lane, s0 + (size_t)j * kBlock);
            }
            if (t + kRopeWarps < k1) load_kv(t + kRopeWarps);
            continue;
        }
        float x[4], y[4];
        kv0.get(x);
        kv1.get(y);
        if (t + kRopeWarps < k1) load_kv(t + kRopeWarps);
        if (is_k) {
            if (lane_turns) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &v = PAIRS ? (e < 2 ? x[2 * e] : y[2 * e - 4]) : x[e];
                    float &w = PAIRS ? (e < 2 ? x[2 * e + 1] : y[2 * e - 3]) : y[e];
                    const double c = c64[4 * m + e], s = s64[4 * m + e], dv = v, dw = w;
                    v = (float)fma(dv, c, -(dw * s));
                    w = (float)fma(dw, c, dv * s);
                }
            }
            store_row16<FMT>(x, y, m, c0, c1, h < H, a.k_codes, a.k_scales, si);
        } else {
            store_v16<FMT>(a, x, y, m, h < H, si);
        }
    }
}

}  // namespace nf
