// nf_rope.cuh -- rotary positions with several axes on a step's queries and
// keys, fused with the quantised append (nf_rope_append_quant).
//
// Mathematics: frequency i of rot / 2 turns one pair of channels by the angle
//   a_i = position[axis(i)] * inv_freq[i]:  (x, y) -> (x cos - y sin, y cos + x sin).
// Positions of a long context put a_i at 10^5 radians and more, where an fp32
// product is off by hundredths of a radian.  So the angle is taken in turns in
// fp64: a = position * inv_freq is exact (31 + 24 bits; one rounding above
// 2^53), and its turns a / 2 pi come as an unevaluated sum of two doubles (the
// product with the leading double of 1 / 2 pi split exactly by an FMA, plus the
// product with the trailing one); the whole turns are dropped exactly and what
// is left, at most half a turn, goes to sincospi.  cos and sin are then good to
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
// Work: a token has num_q_heads + 2 H_kv rows of 128 channels (queries, keys,
// values); a CTA takes one token and a slice of its rows, works out the token's
// cos and sin once in shared memory, and each warp then takes rows of the
// slice, lane l channels 4l .. 4l + 3 (the partner channel of the halves layout
// comes from the lane rot / 8 away).
#pragma once

#include "nf_append.cuh"
#include "nf_common.cuh"

namespace nf {

constexpr int kRopeWarps = 8;

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
    int slices, rows_per_slice;
    uint8_t axis[kHeadDim / 2];
};

// cos and sin of position * f, see above.
__device__ __forceinline__ void rope_angle(int position, float f, double &c, double &s) {
    constexpr double kInv2PiHi = 0x1.45f306dc9c883p-3, kInv2PiLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi) as hi + lo
    const double a = (double)position * (double)f;
    const double hi = a * kInv2PiHi;
    const double lo = fma(a, kInv2PiHi, -hi) + a * kInv2PiLo;
    const double turn = (hi - rint(hi)) + lo;
    sincospi(2.0 * turn, &s, &c);
}

__global__ void __launch_bounds__(kRopeWarps * 32) rope_append_kernel(const __grid_constant__ RopeParams p) {
    __shared__ double2 cs64[kHeadDim / 2];
    __shared__ float2 cs32[kHeadDim / 2];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const AppendParams &a = p.a;
    const long long token = blockIdx.x / p.slices;
    const int slice = blockIdx.x % p.slices;
    const int b = (int)(token / a.n_new), i = (int)(token % a.n_new);
    if (p.n_valid && i >= p.n_valid[b]) return;  // the whole CTA: padding token
    const int half = p.rot >> 1;
    if (threadIdx.x < half) {
        double c, s;
        rope_angle(p.positions[token * p.n_axes + p.axis[threadIdx.x]], p.inv_freq[threadIdx.x], c, s);
        cs64[threadIdx.x] = make_double2(c, s);
        cs32[threadIdx.x] = make_float2((float)c, (float)s);
    }
    __syncthreads();

    // channel c = 4 lane + e of a row: y = x cos + sgn x' sin, x' its partner
    const bool turned = 4 * lane < p.rot;
    const bool second = !p.pairs && 4 * lane >= half;  // the second half: + sin
    const int f0 = !turned ? 0 : p.pairs ? 2 * lane : 4 * lane - (second ? half : 0);  // frequency of channel 4 lane
    const int partner = !turned || p.pairs ? lane : second ? lane - (half >> 2) : lane + (half >> 2);

    const int rows = p.num_q_heads + 2 * a.num_kv_heads;
    const int r0 = slice * p.rows_per_slice, r1 = min(rows, r0 + p.rows_per_slice);

    // where the new token's K and V go
    const int pos = a.seqlens_before[b] + i;
    const int blk_i = pos >> 8;
    int blk = -1;
    if (pos < 0 || blk_i >= a.max_blocks) {
        if (threadIdx.x == 0 && slice == 0) report(NF_DEVERR_TABLE);
    } else {
        blk = a.block_table[(size_t)b * a.max_blocks + blk_i];
        if (blk < 0 || blk >= a.num_blocks) {
            if (threadIdx.x == 0 && slice == 0) report(NF_DEVERR_BLOCK_ID);
            blk = -1;
        }
    }

    for (int r = r0 + warp; r < r1; r += kRopeWarps) {
        float x[4], xp[4];
        if (r < p.num_q_heads) {
            load4(p.q, b * p.q_bs + i * p.q_ts + (size_t)r * kHeadDim + 4 * lane, a.in_f32 != 0, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) xp[e] = p.pairs ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], partner);
            if (turned) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = cs32[p.pairs ? f0 + (e >> 1) : f0 + e];
                    const bool plus = p.pairs ? (e & 1) : second;
                    x[e] = fmaf(x[e], f.x, plus ? xp[e] * f.y : -(xp[e] * f.y));
                }
            }
            const size_t dst = ((size_t)token * p.num_q_heads + r) * kHeadDim + 4 * lane;
            if (a.in_f32)
                *reinterpret_cast<float4 *>(static_cast<float *>(p.q_out) + dst) = make_float4(x[0], x[1], x[2], x[3]);
            else
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.q_out) + dst) =
                    make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
            continue;
        }
        if (blk < 0) continue;
        const bool is_k = r < p.num_q_heads + a.num_kv_heads;
        const int h = r - p.num_q_heads - (is_k ? 0 : a.num_kv_heads);
        const size_t si = ((size_t)blk * a.num_kv_heads + h) * kBlock + (pos & (kBlock - 1));
        if (is_k) {
            load4(a.k_new, b * p.k_bs + i * p.k_ts + (size_t)h * kHeadDim + 4 * lane, a.in_f32 != 0, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) xp[e] = p.pairs ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], partner);
            if (turned) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const double2 f = cs64[p.pairs ? f0 + (e >> 1) : f0 + e];
                    const bool plus = p.pairs ? (e & 1) : second;
                    const double y = (double)xp[e] * f.y;
                    x[e] = (float)fma((double)x[e], f.x, plus ? y : -y);
                }
            }
            store_k_row(a, x, lane, si);
        } else {
            load4(a.v_new, b * p.v_bs + i * p.v_ts + (size_t)h * kHeadDim + 4 * lane, a.in_f32 != 0, x);
            store_v_row(a, x, lane, si);
        }
    }
}

}  // namespace nf
