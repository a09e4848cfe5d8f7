// nf_append.cuh -- quantise-and-append of new K/V tokens into the segmented
// pool (the rk8v4 KV dtype of page "3090 单卡跑 Qwen3.8-27B：NInfer 上机实测",
// section 一.3; bit format as defined in nf.h).
//
// One warp per (sequence, new token, kv-head); lane l owns channels 4l..4l+3.
// K: absmax over the warp -> fp16 scale absmax/127 -> int8 codes (4 bytes per
// lane, a coalesced 128-byte row).  V: absmax over each 8-lane group of 32
// channels -> fp16 scale absmax/7 -> 4 nibbles per lane packed into 2 bytes;
// for the int8 KV dtype (same section, --kv-dtype int8) V takes the K rule; the
// fp8 dtype (--kv-dtype fp8) stores e4m3 codes of x / (absmax / 448) for both;
// the RK4V4-E8 reading (page "影片筆記：NInfer + 千问3.8 27b = 1.5倍速@256K上下文",
// section 三) stores 4-bit codes of both with a power-of-two scale per 32 channels.
// Division and rounding are the IEEE fp32 ones (or proven to give the same code,
// see make_codes), round half to even, subnormals kept, so the codes are
// bit-identical to the format definition.
#pragma once

#include "nf_common.cuh"

namespace nf {

struct AppendParams {
    const void *k_new;
    const void *v_new;
    int in_f32;  // 1: fp32 inputs, 0: bf16 inputs
    int batch, n_new, num_kv_heads;
    const int32_t *block_table;
    int max_blocks;
    const int32_t *seqlens_before;
    int num_blocks;
    int fmt;
    void *k_codes;
    __half *k_scales;
    void *v_codes;
    __half *v_scales;
};

__device__ __forceinline__ void load4(const void *base, size_t elem, bool f32, float (&x)[4]) {
    if (f32) {
        const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + elem);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const uint2 v =
            *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(base) + elem);
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
}

// fp16 scale for absmax a and code limit q: fp32 a / q, then fp16 round half to
// even, saturated at 65504 (clamping first gives the same fp16 value).
__device__ __forceinline__ __half make_scale(float a, float q, float &sigma) {
    const float s32 = fminf(__fdiv_rn(a, q), 65504.0f);
    const __half s16 = __float2half_rn(s32);
    sigma = __half2float(s16);
    return s16;
}

// Codes of four channels: round_half_even(fp32(x / sigma)) clamped to [-q, q], 0
// when sigma is 0.
// QUICK: the IEEE quotient is only worked out where it matters.  t = x *
// rcp(sigma) is within 2^-22 of x / sigma relatively and the fp32 quotient within
// 2^-24, so for |t| <= 128 both lie within 2^-14 of each other, and where t is
// further than 2^-13 from every border n + 1/2 the two round alike (beyond 128
// both are clamped).  About one warp in 30 has a lane that is closer and divides.
// The rotary append takes it for its many rows.  append_quant_kernel divides;
// with it 8192 tokens x 8 heads would take 22.6 instead of 24.8 us (K8/V4), 21.8
// instead of 24.4 (int8) and 22.8 instead of 23.0 (fp8), a step's 1 to 4 tokens
// between 0.17 us less (int8) and 0.08 us more (fp8).
template <bool QUICK>
__device__ __forceinline__ void make_codes(const float (&x)[4], float sigma, int q, int (&code)[4]) {
    const float r = sigma == 0.0f ? 0.0f : rcp_approx(sigma);  // sigma >= 2^-24: normal
    float t[4];
    bool sure = QUICK;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        t[c] = x[c] * r;
        sure = sure && fabsf(t[c] - rintf(t[c])) < 0.5f - 0x1p-13f;  // false for infinities and NaN too
    }
    if (!sure) {
#pragma unroll
        for (int c = 0; c < 4; ++c) t[c] = sigma == 0.0f ? 0.0f : __fdiv_rn(x[c], sigma);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) code[c] = min(max(__float2int_rn(t[c]), -q), q);
}

// Four int8 codes (absmax / 127 scale) in one word.
template <bool QUICK>
__device__ __forceinline__ uint32_t pack_codes8(const float (&x)[4], float sigma) {
    int code[4];
    make_codes<QUICK>(x, sigma, 127, code);
    return prmt(prmt((uint32_t)code[0], (uint32_t)code[1], 0x0040), prmt((uint32_t)code[2], (uint32_t)code[3], 0x0040),
                0x5410);
}
// Four nibbles, channel 0 in the lowest.
__device__ __forceinline__ uint32_t pack_codes4(const int (&code)[4]) {
    return ((uint32_t)code[0] & 0xFu) | (((uint32_t)code[1] & 0xFu) << 4) | (((uint32_t)code[2] & 0xFu) << 8) |
           (((uint32_t)code[3] & 0xFu) << 12);
}

// One 128-channel row held 4 channels per lane -> int8 codes (absmax / 127
// scale, a coalesced 128-byte row) and its fp16 scale.
__device__ __forceinline__ void quant_row8(const float (&x)[4], int lane, int8_t *codes, __half *scale) {
    float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    float sigma;
    const __half h = make_scale(a, 127.0f, sigma);
    *reinterpret_cast<uint32_t *>(codes + 4 * lane) = pack_codes8<false>(x, sigma);
    if (lane == 0) *scale = h;
}

// Four e4m3 codes (absmax / 448 scale) in one word.
template <bool QUICK>
__device__ __forceinline__ uint32_t pack_codes_f8(const float (&x)[4], float sigma) {
    // as make_codes: t is within 2^-22 of the fp32 quotient relatively (about 2
    // fp32 steps); an e4m3 border of a normal result lies where the 20 fp32
    // mantissa bits below the 3 kept ones are 0x80000, so outside 8 steps of it,
    // and above the subnormal results, both round alike
    const float r = sigma == 0.0f ? 0.0f : rcp_approx(sigma);
    float t[4];
    bool sure = QUICK;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        t[c] = x[c] * r;
        const uint32_t low = (__float_as_uint(t[c]) & 0xFFFFFu) - 0x80000u + 8u;
        sure = sure && low > 16u && fabsf(t[c]) >= 0x1p-6f && fabsf(t[c]) < 512.0f;
    }
    if (!sure) {
#pragma unroll
        for (int c = 0; c < 4; ++c) t[c] = sigma == 0.0f ? 0.0f : __fdiv_rn(x[c], sigma);
    }
    return f32x4_to_e4m3(t[0], t[1], t[2], t[3]);
}

// The same row -> e4m3 codes of x / scale (scale absmax / 448), 0 when the
// scale is 0.
__device__ __forceinline__ void quant_row_f8(const float (&x)[4], int lane, uint8_t *codes, __half *scale) {
    float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    float sigma;
    const __half h = make_scale(a, 448.0f, sigma);
    *reinterpret_cast<uint32_t *>(codes + 4 * lane) = pack_codes_f8<false>(x, sigma);
    if (lane == 0) *scale = h;
}

// The exponent e of a group with absmax a (see quant_row_e8) and 2^-e.
__device__ __forceinline__ int e8_exponent(float a, float &inv) {
    const uint32_t sb = __float_as_uint(__fdiv_rn(a, 7.0f));
    const int ef = (int)(sb >> 23);  // biased exponent; 0 for zero and subnormal quotients
    int e = ef == 0 ? -126 : ef - 127 + ((sb & 0x7FFFFFu) != 0u ? 1 : 0);
    e = min(max(e, -126), 127);
    // x / 2^e = x * 2^-e exactly (2^-127 is a subnormal factor; a product below
    // the normal range is rounded as the quotient would be)
    inv = e == 127 ? 0x1p-127f : __int_as_float((127 - e) << 23);
    return e;
}
__device__ __forceinline__ uint32_t pack_codes_e8(const float (&x)[4], float inv) {
    int code[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) code[c] = min(max(__float2int_rn(x[c] * inv), -7), 7);
    return pack_codes4(code);
}

// RK4V4-E8 (both K and V): one power-of-two scale 2^e per 32 channels = 8
// lanes, e the smallest integer with 2^e >= fp32(absmax / 7) (read from the
// bits of the quotient: an exact power of two keeps its exponent, anything
// above it takes the next one), clamped to [-126, 127] and stored as the byte
// e + 127; codes round_half_even(x / 2^e) clamped to [-7, 7], packed two per
// byte (the even channel in the low nibble).
__device__ __forceinline__ void quant_row_e8(const float (&x)[4], int lane, uint8_t *codes, uint8_t *scales) {
    float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    float inv;
    const int e = e8_exponent(a, inv);
    *reinterpret_cast<uint16_t *>(codes + 2 * lane) = (uint16_t)pack_codes_e8(x, inv);
    if ((lane & 7) == 0) scales[lane >> 3] = (uint8_t)(e + 127);
}

// One K row (lane l holds channels 4l..4l+3) into slot si of the pool, in the
// pool's format.
template <int FMT>
__device__ __forceinline__ void store_k_row(const AppendParams &p, const float (&k)[4], int lane, size_t si) {
    if constexpr (FMT == NF_KV_BF16)
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.k_codes) + si * kHeadDim + 4 * lane) =
            make_uint2(pack_bf16(k[0], k[1]), pack_bf16(k[2], k[3]));
    else if constexpr (FMT == NF_KV_K4V4)
        quant_row_e8(k, lane, static_cast<uint8_t *>(p.k_codes) + si * (kHeadDim / 2),
                     reinterpret_cast<uint8_t *>(p.k_scales) + si * (kHeadDim / 32));
    else if constexpr (FMT == NF_KV_F8)
        quant_row_f8(k, lane, static_cast<uint8_t *>(p.k_codes) + si * kHeadDim, p.k_scales + si);
    else  // one int8 scale per (token, kv-head)
        quant_row8(k, lane, static_cast<int8_t *>(p.k_codes) + si * kHeadDim, p.k_scales + si);
}

// One V row likewise.
template <int FMT>
__device__ __forceinline__ void store_v_row(const AppendParams &p, const float (&v)[4], int lane, size_t si) {
    if constexpr (FMT == NF_KV_BF16) {
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.v_codes) + si * kHeadDim + 4 * lane) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else if constexpr (FMT == NF_KV_K4V4) {
        quant_row_e8(v, lane, static_cast<uint8_t *>(p.v_codes) + si * (kHeadDim / 2),
                     reinterpret_cast<uint8_t *>(p.v_scales) + si * (kHeadDim / 32));
    } else if constexpr (FMT == NF_KV_F8) {
        quant_row_f8(v, lane, static_cast<uint8_t *>(p.v_codes) + si * kHeadDim, p.v_scales + si);
    } else if constexpr (FMT == NF_KV_K8V8) {
        // int8 KV: V by the K rule
        quant_row8(v, lane, static_cast<int8_t *>(p.v_codes) + si * kHeadDim, p.v_scales + si);
    } else {
        // K8/V4: one scale per 32 channels = 8 lanes
        float av = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, o));
        float sv;
        const __half hv = make_scale(av, 7.0f, sv);
        int code[4];
        make_codes<false>(v, sv, 7, code);
        *reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(p.v_codes) + si * (kHeadDim / 2) + 2 * lane) =
            (uint16_t)pack_codes4(code);
        if ((lane & 7) == 0) p.v_scales[si * (kHeadDim / kVGroup) + (lane >> 3)] = hv;
    }
}

// One kernel per format: with the format branched on in the kernel, K and V each behind a
// branch of its own, the two rows' reductions and quotients did not overlap (8 heads of
// fp8, 1 / 16384 tokens: 2.23 / 46.8 us, now 1.99 / 45.0; int8 2.35 / 50.1, now 2.10 / 47.9).
template <int FMT>
__global__ void __launch_bounds__(256) append_quant_kernel(const AppendParams p) {
    // let the next kernel place its CTAs at once (it waits for this grid to
    // complete before it reads what this one writes)
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long total = (long long)p.batch * p.n_new * p.num_kv_heads;
    if (item >= total) return;
    const int h = (int)(item % p.num_kv_heads);
    const long long bi = item / p.num_kv_heads;
    const int i = (int)(bi % p.n_new);
    const int b = (int)(bi / p.n_new);

    // the new token's values do not depend on where it goes: load them first,
    // so their latency overlaps the lengths -> block-table lookups
    const size_t src = (size_t)item * kHeadDim + 4 * lane;
    float k[4], v[4];
    load4(p.k_new, src, p.in_f32 != 0, k);
    load4(p.v_new, src, p.in_f32 != 0, v);

    const int pos = p.seqlens_before[b] + i;
    const int blk_i = pos >> 8;
    if (pos < 0 || blk_i >= p.max_blocks) {
        if (lane == 0) report(NF_DEVERR_TABLE);
        return;
    }
    const int blk = p.block_table[(size_t)b * p.max_blocks + blk_i];
    if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) report(NF_DEVERR_BLOCK_ID);
        return;
    }
    const size_t si = ((size_t)blk * p.num_kv_heads + h) * kBlock + (pos & (kBlock - 1));

    store_k_row<FMT>(p, k, lane, si);
    store_v_row<FMT>(p, v, lane, si);
}

}  // namespace nf
