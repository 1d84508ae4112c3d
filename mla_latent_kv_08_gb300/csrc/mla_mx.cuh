// The 8-bit latent cache (MLA_KV_MXFP8): its codes, their scales and a warp's
// quantisation of one token.
//
// A group of 32 latent values shares a scale 2^e, held as the biased exponent e + 127
// in one byte (255: not a number); a value is held as an e4m3 code (sign, 4 exponent
// bits of bias 7, 3 fraction bits; largest 448) of c / 2^e. Both multiplications by 2^e
// are exact in fp32 and in bf16, so the only rounding is that of the code.
//
// e is the least with amax / 2^e <= 448 = 1.75 * 2^8, so no value saturates: for
// amax = 1.f * 2^E it is E - 8 where 1.f <= 1.75 and E - 7 above, read off the bf16 bits.
// e is held within [-110, 119], where every value a code stands for is a normal bf16 or
// zero, so that reading back in bf16 is exact: the smallest is 2^-9 * 2^-110, the largest
// 448 * 2^119 = 1.75 * 2^127 (the few bf16 values above it become it).
#pragma once

#include "mla_internal.cuh"

#include <cuda_fp8.h>

namespace mla {

constexpr int kMxGroup = 32;
constexpr int kMxMinE = -110, kMxMaxE = 119;

// Biased scale exponent of a group whose largest magnitude has the bf16 bits `amax`
// (sign cleared; 0x7f80 and above: infinite or not a number).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    const int E = (int)(amax >> 7);
    if (E == 255) return 255u;
    if (E == 0) return (uint32_t)(kMxMinE + 127);          // zero or subnormal: far below the range
    const int e = E - 127 - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
    return (uint32_t)(max(kMxMinE, min(kMxMaxE, e)) + 127);
}
// 2^(b - 127) in fp32; 255: NaN.
__device__ __forceinline__ float mx_scale_f32(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}
// The same in both halves of a bf16 pair.
__device__ __forceinline__ uint32_t mx_scale_bf162(uint32_t b) {
    const uint32_t h = b == 255u ? 0x7fc0u : b == 0u ? 0x0040u : b << 7;
    return h | (h << 16);
}
constexpr uint32_t kMx2p120 = 0x7b807b80u;                  // 2^120 twice, as a bf16 pair
__device__ __forceinline__ uint32_t mul_bf162(uint32_t a, uint32_t b) {
    const __nv_bfloat162 x = __hmul2(*(const __nv_bfloat162 *)&a, *(const __nv_bfloat162 *)&b);
    return *(const uint32_t *)&x;
}
// Four codes (a word, memory order) as two bf16 pairs of their values times 2^-120: a
// code's exponent and fraction bits placed 4 up in a bf16, whose exponent field is then
// the code's; subnormal codes become subnormal and stay right. The byte permute extends the
// code's sign over the high byte of its half, so that a shift by 4 brings the sign to bit 15
// and one mask clears what the shift put between.
__device__ __forceinline__ void mx_place4(uint32_t w, uint32_t &o0, uint32_t &o1) {
    uint32_t lo, hi;                                       // (the intrinsic has no sign mode)
    asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(w));
    asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(hi) : "r"(w));
    o0 = (lo << 4) & 0x87f087f0u;
    o1 = (hi << 4) & 0x87f087f0u;
}
// Codes 0x7f and 0xff are not a number. Bit 7 of each byte of a word of four: whether it is
// one.
__device__ __forceinline__ uint32_t mx_nan4(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// Whether any of several is one, in fewer steps: adding 1 to a byte changes its bit 7 where the
// seven below are ones. (Of bytes, only 0xff carries into the next, and that is one itself.) The
// check takes 2 to 3 % of a decode or verify call (32 sequences, 156k tokens, 128 heads: 92.3
// -> 94.7 us; ahead of the expanding warps' waits it took as much).
__device__ __forceinline__ uint32_t mx_bit7(uint32_t w) { return (w + 0x01010101u) ^ w; }
__device__ __forceinline__ bool mx_any_nan(uint2 c) { return ((mx_bit7(c.x) | mx_bit7(c.y)) & 0x80808080u) != 0; }
__device__ __forceinline__ uint32_t mx_nan16(const uint4 &c) {
    return (mx_bit7(c.x) | mx_bit7(c.y) | mx_bit7(c.z) | mx_bit7(c.w)) & 0x80808080u;
}
// Eight codes (memory order) as bf16. Both products are exact.
__device__ __forceinline__ uint4 mx_expand8(uint2 c, uint32_t scale) {
    uint4 o;
    mx_place4(c.x, o.x, o.y);
    mx_place4(c.y, o.z, o.w);
    o.x = mul_bf162(mul_bf162(o.x, kMx2p120), scale);
    o.y = mul_bf162(mul_bf162(o.y, kMx2p120), scale);
    o.z = mul_bf162(mul_bf162(o.z, kMx2p120), scale);
    o.w = mul_bf162(mul_bf162(o.w, kMx2p120), scale);
    if (mx_any_nan(c)) {
        uint32_t *w = (uint32_t *)&o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t n = mx_nan4(i < 2 ? c.x : c.y) >> (16 * (i & 1));
            if (n & 0x80u) w[i] = (w[i] & 0xffff0000u) | 0x7fc0u;
            if (n & 0x8000u) w[i] = (w[i] & 0xffffu) | 0x7fc00000u;
        }
    }
    return o;
}
// Sixteen codes (memory order) as bf16: `first` times their placed values, where no scale
// is above 1 the scale and 2^120 in one (mx_scale120), else 2^120 and then `second`. Every
// product is exact. (Codes that are not a number come out as +-480: mx_nan16 finds them.)
__device__ __forceinline__ void mx_expand16(const uint4 &c, uint32_t first, uint4 &o0, uint4 &o1) {
    mx_place4(c.x, o0.x, o0.y);
    mx_place4(c.y, o0.z, o0.w);
    mx_place4(c.z, o1.x, o1.y);
    mx_place4(c.w, o1.z, o1.w);
    uint32_t *a = (uint32_t *)&o0, *b = (uint32_t *)&o1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = mul_bf162(a[i], first);
        b[i] = mul_bf162(b[i], first);
    }
}
__device__ __forceinline__ void mx_expand16(const uint4 &c, uint32_t first, uint32_t second, uint4 &o0, uint4 &o1) {
    mx_expand16(c, first, o0, o1);
    uint32_t *a = (uint32_t *)&o0, *b = (uint32_t *)&o1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = mul_bf162(a[i], second);
        b[i] = mul_bf162(b[i], second);
    }
}
// 2^(b - 127 + 120) in both halves, of byte `sel` of four scale bytes that are all at most
// 127 (scales up to 1).
__device__ __forceinline__ uint32_t mx_scale120(uint32_t bytes, uint32_t sel) {
    return __byte_perm(bytes, 0u, 0x4040u | sel | (sel << 8)) * 128u + 0x3c003c00u;
}
// One code, a number, and its scale byte in fp32 (the CUDA-core kernels).
__device__ __forceinline__ float mx_value(uint32_t code, uint32_t scale_byte) {
    const uint32_t h = ((code & 0x7fu) << 4) | ((code & 0x80u) << 8);
    return __uint_as_float(h << 16) * 0x1p120f * mx_scale_f32(scale_byte);
}

// 1152 bytes in and 656 out a token (51k tokens: 19.6 us, 4.7 TB/s; 13.6 at the copy rate).
// Its instructions bound it: 73 % of the issue slots are taken, the memory is a third busy.
// A new token's codes, by one warp: a lane takes 16 values (two lanes a group), 512 a pass.
// `row()` gives the token row of the cache, or below 0 for none; it is asked for once the
// loads are on their way, which do not depend on it (with the look-up first, its chain of
// four loads stood before them).
template <typename Row>
__device__ __forceinline__ void mx_write_token(const AppendParams &p, const __nv_bfloat16 *c, const __nv_bfloat16 *k, Row row) {
    const int lane = threadIdx.x & 31;
    const int r = p.s.r, dR = p.s.dR, ng = r / kMxGroup;
    uint4 rope = make_uint4(0, 0, 0, 0);
    if (lane < dR / 8) rope = ((const uint4 *)k)[lane];            // d_R <= 128: 16 lanes
    long long at = 0;
    for (int g0 = 0; g0 < ng; g0 += 16) {
        const int g = g0 + (lane >> 1);
        const bool act = g < ng;
        uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (act) {
            const uint4 *src = (const uint4 *)(c + g * kMxGroup + 16 * (lane & 1));
            u[0] = src[0];
            u[1] = src[1];
        }
        if (g0 == 0) {
            at = row();
            if (at < 0) return;
        }
        const uint32_t *w = (const uint32_t *)u;
        __nv_bfloat162 mm = __habs2(*(const __nv_bfloat162 *)&w[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) mm = __hmax2_nan(mm, __habs2(*(const __nv_bfloat162 *)&w[i]));
        uint32_t m = *(const uint32_t *)&mm;
        m = max(m & 0xffffu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const uint32_t sb = mx_scale_byte(m);
        if (!act) continue;
        // 2^-e: exponent field 127 - e = 254 - sb, normal for every e of the range. The products
        // are exact in bf16, but for those below 2^-126, whose code is 0 either way.
        const uint32_t inv = ((254u - min(sb, 254u)) << 7) * 0x10001u;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = mul_bf162(w[2 * i], inv), y = mul_bf162(w[2 * i + 1], inv);
            o[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)),
                                                      __NV_SATFINITE, __NV_E4M3) |
                   ((uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u)),
                                                       __NV_SATFINITE, __NV_E4M3) << 16);
            if (sb == 255u) o[i] = 0x7f7f7f7fu;
        }
        *(uint4 *)(p.codes + (size_t)at * r + g * kMxGroup + 16 * (lane & 1)) = make_uint4(o[0], o[1], o[2], o[3]);
        if ((lane & 1) == 0) p.mx_scale[(size_t)at * ng + g] = (uint8_t)sb;
    }
    if (lane < dR / 8) ((uint4 *)(p.rope + (size_t)at * dR))[lane] = rope;
}

}  // namespace mla
