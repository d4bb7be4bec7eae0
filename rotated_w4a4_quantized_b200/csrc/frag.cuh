// frag.cuh -- register-level pieces shared by the group-scaled linear and the
// 4-bit cache: rotation of 16 or 32 channels a thread, exact widening of packed
// INT4 codes to int8 and f16, and the warp-level matrix products.
//
// Why mma.sync and not tcgen05 here: these kernels have 1 to 32 columns
// (tokens or queries) and are bound by the bytes of the packed codes.  A
// tcgen05 MMA reads its whole 128-row A operand from TMEM whatever its column
// count, and the codes would have to be stored to TMEM first; the warp-level
// product takes the widened codes straight from the registers they were
// widened in.  Measured rates of the warp-level forms, a warp instruction of
// one sub-core: m16n8k16 f16 and m16n8k32 int8 8 cycles each, so int8 has
// twice the rate; with up to 16 columns they are a third of a kernel's cycles
// at most.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "prep.cuh"

namespace frag {

// Codes of one 32-bit word as f16 pairs (c0, c4), 16 (c1, c5), (c2, c6),
// 16 (c3, c7), each code offset by 8 and all times 2^-24.  A nibble XOR 8 is
// u = code + 8, and an f16 whose bits are a small whole number u is the
// subnormal u 2^-24, exactly, which the matrix product takes at its full value:
// one operation a pair and one shift a word, against two a pair for a
// conversion that removes the offset.  The second of two nibbles stays where it
// is and counts 16 times.  Callers put the factors into the other operand or
// the result and take 8 times the other operand's sum off.
constexpr float kCodeUnit = 1.0f / 16777216.0f;   // 2^-24

// The masks are values that the compiler cannot see: as immediates the AND and
// the XOR, one three-input operation between registers, become two, and a
// product by 16 becomes a shift, which the integer pipe has to run.
struct CodeMasks {
    uint32_t low, low8, high, high8, sixteen;
    __device__ __forceinline__ CodeMasks() {
        const uint32_t z = gridDim.z;   // 1
        sixteen = 15u + z;
        low = 0x000F000Eu + z;
        low8 = 0x00080007u + z;
        high = 0x00F000EFu + z;
        high8 = 0x0080007Fu + z;
    }
};

__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t m, uint32_t x) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(m), "r"(x));   // (w & m) ^ x
    return r;
}

__device__ __forceinline__ void codes_f16(const CodeMasks &k, uint32_t w, uint32_t (&o)[4]) {
    const uint32_t w8 = w >> 8;
    o[0] = and_xor(w, k.low, k.low8);
    o[1] = and_xor(w, k.high, k.high8);
    o[2] = and_xor(w8, k.low, k.low8);
    o[3] = and_xor(w8, k.high, k.high8);
}

// Codes of one 32-bit word (8 codes, low nibble first) as int8: 16 times the
// odd codes and 16 times the even codes (a nibble at the top of a byte is the
// signed code times 16).
__device__ __forceinline__ void codes_s8(const CodeMasks &k, uint32_t w, uint32_t &odd, uint32_t &even) {
    odd = w & 0xF0F0F0F0u;
    even = (w * k.sixteen) & 0xF0F0F0F0u;
}

// The codes themselves as f16 pairs (c0, c4), (c1, c5), (c2, c6), (c3, c7): in
// the low mantissa bits of 0x6400 (1024.0, spacing 1) a nibble XOR 8 reads
// 1024 + code + 8, and one nibble further up 1024 + 16 (code + 8).
__device__ __forceinline__ void widen_f16(const CodeMasks &k, uint32_t w, __half2 (&o)[4]) {
    const uint32_t bias = 0x64006400u, w8 = w >> 8;
    const __half2 low = __float2half2_rn(-1032.0f), sixteenth = __float2half2_rn(0.0625f), high = __float2half2_rn(-72.0f);
    auto half2_of = [](uint32_t v) { return *reinterpret_cast<__half2 *>(&v); };
    o[0] = __hadd2(half2_of(and_xor(w, k.low, k.low8 | bias)), low);
    o[1] = __hfma2(half2_of(and_xor(w, k.high, k.high8 | bias)), sixteenth, high);
    o[2] = __hadd2(half2_of(and_xor(w8, k.low, k.low8 | bias)), low);
    o[3] = __hfma2(half2_of(and_xor(w8, k.high, k.high8 | bias)), sixteenth, high);
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D (16 x 8, int32) += A (16 x 32, int8) B (32 x 8, int8), exact.
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B: the same without a first summand.
__device__ __forceinline__ void mma_s8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}

__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The transpose of an 8 x 8 tile of 16-bit values held one row per 4 lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float bf16_f32(uint16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

__device__ __forceinline__ uint16_t f32_bf16(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// 16 bytes into shared memory (this thread's copies, in groups), or zeros.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- rotation
// The unnormalised rotation of 16 or 32 consecutive channels a thread, whole
// groups in neighbouring lanes (channel order = lane order): 4 or 2 lanes for
// n = 64, 16 or 8 for n = 256.  Digits 0 and 1 run in registers, the others
// over lanes; every quadruple is added as (x_0 + x_1) + (x_2 + x_3), the order
// of the prep kernels, so the bits are theirs.  All 32 lanes take part.  With
// 32 channels a thread adds half of each quadruple of digit 2 by itself: one
// shuffle for two channels there, against two for each (16 for the whole
// rotation of 32 channels, against 64).
template <int E>
__device__ __forceinline__ void lane_digit(float (&v)[E], int stride) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        float p0, p1, s0, s1;
        ptx::add2(p0, p1, v[e], v[e + 1], __shfl_xor_sync(0xFFFFFFFFu, v[e], stride), __shfl_xor_sync(0xFFFFFFFFu, v[e + 1], stride));
        ptx::add2(s0, s1, p0, p1, __shfl_xor_sync(0xFFFFFFFFu, p0, 2 * stride), __shfl_xor_sync(0xFFFFFFFFu, p1, 2 * stride));
        ptx::bfly2(v[e], v[e + 1], s0, s1);
    }
}

__device__ __forceinline__ void rotate(float (&v)[16], bool wide) {
    prep::radix4_digit0(v);
    prep::radix4_stage<4>(v);
    lane_digit(v, 1);
    if (wide) lane_digit(v, 4);
}

__device__ __forceinline__ void rotate(float (&v)[32], bool wide) {
    prep::radix4_digit0(v);
    prep::radix4_stage<4>(v);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        float p0, p1, s0, s1;
        ptx::add2(p0, p1, v[e], v[e + 1], v[16 + e], v[17 + e]);
        ptx::add2(s0, s1, p0, p1, __shfl_xor_sync(0xFFFFFFFFu, p0, 1), __shfl_xor_sync(0xFFFFFFFFu, p1, 1));
        ptx::bfly2(v[e], v[e + 1], s0, s1);
        ptx::bfly2(v[16 + e], v[17 + e], s0, s1);
    }
    if (wide) lane_digit(v, 2);
}

// 2^-digits of the normalised matrix.
__device__ __forceinline__ float norm_of(int group) { return group == 64 ? 0.125f : 0.0625f; }

__device__ __forceinline__ void unpack_bf16x8(uint4 a, float *v) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load16(const uint16_t *p, float (&v)[16]) {
    unpack_bf16x8(*reinterpret_cast<const uint4 *>(p), v);
    unpack_bf16x8(*reinterpret_cast<const uint4 *>(p + 8), v + 8);
}

__device__ __forceinline__ void store16(uint16_t *p, const float (&v)[16], float scale) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i] * scale, v[2 * i + 1] * scale);
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// The largest |v| over `lanes` neighbouring lanes, as float bits: an integer
// maximum, so that an infinity or a NaN (larger still) wins.
template <int E>
__device__ __forceinline__ uint32_t absmax_bits(const float (&v)[E], int lanes) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        m = max(max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu), __float_as_uint(v[e + 1]) & 0x7FFFFFFFu);
    for (int s = 1; s < lanes; s <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    return m;
}

// The bf16 scale of a block whose largest unnormalised |u| has the bits
// `amax`, and the factor that takes u to q's argument.  Scales below 2^-100
// count as 0, so that 1 / s stays finite.
__device__ __forceinline__ uint16_t block_scale(uint32_t amax, float norm, float &factor) {
    const uint16_t s = f32_bf16(__fdiv_rn(__uint_as_float(amax) * norm, 7.0f));
    if (s < ((127 - 100) << 7)) {   // positive bf16 bits order like the values
        factor = 0.0f;
        return 0;
    }
    factor = __frcp_rn(bf16_f32(s)) * norm;
    return s;
}

}  // namespace frag
