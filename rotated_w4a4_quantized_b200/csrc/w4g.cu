// w4g.cu -- the group-scaled few-token variant of the rotated linear layer
// (include/convrot_w4g.h).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/convrot_w4g.h"
#include "frag.cuh"
#include "host.cuh"

namespace w4g {

// ------------------------------------------------------------------ weights
// 32 channels a thread over the matrix as one line of values: a rotation group
// (2 or 8 threads) and a scale group (1, 2 or 4 threads) never cross a row,
// because K is a multiple of both.
//
// Runs once a model.  4096 -> 14336 in 37.7 us with groups of 64, 3.9 TB/s of
// reads and writes, bound by the instructions of rotation and rounding (31.7 us,
// 4.7 TB/s, without a rotation).  16 channels a thread need four times the
// shuffles: 52.6 us.
constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads)
quantize_kernel(const uint16_t *__restrict__ w, int64_t threads, int group, int scale_group,
                uint8_t *__restrict__ qw, uint16_t *__restrict__ sg) {
    const int lanes = scale_group / 32;
    const float norm = group ? frag::norm_of(group) : 1.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kRowThreads; i0 < threads; i0 += step) {
        const int64_t i = i0 + threadIdx.x;
        uint4 raw[4] = {};
        if (i < threads)
#pragma unroll
            for (int e = 0; e < 4; ++e) raw[e] = __ldcs(reinterpret_cast<const uint4 *>(w + 32 * i) + e);
        float x[32];
#pragma unroll
        for (int e = 0; e < 4; ++e) frag::unpack_bf16x8(raw[e], x + 8 * e);
        if (group) frag::rotate(x, group == 256);
        float factor;
        const uint16_t s = frag::block_scale(frag::absmax_bits(x, lanes), norm, factor);
        uint32_t packed[4];
        prep::quantize_pack(x, factor, packed);
        if (i < threads) {
            *reinterpret_cast<uint4 *>(qw + 16 * i) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
            if (i % lanes == 0) sg[i / lanes] = s;
        }
    }
}

// ------------------------------------------------------------------ activations
// The product takes 16-bit whole numbers, n, and a factor f for every 256
// channels of a row: x R = n f with the largest of the 256 at 32000, so the
// rounding is at most 2^-16 of it (bf16 would be off by 2^-8 of each value).  A
// number's high and low byte (signed) go through int8 products of their own.
// Blocks below 2^-100 count as 0; one with a NaN or an infinity has a factor of
// NaN.  A word's 8 channels are 16 bytes: the high bytes of the odd channels,
// of the even ones, then the low bytes in the same order.
constexpr int kStage = 256;                  // channels
constexpr int kLanes = kStage / 16;          // lanes of a block, 16 channels each

// The 16 channels of this lane's part of a block; whole warps call it.
__device__ __forceinline__ void whole_numbers(float (&v)[16], int group, uint4 (&words)[2], float &factor) {
    if (group) frag::rotate(v, group == 256);
    const uint32_t amax = frag::absmax_bits(v, kLanes);
    const float top = __uint_as_float(amax);
    const bool zero = amax < (27u << 23);
    const float f = zero ? 0.0f : 32000.0f / top;
    factor = zero ? 0.0f : (group ? frag::norm_of(group) : 1.0f) * (top / 32000.0f);
    if (amax >= 0x7F800000u) factor = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int n = __float2int_rn(v[8 * half + e] * f);
            hi[e] = static_cast<uint32_t>(n + 128) >> 8;
            lo[e] = static_cast<uint32_t>(n);
        }
        auto bytes = [](uint32_t p, uint32_t q, uint32_t r, uint32_t t) {
            return __byte_perm(__byte_perm(p, q, 0x0040), __byte_perm(r, t, 0x0040), 0x5410);
        };
        words[half] = make_uint4(bytes(hi[1], hi[3], hi[5], hi[7]), bytes(hi[0], hi[2], hi[4], hi[6]),
                                 bytes(lo[1], lo[3], lo[5], lo[7]), bytes(lo[0], lo[2], lo[4], lo[6]));
    }
}

__device__ __forceinline__ void load_part(const uint16_t *x, int64_t m, int K, int part, bool live, float (&v)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.0f;
    if (live && 16 * part < K) frag::load16(x + m * K + 16 * part, v);
}

// Where a row's 16 bytes of a word lie among the `pitch` places of the word:
// with 8 or 16 places the rows of neighbouring words are turned against each
// other, so that the 8 lanes of a 128-byte read hit all banks.
__device__ __forceinline__ int place(int word, int row, int pitch) { return pitch >= 8 ? row ^ ((word & 3) << 1) : row; }

// Numbers [block][word][pitch] and factors [block][pitch] of every 16 rows, as
// the product holds them.  16 channels a thread: 16 rows of 4096 are 4096
// threads, less than one CTA an SM, so that latency is all that counts (about
// 2.5 us, much of it behind the product's start).
__global__ void __launch_bounds__(kRowThreads)
prepare_kernel(const uint16_t *__restrict__ x, int64_t M, int K, int group, int pitch, uint4 *__restrict__ numbers,
               float *__restrict__ factors) {
    // the product's CTAs may be placed as soon as there is room: they fetch
    // weights and wait for this grid before they read its numbers
    ptx::launch_dependents();
    const int blocks = (K + kStage - 1) / kStage, lanes = blocks * kLanes;
    const int64_t total = M * lanes, step = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kRowThreads; i0 < total; i0 += step) {
        const int64_t i = i0 + threadIdx.x, m = i / lanes;
        const int part = static_cast<int>(i % lanes);
        float v[16], factor;
        uint4 words[2];
        load_part(x, m, K, part, i < total, v);
        whole_numbers(v, group, words, factor);
        if (i < total) {
            const int64_t chunk = (m >> 4) * blocks;
            const int r = static_cast<int>(m & 15);
            uint4 *dst = numbers + (chunk * (kStage / 8) + 2 * part) * pitch;
            dst[place(2 * part, r, pitch)] = words[0];
            dst[pitch + place(2 * part + 1, r, pitch)] = words[1];
            if (part % kLanes == 0) factors[(chunk + part / kLanes) * pitch + r] = factor;
        }
    }
}

// ------------------------------------------------------------------ product
// y^T (rows x tokens) = sum over blocks f (sum over scale groups s (codes x
// numbers)): the codes as int8 (16 times the code: three operations for 8 of
// them, of which two on the integer pipe) are the A operand of mma.sync
// m16n8k32 (16 weight rows, 32 channels), the numbers its 8 columns.  Up to 4
// tokens fill the 8 columns with both bytes of their numbers; more take a
// product for each byte.  A group's sum is exact in int32 and joins the row's
// with one FMA by the scale, a block's by the factor.
//
// One CTA has R consecutive rows (R spreads N over the SMs) and all of K.  Its
// warps are (tile of 16 rows, part of K): part p of kp takes the 256-code
// stages p, p + kp, ..., each copied to the warp's own ring in shared memory
// with cp.async (16 rows x 128 bytes a stage; no barrier between warps).
// 16-byte chunk c of row r lies at c ^ (r mod 8), so the reads of one word from
// each of 8 rows spread over all banks.  In step j of a stage lane (g, t) has
// word 4 j + t of rows g and g + 8: the 32 channels of a step are consecutive,
// so scale groups of 32 and more never share an accumulator.
//
// Measured (4096 -> 14336, 4.8 us of bytes; CUDA graphs): one token with scale
// groups of 64 in 10.4 us (3.0 TB/s), 16 with groups of 128 in 15.0, of which
// prepare_kernel is 2.5; 12288 -> 8197 (8.7 us of bytes), 5 tokens, groups of
// 32, in 20.4 (2.8 TB/s).  About 5 us of the first are the launch, the rows'
// numbers and the first copies' latency; then the loop's instructions bound it,
// half an instruction a cycle and sub-core: taking the codes apart and, with
// small scale groups, turning int32 sums into fp32 and scaling them.  bf16
// codes and activations took 17.8 us for one token and 31 for 16.
//
// Choices, each with both sides measured on the first layer, us:
// - columns (TOK 4, 8, 16: the smallest that holds the tokens).  One token
//   10.1 with 4, 11.2 with 8, 14.0 with 16; 8 tokens 12.8 with 8, 15.8 with 16.
// - the rows' numbers.  Few rows are turned into numbers by every CTA while its
//   first weights are on their way, more by prepare_kernel once.  Two tokens
//   10.6 in the product, 12.0 with prepare_kernel; 5 tokens 14.0 and 12.4.  They
//   meet at kFusedLanes (4 tokens: 12.1 and 12.3; 1024 -> 4096, 8 tokens: 4.2
//   and 4.9).
// - stages of a ring (depth_of): one on its way while one is used is enough
//   for 16 warps, and more only delay the activations' loads.  Measured for 1,
//   4, 5, 8, 9 and 16 tokens, scale groups of 32, 64 and 128, and 1024 -> 4096,
//   4096 -> 14336, 12288 -> 8197: 5 and 8 tokens with groups of 32 take 0.5, 9
//   and 4% less with 3 stages than with 2 (4096 -> 14336, 5 tokens: 12.6 against
//   13.9); every other class takes between 1% less and 6% more.
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kStageBytes = 16 * kStage / 2;
// Stages of a warp's ring; there is room for kRing of them in every variant, so
// that what else fits does not depend on it.
constexpr int kRing = 3;
__host__ __device__ constexpr int depth_of(int tok, int scale_group) { return tok == 8 && scale_group == 32 ? 3 : 2; }
constexpr int kRingBytes = kWarps * kRing * kStageBytes;
// numbers and factors held at a time
constexpr int kActBytes = 226 * 1024 - kRingBytes;
constexpr int kMaxRows = 128;                // of a CTA
constexpr int kFusedLanes = 2 * kThreads;    // lanes of 16 channels that a CTA turns into numbers itself

struct Args {
    const uint16_t *x;       // [M][K], or NULL: prepared
    const uint4 *numbers;
    const float *factors;
    const uint8_t *qw;
    const uint16_t *sg;
    const uint16_t *bias;
    uint16_t *y;
    int64_t M, N;
    int K, R, group;
    int slice;               // stages of numbers in shared memory at a time
};

// TOK: tokens of a CTA, 4, 8 or 16.  SG: scale group.
template <int TOK, int SG>
__global__ void __launch_bounds__(kThreads) product_kernel(Args a) {
    constexpr bool HALF = TOK == 4;          // columns 0-3 high bytes, 4-7 low bytes
    constexpr int NT = HALF ? 1 : TOK / 8;
    constexpr int GROUPS = kStage / SG;      // scale groups of a stage
    constexpr int STEPS = SG / 32;           // of a group
    constexpr int kDepth = depth_of(TOK, SG);
    static_assert(kDepth <= kRing);
    extern __shared__ uint4 smem[];
    __shared__ uint4 zeros;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 16;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(16), a.M - m0));
    const int pitch = HALF ? tokens : TOK;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * a.R;
    const int rows = static_cast<int>(min(static_cast<int64_t>(a.R), a.N - n0));
    const int stages = (a.K + kStage - 1) / kStage, lanes = stages * kLanes;

    // rows that the CTA turns into numbers itself: their first values first
    uint4 raw[2];
    auto load_raw = [&](int i) {
        const int m = i / lanes, p = i % lanes;
        raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
        if (m < tokens && 16 * p < a.K) {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.x + m * a.K + 16 * p);
            raw[0] = src[0];
            raw[1] = src[1];
        }
    };
    if (a.x) load_raw(tid);
    const int tiles = (rows + 15) / 16;
    const int parts = min(kWarps / tiles, stages);
    const int tile = warp % tiles, part = warp / tiles;
    const bool works = part < parts;
    const int tile_rows = min(16, rows - 16 * tile);
    const int groups = a.K / SG;

    const uint32_t ring = ptx::smem_u32(smem) + warp * (kDepth * kStageBytes);
    uint4 *act = smem + kRingBytes / 16;   // [slice * 32 words][pitch]
    float *fac = reinterpret_cast<float *>(act + a.slice * (kStage / 8) * pitch);   // [slice][pitch]
    // this lane's copies of a stage: rows lane / 8 + 0, 4, 8, 12, chunk lane % 8
    const int chunk = lane & 7, copy_row = lane >> 3;
    const uint8_t *wsrc = a.qw + (n0 + 16 * tile + copy_row) * (a.K / 2) + 16 * chunk;

    uint32_t copy_dst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) copy_dst[i] = ring + (copy_row + 4 * i) * 128 + ((chunk ^ ((copy_row + 4 * i) & 7)) << 4);
    auto request = [&](int stage, int slot) {
        if (works && stage < stages) {
            const uint8_t *src = wsrc + stage * (kStage / 2);
            if (tile_rows == 16 && (stage + 1) * kStage <= a.K) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    prep::cp_async16(copy_dst[i] + slot * kStageBytes, src + static_cast<int64_t>(i) * (2 * a.K));
            } else {
                const bool inside = stage * (kStage / 2) + 16 * chunk < a.K / 2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool live = inside && copy_row + 4 * i < tile_rows;
                    frag::cp_async16_or_zero(copy_dst[i] + slot * kStageBytes,
                                             live ? src + static_cast<int64_t>(i) * (2 * a.K) : a.qw, live);
                }
            }
        }
        prep::cp_async_commit();
    };
    // scales of rows g and g + 8 of a stage, two to a register: one load a row
    // where every row's stages begin on the load's boundary
    constexpr int PAIRS = GROUPS / 2;
    const bool row_a = works && g < tile_rows, row_b = works && g + 8 < tile_rows;
    const uint16_t *srow = a.sg + (n0 + 16 * tile + g) * groups;
    const bool whole = a.K % kStage == 0;
    auto load_row_scales = [&](const uint16_t *p, int left, uint32_t (&s)[PAIRS]) {
        if (whole) {
            if constexpr (PAIRS == 1) s[0] = *reinterpret_cast<const uint32_t *>(p);
            else if constexpr (PAIRS == 2) *reinterpret_cast<uint2 *>(s) = *reinterpret_cast<const uint2 *>(p);
            else *reinterpret_cast<uint4 *>(s) = *reinterpret_cast<const uint4 *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const uint32_t lo = 2 * i < left ? p[2 * i] : 0u, hi = 2 * i + 1 < left ? p[2 * i + 1] : 0u;
                s[i] = lo | hi << 16;
            }
        }
    };
    auto load_scales = [&](int stage, uint32_t (&s)[2][PAIRS]) {
        if (stage >= stages) return;
        const uint16_t *p = srow + stage * GROUPS;
        const int left = groups - stage * GROUPS;
        if (row_a) load_row_scales(p, left, s[0]);
        if (row_b) load_row_scales(p + 8 * static_cast<int64_t>(groups), left, s[1]);
    };

    // the CTA's scales are one run of bytes: into L2 ahead of their loads, which
    // are a stage ahead of their use
    {
        const uint8_t *first = reinterpret_cast<const uint8_t *>(a.sg + n0 * groups);
        for (int64_t at = static_cast<int64_t>(tid) * 128; at < static_cast<int64_t>(rows) * groups * 2; at += kThreads * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(first + at));
    }
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) request(part + i * parts, i);
    uint32_t next[2][PAIRS] = {};
    load_scales(part, next);

    const frag::CodeMasks masks;
    // this lane's column of the numbers: a token's (both bytes', or with HALF
    // one byte's) 8 or 16 bytes of a word; columns without a token read zeros
    const int token = HALF ? g & 3 : g;
    if (tid == 0) zeros = make_uint4(0, 0, 0, 0);
    float acc[NT][4] = {};
    int stage = part, slot = 0;
    if (!a.x) ptx::grid_dependency_wait();
    for (int s0 = 0; s0 < stages; s0 += a.slice) {
        const int s1 = min(stages, s0 + a.slice);
        if (s0) __syncthreads();             // the last slice has been read
        if (a.x) {                           // one slice
#pragma unroll 1
            for (int i0 = 0; i0 < tokens * lanes; i0 += kThreads) {
                const int i = i0 + tid, m = i / lanes, p = i % lanes;
                if (i0) load_raw(i);
                float v[16], factor;
                uint4 words[2];
                frag::unpack_bf16x8(raw[0], v);
                frag::unpack_bf16x8(raw[1], v + 8);
                whole_numbers(v, a.group, words, factor);
                if (m < tokens) {
                    act[2 * p * pitch + place(2 * p, m, pitch)] = words[0];
                    act[(2 * p + 1) * pitch + place(2 * p + 1, m, pitch)] = words[1];
                    if (p % kLanes == 0) fac[p / kLanes * pitch + m] = factor;
                }
            }
        } else {
            // (in the same group of copies as the warp's latest weights)
            const int n = (s1 - s0) * (kStage / 8) * pitch;
            const int64_t from = (static_cast<int64_t>(blockIdx.y) * stages + s0) * pitch;
            const uint4 *src = a.numbers + from * (kStage / 8);
            for (int i = tid; i < n; i += kThreads) frag::cp_async16_or_zero(ptx::smem_u32(act + i), src + i, true);
            for (int i = tid; i < (s1 - s0) * pitch; i += kThreads) fac[i] = a.factors[from + i];
            prep::cp_async_commit();
            frag::cp_async_wait<0>();
        }
        __syncthreads();
        if (!works) continue;
        for (; stage < s1; stage += parts) {
            request(stage + (kDepth - 1) * parts, (slot + kDepth - 1) % kDepth);
            uint32_t sc[2][PAIRS];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                sc[0][i] = next[0][i];
                sc[1][i] = next[1][i];
            }
            load_scales(stage + parts, next);
            frag::cp_async_wait<kDepth - 1>();
            __syncwarp();
            const uint8_t *src = reinterpret_cast<const uint8_t *>(smem) + warp * (kDepth * kStageBytes) + slot * kStageBytes + 128 * g + 4 * t4;
            const uint4 *xs = act + ((stage - s0) * (kStage / 8) + t4) * pitch + (HALF ? token : token ^ (t4 << 1));
            // HALF: lanes without a token read zeros
            const uint2 *xh = reinterpret_cast<const uint2 *>(token < tokens ? xs : &zeros) + (g >> 2);
            const int xh_step = token < tokens ? 8 * pitch : 0;
            float block[NT][4] = {};
            int high[NT][4], low[NT][4];
#pragma unroll
            for (int j = 0; j < kStage / 32; ++j) {
                uint32_t ao, ae, bo, be;
                frag::codes_s8(masks, *reinterpret_cast<const uint32_t *>(src + ((j ^ g) << 4)), ao, ae);
                frag::codes_s8(masks, *reinterpret_cast<const uint32_t *>(src + 1024 + ((j ^ g) << 4)), bo, be);
                const bool begins = j % STEPS == 0;
                if constexpr (HALF) {
                    const uint2 x = xh[j * xh_step];
                    if (begins) frag::mma_s8_first(high[0], ao, bo, ae, be, x.x, x.y);
                    else frag::mma_s8(high[0], ao, bo, ae, be, x.x, x.y);
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (8 * nt + token < tokens) x = xs[4 * j * TOK + 8 * nt];
                        if (begins) {
                            frag::mma_s8_first(high[nt], ao, bo, ae, be, x.x, x.y);
                            frag::mma_s8_first(low[nt], ao, bo, ae, be, x.z, x.w);
                        } else {
                            frag::mma_s8(high[nt], ao, bo, ae, be, x.x, x.y);
                            frag::mma_s8(low[nt], ao, bo, ae, be, x.z, x.w);
                        }
                    }
                }
                if ((j + 1) % STEPS == 0) {
                    constexpr uint32_t upper = 0xFFFF0000u;
                    const int i = j / STEPS;
                    const float fa = __uint_as_float(i & 1 ? sc[0][i >> 1] & upper : sc[0][i >> 1] << 16);
                    const float fb = __uint_as_float(i & 1 ? sc[1][i >> 1] & upper : sc[1][i >> 1] << 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            block[nt][x] = fmaf(x < 2 ? fa : fb, static_cast<float>(HALF ? high[nt][x] : 256 * high[nt][x] + low[nt][x]), block[nt][x]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int m = 8 * nt + (HALF ? 2 * (t4 & 1) : 2 * t4) + x;
                    const float f = m < tokens ? fac[(stage - s0) * pitch + m] : 0.0f;
                    acc[nt][x] = fmaf(f, block[nt][x], acc[nt][x]);
                    acc[nt][2 + x] = fmaf(f, block[nt][2 + x], acc[nt][2 + x]);
                }
            __syncwarp();                    // the slot is free again
            slot = (slot + 1) % kDepth;
        }
    }
    frag::cp_async_wait<0>();

    // ---- join the bytes and the parts of K in their order, add the bias, round
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);   // [parts][tokens][tiles * 16]
    const int columns = tiles * 16;
    if constexpr (HALF)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[0][x] = fmaf(256.0f, acc[0][x], __shfl_xor_sync(0xFFFFFFFFu, acc[0][x], 2));
    if (works) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int m = 8 * nt + 2 * t4 + (x & 1);
                if (m < (HALF ? min(4, tokens) : tokens)) red[(part * tokens + m) * columns + 16 * tile + g + 8 * (x >> 1)] = acc[nt][x] * (1.0f / 16.0f);
            }
    }
    __syncthreads();
    for (int i = tid; i < tokens * rows; i += kThreads) {
        const int m = i / rows, r = i % rows;
        float sum = 0.0f;
        for (int p = 0; p < parts; ++p) sum += red[(p * tokens + m) * columns + r];
        if (a.bias) sum += frag::bf16_f32(a.bias[n0 + r]);
        a.y[(m0 + m) * a.N + n0 + r] = frag::f32_bf16(sum);
    }
}

}  // namespace w4g

// ====================================================================== host

namespace {

using namespace w4g;


template <int TOK, int SG>
bool opt_in() {
    return cudaFuncSetAttribute(product_kernel<TOK, SG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kRingBytes + kActBytes) == cudaSuccess;
}

convrot_status setup(int *dev) {
    return host::device_setup(dev, [] {
        return opt_in<4, 32>() && opt_in<4, 64>() && opt_in<4, 128>() && opt_in<8, 32>() && opt_in<8, 64>() &&
               opt_in<8, 128>() && opt_in<16, 32>() && opt_in<16, 64>() && opt_in<16, 128>();
    });
}

convrot_status check_shape(int64_t rows, int64_t K, int group, int scale_group) {
    if ((group != 0 && group != 64 && group != 256) || (scale_group != 32 && scale_group != 64 && scale_group != 128))
        return CONVROT_ERR_GROUP;
    if (rows < 0 || rows > (int64_t(1) << 30) || K < 64 || K > CONVROT_MAX_K || K % 64 || (group && K % group) ||
        K % scale_group)
        return CONVROT_ERR_SHAPE;
    return CONVROT_OK;
}

unsigned row_grid(int64_t threads, int sms) {
    const int64_t n = (threads + kRowThreads - 1) / kRowThreads;
    return static_cast<unsigned>(n < 8 * sms ? n : 8 * sms);
}

// Places of a word's rows (place()).
int64_t pitch_of(int64_t M) { return M <= 4 ? M : M <= 8 ? 8 : 16; }

// Stages of numbers that the shared memory holds beside the weights' rings.
int64_t stages_held(int64_t M) {
    return kActBytes / ((kStage * 2 + static_cast<int64_t>(sizeof(float))) * pitch_of(M));
}

// Whether every CTA of the product turns the rows into numbers itself: few
// enough of them, all held at once.
bool fused(int64_t M, int64_t K) {
    const int64_t blocks = (K + kStage - 1) / kStage;
    return M <= 16 && M * blocks * kLanes <= kFusedLanes && blocks <= stages_held(M);
}

template <int TOK>
convrot_status launch_product(const Args &a, int scale_group, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.N + a.R - 1) / a.R), static_cast<unsigned>((a.M + 15) / 16));
    const size_t smem = kRingBytes + a.slice * (kStage * 2 + sizeof(float)) * pitch_of(a.M);
    auto go = [&](auto *kernel) {
        if (!a.x) return host::launch_dependent(kernel, grid, dim3(kThreads), smem, stream, a);
        kernel<<<grid, kThreads, smem, stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
    };
    return scale_group == 32 ? go(product_kernel<TOK, 32>)
                             : scale_group == 64 ? go(product_kernel<TOK, 64>) : go(product_kernel<TOK, 128>);
}

}  // namespace

extern "C" {

convrot_status convrot_w4g_quantize_weight(const void *w_bf16, int64_t N, int64_t K, int group,
                                           int scale_group, uint8_t *qw, void *sg_bf16,
                                           convrot_stream_t stream) {
    convrot_status st = check_shape(N, K, group, scale_group);
    if (st != CONVROT_OK) return st;
    if (N == 0) return CONVROT_OK;
    if (!w_bf16 || !qw || !sg_bf16) return CONVROT_ERR_NULL;
    if (!host::aligned16({w_bf16, qw, sg_bf16})) return CONVROT_ERR_ALIGN;
    int dev;
    if ((st = setup(&dev)) != CONVROT_OK) return st;
    if ((st = host::check_device_ptrs(dev, {w_bf16, qw, sg_bf16})) != CONVROT_OK) return st;
    if (host::overlap({{qw, N * K / 2}, {sg_bf16, N * (K / scale_group) * 2}}, {{w_bf16, N * K * 2}})) return CONVROT_ERR_OVERLAP;
    const int64_t threads = N * (K / 32);
    quantize_kernel<<<row_grid(threads, host::g_dev[dev].num_sms), kRowThreads, 0, stream>>>(
        static_cast<const uint16_t *>(w_bf16), threads, group, scale_group, qw, static_cast<uint16_t *>(sg_bf16));
    return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

size_t convrot_w4g_workspace_size(int64_t M, int64_t K) {
    if (M <= 0 || K <= 0 || K > CONVROT_MAX_K || fused(M, K)) return 0;
    const size_t blocks = static_cast<size_t>((M + 15) / 16 * pitch_of(M)) * static_cast<size_t>((K + kStage - 1) / kStage);
    return host::round256(blocks * kStage * 2) + host::round256(blocks * sizeof(float));
}

convrot_status convrot_w4g_linear(const void *x_bf16, const uint8_t *qw, const void *sg_bf16,
                                  const void *bias_bf16, int64_t M, int64_t N, int64_t K,
                                  int group, int scale_group, void *workspace, size_t ws_bytes,
                                  void *y_bf16, convrot_stream_t stream) {
    convrot_status st = check_shape(M, K, group, scale_group);
    if (st != CONVROT_OK) return st;
    if (N < 0 || N > (int64_t(1) << 30) || M > 65535 * 16 || M * N > (int64_t(1) << 40)) return CONVROT_ERR_SHAPE;
    if (M == 0 || N == 0) return CONVROT_OK;
    const size_t need = convrot_w4g_workspace_size(M, K);
    if (!x_bf16 || !qw || !sg_bf16 || !y_bf16 || (need && !workspace)) return CONVROT_ERR_NULL;
    if (need && (ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))) return CONVROT_ERR_WORKSPACE;
    if (!host::aligned16({x_bf16, qw, sg_bf16, bias_bf16, y_bf16})) return CONVROT_ERR_ALIGN;
    int dev;
    if ((st = setup(&dev)) != CONVROT_OK) return st;
    if ((st = host::check_device_ptrs(dev, {x_bf16, qw, sg_bf16, bias_bf16, y_bf16, need ? workspace : nullptr})) != CONVROT_OK)
        return st;
    if (host::overlap({{y_bf16, M * N * 2}, {need ? workspace : nullptr, static_cast<int64_t>(need)}},
                      {{x_bf16, M * K * 2}, {qw, N * K / 2}, {sg_bf16, N * (K / scale_group) * 2}, {bias_bf16, N * 2}}))
        return CONVROT_ERR_OVERLAP;
    const int sms = host::g_dev[dev].num_sms;
    const uint16_t *x = static_cast<const uint16_t *>(x_bf16);
    const int64_t blocks = (K + kStage - 1) / kStage, pitch = pitch_of(M), places = (M + 15) / 16 * pitch;
    uint4 *numbers = nullptr;
    float *factors = nullptr;
    if (need) {
        numbers = static_cast<uint4 *>(workspace);
        factors = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + host::round256(places * blocks * kStage * 2));
        prepare_kernel<<<row_grid(M * blocks * kLanes, sms), kRowThreads, 0, stream>>>(x, M, static_cast<int>(K), group, static_cast<int>(pitch),
                                                                                       numbers, factors);
        if (cudaGetLastError() != cudaSuccess) return CONVROT_ERR_CUDA;
    }
    // rows of a CTA: N spread evenly over whole waves of one CTA an SM
    const int64_t waves = (N + static_cast<int64_t>(sms) * kMaxRows - 1) / (static_cast<int64_t>(sms) * kMaxRows);
    const int R = static_cast<int>((N + sms * waves - 1) / (sms * waves));
    // the numbers' slices: as few as the shared memory allows, of even length
    const int64_t room = stages_held(M), slices = (blocks + room - 1) / room;
    const int64_t slice = (blocks + slices - 1) / slices;
    Args a{need ? nullptr : x, numbers, factors, qw, static_cast<const uint16_t *>(sg_bf16),
           static_cast<const uint16_t *>(bias_bf16), static_cast<uint16_t *>(y_bf16), M, N, static_cast<int>(K), R, group,
           static_cast<int>(slice)};
    return M <= 4 ? launch_product<4>(a, scale_group, stream)
                  : M <= 8 ? launch_product<8>(a, scale_group, stream) : launch_product<16>(a, scale_group, stream);
}

}  // extern "C"
