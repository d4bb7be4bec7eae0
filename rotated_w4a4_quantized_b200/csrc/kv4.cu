// kv4.cu -- the rotated INT4 cache of keys and values (include/convrot_kv4.h):
// the plan of a step, append, read and the attention over the cache.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/convrot_kv4.h"
#include "frag.cuh"
#include "host.cuh"

namespace kv4 {

__device__ __forceinline__ void page_error() { atomicExch(&g_convrot_error, CONVROT_ERR_PAGE); }

struct Cache {
    uint8_t *kc;
    uint16_t *ks;
    uint8_t *vc;
    uint16_t *vs;
    int64_t num_pages;
    int heads, page_shift, D, group;
};

// ------------------------------------------------------------------ plan
// One pass of integer prefix sums over the requests, done by every CTA for
// itself (B is at most 8192: a few loads a thread and block scans, less than a
// second launch would cost), then a grid-stride loop over the new tokens and
// the taken pages, each found by binary search in the prefix sums in shared
// memory.  Nothing that one CTA writes is read by another: pages that come back
// and go out again in the same step are read from the finished request's table
// row, not from the stack.
//
// Bound by latency: 64 requests with a token each in 5.4 us, 1024 requests with
// 145,000 tokens in 7.9 us (1.8 MB; 0.3 us of bytes): the launch, one load of
// the lengths, 32-lane scans with one of the warps' sums (10.5 us with a scan of
// 10 steps over the block), ten steps of a search and one load of a table entry.
constexpr int kPlanThreads = 1024;

struct PlanArgs {
    const int *cached, *fresh;
    int B, page_shift;
    int *table;
    int64_t max_pages;
    int *free_pages;
    int64_t capacity;
    const int *free_count;
    int64_t max_tokens;
    int *seq_lens, *cu_q;
    long long *slots;
    int *positions, *result;
};

// The last b of cu[0 .. B] with cu[b] <= i, among those with cu[b + 1] > i.
__device__ __forceinline__ int find(const int *cu, int B, int i) {
    int lo = 0, hi = B;   // cu[lo] <= i < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
    extern __shared__ int sm[];
    int *cu_q = sm, *cu_take = cu_q + (a.B + 1), *cu_back = cu_take + (a.B + 1), *held_by = cu_back + (a.B + 1);
    __shared__ long long warp_sum[3][32];
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t count = *a.free_count;
    if (tid == 0) bad = 0;
    __syncthreads();

    const int64_t mask = (int64_t(1) << a.page_shift) - 1;
    long long carry[3] = {0, 0, 0};
    for (int base = 0; base < a.B; base += kPlanThreads) {
        const int b = base + tid;
        long long v[3] = {0, 0, 0};
        if (b < a.B) {
            const int64_t c = a.cached[b], n = a.fresh[b];
            held_by[b] = static_cast<int>(c);
            const int64_t have = (c + mask) >> a.page_shift;
            int why = 0;
            if (c < 0 || have > a.max_pages) why = 4;
            else if (n < 0) v[2] = have;
            else {
                const int64_t need = (c + n + mask) >> a.page_shift;
                if (need > a.max_pages || c + n > 0x7FFFFFFF) why = 2;
                else {
                    v[0] = n;
                    v[1] = need - have;
                }
            }
            if (why) atomicMax(&bad, why);
        }
        // inclusive scan over the block: lanes, then the warps' sums
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            for (int s = 1; s < 32; s <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, v[k], s);
                if (lane >= s) v[k] += u;
            }
            if (lane == 31) warp_sum[k][warp] = v[k];
        }
        __syncthreads();
        if (warp < 3) {
            long long w = warp_sum[warp][lane];
            for (int s = 1; s < 32; s <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, w, s);
                if (lane >= s) w += u;
            }
            warp_sum[warp][lane] = w;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            v[k] += carry[k] + (warp ? warp_sum[k][warp - 1] : 0);
            carry[k] += warp_sum[k][31];
        }
        if (b < a.B) {
            // sums beyond 2^31 - 1 are refused below, before any is used
            cu_q[b + 1] = static_cast<int>(v[0]);
            cu_take[b + 1] = static_cast<int>(v[1]);
            cu_back[b + 1] = static_cast<int>(v[2]);
        }
        __syncthreads();
    }
    if (tid == 0) cu_q[0] = cu_take[0] = cu_back[0] = 0;
    __syncthreads();

    const int64_t held = count + carry[2];
    int status = bad;
    if (!status && (count < 0 || held > a.capacity)) status = 4;
    if (!status && (carry[0] > a.max_tokens || carry[0] > 0x7FFFFFFF)) status = 3;
    if (!status && carry[1] > held) status = 1;
    const bool ok = status == 0;
    const int tokens = ok ? static_cast<int>(carry[0]) : 0;
    const int taken = ok ? static_cast<int>(carry[1]) : 0;
    const int returned = ok ? static_cast<int>(carry[2]) : 0;

    // The page at place i of the stack after the returned pages were pushed.
    auto stack_at = [&](int64_t i) -> int {
        if (i < count) return a.free_pages[i];
        const int r = static_cast<int>(i - count);
        const int b = find(cu_back, a.B, r);
        return a.table[b * a.max_pages + (r - cu_back[b])];
    };
    auto taken_page = [&](int p) -> int { return stack_at(held - 1 - p); };

    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    for (int64_t t = first; t < a.max_tokens; t += step) {
        long long slot = -1;
        int pos = -1;
        if (t < tokens) {
            const int b = find(cu_q, a.B, static_cast<int>(t));
            const int c = held_by[b];
            pos = c + static_cast<int>(t) - cu_q[b];
            const int have = static_cast<int>((c + mask) >> a.page_shift);
            const int j = pos >> a.page_shift;
            const int id = j < have ? a.table[b * a.max_pages + j] : taken_page(cu_take[b] + j - have);
            slot = (static_cast<long long>(id) << a.page_shift) + (pos & mask);
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    for (int64_t p = first; p < taken; p += step) {
        const int b = find(cu_take, a.B, static_cast<int>(p));
        const int have = static_cast<int>((held_by[b] + mask) >> a.page_shift);
        a.table[b * a.max_pages + have + static_cast<int>(p) - cu_take[b]] = taken_page(static_cast<int>(p));
    }
    for (int64_t r = first; r < returned; r += step) {
        const int b = find(cu_back, a.B, static_cast<int>(r));
        a.free_pages[count + r] = a.table[b * a.max_pages + (static_cast<int>(r) - cu_back[b])];
    }
    for (int64_t b = first; b <= a.B; b += step) {
        a.cu_q[b] = ok ? cu_q[b] : 0;
        if (b < a.B) {
            const int c = held_by[b], n = a.fresh[b];
            a.seq_lens[b] = !ok ? c : n < 0 ? 0 : c + n;
        }
    }
    if (first == 0) {
        a.result[0] = static_cast<int>(ok ? held - taken : count);
        a.result[1] = taken;
        a.result[2] = tokens;
        a.result[3] = status;
    }
}

// ------------------------------------------------------------------ append, read
// 16 or 32 channels a thread, neighbouring lanes a row, the key's and the
// value's row of a (token, head) by the same threads, so that their loads are
// on the way together.  I: the type of thread numbers, 32 bits where they
// suffice (45.0 against 44.7 us below; 64-bit numbers are there for calls of
// more than 2^31 threads).
//
// 16384 tokens, 8 heads of 128 (12.9 us of bytes each): append in 20.7 us
// (4.1 TB/s), read in 17.7 us (4.8 TB/s).  Append is bound by instruction
// issue, above all shuffles and the roundings to codes.  With 32 channels a
// thread a row takes a quarter of the shuffles, but a call of few rows half of
// the threads, whose latency counts: 16 channels take 26.4 us there and 32 20.7;
// for 64 tokens, append and read, 5.5 and 6.3.  They meet at kFewChannels (4096
// tokens: 17.5 and 17.3).  Read has no rounding and packed arithmetic, and
// 16 channels a thread, whose stores spread over half as many lines an
// instruction, are faster: 17.7 against 20.4 us.
constexpr int kRowThreads = 256;
constexpr int64_t kFewChannels = 24576;   // of the keys, an SM: below, append takes 16 a thread

__device__ __forceinline__ bool slot_ok(const Cache &c, long long slot) {
    if (slot < 0) return false;
    if (slot >= (c.num_pages << c.page_shift)) {
        page_error();
        return false;
    }
    return true;
}

// Row index of (slot, head) in the codes and scales.
__device__ __forceinline__ int64_t row_at(const Cache &c, long long slot, int h) {
    const int64_t id = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
    return ((id * c.heads + h) << c.page_shift) + off;
}

// E: channels of a thread.
template <int D, int E, class I>
__global__ void __launch_bounds__(kRowThreads, 4)
append_kernel(Cache c, const uint16_t *__restrict__ k, int64_t ldk, const uint16_t *__restrict__ v,
              int64_t ldv, const long long *__restrict__ slots, I total) {
    constexpr int LANES = D / E;
    const float norm = frag::norm_of(c.group);
    for (I i0 = static_cast<I>(blockIdx.x) * kRowThreads; i0 < total; i0 += gridDim.x * kRowThreads) {
        const I i = i0 + threadIdx.x, row = i / LANES, t = row / c.heads;
        const int part = static_cast<int>(i % LANES), h = static_cast<int>(row - t * c.heads);
        // (rows that are skipped are loaded too: nothing waits for the slot)
        uint4 raw[2][E / 8] = {};
        long long slot = -1;
        if (i < total) {
            const uint4 *pk = reinterpret_cast<const uint4 *>(k + static_cast<int64_t>(t) * ldk + h * D + E * part);
            const uint4 *pv = reinterpret_cast<const uint4 *>(v + static_cast<int64_t>(t) * ldv + h * D + E * part);
#pragma unroll
            for (int e = 0; e < E / 8; ++e) raw[0][e] = __ldcs(pk + e);
#pragma unroll
            for (int e = 0; e < E / 8; ++e) raw[1][e] = __ldcs(pv + e);
            slot = slots[t];
        }
        const bool live = slot_ok(c, slot);
        const int64_t at = live ? row_at(c, slot, h) : 0;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float x[E], factor;
#pragma unroll
            for (int e = 0; e < E / 8; ++e) frag::unpack_bf16x8(raw[y][e], x + 8 * e);
            frag::rotate(x, c.group == 256);
            const uint16_t s = frag::block_scale(frag::absmax_bits(x, LANES), norm, factor);
            uint32_t packed[E / 8];
            prep::quantize_pack(x, factor, packed);
            if (live) {
                uint8_t *dst = (y ? c.vc : c.kc) + at * (D / 2) + E / 2 * part;
                if constexpr (E == 16) *reinterpret_cast<uint2 *>(dst) = make_uint2(packed[0], packed[1]);
                else *reinterpret_cast<uint4 *>(dst) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
                if (part == 0) (y ? c.vs : c.ks)[at] = s;
            }
        }
    }
}

template <int D, class I>
__global__ void __launch_bounds__(kRowThreads)
read_kernel(Cache c, const long long *__restrict__ slots, I total, uint16_t *__restrict__ k,
            uint16_t *__restrict__ v) {
    constexpr int LANES = D / 16;
    const float norm = frag::norm_of(c.group);
    const frag::CodeMasks masks;
    for (I i0 = static_cast<I>(blockIdx.x) * kRowThreads; i0 < total; i0 += gridDim.x * kRowThreads) {
        const I i = i0 + threadIdx.x, row = i / LANES, t = row / c.heads;
        const int part = static_cast<int>(i % LANES);
        const long long slot = i < total ? slots[t] : -1;
        uint2 w[2] = {};
        float s[2] = {0.0f, 0.0f};
        if (slot_ok(c, slot)) {
            const int64_t at = row_at(c, slot, static_cast<int>(row - t * c.heads));
            w[0] = *reinterpret_cast<const uint2 *>(c.kc + at * (D / 2) + 8 * part);
            w[1] = *reinterpret_cast<const uint2 *>(c.vc + at * (D / 2) + 8 * part);
            s[0] = frag::bf16_f32(c.ks[at]);
            s[1] = frag::bf16_f32(c.vs[at]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            // Sums of up to 256 codes are whole numbers below 2048, exact in
            // f16: two channels an operation and a shuffle.  h[4 u + e]: codes
            // e and e + 4 of word u.
            __half2 h[8];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                __half2 o[4];
                frag::widen_f16(masks, u ? w[y].y : w[y].x, o);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[4 * u + e] = o[e];
            }
            const __half2 minus2 = __float2half2_rn(-2.0f);
#pragma unroll
            for (int u = 0; u < 8; u += 4) {   // digit 0: codes 0-3, 4-7
                const __half2 sum = __hadd2(__hadd2(h[u], h[u + 1]), __hadd2(h[u + 2], h[u + 3]));
#pragma unroll
                for (int e = 0; e < 4; ++e) h[u + e] = __hfma2(minus2, h[u + e], sum);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {      // digit 1: both halves of both words
                const __half2 pair = __hadd2(h[e], h[4 + e]), sum = __hadd2(pair, __lowhigh2highlow(pair));
                h[e] = __hfma2(minus2, h[e], sum);
                h[4 + e] = __hfma2(minus2, h[4 + e], sum);
            }
            auto lane_digit = [&](int stride) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __half2 pair = __hadd2(h[e], __shfl_xor_sync(0xFFFFFFFFu, h[e], stride));
                    h[e] = __hfma2(minus2, h[e], __hadd2(pair, __shfl_xor_sync(0xFFFFFFFFu, pair, 2 * stride)));
                }
            };
            lane_digit(1);
            if (c.group == 256) lane_digit(4);
            // the product with the 8-bit significand of the scale is exact too:
            // one rounding, to bf16
            float x[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = __half22float2(h[e]);
                x[8 * (e >> 2) + (e & 3)] = f.x;
                x[8 * (e >> 2) + (e & 3) + 4] = f.y;
            }
            if (i < total) frag::store16((y ? v : k) + static_cast<int64_t>(row) * D + 16 * part, x, s[y] * norm);
        }
    }
}

// ------------------------------------------------------------------ attention
// Per request and shared head, the rows are the queries of the heads that
// share it times the new tokens, in blocks of ROWS; the keys go by in tiles of
// 64, one tile a warp at a time, with the running maximum and sum of a softmax
// in fp32:
//   S^T (keys x ROWS) = K (codes) Q^T           mma m16n8k32, int8, A = codes
//   P = exp2(S s_k - max)
//   O^T (D x ROWS) += V^T (codes) (P s_v)^T     mma m16n8k16, f16, A = codes
// Codes are the A operand of both products (16 rows an instruction against 8
// of the B side).  K's scale goes into the scores and V's into P, in fp32.
//
// Codes are converted as little as can be, for the integer pipe (half a warp
// instruction a cycle) has most of the loop's work:
// - K: int8, 16 times the code: two ANDs and a product for 8 codes.  The queries
//   are 16-bit whole numbers, the row's largest value at 32000 (off by 2^-16 of
//   it; f16 is off by 2^-11 of each value), as a high and a low byte that make
//   two columns; the sums are exact in int32.  Up to 4 rows fill the 8 columns
//   of one product with both bytes, and each lane then has two scores of a
//   block instead of four.
// - V: f16 subnormals offset by 8 (frag::codes_f16), five operations for 8
//   codes with up to 4 rows, else six; the offset's part of the outputs, -8
//   times the sum of the weights, comes out of one more product with a matrix
//   of ones and is taken off before each tile.
// The softmax's reference is not the running maximum but within 2^8 of it: it
// moves, and the outputs are rescaled, only when a score is more than 8 (log2)
// above it, so most tiles need no maximum over their lanes.  P s_v is f16
// relative to a reference of its own, in the same way: within 2^9 of the row's
// largest weight P s_v so far, of the keys that the row sees, so that neither a
// hidden value nor one without weight costs the others their bits.  2^-11
// relative for weights down to 2^-19 of the row's largest, and 2^-30 of it off
// below.  (One reference for all rows of a warp, of the scales alone, takes 1.8%
// fewer instructions and the same time, 58.0 against 57.8 us.)
//
// Which keys of a 16-key block sit in which row of the product is free as
// long as both products agree.  Row r holds key sigma(r), chosen so that both
// the 16-byte reads of K and the 4 D/64-byte reads of V spread over the banks.
//
// Copies.  Each warp has its own place for a tile's keys and one for its
// values (codes and scales, 64 (D + 4) bytes together), filled by its own
// 16-byte asynchronous copies: no warp waits for another inside a request.
// (Bulk copies take 25 instructions each, a lane at a time: 80 us against 68.)
// The 8 lanes that copy a block of 16 keys look its page up, so that pages of
// any size cost nearly the same (pages of 16: 58.9 us, of 64: 57.5; with a lane's
// copies spread over the blocks pages of 16 took 74.6 where this took 63.2).
// The next tile's keys are requested as soon as this one's scores are there, its
// values after the second product: with 16 warps an SM a warp has several times
// the copy's latency until it needs them, and registers, not bytes on the way,
// are what is short.
//
// Work.  Units of one tile for one (request, head, row block) are laid out in
// one line, with kTurn more behind each (request, head, row block) for the turn
// to the next: queries, joining the warps, and warps without a tile.  CTA c takes
// an even share of the line, so ragged lengths load the GPU evenly and long
// requests are split.  A CTA whose part ends inside a request writes (log2 of the
// softmax's sum, mean of the values) to the workspace and combine_kernel joins
// the parts in their order.
//
// Measured (CUDA graphs), 64 requests of 1500 to 8192 keys, 32 query heads on 8
// of 128: 57.5 us for 268 MB, 4.7 TB/s (41.1 us at the copy rate; the copies
// alone, without arithmetic, took 63.7 us when all of it took 65).  A steady loop of the same copies
// reads 6.1 TB/s; what is missing is the start (6.4 us to the first keys: launch,
// prefix of the lengths, table, latency), uneven ends (CTAs end 7 us after the
// mean) and the joining kernel (4 us).  2 requests of up to 131072 keys, 64 heads
// on 8: 57.6 us, 4.2 TB/s.  16 requests of up to 3001 keys, 5 queries, 16 heads
// on 4 of 256: 24.8 us, latency of few tiles a warp.
//
// Choices, each with both sides measured on the first case, us:
// - rows of a block (block_rows): 57.4 with 4, 63.0 with 8, 92.6 with 16; 8 heads
//   on a shared one (8 rows): 99 with 4, 63.0 with 8; 4 queries of 4 heads: 158
//   with 4, 97.6 with 8, 93.1 with 16.
// - kTurn: 60.3 with 0, 58.3 with 4, 57.4 with 8, 58.1 with 12; the 16 requests
//   32.3, 26.3, 24.8, 26.2.
// - outputs_beside: outputs beside the tiles 57.4, in their place 58.0.
// - four CTAs an SM (128 registers) 57.4, five or six (spills) 65 and 70.
// - four warps a CTA 57.4, two (and twice the CTAs) 59.1, eight 74.
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kMaxCtas = 592;

constexpr int kTile = 64;               // keys
constexpr int kMinUnits = kAttnWarps;   // at least one tile a warp
constexpr int kTurn = 8;                // units that a turn from one request to the next counts
// log2: what a score may be above its reference, where a row's reference weight
// lies in f16 and what a weight may be above it (2^15.1 at most), and the least
// reference, so that a weight of 1 in its unit is a float
constexpr float kRoom = 8.0f;
constexpr float kUnit = 6.0f, kHead = 9.0f;
constexpr float kLeast = -110.0f;
constexpr uint32_t kOnes = 0x3C003C00u;   // two f16

struct AttnArgs {
    Cache c;
    const uint16_t *q;
    int64_t ldq;
    int64_t T;
    int G;                   // query heads that share a head
    const int *table;
    int64_t max_pages;
    const int *seq_lens, *cu_q;
    int B;
    float scale;             // softmax scale * log2(e)
    int4 *desc;              // per CTA: {last CTA of the request it starts and does not end, b, h, row block}
    float *parts;            // per CTA two parts: ROWS (log2 of the softmax's sum, -), then ROWS x D
    uint16_t *out;
};

__device__ __forceinline__ int sigma(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1; }

struct Request {
    int len, q0, nq, tiles, blocks;
    __device__ __forceinline__ long long span() const { return static_cast<long long>(tiles) + kTurn; }
};

// Request b's sizes, clamped to what its buffers hold.
template <int ROWS>
__device__ __forceinline__ Request request_of(const AttnArgs &a, int b) {
    Request r;
    int64_t len = a.seq_lens[b];
    const int64_t most = a.max_pages << a.c.page_shift;
    len = len < 0 ? 0 : len > most ? most : len;
    int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
    q0 = q0 < 0 ? 0 : q0;
    q1 = q1 > a.T ? a.T : q1;
    r.len = static_cast<int>(len);
    r.q0 = static_cast<int>(q0);
    r.nq = q1 > q0 ? static_cast<int>(q1 - q0) : 0;
    r.tiles = len > 0 ? (r.len - 1) / kTile + 1 : 1;
    r.blocks = static_cast<int>((static_cast<int64_t>(r.nq) * a.G + ROWS - 1) / ROWS);
    return r;
}

// 2^x (one instruction; results below the normal range are 0).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// log2 of a bf16 scale: the exponent and the fraction behind it, at most 0.09
// below; -127 for 0, 128 and more for an infinity or a NaN.  (2^23 + bits, less
// 2^23 and the exponent's bias, in units of the fraction's 2^-7.)
__device__ __forceinline__ float level_of(uint32_t bits) {
    return fmaf(__uint_as_float((bits & 0x7FFFu) | 0x4B000000u), 1.0f / 128.0f, -65536.0f - 127.0f);
}

// log2 of the sum of a row's softmax weights; 0 for a row that has none.
// Outputs of several warps or CTAs are joined as means by their shares of the
// sum: a sum of the largest values over many keys would leave fp32.  (The sum's
// rounding as a logarithm, 2^-24 of it, is below that of the scores' own fp32
// products.  With reference and sum apart, and a division a step: 58.3 us
// against 57.5.)
__device__ __forceinline__ float log_of(float sum) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sum));
    return sum > 0.0f || sum != sum ? r : 0.0f;
}

// Output row r of a row block -> rotate back 16 channels a thread and store.
__device__ __forceinline__ void store_row(const AttnArgs &a, const Request &rq, int h, int row,
                                          int part, float (&x)[16]) {
    frag::rotate(x, a.c.group == 256);
    const int i = row / a.G;
    if (i < rq.nq) {
        const int heads = a.G * a.c.heads;
        frag::store16(a.out + ((static_cast<int64_t>(rq.q0) + i) * heads + h * a.G + row % a.G) * a.c.D + 16 * part, x, frag::norm_of(a.c.group));
    }
}

template <int D, int ROWS>
__host__ __device__ constexpr bool outputs_beside() {
    return kAttnWarps * (kTile * (D + 4) + ROWS * (D + 4) * 4) <= 110 * 1024;
}

// One request's part of a CTA's work: a head, a row block and tiles.
struct Segment {
    int b, h, rb, tile0, tile1;
    long long u0, u1;           // its first unit and the one behind its last, of all CTAs
    Request rq;
};

template <int D, int ROWS>
__global__ void __launch_bounds__(kAttnThreads, D > 128 || ROWS > 8 ? 2 : ROWS == 8 ? 3 : 4) attention_kernel(AttnArgs a) {
    constexpr bool HALF = ROWS == 4;    // the columns hold the two bytes of four queries
    constexpr int NT = HALF ? 1 : ROWS / 8;
    constexpr int NS = HALF ? 2 : 4;    // scores a thread, 16-key block and column tile
    constexpr int NW = D / 32;          // K words (8 codes) a thread and key
    constexpr int VW = D / 64;          // V words a thread and key
    constexpr int MT = HALF ? D / 32 : D / 16;   // accumulators of O^T, four values each
    constexpr int LANES = D / 16;
    constexpr int PITCH = D + 4;
    constexpr int TILE = kTile, NB = TILE / 16;
    constexpr int STAGE = TILE * (D + 4);   // codes of keys, of values, scales of keys, of values
    // (the tiles begin on a 32-byte sector: 57.8 us, 16 bytes off 60.0)
    extern __shared__ __align__(128) uint4 smem[];
    // queries as B fragments, {odd, even} channels of a word: HALF: [NW][32
    // lanes], else [NT][NW][high, low byte][32 lanes]
    uint2 *qf = reinterpret_cast<uint2 *>(smem);
    uint8_t *stages = reinterpret_cast<uint8_t *>(qf + (HALF ? 1 : 2 * NT) * NW * 32);
    // outputs of the warps [warps][ROWS][PITCH]: beside the stages, so that the
    // next request's first tiles come in while this one's outputs are joined,
    // or in their place where that leaves two CTAs to an SM
    constexpr bool BESIDE = outputs_beside<D, ROWS>();
    float *osum = reinterpret_cast<float *>(stages + (BESIDE ? kAttnWarps * STAGE : 0));
    __shared__ float qs[ROWS];
    __shared__ int qmax[ROWS];
    __shared__ float wm[kAttnWarps][ROWS], wl[kAttnWarps][ROWS], wunit[kAttnWarps][ROWS];
    __shared__ long long scan[kAttnWarps];
    __shared__ long long start_unit;
    __shared__ int start_b;

    // whether value x of accumulator i belongs to the second nibble of a byte
    auto second_nibble = [](int i, int x) { return HALF && VW == 1 ? (x >> 1) != 0 : (i & 1) != 0; };

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    ptx::launch_dependents();           // the combining CTAs take the places of those that are done
    ptx::grid_dependency_wait();
    // ---- this CTA's part of the line of units
    const int chunk = (a.B + kAttnThreads - 1) / kAttnThreads;
    const int b_lo = min(a.B, tid * chunk), b_hi = min(a.B, b_lo + chunk);
    long long mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const Request r = request_of<ROWS>(a, b);
        mine += r.span() * r.blocks * a.c.heads;
    }
    long long incl = mine;
    for (int s = 1; s < 32; s <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, s);
        if (lane >= s) incl += u;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    // CTA c of the first `ctas` takes units [c total / ctas, (c + 1) total / ctas)
    const long long ctas = min(static_cast<long long>(gridDim.x), (total + kMinUnits - 1) / kMinUnits);
    auto first_of = [&](long long c) {
        const long long n = c * total;
        return n < (1ll << 32) ? static_cast<long long>(static_cast<unsigned>(n) / static_cast<unsigned>(ctas)) : n / ctas;
    };
    if (tid == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (blockIdx.x >= ctas) return;
    const long long u0 = first_of(blockIdx.x), u1 = first_of(blockIdx.x + 1);
    if (mine > 0 && before <= u0 && u0 < before + mine) {
        long long at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            const Request r = request_of<ROWS>(a, b);
            const long long n = r.span() * r.blocks * a.c.heads;
            if (u0 < at + n) {
                start_b = b;
                start_unit = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int b = start_b;
    long long base = start_unit;        // first unit of request b
    const uint8_t *st = stages + warp * STAGE;
    const uint32_t st_s = ptx::smem_u32(st);
    const uint16_t *sks = reinterpret_cast<const uint16_t *>(st + TILE * D), *svs = sks + TILE;
    const int page_mask = (1 << a.c.page_shift) - 1, num_pages = static_cast<int>(a.c.num_pages);
    const frag::CodeMasks masks;
    // this thread's row in a 16-key block, of its first scores
    const int key0 = sigma(g) + (HALF && t4 >= 2 ? 8 : 0);
    const int col0 = HALF ? 2 * (t4 & 1) : 2 * t4;   // and its first query of a column tile
    const bool first = t4 < 2;
    const int weight_mine = first ? 256 : 1, weight_theirs = first ? 1 : 256;
    // HALF: the transposed weights of two keys -> (low, 0) and (high, 0) for
    // columns 0-3, (0, low) and (0, high) for columns 4-7
    const uint32_t pick_low = g < 4 ? 0x4410u : 0x1044u, pick_high = g < 4 ? 0x4432u : 0x3244u;

    auto locate = [&](long long u) {
        Segment sg;
        sg.rq = request_of<ROWS>(a, b);
        long long n = sg.rq.span() * sg.rq.blocks * a.c.heads;
        while (u >= base + n && b + 1 < a.B) {
            base += n;
            sg.rq = request_of<ROWS>(a, ++b);
            n = sg.rq.span() * sg.rq.blocks * a.c.heads;
        }
        const long long at = min(u - base, n - 1);   // (n is 0 only if lengths change under the kernel)
        const int seg = n < 1 ? 0 : at < (1ll << 31) ? static_cast<int>(static_cast<unsigned>(at) / static_cast<unsigned>(sg.rq.span()))
                                                     : static_cast<int>(at / sg.rq.span());
        sg.b = b;
        sg.u0 = base + seg * sg.rq.span();
        sg.u1 = sg.u0 + sg.rq.tiles;
        sg.tile0 = static_cast<int>(min(max(u - sg.u0, 0ll), static_cast<long long>(sg.rq.tiles)));
        sg.tile1 = static_cast<int>(min(u1, sg.u1) - sg.u0);
        const int blocks = max(sg.rq.blocks, 1);
        sg.h = seg / blocks;
        sg.rb = seg % blocks;
        return sg;
    };
    // Request a tile's keys; its values are requested once the last tile's have
    // been read.  A page holds at least 16 keys, so a 16-key block lies in one:
    // the 8 lanes of a block copy its codes, 128 bytes an instruction, and two
    // of them its scales, all from the one page that the lane has looked up.
    const int block = lane >> 3;
    int id = -1;                        // the page of this lane's block, -1: none
    int in_page = 0;                    // the block's first key in it
    auto copy = [&](int h, const uint8_t *codes, const uint16_t *scales, int i) {   // keys (0) or values (1)
        const int64_t row = ((static_cast<int64_t>(id) * a.c.heads + h) << a.c.page_shift) + in_page;
        const bool there = id >= 0;
        // (copies of no bytes name the cache's first block)
        const uint8_t *src = codes + (there ? row * (D / 2) : 0) + 16 * (lane & 7);
        const uint16_t *ssrc = scales + (there ? row : 0) + 8 * (lane & 7);
        const uint32_t dst = st_s + i * (TILE * D / 2) + block * (16 * D / 2) + 16 * (lane & 7);
#pragma unroll
        for (int y = 0; y < D / 16; ++y) frag::cp_async16_or_zero(dst + 128 * y, src + 128 * y, there);
        if ((lane & 7) < 2)
            frag::cp_async16_or_zero(st_s + TILE * D + i * (TILE * 2) + 32 * block + 16 * (lane & 7), ssrc, there);
        prep::cp_async_commit();
    };
    // Table entries are read a tile ahead of their use (-1 behind the
    // request's end), and checked when they are used.
    int ahead = -1;
    auto look_ahead = [&](const Segment &sg, int tile) {
        const int64_t j0 = static_cast<int64_t>(tile) * TILE + 16 * block;
        ahead = j0 < sg.rq.len ? a.table[sg.b * a.max_pages + (j0 >> a.c.page_shift)] : -1;
    };
    auto request = [&](const Segment &sg, int tile) {
        in_page = (tile * TILE + 16 * block) & page_mask;
        id = ahead;
        if (id < 0 || id >= num_pages) {
            id = -1;
            if (tile * TILE + 16 * block < sg.rq.len && (lane & 7) == 0) page_error();
        }
        copy(sg.h, a.c.kc, a.c.ks, 0);
        look_ahead(sg, tile + kAttnWarps);
    };
    // The first of a segment's tiles, and this thread's queries of it.
    uint4 raw[2];
    auto query_at = [&](const Segment &sg, int i) -> const uint16_t * {
        const int row = sg.rb * ROWS + i / LANES, qi = row / a.G;
        if (i >= ROWS * LANES || qi >= sg.rq.nq) return nullptr;
        return a.q + (static_cast<int64_t>(sg.rq.q0) + qi) * a.ldq + static_cast<int64_t>(sg.h * a.G + row % a.G) * D + 16 * (i % LANES);
    };
    auto load_query = [&](const Segment &sg, int i) {
        const uint4 *p = reinterpret_cast<const uint4 *>(query_at(sg, i));
        raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
        if (p) {
            raw[0] = p[0];
            raw[1] = p[1];
        }
    };
    auto start = [&](const Segment &sg) {
        load_query(sg, tid);
        if (sg.tile0 + warp < sg.tile1) {
            look_ahead(sg, sg.tile0 + warp);
            request(sg, sg.tile0 + warp);
            copy(sg.h, a.c.vc, a.c.vs, 1);
        }
    };

    Segment next = locate(u0);
    if (next.tile0 == next.rq.tiles) {  // begins in a turn
        const long long u = next.u0 + next.rq.span();
        if (u >= u1) return;
        next = locate(u);
    }
    start(next);
    for (bool last = false; !last;) {
        const Segment sg = next;
        const Request &rq = sg.rq;
        const int tile0 = sg.tile0, tile1 = sg.tile1, h = sg.h, row0 = sg.rb * ROWS;
        // ---- queries: rotate, round to 16 bits, lay out as B fragments
        for (int i0 = 0; i0 < ROWS * LANES; i0 += kAttnThreads) {
            const int i = i0 + tid;
            const int r = i / LANES, part = i % LANES;
            const int qi = (row0 + r) / a.G;
            if (i0) load_query(sg, i);
            float x[16];
            frag::unpack_bf16x8(raw[0], x);
            frag::unpack_bf16x8(raw[1], x + 8);
            frag::rotate(x, a.c.group == 256);
            const uint32_t amax = frag::absmax_bits(x, LANES);
            // 16-bit whole numbers, the row's largest at 32000; rows below
            // 2^-100 count as 0, rows with a NaN or an infinity give NaN
            const float top = __uint_as_float(amax);
            const bool zero = amax < (27u << 23);
            const float f = zero ? 0.0f : 32000.0f / top;
            if (r < ROWS) {
                if (part == 0) {
                    qs[r] = zero ? 0.0f : a.scale * frag::norm_of(a.c.group) * (top / 32000.0f) / 16.0f;
                    if (amax >= 0x7F800000u) qs[r] = __uint_as_float(0x7FC00000u);
                    qmax[r] = rq.len - rq.nq + min(qi, rq.nq - 1);   // rows past the last query are not stored
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int d = 16 * part + 8 * half;
                    const int tq = D == 64 ? d / 16 : (d % 128) / 32;
                    const int j = D == 64 ? (d % 16) / 8 : 4 * (d / 128) + (d % 32) / 8;
                    // high and low byte (signed) of each, channels 0-7
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int n = __float2int_rn(x[8 * half + e] * f);
                        hi[e] = static_cast<uint32_t>(n + 128) >> 8;
                        lo[e] = static_cast<uint32_t>(n);
                    }
                    auto bytes = [](uint32_t p, uint32_t q, uint32_t u, uint32_t v) {
                        return __byte_perm(__byte_perm(p, q, 0x0040), __byte_perm(u, v, 0x0040), 0x5410);
                    };
                    const uint2 high = make_uint2(bytes(hi[1], hi[3], hi[5], hi[7]), bytes(hi[0], hi[2], hi[4], hi[6]));
                    const uint2 low = make_uint2(bytes(lo[1], lo[3], lo[5], lo[7]), bytes(lo[0], lo[2], lo[4], lo[6]));
                    if constexpr (HALF) {
                        qf[j * 32 + r * 4 + tq] = high;
                        qf[j * 32 + (r + 4) * 4 + tq] = low;
                    } else {
                        qf[(((r >> 3) * NW + j) * 2) * 32 + (r & 7) * 4 + tq] = high;
                        qf[(((r >> 3) * NW + j) * 2 + 1) * 32 + (r & 7) * 4 + tq] = low;
                    }
                }
            }
        }
        __syncthreads();

        // thread's columns of a tile: queries col0 and col0 + 1
        float cs[NT][2];
        int cmax[NT][2];
        int least = 0x7FFFFFFF;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                cs[nt][x] = qs[8 * nt + col0 + x];
                cmax[nt][x] = qmax[8 * nt + col0 + x];
                least = min(least, cmax[nt][x]);
            }
        for (int s = 1; s < 4; s <<= 1) least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, s));
        // the fragments stay in registers where there is room
        uint2 qreg[HALF ? NW : 1];
        if constexpr (HALF)
#pragma unroll
            for (int j = 0; j < NW; ++j) qreg[j] = qf[j * 32 + lane];

        float o[MT][NT][4] = {};
        // reference of the softmax and how far above it (log2) a score may be
        // before the reference moves: not at all until there is one.  limit:
        // how far a weight P s_v may be, kHead above its reference; unit: what
        // weights are taken times, 2^kUnit over their reference
        float m[NT][2], room[NT][2], l[NT][2], limit[NT][2], unit[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                m[nt][x] = 0.0f;
                room[nt][x] = -INFINITY;
                l[nt][x] = 0.0f;
                limit[nt][x] = kUnit + kHead;
                unit[nt][x] = 1.0f;
            }

        for (int tile = tile0 + warp; tile < tile1; tile += kAttnWarps) {
            const int k0 = tile * TILE;
            // 16-key blocks that are there; whether every query sees every key
            const bool mine_here = id >= 0;
            const uint32_t here = __ballot_sync(0xFFFFFFFFu, mine_here);   // bit 8 blk: block blk's
            const bool all = here == 0xFFFFFFFFu && k0 + TILE - 1 <= least;
            frag::cp_async_wait<1>();   // the keys are there, the values may be on their way
            __syncwarp();
            float s[NB][NT][NS];
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                const uint8_t *pa = st + (16 * blk + sigma(g)) * (D / 2), *pb = pa + 8 * (D / 2);
                uint32_t ka[NW], kb[NW];
                if constexpr (D == 64) {
                    *reinterpret_cast<uint2 *>(ka) = *reinterpret_cast<const uint2 *>(pa + 8 * t4);
                    *reinterpret_cast<uint2 *>(kb) = *reinterpret_cast<const uint2 *>(pb + 8 * t4);
                } else {
#pragma unroll
                    for (int i = 0; i < NW / 4; ++i) {
                        reinterpret_cast<uint4 *>(ka)[i] = *reinterpret_cast<const uint4 *>(pa + 64 * i + 16 * t4);
                        reinterpret_cast<uint4 *>(kb)[i] = *reinterpret_cast<const uint4 *>(pb + 64 * i + 16 * t4);
                    }
                }
                int high[NT][4], low[HALF ? 1 : NT][4];
#pragma unroll
                for (int j = 0; j < NW; j += 2) {
                    uint32_t ao[2], ae[2], bo[2], be[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        frag::codes_s8(masks, ka[j + y], ao[y], ae[y]);
                        frag::codes_s8(masks, kb[j + y], bo[y], be[y]);
                    }
                    if constexpr (HALF) {
                        if (j == 0) frag::mma_s8_first(high[0], ao[0], bo[0], ao[1], bo[1], qreg[j].x, qreg[j + 1].x);
                        else frag::mma_s8(high[0], ao[0], bo[0], ao[1], bo[1], qreg[j].x, qreg[j + 1].x);
                        frag::mma_s8(high[0], ae[0], be[0], ae[1], be[1], qreg[j].y, qreg[j + 1].y);
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 *q = qf + (nt * NW + j) * 64 + lane;
                            const uint2 h0 = q[0], l0 = q[32], h1 = q[64], l1 = q[96];
                            if (j == 0) {
                                frag::mma_s8_first(high[nt], ao[0], bo[0], ao[1], bo[1], h0.x, h1.x);
                                frag::mma_s8_first(low[nt], ao[0], bo[0], ao[1], bo[1], l0.x, l1.x);
                            } else {
                                frag::mma_s8(high[nt], ao[0], bo[0], ao[1], bo[1], h0.x, h1.x);
                                frag::mma_s8(low[nt], ao[0], bo[0], ao[1], bo[1], l0.x, l1.x);
                            }
                            frag::mma_s8(high[nt], ae[0], be[0], ae[1], be[1], h0.y, h1.y);
                            frag::mma_s8(low[nt], ae[0], be[0], ae[1], be[1], l0.y, l1.y);
                        }
                    }
                }
                // 256 high + low, exact in 32 bits; scores in units of log2,
                // less the reference
                const float ska = frag::bf16_f32(sks[16 * blk + key0]);
                if constexpr (HALF) {
                    // columns 0-3 have the high bytes' sums and columns 4-7 the
                    // low ones': lanes of columns 0-3 take rows 0-7, the others
                    // rows 8-15
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int mine = first ? high[0][x] : high[0][2 + x];
                        const int theirs = __shfl_xor_sync(0xFFFFFFFFu, first ? high[0][2 + x] : high[0][x], 2);
                        const int sum = mine * weight_mine + theirs * weight_theirs;
                        s[blk][0][x] = fmaf(static_cast<float>(sum), ska * cs[0][x], -m[0][x]);
                    }
                } else {
                    const float skb = frag::bf16_f32(sks[16 * blk + key0 + 8]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            s[blk][nt][x] = fmaf(static_cast<float>(256 * high[nt][x] + low[nt][x]),
                                                 (x < 2 ? ska : skb) * cs[nt][x & 1], -m[nt][x & 1]);
                }
            }
            __syncwarp();               // the keys have been read
            const bool more = tile + kAttnWarps < tile1;
            if (more) request(sg, tile + kAttnWarps);
            else prep::cp_async_commit();   // an empty group: the counts stay
            if (!all) {
                asm volatile("");       // a branch: few tiles take it
                // hidden keys are -inf whatever they hold
#pragma unroll
                for (int blk = 0; blk < NB; ++blk) {
                    const int ja = k0 + 16 * blk + key0;
                    const bool there = (here >> (8 * blk)) & 1;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < NS; ++x)
                            if (!there || ja + 4 * (x & 2) > cmax[nt][x & 1]) s[blk][nt][x] = -INFINITY;
                }
            }
            frag::cp_async_wait<1>();   // the values are there, the next keys may be on their way
            __syncwarp();
            // ---- does a score or a weight leave its reference's room?  Hidden
            // keys' are -inf.  For the weights a lane takes its largest score with
            // its largest scale first, which is no less than its largest weight
            // (without signs: hidden keys' scales are whatever memory held).
            uint32_t scale_bits[NB][NS / 2], wide = 0;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                for (int y = 0; y < NS / 2; ++y) {
                    scale_bits[blk][y] = svs[16 * blk + key0 + 8 * y];
                    wide = max(wide, scale_bits[blk][y] & 0x7FFFu);
                }
            const float widest = level_of(wide);
            // the largest of f(a score, its key's scale) of this lane's keys in a column
            auto largest_of = [&](int nt, int x, auto f) {
                float top = f(s[0][nt][x], scale_bits[0][0]);
#pragma unroll
                for (int i = 1; i < NB * (NS / 2); i += 2) {
                    const int blk = i / (NS / 2), y = i % (NS / 2), blk2 = (i + 1) / (NS / 2) % NB, y2 = (i + 1) % (NS / 2);
                    const float one = f(s[blk][nt][2 * y + x], scale_bits[blk][y]);
                    top = i + 1 < NB * (NS / 2) ? prep::max3(top, one, f(s[blk2][nt][2 * y2 + x], scale_bits[blk2][y2])) : fmaxf(top, one);
                }
                return top;
            };
            auto score = [](float v, uint32_t) { return v; };
            auto weight = [](float v, uint32_t bits) { return v + level_of(bits); };
            bool turn = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float top = largest_of(nt, x, score);
                    turn |= top > room[nt][x] || top + widest > limit[nt][x];
                }
            if (__any_sync(0xFFFFFFFFu, turn)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float mul[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float top = largest_of(nt, x, score), heavy = largest_of(nt, x, weight);
                        for (int k = HALF ? 2 : 4; k < 32; k <<= 1) {
                            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
                            heavy = fmaxf(heavy, __shfl_xor_sync(0xFFFFFFFFu, heavy, k));
                        }
                        mul[x] = 1.0f;
                        if (top > room[nt][x] || heavy > limit[nt][x]) {
                            // of nothing, at first (the room is the column's; l is of
                            // this lane's keys only, and 0 where all of those underflow)
                            const bool none = room[nt][x] == -INFINITY;
                            const float up = none ? top : fmaxf(top, 0.0f), before = limit[nt][x] - kHead - up;
                            const float largest = fmaxf(none ? kLeast : fmaxf(before, kLeast), heavy - up);
                            m[nt][x] += up;
                            room[nt][x] = kRoom;
                            l[nt][x] *= none ? 0.0f : ex2(-up);
                            mul[x] = none ? 0.0f : ex2(before - largest);
                            limit[nt][x] = largest + kHead;
                            unit[nt][x] = ex2(kUnit - largest);
#pragma unroll
                            for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                                for (int y = 0; y < NS; y += 2) s[blk][nt][y + x] -= up;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[i][nt][x] *= mul[x & 1];
                }
            }
#pragma unroll
            for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < NS; ++x) {
                        s[blk][nt][x] = ex2(s[blk][nt][x]);
                        l[nt][x & 1] += s[blk][nt][x];
                    }
            // ---- weights of the values, as f16 fragments, and their sums
            // HALF: p[blk][0][..] are the keys of rows 0-7 (two of them) and rows 8-15
            uint32_t p[NB][NT][HALF ? 4 : 2];
            float psum[NT][4];
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                const float sva = frag::bf16_f32(scale_bits[blk][0]), svb = HALF ? 0.0f : frag::bf16_f32(scale_bits[blk][NS / 2 - 1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[NS];
#pragma unroll
                    for (int x = 0; x < NS; ++x) w[x] = s[blk][nt][x] * unit[nt][x & 1] * (x < 2 ? sva : svb);
                    if (!all) {
                        asm volatile("");
                        // a hidden key's scale may be anything
                        const int ja = k0 + 16 * blk + key0;
                        const bool there = (here >> (8 * blk)) & 1;
#pragma unroll
                        for (int x = 0; x < NS; ++x)
                            if (!there || ja + 4 * (x & 2) > cmax[nt][x & 1]) w[x] = 0.0f;
                    }
                    const uint32_t mine = frag::transpose8x8(frag::pack_f16(w[0], w[1]));
                    if constexpr (HALF) {
                        // lanes of columns 0-3 hold rows 0-7 of a query, those
                        // of columns 4-7 rows 8-15
                        const uint32_t theirs = __shfl_xor_sync(0xFFFFFFFFu, mine, 16);
                        const uint32_t upper = g < 4 ? mine : theirs, lower = g < 4 ? theirs : mine;
                        p[blk][nt][0] = __byte_perm(upper, 0, pick_low);
                        p[blk][nt][1] = __byte_perm(upper, 0, pick_high);
                        p[blk][nt][2] = __byte_perm(lower, 0, pick_low);
                        p[blk][nt][3] = __byte_perm(lower, 0, pick_high);
                    } else {
                        p[blk][nt][0] = mine;
                        p[blk][nt][1] = frag::transpose8x8(frag::pack_f16(w[2], w[3]));
                    }
#pragma unroll
                    for (int y = 0; y < (HALF ? 4 : 2); y += 2)
                        if (blk == 0 && y == 0) frag::mma_f16_first(psum[nt], kOnes, kOnes, kOnes, kOnes, p[blk][nt][y], p[blk][nt][y + 1]);
                        else frag::mma_f16(psum[nt], kOnes, kOnes, kOnes, kOnes, p[blk][nt][y], p[blk][nt][y + 1]);
                }
            }
            // the codes' offset of 8, taken off tile by tile so that it never
            // grows far beyond the sums it is part of
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float one[2] = {-8.0f * frag::kCodeUnit * psum[nt][0], -8.0f * frag::kCodeUnit * psum[nt][1]};
                const float second[2] = {16.0f * one[0], 16.0f * one[1]};
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[i][nt][x] += second_nibble(i, x) ? second[x & 1] : one[x & 1];
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                // columns 2 t4, 2 t4 + 1 of the product are the keys sigma of those
                uint32_t v[4][VW];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = 16 * blk + sigma(2 * t4 + (i & 1)) + 8 * (i >> 1);
                    const uint8_t *p = st + TILE * (D / 2) + key * (D / 2) + 4 * VW * g;
                    if constexpr (VW == 1) v[i][0] = *reinterpret_cast<const uint32_t *>(p);
                    else if constexpr (VW == 2) *reinterpret_cast<uint2 *>(v[i]) = *reinterpret_cast<const uint2 *>(p);
                    else *reinterpret_cast<uint4 *>(v[i]) = *reinterpret_cast<const uint4 *>(p);
                }
                if constexpr (HALF) {
                    // A register has codes i and i + 4 of one key's word: two
                    // rows of O^T that the columns tell apart, so that no
                    // keys have to be put side by side.  Rows r and r + 8 of a
                    // product are neighbouring words (with D = 64, which has
                    // one word a lane, its even and odd pairs).
#pragma unroll
                    for (int y = 0; y < 4; y += 2)
#pragma unroll
                        for (int w = 0; w < VW; w += 2) {
                            uint32_t a0[4], a1[4], a2[4], a3[4];
                            frag::codes_f16(masks, v[y][w], a0);
                            frag::codes_f16(masks, v[y + 1][w], a2);
                            if constexpr (VW > 1) {
                                frag::codes_f16(masks, v[y][w + 1], a1);
                                frag::codes_f16(masks, v[y + 1][w + 1], a3);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (VW > 1)
                                    frag::mma_f16(o[2 * w + i][0], a0[i], a1[i], a2[i], a3[i], p[blk][0][y], p[blk][0][y + 1]);
                                else if (i < 2)
                                    frag::mma_f16(o[i][0], a0[2 * i], a0[2 * i + 1], a2[2 * i], a2[2 * i + 1], p[blk][0][y], p[blk][0][y + 1]);
                            }
                        }
                } else {
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        // halves of two keys side by side: codes 0-3, then 4-7
                        uint32_t lo0[4], lo1[4], hi0[4], hi1[4];
                        frag::codes_f16(masks, __byte_perm(v[0][w], v[1][w], 0x5410), lo0);
                        frag::codes_f16(masks, __byte_perm(v[0][w], v[1][w], 0x7632), hi0);
                        frag::codes_f16(masks, __byte_perm(v[2][w], v[3][w], 0x5410), lo1);
                        frag::codes_f16(masks, __byte_perm(v[2][w], v[3][w], 0x7632), hi1);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                frag::mma_f16(o[4 * w + i][nt], lo0[i], hi0[i], lo1[i], hi1[i], p[blk][nt][0], p[blk][nt][1]);
                    }
                }
            }
            __syncwarp();               // the values have been read
            if (more) copy(h, a.c.vc, a.c.vs, 1);
            else prep::cp_async_commit();
        }
        frag::cp_async_wait<0>();
        const long long end = sg.u0 + rq.span();
        last = end >= u1;

        // ---- join the warps
        if constexpr (!BESIDE) __syncthreads();   // every tile is done
        if (!last) {
            next = locate(end);
            if constexpr (BESIDE) start(next);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                for (int k = HALF ? 2 : 4; k < 32; k <<= 1) l[nt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][x], k);
                if (g == 0) {
                    wm[warp][8 * nt + col0 + x] = room[nt][x] == -INFINITY ? -INFINITY : m[nt][x];
                    wl[warp][8 * nt + col0 + x] = l[nt][x];
                    wunit[warp][8 * nt + col0 + x] = limit[nt][x] - kHead - kUnit;
                }
            }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int d = (D / 8) * g + (HALF ? (first ? 0 : 4) + (VW > 1 ? 8 * (2 * (i >> 2) + (x >> 1)) + (i & 3) : 2 * i + (x >> 1))
                                                      : 8 * (i >> 2) + (i & 3) + 4 * (x >> 1));
                    osum[(warp * ROWS + 8 * nt + col0 + (x & 1)) * PITCH + d] =
                        o[i][nt][x] * (second_nibble(i, x) ? 1.0f / (16.0f * frag::kCodeUnit) : 1.0f / frag::kCodeUnit);
                }
        __syncthreads();
        const bool whole = sg.u0 >= u0 && sg.u1 <= u1;
        float *part_out = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (sg.u0 >= u0 ? 1 : 0)) * (ROWS * (D + 2));
        for (int i0 = 0; i0 < ROWS * LANES; i0 += kAttnThreads) {
            const int i = i0 + tid;
            const int r = min(i / LANES, ROWS - 1), part = i % LANES;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, wm[w][r]);
            const float safe = top == -INFINITY ? 0.0f : top;
            float x[16] = {}, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) sum += ex2(wm[w][r] - safe) * wl[w][r];
            const float log = log_of(sum);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = ex2(wm[w][r] - safe + (wunit[w][r] - log));
                const float4 *src = reinterpret_cast<const float4 *>(osum + (w * ROWS + r) * PITCH + 16 * part);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 y = src[e];
                    x[4 * e] += f * y.x;
                    x[4 * e + 1] += f * y.y;
                    x[4 * e + 2] += f * y.z;
                    x[4 * e + 3] += f * y.w;
                }
            }
            if (whole) {
                store_row(a, rq, h, i < ROWS * LANES ? row0 + r : 0x7FFFFFFF, part, x);
            } else if (i < ROWS * LANES) {
                if (part == 0) part_out[2 * r] = top + log;
                float4 *dst = reinterpret_cast<float4 *>(part_out + 2 * ROWS + r * D + 16 * part);
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
        }
        if (!whole && sg.u0 >= u0 && tid == 0)
            a.desc[blockIdx.x] = make_int4(static_cast<int>((sg.u1 * ctas - 1) / total), sg.b, h, sg.rb);   // the owner of its last unit
        if constexpr (!BESIDE) {
            __syncthreads();            // the outputs have been read
            if (!last) start(next);
        }
    }
}

// CTA c joins the parts of the request that CTA c of attention_kernel began
// and did not end: 16 channels of a row a thread, the parts dealt out to the
// groups of ROWS D / 16 threads that the CTA has, which are joined at the end.
// Bound by latency (about 4 us behind the attention; a launch of its own costs
// less than a count of arrivals and the last CTA joining: 69 and 74 us for the
// two long cases).  256 threads with 64 registers fit into the place of one
// attention CTA that has ended: two parts on the way a thread give 57.4 us, four
// 58.2, 512 threads 59.7.
constexpr int kCombineThreads = 256;

template <int D, int ROWS>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(AttnArgs a) {
    constexpr int LANES = D / 16, USED = ROWS * LANES, WIDTH = USED < 32 ? 32 : USED, GROUPS = kCombineThreads / WIDTH;
    static_assert(WIDTH % 32 == 0 && WIDTH <= kCombineThreads / 2, "whole warps a group");
    __shared__ float4 sums[GROUPS - 1][4][WIDTH];
    __shared__ float2 tops[GROUPS][WIDTH];
    ptx::grid_dependency_wait();
    const int4 d = a.desc[blockIdx.x];
    if (d.x < 0) return;
    const int i = threadIdx.x % WIDTH, group = threadIdx.x / WIDTH, r = min(i / LANES, ROWS - 1), part = i % LANES;
    const int c0 = blockIdx.x, count = d.x - c0 + 1;
    auto at = [&](int k) {   // the k-th part: the first is its CTA's second
        return a.parts + (2 * static_cast<int64_t>(c0 + k) + (k == 0 ? 1 : 0)) * (ROWS * (D + 2));
    };
    // the mean of the group's parts, kBatch on the way at a time, relative to
    // the largest of the references so far
    // (kShare: all parts of a grid together stay below the largest of their means)
    constexpr int kBatch = 2;
    constexpr float kShare = 1.0f / 1024.0f;
    static_assert(kMaxCtas < 1024);
    float x[16] = {}, sum = 0.0f, top = -INFINITY;
    if (group < count) {
#pragma unroll 1
        for (int k0 = group; k0 < count; k0 += kBatch * GROUPS) {
            float log[kBatch];
            float4 y[kBatch][4];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + u * GROUPS;
                const float *p = at(min(k, count - 1));
                const float4 *src = reinterpret_cast<const float4 *>(p + 2 * ROWS + r * D + 16 * part);
                log[u] = k < count ? p[2 * r] : -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[u][e] = k < count ? src[e] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            const float last = top;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) top = fmaxf(top, log[u]);
            const float safe = top == -INFINITY ? 0.0f : top, f0 = ex2(last - safe);
            sum *= f0;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= f0;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const float f = kShare * ex2(log[u] - safe);
                sum += f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[4 * e] += f * y[u][e].x;
                    x[4 * e + 1] += f * y[u][e].y;
                    x[4 * e + 2] += f * y[u][e].z;
                    x[4 * e + 3] += f * y[u][e].w;
                }
            }
        }
        if (group) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[group - 1][e][i] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
        tops[group][i] = make_float2(top, sum);
    }
    __syncthreads();
    if (group) return;
    const Request rq = request_of<ROWS>(a, d.y);
    const int groups = min(GROUPS, count);
    float all = top;
    for (int k = 1; k < groups; ++k) all = fmaxf(all, tops[k][i].x);
    const float safe = all == -INFINITY ? 0.0f : all, f0 = ex2(top - safe);
    sum *= f0;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= f0;
    for (int k = 1; k < groups; ++k) {
        const float2 t = tops[k][i];
        const float f = ex2(t.x - safe);
        sum += f * t.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 y = sums[k - 1][e][i];
            x[4 * e] += f * y.x;
            x[4 * e + 1] += f * y.y;
            x[4 * e + 2] += f * y.z;
            x[4 * e + 3] += f * y.w;
        }
    }
    const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= f;
    store_row(a, rq, d.z, i < USED ? d.w * ROWS + r : 0x7FFFFFFF, part, x);
}

template <int D, int ROWS>
constexpr int attn_smem() {
    constexpr int stages = kTile * (D + 4), outputs = ROWS * (D + 4) * 4;
    return (ROWS / 4) * (D / 32) * 256 +
           kAttnWarps * (outputs_beside<D, ROWS>() ? stages + outputs : stages > outputs ? stages : outputs);
}

}  // namespace kv4

// ====================================================================== host

namespace {

using namespace kv4;

template <class F>
bool set_smem(F *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

convrot_status setup(int *dev) {
    return host::device_setup(dev, [] {
        bool ok = set_smem(plan_kernel, 4 * (CONVROT_KV4_MAX_REQUESTS + 1) * 4);
        ok &= set_smem(attention_kernel<64, 4>, attn_smem<64, 4>());
        ok &= set_smem(attention_kernel<64, 8>, attn_smem<64, 8>());
        ok &= set_smem(attention_kernel<64, 16>, attn_smem<64, 16>());
        ok &= set_smem(attention_kernel<128, 4>, attn_smem<128, 4>());
        ok &= set_smem(attention_kernel<128, 8>, attn_smem<128, 8>());
        ok &= set_smem(attention_kernel<128, 16>, attn_smem<128, 16>());
        ok &= set_smem(attention_kernel<256, 4>, attn_smem<256, 4>());
        ok &= set_smem(attention_kernel<256, 8>, attn_smem<256, 8>());
        return ok;
    });
}

int shift_of(int page) {
    for (int s = 4; s <= 8; ++s)
        if (page == 1 << s) return s;
    return -1;
}

convrot_status check_cache(const convrot_kv4_cache *c) {
    if (!c) return CONVROT_ERR_NULL;
    if (c->group != 64 && c->group != 256) return CONVROT_ERR_GROUP;
    if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->head_dim % c->group)
        return CONVROT_ERR_SHAPE;
    if (shift_of(c->page) < 0 || c->kv_heads < 1 || c->kv_heads > 1024 || c->num_pages < 0 ||
        c->num_pages >= (int64_t(1) << 31) / c->page)
        return CONVROT_ERR_SHAPE;
    return CONVROT_OK;
}

// Pointers of a cache with at least one page.
convrot_status check_cache_ptrs(const convrot_kv4_cache *c) {
    if (!c->num_pages) return CONVROT_OK;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return CONVROT_ERR_NULL;
    return host::aligned16({c->k_codes, c->k_scales, c->v_codes, c->v_scales}) ? CONVROT_OK : CONVROT_ERR_ALIGN;
}

// Bytes of a cache's codes, of its scales, and of T tokens of `row` values with
// ld values between them.
int64_t code_bytes(const convrot_kv4_cache *c) { return c->num_pages * c->kv_heads * c->page * (c->head_dim / 2); }
int64_t scale_bytes(const convrot_kv4_cache *c) { return c->num_pages * c->kv_heads * c->page * 2; }
int64_t token_bytes(int64_t T, int64_t ld, int64_t row) { return ((T - 1) * ld + row) * 2; }

Cache device_cache(const convrot_kv4_cache *c) {
    return Cache{c->k_codes, static_cast<uint16_t *>(c->k_scales), c->v_codes,
                 static_cast<uint16_t *>(c->v_scales), c->num_pages, c->kv_heads,
                 shift_of(c->page), c->head_dim, c->group};
}

convrot_status launched() {
    return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

// One launch of a row kernel over T tokens with E channels a thread: `go` gets
// the head dimension, the number of threads in its type and the grid (up to
// eight CTAs an SM).
template <int E, class F>
convrot_status launch_rows(const convrot_kv4_cache *c, int64_t T, int sms, F go) {
    const int64_t total = T * c->kv_heads * (c->head_dim / E), n = (total + kRowThreads - 1) / kRowThreads;
    const unsigned grid = static_cast<unsigned>(n < 8 * sms ? n : 8 * sms);
    auto with = [&](auto d) {
        // (a thread's number stays below the total and the grid's threads)
        if (total < (int64_t(1) << 31)) go(d, static_cast<uint32_t>(total), grid);
        else go(d, static_cast<uint64_t>(total), grid);
    };
    if (c->head_dim == 64) with(std::integral_constant<int, 64>{});
    else if (c->head_dim == 128) with(std::integral_constant<int, 128>{});
    else with(std::integral_constant<int, 256>{});
    return launched();
}

// Rows of a block: the smallest of 4, 8 and 16 (8 with D = 256, whose
// accumulators fill the registers) that holds an average request's rows.
int block_rows(int64_t T, int64_t B, int G, int D) {
    const int64_t rows = (T + B - 1) / B * G;
    return rows <= 4 ? 4 : rows <= 8 || D == 256 ? 8 : 16;
}

// CTAs that can have work at most, from what the host knows.
int64_t attn_ctas(int64_t T, int64_t B, int G, int kv_heads, int rows, int64_t max_keys) {
    const int64_t blocks = (T * G + rows - 1) / rows + B;
    const int64_t tiles = (max_keys + kTile - 1) / kTile;
    // beyond kMaxCtas the product is not needed, and could overflow
    if (blocks > 8 * kMaxCtas || tiles > 8 * kMaxCtas) return kMaxCtas;
    const int64_t n = (blocks * (tiles > 0 ? tiles : 1) * kv_heads + kMinUnits - 1) / kMinUnits;
    return n < kMaxCtas ? n : kMaxCtas;
}

bool attn_shape_ok(int64_t T, int64_t B, int heads, int kv_heads, int D, int64_t max_keys) {
    return T >= 0 && B >= 0 && B <= CONVROT_KV4_MAX_REQUESTS && T < (int64_t(1) << 31) && kv_heads >= 1 &&
           kv_heads <= 1024 && heads >= kv_heads && heads % kv_heads == 0 && heads <= 65536 &&
           (D == 64 || D == 128 || D == 256) && max_keys >= 0 && max_keys < (int64_t(1) << 31);
}

template <int D, int ROWS>
convrot_status launch_attention(AttnArgs a, int64_t ctas, int sms, cudaStream_t stream) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attention_kernel<D, ROWS>, kAttnThreads,
                                                      attn_smem<D, ROWS>()) != cudaSuccess) {
        cudaGetLastError();
        return CONVROT_ERR_CUDA;
    }
    if (ctas > static_cast<int64_t>(sms) * per_sm) ctas = static_cast<int64_t>(sms) * per_sm;
    const dim3 grid(static_cast<unsigned>(ctas));
    if (host::launch_dependent(attention_kernel<D, ROWS>, grid, dim3(kAttnThreads), attn_smem<D, ROWS>(), stream, a) != CONVROT_OK)
        return CONVROT_ERR_CUDA;
    return host::launch_dependent(combine_kernel<D, ROWS>, grid, dim3(kCombineThreads), 0,
                                  stream, a);
}

}  // namespace

extern "C" {

convrot_status convrot_kv4_plan(const int32_t *cached, const int32_t *new_tokens, int64_t B,
                                int page, int32_t *block_table, int64_t max_pages,
                                int32_t *free_pages, int64_t capacity, const int32_t *free_count,
                                int64_t max_tokens, int32_t *seq_lens, int32_t *cu_q,
                                int64_t *slots, int32_t *positions, int32_t *result,
                                convrot_stream_t stream) {
    const int shift = shift_of(page);
    if (B < 0 || B > CONVROT_KV4_MAX_REQUESTS || shift < 0 || max_pages < 0 || max_pages >= (int64_t(1) << 31) ||
        capacity < 0 || capacity >= (int64_t(1) << 31) || max_tokens < 0 || max_tokens >= (int64_t(1) << 31))
        return CONVROT_ERR_SHAPE;
    if (!free_count || !cu_q || !result || (B && (!cached || !new_tokens || !seq_lens || (max_pages && !block_table))) ||
        (capacity && !free_pages) || (max_tokens && (!slots || !positions)))
        return CONVROT_ERR_NULL;
    if (!host::aligned16({cached, result}) || !host::aligned(8, {slots}) ||
        !host::aligned(4, {new_tokens, block_table, free_pages, free_count, seq_lens, cu_q, positions}))
        return CONVROT_ERR_ALIGN;
    int dev;
    convrot_status st = setup(&dev);
    if (st != CONVROT_OK) return st;
    if ((st = host::check_device_ptrs(dev, {cached, new_tokens, block_table, free_pages, free_count, seq_lens, cu_q,
                                            slots, positions, result})) != CONVROT_OK)
        return st;
    if (host::overlap({{block_table, B * max_pages * 4}, {free_pages, capacity * 4}, {seq_lens, B * 4}, {cu_q, (B + 1) * 4},
                       {slots, max_tokens * 8}, {positions, max_tokens * 4}, {result, 16}},
                      {{cached, B * 4}, {new_tokens, B * 4}, {free_count, 4}}))
        return CONVROT_ERR_OVERLAP;
    PlanArgs a{cached, new_tokens, static_cast<int>(B), shift, block_table, max_pages, free_pages, capacity,
               free_count, max_tokens, seq_lens, cu_q, reinterpret_cast<long long *>(slots), positions, result};
    int64_t grid = (max_tokens + kPlanThreads - 1) / kPlanThreads;
    const int sms = host::g_dev[dev].num_sms;
    grid = grid < 1 ? 1 : grid > sms ? sms : grid;
    plan_kernel<<<static_cast<unsigned>(grid), kPlanThreads, 4 * (B + 1) * 4, stream>>>(a);
    return launched();
}

convrot_status convrot_kv4_append(const convrot_kv4_cache *cache, const void *k_bf16, int64_t ldk,
                                  const void *v_bf16, int64_t ldv, const int64_t *slots, int64_t T,
                                  convrot_stream_t stream) {
    convrot_status st = check_cache(cache);
    if (st != CONVROT_OK) return st;
    const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
    if (T < 0 || T >= (int64_t(1) << 31) || ldk < width || ldv < width || ldk % 8 || ldv % 8) return CONVROT_ERR_SHAPE;
    if (T == 0) return CONVROT_OK;
    if (!k_bf16 || !v_bf16 || !slots) return CONVROT_ERR_NULL;
    if ((st = check_cache_ptrs(cache)) != CONVROT_OK) return st;
    if (!host::aligned16({k_bf16, v_bf16}) || !host::aligned(8, {slots})) return CONVROT_ERR_ALIGN;
    int dev;
    if ((st = setup(&dev)) != CONVROT_OK) return st;
    if ((st = host::check_device_ptrs(dev, {k_bf16, v_bf16, slots, cache->k_codes, cache->k_scales, cache->v_codes,
                                            cache->v_scales})) != CONVROT_OK)
        return st;
    if (host::overlap({{cache->k_codes, code_bytes(cache)}, {cache->k_scales, scale_bytes(cache)},
                       {cache->v_codes, code_bytes(cache)}, {cache->v_scales, scale_bytes(cache)}},
                      {{k_bf16, token_bytes(T, ldk, width)}, {v_bf16, token_bytes(T, ldv, width)}, {slots, T * 8}}))
        return CONVROT_ERR_OVERLAP;
    const int sms = host::g_dev[dev].num_sms;
    auto go = [&](auto e) {
        constexpr int E = decltype(e)::value;
        return launch_rows<E>(cache, T, sms, [&](auto d, auto total, unsigned grid) {
            append_kernel<decltype(d)::value, E, decltype(total)><<<grid, kRowThreads, 0, stream>>>(
                device_cache(cache), static_cast<const uint16_t *>(k_bf16), ldk, static_cast<const uint16_t *>(v_bf16), ldv,
                reinterpret_cast<const long long *>(slots), total);
        });
    };
    return T * width < kFewChannels * sms ? go(std::integral_constant<int, 16>{}) : go(std::integral_constant<int, 32>{});
}

convrot_status convrot_kv4_read(const convrot_kv4_cache *cache, const int64_t *slots, int64_t T,
                                void *k_bf16, void *v_bf16, convrot_stream_t stream) {
    convrot_status st = check_cache(cache);
    if (st != CONVROT_OK) return st;
    if (T < 0 || T >= (int64_t(1) << 31)) return CONVROT_ERR_SHAPE;
    if (T == 0) return CONVROT_OK;
    if (!k_bf16 || !v_bf16 || !slots) return CONVROT_ERR_NULL;
    if ((st = check_cache_ptrs(cache)) != CONVROT_OK) return st;
    if (!host::aligned16({k_bf16, v_bf16}) || !host::aligned(8, {slots})) return CONVROT_ERR_ALIGN;
    int dev;
    if ((st = setup(&dev)) != CONVROT_OK) return st;
    if ((st = host::check_device_ptrs(dev, {k_bf16, v_bf16, slots, cache->k_codes, cache->k_scales, cache->v_codes,
                                            cache->v_scales})) != CONVROT_OK)
        return st;
    const int64_t bytes = T * cache->kv_heads * cache->head_dim * 2;
    if (host::overlap({{k_bf16, bytes}, {v_bf16, bytes}},
                      {{cache->k_codes, code_bytes(cache)}, {cache->k_scales, scale_bytes(cache)},
                       {cache->v_codes, code_bytes(cache)}, {cache->v_scales, scale_bytes(cache)}, {slots, T * 8}}))
        return CONVROT_ERR_OVERLAP;
    return launch_rows<16>(cache, T, host::g_dev[dev].num_sms, [&](auto d, auto total, unsigned grid) {
        read_kernel<decltype(d)::value, decltype(total)><<<grid, kRowThreads, 0, stream>>>(
            device_cache(cache), reinterpret_cast<const long long *>(slots), total, static_cast<uint16_t *>(k_bf16),
            static_cast<uint16_t *>(v_bf16));
    });
}

size_t convrot_kv4_attention_workspace_size(int64_t T, int64_t B, int heads, int kv_heads,
                                            int head_dim, int64_t max_keys) {
    if (!attn_shape_ok(T, B, heads, kv_heads, head_dim, max_keys) || T == 0 || B == 0) return 0;
    const int G = heads / kv_heads, rows = block_rows(T, B, G, head_dim);
    const size_t ctas = static_cast<size_t>(attn_ctas(T, B, G, kv_heads, rows, max_keys));
    return host::round256(ctas * sizeof(int4)) + ctas * 2 * rows * (head_dim + 2) * sizeof(float);
}

convrot_status convrot_kv4_attention(const convrot_kv4_cache *cache, const void *q_bf16,
                                     int64_t ldq, int64_t T, int heads, const int32_t *block_table,
                                     int64_t max_pages, const int32_t *seq_lens,
                                     const int32_t *cu_q, int64_t B, float scale, void *workspace,
                                     size_t ws_bytes, void *out_bf16, convrot_stream_t stream) {
    convrot_status st = check_cache(cache);
    if (st != CONVROT_OK) return st;
    const int D = cache->head_dim;
    if (max_pages < 0 || max_pages >= (int64_t(1) << 31) / cache->page ||
        !attn_shape_ok(T, B, heads, cache->kv_heads, D, max_pages * cache->page) ||
        ldq < static_cast<int64_t>(heads) * D || ldq % 8 || !(scale <= 0x1p100f && scale >= -0x1p100f))
        return CONVROT_ERR_SHAPE;
    if (T == 0 || B == 0) return CONVROT_OK;
    if (!q_bf16 || !seq_lens || !cu_q || !out_bf16 || !workspace || (max_pages && !block_table)) return CONVROT_ERR_NULL;
    if ((st = check_cache_ptrs(cache)) != CONVROT_OK) return st;
    const size_t need = convrot_kv4_attention_workspace_size(T, B, heads, cache->kv_heads, D, max_pages * cache->page);
    if (ws_bytes < need ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return CONVROT_ERR_WORKSPACE;
    if (!host::aligned16({q_bf16, out_bf16}) || !host::aligned(4, {block_table, seq_lens, cu_q})) return CONVROT_ERR_ALIGN;
    int dev;
    if ((st = setup(&dev)) != CONVROT_OK) return st;
    if ((st = host::check_device_ptrs(dev, {q_bf16, block_table, seq_lens, cu_q, out_bf16, workspace, cache->k_codes,
                                            cache->k_scales, cache->v_codes, cache->v_scales})) != CONVROT_OK)
        return st;
    if (host::overlap({{out_bf16, T * heads * D * 2}, {workspace, static_cast<int64_t>(need)}},
                      {{q_bf16, token_bytes(T, ldq, static_cast<int64_t>(heads) * D)}, {block_table, B * max_pages * 4},
                       {seq_lens, B * 4}, {cu_q, (B + 1) * 4}, {cache->k_codes, code_bytes(cache)},
                       {cache->k_scales, scale_bytes(cache)}, {cache->v_codes, code_bytes(cache)}, {cache->v_scales, scale_bytes(cache)}}))
        return CONVROT_ERR_OVERLAP;
    const int G = heads / cache->kv_heads, rows = block_rows(T, B, G, D);
    const int64_t ctas = attn_ctas(T, B, G, cache->kv_heads, rows, max_pages * cache->page);
    AttnArgs a{device_cache(cache), static_cast<const uint16_t *>(q_bf16), ldq, T, G, block_table, max_pages,
               seq_lens, cu_q, static_cast<int>(B), scale * 1.4426950408889634f, static_cast<int4 *>(workspace),
               reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + host::round256(ctas * sizeof(int4))),
               static_cast<uint16_t *>(out_bf16)};
    if (!cache->num_pages) {   // copies of no bytes still name a block's addresses: the workspace holds more
        a.c.kc = a.c.vc = static_cast<uint8_t *>(workspace);
        a.c.ks = a.c.vs = static_cast<uint16_t *>(workspace);
    }
    const int sms = host::g_dev[dev].num_sms;
    auto go = [&](auto d) {
        constexpr int DIM = decltype(d)::value;
        if (rows == 4) return launch_attention<DIM, 4>(a, ctas, sms, stream);
        if (rows == 8) return launch_attention<DIM, 8>(a, ctas, sms, stream);
        return launch_attention<DIM, DIM == 256 ? 8 : 16>(a, ctas, sms, stream);
    };
    return D == 64 ? go(std::integral_constant<int, 64>{})
                   : D == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 256>{});
}

convrot_status convrot_kv4_check_device_error(convrot_stream_t stream) {
    if (cudaStreamSynchronize(stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_convrot_error, sizeof v) != cudaSuccess) return CONVROT_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_convrot_error, &zero, sizeof zero) != cudaSuccess) return CONVROT_ERR_CUDA;
        return static_cast<convrot_status>(v);
    }
    return CONVROT_OK;
}

}  // extern "C"
