// w4g.cu -- the group-scaled few-token variant of the rotated linear layer
// (include/convrot_w4g.h).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/convrot_w4g.h"
#include "frag.cuh"
#include "host.cuh"

namespace w4g {

// ------------------------------------------------------------------ weights, activations
// 16 channels a thread over the matrix as one line of values: a rotation group
// (4 or 16 threads) and a scale group (2, 4 or 8 threads) never cross a row,
// because K is a multiple of both.
constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads)
quantize_kernel(const uint16_t *__restrict__ w, int64_t threads, int group, int scale_group,
                uint8_t *__restrict__ qw, uint16_t *__restrict__ sg) {
    const int lanes = scale_group / 16;
    const float norm = group ? frag::norm_of(group) : 1.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kRowThreads; i0 < threads; i0 += step) {
        const int64_t i = i0 + threadIdx.x;
        float x[16] = {};
        if (i < threads) frag::load16(w + 16 * i, x);
        if (group) frag::rotate16(x, group == 256);
        float factor;
        const uint16_t s = frag::block_scale(frag::absmax_bits(x, lanes), norm, factor);
        uint32_t packed[2];
        prep::quantize_pack(x, factor, packed);
        if (i < threads) {
            *reinterpret_cast<uint2 *>(qw + 8 * i) = make_uint2(packed[0], packed[1]);
            if (i % lanes == 0) sg[i / lanes] = s;
        }
    }
}

__global__ void __launch_bounds__(kRowThreads)
rotate_kernel(const uint16_t *__restrict__ x, int64_t threads, int group, uint16_t *__restrict__ xr) {
    // the product's CTAs may be placed as soon as there is room: they fetch
    // weights and wait for this grid before they read xr
    ptx::launch_dependents();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kRowThreads; i0 < threads; i0 += step) {
        const int64_t i = i0 + threadIdx.x;
        float v[16] = {};
        if (i < threads) frag::load16(x + 16 * i, v);
        frag::rotate16(v, group == 256);
        if (i < threads) frag::store16(xr + 16 * i, v, frag::norm_of(group));
    }
}

// ------------------------------------------------------------------ product
// y^T (rows x tokens) = sum over scale groups of s (codes x tokens): the
// codes, widened exactly to bf16, are the A operand of mma.sync m16n8k16 (16
// weight rows, 16 channels), the tokens its 8 columns.  A group's sum is
// taken in its own fp32 accumulator and joins the row's with one FMA by the
// scale: codes times activations are summed without any rounding of the
// weights.
//
// One CTA has R consecutive rows (R spreads N over the SMs) and all of K.  Its
// warps are (tile of 16 rows, part of K): part p of kp takes the 256-code
// stages p, p + kp, ..., each copied to the warp's own ring in shared memory
// with cp.async (four stages of 16 rows x 128 bytes; no barrier between
// warps).  16-byte chunk c of row r lies at c ^ (r mod 8), so the reads of one
// word from each of 8 rows spread over all banks.  In step j of a stage lane
// (g, t) has word 4 j + t of rows g and g + 8: the 32 channels of a step are
// consecutive, so scale groups of 32 and more never share an accumulator.
// Which channel sits where in the product is free as long as the activations
// agree: they lie in shared memory as 16-byte groups of 8 channels in the
// order (0, 4), (1, 5), (2, 6), (3, 7) of the widened words.
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kStage = 256;                  // codes
constexpr int kStageBytes = 16 * kStage / 2;
constexpr int kDepth = 4;
constexpr int kRing = kWarps * kDepth * kStageBytes;
constexpr int kActBytes = 96 * 1024;         // activations held at a time
constexpr int kMaxRows = 128;                // of a CTA

struct Args {
    const uint16_t *x;       // [M][K], rotated
    const uint8_t *qw;
    const uint16_t *sg;
    const uint16_t *bias;
    uint16_t *y;
    int64_t M, N;
    int K, R;
    int slice;               // stages of activations in shared memory at a time
    int wait;                // a rotation kernel comes before this one
};

// NT: token columns / 8.  SG: scale group.
template <int NT, int SG>
__global__ void __launch_bounds__(kThreads) product_kernel(Args a) {
    constexpr int GROUPS = kStage / SG;      // scale groups of a stage
    extern __shared__ uint4 smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
    const int tokens = static_cast<int>(min(static_cast<int64_t>(8 * NT), a.M - m0));
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * a.R;
    const int rows = static_cast<int>(min(static_cast<int64_t>(a.R), a.N - n0));
    const int stages = (a.K + kStage - 1) / kStage;
    const int tiles = (rows + 15) / 16;
    const int parts = min(kWarps / tiles, stages);
    const int tile = warp % tiles, part = warp / tiles;
    const bool works = part < parts;
    const int tile_rows = min(16, rows - 16 * tile);
    const int groups = a.K / SG;

    const uint32_t ring = ptx::smem_u32(smem) + warp * (kDepth * kStageBytes);
    uint4 *act = smem + kRing / 16;          // [slice * 32 words][tokens]
    const uint8_t *wrow = a.qw + (n0 + 16 * tile) * (a.K / 2);

    auto request = [&](int stage, int slot) {
        if (works && stage < stages) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = (lane >> 3) + 4 * i, c = lane & 7;
                const int byte = stage * (kStage / 2) + 16 * c;
                const bool live = r < tile_rows && byte < a.K / 2;
                frag::cp_async16_or_zero(ring + slot * kStageBytes + r * 128 + ((c ^ (r & 7)) << 4),
                                   live ? wrow + static_cast<int64_t>(r) * (a.K / 2) + byte : a.qw, live);
            }
        }
        prep::cp_async_commit();
    };
    // scales of rows g and g + 8 of a stage
    const uint16_t *srow = a.sg + (n0 + 16 * tile) * groups;
    auto load_scales = [&](int stage, uint16_t (&s)[2][GROUPS]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) {
                const int b = stage * GROUPS + i, r = g + 8 * h;
                s[h][i] = works && r < tile_rows && b < groups ? srow[static_cast<int64_t>(r) * groups + b] : 0;
            }
    };

#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) request(part + i * parts, i);
    uint16_t next[2][GROUPS];
    load_scales(part, next);
    if (a.wait) ptx::grid_dependency_wait();

    float acc[NT][4] = {};
    int stage = part, slot = 0;
    for (int s0 = 0; s0 < stages; s0 += a.slice) {
        const int s1 = min(stages, s0 + a.slice);
        if (s0) __syncthreads();             // the last slice has been read
        const int words = (s1 - s0) * (kStage / 8);
        for (int i = tid; i < words * tokens; i += kThreads) {
            const int m = i / words, w = i % words;
            const int k = (s0 * (kStage / 8) + w) * 8;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (k < a.K) v = *reinterpret_cast<const uint4 *>(a.x + (m0 + m) * a.K + k);
            act[w * tokens + m] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                             __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
        __syncthreads();
        if (!works) continue;
        for (; stage < s1; stage += parts) {
            request(stage + (kDepth - 1) * parts, (slot + kDepth - 1) % kDepth);
            uint16_t sc[2][GROUPS];
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) {
                sc[0][i] = next[0][i];
                sc[1][i] = next[1][i];
            }
            load_scales(stage + parts, next);
            frag::cp_async_wait<kDepth - 1>();
            __syncwarp();
            const uint8_t *src = reinterpret_cast<const uint8_t *>(smem) + warp * (kDepth * kStageBytes) + slot * kStageBytes + 128 * g + 4 * t4;
            const uint4 *xs = act + ((stage - s0) * (kStage / 8) + t4) * tokens + g;
            float part_acc[NT][4] = {};
#pragma unroll
            for (int j = 0; j < kStage / 32; ++j) {
                uint32_t wa[4], wb[4];
                frag::widen_bf16(*reinterpret_cast<const uint32_t *>(src + ((j ^ g) << 4)), wa);
                frag::widen_bf16(*reinterpret_cast<const uint32_t *>(src + 1024 + ((j ^ g) << 4)), wb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (8 * nt + g < tokens) x = xs[4 * j * tokens + 8 * nt];
                    frag::mma_bf16(part_acc[nt], wa[0], wb[0], wa[1], wb[1], x.x, x.y);
                    frag::mma_bf16(part_acc[nt], wa[2], wb[2], wa[3], wb[3], x.z, x.w);
                }
                if ((j + 1) % (SG / 32) == 0) {
                    const int i = j / (SG / 32);
                    const float fa = frag::bf16_f32(sc[0][i]), fb = frag::bf16_f32(sc[1][i]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        acc[nt][0] = fmaf(fa, part_acc[nt][0], acc[nt][0]);
                        acc[nt][1] = fmaf(fa, part_acc[nt][1], acc[nt][1]);
                        acc[nt][2] = fmaf(fb, part_acc[nt][2], acc[nt][2]);
                        acc[nt][3] = fmaf(fb, part_acc[nt][3], acc[nt][3]);
                        part_acc[nt][0] = part_acc[nt][1] = part_acc[nt][2] = part_acc[nt][3] = 0.0f;
                    }
                }
            }
            __syncwarp();                    // the slot is free again
            slot = (slot + 1) % kDepth;
        }
    }
    frag::cp_async_wait<0>();

    // ---- join the parts of K in their order, add the bias, round
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);   // [parts][tokens][tiles * 16]
    const int pitch = tiles * 16;
    if (works) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int m = 8 * nt + 2 * t4 + (x & 1);
                if (m < tokens) red[(part * tokens + m) * pitch + 16 * tile + g + 8 * (x >> 1)] = acc[nt][x];
            }
    }
    __syncthreads();
    for (int i = tid; i < tokens * rows; i += kThreads) {
        const int m = i / rows, r = i % rows;
        float sum = 0.0f;
        for (int p = 0; p < parts; ++p) sum += red[(p * tokens + m) * pitch + r];
        if (a.bias) sum += frag::bf16_f32(a.bias[n0 + r]);
        a.y[(m0 + m) * a.N + n0 + r] = frag::f32_bf16(sum);
    }
}

}  // namespace w4g

// ====================================================================== host

namespace {

using namespace w4g;

template <int NT, int SG>
bool opt_in() {
    return cudaFuncSetAttribute(product_kernel<NT, SG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kRing + kActBytes) == cudaSuccess;
}

convrot_status setup(int *dev) {
    return host::device_setup(dev, [] {
        return opt_in<1, 32>() && opt_in<1, 64>() && opt_in<1, 128>() && opt_in<2, 32>() && opt_in<2, 64>() &&
               opt_in<2, 128>();
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

template <int NT>
convrot_status launch_product(const Args &a, int scale_group, int sms, cudaStream_t stream) {
    const int stages = (a.K + kStage - 1) / kStage;
    const int slice = a.slice < stages ? a.slice : stages;
    const int64_t tokens = a.M < 8 * NT ? a.M : 8 * NT;
    const dim3 grid(static_cast<unsigned>((a.N + a.R - 1) / a.R), static_cast<unsigned>((a.M + 8 * NT - 1) / (8 * NT)));
    const size_t smem = kRing + static_cast<size_t>(slice) * kStage * 2 * tokens;
    auto go = [&](auto *kernel) {
        if (a.wait) return host::launch_dependent(kernel, grid, dim3(kThreads), smem, stream, a);
        kernel<<<grid, kThreads, smem, stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
    };
    return scale_group == 32 ? go(product_kernel<NT, 32>)
                             : scale_group == 64 ? go(product_kernel<NT, 64>) : go(product_kernel<NT, 128>);
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
    const int64_t threads = N * (K / 16);
    quantize_kernel<<<row_grid(threads, host::g_dev[dev].num_sms), kRowThreads, 0, stream>>>(
        static_cast<const uint16_t *>(w_bf16), threads, group, scale_group, qw, static_cast<uint16_t *>(sg_bf16));
    return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

size_t convrot_w4g_workspace_size(int64_t M, int64_t K, int group) {
    if (M <= 0 || K <= 0 || group == 0) return 0;
    return host::round256(static_cast<size_t>(M) * static_cast<size_t>(K) * 2);
}

convrot_status convrot_w4g_linear(const void *x_bf16, const uint8_t *qw, const void *sg_bf16,
                                  const void *bias_bf16, int64_t M, int64_t N, int64_t K,
                                  int group, int scale_group, void *workspace, size_t ws_bytes,
                                  void *y_bf16, convrot_stream_t stream) {
    convrot_status st = check_shape(M, K, group, scale_group);
    if (st != CONVROT_OK) return st;
    if (N < 0 || N > (int64_t(1) << 30) || M > 65535 * 8 || M * N > (int64_t(1) << 40)) return CONVROT_ERR_SHAPE;
    if (M == 0 || N == 0) return CONVROT_OK;
    const size_t need = convrot_w4g_workspace_size(M, K, group);
    if (!x_bf16 || !qw || !sg_bf16 || !y_bf16 || (need && !workspace)) return CONVROT_ERR_NULL;
    if (need && (ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))) return CONVROT_ERR_WORKSPACE;
    if (!host::aligned16({x_bf16, qw, sg_bf16, bias_bf16, y_bf16})) return CONVROT_ERR_ALIGN;
    int dev;
    if ((st = setup(&dev)) != CONVROT_OK) return st;
    if ((st = host::check_device_ptrs(dev, {x_bf16, qw, sg_bf16, bias_bf16, y_bf16, need ? workspace : nullptr})) != CONVROT_OK)
        return st;
    const int sms = host::g_dev[dev].num_sms;
    const uint16_t *x = static_cast<const uint16_t *>(x_bf16);
    if (group) {
        const int64_t threads = M * (K / 16);
        rotate_kernel<<<row_grid(threads, sms), kRowThreads, 0, stream>>>(x, threads, group, static_cast<uint16_t *>(workspace));
        if (cudaGetLastError() != cudaSuccess) return CONVROT_ERR_CUDA;
        x = static_cast<const uint16_t *>(workspace);
    }
    // rows of a CTA: N spread evenly over whole waves of one CTA an SM
    const int64_t waves = (N + static_cast<int64_t>(sms) * kMaxRows - 1) / (static_cast<int64_t>(sms) * kMaxRows);
    const int R = static_cast<int>((N + sms * waves - 1) / (sms * waves));
    const int64_t tokens = M <= 8 ? M : M < 16 ? M : 16;
    Args a{x, qw, static_cast<const uint16_t *>(sg_bf16), static_cast<const uint16_t *>(bias_bf16),
           static_cast<uint16_t *>(y_bf16), M, N, static_cast<int>(K), R,
           static_cast<int>(kActBytes / (kStage * 2 * tokens)), group != 0};
    return M <= 8 ? launch_product<1>(a, scale_group, sms, stream) : launch_product<2>(a, scale_group, sms, stream);
}

}  // extern "C"
