// Rotary positions and head norms over rows of heads, and their gradients.
//
// Mathematics (see include/cli.h).  A head of D elements is cut into slots of
// two chunks of VEC elements that hold whole pairs: chunk A at VEC s and chunk
// B at rotary_dim / 2 + VEC s in the half layout, 2 VEC neighbours in the
// interleaved one; what is not rotated is cut the same way and turned by
// (cos, sin) = (1, 0).  A lane owns the same slots of every head it sees, so
// the (cos, sin) of its pairs are loaded once per row and its gains once per
// call; a head's sums are a few shuffles among its lanes; a warp takes
// 32 / (lanes per head) heads at a time.
//
// Bound: HBM.  Each input is read once and each output written once, in
// 16-byte accesses wherever rotary_dim allows (VEC = 8); the table is read
// once per row and stays in L2.
//
// The gain's gradient: a lane sums its slots over the heads and rows it sees
// in registers, a block adds its lanes' sums in a fixed order into one row of
// partials, and a second kernel adds those rows: no atomics, so the result
// does not depend on the order in which blocks run.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cli_device.cuh"
#include "cli_internal.h"

namespace cli {
namespace rotary {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) { return pack_bf16x2(a, b); }
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

// VEC consecutive elements at p (aligned to VEC elements, at most 16 bytes) as floats, and back.
template <typename T, int VEC>
struct Chunk {
    static __device__ __forceinline__ void load(const T *p, float *v) {
        if constexpr (sizeof(T) == 4) {
            if constexpr (VEC >= 4) {
#pragma unroll
                for (int i = 0; i < VEC; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(p + i);
                    v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
                }
            } else if constexpr (VEC == 2) {
                const float2 f = *reinterpret_cast<const float2 *>(p);
                v[0] = f.x, v[1] = f.y;
            } else {
                v[0] = *p;
            }
        } else if constexpr (VEC == 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<T>(w[i]);
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        } else if constexpr (VEC == 2) {
            const float2 f = unpack2<T>(*reinterpret_cast<const uint32_t *>(p));
            v[0] = f.x, v[1] = f.y;
        } else {
            v[0] = static_cast<float>(*p);
        }
    }
    static __device__ __forceinline__ void store(T *p, const float *v) {
        if constexpr (sizeof(T) == 4) {
            if constexpr (VEC >= 4) {
#pragma unroll
                for (int i = 0; i < VEC; i += 4)
                    *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            } else if constexpr (VEC == 2) {
                *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
            } else {
                *p = v[0];
            }
        } else if constexpr (VEC == 8) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                       pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        } else if constexpr (VEC == 2) {
            *reinterpret_cast<uint32_t *>(p) = pack2<T>(v[0], v[1]);
        } else {
            *p = static_cast<T>(v[0]);
        }
    }
};

enum Mode { kRotate, kNorm, kNormGrad };

// T: element type.  VEC: elements of a chunk.  SPL: slots of a lane (SPL * VEC
// covers 128 pairs over 32 lanes).  INTER: interleaved pairs.
template <typename T, int VEC, bool INTER, Mode MODE>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ RotaryLaunch P) {
    constexpr int SPL = VEC >= 4 ? 1 : 4 / VEC;
    constexpr int N = VEC * SPL;   // pairs of a lane
    using C = Chunk<T, VEC>;
    const RotaryPartLaunch &part = P.part[blockIdx.y];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lph = 1 << P.lph_log2;             // lanes of a head
    const int sub = lane & (lph - 1), group = lane >> P.lph_log2, groups = 32 >> P.lph_log2;
    const int half = P.rotary_dim >> 1, D = P.head_dim;

    // This lane's slots: element offsets of the chunks (-1: none) and whether they are rotated.
    int a_at[SPL], b_at[SPL], pair[SPL];
#pragma unroll
    for (int j = 0; j < SPL; ++j) {
        const int s = sub + j * lph;
        if constexpr (INTER) {
            a_at[j] = 2 * VEC * s < D ? 2 * VEC * s : -1;
            b_at[j] = 2 * VEC * s + VEC < D ? 2 * VEC * s + VEC : -1;
            pair[j] = VEC * s;                   // pairs past rotary_dim / 2 are guarded one by one
        } else {
            const int turned = half / VEC;       // slots of the rotated part
            const int rest = P.rotary_dim + 2 * VEC * (s - turned);
            a_at[j] = s < turned ? VEC * s : rest < D ? rest : -1;
            b_at[j] = s < turned ? half + VEC * s : rest + VEC < D ? rest + VEC : -1;
            pair[j] = s < turned ? VEC * s : -1;
        }
    }
    float gain[2 * N], dg[2 * N];
    if constexpr (MODE != kRotate) {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
            const int j = (i % N) / VEC, at = i < N ? a_at[j] : b_at[j];
            gain[i] = part.gain && at >= 0 ? part.gain[at + i % VEC] : 1.0f;
            dg[i] = 0.0f;
        }
    }

    for (int row = blockIdx.x * kWarps + warp; row < part.rows; row += gridDim.x * kWarps) {
        const int pos = part.positions ? part.positions[row] : row;
        if (pos < 0 || pos >= P.table_rows) {    // the same for the warp
            if (lane == 0) report(P.status, CLI_MALFORMED);
            continue;
        }
        float c[N], s[N];
        const float2 *cs = P.table + static_cast<long long>(pos) * half;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int first = pair[i / VEC], p = first + i % VEC;
            const bool on = INTER ? p < half : first >= 0;
            const float2 f = on ? __ldg(cs + p) : make_float2(1.0f, 0.0f);
            c[i] = f.x;
            s[i] = P.sin_sign * f.y;
        }
        for (int h0 = 0; h0 < part.heads; h0 += groups) {
            const int h = h0 + group;
            const bool on = h < part.heads;
            // v: the chunks of A, then those of B.
            float v[2 * N], x[MODE == kNormGrad ? 2 * N : 1];
            const T *in = static_cast<const T *>(part.in) + row * part.in_row + h * part.in_head;
#pragma unroll
            for (int j = 0; j < 2 * SPL; ++j) {
                const int at = j < SPL ? a_at[j] : b_at[j - SPL];
                if (on && at >= 0) {
                    C::load(in + at, v + j * VEC);
                    if constexpr (MODE == kNormGrad)
                        C::load(static_cast<const T *>(part.x) + row * part.x_row + h * part.x_head + at, x + j * VEC);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        v[j * VEC + i] = 0.0f;
                        if constexpr (MODE == kNormGrad) x[j * VEC + i] = 0.0f;
                    }
                }
            }
            if constexpr (MODE == kNorm) {
                float sq = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) sq = fmaf(v[i], v[i], sq);
                for (int o = 1; o < lph; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                const float r = rsqrtf(sq * P.inv_dim + P.epsilon);
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) v[i] *= r * gain[i];
            }
            // Rotation.  Interleaved pairs lie within a chunk: (2 i, 2 i + 1) of A's, then of B's.
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float a = v[2 * i], b = v[2 * i + 1];
                    v[2 * i] = a * c[i] - b * s[i];
                    v[2 * i + 1] = b * c[i] + a * s[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float a = v[i], b = v[N + i];
                    v[i] = a * c[i] - b * s[i];
                    v[N + i] = b * c[i] + a * s[i];
                }
            }
            if constexpr (MODE == kNormGrad) {   // v is dz here
                float sq = 0.0f, tx = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) {
                    sq = fmaf(x[i], x[i], sq);
                    tx = fmaf(v[i] * gain[i], x[i], tx);
                }
                for (int o = 1; o < lph; o <<= 1) {
                    sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    tx += __shfl_xor_sync(0xffffffffu, tx, o);
                }
                const float r = rsqrtf(sq * P.inv_dim + P.epsilon);
                const float k = r * r * tx * P.inv_dim;
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) {
                    dg[i] = fmaf(v[i], x[i] * r, dg[i]);
                    v[i] = r * (v[i] * gain[i] - k * x[i]);
                }
            }
            T *out = static_cast<T *>(part.out) + row * part.out_row + h * part.out_head;
#pragma unroll
            for (int j = 0; j < 2 * SPL; ++j) {
                const int at = j < SPL ? a_at[j] : b_at[j - SPL];
                if (on && at >= 0) C::store(out + at, v + j * VEC);
            }
        }
    }

    if constexpr (MODE == kNormGrad) {
        if (!part.gain_partials) return;
        // One row of partials per block: element by element over the block's warps and head groups.
        __shared__ float sums[kThreads * 2 * N];   // [warp][group][D <= lph * 2 N]
        float *mine = sums + (warp * groups + group) * D;
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
            const int j = (i % N) / VEC, at = i < N ? a_at[j] : b_at[j];
            if (at >= 0) mine[at + i % VEC] = dg[i];
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < D) {
            float t = 0.0f;
            for (int g = 0; g < kWarps * groups; ++g) t += sums[g * D + threadIdx.x];
            part.gain_partials[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = t;
        }
    }
}

// d_gain[i] = the sum of the blocks' partials, each warp a fixed share of the rows.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const __grid_constant__ RotaryLaunch P, int blocks) {
    const RotaryPartLaunch &part = P.part[blockIdx.y];
    if (!part.gain_partials) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    __shared__ float sums[32][33];
    float t = 0.0f;
    if (i < P.head_dim)
        for (int b = warp; b < blocks; b += 32) t += part.gain_partials[static_cast<size_t>(b) * P.head_dim + i];
    sums[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && i < P.head_dim) {
        t = 0.0f;
        for (int w = 0; w < 32; ++w) t += sums[w][lane];
        part.d_gain[i] = t;
    }
}

struct Frequencies {
    double f[128];
};

__global__ void __launch_bounds__(256) table_kernel(float2 *table, long long cells, int half, double amplitude,
                                                    const __grid_constant__ Frequencies F) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < cells; i += gridDim.x * 256ll) {
        const long long p = i / half;
        double s, c;
        sincos(static_cast<double>(p) * F.f[i - p * half], &s, &c);
        table[i] = make_float2(static_cast<float>(amplitude * c), static_cast<float>(amplitude * s));
    }
}

template <typename T, Mode MODE>
void launch_layout(const RotaryLaunch &L, dim3 grid, int vec, cudaStream_t stream) {
    if (L.interleaved)
        heads_kernel<T, 8, true, MODE><<<grid, kThreads, 0, stream>>>(L);
    else if (vec == 8)
        heads_kernel<T, 8, false, MODE><<<grid, kThreads, 0, stream>>>(L);
    else if (vec == 2)
        heads_kernel<T, 2, false, MODE><<<grid, kThreads, 0, stream>>>(L);
    else
        heads_kernel<T, 1, false, MODE><<<grid, kThreads, 0, stream>>>(L);
}

template <typename T>
void launch_mode(const RotaryLaunch &L, dim3 grid, int vec, cudaStream_t stream) {
    if (!L.norm)
        launch_layout<T, kRotate>(L, grid, vec, stream);
    else if (!L.backward)
        launch_layout<T, kNorm>(L, grid, vec, stream);
    else
        launch_layout<T, kNormGrad>(L, grid, vec, stream);
}

}  // namespace
}  // namespace rotary

cudaError_t launch_rotary_table(float *table, long long positions, int half, const double *frequencies,
                                double amplitude, cudaStream_t stream) {
    rotary::Frequencies F;
    for (int i = 0; i < half; ++i) F.f[i] = frequencies[i];
    const long long cells = positions * half, blocks = (cells + 255) / 256;
    rotary::table_kernel<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), 256, 0, stream>>>(
        reinterpret_cast<float2 *>(table), cells, half, amplitude, F);
    return cudaGetLastError();
}

cudaError_t launch_rotary(RotaryLaunch L, cudaStream_t stream) {
    using namespace rotary;
    // Chunks of 8 where both halves of the rotated part start on a multiple of 8, else the widest that do.
    const int half = L.rotary_dim / 2;
    const int vec = L.interleaved || half % 8 == 0 ? 8 : half % 2 == 0 ? 2 : 1;
    const int slots = (L.head_dim + 2 * vec - 1) / (2 * vec);
    const int spl = vec >= 4 ? 1 : 4 / vec;
    L.lph_log2 = 0;
    while ((spl << L.lph_log2) < slots) ++L.lph_log2;
    const int parts = L.part[1].heads ? 2 : 1;
    const int rows = L.part[0].rows > L.part[1].rows ? L.part[0].rows : L.part[1].rows;
    const int want = (rows + kWarps - 1) / kWarps;
    const int most = rotary_blocks(L.sm_count);
    const int blocks = want < 1 ? 1 : want < most ? want : most;
    const dim3 grid(blocks, parts);
    if (L.dtype == CLI_BF16)
        launch_mode<__nv_bfloat16>(L, grid, vec, stream);
    else if (L.dtype == CLI_F16)
        launch_mode<__half>(L, grid, vec, stream);
    else
        launch_mode<float>(L, grid, vec, stream);
    if (L.part[0].gain_partials || L.part[1].gain_partials)
        gain_sum_kernel<<<dim3((L.head_dim + 31) / 32, parts), 1024, 0, stream>>>(L, blocks);
    return cudaGetLastError();
}

}  // namespace cli
