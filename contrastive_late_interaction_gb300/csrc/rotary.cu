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
// Bound: HBM.  Each input is read once and each output written once, and the
// table is read once per row and stays in L2.  What it takes to stream is to
// have enough on its way: a warp that loads a row, looks its position up,
// loads its angles, computes and stores, waits most of the time (3.2 TB/s for
// the gradients).  stream_kernel, which takes every call whose rotated halves
// start on a multiple of 8, copies what a warp needs two steps from now into
// shared memory (cp.async; a step is 32 / (lanes per head) heads of a row), so
// some 100 KB an SM are under way; the rest go through heads_kernel.  Measured
// in bf16: the norm with rotation of 270336 rows, 32 heads of 64, 355 us (6.2
// TB/s), the gradient of 131072 rows, 16 heads of 128, 279 us (5.8 TB/s).  A step
// does not span rows, so a part with few heads leaves lanes idle: in fp32 the
// rotation of 20011 rows, 8 + 2 heads of 80 (four a step), takes 34 us (3.7
// TB/s), the norm with rotation of 100000 rows, 8 + 1 heads of 64 (eight a
// step), 184 us (1.3 TB/s).  heads_kernel: 131072 rows, 16 heads of 128, 100 of
// each rotated, 251 us (4.3 TB/s), the gradient 700 (2.3 TB/s); 102 rotated, in
// chunks of one, 326 us.
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

// ----------------------------------------------------------------------------
// pieces
// ----------------------------------------------------------------------------

// Rotation of a lane's N pairs.  Interleaved pairs lie within a chunk:
// (2 i, 2 i + 1) of A's, then of B's.
template <bool INTER, int N>
__device__ __forceinline__ void rotate(float (&v)[2 * N], const float (&c)[N], const float (&s)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int p = INTER ? 2 * i : i, q = INTER ? 2 * i + 1 : N + i;
        const float a = v[p], b = v[q];
        v[p] = a * c[i] - b * s[i];
        v[q] = b * c[i] + a * s[i];
    }
}

template <int N>
__device__ __forceinline__ void norm(float (&v)[2 * N], const float (&gain)[2 * N], int lph, float inv_dim, float epsilon) {
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) sq = fmaf(v[i], v[i], sq);
    for (int o = 1; o < lph; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float r = rsqrtf(sq * inv_dim + epsilon);
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) v[i] *= r * gain[i];
}

// dz in v becomes dx; the gain's gradient is added to dg.
template <int N>
__device__ __forceinline__ void norm_grad(float (&v)[2 * N], const float (&x)[2 * N], const float (&gain)[2 * N],
                                          float (&dg)[2 * N], int lph, float inv_dim, float epsilon) {
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
    const float r = rsqrtf(sq * inv_dim + epsilon);
    const float k = r * r * tx * inv_dim;
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
        dg[i] = fmaf(v[i], x[i] * r, dg[i]);
        v[i] = r * (v[i] * gain[i] - k * x[i]);
    }
}

// A block's part of the call, and its place among that part's blocks.
struct Share {
    int part, block, blocks;
};
__device__ __forceinline__ Share share_of(const RotaryLaunch &P) {
    const int b = blockIdx.x;
    return b < P.q_blocks ? Share{0, b, P.q_blocks} : Share{1, b - P.q_blocks, static_cast<int>(gridDim.x) - P.q_blocks};
}

// A call on few rows has no memset of the status before it: block 0 looks at
// every position and writes the word, and nobody else reports.
constexpr int kFewRows = 1024;
__device__ __forceinline__ bool few_rows(const RotaryLaunch &P) { return static_cast<long long>(P.part[0].rows) + P.part[1].rows <= kFewRows; }

__device__ __forceinline__ void write_status(const RotaryLaunch &P) {
    if (blockIdx.x != 0 || !few_rows(P)) return;   // the same for the block
    bool bad = false;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const RotaryPartLaunch &part = P.part[p];
        if (!part.positions) {
            bad |= part.rows > P.table_rows;
            continue;
        }
#pragma unroll 8
        for (int r = threadIdx.x; r < part.rows; r += blockDim.x) {
            const int pos = part.positions[r];
            bad |= pos < 0 || pos >= P.table_rows;
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *P.status = bad ? CLI_MALFORMED : CLI_OK;
}

// One row of partials of the gain's gradient: the block's lanes add up in a fixed order.
template <int N, int VEC, int WARPS>
__device__ __forceinline__ void gain_partial(const RotaryLaunch &P, float *to, const int *a_at, const int *b_at,
                                             const float (&dg)[2 * N], float *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = P.head_dim;
    const int groups = 32 >> P.lph_log2, group = lane >> P.lph_log2;
    float *mine = sums + (warp * groups + group) * D;   // [warp][group][D <= lanes of a head * 2 N]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
        const int j = (i % N) / VEC, at = i < N ? a_at[j] : b_at[j];
        if (at >= 0) mine[at + i % VEC] = dg[i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += WARPS * 32) {
        float t = 0.0f;
        for (int g = 0; g < WARPS * groups; ++g) t += sums[g * D + d];
        to[d] = t;
    }
}

// ----------------------------------------------------------------------------
// streaming kernel: chunks of 8, rotary_dim / 2 a multiple of 8
// ----------------------------------------------------------------------------

constexpr int kStreamWarps = 4;

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// The 8 elements in one unit of 16 bytes (16-bit types) or two (fp32), and back.
template <typename T>
__device__ __forceinline__ void floats_of(const uint4 *u, float *v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(u[i].x), v[4 * i + 1] = __uint_as_float(u[i].y);
            v[4 * i + 2] = __uint_as_float(u[i].z), v[4 * i + 3] = __uint_as_float(u[i].w);
        }
    } else {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(w[i]);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
}

template <typename T, Mode MODE>
struct Stream {
    static constexpr int kUnits = sizeof(T) / 2;                        // 16 bytes each, of a chunk
    static constexpr int kTensors = MODE == kNormGrad ? 2 : 1;
    static constexpr int kStages = 3;   // 2: 396 us where 3 takes 355, 4: 358, 6: 385
    static constexpr int kStageBytes = 2 * kTensors * kUnits * 32 * 16;
    // a warp's stages, and the angles of as many rows as may be under way
    static size_t warp_bytes(int half) { return kStages * kStageBytes + (kStages + 1) * static_cast<size_t>(half) * 8; }
};

template <typename T, bool INTER, Mode MODE>
__global__ void __launch_bounds__(kStreamWarps * 32, MODE == kNormGrad ? 4 : 6)
    stream_kernel(const __grid_constant__ RotaryLaunch P) {
    using S = Stream<T, MODE>;
    constexpr int N = 8, kStages = S::kStages, kUnits = S::kUnits;
    extern __shared__ __align__(16) uint8_t smem[];
    write_status(P);
    const Share share = share_of(P);
    const RotaryPartLaunch &part = P.part[share.part];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lph = 1 << P.lph_log2, sub = lane & (lph - 1), group = lane >> P.lph_log2, groups = 32 >> P.lph_log2;
    const int half = P.rotary_dim >> 1, D = P.head_dim;
    const size_t warp_bytes = kStages * S::kStageBytes + (kStages + 1) * static_cast<size_t>(half) * 8;
    const uint32_t stage0 = smem_u32(smem) + static_cast<uint32_t>(warp * warp_bytes);
    const uint32_t angle0 = smem_u32(smem) + static_cast<uint32_t>(warp * warp_bytes) + kStages * S::kStageBytes;

    // This lane's two chunks (-1: none) and the first of its pairs (-1: not rotated).
    int a_at, b_at, pair;
    if constexpr (INTER) {
        a_at = 16 * sub < D ? 16 * sub : -1;
        b_at = 16 * sub + 8 < D ? 16 * sub + 8 : -1;
        pair = 8 * sub < half ? 8 * sub : -1;
    } else {
        const int turned = half / 8, rest = P.rotary_dim + 16 * (sub - turned);
        a_at = sub < turned ? 8 * sub : rest < D ? rest : -1;
        b_at = sub < turned ? half + 8 * sub : rest + 8 < D ? rest + 8 : -1;
        pair = sub < turned ? 8 * sub : -1;
    }
    // What it copies of a step.  Its own chunks, where the lanes' chunks are neighbours (16-bit halves); elsewhere
    // every 32nd 16 bytes of the step's heads, so that a request still covers whole lines (36 -> 31 us for 20011
    // rows of fp32 pairs), at the price of a head's address for each copy (371 -> 443 us for 270336 rows of halves).
    constexpr bool kOwn = !INTER && sizeof(T) == 2;
    constexpr int kCopies = 2 * kUnits;
    const int head_units = D * static_cast<int>(sizeof(T)) / 16;
    int copy_head[kCopies], copy_at[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies && !kOwn; ++i) {
        const int u = lane + 32 * i;
        copy_head[i] = u < groups * head_units ? u / head_units : 1 << 30;
        copy_at[i] = u % head_units * (16 / static_cast<int>(sizeof(T)));
    }
    float gain[2 * N], dg[2 * N];
    if constexpr (MODE != kRotate) {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
            const int at = i < N ? a_at : b_at;
            gain[i] = part.gain && at >= 0 ? part.gain[at + i % 8] : 1.0f;
            dg[i] = 0.0f;
        }
    }

    // This warp's rows first, first + step, ...; a step takes `groups` heads of one.
    const int first = share.block * kStreamWarps + warp, stride = share.blocks * kStreamWarps;
    const int my_rows = first < part.rows ? (part.rows - 1 - first) / stride + 1 : 0;
    const int head_steps = (part.heads + groups - 1) / groups;
    const long long steps = static_cast<long long>(my_rows) * head_steps;
    auto row_of = [&](int k) { return first + k * static_cast<long long>(stride); };
    // Positions, 32 of the warp's rows at a time, a row a lane; one outside the table is reported and read as 0.
    int positions = 0;
    auto look_up = [&](int k) {
        const int mine = k + lane;
        int p = 0;
        if (mine < my_rows) {
            p = part.positions ? part.positions[row_of(mine)] : static_cast<int>(row_of(mine));
            if (p < 0 || p >= P.table_rows) {
                if (!few_rows(P)) report(P.status, CLI_MALFORMED);
                p = 0;
            }
        }
        positions = p;
    };

    int at_row = 0, at_head = 0;   // of the next step to copy
    auto copy_step = [&](int stage) {
        if (at_row < my_rows) {
            const long long row = row_of(at_row);
            if (at_head == 0) {
                if ((at_row & 31) == 0) look_up(at_row);
                const int p = __shfl_sync(0xffffffffu, positions, at_row & 31);
                const float2 *from = P.table + static_cast<long long>(p) * half;
                const uint32_t to = angle0 + static_cast<uint32_t>(at_row % (kStages + 1)) * half * 8;
                for (int i = 2 * lane; i < half; i += 64) copy16(to + i * 8, from + i);
            }
            const uint32_t to = stage0 + stage * S::kStageBytes + lane * 16;
            if constexpr (kOwn) {
                const int h = at_head * groups + group;
                if (h < part.heads) {
                    const T *in = static_cast<const T *>(part.in) + row * part.in_row + h * part.in_head;
                    const T *x = static_cast<const T *>(part.x) + row * part.x_row + h * part.x_head;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int e = c ? b_at : a_at;
                        if (e < 0) continue;
                        copy16(to + c * 512, in + e);
                        if constexpr (MODE == kNormGrad) copy16(to + (2 + c) * 512, x + e);
                    }
                }
            } else {
                const T *in = static_cast<const T *>(part.in) + row * part.in_row;
                const T *x = static_cast<const T *>(part.x) + row * part.x_row;
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const int h = at_head * groups + copy_head[i];
                    if (h >= part.heads) continue;
                    copy16(to + i * 512, in + h * part.in_head + copy_at[i]);
                    if constexpr (MODE == kNormGrad) copy16(to + (kCopies + i) * 512, x + h * part.x_head + copy_at[i]);
                }
            }
            if (++at_head == head_steps) at_head = 0, ++at_row;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) copy_step(s);

    float c[N], s[N];
    int row_k = 0, head_k = 0, stage = 0;
    for (long long t = 0; t < steps; ++t) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();   // what a lane reads is copied by others
        if (head_k == 0) {
            const uint32_t from = angle0 + static_cast<uint32_t>(row_k % (kStages + 1)) * half * 8 + pair * 8;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                uint4 u = make_uint4(__float_as_uint(1.0f), 0, __float_as_uint(1.0f), 0);
                if (pair >= 0) u = shared16(from + i * 8);
                c[i] = __uint_as_float(u.x), s[i] = P.sin_sign * __uint_as_float(u.y);
                c[i + 1] = __uint_as_float(u.z), s[i + 1] = P.sin_sign * __uint_as_float(u.w);
            }
        }
        const int h = head_k * groups + group;
        const bool on = h < part.heads;
        float v[2 * N], x[MODE == kNormGrad ? 2 * N : 1];
        const uint32_t from = stage0 + stage * S::kStageBytes + (kOwn ? lane : group * head_units) * 16;
#pragma unroll
        for (int k = 0; k < 2 * S::kTensors; ++k) {
            float *to = k < 2 ? v + 8 * k : x + 8 * (k - 2);
            const int e = k & 1 ? b_at : a_at;
            uint4 u[kUnits];
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
                u[i] = on && e >= 0 ? shared16(from + (kOwn ? k * 512 : (k >> 1) * kCopies * 512 + e * static_cast<int>(sizeof(T)) + i * 16))
                                    : make_uint4(0, 0, 0, 0);
            floats_of<T>(u, to);
        }
        // Every lane has read its part of the stage and its angles: the copies go on.
        __syncwarp();
        int next = stage + kStages - 1;
        copy_step(next >= kStages ? next - kStages : next);
        if constexpr (MODE == kNorm) norm<N>(v, gain, lph, P.inv_dim, P.epsilon);
        rotate<INTER, N>(v, c, s);
        if constexpr (MODE == kNormGrad) norm_grad<N>(v, x, gain, dg, lph, P.inv_dim, P.epsilon);
        if (on) {
            T *out = static_cast<T *>(part.out) + row_of(row_k) * part.out_row + h * part.out_head;
            if (a_at >= 0) Chunk<T, 8>::store(out + a_at, v);
            if (b_at >= 0) Chunk<T, 8>::store(out + b_at, v + 8);
        }
        if (++head_k == head_steps) head_k = 0, ++row_k;
        if (++stage == kStages) stage = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (MODE == kNormGrad) {
        if (part.gain_partials)
            gain_partial<N, 8, kStreamWarps>(P, part.gain_partials + static_cast<size_t>(share.block) * D, &a_at, &b_at, dg,
                                             reinterpret_cast<float *>(smem));
    }
}

// ----------------------------------------------------------------------------
// the rest
// ----------------------------------------------------------------------------

// T: element type.  VEC: elements of a chunk.  SPL: slots of a lane (SPL * VEC
// covers 128 pairs over 32 lanes).  INTER: interleaved pairs.
template <typename T, int VEC, bool INTER, Mode MODE>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ RotaryLaunch P) {
    constexpr int SPL = VEC >= 4 ? 1 : 4 / VEC;
    constexpr int N = VEC * SPL;   // pairs of a lane
    using C = Chunk<T, VEC>;
    write_status(P);
    const Share share = share_of(P);
    const RotaryPartLaunch &part = P.part[share.part];
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

    for (long long row = share.block * kWarps + warp; row < part.rows; row += share.blocks * kWarps) {
        int pos = part.positions ? part.positions[row] : static_cast<int>(row);
        if (pos < 0 || pos >= P.table_rows) {    // reported and read as 0, as above; the same for the warp
            if (lane == 0 && !few_rows(P)) report(P.status, CLI_MALFORMED);
            pos = 0;
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
            if constexpr (MODE == kNorm) norm<N>(v, gain, lph, P.inv_dim, P.epsilon);
            rotate<INTER, N>(v, c, s);
            if constexpr (MODE == kNormGrad) norm_grad<N>(v, x, gain, dg, lph, P.inv_dim, P.epsilon);
            T *out = static_cast<T *>(part.out) + row * part.out_row + h * part.out_head;
#pragma unroll
            for (int j = 0; j < 2 * SPL; ++j) {
                const int at = j < SPL ? a_at[j] : b_at[j - SPL];
                if (on && at >= 0) C::store(out + at, v + j * VEC);
            }
        }
    }

    if constexpr (MODE == kNormGrad) {
        __shared__ float sums[kThreads * 2 * N];
        if (part.gain_partials)
            gain_partial<N, VEC, kWarps>(P, part.gain_partials + static_cast<size_t>(share.block) * D, a_at, b_at, dg, sums);
    }
}

// d_gain[i] = the sum of the blocks' partials, each warp a fixed share of the rows.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const __grid_constant__ RotaryLaunch P, int all_blocks) {
    const RotaryPartLaunch &part = P.part[blockIdx.y];
    const int blocks = blockIdx.y ? all_blocks - P.q_blocks : P.q_blocks;
    if (!part.gain_partials) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    __shared__ float sums[32][33];
    float t = 0.0f;
    if (i < P.head_dim) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += 32) t += part.gain_partials[static_cast<size_t>(b) * P.head_dim + i];
    }
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

// Blocks of the parts, in proportion to the heads that they move, at least one
// each.  A warp's time goes by its steps, rows * ceil(heads / heads a step), so
// that a part whose heads do not fill a step has too few blocks (20011 rows, 8 + 2
// heads of 80: 28 steps a warp for the keys, 14 for the queries).
void split(RotaryLaunch &L, int rows_a_block, int most, int &blocks) {
    long long work[2], want[2];
    for (int p = 0; p < 2; ++p) {
        work[p] = L.part[p].heads ? static_cast<long long>(L.part[p].rows) * L.part[p].heads + 1 : 0;
        want[p] = work[p] ? (L.part[p].rows + rows_a_block - 1) / rows_a_block : 0;
        if (work[p] && want[p] < 1) want[p] = 1;
    }
    if (want[0] + want[1] > most) {
        long long q = static_cast<long long>(static_cast<double>(most) * work[0] / (work[0] + work[1]));
        if (q < 1) q = 1;
        if (work[1] && q > most - 1) q = most - 1;
        if (q > want[0]) q = want[0];
        want[0] = q;
        if (want[1] > most - q) want[1] = most - q;
    }
    L.q_blocks = static_cast<int>(want[0]);
    blocks = static_cast<int>(want[0] + want[1]);
}

template <typename T, Mode MODE>
cudaError_t launch_layout(RotaryLaunch L, int vec, int &blocks, cudaStream_t stream) {
    const int half = L.rotary_dim / 2;
    if (half % 8 == 0 && reinterpret_cast<uintptr_t>(L.table) % 16 == 0) {
        using S = Stream<T, MODE>;
        size_t smem = kStreamWarps * S::warp_bytes(half);
        const size_t sums = kStreamWarps * 32 * 16 * sizeof(float);   // the gain's partial sums
        if (MODE == kNormGrad && smem < sums) smem = sums;
        const int fit = static_cast<int>(200 * 1024 / smem), cap = MODE == kNormGrad ? 4 : 6;
        split(L, kStreamWarps, L.sm_count * (fit < cap ? fit : cap), blocks);
        auto kernel = L.interleaved ? stream_kernel<T, true, MODE> : stream_kernel<T, false, MODE>;
        if (smem > 48 * 1024) {   // more than a kernel has without asking
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e != cudaSuccess) return e;
        }
        kernel<<<blocks, kStreamWarps * 32, smem, stream>>>(L);
    } else {
        split(L, kWarps, rotary_blocks(L.sm_count), blocks);
        if (L.interleaved)
            heads_kernel<T, 8, true, MODE><<<blocks, kThreads, 0, stream>>>(L);
        else if (vec >= 2)
            heads_kernel<T, 2, false, MODE><<<blocks, kThreads, 0, stream>>>(L);
        else
            heads_kernel<T, 1, false, MODE><<<blocks, kThreads, 0, stream>>>(L);
    }
    if (MODE == kNormGrad && (L.part[0].gain_partials || L.part[1].gain_partials))
        gain_sum_kernel<<<dim3((L.head_dim + 31) / 32, L.part[1].heads ? 2 : 1), 1024, 0, stream>>>(L, blocks);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_mode(const RotaryLaunch &L, int vec, int &blocks, cudaStream_t stream) {
    if (!L.norm) return launch_layout<T, kRotate>(L, vec, blocks, stream);
    if (!L.backward) return launch_layout<T, kNorm>(L, vec, blocks, stream);
    return launch_layout<T, kNormGrad>(L, vec, blocks, stream);
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
    // Chunks of 8 where both halves of the rotated part start on a multiple of 8 (and the table's rows on 16
    // bytes), else the widest that do.
    const int half = L.rotary_dim / 2;
    const bool whole = half % 8 == 0 && reinterpret_cast<uintptr_t>(L.table) % 16 == 0;
    const int vec = L.interleaved || whole ? 8 : half % 2 == 0 ? 2 : 1;
    const int slots = (L.head_dim + 2 * vec - 1) / (2 * vec);
    const int spl = vec >= 4 ? 1 : 4 / vec;
    L.lph_log2 = 0;
    while ((spl << L.lph_log2) < slots) ++L.lph_log2;
    if (static_cast<long long>(L.part[0].rows) + L.part[1].rows > kFewRows) {
        const cudaError_t e = cudaMemsetAsync(L.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    int blocks = 0;
    if (L.dtype == CLI_BF16) return launch_mode<__nv_bfloat16>(L, vec, blocks, stream);
    if (L.dtype == CLI_F16) return launch_mode<__half>(L, vec, blocks, stream);
    return launch_mode<float>(L, vec, blocks, stream);
}

}  // namespace cli
