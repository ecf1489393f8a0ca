// Kernels of layer norm over rows of 1 to 16384 elements, alone and where a
// dropped-out branch joins a residual stream; norm.cu launches them.
//
// Mathematics (see include/cli.h).  A row z is x itself, or residual + the
// branch through its mask.  The mean m comes from one sum, and the variance
// from the deviations d = z - m, whose own sum corrects both: with
// e = mean d, n = (d - e) r and v = mean d^2 - e^2, so that a mean far from 0
// costs no digits of the spread around it.  The gradient, t = gain d_y:
//     d_z = r (t - mean t - n mean(t n)),  d_gain = sum d_y n,  d_bias = sum d_y.
#pragma once

#include "rows.cuh"

namespace cli {
namespace norm {

using namespace rows;

// Where a thread's chunks of a row lie, and how many elements of each there are.
template <int E>
__device__ __forceinline__ int column_of(const Team &team, int j) { return (j * team.lanes + team.lane) * E; }
template <int E>
__device__ __forceinline__ int elements_of(int at, int width) { return min(max(width - at, 0), E); }

// 1 / sqrt(variance + epsilon) of `width` deviations that sum to `sum` and whose squares sum to `squares`; e: their mean.
__device__ __forceinline__ float deviation(float sum, float squares, float inv_width, float epsilon, float &e) {
    e = sum * inv_width;
    return rsqrtf(fmaxf(squares * inv_width - e * e, 0.0f) + epsilon);
}

// The most threads of a block: one team of the widest rows where it has several warps.
template <int E, int C> constexpr int kForwardThreads = C < 4 ? 256 : static_cast<int>(kMaxRowWidth) / (E * C);

// T: type of the branch and the output.  S: the stream's.  E: elements of a
// chunk; C: chunks of a row that a thread has; R: rows that a team takes at a
// time.  BRANCH: a branch joins.
template <typename T, typename S, int E, int C, int R, bool BRANCH>
__global__ void __launch_bounds__(kForwardThreads<E, C>) forward_kernel(const __grid_constant__ NormLaunch P) {
    extern __shared__ float scratch[];   // teams of several warps: two of 64 floats each
    const Team team(P.lanes);
    const int width = P.width;
    const bool whole = P.whole;
    float *sums = scratch + team.id * 128;
    const Mask mask(P.mask);
    const int first = team.lanes < 32 ? team.index - (threadIdx.x & 31) / team.lanes : team.index;   // of the warp
    for (long long base = 0; base + static_cast<long long>(first) * R < P.rows; base += static_cast<long long>(team.count) * R) {
        const long long row0 = base + static_cast<long long>(team.index) * R;
        float v[R][C][E];
        {
            Chunk<S, E> in[R][C];
            Chunk<T, E> x[BRANCH ? R : 1][C];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const int at = column_of<E>(team, j), n = row0 + r < P.rows ? elements_of<E>(at, width) : 0;
                    take(in[r][j], static_cast<const S *>(P.in) + (row0 + r) * P.in_row + at, n, whole);
                    if constexpr (BRANCH) take(x[r][j], static_cast<const T *>(P.branch) + (row0 + r) * P.branch_row + at, n, whole);
                }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    in[r][j].floats(v[r][j]);
                    if constexpr (BRANCH) {
                        const int at = column_of<E>(team, j), n = row0 + r < P.rows ? elements_of<E>(at, width) : 0;
                        float f[E];
                        x[r][j].floats(f);
                        mask.apply<E>(f, static_cast<uint32_t>(row0 + r), at);
#pragma unroll
                        for (int i = 0; i < E; ++i) v[r][j][i] += f[i];
                        if (P.sum) {
                            Chunk<S, E> c;
                            c.set(v[r][j]);
                            put(c, static_cast<S *>(P.sum) + (row0 + r) * P.sum_row + at, n, whole);
                        }
                    }
                }
        }
        float s[R], s2[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) s[r] += v[r][j][i];   // 0 past the row's end
        }
        team.sum<R>(s, sums);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float m = s[r] * P.inv_width;
            s2[2 * r] = s2[2 * r + 1] = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int n = elements_of<E>(column_of<E>(team, j), width);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float d = (E == 8 ? n > 0 : i < n) ? v[r][j][i] - m : 0.0f;
                    v[r][j][i] = d;
                    s2[2 * r] += d;
                    s2[2 * r + 1] = fmaf(d, d, s2[2 * r + 1]);
                }
            }
        }
        team.sum<2 * R>(s2, sums + 64);
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = deviation(s2[2 * r], s2[2 * r + 1], P.inv_width, P.epsilon, s2[2 * r]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int at = column_of<E>(team, j);
            float gain[E], bias[E];
            vector_of<E>(P.gain, at, width, 1.0f, gain);
            vector_of<E>(P.bias, at, width, 0.0f, bias);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int n = row0 + r < P.rows ? elements_of<E>(at, width) : 0;
                float y[E];
#pragma unroll
                for (int i = 0; i < E; ++i) y[i] = fmaf((v[r][j][i] - s2[2 * r]) * s[r], gain[i], bias[i]);
                Chunk<T, E> c;
                c.set(y);
                put(c, static_cast<T *>(P.out) + (row0 + r) * P.out_row + at, n, whole);
            }
        }
    }
}

// THREADS: the most of a block.
template <typename T, typename S, int E, int C, int THREADS, bool BRANCH>
__global__ void __launch_bounds__(THREADS) backward_kernel(const __grid_constant__ NormLaunch P) {
    extern __shared__ float scratch[];   // teams of several warps: two of 128 floats each; then the block's sums
    const Team team(P.lanes);
    const int width = P.width;
    const bool whole = P.whole;
    float *sums = scratch + team.id * 256;
    const Mask mask(P.mask);
    float gain[C][E], d_gain[C][E], d_bias[C][E];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        vector_of<E>(P.gain, column_of<E>(team, j), width, 1.0f, gain[j]);
#pragma unroll
        for (int i = 0; i < E; ++i) d_gain[j][i] = d_bias[j][i] = 0.0f;
    }
    const int first = team.lanes < 32 ? team.index - (threadIdx.x & 31) / team.lanes : team.index;   // of the warp
    for (long long base = 0; base + first < P.rows; base += team.count) {
        const long long row = base + team.index;
        const bool on = row < P.rows;
        Chunk<S, E> z[C], d_sum[BRANCH ? C : 1];
        Chunk<T, E> d_y[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int at = column_of<E>(team, j), n = on ? elements_of<E>(at, width) : 0;
            take(z[j], static_cast<const S *>(P.in) + row * P.in_row + at, n, whole);
            take(d_y[j], static_cast<const T *>(P.d_out) + row * P.d_out_row + at, n, whole);
            if constexpr (BRANCH) {
                if (P.d_sum)
                    take(d_sum[j], static_cast<const S *>(P.d_sum) + row * P.d_sum_row + at, n, whole);
                else
                    d_sum[j].clear();
            }
        }
        float s[1] = {0.0f}, s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float v[E];
            z[j].floats(v);
#pragma unroll
            for (int i = 0; i < E; ++i) s[0] += v[i];
        }
        team.sum<1>(s, sums);
        const float m = s[0] * P.inv_width;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int n = elements_of<E>(column_of<E>(team, j), width);
            float v[E], g[E];
            z[j].floats(v);
            d_y[j].floats(g);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float d = (E == 8 ? n > 0 : i < n) ? v[i] - m : 0.0f, t = g[i] * gain[j][i];
                s4[0] += d;
                s4[1] = fmaf(d, d, s4[1]);
                s4[2] += t;
                s4[3] = fmaf(t, d, s4[3]);
            }
        }
        team.sum<4>(s4, sums + 128);
        float e;
        const float r = deviation(s4[0], s4[1], P.inv_width, P.epsilon, e);
        const float mean_t = s4[2] * P.inv_width, mean_tn = (s4[3] * P.inv_width - e * mean_t) * r;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int at = column_of<E>(team, j), n = on ? elements_of<E>(at, width) : 0;
            float v[E], g[E], dz[E];
            z[j].floats(v);
            d_y[j].floats(g);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float norm = ((v[i] - m) - e) * r;
                if (on) {
                    d_gain[j][i] = fmaf(g[i], norm, d_gain[j][i]);
                    d_bias[j][i] += g[i];
                }
                dz[i] = r * (g[i] * gain[j][i] - mean_t - norm * mean_tn);
            }
            if constexpr (BRANCH) {
                float more[E];
                d_sum[j].floats(more);
#pragma unroll
                for (int i = 0; i < E; ++i) dz[i] += more[i];
            }
            Chunk<S, E> c;
            c.set(dz);
            put(c, static_cast<S *>(P.d_in) + row * P.d_in_row + at, n, whole);
            if constexpr (BRANCH) {
                if (P.d_branch) {
                    mask.apply<E>(dz, static_cast<uint32_t>(row), at);
                    Chunk<T, E> b;
                    b.set(dz);
                    put(b, static_cast<T *>(P.d_branch) + row * P.d_branch_row + at, n, whole);
                }
            }
        }
    }
    if (!P.partials) return;
    // The block's sums: its teams' in their order.
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *to = P.partials + (static_cast<size_t>(which) * gridDim.x + blockIdx.x) * width;
        if (team.in_block > 1) {
            __syncthreads();
            const int slot = C * E * team.lanes;   // of a team
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) scratch[team.id * slot + column_of<E>(team, j) + i] = which ? d_bias[j][i] : d_gain[j][i];
            __syncthreads();
            for (int c = threadIdx.x; c < width; c += blockDim.x) {
                float t = 0.0f;
                for (int k = 0; k < team.in_block; ++k) t += scratch[k * slot + c];
                to[c] = t;
            }
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int c = column_of<E>(team, j) + i;
                    if (c < width) to[c] = which ? d_bias[j][i] : d_gain[j][i];
                }
        }
    }
}

// The sums of the blocks' partials, 32 columns a block and a fixed share of the rows a warp.
static __global__ void __launch_bounds__(1024) gain_kernel(const __grid_constant__ NormLaunch P, int blocks) {
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float *to = blockIdx.y ? P.d_bias : P.d_gain;
    if (!to) return;
    const float *from = P.partials + static_cast<size_t>(blockIdx.y) * blocks * P.width;
    __shared__ float sums[32][33];
    float t = 0.0f;
    if (c < P.width) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += 32) t += from[static_cast<size_t>(b) * P.width + c];
    }
    sums[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < P.width) {
        t = 0.0f;
        for (int w = 0; w < 32; ++w) t += sums[w][lane];
        to[c] = t;
    }
}

// ----------------------------------------------------------------------------
// launches of one pair of types
// ----------------------------------------------------------------------------

inline int lanes_of(int chunks, int each) {   // of a team whose lanes have `each` chunks at most
    const int need = (chunks + each - 1) / each;
    if (need > 32) return (need + 31) / 32 * 32;
    int lanes = 1;
    while (lanes < need) lanes *= 2;
    return lanes;
}

template <typename T, typename S, int E, int C, int R, bool BRANCH>
cudaError_t forward(NormLaunch L, cudaStream_t stream) {
    L.lanes = lanes_of((L.width + E - 1) / E, C);
    const int threads = L.lanes > 256 ? L.lanes : 256 / L.lanes * L.lanes, teams = threads / L.lanes;
    const long long want = (L.rows + static_cast<long long>(teams) * R - 1) / (static_cast<long long>(teams) * R);
    const long long most = 8ll * L.sm_count;
    const size_t smem = L.lanes > 32 ? teams * 128 * sizeof(float) : 0;
    forward_kernel<T, S, E, C, R, BRANCH><<<static_cast<unsigned>(want < most ? want : most), threads, smem, stream>>>(L);
    return cudaGetLastError();
}

template <typename T, typename S, int E, bool BRANCH>
cudaError_t forward(const NormLaunch &L, cudaStream_t stream) {
    const int chunks = (L.width + E - 1) / E;
    if (chunks <= 32) return forward<T, S, E, 1, 4, BRANCH>(L, stream);
    if (chunks <= 64) return forward<T, S, E, 2, 2, BRANCH>(L, stream);
    return forward<T, S, E, 4, 1, BRANCH>(L, stream);
}

template <typename T, typename S, int E, int C, int THREADS, bool BRANCH>
cudaError_t backward_of(NormLaunch L, cudaStream_t stream) {
    L.lanes = lanes_of((L.width + E - 1) / E, C);
    const int threads = L.lanes > 256 ? L.lanes : 256 / L.lanes * L.lanes, teams = threads / L.lanes;
    long long blocks = (L.rows + teams - 1) / teams, most = 2ll * L.sm_count;
    blocks = blocks < 1 ? 1 : blocks < most ? blocks : most;
    size_t smem = L.lanes > 32 ? teams * 256 * sizeof(float) : 0;
    if (teams > 1) {
        const size_t sums = static_cast<size_t>(threads) * C * E * sizeof(float);
        smem = smem > sums ? smem : sums;
    }
    backward_kernel<T, S, E, C, THREADS, BRANCH><<<static_cast<unsigned>(blocks), threads, smem, stream>>>(L);
    if (!L.partials) return cudaGetLastError();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(gain_kernel, dim3((L.width + 31) / 32, 2), 1024, 0, stream, L, static_cast<int>(blocks));
}

template <typename T, typename S, int E, bool BRANCH>
cudaError_t backward_of(const NormLaunch &L, cudaStream_t stream) {
    constexpr int kEach = 16 / E;   // chunks of a thread
    const int chunks = (L.width + E - 1) / E;
    if (chunks <= 32) return backward_of<T, S, E, 1, 256, BRANCH>(L, stream);
    if (chunks <= 512 * kEach) return backward_of<T, S, E, kEach, 512, BRANCH>(L, stream);
    return backward_of<T, S, E, kEach, 1024, BRANCH>(L, stream);
}

template <typename T, typename S, int E>
cudaError_t launch_chunks(const NormLaunch &L, cudaStream_t stream) {
    if (L.backward) return L.join ? backward_of<T, S, E, true>(L, stream) : backward_of<T, S, E, false>(L, stream);
    return L.join ? forward<T, S, E, true>(L, stream) : forward<T, S, E, false>(L, stream);
}

// One pair of types a source file (norm_*.cu).
template <typename T, typename S>
cudaError_t launch_types(const NormLaunch &L, cudaStream_t stream) {
    return L.wide ? launch_chunks<T, S, 8>(L, stream) : launch_chunks<T, S, 4>(L, stream);
}

}  // namespace norm
}  // namespace cli
