// Kernels of layer norm over rows of 1 to 16384 elements, alone and where a
// dropped-out branch joins a residual stream, and their launches for one pair
// of types (norm_*.cu).
//
// Mathematics (see include/cli.h).  A row z is x itself, or residual + the
// branch through its mask.  The mean m comes from one sum, and the variance
// from the deviations d = z - m, whose own sum corrects both: with
// e = mean d, n = (d - e) r and v = mean d^2 - e^2, so that a mean far from 0
// costs no digits of the spread around it.  The gradient, t = gain d_y:
//     d_z = r (t - mean t - n mean(t n)),  d_gain = sum d_y n,  d_bias = sum d_y.
//
// Work.  A team takes a row, or R of them: 2^k lanes of a warp, or whole
// warps, each thread NE elements of a row in chunks of E.  Teams walk the rows
// at the grid's stride, and what a thread needs some steps from now is on its
// way into its own places in shared memory (rows.cuh).
//
// Bound: HBM, where an element's instructions leave it time.  The norm of
// 270336 x 1024 in bf16 takes 14 an element and 171 us (6.5 TB/s, 95% of the
// copy's rate); the join of as many into an fp32 stream 31 and 509 us (6.5 TB/s).
// The gradients wait: 23 instructions an element and 146 us over 131072 x 1024
// (5.5 TB/s), the join's 40 and 257 us (5.2 TB/s), with 53 to 57% of the issue
// slots used.  16 warps an SM, which is what a thread's 128 registers allow (the
// columns' sums, the row and the generator), do not cover the instruction
// before, shared memory and the team's barrier.  Over 8192 x 8192 without the
// stream's gradient, where the one team of an SM meets at that barrier and has
// fewer bytes an element to wait for, the join's takes 148 us (3.6 TB/s).
#pragma once

#include "rows.cuh"

namespace cli {
namespace norm {

using namespace rows;

constexpr int kThreads = 512;   // the most of a block: one team of the widest rows

// A thread's chunks lie a constant apart unless its team is a part of a warp (SUB).
template <typename T, int E, bool SUB, int MOVES>
using RowLayout = Layout<T, E, MOVES, SUB ? 0 : 32>;
template <typename L, int NE, bool SUB>
__device__ __forceinline__ L layout_of(const Team &team) {
    return SUB ? L(team.lanes, team.lane, 0) : L(32, team.lane & 31, (team.lane >> 5) * (32 * NE));
}

// 1 / sqrt(variance + epsilon) of `width` deviations that sum to `sum` and whose squares sum to `squares`; e: their mean.
// 0 where the squares pass fp32's range: their mean's own square may pass it too, and infinity less infinity is no variance
// (nor does fmaxf let the NaN through).
__device__ __forceinline__ float deviation(float sum, float squares, float inv_width, float epsilon, float &e) {
    e = sum * inv_width;
    const float r = rsqrtf(fmaxf(squares * inv_width - e * e, 0.0f) + epsilon);
    return squares < INFINITY ? r : 0.0f;   // of a NaN too: e, and with it the row, is NaN then
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// v - m for a chunk's elements that are there; the others are 0 and stay so.
template <int E, typename L>
__device__ __forceinline__ void deviations(float2 (&v)[E / 2], float m, uint32_t there) {
#pragma unroll
    for (int i = 0; i < E; i += 2)
        v[i / 2] = __fadd2_rn(v[i / 2], make_float2(there >> (i / L::kPiece) & 1u ? -m : 0.0f, there >> ((i + 1) / L::kPiece) & 1u ? -m : 0.0f));
}

// What a team's lanes need of the mask and the gain in every row, in shared memory: as many registers would displace the
// row.  A lane's blocks and gains lie beside the other lanes', the block's teams share them.
//   keys    3 x 16 bytes: a and b of rounds 4 to 9
//   blocks  [NE / 4][lanes of a team] x 16 bytes, with BLOCKS; else they are worked out again in each row
//   gains   [NE / 4][lanes of a team] x 16 bytes, with GAIN
template <int E, int NE, bool BLOCKS, bool GAIN>
struct Table {
    uint32_t at, blocks, gains, step, row_word, a3;   // step: from a lane's 16 bytes to its next
    Seed seed;
    static __host__ __device__ uint32_t bytes(int lanes) { return 48 + ((BLOCKS ? 1u : 0u) + (GAIN ? 1u : 0u)) * (NE / 4) * lanes * 16; }
    Table() = default;
    template <typename L>
    __device__ __forceinline__ Table(uint32_t base, const NormLaunch &P, const Team &team, const L &layout)
        : at(base), blocks(base + 48 + team.lane * 16), gains(blocks + (BLOCKS ? NE / 4 : 0) * team.lanes * 16),
          step(team.lanes * 16), seed(P.mask) {
        row_word = seed.row_word(), a3 = seed.a(3);
        if (P.mask.least && threadIdx.x < 3) {
            const int i = 4 + 2 * threadIdx.x;
            st_shared_v4(at + threadIdx.x * 16, seed.a(i), seed.b(i), seed.a(i + 1), seed.b(i + 1));
        }
        if (team.id == 0) {
#pragma unroll
            for (int j = 0; j < NE / E; ++j) {
                float2 gain[E / 2];
                if (GAIN) layout.vector(P.gain, j, P.width, 1.0f, gain);
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    const uint32_t to = (j * (E / 4) + i) * step;
                    if (BLOCKS && P.mask.least) {
                        const Block b(seed, P.mask.site, layout.first_of(j, i));
                        st_shared_v4(blocks + to, b.d, b.f, b.g, b.h);
                    }
                    if (GAIN)
                        st_shared_v4(gains + to, __float_as_uint(gain[2 * i].x), __float_as_uint(gain[2 * i].y),
                                     __float_as_uint(gain[2 * i + 1].x), __float_as_uint(gain[2 * i + 1].y));
                }
            }
        }
        __syncthreads();
    }
    __device__ __forceinline__ uint4 two(int i) const { return shared16(at + (i - 4) * 8); }
    __device__ __forceinline__ void gain(int j, float2 (&v)[E / 2]) const {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const uint4 u = shared16(gains + (j * (E / 4) + i) * step);
            v[2 * i] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
            v[2 * i + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        }
    }
    // Chunk j of a row through the mask.
    template <typename L>
    __device__ __forceinline__ void mask(const L &layout, const MaskLaunch &m, float2 (&v)[E / 2], uint32_t row, int j) const {
        if (!m.least) return;
        Block b[E / 4];
        uint4 r[E / 4];
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            if constexpr (BLOCKS) {
                const uint4 u = shared16(blocks + (j * (E / 4) + i) * step);
                b[i].d = u.x, b[i].f = u.y, b[i].g = u.z, b[i].h = u.w;
            } else {
                b[i] = Block(seed, m.site, layout.first_of(j, i));
            }
        }
        draw(b, *this, product(kMul0, row ^ row_word), r);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) hand_round(layout, r[i]);
        keep<E>(v, r, m.least, m.scale);
    }
};

// Waits until all but the last `ahead` of the thread's groups of copies are there.
__device__ __forceinline__ void wait_copies(int ahead) {
    switch (ahead) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

// T: type of the branch and the output.  S: the stream's.  E: elements of a
// chunk; NE: of a row that a thread has; R: rows that a team takes at a time.
// BRANCH: a branch joins.  PIPE: the rows' means come with the sums of the rows
// before them, so that a team meets once a step and not twice, which pays in
// teams of more than two warps (bf16, shares of the copy's rate: 2048 elements
// 0.77 -> 0.81, 4096 0.74 -> 0.79, 8192 0.66 -> 0.72).
template <typename T, typename S, int E, int NE, bool SUB, int R, bool BRANCH, int MOVES, bool PIPE>
__global__ void __launch_bounds__(kThreads) forward_kernel(const __grid_constant__ NormLaunch P) {
    constexpr int C = NE / E;
    const int stages = P.stages;
    constexpr bool kHold = NE <= 16;   // the gain and the bias stay in registers
    extern __shared__ __align__(16) float scratch[];   // teams of several warps: R * 112 floats each; then the feeds
    const Team team(P.lanes);
    float *sums = scratch + team.id * R * 112;
    uint32_t places = smem_u32(scratch) + (team.lanes > 32 ? team.in_block * R * 448 : 0);
    using L = RowLayout<T, E, SUB, MOVES>;
    using Tab = Table<E, NE, true, false>;
    const L layout = layout_of<L, NE, SUB>(team);
    const uint32_t table_at = places;
    if (BRANCH) places += Tab::bytes(team.lanes);
    Feed<S, L, E, C * R, MOVES, true> in(places, stages);
    Feed<T, L, E, C * R, MOVES, true> branch(places + stages * NE * R * static_cast<int>(sizeof(S)) * blockDim.x, BRANCH ? stages : 0);
    const uint32_t there = layout.template there<C>(P.width);
    const uint32_t rows = static_cast<uint32_t>(P.rows), stride = team.count * R, mine = team.index * R;
    const uint32_t first = team.first * R;   // of the warp

    // The copies of a step, rows base + mine to base + mine + R - 1.
    auto copy = [&](uint32_t base, int stage) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = base + mine + r;
            const uint32_t on = row < rows ? there : 0u;
            const S *from = static_cast<const S *>(P.in) + row * P.in_row + layout.column;
            const T *x = static_cast<const T *>(P.branch) + row * P.branch_row + layout.column;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                in.copy(layout, stage, r * C + j, from + layout.chunk(j), on >> (j * L::kPieces));
                if constexpr (BRANCH) branch.copy(layout, stage, r * C + j, x + layout.chunk(j), on >> (j * L::kPieces));
            }
        }
    };
    auto settle = [&](int stage) {
        in.settle(stage);
        if constexpr (BRANCH) branch.settle(stage);
    };
    constexpr bool kHeld = MOVES == kHalves && (BRANCH || sizeof(S) == 2);
    const int ahead = kHeld && stages > 1 ? 1 : stages - 1;   // steps
    for (int k = 0; k < ahead; ++k) {
        copy(k * stride, k);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // While these are on their way, what the rows share.
    const Tab table = [&] {
        if constexpr (BRANCH) return Tab(table_at, P, team, layout);
        else return Tab();
    }();
    float2 gain[kHold ? C : 1][E / 2], bias[kHold ? C : 1][E / 2];
#pragma unroll
    for (int j = 0; j < C && kHold; ++j) {
        layout.vector(P.gain, j, P.width, 1.0f, gain[j]);
        layout.vector(P.bias, j, P.width, 0.0f, bias[j]);
    }
    if (kHeld && ahead) settle(0);
    auto sums_of = [&](int from, float *to) {   // a thread's share of the sums
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 sum = both(0.0f);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float2 z[E / 2];
                in.floats(from, r * C + j, z);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) sum = __fadd2_rn(sum, z[i]);
            }
            to[r] = sum.x + sum.y;
        }
    };
    float s[R];   // the rows' sums, later what their deviations are divided by
    if constexpr (PIPE) {
        wait_copies(ahead - 1);
        sums_of(0, s);
        team.sum<R, !SUB>(s, sums);
    }
    int stage = 0, parity = 0;
    for (uint32_t base = 0; base + first < rows; base += stride) {
        const int next = stage + ahead >= stages ? stage + ahead - stages : stage + ahead;
        copy(base + ahead * stride, next);   // what was there was used up a step ago
        asm volatile("cp.async.commit_group;" ::: "memory");
        wait_copies(PIPE ? ahead - 1 : ahead);
        if (kHeld && !ahead) settle(stage);
        float2 v[R][C][E / 2];
        float s2[PIPE ? 3 * R : 2 * R];   // of the deviations and of their squares; of the next rows
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = base + mine + r;
            const uint32_t on = row < rows ? there : 0u;
            S *total = static_cast<S *>(P.sum) + row * P.sum_row + layout.column;
            float2 sum = both(0.0f);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                in.floats(stage, r * C + j, v[r][j]);
                if constexpr (BRANCH) {
                    float2 f[E / 2];
                    branch.floats(stage, r * C + j, f);
                    table.mask(layout, P.mask, f, row, j);
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) v[r][j][i] = __fadd2_rn(v[r][j][i], f[i]);
                    if (P.sum) {
                        Chunk<S, E> c;
                        c.set(v[r][j]);
                        layout.store(c, total + layout.chunk(j), on >> (j * L::kPieces));
                    }
                }
#pragma unroll
                for (int i = 0; i < E / 2; ++i) sum = __fadd2_rn(sum, v[r][j][i]);   // 0 past the row's end
            }
            if constexpr (!PIPE) s[r] = sum.x + sum.y;
        }
        if constexpr (!PIPE) team.sum<R, !SUB>(s, sums);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float m = s[r] * P.inv_width;
            float2 sum = both(0.0f), squares = sum;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                deviations<E, L>(v[r][j], m, there >> (j * L::kPieces));
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    sum = __fadd2_rn(sum, v[r][j][i]);
                    squares = __ffma2_rn(v[r][j][i], v[r][j][i], squares);
                }
            }
            s2[2 * r] = sum.x + sum.y;
            s2[2 * r + 1] = squares.x + squares.y;
        }
        if constexpr (PIPE) sums_of(stage + 1 == stages ? 0 : stage + 1, s2 + 2 * R);
        team.sum<PIPE ? 3 * R : 2 * R, !SUB>(s2, sums + R * 16 + parity * R * 48);
        if constexpr (PIPE) parity ^= 1;   // two places, which steps alternate between
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = deviation(s2[2 * r], s2[2 * r + 1], P.inv_width, P.epsilon, s2[2 * r]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if constexpr (!kHold) {
                layout.vector(P.gain, j, P.width, 1.0f, gain[0]);
                layout.vector(P.bias, j, P.width, 0.0f, bias[0]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t row = base + mine + r;
                const float2 scale = both(s[r]), shift = both(-s2[2 * r] * s[r]);
                float2 y[E / 2];
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    y[i] = __ffma2_rn(__ffma2_rn(v[r][j][i], scale, shift), gain[kHold ? j : 0][i], bias[kHold ? j : 0][i]);
                Chunk<T, E> c;
                c.set(y);
                layout.store(c, static_cast<T *>(P.out) + row * P.out_row + layout.column + layout.chunk(j), row < rows ? there >> (j * L::kPieces) : 0u);
            }
        }
        if constexpr (PIPE) {
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = s2[2 * R + r];
        }
        if (kHeld && ahead) settle(next);
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Where a backward call's gains are: in registers, or read again in each row from shared memory, or (where that is full of
// stages) from global memory.
enum Gains { kHeldGain, kSharedGain, kGlobalGain };
template <typename S, int NE, bool BRANCH>
constexpr Gains kGains = NE > 8 && sizeof(S) == 2 && (BRANCH || NE > 16) ? kSharedGain : NE <= 16 ? kHeldGain : kGlobalGain;

// Where the blocks are kept for the mask: not beside the widest rows of fp32, which leave no room.
template <typename T, int NE, bool BRANCH> constexpr bool kBlocks = BRANCH && !(NE == 32 && sizeof(T) == 4);

// Where a row's mean comes with the sums of the row before it, so that a team meets once a row (the join's gradient over
// 131072 x 1024 in bf16: 284 -> 259 us, over 8192 x 8192 204 -> 148): with three stages, for which there is room.
template <typename T, typename S, int NE, bool BRANCH, int MOVES>
constexpr bool kPiped = !(MOVES == kHalves && sizeof(T) == 2) &&
                        (NE == 8 || (NE == 16 && !(BRANCH && sizeof(S) == 4)) || (NE == 24 && !BRANCH));

template <typename T, typename S, int E, int NE, bool SUB, bool BRANCH, int MOVES>
__global__ void __launch_bounds__(kThreads) backward_kernel(const __grid_constant__ NormLaunch P) {
    constexpr int C = NE / E;
    constexpr bool kHold = NE <= 16;   // the row's deviations stay in registers
    constexpr Gains kGain = kGains<S, NE, BRANCH>;
    const int stages = P.stages;
    extern __shared__ __align__(16) float scratch[];   // teams of several warps: 176 floats each; then the table and the feeds.  At the end, the block's sums
    const Team team(P.lanes);
    float *sums = scratch + team.id * 176;
    uint32_t places = smem_u32(scratch) + (team.lanes > 32 ? team.in_block * 704 : 0);
    using L = RowLayout<T, E, SUB, MOVES>;
    using Tab = Table<E, NE, kBlocks<T, NE, BRANCH>, kGain == kSharedGain>;
    const L layout = layout_of<L, NE, SUB>(team);
    const Tab table = [&] {
        if constexpr (BRANCH || kGain == kSharedGain) return Tab(places, P, team, layout);
        else return Tab();
    }();
    if (BRANCH || kGain == kSharedGain) places += Tab::bytes(team.lanes);
    Feed<S, L, E, C, MOVES, false> in(places, stages);
    places += stages * NE * static_cast<int>(sizeof(S)) * blockDim.x;
    Feed<T, L, E, C, MOVES, false> d_out(places, stages);
    places += stages * NE * static_cast<int>(sizeof(T)) * blockDim.x;
    Feed<S, L, E, C, MOVES, false> d_sum(places, BRANCH ? stages : 0);
    const uint32_t there = layout.template there<C>(P.width);
    float2 gain[kGain == kHeldGain ? C : 1][E / 2], d_gain[C][E / 2], d_bias[C][E / 2];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        if constexpr (kGain == kHeldGain) layout.vector(P.gain, j, P.width, 1.0f, gain[j]);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) d_gain[j][i] = d_bias[j][i] = both(0.0f);
    }
    const uint32_t rows = static_cast<uint32_t>(P.rows), stride = team.count, mine = team.index, first = team.first;

    auto copy = [&](uint32_t base, int stage) {
        const uint32_t row = base + mine;
        const uint32_t on = row < rows ? there : 0u;
        const S *z = static_cast<const S *>(P.in) + row * P.in_row + layout.column;
        const T *g = static_cast<const T *>(P.d_out) + row * P.d_out_row + layout.column;
        const S *more = static_cast<const S *>(P.d_sum) + row * P.d_sum_row + layout.column;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t pieces = on >> (j * L::kPieces);
            in.copy(layout, stage, j, z + layout.chunk(j), pieces);
            d_out.copy(layout, stage, j, g + layout.chunk(j), pieces);
            if constexpr (BRANCH) d_sum.copy(layout, stage, j, more + layout.chunk(j), P.d_sum ? pieces : 0u);   // none: its places stay 0
        }
    };
    auto settle = [&](int stage) {
        in.settle(stage);
        d_out.settle(stage);
        if constexpr (BRANCH) d_sum.settle(stage);
    };
    constexpr bool kHeld = MOVES == kHalves;
    const int ahead = kHeld && stages > 1 ? 1 : stages - 1;   // steps
    for (int k = 0; k < ahead; ++k) {
        copy(k * stride, k);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (kHeld && ahead) settle(0);
    auto total_of = [&](int from) {   // a thread's
        float2 sum = both(0.0f);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float2 v[E / 2];
            in.floats(from, j, v);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) sum = __fadd2_rn(sum, v[i]);   // 0 past the row's end
        }
        return sum.x + sum.y;
    };
    auto mean_of = [&](int from) {
        float s[1] = {total_of(from)};
        team.sum<1, !SUB>(s, sums);
        return s[0] * P.inv_width;
    };
    constexpr bool kPipe = kPiped<T, S, NE, BRANCH, MOVES>;
    int stage = 0, parity = 0;
    float m = 0.0f;
    if constexpr (kPipe) {
        wait_copies(ahead - 1);
        m = mean_of(0);
    }
    for (uint32_t base = 0; base + first < rows; base += stride) {
        const int next = stage + ahead >= stages ? stage + ahead - stages : stage + ahead;
        copy(base + ahead * stride, next);   // what was there was used up a step ago
        asm volatile("cp.async.commit_group;" ::: "memory");
        wait_copies(kPipe ? ahead - 1 : ahead);
        if (kHeld && !ahead) settle(stage);
        const uint32_t row = base + mine;
        const bool on = row < rows;
        float2 d[kHold ? C : 1][E / 2];
        Chunk<T, E> dy[kHold ? C : 1];
        if constexpr (!kPipe) m = mean_of(stage);
        // A chunk's deviations and gradient: kept with kHold, else computed again where they are used.
        auto load = [&](int j) {
            in.floats(stage, j, d[kHold ? j : 0]);
            deviations<E, L>(d[kHold ? j : 0], m, there >> (j * L::kPieces));
            dy[kHold ? j : 0] = d_out.chunk(stage, j);
        };
        auto gain_of = [&](int j) -> const float2 (&)[E / 2] {
            if constexpr (kGain == kHeldGain) return gain[j];
            if constexpr (kGain == kSharedGain) table.gain(j, gain[0]);
            if constexpr (kGain == kGlobalGain) layout.vector(P.gain, j, P.width, 1.0f, gain[0]);
            return gain[0];
        };
        float s[kPipe ? 5 : 4];
        {
            float2 sum = both(0.0f), squares = sum, sum_t = sum, sum_td = sum;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                load(j);
                const int k = kHold ? j : 0;
                float2 g[E / 2];
                dy[k].floats(g);
                const float2 (&w)[E / 2] = gain_of(j);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    const float2 t = __fmul2_rn(g[i], w[i]);
                    sum = __fadd2_rn(sum, d[k][i]);
                    squares = __ffma2_rn(d[k][i], d[k][i], squares);
                    sum_t = __fadd2_rn(sum_t, t);
                    sum_td = __ffma2_rn(t, d[k][i], sum_td);
                }
            }
            s[0] = sum.x + sum.y, s[1] = squares.x + squares.y, s[2] = sum_t.x + sum_t.y, s[3] = sum_td.x + sum_td.y;
        }
        if constexpr (kPipe) s[4] = total_of(stage + 1 == stages ? 0 : stage + 1);
        team.sum<kPipe ? 5 : 4, !SUB>(s, sums + 16 + parity * 80);   // two places, which steps alternate between
        parity ^= 1;
        float e;
        const float r = deviation(s[0], s[1], P.inv_width, P.epsilon, e);
        // Where the squares pass the range, n and r are 0, whatever t and the deviations sum to.  (As `deviation` asks: with r itself
        // compared the gradient over 516 columns of bf16 runs at 0.52 of the copy's rate, and at 0.59 so.)
        const float mean_t = s[2] * P.inv_width, mean_tn = (s[1] < INFINITY ? s[3] * P.inv_width - e * mean_t : 0.0f) * r;
        const float2 scale = both(r), shift = both(-e * r), less = both(-r * mean_t), less_n = both(-r * mean_tn);
        if (SUB || on) {   // of a warp with several teams all lanes go on together, for the mask
            S *to = static_cast<S *>(P.d_in) + row * P.d_in_row + layout.column;
            T *to_x = static_cast<T *>(P.d_branch) + row * P.d_branch_row + layout.column;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                if constexpr (!kHold) load(j);
                const int k = kHold ? j : 0;
                const uint32_t pieces = on ? there >> (j * L::kPieces) : 0u;
                float2 v[E / 2], g[E / 2];
                dy[k].floats(g);
                const float2 (&w)[E / 2] = gain_of(j);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    const float2 norm = __ffma2_rn(d[k][i], scale, shift);
                    if (on) {
                        d_gain[j][i] = __ffma2_rn(g[i], norm, d_gain[j][i]);
                        d_bias[j][i] = __fadd2_rn(d_bias[j][i], g[i]);
                    }
                    v[i] = __ffma2_rn(__fmul2_rn(g[i], w[i]), scale, __ffma2_rn(norm, less_n, less));
                }
                if constexpr (BRANCH) {
                    d_sum.floats(stage, j, g);
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) v[i] = __fadd2_rn(v[i], g[i]);
                }
                Chunk<S, E> c;
                c.set(v);
                layout.store(c, to + layout.chunk(j), pieces);
                if constexpr (BRANCH) {
                    if (P.d_branch && (L::kPiece != E || pieces)) {   // warps whose lanes have none are spared the mask
                        table.mask(layout, P.mask, v, row, j);
                        Chunk<T, E> b;
                        b.set(v);
                        layout.store(b, to_x + layout.chunk(j), pieces);
                    }
                }
            }
        }
        if constexpr (kPipe) m = s[4] * P.inv_width;
        if (kHeld && ahead) settle(next);
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!P.d_gain && !P.d_bias) return;
    // The block's sums: its teams' in their order.  A block by itself has the gradients.
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *to = P.partials + (static_cast<size_t>(which) * gridDim.x + blockIdx.x) * P.width;
        if (!P.partials) to = which ? P.d_bias : P.d_gain;
        if (!to) continue;
        const int slot = NE * team.lanes;   // of a team
        __syncthreads();
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 v = which ? d_bias[j][i] : d_gain[j][i];
                scratch[team.id * slot + layout.element(j, 2 * i)] = v.x;
                scratch[team.id * slot + layout.element(j, 2 * i + 1)] = v.y;
            }
        __syncthreads();
        for (int c = threadIdx.x; c < P.width; c += blockDim.x) {
            float t = 0.0f;
            for (int k = 0; k < team.in_block; ++k) t += scratch[k * slot + c];
            to[c] = t;
        }
    }
}

// The sums of the blocks' partials, 32 columns a block and a fixed share of the rows a warp.  It is launched ahead, but starts
// when the last block of the gradient's kernel has ended, which does not let it start before.
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

inline int lanes_of(int width, int each) {   // of a team whose lanes have `each` elements at most: whole groups of 4
    const int need = (width + each - 1) / each;
    if (need > 32) return (need + 31) / 32 * 32;
    int lanes = 4;
    while (lanes < need) lanes *= 2;
    return lanes;
}

// Threads of a block: whole teams, 256 of them or the first number above that leaves fewer of an SM's 512 idle.
inline int threads_of(int lanes) {
    int best = lanes;
    for (int t = lanes; t <= 512; t += lanes)
        if (t / lanes <= 15 || lanes <= 32)   // there are 16 barriers
            if (best < 256 ? t <= 256 || 512 / t * t >= 512 / best * best : 512 / t * t > 512 / best * best) best = t;
    return best;
}

// A launch's shape, for `groups` of rows that a team takes at a time: `fixed` bytes of shared memory a block, and `stage`
// for each stage of its threads' places.  As many stages, up to 4 and one more than a team's steps, as leave an SM its 512
// threads of 128 registers; `least` at least, or if one block has no room for them, 1.
struct Shape {
    int stages;
    long long blocks;
    size_t smem;
    Shape(int threads, int teams, long long groups, int sm_count, size_t fixed, size_t stage, int least) {
        constexpr size_t kRoom = 227 * 1024, kBlock = 1024;   // of an SM; of which each block takes some
        const int most = 512 / threads;
        stages = 4;
        while (stages > least && most * (fixed + stages * stage + kBlock) > kRoom + kBlock) --stages;
        if (fixed + stages * stage > kRoom) stages = 1;
        const int fit = static_cast<int>((kRoom + kBlock) / (fixed + stages * stage + kBlock));
        const long long across = static_cast<long long>(fit < most ? fit : most) * sm_count, want = (groups + teams - 1) / teams;
        blocks = want < 1 ? 1 : want < across ? want : across;
        const long long steps = (want + blocks - 1) / blocks;
        if (stages > steps + 1 && stages > least) stages = steps + 1 > least ? static_cast<int>(steps) + 1 : least;
        smem = fixed + stages * stage;
    }
};

template <typename K>
cudaError_t allow(K kernel, size_t smem) {   // more shared memory than a kernel has without asking
    return smem > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) : cudaSuccess;
}

template <typename T, typename S, int E, int NE, bool SUB, int R, bool BRANCH, int MOVES>
cudaError_t forward(NormLaunch L, cudaStream_t stream) {
    L.lanes = lanes_of(L.width, NE);
    const int threads = threads_of(L.lanes), teams = threads / L.lanes;
    const Shape shape(threads, teams, (L.rows + R - 1) / R, L.sm_count,
                      (L.lanes > 32 ? teams * R * 448 : 0) + (BRANCH ? Table<E, NE, true, false>::bytes(L.lanes) : 0),
                      NE * R * (sizeof(S) + (BRANCH ? sizeof(T) : 0)) * threads, 1);
    L.stages = shape.stages;
    auto kernel = forward_kernel<T, S, E, NE, SUB, R, BRANCH, MOVES, false>;
    if constexpr (!BRANCH && !SUB && !(MOVES == kHalves && sizeof(S) == 2)) {
        if (L.lanes > 64 && shape.stages > 2) kernel = forward_kernel<T, S, E, NE, SUB, R, BRANCH, MOVES, true>;
    }
    const cudaError_t e = allow(kernel, shape.smem);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(shape.blocks), threads, shape.smem, stream>>>(L);
    return cudaGetLastError();
}

template <typename T, typename S, int E, int NE, bool SUB, bool BRANCH, int MOVES>
cudaError_t backward(NormLaunch L, cudaStream_t stream) {
    constexpr bool kShared = kGains<S, NE, BRANCH> == kSharedGain;
    L.lanes = lanes_of(L.width, NE);
    const int threads = threads_of(L.lanes), teams = threads / L.lanes;
    constexpr bool kPipe = kPiped<T, S, NE, BRANCH, MOVES>;
    const Shape shape(threads, teams, L.rows, L.sm_count,
                      (L.lanes > 32 ? teams * 704 : 0) + (BRANCH || kShared ? Table<E, NE, kBlocks<T, NE, BRANCH>, kShared>::bytes(L.lanes) : 0),
                      NE * (sizeof(S) * (BRANCH ? 2 : 1) + sizeof(T)) * threads, kPipe ? 3 : 1);
    if (kPipe && shape.stages < 3) return cudaErrorInvalidConfiguration;
    L.stages = shape.stages;
    const size_t sums = static_cast<size_t>(threads) * NE * sizeof(float), smem = shape.smem > sums ? shape.smem : sums;
    const long long blocks = (L.d_gain || L.d_bias) && !L.partials ? 1 : shape.blocks;
    auto kernel = backward_kernel<T, S, E, NE, SUB, BRANCH, MOVES>;
    cudaError_t e = allow(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(blocks), threads, smem, stream>>>(L);
    e = cudaGetLastError();
    if (e != cudaSuccess || !L.partials) return e;
    return launch_after(gain_kernel, dim3((L.width + 31) / 32, 2), 1024, 0, stream, L, static_cast<int>(blocks));
}

// How many elements of a row a thread has, and whether a team is a part of a warp: up to 256 elements (with eight a thread
// the norm runs at 0.75 of the copy's rate at 256 where it has 0.89 with sixteen, its gradient at 0.62 against 0.88).
// Sixteen leave it room for what the row and its columns need from one step to the next.  Measured for 16-bit rows, as
// shares of the copy's rate with 16 | 24 | 32:
//   norm            0.81 | 0.49 | 0.71 at 1024, 0.74 | 0.44 | 0.57 at 4096, 0.66 | 0.42 | 0.55 at 8192 (0.88, 0.78 and
//                   0.73 with sixteen as they are now)
//   its gradient    0.61 | 0.69 | 0.68 at 768, 0.74 | 0.52 | 0.67 at 1024, 0.69 | 0.65 | 0.63 at 1536, 0.63 | 0.64 | 0.68 at
//                   2048, 0.61 | 0.53 | 0.67 at 4096, 0.55 | 0.50 | 0.64 at 8192
//   join's gradient 0.67 | 0.75 | 0.55 at 768, 0.76 | 0.61 | 0.61 at 1024, 0.73 | 0.69 | 0.53 at 2048, 0.64 | 0.57 | 0.43 at
//                   8192
// The gradients' rule is that of rows in pieces as well, where its kernels spill up to 712 bytes a thread and are now the
// faster ones and now the slower (as the rule has it | with sixteen; bf16, halves and then words):
//   norm's gradient 0.24 | 0.23 at 517, 0.23 | 0.27 at 1537, 0.18 | 0.27 at 2051, 0.26 | 0.27 at 3001, 0.21 | 0.18 at 4099,
//                   0.25 | 0.27 at 8191; 0.45 | 0.41 at 1538, 0.36 | 0.43 at 2050, 0.39 | 0.33 at 4098
//   join's gradient 0.22 | 0.19 at 517
template <typename T, typename S, int E, bool BRANCH, int MOVES>
cudaError_t launch_widths(const NormLaunch &L, cudaStream_t stream) {
    const int w = L.width;
    if (L.backward) {
        if (w <= 32) return backward<T, S, E, 8, true, BRANCH, MOVES>(L, stream);
        if (w <= 256) return backward<T, S, E, 16, true, BRANCH, MOVES>(L, stream);
        if constexpr (sizeof(S) == 2) {
            if (w > 512 && w <= 768) return backward<T, S, E, 24, false, BRANCH, MOVES>(L, stream);
            if (!BRANCH && w > 1536) return backward<T, S, E, 32, false, BRANCH, MOVES>(L, stream);
        }
        if (w > 8192) return backward<T, S, E, 32, false, BRANCH, MOVES>(L, stream);
        return backward<T, S, E, 16, false, BRANCH, MOVES>(L, stream);
    }
    // Two rows at a time where there is room for two stages of them, and they need no registers on their way.
    constexpr int kRows = sizeof(S) + (BRANCH ? sizeof(T) : 0) > 6 || MOVES == kHalves ? 1 : 2;
    if (w <= 32) return forward<T, S, E, 8, true, 2 * kRows, BRANCH, MOVES>(L, stream);
    if (w <= 256) return forward<T, S, E, 16, true, kRows, BRANCH, MOVES>(L, stream);
    if (w > 8192) return forward<T, S, E, 32, false, 1, BRANCH, MOVES>(L, stream);
    return forward<T, S, E, 16, false, kRows, BRANCH, MOVES>(L, stream);
}

template <typename T, typename S, int E, int MOVES>
cudaError_t launch_branch(const NormLaunch &L, cudaStream_t stream) {
    return L.join ? launch_widths<T, S, E, true, MOVES>(L, stream) : launch_widths<T, S, E, false, MOVES>(L, stream);
}

// Chunks of 8 for rows of 16-bit types alone, whose 16 bytes are one access; beside fp32 rows, and where rows are not
// aligned to that, chunks of 4.
template <typename T, typename S>
cudaError_t launch_types(const NormLaunch &L, cudaStream_t stream) {
    if constexpr (sizeof(S) == 2) {
        if (L.wide) return launch_branch<T, S, 8, kWhole>(L, stream);
    }
    if constexpr (sizeof(T) == 2) {
        if (L.moves == kHalves) return launch_branch<T, S, 4, kHalves>(L, stream);
    }
    return L.moves == kWhole ? launch_branch<T, S, 4, kWhole>(L, stream) : launch_branch<T, S, 4, kWords>(L, stream);
}

}  // namespace norm
}  // namespace cli
