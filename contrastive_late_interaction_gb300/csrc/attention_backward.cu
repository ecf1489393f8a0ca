// Gradients of cross attention over tapes: the tensor-core backward.
//
// Mathematics.  With p_rj = exp(scale <q_r, k_j> - lse_r) recomputed from the
// forward's lse and delta_r = <dO_r, O_r>:
//     dV_j = sum_r p_rj dO_r,      ds_rj = p_rj (<dO_r, v_j> - delta_r),
//     dQ_r = scale sum_j ds_rj k_j,   dK_j = scale sum_r ds_rj q_r.
//
// Two kernels, each the owner of what it sums, so no sum crosses CTAs and the
// results do not depend on the order in which CTAs run.  dkv_kernel holds 128
// states and walks the item's queries (four products of 128 x 128 x D a block:
// S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q); dq_kernel holds 128
// rows and walks the item's states (three: S, dP, dQ += dS K).  One kernel
// would need five products in the place of seven, but sums dQ across CTAs:
// with fp32 reductions in memory, in whatever order they arrive.
//
// Both keep the scores' tiles in TMEM: S is turned into P in place, dP into dS
// (16-bit, over the first half of the columns of each reader), and the second
// products read them from there as their A operand.  Rows are packed as in the
// forward: the heads of a group lie side by side in a tile.  Warp roles are
// those of the forward, with eight warps for the tiles' arithmetic: each
// thread has one row of TMEM and half of its columns.
//
// Delta.  The output is rounded, so delta_r from it is off by up to u <|dO_r|,
// |O_r|>.  That hardly shows in dQ_r, but where one state has most of a row's
// weight, its ds is a small difference of large terms and an element of dK was
// off by 0.3 to 0.7 of the root mean square of all of dK in items of few rows.
// So dq_kernel runs first, with that delta, and sums each row's ds in 32 bits:
// the sum over a row is 0 but for delta's error, and dkv_kernel takes delta
// with it.  The order costs the time that dq_kernel used to fill at the other's
// end: 32 items of 512 to 2048 x 512 to 1024 rows, 690 -> 783 us.
//
// Rounding.  P and dS are rounded to 16 bits as operands; sums are in 32 bits.
// The error of dV and dK against 64 bits is 1.4 times what one rounding at the
// end leaves (bf16: 0.0023 of the norm, not 0.0017), that of dQ, which has the
// first delta, 1.5 to 2.3 times (0.0026 to 0.0038, the latter where one state has
// most of most rows' weight).  Doubling the operands would double the products;
// delta from a kernel of its own, of S and dP alone, brings dQ to 1.4 times for
// 80 us more, the sums of p k beside those of ds k for 210.
//
// Bound: 32 items of 512 to 2048 x 512 to 1024 rows, 16 heads of 128 in groups
// of 4, take 783 us: stats 54 (HBM: dO and O), dq 311, dkv 419, of which some
// 80 are its end, where CTAs wait for the last units of up to 64 blocks.  The
// rest is the arithmetic between products, for which a block has only two
// products to hide under (8 x 2048 x 1024, 16 heads of 128: 57% of the tensor
// pipe in dq, 68% in dkv), and the items' ends.  Short items (96 of 1 to 300 x 0
// to 700 rows, fp16) are bound by the chain of loads, products and stores of a
// tile of four or five blocks: 127 us.

#include <cuda.h>

#include "attention.cuh"

namespace cli {
namespace attn {
namespace {

constexpr int kThreads = 384;
constexpr int kWorks = 4;
constexpr int kReaders = 11;   // of a published work item: warps 0 to 2, eight arithmetic warps

// What the scores' rows need in the backward, one entry per output row and
// head at stat_at: -lse in powers of two (-infinity where the row kept no
// state, so that p is 0) and -delta of the rounded output, to be added.
__device__ __forceinline__ long long stat_at(const AttentionLaunch &L, int out_rows, int key_head, long long row) {
    return (static_cast<long long>(key_head) * out_rows + row) * L.group;
}

// fp16: the largest square of a norm among the output gradient's rows of heads,
// and among the kept values', as the bits of a float.  Rows that are not
// finite are left out: their own gradients are not finite either.
struct Bounds {
    uint32_t d_o, v;
};
// The largest of a block's threads, in whatever order the blocks come: one request a block, as they all go to one address.
__device__ __forceinline__ void raise_bounds(Bounds *bounds, float d_o, float v) {
    __shared__ float most[2][8];
    for (int w = 16; w; w >>= 1) {
        d_o = fmaxf(d_o, __shfl_xor_sync(0xffffffffu, d_o, w));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, w));
    }
    if ((threadIdx.x & 31) == 0) most[0][threadIdx.x >> 5] = d_o, most[1][threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x > 1) return;
    float mine = 0.0f;
    for (int w = 0; w < 8; ++w) mine = fmaxf(mine, most[threadIdx.x][w]);
    atomicMax(threadIdx.x ? &bounds->v : &bounds->d_o, __float_as_uint(mine));
}

// What dS is multiplied by beside P's 2^14: |dS| <= p (|dP| + |delta|) <= 2 |dO| |v| < 2^(e + 1), and 2^14 2^-e times
// that is below 2^15.
template <typename T>
__device__ __forceinline__ float ds_scale(const Bounds *bounds) {
    if constexpr (Type<T>::bf16) return 1.0f;
    const float most = 2.001f * sqrtf(__uint_as_float(__ldcg(&bounds->d_o))) * sqrtf(__uint_as_float(__ldcg(&bounds->v)));
    return most > 0.0f ? power_of_two(-exponent_of(most)) : 1.0f;
}

// The larger of `most` and the square of the norm of a row of a head, 8 elements a lane of 16.
__device__ __forceinline__ float larger_square(float most, const uint32_t (&w)[4]) {
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = Type<__half>::unpack(w[i]);
        sq = fmaf(v.x, v.x, fmaf(v.y, v.y, sq));
    }
#pragma unroll
    for (int s = 8; s; s >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, s);
    return sq < INFINITY ? fmaxf(most, sq) : most;   // not infinite, and not a NaN
}

// A warp a row, 16 lanes a head, 8 elements a lane, the loads of eight heads
// under way together.
template <typename T>
__global__ void __launch_bounds__(256, 4) stats_kernel(const __grid_constant__ AttentionLaunch L, int out_rows,
                                                    float2 *stats, Bounds *bounds) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    after_previous();
    check_items(L, static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, static_cast<long long>(gridDim.x) * 256);
    const int lane = threadIdx.x & 15, side = (threadIdx.x >> 4) & 1;
    const bool in = 8 * lane < L.head_dim;
    constexpr int kAtOnce = 4;
    float most = 0.0f, most_v = 0.0f;
    for (long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < out_rows;
         row += static_cast<long long>(gridDim.x) * 8) {
        const T *o = static_cast<const T *>(L.o.data) + row * L.o.row + 8 * lane;
        const T *d_o = static_cast<const T *>(L.d_o.data) + row * L.d_o.row + 8 * lane;
        for (int h0 = side; h0 - side < L.query_heads; h0 += 2 * kAtOnce) {
            uint4 a[kAtOnce], b[kAtOnce];
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                const int h = h0 + 2 * x;
                a[x] = b[x] = make_uint4(0, 0, 0, 0);
                if (in && h < L.query_heads) {
                    a[x] = __ldcs(reinterpret_cast<const uint4 *>(o + h * L.o.head));
                    b[x] = __ldg(reinterpret_cast<const uint4 *>(d_o + h * L.d_o.head));
                }
            }
            float d[kAtOnce];
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                const uint32_t wa[4] = {a[x].x, a[x].y, a[x].z, a[x].w}, wb[4] = {b[x].x, b[x].y, b[x].z, b[x].w};
                d[x] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = Type<T>::unpack(wa[i]), v = Type<T>::unpack(wb[i]);
                    d[x] = fmaf(u.x, v.x, fmaf(u.y, v.y, d[x]));
                }
                if constexpr (!Type<T>::bf16) most = larger_square(most, wb);
#pragma unroll
                for (int s = 8; s; s >>= 1) d[x] += __shfl_xor_sync(0xffffffffu, d[x], s);
            }
            if (lane < kAtOnce) {
                float mine = d[0];
#pragma unroll
                for (int x = 1; x < kAtOnce; ++x) mine = lane == x ? d[x] : mine;
                const int h = h0 + 2 * lane;
                if (h < L.query_heads) {
                    const int kh = h / L.group;
                    const float lse = L.lse[row * L.query_heads + h];
                    stats[stat_at(L, out_rows, kh, row) + h - kh * L.group] =
                        make_float2(lse == -INFINITY ? -INFINITY : -lse * kLog2e, -mine);
                }
            }
        }
    }
    if constexpr (!Type<T>::bf16) {
        const long long cells = static_cast<long long>(L.key_rows) * L.key_heads;
        for (long long c0 = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 2 * kAtOnce; c0 < cells;
             c0 += static_cast<long long>(gridDim.x) * 16 * kAtOnce) {
            uint4 a[kAtOnce];
            bool kept[kAtOnce];
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                const long long cell = c0 + 2 * x + side, row = cell / L.key_heads;
                a[x] = make_uint4(0, 0, 0, 0), kept[x] = false;
                if (cell >= cells) continue;
                kept[x] = !L.key_mask || L.key_mask[row] != 0;
                if (in)
                    a[x] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(L.v.data) + row * L.v.row +
                                                                 (cell - row * L.key_heads) * L.v.head + 8 * lane));
            }
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                const uint32_t w[4] = {a[x].x, a[x].y, a[x].z, a[x].w};
                const float with = larger_square(most_v, w);
                most_v = kept[x] ? with : most_v;
            }
        }
        raise_bounds(bounds, most, most_v);
    }
}

// dP - delta, both times the scale of dS (delta has it already).
template <typename T>
__device__ __forceinline__ float2 centred(float2 dp, float2 unit, float2 minus_delta) {
    return Type<T>::bf16 ? __fadd2_rn(dp, minus_delta) : __ffma2_rn(dp, unit, minus_delta);
}

// One CTA's current work: a tile of 128 states or of 128 packed rows.
struct alignas(16) Work {
    int q0, o0, nq, k0, nk, head, part;   // nq, nk: rows of the item to walk, or of the tile; head < 0: no more work
};

// The walked tiles come through two rings.  Those of A (Q, or K) are held
// longest, from the scores of a block to the last product of it, while the
// next block's scores are already wanted: they need three stages (with two,
// the products waited 1100 of 3900 cycles a block).  Those of B (dO, or V) are
// done with earlier.
template <int BOXES>
struct Storage {
    static constexpr uint32_t kA = BOXES == 2 ? 3 : 4, kB = BOXES == 2 ? 2 : 3;
    alignas(1024) uint8_t held[2][BOXES * kBoxBytes];      // K and V, or Q and dO
    alignas(1024) uint8_t ring_a[kA][BOXES * kBoxBytes];
    alignas(1024) uint8_t ring_b[kB][BOXES * kBoxBytes];
    alignas(16) float lse[kB][128], delta[kA][128];        // dkv: of a stage's rows, negated; lse is done with when dO is
    uint32_t bits[4][4];                                    // dq: a block's kept states
    Work work[kWorks];
    uint64_t work_full[kWorks], work_empty[kWorks];
    uint64_t held_full, held_empty, a_full[kA], a_empty[kA], a_ready[kA], b_full[kB], b_empty[kB], b_ready[kB];
    uint64_t s_full[2], dp_full, p_ready, ds_ready[2], sum_full, done;   // the dkv kernel uses the first of two
    uint32_t tmem_base;
    int abort_flag;
};

struct Maps {
    CUtensorMap q, k, v, d_o;
};

template <typename Smem>
__device__ __forceinline__ uint32_t begin(Smem &sm, const Maps &M, int32_t *status) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.ds_ready[i], 8);
        }
        for (uint32_t i = 0; i < Smem::kA; ++i) {
            mbar_init(&sm.a_full[i], 1);
            mbar_init(&sm.a_empty[i], 1);
            mbar_init(&sm.a_ready[i], 1);
        }
        for (uint32_t i = 0; i < Smem::kB; ++i) {
            mbar_init(&sm.b_full[i], 1);
            mbar_init(&sm.b_empty[i], 1);
            mbar_init(&sm.b_ready[i], 1);
        }
        for (int i = 0; i < kWorks; ++i) {
            mbar_init(&sm.work_full[i], 1);
            mbar_init(&sm.work_empty[i], kReaders);
        }
        mbar_init(&sm.held_full, 1);
        mbar_init(&sm.held_empty, 1);
        mbar_init(&sm.dp_full, 1);
        mbar_init(&sm.p_ready, 8);
        mbar_init(&sm.sum_full, 1);
        mbar_init(&sm.done, 1);
        // The tiles use every byte there is, so the array has to start on 1024, as it asks for.
        sm.abort_flag = smem_u32(&sm) % 1024 != 0;
        if (sm.abort_flag) report(status, CLI_INTERNAL);
        fence_mbar_init();
        prefetch_tmap(&M.q);
        prefetch_tmap(&M.k);
        prefetch_tmap(&M.v);
        prefetch_tmap(&M.d_o);
    }
    if (threadIdx.x / 32 == 1) tmem_alloc(&sm.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return sm.tmem_base;
}

template <typename Smem>
__device__ __forceinline__ bool next_work(Smem &sm, const AttentionLaunch &L, uint32_t it, Work &w) {
    if (!wait_warp(&sm.work_full[it % kWorks], (it / kWorks) & 1, &sm.abort_flag, L.status)) return false;
    w = sm.work[it % kWorks];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.work_empty[it % kWorks]);
    return w.head >= 0;
}

// Hands out the work: blocks of `span` states (of_keys) or queries.
template <typename Smem>
__device__ __forceinline__ void hand_out(Smem &sm, const AttentionLaunch &L, bool of_keys, int span, long long tiles,
                                         const Split &cut, unsigned long long *counter) {
    const int lane = threadIdx.x & 31, batch = batch_of(tiles);
    const uint64_t *off = of_keys ? L.k_off : L.q_off;
    const int per_item = off ? 0 : (L.query_rows + span - 1) / span;
    uint32_t it = 0;
    bool ok = true;
    auto publish = [&](const Work &w) {
        if (!wait_warp(&sm.work_empty[it % kWorks], ((it / kWorks) & 1) ^ 1, &sm.abort_flag, L.status)) return false;
        if (lane == 0) {
            sm.work[it % kWorks] = w;
            mbar_arrive(&sm.work_full[it % kWorks]);
        }
        ++it;
        return true;
    };
    while (ok) {
        unsigned long long base = 0;
        if (lane == 0) base = atomicAdd(counter, static_cast<unsigned long long>(batch));
        base = __shfl_sync(0xffffffffu, base, 0);
        if (base >= static_cast<unsigned long long>(tiles)) break;
        const long long id = static_cast<long long>(base) + lane;
        Item t;
        int r0 = 0;
        long long block = id / L.key_heads;
        const int head = static_cast<int>(id - block * L.key_heads);
        int part = 0;
        if (cut.parts > 1) {
            const long long whole = block / cut.parts;
            part = static_cast<int>(block - whole * cut.parts);
            block = whole;
        }
        const bool on = lane < batch && id < tiles && find_block(L, off, span, per_item, of_keys, block, t, r0);
        if (on && cut.parts > 1) part_of(cut, part, t);
        for (uint32_t left = __ballot_sync(0xffffffffu, on); left && ok; left &= left - 1) {
            const int from = __ffs(left) - 1;
            Work w = of_keys ? Work{t.q0, t.o0, t.nq, t.k0 + r0, min(span, t.nk - r0), head, part}
                             : Work{t.q0 + r0, t.o0 + r0, min(span, t.nq - r0), t.k0, t.nk, head, part};
            w.q0 = __shfl_sync(0xffffffffu, w.q0, from);
            w.o0 = __shfl_sync(0xffffffffu, w.o0, from);
            w.nq = __shfl_sync(0xffffffffu, w.nq, from);
            w.k0 = __shfl_sync(0xffffffffu, w.k0, from);
            w.nk = __shfl_sync(0xffffffffu, w.nk, from);
            w.head = __shfl_sync(0xffffffffu, w.head, from);
            w.part = __shfl_sync(0xffffffffu, w.part, from);
            ok = publish(w);
        }
    }
    if (ok) publish({0, 0, 0, 0, 0, -1, 0});
}

// The TMA producer's side.
template <int BOXES, typename Smem>
struct Producer {
    Smem &sm;
    const AttentionLaunch &L;
    uint32_t entry = 0, held = 0;
    __device__ bool wait(uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, &sm.abort_flag, L.status); }
    __device__ void load(uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int head, int row) {
#pragma unroll
        for (int b = 0; b < BOXES; ++b) tma_load_3d(dst + b * kBoxBytes, map, bar, 64 * b, head, row);
    }
    // One thread: the held pair of tiles (bytes: of one), then a stage's pair.
    __device__ bool hold(const CUtensorMap *a, const CUtensorMap *b, uint32_t bytes, int head, int row_a, int row_b) {
        if (!wait(&sm.held_empty, (held & 1) ^ 1)) return false;
        ++held;
        mbar_arrive_expect_tx(&sm.held_full, 2 * bytes);
        load(sm.held[0], a, &sm.held_full, head, row_a);
        load(sm.held[1], b, &sm.held_full, head, row_b);
        return true;
    }
    __device__ bool stage(const CUtensorMap *a, const CUtensorMap *b, uint32_t bytes, int head, int row_a, int row_b) {
        constexpr uint32_t kA = Smem::kA, kB = Smem::kB;
        const uint32_t x = entry % kA, y = entry % kB;
        if (!wait(&sm.a_empty[x], ((entry / kA) & 1) ^ 1)) return false;
        mbar_arrive_expect_tx(&sm.a_full[x], bytes);
        load(sm.ring_a[x], a, &sm.a_full[x], head, row_a);
        if (!wait(&sm.b_empty[y], ((entry / kB) & 1) ^ 1)) return false;
        mbar_arrive_expect_tx(&sm.b_full[y], bytes);
        load(sm.ring_b[y], b, &sm.b_full[y], head, row_b);
        ++entry;
        return true;
    }
    // Lets the loads in flight land before the CTA can exit.
    __device__ void drain() {
        for (uint32_t s = 0; s < Smem::kA; ++s)
            if (entry > s) wait(&sm.a_empty[s], ((entry - 1 - s) / Smem::kA) & 1);
        for (uint32_t s = 0; s < Smem::kB; ++s)
            if (entry > s) wait(&sm.b_empty[s], ((entry - 1 - s) / Smem::kB) & 1);
        if (held) wait(&sm.held_empty, (held - 1) & 1);
    }
};

// ----------------------------------------------------------------------------
// dK, dV
// ----------------------------------------------------------------------------

// TMEM: S^T / P^T | dP^T / dS^T | dV | dK.  The products of block j + 1's
// scores run between those of block j, so that each of the two arithmetic
// steps (P from S, dS from dP) has two products to hide under:
//     ... [dV(j) S(j+1)] [dK(j) dP(j+1)] [dV(j+1) S(j+2)] ...
template <typename T, int BOXES>
__global__ void __launch_bounds__(kThreads, 1)
    dkv_kernel(const __grid_constant__ AttentionLaunch L, const __grid_constant__ Maps M, int rows_per_tile,
               int out_rows, const float2 *stats, const float *ds_sums, const Bounds *bounds, long long tiles,
               unsigned long long *counter) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    using Smem = Storage<BOXES>;
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t tmem = begin(sm, M, L.status);
    after_previous();
    const int group = L.group, dim = L.head_dim;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, &sm.abort_flag, L.status); };
    auto q_blocks = [&](const Work &w) { return (w.nq + rows_per_tile - 1) / rows_per_tile; };
    auto q_rows = [&](const Work &w, int j) { return min(rows_per_tile, w.nq - j * rows_per_tile) * group; };

    if (warp == 0) {
        Producer<BOXES, Smem> P{sm, L};
        const uint32_t q_bytes = BOXES * static_cast<uint32_t>(rows_per_tile * group) * 128u;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            if (lane == 0 && w.nq) {
                ok = P.hold(&M.k, &M.v, BOXES * kBoxBytes, w.head, w.k0, w.k0);
                for (int j = 0; j < q_blocks(w) && ok; ++j)
                    ok = P.stage(&M.q, &M.d_o, q_bytes, w.head * group, w.q0 + j * rows_per_tile, w.o0 + j * rows_per_tile);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) P.drain();
    } else if (warp == 1) {
        const uint32_t idesc_s = idesc_16bit(Type<T>::bf16, 128, 0, 0, 0);   // N by block
        const uint32_t idesc_d = idesc_16bit(Type<T>::bf16, 128, round16(dim), 0, 1);
        constexpr uint32_t kA = Smem::kA, kB = Smem::kB;
        const uint64_t held_desc = desc_rows(smem_u32(sm.held[0]));
        const uint64_t a_rows = desc_rows(smem_u32(sm.ring_a[0])), b_rows = desc_rows(smem_u32(sm.ring_b[0]));
        const uint64_t a_sum = desc_sum(smem_u32(sm.ring_a[0])), b_sum = desc_sum(smem_u32(sm.ring_b[0]));
        constexpr uint64_t kTile = desc_bytes(BOXES * kBoxBytes);
        const int steps = (dim + 15) / 16;
        const uint32_t leader = elected(), tm = uniform(tmem);
        uint32_t entry = 0, held = 0, j_all = 0;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            w.nq = static_cast<int>(uniform(w.nq));
            const int blocks = q_blocks(w);
            if (blocks == 0) continue;
            // A 16-bit TMEM operand whose halves lie 64 columns apart.
            auto sum = [&](uint32_t d, uint32_t a, uint64_t b, int rows, bool more) {
                mma_pairs<4>(leader, d, a, b, idesc_d, rows, more);
                mma_pairs<4>(leader, d, a + 64, b + desc_bytes(4 * 2048), idesc_d, rows - 64, true);
            };
            auto scores = [&](int j, uint32_t e, int which) {
                const uint32_t n = round16(q_rows(w, j));
                mma_rows<BOXES>(leader, tm + which * 128, held_desc + which * kTile,
                                which ? b_rows + e % kB * kTile : a_rows + e % kA * kTile, idesc_s | (n >> 3) << 17, steps);
                issue_commit(leader, which ? &sm.dp_full : &sm.s_full[0]);
            };
            auto a_there = [&](uint32_t e) { return wait(&sm.a_ready[e % kA], (e / kA) & 1); };
            auto b_there = [&](uint32_t e) { return wait(&sm.b_ready[e % kB], (e / kB) & 1); };
            ok = wait(&sm.held_full, held & 1) && a_there(entry);
            ++held;
            tc_fence_after();
            if (ok) {
                scores(0, entry, 0);
                ok = b_there(entry);
            }
            if (ok) {
                tc_fence_after();
                scores(0, entry, 1);
                if (blocks == 1) issue_commit(leader, &sm.held_empty);
            }
            for (int j = 0; j < blocks && ok; ++j, ++j_all) {
                const uint32_t e = entry + j, en = e + 1;
                if (!wait(&sm.p_ready, j_all & 1)) { ok = false; break; }
                tc_fence_after();
                sum(tm + 256, tm, b_sum + e % kB * kTile, q_rows(w, j), j != 0);
                issue_commit(leader, &sm.b_empty[e % kB]);
                if (j + 1 < blocks) {
                    if (!a_there(en)) { ok = false; break; }
                    tc_fence_after();
                    scores(j + 1, en, 0);
                }
                if (!wait(&sm.ds_ready[0], j_all & 1)) { ok = false; break; }
                tc_fence_after();
                sum(tm + 384, tm + 128, a_sum + e % kA * kTile, q_rows(w, j), j != 0);
                issue_commit(leader, &sm.a_empty[e % kA]);
                if (j + 1 < blocks) {
                    if (!b_there(en)) { ok = false; break; }
                    tc_fence_after();
                    scores(j + 1, en, 1);
                    if (j + 2 == blocks) issue_commit(leader, &sm.held_empty);
                } else {
                    issue_commit(leader, &sm.sum_full);
                }
            }
            entry += blocks;
        }
        issue_commit(leader, &sm.done);
        wait(&sm.done, 0);
    } else if (warp == 2) {
        // Rows past the item's end are zeroed (they are summed over), and the rows' lse and corrected delta staged.
        const long long cells = static_cast<long long>(out_rows) * L.query_heads;
        const float ds_unit = ds_scale<T>(bounds);
        uint32_t entry = 0;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            const int blocks = q_blocks(w);
            for (int j = 0; j < blocks; ++j, ++entry) {
                const int n = q_rows(w, j);
                const long long first = stat_at(L, out_rows, w.head, static_cast<long long>(w.o0) + j * rows_per_tile);
                float2 f[4], more[4];   // all on their way together: one after another they held up every block
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 32 * i + lane;
                    f[i] = make_float2(-INFINITY, 0.0f), more[i] = make_float2(0.0f, 0.0f);
                    if (at < n) {
                        f[i] = stats[first + at];
                        more[i] = make_float2(ds_sums[first + at], ds_sums[cells + first + at]);
                    }
                }
                const uint32_t s = entry % Smem::kA, sb = entry % Smem::kB;
                if (!wait(&sm.a_full[s], (entry / Smem::kA) & 1)) { ok = false; break; }
                const uint32_t keep[4] = {first_bits(n, 0), first_bits(n, 1), first_bits(n, 2), first_bits(n, 3)};
                zero_rows<BOXES>(smem_u32(sm.ring_a[s]), round16(n), keep, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.a_ready[s]);
                if (!wait(&sm.b_full[sb], (entry / Smem::kB) & 1)) { ok = false; break; }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sm.lse[sb][32 * i + lane] = f[i].x + weight_shift<T>();
                    sm.delta[s][32 * i + lane] = (f[i].y - (more[i].x + more[i].y)) * ds_unit;
                }
                zero_rows<BOXES>(smem_u32(sm.ring_b[sb]), round16(n), keep, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.b_ready[sb]);
            }
        }
    } else if (warp == 3) {
        hand_out(sm, L, true, 128, tiles, {1, 0}, counter);
    } else {
        const int side = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_at = tmem + lanes + side * 64, dp_at = s_at + 128;
        const float2 sl22 = make_float2(L.scale * kLog2e, L.scale * kLog2e);
        const float ds_unit = ds_scale<T>(bounds);
        const float2 ds_unit2 = make_float2(ds_unit, ds_unit);
        uint32_t j_all = 0, works = 0;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            const int blocks = q_blocks(w);
            const bool mine = row < w.nk, live = mine && (!L.key_mask || L.key_mask[w.k0 + row] != 0);
            for (int j = 0; j < blocks; ++j, ++j_all) {
                const int n = round16(q_rows(w, j)) - side * 64;   // columns of this side
                const uint32_t sb = j_all % Smem::kB;
                if (!wait(&sm.b_ready[sb], (j_all / Smem::kB) & 1) || !wait(&sm.s_full[0], j_all & 1)) { ok = false; break; }
                tc_fence_after();
                // A dropped state's row of scores may be anything; so is its row of P and dS then, which reaches
                // its own row of the sums alone, and that is not written.
                const float4 *lse = reinterpret_cast<const float4 *>(sm.lse[sb] + side * 64);
                const float4 *delta = reinterpret_cast<const float4 *>(sm.delta[j_all % Smem::kA] + side * 64);
                float2 p[32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (32 * c >= n) continue;
                    uint32_t r[32], packed[16];
                    tmem_ld32_async(s_at + 32 * c, r);
                    tmem_wait_ld();
                    tmem_regs_ready(r);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 l = lse[8 * c + i / 4];
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), sl22, make_float2(l.x, l.y));
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), sl22, make_float2(l.z, l.w));
                        x = make_float2(ex2(x.x), ex2(x.y));
                        y = make_float2(ex2(y.x), ex2(y.y));
                        p[16 * c + i / 2] = x;
                        p[16 * c + i / 2 + 1] = y;
                        packed[i / 2] = Type<T>::pack(x.x, x.y);
                        packed[i / 2 + 1] = Type<T>::pack(y.x, y.y);
                    }
                    tmem_st16(s_at + 16 * c, packed);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_ready);
                if (!wait(&sm.dp_full, j_all & 1)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (32 * c >= n) continue;
                    uint32_t r[32], packed[16];
                    tmem_ld32_async(dp_at + 32 * c, r);
                    tmem_wait_ld();
                    tmem_regs_ready(r);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 d = delta[8 * c + i / 4];
                        float2 x = centred<T>(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), ds_unit2, make_float2(d.x, d.y));
                        float2 y = centred<T>(make_float2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), ds_unit2, make_float2(d.z, d.w));
                        x = __fmul2_rn(p[16 * c + i / 2], x);
                        y = __fmul2_rn(p[16 * c + i / 2 + 1], y);
                        packed[i / 2] = Type<T>::pack(x.x, x.y);
                        packed[i / 2 + 1] = Type<T>::pack(y.x, y.y);
                    }
                    tmem_st16(dp_at + 16 * c, packed);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ds_ready[0]);
            }
            if (!ok) break;
            if (blocks) {
                if (!wait(&sm.sum_full, works & 1)) break;
                ++works;
                tc_fence_after();
            }
            const HeadsView &v = side ? L.d_k : L.d_v;
            T *out = static_cast<T *>(v.data) + (static_cast<long long>(w.k0) + row) * v.row + w.head * v.head;
            store_sums<T>(tmem + lanes + 256 + side * 128, dim, weight_unit<T>() * (side ? L.scale / ds_unit : 1.0f), blocks != 0, !live, mine, out);
            tc_fence_before();
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------------------
// dQ
// ----------------------------------------------------------------------------

// TMEM: S / dS of even blocks | of odd blocks | dP | dQ.  p_ready says here
// that dP has been read, so that the next block's may be written.  s_full and
// ds_ready alternate: the scores of block j + 1 are issued before block j's
// are waited for, and dP of block j + 1 before ds of block j is, so with one
// barrier each a phase could pass unseen.
// It runs first: each row's sum of ds, which the two sides' threads leave in
// slots 2 part and 2 part + 1 of `ds_sums`, is what dkv_kernel corrects delta by.
template <typename T, int BOXES>
__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ AttentionLaunch L, const __grid_constant__ Maps M, int rows_per_tile,
              int out_rows, const float2 *stats, float *ds_sums, const Bounds *bounds, float *partials, long long tiles,
              Split cut, unsigned long long *counter) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    using Smem = Storage<BOXES>;
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t tmem = begin(sm, M, L.status);
    after_previous();
    // dkv_kernel may set up on the SMs that this one leaves, where it waits for all of this one.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int group = L.group, dim = L.head_dim;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, &sm.abort_flag, L.status); };

    if (warp == 0) {
        Producer<BOXES, Smem> P{sm, L};
        const uint32_t q_bytes = BOXES * static_cast<uint32_t>(rows_per_tile * group) * 128u;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            if (lane == 0 && w.nk) {
                ok = P.hold(&M.q, &M.d_o, q_bytes, w.head * group, w.q0, w.o0);
                for (int j = 0; j < (w.nk + 127) / 128 && ok; ++j)
                    ok = P.stage(&M.k, &M.v, BOXES * kBoxBytes, w.head, w.k0 + 128 * j, w.k0 + 128 * j);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) P.drain();
    } else if (warp == 1) {
        const uint32_t idesc_s = idesc_16bit(Type<T>::bf16, 128, 0, 0, 0);   // N by block
        const uint32_t idesc_d = idesc_16bit(Type<T>::bf16, 128, round16(dim), 0, 1);
        constexpr uint32_t kA = Smem::kA, kB = Smem::kB;
        const uint64_t held_desc = desc_rows(smem_u32(sm.held[0]));
        const uint64_t a_rows = desc_rows(smem_u32(sm.ring_a[0])), b_rows = desc_rows(smem_u32(sm.ring_b[0]));
        const uint64_t a_sum = desc_sum(smem_u32(sm.ring_a[0])), b_sum = desc_sum(smem_u32(sm.ring_b[0]));
        constexpr uint64_t kTile = desc_bytes(BOXES * kBoxBytes);
        const int steps = (dim + 15) / 16;
        const uint32_t leader = elected(), tm = uniform(tmem);
        uint32_t entry = 0, held = 0, j_all = 0;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            const int nk = static_cast<int>(uniform(w.nk)), blocks = (nk + 127) / 128;
            if (blocks == 0) continue;
            auto scores = [&](int j, uint32_t e, int which) {
                const uint32_t n = round16(min(128, nk - 128 * j));
                const uint32_t d = which ? tm + 256 : tm + (e & 1) * 128;
                mma_rows<BOXES>(leader, d, held_desc + which * kTile, which ? b_rows + e % kB * kTile : a_rows + e % kA * kTile,
                                idesc_s | (n >> 3) << 17, steps);
                if (which) issue_commit(leader, &sm.b_empty[e % kB]);
                issue_commit(leader, which ? &sm.dp_full : &sm.s_full[e & 1]);
            };
            auto a_there = [&](uint32_t e) { return wait(&sm.a_ready[e % kA], (e / kA) & 1); };
            auto b_there = [&](uint32_t e) { return wait(&sm.b_full[e % kB], (e / kB) & 1); };
            ok = wait(&sm.held_full, held & 1) && a_there(entry);
            ++held;
            tc_fence_after();
            if (ok) {
                scores(0, entry, 0);
                ok = b_there(entry);
            }
            if (ok) {
                tc_fence_after();
                scores(0, entry, 1);
                if (blocks == 1) issue_commit(leader, &sm.held_empty);
            }
            for (int j = 0; j < blocks && ok; ++j, ++j_all) {
                const uint32_t e = entry + j, en = e + 1;
                if (j + 1 < blocks) {
                    if (!a_there(en)) { ok = false; break; }
                    tc_fence_after();
                    scores(j + 1, en, 0);
                }
                if (!wait(&sm.p_ready, j_all & 1)) { ok = false; break; }
                tc_fence_after();
                if (j + 1 < blocks) {
                    if (!b_there(en)) { ok = false; break; }
                    tc_fence_after();
                    scores(j + 1, en, 1);
                    if (j + 2 == blocks) issue_commit(leader, &sm.held_empty);
                }
                if (!wait(&sm.ds_ready[j_all & 1], (j_all >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                const int n = min(128, nk - 128 * j);
                const uint32_t a = tm + (e & 1) * 128;
                const uint64_t b = a_sum + e % kA * kTile;
                mma_pairs<4>(leader, tm + 384, a, b, idesc_d, n, j != 0);
                mma_pairs<4>(leader, tm + 384, a + 64, b + desc_bytes(4 * 2048), idesc_d, n - 64, true);
                issue_commit(leader, &sm.a_empty[e % kA]);
                if (j + 1 == blocks) issue_commit(leader, &sm.sum_full);
            }
            entry += blocks;
        }
        issue_commit(leader, &sm.done);
        wait(&sm.done, 0);
    } else if (warp == 2) {
        // Dropped states and those past the item's end: their K rows are zeroed (they are summed over), and
        // their bits staged.  V's rows only reach their own columns of dP, which are not used.
        uint32_t entry = 0;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            const int blocks = (w.nk + 127) / 128;
            for (int j = 0; j < blocks; ++j, ++entry) {
                const int n = min(128, w.nk - 128 * j);
                uint32_t keep[4];
                kept_bits(L, w.k0 + 128 * j, n, lane, keep);
                const uint32_t s = entry % Smem::kA;
                if (!wait(&sm.a_full[s], (entry / Smem::kA) & 1)) { ok = false; break; }
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) sm.bits[entry & 3][k] = keep[k];
                }
                zero_rows<BOXES>(smem_u32(sm.ring_a[s]), round16(n), keep, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.a_ready[s]);
            }
        }
    } else if (warp == 3) {
        hand_out(sm, L, false, rows_per_tile, tiles, cut, counter);
    } else {
        const int side = (warp - 4) >> 2, quad = warp & 3, m_row = quad * 32 + lane;
        const int r_in = m_row / group, head_in = m_row - r_in * group;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t dp_at = tmem + lanes + 256 + side * 64;
        const float sl2 = L.scale * kLog2e, ds_unit = ds_scale<T>(bounds);
        const float2 ds_unit2 = make_float2(ds_unit, ds_unit);
        uint32_t j_all = 0, works = 0;
        bool ok = true;
        Work w;
        for (uint32_t it = 0; ok && next_work(sm, L, it, w); ++it) {
            const int blocks = (w.nk + 127) / 128;
            const bool mine = r_in < w.nq && m_row < rows_per_tile * group;
            float2 st = make_float2(-INFINITY, 0.0f);
            if (mine)
                st = __ldcg(stats + stat_at(L, out_rows, w.head, static_cast<long long>(w.o0) + r_in) + head_in);
            st.x += weight_shift<T>();
            st.y *= ds_unit;
            const float2 sl22 = make_float2(sl2, sl2), shift = make_float2(st.x, st.x), delta = make_float2(st.y, st.y);
            float2 ds_sum = make_float2(0.0f, 0.0f);
            for (int j = 0; j < blocks; ++j, ++j_all) {
                const int n = min(128, w.nk - 128 * j) - side * 64;   // columns of this side
                const bool whole = !L.key_mask && n >= 64;
                const uint32_t s_at = tmem + lanes + (j_all & 1) * 128 + side * 64;
                if (!wait(&sm.a_ready[j_all % Smem::kA], (j_all / Smem::kA) & 1) || !wait(&sm.s_full[j_all & 1], (j_all >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                float2 p[32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (32 * c >= n) continue;
                    uint32_t r[32];
                    tmem_ld32_async(s_at + 32 * c, r);
                    tmem_wait_ld();
                    tmem_regs_ready(r);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), sl22, shift);
                        p[16 * c + i / 2] = make_float2(ex2(x.x), ex2(x.y));
                    }
                }
                if (!wait(&sm.dp_full, j_all & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t packed[2][16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (32 * c >= n) continue;
                    uint32_t r[32];
                    tmem_ld32_async(dp_at + 32 * c, r);
                    tmem_wait_ld();
                    tmem_regs_ready(r);
                    const uint32_t keep = whole ? 0xffffffffu : sm.bits[j_all & 3][2 * side + c];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 x = centred<T>(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), ds_unit2, delta);
                        x = __fmul2_rn(p[16 * c + i / 2], x);
                        if (!whole) {
                            x.x = (keep >> i) & 1u ? x.x : 0.0f;
                            x.y = (keep >> (i + 1)) & 1u ? x.y : 0.0f;
                        }
                        ds_sum = __fadd2_rn(ds_sum, x);
                        packed[c][i / 2] = Type<T>::pack(x.x, x.y);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_ready);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (32 * c < n) tmem_st16(s_at + 16 * c, packed[c]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ds_ready[j_all & 1]);
            }
            if (!ok) break;
            if (blocks) {
                if (!wait(&sm.sum_full, works & 1)) break;
                ++works;
                tc_fence_after();
            }
            const int head = w.head * group + head_in;
            if (mine)
                ds_sums[static_cast<long long>(2 * w.part + side) * out_rows * L.query_heads +
                        stat_at(L, out_rows, w.head, static_cast<long long>(w.o0) + r_in) + head_in] =
                    (ds_sum.x + ds_sum.y) * (weight_unit<T>() / ds_unit);
            // The sides take half of the row's columns each, in whole 16s.
            const int half = (dim / 2 + 15) & ~15;
            const int first = side ? half : 0, count = side ? dim - half : min(half, dim);
            const uint32_t sums = tmem + lanes + 384 + first;
            if (partials) {
                float *out = partials + ((static_cast<long long>(w.part) * out_rows + w.o0 + r_in) * L.query_heads + head) * dim + first;
                store_partials(sums, count, weight_unit<T>() / ds_unit, blocks != 0, mine, out);
            } else {
                T *out = static_cast<T *>(L.d_q.data) + (static_cast<long long>(w.q0) + r_in) * L.d_q.row + head * L.d_q.head + first;
                store_sums<T>(sums, count, weight_unit<T>() * (L.scale / ds_unit), blocks != 0, false, mine, out);
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Where items are cut into parts: the rows' sums of ds of all parts, in a fixed
// order, become those of the first.
__global__ void __launch_bounds__(256) ds_sum_kernel(float *ds_sums, long long cells, int parts) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    after_previous();
    const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;   // of both sides' cells
    if (at >= 2 * cells) return;
    float s = 0.0f;
#pragma unroll 8
    for (int p = 0; p < parts; ++p) s += ds_sums[2 * cells * p + at];
    ds_sums[at] = s;
}

// dQ of shared queries, and of items cut into parts: the sums of all, in a
// fixed order.  A block takes 128 elements, four a lane; its warps take an
// eighth of the sums each, so that many small items do not make one long chain
// of loads (512 items of 17 rows, 16 heads of 64: 144 us with a thread walking
// all of them).
constexpr int kSumElems = 128;
template <typename T>
__global__ void __launch_bounds__(256) dq_sum_kernel(const __grid_constant__ AttentionLaunch L, int sums, const float *partials) {
    __shared__ float4 part[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row_elems = static_cast<long long>(L.query_heads) * L.head_dim, all = row_elems * L.query_rows;
    const long long at = static_cast<long long>(blockIdx.x) * kSumElems + lane * 4;
    const int per = (sums + 7) / 8, from = min(sums, warp * per), to = min(sums, from + per);
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float4 &v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    if (at < all) {
#pragma unroll 8
        for (int i = from; i < to; ++i) add(__ldcs(reinterpret_cast<const float4 *>(partials + i * all + at)));
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp || at >= all) return;
    for (int w = 1; w < 8; ++w) add(part[w][lane]);
    const long long row = at / row_elems;
    const int in_row = static_cast<int>(at - row * row_elems), head = in_row / L.head_dim;
    *reinterpret_cast<uint2 *>(static_cast<T *>(L.d_q.data) + row * L.d_q.row + head * L.d_q.head + in_row - head * L.head_dim) =
        make_uint2(Type<T>::pack(s.x * L.scale, s.y * L.scale), Type<T>::pack(s.z * L.scale, s.w * L.scale));
}

long long cells_of(const AttentionLaunch &L) {
    return static_cast<long long>(L.query_rows) * (L.q_off ? 1 : L.items) * L.query_heads;
}
size_t stats_bytes(const AttentionLaunch &L) { return align256(static_cast<size_t>(cells_of(L)) * sizeof(float2)); }

// dq_kernel's work: slots of tiles of queries, parts along the states, and the sums that this leaves for each row.
struct Cut {
    long long slots;
    Split split;
    int sums;   // 1: none, dQ is stored at once
};
constexpr long long kLeastPart = 512;
Cut cut_of(const AttentionLaunch &L) {
    const int rows_per_tile = 128 / L.group;
    Cut c;
    c.slots = L.q_off ? static_cast<long long>(L.query_rows) / rows_per_tile + L.items
                      : static_cast<long long>(L.items) * ((L.query_rows + rows_per_tile - 1) / rows_per_tile);
    const long long filled = L.q_off ? (L.query_rows + rows_per_tile - 1) / rows_per_tile : c.slots;
    const long long blocks = (filled > L.items ? filled : L.items) * L.key_heads;
    c.split = split_of(L, blocks, 152, kLeastPart);
    c.sums = (L.q_off ? 1 : L.items) * c.split.parts;
    return c;
}

long long joins_of(const AttentionLaunch &L) {
    return (static_cast<long long>(L.query_rows) * L.query_heads * L.head_dim + kSumElems - 1) / kSumElems;
}

// Two slots of a float a part.
size_t ds_sums_bytes(const AttentionLaunch &L, const Cut &c) { return c.split.parts * stats_bytes(L); }

template <typename T, int BOXES>
cudaError_t launch(const AttentionLaunch &L, cudaStream_t stream) {
    const int rows_per_tile = 128 / L.group;
    const int out_rows = L.query_rows * (L.q_off ? 1 : L.items);
    unsigned long long *counters = reinterpret_cast<unsigned long long *>(L.workspace);
    Bounds *bounds = reinterpret_cast<Bounds *>(reinterpret_cast<uint32_t *>(L.workspace) + kBoundsAt);
    const Cut c = cut_of(L);
    uint8_t *at = L.workspace + kCounterBytes;
    float2 *stats = reinterpret_cast<float2 *>(at);
    float *ds_sums = reinterpret_cast<float *>(at += stats_bytes(L));
    float *partials = L.q_off && c.sums == 1 ? nullptr : reinterpret_cast<float *>(at + ds_sums_bytes(L, c));
    Maps M;
    const bool bf16 = Type<T>::bf16;
    if (!encode_heads_tiles(&M.q, L.q, bf16, L.head_dim, L.query_heads, L.query_rows, L.group, rows_per_tile) ||
        !encode_heads_tiles(&M.d_o, L.d_o, bf16, L.head_dim, L.query_heads, out_rows, L.group, rows_per_tile) ||
        !encode_heads_tiles(&M.k, L.k, bf16, L.head_dim, L.key_heads, L.key_rows, 1, kTileRows) ||
        !encode_heads_tiles(&M.v, L.v, bf16, L.head_dim, L.key_heads, L.key_rows, 1, kTileRows))
        return cudaErrorInvalidValue;
    const long long blocks = (static_cast<long long>(out_rows) + 7) / 8, most = 8ll * L.sm_count;
    begin_kernel<<<1, 32, 0, stream>>>(L.status, counters);
    cudaError_t e = launch_after(stats_kernel<T>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, stream, L,
                                 out_rows, stats, bounds);
    if (e != cudaSuccess) return e;

    const size_t smem = sizeof(Storage<BOXES>);
    static_assert(sizeof(Storage<BOXES>) <= 227 * 1024, "shared memory per CTA");
    auto dkv = dkv_kernel<T, BOXES>;
    auto dq = dq_kernel<T, BOXES>;
    e = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    auto grid = [&](long long tiles) { return static_cast<unsigned>(tiles < L.sm_count ? tiles : L.sm_count); };
    const long long q_tiles = c.slots * c.split.parts * L.key_heads;
    e = launch_after(dq, dim3(grid(q_tiles)), kThreads, smem, stream, L, M, rows_per_tile, out_rows, stats, ds_sums, bounds,
                     partials, q_tiles, c.split, counters);
    if (e != cudaSuccess) return e;
    if (c.split.parts > 1) {
        e = launch_after(ds_sum_kernel, dim3(static_cast<unsigned>((2 * cells_of(L) + 255) / 256)), 256, 0, stream, ds_sums,
                         cells_of(L), c.split.parts);
        if (e != cudaSuccess) return e;
    }
    const long long k_tiles = (static_cast<long long>(L.key_rows) / 128 + L.items) * L.key_heads;
    e = launch_after(dkv, dim3(grid(k_tiles)), kThreads, smem, stream, L, M, rows_per_tile, out_rows, stats, ds_sums, bounds,
                     k_tiles, counters + 1);
    if (e != cudaSuccess) return e;
    if (partials) dq_sum_kernel<T><<<static_cast<unsigned>(joins_of(L)), 256, 0, stream>>>(L, c.sums, partials);
    return cudaGetLastError();
}

}  // namespace

long long backward_tiles_joins(const AttentionLaunch &L) {
    const Cut c = cut_of(L);
    const long long folds = c.split.parts > 1 ? (2 * cells_of(L) + 255) / 256 : 0;
    const long long joins = L.q_off && c.sums == 1 ? 0 : joins_of(L);
    return folds > joins ? folds : joins;
}

size_t backward_tiles_workspace(const AttentionLaunch &L) {
    const Cut c = cut_of(L);
    const size_t rows = L.q_off && c.sums == 1 ? 0 : static_cast<size_t>(c.sums) * L.query_rows;
    const size_t partials = rows * L.query_heads * L.head_dim * sizeof(float);
    return kCounterBytes + stats_bytes(L) + ds_sums_bytes(L, c) + align256(partials);
}

// Needs at least one query row and one state (the tensor maps have no empty form).
cudaError_t launch_backward_tiles(const AttentionLaunch &L, cudaStream_t stream) {
    const bool wide = L.head_dim > 64;
    if (L.dtype == CLI_BF16) return wide ? launch<__nv_bfloat16, 2>(L, stream) : launch<__nv_bfloat16, 1>(L, stream);
    return wide ? launch<__half, 2>(L, stream) : launch<__half, 1>(L, stream);
}

}  // namespace attn
}  // namespace cli
