// Cross attention over tapes: the tensor-core forward.
//
// Mathematics.  For a query row with scores s_j = scale <q, k_j>:
//     m = max s_j,  p_j = exp(s_j - m),  l = sum p_j,
//     output = sum p_j v_j / l,  lse = m + ln l,
// in one pass over the states: m, l and the output accumulator are kept
// running, and when the maximum grows the earlier sums are scaled by exp of
// the difference.  Any reference value serves in the place of m as long as
// nothing overflows, so the accumulator is rescaled only when the maximum has
// grown by more than a factor of 2^8 over the reference: rarely after an
// item's first block.
//
// Work.  A tile is 128 rows of (query row, head of the group): the heads that
// share a key head are packed next to one another, so K and V are read once
// for all of them.  A persistent CTA takes two tiles at a time (or one, see
// dispatch) against blocks of 128 states; key heads are handed out before
// items, so that the lines that hold several heads are read together (64 x 4096
// rows, 8 heads of 128: 240 -> 198 us).  Warp roles:
//   0      issues the TMA loads: Q, and K and V blocks through a ring of
//          stages;
//   1      issues the products: S = Q K^T into TMEM, then O += P V with P read
//          from TMEM, alternating between the two tiles so that one tile's
//          softmax runs under the other's products;
//   2      makes the blocks safe: V's rows past the item's end and dropped
//          rows of K and V are zeroed (0 x NaN would reach the output through
//          the product), and for the states to leave out -infinity is added
//          to their scores by the product itself: one more step of 16
//          elements, a column of ones against a column of 0 or -infinity, so
//          that the softmax knows nothing of them;
//   3      hands out the pairs of tiles, some ahead, and checks the offsets of
//          every item;
//   4..11  softmax, four warps a tile, one row a thread: S from TMEM, P back
//          over the same columns, and at the end O / l to global memory.
// TMEM: S0 | S1 | O0 | O1, 128 columns each.
//
// Where the blocks of queries do not fill the SMs, items are also cut along their
// states, and join_parts_kernel adds the parts: 1 x 64 x 8192 rows, 8 heads of
// 128, take 18 us instead of 97.
//
// P is rounded to 16 bits because the product takes it so; l sums the weights
// before that.
//
// Bound: 8 items of 2048 x 4096 rows, 16 heads of 128, run at 1460 TFLOP/s (75%
// of measured), where the two tiles' softmax (about 1700 cycles a block of each,
// half of it exponentials) and products (2100 for both) take turns; 2048 x
// 1024 at 1280, the rest being the rows' way out at every item's end; 64 x 4096
// at 4.9 TB/s, bound by HBM.

#include <cuda.h>

#include "attention.cuh"

namespace cli {
namespace attn {
namespace {

constexpr int kPairs = 4;

struct Pair {
    int q0, o0, rows, k0, nk, head;   // o0: output row, or with parts the partials' row; rows < 0: no more work
};

// TILES: tiles that a CTA works on at a time.
template <int BOXES, int TILES>
struct Storage {
    // K blocks in the even stages, V blocks in the odd ones.
    static constexpr int kStages = TILES == 1 && BOXES == 2 ? 2 : 4;
    alignas(1024) uint8_t q[TILES][BOXES * kBoxBytes];
    alignas(1024) uint8_t kv[kStages][BOXES * kBoxBytes];
    alignas(128) uint8_t ones[kColumnBytes];             // a 1, and 15 zeros, for each of 128 rows
    alignas(128) uint8_t left_out[kStages / 2][kColumnBytes];   // 0 or an infinity, and 15 zeros, for each state of a K stage
    Pair pair[kPairs];
    uint64_t pair_full[kPairs], pair_empty[kPairs];
    uint64_t q_full[TILES], q_empty[TILES], kv_full[kStages], kv_empty[kStages], ready[kStages];
    uint64_t s_full[TILES], p_ready[TILES], o_full[TILES], done;
    uint32_t tmem_base;
    int abort_flag;
};

struct Maps {
    CUtensorMap q, k, v;
};

// CUT: items are cut along their states, and the sums joined afterwards (as a
// branch in the one kernel this cost whole items 2%).
template <typename T, int BOXES, int TILES, bool CUT>
__global__ void __launch_bounds__(128 + 128 * TILES, 3 - TILES)
    forward_kernel(const __grid_constant__ AttentionLaunch L, const __grid_constant__ Maps M, int rows_per_tile,
                   long long tiles, unsigned long long *counter, Split cut, int out_rows, float *part_o, float2 *part_ml) {
    extern __shared__ uint8_t smem_raw[];
    using Smem = Storage<BOXES, TILES>;
    constexpr int kStages = Smem::kStages, kThreads = 128 + 128 * TILES;
    constexpr uint32_t kColumns = TILES * 256, kO = TILES * 128;   // of TMEM: the tiles' scores, then their sums
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < TILES; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_ready[i], 4);
            mbar_init(&sm.o_full[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.kv_full[i], 1);
            mbar_init(&sm.kv_empty[i], 1);
            mbar_init(&sm.ready[i], 1);
        }
        for (int i = 0; i < kPairs; ++i) {
            mbar_init(&sm.pair_full[i], 1);
            mbar_init(&sm.pair_empty[i], 3 + 4 * TILES);   // warps 0 to 2 and the softmax warps read it
        }
        mbar_init(&sm.done, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&M.q);
        prefetch_tmap(&M.k);
        prefetch_tmap(&M.v);
    }
    if (warp == 1) tmem_alloc(&sm.tmem_base, kColumns);
    for (uint32_t i = threadIdx.x; i < kColumnBytes / 16; i += kThreads) {
        const uint32_t at = i * 16;
        st_shared_v4(smem_u32(sm.ones) + at, at < 2048 ? Type<T>::one : 0u, 0, 0, 0);
        for (int k = 0; k < kStages / 2; ++k) st_shared_v4(smem_u32(sm.left_out[k]) + at, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    const uint32_t tmem = sm.tmem_base;
    volatile int *abort_flag = &sm.abort_flag;
    const int group = L.group, dim = L.head_dim, span = TILES * rows_per_tile;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, abort_flag, L.status); };
    auto wait_one = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, L.status); };   // a thread's
    // The next published pair, for a reader; false where there is none or the CTA gave up.
    auto next_pair = [&](uint32_t it, Pair &p) {
        if (!wait(&sm.pair_full[it % kPairs], (it / kPairs) & 1)) return false;
        p = sm.pair[it % kPairs];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pair_empty[it % kPairs]);
        return p.rows >= 0;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        uint32_t entry = 0, q_phase = 0;
        bool ok = true;
        const uint32_t q_bytes = BOXES * static_cast<uint32_t>(rows_per_tile * group) * 128u;
        Pair p;
        for (uint32_t it = 0; ok && next_pair(it, p); ++it) {
            const int blocks = (p.nk + 127) / 128, nt = TILES == 2 && p.rows > rows_per_tile ? 2 : 1;
            if (lane == 0 && blocks) {
                auto load = [&](uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int head, int row) {
#pragma unroll
                    for (int b = 0; b < BOXES; ++b) tma_load_3d(dst + b * kBoxBytes, map, bar, 64 * b, head, row);
                };
                auto load_q = [&](int t) {
                    if (!wait_one(&sm.q_empty[t], ((q_phase >> t) & 1) ^ 1)) return false;
                    q_phase ^= 1u << t;
                    mbar_arrive_expect_tx(&sm.q_full[t], q_bytes);
                    load(sm.q[t], &M.q, &sm.q_full[t], p.head * group, p.q0 + t * rows_per_tile);
                    return true;
                };
                auto load_kv = [&](const CUtensorMap *map, int j) {
                    const uint32_t s = entry % kStages;
                    if (!wait_one(&sm.kv_empty[s], ((entry / kStages) & 1) ^ 1)) return false;
                    mbar_arrive_expect_tx(&sm.kv_full[s], BOXES * kBoxBytes);
                    load(sm.kv[s], map, &sm.kv_full[s], p.head, p.k0 + 128 * j);
                    ++entry;
                    return true;
                };
                ok = load_q(0) && load_kv(&M.k, 0) && (nt == 1 || load_q(1)) && load_kv(&M.v, 0);
                for (int j = 1; j < blocks && ok; ++j) ok = load_kv(&M.k, j) && load_kv(&M.v, j);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // Let the loads in flight land before the CTA can exit.
        if (lane == 0)
            for (int s = 0; s < kStages; ++s) {
                // the last use of stage s: entry - 1 - ((entry - 1 - s) mod kStages), where there is one
                if (entry > static_cast<uint32_t>(s)) {
                    const uint32_t last = (entry - 1 - s) / kStages;
                    wait_one(&sm.kv_empty[s], last & 1);
                }
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        // N by block; with a negative scale the scores are negated here, so that their maximum is the row's
        const uint32_t idesc_s = idesc_16bit(Type<T>::bf16, 128, 0, 0, 0) | (L.scale < 0.0f ? kIdescNegateA : 0u);
        const uint32_t idesc_o = idesc_16bit(Type<T>::bf16, 128, round16(dim), 0, 1);
        const uint64_t q_desc = desc_rows(smem_u32(sm.q[0])), k_desc = desc_rows(smem_u32(sm.kv[0]));
        const uint64_t v_desc = desc_sum(smem_u32(sm.kv[0]));
        const uint64_t ones_desc = desc_column(smem_u32(sm.ones)), out_desc = desc_column(smem_u32(sm.left_out[0]));
        constexpr uint64_t kTile = desc_bytes(BOXES * kBoxBytes);
        const int steps = (dim + 15) / 16;
        const uint32_t leader = elected(), tm = uniform(tmem);
        uint32_t entry = 0, q_phase = 0, p_phase = 0;
        bool ok = true;
        Pair p;
        for (uint32_t it = 0; ok && next_pair(it, p); ++it) {
            const int nk = static_cast<int>(uniform(p.nk)), rows = static_cast<int>(uniform(p.rows));
            const int blocks = (nk + 127) / 128, nt = TILES == 2 && rows > rows_per_tile ? 2 : 1;
            if (blocks == 0) continue;
            auto scores = [&](int t, int j, uint32_t e) {
                const uint32_t n = (min(128, nk - 128 * j) + 31) & ~31;
                mma_rows<BOXES>(leader, tm + t * 128, q_desc + t * kTile, k_desc + (e % kStages) * kTile,
                                idesc_s | (n >> 3) << 17, steps);
                if (L.key_mask || nk - 128 * j < 128)
                    issue_ss(leader, tm + t * 128, ones_desc, out_desc + (e % kStages) / 2 * desc_bytes(kColumnBytes),
                             idesc_s | (n >> 3) << 17, 1);
                issue_commit(leader, &sm.s_full[t]);
                if (j + 1 == blocks) issue_commit(leader, &sm.q_empty[t]);
            };
            ok = wait(&sm.ready[entry % kStages], (entry / kStages) & 1);
            for (int t = 0; t < nt && ok; ++t) {
                ok = wait(&sm.q_full[t], (q_phase >> t) & 1);
                if (!ok) break;
                q_phase ^= 1u << t;
                tc_fence_after();
                scores(t, 0, entry);
            }
            if (ok) issue_commit(leader, &sm.kv_empty[entry % kStages]);
            for (int j = 0; j < blocks && ok; ++j) {
                const uint32_t ev = entry + 2 * j + 1, ek = ev + 1;
                ok = wait(&sm.ready[ev % kStages], (ev / kStages) & 1);
                for (int t = 0; t < nt && ok; ++t) {
                    if (!wait(&sm.p_ready[t], (p_phase >> t) & 1)) { ok = false; break; }
                    p_phase ^= 1u << t;
                    tc_fence_after();
                    mma_pairs<8>(leader, tm + kO + t * 128, tm + t * 128, v_desc + (ev % kStages) * kTile, idesc_o,
                                 min(128, nk - 128 * j), j != 0);
                    if (j + 1 == blocks) {
                        issue_commit(leader, &sm.o_full[t]);
                    } else {
                        if (t == 0 && !wait(&sm.ready[ek % kStages], (ek / kStages) & 1)) { ok = false; break; }
                        tc_fence_after();
                        scores(t, j + 1, ek);
                    }
                }
                if (!ok) break;
                issue_commit(leader, &sm.kv_empty[ev % kStages]);
                if (j + 1 < blocks) issue_commit(leader, &sm.kv_empty[ek % kStages]);
            }
            entry += 2 * blocks;
        }
        issue_commit(leader, &sm.done);
        wait(&sm.done, 0);
    } else if (warp == 2) {
        // ------------------------------------------------------------ blocks made safe, dropped states
        uint32_t entry = 0;
        bool ok = true;
        // -infinity, or its negative where the scores' product is negated
        const uint16_t infinity = Type<T>::infinity | (L.scale < 0.0f ? 0u : 0x8000u);
        Pair p;
        for (uint32_t it = 0; ok && next_pair(it, p); ++it) {
            const int blocks = (p.nk + 127) / 128;
            for (int j = 0; j < blocks && ok; ++j, entry += 2) {
                const int n = min(128, p.nk - 128 * j);
                uint32_t keep[4];
                kept_bits(L, p.k0 + 128 * j, n, lane, keep);
                const uint32_t sk = entry % kStages, sv = (entry + 1) % kStages;
                // Scores are taken 32 at a time: the rows up to there have to be numbers.
                if (!wait(&sm.kv_full[sk], (entry / kStages) & 1)) { ok = false; break; }
                if (L.key_mask || n < 128) {   // the products that read this column last are done: the stage was free
                    const uint32_t column = smem_u32(sm.left_out[sk / 2]);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint16_t v = (keep[w] >> lane) & 1u ? 0 : infinity;
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(column + (32 * w + lane) * 16), "h"(v) : "memory");
                    }
                }
                zero_rows<BOXES>(smem_u32(sm.kv[sk]), (n + 31) & ~31, keep, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ready[sk]);
                if (!wait(&sm.kv_full[sv], ((entry + 1) / kStages) & 1)) { ok = false; break; }
                zero_rows<BOXES>(smem_u32(sm.kv[sv]), (n + 31) & ~31, keep, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ready[sv]);
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ work
        const int per_item = L.q_off ? 0 : (L.query_rows + span - 1) / span, batch = batch_of(tiles);
        uint32_t it = 0;
        bool ok = true;
        auto publish = [&](const Pair &p) {
            if (!wait(&sm.pair_empty[it % kPairs], ((it / kPairs) & 1) ^ 1)) return false;
            if (lane == 0) {
                sm.pair[it % kPairs] = p;
                mbar_arrive(&sm.pair_full[it % kPairs]);
            }
            ++it;
            return true;
        };
        auto hand_out = [&](long long base, int known) {
            const long long id = base + lane;
            Item t;
            int r0 = 0;
            long long block = id / L.key_heads;
            const int head = static_cast<int>(id - block * L.key_heads);
            int part = 0;
            if constexpr (CUT) {
                const long long whole = block / cut.parts;
                part = static_cast<int>(block - whole * cut.parts);
                block = whole;
            }
            const bool on = lane < batch && id < tiles && find_block(L, L.q_off, span, per_item, false, block, t, r0, known);
            if constexpr (CUT) {
                if (on) part_of(cut, part, t);
            }
            for (uint32_t left = __ballot_sync(0xffffffffu, on); left && ok; left &= left - 1) {
                const int from = __ffs(left) - 1;
                Pair p = {t.q0 + r0, part * out_rows + t.o0 + r0, min(span, t.nq - r0), t.k0, t.nk, head};
                p.q0 = __shfl_sync(0xffffffffu, p.q0, from);
                p.o0 = __shfl_sync(0xffffffffu, p.o0, from);
                p.rows = __shfl_sync(0xffffffffu, p.rows, from);
                p.k0 = __shfl_sync(0xffffffffu, p.k0, from);
                p.nk = __shfl_sync(0xffffffffu, p.nk, from);
                p.head = __shfl_sync(0xffffffffu, p.head, from);
                ok = publish(p);
            }
        };
        auto more = [&]() {
            unsigned long long base = 0;
            if (lane == 0) base = atomicAdd(counter, static_cast<unsigned long long>(batch));
            return static_cast<long long>(__shfl_sync(0xffffffffu, base, 0));
        };
        if (batch == 1) {
            // Few pairs a CTA: the way to its first product counts.  The first is its own, without the counter, and
            // the warp searches together (512 items of 32 x 512 rows, 4 key heads of 64: 95 -> 83 us).
            for (long long base = blockIdx.x; ok && base < tiles; base = more() + gridDim.x)
                hand_out(base, L.q_off ? find_item(L.q_off, L.items, span, base / L.key_heads / (CUT ? cut.parts : 1), lane) : -1);
        } else {
            for (long long base = more(); ok && base < tiles; base = more()) hand_out(base, -1);
        }
        if (ok) publish({0, 0, -1, 0, 0, 0});
        check_items(L, static_cast<long long>(blockIdx.x) * 32 + lane, static_cast<long long>(gridDim.x) * 32);
    } else {
        // ------------------------------------------------------------ softmax
        const int t = (warp - 4) >> 2, quad = warp & 3, m_row = quad * 32 + lane;
        const int r_in = m_row / group, head_in = m_row - r_in * group;
        const bool in_tile = r_in < rows_per_tile;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + kO + t * 128;
        const float sl2 = fmaxf(fabsf(L.scale) * kLog2e, 1e-30f);   // above 0, so that -infinity stays that
        const float lazy = 8.0f / sl2;   // in units of a raw score
        const float2 sl22 = make_float2(sl2, sl2);
        uint32_t phase = 0, o_phase = 0;
        bool ok = true;
        Pair p;
        for (uint32_t it = 0; ok && next_pair(it, p); ++it) {
            const int blocks = (p.nk + 127) / 128;
            if (t * rows_per_tile >= p.rows) continue;
            const int row = t * rows_per_tile + r_in;
            const bool mine = in_tile && row < p.rows;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < blocks; ++j) {
                if (!wait(&sm.s_full[t], phase)) { ok = false; break; }
                phase ^= 1;
                tc_fence_after();
                const int n = min(128, p.nk - 128 * j);
                // The maximum of the scores, the first two chunks of 32 staying in registers.
                uint32_t a[32], b[32];
                float top = -INFINITY, top1 = -INFINITY;
                if (n > 64) {
                    tmem_ld32_max_async(s_at + 64, a, top);
                    if (n > 96) tmem_ld32_max_async(s_at + 96, b, top1);
                    tmem_wait_ld();
                    tmem_regs_ready(a, top);
                    tmem_regs_ready(b, top1);
                    top = fmaxf(top, top1);
                    top1 = -INFINITY;
                }
                {
                    float top2;
                    tmem_ld32_max_async(s_at, a, top2);
                    if (n > 32) tmem_ld32_max_async(s_at + 32, b, top1);
                    tmem_wait_ld();
                    tmem_regs_ready(a, top2);
                    tmem_regs_ready(b, top1);
                    top = fmaxf(fmaxf(top, top1), top2);
                }
                // The reference follows the maximum only when that has grown past 2^8, in some row of the item's: rows of
                // the tile that are another's, or hold what was there before, have no say in it.
                if (__any_sync(0xffffffffu, mine && (top > m + lazy || (m == -INFINITY && top > m)))) {
                    const float m1 = fmaxf(m, top);
                    const float c = m1 > m ? ex2((m - m1) * sl2) : 1.0f;
                    m = m1;
                    l *= c;
                    if (j > 0) {   // S of this block is ready, so the product before it is done
#pragma unroll 1
                        for (int x = 0; x < BOXES * 64; x += 32) {
                            uint32_t o[32];
                            tmem_ld32_async(o_at + x, o);
                            tmem_wait_ld();
                            tmem_regs_ready(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * c);
                            tmem_st32(o_at + x, o);
                            tmem_wait_st();
                        }
                    }
                }
                // The weights, stored over the scores as these are done with: chunk w's 16 words end before
                // chunk w + 1's scores begin.
                const float at0 = m == -INFINITY ? 0.0f : -m * sl2;
                const float2 shift = make_float2(at0, at0);
                float2 sum = make_float2(0.0f, 0.0f), sum1 = sum;
                auto weights = [&](const uint32_t (&r)[32], int w) {
                    uint32_t packed[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), sl22, shift);
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), sl22, shift);
                        x = make_float2(ex2(x.x), ex2(x.y));
                        y = make_float2(ex2(y.x), ex2(y.y));
                        sum = __fadd2_rn(sum, x);
                        sum1 = __fadd2_rn(sum1, y);
                        packed[i / 2] = Type<T>::pack(x.x, x.y);
                        packed[i / 2 + 1] = Type<T>::pack(y.x, y.y);
                    }
                    tmem_st16(s_at + 16 * w, packed);
                };
                weights(a, 0);
                if (n > 64) tmem_ld32_async(s_at + 64, a);
                if (n > 32) weights(b, 1);
                if (n > 64) {
                    tmem_wait_ld();
                    tmem_regs_ready(a);
                    if (n > 96) tmem_ld32_async(s_at + 96, b);
                    weights(a, 2);
                }
                if (n > 96) {
                    tmem_wait_ld();
                    tmem_regs_ready(b);
                    weights(b, 3);
                }
                l += (sum.x + sum1.x) + (sum.y + sum1.y);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_ready[t]);
            }
            if (!ok) break;
            if (blocks) {
                if (!wait(&sm.o_full[t], o_phase)) break;
                o_phase ^= 1;
                tc_fence_after();
            }
            const int head = p.head * group + head_in;
            __syncwarp();
            if constexpr (CUT) {   // the sums as they are, and what they are relative to
                const long long cell = (static_cast<long long>(p.o0) + row) * L.query_heads + head;
                store_partials(o_at, dim, 1.0f, blocks != 0, mine, part_o + cell * dim);
                if (mine) part_ml[cell] = make_float2(m * sl2, l);
            } else {
                T *out = static_cast<T *>(L.o.data) + (static_cast<long long>(p.o0) + row) * L.o.row + head * L.o.head;
                store_sums<T>(o_at, dim, 1.0f / l, blocks != 0, l == 0.0f, mine, out);   // no kept state: zero
                if (L.lse && mine)
                    L.lse[(static_cast<long long>(p.o0) + row) * L.query_heads + head] =
                        l == 0.0f ? -INFINITY : m * (sl2 * kLn2) + logf(l);
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kColumns);
}

// Joins the parts of each row in their order: a warp a row and head.
template <typename T>
__global__ void __launch_bounds__(256)
    join_parts_kernel(const __grid_constant__ AttentionLaunch L, int parts, int out_rows, const float *part_o, const float2 *part_ml) {
    after_previous();
    const long long cells = static_cast<long long>(out_rows) * L.query_heads;
    const long long cell = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, dim = L.head_dim, d = 4 * lane;
    if (cell >= cells) return;
    const float2 mine = lane < parts ? part_ml[lane * cells + cell] : make_float2(-INFINITY, 0.0f);
    float m = mine.x;
    for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float c = lane < parts ? ex2(mine.x - (m == -INFINITY ? 0.0f : m)) : 0.0f;
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const float cp = __shfl_sync(0xffffffffu, c, p), lp = __shfl_sync(0xffffffffu, mine.y, p);
        l = fmaf(lp, cp, l);
        if (d < dim) {
            const float4 v = *reinterpret_cast<const float4 *>(part_o + (p * cells + cell) * dim + d);
            o.x = fmaf(v.x, cp, o.x), o.y = fmaf(v.y, cp, o.y), o.z = fmaf(v.z, cp, o.z), o.w = fmaf(v.w, cp, o.w);
        }
    }
    const long long row = cell / L.query_heads;
    const int head = static_cast<int>(cell - row * L.query_heads);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // no kept state: zero
    if (d < dim)
        *reinterpret_cast<uint2 *>(static_cast<T *>(L.o.data) + row * L.o.row + head * L.o.head + d) =
            make_uint2(Type<T>::pack(o.x * inv, o.y * inv), Type<T>::pack(o.z * inv, o.w * inv));
    if (L.lse && lane == 0) L.lse[cell] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
}

int output_rows(const AttentionLaunch &L) { return L.query_rows * (L.q_off ? 1 : L.items); }

// How a call is cut: tiles a CTA, slots of blocks of queries, parts along the states.
struct Cut {
    int tiles;
    long long slots;
    Split split;
};

// Two tiles a CTA share K and V, which is what long queries need (32 x 2048 x
// 1024 rows, 16 heads of 128: 431 us against 521 with one tile a CTA, two CTAs
// an SM; 64 x 512 x 1024, 8 heads of 64: 99 against 106).  One tile a CTA serves
// narrow heads, for which two CTAs of the full ring fit an SM, in items of two
// and a half tiles or less on average (64 x 200 x 1024, 8 heads of 64: 72 us
// against 80; 64 x 300: 88 against 92; 64 of 1 to 512 x 1 to 1024: 62 against
// 66, of 1 to 700: 73 against 72; at heads of 128 the short ring loses what the
// second CTA gains: 64 of 1 to 512: 90 against 78),
// and calls with less than a pair for every other SM (1 x 2048 x 2048 rows, 2
// heads: 35 us against 38, whole).
Cut cut_of(const AttentionLaunch &L) {
    const bool one = static_cast<long long>(output_rows(L)) * L.group <= 320ll * L.items && L.head_dim <= 64;
    const bool small = (static_cast<long long>(output_rows(L)) * L.group / 256 + 1) * L.key_heads <= 76;
    Cut c;
    c.tiles = one || small ? 1 : 2;
    const long long span = c.tiles * (128 / L.group);
    c.slots = L.q_off ? L.query_rows / span + L.items : static_cast<long long>(L.items) * ((L.query_rows + span - 1) / span);
    // at least so many blocks are there: half of the slots may be empty
    const long long filled = (output_rows(L) + span - 1) / span;
    c.split = split_of(L, (filled > L.items ? filled : L.items) * L.key_heads, 152 * (3 - c.tiles), 512);
    return c;
}

size_t part_bytes(const AttentionLaunch &L, const Cut &c) {
    return align256(static_cast<size_t>(c.split.parts) * output_rows(L) * L.query_heads * L.head_dim * sizeof(float));
}

long long joins_of(const AttentionLaunch &L) { return (static_cast<long long>(output_rows(L)) * L.query_heads + 7) / 8; }

template <typename T, int BOXES, int TILES, bool CUT>
cudaError_t launch(const AttentionLaunch &L, const Cut &c, cudaStream_t stream) {
    const int rows_per_tile = 128 / L.group, out_rows = output_rows(L);
    const long long tiles = c.slots * c.split.parts * L.key_heads;
    Maps M;
    const bool bf16 = Type<T>::bf16;
    if (!encode_heads_tiles(&M.q, L.q, bf16, L.head_dim, L.query_heads, L.query_rows, L.group, rows_per_tile) ||
        !encode_heads_tiles(&M.k, L.k, bf16, L.head_dim, L.key_heads, L.key_rows, 1, kTileRows) ||
        !encode_heads_tiles(&M.v, L.v, bf16, L.head_dim, L.key_heads, L.key_rows, 1, kTileRows))
        return cudaErrorInvalidValue;
    const size_t smem = sizeof(Storage<BOXES, TILES>) + 1024;
    auto kernel = forward_kernel<T, BOXES, TILES, CUT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const long long ctas = static_cast<long long>(L.sm_count) * (3 - TILES);
    unsigned long long *counters = reinterpret_cast<unsigned long long *>(L.workspace);
    float *part_o = reinterpret_cast<float *>(L.workspace + kCounterBytes);
    float2 *part_ml = reinterpret_cast<float2 *>(L.workspace + kCounterBytes + part_bytes(L, c));
    begin_kernel<<<1, 32, 0, stream>>>(L.status, counters);
    e = launch_after(kernel, dim3(static_cast<unsigned>(tiles < ctas ? tiles : ctas)), 128 + 128 * TILES, smem, stream, L, M,
                     rows_per_tile, tiles, counters, c.split, out_rows, part_o, part_ml);
    if (e != cudaSuccess || !CUT) return e;
    return launch_after(join_parts_kernel<T>, dim3(static_cast<unsigned>(joins_of(L))), 256, 0, stream, L, c.split.parts,
                        out_rows, part_o, part_ml);
}

template <typename T, int BOXES, int TILES>
cudaError_t launch(const AttentionLaunch &L, const Cut &c, cudaStream_t stream) {
    return c.split.parts > 1 ? launch<T, BOXES, TILES, true>(L, c, stream) : launch<T, BOXES, TILES, false>(L, c, stream);
}

template <typename T>
cudaError_t dispatch(const AttentionLaunch &L, cudaStream_t stream) {
    const Cut c = cut_of(L);
    if (L.head_dim > 64) return c.tiles == 1 ? launch<T, 2, 1>(L, c, stream) : launch<T, 2, 2>(L, c, stream);
    return c.tiles == 1 ? launch<T, 1, 1>(L, c, stream) : launch<T, 1, 2>(L, c, stream);
}

}  // namespace

long long forward_tiles_joins(const AttentionLaunch &L) { return cut_of(L).split.parts == 1 ? 0 : joins_of(L); }

size_t forward_tiles_workspace(const AttentionLaunch &L) {
    const Cut c = cut_of(L);
    if (c.split.parts == 1) return kCounterBytes;
    return kCounterBytes + part_bytes(L, c) +
           align256(static_cast<size_t>(c.split.parts) * output_rows(L) * L.query_heads * sizeof(float2));
}

// Needs at least one query row and one state (the tensor maps have no empty form).
cudaError_t launch_forward_tiles(const AttentionLaunch &L, cudaStream_t stream) {
    return L.dtype == CLI_BF16 ? dispatch<__nv_bfloat16>(L, stream) : dispatch<__half>(L, stream);
}

}  // namespace attn
}  // namespace cli
