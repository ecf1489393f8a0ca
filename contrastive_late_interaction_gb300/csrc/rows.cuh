// What the kernels over whole rows share (layer norm, dropout, the residual
// join): chunks of a row, the counter-based generator behind dropout, and the
// teams of lanes or warps that take a row together.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "cli_device.cuh"
#include "cli_internal.h"
#include "launch.cuh"

namespace cli {
namespace rows {

// ----------------------------------------------------------------------------
// chunks: E consecutive elements of a row, as they lie in memory
// ----------------------------------------------------------------------------

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
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

// How a call's rows can be moved: whole chunks (aligned to their size, and the
// rows a multiple of it), else the widest pieces that their alignment allows,
// words of 4 bytes or halves of 2.
enum Moves { kWhole = 0, kWords = 1, kHalves = 2 };

template <typename T, int E>
struct Chunk {
    static constexpr int kBytes = E * static_cast<int>(sizeof(T)), kWords4 = kBytes / 4;
    static_assert(kBytes == 8 || kBytes == 16, "a chunk is one access");
    uint32_t w[kWords4];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords4; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kBytes == 8) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1] = u.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kBytes == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }

    __device__ __forceinline__ void floats(float2 (&v)[E / 2]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = unpack2<T>(w[i]);
        }
    }
    __device__ __forceinline__ void set(const float2 (&v)[E / 2]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[2 * i] = __float_as_uint(v[i].x), w[2 * i + 1] = __float_as_uint(v[i].y);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[i] = pack2<T>(v[i].x, v[i].y);
        }
    }
};

// Where the elements of a thread's chunks lie in a row of `width`.  The lanes of
// a warp that take the row together, `part` of them, have chunks side by side,
// a chunk being
//   whole: E neighbouring elements, one access;
//   else:  pieces of kPiece elements, each next to the other lanes' pieces, so
//          that an access of the warp's covers whole lines all the same (a
//          thread's words side by side would be written as four parts of every
//          32 bytes: 20011 fp32 rows of 771 took 39 us where these take 31).
// PART: `part` where it is known, else 0.
template <typename T, int E, int MOVES, int PART>
struct Layout {
    static constexpr int kPiece = MOVES == kWhole ? E : MOVES == kWords && sizeof(T) == 2 ? 2 : 1, kPieces = E / kPiece;
    int part_, lane, column;   // column: of the first chunk's first element
    __device__ __forceinline__ Layout(int part, int lane_, int start) : part_(part), lane(lane_), column(start + lane_ * kPiece) {}
    __device__ __forceinline__ int part() const { return PART ? PART : part_; }
    __device__ __forceinline__ int chunk(int j) const { return j * part() * E; }        // from `column`
    __device__ __forceinline__ int piece(int k) const { return k * part() * kPiece; }   // from the chunk's first
    __device__ __forceinline__ int element(int j, int i) const { return column + chunk(j) + piece(i / kPiece) + i % kPiece; }
    // The first column of the i-th block of four columns that a lane draws for chunk j: its own, or where a block lies with
    // several lanes, the one of the piece that is the lane's to draw.
    __device__ __forceinline__ int drawer() const { return lane & (kPieces - 1); }
    __device__ __forceinline__ int first_of(int j, int i) const {
        return kPieces == 1 ? column + chunk(j) + 4 * i : ((column + chunk(j)) & ~3) + piece(drawer());
    }
    // Bit j * kPieces + k: piece k of chunk j is there (a piece is wholly there or not at all).
    template <int C>
    __device__ __forceinline__ uint32_t there(int width) const {
        static_assert(C * kPieces <= 32, "");
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int k = 0; k < kPieces; ++k) bits |= column + chunk(j) + piece(k) < width ? 1u << (j * kPieces + k) : 0u;
        return bits;
    }
    // A float of a vector for each element of chunk j; what lies past it, or its absence, is `otherwise`.
    __device__ __forceinline__ void vector(const float *p, int j, int width, float otherwise, float2 (&v)[E / 2]) const {
        const int at = column + chunk(j);   // a multiple of 4 where chunks are whole
        if (MOVES == kWhole && p && at < width && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(p + at + i));
                v[i / 2] = make_float2(f.x, f.y), v[i / 2 + 1] = make_float2(f.z, f.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const int a = element(j, i), b = element(j, i + 1);
                v[i / 2] = make_float2(p && a < width ? __ldg(p + a) : otherwise, p && b < width ? __ldg(p + b) : otherwise);
            }
        }
    }
    // A chunk as it was loaded: halves a register each, so that nothing waits for them before they are put together.
    template <typename M>
    struct Raw {
        static constexpr bool kApart = MOVES == kHalves && sizeof(M) == 2;
        uint32_t w[kApart ? E : Chunk<M, E>::kWords4];
        __device__ __forceinline__ Chunk<M, E> chunk() const {
            Chunk<M, E> c;
#pragma unroll
            for (int i = 0; i < Chunk<M, E>::kWords4; ++i) c.w[i] = kApart ? __byte_perm(w[kApart ? 2 * i : i], w[kApart ? 2 * i + 1 : i], 0x5410) : w[i];
            return c;
        }
    };
    // The pieces of a chunk that `there` names (from bit 0), at p, which is the chunk's first element; the others are 0.
    template <typename M>
    __device__ __forceinline__ void load(Raw<M> &c, const M *p, uint32_t there) const {
        if constexpr (MOVES == kWhole) {
            Chunk<M, E> whole;
            whole.clear();
            if (there & 1u) whole.load(p);
#pragma unroll
            for (int i = 0; i < Chunk<M, E>::kWords4; ++i) c.w[i] = whole.w[i];
        } else if constexpr (Raw<M>::kApart) {
#pragma unroll
            for (int k = 0; k < E; ++k) c.w[k] = there >> k & 1u ? *reinterpret_cast<const uint16_t *>(p + piece(k)) : 0u;
        } else {
            constexpr int kWords4 = kPiece * static_cast<int>(sizeof(M)) / 4;   // of a piece
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
#pragma unroll
                for (int w = 0; w < kWords4; ++w)
                    c.w[k * kWords4 + w] = there >> k & 1u ? reinterpret_cast<const uint32_t *>(p + piece(k))[w] : 0u;
        }
    }
    template <typename M>
    __device__ __forceinline__ void store(const Chunk<M, E> &c, M *p, uint32_t there) const {
        if constexpr (MOVES == kWhole) {
            if (there & 1u) c.store(p);
        } else {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                if (!(there >> k & 1u)) continue;
                M *to = p + piece(k);
                if constexpr (sizeof(M) == 4) {
#pragma unroll
                    for (int i = 0; i < kPiece; ++i) reinterpret_cast<uint32_t *>(to)[i] = c.w[k * kPiece + i];
                } else if constexpr (kPiece == 2) {
                    *reinterpret_cast<uint32_t *>(to) = c.w[k];
                } else {
                    *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(c.w[k / 2] >> (16 * (k & 1)));
                }
            }
        }
    }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// A thread's chunks of one matrix of type M, N a step, on their way to it
// through its own places in shared memory.  No other thread reads those, so
// that the thread's own wait for its copies is all that a step needs.  Halves,
// which no asynchronous copy takes, wait in registers for one step: each in one
// of its own with APART, else put together as they come, which waits for them
// (rows of 771 in bf16: the join takes 289 us apart and 413 together, its
// gradient, which has no registers left, 543 and 442).
template <typename M, typename L, int E, int N, int MOVES, bool APART>
struct Feed {
    static constexpr bool kHeld = MOVES == kHalves && sizeof(M) == 2;
    // Copies of words go to places a word wide, a thread's side by side with the others', so that they meet no bank twice.
    static constexpr int kBytes = Chunk<M, E>::kBytes, kUnit = MOVES == kWhole || kHeld ? kBytes : 4, kUnits = kBytes / kUnit;
    uint32_t at;   // of chunk 0 of stage 0
    using Raw = typename L::template Raw<M>;
    std::conditional_t<APART, Raw, Chunk<M, E>> held[kHeld ? N : 1];

    // `base`: where the block's places for this matrix start, [stages][N][units][threads].  Places that no copy writes,
    // those past a row's end, are 0.
    __device__ __forceinline__ Feed(uint32_t base, int stages) {
        at = base + threadIdx.x * kUnit;
        for (int i = 0; i < stages * N * kUnits; ++i) {
            const uint32_t to = at + i * blockDim.x * kUnit;
            if constexpr (kUnit == 16)
                st_shared_v4(to, 0, 0, 0, 0);
            else if constexpr (kUnit == 8)
                asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(to), "r"(0) : "memory");
            else
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(0) : "memory");
        }
    }
    __device__ __forceinline__ uint32_t place(int stage, int i, int unit = 0) const {
        return at + ((stage * N + i) * kUnits + unit) * blockDim.x * kUnit;
    }
    // Chunk i of a step, whose first element is at p.
    __device__ __forceinline__ void copy(const L &layout, int stage, int i, const M *p, uint32_t there) {
        if constexpr (kHeld) {
            if constexpr (APART) {
                layout.load(held[i], p, there);
            } else {
                Raw raw;
                layout.load(raw, p, there);
                held[i] = raw.chunk();
            }
        } else if constexpr (MOVES == kWhole) {
            if (there & 1u) copy_async<kUnit>(place(stage, i), p);
        } else {
#pragma unroll
            for (int k = 0; k < L::kPieces; ++k) {
                if (!(there >> k & 1u)) continue;
                constexpr int kWords4 = L::kPiece * static_cast<int>(sizeof(M)) / 4;   // of a piece
#pragma unroll
                for (int w = 0; w < kWords4; ++w)
                    copy_async<4>(place(stage, i, k * kWords4 + w), reinterpret_cast<const uint32_t *>(p + layout.piece(k)) + w);
            }
        }
    }
    // What is held, to its stage.
    __device__ __forceinline__ void settle(int stage) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                Chunk<M, E> c;
                if constexpr (APART) c = held[i].chunk(); else c = held[i];
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(place(stage, i)), "r"(c.w[0]), "r"(c.w[1]) : "memory");
            }
        }
    }
    __device__ __forceinline__ Chunk<M, E> chunk(int stage, int i) const {
        Chunk<M, E> c;
        if constexpr (kUnit == 16) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]) : "r"(place(stage, i)) : "memory");
        } else if constexpr (kUnit == 8) {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(c.w[0]), "=r"(c.w[1]) : "r"(place(stage, i)) : "memory");
        } else {
#pragma unroll
            for (int k = 0; k < kUnits; ++k)
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(c.w[k]) : "r"(place(stage, i, k)) : "memory");
        }
        return c;
    }
    __device__ __forceinline__ void floats(int stage, int i, float2 (&v)[E / 2]) const { chunk(stage, i).floats(v); }
};

// ----------------------------------------------------------------------------
// dropout
// ----------------------------------------------------------------------------

// Philox 4x32 of ten rounds (Salmon, Moraes, Dror, Shaw: Parallel random
// numbers: as easy as 1, 2, 3; 2011): four words of 32 bits from a counter of
// four and a key of two.
constexpr uint32_t kMul0 = 0xD2511F53u, kMul1 = 0xCD9E8D57u, kWeyl0 = 0x9E3779B9u, kWeyl1 = 0xBB67AE85u;
__device__ __forceinline__ uint2 product(uint32_t a, uint32_t b) {   // x: the low word
    const uint64_t p = static_cast<uint64_t>(a) * b;
    return make_uint2(static_cast<uint32_t>(p), static_cast<uint32_t>(p >> 32));
}

// A call's mask as its kernels start: its seed and step are read from the device, so that a captured call draws another
// mask at each step.
struct Seed {
    uint32_t k0, k1, step0, step1;
    Seed() = default;
    __device__ __forceinline__ explicit Seed(const MaskLaunch &m) : k0(0), k1(0), step0(0), step1(0) {
        if (!m.least) return;
        const uint2 key = *reinterpret_cast<const uint2 *>(m.seed), step = *reinterpret_cast<const uint2 *>(m.seed + 1);
        k0 = key.x, k1 = key.y, step0 = step.x, step1 = step.y;
    }
    __device__ __forceinline__ uint32_t a(int i) const { return k0 + i * kWeyl0; }   // the rounds' keys
    __device__ __forceinline__ uint32_t b(int i) const { return k1 + i * kWeyl1; }
    // What the first round makes of the row, but for the row itself.
    __device__ __forceinline__ uint32_t row_word() const { return product(kMul1, step0).y ^ a(0); }
};

// What the first rounds make of a block's columns and of the step before the row has reached every word (counter: column
// block, row, step, step).  A multiplication of 32 x 32 to 64 bits goes out every fourth cycle, so that these decide what
// a mask costs: of 20 a block, 15 are left to each row, and one that the row's blocks share.
struct Block {
    uint32_t d, f, g, h;
    Block() = default;
    __device__ __forceinline__ Block(const Seed &s, uint32_t site, int column) {
        const uint2 p0 = product(kMul0, static_cast<uint32_t>(column >> 2) | site << 16), q0 = product(kMul1, s.step0);
        const uint2 q1 = product(kMul1, p0.y ^ s.step1 ^ s.b(0));
        const uint2 p2 = product(kMul0, q1.y ^ q0.x ^ s.a(1));
        d = p0.x ^ s.b(1), f = q1.x ^ s.a(2), g = p2.y ^ s.b(2), h = p2.x ^ s.b(3);
    }
};

// The words of N blocks of a row, round by round together.  `row`: the row's word, multiplied.  K gives the keys: a3 of
// round 3, and two(i) the a and b of rounds i and i + 1.
template <int N, typename K>
__device__ __forceinline__ void draw(const Block (&b)[N], const K &keys, uint2 row, uint4 (&c)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint2 q = product(kMul1, row.y ^ b[n].d);
        const uint32_t x = q.y ^ b[n].f, y = q.x, z = b[n].g ^ row.x;
        const uint2 p = product(kMul0, x);
        q = product(kMul1, z);
        c[n] = make_uint4(q.y ^ y ^ keys.a3, q.x, p.y ^ b[n].h, p.x);
    }
#pragma unroll
    for (int i = 4; i < 10; i += 2) {
        const uint4 k = keys.two(i);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint2 p = product(kMul0, c[n].x), q = product(kMul1, c[n].z);
            c[n] = make_uint4(q.y ^ c[n].y ^ k.x, q.x, p.y ^ c[n].w ^ k.y, p.x);
            p = product(kMul0, c[n].x), q = product(kMul1, c[n].z);
            c[n] = make_uint4(q.y ^ c[n].y ^ k.z, q.x, p.y ^ c[n].w ^ k.w, p.x);
        }
    }
}

// The words of a lane's elements from the blocks that it drew.  Where a block's four columns lie with several lanes, each
// of these draws another of their blocks, and they hand the words round: the lanes of such a group call this together.
template <typename L>
__device__ __forceinline__ void hand_round(const L &layout, uint4 &r) {
    if constexpr (L::kPieces > 1) {
        const int mine = layout.drawer();
        auto swap = [](uint32_t x, int o) { return __shfl_xor_sync(0xffffffffu, x, o); };
        if constexpr (L::kPieces == 4) {   // r: words x, y, z, w of block `mine`; then word `mine` of blocks 0 to 3
            uint32_t t = swap(mine & 1 ? r.x : r.y, 1), u = swap(mine & 1 ? r.z : r.w, 1);
            if (mine & 1) r.x = t, r.z = u; else r.y = t, r.w = u;
            t = swap(mine & 2 ? r.x : r.z, 2), u = swap(mine & 2 ? r.y : r.w, 2);
            if (mine & 2) r.x = t, r.y = u; else r.z = t, r.w = u;
        } else {   // then words 2 mine and 2 mine + 1 of blocks 0 and 1
            const uint32_t t = swap(mine ? r.x : r.z, 1), u = swap(mine ? r.y : r.w, 1);
            if (mine) r.x = t, r.y = u; else r.z = t, r.w = u;
        }
    }
}

// A chunk through its words: kept elements times scale, the others 0 whatever they hold.
template <int E>
__device__ __forceinline__ void keep(float2 (&v)[E / 2], const uint4 (&r)[E / 4], uint32_t least, float scale) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        const float2 a = __fmul2_rn(v[2 * i], make_float2(scale, scale)), b = __fmul2_rn(v[2 * i + 1], make_float2(scale, scale));
        v[2 * i] = make_float2(r[i].x >= least ? a.x : 0.0f, r[i].y >= least ? a.y : 0.0f);
        v[2 * i + 1] = make_float2(r[i].z >= least ? b.x : 0.0f, r[i].w >= least ? b.y : 0.0f);
    }
}

__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// ----------------------------------------------------------------------------
// teams
// ----------------------------------------------------------------------------

// Sums over a warp of N values, the same in each lane: with several, halves of the warp take some of them each
// and hand them round at the end, 9 shuffles for four sums instead of 20.
template <int N>
__device__ __forceinline__ void warp_sum(float (&v)[N]) {
    const uint32_t lane = threadIdx.x;
    auto swap = [](float x, int o) { return __shfl_xor_sync(0xffffffffu, x, o); };
    if constexpr (N == 1) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v[0] += swap(v[0], o);
    } else if constexpr (N == 2) {
        const bool upper = lane & 16;
        float t = (upper ? v[1] : v[0]) + swap(upper ? v[0] : v[1], 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) t += swap(t, o);
        const float u = swap(t, 16);
        v[0] = upper ? u : t, v[1] = upper ? t : u;
    } else if constexpr (N != 4) {   // as 4 or 2 and the rest: each the same sum as by itself
        constexpr int kHead = N > 4 ? 4 : 2;
        float head[kHead], rest[N - kHead];
#pragma unroll
        for (int i = 0; i < N; ++i) (i < kHead ? head[i < kHead ? i : 0] : rest[i < kHead ? 0 : i - kHead]) = v[i];
        warp_sum(head);
        warp_sum(rest);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < kHead ? head[i < kHead ? i : 0] : rest[i < kHead ? 0 : i - kHead];
    } else {
        const bool upper = lane & 16, odd = lane & 8;
        const float a = (upper ? v[2] : v[0]) + swap(upper ? v[0] : v[2], 16);
        const float b = (upper ? v[3] : v[1]) + swap(upper ? v[1] : v[3], 16);
        float t = (odd ? b : a) + swap(odd ? a : b, 8);
#pragma unroll
        for (int o = 4; o; o >>= 1) t += swap(t, o);
        const float u = swap(t, 8), lo = odd ? u : t, hi = odd ? t : u, lo2 = swap(lo, 16), hi2 = swap(hi, 16);
        v[0] = upper ? lo2 : lo, v[1] = upper ? hi2 : hi, v[2] = upper ? lo : lo2, v[3] = upper ? hi : hi2;
    }
}

// The lanes that take a row together: 2^k lanes of a warp, or whole warps.
struct Team {
    int lane, lanes;      // this thread's place, the team's size
    int index, count;     // the team's place among the grid's
    int first;            // the index of the warp's first team
    int id, in_block;     // its place in the block, the block's teams
    __device__ __forceinline__ explicit Team(int lanes_) : lanes(lanes_) {
        id = threadIdx.x / lanes;
        lane = threadIdx.x - id * lanes;
        in_block = blockDim.x / lanes;
        index = blockIdx.x * in_block + id;
        count = gridDim.x * in_block;
        first = lanes < 32 ? index - (threadIdx.x & 31) / lanes : index;
    }
    // Sums of N values over the team, the same in each lane, in a fixed order.  `scratch`: 16 * N floats of the team's own
    // in shared memory, 16-byte aligned, of two that calls alternate between (a team of several warps needs one barrier a
    // sum, then).  WARPS: the team is one warp or more.
    template <int N, bool WARPS>
    __device__ __forceinline__ void sum(float (&v)[N], float *scratch) const {
        if constexpr (!WARPS) {
            for (int o = 1; o < lanes; o <<= 1) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
            }
        } else {
            warp_sum(v);
            if (lanes > 32) {
                const int warps = lanes >> 5;
                if ((lane & 31) == 0) {
#pragma unroll
                    for (int i = 0; i < N; ++i) scratch[(lane >> 5) * N + i] = v[i];
                }
                named_barrier_sync(1 + id, lanes);
                if (warps == 2) {
#pragma unroll
                    for (int i = 0; i < N; ++i) v[i] = scratch[i] + scratch[N + i];
                } else {   // a warp's sums a lane
                    const int w = threadIdx.x & 31;
#pragma unroll
                    for (int i = 0; i < N; ++i) v[i] = w < warps ? scratch[w * N + i] : 0.0f;
                    warp_sum(v);
                }
            }
        }
    }
};

}  // namespace rows
}  // namespace cli
