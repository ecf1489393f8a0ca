// Cross attention of few query rows: pooling queries and single tokens.
//
// When an item has at most 16 rows of (query, head of the group), a pass over
// its states does a few operations a byte: HBM bounds it, and what counts is
// to keep enough loads in flight.  The unit of work is a warp with one key
// head and a chunk of an item's states.  It holds K, V and everything else in
// registers, with no shared-memory stage between HBM and the products, which
// are mma.sync with the states on the long side: 16 states x 8 rows.  (tcgen05
// works on 128 rows at a time, of which these calls fill a sixteenth or less,
// and takes its operands from shared memory or TMEM.)
//
// Fragments.  With g = lane / 4 and t = lane % 4, a lane's A registers of
// S^T = K Q^T hold states g and g + 8.  A product does not care in which order
// its inner index runs, so the index is dealt out such that a lane's part is
// one 16-byte load: elements 8 t .. 8 t + 7 of each 32 of the head.  Q's
// fragment is dealt out alike.  For O^T += V^T P^T the inner index is the
// state and a register holds a pair of states: lanes load 16 bytes of elements
// 8 g .. 8 g + 7 of states 2 t, 2 t + 1, 2 t + 8, 2 t + 9 and interleave them,
// so that a lane ends up with 8 neighbouring output elements of a row.  P
// comes out of the first product with states on g and goes into the second
// with states on t: an 8 x 8 transposition within the warp (movmatrix).
//
// The softmax follows attention_forward.cu: a running reference that moves
// when a score passes it by 2^8.  A score is compared in the lane that has it,
// and lanes reduce among themselves only when some score is past.
//
// Chunks.  Items longer than a chunk are split, and a second kernel joins the
// parts in a fixed order; results do not depend on the order of execution.
//
// Bound: HBM.  2048 items of 64 to 512 states, one shared query, 16 heads of
// 64: 364 us (6.6 TB/s); 512 of 32 to 1024, 8 heads of 128: 185 us (6.0 TB/s)
// and 432 for the backward (5.1 TB/s, reads and writes mixed; 413 without the
// noting and mending of dK).  One row against 4096 states, 8 heads on 2: 12 us in two
// launches, both latency.

#include "attention.cuh"

namespace cli {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kMostChunk = 512, kSteps = kMostChunk / 16;   // states of a unit; 16 are taken at a time

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (Type<T>::bf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Element (row g, columns 2 t, 2 t + 1) of an 8 x 8 matrix of 16-bit values -> (row g, ...) of its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 2^x with results down to the smallest subnormal.
__device__ __forceinline__ float ex2_full(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two values as a pair of 16-bit pairs that add up to them to twice the type's
// digits.  HBM bounds these kernels, so weights go into the products as both
// halves: their rounding would be half of the results' error.
template <typename T>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = Type<T>::pack(a, b);
    const float2 h = Type<T>::unpack(hi);
    lo = Type<T>::pack(a - h.x, b - h.y);
}

// The 16 bytes at p where `on`, else zeros.  Volatile, as the products are: a
// step's loads then all go out before its first product, however the compiler
// would like to save registers (the kernel below ran at 5.8 or at 6.5 TB/s as
// it chose).
__device__ __forceinline__ void load_if(bool on, const void *p, uint32_t (&r)[4]) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.u32 p, %5, 0;\n"
        " mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
        " @p ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];\n"
        "}\n"
        : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3])
        : "l"(p), "r"(static_cast<uint32_t>(on)));
}

// A warp's unit: states k0 .. k0 + n - 1 of an item for one key head.
struct Unit {
    Item item;
    long long slot;
    int k0, n, head, rows;   // rows: (query, head of the group) pairs; 0: nothing to do
};

__device__ __forceinline__ Unit find_unit(const AttentionLaunch &L, int chunk, long long slot, int head, int lane) {
    Unit u;
    u.slot = slot;
    u.head = head;
    int i;
    long long block;
    if (chunk >= L.max_k) {   // one chunk an item
        i = static_cast<int>(slot);
        block = 0;
    } else {
        i = find_item(L.k_off, L.items, chunk, slot, lane);
        block = slot - (static_cast<long long>(L.k_off[i] / chunk) + i);
    }
    u.item = load_item(L, i);
    const long long at = block * chunk;
    u.rows = u.item.nq * L.group;
    u.k0 = u.item.k0;
    u.n = 0;
    if (!u.item.ok || block < 0 || (at >= u.item.nk && block > 0)) {   // block 0 also writes an empty item's rows
        u.rows = 0;
        return u;
    }
    u.k0 += static_cast<int>(at);
    u.n = min(chunk, u.item.nk - static_cast<int>(at));
    return u;
}

// A call on few items has no memset of the status before it: block 0 checks
// every item and writes the word (what others report until then is what it
// will find).  With more items the grid shares the checks.
constexpr int kFewItems = 256;
__device__ __forceinline__ void check_all(const AttentionLaunch &L, bool reached) {
    if (L.items > kFewItems) {
        if (!reached)   // a unit looks at its item anyway, where each item has one
            check_items(L, static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x,
                        static_cast<long long>(gridDim.x) * blockDim.x);
    } else if (blockIdx.x == 0) {
        bool bad = false;
        for (int i = threadIdx.x; i < L.items; i += blockDim.x) bad |= !load_item(L, i).ok;
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *L.status = bad ? CLI_MALFORMED : CLI_OK;
    }
}

// The kept states among the `count` (at most 32) from k0, as bits.
__device__ __forceinline__ uint32_t kept(const AttentionLaunch &L, int k0, int count, int lane) {
    if (!L.key_mask) return count >= 32 ? 0xffffffffu : (1u << count) - 1u;
    return __ballot_sync(0xffffffffu, lane < count && L.key_mask[k0 + lane] != 0);
}

// Row `row` of the unit's packed rows in a matrix of query rows that starts at `first`.
template <typename T>
__device__ __forceinline__ T *row_ptr(const AttentionLaunch &L, const HeadsView &v, const Unit &u, int first, int row) {
    const int r = row / L.group, h = u.head * L.group + row - r * L.group;
    return static_cast<T *>(v.data) + static_cast<long long>(first + r) * v.row + h * v.head;
}

// ----------------------------------------------------------------------------
// forward
// ----------------------------------------------------------------------------

// DP: the head's elements, rounded up to 64 or 128.  NT: tiles of 8 rows.
// A step takes 8 KB of K and V: 16 states at DP 128, 32 at DP 64.
template <typename T, int DP, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 3)
    forward_kernel(const __grid_constant__ AttentionLaunch L, int chunk, long long slots, float *part_o, float2 *part_ml) {
    constexpr int KC = DP / 32, VB = DP / 64, KG = 128 / DP, kStep = 16 * KG;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel, if there is one
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long id = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    check_all(L, chunk >= L.max_k);
    if (id >= slots * L.key_heads) return;
    const Unit u = find_unit(L, chunk, id / L.key_heads, static_cast<int>(id % L.key_heads), lane);
    if (u.rows == 0) return;
    const int dim = L.head_dim;

    uint32_t q[NT][KC][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = 8 * n + g;
        const T *p = row_ptr<T>(L, L.q, u, u.item.q0, row < u.rows ? row : 0);
#pragma unroll
        for (int c = 0; c < KC; ++c) load_if(row < u.rows && 32 * c + 8 * t < dim, p + 32 * c + 8 * t, q[n][c]);
    }
    float o[VB][4][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[b][i][n][0] = o[b][i][n][1] = o[b][i][n][2] = o[b][i][n][3] = 0.0f;
    }
    const float sl2 = L.scale * kLog2e;
    const T *kbase = static_cast<const T *>(L.k.data) + u.head * L.k.head + 8 * t;
    const T *vbase = static_cast<const T *>(L.v.data) + u.head * L.v.head + 8 * g;

    for (int j = 0; j < u.n; j += kStep) {
        const uint32_t keep = kept(L, u.k0 + j, min(kStep, u.n - j), lane);
        uint32_t kr[KG][2][KC][4], vr[KG][4][VB][4];
#pragma unroll
        for (int x = 0; x < KG; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int s = 16 * x + 8 * y + g;
                const T *p = kbase + static_cast<long long>(u.k0 + j + s) * L.k.row;
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    load_if(((keep >> s) & 1u) && 32 * c + 8 * t < dim, p + 32 * c, kr[x][y][c]);
            }
#pragma unroll
        for (int x = 0; x < KG; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int s = 16 * x + 8 * (y >> 1) + 2 * t + (y & 1);
                const T *p = vbase + static_cast<long long>(u.k0 + j + s) * L.v.row;
#pragma unroll
                for (int b = 0; b < VB; ++b)
                    load_if(((keep >> s) & 1u) && 64 * b + 8 * g < dim, p + 64 * b, vr[x][y][b]);
            }
        // s[..][0..3]: (state g, rows 2t, 2t + 1), (state g + 8, rows 2t, 2t + 1), in powers of two
        float s[KG][NT][4];
        bool past = false;
#pragma unroll
        for (int x = 0; x < KG; ++x)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float c4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    mma16<T>(c4, kr[x][0][c][0], kr[x][1][c][0], kr[x][0][c][1], kr[x][1][c][1], q[n][c][0], q[n][c][1]);
                    mma16<T>(c4, kr[x][0][c][2], kr[x][1][c][2], kr[x][0][c][3], kr[x][1][c][3], q[n][c][2], q[n][c][3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = (keep >> (16 * x + 8 * (i >> 1) + g)) & 1u;
                    s[x][n][i] = on ? c4[i] * sl2 : -INFINITY;
                    past |= s[x][n][i] > m[n][i & 1] + 8.0f;   // also the first finite score: m is -infinity
                }
            }
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float top = m[n][r];
#pragma unroll
                    for (int x = 0; x < KG; ++x) top = fmaxf(top, fmaxf(s[x][n][r], s[x][n][r + 2]));
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                    const float c = top > m[n][r] ? ex2_full(m[n][r] - top) : 1.0f;
                    m[n][r] = top;
                    l[n][r] *= c;
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[b][i][n][r] *= c;
                            o[b][i][n][r + 2] *= c;
                        }
                }
        }
#pragma unroll
        for (int x = 0; x < KG; ++x) {
            uint32_t p[NT][4];   // high halves, then low ones
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float ref = m[n][i & 1] == -INFINITY ? 0.0f : m[n][i & 1];
                    e[i] = ex2_full(s[x][n][i] - ref);
                    l[n][i & 1] += e[i];
                }
                split_pair<T>(e[0], e[1], p[n][0], p[n][2]);
                split_pair<T>(e[2], e[3], p[n][1], p[n][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[n][i] = transpose8(p[n][i]);
            }
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = __byte_perm(vr[x][0][b][i], vr[x][1][b][i], 0x5410);
                    const uint32_t a1 = __byte_perm(vr[x][0][b][i], vr[x][1][b][i], 0x7632);
                    const uint32_t a2 = __byte_perm(vr[x][2][b][i], vr[x][3][b][i], 0x5410);
                    const uint32_t a3 = __byte_perm(vr[x][2][b][i], vr[x][3][b][i], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16<T>(o[b][i][n], a0, a1, a2, a3, p[n][0], p[n][1]);
                        mma16<T>(o[b][i][n], a0, a1, a2, a3, p[n][2], p[n][3]);
                    }
                }
        }
    }

#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float sum = l[n][r];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int row = 8 * n + 2 * t + r;
            if (row >= u.rows) continue;
            if (part_o) {
                const long long at = (u.slot * L.key_heads + u.head) * (static_cast<long long>(L.max_q) * L.group) + row;
                if (g == 0) part_ml[at] = make_float2(m[n][r], sum);
#pragma unroll
                for (int b = 0; b < VB; ++b) {
                    if (64 * b + 8 * g >= dim) continue;
                    float4 *p = reinterpret_cast<float4 *>(part_o + at * dim + 64 * b + 8 * g);
                    p[0] = make_float4(o[b][0][n][r], o[b][0][n][r + 2], o[b][1][n][r], o[b][1][n][r + 2]);
                    p[1] = make_float4(o[b][2][n][r], o[b][2][n][r + 2], o[b][3][n][r], o[b][3][n][r + 2]);
                }
            } else {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // no kept state: zero
                T *p = row_ptr<T>(L, L.o, u, u.item.o0, row);
#pragma unroll
                for (int b = 0; b < VB; ++b) {
                    if (64 * b + 8 * g >= dim) continue;
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = Type<T>::pack(o[b][i][n][r] * inv, o[b][i][n][r + 2] * inv);
                    *reinterpret_cast<uint4 *>(p + 64 * b + 8 * g) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (L.lse && g == 0) {
                    const int rr = row / L.group, h = u.head * L.group + row - rr * L.group;
                    L.lse[static_cast<long long>(u.item.o0 + rr) * L.query_heads + h] =
                        sum == 0.0f ? -INFINITY : m[n][r] * kLn2 + logf(sum);
                }
            }
        }
}

// Joins the parts of each row, four elements a lane, by W warps a row.
template <typename T, int W>
__global__ void __launch_bounds__(256)
    join_kernel(const __grid_constant__ AttentionLaunch L, int chunk, const float *part_o, const float2 *part_ml) {
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long most = static_cast<long long>(L.max_q) * L.group;   // rows of an item and key head
    const long long id = W == 8 ? blockIdx.x : static_cast<long long>(blockIdx.x) * 8 + warp;
    if (id >= static_cast<long long>(L.items) * L.key_heads * most) return;
    const int row = static_cast<int>(id % most), head = static_cast<int>(id / most % L.key_heads);
    const int i = static_cast<int>(id / (most * L.key_heads));
    Unit u;
    u.item = load_item(L, i);
    u.head = head;
    if (!u.item.ok || row >= u.item.nq * L.group) return;
    const long long first = static_cast<long long>(L.k_off[i] / chunk) + i;
    const int parts = max(1, (u.item.nk + chunk - 1) / chunk);
    const long long step = L.key_heads * most, at = (first * L.key_heads + head) * most + row;
    // The largest reference, then the sums at it.
    float m = -INFINITY, l = 0.0f;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, part_ml[at + p * step].x);
    for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float ref = m == -INFINITY ? 0.0f : m;
    const int dim = L.head_dim, d = 4 * lane;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int p = W == 8 ? warp : 0; p < parts; p += W) {
        const float2 ml = part_ml[at + p * step];
        const float c = ex2_full(ml.x - ref);
        l = fmaf(ml.y, c, l);
        if (d < dim) {
            const float4 v = *reinterpret_cast<const float4 *>(part_o + (at + p * step) * dim + d);
            o.x = fmaf(v.x, c, o.x), o.y = fmaf(v.y, c, o.y), o.z = fmaf(v.z, c, o.z), o.w = fmaf(v.w, c, o.w);
        }
    }
    if constexpr (W == 8) {
        __shared__ float4 sum_o[8][32];
        __shared__ float sum_l[8];
        sum_o[warp][lane] = o;
        if (lane == 0) sum_l[warp] = l;
        __syncthreads();
        if (warp != 0) return;
        for (int w = 1; w < 8; ++w) {
            const float4 v = sum_o[w][lane];
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
            l += sum_l[w];
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (d < dim)
        *reinterpret_cast<uint2 *>(row_ptr<T>(L, L.o, u, u.item.o0, row) + d) =
            make_uint2(Type<T>::pack(o.x * inv, o.y * inv), Type<T>::pack(o.z * inv, o.w * inv));
    if (L.lse && lane == 0) {
        const int r = row / L.group, h = head * L.group + row - r * L.group;
        L.lse[static_cast<long long>(u.item.o0 + r) * L.query_heads + h] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
    }
}

// ----------------------------------------------------------------------------
// backward
// ----------------------------------------------------------------------------

// A step loads 8 KB and takes 16 states at a time: S^T = K Q^T and dP^T = V dO^T, then
// dV = P^T dO and dK = dS^T Q of these states (the inner index is the row, P^T
// and dS^T are A operands as they come out of the first products), and
// dQ^T += K^T dS^T.  The fragments of Q and dO, as B operands of the first
// products and transposed as those of the second, stay in shared memory.
// With shared queries a warp keeps one dQ for all the units it takes.
//
// delta is taken from the output, which is rounded.  Where one state has most
// of a row's weight, its ds = p (dp - delta) is a small difference of large
// terms, and that rounding shows: an element of dK was off by as much as the
// root mean square of all of dK.  So the sums of ds are kept too: over a whole
// row sum p (dp - delta) is 0, and what it is instead is delta's error.
// States with a weight of 1/8 or more in some row, or 1/4 with more than 8 rows,
// whose share of an element is less, are noted, and mend() computes their dK
// again with the right delta (512 x 32 to 1024 states, 16 rows, 16 heads of 64:
// 873 us, 848 without; with 1/16 for all 976).  dQ keeps the first delta: its
// error is up to twice that of one rounding (0.0028 to 0.0033 of the norm in
// bf16, with sharp rows).
constexpr float large_weight(int tiles) { return tiles == 1 ? 0.125f : 0.25f; }

// What the backward leaves for mend(): of each unit, the sums of ds of its
// rows, the steps of 16 states with noted ones, and which they are: bit 4 g of
// a step's word is state g, bit 4 g + 1 state g + 8.
struct Notes {
    float *sums;
    uint32_t *steps, *states;
};

template <typename T, int DP, int NT>
__global__ void __launch_bounds__(kWarps / NT * 32, 3)
    backward_kernel(const __grid_constant__ AttentionLaunch L, int chunk, long long slots, long long stride,
                    float *part_dq, Notes notes) {
    constexpr int KC = DP / 32, KG = 128 / DP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr float kLarge = large_weight(NT);
    // [warp][Q, dO, Q^T, dO^T][tile][chunk][lane]
    __shared__ uint4 frag[kWarps / NT][4][NT][KC][32];
    check_all(L, false);
    const long long id = static_cast<long long>(blockIdx.x) * (kWarps / NT) + warp;
    if (id >= stride * L.key_heads) return;
    const int head = static_cast<int>(id % L.key_heads), dim = L.head_dim;
    const long long worker = id / L.key_heads;
    const float sl2 = L.scale * kLog2e;
    // fp16: what dS is multiplied by on its way through the products, P's 2^14 among it.  A power of two that follows the
    // largest dS that the warp has met: that goes in between 2^7 and 2^15.
    float unit = weight_unit<T>() == 1.0f ? 1.0f : 0.0f;   // 0: none met yet
    float dq[KC][2][NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) dq[c][i][n][0] = dq[c][i][n][1] = dq[c][i][n][2] = dq[c][i][n][3] = 0.0f;
    };
    // dq[c][i][n]: elements 32 c + 8 (g / 2) + 4 i + (g % 2), and two further on, of rows 8 n + 2 t, 2 t + 1.
    auto write = [&](long long slot, int rows) {
        const float back = unit == 0.0f ? 1.0f : weight_unit<T>() / unit;
        const long long at = (slot * L.key_heads + head) * (static_cast<long long>(L.max_q) * L.group);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 8 * n + 2 * t + r;
                if (row >= rows) continue;
                float *p = part_dq + (at + row) * dim + 8 * (g >> 1) + (g & 1);
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    if (32 * c + 8 * (g >> 1) >= dim) continue;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        p[32 * c + 4 * i] = dq[c][i][n][r] * back;
                        p[32 * c + 4 * i + 2] = dq[c][i][n][r + 2] * back;
                    }
                }
            }
    };
    clear();
    for (long long slot = worker; slot < slots; slot += stride) {
        const Unit u = find_unit(L, chunk, slot, head, lane);
        const long long slot_unit = slot * L.key_heads + head;
        if (u.rows == 0) {
            if (lane == 0) notes.steps[slot_unit] = 0;
            // an item without queries still has gradients to write, of zero
            if (u.item.ok && u.n > 0) {
                for (int s = g; s < u.n; s += 8)
                    for (int d = 8 * t; d < dim; d += 32) {
                        const long long row = u.k0 + s;
                        *reinterpret_cast<uint4 *>(static_cast<T *>(L.d_k.data) + row * L.d_k.row + head * L.d_k.head + d) =
                            make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(static_cast<T *>(L.d_v.data) + row * L.d_v.row + head * L.d_v.head + d) =
                            make_uint4(0, 0, 0, 0);
                    }
            }
            continue;
        }
        // Fragments, and lse (in powers of two) and delta of rows 2 t and 2 t + 1 of each tile.
        float lse[NT][2], delta[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = 8 * n + g;
            const bool on = row < u.rows;
            const T *pq = row_ptr<T>(L, L.q, u, u.item.q0, on ? row : 0);
            const T *pd = row_ptr<T>(L, L.d_o, u, u.item.o0, on ? row : 0);
            const T *po = row_ptr<T>(L, L.o, u, u.item.o0, on ? row : 0);
            float d = 0.0f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const bool in = on && 32 * c + 8 * t < dim;
                uint32_t fq[4], fd[4], fo[4];
                load_if(in, pq + 32 * c + 8 * t, fq);
                load_if(in, pd + 32 * c + 8 * t, fd);
                load_if(in, po + 32 * c + 8 * t, fo);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = Type<T>::unpack(fd[i]), b = Type<T>::unpack(fo[i]);
                    d = fmaf(a.x, b.x, fmaf(a.y, b.y, d));
                }
                frag[warp][0][n][c][lane] = make_uint4(fq[0], fq[1], fq[2], fq[3]);
                frag[warp][1][n][c][lane] = make_uint4(fd[0], fd[1], fd[2], fd[3]);
                frag[warp][2][n][c][lane] = make_uint4(transpose8(fq[0]), transpose8(fq[1]), transpose8(fq[2]), transpose8(fq[3]));
                frag[warp][3][n][c][lane] = make_uint4(transpose8(fd[0]), transpose8(fd[1]), transpose8(fd[2]), transpose8(fd[3]));
            }
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            d += __shfl_xor_sync(0xffffffffu, d, 2);
            const int rr = row / L.group, h = head * L.group + row - rr * L.group;
            const float e = on ? L.lse[static_cast<long long>(u.item.o0 + rr) * L.query_heads + h] : -INFINITY;
            const float e2 = e == -INFINITY ? INFINITY : e * kLog2e - weight_shift<T>();   // no kept state: p is 0
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                lse[n][r] = __shfl_sync(0xffffffffu, e2, 4 * (2 * t + r));
                delta[n][r] = __shfl_sync(0xffffffffu, d, 4 * (2 * t + r));
            }
        }
        __syncwarp();
        uint32_t noted = 0;
        float ds_sum[NT][2] = {};
        const T *kbase = static_cast<const T *>(L.k.data) + head * L.k.head + 8 * t;
        const T *vbase = static_cast<const T *>(L.v.data) + head * L.v.head + 8 * t;
        T *dkbase = static_cast<T *>(L.d_k.data) + head * L.d_k.head + 8 * t;
        T *dvbase = static_cast<T *>(L.d_v.data) + head * L.d_v.head + 8 * t;
        for (int j0 = 0; j0 < u.n; j0 += 16 * KG) {
            const uint32_t keep0 = kept(L, u.k0 + j0, min(16 * KG, u.n - j0), lane);
            uint32_t kr0[KG][2][KC][4], vr0[KG][2][KC][4];
#pragma unroll
            for (int x = 0; x < KG; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int s = 16 * x + 8 * y + g;
                    const long long row = u.k0 + j0 + s;
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const bool on = ((keep0 >> s) & 1u) && 32 * c + 8 * t < dim;
                        load_if(on, kbase + row * L.k.row + 32 * c, kr0[x][y][c]);
                        load_if(on, vbase + row * L.v.row + 32 * c, vr0[x][y][c]);
                    }
                }
#pragma unroll
            for (int x = 0; x < KG; ++x) {
                const int j = j0 + 16 * x, count = min(16, u.n - j);
                const uint32_t keep = keep0 >> (16 * x);
                auto &kr = kr0[x];
                auto &vr = vr0[x];
                uint32_t p[NT][4], ds[NT][4];   // of states g and g + 8: high halves, then low ones
                bool large0 = false, large1 = false;
                float met = 0.0f, des[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const uint4 q = frag[warp][0][n][c][lane], d = frag[warp][1][n][c][lane];
                        mma16<T>(s4, kr[0][c][0], kr[1][c][0], kr[0][c][1], kr[1][c][1], q.x, q.y);
                        mma16<T>(s4, kr[0][c][2], kr[1][c][2], kr[0][c][3], kr[1][c][3], q.z, q.w);
                        mma16<T>(d4, vr[0][c][0], vr[1][c][0], vr[0][c][1], vr[1][c][1], d.x, d.y);
                        mma16<T>(d4, vr[0][c][2], vr[1][c][2], vr[0][c][3], vr[1][c][3], d.z, d.w);
                    }
                    float pe[4], de[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool on = (keep >> (8 * (i >> 1) + g)) & 1u;
                        pe[i] = on ? ex2_full(fmaf(s4[i], sl2, -lse[n][i & 1])) : 0.0f;
                        de[i] = on ? pe[i] * (d4[i] - delta[n][i & 1]) : 0.0f;
                    }
                    ds_sum[n][0] += de[0] + de[2];
                    ds_sum[n][1] += de[1] + de[3];
                    large0 |= fmaxf(pe[0], pe[1]) >= kLarge / weight_unit<T>();
                    large1 |= fmaxf(pe[2], pe[3]) >= kLarge / weight_unit<T>();
                    split_pair<T>(pe[0], pe[1], p[n][0], p[n][2]);
                    split_pair<T>(pe[2], pe[3], p[n][1], p[n][3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        des[n][i] = de[i];
                        if constexpr (!Type<T>::bf16) met = fmaxf(met, fabsf(de[i]));
                    }
                }
                if constexpr (!Type<T>::bf16) {
                    const bool grow = met * unit > 32768.0f, first = unit == 0.0f && met > 0.0f;
                    if (__any_sync(0xffffffffu, (grow || first) && met < INFINITY)) {
                        if (!(met < INFINITY)) met = 0.0f;   // its results are not finite anyway
                        for (int w = 16; w; w >>= 1) met = fmaxf(met, __shfl_xor_sync(0xffffffffu, met, w));
                        const int e = max(min(7 - exponent_of(met), 100), -100);
                        const float now = power_of_two(e), change = unit == 0.0f ? 1.0f : now / unit;
                        unit = now;
#pragma unroll
                        for (int c = 0; c < KC; ++c)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int r = 0; r < 4; ++r) dq[c][i][n][r] *= change;
                    }
                }
                const float back = unit == 0.0f ? 1.0f : weight_unit<T>() / unit;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    split_pair<T>(des[n][0] * unit, des[n][1] * unit, ds[n][0], ds[n][2]);
                    split_pair<T>(des[n][2] * unit, des[n][3] * unit, ds[n][1], ds[n][3]);
                }
                if (__any_sync(0xffffffffu, large0 || large1)) {   // fold the four lanes of a state
                    uint32_t m0 = __ballot_sync(0xffffffffu, large0), m1 = __ballot_sync(0xffffffffu, large1);
                    m0 |= m0 >> 1, m1 |= m1 >> 1;
                    m0 |= m0 >> 2, m1 |= m1 >> 2;
                    if (lane == 0) notes.states[slot_unit * kSteps + (j >> 4)] = (m0 & 0x11111111u) | (m1 & 0x11111111u) << 1;
                    noted |= 1u << (j >> 4);
                }
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    float av[4][4], ak[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        av[i][0] = av[i][1] = av[i][2] = av[i][3] = ak[i][0] = ak[i][1] = ak[i][2] = ak[i][3] = 0.0f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 q = frag[warp][2][n][c][lane], d = frag[warp][3][n][c][lane];
                        const uint32_t qi[4] = {q.x, q.y, q.z, q.w}, di[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // 8 rows twice: against the high halves and against the low ones
                            mma16<T>(av[i], p[n][0], p[n][1], p[n][2], p[n][3], di[i], di[i]);
                            mma16<T>(ak[i], ds[n][0], ds[n][1], ds[n][2], ds[n][3], qi[i], qi[i]);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const long long row = u.k0 + j + 8 * y + g;
                        const bool live = (keep >> (8 * y + g)) & 1u;   // a dropped state's are 0 times whatever the rows hold
                        uint32_t wv[4], wk[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            wv[i] = live ? Type<T>::pack(av[i][2 * y] * weight_unit<T>(), av[i][2 * y + 1] * weight_unit<T>()) : 0u;
                            wk[i] = live ? Type<T>::pack(ak[i][2 * y] * (L.scale * back), ak[i][2 * y + 1] * (L.scale * back)) : 0u;
                        }
                        if (32 * c + 8 * t < dim && 8 * y + g < count) {
                            __stcs(reinterpret_cast<uint4 *>(dvbase + row * L.d_v.row + 32 * c), make_uint4(wv[0], wv[1], wv[2], wv[3]));
                            __stcs(reinterpret_cast<uint4 *>(dkbase + row * L.d_k.row + 32 * c), make_uint4(wk[0], wk[1], wk[2], wk[3]));
                        }
                    }
                    __syncwarp();   // the products that follow are the whole warp's
                }
                uint32_t bs[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) bs[n][i] = transpose8(ds[n][i]);
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a0 = transpose8(kr[0][c][2 * i]), a1 = transpose8(kr[0][c][2 * i + 1]);
                        const uint32_t a2 = transpose8(kr[1][c][2 * i]), a3 = transpose8(kr[1][c][2 * i + 1]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16<T>(dq[c][i][n], a0, a1, a2, a3, bs[n][0], bs[n][1]);
                            mma16<T>(dq[c][i][n], a0, a1, a2, a3, bs[n][2], bs[n][3]);
                        }
                    }
            }
        }
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float e = ds_sum[n][r];
                for (int w = 4; w < 32; w <<= 1) e += __shfl_xor_sync(0xffffffffu, e, w);
                const int row = 8 * n + 2 * t + r;
                if (g == 0 && row < u.rows)
                    notes.sums[slot_unit * (static_cast<long long>(L.max_q) * L.group) + row] = e * weight_unit<T>();
            }
        if (lane == 0) notes.steps[slot_unit] = noted;
        if (L.q_off) {
            write(slot, u.rows);
            clear();
        }
    }
    if (!L.q_off) write(worker, L.query_rows * L.group);
}

// dQ: the sum of a row's parts in a fixed order, times the scale; of shared
// queries the sum over all workers.  W warps a row, four elements a lane.
template <typename T, int W>
__device__ __forceinline__ void join_dq(const AttentionLaunch &L, int chunk, long long workers, const float *part_dq) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long most = static_cast<long long>(L.max_q) * L.group;
    const int dim = L.head_dim, d = 4 * lane;
    Unit u;
    long long first, parts;
    const long long id = W == 8 ? blockIdx.x : static_cast<long long>(blockIdx.x) * 8 + warp;
    if (id >= (L.q_off ? static_cast<long long>(L.items) : 1) * L.key_heads * most) return;
    const int i = static_cast<int>(id / (most * L.key_heads));
    const int row = static_cast<int>(id % most), head = static_cast<int>(id / most % L.key_heads);
    u.head = head;
    if (L.q_off) {
        u.item = load_item(L, i);
        if (!u.item.ok || row >= u.item.nq * L.group) return;
        first = chunk >= L.max_k ? i : static_cast<long long>(L.k_off[i] / chunk) + i;
        parts = max(1, (u.item.nk + chunk - 1) / chunk);
    } else {
        u.item.q0 = 0;
        first = 0;
        parts = workers;
    }
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (d < dim) {
        const float *src = part_dq + ((first * L.key_heads + head) * most + row) * dim + d;
        const long long step = L.key_heads * most * dim;
#pragma unroll 4
        for (long long p = W == 8 ? warp : 0; p < parts; p += W) {
            const float4 v = *reinterpret_cast<const float4 *>(src + p * step);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    if constexpr (W == 8) {
        __shared__ float4 sums[8][32];
        sums[warp][lane] = s;
        __syncthreads();
        if (warp != 0) return;
        for (int w = 1; w < 8; ++w) {
            const float4 v = sums[w][lane];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    if (d < dim)
        *reinterpret_cast<uint2 *>(row_ptr<T>(L, L.d_q, u, u.item.q0, row) + d) =
            make_uint2(Type<T>::pack(s.x * L.scale, s.y * L.scale), Type<T>::pack(s.z * L.scale, s.w * L.scale));
}

// The dK of a unit's noted states, with delta corrected by the row's sum of ds
// over the item's units, in a fixed order.  A warp a unit: half a warp a row,
// eight elements a lane.
template <typename T>
__device__ __forceinline__ void mend(const AttentionLaunch &L, int chunk, long long slots, long long unit, const Notes &notes) {
    if (unit >= slots * L.key_heads) return;
    uint32_t steps = notes.steps[unit];
    if (!steps) return;
    const int lane = threadIdx.x & 31, head = static_cast<int>(unit % L.key_heads), dim = L.head_dim, d = 8 * (lane & 15);
    const int half = lane >> 4;
    const Unit u = find_unit(L, chunk, unit / L.key_heads, head, lane);
    const long long most = static_cast<long long>(L.max_q) * L.group;
    const long long first = u.slot - (u.k0 - u.item.k0) / chunk;
    const int parts = max(1, (u.item.nk + chunk - 1) / chunk);
    const bool in = d < dim;
    auto load = [&](const T *p, bool on, float (&v)[8]) {
        const uint4 w = in && on ? *reinterpret_cast<const uint4 *>(p + d) : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 y = Type<T>::unpack(x[i]);
            v[2 * i] = y.x, v[2 * i + 1] = y.y;
        }
    };
    auto dot = [&](const float (&a)[8], const float (&b)[8]) {   // each half's
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x = fmaf(a[i], b[i], x);
        for (int w = 8; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        return x;
    };
    // Row r's delta and lse (in powers of two) in lane r and lane r + 16, which share its sums.
    float delta = 0.0f, lse = 0.0f;
    const int row_of = lane & 15;
    if (row_of < u.rows) {
        const int rr = row_of / L.group, h = head * L.group + row_of - rr * L.group;
        const float e = L.lse[static_cast<long long>(u.item.o0 + rr) * L.query_heads + h];
        lse = e == -INFINITY ? INFINITY : e * kLog2e;
        const float *sums = notes.sums + (first * L.key_heads + head) * most + row_of;
#pragma unroll 8
        for (int p = lane >> 4; p < parts; p += 2) delta += sums[p * (L.key_heads * most)];
    }
    delta += __shfl_xor_sync(0xffffffffu, delta, 16);
#pragma unroll 4
    for (int r0 = 0; r0 < u.rows; r0 += 2) {
        const int r = r0 + half;
        const bool on = r < u.rows;
        float a[8], b[8];
        load(row_ptr<T>(L, L.d_o, u, u.item.o0, on ? r : 0), on, a);
        load(row_ptr<T>(L, L.o, u, u.item.o0, on ? r : 0), on, b);
        const float x = dot(a, b), other = __shfl_xor_sync(0xffffffffu, x, 16);
        if ((row_of & ~1) == r0) delta += (row_of & 1) == half ? x : other;
    }
    for (; steps; steps &= steps - 1) {
        const int step = __ffs(steps) - 1;
        for (uint32_t left = notes.states[unit * kSteps + step]; left; left &= left - 1) {
            const int bit = __ffs(left) - 1;
            const long long row = u.k0 + 16 * step + (bit >> 2) + 8 * (bit & 1);
            float k[8], v[8], dk[8] = {};
            load(static_cast<const T *>(L.k.data) + row * L.k.row + head * L.k.head, true, k);
            load(static_cast<const T *>(L.v.data) + row * L.v.row + head * L.v.head, true, v);
#pragma unroll 4
            for (int r0 = 0; r0 < u.rows; r0 += 2) {
                const int r = r0 + half;
                const bool on = r < u.rows;
                float q[8], o[8];
                load(row_ptr<T>(L, L.q, u, u.item.q0, on ? r : 0), on, q);
                load(row_ptr<T>(L, L.d_o, u, u.item.o0, on ? r : 0), on, o);
                const float p = ex2_full(fmaf(dot(q, k), L.scale * kLog2e, -__shfl_sync(0xffffffffu, lse, r & 15)));
                const float ds = p * (dot(o, v) - __shfl_sync(0xffffffffu, delta, r & 15));
#pragma unroll
                for (int i = 0; i < 8; ++i) dk[i] = on ? fmaf(ds, q[i], dk[i]) : dk[i];
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) dk[i] = (dk[i] + __shfl_xor_sync(0xffffffffu, dk[i], 16)) * L.scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = Type<T>::pack(dk[2 * i], dk[2 * i + 1]);
            if (in && half == 0)
                *reinterpret_cast<uint4 *>(static_cast<T *>(L.d_k.data) + row * L.d_k.row + head * L.d_k.head + d) =
                    make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <typename T, int W>
__global__ void __launch_bounds__(256)
    finish_kernel(const __grid_constant__ AttentionLaunch L, int chunk, long long slots, long long workers, unsigned joins,
                  const float *part_dq, Notes notes) {
    after_previous();
    if (blockIdx.x < joins)
        join_dq<T, W>(L, chunk, workers, part_dq);
    else
        mend<T>(L, chunk, slots, static_cast<long long>(blockIdx.x - joins) * 8 + (threadIdx.x >> 5), notes);
}

// ----------------------------------------------------------------------------
// calls without states or without queries
// ----------------------------------------------------------------------------

// Zeroes rows x heads x dim of v, and sets lse to -infinity where there is one.
__global__ void __launch_bounds__(256)
    empty_kernel(const __grid_constant__ AttentionLaunch L, HeadsView v, long long rows, int heads, float *lse) {
    check_items(L, static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, static_cast<long long>(gridDim.x) * 256);
    const int per = L.head_dim / 8;
    const long long all = rows * heads * per;
    for (long long x = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; x < all; x += static_cast<long long>(gridDim.x) * 256) {
        const long long cell = x / per, row = cell / heads;
        const int d = static_cast<int>(x - cell * per) * 8, head = static_cast<int>(cell - row * heads);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(v.data) + row * v.row + head * v.head + d) = make_uint4(0, 0, 0, 0);
        if (lse && d == 0) lse[cell] = -INFINITY;
    }
}

void empty(const AttentionLaunch &L, const HeadsView &v, long long rows, int heads, float *lse, cudaStream_t stream) {
    const long long blocks = (rows * heads * (L.head_dim / 8) + 255) / 256;
    empty_kernel<<<static_cast<unsigned>(blocks < 1 ? 1 : blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(L, v, rows, heads, lse);
}

// How a call is cut.  Some 16 warps fit an SM of 152; a chunk leaves each
// about four units to even out ragged items, within 32 states (below that a
// warp does less than one step of its own) and 512 (a unit of some 10 us).
struct Cut {
    int chunk;
    long long slots, workers;
    long long rows;   // packed rows of an item and key head
};

Cut cut_of(const AttentionLaunch &L) {
    Cut c;
    long long want = static_cast<long long>(L.key_rows) * L.key_heads / (152 * 16 * 4);
    want = (want + 31) / 32 * 32;
    c.chunk = static_cast<int>(want < 32 ? 32 : want > kMostChunk ? kMostChunk : want);
    c.slots = c.chunk >= L.max_k ? L.items : L.key_rows / c.chunk + static_cast<long long>(L.items);
    const long long warps = 152 * 12 / L.key_heads;
    c.workers = L.q_off ? c.slots : warps < 1 ? 1 : warps < c.slots ? warps : c.slots;
    c.rows = static_cast<long long>(L.max_q) * L.group;
    return c;
}

// Eight warps a row join many parts of few rows sooner (1 x 8192 states, 8 heads
// of 64: the backward 17 us against 60), one warp a row the parts of many (64 x
// 4096, 16 rows: 244 us against 260).
bool wide_join(const AttentionLaunch &L, const Cut &c, long long rows) {
    return L.max_k > 8 * static_cast<long long>(c.chunk) && rows <= 152 * 8;
}

size_t part_bytes(const AttentionLaunch &L, long long slots, const Cut &c) {
    return align256(static_cast<size_t>(slots) * L.key_heads * c.rows * L.head_dim * sizeof(float));
}

// A call's two grids: the pass over the states, and what joins its parts (and
// mends, in the backward).  Items times heads pass 32 bits.
struct Grids {
    long long first, joins, mends;
    bool wide;   // eight warps a row join
};
Grids grids_of(const AttentionLaunch &L, const Cut &c, bool back) {
    const long long of_rows = L.q_off || !back ? L.items : 1, rows = of_rows * L.key_heads * c.rows;
    const int warps = back && c.rows > 8 ? kWarps / 2 : kWarps;
    Grids g;
    g.first = ((back ? c.workers : c.slots) * L.key_heads + warps - 1) / warps;
    g.wide = (back && !L.q_off) || wide_join(L, c, rows);
    g.joins = !back && c.chunk >= L.max_k ? 0 : g.wide ? rows : (rows + 7) / 8;
    g.mends = back ? (c.slots * L.key_heads + 7) / 8 : 0;
    return g;
}

template <typename T, int DP, int NT>
cudaError_t forward(const AttentionLaunch &L, cudaStream_t stream) {
    const Cut c = cut_of(L);
    const bool split = c.chunk < L.max_k;
    float *part_o = split ? reinterpret_cast<float *>(L.workspace) : nullptr;
    float2 *part_ml = split ? reinterpret_cast<float2 *>(L.workspace + part_bytes(L, c.slots, c)) : nullptr;
    const Grids g = grids_of(L, c, false);
    forward_kernel<T, DP, NT><<<static_cast<unsigned>(g.first), kWarps * 32, 0, stream>>>(L, c.chunk, c.slots, part_o, part_ml);
    if (g.joins == 0) return cudaGetLastError();   // whole items, or none that may have rows
    const dim3 joins(static_cast<unsigned>(g.joins));
    if (g.wide) return launch_after(join_kernel<T, 8>, joins, 256, 0, stream, L, c.chunk, part_o, part_ml);
    return launch_after(join_kernel<T, 1>, joins, 256, 0, stream, L, c.chunk, part_o, part_ml);
}

// The backward's workspace: dQ's parts, then the notes.
size_t notes_sums_bytes(const AttentionLaunch &L, const Cut &c) {
    return align256(static_cast<size_t>(c.slots) * L.key_heads * c.rows * sizeof(float));
}
size_t notes_steps_bytes(const AttentionLaunch &L, const Cut &c) {
    return align256(static_cast<size_t>(c.slots) * L.key_heads * sizeof(uint32_t));
}

template <typename T, int DP, int NT>
cudaError_t backward(const AttentionLaunch &L, cudaStream_t stream) {
    const Cut c = cut_of(L);
    float *part_dq = reinterpret_cast<float *>(L.workspace);
    char *at = reinterpret_cast<char *>(L.workspace) + part_bytes(L, c.workers, c);
    Notes notes;
    notes.sums = reinterpret_cast<float *>(at);
    notes.steps = reinterpret_cast<uint32_t *>(at + notes_sums_bytes(L, c));
    notes.states = reinterpret_cast<uint32_t *>(at + notes_sums_bytes(L, c) + notes_steps_bytes(L, c));
    const Grids g = grids_of(L, c, true);
    backward_kernel<T, DP, NT><<<static_cast<unsigned>(g.first), kWarps / NT * 32, 0, stream>>>(L, c.chunk, c.slots, c.workers,
                                                                                               part_dq, notes);
    const dim3 grid(static_cast<unsigned>(g.joins + g.mends));
    const unsigned joins = static_cast<unsigned>(g.joins);
    if (g.wide)
        return launch_after(finish_kernel<T, 8>, grid, 256, 0, stream, L, c.chunk, c.slots, c.workers, joins, part_dq, notes);
    return launch_after(finish_kernel<T, 1>, grid, 256, 0, stream, L, c.chunk, c.slots, c.workers, joins, part_dq, notes);
}

template <typename T>
cudaError_t dispatch(const AttentionLaunch &L, bool back, cudaStream_t stream) {
    const bool wide = L.head_dim > 64, two = static_cast<long long>(L.max_q) * L.group > 8;
    if (back) {
        if (wide) return two ? backward<T, 128, 2>(L, stream) : backward<T, 128, 1>(L, stream);
        return two ? backward<T, 64, 2>(L, stream) : backward<T, 64, 1>(L, stream);
    }
    if (wide) return two ? forward<T, 128, 2>(L, stream) : forward<T, 128, 1>(L, stream);
    return two ? forward<T, 64, 2>(L, stream) : forward<T, 64, 1>(L, stream);
}

// Few rows: an item's packed rows fill at most two tiles of 8.  With two of them
// the forward's tensor cores are ahead from some states on (16 rows, 8 heads of
// 128: 1 x 4096 states 13.8 us here and 16.3 there, 1 x 8192 27 and 18; 32 x
// 256 of 64: 16.6 and 11.6; 32 x 2048: 60 and 34; 512 x 32 to 1024 shared, 16
// heads of 64: 301 and 290; with 9 rows, 260).  The backward is ahead here (1 x
// 4096, 8 heads of 128: 18.5 us and 32.8; 8 heads of 64: 32 x 256 28.5 and 37,
// 64 x 4096 288 and 416; 512 x 32 to 1024, 16 heads of 64: 863 and 977, 725 and
// 972 with rows of their own).
bool few_rows(const AttentionLaunch &L, bool back) {
    const long long rows = static_cast<long long>(L.max_q) * L.group;
    return rows <= 8 || (rows <= 16 && (back || static_cast<long long>(L.key_rows) * L.key_heads <= 32768));
}

}  // namespace
}  // namespace attn

bool attention_grids_fit(const AttentionLaunch &L, bool back) {
    using namespace attn;
    constexpr long long kMost = (1ll << 31) - 1;
    if (!L.query_rows || !L.key_rows) return true;   // a grid of their own size
    if (!few_rows(L, back)) return (back ? backward_tiles_joins(L) : forward_tiles_joins(L)) <= kMost;
    const Grids g = grids_of(L, cut_of(L), back);
    return g.first <= kMost && g.joins + g.mends <= kMost;
}

size_t attention_workspace(const AttentionLaunch &L) {
    using namespace attn;
    if (!L.query_rows || !L.key_rows) return 0;
    if (!few_rows(L, false)) return forward_tiles_workspace(L);
    const Cut c = cut_of(L);
    if (c.chunk >= L.max_k) return 0;
    return part_bytes(L, c.slots, c) + align256(static_cast<size_t>(c.slots) * L.key_heads * c.rows * sizeof(float2));
}

size_t attention_backward_workspace(const AttentionLaunch &L) {
    using namespace attn;
    if (!L.query_rows || !L.key_rows) return 0;
    if (!few_rows(L, true)) return backward_tiles_workspace(L);
    const Cut c = cut_of(L);
    return part_bytes(L, c.workers, c) + notes_sums_bytes(L, c) + notes_steps_bytes(L, c) +
           static_cast<size_t>(c.slots) * L.key_heads * kSteps * sizeof(uint32_t);
}

cudaError_t launch_attention(const AttentionLaunch &L, cudaStream_t stream) {
    using namespace attn;
    if (L.query_rows && L.key_rows && !few_rows(L, false)) return launch_forward_tiles(L, stream);
    const bool none = !L.query_rows || !L.key_rows;
    if (none || L.items > kFewItems) {
        const cudaError_t e = cudaMemsetAsync(L.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    const long long out_rows = static_cast<long long>(L.query_rows) * (L.q_off ? 1 : L.items);
    if (none) {
        empty(L, L.o, out_rows, L.query_heads, L.lse, stream);
        return cudaGetLastError();
    }
    return L.dtype == CLI_BF16 ? dispatch<__nv_bfloat16>(L, false, stream) : dispatch<__half>(L, false, stream);
}

cudaError_t launch_attention_backward(const AttentionLaunch &L, cudaStream_t stream) {
    using namespace attn;
    if (L.query_rows && L.key_rows && !few_rows(L, true)) return launch_backward_tiles(L, stream);
    const bool none = !L.query_rows || !L.key_rows;
    if (none || L.items > kFewItems) {
        const cudaError_t e = cudaMemsetAsync(L.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    if (none) {
        empty(L, L.d_q, L.query_rows, L.query_heads, nullptr, stream);
        empty(L, L.d_k, L.key_rows, L.key_heads, nullptr, stream);
        empty(L, L.d_v, L.key_rows, L.key_heads, nullptr, stream);
        return cudaGetLastError();
    }
    return L.dtype == CLI_BF16 ? dispatch<__nv_bfloat16>(L, true, stream) : dispatch<__half>(L, true, stream);
}

}  // namespace cli
