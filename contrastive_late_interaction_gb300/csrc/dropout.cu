// Dropout of rows, forward and backward: the same kernel, as the gradient goes
// through the same mask.
//
// Mathematics: y = x * scale where the element's word of the generator is at
// least rate * 2^32, else 0, with scale = 1 / P(kept).  The word depends on the
// seed, the step, the call's site, the row and the column alone, so the
// backward draws it again and no mask is stored.
//
// Work.  A thread has a chunk of one row in every few, always the same columns:
// what the generator's first rounds make of those and of the step is worked out
// once.  It takes kUnroll rows at a time, the next ones on their way.
//
// Bound: the generator.  A block of four words is 15 multiplications to 64 bits,
// and half of one that the row's two blocks share, which go out every fourth
// cycle, so four elements cost a scheduler 62 cycles on that pipe and some 70 on
// the one of exclusive ors and comparisons (73 in all, alone), beside 88 that
// HBM gives a warp's elements in bf16: 131072 x 2048 take 188 us (5.7 TB/s),
// where the bytes alone would take 158; fp32 runs at 0.98 of the copy's rate.
// Odd 16-bit rows go element by element: 0.42 at 771 columns.

#include "rows.cuh"

namespace cli {
namespace rows {
namespace {

// The rounds' keys in registers.  They come by way of shared memory, or the compiler would add them up again in each row:
// 233 us where these took 195 (131072 x 2048 in bf16, with the blocks' first rounds in registers too).
struct HeldKeys {
    uint32_t a3, k[12];
    __device__ __forceinline__ uint4 two(int i) const { return make_uint4(k[2 * i - 8], k[2 * i - 7], k[2 * i - 6], k[2 * i - 5]); }
    __device__ __forceinline__ explicit HeldKeys(const Seed &seed) {
        __shared__ uint32_t keys[13];
        const int i = threadIdx.x;
        if (i < 13) keys[i] = i == 12 ? seed.a(3) : i & 1 ? seed.b(4 + i / 2) : seed.a(4 + i / 2);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 12; ++j) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(k[j]) : "r"(smem_u32(keys + j)));
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a3) : "r"(smem_u32(keys + 12)));
    }
};

// Rows that a thread takes at a time.  131072 x 2048 in bf16: 2 take 226 us, 4 194, 6 188, 8 189; fp32 rows of 1024, shares
// of the copy's rate: 2 0.95, 4 0.84, 6 0.91, 8 0.87; 30011 rows of 517 in fp16, in pieces: 2 29 us, 3 27, 4 33.  (With the registers that a bound
// of 512 threads alone leaves the compiler to choose, six rows took 221.)
template <typename T, int MOVES> constexpr int kUnroll = MOVES != kWhole ? 3 : sizeof(T) == 2 ? 6 : 2;

// Lanes whose chunks make a span: whole chunks stand for themselves; pieces of 16 lanes are 32 bytes at least.
template <int MOVES> constexpr int kPart = MOVES == kWhole ? 1 : 16;

// spans: that the block has of each row; height: rows that it takes side by side.
template <typename T, int E, int MOVES>
__global__ void __launch_bounds__(512, 1) dropout_kernel(const __grid_constant__ DropoutLaunch P, int spans, int height) {
    constexpr int part = kPart<MOVES>;
    using L = Layout<T, E, MOVES, part>;
    const Seed seed(P.mask);
    const int group = threadIdx.x / part, span = blockIdx.y * spans + group % spans, down = group / spans;
    const L layout(part, threadIdx.x - group * part, span * part * E);
    const uint32_t rows = static_cast<uint32_t>(P.rows), stride = gridDim.x * height;
    const uint32_t there = down < height ? layout.template there<1>(P.width) : 0u;
    const HeldKeys keys(seed);
    Block blocks[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) blocks[i] = Block(seed, P.mask.site, layout.first_of(0, i));
    const uint32_t row_word = seed.row_word();
    const T *in = static_cast<const T *>(P.in) + layout.column;
    T *out = static_cast<T *>(P.out) + layout.column;
    using Raw = typename L::template Raw<T>;
    Raw next[kUnroll<T, MOVES>];
    auto load = [&](uint32_t row) {
#pragma unroll
        for (int u = 0; u < kUnroll<T, MOVES>; ++u, row += stride)
            layout.load(next[u], in + row * P.in_row, row < rows ? there : 0u);
    };
    uint32_t base = blockIdx.x * height;   // of the block
    load(base + down);
    for (; base < rows; base += kUnroll<T, MOVES> * stride) {
        uint32_t row = base + down;
        Raw now[kUnroll<T, MOVES>];
#pragma unroll
        for (int u = 0; u < kUnroll<T, MOVES>; ++u) now[u] = next[u];
        load(row + kUnroll<T, MOVES> * stride);
#pragma unroll
        for (int u = 0; u < kUnroll<T, MOVES>; ++u, row += stride) {
            float2 v[E / 2];
            Chunk<T, E> c = now[u].chunk();
            c.floats(v);
            if (P.mask.least) {
                uint4 r[E / 4];
                draw(blocks, keys, product(kMul0, row ^ row_word), r);
#pragma unroll
                for (int i = 0; i < E / 4; ++i) hand_round(layout, r[i]);
                keep<E>(v, r, P.mask.least, P.mask.scale);
            }
            c.set(v);
            layout.store(c, out + row * P.out_row, row < rows ? there : 0u);
        }
    }
}

template <typename T, int E, int MOVES>
cudaError_t launch(const DropoutLaunch &L, cudaStream_t stream) {
    constexpr int part = kPart<MOVES>;
    const int all = (L.width + part * E - 1) / (part * E);   // spans of a row
    const int pieces = (all * part + 511) / 512, spans = (all + pieces - 1) / pieces;
    // Rows side by side: of the blocks of 256 threads and more the one that wastes least of its last warp.
    int height = 1, threads = 0;
    double best = 0.0;
    for (int h = 1; h * spans * part <= 512; ++h) {
        const int t = (h * spans * part + 31) / 32 * 32;
        const double used = static_cast<double>(h * spans * part) / t;
        if (!threads || t <= 256 || used > best) height = h, threads = t, best = used;
    }
    // Blocks for 1024 threads an SM and piece of a row, twice what it holds of the kernels for whole chunks of 16-bit types
    // (110 to 124 registers): those come in waves, which costs nothing (131072 x 2048 in bf16: 187 us, with blocks for 512
    // threads 188; 32768 x 8192 188 and 184).  The others need them: fp32 rows of 1024 take 162 us and 202, 30011 rows of 517
    // in fp16 24.5 and 31.
    const long long want = (L.rows + height - 1) / height;
    const long long most = static_cast<long long>(L.sm_count) * (1024 / threads);
    long long across = want < most ? want : most;
    dropout_kernel<T, E, MOVES><<<dim3(static_cast<unsigned>(across), pieces), threads, 0, stream>>>(L, spans, height);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const DropoutLaunch &L, cudaStream_t stream) {
    if constexpr (sizeof(T) == 2) {
        if (L.wide) return launch<T, 8, kWhole>(L, stream);
        if (L.moves == kHalves) return launch<T, 4, kHalves>(L, stream);
    }
    return L.moves == kWhole ? launch<T, 4, kWhole>(L, stream) : launch<T, 4, kWords>(L, stream);
}

}  // namespace
}  // namespace rows

cudaError_t launch_dropout(const DropoutLaunch &L, cudaStream_t stream) {
    using namespace rows;
    if (L.dtype == CLI_BF16) return launch<__nv_bfloat16>(L, stream);
    if (L.dtype == CLI_F16) return launch<__half>(L, stream);
    return launch<float>(L, stream);
}

}  // namespace cli
