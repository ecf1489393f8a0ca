// Dropout of rows, forward and backward: the same kernel, as the gradient goes
// through the same mask.
//
// Mathematics: y = x * scale where the element's word of the generator is at
// least rate * 2^32, else 0, with scale = 1 / P(kept).  The word depends on the
// seed, the step, the call's site, the row and the column alone, so the
// backward draws it again and no mask is stored.

#include "rows.cuh"

namespace cli {
namespace rows {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

// The rows' chunks, counted through: a block takes kThreads * kUnroll of them at a time.  magic: 2^32 / chunks of a row,
// rounded up (0 for one chunk); next_row, next_chunk: how far the grid is across.
template <typename T, int E, int MOVES>
__global__ void __launch_bounds__(kThreads)
    dropout_kernel(const __grid_constant__ DropoutLaunch P, uint32_t chunks, uint32_t magic, long long next_row, uint32_t next_chunk) {
    constexpr uint32_t kTile = kThreads * kUnroll;
    const Mask mask(P.mask);
    const unsigned long long start = static_cast<unsigned long long>(blockIdx.x) * kTile;
    long long row0 = static_cast<long long>(start / chunks);
    uint32_t chunk0 = static_cast<uint32_t>(start % chunks);
    for (; row0 < P.rows; row0 += next_row, chunk0 += next_chunk) {
        if (chunk0 >= chunks) {
            chunk0 -= chunks;
            if (++row0 >= P.rows) break;
        }
        Chunk<T, E> c[kUnroll];
        long long row[kUnroll];
        int at[kUnroll], n[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t k = chunk0 + threadIdx.x + u * kThreads;   // k * chunks < 2^32: the quotient is exact
            const uint32_t down = magic ? __umulhi(k, magic) : k;
            row[u] = row0 + down;
            at[u] = static_cast<int>(k - down * chunks) * E;
            n[u] = row[u] < P.rows ? min(E, P.width - at[u]) : 0;
            take<MOVES>(c[u], static_cast<const T *>(P.in) + row[u] * P.in_row + at[u], n[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float2 v[E / 2];
            c[u].floats(v);
            mask.apply<E>(v, static_cast<uint32_t>(row[u]), at[u]);
            c[u].set(v);
            put<MOVES>(c[u], static_cast<T *>(P.out) + row[u] * P.out_row + at[u], n[u]);
        }
    }
}

template <typename T, int E, int MOVES>
cudaError_t launch(const DropoutLaunch &L, cudaStream_t stream) {
    constexpr long long kTile = kThreads * kUnroll;
    const long long chunks = (L.width + E - 1) / E, tiles = (L.rows * chunks + kTile - 1) / kTile;
    const long long most = 8ll * L.sm_count, blocks = tiles < most ? tiles : most;
    const uint32_t magic = chunks == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + chunks - 1) / chunks);
    dropout_kernel<T, E, MOVES><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
        L, static_cast<uint32_t>(chunks), magic, blocks * kTile / chunks, static_cast<uint32_t>(blocks * kTile % chunks));
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
