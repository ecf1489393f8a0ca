// Cross attention over tapes and its gradients.  See include/cli.h for the
// formulas.
//
// One warp per (output row, head) walks its item's kept states with a running
// maximum and sum; the backward walks them again for dQ, and one warp per
// (state, key head) walks the item's queries for dK and dV.

#include "attention.cuh"

namespace cli {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kE = 4;   // elements of a head per lane: head_dim <= 128

template <typename T>
__device__ __forceinline__ void load_row(const HeadsView &v, long long row, int head, int d, float (&x)[kE]) {
    const T *p = static_cast<const T *>(v.data) + row * v.row + head * v.head;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = (threadIdx.x & 31) + 32 * e;
        x[e] = i < d ? static_cast<float>(p[i]) : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store_row(const HeadsView &v, long long row, int head, int d, const float (&x)[kE]) {
    T *p = static_cast<T *>(v.data) + row * v.row + head * v.head;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = (threadIdx.x & 31) + 32 * e;
        if (i < d) p[i] = static_cast<T>(x[e]);
    }
}
__device__ __forceinline__ float dot(const float (&a)[kE], const float (&b)[kE]) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) s = fmaf(a[e], b[e], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The item of row `row` of a tape: the last one whose offset is at most row.
__device__ __forceinline__ int item_of(const uint64_t *off, int items, int row) {
    int lo = 0, hi = items;   // off[lo] <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= static_cast<uint64_t>(row)) lo = mid; else hi = mid;
    }
    return lo;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) forward_kernel(const __grid_constant__ AttentionLaunch L, int out_rows) {
    check_items(L, (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                static_cast<long long>(gridDim.x) * gridDim.y * blockDim.x);
    const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y;
    if (row >= out_rows) return;
    const int i = L.q_off ? item_of(L.q_off, L.items, row) : row / L.query_rows;
    const Item t = load_item(L, i);
    if (!t.ok) return;
    const int kh = h / L.group;
    float q[kE], acc[kE] = {};
    load_row<T>(L.q, t.q0 + row - t.o0, h, L.head_dim, q);
    float m = -INFINITY, l = 0.0f;
    for (int j = t.k0; j < t.k0 + t.nk; ++j) {
        if (L.key_mask && !L.key_mask[j]) continue;
        float k[kE], v[kE];
        load_row<T>(L.k, j, kh, L.head_dim, k);
        load_row<T>(L.v, j, kh, L.head_dim, v);
        const float s = dot(q, k) * L.scale;
        const float m1 = fmaxf(m, s), c = expf(m - m1), p = expf(s - m1);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = acc[e] * c + p * v[e];
        m = m1;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = l == 0.0f ? 0.0f : acc[e] / l;   // no kept state: zero
    store_row<T>(L.o, row, h, L.head_dim, acc);
    if (L.lse && (threadIdx.x & 31) == 0)
        L.lse[static_cast<long long>(row) * L.query_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) dq_kernel(const __grid_constant__ AttentionLaunch L) {
    check_items(L, (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                static_cast<long long>(gridDim.x) * gridDim.y * blockDim.x);
    const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y;
    if (row >= L.query_rows) return;
    const int kh = h / L.group;
    float q[kE], acc[kE] = {};
    load_row<T>(L.q, row, h, L.head_dim, q);
    const int first = L.q_off ? item_of(L.q_off, L.items, row) : 0, last = L.q_off ? first + 1 : L.items;
    for (int i = first; i < last; ++i) {
        const Item t = load_item(L, i);
        if (!t.ok) return;
        const int o_row = t.o0 + row - t.q0;
        float o[kE], d_o[kE];
        load_row<T>(L.o, o_row, h, L.head_dim, o);
        load_row<T>(L.d_o, o_row, h, L.head_dim, d_o);
        const float delta = dot(o, d_o), lse = L.lse[static_cast<long long>(o_row) * L.query_heads + h];
        for (int j = t.k0; j < t.k0 + t.nk; ++j) {
            if (L.key_mask && !L.key_mask[j]) continue;
            float k[kE], v[kE];
            load_row<T>(L.k, j, kh, L.head_dim, k);
            load_row<T>(L.v, j, kh, L.head_dim, v);
            const float ds = expf(dot(q, k) * L.scale - lse) * (dot(d_o, v) - delta);
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[e] = fmaf(ds, k[e], acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] *= L.scale;
    store_row<T>(L.d_q, row, h, L.head_dim, acc);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) dkv_kernel(const __grid_constant__ AttentionLaunch L) {
    check_items(L, (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                static_cast<long long>(gridDim.x) * gridDim.y * blockDim.x);
    const int j = blockIdx.x * kWarps + (threadIdx.x >> 5), kh = blockIdx.y;
    if (j >= L.key_rows) return;
    const Item t = load_item(L, item_of(L.k_off, L.items, j));
    if (!t.ok) return;
    float k[kE], v[kE], dk[kE] = {}, dv[kE] = {};
    if (!L.key_mask || L.key_mask[j]) {
        load_row<T>(L.k, j, kh, L.head_dim, k);
        load_row<T>(L.v, j, kh, L.head_dim, v);
        for (int r = 0; r < t.nq; ++r)
            for (int h = kh * L.group; h < (kh + 1) * L.group; ++h) {
                float q[kE], o[kE], d_o[kE];
                load_row<T>(L.q, t.q0 + r, h, L.head_dim, q);
                load_row<T>(L.o, t.o0 + r, h, L.head_dim, o);
                load_row<T>(L.d_o, t.o0 + r, h, L.head_dim, d_o);
                const float lse = L.lse[static_cast<long long>(t.o0 + r) * L.query_heads + h];
                const float p = expf(dot(q, k) * L.scale - lse);
                const float ds = p * (dot(d_o, v) - dot(o, d_o)) * L.scale;
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    dk[e] = fmaf(ds, q[e], dk[e]);
                    dv[e] = fmaf(p, d_o[e], dv[e]);
                }
            }
    }
    store_row<T>(L.d_k, j, kh, L.head_dim, dk);
    store_row<T>(L.d_v, j, kh, L.head_dim, dv);
}

unsigned blocks(int rows) { return rows ? static_cast<unsigned>((rows + kWarps - 1) / kWarps) : 1u; }

template <typename T>
void forward(const AttentionLaunch &L, cudaStream_t stream) {
    const int out_rows = L.q_off ? L.query_rows : L.query_rows * L.items;
    forward_kernel<T><<<dim3(blocks(out_rows), L.query_heads), kWarps * 32, 0, stream>>>(L, out_rows);
}
template <typename T>
void backward(const AttentionLaunch &L, cudaStream_t stream) {
    dq_kernel<T><<<dim3(blocks(L.query_rows), L.query_heads), kWarps * 32, 0, stream>>>(L);
    dkv_kernel<T><<<dim3(blocks(L.key_rows), L.key_heads), kWarps * 32, 0, stream>>>(L);
}

}  // namespace
}  // namespace attn

size_t attention_workspace(const AttentionLaunch &) { return 0; }
size_t attention_backward_workspace(const AttentionLaunch &L) { return attn::backward_tiles_workspace(L); }

cudaError_t launch_attention(const AttentionLaunch &L, cudaStream_t stream) {
    if (L.query_rows && L.key_rows) return attn::launch_forward_tiles(L, stream);
    if (L.dtype == CLI_BF16) attn::forward<__nv_bfloat16>(L, stream); else attn::forward<__half>(L, stream);
    return cudaGetLastError();
}
cudaError_t launch_attention_backward(const AttentionLaunch &L, cudaStream_t stream) {
    if (L.query_rows && L.key_rows) return attn::launch_backward_tiles(L, stream);
    if (L.dtype == CLI_BF16) attn::backward<__nv_bfloat16>(L, stream); else attn::backward<__half>(L, stream);
    return cudaGetLastError();
}

}  // namespace cli
