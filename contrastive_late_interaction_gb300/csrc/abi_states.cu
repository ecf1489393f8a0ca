// The C ABI of include/cli.h, token states: host-side argument checks and
// launches of the rotation, head-norm and cross-attention verbs.  Nothing here
// allocates device memory.

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/cli.h"
#include "abi_checks.h"
#include "cli_internal.h"

namespace cli {
namespace {

constexpr size_t kRowsLimit = 1ull << 31;
constexpr size_t kTapeLimit = kRowsLimit - 4096;   // of attention: blocks of states are rounded up in 32 bits

size_t dtype_bytes(int dtype) { return dtype == CLI_F32 ? 4 : 2; }

// Heads of rows as bytes: a cli_heads_t with its counts.
struct Heads {
    uintptr_t at;
    size_t rows, heads, inner, row, head;   // inner: bytes of a head; row, head: strides in bytes
    Heads(const cli_heads_t &h, size_t rows_, size_t heads_, size_t dim, size_t esize)
        : at(reinterpret_cast<uintptr_t>(h.data)), rows(rows_), heads(heads_), inner(dim * esize),
          row(bytes_of(h.row_stride, esize)), head(bytes_of(h.head_stride, esize)) {
        if (rows <= 1) row = 0;
        if (heads <= 1) head = 0;
    }
    // past 2^40 elements it is more than heads_ok takes, and stays so
    static size_t bytes_of(size_t stride, size_t esize) { return (stride >> 40 ? 1ull << 40 : stride) * esize; }
    bool empty() const { return rows == 0 || heads == 0; }
    size_t span() const { return empty() ? 0 : (rows - 1) * row + (heads - 1) * head + inner; }
    Range range() const { return {at, at + span()}; }
};

// A data pointer and strides the kernels can address: 16-byte multiples and,
// over all rows and heads, less than 2^62 bytes.
cli_status_t heads_ok(const Heads &h) {
    if (h.empty()) return CLI_OK;
    if (!h.at || h.at % 16 != 0) return CLI_INVALID_ARGUMENT;
    if (h.row % 16 != 0 || h.head % 16 != 0) return CLI_SHAPE_MISMATCH;
    if (h.row >= (1ull << 40) || h.head >= (1ull << 40)) return CLI_SHAPE_MISMATCH;
    if (h.row && h.rows - 1 > (1ull << 61) / h.row) return CLI_SHAPE_MISMATCH;   // heads: 2^16 times 2^40 at most
    return CLI_OK;
}

// True when the rows and heads of h overlap one another (an output's may not).
bool self_overlap(const Heads &h) {
    if (h.empty()) return false;
    const bool rows_outer = (h.heads <= 1 || h.head >= h.inner) &&
                            (h.rows <= 1 || h.row >= (h.heads - 1) * h.head + h.inner);
    const bool heads_outer = (h.rows <= 1 || h.row >= h.inner) &&
                             (h.heads <= 1 || h.head >= (h.rows - 1) * h.row + h.inner);
    return !rows_outer && !heads_outer;
}

// True unless a and b share no byte.  Matrices that interleave in one buffer
// (a packed key-value tensor's halves, say) are told apart by their place
// within a common row stride or head stride.
bool heads_overlap(const Heads &a, const Heads &b) {
    if (a.empty() || b.empty() || !overlaps(a.range(), b.range())) return false;
    auto apart = [](const Heads &x, const Heads &y, size_t stride, size_t xspan, size_t yspan) {
        if (stride == 0 || xspan > stride || yspan > stride) return false;
        const size_t d = static_cast<size_t>(y.at >= x.at ? (y.at - x.at) % stride
                                                           : (stride - (x.at - y.at) % stride) % stride);
        return xspan <= d && d + yspan <= stride;
    };
    const size_t arow = a.row ? a.row : b.row, brow = b.row ? b.row : a.row;
    if (arow == brow &&
        apart(a, b, arow, (a.heads - 1) * a.head + a.inner, (b.heads - 1) * b.head + b.inner))
        return false;
    const size_t ahead = a.head ? a.head : b.head, bhead = b.head ? b.head : a.head;
    if (ahead == bhead && ahead) {
        if (apart(a, b, ahead, (a.rows - 1) * a.row + a.inner, (b.rows - 1) * b.row + b.inner)) return false;
        if (a.row % ahead == 0 && b.row % ahead == 0 && apart(a, b, ahead, a.inner, b.inner)) return false;
    }
    return true;
}

bool heads_range_overlap(const Heads &a, const Range &r) { return !a.empty() && overlaps(a.range(), r); }

bool same_place(const Heads &a, const Heads &b) {
    return a.at == b.at && a.row == b.row && a.head == b.head;
}

// What a launch came to.  A failed one leaves its error with the runtime, where the caller's next check of its own
// would find it.
cli_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return CLI_OK;
    cudaGetLastError();
    return CLI_DEVICE;
}

HeadsView view_of(const cli_heads_t &h) {
    return {h.data, static_cast<long long>(h.row_stride), static_cast<long long>(h.head_stride)};
}

// One rotation call: the two matrices a part reads and the one it writes.
cli_status_t rotary_call(const cli_rotary_t *a, bool norm, bool backward) {
    if (!a || !a->table || !a->device_status) return CLI_INVALID_ARGUMENT;
    if (a->dtype != CLI_BF16 && a->dtype != CLI_F16 && a->dtype != CLI_F32) return CLI_UNSUPPORTED;
    if (a->head_dim == 0 || a->head_dim % 8 != 0) return CLI_SHAPE_MISMATCH;
    if (a->head_dim > 256) return CLI_UNSUPPORTED;
    if (a->rotary_dim < 2 || a->rotary_dim % 2 != 0 || a->rotary_dim > a->head_dim) return CLI_SHAPE_MISMATCH;
    if (a->table_rows == 0 || a->table_rows >= kRowsLimit) return CLI_SHAPE_MISMATCH;
    if (!aligned(a->table, 8) || !aligned(a->device_status, 4)) return CLI_INVALID_ARGUMENT;
    if (norm && (!(a->epsilon > 0.0f) || std::isinf(a->epsilon))) return CLI_INVALID_ARGUMENT;

    const size_t es = dtype_bytes(a->dtype), d = a->head_dim;
    const bool grads = norm && backward;
    const cli_rotary_part_t *parts[2] = {&a->q, &a->k};
    const bool want_gain = grads && (a->q.d_gain || (a->k.heads && a->k.d_gain));
    const size_t ws_bytes = want_gain ? norm_rotary_heads_backward_workspace_bytes(d) : 0;
    if (want_gain && (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < ws_bytes))
        return CLI_INVALID_ARGUMENT;

    RotaryLaunch L = {};
    Heads outs[2] = {Heads({}, 0, 0, d, es), Heads({}, 0, 0, d, es)};
    Heads ins[4] = {outs[0], outs[0], outs[0], outs[0]};
    Range small_in[5] = {range_of(a->table, a->table_rows * (a->rotary_dim / 2) * 8)};
    Range small_out[4] = {range_of(a->device_status, 4), range_of(want_gain ? a->workspace : nullptr, ws_bytes)};
    for (int p = 0; p < 2; ++p) {
        const cli_rotary_part_t &s = *parts[p];
        if (p == 1 && s.heads == 0) continue;
        if (s.rows >= kRowsLimit || s.heads == 0 || s.heads > 65535) return CLI_SHAPE_MISMATCH;
        if (!aligned(s.positions, 4) || (norm && !aligned(s.gain, 4)) || (grads && !aligned(s.d_gain, 4))) return CLI_INVALID_ARGUMENT;
        const cli_heads_t &in = backward ? s.d_y : s.x, &out = backward ? s.d_x : s.y;
        const Heads hin(in, s.rows, s.heads, d, es), hout(out, s.rows, s.heads, d, es);
        const Heads hx(grads ? s.x : cli_heads_t{}, grads ? s.rows : 0, s.heads, d, es);
        for (const Heads *h : {&hin, &hout, &hx}) {
            const cli_status_t st = heads_ok(*h);
            if (st != CLI_OK) return st;
        }
        if (self_overlap(hout)) return CLI_SHAPE_MISMATCH;
        ins[2 * p] = hin;
        ins[2 * p + 1] = hx;
        outs[p] = hout;
        small_in[1 + 2 * p] = range_of(s.positions, s.positions ? s.rows * 4 : 0);
        small_in[2 + 2 * p] = range_of(norm ? s.gain : nullptr, norm && s.gain ? d * 4 : 0);
        small_out[2 + p] = range_of(grads ? s.d_gain : nullptr, grads && s.d_gain ? d * 4 : 0);
        RotaryPartLaunch &t = L.part[p];
        t.rows = static_cast<int>(s.rows);
        t.heads = static_cast<int>(s.heads);
        t.positions = s.positions;
        t.in = in.data;
        t.x = grads ? s.x.data : nullptr;
        t.out = out.data;
        t.in_row = static_cast<long long>(in.row_stride);
        t.in_head = static_cast<long long>(in.head_stride);
        t.x_row = static_cast<long long>(s.x.row_stride);
        t.x_head = static_cast<long long>(s.x.head_stride);
        t.out_row = static_cast<long long>(out.row_stride);
        t.out_head = static_cast<long long>(out.head_stride);
        t.gain = norm ? s.gain : nullptr;
        t.d_gain = grads ? s.d_gain : nullptr;
    }
    // Outputs overlap no input (but for a part's own, in place) and no other output.
    for (int p = 0; p < 2; ++p) {
        for (int i = 0; i < 4; ++i)
            if (heads_overlap(outs[p], ins[i]) && !(i / 2 == p && same_place(outs[p], ins[i])))
                return CLI_INVALID_ARGUMENT;
        for (const Range &r : small_in)
            if (heads_range_overlap(outs[p], r)) return CLI_INVALID_ARGUMENT;
        for (const Range &r : small_out)
            if (heads_range_overlap(outs[p], r)) return CLI_INVALID_ARGUMENT;
    }
    if (heads_overlap(outs[0], outs[1])) return CLI_INVALID_ARGUMENT;
    for (int o = 0; o < 4; ++o) {
        for (const Heads &h : ins)
            if (heads_range_overlap(h, small_out[o])) return CLI_INVALID_ARGUMENT;
        for (const Range &r : small_in)
            if (overlaps(r, small_out[o])) return CLI_INVALID_ARGUMENT;
        for (int q = o + 1; q < 4; ++q)
            if (overlaps(small_out[o], small_out[q])) return CLI_INVALID_ARGUMENT;
    }

    const int sms = sm_count();
    if (sms <= 0) return CLI_DEVICE;
    L.dtype = a->dtype;
    L.interleaved = a->interleaved ? 1 : 0;
    L.norm = norm;
    L.backward = backward;
    L.head_dim = static_cast<int>(d);
    L.rotary_dim = static_cast<int>(a->rotary_dim);
    L.table = reinterpret_cast<const float2 *>(a->table);
    L.table_rows = static_cast<int>(a->table_rows);
    L.epsilon = a->epsilon;
    L.inv_dim = 1.0f / static_cast<float>(d);
    L.sin_sign = backward ? -1.0f : 1.0f;
    L.status = a->device_status;
    L.sm_count = sms;
    float *partials = static_cast<float *>(a->workspace);
    for (int p = 0; p < 2; ++p)
        if (L.part[p].d_gain) L.part[p].gain_partials = partials + p * static_cast<size_t>(rotary_blocks(sms)) * d;
    if (want_gain && 2ull * rotary_blocks(sms) * d * 4 > ws_bytes) return CLI_UNSUPPORTED;
    cudaStream_t stream = static_cast<cudaStream_t>(a->stream);
    return launched(launch_rotary(L, stream));
}

// The sizes of an attention call, checked; `L` receives them.
cli_status_t attention_sizes(const cli_attention_t *a, bool backward, AttentionLaunch &L) {
    if (a->dtype != CLI_BF16 && a->dtype != CLI_F16) return CLI_UNSUPPORTED;
    if (a->items == 0 || a->items >= kRowsLimit || a->query_rows >= kTapeLimit || a->key_rows >= kTapeLimit)
        return CLI_SHAPE_MISMATCH;
    if (a->head_dim == 0 || a->head_dim % 8 != 0) return CLI_SHAPE_MISMATCH;
    if (a->head_dim > 128) return CLI_UNSUPPORTED;
    if (a->query_heads == 0 || a->key_heads == 0 || a->query_heads > 65535 || a->key_heads > 65535 ||
        a->query_heads % a->key_heads != 0)
        return CLI_SHAPE_MISMATCH;
    if (a->query_heads / a->key_heads > 128) return CLI_UNSUPPORTED;
    if (!a->query_offsets && a->items * a->query_rows >= kRowsLimit) return CLI_SHAPE_MISMATCH;
    const size_t mq = a->query_offsets && a->max_query_rows < a->query_rows ? a->max_query_rows : a->query_rows;
    const size_t mk = a->max_key_rows < a->key_rows ? a->max_key_rows : a->key_rows;
    L.dtype = a->dtype;
    L.items = static_cast<int>(a->items);
    L.query_rows = static_cast<int>(a->query_rows);
    L.key_rows = static_cast<int>(a->key_rows);
    L.q_off = a->query_offsets;
    L.k_off = a->key_offsets;
    L.max_q = static_cast<int>(mq);
    L.max_k = static_cast<int>(mk);
    L.query_heads = static_cast<int>(a->query_heads);
    L.key_heads = static_cast<int>(a->key_heads);
    L.group = L.query_heads / L.key_heads;
    L.head_dim = static_cast<int>(a->head_dim);
    return attention_grids_fit(L, backward) ? CLI_OK : CLI_SHAPE_MISMATCH;
}

cli_status_t attention_call(const cli_attention_t *a, bool backward) {
    if (!a) return CLI_INVALID_ARGUMENT;
    AttentionLaunch L = {};
    cli_status_t st = attention_sizes(a, backward, L);
    if (st != CLI_OK) return st;
    if (!a->key_offsets || !a->device_status || !std::isfinite(a->scale)) return CLI_INVALID_ARGUMENT;
    if (!aligned(a->key_offsets, 8) || !aligned(a->query_offsets, 8) || !aligned(a->device_status, 4) ||
        !aligned(a->lse, 4))
        return CLI_INVALID_ARGUMENT;
    const size_t out_rows = a->query_offsets ? a->query_rows : a->items * a->query_rows;
    const size_t d = a->head_dim, hq = a->query_heads, hk = a->key_heads;
    if (backward && !a->lse && out_rows) return CLI_INVALID_ARGUMENT;
    const Heads q(a->q, a->query_rows, hq, d, 2), k(a->k, a->key_rows, hk, d, 2), v(a->v, a->key_rows, hk, d, 2);
    const Heads o(a->output, out_rows, hq, d, 2);
    const size_t bo = backward ? out_rows : 0, bq = backward ? a->query_rows : 0, bk = backward ? a->key_rows : 0;
    const Heads d_o(a->d_output, bo, hq, d, 2), d_q(a->d_q, bq, hq, d, 2), d_k(a->d_k, bk, hk, d, 2),
        d_v(a->d_v, bk, hk, d, 2);
    for (const Heads *h : {&q, &k, &v, &o, &d_o, &d_q, &d_k, &d_v})
        if ((st = heads_ok(*h)) != CLI_OK) return st;
    for (const Heads *h : {&q, &k, &v, &d_o})
        if (!h->empty() && ((h->rows > 1 && h->row < h->inner) || (h->heads > 1 && h->head < h->inner)))
            return CLI_SHAPE_MISMATCH;
    for (const Heads *h : {&o, &d_q, &d_k, &d_v})
        if (self_overlap(*h)) return CLI_SHAPE_MISMATCH;
    const size_t ws_bytes = backward ? attention_backward_workspace(L) : attention_workspace(L);
    if (ws_bytes && (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < ws_bytes))
        return CLI_INVALID_ARGUMENT;

    const Heads *ins[5] = {&q, &k, &v, &d_o, &o};       // the output is an input of the backward
    const Heads *outs[3] = {&d_q, &d_k, &d_v};
    if (!backward) outs[0] = outs[1] = outs[2] = &o;
    const int nin = backward ? 5 : 3, nout = backward ? 3 : 1;
    const size_t lse_bytes = a->lse ? out_rows * hq * 4 : 0;
    const Range small_in[4] = {range_of(a->query_offsets, a->query_offsets ? (a->items + 1) * 8 : 0),
                               range_of(a->key_offsets, (a->items + 1) * 8),
                               range_of(a->key_mask, a->key_mask ? a->key_rows : 0),
                               range_of(a->lse, backward ? lse_bytes : 0)};
    const Range small_out[3] = {range_of(a->device_status, 4), range_of(ws_bytes ? a->workspace : nullptr, ws_bytes),
                                range_of(a->lse, backward ? 0 : lse_bytes)};
    for (int x = 0; x < nout; ++x) {
        for (int i = 0; i < nin; ++i)
            if (heads_overlap(*outs[x], *ins[i])) return CLI_INVALID_ARGUMENT;
        for (int y = x + 1; y < nout; ++y)
            if (heads_overlap(*outs[x], *outs[y])) return CLI_INVALID_ARGUMENT;
        for (const Range &r : small_in)
            if (heads_range_overlap(*outs[x], r)) return CLI_INVALID_ARGUMENT;
        for (const Range &r : small_out)
            if (heads_range_overlap(*outs[x], r)) return CLI_INVALID_ARGUMENT;
    }
    for (int x = 0; x < 3; ++x) {
        for (int i = 0; i < nin; ++i)
            if (heads_range_overlap(*ins[i], small_out[x])) return CLI_INVALID_ARGUMENT;
        for (const Range &r : small_in)
            if (overlaps(r, small_out[x])) return CLI_INVALID_ARGUMENT;
        for (int y = x + 1; y < 3; ++y)
            if (overlaps(small_out[x], small_out[y])) return CLI_INVALID_ARGUMENT;
    }

    L.sm_count = sm_count();
    if (L.sm_count <= 0) return CLI_DEVICE;
    L.scale = a->scale;
    L.key_mask = a->key_mask;
    L.q = view_of(a->q);
    L.k = view_of(a->k);
    L.v = view_of(a->v);
    L.o = view_of(a->output);
    L.d_o = view_of(a->d_output);
    L.d_q = view_of(a->d_q);
    L.d_k = view_of(a->d_k);
    L.d_v = view_of(a->d_v);
    L.lse = a->lse;
    L.workspace = static_cast<uint8_t *>(a->workspace);
    L.status = a->device_status;
    cudaStream_t stream = static_cast<cudaStream_t>(a->stream);
    return launched(backward ? launch_attention_backward(L, stream) : launch_attention(L, stream));
}

size_t attention_bytes(const cli_attention_t *a, bool backward) {
    if (!a) return 0;
    AttentionLaunch L = {};
    if (attention_sizes(a, backward, L) != CLI_OK) return 0;
    return backward ? attention_backward_workspace(L) : attention_workspace(L);
}

}  // namespace
}  // namespace cli

using namespace cli;

extern "C" {

cli_status_t rotary_table(const cli_rotary_table_t *a) {
    if (!a || !a->table || !aligned(a->table, 16)) return CLI_INVALID_ARGUMENT;
    if (a->positions == 0 || a->positions >= kRowsLimit) return CLI_SHAPE_MISMATCH;
    if (a->rotary_dim < 2 || a->rotary_dim % 2 != 0) return CLI_SHAPE_MISMATCH;
    if (a->rotary_dim > 256) return CLI_UNSUPPORTED;
    if (!(a->base > 1.0) || std::isinf(a->base) || !(a->factor >= 1.0) || std::isinf(a->factor))
        return CLI_INVALID_ARGUMENT;
    if (a->scaling < CLI_ROTARY_PLAIN || a->scaling > CLI_ROTARY_YARN) return CLI_UNSUPPORTED;
    if (a->scaling == CLI_ROTARY_NTK && a->rotary_dim == 2) return CLI_SHAPE_MISMATCH;
    if (a->scaling == CLI_ROTARY_YARN && a->trained_positions == 0) return CLI_INVALID_ARGUMENT;
    const int half = static_cast<int>(a->rotary_dim / 2);
    const double n = static_cast<double>(a->rotary_dim), two_pi = 6.283185307179586;
    double base = a->base, amplitude = 1.0, f[128];
    if (a->scaling == CLI_ROTARY_NTK) base *= std::pow(a->factor, n / (n - 2.0));
    // The pair that turns `turns` times over the trained positions L: base^(2 i / n) = L / (2 pi turns).
    auto pair_of = [&](double turns) {
        return n * std::log(static_cast<double>(a->trained_positions) / (two_pi * turns)) / (2.0 * std::log(a->base));
    };
    double lo = 0.0, hi = 0.0;
    if (a->scaling == CLI_ROTARY_YARN) {
        lo = std::fmax(std::floor(pair_of(32.0)), 0.0);
        hi = std::fmin(std::ceil(pair_of(1.0)), n - 1.0);
        if (hi <= lo) hi = lo + 0.001;
        amplitude = 0.1 * std::log(a->factor) + 1.0;
    }
    for (int i = 0; i < half; ++i) {
        f[i] = std::pow(base, -2.0 * i / n);
        if (a->scaling == CLI_ROTARY_LINEAR) f[i] /= a->factor;
        if (a->scaling == CLI_ROTARY_YARN) {
            const double blend = std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);   // 0: kept, 1: divided
            f[i] = f[i] * (1.0 - blend) + f[i] / a->factor * blend;
        }
    }
    return launched(launch_rotary_table(a->table, static_cast<long long>(a->positions), half, f, amplitude,
                                        static_cast<cudaStream_t>(a->stream)));
}

cli_status_t rotary_heads(const cli_rotary_t *a) { return rotary_call(a, false, false); }
cli_status_t rotary_heads_backward(const cli_rotary_t *a) { return rotary_call(a, false, true); }
cli_status_t norm_rotary_heads(const cli_rotary_t *a) { return rotary_call(a, true, false); }
cli_status_t norm_rotary_heads_backward(const cli_rotary_t *a) { return rotary_call(a, true, true); }

size_t norm_rotary_heads_backward_workspace_bytes(size_t head_dim) {
    // One row of partial sums per block and part; 256 SMs cover the GPUs this library is built for.
    return align256(2 * static_cast<size_t>(rotary_blocks(256)) * head_dim * sizeof(float));
}

cli_status_t cross_attention(const cli_attention_t *a) { return attention_call(a, false); }
size_t cross_attention_workspace_bytes(const cli_attention_t *a) { return attention_bytes(a, false); }
cli_status_t cross_attention_backward(const cli_attention_t *a) { return attention_call(a, true); }
size_t cross_attention_backward_workspace_bytes(const cli_attention_t *a) { return attention_bytes(a, true); }

}  // extern "C"
