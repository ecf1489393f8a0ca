// The C ABI of include/cli.h, between a tower's blocks: host-side argument
// checks and launches of layer norm, dropout and the residual join.  Nothing
// here allocates device memory.

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/cli.h"
#include "abi_checks.h"
#include "cli_internal.h"

namespace cli {
namespace {

constexpr size_t kRowsLimit = 1ull << 31;

bool is_dtype(int dtype) { return dtype == CLI_BF16 || dtype == CLI_F16 || dtype == CLI_F32; }

// A cli_rows_t as bytes; none: not part of the call.
struct Rows {
    uintptr_t at = 0;
    size_t rows = 0, inner = 0, row = 0, element = 1;   // inner: bytes of a row; row: stride in bytes, 0 where there is one
    size_t step = 0;                                    // the stride in bytes as it was given, modulo 2^64
    bool none = true;
    Rows() = default;
    Rows(const cli_rows_t &r, size_t rows_, size_t width, int dtype)
        : at(reinterpret_cast<uintptr_t>(r.data)), rows(rows_), element(dtype == CLI_F32 ? 4 : 2), none(false) {
        inner = width * element;
        step = r.row_stride * element;
        // past 2^40 elements it is more than ok() takes, and stays so
        row = rows > 1 ? (r.row_stride >> 40 ? 1ull << 40 : r.row_stride) * element : 0;
    }
    bool empty() const { return none || rows == 0; }
    Range range() const { return {at, at + (empty() ? 0 : (rows - 1) * row + inner)}; }
    cli_status_t ok() const {   // a pointer and a stride that the kernels can address: less than 2^62 bytes in all
        if (empty()) return CLI_OK;
        if (!at || at % element != 0) return CLI_INVALID_ARGUMENT;
        if (row >= (1ull << 40) || (row && rows - 1 > (1ull << 61) / row)) return CLI_SHAPE_MISMATCH;
        return CLI_OK;
    }
    // Rows of whole, aligned pieces.  One row's stride counts too, so that it is moved, and its sums run, as beside others.
    bool pieces(size_t bytes) const {
        return empty() || (at % bytes == 0 && step % bytes == 0 && inner % bytes == 0);
    }
};

// True unless a and b share no byte; columns of one buffer are told apart by their place within the common stride.
bool overlap(const Rows &a, const Rows &b) {
    if (a.empty() || b.empty() || !overlaps(a.range(), b.range())) return false;
    const size_t stride = a.row ? a.row : b.row;
    if (stride == 0 || (b.row && b.row != stride) || a.inner > stride || b.inner > stride) return true;
    const size_t d = static_cast<size_t>(b.at >= a.at ? (b.at - a.at) % stride : (stride - (a.at - b.at) % stride) % stride);
    return !(a.inner <= d && d + b.inner <= stride);
}

bool in_place(const Rows &a, const Rows &b) { return a.at == b.at && a.row == b.row && a.element == b.element; }

// A call's matrices and vectors, checked together: outputs overlap nothing but, in place, an input.
struct Call {
    Rows in[4], out[2];
    Range small_in[3] = {{0, 0}, {0, 0}, {0, 0}}, small_out[3] = {{0, 0}, {0, 0}, {0, 0}};

    cli_status_t check() const {
        for (const Rows &r : in)
            if (r.ok() != CLI_OK) return r.ok();
        for (const Rows &r : out) {
            if (r.ok() != CLI_OK) return r.ok();
            if (!r.empty() && r.rows > 1 && r.row < r.inner) return CLI_SHAPE_MISMATCH;
        }
        if (overlap(out[0], out[1])) return CLI_INVALID_ARGUMENT;
        for (const Rows &o : out) {
            for (const Rows &i : in)
                if (overlap(o, i) && !in_place(o, i)) return CLI_INVALID_ARGUMENT;
            if (o.empty()) continue;
            for (const Range &r : small_in)
                if (overlaps(o.range(), r)) return CLI_INVALID_ARGUMENT;
            for (const Range &r : small_out)
                if (overlaps(o.range(), r)) return CLI_INVALID_ARGUMENT;
        }
        for (int o = 0; o < 3; ++o) {
            for (const Rows &i : in)
                if (!i.empty() && overlaps(i.range(), small_out[o])) return CLI_INVALID_ARGUMENT;
            for (const Range &r : small_in)
                if (overlaps(r, small_out[o])) return CLI_INVALID_ARGUMENT;
            for (int p = o + 1; p < 3; ++p)
                if (overlaps(small_out[o], small_out[p])) return CLI_INVALID_ARGUMENT;
        }
        return CLI_OK;
    }
    template <typename F>
    bool all(F f) const {
        for (const Rows &r : in)
            if (!f(r)) return false;
        for (const Rows &r : out)
            if (!f(r)) return false;
        return true;
    }
    // How the call's chunks of 4 can be moved, and whether chunks of 8 are 16 bytes each.
    int moves() const {
        if (all([](const Rows &r) { return r.pieces(4 * r.element); })) return 0;   // kWhole
        return all([](const Rows &r) { return r.pieces(4); }) ? 1 : 2;              // kWords, kHalves
    }
    bool wide() const {
        return all([](const Rows &r) { return r.empty() || (r.element == 2 && r.pieces(16)); });
    }
};

// What a launch came to.  A failed one leaves its error with the runtime, where the caller's next check of its own
// would find it.
cli_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return CLI_OK;
    cudaGetLastError();
    return CLI_DEVICE;
}

cli_status_t sizes_ok(size_t rows, size_t width) {
    if (rows >= kRowsLimit || width == 0) return CLI_SHAPE_MISMATCH;
    return width > kMaxRowWidth ? CLI_UNSUPPORTED : CLI_OK;
}

cli_status_t mask_of(const cli_dropout_mask_t &m, MaskLaunch &out) {
    if (!(m.rate >= 0.0 && m.rate < 1.0) || m.site > 65535) return CLI_INVALID_ARGUMENT;
    if (m.rate > 0.0 && (!m.seed || !aligned(m.seed, 8))) return CLI_INVALID_ARGUMENT;
    const double words = 4294967296.0, least = std::floor(m.rate * words);
    out.seed = m.seed;
    out.site = m.site;
    out.least = static_cast<uint32_t>(least);
    out.scale = static_cast<float>(words / (words - least));
    return CLI_OK;
}

long long stride_of(const cli_rows_t &r) { return static_cast<long long>(r.row_stride); }

// A norm call, alone or joined: `s` and `t` are the stream's type and the other one.
struct Norm {
    int t, s;
    size_t rows, width;
    bool backward, join;
    cli_rows_t in, branch, sum, out, d_out, d_sum, d_in, d_branch;   // as in NormLaunch
    const float *gain, *bias;
    float *d_gain, *d_bias;
    float epsilon;
    cli_dropout_mask_t mask;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
};

cli_status_t norm_call(const Norm &a) {
    if (!is_dtype(a.t) || !is_dtype(a.s) || (a.s != a.t && a.s != CLI_F32)) return CLI_UNSUPPORTED;
    cli_status_t st = sizes_ok(a.rows, a.width);
    if (st != CLI_OK) return st;
    if (!(a.epsilon > 0.0f) || std::isinf(a.epsilon)) return CLI_INVALID_ARGUMENT;
    const float *gain = a.gain, *bias = a.backward ? nullptr : a.bias;
    float *d_gain = a.backward ? a.d_gain : nullptr, *d_bias = a.backward ? a.d_bias : nullptr;
    for (const float *p : {gain, bias, static_cast<const float *>(d_gain), static_cast<const float *>(d_bias)})
        if (!aligned(p, 4)) return CLI_INVALID_ARGUMENT;
    NormLaunch L = {};
    if ((st = mask_of(a.mask, L.mask)) != CLI_OK) return st;
    const bool sums = d_gain || d_bias;
    const size_t ws_bytes = sums ? layer_norm_backward_workspace_bytes(a.rows, a.width) : 0, vector = a.width * sizeof(float);
    if (ws_bytes && (!a.workspace || !aligned(a.workspace, 256) || a.workspace_bytes < ws_bytes)) return CLI_INVALID_ARGUMENT;

    Call c;
    auto rows = [&](const cli_rows_t &r, int dtype, bool there) { return there ? Rows(r, a.rows, a.width, dtype) : Rows(); };
    c.in[0] = rows(a.in, a.s, true);
    if (a.backward) {
        c.in[1] = rows(a.d_out, a.t, true);
        c.in[2] = rows(a.d_sum, a.s, a.join && a.d_sum.data);
        c.out[0] = rows(a.d_in, a.s, true);
        c.out[1] = rows(a.d_branch, a.t, a.join && a.d_branch.data);
    } else {
        c.in[1] = rows(a.branch, a.t, a.join);
        c.out[0] = rows(a.out, a.t, true);
        c.out[1] = rows(a.sum, a.s, a.join && a.sum.data);
    }
    c.small_in[0] = range_of(gain, gain ? vector : 0);
    c.small_in[1] = range_of(bias, bias ? vector : 0);
    c.small_in[2] = range_of(a.mask.seed, a.mask.rate > 0.0 ? 16 : 0);
    c.small_out[0] = range_of(d_gain, d_gain ? vector : 0);
    c.small_out[1] = range_of(d_bias, d_bias ? vector : 0);
    c.small_out[2] = range_of(ws_bytes ? a.workspace : nullptr, ws_bytes);
    if ((st = c.check()) != CLI_OK) return st;
    if (a.rows == 0 && !sums) return CLI_OK;

    L.sm_count = sm_count();
    if (L.sm_count <= 0) return CLI_DEVICE;
    if (ws_bytes && 2ull * norm_blocks(static_cast<long long>(a.rows), L.sm_count) * vector > ws_bytes) return CLI_UNSUPPORTED;
    L.dtype = a.t;
    L.stream_dtype = a.s;
    L.backward = a.backward;
    L.join = a.join;
    L.rows = static_cast<long long>(a.rows);
    L.width = static_cast<int>(a.width);
    L.wide = c.wide();
    L.moves = c.moves();
    L.inv_width = 1.0f / static_cast<float>(a.width);
    L.epsilon = a.epsilon;
    L.in = a.in.data, L.in_row = stride_of(a.in);
    L.branch = a.branch.data, L.branch_row = stride_of(a.branch);
    L.sum = a.sum.data, L.sum_row = stride_of(a.sum);
    L.out = a.out.data, L.out_row = stride_of(a.out);
    L.d_out = a.d_out.data, L.d_out_row = stride_of(a.d_out);
    L.d_sum = a.d_sum.data, L.d_sum_row = stride_of(a.d_sum);
    L.d_in = a.d_in.data, L.d_in_row = stride_of(a.d_in);
    L.d_branch = a.d_branch.data, L.d_branch_row = stride_of(a.d_branch);
    L.gain = gain;
    L.bias = bias;
    L.d_gain = d_gain;
    L.d_bias = d_bias;
    L.partials = ws_bytes ? static_cast<float *>(a.workspace) : nullptr;
    return launched(launch_norm(L, static_cast<cudaStream_t>(a.stream)));
}

cli_status_t layer_norm_call(const cli_layer_norm_t *a, bool backward) {
    if (!a) return CLI_INVALID_ARGUMENT;
    Norm n = {};
    n.t = a->y_dtype, n.s = a->x_dtype;
    n.rows = a->rows, n.width = a->width;
    n.backward = backward;
    n.in = a->x, n.out = a->y, n.d_out = a->d_y, n.d_in = a->d_x;
    n.gain = a->gain, n.bias = a->bias, n.d_gain = a->d_gain, n.d_bias = a->d_bias;
    n.epsilon = a->epsilon;
    n.workspace = a->workspace, n.workspace_bytes = a->workspace_bytes;
    n.stream = a->stream;
    return norm_call(n);
}

cli_status_t join_call(const cli_dropout_layer_norm_t *a, bool backward) {
    if (!a) return CLI_INVALID_ARGUMENT;
    Norm n = {};
    n.t = a->dtype, n.s = a->stream_dtype;
    n.rows = a->rows, n.width = a->width;
    n.backward = backward, n.join = true;
    n.in = backward ? a->sum : a->residual;
    n.branch = a->x, n.sum = a->sum, n.out = a->y;
    n.d_out = a->d_y, n.d_sum = a->d_sum, n.d_in = a->d_residual, n.d_branch = a->d_x;
    n.gain = a->gain, n.bias = a->bias, n.d_gain = a->d_gain, n.d_bias = a->d_bias;
    n.epsilon = a->epsilon;
    n.mask = a->mask;
    n.workspace = a->workspace, n.workspace_bytes = a->workspace_bytes;
    n.stream = a->stream;
    return norm_call(n);
}

cli_status_t dropout_call(const cli_dropout_t *a, bool backward) {
    if (!a) return CLI_INVALID_ARGUMENT;
    if (!is_dtype(a->dtype)) return CLI_UNSUPPORTED;
    cli_status_t st = sizes_ok(a->rows, a->width);
    if (st != CLI_OK) return st;
    DropoutLaunch L = {};
    if ((st = mask_of(a->mask, L.mask)) != CLI_OK) return st;
    const cli_rows_t &in = backward ? a->d_y : a->x, &out = backward ? a->d_x : a->y;
    Call c;
    c.in[0] = Rows(in, a->rows, a->width, a->dtype);
    c.out[0] = Rows(out, a->rows, a->width, a->dtype);
    c.small_in[0] = range_of(a->mask.seed, a->mask.rate > 0.0 ? 16 : 0);
    if ((st = c.check()) != CLI_OK) return st;
    if (a->rows == 0) return CLI_OK;
    L.sm_count = sm_count();
    if (L.sm_count <= 0) return CLI_DEVICE;
    L.dtype = a->dtype;
    L.rows = static_cast<long long>(a->rows);
    L.width = static_cast<int>(a->width);
    L.wide = c.wide();
    L.moves = c.moves();
    L.in = in.data, L.in_row = stride_of(in);
    L.out = out.data, L.out_row = stride_of(out);
    return launched(launch_dropout(L, static_cast<cudaStream_t>(a->stream)));
}

}  // namespace
}  // namespace cli

using namespace cli;

extern "C" {

cli_status_t layer_norm(const cli_layer_norm_t *a) { return layer_norm_call(a, false); }
cli_status_t layer_norm_backward(const cli_layer_norm_t *a) { return layer_norm_call(a, true); }

size_t layer_norm_backward_workspace_bytes(size_t rows, size_t width) {
    if (sizes_ok(rows, width) != CLI_OK || norm_few(rows, width)) return 0;
    // Two rows of partial sums a block; 256 SMs cover the GPUs this library is built for.
    return align256(2 * static_cast<size_t>(norm_blocks(static_cast<long long>(rows), 256)) * width * sizeof(float));
}

cli_status_t dropout(const cli_dropout_t *a) { return dropout_call(a, false); }
cli_status_t dropout_backward(const cli_dropout_t *a) { return dropout_call(a, true); }
cli_status_t dropout_layer_norm(const cli_dropout_layer_norm_t *a) { return join_call(a, false); }
cli_status_t dropout_layer_norm_backward(const cli_dropout_layer_norm_t *a) { return join_call(a, true); }

}  // extern "C"
