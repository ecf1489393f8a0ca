"""Cases of the operators between a tower's blocks: layer norm, dropout, and both where a branch joins the residual stream.

A block of a byte encoder hands its branch's output, row after row on the batch's tape, to the residual stream: the
branch is dropped out, added to the stream, and the sum normalised for the next block.  Training runs the same way
back: the norm's gradient joins the stream's, the branch gets its share through the same mask, and the gain and the bias
sum theirs over every row of the tape.  The mask is never stored: both directions draw it from a counter-based
generator, whose seed and step are inputs.  The listed cases are those steps at the sizes this repository works with:
widths of 512 to 2048 and a wide one of 8192, tapes of one row for each of 16 items up to 270336 rows.

`run` is one call of an operator; with `own` false it is the plain form in 32 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPSILON = 1e-5


def device():
    return torch.device("cuda")


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def norm(name, direction, dtype, stream_dtype, rows, width, pad=0):
    """Layer norm of rows of `stream_dtype` to rows of `dtype`; `pad`: elements between the inputs' rows."""
    return {"name": name, "kind": "norm", "direction": direction, "dtype": dtype, "stream_dtype": stream_dtype,
            "rows": rows, "width": width, "pad": pad}


def drop(name, direction, dtype, rows, width, rate, pad=0):
    """Dropout of rows of `dtype`."""
    return {"name": name, "kind": "drop", "direction": direction, "dtype": dtype, "rows": rows, "width": width,
            "rate": rate, "pad": pad}


def join(name, direction, dtype, stream_dtype, rows, width, rate, onward, pad=0):
    """A branch of `dtype` into a stream of `stream_dtype`, and the norm of that; `onward`: the stream goes on past the
    norm, so that a gradient comes back along it too."""
    return {"name": name, "kind": "join", "direction": direction, "dtype": dtype, "stream_dtype": stream_dtype,
            "rows": rows, "width": width, "rate": rate, "onward": onward, "pad": pad}


def listed():
    return [
        # The pooled vectors of 16 requests, normalised before they are scored: latency is all.
        norm("norm_token", "forward", "bf16", "bf16", 16, 1024),
        # Every row of a tape of documents at width 1024: the largest norm.
        norm("norm_tape", "forward", "bf16", "bf16", 270336, 1024),
        # Full precision, an odd width whose rows start at any 4 bytes, and a count of rows that no tile divides.
        norm("norm_odd_f32", "forward", "f32", "f32", 20011, 771),
        # The tape's gradient in training, gain and bias summed over 131072 rows.
        norm("norm_grad", "backward", "bf16", "bf16", 131072, 1024),
        # The gradient of a small ragged batch in half precision, rows that start at any 4 bytes.
        norm("norm_grad_f16", "backward", "f16", "f16", 4099, 1002),
        # What a block reads of its tape, dropped out in training.
        drop("drop_tape", "forward", "bf16", 131072, 2048, 0.1),
        # Its gradient where rows lie apart in a wider buffer, at an odd width and a high rate.
        drop("drop_odd_grad", "backward", "f16", 30011, 517, 0.5, 8),
        # One row of each of 16 items joins its stream.
        join("join_token", "forward", "bf16", "bf16", 16, 2048, 0.1, True),
        # Branches in 16 bits, the residual stream in 32: the largest pass.
        join("join_tape", "forward", "bf16", "f32", 270336, 1024, 0.1, True),
        # The join's gradient in training, the stream's own coming back beside the norm's.
        join("join_grad", "backward", "bf16", "bf16", 131072, 1024, 0.1, True),
        # A wide block whose norm closes it: all of the gradient comes through the norm.
        join("join_wide_grad", "backward", "bf16", "bf16", 8192, 8192, 0.1, False),
        # Half precision into a 32-bit stream, a width of 4 elements times an odd number.
        join("join_narrow_grad", "backward", "f16", "f32", 20011, 516, 0.2, True),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    for _ in range(1000):
        c = one_draw(rng)
        if work(c)["bytes"] <= most:
            return c
    raise AssertionError("no draw within the listed cases' work")


def one_draw(rng):
    width = rng.choice([8 * spread(rng, 1, 1024), 8 * spread(rng, 16, 256), 4 * spread(rng, 2, 2048), spread(rng, 8, 8192)])
    rows = spread(rng, 1, 270336)
    direction = rng.choice(["forward", "backward"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    stream = rng.choice([dtype, "f32"])
    rate = rng.choice([0.0, 0.1, 0.1, 0.5, round(rng.random() * 0.9, 3)])
    pad = rng.choice([0, 0, 0, 8, rng.randint(1, 40)])
    kind = rng.choice(["norm", "drop", "join", "join"])
    if kind == "norm":
        c = norm("", direction, dtype, stream, rows, width, pad)
    elif kind == "drop":
        c = drop("", direction, dtype, rows, width, rate, pad)
    else:
        c = join("", direction, dtype, stream, rows, width, rate, rng.random() < 0.6, pad)
    del c["name"]
    return c


def work(case):
    t = BYTES[case["dtype"]]
    values = case["rows"] * case["width"]
    if case["kind"] == "drop":
        return {"bytes": float(2 * t * values + 16), "flops": float(values)}
    s, back = BYTES[case["stream_dtype"]], case["direction"] == "backward"
    if case["kind"] == "norm":
        each = t + 2 * s if back else t + s
    else:   # the sum is written where the stream goes on, and its gradient read
        each = 2 * t + s * ((3 if case["onward"] else 2) if back else 2 if case["onward"] else 1)
    return {"bytes": float(each * values + (12 if back else 8) * case["width"]), "flops": float(values * (14 if back else 8))}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=device())
    g.manual_seed(seed)
    rows, width, pad = case["rows"], case["width"], case["pad"]

    def matrix(dtype, scale=1.0, shift=0.0):   # rows `pad` elements apart
        x = torch.empty(rows, width + pad, dtype=DTYPES[dtype], device=device())
        step = max(1, (1 << 27) // (width + pad))
        for at in range(0, rows, step):
            part = torch.randn(min(step, rows - at), width + pad, generator=g, device=device())
            x[at:at + step] = part.mul_(scale).add_(shift)
        return x[:, :width] if pad else x

    s = {"case": case}
    if case["kind"] != "norm":
        # what a training program keeps on the device: a seed and the step
        s["seed"] = torch.tensor([0x5DEECE66D0000 + seed, 1000 + seed], dtype=torch.int64, device=device())
    back = case["direction"] == "backward"
    if case["kind"] == "drop":
        s["x"] = matrix(case["dtype"])
        return s
    s["gain"] = 1 + 0.2 * torch.randn(width, generator=g, device=device())
    s["bias"] = 0.1 * torch.randn(width, generator=g, device=device())
    if back:
        s["stream"] = matrix(case["stream_dtype"], 1.5, 0.25)
        s["d_output"] = matrix(case["dtype"])
        s["d_sum"] = matrix(case["stream_dtype"]) if case["kind"] == "join" and case["onward"] else None
    else:
        s["stream"] = matrix(case["stream_dtype"], 1.5, 0.25)
        s["x"] = matrix(case["dtype"]) if case["kind"] == "join" else None
    return s


SITE = 3   # the call's place among a model's dropouts


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    import contrastive_late_interaction_gb300 as cli
    case = s["case"]
    back, dtype = case["direction"] == "backward", DTYPES[case["dtype"]]
    if case["kind"] == "drop":
        if back:
            return [cli.dropout_backward(s["x"], case["rate"], s["seed"], site=SITE)["d_x"]]
        return [cli.dropout(s["x"], case["rate"], s["seed"], site=SITE)["output"]]
    if case["kind"] == "norm":
        if back:
            r = cli.layer_norm_backward(s["stream"], s["d_output"], gain=s["gain"], bias=s["bias"], epsilon=EPSILON)
            return [r["d_x"], r["d_gain"], r["d_bias"]]
        return [cli.layer_norm(s["stream"], gain=s["gain"], bias=s["bias"], epsilon=EPSILON, dtype=dtype)["output"]]
    if back:
        r = cli.dropout_layer_norm_backward(s["stream"], s["d_output"], case["rate"], s["seed"], site=SITE,
                                            d_sum=s["d_sum"], gain=s["gain"], bias=s["bias"], epsilon=EPSILON)
        return [r["d_residual"], r["d_x"], r["d_gain"], r["d_bias"]]
    r = cli.dropout_layer_norm(s["x"], s["stream"], case["rate"], s["seed"], site=SITE, gain=s["gain"], bias=s["bias"],
                               epsilon=EPSILON, want_sum=case["onward"])
    return [r["sum"], r["output"]] if case["onward"] else [r["output"]]


def run_plain(s):
    case = s["case"]
    back, dtype = case["direction"] == "backward", DTYPES[case["dtype"]]
    if case["kind"] == "drop":
        return [dropped(s["x"].float(), case["rate"], s["seed"]).to(dtype)]
    stream_dtype = DTYPES[case["stream_dtype"]]
    if not back:
        z = s["stream"].float()
        if case["kind"] == "join":
            z = z + dropped(s["x"].float(), case["rate"], s["seed"])
        y = (normed(z)[0] * s["gain"] + s["bias"]).to(dtype)
        return [z.to(stream_dtype), y] if case["kind"] == "join" and case["onward"] else [y]
    n, r = normed(s["stream"].float())
    dy = s["d_output"].float()
    d_gain, d_bias = (dy * n).sum(dim=0), dy.sum(dim=0)
    t = dy * s["gain"]
    dz = r * (t - t.mean(dim=1, keepdim=True) - n * (t * n).mean(dim=1, keepdim=True))
    if case["kind"] == "norm":
        return [dz.to(stream_dtype), d_gain, d_bias]
    if case["onward"]:
        dz = dz + s["d_sum"].float()
    return [dz.to(stream_dtype), dropped(dz, case["rate"], s["seed"]).to(dtype), d_gain, d_bias]


def normed(x):
    c = x - x.mean(dim=1, keepdim=True)
    r = torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPSILON)
    return c * r, r


def dropped(x, rate, seed):
    """x times 1 / (1 - rate) where the element's word is at least rate * 2^32, and 0 elsewhere."""
    least = int(rate * 2.0 ** 32)
    keep = words(x.shape[0], x.shape[1], seed) >= least
    return torch.where(keep, x * (2.0 ** 32 / (2.0 ** 32 - least)), 0.0)


def words(rows, width, seed):
    """The generator's 32-bit word of every element, as whole numbers [rows, width]: Philox 4x32 of ten rounds (Salmon,
    Moraes, Dror, Shaw 2011), keyed by the seed; word column % 4 of the block at (column / 4 + 2^16 site, row, step)."""
    low = 0xFFFFFFFF
    groups = (width + 3) // 4
    key0, key1 = seed[0] & low, (seed[0] >> 32) & low
    a = torch.arange(groups, device=device()).expand(rows, groups) + (SITE << 16)
    b = torch.arange(rows, device=device())[:, None].expand(rows, groups)
    c, d = (seed[1] & low).expand(rows, groups), ((seed[1] >> 32) & low).expand(rows, groups)
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57      # of 64 bits; what wraps is masked off
        a, b, c, d = ((q >> 32) & low) ^ b ^ key0, q & low, ((p >> 32) & low) ^ d ^ key1, p & low
        key0, key1 = (key0 + 0x9E3779B9) & low, (key1 + 0xBB67AE85) & low
    return torch.stack((a, b, c, d), dim=2).view(rows, 4 * groups)[:, :width]


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    rows, width = case["rows"], case["width"]
    f64 = torch.float64
    step = max(1, (1 << 23) // width)
    back, parts = case["direction"] == "backward", []
    d_gain, d_bias = torch.zeros(width, dtype=f64, device=device()), torch.zeros(width, dtype=f64, device=device())
    for at in range(0, rows, step):
        cut = slice(at, min(at + step, rows))
        factor = None if case["kind"] == "norm" else factors(cut, width, case["rate"], s["seed"].tolist())
        if case["kind"] == "drop":
            parts.append([s["x"][cut].double() * factor])
            continue
        z = s["stream"][cut].double()
        if not back:
            if case["kind"] == "join":
                z = z + s["x"][cut].double() * factor
            sd = torch.sqrt(z.var(dim=1, unbiased=False, keepdim=True) + EPSILON)
            y = (z - z.mean(dim=1, keepdim=True)) / sd * s["gain"].double() + s["bias"].double()
            parts.append([z, y] if case["kind"] == "join" and case["onward"] else [y])
            continue
        centred = z - z.sum(dim=1, keepdim=True) / width
        variance = centred.square().sum(dim=1, keepdim=True) / width + EPSILON
        g = s["d_output"][cut].double()
        d_gain += (g * centred / variance.sqrt()).sum(dim=0)
        d_bias += g.sum(dim=0)
        h = g * s["gain"].double()
        # of (z - mean) / sqrt(variance): the quotient's two terms, then the mean's
        d = h / variance.sqrt() - centred * (h * centred).sum(dim=1, keepdim=True) / (width * variance ** 1.5)
        d = d - (h / variance.sqrt()).sum(dim=1, keepdim=True) / width
        if case["kind"] == "norm":
            parts.append([d])
            continue
        if case["onward"]:
            d = d + s["d_sum"][cut].double()
        parts.append([d, d * factor])
    out = [torch.cat(p) for p in zip(*parts)]
    return out + [d_gain, d_bias] if back and case["kind"] != "drop" else out


def factors(cut, width, rate, seed):
    """[rows, width] of 0 or 1 / (1 - rate) in 64 bits, products taken in halves of 16 bits."""
    mask = 2 ** 32 - 1

    def times(x, m):   # (high, low) words of x * m
        low, mid = (x & 0xFFFF) * (m & 0xFFFF), (x >> 16) * (m & 0xFFFF)
        cross = (x & 0xFFFF) * (m >> 16) + (low >> 16) + (mid & 0xFFFF)
        return (x >> 16) * (m >> 16) + (mid >> 16) + (cross >> 16), ((cross & 0xFFFF) << 16) | (low & 0xFFFF)

    group = torch.arange((width + 3) // 4, device=device())[None, :]
    row = torch.arange(cut.start, cut.stop, device=device())[:, None]
    seed = [v % 2 ** 64 for v in seed]
    shape = (row.shape[0], group.shape[1])
    x = [(group + SITE * 65536).expand(shape), row.expand(shape),
         torch.full(shape, seed[1] % 2 ** 32, device=device()), torch.full(shape, seed[1] >> 32, device=device())]
    for i in range(10):
        k0 = (seed[0] % 2 ** 32 + i * 0x9E3779B9) & mask
        k1 = ((seed[0] >> 32) + i * 0xBB67AE85) & mask
        (h0, l0), (h1, l1) = times(x[0], 0xD2511F53), times(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
    word = torch.stack(x, dim=-1).flatten(1)[:, :width]
    dropped_share = math.floor(rate * 2 ** 32) / 2 ** 32
    return (word.double() / 2 ** 32 >= dropped_share).double() / (1.0 - dropped_share)
