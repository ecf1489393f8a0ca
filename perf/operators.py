"""Cases of the token-state operators: rotary positions, head norms with rotation, cross attention over tapes.

A byte encoder hands on the states of every token of a batch, item after item on one tape.  Its pooling and
cross-modal blocks normalise queries and keys per head, rotate them by their positions, and let a few queries, or
another tape's rows, attend to each item's states.  The listed cases are those steps at the sizes this repository
works with: widths of 512 to 2048, heads of 64 and 128, documents of 32 to 1024 and of 64 to 512 rows, byte rows of
4096, media rows of 1024, batches of 512 to 2048 items.

`run` is one call (or a forward with its backward) of an operator; with `own` false it is the plain form in 32 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def device():
    return torch.device("cuda")


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def rotary(name, direction, dtype, rows, q_heads, k_heads, head_dim, rotary_dim, interleaved, context, scaling):
    return {"name": name, "kind": "rotary", "direction": direction, "dtype": dtype, "rows": rows, "q_heads": q_heads,
            "k_heads": k_heads, "head_dim": head_dim, "rotary_dim": rotary_dim, "interleaved": interleaved,
            "context": context, "scaling": scaling}


def norm_rotary(name, direction, dtype, rows, q_heads, k_heads, head_dim, rotary_dim, interleaved, context):
    return {"name": name, "kind": "norm_rotary", "direction": direction, "dtype": dtype, "rows": rows,
            "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim, "rotary_dim": rotary_dim,
            "interleaved": interleaved, "context": context, "scaling": 1.0}


def attention(name, direction, dtype, items, q_min, q_max, shared, k_min, k_max, q_heads, k_heads, head_dim, masked,
              length_seed):
    return {"name": name, "kind": "attention", "direction": direction, "dtype": dtype, "items": items, "q_min": q_min,
            "q_max": q_max, "shared": shared, "k_min": k_min, "k_max": k_max, "q_heads": q_heads, "k_heads": k_heads,
            "head_dim": head_dim, "masked": masked, "length_seed": length_seed}


def listed():
    return [
        # One new token of each of 16 running requests is rotated before it joins a cache: latency is all.
        rotary("rotary_token", "forward", "bf16", 16, 8, 2, 128, 128, False, 4096, 1.0),
        # A part of each head rotated, adjacent pairs, stretched to eight times the trained 4096 positions, full
        # precision, and a count of rows that no tile divides.
        rotary("rotary_part_f32", "forward", "f32", 20011, 8, 2, 80, 32, True, 32768, 8.0),
        # Queries and keys of a tape of 270,000 document rows at width 1024, before pooling.
        norm_rotary("norm_rotary_tape", "forward", "bf16", 270336, 16, 16, 64, 64, False, 1024),
        # The same step's gradient at width 1024 with heads of 128, both gains trained.
        norm_rotary("norm_rotary_grad", "backward", "bf16", 131072, 8, 8, 128, 128, False, 4096),
        # The gradient for a small ragged batch in half precision with grouped keys and a partly rotated head.
        norm_rotary("norm_rotary_grad_f16", "backward", "f16", 4099, 12, 4, 96, 64, True, 4096),
        # One query against one byte row of 4096 states with grouped heads: a reranker's answer to one request.
        attention("attend_token", "forward", "bf16", 1, 1, 1, False, 4096, 4096, 8, 2, 128, 0.0, 1),
        # The learned pooling query of every item over its states, for 2048 documents of 64 to 512 rows.
        attention("pool_documents", "forward", "bf16", 2048, 1, 1, True, 64, 512, 16, 16, 64, 0.0, 2),
        # The same pooling in training: 512 documents of 32 to 1024 rows, gradients for every state and the query.
        attention("pool_train", "train", "bf16", 512, 1, 1, True, 32, 1024, 8, 8, 128, 0.0, 3),
        # Queries of 8 to 64 tokens reading documents of 32 to 1024 rows, a tenth of whose rows are dropped.
        attention("read_documents", "forward", "f16", 512, 8, 64, False, 32, 1024, 16, 4, 64, 0.1, 4),
        # Byte rows of up to 4096 attending to media rows of 1024 at width 2048: the largest forward.
        attention("read_media", "forward", "bf16", 32, 1024, 4096, False, 1024, 1024, 16, 16, 128, 0.0, 5),
        # Training the same block on shorter rows, grouped keys.
        attention("read_media_train", "train", "bf16", 32, 512, 2048, False, 512, 1024, 16, 4, 128, 0.0, 6),
        # Training with narrow odd heads, dropped rows, short items and some with no states at all.
        attention("read_ragged_train", "train", "f16", 96, 1, 300, False, 0, 700, 6, 2, 72, 0.25, 7),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for key in w:
            most[key] = max(most.get(key, 0), w[key])
    for _ in range(1000):
        c = one_draw(rng)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and padded_bytes(c) <= 12e9:
            return c
    raise AssertionError("no draw within the listed cases' work")


def one_draw(rng):
    kind = rng.choice(["rotary", "norm_rotary", "attention", "attention", "attention"])
    if kind == "attention":
        head_dim = rng.choice([64, 128, 64, 128, 8 * rng.randint(4, 16)])
        k_heads = rng.choice([1, 2, 4, 8, 16])
        q_heads = k_heads * rng.choice([1, 1, 2, 3, 4, 8])
        q_max, k_max = spread(rng, 1, 2048), spread(rng, 16, 4096)
        if rng.random() < 0.3:
            q_max = 1
        c = attention("", rng.choice(["forward", "train"]), rng.choice(["bf16", "bf16", "f16"]), spread(rng, 1, 1024),
                      rng.choice([q_max, max(1, q_max // 8)]), q_max, rng.random() < 0.3,
                      rng.choice([k_max, k_max // 8]), k_max, q_heads, k_heads, head_dim,
                      rng.choice([0.0, 0.0, 0.15]), rng.randrange(1 << 20))
    else:
        head_dim = rng.choice([64, 128, 64, 128, 8 * rng.randint(4, 32)])
        rotary_dim = rng.choice([head_dim, head_dim, 2 * rng.randint(4, head_dim // 2)])
        k_heads = rng.choice([1, 2, 4, 8, 16])
        q_heads = k_heads * rng.choice([1, 2, 3, 4])
        args = ("", rng.choice(["forward", "backward"]), rng.choice(["bf16", "bf16", "f16", "f32"]),
                spread(rng, 1, 200000), q_heads, k_heads, head_dim, rotary_dim, rng.random() < 0.5,
                spread(rng, 256, 32768))
        c = rotary(*args, rng.choice([1.0, 4.0])) if kind == "rotary" else norm_rotary(*args)
    del c["name"]
    return c


def lengths(case):
    """The items' numbers of query rows and of state rows: the case's own, whatever the values' seed."""
    rng = random.Random(case["length_seed"])
    q = [case["q_max"]] if case["shared"] else [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["items"])]
    k = [rng.randint(case["k_min"], case["k_max"]) for _ in range(case["items"])]
    return q, k


def padded_bytes(case):
    """What the plain form's padded scores and states take."""
    if case["kind"] != "attention":
        return 0
    q, k = lengths(case)
    mq, mk = max(q), max(max(k), 1)
    return 4.0 * case["items"] * (case["q_heads"] * mq * mk + mk * case["k_heads"] * case["head_dim"])


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    d = case["head_dim"]
    if case["kind"] == "attention":
        q, k = lengths(case)
        pairs = sum(k) * q[0] if case["shared"] else sum(a * b for a, b in zip(q, k))
        out_rows = q[0] * case["items"] if case["shared"] else sum(q)
        q_row, k_row = case["q_heads"] * d * size, case["k_heads"] * d * size
        read = sum(q) * q_row + sum(k) * 2 * k_row + (sum(k) if case["masked"] else 0)
        flops = 4.0 * pairs * case["q_heads"] * d
        if case["direction"] == "forward":
            return {"bytes": float(read + out_rows * q_row), "flops": flops}
        # with the backward: dO read, dQ, dK and dV written, and five more products of the scores' size
        return {"bytes": float(read + 2 * out_rows * q_row + sum(q) * q_row + sum(k) * 2 * k_row), "flops": 3.5 * flops}
    values = case["rows"] * (case["q_heads"] + case["k_heads"]) * d
    table = min(case["rows"], case["context"]) * case["rotary_dim"] * 4 + 4 * case["rows"]
    passes = 3 if case["kind"] == "norm_rotary" and case["direction"] == "backward" else 2
    return {"bytes": float(passes * values * size + table),
            "flops": float(values * (3 if case["kind"] == "rotary" else 8 if passes == 2 else 20))}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def rotation_table(context, rotary_dim, scaling, dtype=torch.float32):
    """[context, rotary_dim / 2, (cos, sin)] of p * 10000^(-2 i / rotary_dim) / scaling."""
    i = torch.arange(rotary_dim // 2, device=device(), dtype=torch.float64)
    angle = torch.arange(context, device=device(), dtype=torch.float64)[:, None] * (
        10000.0 ** (-2.0 * i / rotary_dim) / scaling)
    return torch.stack((angle.cos(), angle.sin()), dim=-1).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=device())
    g.manual_seed(seed)
    dtype, d = DTYPES[case["dtype"]], case["head_dim"]

    def rand(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g, device=device(), dtype=torch.float32)).to(dtype)

    s = {"case": case}
    if case["kind"] == "attention":
        ql, kl = lengths(case)
        rows_q, rows_k, hq, hk = sum(ql), sum(kl), case["q_heads"], case["k_heads"]
        out_rows = rows_q * case["items"] if case["shared"] else rows_q

        def offsets(n):
            return torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(device())

        s.update(q=rand(rows_q, hq, d, scale=2.0), k=rand(rows_k, hk, d), v=rand(rows_k, hk, d),
                 q_offsets=None if case["shared"] else offsets(ql), k_offsets=offsets(kl), max_q=max(ql), max_k=max(kl),
                 key_mask=None, d_out=rand(out_rows, hq, d) if case["direction"] == "train" else None)
        if case["masked"]:
            keep = torch.rand(rows_k, generator=g, device=device()) >= case["masked"]
            s["key_mask"] = keep.to(torch.uint8)
            drop = ~keep   # rows that were dropped before they were computed: whatever the memory held
            s["k"][drop] = float("nan")
            s["v"][drop] = float("inf")
        return s
    rows, context = case["rows"], case["context"]
    s.update(q=rand(rows, case["q_heads"], d), k=rand(rows, case["k_heads"], d),
             table=rotation_table(context, case["rotary_dim"], case["scaling"]),
             positions=torch.randint(0, context, (rows,), generator=g, device=device(), dtype=torch.int32))
    if case["kind"] == "norm_rotary":
        s["q_gain"] = 1 + 0.2 * torch.randn(d, generator=g, device=device())
        s["k_gain"] = 1 + 0.2 * torch.randn(d, generator=g, device=device())
        if case["direction"] == "backward":
            s["d_q"], s["d_k"] = rand(rows, case["q_heads"], d), rand(rows, case["k_heads"], d)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

EPSILON = 1e-6


def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    import contrastive_late_interaction_gb300 as cli
    case = s["case"]
    if case["kind"] == "rotary":
        if case["direction"] == "forward":
            r = cli.rotary_heads(s["q"], s["table"], s["positions"], k=s["k"], k_positions=s["positions"],
                                 interleaved=case["interleaved"])
            return [r["q"], r["k"]]
        r = cli.rotary_heads_backward(s["q"], s["table"], s["positions"], d_k=s["k"], k_positions=s["positions"],
                                      interleaved=case["interleaved"])
        return [r["d_q"], r["d_k"]]
    if case["kind"] == "norm_rotary":
        if case["direction"] == "forward":
            r = cli.norm_rotary_heads(s["q"], s["table"], s["positions"], q_gain=s["q_gain"], k=s["k"],
                                      k_positions=s["positions"], k_gain=s["k_gain"],
                                      interleaved=case["interleaved"], epsilon=EPSILON)
            return [r["q"], r["k"]]
        r = cli.norm_rotary_heads_backward(s["q"], s["d_q"], s["table"], s["positions"], q_gain=s["q_gain"], k=s["k"],
                                           d_k=s["d_k"], k_positions=s["positions"], k_gain=s["k_gain"],
                                           interleaved=case["interleaved"], epsilon=EPSILON)
        return [r["d_q"], r["d_k"], r["d_q_gain"], r["d_k_gain"]]
    sizes = dict(key_mask=s["key_mask"], max_query_rows=s["max_q"], max_key_rows=s["max_k"])
    f = cli.cross_attention(s["q"], s["q_offsets"], s["k"], s["v"], s["k_offsets"],
                            want_lse=case["direction"] == "train", **sizes)
    if case["direction"] == "forward":
        return [f["output"]]
    b = cli.cross_attention_backward(s["q"], s["q_offsets"], s["k"], s["v"], s["k_offsets"], f["output"], f["lse"],
                                     s["d_out"], **sizes)
    return [f["output"], b["d_q"], b["d_k"], b["d_v"]]


def run_plain(s):
    case = s["case"]
    if case["kind"] == "attention":
        return plain_attention(s)
    cs = s["table"][s["positions"].long()]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if case["direction"] == "backward":
        sin = -sin   # the transposed rotation
    turn = lambda x: rotate(x, cos, sin, case["interleaved"])  # noqa: E731
    dtype = s["q"].dtype
    q, k = s["q"].float(), s["k"].float()
    if case["kind"] == "rotary":
        return [turn(q).to(dtype), turn(k).to(dtype)]
    if case["direction"] == "forward":
        return [turn(normed(q) * s["q_gain"]).to(dtype), turn(normed(k) * s["k_gain"]).to(dtype)]
    dq, dqg = norm_gradient(q, turn(s["d_q"].float()), s["q_gain"])
    dk, dkg = norm_gradient(k, turn(s["d_k"].float()), s["k_gain"])
    return [dq.to(dtype), dk.to(dtype), dqg, dkg]


def rotate(x, cos, sin, interleaved):
    n = 2 * cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y[..., 0:n:2], y[..., 1:n:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        y[..., :n // 2], y[..., n // 2:n] = a * cos - b * sin, b * cos + a * sin
    return y


def normed(x):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPSILON)


def norm_gradient(x, dz, gain):
    """Of z = gain x / sqrt(mean(x^2) + epsilon): dx, and the gain's gradient summed over rows and heads."""
    r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPSILON)
    n = x * r
    t = dz * gain
    return r * (t - n * (t * n).mean(dim=-1, keepdim=True)), (dz * n).sum(dim=(0, 1))


def plain_attention(s):
    case = s["case"]
    items, hq, hk, d = case["items"], case["q_heads"], case["k_heads"], case["head_dim"]
    mq, mk, group, dtype = s["max_q"], max(s["max_k"], 1), hq // hk, s["q"].dtype
    scale = 1.0 / math.sqrt(d)
    rows_q, rows_k = s["q"].shape[0], s["k"].shape[0]

    def places(offsets, rows, most):   # of each row of a tape in [items, most]
        item = torch.repeat_interleave(torch.arange(items, device=device()), offsets.diff(), output_size=rows)
        return item * most + torch.arange(rows, device=device()) - offsets[item]

    kat = places(s["k_offsets"], rows_k, mk)
    qat = None if case["shared"] else places(s["q_offsets"], rows_q, mq)
    keep = torch.ones(rows_k, dtype=torch.bool, device=device()) if s["key_mask"] is None else s["key_mask"] != 0
    valid = torch.zeros(items * mk, dtype=torch.bool, device=device())
    valid[kat] = keep
    valid = valid.view(items, 1, 1, mk)

    def keys(x):   # [items, hk, mk, d], zeros where there is no state or it was dropped
        p = torch.zeros(items * mk, hk, d, device=device())
        p[kat] = torch.where(keep[:, None, None], x.float(), 0.0)
        return p.view(items, mk, hk, d).transpose(1, 2)

    def queries(x, per_item):   # [items, hk, group * mq, d]
        if qat is None:
            p = x.float().view(items if per_item else 1, mq, hk, group, d)
        else:
            p = torch.zeros(items * mq, hq, d, device=device())
            p[qat] = x.float()
            p = p.view(items, mq, hk, group, d)
        return p.permute(0, 2, 3, 1, 4).reshape(p.shape[0], hk, group * mq, d)

    def back(x):   # the inverse of `queries` for results per item: [rows, hq, d]
        x = x.view(items, hk, group, mq, d).permute(0, 3, 1, 2, 4).reshape(items * mq, hq, d)
        return x if qat is None else x[qat]

    q, k, v = queries(s["q"], False), keys(s["k"]), keys(s["v"])
    scores = torch.where(valid, torch.matmul(q * scale, k.transpose(2, 3)), -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, v)
    if case["direction"] == "forward":
        return [back(out).to(dtype)]
    del scores
    do = queries(s["d_out"], True)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = p * (torch.matmul(do, v.transpose(2, 3)) - (do * out).sum(dim=-1, keepdim=True)) * scale
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q.expand(items, -1, -1, -1))
    flat = lambda x: x.transpose(1, 2).reshape(items * mk, hk, d)[kat].to(dtype)  # noqa: E731
    dq = back(dq)
    if case["shared"]:
        dq = dq.view(items, mq, hq, d).sum(dim=0)
    return [back(out).to(dtype), dq.to(dtype), flat(dk), flat(dv)]


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attention":
        return exact_attention(case, s)
    d, n = case["head_dim"], case["rotary_dim"]
    # The rotation as a d x d matrix per position, R[a, b] = what coordinate b adds to coordinate a.
    first = torch.arange(0, n, 2) if case["interleaved"] else torch.arange(n // 2)
    second = first + 1 if case["interleaved"] else first + n // 2
    table = s["table"].double()
    out = []
    for name in ("q", "k"):
        parts, gains = [], torch.zeros(d, dtype=torch.float64, device=device())
        for at in range(0, case["rows"], 2048):
            x = s[name][at:at + 2048].double()
            cs = table[s["positions"][at:at + 2048].long()]
            m = torch.eye(d, dtype=torch.float64, device=device()).repeat(x.shape[0], 1, 1)
            m[:, first, first], m[:, second, second] = cs[..., 0], cs[..., 0]
            m[:, second, first], m[:, first, second] = cs[..., 1], -cs[..., 1]
            if case["kind"] == "rotary":
                y = x @ m if case["direction"] == "backward" else x @ m.transpose(1, 2)
            else:
                gain = s[name + "_gain"].double()
                mean = x.pow(2).sum(-1, keepdim=True) / d + EPSILON
                if case["direction"] == "forward":
                    y = (x / mean.sqrt() * gain) @ m.transpose(1, 2)
                else:
                    dz = s["d_" + name][at:at + 2048].double() @ m
                    gains += (dz * x / mean.sqrt()).sum(dim=(0, 1))
                    y = dz * gain / mean.sqrt() - x * (dz * gain * x).sum(-1, keepdim=True) / (d * mean ** 1.5)
            parts.append(y)
        out.append((torch.cat(parts), gains))
    if case["kind"] == "norm_rotary" and case["direction"] == "backward":
        return [out[0][0], out[1][0], out[0][1], out[1][1]]
    return [out[0][0], out[1][0]]


def exact_attention(case, s):
    if work(case)["flops"] > 6e12:
        return None   # more than about 20 seconds in 64 bits
    ql, kl = lengths(case)
    hq, hk, d = case["q_heads"], case["k_heads"], case["head_dim"]
    if case["items"] * hk > 40000:
        return None
    group, train = hq // hk, case["direction"] == "train"
    out_rows = s["q"].shape[0] * (case["items"] if case["shared"] else 1)
    zeros = lambda rows, heads: torch.zeros(rows, heads, d, dtype=torch.float64, device=device())  # noqa: E731
    out, dq = zeros(out_rows, hq), zeros(s["q"].shape[0], hq)
    dk, dv = zeros(s["k"].shape[0], hk), zeros(s["k"].shape[0], hk)
    q0 = k0 = o0 = 0
    for i in range(case["items"]):
        nq, nk = ql[0] if case["shared"] else ql[i], kl[i]
        qs, os_, ks = slice(q0, q0 + nq), slice(o0, o0 + nq), torch.arange(k0, k0 + nk, device=device())
        if s["key_mask"] is not None:
            ks = ks[s["key_mask"][k0:k0 + nk] != 0]
        if ks.numel():
            q = s["q"][qs].double().view(nq, hk, group, d)
            k, v = s["k"][ks].double(), s["v"][ks].double()
            a = torch.softmax(torch.einsum("rhgd,khd->hgrk", q, k) / d ** 0.5, dim=-1)
            o = torch.einsum("hgrk,khd->rhgd", a, v)
            out[os_] = o.reshape(nq, hq, d)
            if train:
                do = s["d_out"][os_].double().view(nq, hk, group, d)
                da = torch.einsum("rhgd,khd->hgrk", do, v)
                ds = a * (da - (a * da).sum(-1, keepdim=True)) / d ** 0.5
                dq[qs] += torch.einsum("hgrk,khd->rhgd", ds, k).reshape(nq, hq, d)
                dk[ks] = torch.einsum("hgrk,rhgd->khd", ds, q)
                dv[ks] = torch.einsum("hgrk,rhgd->khd", a, do)
        k0 += nk
        o0 += nq
        if not case["shared"]:
            q0 += nq
    return [out, dq, dk, dv] if train else [out]
