"""The token-state operators on the GPU against the 64-bit reference, within the bounds it derives."""

import pytest
import torch

import states_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def cli():
    import contrastive_late_interaction_gb300 as cli
    return cli


def rand(g, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda", dtype=F32)).to(dtype)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def within(got, want, bound, what):
    bad = (got.double() - want).abs() > bound
    assert not bad.any() and torch.isfinite(got).all(), \
        f"{what}: {int(bad.sum())} of {bad.numel()} off, {((got.double() - want).abs() / bound).nan_to_num(posinf=1e9).max():.3g} of the bound"


# ----------------------------------------------------------------------------
# rotation
# ----------------------------------------------------------------------------

def layouts(t, kind):
    """The values of t [rows, heads, dim] in memory of another layout."""
    rows, heads, dim = t.shape
    if kind == "padded":
        wide = torch.full((rows, heads + 1, dim + 8), 7.0, dtype=t.dtype, device=t.device)
        wide[:, :heads, :dim] = t
        return wide[:, :heads, :dim]
    if kind == "heads_first":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    return t


ROTATIONS = [
    # rows, q heads, k heads (0: no keys), dim, rotary_dim, interleaved
    (1, 1, 0, 8, 2, False), (1, 8, 2, 128, 128, False), (3, 5, 3, 64, 64, True), (37, 4, 4, 64, 32, False),
    (129, 3, 1, 80, 76, False), (65, 2, 2, 96, 34, False), (50, 12, 4, 96, 6, True), (33, 33, 1, 256, 256, False),
    (17, 2, 7, 256, 254, True), (9, 1, 1, 104, 16, False), (300, 16, 16, 64, 64, False), (2500, 2, 1, 24, 24, False),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("layout", ["packed", "padded", "heads_first"])
@pytest.mark.parametrize("shape", ROTATIONS)
def test_rotation_and_its_gradient(cli, shape, layout, dtype):
    rows, hq, hk, d, n, inter = shape
    g = gen(rows * d + n)
    tab = ref.table(1000, n).cuda()
    u = ref.UNIT[dtype]
    pos = [torch.randint(0, 1000, (r,), generator=g, device="cuda", dtype=torch.int32) for r in (rows, rows + 2)]
    q = layouts(rand(g, rows, hq, d, dtype=dtype), layout)
    k = layouts(rand(g, rows + 2, hk, d, dtype=dtype), layout) if hk else None
    f = cli.rotary_heads(q, tab, pos[0], k=k, k_positions=pos[1] if hk else None, interleaved=inter)
    b = cli.rotary_heads_backward(q, tab, pos[0], d_k=k, k_positions=pos[1] if hk else None, interleaved=inter)
    cli.check_device_status(f["device_status"])
    cli.check_device_status(b["device_status"])
    for x, p, name in ((q, pos[0], "q"), (k, pos[1], "k")):
        if x is None:
            assert f[name] is None and b["d_" + name] is None
            continue
        for back, got in ((False, f[name]), (True, b["d_" + name])):
            y, m = ref.rotate(x.double(), tab, p.long(), inter, back)
            within(got, y, u * y.abs() + 4 * ref.E * m + ref.TINY[dtype], f"{name} back={back}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("layout", ["packed", "padded"])
@pytest.mark.parametrize("shape", ROTATIONS)
def test_norm_rotation_and_its_gradient(cli, shape, layout, dtype):
    rows, hq, hk, d, n, inter = shape
    g = gen(rows * d + n + 1)
    tab = ref.table(1000, n).cuda()
    u, e, eps = ref.UNIT[dtype], ref.E, 1e-5
    for x_scale in (1.0, 0.01):   # the second one near epsilon
        make = lambda r, h: layouts(rand(g, r, h, d, dtype=dtype, scale=x_scale), layout)  # noqa: E731
        xs = {"q": make(rows, hq), "k": make(rows + 2, hk) if hk else None}
        ds = {"q": layouts(rand(g, rows, hq, d, dtype=dtype), layout),
              "k": layouts(rand(g, rows + 2, hk, d, dtype=dtype), layout) if hk else None}
        gains = {"q": 1 + 0.3 * rand(g, d), "k": 1 + 0.3 * rand(g, d) if rows % 2 else None}
        pos = {"q": torch.randint(0, 1000, (rows,), generator=g, device="cuda", dtype=torch.int32), "k": None}
        kw = dict(q_gain=gains["q"], k=xs["k"], k_gain=gains["k"] if hk else None, interleaved=inter, epsilon=eps)
        if rows + 2 > 1000:
            pos["k"] = torch.arange(rows + 2, device="cuda", dtype=torch.int32) % 1000
        f = cli.norm_rotary_heads(xs["q"], tab, pos["q"], k_positions=pos["k"], **kw)
        b = cli.norm_rotary_heads_backward(xs["q"], ds["q"], tab, pos["q"], d_k=ds["k"], k_positions=pos["k"], **kw)
        cli.check_device_status(f["device_status"])
        cli.check_device_status(b["device_status"])
        for name in ("q", "k"):
            x = xs[name]
            if x is None:
                continue
            p = pos[name].long() if pos[name] is not None else torch.arange(x.shape[0], device="cuda")
            gain = gains[name].double() if gains[name] is not None else torch.ones(d, dtype=torch.float64, device="cuda")
            y, m = ref.norm_rotate(x.double(), gain, tab, p, inter, eps)
            factor = (d / 2 + 8) * e    # of the norm's factor and the products with it
            within(f[name], y, u * y.abs() + (4 * e + factor) * m + ref.TINY[dtype], f"{name} x{x_scale}")
            dx, mx, dg, mg = ref.norm_rotate_backward(x.double(), ds[name].double(), gain, tab, p, inter, eps)
            within(b["d_" + name], dx, u * dx.abs() + (3 * factor + (d + 8) * e) * mx + ref.TINY[dtype],
                   f"d_{name} x{x_scale}")
            got = b[f"d_{name}_gain"]
            if gains[name] is None:
                assert got is None
            else:   # a sum of rows * heads terms in 32 bits, in blocks of at most a few thousand additions each
                within(got, dg, (factor + 8 * e + 4096 * e) * mg, f"d_{name}_gain x{x_scale}")


def test_norm_gradient_matches_differences(cli):
    g = gen(5)
    tab = ref.table(64, 48).cuda()
    x, dy, gain = rand(g, 40, 3, 64), rand(g, 40, 3, 64), 1 + 0.3 * rand(g, 64)
    b = cli.norm_rotary_heads_backward(x, dy, tab, q_gain=gain, epsilon=1e-5)

    def loss(x, gain):
        return (cli.norm_rotary_heads(x, tab, q_gain=gain, epsilon=1e-5)["q"].double() * dy.double()).sum().item()
    h = 2.0 ** -8
    ex, eg = rand(g, 40, 3, 64), rand(g, 64)
    terms = 40 * 3 * 64
    # a difference is off by h^2 (third derivatives, here at most about 10 a term) and by the outputs' rounding over h
    tol = 10 * h * h * terms ** 0.5 * 4 + 8 * ref.E * terms / h
    want = (loss(x + h * ex, gain) - loss(x - h * ex, gain)) / (2 * h)
    assert abs((b["d_q"].double() * ex.double()).sum().item() - want) <= tol
    want = (loss(x, gain + h * eg) - loss(x, gain - h * eg)) / (2 * h)
    assert abs((b["d_q_gain"].double() * eg.double()).sum().item() - want) <= tol


def test_rotation_in_place_and_repeatable(cli):
    g = gen(6)
    tab = ref.table(4096, 64).cuda()
    q = rand(g, 700, 6, 64, dtype=BF16)
    want = cli.rotary_heads(q, tab)["q"]
    work = q.clone()
    got = cli.rotary_heads(work, tab, out={"q": work})["q"]
    assert got.data_ptr() == work.data_ptr() and torch.equal(got, want)
    packed = rand(g, 700, 3, 6, 64, dtype=BF16)     # queries, keys and values of one projection
    r = cli.rotary_heads(packed[:, 0], tab, k=packed[:, 1], out={"q": packed[:, 0], "k": packed[:, 1]})
    cli.check_device_status(r["device_status"])
    dy = rand(g, 700, 6, 64, dtype=BF16)
    gain = torch.ones(64, device="cuda")
    a = cli.norm_rotary_heads_backward(q, dy, tab, q_gain=gain)
    b = cli.norm_rotary_heads_backward(q, dy, tab, q_gain=gain)
    assert torch.equal(a["d_q_gain"], b["d_q_gain"]) and torch.equal(a["d_q"], b["d_q"])


def test_rotation_of_no_rows(cli):
    tab = ref.table(16, 64).cuda()
    q = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    assert cli.rotary_heads(q, tab)["q"].shape == (0, 2, 64)
    gain = torch.ones(64, device="cuda")
    r = cli.norm_rotary_heads_backward(q, q, tab, q_gain=gain)
    assert torch.equal(r["d_q_gain"], torch.zeros(64, device="cuda"))


@pytest.mark.parametrize("bad", [-1, 16, 2 ** 31 - 1, -2 ** 31])
def test_position_outside_the_table_is_reported(cli, bad):
    tab = ref.table(16, 64).cuda()
    q = torch.zeros(9, 2, 64, dtype=BF16, device="cuda")
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    pos[4] = bad
    with pytest.raises(Exception, match="malformed"):
        cli.check_device_status(cli.rotary_heads(q, tab, pos)["device_status"])
    long = torch.zeros(17, 2, 64, dtype=BF16, device="cuda")
    with pytest.raises(Exception, match="malformed"):
        cli.check_device_status(cli.rotary_heads(long, tab)["device_status"])


def test_tables(cli):
    import math
    n, p = 48, 5000
    pos = torch.arange(p, dtype=torch.float64)[:, None]
    i = torch.arange(n // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / n)

    def check(freq, amplitude=1.0, **kw):
        t = cli.rotary_table(p, n, **kw)["table"].cpu().double()
        a = pos * freq
        want = amplitude * torch.stack((a.cos(), a.sin()), -1)
        # one rounding to 32 bits, and angles of at most 5000 rad to 2^-52 of themselves on either side
        assert (t - want).abs().max() <= 2.0 ** -24 * amplitude + 1e-11
    check(f)
    check(f / 4, scaling="linear", factor=4.0)
    check((10000.0 * 4 ** (n / (n - 2))) ** (-2 * i / n), scaling="ntk", factor=4.0)
    pair = lambda turns: n * math.log(4096 / (2 * math.pi * turns)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), n - 1)
    blend = ((i - lo) / (hi - lo)).clamp(0, 1)
    check(f * (1 - blend) + f / 8 * blend, 0.1 * math.log(8) + 1, scaling="yarn", factor=8.0, trained_positions=4096)


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------

def offsets(lengths):
    return torch.tensor([0] + list(lengths), dtype=torch.int64).cumsum(0).cuda()


def attend(cli, q_len, k_len, hq, hk, d, dtype, seed, mask=None, shared=False, layout="packed", scale=None,
           poison=True, q_scale=2.0):
    """Forward and backward on the GPU and the reference's values and bounds."""
    g = gen(seed)
    rows_q, rows_k = (q_len if shared else sum(q_len)), sum(k_len)
    out_rows = rows_q * len(k_len) if shared else rows_q
    q, k, v = rand(g, rows_q, hq, d, dtype=dtype, scale=q_scale), rand(g, rows_k, hk, d, dtype=dtype), \
        rand(g, rows_k, hk, d, dtype=dtype)
    d_o = rand(g, out_rows, hq, d, dtype=dtype)
    keep = None
    if mask is not None:
        keep = (torch.rand(rows_k, generator=g, device="cuda") >= mask).to(torch.uint8)
        at = 0
        for i, n in enumerate(k_len):      # every third item keeps nothing
            if i % 3 == 2:
                keep[at:at + n] = 0
            at += n
    scale = d ** -0.5 if scale is None else scale
    want = ref.attention(q, k, v, None if shared else q_len, k_len, scale, keep, d_o, shared, dtype)
    if keep is not None and poison:
        k[keep == 0] = float("nan")
        v[keep == 0] = float("inf")
    out = {}
    if layout == "packed_kv":
        kv = torch.stack((k, v), dim=1)            # [rows, 2, heads, dim]
        k, v = kv[:, 0], kv[:, 1]
        d_kv = torch.full_like(kv, 9.0)
        out = {"d_k": d_kv[:, 0], "d_v": d_kv[:, 1]}
    elif layout != "packed":
        q, k, v, d_o = (layouts(t, layout) for t in (q, k, v, d_o))
    qo = None if shared else offsets(q_len)
    kw = dict(key_mask=keep, scale=scale, max_query_rows=rows_q if shared else max(q_len), max_key_rows=max(k_len))
    f = cli.cross_attention(q, qo, k, v, offsets(k_len), **kw)
    cli.check_device_status(f["device_status"])
    b = cli.cross_attention_backward(q, qo, k, v, offsets(k_len), f["output"], f["lse"], d_o, out=out, **kw)
    cli.check_device_status(b["device_status"])
    got = {"output": f["output"], "lse": f["lse"], "d_q": b["d_q"], "d_k": b["d_k"], "d_v": b["d_v"]}
    return got, want


def check(got, want):
    lse, bound = want["lse"]
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(got["lse"]) & (got["lse"] < 0), empty)
    assert ((got["lse"].double() - lse)[~empty].abs() <= bound[~empty]).all()
    for name in ("output", "d_q", "d_k", "d_v"):
        within(got[name], *want[name], name)


CASES = [
    # query lengths (a number: shared), state lengths, query heads, key heads, head_dim
    ([1], [1], 1, 1, 8), ([1], [0], 2, 1, 64), ([0, 1], [3, 5], 4, 2, 64), ([1, 1, 1], [300, 0, 17], 8, 2, 128),
    ([5], [4096], 4, 1, 64), ([3, 2, 1], [129, 127, 128], 3, 1, 72), ([16], [1000], 1, 1, 128),
    ([17, 0, 2], [31, 200, 33], 6, 6, 40), ([128], [128], 2, 2, 128), ([129], [127], 2, 2, 128),
    ([127, 1, 255], [257, 384, 1], 2, 1, 64), ([300, 20], [65, 700], 6, 2, 72), ([64, 64], [256, 100], 16, 4, 64),
    ([257], [640], 4, 1, 128), ([40], [130], 7, 1, 96), ([90, 33], [150, 513], 5, 5, 120), ([2, 9], [300, 77], 128, 1, 16),
    ([700], [1100], 3, 3, 128), ([12] * 40, [13] * 40, 2, 2, 32), (1, [64, 0, 500, 1], 4, 4, 64), (1, [700], 8, 1, 128),
    (3, [31, 129, 64], 2, 2, 64), (64, [200, 0, 129], 4, 2, 64), (150, [140, 300], 2, 2, 128), (1, [1] * 70, 2, 2, 8),
    ([385], [129], 3, 1, 88), ([1, 600], [2000, 3], 2, 2, 56),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("mask", [None, 0.3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_and_its_gradient(cli, case, mask, dtype):
    q_len, k_len, hq, hk, d = CASES[case]
    check(*attend(cli, q_len, k_len, hq, hk, d, dtype, 100 + case, mask, shared=isinstance(q_len, int)))


@pytest.mark.parametrize("mask", [None, 0.3])
@pytest.mark.parametrize("q_len, k_len, h, d", [
    ([200], [9000], 2, 128), ([40, 3, 0, 17], [5000, 700, 6000, 0], 3, 72), (20, [4000, 100, 1537], 2, 64),
    ([130], [512 * 5 + 1], 1, 8), ([16] * 40, [70, 130] * 20, 4, 128), (10, [33, 0, 257] * 60, 1, 96),
])
def test_attention_cut_along_the_states_or_into_many_items(cli, q_len, k_len, h, d, mask):
    check(*attend(cli, q_len, k_len, h, h, d, BF16, 310, mask, shared=isinstance(q_len, int)))


@pytest.mark.parametrize("layout", ["padded", "heads_first", "packed_kv"])
@pytest.mark.parametrize("case", [3, 11, 13, 20, 22])
def test_attention_layouts(cli, case, layout):
    q_len, k_len, hq, hk, d = CASES[case]
    check(*attend(cli, q_len, k_len, hq, hk, d, BF16, 300 + case, 0.2, shared=isinstance(q_len, int), layout=layout))


@pytest.mark.parametrize("q_len, k_len", [([200], [400]), ([2], [3000]), (1, [900, 40])])
@pytest.mark.parametrize("q_scale", [1e-3, 30.0])
def test_attention_of_flat_and_sharp_rows(cli, q_len, k_len, q_scale):
    """Nearly equal scores, and scores of hundreds, where one state takes all."""
    check(*attend(cli, q_len, k_len, 4, 2, 64, BF16, 400, shared=isinstance(q_len, int), q_scale=q_scale))


@pytest.mark.parametrize("q_len, k_len", [([200, 30], [400, 77]), ([2], [700]), (1, [300, 40])])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.0])
@pytest.mark.parametrize("mask", [None, 0.3])
def test_attention_scales(cli, q_len, k_len, scale, mask):
    """Scores that are negated, all equal, or not shrunk."""
    check(*attend(cli, q_len, k_len, 4, 2, 64, BF16, 500, mask, shared=isinstance(q_len, int), scale=scale))


@pytest.mark.parametrize("q_len, k_len", [([150, 3], [260, 130]), ([1, 1], [260, 130])])
def test_states_past_an_item_do_not_reach_it(cli, q_len, k_len):
    """Neighbouring items' rows, whatever they hold, change nothing: not in the tile that an item ends in."""
    g = gen(7)
    q, k, v = rand(g, sum(q_len), 4, 64, dtype=BF16), rand(g, sum(k_len), 2, 64, dtype=BF16), \
        rand(g, sum(k_len), 2, 64, dtype=BF16)
    d_o = rand(g, sum(q_len), 4, 64, dtype=BF16)
    kw = dict(max_query_rows=max(q_len), max_key_rows=max(k_len))

    def both(q, k, v, d_o):
        f = cli.cross_attention(q, offsets(q_len), k, v, offsets(k_len), **kw)
        b = cli.cross_attention_backward(q, offsets(q_len), k, v, offsets(k_len), f["output"], f["lse"], d_o, **kw)
        return (f["output"], b["d_q"]), (b["d_k"], b["d_v"])
    a_q, a_k = both(q, k, v, d_o)
    for t, n in ((q, q_len), (k, k_len), (v, k_len), (d_o, q_len)):
        t[n[0]:] = float("nan")            # the second item
    b_q, b_k = both(q, k, v, d_o)
    for a, b in zip(a_q, b_q):
        assert torch.equal(a[:q_len[0]], b[:q_len[0]]) and torch.isnan(b[q_len[0]:]).all()
    for a, b in zip(a_k, b_k):
        assert torch.equal(a[:k_len[0]], b[:k_len[0]])


@pytest.mark.parametrize("q_len, k_len, hq", [([300, 40], [500, 90], 4), ([1, 1], [5000, 9], 8), (2, [900] * 5, 4)])
def test_attention_is_repeatable_and_stream_ordered(cli, q_len, k_len, hq):
    shared = isinstance(q_len, int)
    a, _ = attend(cli, q_len, k_len, hq, 2, 64, BF16, 11, shared=shared)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, _ = attend(cli, q_len, k_len, hq, 2, 64, BF16, 11, shared=shared)
    torch.cuda.current_stream().wait_stream(s)
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("q_len, k_len, hq, hk, d, shared", [
    (1, [200, 37, 1024, 700, 0, 3] * 8, 8, 8, 128, True), ([1, 3, 2], [5000, 90, 400], 8, 2, 64, False),
    ([4], [700], 12, 3, 72, False),
])
def test_gradient_of_a_state_that_has_most_of_a_row(cli, q_len, k_len, hq, hk, d, shared):
    """dK in bf16 where ds = p (dp - delta) is a small difference: with delta from the rounded output alone it is off by up to
    u scale p sum |dO O| |q|, u the type's unit roundoff.  Of that at most a sixteenth may be left (a state with a
    weight above it is computed with delta from 32-bit sums), beside dK's own rounding, two roundings' worth of the
    16-bit halves (u^2) and the sums in 32 bits (2^-15 of their terms, as p and delta take part in all of them)."""
    g, dtype = gen(77), BF16
    rows_q, rows_k = (q_len if shared else sum(q_len)), sum(k_len)
    out_rows = rows_q * len(k_len) if shared else rows_q
    q, k, v = rand(g, rows_q, hq, d, dtype=dtype, scale=4.0), rand(g, rows_k, hk, d, dtype=dtype), rand(g, rows_k, hk, d, dtype=dtype)
    d_o = rand(g, out_rows, hq, d, dtype=dtype)
    qo = None if shared else offsets(q_len)
    kw = dict(max_query_rows=rows_q if shared else max(q_len), max_key_rows=max(k_len))
    f = cli.cross_attention(q, qo, k, v, offsets(k_len), **kw)
    got = cli.cross_attention_backward(q, qo, k, v, offsets(k_len), f["output"], f["lse"], d_o, **kw)["d_k"].double()
    u, scale = 2.0 ** -8, d ** -0.5
    ka = qa = 0
    largest = 0.0
    for i, nk in enumerate(k_len):
        nq = rows_q if shared else q_len[i]
        qi = q[:nq] if shared else q[qa:qa + nq]
        wide = lambda t: t.double().repeat_interleave(hq // hk, 1)  # noqa: E731
        qi, oi, ki, vi = qi.double(), d_o[qa:qa + nq].double(), wide(k[ka:ka + nk]), wide(v[ka:ka + nk])
        p = (torch.einsum("qhd,khd->hqk", qi, ki) * scale).softmax(-1)
        o = torch.einsum("hqk,khd->qhd", p, vi)
        delta = (oi * o).sum(-1).T[:, :, None]
        ds = p * (torch.einsum("qhd,khd->hqk", oi, vi) - delta)
        terms = p * (torch.einsum("qhd,khd->hqk", oi.abs(), vi.abs()) + (oi * o).abs().sum(-1).T[:, :, None])
        spread = p.clamp(max=1 / 16) * u * (oi * o).abs().sum(-1).T[:, :, None] + (2.0 ** -15 + u * u) * terms
        fold = lambda t: t.view(nk, hk, hq // hk, d).sum(2)  # noqa: E731
        want = scale * fold(torch.einsum("hqk,qhd->khd", ds, qi))
        bound = u * want.abs() + scale * fold(torch.einsum("hqk,qhd->khd", spread, qi.abs())) + ref.TINY[dtype]
        if nk:
            largest = max(largest, p.max().item())
            assert ((got[ka:ka + nk] - want).abs() <= bound).all()
        ka, qa = ka + nk, qa + nq
    assert largest > 0.9


def test_attention_without_lse_and_with_loose_maxima(cli):
    g = gen(12)
    q_len, k_len = [1, 1, 1], [40, 500, 7]
    q, k, v = rand(g, 3, 4, 64, dtype=BF16), rand(g, 547, 4, 64, dtype=BF16), rand(g, 547, 4, 64, dtype=BF16)
    a = cli.cross_attention(q, offsets(q_len), k, v, offsets(k_len), want_lse=False, max_query_rows=1, max_key_rows=500)
    b = cli.cross_attention(q, offsets(q_len), k, v, offsets(k_len))       # the tapes' rows bound the items'
    assert a["lse"] is None
    want = ref.attention(q, k, v, q_len, k_len, 0.125)
    within(a["output"], *want["output"], "tight")
    within(b["output"], *want["output"], "loose")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("which, bad", [("k", [0, 9, 5, 20]), ("k", [1, 5, 9, 20]), ("k", [0, 5, 9, 19]),
                                        ("k", [0, 5, 9, 2 ** 62]), ("k", [0, 5, -1, 20]), ("q", [0, 4, 2, 6]),
                                        ("q", [0, 2, 4, 7]), ("q", [2, 2, 4, 6])])
def test_malformed_offsets_are_reported(cli, which, bad, many):
    scale = 100 if many else 1
    q = torch.zeros(6 * scale, 2, 64, dtype=BF16, device="cuda")
    k = torch.zeros(20 * scale, 2, 64, dtype=BF16, device="cuda")
    qo, ko = offsets([2 * scale] * 3), offsets([5 * scale, 4 * scale, 11 * scale])
    bad = torch.tensor([b * scale if abs(b) < 100 else b for b in bad], device="cuda")
    args = (q, bad if which == "q" else qo, k, k, bad if which == "k" else ko)
    f = cli.cross_attention(*args)
    with pytest.raises(Exception, match="malformed"):
        cli.check_device_status(f["device_status"])
    b = cli.cross_attention_backward(*args, torch.zeros_like(q), torch.zeros(6 * scale, 2, device="cuda"), q)
    with pytest.raises(Exception, match="malformed"):
        cli.check_device_status(b["device_status"])
    torch.cuda.synchronize()


@pytest.mark.parametrize("over", [dict(max_query_rows=1), dict(max_key_rows=10)])
def test_an_item_longer_than_the_maxima_is_reported(cli, over):
    q, k = torch.zeros(6, 2, 64, dtype=BF16, device="cuda"), torch.zeros(20, 2, 64, dtype=BF16, device="cuda")
    f = cli.cross_attention(q, offsets([2, 2, 2]), k, k, offsets([5, 4, 11]), **over)
    with pytest.raises(Exception, match="malformed"):
        cli.check_device_status(f["device_status"])


def test_attention_of_no_rows(cli):
    e = lambda n: torch.zeros(n, 2, 64, dtype=BF16, device="cuda")  # noqa: E731
    f = cli.cross_attention(e(0), offsets([0, 0]), e(9), e(9), offsets([4, 5]))
    cli.check_device_status(f["device_status"])
    b = cli.cross_attention_backward(e(0), offsets([0, 0]), e(9), e(9), offsets([4, 5]), f["output"], f["lse"], e(0))
    cli.check_device_status(b["device_status"])
    assert not b["d_k"].any() and not b["d_v"].any()
    f = cli.cross_attention(e(3), offsets([1, 2]), e(0), e(0), offsets([0, 0]))
    cli.check_device_status(f["device_status"])
    assert not f["output"].any() and torch.isinf(f["lse"]).all()
    b = cli.cross_attention_backward(e(3), offsets([1, 2]), e(0), e(0), offsets([0, 0]), f["output"], f["lse"], e(3))
    cli.check_device_status(b["device_status"])
    assert not b["d_q"].any()


def test_offsets_past_32_bits(cli):
    """Rows whose byte offset in a tape passes 2^32 (and whose element offset passes 2^31)."""
    heads, d, rows = 16, 128, 1100000       # 4.5 GB a tensor
    g = gen(13)
    k = torch.zeros(rows, heads, d, dtype=BF16, device="cuda")
    v = torch.zeros(rows, heads, d, dtype=BF16, device="cuda")
    n = 300
    k[-n:], v[-n:] = rand(g, n, heads, d, dtype=BF16), rand(g, n, heads, d, dtype=BF16)
    for nq in (1, 200):
        q, d_o = rand(g, nq, heads, d, dtype=BF16), rand(g, nq, heads, d, dtype=BF16)
        qo, ko = offsets([0, nq]), offsets([rows - n, n])
        f = cli.cross_attention(q, qo, k, v, ko, max_query_rows=nq)
        cli.check_device_status(f["device_status"])
        want = ref.attention(q, k[-n:], v[-n:], [nq], [n], d ** -0.5, d_o=d_o)
        within(f["output"], *want["output"], "output")
        b = cli.cross_attention_backward(q, qo, k, v, ko, f["output"], f["lse"], d_o, max_query_rows=nq)
        cli.check_device_status(b["device_status"])
        within(b["d_k"][-n:], *want["d_k"], "d_k")
        within(b["d_v"][-n:], *want["d_v"], "d_v")
        assert not b["d_k"][:5].any() and not b["d_k"][rows - n - 5:rows - n].any()
        del b


def test_calls_in_a_captured_graph(cli):
    """A captured step (tiles and few rows, forward and backward, rotation before it) replays on new contents."""
    g = gen(21)
    tab = ref.table(512, 64).cuda()
    k_len = [300, 45, 128]
    ko = offsets(k_len)
    k, v = rand(g, sum(k_len), 2, 64, dtype=BF16), rand(g, sum(k_len), 2, 64, dtype=BF16)

    def step(q, qo, d_o, most):
        n = cli.rotary_heads(q, tab, k=k)
        f = cli.cross_attention(n["q"], qo, n["k"], v, ko, max_query_rows=most, max_key_rows=300)
        b = cli.cross_attention_backward(n["q"], qo, n["k"], v, ko, f["output"], f["lse"], d_o, max_query_rows=most,
                                         max_key_rows=300)
        return [f["output"], f["lse"], b["d_q"], b["d_k"], b["d_v"], f["device_status"], b["device_status"]]
    for q_len in ([70, 3, 200], [1, 2, 1]):
        qo = offsets(q_len)
        q, d_o = rand(g, sum(q_len), 8, 64, dtype=BF16), rand(g, sum(q_len), 8, 64, dtype=BF16)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(q, qo, d_o, max(q_len))
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(q, qo, d_o, max(q_len))
        for seed in (22, 23):
            g2 = gen(seed)
            q.copy_(rand(g2, *q.shape, dtype=BF16))
            k.copy_(rand(g2, *k.shape, dtype=BF16))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            for a, b in zip(got, step(q, qo, d_o, max(q_len))):
                assert torch.equal(a, b)


def test_outputs_workspace_and_status_are_the_callers(cli):
    g = gen(31)
    q_len, k_len = [70, 9], [140, 200]
    qo, ko = offsets(q_len), offsets(k_len)
    q, d_o = rand(g, 79, 4, 64, dtype=BF16), rand(g, 79, 4, 64, dtype=BF16)
    k, v = rand(g, 340, 2, 64, dtype=BF16), rand(g, 340, 2, 64, dtype=BF16)
    kw = dict(max_query_rows=70, max_key_rows=200)
    a = cli.cross_attention(q, qo, k, v, ko, **kw)
    b = cli.cross_attention_backward(q, qo, k, v, ko, a["output"], a["lse"], d_o, **kw)
    for names, call, need, want in (
            (("output", "lse"), lambda **o: cli.cross_attention(q, qo, k, v, ko, **kw, **o),
             cli.cross_attention_workspace_bytes(q, qo, k, v, ko, **kw), a),
            (("d_q", "d_k", "d_v"), lambda **o: cli.cross_attention_backward(q, qo, k, v, ko, a["output"], a["lse"], d_o,
                                                                             **kw, **o),
             cli.cross_attention_backward_workspace_bytes(q, qo, k, v, ko, **kw), b)):
        out = {n: torch.full_like(want[n], 9.0) for n in names}
        ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
        st = torch.full((1,), 77, dtype=torch.int32, device="cuda")
        r = call(out=out, workspace=ws[:need], device_status=st)
        assert int(st.item()) == 0 and (ws[need:] == 0xAB).all()
        for n in names:
            assert r[n] is out[n] and torch.equal(out[n], want[n]), n
        with pytest.raises(cli.InvalidArgumentError):
            call(workspace=ws[:need - 1])


def test_pooling_example_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "pool_states.py")
    spec = importlib.util.spec_from_file_location("pool_states", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(items=64, heads=4, dim=64, steps=20, say=lambda s: None)
    assert all(np_isfinite(x) for x in losses) and losses[-1] < 0.8 * losses[0], losses


def np_isfinite(x):
    return x == x and abs(x) != float("inf")
