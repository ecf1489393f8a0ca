"""The token-state operators on the GPU where a call's surroundings matter: other streams, lent buffers, bad offsets and
positions, values that only some rows hold."""

import pytest
import torch

import states_delta as sd
import states_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def cli():
    import contrastive_late_interaction_gb300 as cli
    return cli


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, dtype=BF16, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda", dtype=F32)).to(dtype)


def offsets(lengths):
    return torch.tensor([0] + list(lengths), dtype=torch.int64).cumsum(0).cuda()


# ----------------------------------------------------------------------------
# a stream other than the current one
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("q_len, k_len", [([1, 2], [5000, 300]), ([300, 40], [500, 90]), ([60], [9000])])
def test_scratch_of_a_call_on_another_stream_is_not_handed_out(cli, q_len, k_len):
    """The call is queued behind a delay on its stream; the current stream allocates and overwrites memory meanwhile."""
    g = gen(41)
    q, k, v = rand(g, sum(q_len), 4, 64), rand(g, sum(k_len), 2, 64), rand(g, sum(k_len), 2, 64)
    d_o, gain, tab = rand(g, sum(q_len), 4, 64), 1 + 0.1 * rand(g, 64, dtype=F32), ref.table(10000, 64).cuda()
    qo, ko = offsets(q_len), offsets(k_len)
    kw = dict(max_query_rows=max(q_len), max_key_rows=max(k_len))

    def step(**on):
        n = cli.norm_rotary_heads(q, tab, q_gain=gain, k=k, k_gain=gain, **on)
        f = cli.cross_attention(n["q"], qo, n["k"], v, ko, **kw, **on)
        b = cli.cross_attention_backward(n["q"], qo, n["k"], v, ko, f["output"], f["lse"], d_o, **kw, **on)
        d = cli.norm_rotary_heads_backward(q, b["d_q"], tab, q_gain=gain, k=k, d_k=b["d_k"], k_gain=gain, **on)
        return [t for r in (n, f, b, d) for t in r.values()]
    want = [t.clone() for t in step()]
    need = max(cli.cross_attention_workspace_bytes(q, qo, k, v, ko, **kw),
               cli.cross_attention_backward_workspace_bytes(q, qo, k, v, ko, **kw),
               cli.norm_rotary_heads_backward_workspace_bytes(64))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = step(stream=s)
    fill = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (256, 4096, need, need) for _ in range(8)]
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del fill


# ----------------------------------------------------------------------------
# maxima, offsets and positions that do not fit
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("maxima", [dict(max_query_rows=0), dict(max_key_rows=0), dict(max_query_rows=0, max_key_rows=0),
                                    dict(max_query_rows=0, max_key_rows=300)])
@pytest.mark.parametrize("k_len", [[20, 30], [9000, 700]])
def test_maxima_of_nothing_are_reported_as_malformed(cli, k_len, maxima):
    """Rows longer than a maximum of 0 are the device's to report, whatever the call is cut into."""
    q, k = rand(gen(1), 3, 2, 64), rand(gen(2), sum(k_len), 2, 64)
    qo, ko = offsets([2, 1]), offsets(k_len)
    f = cli.cross_attention(q, qo, k, k, ko, **maxima)
    with pytest.raises(cli.MalformedError):
        cli.check_device_status(f["device_status"])
    b = cli.cross_attention_backward(q, qo, k, k, ko, torch.zeros_like(q), torch.zeros(3, 2, device="cuda"), q, **maxima)
    with pytest.raises(cli.MalformedError):
        cli.check_device_status(b["device_status"])
    assert not q.isnan().any()   # and PyTorch's own launches find no error of the call's


@pytest.mark.parametrize("rotary_dim", [64, 36, 34])    # half a multiple of 8, of 2, odd
@pytest.mark.parametrize("rows", [40, 3000])            # one block looks at every position, or every warp at its own
@pytest.mark.parametrize("part", ["q", "k"])
@pytest.mark.parametrize("bad", [-1, 50, -2 ** 31])
def test_a_row_outside_the_table_is_reported_and_rotated_as_at_0(cli, bad, part, rows, rotary_dim):
    g, tab = gen(rows), ref.table(50, rotary_dim).cuda()
    x = {"q": rand(g, rows, 3, 64), "k": rand(g, rows + 7, 2, 64)}
    gain = 1 + 0.1 * rand(g, 64, dtype=F32)
    good = {n: torch.randint(0, 50, (t.shape[0],), generator=g, device="cuda", dtype=torch.int32) for n, t in x.items()}
    good[part][rows // 2] = 0
    wrong = {n: p.clone() for n, p in good.items()}
    wrong[part][rows // 2] = bad

    def both(pos):
        out = {n: torch.full_like(t, 9.0) for n, t in x.items()}
        f = cli.norm_rotary_heads(x["q"], tab, pos["q"], q_gain=gain, k=x["k"], k_positions=pos["k"], k_gain=gain, out=out)
        out = {"d_" + n: torch.full_like(t, 9.0) for n, t in x.items()}
        b = cli.norm_rotary_heads_backward(x["q"], x["q"], tab, pos["q"], q_gain=gain, k=x["k"], d_k=x["k"],
                                           k_positions=pos["k"], k_gain=gain, out=out)
        r = cli.rotary_heads(x["q"], tab, pos["q"], k=x["k"], k_positions=pos["k"])
        return f, b, r
    for a, w in zip(both(good), both(wrong)):
        cli.check_device_status(a["device_status"])
        with pytest.raises(cli.MalformedError):
            cli.check_device_status(w["device_status"])
        for name in a:
            if name != "device_status":
                assert torch.equal(a[name], w[name]), name


def test_rotation_of_a_packed_projection_in_place(cli):
    """Queries and keys of one [rows, 3, heads, dim] tensor, in place: the same values, and the values left alone."""
    g, tab = gen(6), ref.table(4096, 64).cuda()
    packed = rand(g, 1500, 3, 6, 64)
    want = cli.rotary_heads(packed[:, 0].contiguous(), tab, k=packed[:, 1].contiguous())
    values = packed[:, 2].clone()
    r = cli.rotary_heads(packed[:, 0], tab, k=packed[:, 1], out={"q": packed[:, 0], "k": packed[:, 1]})
    cli.check_device_status(r["device_status"])
    assert torch.equal(packed[:, 0], want["q"]) and torch.equal(packed[:, 1], want["k"])
    assert torch.equal(packed[:, 2], values)


@pytest.mark.parametrize("items", [3, 300])              # one block checks every item, or the grid shares them
@pytest.mark.parametrize("states", [20, 1500])           # whole items, and items cut along their states
@pytest.mark.parametrize("rows", [1, 40])                # few rows, and tiles
@pytest.mark.parametrize("which", ["k", "q"])
@pytest.mark.parametrize("how", ["down", "first", "last", "past"])
def test_malformed_offsets_are_reported_whatever_the_call_is_cut_into(cli, how, which, rows, states, items):
    q, k = torch.zeros(rows * items, 2, 64, dtype=BF16, device="cuda"), torch.zeros(states * items, 2, 64, dtype=BF16, device="cuda")
    n = {"q": rows, "k": states}[which]
    bad = offsets([n] * items)
    at, value = {"down": (items // 2, 0), "first": (0, 1), "last": (items, n * items - 1), "past": (items - 1, 2 ** 62)}[how]
    bad[at] = value
    off = {"q": offsets([rows] * items), "k": offsets([states] * items), which: bad}
    kw = dict(max_query_rows=rows, max_key_rows=states)
    if how == "down" and items // 2 == 1:
        kw["max_" + ("query" if which == "q" else "key") + "_rows"] = 2 * n   # 0, 0, 2n, 3n is a tape of its own
        off[which] = torch.tensor([0, 2 * n, n, 3 * n], device="cuda")
    f = cli.cross_attention(q, off["q"], k, k, off["k"], **kw)
    with pytest.raises(cli.MalformedError):
        cli.check_device_status(f["device_status"])
    b = cli.cross_attention_backward(q, off["q"], k, k, off["k"], q, torch.zeros(rows * items, 2, device="cuda"), q, **kw)
    with pytest.raises(cli.MalformedError):
        cli.check_device_status(b["device_status"])


# ----------------------------------------------------------------------------
# values that only some rows hold
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_len", [[2, 1, 3], [3, 40, 2]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_dropped_states_have_no_gradient_whatever_the_rows_hold(cli, bad, q_len, dtype):
    g = gen(51)
    k_len = [70, 300, 33]
    q, d_o = rand(g, sum(q_len), 4, 64, dtype=dtype), rand(g, sum(q_len), 4, 64, dtype=dtype)
    k, v = rand(g, sum(k_len), 2, 64, dtype=dtype), rand(g, sum(k_len), 2, 64, dtype=dtype)
    q[0, :, 3], d_o[q_len[0] - 1, :, 5] = bad, bad     # of the first item
    keep = (torch.rand(sum(k_len), generator=g, device="cuda") >= 0.4).to(torch.uint8)
    keep[-k_len[2]:] = 0
    kw = dict(key_mask=keep, max_query_rows=max(q_len), max_key_rows=max(k_len))
    f = cli.cross_attention(q, offsets(q_len), k, v, offsets(k_len), **kw)
    b = cli.cross_attention_backward(q, offsets(q_len), k, v, offsets(k_len), f["output"], f["lse"], d_o, **kw)
    for name in ("d_k", "d_v"):
        assert not b[name][keep == 0].any(), name
        assert b[name][k_len[0]:].isfinite().all(), name
    assert b["d_q"][q_len[0]:].isfinite().all()


def exact_backward(q, k, v, d_o, q_len, k_len, scale, shared=False):
    """Of each item, in 64 bits: (p, dP, delta, ds) [heads, rows, states], its slices of the tapes, and wide k, v."""
    group = q.shape[1] // k.shape[1]
    qa = oa = ka = 0
    for i, nk in enumerate(k_len):
        nq = q.shape[0] if shared else q_len[i]
        qi, oi = q[qa:qa + nq].double(), d_o[oa:oa + nq].double()
        ki, vi = (t[ka:ka + nk].double().repeat_interleave(group, 1) for t in (k, v))
        if nk and nq:
            p = (torch.einsum("qhd,khd->hqk", qi, ki) * scale).softmax(-1)
            dp = torch.einsum("qhd,khd->hqk", oi, vi)
            delta = (p * dp).sum(-1, keepdim=True)
            yield slice(qa, qa + nq), slice(ka, ka + nk), qi, oi, ki, vi, p, dp, delta, p * (dp - delta)
        oa, ka = oa + nq, ka + nk
        qa += 0 if shared else nq


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_len, k_len, hq, hk, d, shared", [
    ([1] * 60 + [20], [300, 37, 900] * 20 + [500], 4, 4, 128, False),   # short items in a long call
    ([1, 300, 2], [700, 400, 90], 4, 2, 64, False), ([17, 5], [9000, 700], 2, 2, 128, False),
    (20, [400, 60, 1300], 2, 2, 72, True),
])
def test_gradient_of_a_dominating_state_on_tiles(cli, q_len, k_len, hq, hk, d, shared, dtype):
    """dK of the calls that go through tiles, where ds = p (dp - delta) is a small difference of large terms.  delta comes
    from sums in 32 bits, so what is left of a state's ds is: its rounding as an operand (u |ds|, or half the smallest
    subnormal), p's relative error r (of ds, and of every state's ds through delta), and the 32-bit sums of dP and of the
    row (e (d + 4) and e n of their terms).  r is as in the reference: 2 es + 2^-20 + e |s|."""
    g = gen(78)
    u, e, tiny = ref.UNIT[dtype], ref.E, ref.TINY[dtype]
    rows_q, rows_k = (q_len if shared else sum(q_len)), sum(k_len)
    out_rows = rows_q * len(k_len) if shared else rows_q
    q, k, v = rand(g, rows_q, hq, d, dtype=dtype, scale=4.0), rand(g, rows_k, hk, d, dtype=dtype), rand(g, rows_k, hk, d, dtype=dtype)
    d_o = rand(g, out_rows, hq, d, dtype=dtype)
    qo, scale = None if shared else offsets(q_len), d ** -0.5
    kw = dict(max_query_rows=rows_q if shared else max(q_len), max_key_rows=max(k_len))
    f = cli.cross_attention(q, qo, k, v, offsets(k_len), **kw)
    got = cli.cross_attention_backward(q, qo, k, v, offsets(k_len), f["output"], f["lse"], d_o, **kw)["d_k"].double()
    largest = 0.0
    for _, ks, qi, oi, ki, vi, p, dp, delta, ds in exact_backward(q, k, v, d_o, q_len, k_len, scale, shared):
        es = (d + 4) * e * scale * torch.einsum("qhd,khd->hqk", qi.abs(), ki.abs()).amax(-1, keepdim=True)
        s = scale * torch.einsum("qhd,khd->hqk", qi, ki).abs().amax(-1, keepdim=True)
        r = 2 * es + 2.0 ** -20 + e * s
        mag = torch.einsum("qhd,khd->hqk", oi.abs(), vi.abs())
        # of delta: the row's ds with p's error, its dP sums, and the sum over n states of ds with the first delta, which
        # is off by u sum |dO O| at most
        first = u * torch.einsum("qhd,hqd->hq", oi.abs(), torch.einsum("hqk,khd->hqd", p, vi).abs())[..., None]
        nk = p.shape[2]
        b_delta = (r * ds.abs() + (d + 4) * e * p * mag + nk * e * (ds.abs() + p * first)).sum(-1, keepdim=True) + r * first
        b = (u + r) * ds.abs() + tiny + p * ((d + 4) * e * mag + b_delta)
        fold = lambda t: t.view(nk, hk, hq // hk, d).sum(2)  # noqa: E731
        want = scale * fold(torch.einsum("hqk,qhd->khd", ds, qi))
        sums = fold(torch.einsum("hqk,qhd->khd", ds.abs(), qi.abs()))
        bound = (u + 2.0 ** -20) * want.abs() + scale * fold(torch.einsum("hqk,qhd->khd", b, qi.abs())) + \
            scale * (p.shape[1] * hq // hk + 4) * e * sums + tiny
        largest = max(largest, p.max().item())
        bad = (got[ks] - want).abs() > bound
        assert not bad.any(), (int(bad.sum()), ((got[ks] - want).abs() / bound).max().item())
    assert largest > 0.9


def half_case(q_len, k_len, hq, hk, d, shared, seed, q_scale, k_scale, v_scale):
    g = gen(seed)
    rows_q, rows_k = (q_len if shared else sum(q_len)), sum(k_len)
    q, k, v = (rand(g, n, h, d, dtype=F16, scale=s) for n, h, s in ((rows_q, hq, q_scale), (rows_k, hk, k_scale), (rows_k, hk, v_scale)))
    d_o = torch.randn(rows_q * len(k_len) if shared else rows_q, hq, d, generator=g, device="cuda")
    qo, ko = None if shared else offsets(q_len), offsets(k_len)
    kw = dict(max_query_rows=rows_q if shared else max(q_len), max_key_rows=max(k_len))
    return q, qo, k, v, ko, d_o, kw


HALVES = [([200], [4096], 2, 2, 64, False), ([40, 3, 300], [700, 1000, 90], 4, 2, 72, False),
          (30, [500, 129], 2, 2, 128, True), ([1, 2], [4096, 300], 2, 2, 64, False), ([4] * 8, [900] * 8, 12, 4, 128, False),
          (1, [3000, 40] * 4, 8, 8, 64, True)]


@pytest.mark.parametrize("case", range(len(HALVES)))
def test_half_precision_gradients_scale_with_the_output_gradient(cli, case):
    """Gradients are linear in d_output.  A power of two in it changes no sum's digits, so that the results differ by
    their own rounding alone: u of themselves, or half the smallest subnormal, on either side."""
    q, qo, k, v, ko, d_o, kw = half_case(*HALVES[case], 90 + case, 2.0, 1.0, 1.0)
    small = (d_o * 2.0 ** -12).to(F16)
    f = cli.cross_attention(q, qo, k, v, ko, **kw)
    a = cli.cross_attention_backward(q, qo, k, v, ko, f["output"], f["lse"], small, **kw)
    b = cli.cross_attention_backward(q, qo, k, v, ko, f["output"], f["lse"], small * 2.0 ** 12, **kw)
    u, tiny = ref.UNIT[F16], ref.TINY[F16]
    for name in ("d_q", "d_k", "d_v"):
        x, y = a[name].double(), b[name].double() * 2.0 ** -12
        bound = u * (1 + u) * (x.abs() + y.abs()) + tiny * (1 + 2.0 ** -12)
        bad = (x - y).abs() > bound
        assert y.abs().max() > 0 and not bad.any(), (name, int(bad.sum()), ((x - y).abs() / bound).max().item())


@pytest.mark.parametrize("q_len, shared", [([200, 30], False), ([1, 2], False), (1, True), (40, True)])
def test_half_precision_gradients_of_large_values(cli, q_len, shared):
    """Weights' gradients past the type's range, between inputs and results within it."""
    k_len = [40, 25]
    q, qo, k, v, ko, d_o, kw = half_case(q_len, k_len, 4, 2, 64, shared, 99, 1e-3, 1e-3, 1e4)
    d_o = (60 * d_o).to(F16)
    f = cli.cross_attention(q, qo, k, v, ko, **kw)
    b = cli.cross_attention_backward(q, qo, k, v, ko, f["output"], f["lse"], d_o, **kw)
    want = ref.attention(q, k, v, None if shared else q_len, k_len, 0.125, d_o=d_o, shared=shared, dtype=F16)
    for name in ("d_q", "d_k", "d_v"):
        value, bound = want[name]
        assert value.abs().max() < 65504
        assert ((b[name].double() - value).abs() <= bound).all() and b[name].isfinite().all(), name


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("case", range(len(sd.CASES)))
def test_few_rows_notes_the_states_that_it_says(cli, case, group, dtype):
    """dK where a state's share of delta's error is kept up to the weight at which states are noted, and not above it."""
    rows, k_len, d = sd.CASES[case]
    if rows % group:
        pytest.skip("no whole query rows")
    g, nq, hk = gen(500 + case), rows // group, 2
    q_len = [nq] * len(k_len)
    q, d_o = (rand(g, sum(q_len), hk * group, d, dtype=dtype, scale=s) for s in (4.0, 1.0))
    k, v = (rand(g, sum(k_len), hk, d, dtype=dtype) for _ in range(2))
    kw = dict(max_query_rows=nq, max_key_rows=max(k_len))
    f = cli.cross_attention(q, offsets(q_len), k, v, offsets(k_len), **kw)
    got = cli.cross_attention_backward(q, offsets(q_len), k, v, offsets(k_len), f["output"], f["lse"], d_o, **kw)["d_k"].double()
    ka, largest = 0, 0.0
    for i, n in enumerate(k_len):
        for h in range(hk):
            rows_of = lambda t: t[i * nq:(i + 1) * nq, h * group:(h + 1) * group].double().reshape(rows, d)  # noqa: E731
            ki, vi = k[ka:ka + n, h].double(), v[ka:ka + n, h].double()
            want, bound, _ = sd.item(rows_of(q), ki, vi, rows_of(d_o), rows_of(f["output"]), d ** -0.5, sd.large_weight(rows), dtype)
            ratio = ((got[ka:ka + n, h] - want).abs() / bound).max().item()
            assert ratio <= 1, (i, h, ratio)
            largest = max(largest, ((got[ka:ka + n, h] - want).abs().max() / want.pow(2).mean().sqrt()).item())
        ka += n
    print(f"largest error {largest:.3f} of the root mean square")


# ----------------------------------------------------------------------------
# rows that share a tile
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_len, k_len, group", [([45, 20], [700, 300], 9), ([150, 3], [260, 900], 1), ([33, 70], [2100, 64], 3),
                                                 ([1, 2], [700, 300], 5), ([60, 5], [9000, 300], 1)])
def test_an_items_bits_do_not_depend_on_the_rows_beside_it(cli, q_len, k_len, group, dtype):
    """The second item's rows lie in the tiles that the first one's end in: large or small, they change no bit of it."""
    g, hk = gen(61), 2
    q, d_o = (rand(g, sum(q_len), hk * group, 64, dtype=dtype) for _ in range(2))
    k, v = (rand(g, sum(k_len), hk, 64, dtype=dtype) for _ in range(2))
    kw = dict(max_query_rows=max(q_len), max_key_rows=max(k_len))

    def first(scale):
        x, y = q.clone(), d_o.clone()
        x[q_len[0]:] *= scale
        f = cli.cross_attention(x, offsets(q_len), k, v, offsets(k_len), **kw)
        b = cli.cross_attention_backward(x, offsets(q_len), k, v, offsets(k_len), f["output"], f["lse"], y, **kw)
        return [t[:q_len[0]] for t in (f["output"], f["lse"], b["d_q"])] + [t[:k_len[0]] for t in (b["d_k"], b["d_v"])]
    want = first(1.0)
    for scale in (30.0, 1e-3):
        for a, b in zip(want, first(scale)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("q_len, k_len, group", [([45, 40], [700, 300], 9), ([60], [3000], 7), ([200, 3], [400, 260], 3)])
def test_results_do_not_depend_on_what_ran_before(cli, q_len, k_len, group):
    """Groups that do not divide 128 leave rows of a tile without queries, which hold whatever was there."""
    g, hk = gen(62), 2
    q, d_o = (rand(g, sum(q_len), hk * group, 96) for _ in range(2))
    k, v = (rand(g, sum(k_len), hk, 96) for _ in range(2))
    kw = dict(max_query_rows=max(q_len), max_key_rows=max(k_len))

    def both(q):
        f = cli.cross_attention(q, offsets(q_len), k, v, offsets(k_len), **kw)
        b = cli.cross_attention_backward(q, offsets(q_len), k, v, offsets(k_len), f["output"], f["lse"], d_o, **kw)
        return [f["output"], f["lse"], b["d_q"], b["d_k"], b["d_v"]]
    other = rand(g, 600, 4, 128)
    want = both(q)
    for scale in (100.0, 1e-3, 3e4):    # a call whose tiles are full, with large and small rows
        x = (scale * other).to(BF16)
        cli.cross_attention(x, offsets([600]), x, x, offsets([600]), max_query_rows=600)
        for a, b in zip(want, both(q)):
            assert torch.equal(a, b)
