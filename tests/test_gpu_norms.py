"""Layer norm, dropout and the residual join on the GPU against the 64-bit reference, within the bounds it derives."""

import pytest
import torch

import norms_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SEED, STEP, SITE = -0x123456789ABCDEF, (5 << 32) + 77, 65535   # a seed with its highest bit set


@pytest.fixture(scope="module")
def cli():
    import contrastive_late_interaction_gb300 as cli
    return cli


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda") + shift).to(dtype)


def seed_of(seed=SEED, step=STEP):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def factors(rows, width, rate):
    """The mask of the reference; few rows of it are drawn and the GPU's own dropout checked against them."""
    return ref.factors(rows, width, rate, SEED % 2 ** 64, STEP, SITE).cuda()


def within(got, want, what):
    value, bound = want
    off = (got.double() - value).abs()
    assert torch.isfinite(got).all() and not (off > bound).any(), \
        f"{what}: {int((off > bound).sum())} of {off.numel()} off, {(off / bound).nan_to_num(posinf=1e9).max():.3g} of the bound"


def layout(t, kind):
    """The values of t [rows, width] in memory of another layout; the rest of it is NaN."""
    if kind == "packed":
        return t
    rows, width = t.shape
    off, gap = {"padded": (8, 8), "fours": (4, 12 - width % 4), "odd": (1, 3)}[kind]
    wide = torch.full((rows, off + width + gap), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, off:off + width] = t
    return wide[:, off:off + width]


TYPES = [(BF16, BF16), (F16, F16), (F32, F32), (BF16, F32), (F16, F32)]   # branch and output, stream
# One chunk and less of a row, teams of 1 to 32 lanes and of several warps, widths no chunk divides, the widest.
SHAPES = [(1, 1), (3, 2), (5, 7), (9, 8), (2, 12), (33, 64), (17, 100), (70, 96), (9, 256), (7, 260), (130, 264),
          (5, 520), (6, 1000), (3, 1024), (4, 1026), (11, 1032), (2, 2048), (3, 4100), (2, 8192), (1, 8200), (2, 8193),
          (2, 16384), (1, 16383)]
LAYOUTS = ["packed", "padded", "fours", "odd"]


def vectors(g, width):
    return rand(g, width, scale=0.3, shift=1.0), rand(g, width)


@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("types", TYPES)
def test_layer_norm_and_its_gradient(cli, types, kind):
    dtype, stream = types
    for rows, width in SHAPES:
        what = f"{rows} x {width}"
        g = gen(rows * 20000 + width)
        x, d_y = rand(g, rows, width, dtype=stream, scale=1.5, shift=0.3), rand(g, rows, width, dtype=dtype)
        gain, bias = vectors(g, width)
        xl = layout(x, kind)
        f = cli.layer_norm(xl, gain, bias, dtype=dtype)
        within(f["output"], ref.layer_norm(x, gain, bias, 1e-5, dtype), what)
        b = cli.layer_norm_backward(xl, layout(d_y, kind), gain, bias)
        want = ref.layer_norm_backward(x, d_y, gain, 1e-5, stream)
        for name in ("d_x", "d_gain", "d_bias"):
            within(b[name], want[name], f"{what} {name}")


@pytest.mark.parametrize("rate", [0.0, 0.1, 0.75])
@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("types", TYPES)
def test_join_and_its_gradient(cli, types, kind, rate):
    dtype, stream = types
    seed = seed_of() if rate else None
    for rows, width in SHAPES[::2] if kind == "fours" else SHAPES[1::2]:
        what = f"{rows} x {width}"
        g = gen(rows * 20000 + width + 1)
        x, res = rand(g, rows, width, dtype=dtype), rand(g, rows, width, dtype=stream, shift=0.5)
        d_y, d_sum = rand(g, rows, width, dtype=dtype), rand(g, rows, width, dtype=stream)
        gain, bias = vectors(g, width)
        factor = factors(rows, width, rate)
        f = cli.dropout_layer_norm(layout(x, kind), layout(res, kind), rate, seed, SITE, gain, bias)
        want = ref.join(x, res, factor, gain, bias, 1e-5)
        within(f["sum"], want["sum"], what + " sum")
        within(f["output"], want["output"], what + " output")
        alone = cli.dropout_layer_norm(layout(x, kind), layout(res, kind), rate, seed, SITE, gain, bias, want_sum=False)
        assert alone["sum"] is None and torch.equal(alone["output"], f["output"])
        for ds in (d_sum, None):
            b = cli.dropout_layer_norm_backward(layout(f["sum"], kind), layout(d_y, kind), rate, seed, SITE,
                                                None if ds is None else layout(ds, kind), gain, bias)
            want = ref.join_backward(f["sum"], d_y, ds, factor, gain, 1e-5)
            for name in ("d_residual", "d_x", "d_gain", "d_bias"):
                within(b[name], want[name], f"{what} {name}")
        c = cli.dropout_layer_norm_backward(f["sum"], d_y, rate, seed, SITE, gain=gain, want_d_x=False)
        assert c["d_x"] is None and c["d_bias"] is None
        within(c["d_residual"], want["d_residual"], what)
        within(c["d_gain"], want["d_gain"], what)


@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_dropout_and_its_gradient(cli, dtype, kind):
    for rows, width in SHAPES:
        x = rand(gen(width), rows, width, dtype=dtype)
        for rate in (0.0, 0.3, 0.999):
            want = ref.dropout(x, factors(rows, width, rate), dtype)
            within(cli.dropout(layout(x, kind), rate, seed_of(), SITE)["output"], want, f"{rows} x {width}")
            within(cli.dropout_backward(layout(x, kind), rate, seed_of(), SITE)["d_x"], want, f"{rows} x {width}")


def test_masks_by_seed_step_site_and_rate(cli):
    """The mask is the documented one, whatever the type, and every part of its counter counts."""
    ones = torch.ones(64, 100, device="cuda")
    seen = []
    for seed, step, site in ((0, 0, 0), (1, 0, 0), (1 << 32, 0, 0), (0, 1, 0), (0, 1 << 32, 0), (0, 0, 1), (-1, -1, 7)):
        want = ref.factors(64, 100, 0.5, seed % 2 ** 64, step % 2 ** 64, site).cuda()
        for dtype in (BF16, F32):
            got = cli.dropout(ones.to(dtype), 0.5, seed_of(seed, step), site)["output"]
            assert torch.equal(got.double(), want)
        assert not any(torch.equal(want, s) for s in seen)
        seen.append(want)
    for rate in (2.0 ** -32, 2.0 ** -33, 1 - 2.0 ** -53):   # the least share that drops, one below it, the largest rate
        drop = int(rate * 2 ** 32)
        got = cli.dropout(ones, rate, seed_of(0, 0))["output"]
        assert torch.equal(got.double(), (ref.words(64, 100, 0, 0, 0).cuda() >= drop) * (2.0 ** 32 / (2 ** 32 - drop)))


def test_kept_share(cli):
    """Of 2^24 elements at rate p, sqrt(p (1 - p) 2^24) is a standard deviation: eight of them are allowed."""
    x = torch.ones(4096, 4096, dtype=F16, device="cuda")
    for rate in (0.1, 0.5, 0.9):
        y = cli.dropout(x, rate, seed_of())["output"]
        assert abs(int((y == 0).sum()) - rate * 2 ** 24) <= 8 * (rate * (1 - rate) * 2 ** 24) ** 0.5
        for share in ((y == 0).double().mean(0), (y == 0).double().mean(1)):   # and of each row and column of 4096
            assert ((share - rate).abs() <= 8 * (rate * (1 - rate) / 4096) ** 0.5).all()


def test_dropped_elements_are_zero_whatever_they_hold(cli):
    for width in (64, 63):
        factor = factors(40, width, 0.5)
        x = rand(gen(3), 40, width, dtype=BF16)
        x[factor == 0] = float("nan")
        y = cli.dropout(x, 0.5, seed_of(), SITE)["output"]
        assert torch.isfinite(y).all() and not y[factor == 0].any()
        res = rand(gen(4), 40, width, dtype=BF16)
        x[factor == 0] = float("inf")
        f = cli.dropout_layer_norm(x, res, 0.5, seed_of(), SITE)
        assert torch.isfinite(f["output"]).all() and torch.equal(f["sum"][factor == 0], res[factor == 0])


def test_rows_are_apart(cli):
    """NaN and infinity stay in their rows, and a row's results do not depend on how many others there are."""
    for width in (72, 130, 600, 2056):
        g = gen(width)
        x, d_y = rand(g, 300, width, dtype=BF16), rand(g, 300, width, dtype=BF16)
        gain, bias = vectors(g, width)
        y, d = cli.layer_norm(x, gain, bias)["output"], cli.layer_norm_backward(x, d_y, gain)["d_x"]
        for n in (1, 2, 5, 64):
            assert torch.equal(cli.layer_norm(x[:n], gain, bias)["output"], y[:n])
            assert torch.equal(cli.layer_norm_backward(x[:n], d_y[:n], gain)["d_x"], d[:n])
        bad = x.clone()
        bad[7, 3], bad[100] = float("inf"), float("nan")
        rest = torch.ones(300, dtype=torch.bool, device="cuda")
        rest[[7, 100]] = False
        y2 = cli.layer_norm(bad, gain, bias)["output"]
        d2 = cli.layer_norm_backward(bad, d_y, gain)["d_x"]
        assert torch.equal(y2[rest], y[rest]) and torch.equal(d2[rest], d[rest])
        assert y2[~rest].isnan().all() and d2[~rest].isnan().all()


@pytest.mark.parametrize("shift, scale", [(1000.0, 1.0), (-3e4, 1.0), (0.0, 1e-4), (5.0, 1e3), (0.0, 1e15)])
def test_means_far_from_zero_and_spreads(cli, shift, scale):
    """Rows of fp32 around a mean of up to 3e4 times their spread, of next to no spread, of a large one."""
    for width in (40, 771, 1024, 4096):
        g = gen(9)
        x, d_y = rand(g, 30, width, scale=scale, shift=shift), rand(g, 30, width)
        gain, bias = vectors(g, width)
        within(cli.layer_norm(x, gain, bias)["output"], ref.layer_norm(x, gain, bias, 1e-5, F32), width)
        b, want = cli.layer_norm_backward(x, d_y, gain, bias), ref.layer_norm_backward(x, d_y, gain, 1e-5, F32)
        for name in ("d_x", "d_gain", "d_bias"):
            within(b[name], want[name], f"{width} {name}")


def test_constant_rows(cli):
    """No spread: the normalised row is 0.  Its elements are alike, so every deviation is the same number D <= 70 U |x|, and
    the mean of those is D to within 71 U D; times r = 1 / sqrt(epsilon) that is under 1e-7 |x|."""
    for value in (0.0, 3.0, -0.1, 100.0):
        for width in (1, 3, 64, 1000, 8191):
            x = torch.full((5, width), value, device="cuda")
            gain, bias = vectors(gen(1), width)
            y = cli.layer_norm(x, gain, bias)["output"]
            assert ((y - bias).abs() <= 1e-7 * abs(value) * gain.abs() + 2.0 ** -23 * bias.abs()).all(), (value, width)


def test_gradient_matches_differences(cli):
    """Along random directions, the kernels' gradients against central differences of the 64-bit forward; the terms of the
    inner product are as many roundings off as the reference's bounds say, the difference itself by h^2."""
    g = gen(17)
    rows, width, rate = 20, 130, 0.3
    factor = factors(rows, width, rate)
    x, res = rand(g, rows, width), rand(g, rows, width)
    gain, bias = vectors(g, width)
    d_y, d_sum = rand(g, rows, width), rand(g, rows, width)
    f = cli.dropout_layer_norm(x, res, rate, seed_of(), SITE, gain, bias)
    got = cli.dropout_layer_norm_backward(f["sum"], d_y, rate, seed_of(), SITE, d_sum, gain, bias)
    bounds = ref.join_backward(f["sum"], d_y, d_sum, factor, gain, 1e-5)

    def loss(*args):
        r = ref.join(*args[:2], factor, *args[2:], 1e-5)
        return (r["output"][0] * d_y.double()).sum() + (r["sum"][0] * d_sum.double()).sum()
    args = [t.double() for t in (x, res, gain, bias)]
    for i, name in enumerate(("d_x", "d_residual", "d_gain", "d_bias")):
        direction, h = rand(g, *args[i].shape).double(), 1e-5
        plus, minus = [[v + s * h * direction if j == i else v for j, v in enumerate(args)] for s in (1, -1)]
        want = float(loss(*plus) - loss(*minus)) / (2 * h)
        # the sum that the kernel read is rounded: 2 U relative, through second derivatives below 10 here
        bound = float((bounds[name][1] * direction.abs()).sum()) + 20 * ref.U * float(direction.abs().sum()) + 1e-6 * abs(want) + 1e-6
        assert abs(float((got[name].double() * direction).sum()) - want) <= bound, name


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, width", [(20011, 64), (9000, 200), (5000, 1024), (3001, 517), (1500, 4096), (4000, 1100), (2500, 3200),
                                         (1200, 8192), (700, 12000)])
def test_more_rows_than_the_grid_takes_at_once(cli, rows, width, dtype):
    g = gen(rows)
    x, d_y = rand(g, rows, width, dtype=dtype, shift=0.3), rand(g, rows, width, dtype=dtype)
    gain, bias = vectors(g, width)
    within(cli.layer_norm(x, gain, bias)["output"], ref.layer_norm(x, gain, bias, 1e-5, dtype), "output")
    b, want = cli.layer_norm_backward(x, d_y, gain, bias), ref.layer_norm_backward(x, d_y, gain, 1e-5, dtype)
    for name in ("d_x", "d_gain", "d_bias"):
        within(b[name], want[name], name)
    for n in (3, 700):   # whatever comes after them
        assert torch.equal(cli.layer_norm(x[:n], gain, bias)["output"], cli.layer_norm(x, gain, bias)["output"][:n])
        assert torch.equal(cli.layer_norm_backward(x[:n], d_y[:n], gain, bias)["d_x"], b["d_x"][:n])
    again = cli.layer_norm_backward(x, d_y, gain, bias)
    assert all(torch.equal(b[n], again[n]) for n in b)
    factor = cli.dropout(torch.ones(rows, width, device="cuda"), 0.2, seed_of(), SITE)["output"].double()
    some = [0, 1, rows // 2, rows - 2, rows - 1]   # of the mask's rows, each drawn alone by the reference
    low = 2 ** 32 - 1
    for r in some:
        c = torch.tensor([ref.philox([k + 65536 * SITE, r, STEP & low, STEP >> 32], [SEED & low, (SEED >> 32) & low])
                          for k in range((width + 3) // 4)]).flatten()[:width]
        assert torch.equal(factor[r] != 0, (c >= int(0.2 * 2 ** 32)).cuda())
    f = cli.dropout_layer_norm(x, d_y, 0.2, seed_of(), SITE, gain, bias)
    kept = 2.0 ** 32 / (2 ** 32 - int(0.2 * 2 ** 32))
    want = ref.join(x, d_y, (factor != 0) * kept, gain, bias, 1e-5)
    within(f["sum"], want["sum"], "sum")
    within(f["output"], want["output"], "joined output")
    b = cli.dropout_layer_norm_backward(f["sum"], d_y, 0.2, seed_of(), SITE, x, gain, bias)
    want = ref.join_backward(f["sum"], d_y, x, (factor != 0) * kept, gain, 1e-5)
    for name in ("d_residual", "d_x", "d_gain", "d_bias"):
        within(b[name], want[name], "joined " + name)
    for n in (3, 700):
        few = cli.dropout_layer_norm(x[:n], d_y[:n], 0.2, seed_of(), SITE, gain, bias)
        back = cli.dropout_layer_norm_backward(f["sum"][:n], d_y[:n], 0.2, seed_of(), SITE, x[:n], gain, bias)
        assert torch.equal(few["output"], f["output"][:n]) and torch.equal(few["sum"], f["sum"][:n])
        assert torch.equal(back["d_residual"], b["d_residual"][:n]) and torch.equal(back["d_x"], b["d_x"][:n])


def test_in_place(cli):
    for width in (96, 97, 2048):
        g = gen(width)
        x, res, d_y, d_s = (rand(g, 50, width, dtype=BF16) for _ in range(4))
        gain, bias = vectors(g, width)
        y = cli.layer_norm(x, gain, bias)["output"]
        t = x.clone()
        assert cli.layer_norm(t, gain, bias, out={"output": t})["output"] is t and torch.equal(t, y)
        b = cli.layer_norm_backward(x, d_y, gain, bias)
        for which in (0, 1):
            a = [x.clone(), d_y.clone()]
            assert torch.equal(cli.layer_norm_backward(*a, gain, bias, out={"d_x": a[which]})["d_x"], b["d_x"])
        t = x.clone()
        cli.dropout(t, 0.3, seed_of(), out={"output": t})
        assert torch.equal(t, cli.dropout(x, 0.3, seed_of())["output"])
        f = cli.dropout_layer_norm(x, res, 0.3, seed_of(), 0, gain, bias)
        t, u = x.clone(), res.clone()
        cli.dropout_layer_norm(t, u, 0.3, seed_of(), 0, gain, bias, out={"sum": u, "output": t})
        assert torch.equal(u, f["sum"]) and torch.equal(t, f["output"])
        b = cli.dropout_layer_norm_backward(f["sum"], d_y, 0.3, seed_of(), 0, d_s, gain, bias)
        t, u = d_y.clone(), d_s.clone()
        cli.dropout_layer_norm_backward(f["sum"], t, 0.3, seed_of(), 0, u, gain, bias, out={"d_residual": u, "d_x": t})
        assert torch.equal(u, b["d_residual"]) and torch.equal(t, b["d_x"])


def test_rows_behind_and_between_are_left_alone(cli):
    for width, kind in ((64, "padded"), (61, "odd"), (1028, "fours")):
        g = gen(width)
        x, d_y = rand(g, 37, width, dtype=F16), rand(g, 37, width, dtype=F16)
        off, gap = {"padded": (8, 8), "fours": (4, 12), "odd": (1, 3)}[kind]
        bufs = [torch.full((39, off + width + gap), 7.0, dtype=F16, device="cuda") for _ in range(4)]
        views = [t[1:38, off:off + width] for t in bufs]
        cli.layer_norm(x, out={"output": views[0]})
        cli.layer_norm_backward(x, d_y, out={"d_x": views[1]})
        cli.dropout(x, 0.5, seed_of(), out={"output": views[2]})
        cli.dropout_layer_norm(x, d_y, 0.5, seed_of(), out={"sum": views[3]})
        for t, v in zip(bufs, views):
            v.fill_(7.0)
            assert (t == 7.0).all()


def test_broadcast_rows_and_no_rows(cli):
    g = gen(2)
    x, one = rand(g, 40, 64, dtype=BF16), rand(g, 1, 64, dtype=BF16)
    wide = one.expand(40, 64)
    f, want = cli.dropout_layer_norm(x, wide, 0.0, None), cli.dropout_layer_norm(x, wide.contiguous(), 0.0, None)
    assert torch.equal(f["sum"], want["sum"]) and torch.equal(f["output"], want["output"])
    with pytest.raises(cli.ShapeMismatchError):
        cli.layer_norm(x, out={"output": wide})
    none, gain = x[:0], torch.ones(64, device="cuda")
    assert cli.layer_norm(none)["output"].shape == (0, 64) and cli.dropout(none, 0.5, seed_of())["output"].shape == (0, 64)
    b = cli.layer_norm_backward(none, none, gain, gain)
    assert not b["d_gain"].any() and not b["d_bias"].any() and b["d_x"].shape == (0, 64)
    b = cli.dropout_layer_norm_backward(none, none, 0.1, seed_of(), gain=gain)
    assert not b["d_gain"].any() and b["d_bias"] is None


def test_outputs_and_workspace_are_the_callers(cli):
    g = gen(31)
    x, d_y, d_s = rand(g, 777, 200, dtype=BF16), rand(g, 777, 200, dtype=BF16), rand(g, 777, 200, dtype=BF16)
    gain, bias = vectors(g, 200)
    need = cli.layer_norm_backward_workspace_bytes(777, 200)
    for call in (lambda **o: cli.layer_norm_backward(x, d_y, gain, bias, **o),
                 lambda **o: cli.dropout_layer_norm_backward(x, d_y, 0.1, seed_of(), 0, d_s, gain, bias, **o)):
        want = call()
        out = {n: torch.full_like(t, 9.0) for n, t in want.items()}
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN in every word
        r = call(out=out, workspace=ws[:need])
        assert (ws[need:] == 0xFF).all()
        for n in want:
            assert r[n] is out[n] and torch.equal(out[n], want[n]), n
        with pytest.raises(cli.InvalidArgumentError):
            call(workspace=ws[:need - 1])


def test_calls_on_other_streams(cli):
    g = gen(5)
    x, d_y = rand(g, 3000, 512, dtype=BF16), rand(g, 3000, 512, dtype=BF16)
    gain, bias = vectors(g, 512)
    seed = seed_of()

    def calls(**kw):
        f = cli.dropout_layer_norm(x, d_y, 0.1, seed, 1, gain, bias, **kw)
        b = cli.dropout_layer_norm_backward(f["sum"], d_y, 0.1, seed, 1, f["sum"], gain, bias, **kw)
        n = cli.layer_norm_backward(f["output"], b["d_x"], gain, bias, **kw)
        return [*f.values(), *b.values(), *n.values(), cli.dropout(x, 0.2, seed, **kw)["output"]]
    want = calls()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [calls(stream=s) for s in streams]   # two sets of calls under way at once
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_a_captured_step_draws_the_step_that_is_there(cli):
    g = gen(6)
    x, res, d_y = (rand(g, 300, 256, dtype=BF16) for _ in range(3))
    gain, bias = vectors(g, 256)
    seed = seed_of(11, 0)

    def step():
        f = cli.dropout_layer_norm(x, res, 0.25, seed, 3, gain, bias)
        b = cli.dropout_layer_norm_backward(f["sum"], d_y, 0.25, seed, 3, None, gain, bias)
        d = cli.dropout(x, 0.25, seed, 4)["output"]
        return [*f.values(), *b.values(), d]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
        seed[1] += 1
    seen = []
    for k in range(3):
        x.copy_(rand(gen(60 + k), 300, 256, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert seed.tolist() == [11, k + 1]
        got = [t.clone() for t in out]
        keep = seed.clone()
        seed.copy_(seed_of(11, k))
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        seed.copy_(keep)
        seen.append(got[-1] != 0)
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_rows_past_32_bits(cli):
    """Rows whose element offset passes 2^32 and whose byte offset passes 2^33."""
    rows, width, n = 2200000, 2048, 40   # 9 GB a tensor
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    g = gen(8)
    x[-n:] = rand(g, n, width, dtype=BF16)
    gain, bias = vectors(g, width)
    y = cli.layer_norm(x, gain, bias)["output"]
    within(y[-n:], ref.layer_norm(x[-n:], gain, bias, 1e-5, BF16), "output")
    assert torch.equal(y[5], bias.bfloat16())
    del y
    b = cli.layer_norm_backward(x, x, gain, bias)
    want = ref.layer_norm_backward(x[-n:], x[-n:], gain, 1e-5, BF16)
    within(b["d_x"][-n:], want["d_x"], "d_x")
    within(b["d_gain"], want["d_gain"], "d_gain")   # the other rows give nothing
    within(b["d_bias"], want["d_bias"], "d_bias")
    del b
    d = cli.dropout(x, 0.5, seed_of(), SITE, out={"output": x})["output"]   # in place
    low = 2 ** 32 - 1
    last = torch.tensor([ref.philox([k + 65536 * SITE, rows - 1, STEP & low, STEP >> 32], [SEED & low, (SEED >> 32) & low])
                         for k in range(width // 4)]).flatten().cuda()
    assert not d[-1][last < 2 ** 31].any() and d[-1][last >= 2 ** 31].all()


def test_refusals_of_the_binding(cli):
    x = torch.zeros(4, 8, dtype=BF16, device="cuda")
    seed, host = seed_of(), torch.zeros(4, 8, dtype=BF16)
    for call, error in (
            (lambda: cli.layer_norm(host), cli.InvalidArgumentError),
            (lambda: cli.layer_norm(x[0]), cli.ShapeMismatchError),
            (lambda: cli.layer_norm(x.t()), cli.ShapeMismatchError),
            (lambda: cli.layer_norm(x.double()), cli.UnsupportedError),
            (lambda: cli.layer_norm(x, dtype=F32), cli.UnsupportedError),
            (lambda: cli.layer_norm(x, dtype=F16), cli.UnsupportedError),
            (lambda: cli.layer_norm(x, gain=torch.ones(7, device="cuda")), cli.ShapeMismatchError),
            (lambda: cli.layer_norm(x, gain=torch.ones(8, dtype=BF16, device="cuda")), cli.InvalidArgumentError),
            (lambda: cli.layer_norm(x, epsilon=0.0), cli.InvalidArgumentError),
            (lambda: cli.layer_norm_backward(x, x.float()), cli.UnsupportedError),
            (lambda: cli.layer_norm_backward(x, x[:2]), cli.ShapeMismatchError),
            (lambda: cli.dropout(x, 1.0, seed), cli.InvalidArgumentError),
            (lambda: cli.dropout(x, 0.1, None), cli.InvalidArgumentError),
            (lambda: cli.dropout(x, 0.1, seed.cpu()), cli.InvalidArgumentError),
            (lambda: cli.dropout(x, 0.1, seed.int()), cli.InvalidArgumentError),
            (lambda: cli.dropout(x, 0.1, seed[:1]), cli.ShapeMismatchError),
            (lambda: cli.dropout(x, 0.1, seed, site=-1), cli.InvalidArgumentError),
            (lambda: cli.dropout(x, 0.1, seed, site=65536), cli.InvalidArgumentError),
            (lambda: cli.dropout_layer_norm(x, x.half(), 0.1, seed), cli.UnsupportedError),
            (lambda: cli.dropout_layer_norm(x.float(), x, 0.1, seed), cli.UnsupportedError),
            (lambda: cli.dropout_layer_norm_backward(x, x, 0.1, seed, d_sum=x.float()), cli.InvalidArgumentError),
            (lambda: cli.layer_norm(torch.zeros(2, 16392, device="cuda")), cli.UnsupportedError)):
        with pytest.raises(error):
            call()


def test_a_training_block(cli):
    """A block as it is trained: norm, heads, attention over a tape, dropout into the stream, the next norm, and the whole
    way back, against autograd in 64 bits over the same roundings' places.  The tolerance counts the 16-bit results between
    input and gradient, seven in series at half a step (2^-8) each, in the norm over all elements."""
    g = gen(40)
    heads, dim, lengths, rate = 4, 64, [70, 1, 129], 0.1
    rows, width = sum(lengths), heads * dim
    offsets = torch.tensor([0] + lengths, device="cuda").cumsum(0)
    x = rand(g, rows, width, dtype=BF16)
    gain1, bias1 = vectors(g, width)
    gain2, bias2 = vectors(g, width)
    d_y = rand(g, rows, width, dtype=BF16)
    seed = seed_of()
    # forward
    h = cli.layer_norm(x, gain1, bias1)["output"]
    split = h.view(rows, heads, dim)
    kw = dict(max_query_rows=max(lengths), max_key_rows=max(lengths))
    a = cli.cross_attention(split, offsets, split, split, offsets, **kw)
    j = cli.dropout_layer_norm(a["output"].view(rows, width), x, rate, seed, 5, gain2, bias2)
    # and back
    e = cli.dropout_layer_norm_backward(j["sum"], d_y, rate, seed, 5, None, gain2, bias2)
    b = cli.cross_attention_backward(split, offsets, split, split, offsets, a["output"], a["lse"],
                                     e["d_x"].view(rows, heads, dim), **kw)
    d_h = (b["d_q"].float() + b["d_k"].float() + b["d_v"].float()).bfloat16().view(rows, width)
    n = cli.layer_norm_backward(x, d_h, gain1, bias1)
    d_x = n["d_x"].double() + e["d_residual"].double()
    # in 64 bits
    leaves = [t.double().requires_grad_() for t in (x, gain1, bias1, gain2, bias2)]
    X, G1, B1, G2, B2 = leaves

    def norm(t, w, c):
        u = t - t.mean(1, keepdim=True)
        return u / torch.sqrt((u * u).mean(1, keepdim=True) + 1e-5) * w + c
    H = norm(X, G1, B1).view(rows, heads, dim)
    parts, at = [], 0
    for k in lengths:
        t = H[at:at + k]
        p = torch.einsum("qhd,khd->hqk", t, t).mul(dim ** -0.5).softmax(-1)
        parts.append(torch.einsum("hqk,khd->qhd", p, t))
        at += k
    branch = torch.cat(parts).view(rows, width)
    factor = ref.factors(rows, width, rate, SEED % 2 ** 64, STEP, 5).cuda()
    Y = norm(X + branch * factor, G2, B2)
    Y.backward(d_y.double())
    tolerance = 7 * 2.0 ** -8
    for name, got, want in (("output", j["output"], Y), ("d_x", d_x, X.grad), ("d_gain1", n["d_gain"], G1.grad),
                            ("d_bias1", n["d_bias"], B1.grad), ("d_gain2", e["d_gain"], G2.grad), ("d_bias2", e["d_bias"], B2.grad)):
        assert (got.double() - want).norm() <= tolerance * want.norm(), name
