"""The token-state operators on the GPU where a call's surroundings matter: other streams, lent buffers, bad offsets and
positions, values that only some rows hold."""

import pytest
import torch

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
