"""Tokens from logits on a GB300 against whole numbers in Python: the tokens have to be equal."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from hashed_gram_embedding_engram_gb300 import sample_tokens  # noqa: E402
from oracle import decoding_oracle as O  # noqa: E402

SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7), dict(top_k=1), dict(top_k=5), dict(top_k=40),
            dict(top_p=0.9), dict(top_p=0.3), dict(top_p=0.0), dict(min_p=0.1), dict(min_p=1.0),
            dict(temperature=1.3, top_k=50, top_p=0.8), dict(temperature=0.5, top_k=7, top_p=0.95, min_p=0.02),
            dict(temperature=5.0, top_p=0.999), dict(temperature=0.01, top_p=0.9), dict(temperature=100.0, top_k=1000)]


def check(logits, u, **settings):
    """Every row, its settings a number or its own of a tensor."""
    got = sample_tokens(logits, u, **settings).cpu().tolist()
    l, uu = logits.float().cpu().numpy(), u.cpu().numpy()
    rows = {k: v.cpu().numpy() if isinstance(v, torch.Tensor) else [v] * len(l) for k, v in settings.items()}
    want = [O.sample(l[r], uu[r], **{k: v[r] for k, v in rows.items()}) for r in range(len(l))]
    assert got == want
    return got


def normal(R, V, seed=0, scale=3.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed + V)
    return (torch.randn(R, V, generator=g) * scale).to(dtype).cuda(), torch.rand(R, generator=g).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", SETTINGS, ids=[str(i) for i in range(len(SETTINGS))])
def test_sampling_matches_whole_numbers(settings, dtype):
    for R, V in ((1, 1), (3, 2), (4, 31), (5, 128), (6, 1000), (7, 4099), (2, 20001)):
        check(*normal(R, V, dtype=dtype), **settings)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [129280, 65537, 32000])
def test_large_vocabularies_and_settings_of_each_row(V, dtype):
    R = 6
    logits, u = normal(R, V, 1, dtype=dtype)
    g = torch.Generator().manual_seed(V)
    check(logits, u, temperature=torch.tensor([0.0, 0.3, 1.0, 2.0, 0.8, 1.0]).cuda(),
          top_k=torch.tensor([0, 50, 0, 3000, 1, 0], dtype=torch.int32).cuda(),
          top_p=torch.tensor([1.0, 0.9, 0.5, 0.99, 1.0, 1.0]).cuda(), min_p=(torch.rand(R, generator=g) * 0.01).cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", [dict(temperature=3.0, top_p=0.5), dict(temperature=3.0, top_p=0.97),
                                      dict(temperature=30.0, top_p=0.8), dict(temperature=2.0, top_p=1 - 2.0 ** -20),
                                      dict(top_k=1100), dict(top_k=5000, top_p=0.7), dict(temperature=0.2, top_p=0.9999)],
                         ids=[str(i) for i in range(7)])
def test_more_tokens_than_a_blocks_lists_hold(settings, dtype):
    """Lists that just fit and that do not: flat distributions, large top_k, borders in the far tail."""
    check(*normal(3, 50001, 12, dtype=dtype), **settings)
    check(*normal(2, 129280, 13, dtype=dtype), min_p=1e-4, **settings)


@pytest.mark.parametrize("R", [1, 19, 20, 37, 38, 39, 75, 77, 150, 155, 400])
def test_batches_around_the_sizes_at_which_rows_get_fewer_blocks(R):
    logits, u = normal(R, 9000, R)
    check(logits, u, top_k=30, top_p=0.9)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(dtype):
    """Few distinct values: borders inside ties, over several warps and blocks."""
    g = torch.Generator().manual_seed(4)
    for V in (40, 5000, 70001):
        logits = torch.randint(0, 4, (6, V), generator=g).to(dtype).cuda()
        u = torch.rand(6, generator=g).cuda()
        for settings in (dict(temperature=0.0), dict(top_k=V // 3), dict(top_k=V // 2 + 1, top_p=0.7), dict(top_p=0.35),
                         dict(min_p=0.2), dict(top_k=3)):
            check(logits, u, **settings)
        same = torch.full((2, V), 1.5, dtype=dtype).cuda()
        for settings in (dict(), dict(top_k=V - 1), dict(top_k=7), dict(top_p=0.5), dict(temperature=0.0)):
            check(same, u[:2], **settings)


def test_signed_zeros_are_equal():
    logits = torch.zeros(4, 300)
    logits[:, 1::2] = -0.0
    u = torch.tensor([0.0, 0.3, 0.6, 0.999]).cuda()
    for x in (logits.cuda(), logits.bfloat16().cuda(), -logits.cuda()):
        check(x, u, top_k=9)
        check(x, u, temperature=0.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinities_and_nan(dtype):
    inf, nan = math.inf, math.nan
    g = torch.Generator().manual_seed(5)
    logits = (torch.randn(9, 700, generator=g) * 3).to(dtype)
    logits[0] = -inf
    logits[1] = nan
    logits[2, ::2] = nan
    logits[3, 5:] = -inf
    logits[4, 100] = inf
    logits[5, 100:110] = inf
    logits[5, 50] = nan
    logits[6] = -inf
    logits[6, 321] = -3e38
    logits[7] = 3e38
    logits[7, 9] = -3e38
    logits[8, :699] = nan
    u = torch.rand(9, generator=g).cuda()
    for settings in SETTINGS:
        got = check(logits.cuda(), u, **settings)
        assert got[0] == got[1] == -1 and got[4] == 100 and 100 <= got[5] < 110 and got[6] == 321 and got[8] == 699


def test_settings_at_their_ends():
    logits, u = normal(5, 900, 6)
    f = lambda *x: torch.tensor(x, dtype=torch.float32).cuda()  # noqa: E731
    inf, nan = math.inf, math.nan
    check(logits, u, temperature=f(1e-45, 1e-38, 1e38, inf, -1.0))
    greedy = sample_tokens(logits, u, temperature=nan)
    assert torch.equal(greedy.long(), logits.argmax(1))
    check(logits, u, top_k=torch.tensor([-5, 2 ** 31 - 1, 900, 899, 901], dtype=torch.int32).cuda())
    check(logits, u, top_k=10 ** 30)
    check(logits, u, top_p=f(-1.0, 1 - 2.0 ** -24, 1.5, inf, 2.0 ** -24))
    check(logits, u, min_p=f(-1.0, 2.0, 1e-30, inf, 0.0))
    assert torch.equal(sample_tokens(logits, u, top_p=nan, min_p=nan), sample_tokens(logits, u))


def test_random_numbers_at_their_ends():
    logits, _ = normal(1, 500, 7)
    logits = logits.expand(8, 500).contiguous()
    u = torch.tensor([0.0, 1.0, 1 - 2.0 ** -24, 2.0 ** -25, -3.0, 7.0, math.nan, math.inf]).cuda()
    got = sample_tokens(logits, u).cpu().tolist()
    want = [O.sample(logits[0].cpu().numpy(), x) for x in (0.0, 1.0, 1.0, 0.0, 0.0, 1.0, 0.0, 1.0)]
    assert got == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_apart_and_at_any_element(dtype):
    for V, offset, stride in ((777, 1, 777), (1000, 3, 1029), (8, 5, 9), (5, 2, 64), (33000, 7, 33001)):
        flat, _ = normal(1, offset + 4 * stride, 8, dtype=dtype)
        logits = flat.view(-1)[offset:].as_strided((4, V), (stride, 1))
        check(logits, torch.rand(4, generator=torch.Generator().manual_seed(V)).cuda(), top_k=20, top_p=0.9)
    check(flat.view(-1)[:5000].expand(1, 5000), torch.rand(1).cuda())


@pytest.mark.parametrize("V,dtype", [(300001, torch.float32), (360000, torch.float32), (300003, torch.bfloat16),
                                     (600001, torch.bfloat16), (720001, torch.bfloat16)])
def test_rows_that_just_fit_shared_memory(V, dtype):
    """Pieces of more than 64 KB (one block an SM), of more than 65536 tokens (whose places take 17 bits), and the
    longest that are kept."""
    logits, u = normal(2, V, 14, dtype=dtype)
    for settings in (dict(top_p=0.9), dict(temperature=2.0, top_p=0.7), dict(top_k=60, top_p=0.8), dict(min_p=0.01)):
        check(logits, u, **settings)


def test_rows_too_long_for_shared_memory():
    """Longer than a cluster's shared memory holds: read again from device memory."""
    for V, dtype in ((600001, torch.float32), (1100003, torch.bfloat16)):
        logits, u = normal(2, V, 9, dtype=dtype)
        for settings in (dict(temperature=0.8), dict(top_k=100, top_p=0.9), dict(temperature=0.0)):
            check(logits, u, **settings)


def test_no_rows_and_given_outputs():
    logits, u = normal(3, 50)
    assert sample_tokens(logits[:0], u[:0]).shape == (0,)
    tokens = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    assert sample_tokens(logits, u, tokens=tokens) is tokens and tokens.cpu().tolist() == check(logits, u)


def test_the_draw_follows_the_weights():
    """Over a grid of random numbers every token comes up as often as its weight says."""
    V, n = 9, 4096
    logits, _ = normal(1, V, 10, scale=1.0)
    u = (torch.arange(n, dtype=torch.float32) + 0.5).cuda() / n
    got = torch.bincount(sample_tokens(logits.expand(n, V).contiguous(), u).long(), minlength=V).double().cpu() / n
    # each of the V borders is off by at most one step of the grid, and the weights by 2^-22
    assert (got - torch.softmax(logits[0].double().cpu(), 0)).abs().max() <= 2.0 / n + 2.0 ** -22


def test_weights_are_exponentials():
    """2^38 P(f) 2^-n against 2^(38 - a): 1.0e-7 from the polynomial with its roundings, the roundings of
    m - l, of c and of the product (three halves of 2^-23 of a at most, a ln 2 < 28 of them), and the
    fraction that is cut off."""
    l = np.linspace(-30, 5, 5001).astype(np.float32)
    for t in (0.5, 1.0, 2.7):
        a = (5.0 - l.astype(np.float64)) * math.log2(math.e) / t
        want = 2.0 ** (38 - a)
        near = np.abs(np.array([float(x) for x in O.weights(l, t)]) - want)
        assert (near <= want * (1.01e-7 + 3 * 2.0 ** -24 * a * math.log(2)) + 1).all()


def test_two_streams_give_the_same_tokens():
    inputs = [normal(40, 30000, i, dtype=t) for i, t in enumerate((torch.float32, torch.bfloat16))]
    kw = dict(temperature=1.1, top_p=0.9)
    want = [sample_tokens(*x, **kw) for x in inputs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in inputs], []
    for _ in range(20):
        for i, (x, s) in enumerate(zip(inputs, streams)):
            with torch.cuda.stream(s):
                got.append((i, sample_tokens(*x, **kw)))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i, t in got)


def test_graph_replay():
    logits, u = normal(4, 3000, 11)
    k = torch.tensor([0, 1, 20, 300], dtype=torch.int32, device="cuda")
    tokens = torch.empty(4, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sample_tokens(logits, u, top_k=k, tokens=tokens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sample_tokens(logits, u, top_k=k, tokens=tokens)
    torch.cuda.current_stream().wait_stream(s)
    for seed in (1, 2):
        logits.copy_(normal(4, 3000, seed)[0])
        u.copy_(torch.rand(4, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        assert tokens.cpu().tolist() == check(logits, u, top_k=k)
