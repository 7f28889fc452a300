"""pa_verify_drafts against the definition in 64 bits: chains and trees, with and
without draft probabilities, small and large vocabularies, padded and ragged batches,
special values, and what it is for: the distribution of the kept tokens."""
import numpy as np
import pytest
import torch

import speclib
from paged_kv_cache_251_gb300 import pa

pytestmark = pytest.mark.gpu


def outputs(n, t):
    return (torch.full((n,), -7, dtype=torch.int32, device="cuda"),
            torch.full((n, t), -7, dtype=torch.int32, device="cuda"),
            torch.full((n, t + 1), -7, dtype=torch.int32, device="cuda"))


def probs(gen, shape, near=None, noise=0.7):
    x = 2.5 * torch.randn(shape, generator=gen)
    if near is not None:
        x = near + noise * torch.randn(shape, generator=gen)
    return x, x.softmax(-1)


def problem(seed, n, t, v, tree, with_q, dtype):
    gen = torch.Generator().manual_seed(seed)
    logits, target = probs(gen, (n, t + 1, v))
    draft = probs(gen, (n, t, v), near=logits[:, :t])[1] if with_q else None
    parents = None
    at = torch.arange(t).expand(n, t)
    if tree:
        parents = (torch.arange(t) - torch.randint(1, 4, (n, t), generator=gen)).clamp_min(-1)
        at = parents + 1
    source = draft if with_q else target[:, :t]
    tokens = torch.stack([torch.stack([torch.multinomial(source[s, at[s, i]], 1, generator=gen)[0]
                                       for i in range(t)]) for s in range(n)])
    lens = torch.randint(0, t + 1, (n,), generator=gen)
    u = torch.rand((n, t + 1), generator=gen)
    return dict(target=target.to(dtype), draft=None if draft is None else draft.to(dtype), tokens=tokens.int(),
                uniforms=u, lens=lens.int(), parents=None if parents is None else parents.int())


def run(pr, stream=None, err=None):
    n, t = pr["tokens"].shape
    out = outputs(n, t)
    dev = {k: None if x is None else x.cuda() for k, x in pr.items()}
    pa.pa_verify_drafts(*out, dev["target"], dev["tokens"], dev["uniforms"], draft_probs=dev["draft"],
                        draft_lens=dev["lens"], parents=dev["parents"], err_word=err, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in out]


def expected(pr):
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    g = lambda x: None if x is None else x.numpy()  # noqa: E731
    return speclib.verify(f(pr["target"]), f(pr["draft"]), g(pr["tokens"]), g(pr["uniforms"]), g(pr["lens"]),
                          g(pr["parents"]))


def check(pr):
    for got, want in zip(run(pr), expected(pr)):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("n,t,v", [(1, 1, 1), (3, 1, 2), (2, 4, 37), (5, 7, 1000), (40, 3, 257), (7, 16, 4099),
                                   (2, 30, 8192), (1, 5, 50257), (3, 2, 128000)])
def test_definition(n, t, v, tree, with_q, dtype):
    check(problem(n * 1000 + t, n, t, v, tree, with_q, dtype))


def test_many_sequences_and_the_longest_tree():
    check(problem(1, 700, 4, 640, False, True, torch.float32))
    check(problem(2, 2, 256, 300, True, True, torch.float32))
    check(problem(3, 2, 256, 301, True, False, torch.bfloat16))


@pytest.mark.parametrize("with_q", [True, False])
def test_siblings_and_repeated_tokens(with_q):
    """Many children of one node, the same token among them again."""
    pr = problem(4, 12, 24, 50, True, with_q, torch.float32)
    pr["parents"] = torch.full((12, 24), -1, dtype=torch.int32)
    pr["lens"] = torch.full((12,), 24, dtype=torch.int32)
    pr["tokens"][:, 1::2] = pr["tokens"][:, 0::2]
    pr["uniforms"][:, :24] = 0.97 + 0.03 * pr["uniforms"][:, :24]
    pr["uniforms"].clamp_(max=1 - 2.0 ** -24)
    check(pr)


@pytest.mark.parametrize("v,dtype", [(8200, torch.float32), (17001, torch.bfloat16), (40000, torch.float16),
                                     (40003, torch.float32)])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("same", [False, True])
def test_rejections_over_long_rows(v, dtype, with_q, same):
    """Many sums of a row that several CTAs share; same: where p and q are alike nothing is left of p."""
    if same and not with_q:
        pytest.skip("without q nothing is alike")
    n, t = 3, 9
    pr = problem(40, n, t, v, True, with_q, dtype)
    if same:
        pr["draft"] = pr["target"][:, :t].clone()
        pr["uniforms"][:, :t] = 1.0  # (every draft rejected)
    else:
        pr["uniforms"][:, :t].clamp_(min=0.9, max=1 - 2.0 ** -24)
    pr["parents"] = torch.tensor([-1, -1, -1, -1, 0, 0, 1, 2, 2], dtype=torch.int32).expand(n, t).contiguous()
    pr["lens"] = torch.full((n,), t, dtype=torch.int32)
    check(pr)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_distributions_keep_everything(dtype):
    pr = problem(5, 6, 5, 999, False, True, dtype)
    pr["draft"] = pr["target"][:, :5].clone()
    pr["lens"] = None
    got = run(pr)
    assert (got[0] == 5).all()
    check(pr)


def test_certain_target():
    """One-hot targets (greedy decoding): drafted tokens are kept while they agree."""
    n, t, v = 4, 6, 1003
    hot = torch.randint(0, v, (n, t + 1), generator=torch.Generator().manual_seed(6))
    target = torch.zeros((n, t + 1, v)).scatter_(2, hot[:, :, None], 1.0)
    tokens = hot[:, :t].clone().int()
    for s in range(n):
        if s < t:
            tokens[s, s] = (tokens[s, s] + 1) % v
    pr = dict(target=target, draft=None, tokens=tokens, uniforms=torch.full((n, t + 1), 0.5), lens=None, parents=None)
    got = run(pr)
    assert got[0].tolist() == [0, 1, 2, 3]
    assert [int(got[2][s, s]) for s in range(n)] == [int(hot[s, s]) for s in range(n)]
    check(pr)


@pytest.mark.parametrize("v", [64, 1001])
@pytest.mark.parametrize("with_q", [True, False])
def test_random_numbers_at_the_ends(v, with_q):
    pr = problem(7, 6, 3, v, False, with_q, torch.float32)
    pr["target"][:, :, v - 5:] = 0  # no weight at the end of the vocabulary
    for u in (0.0, 1 - 2.0 ** -24):
        pr["uniforms"][:] = u
        check(pr)
    pr["uniforms"][:] = 1.0  # beyond [0, 1): the last token with any weight
    got = run(pr)
    assert ((got[2] >= -1) & (got[2] < v)).all()
    rows = np.arange(6)
    assert (got[2][rows, got[0]] >= 0).all()


def test_values_that_are_no_probabilities():
    """NaN counts as no weight; infinities and negative numbers give some token, and nothing else breaks."""
    pr = problem(8, 5, 3, 777, False, True, torch.float32)
    pr["target"][:, :, 3] = float("nan")
    pr["draft"][:, :, 9] = float("nan")
    pr["tokens"][0, 0] = 3
    pr["tokens"][1, 0] = 9
    check(pr)
    for bad in (float("inf"), -1.0, 3e38):
        pr["target"][:, :, 5] = bad
        pr["draft"][:, :, 700] = -bad
        got = run(pr)
        assert ((got[2] >= -1) & (got[2] < 777)).all() and ((got[0] >= 0) & (got[0] <= 3)).all()


def test_rows_without_any_weight():
    pr = problem(9, 3, 2, 515, False, True, torch.float32)
    pr["target"][:] = 0
    got = run(pr)
    assert (got[0] == 0).all() and (got[2] == -1).all() and (got[1] == -1).all()
    pr["target"][1, 0, 400] = 1e-30  # far below a rounding of the sum
    check(pr)
    pr["draft"] = None
    check(pr)


def test_bad_contents_are_left_out_and_flagged():
    pr = problem(10, 4, 6, 300, True, True, torch.float32)
    pr["lens"] = torch.tensor([6, 9, -2, 6], dtype=torch.int32)
    pr["tokens"][0, 0] = 300
    pr["tokens"][0, 1] = -1
    pr["parents"][3, 2] = 2
    pr["parents"][3, 3] = 99
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(pr, err=err)
    for a, b in zip(got, expected(pr)):
        np.testing.assert_array_equal(a, b)
    assert err.item() == pa.DEVERR_BAD_INDEX | pa.DEVERR_BAD_LEN


@pytest.mark.parametrize("pad", [3, 8])
def test_rows_of_a_wider_array(pad):
    pr = problem(11, 3, 4, 504, False, True, torch.bfloat16)
    want = expected(pr)
    wide_t = torch.full((3, 5, 504 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    wide_q = torch.full((3, 4, 504 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    wide_t[:, :, :504] = pr["target"].cuda()
    wide_q[:, :, :504] = pr["draft"].cuda()
    out = outputs(3, 4)
    pa.pa_verify_drafts(*out, wide_t[:, :, :504], pr["tokens"].cuda(), pr["uniforms"].cuda(),
                        draft_probs=wide_q[:, :, :504], draft_lens=pr["lens"].cuda())
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_large_offsets():
    """Rows beyond 2^31 elements from the first."""
    n, t, v = 9, 15, 1 << 24
    target = torch.zeros((n, t + 1, v), dtype=torch.float16, device="cuda")
    want = torch.randint(0, v, (n, t + 1), generator=torch.Generator().manual_seed(12))
    target.scatter_(2, want[:, :, None].cuda(), 1.0)
    out = outputs(n, t)
    pa.pa_verify_drafts(*out, target, want[:, :t].int().cuda(), torch.full((n, t + 1), 0.5, device="cuda"))
    assert torch.equal(out[2].cpu(), want.int()) and (out[0] == t).all()


def test_same_bits_on_a_stream_and_in_a_graph():
    pr = problem(13, 20, 6, 3001, True, True, torch.float32)
    want = expected(pr)
    side = torch.cuda.Stream()
    for a, b in zip(run(pr, stream=side), want):
        np.testing.assert_array_equal(a, b)
    dev = {k: x.cuda() for k, x in pr.items()}
    out = outputs(20, 6)
    call = lambda: pa.pa_verify_drafts(*out, dev["target"], dev["tokens"], dev["uniforms"],  # noqa: E731
                                       draft_probs=dev["draft"], draft_lens=dev["lens"], parents=dev["parents"])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (14, 15):
        pr2 = problem(seed, 20, 6, 3001, True, True, torch.float32)
        for k in dev:
            dev[k].copy_(pr2[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, expected(pr2)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("with_q", [True, False])
def test_kept_tokens_follow_the_target(with_q):
    """The first token is distributed as the target's first row, whatever was drafted: 200000
    sequences of one two-way tree; each count is binomial, so 5 standard deviations bound it
    (16 counts: a chance of 1e-5 at a fixed seed)."""
    n, t, v = 200000, 2, 16
    gen = torch.Generator(device="cuda").manual_seed(16)
    p = torch.rand(v, generator=gen, device="cuda").square()
    q = torch.rand(v, generator=gen, device="cuda").square()
    p, q = p / p.sum(), q / q.sum()
    if with_q:
        tokens = torch.multinomial(q, n * t, replacement=True, generator=gen).view(n, t)
    else:
        tokens = torch.randint(0, v, (n, t), generator=gen, device="cuda")
    out = outputs(n, t)
    pa.pa_verify_drafts(*out, p.expand(n, t + 1, v).contiguous(), tokens.int().contiguous(),
                        torch.rand((n, t + 1), generator=gen, device="cuda"),
                        draft_probs=q.expand(n, t, v).contiguous() if with_q else None,
                        parents=torch.full((n, t), -1, dtype=torch.int32, device="cuda"))
    got = torch.bincount(out[2][:, 0].long(), minlength=v).double()
    sd = (n * p.double() * (1 - p.double())).sqrt()
    assert ((got - n * p.double()).abs() <= 5 * sd + 1).all()
