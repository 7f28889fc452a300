"""pa_verify_drafts over rows that are not normalised: sums far above one are drawn from as given."""
import pytest
import torch

from test_gpu_verify import check, expected, problem, run

pytestmark = pytest.mark.gpu


def undrafted(seed, n, target):
    """A batch whose tokens after the context are drawn at once."""
    gen = torch.Generator().manual_seed(seed)
    t = target.shape[1] - 1
    u = torch.rand((n, t + 1), generator=gen)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    return dict(target=target, draft=None, tokens=torch.zeros((n, t), dtype=torch.int32), uniforms=u,
                lens=torch.zeros(n, dtype=torch.int32), parents=None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("v", [15, 16, 17, 512, 1024, 2048, 4099, 32000, 32768, 65536, 128000])
def test_rows_of_ones(v, dtype):
    """Token floor(u v): sums of 16 up to 128000, in one CTA and in clusters."""
    pr = undrafted(v, 8, torch.ones((8, 2, v), dtype=dtype))
    want = torch.floor(pr["uniforms"][:, 1].double() * v).long()
    assert (torch.from_numpy(expected(pr)[2][:, 0]) == want).all()
    check(pr)


@pytest.mark.parametrize("v", [700, 4099, 50257, 128000])
@pytest.mark.parametrize("size", [1.0, 1e-6, 2.0 ** 40])
def test_rows_of_exponentials(v, size):
    """exp(logit) without its division by the sum."""
    x = torch.exp(2.5 * torch.randn((6, 2, v), generator=torch.Generator().manual_seed(v))) * size
    check(undrafted(v, 6, x))


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("v,dtype", [(300, torch.float32), (5000, torch.bfloat16), (33000, torch.float32),
                                     (70001, torch.float16)])
def test_drafts_over_entries_up_to_one(with_q, tree, v, dtype):
    """Every entry in [0, 1], rows summing to v / 2: rejections sum them, too."""
    pr = problem(60 + v, 5, 6, v, tree, with_q, torch.float32)
    gen = torch.Generator().manual_seed(v)
    pr["target"] = torch.rand((5, 7, v), generator=gen).to(dtype)
    if with_q:
        pr["draft"] = (torch.rand((5, 6, v), generator=gen) * 1.4).clamp(max=1.0).to(dtype)
    pr["lens"] = torch.full((5,), 6, dtype=torch.int32)
    pr["uniforms"][:3, :6] = 0.95
    check(pr)


def test_one_large_entry():
    """A lane's, a warp's, a CTA's sum alone above the limit of its units."""
    v = 40000
    for at in (0, 17, 9000, v - 1):
        x = torch.full((6, 2, v), 1e-4)
        x[:, :, at] = 1000.0
        check(undrafted(at, 6, x))


def test_infinite_entries_end():
    """Sums that no units hold: some token, and the call returns."""
    x = torch.rand((6, 2, 9000))
    x[:, :, 77] = float("inf")
    x[3:, :, 8000] = float("inf")
    got = run(undrafted(3, 6, x))
    assert ((got[2][:, 0] >= -1) & (got[2][:, 0] < 9000)).all()
