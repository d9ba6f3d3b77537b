"""Head norms of elements whose squares leave fp32, with an eps as small, against the
formula in 64 bits."""
import pytest
import torch

import kv8util as ref
from test_gpu_qk_rope import check, formula, projection, w4, weights  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,interleaved", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-30, 1e-6])
@pytest.mark.parametrize("tokens", [3, 700, 9000])
def test_small_heads(w4, dim, interleaved, eps, tokens):
    """Heads of one size each, from the smallest bf16 to 2^50, side by side in a warp, and
    some whose elements are of all sizes. fp32 holds eps 1e-44 as a subnormal number."""
    x = projection(tokens, 5, dim, "bf16", 30, spread=0)
    size = torch.linspace(-130, 50, 5 * tokens, device="cuda").round().view(tokens, 5, 1)
    size = size.flatten()[torch.randperm(5 * tokens, device="cuda", generator=torch.Generator("cuda").manual_seed(1))]
    wide = (x.double() * torch.exp2(size.double().view(tokens, 5, 1))).to(torch.bfloat16)
    each = torch.linspace(-140, -50, dim, device="cuda").double().exp2()
    wide[0] = (x[0].double() * each).to(torch.bfloat16)
    wide[tokens // 2, 1:4] = (x[tokens // 2, 1:4].double() * each * 2.0 ** 40).to(torch.bfloat16)
    wide = torch.where((wide == 0).all(-1, keepdim=True), torch.full_like(wide, 2.0 ** -133), wide)
    pos, table = ref.ints(list(range(tokens))), w4.rope_table(tokens, dim)
    wq, wk = weights(dim, 31)
    exact = float(torch.tensor(eps, dtype=torch.float32))
    for norms in ((wq, wk), (wq, None), (None, wk)):
        got = w4.qk_norm_rope(wide[:, :3], wide[:, 3:], pos, table, *norms, exact, interleaved)
        for y, z, w in zip(got, (wide[:, :3], wide[:, 3:]), norms):
            want, tol = formula(z, w, pos, table, interleaved, exact)
            # (results below bf16's normal range are off by half a step of 2^-133 more)
            check(y, want, tol + 2.0 ** -134)
            assert torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_heads_of_zeros(w4, dtype):
    """NaN with eps 0, as the formula says, zeros with any other; their neighbours are not touched."""
    x = projection(9, 7, 64, dtype, 32)
    x[2, 3] = 0
    x[8, 6] = -0.0
    wq, wk = weights(64, 33)
    for eps in (0.0, 1e-44, 1e-6):
        exact = float(torch.tensor(eps, dtype=torch.float32))
        got = torch.cat(w4.qk_norm_rope(x[:, :5], x[:, 5:], None, None, wq, wk, exact), 1)
        want, tol = (torch.cat(z, 1) for z in zip(formula(x[:, :5], wq, None, None, False, exact),
                                                  formula(x[:, 5:], wk, None, None, False, exact)))
        assert got[2, 3].isnan().all() == (eps == 0) == got[8, 6].isnan().all()
        check(got, want, tol)


def test_the_smallest_fp16(w4):
    x = torch.full((4, 2, 128), 2.0 ** -24, dtype=torch.float16, device="cuda")
    x[1::2, :, ::3] *= -1
    w = torch.ones(128, device="cuda")
    q, _ = w4.qk_norm_rope(x, None, None, None, w, None, 0.0)
    assert torch.equal(q, torch.sign(x))
