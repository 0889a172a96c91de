"""The beams' sums of exponentials, by scores near 0: where one token of a late
round has nearly all of a row, its exponential is what the sum's error is."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


def errors(d, x):
    """Of the best token's log-probability: cum is its size, so that the score is
    near 0 and its rounding to fp32 is nothing."""
    top, at = x.double().max(1)
    lse = torch.logsumexp(x.double(), 1)
    cum = (lse - top).float()
    t, _, s = d.beam_select(x.view(x.shape[0], 1, -1), cum.view(-1, 1), 1)
    assert torch.equal(x.gather(1, t.long()), x.gather(1, at.view(-1, 1)))
    return (s.view(-1).double() - (cum.double() + (top - lse))).abs()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("height", [24, 31, 38, 44, 52, 75])
def test_one_token_has_nearly_everything(d, dtype, height):
    # 512 rows in pieces of 8 rounds; a value of the first rounds in every 97 tokens, so
    # that a warp has a reference and little else
    rows, V = 512, 131072
    g = torch.Generator(device="cuda").manual_seed(height)
    x = torch.full((rows, V), -math.inf, device="cuda")
    x[:, ::97] = torch.rand(rows, -(-V // 97), generator=g, device="cuda")
    x[:, 9000] = height + torch.rand(rows, generator=g, device="cuda")
    # the exponential's 2^-22; two roundings of its argument, which is below 8 (and as
    # much as its limit's rounding more: 2^-21 each), times log 2; the logarithm's 2^-29;
    # the other tokens' part of a warp's sum, 43 e^-23, is lost at most
    bound = 2.0 ** -22 + math.log(2) * 2 * 2.0 ** -21 + 2.0 ** -29 + 43 * math.exp(1 - height)
    assert float(errors(d, x.to(dtype)).max()) <= bound


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("height", [0, 5, 12, 20, 30])
def test_usual_rows(d, dtype, height):
    rows, V = 512, 131072
    g = torch.Generator(device="cuda").manual_seed(height)
    x = 2.5 * torch.randn(rows, V, generator=g, device="cuda")
    if height:
        x[:, 9000] = height + torch.rand(rows, generator=g, device="cuda")
    # the header's: 2^-22, an argument's 2^-19.5, 71 additions
    e = errors(d, x.to(dtype))
    assert float(e.max()) <= 2.0 ** -22 + 2.0 ** -19.5 + 71 * 2.0 ** -24 + 2.0 ** -29 <= 2.0 ** -17
