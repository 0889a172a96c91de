"""Walks of many clusters at once, while other work holds the SMs: a cluster's CTAs
then start apart, and every walk has to come out as alone. With requests that
have no node among the others."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_candidates import check_walk, drafted  # noqa: E402
from test_gpu_paged import i32  # noqa: E402


@pytest.fixture(scope="module")
def d():
    import decode_dsa_kv_gb300 as mod
    return mod


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V, B", [(300, 400), (5003, 100), (20000, 12)])
def test_walks_beside_other_work(d, sampled, V, B):
    rng = np.random.default_rng(V)
    depth, sizes = 3, [int(x) for x in rng.integers(0, 4, B)]
    sizes[0], sizes[-1] = 0, 3
    p, parents, tokens = drafted(rng, V, sizes, sharp=4.0)
    u = rng.random((B, depth + 1)).astype(np.float32) if sampled else None
    args = (i32(tokens), i32(parents), i32(np.cumsum([0] + sizes)), torch.from_numpy(p).cuda(),
            torch.from_numpy(u).cuda() if sampled else None, depth)
    first = d.verify_tree(*args)
    check_walk(d, p, parents, tokens, sizes, u, depth, first)
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(60):
        with torch.cuda.stream(other):
            b = a @ a
        got = d.verify_tree(*args)
        assert all(torch.equal(x, y) for x, y in zip(got, first))
    torch.cuda.synchronize()
    assert b.shape == a.shape
