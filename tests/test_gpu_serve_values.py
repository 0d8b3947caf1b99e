"""The operators of a serving step at values and in orders where a mistake would be small or rare."""
import pytest

from test_gpu_serve import af, lora_call, lora_ref  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---------------------------------------------------------------- adapters: factors far from one

@pytest.mark.parametrize("xs,a_s,bs", [(1e-30, 1e33, 1.0), (1e33, 1e-30, 1.0), (1e-36, 1e36, 1.0), (1e-30, 1.0, 1e33),
                                       (1e30, 1.0, 1e-30), (1e-20, 1e-15, 1e36), (1.0, 1.0, 1.0)])
@pytest.mark.parametrize("n,m,r,K,N", [(1, 1, 16, 96, 128), (9, 1, 24, 512, 77), (40, 3, 64, 256, 260), (70, 2, 8, 64, 64)])
def test_lora_factors_far_from_one(af, xs, a_s, bs, n, m, r, K, N):
    """fp32 weights and rows whose sizes are far apart while their products are not: as with neither of them scaled."""
    g = torch.Generator(device="cuda").manual_seed(n + r)
    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, a, b = normal(n, K) * xs, normal(m, r, K) * a_s, normal(m, N, r) * bs
    ids = torch.randint(0, m, (n,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.empty(n, N, device="cuda")
    lora_call(af, x, ids, a, b, None, None, None, y, N)
    ref, tol = lora_ref(x, ids, a, b, None, None, torch.zeros(n, N, device="cuda"))
    assert torch.isfinite(y).all()
    assert ((y.double() - ref).abs() <= tol).all(), ((y.double() - ref).abs() / tol).max()


def test_lora_large_factors_that_do_not_meet(af):
    """The largest of x meet zeros of A and the other way round: what is left is the small sums."""
    n, m, r, K, N = 20, 1, 16, 64, 48
    g = torch.Generator(device="cuda").manual_seed(2)
    x, a = torch.zeros(n, K, device="cuda"), torch.zeros(m, r, K, device="cuda")
    x[:, ::4], a[:, :, 1::4] = 1e38, 1e38
    x[:, 2::4] = torch.randn(n, K // 4, generator=g, device="cuda") * 1e30
    a[:, :, 2::4] = torch.randn(m, r, K // 4, generator=g, device="cuda") * 1e-30
    b = torch.randn(m, N, r, generator=g, device="cuda")
    y = torch.empty(n, N, device="cuda")
    lora_call(af, x, torch.zeros(n, dtype=torch.int32, device="cuda"), a, b, None, None, None, y, N)
    assert torch.isfinite(y).all()
