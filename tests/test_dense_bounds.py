"""What the bounds of tests/dense_ref.py can see of a sum that lost 64 of its products (no GPU)."""

import pytest
import torch

import dense_ref as ref

BF, HF = torch.bfloat16, torch.float16
SIZES = [(1, 76, 12289), (16, 76, 13679), (32, 64, 12288), (64, 40, 4096), (150, 33, 20001)]


def rnd(g, rows, cols, dtype, scale=1.0):
    return (torch.randn(rows, cols, generator=g) * scale).to(dtype)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_lost_block_shows_in_the_root_mean_square(m, n, k, dtype):
    g = torch.Generator().manual_seed(k)
    x, w, w2 = rnd(g, m, k, dtype), rnd(g, n, k, dtype, k ** -0.5), rnd(g, n, k, dtype, k ** -0.5)
    b = rnd(g, 1, n, dtype)[0]
    short = x.clone()
    short[:, k - 64:] = 0
    for act in ("gelu", "none"):
        whole = ref.linear(x, w, b, None, act, dtype, dtype)[0]
        ref.assert_rms(whole[0].to(dtype), whole, dtype)
        lost = ref.linear(short, w, b, None, act, dtype, dtype)[0][0].to(dtype)
        with pytest.raises(AssertionError):
            ref.assert_rms(lost, whole, dtype)
    for right, wrong in zip(ref.gated(x, w, w2, "silu", dtype),
                            ref.gated(short, w, w2, "silu", dtype)):
        ref.assert_rms(right[0].to(dtype), right, dtype)
        with pytest.raises(AssertionError):
            ref.assert_rms(wrong[0].to(dtype), right, dtype)


@pytest.mark.parametrize("m,n,k", [(20001, 150, 33), (33, 16384, 64)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_lost_block_of_a_gradient_too(m, n, k, dtype):
    """dW sums over tokens, dx over outputs."""
    g = torch.Generator().manual_seed(m)
    x, w, w2 = rnd(g, m, k, dtype), rnd(g, n, k, dtype, .05), rnd(g, n, k, dtype, .05)
    dy, z, u = (rnd(g, m, n, dtype) for _ in range(3))
    short = dy.clone()
    if m > n:
        short[m - 64:] = 0
    else:
        short[:, n - 64:] = 0
    i = 1 if m > n else 0   # of the gradients, the one with the long sum
    for f in (lambda d: ref.linear_bwd(d, z, x, w, "gelu", dtype, dtype)[i],
              lambda d: ref.gated_bwd(d, z, u, x, w, w2, "silu", dtype, dtype)[i]):
        right, wrong = f(dy), f(short)
        ref.assert_rms(right[0].to(dtype), right, dtype, times=2.0)
        with pytest.raises(AssertionError):
            ref.assert_rms(wrong[0].to(dtype), right, dtype, times=2.0)
