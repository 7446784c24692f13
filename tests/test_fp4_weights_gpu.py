"""What fp32 attention over the 4-bit cache keeps of small weights: a first key that
outweighs every other by up to 2^18, the others alike, so that what a weight loses is lost
in every one of them."""
import numpy as np
import pytest
import torch

from fp4_step import Batch, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head_dim", [16, 64])
@pytest.mark.parametrize("drop", [10.3, 13.7, 16.3, 17.15, 17.7, 18.0])
def test_small_weights_keep_22_bits(drop, head_dim):
    """Off relatively by at most: 2^-21 for a weight in two f16 terms and 2^-22 for exp2; a
    score's roundings, four of 2^-24 at its magnitude (the factor, the reference, their
    difference), as a factor of the weight (ln 2); sums over the blocks, half a step of 2^-24
    of the output's and half a step of 2^-19 of the sum of the weights, which is 16 or more
    (the first key's), a block; and 2^-22 for the product of a block, whose sum is cut off."""
    n, blocks = 1025, 65
    bt = Batch([n], n_kv=1, head_dim=head_dim, dtype="f32", scale=2.0 ** -3)
    k, v = torch.zeros(n, 1, head_dim), torch.ones(n, 1, head_dim)
    k[0, 0, 0] = 6.0
    v[0] = 0.0
    v[1:] *= 1.0 + torch.arange(head_dim) / 32.0
    bt.write(bt.slots([n], [n]), k, v)
    scale = 1.0 / np.sqrt(head_dim)
    q = torch.zeros(1, 1, head_dim)
    q[0, 0, 0] = float(np.float16(drop / (scale * np.log2(np.e) * 6.0)))
    outs = [bt.decode(q, max_ctas=c) for c in (0, 1, 3)] + [bt.prefill(q, [n], [1])]
    bt.no_error()
    K, V = bt.rows(0, n)
    s = scale * (K[:, 0] @ f64(q)[0, 0])
    p = np.exp(s - s.max())
    ref = (p @ V[:, 0]) / p.sum()
    tol = (2.0 ** -21 + 2 * 2.0 ** -22 + np.log(2) * 4 * 2.0 ** -24 * (drop + 4) + blocks * 2.0 ** -24
           + blocks * 2.0 ** -20 / 16)
    for out in outs:
        off = np.abs(f64(out)[0, 0] / ref - 1).max()
        assert off <= tol, (off, tol)


@pytest.mark.parametrize("head_dim", [32, 128])
def test_bf16_sums_over_a_very_long_sequence(head_dim):
    """Output sums that one CTA takes over the whole sequence are cut off at every product:
    too small by up to 2^-23 for each 16 tokens, beside the output's own half step, and its
    weights' 2^-11 (f16), of either sign."""
    n = 131_077
    bt = Batch([n], n_kv=1, head_dim=head_dim, seed=2, scale=2.0 ** -4)
    k, v = bt.draw(n, 0.2), (1.0 + 0.25 * torch.randn(n, 1, head_dim, generator=bt.g)).to(bt.dtype)
    bt.write(bt.slots([n], [n]), k, v)
    q = bt.queries(3, 2, mag=0.3)
    outs = [(bt.decode(q[-1:], max_ctas=1), [n - 1]), (bt.prefill(q, [n], [3]), range(n - 3, n))]
    bt.no_error()
    for out, lasts in outs:
        for i, last in enumerate(lasts):
            ref, _ = bt.reference(f64(q[i - len(lasts)]), 0, last)
            off = np.abs(f64(out[i]) - ref) / np.abs(ref)
            assert off.max() <= 2.0 ** -8 + n / 16 * 2.0 ** -23 + 2.0 ** -11, off.max()
