"""The 4-bit product along long axes, where a part of K that is lost or taken twice has
to show among very many terms.

Two kinds of inputs.  Small whole numbers with scales of 1 and 2: every sum of terms,
in any order, is a whole number below 2^24, so the product is exact and the comparison
too.  And states as they are used, with a tolerance from the way sums are held: within
a group at most 24 roundings (or cuts) of u = 2^-24 on sums no larger than the sum of
its terms' magnitudes; a group's sum is then added to others that follow one another
along K, whose sum is the difference of two prefixes, one rounding each; parts of x and
of K add as many as there are groups at most.  In all 2 u P (G + 64) + 24 u sum |w x|
+ u |y|, P the largest magnitude of a prefix, G the number of groups."""
import numpy as np
import pytest
import torch

import readout_oracle as ro

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# 12 warps in whole tiles, slabs, 16 warps (long runs), two column tiles, batches with K in
# one run and in several
SIZES = [(1, 20001, 7), (1, 40000, 100), (4, 211577, 40), (1, 211577, 4096), (3, 100001, 3000), (16, 60000, 500),
         (20, 40000, 100), (32, 9000, 2000), (33, 211577, 300), (96, 20001, 257)]


def packed(nibbles):
    V, K = nibbles.shape
    n = (K + 1) // 2
    q = torch.zeros(V, -(-n // 16) * 16, dtype=torch.uint8, device="cuda")[:, :n]
    full = torch.nn.functional.pad(nibbles, (0, K % 2))
    q.copy_(full[:, 0::2] + 16 * full[:, 1::2])
    return q


def inputs(M, K, V, group, zeros, whole, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *a, **kw: torch.randint(*a, generator=g, device="cuda", **kw)  # noqa: E731
    G = -(-K // group)
    nibbles = rand(0, 16, (V, K), dtype=torch.uint8)
    z = rand(0, 16, (V, G), dtype=torch.uint8) if zeros else None
    if whole:
        x, s = rand(-1, 2, (M, K)).double(), 2.0 ** rand(0, 2, (V, G)).double()
    else:
        x = torch.tanh(torch.randn(M, K, generator=g, device="cuda")).double()
        s = ((0.5 + torch.rand(V, G, generator=g, device="cuda")) / K ** 0.5).half().double()
    return nibbles, z, x, s


def terms(nibbles, z, s, group, rows):
    """The weights, in 64 bits, of some rows of V."""
    K = nibbles.shape[1]
    at = torch.arange(K, device="cuda") // group
    zero = 8.0 if z is None else z[rows].double()[:, at]
    return (nibbles[rows].double() - zero) * s[rows][:, at]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("M,K,V", SIZES)
def test_whole_numbers_are_exact(M, K, V, group, zeros, dtype):
    import sparse_graph_recurrent_gb300 as ck
    nibbles, z, x, s = inputs(M, K, V, group, zeros, True, M + K + group)
    assert K * 15 * 2 < 2 ** 24
    y = ck.int4_matvec(x.to(dtype), packed(nibbles), s.to(dtype), z, group_size=group)
    for r in range(0, V, 256):
        rows = slice(r, r + 256)
        w = terms(nibbles, z, s, group, rows)
        assert torch.equal(y[:, rows], (x @ w.t()).to(dtype)), r
        if r == 0:
            # no 64 columns can be left out or taken twice unseen
            pad = (0, -K % 64)
            steps = torch.einsum("kj,vkj->vk", torch.nn.functional.pad(x[:1], pad).view(-1, 64),
                                 torch.nn.functional.pad(w[:32], pad).view(min(V, 32), -1, 64))
            assert (steps != 0).any(0).all()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("M,K,V", [(1, 40000, 100), (4, 211577, 40), (1, 211577, 4096), (20, 40000, 100), (33, 211577, 300)])
def test_states_within_what_sums_lose(M, K, V, group):
    import sparse_graph_recurrent_gb300 as ck
    nibbles, z, x, s = inputs(M, K, V, group, True, False, K + V)
    x = x.float()
    y = ck.int4_matvec(x, packed(nibbles), s.half(), z, group_size=group).double()
    G = -(-K // group)
    for r in sorted({0, max(0, V - 64)}):
        rows = slice(r, r + 64)
        w = terms(nibbles, z, s, group, rows)
        for m in sorted({0, M - 1}):
            t = w * x[m].double()
            prefix = t.cumsum(1)
            tol = 2 * U * prefix.abs().max(1).values * (G + 64) + 24 * U * t.abs().sum(1) + U * prefix[:, -1].abs()
            err = (y[m, rows] - prefix[:, -1]).abs()
            assert (err <= tol).all(), float((err / tol).max())
            # the definition without 64 columns of K lies outside of it, in most rows
            for at in (0, K // 128 * 64, K - 64):
                assert (t[:, at:at + 64].sum(1).abs() > 2 * tol).float().mean() > 0.5


@pytest.mark.parametrize("M,K,V", [(1, 211577, 33), (4, 40000, 40), (20, 40000, 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_single_columns_at_the_edges(M, K, V, dtype):
    """x is 1 in one column and 0 elsewhere: y is that column of the weights."""
    import sparse_graph_recurrent_gb300 as ck
    nibbles, z, _, s = inputs(M, K, V, 64, True, True, K)
    q, st, w = packed(nibbles), s.to(dtype), terms(nibbles, z, s, 64, slice(0, V))
    edges = {0, K - 1, K - 2}
    for step in (32, 64, 128, 256, 2048, 8192, 14336, 32768):
        for k in (1, K // step // 2, K // step):
            edges |= {k * step - 1, k * step}
    at = sorted(e for e in edges if 0 <= e < K)
    for i in range(0, len(at), M):
        cols = at[i:i + M]
        x = torch.zeros(M, K, dtype=dtype, device="cuda")
        for m, k in enumerate(cols):
            x[m, k] = 1
        y = ck.int4_matvec(x, q, st, z, group_size=64)
        assert torch.equal(y[:len(cols)].double(), w[:, cols].t())
        assert not y[len(cols):].any()


@pytest.mark.parametrize("M", [1, 4, 20])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_every_output_of_a_row_that_is_not_finite(M, dtype):
    import sparse_graph_recurrent_gb300 as ck
    nibbles, z, x, s = inputs(M, 9001, 333, 32, True, False, 3)
    q, x, s = packed(nibbles), x.to(dtype), s.to(dtype)
    clean = ck.int4_matvec(x, q, s, z, group_size=32)
    assert torch.isfinite(clean).all()
    for bad in (float("inf"), -float("inf"), float("nan")):
        for k in (0, 4097, 9000):
            v = x.clone()
            v[M // 2, k] = bad
            y = ck.int4_matvec(v, q, s, z, group_size=32)
            assert not torch.isfinite(y[M // 2]).any()
            rest = torch.arange(M, device="cuda") != M // 2
            assert torch.equal(y[rest], clean[rest])


def test_the_oracle_agrees_with_the_weights_here():
    nibbles, z, _, s = inputs(1, 333, 9, 32, True, False, 5)
    w = ro.dequantize(packed(nibbles).cpu().numpy(), s.cpu().numpy(), z.cpu().numpy(), 333, 32)
    assert np.allclose(terms(nibbles, z, s, 32, slice(0, 9)).cpu().numpy(), w, rtol=1e-15)
