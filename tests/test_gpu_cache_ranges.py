"""Attention over caches whose grids, queries or lengths leave the usual range: every legal finite
input is within the bound of oracle.attend_bound."""
import numpy as np
import pytest
import torch

import oracle
from cache_util import DEV, HostCache, check_attend, dev
from post_weight_quantization_12_b200 import _lib

pytestmark = pytest.mark.gpu


def _host(k, v, bits, group, page=16):
    """A cache of one head whose slots hold k and v [tokens, dim], page after page."""
    host = HostCache.__new__(HostCache)
    host.bits, host.dim, host.page, host.heads = bits, k.shape[1], page, 1
    pages = -(-k.shape[0] // page)
    host.part = {}
    for half, x in (("k", k), ("v", v)):
        full = np.zeros((pages * page, k.shape[1]), np.float32)
        full[:len(x)] = x
        host.part[half] = oracle.grid_quantize(full.reshape(pages, 1, page, -1), bits, group)
    return host


def _queries(n, dim, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, 1, dim, generator=g).to(torch.bfloat16)


def _attend(host, tokens, q, scale=None, rows=None):
    """Every row of q [rows, 1, dim] meets the first `tokens` positions: as the query heads of one
    token, and as a shared prefix (from 33 rows on by the kernel for many rows)."""
    scale = host.dim ** -0.5 if scale is None else scale
    pages = host.part["k"][0].shape[0]
    table = np.arange(pages, dtype=np.int32)
    n, cache = q.shape[0], host.device()
    one = q.transpose(0, 1)
    own = cache.attend(one.contiguous().to(DEV), dev(table[None]),
                       dev(np.array([tokens], np.int32)), scale=scale)
    pre = cache.attend_shared(q.to(DEV), dev(table), tokens, dev(np.zeros((n, 1), np.int32)),
                              dev(np.zeros(n, np.int32)), scale=scale)
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0
    args = [p[:, 0].reshape(-1, p.shape[-1])[:tokens] for half in "kv" for p in host.part[half]]
    for i in range(n) if rows is None else rows:
        for got, many in ((own[0, i], False), (pre[i, 0], n > 32)):
            ref, tol = oracle.attend_bound(q[i, 0].double().numpy(), *args, scale,
                                           many_rows=many)
            err = np.abs(got.double().cpu().numpy() - ref)
            assert np.all(err <= tol), (i, many, float((err / tol).max()), int((err > tol).sum()))


FORMATS = [(128, 4, 128), (128, 8, 128), (128, 4, 32), (128, 8, 64), (64, 4, 64), (64, 8, 32)]


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("small,large,every", [(-60, 70, 9), (-60, 60, 9), (-90, 90, 5),
                                               (-80, 60, 150)])
def test_value_scales_far_apart(dim, bits, group, n, small, large, every):
    """Even weights: the tokens with the small scales count in the sum of the weights in full, and
    where there are no large ones among a run's tokens their values do, too."""
    rng = np.random.default_rng(every)
    k, v = (rng.standard_normal((150, dim)).astype(np.float32) for _ in range(2))
    e = np.where(np.arange(150) % every == 4, large, small).astype(np.float32)
    host = _host(k, v * np.exp2(e)[:, None], bits, group)
    _attend(host, 150, torch.zeros(n, 1, dim, dtype=torch.bfloat16))
    _attend(host, 150, _queries(n, dim, 1))


@pytest.mark.parametrize("n", [1, 12])
def test_value_scales_far_apart_in_a_long_sequence(n):
    """The same over many runs, which are joined."""
    rng = np.random.default_rng(2)
    k, v = (rng.standard_normal((9000, 64)).astype(np.float32) for _ in range(2))
    e = np.where(rng.random(9000) < 0.01, 65.0, -60.0).astype(np.float32)
    host = _host(k, v * np.exp2(e)[:, None], 8, 64)
    _attend(host, 9000, torch.zeros(n, 1, 64, dtype=torch.bfloat16))


@pytest.mark.parametrize("dim,bits,group", [(128, 4, 32), (128, 8, 32), (128, 4, 64), (64, 8, 32)])
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("size,other", [(1e-4, 0.0), (1e-8, 0.0), (1e-8, 1.0), (1e-4, 1e4),
                                        (2.0 ** -40, 2.0 ** 40)])
def test_groups_of_different_size(dim, bits, group, n, size, other):
    """The first group's values are of size `other` (0: a head dimension padded up), the others'
    of `size`; with even weights and with one token far above the rest."""
    rng = np.random.default_rng(3)
    k, v = (rng.standard_normal((700, dim)).astype(np.float32) for _ in range(2))
    v *= np.where(np.arange(dim) < group, other, size).astype(np.float32)
    host = _host(k, v, bits, group)
    _attend(host, 700, torch.zeros(n, 1, dim, dtype=torch.bfloat16))
    q = np.repeat(k[None, 400:401], n, 0) * np.float32(14 * dim ** 0.5 / (k[400] @ k[400]))
    _attend(host, 700, torch.from_numpy(q).to(torch.bfloat16))      # a score of 14


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("size", [1e-4, 1e-8])
def test_tokens_whose_values_are_zero(dim, bits, group, n, size):
    """A third of the tokens has no values at all (their grid is [-1, 1] all the same)."""
    rng = np.random.default_rng(4)
    k, v = (rng.standard_normal((500, dim)).astype(np.float32) for _ in range(2))
    v *= np.float32(size)
    v[rng.random(500) < 0.33] = 0
    v[37, group // 2:] = 0                # and one has some of them only
    host = _host(k, v, bits, group)
    _attend(host, 500, _queries(n, dim, 2))
    v[:] = 0                              # and a sequence without any
    _attend(_host(k, v, bits, group), 500, _queries(n, dim, 2))


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("up", [124, 118, 100, -110])
def test_queries_and_keys_of_opposite_size(dim, bits, group, n, up):
    """Products of the usual size from queries of 2^up and keys of 2^-up."""
    rng = np.random.default_rng(5)
    k, v = (rng.standard_normal((90, dim)).astype(np.float32) for _ in range(2))
    host = _host(k * np.float32(2.0 ** (2 - up)), v, bits, group)
    q = (_queries(n, dim, 3).float() * 2.0 ** (up - 2)).to(torch.bfloat16)
    assert torch.isfinite(q).all()
    _attend(host, 90, q)


# ------------------------------------------------------------------------------------------------
# a prefix that many rows meet
# ------------------------------------------------------------------------------------------------
ROWS = (0, 17, 39, 139)


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("n", [40, 140])
@pytest.mark.parametrize("outliers,kx,qx", [(0, 1, 1), (2, 15, 8), (4, 20, 20)])
def test_prefix_keys_with_outlier_channels(dim, bits, group, n, outliers, kx, qx):
    """A few channels far above the others, in keys and queries: the scores' error must not grow
    with the scores. Six tokens stand out and share the weight, so an error of their scores shows."""
    rng = np.random.default_rng(8)
    k, v = (rng.standard_normal((600, dim)).astype(np.float32) for _ in range(2))
    at = rng.permutation(dim)[:outliers]
    k[:, at] *= kx / 4
    k[np.ix_(range(50, 590, 100), at)] = kx
    q = _queries(n, dim, 9).float()
    q[:, 0, at] = qx
    _attend(_host(k, v, bits, group), 600, q.to(torch.bfloat16), rows=[r for r in ROWS if r < n])


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("n", [40, 140])
@pytest.mark.parametrize("up", [20, 40, 70])
def test_prefix_of_one_large_value_without_weight(dim, bits, group, n, up):
    """An early token with a huge value that no row gives any weight, and one with a small value:
    the others' values are kept as well as without them."""
    rng = np.random.default_rng(10)
    k, v = (rng.standard_normal((600, dim)).astype(np.float32) for _ in range(2))
    q = _queries(n, dim, 11).float()
    q[:, 0, 3] = 6.0
    k[5], v[5] = 0, v[5] * np.float32(2.0 ** up)
    k[5, 3] = -60 * dim ** 0.5 - up             # its weight: e^-6(60 + up / dim^0.5)
    v[400] *= np.float32(2.0 ** -up)
    _attend(_host(k, v, bits, group), 600, q.to(torch.bfloat16), rows=[r for r in ROWS if r < n])


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("n", [40, 140])
@pytest.mark.parametrize("size", [1e-4, 1e-8])
def test_prefix_tokens_whose_values_are_zero(dim, bits, group, n, size):
    rng = np.random.default_rng(12)
    k, v = (rng.standard_normal((500, dim)).astype(np.float32) for _ in range(2))
    v *= np.float32(size)
    v[rng.random(500) < 0.33] = 0
    v[37, group // 2:] = 0
    if group < dim:
        v[:, :group] = 0                  # a head dimension padded up
    host = _host(k, v, bits, group)
    _attend(host, 500, _queries(n, dim, 13), rows=[r for r in ROWS if r < n])


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("n", [40, 140])
@pytest.mark.parametrize("small,large", [(-40, 40), (-60, 70)])
def test_prefix_value_scales_far_apart(dim, bits, group, n, small, large):
    rng = np.random.default_rng(14)
    k, v = (rng.standard_normal((600, dim)).astype(np.float32) for _ in range(2))
    e = np.where((np.arange(600) // 128) % 2 == 1, large, small) + rng.integers(-9, 9, 600)
    host = _host(k, v * np.exp2(e.astype(np.float32))[:, None], bits, group)
    rows = [r for r in ROWS if r < n]
    _attend(host, 600, torch.zeros(n, 1, dim, dtype=torch.bfloat16), rows=rows)
    _attend(host, 600, _queries(n, dim, 15), rows=rows)


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("up", [124, 100, -110])
def test_prefix_queries_and_keys_of_opposite_size(dim, bits, group, up):
    rng = np.random.default_rng(16)
    k, v = (rng.standard_normal((300, dim)).astype(np.float32) for _ in range(2))
    host = _host(k * np.float32(2.0 ** (2 - up)), v, bits, group)
    q = (_queries(40, dim, 17).float() * 2.0 ** (up - 2)).to(torch.bfloat16)
    _attend(host, 300, q, rows=[0, 17, 39])


# ------------------------------------------------------------------------------------------------
# lengths
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("news,ratio", [(3, 2), (20, 3)])
@pytest.mark.parametrize("over", [1, 2, 15, 1000])
def test_rows_at_positions_past_the_page_table(news, ratio, over):
    """A length past the table: the positions past it are left out, those before it stay where they
    are, also for the rows whose own position lies before the table's end."""
    host = HostCache(4, 2, 16, 64, 8, 64, seed=6)
    table = np.array([[2, 0, 3]], np.int32)
    lengths, starts = np.array([48 + over], np.int32), np.array([0, news], np.int32)
    g = torch.Generator().manual_seed(7)
    q = torch.randn(news, 2 * ratio, 64, generator=g).to(torch.bfloat16)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(table), dev(lengths), dev(starts))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == _lib.GPTQ_INFO_BAD_PAGE
    for i in range(news):
        limit = min(48 + over - news + i + 1, 48)
        check_attend(out[i:i + 1], host, table, [limit], [0, 1], q[i:i + 1], 0.125)
