"""Attention whose work gives every part of the kernels several rounds: warps that go over many steps
of a ring, runs of many tiles and their joins, and units of the prefix kernel that follow one another
on a CTA. The shapes are checked against the device, so that they keep reaching those paths."""
import numpy as np
import pytest
import torch

import oracle
from cache_util import DEV, HostCache, dev
from post_weight_quantization_12_b200 import _lib

pytestmark = pytest.mark.gpu

FORMATS = [(64, 4, 32), (64, 4, 64), (64, 8, 32), (64, 8, 64), (128, 4, 32), (128, 4, 64),
           (128, 4, 128), (128, 8, 32), (128, 8, 64), (128, 8, 128)]


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _parts(host, table_row, length, head, skip=()):
    pos = np.array([p for p in range(length) if p // host.page not in skip])
    pg, off = np.asarray(table_row)[pos // host.page], pos % host.page
    return [a[pg, head, off] for half in "kv" for a in host.part[half]], pos


def _aim(host, parts, at, seed):
    """A query (bf16) under which the token in row `at` of parts has about as much weight as all the
    others together: were it lost, or met twice, the result would leave the bound."""
    k = oracle.cache_values(*parts[:3])
    rng = np.random.default_rng(seed)
    target = k[at] + 0.3 * rng.standard_normal(host.dim)
    scores = (k @ target) * host.dim ** -0.5
    lo, hi = 0.0, 50.0
    for _ in range(30):
        a = (lo + hi) / 2
        x = a * scores
        x -= x.max()
        w = np.exp(x)
        lo, hi = (a, hi) if w[at] < 0.5 * w.sum() else (lo, a)
    return torch.from_numpy(target * hi).float().to(torch.bfloat16)


def _check(got, q, parts, scale, **kw):
    ref, tol = oracle.attend_bound(q.double().numpy(), *parts, scale, **kw)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), (float((err / tol).max()), int((err > tol).sum()))


def _aimed_rows(host, tables, lengths, ratio, picks, page_skip=None):
    """Queries [batch, heads ratio, dim], one token a sequence, random but for the picked
    (sequence, query head, position) ones; and those with what they meet."""
    g = torch.Generator().manual_seed(1)
    q = torch.randn(len(lengths), host.heads * ratio, host.dim, generator=g).to(torch.bfloat16)
    want = []
    for n, (b, qh, position) in enumerate(picks):
        skip = (page_skip or {}).get(b, ())
        parts, pos = _parts(host, tables[b], lengths[b], qh // ratio, skip)
        q[b, qh] = _aim(host, parts, int(np.searchsorted(pos, position)), n)
        want.append((b, qh, parts))
    return q, want


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("ratio", [2, 11])
def test_runs_of_many_tiles(dim, bits, group, ratio):
    """Sequences of 160 tiles of 64 tokens, all on the same pages in orders of their own, cut into
    runs of more than 33 tiles: rings that are filled many times, page numbers fetched in a second
    batch of 32, items shared by several runs."""
    heads, page, pages, batch = 4, 64, 160, 32
    runs = _sms() * (4 if ratio <= 8 else 2)
    assert batch * heads * pages / runs > 33
    host = HostCache(pages, heads, page, dim, bits, group, seed=dim + bits + group)
    rng = np.random.default_rng(ratio)
    tables = np.stack([rng.permutation(pages) for _ in range(batch)]).astype(np.int32)
    lengths = (pages * page - rng.integers(0, 64, batch)).astype(np.int32)
    cuts = np.unique((np.arange(1, runs) * (batch * heads * pages) // runs) % pages)
    places = [0, 15, 16, 63, 64, 31 * 64, 32 * 64 - 1, 32 * 64, 33 * 64 + 17, int(lengths[5]) - 1] + \
        [int(64 * t) for t in cuts[:: max(1, len(cuts) // 6)]][:6]
    picks = [(int(rng.integers(0, batch)) if i != 9 else 5, int(rng.integers(0, heads * ratio)), at)
             for i, at in enumerate(places)]
    picks = [(b, qh, min(at, int(lengths[b]) - 1)) for b, qh, at in picks]
    q, want = _aimed_rows(host, tables, lengths, ratio, picks)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(tables), dev(lengths))
    again = cache.attend(q.to(DEV), dev(tables), dev(lengths))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0 and torch.equal(out, again)
    for b, qh, parts in want:
        _check(out[b, qh], q[b, qh], parts, dim ** -0.5)


def test_a_bad_page_late_in_a_run():
    """Pages that do not exist, past the first 32 steps of a run and at its next ones."""
    heads, page, pages, batch = 4, 64, 160, 32
    host = HostCache(pages, heads, page, 64, 8, 64, seed=3)
    rng = np.random.default_rng(4)
    tables = np.stack([rng.permutation(pages) for _ in range(batch)]).astype(np.int32)
    lengths = np.full(batch, pages * page, np.int32)
    skip = {3: {33, 34, 70}, 9: {0, 159}, 20: set(range(30, 70))}
    for b, ks in skip.items():
        tables[b, sorted(ks)] = [(-1, 10 ** 6)[i % 2] for i in range(len(ks))]
    picks = [(3, 1, 35 * 64), (3, 6, 32 * 64 + 63), (9, 0, 64), (20, 7, 70 * 64 + 1), (4, 2, 34 * 64)]
    q, want = _aimed_rows(host, tables, lengths, 2, picks, skip)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(tables), dev(lengths))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == _lib.GPTQ_INFO_BAD_PAGE
    for b, qh, parts in want:
        _check(out[b, qh], q[b, qh], parts, 0.125)


@pytest.mark.parametrize("dim,bits,group", [(128, 8, 128), (64, 4, 32), (128, 4, 64)])
def test_an_item_per_warp_of_many_steps(dim, bits, group):
    """Enough sequences times heads for every warp to work on its own, over items of 10 to 80 steps:
    runs that end and begin inside items."""
    heads, page, pages, batch = 4, 16, 80, 640
    assert batch * heads >= _sms() * 16
    host = HostCache(pages, heads, page, dim, bits, group, seed=bits)
    rng = np.random.default_rng(5)
    tables = np.stack([rng.permutation(pages) for _ in range(batch)]).astype(np.int32)
    lengths = rng.integers(150, pages * page + 1, batch).astype(np.int32)
    lengths[[7, 300]] = [pages * page, 0]
    picks = [(7, 0, 0), (7, 1, 31 * 16 + 15), (7, 2, 32 * 16), (7, 3, 1279), (639, 4, 149)]
    picks += [(int(b), int(qh), 16 * int(rng.integers(0, 9))) for b, qh in
              zip(rng.integers(301, 639, 12), rng.integers(0, 8, 12))]
    q, want = _aimed_rows(host, tables, lengths, 2, picks)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(tables), dev(lengths))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0 and torch.all(out[300] == 0)
    for b, qh, parts in want:
        _check(out[b, qh], q[b, qh], parts, dim ** -0.5)


# ------------------------------------------------------------------------------------------------
# units of the prefix kernel
# ------------------------------------------------------------------------------------------------
def _units(heads, rows, prefix):
    """(units, steps of the longest) of the prefix kernel: per item of up to 256 rows the split with
    the fewest rounds times their length."""
    sms, tiles = _sms(), -(-prefix // 128)
    items = heads * -(-rows // 256)
    most = min(tiles, max(max(items, 2 * sms) // items, 1))
    cost = {s: -(-items * s // sms) * (-(-tiles // s) + 2) for s in range(1, most + 1)}
    s = min(cost, key=lambda k: (cost[k], k))
    return items * s, -(-tiles // s)


def _prefix_case(heads, n, ratio, prefix, dim, bits, group, picks, scales=False, page=128):
    pages = -(-prefix // page)
    host = HostCache(pages, heads, page, dim, bits, group, seed=heads + n)
    if scales:          # V's grids rise and fall from tile to tile
        e = np.array([0, 11, -12, 3, 14, -10, 12, 0, -14, 5])[np.arange(pages * page) // 128 % 10]
        host.part["v"][1][:] *= np.exp2(e).astype(np.float32).reshape(pages, 1, page, 1)
    ptable = np.random.default_rng(n).permutation(pages).astype(np.int32)
    if scales:
        ptable = np.arange(pages, dtype=np.int32)
    tables = np.repeat(ptable[None], n, 0)
    q, want = _aimed_rows(host, tables, np.full(n, prefix), ratio, picks)
    cache = host.device()
    args = (q.to(DEV), dev(ptable), prefix, dev(np.zeros((n, 1), np.int32)),
            dev(np.zeros(n, np.int32)))
    out = cache.attend_shared(*args)
    again = cache.attend_shared(*args)
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0 and torch.equal(out, again)
    for i, qh, parts in want:
        _check(out[i, qh], q[i, qh], parts, dim ** -0.5, many_rows=True)


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("scales", [False, True])
def test_units_of_two_and_one_row_tiles_on_one_cta(dim, bits, group, scales):
    """192 items of 32 heads, the last of each head with 20 rows: CTAs that take a second unit, of
    the other kind too."""
    heads, n, prefix = 32, 260, 700
    units, steps = _units(heads, n * 5, prefix)
    assert units > _sms() and steps >= 5
    rng = np.random.default_rng(6)
    picks = [(i, int(rng.integers(0, heads)) * 5 + r, at) for i, r, at in (
        (0, 0, 0), (51, 0, 699), (51, 1, 128), (51, 2, 127), (102, 3, 383), (255, 4, 600),
        (256, 0, 512), (259, 4, 640), (258, 2, 1), (130, 1, 300))]
    picks += [(257, 31 * 5, 699), (256, 31 * 5 + 1, 5), (0, 31 * 5 + 2, 511), (140, 30 * 5, 256)]
    _prefix_case(heads, n, 5, prefix, dim, bits, group, picks, scales)


@pytest.mark.parametrize("heads,prefix", [(100, 640), (100, 700), (150, 1150), (74, 2500)])
@pytest.mark.parametrize("n,scales", [(40, False), (128, True)])
def test_units_of_one_row_tile(heads, prefix, n, scales):
    """Items near the number of SMs, at most 128 rows: both softmax groups over every other tile,
    for odd and even counts."""
    units, steps = _units(heads, n, prefix)
    assert steps >= 5
    rng = np.random.default_rng(7)
    picks = [(int(rng.integers(0, n)), int(rng.integers(0, heads)), at) for at in
             (0, 127, 128, 255, 256, 511, 512, 639, prefix - 1, prefix - 130)]
    dim, bits, group = ((64, 8, 32), (64, 4, 64))[scales]
    _prefix_case(heads, n, 1, prefix, dim, bits, group, picks, scales)


@pytest.mark.parametrize("dim,bits,group", [(128, 4, 128), (128, 8, 32)])
def test_units_of_many_steps(dim, bits, group):
    """A prefix of more than 20 tiles a unit, grids that rise and fall."""
    heads, n, prefix = 20, 300, 22 * 128 * 7 + 77
    units, steps = _units(heads, n, prefix)
    assert steps >= 20
    picks = [(i, qh, at) for i, qh, at in ((0, 0, 128 * 21), (255, 7, 128 * 22 + 1), (256, 19, 77),
                                           (299, 3, prefix - 1), (130, 12, 128 * 44), (7, 9, 5000))]
    _prefix_case(heads, n, 1, prefix, dim, bits, group, picks, scales=True)
