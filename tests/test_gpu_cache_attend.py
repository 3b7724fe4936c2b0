"""Attention over the quantized cache on the GPU, against the fp64 oracle within the bound that
oracle.attend_bound derives from the arithmetic."""
import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import DEV, HostCache, check_attend, dev, make_table
from post_weight_quantization_12_b200 import _lib, api

pytestmark = pytest.mark.gpu

FORMATS = [(64, 4, 32), (64, 4, 64), (64, 8, 32), (64, 8, 64), (128, 4, 32), (128, 4, 64),
           (128, 4, 128), (128, 8, 32), (128, 8, 64), (128, 8, 128)]


def _starts(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


def _q(n, heads, dim, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, dim, generator=g).to(torch.bfloat16)


def _run(host, lengths, news, ratio, seed=0, rows=None, scale=None, width=None, table=None, q=None,
         pages=None):
    lengths = np.asarray(lengths, np.int32)
    starts = _starts(news)
    if table is None:
        table = make_table(lengths, host.page, host.part["k"][0].shape[0], seed, width=width)
    if q is None:
        q = _q(int(starts[-1]), host.heads * ratio, host.dim, seed + 1)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(table), dev(lengths), dev(starts), scale=scale)
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0
    check_attend(out, host, table, lengths, starts, q,
                 host.dim ** -0.5 if scale is None else scale, rows=rows)
    return out


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("ratio", [1, 5, 8, 12])
def test_formats_and_head_ratios(dim, bits, group, ratio):
    host = HostCache(40, 2, 16, dim, bits, group, seed=dim + bits + ratio)
    _run(host, [1, 37, 130, 16, 65], [1, 1, 1, 1, 1], ratio, seed=ratio)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_lengths_around_steps_tiles_and_pages(length, page):
    host = HostCache(max(3, -(-length // page) + 1), 1, page, 128, 4, 128, seed=length)
    _run(host, [length], [1], 4)


@pytest.mark.parametrize("news", [[2, 1, 5, 0, 3], [1, 20, 7, 0, 40], [33, 0, 0, 64, 1]])
@pytest.mark.parametrize("ratio", [1, 3, 8])
def test_several_tokens_per_sequence(news, ratio):
    """Causal within the new tokens; row tiles that hold several tokens and end inside a head
    group."""
    past = [0, 40, 100, 9, 63]
    host = HostCache(60, 2, 16, 64, 8, 32, seed=sum(news))
    _run(host, [p + n for p, n in zip(past, news)], news, ratio)


def test_rows_that_meet_nothing():
    """Length 0, and more new rows than the sequence is long: such rows give 0 and the others are
    right."""
    host = HostCache(10, 2, 16, 128, 4, 64, seed=3)
    out = _run(host, [0, 3, 17, 0], [1, 5, 1, 2], 2)
    assert torch.all(out[0] == 0) and torch.all(out[1:3] == 0) and torch.all(out[7:] == 0)
    assert torch.all(out[3:7].abs().amax((1, 2)) > 0)


def test_long_sequences_are_split_and_joined():
    host = HostCache(200, 1, 64, 128, 8, 128, seed=8)
    _run(host, [12000], [1], 4)
    host = HostCache(300, 2, 32, 64, 4, 32, seed=9)
    _run(host, [4000, 17, 5000], [1, 2, 3], 2, rows=[0, 1, 2, 5])


def test_many_short_sequences():
    rng = np.random.default_rng(1)
    lengths = rng.integers(1, 60, 700)
    host = HostCache(2800, 2, 16, 64, 4, 64, seed=10)
    _run(host, lengths, [1] * 700, 3, rows=set(range(0, 700, 17)) | {699})


def test_lengths_that_differ_widely():
    host = HostCache(260, 4, 16, 128, 4, 128, seed=11)
    _run(host, [1, 3000, 1, 1, 700, 2, 1, 150], [1] * 8, 4)


def test_scales_that_span_the_range():
    """V grids from 2^-40 to 2^40 within a tile: the small ones must count where the weights are
    theirs."""
    host = HostCache(12, 1, 16, 128, 4, 32, seed=12, spread=40.0)
    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16)      # even weights
    _run(host, [150], [1], 2, q=q)
    c, s, z = host.part["v"]
    host.part["k"] = HostCache(12, 1, 16, 128, 4, 32, seed=13).part["k"]
    _run(host, [150], [1], 2)
    # one token a page with a scale 2^60 below the others
    host = HostCache(12, 1, 16, 128, 4, 128, seed=14)
    s = host.part["v"][1]
    s[:, :, 3] *= np.float32(2.0 ** -60)
    _run(host, [150], [1], 2, scale=0.5)


def test_queries_of_any_magnitude():
    host = HostCache(10, 1, 16, 64, 8, 64, seed=15)
    q = _q(3, 2, 64, 1).float() * torch.tensor([2.0 ** -100, 1.0, 0.0])[:, None, None]
    q[1, 0, 5] = 2.0 ** 9
    _run(host, [40, 50, 20], [1, 1, 1], 2, q=q.to(torch.bfloat16))
    q = (_q(1, 1, 64, 2).float() * 2.0 ** 100).to(torch.bfloat16)
    _run(host, [40], [1], 1, q=q, scale=2.0 ** -103)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-6])
def test_any_scale(scale):
    host = HostCache(30, 1, 16, 128, 4, 128, seed=22)
    q = _q(3, 4, 128, 9)
    lengths, starts = np.array([100, 37], np.int32), np.array([0, 1, 3], np.int32)
    table = make_table(lengths, 16, 30, 1, first=9)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(table), dev(lengths), dev(starts), scale=scale)
    torch.cuda.synchronize()
    check_attend(out, host, table, lengths, starts, q, abs(scale) or 1.0, flip=scale)
    q = _q(40, 4, 128, 10)
    starts = np.array([0, 17, 40], np.int32)
    ptable = np.arange(9, dtype=np.int32)
    out = cache.attend_shared(q.to(DEV), dev(ptable), 140, dev(table), dev(lengths), dev(starts),
                              scale=scale)
    torch.cuda.synchronize()
    check_attend(out, host, table, lengths, starts, q, abs(scale) or 1.0, flip=scale,
                 prefix=(ptable, 140), image16=True, rows={0, 16, 20, 39})


def test_a_cache_past_four_gigabytes():
    """Pages whose codes lie 5 GB into the tensors: written, read, attended to, as a prefix too."""
    heads, dim, page = 8, 128, 64
    pages = 5 * 2 ** 30 // (heads * page * dim) + 8
    t = [torch.empty(pages, heads, page, n, dtype=dt, device=DEV) for _ in range(2)
         for n, dt in ((dim // 4, torch.int32), (1, torch.bfloat16), (1, torch.uint8))]
    cache = api.QuantizedCache.of_tensors(*t, dim=dim)
    g = torch.Generator().manual_seed(11)
    K, V = (torch.randn(100, heads, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    table = np.array([[pages - 1, pages - 3]], np.int32)
    lengths, starts = np.array([100], np.int32), np.array([0, 100], np.int32)
    hat = [torch.empty_like(K, device=DEV) for _ in range(2)]
    cache.append(K.to(DEV), V.to(DEV), dev(table), dev(lengths), dev(starts), *hat)
    back = cache.read(dev(table), dev(lengths), dev(starts), n=100)
    torch.cuda.synchronize()
    assert torch.equal(back[0], hat[0]) and torch.equal(back[1], hat[1])
    parts = [oracle.grid_quantize(x.float().numpy(), 8, dim) for x in (K, V)]
    assert torch.equal(hat[0].cpu(), torch.from_numpy(oracle.cache_values(*parts[0]))
                       .to(torch.bfloat16))
    q = _q(1, 16, dim, 12)
    o1 = cache.attend(q.to(DEV), dev(table), dev(lengths))
    qs = q.expand(20, -1, -1).contiguous()
    o2 = cache.attend_shared(qs.to(DEV), dev(table[0]), 100, dev(np.zeros((20, 1), np.int32)),
                             dev(np.zeros(20, np.int32)))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0
    for h in range(16):
        args = [p[:, h // 2] for part in parts for p in part]
        for got, image in ((o1[0], False), (o2[0], True), (o2[19], True)):
            ref, tol = oracle.attend_bound(q[0, h].double().numpy(), *args, dim ** -0.5, image)
            assert np.all(np.abs(got[h].double().cpu().numpy() - ref) <= tol)


def test_slots_behind_a_sequence_hold_anything():
    """NaN scales and garbage past the end, and on pages that are not the sequence's."""
    host = HostCache(6, 2, 16, 128, 4, 128, seed=16)
    lengths, table = np.array([37], np.int32), np.array([[4, 0, 2, 5]], np.int32)
    for half in "kv":
        c, s, z = host.part[half]
        s[2, :, 5:] = np.nan
        s[[1, 3, 5]] = np.inf
        c[2, :, 5:] = 255 >> 4
    _run(host, lengths, [1], 2, table=table)


def test_not_finite_entries_reach_their_rows_only():
    host = HostCache(6, 1, 16, 128, 4, 64, seed=17)
    table = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    host.part["k"][1][2, 0, 3, 0] = np.nan        # sequence 1: a key
    host.part["v"][1][4, 0, 2, 1] = np.nan        # sequence 2: the upper half of a value
    lengths, starts = np.array([20, 20, 20], np.int32), np.arange(4, dtype=np.int32)
    q = _q(3, 2, 128, 3)
    out = host.device().attend(q.to(DEV), dev(table), dev(lengths), dev(starts))
    torch.cuda.synchronize()
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()
    assert torch.isfinite(out[2, :, :64]).all() and torch.isnan(out[2, :, 64:]).all()
    # before the entry, a row of the same sequence is whole
    out = host.device().attend(_q(18, 2, 128, 4).to(DEV), dev(table[1:2]), dev(lengths[:1]),
                               dev(np.array([0, 18], np.int32)))
    torch.cuda.synchronize()
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1:]).all()
    q[0, 1, 7] = float("nan")
    out = host.device().attend(q.to(DEV), dev(table), dev(lengths), dev(starts))
    torch.cuda.synchronize()
    assert torch.isfinite(out[0, 0]).all() and torch.isnan(out[0, 1]).all()


def test_strided_queries_and_outputs_and_padding():
    host = HostCache(8, 2, 16, 64, 4, 64, seed=18)
    lengths, starts = np.array([20, 33], np.int32), np.array([0, 2, 3], np.int32)
    table = make_table(lengths, 16, 8, 1)
    q = _q(6, 4, 64, 5)
    big = torch.zeros(6, 10, 64, dtype=torch.bfloat16, device=DEV)
    big[:, 3:7] = q.to(DEV)
    out = torch.full((6, 9, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    cache = host.device()
    assert cache.attend(big[:, 3:7], dev(table), dev(lengths), dev(starts),
                        out=out[:, 2:6]).data_ptr() == out[:, 2:6].data_ptr()
    torch.cuda.synchronize()
    check_attend(out[:, 2:6], host, table, lengths, starts, q, 0.125)
    assert torch.all(out[3:] == 7.0)                      # rows behind the last sequence
    assert torch.all(out[:, :2] == 7.0) and torch.all(out[:, 6:] == 7.0)


@pytest.mark.parametrize("table,lengths", [
    ([[0, 1], [9, 3]], [20, 20]), ([[0, 1], [-1, 3]], [20, 20]), ([[0, 1], [2, 3]], [20, 60]),
    ([[0, 1], [2, 3]], [20, -4]),
])
def test_positions_without_a_page_are_left_out(table, lengths):
    """The wrong pages of sequence 1 are not met, the status word says so, sequence 0 is whole."""
    host = HostCache(4, 1, 16, 64, 8, 64, seed=19)
    table, lengths = np.array(table, np.int32), np.array(lengths, np.int32)
    q = _q(2, 2, 64, 6)
    cache = host.device()
    out = cache.attend(q.to(DEV), dev(table), dev(lengths))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == _lib.GPTQ_INFO_BAD_PAGE
    check_attend(out[:1], host, table[:1], lengths[:1], [0, 1], q[:1], 0.125)
    assert torch.isfinite(out).all()
    if table[1, 0] != 2:           # page 3 holds positions 16 .. 19: the only ones left
        check_attend(out[1:], host, np.array([[3]]), [4], [0, 1], q[1:], 0.125)
    elif lengths[1] > 32:          # cut to the table
        check_attend(out[1:], host, table[1:], [32], [0, 1], q[1:], 0.125)
    else:
        assert torch.all(out[1] == 0)


def test_deterministic_and_independent_of_what_runs_beside():
    """The same call twice, and two calls at once on two streams."""
    host = HostCache(200, 4, 32, 128, 4, 128, seed=20)
    lengths = np.array([3000, 100, 1500, 900], np.int32)
    table = make_table(lengths, 32, 200, 2)
    q = _q(4, 16, 128, 7).to(DEV)
    cache, t, n = host.device(), dev(table), dev(lengths)
    first = cache.attend(q, t, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [cache.attend(q, t, n, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


def test_replayed_step_with_growing_lengths():
    """append + attend captured once, replayed over a sequence's first 40 tokens."""
    host = HostCache(8, 2, 16, 64, 8, 32, seed=21)
    cache = host.device()
    table = np.array([[3, 1, 6], [0, 5, 2]], np.int32)
    t, lengths = dev(table), dev(np.array([1, 1], np.int32))
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    q = _q(2, 4, 64, 8).to(DEV)
    cache.append(kv, kv, t, lengths)
    cache.attend(q, t, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(kv, kv, t, lengths)
        out = cache.attend(q, t, lengths)
    rng = np.random.default_rng(0)
    for n in range(1, 41):
        x = torch.from_numpy(rng.standard_normal((2, 2, 64)).astype(np.float32)).to(torch.bfloat16)
        kv.copy_(x)
        lengths.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        parts = oracle.grid_quantize(x.float().numpy(), 8, 32)
        for half in "kv":
            for b in range(2):
                for a, p in zip(host.part[half], parts):
                    a[table[b, (n - 1) // 16], :, (n - 1) % 16] = p[b]
        check_attend(out, host, table, [n, n], [0, 1, 2], q.cpu(), 0.125)
    assert int(cache.info.item()) == 0


# ------------------------------------------------------------------------------------------------
# a common prefix
# ------------------------------------------------------------------------------------------------
def _shared(host, prefix, lengths, news, ratio, seed=0, rows=None, scale=None, q=None):
    lengths = np.asarray(lengths, np.int32)
    starts = _starts(news)
    pages = host.part["k"][0].shape[0]
    k = -(-prefix // host.page)
    ptable = np.random.default_rng(seed).permutation(max(k, 1)).astype(np.int32)[:k]
    table = make_table(lengths, host.page, pages, seed, first=k)
    if q is None:
        q = _q(int(starts[-1]), host.heads * ratio, host.dim, seed + 1)
    cache = host.device()
    out = cache.attend_shared(q.to(DEV), dev(ptable), prefix, dev(table), dev(lengths), dev(starts),
                              scale=scale)
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0
    check_attend(out, host, table, lengths, starts, q,
                 host.dim ** -0.5 if scale is None else scale, prefix=(ptable, prefix),
                 image16=True, rows=rows)
    return out


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("batch,ratio", [(3, 1), (20, 3), (40, 8)])
def test_shared_formats(dim, bits, group, batch, ratio):
    host = HostCache(14 + 4 * batch, 2, 16, dim, bits, group, seed=dim + batch)
    lengths = (np.arange(batch) * 7) % 50 + 1
    _shared(host, 200, lengths, [1] * batch, ratio, rows={0, 1, batch // 2, batch - 1})


@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("page", [16, 128])
def test_shared_prefix_lengths(prefix, page):
    host = HostCache(-(-prefix // page) + 4, 1, page, 128, 4, 128, seed=prefix)
    _shared(host, prefix, [5, 1, 9], [1, 1, 2], 12)


def test_shared_rows_of_any_count():
    """Row counts around the row tiles, several tokens a sequence, sequences with none."""
    for batch, news, ratio in ((1, 1, 1), (33, 1, 4), (31, 1, 4), (16, 2, 8), (65, 1, 4), (9, 5, 7)):
        host = HostCache(40 + 2 * batch, 1, 16, 64, 4, 64, seed=batch)
        n = [news] * batch
        n[batch // 2] = 0 if batch > 1 else news
        _shared(host, 300, [news + b % 9 for b in range(batch)], n, ratio,
                rows={0, 1, sum(n) // 2, sum(n) - 1})


def test_shared_without_own_positions_or_prefix():
    """Own lengths of 0 meet the prefix alone; a prefix of 0 leaves plain attention; both: 0."""
    host = HostCache(20, 2, 16, 128, 8, 64, seed=30)
    _shared(host, 100, [0, 7, 0], [1, 1, 1], 4)
    out = _shared(host, 0, [0, 7, 40], [1, 2, 1], 4)
    assert torch.all(out[0] == 0)


def test_shared_many_rows_long_prefix():
    host = HostCache(110, 2, 64, 128, 4, 128, seed=31)
    _shared(host, 5000, [3] * 25, [1] * 25, 16, rows={0, 12, 24})


def test_shared_grids_that_span_the_range():
    host = HostCache(20, 1, 16, 128, 4, 32, seed=32, spread=12.0)
    host.part["k"] = HostCache(20, 1, 16, 128, 4, 32, seed=33).part["k"]
    _shared(host, 180, [20, 3], [1, 1], 4)
    host = HostCache(20, 1, 16, 64, 8, 64, seed=34)
    host.part["k"][1][:] *= np.float32(2.0 ** 40)
    _shared(host, 180, [20, 3], [1, 1], 4, scale=2.0 ** -43)


def test_shared_garbage_behind_the_prefix_and_not_finite_entries():
    host = HostCache(12, 1, 16, 128, 4, 64, seed=35)
    for half in "kv":
        host.part[half][1][7, :, 5:] = np.nan         # behind a prefix of 117 on pages 0 .. 7
    q, lengths = _q(2, 4, 128, 1), np.array([3, 4], np.int32)
    table = np.array([[9], [10]], np.int32)
    ptable = np.arange(8, dtype=np.int32)
    starts = [0, 1, 2]
    cache = host.device()
    out = cache.attend_shared(q.to(DEV), dev(ptable), 117, dev(table), dev(lengths))
    torch.cuda.synchronize()
    check_attend(out, host, table, lengths, starts, q, 128 ** -0.5, prefix=(ptable, 117),
                 image16=True)
    host.part["v"][1][3, 0, 2, 1] = np.nan
    out = host.device().attend_shared(q.to(DEV), dev(ptable), 117, dev(table), dev(lengths))
    torch.cuda.synchronize()
    assert torch.isfinite(out[:, :, :64]).all() and torch.isnan(out[:, :, 64:]).all()
    host.part["k"][1][9, 0, 1, 0] = np.nan            # an own key of sequence 0
    out = host.device().attend_shared(q.to(DEV), dev(ptable), 117, dev(table), dev(lengths))
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1, :, :64]).all()
    q[1, 2, 3] = float("inf")
    out = host.device().attend_shared(q.to(DEV), dev(ptable), 117, dev(table), dev(lengths))
    torch.cuda.synchronize()
    assert torch.isnan(out[1, 2]).all() and torch.isfinite(out[1, [0, 1, 3], :64]).all()


def test_shared_bad_pages_are_left_out():
    host = HostCache(12, 1, 16, 64, 4, 64, seed=36)
    q, lengths, table = _q(1, 4, 64, 2), np.array([3], np.int32), np.array([[9]], np.int32)
    cache = host.device()
    out = cache.attend_shared(q.to(DEV), dev(np.array([0, 50, 2, -1, 4], np.int32)), 75, dev(table),
                              dev(lengths))
    torch.cuda.synchronize()
    assert int(cache.info.item()) == _lib.GPTQ_INFO_BAD_PAGE
    # pages 0, 2 and 4 (11 positions) are met
    check_attend(out, host, table, lengths, [0, 1], q, 0.125,
                 prefix=(np.array([0, 2, 4], np.int32), 43), image16=True)


def test_shared_padding_determinism_and_refusals():
    host = HostCache(40, 2, 16, 128, 4, 128, seed=37)
    lengths, starts = np.array([20, 33], np.int32), np.array([0, 2, 3], np.int32)
    table, ptable = make_table(lengths, 16, 40, 1, first=20), np.arange(20, dtype=np.int32)
    q = _q(40, 8, 128, 5)
    cache = host.device()
    args = (dev(ptable), 310, dev(table), dev(lengths), dev(starts))
    outs = []
    for _ in range(2):
        out = torch.full((40, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        outs.append(cache.attend_shared(q.to(DEV), *args, out=out))
    torch.cuda.synchronize()
    assert torch.all(outs[0][3:] == 7.0) and torch.equal(outs[0], outs[1])
    check_attend(outs[0][:3], host, table, lengths, starts, q[:3], 128 ** -0.5,
                 prefix=(ptable, 310), image16=True)
    with pytest.raises(ValueError):
        cache.attend_shared(q.to(DEV), dev(ptable), 321, *args[2:])
    with pytest.raises(ValueError):
        cache.attend(q[:, :3].to(DEV), *args[2:])
    with pytest.raises(ValueError):
        cache.attend(q, *args[2:])                       # a host tensor


# ------------------------------------------------------------------------------------------------
# a step of a quantized layer
# ------------------------------------------------------------------------------------------------
def test_decode_steps_of_a_quantized_attention_layer():
    """The run of calls of a served layer: the fused projection from packed 4-bit weights, queries
    and keys rotated (which leaves q . k as it was), the new keys and values appended, attention over
    the cache, and, beside it, the same where the prompt is a prefix that two sequences share."""
    hidden, kv, ratio, dim, page = 512, 2, 2, 128, 16
    g = torch.Generator().manual_seed(40)
    rows = (kv * ratio + 2 * kv) * dim
    codes = torch.randint(0, 16, (rows, hidden), generator=g, dtype=torch.uint8)
    layer = api.QuantizedLayer(codes.to(DEV), torch.full((rows, 4), 0.02, device=DEV),
                               torch.full((rows, 4), 8, dtype=torch.uint8, device=DEV), None, None,
                               0)
    lin = api.pack_4bit(layer)

    def project(x):
        y = lin(x.to(DEV)).to(torch.bfloat16).reshape(-1, kv * ratio + 2 * kv, dim)
        q, k = y[:, :kv * ratio].contiguous(), y[:, kv * ratio:-kv].contiguous()
        return (api.rotate(q.view(-1, dim)).view(q.shape), api.rotate(k.view(-1, dim)).view(k.shape),
                y[:, -kv:])

    prompt = torch.randn(45, hidden, generator=g).to(torch.bfloat16)
    steps = [torch.randn(2, hidden, generator=g).to(torch.bfloat16) for _ in range(3)]
    cache = api.QuantizedCache(16, kv, dim, page, 4)
    table = np.array([[0, 1, 2, 3], [8, 9, 10, 11]], np.int32)
    own = np.array([[4], [12]], np.int32)
    q, k, v = project(prompt)
    for b in range(2):          # the prompt on both sequences' pages
        cache.append(k, v, dev(table[b:b + 1]), dev(np.array([45], np.int32)),
                     dev(np.array([0, 45], np.int32)))
    full = cache.attend(q, dev(table[:1]), dev(np.array([45], np.int32)),
                        dev(np.array([0, 45], np.int32)))
    held = {"k": [[], []], "v": [[], []]}
    for half, x in (("k", k), ("v", v)):
        for b in range(2):
            held[half][b].append(x.float().cpu().numpy())
    for n, x in enumerate(steps):
        q, k, v = project(x)
        lengths = dev(np.array([46 + n] * 2, np.int32))
        mine = dev(np.array([n + 1] * 2, np.int32))
        cache.append(k, v, dev(table), lengths)
        cache.append(k, v, dev(own), mine)
        a = cache.attend(q, dev(table), lengths)
        s = cache.attend_shared(q, dev(table[0, :3].copy()), 45, dev(own), mine)
        torch.cuda.synchronize()
        for b in range(2):
            for half, t in (("k", k), ("v", v)):
                held[half][b].append(t[b:b + 1].float().cpu().numpy())
            parts = {h: oracle.grid_quantize(np.concatenate(held[h][b]), 4, dim) for h in "kv"}
            for h in range(kv * ratio):
                args = [p[:, h // ratio] for half in "kv" for p in parts[half]]
                for got, image in ((a, False), (s, True)):
                    ref, tol = oracle.attend_bound(q[b, h].double().cpu().numpy(), *args,
                                                   dim ** -0.5, image)
                    assert np.all(np.abs(got[b, h].double().cpu().numpy() - ref) <= tol)
    assert int(cache.info.item()) == 0 and torch.isfinite(full).all()


def test_an_item_per_warp():
    """Enough sequences times heads for every warp of the device to work on its own: one, several
    and no tiles a sequence, items that two warps share, empty sequences between."""
    heads, batch = 24, 130
    rng = np.random.default_rng(5)
    lengths = rng.integers(1, 70, batch)
    lengths[[0, 7, 64, 129]] = [0, 300, 16, 250]
    news = np.ones(batch, int)
    news[[3, 50, 51]] = 0
    host = HostCache(int(sum(-(-n // 16) for n in lengths)) + 1, heads, 16, 64, 4, 32, seed=50)
    _run(host, lengths, news, 2, rows={0, 1, 6, 7, 60, 62, 100, 126})
    news = np.minimum(rng.integers(1, 4, batch), 3)
    _run(host, lengths, news, 2, rows={0, 1, 2, 14, 15, 100, 200})


# ------------------------------------------------------------------------------------------------
# calls at once, captured, replayed
# ------------------------------------------------------------------------------------------------
def _shared_call(seed, batch=40):
    """A cache and the arguments of a call over a prefix of up to 704 positions, met by more than 32
    rows."""
    host = HostCache(44 + 4 * batch, 2, 16, 128, 4, 64, seed=seed)
    lengths = ((np.arange(batch) * 11) % 50 + 1).astype(np.int32)
    ptable = np.random.default_rng(seed).permutation(44).astype(np.int32)
    table = make_table(lengths, 16, 44 + 4 * batch, seed, first=44)
    return host, ptable, table, lengths, _q(batch, 8, 128, seed)


def test_shared_calls_at_once_and_behind_one_another():
    """Calls on two streams at once, several behind one another on each, every one with a workspace
    of its own: each result is the one of a call alone. Tables of one page leave the sequences' own
    level one kernel, without a join in front of the prefix's."""
    calls = []
    for seed, batch, prefix in ((61, 40, 700), (62, 100, 130), (63, 33, 650)):
        host, ptable, table, lengths, q = _shared_call(seed, batch)
        if seed == 63:
            lengths, table = np.ones_like(lengths), table[:, :1].copy()
        cache = host.device()
        args = (q.to(DEV), dev(ptable), prefix, dev(table), dev(lengths))
        alone = cache.attend_shared(*args)
        torch.cuda.synchronize()
        check_attend(alone, host, table, lengths, np.arange(batch + 1), q, 128 ** -0.5,
                     prefix=(ptable, prefix), image16=True, rows={0, batch // 2, batch - 1})
        calls.append((cache, args, alone))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for k in range(4):
        for s in streams:
            for cache, args, alone in calls if s is streams[k % 2] else reversed(calls):
                outs.append((cache.attend_shared(*args, stream=s), alone))
    torch.cuda.synchronize()
    for out, alone in outs:
        assert torch.equal(out, alone)


def test_shared_step_replayed_with_new_queries_and_lengths():
    """append + attend_shared captured once; each replay equals the same calls made eagerly."""
    host, ptable, table, lengths, q = _shared_call(64)
    batch = len(lengths)
    caches = [host.device() for _ in range(2)]
    pt, t = dev(ptable), dev(np.where(table < 0, 0, table).astype(np.int32))
    n = dev(np.ones(batch, np.int32))
    kv = torch.zeros(batch, 2, 128, dtype=torch.bfloat16, device=DEV)
    qd = q.to(DEV)
    # each sequence on its first page only: 16 positions of its own
    t = t[:, :1].contiguous()

    def step(cache):
        cache.append(kv, kv, t, n)
        return cache.attend_shared(qd, pt, 700, t, n)
    step(caches[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0])
    g = torch.Generator().manual_seed(4)
    for length in (1, 2, 9, 16):
        kv.copy_(torch.randn(batch, 2, 128, generator=g))
        qd.copy_(torch.randn(batch, 8, 128, generator=g))
        n.fill_(length)
        for _ in range(2):                # the same step twice over: same codes, same result
            graph.replay()
        want = step(caches[1])
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(caches[0].k_codes, caches[1].k_codes)
    assert int(caches[0].info.item()) == 0 and int(caches[1].info.item()) == 0


def test_first_calls_of_a_process_under_capture():
    """Nothing has to run before a capture: a fresh process captures every call as its first."""
    import os
    import subprocess
    import sys
    code = """
import torch
from post_weight_quantization_12_b200 import api
dev = "cuda"
cache = api.QuantizedCache(64, 2, 128, 16, 4)
i32 = dict(dtype=torch.int32, device=dev)
table, lengths = torch.arange(20, 60, **i32)[:, None], torch.ones(40, **i32)
pt, starts = torch.arange(20, **i32), torch.tensor([0, 300], **i32)
x = torch.randn(40, 2, 128, device=dev).bfloat16()
pre = torch.randn(300, 2, 128, device=dev).bfloat16()
plen = torch.tensor([300], **i32)
q = torch.randn(40, 8, 128, device=dev).bfloat16()
torch.cuda.synchronize()
def step():
    cache.append(pre, pre, pt[None], plen, starts)
    cache.append(x, x, table, lengths)
    return (cache.attend(q, table, lengths), cache.attend_shared(q, pt, 300, table, lengths),
            cache.attend_shared(q[:4], pt, 300, table[:4], lengths[:4]), *cache.read(table, lengths))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
torch.cuda.synchronize()
eager = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
assert torch.isfinite(eager[1]).all() and int(cache.info.item()) == 0
print("as eager")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "as eager" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_shared_queries_that_are_not_finite_stay_in_their_row(bad):
    host, ptable, table, lengths, q = _shared_call(65)
    cache = host.device()
    args = (dev(ptable), 700, dev(table), dev(lengths))
    clean = cache.attend_shared(q.to(DEV), *args)
    q[3, 5, 17] = bad
    out = cache.attend_shared(q.to(DEV), *args)
    own = cache.attend(q.to(DEV), *args[2:])
    torch.cuda.synchronize()
    if math.isnan(bad):
        assert torch.isnan(out[3, 5]).all()
    clean[3, 5], out[3, 5] = 0, 0
    assert torch.equal(out, clean)
    own[3, 5] = 0
    assert torch.isfinite(own).all()


def test_one_row_cut_from_a_wider_tensor():
    """A single row whose tensor has an odd row stride, for queries, keys and outputs."""
    host = HostCache(4, 2, 16, 128, 4, 128, seed=66)
    cache, table, lengths = host.device(), np.array([[2, 1]], np.int32), np.array([20], np.int32)
    q = _q(1, 4, 128, 67)
    wide = torch.zeros(4 * 128 + 8, dtype=torch.bfloat16, device=DEV)
    odd = wide.as_strided((1, 4, 128), (4 * 128 + 3, 128, 1))
    odd.copy_(q)
    out = cache.attend(odd, dev(table), dev(lengths))
    torch.cuda.synchronize()
    check_attend(out, host, table, lengths, [0, 1], q, 128 ** -0.5)
    want = cache.attend(q.to(DEV), dev(table), dev(lengths))
    assert torch.equal(out, want)
