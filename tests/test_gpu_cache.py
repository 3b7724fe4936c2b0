"""Writing the quantized cache and reading it back, on the GPU, against the oracle: codes, scales and
zero points bit for bit, values exactly (or rounded once to bf16), and everything that a call must
leave alone."""
import numpy as np
import pytest
import torch

import oracle
from cache_util import DEV, HostCache, dev, make_table, words_of
from post_weight_quantization_12_b200 import _lib, api

pytestmark = pytest.mark.gpu

FORMATS = [(64, 4, 32), (64, 4, 64), (64, 8, 32), (64, 8, 64), (128, 4, 32), (128, 4, 64),
           (128, 4, 128), (128, 8, 32), (128, 8, 64), (128, 8, 128)]


def _starts(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


def _random_state(cache, seed):
    """Fills the cache's tensors with anything and returns copies."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    for h in "kv":
        for part in ("codes", "scales", "zeros"):
            t = getattr(cache, f"{h}_{part}")
            t.view(torch.uint8).random_(0, 256, generator=g) if t.dtype != torch.bfloat16 else \
                t.uniform_(0.5, 1, generator=g)
    return {f"{h}_{p}": getattr(cache, f"{h}_{p}").clone() for h in "kv"
            for p in ("codes", "scales", "zeros")}


def _expect(before, x, half, table, lengths, starts, page, bits, group):
    """The cache's tensors after x has been written over `before`."""
    q, s, z = oracle.grid_quantize(x, bits, group)
    out = {p: before[f"{half}_{p}"].cpu().clone() for p in ("codes", "scales", "zeros")}
    for b in range(len(lengths)):
        for i in range(starts[b], starts[b + 1]):
            pos = lengths[b] - starts[b + 1] + i
            at = (int(table[b, pos // page]), slice(None), pos % page)
            out["codes"][at] = words_of(q[i], bits)
            out["scales"][at] = torch.from_numpy(s[i]).to(torch.bfloat16)
            out["zeros"][at] = torch.from_numpy(z[i])
    return out, oracle.cache_values(q, s, z)


def _bits_equal(a, b):
    a, b = a.cpu(), b.cpu()
    if a.dtype == torch.bfloat16:      # NaN scales compare as NaN
        return torch.equal(torch.nan_to_num(a.float(), nan=-1), torch.nan_to_num(b.float(), nan=-1))
    return torch.equal(a, b)


def _check_append(cache, K, V, table, lengths, starts, hats=True, stream=None):
    before = _random_state(cache, 9)
    Kd, Vd = K.to(DEV), V.to(DEV)
    hat = [torch.full(K.shape, 7.0, dtype=K.dtype, device=DEV) for _ in range(2)] if hats \
        else [None, None]
    cache.append(Kd, Vd, dev(table), dev(lengths), None if starts is None else dev(starts),
                 K_hat=hat[0], V_hat=hat[1], stream=stream)
    torch.cuda.synchronize()
    st = np.arange(len(lengths) + 1) if starts is None else starts
    for half, x, h in (("k", K, hat[0]), ("v", V, hat[1])):
        want, vals = _expect(before, x.float().numpy(), half, table, lengths, st, cache.page,
                             cache.bits, cache.group)
        for part in ("codes", "scales", "zeros"):
            assert _bits_equal(getattr(cache, f"{half}_{part}"), want[part]), (half, part)
        if hats:
            n = st[-1]
            ref = torch.from_numpy(vals[:n]).to(K.dtype)
            assert torch.equal(torch.nan_to_num(h[:n].cpu(), nan=-5.0),
                               torch.nan_to_num(ref, nan=-5.0))
            assert torch.all(h[n:] == 7.0)
    return before


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_bit_exact(dim, bits, group, dtype):
    heads, page, news, past = 3, 16, [5, 1, 17, 33], [0, 15, 30, 7]
    lengths = np.array([p + n for p, n in zip(past, news)], np.int32)
    cache = api.QuantizedCache(20, heads, dim, page, bits, group)
    g = torch.Generator().manual_seed(dim + bits + group)
    K, V = (torch.randn(sum(news), heads, dim, generator=g) for _ in range(2))
    K *= torch.exp2(torch.randint(-20, 20, (sum(news), heads, 1), generator=g).float())
    _check_append(cache, K.to(dtype), V.to(dtype), make_table(lengths, page, 20, 1), lengths,
                  _starts(news))
    assert int(cache.info.item()) == 0


@pytest.mark.parametrize("heads,batch,page", [(1, 1, 32), (8, 70, 16), (2, 1100, 16), (5, 33, 64)])
def test_append_one_row_each(heads, batch, page):
    """A decode step: without starts, and the same with starts."""
    rng = np.random.default_rng(batch)
    lengths = rng.integers(1, 3 * page, batch).astype(np.int32)
    pages = 3 * batch
    table = make_table(lengths, page, pages, 2)
    g = torch.Generator().manual_seed(batch)
    K, V = (torch.randn(batch, heads, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    cache = api.QuantizedCache(pages, heads, 128, page, 4)
    _check_append(cache, K, V, table, lengths, None)
    _check_append(cache, K, V, table, lengths, np.arange(batch + 1, dtype=np.int32))
    assert int(cache.info.item()) == 0


def test_append_uneven_and_empty_sequences():
    """Sequences without new rows among the others, many of them, first and last too."""
    rng = np.random.default_rng(5)
    news = rng.integers(0, 4, 300)
    news[[0, 1, 50, 298, 299]] = 0
    news[120:200] = 0
    lengths = (news + rng.integers(0, 20, 300)).astype(np.int32)
    table = make_table(lengths, 16, 700, 3)
    g = torch.Generator().manual_seed(1)
    K, V = (torch.randn(int(news.sum()), 2, 64, generator=g) for _ in range(2))
    cache = api.QuantizedCache(700, 2, 64, 16, 8, 32)
    _check_append(cache, K, V, table, lengths, _starts(news), hats=False)
    assert int(cache.info.item()) == 0


def test_append_special_values():
    """Zero groups, constants, subnormals, values at the end of the range, NaN and infinities,
    quotients at half-integers."""
    x = torch.zeros(14, 1, 128)
    x[1] = 3.0
    x[2] = -2.5
    x[3, 0, ::2] = 1e-45
    x[4] = torch.linspace(-1e-40, 2e-40, 128)
    x[5] = torch.linspace(-1.6e38, 1.6e38, 128)
    x[6, 0, 5], x[6, 0, 9] = 3e38, -3e38                 # the step overflows
    x[7, 0, 17] = float("nan")
    x[8, 0, 80] = float("inf")
    x[9, 0, 31] = -float("inf")
    x[10] = (torch.arange(128) % 31 - 15) * 0.5           # s = 1 at 4 bits: ties to even
    x[11] = torch.arange(128).float() * 0.5 * 1.0
    x[12] = -x[11]
    x[13, 0, 3] = 3.3895313892515355e38                   # the largest bf16
    lengths, starts = np.array([14], np.int32), np.array([0, 14], np.int32)
    for bits in (4, 8):
        for group in (32, 64, 128):
            for dtype in (torch.float32, torch.bfloat16):
                cache = api.QuantizedCache(2, 1, 128, 16, bits, group)
                _check_append(cache, x.to(dtype), x.flip(0).to(dtype), np.array([[1]], np.int32),
                              lengths, starts)


def test_append_near_ties_match_the_division():
    """Quotients within a few ulps of half-integers, where x * (1 / s) and x / s part."""
    g = torch.Generator().manual_seed(11)
    k = torch.randint(-120, 120, (400, 2, 64), generator=g).float() + 0.5
    s = (torch.rand(400, 2, 1, generator=g) + 0.5)
    x = k * s
    x = torch.nextafter(x, x + torch.randint(-1, 2, x.shape, generator=g))
    lengths, starts = np.array([400], np.int32), np.array([0, 400], np.int32)
    cache = api.QuantizedCache(26, 2, 64, 16, 8, 32)
    _check_append(cache, x, -x, make_table(lengths, 16, 26, 0), lengths, starts)


def test_append_from_a_fused_projection():
    """K and V as column ranges of one [n, (q + 2 kv) dim] tensor."""
    n, heads, dim = 37, 4, 128
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(n, 16 + 2 * heads, dim, generator=g).to(torch.bfloat16).to(DEV)
    K, V = qkv[:, 16:16 + heads], qkv[:, 16 + heads:]
    lengths, starts = np.array([20, 30], np.int32), np.array([0, 20, 37], np.int32)
    table = make_table(lengths, 32, 4, 4)
    a, b = (api.QuantizedCache(4, heads, dim, 32) for _ in range(2))
    a.append(K, V, dev(table), dev(lengths), dev(starts))
    b.append(K.contiguous(), V.contiguous(), dev(table), dev(lengths), dev(starts))
    for part in ("k_codes", "v_codes", "k_scales", "v_scales", "k_zeros", "v_zeros"):
        assert torch.equal(getattr(a, part), getattr(b, part))
        assert torch.count_nonzero(getattr(a, part)) > 0


def test_append_in_place():
    """The stored values written over the dense inputs."""
    lengths, starts = np.array([40], np.int32), np.array([0, 40], np.int32)
    table = np.array([[1, 2, 0]], np.int32)
    g = torch.Generator().manual_seed(12)
    K, V = (torch.randn(40, 5, 64, generator=g) for _ in range(2))
    a, b = K.to(DEV), V.to(DEV)
    cache = api.QuantizedCache(3, 5, 64, 16, 4, 32)
    cache.append(a, b, dev(table), dev(lengths), dev(starts), K_hat=a, V_hat=b)
    torch.cuda.synchronize()
    for x, got in ((K, a), (V, b)):
        want = oracle.cache_values(*oracle.grid_quantize(x.numpy(), 4, 32))
        assert torch.equal(got.cpu(), torch.from_numpy(want).float())


def test_rows_behind_the_last_sequence_are_ignored():
    """A padded batch: rows from starts[batch] on change neither the cache nor the outputs."""
    lengths, starts = np.array([4, 9], np.int32), np.array([0, 3, 5], np.int32)
    g = torch.Generator().manual_seed(3)
    K, V = (torch.randn(50, 2, 64, generator=g) for _ in range(2))
    cache = api.QuantizedCache(3, 2, 64, 16, 4)
    _check_append(cache, K, V, np.array([[2], [0]], np.int32), lengths, starts)
    out = [torch.full((50, 2, 64), 7.0, device=DEV) for _ in range(2)]
    cache.read(dev(np.array([[2], [0]], np.int32)), dev(lengths), dev(starts), K_out=out[0],
               V_out=out[1])
    torch.cuda.synchronize()
    assert torch.all(out[0][5:] == 7.0) and torch.all(out[1][5:] == 7.0)
    assert torch.all(out[0][:5] != 7.0)
    assert int(cache.info.item()) == 0


@pytest.mark.parametrize("table,lengths", [
    ([[0], [7]], [3, 3]),            # a page past the cache
    ([[0], [-1]], [3, 3]),           # no page
    ([[0], [1]], [3, 40]),           # a position past the table
    ([[0], [1]], [3, 1]),            # more new rows than the sequence is long
    ([[0], [2 ** 31 - 1]], [3, 3]),
    ([[0], [1]], [3, 2 ** 31 - 1]),
    ([[0], [1]], [3, -5]),
])
def test_positions_without_a_page(table, lengths):
    """Sequence 1 is wrong: its rows are left out, the status word says so, sequence 0 is whole.
    (The lookups are bounds-checked in the kernels; nothing is read or written out of range.)"""
    table, lengths = np.array(table, np.int32), np.array(lengths, np.int32)
    starts = np.array([0, 2, 4], np.int32)
    cache = api.QuantizedCache(4, 1, 64, 16, 4)
    before = _random_state(cache, 1)
    g = torch.Generator().manual_seed(4)
    K = torch.randn(4, 1, 64, generator=g)
    hat = torch.full((4, 1, 64), 7.0, device=DEV)
    cache.append(K.to(DEV), K.to(DEV), dev(table), dev(lengths), dev(starts), K_hat=hat)
    torch.cuda.synchronize()
    assert int(cache.info.item()) == _lib.GPTQ_INFO_BAD_PAGE
    # the rows of sequence 1 that have a position in range are stored where it says
    ok1 = [i for i in (2, 3) if 0 <= lengths[1] - 4 + i < 16 and 0 <= table[1, 0] < 4]
    want, vals = before["k_codes"].cpu().clone(), None
    q, s, z = oracle.grid_quantize(K.numpy(), 4, 64)
    for i in (0, 1):
        want[0, :, 1 + i] = words_of(q[i], 4)
    for i in ok1:
        want[int(table[1, 0]), :, int(lengths[1]) - 4 + i] = words_of(q[i], 4)
    assert torch.equal(cache.k_codes.cpu(), want)
    assert torch.all(hat[:2] != 7.0)
    for i in (2, 3):
        if i not in ok1:
            assert torch.all(hat[i] == 7.0)
    cache.info.zero_()
    out, _ = cache.read(dev(table), dev(lengths), dev(starts), n=4, dtype=torch.float32)
    torch.cuda.synchronize()
    assert int(cache.info.item()) == _lib.GPTQ_INFO_BAD_PAGE
    for i in (2, 3):
        if i not in ok1:
            assert torch.all(out[i] == 0)
    assert torch.equal(out[:2], hat[:2])


@pytest.mark.parametrize("dim,bits,group", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_exact(dim, bits, group, dtype):
    heads, page = 3, 16
    host = HostCache(30, heads, page, dim, bits, group, seed=dim + group, spread=10.0)
    cache = host.device()
    lengths = np.array([50, 1, 0, 33, 100], np.int32)
    table = make_table(lengths, page, 30, 5)
    for news in (lengths, np.array([7, 1, 0, 33, 18])):    # whole sequences, and their ends
        starts = _starts(news)
        K, V = cache.read(dev(table), dev(lengths), dev(starts), n=int(starts[-1]), dtype=dtype)
        torch.cuda.synchronize()
        for half, got in (("k", K), ("v", V)):
            want = np.concatenate([np.stack([oracle.cache_values(
                *host.rows(half, table[b], lengths[b] - news[b], lengths[b], h))
                for h in range(heads)], 1) for b in range(5)])
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype))
    assert int(cache.info.item()) == 0


def test_read_one_half_and_empty():
    cache = HostCache(2, 1, 16, 64, 4, 64, 1).device()
    table, lengths = dev(np.array([[1]], np.int32)), dev(np.array([16], np.int32))
    K, V = cache.read(table, lengths)
    k = torch.empty_like(K)
    assert cache.read(table, lengths, K_out=k) == (k, None)
    torch.cuda.synchronize()
    assert torch.equal(k, K) and K.shape == (1, 1, 64)
    K, V = cache.read(table[:0], lengths[:0])
    assert K.shape == (0, 1, 64)
    cache.append(K, V, table[:0], lengths[:0])
    torch.cuda.synchronize()
    assert int(cache.info.item()) == 0


def test_write_then_read_on_another_stream_and_from_a_graph():
    """A captured step replayed with new lengths, and the same calls on a side stream."""
    heads, dim, page = 2, 128, 16
    cache = api.QuantizedCache(8, heads, dim, page, 8)
    table = dev(np.array([[3, 1], [0, 5]], np.int32))
    lengths = dev(np.array([1, 1], np.int32))
    g = torch.Generator().manual_seed(6)
    xs = [torch.randn(2, heads, dim, generator=g).to(torch.bfloat16).to(DEV) for _ in range(20)]
    K = xs[0].clone()
    out = torch.empty_like(K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.append(K, K, table, lengths, stream=side)          # warm-up before the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(K, K, table, lengths)
        cache.read(table, lengths, K_out=out)
    for step in range(20):
        K.copy_(xs[step])
        lengths.fill_(step + 1)
        graph.replay()
        torch.cuda.synchronize()
        q = oracle.cache_values(*oracle.grid_quantize(xs[step].float().cpu().numpy(), 8, dim))
        assert torch.equal(out.cpu(), torch.from_numpy(q).to(torch.bfloat16))
    starts = dev(np.array([0, 20, 40], np.int32))
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
    allK, _ = cache.read(table, lengths, starts, n=40, stream=side)
    side.synchronize()
    want = torch.stack([torch.from_numpy(oracle.cache_values(*oracle.grid_quantize(
        x.float().cpu().numpy(), 8, dim))).to(torch.bfloat16) for x in xs])     # [20, 2, h, d]
    assert torch.equal(allK.cpu(), want.transpose(0, 1).reshape(40, heads, dim))
