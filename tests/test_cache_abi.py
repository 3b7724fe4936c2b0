"""Refusals of the cache entry points: on the host, before anything is enqueued. No pointer given
here is ever dereferenced."""
import ctypes

import pytest
import torch

from post_weight_quantization_12_b200 import _lib, api

E, U, W, OK = (_lib.GPTQ_EINVAL, _lib.GPTQ_EUNSUPPORTED, _lib.GPTQ_EWORKSPACE, _lib.GPTQ_OK)
BF, F32 = _lib.GPTQ_BF16, _lib.GPTQ_FP32


def cache(**kw):
    d = dict(pages=4, heads=2, page=16, dim=128, bits=4, group=128)
    ptr = dict(k_codes=0x10000, k_scales=0x20000, k_zeros=0x30000, v_codes=0x40000,
               v_scales=0x50000, v_zeros=0x60000)
    for k, v in kw.items():
        (d if k in d else ptr)[k] = v
    return _lib.Cache(*ptr.values(), *d.values())


def rows(**kw):
    d = dict(table=0x70000, ld_table=4, width=4, lengths=0x71000, starts=0x72000, batch=3, n=5)
    d.update(kw)
    return _lib.CacheRows(*d.values())


def append(c=None, r=None, k=0x80000, ldk=256, v=0x90000, ldv=256, dtype=BF, kh=None, vh=None):
    return _lib.load().gptq_cache_append(c or cache(), r or rows(), k, ldk, v, ldv, dtype, kh, vh,
                                         None, None)


def read(c=None, r=None, k=0x80000, v=0x90000, dtype=BF):
    return _lib.load().gptq_cache_read(c or cache(), r or rows(), k, v, dtype, None, None)


def attend(c=None, r=None, q=0x80000, ldq=512, ratio=2, scale=0.1, out=0x90000, ldo=512,
           ws=0x100000, size=1 << 40, prefix=None):
    lib = _lib.load()
    tail = (q, ldq, ratio, scale, out, ldo, ws, size, None, None)
    if prefix is None:
        return lib.gptq_cache_attend(c or cache(), r or rows(), *tail)
    return lib.gptq_cache_attend_shared(c or cache(), r or rows(), *prefix, *tail)


CALLS = [append, read, attend, lambda **kw: attend(prefix=(0xA0000, 100), **kw)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,st", [
    (dict(dim=96, group=96), U), (dict(dim=256), U), (dict(group=48), E), (dict(group=16), U),
    (dict(bits=3), U), (dict(bits=16), U), (dict(page=8), U), (dict(page=48), U),
    (dict(page=65536), U), (dict(page=0), E), (dict(pages=0), E), (dict(heads=0), E),
    (dict(heads=1 << 17), U), (dict(pages=1 << 40), U), (dict(k_codes=None), E),
    (dict(v_zeros=None), E), (dict(k_scales=0x20008), E), (dict(v_codes=0x10000), E),
    (dict(dim=0), E), (dict(group=0), E),
])
def test_bad_caches(built_lib, call, kw, st):
    assert call(c=cache(**kw)) == st


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,st", [
    (dict(n=-1), E), (dict(batch=-1), E), (dict(width=-1), E), (dict(ld_table=3), E),
    (dict(starts=None), E),                          # 5 rows of 3 sequences need starts
    (dict(lengths=None), E), (dict(table=None), E), (dict(table=0x70002), E),
    (dict(n=1 << 40), U), (dict(batch=1 << 33), U), (dict(n=0), OK), (dict(batch=0), OK),
    (dict(n=0, table=None, lengths=None, starts=None), OK),
])
def test_bad_rows(built_lib, call, kw, st):
    assert call(r=rows(**kw)) == st


def test_bad_tensors(built_lib):
    assert append(k=None) == E and append(v=None) == E
    assert append(ldk=128) == E and append(ldv=252) == E and append(ldk=260) == E
    assert append(dtype=7) == E and append(k=0x80008) == E and append(kh=0x80008) == E
    # in place only if dense; outputs distinct from everything else
    assert append(k=0x80000, kh=0x80000, ldk=512) == E
    assert append(kh=0xB0000, vh=0xB0000) == E and append(kh=0x90000) == E
    assert append(vh=0x80000) == E and read(k=0x80000, v=0x80000) == E
    assert attend(c=cache(heads=1024), ratio=512, ldq=1 << 27, ldo=1 << 27) == U
    assert attend(r=rows(n=1 << 22), ratio=1000, ldq=1 << 20, ldo=1 << 20) == U
    assert read(k=None, v=None) == E and read(dtype=9) == E and read(k=0x80004) == E
    assert attend(q=None) == E and attend(out=None) == E and attend(q=0x90000) == E
    assert attend(ldq=256) == E and attend(ldo=514) == E and attend(ratio=0) == E
    assert attend(ratio=2000) == E and attend(scale=float("nan")) == E
    assert attend(scale=float("inf")) == E
    assert attend(ws=None) == W and attend(ws=0x100080) == W and attend(size=1000) == W
    assert attend(prefix=(0xA0000, -1)) == E and attend(prefix=(None, 10)) == E
    assert attend(prefix=(0xA0000, 1 << 31)) == U


def test_workspace_size(built_lib):
    c = cache()
    plain, shared = (_lib.cache_workspace_size(c, 64, 4, s) for s in (0, 1))
    assert plain > 0 and plain % 256 == 0
    assert shared >= plain + 64 * 8 * (128 + 1) * 4
    assert _lib.cache_workspace_size(cache(bits=5), 64, 4, 0) == 0
    assert _lib.cache_workspace_size(c, -1, 4, 0) == 0
    assert _lib.cache_workspace_size(c, 1, 0, 0) == 0


def test_status_of_a_bad_page(built_lib):
    assert _lib.info_status(_lib.GPTQ_INFO_BAD_PAGE) == E


def _cpu_tensors(**kw):
    t = dict(k_codes=torch.zeros(3, 2, 16, 16, dtype=torch.int32),
             k_scales=torch.zeros(3, 2, 16, 1, dtype=torch.bfloat16),
             k_zeros=torch.zeros(3, 2, 16, 1, dtype=torch.uint8))
    t.update({"v" + k[1:]: v.clone() for k, v in list(t.items())})
    t.update(kw)
    return t


@pytest.mark.parametrize("kw", [
    dict(v_codes=torch.zeros(3, 2, 16, 32, dtype=torch.int32)),
    dict(k_scales=torch.zeros(3, 2, 16, 1)),
    dict(v_zeros=torch.zeros(3, 2, 16, 2, dtype=torch.uint8)),
    dict(k_codes=torch.zeros(3, 2, 16, 16, dtype=torch.int32).transpose(0, 1)),
    dict(k_codes=torch.zeros(3, 16, 16, dtype=torch.int32)),
])
def test_of_tensors_refuses(kw):
    with pytest.raises(ValueError):
        api.QuantizedCache.of_tensors(**_cpu_tensors(**kw), dim=128)


def test_of_tensors_tells_the_format():
    c = api.QuantizedCache.of_tensors(**_cpu_tensors(), dim=128)
    assert (c.bits, c.group, c.page, c.heads, c.pages) == (4, 128, 16, 2, 3)
    c = api.QuantizedCache.of_tensors(**_cpu_tensors(), dim=64)
    assert (c.bits, c.group) == (8, 64)
    with pytest.raises(ValueError):
        api.QuantizedCache.of_tensors(**_cpu_tensors(), dim=96)
    with pytest.raises(ValueError):
        api.QuantizedCache(4, 2, 128, group=48, device="cpu")
    with pytest.raises(ValueError):
        api.QuantizedCache(4, 2, 128, bits=3, device="cpu")


def test_marshalling_refuses():
    c, i32 = cache(), torch.int32
    table, lengths = torch.zeros(3, 4, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(TypeError):
        _lib.cache_rows(3, table.long(), lengths, None)
    with pytest.raises(TypeError):
        _lib.cache_rows(3, table, lengths.float(), None)
    with pytest.raises(ValueError):
        _lib.cache_rows(3, table, lengths[:2], None)
    with pytest.raises(ValueError):
        _lib.cache_rows(3, table, lengths, torch.zeros(3, dtype=i32))
    r = _lib.cache_rows(3, table, lengths, None)
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _lib.cache_append(c, r, x, x[:2])
    with pytest.raises(ValueError):
        _lib.cache_append(c, r, x, x.float())
    with pytest.raises(ValueError):
        _lib.cache_append(c, r, x[:, :1], x[:, :1])
    with pytest.raises(ValueError):
        _lib.cache_append(c, r, x, x, K_hat=x.float())
    with pytest.raises(ValueError):
        _lib.cache_append(c, r, x.transpose(0, 1).contiguous().transpose(0, 1), x)
    with pytest.raises(TypeError):
        _lib.cache_append(c, r, x.half(), x.half())
    with pytest.raises(ValueError):
        _lib.cache_read(c, r, None, None)
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(TypeError):
        _lib.cache_attend(c, r, x.float(), x.float(), 1, 0.1, ws)
    with pytest.raises(ValueError):
        _lib.cache_attend(c, r, x, x[:2], 1, 0.1, ws)


def test_structs_match_the_header():
    """Field for field, in the header's order."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "gptq.h")).read(), flags=re.S)
    for name, struct in (("gptq_cache", _lib.Cache), ("gptq_cache_rows", _lib.CacheRows)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = []
        for decl in body.split(";"):
            decl = decl.strip()
            if decl:
                first, *rest = decl.split(",")
                fields += [re.findall(r"(\w+)$", f.strip())[0] for f in [first, *rest]]
        assert [f.replace("_dev", "") for f in fields] == [f for f, _ in struct._fields_]
    assert ctypes.sizeof(_lib.Cache) == 6 * 8 + 8 + 5 * 4 + 4


def test_one_row_has_the_stride_of_its_width():
    """A single row cut from any tensor: its row stride says nothing and is not passed on."""
    base = torch.zeros(7 * 300 + 1, dtype=torch.bfloat16)
    for stride in (1, 256, 301, 2048):
        x = base.as_strided((1, 2, 128), (stride, 128, 1))
        assert _lib._heads_ld(x, "x", 2, 128) == 256
    assert _lib._heads_ld(base.as_strided((3, 2, 128), (264, 128, 1)), "x", 2, 128) == 264


def test_no_workspace_size_for_refused_calls(built_lib):
    """Shapes that the attention calls refuse have no size; the largest that they take have one that
    fits in 64 bits."""
    size = _lib.cache_workspace_size
    for shared in (0, 1):
        assert size(cache(heads=1 << 16), (1 << 31) - 1, 1024, shared) == 0
        assert size(cache(heads=1024), 5, 512, shared) == 0
        assert size(cache(), 1 << 22, 1000, shared) == 0
        assert size(cache(), 1 << 30, 1, shared) > 0
    n, ratio, heads = (1 << 31) // 1024 - 1, 1024, 256
    assert size(cache(heads=heads), n, ratio, 1) > n * ratio * heads * 128 * 4
