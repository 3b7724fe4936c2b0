"""The measured cases of the quantized key/value cache: writing it, reading it back, and the
attention of decode steps over it, each in a plain form and as the package's own calls.

The cache holds one k-bit grid per (token, head, group of `group` head dimensions), asymmetric like
the layer quantizer's: codes q, a scale s and a zero point z, standing for s (q - z). It is paged:
position p of sequence b is token p % page of page table[b][p // page]. A call works on `n` rows;
rows starts[b] .. starts[b + 1] - 1 belong to sequence b and sit at its last positions, the last one
at lengths[b] - 1.

  append   quantizes K and V rows as they are written; returns what the cache now stands for
  read     returns the values of the last positions of every sequence
  attend   softmax attention of the rows' queries over their own sequence up to their position
  shared   the same where every sequence continues one common prefix, held once
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, new=1, ragged=False, past_lo=0, past_hi=0, prefix=0,
             heads=8, ratio=4, dim=128, bits=4, group=128, page=64, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a small batch: one token's K and V per sequence, the latency case
        _case("append_step", "append", batch=16, new=1, past_lo=40, past_hi=4000),
        # prompts of a batch entering the cache: a bandwidth case
        _case("append_prompts", "append", batch=4, new=16384, ragged=True, page=128),
        # 8-bit codes, narrow heads, fine groups, fp32 inputs, pages that end anywhere
        _case("append_fp32_8bit", "append", batch=3, new=1237, ragged=True, past_lo=5, past_hi=77,
              heads=12, dim=64, bits=8, group=32, page=16, dtype="fp32"),
        # one sequence copied out of the cache, e.g. to move it elsewhere
        _case("read_one", "read", new=777, heads=8),
        # a whole batch read back at once
        _case("read_batch", "read", batch=16, new=8192, ragged=True, page=128),
        # a chat turn just begun: the smallest attention call
        _case("attend_short", "attend", past_lo=36, past_hi=36, heads=32, ratio=1),
        # a decode step of a serving batch whose sequences differ in length
        _case("attend_batch", "attend", batch=32, past_lo=100, past_hi=16000),
        # one sequence with a long context, 8-bit codes: the work must be split along it
        _case("attend_long", "attend", past_lo=131071, past_hi=131071, bits=8, page=128),
        # several tokens a sequence checked at once, narrow heads with fine groups
        _case("attend_several", "attend", batch=8, new=4, past_lo=900, past_hi=5000, heads=32,
              ratio=1, dim=64, bits=8, group=32, page=16),
        # a few requests that share an instruction of a thousand tokens
        _case("shared_few", "shared", batch=8, prefix=1000, past_lo=3, past_hi=64),
        # many samples of one long document, 4-bit codes
        _case("shared_document", "shared", batch=128, prefix=32768, past_lo=16, past_hi=500,
              page=128),
        # as many key heads as query heads and 8-bit codes: fewer rows meet each prefix byte
        _case("shared_full_heads", "shared", batch=96, prefix=8192, past_lo=1, past_hi=300, heads=32,
              ratio=1, bits=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_MOST = {}


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "shared", "shared"])
    if not _MOST:
        for c in listed():
            w = work(c)
            m = _MOST.setdefault(c["op"], {"bytes": 0, "flops": 0})
            m["bytes"], m["flops"] = max(m["bytes"], w["bytes"]), max(m["flops"], w["flops"])
    while True:
        dim = rng.choice([64, 128])
        c = _case("", op, heads=_log(rng, 1, 32), dim=dim, bits=rng.choice([4, 8]),
                  group=rng.choice([g for g in (32, 64, 128) if g <= dim]),
                  page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7,
                  ratio=rng.choice([1, 2, 3, 4, 5, 7, 8, 12]))
        if op in ("append", "read"):
            c.update(batch=_log(rng, 1, 64), new=_log(rng, 1, 16384), past_lo=rng.randint(0, 50),
                     past_hi=rng.randint(50, 2000), dtype=rng.choice(["bf16", "bf16", "fp32"]))
        else:
            hi = _log(rng, 16, 131072 if op == "attend" else 600)
            c.update(batch=_log(rng, 1, 96), new=rng.choice([1, 1, 1, 2, 3, 5]), past_hi=hi,
                     past_lo=rng.randint(0, hi))
            if op == "shared":
                c["prefix"] = _log(rng, 64, 32768)
        w, m = work(c), _MOST[op]
        # the padded intermediates of the plain form stay within a few GB
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and _padded(c) <= 1 << 30:
            del c["name"]
            return c


def _padded(c):
    """Values of K that the plain form holds at once, each sequence padded to the longest."""
    if c["op"] in ("append", "read"):
        return 0
    per = c["heads"] * max(c["dim"], c["ratio"] * c["new"])
    return per * (c["batch"] * (c["past_hi"] + c["new"]) + c["prefix"])


def _spread(lo, hi, batch):
    """Lengths from lo to hi in a mixed order: the same for every seed."""
    return [lo + ((hi - lo) * ((7 * b) % batch)) // max(1, batch - 1) for b in range(batch)]


def _sizes(c):
    """(new rows, length after them) of every sequence."""
    news = [c["new"]] * c["batch"]
    if c["ragged"]:
        news = [max(1, c["new"] - (c["new"] * ((5 * b) % c["batch"])) // (2 * c["batch"]))
                for b in range(c["batch"])]
    past = _spread(c["past_lo"], c["past_hi"], c["batch"])
    return news, [p + n for p, n in zip(past, news)]


def work(case):
    news, lens = _sizes(case)
    n, H, D = sum(news), case["heads"], case["dim"]
    # stored bytes of K and V of one token: the codes, a 2-byte scale and a 1-byte zero per group
    token = 2 * H * (D * case["bits"] // 8 + 3 * (D // case["group"]))
    if case["op"] == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (token + 2 * H * D * (e + e)), "flops": 2 * n * H * D * 8}
    if case["op"] == "read":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (token + 2 * H * D * e), "flops": 2 * n * H * D * 2}
    # every row meets the prefix and its own sequence up to its position
    pairs = sum(m * (case["prefix"] + L) - m * (m - 1) // 2 for m, L in zip(news, lens))
    io = 2 * n * H * case["ratio"] * D * 2
    return {"bytes": (case["prefix"] + sum(lens)) * token + io,
            "flops": 4 * pairs * H * case["ratio"] * D}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _grid_values(x, bits, group):
    """Codes, scales and zero points of x [..., D] (fp32), in elementary fp32 operations: the grid
    spans [min(0, min), max(0, max)] of a group, its step rounded up to bfloat16; a group whose step
    is zero takes [-1, 1]; one with a value that is not finite (or whose step is not) has a NaN
    scale and zero codes."""
    v = x.reshape(*x.shape[:-1], -1, group)
    top = torch.full((), float(2 ** bits - 1), device=x.device)
    ok = torch.isfinite(v).all(-1)
    lo = torch.clamp(v.amin(-1), max=0.0)
    hi = torch.clamp(v.amax(-1), min=0.0)
    step = (hi - lo) / top
    flat = step == 0
    lo = torch.where(flat, torch.full_like(lo, -1.0), lo)
    step = torch.where(flat, torch.full_like(step, 2.0) / top, step)
    s = ((step.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
    ok = ok & torch.isfinite(s)
    z = torch.clamp(torch.round(-lo / s), min=0.0).minimum(top)
    q = torch.clamp(torch.round(v / s[..., None]) + z[..., None], min=0.0).minimum(top)
    s = torch.where(ok, s, torch.full_like(s, float("nan")))
    z = torch.where(ok, z, torch.zeros_like(z))
    q = torch.where(ok[..., None], q, torch.zeros_like(q))
    return q.reshape(x.shape), s, z


def _pack(q, bits):
    """fp32 codes [..., D] -> int32 words, code c of a word in bits bits * c and up."""
    per = 32 // bits
    w = q.to(torch.int64).reshape(*q.shape[:-1], -1, per)
    shift = torch.arange(0, 32, bits, device=q.device)
    w = (w << shift).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _unpack(words, bits):
    shift = torch.arange(0, 32, bits, device=words.device, dtype=torch.int32)
    q = (words[..., None] >> shift) & (2 ** bits - 1)
    return q.reshape(*words.shape[:-1], -1)


def _normal(shape, g, channels):
    """N(0, 1) with a few head dimensions larger than the rest, as keys have them."""
    x = torch.randn(shape, generator=g, device=DEV)
    return x if channels is None else x * channels


def _paged(c, g):
    """Inputs that every operator has: the page tables, lengths, starts and the cache's tensors,
    filled for what the operator reads."""
    news, lens = _sizes(c)
    P, H, D, B = c["page"], c["heads"], c["dim"], c["batch"]
    own_pages = [-(-L // P) for L in lens]
    prefix_pages = -(-c["prefix"] // P)
    pages = sum(own_pages) + prefix_pages + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.zeros(B, max(own_pages) + 1, dtype=torch.int32)
    at = prefix_pages
    for b, k in enumerate(own_pages):
        table[b, :k] = order[at:at + k]
        at += k
    starts = torch.zeros(B + 1, dtype=torch.int32)
    starts[1:] = torch.cumsum(torch.tensor(news), 0)
    s = dict(case=c, table=table.to(DEV), lengths=torch.tensor(lens, dtype=torch.int32, device=DEV),
             starts=starts.to(DEV), longest=max(lens), most=max(news),
             prefix_table=order[:prefix_pages].to(DEV))
    channels = torch.ones(D, device=DEV)
    channels[torch.randperm(D, generator=g, device=DEV)[:max(1, D // 32)]] = 4.0
    G = D // c["group"]
    if c["op"] == "append":
        for k in "kv":
            s[k + "_codes"] = torch.zeros(pages, H, P, D * c["bits"] // 32, dtype=torch.int32,
                                          device=DEV)
            s[k + "_scales"] = torch.zeros(pages, H, P, G, dtype=torch.bfloat16, device=DEV)
            s[k + "_zeros"] = torch.zeros(pages, H, P, G, dtype=torch.uint8, device=DEV)
        return s, channels
    for k in "kv":
        x = _normal((pages, H, P, D), g, channels if k == "k" else None)
        q, sc, z = _grid_values(x, c["bits"], c["group"])
        del x
        s[k + "_codes"] = _pack(q, c["bits"])
        s[k + "_scales"], s[k + "_zeros"] = sc.to(torch.bfloat16), z.to(torch.uint8)
    return s, channels


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s, channels = _paged(case, g)
    news, _ = _sizes(case)
    n, H, D = sum(news), case["heads"], case["dim"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "append":
        s["K"] = _normal((n, H, D), g, channels).to(dt)
        s["V"] = _normal((n, H, D), g, None).to(dt)
        s["K_hat"], s["V_hat"] = torch.empty_like(s["K"]), torch.empty_like(s["V"])
    elif case["op"] == "read":
        s["K_hat"] = torch.empty(n, H, D, dtype=dt, device=DEV)
        s["V_hat"] = torch.empty_like(s["K_hat"])
    else:
        s["Q"] = torch.randn(n, H * case["ratio"], D, generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["Q"])
    if own:
        from post_weight_quantization_12_b200 import api
        s["cache"] = api.QuantizedCache.of_tensors(
            s["k_codes"], s["k_scales"], s["k_zeros"], s["v_codes"], s["v_scales"], s["v_zeros"],
            dim=case["dim"])
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def _rows(s, n):
    """Sequence and position of every row."""
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(s["starts"][1:].long(), row, right=True)
    pos = s["lengths"][seq].long() - s["starts"][seq + 1].long() + row
    return seq, pos


def _slots(s, seq, pos):
    """(page, token) of positions of sequences."""
    P = s["case"]["page"]
    return s["table"][seq, pos // P].long(), pos % P


def _values(s, which, page, token):
    """fp32 values [..., heads, dim] of cached tokens."""
    c = s["case"]
    q = _unpack(s[which + "_codes"][page, :, token], c["bits"]).float()
    sc = s[which + "_scales"][page, :, token].float()
    z = s[which + "_zeros"][page, :, token].float()
    v = q.reshape(*sc.shape, c["group"])
    return (sc[..., None] * (v - z[..., None])).reshape(q.shape)


def _plain_append(s):
    c = s["case"]
    page, token = _slots(s, *_rows(s, s["K"].shape[0]))
    for which, x, hat in (("k", s["K"], s["K_hat"]), ("v", s["V"], s["V_hat"])):
        q, sc, z = _grid_values(x.float(), c["bits"], c["group"])
        s[which + "_codes"][page, :, token] = _pack(q, c["bits"])
        s[which + "_scales"][page, :, token] = sc.to(torch.bfloat16)
        s[which + "_zeros"][page, :, token] = z.to(torch.uint8)
        v = q.reshape(*sc.shape, c["group"])
        hat.copy_((sc[..., None] * (v - z[..., None])).reshape(q.shape))
    return s["K_hat"], s["V_hat"]


def _plain_read(s):
    page, token = _slots(s, *_rows(s, s["K_hat"].shape[0]))
    for which, hat in (("k", s["K_hat"]), ("v", s["V_hat"])):
        hat.copy_(_values(s, which, page, token))
    return s["K_hat"], s["V_hat"]


def _plain_attend(s):
    """Attention with every sequence padded to the longest one, in fp32."""
    c = s["case"]
    H, R, D, B, M = c["heads"], c["ratio"], c["dim"], c["batch"], s["most"]
    dev = s["Q"].device
    # rows padded to M per sequence, [B, H, M R, D]
    j = torch.arange(M, device=dev)
    starts, lengths = s["starts"].long(), s["lengths"].long()
    count = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + j).clamp(max=s["Q"].shape[0] - 1)
    q = s["Q"][row].float().reshape(B, M, H, R, D).transpose(1, 2).reshape(B, H, M * R, D)
    # own positions, [B, L]
    p = torch.arange(s["longest"], device=dev)
    page = s["table"][:, p // c["page"]].long()
    token = (p % c["page"]).expand(B, -1)
    k = _values(s, "k", page, token).permute(0, 2, 3, 1)
    x = torch.matmul(q, k).reshape(B, H, M, R, -1) / math.sqrt(D)
    del k
    at = lengths[:, None] - count[:, None] + j                        # [B, M] the rows' positions
    x = x.masked_fill((p > at[:, :, None])[:, None, :, None], -math.inf)
    v = _values(s, "v", page, token).transpose(1, 2)
    if c["prefix"]:
        pp = torch.arange(c["prefix"], device=dev)
        ppage, ptoken = s["prefix_table"][pp // c["page"]].long(), pp % c["page"]
        qa = q.transpose(0, 1).reshape(H, B * M * R, D)
        y = torch.matmul(qa, _values(s, "k", ppage, ptoken).permute(1, 2, 0)) / math.sqrt(D)
        y = y.reshape(H, B, M, R, -1).transpose(0, 1)
        top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
        x, y = torch.exp(x - top), torch.exp(y - top)
        total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
        o = torch.matmul(x.reshape(B, H, M * R, -1), v).reshape(B, H, M, R, D)
        ya = y.transpose(0, 1).reshape(H, B * M * R, -1)
        del x, y
        pv = torch.matmul(ya, _values(s, "v", ppage, ptoken).transpose(0, 1))
        o = (o + pv.reshape(H, B, M, R, D).transpose(0, 1)) / total
    else:
        x = torch.exp(x - x.amax(-1, keepdim=True))
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x.reshape(B, H, M * R, -1), v).reshape(B, H, M, R, D) / total
    o = o.transpose(1, 2).reshape(B, M, H * R, D)
    s["out"].copy_(o[(j < count[:, None])])
    return s["out"]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        return _plain_read(s) if op == "read" else _plain_attend(s)
    cache = s["cache"]
    if op == "append":
        cache.append(s["K"], s["V"], s["table"], s["lengths"], s["starts"], K_hat=s["K_hat"],
                     V_hat=s["V_hat"])
        return s["K_hat"], s["V_hat"]
    if op == "read":
        return cache.read(s["table"], s["lengths"], s["starts"], K_out=s["K_hat"],
                          V_out=s["V_hat"])
    if op == "attend":
        return cache.attend(s["Q"], s["table"], s["lengths"], s["starts"], out=s["out"])
    return cache.attend_shared(s["Q"], s["prefix_table"], s["case"]["prefix"], s["table"],
                               s["lengths"], s["starts"], out=s["out"])


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _f32(x):
    """Rounds once to fp32. A quotient of two fp32 numbers taken in 64 bits first keeps its value."""
    return x.to(torch.float32).double()


def _stands_for(x, bits, group):
    """s (q - z) of each value of x (fp64 holding fp32 values), each step as the grid defines it."""
    rows = x.reshape(-1, group)
    top = float(2 ** bits - 1)
    zero = torch.zeros(rows.shape[0], 1, dtype=torch.float64, device=x.device)
    both = torch.cat([rows, zero], 1)
    lo, hi = both.min(1, keepdim=True).values, both.max(1, keepdim=True).values
    step = _f32(_f32(hi - lo) / top)
    lo = torch.where(step > 0, lo, -torch.ones_like(lo))
    step = torch.where(step > 0, step, _f32(torch.full_like(step, 2.0) / top))
    near = step.to(torch.bfloat16).double()                 # nearest, then up where it fell short
    ulp = torch.exp2(torch.floor(torch.log2(near.clamp(min=2.0 ** -126))) - 7)
    s = torch.where(near < step, near + ulp, near)
    z = torch.round(_f32(-lo / s)).clamp(0, top)
    q = (torch.round(_f32(rows / s)) + z).clamp(0, top)
    return (s * (q - z)).reshape(x.shape)


def _stored(s, which, seq_table, L):
    """fp64 values [heads, L, dim] of the first L positions behind one row of a page table."""
    c = s["case"]
    pages = seq_table[:-(-L // c["page"])].long()
    words = s[which + "_codes"][pages].transpose(0, 1).flatten(1, 2)[:, :L]
    scale = s[which + "_scales"][pages].transpose(0, 1).flatten(1, 2)[:, :L].double()
    zero = s[which + "_zeros"][pages].transpose(0, 1).flatten(1, 2)[:, :L].double()
    byte = words.contiguous().view(torch.uint8)
    if c["bits"] == 4:
        byte = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    group = torch.arange(c["dim"], device=byte.device) // c["group"]
    return scale[..., group] * (byte.double() - zero[..., group])


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "append":
        return tuple(_stands_for(x.double(), c["bits"], c["group"]) for x in (s["K"], s["V"]))
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    if c["op"] == "read":
        return tuple(torch.cat([_stored(s, w, s["table"][b], lengths[b])
                                [:, lengths[b] - (starts[b + 1] - starts[b]):].transpose(0, 1)
                                for b in range(c["batch"])]) for w in "kv")
    if c["prefix"]:
        pk, pv = (_stored(s, w, s["prefix_table"], c["prefix"]) for w in "kv")
    outs = []
    for b in range(c["batch"]):
        L, m = lengths[b], starts[b + 1] - starts[b]
        k, v = (_stored(s, w, s["table"][b], L) for w in "kv")
        q = s["Q"][starts[b]:starts[b + 1]].double()
        q = q.reshape(m, c["heads"], c["ratio"], c["dim"]).permute(1, 0, 2, 3)
        x = torch.einsum("hmrd,hld->hmrl", q, k) * c["dim"] ** -0.5
        i = torch.arange(m, device=x.device)[:, None]
        x[:, (torch.arange(L, device=x.device) > L - m + i)[:, None].expand(-1, c["ratio"], -1)] \
            = -math.inf
        if c["prefix"]:
            x = torch.cat([torch.einsum("hmrd,hld->hmrl", q, pk) * c["dim"] ** -0.5, x], -1)
        a = torch.softmax(x, -1)
        o = torch.einsum("hmrl,hld->hmrd", a[..., c["prefix"]:], v)
        if c["prefix"]:
            o = o + torch.einsum("hmrl,hld->hmrd", a[..., :c["prefix"]], pv)
        outs.append(o.permute(1, 0, 2, 3).reshape(m, c["heads"] * c["ratio"], c["dim"]))
    return torch.cat(outs)
