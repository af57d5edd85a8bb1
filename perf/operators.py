"""Cases and plain forms of the quantised key/value cache and the attention that reads it.

Four kinds of pass, each over a paged cache of 8-bit codes with one fp32 scale per token and head:

``append``  quantises new keys and values into the cache and reads the written tokens back
``read``    reads whole sequences back as bf16
``attend``  attention of each sequence's newest tokens over its cached keys, causal from the end
``prefix``  the same for a batch whose sequences begin with one shared prefix

The cache is ``k, v`` [pages, kv heads, page size, d] codes (int8, or e4m3 bytes) and ``k_scale, v_scale``
[pages, kv heads, page size] fp32; a code stands for code * scale.  ``own`` selects the framework's calls; where it
is false the passes are elementary torch operations in 32 bits, and in 64 at the borders of the quantisation.
"""
import math
import random

import torch

own = False

CODE_MAX = {"int8": 127.0, "fp8": 448.0}  # largest code of each format


def listed():
    return [
        # one decoding step of a running batch: 16 sequences write a token each
        dict(name="append_step", kind="append", fmt="int8", page=16, B=16, new_lo=1, new_hi=1, past_lo=512, past_hi=8192, Hkv=8, d=128),
        # a few tokens for some sequences, odd head count, narrow heads
        dict(name="append_odd", kind="append", fmt="fp8", page=32, B=5, new_lo=1, new_hi=37, past_lo=0, past_hi=700, Hkv=3, d=64),
        # prompts of 512 to 8192 tokens written at once
        dict(name="append_prompts", kind="append", fmt="fp8", page=64, B=16, new_lo=512, new_hi=8192, past_lo=0, past_hi=0, Hkv=16,
             d=128),
        # short sequences handed on as bf16
        dict(name="read_short", kind="read", fmt="int8", page=16, B=3, len_lo=1, len_hi=700, Hkv=4, d=64),
        # a long context handed to a dense kernel or another machine
        dict(name="read_long", kind="read", fmt="fp8", page=128, B=1, len_lo=65536, len_hi=65536, Hkv=8, d=128),
        # one user, one token, a short context: latency
        dict(name="attend_one", kind="attend", fmt="int8", page=16, B=1, q_lo=1, q_hi=1, len_lo=2048, len_hi=2048, Hq=16, Hkv=2,
             d=64),
        # one user deep in a long context
        dict(name="attend_long", kind="attend", fmt="fp8", page=64, B=1, q_lo=1, q_hi=1, len_lo=65536, len_hi=65536, Hq=16, Hkv=4,
             d=128),
        # a decoding step of a ragged batch
        dict(name="attend_batch", kind="attend", fmt="int8", page=16, B=64, q_lo=1, q_hi=1, len_lo=512, len_hi=8192, Hq=32, Hkv=8,
             d=128),
        # drafts of 1 to 5 tokens to verify, odd group of heads
        dict(name="attend_draft", kind="attend", fmt="fp8", page=32, B=16, q_lo=1, q_hi=5, len_lo=5, len_hi=4096, Hq=24, Hkv=4,
             d=128),
        # chunks of prompts over what is cached already, one key head per query head
        dict(name="attend_chunk", kind="attend", fmt="int8", page=64, B=4, q_lo=256, q_hi=2048, len_lo=2048, len_hi=8192, Hq=16,
             Hkv=16, d=128),
        # a few answers drawn from one prompt
        dict(name="prefix_small", kind="prefix", fmt="int8", page=16, B=8, q_lo=1, q_hi=1, prefix=2048, len_lo=1, len_hi=129, Hq=16,
             Hkv=4, d=64),
        # many users behind one long document
        dict(name="prefix_large", kind="prefix", fmt="fp8", page=64, B=64, q_lo=1, q_hi=1, prefix=32768, len_lo=64, len_hi=1024,
             Hq=32, Hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "read", "attend", "attend", "prefix", "prefix"])
    c = dict(kind=kind, fmt=rng.choice(["int8", "fp8"]), page=rng.choice([16, 32, 64, 128]),
             d=rng.choice([64, 128]), Hkv=rng.randint(1, 16))
    if kind == "append":
        c["B"] = _log_int(rng, 1, 64)
        top = _log_int(rng, 1, min(8192, 65536 // c["B"]))
        c["new_lo"], c["new_hi"] = max(1, top // rng.randint(1, 16)), top
        past = rng.choice([0, _log_int(rng, 1, 2048)])
        c["past_lo"], c["past_hi"] = past // 2, past
        return c
    if kind == "read":
        c["B"] = _log_int(rng, 1, 64)
        top = _log_int(rng, 1, 32768 // c["B"])
        c["len_lo"], c["len_hi"] = max(1, top // rng.randint(1, 16)), top
        return c
    c["Hkv"] = rng.randint(1, 8)
    c["Hq"] = c["Hkv"] * rng.randint(1, 8)
    c["B"] = _log_int(rng, 1, 64)
    wide = rng.random() < 0.25
    c["q_lo"], c["q_hi"] = 1, rng.choice([1, 1, 1, rng.randint(2, 9)])
    if wide:
        c["B"] = rng.randint(1, 4)
        top = _log_int(rng, 16, 1024)
        c["q_lo"], c["q_hi"] = max(1, top // rng.randint(1, 4)), top
    if kind == "prefix":
        c["prefix"] = c["page"] * max(1, _log_int(rng, 128, 16384) // c["page"])
        top = c["q_hi"] + _log_int(rng, 1, 1024)
        c["len_lo"], c["len_hi"] = c["q_hi"], top
    else:
        top = c["q_hi"] + _log_int(rng, 1, 8192)
        c["len_lo"], c["len_hi"] = max(c["q_hi"], top // rng.randint(1, 16)), top
    return c


def _lengths(case):
    """(query or new tokens, cached tokens in all) of each sequence; part of the case, not of the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B = case["B"]
    if case["kind"] == "append":
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
        return new, [rng.randint(case["past_lo"], case["past_hi"]) + n for n in new]
    if case["kind"] == "read":
        lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(B)]
        return lens, lens
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(B)]
    return q, [case.get("prefix", 0) + rng.randint(case["len_lo"], case["len_hi"]) for _ in range(B)]


def _quantise(x, fmt):
    """Codes and fp32 scales of the rows of x (any leading shape, d last)."""
    top = CODE_MAX[fmt]
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    y = torch.where(amax > 0, x * top / amax, torch.zeros_like(x))
    code = torch.round(y).to(torch.int8) if fmt == "int8" else y.float().to(torch.float8_e4m3fn)
    return code, (amax[..., 0] / top).float()


def _rows(shape, gen, heavy):
    """Normal values; keys have some channels several times the others' size, as trained models' keys do."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if heavy:
        x[..., ::16] *= 4.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    Hkv, d, page, fmt = case["Hkv"], case["d"], case["page"], case["fmt"]
    news, lens = _lengths(case)
    B, T = case["B"], sum(news)
    shared = case.get("prefix", 0) // page
    own_pages = [-(-n // page) - shared for n in lens]
    pages = shared + sum(own_pages) + 3
    order = torch.randperm(pages, generator=cpu, dtype=torch.int64).to(torch.int32)
    table = torch.zeros((B, shared + max(own_pages)), dtype=torch.int32)
    at = shared
    for b in range(B):
        table[b, :shared] = order[:shared]
        table[b, shared:shared + own_pages[b]] = order[at:at + own_pages[b]]
        at += own_pages[b]
    cu = torch.tensor([0] + news, dtype=torch.int64).cumsum(0).to(torch.int32)
    code = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    st = dict(case=case, news=news, lens=lens, table=table.cuda(), cu=cu.cuda(),
              seqlens=torch.tensor(lens, dtype=torch.int32).cuda(),
              past=torch.tensor([n - m for n, m in zip(lens, news)], dtype=torch.int32).cuda())
    for name in ("k", "v"):
        st[name] = torch.zeros((pages, Hkv, page, d), dtype=code, device="cuda")
        st[name + "_scale"] = torch.zeros((pages, Hkv, page), dtype=torch.float32, device="cuda")
        if case["kind"] == "append":
            st[name + "_new"] = _rows((T, Hkv, d), gen, name == "k")
        else:
            step = max(1, (1 << 26) // (Hkv * page * d))
            for p in range(0, pages, step):
                n = min(step, pages - p)
                st[name][p:p + n], st[name + "_scale"][p:p + n] = _quantise(_rows((n, Hkv, page, d), gen, name == "k"),
                                                                           fmt)
    if "Hq" in case:
        st["q"] = _rows((T, case["Hq"], d), gen, False)
    if own:
        from io_aware_exact_25_b200.kvcache import KVCache
        st["cache"] = KVCache.from_tensors(st["k"], st["v"], st["k_scale"], st["v_scale"])
    return st


def run(st):
    kind = st["case"]["kind"]
    if own:
        return _run_own(st, kind)
    if kind == "append":
        return _plain_append(st)
    if kind == "read":
        return _plain_read(st)
    return _plain_attend(st)


def _run_own(st, kind):
    cache = st["cache"]
    if kind == "append":
        cache.append(st["k_new"], st["v_new"], st["table"], st["past"], cu_seqlens=st["cu"])
        k, v = cache.read(st["table"], st["cu"], total_tokens=st["k_new"].shape[0], starts=st["past"])
        return k, v, st["k_scale"], st["v_scale"]
    if kind == "read":
        return cache.read(st["table"], st["cu"], total_tokens=sum(st["lens"]))
    from io_aware_exact_25_b200.kvcache import flash_attention_kvcache
    return flash_attention_kvcache(st["q"], cache, st["table"], st["seqlens"], cu_seqlens_q=st["cu"],
                                   max_seqlen_q=max(st["news"]), causal=True, prefix_len=st["case"].get("prefix", 0),
                                   return_lse=True)


def _slots(st, b, first, count):
    """Page and slot of positions [first, first + count) of sequence b."""
    page = st["case"]["page"]
    pos = torch.arange(first, first + count, device="cuda")
    return st["table"][b].long()[pos // page], pos % page


def _values(st, name, b, first, count):
    """fp32 values [count, Hkv, d] of positions [first, first + count) of sequence b."""
    p, s = _slots(st, b, first, count)
    return st[name][p, :, s].float() * st[name + "_scale"][p, :, s][..., None]


def _plain_append(st):
    at = 0
    for b, (n, total) in enumerate(zip(st["news"], st["lens"])):
        p, s = _slots(st, b, total - n, n)
        for name in ("k", "v"):
            code, scale = _quantise(st[name + "_new"][at:at + n], st["case"]["fmt"])
            st[name].view(torch.uint8)[p, :, s] = code.view(torch.uint8)
            st[name + "_scale"][p, :, s] = scale
        at += n
    return (*_plain_read(st), st["k_scale"], st["v_scale"])


def _plain_read(st):
    return tuple(torch.cat([_values(st, name, b, total - n, n)
                            for b, (n, total) in enumerate(zip(st["news"], st["lens"]))]).to(torch.bfloat16)
                 for name in ("k", "v"))


def _plain_attend(st):
    case = st["case"]
    Hkv, Hq, d = case["Hkv"], case["Hq"], case["d"]
    g = Hq // Hkv
    outs, lses = [], []
    at = 0
    for b, (n, total) in enumerate(zip(st["news"], st["lens"])):
        k, v = _values(st, "k", b, 0, total), _values(st, "v", b, 0, total)
        q = st["q"][at:at + n].float().view(n, Hkv, g, d).permute(1, 2, 0, 3).reshape(Hkv, g * n, d)
        x = torch.matmul(q, k.permute(1, 2, 0)) / math.sqrt(d)
        sees = torch.arange(total, device="cuda")[None] <= (total - n + torch.arange(n, device="cuda"))[:, None]
        x = x.masked_fill(~sees.repeat(g, 1), -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1, keepdim=True)
        o = torch.matmul(e, v.transpose(0, 1)) / z
        outs.append(o.view(Hkv, g, n, d).permute(2, 0, 1, 3).reshape(n, Hq, d))
        lses.append((m + torch.log(z)).view(Hq, n))
        at += n
    return torch.cat(outs).to(torch.bfloat16), torch.cat(lses, 1)


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    Hkv, d = case["Hkv"], case["d"]
    news, lens = _lengths(case)
    T, row = sum(news), 2 * Hkv * (d + 4)  # bytes of a cached token: K and V codes and scales
    if case["kind"] == "append":
        # the new keys and values in, their codes and scales out and in again, the values out
        return dict(bytes=T * (2 * (2 * Hkv * d * 2) + 2 * row), flops=T * Hkv * d * 2 * 4)
    if case["kind"] == "read":
        return dict(bytes=T * (2 * Hkv * d * 2 + row), flops=T * Hkv * d * 2)
    shared = case.get("prefix", 0)
    cached = shared + sum(n - shared for n in lens)
    pairs = sum(n * (total - n) + n * (n + 1) // 2 for n, total in zip(news, lens))
    return dict(bytes=cached * row + T * case["Hq"] * (2 * d * 2 + 4), flops=4 * case["Hq"] * d * pairs)


def exact(case, seed):
    """The passes' results from their definitions in 64 bits."""
    st = prepare(case, seed)
    news, lens = _lengths(case)
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    table = st["table"].tolist()
    if case["kind"] == "append":
        top = CODE_MAX[case["fmt"]]
        out = []
        scales = []
        for name in ("k", "v"):
            x = st[name + "_new"].double()
            amax = x.abs().max(dim=2).values
            scale = amax / top
            unit = x / scale.unsqueeze(2).clamp_min(1e-300)
            if case["fmt"] == "int8":
                # the nearest whole number; a tie (up to the quotient's own error) goes to the even one
                low = torch.floor(unit)
                frac = unit - low
                up = (frac > 0.5 + 1e-9) | (((frac - 0.5).abs() <= 1e-9) & (low % 2 == 1))
                code = low + up
            else:
                # e4m3: steps of 2^(exponent - 3), exponent >= -6; a tie goes to the even step
                e = torch.floor(torch.log2(unit.abs().clamp_min(2.0 ** -6)) + 1e-13).clamp(-6, 8)
                stepsize = torch.pow(2.0, e - 3)
                steps = unit / stepsize
                low = torch.floor(steps)
                frac = steps - low
                up = (frac > 0.5 + 1e-9) | (((frac - 0.5).abs() <= 1e-9) & (low % 2 == 1))
                code = (low + up) * stepsize
            out.append(code * scale.unsqueeze(2))
            whole = torch.zeros(st[name + "_scale"].shape, dtype=torch.float64, device="cuda")
            t = 0
            for b, (n, total) in enumerate(zip(news, lens)):
                pos = range(total - n, total)
                pp = torch.tensor([table[b][i // page] for i in pos], device="cuda")
                ss = torch.tensor([i % page for i in pos], device="cuda")
                whole[pp, :, ss] = scale[t:t + n]
                t += n
            scales.append(whole)
        return (*out, *scales)

    def values(name, b, head=None):
        pp = torch.tensor(table[b][:-(-lens[b] // page)], device="cuda")
        codes = st[name][pp].float().double()              # [pages, Hkv, page, d]
        full = codes * st[name + "_scale"][pp].double().unsqueeze(3)
        full = full.transpose(0, 1).reshape(Hkv, -1, d)[:, :lens[b]]
        return full

    if case["kind"] == "read":
        return tuple(torch.cat([values(name, b).transpose(0, 1) for b in range(case["B"])]) for name in ("k", "v"))
    Hq = case["Hq"]
    T = sum(news)
    o = torch.empty((T, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((Hq, T), dtype=torch.float64, device="cuda")
    t = 0
    for b in range(case["B"]):
        n, total = news[b], lens[b]
        k, v = values("k", b), values("v", b)
        end = torch.arange(total - n, total, device="cuda") + 1        # keys that each query sees
        hidden = torch.arange(total, device="cuda").unsqueeze(0) >= end.unsqueeze(1)
        for h in range(Hq):
            kv = h * Hkv // Hq
            score = st["q"][t:t + n, h].double() @ k[kv].t() * (d ** -0.5)
            score[hidden] = -math.inf
            lse[h, t:t + n] = torch.logsumexp(score, 1)
            o[t:t + n, h] = torch.exp(score - lse[h, t:t + n].unsqueeze(1)) @ v[kv]
        t += n
    return o, lse
