"""The prompt-side operators of the library, as they are measured.

Three operators take a batch of prompts into the verify loop and report on its
tokens:

prompt_attn       causal attention of packed prompts of different lengths over
                  their own bf16 keys and values (grouped heads)
kv_append_packed  the same packed keys and values quantised into the paged
                  cache, behind what each lane has cached already
token_logprobs    log probability of a given token per logits row, the row's
                  entropy, and its most probable tokens

``run`` with ``own`` false computes them in plain torch operations in 32 bits;
with ``own`` true it makes the library's calls.  ``exact`` states them again
in 64 bits.
"""
import math

import torch

own = False

PAGE = 64
D = 128
FORMATS = {"fp8": 0, "int4": 1, "int8": 2, "fp8row": 3}  # the cache formats' numbers in the library
LOGITS = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def ints(text):
    return [int(x) for x in str(text).split()]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def attn(lens, hq, hkv, fused=False, outliers=False):
    return {"op": "prompt_attn", "lens": " ".join(map(str, lens)), "hq": hq, "hkv": hkv, "fused": fused,
            "outliers": outliers}


def append(fmt, lens, cached, hkv, fused=False):
    return {"op": "kv_append_packed", "format": fmt, "lens": " ".join(map(str, lens)),
            "cached": " ".join(map(str, cached)), "hkv": hkv, "fused": fused}


def score(rows, vocab, dtype, top, skipped=0.0, masked=0.0):
    return {"op": "token_logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "skipped": skipped,
            "masked": masked}


def listed():
    cases = {
        # one short request reaches an idle engine: nothing but latency
        "attn_40": attn([40], 24, 4),
        # a scheduler's prefill batch: prompts of all lengths, q/k/v slices of one projection's output
        "attn_ragged_8": attn([1, 63, 64, 65, 517, 1030, 2011, 777], 24, 4, fused=True),
        # heads that share nothing, odd lengths, keys with the outlier channels that real models have
        "attn_mha_odd": attn([1501, 999, 2047, 3], 8, 8, outliers=True),
        # a long document in one piece
        "attn_16384": attn([16384], 24, 4),
        # a second turn of a chat: a few tokens behind a cached prefix that ends inside a page
        "append_fp8_turn": append("fp8", [100], [30], 4),
        # a prefill batch into the default format
        "append_fp8_batch": append("fp8", [8192, 4097, 6000, 12345, 640, 7000, 1, 2900], [0] * 8, 4, fused=True),
        # lanes that go on where a shared prefix ended
        "append_int8_prefix": append("int8", [3000, 17, 2500, 64, 63, 1900, 4000, 1, 555, 1234, 800, 2222],
                                     [1024, 5, 0, 64, 127, 700, 2048, 63, 1, 100, 333, 0], 4),
        # one long document, a scale per token
        "append_fp8row_long": append("fp8row", [65001], [0], 4),
        # the bonus token of one lane, with twenty alternatives
        "logprobs_1": score(1, 151936, "float32", 20),
        # an 8-lane verify step of 16 window rows; rows after the accepted prefix are not scored
        "logprobs_step": score(128, 151936, "float32", 5, skipped=0.4),
        # scoring the tokens of a prompt, logits as the model wrote them
        "logprobs_prompt": score(4096, 151936, "bfloat16", 5),
        # a small odd vocabulary under a grammar that forbids most tokens
        "logprobs_odd": score(333, 32003, "float16", 8, masked=0.9),
    }
    return [{"name": n, **c} for n, c in cases.items()]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prompt_attn", "kv_append_packed", "token_logprobs"])
    if op == "prompt_attn":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        longest, num = log_int(rng, 1, 16384), log_int(rng, 1, 24)
        most = 24 * 16384 ** 2  # the padded products of the largest listed case
        while num * hq * longest ** 2 > most:
            num, longest = max(1, num // 2), longest if num > 1 else longest // 2
        lens = [longest] + [rng.choice([log_int(rng, 1, longest), rng.randint(0, longest)]) for _ in range(num - 1)]
        rng.shuffle(lens)
        return attn(lens, hq, hkv, rng.random() < 0.5, rng.random() < 0.3)
    if op == "kv_append_packed":
        hkv, num = rng.choice([1, 2, 4, 8]), log_int(rng, 1, 64)
        total = log_int(rng, num, 65000 * 4 // hkv)
        cuts = sorted(rng.randint(0, total) for _ in range(num - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        cached = [rng.choice([0, 0, rng.randint(0, 300), 64 * rng.randint(0, 8)]) for _ in lens]
        return append(rng.choice(list(FORMATS)), lens, cached, hkv, rng.random() < 0.5)
    vocab = log_int(rng, 100, 160000)
    dtype = rng.choice(list(LOGITS))
    rows = log_int(rng, 1, max(1, min(20000, 300_000_000 // vocab)))
    return score(rows, vocab, dtype, rng.choice([0, 1, 5, 8, 20, 32]) if vocab >= 32 else 1,
                 rng.choice([0.0, 0.0, 0.4]), rng.choice([0.0, 0.0, 0.5, 0.95]))


def work(case):
    if case["op"] == "prompt_attn":
        lens, hq, hkv = ints(case["lens"]), case["hq"], case["hkv"]
        t = sum(lens)
        return {"bytes": t * (4 * hq * D + 4 * hkv * D + 4 * hq), "flops": sum(2 * D * hq * n * (n + 1) for n in lens)}
    if case["op"] == "kv_append_packed":
        t, h = sum(ints(case["lens"])), case["hkv"]
        code = {"fp8": D, "fp8row": D + 4, "int8": D + 4, "int4": D // 2 + 8}[case["format"]]
        return {"bytes": 2 * t * h * (2 * D + code), "flops": 4 * t * h * D}
    scored = max(1, round(case["rows"] * (1 - case["skipped"])))
    size = 4 if case["dtype"] == "float32" else 2
    return {"bytes": scored * case["vocab"] * size + case["rows"] * (12 + 8 * case["top"]),
            "flops": 5 * scored * case["vocab"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def heads(t, *counts):
        """bf16 [t][count][128] for each count: tensors of their own, or slices of one projection's output."""
        x = [normal(t, n, D).to(torch.bfloat16) for n in counts]
        return list(torch.cat(x, 1).split(counts, 1)) if case["fused"] else x

    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "token_logprobs":
        n, v = case["rows"], case["vocab"]
        # peaked and flat rows, each with a favourite
        x = normal(n, v) * torch.empty(n, 1, device="cuda").uniform_(0.3, 3.0, generator=g)
        x[torch.arange(n, device="cuda"), torch.randint(v, (n,), generator=g, device="cuda")] += 8.0
        if case["masked"]:
            x[torch.rand((n, v), generator=g, device="cuda") < case["masked"]] = -math.inf
            x[:, 0] = normal(n)
        tokens = torch.randint(v, (n,), generator=g, **i32)
        tokens[torch.rand(n, generator=g, device="cuda") < 0.5] = 0
        k = round(n * case["skipped"])
        tokens[torch.randperm(n, generator=g, device="cuda")[:k]] = -1
        return {"case": case, "logits": x.to(LOGITS[case["dtype"]]), "tokens": tokens,
                "logprobs": torch.empty(n, device="cuda"), "entropy": torch.empty(n, device="cuda"),
                "top_tokens": torch.empty((n, case["top"]), **i32) if case["top"] else None,
                "top_logprobs": torch.empty((n, case["top"]), device="cuda") if case["top"] else None}

    lens = ints(case["lens"])
    cu = torch.tensor([0] + lens, **i32).cumsum(0).to(torch.int32)
    t = sum(lens)
    if case["op"] == "prompt_attn":
        hq, hkv = case["hq"], case["hkv"]
        q, k, v = heads(t, hq, hkv, hkv)
        if case["outliers"]:
            k[:, :, ::32] *= 8.0
        return {"case": case, "q": q, "k": k, "v": v, "cu": cu, "num": len(lens), "longest": max(lens),
                "out": torch.empty((t, hq, D), dtype=torch.bfloat16, device="cuda"),
                "lse": torch.empty((t, hq), device="cuda")}

    cached, h, fmt = ints(case["cached"]), case["hkv"], case["format"]
    k, v = heads(t, h, h)
    need = [-(-(c + n) // PAGE) for c, n in zip(cached, lens)]
    pages, row = sum(need) + 3, max(max(need), 1)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    lane = torch.repeat_interleave(torch.arange(len(need)), torch.tensor(need))
    slot = torch.cat([torch.arange(m) for m in need])
    table = torch.full((len(need), row), -1, **i32)
    table[lane.cuda(), slot.cuda()] = ids[:sum(need)]

    def codes():
        if fmt == "int8":
            return torch.randint(-127, 128, (pages, h, PAGE, D), generator=g, device="cuda").to(torch.int8).view(torch.uint8)
        if fmt == "int4":
            lo, hi = (torch.randint(-7, 8, (pages, h, PAGE, D // 2), generator=g, device="cuda") & 15 for _ in range(2))
            return (lo | hi << 4).to(torch.uint8)
        return (normal(pages, h, PAGE, D) * 120).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales():
        shape = {"fp8": (pages, h), "fp8row": (pages, h, PAGE), "int8": (pages, h, PAGE, 2), "int4": (pages, h, PAGE, 4)}
        top = {"fp8": 448, "fp8row": 448, "int8": 127, "int4": 7}[fmt]
        s = torch.empty(shape[fmt], device="cuda").uniform_(2.5 / top, 4.0 / top, generator=g)
        return s if fmt.startswith("fp8") else s.to(torch.float16)

    s = {"case": case, "k": k, "v": v, "cu": cu, "lens": torch.tensor(cached, **i32), "table": table,
         "cache": [codes(), codes(), scales(), scales()]}
    # the plain form's offsets of every packed token; the library derives them from cu, lens and table
    lane = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
    s["lane"], s["pos"] = lane, torch.arange(t, device="cuda") - cu.long()[lane] + s["lens"].long()[lane]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"prompt_attn": run_attn, "kv_append_packed": run_append, "token_logprobs": run_logprobs}[s["case"]["op"]](s)


def run_attn(s):
    if own:
        import speculative_decode_verify_append_gb300 as sdva
        sdva.prompt_attn(s["q"], s["k"], s["v"], s["cu"], 1 / math.sqrt(D), s["out"], s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    # a padded batch: every prompt at the longest one's length
    n, m, hq, hkv = s["num"], s["longest"], s["case"]["hq"], s["case"]["hkv"]
    cu = s["cu"].long()
    at = cu[:-1, None] + torch.arange(m, device="cuda")
    real = at < cu[1:, None]
    at = at.clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(n, m, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[at].permute(0, 2, 3, 1).unsqueeze(2)
    v = s["v"].float()[at].permute(0, 2, 1, 3).unsqueeze(2)
    x = torch.matmul(q * (1 / math.sqrt(D)), k)
    x.masked_fill_(torch.ones((m, m), dtype=torch.bool, device="cuda").triu_(1), -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / total
    lse = (top + total.log()).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(n, m, hq, D)[real].to(torch.bfloat16),
            "lse": lse.permute(0, 3, 1, 2).reshape(n, m, hq)[real]}


def e4m3(x):
    """fp32 -> E4M3 codes, to nearest even, saturating."""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def append_plain(s, new, codes, scales):
    fmt, x = s["case"]["format"], new.float()
    page, off = s["table"].long()[s["lane"], s["pos"] // PAGE], s["pos"] % PAGE
    if fmt != "fp8":
        group, top = {"fp8row": (D, 448.0), "int8": (64, 127.0), "int4": (32, 7.0)}[fmt]
        x = x.view(x.shape[0], x.shape[1], D // group, group)
        amax = x.abs().amax(-1)
        sc = amax / top if fmt == "fp8row" else (amax / top).clamp(max=65504.0).to(torch.float16)
        d = torch.where(sc != 0, sc.float(), 1.0)[..., None]
        y = torch.where(sc[..., None] != 0, x / d, 0.0).flatten(2)
        if fmt == "fp8row":
            c = e4m3(y)
        elif fmt == "int8":
            c = y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        else:
            y = y.round().clamp(-7, 7).to(torch.int32) & 15
            c = (y[..., 0::2] | y[..., 1::2] << 4).to(torch.uint8)
        codes[page, :, off] = c
        scales[page, :, off] = sc.squeeze(-1) if fmt == "fp8row" else sc
        return
    # a page's scale: that of its new tokens where the page starts here, else no smaller than it was
    h = x.shape[1]
    cand = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax") / 448.0
    starts = torch.zeros(scales.shape[0], dtype=torch.int32, device="cuda").index_add_(0, page, (off == 0).int()) > 0
    first = s["lens"].long() % PAGE  # cached tokens of a lane's first page, moved to the larger scale
    lane = torch.arange(first.numel(), device="cuda")
    has = ((s["cu"][1:] > s["cu"][:-1]) & (first > 0)).nonzero().squeeze(1)
    old = s["table"].long()[lane[has], s["lens"].long()[has] // PAGE]
    new_scale = torch.where(starts[:, None], cand, torch.maximum(scales, cand))
    was, now = scales[old], new_scale[old]
    moved = codes[old].view(torch.float8_e4m3fn).float() * was[:, :, None, None] / torch.where(now != 0, now, 1.0)[:, :, None, None]
    keep = (now > was)[:, :, None, None] & (torch.arange(PAGE, device="cuda") < first[has, None])[:, None, :, None]
    codes[old] = torch.where(keep, e4m3(moved), codes[old])
    scales.copy_(new_scale)
    d = new_scale[page][..., None]
    codes[page, :, off] = e4m3(torch.where(d != 0, x / torch.where(d != 0, d, 1.0), 0.0)).view(-1, h, D)


def values(fmt, codes):
    """The numbers that the codes stand for, before their scale."""
    if fmt == "int8":
        return codes.view(torch.int8)
    if fmt == "int4":
        c = torch.stack([codes << 4, codes & 0xF0], -1).flatten(-2)
        return c.view(torch.int8) >> 4
    return codes.view(torch.float8_e4m3fn)


def run_append(s):
    kc, vc, ks, vs = s["cache"]
    fmt = s["case"]["format"]
    if own:
        import speculative_decode_verify_append_gb300 as sdva
        cache = sdva.KVCache(FORMATS[fmt], kc.shape[0], kc.shape[1], tensors=s["cache"])
        sdva.kv_append_packed(cache, s["k"], s["v"], s["cu"], s["table"], s["lens"])
    else:
        append_plain(s, s["k"], kc, ks)
        append_plain(s, s["v"], vc, vs)
    return {"k": values(fmt, kc), "v": values(fmt, vc), "k_scales": ks, "v_scales": vs}


def run_logprobs(s):
    top = s["case"]["top"]
    if own:
        import speculative_decode_verify_append_gb300 as sdva
        sdva.token_logprobs(s["logits"], s["tokens"], s["logprobs"], s["entropy"], s["top_tokens"], s["top_logprobs"])
        r = {"logprobs": s["logprobs"], "entropy": s["entropy"]}
        return {**r, "top_tokens": s["top_tokens"], "top_logprobs": s["top_logprobs"]} if top else r
    scored = s["tokens"] >= 0
    x = s["logits"].float()
    x = x - x.amax(-1, keepdim=True)
    e = x.exp()
    total = e.sum(-1)
    z = total.log()
    # a forbidden token has no part in the entropy
    entropy = z - (e * torch.where(e > 0, x, 0.0)).sum(-1) / total
    logprobs = x.gather(1, s["tokens"].clamp(min=0).long()[:, None]).squeeze(1) - z
    r = {"logprobs": torch.where(scored, logprobs, 0.0), "entropy": torch.where(scored, entropy, 0.0)}
    if top:
        # largest logit first, equal ones by index: one 64-bit key holds both
        y = (s["logits"].float() + 0.0).view(torch.int32)  # + 0.0: the zeros are one number
        key = torch.where(y >= 0, y, y ^ 0x7FFFFFFF).long() << 32
        key += torch.arange(x.shape[1] - 1, -1, -1, device="cuda")
        at = x.shape[1] - 1 - (key.topk(top, -1).values & 0xFFFFFFFF)
        r["top_tokens"] = torch.where(scored[:, None], at, -1).to(torch.int32)
        r["top_logprobs"] = torch.where(scored[:, None], x.gather(1, at) - z[:, None], 0.0)
    return r


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt_attn": exact_attn, "kv_append_packed": exact_append, "token_logprobs": exact_logprobs}[case["op"]](s)


def exact_attn(s):
    t, hq, hkv = s["q"].shape[0], s["case"]["hq"], s["case"]["hkv"]
    out = torch.empty((t, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((t, hq), dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for a, b in zip(cu, cu[1:]):
        for h in range(hq):
            k, v = (s[n][a:b, h * hkv // hq].double() for n in ("k", "v"))
            for i in range(a, b, 4096):
                j = min(i + 4096, b)
                x = s["q"][i:j, h].double() @ k[:j - a].T / math.sqrt(D)
                x = x.masked_fill(torch.arange(a, j, device="cuda") > torch.arange(i, j, device="cuda")[:, None], -math.inf)
                lse[i:j, h] = x.logsumexp(-1)
                out[i:j, h] = (x - lse[i:j, h, None]).exp() @ v[:j - a]
    return {"out": out, "lse": lse}


def round_e4m3(x):
    """x to the nearest number sign * m * 2^e with 3 bits behind the point (2^-9 apart below 2^-6), halves to even."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def exact_append(s):
    """Lane by lane and page by page; codes that are whole numbers have no value in 64 bits."""
    fmt = s["case"]["format"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    r = {}
    for name, codes, scales in zip("kv", s["cache"][:2], s["cache"][2:]):
        sc = scales.double()
        c = codes.view(torch.float8_e4m3fn).double() if fmt.startswith("fp8") else None
        for b, (i, j) in enumerate(zip(cu, cu[1:])):
            pos = lens[b]
            while i < j:
                o = pos % PAGE
                m = min(PAGE - o, j - i)
                p = table[b][pos // PAGE]
                x = s[name][i:i + m].double().transpose(0, 1)
                if fmt == "fp8":
                    was, now = sc[p].clone(), x.abs().amax((1, 2)) / 448
                    sc[p] = now if o == 0 else torch.maximum(was, now)
                    w, d = was[:, None, None], sc[p][:, None, None]
                    c[p, :, :o] = torch.where(d > w, round_e4m3(c[p, :, :o] * w / d), c[p, :, :o])
                    c[p, :, o:o + m] = round_e4m3(x / d)
                elif fmt == "fp8row":
                    sc[p, :, o:o + m] = x.abs().amax(-1) / 448
                    c[p, :, o:o + m] = round_e4m3(x / sc[p, :, o:o + m, None])
                else:
                    group, top = {"int8": (64, 127), "int4": (32, 7)}[fmt]
                    sc[p, :, o:o + m] = x.unflatten(-1, (-1, group)).abs().amax(-1) / top
                i, pos = i + m, pos + m
        r[name], r[name + "_scales"] = c, sc
    return r


def exact_logprobs(s):
    n, top = s["case"]["rows"], s["case"]["top"]
    lp, en = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    tl = torch.zeros((n, max(top, 1)), dtype=torch.float64, device="cuda")
    for i in range(0, n, 256):
        x = s["logits"][i:i + 256].double()
        logp = x - x.logsumexp(-1, keepdim=True)
        t = s["tokens"][i:i + 256].long()
        on = t >= 0
        lp[i:i + 256] = torch.where(on, logp.gather(1, t.clamp(min=0)[:, None]).squeeze(1), 0.0)
        en[i:i + 256] = torch.where(on, -torch.special.xlogy(logp.exp(), logp.exp()).sum(-1), 0.0)
        if top:
            tl[i:i + 256] = torch.where(on[:, None], logp.topk(top, -1).values, 0.0)
    r = {"logprobs": lp, "entropy": en}
    return {**r, "top_tokens": None, "top_logprobs": tl} if top else r
