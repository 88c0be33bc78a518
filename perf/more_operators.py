"""The operators of a layer around the cache, as they are measured.

A hybrid model puts two kinds of context memory into its layers: the paged,
quantised cache of its attention layers, and the state matrices of its
recurrent layers (the gated delta rule).  Five operators take a prompt batch or
a verify window through either of them:

kv_append_rope         a verify window's queries and keys rotated to their
                       positions, its keys and values quantised into the cache
kv_append_packed_rope  the same for a packed batch of prompts
prompt_delta           the gated delta rule over packed prompts, which leaves
                       each lane's state behind its last token
verify_delta           the gated delta rule over a verify window (a chain or a
                       tree of drafts) from each lane's state: either the
                       tokens' updates are recorded and the state stays, or the
                       whole window is committed (a plain decode step)
commit_delta           the state moved by the recorded updates of the accepted
                       tokens

For a head with state S (128 values by 128 keys), log decay g_t, strength b_t
and normalised q_t, k_t, and p the token before t (a tree: its parent):
    u_t = b_t (v_t - e^g_t S_p k_t)
    S_t = e^g_t S_p + u_t k_t'
    o_t = scale S_t q_t

``run`` with ``own`` false computes them in plain torch operations in 32 bits;
with ``own`` true it makes the library's calls.  ``exact`` states them again
in 64 bits.
"""
import math

import torch

own = False

PAGE = 64
D = 128
EPS = 1e-6
SCALE = 1 / math.sqrt(D)
FORMATS = {"fp8": 0, "int4": 1, "int8": 2, "fp8row": 3}  # the cache formats' numbers in the library


def ints(text):
    return [int(x) for x in str(text).split()]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def rope_window(fmt, lanes, window, longest, hq, hkv, rot, interleaved=False, ragged=False, tree=False):
    return {"op": "kv_append_rope", "format": fmt, "lanes": lanes, "window": window, "longest": longest, "hq": hq,
            "hkv": hkv, "rot": rot, "interleaved": interleaved, "ragged": ragged, "tree": tree}


def rope_packed(fmt, lens, cached, hq, hkv, rot, interleaved=False):
    return {"op": "kv_append_packed_rope", "format": fmt, "lens": " ".join(map(str, lens)),
            "cached": " ".join(map(str, cached)), "hq": hq, "hkv": hkv, "rot": rot, "interleaved": interleaved}


def prompt(lens, cached, hk, hv, fused=False):
    return {"op": "prompt_delta", "lens": " ".join(map(str, lens)), "cached": " ".join(map(str, cached)), "hk": hk,
            "hv": hv, "fused": fused}


def verify(lanes, window, hk, hv, keep=True, ragged=False, tree=False, fused=False):
    return {"op": "verify_delta", "lanes": lanes, "window": window, "hk": hk, "hv": hv, "keep": keep,
            "ragged": ragged, "tree": tree, "fused": fused}


def commit(lanes, window, hk, hv, tree=False):
    return {"op": "commit_delta", "lanes": lanes, "window": window, "hk": hk, "hv": hv, "tree": tree}


def listed():
    cases = {
        # a plain decode step of one request deep in its context: nothing but latency
        "rope_decode_1": rope_window("fp8", 1, 1, 240000, 24, 4, 128),
        # a full server's verify step, lanes that drafted trees of different sizes, half of each head rotated
        "rope_window_64": rope_window("int8", 64, 16, 65536, 24, 4, 64, ragged=True, tree=True),
        # a second turn of a chat behind a cached prefix that ends inside a page
        "rope_turn": rope_packed("int4", [100], [30], 24, 4, 128, interleaved=True),
        # a scheduler's prefill batch into the default format
        "rope_batch": rope_packed("fp8", [8192, 4097, 6000, 12345, 640, 7000, 1, 2900], [0] * 8, 24, 4, 128),
        # one short request reaches an idle engine
        "delta_prompt_40": prompt([40], [0], 4, 8),
        # prompts of all lengths, some of them the later part of one: slices of one projection's output
        "delta_prompt_ragged": prompt([1, 63, 64, 65, 517, 1030, 2011, 777], [0, 64, 0, 1, 2048, 0, 0, 5], 8, 24, True),
        # a long document in one piece
        "delta_prompt_16384": prompt([16384], [0], 16, 32),
        # one plain decode step of many requests
        "delta_decode_64": verify(64, 1, 16, 32, keep=False, fused=True),
        # an 8-lane verify step of 16 window rows
        "delta_verify_8": verify(8, 16, 16, 32),
        # a full server's verify step with draft trees, padded windows
        "delta_verify_64": verify(64, 16, 16, 32, ragged=True, tree=True),
        # the accepted tokens of one request
        "delta_commit_1": commit(1, 6, 16, 32),
        # and of a full server, along the accepted paths of their trees
        "delta_commit_64": commit(64, 16, 16, 32, tree=True),
    }
    return [{"name": n, **c} for n, c in cases.items()]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["kv_append_rope", "kv_append_packed_rope", "prompt_delta", "prompt_delta", "verify_delta",
                     "verify_delta", "commit_delta"])
    flag = lambda p: rng.random() < p  # noqa: E731
    if op.startswith("kv"):
        hkv = rng.choice([1, 2, 4, 8])
        heads = (hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), hkv, rng.choice([16, 32, 64, 128, 128]), flag(0.3))
        fmt = rng.choice(list(FORMATS))
        if op == "kv_append_rope":
            return rope_window(fmt, log_int(rng, 1, 128), rng.randint(1, 16), log_int(rng, 1, 240000), *heads,
                               ragged=flag(0.5), tree=flag(0.4))
        num = log_int(rng, 1, 32)
        total = log_int(rng, num, 41000 * 28 // (heads[0] + hkv))
        total = min(total, 82000)
        cuts = sorted(rng.randint(0, total) for _ in range(num - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return rope_packed(fmt, lens, [rng.choice([0, 0, rng.randint(0, 300), 64 * rng.randint(0, 8)]) for _ in lens],
                           *heads)
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 2, 3, 4] if hk <= 8 else [1, 2])
    if op == "prompt_delta":
        longest, num = log_int(rng, 1, 16384), log_int(rng, 1, 24)
        while num * hv * longest > 16384 * 32:
            num, longest = max(1, num // 2), longest if num > 1 else longest // 2
        lens = [longest] + [rng.choice([log_int(rng, 1, longest), rng.randint(0, longest)]) for _ in range(num - 1)]
        rng.shuffle(lens)
        return prompt(lens, [rng.choice([0, 0, rng.randint(1, 5000)]) for _ in lens], hk, hv, flag(0.5))
    lanes = log_int(rng, 1, 64 * 32 // hv)
    window = rng.choice([1, rng.randint(1, 16)])
    if op == "verify_delta":
        keep = flag(0.7)
        return verify(lanes, window, hk, hv, keep, flag(0.5), keep and flag(0.4), flag(0.5))
    return commit(lanes, window, hk, hv, flag(0.5))


def work(case):
    if case["op"].startswith("kv"):
        t = sum(ints(case["lens"])) if "lens" in case else case["lanes"] * case["window"]
        hq, h = case["hq"], case["hkv"]
        code = {"fp8": D, "fp8row": D + 4, "int8": D + 4, "int4": D // 2 + 8}[case["format"]]
        out = 2 * D * hq + (2 * D * h if "lens" in case else 0)
        return {"bytes": t * (2 * D * (hq + 2 * h) + 2 * code * h + out + 4 * case["rot"]),
                "flops": t * (3 * (hq + h) * case["rot"] + 4 * h * D)}
    hk, hv = case["hk"], case["hv"]
    t = sum(ints(case["lens"])) if "lens" in case else case["lanes"] * case["window"]
    b = len(ints(case["lens"])) if "lens" in case else case["lanes"]
    state = b * hv * D * D * 4
    if case["op"] == "commit_delta":
        return {"bytes": 2 * state + t * (2 * D * hk + 4 * D * hv + 4 * hv), "flops": t * hv * 2 * D * D}
    size = state * (1 if case.get("keep") else 2) + t * (4 * D * hk + 4 * D * hv + 8 * hv)
    if case.get("keep"):
        size += t * hv * D * 4
    return {"bytes": size, "flops": t * hv * 6 * D * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
I32 = dict(dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return (prepare_rope if case["op"].startswith("kv") else prepare_delta)(case, g)


def trees(g, lanes, window):
    """A parent for every slot (an earlier one, more often the slot just before) and every slot's depth."""
    parent = torch.arange(-1, window - 1, device="cuda").repeat(lanes, 1)
    other = (torch.rand((lanes, window), generator=g, device="cuda") * torch.arange(window, device="cuda")).long()
    parent = torch.where(torch.rand((lanes, window), generator=g, device="cuda") < 0.5, parent, other)
    parent[:, 0] = -1
    depth = torch.zeros((lanes, window), dtype=torch.long, device="cuda")
    for i in range(1, window):
        depth[:, i] = depth.gather(1, parent[:, i:i + 1]).squeeze(1) + 1
    return parent, depth


def prepare_rope(case, g):
    fmt, hq, h, rot = case["format"], case["hq"], case["hkv"], case["rot"]
    window = case["op"] == "kv_append_rope"
    if window:
        b, w = case["lanes"], case["window"]
        lens = torch.randint(0, case["longest"] + 1, (b,), generator=g, device="cuda")
        lens[0] = case["longest"]
        count = torch.randint(0, w + 1, (b,), generator=g, device="cuda") if case["ragged"] else torch.full((b,), w, device="cuda")
        row = torch.arange(w, device="cuda").repeat(b, 1)
        lane, slot = (row < count[:, None]).nonzero(as_tuple=True)
        at = lane * w + slot  # the tokens' rows in the window
        rows = b * w
    else:
        count, lens = (torch.tensor(ints(case[n]), device="cuda") for n in ("lens", "cached"))
        b, rows = len(count), int(count.sum())
        lane = torch.repeat_interleave(torch.arange(b, device="cuda"), count)
        slot = torch.arange(rows, device="cuda") - (count.cumsum(0) - count)[lane]
        at = torch.arange(rows, device="cuda")
    pos = lens[lane] + slot

    # queries, keys and values are slices of one projection's output
    x = torch.randn((rows, hq + 2 * h, D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x.split((hq, h, h), 1)
    # the pages that the new tokens touch, in any order; the others are not read
    first, last = lens // PAGE, torch.where(count > 0, (lens + count - 1) // PAGE, lens // PAGE - 1)
    used = (last - first + 1).clamp(min=0)
    pages = 3 + (b * ((w + PAGE - 2) // PAGE + 1) if window else int(used.sum()))
    table = torch.full((b, int(((lens + count + PAGE - 1) // PAGE).max()) + 1), -1, **I32)
    tl = torch.repeat_interleave(torch.arange(b, device="cuda"), used)
    ts = torch.arange(tl.numel(), device="cuda") - (used.cumsum(0) - used)[tl] + first[tl]
    table[tl, ts] = torch.randperm(pages, generator=g, device="cuda")[:tl.numel()].to(torch.int32)

    def codes():
        if fmt == "int8":
            return torch.randint(-127, 128, (pages, h, PAGE, D), generator=g, device="cuda").to(torch.int8).view(torch.uint8)
        if fmt == "int4":
            lo, hi = (torch.randint(-7, 8, (pages, h, PAGE, D // 2), generator=g, device="cuda") & 15 for _ in range(2))
            return (lo | hi << 4).to(torch.uint8)
        c = torch.randn((pages, h, PAGE, D), generator=g, device="cuda") * 120
        return c.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales():
        shape = {"fp8": (pages, h), "fp8row": (pages, h, PAGE), "int8": (pages, h, PAGE, 2), "int4": (pages, h, PAGE, 4)}
        top = {"fp8": 448, "fp8row": 448, "int8": 127, "int4": 7}[fmt]
        s = torch.empty(shape[fmt], device="cuda").uniform_(2.5 / top, 4.0 / top, generator=g)
        return s if fmt.startswith("fp8") else s.to(torch.float16)

    where = pos
    if window and case["tree"]:
        depth = trees(g, b, w)[1]
        where = lens[lane] + depth[lane, slot]
    far = int((lens + count).max()) + 1
    angle = torch.arange(far, device="cuda").double()[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)
    s = {"case": case, "q": q, "k": k, "v": v, "lens": lens.to(torch.int32), "table": table,
         "rope": torch.cat([angle.cos(), angle.sin()], 1).float(),
         "cache": [codes(), codes(), scales(), scales()],
         "q_out": torch.zeros((rows, hq, D), dtype=torch.bfloat16, device="cuda"),
         # the plain form's rows, lanes and positions of the tokens; the library derives them
         "at": at, "lane": lane, "pos": pos, "where": where}
    if window:
        s["n_lane"] = count.to(torch.int32) if case["ragged"] else None
        s["positions"] = (lens[:, None] + depth).to(torch.int32) if case["tree"] else None
        s["shape"] = (b, w)
    else:
        s["cu"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
        s["k_out"] = torch.zeros((rows, h, D), dtype=torch.bfloat16, device="cuda")
    return s


def prepare_delta(case, g):
    hk, hv = case["hk"], case["hv"]
    packed = case["op"] == "prompt_delta"
    lens = ints(case["lens"]) if packed else None
    b = len(lens) if packed else case["lanes"]
    lead = (sum(lens),) if packed else (b, case["window"])

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # a head's keys have a direction in common, as a model's have
    q, k, v = normal(*lead, hk, D), normal(*lead, hk, D) + 0.5 * normal(hk, D), normal(*lead, hv, D)
    x = [y.to(torch.bfloat16) for y in (q, k, v)]
    q, k, v = torch.cat(x, -2).split((hk, hk, hv), -2) if case.get("fused") else x
    # decays from a rate and a step of each head, some of which forget within a few tokens and some hardly at all
    rate, step = 16 * torch.rand(hv, generator=g, device="cuda") + 0.01, torch.exp(normal(hv) - 4)
    log_decay = -rate * torch.nn.functional.softplus(normal(*lead, hv) + torch.log(torch.expm1(step)))
    beta = torch.sigmoid(normal(*lead, hv))
    slots = torch.randperm(b + 2, generator=g, device="cuda")[:b].to(torch.int32)
    s = {"case": case, "q": q, "k": k, "v": v, "log_decay": log_decay, "beta": beta, "slots": slots,
         "state": normal(b + 2, hv, D, D) * 0.2, "n_lane": None, "parent": None, "deltas": None}
    if packed:
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["seq_lens"] = torch.tensor(ints(case["cached"]), **I32)
        s["lens"], s["longest"] = torch.tensor(lens, device="cuda"), max(lens)
        s["out"] = torch.zeros((*lead, hv, D), dtype=torch.bfloat16, device="cuda")
        if own:  # what a user's program allocates once
            import speculative_decode_verify_append_gb300 as sdva
            s["workspace"] = torch.empty(sdva.prompt_delta_workspace_size(lead[0], b, hk, hv), dtype=torch.uint8, device="cuda")
        return s
    w = case["window"]
    parent, depth = trees(g, b, w)
    if case["tree"]:
        s["parent"] = parent.to(torch.int32)
    if case["op"] == "verify_delta":
        if case["ragged"]:
            s["n_lane"] = torch.randint(0, w + 1, (b,), generator=g, **I32)
        s["out"] = torch.zeros((b, w, hv, D), dtype=torch.bfloat16, device="cuda")
        if case["keep"]:
            s["deltas"] = torch.zeros((b, w, hv, D), device="cuda")
        return s
    # recorded updates, and an accepted chain or path that ends at any slot
    s["deltas"] = normal(b, w, hv, D) * 0.1
    end = torch.randint(0, w, (b,), generator=g, device="cuda")
    if not case["tree"]:
        s["accept_len"], s["path"] = end.to(torch.int32), None
        return s
    s["accept_len"] = depth.gather(1, end[:, None]).squeeze(1).to(torch.int32)
    path = torch.full((b, w), -1, device="cuda")
    for _ in range(w):
        on = end >= 0
        d = depth.gather(1, end.clamp(min=0)[:, None])
        path.scatter_(1, d, torch.where(on[:, None], end[:, None], path.gather(1, d)))
        end = torch.where(on, parent.gather(1, end.clamp(min=0)[:, None]).squeeze(1), end)
    s["path"] = path.to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"kv_append_rope": run_rope, "kv_append_packed_rope": run_rope, "prompt_delta": run_prompt,
            "verify_delta": run_verify, "commit_delta": run_commit}[s["case"]["op"]](s)


def rotate(x, table, where, rot, interleaved):
    """The first rot dims of x [t][heads][128] turned by their position's angles; products and sums of 32 bits, each rounded."""
    c, n = (y[:, None, :] for y in table[where].chunk(2, -1))
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    p, r = a * c - b * n, b * c + a * n
    turned = torch.stack([p, r], -1).flatten(-2) if interleaved else torch.cat([p, r], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16)


def e4m3(x):
    """fp32 -> E4M3 codes, to nearest even, saturating."""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def append_plain(s, x, codes, scales):
    """bf16 rows x of the tokens (s["lane"], s["pos"]) into the cache."""
    fmt, x, h = s["case"]["format"], x.float(), x.shape[1]
    page, off = s["table"].long()[s["lane"], s["pos"] // PAGE], s["pos"] % PAGE
    if fmt != "fp8":
        group, top = {"fp8row": (D, 448.0), "int8": (64, 127.0), "int4": (32, 7.0)}[fmt]
        x = x.unflatten(-1, (-1, group))
        amax = x.abs().amax(-1)
        sc = amax / top if fmt == "fp8row" else (amax / top).clamp(max=65504.0).to(torch.float16)
        y = torch.where(sc[..., None] != 0, x / torch.where(sc != 0, sc.float(), 1.0)[..., None], 0.0).flatten(2)
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
    top = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax") / 448.0
    new = torch.zeros(scales.shape[0], dtype=torch.int32, device="cuda").index_add_(0, page, (off == 0).int()) > 0
    now = torch.where(new[:, None], top, torch.maximum(scales, top))
    # cached tokens of a lane's first page move to the larger scale
    behind = torch.zeros(scales.shape[0], dtype=torch.long, device="cuda")
    behind.index_reduce_(0, page, off, "amin", include_self=False)
    moves = (now > scales) & ~new[:, None]
    keep = moves[:, :, None, None] & (torch.arange(PAGE, device="cuda") < behind[:, None])[:, None, :, None]
    d = torch.where(now != 0, now, 1.0)
    moved = codes.view(torch.float8_e4m3fn).float() * scales[:, :, None, None] / d[:, :, None, None]
    codes.copy_(torch.where(keep, e4m3(moved), codes))
    scales.copy_(now)
    codes[page, :, off] = e4m3(torch.where(now[page][..., None] != 0, x / d[page][..., None], 0.0)).view(-1, h, D)


def values(fmt, codes):
    """The numbers that the codes stand for, before their scale."""
    if fmt == "int8":
        return codes.view(torch.int8)
    if fmt == "int4":
        c = torch.stack([codes << 4, codes & 0xF0], -1).flatten(-2)
        return c.view(torch.int8) >> 4
    return codes.view(torch.float8_e4m3fn)


def run_rope(s):
    case = s["case"]
    fmt, (kc, vc, ks, vs) = case["format"], s["cache"]
    if own:
        import speculative_decode_verify_append_gb300 as sdva
        cache = sdva.KVCache(FORMATS[fmt], kc.shape[0], kc.shape[1], tensors=s["cache"])
        if "cu" in s:
            sdva.kv_append_packed_rope(cache, s["q"], s["k"], s["v"], s["cu"], s["rope"], s["table"], s["lens"],
                                       s["q_out"], s["k_out"], interleaved=case["interleaved"])
        else:
            q, k, v, q_out = (s[n].unflatten(0, s["shape"]) for n in ("q", "k", "v", "q_out"))
            sdva.kv_append_rope(cache, q, k, v, s["rope"], s["table"], s["lens"], q_out, n_lane=s["n_lane"],
                                positions=s["positions"], interleaved=case["interleaved"])
    else:
        at = s["at"]
        how = (s["rope"], s["where"], case["rot"], case["interleaved"])
        k = rotate(s["k"][at], *how)
        s["q_out"][at] = rotate(s["q"][at], *how)
        if "k_out" in s:
            s["k_out"][at] = k
        append_plain(s, k, kc, ks)
        append_plain(s, s["v"][at], vc, vs)
    r = {"q": s["q_out"], "k": values(fmt, kc), "v": values(fmt, vc), "k_scales": ks, "v_scales": vs}
    return {**r, "k_out": s["k_out"]} if "k_out" in s else r


def unit(x):
    x = x.float()
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)


def run_prompt(s):
    if own:
        import speculative_decode_verify_append_gb300 as sdva
        sdva.prompt_delta(s["state"], s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["cu"], s["slots"], SCALE,
                          s["out"], s["workspace"], s["seq_lens"], EPS)
        return {"out": s["out"], "state": s["state"]}
    # a padded batch, [lane * head][chunk][64], the padding with nothing in it
    b, hk, hv, c = len(s["lens"]), s["case"]["hk"], s["case"]["hv"], 64
    n = -(-s["longest"] // c)
    row = torch.arange(n * c, device="cuda")
    real = row < s["lens"][:, None]
    at = (s["cu"][:-1, None].long() + row).clamp(max=s["q"].shape[0] - 1)

    def chunks(x, scale=1.0):
        x = torch.where(real.view(*real.shape, *[1] * (x.dim() - 1)), x[at] * scale, 0.0)
        x = x.repeat_interleave(hv // x.shape[2], 2).transpose(1, 2)
        return x.reshape(b * hv, n, c, *x.shape[3:])

    q, k, v = chunks(unit(s["q"]), SCALE), chunks(unit(s["k"])), chunks(s["v"].float())
    fall, beta = chunks(s["log_decay"].double()).cumsum(-1), chunks(s["beta"])
    lower = torch.ones((c, c), dtype=torch.bool, device="cuda").tril_()
    decay = (fall[..., :, None] - fall[..., None, :]).masked_fill_(~lower, -math.inf).exp_().float()
    scores = torch.matmul(q, k.transpose(-1, -2)) * decay
    # the updates of a chunk depend on one another: inv (1 + a) = 1, row by row
    a = torch.matmul(k, k.transpose(-1, -2)) * decay * beta[..., None]
    inv = torch.eye(c, device="cuda").repeat(b * hv, n, 1, 1)
    for i in range(1, c):
        inv[..., i, :i] = -torch.matmul(a[..., i, None, :i], inv[..., :i, :i]).squeeze(-2)
    inv *= beta[..., None, :]
    rest, fall = (fall[..., -1:] - fall).exp().float()[..., None], fall.exp().float()[..., None]
    state = torch.where((s["seq_lens"] > 0)[:, None, None, None], s["state"][s["slots"].long()], 0.0).view(-1, D, D)
    out = torch.empty((b * hv, n, c, D), device="cuda")
    for i in range(n):
        left = state.transpose(-1, -2)
        u = torch.matmul(inv[:, i], v[:, i] - fall[:, i] * torch.matmul(k[:, i], left))
        out[:, i] = fall[:, i] * torch.matmul(q[:, i], left) + torch.matmul(scores[:, i], u)
        state = state * fall[:, i, -1:] + torch.matmul((u * rest[:, i]).transpose(-1, -2), k[:, i])
    # a lane without tokens keeps what it has
    had = s["state"][s["slots"].long()]
    s["state"][s["slots"].long()] = torch.where((s["lens"] > 0)[:, None, None, None], state.view_as(had), had)
    s["out"].copy_(out.view(b, hv, n * c, D).transpose(1, 2)[real])
    return {"out": s["out"], "state": s["state"]}


def run_verify(s):
    keep = s["case"]["keep"]
    if own:
        import speculative_decode_verify_append_gb300 as sdva
        sdva.verify_delta(s["state"], s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["slots"], SCALE, s["out"],
                          s["deltas"], s["n_lane"], s["parent"], EPS)
        return {"out": s["out"], "deltas": s["deltas"]} if keep else {"out": s["out"], "state": s["state"]}
    w, hv = s["case"]["window"], s["case"]["hv"]
    q, k, raw = (x.repeat_interleave(hv // x.shape[2], 2) for x in (unit(s["q"]), unit(s["k"]), s["k"].float()))
    norm = torch.rsqrt(raw.square().sum(-1, keepdim=True) + EPS)
    v, fall, b = s["v"].float(), s["log_decay"].exp(), s["beta"]
    lane = torch.arange(v.shape[0], device="cuda")
    # the state in front of the window, then the one behind each slot
    states = [s["state"][s["slots"].long()]]
    out, deltas = torch.zeros_like(v), torch.zeros_like(v)
    count = s["n_lane"]
    for i in range(w):
        on = torch.ones_like(lane, dtype=torch.bool) if count is None else i < count
        if s["parent"] is None or i == 0:
            before = states[-1]
        else:
            before = torch.stack(states)[s["parent"][:, i].long() + 1, lane]
        x = before * fall[:, i, :, None, None]
        u = b[:, i, :, None] * (v[:, i] - torch.matmul(x, k[:, i, :, :, None]).squeeze(-1))
        x = x + u[..., None] * k[:, i, :, None, :]
        states.append(torch.where(on[:, None, None, None], x, before))
        out[:, i] = torch.where(on[:, None, None], SCALE * torch.matmul(x, q[:, i, :, :, None]).squeeze(-1), 0.0)
        deltas[:, i] = torch.where(on[:, None, None], u * norm[:, i], 0.0)
    s["out"].copy_(out)
    if keep:
        s["deltas"].copy_(deltas)
        return {"out": s["out"], "deltas": s["deltas"]}
    s["state"][s["slots"].long()] = states[-1]
    return {"out": s["out"], "state": s["state"]}


def run_commit(s):
    if own:
        import speculative_decode_verify_append_gb300 as sdva
        sdva.commit_delta(s["state"], s["k"], s["log_decay"], s["deltas"], s["slots"], s["accept_len"], s["path"])
        return {"state": s["state"]}
    w, hv = s["case"]["window"], s["case"]["hv"]
    k, d, g = s["k"].float().repeat_interleave(hv // s["k"].shape[2], 2), s["deltas"], s["log_decay"].double()
    row = torch.arange(w, device="cuda")
    at = row.expand(k.shape[0], -1) if s["path"] is None else s["path"].long().clamp(min=0)
    on = (row <= s["accept_len"][:, None])[..., None]
    g = torch.where(on, g.gather(1, at[..., None].expand(-1, -1, hv)), 0.0)
    at = at[..., None, None].expand(-1, -1, hv, D)
    behind = g.flip(1).cumsum(1).flip(1) - g
    d = d.gather(1, at) * torch.where(on, behind.exp(), 0.0).float()[..., None]
    state = s["state"][s["slots"].long()] * g.sum(1).exp().float()[..., None, None]
    s["state"][s["slots"].long()] = state + torch.matmul(d.permute(0, 2, 3, 1), k.gather(1, at).transpose(1, 2))
    return {"state": s["state"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"kv_append_rope": exact_rope, "kv_append_packed_rope": exact_rope, "prompt_delta": exact_prompt,
            "verify_delta": exact_verify, "commit_delta": exact_commit}[case["op"]](s)


def round_e4m3(x):
    """x to the nearest number sign * m * 2^e with 3 bits behind the point (2^-9 apart below 2^-6), halves to even."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def exact_rope(s):
    """Token by token of a lane's page.  The cache takes the rotated key as the definition rounds it: each product
    and the sum to 32 bits, then to bf16; codes that are whole numbers have no value in 64 bits."""
    case, fmt = s["case"], s["case"]["format"]
    rot, half = case["rot"], case["rot"] // 2
    first = list(range(0, rot, 2)) if case["interleaved"] else list(range(half))
    second = list(range(1, rot, 2)) if case["interleaved"] else list(range(half, rot))
    angle = s["rope"].double()[s["where"]]
    c, n = angle[:, None, :half], angle[:, None, half:]

    def turn(x, narrow):
        y = x.double()[s["at"]]
        a, b = y[..., first], y[..., second]
        z = y.clone()
        z[..., first], z[..., second] = narrow(narrow(a * c) - narrow(b * n)), narrow(narrow(b * c) + narrow(a * n))
        return z

    def whole(x, z):
        r = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        r[s["at"]] = z
        return r

    r = {"q": whole(s["q"], turn(s["q"], lambda x: x))}
    if "k_out" in s:
        r["k_out"] = whole(s["k"], turn(s["k"], lambda x: x))
    new = {"k": turn(s["k"], lambda x: x.float().double()).float().bfloat16().double(), "v": s["v"].double()[s["at"]]}
    page, off = s["table"].long()[s["lane"], s["pos"] // PAGE], s["pos"] % PAGE
    order = torch.argsort(page * PAGE + off)
    ids, sizes = page[order].unique_consecutive(return_counts=True)
    for name, codes, scales in zip("kv", s["cache"][:2], s["cache"][2:]):
        x, sc = new[name], scales.double()
        cd = codes.view(torch.float8_e4m3fn).double() if fmt.startswith("fp8") else None
        if fmt == "fp8row":
            sc[page, :, off] = x.abs().amax(-1) / 448
            cd[page, :, off] = round_e4m3(x / sc[page, :, off][..., None])
        elif fmt != "fp8":
            group, top = {"int8": (64, 127), "int4": (32, 7)}[fmt]
            sc[page, :, off] = x.unflatten(-1, (-1, group)).abs().amax(-1) / top
        else:
            i = 0
            for p, m in zip(ids.tolist(), sizes.tolist()):
                y, o = x[order[i:i + m]].transpose(0, 1), int(off[order[i]])
                was, now = sc[p].clone(), y.abs().amax((1, 2)) / 448
                sc[p] = now if o == 0 else torch.maximum(was, now)
                a, d = was[:, None, None], sc[p][:, None, None]
                cd[p, :, :o] = torch.where(d > a, round_e4m3(cd[p, :, :o] * a / d), cd[p, :, :o])
                cd[p, :, o:o + m] = round_e4m3(y / d)
                i += m
        r[name], r[name + "_scales"] = cd, sc
    return r


def step64(state, q, k, v, g, b):
    """One token of every lane: state [n][h][128][128], q, k [n][h][128] normalised, v [n][h][128], g, b [n][h]."""
    state = state * g.exp()[..., None, None]
    u = b[..., None] * (v - (state @ k[..., None]).squeeze(-1))
    state = state + u[..., :, None] * k[..., None, :]
    return state, u, SCALE * (state @ q[..., None]).squeeze(-1)


def unit64(x, hv):
    x = x.double()
    x = x / (x.square().sum(-1, keepdim=True) + EPS).sqrt()
    return x.repeat_interleave(hv // x.shape[-2], -2)


def exact_prompt(s):
    hv, cu = s["case"]["hv"], s["cu"].long()
    q, k, v, g, b = unit64(s["q"], hv), unit64(s["k"], hv), s["v"].double(), s["log_decay"].double(), s["beta"].double()
    whole, out = s["state"].double(), torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    state = whole[s["slots"].long()]
    state[(s["seq_lens"] == 0) & (s["lens"] > 0)] = 0.0
    lens = s["lens"].tolist()
    for i in range(s["longest"]):
        on = [j for j, n in enumerate(lens) if n > i]
        every = len(on) == len(lens)
        at = cu[on] + i
        new, _, o = step64(state if every else state[on], q[at], k[at], v[at], g[at], b[at])
        if every:
            state = new
        else:
            state[on] = new
        out[at] = o
    whole[s["slots"].long()] = state
    return {"out": out, "state": whole}


def exact_verify(s):
    case = s["case"]
    w, hv = case["window"], case["hv"]
    q, k, v, g, b = unit64(s["q"], hv), unit64(s["k"], hv), s["v"].double(), s["log_decay"].double(), s["beta"].double()
    norm = (s["k"].double().square().sum(-1, keepdim=True) + EPS).sqrt().repeat_interleave(hv // case["hk"], 2)
    whole = s["state"].double()
    out, deltas = torch.zeros_like(v), torch.zeros_like(v)
    for lane, slot in enumerate(s["slots"].tolist()):
        count = w if s["n_lane"] is None else int(s["n_lane"][lane])
        parent = list(range(-1, w - 1)) if s["parent"] is None else s["parent"][lane].tolist()
        states = {-1: whole[slot][None]}
        for i in range(count):
            row = (x[lane:lane + 1, i] for x in (q, k, v, g, b))
            states[i], u, o = step64(states[parent[i] if i else -1], *row)
            out[lane, i], deltas[lane, i] = o[0], u[0] / norm[lane, i]
        if not case["keep"]:
            whole[slot] = states[count - 1][0]
    return {"out": out, "deltas": deltas} if case["keep"] else {"out": out, "state": whole}


def exact_commit(s):
    case = s["case"]
    k, d, g = s["k"].double().repeat_interleave(case["hv"] // case["hk"], 2), s["deltas"].double(), s["log_decay"].double()
    whole = s["state"].double()
    for lane, slot in enumerate(s["slots"].tolist()):
        for j in range(int(s["accept_len"][lane]) + 1):
            i = j if s["path"] is None else int(s["path"][lane, j])
            whole[slot] = whole[slot] * g[lane, i].exp()[:, None, None] + d[lane, i][:, :, None] * k[lane, i][:, None, :]
    return {"state": whole}
