"""prompt_attn, kv_append_packed and token_logprobs on the GPU against plain
64-bit statements, and a run of them together with the verify step."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import ALL_KV, KV_NAMES, SM_SCALE, bf16_dev, cache_to_host, i32_dev

pytestmark = pytest.mark.gpu

D = 128
NAN, INF = float("nan"), float("inf")


def _cu(lens, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _qkv(g, T, hq, hkv, fused=False):
    x = torch.randn((T, hq + 2 * hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x.split([hq, hkv, hkv], 1)
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# prompt_attn
# ---------------------------------------------------------------------------
def _attn_ref(q, k, v, lens, scale, start=0):
    """out, lse and their error bounds, fp64.

    Bounds.  A score is 128 products added in fp32: off by at most
    E = 128 * 2^-22 * scale * sum |q_i k_i| (2^-22 a step: the tensor core may
    truncate where fp32 would round), plus 2^-22 |s| for the scaling.  That
    moves a weight by a factor within exp(+-2E) and lse by E; exp2 and the
    sums add 2^-20.  Weights are rounded to bf16 (2^-8 of each), the output
    once more (2^-8 of it)."""
    T, hq = q.shape[:2]
    G = hq // k.shape[1]
    out = torch.zeros((T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, hq), dtype=torch.float64, device="cuda")
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    a = start
    for n in lens:
        if n:
            qq = q[a:a + n].double().transpose(0, 1)
            kk, vv = (x[a:a + n].double().transpose(0, 1).repeat_interleave(G, 0) for x in (k, v))
            s = qq @ kk.transpose(1, 2) * scale
            mag = qq.abs() @ kk.abs().transpose(1, 2) * scale
            mask = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
            s, mag = s.masked_fill(mask, -INF), mag.masked_fill(mask, 0.0)
            e = 128 * 2.0 ** -22 * mag.amax(-1) + 2.0 ** -22 * s.masked_fill(mask, 0.0).abs().amax(-1)
            z = s.logsumexp(-1)
            p = (s - z[..., None]).exp().masked_fill(mask, 0.0)
            o = p @ vv
            out[a:a + n], lse[a:a + n] = o.transpose(0, 1), z.transpose(0, 1)
            av = p @ vv.abs()
            near = (2.0 ** -8 + 4 * e[..., None] + 2.0 ** -18) * av * 1.01
            tol_o[a:a + n] = (2.0 ** -8 * o.abs() + near).transpose(0, 1)
            tol_l[a:a + n] = (e + 2.0 ** -20 * (1 + z.abs())).transpose(0, 1)
        a += n
    return out, lse, tol_o, tol_l


def _run_attn(q, k, v, cu, scale=float(SM_SCALE), status=None):
    import speculative_decode_verify_append_gb300 as sdva
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    sdva.prompt_attn(q, k, v, cu, scale, out, lse, status)
    torch.cuda.synchronize()
    return out, lse


def _check_attn(q, k, v, lens, scale=float(SM_SCALE), start=0):
    st = _status()
    out, lse = _run_attn(q, k, v, _cu(lens, start), scale, st)
    assert int(st.item()) == 0
    ro, rl, to, tl = _attn_ref(q, k, v, lens, scale, start)
    end = start + sum(lens)
    for got, want, tol in ((out, ro, to), (lse, rl, tl)):
        err = (got[start:end].double() - want[start:end]).abs()
        bad = (~(err <= tol[start:end])).nonzero()
        assert bad.numel() == 0, (lens, len(bad), bad[:5].tolist(), float(err.nan_to_num().max()))
        assert (got[:start] == 7.0).all() and (got[end:] == 7.0).all()


@pytest.mark.parametrize("lens", [[1], [2], [21], [22], [63, 0, 64, 65], [127], [128], [129], [255, 257], [42, 43],
                                  [0, 0, 5, 0], [1] * 40, [300, 1, 700], [1025]])
@pytest.mark.parametrize("hq,hkv", [(24, 4), (4, 1), (2, 2)])
def test_prompt_attn_lengths(lens, hq, hkv):
    q, k, v = _qkv(_gen(len(lens) * 7 + hq), sum(lens), hq, hkv)
    _check_attn(q, k, v, lens)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (7, 1), (12, 1), (16, 2), (24, 1), (32, 2), (48, 1),
                                    (64, 1), (100, 1), (128, 1), (8, 8), (40, 8)])
def test_prompt_attn_head_layouts(hq, hkv):
    lens = [150, 3, 260]
    q, k, v = _qkv(_gen(hq), sum(lens), hq, hkv, fused=True)
    _check_attn(q, k, v, lens)


@pytest.mark.parametrize("lens", [[256], [257], [383], [384], [385], [511, 130], [640, 1, 900], [2048], [3001]])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (1, 1), (12, 2), (7, 1)])
def test_prompt_attn_few_long_tiles(lens, hq, hkv):
    """Fewer tiles than SMs, of every number of blocks; flat and peaked scores."""
    q, k, v = _qkv(_gen(len(lens) + 10 * hq), sum(lens), hq, hkv)
    _check_attn(q, k, v, lens)
    k[:, :, ::32] *= 16.0
    _check_attn(q, k, v, lens)


def test_prompt_attn_rows_outside_the_lanes_are_left():
    """Lanes that start behind row 0 and end before the last row; the rows
    around them hold NaN, which reaches nothing."""
    lens, start = [70, 130], 9
    q, k, v = _qkv(_gen(3), 230, 6, 2)
    for x in (q, k, v):
        x[:start] = NAN
        x[start + 200:] = NAN
    _check_attn(q, k, v, lens, start=start)


def test_prompt_attn_long_and_many():
    g = _gen(11)
    q, k, v = _qkv(g, 5000, 8, 2, fused=True)
    _check_attn(q, k, v, [5000])
    lens = [int(x) for x in torch.randint(0, 12, (1000,), generator=torch.Generator().manual_seed(2))]
    q, k, v = _qkv(g, sum(lens), 6, 1)
    _check_attn(q, k, v, lens)


@pytest.mark.parametrize("gain", [0.0, 1e-3, 30.0])
def test_prompt_attn_flat_and_peaked(gain):
    """Equal scores, nearly equal ones, and one key that takes all; maxima
    that grow along the row, so that the running one is outgrown often."""
    q, k, v = _qkv(_gen(5), 700, 4, 2)
    q = (q * gain).to(torch.bfloat16)
    k = (k * torch.linspace(0.1, 1.0, 700, device="cuda")[:, None, None]).to(torch.bfloat16)
    _check_attn(q, k, v, [333, 367])


def test_prompt_attn_infinities_and_nan_stay_behind_the_mask():
    """A row sees only rows up to its own: whatever follows it, in its lane or
    the next, leaves it bit for bit as it was.  Rows that do see it are NaN
    (a NaN key or value, opposite infinities) or infinite (one infinity in V)."""
    lens = [200, 150]
    q, k, v = _qkv(_gen(6), 350, 6, 2)
    cu = _cu(lens)
    out0, lse0 = _run_attn(q, k, v, cu)
    for at, name, value in ((150, "v", NAN), (150, "v", INF), (131, "v", -INF), (199, "k", NAN), (60, "k", INF),
                            (10, "q", NAN), (0, "v", INF), (349, "v", NAN), (200, "v", INF)):
        x = {"q": q, "k": k, "v": v}
        x[name] = x[name].clone()
        x[name][at, -1, 5] = value
        out, lse = _run_attn(x["q"], x["k"], x["v"], cu)
        end = 200 if at < 200 else 350
        rows = torch.zeros(350, dtype=torch.bool, device="cuda")
        rows[at:end] = name != "q"
        rows[at] = True
        heads = slice(5, 6) if name == "q" else slice(3, 6)
        same = torch.ones_like(out, dtype=torch.bool)
        same[rows, heads] = False
        assert torch.equal(out[same], out0[same]), (at, name, value)
        got = out[rows, heads]
        if name == "v":
            assert torch.equal(lse, lse0)
            assert torch.equal(got[..., :5], out0[rows, heads][..., :5])
            assert torch.equal(got[..., 6:], out0[rows, heads][..., 6:])
            hit = got[..., 5]
            # a weight that underflows to 0 makes 0 * inf a NaN, as the formula in floating point does
            assert (hit.isnan() if value != value else (hit == value) | hit.isnan()).all()
            assert value != value or hit[0].isinf().all()
        elif value != value:
            assert got.isnan().all() and lse[rows, heads].isnan().all()


def test_prompt_attn_first_keys_without_weight():
    """Scores of -inf over the whole first block of keys and more: the rows
    behind them weigh the other keys alone; rows that see nothing else are NaN
    with lse -inf, as the formula's 0 / 0."""
    q, k, v = _qkv(_gen(12), 400, 4, 2)
    q[:, :, 0] = 1.0
    k[:150, :, 0] = -INF
    out, lse = _run_attn(q, k, v, _cu([400]))
    assert out[:150].isnan().all() and (lse[:150] == -INF).all()
    for t in (150, 151, 260, 399):
        want, wl, to, tl = _attn_ref(q[150:t + 1], k[150:t + 1], v[150:t + 1], [t - 149], float(SM_SCALE))
        assert ((out[t].double() - want[-1]).abs() <= to[-1]).all()
        assert ((lse[t].double() - wl[-1]).abs() <= tl[-1]).all()


@pytest.mark.parametrize("lens", [[1501, 999, 2047, 3], [4000]])
def test_prompt_attn_outlier_channels(lens):
    """A few key channels eight times the rest, as real models have them."""
    q, k, v = _qkv(_gen(13), sum(lens), 8, 4)
    k[:, :, ::32] *= 8.0
    _check_attn(q, k, v, lens)


@pytest.mark.parametrize("hq,hkv", [(24, 4), (8, 8), (16, 1)])
def test_prompt_attn_rows_keep_their_bits(hq, hkv):
    """A row's bits depend on its lane's rows up to it alone: not on the rows
    behind them, nor on the other lanes.  Of one key the output is its value."""
    q, k, v = _qkv(_gen(21), 1000, hq, hkv)
    out, lse = _run_attn(q, k, v, _cu([1000]))
    assert torch.equal(out[0], v[0].repeat_interleave(hq // hkv, 0))
    for n in (1, 5, 127, 128, 129, 300, 999):
        o, z = _run_attn(q[:n], k[:n], v[:n], _cu([n]))
        assert torch.equal(o, out[:n]) and torch.equal(z, lse[:n]), n
    junk = torch.randn_like(q[:700])
    kv = torch.randn_like(k[:700])
    o, z = _run_attn(torch.cat([junk, q]), torch.cat([kv, k]), torch.cat([kv, v]), _cu([1, 400, 299, 1000]))
    assert torch.equal(o[700:], out) and torch.equal(z[700:], lse)


def test_prompt_attn_opposite_infinities():
    q, k, v = _qkv(_gen(7), 100, 2, 1)
    v[40, 0, 3], v[45, 0, 3] = INF, -INF
    out, _ = _run_attn(q, k, v, _cu([100]))
    c = out[:, :, 3]
    assert c[:40].isfinite().all() and (c[40:45] == INF).all() and c[45:].isnan().all()


@pytest.mark.parametrize("cu", [[0, 5, 4, 10], [-1, 5, 6, 10], [0, 5, 6, 11], [3, 2, 1, 0], [0, 11, 10, 10]])
def test_bad_offsets_write_nothing(cu):
    import speculative_decode_verify_append_gb300 as sdva
    q, k, v = _qkv(_gen(1), 10, 4, 2)
    cu, st = torch.tensor(cu, dtype=torch.int32, device="cuda"), _status()
    out, lse = _run_attn(q, k, v, cu, status=st)
    assert int(st.item()) == sdva.STATUS_BAD_COUNT and (out == 7.0).all() and (lse == 7.0).all()
    for kind in ALL_KV:
        cache, st = sdva.KVCache(kind, 4, 2), _status()
        for x in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
            x.fill_(3)
        table = torch.arange(3, dtype=torch.int32, device="cuda").view(3, 1)
        sdva.kv_append_packed(cache, k, v, cu, table, torch.zeros(3, dtype=torch.int32, device="cuda"), st)
        assert int(st.item()) == sdva.STATUS_BAD_COUNT
        assert all((x == 3).all() for x in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))


def test_prompt_attn_runs_repeat_bit_for_bit_and_replay():
    """Twice eager, on another stream, and replayed from a graph with new
    inputs in the same buffers; without lse."""
    import speculative_decode_verify_append_gb300 as sdva
    lens = [700, 1, 333, 64]
    q, k, v = _qkv(_gen(8), sum(lens), 12, 2)
    cu = _cu(lens)
    a, la = _run_attn(q, k, v, cu)
    b, lb = _run_attn(q, k, v, cu)
    assert torch.equal(a, b) and torch.equal(la, lb)
    out = torch.empty_like(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sdva.prompt_attn(q, k, v, cu, float(SM_SCALE), out, stream=s)
    s.synchronize()
    assert torch.equal(a, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdva.prompt_attn(q, k, v, cu, float(SM_SCALE), out)
    q.copy_(torch.randn_like(q))
    cu.copy_(_cu([10, 600, 488, 0]))
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _run_attn(q, k, v, cu)
    assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# kv_append_packed
# ---------------------------------------------------------------------------
def _oracle_append(cache, k, v, lens, table, cached):
    a = 0
    for b, n in enumerate(lens):
        if n:
            st = oracle.append(cache, k[None, a:a + n], v[None, a:a + n], table[b:b + 1],
                               np.array(cached[b:b + 1], np.int32))
            assert st == 0
        a += n


def _packed_case(kind, lens, cached, hkv, seed, fused=False):
    """A cache that holds `cached` tokens a lane, on the GPU and in the oracle, and new packed rows."""
    import speculative_decode_verify_append_gb300 as sdva
    rng = np.random.default_rng(seed)
    need = [-(-(c + n) // 64) for c, n in zip(cached, lens)]
    row = max(max(need), 1)
    ids = rng.permutation(sum(need) + 2).astype(np.int32)
    table = np.full((len(lens), row), -7, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    gc, oc = sdva.KVCache(kind, len(ids), hkv), oracle.Cache(kind, len(ids), hkv)
    st = _status()
    for rows, done in ((cached, [0] * len(lens)), (lens, cached)):
        k, v = (synth.to_bf16_bits(rng.standard_normal((sum(rows), hkv, D), dtype=np.float32) *
                                   np.exp2(rng.integers(-3, 4, (sum(rows), 1, 1))).astype(np.float32)) for _ in "kv")
        dk, dv = bf16_dev(k), bf16_dev(v)
        if fused:
            both = torch.cat([dk, dv], 1)
            dk, dv = both[:, :hkv], both[:, hkv:]
        sdva.kv_append_packed(gc, dk, dv, _cu(rows), i32_dev(table), i32_dev(np.array(done)), st)
        _oracle_append(oc, k, v, rows, table, done)
    assert int(st.item()) == 0
    return gc, oc


@pytest.mark.parametrize("kind", ALL_KV, ids=[KV_NAMES[k] for k in ALL_KV])
@pytest.mark.parametrize("lens,cached", [([1], [0]), ([64], [0]), ([65], [0]), ([130], [0]), ([5, 0, 7], [0, 30, 63]),
                                         ([64, 64], [1, 63]), ([2, 66, 200], [63, 63, 100]),
                                         ([0, 1, 0, 300, 0], [0, 64, 5, 31, 128])])
def test_packed_append_matches_the_oracle(kind, lens, cached):
    gc, oc = _packed_case(kind, lens, cached, 3, 17 + len(lens), fused=len(lens) % 2 == 1)
    host = cache_to_host(gc)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        want = getattr(oc, name)
        assert np.array_equal(host[name].view(np.uint8), np.ascontiguousarray(want).view(np.uint8)), name


@pytest.mark.parametrize("kind", ALL_KV, ids=[KV_NAMES[k] for k in ALL_KV])
def test_packed_append_equals_single_lane_calls(kind):
    """Forty lanes of 0 .. 400 tokens in one call, against kv_append_quant lane by lane."""
    import speculative_decode_verify_append_gb300 as sdva
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 400, 40)]
    lens[3] = lens[39] = 0
    cached = [int(x) for x in rng.integers(0, 200, 40)]
    T, row = sum(lens), 12
    table = torch.from_numpy(rng.permutation(40 * row).astype(np.int32).reshape(40, row)).cuda()
    g = _gen(9)
    _, k, v = _qkv(g, T, 1, 4, fused=True)
    k[::7] *= 4.0
    caches = [sdva.KVCache(kind, 40 * row, 4) for _ in range(2)]
    pre_k, pre_v = (torch.randn((40, 200, 4, D), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    zero = torch.zeros(40, dtype=torch.int32, device="cuda")
    for c in caches:
        sdva.kv_append_quant_ragged(c, pre_k, pre_v, i32_dev(np.array(cached)), table, zero)
    st = _status()
    sdva.kv_append_packed(caches[0], k, v, _cu(lens), table, i32_dev(np.array(cached)), st)
    a = 0
    for b, n in enumerate(lens):
        if n:
            sdva.kv_append_quant(caches[1], k[None, a:a + n].contiguous(), v[None, a:a + n].contiguous(),
                                 table[b:b + 1], i32_dev(np.array(cached[b:b + 1])))
        a += n
    assert int(st.item()) == 0
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(getattr(caches[0], name).view(torch.uint8), getattr(caches[1], name).view(torch.uint8)), name


@pytest.mark.parametrize("kind", ALL_KV, ids=[KV_NAMES[k] for k in ALL_KV])
def test_packed_append_skips_bad_lanes_alone(kind):
    """A lane that does not fit, one with a bad page id, one with a negative
    length: each flagged and left; the others written."""
    import speculative_decode_verify_append_gb300 as sdva
    lens = [70, 70, 70, 70, 0]
    _, k, v = _qkv(_gen(2), sum(lens), 1, 2)
    table = torch.tensor([[0, 1], [2, 3], [4, 99], [6, 7], [-1, -1]], dtype=torch.int32, device="cuda")
    st, cache = _status(), sdva.KVCache(kind, 8, 2)
    sdva.kv_append_packed(cache, k, v, _cu(lens), table, i32_dev(np.array([10, 100, 0, -1, 500])), st)
    assert int(st.item()) == sdva.STATUS_OVERFLOW | sdva.STATUS_BAD_PAGE
    assert cache.k_codes[:2].any() and cache.v_codes[:2].any()
    for x in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
        assert not x[2:].any()


def test_packed_append_hostile_values():
    """Zeros of both signs, the smallest subnormals, the largest finite
    values: codes and scales as the oracle's in every format."""
    import speculative_decode_verify_append_gb300 as sdva
    bits = np.array([0x0000, 0x8000, 0x0001, 0x8001, 0x0080, 0x7F7F, 0xFF7F, 0x3F80, 0xBF81, 0x4000], np.uint16)
    rng = np.random.default_rng(1)
    x = rng.choice(bits, (96, 2, D))
    x[:20] = rng.choice(bits[:2], (20, 2, D))
    x[20:40] = rng.choice(bits[:4], (20, 2, D))
    x[64:] = rng.choice(bits[:5], (32, 2, D))
    table = np.array([[1, 0]], np.int32)
    for kind in ALL_KV:
        gc, oc = sdva.KVCache(kind, 2, 2), oracle.Cache(kind, 2, 2)
        sdva.kv_append_packed(gc, bf16_dev(x), bf16_dev(x[::-1]), _cu([96]), i32_dev(table), i32_dev(np.array([0])))
        assert oracle.append(oc, x[None], x[None, ::-1].copy(), table, np.array([0], np.int32)) == 0
        host = cache_to_host(gc)
        for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
            assert np.array_equal(host[name].view(np.uint8), np.ascontiguousarray(getattr(oc, name)).view(np.uint8)), (
                KV_NAMES[kind], name)


@pytest.mark.parametrize("exponent", [127, 127 - 75, 127 + 100])
@pytest.mark.parametrize("kind", ALL_KV, ids=[KV_NAMES[k] for k in ALL_KV])
def test_packed_append_every_significand(kind, exponent):
    """Every bf16 significand under every scale significand (a scale comes from
    a bf16 maximum), the values 0 .. 13 binades below it: the codes' quotients
    are exact where the kernel replaces the division, and where it does not."""
    import speculative_decode_verify_append_gb300 as sdva
    m = np.arange(128, dtype=np.uint32)
    a, e = np.repeat(m, 14), np.tile(np.arange(14, dtype=np.uint32), 128)
    top = (exponent << 7) | a
    x = ((exponent - e[:, None]) << 7) | m[None, :]
    x = np.minimum(x, top[:, None])
    x[:, ::32] = top[:, None]
    x = (x | ((m & 1) << 15)[None, :]).astype(np.uint16)[:, None, :]
    n = x.shape[0]
    pages = n // 64
    # page scales: one maximum to a page, so the pages' rows share theirs
    if kind == synth.KV_FP8:
        x = np.sort(x.view(np.int16), axis=0).view(np.uint16)
    table = np.arange(pages, dtype=np.int32)[None]
    gc, oc = sdva.KVCache(kind, pages, 1), oracle.Cache(kind, pages, 1)
    st = _status()
    sdva.kv_append_packed(gc, bf16_dev(x), bf16_dev(x[:, :, ::-1]), _cu([n]), i32_dev(table), i32_dev(np.array([0])),
                          st)
    assert oracle.append(oc, x[None], x[None, :, :, ::-1].copy(), table, np.array([0], np.int32)) == 0
    assert int(st.item()) == 0
    host = cache_to_host(gc)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert np.array_equal(host[name].view(np.uint8), np.ascontiguousarray(getattr(oc, name)).view(np.uint8)), name


# ---------------------------------------------------------------------------
# token_logprobs
# ---------------------------------------------------------------------------
def _score(logits, tokens, top, status=None):
    import speculative_decode_verify_append_gb300 as sdva
    lead = tuple(tokens.shape)
    lp, en = (torch.full(lead, 7.0, device="cuda") for _ in range(2))
    tt = torch.full(lead + (top,), 77, dtype=torch.int32, device="cuda") if top else None
    tl = torch.full(lead + (top,), 7.0, device="cuda") if top else None
    sdva.token_logprobs(logits, tokens, lp, en, tt, tl, status)
    torch.cuda.synchronize()
    return lp, en, tt, tl


def _order(x, top):
    """The first `top` indices by (value descending, index ascending), NaN last."""
    x = x.double() + 0.0
    key = torch.where(x.isnan(), torch.tensor(-INF, dtype=torch.float64, device=x.device), x)
    nan = x.isnan().to(torch.int8)
    idx = torch.argsort(key, dim=-1, descending=True, stable=True)
    idx = idx.gather(-1, torch.argsort(nan.gather(-1, idx), dim=-1, stable=True))
    return idx[..., :top]


def _check_scores(logits, tokens, top):
    """Bounds: S adds V terms in fp32, no thread more than V / 128 + 64 of
    them in a row (2^-24 each); a term's exponent d log2 e is rounded
    (|d| 2^-23 of the term) and exp2 is off by 2^-22.  So S is off by
    c = 2^-22 (V / 512 + 32) (1 + E|d|) of itself, T / S by the same with
    E|d| + E d^2, and a log probability by c plus the rounding of its two
    terms."""
    st = _status()
    lp, en, tt, tl = _score(logits, tokens, top, st)
    assert int(st.item()) == 0
    x = logits.double()
    V = x.shape[-1]
    on = tokens >= 0
    t = tokens.clamp(min=0).long()
    x = x - x.amax(-1, keepdim=True)  # first: near the type's lowest value the difference alone is exact
    z = x.logsumexp(-1, keepdim=True)
    p = (x - z).exp()
    d = torch.where(p > 0, x, 0.0)
    ed, ed2 = (p * d.abs()).sum(-1), (p * d * d).sum(-1)
    ent = z.squeeze(-1) + ed
    c = 2.0 ** -22 * (V / 512 + 32)
    want = torch.where(on, (x.gather(-1, t[..., None]) - z).squeeze(-1), 0.0)

    def near(got, want, tol, what):
        same = (got.double() == want) | ((got.double() - want).abs() <= tol)
        assert same.all(), (what, (~same).nonzero()[:4].tolist(), got[~same][:4].tolist(), want[~same][:4].tolist())

    tol = c * (1 + ed) + 2.0 ** -22 * (1 + z.squeeze(-1))
    near(lp, want, tol + 2.0 ** -22 * want.abs().nan_to_num(posinf=0.0), "logprobs")
    near(en, torch.where(on, ent, 0.0), c * (1 + 2 * ed + ed2) + 2.0 ** -22 * (1 + ent), "entropy")
    if top:
        idx = _order(logits, top)
        assert torch.equal(tt, torch.where(on[..., None], idx, -1).to(torch.int32))
        want = torch.where(on[..., None], x.gather(-1, idx) - z, 0.0)
        near(tl, want, tol[..., None] + 2.0 ** -22 * want.abs().nan_to_num(posinf=0.0), "top_logprobs")


def _logits(g, n, V, dtype, spread=3.0):
    x = torch.randn((n, V), generator=g, device="cuda") * spread * torch.rand((n, 1), generator=g, device="cuda")
    return x.to(dtype)


DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,V,top", [(1, 1, 1), (1, 7, 7), (3, 32, 32), (5, 33, 32), (2, 100, 0), (4, 1000, 5),
                                     (1, 4096, 20), (7, 5003, 8), (3, 32001, 32), (200, 257, 3), (1, 151936, 20),
                                     (9, 151936, 5), (130, 65537, 1), (600, 8191, 2)])
def test_token_logprobs_sizes(dtype, n, V, top):
    g = _gen(n + V)
    x = _logits(g, n, V, dtype)
    tokens = torch.randint(V, (n,), generator=g, device="cuda", dtype=torch.int32)
    _check_scores(x, tokens, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,V,top", [(330, 9999, 4), (400, 16003, 32), (160, 32001, 5), (609, 16003, 5), (20, 8195, 1),
                                     (300, 16383, 0)])
def test_token_logprobs_short_rows_few_and_many(dtype, n, V, top):
    """Blocks with eight and with four vectors in flight, alone and in clusters."""
    g = _gen(V + n)
    x = _logits(g, n, V, dtype)
    x[::7, ::3] = -INF
    tokens = torch.randint(V, (n,), generator=g, device="cuda", dtype=torch.int32)
    _check_scores(x, tokens, top)


@pytest.mark.parametrize("dtype", DTYPES)
def test_token_logprobs_strided_and_unaligned_rows(dtype):
    """Rows behind one another with a gap, starting at an odd element."""
    g = _gen(4)
    big = _logits(g, 6, 10007, dtype)
    tokens = torch.randint(5000, (6,), generator=g, device="cuda", dtype=torch.int32)
    for lo, V in ((0, 10000), (1, 9999), (3, 5001), (8, 9984)):
        _check_scores(big[:, lo:lo + V], tokens, 6)
    wide = _logits(g, 6, 5120, dtype)
    _check_scores(wide[:, 16:5000 + 16], tokens, 6)


@pytest.mark.parametrize("V", [64, 1500, 20000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_token_logprobs_ties_and_orders(dtype, V):
    """Rows of one value, of few values, rising and falling ones, zeros of
    both signs, one token far above the rest, the type's lowest values."""
    g = _gen(V)
    lowest = torch.finfo(dtype).min
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    rows = [torch.zeros(V, device="cuda"), torch.randint(3, (V,), generator=g, device="cuda").float(), i / V * 8,
            -i / V * 8, torch.where(torch.rand(V, generator=g, device="cuda") < 0.5, 0.0, -0.0),
            torch.where(i == V - 1, 60.0, 0.0), torch.full((V,), lowest, device="cuda"),
            torch.where(i % 5 == 3, torch.randn(V, generator=g, device="cuda"), torch.full_like(i, lowest)),
            torch.randn(V, generator=g, device="cuda").round() * 0.25, i % 16]
    x = torch.stack(rows).to(dtype)
    tokens = torch.randint(V, (len(rows),), generator=g, device="cuda", dtype=torch.int32)
    for top in (1, 20, 32):
        _check_scores(x, tokens, top)


@pytest.mark.parametrize("share", [0.5, 0.99, 1.0])
def test_token_logprobs_forbidden_tokens(share):
    """-inf entries: probability 0, no part in the entropy; a row may keep one
    token only, and the list goes on with forbidden ones by index."""
    g = _gen(3)
    x = _logits(g, 8, 3001, torch.float32)
    x[torch.rand(x.shape, generator=g, device="cuda") < share] = -INF
    keep = torch.randint(3001, (8,), generator=g, device="cuda")
    x[torch.arange(8, device="cuda"), keep] = 1.5
    tokens = keep.to(torch.int32)
    tokens[::2] = 17
    _check_scores(x, tokens, 10)


def test_token_logprobs_rows_without_a_distribution():
    """All -inf, a NaN, +inf: NaN scores, and the list in order, NaN last."""
    x = torch.randn((6, 2100), generator=_gen(1), device="cuda")
    x[0] = -INF
    x[1, 700] = NAN
    x[2, 2099] = INF
    x[3] = NAN
    x[4, 5:] = NAN
    tokens = torch.full((6,), 3, dtype=torch.int32, device="cuda")
    lp, en, tt, tl = _score(x, tokens, 9)
    assert lp[:5].isnan().all() and en[:5].isnan().all() and tl[:5].isnan().all()
    assert lp[5].isfinite() and en[5].isfinite() and tl[5].isfinite().all()
    assert torch.equal(tt, _order(x, 9).to(torch.int32))


def test_token_logprobs_rows_that_are_not_scored():
    """-1 rows are not read (NaN there changes nothing) and give 0, -1; other
    ids outside the vocabulary are flagged and give the same."""
    import speculative_decode_verify_append_gb300 as sdva
    x = torch.randn((4, 3, 999), generator=_gen(1), device="cuda")
    x[1, 1] = NAN
    tokens = torch.randint(999, (4, 3), dtype=torch.int32, device="cuda")
    tokens[1, 1] = tokens[3, 2] = -1
    st = _status()
    lp, en, tt, tl = _score(x, tokens, 4, st)
    assert int(st.item()) == 0
    off = tokens < 0
    assert not lp[off].any() and not en[off].any() and (tt[off] == -1).all() and not tl[off].any()
    assert lp[~off].isfinite().all() and (lp[~off] < 0).all()
    tokens[0, 0], tokens[2, 2] = 999, -5
    lp2, en2, tt2, tl2 = _score(x, tokens, 4, st)
    assert int(st.item()) == sdva.STATUS_BAD_DRAFT
    off2 = (tokens < 0) | (tokens >= 999)
    assert not lp2[off2].any() and not en2[off2].any() and (tt2[off2] == -1).all() and not tl2[off2].any()
    on = ~off2
    assert torch.equal(lp2[on], lp[on]) and torch.equal(en2[on], en[on]) and torch.equal(tt2[on], tt[on])


@pytest.mark.parametrize("dtype", DTYPES)
def test_token_logprobs_rows_that_stream_past_long_lists(dtype):
    """Several rows to a block, lists of 32: the end of a row takes longer than
    the next row's copies, which must not overtake its readers."""
    g = _gen(58)
    x = _logits(g, 1000, 58010, dtype)
    tokens = torch.randint(58010, (1000,), generator=g, device="cuda", dtype=torch.int32)
    for _ in range(3):
        _check_scores(x, tokens, 32)


@pytest.mark.parametrize("n", [1, 40])
def test_token_logprobs_without_the_optional_outputs_and_replayed(n):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(n)
    x = _logits(g, n, 40000, torch.float32)
    tokens = torch.randint(40000, (n,), generator=g, device="cuda", dtype=torch.int32)
    lp0, en0, tt0, tl0 = _score(x, tokens, 7)
    lp = torch.empty(n, device="cuda")
    sdva.token_logprobs(x, tokens, lp)
    assert torch.equal(lp, lp0)
    en, tt, tl = torch.empty_like(lp), torch.empty_like(tt0), torch.empty_like(tl0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdva.token_logprobs(x, tokens, lp, en, tt, tl)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lp, lp0) and torch.equal(en, en0) and torch.equal(tt, tt0) and torch.equal(tl, tl0)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ALL_KV, ids=[KV_NAMES[k] for k in ALL_KV])
def test_prompts_into_verify_steps(kind):
    """Prompts packed into the cache in one pass, then a verify step and the
    scores of its tokens, all in one captured graph: the cache and the step's
    results are those of lane-by-lane appends, byte for byte."""
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import PromptStep, VerifyStep, fill_context
    lens, hq, hkv, W, V = [300, 1, 64, 129], 12, 2, 4, 5003
    B, T = len(lens), sum(lens)
    g = _gen(21)
    q, k, v = _qkv(g, T, hq, hkv, fused=True)
    rows = 8
    table = torch.randperm(B * rows, generator=g, device="cuda").to(torch.int32).view(B, rows)
    win = [torch.randn((B, W, n, D), generator=g, device="cuda").to(torch.bfloat16) for n in (hq, hkv, hkv)]
    logits = torch.randn((B, W, V), generator=g, device="cuda") * 3
    drafts = logits[:, :-1].argmax(-1).to(torch.int32)
    drafts[0, 1] = drafts[2, 0] = 7
    caches = [sdva.KVCache(kind, B * rows, hkv) for _ in range(2)]
    prompt = PromptStep(T + 50, hq)
    steps = [VerifyStep(B, W, hq, hkv, 512, V, num_top=6) for _ in range(2)]
    zero, cu = torch.zeros(B, dtype=torch.int32, device="cuda"), _cu(lens)
    seq = [torch.tensor(lens, dtype=torch.int32, device="cuda") for _ in range(2)]

    def one_pass():
        out, lse = prompt.run(caches[0], q, k, v, cu, table, zero)
        steps[0].append(caches[0], win[1], win[2], table, seq[0])
        steps[0].attend(caches[0], win[0], table, seq[0])
        steps[0].accept_lazy(logits, drafts)
        steps[0].score(logits)
        return out, lse

    one_pass()  # eager, also before a capture loads the code
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = one_pass()
    out.fill_(7.0)
    steps[0].out.fill_(7.0)
    steps[0].logprobs.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert int(prompt.status.item()) == 0 and int(steps[0].status.item()) == 0

    a = 0
    for b, n in enumerate(lens):
        fill_context(caches[1], k[a:a + n].contiguous(), v[a:a + n].contiguous(), table[b])
        a += n
    steps[1].append(caches[1], win[1], win[2], table, seq[1])
    steps[1].attend(caches[1], win[0], table, seq[1])
    steps[1].accept_lazy(logits, drafts)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        x, y = (getattr(c, name)[table.long()[torch.arange(B), [n // 64 for n in lens]]] for c in caches)
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name
    assert torch.equal(steps[0].out, steps[1].out)
    assert torch.equal(steps[0].out_tokens, steps[1].out_tokens)
    assert torch.equal(steps[0].accept_len, steps[1].accept_len)
    ro, rl, to, tl = _attn_ref(q, k, v, lens, float(SM_SCALE))
    assert ((out.double() - ro).abs() <= to).all() and ((lse.double() - rl).abs() <= tl).all()
    tok = steps[0].out_tokens
    on = tok >= 0
    assert on.sum(-1).tolist() == (steps[0].accept_len + 1).tolist()
    lp = logits.double().log_softmax(-1)
    want = lp.gather(-1, tok.clamp(min=0).long()[..., None]).squeeze(-1)
    # 2^-22 (V / 512 + 32) of the sum, as in _check_scores, with E|d| below 64 here
    assert ((steps[0].logprobs.double() - want).abs()[on] <= 2.0 ** -22 * (V / 512 + 32) * 65).all()
    assert not steps[0].logprobs[~on].any() and (steps[0].top_tokens[~on] == -1).all()
    assert torch.equal(steps[0].top_tokens[on], _order(logits, 6)[on].to(torch.int32))


def test_prompt_rows_agree_with_the_cache():
    """The last rows of a prompt by prompt_attn, and by verify_attn as a window
    over the INT8 cache that kv_append_packed filled.

    Bounds.  A cached element is off by at most half a step of its group's
    scale, s / 2 <= amax / 254 (1 + 2^-11), and once more by 2^-11 of itself
    when it is widened to fp16; a score then by e = scale * sum |q| (amax_K / 253 +
    2^-11 amax_K), a weight by a factor within exp(+-2e), an output by
    amax_V (1 / 253 + 2^-11) more.  Weights and outputs are rounded on both
    sides (2^-8 of sum p |v| and of the output each; q to fp16, 2^-11, on one)."""
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import PromptStep, VerifyStep
    lens, hq, hkv, W = [500, 77], 6, 2, 5
    q, k, v = _qkv(_gen(31), sum(lens), hq, hkv)
    cache = sdva.KVCache(sdva.KV_INT8_G64, 20, hkv)
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    prompt = PromptStep(sum(lens), hq)
    out, _ = prompt.run(cache, q, k, v, _cu(lens), table, torch.zeros(2, dtype=torch.int32, device="cuda"))
    step = VerifyStep(2, W, hq, hkv, 512, None)
    last = torch.tensor([list(range(n - W, n)) for n in (500, 577)], device="cuda")
    step.attend(cache, q[last].contiguous(), table,
                torch.tensor([n - W for n in lens], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(prompt.status.item()) == 0 and int(step.status.item()) == 0
    scale = float(SM_SCALE)
    for b, (start, n) in enumerate(((0, 500), (500, 77))):
        for i in range(W):
            t = start + n - W + i
            for h in range(hq):
                kk, vv = k[start:t + 1, h // 3].double(), v[start:t + 1, h // 3].double()
                qq = q[t, h].double()
                p = (kk @ qq * scale).softmax(0)
                e = scale * float(qq.abs().sum()) * float(kk.abs().max()) * (1 / 253 + 2.0 ** -11 + 2.0 ** -11)
                av = p @ vv.abs()
                tol = (math.expm1(2 * e) + 2 * 2.0 ** -8) * av + float(vv.abs().max()) * (1 / 253 + 2.0 ** -11) + \
                    2 * 2.0 ** -8 * (p @ vv).abs()
                err = (out[t, h].double() - step.out[b, i, h].double()).abs()
                assert (err <= tol).all(), (b, i, h, float((err / tol).max()))


# ---------------------------------------------------------------------------
# arguments
# ---------------------------------------------------------------------------
def test_refusals_of_the_binding():
    import speculative_decode_verify_append_gb300 as sdva
    q, k, v = _qkv(_gen(1), 10, 4, 2)
    cu = _cu([10])
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        sdva.prompt_attn(q.float(), k, v, cu, 0.1, out)
    with pytest.raises(ValueError):
        sdva.prompt_attn(q, k[:9], v, cu, 0.1, out)
    with pytest.raises(ValueError):
        sdva.prompt_attn(q, k, v[:, :1], cu, 0.1, out)
    with pytest.raises(ValueError):
        sdva.prompt_attn(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cu, 0.1, out)
    with pytest.raises(ValueError):
        sdva.prompt_attn(q, k, v, cu.long(), 0.1, out)
    with pytest.raises(ValueError):
        sdva.prompt_attn(q, k, v, cu, 0.1, out[:, ::2])
    with pytest.raises(ValueError):
        sdva.prompt_attn(q, k, v, cu.cpu(), 0.1, out)
    for scale in (0.0, -1.0, NAN, INF):
        with pytest.raises(sdva.SdvaError) as e:
            sdva.prompt_attn(q, k, v, cu, scale, out)
        assert e.value.code == sdva.ERR_INVALID
    with pytest.raises(sdva.SdvaError) as e:  # 129 q heads to a kv head
        sdva.prompt_attn(*_qkv(_gen(1), 2, 129, 1), cu, 0.1,
                         torch.empty((2, 129, D), dtype=torch.bfloat16, device="cuda"))
    assert e.value.code == sdva.ERR_UNSUPPORTED
    cache = sdva.KVCache(sdva.KV_FP8_E4M3, 2, 2)
    table, lens = i32_dev(np.array([[0, 1]])), i32_dev(np.array([0]))
    with pytest.raises(ValueError):
        sdva.kv_append_packed(cache, k[:, :1], v[:, :1], cu, table, lens)
    with pytest.raises(ValueError):
        sdva.kv_append_packed(cache, k, v, _cu([5, 5]), table, lens)
    with pytest.raises(ValueError):
        sdva.kv_append_packed(cache, k, v, cu, i32_dev(np.array([[0], [1]])), lens)
    x, t, lp = torch.randn((3, 50), device="cuda"), i32_dev(np.array([1, 2, 3])), torch.empty(3, device="cuda")
    with pytest.raises(ValueError):
        sdva.token_logprobs(x.double(), t, lp)
    with pytest.raises(ValueError):
        sdva.token_logprobs(x, t[:2], lp)
    with pytest.raises(ValueError):
        sdva.token_logprobs(x.T.contiguous().T, t, lp)
    with pytest.raises(ValueError):
        sdva.token_logprobs(x, t, lp, None, torch.empty((3, 2), dtype=torch.int32, device="cuda"))
    from speculative_decode_verify_append_gb300.step import VerifyStep
    with pytest.raises(ValueError):
        VerifyStep(1, 1, 4, 2, 64, 50).score(x[:1].view(1, 1, 50))
    for top, code in ((33, sdva.ERR_UNSUPPORTED), (51, sdva.ERR_INVALID)):
        with pytest.raises(sdva.SdvaError) as e:
            sdva.token_logprobs(x, t, lp, None, torch.empty((3, top), dtype=torch.int32, device="cuda"),
                                torch.empty((3, top), device="cuda"))
        assert e.value.code == code


def test_empty_calls_do_nothing():
    import speculative_decode_verify_append_gb300 as sdva
    q, k, v = _qkv(_gen(1), 0, 4, 2)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    sdva.prompt_attn(q, k, v, cu, 0.1, torch.empty_like(q), torch.empty((0, 4), device="cuda"))
    cache = sdva.KVCache(sdva.KV_INT8_G64, 2, 2)
    sdva.kv_append_packed(cache, k, v, cu, i32_dev(np.array([[0], [1]])), i32_dev(np.array([0, 0])))
    e = torch.empty(0, device="cuda")
    sdva.token_logprobs(torch.empty((0, 9), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), e, e)
    torch.cuda.synchronize()


def test_shapes_with_the_wrong_number_of_axes_are_refused():
    import speculative_decode_verify_append_gb300 as sdva
    q, k, v = _qkv(_gen(1), 10, 4, 2)
    cu, out = _cu([10]), torch.empty_like(q)
    cache = sdva.KVCache(sdva.KV_INT4_G32, 1, 2)
    table, lens = i32_dev(np.array([[0]])), i32_dev(np.array([0]))
    for bad in (k.view(10, -1), k[None]):
        with pytest.raises(ValueError):
            sdva.kv_append_packed(cache, bad, v, cu, table, lens)
        with pytest.raises(ValueError):
            sdva.kv_append_packed(cache, k, bad, cu, table, lens)
        with pytest.raises(ValueError):
            sdva.prompt_attn(q, bad, v, cu, 0.1, out)
    with pytest.raises(ValueError):
        sdva.kv_append_packed(cache, k, v, cu, table[0], lens)
    with pytest.raises(ValueError):
        sdva.kv_append_packed(cache, k, v, cu, table, lens[0])
    with pytest.raises(ValueError):
        sdva.prompt_attn(q, k, v, cu[0], 0.1, out)
    with pytest.raises(ValueError):
        sdva.token_logprobs(torch.zeros(9, device="cuda"), lens, torch.empty(1, device="cuda"))


def test_one_row_of_any_stride():
    """One token has no row stride that means anything: slices whose stride is
    odd, shorter than the row or 0 are as good as a tensor of their own."""
    import speculative_decode_verify_append_gb300 as sdva
    q, k, v = _qkv(_gen(2), 1, 4, 2)

    def odd(x, stride):
        return x.as_strided(x.shape, (stride, D, 1))

    cu = _cu([1])
    want, got = torch.empty_like(q), torch.empty_like(q)
    sdva.prompt_attn(q, k, v, cu, np.float32(0.1), want)
    sdva.prompt_attn(odd(q, 0), odd(k, 13), odd(v, 1001), cu, 0.1, got)
    table, lens = i32_dev(np.array([[0]])), i32_dev(np.array([0]))
    a, b = sdva.KVCache(sdva.KV_INT8_G64, 1, 2), sdva.KVCache(sdva.KV_INT8_G64, 1, 2)
    sdva.kv_append_packed(a, k, v, cu, table, lens)
    sdva.kv_append_packed(b, odd(k, 13), odd(v, 0), cu, table, lens)
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)
    x = torch.randn((1, 40), device="cuda")
    lp = [torch.empty(1, device="cuda") for _ in range(2)]
    sdva.token_logprobs(x, lens, lp[0])
    sdva.token_logprobs(x.as_strided((1, 40), (0, 1)), lens, lp[1])
    torch.cuda.synchronize()
    assert torch.equal(*lp)


def test_calls_at_once_on_several_streams():
    """Kernels of several calls, each on its own stream, share the GPU: what
    they write is what they write one after the other."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(12)
    lens = [900, 64, 2000, 1]
    q, k, v = _qkv(g, sum(lens), 24, 4)
    cu = _cu(lens)
    pages = [n // 64 + 1 for n in lens]
    table = torch.full((4, max(pages)), -1, dtype=torch.int32, device="cuda")
    for b in range(4):
        table[b, :pages[b]] = torch.arange(pages[b], dtype=torch.int32, device="cuda") + sum(pages[:b])
    start = torch.zeros(4, dtype=torch.int32, device="cuda")
    long, short = _logits(g, 200, 50000, torch.bfloat16), _logits(g, 300, 9000, torch.float32)
    tokens = torch.randint(9000, (300,), generator=g, device="cuda", dtype=torch.int32)
    status = _status()

    def calls(streams):
        results = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i % 4 == 0:
                    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
                    sdva.prompt_attn(q, k, v, cu, float(SM_SCALE), out, lse, status)
                    results += [out, lse]
                elif i % 4 == 1:
                    cache = sdva.KVCache(sdva.KV_FP8_E4M3, sum(pages), 4)
                    sdva.kv_append_packed(cache, k, v, cu, table, start, status)
                    results += [cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales]
                else:
                    x = long if i % 4 == 2 else short
                    n = x.shape[0]
                    lp, en = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
                    tt, tl = torch.zeros((n, 9), dtype=torch.int32, device="cuda"), torch.zeros((n, 9), device="cuda")
                    sdva.token_logprobs(x, tokens[:n], lp, en, tt, tl, status)
                    results += [lp, en, tt, tl]
        torch.cuda.synchronize()
        return results

    one = calls([torch.cuda.current_stream()] * 8)
    streams = [torch.cuda.Stream() for _ in range(8)]
    for _ in range(3):
        for a, b in zip(one, calls(streams)):
            assert torch.equal(a, b)
    assert int(status.item()) == 0


@pytest.mark.parametrize("what", ["prompt_attn", "rows", "few_rows"])
def test_wait_that_runs_out_is_reported_and_recovered(what):
    """With a limit of zero cycles a wait that is not over when its sleep ends
    (some 200 us) gives up; the sizes have one warp wait through more of
    another's work than that.  The call reports it and returns, and the next
    one is right."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(13)
    if what == "prompt_attn":
        q, k, v = _qkv(g, 80000, 2, 1)

        def run(st):
            return _run_attn(q, k, v, _cu([80000]), status=st)
    else:
        n, V = (160, 3000000) if what == "rows" else (3, 30000000)
        x = torch.randn((n, V), generator=g, device="cuda")
        tokens = torch.zeros(n, dtype=torch.int32, device="cuda")

        def run(st):
            return _score(x, tokens, 4, st)
    want = run(None)
    st = _status()
    prev = sdva.sdva_debug_set_wait_limit(0)
    try:
        run(st)
    finally:
        sdva.sdva_debug_set_wait_limit(prev)
    assert int(st.item()) == sdva.STATUS_TIMEOUT
    for _ in range(2):
        st = _status()
        got = run(st)
        assert int(st.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
