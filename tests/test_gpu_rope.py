"""kv_append_rope and kv_append_packed_rope on the GPU: the turned queries and
keys against 64 bits and bit for bit against their definition, and the cache
byte for byte against kv_append_quant of the turned keys."""
import numpy as np
import pytest
import torch

from gpu_util import ALL_KV, KV_NAMES

pytestmark = pytest.mark.gpu

D = 128
NAN = float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _qkv(g, lead, hq, hkv):
    x = torch.randn((*lead, hq + 2 * hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    return x.split([hq, hkv, hkv], -2)


def _turn(x, rope, pos, interleaved):
    """The definition: fp32 products and sums, each rounded, then bf16; x [..., H, 128], pos [...]."""
    rot = rope.shape[1]
    c, s = (y.unsqueeze(-2) for y in rope[pos.long()].chunk(2, -1))
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    p, r = a * c - b * s, b * c + a * s
    t = torch.stack([p, r], -1).flatten(-2) if interleaved else torch.cat([p, r], -1)
    return torch.cat([t, y[..., rot:]], -1).to(torch.bfloat16)


def _turn64(x, rope, pos, interleaved):
    rot = rope.shape[1]
    ang = rope[pos.long()].double().unsqueeze(-2)
    y = x.double()
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(ang[..., :rot // 2], ang[..., rot // 2:])
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _check64(got, x, rope, pos, interleaved):
    """Half a step of bf16 (2^-8), and three roundings of fp32 (2^-24 each) of the products' magnitudes."""
    want = _turn64(x, rope, pos, interleaved)
    mag = _turn64(x.abs(), rope.abs(), pos, interleaved).abs() + x.double().abs() + want.abs()
    # |x1 c| + |x2 s| <= |x1| + |x2| of the pair: the sum of the pair's magnitudes
    rot = rope.shape[1]
    y = x.double().abs()
    pair = y.clone()
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    pair[..., first] = pair[..., second] = y[..., first] + y[..., second]
    err = (got.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 1.01 * 3 * 2.0 ** -24 * (pair + mag)).all()


def _cache(dtype, pages, hkv, g):
    """A cache that holds other lanes' leftovers."""
    import speculative_decode_verify_append_gb300 as sdva
    c = sdva.KVCache(dtype, pages, hkv)
    for n in ("k_codes", "v_codes"):
        t = getattr(c, n)
        if dtype in (sdva.KV_FP8_E4M3, sdva.KV_FP8_ROW):
            t.copy_((torch.randn(t.shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
                    .view(torch.uint8))
        else:
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda").to(torch.uint8))
    for n in ("k_scales", "v_scales"):
        getattr(c, n).uniform_(0.004, 0.008, generator=g)
    return c


def _copy(c):
    import speculative_decode_verify_append_gb300 as sdva
    return sdva.KVCache(c.dtype, c.num_pages, c.num_kv_heads,
                        tensors=[getattr(c, n).clone() for n in ("k_codes", "v_codes", "k_scales", "v_scales")])


def _same(a, b):
    for n in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def _table(g, lens, counts, extra=2):
    """Pages of the lanes' new tokens in any order; the pages in front of them are not mapped."""
    rows = max((L + n + 63) // 64 for L, n in zip(lens, counts)) + 1
    need = [(L // 64, (L + n - 1) // 64) if n else (0, -1) for L, n in zip(lens, counts)]
    pages = sum(b - a + 1 for a, b in need) + extra
    ids = torch.randperm(pages, generator=g, device="cuda").tolist()
    t = np.full((len(lens), rows), -1, np.int32)
    for row, (a, b) in zip(t, need):
        for p in range(a, b + 1):
            row[p] = ids.pop()
    return torch.from_numpy(t).cuda(), pages


def _rope(positions, rot, base=10000.0):
    from speculative_decode_verify_append_gb300.step import rope_table
    return rope_table(positions, rot, base)


def test_rope_table():
    t = _rope(240001, 64)
    assert t.shape == (240001, 64) and t.dtype == torch.float32
    for p in (0, 1, 77, 240000):
        a = p * 10000.0 ** (-np.arange(0, 64, 2) / 64)
        want = np.concatenate([np.cos(a), np.sin(a)])
        # half a step of fp32 at most 1 in magnitude, and the angle's own rounding in 64 bits (2^-52 of it)
        assert np.abs(t[p].cpu().numpy() - want).max() <= 2.0 ** -25 + 4 * 2.0 ** -52 * p + 1e-12


def _window(dtype, rot, interleaved, lanes, W, hq, hkv, seed, ragged=False, tree=False, lens=None):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(seed)
    cpu = np.random.default_rng(seed)
    lens = [int(x) for x in cpu.integers(0, 700, lanes)] if lens is None else lens
    counts = [int(x) for x in cpu.integers(0, W + 1, lanes)] if ragged else [W] * lanes
    q, k, v = _qkv(g, (lanes, W), hq, hkv)
    for b, n in enumerate(counts):  # rows behind a lane's count are not read
        for x in (q, k, v):
            x[b, n:] = NAN
    table, pages = _table(g, lens, counts)
    pos = torch.tensor(lens, device="cuda")[:, None] + torch.arange(W, device="cuda")
    if tree:
        pos = torch.tensor(lens, device="cuda")[:, None] + torch.from_numpy(
            np.minimum(cpu.integers(0, W, (lanes, W)), np.arange(W))).cuda()
    rope = _rope(max(lens) + W, rot)
    seq, n_lane = _i32(lens), _i32(counts)
    cache = _cache(dtype, pages, hkv, g)
    other, before = _copy(cache), _copy(cache)
    q_out, k_out = (torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k))
    st = _status()
    sdva.kv_append_rope(cache, q, k, v, rope, table, seq, q_out, k_out, n_lane if ragged else None,
                        pos.to(torch.int32) if tree else None, interleaved, st)
    kt = _turn(k, rope, pos, interleaved)
    sdva.kv_append_quant_ragged(other, kt, v.contiguous(), n_lane, table, seq, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _same(cache, other)
    for b, n in enumerate(counts):
        assert torch.equal(q_out[b, :n], _turn(q[b, :n], rope, pos[b, :n], interleaved))
        assert torch.equal(k_out[b, :n], kt[b, :n])
        assert (q_out[b, n:] == 7.0).all() and (k_out[b, n:] == 7.0).all()
        _check64(q_out[b, :n], q[b, :n], rope, pos[b, :n], interleaved)
    # without the turned keys, the same cache
    sdva.kv_append_rope(before, q, k, v, rope, table, seq, q_out, None, n_lane if ragged else None,
                        pos.to(torch.int32) if tree else None, interleaved, st)
    _same(before, other)


@pytest.mark.parametrize("dtype", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("rot", [16, 32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_window(dtype, rot, interleaved):
    _window(dtype, rot, interleaved, 5, 16, 6, 2, rot + dtype)


@pytest.mark.parametrize("dtype", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("hq,hkv", [(24, 4), (1, 1), (7, 7), (5, 1), (8, 8), (64, 2)])
@pytest.mark.parametrize("W", [1, 2, 7])
def test_window_heads_ragged_and_trees(dtype, hq, hkv, W):
    _window(dtype, 128 if W == 2 else 64, W == 7, 9, W, hq, hkv, hq + W, ragged=True, tree=True)


@pytest.mark.parametrize("dtype", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("lens", [[0], [63], [64], [48], [49], [1, 60, 127, 64]])
def test_window_page_edges(dtype, lens):
    _window(dtype, 128, False, len(lens), 16, 4, 2, 3, lens=lens)


def test_a_long_window_and_far_positions():
    _window(0, 128, False, 2, 300, 4, 2, 8, lens=[239000, 17])
    _window(2, 64, True, 3, 130, 3, 1, 9, ragged=True, tree=True, lens=[120000, 1, 0])


def test_window_of_one_row_of_any_stride():
    """Lanes of one row are one stride apart whatever the axis of one says."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(4)
    x = torch.randn((6, 1, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    rope, table, seq = _rope(100, 128), _i32([[i] for i in range(6)]), _i32([0] * 6)
    caches = [sdva.KVCache(0, 6, 2) for _ in range(2)]
    outs = [torch.empty((6, 1, 4, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, k, v = x.split([4, 2, 2], 2)
    sdva.kv_append_rope(caches[0], q, k, v, rope, table, seq, outs[0])
    sdva.kv_append_rope(caches[1], q.contiguous(), k.contiguous(), v.contiguous(), rope, table, seq, outs[1])
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    _same(*caches)


def _packed(dtype, rot, interleaved, lens, cached, hq, hkv, seed, start=0, tail=0):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(seed)
    T = start + sum(lens) + tail
    q, k, v = _qkv(g, (T,), hq, hkv)
    cu = _i32(np.concatenate([[start], start + np.cumsum(lens)]))
    end = start + sum(lens)
    for x in (q, k, v):
        x[:start] = NAN
        x[end:] = NAN
    table, pages = _table(g, cached, lens)
    rope = _rope(max(c + n for c, n in zip(cached, lens)), rot)
    cache = _cache(dtype, pages, hkv, g)
    other = _copy(cache)
    q_out, k_out = (torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k))
    seq, st = _i32(cached), _status()
    sdva.kv_append_packed_rope(cache, q, k, v, cu, rope, table, seq, q_out, k_out, interleaved, st)
    pos = torch.zeros(T, dtype=torch.long, device="cuda")
    a = start
    for n, c in zip(lens, cached):
        pos[a:a + n] = c + torch.arange(n, device="cuda")
        a += n
    kt = _turn(k, rope, pos, interleaved)
    sdva.kv_append_packed(other, kt, v, cu, table, seq, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _same(cache, other)
    assert torch.equal(q_out[start:end], _turn(q, rope, pos, interleaved)[start:end])
    assert torch.equal(k_out[start:end], kt[start:end])
    for x in (q_out, k_out):
        assert (x[:start] == 7.0).all() and (x[end:] == 7.0).all()
    _check64(q_out[start:end], q[start:end], rope, pos[start:end], interleaved)


@pytest.mark.parametrize("dtype", ALL_KV, ids=KV_NAMES.get)
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (16, True)])
@pytest.mark.parametrize("lens,cached", [([1], [0]), ([64], [0]), ([65, 0, 63, 1, 700], [0, 5, 127, 64, 40]),
                                         ([1] * 30, list(range(50, 80)))])
def test_packed(dtype, rot, interleaved, lens, cached):
    _packed(dtype, rot, interleaved, lens, cached, 6, 2, len(lens) + rot, start=3, tail=5)


@pytest.mark.parametrize("dtype", ALL_KV, ids=KV_NAMES.get)
def test_packed_long(dtype):
    _packed(dtype, 128, False, [5000, 3, 2100], [300, 0, 9], 24, 4, 1)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("what", ["page", "length", "negative", "position_table", "positions_low", "positions_high", "count"])
def test_bad_lanes_are_skipped_whole(packed, what):
    import speculative_decode_verify_append_gb300 as sdva
    if packed and (what.startswith("positions") or what == "count"):
        pytest.skip("windows only")
    g = _gen(6)
    W, B = 8, 3
    q, k, v = _qkv(g, (B, W), 4, 2)
    lens, pages = [60, 10, 0], 8
    t = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    pos = np.array(lens)[:, None] + np.arange(W)
    positions, n_lane, far = None, None, 200
    want = sdva.STATUS_OVERFLOW
    if what == "page":
        t[0, 1], want = pages, sdva.STATUS_BAD_PAGE
    elif what == "length":
        lens[0] = 121
    elif what == "negative":
        lens[0] = -1
    elif what == "position_table":
        far = 67
    elif what == "positions_low":
        positions = pos.copy()
        positions[0, 7] = -1
    elif what == "positions_high":
        positions = pos.copy()
        positions[0, 3] = far
    else:
        n_lane, want = _i32([W + 1, W, 2]), sdva.STATUS_BAD_COUNT
    rope, table, seq, st = _rope(far, 64), torch.from_numpy(t).cuda(), _i32(lens), _status()
    cache = _cache(0, pages, 2, g)
    other = _copy(cache)
    q_out, k_out = (torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k))
    if packed:
        cu = _i32([0, 8, 16, 24])
        sdva.kv_append_packed_rope(cache, q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), cu, rope, table, seq,
                                   q_out.flatten(0, 1), k_out.flatten(0, 1), status=st)
    else:
        sdva.kv_append_rope(cache, q, k, v, rope, table, seq, q_out, k_out, n_lane,
                            None if positions is None else _i32(positions), status=st)
    good = [8, 2] if n_lane is not None else [8, 8]
    for b, n in zip((1, 2), good):
        kt = _turn(k[b:b + 1, :n], rope, torch.from_numpy(pos[b:b + 1, :n]).cuda(), False)
        sdva.kv_append_quant(other, kt, v[b:b + 1, :n].contiguous(), table[b:b + 1], seq[b:b + 1])
        assert torch.equal(k_out[b, :n], kt[0])
    torch.cuda.synchronize()
    assert int(st.item()) == want
    _same(cache, other)
    assert (q_out[0] == 7.0).all() and (k_out[0] == 7.0).all() and not (q_out[1] == 7.0).any()


def test_packed_offsets_out_of_order_write_nothing():
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(7)
    q, k, v = _qkv(g, (20,), 4, 2)
    rope, table, seq = _rope(100, 128), _i32([[0], [1]]), _i32([0, 0])
    for cu in ([0, 12, 9], [-1, 5, 20], [0, 5, 21]):
        cache, st = _cache(3, 4, 2, g), _status()
        other = _copy(cache)
        q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        sdva.kv_append_packed_rope(cache, q, k, v, _i32(cu), rope, table, seq, q_out, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == sdva.STATUS_BAD_COUNT
        _same(cache, other)
        assert (q_out == 7.0).all()


def test_the_binding_refuses():
    import speculative_decode_verify_append_gb300 as sdva
    q, k, v = _qkv(_gen(1), (2, 4), 4, 2)
    out, rope, table, seq = torch.empty_like(q, memory_format=torch.contiguous_format), _rope(64, 128), _i32([[0], [1]]), _i32([0, 0])
    cache = sdva.KVCache(0, 2, 2)
    good = dict(cache=cache, q=q, k_new=k, v_new=v, rope=rope, page_table=table, seq_lens=seq, q_out=out)
    sdva.kv_append_rope(**good)
    for change in (dict(q=q.float()), dict(k_new=k[:, :3]), dict(v_new=v.transpose(0, 1)), dict(q=q.cpu()),
                   dict(rope=rope.double()), dict(rope=rope[:, :100]), dict(rope=rope[::2]), dict(seq_lens=seq[:1]),
                   dict(q_out=out[:, :, :2]), dict(q_out=q), dict(positions=seq), dict(n_lane=_i32([1])),
                   dict(page_table=table[0]), dict(k_out=out), dict(k_new=q)):
        with pytest.raises((ValueError, sdva.SdvaError)):
            sdva.kv_append_rope(**{**good, **change})
    with pytest.raises(sdva.SdvaError) as e:
        sdva.kv_append_rope(**{**good, "rope": _rope(64, 48)})
    assert e.value.code == sdva.ERR_UNSUPPORTED


@pytest.mark.parametrize("packed", [False, True])
def test_a_captured_graph_replays(packed):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(2)
    q, k, v = (x.contiguous() for x in _qkv(g, (3, 8), 4, 2))
    rope, table, seq = _rope(300, 128), _i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]]), _i32([5, 60, 100])
    cu = _i32([0, 8, 16, 24])
    q_out = torch.zeros_like(q)
    cache = sdva.KVCache(1, 9, 2)

    def call(c, out):
        if packed:
            sdva.kv_append_packed_rope(c, q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), cu, rope, table, seq,
                                       out.flatten(0, 1))
        else:
            sdva.kv_append_rope(c, q, k, v, rope, table, seq, out)

    call(cache, q_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cache, q_out)
    for seed in (1, 2):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=_gen(seed), device="cuda"))
        seq += 3
        graph.replay()
        other, out = _copy(cache), torch.zeros_like(q)
        call(other, out)
        torch.cuda.synchronize()
        _same(cache, other)
        assert torch.equal(out, q_out)
