"""The attention over a paged cache where it can go wrong: rows that see nothing, layouts, lengths and
pages that break the rules, many sequences, far offsets, streams, workspaces and captured replays."""
import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from oracle import attn as ref
from tests.parity import host32, say
from tests.test_gpu_paged_attn import BF16, DEV, F32, U16, call, check, make, tokens

pytestmark = pytest.mark.gpu


def test_tokens_that_see_nothing():
    c = ([5, 3, 70], [0, 10, 0], 4, 2, 64, 64, 16, 0, True)
    x = make(c)
    x["kv_lens"] = torch.tensor([2, 0, 40], dtype=torch.int32, device=DEV)      # fewer positions than new tokens
    o, lse = call(c, x)
    check(c, x, o, lse)
    assert not tokens(o, True)[:3].any() and np.isneginf(tokens(lse, True)[:3]).all()
    assert not tokens(o, True)[5:8].any() and not tokens(o, True)[8:38].any()
    c = ([1, 1], [0, 0], 4, 2, 128, 128, 16, 0, False)
    x = make(c)
    x["kv_lens"].zero_()
    o, lse = call(c, x)
    assert not o.any() and torch.isneginf(lse).all()


def test_layouts_of_rows_and_caches():
    c = ([40, 40], [100, 20], 6, 2, 128, 128, 64, 0, False)
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)
    # q sliced from a projection, o written head-major, lse given
    wide = torch.full((2, 40, 10, 128), float("nan"), dtype=BF16, device=DEV)
    wide[:, :, 1:7] = x["q"].transpose(1, 2)
    out, out_l = torch.empty(2, 6, 40, 128, dtype=BF16, device=DEV), torch.empty(2, 6, 40, device=DEV)
    y = dict(x, q=wide[:, :, 1:7].transpose(1, 2))
    a, al = call(c, y, o=out, lse=out_l)
    assert a is out and al is out_l and torch.equal(a, o) and torch.equal(al, lse)
    assert torch.equal(kda.paged_attn(y["q"], x["kc"], x["vc"], x["table"], x["kv_lens"]), o)       # without lse
    # keys and values in one buffer; rows and pages padded; rows before heads
    both = torch.stack((x["kc"], x["vc"]), 1)
    a, _ = call(c, dict(x, kc=both[:, 0], vc=both[:, 1]))
    assert torch.equal(a, o)
    pad = torch.full((x["kc"].shape[0], 2, 67, 152), float("nan"), dtype=BF16, device=DEV)
    pad[:, :, :64, :128] = x["kc"]
    a, _ = call(c, dict(x, kc=pad[:, :, :64, :128]))
    assert torch.equal(a, o)
    rows = x["vc"].transpose(1, 2).contiguous().transpose(1, 2)
    a, _ = call(c, dict(x, vc=rows))
    assert torch.equal(a, o)
    # a window of a wider table
    big = torch.cat((x["table"], torch.full_like(x["table"], 12345)), 1)
    a, _ = call(c, dict(x, table=big[:, :x["table"].shape[1]]))
    assert torch.equal(a, o)


@pytest.mark.parametrize("d", [(64, 128), (128, 64)])
def test_narrow_tiles_of_padded_rows(d):
    c = ([1, 1, 1], [300, 5, 64], 4, 1, d[0], d[1], 16, 0, False)
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)
    pk = torch.full((x["kc"].shape[0], 1, 16, d[0] + 24), float("nan"), dtype=BF16, device=DEV)
    pv = torch.full((x["kc"].shape[0], 1, 16, d[1] + 8), float("nan"), dtype=BF16, device=DEV)
    pk[..., :d[0]], pv[..., :d[1]] = x["kc"], x["vc"]
    a, al = call(c, dict(x, kc=pk[..., :d[0]], vc=pv[..., :d[1]]))
    assert torch.equal(a, o) and torch.equal(al, lse)


def test_rows_in_no_sequence_stay():
    c = ([5, 40], [30, 100], 4, 2, 64, 64, 16, 0, True)
    x = make(c)
    o, lse = call(c, x)
    wide = torch.cat((x["q"][:, :3], x["q"], x["q"][:, :2]), 1)
    out = torch.full((4, 50, 64), 7.0, dtype=BF16, device=DEV)
    out_l = torch.full((4, 50), 7.0, device=DEV)
    call(c, dict(x, q=wide, cu=x["cu"] + 3), o=out, lse=out_l)
    assert torch.equal(out[:, 3:48], o) and torch.equal(out_l[:, 3:48], lse)
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 48:] == 7).all()) and bool((out_l[:, 48:] == 7).all())


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 3.0])
def test_scales(scale):
    for c in (([1, 1], [200, 40], 4, 2, 64, 64, 16, 0, False), ([50], [20], 4, 2, 64, 64, 16, 0, False)):
        x = make(c)
        o, lse = call(c, x, scale=scale)
        check(c, x, o, lse, scale=scale)


def test_peaked_scores():
    for c in (([3, 3], [300, 40], 4, 2, 128, 128, 16, 0, False), ([100], [200], 4, 2, 128, 128, 16, 0, False)):
        x = make(c, qs=40.0)
        o, lse = call(c, x)
        check(c, x, o, lse)


def test_scores_that_rise_all_along():
    """Every block raises the running reference: keys along the query, longer from row to row."""
    c = ([70], [500], 2, 1, 64, 64, 64, 0, False)
    x = make(c)
    u = torch.randn(64, device=DEV)
    u /= u.norm()
    flat = torch.arange(1, 640 + 1, device=DEV, dtype=F32)[:, None] * u * 0.2
    for i, p in enumerate(x["table"][0, :9].tolist()):
        x["kc"][p, 0, :] = flat[i * 64:(i + 1) * 64].to(BF16)
    x["q"] = (u * 8.0).expand(1, 2, 70, 64).to(BF16).contiguous()
    o, lse = call(c, x)
    check(c, x, o, lse)


@pytest.mark.parametrize("n", [65, 300, 4100])
def test_many_sequences(n):
    rng = np.random.default_rng(n)
    c = ([1] * n, rng.integers(0, 40, n).tolist(), 1, 1, 64, 64, 16, 0, False)
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)
    new = rng.integers(0, 4, n).tolist()
    new[3], new[n - 2] = 40, 70
    c = (new, rng.integers(0, 40, n).tolist(), 1, 1, 64, 64, 16, 0, True)
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)


def test_page_sizes_of_the_prefix_cache():
    for page in (48, 512, 6144):
        c = ([30, 1], [700, 6200], 4, 2, 64, 64, page, 0, True)
        x = make(c)
        o, lse = call(c, x)
        check(c, x, o, lse)


def test_broken_tables_and_lengths_touch_nothing_else():
    c = ([1, 40, 1, 33], [200, 100, 64, 0], 4, 2, 64, 64, 16, 0, True)
    x = make(c)
    o, lse = call(c, x)
    keep = torch.ones(75, dtype=torch.bool, device=DEV)
    keep[1:41] = False                                            # the second sequence
    for what in ("page", "far page", "long", "negative"):
        y = dict(x, table=x["table"].clone(), kv_lens=x["kv_lens"].clone())
        if what == "page":
            y["table"][1] = -1
        elif what == "far page":
            y["table"][1] = torch.tensor([2147483647, 1 << 20, y["kc"].shape[0]], device=DEV, dtype=torch.int32).repeat(5)[:y["table"].shape[1]]
        elif what == "long":
            y["kv_lens"][1] = 2147483647
        else:
            y["kv_lens"][1] = -2147483648
        a, al = call(c, y)
        assert torch.equal(a[:, keep], o[:, keep]) and torch.equal(al[:, keep], lse[:, keep]), what
    for cu in ([0, 41, 41, 42, 75], [0, 1, 0, 42, 75], [0, 1, 41, 42, 1000], [-5, 1, 41, 42, 75]):
        y = dict(x, cu=torch.tensor(cu, dtype=torch.int32, device=DEV))
        a, _ = call(c, y, o=torch.zeros_like(o))
        s = 3 if cu[4] == 75 else 2                              # a sequence whose own bounds are right
        lo, hi = (42, 75) if s == 3 else (41, 42)
        assert torch.equal(a[:, lo:hi], o[:, lo:hi]), cu


def test_offsets_past_32_bits():
    """Pages behind the first 2^32 elements of a cache."""
    Hk, page, d = 8, 64, 128
    pages = (1 << 32) // (Hk * page * d) + 40
    kc, vc = (torch.empty(pages, Hk, page, d, dtype=BF16, device=DEV) for _ in range(2))
    for c in (([1, 1], [500, 70], 16, Hk, d, d, page, 0, False), ([60], [300], 8, Hk, d, d, page, 0, False)):
        x = make(c)
        o, lse = call(c, x)
        n = x["kc"].shape[0]
        kc[pages - n:], vc[pages - n:] = x["kc"], x["vc"]
        t = torch.where(x["table"] >= 0, x["table"] + (pages - n), x["table"])
        a, al = call(c, dict(x, kc=kc, vc=vc, table=t))
        assert torch.equal(a, o) and torch.equal(al, lse)
    # the append reaches them too
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    k = torch.randn(2, Hk, 1, d, generator=g, device=DEV).to(BF16)
    table = torch.tensor([[pages - 1], [pages - 2]], dtype=torch.int32, device=DEV)
    kda.kv_append(None, k, k, kc, vc, table, torch.tensor([64, 3], dtype=torch.int32, device=DEV), norm=False)
    assert torch.equal(kc[pages - 1, :, 63], k[0, :, 0]) and torch.equal(vc[pages - 2, :, 2], k[1, :, 0])


def test_long_context():
    """One token and a chunk over 100001 positions, every key head, against fp64 on the GPU."""
    for n in (1, 300):
        c = ([n], [100001 - n], 8, 2, 128, 128, 64, 0, False)
        x = make(c)
        o, lse = call(c, x)
        pg = x["table"][0, :-(-100001 // 64)].long()
        for h in range(8):
            K, V = (x[t][pg, h // 4].reshape(-1, 128)[:100001].double() for t in ("kc", "vc"))
            s = x["q"][0, h].double() @ K.t() * float(np.float32(128 ** -0.5))
            j, pos = torch.arange(100001, device=DEV), torch.arange(100001 - n, 100001, device=DEV)[:, None]
            s = torch.where(j <= pos, s, torch.full_like(s, float("-inf")))
            L = torch.logsumexp(s, -1)
            P = torch.exp(s - L[:, None])
            want, mag = P @ V, P @ V.abs()
            # probabilities in bf16, the rest in fp32: 2^-8 of the magnitude and 2^-8 of the result
            assert bool(((o[0, h].double() - want).abs() <= 1.05 * U16 * (mag + want.abs())).all())
            # each of a lane's sums has 100001 / 64 terms of one rounding, the scores 130 of 2^-24 of |q||k|, 25
            assert bool(((lse[0, h].double() - L).abs() <= 2.0 ** -24 * (100001 / 64 + 130 * 60 + 4 * L.abs())).all())


def test_repeats_and_a_dirty_workspace():
    for c in (([1, 1, 1], [3000, 70, 900], 8, 2, 128, 128, 64, 0, False), ([300, 2], [2000, 100], 8, 1, 64, 64, 16, 0, True)):
        x = make(c)
        o, lse = call(c, x)
        for fill in (255, 0, 127):
            ws = torch.full((256 << 20,), fill, dtype=torch.uint8, device=DEV)
            a, al = call(c, x, workspace=ws)
            assert torch.equal(a, o) and torch.equal(al, lse)
        with pytest.raises(ValueError):
            call(c, x, workspace=torch.empty(64, dtype=torch.uint8))


def test_two_streams_at_once():
    cs = [([1, 1], [4000, 300], 8, 2, 128, 128, 64, 0, False), ([200], [1000], 8, 2, 128, 128, 64, 0, False)]
    xs = [make(c) for c in cs]
    want = [call(c, x) for c, x in zip(cs, xs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append([call(c, x, stream=s) for c, x, s in zip(cs, xs, streams)])
    torch.cuda.synchronize()
    for g in got:
        for (a, al), (b, bl) in zip(g, want):
            assert torch.equal(a, b) and torch.equal(al, bl)


def test_captured_replays_follow_the_lengths():
    """Lengths, table and rows are read on the device: a captured append and attention serve every step."""
    c = ([1, 1, 1], [1, 40, 700], 8, 2, 64, 64, 16, 0, False)
    x = make(c, fill=0.0)
    start = x["kv_lens"] - 1
    width = x["table"].shape[1]
    spare = iter(range(x["kc"].shape[0], x["kc"].shape[0] + 40))
    kc, vc = (torch.cat((x[t], torch.zeros(40, *x[t].shape[1:], dtype=BF16, device=DEV))) for t in ("kc", "vc"))
    table = torch.full((3, width + 3), -1, dtype=torch.int32, device=DEV)
    table[:, :width] = x["table"]
    f = torch.tensor(10000.0 ** (-np.arange(0, 64, 2) / 64), dtype=F32, device=DEV)
    row = torch.zeros(3, 1, 12, 64, dtype=BF16, device=DEV)
    lens = start.clone()
    q, k, v = row[:, :, :8].transpose(1, 2), row[:, :, 8:10].transpose(1, 2), row[:, :, 10:].transpose(1, 2)

    def step(cache_k, cache_v):
        qr = kda.kv_append(q, k, v, cache_k, cache_v, table, lens, f)
        return kda.paged_attn(qr, cache_k, cache_v, table, lens)

    lens += 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kc.clone(), vc.clone())
    torch.cuda.synchronize()
    ke, ve = kc.clone(), vc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(kc, vc)
    lens.copy_(start)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for i in range(20):
        row.copy_(torch.randn(3, 1, 12, 64, generator=g, device=DEV).to(BF16))
        lens += 1
        for s, n in enumerate(lens.tolist()):
            if table[s, (n - 1) // 16] < 0:
                table[s, (n - 1) // 16] = next(spare)
        want = step(ke, ve)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kc, ke) and torch.equal(vc, ve), i


def test_two_graphs_of_one_pool():
    cs = [([1, 1], [3000, 300], 8, 2, 128, 128, 64, 0, False), ([64], [2000], 8, 2, 128, 128, 64, 0, False)]
    xs = [make(c) for c in cs]
    want = [call(c, x) for c, x in zip(cs, xs)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c, x in zip(cs, xs):
            call(c, x)
    torch.cuda.synchronize()
    pool, graphs, outs = torch.cuda.graph_pool_handle(), [], []
    for c, x in zip(cs, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(call(c, x))
        graphs.append(g)
    for _ in range(4):
        for g, o, w in zip(graphs, outs, want):
            for t in o:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_rope_captured_streams_and_far_rows():
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    q = torch.randn(1, 4, 300, 128, generator=g, device=DEV).to(BF16)
    k = torch.randn(1, 2, 300, 128, generator=g, device=DEV).to(BF16)
    w = 1.0 + 0.1 * torch.randn(128, generator=g, device=DEV)
    f = torch.tensor(10000.0 ** (-np.arange(0, 128, 2) / 128), dtype=F32, device=DEV)
    both = lambda **kw: (*kda.head_rope_fwd(q, k, f, q_weight=w, k_weight=w, **kw),
                         *kda.head_rope_bwd(q, k, f, k.repeat(1, 2, 1, 1), k, q_weight=w, k_weight=w, **kw))
    want = both()
    again = both()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = both(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    # rows behind 2^32 elements: the last block of a tensor expanded nowhere
    far = torch.empty((1 << 32) // (300 * 128) + 2, 300, 128, dtype=BF16, device=DEV)
    far[-1], far[0] = k[0, 0], k[0, 1]
    view = far.as_strided((1, 2, 300, 128), (0, (far.shape[0] - 1) * 300 * 128, 128, 1))
    with pytest.raises(kda.KDAError):
        kda.head_rope_fwd(None, view, f)                          # a head stride past 32 bits
    view = far.as_strided((2, 1, 300, 128), ((far.shape[0] - 1) * 300 * 128, 0, 128, 1))
    _, z = kda.head_rope_fwd(None, view, f, k_weight=w)
    assert torch.equal(z[1, 0], want[1][0, 0]) and torch.equal(z[0, 0], want[1][0, 1])


def test_streams_of_another_device_are_refused():
    class Other:
        device = torch.device("cuda:1")
    c = ([1], [10], 2, 1, 64, 64, 16, 0, False)
    x = make(c)
    with pytest.raises(ValueError, match="stream is on"):
        call(c, x, stream=Other())


@pytest.mark.parametrize("c", [
    ([1], [40], 4, 2, 128, 128, 16, 0, False),          # one chunk
    ([1], [6000], 2, 1, 64, 64, 16, 0, False),          # many chunks of a narrow tile, more than a wave joins
    ([1, 1, 1], [900, 64, 1], 4, 2, 128, 64, 16, 64, False),
    ([40, 1, 20], [3000, 500, 3], 8, 2, 64, 128, 64, 0, True),
    ([150], [20000], 2, 1, 128, 128, 512, 0, False),    # many chunks of a wide tile
])
def test_nan_queries(c):
    """A query that holds a NaN has NaN outputs, also where every score of a wave's keys is one; no other row is
    touched."""
    x = make(c)
    clean, clean_l = call(c, x)
    q = x["q"].clone()
    q[..., 1, -1, 5] = float("nan")             # head 1, the last token (of every sequence, or of the last one)
    if not c[8]:
        q[0, 0, 0, 0] = float("nan")
    o, lse = call(c, dict(x, q=q))
    hit = torch.isnan(q).any(-1)
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_l[~hit])
    check(c, x, clean, clean_l)


@pytest.mark.parametrize("c", [
    ([1], [50000], 16, 1, 64, 64, 16, 0, False),
    ([2, 1, 1], [30000, 100, 0], 4, 2, 64, 128, 64, 0, True),
    ([1, 1], [20000, 15], 8, 1, 128, 64, 16, 0, False),
    ([300, 30, 5], [9000, 10, 200], 2, 1, 128, 128, 64, 0, True),
    ([520, 3], [1500, 0], 3, 3, 64, 64, 32, 0, True),
])
def test_long_caches_cut_into_many_chunks(c):
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)
    a, al = call(c, x)
    assert torch.equal(a, o) and torch.equal(al, lse)


@pytest.mark.parametrize("c", [
    ([33, 128, 129, 64, 32, 1], [0, 70, 300, 2000, 9000, 128], 2, 2, 64, 64, 16, 0, True),
    ([16, 9, 5], [4000, 100, 0], 8, 1, 64, 64, 64, 0, True),
    ([12] * 3, [1500, 31, 700], 10, 1, 64, 64, 32, 40, False),
    ([43], [9000], 3, 1, 64, 64, 16, 0, False),
])
def test_heads_of_64_around_the_widths_of_tiles(c):
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)


@pytest.mark.parametrize("c", [
    ([1500], [0], 16, 8, 128, 128, 16, 0, False),       # more pages in one chunk than a wave holds addresses of
    ([700, 900], [650, 300], 16, 8, 64, 128, 32, 0, True),
    ([600, 600], [500, 700], 16, 8, 128, 64, 16, 0, False),
    ([1300], [200], 16, 8, 64, 64, 16, 700, False),
])
def test_small_pages_in_wide_tiles(c):
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)


@pytest.mark.parametrize("n", [65, 256, 257, 4097, 4500])
def test_numbers_of_sequences_around_the_scan(n):
    """Rounds of 64 sequences, four lengths a lane at a time: every row against the same call in pieces, and cut
    sequences among them."""
    new = [(s * 5) % 4 if s % 7 else 1 for s in range(n)]
    past = [(s * 13) % 40 for s in range(n)]
    past[n // 3], past[n - 1], new[n - 1] = 3000, 5000, 2
    c = (new, past, 2, 1, 64, 64, 16, 0, True)
    x = make(c)
    o, lse = call(c, x)
    check(c, x, o, lse)


def test_overlapping_sequences_stay_within_the_tensors():
    """cu_seqlens that go back and forth: the same rows in many sequences, more tiles and cuts than the rows allow.
    Numbers are undefined, accesses are not; what surrounds the outputs keeps its bits."""
    for T, N, kv, Hq, Hk, d in ((4, 40, 3000, 2, 2, 64), (300, 30, 4000, 2, 1, 128), (1, 600, 900, 1, 1, 64)):
        q = torch.randn(Hq, T, d, device=DEV).to(BF16)
        pages = 70
        kc, vc = (torch.randn(pages, Hk, 64, d, device=DEV).to(BF16) for _ in range(2))
        table = torch.randint(0, pages, (N, (kv + 63) // 64), dtype=torch.int32, device=DEV)
        cu = torch.tensor([0 if s % 2 == 0 else T for s in range(N + 1)], dtype=torch.int32, device=DEV)
        lens = torch.full((N,), kv, dtype=torch.int32, device=DEV)
        wide = torch.full((Hq, T + 2, d), 7.0, dtype=BF16, device=DEV)
        kda.paged_attn(q, kc, vc, table, lens, cu_seqlens=cu, o=wide[:, 1:T + 1])
        torch.cuda.synchronize()
        assert bool((wide[:, 0] == 7).all()) and bool((wide[:, T + 1] == 7).all())
