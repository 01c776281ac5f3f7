"""GPU parity of pa_prefill and pa_cross_attention against the fp64 oracle:
head layouts, block sizes, lengths around every tile border, empty and
one-token sequences, padded batches, work partitions, scales, streams,
graphs, and the data-dependent errors (flagged, never a fault)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_228_gb300 import pa

from prompt_cases import Prompt, assert_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_cache_228_gb300 import build
    build.build()
    pa.pa_get_device_error()


def _ws(c, splits=0):
    n = pa.pa_attention_workspace_size(len(c.news), c.hq, c.hkv, c.d, splits)
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


def _run(c, causal, splits=0, scale=None, dev=None, single=False, stream=None, ws=None):
    x = dev or c.device()
    out = torch.full(x["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    fn = pa.pa_prefill if causal else pa.pa_cross_attention
    fn(x["q"], x["k"], x["v"], x["tab"], None if single else x["start"], x["lens"],
       c.scale if scale is None else scale, out, _ws(c, splits) if ws is None else ws,
       k_scale=x["ks"], v_scale=x["vs"], num_splits=splits, stream=stream)
    return out


def _check(c, causal, what="", splits=0, scale=None, **kw):
    out = _run(c, causal, splits, scale, **kw)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    assert_rows(out, *c.oracle(causal, scale), what=what)
    return out


FP8 = [pytest.param(False, id="bf16"), pytest.param(True, id="fp8")]


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_tiny(d, causal, fp8):
    c = Prompt([7, 16, 33, 50], [7, 16, 33, 50], 4, 2, d, 16, seed=1, fp8=fp8)
    _check(c, causal, f"tiny d={d}")


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 1, 128, 16), (4, 4, 128, 8), (6, 2, 128, 32),
                                         (4, 1, 64, 64), (7, 1, 64, 16), (16, 1, 128, 128),
                                         (64, 1, 64, 256), (2, 1, 128, 256), (5, 1, 64, 8)])
def test_head_layouts_and_block_sizes(hq, hkv, d, bs, fp8):
    # prompts, chunks behind a cache, one token, an empty sequence
    news, ctx = [130, 3, 0, 1, 61], [0, 517, 40, 255, 128]
    c = Prompt(news, [a + b for a, b in zip(news, ctx)], hq, hkv, d, bs, seed=2, fp8=fp8,
               pad_rows=3)
    _check(c, True, "causal")
    _check(c, False, "cross")


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 385])
def test_lengths_around_chunks(n):
    c = Prompt([n, 1, max(1, n - 1)], [n, n, n + 1], 4, 2, 128, 16, seed=n)
    _check(c, True, f"causal {n}")
    _check(c, False, f"cross {n}")


@pytest.mark.parametrize("nq", [31, 32, 33, 63, 64, 65, 127, 129])
def test_query_counts_around_tiles(nq):
    # G = 4: 128 rows are 32 tokens, an item 64
    c = Prompt([nq, nq], [nq, nq + 200], 4, 1, 64, 16, seed=nq)
    _check(c, True, f"causal {nq}")
    _check(c, False, f"cross {nq}")


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40, 152, 500])
def test_work_partitions(splits, fp8):
    # few items over long caches: pieces of one item in many CTAs
    c = Prompt([5, 90, 1], [2000, 1111, 700], 8, 2, 128, 16, seed=3, fp8=fp8)
    _check(c, True, f"causal splits {splits}", splits=splits)
    _check(c, False, f"cross splits {splits}", splits=splits)


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("splits", [1, 3, 0])
def test_long_runs_through_the_rings(splits, d, fp8):
    # every ring goes round many times in one CTA: items of one tile (both
    # tiles take chunks in turn), of two, and of one chunk, behind each other
    news = [1, 3, 70, 200, 1, 64, 2]
    lens = [3000, 100, 2500, 200, 1500, 1700, 129]
    c = Prompt(news, lens, 4, 1, d, 16, seed=20, fp8=fp8)
    _check(c, True, "causal", splits=splits)
    _check(c, False, "cross", splits=splits)


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("d", [64, 128])
def test_many_one_token_sequences_with_offsets(d, fp8):
    # a batch of more than 32 sequences, each an item of one tile over several
    # chunks
    rng = np.random.default_rng(21)
    lens = rng.integers(1, 2000, 64).tolist()
    c = Prompt([1] * 64, lens, 4, 2, d, 32, seed=21, fp8=fp8)
    for _ in range(3):
        _check(c, False, "one token each")


def test_partition_does_not_depend_on_blocks_and_repeats_bit_for_bit():
    c = Prompt([40, 300], [900, 300], 8, 2, 128, 16, seed=4)
    a, b = _run(c, True), _run(c, True)
    perm = torch.randperm(c.nb)
    x = c.device()
    x["k"], x["v"] = torch.empty_like(x["k"]), torch.empty_like(x["v"])
    x["k"][perm.cuda()], x["v"][perm.cuda()] = c.k.cuda(), c.v.cuda()
    t = torch.from_numpy(c.tab).long()
    x["tab"] = torch.where(t >= 0, perm[t.clamp(min=0)], -1).to(torch.int32).cuda()
    d = _run(c, True, dev=x)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(a.view(torch.int16), d.view(torch.int16))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-42, 4.0])
def test_scales(scale, fp8):
    c = Prompt([70, 2], [70, 333], 4, 2, 64, 16, seed=5, fp8=fp8)
    _check(c, True, f"scale {scale}", scale=scale)


def test_large_scores_stay_finite_and_the_maximum_moves():
    # keys grow along the sequence, so the running maximum moves by more than
    # the rescale threshold again and again
    c = Prompt([64, 10], [700, 900], 4, 2, 128, 16, seed=6)
    for b, n in enumerate(c.lens):
        for t in range(n):
            blk, off = c.tab[b][t // 16], t % 16
            c.k[blk, :, off] = (c.k[blk, :, off].float() * (0.2 + t / 60)).to(torch.bfloat16)
    for causal in (True, False):
        out = _run(c, causal)
        torch.cuda.synchronize()
        ref, spread = c.oracle(causal)
        # scores of magnitude s lose D 2^-24 of sum|q k| each: here up to
        # scale sum|q k| ~ 150, so a weight is off by up to 2 * 150 * 128 * 2^-24
        # = 2.3e-3, less than 2^-8: allow that much of the spread on top
        assert_rows(out, ref, spread * 1.8, "growing keys")
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("d", [64, 128])
def test_the_first_scores_are_far_below_the_maximum(d, fp8):
    # the running maximum starts from a chunk's first 32 scores: here those
    # are 2^40 and more below the rest in weight, in every chunk and piece
    c = Prompt([40, 3], [700, 900], 4, 2, d, 16, seed=23)
    for b, n in enumerate(c.lens):
        t = np.arange(n)
        low = torch.from_numpy(t % 128 < 32)
        k = torch.ones(n, c.hkv, d)
        k[low] = -1
        k += torch.randn(n, c.hkv, d, generator=torch.Generator().manual_seed(b)) * 0.05
        c.k[torch.from_numpy(c.tab[b][t // 16]).long(), :, torch.from_numpy(t % 16)] = k.to(torch.bfloat16)
    c.q = (torch.ones_like(c.q.float()) + c.q.float() * 0.05).to(torch.bfloat16)
    scale = 40.0 / d
    if fp8:
        kn, vn = c.k.nan_to_num().float().numpy(), c.v.nan_to_num().float().numpy()
        ids, full = list(range(c.nb)), [16] * c.nb
        from oracle import quantize as OQ
        kq, ks = OQ.quantize_blocks(kn, ids, full)
        vq, vs = OQ.quantize_blocks(vn, ids, full)
        c.k, c.v, c.ks, c.vs = (torch.from_numpy(x) for x in (kq, vq, ks, vs))
    for causal in (True, False):
        for splits in (0, 1, 5):
            out = _run(c, causal, splits, scale=scale)
            torch.cuda.synchronize()
            ref, spread = c.oracle(causal, scale)
            # scores of magnitude 40 lose at most D 2^-24 sum|q k| scale = 128 *
            # 2^-24 * 44 = 3.4e-4: less than the 2^-10 allowed
            assert_rows(out, ref, spread, f"low first scores, splits {splits}")
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_keys_with_scores_of_minus_infinity_have_no_weight(d):
    # the first 32 scores of every row are -inf, the others about -120, whose
    # exponentials against any maximum but their own underflow
    c = Prompt([40, 3], [700, 200], 4, 2, d, 16, seed=29)
    c.q = c.q * 0.05
    c.q[..., 0] = 1
    c.k = c.k * 0.5
    for b, n in enumerate(c.lens):
        t = np.arange(n)
        at = torch.from_numpy(c.tab[b][t // 16]).long(), torch.from_numpy(t % 16)
        first = torch.full((n, c.hkv), -120.0 * d ** 0.5)
        first[:32] = float("-inf")
        c.k[at[0], :, at[1], 0] = first.to(torch.bfloat16)
    for causal in (True, False):
        for splits in (0, 1, 5):
            out = _run(c, causal, splits)
            torch.cuda.synchronize()
            ref, spread = c.oracle(causal)
            # scores are off by at most D 2^-24 sum|q k| scale < 128 * 2^-24 *
            # 121 = 9.3e-4: less than the 2^-10 allowed
            assert_rows(out, ref, spread, f"scores of -inf, splits {splits}")
    assert pa.pa_get_device_error() == 0


def test_fp8_chunks_are_read_before_the_copies_refill_their_stage():
    # K = 0: every visible token weighs the same; V of chunk j is 1 in column j
    # and 0 elsewhere: column j of a row counts its visible tokens of chunk j.
    # Calls back to back, each with an output of its own.
    d, bs, hkv, hq = 128, 16, 8, 64
    news, lens = [1021, 1021], [9237, 9982]
    need = [-(-n // bs) for n in lens]
    nb = sum(need)
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(31)).int()
    tab = torch.full((2, max(need)), -1, dtype=torch.int32)
    tab[0, :need[0]], tab[1, :need[1]] = ids[:need[0]], ids[need[0]:]
    k = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8)
    want = torch.zeros(sum(news), d, dtype=torch.float64)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        v[tab[b][t // bs].long(), :, t % bs, t // 128] = 0x38  # 1.0
        lim = torch.arange(n - news[b], n) + 1
        seen = (lim[:, None] - 128 * torch.arange(d)[None, :]).clamp(0, 128)
        want[sum(news[:b]):sum(news[:b + 1])] = seen / lim[:, None]
    one = torch.ones(nb, hkv, device="cuda")
    q = torch.randn(sum(news), hq, d, device="cuda").to(torch.bfloat16)
    start = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device="cuda")
    kv, tab, v = torch.tensor(lens, dtype=torch.int32, device="cuda"), tab.cuda(), v.cuda()
    ws = torch.empty(pa.pa_attention_workspace_size(2, hq, hkv, d), dtype=torch.uint8,
                     device="cuda")
    # weights and their sum are exact or nearly so (2^-10); one rounding to
    # bf16, 2^-8.  One token of another chunk is 1 / 128 of the value: more.
    want = want.cuda()[:, None, :]
    outs = [torch.full_like(q, float("nan")) for _ in range(20)]
    torch.cuda.synchronize()
    for out in outs:
        pa.pa_prefill(q, k, v, tab, start, kv, d ** -0.5, out, ws, k_scale=one, v_scale=one)
    for i, out in enumerate(outs):
        err = (out.double() - want).abs() - (2.0 ** -8 + 2.0 ** -10) * want
        assert bool((err <= 0).all()), f"call {i}: {int((err > 0).sum())} values off"
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq", [16, 12])
def test_calls_back_to_back_give_the_same_bits(hq, causal, d, fp8):
    # two batches in turn over one workspace, nothing between the launches; 12
    # heads over 4: groups of 3 leave rows of a tile without a token
    cases = (Prompt([130, 1, 300, 7], [900, 400, 300, 4100], hq, 4, d, 16, seed=37, fp8=fp8),
             Prompt([5] * 9, [700 + 90 * i for i in range(9)], hq, 4, d, 32, seed=38, fp8=fp8,
                    std=2.0))
    devs = [c.device() for c in cases]
    ws = torch.full((max(_ws(c).numel() for c in cases),), 255, dtype=torch.uint8, device="cuda")
    fn = pa.pa_prefill if causal else pa.pa_cross_attention
    outs = [torch.full(devs[i % 2]["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            for i in range(24)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        c, x = cases[i % 2], devs[i % 2]
        fn(x["q"], x["k"], x["v"], x["tab"], x["start"], x["lens"], c.scale, out, ws,
           k_scale=x["ks"], v_scale=x["vs"])
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for i, out in enumerate(outs):
        if i < 2:
            assert_rows(out, *cases[i].oracle(causal), what=f"batch {i}")
        assert torch.equal(out, outs[i % 2]), f"call {i}"


def test_empty_encoder_gives_zeros_and_padded_rows_stay():
    c = Prompt([3, 5, 0], [0, 17, 9], 8, 2, 128, 16, seed=7, pad_rows=9)
    out = _check(c, False, "empty encoder")
    assert (out[:3] == 0).all()


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1)])
def test_one_token_a_sequence(hq, hkv, fp8):
    # without offsets (the decode step) and with them: the same attention
    c = Prompt([1] * 9, [1, 5, 0, 128, 129, 700, 64, 17, 1500], hq, hkv, 128, 16, seed=8,
               fp8=fp8)
    for causal in (False, True):
        ref, spread = c.oracle(False)
        if causal:  # a causal query has its own token in the cache
            x = c.device()
            x["lens"] = x["lens"].clamp(min=1)
        out = _run(c, False, single=True)
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        # FP8 decode at head_dim 128 also splits its weights in E4M3 pairs
        # (2^-8 of each plus 2^-18 of the largest): one more 2^-8
        assert_rows(out, ref, spread * (2 if fp8 else 1), "no offsets")
        out = _run(c, False)
        torch.cuda.synchronize()
        assert_rows(out, ref, spread, "offsets")
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", FP8)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1500], [3, 2100], [0], [1, 1024, 700], [2000, 0, 129, 1],
                                  [1100, 5, 600, 64, 1]])
def test_one_token_of_few_sequences_over_a_long_table(lens, d, fp8):
    # up to four sequences (two for FP8) over tables of 1024 tokens and more
    # take another split than batches do
    c = Prompt([1] * len(lens), lens, 8, 2, d, 16, seed=22, fp8=fp8)
    c.tab = np.pad(c.tab, ((0, 0), (0, 70)), constant_values=-1)
    out = _run(c, False, single=True)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    ref, spread = c.oracle(False)
    # as above: FP8 decode at head_dim 128 has one more rounding per weight
    assert_rows(out, ref, spread * (2 if fp8 else 1), "no offsets")


def test_single_token_over_one_state_is_its_value():
    c = Prompt([1, 1], [1, 1], 8, 2, 128, 16, seed=9)
    out = _run(c, True)
    torch.cuda.synchronize()
    for b in range(2):
        assert torch.equal(out[b].cpu(), c.v[c.tab[b][0], :, 0].repeat_interleave(4, 0))


def test_shared_blocks_between_sequences():
    # two decoder branches read one encoder's blocks
    c = Prompt([20, 30], [100, 100], 8, 2, 64, 16, seed=10)
    c.tab[1] = c.tab[0]
    _check(c, False, "shared encoder")


def test_many_small_sequences():
    rng = np.random.default_rng(11)
    news = rng.integers(0, 4, 900).tolist()
    c = Prompt(news, [n + int(x) for n, x in zip(news, rng.integers(0, 40, 900))], 4, 2, 64, 8,
               seed=11)
    _check(c, True, "900 sequences")


def test_errors_are_flagged_and_never_fault():
    c = Prompt([8, 8], [40, 40], 8, 2, 128, 16, seed=12)
    x = c.device()
    x["tab"][0, 1] = c.nb + 5
    x["tab"][1, 0] = -7
    _run(c, True, dev=x)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.DEVERR_BAD_BLOCK_ID
    # more queries than tokens: zeros for that sequence, the other as ever
    x = c.device()
    x["lens"][0] = 7
    out = _run(c, True, dev=x)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == pa.DEVERR_BAD_SEQ_LEN
    assert (out[:8] == 0).all()
    ref, spread = c.oracle(True)
    ref[:8] = spread[:8] = 0
    assert_rows(out, ref, spread, "the other sequence")
    # a length past the table is clamped to it (the entry there is -1: zeros)
    x = c.device()
    x["lens"][1] = 1 << 30
    _run(c, False, dev=x)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() & pa.DEVERR_BAD_SEQ_LEN
    # offsets out of order or range: nothing is written
    for start in ([0, 9, 8], [-1, 8, 16], [0, 8, 17], [5, 3, 16]):
        x = c.device()
        x["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        out = _run(c, True, dev=x)
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == pa.DEVERR_BAD_QUERY, start
        assert torch.isnan(out.float()).all()
    _check(c, True, "afterwards")


def test_streams_graphs_and_separate_workspaces():
    a = Prompt([33, 5], [300, 1200], 8, 2, 128, 16, seed=13)
    b = Prompt([64, 1], [64, 2000], 8, 2, 128, 16, seed=14)
    xa, xb = a.device(), b.device()
    wa, wb = _ws(a), _ws(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            oa = _run(a, True, dev=xa, ws=wa)
        with torch.cuda.stream(s2):
            ob = _run(b, False, dev=xb, ws=wb)
        outs.append((oa, ob))
    torch.cuda.synchronize()
    for oa, ob in outs:
        assert_rows(oa, *a.oracle(True), "stream 1")
        assert_rows(ob, *b.oracle(False), "stream 2")
    g = torch.cuda.CUDAGraph()
    out = torch.full(xa["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    with torch.cuda.graph(g):
        pa.pa_prefill(xa["q"], xa["k"], xa["v"], xa["tab"], xa["start"], xa["lens"], a.scale, out,
                      wa)
    # new lengths between replays: the plan is made on the device
    for shrink in (0, 17):
        xa["lens"].copy_(torch.tensor([300 - shrink, 1200 - shrink], dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        a.lens = [300 - shrink, 1200 - shrink]
        assert_rows(out, *a.oracle(True), f"replay {shrink}")
    assert pa.pa_get_device_error() == 0


def test_pool_past_32_bit_offsets():
    # a pool of more than 2^31 elements and 2^32 bytes; the blocks used lie
    # at its end
    hkv, bs, d = 8, 16, 128
    nb = (1 << 31) // (hkv * bs * d) + 4096
    c = Prompt([40, 3], [40, 700], 16, hkv, d, bs, seed=15)
    x = c.device()
    for n in ("k", "v"):
        pool = torch.empty((nb, hkv, bs, d), dtype=torch.bfloat16, device="cuda")
        pool[nb - c.nb:] = x[n]
        x[n] = pool
    x["tab"] = torch.where(x["tab"] >= 0, x["tab"] + (nb - c.nb), -1)
    _check(c, True, "large pool", dev=x)


def test_workspace_too_small_is_refused():
    c = Prompt([8], [40], 8, 2, 128, 16, seed=16)
    with pytest.raises(pa.PAError) as e:
        _run(c, True, ws=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pa.PA_ERR_WORKSPACE
    x = c.device()
    with pytest.raises(ValueError):
        pa.pa_prefill(x["q"], x["k"], x["v"], x["tab"], x["start"], x["lens"].cpu(), c.scale,
                      torch.empty_like(x["q"]), _ws(c))
