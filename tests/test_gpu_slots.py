"""GPU parity of pa_append_slots_device / pa_trim_slots_device, bit for bit,
against the oracle's list model of the block manager: random grow / shrink
runs in place, batches past one tile of 1024 sequences, every way a batch
stops, bad ids, in-place and separate outputs, graph replay; and the whole
prompt-side run: append, cache write, prefill, decode, trim, cross."""
import numpy as np
import pytest
import torch

from oracle import block_manager as BM
from oracle import prompt as OP
from paged_kv_cache_228_gb300 import pa

from prompt_cases import assert_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_cache_228_gb300 import build
    build.build()
    pa.pa_get_device_error()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Device:
    """The device's side of a batch: tables, free stack, lengths."""

    def __init__(self, model, B, width, bs):
        self.bs, self.B = bs, B
        self.free = torch.full((model.num_blocks,), -1, dtype=torch.int32, device="cuda")
        self.free[:len(model.free_stack)] = _i32(model.free_stack)
        self.num_free = _i32([len(model.free_stack)])
        self.tab = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.done = _i32([-1])

    def append(self, n_new, capacity):
        slots = torch.full((capacity,), -99, dtype=torch.int64, device="cuda")
        start = torch.full((self.B + 1,), -99, dtype=torch.int32, device="cuda")
        pa.pa_append_slots_device(self.lens, n_new, self.tab, self.free, self.num_free, self.bs,
                                  slots, start, self.lens, self.num_free, self.done)
        return slots, start

    def trim(self, new_lens):
        pa.pa_trim_slots_device(self.lens, new_lens, self.tab, self.free, self.num_free, self.bs,
                                self.lens, self.num_free)


def _same_state(dev, model, tables, lens):
    assert dev.lens.tolist() == lens
    n = int(dev.num_free)
    assert dev.free[:n].tolist() == model.free_stack
    got = dev.tab.tolist()
    for b, t in enumerate(tables):
        assert got[b][:len(t)] == t, b


@pytest.mark.parametrize("B,bs,nb,top,seed", [(5, 16, 200, 90, 0), (64, 8, 4000, 300, 1),
                                              (1, 32, 64, 700, 2), (1500, 16, 9000, 40, 3),
                                              (2100, 256, 9000, 400, 4)])
def test_random_runs_match_the_model_in_place(B, bs, nb, top, seed):
    rng = np.random.default_rng(seed)
    model = BM.BlockManagerModel(nb)
    tables, lens = [[] for _ in range(B)], [0] * B
    width = -(-4 * top // bs)
    dev = Device(model, B, width, bs)
    for step in range(6):
        kind = step % 3
        if kind < 2:
            n_new = rng.integers(0, top if kind == 0 else 2, B).tolist()
            slots, start = dev.append(_i32(n_new), sum(n_new) + 7)
            want = []
            for b in range(B):
                st, s, pairs = model.append_slots(tables[b], lens[b], n_new[b], bs, width)
                assert st == BM.OK and not pairs
                want += s
                lens[b] += n_new[b]
            assert slots.tolist() == want + [-1] * 7
            assert start.tolist() == np.concatenate([[0], np.cumsum(n_new)]).tolist()
            assert dev.done.tolist() == [B]
        else:
            to = [0 if rng.random() < 0.3 else max(0, n - int(rng.integers(0, 40))) for n in lens]
            dev.trim(_i32(to))
            for b in range(B):
                keep = -(-to[b] // bs)
                assert model.free(tables[b][keep:]) == BM.OK
                del tables[b][keep:]
            lens = to
        _same_state(dev, model, tables, lens)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("B", [4, 1300])
def test_out_of_blocks_stops_the_batch_there(B):
    bs, width = 8, 20
    model = BM.BlockManagerModel(2 * B)
    tables, lens = [[] for _ in range(B)], [0] * B
    dev = Device(model, B, width, bs)
    n_new = [5 + (7 * b) % 60 for b in range(B)]
    slots, start = dev.append(_i32(n_new), sum(n_new))
    want, done = [], None
    for b in range(B):
        st = BM.OUT_OF_BLOCKS
        if done is None:
            st, s, _ = model.append_slots(tables[b], 0, n_new[b], bs, width)
        if st == BM.OK:
            want += s
            lens[b] = n_new[b]
        else:
            done = b if done is None else done
            want += [-1] * n_new[b]
    assert done is not None
    assert slots.tolist() == want
    assert dev.done.tolist() == [done]
    _same_state(dev, model, tables, lens)
    assert pa.pa_get_device_error() == pa.DEVERR_OUT_OF_BLOCKS
    # what failed goes through once blocks are back
    dev.trim(torch.zeros_like(dev.lens))
    assert int(dev.num_free) == 2 * B
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("lens,n_new,cap,err", [
    ([0, -1, 0], [3, 1, 2], 6, "DEVERR_BAD_SEQ_LEN"), ([0, 0, 0], [3, -1, 2], 5, "DEVERR_BAD_SEQ_LEN"),
    ([0, 60, 0], [3, 5, 2], 10, "DEVERR_BAD_SEQ_LEN"), ([0, 0, 0], [3, 5, 2], 7, "DEVERR_BAD_QUERY"),
    ([0, 2147483647, 0], [3, 2147483647, 2], 10, "DEVERR_BAD_SEQ_LEN")])
def test_bad_lengths_stop_the_batch(lens, n_new, cap, err):
    model = BM.BlockManagerModel(50)
    dev = Device(model, 3, 8, 8)
    dev.lens = _i32(lens)
    slots, start = dev.append(_i32(n_new), cap)
    assert dev.lens.tolist() == [3] + lens[1:]
    assert dev.done.tolist() == [1] and int(dev.num_free) == 49
    assert slots.tolist()[3:] == [-1] * (cap - 3) and (slots[:3] >= 0).all()
    assert all(0 <= x <= cap for x in start.tolist())
    assert pa.pa_get_device_error() == getattr(pa, err)


def test_bad_ids_are_flagged():
    dev = Device(BM.BlockManagerModel(10), 2, 8, 8)
    dev.free[9] = 77          # the first id popped lies outside the pool
    slots, _ = dev.append(_i32([3, 4]), 7)
    assert slots.tolist()[:3] == [-1] * 3 and (slots[3:] >= 0).all()
    assert pa.pa_get_device_error() == pa.DEVERR_BAD_BLOCK_ID
    # its owner then cannot give it back: it keeps length and block, the
    # other sequence's block moves up in the stack
    keep = dev.tab[1, 0].item()
    dev.trim(_i32([0, 0]))
    assert dev.lens.tolist() == [3, 0] and int(dev.num_free) == 9
    assert dev.free[8].item() == keep
    assert pa.pa_get_device_error() == pa.DEVERR_BAD_BLOCK_ID
    # new lengths out of range
    dev.trim(_i32([4, 0]))
    assert dev.lens.tolist() == [3, 0]
    assert pa.pa_get_device_error() == pa.DEVERR_BAD_SEQ_LEN
    # more blocks than the pool has room for
    full = Device(BM.BlockManagerModel(4), 1, 4, 8)
    full.lens, full.tab[0, 0] = _i32([5]), 2
    full.trim(_i32([0]))
    assert full.lens.tolist() == [5] and int(full.num_free) == 4
    assert pa.pa_get_device_error() == pa.DEVERR_BAD_BLOCK_ID


def test_bad_ids_in_a_cluster_trim():
    # wide tables take the 8-CTA form; bad entries in several sequences
    B, bs, width = 300, 8, 500
    dev = Device(BM.BlockManagerModel(B * 12), B, width, bs)
    dev.append(_i32([90] * B), 90 * B)
    before = dev.tab[:, :12].clone()
    n0 = int(dev.num_free)
    bad = [3, 77, 299]
    for b in bad:
        dev.tab[b, 4] = -5
    dev.trim(_i32([0] * B))
    want = [x for b in range(B) if b not in bad for x in before[b].tolist()]
    assert int(dev.num_free) == n0 + len(want)
    assert dev.free[n0:n0 + len(want)].tolist() == want
    assert [b for b, n in enumerate(dev.lens.tolist()) if n] == bad
    assert pa.pa_get_device_error() == pa.DEVERR_BAD_BLOCK_ID


def test_separate_outputs_repeat():
    # with outputs of their own the inputs stay, so a call can be repeated
    dev = Device(BM.BlockManagerModel(100), 3, 8, 8)
    got = []
    for _ in range(2):
        slots = torch.empty(30, dtype=torch.int64, device="cuda")
        start, lens, nf = _i32([0] * 4), _i32([0] * 3), _i32([0])
        pa.pa_append_slots_device(dev.lens, _i32([9, 0, 21]), dev.tab, dev.free, dev.num_free, 8,
                                  slots, start, lens, nf, dev.done)
        got.append((slots.tolist(), start.tolist(), lens.tolist(), nf.tolist()))
    assert got[0] == got[1] and got[0][3] == [95]
    assert int(dev.num_free) == 100 and dev.lens.tolist() == [0, 0, 0]


@pytest.mark.parametrize("B,top", [(60, 300), (1100, 30)])
def test_long_maps_with_separate_outputs(B, top):
    # outputs apart from the inputs: the slot map is shared by a whole grid
    rng = np.random.default_rng(B)
    n_new = rng.integers(0, top, B).tolist()
    assert sum(n_new) > 4096
    model = BM.BlockManagerModel(sum(n_new))
    dev = Device(model, B, 64, 8)
    slots = torch.empty(sum(n_new), dtype=torch.int64, device="cuda")
    start, lens, nf = _i32([0] * (B + 1)), _i32([0] * B), _i32([0])
    pa.pa_append_slots_device(dev.lens, _i32(n_new), dev.tab, dev.free, dev.num_free, 8, slots,
                              start, lens, nf, dev.done)
    tables, want = [[] for _ in range(B)], []
    for b in range(B):
        _, s, _ = model.append_slots(tables[b], 0, n_new[b], 8, 64)
        want += s
    assert slots.tolist() == want and lens.tolist() == n_new and dev.done.tolist() == [B]
    assert int(nf) == len(model.free_stack)
    got = dev.tab.tolist()
    assert all(got[b][:len(t)] == t for b, t in enumerate(tables))
    assert pa.pa_get_device_error() == 0


def test_captured_steps_advance_in_place():
    B, bs, width = 40, 16, 30
    model = BM.BlockManagerModel(2000)
    tables, lens = [[] for _ in range(B)], [0] * B
    dev = Device(model, B, width, bs)
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    start = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_append_slots_device(dev.lens, one, dev.tab, dev.free, dev.num_free, bs, slots,
                                  start, dev.lens, dev.num_free, dev.done)
    for _ in range(37):
        g.replay()
        want = []
        for b in range(B):
            _, s, _ = model.append_slots(tables[b], lens[b], 1, bs, width)
            want += s
            lens[b] += 1
        assert slots.tolist() == want
    _same_state(dev, model, tables, lens)
    assert pa.pa_get_device_error() == 0


def test_a_served_batch_end_to_end():
    """Prompts are admitted, prefilled in two chunks, decode three steps,
    attend to an encoder, take back drafts and finish: every output against
    the oracle on a host copy of the caches."""
    rng = np.random.default_rng(5)
    B, hq, hkv, d, bs, nb, width = 5, 8, 2, 128, 16, 120, 24
    scale = d ** -0.5
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    dev = Device(BM.BlockManagerModel(nb), B, width, bs)
    k = torch.full((nb, hkv, bs, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    enc_lens = [0, 40, 130, 17, 64]
    enc = Device(BM.BlockManagerModel(40), B, 10, bs)
    ek, ev = (torch.full((40, hkv, bs, d), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    es, _ = enc.append(_i32(enc_lens), sum(enc_lens))
    pa.pa_cache_write(rnd(sum(enc_lens), hkv, d), rnd(sum(enc_lens), hkv, d), es, ek, ev)
    ws = torch.empty(max(pa.pa_attention_workspace_size(B, hq, hkv, d),
                         pa.pa_decode_workspace_size(B, hq, hkv, d)), dtype=torch.uint8,
                     device="cuda")
    host = lambda t: t.float().cpu().numpy()  # noqa: E731
    for n_new in (rng.integers(1, 150, B).tolist(), rng.integers(0, 90, B).tolist(), [1] * B,
                  [1] * B, [4] * B):
        T = sum(n_new)
        slots, start = dev.append(_i32(n_new), T + 2)
        kn, vn, q = rnd(T + 2, hkv, d), rnd(T + 2, hkv, d), rnd(T + 2, hq, d)
        pa.pa_cache_write(kn, vn, slots, k, v)
        out = torch.full_like(q, float("nan"))
        if n_new == [1] * B:
            pa.pa_decode(q[:B], k, v, dev.tab, dev.lens, scale, out[:B], ws)
        else:
            pa.pa_prefill(q, k, v, dev.tab, start, dev.lens, scale, out, ws)
        cross = torch.full_like(q, float("nan"))
        if n_new == [1] * B:
            pa.pa_cross_attention(q[:B], ek, ev, enc.tab, None, enc.lens, scale, cross[:B], ws)
        else:
            pa.pa_cross_attention(q, ek, ev, enc.tab, start, enc.lens, scale, cross, ws)
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        lens, tab, st = dev.lens.tolist(), dev.tab.cpu().numpy(), start.tolist()
        assert_rows(out, *OP.attend_rows(host(q), host(k), host(v), tab, st, lens, scale, True),
                    what=f"self {n_new}")
        assert_rows(cross, *OP.attend_rows(host(q), host(ek), host(ev), enc.tab.cpu().numpy(), st,
                                           enc_lens, scale, False), what=f"cross {n_new}")
    # two of the four drafted tokens are rejected, then everyone finishes
    dev.trim(dev.lens - 2)
    dev.trim(torch.zeros_like(dev.lens))
    assert int(dev.num_free) == nb and sorted(dev.free.tolist()) == list(range(nb))
    assert pa.pa_get_device_error() == 0
