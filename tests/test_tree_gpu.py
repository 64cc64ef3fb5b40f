"""GPU parity of the draft-tree attention (bf16 and FP8 pools) with the fp64 oracle, and its plan."""
import os

import numpy as np
import pytest
import torch

import paged_kv_flashattention_split_b200 as pa
from tests.helpers import alloc_ws
from tests.tree_cases import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_flashattention_split_b200 import build
        build.build()
    pa.lib()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,hq,hkv", [(1, 8, 2), (2, 4, 4), (4, 16, 2), (16, 32, 8), (64, 6, 3), (256, 8, 1)])
def test_page_sizes_and_head_layouts(page, hq, hkv, fp8):
    c = Case([(17, 1), (300, 5), (0, 3), (129, 33), (511, 12)], hq, hkv, page, fp8, unused=0.1, seed=page)
    c.check(*c.run(), f"P={page} hq={hq} hkv={hkv}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("n", [1, 16, 31, 32, 33, 63, 65, 128, 129, 255, 256])
def test_node_counts(n, group, fp8):
    """Query tiles of every fill, one and several to a request."""
    c = Case([(200, n), (1, max(1, n // 2))], 2 * group, 2, 16, fp8, shape="tree", unused=0.05, seed=n)
    c.check(*c.run(), f"n={n} G={group}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix", [0, 1, 15, 112, 127, 128, 129, 240, 255, 256, 257, 384, 1000])
def test_prefixes_at_the_borders_of_key_tiles(prefix, fp8):
    c = Case([(prefix, 1), (prefix, 16), (prefix, 70)], 8, 2, 8, fp8, seed=prefix)
    c.check(*c.run(), f"prefix={prefix}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape,unused", [("chain", 0.0), ("chain", 0.1), ("tree", 0.5), ("forest", 0.2),
                                          ("tree", 1.0)])
def test_tree_shapes(shape, unused, fp8):
    c = Case([(90, 40), (0, 40), (400, 7)], 8, 4, 4, fp8, shape=shape, unused=unused, seed=11)
    c.check(*c.run(), f"{shape} {unused}")


@pytest.mark.parametrize("fp8", [False, True])
def test_requests_without_nodes(fp8):
    c = Case([(100, 0), (50, 4), (0, 0), (200, 9), (64, 0)], 8, 2, 16, fp8, seed=5)
    c.check(*c.run(), "empty requests")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv,hq,n", [(1, 8, 40), (8, 32, 16), (3, 3, 200), (8, 64, 32)])
def test_long_prefixes_are_split(hkv, hq, n, fp8):
    """One long request among short ones: its key tiles spread over many CTA slots."""
    c = Case([(9000, n), (130, 3)], hq, hkv, 16, fp8, seed=hkv)
    c.check(*c.run(), "split")


@pytest.mark.parametrize("num_sms", [1, 3, 40])
def test_fewer_sms_than_the_device(num_sms):
    c = Case([(1000, 20), (3, 2), (257, 64)], 16, 4, 16, seed=num_sms)
    c.check(*c.run(num_sms=num_sms), f"sms={num_sms}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("peak,scale", [(8.0, None), (1.0, 0.0), (1.0, -0.1), (4.0, 1.0)])
def test_peaked_scores_and_scales(peak, scale, fp8):
    c = Case([(700, 20), (10, 4)], 8, 2, 16, fp8, peak=peak, scale=scale, seed=3)
    c.check(*c.run(), f"peak={peak} scale={scale}")


def test_large_and_small_queries_over_an_fp8_cache():
    """Query values outside the f16 range, and rows of very different size."""
    c = Case([(300, 24)], 8, 2, 16, True, seed=8, scale=2.0 ** -20)
    c.q[::2] *= 2.0 ** 17
    c.q[1::4] *= 2.0 ** -30
    c.check(*c.run(), "large q")
    c = Case([(300, 24)], 8, 2, 16, True, seed=9)
    c.q[3] = 0
    c.q[5] *= 2.0 ** -100
    c.check(*c.run(), "small q")


def test_lse_is_optional_and_the_output_repeats():
    c = Case([(4000, 16), (30, 3)], 32, 8, 16, seed=6)
    a, _ = c.run()
    params, (out, _) = c.params(), c.outputs()
    ws = alloc_ws(params)
    for _ in range(3):
        pa.attn_plan_tree(params, c.seq_lens, c.cu, c.parent, ws)
        c.attend(params, ws, out, None)
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), out.view(torch.int16))


def test_bounds_larger_than_the_batch():
    """A plan sized for longer sequences and more nodes gives the same result."""
    c = Case([(200, 9), (0, 5)], 8, 2, 16, extra_pitch=500, seed=12)
    c.check(*c.run(max_kv_len=4096, max_q_tokens=2000), "bounds")


def test_plan_covers_every_unit_once():
    c = Case([(9000, 130), (0, 1), (5, 0), (260, 70)], 16, 2, 16, shape="chain", seed=1)
    params = c.params()
    ws = alloc_ws(params)
    pa.attn_plan_tree(params, c.seq_lens, c.cu, c.parent, ws)
    assert pa.pa_read_device_error(ws) == pa.PA_OK
    raw = ws.cpu().numpy()
    hdr = raw[:64].view(np.int32)
    n_items, per, slots, n_cut = hdr[7], hdr[10], hdr[14], hdr[15]
    B, tile_nodes = c.B, 256 // 8
    off = 64 + 4 * (5 * B + 1)
    off = (off + 15) // 16 * 16
    items = raw[off:off + 16 * n_items].view(np.int32).reshape(-1, 4)
    off = (off + 16 * int(hdr[8]) + 255) // 256 * 256
    first = raw[off:off + 4 * (slots + 1)].view(np.int32)
    want = [(r, t) for r in range(B) for t in range(-(-c.n[r] // tile_nodes))]
    assert n_cut == sum(((items[:, 0] == r) & (items[:, 1] == t)).sum() > 1 for r, t in want)
    for r, t in want:
        pieces = items[(items[:, 0] == r) & (items[:, 1] == t)]
        assert pieces[0, 2] == 0 and pieces[-1, 3] == -(-c.lens[r] // 128)
        assert np.array_equal(pieces[1:, 2], pieces[:-1, 3])
    assert first[0] == 0 and first[-1] == n_items
    for s in range(slots):
        mine = items[first[s]:first[s + 1]]
        assert (mine[:, 3] - mine[:, 2]).sum() <= per


def test_bad_inputs_are_skipped_and_flagged():
    def run(c, params=None):
        params = params or c.params()
        ws = alloc_ws(params)
        out, lse = c.outputs()
        pa.attn_plan_tree(params, c.seq_lens, c.cu, c.parent, ws)
        c.attend(params, ws, out, lse)
        torch.cuda.synchronize()
        return pa.pa_read_device_error(ws), out, lse

    sizes = [(100, 8), (60, 8), (30, 4)]
    good = Case(sizes, seed=2)
    st, ref, ref_lse = run(good)
    assert st == pa.PA_OK
    # a parent that is not an earlier node: the node is unused
    for bad in (5, 7, -3, 1 << 30):
        c = Case(sizes, seed=2, shape="chain")
        c.parent[8 + 5] = bad
        st, out, lse = run(c)
        assert st == pa.PA_ERR_DEVICE_INDEX
        c.parent[8 + 5] = -2
        assert torch.all(out[8 + 5].float() == 0) and torch.all(torch.isneginf(lse[8 + 5]))
        c.parents[1][5] = -2
        c.check(out, lse, f"parent {bad}")
    # a request longer than max_kv_len, of negative length, or with more nodes than keys: left out
    for r, L in ((1, 200), (1, -5), (1, 7)):
        c = Case(sizes, seed=2)
        c.seq_lens[r] = L
        st, out, lse = run(c)
        assert st == pa.PA_ERR_DEVICE_INDEX
        assert torch.all(torch.isnan(out[8:16])) and torch.all(torch.isnan(lse[8:16]))
        for lo, hi in ((0, 8), (16, 20)):
            assert torch.equal(out[lo:hi].view(torch.int16), ref[lo:hi].view(torch.int16))
    # rows outside max_q_tokens
    c = Case(sizes, seed=2)
    c.cu[3] = 21
    st, out, lse = run(c)
    assert st == pa.PA_ERR_DEVICE_INDEX and torch.all(torch.isnan(out[16:]))
    assert torch.equal(out[:16].view(torch.int16), ref[:16].view(torch.int16))
    # pages outside the pool read as zero rows
    c = Case(sizes, seed=2)
    c.table[2, 0] = 1 << 30
    st, out, lse = run(c)
    assert st == pa.PA_ERR_DEVICE_INDEX
    assert torch.equal(out[:16].view(torch.int16), ref[:16].view(torch.int16)) and torch.all(torch.isfinite(out[16:20]))
    # requests that share rows of Q beyond the plan's bound on its tiles
    c = Case([(10, 200)] * 6, 16, 2, 16, seed=2)
    c.cu[:] = torch.tensor([0, 200, 0, 200, 0, 200, 0], dtype=torch.int32)
    st, out, lse = run(c, c.params(max_q_tokens=200))
    assert st == pa.PA_ERR_DEVICE_INDEX


def test_attention_without_a_tree_plan_is_refused_on_the_device():
    c = Case([(100, 8)], seed=2)
    params, (out, lse) = c.params(), c.outputs()
    ws = alloc_ws(params)                                     # zeros: no plan
    c.attend(params, ws, out, lse)
    torch.cuda.synchronize()
    assert pa.pa_read_device_error(ws) == pa.PA_ERR_WORKSPACE
    assert torch.all(torch.isnan(out))


@pytest.mark.parametrize("fp8", [False, True])
def test_other_streams_and_two_calls_at_once(fp8):
    cs = [Case([(3000, 32), (70, 5)], 16, 4, 16, fp8, seed=s) for s in (1, 2)]
    want = [c.run() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    state = []
    for c in cs:
        params = c.params()
        state.append((params, alloc_ws(params), *c.outputs()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, (params, ws, out, lse) in zip(cs, streams, state):
            pa.attn_plan_tree(params, c.seq_lens, c.cu, c.parent, ws, stream=s)
            c.attend(params, ws, out, lse, stream=s)
    torch.cuda.synchronize()
    for (out, lse), (_, _, o, l) in zip(want, state):
        assert torch.equal(out.view(torch.int16), o.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), l.view(torch.int32))


def test_graph_replays_with_new_lengths_and_trees():
    """Captured at one size; replayed with other lengths, trees, tables and queries in the same buffers."""
    sizes = [[(500, 16), (40, 16)], [(17, 16), (511, 16)], [(0, 16), (128, 16)]]
    cases = [Case(s, 16, 4, 16, shape="tree", unused=0.2, seed=i, extra_pitch=40) for i, s in enumerate(sizes)]
    cap = 640
    slots = max(c.slots for c in cases)
    pitch = max(c.table.shape[1] for c in cases)
    buf = Case(sizes[0], 16, 4, 16, seed=0)
    buf.k = torch.zeros(slots, 4, 128, dtype=torch.bfloat16, device="cuda")
    buf.v = torch.zeros_like(buf.k)
    buf.table = torch.zeros(2, pitch, dtype=torch.int32, device="cuda")
    params = buf.params(max_kv_len=cap)
    ws = alloc_ws(params)
    out, lse = buf.outputs()

    def load(c):
        buf.k[:c.slots].copy_(c.k)
        buf.v[:c.slots].copy_(c.v)
        buf.table.zero_()
        buf.table[:, :c.table.shape[1]].copy_(c.table)
        buf.q.copy_(c.q)
        buf.seq_lens.copy_(c.seq_lens)
        buf.cu.copy_(c.cu)
        buf.parent.copy_(c.parent)

    def step():
        pa.attn_plan_tree(params, buf.seq_lens, buf.cu, buf.parent, ws)
        for _ in range(2):                                    # two layers of one plan
            buf.attend(params, ws, out, lse)

    load(cases[0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c in cases:
        load(c)
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert pa.pa_read_device_error(ws) == pa.PA_OK
        c.check(out, lse, "replay")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [12, 40])
@pytest.mark.parametrize("order", ["rising", "falling", "late", "within"])
def test_scores_that_rise_and_fall_along_the_keys(order, n, fp8):
    """Key rows along the query direction whose scores rise from tile to tile by more than the references may
    lag, fall, jump once near the end, or rise inside one key tile."""
    c = Case([(1500, n), (130, 3)], 16, 4, 16, fp8, seed=31, scale=0.5)
    one = torch.full((128,), 0.25, device="cuda")
    c.q[:] = (one + 0.01 * torch.randn(c.q.shape, device="cuda")).to(torch.bfloat16)
    import oracle.tree as ot
    for r in range(c.B):
        L = c.lens[r]
        slots = torch.from_numpy(ot.gather_slots(c.table.cpu().numpy(), c.prefix[r], c.page, r)).cuda()
        pos = torch.arange(c.prefix[r], device="cuda", dtype=torch.float32)
        size = {"rising": pos / 64, "falling": (L - pos) / 64, "late": 12.0 * (pos > c.prefix[r] - 70),
                "within": 3.0 * ((pos % 128) / 32).floor()}[order]
        k = size[:, None, None] * one * 2 + 0.05 * torch.randn(len(slots), c.hkv, 128, device="cuda")
        if fp8:
            c.k[slots] = (k / c.ks).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            c.k[slots] = k.to(torch.bfloat16)
    c.check(*c.run(), order)


def test_every_fp8_code():
    """Subnormal, normal and extreme E4M3 codes of both signs, in K and in V."""
    c = Case([(512, 9)], 8, 2, 16, True, seed=33, scale=0.002)
    codes = torch.tensor([x for x in range(256) if x & 0x7F != 0x7F], dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for pool in (c.k, c.v):
        live = pool != 0x7F
        pool[live] = codes[torch.randint(0, len(codes), (int(live.sum()),), generator=g, device="cuda")]
    c.check(*c.run(), "all codes")
    for lo, hi in ((1, 8), (8, 16)):                         # the subnormals alone, and the smallest normals
        live = c.v != 0x7F
        c.v[live] = torch.randint(lo, hi, (int(live.sum()),), generator=g, device="cuda").to(torch.uint8)
        c.check(*c.run(), f"codes {lo}..{hi}")


@pytest.mark.parametrize("fp8", [False, True])
def test_unused_nodes_may_hold_anything_and_disturb_nothing(fp8):
    """NaN, infinities and the largest values in the queries, keys and values of nodes that are not in use."""
    sizes, parents = [(200, 40), (3, 9)], [[-1] + [(i - 1) if i % 3 else -2 for i in range(1, 40)],
                                           [-1, 0, -2, 0, 3, -2, 4, 6, 5]]
    c = Case(sizes, 8, 2, 16, fp8, seed=35, parents=parents)
    out, lse = c.run()
    c.check(out, lse, "unused")
    import oracle.tree as ot
    dead = np.concatenate([~ot.visibility(p).any(1) for p in parents])
    for junk in (float("nan"), float("inf"), -float("inf"), 3e38):
        c.q[:c.T][torch.from_numpy(dead).cuda()] = junk
        again, lse2 = c.run()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


@pytest.mark.parametrize("fp8", [False, True])
def test_many_heads_and_many_requests(fp8):
    """More KV heads than SMs (one slot), and more requests than a small plan block takes."""
    c = Case([(70, 3), (200, 2)], 160, 160, 16, fp8, seed=36)
    c.check(*c.run(), "heads")
    c = Case([(5 + (37 * i) % 90, 1 + i % 4) for i in range(300)], 2, 1, 4, fp8, seed=37, unused=0.1)
    c.check(*c.run(), "requests")


def test_values_of_any_size():
    """V near the top of bf16's range: the weights' common factor must not overflow the sums."""
    c = Case([(900, 20)], 8, 2, 16, seed=38)
    c.v.copy_((c.v.float() * 2.0 ** 80).to(torch.bfloat16))
    c.check(*c.run(), "large V")
    c = Case([(900, 20)], 8, 2, 16, seed=39)
    c.v.copy_((c.v.float() * 2.0 ** -80).to(torch.bfloat16))
    c.check(*c.run(), "small V")


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_far_behind_four_gigabytes(fp8):
    """The same cache at the end of pools of more than 2^32 bytes: bit for bit the same results."""
    c = Case([(700, 20), (0, 40), (5000, 3)], 16, 8, 16, fp8=fp8, seed=41)
    want = c.run()
    slots = (2 ** 32 // (8 * 128 * c.k.element_size()) // 16 + 8) * 16 + c.slots
    pools = []
    for x in (c.k, c.v):
        pools.append(torch.empty((slots,) + tuple(x.shape[1:]), dtype=x.dtype, device=x.device))
        pools[-1][-c.slots:] = x
    assert c.slots % 16 == 0 and (slots - c.slots) * 8 * 128 * c.k.element_size() > 2 ** 32
    c.k, c.v = pools
    c.table += (slots - c.slots) // 16
    for a, b in zip(want, c.run()):
        assert torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("skip", [1, 3, 700])
def test_tree_rows_behind_other_rows(skip, fp8):
    """Offsets that start behind the rows of something else (prefill tokens of a mixed batch): no error is
    recorded, nothing of those rows is read or written, and the results are the same bit for bit."""
    sizes = [(300, 17), (0, 5), (40, 33)]
    plain = Case(sizes, 8, 2, 16, fp8, unused=0.1, seed=61)
    want, want_lse = plain.run()
    c = Case(sizes, 8, 2, 16, fp8, unused=0.1, seed=61)
    c.q = torch.cat([torch.full((skip, 8, 128), float("nan"), dtype=c.q.dtype, device=c.q.device), c.q])
    c.parent = torch.cat([torch.tensor([7, -9, 1 << 30], dtype=torch.int32, device=c.q.device).repeat(skip)[:skip], c.parent])
    c.cu += skip
    out, lse = c.run(max_q_tokens=c.T + skip)                 # run() checks that no error was recorded
    assert torch.all(torch.isnan(out[:skip])) and torch.all(torch.isnan(lse[:skip]))
    for a, b in ((out[skip:], want), (lse[skip:], want_lse)):
        assert torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))
    # a wrong parent is still found there
    params = c.params(max_q_tokens=c.T + skip)
    ws = alloc_ws(params)
    c.parent[skip + c.T - 1] = 33
    pa.attn_plan_tree(params, c.seq_lens, c.cu, c.parent, ws)
    assert pa.pa_read_device_error(ws) == pa.PA_ERR_DEVICE_INDEX


def test_queries_at_the_top_of_bf16_over_an_fp8_cache():
    """Rows whose largest value is 2^127 or more keep the promised 2^-17 of it.  Subnormal key codes and small scales
    bring the scores to a few units."""
    c = Case([(300, 24), (20, 9)], 8, 2, 16, True, seed=62, scale=2.0 ** -62)
    c.ks = 2.0 ** -60
    g = torch.Generator(device="cuda").manual_seed(2)
    live = c.k != 0x7F
    code = torch.randint(1, 8, (int(live.sum()),), generator=g, device="cuda")
    sign = 128 * torch.randint(0, 2, (int(live.sum()),), generator=g, device="cuda")
    c.k[live] = (code + sign).to(torch.uint8)

    def values(lo, hi):
        x = lo + (hi - lo) * torch.rand(c.q.shape, generator=g, device="cuda")
        return x * (1 - 2 * torch.randint(0, 2, c.q.shape, generator=g, device="cuda"))

    def load(x, exponent):
        c.q.copy_((x.to(torch.bfloat16).float() * 2.0 ** exponent).to(torch.bfloat16))
        assert torch.all(torch.isfinite(c.q.float()))

    load(values(1.75, 1.98), 127)                             # 8 significant bits in the upper quarter of the binade
    c.check(*c.run(), "top")
    x = values(1.0, 1.98)
    x[:, :, 1::2] *= 2.0 ** -9                                # one part of the row at the split's lower end
    load(x, 127)
    c.check(*c.run(), "top and 2^-9 of it")
    load(values(1.0, 1.98), 126)
    c.check(*c.run(), "2^126")


def test_host_tensors():
    """Pinned host memory is within the kernel's reach; other host memory is refused before a launch."""
    c = Case([(100, 8), (33, 5)], 8, 2, 16, seed=64)
    want, _ = c.run()
    for name in ("seq_lens", "cu", "parent"):
        setattr(c, name, getattr(c, name).cpu().pin_memory())
    out, lse = c.run()
    assert torch.equal(out.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
    for name in ("seq_lens", "cu", "parent", "q", "k", "table"):
        d = Case([(100, 8), (33, 5)], 8, 2, 16, seed=64)
        setattr(d, name, getattr(d, name).cpu())
        with pytest.raises(ValueError, match="current device"):
            d.run()


def read_tree_plan(ws, params):
    """The workspace's arrays, from the layout documented at attn_plan_tree."""
    raw, up = ws.cpu().numpy(), lambda x: -(-x // 256) * 256   # noqa: E731
    hdr = raw[:64].view(np.int32)
    B, at, out = params.batch, 64, {}

    def take(n, dtype=np.int32):
        nonlocal at
        a = raw[at:at + 4 * n].view(dtype)
        at += 4 * n
        return a

    for name, n in (("tiles", B), ("base", B + 1), ("lens", B), ("row0", B), ("prefix", B)):
        out[name] = take(n)
    at = -(-at // 16) * 16
    out["items"] = take(4 * int(hdr[8])).reshape(-1, 4)[:hdr[7]]
    at = up(at)
    out["slot_first"] = take(int(hdr[14]) + 1)
    at = up(at)
    T = params.max_q_tokens // (256 // (params.hq // params.hkv)) + B
    out["cut"] = take(2 * min(max(1, int(hdr[14]) - 1), T)).reshape(-1, 2)[:hdr[15]]
    at = up(at)
    out["bits"] = take(8 * params.max_q_tokens, np.uint32).reshape(-1, 8)
    out.update(per=int(hdr[10]), slots=int(hdr[14]), header=hdr)
    return out


@pytest.mark.parametrize("batch,seed", [(b, s) for s in range(4) for b in (1, 2, 7, 33)] +
                         [(256, 0), (257, 1), (1023, 2), (1025, 3), (3000, 4)])
def test_plan_bit_exact(batch, seed):
    """Every array of the plan against the oracle: both block sizes, several requests a thread, empty requests,
    requests out of range, offsets behind other rows, plans for fewer SMs."""
    import oracle.tree as ot
    rng = np.random.default_rng(1000 * batch + seed)
    hq, hkv = [(8, 8), (8, 4), (32, 8), (8, 1)][seed % 4]
    n = rng.integers(0, 257 if batch < 40 else 6, batch)
    n[rng.random(batch) < 0.2] = 0
    lens = n + rng.integers(0, 3000 if batch < 40 else 200, batch)
    cu = int(rng.integers(0, 40)) + np.concatenate([[0], np.cumsum(n)])
    parent = [7] * int(cu[0])
    for k in n:
        parent += [int(rng.integers(max(-2, i - 5) if rng.random() < 0.9 else -2, i)) for i in range(int(k))]
    bad = seed % 2 == 1
    if bad:
        lens[rng.random(batch) < 0.1] = 4000
    rows, sms = int(cu[-1]) + int(rng.integers(1, 50)), int(rng.integers(1, 149))
    params = pa.make_params(pa.PA_MODE_TREE, batch, hq, hkv, 128, 16, max_kv_len=3400, max_q_tokens=rows, num_sms=sms)
    ws = alloc_ws(params)
    ws.fill_(0)
    t = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")   # noqa: E731
    pa.attn_plan_tree(params, t(lens), t(cu), t(parent or [-1]), ws)
    got = read_tree_plan(ws, params)
    want = ot.plan_tree(lens, cu, parent, hq, hkv, 3400, rows, sms)
    expect = pa.PA_ERR_DEVICE_INDEX if bad and np.any(lens == 4000) else pa.PA_OK
    assert pa.pa_read_device_error(ws) == expect
    assert (got["per"], got["slots"]) == (want["per"], want["slots"])
    assert got["header"][1:7].tolist() == [pa.PA_MODE_TREE, batch, hq, hkv, 128, 16]
    assert np.array_equal(got["lens"], lens) and np.array_equal(got["row0"], cu[:-1])
    for name in ("tiles", "base", "prefix", "slot_first"):
        assert np.array_equal(got[name], want[name]), name
    for name, width in (("items", 4), ("cut", 2)):
        assert np.array_equal(got[name], np.array(want[name], np.int32).reshape(-1, width)), name
    assert np.array_equal(got["bits"], want["bits"])           # rows of nobody stay as they were


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [12, 40])
@pytest.mark.parametrize("shape", ["lag", "stairs"])
def test_large_values_behind_references_that_lag(shape, n, fp8):
    """V up to 2^90 under weights near the top of what a row's reference allows: the keys that set the reference (the
    first half of each stream's first tile) score just less below the others than what would raise it, over 4096 keys
    of one slot; or the scores climb such a step every 512 keys.  Sums reach 2^16 x 4096 x 2^90 < 2^128."""
    import oracle.tree as ot
    lag = 7.9 if fp8 else 15.9
    c = Case([(4096, n)], 4, 1, 16, fp8, seed=43)
    if fp8:
        c.vs = 2.0 ** 90 / 448
    c.q[:] = 0.25                                             # q . k = 32 t for a key row of t's
    c.scale = lag * np.log(2) / (32 * (c.ks or 1.0))
    slots = torch.from_numpy(ot.gather_slots(c.table.cpu().numpy(), 4096, c.page, 0)).cuda()
    pos = torch.arange(4096, device="cuda")
    level = 1.0 + (pos // 512 if shape == "stairs" else 0 * pos)
    level[(pos < 64) | ((pos >= 128) & (pos < 192))] = 0
    g = torch.Generator(device="cuda").manual_seed(3)
    k = level[:, None, None].expand(-1, 1, 128)
    v = 0.5 + 0.5 * torch.rand(4096 + n, 1, 128, generator=g, device="cuda")
    every = torch.from_numpy(ot.gather_slots(c.table.cpu().numpy(), 4096 + n, c.page, 0)).cuda()
    if fp8:
        c.k[slots] = k.to(torch.float8_e4m3fn).view(torch.uint8)
        c.v[every] = (448 * v).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        c.k[slots] = k.to(torch.bfloat16)
        c.v[every] = (2.0 ** 90 * v).to(torch.bfloat16)
    out, lse = c.run(num_sms=1)
    assert torch.all(torch.isfinite(out[:c.T].float()))
    c.check(out, lse, shape)


def test_far_keys_under_a_peak_without_value_over_an_fp8_cache():
    """A key that takes nearly all the weight and has V = 0: what is left of O are the far keys' shares, each taken to
    within 2^-11 of itself or 2^-31 (the step of f16 at its lower end, 2^-25, over a row's sum of at least 2^6)."""
    import oracle.tree as ot
    for gap in (10.0, 16.0, 22.0, 40.0):
        c = Case([(700, 9), (300, 40)], 8, 2, 16, True, seed=65, scale=gap / 32.0)
        c.q[:] = 0.25                                         # q . k = 32 t for a key row of t's
        table = c.table.cpu().numpy()
        limit = []
        for r in range(c.B):
            slots = torch.from_numpy(ot.gather_slots(table, c.lens[r], c.page, r)).cuda()
            c.k[slots] = 0
            peak = slots[137]
            c.k[peak] = int(torch.tensor(1.0 / c.ks).to(torch.float8_e4m3fn).view(torch.uint8))
            c.v[peak] = 0
            v = c.vs * c.v[slots].view(torch.float8_e4m3fn).double().abs().sum(0)             # [Hkv, D]
            limit.append(v.repeat_interleave(4, 0).expand(c.n[r], -1, -1))
        out, lse = c.run()
        ref, ref_lse, mag = c.oracle()
        err = np.abs(out[:c.T].double().cpu().numpy() - ref[:c.T])
        tol = (2.0 ** -8 + 2.0 ** -11 + 2 * c.score_error() + 2.0 ** -16) * mag[:c.T]       # 2^-8: O in bf16
        tol += 2.0 ** -31 * torch.cat(limit).cpu().numpy()
        assert np.all(err <= tol), (gap, np.max(err / tol))
        assert np.all(np.abs(lse[:c.T].cpu().numpy() - ref_lse[:c.T]) <= c.score_error() + 2.0 ** -16 + 2.0 ** -20 * np.abs(ref_lse[:c.T]))
