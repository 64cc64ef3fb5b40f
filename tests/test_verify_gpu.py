"""GPU tests of the draft verification and of the compaction of accepted rows: exact against the oracle."""
import os

import numpy as np
import pytest
import torch

import paged_kv_flashattention_split_b200 as pa
from oracle import tree as ot
from tests.helpers import alloc_ws, bits16
from tests.tree_cases import Case, random_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_flashattention_split_b200 import build
        build.build()
    pa.lib()


class Drafts:
    """Requests of the given node counts; rows as numpy fp32, tokens drawn from the draft rows."""

    def __init__(self, counts, vocab, drafts=True, shape="tree", unused=0.0, seed=0, temp=3.0, near=1.0, parents=None):
        rng = np.random.default_rng(seed)
        self.vocab, self.B, self.T = vocab, len(counts), sum(counts)
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        rows = parents or [random_parents(rng, n, shape, unused) for n in counts]
        for row in rows if parents is None else []:
            if row:
                row[0] = -1
        self.parent = np.array([p for row in rows for p in row] or [-1], dtype=np.int32)
        T = max(self.T, 1)
        logits = rng.standard_normal((T, vocab)) * temp
        softmax = lambda x: (lambda e: e / e.sum(-1, keepdims=True))(np.exp(x - x.max(-1, keepdims=True)))   # noqa: E731
        self.target = softmax(logits).astype(np.float32)
        self.draft = softmax(logits + near * rng.standard_normal((T, vocab))).astype(np.float32)
        self.tokens = np.zeros(T, dtype=np.int32)
        for r in range(self.B):
            for i in range(counts[r]):
                row = self.cu[r] + max(int(rows[r][i]), 0)
                cdf = np.cumsum(self.draft[row].astype(np.float64))
                self.tokens[self.cu[r] + i] = min(vocab - 1, np.searchsorted(cdf, rng.random() * cdf[-1], "right"))
        if not drafts:
            self.draft = None
        self.u_accept = rng.random(T).astype(np.float32)
        self.u_final = rng.random(self.B).astype(np.float32)

    def run(self, pitch=None, ws=None, row_pad=0, stream=None):
        pitch = max(1, int(np.diff(self.cu).max(initial=1))) if pitch is None else pitch

        def dev(a):
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)

        def rows(a):
            if a is None or not row_pad:
                return dev(a)
            wide = torch.full((a.shape[0], a.shape[1] + row_pad), float("nan"), device=DEV)
            wide[:, :a.shape[1]] = dev(a)
            return wide[:, :a.shape[1]]

        n, nxt = (torch.full((self.B,), 77, dtype=torch.int32, device=DEV) for _ in range(2))
        path = torch.full((self.B, pitch), 77, dtype=torch.int32, device=DEV)
        pa.attn_tree_verify(dev(self.cu), dev(self.parent), dev(self.tokens), rows(self.target), rows(self.draft),
                            dev(self.u_accept), dev(self.u_final), n, path, nxt, ws=ws, stream=stream)
        torch.cuda.synchronize()
        return n.cpu().numpy(), path.cpu().numpy(), nxt.cpu().numpy()

    def check(self, **kw):
        got = self.run(**kw)
        want = ot.verify(self.cu, self.parent, self.tokens, self.target, self.draft, self.u_accept, self.u_final,
                         got[1].shape[1])
        for a, b, name in zip(got, want, ("accept_len", "path", "next_token")):
            assert np.array_equal(a, b), (name, a, b)
        return got


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 3, 127, 1000, 1024, 1025, 4097, 32000, 50257])
def test_vocabularies(vocab, drafts):
    Drafts([1, 8, 5, 12], vocab, drafts, seed=vocab).check()


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("shape,unused", [("chain", 0.0), ("chain", 0.2), ("tree", 0.0), ("tree", 0.3), ("forest", 0.1)])
def test_tree_shapes(shape, unused, drafts):
    for seed in range(4):
        Drafts([7, 20, 1, 64, 33], 300, drafts, shape, unused, seed=seed, near=0.3).check()


@pytest.mark.parametrize("drafts", [True, False])
def test_the_widest_trees_and_many_siblings(drafts):
    star = [[-1] + [0] * 255, [-1] + [0] * 20 + [3] * 20]
    got = Drafts([256, 41], 5000, drafts, seed=4, near=6.0, temp=1.0, parents=star).check()
    assert got[1].shape == (2, 256)
    Drafts([256], 64, drafts, "chain", seed=4, near=0.0).check()


@pytest.mark.parametrize("batch", [1, 3, 40, 200])
def test_batches(batch):
    counts = [1 + (7 * i) % 9 for i in range(batch)]
    Drafts(counts, 2000, True, seed=batch).check()


def test_odd_vocabulary_and_row_strides():
    for pad in (1, 2, 3, 4, 7):
        Drafts([9, 4], 1001, True, seed=pad).check(row_pad=pad)
        Drafts([9, 4], 1001, False, seed=pad).check(row_pad=pad)


def test_requests_without_work_and_short_paths():
    d = Drafts([0, 5, 0, 3], 100, True, seed=1)
    d.parent[d.cu[3]] = -2                                     # an idle request: node 0 not in use
    got = d.check()
    assert got[0][0] == 0 and got[2][0] == -1 and got[2][3] == -1 and np.all(got[1][3] == -1)
    d = Drafts([12], 50, True, "chain", seed=2, near=0.0)
    for pitch in (1, 2, 5, 12, 20):
        assert d.check(pitch=pitch)[0][0] <= pitch - 1


def test_identical_draft_and_target_accept_every_token():
    d = Drafts([9], 200, True, "chain", seed=3, near=0.0)
    d.draft = d.target.copy()
    assert d.check()[0][0] == 8


def test_random_numbers_at_the_ends_of_their_range():
    for u in (0.0, np.float32(1.0 - 2.0 ** -24)):
        d = Drafts([6, 6], 500, True, seed=5)
        d.u_accept[:], d.u_final[:] = u, u
        d.check()
        d = Drafts([6, 6], 500, False, seed=6)
        d.u_accept[:], d.u_final[:] = u, u
        d.check()
    # u_final = 1 (outside the promised range) still gives a token with weight
    d = Drafts([1], 500, True, seed=5)
    d.target[0, 250:] = 0
    d.u_final[:] = 1.0
    assert d.check()[2][0] == 249


def test_rows_with_zeros_and_without_weight():
    d = Drafts([4, 4, 1], 600, True, "chain", seed=7)
    d.target[0, :] = 0
    d.target[0, 599] = 1.0
    d.target[d.cu[1]] = np.nan                                 # no usable weight: no token
    d.target[d.cu[2], :] = 0
    got = d.check()
    assert got[2][1] == -1 and got[2][2] == -1
    # a draft row that covers all of the target's weight leaves no residual: the row itself is taken
    d = Drafts([2], 600, True, "chain", seed=8)
    d.target[0], d.draft[0] = 0, 0
    d.target[0, 5], d.draft[0, 5], d.draft[0, 9] = 0.5, 0.75, 0.25
    d.tokens[1], d.u_accept[1] = 9, 0.5
    got = d.check()
    assert got[0][0] == 0 and got[2][0] == 5


def test_bad_rows_parents_and_tokens_are_flagged():
    params = pa.make_params(pa.PA_MODE_DECODE, 1, 8, 8, 128, 1, max_kv_len=1)
    ws = alloc_ws(params)
    pa.attn_plan(params, torch.zeros(1, dtype=torch.int32, device=DEV), None, ws)
    d = Drafts([6, 6], 100, True, "chain", seed=9, near=0.0)
    d.check(ws=ws)
    assert pa.pa_read_device_error(ws) == pa.PA_OK
    for bad_token in (100, -1, 1 << 30):
        d = Drafts([6, 6], 100, True, "chain", seed=9, near=0.0)
        d.tokens[3] = bad_token
        assert d.check(ws=ws)[0][0] <= 2
        assert pa.pa_read_device_error(ws) == pa.PA_ERR_DEVICE_INDEX
    d = Drafts([6, 6], 100, True, "chain", seed=9, near=0.0)
    d.parent[2] = 4
    d.check(ws=ws)
    assert pa.pa_read_device_error(ws) == pa.PA_ERR_DEVICE_INDEX
    d.run()                                                    # without a workspace: skipped just the same
    d = Drafts([6, 6], 100, True, "chain", seed=9, near=0.0)
    d.cu[2] = 13
    got = d.run(ws=ws, pitch=6)
    assert got[0][1] == 0 and got[2][1] == -1 and np.all(got[1][1] == -1)
    assert pa.pa_read_device_error(ws) == pa.PA_ERR_DEVICE_INDEX


def test_the_verified_tokens_are_distributed_as_the_target():
    """A depth-one tree of 3 siblings, 20000 walks: the first token's frequencies match the target's row.

    The count of a token of probability p over N walks has deviation sqrt(N p (1 - p)); 5.5 deviations on
    12 tokens fail by chance with probability below 12 * 4e-8."""
    N, V = 20000, 12
    for drafts in (True, False):
        d = Drafts([4], V, True, seed=10, temp=1.0, near=1.0, parents=[[-1, 0, 0, 0]])
        rng = np.random.default_rng(1)
        row, q = d.target[0].astype(np.float64), d.draft[0].astype(np.float64)
        big = Drafts([4] * 1, V, drafts, seed=10, parents=[[-1, 0, 0, 0]])
        big.B, big.T = N, 4 * N
        big.cu = (4 * np.arange(N + 1)).astype(np.int32)
        big.parent = np.tile(np.array([-1, 0, 0, 0], np.int32), N)
        big.target = np.tile(d.target, (N, 1))
        big.draft = np.tile(d.draft, (N, 1)) if drafts else None
        if drafts:
            big.tokens = rng.choice(V, size=4 * N, p=q / q.sum()).astype(np.int32)
        else:
            big.tokens = np.tile(np.array([0, 3, 1, 7], np.int32), N)
        big.u_accept, big.u_final = rng.random(4 * N).astype(np.float32), rng.random(N).astype(np.float32)
        assert N > 8192                                        # run in parts of the largest batch
        first = []
        for a in range(0, N, 5000):
            part = Drafts([4], V, drafts, seed=0, parents=[[-1, 0, 0, 0]])
            part.B, part.T, part.cu = 5000, 20000, (4 * np.arange(5001)).astype(np.int32)
            s = slice(4 * a, 4 * a + 20000)
            part.parent, part.tokens, part.target = big.parent[s], big.tokens[s], big.target[s]
            part.draft = big.draft[s] if drafts else None
            part.u_accept, part.u_final = big.u_accept[s], big.u_final[a:a + 5000]
            n, path, nxt = part.run()
            tok = part.tokens.reshape(5000, 4)[np.arange(5000), np.maximum(path[:, 1], 0)]
            first.append(np.where(n > 0, tok, nxt))
        count = np.bincount(np.concatenate(first), minlength=V)
        p = row / row.sum()
        assert np.all(np.abs(count - N * p) <= 5.5 * np.sqrt(N * p * (1 - p))), (drafts, count, N * p)


def test_verify_on_another_stream():
    d = Drafts([9, 3, 17], 3000, True, seed=13)
    want = d.check()
    s = torch.cuda.Stream()
    for a, b in zip(want, d.run(stream=s)):
        assert np.array_equal(a, b)


# ------------------------------------------------------------------------------------- compaction

def compact_case(sizes, page, hkv, item, layers, seed):
    """Random accepted paths over random trees; pools of random bits."""
    rng = np.random.default_rng(seed)
    c = Case(sizes, 2 * hkv, hkv, page, seed=seed, shape="tree")
    pools = [torch.from_numpy(rng.integers(0, 256, (c.slots, hkv, 128 * item)).astype(np.uint8)).to(DEV)
             for _ in range(2 * layers)]
    pools = [p.view(torch.bfloat16) if item == 2 else p for p in pools]
    pitch = max(c.n + [1])
    path, length = np.full((c.B, pitch), -1, np.int32), np.zeros(c.B, np.int32)
    for r in range(c.B):
        if c.n[r] == 0:
            continue
        walk = [0]
        while True:
            kids = [i for i in range(c.n[r]) if c.parents[r][i] == walk[-1]]
            if not kids or rng.random() < 0.1:
                break
            walk.append(int(rng.choice(kids)))
        path[r, :len(walk)], length[r] = walk, len(walk) - 1
    return c, pools, path, length


def raw(p):
    return p.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("item", [1, 2])
@pytest.mark.parametrize("page,hkv,layers", [(1, 1, 1), (4, 3, 5), (16, 8, 16), (64, 2, 1), (256, 8, 2)])
def test_compaction_moves_the_accepted_rows(page, hkv, layers, item):
    c, pools, path, length = compact_case([(0, 9), (33, 40), (100, 1), (70, 0), (5, 256)], page, hkv, item, layers, page)
    want, lens = ot.kv_compact([raw(p) for p in pools], c.cu.cpu().numpy(), c.lens, length, path,
                               c.table.cpu().numpy(), page)
    out = torch.full((c.B,), 77, dtype=torch.int32, device=DEV)
    pa.attn_kv_compact(pa.make_pool_list(pools), c.seq_lens, c.cu, torch.from_numpy(length).to(DEV),
                       torch.from_numpy(path).to(DEV), c.table, page, out)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), lens)
    for p, w in zip(pools, want):
        assert np.array_equal(raw(p), w)


def test_compaction_of_dense_paths_that_overlap_themselves():
    """Every second node of a chain of 256, and of one where all are kept: each row is read before it is written."""
    for step in (1, 2, 3, 37):
        c, pools, path, length = compact_case([(20, 256), (7, 256)], 8, 2, 2, 2, step)
        walk = np.arange(0, 256, step)
        path[:, :] = -1
        path[0, :len(walk)], length[0] = walk, len(walk) - 1
        path[1, :2], length[1] = [0, 255], 1
        want, lens = ot.kv_compact([raw(p) for p in pools], c.cu.cpu().numpy(), c.lens, length, path,
                                   c.table.cpu().numpy(), 8)
        pa.attn_kv_compact(pa.make_pool_list(pools), c.seq_lens, c.cu, torch.from_numpy(length).to(DEV),
                           torch.from_numpy(path).to(DEV), c.table, 8)
        torch.cuda.synchronize()
        for p, w in zip(pools, want):
            assert np.array_equal(raw(p), w), step


def test_compaction_skips_and_flags_bad_entries():
    params = pa.make_params(pa.PA_MODE_DECODE, 1, 8, 8, 128, 1, max_kv_len=1)
    ws = alloc_ws(params)
    pa.attn_plan(params, torch.zeros(1, dtype=torch.int32, device=DEV), None, ws)

    def run(change, untouched):
        c, pools, path, length = compact_case([(20, 30), (9, 30)], 4, 2, 2, 1, 3)
        path[:, :] = -1
        path[:, :4], length[:] = [0, 3, 9, 20], 3
        before = [raw(p) for p in pools]
        good, _ = ot.kv_compact(before, c.cu.cpu().numpy(), c.lens, length, path, c.table.cpu().numpy(), 4)
        table = c.table.cpu().numpy().copy()
        t = dict(lens=c.seq_lens, cu=c.cu, path=torch.from_numpy(path).to(DEV), table=c.table,
                 length=torch.from_numpy(length).to(DEV))
        change(t)
        out = torch.zeros(2, dtype=torch.int32, device=DEV)
        pa.attn_kv_compact(pa.make_pool_list(pools), t["lens"], t["cu"], t["length"], t["path"], t["table"], 4, out,
                           ws=ws, max_q_tokens=60)
        assert pa.pa_read_device_error(ws) == pa.PA_ERR_DEVICE_INDEX
        for p, w, b in zip(pools, good, before):
            w = w.copy()
            for r, k in untouched:                             # rows that must not have moved
                slot = ot.gather_slots(table, c.lens[r], 4, r)[c.prefix[r] + k]
                w[slot] = b[slot]
            assert np.array_equal(raw(p), w)
        return out.cpu().numpy()

    def put(name, index, value):
        def change(t):
            t[name][index] = value
        return change

    run(put("path", (0, 2), 30), [(0, 2)])                     # not a node
    run(put("path", (0, 2), 1), [(0, 2)])                      # behind its own position
    run(put("path", (0, 2), -1), [(0, 2)])
    assert run(put("length", 1, 31), [(1, 1), (1, 2), (1, 3)])[1] == 39
    assert run(put("length", 1, -1), [(1, 1), (1, 2), (1, 3)])[1] == 39
    run(put("cu", 2, 61), [(1, 1), (1, 2), (1, 3)])
    run(put("lens", 1, 12), [(1, 1), (1, 2), (1, 3)])


def test_a_speculative_step_leads_to_the_cache_of_the_accepted_tokens():
    """Attention over the tree, verification, compaction: the next step over the compacted cache gives what a
    cache filled with the accepted tokens alone gives, in one captured graph as well."""
    c = Case([(150, 16), (31, 12), (0, 5)], 16, 4, 16, shape="tree", seed=21)
    d = Drafts(c.n, 500, True, seed=21, near=0.2, parents=c.parents)
    t = {k: torch.from_numpy(getattr(d, k)).to(DEV) for k in ("tokens", "target", "draft", "u_accept", "u_final")}
    params = c.params()
    ws = alloc_ws(params)
    out, lse = c.outputs()
    n, nxt, lens = (torch.zeros(c.B, dtype=torch.int32, device=DEV) for _ in range(3))
    path = torch.zeros(c.B, max(c.n), dtype=torch.int32, device=DEV)
    k0, v0 = c.k.clone(), c.v.clone()
    pools = pa.make_pool_list([c.k, c.v])

    def step():
        pa.attn_plan_tree(params, c.seq_lens, c.cu, c.parent, ws)
        c.attend(params, ws, out, lse)
        pa.attn_tree_verify(c.cu, c.parent, t["tokens"], t["target"], t["draft"], t["u_accept"], t["u_final"], n,
                            path, nxt, ws=ws)
        pa.attn_kv_compact(pools, c.seq_lens, c.cu, n, path, c.table, c.page, lens, ws=ws)

    def results():
        torch.cuda.synchronize()
        assert pa.pa_read_device_error(ws) == pa.PA_OK
        return [x.clone() for x in (out[:c.T], lse[:c.T], n, path, nxt, lens, c.k, c.v)]

    step()
    eager = results()
    c.k.copy_(k0)
    c.v.copy_(v0)
    c.check(out, lse, "tree")
    want = ot.verify(d.cu, d.parent, d.tokens, d.target, d.draft, d.u_accept, d.u_final, path.shape[1])
    for a, b in zip((n, path, nxt), want):
        assert np.array_equal(a.cpu().numpy(), b)
    wk, wl = ot.kv_compact([bits16(k0), bits16(v0)], d.cu, c.lens, want[0], want[1], c.table.cpu().numpy(), c.page)
    assert np.array_equal(bits16(eager[6]), wk[0]) and np.array_equal(bits16(eager[7]), wk[1])
    assert np.array_equal(lens.cpu().numpy(), wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.k.copy_(k0)
    c.v.copy_(v0)
    graph.replay()
    for a, b in zip(eager, results()):
        assert torch.equal(a.view(torch.int32) if a.dtype == torch.float32 else a.view(torch.int16),
                           b.view(torch.int32) if b.dtype == torch.float32 else b.view(torch.int16))
    # decode over the compacted cache: the accepted tokens as an ordinary prefix
    dparams = pa.make_params(pa.PA_MODE_DECODE, c.B, c.hq, c.hkv, 128, c.page, max_kv_len=c.L_max)
    dws = alloc_ws(dparams)
    q = torch.randn(c.B, c.hq, 128, device=DEV).to(torch.bfloat16)
    o = torch.empty_like(q)
    pa.attn_plan(dparams, lens, None, dws)
    pa.attn_decode_paged(dparams, dws, q, c.k, c.v, c.table, c.scale, o)
    from oracle import attention as oa
    from tests.helpers import assert_bf16_close
    ref, _ = oa.decode(bits16(q), wk[0], wk[1], c.table.cpu().numpy(), wl, c.page, c.scale)
    assert_bf16_close(o, ref, "decode after compaction")


def test_compaction_far_behind_four_gigabytes():
    c, pools, path, length = compact_case([(33, 40), (100, 9)], 16, 8, 2, 1, 51)
    length[:], path[:] = 0, -1
    for r, walk in enumerate(([0, 2, 3, 17, 39], [0, 8])):
        path[r, :len(walk)], length[r] = walk, len(walk) - 1
    want, lens = ot.kv_compact([raw(p) for p in pools], c.cu.cpu().numpy(), c.lens, length, path,
                               c.table.cpu().numpy(), 16)
    slots = (2 ** 32 // 2048 // 16 + 8) * 16 + c.slots
    big = [torch.empty((slots,) + tuple(p.shape[1:]), dtype=p.dtype, device=DEV) for p in pools]
    for b, p in zip(big, pools):
        b[-c.slots:] = p
    out = torch.full((c.B,), 77, dtype=torch.int32, device=DEV)
    pa.attn_kv_compact(pa.make_pool_list(big), c.seq_lens, c.cu, torch.from_numpy(length).to(DEV),
                       torch.from_numpy(path).to(DEV), c.table + (slots - c.slots) // 16, 16, out)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), lens)
    for b, w in zip(big, want):
        assert np.array_equal(raw(b[-c.slots:]), w)


def test_probability_rows_far_behind_2_to_the_31():
    d = Drafts([17, 4], 1000, seed=52)
    n, path, nxt = d.run()
    pitch = 2 ** 27 + 4
    assert (d.T - 1) * pitch > 2 ** 31
    rows = []
    for a in (d.target, d.draft):
        wide = torch.empty(d.T * pitch, device=DEV).view(d.T, pitch)[:, :1000]
        wide.copy_(torch.from_numpy(a))
        rows.append(wide)
    t = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    got = [torch.full_like(t(a), 77) for a in (n, path, nxt)]
    pa.attn_tree_verify(t(d.cu), t(d.parent), t(d.tokens), rows[0], rows[1], t(d.u_accept), t(d.u_final), *got)
    torch.cuda.synchronize()
    for a, b in zip(got, (n, path, nxt)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_draft_probabilities_of_either_zero(zero):
    """A draft probability of zero, of either sign, leaves the token's weight as it is."""
    for seed in range(6):
        d = Drafts([3, 9, 5], 700, True, seed=seed, near=4.0, temp=1.0)
        d.draft[:, ::3] = zero
        d.u_accept[:] = 0.999
        d.check()
    # the only weight that a rejection leaves lies on such tokens
    d = Drafts([2], 700, True, "chain", seed=9)
    d.target[0], d.draft[0] = 0, zero
    d.target[0, 5], d.target[0, 600], d.draft[0, 5], d.tokens[1], d.u_accept[1] = 0.25, 0.75, 1.0, 5, 0.5
    assert d.check()[2][0] == 600


def test_a_step_whose_rows_start_behind_others():
    """Verification and compaction with offsets that do not start at 0."""
    skip = 37
    for drafts in (True, False):
        d = Drafts([6, 9, 1], 1001, drafts, seed=63)
        want = d.run()
        for name in ("target", "draft"):
            rows = getattr(d, name)
            if rows is not None:
                setattr(d, name, np.concatenate([np.full((skip, 1001), np.nan, np.float32), rows]))
        d.parent = np.concatenate([np.full(skip, 9, np.int32), d.parent])
        d.tokens = np.concatenate([np.full(skip, -5, np.int32), d.tokens])
        d.u_accept = np.concatenate([np.full(skip, np.nan, np.float32), d.u_accept])
        d.cu = d.cu + np.int32(skip)
        params = pa.make_params(pa.PA_MODE_DECODE, 1, 8, 8, 128, 1, max_kv_len=1)
        ws = alloc_ws(params)
        pa.attn_plan(params, torch.zeros(1, dtype=torch.int32, device=DEV), None, ws)
        for a, b in zip(d.check(pitch=9, ws=ws), want):
            assert np.array_equal(a, b)
        assert pa.pa_read_device_error(ws) == pa.PA_OK
    c, pools, path, length = compact_case([(20, 30), (9, 12)], 4, 2, 2, 1, 3)
    want, lens = ot.kv_compact([raw(p) for p in pools], c.cu.cpu().numpy(), c.lens, length, path,
                               c.table.cpu().numpy(), 4)
    out = torch.zeros(2, dtype=torch.int32, device=DEV)
    pa.attn_kv_compact(pa.make_pool_list(pools), c.seq_lens, c.cu + skip, torch.from_numpy(length).to(DEV),
                       torch.from_numpy(path).to(DEV), c.table, 4, out, ws=ws, max_q_tokens=c.T + skip)
    assert pa.pa_read_device_error(ws) == pa.PA_OK
    assert np.array_equal(out.cpu().numpy(), lens)
    for p, w in zip(pools, want):
        assert np.array_equal(raw(p), w)


def test_compaction_needs_no_bound_on_the_rows():
    """Offsets far behind other rows (a long prefill in the same batch), without max_q_tokens."""
    c, pools, path, length = compact_case([(20, 30), (9, 12)], 4, 2, 2, 1, 5)
    length[:], path[:] = 0, -1
    for r, walk in enumerate(([0, 2, 17, 29], [0, 11])):
        path[r, :len(walk)], length[r] = walk, len(walk) - 1
    want, lens = ot.kv_compact([raw(p) for p in pools], c.cu.cpu().numpy(), c.lens, length, path,
                               c.table.cpu().numpy(), 4)
    out = torch.zeros(2, dtype=torch.int32, device=DEV)
    pa.attn_kv_compact(pa.make_pool_list(pools), c.seq_lens, c.cu + 100000, torch.from_numpy(length).to(DEV),
                       torch.from_numpy(path).to(DEV), c.table, 4, out)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), lens)
    for p, w in zip(pools, want):
        assert np.array_equal(raw(p), w)


class WideRows(Drafts):
    """Few nodes over a long vocabulary, rows cheap to make: target and draft from uniform numbers."""

    def __init__(self, counts, vocab, drafts, seed):
        super().__init__(counts, 2, drafts, "chain", seed=seed)
        rng = np.random.default_rng(seed)
        self.vocab = vocab
        self.target, draft = (rng.random((self.T, vocab), dtype=np.float32) for _ in range(2))
        self.target /= self.target.sum(-1, keepdims=True)
        draft /= draft.sum(-1, keepdims=True)
        self.draft = draft if drafts else None
        self.tokens = rng.integers(0, vocab, self.T).astype(np.int32)


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("counts,vocab", [
    ([3, 2], 128256),                                          # 8 CTAs a request, 32 chunks of 512 tokens each
    ([2] * 80, 128256),                                        # 4 CTAs, 63 chunks
    ([1] * 310, 50001),                                        # 1 CTA, 98 chunks
    ([2, 1], 1 << 20),                                         # 8 CTAs, 256 chunks
])
def test_long_vocabularies_in_many_chunks(counts, vocab, drafts):
    """More chunks than warps and than lanes of the final search, drawn all along the vocabulary."""
    d = WideRows(counts, vocab, drafts, seed=vocab % 1000 + len(counts))
    d.u_final[:] = ((np.arange(d.B) + 0.5) / d.B).astype(np.float32)
    d.check()
    for u in (0.0, 0.03, 0.5, 0.97, 1 - 2.0 ** -24):
        d.u_final[:] = np.float32(u)
        d.check()


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("batch,vocab", [(2, 1 << 20), (3, (1 << 20) - 511), (310, 50001)])
def test_weight_in_few_chunks_of_a_long_vocabulary(batch, vocab, drafts):
    """All weight in the last chunk, or at single tokens of the first, a middle and the last chunk: the sums carried
    over the chunks before have to be right."""
    d = WideRows([1] * batch, vocab, drafts, seed=7)
    d.target[:] = 0
    d.target[:, -5:] = [0.25, 0, 0.25, 0.25, 0.25]
    got = d.check()
    assert np.all(got[2] >= vocab - 5)
    d.target[:] = 0
    at = [3, 511, 512, vocab // 2, vocab - 20000, vocab - 1]
    d.target[:, at] = 1 / 6
    for i, x in enumerate(at):
        d.u_final[:] = np.float32((i + 0.5) / 6)
        assert np.all(d.check()[2] == x)
