"""Host-side checks of the speculative-decoding entry points (no GPU needed), and the oracle's pins."""
import ctypes
import os

import numpy as np
import pytest
import torch

import paged_kv_flashattention_split_b200 as pa
from oracle import attention as oa
from oracle import tree as ot
from paged_kv_flashattention_split_b200 import build as pa_build

INVALID, UNSUPPORTED, WORKSPACE = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pa.LIB_PATH):
        pa_build.build()
    return pa.lib()


def P(**kw):
    base = dict(mode=pa.PA_MODE_TREE, batch=4, hq=8, hkv=2, head_dim=128, page_size=16, max_kv_len=300,
                max_q_tokens=64, num_sms=148)
    base.update(kw)
    return pa.make_params(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(max_q_tokens=0), INVALID),
    (dict(max_splits=1), INVALID),
    (dict(sage_k_block=64), INVALID),
    (dict(head_dim=64), UNSUPPORTED),
    (dict(page_size=3), UNSUPPORTED),
    (dict(hq=32, hkv=2), UNSUPPORTED),
    (dict(hq=6, hkv=4), INVALID),
    (dict(batch=0), INVALID),
    (dict(batch=8193), INVALID),
    (dict(batch=8192, max_q_tokens=2 ** 30), UNSUPPORTED),
    (dict(max_kv_len=2 ** 31 - 2048, batch=200), UNSUPPORTED),    # the plan counts key tiles in 32 bits
    (dict(max_kv_len=2 ** 22, batch=8192, hq=64, hkv=8), UNSUPPORTED),   # whatever the rows' offsets hold
    (dict(max_kv_len=2 ** 31 - 1, batch=1, max_q_tokens=1), UNSUPPORTED),   # so are key positions, read ahead
])
def test_plan_parameters(lib, kw, status):
    assert pa.pa_plan_workspace_size(P(**kw), raise_on_error=False) == status


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2), (24, 3)])
def test_workspace_size_is_the_documented_layout(lib, hq, hkv):
    up = lambda x: -(-x // 256) * 256   # noqa: E731
    B, Tq, C = 4, 1000, max(1, 148 // hkv)
    tiles = Tq // (256 // (hq // hkv)) + B
    off = 64 + 4 * (5 * B + 1)
    off = up(-(-off // 16) * 16 + 16 * (C + tiles))
    off = up(off + 4 * (C + 1))
    off = up(off + 8 * min(max(1, C - 1), tiles))
    off = up(off + 4 * 8 * Tq)
    off = up(off + 4 * 2 * C * hkv * 256 * 128)
    off = up(off + 4 * 2 * C * hkv * 256)
    assert pa.pa_plan_workspace_size(P(hq=hq, hkv=hkv, max_q_tokens=Tq)) == off


def test_plan_and_attention_refusals(lib):
    p, big = P(), 1 << 40
    ref = ctypes.byref
    assert lib.attn_plan(ref(p), 16, 32, 256, big, None) == INVALID             # a tree plan needs the parents
    assert lib.attn_plan_tree(None, 16, 32, 48, 256, big, None) == INVALID
    assert lib.attn_plan_tree(ref(P(mode=pa.PA_MODE_DECODE, max_q_tokens=0)), 16, 32, 48, 256, big, None) == INVALID
    for i in range(4):
        args = [16, 32, 48, 256]
        args[i] = None
        assert lib.attn_plan_tree(ref(p), *args, big, None) == INVALID
    assert lib.attn_plan_tree(ref(p), 16, 32, 48, 264, big, None) == INVALID
    assert lib.attn_plan_tree(ref(p), 16, 32, 48, 256, 4096, None) == WORKSPACE

    def tree(params=p, ws=256, nbytes=big, q=256, k=256, v=256, slots=1000, table=256, pitch=19, out=256, lse=None):
        a = lib.attn_tree_paged(ref(params), ws, nbytes, q, k, v, slots, table, pitch, 1.0, out, lse, None)
        b = lib.attn_tree_paged_fp8(ref(params), ws, nbytes, q, k, v, 1.0, 1.0, slots, table, pitch, 1.0, out, lse, None)
        assert a == b
        return a

    for name in ("ws", "q", "k", "v", "table", "out"):
        assert tree(**{name: None}) == INVALID
    for name in ("ws", "q", "k", "v", "out"):
        assert tree(**{name: 264}) == INVALID
    assert tree(lse=258) == INVALID
    assert tree(pitch=18) == INVALID                                             # fewer than ceil(300 / 16) entries
    assert tree(slots=0) == INVALID
    assert tree(slots=1 << 31) == INVALID
    assert tree(nbytes=4096) == WORKSPACE
    assert tree(params=P(mode=pa.PA_MODE_EXTEND)) == WORKSPACE
    assert tree(params=P(mode=pa.PA_MODE_DECODE, max_q_tokens=0)) == WORKSPACE


def test_verify_refusals(lib):
    def verify(batch=2, rows=8, vocab=100, cu=16, parent=16, tokens=16, target=16, tp=100, draft=16, dp=100, ua=16,
               uf=16, n=16, path=16, pitch=4, nxt=16, ws=None):
        return lib.attn_tree_verify(batch, rows, vocab, cu, parent, tokens, target, tp, draft, dp, ua, uf, n, path,
                                    pitch, nxt, ws, None)

    for kw in (dict(batch=0), dict(batch=8193), dict(rows=0), dict(vocab=0), dict(pitch=0), dict(tp=99), dict(dp=99),
               dict(draft=None), dict(draft=None, dp=-1), dict(ws=8)):
        assert verify(**kw) == INVALID, kw
    assert verify(vocab=(1 << 20) + 1, tp=1 << 21, dp=1 << 21) == UNSUPPORTED
    for name in ("cu", "parent", "tokens", "target", "ua", "uf", "n", "path", "nxt"):
        assert verify(**{name: None}) == INVALID, name
        assert verify(**{name: 18}) == INVALID, name
    assert verify(draft=18) == INVALID


def test_compact_refusals(lib):
    def compact(pools=(256, 512), count=None, hkv=2, d=128, item=2, slots=100, batch=2, rows=8, lens=16, cu=16, n=16,
                path=16, pp=4, table=16, pitch=4, page=16, out=None, ws=None):
        array = (ctypes.c_void_p * max(1, len(pools)))(*pools)
        return lib.attn_kv_compact(array, len(pools) if count is None else count, hkv, d, item, slots, batch, rows,
                                   lens, cu, n, path, pp, table, pitch, page, out, ws, None)

    for kw in (dict(count=0), dict(hkv=0), dict(batch=0), dict(batch=8193), dict(rows=0), dict(pp=0), dict(pitch=0),
               dict(slots=0), dict(slots=1 << 31), dict(pools=(256, None)), dict(pools=(256, 264)),
               dict(pools=(256, 256)), dict(out=16), dict(ws=8), dict(out=18)):
        assert compact(**kw) == INVALID, kw
    for kw in (dict(d=64), dict(item=4), dict(page=0), dict(page=3), dict(page=512),
               dict(pools=tuple(256 * (i + 1) for i in range(257)))):
        assert compact(**kw) == UNSUPPORTED, kw
    for name in ("lens", "cu", "n", "path", "table"):
        assert compact(**{name: None}) == INVALID, name
        assert compact(**{name: 18}) == INVALID, name


def test_binding_refusals():
    with pytest.raises(ValueError):
        pa.make_pool_list([torch.zeros(4, 2, 128), torch.zeros(5, 2, 128)])
    with pytest.raises(ValueError):
        pa.make_pool_list([torch.zeros(4, 128, 2).transpose(1, 2)])
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.attn_tree_verify(torch.zeros(2, **i32), torch.zeros(4, **i32), torch.zeros(4, **i32),
                            torch.zeros(10, 4).t(), None, torch.zeros(4), torch.zeros(1), torch.zeros(1, **i32),
                            torch.zeros(1, 4, **i32), torch.zeros(1, **i32))
    with pytest.raises(ValueError):
        pa.make_pool_list([])
    with pytest.raises(ValueError):
        pa.make_pool_list([torch.zeros(4, 128)])
    with pytest.raises(ValueError):                                # a view of longer rows, shorter than the target's
        pa.attn_tree_verify(torch.zeros(2, **i32), torch.zeros(4, **i32), torch.zeros(4, **i32), torch.zeros(4, 10),
                            torch.zeros(4, 10)[:, :8], torch.zeros(4), torch.zeros(1), torch.zeros(1, **i32),
                            torch.zeros(1, 4, **i32), torch.zeros(1, **i32))


# ------------------------------------------------------------------------------------- oracle pins

def test_visibility():
    see = ot.visibility([-1, 0, 0, 2, -2, 4, -1, 9, 6])
    want = np.zeros((9, 9), bool)
    for i, js in enumerate([[0], [0, 1], [0, 2], [0, 2, 3], [], [], [6], [], [6, 8]]):
        want[i, js] = True
    assert np.array_equal(see, want)


def test_a_chain_is_the_causal_extend():
    rng = np.random.default_rng(0)
    bits = lambda *s: (rng.standard_normal(s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)   # noqa: E731
    q, k, v = bits(9, 4, 128), bits(64, 2, 128), bits(64, 2, 128)
    cu, lens = np.array([0, 4, 9]), np.array([20, 5])
    table = rng.permutation(16).reshape(2, 8)
    parent = [-1, 0, 1, 2, -1, 0, 1, 2, 3]
    o, lse, _ = ot.tree_attention(q, cu, parent, k, v, table, lens, 4, 0.1)
    ref, ref_lse = oa.extend(q, cu, k, v, table, lens, 4, 0.1)
    assert np.allclose(o, ref, atol=1e-13) and np.allclose(lse, ref_lse, atol=1e-13)


@pytest.mark.parametrize("drafts", [True, False])
def test_verification_preserves_the_target_distribution(drafts):
    """The exact distribution of the first token: sums over the drafted tokens, integrals over u by the rule itself.

    With independent siblings drawn from q, P(first token = x) = target(x) for every number of siblings."""
    rng = np.random.default_rng(3)
    V, N = 5, 60000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    target, draft = np.tile(p.astype(np.float32), (3, 1)), np.tile(q.astype(np.float32), (3, 1))
    count = np.zeros(V)
    for _ in range(N // 20):
        tok = np.array([0, *rng.choice(V, size=2, p=q)]) if drafts else np.array([0, 1, 4])
        n, path, nxt = ot.verify([0, 3], [-1, 0, 0], tok, target, draft if drafts else None, rng.random(3),
                                 rng.random(1), 3)
        count[tok[path[0, 1]] if n[0] else nxt[0]] += 1
    m = N // 20
    assert np.all(np.abs(count - m * p) <= 5.5 * np.sqrt(m * p * (1 - p)))


def test_compaction_oracle():
    pool = np.arange(12)[:, None].copy()
    (new,), lens = ot.kv_compact([pool], [0, 4, 6], [6, 3], np.array([2, 0]), np.array([[0, 2, 3], [-1, -1, -1]]),
                                 np.array([[2, 0, 1], [3, 4, 5]]), 2)
    # request 0: prefix 2 at slots 4 5, nodes at 0 1 2 3; node 2 -> position 3 (slot 1), node 3 -> position 4 (slot 2)
    assert new[:, 0].tolist() == [0, 2, 3, 3, 4, 5, 6, 7, 8, 9, 10, 11] and lens.tolist() == [5, 1]


# ------------------------------------------------------------------------------------- arguments of the binding

def step_arguments(B=2, T=6, vocab=40, pitch=4):
    """Arguments of a verification and of a compaction over host memory: they are to be refused before any launch."""
    i32 = dict(dtype=torch.int32)
    verify = dict(cu_seqlens_q=torch.zeros(B + 1, **i32), parent=torch.zeros(T, **i32), tokens=torch.zeros(T, **i32),
                  target_probs=torch.zeros(T, vocab), draft_probs=torch.zeros(T, vocab), u_accept=torch.zeros(T),
                  u_final=torch.zeros(B), accept_len=torch.zeros(B, **i32), accept_path=torch.zeros(B, pitch, **i32),
                  next_token=torch.zeros(B, **i32))
    compact = dict(pool_list=pa.make_pool_list([torch.zeros(16, 2, 128, dtype=torch.bfloat16)]),
                   seq_lens=torch.zeros(B, **i32), cu_seqlens_q=torch.zeros(B + 1, **i32),
                   accept_len=torch.zeros(B, **i32), accept_path=torch.zeros(B, pitch, **i32),
                   page_table=torch.zeros(B, 4, **i32), page_size=4, seq_lens_out=torch.zeros(B, **i32))
    return verify, compact


@pytest.mark.parametrize("path", [
    lambda: torch.zeros(2, 10, dtype=torch.int32)[:, 2:8],         # columns inside longer rows
    lambda: torch.zeros(2, 10, dtype=torch.int32)[:, :4],
    lambda: torch.zeros(4, 2, dtype=torch.int32).t(),
    lambda: torch.zeros(8, dtype=torch.int32),                     # no rows
    lambda: torch.zeros(1, 4, dtype=torch.int32),                  # fewer rows than requests
])
def test_accepted_paths_are_dense_rows(lib, path):
    """The kernels take the width of a path for its stride: a fill of wider rows would leave the view."""
    verify, compact = step_arguments()
    with pytest.raises(ValueError, match="path"):
        pa.attn_tree_verify(**dict(verify, accept_path=path()))
    with pytest.raises(ValueError, match="path"):
        pa.attn_kv_compact(**dict(compact, accept_path=path()))


def test_one_accepted_path_out_of_longer_rows_has_its_own_width(lib, monkeypatch):
    """A single row is dense whatever its stride; its pitch is its width."""
    verify, compact = step_arguments(B=1, T=3)
    view = torch.zeros(1, 10, dtype=torch.int32)[:, 2:8]
    seen = {}

    class Fake:
        def attn_tree_verify(self, *args):
            seen["verify"] = args[14]
            return pa.PA_OK

        def attn_kv_compact(self, *args):
            seen["compact"] = args[12]
            return pa.PA_OK

    monkeypatch.setattr(pa._binding, "lib", lambda: Fake())
    pa.attn_tree_verify(**dict(verify, accept_path=view))
    pa.attn_kv_compact(**dict(compact, accept_path=view))
    assert seen == dict(verify=6, compact=6)


@pytest.mark.parametrize("name,wrong", [
    (name, wrong) for name in ("cu_seqlens_q", "parent", "tokens", "accept_len", "accept_path", "next_token")
    for wrong in (torch.int64, torch.float32)] + [
    (name, wrong) for name in ("target_probs", "draft_probs", "u_accept", "u_final")
    for wrong in (torch.bfloat16, torch.float64, torch.int32)])
def test_verification_refuses_other_types(lib, name, wrong):
    """The kernel reads 32-bit words: 64-bit tokens (as argmax and topk give) would be taken for other tokens."""
    verify, _ = step_arguments()
    with pytest.raises(ValueError, match=name):
        pa.attn_tree_verify(**dict(verify, **{name: verify[name].to(wrong)}))


@pytest.mark.parametrize("name", ["cu_seqlens_q", "parent", "tokens", "u_accept", "u_final", "accept_len", "next_token"])
def test_verification_refuses_strided_vectors(lib, name):
    verify, _ = step_arguments()
    strided = torch.zeros(len(verify[name]), 2, dtype=verify[name].dtype)[:, 0]
    with pytest.raises(ValueError, match=name):
        pa.attn_tree_verify(**dict(verify, **{name: strided}))


@pytest.mark.parametrize("name", ["cu_seqlens_q", "u_final", "next_token"])
def test_verification_refuses_vectors_shorter_than_the_batch(lib, name):
    verify, _ = step_arguments()
    with pytest.raises(ValueError, match=name):
        pa.attn_tree_verify(**dict(verify, **{name: verify[name][:-1]}))


@pytest.mark.parametrize("name", ["seq_lens", "cu_seqlens_q", "accept_len", "accept_path", "page_table", "seq_lens_out"])
def test_compaction_refuses_other_types_and_strides(lib, name):
    _, compact = step_arguments()
    t = compact[name]
    wrong = [t.to(torch.int64), t.to(torch.float32), torch.stack([t, t], -1)[..., 0]]
    for bad in wrong:
        with pytest.raises(ValueError, match="path" if name == "accept_path" else name):
            pa.attn_kv_compact(**dict(compact, **{name: bad}))
    if name in ("seq_lens", "cu_seqlens_q", "page_table", "seq_lens_out"):
        with pytest.raises(ValueError, match=name):
            pa.attn_kv_compact(**dict(compact, **{name: t[:-1]}))


def test_addresses_are_taken_as_they_are(lib, monkeypatch):
    """A device address instead of a tensor has no type to check."""
    verify, compact = step_arguments()
    seen = []

    class Fake:
        def attn_tree_verify(self, *args):
            seen.append(args)
            return pa.PA_OK

        def attn_kv_compact(self, *args):
            seen.append(args)
            return pa.PA_OK

    monkeypatch.setattr(pa._binding, "lib", lambda: Fake())
    pa.attn_tree_verify(**dict(verify, tokens=4096, u_accept=8192, draft_probs=None))
    pa.attn_kv_compact(**dict(compact, seq_lens=4096, seq_lens_out=None))
    assert seen[0][5] == 4096 and seen[0][10] == 8192 and seen[0][8] is None and seen[0][9] == 0
    assert seen[1][8] == 4096 and seen[1][16] is None


def attention_arguments(fp8=False, B=2, T=6):
    """Arguments of a tree plan and of one layer's attention over host memory."""
    i32 = dict(dtype=torch.int32)
    params = P(batch=B, max_q_tokens=T, max_kv_len=30)
    ws = torch.zeros(64, dtype=torch.uint8)
    plan = dict(params=params, seq_lens=torch.zeros(B, **i32), cu_seqlens_q=torch.zeros(B + 1, **i32),
                parent=torch.zeros(T, **i32), ws=ws)
    kind = torch.uint8 if fp8 else torch.bfloat16
    pools = [torch.zeros(64, 2, 128, dtype=kind) for _ in range(2)]
    layer = dict(params=params, ws=ws, q=torch.zeros(T, 8, 128, dtype=torch.bfloat16), page_table=torch.zeros(B, 4, **i32),
                 sm_scale=0.1, out=torch.zeros(T, 8, 128, dtype=torch.bfloat16), lse_out=torch.zeros(T, 8))
    layer.update(dict(k8_pool=pools[0], v8_pool=pools[1], k_scale=1.0, v_scale=1.0) if fp8 else
                 dict(k_pool=pools[0], v_pool=pools[1]))
    return plan, layer


@pytest.mark.parametrize("name", ["seq_lens", "cu_seqlens_q", "parent"])
def test_tree_plan_refuses_other_types_and_strides(lib, name):
    """A tree built by torch.tensor of Python integers is 64-bit: its words would be read as another tree."""
    plan, _ = attention_arguments()
    t = plan[name]
    bad = [t.to(torch.int64), t.to(torch.float32), torch.stack([t, t], -1)[..., 0]]
    bad += [] if name == "parent" else [t[:-1]]
    for x in bad:
        with pytest.raises(ValueError, match=name):
            pa.attn_plan_tree(**dict(plan, **{name: x}))


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_refuses_other_types_and_strides(lib, fp8):
    _, layer = attention_arguments(fp8)
    call = pa.attn_tree_paged_fp8 if fp8 else pa.attn_tree_paged
    k, v = ("k8_pool", "v8_pool") if fp8 else ("k_pool", "v_pool")
    wide = torch.zeros(6, 12, 128, dtype=torch.bfloat16)                       # queries inside a fused projection
    bad = [("q", wide[:, :8]), ("out", wide[:, :8]), ("q", layer["q"].float()), ("out", layer["out"].half()),
           ("lse_out", layer["lse_out"].double()), ("lse_out", torch.zeros(6, 12)[:, :8]),
           ("page_table", layer["page_table"].long()), ("page_table", torch.zeros(2, 8, dtype=torch.int32)[:, :4]),
           ("page_table", layer["page_table"][:1])]
    for name in (k, v):
        other = torch.bfloat16 if fp8 else torch.uint8
        bad += [(name, layer[name].to(other)), (name, layer[name].float()), (name, layer[name].transpose(0, 1))]
    for name, x in bad:
        with pytest.raises(ValueError, match=name):
            call(**dict(layer, **{name: x}))


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_takes_bit_patterns_and_a_given_pitch(lib, monkeypatch, fp8):
    """Raw 16-bit patterns, torch's own E4M3 type, and a table inside longer rows with its pitch given."""
    _, layer = attention_arguments(fp8)
    seen = []

    class Fake:
        def attn_tree_paged(self, *args):
            seen.append(args[8])
            return pa.PA_OK

        def attn_tree_paged_fp8(self, *args):
            seen.append(args[10])
            return pa.PA_OK

    monkeypatch.setattr(pa._binding, "lib", lambda: Fake())
    table = torch.zeros(2, 9, dtype=torch.int32)
    layer.update(q=layer["q"].view(torch.int16), out=layer["out"].view(torch.uint16), page_table=table[:, 2:6], pt_pitch=9)
    if fp8:
        layer.update(k8_pool=layer["k8_pool"].view(torch.float8_e4m3fn), v8_pool=layer["v8_pool"].view(torch.int8))
        pa.attn_tree_paged_fp8(**layer)
    else:
        layer.update(k_pool=layer["k_pool"].view(torch.int16))
        pa.attn_tree_paged(**layer)
    assert seen == [9]


def test_compaction_refuses_pools_that_overlap(lib, monkeypatch):
    """Rows in two pools of a list would move twice, in no order."""
    monkeypatch.setenv("PAGEDATTN_TEST_FORCE_ARCH", "90")          # what is accepted ends before a launch
    row, slots = 2 * 128 * 2, 100

    def compact(*pools):
        return lib.attn_kv_compact((ctypes.c_void_p * len(pools))(*pools), len(pools), 2, 128, 2, slots, 2, 8, 16, 16, 16,
                                   16, 4, 16, 4, 16, None, None, None)

    a = 1 << 30
    for other in (a, a + 16, a + (slots - 1) * row, a + slots * row - 16, a - 16, a - slots * row + 16):
        assert compact(a, other) == INVALID
        assert compact(a + 4 * slots * row, a, a + 2 * slots * row, other) == INVALID
    for other in (a + slots * row, a - slots * row, a + 9 * slots * row):
        assert compact(a, other) in (pa.PA_ERR_ARCH, pa.PA_ERR_CUDA)


def test_host_tensors_are_refused_where_there_is_a_device(lib, monkeypatch):
    """A tree built on the host and forgotten there is refused, not read by the kernel; pinned memory is in reach."""
    calls = []

    class Fake:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or pa.PA_OK

    monkeypatch.setattr(pa._binding, "lib", lambda: Fake())
    monkeypatch.setattr(pa._binding, "_stream_of", lambda here, stream: None)
    plan, layer = attention_arguments()
    _, layer8 = attention_arguments(fp8=True)
    verify, compact = step_arguments()
    for call, args in ((pa.attn_plan_tree, plan), (pa.attn_tree_paged, layer), (pa.attn_tree_paged_fp8, layer8),
                       (pa.attn_tree_verify, verify), (pa.attn_kv_compact, compact)):
        monkeypatch.setattr(pa._binding, "_here", lambda: -1)
        call(**args)                                               # host tensors, no device: the library answers
        monkeypatch.setattr(pa._binding, "_here", lambda: 0)
        for name in [k for k, v in args.items() if isinstance(v, (torch.Tensor, pa._binding.PoolList))]:
            # all other tensors count as pinned
            monkeypatch.setattr(pa._binding, "_elsewhere",
                                lambda n, t, name=name: elsewhere(n, t) if n == name.replace("pool_list", "pools") else None)
            with pytest.raises(ValueError, match="not on the current device"):
                call(**args)
    assert calls == ["attn_plan_tree", "attn_tree_paged", "attn_tree_paged_fp8", "attn_tree_verify", "attn_kv_compact"]


elsewhere = pa._binding._elsewhere


# ------------------------------------------------------------------------------------- more pins of the oracle

def bits_of(rng, *shape):
    return (rng.standard_normal(shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_one_node_is_the_decode():
    rng = np.random.default_rng(4)
    q, k, v = bits_of(rng, 3, 4, 128), bits_of(rng, 64, 2, 128), bits_of(rng, 64, 2, 128)
    lens, table = np.array([20, 1, 32]), rng.permutation(16)[None, :8].repeat(3, 0)
    o, lse, _ = ot.tree_attention(q, np.arange(4), [-1, -1, -1], k, v, table, lens, 4, 0.1)
    ref, ref_lse = oa.decode(q, k, v, table, lens, 4, 0.1)
    assert np.allclose(o, ref, atol=1e-13) and np.allclose(lse, ref_lse, atol=1e-13)


def test_the_fp8_form_is_the_bf16_form_of_the_dequantised_cache():
    """Scales that are powers of two: every dequantised value is a bf16 value."""
    rng = np.random.default_rng(5)
    codes = np.array([x for x in range(256) if x & 0x7F != 0x7F], dtype=np.uint8)
    q = bits_of(rng, 9, 4, 128)
    k8, v8 = rng.choice(codes, (64, 2, 128)), rng.choice(codes, (64, 2, 128))
    table, lens, cu = rng.permutation(16).reshape(2, 8), np.array([20, 5]), np.array([0, 4, 9])
    parent = [-1, 0, 0, 1, -1, -2, 0, 1, 2]
    from oracle.codecs import e4m3_to_f64
    as_bf16 = lambda c, s: ((e4m3_to_f64(c) * s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)   # noqa: E731
    a = ot.tree_attention(q, cu, parent, k8, v8, table, lens, 4, 0.01, 2.0 ** -4, 2.0 ** -6)
    b = ot.tree_attention(q, cu, parent, as_bf16(k8, 2.0 ** -4), as_bf16(v8, 2.0 ** -6), table, lens, 4, 0.01)
    for x, y in zip(a, b):
        assert np.array_equal(np.isneginf(x), np.isneginf(y)) and np.allclose(x, y, atol=1e-13)


def test_unused_nodes_give_and_change_nothing():
    rng = np.random.default_rng(6)
    q, k, v = bits_of(rng, 5, 2, 128), bits_of(rng, 16, 1, 128), bits_of(rng, 16, 1, 128)
    args = ([0, 5], [-1, -2, 0, 1, 2], k, v, np.arange(16)[None], [12], 1, 0.1)      # node 3 hangs below node 1
    o, lse, _ = ot.tree_attention(q, *args)
    assert np.all(o[[1, 3]] == 0) and np.all(np.isneginf(lse[[1, 3]])) and np.all(np.isfinite(lse[[0, 2, 4]]))
    for x in (k, v):
        x[[8, 10]] = 0x7FC0                                                          # their rows: NaN
    again, lse2, _ = ot.tree_attention(q, *args)
    assert np.array_equal(o, again) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("seed", range(12))
def test_plan_invariants(seed):
    """Every (query tile, key tile) unit once and in order, runs of at most `per` a slot, cut tiles listed."""
    rng = np.random.default_rng(seed)
    B, (hq, hkv) = int(rng.integers(1, 9)), [(8, 8), (8, 4), (16, 4), (32, 4)][seed % 4]
    n = rng.integers(0, 60, B)
    lens = n + rng.integers(0, 900, B)
    cu = int(rng.integers(0, 5)) + np.concatenate([[0], np.cumsum(n)])
    parent = [-2] * int(cu[0])
    for k in n:
        parent += [int(rng.integers(-2, i)) for i in range(int(k))]
    p = ot.plan_tree(lens, cu, parent, hq, hkv, 2000, int(cu[-1]), int(rng.integers(1, 160)))
    units = [(r, t, u) for r, t, a, b in p["items"] for u in range(a, b)]
    nodes = 256 // (hq // hkv)
    want = [(r, t, u) for r in range(B) for t in range(-(-int(n[r]) // nodes)) for u in range(-(-int(lens[r]) // 128))]
    assert units == want and p["base"][-1] == len(want)
    first = p["slot_first"]
    assert first[0] == 0 and first[-1] == len(p["items"]) and len(first) == p["slots"] + 1
    for a, b in zip(first, first[1:]):
        assert a <= b and sum(i[3] - i[2] for i in p["items"][a:b]) <= p["per"]
    pieces = [i[:2] for i in p["items"]]
    assert p["cut"] == [x for x in dict.fromkeys(pieces) if pieces.count(x) > 1]
    for r in range(B):
        see = ot.visibility(parent[cu[r]:cu[r + 1]])
        got = (p["bits"][cu[r]:cu[r + 1], :, None] >> np.arange(32)) & 1
        assert np.array_equal(got.reshape(int(n[r]), 256)[:, :int(n[r])], see) and got.sum() == see.sum()


def bisect_unit(f):
    """Largest-but-eps u in [0, 1] with f(u) true, for an f that is true below a threshold."""
    lo, hi = 0.0, 1.0
    if not f(0.0):
        return 0.0
    if f(1.0 - 2.0 ** -53):
        return 1.0
    for _ in range(52):
        mid = 0.5 * (lo + hi)
        lo, hi = (mid, hi) if f(mid) else (lo, mid)
    return hi


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("siblings", [1, 2, 3])
def test_verification_enumerated(drafts, siblings):
    """P(first token = x) = target(x), by enumeration: all drafted tokens with their probabilities under q, and the
    random numbers integrated by finding the oracle's own thresholds.  Probabilities are multiples of 1/16."""
    V = 3
    p, q = np.array([8, 3, 5]) / 16, np.array([3, 9, 4]) / 16
    rows = siblings + 1
    target, draft = (np.tile(x.astype(np.float32), (rows, 1)) for x in (p, q))
    cu, parent = [0, rows], [-1] + [0] * siblings

    def walk(tokens, u_accept, u_final):
        n, path, nxt = ot.verify(cu, parent, [0, *tokens], target, draft if drafts else None, np.array([0.0, *u_accept]),
                                 np.array([u_final]), rows)
        return (int(path[0, 1]) if n[0] else 0), int(nxt[0])

    first = np.zeros(V)
    cases = list(np.ndindex(*(V,) * siblings)) if drafts else [(2, 1, 0)[:siblings]]
    for tokens in cases:
        weight = np.prod(q[list(tokens)]) if drafts else 1.0
        refused = []                                               # u = 1 is never below a ratio of at most 1
        for c in range(siblings):
            t = bisect_unit(lambda u: walk(tokens, refused + [u] + [1.0] * (siblings - c - 1), 0.0)[0] == c + 1)
            first[tokens[c]] += weight * t
            weight *= 1.0 - t
            # a ratio above 1 accepts whatever u is: nothing is left then
            refused.append(1.0)
            if weight == 0.0:
                break
        if weight > 0.0:
            edges = [0.0]
            for x in range(V - 1):
                edges.append(bisect_unit(lambda u: walk(tokens, refused, u)[1] <= x))
            first += weight * np.diff(edges + [1.0])
    assert np.allclose(first, p, atol=1e-12), (first, p)


def test_accepted_tokens_lead_to_the_next_row():
    """Two levels: after an accepted child the next token comes from that child's row."""
    target = np.array([[0.5, 0.5, 0], [0, 0.25, 0.75], [1, 0, 0]], dtype=np.float32)
    draft = np.tile(np.array([0.5, 0.25, 0.25], dtype=np.float32), (3, 1))
    n, path, nxt = ot.verify([0, 3], [-1, 0, 1], [9, 1, 2], target, draft, np.array([0, 0.999, 0.999]), [0.5], 3)
    # child 1 (token 1): 0.999 * 0.25 < 0.5; child 2 (token 2): 0.999 * 0.25 < 0.75; then row 2: token 0
    assert n[0] == 2 and path[0].tolist() == [0, 1, 2] and nxt[0] == 0
