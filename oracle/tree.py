"""fp64 reference of the speculative-decoding steps (test infrastructure only).

A request r brings n_r tree nodes behind its cached prefix of p_r = L_r - n_r keys; ``parent``
holds each node's parent inside its request (-1 a root, -2 a node that is not in use).  Not on the
source pages; the definitions are those of include/pagedattn.h:

* attention: node i sees the prefix, itself and its ancestors; a node that is not in use, or
  below one that is not, gives O = 0, lse = -inf;
* verification: the walk from node 0 with residual weights w <- max(w - Z q, 0), Z <- sum w;
* compaction: the accepted rows move to the positions behind the prefix.

All arithmetic is float64 and written node by node, one request at a time.
"""
from __future__ import annotations

import numpy as np

from .attention import gather_slots, softmax_attend
from .codecs import bf16_bits_to_f64, e4m3_to_f64


def visibility(parent) -> np.ndarray:
    """bool [n, n]: node j is node i or one of its ancestors; the row of an unused node is empty."""
    n = len(parent)
    see = np.zeros((n, n), dtype=bool)
    for i in range(n):
        p = int(parent[i])
        if p == -1 or (0 <= p < i and see[p, p]):
            if p >= 0:
                see[i] = see[p]
            see[i, i] = True
    return see


def tree_attention(q_bits, cu_seqlens_q, parent, k_pool, v_pool, page_table, seq_lens, page_size, sm_scale,
                   k_scale=None, v_scale=None):
    """O, lse and A = sum_j p_j |V_j| (the scale of the rounding of p) of every node and query head.

    Pools: uint16 bf16 patterns, or uint8 E4M3 codes with k_scale and v_scale given.
    """
    T, hq, D = q_bits.shape
    hkv = k_pool.shape[1]
    G = hq // hkv
    q = bf16_bits_to_f64(q_bits)
    out, mag = np.zeros((T, hq, D)), np.zeros((T, hq, D))
    lse = np.full((T, hq), -np.inf)
    for r in range(len(seq_lens)):
        q0, q1, L = int(cu_seqlens_q[r]), int(cu_seqlens_q[r + 1]), int(seq_lens[r])
        n = q1 - q0
        if n == 0:
            continue
        see = visibility(parent[q0:q1])
        vis = np.concatenate([np.repeat(see.any(1)[:, None], L - n, 1), see], 1)
        slots = gather_slots(page_table, L, page_size, r)
        seen = vis.any(0)
        for h in range(hkv):
            if k_scale is None:
                k, v = bf16_bits_to_f64(k_pool[slots, h]), bf16_bits_to_f64(v_pool[slots, h])
            else:
                k, v = k_scale * e4m3_to_f64(k_pool[slots, h]), v_scale * e4m3_to_f64(v_pool[slots, h])
            k, v = np.where(seen[:, None], k, 0.0), np.where(seen[:, None], v, 0.0)
            for g in range(G):
                qh = q[q0:q1, h * G + g]
                out[q0:q1, h * G + g], lse[q0:q1, h * G + g] = softmax_attend(qh, k, v, sm_scale, vis)
                mag[q0:q1, h * G + g], _ = softmax_attend(qh, k, np.abs(v), sm_scale, vis)
    return out, lse, mag


def verify(cu_seqlens_q, parent, tokens, target, draft, u_accept, u_final, path_pitch):
    """(accept_len [B], path [B, path_pitch], next_token [B]) of the walks."""
    B = len(cu_seqlens_q) - 1
    accept_len = np.zeros(B, dtype=np.int32)
    path = np.full((B, path_pitch), -1, dtype=np.int32)
    nxt = np.full(B, -1, dtype=np.int32)
    for r in range(B):
        q0, n = int(cu_seqlens_q[r]), int(cu_seqlens_q[r + 1] - cu_seqlens_q[r])
        if n == 0 or parent[q0] != -1:
            continue
        used = visibility(parent[q0:q0 + n]).any(1)
        walk = [0]
        while True:
            row = q0 + walk[-1]
            w, z, found = np.maximum(np.nan_to_num(target[row].astype(np.float64), nan=0.0), 0.0), 1.0, None
            for c in range(walk[-1] + 1, n):
                if not used[c] or parent[q0 + c] != walk[-1] or len(walk) >= path_pitch:
                    continue
                x = int(tokens[q0 + c])
                if not 0 <= x < target.shape[1]:
                    continue
                q = draft[row].astype(np.float64) if draft is not None else (np.arange(target.shape[1]) == x) * 1.0
                if float(u_accept[q0 + c]) * q[x] * z < w[x]:
                    found = c
                    break
                if draft is not None:
                    w = np.maximum(w - z * q, 0.0)
                    z = float(w.sum())
                else:
                    z = max(z - w[x], 0.0)
                    w = w.copy()
                    w[x] = 0.0
            if found is None:
                break
            walk.append(found)
        if not w.sum() > 0:
            w = np.maximum(np.nan_to_num(target[row].astype(np.float64), nan=0.0), 0.0)
        path[r, :len(walk)] = walk
        accept_len[r] = len(walk) - 1
        if w.sum() > 0:
            over = np.flatnonzero(np.cumsum(w) > float(u_final[r]) * w.sum())
            nxt[r] = over[0] if len(over) else np.flatnonzero(w > 0)[-1]
    return accept_len, path, nxt


def kv_compact(pools, cu_seqlens_q, seq_lens, accept_len, path, page_table, page_size):
    """(new pools, new lengths); the pools are arrays [slots, ...], left as they were."""
    pools = [p.copy() for p in pools]
    lens = np.array(seq_lens, dtype=np.int32).copy()
    for r in range(len(lens)):
        n = int(cu_seqlens_q[r + 1] - cu_seqlens_q[r])
        if n == 0:
            continue
        prefix = int(lens[r]) - n
        if path[r, 0] < 0:
            lens[r] = prefix
            continue
        slots = gather_slots(page_table, int(lens[r]), page_size, r)
        k = np.arange(1, int(accept_len[r]) + 1)
        for p in pools:
            p[slots[prefix + k]] = p[slots[prefix + path[r, k]]]
        lens[r] = prefix + 1 + int(accept_len[r])
    return pools, lens


def plan_tree(seq_lens, cu_seqlens_q, parent, hq, hkv, max_kv_len, max_q_tokens, num_sms):
    """The plan's arrays as attn_plan_tree documents them, for requests in range; a request out of range
    (more keys than max_kv_len, more nodes than keys or than 256, rows outside max_q_tokens) has no work.

    Returns a dict: tiles, base (units before each request, then all), prefix, items (r, tile, first key tile,
    end key tile), slot_first, cut (query tiles cut into pieces), per, slots, bits (one row of 8 words a node).
    """
    B, nodes = len(seq_lens), 256 // (hq // hkv)
    slots = max(1, num_sms // hkv)
    cu = [int(x) for x in cu_seqlens_q]
    tiles, ktiles, prefix = [], [], []
    bits = np.zeros((max_q_tokens, 8), dtype=np.uint32)
    for r in range(B):
        L, n = int(seq_lens[r]), cu[r + 1] - cu[r]
        if not (0 <= L <= max_kv_len and 0 <= cu[r] and cu[r + 1] <= max_q_tokens and 0 <= n <= min(L, 256)):
            n = 0
        tiles.append((n + nodes - 1) // nodes)
        ktiles.append((L + 127) // 128 if n else 0)
        prefix.append(L - n)
        see = visibility(parent[cu[r]:cu[r] + n])
        for i in range(n):
            for j in np.flatnonzero(see[i]):
                bits[cu[r] + i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    base = [0]
    for r in range(B):
        base.append(base[-1] + tiles[r] * ktiles[r])
    per = max(1, -(-base[-1] // slots))
    items, item_slot, cut = [], [], []
    for r in range(B):
        for t in range(tiles[r]):
            u0 = base[r] + t * ktiles[r]
            owners = sorted({u // per for u in range(u0, u0 + ktiles[r])})
            if len(owners) > 1:
                cut.append((r, t))
            for c in owners:
                mine = [u for u in range(u0, u0 + ktiles[r]) if u // per == c]
                items.append((r, t, mine[0] - u0, mine[-1] + 1 - u0))
                item_slot.append(c)
    slot_first = [sum(s < c for s in item_slot) for c in range(slots + 1)]
    return dict(tiles=tiles, base=base, prefix=prefix, items=items, slot_first=slot_first, cut=cut, per=per, slots=slots,
                bits=bits)
