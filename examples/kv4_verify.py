"""Speculative verify rounds with the attention half of the step on the 4-bit KV cache.

One layer of a small model, several sequences.  Each round
  1. selects draft nodes of every sequence's tree (the control path of the MoE verify step),
  2. writes the keys and values of the verify tokens (root and selected nodes) behind the context,
  3. attends: a token sees the context, its ancestors in the tree and itself,
  4. adds the attention weights to every slot's account,
  5. accepts a path (here: drawn at random) and commits it: the accepted tokens are written again, side by side
     (the others need no rollback: no later call looks beyond the length it is given),
  6. where a sequence has outgrown its budget, evicts the slots of least weight.

Run from the repository's root: python examples/kv4_verify.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import serving_router_softmax_gb300 as mv  # noqa: E402
from workload import gen  # noqa: E402


def tree_masks(ancestors: torch.Tensor, selected: torch.Tensor, gamma) -> torch.Tensor:
    """Visibility masks of the verify tokens, sequence after sequence: token 0 is the root, token 1 + i the i-th selected
    node; each sees the root, its selected ancestors and itself.  ``ancestors`` [N, N]: entry (a, b) is true where b is a
    or above it."""
    rows = []
    for s, g in enumerate(gamma):
        sel = selected[s, :g].long()
        sees = ancestors[sel][:, sel].long()
        bits = (sees << torch.arange(1, g + 1, device=sel.device)).sum(1) | 1
        rows.append(torch.cat([torch.ones(1, dtype=torch.int64, device=sel.device), bits]))
    return torch.cat(rows)


def plain_attention(cache, q, q_start, base, visible, scale):
    """The same attention in fp32 torch operations over the values that the cache holds."""
    out = torch.empty_like(q, dtype=torch.float32)
    G = q.shape[1] // cache.n_kv_heads
    for s in range(cache.n_seq):
        a, b, n = q_start[s], q_start[s + 1], base[s] + q_start[s + 1] - q_start[s]
        where = torch.arange(n, dtype=torch.int32, device=q.device)
        k, v = mv.kv4_read(cache, torch.full_like(where, s), where, torch.float32)
        sees = torch.ones((b - a, n), dtype=torch.bool, device=q.device)
        sees[:, base[s]:] = (visible[a:b, None] >> torch.arange(b - a, device=q.device)) & 1 > 0
        x = torch.einsum("thd,jhd->thj", q[a:b].float(), k.repeat_interleave(G, 1)) * scale
        p = torch.softmax(x.masked_fill(~sees[:, None], float("-inf")), 2)
        out[a:b] = torch.einsum("thj,jhd->thd", p, v.repeat_interleave(G, 1))
    return out


def main(rounds: int = 40, context: int = 180, budget: int = 256, recent: int = 32, seed: int = 0, say=print) -> dict:
    dev = torch.device("cuda")
    cfg = gen.small_case("kv4_example", L=1, E=16, k=4, nseq=3, gamma=4, seed=seed)
    wl = gen.make_workload(cfg)
    Hq, Hkv, D, page = 16, 2, 128, 32
    gamma = wl.gamma.tolist()
    spec = mv.StepSpec(L=1, nseq=cfg.nseq, N=len(wl.parent), W=cfg.W, E=cfg.E, k=cfg.k, H=cfg.H, I=cfg.I, dtype=cfg.dtype,
                       T=wl.T, gamma_max=max(gamma))
    plan = mv.VerifyPlan(spec, dev)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
    tree = [t(wl.P), t(np.tile(wl.parent, (cfg.nseq, 1))), t(wl.own_fp.view(np.int32)), t(wl.gamma), t(wl.logits)]
    N = len(wl.parent)
    ancestors = torch.eye(N, dtype=torch.bool)
    for x in range(N):
        if wl.parent[x] >= 0:
            ancestors[x] |= ancestors[wl.parent[x]]
    ancestors = ancestors.to(dev)

    # A cache of a context, the budget's growth between evictions and one round's tokens.
    pages_each = -(-(max(budget, context) + 3 * max(gamma) + 8) // page)
    cache = mv.Kv4Cache.new(cfg.nseq * pages_each, Hkv, page, D, cfg.nseq, pages_each, dev)
    cache.table.copy_(torch.randperm(cfg.nseq * pages_each, device=dev).view(cfg.nseq, pages_each))
    mass = cache.new_mass()
    g = torch.Generator(device=dev).manual_seed(seed)
    r = np.random.default_rng(seed)
    err = mv.new_dev_err()
    scale = D ** -0.5
    rows = lambda n: torch.randn((n, Hq + 2 * Hkv, D), generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    base = [context] * cfg.nseq
    seq = t(np.repeat(np.arange(cfg.nseq), base).astype(np.int32))
    slot = t(np.concatenate([np.arange(b) for b in base]).astype(np.int32))
    kv = rows(len(seq))
    mv.kv4_append(cache, kv[:, Hq:Hq + Hkv], kv[:, Hq + Hkv:], seq, slot, dev_err=err)
    fresh = [n + 1 for n in gamma]
    q_start = np.concatenate([[0], np.cumsum(fresh)]).astype(np.int32)
    seq = t(np.repeat(np.arange(cfg.nseq), fresh).astype(np.int32))
    worst, evictions, committed = 0.0, 0, 0
    for step in range(rounds):
        plan(*tree)
        visible = tree_masks(ancestors, plan.selected, gamma)
        qkv = rows(int(q_start[-1]))
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        base_d = t(np.asarray(base, np.int32))
        slot = t(np.concatenate([b + np.arange(n) for b, n in zip(base, fresh)]).astype(np.int32))
        mv.kv4_append(cache, k, v, seq, slot, dev_err=err)
        out, lse = mv.kv4_attend(cache, q, t(q_start), base_d, max(fresh), visible=visible, scale=scale, dev_err=err)
        mv.kv4_weigh(cache, q, t(q_start), base_d, max(fresh), lse, mass, visible=visible, scale=scale, dev_err=err)
        if step % 10 == 0:
            want = plain_attention(cache, q, q_start, base, visible, scale)
            worst = max(worst, float((out.float() - want).norm() / want.norm()))
        # Accept: from the root down to a token drawn at random; its ancestors are the set bits of its mask.
        seen = visible.cpu().numpy()
        slots = np.full(int(q_start[-1]), -1, np.int32)
        kept = []
        for s in range(cfg.nseq):
            last = q_start[s] + int(r.integers(0, fresh[s]))
            path = [q_start[s] + i for i in range(fresh[s]) if (int(seen[last]) >> i) & 1]
            slots[path] = base[s] + np.arange(len(path))
            kept.append(len(path))
        committed += sum(kept)
        # The path's weights move with it; the rejected tokens' are dropped.
        for s in range(cfg.nseq):
            new = mass[s, :, base[s]:base[s] + fresh[s]].clone()
            mass[s, :, base[s]:base[s] + fresh[s]] = 0
            at = [i for i in range(fresh[s]) if slots[q_start[s] + i] >= 0]
            mass[s, :, base[s]:base[s] + len(at)] = new[:, at]
        mv.kv4_append(cache, k, v, seq, t(slots), dev_err=err)
        base = [b + n for b, n in zip(base, kept)]
        if max(base) > budget:
            new_len, _, _ = mv.kv4_evict(cache, mass, t(np.asarray(base, np.int32)), budget - 2 * max(fresh), recent, dev_err=err)
            base = new_len.tolist()
            evictions += 1
    torch.cuda.synchronize()
    assert err.item() == 0, f"device error bits {err.item()}"
    say(f"{rounds} rounds, {committed} tokens committed, {evictions} evictions, lengths {base}, attention within {worst:.1e} of fp32")
    return {"worst": worst, "evictions": evictions, "committed": committed, "lengths": base, "mass": mass}


if __name__ == "__main__":
    main()
