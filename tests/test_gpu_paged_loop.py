"""The paged step as a server uses it, against the oracle running the same loop:
prompts of different lengths appended, steps of heads, tree, append in two
layers, attention, acceptance, commit and trim, a sequence forked into an idle
row, a request leaving, and the last step captured in a CUDA graph.

The oracle follows the GPU's written keys bit for bit (each checked against the
fp64 rotation first), so that attention is compared on the same cache.
"""
import numpy as np
import pytest

import medusa_draft_heads_b200 as md
from medusa_draft_heads_b200.step import PagedMedusaStep
from oracle import accept as oacc
from oracle import heads as oh
from oracle import paged as op
from oracle import tree as ot
from oracle.heads import bf16_to_f64
from seeded_inputs import gen, synth
from seeded_inputs.workloads import TREE_ACCEPT

from .helpers import bf16_tensor, f32, i32, to_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_paged_decode_loop_matches_oracle():
    B, d, V, K, kph, n = 4, 256, 2048, 4, (4, 3, 2, 2), 16
    Hq, Hkv, dh, page, width, pool, layers = 4, 2, 64, 16, 8, 24, 2
    T = n + 1
    parent, rank, _ = ot.spec_from_tuples(ot.select_tree(kph, TREE_ACCEPT, n))
    step = PagedMedusaStep(B=B, M=B, d=d, V=V, K=K, k_per_head=kph, tree_tuples=md.select_tree(kph, TREE_ACCEPT, n), Hq=Hq,
                           Hkv=Hkv, dh=dh, page_size=page, max_pages=width, pool_pages=pool, out_dtype=torch.bfloat16)
    W1, b1, Wv = (gen.normal_bf16(0, s, sh, 0.02) for s, sh in (("W1", (K, d, d)), ("b1", (K, d)), ("Wv", (K, d, V))))
    gW = [bf16_tensor(x) for x in (W1, b1, Wv)]
    qn, kn = gen.normal_bf16(0, "q", (dh,), 1.0), gen.normal_bf16(1, "q", (dh,), 1.0)
    freq = (10000.0 ** (-np.arange(dh // 2) / (dh // 2))).astype(np.float32)
    k = np.full((layers, pool, Hkv, page, dh), 0x7FC0, dtype=np.uint16)       # the pools start as NaN
    v = k.copy()
    gk, gv = bf16_tensor(k), bf16_tensor(v)
    table, cnt, ref = np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.zeros(pool, np.int32)

    def pages_equal():
        for got, want in ((step.block_table, table), (step.n_pages, cnt), (step.refcount, ref)):
            assert np.array_equal(got.cpu().numpy(), want)

    def append(seed, width_t, pos, prefix, n_new, q_out=None):
        """Both layers' new tokens on the GPU; the oracle's pools take the checked bits."""
        outs = []
        for layer in range(layers):
            qkv = gen.normal_bf16(seed + layer, "q", (B, width_t, Hq + 2 * Hkv, dh), 1.0)
            gq, gkk, gvv = bf16_tensor(qkv).split([Hq, Hkv, Hkv], dim=2)
            out = torch.zeros((B, width_t, Hq, dh), dtype=torch.bfloat16, device="cuda")
            step.append(gq, gkk, gvv, i32(pos), torch.from_numpy(freq).cuda(), gk[layer], gv[layer], i32(prefix),
                        q_norm=bf16_tensor(qn), k_norm=bf16_tensor(kn), n_new=None if n_new is None else i32(n_new), q_out=out)
            _, written = op.qk_rope_append(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:], pos, freq, table, prefix,
                                           k[layer].shape, qn, kn, 1e-6, False, n_new)
            bits = to_bits(gk[layer])
            for (pg, row), (kr, vr) in written.items():
                got = bf16_to_f64(bits[pg, :, row])
                assert (np.abs(got - kr) <= 2.0 ** -8 * np.abs(kr) + 2.0 ** -20 * np.abs(kr).max()).all()
                k[layer, pg, :, row], v[layer, pg, :, row] = bits[pg, :, row], vr
            assert np.array_equal(bits, k[layer]) and np.array_equal(to_bits(gv[layer]), v[layer])
            outs.append(out)
        return outs

    # ---- prompts: 37, 16 and 5 tokens; row 3 is idle ----
    lens = np.array([37, 16, 5, -1], dtype=np.int32)
    step.prefill_pages(i32(lens))
    table, cnt, ref, _ = op.pages_resize(table, cnt, ref, lens, page)
    pages_equal()
    start = np.where(lens < 0, -1, 0).astype(np.int32)
    append(50, 40, np.tile(np.arange(40), (B, 1)), start, np.maximum(lens, 0))
    P = lens.copy()
    root = synth.root_tokens(0, B, V)
    for s in range(3):
        seed = 100 + 10 * s
        if s == 1:                                        # row 0 goes on twice; row 2 leaves
            P[2] = -1
            gP = i32(P)
            step.prefill_pages(gP)
            table, cnt, ref, _ = op.pages_resize(table, cnt, ref, P, page)
            step.fork(gk, gv, i32([0, -1]), i32([3, 0]), gP)
            k, v, table, cnt, ref, P = op.pages_fork(k, v, table, cnt, ref, np.array([0, -1]), np.array([3, 0]), P)
            root[3] = root[0]
            assert gP.cpu().tolist() == P.tolist()
            assert np.array_equal(to_bits(gk), k) and np.array_equal(to_bits(gv), v)
            pages_equal()
        gP, groot = i32(P), i32(root)
        h = gen.normal_bf16(seed, "h", (B, d), 1.0)
        rid, _, _, _ = oh.medusa_heads(h, W1, b1, Wv, kph)
        live = [b for b in range(B) if P[b] >= 0]
        rtok, _, _, rpos = ot.tree_build(parent, rank, rid, root, P)
        step.heads(bf16_tensor(h), *gW)
        step.build(groot, gP)
        assert np.array_equal(step.tokens.cpu().numpy()[live], rtok[live])
        assert np.array_equal(step.pos.cpu().numpy()[live], rpos[live])
        step.reserve(gP)
        table, cnt, ref, short = op.pages_resize(table, cnt, ref, P, page, T)
        assert not short
        pages_equal()
        qs = append(seed, T, rpos, P, None)
        for layer in range(layers):
            step.attention(qs[layer], gk[layer], gv[layer], gP)
            q = to_bits(qs[layer])
            want = op.tree_attention_paged(q, k[layer], v[layer], table, P, parent)
            absv = op.tree_attention_paged(q, k[layer], v[layer] & 0x7FFF, table, P, parent)
            got = step.attn_out.float().cpu().numpy()
            assert (np.abs(got - want) <= 2 * (2.0 ** -13 + 2.0 ** -8) * absv + 2.0 ** -8 * np.abs(want)).all()
        logits = synth.planted_logits(seed, parent, rtok, V, TREE_ACCEPT)
        L, path, bonus, _ = oacc.greedy_accept(logits, rtok, parent, K)
        glog = f32(logits)
        if s < 2:
            step.accept(glog)
            step.commit(gk, gv, gP)
            step.trim()
        else:                                             # the tail of the step from a graph
            state = gk.view(torch.int16), gv.view(torch.int16), step.block_table, step.n_pages, step.refcount
            before = [x.clone() for x in state]
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step.accept(glog)
                step.commit(gk, gv, gP)
                step.trim()
            assert all(torch.equal(a, b) for a, b in zip(before, state))     # nothing ran yet
            g.replay()
        k, v, P2, root2, _ = op.tree_commit_paged(k, v, table, P, L, path, bonus, T)
        assert np.array_equal(to_bits(gk), k) and np.array_equal(to_bits(gv), v)
        assert step.new_prefix_len.cpu().tolist() == P2.tolist() and step.next_root.cpu().tolist() == root2.tolist()
        table, cnt, ref, _ = op.pages_resize(table, cnt, ref, P2, page)
        pages_equal()
        assert md.device_status() == 0
        P, root = P2.astype(np.int32), np.maximum(root2, 0).astype(np.int32)
    # the fork's sequences went on in pages of their own, sharing the first
    assert ref.max() == 2 and table[0, 0] == table[3, 0] and table[0, 2] != table[3, 2]


def test_a_captured_fork_replays_after_larger_ones():
    """A fork of one row captured, then eager forks of many rows and other allocations, then the graph again."""
    B, Hkv, dh, page, width, pool = 48, 2, 64, 16, 4, 200
    kph = (4, 3, 2, 2)
    step = PagedMedusaStep(B=B, M=B, d=256, V=2048, K=4, k_per_head=kph, tree_tuples=md.select_tree(kph, TREE_ACCEPT, 16), Hq=4,
                           Hkv=Hkv, dh=dh, page_size=page, max_pages=width, pool_pages=pool, out_dtype=torch.bfloat16)
    k = gen.normal_bf16(1, "k_cache", (2, pool, Hkv, page, dh), 1.0)
    v = gen.normal_bf16(1, "v_cache", (2, pool, Hkv, page, dh), 1.0)
    gk, gv = bf16_tensor(k), bf16_tensor(v)
    length = np.full(B, -1, dtype=np.int32)
    length[:20] = 17 + np.arange(20)
    table, cnt, ref = np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.zeros(pool, np.int32)
    glen, one = i32(length), (i32([3]), i32([47]))
    step.prefill_pages(glen)
    table, cnt, ref, _ = op.pages_resize(table, cnt, ref, length, page)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.fork(gk, gv, *one, glen)
    many = np.arange(20), np.arange(20) + 20
    step.fork(gk, gv, i32(many[0]), i32(many[1]), glen)
    k, v, table, cnt, ref, length = op.pages_fork(k, v, table, cnt, ref, *many, length)
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (256, 512, 1024, 16384) for _ in range(8)]
    g.replay()
    k, v, table, cnt, ref, length = op.pages_fork(k, v, table, cnt, ref, np.array([3]), np.array([47]), length)
    assert md.device_status() == 0
    assert np.array_equal(to_bits(gk), k) and np.array_equal(to_bits(gv), v)
    for got, want in ((step.block_table, table), (step.n_pages, cnt), (step.refcount, ref), (glen, length)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert all(bool((x == 0x7F).all()) for x in junk)


@pytest.mark.parametrize("mode", ["greedy", "typical", "sample", "rejection"])
def test_padded_batch_feeds_its_own_outputs_back(mode):
    """Rows that hold no request beside rows that do: root, prefix and head row of each step
    are the commit's of the step before, untouched by the host, and no status bit is ever set.
    The target's logits of the idle rows are NaN."""
    B, d, V, K, kph, n = 4, 256, 2048, 4, (4, 3, 2, 2), 16
    Hq, Hkv, dh, page, width, pool = 4, 2, 64, 16, 8, 24
    T = n + 1
    parent, rank, depth = ot.spec_from_tuples(ot.select_tree(kph, TREE_ACCEPT, n))
    step = PagedMedusaStep(B=B, M=B * T, d=d, V=V, K=K, k_per_head=kph, tree_tuples=md.select_tree(kph, TREE_ACCEPT, n),
                           Hq=Hq, Hkv=Hkv, dh=dh, page_size=page, max_pages=width, pool_pages=pool, mode=mode)
    gW = [bf16_tensor(gen.normal_bf16(0, s, sh, 0.02)) for s, sh in (("W1", (K, d, d)), ("b1", (K, d)), ("Wv", (K, d, V)))]
    freq = torch.ones(dh // 2, device="cuda")
    gk = torch.full((1, pool, Hkv, page, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    gv = gk.clone()
    P = np.array([20, -1, 5, -1], dtype=np.int32)
    gP, root, head_row = i32(P), i32([3, -1, 1000, -1]), i32([0, -1, 2 * T, -1])
    rng = np.random.default_rng(1)
    md.device_status(clear=True)
    step.prefill_pages(gP)
    gk[:, step.block_table[[0, 2]][step.block_table[[0, 2]] >= 0].long()] = 0
    gv.copy_(gk)
    hosts = root.cpu().numpy(), head_row.cpu().numpy()
    for s in range(4):
        if s == 2:                                        # row 2's request ends
            P[2] = -1
            gP.copy_(i32(P))
            step.prefill_pages(gP)
        live = [b for b in range(B) if P[b] >= 0]
        h = gen.normal_bf16(10 + s, "h", (B * T, d), 1.0)
        if mode == "rejection":
            step.u_draft.copy_(torch.rand(step.u_draft.shape, generator=torch.Generator().manual_seed(s)))
        step.heads(bf16_tensor(h), *gW)
        step.build(root, gP, head_row=head_row)
        rtok, _, _, rpos = ot.tree_build(parent, rank, step.topk_ids.cpu().numpy(), hosts[0], P, head_row=hosts[1])
        assert np.array_equal(step.tokens.cpu().numpy(), rtok) and np.array_equal(step.pos.cpu().numpy(), rpos)
        assert (rtok >= 0).all() and (rtok < V).all() and (rpos >= 0).all()
        step.reserve(gP)
        qkv = bf16_tensor(gen.normal_bf16(s, "q", (B, T, Hq + 2 * Hkv, dh), 1.0))
        step.append(*qkv.split([Hq, Hkv, Hkv], dim=2), step.pos, freq, gk[0], gv[0], gP)
        step.attention(step.q, gk[0], gv[0], gP)
        idle = [b for b in range(B) if P[b] < 0]
        assert not step.attn_out[idle].any() and torch.isfinite(step.attn_out).all()
        logits = synth.planted_logits(20 + s, parent, rtok, V, TREE_ACCEPT)
        logits[idle] = np.nan
        step.accept(f32(logits))
        step.commit(gk, gv, gP)
        step.trim()
        L, new = step.accept_len.cpu().numpy(), step.new_prefix_len.cpu().numpy()
        assert md.device_status() == 0
        assert (new[live] == P[live] + L[live] + 1).all() and (new[idle] == -1).all()
        assert step.n_pages.cpu().tolist() == [max(0, -(-int(p) // page)) for p in new]
        gP.copy_(step.new_prefix_len)
        root, head_row, P = step.next_root, step.next_head_row, new.copy()
        hosts = root.cpu().numpy(), head_row.cpu().numpy()
        assert (hosts[0][idle] == -1).all() and (hosts[1][idle] == -1).all() and (hosts[1][live] >= 0).all()
