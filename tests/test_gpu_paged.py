"""GPU parity of the paged-cache calls against the oracle (fp64, integers).

Tolerances. A weight's relative error: the score's fp32 sum of dh products
(at most dh * 2^-24 * scale * sum|q k|, under 2^-13 for these inputs) and, for bf16
results, its rounding, half a step = 2^-8 (fp32 results keep all 24 bits). Numerator
and denominator together move a result by at most twice that times
A = sum_j w_j |v_j|; a bf16 result is rounded once more.
The rotation is fp32 with one rounding: 2^-8 of the value, and 2^-20 of the
row's largest for the fp32 steps before it.
"""
import numpy as np
import pytest

import medusa_draft_heads_b200 as md
from oracle import paged as op
from oracle import tree as ot
from oracle.heads import bf16_to_f64
from seeded_inputs import gen
from seeded_inputs.workloads import TREE_ACCEPT

from .helpers import bf16_tensor, i32, to_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN = 0x7FC0


def _tree(n, kph=(10, 10, 10, 10)):
    if n == 0:
        return [-1], [0]
    parent, rank, _ = ot.spec_from_tuples(ot.select_tree(kph, TREE_ACCEPT, n))
    return list(parent), list(rank)


def _table(rng, P, T, page, spare=3, width=None):
    counts = [0 if p < 0 else -(-(p + T) // page) for p in P]
    pool = sum(counts) + spare
    width = width or max(max(counts), 1)
    ids = rng.permutation(pool)
    table, at = np.full((len(P), width), -1, dtype=np.int32), 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pool


def _attention(q, kp, vp, table, P, parent, rank, out_dtype, scale=0.0, ws=None, stream=None, out=None):
    B, T, Hq, dh = q.shape
    tree = md.Tree(parent, rank, [16] * 8)
    out = torch.full((B, T, Hq, dh), 7.0, dtype=out_dtype, device="cuda") if out is None else out
    if ws is None:
        ws = md.workspace(md.attention_paged_workspace_bytes(B, T, Hq, kp.shape[1], dh, kp.shape[2], table.shape[1]))
        ws.fill_(0xA5)
    md.tree_attention_paged(q, kp, vp, table, P, tree, out, ws, scale=scale, stream=stream)
    return out


def _check_attention(out, q, kp, vp, table, P, parent, scale=None):
    ref = op.tree_attention_paged(q, kp, vp, table, P, parent, scale)
    absv = op.tree_attention_paged(q, kp, vp & 0x7FFF, table, P, parent, scale)      # A = sum w |v|
    got = out.float().cpu().numpy().astype(np.float64)
    tol = 2 * 2.0 ** -13 * absv
    if out.dtype == torch.bfloat16:
        tol = 2 * (2.0 ** -13 + 2.0 ** -8) * absv + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3], tol[bad][:3])


CASES = [
    # nodes, Hq, Hkv, dh, page, prefixes
    ("decode-empty", 0, 4, 2, 64, 16, [0]),
    ("decode-ragged", 0, 32, 8, 128, 16, [0, 1, 127, 128, 129, 1000]),
    ("decode-long-many-splits", 0, 8, 1, 128, 64, [6001]),
    ("pair", 1, 8, 2, 64, 32, [5, 254, 255]),
    ("tiny", 16, 4, 2, 64, 16, [128]),
    ("mha", 16, 4, 4, 128, 32, [0, 200]),
    ("g3-page48", 16, 6, 2, 128, 48, [77, 300]),
    ("g7", 20, 28, 4, 128, 64, [0, 37, 511]),
    ("g12-page256", 64, 12, 1, 64, 256, [1000]),
    ("g16-many-tiles", 64, 16, 1, 64, 128, [700, 65]),
    ("second-tile-of-one-node", 16, 16, 2, 128, 16, [400, 90]),
    ("70b", 64, 64, 8, 128, 64, [601]),
    ("full-tree", 127, 8, 4, 128, 16, [3, 250]),
    ("chunk-edges", 64, 8, 2, 128, 32, [63, 64, 127, 128, 191]),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("name,nodes,Hq,Hkv,dh,page,P", CASES, ids=[c[0] for c in CASES])
def test_attention_matches_oracle(name, nodes, Hq, Hkv, dh, page, P, dtype):
    rng = np.random.default_rng(nodes + Hq + page)
    parent, rank = _tree(nodes)
    T, B = len(parent), len(P)
    table, pool = _table(rng, P, T, page)
    q = gen.normal_bf16(3, "q", (B, T, Hq, dh), 1.0)
    kp = gen.normal_bf16(3, "k_cache", (pool, Hkv, page, dh), 1.0)
    vp = gen.normal_bf16(3, "v_cache", (pool, Hkv, page, dh), 1.0)
    md.device_status(clear=True)
    out = _attention(bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(P), parent, rank, dtype)
    again = _attention(bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(P), parent, rank, dtype)
    assert md.device_status() == 0
    _check_attention(out, q, kp, vp, table, P, parent)
    assert torch.equal(out, again)


@pytest.mark.parametrize("nodes,Hq,Hkv,dh,page,P", [(16, 8, 2, 128, 16, [77, 0, -1, 300]), (0, 8, 2, 64, 32, [77, 0, -1, 300]),
                                                    (64, 16, 2, 64, 64, [-1, 129])])
def test_unused_slots_may_hold_nan_and_idle_rows_are_zero(nodes, Hq, Hkv, dh, page, P):
    """Every slot that no request uses holds NaN; the table is wider than any sequence."""
    rng = np.random.default_rng(9)
    parent, rank = _tree(nodes)
    T, B = len(parent), len(P)
    table, pool = _table(rng, P, T, page, width=400)
    q = gen.normal_bf16(5, "q", (B, T, Hq, dh), 1.0)
    k = gen.normal_bf16(5, "k_cache", (pool, Hkv, page, dh), 1.0)
    v = gen.normal_bf16(5, "v_cache", (pool, Hkv, page, dh), 1.0)
    kp, vp = np.full_like(k, NAN), np.full_like(v, NAN)
    for b in range(B):
        for s in range(P[b] + T if P[b] >= 0 else 0):
            at = (table[b, s // page], slice(None), s % page)
            kp[at], vp[at] = k[at], v[at]
    for dtype in (torch.float32, torch.bfloat16):
        md.device_status(clear=True)
        out = _attention(bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(P), parent, rank, dtype)
        assert md.device_status() == 0
        _check_attention(out, q, kp, vp, table, P, parent)
        assert not out[[b for b in range(B) if P[b] < 0]].any()


@pytest.mark.parametrize("Hq,P", [(4, [250, 3]), (32, [250, 3])])     # one row tile; two
def test_a_node_that_is_not_finite_reaches_only_its_descendants(Hq, P):
    rng = np.random.default_rng(2)
    parent, rank = _tree(16)
    T, Hkv, dh, page = 17, 2, 64, 16
    table, pool = _table(rng, P, T, page)
    q = gen.normal_bf16(6, "q", (2, T, Hq, dh), 1.0)
    kp = gen.normal_bf16(6, "k_cache", (pool, Hkv, page, dh), 1.0)
    vp = gen.normal_bf16(6, "v_cache", (pool, Hkv, page, dh), 1.0)
    clean_k, clean_v = kp.copy(), vp.copy()
    node = {0: 2, 1: 5}                    # request 0: K and V of node 2 are NaN; request 1: V of node 5 holds infinities
    sees = [[any(a == node[b] for a in _ancestors(parent, t)) for t in range(T)] for b in range(2)]
    s0, s1 = P[0] + node[0], P[1] + node[1]
    kp[table[0, s0 // page], :, s0 % page] = NAN
    vp[table[0, s0 // page], :, s0 % page] = NAN
    vp[table[1, s1 // page], :, s1 % page, 3] = 0x7F80
    vp[table[1, s1 // page], :, s1 % page, 4] = 0xFF80
    for dtype in (torch.float32, torch.bfloat16):
        out = _attention(bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(P), parent, rank, dtype)
        ref = _attention(bf16_tensor(q), bf16_tensor(clean_k), bf16_tensor(clean_v), i32(table), i32(P), parent, rank, dtype)
        for t in range(T):
            if sees[0][t]:
                assert torch.isnan(out[0, t]).all()
            else:
                assert torch.equal(out[0, t], ref[0, t])
            if sees[1][t]:
                assert (out[1, t, :, 3] == np.inf).all() and (out[1, t, :, 4] == -np.inf).all()
                keep = [e for e in range(dh) if e not in (3, 4)]
                assert torch.equal(out[1, t][:, keep], ref[1, t][:, keep])
            else:
                assert torch.equal(out[1, t], ref[1, t])
    assert any(sees[0]) and not all(sees[0]) and any(sees[1]) and not all(sees[1])


def _ancestors(parent, t):
    while t >= 0:
        yield t
        t = parent[t]


def test_attention_flags_bad_prefixes_and_pages():
    rng = np.random.default_rng(4)
    parent, rank = _tree(16)
    T, page, P = 17, 16, [40, 60, 5]
    table, pool = _table(rng, P, T, page, width=6)
    q = gen.normal_bf16(8, "q", (3, T, 4, 64), 1.0)
    kp = gen.normal_bf16(8, "k_cache", (pool, 2, page, 64), 1.0)
    vp = gen.normal_bf16(8, "v_cache", (pool, 2, page, 64), 1.0)
    call = lambda tb, p: _attention(bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(tb), i32(p), parent, rank,  # noqa: E731
                                    torch.float32)
    for bad in (80, -2, 2 ** 31 - 1):                 # 80 + 17 > 6 pages of 16
        md.device_status(clear=True)
        out = call(table, [40, bad, 5])
        assert md.device_status(clear=True) == md.binding.DEV_BAD_PREFIX
        assert not out[1].any()
        _check_attention(out[[0, 2]], q[[0, 2]], kp, vp, table[[0, 2]], [40, 5], parent)
    for page_id in (-1, pool, 2 ** 31 - 1, -2 ** 31):
        t2 = table.copy()
        t2[1, 1] = page_id                             # slots 16 .. 31 read as zeros
        md.device_status(clear=True)
        out = call(t2, P)
        assert md.device_status(clear=True) == md.binding.DEV_BAD_PAGE
        kz, vz = np.concatenate([kp, np.zeros_like(kp[:1])]), np.concatenate([vp, np.zeros_like(vp[:1])])
        t2[1, 1] = pool
        _check_attention(out, q, kz, vz, t2, P, parent)


def test_attention_of_a_layer_of_a_pool_past_32_bit_offsets():
    """Pools of 2^31 + elements: pages at the far end, and the last layer of a stack."""
    Hkv, page, dh = 8, 64, 128
    per = Hkv * page * dh
    pool = (1 << 31) // per + 40
    kp = torch.zeros((1, pool, Hkv, page, dh), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    P, parent, rank = [200], *_tree(16)
    T = 17
    k = gen.normal_bf16(1, "k_cache", (4, Hkv, page, dh), 1.0)
    v = gen.normal_bf16(1, "v_cache", (4, Hkv, page, dh), 1.0)
    ids = [pool - 1, pool - 7, 3, pool - 2]
    for i, p in enumerate(ids):
        kp[0, p], vp[0, p] = bf16_tensor(k[i]), bf16_tensor(v[i])
    q = gen.normal_bf16(1, "q", (1, T, 64, dh), 1.0)
    out = _attention(bf16_tensor(q), kp[0], vp[0], i32([ids]), i32(P), parent, rank, torch.bfloat16)
    assert md.device_status() == 0
    _check_attention(out, q, k, v, np.arange(4)[None], P, parent)
    # the accepted path moves in the far pages too
    newp, root, row = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3))
    path = np.array([[0, 3, -1, -1, -1, -1, -1, -1, -1]])
    md.tree_commit_paged(kp, vp, i32([ids]), md.Tree(parent, rank, [16] * 8), i32(P), i32([1]), i32(path), i32([9]), newp,
                         root, row)
    assert md.device_status() == 0 and newp.item() == 202
    assert np.array_equal(to_bits(kp[0, pool - 2, :, 201 - 192]), k[3][:, 203 - 192])


def test_calls_on_another_stream_captured_and_replayed():
    """A step's paged calls in one graph, replayed on new contents of the same buffers."""
    rng = np.random.default_rng(12)
    parent, rank = _tree(16)
    T, B, Hq, Hkv, dh, page = 17, 2, 8, 2, 64, 16
    tree = md.Tree(parent, rank, [16] * 8)
    P = [70, 33]
    table, pool = _table(rng, P, T, page)
    q, out = torch.empty((B, T, Hq, dh), dtype=torch.bfloat16, device="cuda"), None
    kp = torch.empty((pool, Hkv, page, dh), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    qkv = torch.empty((B, T, Hq + 2 * Hkv, dh), dtype=torch.bfloat16, device="cuda")
    pos = i32(np.array(P)[:, None] + np.arange(T)[None])
    freq = torch.tensor(10000.0 ** (-np.arange(dh // 2) / (dh // 2)), dtype=torch.float32, device="cuda")
    out = torch.empty((B, T, Hq, dh), dtype=torch.float32, device="cuda")
    ws = md.workspace(md.attention_paged_workspace_bytes(B, T, Hq, Hkv, dh, page, table.shape[1]))
    tb, Pd = i32(table), i32(P)

    def step(stream=None):
        qs, ks, vs = qkv.split([Hq, Hkv, Hkv], dim=2)
        md.qk_rope_append(qs, ks, vs, pos, freq, q, kp, vp, tb, Pd, stream=stream)
        md.tree_attention_paged(q, kp, vp, tb, Pd, tree, out, ws, stream=stream)

    def fill(seed):
        qkv.copy_(bf16_tensor(gen.normal_bf16(seed, "q", tuple(qkv.shape), 1.0)))
        kp.copy_(bf16_tensor(gen.normal_bf16(seed, "k_cache", tuple(kp.shape), 1.0)))
        vp.copy_(bf16_tensor(gen.normal_bf16(seed, "v_cache", tuple(vp.shape), 1.0)))

    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)                                  # eager, on a stream that is not current
    torch.cuda.current_stream().wait_stream(side)
    eager = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (2, 1):
        fill(seed)
        g.replay()
        torch.cuda.synchronize()
        _check_attention(out, to_bits(q), to_bits(kp), to_bits(vp), table, P, parent)
    assert torch.equal(out, eager)


def test_attention_timeout_flags_and_recovers():
    """As the contiguous kernel's: one chunk's copies withheld, waits of 1 ms."""
    rng = np.random.default_rng(3)
    parent, rank = _tree(64)
    for Hq, Hkv, P, chunk in ((64, 8, [3000], 1), (4, 2, [900], 0)):
        T, dh, page = 65, 128, 64
        table, pool = _table(rng, P, T, page)
        q = gen.normal_bf16(7, "q", (1, T, Hq, dh), 1.0)
        kp = gen.normal_bf16(7, "k_cache", (pool, Hkv, page, dh), 1.0)
        vp = gen.normal_bf16(7, "v_cache", (pool, Hkv, page, dh), 1.0)
        args = [bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(P), parent, rank, torch.float32]
        good = _attention(*args)
        md.device_status(clear=True)
        md.set_wait_limit(1_000_000)
        md.binding.withhold_attention_chunk_for_test(chunk)
        try:
            _attention(*args)
            torch.cuda.synchronize()
            status = md.device_status(clear=True)
        finally:
            md.binding.withhold_attention_chunk_for_test(-1)
            md.set_wait_limit(0)
        assert status & md.binding.DEV_TIMEOUT
        assert torch.equal(_attention(*args), good) and md.device_status() == 0


# ------------------------------------------------------------------- append

APPEND = [
    # B, T, Hq, Hkv, dh, page, rot, norm, interleaved, ragged, prefixes
    ("tree", 2, 17, 4, 2, 64, 16, 64, True, False, False, [0, 37]),
    ("one-token", 3, 1, 8, 1, 128, 16, 128, True, True, False, [15, 16, 0]),
    ("partial-rotation", 1, 5, 3, 1, 128, 48, 48, False, False, False, [100]),
    ("partial-interleaved", 2, 9, 7, 7, 64, 7, 32, True, True, True, [3, 90]),
    ("prompt-idle-rows", 4, 70, 12, 4, 64, 32, 64, True, False, True, [0, -1, 31, 32]),
    ("one-page-a-request", 3, 6, 40, 8, 128, 100, 128, False, False, False, [0, 50, 94]),
    ("far-positions", 2, 3, 4, 2, 128, 64, 128, False, True, False, [10, 61]),
]


@pytest.mark.parametrize("name,B,T,Hq,Hkv,dh,page,rot,norm,inter,ragged,P", APPEND, ids=[c[0] for c in APPEND])
def test_append_matches_oracle(name, B, T, Hq, Hkv, dh, page, rot, norm, inter, ragged, P):
    rng = np.random.default_rng(T + rot)
    table, pool = _table(rng, P, T, page)
    qkv = gen.normal_bf16(11, "q", (B, T, Hq + 2 * Hkv, dh), 2.0)
    qw = gen.normal_bf16(11, "W1", (dh,), 1.0) if norm else None
    kw = gen.normal_bf16(11, "b1", (dh,), 1.0) if norm else None
    freq = (500000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    pos = (np.array(P)[:, None] + rng.integers(0, 5, (B, T))).astype(np.int32)
    if name == "far-positions":
        pos = np.array([[1 << 20, 999_983, 131_071], [2 ** 31 - 1, 77_777_777, -5]], dtype=np.int32)
    n_new = rng.integers(0, T + 1, B).astype(np.int32) if ragged else None
    k0 = gen.normal_bf16(12, "k_cache", (pool, Hkv, page, dh), 1.0)
    v0 = gen.normal_bf16(12, "v_cache", (pool, Hkv, page, dh), 1.0)
    kp, vp = bf16_tensor(k0), bf16_tensor(v0)
    fused = bf16_tensor(qkv)
    q, k, v = fused.split([Hq, Hkv, Hkv], dim=2)
    q_out = torch.full((B, T, Hq, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    md.device_status(clear=True)
    md.qk_rope_append(q, k, v, i32(pos), torch.from_numpy(freq).cuda(), q_out, kp, vp, i32(table), i32(P),
                      q_norm=None if qw is None else bf16_tensor(qw), k_norm=None if kw is None else bf16_tensor(kw),
                      eps=1e-5, interleaved=inter, n_new=None if n_new is None else i32(n_new))
    assert md.device_status() == 0
    rq, written = op.qk_rope_append(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:], pos, freq, table, P,
                                    k0.shape, qw, kw, 1e-5, inter, n_new)
    got = q_out.float().cpu().numpy()
    skip = np.isnan(rq)
    assert (got[skip] == 7.0).all()                     # rows behind a request's tokens are left alone
    tol = 2.0 ** -8 * np.abs(rq) + 2.0 ** -20 * np.max(np.abs(rq), axis=-1, keepdims=True)
    assert (np.abs(got - rq)[~skip] <= tol[~skip]).all()
    gk, gv = to_bits(kp), to_bits(vp)
    for (pg, row), (kr, vr) in written.items():
        tol = 2.0 ** -8 * np.abs(kr) + 2.0 ** -20 * np.max(np.abs(kr), axis=-1, keepdims=True)
        assert (np.abs(bf16_to_f64(gk[pg, :, row]) - kr) <= tol).all()
        assert np.array_equal(gv[pg, :, row], vr)       # values go through bit for bit
        k0[pg, :, row], v0[pg, :, row] = gk[pg, :, row], gv[pg, :, row]
    assert np.array_equal(gk, k0) and np.array_equal(gv, v0)          # nothing else was written
    assert len(written) > 0


def test_append_in_place_other_strides_and_bad_slots():
    B, T, Hq, Hkv, dh, page = 3, 4, 4, 2, 64, 16
    q0 = gen.normal_bf16(1, "q", (B, Hq, T, dh), 1.0)                 # heads before tokens
    k0 = gen.normal_bf16(2, "q", (B, Hkv, T, dh), 1.0)
    pos = np.arange(B * T).reshape(B, T).astype(np.int32)
    freq = np.ones(dh // 2, dtype=np.float32)
    table = np.array([[0, 1], [2, 9], [3, -1]], dtype=np.int32)       # request 1: a page outside the pool of 5
    P = [30, 14, -7]                                                  # request 0: slots 32, 33 past the table; 2: bad
    q, k = bf16_tensor(q0).transpose(1, 2), bf16_tensor(k0).transpose(1, 2)
    kp = torch.zeros((5, Hkv, page, dh), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    dense = q.contiguous()
    md.device_status(clear=True)
    md.qk_rope_append(q, k, k, i32(pos), torch.from_numpy(freq).cuda(), torch.empty_like(dense), kp, vp, i32(table), i32(P))
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PREFIX | md.binding.DEV_BAD_PAGE
    first = kp.clone()
    md.qk_rope_append(dense, k.contiguous(), k.contiguous(), i32(pos), torch.from_numpy(freq).cuda(), dense, kp, vp,
                      i32(table), i32(P))                             # q_out is q
    md.device_status(clear=True)
    rq, written = op.qk_rope_append(q0.transpose(0, 2, 1, 3), k0.transpose(0, 2, 1, 3), k0.transpose(0, 2, 1, 3), pos, freq,
                                    table, [30, 14, 0], kp.shape)
    got = dense.float().cpu().numpy()
    assert (np.abs(got - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -20 * np.abs(rq).max()).all()   # queries in every row
    assert torch.equal(first, kp)
    rows = {(p, r) for p in range(5) for r in range(page) if bool(kp[p, :, r].any())}
    assert rows == {pr for pr in written if pr[0] != 3}               # nothing for request 2 (page 3)


# ------------------------------------------------------------------- commit

@pytest.mark.parametrize("layers,Hkv,dh,page,P", [(1, 2, 64, 16, [0, 15, -1, 33]), (3, 8, 128, 64, [100, -1, 5, 61]),
                                                  (5, 1, 128, 5, [0, 3, 4, 29])])
def test_commit_matches_oracle(layers, Hkv, dh, page, P):
    """Paths that cross pages, whose sources are also destinations, of every length."""
    rng = np.random.default_rng(page)
    # a tree whose deep path (0, 2, 3, 5, 6, ...) reads slots it also writes
    parent = [-1, 0, 0, 2, 2, 3, 5, 6, 7, 8]
    rank = [0, 0, 1, 0, 1, 0, 0, 0, 0, 0]
    T, B = len(parent), len(P)
    tree = md.Tree(parent, rank, [16] * 8)
    table, pool = _table(rng, P, T, page)
    k0 = gen.normal_bf16(1, "k_cache", (layers, pool, Hkv, page, dh), 1.0)
    v0 = gen.normal_bf16(1, "v_cache", (layers, pool, Hkv, page, dh), 1.0)
    leaves = [9, 1, 0, 4]
    path = np.full((B, 9), -1, dtype=np.int32)
    L = np.zeros(B, dtype=np.int32)
    for b in range(B):
        p = list(_ancestors(parent, leaves[b % 4]))[::-1]
        path[b, :len(p)], L[b] = p, len(p) - 1
    bonus = rng.integers(0, 1000, B)
    kp, vp = bf16_tensor(k0), bf16_tensor(v0)
    outs = [torch.full((B,), 77, dtype=torch.int32, device="cuda") for _ in range(3)]
    md.device_status(clear=True)
    squeeze = (lambda x: x[0]) if layers == 1 else (lambda x: x)      # a single layer may be 4-D
    md.tree_commit_paged(squeeze(kp), squeeze(vp), i32(table), tree, i32(P), i32(L), i32(path), i32(bonus), *outs)
    assert md.device_status() == 0
    rk, rv, newp, root, row = op.tree_commit_paged(k0, v0, table, P, L, path, bonus, T)
    assert np.array_equal(to_bits(kp), rk) and np.array_equal(to_bits(vp), rv)
    for got, want in zip(outs, (newp, root, row)):
        assert got.cpu().tolist() == want.tolist()


def test_commit_leaves_bad_requests_alone():
    parent, rank = [-1, 0, 0, 1], [0, 0, 1, 0]
    tree = md.Tree(parent, rank, [2, 1])
    k0 = gen.normal_bf16(1, "k_cache", (4, 1, 8, 64), 1.0)
    table = np.array([[0, -1], [1, 9], [2, -1], [3, -1]], dtype=np.int32)
    P, L = [2, 5, 6, 1], [2, 2, 1, 3]
    path = np.array([[0, 2, 3], [0, 1, 3], [0, 2, -1], [0, 1, 3]])    # 0: 3 is no child of 2; 1: slot 8 in a bad page;
    kp = bf16_tensor(k0)                                              # 2: slot 8 has no page; 3: longer than the tree is deep
    outs = [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(3)]
    md.device_status(clear=True)
    md.tree_commit_paged(kp, kp.clone(), i32(table), tree, i32(P), i32(L), i32(path), i32([1, 2, 3, 4]), *outs)
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PATH | md.binding.DEV_BAD_PAGE
    assert np.array_equal(to_bits(kp), k0)
    assert outs[0].cpu().tolist() == P and outs[2].cpu().tolist() == [-1] * 4
    assert outs[1].cpu().tolist() == [1, 2, 3, 4]


def test_commit_refuses_nodes_without_a_page():
    """A resize that ran short leaves rows without pages for their tree: nothing of theirs is
    accepted, not even what would stay where it is, and the next resize frees no foreign slots."""
    parent, rank = [-1, 0, 0, 1], [0, 0, 1, 0]
    T, page, pool, width = 4, 16, 5, 3
    tree = md.Tree(parent, rank, [2, 1])
    table, n, ref = _state(4, width, pool)
    P = np.array([16, 31, 16, -1], dtype=np.int32)
    g = [i32(x) for x in (table, n, ref)]
    md.device_status(clear=True)
    md.pages_resize(*g, i32(P), page)
    md.pages_resize(*g, i32(P), page, extra=T)                 # three rows need one more page each, one is left
    assert md.device_status(clear=True) == md.binding.DEV_NO_PAGES
    held = g[0].cpu().numpy()
    assert g[1].cpu().tolist() == [2, 2, 1, 0]
    k0 = gen.normal_bf16(1, "k_cache", (2, pool, 1, page, 64), 1.0)
    kp, vp = bf16_tensor(k0), bf16_tensor(k0)
    ref_k = k0
    bonus = [1, 2, 3, 4]
    # paths of the root alone; of nodes in place; moved ones. Row 1's root has a page, its node 1 none.
    for L, path in (([0, 0, 0, 0], [[0, -1, -1]] * 4), ([1] * 4, [[0, 1, -1]] * 4), ([2] * 4, [[0, 1, 3]] * 4)):
        outs = [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(3)]
        md.tree_commit_paged(kp, vp, g[0], tree, i32(P), i32(L), i32(path), i32(bonus), *outs)
        assert md.device_status(clear=True) == md.binding.DEV_BAD_PAGE
        ref_k, _, newp, root, row = op.tree_commit_paged(ref_k, ref_k, held, P, L, np.array(path), bonus, T)
        assert newp.tolist() == [17 + L[0], 32 if L[0] == 0 else 31, 16, -1]
        assert [x.cpu().tolist() for x in outs] == [newp.tolist(), root.tolist(), row.tolist()]
        assert np.array_equal(to_bits(kp), ref_k) and np.array_equal(to_bits(vp), ref_k)
    md.pages_resize(*g, outs[0], page)                         # trim: the refused rows keep what their prefixes need
    assert md.device_status(clear=True) == 0 and g[1].cpu().tolist() == [2, 2, 1, 0]


# -------------------------------------------------------------------- pages

def _state(B, width, pool):
    return (np.full((B, width), -1, dtype=np.int32), np.zeros(B, dtype=np.int32), np.zeros(pool, dtype=np.int32))


@pytest.mark.parametrize("B,width,pool,page", [(1, 1, 1, 16), (5, 7, 20, 16), (40, 30, 900, 1), (3, 5000, 9001, 64),
                                               (1500, 8, 20000, 32), (300, 300, 60001, 16)])
def test_resize_matches_oracle(B, width, pool, page):
    rng = np.random.default_rng(pool)
    table, n, ref = _state(B, width, pool)
    g = [i32(x) for x in (table, n, ref)]
    seen_short = False
    for step in range(6):
        length = rng.integers(-1, width * page + 1, B)
        length[rng.random(B) < 0.2] = -1
        extra = int(rng.integers(0, 2 * page)) if step % 2 else 0
        length = np.minimum(length, width * page - extra).astype(np.int32)
        md.device_status(clear=True)
        md.pages_resize(*g, i32(length), page, extra=extra)
        table, n, ref, short = op.pages_resize(table, n, ref, length, page, extra)
        assert md.device_status(clear=True) == (md.binding.DEV_NO_PAGES if short else 0)
        for got, want in zip(g, (table, n, ref)):
            assert np.array_equal(got.cpu().numpy(), want), step
        seen_short |= short
    assert seen_short or pool != 20        # 5 rows of 3.5 pages on average: the pool of 20 runs short


def test_resize_leaves_impossible_rows_alone():
    table = np.array([[0, 1, -1], [2, -1, -1], [3, -1, -1], [9, -1, -1]], dtype=np.int32)
    n, ref = np.array([2, 1, 7, 1], dtype=np.int32), np.array([1, 1, 1, 1, 0, 0], dtype=np.int32)
    g = [i32(x) for x in (table, n, ref)]
    # row 0 wants more than the table holds, row 2's count is impossible, row 3 gives back a page outside the pool
    md.device_status(clear=True)
    md.pages_resize(*g, i32([49, 17, 16, -1]), 16)
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PREFIX | md.binding.DEV_BAD_PAGE
    assert g[0].cpu().tolist() == [[0, 1, -1], [2, 4, -1], [3, -1, -1], [-1, -1, -1]]
    assert g[1].cpu().tolist() == [2, 2, 7, 0]
    assert g[2].cpu().tolist() == [1, 1, 1, 1, 1, 0]
    # a page that nobody holds is given back: flagged, its count stays 0
    g = [i32([[5, 5]]), i32([2]), i32([0, 0, 0, 0, 0, 1])]
    md.pages_resize(*g, i32([-1]), 16)
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PAGE and g[2].cpu().tolist() == [0] * 6
    g = [i32([[-1, -1]]), i32([0]), i32([0, 0])]
    md.pages_resize(*g, i32([2 ** 31 - 1]), 16, extra=2 ** 31 - 1)
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PREFIX and g[1].cpu().tolist() == [0]


def test_resize_leaves_rows_with_negative_counts_alone():
    """Counts below zero: nothing is given to such a row, nothing written through it. The
    table lies between guard rows, as a row's first entry minus its count would reach them."""
    width, pool = 4, 12
    counts = [-5, -1, 2, -2, -2 ** 31, 1, -2 ** 31 + 1, -5]
    B = len(counts)
    full = np.full((B + 8, width), 77, dtype=np.int32)
    table = full[4:4 + B]
    table[:] = 33                                          # what a row with a bad count holds means nothing
    table[2], table[5] = [0, 1, -1, -1], [2, -1, -1, -1]
    ref = np.array([1, 1, 1] + [0] * (pool - 3), dtype=np.int32)
    length = [64, 1, 48, 64, 64, 64, 0, -1]
    gfull, gn, gref = i32(full), i32(counts), i32(ref)
    md.device_status(clear=True)
    md.pages_resize(gfull[4:4 + B], gn, gref, i32(length), 16)
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PAGE
    rt, rn, rr, short = op.pages_resize(table, np.array(counts), ref, np.array(length), 16)
    assert not short and rn.tolist() == [-5, -1, 3, -2, -2 ** 31, 4, -2 ** 31 + 1, -5]
    full[4:4 + B] = rt
    assert np.array_equal(gfull.cpu().numpy(), full)
    assert gn.cpu().tolist() == rn.tolist() and np.array_equal(gref.cpu().numpy(), rr)
    # one row alone, the first of its table; the pool is not drained
    gfull, gn, gref = i32(np.full((3, width), 77)), i32([-5]), i32(np.zeros(pool))
    md.pages_resize(gfull[1:2], gn, gref, i32([64]), 16, extra=16)
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PAGE
    assert (gfull == 77).all() and gn.item() == -5 and not gref.any()


@pytest.mark.parametrize("layers,Hkv,dh,page,B,n", [(1, 1, 64, 16, 6, 2), (3, 2, 128, 7, 9, 4), (2, 8, 128, 64, 40, 19)])
def test_fork_matches_oracle(layers, Hkv, dh, page, B, n):
    rng = np.random.default_rng(page + n)
    width, pool = 6, 4 * B
    table, cnt, ref = _state(B, width, pool)
    k = gen.normal_bf16(1, "k_cache", (layers, pool, Hkv, page, dh), 1.0)
    v = gen.normal_bf16(1, "v_cache", (layers, pool, Hkv, page, dh), 1.0)
    length = rng.integers(0, 3 * page + 1, B).astype(np.int32)
    length[:3] = [-1, 0, 2 * page]                     # an idle row, an empty one, a full last page
    table, cnt, ref, _ = op.pages_resize(table, cnt, ref, length, page)
    g = [bf16_tensor(k), bf16_tensor(v)] + [i32(x) for x in (table, cnt, ref)]
    glen = i32(length)
    ws = md.workspace(md.pages_fork_workspace_bytes(B, n))
    for step in range(5):
        rows = rng.permutation(B)
        src, dst = rows[:n].copy(), rows[n:2 * n].copy()
        if step == 0:
            src[:2] = [0, 2]
            dst = np.array([r for r in range(3, B) if r not in src][:n])
        if step == 1:
            src[:] = src[0]                            # one source, several destinations
        if step == 2:
            src[n // 2:] = -1                          # unused entries
        md.device_status(clear=True)
        md.pages_fork(*g, i32(src), i32(dst), glen, ws)
        assert md.device_status(clear=True) == 0
        k, v, table, cnt, ref, length = op.pages_fork(k, v, table, cnt, ref, src, dst, length)
        assert np.array_equal(to_bits(g[0]), k) and np.array_equal(to_bits(g[1]), v)
        for got, want in zip(g[2:] + [glen], (table, cnt, ref, length)):
            assert np.array_equal(got.cpu().numpy(), want), step


def test_fork_leaves_out_what_cannot_be():
    page, pool = 16, 6
    table = np.array([[0, 1], [2, -1], [3, -1], [-1, -1], [4, -1]], dtype=np.int32)
    cnt, ref = np.array([2, 1, 1, 0, 1], dtype=np.int32), np.array([1, 1, 1, 1, 1, 0], dtype=np.int32)
    length = np.array([20, 16, 40, -1, 3], dtype=np.int32)             # row 2: longer than its pages
    k = gen.normal_bf16(1, "k_cache", (1, pool, 1, page, 64), 1.0)

    def call(src, dst, ref=ref):
        g = [bf16_tensor(k), bf16_tensor(k)] + [i32(x) for x in (table, cnt, ref, length)]
        md.device_status(clear=True)
        md.pages_fork(g[0], g[1], g[2], g[3], g[4], i32(src), i32(dst), g[5], md.workspace(4096))
        return md.device_status(clear=True), g

    same = lambda g: all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(g[2:], (table, cnt, ref, length)))  # noqa: E731
    for src, dst in (([0], [0]), ([0], [5]), ([7], [1]), ([-2], [1]), ([0, 1], [1, 3][:1] + [0])):
        status, g = call(src, dst)
        assert status == md.binding.DEV_BAD_ROW and same(g), (src, dst)
    status, g = call([2], [3])
    assert status == md.binding.DEV_BAD_PREFIX and same(g)
    status, g = call([0, 1], [3, 3])                                   # the second fork into row 3 is left out
    assert status == md.binding.DEV_BAD_ROW
    assert g[2].cpu().tolist()[3] == [0, 5] and g[4].cpu().tolist() == [2, 1, 1, 1, 1, 1]
    assert g[5].cpu().tolist() == [20, 16, 40, 20, 3]
    assert np.array_equal(to_bits(g[0])[0, 5, 0, :4], k[0, 1, 0, :4]) and np.array_equal(to_bits(g[0])[0, 5, 0, 4:], k[0, 5, 0, 4:])
    status, g = call([0], [4], ref=np.array([1, 1, 1, 1, 1, 1], dtype=np.int32))     # row 4's own page serves
    assert status == 0 and g[2].cpu().tolist()[4] == [0, 4]
    status, g = call([0], [3], ref=np.array([1, 1, 1, 1, 1, 1], dtype=np.int32))     # no page left: row 3 stays empty
    assert status == md.binding.DEV_NO_PAGES and g[5].cpu().tolist()[3] == -1 and g[3].cpu().tolist()[3] == 0
    assert g[4].cpu().tolist() == [1, 1, 1, 1, 1, 1]


@pytest.mark.parametrize("bad", [-1, 6, -2 ** 31])
def test_fork_is_left_out_without_a_page_to_copy(bad):
    """The source ends inside a page outside the pool: the destination stays as it is, and no page is taken."""
    page, pool = 16, 6
    table = np.array([[0, bad], [2, -1], [3, bad], [-1, -1], [-1, -1]], dtype=np.int32)
    cnt, ref = np.array([2, 1, 2, 0, 0], dtype=np.int32), np.array([1, 0, 1, 1, 0, 0], dtype=np.int32)
    length = np.array([20, 9, 32, -1, -1], dtype=np.int32)             # row 2 ends with its pages: nothing to copy
    k = gen.normal_bf16(1, "k_cache", (1, pool, 1, page, 64), 1.0)
    src, dst = np.array([0, 1]), np.array([3, 4])
    g = [bf16_tensor(k), bf16_tensor(k)] + [i32(x) for x in (table, cnt, ref, length)]
    md.device_status(clear=True)
    md.pages_fork(g[0], g[1], g[2], g[3], g[4], i32(src), i32(dst), g[5], md.workspace(4096))
    assert md.device_status(clear=True) == md.binding.DEV_BAD_PAGE
    k2, _, t2, c2, r2, l2 = op.pages_fork(k, k, table, cnt, ref, src, dst, length)
    assert t2[3].tolist() == [-1, -1] and t2[4].tolist() == [1, -1] and r2.tolist() == [1, 1, 1, 1, 0, 0]
    assert np.array_equal(to_bits(g[0]), k2) and np.array_equal(to_bits(g[1]), k2)
    for got, want in zip(g[2:], (t2, c2, r2, l2)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_two_streams_with_workspaces_of_their_own():
    """Attention calls of two streams at once, and one call's result on a side stream."""
    rng = np.random.default_rng(21)
    parent, rank = _tree(16)
    T, Hq, Hkv, dh, page, P = 17, 8, 2, 128, 32, [900, 33]
    table, pool = _table(rng, P, T, page)
    q = bf16_tensor(gen.normal_bf16(2, "q", (2, T, Hq, dh), 1.0))
    kp = bf16_tensor(gen.normal_bf16(2, "k_cache", (pool, Hkv, page, dh), 1.0))
    vp = bf16_tensor(gen.normal_bf16(2, "v_cache", (pool, Hkv, page, dh), 1.0))
    tb, Pd = i32(table), i32(P)
    want = _attention(q, kp, vp, tb, Pd, parent, rank, torch.bfloat16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(want) for _ in range(8)] for _ in streams]
    wss = [md.workspace(md.attention_paged_workspace_bytes(2, T, Hq, Hkv, dh, page, table.shape[1])) for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                _attention(q, kp, vp, tb, Pd, parent, rank, torch.bfloat16, ws=wss[s], out=outs[s][i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for per in outs for o in per) and md.device_status() == 0


@pytest.mark.parametrize("B,T,Hq,Hkv,page,P", [(40, 1, 8, 1, 16, (0, 700)), (70, 17, 8, 2, 32, (1, 300)), (24, 65, 8, 4, 64, (0, 400)), (300, 1, 2, 1, 16, (0, 90))])
def test_more_units_than_one_wave(B, T, Hq, Hkv, page, P):
    """Grids past one wave, requests taken from the longest down."""
    rng = np.random.default_rng(B)
    parent, rank = _tree(T - 1)
    lens = [int(x) for x in rng.integers(P[0], P[1], B)]
    lens[3] = -1
    table, pool = _table(rng, lens, T, page)
    q = gen.normal_bf16(4, "q", (B, T, Hq, 64), 1.0)
    kp = gen.normal_bf16(4, "k_cache", (pool, Hkv, page, 64), 1.0)
    vp = gen.normal_bf16(4, "v_cache", (pool, Hkv, page, 64), 1.0)
    out = _attention(bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(lens), parent, rank, torch.bfloat16)
    assert md.device_status() == 0
    _check_attention(out, q, kp, vp, table, lens, parent)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,dh,page,longest", [(170, 1, 4, 1, 128, 16, 300), (90, 7, 6, 2, 64, 48, 200),
                                                        (80, 17, 8, 4, 128, 64, 150), (160, 64, 2, 1, 64, 16, 130),
                                                        (150, 64, 1, 1, 128, 128, 90), (150, 64, 8, 1, 128, 32, 90)])
def test_many_short_requests(B, T, Hq, Hkv, dh, page, longest, dtype):
    """More CTAs than SMs, few keys each. Slots that no request uses hold NaN, and the
    last node's V is infinite in one column: that reaches the node's own rows alone."""
    rng = np.random.default_rng(B + T)
    parent, rank = _tree(T - 1)
    lens = [int(x) for x in rng.integers(0, longest, B)]
    lens[:8] = [0, -1, 63, 64, 65, 1, 127, 128 - T if T < 128 else 0]
    lens = [min(p, longest) for p in lens]
    table, pool = _table(rng, lens, T, page)
    q = gen.normal_bf16(6, "q", (B, T, Hq, dh), 1.0)
    k = gen.normal_bf16(6, "k_cache", (pool, Hkv, page, dh), 1.0)
    v = gen.normal_bf16(6, "v_cache", (pool, Hkv, page, dh), 1.0)
    kp, vp = np.full_like(k, NAN), np.full_like(v, NAN)
    for b, p in enumerate(lens):
        for s in range(p + T if p >= 0 else 0):
            at = (table[b, s // page], slice(None), s % page)
            kp[at], vp[at] = k[at], v[at]
    args = (bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(lens), parent, rank, dtype)
    md.device_status(clear=True)
    out, again = _attention(*args), _attention(*args)
    assert md.device_status() == 0
    _check_attention(out, q, kp, vp, table, lens, parent)
    assert torch.equal(out, again) and not out[1].any()
    if T > 1:
        inf = vp.copy()
        for b, p in enumerate(lens):
            if p >= 0:
                inf[table[b, (p + T - 1) // page], :, (p + T - 1) % page, 5] = 0x7F80
        bad = _attention(args[0], args[1], bf16_tensor(inf), *args[3:])
        live = [b for b in range(B) if lens[b] >= 0]
        assert torch.isinf(bad[live, T - 1, :, 5]).all()
        bad[:, T - 1, :, 5] = out[:, T - 1, :, 5]
        assert torch.equal(bad, out)


def test_many_short_requests_timeout_flags_and_recovers():
    rng = np.random.default_rng(4)
    parent, rank = _tree(4)
    for P, chunk in ((300, 1), (40, 0)):
        B, T, Hq, Hkv, dh, page = 170, 5, 4, 1, 64, 16
        table, pool = _table(rng, [P] * B, T, page)
        q = gen.normal_bf16(8, "q", (B, T, Hq, dh), 1.0)
        kp = gen.normal_bf16(8, "k_cache", (pool, Hkv, page, dh), 1.0)
        vp = gen.normal_bf16(8, "v_cache", (pool, Hkv, page, dh), 1.0)
        args = [bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32([P] * B), parent, rank, torch.bfloat16]
        good = _attention(*args)
        md.device_status(clear=True)
        md.set_wait_limit(1_000_000)
        md.binding.withhold_attention_chunk_for_test(chunk)
        try:
            _attention(*args)
            torch.cuda.synchronize()
            status = md.device_status(clear=True)
        finally:
            md.binding.withhold_attention_chunk_for_test(-1)
            md.set_wait_limit(0)
        assert status & md.binding.DEV_TIMEOUT
        assert torch.equal(_attention(*args), good) and md.device_status() == 0


def test_scores_far_apart_and_rows_of_nan():
    """Maxima that climb by thousands from chunk to chunk (the running maximum moves,
    the result is rescaled), a prefix key of NaN, and a query of NaN."""
    T, Hq, Hkv, dh, page, P = 1, 4, 2, 64, 16, [1000, 1000, 1000]
    rng = np.random.default_rng(8)
    table, pool = _table(rng, P, T, page)
    q = gen.normal_bf16(5, "q", (3, T, Hq, dh), 1.0)
    kf = bf16_to_f64(gen.normal_bf16(5, "k_cache", (pool, Hkv, page, dh), 1.0))
    for b in range(3):
        for i, pg in enumerate(table[b]):
            kf[pg] *= 1.0 + 2.0 * i if pg >= 0 else 1.0
    kp = to_bits(torch.from_numpy(kf).to(torch.bfloat16))
    vp = gen.normal_bf16(5, "v_cache", (pool, Hkv, page, dh), 1.0)
    kp[table[1, 5], 0, 3] = NAN                            # KV head 0 of request 1
    q[2, 0, 1] = NAN                                       # query head 1 of request 2
    for dtype in (torch.float32, torch.bfloat16):
        out = _attention(bf16_tensor(q), bf16_tensor(kp), bf16_tensor(vp), i32(table), i32(P), [-1], [0], dtype)
        nan = torch.isnan(out).all(dim=-1).cpu().numpy()
        want = np.zeros_like(nan)
        want[1, 0, :2] = True
        want[2, 0, 1] = True
        assert np.array_equal(nan, want) and np.array_equal(torch.isnan(out).any(dim=-1).cpu().numpy(), want)
        ref = op.tree_attention_paged(q, kp, vp, table, P, [-1])
        absv = op.tree_attention_paged(q, kp, vp & 0x7FFF, table, P, [-1])
        got = out.float().cpu().numpy()
        # scores of up to 64 * 127 * 3.5^2 / 8 in fp32: off by 2^-24 of that and of their products' sum
        wide = 2.0 ** -7
        tol = 2 * (wide + 2.0 ** -8) * absv + 2.0 ** -8 * np.abs(ref)
        assert (np.abs(got - ref) <= tol)[~want].all()


def _climbing(rng, slots):
    """Levels of the slots, one for 64 of them: rising by up to 12 a step to at most 60, then from 0 again.
    The steps lie on both sides of 8, where a running reference maximum moves."""
    out, level = [], 0.0
    for i in range(-(-slots // 64)):
        if i and rng.random() < 0.06:
            level = 0.0
        out += [level] * 64
        level = min(level + rng.choice([0.0, 4.0, 7.75, 8.25, 9.0, 12.0]), 60.0)
    return np.array(out[:slots])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,dh,page,P", [(1, 1, 4, 1, 128, 64, (20001, 20001)),     # one tile, cut over a cluster
                                                  (80, 1, 8, 2, 64, 16, (500, 1180)),        # one tile, whole
                                                  (20, 40, 16, 4, 128, 64, (900, 1950)),     # two tiles
                                                  (400, 5, 4, 1, 64, 16, (200, 590))],       # half a CTA's form
                         ids=["cluster", "one-tile", "two-tiles", "short"])
def test_maxima_that_climb_along_a_walk(B, T, Hq, Hkv, dh, page, P, dtype):
    """Walks of 8 to 20 jobs of 64 keys whose scores climb: sums and results are rescaled on the way,
    inside and between stretches of 128 keys. A key's weight is about 2^level and its value about
    2^-level, so that every step of the climb counts alike: a rescaling left out or done twice is
    off by the result's size.

    Tolerance: scores of up to 62 in log2 units, sums of dh products in fp32, each off by at most
    dh 2^-24 of that, so a weight by ln 2 times 62 dh 2^-24; numerator and denominator twice that of A.
    bf16 results: the weights' and the result's rounding, 2^-8 each, on top."""
    rng = np.random.default_rng(B + T)
    parent, rank = _tree(T - 1)
    lens = [int(x) for x in rng.integers(P[0], P[1] + 1, B)]
    table, pool = _table(rng, lens, T, page)
    q = bf16_to_f64(gen.normal_bf16(31, "q", (B, T, Hq, dh), 0.25))
    k = bf16_to_f64(gen.normal_bf16(31, "k_cache", (pool, Hkv, page, dh), 0.25))
    v = bf16_to_f64(gen.normal_bf16(31, "v_cache", (pool, Hkv, page, dh), 1.0))
    q[..., 0] = np.resize([1.0, 0.75, 0.5], Hq)
    for b, p in enumerate(lens):
        level = _climbing(rng, p + T)
        level[p:] = level[p - 1]                              # the tree's nodes: the last level
        for i in range(-(-(p + T) // page)):
            at = level[i * page:(i + 1) * page]
            k[table[b, i], :, :len(at), 0] = at
            v[table[b, i], :, :len(at)] *= (2.0 ** -at)[None, :, None]
    bits = [to_bits(torch.from_numpy(x).to(torch.bfloat16)) for x in (q, k, v)]
    scale = float(np.float32(np.log(2.0)))
    md.device_status(clear=True)
    out = _attention(*(bf16_tensor(x) for x in bits), i32(table), i32(lens), parent, rank, dtype, scale=scale)
    assert md.device_status() == 0
    ref = op.tree_attention_paged(*bits, table, lens, parent, scale)
    absv = op.tree_attention_paged(bits[0], bits[1], bits[2] & 0x7FFF, table, lens, parent, scale)
    off = 2 * np.log(2.0) * 62 * dh * 2.0 ** -24
    tol = off * absv
    if dtype == torch.bfloat16:
        tol = (off + 2 * 2.0 ** -8) * absv + 2.0 ** -8 * np.abs(ref)
    got = out.float().cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3], tol[bad][:3])


@pytest.mark.parametrize("positive", [False, True], ids=["values-of-both-signs", "values-of-one-sign"])
@pytest.mark.parametrize("T,P", [(1, 660_000), (65, 330_000), (17, 128)], ids=["one-tile", "two-tiles", "short"])
def test_fp32_results_keep_their_bits_at_any_length(T, P, positive):
    """fp32 results of over 20000 keys a stream against 64 bits, N(0, 1) inputs.

    Bounds. A score: dh / 16 = 4 steps of the tensor cores' sum, each dropping less than 2^-23 of a
    partial sum of at most 6 (in units of the scaled score): a weight is off by at most 2.9e-6, and its
    exponential by 2^-22 more. With values of both signs the weights' errors and the result are sums
    of the same random signs: 3.2e-6 of the result in the 2-norm (weights of two bf16 parts alone would
    give 2^-16 / sqrt(3) = 8.8e-6). With values of one sign what the accumulator drops adds up: 8 steps
    and 3 parts in a stretch of 128 keys, below 24 * 2^-23 = 2.9e-6, with the weights 6.1e-6 of A."""
    parent, rank = _tree(T - 1)
    Hq, dh, page = 4, 64, 64
    n = -(-(P + T) // page)
    g = torch.Generator(device="cuda").manual_seed(T)
    kp, vp = (torch.randn((n, 1, page, dh), generator=g, device="cuda").bfloat16() for _ in range(2))
    vp = vp.abs() if positive else vp
    q = torch.randn((1, T, Hq, dh), generator=g, device="cuda").bfloat16()
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    md.device_status(clear=True)
    out = _attention(q, kp, vp, table, i32([P]), parent, rank, torch.float32)
    assert md.device_status() == 0
    k, v = (x[table[0].long(), 0].reshape(-1, dh)[:P + T].double() for x in (kp, vp))
    hide = torch.ones((T, T), dtype=torch.bool)
    for t in range(T):
        hide[t, list(_ancestors(parent, t))] = False
    err = size = 0.0
    for h in range(Hq):
        x = q[0, :, h].double() @ k.T / dh ** 0.5
        x[:, P:].masked_fill_(hide.cuda(), float("-inf"))
        w = torch.softmax(x, dim=1)
        ref = w @ v
        off = (out[0, :, h].double() - ref).abs()
        assert (off <= 6.1e-6 * (w @ v.abs())).all(), float((off / (w @ v.abs())).max())
        err, size = err + float(off.square().sum()), size + float(ref.square().sum())
    if not positive:
        assert (err / size) ** 0.5 <= 3.2e-6, (err / size) ** 0.5
