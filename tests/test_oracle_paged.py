"""Pins of the paged-cache oracle (CPU): against the contiguous oracles, closed
forms of the rotation, and conservation of the pages."""
import numpy as np
import pytest

from oracle import attention as oa
from oracle import commit as oc
from oracle import paged as op
from oracle import tree as ot
from oracle.heads import bf16_to_f64
from seeded_inputs import gen
from seeded_inputs.workloads import TREE_ACCEPT


def scatter(rng, cache, page, spare=3):
    """A contiguous cache [B, Hkv, S, dh] as pages in random order: pool and table."""
    B, H, S, dh = cache.shape
    width = -(-S // page)
    n = B * width + spare
    table = rng.permutation(n)[:B * width].reshape(B, width).astype(np.int32)
    pool = np.zeros((n, H, page, dh), dtype=cache.dtype)
    for b in range(B):
        for s in range(S):
            pool[table[b, s // page], :, s % page] = cache[b, :, s]
    return pool, table


def test_paged_attention_and_commit_reduce_to_the_contiguous_oracles():
    rng = np.random.default_rng(0)
    parent, _, _ = ot.spec_from_tuples(ot.select_tree((4, 3, 2, 2), TREE_ACCEPT, 16))
    T, B, P = len(parent), 3, [0, 21, 50]
    q = gen.normal_bf16(1, "q", (B, T, 4, 64), 1.0)
    kc = gen.normal_bf16(1, "k_cache", (B, 2, 80, 64), 1.0)
    vc = gen.normal_bf16(1, "v_cache", (B, 2, 80, 64), 1.0)
    state = rng.bit_generator.state
    kp, table = scatter(rng, kc, 16)
    rng.bit_generator.state = state
    vp, _ = scatter(rng, vc, 16)
    ref = oa.tree_attention(q, kc, vc, P, parent)
    assert np.array_equal(op.tree_attention_paged(q, kp, vp, table, P, parent), ref)
    assert not op.tree_attention_paged(q, kp, vp, table, [0, -1, 50], parent)[1].any()
    path = np.array([[0, 2, 4, -1, -1], [0, -1, -1, -1, -1], [0, 1, 3, 7, -1]])
    L = [2, 0, 3]
    k2, v2, newp, root, row = op.tree_commit_paged(kp[None], vp[None], table, P, L, path, [5, 6, 7], T)
    rk, rv, rp, rr, rrow = oc.tree_commit(kc, vc, P, L, path, [5, 6, 7], T)
    for b in range(B):
        assert np.array_equal(op.gather(k2[0], table[b], 80), rk[b])
        assert np.array_equal(op.gather(v2[0], table[b], 80), rv[b])
    assert newp.tolist() == rp.tolist() and root.tolist() == rr.tolist() and row.tolist() == rrow.tolist()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal(64)
    f = np.array([np.pi / 2] + [0.0] * 31)
    y = op.norm_rotate(x, None, 1, f, 0.0, interleaved)
    i, j = (0, 1) if interleaved else (0, 32)
    assert np.isclose(y[i], -x[j]) and np.isclose(y[j], x[i])           # a quarter turn of the first pair
    rest = [e for e in range(64) if e not in (i, j)]
    assert np.array_equal(y[rest], x[rest])
    # a rotation keeps lengths, and scores depend on the difference of positions alone
    g = 10.0 ** -np.linspace(0, 4, 32)
    a, b = rng.standard_normal(64), rng.standard_normal(64)
    rot = lambda v, p: op.norm_rotate(v, None, p, g, 0.0, interleaved)   # noqa: E731
    assert np.isclose(np.linalg.norm(rot(a, 123456)), np.linalg.norm(a))
    assert np.isclose(rot(a, 1007) @ rot(b, 1000), rot(a, 7) @ rot(b, 0))
    n = op.norm_rotate(x, np.full(64, 2.0), 0, g, 0.0, interleaved)
    assert np.isclose(np.mean(n * n), 4.0)                              # RMS 1, times the weight


def test_append_skips_padding_idle_rows_and_slots_without_a_page():
    q = gen.normal_bf16(2, "q", (3, 4, 2, 64), 1.0)
    k = gen.normal_bf16(2, "k_cache", (3, 4, 1, 64), 1.0)
    pos = np.arange(12).reshape(3, 4)
    table = np.array([[3, 1], [0, 2], [2, 9]], dtype=np.int32)
    out, w = op.qk_rope_append(q, k, k, pos, np.zeros(32), table, [14, -1, 30], (4, 1, 16, 64), n_new=[3, 4, 4])
    assert np.isnan(out[0, 3]).all() and np.isnan(out[1]).all() and np.array_equal(out[0, 0], bf16_to_f64(q[0, 0]))
    assert sorted(w) == [(1, 0), (3, 14), (3, 15)]     # request 2: slots 30, 31 in a page outside the pool, 32 and 33 past the table


def test_commit_keeps_a_request_without_pages_as_it_is():
    k = gen.normal_bf16(3, "k_cache", (1, 4, 1, 4, 64), 1.0)
    table = np.array([[0, -1], [1, 9], [2, 3]])
    # row 0: the root has a page at first, its child none; row 1: a page outside the pool
    for P, L, path, newp, row in (([3, 4, 4], 0, [0, -1], [4, 4, 5], [0, -1, 8]), ([3, 4, 4], 1, [0, 1], [3, 4, 6], [-1, -1, 9]),
                                  ([4, 4, 4], 0, [0, -1], [4, 4, 5], [-1, -1, 8])):
        k2, _, got, root, head = op.tree_commit_paged(k, k, table, P, [L] * 3, np.array([path] * 3), [1, 2, 3], 4)
        assert got.tolist() == newp and root.tolist() == [1, 2, 3] and head.tolist() == row
        assert np.array_equal(k2, k)                            # nothing moves on these paths


def _consistent(table, n_pages, ref):
    count = np.zeros_like(ref)
    for b in range(len(n_pages)):
        assert (table[b, :n_pages[b]] >= 0).all() and (table[b, n_pages[b]:] == -1).all()
        for p in table[b, :n_pages[b]]:
            count[p] += 1
    assert np.array_equal(count, ref)


def test_resize_and_fork_conserve_pages():
    rng = np.random.default_rng(5)
    B, width, pool, page = 6, 5, 24, 16
    table = np.full((B, width), -1, dtype=np.int32)
    n, ref = np.zeros(B, dtype=np.int32), np.zeros(pool, dtype=np.int32)
    length = np.full(B, -1, dtype=np.int32)
    k = np.zeros((1, pool, 1, page, 8), dtype=np.uint16)
    for step in range(60):
        length = np.where(rng.random(B) < 0.3, rng.integers(-1, width * page, B), length).astype(np.int32)
        table, n, ref, short = op.pages_resize(table, n, ref, length, page)
        _consistent(table, n, ref)
        if short:
            assert (ref == 0).sum() < width * B
        length = np.where(n * page >= length, length, n * page).astype(np.int32)
        if step % 3 == 2:
            s, d = rng.permutation(B)[:2]
            k[0, :, 0, :, 0] = rng.integers(0, 60000, (pool, page))
            k2, _, table, n, ref, length = op.pages_fork(k, k, table, n, ref, [s], [d], length)
            _consistent(table, n, ref)
            if length[d] > 0:
                assert length[d] == length[s]
                a = op.gather(k2[0], table[s], length[s])
                assert np.array_equal(a, op.gather(k2[0], table[d], length[s]))
                own = length[s] // page
                assert n[d] == own or ref[table[d, own]] == 1        # the page the sequence goes on in is its own
    assert ref.max() > 1                                             # pages were shared


def test_resize_serves_no_row_whose_count_is_impossible():
    table = np.array([[33, 33], [0, -1], [33, 33], [33, 33]], dtype=np.int32)
    n = np.array([-2 ** 31, 1, -2, 3], dtype=np.int32)
    ref = np.array([1, 0, 0, 0], dtype=np.int32)
    t2, n2, r2, short = op.pages_resize(table, n, ref, np.array([32, 32, 32, 32]), 16)
    assert not short and t2.tolist() == [[33, 33], [0, 1], [33, 33], [33, 33]]
    assert n2.tolist() == [-2 ** 31, 2, -2, 3] and r2.tolist() == [1, 1, 0, 0]
