"""Refusals of the paged calls (CPU only): wrong types, shapes, devices and
sizes stop in Python or in the C ABI's checks, before anything is launched."""
import ctypes

import pytest

import medusa_draft_heads_b200 as md
from medusa_draft_heads_b200 import binding
from medusa_draft_heads_b200.step import PagedMedusaStep
from seeded_inputs.workloads import TREE_ACCEPT

torch = pytest.importorskip("torch")

B, T, Hq, Hkv, dh, page, pages, width = 2, 17, 4, 2, 64, 16, 8, 3


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.fixture(scope="module")
def tree():
    return md.Tree(*md.tree_arrays(md.select_tree((4, 3, 2, 2), TREE_ACCEPT, 16)), (4, 3, 2, 2))


def _attention(tree, **kw):
    a = dict(q=bf(B, T, Hq, dh), k_pages=bf(pages, Hkv, page, dh), v_pages=bf(pages, Hkv, page, dh),
             block_table=i32(B, width), prefix_len=i32(B), tree=tree, out=torch.zeros(B, T, Hq, dh),
             ws=torch.zeros(256, dtype=torch.uint8))
    a.update(kw)
    md.tree_attention_paged(**a)


@pytest.mark.parametrize("kw,error,match", [
    (dict(q=bf(B, T, Hq)), ValueError, "q: expected 4 dims"),
    (dict(q=None), TypeError, "q: expected a torch.Tensor"),
    (dict(q=bf(B, T + 1, Hq, dh)), ValueError, "T has shape"),
    (dict(q=torch.zeros(B, T, Hq, dh)), TypeError, "q: expected torch.bfloat16"),
    (dict(k_pages=bf(1, pages, Hkv, page, dh)), ValueError, "k_pages: expected 4 dims"),
    (dict(k_pages=bf(pages, Hkv, page, 2 * dh)), ValueError, "k_pages has shape"),
    (dict(v_pages=bf(pages + 1, Hkv, page, dh)), ValueError, "v_pages has shape"),
    (dict(block_table=i32(B + 1, width)), ValueError, "block_table has shape"),
    (dict(block_table=torch.zeros((B, width), dtype=torch.int64)), TypeError, "block_table: expected torch.int32"),
    (dict(out=torch.zeros(B, T, Hq, dh, dtype=torch.float16)), TypeError, "out: expected torch.float32 or torch.bfloat16"),
    (dict(out=torch.zeros(B, T, dh, Hq)), ValueError, "out has shape"),
    (dict(), ValueError, "q: must be a CUDA tensor"),
])
def test_attention_arguments(tree, kw, error, match):
    with pytest.raises(error, match=match):
        _attention(tree, **kw)


def test_pointer_check_names_what_is_wrong():
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        binding._ptrs("x", -1, (i32(3), "a", torch.int32, (3,)))
    with pytest.raises(ValueError, match="a has shape"):
        binding._ptrs("x", 0, (i32(3), "a", torch.int32, (4,)))
    with pytest.raises(TypeError, match="expected a torch.Tensor"):
        binding._ptrs("x", 0, ([1, 2], "a", torch.int32, (2,)))


def test_append_views():
    qkv = bf(B, T, Hq + 2 * Hkv, dh)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=2)
    args = dict(pos=i32(B, T), inv_freq=torch.zeros(dh // 2), q_out=bf(B, T, Hq, dh), k_pages=bf(pages, Hkv, page, dh),
                v_pages=bf(pages, Hkv, page, dh), block_table=i32(B, width), prefix_len=i32(B))
    with pytest.raises(ValueError, match="q: must be a CUDA tensor"):
        md.qk_rope_append(q, k, v, **args)
    with pytest.raises(TypeError, match="q: expected torch.bfloat16"):
        md.qk_rope_append(q.float(), k, v, **args)
    with pytest.raises(ValueError, match="k: expected 4 dims"):
        md.qk_rope_append(q, k[0], v, **args)
    with pytest.raises(ValueError, match="inv_freq: expected 1 dims"):
        md.qk_rope_append(q, k, v, **dict(args, inv_freq=torch.zeros(1, dh // 2)))


def test_page_calls_arguments():
    with pytest.raises(ValueError, match="block_table: expected 2 dims"):
        md.pages_resize(i32(B), i32(B), i32(pages), i32(B), page)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        md.pages_resize(i32(B, width), i32(B), i32(pages), i32(B), page)
    for bad in (dict(page_size=0), dict(page_size=2 ** 32 + 16), dict(page_size=16, extra=-1), dict(page_size=16, extra=2 ** 31)):
        with pytest.raises(ValueError, match="out of range"):
            md.pages_resize(i32(B, width), i32(B), i32(pages), i32(B), **bad)
    with pytest.raises(ValueError, match="k_pages: expected 4 or 5 dims"):
        md.pages_fork(bf(page, dh), bf(page, dh), i32(B, width), i32(B), i32(pages), i32(1), i32(1), i32(B),
                      torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="path: expected 2 dims"):
        md.tree_commit_paged(bf(pages, Hkv, page, dh), bf(pages, Hkv, page, dh), i32(B, width), None, i32(B), i32(B), i32(B),
                             i32(B), i32(B), i32(B), i32(B))


def test_c_checks_come_before_any_launch(tree):
    """Sizes and pointers the C ABI refuses: pointers are never followed."""
    L = md.lib()
    n = ctypes.c_size_t()
    ws = lambda *a: L.md_attention_paged_workspace(*a, ctypes.byref(n))     # noqa: E731
    assert ws(1, 17, 4, 2, 64, 16, 8) == 0 and n.value > 0
    assert ws(0, 17, 4, 2, 64, 16, 8) == -1 and ws(1, 17, 4, 2, 64, 0, 8) == -1
    for bad in ((1, 129, 4, 2, 64, 16, 8), (1, 17, 5, 2, 64, 16, 8), (1, 17, 34, 2, 64, 16, 8), (1, 17, 4, 2, 96, 16, 8),
                (1, 17, 4, 2, 64, 24, 8), (65536, 17, 4, 2, 64, 16, 8), (1, 17, 4, 2, 64, 16, 1 << 27),
                (60000, 17, 4, 2, 64, 16, 40000), (1, 17, 4096, 4096, 64, 16, 8)):
        assert ws(*bad) == -2, bad
    p = 1 << 20

    def attention(q=p, k=p, tb=p, pool=8, ps=16, w=8, scale=0.0, out=p + 4096, kind=0, wsp=p, wsn=4096):
        return L.md_tree_attention_paged(q, k, p, pool, ps, tb, w, p, tree.handle, 2, 4, 2, 64, scale, out, kind, wsp, wsn, None)

    assert attention(q=None) == -1 and attention(tb=None) == -1 and attention(out=None) == -1
    assert attention(q=p + 2) == -1 and attention(k=p + 8) == -1 and attention(out=p + 4) == -1
    assert attention(q=p, out=p) == -1                 # results over the queries that other CTAs still read
    assert attention(scale=-1.0) == -1 and attention(scale=float("nan")) == -1 and attention(kind=2) == -1
    assert attention(pool=0) == -1 and attention(pool=1 << 30) == -2
    assert attention(wsp=None) == -4 and attention(wsn=8) == -4 and attention(wsp=p + 16) == -4

    strides = lambda *s: (ctypes.c_int64 * 9)(*s)      # noqa: E731
    ok = (4096, 512, 64) * 3

    def append(st=ok, rot=64, eps=1e-6, q=p, T_=4, d=64, hq=4, ps=7):
        return L.md_qk_rope_append(q, p, p, strides(*st), p, p, rot, 0, None, None, eps, p, p, p, 8, ps, p, 8, p, None, 2, T_, hq, 2,
                                   d, None)

    assert append(q=None) == -1 and append(q=p + 8) == -1 and append(st=(4,) + ok[1:]) == -1
    assert append(eps=-1.0) == -1 and append(eps=float("inf")) == -1 and append(T_=0) == -1 and append(ps=0) == -1
    assert append(rot=8) == -2 and append(rot=72) == -2 and append(rot=80) == -2 and append(d=80) == -2
    assert append(T_=1 << 30) == -2 and append(hq=65536) == -2

    def commit(k=p, newp=p, K=4, layers=1, d=64):
        return L.md_tree_commit_paged(k, p, layers, 8, 16, p, 8, 2, d, tree.handle, 2, p + 64, p, p, K, p, newp, p, p, None)

    assert commit(k=None) == -1 and commit(newp=p + 64) == -1 and commit(K=3) == -1 and commit(K=9) == -1
    assert commit(layers=0) == -1 and commit(d=32) == -2 and commit(k=p + 2) == -1

    def resize(tb=p, ref=p, b=2, extra=0, ps=16, pool=8):
        return L.md_pages_resize(tb, p, ref, p, b, 8, pool, ps, extra, None)

    assert resize(tb=None) == -1 and resize(ref=p + 4) == -1 and resize(extra=-1) == -1 and resize(ps=0) == -1
    assert resize(b=16385) == -2 and resize(b=0) == -1 and resize(pool=0) == -1

    assert L.md_pages_fork_workspace(2, 1024, ctypes.byref(n)) == 0 and n.value >= 1024 * 16
    assert L.md_pages_fork_workspace(2, 1025, ctypes.byref(n)) == -2
    assert L.md_pages_fork_workspace(2, 0, ctypes.byref(n)) == -1

    def fork(k=p, layers=1, n_=2, wsp=p, wsn=4096, d=64, ref=p):
        return L.md_pages_fork(k, p, layers, 8, 2, 16, d, p, p, ref, p, 2, 8, p, p, n_, wsp, wsn, None)

    assert fork(k=None) == -1 and fork(layers=0) == -1 and fork(n_=0) == -1 and fork(ref=p + 8) == -1
    assert fork(n_=1025) == -2 and fork(d=80) == -2 and fork(wsp=None) == -4 and fork(wsn=16) == -4


def test_paged_step_is_a_medusa_step():
    from medusa_draft_heads_b200.step import MedusaStep
    assert issubclass(PagedMedusaStep, MedusaStep)
    for name in ("prefill_pages", "reserve", "append", "attention", "commit", "trim", "fork"):
        assert callable(getattr(PagedMedusaStep, name))


def test_fork_workspace_stays_where_it_is(monkeypatch):
    """A graph that captured a fork keeps the workspace's address: calls of any size use the same one."""
    from medusa_draft_heads_b200 import step as step_module
    seen = []

    def fork(kp, vp, table, n_pages, refcount, src, dst, length, ws, stream=None):
        assert ws.numel() >= md.pages_fork_workspace_bytes(B, src.shape[0])
        seen.append((ws.data_ptr(), ws.numel()))

    monkeypatch.setattr(step_module, "pages_fork", fork)
    step = PagedMedusaStep(B=B, M=B, d=256, V=2048, K=4, k_per_head=(4, 3, 2, 2), Hq=Hq, Hkv=Hkv, dh=dh, page_size=page,
                           tree_tuples=md.select_tree((4, 3, 2, 2), TREE_ACCEPT, 16), max_pages=width, pool_pages=pages,
                           device="cpu")
    pool = bf(1, pages, Hkv, page, dh)
    for n in (1, 16, 17, 1, 1024):
        step.fork(pool, pool, i32(n), i32(n), i32(B))
    assert len(set(seen)) == 1


def test_fork_refuses_pages_it_cannot_count():
    """Of a page of 2^27 slots of 128 the copy's 32-bit count of 16-byte pieces would overflow."""
    p = 1 << 20

    def fork(page_size, d):
        return md.lib().md_pages_fork(p, p, 1, 2, 1, page_size, d, p, p, p, p, 2, 1, p, p, 1, None, 0, None)

    assert fork(1 << 27, 128) == -2 and fork((1 << 27) - 1, 128) == -2 and fork(1 << 28, 64) == -2
    assert fork((1 << 27) - 65, 128) == -4 and fork(1 << 27, 64) == -4      # taken, but for the missing workspace
