"""One Medusa draft-and-verify step through the C ABI.

Owns the output buffers and workspaces of the four calls and issues them in
order on one stream: heads + top-k -> tree build -> tree attention (one layer
of the verification pass) -> acceptance. No arithmetic happens here.
"""
from __future__ import annotations

import torch

from .binding import (Tree, accept_workspace_bytes, attention_paged_workspace_bytes, attention_workspace_bytes,
                      heads_shared_workspace_bytes, heads_workspace_bytes, medusa_heads, medusa_heads_sampled,
                      medusa_heads_shared, pages_fork, pages_fork_workspace_bytes, pages_resize, qk_rope_append,
                      tree_accept, tree_accept_rejection, tree_accept_sampled, tree_attention, tree_attention_paged,
                      tree_build, tree_commit, tree_commit_paged, workspace)
from .tree_spec import tree_arrays


class MedusaStep:
    def __init__(self, *, B, M, d, V, K, k_per_head, tree_tuples, Hq, Hkv, dh, S_max, mode="greedy",
                 temperature=0.7, eps=0.09, alpha=0.3, device="cuda", keep_logits=False, shared_vocab=False):
        parent, rank = tree_arrays(tree_tuples)
        self.tree = Tree(parent, rank, k_per_head)
        self.B, self.M, self.d, self.V, self.K = B, M, d, V, K
        self.k_per_head = list(k_per_head)
        self.kmax = max(k_per_head)
        self.T = self.tree.T
        self.Hq, self.Hkv, self.dh, self.S_max = Hq, Hkv, dh, S_max
        self.mode, self.temperature, self.eps, self.alpha = mode, temperature, eps, alpha
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        self.topk_ids = torch.empty((M, K, self.kmax), **i32)
        self.topk_vals = torch.empty((M, K, self.kmax), **f32)
        # mode "rejection": candidates drawn from the heads' distributions, whose
        # logits the lossless acceptance reads, so they are always kept
        keep_logits = keep_logits or mode == "rejection"
        self.logits_dbg = torch.empty((M, K, V), **f32) if keep_logits else None
        self.tokens = torch.empty((B, self.T), **i32)
        self.parent = torch.empty((self.T,), **i32)
        self.anc = torch.empty((self.T, (self.T + 31) // 32), **i32)
        self.pos = torch.empty((B, self.T), **i32)
        self.attn_out = torch.empty((B, self.T, Hq, dh), **f32)
        # the step's result in one buffer (accept_len [B], path [B, K+1],
        # bonus [B]), so a caller reads it back with one copy
        self.result = torch.empty((B * (K + 3),), **i32)
        self.accept_len = self.result[:B]
        self.path = self.result[B:B * (K + 2)].view(B, K + 1)
        self.bonus = self.result[B * (K + 2):]
        self.new_prefix_len = torch.empty((B,), **i32)
        self.next_root = torch.empty((B,), **i32)
        self.next_head_row = torch.empty((B,), **i32)
        self.shared_vocab = shared_vocab
        # mode "sample": one uniform in [0, 1) per tree row, supplied by the caller
        self.uniforms = torch.full((B, self.T), 0.5, **f32) if mode == "sample" else None
        # mode "rejection": uniforms for the draws [M, K, V] and for the tests
        # and bonus draws [B, T] each; the caller refills them every step
        self.u_draft = torch.full((M, K, V), 0.5, **f32) if mode == "rejection" else None
        self.u_accept = torch.full((B, self.T), 0.5, **f32) if mode == "rejection" else None
        self.u_residual = torch.full((B, self.T), 0.5, **f32) if mode == "rejection" else None
        self.head_row = None
        ws_fn = heads_shared_workspace_bytes if shared_vocab else heads_workspace_bytes
        self.ws_heads = workspace(ws_fn(M, d, V, K, self.kmax), dev)
        self.ws_attn = workspace(self._attention_workspace_bytes(), dev)
        self.ws_acc = workspace(accept_workspace_bytes(B, self.T, V), dev)

    def _attention_workspace_bytes(self):
        return attention_workspace_bytes(self.B, self.T, self.Hq, self.Hkv, self.dh, self.S_max)

    def heads(self, h, W1, b1, Wv, stream=None):
        if self.mode == "rejection":
            medusa_heads_sampled(h, W1, b1, Wv, self.k_per_head, self.u_draft, self.topk_ids, self.topk_vals,
                                 self.logits_dbg, self.ws_heads, temperature=self.temperature, stream=stream)
            return
        fn = medusa_heads_shared if self.shared_vocab else medusa_heads
        fn(h, W1, b1, Wv, self.k_per_head, self.topk_ids, self.topk_vals, self.ws_heads,
           logits_dbg=self.logits_dbg, stream=stream)

    def build(self, root_token, prefix_len, head_row=None, stream=None):
        self.head_row = head_row
        tree_build(self.tree, self.topk_ids, root_token, prefix_len, self.tokens, self.parent, self.anc,
                   self.pos, head_row=head_row, stream=stream)

    def attention(self, q, k_cache, v_cache, prefix_len, stream=None):
        tree_attention(q, k_cache, v_cache, prefix_len, self.tree, self.attn_out, self.ws_attn, stream=stream)

    def accept(self, logits, stream=None, uniforms=None):
        """Greedy / typical acceptance, (mode "sample") the lossless sampled
        rule with one uniform per tree row ([B, T] fp32: `uniforms`, else the
        step's own `self.uniforms`, which the caller refills each step), or
        (mode "rejection") lossless acceptance of drafts sampled from the heads."""
        if self.mode == "rejection":
            tree_accept_rejection(logits, self.tokens, self.tree, self.logits_dbg, self.u_accept, self.u_residual,
                                  self.accept_len, self.path, self.bonus, temperature=self.temperature,
                                  temperature_q=self.temperature, head_row=self.head_row, stream=stream)
            return
        if self.mode == "sample":
            u = self.uniforms if uniforms is None else uniforms
            tree_accept_sampled(logits, self.tokens, self.tree, u, self.accept_len, self.path, self.bonus,
                                self.ws_acc, temperature=self.temperature, stream=stream)
            return
        tree_accept(logits, self.tokens, self.tree, self.accept_len, self.path, self.bonus, self.ws_acc,
                    mode=self.mode, temperature=self.temperature, eps=self.eps, alpha=self.alpha, stream=stream)

    def commit(self, k_cache, v_cache, prefix_len, stream=None):
        tree_commit(k_cache, v_cache, self.tree, prefix_len, self.accept_len, self.path, self.bonus,
                    self.new_prefix_len, self.next_root, self.next_head_row, stream=stream)

    def run(self, h, W1, b1, Wv, root_token, prefix_len, q, k_cache, v_cache, logits, head_row=None,
            stream=None):
        self.heads(h, W1, b1, Wv, stream)
        self.build(root_token, prefix_len, head_row, stream)
        self.attention(q, k_cache, v_cache, prefix_len, stream)
        self.accept(logits, stream)


MAX_FORKS = 1024   # entries of one pages_fork call


class PagedMedusaStep(MedusaStep):
    """The step over a KV cache held in pages.

    The caller owns the pools ([layers, pool_pages, Hkv, page_size, dh] bf16, K
    and V); this object owns which request holds which page (`block_table`,
    `n_pages`, `refcount`, all on the device) and the rotated queries `q` of the
    layer at hand. A request is a row of the batch; prefix_len[b] = -1 marks a
    row that holds none, so rows come and go without a change of shapes:

        step.prefill_pages(length)                     # a new request's pages
        step.append(q, k, v, pos, inv_freq, k_pages[i], v_pages[i], prefix_len, n_new=n)     # its prompt, layer i
        step.heads(...); step.build(root_token, prefix_len)
        step.reserve(prefix_len)                       # pages for the tree's T slots
        step.append(q, k, v, step.pos, inv_freq, k_pages[i], v_pages[i], prefix_len)         # every layer i
        step.attention(step.q, k_pages[i], v_pages[i], prefix_len)
        step.accept(logits); step.commit(k_pages, v_pages, prefix_len)                       # all layers at once
        step.trim()                                    # pages past the new prefixes go back
        prefix_len.copy_(step.new_prefix_len)          # and step.next_root, step.next_head_row as they are

    A row whose commit was refused (next_head_row -1 where prefix_len is not: it had no
    pages, or its path was none) keeps its prefix; its root token is still tokens[b, 0].
    out_dtype: of the attention's results; bfloat16 halves its time over long prefixes
    and takes 8 bits of the softmax weights instead of 24.
    """

    def __init__(self, *, page_size, max_pages, pool_pages, out_dtype=torch.float32, **kw):
        self.page_size, self.max_pages = page_size, max_pages
        super().__init__(S_max=page_size * max_pages, **kw)
        dev = self.tokens.device
        i32 = dict(dtype=torch.int32, device=dev)
        self.block_table = torch.full((self.B, max_pages), -1, **i32)
        self.n_pages = torch.zeros((self.B,), **i32)
        self.refcount = torch.zeros((pool_pages,), **i32)
        self.attn_out = torch.empty((self.B, self.T, self.Hq, self.dh), dtype=out_dtype, device=dev)
        self.q = torch.empty((self.B, self.T, self.Hq, self.dh), dtype=torch.bfloat16, device=dev)
        # for the largest call, and never replaced: a captured graph keeps its address
        self.ws_fork = workspace(pages_fork_workspace_bytes(self.B, MAX_FORKS), dev)

    def _attention_workspace_bytes(self):
        return attention_paged_workspace_bytes(self.B, self.T, self.Hq, self.Hkv, self.dh, self.page_size, self.max_pages)

    def prefill_pages(self, length, stream=None):
        """Every row holds exactly the pages of length[b] slots (-1: none)."""
        pages_resize(self.block_table, self.n_pages, self.refcount, length, self.page_size, stream=stream)

    def reserve(self, prefix_len, stream=None):
        """Pages for the prefix and the tree behind it."""
        pages_resize(self.block_table, self.n_pages, self.refcount, prefix_len, self.page_size, extra=self.T,
                     stream=stream)

    def trim(self, stream=None):
        """After commit: the pages past the new prefixes go back."""
        self.prefill_pages(self.new_prefix_len, stream)

    def append(self, q, k, v, pos, inv_freq, k_pages, v_pages, prefix_len, q_norm=None, k_norm=None, eps=1e-6,
               interleaved=False, n_new=None, q_out=None, stream=None):
        """Norms, rotation and cache write of one layer's new tokens; the queries
        go to q_out (default: `self.q`, a tree's)."""
        qk_rope_append(q, k, v, pos, inv_freq, self.q if q_out is None else q_out, k_pages, v_pages, self.block_table,
                       prefix_len, q_norm=q_norm, k_norm=k_norm, eps=eps, interleaved=interleaved, n_new=n_new,
                       stream=stream)

    def attention(self, q, k_pages, v_pages, prefix_len, stream=None):
        tree_attention_paged(q, k_pages, v_pages, self.block_table, prefix_len, self.tree, self.attn_out, self.ws_attn,
                             stream=stream)

    def commit(self, k_pages, v_pages, prefix_len, stream=None):
        tree_commit_paged(k_pages, v_pages, self.block_table, self.tree, prefix_len, self.accept_len, self.path,
                          self.bonus, self.new_prefix_len, self.next_root, self.next_head_row, stream=stream)

    def fork(self, k_pages, v_pages, src, dst, prefix_len, stream=None):
        """Rows dst continue the sequences of rows src; prefix_len[dst] is set. At most
        MAX_FORKS entries a call."""
        pages_fork(k_pages, v_pages, self.block_table, self.n_pages, self.refcount, src, dst, prefix_len, self.ws_fork,
                   stream=stream)
