"""One chunk of the FAST-AR attention path on preallocated device buffers.

The order follows the method: hash the chunk's queries, its new keys and
the prompt keys once (FAST-AR analysis, paper.rainbus.top: the encoding is
computed once and serves all three modules); merge the new frames into the
TempCache; prune the prompt per frame (AnnCA); cross-attend; then
self-attend over the merged cache with the bucket restriction (AnnSA).
Every step is one C-ABI call; this class only owns the buffers.
"""
from __future__ import annotations

import ctypes
import functools
from types import SimpleNamespace

import torch

from . import (Cache, OP_ANNCA, OP_ANNSA, OP_ANNSA_PARTS, OP_MERGE, PagedKV, PageMass, Prefix, _stream, branch_workspace_size,
               fastar_annca_attention, fastar_annca_prune, fastar_annsa_attention, fastar_annsa_attention_part,
               fastar_annsa_combine, fastar_branch_attention, fastar_bucket_csr, fastar_hash, fastar_hash_many,
               fastar_page_append, fastar_page_evict, fastar_page_keep, fastar_page_mass, fastar_tempcache_merge,
               fastar_tree_attention, fastar_workspace_size, mass_workspace_size)

DENSE_FRAC = 0.3  # sparse attention is off for this share of a chunk's denoising steps


class ChunkPath:
    """Buffers and calls of one layer's per-chunk path."""

    def __init__(self, H, D, n_f, F, P, T, B, C, tau, dtype=torch.bfloat16, device="cuda", rep="last",
                 share=None, search="prev"):
        """rep: TempCache representative, "last" (the method) or "mean";
        search: where a new key's group is looked for, "prev" (the previous
        frame's groups, the method) or "lsh" (every earlier group sharing an
        LSH bucket);
        share: another ChunkPath of the same shapes whose workspaces and
        streams this one reuses (layers run one after the other on the same
        streams, so their scratch never overlaps in time); caches, codes,
        outputs and events stay per layer."""
        self.H, self.D, self.n_f, self.F, self.P = H, D, n_f, F, P
        self.rep = rep  # TempCache representative: "last" (the method) or "mean" (ablation)
        self.search = search
        self.T, self.B, self.C, self.tau, self.dtype = T, B, C, tau, dtype
        self.Nq = F * n_f
        self.scale = D ** -0.5
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.cache = Cache(H, C, D, T, B, dtype, dev)
        self.planes = torch.zeros(T * B, D, dtype=dtype, device=dev)
        Nq = self.Nq
        self.q_codes = torch.zeros(H, T, Nq, **i32)
        self.q_perm = torch.zeros(H, T, Nq, **i32)
        self.q_offsets = torch.zeros(H, T, (1 << B) + 1, **i32)
        self.k_codes = torch.zeros(H, T, Nq, **i32)
        self.p_codes = torch.zeros(H, T, max(P, 1), **i32)
        self.kept_idx = torch.zeros(H, F, max(P, 1), **i32)
        self.kept_cnt = torch.zeros(H, F, **i32)
        self.match = torch.zeros(H, Nq, **i32)
        self.o_ca = torch.zeros(H, Nq, D, dtype=dtype, device=dev)
        self.o_sa = torch.zeros(H, Nq, D, dtype=dtype, device=dev)
        self.lse = torch.zeros(H, Nq, dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, **i32)
        if share is not None:
            if (share.H, share.D, share.n_f, share.F, share.P, share.T, share.B, share.C) != \
                    (H, D, n_f, F, P, T, B, C):
                raise ValueError("a shared path must have the same shapes")
            self.ws_merge, self.ws_annsa, self.ws_annca = share.ws_merge, share.ws_annsa, share.ws_annca
            self._side, self._copy_in, self._copy_out = share._side, share._copy_in, share._copy_out
        else:
            self.ws_merge = torch.empty(max(1, fastar_workspace_size(OP_MERGE, H, n_f, D, T, B, C)),
                                        dtype=torch.uint8, device=dev)
            self.ws_annsa = torch.empty(max(1, fastar_workspace_size(OP_ANNSA, H, Nq, D, T, B, C)),
                                        dtype=torch.uint8, device=dev)
            self.ws_annca = torch.empty(max(1, fastar_workspace_size(OP_ANNCA, H, F, D, T, B, P)),
                                        dtype=torch.uint8, device=dev)
            # the second stream (query CSR, cross-attention branch)
            self._side = torch.cuda.Stream(device=dev)
            # host-to-host chunks: the streams that copy inputs in and outputs out
            self._copy_in = torch.cuda.Stream(device=dev)
            self._copy_out = torch.cuda.Stream(device=dev)
        # the events that fork and join the second stream
        self._fork = torch.cuda.Event()
        self._codes_ready = torch.cuda.Event()
        self._csr_done = torch.cuda.Event()
        # host-to-host chunks: device copies of the inputs and the events
        # that release each branch and each output
        self._dev_in = None
        self._in_k = torch.cuda.Event()
        self._in_v = torch.cuda.Event()
        self._in_qp = torch.cuda.Event()
        self._in_vp = torch.cuda.Event()
        self._cross_done = torch.cuda.Event()
        self._ca_done = torch.cuda.Event()
        self._sa_done = torch.cuda.Event()
        self._out_done = torch.cuda.Event()

    # -- pieces -----------------------------------------------------------
    def merge(self, k, v, first_frame, F=None, stream=None):
        """Hash new keys k [H][F*n_f][D] and merge them (cache building).

        Returns (codes [H][T][F*n_f], match [H][F*n_f]) of this call.
        """
        F = self.F if F is None else F
        n = F * self.n_f
        if F == self.F:
            codes, match = self.k_codes, self.match
        else:
            codes = torch.empty(self.H, self.T, n, dtype=torch.int32, device=k.device)
            match = torch.empty(self.H, n, dtype=torch.int32, device=k.device)
        fastar_hash(k, self.planes, self.T, self.B, codes, status=self.status, stream=stream)
        fastar_tempcache_merge(self.cache, k, v, codes, F, self.n_f, first_frame, self.tau,
                               match_out=match, ws=self.ws_merge, status=self.status,
                               stream=stream, rep=self.rep, planes=self.planes,
                               search=self.search)
        return codes, match

    def step(self, q, k, v, kp, vp, first_frame, stream=None):
        """The whole path for one chunk: q, k, v [H][F*n_f][D]; kp, vp [H][P][D].

        The second stream hashes the chunk while the merge starts (its first
        NN search and plan need only the keys and the cache; it waits for
        the key codes before its first apply), then builds the query CSR and
        runs the cross-attention branch (prune, AnnCA), which needs the codes
        but not the merged cache; AnnSA waits for the CSR, and `stream`
        (default: the current stream) waits for both branches before this
        returns, so later work on it sees every output."""
        self._run(q, k, v, kp, vp, first_frame, self._main(stream))

    def step_host(self, hq, hk, hv, hkp, hvp, ho_ca, ho_sa, first_frame, stream=None, dev_in=None,
                  join=True):
        """The chunk from host memory to host memory (pinned tensors, same
        shapes as step's; ho_ca, ho_sa receive o_ca and o_sa).

        The inputs are copied in on one copy stream in the order the
        branches need them (k and v for the merge branch, then q, the prompt
        keys and the prompt values for the cross-attention branch, which
        also builds the query CSR that AnnSA needs; one host-to-device stream
        beside the device-to-host one moves more in total than two), each
        branch hashes and starts as soon as its inputs have landed, and each
        output is copied out on a second stream as soon as it is final.  The copies into this
        path's device buffers (dev_in: (q, k, v, kp, vp) tensors to use; by
        default buffers of its own) wait only for the previous chunk of this
        path to have read them, so with several paths (layers) the copies of
        one run ahead of the kernels of another.  With join (the default)
        `stream` (default: the current stream) waits for all of it, so the
        host buffers are complete once it has synchronised; without, call
        join_outputs before reading them."""
        main = self._main(stream)
        dev = self.q_codes.device
        if dev_in is not None:
            self._dev_in = list(dev_in)
        elif self._dev_in is None or self._dev_in[0].shape != hq.shape or self._dev_in[3].shape != hkp.shape:
            self._dev_in = [torch.empty(x.shape, dtype=x.dtype, device=dev) for x in (hq, hk, hv, hkp, hvp)]
        dq, dk, dv, dkp, dvp = self._dev_in
        # the device inputs and outputs are free once this path's previous
        # chunk has finished and its outputs have been copied out (never
        # recorded before the first chunk); every stream of this chunk waits
        # for that through the copies it depends on
        ci = self._copy_in
        ci.wait_event(self._out_done)
        with torch.cuda.stream(ci):
            dk.copy_(hk, non_blocking=True)
            self._in_k.record(ci)
            dv.copy_(hv, non_blocking=True)
            self._in_v.record(ci)
            dq.copy_(hq, non_blocking=True)
            dkp.copy_(hkp, non_blocking=True)
            self._in_qp.record(ci)
            dvp.copy_(hvp, non_blocking=True)
            self._in_vp.record(ci)
        main.wait_event(self._out_done)
        self._run(dq, dk, dv, dkp, dvp, first_frame, main, host_out=(ho_ca, ho_sa))
        co = self._copy_out
        co.wait_event(self._ca_done)
        with torch.cuda.stream(co):
            ho_ca.copy_(self.o_ca, non_blocking=True)
        co.wait_event(self._sa_done)
        with torch.cuda.stream(co):
            ho_sa.copy_(self.o_sa, non_blocking=True)
        self._out_done.record(co)
        if join:
            self.join_outputs(main)

    def join_outputs(self, stream=None):
        """Make `stream` (default: the current stream) wait until the host
        outputs of this path's last step_host are complete."""
        self._main(stream).wait_event(self._out_done)

    # -- denoising steps -----------------------------------------------------
    def denoise_step(self, s, S, q, k, v, kp, vp, first_frame, dense_frac=DENSE_FRAC, reuse=False):
        """Step s of the S denoising steps of a chunk (FAST-AR analysis,
        paper.rainbus.top: sparse attention is off for the first 30 % of the
        steps; each chunk is denoised conditioned on the history).

        Step s is dense iff s < dense_frac * S.  A step before the last
        attends the cache together with its own keys (count 1; the cache is
        not written): two partial AnnSA calls, one over the cache and one
        over a cache description of the step's keys, merged exactly by
        fastar_annsa_combine; dense steps give both key sets one table of one
        bit with every code 0, and keep every prompt token.  The last step
        merges its keys into the cache and attends the merged cache, as
        `step` does (dense per the schedule).  Outputs: o_sa, lse, o_ca.

        reuse: the codes (queries, the step's keys, the prompt), the query
        CSR and the kept prompt lists are computed at the chunk's first
        sparse step only and reused by its later sparse steps; the last step
        still hashes its keys, whose codes the merge stores with them."""
        dense = s < dense_frac * S
        first_sparse = not dense and (s == 0 or (s - 1) < dense_frac * S)
        reuse_now = reuse and not dense and not first_sparse
        dn = self._denoise_views()
        st = self.status
        if s + 1 == S and not dense:
            if not reuse_now:
                self.step(q, k, v, kp, vp, first_frame)
                return
            fastar_hash(k, self.planes, self.T, self.B, self.k_codes, status=st)
            fastar_tempcache_merge(self.cache, k, v, self.k_codes, self.F, self.n_f, first_frame, self.tau,
                                   match_out=self.match, ws=self.ws_merge, status=st, rep=self.rep,
                                   planes=self.planes, search=self.search)
            fastar_annsa_attention(q, self.q_codes, self.q_perm, self.q_offsets, self.cache, self.scale, self.o_sa,
                                   self.lse, ws=self.ws_annsa, status=st)
            fastar_annca_attention(q, kp, vp, self.kept_idx, self.kept_cnt, self.F, self.n_f, self.scale,
                                   self.o_ca, ws=self.ws_annca, status=st)
            return
        if s + 1 == S:
            fastar_hash(k, self.planes, self.T, self.B, self.k_codes, status=st)
            fastar_tempcache_merge(self.cache, k, v, self.k_codes, self.F, self.n_f, first_frame, self.tau,
                                   match_out=self.match, ws=self.ws_merge, status=st, rep=self.rep,
                                   planes=self.planes)
            fastar_annsa_attention_part(q, dn.qc0, dn.qp0, dn.qo0, dn.cache_dense, self.scale, 0, 1, dn.ws,
                                        status=st)
            fastar_annsa_combine(1, dn.ws, self.o_sa, self.lse, status=st)
        elif dense:
            chunk = self._chunk_view(k, v, dense=True)
            fastar_annsa_attention_part(q, dn.qc0, dn.qp0, dn.qo0, dn.cache_dense, self.scale, 0, 2, dn.ws,
                                        status=st)
            fastar_annsa_attention_part(q, dn.qc0, dn.qp0, dn.qo0, chunk, self.scale, 1, 2, dn.ws, status=st)
            fastar_annsa_combine(2, dn.ws, self.o_sa, self.lse, status=st)
        else:
            T = self.T
            jobs = [(q, self.q_codes, self.q_perm, self.q_offsets), (k, self.k_codes, dn.k_perm, dn.k_off)]
            if self.P:
                jobs.append((kp, self.p_codes, None, None))
            if not reuse_now:
                fastar_hash_many(jobs, self.planes, T, self.B, status=st)
            chunk = self._chunk_view(k, v, dense=False)
            fastar_annsa_attention_part(q, self.q_codes, self.q_perm, self.q_offsets, self.cache, self.scale, 0,
                                        2 * T, dn.ws, status=st)
            fastar_annsa_attention_part(q, self.q_codes, self.q_perm, self.q_offsets, chunk, self.scale, T,
                                        2 * T, dn.ws, status=st)
            fastar_annsa_combine(2 * T, dn.ws, self.o_sa, self.lse, status=st)
        if dense:
            kept, cnt = dn.kept_all, dn.cnt_all
        elif reuse_now:
            kept, cnt = self.kept_idx, self.kept_cnt
        else:
            fastar_annca_prune(self.q_codes, self.p_codes[:, :, :self.P], self.F, self.n_f, self.B,
                               self.kept_idx, self.kept_cnt, status=st)
            kept, cnt = self.kept_idx, self.kept_cnt
        fastar_annca_attention(q, kp, vp, kept, cnt, self.F, self.n_f, self.scale, self.o_ca, ws=self.ws_annca,
                               status=st)

    def _chunk_view(self, k, v, dense):
        dn = self._denoise_views()
        if dense:
            return Cache.view(1, 1, K=k, V=v, m=dn.ones, codes=dn.qc0, last_frame=dn.lf, size=dn.nq,
                              inserted=dn.cnt64, evicted=dn.cnt64, perm=dn.qp0, offsets=dn.qo0)
        return Cache.view(self.T, self.B, K=k, V=v, m=dn.ones, codes=self.k_codes, last_frame=dn.lf,
                          size=dn.nq, inserted=dn.cnt64, evicted=dn.cnt64, perm=dn.k_perm, offsets=dn.k_off)

    def _denoise_views(self):
        """Buffers of the denoising steps, built once: one-bucket (dense)
        views of the queries, of the cache and of a step's keys (codes 0; the
        CSR kernel turns them into an identity order and offsets (0, N, N)),
        every prompt token kept (the prune of all-zero codes), and a step's
        keys described as a cache (m = 1, size = Nq, their own CSR)."""
        if getattr(self, "_dn", None) is not None:
            return self._dn
        if 2 * self.T > 4:
            raise ValueError("denoising steps need T <= 2 (2 T partial results per query)")
        H, C, Nq, F, P, D = self.H, self.C, self.Nq, self.F, self.P, self.D
        dev = self.q_codes.device
        i32 = dict(dtype=torch.int32, device=dev)
        dn = SimpleNamespace()

        def one_bucket(n):
            codes = torch.zeros(H, 1, n, **i32)
            perm = torch.empty(H, 1, n, **i32)
            off = torch.empty(H, 1, 3, **i32)
            fastar_bucket_csr(codes, 1, perm, off, status=self.status)
            return codes, perm, off

        dn.qc0, dn.qp0, dn.qo0 = one_bucket(Nq)
        cc0, cp0, co0 = one_bucket(C)
        c = self.cache
        dn.cache_dense = Cache.view(1, 1, K=c.K, V=c.V, m=c.m, codes=cc0, last_frame=c.last_frame, size=c.size,
                                    inserted=c.inserted, evicted=c.evicted, perm=cp0, offsets=co0)
        dn.kept_all = torch.empty(H, F, max(P, 1), **i32)
        dn.cnt_all = torch.empty(H, F, **i32)
        fastar_annca_prune(dn.qc0, torch.zeros(H, 1, P, **i32), F, self.n_f, 1, dn.kept_all, dn.cnt_all,
                           status=self.status)
        dn.ones = torch.ones(H, Nq, **i32)
        dn.lf = torch.zeros(H, Nq, **i32)
        dn.nq = torch.full((H,), Nq, **i32)
        dn.cnt64 = torch.zeros(H, dtype=torch.int64, device=dev)
        dn.k_perm = torch.empty(H, self.T, Nq, **i32)
        dn.k_off = torch.empty(H, self.T, (1 << self.B) + 1, **i32)
        dn.ws = torch.empty(fastar_workspace_size(OP_ANNSA_PARTS, H, Nq, D, 2 * self.T, self.B, C),
                            dtype=torch.uint8, device=dev)
        self._dn = dn
        return dn

    # -- branches ------------------------------------------------------------
    def branches(self, B, tokens, max_len, **kw):
        """B rollouts that continue this layer's merged history (its cache is
        read, not written): a BranchRollout over the live groups with their
        + ln m.  Arguments as for BranchRollout; the scale is this layer's."""
        kw.setdefault("scale", self.scale)
        return BranchRollout(B, self.H, self.D, tokens, max_len, prefix=Prefix.of(self.cache),
                             dtype=self.dtype, device=self.q_codes.device, **kw)

    # -- internals ----------------------------------------------------------
    @staticmethod
    def _main(stream):
        if stream is None:
            return torch.cuda.current_stream()
        return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))

    def _run(self, q, k, v, kp, vp, first_frame, main, host_out=None):
        st = self.status
        staged = host_out is not None
        side = self._side
        cross = [(q, self.q_codes, None, None)]
        if self.P:
            cross.append((kp, self.p_codes, None, None))
        # The second stream hashes the chunk while the merge starts on `main`
        # (candidate setup, the first frame's NN search and plan need only k
        # and the cache); the merge waits for the key codes (and v) right
        # before its first apply.
        # the second stream starts after the work already on `main` (so that
        # layers run one after the other, as in a model)
        self._fork.record(main)
        side.wait_event(self._fork)
        if staged:
            main.wait_event(self._in_k)
            side.wait_event(self._in_k)
            fastar_hash_many([(k, self.k_codes, None, None)], self.planes, self.T, self.B, status=st,
                             stream=side)
            side.wait_event(self._in_v)
            self._codes_ready.record(side)
            side.wait_event(self._in_qp)
            fastar_hash_many(cross, self.planes, self.T, self.B, status=st, stream=side)
        else:
            fastar_hash_many([(k, self.k_codes, None, None)] + cross, self.planes, self.T, self.B,
                             status=st, stream=side)
            self._codes_ready.record(side)
        fastar_bucket_csr(self.q_codes, self.B, self.q_perm, self.q_offsets, status=st, stream=side)
        self._csr_done.record(side)
        fastar_annca_prune(self.q_codes, self.p_codes[:, :, :self.P], self.F, self.n_f, self.B,
                           self.kept_idx, self.kept_cnt, status=st, stream=side)
        if staged:
            side.wait_event(self._in_vp)
        fastar_annca_attention(q, kp, vp, self.kept_idx, self.kept_cnt, self.F, self.n_f,
                               self.scale, self.o_ca, ws=self.ws_annca, status=st, stream=side)
        if staged:
            self._ca_done.record(side)
        self._cross_done.record(side)
        fastar_tempcache_merge(self.cache, k, v, self.k_codes, self.F, self.n_f, first_frame,
                               self.tau, match_out=self.match, ws=self.ws_merge, status=st,
                               stream=main, codes_ready=self._codes_ready, rep=self.rep, planes=self.planes,
                               search=self.search)
        main.wait_event(self._csr_done)
        fastar_annsa_attention(q, self.q_codes, self.q_perm, self.q_offsets, self.cache,
                               self.scale, self.o_sa, self.lse, ws=self.ws_annsa, status=st,
                               stream=main)
        if staged:
            self._sa_done.record(main)
        main.wait_event(self._cross_done)


class ChunkStack:
    """The per-chunk path of several independent layers of one model.

    One ChunkPath per layer (own cache, codes and outputs) sharing one set
    of workspaces and streams; `step` runs the layers one after the other on
    the calling stream, as the attention layers of a model run (a layer's
    second stream starts after the previous layer's work)."""

    def __init__(self, layers, H, D, n_f, F, P, T, B, C, tau, dtype=torch.bfloat16, device="cuda", rep="last",
                 search="prev"):
        self.paths = []
        for _ in range(layers):
            self.paths.append(ChunkPath(H, D, n_f, F, P, T, B, C, tau, dtype, device, rep,
                                        share=self.paths[0] if self.paths else None, search=search))

    def __len__(self):
        return len(self.paths)

    def step(self, inputs, first_frame, stream=None):
        """inputs[l] = (q, k, v, kp, vp) of layer l, as for ChunkPath.step."""
        if len(inputs) != len(self.paths):
            raise ValueError("one input tuple per layer")
        for p, x in zip(self.paths, inputs):
            p.step(*x, first_frame, stream=stream)

    def step_host(self, host_inputs, host_outputs, first_frame, stream=None, dev_in=None):
        """Host-to-host chunk of every layer: host_inputs[l] = (q, k, v, kp,
        vp) pinned, host_outputs[l] = (o_ca, o_sa) pinned; dev_in[l] optional
        device buffers for layer l's inputs.  The copies of later layers run
        ahead of the kernels of earlier ones; `stream` waits for every output."""
        if len(host_inputs) != len(self.paths) or len(host_outputs) != len(self.paths):
            raise ValueError("one input and one output tuple per layer")
        for i, p in enumerate(self.paths):
            p.step_host(*host_inputs[i], *host_outputs[i], first_frame, stream=stream,
                        dev_in=None if dev_in is None else dev_in[i], join=False)
        for p in self.paths:
            p.join_outputs(stream)


@functools.cache
def _driver():
    return ctypes.CDLL("libcuda.so.1")


class BranchRollout:
    """B rollouts ("branches") of one layer that continue one history.

    The history is a prefix that every branch attends (a Prefix, e.g. a merged
    cache; None: none); each branch's own keys and values lie in pages of a
    pool.  `step` adds tokens to the branches and attends: it rotates the new
    queries and keys, puts keys and values into the pages and runs the
    attention of all branches over the prefix and their pages.  Page ids and
    lengths are counted on the host and copied to the device by `extend`;
    `step` itself can be captured in a graph between two `extend`s.

    tokens: most tokens of one step, all branches together (every step's calls
    are made for that many rows, so an object whose steps are much smaller than
    its largest one pays for the difference); max_len: most positions of a
    branch, whose table and pages are sized by it (under a budget at most 2^19, or
    `evict` raises); Hq: query heads (a multiple of H, default H); plan:
    RopePlan (None: queries and keys are taken as they are); block: 0, every
    new token sees all positions of its branch, or n, those of its own and
    earlier blocks of n positions (a frame's tokens, 1 for text).

    Branches are independent: infinities and NaN among the keys and values of
    one reach no other's outputs.

    Drafts: `extend(new, parents)` makes the next step's tokens of each branch a
    tree, of which `accept` keeps one path.  Drafts are single tokens: with block > 1
    they are refused, for a path of any length would leave later frames across the
    borders of blocks.

    budget: rows that a branch holds per head after `evict`.  Every call of `step` then
    adds its tokens' attention weights to the masses of the rows (older ones fade by
    `decay`): tokens that are attended several times, a frame's once per denoising
    step, are weighed in one of the calls and attended with weigh=False in the others
    (so is a warm-up before a capture).  `evict` keeps the rows of the first `first` and the last `recent`
    tokens and those of the largest masses.  With block > 1 the budget is whole
    blocks, and so is the length of a branch that is cut to it (`evict` refuses one
    whose last frame is not full), so that later tokens' blocks begin where they did.

    Order of the calls: `accept` takes drafts that were attended, `evict` (and under a
    budget the next `extend`) rows that were weighed, both after an `extend` of their
    own; they raise otherwise.  After `accept`, and after an `evict` that took rows, the
    next step needs another `extend`.  A step that was captured marks on the device that
    it was replayed; `stepped` says that a step was made of its parts' calls."""
    budget = mass = drafts = _asked = _graphs = None
    block, _pending, _over = 0, frozenset(), False

    def __init__(self, B, H, D, tokens, max_len, prefix=None, Hq=None, page=64, n_pages=None, plan=None, block=0,
                 scale=None, dtype=torch.bfloat16, device="cuda", budget=None, first=0, recent=0, decay=1.0):
        dev = torch.device(device)
        most = -(-max_len // page)
        if budget is not None and (first < 0 or recent < 0 or first + recent > budget or
                                   (block > 1 and budget % block)):
            raise ValueError("a budget holds the first and the recent rows, and whole blocks")
        self.budget, self.first, self.recent, self.decay = budget, first, recent, decay
        self.B, self.H, self.D, self.Hq, self.max_len, self.tokens = B, H, D, Hq or H, max_len, tokens
        self.prefix, self.plan, self.block = prefix, plan, block
        self.scale = D ** -0.5 if scale is None else scale
        self.pages = PagedKV(H, D, page, n_pages or B * most, B, most, dtype, dev)
        self.cu = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        self.q = torch.zeros(self.Hq, tokens, D, dtype=dtype, device=dev)  # rotated queries
        self.out = torch.zeros(self.Hq, tokens, D, dtype=dtype, device=dev)
        self.lse = torch.zeros(self.Hq, tokens, dtype=torch.float32, device=dev)
        self.ws = torch.empty(branch_workspace_size(self.Hq, H, tokens, D), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.parent = torch.zeros(tokens, dtype=torch.int32, device=dev)
        self.drafts = None                           # parents of the step's tokens, branch by branch
        # The step since the last `extend`: its drafts' queries, once attended; the
        # branches whose new rows are not weighed; whether it is over.  The captured
        # steps, as (queries, of drafts), and the number (from 1) of the one replayed last.
        self._asked, self._pending, self._over = None, frozenset(), False
        self._graphs, self._replayed = [], torch.zeros(1, dtype=torch.int32, device=dev)
        if budget is not None:
            self.mass = PageMass(self.pages)
            self.ws_mass = torch.empty(max(1, mass_workspace_size(self.Hq, H, tokens, D)), dtype=torch.uint8, device=dev)
        self.lengths = [0] * B
        self.totals = [0] * B                        # tokens that each branch has had
        self.held = [[] for _ in range(B)]           # page ids of each branch
        self.free = list(range(self.pages.n_pages))[::-1]
        # the fills above are over before another stream's `extend` or `step`
        torch.cuda.current_stream(dev).synchronize()

    def extend(self, new, stream=None, parents=None):
        """Make room for new[b] more positions of each branch: the next step's
        tokens, laid out branch after branch.  The copies to the device go to
        `stream` (default: the current one), which is also the next step's.

        parents: the tokens are drafts; parents[b][i] < i is the draft of branch b
        that its draft i follows, -1: the branch's last position.  `accept` ends
        their step."""
        if self.drafts is not None:
            raise ValueError("the drafts of the last step are not accepted yet")
        if parents is not None and self.block > 1:
            raise ValueError("drafts are single tokens: block is 0 or 1")
        if parents is not None and ([len(p) for p in parents] != list(new) or
                                    any(not -1 <= q < i for p in parents for i, q in enumerate(p))):
            raise ValueError("one parent per draft, an earlier one of its branch or -1")
        if len(new) != self.B or any(n < 0 for n in new) or sum(new) > self.tokens:
            raise ValueError("one count of new tokens per branch, at most `tokens` in all")
        lengths = [a + n for a, n in zip(self.lengths, new)]
        if max(lengths, default=0) > self.max_len:
            raise ValueError("a branch is longer than max_len")
        if self.mass is not None:
            self._weighed(stream)
        page = self.pages.page
        need = [-(-a // page) - len(h) for a, h in zip(lengths, self.held)]
        if sum(need) > len(self.free):
            raise ValueError("no pages left")
        for h, n in zip(self.held, need):
            h.extend(self.free.pop() for _ in range(n))
        self.lengths = lengths
        most = self.pages.max_pages
        offsets = [0]
        for n in new:
            offsets.append(offsets[-1] + n)
        i32 = dict(dtype=torch.int32)
        self._asked, self._over = None, False
        if self._graphs is not None:
            self._pending = {b for b, n in enumerate(new) if n}
        with self._on(stream):
            if self._graphs:
                self._replayed.zero_()
            if any(need):  # (a released branch's old entries are not read)
                table = [h + [0] * (most - len(h)) for h in self.held]
                self.pages.table.copy_(torch.tensor(table, **i32).view(self.B, most))
            self.pages.len.copy_(torch.tensor(lengths, **i32))
            self.cu.copy_(torch.tensor(offsets, **i32))
            if self.mass is not None:
                self.totals = [a + n for a, n in zip(self.totals, new)]
                self.mass.total.copy_(torch.tensor(self.totals, **i32))
            if parents is not None:
                self.drafts = [list(p) for p in parents]
                flat = [q for p in parents for q in p]
                self.parent[:len(flat)].copy_(torch.tensor(flat, **i32))

    def release(self, b):
        """Branch b starts again: its pages return to the pool."""
        if self.drafts is not None:
            raise ValueError("the drafts of the last step are not accepted yet")
        self.free.extend(self.held[b][::-1])
        self.held[b], self.lengths[b] = [], 0
        self._pending = self._pending - {b}
        if self.mass is not None:
            self.totals[b] = 0

    @staticmethod
    def _on(stream):
        return torch.cuda.stream(None if stream is None else ChunkPath._main(stream))

    @staticmethod
    def _capturing(stream):
        """Whether calls on the stream go into a graph.  (Asked of the driver for a
        stream that need not be the current one: to make it the current one takes 12 us
        of a small step's 23.)"""
        if stream is None:
            return torch.cuda.is_current_stream_capturing()
        handle = _stream(stream)
        if not handle:
            return False  # (the legacy default stream cannot be captured)
        state = ctypes.c_int(0)
        rc = _driver().cuStreamIsCapturing(ctypes.c_void_p(handle), ctypes.byref(state))
        if rc:
            raise RuntimeError(f"cuStreamIsCapturing: CUDA driver error {rc}")
        return state.value != 0

    def _made(self, q, of_drafts):
        """A step of these queries has run since `extend`."""
        if self.drafts is None and not of_drafts:
            self._pending = frozenset()
        elif self.drafts is not None and of_drafts:
            self._asked = q

    def _settle(self, stream):
        """Takes note of a step that was replayed since `extend` (waits for it)."""
        if not self._graphs:
            return
        with self._on(stream):
            n = int(self._replayed)
        if n:
            self._made(*self._graphs[n - 1])

    def _weighed(self, stream):
        if self._pending:
            self._settle(stream)
        if self._pending:
            raise ValueError("the tokens of the last extend are not weighed yet")

    def stepped(self, q=None):
        """Says that the tokens of the last `extend` were appended and attended (under a
        budget plain tokens also weighed) by calls of their own and not by `step`.  q:
        the drafts' queries as they were attended, [Hq][tokens][D] (default, with a
        plan: this object's buffer of rotated ones)."""
        if self.drafts is not None and self.mass is not None and q is None and self.plan is None:
            raise ValueError("the drafts' queries are not in this object's buffer")
        self._made(self.q if q is None else q, self.drafts is not None)

    def _shrink(self, lengths):
        """The branches hold `lengths` positions now; pages behind return to the
        pool.  (Their entries of the table are not read any more.)"""
        self.lengths = lengths
        for held, n in zip(self.held, lengths):
            while len(held) > -(-n // self.pages.page):
                self.free.append(held.pop())
        self.pages.len.copy_(torch.tensor(lengths, dtype=torch.int32))

    def accept(self, leaves, stream=None):
        """Ends a step of drafts: of each branch the draft leaves[b] and those
        above it stay (-1: none), in the order of their positions.  Returns their
        numbers within the step's rows, branch by branch.  (Under a budget their
        queries are read again: without a plan, the step's q is as it was.)"""
        if self.drafts is None:
            raise ValueError("the last step had no drafts")
        self._settle(stream)
        if self._asked is None:
            raise ValueError("the drafts have not been attended yet")
        if len(leaves) != self.B or any(not -1 <= x < len(p) for x, p in zip(leaves, self.drafts)):
            raise ValueError("one draft per branch, or -1")
        kept, first = [], 0
        for x, p in zip(leaves, self.drafts):
            path = []
            while x >= 0:
                path.append(first + x)
                x = p[x]
            kept.append(path[::-1])
            first += len(p)
        gone = [len(p) - len(k) for p, k in zip(self.drafts, kept)]
        cu = [0]
        for k in kept:
            cu.append(cu[-1] + len(k))
        i32 = dict(dtype=torch.int32, device=self.cu.device)
        with self._on(stream):
            rows = torch.tensor([r for k in kept for r in k], **i32)
            keep = torch.tensor(cu, **i32)
            fastar_page_keep(self.pages, self.cu, rows, keep, status=self.status)
            self._shrink([n - g for n, g in zip(self.lengths, gone)])
            self.cu.copy_(keep)
            if self.mass is not None:
                self.totals = [n - g for n, g in zip(self.totals, gone)]
                self.mass.total.copy_(torch.tensor(self.totals, dtype=torch.int32))
                fastar_page_mass(self.pages, self._asked, self.lse, self.cu, self.scale, self.mass, block=1, rows=rows,
                                 decay=self.decay, ws=self.ws_mass, status=self.status)
        self.drafts = self._asked = None
        self._pending, self._over = frozenset(), True
        return kept

    def evict(self, stream=None):
        """Every branch of more than `budget` positions keeps, in each head,
        `budget` of its rows, and returns the pages behind.  With block > 1 such a
        branch holds whole blocks."""
        if self.budget is None:
            raise ValueError("this rollout has no budget")
        if self.drafts is not None:
            raise ValueError("the drafts of the last step are not accepted yet")
        if self.block > 1 and any(n > self.budget and n % self.block for n in self.lengths):
            raise ValueError("a branch over the budget is not whole blocks")
        self._weighed(stream)
        with self._on(stream):
            fastar_page_evict(self.pages, self.mass, self.budget, first=self.first, recent=self.recent,
                              status=self.status)
            self._over = self._over or any(n > self.budget for n in self.lengths)
            self._shrink([min(n, self.budget) for n in self.lengths])

    def step(self, q, k, v, pos=None, stream=None, weigh=True):
        """The new tokens of the last `extend`: q [Hq][tokens][D], k, v
        [H][tokens][D] (any head and token strides, but a q that is not rotated
        is contiguous; the rows behind the last branch's are ignored), pos [tokens][axes] int32 with a plan.  Returns
        (out [Hq][tokens][D], lse [Hq][tokens]), buffers of this object.

        weigh: add the tokens' weights to the masses, under a budget.  Each call
        that weighs adds them (and fades the older rows) again.  Drafts are weighed by
        `accept` alone."""
        captured = (self._over or self.drafts is not None or self.mass is not None) and self._capturing(stream)
        if self._over and not captured:
            raise ValueError("the last step is over: extend comes first")
        rotated = self.q if self.plan is not None else q
        fastar_page_append(self.pages, k, v, self.cu, pos=pos, plan=self.plan,
                           q=q if self.plan is not None else None, q_out=self.q if self.plan is not None else None,
                           status=self.status, stream=stream)
        if self.drafts is not None:
            fastar_tree_attention(rotated, self.cu, self.parent, self.prefix, self.pages, self.scale, self.out,
                                  lse=self.lse, ws=self.ws, status=self.status, stream=stream)
            self._note(rotated, True, captured, stream)  # (`accept` weighs the tokens that stay)
            return self.out, self.lse
        fastar_branch_attention(rotated, self.cu, self.prefix, self.pages, self.scale, self.out, lse=self.lse,
                                block=self.block, ws=self.ws, status=self.status, stream=stream)
        if self.mass is not None and weigh:
            fastar_page_mass(self.pages, rotated, self.lse, self.cu, self.scale, self.mass, block=self.block,
                             decay=self.decay, ws=self.ws_mass, status=self.status, stream=stream)
            if captured:
                self._note(None, False, True, stream)
            else:
                self._pending = frozenset()
        return self.out, self.lse

    def _note(self, q, of_drafts, captured, stream):
        """A step ran, or was captured: then its replays leave its number."""
        if captured:
            self._graphs.append((q, of_drafts))
        else:
            self._made(q, of_drafts)
        if captured or (of_drafts and self._graphs):
            with self._on(stream):
                self._replayed.fill_(len(self._graphs) if captured else 0)
