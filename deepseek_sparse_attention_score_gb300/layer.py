"""One DSA layer step on a resident batch, built from the C-ABI calls.

Every layer first writes its new tokens' rows into the paged caches (the
latent row of every layer, the indexer key on full layers; the backend's
_scatter_paged step that precedes the path). Decode batches then run indexer
-> token top-k (or page top-k with a page budget) -> sparse MLA decode.
Prefill / mixed batches run, on full layers, the indexer once for both the
page top-k (K_p = ceil(k/ps), what the attention consumes) and the token
top-k, then the block union and the query-block sparse MLA; shared layers
(IndexShare, ref.py build_index_share_map) reuse the top-k and union tables of
their source slot and run the attention only.

A step may also start from less than finished inputs: with ``tables`` it
builds its metadata on the GPU from the requests' lengths, with ``rope`` it
rotates queries and keys for the positions found there, and with
``cache_bits=4`` it keeps the latent cache in 4 bits.

All buffers are allocated once up front, so a step only enqueues kernels and
can be captured in a CUDA graph.
"""
from __future__ import annotations

import torch

from . import abi


class LayerRunner:
    def __init__(self, wl, device, page_budget=None, prefill=None, cache_bits=16, tables=False, rope=None,
                 spare_pages=(), PTW=None, max_kv=None):
        """``wl``: a dsa_inputs.Workload whose tensors already live on ``device``
        (or on the CPU; they are moved). ``page_budget``: decode page-budget
        mode with that many pages. ``prefill``: force the prefill path
        (default: any request with more than one new token).
        ``cache_bits``: 16, or 4 for a 4-bit latent cache (quantised from the
        workload's; prefill tokens then attend to their own page selections
        through the 4-bit decode call, one by one instead of by query blocks).
        ``tables``: build the metadata every step with dsa_build_page_tables,
        from ``lens`` (q_lens, seq_lens), ``block_table`` and ``free_pages``.
        Lengths that the caller advances between steps (also between replays
        of a captured one) make each step take its pages behind those of the
        steps before; a step with unchanged lengths is the last one again
        (``free_state``, see dsa_build_page_tables; zero it when
        ``free_pages`` is filled anew). Room to grow:
        ``spare_pages``, page ids that later steps may take; ``PTW``, the
        page-table entries (by default the workload's and the spare pages);
        ``max_kv``, the longest length a request may reach (by default the
        workload's longest).
        ``rope``: (freqs, scale, layout), with ``tables``: the workload's
        rotary columns (the last 64 of latent rows and queries, the first 64
        of indexer queries and keys) are taken as not rotated yet, and every
        step rotates its tokens'; indexer columns pair by halves. ``scale`` is
        that of the rotated columns alone: YaRN's temperature of the logits
        belongs in the workload's ``sm_scale`` (dsa_rope_attention_scales)."""
        if cache_bits not in (4, 16):
            raise ValueError(f"cache_bits must be 4 or 16, got {cache_bits}")
        if rope is not None and not tables:
            raise ValueError("rope needs the positions that tables=True finds")
        if not tables and (len(spare_pages) or PTW is not None or max_kv is not None):
            raise ValueError("spare_pages, PTW and max_kv are for tables=True")
        rg = wl.rg
        if PTW is not None and PTW < rg.PTW or max_kv is not None and max_kv < rg.max_kv:
            raise ValueError(f"the workload needs {rg.PTW} page-table entries and lengths of {rg.max_kv}")
        self.wl = wl
        self.dev = torch.device(device)
        dev = self.dev
        self.rg = rg
        self.T, self.S, self.P, self.PTW, self.ps = rg.T, rg.S, rg.num_pages, rg.PTW, rg.page_size
        self.max_kv = max(1, rg.max_kv, max_kv or 0)
        if tables:
            self.PTW = rg.PTW + len(spare_pages) if PTW is None else PTW
        self.k = wl.k
        self.k_pages = wl.k_pages if page_budget is None else page_budget
        self.page_budget = page_budget
        self.prefill = bool((rg.q_lens > 1).any()) if prefill is None else prefill
        to = lambda a: torch.from_numpy(a).to(dev)
        self.meta = [to(rg.seq_lens), to(rg.cu_q_lens), to(rg.cu_kv_lens), to(rg.page_indices)]
        self.q_idx = wl.q_idx.to(dev)
        self.w = wl.w.to(dev)
        self.kcache = [c.to(dev) for c in wl.kcache]
        self.q = [x.to(dev) for x in wl.q]
        self.kv = [x.to(dev) for x in wl.kv]
        self.types = list(wl.indexer_types) if wl.indexer_types else [0]
        self.full_slot, self.src_slot, self.num_full = abi.dsa_index_build_share_map(self.types, len(self.types))
        # the new tokens' rows (latent rows per layer, indexer keys per full
        # slot): taken from the synthetic caches, which already hold them, so
        # writing them back leaves every cache as generated
        tseq, tpos = rg.token_seq(), rg.token_pos()
        ent = rg.cu_kv_lens[tseq] // rg.page_size + tpos // rg.page_size
        rows = torch.from_numpy(rg.page_indices[ent].astype("int64") * rg.page_size + tpos % rg.page_size).to(dev)
        self.new_kv = [c.view(-1, c.shape[-1]).index_select(0, rows)[:, :576].contiguous() for c in self.kv]
        self.new_k = [c.view(-1, c.shape[-1]).index_select(0, rows).contiguous() for c in self.kcache]
        T, H = self.T, wl.H
        self.H = H
        self.cache_bits = cache_bits
        if cache_bits == 4:
            self.kv4 = [self._quantised(c) for c in self.kv]
            self.kv = None
        self.tables = self._make_tables(rg, spare_pages) if tables else None
        self.rope = None
        if rope is not None:
            freqs, scale, layout = rope
            self.rope = torch.as_tensor(freqs, dtype=torch.float64).to(dev)
            raw = lambda x, cols: x.view(T, -1, x.shape[-1])[:, :, cols].clone()
            qk, ki = slice(512, 576), slice(0, 64)
            turn = lambda x, cols, s, lay: abi.RopeTarget(raw(x, cols), x.view(T, -1, x.shape[-1])[:, :, cols],
                                                          layout=lay, scale=s)
            # layer -> what it rotates; the indexer's queries with the first layer
            self.rope_targets = []
            for layer in range(len(self.types)):
                g = [turn(self.q[layer], qk, scale, layout), turn(self.new_kv[layer], qk, scale, layout)]
                if self.full_slot[layer] >= 0:
                    g.append(turn(self.new_k[self.full_slot[layer]], ki, 1.0, "half"))
                if layer == 0:
                    g.append(turn(self.q_idx, ki, 1.0, "half"))
                self.rope_targets.append(g)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ws_idx = torch.empty(max(1, abi.dsa_indexer_workspace_size(T, self.S, self.max_kv, self.ps)),
                                  dtype=torch.uint8, device=dev)
        if cache_bits == 16:  # the split scratch of the bf16 decode; the 4-bit form merges inside clusters
            self.ws_att = torch.empty(max(1, abi.dsa_sparse_mla_decode_workspace_size(T, H)), dtype=torch.uint8,
                                      device=dev)
        nl = len(self.types)
        self.topk = [torch.empty((T, self.k), dtype=torch.int32, device=dev) for _ in range(self.num_full)]
        self.topk_pages = [torch.empty((T, self.k_pages), dtype=torch.int32, device=dev)
                           for _ in range(self.num_full)]
        self.o = [torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev) for _ in range(nl)]
        if self.prefill and cache_bits == 16:  # query blocks; 4-bit prefill tokens attend one by one
            self.QB = wl.QB
            self.u_max = wl.u_max if wl.u_max > 0 else min(self.QB * self.k_pages, self.PTW)
            nqb = (T + self.QB - 1) // self.QB
            self.units = [torch.empty((nqb, self.u_max), dtype=torch.int32, device=dev) for _ in range(self.num_full)]
            self.member = [torch.empty((nqb, self.u_max, self.QB // 32), dtype=torch.int32, device=dev)
                           for _ in range(self.num_full)]
            self.counts = [torch.empty((nqb,), dtype=torch.int32, device=dev) for _ in range(self.num_full)]

    def _quantised(self, cache):
        """The 4-bit form of a bf16 cache [P, ps, W]: every row written back
        to where it is (one request that owns the whole pool)."""
        P, ps = cache.shape[:2]
        out = torch.zeros((P, ps, abi.Q4_ROW_BYTES), dtype=torch.uint8, device=self.dev)
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=self.dev)
        abi.dsa_q4_write_back(cache.view(P * ps, -1), out, i32(P * ps), i32(0, P * ps), i32(0, P * ps),
                              torch.arange(P, dtype=torch.int32, device=self.dev))
        return out

    def _make_tables(self, rg, spare_pages):
        """Inputs and outputs of dsa_build_page_tables for the workload's
        batch: the pages that its new tokens are the first to need wait in
        ``free_pages``, the spare ones behind them, the others in
        ``block_table``. ``meta`` becomes the outputs."""
        had = -(-(rg.seq_lens - rg.q_lens) // self.ps)
        need = -(-rg.seq_lens // self.ps)
        bt = torch.full((self.S, -(-self.max_kv // self.ps)), -1, dtype=torch.int32)
        free = []
        for s in range(self.S):
            pages = rg.page_indices[rg.cu_kv_lens[s] // self.ps:][: need[s]]
            bt[s, : had[s]] = torch.from_numpy(pages[: had[s]])
            free.extend(pages[had[s]:].tolist())
        self.lens = [torch.from_numpy(rg.q_lens.astype("int32")).to(self.dev), self.meta[0]]
        self.block_table = bt.to(self.dev)
        self.free_pages = torch.tensor(free + list(spare_pages), dtype=torch.int32, device=self.dev)
        self.free_state = torch.zeros(3 + 2 * self.S, dtype=torch.int32, device=self.dev)
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=self.dev)
        out = abi.PageTables(i32(self.S + 1), i32(self.S + 1), i32(self.PTW), i32(self.T), i32(self.T), i32(self.T),
                             i32(1))
        self.meta = [self.meta[0], out.cu_q_lens, out.cu_kv_lens, out.page_indices]
        return out

    # -- stages ---------------------------------------------------------------
    def begin_step(self):
        """The step's metadata from its lengths (with ``tables``)."""
        if self.tables is not None:
            abi.dsa_build_page_tables(*self.lens, self.block_table, self.free_pages, T=self.T, PTW=self.PTW,
                                      ps=self.ps, free_state=self.free_state, out=self.tables,
                                      dev_status=self.status)

    def rotate(self, layer):
        """The layer's queries, latent rows and indexer keys at their
        positions (with ``rope``)."""
        if self.rope is not None:
            abi.dsa_rope(self.rope_targets[layer], self.tables.positions, self.rope)

    def write_back(self, layer):
        """The layer's new latent rows, and on a full layer its new indexer
        keys, into their slots of the paged caches."""
        if self.cache_bits == 4:
            abi.dsa_q4_write_back(self.new_kv[layer], self.kv4[layer], *self.meta, dev_status=self.status)
            if self.full_slot[layer] >= 0:
                slot = self.full_slot[layer]
                abi.dsa_paged_write_back(self.new_k[slot], self.kcache[slot], *self.meta, D=128,
                                         dev_status=self.status)
        elif self.full_slot[layer] >= 0:  # both caches share the page table: one launch
            slot = self.full_slot[layer]
            abi.dsa_paged_write_back_pair(self.new_kv[layer], self.kv[layer], self.new_k[slot], self.kcache[slot],
                                          *self.meta, D0=576, D1=128, dev_status=self.status)
        else:
            abi.dsa_paged_write_back(self.new_kv[layer], self.kv[layer], *self.meta, D=576, dev_status=self.status)

    def index(self, slot):
        if self.prefill or self.page_budget is not None:
            abi.dsa_indexer_page_topk(self.q_idx, self.w, self.kcache[slot], *self.meta, k_pages=self.k_pages,
                                      max_kv=self.max_kv, topk_pages=self.topk_pages[slot], k=self.k,
                                      topk=self.topk[slot] if self.prefill else None, ws=self.ws_idx,
                                      dev_status=self.status)
        else:
            abi.dsa_indexer_topk(self.q_idx, self.w, self.kcache[slot], *self.meta, k=self.k, max_kv=self.max_kv,
                                 topk=self.topk[slot], ws=self.ws_idx, dev_status=self.status)

    def union(self, slot):
        abi.dsa_build_block_union(self.topk_pages[slot], QB=self.QB, u_max=self.u_max, cu_q_lens=self.meta[1],
                                  cu_kv_lens=self.meta[2], ps=self.ps, PTW=self.PTW, units=self.units[slot],
                                  member=self.member[slot], counts=self.counts[slot], dev_status=self.status)

    def attend(self, layer, t_range=None):
        """The layer's attention; ``t_range=(b, e)`` (prefill batches) writes
        only the output rows of tokens b .. e-1."""
        slot = self.src_slot[layer]
        if self.cache_bits == 4:
            paged = self.prefill or self.page_budget is not None
            abi.dsa_sparse_mla_decode_q4(self.q[layer], self.kv4[layer], *self.meta,
                                         (self.topk_pages if paged else self.topk)[slot],
                                         unit=self.ps if paged else 1, sm_scale=self.wl.sm_scale, o=self.o[layer],
                                         dev_status=self.status)
        elif self.prefill:
            abi.dsa_sparse_mla_prefill_qblock(self.q[layer], self.kv[layer], *self.meta, self.units[slot],
                                              self.member[slot], self.counts[slot], QB=self.QB,
                                              sm_scale=self.wl.sm_scale, o=self.o[layer], dev_status=self.status,
                                              t_range=t_range)
        elif self.page_budget is not None:
            abi.dsa_sparse_mla_decode(self.q[layer], self.kv[layer], *self.meta, self.topk_pages[slot],
                                      unit=self.ps, sm_scale=self.wl.sm_scale, o=self.o[layer], ws=self.ws_att,
                                      dev_status=self.status)
        else:
            abi.dsa_sparse_mla_decode(self.q[layer], self.kv[layer], *self.meta, self.topk[slot], unit=1,
                                      sm_scale=self.wl.sm_scale, o=self.o[layer], ws=self.ws_att,
                                      dev_status=self.status)

    def layer_step(self, layer):
        self.rotate(layer)
        self.write_back(layer)
        if self.full_slot[layer] >= 0:
            slot = self.full_slot[layer]
            self.index(slot)
            if self.prefill and self.cache_bits == 16:
                self.union(slot)
        self.attend(layer)

    def step(self):
        """Every layer of the workload once (IndexShare across layers)."""
        self.begin_step()
        for layer in range(len(self.types)):
            self.layer_step(layer)

    def step_host(self, h_q_idx, h_w, h_q, h_meta, h_topk, h_o, side, h_new_kv=None, h_new_k=None, out_side=None,
                  last_chunks=4):
        """One step from and to pinned host buffers (same shapes as the device
        tensors). The indexer inputs, the metadata and the new tokens' rows
        are copied first, on the current stream: host-to-device copies of all
        streams share one copy queue, so anything issued after the queries
        would wait for them. Each layer's attention queries (the largest
        inputs, needed only by that layer's attention) follow on the stream
        ``side``, in layer order, while the earlier layers compute; each
        layer's output is read back on the stream ``out_side`` (one of the
        runner's own if None) as soon as that layer's attention has written it,
        and the token selections of the first full slot once they exist. On a
        prefill batch the first layer's queries arrive, and its attention runs,
        in ``last_chunks`` token ranges (the attention of the first range
        starts when its queries have landed, not all of them), and the last
        layer's attention runs in as many ranges, each read back as soon as it
        is written, so little of the final read-back is left after the last
        kernel. The current stream joins both side streams before it returns,
        so the step ends when every copy has landed. Can be captured in a CUDA
        graph. With ``tables``, ``h_meta`` is (q_lens, seq_lens). Queries and
        rows arrive rotated: not with ``rope``. A 4-bit cache's attention runs
        in one range."""
        if self.rope is not None:
            raise ValueError("step_host takes rotated queries and rows: use it without rope")
        cur = torch.cuda.current_stream(self.dev)
        if out_side is None:
            if getattr(self, "_out_side", None) is None:
                self._out_side = torch.cuda.Stream(self.dev)
            out_side = self._out_side
        nl = len(self.types)

        def ranges(layer):
            # token ranges on query-block boundaries (first and last layer of a
            # prefill batch), else the whole batch
            split = self.prefill and self.cache_bits == 16 and layer in (0, nl - 1)
            nch = max(1, min(last_chunks, self.T // self.QB)) if split else 1
            if nch == 1:
                return [(0, self.T)]
            nqb = -(-self.T // self.QB)
            b = [min(self.T, (nqb * c // nch) * self.QB) for c in range(nch)] + [self.T]
            return list(zip(b[:-1], b[1:]))

        self.q_idx.copy_(h_q_idx, non_blocking=True)
        self.w.copy_(h_w, non_blocking=True)
        for d, h in zip(self.meta if self.tables is None else self.lens, h_meta):
            d.copy_(h, non_blocking=True)
        for d, h in zip(self.new_kv, h_new_kv or []):
            d.copy_(h, non_blocking=True)
        for d, h in zip(self.new_k, h_new_k or []):
            d.copy_(h, non_blocking=True)
        # the previous step's kernels have finished reading q (its read-backs
        # were joined into the current stream when it returned)
        side.wait_stream(cur)
        q_ready = []  # per layer: one event per token range of its attention
        with torch.cuda.stream(side):
            for layer, (d, h) in enumerate(zip(self.q, h_q)):
                evs = []
                for b, e in ranges(layer) if layer == 0 else [(0, self.T)]:
                    d[b:e].copy_(h[b:e], non_blocking=True)
                    ev = torch.cuda.Event()
                    ev.record(side)
                    evs.append(ev)
                q_ready.append(evs)
        topk_read = False
        self.begin_step()
        for layer in range(nl):
            self.write_back(layer)
            if self.full_slot[layer] >= 0:
                slot = self.full_slot[layer]
                self.index(slot)
                if self.prefill and self.cache_bits == 16:
                    self.union(slot)
                if not topk_read:
                    out_side.wait_stream(cur)
                    with torch.cuda.stream(out_side):
                        h_topk.copy_(self.topk[0], non_blocking=True)
                    topk_read = True
            rs = ranges(layer)
            for i, (b, e) in enumerate(rs):
                evs = q_ready[layer]
                cur.wait_event(evs[min(i, len(evs) - 1)])
                self.attend(layer, (b, e) if len(rs) > 1 else None)
                out_side.wait_stream(cur)
                with torch.cuda.stream(out_side):
                    h_o[layer][b:e].copy_(self.o[layer][b:e], non_blocking=True)
        cur.wait_stream(side)
        cur.wait_stream(out_side)
