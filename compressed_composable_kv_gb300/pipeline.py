"""Request-batch runtime over the C ABI: owns the device caches, the length
arrays and the attention scratch of a batch of composed requests.

It only allocates device memory (torch) and sequences C-ABI calls; every
step of the path (composition, re-rotation, append, attention) runs in the
CUDA library.  C2KV explainer (paper-daily.com), section "pipeline: extract,
store, concatenate": compose the retrieved documents, append the question,
then generate.
"""
from __future__ import annotations

import weakref
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

from . import binding as B


def _stream_on(device: torch.device, stream):
    """The stream of a call (None: the device's current one, or a handle) as a torch stream; None on the host."""
    if device.type != "cuda":
        return None
    if stream is None:
        return torch.cuda.current_stream(device)
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device)


@dataclass
class RequestSpec:
    doc_ids: List[int]
    order: Optional[List[int]] = None


class RequestBatch:
    """Device state of `len(requests)` composed requests sharing one store.

    page8: tokens of a page (16, 32, 64 or 128) to decode over an 8-bit paged
    cache, which reads half the bytes of the bf16 one (that stays allocated beside
    it: composition and prefill write there): after composition and question
    prefill, fill_pages8 takes the bf16 rows over, and decode appends to and
    attends over the pages.  `filled` holds the layers whose pages hold the rows
    (a program that writes pages by calls of its own adds to it); decode refuses
    the others, but not while a graph is captured.  spare_pages: further pages of the
    pool, for `answers`.
    """

    def __init__(self, store: int, geom, requests: Sequence[RequestSpec], k: int, q_len: int,
                 decode_steps: int, device: str = "cuda", cap_multiple: int = 32, realign: bool = True,
                 page8: Optional[int] = None, spare_pages: int = 0):
        if spare_pages < 0 or (spare_pages and page8 is None):
            raise ValueError("spare_pages must be >= 0, and go with page8")
        if page8 not in (None, 16, 32, 64, 128):
            raise ValueError(f"page8 must be None, 16, 32, 64 or 128, not {page8}")
        self.store, self.geom, self.k = store, geom, k
        # realign=False: the "no position re-alignment" ablation (documents
        # keep their extraction positions)
        self.compose_flags = 0 if realign else B.C2KV_COMPOSE_NO_REALIGN
        self.requests = list(requests)
        self.q_len, self.decode_steps = q_len, decode_steps
        self.batch = len(self.requests)
        L, H, D = geom.n_layers, geom.n_kv_heads, geom.head_dim
        self.n_slots, self.l_tot = [], []
        for r in self.requests:
            nt, ns = [], []
            for d in r.doc_ids:
                a, b, _ = B.c2kv_store_lookup(store, d)
                nt.append(a)
                ns.append(b)
            _, _, n, lt = B.c2kv_plan(nt, ns, r.order)
            self.n_slots.append(n)
            self.l_tot.append(lt)
        need = max(self.n_slots) + q_len + decode_steps
        self.cap = max(cap_multiple, -(-need // cap_multiple) * cap_multiple)
        self.k_caches = [torch.empty((L, H, self.cap, D), dtype=torch.bfloat16, device=device)
                         for _ in range(self.batch)]
        self.v_caches = [torch.empty_like(t) for t in self.k_caches]
        self.pos = [torch.full((self.cap,), -1, dtype=torch.int32, device=device)
                    for _ in range(self.batch)]
        tb = B.c2kv_rope_table_bytes(geom, self.cap)
        # one allocation, so that it is also the table of the paged calls, where
        # request b's row r is row b * cap + r
        self.rope_table = torch.empty((self.batch, tb // 4), dtype=torch.float32, device=device)
        self.rope_tables = list(self.rope_table)
        # the lengths, and behind them the RoPE rows that go with them
        self._lengths = torch.zeros((2, self.batch), dtype=torch.int32, device=device)
        self.n_cached_dev, self._rope_row = self._lengths
        self._own_lengths = self.n_cached_dev
        self._rope_start = torch.arange(self.batch, dtype=torch.int32, device=device) * self.cap
        self.max_keys_decode = max(self.n_slots) + q_len + decode_steps
        ws = 256
        if q_len > 0:
            ws = max(ws, B.c2kv_attend_workspace_size(geom, self.batch, q_len, max(self.n_slots) + q_len))
        ws = max(ws, B.c2kv_attend_workspace_size(geom, self.batch, 1, self.max_keys_decode))
        self.page8 = page8
        self.filled = set()
        self._fill_before = False   # the batch's last call was fill_pages8
        self._answers = lambda: None   # the sequences that have the pool's pages, while they are there
        if page8 is not None:
            most = -(-self.max_keys_decode // page8)
            self.page_table = torch.arange(most * self.batch, dtype=torch.int32, device=device).reshape(self.batch, most)
            n_pages = most * self.batch + spare_pages
            self.k8 = torch.empty((L, n_pages, H, page8, D), dtype=torch.float8_e4m3fn, device=device)
            self.v8 = torch.empty_like(self.k8)
            self.k_scale = torch.empty((L, n_pages, H), dtype=torch.float32, device=device)
            self.v_scale = torch.empty_like(self.k_scale)
            # of its own: the other calls' scratch would overwrite its counters
            self.workspace8 = torch.zeros(B.c2kv_attend_pages8_workspace_size(geom, self.batch, self.max_keys_decode),
                                          dtype=torch.uint8, device=device)
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=device)
        B.c2kv_workspace_init(self.workspace)
        start = [n + q_len for n in self.n_slots]
        self._dec_start = torch.tensor([start, [b * self.cap + n for b, n in enumerate(start)]], dtype=torch.int32)

    @property
    def rope_row_dev(self) -> torch.Tensor:
        """Each request's row of rope_table for its next token, from the lengths
        as they are (on the current stream).  The same tensor each time; it moves
        with reset_decode and advance.  decode does not need it."""
        return torch.add(self._rope_start, self.n_cached_dev, out=self._rope_row)

    def compose(self, stream=None) -> None:
        self.compose_layers(0, self.geom.n_layers, stream)

    def compose_layers(self, layer_begin: int, layer_end: int, stream=None) -> None:
        """Compose layers [layer_begin, layer_end) of every request.  A call
        with layer_begin > 0 continues the composition of the call before it
        (C2KV_COMPOSE_CONTINUE): its copies follow that call's copies, so work
        enqueued in between on the earlier layers (the question prefill)
        overlaps them ("the problem": loading the cache dominates TTFT)."""
        flags = self.compose_flags | (B.C2KV_COMPOSE_CONTINUE if layer_begin > 0 else 0)
        for b, r in enumerate(self.requests):
            n, nxt = B.c2kv_compose_layers(self.store, r.doc_ids, r.order, self.k, flags, layer_begin,
                                           layer_end, self.k_caches[b], self.v_caches[b], self.cap,
                                           self.rope_tables[b], self.pos[b], stream)
            assert n == self.n_slots[b] and nxt == self.l_tot[b]
        self._rows_change(range(layer_begin, layer_end), stream)

    def _capturing(self, stream) -> bool:
        if not self.n_cached_dev.is_cuda:
            return False
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()

    def _rows_change(self, layers, stream) -> None:
        """The bf16 rows of these layers are no longer what their pages hold."""
        if self.filled and not self._capturing(stream):
            self.filled.difference_update(layers)

    def prefill(self, layer: int, q, k_new, v_new, out, stream=None) -> None:
        B.c2kv_attend_prefill(self.geom, layer, self.k_caches, self.v_caches, self.rope_tables, self.cap,
                              self.n_slots, q, k_new, v_new, out, self.workspace, stream)
        self._rows_change((layer,), stream)

    def reset_decode(self, stream=None) -> None:
        """Point the device lengths at the first decode step (after the question)."""
        s = torch.cuda.current_stream() if stream is None else stream
        with torch.cuda.stream(s):
            if self.n_cached_dev is self._own_lengths:
                self._lengths.copy_(self._dec_start, non_blocking=True)
            else:   # a program's own tensor
                self.n_cached_dev.copy_(self._dec_start[0], non_blocking=True)

    def fill_pages8(self, layer_begin: int = 0, layer_end: Optional[int] = None, stream=None) -> None:
        """The composed and prefilled rows of layers [layer_begin, layer_end) to the 8-bit pages."""
        if self.page8 is None:
            raise ValueError("this batch was made without page8")
        self._refuse_lent_pool()
        layer_end = self.geom.n_layers if layer_end is None else layer_end
        B.c2kv_pages8_fill(self.geom, layer_begin, layer_end, self.k_caches, self.v_caches, self.cap,
                           [n + self.q_len for n in self.n_slots], self.k8, self.v8, self.k_scale, self.v_scale,
                           self.page_table, stream)
        self.filled.update(range(layer_begin, layer_end))
        self._fill_before = True

    def decode(self, layer: int, q, k_new, v_new, out, stream=None, overlap_previous: Optional[bool] = None) -> None:
        """One decode step of one layer.  By default a layer > 0 call may start
        while the previous kernel on the stream (this batch's decode of the
        layer before) finishes: see C2KV_DECODE_OVERLAP_PREVIOUS.  A call right
        behind fill_pages8, which writes what it reads, does not."""
        if overlap_previous is None:
            overlap_previous = layer > 0 and not self._fill_before
        flags = B.C2KV_DECODE_OVERLAP_PREVIOUS if overlap_previous else 0
        if self.page8 is not None:
            self._refuse_lent_pool()
            if layer not in self.filled and 0 <= layer < self.geom.n_layers and not self._capturing(stream):
                raise ValueError(f"the pages of layer {layer} do not hold the batch's rows: fill_pages8 comes first")
            B.c2kv_attend_pages8(self.geom, layer, self.k8, self.v8, self.k_scale, self.v_scale, self.page_table,
                                 self.n_cached_dev, self.max_keys_decode, q.view(self.batch, -1, self.geom.head_dim),
                                 k_new.view(self.batch, -1, self.geom.head_dim),
                                 v_new.view(self.batch, -1, self.geom.head_dim), self.rope_table, self._rope_start,
                                 out.view(self.batch, -1, self.geom.head_dim), self.workspace8, stream,
                                 flags | B.C2KV_DECODE_ROW_AT_LENGTH)
            self._fill_before = False
            return
        B.c2kv_attend_decode(self.geom, layer, self.k_caches, self.v_caches, self.rope_tables, self.cap,
                             self.n_cached_dev, self.max_keys_decode, q, k_new, v_new, out, self.workspace,
                             stream, flags)

    def _refuse_lent_pool(self) -> None:
        seqs = self._answers()
        if seqs is not None and not seqs.released:
            raise ValueError("the pool's pages are those of the sequences that answers made: their release() comes first")

    def advance(self, stream=None) -> None:
        own = self.n_cached_dev is self._own_lengths
        B.c2kv_seq_advance(self._lengths if own else self.n_cached_dev, 1, stream)

    def answers(self, n: int = 1, room: int = 1, stream=None) -> "PagedSequences":
        """n sequences for each request, on the pool's pages: they share the composed
        cache and the question, each with room for `room` tokens of its own.  The pool
        is theirs from here on (all layers of it have to be filled): while they are there,
        fill_pages8 and decode of this batch are refused, until their release().  (The next
        composition and prefill, which write bf16 rows, are not.)"""
        if self.page8 is None:
            raise ValueError("this batch was made without page8")
        self._refuse_lent_pool()
        missing = sorted(set(range(self.geom.n_layers)) - self.filled)
        if missing:
            raise ValueError(f"the pages of layers {missing} do not hold the batch's rows: fill_pages8 comes first")
        if n < 1:
            raise ValueError("n must be at least 1")
        dev = self.page_table.device
        rows = [s + self.q_len for s in self.n_slots]
        with torch.cuda.stream(_stream_on(dev, stream)):
            held = torch.tensor([-(-r // self.page8) for r in rows], device=dev)[:, None]
            width = self.page_table.shape[1]
            mine = torch.arange(width, device=dev) < held
            seqs = PagedSequences(self.geom, self.k8, self.v8, self.k_scale, self.v_scale, self.rope_table,
                                  max_keys=self.max_keys_decode)
            seqs.page_table = torch.where(mine, self.page_table, -1).to(torch.int32)
            seqs.refs.index_add_(0, self.page_table[mine].long(), torch.ones_like(self.page_table[mine]))
            seqs.n_cached_dev = torch.tensor(rows, dtype=torch.int32, device=dev)
            seqs.rope_start = self._rope_start.clone()
        seqs.fork([b for b in range(self.batch) for _ in range(n)], room, stream)
        self.filled.clear()
        self._answers = weakref.ref(seqs)
        return seqs


class PagedSequences:
    """Sequences on the pages of a pool that they may share (RequestBatch.answers):
    parallel answers, beams, further questions.

    page_table int32 [sequences][max_pages] (-1 behind a sequence's pages),
    n_cached_dev their lengths (-1: an empty place), rope_start where a sequence's
    rows begin in rope_table, refs [n_pages] how many sequences hold each page.  A
    fork makes new tensors of them, so a graph is captured anew behind it; compact
    changes them in place.  Tokens are written to pages that `fork` has taken: its
    `room` says how many may follow before the next one.  A fork that finds too few free
    pages, no place for `room` more tokens in a row of the table, or a parent that is none
    records C2KV_EDEVICE and leaves all places empty; `restore` brings the sequences back.
    """

    def __init__(self, geom, k8: torch.Tensor, v8: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 rope_table: torch.Tensor, max_keys: int):
        self.geom, self.max_keys = geom, max_keys
        self.k8, self.v8, self.k_scale, self.v_scale, self.rope_table = k8, v8, k_scale, v_scale, rope_table
        dev = k8.device
        n_pages, self.page = k8.shape[1], k8.shape[3]
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        self.page_table = torch.full((1, -(-max_keys // self.page)), -1, dtype=torch.int32, device=dev)
        self.n_cached_dev = torch.full((1,), -1, dtype=torch.int32, device=dev)
        self.rope_start = torch.zeros(1, dtype=torch.int32, device=dev)
        # page_table, n_cached_dev and rope_start lie one behind the other, each with room for
        # as many places (the rest is -1), here and as the last fork that found a sequence found them
        self._state = self._kept = self.refs[:0]
        self._same = torch.arange(-1, n_pages, dtype=torch.int32, device=dev)
        self._parts = ()
        self._chunk_ws: List[torch.Tensor] = []   # the last one serves; captured graphs hold the others
        self._chunk_ws_held = False   # by a graph, the last one
        self._chunk_ws_stream = None  # that it was allocated on
        # zeroed here, not by a first call that may be a graph's; of a size that the
        # number of sequences does not change
        self._decode_ws = torch.zeros(B.c2kv_attend_pages8_workspace_size(geom, 1, max_keys), dtype=torch.uint8, device=dev)
        self.released = False
        self._pages_change = True   # the last call wrote pages or lengths: what reads some early waits

    @property
    def batch(self) -> int:
        return self.page_table.shape[0]

    def _pool(self):
        if self.released:
            raise ValueError("these sequences were released: the pool is the batch's again")
        return self.k8, self.v8, self.k_scale, self.v_scale

    def fork(self, parents, room: int = 1, stream=None) -> None:
        """Place i goes on with sequence parents[i] (a list, or int32 on the device;
        negative: an empty place): more answers, beams moved or dropped, sequences
        ended.  Each gets room for `room` more tokens."""
        dev = self.page_table.device
        s = self._stream(stream)
        with torch.cuda.stream(s):
            if not isinstance(parents, torch.Tensor):
                parents = torch.tensor(list(parents), dtype=torch.int32).to(dev, non_blocking=True)
            n, width = parents.numel(), self.page_table.shape[1]
            now = self._packed(n, s)
            # (all places are empty behind a fork that failed: what it found is kept)
            torch.where(self.n_cached_dev.max() >= 0, now, self._kept, out=self._kept)
            # a call that fails writes nothing: all places then stay empty
            state = torch.full_like(now, -1)
            table, lengths, rope = self._views(state, n, width)
            ws = torch.empty(B.c2kv_pages8_plan_workspace_size(self.refs.numel(), max(n, self.batch), width),
                             dtype=torch.uint8, device=dev)
            B.c2kv_pages8_fork(self.geom, *self._pool(), self.refs, self.page_table, self.n_cached_dev, parents, room,
                               self.refs, table, lengths, ws, stream)
            torch.index_select(self.rope_start, 0, parents.clamp(min=0, max=self.batch - 1), out=rope)
            self._let_go(s, self.page_table, self.n_cached_dev, self.rope_start, parents)
            self._adopt(state, n, width)
        self._pages_change = True

    def restore(self, stream=None) -> bool:
        """Behind a fork that failed (C2KV_EDEVICE): the sequences as that fork found them,
        however many steps, forks and compactions came after it.  False, and nothing is
        changed, where none has failed.  Waits for the stream."""
        s = self._stream(stream)
        with torch.cuda.stream(s):
            width = self.page_table.shape[1]
            table, lengths, rope = self._views(self._kept, None, width)
            if table.shape[0] == 0 or bool((self.n_cached_dev >= 0).any()):
                return False
            n = int((rope >= 0).sum())
            held = (table >= 0).cumprod(1).bool()
            ids = table[held].long()
            if n == 0 or bool((ids >= self.refs.numel()).any()):
                return False   # pages that are none: not of a fork
            uses = torch.bincount(ids, minlength=self.refs.numel())
            if bool((self.refs < uses).any()) or bool((held.sum(1) * self.page < lengths).any()):
                return False   # ended by a fork: their pages were given back
            self._let_go(s, self.page_table, self.n_cached_dev, self.rope_start)
            self._adopt(self._kept.clone(), n, width)
        self._pages_change = True
        return True

    @staticmethod
    def _let_go(s, *tensors) -> None:
        """These are let go while calls on the stream may still read them, and may be of other streams."""
        if s is not None and not torch.cuda.is_current_stream_capturing():
            for x in tensors:
                x.record_stream(s)

    @staticmethod
    def _views(state, n, width):
        """Page table, lengths and RoPE rows of n places (None: of all) in a state."""
        cap = state.numel() // (width + 2)
        if n is None or n == cap:
            table, lengths, rope = state.split_with_sizes((cap * width, cap, cap))
        else:
            rest = cap - n
            table, _, lengths, _, rope, _ = state.split_with_sizes((n * width, rest * width, n, rest, n, rest))
        return table.view(-1, width), lengths, rope

    def _adopt(self, state, n, width) -> None:
        self._state = state
        self._parts = self.page_table, self.n_cached_dev, self.rope_start = self._views(state, n, width)

    def _packed(self, n, s) -> torch.Tensor:
        """The present state, with room for n places; what is kept gets as much."""
        width, now = self.page_table.shape[1], (self.page_table, self.n_cached_dev, self.rope_start)
        cap = max(n, self.batch)
        if all(x is y for x, y in zip(now, self._parts)) and len(self._parts) == 3 and self._state.numel() >= cap * (width + 2):
            return self._state
        cap = max(cap, self._kept.numel() // (width + 2))

        def pack(parts):
            state = torch.full((cap * (width + 2),), -1, dtype=torch.int32, device=self.refs.device)
            for dst, src in zip(self._views(state, parts[0].shape[0], width), parts):
                dst.copy_(src)
            return state

        if self._kept.numel() < cap * (width + 2):
            self._let_go(s, self._kept)
            self._kept = pack(self._views(self._kept, None, width))
        return pack(now)

    def release(self) -> None:
        """The pool goes back to the batch that made these sequences; they take no more calls."""
        self.released = True

    def compact(self, stream=None) -> None:
        """The pages in use to the front of the pool."""
        with torch.cuda.stream(self._stream(stream)):
            width = self.page_table.shape[1]
            ws = torch.empty(B.c2kv_pages8_plan_workspace_size(self.refs.numel(), self.batch, width),
                             dtype=torch.uint8, device=self.refs.device)
            to = self._same.clone()   # where page i is, in place 1 + i; -1 in place 0 and of free pages
            B.c2kv_pages8_compact(self.geom, *self._pool(), self.refs, self.page_table, self.refs, self.page_table,
                                  to[1:], ws, stream)
            kept = self._views(self._kept, None, width)[0].view(-1)   # what a failed fork found has moved, too
            torch.index_select(to, 0, torch.clamp(kept, -1, to.numel() - 2).add_(1), out=kept)
        self._pages_change = True

    def chunk(self, layer: int, q, k_new, v_new, out, n_new: Optional[torch.Tensor] = None, stream=None) -> None:
        """Attention of t_len new tokens of each sequence (q, out [batch][t_len][n_q_heads]
        [head_dim]) over its pages, their append included; n_new: int32 [batch], the
        tokens of a padded batch."""
        need = B.c2kv_attend_pages8_chunk_workspace_size(self.geom, self.batch, q.shape[1], self.max_keys)
        B.c2kv_attend_pages8_chunk(self.geom, layer, *self._pool(), self.page_table, self.n_cached_dev, self.max_keys, q,
                                   k_new, v_new, self.rope_table, self.rope_start, out, self._chunk_workspace(need, stream),
                                   n_new, stream, B.C2KV_DECODE_ROW_AT_LENGTH)
        self._pages_change = True

    def _chunk_workspace(self, need: int, stream) -> torch.Tensor:
        """Scratch of at least `need` bytes for a call on this stream.  One that has become too
        small is let go, unless a captured graph works on it."""
        s = self._stream(stream)
        with torch.cuda.stream(s):
            if not self._chunk_ws or self._chunk_ws[-1].numel() < need:
                if self._chunk_ws:
                    need = max(need, self._chunk_ws[-1].numel() * 3 // 2)   # so few of them, whatever is asked for
                    if not self._chunk_ws_held:
                        self._chunk_ws.pop()
                self._chunk_ws.append(torch.empty(need, dtype=torch.uint8, device=self.refs.device))
                self._chunk_ws_held, self._chunk_ws_stream = False, s
            ws = self._chunk_ws[-1]
            if s is not None:
                if torch.cuda.is_current_stream_capturing():
                    self._chunk_ws_held = True
                elif s != self._chunk_ws_stream:
                    ws.record_stream(s)
        return ws

    def decode(self, layer: int, q, k_new, v_new, out, stream=None, overlap_previous: Optional[bool] = None) -> None:
        """One token of each sequence, as RequestBatch.decode over pages."""
        if overlap_previous is None:
            overlap_previous = layer > 0 and not self._pages_change
        d = self.geom.head_dim
        B.c2kv_attend_pages8(self.geom, layer, *self._pool(), self.page_table, self.n_cached_dev, self.max_keys,
                             q.view(self.batch, -1, d), k_new.view(self.batch, -1, d), v_new.view(self.batch, -1, d),
                             self.rope_table, self.rope_start, out.view(self.batch, -1, d), self._decode_ws, stream,
                             (B.C2KV_DECODE_OVERLAP_PREVIOUS if overlap_previous else 0) | B.C2KV_DECODE_ROW_AT_LENGTH)
        self._pages_change = False

    def advance(self, stream=None, n=1) -> None:
        """The lengths by n tokens: a number, or int32 [batch] (the n_new of a chunk).
        Empty places stay empty."""
        with torch.cuda.stream(self._stream(stream)):
            self.n_cached_dev.add_(torch.where(self.n_cached_dev >= 0, n, 0).to(torch.int32))
        self._pages_change = True

    def _stream(self, stream):
        return _stream_on(self.refs.device, stream)


class DecoderModel:
    """A synthetic-weight decoder stack around a RequestBatch's attention, on
    the device (C2KV explainer, section "the problem", Fig. 1: the decode rate
    of the whole model).  The layer is the Llama-3 one (no biases):
        h = rmsnorm(x) * w_attn; q | k | v = h W_qkv^T (split by the epilogue)
        x += attention(q, k, v) W_o^T          (the batch's composed caches)
        h = rmsnorm(x) * w_mlp;  x += (silu(h W_g^T) * h W_u^T) W_d^T
    then rmsnorm and the LM head.  Every step is a C-ABI call; launches after
    the first may overlap the tail of the one before (programmatic dependent
    launch): each kernel touches its activations only after the previous one
    has finished.

    weights: dict as synth.make_decoder_weights, values device bf16 tensors.
    """

    def __init__(self, geom, shape, weights: dict, batch: int, device: str = "cuda", top_k: int = 0):
        self.geom, self.shape, self.w = geom, shape, weights
        self.batch = batch
        d = geom.head_dim
        self.nq, self.nkv = geom.n_q_heads * d, geom.n_kv_heads * d
        nb, dim, F = batch, shape.dim, shape.ffn
        bf = torch.bfloat16

        def buf(*sz):
            return torch.zeros(sz, dtype=bf, device=device)

        self.x, self.h = buf(nb, dim), buf(nb, dim)
        self.q, self.k, self.v = buf(nb, self.nq), buf(nb, self.nkv), buf(nb, self.nkv)
        self.att, self.m = buf(nb, self.nq), buf(nb, F)
        has_head = "lm_head" in weights
        self.logits = buf(nb, shape.vocab) if has_head else None
        # token_logprobs' results
        self.logprob, self.entropy = (torch.zeros(nb, device=device) for _ in range(2))
        self.top_ids = torch.zeros((nb, top_k), dtype=torch.int32, device=device)
        self.top_logprobs = torch.zeros((nb, top_k), device=device)
        widest = max(self.nq + 2 * self.nkv, 2 * F, dim, shape.vocab if has_head else 0)
        self.workspace = torch.zeros(B.c2kv_linear_workspace_size(nb, widest), dtype=torch.uint8, device=device)
        B.c2kv_workspace_init(self.workspace)

    def layer(self, l: int, rb: "RequestBatch", stream=None) -> None:
        w = self.w["layers"][l]
        ov = B.C2KV_LINEAR_OVERLAP_PREVIOUS
        eps = self.shape.eps
        B.c2kv_rmsnorm(self.x, w["attn_norm"], self.h, eps, stream, ov)
        B.c2kv_linear(self.h, w["qkv"], self.q, self.workspace, B.C2KV_LINEAR_SPLIT3, y2=self.k, y3=self.v,
                       split1=self.nq, split2=self.nq + self.nkv, stream=stream, flags=ov)
        rb.decode(l, self.q, self.k, self.v, self.att, stream, overlap_previous=True)
        B.c2kv_linear(self.att, w["o"], self.x, self.workspace, B.C2KV_LINEAR_ADD, residual=self.x,
                       stream=stream, flags=ov)
        B.c2kv_rmsnorm(self.x, w["mlp_norm"], self.h, eps, stream, ov)
        B.c2kv_linear(self.h, w["gate_up"], self.m, self.workspace, B.C2KV_LINEAR_SWIGLU, stream=stream,
                       flags=ov)
        B.c2kv_linear(self.m, w["down"], self.x, self.workspace, B.C2KV_LINEAR_ADD, residual=self.x,
                       stream=stream, flags=ov)

    def decode_step(self, rb: "RequestBatch", stream=None) -> None:
        """One answer token per sequence: every layer, the LM head (if the
        weights have one), then the batch's lengths advance.  x holds the
        step's input embeddings and is updated in place."""
        for l in range(len(self.w["layers"])):
            self.layer(l, rb, stream)
        if self.logits is not None:
            B.c2kv_rmsnorm(self.x, self.w["final_norm"], self.h, self.shape.eps, stream,
                            B.C2KV_LINEAR_OVERLAP_PREVIOUS)
            B.c2kv_linear(self.h, self.w["lm_head"], self.logits, self.workspace, stream=stream,
                           flags=B.C2KV_LINEAR_OVERLAP_PREVIOUS)
        rb.advance(stream)

    def token_logprobs(self, tokens: torch.Tensor, stream=None) -> None:
        """Of the last step's logits: logprob of tokens [batch] (int32 on the
        device; negative: none), entropy, and the top_k alternatives in top_ids
        and top_logprobs."""
        if self.logits is None:
            raise ValueError("the model's weights have no lm_head: there are no logits")
        B.c2kv_token_logprobs(self.logits, tokens, self.top_ids.shape[1], self.logprob, self.entropy, self.top_ids,
                              self.top_logprobs, stream)

    def linears_only(self, stream=None) -> None:
        """The step's linear layers and norms without the attention (their
        own weight-streaming rate, for the roofline)."""
        ov = B.C2KV_LINEAR_OVERLAP_PREVIOUS
        eps = self.shape.eps
        for w in self.w["layers"]:
            B.c2kv_rmsnorm(self.x, w["attn_norm"], self.h, eps, stream, ov)
            B.c2kv_linear(self.h, w["qkv"], self.q, self.workspace, B.C2KV_LINEAR_SPLIT3, y2=self.k,
                           y3=self.v, split1=self.nq, split2=self.nq + self.nkv, stream=stream, flags=ov)
            B.c2kv_linear(self.att, w["o"], self.x, self.workspace, B.C2KV_LINEAR_ADD, residual=self.x,
                           stream=stream, flags=ov)
            B.c2kv_rmsnorm(self.x, w["mlp_norm"], self.h, eps, stream, ov)
            B.c2kv_linear(self.h, w["gate_up"], self.m, self.workspace, B.C2KV_LINEAR_SWIGLU, stream=stream,
                           flags=ov)
            B.c2kv_linear(self.m, w["down"], self.x, self.workspace, B.C2KV_LINEAR_ADD, residual=self.x,
                           stream=stream, flags=ov)
        if self.logits is not None:
            B.c2kv_rmsnorm(self.x, self.w["final_norm"], self.h, self.shape.eps, stream, ov)
            B.c2kv_linear(self.h, self.w["lm_head"], self.logits, self.workspace, stream=stream, flags=ov)

    def weight_bytes(self) -> int:
        n = sum(t.numel() for w in self.w["layers"] for t in w.values())
        if self.logits is not None:
            n += self.w["lm_head"].numel() + self.w["final_norm"].numel()
        return 2 * n
