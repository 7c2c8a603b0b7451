"""Python front end of what surrounds the verified context: per-head norms with the position
rotation, and a paged cache, in 16 or in 4 bits, for tokens that have no place in the compressed context
-- those decoded since, and prompts that a batch shares -- from which those of least attention weight can
be evicted.  PyTorch allocates the memory and supplies the stream; the work is libverkv's (verkv_norm_rotate, verkv_paged_append, verkv_paged_attend,
verkv_paged_values, verkv_paged_weigh, verkv_paged_evict).

    rope = Rope(inv_freq)                                     # float64 frequencies, once
    cache = PagedKV(kv_heads, q_per_kv, head_dim, num_pages=..., layers=...)
    q = cache.append(layer, k, v, seq, index, table, positions=pos, rope=rope, q=q, ...)
    o, lse = cache.attend(layer, q, table, lengths, max_length, prior=(eng.o, eng.lse))
    cache.weigh(layer, q, lse, table, lengths, max_length, weights[layer])     # who is looked at
    cache.evict(layer, table, lengths, max_length, weights[layer], keep=2048)  # now and then
"""
import torch

from . import binding as B

# The current stream's handle without a Stream object around it, where torch offers that.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing

# New CUDA tensors by a call that goes past the dispatcher, whose code a launch has driven out of the host's caches
# (behind one torch.empty takes 5 to 7 us, this 3), where torch offers that and nobody has changed what torch.empty does:
# it passes by dispatch modes, which may count or replace tensors, and by the filling of deterministic algorithms.
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
_dispatch_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
_deterministic = getattr(torch._C, "_get_deterministic_algorithms", None)
if _dispatch_modes is None or _deterministic is None:
    _empty_strided = None
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

_DTYPES = {torch.bfloat16: B.VERKV_BF16, torch.float16: B.VERKV_F16}
_PACKED = {torch.bfloat16: B.VERKV_BF16_Q4, torch.float16: B.VERKV_F16_Q4}


class Rope:
    """The rotation of the first 2 * len(inv_freq) channels: pair j turns by position * inv_freq[j]
    (float64 values; whatever scaling a model gives its frequencies is in them).  interleaved: pairs
    are neighbours, else rotary_dim / 2 channels apart."""

    def __init__(self, inv_freq, interleaved=False, device=None):
        f = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").reshape(-1).tolist()
        self.dev = torch.device("cuda" if device is None else device)
        if self.dev.index is None:
            self.dev = torch.device("cuda", torch.cuda.current_device())
        turns = torch.frombuffer(B.verkv_rope_turns(f), dtype=torch.int64) if f else torch.empty(0, dtype=torch.int64)
        self.turns = turns.to(self.dev)
        self.desc = B.verkv_rope(2 * len(f), int(bool(interleaved)), self.turns.data_ptr())


class PagedKV:
    """A pool of pages [layers][num_pages][kv_heads][page_tokens][2][head_dim] and the calls on it.
    With bits=4 pages hold 4-bit codes with a floor and a step for every 32 channels (include/verkv.h
    has the layout), a pool is uint8 [layers][num_pages][kv_heads][page_tokens / 16][2][10 head_dim],
    0.31 of a 16-bit one's bytes, and dtype is that of the queries, keys and values.
    Work is issued on the stream that is current when the object is made; a call made while another
    is current is refused.  One object's calls share its workspace: graphs that may run at the same
    time need an object each (kv= adopts an existing pool), and a graph needs its object as long as it
    is replayed.  With num_pages=0 it has no pool and only norm_rotate."""

    def __init__(self, kv_heads, q_per_kv, head_dim, page_tokens=64, num_pages=0, layers=1,
                 dtype=torch.bfloat16, device=None, kv=None, bits=16):
        self.ctx = None
        if bits not in (4, 16):
            raise ValueError("bits: 16 or 4")
        if bits == 4 and kv is None and page_tokens % 16:
            raise ValueError("page_tokens: 16, 32, 64, 128 or 256")
        if kv is not None and bits == 4:
            if kv.dim() != 6 or kv.shape[2] != kv_heads or kv.shape[4] != 2 or kv.shape[5] != 10 * head_dim or kv.dtype is not torch.uint8:
                raise ValueError("kv: uint8 [layers][pages][kv_heads][page_tokens / 16][2][10 head_dim] is required")
            if not kv.is_cuda or not kv.is_contiguous():
                raise ValueError("kv: a contiguous CUDA tensor is required")
            device = kv.device
            layers, num_pages, page_tokens = kv.shape[0], kv.shape[1], kv.shape[3] * 16
        elif kv is not None:
            if kv.dim() != 6 or kv.shape[2] != kv_heads or kv.shape[4] != 2 or kv.shape[5] != head_dim:
                raise ValueError("kv: [layers][pages][kv_heads][page_tokens][2][head_dim] is required")
            if not kv.is_cuda or not kv.is_contiguous():
                raise ValueError("kv: a contiguous CUDA tensor is required")
            dtype, device = kv.dtype, kv.device
            layers, num_pages, page_tokens = kv.shape[0], kv.shape[1], kv.shape[3]
        if dtype not in _DTYPES:
            raise ValueError("dtype: torch.bfloat16 or torch.float16")
        self.dev = torch.device("cuda" if device is None else device)
        if self.dev.index is None:
            self.dev = torch.device("cuda", torch.cuda.current_device())
        self.dtype, self.h, self.hq, self.d = dtype, kv_heads, kv_heads * q_per_kv, head_dim
        self.layers = layers
        self.shape = B.verkv_shape(1, 1, kv_heads, q_per_kv, head_dim, 1, 1)
        ws = B.verkv_workspace_size(self.shape)
        if ws == 0:
            raise B.VerkvError(B.VERKV_EINVAL, "invalid shape")
        if kv is None and num_pages > 0:
            if bits == 4:
                kv = torch.zeros((layers, num_pages, kv_heads, page_tokens // 16, 2, 10 * head_dim), dtype=torch.uint8, device=self.dev)
            else:
                kv = torch.zeros((layers, num_pages, kv_heads, page_tokens, 2, head_dim), dtype=dtype, device=self.dev)
        self.kv = kv
        self._base = kv.data_ptr() if kv is not None else 0
        self.bits = bits
        self._layer_bytes = num_pages * kv_heads * page_tokens * 4 * head_dim * (10 if bits == 4 else 32) // 32
        self._code = _DTYPES[dtype]
        self._pages = B.verkv_pages(_PACKED[dtype] if bits == 4 else self._code, page_tokens, num_pages, self._base)
        with torch.cuda.device(self.dev):
            self.stream = torch.cuda.current_stream(self.dev)
            self._ctx_ws = torch.empty(ws, dtype=torch.uint8, device=self.dev)
            self.ctx = B.verkv_create(self.dev.index, self.stream.cuda_stream, self.shape,
                                      self._ctx_ws.data_ptr(), ws)
        self._raw_stream = self.stream.cuda_stream
        self._index, self._lib = self.dev.index, B.lib()
        # Workspaces of attend and evict, the one in use last: those before it are held by captured graphs.  And how
        # many bytes each size of call needs.
        self._spaces, self._needs = [], {}
        self._space_at, self._space_bytes, self._space_held = None, 0, True

    # --------------------------------------------------------------------------------------------
    # Checks and descriptors.  A decode step makes these calls once a layer, so they take the tensors'
    # attributes once each and call the library directly.
    def _ready(self):
        if _current_stream(self._index) != self._raw_stream:
            raise ValueError("another stream is current than the one this object was made on")

    def _empty(self, shape, dtype):
        if _empty_strided is None or _dispatch_modes() or _deterministic() or min(shape) < 1 or _current_device() != self._index:
            return torch.empty(shape, dtype=dtype, device=self.dev)
        if len(shape) == 3:
            return _empty_strided(shape, (shape[1] * shape[2], shape[2], 1), dtype)
        strides = [1]
        for size in shape[:0:-1]:
            strides.append(strides[-1] * size)
        return _empty_strided(shape, tuple(strides[::-1]), dtype)

    def _fail(self, status):
        raise B.VerkvError(status, B.verkv_last_error(self.ctx))

    def _rows(self, t, tokens, heads, name):
        s = t.shape
        if t.dtype is not self.dtype or t.device != self.dev or len(s) != 3 or s[0] != tokens or s[1] != heads or s[2] != self.d:
            raise ValueError(f"{name}: a {self.dtype} tensor [{tokens}][{heads}][{self.d}] on {self.dev} is required")
        a, b, c = t.stride()
        if c != 1 and tokens:
            raise ValueError(f"{name}: channels must be contiguous")
        return B.verkv_rows(t.data_ptr(), a if tokens > 1 else 0, b if heads > 1 else 0)

    def _out(self, out, tokens, heads, name):
        """An output of the caller's, or a new one: the tensor and its descriptor."""
        if out is not None:
            return out, self._rows(out, tokens, heads, name)
        d = self.d
        out = self._empty((tokens, heads, d), self.dtype)
        return out, B.verkv_rows(out.data_ptr(), heads * d, d)

    def _ints(self, t, shape, name):
        if t.dtype is not torch.int32 or t.device != self.dev or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous int32 {list(shape)} tensor on {self.dev} is required")
        return t.data_ptr()

    def _table(self, t, name):
        s = t.shape
        if len(s) != 2:
            raise ValueError(f"{name}: an int32 tensor of page ids [rows][pages] is required")
        return self._ints(t, s, name), s[0], s[1]

    def _weight(self, t, name):
        if t is None:
            return None
        if t.dtype is not self.dtype or t.device != self.dev or t.shape != (self.d,) or not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous {self.dtype} [{self.d}] tensor on {self.dev} is required")
        return t.data_ptr()

    def _norm(self, q_weight, k_weight, eps):
        if q_weight is None and k_weight is None:
            return None
        return B.verkv_head_norm(self._weight(q_weight, "q_weight"), self._weight(k_weight, "k_weight"), eps)

    def _turn(self, rope, positions, tokens):
        """Descriptor of the rotation and address of the positions."""
        if rope is None:
            return None, None
        if rope.dev != self.dev:
            raise ValueError(f"rope: made for {rope.dev}, not {self.dev}")
        if positions is None:
            raise ValueError("positions: needed for a rotation")
        return rope.desc, self._ints(positions, (tokens,), "positions")

    def _layer(self, layer):
        if self.kv is None:
            raise ValueError("this object has no pages")
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer: 0 .. {self.layers - 1}")
        self._pages.kv = self._base + layer * self._layer_bytes
        return self._pages

    # --------------------------------------------------------------------------------------------
    def norm_rotate(self, q, k, positions=None, rope=None, q_weight=None, k_weight=None, eps=1e-6,
                    q_out=None, k_out=None):
        """rotate(norm(q)) and rotate(norm(k)): q [tokens][heads][head_dim] and k
        [tokens][kv_heads][head_dim], either None, with any token and head strides of whole 16
        bytes.  An output may be the input itself; by default it is new.  A weight of None leaves
        those heads as long as they are.  Returns (q_out, k_out)."""
        self._ready()
        if q is None and k is None:
            raise ValueError("q or k is required")
        if (q is None and q_out is not None) or (k is None and k_out is not None):
            raise ValueError("an output is given without its input")
        tokens = (k if q is None else q).shape[0]
        rq = ro = rk = rl = None
        if q is not None:
            rq = self._rows(q, tokens, self.hq, "q")
            q_out, ro = self._out(q_out, tokens, self.hq, "q_out")
        if k is not None:
            rk = self._rows(k, tokens, self.h, "k")
            k_out, rl = self._out(k_out, tokens, self.h, "k_out")
        turn, pos = self._turn(rope, positions, tokens)
        norm = self._norm(q_weight, k_weight, eps)
        st = self._lib.verkv_norm_rotate(self.ctx, self._code, tokens, rq, ro, rk, rl, norm, turn, pos)
        if st:
            self._fail(st)
        return q_out, k_out

    def append(self, layer, k, v, seq, index, table, positions=None, rope=None, k_weight=None,
               eps=1e-6, q=None, q_weight=None, q_out=None):
        """Append tokens to the pages of their sequences: token t of k and v
        [tokens][kv_heads][head_dim] becomes token index[t] of sequence seq[t] (-1: padding, nothing
        is written), page table[seq[t]][index[t] // page_tokens]; k is normalised and rotated on the
        way, and q [tokens][heads][head_dim] in the same launch if it is given.  seq, index and
        positions: int32 [tokens]; table: int32 [sequences][pages].  Returns q_out (None without q)."""
        self._ready()
        tokens = k.shape[0]
        rk, rv = self._rows(k, tokens, self.h, "k"), self._rows(v, tokens, self.h, "v")
        rq = ro = None
        if q is not None:
            rq = self._rows(q, tokens, self.hq, "q")
            q_out, ro = self._out(q_out, tokens, self.hq, "q_out")
        elif q_out is not None:
            raise ValueError("q_out: given without q")
        at, rows, stride = self._table(table, "table")
        turn, pos = self._turn(rope, positions, tokens)
        norm = self._norm(q_weight if q is not None else None, k_weight, eps)
        ps, pi = self._ints(seq, (tokens,), "seq"), self._ints(index, (tokens,), "index")
        st = self._lib.verkv_paged_append(self.ctx, self._layer(layer), tokens, rk, rv, rq, ro, norm, turn, pos, ps, pi,
                                          B.verkv_span(at, rows, stride, None, 0))
        if st:
            self._fail(st)
        return q_out

    def attend(self, layer, q, table, lengths, max_length, q_start=None, prefix_table=None,
               prefix_lengths=None, max_prefix=0, group_start=None, scale=0.0, prior=None, out=None,
               lse=None):
        """Attention of q [queries][heads][head_dim] over each sequence's own tokens and, where it
        is given, the prefix its group shares.

        table, lengths: int32 [sequences][pages] and [sequences] of the own tokens, max_length a
        bound of the lengths known here (both None: no own tokens).  q_start: int32
        [sequences + 1], sequence s has the queries q_start[s] .. q_start[s + 1] - 1, which are its
        last tokens; None: one query each.  prefix_table, prefix_lengths, max_prefix: the same of
        the shared prefixes; group_start: int32 [prefixes + 1] of sequences, None with one prefix.
        scale: of the logits, 0 for 1 / sqrt(head_dim).  prior: (o, lse) float32 of attention over
        other tokens (VerKV.fetch_refine's, say), joined to the result.

        Returns (o [queries][heads][head_dim] of the pool's type, lse float32 [queries][heads])."""
        self._ready()
        tokens, hq, dev = q.shape[0], self.hq, self.dev
        rq = self._rows(q, tokens, hq, "q")
        own = prefix = ps = pg = po = pl = None
        groups = 0
        if (table is None) != (lengths is None) or (prefix_table is None) != (prefix_lengths is None):
            raise ValueError("a table and its lengths come together")
        if table is not None:
            at, n, stride = self._table(table, "table")
            if n:
                own = B.verkv_span(at, n, stride, self._ints(lengths, (n,), "lengths"), max_length)
        else:
            n = tokens if q_start is None else q_start.shape[0] - 1
        if q_start is not None:
            ps = self._ints(q_start, (n + 1,), "q_start")
        if prefix_table is not None:
            at, groups, stride = self._table(prefix_table, "prefix_table")
            prefix = B.verkv_span(at, groups, stride, self._ints(prefix_lengths, (groups,), "prefix_lengths"), max_prefix)
        if group_start is not None:
            pg = self._ints(group_start, (groups + 1,), "group_start")
        if prior is not None:
            o, l = prior
            for t, size, name in ((o, tokens * hq * self.d, "prior o"), (l, tokens * hq, "prior lse")):
                if t.dtype is not torch.float32 or t.device != dev or t.numel() != size or not t.is_contiguous():
                    raise ValueError(f"{name}: a contiguous float32 tensor of {size} values on {dev} is required")
            po, pl = o.data_ptr(), l.data_ptr()
        shape = (tokens, hq, self.d)
        if out is None:
            out = self._empty(shape, self.dtype)
        elif out.dtype is not self.dtype or out.device != dev or out.shape != shape or not out.is_contiguous():
            raise ValueError(f"out: a contiguous {self.dtype} {list(shape)} tensor on {dev} is required")
        if lse is None:
            lse = self._empty((tokens, hq), torch.float32)
        elif lse.dtype is not torch.float32 or lse.device != dev or lse.shape != (tokens, hq) or not lse.is_contiguous():
            raise ValueError(f"lse: a contiguous float32 [{tokens}][{hq}] tensor on {dev} is required")
        pages = self._layer(layer)
        if not tokens:
            return out, lse
        ws, nbytes = self._space(n, groups, tokens)
        st = self._lib.verkv_paged_attend(self.ctx, pages, n, tokens, rq, ps, own, prefix, pg, scale, po, pl,
                                          out.data_ptr(), lse.data_ptr(), ws, nbytes)
        if st:
            self._fail(st)
        return out, lse

    def values(self, layer, out=None):
        """The values that a layer of a 4-bit pool stands for: [num_pages][kv_heads][page_tokens][2][head_dim]
        of the rows' type, rounded once."""
        self._ready()
        pages = self._layer(layer)
        if self.bits != 4:
            raise ValueError("values: of a pool of 4-bit pages")
        shape = (pages.num_pages, self.h, pages.page_tokens, 2, self.d)
        if out is None:
            out = self._empty(shape, self.dtype)
        elif out.dtype is not self.dtype or out.device != self.dev or out.shape != shape or not out.is_contiguous():
            raise ValueError(f"out: a contiguous {self.dtype} {list(shape)} tensor on {self.dev} is required")
        st = self._lib.verkv_paged_values(self.ctx, pages, out.data_ptr())
        if st:
            self._fail(st)
        return out

    def _weights(self, t, shape, name):
        if t.dtype is not torch.float32 or t.device != self.dev or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous float32 {list(shape)} tensor on {self.dev} is required")
        return t.data_ptr()

    def _places(self, seqs, places, max_length):
        """Sizes as the library takes them: of 32 bits, and with room for the lengths (of any sequences)."""
        if seqs and not 0 <= max_length <= places <= 1 << 30:
            raise ValueError(f"places: as many as max_length ({max_length}) or more, and at most 2^30, are required")

    def _apart(self, a, b, shape):
        """Weights at a and at b: in one place, or without an overlap.  Returns b."""
        if a != b and abs(a - b) < 4 * shape[0] * shape[1] * shape[2]:
            raise ValueError("out: overlaps weights, but is not the same")
        return b

    def weigh(self, layer, q, lse, table, lengths, max_length, weights=None, out=None, q_start=None, scale=0.0):
        """The attention weight that each sequence's own cached tokens get from the queries q
        [queries][heads][head_dim], added up over queries and a KV head's query heads: exp(logit - lse),
        with lse float32 [queries][heads] as attend has returned it for these queries (over prefixes and a
        prior too).

        table, lengths, max_length, q_start, scale: as in attend.  weights: float32
        [sequences][kv_heads][places] with max_length places or more, the sums so far, None for zeros.
        out: the new sums, by default in weights' place (places behind a length stay as they are), or,
        without weights, a new tensor of max_length places.  Returns out."""
        self._ready()
        tokens, hq = q.shape[0], self.hq
        rq = self._rows(q, tokens, hq, "q")
        at, n, stride = self._table(table, "table")
        own = B.verkv_span(at, n, stride, self._ints(lengths, (n,), "lengths"), max_length)
        ps = self._ints(q_start, (n + 1,), "q_start") if q_start is not None else None
        if lse.dtype is not torch.float32 or lse.device != self.dev or lse.shape != (tokens, hq) or not lse.is_contiguous():
            raise ValueError(f"lse: a contiguous float32 [{tokens}][{hq}] tensor on {self.dev} is required")
        if out is None and weights is None:
            self._places(n, max_length, max_length)
            out = self._empty((n, self.h, max_length), torch.float32)
        elif out is None:
            out = weights
        shape = out.shape
        if len(shape) != 3:
            raise ValueError("out: a float32 tensor [sequences][kv_heads][places] is required")
        shape = (n, self.h, shape[2])
        self._places(n, shape[2], max_length)
        po = self._weights(out, shape, "out")
        pi = None
        if weights is not None:
            pi = po if weights is out else self._apart(po, self._weights(weights, shape, "weights"), shape)
        pages = self._layer(layer)
        if not n and tokens:
            raise ValueError("queries of no sequence")
        if not n or not shape[2]:
            return out
        st = self._lib.verkv_paged_weigh(self.ctx, pages, n, tokens, rq, ps, own, scale, lse.data_ptr(), pi, po, shape[2])
        if st:
            self._fail(st)
        return out

    def evict(self, layer, table, lengths, max_length, weights, keep, first=4, last=32, out=None, kept=None):
        """Evict tokens: each KV head of a sequence with more than `keep` of them keeps the first, the last
        and, between, those with the largest weights (float32 [sequences][kv_heads][places], as weigh adds
        them up).  Their rows move together in the sequence's pages, none of which may stand twice in the call's
        tables up to the lengths; afterwards every sequence has min(length, keep) tokens, and the caller sets the lengths once
        every layer's call is made.  From then on a token's place is not its position: append's index goes on from
        the new lengths, its positions from the old ones.  out: the weights in their tokens' new places, 0 behind them; by default
        in weights' place.

        Returns (out, kept): kept int32 [sequences][kv_heads][keep] is the former place of the token that
        now has this one, -1 behind the last."""
        self._ready()
        at, n, stride = self._table(table, "table")
        own = B.verkv_span(at, n, stride, self._ints(lengths, (n,), "lengths"), max_length)
        shape = weights.shape
        if len(shape) != 3:
            raise ValueError("weights: a float32 tensor [sequences][kv_heads][places] is required")
        shape = (n, self.h, shape[2])
        self._places(n, shape[2], max_length)
        pi = po = self._weights(weights, shape, "weights")
        if out is None:
            out = weights
        elif out is not weights:
            po = self._apart(pi, self._weights(out, shape, "out"), shape)
        if not 1 <= keep < 1 << 31:
            raise ValueError("keep: 1 or more")
        if n and (first < 0 or last < 0 or first + last > keep):
            raise ValueError("keep: must hold the first and the last")
        if kept is None:
            kept = self._empty((n, self.h, keep), torch.int32)
            pk = kept.data_ptr()
        else:
            pk = self._ints(kept, (n, self.h, keep), "kept")
        pages = self._layer(layer)
        if not n:
            return out, kept
        if not shape[2]:  # no places, and so no tokens: kept alone is written
            pi = po = pk
        key = ("evict", n, max_length, keep)
        need = self._needs.get(key)
        if need is None:
            need = self._known(key, B.verkv_paged_evict_workspace_size(self.shape, n, max_length, keep))
        ws, nbytes = self._room(need)
        st = self._lib.verkv_paged_evict(self.ctx, pages, n, own, keep, first, last, pi, po, shape[2], pk, ws, nbytes)
        if st:
            self._fail(st)
        return out, kept

    def _space(self, seqs, groups, tokens):
        key = (seqs, groups, tokens)
        need = self._needs.get(key)
        if need is None:
            need = self._known(key, B.verkv_paged_workspace_size(self.shape, seqs, groups, tokens))
        return self._room(need)

    def _known(self, key, need):
        """Remembers how many bytes of workspace a size of call needs (0: it is out of range)."""
        if need == 0:
            raise B.VerkvError(B.VERKV_EINVAL, "too many sequences, prefixes or queries, or another size out of range")
        if len(self._needs) >= 4096:
            self._needs.clear()
        self._needs[key] = need
        return need

    def _room(self, need):
        """A workspace of that many bytes."""
        if need > self._space_bytes:
            if not self._space_held:
                self._spaces.pop()
            # by half at least: calls that grow one by one make few of them
            size = max(need, self._space_bytes + self._space_bytes // 2)
            self._spaces.append(torch.empty(size, dtype=torch.uint8, device=self.dev))
            self._space_at, self._space_bytes, self._space_held = self._spaces[-1].data_ptr(), size, False
        if not self._space_held and _capturing():
            self._space_held = True
        return self._space_at, self._space_bytes

    def sync(self):
        """Wait, and raise what the device has reported since the last call."""
        B.verkv_sync(self.ctx)

    def close(self):
        if self.ctx is not None:
            B.verkv_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 -- interpreter shutdown
            pass
