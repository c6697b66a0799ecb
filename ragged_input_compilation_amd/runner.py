"""Step driver: runs one workload through libric with PyTorch-owned device
memory and streams.

PyTorch supplies device buffers (workspace, K/V sources, caches, hidden
states) and the stream; every step computation is a libric call.  The driver
only sequences the calls: load the request history into the persistent batch
(adds, removals, condense, refills), schedule, compile, write K/V for every
layer, gather hidden rows."""
from __future__ import annotations

import contextlib
import os
from dataclasses import dataclass
from typing import List, Optional

import numpy as np
import torch

from . import _ric as ric

_TORCH_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
DEBUG = os.environ.get("RIC_DEBUG", "") not in ("", "0")


def config_of(w) -> ric.ric_config:
    return ric.make_config(max_num_reqs=w.max_num_reqs, max_model_len=w.max_model_len,
                           block_size=w.block_size, max_blocks_per_req=w.max_blocks_per_req,
                           max_num_batched_tokens=w.max_num_batched_tokens,
                           num_kv_blocks=w.num_kv_blocks, null_block=w.null_block, staging_bytes=0)


def current_stream() -> int:
    return int(torch.cuda.current_stream().cuda_stream)


class Batch:
    """A libric handle whose workspace is a torch tensor."""

    def __init__(self, cfg: ric.ric_config, device="cuda", stream: Optional[int] = None):
        self.cfg = cfg
        self.stream = current_stream() if stream is None else stream
        nbytes = ric.ric_workspace_bytes(cfg)
        if nbytes == 0:
            raise ric.RicError(ric.RIC_EINVAL, ric.ric_last_error())
        # torch's caching allocator returns blocks aligned to at least 512 bytes
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.h = ric.ric_create(cfg, self.stream, self.workspace.data_ptr(), nbytes)

    def close(self):
        if self.h:
            ric.ric_destroy(self.h)
            self.h = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # history -------------------------------------------------------------
    def add(self, r) -> int:
        return ric.ric_add_request(self.h, r.req_id, r.tokens, r.num_prompt, r.num_computed, r.blocks,
                                   (r.temperature, r.top_p, r.rep_penalty, r.top_k))

    def load_history(self, w) -> int:
        """Add the initial requests, remove the finished ones, condense, add the
        refills.  Returns the number of rows condense moved."""
        for r in w.initial:
            self.add(r)
        for rid in w.finished:
            ric.ric_remove_request(self.h, rid)
        moved = ric.ric_condense(self.h) if w.finished else 0
        for r in w.refill:
            self.add(r)
        ric.ric_flush(self.h)
        return moved

    def row_order(self) -> List[int]:
        n = ric.ric_num_reqs(self.h)
        return [ric.ric_req_at(self.h, i) for i in range(n)]

    def schedule_from(self, w, order: Optional[List[int]] = None) -> None:
        """Schedule every live request with its workload (c, q), rows in
        ``order`` (request ids by row; default: the handle's own rows)."""
        order = self.row_order() if order is None else order
        by_id = w.by_id()
        ric.ric_schedule(self.h, [by_id[i].num_computed for i in order], [by_id[i].num_scheduled for i in order])

    def compile(self, n_pad: int) -> ric.ric_step:
        s = ric.ric_compile(self.h, n_pad)
        if DEBUG:
            self.debug_dump(s)
        return s

    def slot_collisions(self, s: ric.ric_step) -> tuple:
        """(collisions, out-of-range slots) among the step's real tokens, by
        the library's device-side check (debugging; synchronises)."""
        res = torch.zeros(2, dtype=torch.int32, device=self.workspace.device)
        num_slots = self.cfg.num_kv_blocks * self.cfg.block_size
        if num_slots <= ric.RIC_CHECK_SLOTS_NOALLOC_MAX_SLOTS:
            ric.ric_check_slots_noalloc(s.slot_mapping, s.num_tokens_padded, num_slots, res.data_ptr(),
                                        dev_num_tokens=s.dev_scalars + 4, stream=self.stream)
        else:
            nbytes = ric.ric_check_slots_workspace_bytes(num_slots)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.workspace.device)
            ric.ric_check_slots(s.slot_mapping, s.num_tokens_padded, num_slots, ws.data_ptr(), nbytes,
                                res.data_ptr(), dev_num_tokens=s.dev_scalars + 4, stream=self.stream)
        torch.cuda.synchronize()
        return tuple(int(x) for x in res.tolist())

    def debug_dump(self, s: ric.ric_step, limit: int = 32) -> None:
        """Print the small per-step arrays a developer checks first when a step
        goes wrong (request order, counts, boundaries, positions, slots,
        logits rows, discard), not the tables, and the device-side count of
        real tokens sharing a slot.  Synchronises: debugging only, enabled by
        RIC_DEBUG=1."""
        R, n = s.num_reqs, s.num_tokens_padded
        cols = ric.ric_get_columns(self.h)
        show = lambda a: " ".join(str(int(x)) for x in a[:limit]) + (" ..." if len(a) > limit else "")
        print(f"[ric] R={R} N={s.num_actual_tokens} N_pad={n} max_q={s.max_query_len} "
              f"max_seq={s.max_seq_len} sampled={s.num_sampled}")
        print(f"[ric] req_ids    {show(self.row_order())}")
        print(f"[ric] computed   {show(self.device_i32(cols.num_computed, R))}")
        print(f"[ric] scheduled  {show(self.device_i32(cols.num_scheduled, R))}")
        print(f"[ric] qsl        {show(self.device_i32(s.query_start_loc, R + 1))}")
        print(f"[ric] positions  {show(self.device_i32(s.positions, n))}")
        print(f"[ric] seq_lens   {show(self.device_i32(s.seq_lens, R))}")
        print(f"[ric] slots      {show(self.device_i32(s.slot_mapping, n))}")
        print(f"[ric] logits     {show(self.device_i32(s.logits_indices, R))}")
        print(f"[ric] discard    {show(self.device_u8(s.discard, R))}")
        dup, bad = self.slot_collisions(s)
        print(f"[ric] slot collisions {dup}, out-of-range slots {bad}", flush=True)

    def block_table(self, group: int = 0) -> torch.Tensor:
        """The handle's own block table of a KV-cache group, [max_num_reqs, stride]
        int32 (entries past a row's count are stale): what an attention call reads."""
        cols = ric.ric_get_columns(self.h)
        stride = cols.group_block_stride[group]
        n = self.cfg.max_num_reqs * stride
        return _view_u8(self.workspace, cols.group_blocks[group], 4 * n).view(torch.int32).view(-1, stride)

    # inspection (tests) ------------------------------------------------------
    def device_i32(self, ptr: int, n: int) -> np.ndarray:
        """Copy n int32 values from a device address to the host (test use)."""
        if n == 0:
            return np.zeros(0, np.int32)
        t = torch.empty(n, dtype=torch.int32, device=self.workspace.device)
        nbytes = 4 * n
        src = _view_u8(self.workspace, ptr, nbytes)
        t.view(torch.uint8).copy_(src)
        return t.cpu().numpy()

    def device_u8(self, ptr: int, n: int) -> np.ndarray:
        if n == 0:
            return np.zeros(0, np.uint8)
        return _view_u8(self.workspace, ptr, n).cpu().numpy()

    def step_outputs(self, s: ric.ric_step) -> dict:
        MR = self.cfg.max_num_reqs
        n = s.num_tokens_padded
        out = {
            "input_ids": self.device_i32(s.input_ids, n),
            "positions": self.device_i32(s.positions, n),
            "req_indices": self.device_i32(s.req_indices, n),
            "slot_mapping": self.device_i32(s.slot_mapping, n),
            "query_start_loc": self.device_i32(s.query_start_loc, MR + 1),
            "cu_seqlens_k": self.device_i32(s.cu_seqlens_k, MR + 1),
            "seq_lens": self.device_i32(s.seq_lens, MR),
            "logits_indices": self.device_i32(s.logits_indices, MR),
            "discard": self.device_u8(s.discard, MR),
            "sample_indices": self.device_i32(s.sample_indices, MR),
            "dev_scalars": self.device_i32(s.dev_scalars, 8),
        }
        out["num_sampled"] = int(out["dev_scalars"][5])
        return out


def _view_u8(anchor: torch.Tensor, ptr: int, nbytes: int) -> torch.Tensor:
    """A uint8 view of [ptr, ptr+nbytes) inside the anchor tensor's storage."""
    base = anchor.data_ptr()
    off = ptr - base
    if off < 0 or off + nbytes > anchor.numel():
        raise ValueError("address outside the workspace")
    return anchor.view(torch.uint8)[off:off + nbytes]


@dataclass
class KVSet:
    """Per-layer K/V sources [n_pad, H, D] and paged caches [num_blocks, B, H, D]."""
    k: List[torch.Tensor]
    v: List[torch.Tensor]
    kc: List[torch.Tensor]
    vc: List[torch.Tensor]
    row_bytes: int
    num_slots: int


def alloc_caches(w, num_layers: Optional[int] = None, device="cuda", fill: Optional[int] = None):
    L = w.num_layers if num_layers is None else num_layers
    dt = _TORCH_DT[w.kv_dtype]
    shape = (w.num_kv_blocks, w.block_size, w.kv_heads, w.head_dim)
    kc, vc = [], []
    for _ in range(L):
        for lst in (kc, vc):
            t = torch.empty(shape, dtype=dt, device=device)
            if fill is not None:
                t.view(torch.int16).fill_(fill)
            lst.append(t)
    return kc, vc


def alloc_sources(w, n_tokens: int, seed: int, num_layers: Optional[int] = None, device="cuda",
                  host: bool = False):
    """Seeded N(0,1) K/V sources per layer; ``host`` draws them with numpy
    (bit-reproducible on the CPU) and uploads them."""
    from workloads import payload_numpy, payload_torch  # seeded generators only
    L = w.num_layers if num_layers is None else num_layers
    shape = (n_tokens, w.kv_heads, w.head_dim)
    k, v = [], []
    for l in range(L):
        for j, lst in enumerate((k, v)):
            s = seed + 2 * l + j
            if host:
                bits = payload_numpy(np.random.default_rng(s), shape, w.kv_dtype)
                t = torch.from_numpy(bits.view(np.int16)).to(device).view(_TORCH_DT[w.kv_dtype])
            else:
                t = payload_torch(shape, w.kv_dtype, s, device)
            lst.append(t)
    return k, v


def reshape_and_cache(kv: KVSet, slot_mapping: int, num_tokens: int, dev_status: int = 0,
                      stream: Optional[int] = None, flags: int = 0) -> None:
    ric.ric_reshape_and_cache([t.data_ptr() for t in kv.k], [t.data_ptr() for t in kv.v],
                              [t.data_ptr() for t in kv.kc], [t.data_ptr() for t in kv.vc],
                              slot_mapping, num_tokens, kv.row_bytes, kv.num_slots,
                              src_row_stride=kv.k[0].stride(0) * kv.k[0].element_size(),
                              dev_status=dev_status, flags=flags,
                              stream=current_stream() if stream is None else stream)


def compile_and_cache(batch: "Batch", n_pad: int, kv: KVSet, dev_status: int = 0, flags: int = 0) -> ric.ric_step:
    """Compile plus the K/V write of every layer in one library call (one
    kernel for rows of 128 B to 8 KiB, unless the rows are 1 KiB or more and
    the step is mostly long chunks; flags RIC_FUSE_ALWAYS / RIC_FUSE_NEVER
    force the path)."""
    return ric.ric_compile_and_cache(batch.h, n_pad, [t.data_ptr() for t in kv.k], [t.data_ptr() for t in kv.v],
                                     [t.data_ptr() for t in kv.kc], [t.data_ptr() for t in kv.vc], kv.row_bytes,
                                     kv.num_slots, src_row_stride=kv.k[0].stride(0) * kv.k[0].element_size(),
                                     dev_status=dev_status, flags=flags)


def gather(hidden: torch.Tensor, idx_ptr: int, dev_count_ptr: int, max_rows: int, out: torch.Tensor,
           dev_status: int = 0, stream: Optional[int] = None) -> None:
    row_bytes = hidden.shape[1] * hidden.element_size()
    ric.ric_gather_rows(hidden.data_ptr(), hidden.stride(0) * hidden.element_size(), hidden.shape[0],
                        idx_ptr, dev_count_ptr, max_rows, row_bytes, out.data_ptr(),
                        out.stride(0) * out.element_size(), dev_status,
                        current_stream() if stream is None else stream)


# ---- operators around the step ------------------------------------------------------

_DTYPE = {torch.float16: ric.RIC_F16, torch.bfloat16: ric.RIC_BF16, torch.float32: ric.RIC_F32}


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _allocating_on(stream: int):
    """Context in which torch allocates for work on ``stream``."""
    return contextlib.nullcontext() if stream == current_stream() else torch.cuda.stream(torch.cuda.ExternalStream(stream))


def _attention(q, k_cache, scale=None, softcap=0.0, window=0, alibi_slopes=None, prefix_lens=None) -> ric.ric_attention:
    dtype = _DTYPE.get(q.dtype, ric.RIC_F32)
    if dtype == ric.RIC_F32 or k_cache.dtype is not q.dtype:
        raise ValueError("q and the caches must be float16 or bfloat16, and alike")
    _, heads, dim = q.shape
    _, block, kv_heads, _ = k_cache.shape
    return ric.ric_attention(dtype, heads, kv_heads, dim, block, dim ** -0.5 if scale is None else scale, softcap, window,
                             alibi_slopes.data_ptr() if alibi_slopes is not None else None,
                             prefix_lens.data_ptr() if prefix_lens is not None else None)


def _on_current_device(*tensors: Optional[torch.Tensor]) -> None:
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must lie on the current device (cuda:{dev})")


def _counts_ok(t: torch.Tensor, n: int) -> bool:
    return t.dtype is torch.int32 and t.shape == (n,) and t.is_contiguous()


def attention_workspace(q: torch.Tensor, k_cache: torch.Tensor, num_reqs: int, max_query_len: int,
                        max_seq_len: int) -> Optional[torch.Tensor]:
    """A workspace for paged_attention calls with these counts and bounds (None:
    none needed).  Fewer requests may be cut further and need more.  Calls that
    may run at the same time need one each."""
    n = ric.ric_paged_attention_workspace_bytes(_attention(q, k_cache), num_reqs, q.shape[0], max_query_len, max_seq_len)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    query_start_loc: torch.Tensor, seq_lens: torch.Tensor, max_query_len: int, max_seq_len: int,
                    out: torch.Tensor, scale: Optional[float] = None, softcap: float = 0.0, window: int = 0,
                    alibi_slopes: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, dev_status: int = 0) -> torch.Tensor:
    """Attention of q [num_tokens, heads, head_dim] over the pages of each
    request (ric_paged_attention), on the current stream.  k_cache, v_cache
    [num_blocks, block_size, kv_heads, head_dim]; block_table [num_reqs, width]
    int32; query_start_loc [num_reqs + 1], seq_lens [num_reqs] int32.  Without a
    workspace one is allocated where the call needs it."""
    a = _attention(q, k_cache, scale, softcap, window, alibi_slopes, prefix_lens)
    tokens, heads, dim = shape = q.shape
    n = seq_lens.shape[0]
    if k_cache.shape != v_cache.shape or v_cache.dtype is not q.dtype or k_cache.shape[3] != dim:
        raise ValueError("k_cache and v_cache must be [num_blocks, block_size, kv_heads, head_dim] of q's type")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous")
    if out.shape != shape or out.dtype is not q.dtype:
        raise ValueError("out must be like q")
    sq, so = q.stride(), out.stride()
    if tokens and ((dim > 1 and (sq[2] != 1 or so[2] != 1)) or (heads > 1 and (sq[1] != dim or so[1] != dim))):
        raise ValueError("the heads of a token must be contiguous")
    if tokens > 1 and (sq[0] < heads * dim or so[0] < heads * dim):
        raise ValueError("the tokens of q and out must not overlap")
    if not (_counts_ok(query_start_loc, n + 1) and _counts_ok(seq_lens, n) and
            (prefix_lens is None or _counts_ok(prefix_lens, n))):
        raise ValueError(f"query_start_loc [{n + 1}], seq_lens and prefix_lens [{n}] must be contiguous int32")
    rows, width = block_table.shape
    st = block_table.stride()
    if block_table.dtype is not torch.int32 or rows < n or (width > 1 and st[1] != 1) or (rows > 1 and st[0] < width):
        raise ValueError("block_table must be int32 [num_reqs, width] with contiguous rows of their own")
    if alibi_slopes is not None and (alibi_slopes.dtype is not torch.float32 or alibi_slopes.shape != (heads,) or
                                     not alibi_slopes.is_contiguous()):
        raise ValueError("alibi_slopes must be contiguous float32 [heads]")
    _on_current_device(q, k_cache, v_cache, block_table, query_start_loc, seq_lens, out, alibi_slopes, prefix_lens, workspace)
    if workspace is None:
        workspace = attention_workspace(q, k_cache, n, max_query_len, max_seq_len)
    ws, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    many = tokens > 1
    ric.ric_paged_attention(a, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_cache.shape[0],
                            block_table.data_ptr(), max(st[0], width), width, query_start_loc.data_ptr(),
                            seq_lens.data_ptr(), n, tokens, max_query_len, max_seq_len, out.data_ptr(),
                            sq[0] * 2 if many else 0, so[0] * 2 if many else 0, ws, ws_bytes, dev_status,
                            current_stream())
    return out


def step_attention(batch: "Batch", step: ric.ric_step, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   out: torch.Tensor, group: int = 0, workspace: Optional[torch.Tensor] = None, dev_status: int = 0,
                   **kw) -> torch.Tensor:
    """One layer's attention of a compiled step: q [num_tokens_padded, heads,
    head_dim] over the caches its K/V rows were written to, through the handle's
    own query_start_loc, seq_lens and block table.  Enqueued on the handle's
    stream; ``kw``: scale, softcap, window, alibi_slopes, prefix_lens."""
    a = _attention(q, k_cache, **kw)
    _pool(batch, group)                             # a group the handle may have
    cols = ric.ric_get_columns(batch.h)
    if q.shape[0] != step.num_tokens_padded or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q and out must hold the step's padded tokens")
    if k_cache.shape != v_cache.shape or v_cache.dtype != q.dtype or k_cache.shape[3] != q.shape[2] or \
            not (k_cache.is_contiguous() and v_cache.is_contiguous() and q.is_contiguous() and out.is_contiguous()):
        raise ValueError("contiguous q, out and caches of one type are needed")
    cfg = batch.cfg
    if k_cache.shape[1] != (cfg.block_size if group == 0 else cfg.group_block_size[group]):
        raise ValueError("the caches' block size is not the group's")
    prefix, slopes = kw.get("prefix_lens"), kw.get("alibi_slopes")
    if (prefix is not None and not _counts_ok(prefix, step.num_reqs)) or \
            (slopes is not None and (slopes.dtype is not torch.float32 or slopes.shape != (q.shape[1],) or
                                     not slopes.is_contiguous())):
        raise ValueError("prefix_lens must be contiguous int32 [num_reqs], alibi_slopes contiguous float32 [heads]")
    dev = batch.workspace.get_device()
    if any(t is not None and t.get_device() != dev for t in (q, out, k_cache, v_cache, workspace, prefix, slopes)):
        raise ValueError("every tensor must lie on the batch's device")
    with torch.cuda.device(dev):
        if workspace is None:
            with _allocating_on(batch.stream):
                workspace = attention_workspace(q, k_cache, step.num_reqs, step.max_query_len, step.max_seq_len)
        ric.ric_paged_attention(a, _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], cols.group_blocks[group] or 0,
                                cols.group_block_stride[group], cols.group_block_stride[group], step.query_start_loc,
                                step.seq_lens, step.num_reqs, q.shape[0], step.max_query_len, step.max_seq_len,
                                _ptr(out), workspace=_ptr(workspace),
                                workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size(),
                                dev_status=dev_status, stream=batch.stream)
    return out


@dataclass
class Logprobs:
    """Outputs of token_logprobs: [rows] float32, int32, float32; [rows, top_k]."""
    logprob: torch.Tensor
    rank: torch.Tensor
    entropy: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor
    workspace: Optional[torch.Tensor]


def alloc_logprobs(rows: int, vocab: int, top_k: int, device="cuda") -> Logprobs:
    """Output and workspace tensors for token_logprobs calls of up to ``rows`` rows
    of up to ``vocab`` logits."""
    f = lambda *s: torch.empty(s, dtype=torch.float32, device=device)
    i = lambda *s: torch.empty(s, dtype=torch.int32, device=device)
    n = ric.ric_token_logprobs_workspace_bytes(rows, vocab, top_k)
    return Logprobs(f(rows), i(rows), f(rows), i(rows, top_k), f(rows, top_k),
                    torch.empty(n, dtype=torch.uint8, device=device) if n else None)


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor], top_k: int = 0,
                   out: Optional[Logprobs] = None, dev_count: int = 0, dev_status: int = 0) -> Logprobs:
    """Log probability, rank, entropy and top_k alternatives of each row of
    logits [rows, vocab] (ric_token_logprobs), on the current stream.  With
    ``out`` the first ``rows`` rows of its tensors are written."""
    if logits.dim() != 2 or logits.dtype not in _DTYPE or (logits.numel() and logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [rows, vocab] of float16, bfloat16 or float32 with contiguous rows")
    rows, vocab = logits.shape
    if rows > 1 and logits.stride(0) < vocab:
        raise ValueError("the rows of logits must not overlap")
    if targets is not None and (targets.dtype != torch.int32 or targets.shape != (rows,) or not targets.is_contiguous()):
        raise ValueError("targets must be contiguous int32 [rows]")
    if out is None:
        out = alloc_logprobs(rows, vocab, top_k, logits.device)
    elif out.logprob.shape[0] < rows or out.top_ids.shape[1] != top_k:
        raise ValueError("out is too small, or of another top_k")
    has = targets is not None
    _on_current_device(logits, targets, out.logprob, out.rank, out.entropy, out.top_ids, out.top_logprobs, out.workspace)
    ric.ric_token_logprobs(_ptr(logits), _DTYPE[logits.dtype], _ptr(targets), rows, vocab, top_k,
                           _ptr(out.logprob) if has else 0, _ptr(out.rank) if has else 0, _ptr(out.entropy),
                           _ptr(out.top_ids) if top_k else 0, _ptr(out.top_logprobs) if top_k else 0,
                           row_stride=logits.stride(0) * logits.element_size() if rows > 1 else 0, dev_count=dev_count,
                           workspace=_ptr(out.workspace),
                           workspace_bytes=0 if out.workspace is None else out.workspace.numel(),
                           dev_status=dev_status, stream=current_stream())
    return out


def _pool(batch: "Batch", group: int) -> int:
    """Pages of the group's pool."""
    c = batch.cfg
    if not 0 <= group < max(1, c.num_kv_groups):
        raise ValueError(f"group {group} outside [0, {max(1, c.num_kv_groups)})")
    return c.num_kv_blocks if group == 0 or c.group_num_kv_blocks[group] <= 0 else c.group_num_kv_blocks[group]


def _pages(batch: "Batch", kc: List[torch.Tensor], vc: List[torch.Tensor], group: int, *named):
    """Addresses of the layers' caches and the bytes of a page; ``named``: lists of
    the pages that the call is given."""
    if len(kc) != len(vc):
        raise ValueError("kc and vc must hold one cache per layer each")
    if not kc:
        return [], [], 0
    device = batch.workspace.get_device()
    both = [*kc, *vc]
    pages = kc[0].shape[0]                          # ids are checked against the group's pool by the call
    if pages < _pool(batch, group) and any(len(ids) and np.max(ids) >= pages for ids in named):
        raise ValueError("a page lies past the caches' end")
    if len({t.numel() for t in both}) != 1 or len({t.dtype for t in both}) != 1 or \
            {t.get_device() for t in both} != {device} or \
            not all([t.is_contiguous() for t in both]):
        raise ValueError("the layers' caches must be contiguous, alike and on the batch's device")
    return [t.data_ptr() for t in kc], [t.data_ptr() for t in vc], kc[0][0].numel() * kc[0].element_size()


def copy_blocks(batch: "Batch", src, dst, kc: List[torch.Tensor], vc: List[torch.Tensor], group: int = 0) -> None:
    """Page src[k] -> page dst[k] in every layer's caches [num_blocks, ...] (ric_copy_blocks)."""
    k, v, n = _pages(batch, kc, vc, group, src, dst)
    ric.ric_copy_blocks(batch.h, src, dst, k, v, n, group)


def move_blocks(batch: "Batch", src, dst, kc: List[torch.Tensor], vc: List[torch.Tensor], group: int = 0) -> None:
    """copy_blocks, and the live requests' block tables follow (ric_move_blocks)."""
    k, v, n = _pages(batch, kc, vc, group, src, dst)
    ric.ric_move_blocks(batch.h, src, dst, k, v, n, group)


def block_refs(batch: "Batch", group: int = 0) -> torch.Tensor:
    """Table entries that name each page of the group's pool, int32 (ric_block_refs),
    written on the handle's stream."""
    pool = _pool(batch, group)
    with _allocating_on(batch.stream):
        refs = torch.empty(pool, dtype=torch.int32, device=batch.workspace.device)
    ric.ric_block_refs(batch.h, refs.data_ptr(), group)
    return refs


def fork_request(batch: "Batch", parent_id: int, child_id: int, num_tokens: int, num_computed: int, new_blocks,
                 kc: List[torch.Tensor], vc: List[torch.Tensor], sampling=None) -> int:
    """A new request over the parent's history, sharing its full pages (ric_fork_request)."""
    k, v, n = _pages(batch, kc, vc, 0, new_blocks[:1])
    return ric.ric_fork_request(batch.h, parent_id, child_id, num_tokens, num_computed, new_blocks, k, v,
                                n // batch.cfg.block_size, sampling)
