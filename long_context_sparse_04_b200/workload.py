"""Device-side plumbing: put a workload's tensors in HBM and call the C ABI.

PyTorch provides device memory and streams only; every stage runs in
libdsa.so through the binding in ``_native``.
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _native as N


def _vp(x):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def to_device(a: np.ndarray | None, device):
    import torch
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:                       # bf16 bit patterns
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(a).to(device)


def q_group_for(cfg) -> int:
    if cfg.prefill:
        return 4
    return cfg.rows_per_seq if cfg.rows_per_seq in (1, 2, 4) else 1


def pack_latents(dims, latent):
    """Packed 4-bit rows (uint8 [n, row bytes]) of bf16 latent rows on a device."""
    import torch
    n = latent.shape[0]
    if not latent.is_cuda:
        raise ValueError("latent: a tensor on a CUDA device expected")
    new = _tensor(latent, "latent", (n, dims.d_c + dims.d_r), (torch.bfloat16,), latent.device)
    packed = torch.empty((n, N.dsa_latent_row_bytes(dims)), dtype=torch.uint8, device=latent.device)
    if n == 0:
        return packed
    slot = torch.arange(n, dtype=torch.int64, device=latent.device)
    ws = torch.zeros(N.dsa_workspace_size(dims, None, N.DSA_OP_CACHE_APPEND), dtype=torch.uint8, device=latent.device)
    cache = N.dsa_cache(latent=_vp(packed), num_seqs=1, num_tokens=n)
    stream = ctypes.c_void_p(torch.cuda.current_stream(latent.device).cuda_stream)
    with torch.cuda.device(latent.device):
        N.dsa_cache_append_slots(dims, cache, n, _vp(slot), None, new, _vp(ws), ws.numel(), stream)
        st = N.dsa_read_device_status(_vp(ws), stream)
    if st != (0, -1):
        raise ValueError(f"latent row {st[1]} has an infinity or NaN")
    return packed


class DeviceWorkload:
    """One workload resident on a CUDA device, with the C-ABI descriptors."""

    def __init__(self, inp: dict, device="cuda", algo: int = N.DSA_ALGO_AUTO,
                 q_group: int | None = None, int4: bool = False):
        """int4: keep the latent cache in packed 4-bit rows (bf16 workloads)."""
        import torch
        self.torch = torch
        self.inp = inp
        self.device = torch.device(device)
        cfg = inp["cfg"]
        self.cfg = cfg
        dev = self.device
        self.row_seq = to_device(inp["row_seq"].astype(np.int32), dev)
        self.row_klen = to_device(inp["row_klen"].astype(np.int32), dev)
        self.q_idx = to_device(inp["q_idx"], dev)
        self.q_scale = to_device(inp["q_scale"], dev)
        self.w = to_device(inp["w"].astype(np.float32), dev)
        self.k_idx = to_device(inp["k_idx"], dev)
        self.k_scale = to_device(inp["k_scale"], dev)
        self.latent = to_device(inp["latent"], dev)
        self.q = to_device(inp["q"], dev) if inp.get("q") is not None else None
        c = inp["cache"]
        self.seq_start = to_device(c["seq_start"], dev) if c.get("seq_start") is not None else None
        self.block_table = to_device(c["block_table"], dev) if c.get("block_table") is not None else None
        T = int(inp["row_seq"].shape[0])
        self.T = T
        self.max_klen = int(inp["row_klen"].max()) if T else 0
        self.ld = ((self.max_klen + 127) // 128) * 128
        self.topk = int(inp["topk"])
        self.H = int(inp["n_heads"])
        self.d_c = int(inp["d_c"])
        self.mla_bf16 = inp["mla_dtype"] == "bf16"
        self.dims = N.dsa_dims(
            n_idx_heads=int(inp["h_idx"]), d_idx=int(inp["d_idx"]), n_heads=self.H,
            d_c=self.d_c, d_r=int(inp["d_r"]), topk=self.topk,
            idx_dtype=N.DSA_FP8_E4M3 if inp["idx_dtype"] == "e4m3" else N.DSA_F32,
            mla_dtype=N.DSA_INT4 if int4 else N.DSA_BF16 if self.mla_bf16 else N.DSA_F32,
            sm_scale=float(inp["sm_scale"]), algo=algo)
        if int4:
            assert self.mla_bf16, "packed latent rows are made of bf16 rows"
            self.latent = pack_latents(self.dims, self.latent)
        self.rows = N.dsa_rows(num_rows=T, row_seq=_vp(self.row_seq), row_klen=_vp(self.row_klen),
                               max_klen=self.max_klen,
                               q_group=q_group if q_group is not None else q_group_for(cfg))
        n_tok = int(inp["k_idx"].shape[0])
        bt = c.get("block_table")
        self.cache = N.dsa_cache(
            latent=_vp(self.latent), idx_k=_vp(self.k_idx), idx_k_scale=_vp(self.k_scale),
            seq_start=_vp(self.seq_start), block_table=_vp(self.block_table),
            page_size=int(c["page_size"]) if bt is not None else 0,
            max_pages_per_seq=int(bt.shape[1]) if bt is not None else 0,
            num_seqs=int(len(c["seq_start"]) if bt is None else bt.shape[0]), num_tokens=n_tok)
        self._ws = {}

    # ------------------------------------------------------------------ helpers
    @property
    def stream(self):
        return ctypes.c_void_p(self.torch.cuda.current_stream(self.device).cuda_stream)

    def workspace(self, op: int):
        if op not in self._ws:
            n = N.dsa_workspace_size(self.dims, self.rows, op)
            assert n > 0, "dsa_workspace_size returned 0"
            ws = self.torch.empty(n, dtype=self.torch.uint8, device=self.device)
            N.dsa_workspace_init(_vp(ws), n, self.stream)
            self._ws[op] = (ws, n)
        return self._ws[op]

    def status(self, op: int):
        ws, _ = self.workspace(op)
        return N.dsa_read_device_status(_vp(ws), self.stream)

    def kernels_ran(self, op: int) -> int:
        ws, _ = self.workspace(op)
        return N.dsa_read_kernel_trace(_vp(ws), self.stream)

    def out_dtype(self):
        return self.torch.bfloat16 if self.mla_bf16 else self.torch.float32

    # ------------------------------------------------------------------ stages
    def indexer(self, scores=None):
        torch = self.torch
        if scores is None:
            scores = torch.full((self.T, self.ld), float("nan"), dtype=torch.float32, device=self.device)
        ws, n = self.workspace(N.DSA_OP_INDEXER)
        N.dsa_indexer_scores(self.dims, self.rows, self.cache, _vp(self.q_idx), _vp(self.q_scale),
                             _vp(self.w), _vp(scores), self.ld, _vp(ws), n, self.stream)
        return scores

    def topk_(self, scores, idx=None):
        torch = self.torch
        if idx is None:
            idx = torch.empty((self.T, self.topk), dtype=torch.int32, device=self.device)
        ws, n = self.workspace(N.DSA_OP_TOPK)
        N.dsa_topk(self.dims, self.rows, _vp(scores), scores.shape[1], _vp(idx), _vp(ws), n,
                   self.stream)
        return idx

    def mla(self, idx, out=None, lse=None):
        torch = self.torch
        if out is None:
            out = torch.empty((self.T, self.H, self.d_c), dtype=self.out_dtype(), device=self.device)
        if lse is None:
            lse = torch.empty((self.T, self.H), dtype=torch.float32, device=self.device)
        ws, n = self.workspace(N.DSA_OP_SPARSE_MLA)
        N.dsa_sparse_mla_fwd(self.dims, self.rows, self.cache, _vp(self.q), _vp(idx), _vp(out),
                             _vp(lse), _vp(ws), n, self.stream)
        return out, lse

    def decode_step(self, out=None, lse=None, debug=False):
        torch = self.torch
        if out is None:
            out = torch.empty((self.T, self.H, self.d_c), dtype=self.out_dtype(), device=self.device)
        if lse is None:
            lse = torch.empty((self.T, self.H), dtype=torch.float32, device=self.device)
        dbg_s = dbg_i = None
        if debug:
            dbg_s = torch.full((self.T, self.ld), float("nan"), dtype=torch.float32, device=self.device)
            dbg_i = torch.empty((self.T, self.topk), dtype=torch.int32, device=self.device)
        ws, n = self.workspace(N.DSA_OP_DECODE_STEP)
        N.dsa_decode_step(self.dims, self.rows, self.cache, _vp(self.q_idx), _vp(self.q_scale),
                          _vp(self.w), _vp(self.q), _vp(out), _vp(lse), _vp(dbg_s), _vp(dbg_i),
                          _vp(ws), n, self.stream)
        return out, lse, dbg_s, dbg_i

    def forward(self, out=None, lse=None, idx=None):
        torch = self.torch
        if out is None:
            out = torch.empty((self.T, self.H, self.d_c), dtype=self.out_dtype(), device=self.device)
        if lse is None:
            lse = torch.empty((self.T, self.H), dtype=torch.float32, device=self.device)
        if idx is None:
            idx = torch.empty((self.T, self.topk), dtype=torch.int32, device=self.device)
        ws, n = self.workspace(N.DSA_OP_FORWARD)
        N.dsa_forward(self.dims, self.rows, self.cache, _vp(self.q_idx), _vp(self.q_scale),
                      _vp(self.w), _vp(self.q), _vp(out), _vp(lse), _vp(idx), _vp(ws), n,
                      self.stream)
        return out, lse, idx

    def append(self, tok_seq, tok_pos, k_new, latent_new, check=True):
        """dsa_cache_append of new tokens (device tensors: int32 [n], int32 [n],
        fp32 [n, d_I], latent rows [n, d_c+d_r]) into this workload's caches."""
        ws, n = self.workspace(N.DSA_OP_CACHE_APPEND)
        return N.dsa_cache_append(self.dims, self.cache, int(tok_seq.shape[0]), _vp(tok_seq),
                                  _vp(tok_pos), _vp(k_new), _vp(latent_new), _vp(ws), n,
                                  self.stream, check=check)

    def caches_to_host(self):
        """(k_idx, k_scale, latent) in their storage formats (bf16 as uint16 bits)."""
        torch = self.torch
        lat = self.latent
        lat = lat.view(torch.int16).cpu().numpy().view(np.uint16) if lat.dtype == torch.bfloat16 \
            else lat.cpu().numpy()
        ks = None if self.k_scale is None else self.k_scale.cpu().numpy()
        return self.k_idx.cpu().numpy(), ks, lat


def _tensor(x, name: str, shape, dtypes, device):
    """Device pointer of an argument that a kernel will take at its word."""
    if tuple(x.shape) != tuple(shape) or x.dtype not in dtypes or x.device != device or not x.is_contiguous():
        want = " or ".join(str(d) for d in dtypes)
        raise ValueError(f"{name}: contiguous {want} of shape {tuple(shape)} on {device} expected, got {x.dtype} of shape "
                         f"{tuple(x.shape)} on {x.device}{'' if x.is_contiguous() else ', not contiguous'}")
    return _vp(x)


class DevicePlanner:
    """The paging state of a batch of request slots, planned on the GPU: lengths,
    block table and free list live in device memory and each plan() (one
    dsa_batch_plan, in place) advances them by ``n_new`` and ``release``."""

    def __init__(self, num_seqs: int, page_size: int, num_pages: int, max_pages_per_seq: int, max_tokens: int,
                 device="cuda"):
        import torch
        self.torch = torch
        dev = self.device = torch.device(device)
        self.num_seqs, self.max_tokens, self.max_len = num_seqs, max_tokens, max_pages_per_seq * page_size
        zeros = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device=dev)  # noqa: E731
        self.seq_len, self.n_new, self.release = zeros(num_seqs), zeros(num_seqs), zeros(num_seqs)
        self.block_table = torch.full((num_seqs, max_pages_per_seq), -1, dtype=torch.int32, device=dev)
        self.free_pages = torch.arange(num_pages, dtype=torch.int32, device=dev)
        self.free_count = torch.full((1,), num_pages, dtype=torch.int32, device=dev)
        self.tok_start, self.totals = zeros(num_seqs + 1), zeros(4)
        self.row_seq, self.row_klen, self.tok_pos = zeros(max_tokens), zeros(max_tokens), zeros(max_tokens)
        self.slot = zeros(max_tokens, dtype=torch.int64)
        self.cache = N.dsa_cache(block_table=_vp(self.block_table), page_size=page_size,
                                 max_pages_per_seq=max_pages_per_seq, num_seqs=num_seqs,
                                 num_tokens=num_pages * page_size)
        self._plan = N.dsa_plan(
            seq_len=_vp(self.seq_len), n_new=_vp(self.n_new), release=_vp(self.release),
            seq_len_out=_vp(self.seq_len), free_count=_vp(self.free_count), free_count_out=_vp(self.free_count),
            free_pages=_vp(self.free_pages), free_capacity=num_pages, max_tokens=max_tokens,
            tok_start=_vp(self.tok_start), row_seq=_vp(self.row_seq), row_klen=_vp(self.row_klen),
            tok_pos=_vp(self.tok_pos), slot=_vp(self.slot), totals=_vp(self.totals))
        self._ws = zeros(N.dsa_workspace_size(None, None, N.DSA_OP_BATCH_PLAN), dtype=torch.uint8)

    @property
    def stream(self):
        return ctypes.c_void_p(self.torch.cuda.current_stream(self.device).cuda_stream)

    def on_device(self):
        """The library launches on the current device: this makes it the planner's."""
        return self.torch.cuda.device(self.device)

    def plan(self):
        with self.on_device():
            N.dsa_batch_plan(self.cache, self._plan, _vp(self._ws), self._ws.numel(), self.stream)

    def status(self):
        with self.on_device():
            return N.dsa_read_device_status(_vp(self._ws), self.stream)

    def rows(self, q_group: int = 1):
        """dsa_rows of the whole (padded) batch."""
        return N.dsa_rows(num_rows=self.max_tokens, row_seq=_vp(self.row_seq), row_klen=_vp(self.row_klen),
                          max_klen=self.max_len, q_group=q_group)


class PagedCache:
    """The caches of one layer behind a DevicePlanner: FP8 indexer keys, and the
    latents in bf16 or in packed 4-bit rows.

    workspace_of: the cache of another layer of the same planner and sizes, whose workspace
    (the scores of a step above all: rows x context x 4 bytes) this one then uses.  The
    layers' calls must run one after the other, and share one status word.
    q_group: as in dsa_rows; above 1 every request must get a multiple of it in each plan."""

    def __init__(self, planner: DevicePlanner, n_heads: int = 128, topk: int = 2048, int4: bool = True,
                 sm_scale: float | None = None, q_group: int = 1, workspace_of: "PagedCache | None" = None):
        torch = self.torch = planner.torch
        self.planner = planner
        d_c, d_r, d_idx = 512, 64, 128
        self.sm_scale = (d_c + d_r) ** -0.5 if sm_scale is None else sm_scale
        self.dims = N.dsa_dims(n_idx_heads=64, d_idx=d_idx, n_heads=n_heads, d_c=d_c, d_r=d_r, topk=topk,
                               idx_dtype=N.DSA_FP8_E4M3, mla_dtype=N.DSA_INT4 if int4 else N.DSA_BF16,
                               sm_scale=self.sm_scale, algo=N.DSA_ALGO_AUTO)
        p, dev = planner, planner.device
        n = int(p.cache.num_tokens)
        self.latent = torch.zeros((n, N.dsa_latent_row_bytes(self.dims)), dtype=torch.uint8, device=dev)
        self.idx_k = torch.zeros((n, d_idx), dtype=torch.uint8, device=dev)
        self.idx_k_scale = torch.ones(n, dtype=torch.float32, device=dev)
        self.cache = N.dsa_cache(latent=_vp(self.latent), idx_k=_vp(self.idx_k), idx_k_scale=_vp(self.idx_k_scale),
                                 block_table=p.cache.block_table, page_size=p.cache.page_size,
                                 max_pages_per_seq=p.cache.max_pages_per_seq, num_seqs=p.num_seqs, num_tokens=n)
        self.rows = p.rows(q_group)
        self.idx = torch.full((p.max_tokens, topk), -1, dtype=torch.int32, device=dev)
        with p.on_device():
            nb = N.dsa_workspace_size(self.dims, self.rows, N.DSA_OP_DECODE_STEP)
            if workspace_of is None:
                self._ws = torch.empty(nb, dtype=torch.uint8, device=dev)
                N.dsa_workspace_init(_vp(self._ws), nb, p.stream)
            elif workspace_of.planner is not planner:
                raise ValueError("workspace_of: a layer of another planner")
            elif bytes(workspace_of.dims) != bytes(self.dims) or workspace_of.rows.q_group != q_group:
                # (captured graphs count on what lies where: a step leaves its histograms zero)
                raise ValueError("workspace_of: a layer of other sizes")
            else:
                self._ws = workspace_of._ws

    def _args(self):
        return _vp(self._ws), self._ws.numel(), self.planner.stream

    def _arg(self, x, name, shape, *dtypes):
        return _tensor(x, name, shape, dtypes, self.planner.seq_len.device)

    def append(self, k_new, latent_new):
        """The planned step's tokens into the caches: max_tokens rows, in the plan's order,
        whatever lies behind the last."""
        torch, M, d = self.torch, self.planner.max_tokens, self.dims
        k = self._arg(k_new, "k_new", (M, d.d_idx), torch.float32)
        lat = self._arg(latent_new, "latent_new", (M, d.d_c + d.d_r), torch.bfloat16)
        with self.planner.on_device():
            N.dsa_cache_append_slots(d, self.cache, M, _vp(self.planner.slot), k, lat, *self._args())

    def read(self, slot, k_out=None, latent_out=None):
        """Cached tokens by physical row, as the values they stand for."""
        torch, n, d = self.torch, int(slot.shape[0]), self.dims
        at = self._arg(slot, "slot", (n,), torch.int64)
        k = None if k_out is None else self._arg(k_out, "k_out", (n, d.d_idx), torch.float32)
        lat = None if latent_out is None else self._arg(latent_out, "latent_out", (n, d.d_c + d.d_r), torch.bfloat16)
        with self.planner.on_device():
            N.dsa_cache_read(d, self.cache, n, at, k, lat, *self._args())

    def decode_step(self, q_idx, q_scale, w, q, out, lse=None):
        """The three stages over the planned rows (max_tokens rows in every tensor); rows
        behind the last give 0 and -inf."""
        torch, M, d = self.torch, self.planner.max_tokens, self.dims
        args = (self._arg(q_idx, "q_idx", (M, d.n_idx_heads, d.d_idx), torch.uint8, torch.float8_e4m3fn),
                self._arg(q_scale, "q_scale", (M, d.n_idx_heads), torch.float32),
                self._arg(w, "w", (M, d.n_idx_heads), torch.float32),
                self._arg(q, "q", (M, d.n_heads, d.d_c + d.d_r), torch.bfloat16),
                self._arg(out, "out", (M, d.n_heads, d.d_c), torch.bfloat16),
                None if lse is None else self._arg(lse, "lse", (M, d.n_heads), torch.float32))
        with self.planner.on_device():
            N.dsa_decode_step(d, self.rows, self.cache, *args, None, _vp(self.idx), *self._args())
        return out, lse

    def indices(self):
        """The last step's selection [max_tokens, topk]."""
        return self.idx

    def status(self):
        with self.planner.on_device():
            return N.dsa_read_device_status(*self._args()[::2])
