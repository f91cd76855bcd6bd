"""Device-side model: places a synthetic host model's tensors in HBM (torch
allocations) and drives the C ABI's decode step.  Marshalling only: every
step of the computation runs in libnt.so's kernels."""
from __future__ import annotations

import numpy as np
import torch

from . import nt

LAYER = ("wq", "wk", "wv", "wo", "wg", "wu", "wd")


def _h(a) -> torch.Tensor:
    """A host array as a tensor (read-only views, e.g. of a mapped file, are copied)."""
    return torch.from_numpy(a if a.flags.writeable else np.array(a))


def model_desc(spec, stream_slots: int = 0) -> nt.nt_model_desc:
    f = spec.fmt
    return nt.nt_model_desc(spec.n_layers, spec.d_model, spec.n_qh, spec.n_kvh, spec.head_dim, spec.ffn, spec.vocab,
                            spec.eps, spec.theta, spec.kv_cap, f["wq"], f["wk"], f["wv"], f["wo"], f["wg"], f["wu"],
                            f["wd"], f["embd"], f["out"], stream_slots)


def _row_bytes(spec, name):
    r, c = spec.tensor_shape(name)
    f = spec.fmt[name]
    return r, (c // nt.nt_block_elems(f)) * nt.nt_block_bytes(f)


class HostBlobs:
    """Page-locked host memory for the streamed layers of a model (layers
    n_resident..n_layers-1, each one blob in the library's blob layout) and,
    for streamed models, the embedding table.  ``view`` hands the generator
    numpy views to write the weights into, so they are never copied."""

    def __init__(self, spec, stream_slots: int = 0):
        self.spec = spec
        n_res = spec.n_layers if spec.n_resident < 0 else spec.n_resident
        self.layers = list(range(n_res, spec.n_layers))
        self.offsets, self.nbytes = nt.nt_layer_blob_layout(model_desc(spec, stream_slots))
        self.blob = {l: torch.empty(self.nbytes, dtype=torch.uint8, pin_memory=True) for l in self.layers}
        self.embd = None
        if self.layers:
            r, rb = _row_bytes(spec, "embd")
            self.embd = torch.empty((r, rb), dtype=torch.uint8, pin_memory=True)

    def view(self, layer: int, name: str):
        if layer < 0:
            return self.embd.numpy() if (name == "embd" and self.embd is not None) else None
        if layer not in self.blob:
            return None
        i = LAYER.index(name)
        r, rb = _row_bytes(self.spec, name)
        o = self.offsets[i]
        return self.blob[layer].numpy()[o:o + r * rb].reshape(r, rb)


_ROW_FMT = {torch.float32: nt.F32, torch.float16: nt.F16}


class KV8Cache:
    """One layer's 8-bit KV cache in HBM (torch allocations, or `buffers`: a dict
    of tensors k, v, kscale, vscale and, for block selection, kmin, kmax) and the
    calls on it.  fmt: nt.KV8_I8 or nt.KV8_E4M3.  Tensors must be contiguous
    where no stride is named.  pos_dev: an int64 tensor on the cache's device (or
    its address) that the call reads its position from."""

    def __init__(self, ctx: nt.Context, fmt: int, n_kvh: int, head_dim: int, kv_stride: int, device: str = "cuda",
                 bounds: bool = True, buffers: dict | None = None):
        self.ctx, self.n_kvh, self.head_dim, self.kv_stride = ctx, n_kvh, head_dim, kv_stride
        nb = (kv_stride + nt.KV8_BLOCK - 1) // nt.KV8_BLOCK
        shapes = {"k": ((n_kvh, kv_stride, head_dim), torch.uint8), "v": ((n_kvh, kv_stride, head_dim), torch.uint8),
                  "kscale": ((n_kvh, nb), torch.float32), "vscale": ((n_kvh, nb), torch.float32),
                  "kmin": ((n_kvh, nb, head_dim), torch.int8), "kmax": ((n_kvh, nb, head_dim), torch.int8)}
        if buffers is None:
            names = list(shapes) if bounds else list(shapes)[:4]
            buffers = {n: torch.zeros(shapes[n][0], dtype=shapes[n][1], device=device) for n in names}
        self.device, self.index = buffers["k"].device, buffers["k"].get_device()  # index -1: host memory
        for n, t in buffers.items():
            if (tuple(t.shape) != shapes[n][0] or t.dtype != shapes[n][1] or not t.is_contiguous()
                    or t.device != self.device):
                raise ValueError(f"{n}: need a contiguous {shapes[n][1]} tensor of shape {shapes[n][0]}, all on one device")
        if ctx is not None and self.index != ctx.device:
            raise ValueError("the cache must be on the context's device")
        self.buffers = buffers
        self.desc = nt.nt_kv8(fmt, n_kvh, head_dim, kv_stride,
                              *[nt._ptr(buffers.get(n)) for n in ("k", "v", "kscale", "vscale", "kmin", "kmax")])

    def _rows(self, k, v, tok, head):
        shape, stride, dtype = k.shape, k.stride(), k.dtype
        if (len(shape) != 3 or shape[head] != self.n_kvh or shape[2] != self.head_dim or stride[2] != 1
                or v.stride() != stride or v.shape != shape or v.dtype is not dtype
                or k.get_device() != self.index or v.get_device() != self.index):
            raise ValueError("k and v: rows of n_kvh heads of head_dim channels on the cache's device, alike in layout")
        fmt = _ROW_FMT.get(dtype)
        if fmt is None:
            raise ValueError("rows must be float32 or float16")
        return fmt, shape[tok], stride[tok], stride[head]

    def _pos(self, pos_dev):
        if (not isinstance(pos_dev, int) and (pos_dev.dtype is not torch.int64 or pos_dev.numel() < 1
                                              or pos_dev.get_device() != self.index)):
            raise ValueError("pos_dev: an int64 tensor on the cache's device, or a device address")

    def append(self, k, v, pos: int, pos_dev=None, stream=None):
        """Rows [n][n_kvh][head_dim] (fp32 or f16, any strides between rows and heads) to positions pos .."""
        fmt, n, ts, hs = self._rows(k, v, 0, 1)
        if pos_dev is not None:
            self._pos(pos_dev)
        nt.nt_kv8_append(self.ctx, self.desc, fmt, k, v, n, ts, hs, pos, pos_dev, stream)

    def append_from_heads(self, k, v, pos: int, pos_dev=None, stream=None):
        """Rows [n_kvh][n][head_dim], the layout of an F16 cache (a slice of its positions), to positions pos .."""
        fmt, n, ts, hs = self._rows(k, v, 1, 0)
        if pos_dev is not None:
            self._pos(pos_dev)
        nt.nt_kv8_append(self.ctx, self.desc, fmt, k, v, n, ts, hs, pos, pos_dev, stream)

    def read(self, pos0: int, k, v, stream=None):
        """Positions pos0 .. into k and v [n_kvh][n][head_dim] (fp32 or f16; rows of a head contiguous)."""
        fmt, n, ts, hs = self._rows(k, v, 1, 0)
        if n > 1 and ts != self.head_dim:
            raise ValueError("the rows of a head must be contiguous")
        nt.nt_kv8_read(self.ctx, self.desc, pos0, n, fmt, k, v, hs, stream)

    def _queries(self, q, out=None):
        shape = q.shape
        if (len(shape) != 3 or shape[2] != self.head_dim or q.dtype is not torch.float32 or not q.is_contiguous()
                or q.get_device() != self.index):
            raise ValueError("q: contiguous float32 [n_query][n_qh][head_dim] on the cache's device")
        if out is not None and (out.shape != shape or out.dtype is not torch.float32 or not out.is_contiguous()
                                or out.get_device() != self.index):
            raise ValueError("out: like q")
        return shape[0], shape[1]

    def attend(self, q, out, n_pos: int, pos_dev=None, stream=None):
        """Attention of q [n_query][n_qh][head_dim] into out; query i sees n_pos + i positions."""
        nq, n_qh = self._queries(q, out)
        if pos_dev is not None:
            self._pos(pos_dev)
        nt.nt_attn_kv8(self.ctx, q, self.desc, out, n_qh, n_pos, nq, pos_dev, stream)

    def _list(self, idx, nq):
        shape = idx.shape
        if (len(shape) != 3 or shape[0] != nq or shape[1] != self.n_kvh or idx.dtype is not torch.int32
                or not idx.is_contiguous() or idx.get_device() != self.index):
            raise ValueError("idx: contiguous int32 [n_query][n_kvh][n_sel] on the cache's device")
        return shape[2]

    def select(self, q, idx, n_pos: int, n_first: int = 0, n_last: int = 1, pos_dev=None, stream=None):
        """The blocks each query reads into idx [n_query][n_kvh][n_sel]."""
        nq, n_qh = self._queries(q)
        if pos_dev is not None:
            self._pos(pos_dev)
        nt.nt_kv8_select(self.ctx, q, self.desc, n_qh, n_pos, nq, self._list(idx, nq), n_first, n_last, idx, pos_dev,
                         stream)

    def attend_blocks(self, q, out, n_pos: int, idx, pos_dev=None, stream=None):
        """Attention over the listed blocks only."""
        nq, n_qh = self._queries(q, out)
        if pos_dev is not None:
            self._pos(pos_dev)
        nt.nt_attn_kv8_blocks(self.ctx, q, self.desc, out, n_qh, n_pos, nq, idx, self._list(idx, nq), pos_dev, stream)


class DeviceModel:
    """spec: shapes/formats; hm: host arrays (layers list of dicts, embd, out,
    out_norm, kcache/vcache float16 [L, kvh, cap, hd]).  With ``blobs`` the
    layers it holds are streamed from its page-locked host memory and the
    embedding table is read from host memory; their host arrays in ``hm``
    must be the blobs' views (make_host_model(..., out_view=blobs.view))."""

    def __init__(self, ctx: nt.Context, spec, hm, device: str = "cuda", blobs: HostBlobs | None = None,
                 stream_slots: int = 0):
        self.ctx, self.spec, self.blobs = ctx, spec, blobs
        self.n_slots = (stream_slots or 2) if (blobs is not None and blobs.layers) else 0
        dev = torch.device(device)
        self.layers = []
        for i, L in enumerate(hm.layers):
            if blobs is not None and i in blobs.blob:
                d = {n: _h(L[n]).to(dev) for n in ("attn_norm", "ffn_norm")}
                d["host_blob"] = blobs.blob[i]
            else:
                d = {n: _h(L[n]).to(dev) for n in LAYER + ("attn_norm", "ffn_norm")}
            d["kcache"] = torch.from_numpy(np.ascontiguousarray(hm.kcache[i])).to(dev)
            d["vcache"] = torch.from_numpy(np.ascontiguousarray(hm.vcache[i])).to(dev)
            self.layers.append(d)
        if blobs is not None and blobs.embd is not None:
            self.embd = blobs.embd
        else:
            self.embd = _h(hm.embd).to(dev)
        self.out = _h(hm.out).to(dev)
        self.out_norm = _h(hm.out_norm).to(dev)
        self.logits = torch.empty(spec.vocab, dtype=torch.float32, device=dev)
        self.next_token = torch.zeros(1, dtype=torch.int32, device=dev)
        self.handle = nt.nt_model_init(ctx, model_desc(spec, stream_slots), self.layers, self.embd, self.out,
                                       self.out_norm)

    def hbm_weight_bytes(self) -> int:
        """Weight bytes this model keeps in HBM: resident layers, LM head,
        embedding table when resident, streaming slots."""
        n = sum(t.numel() for L in self.layers for k, t in L.items() if k in LAYER)
        n += self.out.numel() + (self.embd.numel() if isinstance(self.embd, torch.Tensor) and self.embd.is_cuda else 0)
        return n + self.n_slots * (self.blobs.nbytes if self.blobs is not None else 0)

    def step(self, token: int, pos: int, skip=None, stream=None):
        """One decode step; token < 0 continues from the device state."""
        nt.nt_decode_step(self.ctx, self.handle, token, pos, skip, self.logits, self.next_token, stream)
        return self.logits

    def set_sampler(self, temperature: float, top_p: float = 1.0, seed: int = 0):
        """Later decode steps sample (temperature, top-p); temperature <= 0 is greedy."""
        nt.nt_model_set_sampler(self.ctx, self.handle, temperature, top_p, seed)

    def prefill(self, tokens, pos0: int, stream=None):
        """Run a prompt through the model (KV written for pos0 ..); returns the
        logits after its last token.  Decoding continues with step(-1, 0)."""
        nt.nt_prefill(self.ctx, self.handle, tokens, pos0, self.logits, self.next_token, stream)
        return self.logits

    def spec_step(self, token: int, pos: int, k: int, n_draft_layers: int = 0, stream=None):
        """One self-speculative step (token < 0 continues from the device
        state); returns (tokens [k + 1] int32 device tensor, count [1] int32
        device tensor, verify logits [k + 1, vocab]).  The first count tokens
        are the step's output."""
        if not hasattr(self, "spec_tokens"):
            dev = self.logits.device
            self.spec_tokens = torch.zeros(8, dtype=torch.int32, device=dev)
            self.spec_count = torch.zeros(1, dtype=torch.int32, device=dev)
            self.spec_logits = torch.empty(16, self.spec.vocab, dtype=torch.float32, device=dev)
        nt.nt_spec_step(self.ctx, self.handle, token, pos, k, n_draft_layers, self.spec_tokens, self.spec_count,
                        self.spec_logits, stream)
        # with the sampler set, the draft logits follow the verify rows
        self.draft_logits = self.spec_logits[k + 1:2 * k + 1]
        return self.spec_tokens, self.spec_count, self.spec_logits[:k + 1]

    def calibrate(self, token: int, pos: int, n_skip: int, stream=None):
        return nt.nt_layer_skip_calibrate(self.ctx, self.handle, token, pos, n_skip, self.spec.n_layers,
                                          self.logits, self.next_token, stream)

    def kv(self, layer: int):
        return self.layers[layer]["kcache"], self.layers[layer]["vcache"]

    def close(self):
        if self.handle:
            nt.nt_model_destroy(self.ctx, self.handle)
            self.handle = None
