"""Coded activation checkpoints: the 8-bit rows that a forward pass saves are kept entropy coded until
the backward pass reads them.

The bytes of 8-bit rows (hx.quantize_rows, hx.gated_forward, hx.head_norm_rope_forward) are e4m3 or
INT8 symbols, which the fixed-codebook coder shortens without loss ("Single-Stage Huffman Encoder for ML
Compression", abstract: the codebook comes from earlier batches, so coding needs no pass of its own
over the data). The scales, one per row, stay as they are.

    store = CheckpointStore(tables)          # a table block (Codebook.upload)
    key = store.put(data, scale)             # forward: coded on the current stream
    store.seal()                             # streams trimmed to their size (reads the sizes: one wait)
    data, scale = store.take(key)            # backward: decoded, and forgotten by the store
    store.check()                            # once per step: raises if a coding or decoding failed
"""
from __future__ import annotations

from dataclasses import dataclass

from . import hx


@dataclass
class _Entry:
    stream: object
    scale: object
    status: object  # the encoder's status word; None once sealed
    shape: tuple


class CheckpointStore:
    """Coded 8-bit rows by key, on the device of the table block, whichever is current. All calls of a store are made on one
    CUDA stream. `hist` (int32[256] on the
    device), if given, accumulates the histogram of all bytes put, for the next codebook. Errors in the data
    (a byte without a code, a stream that does not decode) are kept on the device until seal() or check() reads
    them; what take() gave before that is not to be relied on."""

    def __init__(self, tables, kind: int = hx.KIND_HUFFMAN, hist=None):
        self.tables, self.kind, self.hist = tables, kind, hist
        self._status = hx.new_status(tables.device)
        self._entries: dict[int, _Entry] = {}
        self._next = 0
        self._scratch = None

    def put(self, data, scale) -> int:
        """Codes the bytes of 8-bit rows and keeps them with their scales; returns their key. `data` is not
        needed afterwards. `scale` is kept as it is, not copied: take() gives back the same tensor, so it must not be
        written until then (quantize_rows(x, scale=buffer) with one buffer for several layers needs a clone here).
        check() does not notice. Fewer than 2^32 bytes, contiguous, aligned as a torch allocation."""
        import torch
        if data.dtype is not torch.uint8 or not data.is_contiguous():
            raise TypeError("data must be contiguous uint8")
        if data.device != self.tables.device:
            raise ValueError("data must be on the table block's device")
        flat = data.view(-1)
        n = flat.numel()
        if n >= 1 << 32:
            raise ValueError("a stream codes fewer than 2^32 bytes")
        need = hx.scratch_bytes(n)
        if self._scratch is None or self._scratch.numel() < need:
            self._scratch = torch.empty(need, dtype=torch.uint8, device=data.device)
        with torch.cuda.device(self.tables.device):  # the coder launches on the current device
            stream, status = hx.encode(self.tables, flat, scratch=self._scratch, hist=self.hist, kind=self.kind)
        key, self._next = self._next, self._next + 1
        self._entries[key] = _Entry(stream, scale, status, tuple(data.shape))
        return key

    def seal(self) -> None:
        """Moves every stream put since the last call into a buffer of its own size. Waits for the device
        once. Raises HxError if a byte had no code (the entry is dropped, the others are sealed)."""
        import torch
        fresh = [(k, e) for k, e in self._entries.items() if e.status is not None]
        if not fresh:
            return
        words = torch.stack([e.stream[32:40].view(torch.int64)[0] for _, e in fresh])
        codes = torch.cat([e.status for _, e in fresh])
        words, codes = words.cpu().tolist(), codes.cpu().tolist()
        failed = 0
        for (key, e), w, code in zip(fresh, words, codes):
            if code:
                failed |= code
                del self._entries[key]
                continue
            n = 1
            for d in e.shape:
                n *= d
            e.stream, e.status = e.stream[:hx.stream_bytes(n, w)].clone(), None
        if failed:
            raise hx.HxError(failed, "CheckpointStore.seal")

    def take(self, key: int):
        """Decodes the rows of `key`: (bytes, scale). The store forgets them."""
        import torch
        e = self._entries.pop(key)
        if e.status is not None:  # not sealed: what its coding raised is read by check()
            self._status |= e.status
        n = 1
        for d in e.shape:
            n *= d
        out = torch.empty(max(n, 1), dtype=torch.uint8, device=e.stream.device)[:n]
        with torch.cuda.device(self.tables.device):
            hx.decode(self.tables, e.stream, n, out=out, status=self._status, kind=self.kind)
        return out.view(e.shape), e.scale

    def check(self) -> None:
        """Waits for the device and raises HxError if anything taken so far was not coded or decoded exactly."""
        code = int(self._status.item())
        if code:
            self._status.zero_()
            raise hx.HxError(code, "CheckpointStore.check")

    def nbytes(self) -> int:
        """Device bytes of the streams and scales held."""
        return sum(e.stream.numel() + e.scale.numel() * e.scale.element_size() for e in self._entries.values())

    def __len__(self) -> int:
        return len(self._entries)
