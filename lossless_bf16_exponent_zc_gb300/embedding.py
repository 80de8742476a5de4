"""The rows of an embedding table for a run of token ids, scaled: where the residual stream starts.

    x = embedding.lookup(ids, table, status, scale=hidden ** 0.5)                     # [tokens, hidden]
    dtable = embedding.lookup_backward(dx, ids, len(table), ws, status, scale=hidden ** 0.5)

The gradient sorts the tokens by id, adds up every id's rows in float32, in the order of its tokens within runs of up to 32
sorted tokens and then run by run, and writes each row of the table once.  So the same inputs give the same bits on one kind
of GPU (the runs' length follows from its SMs).  Kernels: zc_embedding and zc_embedding_backward (include/zc.h);
arguments are checked, and outputs that are not given allocated, in the native extension (csrc/zc_torch.cpp).  The rows
are bfloat16, float16 or float32; the table has their type or float32.  ids: int32 or int64 [tokens]; a negative id is
no token, an id beyond the table sets ERR_BAD_INDEX in status and is taken for none.

Calls run on the current torch stream, or on the one given as ``stream``.  On a given stream, what it reads and the
outputs it is handed must be ready there (``stream.wait_stream(...)``) and stay alive until it has run; outputs it makes
are that stream's, to be used elsewhere once that place waits for it.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import zc


@functools.lru_cache(maxsize=4096)
def workspace_size(tokens: int, vocab: int, hidden: int) -> int:
    out = ctypes.c_uint64()
    zc._check(zc.load().zc_embedding_workspace_size(int(tokens), int(vocab), int(hidden), ctypes.byref(out)),
              "zc_embedding_workspace_size")
    return out.value


def workspace(tokens: int, vocab: int, hidden: int, device="cuda") -> torch.Tensor:
    """A workspace for the gradients of up to so many tokens; calls that share it must be ordered on one stream."""
    return torch.empty(workspace_size(tokens, vocab, hidden), dtype=torch.uint8, device=device)


def lookup(ids: torch.Tensor, table: torch.Tensor, status: torch.Tensor, *, scale: float = 1.0,
           dtype: torch.dtype | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """scale * table[ids]: [tokens, hidden], of type dtype (None: the table's).  The rows of negative ids are zero."""
    return zc.native().embedding(ids, table, status, scale, dtype, out, stream)[0]


def lookup_backward(dout: torch.Tensor, ids: torch.Tensor, vocab: int, ws: torch.Tensor, status: torch.Tensor, *,
                    scale: float = 1.0, dtype: torch.dtype | None = None, dtable: torch.Tensor | None = None,
                    accumulate: bool = False, stream=None) -> torch.Tensor:
    """Gradient of the table, [vocab, hidden] of type dtype (None: dtable's, or dout's): zero for ids without a token.
    With accumulate the sums are added to what dtable holds, and other rows are left alone."""
    return zc.native().embedding_backward(dout, ids, vocab, ws, status, scale, dtype, dtable, accumulate, stream)[0]
