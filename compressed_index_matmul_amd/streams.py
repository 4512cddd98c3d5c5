"""The stream a call runs on, and memory for what the call allocates itself.

torch's caching allocator hands a block that was freed on a stream out again
for that same stream at once, while work queued there may still use it.  What
a call writes on a stream of its own therefore has to come from that stream's
blocks: memory of the current stream's would need an order between the two.
"""
from __future__ import annotations

import torch

# The current stream's handle without building Python objects (2 us a call);
# the public call where this torch has no such name.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


def resolve(stream, dev):
    """(raw handle of the stream to launch on, torch stream to allocate under).
    `stream`: a torch stream, a raw handle or None for `dev`'s current stream;
    the second is None where that one is meant."""
    current = _raw_stream(dev.index)
    if stream is None:
        return current, None
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == current:
        return handle, None
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    return handle, stream


def empty(shape, dtype, dev, st, returned: bool = True):
    """A new tensor for a call that runs on `st` (None: the current stream), in
    memory of that stream.  `returned`: the caller gets it and may use it on
    the current stream too, so it is kept from reuse for that one as well."""
    if st is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(st):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if returned:
        t.record_stream(torch.cuda.current_stream(dev))
    return t
