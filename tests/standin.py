"""Stand-ins for CUDA tensors, streams and the library behind the C half of the
binding, so that what it does before and around a call can be looked at
without a GPU: a tensor that says it is on device 0, and library functions
that record their arguments and return 0."""
import contextlib
import ctypes
import types

import newton_schulz_fp32_gb300 as nsg

P, I, I64, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "muon_embedding": (P, I, I64, I, I, P, I, I64, F, P, I, I64, P),
    "muon_embedding_grad": (P, I64, P, I, I64, P, I, I64, F, I, P, P, I, P, S, P),
    "muon_token_logprobs": (P, I, I64, I64, I, P, I, F, P, P),
    "muon_policy_loss": (P, I, I64, I64, I, P, I, P, P, P, P, F, F, F, F, P, P, P, I64, P),
    "muon_preference_loss": (P, I, I64, I64, I, P, I, P, I, I, P, P, F, F, F, P, P, P, P, I64, P, S, P)}
REAL = ("muon_last_error", "muon_embedding_grad_workspace", "muon_preference_loss_workspace")


class Tensor:
    """A CPU tensor that says it is on a CUDA device."""

    def __init__(self, t, machine, index=0):
        self.t, self.machine, self.index = t, machine, index
        self.shape, self.dtype = t.shape, t.dtype
        self.device = types.SimpleNamespace(type="cuda", index=index)

    def _of(self, t):
        if t.untyped_storage().data_ptr() != self.t.untyped_storage().data_ptr():
            self.machine.copies.append(self.machine.stream)
        return Tensor(t, self.machine, self.index)

    def get_device(self):
        return self.index

    def reshape(self, *shape):
        return self._of(self.t.reshape(*shape))

    def view(self, *shape):
        return self._of(self.t.view(*shape))

    def narrow(self, *a):
        return self._of(self.t.narrow(*a))

    def __getattr__(self, name):   # stride, numel, is_contiguous, data_ptr, element_size, dim
        return getattr(self.t, name)


class Machine:
    """Torch's current device and stream, the copies made (by stream) and the
    library's calls: (name, arguments)."""

    def __init__(self, torch):
        self.torch, self.device, self.stream = torch, 0, 0
        self.copies, self.calls, self.made = [], [], []

    def tensor(self, t, index=0):
        return Tensor(t, self, index)

    def empty(self, size, dtype=None, device=None):
        self.made.append(Tensor(self.torch.empty(size, dtype=dtype), self, device.index))
        return self.made[-1]

    def on_stream(self, handle, index=0):
        """A torch stream."""
        return types.SimpleNamespace(cuda_stream=handle, device=types.SimpleNamespace(type="cuda", index=index))

    @contextlib.contextmanager
    def enter(self, device=None, stream=None):
        old = self.device, self.stream
        if device is not None:
            self.device = getattr(device, "index", device)
        if stream is not None:
            self.device, self.stream = stream.device.index, stream.cuda_stream
        try:
            yield
        finally:
            self.device, self.stream = old


@contextlib.contextmanager
def machine(monkeypatch):
    """The binding over stand-ins."""
    import torch
    nsg.build()
    m = Machine(torch)
    keep = []

    def recorder(name):
        def call(*args):
            m.calls.append((name, args))
            return 0
        f = ctypes.CFUNCTYPE(I, *SIGNATURES[name])(call)
        keep.append(f)
        return ctypes.cast(f, P).value

    table = {name: recorder(name) for name in SIGNATURES}
    table.update({name: ctypes.cast(getattr(nsg.lib(), name), P).value for name in REAL})
    fake = types.SimpleNamespace(empty=m.empty, bfloat16=torch.bfloat16, float32=torch.float32, int32=torch.int32,
                                 int64=torch.int64, uint8=torch.uint8)
    monkeypatch.setattr(torch.cuda, "device", lambda d: m.enter(device=d))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: m.enter(stream=s))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: m.on_stream(h, device.index))
    nsg._native().init(fake, lambda: m.device, lambda d: m.stream, nsg.MuonError, table)
    try:
        yield m
    finally:
        nsg._bound = None   # the next call binds the library itself
        nsg._native()
