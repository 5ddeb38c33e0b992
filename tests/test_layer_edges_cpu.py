"""The layer operators on the host: whose memory a call takes."""
import contextlib

import pytest
import torch

from nvfp4_block_scaled_amax_amd import _binding, api


class Streams:
    """torch's streams and the library, without a device: which stream was current
    when a buffer was made, and what every library call was given."""

    def __init__(self, monkeypatch):
        self.now, self.made, self.calls = "current", {}, []
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, **kw: f"handle {h}")
        monkeypatch.setattr(api, "_empty", self.empty)
        for name in ("mxq_moe_route", "mxq_moe_combine", "mxq_nvfp4_expert_gateup",
                     "mxq_nvfp4_expert_matvec", "mxq_nvfp4_attention"):
            monkeypatch.setattr(_binding, name, lambda *a: self.calls.append(a))
        for name in ("mxq_moe_route_workspace", "mxq_nvfp4_attention_workspace"):
            monkeypatch.setattr(_binding, name, lambda *a: 256)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    def empty(self, shape, dtype, like):
        t = torch.zeros(shape, dtype=dtype)
        self.made[id(t)] = (t, self.now)
        return t

    def hidden(self, result):
        """The streams of the buffers that the library used and the caller does not hold."""
        kept = {id(t) for t in (result if isinstance(result, tuple) else (result,))}
        used = {id(a) for c in self.calls for a in c if isinstance(a, torch.Tensor)}
        return [s for i, (_, s) in self.made.items() if i in used and i not in kept]


def nvfp4(*shape):
    return api.NVFP4(torch.zeros(*shape[:-1], shape[-1] // 2, dtype=torch.uint8),
                     torch.zeros(*shape[:-1], shape[-1] // 16, dtype=torch.uint8),
                     torch.zeros(shape[0]))


def calls():
    i64 = torch.int64
    maps = api.Routing(torch.zeros(4, 2), torch.zeros(4, 2, dtype=i64),
                       torch.zeros(4, 2, dtype=i64), torch.zeros(8, dtype=i64),
                       torch.zeros(4, dtype=i64))
    up, dn = nvfp4(3, 32, 64), nvfp4(3, 64, 32)
    pair = api.GateUpNVFP4(*up[:2], *up[:2], up[2])
    down = api.GateUpNVFP4(*dn[:2], None, None, dn[2])
    x, q = torch.zeros(4, 64).bfloat16(), torch.zeros(1, 1, 4, 64).bfloat16()
    return [
        (1, lambda s: api.moe_route(torch.zeros(4, 3), 2, stream=s)),
        (2, lambda s: api.nvfp4_expert_layer(x, maps, pair, down, stream=s)),
        (1, lambda s: api.nvfp4_attention(q, nvfp4(64, 64), nvfp4(64, 64),
                                          torch.zeros(1, 2, dtype=i64),
                                          torch.zeros(1, dtype=i64), 2, 16, stream=s)),
    ]


@pytest.mark.parametrize("stream,owner", [(None, "current"), ("side", "side"), (77, "handle 77")])
def test_what_a_call_lets_go_on_return_belongs_to_its_stream(monkeypatch, stream, owner):
    """Otherwise the current stream's next allocation could take it while the
    kernels on `stream` still use it."""
    for n, call in calls():
        s = Streams(monkeypatch)
        assert s.hidden(call(stream)) == [owner] * n
        assert all(c[-1] == stream for c in s.calls)
