"""Workspaces that the older blocks allocate themselves, for a call on a given stream: they are
allocated with that stream as the current one, so that the allocator orders their reuse by it."""
import pytest
import torch

import linear_attention_recurrence_10_b200 as gdr
from gdr_testutil import run_prefill
from linear_attention_recurrence_10_b200 import synth

pytestmark = pytest.mark.gpu


def _prefill(stream):
    return run_prefill(synth.make_inputs([70, 200], 2, 4, 128, seed=5, s0_std=0.02), stream=stream)[0]


def _attn(stream):
    g = torch.Generator().manual_seed(6)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    out = torch.empty(2, 16, 256, device="cuda")
    q, gate, k, v, kc, vc = bf(2, 16, 256), bf(2, 16, 256), bf(2, 2, 256), bf(2, 2, 256), \
        bf(2, 2, 900, 256), bf(2, 2, 900, 256)
    lens = torch.tensor([800, 17], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    return gdr.attn_decode_step(q, gate, k, v, kc, vc, lens, out, kv_bound=850, stream=stream)


def _moe(stream):
    g = torch.Generator().manual_seed(7)
    bf = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16).cuda()
    out = torch.empty(3, 256, device="cuda")
    args = bf(3, 256), bf(16, 256), bf(16, 128, 256), bf(16, 256, 64)
    torch.cuda.synchronize()
    return gdr.moe_decode(*args, out, top_k=4, stream=stream)


@pytest.mark.parametrize("call", [_prefill, _attn, _moe], ids=lambda f: f.__name__[1:])
def test_workspace_belongs_to_the_stream(monkeypatch, call):
    want = call(None).clone()
    torch.cuda.synchronize()
    streams, empty = [], torch.empty

    def spy(*a, **kw):
        if kw.get("dtype") is torch.uint8:
            streams.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", spy)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        streams.clear()
        got = call(stream)
        assert streams == [side.cuda_stream]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
