"""Edges of the paged cache's operators (gdr_kv_append, gdr_kv_gather, gdr_attn_paged) against
their formulas in 64 bits; bounds in paged_testutil where a test states no other."""
import pytest
import torch

import linear_attention_recurrence_10_b200 as gdr
from paged_testutil import D, NAN, U8, Problem, rope64, status_of

pytestmark = pytest.mark.gpu


# ------------------------------------------------- rows past a sequence's end


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_last_tiles_of_every_length(kind):
    """Chunks that end at every place of a step of the products (16 keys, 32 codes), at either
    half of a tile: what the pages hold behind them (NaN) is cleared before it is multiplied, by
    both blocks of a pair for both, and every call gives the first one's bits."""
    past = [0, 64, 128, 300]
    for i in range(8):
        new = [257 + 5 * i + j for j in range(4)]
        p = Problem(new=new, past=past, page=[16, 64, 128, 256][i % 4], kind=kind, seed=400 + i)
        assert p.rows * 8 >= 256 * p.n_seq  # (pairs, for bf16)
        p.put_plain()
        out, lse, ws = p.attend()
        assert status_of(ws) == 0
        p.check_attend(out, lse, what=i)
        for _ in range(20):
            again, lse2, _ = p.attend(workspace=ws)
            assert torch.equal(out, again) and torch.equal(lse, lse2)


# ------------------------------------------------- workspaces that a call allocates


def given_workspace(monkeypatch):
    """The workspaces' addresses of the calls to come."""
    seen, queue = [], gdr._queue

    def spy(f, name, packed, more, stream, *tensors):
        seen.append(more[0] if more else None)
        return queue(f, name, packed, more, stream, *tensors)

    monkeypatch.setattr(gdr, "_queue", spy)
    return seen


@pytest.mark.parametrize("handle", ["stream", "integer"])
def test_allocated_workspace_is_not_in_use_elsewhere(monkeypatch, handle):
    """A call on a stream of its own while the current stream still has work on a block of the
    workspace's size that has just been freed: the call does not get that block, and neither
    the call's result nor the block's last values change."""
    p = Problem(new=[300], past=[3000], page=64, seed=320)
    p.put_plain()
    want, _, ws = p.attend()
    n = ws.numel()
    del ws
    seen = given_workspace(monkeypatch)
    a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    b, out = torch.empty_like(a), torch.empty_like(p.q)
    s = torch.cuda.Stream()
    # (A block of this size comes from no larger one: the pool holds none that is free.)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        for _ in range(40):
            torch.mm(a, a, out=b)
        block = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        at, low = block.data_ptr(), block.amin()
        del block
        gdr.attn_paged(p.q, *p.pages, p.cache_len, out, gate=p.gate,
                       stream=s if handle == "stream" else s.cuda_stream)
        assert seen[-1] != at
        torch.cuda.synchronize()
        assert int(low) == 0xFF and torch.equal(out, want)


def test_allocated_workspace_on_the_default_stream_by_its_handle(monkeypatch):
    """stream=0 is the device's default stream, whichever is current."""
    p = Problem(new=[40], past=[300], page=64, seed=321)
    p.put_plain()
    want, _, ws = p.attend()
    n, out = ws.numel(), torch.empty_like(p.q)
    del ws
    seen = given_workspace(monkeypatch)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block = torch.empty(n, dtype=torch.uint8, device="cuda")
        at = block.data_ptr()
        del block
        gdr.attn_paged(p.q, *p.pages, p.cache_len, out, gate=p.gate, stream=0)
    assert seen[-1] != at
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ gates


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,past", [([1] * 300, [90] * 300),        # items in one piece, most of them
                                      ([1, 3], [9000, 20]),           # an item in many pieces
                                      ([260, 300, 280], [0, 40, 0])])  # (pairs, for bf16)
def test_gates_of_any_value(kind, new, past):
    """NaN, infinite and far gates change their own value alone, whether or not the split of
    the work has cut their item.  Beside the same call without gates, in fp32, an output is off by
    the sigmoid: u = g log2(e) is rounded twice, |u| <= 128 (2^-24 + 2^-24), its power, the
    reciprocal and the products add less than 2^-20 in all: 2^-16 relative; below 2^-126 it may
    be 0.  A bf16 output rounds by U8 relative, and below 2^-126, where bf16's steps are
    2^-126 2^-7 = 2^-133, by half of one."""
    p = Problem(new=new, past=past, page=64, kind=kind, seed=420)
    p.put_plain()
    plain, _, ws = p.attend(gate=False, out_dtype=torch.float32)
    assert status_of(ws) == 0
    p.check_attend(plain, None, gate=False)
    values = [NAN, float("inf"), -float("inf"), -41.5, -41.75, -50.0, -80.0, -87.5, -100.0, -3e38, 41.75, 60.0,
              3e38, -NAN, 0.0]
    g = torch.Generator().manual_seed(421)
    for share in (0.002, 0.5):  # one of a row's gates, now and then; half of them
        at = (torch.rand(p.gate.shape, generator=g) < share).cuda()
        which = torch.randint(0, len(values), p.gate.shape, generator=g).cuda()
        p.gate = torch.where(at, torch.tensor(values, device="cuda").bfloat16()[which], p.gate)
        want = plain.double() * torch.sigmoid(p.gate.double())
        bad = torch.isnan(p.gate)
        assert bad.any() and torch.equal(torch.isnan(want), bad)
        for dtype in (torch.float32, torch.bfloat16):
            out, _, ws = p.attend(out_dtype=dtype)
            assert status_of(ws) == 0
            assert torch.equal(torch.isnan(out), bad)
            half = 2.0 ** -16 + (U8 if dtype is torch.bfloat16 else 0)
            off = (out.double() - want).abs() - half * want.abs() - 2.0 ** -125 * plain.double().abs()
            if dtype is torch.bfloat16:
                off = off - 2.0 ** -134
            assert (off[~bad] <= 0).all(), (dtype, float(off[~bad].max()))
