"""Edges of the paged cache's operators (gdr_kv_append, gdr_kv_gather, gdr_attn_paged) against
their formulas in 64 bits; bounds in paged_testutil where a test states no other."""
import math
import time

import pytest
import torch

import linear_attention_recurrence_10_b200 as gdr
from linear_attention_recurrence_10_b200 import _abi
from paged_testutil import D, NAN, U8, Problem, rope64, status_of
from test_paged_gpu import check_append, snapshot

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


# ------------------------------------- weights far below the largest, over codes


def shaped_codes(bits, v, H_q, H_kv, new, n_seq, seed):
    """n_seq sequences over the same pages of codes: token j's score is about bits[j, h] (log2) for
    kv head h, its value v[j, h].  The last `new` tokens of each are its new ones."""
    n = bits.shape[0]
    p = Problem(new=[1], past=[0], H_q=H_q, H_kv=H_kv, page=128, kind="e4m3", seed=seed)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(n_seq * new, H_q, D, generator=g)
    k = 0.15 * torch.randn(n, H_kv, D, generator=g)  # scores of about 0.2 besides
    q[..., 0], k[..., 0] = 32.0, bits * (math.log(2) * D ** 0.5 / 32.0)
    n_pages = -(-n // 128)
    order = torch.randperm(n_pages, generator=g)

    def quantised(x):
        x = torch.cat([x, x.new_full((n_pages * 128 - n, H_kv, D), NAN)])
        x = x.view(n_pages, 128, H_kv, D).transpose(1, 2)[order.argsort()].contiguous().cuda()
        scale = (x.abs().amax(-1) / 448).clamp_min(2.0 ** -40)
        return (x / scale[..., None]).to(torch.float8_e4m3fn), scale

    p.k_pages, p.k_scale = quantised(k)
    p.v_pages, p.v_scale = quantised(v)
    p.q = q.bfloat16().cuda()
    p.gate = torch.full_like(p.q, -41.5)
    p.table = order.to(torch.int32).repeat(n_seq, 1).cuda().contiguous()
    p.new, p.past, p.len = [new] * n_seq, [n - new] * n_seq, [n] * n_seq
    p.n_seq, p.rows, p.n_tok, p.n_pages, p.width = n_seq, n_seq * new, n_seq * new, n_pages, n_pages
    p.cu = (torch.arange(n_seq + 1) * new).to(torch.int32).cuda()
    p.cache_len = torch.full((n_seq,), n - new, dtype=torch.int32, device="cuda")
    return p


def check_codes(p, out, lse, tag):
    """Against the formula, with a bound that does not grow with the number of keys.

    A weight is off by (u8 + 2^-11) of itself or by 2^-14 + 2^-17 < 2^-13.8 where it is below 2^-6,
    at a scale where the reference is 2^6: 2^-19.8 of the reference, which is at most 2^5 times
    the largest weight of the tile of 128 keys, or 2^-40 times the row's largest of all.  d, as
    elsewhere, is the scores' error: fp32 sums, and Q's parts, off by 2^-17 of the row's largest
    value each."""
    n, rows = p.len[0], p.rows
    k, _ = p.cached("k", 0)
    v, vs = p.cached("v", 0)
    q = p.q.double().unflatten(1, (p.H_kv, -1))
    last = p.past[0] + torch.arange(rows, device="cuda") % p.new[0]
    at_tile = torch.arange(n, device="cuda") // 128
    n_tile = int(at_tile[-1]) + 1
    worst = 0.0
    for h in range(p.H_kv):
        for r in range(q.shape[2]):
            x = q[:, h, r]
            off = torch.arange(n, device="cuda") > last[:, None]
            a = (x @ k[:, h].t() * D ** -0.5).masked_fill(off, -math.inf)
            ref_lse = torch.logsumexp(a, -1)
            P = torch.exp(a - ref_lse[:, None])
            y = P @ v[:, h]
            # (a score far below the row's largest does not matter: bounded by those that weigh)
            heavy = P > 2.0 ** -40
            d = (x.abs() @ k[:, h].abs().t() * 256 * 2.0 ** -24
                 + x.abs().amax(-1, keepdim=True) * 2.0 ** -17 * k[:, h].abs().sum(-1)) * D ** -0.5
            d = torch.where(heavy, d, 0).amax(-1, keepdim=True)
            W = P * vs[:, h]
            top = torch.zeros(rows, n_tile, dtype=torch.float64, device="cuda").scatter_reduce(
                1, at_tile.expand(rows, -1), W, "amax") + 2.0 ** -45 * W.amax(-1, keepdim=True)
            codes = torch.zeros(n_tile, D, dtype=torch.float64, device="cuda").index_add(
                0, at_tile, (v[:, h] / vs[:, h, None]).abs())
            tol = (U8 + 2.0 ** -11 + 2 * d + 2.0 ** -19) * (P @ v[:, h].abs()) + 2.0 ** -14.8 * (top @ codes)
            head = h * q.shape[2] + r
            err = (out[:, head].double() - y).abs()
            assert (err <= tol).all(), (tag, head, float((err / tol).max()))
            e = (lse[:, head].double() - ref_lse).abs()
            assert (e <= d[:, 0] + 2.0 ** -19 + 2.0 ** -21 * ref_lse.abs()).all(), (tag, head, float(e.max()))
            worst = max(worst, float(err.norm() / y.norm()))
    # the weights' roundings are independent: u8 / sqrt(3), as elsewhere; 20 rows estimate it within 1.25
    assert worst <= 1.25 * U8 / math.sqrt(3), (tag, worst)


@pytest.mark.parametrize("layout", [(8, 8, 1, 20), (16, 2, 200, 1)])
@pytest.mark.parametrize("shape", ["first key", "first value", "first tile", "falling", "steps"])
def test_codes_keep_weights_far_below_the_largest(shape, layout):
    """Long caches of codes in which the weights' sizes change along the sequence, with values
    whose mean is not zero, so that what is lost shows: one dominant key and many keys of a 2^8th to
    a 2^20th of its weight; a value row of another size; scores that fall, or go up and down."""
    H_q, H_kv, new, n_seq = layout
    n = 32768 if new == 1 else 20001
    g = torch.Generator().manual_seed(431)
    j = torch.arange(n)[:, None]
    step = (torch.tensor([8.0, 11.0, 13.0, 14.0, 15.0, 16.0, 17.0, 20.0]) if H_kv == 8 else
            torch.tensor([13.0, 16.0]))
    v = 1 + 0.5 * torch.randn(n, H_kv, D, generator=g)
    if shape == "first key":
        bits = torch.where(j == 0, step, 0.0)
        v[0] = -v[0]
    elif shape == "first value":
        bits = torch.where(j == 0, step - 10, 0.0)
        v[0] *= -1024
    elif shape == "first tile":
        bits = torch.where(j < 100, step - 3, 0.0)
        v[:100] *= -1
    elif shape == "falling":
        bits = step * (1 - 2.5 * j / n)
        v[: n // 3] *= -1
    else:
        bits = torch.where((j // 700) % 2 == 0, step * 0.75, 0.0) + 4 * torch.sin(j / 3000.0)
        v = torch.where(((j // 700) % 2 == 0)[..., None], v, -2 * v)
    p = shaped_codes(bits, v, H_q, H_kv, new, n_seq, seed=430)
    out, lse, ws = p.attend(gate=False, out_dtype=torch.float32)
    assert status_of(ws) == 0
    check_codes(p, out, lse, shape)
    again, _, _ = p.attend(gate=False, out_dtype=torch.float32)
    assert torch.equal(out, again)
    # Gates of -41.5: what is left of 2^-60 keeps its relative precision (bound: test_gates_of_any_value).
    small, _, _ = p.attend(out_dtype=torch.float32)
    want = out.double() * torch.sigmoid(p.gate.double())
    assert ((small.double() - want).abs() <= 2.0 ** -16 * want.abs()).all()


# ---------------------------------------------------------- the longest sequences


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_longest_sequence(kind):
    """A sequence has fewer than 2^31 - 256 tokens: the last one that may be is written, read back
    and rotated, the next is refused by every call, although the table has a page for it."""
    p = Problem(new=[2], past=[0], page=1024, kind=kind, seed=440)
    last = (1 << 31) - 258  # its position
    table = torch.full((1, 1 << 21), -1, dtype=torch.int32, device="cuda")
    table[0, last // 1024] = p.table[0, 0]
    p.table, p.cache_len = table, torch.tensor([last], dtype=torch.int32, device="cuda")
    before = p.k_pages.clone(), p.v_pages.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = p.append(status=status)
    assert int(status) == 1
    want, slack = rope64(p.q[:1], torch.tensor([last], device="cuda"), 64, 1e7)
    assert ((q_out[:1].double() - want).abs() <= U8 * want.abs() * (1 + U8) + slack).all()
    page, row = int(table[0, last // 1024]), last % 1024
    for now, old in zip((p.k_pages, p.v_pages), before):
        changed = (now.view(torch.uint8) != old.view(torch.uint8)).flatten(3).any(-1).nonzero()
        assert changed.cpu().tolist() == [[page, 0, row], [page, 1, row]]
    v = torch.full((2, 2, D), NAN, device="cuda")
    status.zero_()
    gdr.kv_gather(*p.pages, None, v, **p.scales, first=p.cache_len, status=status)
    assert int(status) == 1
    half = 2.0 ** -4 * 1.01 if kind == "e4m3" else 0.0
    top = p.v[0].double().abs().amax(-1, keepdim=True)
    assert ((v[0].double() - p.v[0].double()).abs() <= half * p.v[0].double().abs() +
            (2.0 ** -18 * top if kind == "e4m3" else 0)).all()
    p.cache_len += 1
    p.cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out, lse, ws = p.attend()
    assert status_of(ws) == 1


# ------------------------------------------------- prompts, and long read-backs


def many(n, seed):
    """Lengths that sum to about n: many empty sequences and of one token, some of tens, a few
    of hundreds, in any order."""
    g = torch.Generator().manual_seed(seed)
    out = []
    while sum(out) < n:
        most = [0, 1, 1, 9, 40, 400][int(torch.randint(0, 6, (1,), generator=g))]
        out.append(int(torch.randint(0, most + 1, (1,), generator=g)))
    out[-1] -= sum(out) - n
    return out


def pasts(count, seed):
    g = torch.Generator().manual_seed(seed + 1)
    return torch.randint(0, 60, (count,), generator=g).tolist()


LONG = [(593, (16, 2), 64, 64), (601, (8, 8), 16, 30), (3001, (16, 2), 32, 64), (2999, (3, 1), 128, 30),
        (4096, (8, 8), 256, 256), (1237, (128, 1), 16, 64)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,heads,page,rot_dim", LONG)
def test_append_prompts(n, heads, page, rot_dim, kind):
    """More packed rows than blocks take one by one: blocks of several tokens, whose sequences
    begin, end and are empty inside a block, and a last block that is not full."""
    new = many(n, n)
    p = Problem(new=new, past=pasts(len(new), n), H_q=heads[0], H_kv=heads[1], page=page, kind=kind, seed=n,
                tail=n % 7)
    before = snapshot(p)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = p.append(rot_dim=rot_dim, status=status)
    assert int(status) == 0
    check_append(p, q_out, before, rot_dim)
    after = snapshot(p)
    # in place and without queries: the same rows
    for name, t in before.items():
        getattr(p, name).copy_(t)
    q = p.q.clone()
    assert p.append(q=q, q_out=q, rot_dim=rot_dim) is q
    assert torch.equal(q[:n], q_out[:n]) and torch.equal(q[n:], p.q[n:])
    for name, t in after.items():
        assert torch.equal(getattr(p, name).view(torch.uint8), t.view(torch.uint8)), name
        getattr(p, name).copy_(before[name])
    gdr.kv_append(p.k, p.v, p.k_pages, p.v_pages, p.table, p.cu, p.cache_len, rot_dim=rot_dim, **p.scales)
    for name, t in after.items():
        assert torch.equal(getattr(p, name).view(torch.uint8), t.view(torch.uint8)), name


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_prompts_with_bad_pages(kind):
    """Bad pages and lengths inside blocks of several tokens: the tokens around them are written."""
    p = Problem(new=[700, 5, 800, 0, 90], past=[3, 0, 0, 4, 1], page=16, kind=kind, seed=450)
    before = snapshot(p)
    good = p.table.clone()
    bad = [(0, 7), (2, 20), (2, 21)]
    for s, i in bad:
        p.table[s, i] = [-1, p.n_pages, 1 << 30][i % 3]
    p.cache_len[1] = -3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = p.append(status=status)
    assert int(status) == 1
    # what was not written is put there by hand, and the rest has to be right
    want = Problem(new=p.new, past=p.past, page=16, kind=kind, seed=450)
    want.append()
    p.table, p.cache_len = good, want.cache_len
    lost = torch.zeros(p.n_pages, 16, dtype=torch.bool, device="cuda")
    for s, i in bad:
        lost[good[s, i].long()] = True
    lost[good[1, 0].long(), :5] = True
    for name, old in before.items():
        bits = torch.int32 if name.endswith("scale") else torch.uint8
        now, ref, old = (t.view(bits) for t in (getattr(p, name), getattr(want, name), old))
        at = lost[:, None].expand(now.shape[:3])
        assert torch.equal(now[at], old[at]), name
        now[at] = ref[at]
    q_out[700:705] = rope64(p.q[700:705], torch.arange(5, device="cuda"), 64, 1e7)[0].bfloat16()
    check_append(p, q_out, before)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,heads,page,_", LONG)
def test_gather_many(n, heads, page, _, dtype, kind):
    """More packed rows than blocks take one by one, from the middle of sequences, both sides and
    one, into rows of a wider tensor."""
    past = [m + 70 for m in many(n, n + 1)]
    p = Problem(new=[0] * len(past), past=past, H_q=heads[0], H_kv=heads[1], page=page, kind=kind, seed=n + 2)
    take = [m - 70 for m in past]
    first = pasts(len(past), n + 3)
    cu = torch.tensor([0] + take).cumsum(0).to(torch.int32).cuda()
    begin = torch.tensor(first, dtype=torch.int32, device="cuda")
    want = [torch.cat([p.cached(name, s)[0][f:f + t] for s, (f, t) in enumerate(zip(first, take))]).float().to(dtype)
            for name in "kv"]
    wide = torch.full((n + 5, 2 * heads[1] + 1, D), NAN, dtype=dtype, device="cuda")
    k, v = wide[:, :heads[1]], wide[:, heads[1]:2 * heads[1]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdr.kv_gather(*p.pages[:3], cu, k, v, **p.scales, first=begin, status=status)
    assert int(status) == 0
    assert torch.equal(k[:n], want[0]) and torch.equal(v[:n], want[1])
    assert torch.isnan(wide[n:]).all() and torch.isnan(wide[:, -1]).all()
    for side in range(2):
        one = torch.full((n + 5, heads[1], D), NAN, dtype=dtype, device="cuda")
        gdr.kv_gather(*p.pages[:3], cu, *((one, None) if side == 0 else (None, one)), **p.scales, first=begin)
        assert torch.equal(one[:n], want[side]) and torch.isnan(one[n:]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_gather_many_with_bad_pages(kind):
    p = Problem(new=[0, 0, 0], past=[900, 30, 700], page=16, kind=kind, seed=460)
    good = p.table.clone()
    want = [torch.cat([p.cached(name, s)[0] for s in range(3)]).bfloat16() for name in "kv"]
    p.table[0, 9], p.table[2, 33] = -5, p.n_pages
    cu = torch.tensor([0, 900, 930, 1630], dtype=torch.int32, device="cuda")
    out = [torch.full((1630, 2, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdr.kv_gather(*p.pages[:3], cu, *out, **p.scales, status=status)
    assert int(status) == 1 and not torch.equal(p.table, good)
    keep = torch.ones(1630, dtype=torch.bool, device="cuda")
    keep[9 * 16:10 * 16] = False
    keep[930 + 33 * 16:930 + 34 * 16] = False
    for got, ref in zip(out, want):
        assert torch.equal(got[keep], ref[keep])


def test_append_and_gather_many_on_a_captured_stream():
    """A prompt's append and the read-back captured once, replayed with other lengths."""
    sizes = [[700, 300, 0], [0, 1, 900], [333, 333, 334]]
    p = Problem(new=sizes[0], past=[0, 50, 7], page=64, kind="e4m3", seed=470, width=20, spare=30)
    q_out = torch.empty_like(p.q)
    k, v = (torch.empty(1000, 2, D, device="cuda") for _ in "kv")
    calls = lambda: (gdr.kv_append(p.k, p.v, p.k_pages, p.v_pages, p.table, p.cu, p.cache_len, q=p.q, q_out=q_out,
                                   **p.scales),
                     gdr.kv_gather(*p.pages, k, v, first=p.cache_len, **p.scales))
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i, new in enumerate(sizes):
        x = Problem(new=new, past=[0, 50, 7], page=64, kind="e4m3", seed=471 + i, width=20,
                    tail=1000 - sum(new))
        assert x.n_pages <= p.n_pages
        for name in ("q", "k", "v", "table", "cu", "cache_len"):
            getattr(p, name).copy_(getattr(x, name))
        for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
            getattr(p, name)[:x.n_pages].copy_(getattr(x, name))
        before = snapshot(x)
        for t in (q_out, k, v):
            t.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for name in before:
            setattr(x, name, getattr(p, name)[:x.n_pages].clone())
        check_append(x, q_out, before)
        n = sum(new)
        for name, got in (("k", k), ("v", v)):
            want = torch.cat([x.cached(name, s)[0][x.past[s]:] for s in range(3)])
            assert torch.equal(got[:n], want.float()) and torch.isnan(got[n:]).all()
    del graph


@pytest.mark.parametrize("times", [16, 1024])
def test_codes_queries_with_an_outlying_value(times):
    """Over codes a query's values are held to 2^-17 of the row's largest: one value `times` the
    others', where the keys have nothing or little, leaves the others coarser (d in check_codes)."""
    n = 3000
    g = torch.Generator().manual_seed(480)
    v = 1 + 0.5 * torch.randn(n, 2, D, generator=g)
    p = shaped_codes(torch.zeros(n, 2), v, 16, 2, 40, 1, seed=481)
    p.q[..., 0] = 0
    p.q[..., 77] = 3.0 * times
    codes = p.k_pages.view(torch.uint8)
    codes[..., 77] = 0
    codes[:, :, ::5, 77] = torch.tensor(1024.0 / times).clamp_max(64).to(torch.float8_e4m3fn).view(torch.uint8).item()
    out, lse, ws = p.attend(gate=False, out_dtype=torch.float32)
    assert status_of(ws) == 0
    check_codes(p, out, lse, times)


# ------------------------------------------------------------- waits that run out


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 3], [300, 400]])  # (the second by pairs of blocks, for bf16)
def test_wait_expiry_reports_timeout_and_leaves_gpu_usable(kind, new):
    """Every wait of the attention kernel is bounded.  The self-test runs the ordinary kernels with
    a limit of 20 ms and no query tile ever delivered (a barrier nothing arrives at): the roles give
    up, wait for their copies in flight, free the tensor memory and return, with the status word set.
    An ordinary call right after, which takes all of an SM's tensor memory, is right.  With few
    keys the loads end before the ring is full, with many they wait for it."""
    for past in (0, 3000):
        p = Problem(new=new, past=[past] * len(new), page=64, kind=kind, seed=490)
        p.put_plain()
        out, lse = torch.empty_like(p.q), torch.empty(p.rows, 16, device="cuda")
        a = gdr._attn_paged_args(p.q, *p.pages, p.cache_len, out, p.k_scale, p.v_scale, p.gate, lse, None)
        n = gdr.attn_paged_workspace_size(p.q, *p.pages, p.cache_len, out, **p.scales)
        ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        start = time.perf_counter()
        st = _abi.lib().gdr_attn_paged_selftest_wait_expiry(a, ws.data_ptr(), n, 20_000_000,
                                                            torch.cuda.current_stream().cuda_stream)
        assert st == 0, gdr.status_string(st)
        torch.cuda.synchronize()
        # At most: the ring's slots, Q twice and the last product, 20 ms each.
        assert time.perf_counter() - start < 2.0
        assert status_of(ws) == 6  # GDR_ERR_TIMEOUT
        out, lse, ws = p.attend(workspace=ws)
        assert status_of(ws) == 0
        p.check_attend(out, lse)
