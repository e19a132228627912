"""The paged key/value cache and its attention (gdr_kv_append, gdr_kv_gather, gdr_attn_paged)
against their formulas in 64 bits; bounds in paged_testutil."""
import pytest
import torch

import linear_attention_recurrence_10_b200 as gdr
from paged_testutil import D, NAN, U8, Problem, rope64, status_of

pytestmark = pytest.mark.gpu

HEADS = [(16, 2), (2, 2), (8, 8), (6, 2), (32, 2)]
RAGGED = dict(new=[3, 0, 1, 40, 17, 1], past=[0, 5, 130, 7, 255, 16])


# ------------------------------------------------------------------ append


def check_append(p, q_out, before, rot_dim=64, theta=1e7):
    """q_out and every cache row against the definition; rows of no new token as they were."""
    pos = torch.cat([torch.arange(a, a + n) for n, a in zip(p.new, p.past)]).cuda()
    n = p.n_tok
    want, slack = rope64(p.q[:n], pos, rot_dim, theta)
    assert ((q_out[:n].double() - want).abs() <= U8 * want.abs() * (1 + U8) + slack).all()
    assert torch.isnan(q_out[n:]).all()
    who = torch.cat([torch.full((m,), s) for s, m in enumerate(p.new)]).cuda()
    at = (p.table.long()[who, pos // p.page], pos % p.page)
    written = torch.zeros(p.n_pages, p.page, dtype=torch.bool, device="cuda")
    written[at] = True
    for name in ("k", "v"):
        pages, scales = getattr(p, name + "_pages"), getattr(p, name + "_scale")
        if name == "k":
            want, slack = rope64(p.k[:n], pos, rot_dim, theta)
        else:
            want, slack = p.v[:n].double(), torch.zeros(1, device="cuda", dtype=torch.float64)
        got = pages[at[0], :, at[1]]
        if scales is None:
            assert ((got.double() - want).abs() <= (U8 * want.abs() * (1 + U8) + slack if name == "k" else 0)).all()
        else:
            sc = scales[at[0], :, at[1]].double()
            top = want.abs().amax(-1)
            ref = (top / 448).clamp_min(2.0 ** -40)
            assert ((sc - ref).abs() <= ref * 2.0 ** -21).all()
            half = torch.maximum(want.abs() * 2.0 ** -4, 2.0 ** -10 * sc[..., None])
            assert ((got.double() * sc[..., None] - want).abs() <= half * (1 + 2.0 ** -18) + slack).all()
        same = ~written[:, None].expand(pages.shape[:3])
        old = before[name + "_pages"]
        assert torch.equal(pages.view(torch.uint8)[same], old.view(torch.uint8)[same])
        if scales is not None:
            assert torch.equal(scales.view(torch.int32)[same], before[name + "_scale"].view(torch.int32)[same])


def snapshot(p):
    return {n: getattr(p, n).clone() for n in ("k_pages", "v_pages", "k_scale", "v_scale")
            if getattr(p, n) is not None}


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page", list(zip(HEADS, [16, 32, 64, 128, 256])))
def test_append(heads, page, kind):
    p = Problem(**RAGGED, H_q=heads[0], H_kv=heads[1], page=page, kind=kind, seed=page, tail=3)
    before = snapshot(p)
    check_append(p, p.append(), before)


@pytest.mark.parametrize("rot_dim", [0, 2, 30, 64, 192, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_rotary_dims(rot_dim, kind):
    """Pairs inside a lane's 8 values, across lanes, and at every alignment between."""
    p = Problem(new=[5, 2], past=[301, 11], kind=kind, seed=rot_dim)
    before = snapshot(p)
    check_append(p, p.append(rot_dim=rot_dim, rope_theta=10000.0), before, rot_dim, 10000.0)


def test_append_far_position():
    """A position of ten million: the angle keeps its precision (one page is mapped)."""
    p = Problem(new=[4], past=[0], page=16, seed=5)
    far = 10_000_000
    table = torch.full((1, far // 16 + 1), -1, dtype=torch.int32, device="cuda")
    table[0, far // 16] = p.table[0, 0]
    q_out = torch.empty_like(p.q)
    gdr.kv_append(p.k, p.v, p.k_pages, p.v_pages, table, p.cu,
                  torch.tensor([far], dtype=torch.int32, device="cuda"), q=p.q, q_out=q_out)
    pos = far + torch.arange(4, device="cuda")
    want, slack = rope64(p.q, pos, 64, 1e7)
    assert ((q_out.double() - want).abs() <= U8 * want.abs() * (1 + U8) + slack).all()
    want, slack = rope64(p.k, pos, 64, 1e7)
    got = p.k_pages[p.table[0, 0].long(), :, :4].transpose(0, 1).double()
    assert ((got - want).abs() <= U8 * want.abs() * (1 + U8) + slack).all()


@pytest.mark.parametrize("rot_dim", [64, 30])
def test_append_in_place_and_strided(rot_dim):
    """q_out == q, and q, k, v as views of one projection's output."""
    p = Problem(new=[9, 1], past=[3, 20], kind="e4m3", seed=3)
    want = p.append(rot_dim=rot_dim)
    codes, scale = p.k_pages.clone(), p.v_scale.clone()
    qkv = torch.cat([p.q, p.k, p.v], 1)
    p.q, p.k, p.v = qkv[:, :16], qkv[:, 16:18], qkv[:, 18:]
    got = p.append(q_out=p.q, rot_dim=rot_dim)
    assert torch.equal(got, want) and torch.equal(qkv[:, :16], want)
    assert torch.equal(p.k_pages.view(torch.uint8), codes.view(torch.uint8))
    assert torch.equal(p.v_scale.view(torch.int32), scale.view(torch.int32))


def test_append_without_queries():
    p = Problem(**RAGGED, kind="e4m3", seed=8)
    before = snapshot(p)
    q_out = p.append()
    after = snapshot(p)
    for n, t in before.items():
        getattr(p, n).copy_(t)
    assert gdr.kv_append(p.k, p.v, p.k_pages, p.v_pages, p.table, p.cu, p.cache_len, **p.scales) is None
    for n, t in after.items():
        assert torch.equal(getattr(p, n).view(torch.uint8), t.view(torch.uint8)), n
    assert q_out is not None


def test_append_zero_and_non_finite_rows():
    """A row of zeros has codes 0 and the smallest scale; a row with an infinity or a NaN
    reads back as not finite, and only that row."""
    p = Problem(new=[4], past=[0], kind="e4m3", seed=9)
    p.v[0] = 0
    p.v[1, 0, 7] = float("inf")
    p.v[2, 1, 100] = NAN
    p.append()
    page = p.table[0, 0].long()
    assert (p.v_pages[page, :, 0].float() == 0).all() and (p.v_scale[page, :, 0] == 2.0 ** -40).all()
    out = torch.empty(4, 2, D, device="cuda")
    gdr.kv_gather(*p.pages, None, out, **p.scales)
    bad = ~torch.isfinite(out).all(-1)
    assert bad.cpu().tolist() == [[False, False], [True, False], [False, True], [False, False]]


def test_append_bad_pages_are_reported_and_skipped():
    p = Problem(new=[20, 20, 2, 3], past=[0, 0, 0, 0], page=16, seed=10)
    p.table[0, 1] = p.n_pages       # past the pool
    p.table[1, 0] = -7
    p.cache_len[2] = 31             # past the table's two pages after one token
    p.cache_len[3] = -1
    before = snapshot(p)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p.append(status=status)
    assert int(status) == 1
    good = p.table[0, 0].long()
    want, slack = rope64(p.k[:16], torch.arange(16, device="cuda"), 64, 1e7)
    got = p.k_pages[good].transpose(0, 1).double()
    assert ((got - want).abs() <= U8 * want.abs() * (1 + U8) + slack).all()
    assert torch.equal(p.v_pages[p.table[1, 1].long(), :, :4].transpose(0, 1), p.v[36:40])
    last = p.table[2, 1].long()
    if last >= 0:
        assert torch.equal(p.v_pages[last, :, 15], p.v[40])
    pages = {int(good), int(p.table[1, 1]), int(last)}
    rest = [i for i in range(p.n_pages) if i not in pages]
    for n in ("k_pages", "v_pages"):
        assert torch.equal(getattr(p, n)[rest].view(torch.int16), before[n][rest].view(torch.int16))
    status.zero_()
    ok = Problem(new=[2], past=[3], seed=1)
    ok.append(status=status)
    assert int(status) == 0


# ------------------------------------------------------------------ gather


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,heads", [(16, (16, 2)), (128, (8, 8)), (1024, (3, 1))])
def test_gather(page, heads, dtype, kind):
    p = Problem(new=[0] * 5, past=[70, 1, 0, 33, 300], H_q=heads[0], H_kv=heads[1], page=page, kind=kind,
                seed=20)
    cu = torch.tensor([0, 70, 71, 71, 104, 404], dtype=torch.int32, device="cuda")
    out = [torch.full((404 + 2, heads[1], D), NAN, dtype=dtype, device="cuda") for _ in "kv"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdr.kv_gather(p.k_pages, p.v_pages, p.table, cu, *out, **p.scales, status=status)
    assert int(status) == 0
    for name, got in zip("kv", out):
        want = torch.cat([p.cached(name, s)[0] for s in range(5)])
        # one product in fp32, then the output's rounding: exact but for it
        assert torch.equal(got[:404], want.float().to(dtype))
        assert torch.isnan(got[404:]).all()


def test_gather_from_the_middle_and_one_side():
    p = Problem(new=[0, 0], past=[100, 60], kind="e4m3", seed=21)
    cu = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    first = torch.tensor([85, 30], dtype=torch.int32, device="cuda")
    wide = torch.full((40, 2, 2, D), NAN, device="cuda")
    gdr.kv_gather(p.k_pages, p.v_pages, p.table, cu, None, wide[:, 1], **p.scales, first=first)
    v = [p.cached("v", s)[0].float() for s in range(2)]
    assert torch.equal(wide[:, 1], torch.cat([v[0][85:95], v[1][30:60]]))
    assert torch.isnan(wide[:, 0]).all()


def test_gather_bad_pages_are_reported():
    p = Problem(new=[0, 0], past=[40, 20], seed=22)
    p.table[0, 1] = 1 << 30
    cu = torch.tensor([0, 40, 60], dtype=torch.int32, device="cuda")
    k, v = (torch.full((60, 2, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdr.kv_gather(*p.pages[:3], cu, k, v, status=status)
    assert int(status) == 1
    assert torch.equal(k[40:].double(), p.cached("k", 1)[0]) and torch.isfinite(k[:16]).all()
    status.zero_()
    first = torch.tensor([0, 13 + (1 << 30)], dtype=torch.int32, device="cuda")
    gdr.kv_gather(*p.pages[:3], cu, k, v, status=status, first=first)
    assert int(status) == 1


# --------------------------------------------------------------- attention


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page", list(zip(HEADS + [(128, 1), (10, 1)], [16, 32, 64, 128, 256, 16, 1024])))
def test_attend_ragged(heads, page, kind):
    p = Problem(**RAGGED, H_q=heads[0], H_kv=heads[1], page=page, kind=kind, seed=100 + page, tail=2)
    p.put_plain()
    out, lse, ws = p.attend()
    assert status_of(ws) == 0
    p.check_attend(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 127, 128, 129, 191, 256, 257, 1000])
def test_attend_one_token(length, kind):
    """A chunk of one, at lengths around the tiles of 64 and 128 tokens and the pages."""
    p = Problem(new=[1, 1], past=[length - 1, 0], page=32, kind=kind, seed=length)
    p.put_plain()
    out, lse, ws = p.attend()
    assert status_of(ws) == 0
    p.check_attend(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,past", [(15, 0), (16, 0), (17, 0), (128, 0), (129, 1), (300, 0), (100, 500),
                                      (257, 127)])
def test_attend_chunks(new, past, kind):
    p = Problem(new=[new], past=[past], page=64, kind=kind, seed=new + past)
    p.put_plain()
    out, lse, ws = p.attend()
    assert status_of(ws) == 0
    p.check_attend(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page", list(zip(HEADS + [(128, 1), (10, 1)], [32, 64, 16, 128, 1024, 256, 16])))
def test_attend_long_chunks(heads, page, kind):
    """New tokens that fill 256 rows and more per key head (the tiles are then shared by two
    thread blocks): lengths that leave the second one few rows, none, and few keys."""
    rep = heads[0] // heads[1]
    big = -(-700 // rep)
    p = Problem(new=[big, 3 + 128 // rep, big + 5, 1], past=[0, 77, 130, 40], H_q=heads[0], H_kv=heads[1],
                page=page, kind=kind, seed=300 + page, tail=3)
    assert p.rows * rep >= 256 * p.n_seq  # the rule for it
    p.put_plain()
    for dtype in (torch.bfloat16, torch.float32):
        out, lse, ws = p.attend(out_dtype=dtype)
        assert status_of(ws) == 0
        p.check_attend(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("fault", ["page", "length"])
def test_attend_long_chunks_bad_pages(fault, kind):
    p = Problem(new=[200, 200, 200], past=[10, 20, 30], page=32, kind=kind, seed=310)
    p.put_plain()
    good = p.table.clone(), p.cache_len.clone()
    if fault == "page":
        p.table[1, 3] = -1
    else:
        p.cache_len[1] = 1 << 30
    out, lse, ws = p.attend()
    assert status_of(ws) == 1
    p.table, p.cache_len = good
    out[200:400] = 0
    p.check_attend(out, lse, only=(0, 2))


def test_attend_allocates_its_workspace_for_the_stream():
    """No workspace given, on a stream of its own: what is allocated is not handed out again
    while the call may still run."""
    p = Problem(new=[300], past=[3000], page=64, seed=320)
    p.put_plain()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        out = torch.empty_like(p.q)
        gdr.attn_paged(p.q, *p.pages, p.cache_len, out, gate=p.gate, stream=s)
        torch.empty(39 << 20, dtype=torch.uint8, device="cuda").fill_(0xFF)
        outs.append(out)
    torch.cuda.synchronize()
    for out in outs:
        p.check_attend(out, None)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attend_options(kind):
    """fp32 output, no gate, no lse, another scale; strided q, gate, out, lse and table."""
    p = Problem(**RAGGED, kind=kind, seed=130)
    p.put_plain()
    for gate in (False, True):
        out, _, ws = p.attend(gate=gate, out_dtype=torch.float32, lse=False, scale=0.2)
        assert status_of(ws) == 0
        p.check_attend(out, None, gate=gate, scale=0.2)
    ref, ref_lse, _ = p.attend()
    wide = torch.full((p.rows, 50, D), NAN, dtype=torch.bfloat16, device="cuda")
    wide[:, :16], wide[:, 16:32] = p.q, p.gate
    table = torch.full((p.n_seq, p.width + 5), -1, dtype=torch.int32, device="cuda")
    table[:, :p.width] = p.table
    lse = torch.full((p.rows, 20), NAN, device="cuda")
    gdr.attn_paged(wide[:, :16], p.k_pages, p.v_pages, table[:, :p.width], p.cu, p.cache_len,
                   wide[:, 32:48], gate=wide[:, 16:32], lse=lse[:, :16], **p.scales)
    assert torch.equal(wide[:, 32:48], ref) and torch.equal(lse[:, :16], ref_lse)
    assert torch.isnan(wide[:, 48:]).all() and torch.isnan(lse[:, 16:]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attend_peaked_and_flat_scores(kind):
    """Scores that grow along the sequence (the running maximum moves in every tile), one key
    that takes all the weight, and keys that are all alike."""
    p = Problem(new=[20, 20, 20], past=[500, 500, 500], page=64, kind=kind, seed=140)
    if kind == "bf16":
        for s, f in ((0, None), (1, 60.0), (2, 0.0)):
            t = torch.arange(500, device="cuda")
            at = (p.table[s].long()[t // 64], t % 64)
            k = p.k_pages[at[0], :, at[1]].float()
            if s == 0:
                k = p.q[:1, :2].float() * t[:, None, None] * 0.02
            elif s == 1:
                k[321] = p.q[20, :2].float() * 4
            else:
                k[:] = 1.0
            p.k_pages[at[0], :, at[1]] = k.bfloat16()
    else:
        p.k_scale[p.table[0].long().clamp_min(0)] *= 8
        p.k_scale[p.table[2].long().clamp_min(0)] *= 2.0 ** -12
    p.put_plain()
    out, lse, ws = p.attend()
    assert status_of(ws) == 0
    p.check_attend(out, lse)


def test_attend_scales_of_many_sizes():
    """Value rows whose scales differ by factors of thousands, rows of zeros among them."""
    p = Problem(new=[30, 1], past=[400, 300], page=32, kind="e4m3", seed=150, v_scale_spread=3.0)
    p.v[3] = 0
    t = torch.arange(50, 90, device="cuda")
    at = (p.table[0].long()[t // 32], t % 32)
    p.v_pages.view(torch.uint8)[at[0], :, at[1]] = 0
    p.v_scale[at[0], :, at[1]] = 2.0 ** -40
    p.put_plain()
    out, lse, ws = p.attend()
    assert status_of(ws) == 0
    p.check_attend(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attend_large_batches(kind):
    """More work items than SMs, and sequences cut into many parts: a long one among short."""
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 70, (40,), generator=g).tolist() + [600, 1]
    past = torch.randint(0, 500, (40,), generator=g).tolist() + [0, 9000]
    p = Problem(new=new, past=past, page=128, kind=kind, seed=160)
    p.put_plain()
    out, lse, ws = p.attend()
    assert status_of(ws) == 0
    p.check_attend(out, lse)
    again, lse2, _ = p.attend()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_attend_many_sequences():
    """More sequences than threads in a block, most of them empty."""
    new = [(1 if s % 7 == 0 else 0) for s in range(1500)]
    past = [(s * 13) % 97 for s in range(1500)]
    p = Problem(new=new, past=past, page=16, seed=170)
    p.put_plain()
    out, lse, ws = p.attend()
    assert status_of(ws) == 0
    p.check_attend(out, lse)


def test_attend_nothing():
    p = Problem(new=[0, 0], past=[5, 0], seed=180, tail=4)
    out, lse, ws = p.attend()
    assert torch.isnan(out).all() and torch.isnan(lse).all() and status_of(ws) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attend_bad_pages_and_lengths_are_reported(kind):
    """A wrong page, a length past the table and a negative one leave the other sequences
    right, and are reported."""
    for fault in range(3):
        p = Problem(new=[2, 20, 2], past=[150, 100, 30], page=16, kind=kind, seed=190)
        p.put_plain()
        good = p.table.clone(), p.cache_len.clone()
        if fault == 0:
            p.table[1, 2] = p.n_pages + 5
        elif fault == 1:
            p.cache_len[1] = 16 * p.width + 1000
        else:
            p.cache_len[1] = -1000
        out, lse, ws = p.attend()
        assert status_of(ws) == 1
        p.table, p.cache_len = good
        p.check_attend(torch.cat([out[:2], torch.zeros_like(out[2:22]), out[22:]]), lse, only=(0, 2))


def test_attend_offsets_past_32_bits():
    """Cache rows whose element offsets pass 2^31 (and byte offsets 2^32)."""
    rows = (1 << 31) // D + 4096
    n_pages = rows // (2 * 64)
    small = Problem(new=[5], past=[300], page=64, seed=200)
    small.put_plain()
    k = torch.empty(n_pages, 2, 64, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = small.table.clone()
    n = small.width
    for i in range(n):
        k[n_pages - n + i] = small.k_pages[small.table[0, i].long()]
        v[n_pages - n + i] = small.v_pages[small.table[0, i].long()]
        table[0, i] = n_pages - n + i
    small.k_pages, small.v_pages, small.table = k, v, table
    out, lse, ws = small.attend()
    assert status_of(ws) == 0
    small.check_attend(out, lse)
    back = torch.empty(305, 2, D, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 305], dtype=torch.int32, device="cuda")
    gdr.kv_gather(k, v, table, cu, back, None)
    assert torch.equal(back.double(), small.cached("k", 0)[0])
    small.append()
    want, slack = rope64(small.k, 300 + torch.arange(5, device="cuda"), 64, 1e7)
    assert ((small.cached("k", 0)[0][300:] - want).abs() <= U8 * want.abs() * (1 + U8) + slack).all()


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prompt_in_chunks_then_tokens(kind):
    """A prompt appended and attended in chunks, then token by token, gives what one call over
    the whole gives; what was written reads back."""
    n = 150
    whole = Problem(new=[n], past=[0], page=32, kind=kind, seed=210)
    q = whole.append()
    ref, ref_lse, _ = whole.attend(q=q)
    whole.check_attend(ref, ref_lse, q=q)
    parts = Problem(new=[n], past=[0], page=32, kind=kind, seed=210)
    at, out, lse = 0, torch.empty_like(ref), torch.empty_like(ref_lse)
    for step in (70, 1, 33, 40) + (1,) * 6:
        r = slice(at, at + step)
        cu = torch.tensor([0, step], dtype=torch.int32, device="cuda")
        past = torch.tensor([at], dtype=torch.int32, device="cuda")
        qr = gdr.kv_append(parts.k[r], parts.v[r], parts.k_pages, parts.v_pages, parts.table, cu, past,
                           q=parts.q[r], q_out=torch.empty_like(parts.q[r]), **parts.scales)
        assert torch.equal(qr, q[r])
        gdr.attn_paged(qr, parts.k_pages, parts.v_pages, parts.table, cu, past, out[r],
                       gate=parts.gate[r], lse=lse[r], **parts.scales)
        at += step
    whole.check_attend(out, lse, q=q, what="in parts")
    assert torch.equal(parts.k_pages.view(torch.uint8), whole.k_pages.view(torch.uint8))
    k = torch.empty(n, 2, D, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    gdr.kv_gather(parts.k_pages, parts.v_pages, parts.table, cu, k, None, **parts.scales)
    want, _ = rope64(whole.k, torch.arange(n, device="cuda"), 64, 1e7)
    half = 2.0 ** -4 if kind == "e4m3" else U8
    top = want.abs().amax(-1, keepdim=True)
    assert ((k.double() - want).abs() <= half * want.abs() * 1.01 + top * 2.0 ** -18).all()


def test_same_as_the_contiguous_decode_step():
    """One token over a bf16 paged cache and gdr_attn_decode_step over the same tokens in a
    contiguous one: both within their bounds of the formula, so of each other."""
    B, L = 5, [0, 37, 255, 128, 1]
    p = Problem(new=[1] * B, past=L, page=16, seed=220)
    kc = torch.zeros(B, 2, 300, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    for s in range(B):
        if L[s]:
            kc[s, :, :L[s]] = p.cached("k", s, L[s])[0].bfloat16().transpose(0, 1)
            vc[s, :, :L[s]] = p.cached("v", s, L[s])[0].bfloat16().transpose(0, 1)
    step = torch.empty(B, 16, D, device="cuda")
    gdr.attn_decode_step(p.q, p.gate, p.k, p.v, kc, vc, p.cache_len, step, kv_bound=299)
    q = p.append()
    out, lse, _ = p.attend(q=q, out_dtype=torch.float32)
    p.check_attend(out, lse, q=q)
    assert (out - step).norm() <= 2 * 1.25 * U8 / 3 ** 0.5 * step.norm()
    for s in range(B):
        assert torch.equal(p.cached("k", s)[0], kc[s, :, :L[s] + 1].transpose(0, 1).double())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_step_replayed_with_other_lengths(kind):
    """Append and attention captured once; replayed as the sequences grow and as a batch slot
    changes from one token to several."""
    cap = Problem(new=[1, 1, 6], past=[60, 126, 10], page=32, kind=kind, seed=230, width=8, spare=12)
    rows = cap.rows
    q_out = torch.empty_like(cap.q)
    out = torch.empty_like(cap.q)
    lse = torch.empty(rows, 16, device="cuda")
    ws = torch.empty(gdr.attn_paged_workspace_size(cap.q, *cap.pages, cap.cache_len, out, **cap.scales),
                     dtype=torch.uint8, device="cuda")

    def step():
        gdr.kv_append(cap.k, cap.v, cap.k_pages, cap.v_pages, cap.table, cap.cu, cap.cache_len, q=cap.q,
                      q_out=q_out, **cap.scales)
        gdr.attn_paged(q_out, *cap.pages, cap.cache_len, out, gate=cap.gate, lse=lse, workspace=ws,
                       **cap.scales)

    pools = ("k_pages", "v_pages", "k_scale", "v_scale")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new, past in (([1, 1, 6], [60, 126, 10]), ([3, 4, 1], [0, 128, 200]), ([0, 8, 0], [5, 1, 9])):
        p = Problem(new=new, past=past, page=32, kind=kind, seed=231, width=8, tail=rows - sum(new))
        keep = p.n_pages
        assert keep <= cap.n_pages  # the captured pool holds every case's
        for n in pools:
            if getattr(cap, n) is not None:
                getattr(cap, n)[:keep].copy_(getattr(p, n))
        for n in ("q", "gate", "k", "v", "table", "cu", "cache_len"):
            getattr(cap, n).copy_(getattr(p, n))
        out.fill_(NAN)
        lse.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for n in pools:
            if getattr(cap, n) is not None:
                setattr(p, n, getattr(cap, n)[:keep].clone())
        assert status_of(ws) == 0
        p.check_attend(out, lse, q=q_out)
    del graph


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_chunk_replayed_beside_eager_calls(kind):
    """A captured chunk (of paired blocks) replayed with other lengths, between eager calls on
    another stream with a workspace of their own."""
    p = Problem(new=[300, 200], past=[100, 900], page=64, kind=kind, seed=260, spare=8)  # holds every case
    p.put_plain()
    other = Problem(new=[77], past=[400], page=64, kind=kind, seed=261)
    other.put_plain()
    out, lse = torch.empty_like(p.q), torch.empty(p.rows, 16, device="cuda")
    args = (p.q, *p.pages, p.cache_len, out)
    kw = dict(**p.scales, gate=p.gate, lse=lse)
    ws = torch.empty(gdr.attn_paged_workspace_size(*args, **kw), dtype=torch.uint8, device="cuda")
    gdr.attn_paged(*args, **kw, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.attn_paged(*args, **kw, workspace=ws)
    side = torch.cuda.Stream()
    for new, past in (([300, 200], [100, 900]), ([450, 50], [0, 1050]), ([0, 500], [5, 600])):
        p.new, p.past, p.len = new, past, [a + b for a, b in zip(new, past)]
        q = Problem(new=new, past=past, page=64, kind=kind, seed=262, width=p.width)
        q.put_plain()
        assert q.n_pages <= p.n_pages
        for n in ("k_pages", "v_pages", "k_scale", "v_scale"):
            if getattr(p, n) is not None:
                getattr(p, n)[:q.n_pages].copy_(getattr(q, n))
        for n in ("q", "gate", "table", "cu", "cache_len"):
            getattr(p, n).copy_(getattr(q, n))
        out.fill_(NAN)
        lse.fill_(NAN)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            first = other.attend()
        graph.replay()
        with torch.cuda.stream(side):
            second = other.attend()
        torch.cuda.synchronize()
        assert status_of(ws) == 0
        p.check_attend(out, lse)
        assert torch.equal(first[0], second[0])
        other.check_attend(*first[:2])
    del graph


def test_two_streams_at_once():
    """Two calls in flight, each on its own stream with its own workspace."""
    ps = [Problem(new=[200, 1], past=[100 * i, 2000], page=64, kind=k, seed=240 + i)
          for i, k in enumerate(["bf16", "e4m3"])]
    for p in ps:
        p.put_plain()
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                got.append((p, p.attend()))
    torch.cuda.synchronize()
    for p, (out, lse, ws) in got:
        assert status_of(ws) == 0
        p.check_attend(out, lse)


@pytest.mark.slow
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_serving_batch_repeats_bit_for_bit(kind):
    """64 sequences of 4096 tokens and a chunk of a long prompt, ten calls from an evicted L2:
    every call gives the first one's bits; the first is checked against the formula."""
    p = Problem(new=[1] * 63 + [700], past=[4095] * 63 + [3000], page=64, kind=kind, seed=250)
    p.put_plain()
    evict = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(10):
        evict.fill_(i)
        out, lse, ws = p.attend()
        assert status_of(ws) == 0
        if first is None:
            first = out, lse
            p.check_attend(out, lse)
        else:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
