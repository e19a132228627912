"""The paged key/value cache of the gated full-attention layer: its three operators, in plain form
and as calls of the library.

    append  the new tokens of packed sequences are rotated (q and k) and written into their pages,
            as bf16 or as e4m3 codes with one scale per token and head
    gather  cached tokens are read back into packed rows
    attend  the new tokens attend over their sequence's pages, causally, and are gated

The heads, head size, rotary dims and batch sizes are those of the decode step's benchmark and
tests (16 query over 2 key/value heads of 256 dims, 64 sequences of 4096 cached tokens, 4 prompts of
4096 tokens) and the other head layouts its tests use.
"""
import random

import torch

own = False

D = 256
ROT = 64
THETA = 1e7
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -40


def listed():
    base = dict(H_q=16, H_kv=2, page=64, kind="e4m3", single=0.0, even=True, shape=1)
    return [
        # one sequence generates a token: nothing but latency
        dict(base, name="append one token", op="append", n_seq=1, new=1, past=1000),
        # a serving batch generates a token each, into a bf16 cache
        dict(base, name="append 64 tokens bf16", op="append", n_seq=64, new=1, past=4095, kind="bf16"),
        # four prompts are written as codes
        dict(base, name="append 4 prompts", op="append", n_seq=4, new=4096, past=0),
        # a few short ragged sequences leave a bf16 cache with small pages
        dict(base, name="gather short bf16", op="gather", n_seq=5, new=37, past=263, page=16,
             kind="bf16", even=False),
        # a serving batch's whole cache is read back
        dict(base, name="gather 64x4096", op="gather", n_seq=64, new=0, past=4096),
        # one sequence, one token, a short ragged cache with small pages
        dict(base, name="attend one token", op="attend", n_seq=1, new=1, past=1000, page=16,
             kind="bf16"),
        # the serving batch's decode step on a bf16 cache, and on codes
        dict(base, name="attend decode bf16", op="attend", n_seq=64, new=1, past=4095, kind="bf16"),
        dict(base, name="attend decode", op="attend", n_seq=64, new=1, past=4095),
        # a few drafted tokens per sequence are checked at once, on ragged caches
        dict(base, name="attend drafts", op="attend", n_seq=16, new=5, past=2000, page=16, even=False),
        # one chunk of a long prompt
        dict(base, name="attend chunk bf16", op="attend", n_seq=1, new=2048, past=6144, kind="bf16"),
        # whole prompts
        dict(base, name="attend 4 prompts bf16", op="attend", n_seq=4, new=4096, past=0, kind="bf16"),
        # prompts' chunks and generated tokens in one ragged batch
        dict(base, name="attend mixed", op="attend", n_seq=24, new=1000, past=3001, page=32,
             even=False, single=0.75),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(lo * (hi / lo) ** rng.random() + rng.random()))

    H_q, H_kv = rng.choice([(16, 2), (16, 2), (8, 8), (32, 2), (2, 2), (6, 2)])
    c = dict(op=rng.choice(["append", "gather", "attend", "attend", "attend"]), H_q=H_q, H_kv=H_kv,
             page=rng.choice([16, 32, 64, 128, 256]), kind=rng.choice(["bf16", "e4m3"]),
             n_seq=log(1, 64), new=log(1, 4096), past=log(1, 8192), single=rng.choice([0.0, 0.0, 0.7]),
             even=rng.random() < 0.3, shape=rng.randrange(1 << 30))
    if c["op"] == "attend":  # the plain form holds a score for every (row, cached token) pair
        while c["n_seq"] * c["new"] * H_q * (c["past"] + c["new"]) > 4 * 4096 * 16 * 4096:
            c["new"] = max(1, c["new"] // 2)
            c["n_seq"] = max(1, c["n_seq"] * 2 // 3)
    while c["n_seq"] * c["new"] * max(H_q, 2 * H_kv) > 4 * 4096 * 16:
        c["new"] = max(1, c["new"] // 2)
    while c["n_seq"] * (c["past"] + c["new"]) * H_kv > 64 * 4096 * 2:
        c["past"] = c["past"] // 2
    return c


def lengths(case):
    """(new, past) tokens of each sequence, from the case alone."""
    r = random.Random(case["shape"])
    new, past = [], []
    for s in range(case["n_seq"]):
        one = s > 0 and r.random() < case["single"]
        n, p = r.randint(min(1, case["new"]), case["new"]), r.randint(0, case["past"])
        if case["even"] or s == 0:
            n, p = case["new"], case["past"]
        new.append(1 if one else n)
        past.append(p)
    return new, past


def quantise(x):
    """e4m3 codes of rows of D values, and each row's scale."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, past = lengths(case)
    n_seq, n_tok, ps, H_q, H_kv = len(new), sum(new), case["page"], case["H_q"], case["H_kv"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    need = [-(-(n + p) // ps) for n, p in zip(new, past)]
    width, n_pages = max(need), sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.zeros(n_seq, width, dtype=torch.int32)
    at = 0
    order = order.cpu()
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    cache = []
    for _ in range(2):
        pages = normal(n_pages, H_kv, ps, D)
        if case["kind"] == "e4m3":
            cache.append(quantise(pages.float()))
        else:
            cache.append((pages, None))
    (k_pages, k_scale), (v_pages, v_scale) = cache
    cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0)
    st = dict(op=case["op"], k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale,
              table=table.cuda(), cu=cu.to(torch.int32).cuda(),
              past=torch.tensor(past, dtype=torch.int32).cuda())
    if case["op"] == "gather":
        total = torch.tensor([0] + [n + p for n, p in zip(new, past)], dtype=torch.int64).cumsum(0)
        st.update(cu=total.to(torch.int32).cuda(), n_rows=int(total[-1]))
        return st
    st.update(q=normal(n_tok, H_q, D))
    if case["op"] == "append":
        st.update(k=normal(n_tok, H_kv, D), v=normal(n_tok, H_kv, D))
    else:
        st.update(gate=normal(n_tok, H_q, D), max_new=max(new))
    return st


# ---------------------------------------------------------------- plain forms


def sequence_of(cu, n):
    """The sequence of each of n packed rows, and the row's index in it."""
    rows = torch.arange(n, device=cu.device, dtype=cu.dtype)
    s = torch.bucketize(rows, cu[1:], right=True)
    return s, rows - cu[s]


def rotated(x, pos):
    """x [n, H, D] with its first ROT dims turned by pos * theta^(-2i/ROT); angles in 64 bits."""
    half = ROT // 2
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * THETA ** (-2 * i / ROT)
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    a, b = x[..., :half], x[..., half:ROT]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., ROT:]], -1)


def plain_append(st):
    ps = st["k_pages"].shape[2]
    s, i = sequence_of(st["cu"], st["q"].shape[0])
    pos = (st["past"][s] + i).long()
    page, row = st["table"][s, pos // ps].long(), pos % ps
    for x, pages, scales in ((rotated(st["k"], pos), st["k_pages"], st["k_scale"]),
                             (st["v"].float(), st["v_pages"], st["v_scale"])):
        if scales is None:
            pages[page, :, row] = x.to(torch.bfloat16)
        else:
            codes, scale = quantise(x)
            pages.view(torch.uint8)[page, :, row] = codes.view(torch.uint8)
            scales[page, :, row] = scale
    return rotated(st["q"], pos).to(torch.bfloat16)


def plain_rows(pages, scales, page, row):
    """Cached rows (page, row) in 32 bits: [..., H_kv, D]."""
    x = pages[page, :, row].float()
    return x if scales is None else x * scales[page, :, row][..., None]


def plain_gather(st):
    ps = st["k_pages"].shape[2]
    s, t = sequence_of(st["cu"], st["n_rows"])
    t = t.long()
    page, row = st["table"][s, t // ps].long(), t % ps
    return [plain_rows(st[k + "_pages"], st[k + "_scale"], page, row).to(torch.bfloat16) for k in "kv"]


def plain_attend(st):
    n_seq, ps, dev = st["table"].shape[0], st["k_pages"].shape[2], st["q"].device
    n, H_q, _ = st["q"].shape
    H_kv = st["k_pages"].shape[1]
    s, i = sequence_of(st["cu"], n)
    q = torch.zeros(n_seq, st["max_new"], H_q, D, device=dev)
    q[s, i] = st["q"].float()
    q = q.view(n_seq, -1, H_kv, H_q // H_kv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    t = torch.arange(st["table"].shape[1] * ps, device=dev)
    page, row = st["table"].long()[:, t // ps], (t % ps).expand(n_seq, -1)
    k = plain_rows(st["k_pages"], st["k_scale"], page, row).permute(0, 2, 3, 1)
    pos = st["past"][:, None] + torch.arange(st["max_new"], device=dev)
    length = st["past"] + (st["cu"][1:] - st["cu"][:-1])
    keep = (t <= pos[..., None]) & (t < length[:, None, None])
    score = torch.matmul(q, k) * D ** -0.5
    del k
    score = score.view(n_seq, H_kv, -1, st["max_new"], t.numel())
    score.masked_fill_(~keep[:, None, None], -torch.inf)
    top = score.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    score.div_(total)
    v = plain_rows(st["v_pages"], st["v_scale"], page, row).permute(0, 2, 1, 3)
    v = torch.where((t < length[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(score.flatten(2, 3), v).view(n_seq, H_kv, -1, st["max_new"], D)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s, i]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[s, i]
    return (o / (1 + torch.exp(-st["gate"].float()))).to(torch.bfloat16), lse


# -------------------------------------------------------- the library's calls


def own_append(st):
    import linear_attention_recurrence_10_b200 as gdr
    q_out = torch.empty_like(st["q"])
    gdr.kv_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["cu"], st["past"],
                  k_scale=st["k_scale"], v_scale=st["v_scale"], q=st["q"], q_out=q_out, rot_dim=ROT,
                  rope_theta=THETA)
    return q_out


def own_gather(st):
    import linear_attention_recurrence_10_b200 as gdr
    out = [torch.empty(st["n_rows"], st["k_pages"].shape[1], D, dtype=torch.bfloat16, device="cuda")
           for _ in "kv"]
    gdr.kv_gather(st["k_pages"], st["v_pages"], st["table"], st["cu"], *out,
                  k_scale=st["k_scale"], v_scale=st["v_scale"])
    return out


def own_attend(st):
    import linear_attention_recurrence_10_b200 as gdr
    out = torch.empty_like(st["q"])
    lse = torch.empty(st["q"].shape[:2], device="cuda")
    args = (st["q"], st["k_pages"], st["v_pages"], st["table"], st["cu"], st["past"], out)
    kw = dict(k_scale=st["k_scale"], v_scale=st["v_scale"], gate=st["gate"], lse=lse)
    if "workspace" not in st:  # kept, as a serving loop keeps it
        st["workspace"] = torch.empty(gdr.attn_paged_workspace_size(*args, **kw), dtype=torch.uint8,
                                      device="cuda")
    gdr.attn_paged(*args, **kw, workspace=st["workspace"])
    return out, lse


def run(state):
    op = state["op"]
    if op == "append":
        q_out = own_append(state) if own else plain_append(state)
        return dict(q=q_out, **{n: state[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")})
    if op == "gather":
        k, v = own_gather(state) if own else plain_gather(state)
        return dict(k=k, v=v)
    out, lse = own_attend(state) if own else plain_attend(state)
    return dict(out=out, lse=lse)


def work(case):
    new, past = lengths(case)
    n_tok, total = sum(new), sum(new) + sum(past)
    H_q, H_kv = case["H_q"], case["H_kv"]
    row = 2 * H_kv * (2 * D if case["kind"] == "bf16" else D + 4)  # a token's K and V in the cache
    if case["op"] == "append":
        turned = 6 * ROT * (H_q + H_kv) // 2  # a turn of a pair is 6 operations
        return dict(bytes=n_tok * (2 * H_q * 2 * D + 2 * H_kv * 2 * D + row), flops=n_tok * turned)
    if case["op"] == "gather":
        return dict(bytes=total * (row + 2 * H_kv * 2 * D), flops=0 if case["kind"] == "bf16" else
                    total * 2 * H_kv * D)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    return dict(bytes=n_tok * H_q * (3 * 2 * D + 4) + total * row, flops=4 * D * H_q * pairs)


# ------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    new, past = lengths(case)
    ps, H_kv = case["page"], case["H_kv"]
    kept = {}
    for n in "kv":
        pages = st[n + "_pages"].double()
        kept[n] = pages if st[n + "_scale"] is None else pages * st[n + "_scale"].double()[..., None]

    def cached(n, s, length):
        t = torch.arange(length, device="cuda")
        return kept[n][st["table"][s].long()[t // ps], :, t % ps]

    if case["op"] == "gather":
        return dict(k=torch.cat([cached("k", s, a + b) for s, (a, b) in enumerate(zip(new, past))]),
                    v=torch.cat([cached("v", s, a + b) for s, (a, b) in enumerate(zip(new, past))]))

    where = torch.cat([torch.arange(p, p + n, device="cuda") for n, p in zip(new, past)])
    who = torch.cat([torch.full((n,), s, device="cuda") for s, n in enumerate(new)])
    if case["op"] == "append":
        freq = torch.exp2(torch.arange(ROT // 2, device="cuda", dtype=torch.float64) / (ROT // 2)
                          * -torch.log2(torch.tensor(THETA, dtype=torch.float64)))
        turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                           where.double()[:, None] * freq)

        def rope(x):
            x = x.double()
            z = torch.complex(x[..., :ROT // 2], x[..., ROT // 2:ROT]) * turn[:, None]
            return torch.cat([z.real, z.imag, x[..., ROT:]], -1)

        out = dict(q=rope(st["q"]), k_scale=None, v_scale=None)
        at = (st["table"].long()[who, where // ps], where % ps)
        for n, x in (("k", rope(st["k"])), ("v", st["v"].double())):
            pages = st[n + "_pages"].double()
            if case["kind"] == "e4m3":
                scale = torch.clamp(x.abs().max(-1).values / E4M3_MAX, min=SCALE_MIN)
                x = x / scale[..., None]
                step = torch.exp2(torch.clamp(torch.frexp(x).exponent - 1, min=-6).double() - 3)
                x = torch.clamp(torch.round(x / step) * step, -E4M3_MAX, E4M3_MAX)
                scales = st[n + "_scale"].double()
                scales[at[0], :, at[1]] = scale
                out[n + "_scale"] = scales
            pages[at[0], :, at[1]] = x
            out[n + "_pages"] = pages
        return out

    q, gate = st["q"].double(), st["gate"].double()
    out, lse, at = torch.empty_like(q), torch.empty(q.shape[:2], dtype=q.dtype, device="cuda"), 0
    for s, (n, p) in enumerate(zip(new, past)):
        k, v = cached("k", s, n + p), cached("v", s, n + p)
        for r in range(at, at + n, 512):
            rows = slice(r, min(r + 512, at + n))
            qs = q[rows].unflatten(1, (H_kv, -1))
            score = torch.einsum("igrd,tgd->igrt", qs, k) / D ** 0.5
            last = p + torch.arange(r - at, rows.stop - at, device="cuda")
            score[(torch.arange(n + p, device="cuda") > last[:, None])[:, None, None].expand_as(score)] = -torch.inf
            lse[rows] = torch.logsumexp(score, -1).flatten(1)
            o = torch.einsum("igrt,tgd->igrd", torch.softmax(score, -1), v).flatten(1, 2)
            out[rows] = o * torch.sigmoid(gate[rows])
        at += n
    return dict(out=out, lse=lse)
