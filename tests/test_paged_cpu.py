"""The paged cache's entry points without a GPU: refusals of the C ABI (made-up addresses, so
only where no CUDA device is present), the binding's own refusals, and every call carried
to the launch."""
import ctypes

import pytest
import torch

import linear_attention_recurrence_10_b200 as gdr
from linear_attention_recurrence_10_b200 import _abi, build

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5
FAKE = 0x7f0000000000

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="host-only validation with made-up addresses")


@pytest.fixture(scope="module")
def lib():
    build.build(quiet=True)
    return _abi.lib()


def _addresses(a, names):
    for name in names:
        setattr(a, name, FAKE + (_addresses.at << 32))
        _addresses.at += 1


_addresses.at = 0


def _pages(**kw):
    c = _abi.KvPages(n_seq=3, H_kv=2, d=256, page_size=64, n_pages=20, table_width=4,
                     kv_dtype=_abi.GDR_E4M3)
    _addresses(c, ["k", "v", "k_scale", "v_scale", "page_table", "cu_seqlens"])
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _split(kw):
    fields = {f for f, _ in _abi.KvPages._fields_}
    return {k: v for k, v in kw.items() if k in fields}, {k: v for k, v in kw.items() if k not in fields}


def _append(**kw):
    pages, kw = _split(kw)
    a = _abi.KvAppendArgs(pages=_pages(**pages), n_tok=7, H_q=16, rot_dim=64, rope_theta=1e7)
    _addresses(a, ["q", "k", "v", "q_out", "cache_len", "status"])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _gather(**kw):
    pages, kw = _split(kw)
    a = _abi.KvGatherArgs(pages=_pages(**pages), n_tok=7, out_dtype=_abi.GDR_BF16)
    _addresses(a, ["k_out", "v_out", "first", "status"])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _attn(**kw):
    pages, kw = _split(kw)
    a = _abi.AttnPagedArgs(pages=_pages(**pages), n_tok=7, H_q=16, out_dtype=_abi.GDR_BF16,
                           scale=1.0 / 16)
    _addresses(a, ["q", "gate", "cache_len", "out", "lse"])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


PAGES = [
    ("negative_n_seq", dict(n_seq=-1), INVALID),
    ("no_heads", dict(H_kv=0), INVALID),
    ("d128", dict(d=128), UNSUPPORTED),
    ("page_8", dict(page_size=8), UNSUPPORTED),
    ("page_48", dict(page_size=48), UNSUPPORTED),
    ("page_2048", dict(page_size=2048), UNSUPPORTED),
    ("page_0", dict(page_size=0), INVALID),
    ("negative_pages", dict(n_pages=-1), INVALID),
    ("rows_past_int32", dict(n_pages=1 << 25), UNSUPPORTED),
    ("too_many_heads", dict(H_kv=1 << 16, H_q=1 << 16), UNSUPPORTED),
    ("rows_at_int32", dict(H_kv=1, H_q=1, page_size=1024, n_pages=1 << 21), UNSUPPORTED),
    ("fp32_cache", dict(kv_dtype=0), INVALID),
    ("unknown_cache_type", dict(kv_dtype=3), INVALID),
    ("scales_with_bf16", dict(kv_dtype=1), INVALID),
    ("codes_without_scale", dict(v_scale=None), INVALID),
    ("null_pages", dict(k=None), INVALID),
    ("no_pages", dict(n_pages=0), INVALID),
    ("no_table", dict(table_width=0), INVALID),
    ("null_table", dict(page_table=None), INVALID),
    ("null_cu", dict(cu_seqlens=None), INVALID),
    ("table_stride_small", dict(table_stride=3), INVALID),
    ("table_stride_negative", dict(table_stride=-4), INVALID),
    ("negative_width", dict(table_width=-1), INVALID),
    ("reserved_pages", {}, INVALID),
    ("misaligned_pages", dict(v=FAKE + 8), MISALIGNED),
    ("misaligned_scale", dict(k_scale=FAKE + 8), MISALIGNED),
    ("misaligned_table", dict(page_table=FAKE + 1), MISALIGNED),
    ("misaligned_cu", dict(cu_seqlens=FAKE + 2), MISALIGNED),
    ("negative_tokens", dict(n_tok=-1), INVALID),
    ("too_many_tokens", dict(n_tok=(1 << 31) - 128), UNSUPPORTED),
]


@host_only
@pytest.mark.parametrize("name,kw,want", PAGES, ids=[c[0] for c in PAGES])
def test_pages_validation(lib, name, kw, want):
    """Each of the three calls checks the cache in the same way."""
    ws, n = FAKE + (1 << 44), ctypes.c_size_t(1 << 30)
    calls = [(lib.gdr_kv_append, _append(**kw), ()), (lib.gdr_attn_paged, _attn(**kw), (ws, n))]
    if "H_q" not in kw:
        calls.append((lib.gdr_kv_gather, _gather(**kw), ()))
    for f, a, more in calls:
        if name == "reserved_pages":
            a.pages.reserved = 1
        assert f(ctypes.byref(a), *more, None) == want, f


APPEND = [
    ("null_k", dict(k=None), INVALID),
    ("null_cache_len", dict(cache_len=None), INVALID),
    ("q_without_q_out", dict(q_out=None), INVALID),
    ("q_out_without_q", dict(q=None), INVALID),
    ("heads_without_q", dict(q=None, q_out=None), INVALID),
    ("q_without_heads", dict(H_q=0), INVALID),
    ("odd_rot_dim", dict(rot_dim=33), INVALID),
    ("rot_dim_past_d", dict(rot_dim=258), INVALID),
    ("theta_zero", dict(rope_theta=0.0), INVALID),
    ("theta_nan", dict(rope_theta=float("nan")), INVALID),
    ("theta_inf", dict(rope_theta=float("inf")), INVALID),
    ("reserved", dict(reserved=1), INVALID),
    ("stride_small", dict(k_stride=256), INVALID),
    ("stride_not_16_bytes", dict(v_stride=516), MISALIGNED),
    ("misaligned_q", dict(q=FAKE + 8), MISALIGNED),
    ("misaligned_status", dict(status=FAKE + 2), MISALIGNED),
    ("in_place_other_stride", dict(q=FAKE, q_out=FAKE, q_stride=8192, q_out_stride=4096), INVALID),
]


@host_only
@pytest.mark.parametrize("name,kw,want", APPEND, ids=[c[0] for c in APPEND])
def test_append_validation(lib, name, kw, want):
    assert lib.gdr_kv_append(ctypes.byref(_append(**kw)), None) == want


GATHER = [
    ("no_output", dict(k_out=None, v_out=None), INVALID),
    ("codes_as_output", dict(out_dtype=2), INVALID),
    ("reserved", dict(reserved=1), INVALID),
    ("stride_small", dict(k_out_stride=256), INVALID),
    ("misaligned_out", dict(v_out=FAKE + 4), MISALIGNED),
    ("misaligned_first", dict(first=FAKE + 1), MISALIGNED),
]


@host_only
@pytest.mark.parametrize("name,kw,want", GATHER, ids=[c[0] for c in GATHER])
def test_gather_validation(lib, name, kw, want):
    assert lib.gdr_kv_gather(ctypes.byref(_gather(**kw)), None) == want


ATTN = [
    ("null_q", dict(q=None), INVALID),
    ("null_out", dict(out=None), INVALID),
    ("null_cache_len", dict(cache_len=None), INVALID),
    ("heads_not_multiple", dict(H_q=15), INVALID),
    ("no_heads", dict(H_q=0), INVALID),
    ("too_many_query_heads", dict(H_q=258), UNSUPPORTED),
    ("codes_as_output", dict(out_dtype=2), INVALID),
    ("scale_zero", dict(scale=0.0), INVALID),
    ("scale_negative", dict(scale=-0.1), INVALID),
    ("scale_nan", dict(scale=float("nan")), INVALID),
    ("scale_inf", dict(scale=float("inf")), INVALID),
    ("reserved", dict(reserved=2), INVALID),
    ("stride_small", dict(gate_stride=256), INVALID),
    ("lse_stride_small", dict(lse_stride=15), INVALID),
    ("misaligned_out", dict(out=FAKE + 8), MISALIGNED),
    ("misaligned_lse", dict(lse=FAKE + 2), MISALIGNED),
]


@host_only
@pytest.mark.parametrize("name,kw,want", ATTN, ids=[c[0] for c in ATTN])
def test_attn_paged_validation(lib, name, kw, want):
    a = _attn(**kw)
    assert lib.gdr_attn_paged(ctypes.byref(a), FAKE + (1 << 44), ctypes.c_size_t(1 << 30), None) == want


@host_only
def test_workspace_and_empty_calls(lib):
    n = ctypes.c_size_t(0)
    a = _attn()
    assert lib.gdr_attn_paged_workspace_size(ctypes.byref(a), ctypes.byref(n)) == OK and n.value > 0
    ws = FAKE + (1 << 44)
    assert lib.gdr_attn_paged(ctypes.byref(a), ws, n.value - 1, None) == WORKSPACE
    assert lib.gdr_attn_paged(ctypes.byref(a), None, n.value, None) == WORKSPACE
    assert lib.gdr_attn_paged(ctypes.byref(a), ws + 8, n.value, None) == MISALIGNED
    assert lib.gdr_attn_paged_workspace_size(ctypes.byref(a), None) == INVALID
    assert lib.gdr_attn_paged_workspace_size(ctypes.byref(_attn(d=64)), ctypes.byref(n)) == UNSUPPORTED
    for empty in (dict(n_tok=0), dict(n_seq=0)):
        b = _attn(**empty)
        assert lib.gdr_attn_paged_workspace_size(ctypes.byref(b), ctypes.byref(n)) == OK and n.value == 0
        assert lib.gdr_attn_paged(ctypes.byref(b), None, 0, None) == OK
        assert lib.gdr_kv_append(ctypes.byref(_append(**empty)), None) == OK
        assert lib.gdr_kv_gather(ctypes.byref(_gather(**empty)), None) == OK
    assert lib.gdr_attn_paged(None, ws, 0, None) == INVALID
    assert lib.gdr_kv_append(None, None) == INVALID and lib.gdr_kv_gather(None, None) == INVALID


def _tensors(kind="e4m3"):
    pages = lambda: torch.zeros(6, 2, 16, 256).to(torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16)
    scale = (lambda: torch.ones(6, 2, 16)) if kind == "e4m3" else (lambda: None)
    return dict(k_pages=pages(), v_pages=pages(), page_table=torch.arange(6, dtype=torch.int32).view(2, 3),
                cu_seqlens=torch.tensor([0, 2, 5], dtype=torch.int32), k_scale=scale(), v_scale=scale())


def _rows(H, n=5, dtype=torch.bfloat16):
    return torch.zeros(n, H, 256, dtype=dtype)


def _calls(c, **kw):
    """The three calls on the tensors of `c`, with `kw` in the place of theirs."""
    cache_len = kw.pop("cache_len", torch.tensor([3, 40], dtype=torch.int32))
    q, k, v, gate, out = (kw.pop(n, _rows(H)) for n, H in (("q", 16), ("k", 2), ("v", 2), ("gate", 16),
                                                           ("out", 16)))
    lse = kw.pop("lse", torch.zeros(5, 16))
    head = [c[n] for n in ("k_pages", "v_pages", "page_table", "cu_seqlens")]
    scales = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    assert not kw
    return {
        "gdr_kv_append": lambda: gdr.kv_append(k, v, *head, cache_len, **scales, q=q, q_out=out, stream=0),
        "gdr_kv_gather": lambda: gdr.kv_gather(*head, k, v, **scales, stream=0),
        "gdr_attn_paged": lambda: gdr.attn_paged(q, *head, cache_len, out, **scales, gate=gate, lse=lse,
                                                 stream=0),
    }


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_every_call_reaches_the_launch_without_a_device(kind):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present: the GPU tests cover these calls")
    for name, call in _calls(_tensors(kind)).items():
        with pytest.raises(gdr.GdrError) as e:
            call()
        assert e.value.status == CUDA and name in str(e.value), (name, str(e.value))


@host_only
@pytest.mark.parametrize("change", [
    dict(k_pages=torch.zeros(6, 2, 16, 256, dtype=torch.float16)),
    dict(v_pages=torch.zeros(6, 2, 16, 256, dtype=torch.bfloat16)),
    dict(v_pages=torch.zeros(5, 2, 16, 256).to(torch.float8_e4m3fn)),
    dict(k_pages=torch.zeros(6, 16, 2, 256).to(torch.float8_e4m3fn).transpose(1, 2)),
    dict(k_scale=None),
    dict(v_scale=torch.ones(6, 2, 17)),
    dict(k_scale=torch.ones(6, 2, 16, dtype=torch.float64)),
    dict(page_table=torch.zeros(2, 3, dtype=torch.int64)),
    dict(page_table=torch.zeros(1, 3, dtype=torch.int32).expand(2, 3)),
    dict(page_table=torch.zeros(3, 2, dtype=torch.int32).t()),
    dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)),
    dict(cu_seqlens=torch.zeros(3, dtype=torch.int64)),
])
def test_binding_refuses_the_cache(change):
    for call in _calls(dict(_tensors(), **change)).values():
        with pytest.raises((TypeError, ValueError)):
            call()


@host_only
@pytest.mark.parametrize("change", [
    dict(q=_rows(16, dtype=torch.float16)),
    dict(q=_rows(16, n=4)),
    dict(q=_rows(16, n=1).expand(5, -1, -1)),
    dict(cache_len=torch.zeros(3, dtype=torch.int32)),
    dict(cache_len=torch.zeros(2)),
    dict(cache_len=torch.zeros(1, dtype=torch.int32).expand(2)),
])
def test_binding_refuses_the_rows(change):
    calls = _calls(_tensors(), **change)
    for name in ("gdr_kv_append", "gdr_attn_paged"):
        with pytest.raises((TypeError, ValueError)):
            calls[name]()


@host_only
@pytest.mark.parametrize("name,change", [
    ("gdr_kv_append", dict(k=_rows(4))),
    ("gdr_kv_append", dict(v=_rows(2, dtype=torch.float32))),
    ("gdr_kv_append", dict(out=_rows(16, dtype=torch.float32))),
    ("gdr_kv_gather", dict(k=_rows(2, dtype=torch.float32))),
    ("gdr_kv_gather", dict(v=_rows(2, n=4))),
    ("gdr_kv_gather", dict(k=_rows(2, dtype=torch.float16), v=_rows(2, dtype=torch.float16))),
    ("gdr_attn_paged", dict(gate=_rows(8))),
    ("gdr_attn_paged", dict(gate=_rows(16, n=1).expand(5, -1, -1))),
    ("gdr_attn_paged", dict(out=_rows(16, dtype=torch.float16))),
    ("gdr_attn_paged", dict(out=_rows(16, n=6))),
    ("gdr_attn_paged", dict(lse=torch.zeros(5, 16, dtype=torch.float64))),
    ("gdr_attn_paged", dict(lse=torch.zeros(16, 5).t())),
])
def test_binding_refuses_an_argument(name, change):
    with pytest.raises((TypeError, ValueError)):
        _calls(_tensors(), **change)[name]()


def test_packed_structs_are_the_declared_ones():
    """The binding packs the argument structs by struct formats: the bytes of each are those of
    the ctypes mirror of include/gdr.h, field for field."""
    for fmt, cls in ((gdr._PACK_APPEND, _abi.KvAppendArgs), (gdr._PACK_GATHER, _abi.KvGatherArgs),
                     (gdr._PACK_ATTN, _abi.AttnPagedArgs)):
        flat = []

        def fields(c, base=0):
            for name, t in c._fields_:
                if issubclass(t, ctypes.Structure):
                    fields(t, base + getattr(c, name).offset)
                else:
                    flat.append((base + getattr(c, name).offset, t))

        fields(cls)
        assert fmt.size == ctypes.sizeof(cls)
        values = [i + 1 for i in range(len(flat))]
        data = fmt.pack(*values)
        for (offset, t), want in zip(flat, values):
            assert t.from_buffer_copy(data, offset).value == want, (cls.__name__, offset)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_host_tensors_are_refused_where_there_is_a_gpu(monkeypatch, kind):
    """Tensors in host memory never reach the library on a machine with a GPU (here: a stand-in
    for the library, and a torch that says it has one)."""
    class Library:
        def __getattr__(self, name):
            def call(*args):
                assert name.endswith("workspace_size"), f"{name} was called with host addresses"
                return OK
            return call

    monkeypatch.setattr(_abi, "lib", Library)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    for name, call in _calls(_tensors(kind)).items():
        with pytest.raises(ValueError, match=f"{name}.*CUDA device"):
            call()


@host_only
def test_selftest_wait_expiry_refusals(lib):
    """The wait-expiry self-test has gdr_attn_paged's checks, a range for its limit, and no empty call."""
    f, ws, n = lib.gdr_attn_paged_selftest_wait_expiry, FAKE + (1 << 44), ctypes.c_size_t(1 << 30)
    a = _attn()
    for wait_ns in (0, 99_999, 2_000_000_001):
        assert f(ctypes.byref(a), ws, n, wait_ns, None) == INVALID
    assert f(None, ws, n, 20_000_000, None) == INVALID
    assert f(ctypes.byref(a), ws, 16, 20_000_000, None) == WORKSPACE
    for kw, want in ((dict(n_tok=0), INVALID), (dict(n_seq=0), INVALID), (dict(d=128), UNSUPPORTED),
                     (dict(q=None), INVALID), (dict(out=FAKE + 8), MISALIGNED)):
        assert f(ctypes.byref(_attn(**kw)), ws, n, 20_000_000, None) == want, kw
