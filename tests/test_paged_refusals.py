"""The serving calls refuse what they cannot serve on the host, with the reason
(no GPU needed: validation comes first)."""
import ctypes

import pytest

from quantized_attention_smooth_gb300 import sage

FAKE = 0x100000      # never dereferenced: validation fails first
L = sage.lib
N = sage.workspace_bytes_paged()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=0, k_mean=0, v_scale=0, num_pages=4, page_size=16, Hkv=2,
             D=64, page_stride=2048, token_stride=128, head_stride=64, kind=sage.BF16)
    a.update(kw)
    return sage._CacheC(**a)


def batch(**kw):
    a = dict(cu_q=FAKE, kv_lens=FAKE, block_table=FAKE, nseq=2, total_q=5, table_stride=3,
             table_width=3, max_q=4, max_kv=40)
    a.update(kw)
    return sage._BatchC(**a)


def ref(struct):
    return None if struct is None else ctypes.byref(struct)


def strides(s):
    return None if s is None else (ctypes.c_int64 * 2)(*s)


def attn(c, b, q=FAKE, out=FAKE, lse=0, dtype=sage.BF16, Hq=4, qs=None, window=0, sinks=0,
         scale=0.0, ws=FAKE, n=N):
    return L.sage_attn_paged(ref(c), ref(b), q, out, lse, dtype, Hq, strides(qs), window, sinks, scale, ws,
                             n, None)


def append(c, b, k=FAKE, v=FAKE, q=0, qo=0, dtype=sage.BF16, Hq=4, ks=None, f=0, R=64, ws=FAKE,
           n=N):
    return L.sage_kv_append(ref(c), ref(b), k, v, q, qo, dtype, Hq, strides(ks), None, None, None, f, R, 0,
                            1.0, ws, n, None)


INV, UNS, WSP = sage.ERR_INVALID_ARG, sage.ERR_UNSUPPORTED, sage.ERR_WORKSPACE
COMMON = [
    (dict(D=60), {}, UNS, "head_dim"), (dict(D=136), {}, UNS, "head_dim"),
    (dict(D=0), {}, UNS, "head_dim"), (dict(page_size=24), {}, UNS, "page_size"),
    (dict(page_size=0), {}, UNS, "page_size"), (dict(page_size=1 << 17), {}, UNS, "page_size"),
    (dict(kind=5), {}, INV, "kind"), (dict(Hkv=0), {}, INV, "Hkv"),
    (dict(num_pages=0), {}, INV, "num_pages"), (dict(k=0), {}, INV, "16-byte"),
    (dict(v=FAKE + 8), {}, INV, "16-byte"), (dict(token_stride=0), {}, UNS, "strides"),
    (dict(page_stride=2049), {}, UNS, "strides"), (dict(head_stride=-64), {}, UNS, "strides"),
    (dict(token_stride=1 << 39), {}, UNS, "strides"),
    (dict(num_pages=2 ** 31 - 1, page_stride=(1 << 39) - 8), {}, UNS, "extent"),
    (dict(kind=sage.Q8), {}, INV, "k_scale"),
    ({}, dict(nseq=-1), INV, "negative"), ({}, dict(max_kv=-1), INV, "negative"),
    ({}, dict(max_kv=49), INV, "max_kv"), ({}, dict(nseq=(1 << 20) + 1), UNS, "sequences"),
    ({}, dict(cu_q=0), INV, "cu_q"), ({}, dict(kv_lens=FAKE + 2), INV, "kv_lens"),
    ({}, dict(block_table=0), INV, "block_table"), ({}, dict(table_stride=2), INV, "table_stride"),
]


@pytest.mark.parametrize("ckw,bkw,status,needle", COMMON)
def test_cache_and_batch(ckw, bkw, status, needle):
    for call in (attn, append):
        assert call(cache(**ckw), batch(**bkw)) == status
        assert needle in sage.last_error()


def test_null_structs_and_workspace():
    for call in (attn, append):
        assert call(None, batch()) == INV and "null" in sage.last_error()
        assert call(cache(), None) == INV
        assert call(cache(), batch(), ws=0) == WSP and "256-byte" in sage.last_error()
        assert call(cache(), batch(), ws=FAKE + 16) == WSP
        assert call(cache(), batch(), n=N - 1) == WSP and "needs" in sage.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=3), INV, "dtype"), (dict(dtype=sage.F16), INV, "kind"),
    (dict(Hq=3), INV, "multiple"), (dict(Hq=0), INV, "multiple"),
    (dict(window=-1), INV, "window"), (dict(sinks=-1), INV, "sinks"),
    (dict(scale=float("nan")), INV, "finite"), (dict(scale=float("inf")), INV, "finite"),
    (dict(q=0), INV, "q must"), (dict(out=FAKE + 8), INV, "out"), (dict(lse=FAKE + 2), INV, "lse"),
    (dict(qs=(0, 64)), UNS, "positive"), (dict(qs=(256, -64)), UNS, "positive"),
])
def test_attention(kw, status, needle):
    assert attn(cache(), batch(), **kw) == status
    assert needle in sage.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=3), INV, "dtype"), (dict(dtype=sage.F16), INV, "kind"),
    (dict(q=FAKE), INV, "inv_freq"), (dict(q=FAKE, f=FAKE), INV, "q_out"),
    (dict(q=FAKE, qo=FAKE, f=FAKE, Hq=0), INV, "Hq"), (dict(f=FAKE, R=3), INV, "even"),
    (dict(f=FAKE, R=66), INV, "even"), (dict(f=FAKE + 4), INV, "inv_freq"),
    (dict(k=0), INV, "k, v"), (dict(v=FAKE + 1), INV, "k, v"), (dict(ks=(0, 64)), UNS, "positive"),
])
def test_append(kw, status, needle):
    assert append(cache(), batch(), **kw) == status
    assert needle in sage.last_error()


def rope(**kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, dtype=sage.F16, T=3, Hq=2, Hkv=2, D=64, qs=None,
             ks=None, qos=None, kos=None, pos=FAKE, bits=64, f=FAKE, R=64)
    a.update(kw)
    return L.sage_rope(a["q"], a["k"], a["qo"], a["ko"], a["dtype"], a["T"], a["Hq"], a["Hkv"],
                       a["D"], strides(a["qs"]), strides(a["ks"]), strides(a["qos"]),
                       strides(a["kos"]), a["pos"], a["bits"], a["f"], a["R"], 0, 1.0, 0, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), INV, "dtype"), (dict(D=0), UNS, "head_dim"), (dict(D=129), UNS, "head_dim"),
    (dict(R=65), INV, "even"), (dict(R=66), INV, "even"), (dict(R=0), INV, "even"),
    (dict(k=0), INV, "k is null"), (dict(Hq=0), INV, "Hq"), (dict(T=-1), INV, "T="),
    (dict(q=0), INV, "2-byte"), (dict(ko=0), INV, "2-byte"), (dict(q=FAKE + 1), INV, "2-byte"),
    (dict(bits=16), INV, "pos_bits"), (dict(pos=0), INV, "pos"), (dict(pos=FAKE + 4), INV, "pos"),
    (dict(f=0), INV, "inv_freq"), (dict(qs=(0, 64)), UNS, "positive"),
    (dict(kos=(1 << 39, 64)), UNS, "2^39"), (dict(qs=(256, 64), qos=(128, 64)), INV, "in place"),
])
def test_rope(kw, status, needle):
    assert rope(**kw) == status
    assert needle in sage.last_error()


def test_empty_calls_do_nothing():
    assert rope(T=0) == sage.OK
    assert attn(cache(), batch(total_q=0)) == sage.OK
    assert attn(cache(), batch(nseq=0)) == sage.OK
    assert append(cache(), batch(total_q=0)) == sage.OK
    assert append(cache(), batch(nseq=0, total_q=5)) == sage.OK


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    f = torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        sage.rope(x, None, torch.arange(3), f)
    p = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sage.PagedCache(p, p)
    with pytest.raises(TypeError, match="int8"):
        sage.PagedCache(p, p.half())
    with pytest.raises(ValueError, match="one shape"):
        sage.PagedCache(p, p[:2])
    with pytest.raises(ValueError, match="CUDA"):
        sage.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                        torch.zeros(1, 3, dtype=torch.int32), 1, 40)
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, scaling="x"),
                dict(rotary_dim=8, factor=0.5), dict(rotary_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            sage.rope_freqs(device="cpu", **bad)
