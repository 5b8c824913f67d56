"""What the 4-bit cache, the page pool and rotations of several axes refuse on the host (no
GPU needed: validation comes first)."""
import ctypes

import pytest

from quantized_attention_smooth_gb300 import sage

FAKE = 0x100000      # never dereferenced: validation fails first
L = sage.lib
N = sage.workspace_bytes_paged()
INV, UNS, WSP = sage.ERR_INVALID_ARG, sage.ERR_UNSUPPORTED, sage.ERR_WORKSPACE


def struct(cls, base, kw):
    return cls(**{**base, **kw})


def cache(**kw):
    return struct(sage._CacheC, dict(k=FAKE, v=FAKE, k_scale=0, k_mean=FAKE, v_scale=FAKE, num_pages=4,
                                     page_size=16, Hkv=2, D=72, page_stride=1536, token_stride=96,
                                     head_stride=48, kind=sage.Q4, k_groups=FAKE, v_groups=FAKE), kw)


def batch(**kw):
    return struct(sage._BatchC, dict(cu_q=FAKE, kv_lens=FAKE, block_table=FAKE, nseq=2, total_q=5,
                                     table_stride=3, table_width=3, max_q=4, max_kv=40), kw)


def ref(s):
    return None if s is None else ctypes.byref(s)


def strides(s):
    return None if s is None else (ctypes.c_int64 * 2)(*s)


def attn(c, b, dtype=sage.BF16, ws=FAKE, n=N):
    return L.sage_attn_paged(ref(c), ref(b), FAKE, FAKE, 0, dtype, 4, None, 0, 0, 0.0, ws, n, None)


def append(c, b, dtype=sage.BF16, ws=FAKE, n=N):
    return L.sage_kv_append(ref(c), ref(b), FAKE, FAKE, 0, 0, dtype, 4, None, None, None, None, 0, 0, 0,
                            1.0, ws, n, None)


def gather(c, b, k=FAKE, v=FAKE, dtype=sage.BF16, ks=None, ws=FAKE, n=N):
    return L.sage_kv_gather(ref(c), ref(b), k, v, dtype, strides(ks), None, ws, n, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(k_groups=0), INV, "k_groups"), (dict(v_groups=0), INV, "v_groups"),
    (dict(k_mean=0), INV, "k_mean"), (dict(v_scale=FAKE + 8), INV, "16-byte"),
    (dict(k_groups=FAKE + 2), INV, "16-byte"), (dict(token_stride=32), UNS, "strides"),
    (dict(token_stride=104), UNS, "multiples of 16"), (dict(head_stride=40), UNS, "strides"),
    (dict(page_stride=1544), UNS, "strides"), (dict(D=60), UNS, "head_dim"),
    (dict(page_size=24), UNS, "page_size"), (dict(kind=4), INV, "kind"),
])
def test_a_4_bit_cache(kw, status, needle):
    for call in (attn, append, gather):
        assert call(cache(**kw), batch()) == status
        assert needle in sage.last_error()


def test_gather():
    assert gather(cache(), batch(), dtype=3) == INV and "dtype" in sage.last_error()
    half = cache(kind=sage.F16, D=64, token_stride=128, head_stride=64, page_stride=2048)
    assert gather(half, batch()) == INV and "kind" in sage.last_error()
    assert gather(cache(), batch(), k=0) == INV and "k and v" in sage.last_error()
    assert gather(cache(), batch(), v=FAKE + 1) == INV
    assert gather(cache(), batch(), ks=(0, 72)) == UNS and "positive" in sage.last_error()
    assert gather(cache(), batch(), ws=FAKE + 16) == WSP and "256-byte" in sage.last_error()
    assert gather(cache(), batch(), n=N - 1) == WSP
    assert gather(None, batch()) == INV and gather(cache(), None) == INV
    assert gather(cache(), batch(total_q=0)) == sage.OK


# ------------------------------------------------------------------- axes
def rope(pos=FAKE, bits=64, naxes=3, step=3, axis_of=FAKE, f=FAKE, R=64, T=3):
    return L.sage_rope_axes(FAKE, FAKE, FAKE, FAKE, sage.F16, T, 2, 2, 64, None, None, None, None, pos,
                            bits, naxes, step, axis_of, f, R, 0, 1.0, 0, None)


def append_axes(c=None, b=None, pos=FAKE, bits=64, naxes=3, step=5, f=FAKE, R=64):
    return L.sage_kv_append_axes(ref(c or cache()), ref(b or batch()), FAKE, FAKE, 0, 0, sage.BF16, 4,
                                 None, None, None, None, pos, bits, naxes, step, FAKE, f, R, 0, 1.0, FAKE,
                                 N, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(naxes=0), UNS, "naxes"), (dict(naxes=9), UNS, "naxes"), (dict(step=2), INV, "axis_stride"),
    (dict(step=1 << 39), INV, "axis_stride"), (dict(bits=16), INV, "pos_bits"),
    (dict(pos=0), INV, "pos must"), (dict(pos=FAKE + 4), INV, "pos must"),
    (dict(f=0), INV, "inv_freq"), (dict(R=74), INV, "even"),
])
def test_axes(kw, status, needle):
    for call in (rope, append_axes):
        assert call(**kw) == status
        assert needle in sage.last_error()


def test_axes_of_nothing():
    assert rope(T=0, step=0) == sage.OK
    assert append_axes(b=batch(total_q=0)) == sage.OK
    assert L.sage_kv_append_axes(ref(cache()), None, FAKE, FAKE, 0, 0, sage.BF16, 4, None, None, None, None,
                                 FAKE, 64, 1, 5, FAKE, FAKE, 64, 0, 1.0, FAKE, N, None) == INV


# ------------------------------------------------------------------- pool
def pool(**kw):
    return struct(sage._PoolC, dict(free_pages=FAKE, left=FAKE, table=FAKE, lens=FAKE, marks=FAKE,
                                    num_pages=8, page_size=16, max_requests=4, table_stride=3,
                                    table_width=3), kw)


def plan(**kw):
    return struct(sage._PlanC, dict(cu_q=FAKE, kv_lens=FAKE, block_table=FAKE, positions=FAKE, slots=FAKE,
                                    denied=FAKE, n=2, rows=9, table_stride=3, table_width=3, max_q=5,
                                    max_kv=48), kw)


def step(p, q, requests=FAKE, new=FAKE, ws=FAKE, n=N):
    return L.sage_paged_step(ref(p), ref(q), requests, new, ws, n, None)


def trim(p, q=None, requests=FAKE, keep=0, ws=FAKE, n=N, count=2):
    return L.sage_paged_trim(ref(p), requests, keep, count, ws, n, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(page_size=0), UNS, "page_size"), (dict(page_size=20), UNS, "page_size"),
    (dict(num_pages=0), INV, "num_pages"), (dict(num_pages=1 << 31), INV, "num_pages"),
    (dict(max_requests=0), INV, "max_requests"), (dict(table_width=0), INV, "table_width"),
    (dict(table_stride=2), INV, "table_stride"), (dict(free_pages=0), INV, "free_pages"),
    (dict(left=FAKE + 2), INV, "left"), (dict(marks=0), INV, "marks"), (dict(lens=0), INV, "lens"),
])
def test_pools(kw, status, needle):
    for call in (step, trim):
        assert call(pool(**kw), plan()) == status
        assert needle in sage.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(n=-1), UNS, "sequences"), (dict(n=65537), UNS, "sequences"), (dict(rows=-1), INV, "plan sizes"),
    (dict(rows=1 << 31), INV, "plan sizes"), (dict(max_q=-1), INV, "plan sizes"),
    (dict(table_width=-1), INV, "plan sizes"), (dict(table_stride=2), INV, "table_stride"),
    (dict(cu_q=0), INV, "cu_q"), (dict(kv_lens=FAKE + 2), INV, "kv_lens"), (dict(denied=0), INV, "denied"),
    (dict(block_table=0), INV, "block_table"), (dict(positions=FAKE + 4), INV, "8-byte"),
    (dict(slots=FAKE + 4), INV, "8-byte"),
])
def test_plans(kw, status, needle):
    assert step(pool(), plan(**kw)) == status
    assert needle in sage.last_error()


def test_pool_calls():
    assert step(None, plan()) == INV and step(pool(), None) == INV and trim(None) == INV
    assert "null" in sage.last_error()
    assert step(pool(), plan(), requests=0) == INV and "requests" in sage.last_error()
    assert step(pool(), plan(), new=FAKE + 1) == INV and "new_lens" in sage.last_error()
    assert trim(pool(), requests=FAKE + 2) == INV and "requests" in sage.last_error()
    assert trim(pool(), keep=FAKE + 2) == INV and "keep_lens" in sage.last_error()
    assert trim(pool(), count=65537) == UNS and "sequences" in sage.last_error()
    for call in (step, trim):
        assert call(pool(), plan(), ws=0) == WSP and "256-byte" in sage.last_error()
        assert call(pool(), plan(), n=N - 1) == WSP and "needs" in sage.last_error()
    assert trim(pool(), requests=0, count=0) == sage.OK


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sage.PagePool(torch.zeros(8, **i32), torch.zeros(1, **i32), torch.zeros(2, 3, **i32),
                      torch.zeros(2, **i32), 16)
    b = torch.zeros(4, 16, 2, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        sage.PagedCache(b, b, head_dim=64)
    with pytest.raises(ValueError, match="rows of"):
        sage.PagedCache(b, b, head_dim=72)
    with pytest.raises(TypeError, match="uint8"):
        sage.PagedCache(b, b.to(torch.int8), head_dim=64)
    for bad in ((), (65,), (-1, 3), (1,) * 9, (0, 0)):
        with pytest.raises(ValueError, match="sections"):
            sage.rope_axes(bad, device="cpu")


def test_the_axis_of_each_pair():
    pytest.importorskip("torch")
    assert sage.rope_axes((2, 3, 1), device="cpu").tolist() == [0, 0, 1, 1, 1, 2]
    assert sage.rope_axes((2, 3, 1), in_turn=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 1]
    assert sage.rope_axes((0, 2), in_turn=True, device="cpu").tolist() == [1, 1]
