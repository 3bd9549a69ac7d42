"""Latent attention without a GPU: sizes, host-side refusals of the C ABI and of the binding (all
answered before any launch), and pins of the codec reference the GPU tests compare with."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import latent_ref as ref  # noqa: E402
from compressed_paged_kv_quant_gb300 import build, kvq  # noqa: E402


@pytest.fixture(scope="module")
def L():
    build.build()
    return kvq.lib()


def test_sizes(L):
    gb, gm = kvq.latent_geom(kvq.LATENT_BF16, 3, 128), kvq.latent_geom(kvq.LATENT_MXFP8, 3, 128)
    assert kvq.latent_page_bytes(gb) == 3 * 64 * 1152 and kvq.latent_token_bytes(gb) == 3 * 1152
    assert kvq.latent_page_bytes(gm) == 3 * 64 * 656 and kvq.latent_token_bytes(gm) == 3 * 656
    assert kvq.latent_workspace_bytes(gb, 8, 1, 40960) > 0
    assert kvq.latent_workspace_bytes(gb, 0, 0, 0) > 0
    assert kvq.latent_workspace_bytes(gb, -1, 1, 64) == 0
    assert kvq.latent_prefill_workspace_bytes(1, 16, 8, 8, 64) > 0
    assert kvq.latent_prefill_workspace_bytes(1, 129, 8, 8, 64) == 0


@pytest.mark.parametrize("bad", [dict(format=2), dict(latent_dim=256), dict(rope_dim=32), dict(page_tokens=32),
                                 dict(num_q_heads=129), dict(num_q_heads=0), dict(num_layers=0)])
def test_unsupported_geometry_is_refused(L, bad):
    args = dict(format=0, num_layers=2, num_q_heads=16, latent_dim=512, rope_dim=64, page_tokens=64)
    args.update(bad)
    g = kvq.LatentGeom(*[args[k] for k, _ in kvq.LatentGeom._fields_])
    assert kvq.latent_page_bytes(g) == 0 and kvq.latent_workspace_bytes(g, 1, 1, 64) == 0
    assert _attn(L, g) in (kvq.ERR_UNSUPPORTED, kvq.ERR_INVALID_ARG)
    assert _append(L, g) in (kvq.ERR_UNSUPPORTED, kvq.ERR_INVALID_ARG)


def _rows(ptr, row=512, head=0):
    return ctypes.byref(kvq.Rows(ptr, row, head))


def _append(L, g, fn="kvq_latent_append", **kw):
    a = dict(layer=0, pool=256, pool_bytes=1 << 24, pt=768, max_pages=4, lanes=1, start=1024, n=1040, off=1056,
             most=1, rows=8, lat=_rows(4096), rope=_rows(8192, 64), status=2048)
    a.update(kw)
    return getattr(L, fn)(ctypes.byref(g), a["layer"], a["pool"], a["pool_bytes"], a["pt"], a["max_pages"],
                          a["lanes"], a["start"], a["n"], a["off"], a["most"], a["rows"], a["lat"], a["rope"],
                          a["status"], None)


@pytest.mark.parametrize("fn", ["kvq_latent_append", "kvq_latent_read"])
def test_token_calls_are_refused_on_the_host(L, fn):
    g = kvq.latent_geom(kvq.LATENT_MXFP8, 2, 16)
    for kw in (dict(layer=2), dict(layer=-1), dict(lanes=-1), dict(most=-1), dict(rows=-1), dict(pool=None),
               dict(pt=None), dict(start=None), dict(n=None), dict(off=None), dict(status=None), dict(lat=None),
               dict(rope=_rows(None)), dict(pool_bytes=1000), dict(max_pages=1 << 26)):
        assert _append(L, g, fn, **kw) == kvq.ERR_INVALID_ARG, kw
    for kw in (dict(pool=264), dict(lat=_rows(4100)), dict(lat=_rows(4096, 515)), dict(rope=_rows(8192, 68))):
        assert _append(L, g, fn, **kw) == kvq.ERR_ALIGNMENT, kw
    assert _append(L, g, fn, lanes=0) == kvq.OK and _append(L, g, fn, most=0) == kvq.OK


def _attn(L, g, **kw):
    a = dict(layer=0, pool=256, pool_bytes=1 << 24, pt=768, max_pages=4, lanes=1, pos=1024, nq=1040, off=1056,
             most=1, rows=8, seq=1072, max_seq=256, ql=_rows(4096, 8192, 512), qr=_rows(8192, 1024, 64), scale=0.07,
             ws=1536, ws_bytes=1 << 40, out=_rows(16384, 8192, 512), status=2048)
    a.update(kw)
    return L.kvq_paged_latent_attn(ctypes.byref(g), a["layer"], a["pool"], a["pool_bytes"], a["pt"], a["max_pages"],
                                   a["lanes"], a["pos"], a["nq"], a["off"], a["most"], a["rows"], a["seq"],
                                   a["max_seq"], a["ql"], a["qr"], a["scale"], a["ws"], a["ws_bytes"], a["out"],
                                   a["status"], None)


def test_paged_attention_is_refused_on_the_host(L):
    g = kvq.latent_geom(kvq.LATENT_BF16, 2, 16)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(layer=2), dict(max_seq=257), dict(max_seq=-1), dict(most=-1), dict(rows=-1), dict(pool=None),
               dict(pos=None), dict(nq=None), dict(off=None), dict(seq=None), dict(ws=None), dict(status=None),
               dict(ql=None), dict(qr=None), dict(out=None), dict(pool_bytes=100), dict(scale=nan), dict(scale=inf),
               dict(scale=-0.1)):
        assert _attn(L, g, **kw) == kvq.ERR_INVALID_ARG, kw
    for kw in (dict(ql=_rows(4104, 8192, 512)), dict(ql=_rows(4096, 8192, 516)), dict(out=_rows(16384, 8190, 512)),
               dict(ws=1544)):
        assert _attn(L, g, **kw) == kvq.ERR_ALIGNMENT, kw
    assert _attn(L, g, ws_bytes=0) == kvq.ERR_WORKSPACE_TOO_SMALL
    assert _attn(L, g, lanes=0) == kvq.OK and _attn(L, g, most=0) == kvq.OK


def test_prefill_is_refused_on_the_host(L):
    def pre(**kw):
        a = dict(heads=16, lanes=1, pos=1024, nq=1040, off=1056, most=4, rows=8, nk=1072, koff=1088, max_k=64,
                 krows=64, qn=_rows(4096, 2048, 128), qr=_rows(8192, 1024, 64), kn=_rows(4096, 2048, 128),
                 kr=_rows(8192, 64), v=_rows(4096, 2048, 128), scale=0.07, ws=1536, ws_bytes=1 << 40,
                 out=_rows(16384, 2048, 128), status=2048)
        a.update(kw)
        return L.kvq_latent_prefill_attn(a["heads"], a["lanes"], a["pos"], a["nq"], a["off"], a["most"], a["rows"],
                                         a["nk"], a["koff"], a["max_k"], a["krows"], a["qn"], a["qr"], a["kn"],
                                         a["kr"], a["v"], a["scale"], a["ws"], a["ws_bytes"], a["out"], a["status"],
                                         None)
    for kw in (dict(heads=0), dict(lanes=-1), dict(most=-1), dict(rows=-1), dict(max_k=-1), dict(krows=-1),
               dict(pos=None), dict(nq=None), dict(nk=None), dict(koff=None), dict(off=None), dict(ws=None),
               dict(status=None), dict(qn=None), dict(kn=None), dict(kr=_rows(None)), dict(v=None), dict(out=None),
               dict(scale=-1.0)):
        assert pre(**kw) == kvq.ERR_INVALID_ARG, kw
    assert pre(heads=129) == kvq.ERR_UNSUPPORTED
    assert pre(v=_rows(4096, 2048, 100)) == kvq.ERR_ALIGNMENT and pre(qr=_rows(8196)) == kvq.ERR_ALIGNMENT
    assert pre(ws_bytes=0) == kvq.ERR_WORKSPACE_TOO_SMALL
    assert pre(lanes=0) == kvq.OK and pre(most=0) == kvq.OK


def test_binding_refuses_host_tensors(L):
    """The binding answers with the library's error before it touches a device."""
    g = kvq.latent_geom(kvq.LATENT_BF16, 1, 16)
    i = torch.zeros(1, dtype=torch.int32)
    pool = torch.zeros(kvq.latent_page_bytes(g), dtype=torch.uint8)
    lat, rope = torch.zeros(1, 512, dtype=torch.bfloat16), torch.zeros(1, 64, dtype=torch.bfloat16)
    q, qr = torch.zeros(1, 16, 512, dtype=torch.bfloat16), torch.zeros(1, 16, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: kvq.latent_append(g, 0, pool, t, i, i, i, 1, lat, rope, i),
                 lambda: kvq.latent_read(g, 0, pool, t, i, i, i, 1, lat, rope, i),
                 lambda: kvq.paged_latent_attn(g, 0, pool, t, i, i, i, 1, i, 64, q, qr, 0.1, pool, q, i),
                 lambda: kvq.latent_prefill_attn(i, i, i, 1, i, i, 1, qr, qr, qr, lat, qr, 0.1, pool, qr, i)):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert e.value.code == kvq.ERR_INVALID_ARG
    with pytest.raises(kvq.KvqError):
        kvq.LatentCache(kvq.latent_geom(kvq.LATENT_BF16, 1, 16, latent_dim=256), 1, device="cpu")


def test_reference_codec():
    """The tests' codec: codes equal torch's E4M3 conversion of the scaled values, a decoded value
    is exact in bf16, and the scale is the least that keeps the group within 448."""
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(64, 512, generator=g) * torch.exp(6 * torch.randn(64, 512, generator=g))).clamp(-57344, 57344)
    x[0], x[1] = 0.0, 448.0
    x[2], x[3] = 2.0 ** -126, 57344.0
    x[4, ::2], x[4, 1::2] = 449.0, 17.0
    x = x.bfloat16()
    code, scale = ref.encode(x)
    e = scale.double() - 127
    y = (x.double().view(64, 16, 32) * torch.exp2(-e)[..., None]).view(64, 512)
    assert torch.equal(y.float().to(torch.float8_e4m3fn).view(torch.uint8), code)
    val = ref.decode(code, scale)
    assert torch.equal(val, val.bfloat16().double())
    assert torch.equal(val, (code.view(torch.float8_e4m3fn).double().view(64, 16, 32) * torch.exp2(e)[..., None]).view(64, 512))
    a = x.double().abs().view(64, 16, 32).amax(-1)
    assert bool((a <= 448 * torch.exp2(e)).all()) and bool(((a > 224 * torch.exp2(e)) | (e == -120)).all())


def _prefill(L, **kw):
    a = dict(heads=16, most=4, rows=8, max_k=64, krows=64, qn=_rows(4096, 2048, 128), qr=_rows(8192, 1024, 64),
             kn=_rows(4096, 2048, 128), kr=_rows(8192, 64), v=_rows(4096, 2048, 128), out=_rows(16384, 2048, 128))
    a.update(kw)
    return L.kvq_latent_prefill_attn(a["heads"], 1, 1024, 1040, 1056, a["most"], a["rows"], 1072, 1088, a["max_k"],
                                     a["krows"], a["qn"], a["qr"], a["kn"], a["kr"], a["v"], 0.07, 1536, 1 << 60,
                                     a["out"], 2048, None)


def test_overlapping_outputs_are_refused(L):
    """Rows or heads of an output that share one place would race."""
    g = kvq.latent_geom(kvq.LATENT_BF16, 2, 16)
    assert _attn(L, g, out=_rows(16384, 0, 512)) == kvq.ERR_INVALID_ARG
    assert _attn(L, g, out=_rows(16384, 8192, 0)) == kvq.ERR_INVALID_ARG
    assert _append(L, g, "kvq_latent_read", lat=_rows(4096, 0)) == kvq.ERR_INVALID_ARG
    assert _append(L, g, "kvq_latent_read", rope=_rows(8192, 0)) == kvq.ERR_INVALID_ARG
    assert _prefill(L, out=_rows(16384, 0, 128)) == kvq.ERR_INVALID_ARG
    assert _prefill(L, out=_rows(16384, 2048, 0)) == kvq.ERR_INVALID_ARG


def test_prefill_strides_that_no_tensor_map_takes(L):
    for kw in (dict(qn=_rows(4096, 0, 128)), dict(qr=_rows(8192, -1024, 64)), dict(kn=_rows(4096, 2048, -128)),
               dict(kr=_rows(8192, 0)), dict(v=_rows(4096, 1 << 39, 128)), dict(kn=_rows(4096, 2048, 1 << 40))):
        assert _prefill(L, **kw) == kvq.ERR_UNSUPPORTED, kw
    assert _prefill(L, krows=0) == kvq.ERR_INVALID_ARG


def test_sizes_past_32_bits_are_refused(L):
    """The largest counts that the types allow: refused before any arithmetic on them could wrap."""
    big = 2 ** 31 - 1
    g = kvq.latent_geom(kvq.LATENT_BF16, 2, 128)
    assert kvq.latent_workspace_bytes(g, 1, big, 64) == 0
    assert _attn(L, g, most=big, rows=big) == kvq.ERR_UNSUPPORTED
    assert kvq.latent_prefill_workspace_bytes(1, 16, 8, big, 64) == 0
    assert kvq.latent_prefill_workspace_bytes(1, 16, 8, 8, big) == 0
    assert _prefill(L, most=big) == kvq.ERR_UNSUPPORTED and _prefill(L, max_k=big) == kvq.ERR_UNSUPPORTED
    assert _attn(L, g, lanes=big, max_pages=1 << 20, max_seq=1 << 26, ws_bytes=(1 << 62)) == kvq.ERR_UNSUPPORTED
    assert _append(L, g, lanes=big, most=big) == kvq.ERR_UNSUPPORTED
    assert _append(L, g, "kvq_latent_read", lanes=big, most=big) == kvq.ERR_UNSUPPORTED


@pytest.mark.parametrize("heads", [1, 16, 24, 100, 128])
def test_workspace_for_the_most_serves_every_smaller_call(L, heads):
    """A server sizes one workspace for its largest call and makes all of its calls with it."""
    g = kvq.latent_geom(kvq.LATENT_BF16, 2, heads)
    lanes, most, long = (1, 7, 64, 300), (0, 1, 2, 3, 16, 38, 39, 64, 512), (0, 64, 512, 513, 5000, 40960, 2 ** 31 - 1)
    for i, b in enumerate(lanes):
        for j, n in enumerate(most):
            for k, m in enumerate(long):
                size = kvq.latent_workspace_bytes(g, b, n, m)
                assert size > 0
                for less in ((lanes[i - 1], n, m) if i else None, (b, most[j - 1], m) if j else None,
                             (b, n, long[k - 1]) if k else None):
                    assert less is None or kvq.latent_workspace_bytes(g, *less) <= size, (b, n, m, less)


def test_prefill_workspace_for_the_most_serves_every_smaller_call(L):
    """The same for the expanded form, whose split depends on lanes, heads, queries and keys."""
    axes = [(1, 2, 8, 9, 300), (1, 16, 25, 32, 128), (1, 100, 256, 257, 1024, 2048, 2 ** 31 - 257),
            (1, 1000, 1920, 1921, 5000, 16000, 65536, 2 ** 31 - 257)]
    size = {}
    for lanes in axes[0]:
        for heads in axes[1]:
            for n in axes[2]:
                for m in axes[3]:
                    size[lanes, heads, n, m] = kvq.latent_prefill_workspace_bytes(lanes, heads, 4096, n, m)
    for at, here in size.items():
        assert here > 0
        for i, axis in enumerate(axes):
            j = axis.index(at[i])
            if j:
                assert size[at[:i] + (axis[j - 1],) + at[i + 1:]] <= here, (at, i)
    rows = {kvq.latent_prefill_workspace_bytes(2, 16, r, 256, 16000) for r in (1, 512, 4096, 2 ** 31 - 1)}
    assert len(rows) == 1


def _prefill_short(L, **kw):
    """Without a workspace: stopped by the check of its size, the last one."""
    a = dict(heads=16, rows=8, krows=64, qn=_rows(4096, 2048, 128), qr=_rows(8192, 1024, 64), kn=_rows(4096, 2048, 128),
             kr=_rows(8192, 64), v=_rows(4096, 2048, 128), out=_rows(16384, 2048, 128))
    a.update(kw)
    return L.kvq_latent_prefill_attn(a["heads"], 1, 1024, 1040, 1056, 4, a["rows"], 1072, 1088, 64, a["krows"], a["qn"],
                                     a["qr"], a["kn"], a["kr"], a["v"], 0.07, 1536, 0, a["out"], 2048, None)


def test_unused_strides_may_be_anything(L):
    """Head strides of rows without heads or with one, and row strides of one row: a caller need not set them.  (Each call
    is stopped by a later check.)"""
    odd = 12345
    big = dict(lanes=2 ** 31 - 1, most=2 ** 31 - 1)
    g, one = kvq.latent_geom(kvq.LATENT_BF16, 2, 16), kvq.latent_geom(kvq.LATENT_BF16, 2, 1)
    for fn in ("kvq_latent_append", "kvq_latent_read"):
        assert _append(L, g, fn, lat=_rows(4096, 512, odd), rope=_rows(8192, 64, odd), **big) == kvq.ERR_UNSUPPORTED
        assert _append(L, g, fn, rows=1, lat=_rows(4096, odd), rope=_rows(8192, odd), **big) == kvq.ERR_UNSUPPORTED
    short = dict(ws_bytes=0)
    assert _attn(L, one, ql=_rows(4096, 512, odd), qr=_rows(8192, 64, odd), out=_rows(16384, 512, odd), **short) == kvq.ERR_WORKSPACE_TOO_SMALL
    assert _attn(L, g, rows=1, ql=_rows(4096, odd, 512), qr=_rows(8192, odd, 64), out=_rows(16384, odd, 512), **short) == kvq.ERR_WORKSPACE_TOO_SMALL
    assert _prefill_short(L, kr=_rows(8192, 64, odd)) == kvq.ERR_WORKSPACE_TOO_SMALL
    assert _prefill_short(L, heads=1, qn=_rows(4096, 128, odd), qr=_rows(8192, 64, odd), kn=_rows(4096, 128, odd), v=_rows(4096, 128, odd),
                          out=_rows(16384, 128, odd)) == kvq.ERR_WORKSPACE_TOO_SMALL
    assert _prefill_short(L, rows=1, krows=1, qn=_rows(4096, odd, 128), qr=_rows(8192, odd, 64), kn=_rows(4096, odd, 128), kr=_rows(8192, odd),
                          v=_rows(4096, odd, 128), out=_rows(16384, odd, 128)) == kvq.ERR_WORKSPACE_TOO_SMALL
    assert _attn(L, g, ql=_rows(4096, 8192, odd), **short) == kvq.ERR_ALIGNMENT
    assert _attn(L, one, ql=_rows(4096, odd), **short) == kvq.ERR_ALIGNMENT


def _shared(row, head, rows, heads, dims):
    """By definition: does any element belong to two rows?"""
    at = [r * row + h * head for r in range(rows) for h in range(heads)]
    at.sort()
    return any(b - a < dims for a, b in zip(at, at[1:]))


def test_outputs_that_overlap_in_part_are_refused(L):
    """Every layout of rows and heads whose elements meet, and no other (the accepted ones are stopped by the check of the
    workspace, or of the grid)."""
    g = kvq.latent_geom(kvq.LATENT_BF16, 2, 16)
    three = kvq.latent_geom(kvq.LATENT_BF16, 2, 3)
    seen = set()
    for row in (8, 256, 504, 512, 520, 1016, 1024, 1032, 1536, 2048, 3080, 4096, 7680, 8192, -512, -1024, -8192, 1 << 40, 1 << 62):
        for head in (8, 504, 512, 520, 1024, 1536, 1544, 2048, 4096, 8192, 16384, -512, -1032, -4096, -8192, 1 << 40, 1 << 62):
            for geom, heads in ((g, 16), (three, 3)):
                for rows in (1, 2, 3, 8):
                    want = _shared(row, head, rows, heads, 512)
                    got = _attn(L, geom, rows=rows, out=_rows(16384, row, head), ws_bytes=0)
                    assert got == (kvq.ERR_INVALID_ARG if want else kvq.ERR_WORKSPACE_TOO_SMALL), (row, head, rows, heads)
                    seen.add((want, rows > 1))
    assert len(seen) == 4
    for row, head in ((8, 128), (120, 128 * 8), (2048, 120), (128 * 3, 128), (256, 128)):
        assert _prefill_short(L, out=_rows(16384, row, head)) == kvq.ERR_INVALID_ARG, (row, head)
    for row, head in ((128, 128 * 8), (2048, 128), (2176, 136)):
        assert _prefill_short(L, out=_rows(16384, row, head)) == kvq.ERR_WORKSPACE_TOO_SMALL, (row, head)
    big = dict(lanes=2 ** 31 - 1, most=2 ** 31 - 1)
    for lat, rope, rc in ((504, 64, kvq.ERR_INVALID_ARG), (512, 56, kvq.ERR_INVALID_ARG), (-504, 64, kvq.ERR_INVALID_ARG),
                          (512, 64, kvq.ERR_UNSUPPORTED), (-512, -64, kvq.ERR_UNSUPPORTED), (576, 576, kvq.ERR_UNSUPPORTED)):
        assert _append(L, g, "kvq_latent_read", lat=_rows(4096, lat), rope=_rows(8192, rope), **big) == rc, (lat, rope)
