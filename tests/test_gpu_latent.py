"""Latent attention on the GPU against a plain 64-bit reference: pool bytes bit for bit, reads
exact, attention within a tolerance derived in latent_ref.tolerance."""
import math

import pytest

torch = pytest.importorskip("torch")

import latent_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, MXFP8 = 0, 1
FORMATS = pytest.mark.parametrize("fmt", [BF16, MXFP8], ids=["bf16", "mxfp8"])


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_paged_kv_quant_gb300 import build, kvq as k
    build.build()
    k.lib()
    return k


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rnd(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).bfloat16()


def offsets(counts, gap=0):
    out, at = [], gap
    for n in counts:
        out.append(at)
        at += n
    return out, at + gap


def page_table(lens, gen, spare=3):
    """Permuted pages of the lanes, with `spare` pages that belong to nobody."""
    need = [-(-n // 64) for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=gen)
    table, at = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        at += n
    return table, sum(need) + spare


# ------------------------------------------------------------------------------------- the cache
@FORMATS
def test_append_and_read_bit_for_bit(kvq, fmt):
    """Ragged lanes (one without tokens) in two calls, strided inputs, dirty pool: every byte of the
    pool is the reference's, other layers, slots and pages are untouched; reads are exact and leave
    the rows of nobody as they were."""
    gen = torch.Generator().manual_seed(1 + fmt)
    layers, layer = 3, 1
    first, second = [5, 0, 64, 130, 1], [60, 3, 1, 0, 200]
    total = [x + y for x, y in zip(first, second)]
    table, pages = page_table(total, gen)
    want = ref.Pool(fmt, layers, pages)
    pool = want.bytes.reshape(-1).cuda()
    g = kvq.latent_geom(fmt, layers, 16)
    assert pool.numel() == pages * kvq.latent_page_bytes(g)
    status, start, held = i32([0]), [0] * 5, []
    for counts in (first, second):
        off, rows = offsets(counts, gap=2)
        both = rnd(gen, rows, 592, scale=3.0)
        both[::3] *= torch.exp(3 * torch.randn(both[::3].shape, generator=gen)).bfloat16()
        both.clamp_(-57344, 57344)
        dev = both.cuda()
        kvq.latent_append(g, layer, pool, table.cuda(), i32(start), i32(counts), i32(off), max(counts),
                          dev[:, :512], dev[:, 520:584], status)
        for b, n in enumerate(counts):
            r = slice(off[b], off[b] + n)
            want.write(layer, table[b], range(start[b], start[b] + n), both[r, :512], both[r, 520:584])
        start = [x + y for x, y in zip(start, counts)]
    assert status.item() == 0
    assert torch.equal(pool.cpu(), want.bytes.reshape(-1))

    lo = [3, 0, 63, 10, 1]
    count = [n - x for n, x in zip(total, lo)]
    off, rows = offsets(count, gap=1)
    out = torch.full((rows, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    kvq.latent_read(g, layer, pool, table.cuda(), i32(lo), i32(count), i32(off), max(count), out[:, :512],
                    out[:, 528:592], status)
    assert status.item() == 0
    expect = torch.full((rows, 600), 7.0, dtype=torch.float64)
    for b, n in enumerate(count):
        lat, rope = want.read(layer, table[b], range(lo[b], total[b]))
        expect[off[b]:off[b] + n, :512], expect[off[b]:off[b] + n, 528:592] = lat, rope
    assert torch.equal(out.cpu().double(), expect)


def test_append_extreme_values(kvq):
    """Groups of zeros, subnormals, ties, the largest value, and one large value among small ones."""
    x = torch.zeros(64, 512)
    g = torch.Generator().manual_seed(3)
    x[1] = 57344.0
    x[2] = 2.0 ** -133
    x[3] = 2.0 ** -120
    x[4, ::32] = 448.0
    x[4, 1::2] = torch.linspace(0.0, 1.0, 256)
    x[5] = torch.linspace(-449, 449, 512)
    x[6, ::32] = 1.75
    x[7, ::32] = 1.7578125
    x[8] = -57344.0
    for i in range(9, 64):
        x[i] = torch.randn(512, generator=g) * 2.0 ** torch.randint(-130, 13, (1,), generator=g).item()
    x = x.bfloat16()
    rope = torch.zeros(64, 64).bfloat16()
    rope[0] = 3.0e38
    want = ref.Pool(MXFP8, 1, 1)
    want.write(0, [0], range(64), x, rope)
    pool, status = torch.full((41984,), 0x5A, dtype=torch.uint8, device="cuda"), i32([0])
    geom = kvq.latent_geom(MXFP8, 1, 1)
    kvq.latent_append(geom, 0, pool, i32([[0]]), i32([0]), i32([64]), i32([0]), 64, x.cuda(), rope.cuda(), status)
    assert status.item() == 0
    assert torch.equal(pool.cpu(), want.bytes.reshape(-1))
    lat, rp = torch.zeros(64, 512).bfloat16().cuda(), torch.zeros(64, 64).bfloat16().cuda()
    kvq.latent_read(geom, 0, pool, i32([[0]]), i32([0]), i32([64]), i32([0]), 64, lat, rp, status)
    assert torch.equal(lat.cpu().double(), want.read(0, [0], range(64))[0])


@FORMATS
def test_bad_tokens_and_lanes_are_flagged_and_skipped(kvq, fmt):
    gen = torch.Generator().manual_seed(5)
    g = kvq.latent_geom(fmt, 1, 1)
    lat, rope = rnd(gen, 6, 512), rnd(gen, 6, 64)
    lat[1, 17], rope[2, 5] = float("nan"), float("inf")
    if fmt == MXFP8:
        lat[3, 511] = 57600.0
    want = ref.Pool(fmt, 1, 2)
    for i in (0, 4, 5) if fmt == MXFP8 else (0, 3, 4, 5):
        want.write(0, [1], [62 + i if i < 2 else i - 2], lat[i:i + 1], rope[i:i + 1]) if i >= 2 else \
            want.write(0, [0], [62 + i], lat[i:i + 1], rope[i:i + 1])
    pool, status = torch.full_like(want.bytes, 0xA5).cuda().reshape(-1), i32([0])
    kvq.latent_append(g, 0, pool, i32([[0, 1]]), i32([62]), i32([6]), i32([0]), 6, lat.cuda(), rope.cuda(), status)
    assert status.item() == kvq.STATUS_BAD_INPUT
    assert torch.equal(pool.cpu(), want.bytes.reshape(-1))

    good, rp = rnd(gen, 8, 512).cuda(), rnd(gen, 8, 64).cuda()
    before = pool.clone()
    for table, start, n, off, most, bit in (([[2]], 0, 1, 0, 1, kvq.STATUS_PAGE_OOB),
                                            ([[-1]], 0, 1, 0, 1, kvq.STATUS_PAGE_OOB),
                                            ([[0]], 64, 1, 0, 1, kvq.STATUS_LEN_GT_TABLE),
                                            ([[0]], 2 ** 31 - 1, 1, 0, 1, kvq.STATUS_LEN_GT_TABLE),
                                            ([[0]], 0, -1, 0, 1, kvq.STATUS_BAD_LEN),
                                            ([[0]], 0, 3, 0, 2, kvq.STATUS_BAD_LEN),
                                            ([[0]], 0, 1, 8, 1, kvq.STATUS_BAD_LEN),
                                            ([[0]], 0, 1, -1, 1, kvq.STATUS_BAD_LEN),
                                            ([[0]], -1, 1, 0, 1, kvq.STATUS_BAD_LEN)):
        for call in (kvq.latent_append, kvq.latent_read):
            status.zero_()
            call(g, 0, pool, i32(table), i32([start]), i32([n]), i32([off]), most, good.clone(), rp.clone(), status)
            assert status.item() == bit, (call.__name__, start, n, off)
    assert torch.equal(pool, before)


# ------------------------------------------------------------------------------------- absorbed
class Absorbed:
    """A filled cache and a call of paged_latent_attn over it."""

    def __init__(self, kvq, fmt, heads, lens, nqs, seed, layers=2, layer=1, head_first=True, q_scale=1.0, garbage=0xFF,
                 gap=1):
        gen = torch.Generator().manual_seed(seed)
        self.kvq, self.fmt, self.heads, self.lens, self.nqs, self.layer = kvq, fmt, heads, lens, nqs, layer
        self.table, pages = page_table(lens, gen)
        self.g = kvq.latent_geom(fmt, layers, heads)
        # every byte that no token owns is 0xFF: NaN in bf16, in E4M3 and as a scale
        self.pool = torch.full((pages * kvq.latent_page_bytes(self.g),), garbage, dtype=torch.uint8, device="cuda")
        self.status = i32([0])
        off, rows = offsets(lens)
        lat = (torch.randn(max(rows, 1), 512, generator=gen) * torch.exp(0.4 * torch.randn(512, generator=gen))).bfloat16()
        self.lat, self.rope = lat.cuda(), rnd(gen, max(rows, 1), 64).cuda()
        kvq.latent_append(self.g, layer, self.pool, self.table.cuda(), i32([0] * len(lens)), i32(lens), i32(off),
                          max(lens + [1]), self.lat, self.rope, self.status)
        self.off, self.rows = offsets(nqs, gap=gap)
        n = self.rows
        if head_first:
            self.ql = rnd(gen, heads, n, 512, scale=q_scale).cuda().transpose(0, 1)
            wide = rnd(gen, n, heads, 192, scale=q_scale).cuda()
            self.qr = wide[..., 128:]
            self.out = torch.full((heads, n, 512), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        else:
            self.ql, self.qr = rnd(gen, n, heads, 512, scale=q_scale).cuda(), rnd(gen, n, heads, 64, scale=q_scale).cuda()
            self.out = torch.full((n, heads, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        self.scale = 1 / math.sqrt(192)
        self.max_nq, self.max_len = max(nqs), max(lens)
        self.seq_len, self.n_q, self.q_off = i32(lens), i32(nqs), i32(self.off)
        self.pos = i32([max(0, n - q) for n, q in zip(lens, nqs)])
        self.dtable = self.table.cuda()
        self.ws = torch.full((kvq.latent_workspace_bytes(self.g, len(lens), self.max_nq, self.max_len),), 0xFF,
                             dtype=torch.uint8, device="cuda")

    def call(self, **kw):
        a = dict(stream=None)
        a.update(kw)
        self.kvq.paged_latent_attn(self.g, self.layer, self.pool, self.dtable, self.pos, self.n_q, self.q_off,
                                   self.max_nq, self.seq_len, self.max_len, self.ql, self.qr, self.scale, self.ws,
                                   self.out, self.status, **a)

    def keys(self, b):
        """What the cache holds of lane b, in float64 (codes of the reference for MXFP8)."""
        o, _ = offsets(self.lens)
        lat, rope = self.lat[o[b]:o[b] + self.lens[b]], self.rope[o[b]:o[b] + self.lens[b]].double()
        if self.fmt == BF16:
            return lat.double(), rope
        code, scale = ref.encode(lat)
        return ref.decode(code, scale), rope

    def check(self, skip=()):
        mine = torch.zeros(self.rows, dtype=torch.bool)
        for b, (n, nq) in enumerate(zip(self.lens, self.nqs)):
            if nq == 0 or b in skip:
                continue
            r = slice(self.off[b], self.off[b] + nq)
            mine[r] = True
            lat, rope = self.keys(b)
            q = torch.cat([self.ql[r], self.qr[r]], -1).double().transpose(0, 1)
            k = torch.cat([lat, rope], 1)[None]
            out, weight, mag = ref.attend(q, k, lat[None], self.scale, self.pos[b].item())
            err = (self.out[r].double().transpose(0, 1) - out).abs()
            tol = ref.tolerance(out, weight, mag, self.scale, 576)
            assert bool((err <= tol).all()), f"lane {b}: {(err / tol).max().item():.3g} of the tolerance"
        assert bool((self.out[~mine.cuda()] == 3.0).all()), "rows of nobody were written"


@FORMATS
@pytest.mark.parametrize("heads", [1, 5, 16, 24, 64, 100, 128])
def test_decode_ragged(kvq, fmt, heads):
    """One query a lane over lengths around the page size, one lane without a query."""
    c = Absorbed(kvq, fmt, heads, [1, 2, 63, 64, 65, 128, 700, 0, 1000], [1, 1, 1, 1, 1, 1, 1, 0, 1], 10 + heads)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
@pytest.mark.parametrize("heads,nqs", [(16, [4, 1, 0, 7]), (128, [2, 3, 1, 2]), (8, [1, 8, 9, 16]), (40, [3, 5, 2, 1]),
                                       (128, [65, 1, 0, 4])])
def test_chunk_of_new_tokens_is_causal(kvq, fmt, heads, nqs):
    c = Absorbed(kvq, fmt, heads, [200, 9, 64, 131], nqs, 30 + heads, head_first=False)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
@pytest.mark.parametrize("heads,lens,nqs", [(16, [20011], [1]), (128, [9000, 40, 5121], [1, 1, 1]),
                                            (32, [16384, 1], [2, 1]), (128, [3000] * 20, [1] * 20)])
def test_long_lanes_are_split_and_joined(kvq, fmt, heads, lens, nqs):
    c = Absorbed(kvq, fmt, heads, lens, nqs, 50 + heads)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
def test_whole_prompt_through_the_pages(kvq, fmt):
    """A chunk as long as its lane: every position from the first."""
    c = Absorbed(kvq, fmt, 16, [300, 129], [300, 129], 60)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
def test_large_scores_and_rising_maxima(kvq, fmt):
    """Scores that span hundreds: one key takes all, and the running maximum rises late in the lane."""
    c = Absorbed(kvq, fmt, 16, [1500, 700], [1, 2], 61, q_scale=8.0)
    c.call()
    assert c.status.item() == 0
    c.check()
    c.scale = 0.0                        # every weight equal
    c.call()
    c.check()


@FORMATS
def test_first_pages_far_below(kvq, fmt):
    """Keys whose scores rise steadily with the position, so every tile moves the maximum."""
    c = Absorbed(kvq, fmt, 16, [2000], [1], 62)
    q = c.ql[1, 0].double()
    c.lat[:2000] = (torch.linspace(-40, 40, 2000, device="cuda")[:, None] * (q / q.norm())).bfloat16()
    c.kvq.latent_append(c.g, c.layer, c.pool, c.dtable, i32([0]), i32([2000]), i32([0]), 2000, c.lat, c.rope, c.status)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
def test_refused_lanes_and_pages(kvq, fmt):
    """Bad lanes are skipped and flagged, the others are answered; a page outside the pool is not
    attended; a lane without any page of its own gives zeros."""
    lens, nqs = [100, 200, 300, 64], [1, 2, 1, 1]
    for field, b, value, bit in (("seq_len", 1, -1, kvq.STATUS_BAD_LEN), ("seq_len", 1, 301, kvq.STATUS_BAD_LEN),
                                 ("n_q", 1, 3, kvq.STATUS_BAD_LEN), ("n_q", 1, -1, kvq.STATUS_BAD_LEN),
                                 ("pos", 1, 199, kvq.STATUS_BAD_LEN), ("pos", 1, -1, kvq.STATUS_BAD_LEN),
                                 ("q_off", 1, 6, kvq.STATUS_BAD_LEN), ("q_off", 1, -1, kvq.STATUS_BAD_LEN)):
        c = Absorbed(kvq, fmt, 16, lens, nqs, 63)
        getattr(c, field)[b] = value
        c.call()
        assert c.status.item() == bit, (field, value)
        c.check(skip=(b,)) if field != "n_q" else None
    c = Absorbed(kvq, fmt, 16, lens, nqs, 64)
    c.dtable[3, 0] = 10 ** 6
    c.dtable[2, 1] = -7
    c.call()
    assert c.status.item() == kvq.STATUS_PAGE_OOB
    assert bool((c.out[c.off[3]] == 0).all())
    lat, rope = c.keys(2)
    keep = torch.cat([torch.arange(64), torch.arange(128, 300)]).cuda()
    q = torch.cat([c.ql[c.off[2]:c.off[2] + 1], c.qr[c.off[2]:c.off[2] + 1]], -1).double().transpose(0, 1)
    out, weight, mag = ref.attend(q, torch.cat([lat, rope], 1)[None, keep], lat[None, keep], c.scale, 10 ** 6)
    err = (c.out[c.off[2]:c.off[2] + 1].double().transpose(0, 1) - out).abs()
    assert bool((err <= ref.tolerance(out, weight, mag, c.scale, 576)).all())


@FORMATS
def test_pool_past_32_bits(kvq, fmt):
    """Pages whose byte offsets pass 4 GiB: the lane's pages are the last of a large pool."""
    g = kvq.latent_geom(fmt, 16, 16)
    pages = (5 << 30) // kvq.latent_page_bytes(g)
    c = Absorbed(kvq, fmt, 16, [300], [1], 65, layers=16, layer=15)
    c.pool = torch.empty(pages * kvq.latent_page_bytes(g), dtype=torch.uint8, device="cuda")
    c.dtable = (pages - 1 - torch.arange(5, dtype=torch.int32, device="cuda")).int()[None]
    c.kvq.latent_append(c.g, 15, c.pool, c.dtable, i32([0]), i32([300]), i32([0]), 300, c.lat, c.rope, c.status)
    c.call()
    assert c.status.item() == 0
    c.check()
    lat, rope = torch.empty_like(c.lat), torch.empty_like(c.rope)
    kvq.latent_read(c.g, 15, c.pool, c.dtable, i32([0]), i32([300]), i32([0]), 300, lat, rope, c.status)
    assert torch.equal(lat.double(), c.keys(0)[0]) and torch.equal(rope, c.rope)


@FORMATS
def test_same_bits_again_in_a_graph_and_on_a_side_stream(kvq, fmt):
    """Two calls, a captured and replayed one with new queries, and calls on two streams with their
    own workspaces give the same bits."""
    c, d = Absorbed(kvq, fmt, 128, [5000, 300, 1], [1, 1, 1], 66), Absorbed(kvq, fmt, 128, [4000, 3000], [2, 1], 67)
    c.call()
    d.call()
    first, other = c.out.clone(), d.out.clone()
    c.out.fill_(3.0)
    c.call()
    assert torch.equal(c.out, first)
    side, more = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            c.call()
        d.call(stream=more)
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and torch.equal(d.out, other)
    graph, q = torch.cuda.CUDAGraph(), c.ql.clone()
    with torch.cuda.graph(graph):
        c.call()
    c.ql.copy_(torch.flip(q, (0,)))
    c.ws.fill_(0xFF)
    graph.replay()
    c.check()
    c.ql.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and c.status.item() == 0 and d.status.item() == 0


# ------------------------------------------------------------------------------------- expanded
class Expanded:
    def __init__(self, kvq, heads, nqs, prefix, seed, packed=True, scale=1.0, gap=1):
        gen = torch.Generator().manual_seed(seed)
        self.kvq, self.heads, self.nqs = kvq, heads, nqs
        self.nks = [n + p for n, p in zip(nqs, prefix)]
        self.prefix = prefix
        self.off, self.rows = offsets(nqs, gap=gap)
        self.koff, self.krows = offsets(self.nks, gap=gap)
        q = rnd(gen, self.rows, heads, 192, scale=scale).cuda()
        if packed:
            kv = rnd(gen, self.krows, heads, 256).cuda()
            self.kn, self.v = kv[..., :128], kv[..., 128:]
        else:
            self.kn, self.v = (rnd(gen, heads, self.krows, 128).cuda().transpose(0, 1) for _ in range(2))
        self.qn, self.qr, self.kr = q[..., :128], q[..., 128:], rnd(gen, self.krows, 80).cuda()[:, :64]
        used = torch.zeros(self.krows, dtype=torch.bool, device="cuda")
        for o, n in zip(self.koff, self.nks):
            used[o:o + n] = True
        self.kn[~used], self.v[~used], self.kr[~used] = float("nan"), float("inf"), float("nan")
        self.out = torch.full((self.rows, heads, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        self.scale, self.status = 1 / math.sqrt(192), i32([0])
        self.pos, self.n_q, self.q_off = i32(prefix), i32(nqs), i32(self.off)
        self.n_k, self.k_off = i32(self.nks), i32(self.koff)
        self.most, self.most_k = max(nqs), max(self.nks)
        self.ws = torch.full((kvq.latent_prefill_workspace_bytes(len(nqs), heads, self.rows, self.most, self.most_k),),
                             0xFF, dtype=torch.uint8, device="cuda")

    def call(self, **kw):
        self.kvq.latent_prefill_attn(self.pos, self.n_q, self.q_off, self.most, self.n_k, self.k_off, self.most_k,
                                     self.qn, self.qr, self.kn, self.kr, self.v, self.scale, self.ws, self.out,
                                     self.status, **kw)

    def check(self, skip=()):
        mine = torch.zeros(self.rows, dtype=torch.bool)
        for b, (nq, nk) in enumerate(zip(self.nqs, self.nks)):
            if nq == 0 or b in skip:
                continue
            r, kr = slice(self.off[b], self.off[b] + nq), slice(self.koff[b], self.koff[b] + nk)
            mine[r] = True
            q = torch.cat([self.qn[r], self.qr[r]], -1).double().transpose(0, 1)
            k = torch.cat([self.kn[kr], self.kr[kr][:, None].expand(-1, self.heads, -1)], -1).double().transpose(0, 1)
            out, weight, mag = ref.attend(q, k, self.v[kr].double().transpose(0, 1), self.scale, self.prefix[b])
            err = (self.out[r].double().transpose(0, 1) - out).abs()
            tol = ref.tolerance(out, weight, mag, self.scale, 192)
            assert bool((err <= tol).all()), f"lane {b}: {(err / tol).max().item():.3g} of the tolerance"
        assert bool((self.out[~mine.cuda()] == 3.0).all()), "rows of nobody were written"


@pytest.mark.parametrize("heads,nqs,prefix,packed", [
    (1, [1], [0], True), (3, [1, 2, 0, 127, 128, 129], [0, 5, 9, 0, 3, 0], True), (16, [64, 65, 255, 256, 257], [0] * 5, False),
    (8, [1, 1, 1], [0, 1000, 4095], True), (4, [300, 40], [700, 1], False), (128, [33], [0], True), (2, [1000], [0], True),
    (5, [513, 200], [1, 900], False)])
def test_expanded_ragged(kvq, heads, nqs, prefix, packed):
    c = Expanded(kvq, heads, nqs, prefix, 70 + heads, packed)
    c.call()
    assert c.status.item() == 0
    c.check()


@pytest.mark.parametrize("heads,nqs,prefix", [(2, [40], [6000]), (16, [256], [3000]), (1, [2, 130], [9000, 2000])])
def test_expanded_few_rows_over_long_keys(kvq, heads, nqs, prefix):
    c = Expanded(kvq, heads, nqs, prefix, 90 + heads)
    c.call()
    assert c.status.item() == 0
    c.check()


def test_expanded_large_scores(kvq):
    c = Expanded(kvq, 4, [700, 30], [0, 500], 91, scale=12.0)
    c.call()
    assert c.status.item() == 0
    c.check()
    c.scale = 0.0
    c.call()
    c.check()


def test_expanded_rising_maxima(kvq):
    """Scores that rise with the position by hundreds: every tile moves the running maximum."""
    c = Expanded(kvq, 2, [600], [200], 92)
    ramp = torch.linspace(-60, 60, 800, device="cuda")
    u = c.qn[100, 0].double()
    c.kn[c.koff[0]:c.koff[0] + 800] = (ramp[:, None, None] * (u / u.norm())).bfloat16()
    c.qn[c.off[0]:c.off[0] + 600] = (u * 3).bfloat16()
    c.call()
    assert c.status.item() == 0
    c.check()


def test_expanded_refused_lanes(kvq):
    for field, value in (("n_q", -1), ("n_q", 301), ("n_k", -1), ("n_k", 2000), ("pos", -1), ("pos", 101), ("q_off", -1),
                         ("q_off", 500), ("k_off", -1), ("k_off", 900)):
        c = Expanded(kvq, 2, [300, 100, 10], [0, 100, 5], 93)
        getattr(c, field)[1] = value
        c.call()
        assert c.status.item() == kvq.STATUS_BAD_LEN, (field, value)
        c.check(skip=(1,))


def test_expanded_broadcast_heads_and_graph(kvq):
    """Keys and values shared by all heads through a zero head stride; a captured call replayed on
    new values; two streams with their own workspaces; the same bits each time."""
    c, d = Expanded(kvq, 8, [200, 50], [300, 0], 94), Expanded(kvq, 4, [150], [700], 95)
    c.kn = c.kn[:, :1].contiguous().expand(-1, 8, -1)
    c.v = c.v[:, :1].contiguous().expand(-1, 8, -1)
    c.call()
    d.call()
    c.check()
    first, other = c.out.clone(), d.out.clone()
    side, more = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            c.call()
        d.call(stream=more)
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and torch.equal(d.out, other)
    graph, q = torch.cuda.CUDAGraph(), c.qn.clone()
    with torch.cuda.graph(graph):
        c.call()
    c.qn.copy_(torch.flip(q, (0,)))
    c.ws.fill_(0xFF)
    graph.replay()
    c.check()
    c.qn.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and c.status.item() == 0


# ------------------------------------------------------------------------------------- together
@FORMATS
def test_serving_run(kvq, fmt):
    """Two lanes served as a program would: each prompt's latents are appended, read back, expanded
    and attended in the expanded form; a second chunk goes after the prefix; then drafted tokens and
    single tokens go through the absorbed form.  Every step is compared with the 64-bit formulas on
    what the cache holds, and the absorbed output, expanded by the value weights, with the expanded
    form's."""
    gen = torch.Generator().manual_seed(100 + fmt)
    heads, lanes, cap = 16, 2, 640
    table, pages = page_table([cap] * lanes, gen)
    g = kvq.latent_geom(fmt, 1, heads)
    cache = kvq.LatentCache(g, pages, fill=0xFF)
    wk = (torch.randn(heads, 128, 512, generator=gen) / math.sqrt(512)).bfloat16().cuda()   # key expansion
    wv = (torch.randn(heads, 512, 128, generator=gen) / math.sqrt(512)).bfloat16().cuda()   # value expansion
    dt, lens, scale = table.cuda(), [0, 0], 1 / math.sqrt(192)
    for step, (new, form) in enumerate([([200, 77], "expanded"), ([130, 1], "expanded"), ([4, 3], "absorbed"),
                                        ([1, 1], "absorbed"), ([1, 0], "absorbed"), ([1, 1], "both")]):
        off, rows = offsets(new)
        lat, rope = rnd(gen, rows, 512).cuda(), rnd(gen, rows, 64).cuda()
        q = rnd(gen, rows, heads, 192).cuda()
        kvq.latent_append(g, 0, cache.pool, dt, i32(lens), i32(new), i32(off), max(new), lat, rope, cache.status)
        pos, lens = list(lens), [x + y for x, y in zip(lens, new)]
        koff, krows = offsets(lens)
        held, hrope = torch.empty(krows, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(krows, 64, dtype=torch.bfloat16, device="cuda")
        kvq.latent_read(g, 0, cache.pool, dt, i32([0] * lanes), i32(lens), i32(koff), max(lens), held, hrope, cache.status)
        kn = torch.einsum("tc,hdc->thd", held, wk)
        v = torch.einsum("tc,hcd->thd", held, wv)
        q_lat = torch.einsum("rhd,hdc->hrc", q[..., :128], wk).transpose(0, 1)
        got = {}
        if form != "absorbed":
            out = torch.empty(rows, heads, 128, dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(kvq.latent_prefill_workspace_bytes(lanes, heads, rows, max(new), max(lens)), dtype=torch.uint8, device="cuda")
            kvq.latent_prefill_attn(i32(pos), i32(new), i32(off), max(new), i32(lens), i32(koff), max(lens), q[..., :128],
                                    q[..., 128:], kn, hrope, v, scale, ws, out, cache.status)
            got["expanded"] = out
        if form != "expanded":
            out = torch.empty(rows, heads, 512, dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(kvq.latent_workspace_bytes(g, lanes, max(new), max(lens)), dtype=torch.uint8, device="cuda")
            kvq.paged_latent_attn(g, 0, cache.pool, dt, i32(pos), i32(new), i32(off), max(new), i32(lens), max(lens), q_lat,
                                  q[..., 128:], scale, ws, out, cache.status)
            got["absorbed"] = out
        assert cache.read_status() == 0
        for b in range(lanes):
            if not new[b]:
                continue
            r, kr = slice(off[b], off[b] + new[b]), slice(koff[b], koff[b] + lens[b])
            hr = hrope[kr].double()
            if "expanded" in got:
                qq = q[r].double().transpose(0, 1)
                k = torch.cat([kn[kr], hrope[kr][:, None].expand(-1, heads, -1)], -1).double().transpose(0, 1)
                o, w, mag = ref.attend(qq, k, v[kr].double().transpose(0, 1), scale, pos[b])
                assert bool(((got["expanded"][r].double().transpose(0, 1) - o).abs() <= ref.tolerance(o, w, mag, scale, 192)).all()), step
            if "absorbed" in got:
                qq = torch.cat([q_lat[r], q[r][..., 128:]], -1).double().transpose(0, 1)
                k = torch.cat([held[kr].double(), hr], -1)[None]
                o, w, mag = ref.attend(qq, k, held[kr].double()[None], scale, pos[b])
                assert bool(((got["absorbed"][r].double().transpose(0, 1) - o).abs() <= ref.tolerance(o, w, mag, scale, 576)).all()), step
        if form == "both":
            # bf16 roundings of q_lat, k, v and both outputs: a few bf16 steps of values of order one
            a = torch.einsum("rhc,hcd->rhd", got["absorbed"].float(), wv.float())
            assert (a - got["expanded"].float()).norm() <= 0.05 * a.norm()


def test_smallest_calls(kvq):
    """One token, one head, one key; and calls with nothing to do."""
    for fmt in (BF16, MXFP8):
        c = Absorbed(kvq, fmt, 1, [1], [1], 110)
        c.call()
        c.check()
    e = Expanded(kvq, 1, [1], [0], 111)
    e.call()
    e.check()
    before = c.out.clone()
    c.n_q.zero_()
    c.call()
    assert torch.equal(c.out, before) and c.status.item() == 0
    e.n_q.zero_()
    e.out.fill_(3.0)
    e.call()
    assert bool((e.out == 3.0).all()) and e.status.item() == 0


# ------------------------------------------------------------------------------------- further calls
@FORMATS
def test_read_of_many_tokens(kvq, fmt):
    """So many tokens that a warp takes two; odd counts, a short lane, a lane without tokens."""
    gen = torch.Generator().manual_seed(120 + fmt)
    lens = [20000, 19983, 5, 0]
    table, pages = page_table(lens, gen)
    g, status = kvq.latent_geom(fmt, 1, 1), i32([0])
    pool = torch.full((pages * kvq.latent_page_bytes(g),), 0xFF, dtype=torch.uint8, device="cuda")
    off, rows = offsets(lens)
    lat, rope = rnd(gen, rows, 512, scale=2.0).cuda(), rnd(gen, rows, 64).cuda()
    kvq.latent_append(g, 0, pool, table.cuda(), i32([0] * 4), i32(lens), i32(off), max(lens), lat, rope, status)
    lo = [1, 16, 0, 0]
    count = [n - x for n, x in zip(lens, lo)]
    to, out_rows = offsets(count, gap=3)
    got, got_rope = torch.full((out_rows, 512), 7.0).bfloat16().cuda(), torch.full((out_rows, 64), 7.0).bfloat16().cuda()
    kvq.latent_read(g, 0, pool, table.cuda(), i32(lo), i32(count), i32(to), max(count), got, got_rope, status)
    assert status.item() == 0
    want = lat.double() if fmt == BF16 else ref.decode(*ref.encode(lat))
    mine = torch.zeros(out_rows, dtype=torch.bool, device="cuda")
    for b, n in enumerate(count):
        src = slice(off[b] + lo[b], off[b] + lens[b])
        assert torch.equal(got[to[b]:to[b] + n].double(), want[src]) and torch.equal(got_rope[to[b]:to[b] + n], rope[src])
        mine[to[b]:to[b] + n] = True
    assert bool((got[~mine] == 7.0).all()) and bool((got_rope[~mine] == 7.0).all())


@FORMATS
@pytest.mark.parametrize("heads,most", [(16, 1), (128, 1), (24, 3)])
def test_more_lanes_than_ranges(kvq, fmt, heads, most):
    """A batch of 200 ragged lanes, padded with lanes that have no tokens or no queries: borders fall in some
    lanes and not in others, several lanes lie in one range, and one lane spans many."""
    gen = torch.Generator().manual_seed(130)
    lens = torch.randint(0, 900, (200,), generator=gen).tolist()
    lens[3], lens[77], lens[150], lens[199] = 0, 6400, 64, 1
    nqs = [min(n, int(q)) for n, q in zip(lens, torch.randint(0, most + 1, (200,), generator=gen))]
    nqs[77] = most
    c = Absorbed(kvq, fmt, heads, lens, nqs, 131 + heads, head_first=False)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
def test_lanes_share_pages(kvq, fmt):
    """Lanes whose page tables name the same pages (a shared prefix), one lane a page three times over."""
    c = Absorbed(kvq, fmt, 16, [1300, 700, 192], [1, 2, 1], 140)
    src, _ = offsets(c.lens)
    c.dtable[1, :10] = c.dtable[0, :10]
    c.dtable[2, :3] = c.dtable[0, 4]
    for t in (c.lat, c.rope):
        t[src[1]:src[1] + 640] = t[:640].clone()
        t[src[2]:src[2] + 192] = t[256:320].repeat(3, 1)
    # (lane 1's tail once more, with its own values: pages of its own)
    kvq.latent_append(c.g, c.layer, c.pool, c.dtable, i32([0, 640, 0]), i32([0, 60, 0]), i32([0, src[1] + 640, 0]), 60,
                      c.lat, c.rope, c.status)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
def test_two_graphs_share_a_workspace(kvq, fmt):
    """Captured calls of different shapes over one workspace, replayed in turn on one stream."""
    c, d = Absorbed(kvq, fmt, 16, [4000, 30], [1, 1], 150), Absorbed(kvq, fmt, 128, [900, 2500], [3, 1], 151)
    d.ws = c.ws = max((c.ws, d.ws), key=lambda t: t.numel())
    e = Expanded(kvq, 2, [40], [6000], 152)
    e.ws = c.ws if c.ws.numel() >= e.ws.numel() else e.ws
    graphs = []
    for x in (c, d, e):
        x.call()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.call()
    for x in (c, d, e):
        x.out.fill_(3.0)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    for x in (c, d, e):
        assert x.status.item() == 0
        x.check()


def test_expanded_keys_past_the_queries(kvq):
    """A lane may bring keys behind its last query (a padded batch): they may hold anything."""
    for nq, prefix in ((130, 90), (1, 300), (256, 0), (300, 1000)):
        c = Expanded(kvq, 3, [nq], [prefix], 160, gap=70)
        c.n_k += 60                       # the rows behind the lane's own are NaN and infinity
        c.most_k += 60
        c.ws = torch.empty(kvq.latent_prefill_workspace_bytes(1, 3, c.rows, c.most, c.most_k), dtype=torch.uint8, device="cuda")
        c.call()
        assert c.status.item() == 0
        c.check()


def test_binding_refuses_what_the_kernels_cannot_take(kvq):
    c, e = Absorbed(kvq, BF16, 2, [70], [2], 170, head_first=False), Expanded(kvq, 2, [3], [0], 171)
    out, keys = c.out, e.kn
    for bad in (out[:, :1].expand(-1, 2, -1), out[:1].expand(c.rows, -1, -1), out.float(), out.cpu(), out[..., :256]):
        c.out = bad
        with pytest.raises(kvq.KvqError) as err:
            c.call()
        assert err.value.code == kvq.ERR_INVALID_ARG
    c.out = torch.empty(out.numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view_as(out)
    with pytest.raises(kvq.KvqError) as err:
        c.call()
    assert err.value.code == kvq.ERR_ALIGNMENT
    e.kn = keys[:1].expand(e.krows, -1, -1)
    with pytest.raises(kvq.KvqError) as err:
        e.call()
    assert err.value.code == kvq.ERR_UNSUPPORTED
    c.out, e.kn = out, keys
    c.call()
    e.call()
    c.check()
    e.check()


@FORMATS
def test_capture_behind_joined_streams(kvq, fmt):
    """Captured calls whose inputs come from another captured stream, right behind one another and behind a
    copy: each sees what was written before it."""
    c, d = Absorbed(kvq, fmt, 16, [3000, 50], [1, 1], 180), Absorbed(kvq, fmt, 16, [100], [1], 181)
    for x in (c, d):
        x.call()
    torch.cuda.synchronize()
    q, lat = c.ql.clone(), d.lat.clone()
    side, main, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            c.ql.copy_(q)
            kvq.latent_append(d.g, d.layer, d.pool, d.dtable, i32_like(d, 0), d.seq_len, i32_like(d, 0), 100, lat, d.rope, d.status)
        c.out.fill_(3.0)
        main.wait_stream(side)
        c.call()
        d.call()
        c.call()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            d.call()
        main.wait_stream(side)
    for _ in range(3):
        c.ql.zero_()
        d.pool.fill_(0)
        d.out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
    torch.cuda.synchronize()
    assert c.status.item() == 0 and d.status.item() == 0
    c.check()
    d.check()


def i32_like(c, value):
    return torch.full_like(c.seq_len, value)


@pytest.mark.parametrize("heads,nqs,prefix", [(80, [100], [6000]), (20, [260, 3], [6000, 100]), (40, [1, 200], [5600, 6000])])
def test_expanded_tails_on_the_free_sms(kvq, heads, nqs, prefix):
    """CTAs for more than half of the SMs behind a long prefix: the last key tiles of each are split off."""
    c = Expanded(kvq, heads, nqs, prefix, 190 + heads)
    assert c.ws.numel() > 256
    c.call()
    assert c.status.item() == 0
    c.check()


def far_below(c, b):
    """Gives lane b keys whose scores are all near -600 (in powers of two): any reference above them loses all."""
    first, n = offsets(c.lens)[0][b], c.lens[b]
    u = torch.randn(512, generator=torch.Generator().manual_seed(7)).double().cuda()
    u /= u.norm()
    c.lat[first:first + n] = (c.lat[first:first + n].double() * 0.25 - 40 * u).bfloat16()
    c.ql[c.off[b]:c.off[b] + c.nqs[b]] += (144 * u).bfloat16()
    c.kvq.latent_append(c.g, c.layer, c.pool, c.dtable, i32([0] * len(c.lens)), i32(c.lens), i32(offsets(c.lens)[0]),
                        max(c.lens), c.lat, c.rope, c.status)


@FORMATS
@pytest.mark.parametrize("heads", [16, 32, 128])
def test_low_scores_behind_pages_outside_the_pool(kvq, fmt, heads):
    """The first pages of a lane are not in the pool and the scores of the others lie far below zero."""
    c = Absorbed(kvq, fmt, heads, [300, 130], [1, 1], 200 + heads)
    far_below(c, 0)
    c.dtable[0, :2] = -1
    c.call()
    assert c.status.item() == kvq.STATUS_PAGE_OOB
    lat, rope = c.keys(0)
    q = torch.cat([c.ql[c.off[0]:c.off[0] + 1], c.qr[c.off[0]:c.off[0] + 1]], -1).double().transpose(0, 1)
    out, weight, mag = ref.attend(q, torch.cat([lat, rope], 1)[None, 128:], lat[None, 128:], c.scale, 10 ** 6)
    err = (c.out[c.off[0]:c.off[0] + 1].double().transpose(0, 1) - out).abs()
    assert bool((err <= ref.tolerance(out, weight, mag, c.scale, 576)).all())
    c.out[c.off[0]] = 3.0
    c.check(skip=(0,))


@FORMATS
@pytest.mark.parametrize("heads,nq", [(16, 8), (5, 9), (128, 8)])
def test_parts_without_keys_for_some_rows(kvq, fmt, heads, nq):
    """Ranges of four pages: the last part of lane 0 holds keys for its later queries only, with scores far below
    zero, so that an empty part's reference must not count."""
    c = Absorbed(kvq, fmt, heads, [262, 700, 519], [nq, 1, nq], 210 + heads)
    for b in (0, 2):
        far_below(c, b)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
def test_calls_right_behind_one_another(kvq, fmt):
    """Calls that rewrite what the call before read, with nothing between them: each starts while the one before
    ends, and the bits are those of calls with a wait between."""
    c = Absorbed(kvq, fmt, 16, [5000, 70], [1, 1], 220)
    off, rows = offsets(c.lens)
    values = [(c.lat, c.rope), (torch.flip(c.lat, (0,)).contiguous(), torch.flip(c.rope, (0,)).contiguous())]
    back = torch.empty_like(c.lat), torch.empty_like(c.rope)

    def step(v):
        kvq.latent_append(c.g, c.layer, c.pool, c.dtable, i32_zero, c.seq_len, i32_off, 5000, *values[v], c.status)
        c.call()
        kvq.latent_read(c.g, c.layer, c.pool, c.dtable, i32_zero, c.seq_len, i32_off, 5000, *back, c.status)

    i32_zero, i32_off, want = i32([0, 0]), i32(off), []
    for v in (0, 1):
        step(v)
        torch.cuda.synchronize()
        want.append((c.out.clone(), back[0].clone(), back[1].clone()))
    assert not torch.equal(want[0][0], want[1][0])
    got = []
    for i in range(12):
        step(i & 1)
        got.append((c.out.clone(), back[0].clone(), back[1].clone()))
        step(1 - (i & 1))
    torch.cuda.synchronize()
    assert c.status.item() == 0
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i & 1])), i
    assert torch.equal(back[1], values[0][1][:rows]) and torch.equal(c.out, want[0][0])


@pytest.mark.parametrize("heads,nqs,prefix", [(20, [1024], [4500]), (27, [721], [5000])])
def test_expanded_two_splits_of_many_rows(kvq, heads, nqs, prefix):
    """The merge that takes several rows a warp: odd counts of rows and heads."""
    c = Expanded(kvq, heads, nqs, prefix, 230 + heads)
    assert c.ws.numel() > 256 and c.most * heads >= 2 * 64 * 152
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
@pytest.mark.parametrize("heads", [16, 128])
def test_one_workspace_for_all_calls_of_a_server(kvq, fmt, heads):
    """A workspace sized for the largest call (chunks of up to 64 queries, 16 lanes, 8,192 tokens) serves single
    tokens, drafted tokens and chunks, and nothing behind it is touched."""
    size = kvq.latent_workspace_bytes(kvq.latent_geom(fmt, 2, heads), 16, 64, 8192)
    whole = torch.full((size + 65536,), 0xEE, dtype=torch.uint8, device="cuda")
    for lens, nqs in (([8192, 100], [1, 1]), ([3000, 2000, 700], [4, 1, 2]), ([1500, 700], [30, 1]), ([900, 300], [64, 1]),
                      ([700 + 13 * i for i in range(16)], [1] * 16)):
        c = Absorbed(kvq, fmt, heads, lens, nqs, 240 + heads, head_first=False)
        c.ws = whole[:size]
        c.call()
        assert c.status.item() == 0
        c.check()
    assert bool((whole[size:] == 0xEE).all())


def test_one_workspace_for_all_expanded_calls_of_a_server(kvq):
    """A workspace sized for the largest call (8 lanes, 32 heads, chunks of 2,048 over 16,000 keys) serves every smaller
    one, also from rows in the middle of large buffers, and nothing behind it is touched."""
    size = kvq.latent_prefill_workspace_bytes(8, 32, 16384, 2048, 16000)
    whole = torch.full((size + 65536,), 0xEE, dtype=torch.uint8, device="cuda")
    for heads, nqs, prefix, gap in ((32, [256], [3000], 1), (20, [1024], [4500], 3), (16, [40, 1], [2500, 2100], 3000),
                                    (4, [300, 7, 256], [2000, 2300, 0], 700), (2, [130] * 8, [2100] * 8, 1), (32, [2048], [0], 1)):
        c = Expanded(kvq, heads, nqs, prefix, 250 + heads, gap=gap)
        c.ws = whole[:size]
        c.call()
        assert c.status.item() == 0
        c.check()
    assert bool((whole[size:] == 0xEE).all())


@pytest.mark.parametrize("heads,nqs,prefix", [(2, [40, 300], [6000, 3000]), (20, [260, 3], [6000, 100]), (1, [9, 257], [2500, 2000])])
def test_expanded_parts_stay_in_their_workspace(kvq, heads, nqs, prefix):
    """The bytes that this very call needs, with a guard behind them."""
    c = Expanded(kvq, heads, nqs, prefix, 260 + heads, gap=900)
    tiles, ctas = -(-c.most_k // 128), len(nqs) * heads * -(-c.most // 256)
    splits = 2 if 2 * ctas > 152 else -(-tiles // max(8, -(-tiles // (152 // ctas))))
    size = len(nqs) * c.most * heads * splits * 130 * 4 + 256
    assert size <= c.ws.numel()
    whole = torch.full((size + 65536,), 0xEE, dtype=torch.uint8, device="cuda")
    c.ws = whole[:size]
    c.call()
    assert c.status.item() == 0 and bool((whole[size:] == 0xEE).all())
    c.check()


@FORMATS
@pytest.mark.parametrize("value", [3, -1])
def test_lanes_beside_a_refused_count_are_answered(kvq, fmt, value):
    """A lane with a bad count of queries is skipped: the other lanes are answered and its own rows left as they were."""
    for lens in ([100, 200, 300, 64], [100, 900, 3000, 64]):
        c = Absorbed(kvq, fmt, 16, lens, [1, 2, 1, 1], 270)
        c.n_q[1] = value
        c.call()
        assert c.status.item() == kvq.STATUS_BAD_LEN
        c.check(skip=(1,))


@FORMATS
@pytest.mark.parametrize("heads,lens,nqs", [(128, [1500, 700], [30, 1]), (128, [1500, 700], [40, 1]), (128, [2000, 5], [38, 3]),
                                            (128, [700, 1300, 90], [12, 26, 2]), (100, [3000], [33]), (16, [1400, 600], [120, 304]),
                                            (24, [900, 2500, 1], [70, 11, 1]), (128, [2600, 90], [10, 2]), (128, [1700], [25])])
def test_chunks_of_many_row_tiles(kvq, fmt, heads, lens, nqs):
    """Chunks whose rows take 20 to 80 tiles: few ranges of the page list (7, 5, 3 or 2) with a merge, and, above 76 tiles,
    long lanes in one piece."""
    c = Absorbed(kvq, fmt, heads, lens, nqs, 280 + heads, head_first=False)
    c.call()
    assert c.status.item() == 0
    c.check()


@FORMATS
def test_inputs_that_share_rows_or_heads(kvq, fmt):
    """Queries, latents and rotary keys broadcast through zero strides."""
    c = Absorbed(kvq, fmt, 16, [700, 90], [3, 1], 290, head_first=False)
    c.ql = c.ql[:1].contiguous().expand(c.rows, -1, -1)
    c.qr = c.qr[:, :1].contiguous().expand(-1, 16, -1)
    c.lat, c.rope = c.lat[:1].expand(790, -1), c.rope[5:6].expand(790, -1)
    kvq.latent_append(c.g, c.layer, c.pool, c.dtable, i32([0, 0]), c.seq_len, i32([0, 700]), 700, c.lat, c.rope, c.status)
    c.call()
    assert c.status.item() == 0
    c.check()
