"""The paged cache operators on the GPU against plain 64-bit forms.

Pools start full of what must never matter (NaN in 16-bit and e4m3 pages and
in scales, random codes in int8 ones); only the positions a sequence holds
are finite.  Row buffers have rows behind the last sequence, which must stay
as they were.
"""
import math

import numpy as np
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FORMATS = ("f16", "bf16", "int8", "e4m3")
TORCH = {"f32": "float32", "f16": "float16", "bf16": "bfloat16", "int8": "int8", "e4m3": "float8_e4m3fn"}
LARGEST = {"int8": 127.0, "e4m3": 448.0}


def dt(name):
    return getattr(torch, TORCH[name])


@pytest.fixture(scope="module")
def q2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import qwen2_decoder_forward_gb300 as m
    from qwen2_decoder_forward_gb300 import build
    build.build()
    return m


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def coded(x, kind):
    """(codes as floats, scale) of 64-bit heads x, by the format's definition."""
    largest = x.abs().amax(-1, keepdim=True)
    scale = torch.where(largest == 0, torch.ones_like(largest), largest / LARGEST[kind])
    y = x / scale
    if kind == "e4m3":
        return y.float().to(torch.float8_e4m3fn).double(), scale
    return torch.sign(y) * torch.floor(y.abs() + 0.5), scale


class Case:
    """A batch of sequences given as (rows, cached positions) pairs."""

    def __init__(self, q2, seqs, heads, fmt, page, layout="head", seed=0, spare_rows=3, before=0):
        self.q2, self.seqs, self.fmt, self.page = q2, seqs, fmt, page
        self.nh, self.nkv, self.hd = heads
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-kv // page) for _, kv in seqs]
        n_pages = before + sum(need) + 2      # `before`: pages in front that nothing uses
        order = before + torch.randperm(n_pages - before, generator=g, device="cuda").to(torch.int32)
        self.width = max(need) + 1
        pages = torch.full((len(seqs), self.width), -7, dtype=torch.int32, device="cuda")   # unused entries: bad ids
        at = 0
        for s, n in enumerate(need):
            pages[s, :n] = order[at:at + n]
            at += n
        starts = np.concatenate([[0], np.cumsum([n for n, _ in seqs])])
        self.starts, self.rows = [int(x) for x in starts], int(starts[-1]) + spare_rows
        self.live = int(starts[-1])
        self.pages = pages
        self.batch = q2.PagedBatch(torch.tensor(self.starts, dtype=torch.int32, device="cuda"),
                                   torch.tensor([kv for _, kv in seqs], dtype=torch.int32, device="cuda"), pages,
                                   max(1, max(n for n, _ in seqs)))
        self.quant = fmt in LARGEST
        base = torch.int8 if self.quant else dt(fmt)
        if layout == "head":       # [page][head][token]
            raw = torch.empty((2, n_pages, self.nkv, page, self.hd), dtype=base, device="cuda").permute(0, 1, 3, 2, 4)
        elif layout == "token":    # [page][token][head]
            raw = torch.empty((2, n_pages, page, self.nkv, self.hd), dtype=base, device="cuda")
        else:                      # K and V of a page side by side, heads padded
            pad = 16 if self.quant else 8
            raw = torch.empty((n_pages, 2, page, self.nkv, self.hd + pad), dtype=base, device="cuda")[..., :self.hd]
            raw = raw.permute(1, 0, 2, 3, 4)
        if self.quant:
            raw.copy_(torch.randint(-128, 128, raw.shape, generator=g, device="cuda").to(torch.int8))
            if fmt == "e4m3":
                raw.fill_(127)     # NaN
            ks, vs = (torch.full((n_pages, self.nkv, page), math.nan, device="cuda") for _ in range(2))
            self.kv = q2.PagedKV(raw[0].view(dt(fmt)), raw[1].view(dt(fmt)), ks, vs)
        else:
            raw.fill_(math.nan)
            self.kv = q2.PagedKV(raw[0], raw[1])

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float64)

    def fill(self, spread=1.0):
        """Puts random K and V at every sequence's positions; returns their
        exact 64-bit values per sequence."""
        held = []
        for s, (_, kv) in enumerate(self.seqs):
            values = []
            for which in range(2):
                x = self.normal(kv, self.nkv, self.hd) * (torch.exp(spread * self.normal(kv, self.nkv, 1)) if spread else 1)
                pos = torch.arange(kv, device="cuda")
                pg, off = self.pages[s][pos // self.page].long(), pos % self.page
                pool, scales = ((self.kv.k, self.kv.k_scale), (self.kv.v, self.kv.v_scale))[which]
                if self.quant:
                    codes, scale = coded(x, self.fmt)
                    scale = scale.float()
                    scales[pg, :, off] = scale[..., 0]
                    pool.view(torch.int8)[pg, off] = (codes.to(torch.int8) if self.fmt == "int8" else
                                                      codes.float().to(torch.float8_e4m3fn).view(torch.int8))
                    values.append((codes * scale.double(), codes, scale.double()))
                else:
                    pool[pg, off] = x.to(pool.dtype)
                    values.append((x.to(pool.dtype).double(), None, None))
            held.append(values)
        return held

    def queries(self, dtype, gain=1.0):
        q = (gain * self.normal(self.rows, self.nh, self.hd)).to(dtype)
        return q


def check_attention(c, q, held, o, lse, scale, causal, out_fill):
    """|o - exact| by arithmetic: with A = sum w |v| / sum w,
      * each probability is rounded to the product's 16-bit type, q's own (f16 over 8-bit pages where a sequence
        has at most 32 rows of a kv head's group): A u_P;
      * a score's error d (f32 products of hd terms, its scaling and the
        exponential's 2^-22) turns into a factor 1 +- 2 d on weights: 4 d A
        over numerator and denominator;
      * a probability below the smallest normal 16-bit number is off by half
        a subnormal step (f16: 2^-25) times |v| (8-bit: times the largest
        scale, rounded up to a power of two, times the code);
      * the output's own rounding u_o |o|."""
    few = c.batch.max_q * (c.nh // c.nkv) <= 32
    p_type = torch.float16 if q.dtype == torch.float16 or (c.quant and few) else torch.bfloat16
    sub = 2.0 ** -25 if p_type == torch.float16 else 2.0 ** -134
    for s, (n, kv) in enumerate(c.seqs):
        if n == 0:
            continue
        rows = slice(c.starts[s], c.starts[s] + n)
        (k, _, _), (v, codes, vscale) = held[s]
        for h in range(c.nh):
            hk = h * c.nkv // c.nh
            qq, kk, vv = q[rows, h].double(), k[:, hk], v[:, hk]
            if kv == 0:
                assert (o[rows, h] == 0).all()
                if lse is not None:
                    assert (lse[rows, h] == -math.inf).all()
                continue
            sc = qq @ kk.T * scale
            if causal:
                late = torch.arange(kv, device="cuda")[None] > torch.arange(n, device="cuda")[:, None] + (kv - n)
                sc = sc.masked_fill(late, -math.inf)
            top = sc.amax(-1, keepdim=True)
            empty = torch.isinf(top[:, 0])
            w = torch.exp(sc - torch.where(torch.isinf(top), 0.0, top))
            total = w.sum(-1, keepdim=True)
            safe = torch.where(total == 0, 1.0, total)
            ref = (w @ vv) / safe
            a = (w @ vv.abs()) / safe
            mag = (qq.abs() @ kk.abs().T * abs(scale)).amax(-1, keepdim=True)
            d = c.hd * 2.0 ** -23 * mag + 2.0 ** -20
            tiny = sub / safe * (vv.abs().sum(0)[None] if not c.quant else
                                 2 * vscale[:, hk].max() * codes[:, hk].abs().sum(0)[None])
            bound = a * (half_step(p_type) + 4 * d) + tiny + half_step(q.dtype) * ref.abs() + 2.0 ** -24
            got = o[rows, h].double()
            err = (got - ref).abs()
            assert bool((err <= bound).all()), (
                f"sequence {s} (rows {n}, kv {kv}) head {h}: worst {float((err / bound).max()):.2f} of the bound, "
                f"error {float(err.max()):.3e}")
            assert bool((got[empty] == 0).all())
            if lse is not None:
                want = top[:, 0] + torch.log(total[:, 0])
                got_l = lse[rows, h].double()
                assert bool((got_l[empty] == -math.inf).all())
                e = (got_l - want)[~empty].abs()
                lim = (2 * d[:, 0] + 2.0 ** -22 * want.abs() + 2.0 ** -20)[~empty]
                assert bool((e <= lim).all()), f"lse off by {float(e.max()):.3e}"
    assert bool((o[c.live:] == out_fill).all()), "rows behind the last sequence were written"


HEADS = [(14, 2, 64), (4, 4, 64), (28, 4, 128), (8, 1, 128), (16, 1, 64), (6, 2, 128)]
MIXES = {
    "tokens": [(1, 1), (1, 15), (1, 16), (1, 17), (1, 64), (1, 65), (1, 300), (1, 1111), (0, 40), (1, 128)],
    "few": [(3, 3), (5, 70), (2, 500), (8, 130), (4, 0), (7, 3), (0, 0), (1, 63)],
    "chunks": [(37, 37), (64, 301), (1, 90), (130, 131), (20, 1000)],
    "prompt": [(419, 419)],
    "long": [(1, 5000)],
    "big chunk": [(300, 1800), (3, 1000)],
}


def run_attention(c, dtype, causal=True, scale=None, gain=1.0, spread=0.5, lse=True):
    held = c.fill(spread)
    q = c.queries(dtype, gain)
    out = torch.full((c.rows, c.nh, c.hd), 7.0, dtype=dtype, device="cuda")
    r = c.q2.paged_attention(c.kv, c.batch, q, out=out, scale=scale, causal=causal, return_lse=lse)
    c.batch.check()
    o, l = r if lse else (r, None)
    assert o is out
    check_attention(c, q, held, o, l, c.hd ** -0.5 if scale is None else scale, causal, 7.0)
    return o


@pytest.mark.parametrize("mix", list(MIXES))
@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "f16"), ("int8", "bf16"),
                                       ("e4m3", "f16"), ("e4m3", "bf16")])
def test_attention_matches_the_formula(q2, mix, fmt, dtype):
    for i, heads in enumerate(HEADS):
        c = Case(q2, MIXES[mix], heads, fmt, (16, 32, 64, 128, 256)[i % 5], ("head", "token", "padded")[i % 3], seed=i)
        run_attention(c, dt(dtype), causal=not (mix == "chunks" and i % 2))


def test_attention_to_another_sequences_states(q2):
    """Causal off: rows see all kv_len positions, more rows than positions included."""
    for heads in HEADS[:3]:
        c = Case(q2, [(9, 4), (3, 200), (150, 77), (1, 0), (40, 1)], heads, "bf16", 32, seed=3)
        run_attention(c, torch.bfloat16, causal=False)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_attention_with_other_scales(q2, scale):
    for seqs in ([(2, 90), (1, 33)], [(200, 700)]):
        run_attention(Case(q2, seqs, (14, 2, 64), "f16", 16, seed=5), torch.float16, scale=scale)


def test_sharp_and_large_scores(q2):
    """Scores in the hundreds: the running maximum moves and most weights vanish."""
    for seqs in ([(1, 700), (3, 200)], [(260, 900)]):
        for fmt in ("f16", "int8"):
            run_attention(Case(q2, seqs, (8, 2, 128), fmt, 64, seed=6), torch.float16, gain=30.0, spread=0.0)


def test_growing_scores_move_the_maximum_every_tile(q2):
    """Keys that grow along the sequence: each tile's maximum is above the last one's by more than a rescale
    threshold could hide."""
    for n in (1, 300):
        c = Case(q2, [(n, 1500)], (8, 2, 64), "bf16", 32, seed=7)
        held = c.fill(0.0)
        ramp = torch.linspace(0, 40, 1500, device="cuda", dtype=torch.float64)[:, None, None]
        k = ramp.expand(1500, c.nkv, c.hd).to(torch.bfloat16)
        pos = torch.arange(1500, device="cuda")
        c.kv.k[c.pages[0][pos // 32].long(), pos % 32] = k
        held[0][0] = (k.double(), None, None)
        q = c.queries(torch.bfloat16).abs()
        out = torch.full_like(q, 7.0)
        _, lse = q2.paged_attention(c.kv, c.batch, q, out=out, return_lse=True)
        c.batch.check()
        check_attention(c, q, held, out, lse, c.hd ** -0.5, True, 7.0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scales_that_span_many_powers_of_two(q2, fmt):
    """v scales from 2^-20 to 2^10 in one sequence, zero heads among them (scale 1, codes 0)."""
    for n in (1, 200):
        c = Case(q2, [(n, 900)], (8, 2, 128), fmt, 64, seed=8)
        held = c.fill(0.0)
        pos = torch.arange(900, device="cuda")
        pg, off = c.pages[0][pos // 64].long(), pos % 64
        sc = 2.0 ** torch.randint(-20, 11, (900, c.nkv), generator=c.g, device="cuda").double()
        zero = torch.rand(900, c.nkv, generator=c.g, device="cuda") < 0.1
        sc[zero] = 1.0
        codes = held[0][1][1] * (~zero)[..., None]
        c.kv.v_scale[pg, :, off] = sc.float()
        raw = codes.to(torch.int8) if fmt == "int8" else codes.float().to(torch.float8_e4m3fn).view(torch.int8)
        c.kv.v.view(torch.int8)[pg, off] = raw
        held[0][1] = (codes * sc[..., None], codes, sc[..., None])
        q = c.queries(torch.bfloat16)
        out = torch.full_like(q, 7.0)
        q2.paged_attention(c.kv, c.batch, q, out=out)
        c.batch.check()
        check_attention(c, q, held, out, None, c.hd ** -0.5, True, 7.0)


def test_attention_is_repeatable_and_other_streams_agree(q2):
    c = Case(q2, MIXES["chunks"] + MIXES["tokens"], (14, 2, 64), "f16", 32, seed=9)
    c.fill()
    q = c.queries(torch.float16)
    first = q2.paged_attention(c.kv, c.batch, q)[:c.live].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [q2.paged_attention(c.kv, c.batch, q) for _ in range(3)]
    other = q2.paged_attention(c.kv, c.batch, q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for o in again + [other]:
        assert torch.equal(o[:c.live], first)


def test_strided_queries_and_outputs(q2):
    """q as a slice of fused projection rows, out as a slice of a wider buffer."""
    c = Case(q2, MIXES["few"], (14, 2, 64), "bf16", 16, seed=10)
    held = c.fill()
    fused = torch.randn((c.rows, 14 + 4, 64), generator=c.g, device="cuda").to(torch.bfloat16)
    wide = torch.full((c.rows, 15, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    q, out = fused[:, 2:16], wide[:, 1:, :64]
    q2.paged_attention(c.kv, c.batch, q, out=out)
    c.batch.check()
    check_attention(c, q, held, out, None, 0.125, True, 7.0)
    assert (wide[:, 0] == 7).all() and (wide[..., 64:] == 7).all()


def test_graph_replays_read_lengths_and_pages_anew(q2):
    """A decode step (write, attention) captured once; replays follow lengths and pages changed in place."""
    c = Case(q2, [(1, 200), (1, 77), (1, 31)], (14, 2, 64), "int8", 16, seed=11, spare_rows=0)
    c.fill(0.0)
    table = torch.from_numpy(q2.rope_table(512, 64)).cuda()
    x = c.normal(3, 18, 64).float()

    def step():
        q = q2.paged_write(c.kv, c.batch, x[:, 14:16], x[:, 16:], q=x[:, :14], rope=table)
        return q2.paged_attention(c.kv, c.batch, q)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    spare = [i for i in range(c.kv.n_pages) if not (c.pages == i).any()]
    for lens in ([200, 77, 31], [199, 78, 32], [150, 79, 33], [3, 1, 17]):
        x.copy_(c.normal(3, 18, 64))
        c.batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        if lens[2] == 33:
            c.pages[2, 2] = spare[0]          # sequence 2 grows into a new page
        graph.replay()
        captured = out.clone()
        assert torch.equal(captured, step())  # the same call outside the graph
    c.batch.check()


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 65, 127, 129])
def test_row_counts_around_the_tiles(q2, n, fmt, dtype):
    """As many packed rows as a tile has, one fewer and one more, for one query head a kv head."""
    c = Case(q2, [(n, n), (n, 200), (max(n - 1, 0), 333), (1, 65)], (2, 2, 128), fmt, 64, seed=20 + n)
    run_attention(c, dt(dtype))


@pytest.mark.parametrize("heads", [(64, 1, 64), (64, 1, 128), (33, 3, 64), (80, 2, 64)])
def test_wide_groups(q2, heads):
    for fmt, dtype in (("f16", "f16"), ("int8", "bf16")):
        run_attention(Case(q2, [(1, 100), (1, 700), (0, 3)], heads, fmt, 32, seed=21), dt(dtype))
        run_attention(Case(q2, [(5, 70), (40, 40), (1, 9)], heads, fmt, 32, seed=22), dt(dtype))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("int8", "f16"), ("e4m3", "bf16")])
def test_page_sizes_of_both_kernels(q2, page, fmt, dtype):
    for i, layout in enumerate(("head", "token", "padded")):
        seqs = [(150, 700), (1, 257), (1, 256), (90, 90)]
        run_attention(Case(q2, seqs, (14, 2, 64), fmt, page, layout, seed=23 + i), dt(dtype))
        run_attention(Case(q2, [(1, 257), (1, 16), (1, 255)], (14, 2, 64), fmt, page, layout, seed=26 + i), dt(dtype))


@pytest.mark.parametrize("n_seq", [31, 32, 33, 64, 65, 100, 1025, 4096])
def test_many_sequences(q2, n_seq):
    """Work lists of more sequences than a warp takes at a time; some hold no rows, and with `long` some have
    several causal tiles."""
    for long in (False, True):
        lens = np.random.default_rng(n_seq).integers(1, 40, n_seq)
        seqs = [(int(i % 5 != 3), int(x)) for i, x in enumerate(lens)]
        if long:
            for i in range(0, n_seq, 1 + n_seq // 7):
                seqs[i] = (70 + i % 3 * 40, 150)
        run_attention(Case(q2, seqs, (2, 1, 64), "f16", 16, seed=n_seq), torch.float16)


def test_other_rows_that_are_not_finite(q2):
    """NaN and infinite queries of one sequence and behind the last one reach no other sequence's rows."""
    for seqs in ([(1, 90), (1, 200), (2, 64)], [(100, 400), (130, 130), (70, 300), (1, 90)]):
        c = Case(q2, seqs, (14, 2, 64), "f16", 32, seed=28)
        c.fill()
        q = c.queries(torch.float16)
        want = q2.paged_attention(c.kv, c.batch, q)[:c.live].clone()
        q[c.starts[1]:c.starts[2]] = math.nan
        q[c.starts[1]] = math.inf
        q[c.live:] = math.nan
        got = q2.paged_attention(c.kv, c.batch, q)[:c.live]
        for s in range(len(seqs)):
            if s != 1:
                rows = slice(c.starts[s], c.starts[s + 1])
                assert torch.equal(got[rows], want[rows])


@pytest.mark.parametrize("n", [1, 3, 7, 200])
def test_scales_that_grow_with_rows_of_every_tile(q2, n):
    """v scales that double every 60 positions move G again and again, for each form of the row tiles."""
    c = Case(q2, [(n, 900)], (8, 2, 128), "int8", 64, seed=29)
    held = c.fill(0.0)
    pos = torch.arange(900, device="cuda")
    pg, off = c.pages[0][pos // 64].long(), pos % 64
    sc = (2.0 ** (pos // 60).double() * 1e-3)[:, None].expand(900, c.nkv).float()
    c.kv.v_scale[pg, :, off] = sc
    codes = held[0][1][1]
    held[0][1] = (codes * sc.double()[..., None], codes, sc.double()[..., None])
    q = c.queries(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    q2.paged_attention(c.kv, c.batch, q, out=out)
    c.batch.check()
    check_attention(c, q, held, out, None, c.hd ** -0.5, True, 7.0)


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("int8", "bf16")])
def test_pages_beyond_four_gigabytes(q2, fmt, dtype):
    """Every page in use lies more than 2^32 elements into the pool."""
    before = (1 << 32) // (256 * 4 * 128) + 1
    for seqs in ([(1, 700), (1, 30)], [(150, 600), (1, 40)]):
        c = Case(q2, seqs, (8, 4, 128), fmt, 256, "token", seed=31, before=before)
        run_attention(c, dt(dtype))
        k, v = (c.normal(c.rows, 4, 128).to(dt(dtype)) for _ in range(2))
        q2.paged_write(c.kv, c.batch, k, v)
        n = sum(kv for _, kv in seqs)
        starts = torch.tensor([0] + list(np.cumsum([kv for _, kv in seqs])), dtype=torch.int32, device="cuda")
        gk, gv = q2.paged_read(c.kv, c.batch, starts, n)
        c.batch.check()
        for s, (rows, kv) in enumerate(seqs):
            last = slice(int(starts[s]) + kv - rows, int(starts[s]) + kv)
            for got, x in ((gk, k), (gv, v)):
                x = x[c.starts[s]:c.starts[s] + rows].double()
                # f16 holds it exactly; int8 is off by half a code and f32's roundings of scale and product.
                off = 0 if fmt == "f16" else x.abs().amax(-1, keepdim=True) / 127 * (0.5 + 2.0 ** -15)
                assert bool(((got[last].double() - x).abs() <= off).all())
        del c, k, v, gk, gv
        torch.cuda.empty_cache()


def test_threads_and_graphs_at_the_same_time(q2):
    """Two threads share a pool and a batch on streams of their own with different row buffers; two graphs of
    the same call are replayed side by side."""
    import threading
    c = Case(q2, MIXES["chunks"] + MIXES["tokens"], (14, 2, 64), "int8", 32, seed=30)
    c.fill()
    q = c.queries(torch.float16)
    qs = [q, torch.cat([q, q[:9]])]
    want = [q2.paged_attention(c.kv, c.batch, x)[:c.live].clone() for x in qs]
    assert torch.equal(want[0], want[1])
    torch.cuda.synchronize()
    bad = []

    def work(i, own):
        try:
            stream = torch.cuda.Stream() if own else None
            for _ in range(40):
                o = q2.paged_attention(c.kv, c.batch, qs[i], stream=stream)
                (stream or torch.cuda.current_stream()).synchronize()
                if o.shape != qs[i].shape or not torch.equal(o[:c.live], want[0]):
                    bad.append(i)
        except Exception as e:      # noqa: BLE001
            bad.append(e)
    for own in (True, False):       # streams of their own, then one stream
        threads = [threading.Thread(target=work, args=(i, own)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(q2.paged_attention(c.kv, c.batch, q))
        graphs.append(g)
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[:c.live], want[0])
    c.batch.check()


# ---- the write and the read ---------------------------------------------------------------


def written(c, x, norm, table, interleaved, first):
    """64-bit rows after the norm and the rotation."""
    x = x.double()
    if norm is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * norm.double()
    if table is None:
        return x
    t = table[first:first + x.shape[0]].double()
    half = t.shape[1]
    cs, sn = t[:, None, :, 0], t[:, None, :, 1]
    out = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out[..., a] = x[..., a] * cs - x[..., b] * sn
    out[..., b] = x[..., b] * cs + x[..., a] * sn
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_write_then_read(q2, fmt, x):
    """Every option over ragged batches; f32 arithmetic, then one rounding."""
    combos = [(None, None, False), (64, None, False), (32, "norm", True), (16, "norm", False), (128, None, True),
              (None, "norm", False)]
    for i, heads in enumerate(HEADS):
        rotary, norm, inter = combos[i]
        if rotary and rotary > heads[2]:
            rotary = heads[2]
        seqs = [(1, 1), (5, 40), (0, 3), (33, 33), (1, 500), (17, 16)]     # the last one's first row has no position
        c = Case(q2, seqs, heads, fmt, (16, 64, 256)[i % 3], ("head", "token", "padded")[i % 3], seed=20 + i)
        held = c.fill(0.3)
        rows = torch.randn((c.rows, c.nh + 2 * c.nkv, c.hd), generator=c.g, device="cuda").to(dt(x))
        rows[2, c.nh:] = 0                                                  # a head of zeros: scale 1
        q, k, v = rows[:, :c.nh], rows[:, c.nh:c.nh + c.nkv], rows[:, c.nh + c.nkv:]
        qn, kn = (1 + 0.1 * torch.randn(c.hd, generator=c.g, device="cuda") for _ in range(2)) if norm else (None, None)
        table = torch.from_numpy(q2.rope_table(600, rotary)).cuda() if rotary else None
        out_type = torch.bfloat16 if fmt == "bf16" else torch.float16
        q_out = torch.full((c.rows, c.nh, c.hd), 7.0, dtype=out_type, device="cuda")
        got = q2.paged_write(c.kv, c.batch, k, v, q=q, q_out=q_out, q_norm=qn, k_norm=kn, rope=table, interleaved=inter)
        assert got is q_out and (q_out[c.live:] == 7).all()
        with pytest.raises(q2.Qwen2Error) as e:                             # (17, 16): position -1
            c.batch.check()
        assert e.value.code == q2.QWEN2_E_DEVICE_GUARD
        ends = [0]
        for _, kv in seqs:
            ends.append(ends[-1] + kv + 1)                                  # one row between the sequences
        start = torch.tensor(ends, dtype=torch.int32, device="cuda")
        ko, vo = (torch.full((ends[-1] + 2, c.nkv, c.hd), 7.0, device="cuda") for _ in range(2))
        q2.paged_read(c.kv, c.batch, start, ends[-1] + 2, k_out=ko, v_out=vo)
        c.batch.check()
        for s, (n, kv) in enumerate(seqs):
            assert (ko[ends[s] + kv:ends[s + 1]] == 7).all() and (vo[ends[s] + kv:ends[s + 1]] == 7).all()
            at = slice(c.starts[s], c.starts[s] + n)
            skip = max(0, n - kv)
            first = kv - n + skip
            assert (q_out[c.starts[s]:c.starts[s] + skip] == 7).all()
            at = slice(at.start + skip, at.stop)
            n -= skip
            # f32 work: the norm's sum of hd squares (relative (hd / 2 + 3) steps of its root), two products
            # and one sum of the rotation.
            work = (c.hd / 2 + 8) * 2.0 ** -24
            ref = written(c, q[at], qn, table, inter, first)
            big = ref.abs().amax(-1, keepdim=True) * 2 ** 0.5
            err = (q_out[at].double() - ref).abs()
            assert bool((err <= half_step(out_type) * ref.abs() + work * big + 2.0 ** -25).all())
            for name, src, nrm, tab, res, old in (("k", k, kn, table, ko, held[s][0][0]), ("v", v, None, None, vo, held[s][1][0])):
                ref = written(c, src[at], nrm, tab, inter, first)
                big = ref.abs().amax(-1, keepdim=True) * 2 ** 0.5
                rd = res[ends[s]:ends[s] + kv].double()
                # What was there before and is not this call's stays.
                assert bool(((rd[:first] - old[:first]).abs() <= 2.0 ** -23 * old[:first].abs()).all())
                rd = rd[first:]
                err = (rd - ref).abs()
                if fmt not in LARGEST:
                    assert bool((err <= half_step(dt(fmt)) * ref.abs() + work * big + 2.0 ** -25).all()), name
                    continue
                codes, scale = coded(ref, fmt)
                slack = 8 * work * big / scale            # in codes: the f32 work, and the division's
                y = ref / scale
                if fmt == "int8":
                    step = torch.full_like(y, 0.5)
                else:
                    step = half_step(torch.float8_e4m3fn) * y.abs().clamp(min=2.0 ** -6)
                assert bool((err / scale <= step * (1 + 1e-5) + slack).all()), name
                # Away from the borders of rounding the code is the definition's.
                got_codes = rd / scale
                border = (y - (torch.floor(y.abs()) + 0.5) * torch.sign(y)).abs() if fmt == "int8" else None
                if fmt == "int8":
                    sure = border > 2 * slack
                    assert bool(((got_codes - codes).abs()[sure] < 1e-2).all())


def test_int8_rounds_half_away_from_zero(q2):
    c = Case(q2, [(1, 1)], (2, 2, 64), "int8", 16, seed=1)
    x = torch.zeros((c.rows, 2, 64), device="cuda")
    x[0, 0, :7] = torch.tensor([127.0, 0.5, -0.5, 1.5, -2.5, 0.49999997, -126.5])   # scale 1
    q2.paged_write(c.kv, c.batch, x, x)
    c.batch.check()
    pg = int(c.pages[0, 0])
    got = c.kv.k[pg, 0, 0, :7].cpu().tolist()
    assert got == [127, 1, -1, 2, -3, 0, -127]
    assert float(c.kv.k_scale[pg, 0, 0]) == 1.0 and float(c.kv.k_scale[pg, 1, 0]) == 1.0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_read_is_the_exact_value_rounded_once(q2, fmt, out):
    for i, heads in enumerate(HEADS[:4]):
        c = Case(q2, [(0, 1), (0, 130), (0, 0), (0, 77)], heads, fmt, 32, ("head", "token", "padded")[i % 3], seed=30 + i)
        c.fill()
        start = torch.tensor([0, 1, 131, 131, 208], dtype=torch.int32, device="cuda")
        k, v = q2.paged_read(c.kv, c.batch, start, 208, dtype=dt(out))
        c.batch.check()
        for got, pool, scales in ((k, c.kv.k, c.kv.k_scale), (v, c.kv.v, c.kv.v_scale)):
            at = 0
            for s, (_, kv) in enumerate(c.seqs):
                pos = torch.arange(kv, device="cuda")
                pg, off = c.pages[s][pos // 32].long(), pos % 32
                x = pool.view(torch.int8)[pg, off].view(pool.dtype).float() if c.quant else pool[pg, off].float()
                if c.quant:
                    x = x * scales[pg, :, off][..., None]
                assert torch.equal(got[at:at + kv], x.to(dt(out)))
                at += kv


def test_a_nan_in_a_head_is_not_lost_by_quantising(q2):
    for fmt in LARGEST:
        c = Case(q2, [(2, 2)], (2, 2, 64), fmt, 16, seed=2)
        x = torch.ones((c.rows, 2, 64), device="cuda")
        x[0, 1, 5] = math.nan
        q2.paged_write(c.kv, c.batch, x, x)
        k, _ = q2.paged_read(c.kv, c.batch, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), 2)
        assert torch.isnan(k[0, 1]).all() and torch.isfinite(k[0, 0]).all() and torch.isfinite(k[1]).all()


# ---- values in device memory that are wrong -------------------------------------------------


def guard_of(c, q2):
    with pytest.raises(q2.Qwen2Error) as e:
        c.batch.check()
    assert e.value.code == q2.QWEN2_E_DEVICE_GUARD
    c.batch.check()         # reported once
    return str(e.value)


def test_bad_pages_are_reported_and_left_out(q2):
    for bad in (-1, 1 << 30):
        for n in (1, 200):
            c = Case(q2, [(n, 300), (n, 400)], (8, 2, 64), "f16", 64, seed=40)
            held = c.fill(0.0)
            good = int(c.pages[0, 2])
            c.pages[0, 2] = bad
            q = c.queries(torch.float16)
            out = torch.full_like(q, 7.0)
            q2.paged_attention(c.kv, c.batch, q, out=out)
            assert "page" in guard_of(c, q2)
            # Sequence 1 is untouched by it; sequence 0 attends to the other keys.
            keep = torch.ones(300, dtype=torch.bool, device="cuda")
            keep[128:192] = False
            live = Case.__new__(Case)
            live.__dict__.update(c.__dict__)
            live.seqs = [(0, 0), (n, 400)]
            check_attention(live, q, held, out, None, 0.125, True, 7.0)
            if n == 1:
                k, v = (held[0][i][0][keep] for i in (0, 1))
                for h in range(8):
                    w = torch.softmax(k[:, h // 4] @ q[0, h].double() * 0.125, 0)
                    assert (out[0, h].double() - w @ v[:, h // 4]).abs().max() < 2e-3
            k, _ = q2.paged_read(c.kv, c.batch, torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda"), 700,
                                 k_out=torch.full((700, 2, 64), 7.0, device="cuda"),
                                 v_out=torch.full((700, 2, 64), 7.0, device="cuda"))
            assert "page" in guard_of(c, q2)
            assert (k[128:192] == 7).all() and not (k[:128] == 7).all(-1).any()
            c.pages[0, 2] = good
            before = c.kv.k.clone()
            c.pages[0, 299 // 64] = bad
            x = torch.randn((c.rows, 2, 64), device="cuda")
            q2.paged_write(c.kv, c.batch, x, x)
            assert "page" in guard_of(c, q2)
            others = torch.ones(c.kv.n_pages, dtype=torch.bool, device="cuda")
            others[c.pages[0, :4].long()] = False
            others[c.pages[1, :7].long()] = False
            assert torch.equal(c.kv.k[others].view(torch.int16), before[others].view(torch.int16))


def test_bad_starts_and_lengths_are_reported(q2):
    c = Case(q2, [(2, 100), (3, 100)], (8, 2, 64), "f16", 64, seed=41)
    c.fill(0.0)
    q = c.queries(torch.float16)
    x = torch.randn((c.rows, 2, 64), device="cuda")
    for field, values in (("q_start", [0, 5, 2]), ("q_start", [-1, 2, 5]), ("q_start", [0, 2, 100]),
                          ("q_start", [0, 5, 8]), ("kv_len", [100, 1 << 20]), ("kv_len", [-5, 100])):
        t = getattr(c.batch, field)
        old = t.clone()
        t.copy_(torch.tensor(values, dtype=torch.int32))
        q2.paged_attention(c.kv, c.batch, q)
        guard_of(c, q2)
        q2.paged_write(c.kv, c.batch, x, x)
        if values != [-1, 2, 5]:      # rows 0 and 1 are outside every sequence there: nothing to report
            guard_of(c, q2)
        t.copy_(old)
        c.batch.guard.zero_()
    table = torch.from_numpy(q2.rope_table(99, 64)).cuda()     # position 99 is past it
    q2.paged_write(c.kv, c.batch, x, x, rope=table)
    assert "position" in guard_of(c, q2)


def test_a_batch_with_no_rows_at_all(q2):
    c = Case(q2, [(0, 5), (0, 0)], (8, 2, 64), "f16", 64, seed=42)
    c.fill()
    q = c.queries(torch.float16)
    out = torch.full_like(q, 7.0)
    q2.paged_attention(c.kv, c.batch, q, out=out)
    c.batch.check()
    assert (out == 7).all()


def test_rows_against_a_bound_of_none(q2):
    """max_q = 0: nothing to do if no sequence has a row, a guard code if one has."""
    c = Case(q2, [(0, 5), (0, 9)], (8, 2, 64), "f16", 64, seed=43)
    c.fill()
    q = c.queries(torch.float16)
    for starts, bad in (([0, 0, 0], False), ([0, 1, 2], True)):
        b = q2.PagedBatch(torch.tensor(starts, dtype=torch.int32, device="cuda"), c.batch.kv_len, c.pages, 0)
        out = torch.full_like(q, 7.0)
        q2.paged_attention(c.kv, b, q, out=out)
        if bad:
            with pytest.raises(q2.Qwen2Error, match="q_start"):
                b.check()
        else:
            b.check()
        assert (out == 7).all()


# ---- together, and with the model -------------------------------------------------------------


def test_a_layer_over_the_paged_cache_matches_the_models_own(q2):
    """A prompt in two chunks and decode steps through paged_write and paged_attention, for the first layer of
    the toy model: its rotated keys are the model's own cache rows, and the attention output is the formula's."""
    shape = synth.SHAPES["toy"]
    w = synth.make_weights(shape, 0)
    toks = synth.make_tokens(shape.vocab, 50, 3)
    nh, nkv, hd = shape.n_head, shape.n_kv_head, shape.head_dim
    lw = w["layers"][0]
    x = torch.from_numpy(np.asarray(w["embed"], dtype=np.float64)[toks]).cuda()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + shape.rms_eps) * torch.from_numpy(
        np.asarray(lw["attn_norm"], dtype=np.float64)).cuda()
    cat = [torch.from_numpy(np.asarray(lw[k], dtype=np.float64)).cuda() for k in ("wq", "wk", "wv", "bq", "bk", "bv")]
    proj = [(x @ cat[i].T + cat[i + 3]).float().view(50, -1, hd) for i in range(3)]
    table = torch.from_numpy(q2.rope_table(64, hd, shape.rope_theta)).cuda()
    pool = q2.PagedKV.zeros(6, 16, nkv, hd, q2.KV_F16)
    pages = torch.tensor([[4, 0, 3, 1]], dtype=torch.int32, device="cuda")
    outs, at = [], 0
    for n in (20, 17, 1, 1, 1, 10):
        batch = q2.PagedBatch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                              torch.tensor([at + n], dtype=torch.int32, device="cuda"), pages, n)
        rows = slice(at, at + n)
        q = q2.paged_write(pool, batch, proj[1][rows], proj[2][rows], q=proj[0][rows], rope=table)
        outs.append(q2.paged_attention(pool, batch, q))
        batch.check()
        at += n
    o = torch.cat(outs)
    with q2.Qwen2Model(shape, w, n_ctx=64, max_seqs=1, max_tokens=64) as m:
        m.prefill([0], [toks])
        cache = m.kv_cache()[0, 0].clone().double()          # [2, nkv, n_ctx, hd]
        m.synchronize()
    k, v = q2.paged_read(pool, batch, torch.tensor([0, 50], dtype=torch.int32, device="cuda"), 50)
    # f16 pages against the model's f32 rows: half a step, and the model's f32 products.
    for got, ref in ((k, cache[0, :, :50]), (v, cache[1, :, :50])):
        ref = ref.transpose(0, 1)
        assert bool(((got.double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 1e-5).all())
    t = table[:50].double()
    qr = proj[0].double()
    lo, hi = qr[..., :hd // 2], qr[..., hd // 2:]
    qr = torch.cat((lo * t[:, None, :, 0] - hi * t[:, None, :, 1], hi * t[:, None, :, 0] + lo * t[:, None, :, 1]), -1)
    late = torch.ones(50, 50, device="cuda").triu(1).bool()
    for h in range(nh):
        kk, vv = cache[0, h * nkv // nh, :50], cache[1, h * nkv // nh, :50]
        a = torch.softmax((qr[:, h] @ kk.T / hd ** 0.5).masked_fill(late, -math.inf), -1)
        # q, k, v, the probabilities and the output each rounded to f16 once; |scores| stay below 8.
        assert (o[:, h].double() - a @ vv).abs().max() <= 2.0 ** -11 * (2 * 8 + 3) * float(vv.abs().max())


@pytest.mark.parametrize("fmt", ["f16", "int8"])
def test_model_sequences_are_parked_in_pages_and_resumed(q2, fmt):
    """save_pages / load_pages: a conversation moved through pages into another slot goes on with the same ids
    (f16) and holds the values the format stands for."""
    shape = synth.SHAPES["toy"]
    w = synth.make_weights(shape, 0)
    prompt = synth.make_tokens(shape.vocab, 40, 5)
    with q2.Qwen2Model(shape, w, n_ctx=64, max_seqs=2, max_tokens=64) as m:
        _, ids = m.prefill([0], [prompt])
        first = int(ids[0])
        pools = [q2.PagedKV.zeros(4, 16, shape.n_kv_head, shape.head_dim, getattr(q2, "KV_" + fmt.upper()))
                 for _ in range(shape.n_layer)]
        pages = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
        m.save_pages(0, 40, pools, pages)
        m.load_pages(1, 40, pools, pages)
        cache = m.kv_cache().double()
        a, b = cache[0, :, :, :, :40], cache[1, :, :, :, :40]
        if fmt == "f16":
            assert bool(((a - b).abs() <= 2.0 ** -11 * a.abs() + 2.0 ** -25).all())
        else:
            assert bool(((a - b).abs() <= a.abs().amax(-1, keepdim=True) / 127 * 0.5001).all())
        assert (cache[1, :, :, :, 40:] == 0).all()
        if fmt == "f16":
            x = m.decode_steps([0], [first], [40], 12).cpu().numpy()
            y = m.decode_steps([1], [first], [40], 12).cpu().numpy()
            assert (x[:4] == y[:4]).all()
        for bad in ((2, 40), (0, 0), (0, 65), (0, 49)):
            with pytest.raises(q2.Qwen2Error):
                m.save_pages(*bad, pools, pages)
        with pytest.raises(q2.Qwen2Error):
            m.save_pages(0, 40, pools[:1], pages)
        m.synchronize()


def test_parking_in_a_page_that_is_none_is_reported(q2):
    """A page id outside the pools is left out, and check() of the returned batch says so; the rest is kept."""
    shape = synth.SHAPES["toy"]
    with q2.Qwen2Model(shape, synth.make_weights(shape, 0), n_ctx=64, max_seqs=2, max_tokens=64) as m:
        m.prefill([0], [synth.make_tokens(shape.vocab, 40, 5)])
        pools = [q2.PagedKV.zeros(4, 16, shape.n_kv_head, shape.head_dim, q2.KV_F16) for _ in range(shape.n_layer)]
        pages = torch.tensor([2, 4, 3], dtype=torch.int32, device="cuda")
        for call in (m.save_pages, m.load_pages):
            with pytest.raises(q2.Qwen2Error, match="page id"):
                call(0 if call == m.save_pages else 1, 40, pools, pages).check()
        cache = m.kv_cache()
        for rows in (slice(0, 16), slice(32, 40)):
            assert torch.equal(cache[1, :, :, :, rows], cache[0, :, :, :, rows].half().float())
        assert (cache[1, :, :, :, 16:32] == 0).all()
        m.synchronize()


def test_binding_refuses_mismatched_tensors(q2):
    c = Case(q2, [(1, 5)], (8, 2, 64), "f16", 64, seed=43)
    q = c.queries(torch.float16)
    x = torch.zeros((c.rows, 2, 64), device="cuda")
    for call in (lambda: q2.paged_attention(c.kv, c.batch, q.cpu()),
                 lambda: q2.paged_attention(c.kv, c.batch, q[..., :32]),
                 lambda: q2.paged_attention(c.kv, c.batch, q, out=q[:1].clone()),
                 lambda: q2.paged_attention(c.kv, c.batch, q.transpose(1, 2)),
                 lambda: q2.paged_attention(c.kv, c.batch, q, workspace=torch.empty(8, device="cuda")),
                 lambda: q2.paged_write(c.kv, c.batch, x, x[:1]),
                 lambda: q2.paged_write(c.kv, c.batch, x, x, q_norm=x[0, 0]),
                 lambda: q2.paged_write(c.kv, c.batch, x, x, k_norm=x[0, 0, :32]),
                 lambda: q2.paged_write(c.kv, c.batch, x, x, rope=x[0]),
                 lambda: q2.paged_read(c.kv, c.batch, c.batch.kv_len, 4),
                 lambda: q2.paged_read(c.kv, c.batch, c.batch.q_start, 4, k_out=x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: q2.paged_attention(c.kv, c.batch, q.bfloat16()),
                 lambda: q2.paged_attention(c.kv, c.batch, q[:, :7]),
                 lambda: q2.paged_attention(c.kv, c.batch, q, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(q2.Qwen2Error):
            call()
