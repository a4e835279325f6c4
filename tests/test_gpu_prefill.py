"""gqla_prefill_gqa on the GPU against the attention formula in float64.

Tolerances, per element, with u = 2^-8 (half a bf16 step, relative) and e = 2^-24:
  * the scores: 192 exact bf16 products summed in fp32, |ds| <= 192 e scale sum|q k| (D);
  * P is rounded to bf16 (u), 2^x and the sum of P add less than 2^-21 + (L / 32) e, and the
    scores move p by a factor within 2 D of 1, numerator and denominator alike:
      |do| <= A (u + 4 D + 2^-20 + L e) + u |o|,  A = sum_t p_t |v_t|;
  * the merge of partials adds a few fp32 roundings, inside the 2^-20;
  * lse: |d| <= D + 2^-20 + L e + 2^-22 |lse|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24
SCALE = 1.0 / math.sqrt(192)


def make(h, g, new, ctx, seed=0, spare=3, tail=float("nan"), gap=0):
    """A ragged batch over a paged expanded cache on the GPU. Slots that hold no token are
    `tail`; unused page-table entries name no page; `gap` query rows before and after the
    batch belong to no sequence."""
    gen = torch.Generator().manual_seed(seed)
    lens = [n + c for n, c in zip(new, ctx)]
    need = [(x + 63) // 64 for x in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(new), max(max(need), 1) + 1), -7, dtype=torch.int32)
    kv = torch.full((g, pages * 64, 256), tail, dtype=torch.bfloat16)
    rope = torch.full((pages * 64, 64), tail, dtype=torch.bfloat16)
    at, slots = 0, []
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
        t = torch.arange(lens[b])
        sl = table[b].long()[t // 64] * 64 + t % 64
        kv[:, sl] = torch.randn(g, lens[b], 256, generator=gen).to(torch.bfloat16)
        rope[sl] = torch.randn(lens[b], 64, generator=gen).to(torch.bfloat16)
        slots.append(sl.cuda())
    starts = [gap]
    for n in new:
        starts.append(starts[-1] + n)
    q = torch.randn(starts[-1] + gap, h, 192, generator=gen).to(torch.bfloat16)
    return dict(h=h, g=g, new=new, lens=lens, pages=pages, table=table.cuda(), kv=kv.cuda(), rope=rope.cuda(),
                q=q.cuda(), starts=torch.tensor(starts, dtype=torch.int32).cuda(), slots=slots,
                seqlens=torch.tensor(lens, dtype=torch.int32).cuda(), row0=starts)


def reference(c):
    """(out, lse, tolerance of out, tolerance of lse) in float64; rows of no sequence are NaN."""
    h, g = c["h"], c["g"]
    G, total = h // g, c["q"].shape[0]
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.full((total, h, 128), math.nan, **f64), torch.full((total, h), math.nan, **f64)
    tol_o, tol_l = out.clone(), lse.clone()
    for b, n in enumerate(c["new"]):
        if n == 0:
            continue
        L, sl, r = c["lens"][b], c["slots"][b], slice(c["row0"][b], c["row0"][b + 1])
        kv, rope = c["kv"][:, sl].double(), c["rope"][sl].double()
        k = torch.cat([kv[..., :128], rope.expand(g, L, 64)], -1)
        q = c["q"][r].double().view(n, g, G, 192)
        s = torch.einsum("nghd,gtd->nght", q, k) * SCALE
        mag = torch.einsum("nghd,gtd->nght", q.abs(), k.abs()) * SCALE
        seen = torch.arange(L, device="cuda") <= (L - n + torch.arange(n, device="cuda"))[:, None]
        s.masked_fill_(~seen[:, None, None, :], -math.inf)
        z = torch.logsumexp(s, -1)
        p = (s - z[..., None]).exp()
        o = torch.einsum("nght,gtd->nghd", p, kv[..., 128:])
        A = torch.einsum("nght,gtd->nghd", p, kv[..., 128:].abs())
        D = (192 * E * mag.masked_fill(~seen[:, None, None, :], 0.0).amax(-1)).view(n, h)
        out[r], lse[r] = o.reshape(n, h, 128), z.reshape(n, h)
        tol_o[r] = A.reshape(n, h, 128) * (U + 4 * D + 2.0 ** -20 + L * E)[..., None] + U * out[r].abs()
        tol_l[r] = D + 2.0 ** -20 + L * E + 2.0 ** -22 * lse[r].abs()
    return out, lse, tol_o, tol_l


def call(c, splits=None, lse=True, fill=7.0, stream=None):
    """(out, lse, device error) of one call; output rows start out as `fill`."""
    from decode_attention_06_b200 import gqla
    dims = gqla.make_dims(c["h"], c["g"])
    kv = gqla.make_kv_index(c["table"], c["seqlens"], c["pages"])
    if splits is None:
        splits = gqla.plan_prefill(dims, c["new"], c["lens"])
    bufs = gqla.PrefillBuffers(dims, c["q"].shape[0], splits)
    bufs.out.fill_(fill)
    bufs.lse.fill_(fill)
    if bufs.o_part is not None:
        bufs.o_part.fill_(math.nan)
        bufs.lse_part.fill_(math.nan)
    torch.cuda.synchronize()
    gqla.gqla_prefill_gqa(dims, c["q"], c["starts"], c["kv"], c["rope"], kv, splits, bufs.o_part, bufs.lse_part,
                          bufs.out, bufs.lse if lse else None, bufs.workspace, stream)
    torch.cuda.synchronize()
    return bufs.out, bufs.lse, gqla.gqla_read_device_error(bufs.workspace)


def check(c, got, lse, fill=7.0):
    out, z, tol_o, tol_l = reference(c)
    mine = ~torch.isnan(z)
    assert bool((got[~mine.any(-1)] == fill).all()) and bool((lse[~mine.any(-1)] == fill).all())
    rows = mine.any(-1)
    d = (got[rows].double() - out[rows]).abs()
    assert bool((d <= tol_o[rows]).all()), f"out: {float((d / tol_o[rows]).max()):.3f} of the tolerance"
    d = (lse[rows].double() - z[rows]).abs()
    assert bool((d <= tol_l[rows]).all()), f"lse: {float((d / tol_l[rows]).max()):.3f} of the tolerance"


SHAPES = {
    "one_token": (32, 8, [1], [0]),
    "one_token_ctx": (128, 8, [1], [64]),
    "verify": (32, 8, [5], [251]),
    "tile_edge": (128, 8, [8, 9, 16, 17], [120, 119, 112, 111]),
    "page_edge": (128, 8, [63, 64, 65], [1, 64, 63]),
    "prompt_odd": (128, 8, [333], [0]),
    "empty_ones": (128, 8, [0, 3, 0, 0, 40, 0], [0, 200, 77, 0, 129, 5]),
    "g4_heads32": (128, 4, [1, 2, 7, 33], [500, 0, 127, 64]),
    "heads4": (32, 8, [130, 1, 31, 32, 33], [3, 260, 0, 100, 95]),
    "heads1": (8, 8, [150, 257], [10, 0]),
    "heads12": (24, 2, [23, 5, 41], [100, 300, 0]),
    "heads128": (128, 1, [3, 2], [130, 0]),
    "heads3_groups5": (15, 5, [85, 90], [40, 0]),
    "long": (32, 8, [4, 70], [5000, 2500]),
}


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("splits", [None, 1, 5, 37, -1, -6, -50])
def test_prefill_matches_the_formula(name, splits):
    h, g, new, ctx = SHAPES[name]
    c = make(h, g, new, ctx, seed=len(name), gap=3)
    out, lse, err = call(c, splits)
    assert err[0] == 0
    check(c, out, lse)


def test_prefill_without_lse_leaves_it_alone():
    c = make(32, 8, [7, 40], [100, 3], seed=2)
    out, lse, err = call(c, lse=False)
    assert err[0] == 0 and bool((lse == 7.0).all())
    want, _, tol, _ = reference(c)
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("factor", [4.0, 30.0])
@pytest.mark.parametrize("splits", [None, -3, 11])
def test_prefill_rising_scores(factor, splits):
    """Keys that grow along the sequence: the running maximum rises by more than 2^8 tile after
    tile, so O is rescaled all along (the decreasing order leaves every later tile negligible)."""
    for flip in (False, True):
        c = make(128, 8, [50, 3], [900, 1300], seed=9)
        for b, L in enumerate(c["lens"]):
            ramp = 1.0 + factor * torch.arange(L, device="cuda") / L
            if flip:
                ramp = ramp.flip(0)
            sl = c["slots"][b]
            c["rope"][sl] = (c["rope"][sl].float() * ramp[:, None]).to(torch.bfloat16)
        out, lse, err = call(c, splits)
        assert err[0] == 0
        check(c, out, lse)


def test_prefill_masked_keys_of_any_value():
    """Keys and values that no row of a sequence sees hold NaN and infinities: tail slots, and the
    pages of another sequence."""
    for tail in (float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min):
        c = make(32, 8, [33, 1, 70], [95, 64, 57], seed=4, tail=tail)
        out, lse, err = call(c)
        assert err[0] == 0
        check(c, out, lse)


def test_prefill_later_tokens_do_not_reach_earlier_blocks():
    """A NaN in a later token of the same sequence changes nothing for query blocks that end before it."""
    c = make(128, 8, [200], [40], seed=5)
    ref, ref_lse, _ = call(c, -5)
    c["kv"][:, c["slots"][0][-9:]] = float("nan")  # blocks of 32 tokens: only the last two see or hold these
    out, lse, err = call(c, -5)
    assert err[0] == 0
    assert torch.equal(out[:160], ref[:160]) and torch.equal(lse[:160], ref_lse[:160])


def test_prefill_reports_inconsistent_sequences_and_finishes_the_rest():
    c = make(32, 8, [20, 30, 40, 50], [5, 200, 0, 70], seed=6)
    want, want_lse, tol, tol_l = reference(c)
    for bad, change in ((1, lambda s, L: L.__setitem__(1, 29)), (3, lambda s, L: L.__setitem__(3, 10 ** 6)),
                        (3, lambda s, L: s.__setitem__(4, 141)), (2, lambda s, L: L.__setitem__(2, -5))):
        d = dict(c, starts=c["starts"].clone(), seqlens=c["seqlens"].clone())
        change(d["starts"], d["seqlens"])
        for splits in (None, 9):
            out, lse, err = call(d, splits)
            assert err == (-5, bad)
            rows = slice(c["row0"][bad], c["row0"][bad + 1])
            assert bool((out[rows] == 7.0).all()) and bool((lse[rows] == 7.0).all())
            keep = torch.ones(out.shape[0], dtype=torch.bool, device="cuda")
            keep[rows] = False
            assert bool(((out[keep].double() - want[keep]).abs() <= tol[keep]).all())
            assert bool(((lse[keep].double() - want_lse[keep]).abs() <= tol_l[keep]).all())


def test_prefill_reports_pages_outside_the_pool():
    c = make(32, 8, [20, 30, 40], [200, 200, 0], seed=7)
    want, _, tol, _ = reference(c)
    for page in (-1, c["pages"], 2 ** 31 - 1):
        d = dict(c, table=c["table"].clone())
        d["table"][1, 2] = page
        out, _, err = call(d)
        assert err == (-5, 1)
        for b in (0, 2):
            rows = slice(c["row0"][b], c["row0"][b + 1])
            assert bool(((out[rows].double() - want[rows]).abs() <= tol[rows]).all())


def test_prefill_far_offsets():
    """Pages whose elements lie beyond 2^31 in the expanded cache."""
    from decode_attention_06_b200 import gqla
    pages = 140_000  # 140000 * 64 * 256 elements a group
    c = make(16, 1, [37, 5], [300, 1000], seed=8)
    move = torch.arange(pages - c["pages"], pages, device="cuda")
    kv = torch.empty(1, pages * 64, 256, dtype=torch.bfloat16, device="cuda")
    rope = torch.empty(pages * 64, 64, dtype=torch.bfloat16, device="cuda")
    kv.view(1, pages, 64, 256)[:, move] = c["kv"].view(1, -1, 64, 256)
    rope.view(pages, 64, 64)[move] = c["rope"].view(-1, 64, 64)
    far = dict(c, table=torch.where(c["table"] >= 0, c["table"] + (pages - c["pages"]), c["table"]), kv=kv, rope=rope,
               pages=pages)
    out, lse, err = call(far)
    assert err[0] == 0
    check(c, out, lse)
    del gqla


def test_prefill_repeats_bit_for_bit():
    c = make(128, 8, [300, 1, 17], [700, 3000, 0], seed=10)
    ref = call(c, 29)
    for _ in range(3):
        out, lse, _ = call(c, 29)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_prefill_on_another_stream_and_in_a_graph():
    from decode_attention_06_b200 import gqla
    c = make(128, 8, [60, 9], [400, 1500], seed=11)
    want, want_lse, tol, tol_l = reference(c)
    side = torch.cuda.Stream()
    out, lse, err = call(c, 21, stream=side)
    assert err[0] == 0
    check(c, out, lse)
    # captured twice (divided and whole plans) into graphs that share the workspace and are replayed
    # in turn, with new lengths and queries in place: the plan follows the device's numbers
    dims = gqla.make_dims(c["h"], c["g"])
    kv = gqla.make_kv_index(c["table"], c["seqlens"], c["pages"])
    bufs = [gqla.PrefillBuffers(dims, c["q"].shape[0], s) for s in (21, -16)]
    bufs[1].workspace = bufs[0].workspace
    graphs = []
    for b in bufs:
        gqla.prefill_step(dims, b, c["q"], c["starts"], kv, c["kv"], c["rope"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gqla.prefill_step(dims, b, c["q"], c["starts"], kv, c["kv"], c["rope"])
        graphs.append(g)
    for new in ([60, 9], [31, 38], [1, 0], [69, 0]):
        d = dict(c, new=new, lens=[400 + new[0], 1500 + new[1]], row0=[0, new[0], sum(new)])
        if max(d["lens"][0] - c["lens"][0], d["lens"][1] - c["lens"][1]) > 0:
            d["lens"] = [min(a, b) for a, b in zip(d["lens"], c["lens"])]
        c["seqlens"].copy_(torch.tensor(d["lens"], dtype=torch.int32))
        c["starts"].copy_(torch.tensor(d["row0"], dtype=torch.int32))
        d["slots"] = [s[:n] for s, n in zip(c["slots"], d["lens"])]
        c["q"].copy_(torch.randn_like(c["q"], dtype=torch.float32).to(torch.bfloat16))
        for b, g in zip(bufs, graphs):
            b.out.fill_(7.0)
            b.lse.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert gqla.gqla_read_device_error(b.workspace)[0] == 0
            check(d, b.out, b.lse)


def test_prefill_refuses_wrong_tensors():
    from decode_attention_06_b200 import gqla
    c = make(32, 8, [4], [3], seed=1)
    dims = gqla.make_dims(32, 8)
    kv = gqla.make_kv_index(c["table"], c["seqlens"], c["pages"])
    b = gqla.PrefillBuffers(dims, 4, -8)
    with pytest.raises(ValueError, match="contiguous"):
        gqla.prefill_step(dims, b, c["q"].transpose(0, 1).contiguous().transpose(0, 1), c["starts"], kv, c["kv"], c["rope"])
    with pytest.raises(ValueError, match="shape"):
        gqla.prefill_step(dims, b, c["q"], c["starts"][:1], kv, c["kv"], c["rope"])
    with pytest.raises(ValueError, match="bfloat16"):
        gqla.prefill_step(dims, b, c["q"].float(), c["starts"], kv, c["kv"], c["rope"])
    with pytest.raises(ValueError, match="CUDA"):
        gqla.prefill_step(dims, b, c["q"].cpu(), c["starts"], kv, c["kv"], c["rope"])
    with pytest.raises(ValueError, match="buffers hold"):
        gqla.prefill_step(dims, gqla.PrefillBuffers(dims, 3, -8), c["q"], c["starts"], kv, c["kv"], c["rope"])
    with pytest.raises(gqla.GqlaError) as e:
        gqla.gqla_prefill_gqa(dims, c["q"], c["starts"], c["kv"], c["rope"], kv, 4, None, None, b.out, b.lse, b.workspace)
    assert e.value.status == -1


@pytest.mark.parametrize("splits,unit", [(-8, 0), (5, 1)])
def test_prefill_wait_that_runs_out_is_reported(splits, unit):
    """A V load that never comes: the wait for it runs out after about two seconds, both CTAs of the pair
    give up together, the call records GQLA_ERR_TIMEOUT, and the next call is correct."""
    from decode_attention_06_b200 import gqla
    c = make(32, 8, [40, 3], [300, 500], seed=12)
    gqla.gqla_debug_drop_v_load(unit)
    _, _, err = call(c, splits)
    assert err[0] == -6
    out, lse, err = call(c, splits)
    assert err[0] == 0
    check(c, out, lse)


@pytest.mark.parametrize("batch,every,n", [(900, 1, 1), (1500, 400, 30), (1000, 7, 3)])
@pytest.mark.parametrize("splits", [None, 1, -9])
def test_prefill_large_batches(batch, every, n, splits):
    """More sequences than a CTA has threads, most of them without new tokens; more in a chunk than
    its list holds."""
    new = [n if b % every == 0 else 0 for b in range(batch)]
    c = make(16, 2, new, [(b * 37) % 150 for b in range(batch)], seed=13)
    out, lse, err = call(c, splits)
    assert err[0] == 0
    check(c, out, lse)


@pytest.mark.parametrize("shape", ["verify", "tile_edge", "heads4", "heads12", "g4_heads32"])
@pytest.mark.parametrize("splits", [None, 7, -3])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_prefill_nan_scores_reach_their_rows_only(shape, splits, what):
    """A query row that holds NaN or infinity and a key that does: NaN in the rows that see them, in
    out and in the LSE, and the formula everywhere else."""
    h, g, new, ctx = SHAPES[shape]
    c = make(h, g, new, ctx, seed=8, gap=2)
    b = len(new) - 1  # the key: the last sequence's second new token's, of group 0
    c["kv"][0, c["slots"][b][ctx[b] + 1], 7] = what
    c["q"][c["row0"][0], 1, 5] = what
    c["q"][c["row0"][0], 1, 9] = -what  # with infinities the scores differ in sign, or are NaN
    nan = torch.zeros(c["q"].shape[0], h, dtype=torch.bool, device="cuda")
    nan[c["row0"][0], 1] = True
    nan[c["row0"][b] + 1:c["row0"][b + 1], :h // g] = True
    if what == math.inf:  # an infinite score of either sign is right or NaN, as the formula is
        clean = dict(c, kv=c["kv"].clone(), q=c["q"].clone())
        clean["kv"][0, c["slots"][b][ctx[b] + 1], 7] = 0
        clean["q"][c["row0"][0], 1, [5, 9]] = 0
    else:
        clean = dict(c, kv=c["kv"].nan_to_num(0.0), q=c["q"].nan_to_num(0.0))
    out, z, tol_o, tol_l = reference(clean)
    got, lse, err = call(c, splits)
    assert err[0] == 0
    if what != math.inf:
        assert bool(torch.isnan(got[nan]).all()) and bool(torch.isnan(lse[nan]).all())
    keep = ~nan & ~torch.isnan(z)
    assert bool(((got.double() - out).abs() <= tol_o)[keep].all())
    assert bool(((lse.double() - z).abs() <= tol_l)[keep].all())


def test_prefill_calls_at_once_on_two_streams():
    """Two calls with buffers of their own, again and again at the same time: each the bits of its
    call alone."""
    from decode_attention_06_b200 import gqla
    cases = [make(128, 8, [333, 1, 40], [0, 700, 129], seed=21), make(32, 8, [130, 5, 64], [300, 2000, 0], seed=22)]
    sides = []
    for c, splits in zip(cases, (37, -9)):
        dims = gqla.make_dims(c["h"], c["g"])
        kv = gqla.make_kv_index(c["table"], c["seqlens"], c["pages"])
        want, want_lse, err = call(c, splits)
        assert err[0] == 0
        sides.append((c, dims, kv, gqla.PrefillBuffers(dims, c["q"].shape[0], splits), torch.cuda.Stream(), want, want_lse))
    torch.cuda.synchronize()
    for _ in range(30):
        for c, dims, kv, bufs, stream, _, _ in sides:
            gqla.prefill_step(dims, bufs, c["q"], c["starts"], kv, c["kv"], c["rope"], stream=stream)
    torch.cuda.synchronize()
    for _, _, _, bufs, _, want, want_lse in sides:
        assert gqla.gqla_read_device_error(bufs.workspace)[0] == 0
        assert torch.equal(bufs.out, want) and torch.equal(bufs.lse, want_lse)


@pytest.mark.parametrize("h,g,splits", [(128, 8, 74), (128, 8, -40), (32, 8, -16)])
def test_prefill_rows_past_the_keys_never_enter(h, g, splits):
    """Blocks that end at every kind of place in a key tile (in the first page, which one CTA of the pair
    clears, in the second, at its start), with NaN in the slots behind them: call after call the bits
    that zeros there give."""
    new = [1, 5, 33, 40, 17, 64, 3, 90]
    ctx = [0, 59, 31, 89, 110, 65, 253, 166]  # ends 1, 64, 64, 129, 127, 129, 256, 256
    ctx += [c + 1 for c in ctx] + [c + 70 for c in ctx]
    zeros = make(h, g, new * 3, ctx, seed=31, tail=0.0)
    nans = make(h, g, new * 3, ctx, seed=31)
    want = call(zeros, splits)
    check(zeros, want[0], want[1])
    for _ in range(40):
        out, lse, err = call(nans, splits)
        assert err[0] == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_prefill_length_of_31_bits():
    """A sequence of 2^31 - 1 tokens over a few pages named again and again; its very last page is one of
    its own, with a key that outweighs all others: the answer is that key's value."""
    from decode_attention_06_b200 import gqla
    most, width, pages = (1 << 31) - 1, 1 << 25, 5
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    kv, rope, q = rnd(1, pages * 64, 256), rnd(pages * 64, 64) * 0.01, rnd(2, 16, 192)
    table = (torch.arange(width, device="cuda", dtype=torch.int32) % 4).view(1, -1)
    table[0, -1] = 4
    # the last two tokens are the queries; scores of 1000 for key 2^31 - 3, -1000 for the very last one,
    # a few units for the rest: 2^31 of them weigh e^(22 + 30 - 1000), nothing in float32
    q[..., 128:] = 0
    q[..., 128] = 100.0
    rope[:, 0] = 0
    rope[4 * 64 + 61, 0], rope[4 * 64 + 62, 0] = 144.0, -144.0
    starts = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    idx = gqla.make_kv_index(table, torch.tensor([most], dtype=torch.int32, device="cuda"), pages)
    dims = gqla.make_dims(16, 1)
    bufs = gqla.PrefillBuffers(dims, 2, gqla.plan_prefill(dims, [2], [most]))
    out, lse = gqla.prefill_step(dims, bufs, q, starts, idx, kv, rope)
    torch.cuda.synchronize()
    assert gqla.gqla_read_device_error(bufs.workspace)[0] == 0
    k = torch.cat([kv[0, 4 * 64 + 61, :128], rope[4 * 64 + 61]]).double()
    score = torch.einsum("nhd,d->nh", q.double(), k) * SCALE
    assert bool((score > 900).all())
    mag = torch.einsum("nhd,d->nh", q.double().abs(), k.abs()) * SCALE
    assert bool(((lse.double() - score).abs() <= 192 * E * mag + 2.0 ** -20 + 2.0 ** -22 * score).all())
    # P is 1 for that key (or a power of two off it by the score's rounding, the same in O and l), 0 elsewhere
    v = kv[0, 4 * 64 + 61, 128:].double()
    assert bool(((out.double() - v).abs() <= (2 * U + 2.0 ** -20) * v.abs()).all())


@pytest.mark.parametrize("step", [5.0, 12.0, 70.0])
@pytest.mark.parametrize("splits", [None, 1, -7, 23])
@pytest.mark.parametrize("values", [0, 100])
def test_prefill_scores_that_step_with_every_tile(step, splits, values):
    """Scores that rise by `step` powers of two with every key tile in some rows, by half of that in
    others, fall in others and stay level in the rest, side by side in a warp: bases that are raised
    seldom, with every tile, or once the sum has grown over several; in blocks of two MMA tiles, in the
    even and odd halves of blocks of one, and in pieces. And with values near 2^100, inside the range
    that the header gives (2^118 / L)."""
    c = make(128, 8, [50, 3, 16, 1], [900, 1300, 640, 2000], seed=17)
    per_tile = step * math.log(2.0) / SCALE
    for b, L in enumerate(c["lens"]):
        c["rope"][c["slots"][b], 0] = (per_tile * (torch.arange(L, device="cuda") // 128)).to(torch.bfloat16)
    kind = (torch.arange(c["q"].shape[0], device="cuda")[:, None] + torch.arange(128, device="cuda")) % 5
    c["q"][..., 128] = torch.tensor([1.0, 0.0, -1.0, 0.5, 0.0], device="cuda")[kind].to(torch.bfloat16)
    c["kv"][..., 128:] *= 2.0 ** values
    out, lse, err = call(c, splits)
    assert err[0] == 0
    check(c, out, lse)


@pytest.mark.parametrize("h,g", [(64, 16), (37, 37), (80, 20), (48, 2), (40, 1), (200, 2), (127, 1)])
@pytest.mark.parametrize("splits", [None, 1, 26, -9])
def test_prefill_of_other_head_layouts(h, g, splits):
    """More groups than 8, and group sizes that leave rows of the tile unused (24, 40, 100, 127 heads)."""
    c = make(h, g, [1, 6, 0, 45], [130, 250, 9, 71], seed=h, gap=2)
    out, lse, err = call(c, splits)
    assert err[0] == 0
    check(c, out, lse)
