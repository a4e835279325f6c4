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
