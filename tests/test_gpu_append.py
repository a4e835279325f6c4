"""gqla_append_cache on the GPU against the projections in float64.

Tolerance: one bf16 rounding (2^-8 relative) and the fp32 accumulation of 512 products,
|x - exact| <= 2^-8 |exact| + 2^-15 sum_k |c_k w_k| (the bound of gqla_expand_cache_tc); the latent
rows and the RoPE keys are copied exactly, everything else in the caches stays as it was.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def make(g, new, ctx, seed=0, gap=0, spare=2, h=None):
    gen = torch.Generator().manual_seed(seed)
    lens = [n + c for n, c in zip(new, ctx)]
    need = [(x + 63) // 64 for x in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(new), max(max(need), 1) + 1), -5, dtype=torch.int32)
    starts, at = [gap], 0
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
        starts.append(starts[-1] + new[b])
    bf = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    w = lambda: (torch.randn(g, 512, 128, generator=gen) / math.sqrt(512)).to(torch.bfloat16).cuda()  # noqa: E731
    return dict(g=g, h=h or 16 * g, new=new, lens=lens, pages=pages, table=table.cuda(), starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                row0=starts, seqlens=torch.tensor(lens, dtype=torch.int32).cuda(), rows=bf(starts[-1] + gap, 576),
                w_uk=w(), w_uv=w(), latent=bf(pages, 64, 576), kv=bf(g, pages * 64, 256), rope=bf(pages * 64, 64))


def run(c, latent=True, expanded=True):
    from decode_attention_06_b200 import gqla
    dims = gqla.make_dims(c["h"], c["g"])
    idx = gqla.make_kv_index(c["table"], c["seqlens"], c["pages"])
    ws = gqla.new_workspace()
    out = {k: c[k].clone() for k in ("latent", "kv", "rope")}
    gqla.gqla_append_cache(dims, c["rows"], c["starts"], idx, ws, latent_cache=out["latent"] if latent else None,
                           **(dict(w_uk=c["w_uk"], w_uv=c["w_uv"], kv_expanded=out["kv"], k_rope=out["rope"])
                              if expanded else {}))
    torch.cuda.synchronize()
    return out, gqla.gqla_read_device_error(ws)


def check(c, out, latent=True, expanded=True, skip=()):
    want = {k: c[k].clone() for k in ("latent", "kv", "rope")}
    touched = torch.zeros(c["pages"] * 64, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c["new"]):
        if n == 0 or b in skip:
            continue
        t = torch.arange(c["lens"][b] - n, c["lens"][b], device="cuda")
        slot = c["table"][b, t // 64].long() * 64 + t % 64
        rows = c["rows"][c["row0"][b]:c["row0"][b + 1]]
        touched[slot] = True
        if latent:
            want["latent"].view(-1, 576)[slot] = rows
        if expanded:
            want["rope"][slot] = rows[:, 512:]
            cd, w = rows[:, :512].double(), torch.cat([c["w_uk"], c["w_uv"]], -1).double()
            exact = torch.matmul(cd, w)
            tol = 2.0 ** -8 * exact.abs() + 2.0 ** -15 * torch.matmul(cd.abs(), w.abs())
            d = (out["kv"][:, slot].double() - exact).abs()
            assert bool((d <= tol).all()), float((d / tol).max())
    assert torch.equal(out["latent"], want["latent"])
    assert torch.equal(out["rope"], want["rope"])
    keep = ~touched if expanded else torch.ones_like(touched)
    assert torch.equal(out["kv"][:, keep], c["kv"][:, keep])


CASES = {
    "one": (8, [1], [0]),
    "one_deep": (8, [1], [127]),
    "step": (8, [2] * 64, list(range(0, 640, 10))),
    "page_edges": (4, [63, 64, 65, 1], [1, 0, 63, 64]),
    "empty_ones": (2, [0, 5, 0, 0, 130, 0], [3, 0, 0, 64, 70, 9]),
    "tile_edge": (8, [127, 1, 128, 129], [0, 64, 1, 63]),
    "groups1": (1, [200, 31], [5, 0]),
    "groups3": (3, [300, 7], [0, 20]),
    "groups6_many": (6, [700, 900, 1100], [10, 0, 33]),
    "many": (8, [3001, 2000, 1500, 777], [0, 100, 0, 5]),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("what", ["both", "expanded", "latent"])
def test_append_matches_the_projections(name, what):
    c = make(*CASES[name], seed=len(name), gap=3)
    out, err = run(c, latent=what != "expanded", expanded=what != "latent")
    assert err[0] == 0
    check(c, out, latent=what != "expanded", expanded=what != "latent")


def test_append_leaves_out_what_is_inconsistent_and_reports_it():
    c = make(2, [20, 30, 40], [5, 100, 0], seed=3)
    for bad, change in ((1, lambda d: d["seqlens"].__setitem__(1, 29)), (2, lambda d: d["seqlens"].__setitem__(2, 10 ** 6)),
                        (0, lambda d: d["starts"].__setitem__(0, -1)), (2, lambda d: d["starts"].__setitem__(3, 91))):
        d = dict(c, starts=c["starts"].clone(), seqlens=c["seqlens"].clone())
        change(d)
        out, err = run(d)
        assert err == (-5, bad)
        check(c, out, skip=(bad,))


def test_append_skips_pages_outside_the_pool():
    c = make(2, [20, 30], [5, 100], seed=4)
    for page in (-1, c["pages"]):
        d = dict(c, table=c["table"].clone())
        d["table"][1, 2] = page  # tokens 128 and 129 of sequence 1
        out, err = run(d)
        assert err == (-5, 1)
        e = dict(c, new=[20, 28], lens=[25, 128], row0=[0, 20, 48])
        check(e, out)


def test_append_far_offsets():
    from decode_attention_06_b200 import gqla
    c = make(1, [37, 5], [300, 60], seed=8)
    pages = 140_000
    far = dict(c, table=torch.where(c["table"] >= 0, c["table"] + (pages - c["pages"]), c["table"]), pages=pages)
    kv = torch.zeros(1, pages * 64, 256, dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros(pages * 64, 64, dtype=torch.bfloat16, device="cuda")
    latent = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    n = c["pages"]
    kv.view(1, pages, 64, 256)[:, -n:] = c["kv"].view(1, n, 64, 256)
    rope.view(pages, 64, 64)[-n:] = c["rope"].view(n, 64, 64)
    latent[-n:] = c["latent"]
    ws = gqla.new_workspace()
    gqla.gqla_append_cache(gqla.make_dims(16, 1), c["rows"], c["starts"], gqla.make_kv_index(far["table"], c["seqlens"], pages),
                           ws, latent_cache=latent, w_uk=c["w_uk"], w_uv=c["w_uv"], kv_expanded=kv, k_rope=rope)
    torch.cuda.synchronize()
    assert gqla.gqla_read_device_error(ws)[0] == 0
    check(c, {"latent": latent[-n:], "kv": kv.view(1, pages, 64, 256)[:, -n:].reshape(1, n * 64, 256),
              "rope": rope.view(pages, 64, 64)[-n:].reshape(n * 64, 64)})
    assert not bool(kv.view(pages, -1)[:-n].any()) and not bool(latent[:-n].any())


@pytest.mark.parametrize("at,value,skip", [(1, 95, (0, 1)), (2, 10, (1, 2)), (1, -3, (0, 1))])
def test_append_does_the_sequences_beside_starts_that_descend(at, value, skip):
    c = make(2, [20, 30, 40], [5, 100, 0], seed=5)  # starts 0, 20, 50, 90
    d = dict(c, starts=c["starts"].clone())
    d["starts"][at] = value
    for what in (dict(), dict(expanded=False)):
        out, err = run(d, **what)
        assert err[0] == -5 and err[1] in skip
        check(c, out, skip=skip, **what)


@pytest.mark.parametrize("g", [16, 20, 37, 40])
@pytest.mark.parametrize("new,ctx", [([1], [200]), ([40, 3, 129], [0, 64, 61]), ([1500, 700], [10, 0])])
def test_append_of_many_groups(g, new, ctx):
    """One product to a pair as long as all fit on the SMs, several beyond; group counts that few powers
    of two divide."""
    c = make(g, new, ctx, seed=g, gap=2, h=2 * g)
    out, err = run(c)
    assert err[0] == 0
    check(c, out)
