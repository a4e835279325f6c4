"""The serving calls together, as a program runs them: pages extended, tokens appended, prompts and
chunks prefilled, sequences forked (their last pages copied), decoded through both paths, freed, the
pool compacted; checked at every step against attention in float64 over the tokens' latent rows.

Tolerances: those of the decode parity tests (max-abs 2e-2, relative Frobenius 1e-2): the caches
are bf16 and the reference starts from the latent rows, so K and V carry their own rounding.
"""
import math
import random

import pytest
import torch

from tests.helpers import compare

pytestmark = pytest.mark.gpu
H, G = 32, 8


class Server:
    def __init__(self, batch=6, width=12, pages=60, seed=0):
        from decode_attention_06_b200 import gqla
        self.gqla, self.gen, self.batch = gqla, torch.Generator(device="cuda").manual_seed(seed), batch
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lens, self.refs = z(batch, width), z(batch), z(pages)
        self.pool = gqla.make_page_pool(self.table, self.lens, self.refs)
        self.index = gqla.make_kv_index(self.table, self.lens, pages)
        nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.pages = pages
        self.latent, self.kv, self.rope = nan(pages, 64, 576), nan(G, pages * 64, 256), nan(pages * 64, 64)
        self.w = [(self.randn(G, 512, 128) / math.sqrt(512)).to(torch.bfloat16) for _ in range(2)]
        self.dims, self.ws = gqla.make_dims(H, G), gqla.new_workspace()
        self.rows = [torch.empty(0, 576, dtype=torch.bfloat16, device="cuda") for _ in range(batch)]  # what each holds

    def randn(self, *s):
        return torch.randn(*s, generator=self.gen, device="cuda")

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def append(self, new):
        """`new[b]` random tokens to every sequence: pages, then rows into both caches."""
        rows = self.randn(sum(new), 576).to(torch.bfloat16)
        starts = [0]
        for b, n in enumerate(new):
            self.rows[b] = torch.cat([self.rows[b], rows[starts[-1]:starts[-1] + n]])
            starts.append(starts[-1] + n)
        self.starts = self.i32(starts)
        self.gqla.gqla_extend_sequences(self.pool, self.i32(new), self.ws)
        self.gqla.gqla_append_cache(self.dims, rows, self.starts, self.index, self.ws, latent_cache=self.latent,
                                    w_uk=self.w[0], w_uv=self.w[1], kv_expanded=self.kv, k_rope=self.rope)

    def prefill(self, new):
        q = self.randn(sum(new), H, 192).to(torch.bfloat16)
        lens = [r.shape[0] for r in self.rows]
        bufs = self.gqla.PrefillBuffers(self.dims, sum(new), self.gqla.plan_prefill(self.dims, new, lens))
        out, lse = self.gqla.prefill_step(self.dims, bufs, q, self.starts, self.index, self.kv, self.rope)
        self.check(q, new, out)
        assert self.gqla.gqla_read_device_error(bufs.workspace)[0] == 0
        return q, out, lse

    def reference(self, q, b, n):
        """Attention of the last n tokens of sequence b over its latent rows, in float64."""
        rows, L = self.rows[b].double(), self.rows[b].shape[0]
        k = torch.einsum("tc,gcd->gtd", rows[:, :512], self.w[0].double())
        v = torch.einsum("tc,gcd->gtd", rows[:, :512], self.w[1].double())
        qd = q.double().view(n, G, H // G, 192)
        s = torch.einsum("nghd,gtd->nght", qd[..., :128], k) + torch.einsum("nghd,td->nght", qd[..., 128:], rows[:, 512:])
        seen = torch.arange(L, device="cuda") <= (L - n + torch.arange(n, device="cuda"))[:, None]
        p = (s / math.sqrt(192)).masked_fill(~seen[:, None, None, :], -math.inf).softmax(-1)
        return torch.einsum("nght,gtd->nghd", p, v).reshape(n, H, 128)

    def check(self, q, new, out):
        at = 0
        for b, n in enumerate(new):
            if n:
                compare(out[at:at + n], self.reference(q[at:at + n], b, n).cpu().numpy(), what=f"sequence {b}")
            at += n

    def decode(self):
        """One decode step through both paths for the sequences as they are; returns both outputs."""
        g, B = self.gqla, self.batch
        q = self.randn(B, 1, H, 192).to(torch.bfloat16)
        for path in ("gqa", "absorb"):
            bufs = g.DecodeBuffers(self.dims, B, 1, 5, path)
            out, _ = g.decode_step(self.dims, bufs, q, *self.w, self.index, latent_cache=self.latent,
                                   kv_expanded=self.kv, k_rope=self.rope)
            torch.cuda.synchronize()
            for b in range(B):
                if self.rows[b].shape[0]:
                    compare(out[b], self.reference(q[b], b, 1).cpu().numpy(), what=f"{path} sequence {b}")
            assert g.gqla_read_device_error(bufs.workspace)[0] == 0

    def fork(self, forks):
        pairs = self.i32([[9, 9]] * len(forks))
        self.gqla.gqla_fork_sequences(self.pool, self.i32(forks), pairs, self.ws)
        self.copy(pairs)
        for a, c in forks:
            self.rows[c] = self.rows[a]

    def copy(self, pairs):
        self.gqla.gqla_copy_pages(self.dims, pairs, self.pages, self.ws, latent_cache=self.latent,
                                  kv_expanded=self.kv, k_rope=self.rope)

    def free(self, ids):
        self.gqla.gqla_free_sequences(self.pool, self.i32(ids), self.ws)
        for b in ids:
            self.rows[b] = self.rows[b][:0]

    def compact(self):
        pairs = self.i32([[9, 9]] * (self.pages // 2))
        counts = self.i32([0, 0])
        self.gqla.gqla_compact_pages(self.pool, self.table, self.refs, pairs, counts, self.ws)
        self.copy(pairs)
        return counts.tolist()

    def error(self):
        return self.gqla.gqla_read_device_error(self.ws)


def test_a_serving_run():
    s = Server()
    prompts = [150, 33, 0, 64, 0, 1]
    s.append(prompts)
    s.prefill(prompts)
    s.decode()
    s.fork([(0, 2), (0, 4)])           # two more continuations of sequence 0
    new = [5, 1, 3, 0, 8, 2]           # drafts, verified
    s.append(new)
    s.prefill(new)
    s.decode()
    s.free([0, 3])                     # its forks keep its pages
    s.decode()
    live = s.compact()[0]
    assert live == int((s.refs > 0).sum()) and not bool((s.refs[live:] != 0).any())
    s.decode()
    chunk = [70, 0, 100, 129, 0, 64]   # chunked prefill over freed and moved pages
    s.append(chunk)
    s.prefill(chunk)
    s.decode()
    assert s.error()[0] == 0


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_random_serving_runs(seed):
    rng = random.Random(seed)
    s = Server(batch=5, width=10, pages=50, seed=seed)
    for _ in range(10):
        lens = [r.shape[0] for r in s.rows]
        what = rng.choice(["append", "append", "fork", "free", "compact"])
        if what == "append":
            new = [rng.choice([0, 1, rng.randint(1, 90)]) if x < 500 else 0 for x in lens]
            if sum(new):
                s.append(new)
                s.prefill(new)
        elif what == "fork" and 0 in lens and max(lens):
            s.fork([(lens.index(max(lens)), lens.index(0))])
        elif what == "free":
            s.free([rng.randrange(5)])
        elif what == "compact":
            s.compact()
        s.decode()
    assert s.error()[0] == 0


def test_prefill_of_one_and_two_tokens_is_the_decode_step():
    """Same cache, same queries: the chunk attention and the decode agree to their roundings."""
    from decode_attention_06_b200 import gqla
    s = Server(batch=4, width=40, pages=120)
    s.append([500, 63, 1200, 2])
    for n in (1, 2):
        q = s.randn(4, n, H, 192).to(torch.bfloat16)
        s.starts = s.i32([n * i for i in range(5)])
        bufs = gqla.PrefillBuffers(s.dims, 4 * n, gqla.plan_prefill(s.dims, [n] * 4, [500, 63, 1200, 2]))
        out, lse = gqla.prefill_step(s.dims, bufs, q.view(4 * n, H, 192), s.starts, s.index, s.kv, s.rope)
        dec = gqla.DecodeBuffers(s.dims, 4, n, 7, "gqa")
        want, want_lse = gqla.decode_step(s.dims, dec, q, None, None, s.index, kv_expanded=s.kv, k_rope=s.rope)
        torch.cuda.synchronize()
        compare(out, want.view(4 * n, H, 128).double().cpu().numpy(), what=f"{n} tokens")
        assert float((lse - want_lse.view(4 * n, H)).abs().max()) <= 1e-2


def test_append_is_the_expansion_of_the_rows():
    """The rows that append writes are those that the one-shot expansion computes from them."""
    from decode_attention_06_b200 import gqla
    s = Server(batch=3, width=12, pages=40)
    s.append([300, 65, 128])
    n = s.pages * 64
    lat = torch.nan_to_num(s.latent)
    kv, rope = torch.empty(G, n, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 64, dtype=torch.bfloat16, device="cuda")
    gqla.gqla_expand_cache_tc(s.dims, lat, *s.w, kv, rope)
    torch.cuda.synchronize()
    used = ~torch.isnan(s.rope[:, 0])
    assert torch.equal(s.rope[used], rope[used])
    a, b = s.kv[:, used].double(), kv[:, used].double()
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -14).all())


def test_a_batch_without_new_tokens():
    """No token at all: nothing is launched and nothing changes."""
    from decode_attention_06_b200 import gqla
    s = Server(batch=3)
    s.append([70, 0, 5])
    before = [x.clone() for x in (s.table, s.lens, s.refs)]
    s.append([0, 0, 0])
    bufs = gqla.PrefillBuffers(s.dims, 4, gqla.plan_prefill(s.dims, [0, 0, 0], [70, 0, 5]))
    out, lse = gqla.prefill_step(s.dims, bufs, torch.empty(0, H, 192, dtype=torch.bfloat16, device="cuda"), s.starts,
                                 s.index, s.kv, s.rope)
    torch.cuda.synchronize()
    assert out.shape == (0, H, 128) and lse.shape == (0, H) and s.error()[0] == 0
    assert all(torch.equal(a, b) for a, b in zip(before, (s.table, s.lens, s.refs)))
