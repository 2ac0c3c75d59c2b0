"""The operators around latent rows one after another, as a decode loop over a pool and its hot
rows uses them: the residual's norm, the projections, the token's latent row to the pool and to
its request's newest hot row, the swap-in of the rows a selection names, attention over them;
eagerly, and as one captured graph that is given the next step's inputs in place."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import cases
from latent_cases import GROUP, check_codes, latent_plain, make_rows, norm_error, norm_plain
from paged_cases import U32, half_step, norm_rope_plain

pytestmark = pytest.mark.gpu
EPS = 1e-6
LENS = [60, 300, 61, 500, 11]
B, K, HOT, LEN, D, HEADS, R, P = 5, 96, 160, 700, 320, 16, 512, 64


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


class Layer:
    def __init__(self, dev, seed=0):
        import sparse_attention_kv_row_gb300 as hs

        self.hs, self.dev = hs, dev
        rng = np.random.default_rng(seed)
        c = cases.random_case(rng, B=B, K=K, H=HOT, S=656, R=B, seq_len=LEN)
        # Every token of every request has a pool row of its own.
        c.pool_rows = rng.permutation(c.pool_k.shape[0]).reshape(c.pool_rows.shape)
        self.pool_rows = c.pool_rows
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        values = torch.randn(c.pool_k.shape[0], R + P, generator=g)
        self.pool = make_rows(values, "fp8", bf)[0].to(dev)
        self.hot = torch.full(c.hot_k.shape, 0xFF, dtype=torch.uint8, device=dev)  # NaN until it is filled
        self.req_host, self.slot_rows = c.req_state, c.rows
        for i, n in enumerate(LENS):  # (a request that fits has its token t in slot t)
            if n <= HOT:
                state = c.req_state[i]
                self.hot[t(c.rows[state, :n]).long()] = self.pool[t(c.pool_rows[state, :n])]
        self.req, self.pool_map = t(c.req_state), t(c.pool_rows)
        self.tokens, self.slots, self.lru = t(c.tokens), t(c.rows), t(c.lru)
        half = P // 2
        a = torch.arange(LEN, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        self.cs = torch.cat([a.cos(), a.sin()], 1).float()
        w = lambda n: (1 + 0.2 * torch.randn(n, generator=g)).to(bf)  # noqa: E731
        self.w1, self.w2 = w(D), w(R)
        self.wkv = (torch.randn(D, R + P, generator=g) * D ** -0.5).to(bf)
        self.wq = (torch.randn(D, HEADS * (R + P), generator=g) * D ** -0.5).to(bf)
        self.d = dict(cs=self.cs.to(dev), w1=self.w1.to(dev), w2=self.w2.to(dev), wkv=self.wkv.to(dev),
                      wq=self.wq.to(dev))
        z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
        i32, i64 = torch.int32, torch.int64
        self.b = dict(x=z(B, D), res=z(B, D), y=z(B, D), kv=z(B, R + P), q=z(B, HEADS, R + P), out=z(B, HEADS, R),
                      pos=z(B, dt=i64), loc=z(B, dt=i64), hot_loc=z(B, dt=i64), seq=z(B, dt=i64),
                      topk=z(B, K, dt=i32), rows=z(B, K, dt=i32), st=z(1, dt=i32), swap_st=z(B, dt=i32),
                      attn_st=z(B, dt=i32), lse=z(B, HEADS, dt=torch.float32))
        self.scale = (R + P) ** -0.5

    def load(self, step, seed=0):
        """The inputs of one step; returns what the host keeps of them."""
        g = torch.Generator().manual_seed(1000 * seed + step)
        rng = np.random.default_rng(1000 * seed + step)
        seq = np.array(LENS) + step
        topk = np.full((B, K), -1, np.int32)
        for i in range(B):
            n = min(K, int(seq[i]))
            topk[i, :n] = rng.permutation(int(seq[i]))[:n]
            topk[i, rng.integers(0, n)] = seq[i] - 1  # the newest token is among them
            _, first = np.unique(topk[i], return_index=True)
            twice = np.setdiff1d(np.arange(K), first)
            topk[i, twice] = -1
        loc = self.pool_rows[self.req_host, seq - 1]
        hot_loc = self.slot_rows[self.req_host, np.where(seq <= HOT, seq - 1, HOT)]
        x, res = (torch.randn(B, D, generator=g).to(torch.bfloat16) for _ in range(2))
        for name, v in (("x", x), ("res", res), ("pos", torch.from_numpy(seq - 1)), ("loc", torch.from_numpy(loc)),
                        ("hot_loc", torch.from_numpy(hot_loc.astype(np.int64))),
                        ("seq", torch.from_numpy(seq)), ("topk", torch.from_numpy(topk))):
            self.b[name].copy_(v)
        return dict(x=x, res=res, seq=seq, topk=topk, loc=loc)

    def step(self):
        hs, b, d = self.hs, self.b, self.d
        hs.add_rms_norm(b["x"], d["w1"], b["y"], residual=b["res"], eps=EPS)
        torch.mm(b["y"], d["wkv"], out=b["kv"])
        torch.mm(b["y"], d["wq"], out=b["q"].view(B, -1))
        self.turned = b["q"][..., R:]
        for rows, loc, q in ((self.pool, "loc", None), (self.hot, "hot_loc", self.turned)):
            hs.latent_norm_rope_store(b["kv"][:, :R], b["kv"][:, R:], d["w2"], d["cs"], b["pos"], rows, b[loc],
                                      q_pe=q, q_out=q, eps=EPS, status=b["st"])
        hs.swap_in(topk_ids=b["topk"], seq_lens=b["seq"], req_state=self.req, slot_tokens=self.tokens,
                   slot_rows=self.slots, lru=self.lru, pool_rows=self.pool_map, pool_k=self.pool,
                   hot_k=self.hot, out_rows=b["rows"], hot_size=HOT, status=b["swap_st"])
        hs.latent_attention(b["q"], self.hot, b["rows"], b["out"], scale=self.scale, lse=b["lse"],
                            status=b["attn_st"])

    def check(self, host):
        torch.cuda.synchronize()
        b = {k: v.cpu() for k, v in self.b.items()}
        assert not any(bool(b[k].any()) for k in ("st", "swap_st", "attn_st"))
        total = (host["x"] + host["res"])
        assert torch.equal(b["res"], total)
        want = norm_plain(total, self.w1, EPS)
        assert bool(((b["y"].double() - want).abs() <= 1.01 * (norm_error(D) + half_step(torch.bfloat16)) * want.abs()).all())
        # the token's row, in the pool and in the newest hot row
        row = self.pool.cpu()[torch.from_numpy(host["loc"])]
        assert torch.equal(row, self.hot.cpu()[b["hot_loc"]])
        codes, scales = row[:, :R], row[:, R:R + 16].contiguous().view(torch.float32)
        check_codes(norm_plain(b["kv"][:, :R], self.w2, EPS), norm_error(R), codes, scales, GROUP, False)
        turn = self.cs[b["pos"]]
        z, both = norm_rope_plain(b["kv"][:, None, R:], None, turn, EPS, False)
        got = row[:, R + 16:].contiguous().view(torch.bfloat16).double()
        assert bool(((got - z[:, 0]).abs() <= 1.01 * (4 * U32 * both[:, 0] + half_step(torch.bfloat16) * z[:, 0].abs())).all())
        # attention over what the selection names, in the pool
        pool = self.pool.cpu()
        held = torch.cat([(pool[:, :R].view(torch.float8_e4m3fn).double().unflatten(1, (-1, GROUP))
                           * pool[:, R:R + 16].contiguous().view(torch.float32).double()[..., None]).flatten(1),
                          pool[:, R + 16:].contiguous().view(torch.bfloat16).double()], 1)
        lists = [[int(self.pool_rows[self.req_host[i], t]) for t in host["topk"][i] if t >= 0] for i in range(B)]
        out, lse, size, unit, n, wide = latent_plain(b["q"], held, lists, R, self.scale)
        h16 = half_step(torch.float16)
        es = ((R + P + 8) * U32 + h16) * unit + 2.0 ** -33 * wide
        rel = 2 * es + (2 * n[:, None] + 16) * U32 + 2 * h16 + 4 * U32
        small = 2.0 ** -29 * float(held[:, :R].abs().max())
        tol = 1.01 * (rel[..., None] * size + half_step(torch.bfloat16) * out.abs() + small * n[:, None, None])
        assert bool(((b["out"].double() - out).abs() <= tol).all())
        assert bool(((b["lse"].double() - lse).abs() <= 1.01 * (es + (n[:, None] + 16) * U32 + 4 * U32 * lse.abs())).all())


def test_decode_steps(dev):
    layer = Layer(dev)
    for step in range(4):
        host = layer.load(step)
        layer.step()
        layer.check(host)


def test_captured_decode_steps(dev):
    """Replays of one captured step against an eager twin: the same state and the same bits."""
    eager, graphed = Layer(dev, 1), Layer(dev, 1)
    for layer in (eager, graphed):
        layer.load(0)
        layer.step()  # (sets up what is set up once)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for step in range(1, 5):
        host = eager.load(step)
        eager.step()
        eager.check(host)
        graphed.load(step)
        graph.replay()
        torch.cuda.synchronize()
        for name, v in eager.b.items():
            assert torch.equal(v, graphed.b[name]), name
        for name in ("pool", "tokens", "lru", "hot"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), name
